// The few-row product's operands, and how both of its kernels stage the columns of A^T: the
// bfloat16 pieces of the rows of A, scaled for the plain form of the weights (q4.cuh), with
// their sums over each group of n.
#pragma once
#include "internal.cuh"
#include "q4.cuh"

namespace sgemm {

// C = A . B. "Columns" are the pieces of A's rows, an unused one after three.
struct Q4Product {
    const void* A;
    size_t lda;
    int M, dtype;
    int row_columns;  // of a row of A: 1, 2 or 4
    const uint8_t* data;
    Q4Geom geom;
    void* C;
    size_t ldc;
    bool vec;  // rows of A start on 16-byte boundaries
    int* err;
};

// Few columns: warp-level matrix instructions (q4_warp.cu). More: tcgen05 (q4_tensor.cu).
// cudaErrorInvalidConfiguration where so many columns of this N do not fit.
cudaError_t launch_q4_warp(const Q4Product& p, int sm_count, cudaStream_t stream);
cudaError_t launch_q4_tensor(const Q4Product& p, int most_columns, int sm_count, cudaStream_t stream);

namespace {

// What a CTA stages of the columns: rows of A, n from n0 on, `octets` of 8 values (a multiple
// of 16), and factor times their sums over each group of 8 << log_octets values.
struct Staging {
    const void* A;
    size_t lda;
    int dtype, rows, n0, N, octets, threads;
    bool vec;
    uint8_t* xs;  // 16 bytes for each octet and column, so many bytes from one to the next:
    int octet_stride, column_stride;
    float* xsum;  // [group][column], sum_pitch floats a group
    int sum_pitch, log_octets;
    float factor;
    int turn, turns;  // this CTA's number among those that stage the same rows
};

// Writes the pieces of the rows to their columns, and their sums (for the centred form, what their
// products are to be multiplied with); true where the plain form cannot take one of the thread's values. A group's octets lie in
// neighbouring lanes of a warp, so that shuffles add them.
template <class T>
__device__ __noinline__ bool stage_rows(const Staging s, bool plain) {
    constexpr int P = pieces_of_type<T>();
    constexpr int AHEAD = 4;  // loads in flight
    constexpr int COLS = P == 3 ? 4 : P;  // of a row
    const T* A = static_cast<const T*>(s.A);
    // Warps take 32 octets at a time, of all rows in order, and each CTA starts elsewhere: lines that
    // all of them want at once, and that L2 does not hold, come some three times as slowly.
    const int items = s.octets * s.rows, lane = threadIdx.x & 31, warps = s.threads / 32;
    const int bundles = (items + 31) / 32;
    const int start = int(uint64_t(uint32_t(bundles)) * s.turn / s.turns);
    const uint32_t reciprocal = 0xffffffffu / uint32_t(max(s.octets, 1)) + 1;  // items * octets < 2^32
    const int group_mask = (1 << s.log_octets) - 1;
    Magnitudes magnitudes;
    for (int i = threadIdx.x / 32; i < bundles; i += AHEAD * warps) {
        Raw8<T> raw[AHEAD];
        int rows[AHEAD], octets[AHEAD];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            rows[j] = -1;
            int bundle = i + j * warps + start;
            if (bundle >= bundles) bundle -= bundles;
            const int item = bundle * 32 + lane;
            if (i + j * warps < bundles && item < items) {
                const int row = int(__umulhi(uint32_t(item), reciprocal));
                rows[j] = row;
                octets[j] = item - row * s.octets;
                raw[j] = load_raw8(A + row * s.lda, s.n0 + octets[j] * 8, s.N, s.vec);
            }
        }
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            float sum[P];
#pragma unroll
            for (int p = 0; p < P; ++p) sum[p] = 0.0f;
            float back = 1.0f, down = 1.0f;
            if (!plain && i + j * warps < bundles) {
                uint32_t most = rows[j] >= 0 ? largest_bits(raw[j]) : 0;
                for (int o = 1; o <= group_mask; o *= 2)
                    most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
                const CentredScale scale(most);
                back = scale.back;
                down = scale.down;
            }
            if (rows[j] >= 0) {
                uint4 piece[P];
                if (plain)
                    split_plain<P>(raw[j], magnitudes, piece, sum);
                else
                    split_centred<P>(raw[j], down, piece);
#pragma unroll
                for (int p = 0; p < P; ++p)
                    *reinterpret_cast<uint4*>(s.xs + octets[j] * s.octet_stride +
                                              (rows[j] * COLS + p) * s.column_stride) =
                        piece[p];
            }
            if (i + j * warps >= bundles) continue;  // the same in the whole warp
#pragma unroll
            for (int p = 0; p < P; ++p) {
                for (int o = 1; o <= group_mask; o *= 2)
                    sum[p] += __shfl_xor_sync(0xffffffffu, sum[p], o);
                if (rows[j] >= 0 && (octets[j] & group_mask) == 0)
                    s.xsum[(octets[j] >> s.log_octets) * s.sum_pitch + rows[j] * COLS + p] =
                        plain ? sum[p] * s.factor : back;
            }
        }
    }
    return magnitudes.special<T>();
}

__device__ __forceinline__ bool stage_any(const Staging s, bool plain) {
    if (s.dtype == SGEMM_BFLOAT16) return stage_rows<__nv_bfloat16>(s, plain);
    if (s.dtype == SGEMM_FLOAT16) return stage_rows<__half>(s, plain);
    return stage_rows<float>(s, plain);
}

// Stages the columns for the plain form; true where that form cannot take one of the values,
// and then they are staged for the centred one. All threads of the CTA.
__device__ __noinline__ bool stage_columns(const Staging s) {
    const bool special = __syncthreads_or(stage_any(s, true));
    if (special) stage_any(s, false);
    ptx::fence_proxy_async_smem();  // tcgen05 reads them through the async proxy
    __syncthreads();
    return special;
}

}  // namespace
}  // namespace sgemm
