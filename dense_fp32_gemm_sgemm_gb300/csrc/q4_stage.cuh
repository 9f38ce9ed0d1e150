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
};

// Writes the pieces of the rows to their columns, and their sums (zeros for the centred form);
// true where the plain form cannot take one of the thread's values. A group's octets lie in
// neighbouring lanes of a warp, so that shuffles add them.
template <class T>
__device__ __noinline__ bool stage_rows(const Staging s, bool plain) {
    constexpr int P = pieces_of_type<T>();
    constexpr int AHEAD = 4;  // loads in flight
    constexpr int COLS = P == 3 ? 4 : P;  // of a row
    const T* A = static_cast<const T*>(s.A);
    const int items = s.octets * s.rows;
    const int group_mask = (1 << s.log_octets) - 1;
    int row = 0, u = threadIdx.x;
    Magnitudes magnitudes;
    for (int i = threadIdx.x; i - int(threadIdx.x & 31) < items; i += AHEAD * s.threads) {
        Raw8<T> raw[AHEAD];
        int rows[AHEAD], octets[AHEAD];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            rows[j] = -1;
            if (i + j * s.threads < items) {
                while (u >= s.octets) {
                    u -= s.octets;
                    ++row;
                }
                rows[j] = row;
                octets[j] = u;
                raw[j] = load_raw8(A + row * s.lda, s.n0 + u * 8, s.N, s.vec);
                u += s.threads;
            }
        }
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            float sum[P];
#pragma unroll
            for (int p = 0; p < P; ++p) sum[p] = 0.0f;
            if (rows[j] >= 0) {
                uint4 piece[P];
                if (plain)
                    split_plain<P>(raw[j], magnitudes, piece, sum);
                else
                    split_centred<P>(raw[j], piece);
#pragma unroll
                for (int p = 0; p < P; ++p)
                    *reinterpret_cast<uint4*>(s.xs + octets[j] * s.octet_stride +
                                              (rows[j] * COLS + p) * s.column_stride) =
                        piece[p];
            }
            if (i - int(threadIdx.x & 31) + j * s.threads >= items) continue;  // warp-uniform
#pragma unroll
            for (int p = 0; p < P; ++p) {
                for (int o = 1; o <= group_mask; o *= 2)
                    sum[p] += __shfl_xor_sync(0xffffffffu, sum[p], o);
                if (rows[j] >= 0 && (octets[j] & group_mask) == 0)
                    s.xsum[(octets[j] >> s.log_octets) * s.sum_pitch + rows[j] * COLS + p] =
                        sum[p] * s.factor;
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
