// Into and out of the packed 4-bit format: quantisation of a dense matrix, layout of codes
// that are quantised already, and dequantisation to FP32 (definitions in sgemm.h, layout in
// q4.cuh).
//
// All three move a tile of 128 n x 64 columns (half a unit) through shared memory, because a
// column's codes run along n while a dense matrix is contiguous along k (or, transposed, the
// other way round): global memory is read and written in whole lines on both sides.
#include "internal.cuh"
#include "q4.cuh"

namespace sgemm {
namespace {

constexpr int TILE_K = 64;
constexpr int PITCH = TILE_K + 1;  // column and row walks of the tile are free of conflicts
constexpr int THREADS = 256;

enum class Source { values, codes };

// The nibble of a word that holds the e-th of its 8 codes.
__device__ constexpr int nibble_of(int e) { return (e >> 1) + 4 * (e & 1); }

// The unit that a CTA works on, and its first column there.
__device__ __forceinline__ uint8_t* unit_at(uint8_t* data, const Q4Geom& geom) {
    return data + size_t(blockIdx.z) * geom.matrix_bytes() +
           (blockIdx.x / (kQ4UnitK / TILE_K)) * geom.tile_bytes() +
           size_t(blockIdx.y) * geom.unit_bytes;
}
__device__ __forceinline__ int first_column() {
    return int(blockIdx.x) % (kQ4UnitK / TILE_K) * TILE_K;
}

template <Source SOURCE>
__global__ void __launch_bounds__(THREADS)
    q4_pack_kernel(const void* __restrict__ src, int dtype, bool transposed,
                   const uint16_t* __restrict__ scales, const uint8_t* __restrict__ zeros,
                   uint8_t* __restrict__ out, Q4Geom geom) {
    __shared__ float tile[kQ4UnitN][PITCH];
    __shared__ float lo_s[4][TILE_K], hi_s[4][TILE_K];  // of 32 n each
    __shared__ float scale_s[4][TILE_K];                // of a group each
    __shared__ float zero_s[4][TILE_K];
    const int tid = threadIdx.x;
    const int n0 = blockIdx.y * kQ4UnitN, k0 = blockIdx.x * TILE_K;
    const int N = geom.N, K = geom.K;
    const size_t mat = size_t(blockIdx.z) * N * K;
    const int blocks = geom.group / 32, groups = kQ4UnitN / geom.group;

#pragma unroll 8
    for (int i = 0; i < kQ4UnitN * TILE_K / THREADS; ++i) {
        const int n = transposed ? tid % kQ4UnitN : tid / TILE_K + i * (THREADS / TILE_K);
        const int k = transposed ? tid / kQ4UnitN + i * (THREADS / kQ4UnitN) : tid % TILE_K;
        float v = 0.0f;
        if (n0 + n < N && k0 + k < K) {
            const size_t at =
                mat + (transposed ? size_t(k0 + k) * N + n0 + n : size_t(n0 + n) * K + k0 + k);
            if constexpr (SOURCE == Source::values)
                v = load_as_float(src, dtype, at);
            else
                v = float(static_cast<const uint8_t*>(src)[at] & 15);
        }
        tile[n][k] = v;
    }
    __syncthreads();

    const int k = tid % TILE_K, part = tid / TILE_K;
    if constexpr (SOURCE == Source::values) {
        float lo = 0.0f, hi = 0.0f;
#pragma unroll 8
        for (int i = 0; i < 32; ++i) {
            const float v = tile[part * 32 + i][k];
            lo = fminf(lo, v);
            hi = fmaxf(hi, v);
        }
        lo_s[part][k] = lo;
        hi_s[part][k] = hi;
        __syncthreads();
    }
    if (part < groups) {
        float s = 0.0f, z = geom.zeros ? 0.0f : 8.0f;
        if constexpr (SOURCE == Source::values) {
            float lo = 0.0f, hi = 0.0f;
            for (int b = part * blocks; b < (part + 1) * blocks; ++b) {
                lo = fminf(lo, lo_s[b][k]);
                hi = fmaxf(hi, hi_s[b][k]);
            }
            s = geom.zeros ? __fsub_rn(__fdiv_rn(hi, 15.0f), __fdiv_rn(lo, 15.0f))
                           : __fdiv_rn(fmaxf(hi, -lo), 7.0f);
            s = __bfloat162float(__float2bfloat16_rn(s));
            if (geom.zeros && s > 0.0f)
                z = fminf(fmaxf(rintf(__fdiv_rn(-lo, s)), 0.0f), 15.0f);
            scale_s[part][k] = s;
            zero_s[part][k] = z;
        }
        const int group = (n0 + part * geom.group) / geom.group;
        const int all_groups = (N + geom.group - 1) / geom.group;
        uint16_t bits = 0;
        if constexpr (SOURCE == Source::values) {
            bits = uint16_t(__float_as_uint(s) >> 16);
        } else {
            if (group < all_groups && k0 + k < K) {
                const size_t at = size_t(blockIdx.z) * all_groups * K +
                                  (transposed ? size_t(k0 + k) * all_groups + group
                                              : size_t(group) * K + k0 + k);
                bits = scales[at];
                if (geom.zeros) z = fminf(float(zeros[at]), 15.0f);
            }
            zero_s[part][k] = z;
        }
        uint8_t* unit = unit_at(out, geom);
        const int at = part * kQ4UnitK + first_column() + k;
        reinterpret_cast<uint16_t*>(unit + kQ4CodeBytes)[at] = bits;
        if (geom.zeros) unit[kQ4CodeBytes + groups * kQ4UnitK * 2 + at] = uint8_t(z);
    }
    __syncthreads();

    // 16 bytes of codes a thread: part is the block of 32 n
    auto code = [&](int n, int kk) -> uint32_t {
        const int g = n / geom.group;
        const float z = zero_s[g][kk];
        if (n0 + n >= N || k0 + kk >= K) return uint32_t(z);
        if constexpr (SOURCE == Source::codes) return uint32_t(tile[n][kk]);
        const float s = scale_s[g][kk];
        const float low = geom.zeros ? 0.0f : -8.0f, high = geom.zeros ? 15.0f : 7.0f;
        if (!(s > 0.0f)) return uint32_t(z);
        float q = rintf(__fdiv_rn(tile[n][kk], s));
        if (geom.zeros) q += z;
        q = fminf(fmaxf(q, low), high);
        return uint32_t(int(geom.zeros ? q : q + 8.0f));
    };
    uint32_t word[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t w = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) w |= code(part * 32 + 8 * i + e, k) << (4 * nibble_of(e));
        word[i] = w;
    }
    reinterpret_cast<uint4*>(unit_at(out, geom))[part * kQ4UnitK + first_column() + k] =
        make_uint4(word[0], word[1], word[2], word[3]);
}

__global__ void __launch_bounds__(THREADS)
    q4_dequantize_kernel(const uint8_t* __restrict__ data, float* __restrict__ B, Q4Geom geom) {
    __shared__ float tile[kQ4UnitN][PITCH];
    const int tid = threadIdx.x;
    const int n0 = blockIdx.y * kQ4UnitN, k0 = blockIdx.x * TILE_K;
    const int N = geom.N, K = geom.K;
    const int k = tid % TILE_K, part = tid / TILE_K;
    {
        const uint8_t* unit = unit_at(const_cast<uint8_t*>(data), geom);
        const int col = first_column() + k, g = part * 32 / geom.group;
        const int groups = kQ4UnitN / geom.group;
        const uint4 w4 = __ldcs(reinterpret_cast<const uint4*>(unit) + part * kQ4UnitK + col);
        const uint32_t word[4] = {w4.x, w4.y, w4.z, w4.w};
        const float s = q4_scale(
            reinterpret_cast<const uint16_t*>(unit + kQ4CodeBytes)[g * kQ4UnitK + col], geom.fp16);
        const int z =
            geom.zeros ? unit[kQ4CodeBytes + groups * kQ4UnitK * 2 + g * kQ4UnitK + col] : 8;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                tile[part * 32 + 8 * i + e][k] =
                    s * float(int((word[i] >> (4 * nibble_of(e))) & 15) - z);
    }
    __syncthreads();
    float* out = B + size_t(blockIdx.z) * N * K;
    if (k0 + k >= K) return;
#pragma unroll 8
    for (int i = 0; i < kQ4UnitN * TILE_K / THREADS; ++i) {
        const int n = tid / TILE_K + i * (THREADS / TILE_K);
        if (n0 + n < N) __stcs(out + size_t(n0 + n) * K + k0 + k, tile[n][k]);
    }
}

dim3 tile_grid(const Q4Geom& g, int count) {
    return dim3(g.tiles * (kQ4UnitK / TILE_K), g.units, count);
}

// Checks shared by the three entry points; SGEMM_OK or an error.
int check_packed(const sgemm_q4* w, const void* dense) {
    if (!q4_valid(w) || !w->data || !dense) return SGEMM_ERR_ARG;
    if (!aligned16(w->data)) return SGEMM_ERR_ARG;
    return SGEMM_OK;
}

}  // namespace
}  // namespace sgemm

using namespace sgemm;

extern "C" {

long long sgemm_q4_bytes(const sgemm_q4* w) {
    if (!q4_valid(w)) return SGEMM_ERR_ARG;
    return static_cast<long long>(q4_bytes(*w));
}

int sgemm_q4_quantize(const void* B, int dtype, int transposed, const sgemm_q4* w, void* stream) {
    const int rc = check_packed(w, B);
    if (rc != SGEMM_OK) return rc;
    if (!dtype_valid(dtype)) return SGEMM_ERR_ARG;
    if (w->flags & SGEMM_Q4_SCALE_FP16) return SGEMM_ERR_UNSUPPORTED;
    const size_t dense = size_t(w->count) * w->N * w->K * dtype_bytes(dtype);
    if (ranges_overlap(w->data, q4_bytes(*w), B, dense)) return SGEMM_ERR_OVERLAP;
    if (!aligned_to(B, dtype_bytes(dtype))) return SGEMM_ERR_ARG;
    if (!current_device(nullptr)) return SGEMM_ERR_NO_DEVICE;
    const Q4Geom g = q4_geom(*w);
    q4_pack_kernel<Source::values>
        <<<tile_grid(g, w->count), THREADS, 0, static_cast<cudaStream_t>(stream)>>>(
            B, dtype, transposed != 0, nullptr, nullptr, static_cast<uint8_t*>(w->data), g);
    count_launch();
    return cudaGetLastError() == cudaSuccess ? SGEMM_OK : SGEMM_ERR_CUDA;
}

int sgemm_q4_pack(const unsigned char* codes, const void* scales, const unsigned char* zeros,
                  int transposed, const sgemm_q4* w, void* stream) {
    const int rc = check_packed(w, codes);
    if (rc != SGEMM_OK) return rc;
    if (!scales || ((w->flags & SGEMM_Q4_ZEROS) && !zeros)) return SGEMM_ERR_ARG;
    const Q4Geom g = q4_geom(*w);
    const size_t bytes = q4_bytes(*w), dense = size_t(w->count) * w->N * w->K;
    const size_t side = size_t(w->count) * ((w->N + w->group - 1) / w->group) * w->K;
    if (ranges_overlap(w->data, bytes, codes, dense) ||
        ranges_overlap(w->data, bytes, scales, 2 * side) ||
        ((w->flags & SGEMM_Q4_ZEROS) && ranges_overlap(w->data, bytes, zeros, side)))
        return SGEMM_ERR_OVERLAP;
    if (!aligned_to(scales, 2)) return SGEMM_ERR_ARG;
    if (!current_device(nullptr)) return SGEMM_ERR_NO_DEVICE;
    q4_pack_kernel<Source::codes>
        <<<tile_grid(g, w->count), THREADS, 0, static_cast<cudaStream_t>(stream)>>>(
            codes, 0, transposed != 0, static_cast<const uint16_t*>(scales), zeros,
            static_cast<uint8_t*>(w->data), g);
    count_launch();
    return cudaGetLastError() == cudaSuccess ? SGEMM_OK : SGEMM_ERR_CUDA;
}

int sgemm_q4_dequantize(const sgemm_q4* w, float* B, void* stream) {
    const int rc = check_packed(w, B);
    if (rc != SGEMM_OK) return rc;
    const size_t dense = size_t(w->count) * w->N * w->K * sizeof(float);
    if (ranges_overlap(B, dense, w->data, q4_bytes(*w))) return SGEMM_ERR_OVERLAP;
    if (!aligned_to(B, sizeof(float))) return SGEMM_ERR_ARG;
    if (!current_device(nullptr)) return SGEMM_ERR_NO_DEVICE;
    const Q4Geom g = q4_geom(*w);
    q4_dequantize_kernel<<<tile_grid(g, w->count), THREADS, 0, static_cast<cudaStream_t>(stream)>>>(
        static_cast<const uint8_t*>(w->data), B, g);
    count_launch();
    return cudaGetLastError() == cudaSuccess ? SGEMM_OK : SGEMM_ERR_CUDA;
}

}  // extern "C"
