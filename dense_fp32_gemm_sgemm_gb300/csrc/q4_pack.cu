// Into and out of the packed 4-bit format: quantisation of a dense matrix, layout of codes
// that are quantised already, and dequantisation to FP32 (definitions in sgemm.h, layout in
// q4.cuh).
//
// All three have to read the dense matrix once and write the packed one, or the reverse. A thread of
// the quantisation owns 32 n of a column, in registers, which is what 16 bytes of codes hold; a
// warp's loads run along the matrix' rows. Groups of 64 and 128 n meet in shared memory for their
// extremes only. From a transposed matrix, a lane reads its column's n itself, in whole aligned
// 16 bytes whatever the row's alignment. Two columns a thread measured 71 us where one takes 62
// (fewer warps to hide the loads). Dequantisation holds 32 n of four columns a thread and writes rows.
//
// Measured at 8192 x 8192, group 128: quantisation 62 us from float32 (4.9 TB/s) and 56 from bfloat16,
// which is bound by some 20 instructions an element; dequantisation 48 us (6.2 TB/s, 93 % of a copy).
#include "internal.cuh"
#include "q4.cuh"

namespace sgemm {
namespace {

constexpr int TILE_K = 64;
constexpr int PITCH = TILE_K + 1;  // column and row walks of the tile are free of conflicts
constexpr int THREADS = 256;

// Quantisation: 32 n of a column a thread, 32 columns a CTA
constexpr int Q_WIDTH = 32, Q_THREADS = 128, Q_CTAS = 7;

// The nibble of a word that holds the e-th of its 8 codes.
__device__ constexpr int nibble_of(int e) { return (e >> 1) + 4 * (e & 1); }

// The unit that a CTA of the layout kernel works on, and its first column there.
__device__ __forceinline__ uint8_t* unit_at(uint8_t* data, const Q4Geom& geom) {
    return data + size_t(blockIdx.z) * geom.matrix_bytes() +
           (blockIdx.x / (kQ4UnitK / TILE_K)) * geom.tile_bytes() +
           size_t(blockIdx.y) * geom.unit_bytes;
}
__device__ __forceinline__ int first_column() {
    return int(blockIdx.x) % (kQ4UnitK / TILE_K) * TILE_K;
}

// A tile of 128 n x 64 columns (half a unit) through shared memory: global memory is read and
// written in whole lines on both sides.
__global__ void __launch_bounds__(THREADS)
    q4_pack_kernel(const uint8_t* __restrict__ src, bool transposed,
                   const uint16_t* __restrict__ scales, const uint8_t* __restrict__ zeros,
                   uint8_t* __restrict__ out, Q4Geom geom) {
    __shared__ uint8_t tile[kQ4UnitN][PITCH];
    __shared__ uint8_t zero_s[4][TILE_K];  // of a group each
    const int tid = threadIdx.x;
    const int n0 = blockIdx.y * kQ4UnitN, k0 = blockIdx.x * TILE_K;
    const int N = geom.N, K = geom.K;
    const size_t mat = size_t(blockIdx.z) * N * K;
    const int groups = kQ4UnitN / geom.group;

#pragma unroll 8
    for (int i = 0; i < kQ4UnitN * TILE_K / THREADS; ++i) {
        const int n = transposed ? tid % kQ4UnitN : tid / TILE_K + i * (THREADS / TILE_K);
        const int k = transposed ? tid / kQ4UnitN + i * (THREADS / kQ4UnitN) : tid % TILE_K;
        uint8_t v = 0;
        if (n0 + n < N && k0 + k < K)
            v = src[mat + (transposed ? size_t(k0 + k) * N + n0 + n : size_t(n0 + n) * K + k0 + k)];
        tile[n][k] = v & 15;
    }
    const int k = tid % TILE_K, part = tid / TILE_K;
    if (part < groups) {
        const int group = n0 / geom.group + part;
        const int all_groups = (N + geom.group - 1) / geom.group;
        uint16_t bits = 0;
        uint8_t z = geom.zeros ? 0 : 8;
        if (group < all_groups && k0 + k < K) {
            const size_t at = size_t(blockIdx.z) * all_groups * K +
                              (transposed ? size_t(k0 + k) * all_groups + group
                                          : size_t(group) * K + k0 + k);
            bits = scales[at];
            if (geom.zeros) z = zeros[at] < 15 ? zeros[at] : 15;
        }
        zero_s[part][k] = z;
        uint8_t* unit = unit_at(out, geom);
        const int at = part * kQ4UnitK + first_column() + k;
        reinterpret_cast<uint16_t*>(unit + kQ4CodeBytes)[at] = bits;
        if (geom.zeros) unit[kQ4CodeBytes + groups * kQ4UnitK * 2 + at] = z;
    }
    __syncthreads();

    // 16 bytes of codes a thread: part is the block of 32 n
    const uint32_t z = zero_s[part * 32 / geom.group][k];
    uint32_t word[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t w = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int n = part * 32 + 8 * i + e;
            const uint32_t code = n0 + n < N && k0 + k < K ? tile[n][k] : z;
            w |= code << (4 * nibble_of(e));
        }
        word[i] = w;
    }
    reinterpret_cast<uint4*>(unit_at(out, geom))[part * kQ4UnitK + first_column() + k] =
        make_uint4(word[0], word[1], word[2], word[3]);
}

// The code of v by the definition, as it is written down. z: 8 without zero points.
__device__ __forceinline__ uint32_t code_of(float v, float s, float z, bool zeros) {
    if (!(s > 0.0f)) return uint32_t(z);
    float q = rintf(__fdiv_rn(v, s));
    if (zeros) q += z;
    q = fminf(fmaxf(q, zeros ? 0.0f : -8.0f), zeros ? 15.0f : 7.0f);
    return uint32_t(int(zeros ? q : q + 8.0f));
}
__device__ __noinline__ uint32_t word_of(const float* v, float s, float z, bool zeros) {
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) w |= code_of(v[e], s, z, zeros) << (4 * nibble_of(e));
    return w;
}

// 8 codes of a word. The definition divides and rounds to nearest, ties to even. v times the
// rounded reciprocal is within 15.1 * 2^-23 of the quotient; rounding it to a grid of 2^-14 first
// (by adding 768) puts ties, which quotients of short numbers often are, back where they belong,
// and a quotient that this moves across a tie leaves a remainder of more than s / 2. The remainder
// v - s q is exact (8 by 5 bits, and no larger than v), so where it is no more than s / 2, q is
// the definition's: the rounded quotient is a tie only if the quotient is, since neighbours of
// s (q + 1/2) in 24 bits are further off than half a place of the quotient. Else, for NaN, and
// for scales far from one, the word is made by the definition.
template <bool ZEROS>
__device__ __forceinline__ uint32_t quick_word(const float (&v)[8], float s, float r, float z) {
    constexpr float GRID = 768.0f, ROUND = 12582912.0f;  // 1.5 * 2^9, 1.5 * 2^23
    constexpr uint32_t BITS = 0x4b400000u;               // ROUND's
    float most = 0.0f;  // of the remainders; NaN if one is
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float u = __fadd_rn(__fmaf_rn(v[e], r, GRID), ROUND - GRID);
        const float rest = __fmaf_rn(-s, __fsub_rn(u, ROUND), v[e]);
        asm("max.NaN.f32 %0, %0, %1;" : "+f"(most) : "f"(fabsf(rest)));
        uint32_t code = __float_as_uint(u);
        if (ZEROS) code = uint32_t(min(max(int(code - BITS) + int(z), 0), 15));
        w += code << (4 * nibble_of(e));
    }
    // without zero points no quotient passes 7 * (1 + 2^-8), so none is clipped
    if (!ZEROS) w += (8u - BITS) * 0x11111111u;
    return s >= 0x1p-100f && s <= 0x1p100f && most <= 0.5f * s ? w : word_of(v, s, z, ZEROS);
}

template <class T>
__device__ __forceinline__ float as_float(T v) { return float(v); }

// v[i] = row[n0 + i], zeros from N on. Aligned 16-byte loads cover the 32 values, and are shifted
// into place; those that reach beyond [begin, end) of the matrix are read value by value.
template <class T>
__device__ __forceinline__ void load_along(const T* row, int n0, int N, const char* begin,
                                           const char* end, float (&v)[32]) {
    constexpr int CHUNKS = 32 * int(sizeof(T)) / 16 + 1;
    const char* from = reinterpret_cast<const char*>(row + n0);
    const int shift = int(reinterpret_cast<uintptr_t>(from) & 15);
    const char* at = from - shift;
    const char* stop = reinterpret_cast<const char*>(row + N);  // nothing after is wanted
    if (n0 + 32 > N || at < begin || at + CHUNKS * 16 > end) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = n0 + i < N ? as_float(row[n0 + i]) : 0.0f;
        return;
    }
    uint32_t w[CHUNKS * 4];
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
        uint4 c = make_uint4(0, 0, 0, 0);
        if (at + i * 16 < stop) c = *reinterpret_cast<const uint4*>(at + i * 16);
        w[4 * i] = c.x;
        w[4 * i + 1] = c.y;
        w[4 * i + 2] = c.z;
        w[4 * i + 3] = c.w;
    }
    constexpr int WORDS = 32 * int(sizeof(T)) / 4;
#pragma unroll
    for (int i = 0; i < WORDS + 2; ++i) w[i] = (shift & 8) ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < WORDS + 1; ++i) w[i] = (shift & 4) ? w[i + 1] : w[i];
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(w[i]);
    } else {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) {
            const uint32_t pair = __funnelshift_r(w[i], w[i + 1], (shift & 2) * 8);
            const T* half = reinterpret_cast<const T*>(&pair);
            v[2 * i] = as_float(half[0]);
            v[2 * i + 1] = as_float(half[1]);
        }
    }
}

template <class T, bool TRANSPOSED, bool ZEROS>
__global__ void __launch_bounds__(Q_THREADS, Q_CTAS)
    q4_quantize_kernel(const T* __restrict__ src, size_t values, uint8_t* __restrict__ out,
                       Q4Geom geom) {
    __shared__ float lo_s[4][Q_WIDTH], hi_s[4][Q_WIDTH];  // of 32 n each
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int block = warp;  // of 32 n
    const int n0 = blockIdx.y * kQ4UnitN + block * 32, k0 = blockIdx.x * Q_WIDTH;
    const int N = geom.N, K = geom.K;
    const T* mat = src + size_t(blockIdx.z) * N * K;

    const int k = k0 + lane;
    float v[32];
    if constexpr (TRANSPOSED) {
        const char* begin = reinterpret_cast<const char*>(src);
        load_along(mat + size_t(k) * N, n0, k < K ? N : 0, begin, begin + values * sizeof(T), v);
    } else if (n0 + 32 <= N && k0 + Q_WIDTH <= K) {
        // the CTA's corner and a 32-bit offset: one addition a load
        const T* corner = mat + size_t(blockIdx.y) * kQ4UnitN * K + k0;
        const uint32_t at = uint32_t(block * 32) * K + lane;
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = as_float(__ldcs(corner + (at + uint32_t(i) * K)));
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            v[i] = n0 + i < N && k < K ? as_float(mat[size_t(n0 + i) * K + k]) : 0.0f;
    }
    float lo = 0.0f, hi = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        lo = fminf(lo, v[i]);
        hi = fmaxf(hi, v[i]);
    }
    const int blocks = geom.group / 32, g = block / blocks;
    if (blocks > 1) {
        lo_s[block][lane] = lo;
        hi_s[block][lane] = hi;
        __syncthreads();
        for (int b = g * blocks; b < (g + 1) * blocks; ++b) {
            lo = fminf(lo, lo_s[b][lane]);
            hi = fmaxf(hi, hi_s[b][lane]);
        }
    }
    uint8_t* unit = out + size_t(blockIdx.z) * geom.matrix_bytes() +
                    k0 / kQ4UnitK * geom.tile_bytes() + size_t(blockIdx.y) * geom.unit_bytes;
    const int column = k0 % kQ4UnitK + lane;
    float s = ZEROS ? __fsub_rn(__fdiv_rn(hi, 15.0f), __fdiv_rn(lo, 15.0f))
                    : __fdiv_rn(fmaxf(hi, -lo), 7.0f);
    s = __bfloat162float(__float2bfloat16_rn(s));
    float z = ZEROS ? 0.0f : 8.0f;
    if (ZEROS && s > 0.0f) z = fminf(fmaxf(rintf(__fdiv_rn(-lo, s)), 0.0f), 15.0f);
    if (block % blocks == 0) {
        const int at = g * kQ4UnitK + column;
        reinterpret_cast<uint16_t*>(unit + kQ4CodeBytes)[at] = uint16_t(__float_as_uint(s) >> 16);
        if (ZEROS) unit[kQ4CodeBytes + kQ4UnitN / geom.group * kQ4UnitK * 2 + at] = uint8_t(z);
    }
    uint32_t word[4];
    if (s > 0.0f) {
        const float r = __fdiv_rn(1.0f, s);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float v8[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v8[e] = v[8 * i + e];
            word[i] = quick_word<ZEROS>(v8, s, r, z);
        }
    } else {
        word[0] = word[1] = word[2] = word[3] = uint32_t(z) * 0x11111111u;
    }
    reinterpret_cast<uint4*>(unit)[block * kQ4UnitK + column] =
        make_uint4(word[0], word[1], word[2], word[3]);
}

// Rows of 16-byte multiples are written 16 bytes at a time (VEC: a thread's four columns are
// neighbours), others 4 (a thread's columns are 32 apart).
template <bool VEC>
__global__ void __launch_bounds__(THREADS)
    q4_dequantize_kernel(const uint8_t* __restrict__ data, float* __restrict__ B, Q4Geom geom) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int y = blockIdx.y * 2 + (warp >> 2), block = warp & 3;
    const int n0 = y * kQ4UnitN + block * 32, k0 = blockIdx.x * kQ4UnitK;
    const int N = geom.N, K = geom.K;
    if (n0 >= N) return;
    const uint8_t* unit = data + size_t(blockIdx.z) * geom.matrix_bytes() +
                          blockIdx.x * geom.tile_bytes() + size_t(y) * geom.unit_bytes;
    const int g = block * 32 / geom.group;
    const uint16_t* scales = reinterpret_cast<const uint16_t*>(unit + kQ4CodeBytes) + g * kQ4UnitK;
    const uint8_t* zeros = unit + kQ4CodeBytes + kQ4UnitN / geom.group * kQ4UnitK * 2 + g * kQ4UnitK;
    uint32_t word[4][4];
    float s[4], z[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int column = VEC ? lane * 4 + j : lane + 32 * j;
        const uint4 w = __ldcs(reinterpret_cast<const uint4*>(unit) + block * kQ4UnitK + column);
        word[j][0] = w.x;
        word[j][1] = w.y;
        word[j][2] = w.z;
        word[j][3] = w.w;
        s[j] = q4_scale(scales[column], geom.fp16);
        // 2^23 + code less 2^23 + z: the difference is exact
        z[j] = 8388608.0f + (geom.zeros ? float(zeros[column]) : 8.0f);
    }
    float* row = B + (size_t(blockIdx.z) * N + n0) * K + k0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (n0 + 8 * i + e >= N) return;
            float f[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t code = (word[j][i] >> (4 * nibble_of(e))) & 15u;
                f[j] = s[j] * (__uint_as_float(0x4b000000u | code) - z[j]);
            }
            if (VEC) {
                if (k0 + lane * 4 < K)
                    __stcs(reinterpret_cast<float4*>(row) + lane, make_float4(f[0], f[1], f[2], f[3]));
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (k0 + lane + 32 * j < K) __stcs(row + lane + 32 * j, f[j]);
            }
            row += K;
        }
}

template <class T>
void launch_quantize(const void* B, bool transposed, size_t values, uint8_t* out, const Q4Geom& g,
                     int count, cudaStream_t stream) {
    const dim3 grid(g.tiles * (kQ4UnitK / Q_WIDTH), g.units, count);
    const T* src = static_cast<const T*>(B);
    if (transposed) {
        if (g.zeros)
            q4_quantize_kernel<T, true, true><<<grid, Q_THREADS, 0, stream>>>(src, values, out, g);
        else
            q4_quantize_kernel<T, true, false><<<grid, Q_THREADS, 0, stream>>>(src, values, out, g);
    } else {
        if (g.zeros)
            q4_quantize_kernel<T, false, true><<<grid, Q_THREADS, 0, stream>>>(src, values, out, g);
        else
            q4_quantize_kernel<T, false, false><<<grid, Q_THREADS, 0, stream>>>(src, values, out, g);
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
    const size_t values = size_t(w->count) * w->N * w->K;
    uint8_t* out = static_cast<uint8_t*>(w->data);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == SGEMM_FLOAT32)
        launch_quantize<float>(B, transposed != 0, values, out, g, w->count, s);
    else if (dtype == SGEMM_BFLOAT16)
        launch_quantize<__nv_bfloat16>(B, transposed != 0, values, out, g, w->count, s);
    else
        launch_quantize<__half>(B, transposed != 0, values, out, g, w->count, s);
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
    q4_pack_kernel<<<tile_grid(g, w->count), THREADS, 0, static_cast<cudaStream_t>(stream)>>>(
        codes, transposed != 0, static_cast<const uint16_t*>(scales), zeros,
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
    const dim3 grid(g.tiles, (g.units + 1) / 2, w->count);
    const uint8_t* data = static_cast<const uint8_t*>(w->data);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (w->K % 4 == 0 && aligned16(B))
        q4_dequantize_kernel<true><<<grid, THREADS, 0, s>>>(data, B, g);
    else
        q4_dequantize_kernel<false><<<grid, THREADS, 0, s>>>(data, B, g);
    count_launch();
    return cudaGetLastError() == cudaSuccess ? SGEMM_OK : SGEMM_ERR_CUDA;
}

}  // extern "C"
