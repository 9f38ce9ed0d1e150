// The packed 4-bit format and the pieces of the product on it that the packing kernels
// (q4_pack.cu), the few-row product (q4_matmul.cu) and the expert layer (moe.cu) share.
//
// With M of a few rows the bytes of B are the cost (2 M operations for half a byte), so the
// format is built for few instructions a weight. The products run on the tensor core with B^T
// as the operand of many rows: 16 in a warp's registers for few columns (q4_warp.cuh), 128 in
// tensor memory for more (q4_tensor.cu), where a thread owns one column of B (a row of B^T),
// turns its codes into operand words and stores them to its lane.
//
// Operand words cost 5 instructions for 8 weights. The bfloat16 with the bit pattern of an
// integer I in 0 .. 255 is I * 2^-133 exactly: its subnormals and its first binade lie on one
// line, and the tensor core takes subnormal operands as they are. So with a word of 8 codes
//   w & 0x000f000f, w & 0x00f000f0, (w >> 8) & 0x000f000f, (w >> 8) & 0x00f000f0
// are four operand words of two weights each: q, 16 q, q and 16 q. The columns of A^T are
// staged times 2^96 to bring the products back into FP32's range, those that meet 16 q
// times 2^92, and a group's sum is (sum of q x) - z (sum of x), the second sum taken once when
// the columns are staged. Where a staged value is an infinity, a NaN or outside [2^-64, 2^24)
// the scaled product could leave FP32's range; such columns meet the centred form: 0x4300 | q
// is the bfloat16 128 + q, and subtracting 128 + z leaves q - z (eleven instructions). They are
// staged times a power of two that brings the largest of a group (of 32 n, in the expert layer)
// near one, so that neither the sums overflow nor low pieces fall out of bfloat16's range.
//
// What the plain form costs in accuracy: both matrix pipes cut the addends of an instruction (16
// products and the accumulator) at 2^-25 of the largest product's exponent, and take a subnormal's
// exponent for 2^-126, which is that of q = 128. So an addend loses what is below 2^-18 |x|, x the
// largest value of the 16, in units of the scale: 17 2^-18 an instruction, 2^-10 a group of 128 at
// most. The errors are of any sign: at 6144 x 4096 float32 rows are 1.1e-7 of the result's norm off
// 64 bits, where a float32 sum of the dequantised products is 2.5e-7 off. Words of 16 q alone would
// keep four bits more for seven instructions instead of five.
//
// A unit is 128 columns of B times 128 n. In memory:
//   codes: [block of 32 n][column][4 words]; word i of a column's block holds n = 8 i + e of the
//     block, e = 0 .. 7, in nibbles 0, 4, 1, 5, 2, 6, 3, 7 (so that the four operand words hold
//     e = 0, 1; 2, 3; 4, 5; 6, 7);
//   scales: [group][column], 16 bits each;
//   zero points, if any: [group][column], a byte each.
// The units of 128 columns follow one another, n ascending; then the next 128 columns. A warp's
// loads of codes, scales and zero points are consecutive in its lanes. Columns past K and n
// past N are held as zero weights.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "ptx.cuh"
#include "sgemm.h"

namespace sgemm {

constexpr int kQ4UnitN = 128;
constexpr int kQ4UnitK = 128;
constexpr int kQ4CodeBytes = kQ4UnitN * kQ4UnitK / 2;
constexpr int kQ4MaxUnit = kQ4CodeBytes + 4 * kQ4UnitK * 3;

struct Q4Geom {
    int N, K;
    int units;       // along n
    int tiles;       // of 128 columns
    int group;       // 32, 64 or 128
    int zeros;       // 1: groups have zero points
    int fp16;        // 1: scales are float16
    int unit_bytes;  // codes, scales, zero points
    __host__ __device__ size_t tile_bytes() const { return size_t(units) * unit_bytes; }
    __host__ __device__ size_t matrix_bytes() const { return tiles * tile_bytes(); }
};

inline Q4Geom q4_geom(const sgemm_q4& w) {
    Q4Geom g;
    g.N = w.N;
    g.K = w.K;
    g.units = (w.N + kQ4UnitN - 1) / kQ4UnitN;
    g.tiles = (w.K + kQ4UnitK - 1) / kQ4UnitK;
    g.group = w.group;
    g.zeros = (w.flags & SGEMM_Q4_ZEROS) != 0;
    g.fp16 = (w.flags & SGEMM_Q4_SCALE_FP16) != 0;
    g.unit_bytes = kQ4CodeBytes + (kQ4UnitN / w.group) * kQ4UnitK * (2 + g.zeros);
    return g;
}

// The descriptor's limits (its data pointer is not looked at).
inline bool q4_valid(const sgemm_q4* w) {
    return w && w->count >= 1 && w->count <= 4096 && w->N >= 1 && w->N <= 65536 && w->K >= 1 &&
           w->K <= (1 << 20) && (w->group == 32 || w->group == 64 || w->group == 128) &&
           (w->flags & ~(SGEMM_Q4_ZEROS | SGEMM_Q4_SCALE_FP16)) == 0;
}
inline size_t q4_bytes(const sgemm_q4& w) { return size_t(w.count) * q4_geom(w).matrix_bytes(); }

__host__ __device__ constexpr int dtype_bytes(int dtype) { return dtype == SGEMM_FLOAT32 ? 4 : 2; }
inline bool dtype_valid(int dtype) { return dtype >= SGEMM_FLOAT32 && dtype <= SGEMM_FLOAT16; }

// bfloat16 pieces that a value of this type is split into, exactly: 8 of the significant
// bits each, of 8, 11 and 24.
__host__ __device__ constexpr int pieces_of(int dtype) {
    return dtype == SGEMM_FLOAT32 ? 3 : dtype == SGEMM_FLOAT16 ? 2 : 1;
}

// ---- device side -----------------------------------------------------------------------

__device__ __forceinline__ float load_as_float(const void* p, int dtype, size_t i) {
    if (dtype == SGEMM_FLOAT32) return static_cast<const float*>(p)[i];
    if (dtype == SGEMM_BFLOAT16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
    return __half2float(static_cast<const __half*>(p)[i]);
}
__device__ __forceinline__ void store_from_float(void* p, int dtype, size_t i, float v) {
    if (dtype == SGEMM_FLOAT32)
        static_cast<float*>(p)[i] = v;
    else if (dtype == SGEMM_BFLOAT16)
        static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
    else
        static_cast<__half*>(p)[i] = __float2half_rn(v);
}

constexpr float kQ4Low = 0x1p-64f, kQ4High = 0x1p24f;
constexpr float kQ4Scale = 0x1p96f;        // of staged values that meet q
constexpr float kQ4Scale16 = 0x1p92f;      // and 16 q
constexpr float kQ4Unscale = 0x1p37f;      // 2^133 / 2^96

// Splits x into P pieces whose sum it is: each takes the leading 8 significant bits of what
// is left by truncation, so no piece overflows and the remainder is exact. An infinity or
// NaN is its own first piece and leaves nothing (a difference of infinities would turn it
// into NaN). A NaN is made quiet: one whose upper half is an infinity's would become one.
template <int P>
__device__ __forceinline__ void split_pieces(float x, float (&piece)[P]) {
    const bool finite = fabsf(x) <= 3.402823466e38f;
    if (x != x) x = __uint_as_float(__float_as_uint(x) | 0x00400000u);
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const float hi =
            finite ? __uint_as_float(__float_as_uint(x) & 0xffff0000u) : (p == 0 ? x : 0.0f);
        piece[p] = hi;
        x -= hi;
    }
}
// Two such pieces (their low 16 bits are zero) as a pair of bfloat16.
__device__ __forceinline__ uint32_t pack_pieces(float lo, float hi) {
    return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
}

// The four operand words of a word of codes, plain form.
__device__ __forceinline__ void q4_plain(uint32_t w, uint32_t (&a)[4]) {
    a[0] = w & 0x000f000fu;
    a[1] = w & 0x00f000f0u;
    a[2] = (w >> 8) & 0x000f000fu;
    a[3] = (w >> 8) & 0x00f000f0u;
}
// The same, centred; base: the bfloat16 128 + z twice.
__device__ __forceinline__ void q4_centred(uint32_t w, uint32_t base, uint32_t (&a)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t v = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
        const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v),
                                         *reinterpret_cast<const __nv_bfloat162*>(&base));
        a[i] = *reinterpret_cast<const uint32_t*>(&d);
    }
}
__device__ __forceinline__ float q4_scale(uint16_t bits, int fp16) {
    return fp16 ? __half2float(__ushort_as_half(bits)) : __uint_as_float(uint32_t(bits) << 16);
}

template <class T>
__host__ __device__ constexpr int pieces_of_type() { return sizeof(T) == 4 ? 3 : 1; }
template <>
__host__ __device__ constexpr int pieces_of_type<__half>() { return 2; }

// 8 consecutive values of a row as they lie in memory.
template <class T>
struct Raw8 {
    uint4 v[sizeof(T) / 2];
};
// row[n .. n + 8), zeros from N on. vec: rows start on 16-byte boundaries (n is a multiple
// of 8).
template <class T>
__device__ __forceinline__ Raw8<T> load_raw8(const T* row, int n, int N, bool vec) {
    Raw8<T> raw;
    if (vec && n + 8 <= N) {
#pragma unroll
        for (int i = 0; i < int(sizeof(T) / 2); ++i)
            raw.v[i] = reinterpret_cast<const uint4*>(row + n)[i];
    } else {
        T e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = n + i < N ? row[n + i] : T(0.0f);
        raw = *reinterpret_cast<const Raw8<T>*>(e);
    }
    return raw;
}
// The magnitudes of a thread's values, as integers (two 16-bit ones in a word, or one of 32): the
// largest, and the smallest but for zero, less one (zero less one is the largest integer).
struct Magnitudes {
    uint32_t most = 0, least = 0xffffffffu;
    __device__ __forceinline__ void add2(uint32_t w) {
        const uint32_t a = w & 0x7fff7fffu;
        most = __vmaxu2(most, a);
        least = __vminu2(least, __vsub2(a, 0x00010001u));
    }
    __device__ __forceinline__ void add(uint32_t w) {
        const uint32_t a = w & 0x7fffffffu;
        most = max(most, a);
        least = min(least, a - 1);
    }
    // whether the centred form is wanted, by the type's bits of the limits
    template <class T>
    __device__ __forceinline__ bool special() const {
        if constexpr (sizeof(T) == 4)
            return most >= __float_as_uint(kQ4High) || least < __float_as_uint(kQ4Low) - 1;
        const uint32_t m = max(most & 0xffffu, most >> 16), l = min(least & 0xffffu, least >> 16);
        if constexpr (sizeof(T) == 2 && pieces_of_type<T>() == 2)
            return m >= 0x7c00u;  // an infinity or NaN: all other float16 are within the limits
        else
            return m >= __float_as_uint(kQ4High) >> 16 || l < (__float_as_uint(kQ4Low) >> 16) - 1;
    }
};

// The P pieces of 8 values (uint4: places 0 .. 7), for the plain form: times 2^96 and, at places
// 2, 3, 6 and 7 (which meet 16 q), 2^92; and their sums, unscaled, added to `sum`. Not for values that the plain
// form cannot take; those show in `magnitudes`.
template <int P, class T>
__device__ __forceinline__ void split_plain(const Raw8<T>& raw, Magnitudes& magnitudes,
                                            uint4 (&out)[P], float (&sum)[P]) {
    const __nv_bfloat162 scale = __float2bfloat162_rn(kQ4Scale);
    const __nv_bfloat162 scale16 = __float2bfloat162_rn(kQ4Scale16);
    uint32_t word[P][4];
    const uint32_t* in = reinterpret_cast<const uint32_t*>(&raw);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (P == 1) {
            magnitudes.add2(in[i]);
            word[0][i] = in[i];
            sum[0] += __uint_as_float(in[i] << 16) + __uint_as_float(in[i] & 0xffff0000u);
        } else {
            float x[2];
            if constexpr (P == 2) {
                magnitudes.add2(in[i]);
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&in[i]));
                x[0] = f.x;
                x[1] = f.y;
            } else {
                magnitudes.add(in[2 * i]);
                magnitudes.add(in[2 * i + 1]);
                x[0] = __uint_as_float(in[2 * i]);
                x[1] = __uint_as_float(in[2 * i + 1]);
            }
#pragma unroll
            for (int p = 0; p < P; ++p) {
                // the leading 8 significant bits of what is left, by truncation
                word[p][i] = pack_pieces(x[0], x[1]);
                const float lo = __uint_as_float(word[p][i] << 16);
                const float hi = __uint_as_float(word[p][i] & 0xffff0000u);
                sum[p] += lo + hi;
                x[0] -= lo;
                x[1] -= hi;
            }
        }
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&word[p][i]),
                                             (i & 1) ? scale16 : scale);
            word[p][i] = *reinterpret_cast<const uint32_t*>(&v);
        }
    }
#pragma unroll
    for (int p = 0; p < P; ++p) out[p] = make_uint4(word[p][0], word[p][1], word[p][2], word[p][3]);
}
// The power of two that values are staged with for the centred form, from the bits of the largest
// magnitude among them (or an infinity's or NaN's), and its reciprocal, which their sums are
// multiplied with. Within 2^100, which leaves both and what they are multiplied with normal.
struct CentredScale {
    float down, back;
    __device__ __forceinline__ explicit CentredScale(uint32_t most) {
        const int k = min(max(127 - int(most >> 23), -100), 100);
        down = __uint_as_float(uint32_t(127 + k) << 23);
        back = __uint_as_float(uint32_t(127 - k) << 23);
    }
};
// total + s * back * acc, the factors in the order in which nothing overflows or is lost below
// FP32's normal range that would not be in the result.
__device__ __forceinline__ float add_centred(float s, float back, float acc, float total) {
    return (back >= 1.0f) == (fabsf(s) < 1.0f) ? fmaf(s * back, acc, total)
                                               : fmaf(s, back * acc, total);
}
template <class T>
__device__ __forceinline__ uint32_t largest_bits(const Raw8<T>& raw) {
    const T* e = reinterpret_cast<const T*>(&raw);
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) most = max(most, __float_as_uint(float(e[i])) & 0x7fffffffu);
    return most;
}
// The pieces of 8 values times a power of two, for the centred form.
template <int P, class T>
__device__ __forceinline__ void split_centred(const Raw8<T>& raw, float scale, uint4 (&out)[P]) {
    const T* e = reinterpret_cast<const T*>(&raw);
    float piece[8][P];
#pragma unroll
    for (int i = 0; i < 8; ++i) split_pieces<P>(float(e[i]) * scale, piece[i]);
#pragma unroll
    for (int p = 0; p < P; ++p)
        out[p] = make_uint4(pack_pieces(piece[0][p], piece[1][p]),
                            pack_pieces(piece[2][p], piece[3][p]),
                            pack_pieces(piece[4][p], piece[5][p]),
                            pack_pieces(piece[6][p], piece[7][p]));
}

}  // namespace sgemm
