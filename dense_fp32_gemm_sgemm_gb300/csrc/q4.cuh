// The packed 4-bit format and the inner product on it, shared by the packing kernels
// (q4_pack.cu), the few-row product (q4_matmul.cu) and the expert layer (moe.cu).
//
// The product runs on the warp-level matrix instruction m16n8k16 with the weights as its
// 16 x 16 operand: 16 columns of B by 16 steps of n, so that one 32-bit word of a lane
// holds exactly its 8 codes of one instruction. With M of a few rows the bytes of B are
// the cost (2 M operations for half a byte), and this form turns codes into operands in
// registers, without a trip through shared or tensor memory.
//
// A chunk is 16 columns x 128 n. Lane l = 4 r + c of a warp works on columns r and r + 8
// of the 16; in the 32-n block b of the chunk it multiplies n = 32 b + 8 c .. + 7, four of
// them in each of two instructions t = 0, 1 (the n order inside an instruction is free as
// long as both operands agree, and 8 consecutive n let a lane load its part of A as one
// 16-byte word). Word (b, t) of a lane holds, with n0 = 32 b + 8 c + 4 t, in nibbles 0..7:
//   q(r, n0)  q(r+8, n0)  q(r, n0+2)  q(r+8, n0+2)  q(r, n0+1)  q(r+8, n0+1)  q(r, n0+3)  q(r+8, n0+3)
// so that nibbles j and j + 4 (one mask of the word shifted right by 4 j) are the operand's
// register j. A chunk in memory: 2 x 512 bytes of codes (16 bytes a lane: words 0..3, then
// 4..7), then for each of its groups 16 scales, then for each group 16 zero-point bytes if
// any, both in the order r = 0: columns 0, 8; r = 1: columns 1, 9; ...
// A strip is the chunks of 16 columns, n ascending; strips follow one another.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "ptx.cuh"
#include "sgemm.h"

namespace sgemm {

constexpr int kQ4ChunkN = 128;
constexpr int kQ4StripK = 16;
constexpr int kQ4CodeBytes = 1024;  // codes of a chunk

struct Q4Geom {
    int N, K;
    int chunks;       // of a strip
    int strips;       // of a matrix
    int group;        // 32, 64 or 128
    int zeros;        // 1: groups have zero points
    int fp16;         // 1: scales are float16
    int chunk_bytes;  // codes, scales, zero points
    __host__ __device__ size_t strip_bytes() const { return size_t(chunks) * chunk_bytes; }
    __host__ __device__ size_t matrix_bytes() const { return strips * strip_bytes(); }
};

inline Q4Geom q4_geom(const sgemm_q4& w) {
    Q4Geom g;
    g.N = w.N;
    g.K = w.K;
    g.chunks = (w.N + kQ4ChunkN - 1) / kQ4ChunkN;
    g.strips = (w.K + kQ4StripK - 1) / kQ4StripK;
    g.group = w.group;
    g.zeros = (w.flags & SGEMM_Q4_ZEROS) != 0;
    g.fp16 = (w.flags & SGEMM_Q4_SCALE_FP16) != 0;
    g.chunk_bytes = kQ4CodeBytes + (kQ4ChunkN / w.group) * (32 + 16 * g.zeros);
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

// Splits x into pieces whose sum it is: each takes the leading 8 significant bits of what
// is left by truncation, so no piece overflows and the remainder is exact. An infinity or
// NaN is its own first piece and leaves nothing (a difference of infinities would turn it
// into NaN).
template <int P>
__device__ __forceinline__ void split_pieces(float x, float (&piece)[P]) {
    const bool finite = fabsf(x) <= 3.402823466e38f;
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

// Two forms of the weight operand, register j from nibbles j and j + 4 of a word:
//
//  * Plain (five instructions for eight weights). The bfloat16 with the bit pattern of an
//    integer I in 0 .. 255 is I * 2^-133 exactly: its subnormals and its first binade lie on
//    one line, and the matrix instruction takes subnormal operands as they are. So one mask
//    makes an operand: q from the low nibble of each half of the word, 16 q from the next
//    one (columns r + 8, whose sums are scaled by 1/16 afterwards), and one shift by 8 gives
//    the other two. The columns of A^T are staged times 2^96 to bring the products back into
//    FP32's range, and a group's sum is (sum of q x) - z (sum of x), the second sum taken
//    once when the columns are staged.
//  * Centred (eleven): 0x4300 | q is the bfloat16 128 + q, and subtracting 128 + z leaves
//    q - z. Works for every x; taken where a staged value is an infinity, a NaN or outside
//    [2^-64, 2^24), where the scaled product could leave FP32's range.
constexpr float kQ4Low = 0x1p-64f, kQ4High = 0x1p24f;
constexpr float kQ4Scale = 0x1p96f;
constexpr float kQ4Unscale = 0x1p37f;      // 2^133 / 2^96
constexpr float kQ4Unscale16 = 0x1p33f;    // and of 16 q

// Whether x must be multiplied in the centred form.
__device__ __forceinline__ bool q4_special(float x) {
    const float a = fabsf(x);
    return !(a < kQ4High) || (a < kQ4Low && a != 0.0f);
}

// 0x000f000f in a register that the compiler does not see through: with two constants it
// would split the and-or of the centred form into two instructions.
__device__ __forceinline__ uint32_t q4_mask() {
    uint32_t m;
    asm("mov.b32 %0, 0x000f000f;" : "=r"(m));
    return m;
}
__device__ __forceinline__ uint32_t q4_centred(uint32_t shifted_word, uint32_t mask, uint32_t base) {
    uint32_t v;
    asm("lop3.b32 %0, %1, %2, 0x43004300, 0xea;" : "=r"(v) : "r"(shifted_word), "r"(mask));
    const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v),
                                     *reinterpret_cast<const __nv_bfloat162*>(&base));
    return *reinterpret_cast<const uint32_t*>(&d);
}

// D (16 x 8, FP32) = A (16 x 16) . B (16 x 8) + D.
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
        " {%8, %9}, {%0, %1, %2, %3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// D (16 x 8, FP32) = A (16 x 16) . B (16 x 8).
__device__ __forceinline__ void mma_bf16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                               uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
        " {%8, %9}, {%10, %10, %10, %10};\n"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}

// A lane's two scales (columns r and r + 8) from the pair of 16-bit values.
__device__ __forceinline__ void q4_scales(uint32_t pair, int fp16, float& lo, float& hi) {
    if (fp16) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&pair));
        lo = f.x;
        hi = f.y;
    } else {
        lo = __uint_as_float(pair << 16);
        hi = __uint_as_float(pair & 0xffff0000u);
    }
}

// One chunk of MT strips times NT tiles of 8 columns of A^T (a column is a bfloat16 piece of
// a row of A): total[m][nt][0..3] += columns (r, 2c), (r, 2c + 1), (r + 8, 2c), (r + 8, 2c + 1)
// of the 16 x 8 products. chunk(m): the chunk of strip m in shared memory; A(b, nt): the
// lane's 8 consecutive bfloat16 of 32-n block b for column 8 nt + r, as a uint4; in the plain
// form scaled, and sum(g, nt) the pair of -(sum of x) over group g of the chunk for columns
// 8 nt + 2 c and + 1, times 8 without zero points. Each group's product is a sum of integers
// times x, and its scale is applied in FP32, so no weight is rounded.
template <int MT, int NT, int GROUP, bool ZEROS, class Chunk, class LoadA, class Sum>
__device__ __forceinline__ void q4_chunk(Chunk&& chunk, int fp16, int lane, LoadA&& A, Sum&& sum,
                                         float (&total)[MT][NT][4]) {
    constexpr int BLOCKS = GROUP / 32, GROUPS = kQ4ChunkN / GROUP;
    const int r = lane >> 2;
    uint4 word[MT];  // of half a chunk: blocks 2 h and 2 h + 1, two instructions each
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
        uint32_t pair[MT], zero[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const uint8_t* side = chunk(m) + kQ4CodeBytes;
            pair[m] = *reinterpret_cast<const uint32_t*>(side + g * 32 + r * 4);
            zero[m] = 0;
            if constexpr (ZEROS)
                zero[m] = *reinterpret_cast<const uint16_t*>(side + GROUPS * 32 + g * 16 + r * 2);
        }
        float acc[MT][NT][4];
#pragma unroll
        for (int k = 0; k < BLOCKS; ++k) {
            const int b = g * BLOCKS + k;
            if (b % 2 == 0) {
#pragma unroll
                for (int m = 0; m < MT; ++m)
                    word[m] = reinterpret_cast<const uint4*>(chunk(m) + (b / 2) * 512)[lane];
            }
            uint4 x[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) x[nt] = A(b, nt);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const uint32_t w = b % 2 == 0 ? (t == 0 ? word[m].x : word[m].y)
                                                  : (t == 0 ? word[m].z : word[m].w);
                    const uint32_t a[4] = {w & 0x000f000fu, w & 0x00f000f0u,
                                           (w >> 8) & 0x000f000fu, (w >> 8) & 0x00f000f0u};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const uint32_t b0 = t == 0 ? x[nt].x : x[nt].z;
                        const uint32_t b1 = t == 0 ? x[nt].y : x[nt].w;
                        if (k == 0 && t == 0)
                            mma_bf16_first(acc[m][nt], a, b0, b1);
                        else
                            mma_bf16(acc[m][nt], a, b0, b1);
                    }
                }
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const float2 xs = sum(g, nt);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                float z0 = 1.0f, z1 = 1.0f;
                if constexpr (ZEROS) {  // 0x4300 | z is the upper half of the float 128 + z
                    z0 = __uint_as_float(__byte_perm(zero[m], 0x43u, 0x4055)) - 128.0f;
                    z1 = __uint_as_float(__byte_perm(zero[m], 0x43u, 0x4155)) - 128.0f;
                }
                acc[m][nt][0] = fmaf(acc[m][nt][0], kQ4Unscale, z0 * xs.x);
                acc[m][nt][1] = fmaf(acc[m][nt][1], kQ4Unscale, z0 * xs.y);
                acc[m][nt][2] = fmaf(acc[m][nt][2], kQ4Unscale16, z1 * xs.x);
                acc[m][nt][3] = fmaf(acc[m][nt][3], kQ4Unscale16, z1 * xs.y);
            }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            float s0, s1;
            q4_scales(pair[m], fp16, s0, s1);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                total[m][nt][0] = fmaf(s0, acc[m][nt][0], total[m][nt][0]);
                total[m][nt][1] = fmaf(s0, acc[m][nt][1], total[m][nt][1]);
                total[m][nt][2] = fmaf(s1, acc[m][nt][2], total[m][nt][2]);
                total[m][nt][3] = fmaf(s1, acc[m][nt][3], total[m][nt][3]);
            }
        }
    }
}

// One chunk of one strip times a tile of 8 columns in the centred form, added to total. x: the
// lane's word of block 0 of its column, as it is; a block is 64 bytes. Rarely run, so kept
// small rather than unrolled.
template <int GROUP, bool ZEROS>
__device__ __forceinline__ void q4_chunk_centred(const uint8_t* chunk, const uint8_t* x, int fp16,
                                                 int lane, float (&total)[4]) {
    constexpr int BLOCKS = GROUP / 32, GROUPS = kQ4ChunkN / GROUP;
    const int r = lane >> 2;
    const uint32_t mask = q4_mask();
    const uint8_t* side = chunk + kQ4CodeBytes;
#pragma unroll 1
    for (int g = 0; g < GROUPS; ++g) {
        uint32_t z = 0x0808u;
        if constexpr (ZEROS)
            z = *reinterpret_cast<const uint16_t*>(side + GROUPS * 32 + g * 16 + r * 2);
        const uint32_t base0 = __byte_perm(z, 0x43u, 0x4040), base1 = __byte_perm(z, 0x43u, 0x4141);
        float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
        for (int i = 0; i < 2 * BLOCKS; ++i) {
            const int b = g * BLOCKS + i / 2;
            const uint32_t w = *reinterpret_cast<const uint32_t*>(chunk + (b / 2) * 512 + lane * 16 +
                                                                  (b & 1) * 8 + (i & 1) * 4);
            const uint2 xb = *reinterpret_cast<const uint2*>(x + b * 64 + (i & 1) * 8);
            const uint32_t a[4] = {q4_centred(w, mask, base0), q4_centred(w >> 4, mask, base1),
                                   q4_centred(w >> 8, mask, base0),
                                   q4_centred(w >> 12, mask, base1)};
            mma_bf16(acc, a, xb.x, xb.y);
        }
        float s0, s1;
        q4_scales(reinterpret_cast<const uint32_t*>(side + g * 32)[r], fp16, s0, s1);
        total[0] = fmaf(s0, acc[0], total[0]);
        total[1] = fmaf(s0, acc[1], total[1]);
        total[2] = fmaf(s1, acc[2], total[2]);
        total[3] = fmaf(s1, acc[3], total[3]);
    }
}

// Copies `bytes` (a multiple of 16, at most kQ4MaxChunk) of a chunk to shared memory,
// asynchronously: 16 bytes a lane and step.
constexpr int kQ4MaxChunk = kQ4CodeBytes + 4 * 48;
__device__ __forceinline__ void q4_fetch(uint32_t dst, const uint8_t* src, bool tail) {
    ptx::cp_async_16(dst, src, true);
    ptx::cp_async_16(dst + 512, src + 512, true);
    if (tail) ptx::cp_async_16(dst + 1024, src + 1024, true);
}

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
// The P pieces of 8 values, times `scale` (a power of two), and their sums; sets `special` where the plain
// form cannot take one of them.
template <int P, class T>
__device__ __forceinline__ void split_raw8(const Raw8<T>& raw, float scale, bool& special,
                                           uint4 (&out)[P], float (&sum)[P]) {
    const T* e = reinterpret_cast<const T*>(&raw);
    float piece[8][P];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float x = float(e[i]);
        special |= q4_special(x);
        split_pieces<P>(x, piece[i]);
#pragma unroll
        for (int p = 0; p < P; ++p) {
            sum[p] += piece[i][p];
            piece[i][p] *= scale;
        }
    }
#pragma unroll
    for (int p = 0; p < P; ++p)
        out[p] = make_uint4(pack_pieces(piece[0][p], piece[1][p]),
                            pack_pieces(piece[2][p], piece[3][p]),
                            pack_pieces(piece[4][p], piece[5][p]),
                            pack_pieces(piece[6][p], piece[7][p]));
}
}  // namespace sgemm
