// The product on packed weights with warp-level matrix instructions, for few columns of A^T:
// shared by the few-row product (q4_warp.cu) and the expert layer (moe.cu).
//
// The weights are the 16 x 16 operand of m16n8k16, so a warp works on strips of 16 columns of B.
// Lane 4 r + c takes word c of the codes of columns r and r + 8 of a strip: n = 8 c .. 8 c + 7 of
// a block of 32, four of them in each of two instructions (the order of n in an instruction is
// free as long as both operands agree). The matrix pipe takes one such instruction every two
// cycles an SM, 128 weights a cycle and 8 columns, three times what HBM brings; what bounds the
// product is the instructions around it.
#pragma once
#include "q4.cuh"

namespace sgemm {

constexpr int kQ4StripK = 16;
constexpr int kQ4StripsOfTile = kQ4UnitK / kQ4StripK;
constexpr int kQ4ChunkCodes = kQ4CodeBytes / kQ4StripsOfTile;  // of a strip's part of a unit

// Bytes of a strip's part of a unit in shared memory: codes [block][column][16 bytes], scales
// [group][column], zero points [group][column].
__host__ __device__ constexpr int q4_chunk_bytes(int group, int zeros) {
    return kQ4ChunkCodes + kQ4UnitN / group * kQ4StripK * (2 + zeros);
}

// What a lane copies of a chunk besides two times 16 bytes of codes: 16 bytes of scales or zero
// points, if any, at `from` in the unit of the tile's first strip, `step` further for each next
// strip.
struct Q4Side {
    int from, step;
    bool any;
};
template <int GROUP, bool ZEROS>
__device__ __forceinline__ Q4Side q4_side(int lane) {
    constexpr int GROUPS = kQ4UnitN / GROUP;
    Q4Side s;
    if (lane < 2 * GROUPS) {
        s.step = kQ4StripK * 2;
        s.from = kQ4CodeBytes + (lane >> 1) * kQ4UnitK * 2 + (lane & 1) * 16;
    } else {
        s.step = kQ4StripK;
        s.from = kQ4CodeBytes + GROUPS * kQ4UnitK * 2 + (lane - 2 * GROUPS) * kQ4UnitK;
    }
    s.any = lane < (2 + ZEROS) * GROUPS;
    return s;
}
// Copies the chunks of MT strips, from `strip` of the tile on, of a unit to shared memory,
// asynchronously; those past `valid` are left out. dst: the first chunk there; all lanes.
template <int MT>
__device__ __forceinline__ void q4_fetch(uint32_t dst, int chunk_bytes, const uint8_t* unit, int strip,
                                         int valid, int lane, const Q4Side& side) {
    // lane l: column l % 16 of blocks l / 16 and 2 + l / 16
    const uint8_t* codes = unit + (lane >> 4) * (kQ4UnitK * 16) + (strip * kQ4StripK + (lane & 15)) * 16;
    const uint8_t* rest = unit + side.from + strip * side.step;
    dst += lane * 16;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        if (m < valid) {
            ptx::cp_async_16(dst, codes, true);
            ptx::cp_async_16(dst + 512, codes + 2 * kQ4UnitK * 16, true);
            if (side.any) ptx::cp_async_16(dst + kQ4ChunkCodes, rest, true);
        }
        dst += chunk_bytes;
        codes += kQ4StripK * 16;
        rest += side.step;
    }
}

// D (16 x 8, FP32) = A (16 x 16) . B (16 x 8) + D.
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
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

// One chunk of MT strips times NT tiles of 8 columns of A^T: total[m][nt][0..3] += columns
// (r, 2c), (r, 2c + 1), (r + 8, 2c), (r + 8, 2c + 1) of the 16 x 8 products. chunk(m): the chunk of
// strip m in shared memory; A(b, nt): the lane's 8 consecutive bfloat16 of 32-n block b for column
// 8 nt + r, as a uint4, staged for the plain form; sum(g, nt): the pair of -(sum of x) over group
// g of the chunk for columns 8 nt + 2 c and + 1, times 8 without zero points. Each group's product
// is a sum of integers times x, and its scale is applied in FP32, so no weight is rounded.
template <int MT, int NT, int GROUP, bool ZEROS, class Chunk, class LoadA, class Sum>
__device__ __forceinline__ void q4_chunk(Chunk&& chunk, int fp16, int lane, LoadA&& A, Sum&& sum,
                                         float (&total)[MT][NT][4]) {
    constexpr int BLOCKS = GROUP / 32, GROUPS = kQ4UnitN / GROUP;
    const int r = lane >> 2;
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
        float acc[MT][NT][4];
#pragma unroll
        for (int k = 0; k < BLOCKS; ++k) {
            const int b = g * BLOCKS + k;
            uint4 x[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) x[nt] = A(b, nt);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const uint32_t* codes = reinterpret_cast<const uint32_t*>(chunk(m) + b * 256) + lane;
                uint32_t lo[4], hi[4];
                q4_plain(codes[0], lo);
                q4_plain(codes[32], hi);
                const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]};
                const uint32_t a1[4] = {lo[2], hi[2], lo[3], hi[3]};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    if (k == 0)
                        mma_bf16_first(acc[m][nt], a0, x[nt].x, x[nt].y);
                    else
                        mma_bf16(acc[m][nt], a0, x[nt].x, x[nt].y);
                    mma_bf16(acc[m][nt], a1, x[nt].z, x[nt].w);
                }
            }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const uint8_t* side = chunk(m) + kQ4ChunkCodes;
            const uint16_t* scales = reinterpret_cast<const uint16_t*>(side) + g * kQ4StripK + r;
            const float s0 = q4_scale(scales[0], fp16), s1 = q4_scale(scales[8], fp16);
            float z0 = 1.0f, z1 = 1.0f;
            if constexpr (ZEROS) {  // 0x4300 | z is the upper half of the float 128 + z
                const uint8_t* z = side + GROUPS * kQ4StripK * 2 + g * kQ4StripK + r;
                z0 = __uint_as_float(0x43000000u | uint32_t(z[0]) << 16) - 128.0f;
                z1 = __uint_as_float(0x43000000u | uint32_t(z[8]) << 16) - 128.0f;
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float2 xs = sum(g, nt);
                total[m][nt][0] =
                    fmaf(s0, fmaf(acc[m][nt][0], kQ4Unscale, z0 * xs.x), total[m][nt][0]);
                total[m][nt][1] =
                    fmaf(s0, fmaf(acc[m][nt][1], kQ4Unscale, z0 * xs.y), total[m][nt][1]);
                total[m][nt][2] =
                    fmaf(s1, fmaf(acc[m][nt][2], kQ4Unscale, z1 * xs.x), total[m][nt][2]);
                total[m][nt][3] =
                    fmaf(s1, fmaf(acc[m][nt][3], kQ4Unscale, z1 * xs.y), total[m][nt][3]);
            }
        }
    }
}

// One chunk of one strip times a tile of 8 columns in the centred form, added to total. A(b): the
// lane's word of block b of its column, staged for that form; back(g): what the sums of group g are
// to be multiplied with, for columns 2 c and 2 c + 1. Rarely run, so kept small rather than unrolled.
template <int GROUP, bool ZEROS, class LoadA, class Back>
__device__ __forceinline__ void q4_chunk_centred(const uint8_t* chunk, int fp16, int lane, LoadA&& A,
                                                 Back&& back, float (&total)[4]) {
    constexpr int BLOCKS = GROUP / 32, GROUPS = kQ4UnitN / GROUP;
    const int r = lane >> 2;
    const uint8_t* side = chunk + kQ4ChunkCodes;
#pragma unroll 1
    for (int g = 0; g < GROUPS; ++g) {
        uint32_t z0 = 8, z1 = 8;
        if constexpr (ZEROS) {
            const uint8_t* z = side + GROUPS * kQ4StripK * 2 + g * kQ4StripK + r;
            z0 = z[0];
            z1 = z[8];
        }
        const uint32_t base0 = 0x43004300u | z0 * 0x00010001u, base1 = 0x43004300u | z1 * 0x00010001u;
        float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
        for (int b = g * BLOCKS; b < (g + 1) * BLOCKS; ++b) {
            const uint32_t* codes = reinterpret_cast<const uint32_t*>(chunk + b * 256) + lane;
            const uint4 x = A(b);
            uint32_t lo[4], hi[4];
            q4_centred(codes[0], base0, lo);
            q4_centred(codes[32], base1, hi);
            const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]};
            const uint32_t a1[4] = {lo[2], hi[2], lo[3], hi[3]};
            mma_bf16(acc, a0, x.x, x.y);
            mma_bf16(acc, a1, x.z, x.w);
        }
        const uint16_t* scales = reinterpret_cast<const uint16_t*>(side) + g * kQ4StripK + r;
        const float s0 = q4_scale(scales[0], fp16), s1 = q4_scale(scales[8], fp16);
        const float2 f = back(g);
        total[0] = add_centred(s0, f.x, acc[0], total[0]);
        total[1] = add_centred(s0, f.y, acc[1], total[1]);
        total[2] = add_centred(s1, f.x, acc[2], total[2]);
        total[3] = add_centred(s1, f.y, acc[3], total[3]);
    }
}

}  // namespace sgemm
