// A mixture-of-experts layer for a few tokens (definition in sgemm.h), in two kernels. The cost is
// reading the weights of the experts that some token picked, once.
//
// moe_route_kernel: a cluster of 8 CTAs a token shares the router's rows, writes the token as
// bfloat16 pieces (staged for the plain form of the weights and, once more, for the centred
// form), and its first CTA chooses the experts.
//
// moe_expert_kernel: every CTA builds the same lists of the picked experts' tokens, cut into tiles
// of so many tokens that an expert's weights are read once for each tile. Then the CTAs take work
// items in order from a counter:
//   first items: one tile x some sets of 32 hidden values, gate and up; h = silu(g) u times
//     the token's weight goes to scratch as bfloat16 pieces;
//   second items: one tile x some sets of 64 columns of the output: the rows of h times down go to
//     scratch in FP32, one row for each token and expert;
//   sum items: 32 columns of 16 tokens' output, each token's rows added in the order of its experts.
// So a token's result does not depend on which other tokens there are. An item that needs earlier
// ones waits for a count of them. Those have been taken before it, by CTAs that are running and
// wait for still earlier ones at most, so every wait ends whatever the number of CTAs that are
// resident. Meanwhile each warp's ring of cp.async stages already fills with the item's weights:
// HBM stays busy across items and across the waits.
//
// The inner product is that of q4_warp.cuh, on sets of four chunks (two strips of gate and of up, or
// four of down), so that a column's words serve four strips (at the largest case below two gave 428 us
// instead of 338, with two pieces a hidden value). The sums of x that zero points take are kept beside the pieces, for each 32 n
// (a group's hidden values may come from several CTAs, but 32 of them come from one). Taken by one
// more matrix instruction on a constant operand, whose sums are truncated, they more than doubled the
// error of float32 layers with zero points (5.8e-7 instead of 2.4e-7 of the result's norm).
//
// Measured, experts of 4096 x 2048, 8 of 64 picked, group 128, bfloat16: one token 42 us (its
// weights take 15.6 at HBM's rate), 64 tokens 410 us (124). 2 of 8 experts of 512 x 512, one token:
// 17 us. What bounds it: with few items, latencies, a third of them for instructions that come from
// far (routing 6 us, lists 2, each phase 4 and its products); with many, the instructions of a set,
// some 400 for one tile of columns, at 16 warps an SM, and in the second product of tiles of more
// than four tokens the matrix instructions, 96 a set at two cycles. A token whose input the centred
// form takes costs more: 79 us instead of 42 for the one token, 580 instead of 410 for one of 64.
#include <cmath>
#include <type_traits>

#include "internal.cuh"
#include "q4_warp.cuh"
#include "wait.cuh"

namespace sgemm {
namespace {

constexpr int kMoeMaxT = 64;
constexpr int kMoeMaxDim = 16384;
constexpr int kMoeMaxE = 256;
constexpr int kMoeMaxTop = 16;

constexpr int ROUTE_CTAS = 8;  // of a token
constexpr int ROUTE_THREADS = 512, ROUTE_WARPS = ROUTE_THREADS / 32;

constexpr int SET = 4;          // chunks that a warp multiplies with the same columns
constexpr int DEPTH = 2;        // stages of a warp's ring, a set of chunks each
constexpr int SUM_COLUMNS = 32, SUM_TOKENS = 16;  // of a sum item
constexpr int WARPS = 8, THREADS = WARPS * 32;
constexpr int SMEM_LIMIT = 227 * 1024;
constexpr int TILE = 8;  // the most tokens of a tile, and columns whose sums are exchanged
constexpr int PITCH = TILE * 17;  // floats of a chunk's sums
// Pieces of a hidden value, whatever the layer's type: all 24 significant bits.
constexpr int H_PIECES = 3;

struct MoeArgs {
    const void* x;
    size_t ldx;
    const void* router;
    int router_dtype, dtype, T, D, F, E, top, renormalize;
    const uint8_t* live;
    int* ids;        // T x top, -1 for a token that is not live
    float* weights;  // T x top
    void* y;
    size_t ldy;
    bool vec;  // rows of x and the router start on 16-byte boundaries
    // scratch
    // pieces as bfloat16, first staged for the plain form, then, x_form and h_form further, for the
    // centred form, each 32 n of a row with a power of two of their own
    uint16_t* xp;      // of x: [token][piece][D padded to units]
    uint16_t* hp;      // of the hidden values: [token and slot][piece][F padded]
    size_t x_form, h_form;
    // sums of 32 values of each piece, times -8 or, where the weights have zero points, -1
    float *x_sum, *h_sum;
    float x_factor, h_factor;
    float *x_back, *h_back;  // what products of 32 values in the centred form are multiplied with
    int* x_special;    // [token]: nonzero where the plain form cannot take some value
    int* h_special;    // [token and slot]
    // 0: next item, 1: first items done, 2: whether some h_special is set, 3 ..: second items done
    // of a group
    int* counters;
    float* z;          // [token and slot][D]
    int* err;
};

struct Stack {
    const uint8_t* data;
    Q4Geom geom;
};

// How the expert kernel cuts its work.
struct MoePlan {
    int capacity;                 // tokens of a tile
    int x_pieces;                 // of a token of x
    int wn1, wn2;                 // warps that split n in first and second items
    int step1, step2;             // bytes from a warp's unit to its next
    ptrdiff_t gate_to_up;
    int sets1, sets2;             // sets of a tile's hidden values (32) and of the output (64)
    int chunk, smem;
};

// ---- routing ---------------------------------------------------------------------------

// The lane's part of x . w: octets lane, lane + 32, ... of [from, to).
template <class T, class R>
__device__ __forceinline__ float dot(const T* x, const R* w, int from, int to, int D, bool vec,
                                     int lane) {
    constexpr int AHEAD = sizeof(T) + sizeof(R) > 4 ? 4 : 8;  // octets in flight
    float s = 0.0f;
    for (int u = from + lane; u < to; u += 32 * AHEAD) {
        Raw8<T> p[AHEAD];
        Raw8<R> q[AHEAD];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j)
            if (u + 32 * j < to) {
                p[j] = load_raw8(x, (u + 32 * j) * 8, D, vec);
                q[j] = load_raw8(w, (u + 32 * j) * 8, D, vec);
            }
#pragma unroll
        for (int j = 0; j < AHEAD; ++j)
            if (u + 32 * j < to) {
                const T* a = reinterpret_cast<const T*>(&p[j]);
                const R* b = reinterpret_cast<const R*>(&q[j]);
#pragma unroll
                for (int i = 0; i < 8; ++i) s = fmaf(float(a[i]), float(b[i]), s);
            }
    }
    return s;
}

// This CTA's share of the token's octets as pieces; true where the plain form cannot take one.
template <class T>
__device__ __forceinline__ bool write_pieces(const MoeArgs& a, int t, int rank, int padded) {
    constexpr int P = pieces_of_type<T>();
    const T* x = static_cast<const T*>(a.x) + t * a.ldx;
    Magnitudes magnitudes;
    const int octets = padded / 8, lane = threadIdx.x & 31;
    for (int first = rank * ROUTE_THREADS + threadIdx.x - lane; first < octets;
         first += ROUTE_CTAS * ROUTE_THREADS) {
        const int u = first + lane;  // octets are a multiple of four
        float sums[P];
#pragma unroll
        for (int p = 0; p < P; ++p) sums[p] = 0.0f;
        Raw8<T> raw;
        uint32_t most = 0;
        if (u < octets) {
            raw = load_raw8(x, u * 8, a.D, a.vec);
            most = largest_bits(raw);
        }
        most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
        most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
        const CentredScale scale(most);
        if (u < octets) {
            uint4 plain[P], centred[P];
            split_plain<P>(raw, magnitudes, plain, sums);
            split_centred<P>(raw, scale.down, centred);
            if (lane % 4 == 0) a.x_back[size_t(t) * (padded / 32) + u / 4] = scale.back;
#pragma unroll
            for (int p = 0; p < P; ++p) {
                uint16_t* to = a.xp + (size_t(t) * P + p) * padded;
                reinterpret_cast<uint4*>(to)[u] = plain[p];
                reinterpret_cast<uint4*>(to + a.x_form)[u] = centred[p];
            }
        }
#pragma unroll
        for (int p = 0; p < P; ++p) {
            sums[p] += __shfl_xor_sync(0xffffffffu, sums[p], 1);
            sums[p] += __shfl_xor_sync(0xffffffffu, sums[p], 2);
            if (u < octets && lane % 4 == 0)
                a.x_sum[(size_t(t) * P + p) * (padded / 32) + u / 4] = sums[p] * a.x_factor;
        }
    }
    return magnitudes.special<T>();
}

// The top experts of a token's logits in ascending order, and their weights; all threads of the
// CTA, a thread an expert. An expert is among them if fewer than `top` others go before it: a
// larger logit, or an equal one and a lower index.
__device__ __forceinline__ void choose(const MoeArgs& a, const float* logit, int t) {
    __shared__ float part[3][ROUTE_WARPS];
    __shared__ int count[ROUTE_WARPS];
    const int e = threadIdx.x, lane = e & 31, warp = e >> 5;
    const float mine = e < a.E ? logit[e] : -INFINITY;
    float biggest = mine;
    for (int o = 16; o > 0; o >>= 1)
        biggest = fmaxf(biggest, __shfl_xor_sync(0xffffffffu, biggest, o));
    if (lane == 0) part[0][warp] = biggest;
    int before = 0;
    if (e < a.E)
#pragma unroll 8
        for (int i = 0; i < a.E; ++i) before += logit[i] > mine || (logit[i] == mine && i < e);
    const bool chosen = e < a.E && before < a.top;
    __syncthreads();
    for (int w = 0; w < ROUTE_WARPS; ++w) biggest = fmaxf(biggest, part[0][w]);
    // an infinite logit shares the weight with its equals, and so do logits that are all -infinity
    const float power = e < a.E ? (mine == biggest ? 1.0f : expf(mine - biggest)) : 0.0f;
    float all = power, some = chosen ? power : 0.0f;
    for (int o = 16; o > 0; o >>= 1) {
        all += __shfl_xor_sync(0xffffffffu, all, o);
        some += __shfl_xor_sync(0xffffffffu, some, o);
    }
    const uint32_t mask = __ballot_sync(0xffffffffu, chosen);
    if (lane == 0) {
        part[1][warp] = all;
        part[2][warp] = some;
        count[warp] = __popc(mask);
    }
    __syncthreads();
    float total = 0.0f;
    for (int w = 0; w < ROUTE_WARPS; ++w) total += part[a.renormalize ? 2 : 1][w];
    int slot = __popc(mask & ((1u << lane) - 1));
    for (int w = 0; w < warp; ++w) slot += count[w];
    if (chosen) {
        a.ids[t * a.top + slot] = e;
        a.weights[t * a.top + slot] = power / total;
    }
}

template <class T, class R>
__global__ void __launch_bounds__(ROUTE_THREADS) moe_route_kernel(const MoeArgs a, int counters,
                                                                  int padded) {
    __shared__ float mine[ROUTE_WARPS];
    __shared__ float logit[kMoeMaxE];          // of the first CTA
    __shared__ int special_of[ROUTE_CTAS];     // and there, each CTA's
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = int(ptx::cluster_ctarank()), t = blockIdx.y;
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    if (t == 0)
        for (int i = rank * ROUTE_THREADS + threadIdx.x; i < counters;
             i += ROUTE_CTAS * ROUTE_THREADS)
            a.counters[i] = 0;
    const bool live = !a.live || a.live[t];  // the same in the whole cluster
    if (!live) {
        if (rank == 0 && threadIdx.x < a.top) {
            a.ids[t * a.top + threadIdx.x] = -1;
            a.weights[t * a.top + threadIdx.x] = 0.0f;
        }
        return;
    }
    // Experts rank, rank + 8, ...: so many warps for each that all have work.
    const int experts = (a.E - rank + ROUTE_CTAS - 1) / ROUTE_CTAS;  // of this CTA
    int split = 1;
    while (split < ROUTE_WARPS && experts * split * 2 <= ROUTE_WARPS) split *= 2;
    const int octets = (a.D + 7) / 8, per = (octets + split - 1) / split;
    ptx::cluster_sync();  // the first CTA is there for what is stored to it
    for (int i0 = 0; i0 < experts; i0 += ROUTE_WARPS / split) {
        const int i = i0 + warp / split, part = warp % split;
        float s = 0.0f;
        if (i < experts) {
            const int e = rank + ROUTE_CTAS * i, from = part * per, to = min(octets, from + per);
            s = dot(static_cast<const T*>(a.x) + t * a.ldx,
                    static_cast<const R*>(a.router) + size_t(e) * a.D, from, to, a.D, a.vec, lane);
        }
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (split > 1) {
            if (lane == 0) mine[warp] = s;
            __syncthreads();
            s = 0.0f;
            for (int w = 0; w < split; ++w) s += mine[warp / split * split + w];
            __syncthreads();
        }
        if (lane == 0 && part == 0 && i < experts)
            ptx::st_shared_cluster_f32(
                ptx::mapa_shared(ptx::smem_u32(logit + rank + ROUTE_CTAS * i), 0),
                s == s ? s : -INFINITY);
    }
    const bool special = __syncthreads_or(write_pieces<T>(a, t, rank, padded));
    if (threadIdx.x == 0)
        ptx::st_shared_cluster_f32(ptx::mapa_shared(ptx::smem_u32(special_of + rank), 0),
                                   __int_as_float(special));
    ptx::cluster_sync();
    if (rank != 0) return;
    choose(a, logit, t);
    if (threadIdx.x < a.top) a.h_special[t * a.top + threadIdx.x] = 0;
    if (threadIdx.x == 0) {
        int any = 0;
        for (int q = 0; q < ROUTE_CTAS; ++q) any |= special_of[q];
        a.x_special[t] = any;
    }
}

// ---- experts -------------------------------------------------------------------------------

// Where the expert kernel's shared memory holds what, in bytes.
struct MoeOffsets {
    int tiles;    // int4 each: expert, first member, members, which of them want the centred form (-1: all)
    int members;  // token and slot, by expert
    int sums;     // [wn][set][chunk][column, TILE of them][17]
    int masks;    // in the same place before: [expert][form][2], and [expert]
    int ring;
    int end;
};
__host__ __device__ constexpr MoeOffsets moe_offsets(int chunk, int tiles, int slots, int E) {
    MoeOffsets o{};
    o.tiles = 0;
    o.members = tiles * 16;
    o.sums = (o.members + slots * 2 + 15) / 16 * 16;
    o.masks = o.sums;
    int most = WARPS * SET * PITCH * 4;
    if (most < E * 20) most = E * 20;
    o.ring = o.sums + (most + 15) / 16 * 16;
    o.end = o.ring + WARPS * DEPTH * SET * chunk;
    return o;
}

// Waits until other CTAs have counted up to `count`; all threads of the CTA. Bounded: when it gives
// up, the rest is computed from what the scratch holds.
__device__ __forceinline__ void wait_count(const int* counter, int count, volatile int* abort_flag,
                                           int* err) {
    if (threadIdx.x == 0 && !*abort_flag) {
        const unsigned long long t0 = ptx::globaltimer_ns();
        while (ptx::ld_acquire_gpu(counter) < count)
            if (ptx::globaltimer_ns() - t0 > WAIT_LIMIT_NS) {
                *abort_flag = 1;
                atomicExch(err, kErrWaitTimeout);
                break;
            }
    }
    __syncthreads();
}

// Tiles of the picked experts' tokens: an expert has at most two that are not full.
__host__ __device__ constexpr int most_tiles(int E, int slots, int capacity) {
    return slots / capacity + 2 * (E < slots ? E : slots);
}

// MT chunks (at stage, stage + chunk, ...) times NT tiles of 8 columns, added to total as in
// q4_chunk. x(b, nt): the lane's 8 values of block b of column 8 nt + r, staged for the plain form;
// sum(g, nt): the kept sums over group g of columns 8 nt + 2 c and + 1. JOIN: joined(b) is multiplied
// too, into the sums of the last tile of columns.
// GROUP 0: the stack's own group size and zero points.
template <int MT, int NT, bool JOIN, int GROUP, bool ZEROS, class X, class Joined, class Sum>
__device__ __forceinline__ void chunk_set(const uint8_t* stage, int chunk, const Q4Geom& geom, int lane,
                                          X&& x, Joined&& joined, Sum&& sum, float (*total)[NT][4]) {
    const int r = lane >> 2;
    const int blocks = GROUP ? GROUP / 32 : geom.group / 32;
    const int groups = GROUP ? kQ4UnitN / (GROUP ? GROUP : 32) : kQ4UnitN / geom.group;
    const bool zeros = GROUP ? ZEROS : geom.zeros != 0;
    constexpr int BLOCKS = GROUP ? GROUP / 32 : 1;
#pragma unroll(NT == 1 && GROUP ? 4 : 1)
    for (int g = 0; g < groups; ++g) {
        float acc[MT][NT][4];
        auto block = [&](int b, bool first) {
            uint4 v[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) v[nt] = x(b, nt);
            uint4 more;
            if constexpr (JOIN) more = joined(b);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const uint32_t* codes =
                    reinterpret_cast<const uint32_t*>(stage + m * chunk + b * 256) + lane;
                uint32_t lo[4], hi[4];
                q4_plain(codes[0], lo);
                q4_plain(codes[32], hi);
                const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]};
                const uint32_t a1[4] = {lo[2], hi[2], lo[3], hi[3]};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    if (first)
                        mma_bf16_first(acc[m][nt], a0, v[nt].x, v[nt].y);
                    else
                        mma_bf16(acc[m][nt], a0, v[nt].x, v[nt].y);
                    mma_bf16(acc[m][nt], a1, v[nt].z, v[nt].w);
                }
                if constexpr (JOIN) {
                    mma_bf16(acc[m][NT - 1], a0, more.x, more.y);
                    mma_bf16(acc[m][NT - 1], a1, more.z, more.w);
                }
            }
        };
        if constexpr (GROUP != 0) {
#pragma unroll
            for (int k = 0; k < BLOCKS; ++k) block(g * BLOCKS + k, k == 0);
        } else {
            block(g * blocks, true);
#pragma unroll 1
            for (int k = 1; k < blocks; ++k) block(g * blocks + k, false);
        }
        float2 xs[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) xs[nt] = sum(g, nt);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const uint8_t* side = stage + m * chunk + kQ4ChunkCodes;
            const uint16_t* scales = reinterpret_cast<const uint16_t*>(side) + g * kQ4StripK + r;
            const float s0 = q4_scale(scales[0], geom.fp16), s1 = q4_scale(scales[8], geom.fp16);
            float z0 = 1.0f, z1 = 1.0f;
            if (zeros) {  // 0x4300 | z is the upper half of the float 128 + z
                const uint8_t* z = side + groups * kQ4StripK * 2 + g * kQ4StripK + r;
                z0 = __uint_as_float(0x43000000u | uint32_t(z[0]) << 16) - 128.0f;
                z1 = __uint_as_float(0x43000000u | uint32_t(z[8]) << 16) - 128.0f;
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float d = fmaf(acc[m][nt][i], kQ4Unscale,
                                         (i < 2 ? z0 : z1) * (i & 1 ? xs[nt].y : xs[nt].x));
                    total[m][nt][i] = fmaf(i < 2 ? s0 : s1, d, total[m][nt][i]);
                }
        }
    }
}
// A group's sum of the kept sums of a unit's four blocks of 32 n.
template <int GROUP>
__device__ __forceinline__ float group_sum(const float* block, int g, int group) {
    if constexpr (GROUP == 32) return block[g];
    if constexpr (GROUP == 64) return block[2 * g] + block[2 * g + 1];
    if constexpr (GROUP == 128) return (block[0] + block[1]) + (block[2] + block[3]);
    float s = 0.0f;
    for (int k = 0; k < group / 32; ++k) s += block[g * (group / 32) + k];
    return s;
}
// What a product reads of a unit of its tile's columns, NT tiles of 8 of them.
struct Columns {
    const uint16_t* x;     // the lane's column of the first tile, staged for the plain form
    const uint16_t* more;  // joined to the sums of the last tile's column, or null
    int padded;            // from a tile's columns to the next one's, and from row to row
    size_t form;           // to the same as they are, for the centred form
    const float* sums;     // of 32 values each; those of columns 2 c and 2 c + 1 of the first tile:
    uint32_t sum_at[2];
    const float* back;     // what products of 32 values in the centred form are multiplied with,
    uint32_t back_at[2];   // for the same columns, in all tiles
    template <int NT, bool JOIN, int GROUP>
    __device__ __forceinline__ float2 group_sums(int g, int nt, int group) const {
        const float* block = sums + nt * (padded / 32);
        float2 s = make_float2(group_sum<GROUP>(block + sum_at[0], g, group),
                               group_sum<GROUP>(block + sum_at[1], g, group));
        if (JOIN && nt == NT - 1) {
            block += padded / 32;
            if (NT == 2) s.x += group_sum<GROUP>(block + sum_at[0], g, group);
            s.y += group_sum<GROUP>(block + sum_at[1], g, group);
        }
        return s;
    }
    // Adds a block's products with the tile nt of columns; at: where the block is in them.
    template <int NT, bool JOIN>
    __device__ __forceinline__ void multiply(const uint32_t (&a0)[4], const uint32_t (&a1)[4], int nt,
                                             size_t at, float (&acc)[4]) const {
        const uint4 v = *reinterpret_cast<const uint4*>(x + nt * padded + at);
        mma_bf16(acc, a0, v.x, v.y);
        mma_bf16(acc, a1, v.z, v.w);
        if (JOIN && nt == NT - 1) {
            uint4 w = make_uint4(0, 0, 0, 0);
            if (more) w = *reinterpret_cast<const uint4*>(more + at);
            mma_bf16(acc, a0, w.x, w.y);
            mma_bf16(acc, a1, w.z, w.w);
        }
    }
};

// A block of 32 n of a strip in the centred form, for the lane's columns r and r + 8 of it.
struct CentredBlock {
    float scale[2], zero[2];  // the zero points: 1 where there are none, for sums times -8
    uint32_t a0[4], a1[4];
    __device__ __forceinline__ CentredBlock(const uint8_t* strip, int b, int g, int group, int zeros,
                                            int fp16) {
        const int lane = threadIdx.x & 31, r = lane >> 2;
        const uint8_t* side = strip + kQ4ChunkCodes;
        const uint16_t* scales = reinterpret_cast<const uint16_t*>(side) + g * kQ4StripK + r;
        const uint32_t* codes = reinterpret_cast<const uint32_t*>(strip + b * 256) + lane;
        uint32_t word[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t z = 8;
            if (zeros) z = side[kQ4UnitN / group * kQ4StripK * 2 + g * kQ4StripK + r + 8 * h];
            scale[h] = q4_scale(scales[8 * h], fp16);
            zero[h] = zeros ? float(z) : 1.0f;
            q4_centred(codes[32 * h], 0x43004300u | z * 0x00010001u, word[h]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a0[i] = word[i & 1][i >> 1];
            a1[i] = word[i & 1][2 + (i >> 1)];
        }
    }
};

// chunk_set of SET chunks in the centred form, whose sums are of 32 n each. Rarely run, so kept small
// rather than unrolled, and a function of its own, which leaves the plain form its registers.
template <int NT, bool JOIN>
__device__ __noinline__ void chunk_set_centred(const uint8_t* stage, int chunk, int group, int zeros, int fp16,
                                               const Columns col, float* kept) {
    const int group_log = 31 - __clz(group / 32);
    float total[SET][NT][4];
#pragma unroll
    for (int i = 0; i < SET * NT * 4; ++i) total[i / (4 * NT)][i / 4 % NT][i % 4] = kept[i];
#pragma unroll
    for (int m = 0; m < SET; ++m)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll 1
            for (int b = 0; b < 4; ++b) {
                const CentredBlock w(stage + m * chunk, b, b >> group_log, group, zeros, fp16);
                float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                col.multiply<NT, JOIN>(w.a0, w.a1, nt, col.form + b * 32, acc);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    total[m][nt][j] =
                        add_centred(w.scale[j >> 1], col.back[col.back_at[j & 1] + b], acc[j], total[m][nt][j]);
            }
#pragma unroll
    for (int i = 0; i < SET * NT * 4; ++i) kept[i] = total[i / (4 * NT)][i / 4 % NT][i % 4];
}

// The same where some columns want that form (special: bits 0 and 1 for columns 2 c and 2 c + 1) and
// some the plain one: both are multiplied, and each column keeps the sums of its own, which are those
// that it has in a tile of one form. So a token's bits do not depend on the others of its tile.
template <int NT, bool JOIN, int GROUP>
__device__ __noinline__ void chunk_set_mixed(const uint8_t* stage, int chunk, int group, int zeros, int fp16,
                                             const Columns col, int special, float* total) {
    const int group_log = 31 - __clz(group / 32), lane = threadIdx.x & 31;
#pragma unroll 1
    for (int i = 0; i < SET * NT; ++i, total += 4) {
        const int m = i / NT, nt = i - m * NT;
        const uint8_t* strip = stage + m * chunk;
        float plain[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
        for (int b = 0; b < 4; ++b) {
            const int g = b >> group_log;
            const CentredBlock w(strip, b, g, group, zeros, fp16);
            float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            col.multiply<NT, JOIN>(w.a0, w.a1, nt, col.form + b * 32, acc);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (special >> (j & 1) & 1)
                    total[j] = add_centred(w.scale[j >> 1], col.back[col.back_at[j & 1] + b], acc[j], total[j]);
            const uint32_t* codes = reinterpret_cast<const uint32_t*>(strip + b * 256) + lane;
            uint32_t lo[4], hi[4];
            q4_plain(codes[0], lo);
            q4_plain(codes[32], hi);
            const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]}, a1[4] = {lo[2], hi[2], lo[3], hi[3]};
            col.multiply<NT, JOIN>(a0, a1, nt, b * 32, plain);
            if ((b + 1) >> group_log == g) continue;
            const float2 xs = col.group_sums<NT, JOIN, GROUP>(g, nt, group);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float d = fmaf(plain[j], kQ4Unscale, w.zero[j >> 1] * (j & 1 ? xs.y : xs.x));
                if (!(special >> (j & 1) & 1)) total[j] = fmaf(w.scale[j >> 1], d, total[j]);
                plain[j] = 0.0f;
            }
        }
    }
}

// The columns of A^T of a tile of tokens. Where tiles are of one or two tokens, a piece has a column
// of its own (NT_MOST 1). With larger ones a token has two columns at most, and a third piece is
// multiplied into the sums of the second: with a column of its own it would take eight tokens to 24
// columns and more registers than there are (64 tokens: 430 us instead of 410). One tile of columns
// holds all of them (column `columns` * m + p) where they fit; else there are two, and column m of
// each is token m's: a thread then adds its tokens' sums before they are exchanged. So the order of
// a token's sums does not depend on how many share the tile.
__device__ __forceinline__ bool packed_columns(int tokens, int columns) { return tokens * columns <= TILE; }

// NT_MOST: tiles of 8 columns that a tile of tokens may take.
template <int NT_MOST, int GROUP, bool ZEROS>
__global__ void __launch_bounds__(THREADS, 2)
    moe_expert_kernel(const MoeArgs a, const Stack gate, const Stack down,
                      const MoePlan plan) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int scan_s[WARPS], tiles_s, item_s;
    // the item after the current one, -1 while it is not known; two places in turn
    __shared__ volatile int next_s[2];
    __shared__ volatile int abort_s;
    constexpr int warps = WARPS, threads = THREADS;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = lane >> 2, c = lane & 3;
    const int slots = a.T * a.top;
    const int max_tiles = most_tiles(a.E, slots, plan.capacity);
    const MoeOffsets at =
        moe_offsets(plan.chunk, max_tiles, slots, a.E);
    int4* tile_s = reinterpret_cast<int4*>(smem + at.tiles);
    uint16_t* member_s = reinterpret_cast<uint16_t*>(smem + at.members);
    float* sums = reinterpret_cast<float*>(smem + at.sums);
    uint8_t* ring = smem + at.ring + warp * DEPTH * SET * plan.chunk;
    // first items: wm1 sets of wn1 warps each; second items: wm2 sets of wn2 warps each
    const int wn1 = warp & (plan.wn1 - 1), wm1 = warp / plan.wn1, sets1_item = warps / plan.wn1;
    const int wn2 = warp & (plan.wn2 - 1), wm2 = warp / plan.wn2, sets2_item = warps / plan.wn2;

    // what does not depend on the routing, while that runs
    const int groups1 = (plan.sets1 + sets1_item - 1) / sets1_item;
    const int groups2 = (plan.sets2 + sets2_item - 1) / sets2_item;
    const int sum_columns = (a.D + SUM_COLUMNS - 1) / SUM_COLUMNS;
    const int x_padded = gate.geom.units * kQ4UnitN, h_padded = down.geom.units * kQ4UnitN;
    // what a lane copies besides codes, for the gate and up stacks and for down
    auto side_of = [&](const Q4Geom& g) {
        const int groups = kQ4UnitN / g.group;
        Q4Side s;
        const bool zero = lane >= 2 * groups;  // zero points
        s.step = zero ? kQ4StripK : kQ4StripK * 2;
        s.from = kQ4CodeBytes + (zero ? groups * kQ4UnitK * 2 + (lane - 2 * groups) * kQ4UnitK
                                      : (lane >> 1) * kQ4UnitK * 2 + (lane & 1) * 16);
        s.any = lane < (2 + g.zeros) * groups;
        return s;
    };
    // [expert][form][2], and [expert]
    uint32_t* mask_s = reinterpret_cast<uint32_t*>(smem + at.masks);
    int* first_s = reinterpret_cast<int*>(mask_s + 4 * a.E);
    for (int i = tid; i < 4 * a.E; i += threads) mask_s[i] = 0;
    if (tid == 0) {
        abort_s = 0;
        next_s[0] = next_s[1] = -1;
    }
    __syncthreads();
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    int claimed = 0;
    if (tid == 0) claimed = atomicAdd(a.counters, 1);

    // The tokens of each expert, in order, in tiles; the same in every CTA. Tokens that want the
    // centred form have tiles of their own, so that the others need not take its time. A token
    // picks an expert once, so an expert's tokens are a 64-bit mask (one for each form).
    {
        for (int i = tid; i < slots; i += threads) {
            const int e = a.ids[i], t = i / a.top;
            const int form = a.x_special[t] != 0;
            if (e >= 0) atomicOr(mask_s + 4 * e + 2 * form + (t >> 5), 1u << (t & 31));
        }
        __syncthreads();
        int plain = 0, centred = 0;
        if (tid < a.E) {
            plain = __popc(mask_s[4 * tid]) + __popc(mask_s[4 * tid + 1]);
            centred = __popc(mask_s[4 * tid + 2]) + __popc(mask_s[4 * tid + 3]);
        }
        const int plain_tiles = (plain + plan.capacity - 1) / plan.capacity;
        const int my_tiles = plain_tiles + (centred + plan.capacity - 1) / plan.capacity;
        // tiles and members before this expert's: a scan over the threads
        const int own = my_tiles << 16 | (plain + centred);
        int scan = own;
        for (int o = 1; o < 32; o *= 2) {
            const int v = __shfl_up_sync(0xffffffffu, scan, o);
            if (lane >= o) scan += v;
        }
        if (lane == 31) scan_s[warp] = scan;
        __syncthreads();
        int before = scan - own;
        for (int w = 0; w < warp; ++w) before += scan_s[w];
        const int first_tile = before >> 16, first = before & 0xffff;
        if (tid < a.E) {
            first_s[tid] = first;
            for (int k = 0; k < my_tiles; ++k) {
                const bool other = k >= plain_tiles;
                const int from = (other ? k - plain_tiles : k) * plan.capacity;
                int4 tile;
                tile.x = tid;
                tile.y = first + (other ? plain : 0) + from;
                tile.z = min(plan.capacity, (other ? centred : plain) - from);
                tile.w = other ? -1 : 0;
                tile_s[first_tile + k] = tile;
            }
        }
        if (tid == threads - 1) tiles_s = (before + own) >> 16;
        if (tid == 0) item_s = claimed;
        __syncthreads();
        for (int i = tid; i < slots; i += threads) {
            const int e = a.ids[i], t = i / a.top;
            if (e < 0) continue;
            const uint32_t* mask = mask_s + 4 * e;
            const bool other = (mask[2 + (t >> 5)] >> (t & 31)) & 1;
            const uint32_t* own_mask = mask + (other ? 2 : 0);
            int n = first_s[e] + __popc(own_mask[t >> 5] & ((1u << (t & 31)) - 1));
            if (t >= 32) n += __popc(own_mask[0]);
            if (other) n += __popc(mask[0]) + __popc(mask[1]);
            member_s[n] = uint16_t(i);
        }
        __syncthreads();
    }
    auto columns_of = [&](int pieces) { return NT_MOST == 1 ? pieces : min(pieces, 2); };
    const int tiles = tiles_s;
    const int first_items = tiles * groups1, second_items = tiles * groups2;
    const int items = first_items + second_items +
                      sum_columns * ((a.T + SUM_TOKENS - 1) / SUM_TOKENS);

    // Where a warp is in an item. kind 0: strips `strip` and + 1 of gate and up of the tile's
    // expert, units wn1, wn1 + plan.wn1, ...; 1: strips `strip` .. + 3 of down, units wn2, ...;
    // 2: nothing to fetch. The packed columns are a multiple of eight strips.
    struct Walk {
        int kind, strip, tile, unit, left;
    };
    auto walk = [&](int item) {
        Walk w;
        w.kind = 2;
        w.strip = w.tile = w.unit = w.left = 0;
        if (item < first_items) {
            w.kind = 0;
            w.tile = item / groups1;
            const int set = (item - w.tile * groups1) * sets1_item + wm1;
            w.strip = 2 * set;
            w.unit = wn1;
            if (set < plan.sets1) w.left = (gate.geom.units - wn1 + plan.wn1 - 1) / plan.wn1;
        } else if (item < first_items + second_items) {
            item -= first_items;
            w.kind = 1;
            w.tile = item / groups2;
            const int set = (item - w.tile * groups2) * sets2_item + wm2;
            w.strip = 4 * set;
            w.unit = wn2;
            if (set < plan.sets2) w.left = (down.geom.units - wn2 + plan.wn2 - 1) / plan.wn2;
        }
        return w;
    };
    auto advance = [&](Walk& w) {
        --w.left;
        w.unit += w.kind == 0 ? plan.wn1 : plan.wn2;
    };

    // ---- the ring
    const uint32_t ring_u32 = ptx::smem_u32(ring);
    uint32_t fetch_to = ring_u32;
    const int stage_bytes = SET * plan.chunk;
    int turn = 0;   // of next_s
    int claim_at = 0;  // units left when the next item is claimed
    int f_on = 0;   // the walk is in the current item (0) or the next (1)
    int ahead = 0;  // stages fetched and not used up
    Walk f = walk(item_s);
    // where the lane's next codes and scales or zero points are, and the latter's step to the next
    // strip
    const uint8_t *f_codes = nullptr, *f_rest = nullptr;
    int f_side = 0;
    bool f_any = false;
    auto locate = [&]() {
        if (f.left == 0) return;
        const Stack& stack = f.kind == 0 ? gate : down;
        const int in_tile = f.strip % kQ4StripsOfTile;
        const Q4Side side = side_of(stack.geom);
        const uint8_t* unit = stack.data + tile_s[f.tile].x * stack.geom.matrix_bytes() +
                              size_t(f.strip / kQ4StripsOfTile) * stack.geom.tile_bytes() +
                              size_t(f.unit) * stack.geom.unit_bytes;
        f_codes = unit + (lane >> 4) * (kQ4UnitK * 16) + (in_tile * kQ4StripK + (lane & 15)) * 16;
        f_rest = unit + side.from + in_tile * side.step;
        f_side = side.step;
        f_any = side.any;
    };
    auto fetch = [&]() -> bool {
        if (f.left == 0) {
            if (f_on == 1) return false;
            const int next = __shfl_sync(0xffffffffu, next_s[turn], 0);
            if (next < 0) return false;
            f = walk(next);
            locate();
            f_on = 1;
            if (f.left == 0) return false;
        }
        uint32_t to = fetch_to + lane * 16;
        const uint8_t *codes = f_codes, *rest = f_rest;
        // from a chunk to the second (as from the third to the fourth), and to the third
        const bool second = f.kind != 0;
        const ptrdiff_t codes2 = second ? kQ4StripK * 16 : plan.gate_to_up;
        const ptrdiff_t rest2 = second ? f_side : plan.gate_to_up;
        const int codes3 = second ? 2 * kQ4StripK * 16 : kQ4StripK * 16;
        const int rest3 = second ? 2 * f_side : f_side;
#pragma unroll
        for (int m = 0; m < SET; m += 2) {
            const uint32_t to2 = to + plan.chunk;
            ptx::cp_async_16(to, codes, true);
            ptx::cp_async_16(to + 512, codes + 2 * kQ4UnitK * 16, true);
            ptx::cp_async_16(to2, codes + codes2, true);
            ptx::cp_async_16(to2 + 512, codes + codes2 + 2 * kQ4UnitK * 16, true);
            if (f_any) {
                ptx::cp_async_16(to + kQ4ChunkCodes, rest, true);
                ptx::cp_async_16(to2 + kQ4ChunkCodes, rest + rest2, true);
            }
            to = to2 + plan.chunk;
            codes += codes3;
            rest += rest3;
        }
        ptx::cp_async_commit();
        const int step = second ? plan.step2 : plan.step1;
        f_codes += step;
        f_rest += step;
        --f.left;
        ++ahead;
        fetch_to += stage_bytes;
        if (fetch_to == ring_u32 + DEPTH * stage_bytes) fetch_to = ring_u32;
        return true;
    };
    // Fills up the ring again, the stage used before being free, and waits for the oldest.
    static_assert(DEPTH == 2, "the waits");
    auto acquire = [&]() {
        __syncwarp();
        if (ahead < DEPTH && fetch() && ahead < DEPTH) fetch();
        if (ahead == DEPTH)
            ptx::cp_async_wait<DEPTH - 1>();
        else
            ptx::cp_async_wait<0>();
        __syncwarp();
    };
    const uint8_t* stage = ring;
    auto release = [&]() {
        --ahead;
        stage += stage_bytes;
        if (stage == ring + DEPTH * stage_bytes) stage = ring;
    };
    locate();
#pragma unroll 1
    while (ahead < DEPTH && fetch()) {
    }

    // The first thread's claim of the next item: none or through (0), wanted (1), asked for (2).
    int claim = 0, ticket = 0;
    auto claim_step = [&]() {
        if (claim == 1)
            ticket = atomicAdd(a.counters, 1);
        else if (claim == 2)
            next_s[turn] = ticket;
        claim = claim == 1 ? 2 : 0;
    };

    // Multiplies the warp's set of an item with the columns of its tile of tokens and puts the sums
    // to [wn][set][chunk][column][17]. One copy of this code serves both kinds of items: it is most
    // of the kernel, and where there are few items its instructions come from far.
    auto product = [&](const int4& tile, Walk& w) {
        const bool second = w.kind != 0;
        const Q4Geom& geom = second ? down.geom : gate.geom;
        const int pieces = second ? H_PIECES : plan.x_pieces;
        const int token_columns = columns_of(pieces);
        const bool packed = packed_columns(tile.z, token_columns);
        const int padded = second ? h_padded : x_padded;
        const uint32_t per_row = second ? 1 : a.top;
        const int place = second ? wn2 * sets2_item + wm2 : wn1 * sets1_item + wm1;
        const float* sum_rows = second ? a.h_sum : a.x_sum;
        const uint16_t* rows = second ? a.hp : a.xp;
        auto run = [&](auto nt_, auto join_) {
            constexpr int NT = decltype(nt_)::value;
            constexpr bool JOIN = decltype(join_)::value;
            // columns that do not exist repeat the first, and their sums are not used
            const int apart = NT == 1 ? token_columns : 1;
            auto token_of = [&](int j) { return apart == 1 ? j : apart == 2 ? j >> 1 : j * 11 >> 5; };
            auto token_row = [&](int m) {
                return uint32_t(member_s[tile.y + (m < tile.z ? m : 0)]) / per_row;
            };
            auto row_of = [&](int j) {
                const int m = token_of(j), p = j - m * apart;
                return token_row(m) * pieces + (m < tile.z ? p : 0);
            };
            // of the first tile of columns; the next piece's are `padded` further. The third
            // piece of first columns is nothing.
            const uint16_t* const col = rows + size_t(row_of(r)) * padded + c * 8;
            const bool joins = NT == 2 || (r & 1);
            // of columns 2 c and 2 c + 1, in their units' first block
            const uint32_t sum_at[2] = {row_of(2 * c) * uint32_t(padded / 32),
                                        row_of(2 * c + 1) * uint32_t(padded / 32)};
            float total[SET][NT][4];
#pragma unroll
            for (int m = 0; m < SET; ++m)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) total[m][nt][i] = 0.0f;
#pragma unroll 1
            while (w.left > 0) {
                if (warp == 0 && w.left <= claim_at) claim_step();
                Columns here;
                here.x = col + w.unit * kQ4UnitN;
                here.more = joins ? here.x + NT * padded : nullptr;
                here.padded = padded;
                here.form = second ? a.h_form : a.x_form;
                here.sums = sum_rows + w.unit * (kQ4UnitN / 32);
                here.sum_at[0] = sum_at[0];
                here.sum_at[1] = sum_at[1];
                const int unit = w.unit;
                auto more = [&](int b) {
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (joins) v = *reinterpret_cast<const uint4*>(here.more + b * 32);
                    return v;
                };
                advance(w);
                if (tile.w) {
                    const int special =
                        (tile.w >> token_of(2 * c) & 1) | (tile.w >> token_of(2 * c + 1) & 1) << 1;
                    here.back = (second ? a.h_back : a.x_back) + unit * (kQ4UnitN / 32);
                    for (int i = 0; i < 2; ++i)
                        here.back_at[i] = token_row(token_of(2 * c + i)) * uint32_t(padded / 32);
                    float kept[SET * NT * 4];
                    auto move = [&](bool back) {
#pragma unroll
                        for (int i = 0; i < SET * NT * 4; ++i) {
                            float& t = total[i / (4 * NT)][i / 4 % NT][i % 4];
                            back ? t = kept[i] : kept[i] = t;
                        }
                    };
                    acquire();
                    move(false);
                    if (tile.w == -1)
                        chunk_set_centred<NT, JOIN>(stage, plan.chunk, geom.group, geom.zeros, geom.fp16,
                                                    here, kept);
                    else
                        chunk_set_mixed<NT, JOIN, GROUP>(stage, plan.chunk, geom.group, geom.zeros,
                                                         geom.fp16, here, special, kept);
                    move(true);
                } else {
                    if constexpr (NT == 1 && GROUP != 0 && !JOIN) {
                        // all four blocks' words at once, while the stage is waited for
                        uint4 x[4];
#pragma unroll
                        for (int b = 0; b < 4; ++b)
                            x[b] = *reinterpret_cast<const uint4*>(here.x + b * 32);
                        __align__(16) float block[2][4];
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            *reinterpret_cast<float4*>(block[i]) =
                                *reinterpret_cast<const float4*>(here.sums + sum_at[i]);
                        acquire();
                        chunk_set<SET, 1, false, GROUP, ZEROS>(
                            stage, plan.chunk, geom, lane, [&](int b, int) { return x[b]; }, more,
                            [&](int g, int) {
                                return make_float2(group_sum<GROUP>(block[0], g, GROUP),
                                                   group_sum<GROUP>(block[1], g, GROUP));
                            },
                            total);
                    } else {
                        // no registers for words ahead, and with more columns for two chunks at a time
                        constexpr int MT = NT == 1 ? SET : 2;
                        acquire();
#pragma unroll
                        for (int m = 0; m < SET; m += MT)
                            chunk_set<MT, NT, JOIN, GROUP, ZEROS>(
                                stage + m * plan.chunk, plan.chunk, geom, lane,
                                [&](int b, int nt) {
                                    return *reinterpret_cast<const uint4*>(here.x + nt * padded + b * 32);
                                },
                                more,
                                [&](int g, int nt) {
                                    return here.template group_sums<NT, JOIN, GROUP>(g, nt, geom.group);
                                },
                                total + m);
                    }
                }
                release();
            }
            float* mine = sums + place * SET * PITCH + r;
            const int columns = NT == 1 ? tile.z * token_columns : tile.z;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int j = 2 * c + i;
                if (j < columns)
#pragma unroll
                    for (int m = 0; m < SET; ++m) {
                        float v = total[m][0][i], v8 = total[m][0][i + 2];
#pragma unroll
                        for (int nt = 1; nt < NT; ++nt) {
                            v += total[m][nt][i];
                            v8 += total[m][nt][i + 2];
                        }
                        mine[m * PITCH + j * 17] = v;
                        mine[m * PITCH + j * 17 + 8] = v8;
                    }
            }
        };
        constexpr std::integral_constant<int, 1> one{};
        constexpr std::integral_constant<int, 2> two{};
        if constexpr (NT_MOST == 1) {
            run(one, std::false_type());
        } else if (pieces == 3) {
            if (packed)
                run(one, std::true_type());
            else
                run(two, std::true_type());
        } else {
            if (packed)
                run(one, std::false_type());
            else
                run(two, std::false_type());
        }
    };
    // A token's sum from one warp of those that split n: its pieces' that are there.
    auto sum_of = [&](const float* from, int apart) {
        float v = from[0];
        if (apart > 1) v += from[17];
        if (apart > 2) v += from[34];
        return v;
    };

    // ---- the items
    bool hidden_ready = false;
    int item = item_s;
    while (item < items) {
        // The next item is claimed when the first warp is near this one's end, not before: where
        // there is about one item for each CTA, none should hold two. Far from the end of a phase
        // it may be claimed at once.
        claim = tid == 0;
        const int phase_end = item < first_items ? first_items : first_items + second_items;
        claim_at = item + 3 * int(gridDim.x) < phase_end ? INT_MAX : DEPTH + 1;
        Walk w = walk(item);
#pragma unroll 1
        while (ahead < DEPTH && fetch()) {
        }
        if (item >= first_items && item < first_items + second_items && !hidden_ready) {
            wait_count(a.counters + 1, first_items, &abort_s, a.err);
            // members with a hidden value that the plain form cannot take
            const bool some = __ldcg(a.counters + 2) != 0;
            for (int k = tid; k < tiles; k += threads) {
                const int4 tile = tile_s[k];
                int special = 0;
                if (some)
                    for (int i = 0; i < tile.z; ++i)
                        special |= (__ldcg(a.h_special + member_s[tile.y + i]) != 0) << i;
                tile_s[k].w = special == (1 << tile.z) - 1 ? -1 : special;
            }
            __syncthreads();
            hidden_ready = true;
        }
        int4 tile = make_int4(0, 0, 0, 0);
        if (item < first_items + second_items) {
            tile = tile_s[w.tile];
            product(tile, w);
            __syncthreads();
        }
        if (item < first_items) {
            const int width = sets1_item * 32, f0 = (item - w.tile * groups1) * width;
            const int token_columns = columns_of(plan.x_pieces);
            const int apart = packed_columns(tile.z, token_columns) ? token_columns : 1;
            for (int i = tid; i < tile.z * width; i += threads) {
                const int m = i / width, k = i - m * width;
                const int f_at = f0 + k;
                if (f_at >= plan.sets1 * 32) continue;
                float g = 0.0f, u = 0.0f;
                const float* from = sums + (k / kQ4StripK) * 2 * PITCH +  // two of a set
                                    m * apart * 17 + k % kQ4StripK;
#pragma unroll 4
                for (int q = 0; q < plan.wn1; ++q) {
                    g += sum_of(from + q * sets1_item * SET * PITCH, apart);
                    u += sum_of(from + q * sets1_item * SET * PITCH + PITCH, apart);
                }
                const int slot = member_s[tile.y + m];
                const float h = f_at < a.F ? g / (1.0f + expf(-g)) * u * a.weights[slot] : 0.0f;
                float piece[H_PIECES];
                split_pieces<H_PIECES>(h, piece);
                Magnitudes magnitude;
                magnitude.add(__float_as_uint(h));
                if (magnitude.special<float>()) {
                    a.h_special[slot] = 1;
                    a.counters[2] = 1;
                }
                const float scale = (f_at & 2) ? kQ4Scale16 : kQ4Scale;  // by place, as in x
                // a warp's 32 values are one token's
                const CentredScale centred(
                    __reduce_max_sync(0xffffffffu, __float_as_uint(h) & 0x7fffffffu));
                float centred_piece[H_PIECES];
                split_pieces<H_PIECES>(h * centred.down, centred_piece);
                if (lane == 0) a.h_back[size_t(slot) * (h_padded / 32) + f_at / 32] = centred.back;
#pragma unroll
                for (int p = 0; p < H_PIECES; ++p) {
                    float sum = piece[p];
                    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    if (lane == 0)
                        a.h_sum[(size_t(slot) * H_PIECES + p) * (h_padded / 32) + f_at / 32] =
                            sum * a.h_factor;
                    uint16_t* to = a.hp + (size_t(slot) * H_PIECES + p) * h_padded + f_at;
                    to[0] = uint16_t(__float_as_uint(piece[p] * scale) >> 16);
                    to[a.h_form] = uint16_t(__float_as_uint(centred_piece[p]) >> 16);
                }
            }
            // past F: down's weights are zero there, but not whatever the scratch holds
            if (f0 + width >= plan.sets1 * 32) {
                const int from = plan.sets1 * 32, rest = h_padded - from;
                for (int i = tid; i < tile.z * H_PIECES * rest; i += threads) {
                    const int line = i / rest, m = line / H_PIECES;
                    const size_t row = size_t(member_s[tile.y + m]) * H_PIECES + line % H_PIECES;
                    uint16_t* to = a.hp + row * h_padded + from + i % rest;
                    to[0] = to[a.h_form] = 0;
                    if (i % rest % 32 == 0) {
                        a.h_sum[row * (h_padded / 32) + (from + i % rest) / 32] = 0.0f;
                        a.h_back[row / H_PIECES * (h_padded / 32) + (from + i % rest) / 32] = 1.0f;
                    }
                }
            }
            __syncthreads();
            if (tid == 0) ptx::red_release_gpu_add(a.counters + 1, 1);
        } else if (item < first_items + second_items) {
            const int group = item - first_items - w.tile * groups2;
            const int width = sets2_item * 64;
            const int token_columns = columns_of(H_PIECES);
            const int apart = packed_columns(tile.z, token_columns) ? token_columns : 1;
            for (int i = tid; i < tile.z * width; i += threads) {
                const int m = i / width, k = i - m * width, d = group * width + k;
                if (d >= a.D) continue;
                float v = 0.0f;
                const float* from = sums + (k / kQ4StripK) * PITCH + m * apart * 17 + k % kQ4StripK;
#pragma unroll 4
                for (int q = 0; q < plan.wn2; ++q) v += sum_of(from + q * sets2_item * SET * PITCH, apart);
                a.z[size_t(member_s[tile.y + m]) * a.D + d] = v;
            }
            __syncthreads();
            if (tid == 0) ptx::red_release_gpu_add(a.counters + 3 + group, 1);
        } else {
            // some columns of some tokens' output: their rows in the order of the experts
            const int at = item - first_items - second_items;
            const int d0 = at % sum_columns * SUM_COLUMNS, t0 = at / sum_columns * SUM_TOKENS;
            wait_count(a.counters + 3 + d0 / (64 * sets2_item), tiles, &abort_s, a.err);
            for (int i = tid; i < SUM_TOKENS * SUM_COLUMNS; i += threads) {
                const int t = t0 + i / SUM_COLUMNS, d = d0 + i % SUM_COLUMNS;
                if (t >= a.T || d >= a.D) continue;
                float v = 0.0f;
                if (a.ids[t * a.top] >= 0)
                    for (int j0 = 0; j0 < a.top; j0 += 8) {
                        float z[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            z[j] = j0 + j < a.top ? __ldcg(a.z + size_t(t * a.top + j0 + j) * a.D + d)
                                                  : 0.0f;
#pragma unroll
                        for (int j = 0; j < 8; ++j) v += z[j];
                    }
                store_from_float(a.y, a.dtype, t * a.ldy + d, v);
            }
        }
        // all have read the other place since they took this item from it
        if (tid == 0) next_s[turn ^ 1] = -1;
        if (claim == 1) claim_step();
        if (claim == 2) claim_step();
        __syncthreads();
        item = next_s[turn];
        turn ^= 1;
        if (f_on == 0) {  // the walk is through the item that was
            f = walk(item);
            locate();
        }
        f_on = 0;
    }
    ptx::cp_async_wait<0>();
}

template <class T>
cudaError_t launch_route(const cudaLaunchConfig_t& config, const MoeArgs& a, int counters, int padded) {
    if (a.router_dtype == SGEMM_FLOAT32)
        return cudaLaunchKernelEx(&config, moe_route_kernel<T, float>, a, counters, padded);
    if (a.router_dtype == SGEMM_BFLOAT16)
        return cudaLaunchKernelEx(&config, moe_route_kernel<T, __nv_bfloat16>, a, counters, padded);
    return cudaLaunchKernelEx(&config, moe_route_kernel<T, __half>, a, counters, padded);
}

template <int NT_MOST, int GROUP, bool ZEROS>
cudaError_t launch_expert_kernel(const cudaLaunchConfig_t& config, const MoeArgs& a, const Stack& gate,
                                 const Stack& down, const MoePlan& plan) {
    constexpr auto kernel = moe_expert_kernel<NT_MOST, GROUP, ZEROS>;
    const cudaError_t err = set_smem_limit_once<kernel>(SMEM_LIMIT - 2048);
    if (err != cudaSuccess) return err;
    count_launch();
    return cudaLaunchKernelEx(&config, kernel, a, gate, down, plan);
}

// The stacks' group size and zero points are known to the kernel where they are the same.
template <int NT_MOST>
cudaError_t launch_experts(const cudaLaunchConfig_t& config, const MoeArgs& a, const Stack& gate,
                           const Stack& down, const MoePlan& plan) {
    if (gate.geom.group != down.geom.group || gate.geom.zeros != down.geom.zeros)
        return launch_expert_kernel<NT_MOST, 0, false>(config, a, gate, down, plan);
    switch (gate.geom.group + gate.geom.zeros) {
        case 32: return launch_expert_kernel<NT_MOST, 32, false>(config, a, gate, down, plan);
        case 33: return launch_expert_kernel<NT_MOST, 32, true>(config, a, gate, down, plan);
        case 64: return launch_expert_kernel<NT_MOST, 64, false>(config, a, gate, down, plan);
        case 65: return launch_expert_kernel<NT_MOST, 64, true>(config, a, gate, down, plan);
        case 128: return launch_expert_kernel<NT_MOST, 128, false>(config, a, gate, down, plan);
        default: return launch_expert_kernel<NT_MOST, 128, true>(config, a, gate, down, plan);
    }
}

// How many warps split n, so that the CTAs are done first with `tiles` times `sets` pieces of
// work of `units` chunk sets each; an item costs some sets besides.
int choose_split(double tiles, int sets, int units, int ctas) {
    constexpr double FIXED = 2.0;
    double best_cost = 1e30;
    int best = 1;
    for (int wn = 1; wn <= WARPS; wn *= 2) {
        if (wn > 1 && wn > units) break;
        const int groups = (sets + WARPS / wn - 1) / (WARPS / wn);
        const double rounds = std::ceil(tiles * groups / ctas);
        const double cost = rounds * ((units + wn - 1) / wn + FIXED + 0.125 * wn);
        if (cost < best_cost) {
            best_cost = cost;
            best = wn;
        }
    }
    return best;
}

// Whether tiles are of two tokens at most, all of whose pieces have columns of their own. Larger
// ones save reading an expert's weights again, from L2, but take two matrix instructions or three
// where these take one. 8 of 64 experts of 4096 x 2048, bfloat16: 3, 8, 16, 24 and 32 tokens take 87,
// 141, 218, 264 and 344 us with small tiles, 110, 183, 232, 273 and 292 with large ones.
bool small_tiles(const sgemm_moe_layer& m, int T) { return T <= 2 || T * m.top_k <= 3 * m.E; }

MoePlan make_plan(const sgemm_moe_layer& m, const Q4Geom& g, const Q4Geom& gd, int T, int sm_count) {
    MoePlan p;
    const int slots = T * m.top_k;
    p.x_pieces = pieces_of(m.dtype);
    p.capacity = small_tiles(m, T) ? (T < 2 ? T : 2) : TILE;
    const int chunk1 = q4_chunk_bytes(g.group, g.zeros), chunk2 = q4_chunk_bytes(gd.group, gd.zeros);
    p.chunk = chunk1 > chunk2 ? chunk1 : chunk2;
    p.smem = moe_offsets(p.chunk, most_tiles(m.E, slots, p.capacity), slots, m.E).end;
    p.sets1 = (m.F + 31) / 32;
    p.sets2 = (m.D + 63) / 64;
    // tiles, about, if tokens picked experts at random
    double missed = 1.0;
    for (int t = 0; t < T; ++t) missed *= 1.0 - double(m.top_k) / m.E;
    double tiles = m.E * (1.0 - missed);
    if (tiles < double(slots) / p.capacity) tiles = double(slots) / p.capacity;
    const int ctas = 2 * sm_count;
    p.wn1 = choose_split(tiles, p.sets1, g.units, ctas);
    p.wn2 = choose_split(tiles, p.sets2, gd.units, ctas);
    p.step1 = p.wn1 * g.unit_bytes;
    p.step2 = p.wn2 * gd.unit_bytes;
    p.gate_to_up = static_cast<const uint8_t*>(m.up.data) - static_cast<const uint8_t*>(m.gate.data);
    return p;
}

bool stack_fits(const sgemm_q4& w, int E, int N, int K) {
    return q4_valid(&w) && w.data && aligned16(w.data) && w.count == E && w.N == N && w.K == K;
}

}  // namespace
}  // namespace sgemm

using namespace sgemm;

extern "C" int sgemm_moe(const sgemm_moe_layer* layer, const void* x, long long ldx, int T,
                         const unsigned char* live, void* y, long long ldy, int* ids,
                         float* weights, void* stream) {
    if (!layer || !layer->router || !dtype_valid(layer->dtype) || !dtype_valid(layer->router_dtype))
        return SGEMM_ERR_ARG;
    const sgemm_moe_layer& m = *layer;
    if (m.D < 1 || m.D > kMoeMaxDim || m.F < 1 || m.F > kMoeMaxDim || m.E < 1 || m.E > kMoeMaxE ||
        m.top_k < 1 || m.top_k > kMoeMaxTop || m.top_k > m.E)
        return SGEMM_ERR_ARG;
    if (!stack_fits(m.gate, m.E, m.D, m.F) || !stack_fits(m.up, m.E, m.D, m.F) ||
        !stack_fits(m.down, m.E, m.F, m.D) || m.gate.group != m.up.group ||
        m.gate.flags != m.up.flags)
        return SGEMM_ERR_ARG;
    if (T < 0 || T > kMoeMaxT || ldx < m.D || ldy < m.D || ldx > (1ll << 40) || ldy > (1ll << 40))
        return SGEMM_ERR_ARG;
    if (T == 0) return SGEMM_OK;
    if (!x || !y) return SGEMM_ERR_ARG;
    const size_t size = dtype_bytes(m.dtype), side = size_t(T) * m.top_k * 4;
    const size_t router_size = dtype_bytes(m.router_dtype);
    const struct { const void* p; size_t bytes; } outs[3] = {
        {y, (size_t(T - 1) * ldy + m.D) * size}, {ids, ids ? side : 0}, {weights, weights ? side : 0}};
    const struct { const void* p; size_t bytes; } ins[6] = {
        {x, (size_t(T - 1) * ldx + m.D) * size},
        {m.router, size_t(m.E) * m.D * router_size},
        {live, live ? size_t(T) : 0},
        {m.gate.data, q4_bytes(m.gate)}, {m.up.data, q4_bytes(m.up)}, {m.down.data, q4_bytes(m.down)}};
    for (int i = 0; i < 3; ++i) {
        if (!outs[i].bytes) continue;
        for (const auto& in : ins)
            if (in.bytes && ranges_overlap(outs[i].p, outs[i].bytes, in.p, in.bytes))
                return SGEMM_ERR_OVERLAP;
        for (int j = 0; j < i; ++j)
            if (outs[j].bytes && ranges_overlap(outs[i].p, outs[i].bytes, outs[j].p, outs[j].bytes))
                return SGEMM_ERR_OVERLAP;
    }
    if (!aligned_to(x, size) || !aligned_to(y, size) || !aligned_to(m.router, router_size) ||
        !aligned_to(ids, 4) || !aligned_to(weights, 4))
        return SGEMM_ERR_ARG;
    int dev = -1;
    const DeviceInfo* info = current_device(&dev);
    if (!info) return SGEMM_ERR_NO_DEVICE;
    const Q4Geom g = q4_geom(m.gate), gd = q4_geom(m.down);
    const int slots = T * m.top_k;
    const MoePlan plan = make_plan(m, g, gd, T, info->sm_count);

    const int x_padded = g.units * kQ4UnitN, h_padded = gd.units * kQ4UnitN;
    const int counters = 3 + plan.sets2;
    size_t bytes = 0;
    auto take = [&](size_t n) {
        const size_t at = bytes;
        bytes += (n + 255) / 256 * 256;
        return at;
    };
    const size_t at_xp = take(size_t(T) * plan.x_pieces * x_padded * 4);
    const size_t at_hp = take(size_t(slots) * H_PIECES * h_padded * 4);
    const size_t at_xs = take(size_t(T) * 4), at_hs = take(size_t(slots) * 4);
    const size_t at_counters = take(size_t(counters) * 4);
    const size_t at_z = take(size_t(slots) * m.D * 4);
    const size_t at_xsum = take(size_t(T) * plan.x_pieces * (x_padded / 32) * 4);
    const size_t at_hsum = take(size_t(slots) * H_PIECES * (h_padded / 32) * 4);
    const size_t at_xback = take(size_t(T) * (x_padded / 32) * 4);
    const size_t at_hback = take(size_t(slots) * (h_padded / 32) * 4);
    const size_t at_ids = take(ids ? 0 : side), at_weights = take(weights ? 0 : side);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    Scratch ws;
    if (ws.alloc(dev, bytes, s) != cudaSuccess) return SGEMM_ERR_CUDA;
    uint8_t* base = static_cast<uint8_t*>(ws.ptr);

    MoeArgs a;
    a.x = x;
    a.ldx = size_t(ldx);
    a.router = m.router;
    a.router_dtype = m.router_dtype;
    a.dtype = m.dtype;
    a.T = T;
    a.D = m.D;
    a.F = m.F;
    a.E = m.E;
    a.top = m.top_k;
    a.renormalize = m.renormalize;
    a.live = live;
    a.ids = ids ? ids : reinterpret_cast<int*>(base + at_ids);
    a.weights = weights ? weights : reinterpret_cast<float*>(base + at_weights);
    a.y = y;
    a.ldy = size_t(ldy);
    a.vec = aligned16(x) && size_t(ldx) * size % 16 == 0 && aligned16(m.router) &&
            size_t(m.D) * router_size % 16 == 0;
    a.xp = reinterpret_cast<uint16_t*>(base + at_xp);
    a.hp = reinterpret_cast<uint16_t*>(base + at_hp);
    a.x_sum = reinterpret_cast<float*>(base + at_xsum);
    a.h_sum = reinterpret_cast<float*>(base + at_hsum);
    a.x_back = reinterpret_cast<float*>(base + at_xback);
    a.h_back = reinterpret_cast<float*>(base + at_hback);
    a.x_factor = g.zeros ? -1.0f : -8.0f;
    a.h_factor = gd.zeros ? -1.0f : -8.0f;
    a.x_form = size_t(T) * plan.x_pieces * x_padded;
    a.h_form = size_t(slots) * H_PIECES * h_padded;
    a.x_special = reinterpret_cast<int*>(base + at_xs);
    a.h_special = reinterpret_cast<int*>(base + at_hs);
    a.counters = reinterpret_cast<int*>(base + at_counters);
    a.z = reinterpret_cast<float*>(base + at_z);
    a.err = info->error_word;

    cudaLaunchAttribute attrs[2];
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = ROUTE_CTAS;
    attrs[1].val.clusterDim.y = 1;
    attrs[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t config = {};
    config.stream = s;
    config.attrs = attrs;
    config.gridDim = dim3(ROUTE_CTAS, T);
    config.blockDim = dim3(ROUTE_THREADS);
    config.numAttrs = 2;
    cudaError_t err = m.dtype == SGEMM_FLOAT32    ? launch_route<float>(config, a, counters, x_padded)
                      : m.dtype == SGEMM_BFLOAT16 ? launch_route<__nv_bfloat16>(config, a, counters, x_padded)
                                                  : launch_route<__half>(config, a, counters, x_padded);
    if (err != cudaSuccess) return SGEMM_ERR_CUDA;
    count_launch();
    config.gridDim = dim3(2 * info->sm_count);
    config.blockDim = dim3(THREADS);
    config.dynamicSmemBytes = plan.smem;
    config.numAttrs = 1;
    const Stack gate{static_cast<const uint8_t*>(m.gate.data), g};
    const Stack down{static_cast<const uint8_t*>(m.down.data), gd};
    if (small_tiles(m, T))
        err = launch_experts<1>(config, a, gate, down, plan);
    else
        err = launch_experts<2>(config, a, gate, down, plan);
    return err == cudaSuccess ? SGEMM_OK : SGEMM_ERR_CUDA;
}
