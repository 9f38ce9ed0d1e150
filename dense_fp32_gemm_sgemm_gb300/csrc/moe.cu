// A mixture-of-experts layer for a few tokens (definition in sgemm.h), in two kernels. The cost is
// reading the weights of the experts that some token picked, once.
//
// moe_route_kernel: a cluster of 8 CTAs a token shares the router's rows, writes the token as
// bfloat16 pieces, and its first CTA chooses the experts.
//
// moe_expert_kernel: every CTA builds the same lists of the picked experts' tokens, cut into tiles
// of so many tokens that an expert's weights are read once for each tile. Then the CTAs take work
// items in order from a counter:
//   first items: one tile x 16 hidden values: the strips of gate and up, n = D split over the
//     CTA's warps; h = silu(g) u times the token's weight goes to scratch as bfloat16 pieces;
//   then items: 32 columns of the output x a part of the tiles: two strips of down, with the
//     (tile, n = F) chunks of all the part's experts dealt out to the warps in turn. Each warp
//     adds its sums to a slab of its own, [token][32], and the slabs are added in warp order; the
//     last part of a column block to finish adds the parts in their order.
// An item of the second kind needs all of the first kind. Those have been taken before it, by CTAs
// that are running and wait for nothing, so its wait ends whatever the number of CTAs that are
// resident. Meanwhile each warp's ring of cp.async stages already fills with the item's weights:
// HBM stays busy across items and across the wait.
//
// The inner product is that of q4_warp.cuh, on chunk pairs (gate and up, or two strips of down), so
// that a column's words serve two strips. The sums of x that zero points take come from one more
// matrix instruction on a constant operand (z's place taken by 8, or by 1 and multiplied by z
// afterwards): hidden values of a group come from several CTAs, so they cannot be summed beforehand.
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
constexpr int ROUTE_THREADS = 256;

constexpr int DEPTH = 4;        // stages of a warp's ring, a pair of chunks each
constexpr int MAX_WARPS = 16;
constexpr int MAX_PARTS = 16;
constexpr int SMEM_SM = 228 * 1024;
constexpr int SMEM_LIMIT = 227 * 1024;

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
    uint16_t* xp;      // pieces of x as bfloat16: [token][piece][D padded to units]
    uint16_t* hp;      // pieces of the hidden values: [token and slot][piece][F padded]
    int* x_special;    // [token]: nonzero where the plain form cannot take some value
    int* h_special;    // [token and slot]
    int* counters;     // 0: next item, 1: finished first items, 2 ..: parts done of a column block
    float* parts;      // [part][token][D]
    int* err;
};

struct Stack {
    const uint8_t* data;
    Q4Geom geom;
};

// How the expert kernel cuts its work.
struct MoePlan {
    int warps;
    int capacity;   // tokens of a tile
    int x_pieces, x_columns;  // pieces of a token of x, and columns that they take
    int h_pieces, h_columns;  // and of a hidden row
    int blocks;     // column blocks of 32 of the output
    int parts;      // at most, of the tiles of a column block
    int chunk, smem;
};

// ---- routing ---------------------------------------------------------------------------

template <class T, class R>
__device__ __forceinline__ float dot(const T* x, const R* w, int D, bool vec, int lane) {
    float s = 0.0f;
    if (vec && D % 8 == 0) {
#pragma unroll 4
        for (int d = lane * 8; d < D; d += 256) {
            const Raw8<T> a = load_raw8(x, d, D, true);
            const Raw8<R> b = load_raw8(w, d, D, true);
            const T* p = reinterpret_cast<const T*>(&a);
            const R* q = reinterpret_cast<const R*>(&b);
#pragma unroll
            for (int i = 0; i < 8; ++i) s = fmaf(float(p[i]), float(q[i]), s);
        }
    } else {
        for (int d = lane; d < D; d += 32) s = fmaf(float(x[d]), float(w[d]), s);
    }
    return s;
}

template <class T>
__device__ __forceinline__ float router_dot(const MoeArgs& a, int t, int e, int lane) {
    const T* x = static_cast<const T*>(a.x) + t * a.ldx;
    const size_t at = size_t(e) * a.D;
    if (a.router_dtype == SGEMM_FLOAT32)
        return dot(x, static_cast<const float*>(a.router) + at, a.D, a.vec, lane);
    if (a.router_dtype == SGEMM_BFLOAT16)
        return dot(x, static_cast<const __nv_bfloat16*>(a.router) + at, a.D, a.vec, lane);
    return dot(x, static_cast<const __half*>(a.router) + at, a.D, a.vec, lane);
}

// This CTA's share of the token's octets as pieces; true where the plain form cannot take one.
template <class T>
__device__ __forceinline__ bool write_pieces(const MoeArgs& a, int t, int rank, int padded) {
    constexpr int P = pieces_of_type<T>();
    const T* x = static_cast<const T*>(a.x) + t * a.ldx;
    Magnitudes magnitudes;
    const int octets = padded / 8;
    for (int u = rank * ROUTE_THREADS + threadIdx.x; u < octets; u += ROUTE_CTAS * ROUTE_THREADS) {
        const Raw8<T> raw = load_raw8(x, u * 8, a.D, a.vec);
        const uint32_t* words = reinterpret_cast<const uint32_t*>(&raw);
#pragma unroll
        for (int i = 0; i < int(sizeof(T)) * 2; ++i) {
            if constexpr (sizeof(T) == 4)
                magnitudes.add(words[i]);
            else
                magnitudes.add2(words[i]);
        }
        uint4 piece[P];
        split_centred<P>(raw, piece);
#pragma unroll
        for (int p = 0; p < P; ++p)
            reinterpret_cast<uint4*>(a.xp + (size_t(t) * P + p) * padded)[u] = piece[p];
    }
    return magnitudes.special<T>();
}

// The top experts of a token's logits (shared memory, one warp) in ascending order, and their
// weights.
__device__ __forceinline__ void choose(const MoeArgs& a, const float* logit, int t, int lane) {
    float biggest = -INFINITY;
    for (int e = lane; e < a.E; e += 32) biggest = fmaxf(biggest, logit[e]);
    for (int o = 16; o > 0; o >>= 1)
        biggest = fmaxf(biggest, __shfl_xor_sync(0xffffffffu, biggest, o));
    // an infinite logit shares the weight with its equals, and so do logits that are all -infinity
    auto power = [&](float l) { return l == biggest ? 1.0f : expf(l - biggest); };
    float sum = 0.0f;
    for (int e = lane; e < a.E; e += 32) sum += power(logit[e]);
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    uint32_t taken = 0;  // bit i: expert lane + 32 i
    float chosen = 0.0f;
    for (int j = 0; j < a.top; ++j) {
        float best = -INFINITY;
        int at = kMoeMaxE;
        for (int i = 0; lane + 32 * i < a.E; ++i) {
            const float l = logit[lane + 32 * i];
            if (!((taken >> i) & 1) && (l > best || at == kMoeMaxE)) {
                best = l;
                at = lane + 32 * i;
            }
        }
        for (int o = 16; o > 0; o >>= 1) {
            const float other = __shfl_xor_sync(0xffffffffu, best, o);
            const int other_at = __shfl_xor_sync(0xffffffffu, at, o);
            if (other_at < kMoeMaxE &&
                (at == kMoeMaxE || other > best || (other == best && other_at < at))) {
                best = other;
                at = other_at;
            }
        }
        if ((at & 31) == lane) taken |= 1u << (at >> 5);
        chosen += power(best);
    }
    int slot = 0;
    for (int i = 0; 32 * i < a.E; ++i) {
        const bool mine = (taken >> i) & 1;
        const uint32_t mask = __ballot_sync(0xffffffffu, mine);
        if (mine) {
            const int at = t * a.top + slot + __popc(mask & ((1u << lane) - 1));
            a.ids[at] = lane + 32 * i;
            a.weights[at] = power(logit[lane + 32 * i]) / (a.renormalize ? chosen : sum);
        }
        slot += __popc(mask);
    }
}

__global__ void __launch_bounds__(ROUTE_THREADS) moe_route_kernel(const MoeArgs a, int counters,
                                                                  int padded) {
    __shared__ float mine[kMoeMaxE / ROUTE_CTAS];
    __shared__ float logit[kMoeMaxE];
    __shared__ float special_s;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = int(ptx::cluster_ctarank()), t = blockIdx.y;
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    if (t == 0)
        for (int i = rank * ROUTE_THREADS + threadIdx.x; i < counters;
             i += ROUTE_CTAS * ROUTE_THREADS)
            a.counters[i] = 0;
    const bool live = !a.live || a.live[t];  // the same in the whole cluster
    bool special = false;
    if (live) {
        for (int i = warp; rank + ROUTE_CTAS * i < a.E; i += ROUTE_THREADS / 32) {
            const int e = rank + ROUTE_CTAS * i;
            float s = a.dtype == SGEMM_FLOAT32    ? router_dot<float>(a, t, e, lane)
                      : a.dtype == SGEMM_BFLOAT16 ? router_dot<__nv_bfloat16>(a, t, e, lane)
                                                  : router_dot<__half>(a, t, e, lane);
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            if (lane == 0) mine[i] = s == s ? s : -INFINITY;
        }
        special = a.dtype == SGEMM_FLOAT32    ? write_pieces<float>(a, t, rank, padded)
                  : a.dtype == SGEMM_BFLOAT16 ? write_pieces<__nv_bfloat16>(a, t, rank, padded)
                                              : write_pieces<__half>(a, t, rank, padded);
    }
    special = __syncthreads_or(special);
    if (threadIdx.x == 0) special_s = special ? 1.0f : 0.0f;
    if (!live) {
        if (rank == 0 && threadIdx.x < a.top) {
            a.ids[t * a.top + threadIdx.x] = -1;
            a.weights[t * a.top + threadIdx.x] = 0.0f;
        }
        return;
    }
    ptx::cluster_sync();
    if (rank == 0) {
        for (int e = threadIdx.x; e < a.E; e += ROUTE_THREADS)
            logit[e] = ptx::ld_shared_cluster_f32(
                ptx::mapa_shared(ptx::smem_u32(mine + e / ROUTE_CTAS), e % ROUTE_CTAS));
        if (threadIdx.x < a.top) a.h_special[t * a.top + threadIdx.x] = 0;
        float any = 0.0f;
        if (threadIdx.x == 0) {
            for (int q = 0; q < ROUTE_CTAS; ++q)
                any += ptx::ld_shared_cluster_f32(ptx::mapa_shared(ptx::smem_u32(&special_s), q));
            a.x_special[t] = any > 0.0f;
        }
        __syncthreads();
    }
    ptx::cluster_sync();  // the others' shared memory has been read
    if (rank == 0 && warp == 0) choose(a, logit, t, lane);
}

// ---- experts -------------------------------------------------------------------------------

// Where the expert kernel's shared memory holds what, in bytes.
struct MoeOffsets {
    int tiles;    // int4 each: expert, first member, members, special
    int members;  // token and slot, by expert
    int sums;     // first items: [warp][gate, up][column][17]; second: [warp][token][32]
    int ring;
    int end;
};
__host__ __device__ constexpr MoeOffsets moe_offsets(int warps, int T, int max_columns, int chunk,
                                                     int tiles, int slots) {
    MoeOffsets o{};
    o.tiles = 0;
    o.members = tiles * 16;
    o.sums = (o.members + slots * 2 + 15) / 16 * 16;
    const int first = warps * 2 * max_columns * 17 * 4, second = warps * T * 32 * 4;
    o.ring = o.sums + (((first > second ? first : second) + 15) / 16) * 16;
    o.end = o.ring + warps * DEPTH * 2 * chunk;
    return o;
}

// Tiles of the picked experts' tokens: an expert has at most two that are not full.
__host__ __device__ constexpr int most_tiles(int E, int slots, int capacity) {
    return slots / capacity + 2 * (E < slots ? E : slots);
}

// One pair of chunks (strips m = 0, 1 at stage and stage + chunk) times NT tiles of 8 columns, added
// to total as in q4_chunk. col[nt]: the lane's column 8 nt + r at the unit, plus 8 c values; its
// pieces are as they are and scaled here. The group size and zero points are the stack's.
template <int NT, bool CENTRED>
__device__ __forceinline__ void chunk_pair(const uint8_t* stage, int chunk, const Q4Geom& geom, int lane,
                                           const uint16_t* const (&col)[NT], float (&total)[2][NT][4]) {
    constexpr int AHEAD = NT == 4 ? 1 : 4;  // blocks whose columns are loaded ahead
    const int r = lane >> 2;
    const int blocks = geom.group / 32, groups = kQ4UnitN / geom.group;
    const __nv_bfloat162 scale = __float2bfloat162_rn(kQ4Scale);
    const __nv_bfloat162 scale16 = __float2bfloat162_rn(kQ4Scale16);
    const uint32_t one = geom.zeros ? 0x00010001u : 0x00080008u;
    const uint32_t ones[4] = {one, one, one << 4, one << 4};
    uint4 x[AHEAD][NT];
    auto load = [&](int b) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            x[b % AHEAD][nt] = *reinterpret_cast<const uint4*>(col[nt] + b * 32);
    };
#pragma unroll
    for (int b = 0; b < AHEAD; ++b) load(b);
    float acc[2][NT][4], sum[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[0][nt][i] = acc[1][nt][i] = sum[nt][i] = 0.0f;
    int left = blocks;  // of the group
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        uint32_t xs[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const uint4 v = x[b % AHEAD][nt];
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                xs[nt][i] = w[i];
                if constexpr (!CENTRED) {
                    const __nv_bfloat162 s = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]),
                                                     (i & 1) ? scale16 : scale);
                    xs[nt][i] = *reinterpret_cast<const uint32_t*>(&s);
                }
            }
        }
        if (AHEAD == 1 && b < 3) load(b + 1);
        const int g = b / blocks;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const uint32_t* codes =
                reinterpret_cast<const uint32_t*>(stage + m * chunk + b * 256) + lane;
            uint32_t lo[4], hi[4];
            if constexpr (CENTRED) {
                uint32_t z0 = 8, z1 = 8;
                if (geom.zeros) {
                    const uint8_t* z = stage + m * chunk + kQ4ChunkCodes + groups * kQ4StripK * 2 +
                                       g * kQ4StripK + r;
                    z0 = z[0];
                    z1 = z[8];
                }
                q4_centred(codes[0], 0x43004300u | z0 * 0x00010001u, lo);
                q4_centred(codes[32], 0x43004300u | z1 * 0x00010001u, hi);
            } else {
                q4_plain(codes[0], lo);
                q4_plain(codes[32], hi);
            }
            const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]};
            const uint32_t a1[4] = {lo[2], hi[2], lo[3], hi[3]};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                mma_bf16(acc[m][nt], a0, xs[nt][0], xs[nt][1]);
                mma_bf16(acc[m][nt], a1, xs[nt][2], xs[nt][3]);
            }
        }
        if constexpr (!CENTRED) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                mma_bf16(sum[nt], ones, xs[nt][0], xs[nt][1]);
                mma_bf16(sum[nt], ones, xs[nt][2], xs[nt][3]);
            }
        }
        if (--left > 0) continue;
        left = blocks;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const uint8_t* side = stage + m * chunk + kQ4ChunkCodes;
            const uint16_t* scales = reinterpret_cast<const uint16_t*>(side) + g * kQ4StripK + r;
            const float s0 = q4_scale(scales[0], geom.fp16), s1 = q4_scale(scales[8], geom.fp16);
            float z0 = 1.0f, z1 = 1.0f;
            if (!CENTRED && geom.zeros) {  // 0x4300 | z is the upper half of the float 128 + z
                const uint8_t* z = side + groups * kQ4StripK * 2 + g * kQ4StripK + r;
                z0 = __uint_as_float(0x43000000u | uint32_t(z[0]) << 16) - 128.0f;
                z1 = __uint_as_float(0x43000000u | uint32_t(z[8]) << 16) - 128.0f;
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float s = i < 2 ? s0 : s1, z = i < 2 ? z0 : z1;
                    float v = acc[m][nt][i];
                    // the sums are alike in all rows of the constant operand
                    if constexpr (!CENTRED) v = fmaf(-z, sum[nt][i & 1], v) * kQ4Unscale;
                    total[m][nt][i] = fmaf(s, v, total[m][nt][i]);
                    acc[m][nt][i] = 0.0f;
                }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[nt][i] = 0.0f;
    }
}

// Adds up a warp's columns of a tile, column by column: NT as few as hold `columns`.
template <class Body>
__device__ __forceinline__ void by_tiles(int columns, bool special, Body&& body) {
    if (columns <= 8) {
        if (special)
            body(std::integral_constant<int, 1>(), std::true_type());
        else
            body(std::integral_constant<int, 1>(), std::false_type());
    } else if (columns <= 16) {
        if (special)
            body(std::integral_constant<int, 2>(), std::true_type());
        else
            body(std::integral_constant<int, 2>(), std::false_type());
    } else {
        if (special)
            body(std::integral_constant<int, 4>(), std::true_type());
        else
            body(std::integral_constant<int, 4>(), std::false_type());
    }
}

__global__ void __launch_bounds__(MAX_WARPS * 32, 1)
    moe_expert_kernel(const MoeArgs a, const Stack gate, const Stack up, const Stack down,
                      const MoePlan plan) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int scan_s[MAX_WARPS], tiles_s, item_s[2], last_s;
    __shared__ volatile int abort_s;
    const int warps = plan.warps, threads = warps * 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = lane >> 2, c = lane & 3;
    const int slots = a.T * a.top;
    const int max_tiles = most_tiles(a.E, slots, plan.capacity);
    const int max_columns = plan.capacity * max(plan.x_columns, plan.h_columns);
    const MoeOffsets at = moe_offsets(warps, a.T, max_columns, plan.chunk, max_tiles, slots);
    int4* tile_s = reinterpret_cast<int4*>(smem + at.tiles);
    uint16_t* member_s = reinterpret_cast<uint16_t*>(smem + at.members);
    float* sums = reinterpret_cast<float*>(smem + at.sums);
    uint8_t* ring = smem + at.ring + warp * DEPTH * 2 * plan.chunk;

    if (tid == 0) abort_s = 0;
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();

    // The tokens of each expert, in order, in tiles; the same in every CTA. The slots' experts are
    // put where the sums will be.
    {
        int* id_s = reinterpret_cast<int*>(sums);
        // an expert's number, and beside it whether the token wants the centred form: such tokens
        // have tiles of their own, so that they change nothing for the others
        for (int i = tid; i < slots; i += threads) {
            const int e = a.ids[i];
            id_s[i] = e < 0 ? -1 : 2 * e + (a.x_special[i / a.top] != 0);
        }
        __syncthreads();
        int count = 0, plain = 0;
        if (tid < a.E)
            for (int i = 0; i < slots; ++i) {
                count += id_s[i] >> 1 == tid;
                plain += id_s[i] == 2 * tid;
            }
        const int plain_tiles = (plain + plan.capacity - 1) / plan.capacity;
        const int my_tiles = plain_tiles + (count - plain + plan.capacity - 1) / plan.capacity;
        // tiles and members before this expert's: a scan over the threads
        int scan = my_tiles << 16 | count;
        for (int o = 1; o < 32; o *= 2) {
            const int v = __shfl_up_sync(0xffffffffu, scan, o);
            if (lane >= o) scan += v;
        }
        if (lane == 31) scan_s[warp] = scan;
        __syncthreads();
        int before = scan - (my_tiles << 16 | count);
        for (int w = 0; w < warp; ++w) before += scan_s[w];
        const int first_tile = before >> 16, first = before & 0xffff;
        if (tid < a.E && count > 0) {
            int n = first, special = first + plain;
            for (int i = 0; i < slots; ++i)
                if (id_s[i] >> 1 == tid) member_s[(id_s[i] & 1) ? special++ : n++] = uint16_t(i);
            for (int k = 0; k < my_tiles; ++k) {
                const bool centred = k >= plain_tiles;
                const int from = (centred ? k - plain_tiles : k) * plan.capacity;
                int4 tile;
                tile.x = tid;
                tile.y = first + (centred ? plain : 0) + from;
                tile.z = min(plan.capacity, (centred ? count - plain : plain) - from);
                tile.w = centred;
                tile_s[first_tile + k] = tile;
            }
        }
        if (tid == threads - 1) tiles_s = (before + (my_tiles << 16 | count)) >> 16;
        if (tid == 0) {
            item_s[0] = atomicAdd(a.counters, 1);
            item_s[1] = atomicAdd(a.counters, 1);
        }
        __syncthreads();
    }
    const int tiles = tiles_s;
    const int strips = (a.F + kQ4StripK - 1) / kQ4StripK;
    const int parts = max(1, min(plan.parts, tiles));
    const int first_items = tiles * strips, items = first_items + plan.blocks * parts;
    const int x_padded = gate.geom.units * kQ4UnitN, h_padded = down.geom.units * kQ4UnitN;

    // Where an item's chunks are: first items: strip `strip` of gate and up of the tile's expert,
    // units warp, warp + warps, ...; second items: strips 2 block and + 1 of down, tiles from .. to,
    // (tile, unit) pairs warp, warp + warps, ... of them.
    struct Walk {
        int kind;  // 0, 1; 2: nothing
        int tile, to, unit, strip;
    };
    auto walk = [&](int item) {
        Walk w;
        if (item < first_items) {
            w.kind = 0;
            w.tile = item / strips;
            w.strip = item - w.tile * strips;
            w.to = w.tile + 1;
            w.unit = warp;
        } else if (item < items) {
            const int i = item - first_items, block = i / parts, part = i - block * parts;
            w.kind = 1;
            w.strip = 2 * block;
            w.tile = part * tiles / parts;
            w.to = (part + 1) * tiles / parts;
            w.unit = warp;
            while (w.unit >= down.geom.units && w.tile < w.to) {
                w.unit -= down.geom.units;
                ++w.tile;
            }
        } else {
            w.kind = 2;
            w.tile = w.to = w.unit = w.strip = 0;
        }
        return w;
    };
    auto done = [&](const Walk& w) {
        return w.kind == 0 ? w.unit >= gate.geom.units : w.tile >= w.to;
    };
    auto advance = [&](Walk& w) {
        w.unit += warps;
        if (w.kind == 1)
            while (w.unit >= down.geom.units && w.tile < w.to) {
                w.unit -= down.geom.units;
                ++w.tile;
            }
    };

    const uint32_t ring_u32 = ptx::smem_u32(ring);
    uint32_t fetch_to = ring_u32;
    const int stage_bytes = 2 * plan.chunk;
    // what a lane copies besides codes, for the gate and up stacks and for down
    auto side_of = [&](const Q4Geom& g) {
        const int groups = kQ4UnitN / g.group;
        Q4Side s;
        const bool zero = lane >= 2 * groups;
        s.step = zero ? kQ4StripK : kQ4StripK * 2;
        s.from = kQ4CodeBytes + (zero ? groups * kQ4UnitK * 2 + (lane - 2 * groups) * kQ4UnitK
                                      : (lane >> 1) * kQ4UnitK * 2 + (lane & 1) * 16);
        s.any = lane < (2 + g.zeros) * groups;
        return s;
    };
    const Q4Side side1 = side_of(gate.geom), side2 = side_of(down.geom);
    int next_item = item_s[1];
    Walk f = walk(item_s[0]);
    int f_on = 0;   // the walk is in the current item (0), the next (1) or through both (2)
    int ahead = 0;  // stages fetched and not used up
    auto fetch = [&]() -> bool {
        while (f_on < 2 && done(f))
            if (++f_on == 1) f = walk(next_item);
        if (f_on == 2) return false;
        const int e = tile_s[f.tile].x, in_tile = f.strip % kQ4StripsOfTile;
        if (f.kind == 0) {
            const size_t from = e * gate.geom.matrix_bytes() +
                                size_t(f.strip / kQ4StripsOfTile) * gate.geom.tile_bytes() +
                                size_t(f.unit) * gate.geom.unit_bytes;
            q4_fetch<1>(fetch_to, plan.chunk, gate.data + from, in_tile, 1, lane, side1);
            q4_fetch<1>(fetch_to + plan.chunk, plan.chunk, up.data + from, in_tile, 1, lane, side1);
        } else {
            const size_t from = e * down.geom.matrix_bytes() +
                                size_t(f.strip / kQ4StripsOfTile) * down.geom.tile_bytes() +
                                size_t(f.unit) * down.geom.unit_bytes;
            q4_fetch<2>(fetch_to, plan.chunk, down.data + from, in_tile, 2, lane, side2);
        }
        ptx::cp_async_commit();
        advance(f);
        ++ahead;
        fetch_to += stage_bytes;
        if (fetch_to == ring_u32 + DEPTH * stage_bytes) fetch_to = ring_u32;
        return true;
    };
    // Waits for the oldest stage and fills up the ring again; the stage used before it is free.
    auto acquire = [&]() {
        if (ahead == 0) fetch();
        switch (ahead) {
            case 1: ptx::cp_async_wait<0>(); break;
            case 2: ptx::cp_async_wait<1>(); break;
            case 3: ptx::cp_async_wait<2>(); break;
            default: ptx::cp_async_wait<DEPTH - 1>(); break;
        }
        __syncwarp();
        while (ahead < DEPTH && fetch()) {
        }
    };
    while (ahead < DEPTH && fetch()) {
    }
    const uint8_t* stage = ring;
    auto release = [&]() {
        --ahead;
        stage += stage_bytes;
        if (stage == ring + DEPTH * stage_bytes) stage = ring;
    };

    bool hidden_ready = false;
    int item = item_s[0];
    while (item < items) {
        __syncthreads();  // the sums and item_s are free again
        int claimed = 0;  // the item after the next
        if (tid == 0) claimed = atomicAdd(a.counters, 1);
        Walk w = walk(item);
        if (w.kind == 0) {
            const int4 tile = tile_s[w.tile];
            const int columns = tile.z * plan.x_columns;
            by_tiles(columns, tile.w != 0, [&](auto nt_, auto centred) {
                constexpr int NT = decltype(nt_)::value;
                constexpr bool CENTRED = decltype(centred)::value;
                // columns that do not exist repeat the first, and their sums are not used
                const uint16_t* col[NT];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const int j = nt * 8 + r, m = j / plan.x_columns, p = j - m * plan.x_columns;
                    const bool is = m < tile.z && p < plan.x_pieces;
                    const int token = member_s[tile.y + (is ? m : 0)] / a.top;
                    col[nt] = a.xp + (size_t(token) * plan.x_pieces + (is ? p : 0)) * x_padded + c * 8;
                }
                float total[2][NT][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) total[0][nt][i] = total[1][nt][i] = 0.0f;
#pragma unroll 1
                for (; !done(w); advance(w)) {
                    acquire();
                    const uint16_t* here[NT];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) here[nt] = col[nt] + w.unit * kQ4UnitN;
                    chunk_pair<NT, CENTRED>(stage, plan.chunk, gate.geom, lane, here, total);
                    release();
                }
                float* mine = sums + warp * 2 * max_columns * 17 + r;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int j = nt * 8 + 2 * c + i;
                        if (j < columns)
#pragma unroll
                            for (int m = 0; m < 2; ++m) {
                                mine[(m * max_columns + j) * 17] = total[m][nt][i];
                                mine[(m * max_columns + j) * 17 + 8] = total[m][nt][i + 2];
                            }
                    }
            });
            __syncthreads();
            for (int i = tid; i < tile.z * kQ4StripK; i += threads) {
                const int m = i / kQ4StripK, k = i % kQ4StripK, f_at = w.strip * kQ4StripK + k;
                float g = 0.0f, u = 0.0f;
                for (int p = 0; p < plan.x_pieces; ++p) {
                    const float* from = sums + (m * plan.x_columns + p) * 17 + k;
                    for (int q = 0; q < warps; ++q) {
                        g += from[q * 2 * max_columns * 17];
                        u += from[(q * 2 + 1) * max_columns * 17];
                    }
                }
                const int slot = member_s[tile.y + m];
                const float h =
                    f_at < a.F ? g / (1.0f + expf(-g)) * u * a.weights[slot] : 0.0f;
                float piece[3];
                split_pieces<3>(h, piece);
                if (plan.h_pieces == 2 && fabsf(h) < 1e38f) {
                    // the second piece rounded to nearest: 2^-16 of the value at most
                    piece[1] = __bfloat162float(__float2bfloat16_rn(h - piece[0]));
                }
                Magnitudes magnitude;
                magnitude.add(__float_as_uint(h));
                if (magnitude.special<float>()) atomicOr(a.h_special + slot, 1);
                for (int p = 0; p < plan.h_pieces; ++p)
                    a.hp[(size_t(slot) * plan.h_pieces + p) * h_padded + f_at] =
                        uint16_t(__float_as_uint(piece[p]) >> 16);
            }
            // past F: down's weights are zero there, but not whatever the scratch holds
            if (w.strip == strips - 1) {
                const int from = strips * kQ4StripK, width = h_padded - from;
                for (int i = tid; i < tile.z * plan.h_pieces * width; i += threads) {
                    const int row = i / width, m = row / plan.h_pieces;
                    a.hp[(size_t(member_s[tile.y + m]) * plan.h_pieces + row % plan.h_pieces) *
                             h_padded +
                         from + i % width] = 0;
                }
            }
            __syncthreads();
            if (tid == 0) ptx::red_release_gpu_add(a.counters + 1, 1);
        } else {
            if (!hidden_ready) {
                // bounded; when it gives up, the rest is computed from what the scratch holds
                if (tid == 0) {
                    const unsigned long long t0 = ptx::globaltimer_ns();
                    while (ptx::ld_acquire_gpu(a.counters + 1) < first_items && !abort_s)
                        if (ptx::globaltimer_ns() - t0 > WAIT_LIMIT_NS) {
                            abort_s = 1;
                            atomicExch(a.err, kErrWaitTimeout);
                        }
                }
                __syncthreads();
                __threadfence();
                hidden_ready = true;
            }
            float* slab = sums + warp * a.T * 32;
            for (int i = lane; i < a.T * 32; i += 32) slab[i] = 0.0f;
            __syncwarp();
            while (!done(w)) {
                const int4 tile = tile_s[w.tile];
                const int columns = tile.z * plan.h_columns;
                int special = 0;
                for (int i = lane; i < tile.z; i += 32) special |= a.h_special[member_s[tile.y + i]];
                special = __any_sync(0xffffffffu, special);
                by_tiles(columns, special != 0, [&](auto nt_, auto centred) {
                    constexpr int NT = decltype(nt_)::value;
                    constexpr bool CENTRED = decltype(centred)::value;
                    const uint16_t* col[NT];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const int j = nt * 8 + r, m = j / plan.h_columns, p = j - m * plan.h_columns;
                        const bool is = m < tile.z && p < plan.h_pieces;
                        const int slot = member_s[tile.y + (is ? m : 0)];
                        col[nt] =
                            a.hp + (size_t(slot) * plan.h_pieces + (is ? p : 0)) * h_padded + c * 8;
                    }
                    float total[2][NT][4];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 4; ++i) total[0][nt][i] = total[1][nt][i] = 0.0f;
                    const int this_tile = w.tile;
#pragma unroll 1
                    for (; !done(w) && w.tile == this_tile; advance(w)) {
                        acquire();
                        const uint16_t* here[NT];
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) here[nt] = col[nt] + w.unit * kQ4UnitN;
                        chunk_pair<NT, CENTRED>(stage, plan.chunk, down.geom, lane, here, total);
                        release();
                    }
                    // a token's pieces: two columns of this lane, or these and the first of the
                    // next lane's
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const int j = nt * 8 + 2 * c, m = j / plan.h_columns;
                        const int token = m < tile.z ? member_s[tile.y + m] / a.top : 0;
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int i = 0; i < 4; i += 2) {
                                float v = total[h][nt][i] + total[h][nt][i + 1];
                                if (plan.h_columns == 4) {
                                    const float third =
                                        __shfl_down_sync(0xffffffffu, total[h][nt][i], 1);
                                    v += third;
                                    if (c & 1) continue;
                                }
                                if (m < tile.z) slab[token * 32 + h * 16 + r + 4 * i] += v;
                            }
                    }
                    __syncwarp();
                });
            }
            __syncthreads();
            const int i2 = item - first_items, block = i2 / parts, part = i2 - block * parts;
            auto put = [&](int t, int d, float v) {
                if (d < a.D) store_from_float(a.y, a.dtype, t * a.ldy + d, v);
            };
            for (int i = tid; i < a.T * 32; i += threads) {
                float v = 0.0f;
                for (int q = 0; q < warps; ++q) v += sums[q * a.T * 32 + i];
                const int t = i / 32, d = block * 32 + i % 32;
                if (parts == 1)
                    put(t, d, v);
                else if (d < a.D)
                    a.parts[(size_t(part) * a.T + t) * a.D + d] = v;
            }
            if (parts > 1) {
                __syncthreads();
                if (tid == 0) {
                    __threadfence();
                    last_s = atomicAdd(a.counters + 2 + block, 1) == parts - 1;
                    __threadfence();
                }
                __syncthreads();
                if (last_s)
                    for (int i = tid; i < a.T * 32; i += threads) {
                        const int t = i / 32, d = block * 32 + i % 32;
                        if (d >= a.D) continue;
                        float v = 0.0f;
                        for (int q = 0; q < parts; ++q)
                            v += __ldcg(a.parts + (size_t(q) * a.T + t) * a.D + d);
                        put(t, d, v);
                    }
            }
        }
        if (tid == 0) item_s[0] = claimed;
        __syncthreads();
        item = next_item;
        next_item = item_s[0];
        if (f_on == 0)  // the walk is through the item that was
            f = walk(item);
        else if (--f_on == 1)  // and through the one that is
            f = walk(next_item);
    }
    ptx::cp_async_wait<0>();
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
    if (set_smem_limit_once<moe_expert_kernel>(SMEM_LIMIT - 2048) != cudaSuccess)
        return SGEMM_ERR_CUDA;

    const Q4Geom g = q4_geom(m.gate), gd = q4_geom(m.down);
    const int slots = T * m.top_k;
    MoePlan plan;
    plan.x_pieces = pieces_of(m.dtype);
    plan.x_columns = m.dtype == SGEMM_FLOAT32 ? 4 : plan.x_pieces;
    // the hidden values: all 24 significant bits for float32, 16 for the 16-bit types
    plan.h_pieces = m.dtype == SGEMM_FLOAT32 ? 3 : 2;
    plan.h_columns = m.dtype == SGEMM_FLOAT32 ? 4 : 2;
    plan.capacity = 32 / plan.h_columns;  // 32 columns at most
    if (plan.capacity > T) plan.capacity = T;
    const int chunk1 = q4_chunk_bytes(g.group, g.zeros), chunk2 = q4_chunk_bytes(gd.group, gd.zeros);
    plan.chunk = chunk1 > chunk2 ? chunk1 : chunk2;
    const int max_columns =
        plan.capacity * (plan.x_columns > plan.h_columns ? plan.x_columns : plan.h_columns);
    const int max_tiles = most_tiles(m.E, slots, plan.capacity);
    // two CTAs of 8 warps on an SM while their slabs leave room for it, else one of 12
    int resident = 2;
    plan.warps = 8;
    plan.smem = moe_offsets(8, T, max_columns, plan.chunk, max_tiles, slots).end;
    if ((plan.smem + 2048) * 2 > SMEM_SM) {
        resident = 1;
        plan.warps = 12;
        plan.smem = moe_offsets(12, T, max_columns, plan.chunk, max_tiles, slots).end;
    }
    const int ctas = info->sm_count * resident;
    plan.blocks = (m.D + 31) / 32;
    plan.parts = (2 * ctas + plan.blocks - 1) / plan.blocks;
    if (plan.parts > MAX_PARTS) plan.parts = MAX_PARTS;
    if (plan.parts > max_tiles) plan.parts = max_tiles;

    const int x_padded = g.units * kQ4UnitN, h_padded = gd.units * kQ4UnitN;
    const int counters = 2 + plan.blocks;
    size_t bytes = 0;
    auto take = [&](size_t n) {
        const size_t at = bytes;
        bytes += (n + 255) / 256 * 256;
        return at;
    };
    const size_t at_xp = take(size_t(T) * plan.x_pieces * x_padded * 2);
    const size_t at_hp = take(size_t(slots) * plan.h_pieces * h_padded * 2);
    const size_t at_xs = take(size_t(T) * 4), at_hs = take(size_t(slots) * 4);
    const size_t at_counters = take(size_t(counters) * 4);
    const size_t at_parts = take(plan.parts > 1 ? size_t(plan.parts) * T * m.D * 4 : 0);
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
    a.x_special = reinterpret_cast<int*>(base + at_xs);
    a.h_special = reinterpret_cast<int*>(base + at_hs);
    a.counters = reinterpret_cast<int*>(base + at_counters);
    a.parts = reinterpret_cast<float*>(base + at_parts);
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
    cudaError_t err = cudaLaunchKernelEx(&config, moe_route_kernel, a, counters, x_padded);
    if (err != cudaSuccess) return SGEMM_ERR_CUDA;
    count_launch();
    config.gridDim = dim3(ctas);
    config.blockDim = dim3(plan.warps * 32);
    config.dynamicSmemBytes = plan.smem;
    config.numAttrs = 1;
    const Stack gate{static_cast<const uint8_t*>(m.gate.data), g};
    const Stack up{static_cast<const uint8_t*>(m.up.data), g};
    const Stack down{static_cast<const uint8_t*>(m.down.data), gd};
    err = cudaLaunchKernelEx(&config, moe_expert_kernel, a, gate, up, down, plan);
    count_launch();
    return err == cudaSuccess ? SGEMM_OK : SGEMM_ERR_CUDA;
}
