// Matrix products of 16-bit operands on the tensor cores, with a fused epilogue: the core of
// the cross entropy (cross_entropy.cu) and of the Newton-Schulz products (orthogonalize.cu).
//
// D[M x N] = sum over k of A[m][k] * B[k][n]; either operand may be stored with k or with its
// other index contiguous, as one or more planes (pieces of a longer type) whose products are
// added up in one accumulation. A pair of CTAs computes a tile of 256 x BN with
// tcgen05.mma.cta_group::2; each CTA stages its 128 rows of A and its half of B's columns.
//
// Roles in a CTA: warp 0 issues A's TMA loads, warp 2 B's (a step takes one warp some 450 cycles for
// both, the MMAs 512); in the pair's first CTA warp 1 issues the MMAs and warp 3 hands out units of
// work, each when the loads of the one before begin (when they ended that cost 3 us a unit); warps
// 4-11 run the epilogue.
//
// Accumulation. The tensor core cuts off, rather than rounds, the bits that an addition to its
// FP32 accumulator shifts out, always towards zero. Measured in sums of one sign, FP16 operands: 0.8 ulps of
// the accumulator (an ulp is 2^-23 of it at most) an MMA in sums of 4 MMAs, 1.9 in sums of 32, 2.2 in the worst
// sum; bfloat16 products have fewer bits to lose, 0.3. So n MMAs cost up to n 2^-23 of an evenly growing sum.
// After seg_steps stages (4 MMAs each) the accumulator is therefore added to FP32 registers, rounded to
// nearest, and starts again at zero. The two accumulators of a CTA pair alternate, so the additions overlap
// the next stages' MMAs, and so does the epilogue as far as two segments reach (a stage of 256 columns
// takes 512 cycles): short segments are for results in FP32, long ones let a long epilogue pass unnoticed.
//
// Where two planes share a stage (Ring), the second is what the first leaves of a value, times 2^11: an FP16
// piece of it then is a normal number down to 2^-25 in the first one's scale instead of 2^-14, with steps of
// 2^-35 below. Both products that have a second plane are summed in accumulators of their own, a unit's whole
// reduction in one, and added with 2^-11 to the unit's last segment; what these cut off is 2^-11 of the other's.
//
// Measured: 522 cycles a stage of 256 columns, where the MMAs take 512 and 32 KiB arrive at 62 bytes
// a cycle and SM; the tensor pipe is active 88 to 90 % of the time in products of 2048 x 4096 by 16384
// and at the power cap in larger ones.
//
// Units are claimed from a counter, so that long and short ones may be mixed in a launch. Which
// pair computes a unit does not change what is computed.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.cuh"
#include "ptx.cuh"
#include "wait.cuh"

namespace sgemm {
namespace hg {

constexpr int BM = 256;       // rows of a tile (both CTAs)
constexpr int HALF_M = 128;   // rows of one CTA
constexpr int BK = 64;        // reduction elements in a stage: 128 bytes
constexpr int MAX_STAGES = 6;
constexpr int SLOTS = 4;      // units handed out and not yet taken by all
constexpr int EPI_WARPS = 8;
constexpr int EPI_WARP0 = 4;
constexpr int THREADS = 32 * (EPI_WARP0 + EPI_WARPS);
// Registers: 168 a thread at launch (384 threads); the first warpgroup gives most of its own to
// the epilogue's, whose threads hold 128 sums. 72 + 216 + 216 = 3 * 168.
constexpr int REGS_FEW = 72;
constexpr int REGS_MANY = 216;
constexpr int A_BYTES = HALF_M * BK * 2;
constexpr int CHUNK_BYTES = 64 * BK * 2;  // 64 elements of the other index by 64 of k
constexpr int STAGING = 4096;             // bytes of a staging block
constexpr int NUM_BARS = 2 * MAX_STAGES + 6 + 2 * SLOTS + 2 * EPI_WARPS;
constexpr int MAX_PRODUCTS = 6;
constexpr float SECOND_UP = 0x1p11f, SECOND_DOWN = 0x1p-11f;  // of the second of two planes in a stage

template <int BN>
constexpr int B_BYTES = BN / 2 * BK * 2;
// A stage: 64 k of both operands, of one plane each (then every product has a stage to itself), or
// of both planes of them (a value and 2^11 times what that leaves), which three products share: all but
// the one of the second planes. A stage of one product and 128 columns takes some 430 cycles to wait for,
// issue and hand on where its MMAs take 256, and its 24 KiB 384 to arrive; with two planes three products
// share 48 KiB, a wait and a commit.
template <class EPI>
struct Ring {
    static constexpr int BN = EPI::BN, PLANES = EPI::PLANES;
    static constexpr int B_AT = PLANES * A_BYTES;  // of B in a stage
    static constexpr int STAGE_BYTES = PLANES * (A_BYTES + B_BYTES<BN>);
    static constexpr int STAGES = PLANES == 1 ? 6 : 3;
    // staging blocks of an epilogue warp
    static constexpr int BLOCKS = BN == 256 ? 1 : 2;
    static constexpr int SMEM_BYTES =
        STAGES * STAGE_BYTES + BLOCKS * EPI_WARPS * STAGING + 512 + 1024;
    static_assert(SMEM_BYTES <= 232448, "shared memory of an SM");
    static_assert(STAGES <= MAX_STAGES && (PLANES == 1 || (PLANES == 2 && BN == 128)), "see above");
    // of tensor memory: two accumulators, and with two planes two more
    static constexpr int TMEM_COLUMNS = 2 * PLANES * BN;
};

// One product of a launch. Sizes are in elements; `live` may replace one of them on the device.
struct Problem {
    int M, N, K;
    int batch;          // independent products, the maps' outermost coordinate / planes
    int dyn;            // 0: as given; 1: M, 2: K is the number of live rows
    int splits;         // parts of the reduction, each a unit
    int group;          // tile rows that are worked through column by column
    int symmetric;      // only tiles that reach the diagonal or lie below it (M == N)
    int a_mn, b_mn;     // operand stored with its other index contiguous (else with k)
    int a_row, b_row;   // added to the row coordinate (k or the other index, whichever is a row)
    int planes_a, planes_b;
    int products;       // pairs of planes, smallest products first (1 where a stage holds two planes)
    unsigned char pa[MAX_PRODUCTS], pb[MAX_PRODUCTS];
    unsigned idesc;     // instruction descriptor without N
};

template <int PROBLEMS>
struct Args {
    CUtensorMap a[PROBLEMS], b[PROBLEMS];  // 3-D: contiguous index, row, batch * planes + plane
    Problem p[PROBLEMS];
    int problems;
    const int* live;  // number of rows in all, or null
    int live0;        // rows before this launch's
    int live_max;     // rows of this launch at most
    int* counter;     // claimed units, zero before the launch
    int* err;
    // A chain of products that build on one another: rounds of three problems, the odd rounds with
    // the last three. done[i * batch + e] counts the epilogue warps' finished units of product e of
    // phase i = 3 round + problem, zero before the launch.
    int rounds;
    int* done;
    int seg_steps;  // stages in an accumulator segment
};

// A unit of work.
struct Unit {
    int problem, batch, split;
    int row0, col0;  // of the tile
    int kb0, kb1;    // blocks of the reduction
    int phase;       // of a chain
};

__host__ __device__ inline int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Tiles of a product of `tiles_m` tile rows; with `symmetric` tile row r has the tiles that
// begin at or before its last row.
template <int BN>
__host__ __device__ inline int tile_count(const Problem& p, int tiles_m, int tiles_n) {
    if (!p.symmetric) return tiles_m * tiles_n;
    constexpr int R = BM / BN;
    return R * (tiles_m - 1) * tiles_m / 2 + (tiles_m * R < tiles_n ? tiles_m * R : tiles_n);
}

template <int BN>
__host__ __device__ inline int unit_count(const Problem& p, int live) {
    const int m = p.dyn == 1 ? live : p.M;
    if (m <= 0) return 0;
    return p.batch * p.splits * tile_count<BN>(p, ceil_div(m, BM), ceil_div(p.N, BN));
}

// Units of the launch's problems, and of all together.
struct Units {
    int first, second, third, all;
    template <int BN, bool CHAIN, class ARGS>
    static __device__ __forceinline__ Units of(const ARGS& g, int live) {
        Units n;
        n.first = unit_count<BN>(g.p[0], live);
        n.second = n.third = 0;
        if (CHAIN || g.problems > 1) n.second = unit_count<BN>(g.p[1], live);
        if constexpr (CHAIN) n.third = unit_count<BN>(g.p[2], live);
        n.all = n.first + n.second + n.third;
        if (CHAIN) n.all *= g.rounds;
        return n;
    }
};

// Unit u of the launch; u counts over all its problems.
template <int BN, bool CHAIN, class ARGS>
__device__ inline Unit unit_at(const ARGS& g, const Units& n, int u, int live) {
    Unit t;
    t.problem = 0;
    t.phase = 0;
    if constexpr (CHAIN) {
        const int each = n.first + n.second + n.third;
        const int round = u / each;
        u -= round * each;
        if (u >= n.first) {
            u -= n.first;
            t.problem = 1;
            if (u >= n.second) {
                u -= n.second;
                t.problem = 2;
            }
        }
        t.phase = 3 * round + t.problem;
        t.problem += 3 * (round & 1);
    } else if (u >= n.first) {
        t.problem = 1;
        u -= n.first;
    }
    const Problem& p = g.p[t.problem];
    const int tiles_m = ceil_div(p.dyn == 1 ? live : p.M, BM), tiles_n = ceil_div(p.N, BN);
    const int tiles = tile_count<BN>(p, tiles_m, tiles_n);
    const int each = tiles * p.splits;
    t.batch = u / each;
    u -= t.batch * each;
    t.split = u / tiles;
    u -= t.split * tiles;
    int tm, tn;
    if (p.symmetric) {
        constexpr int R = BM / BN;
        tm = 0;
        while (tm + 1 < tiles_m && u >= (tm + 1) * R) u -= ++tm * R;
        tn = u;
    } else {
        const int grouped = p.group * tiles_n;
        const int gi = u / grouped;
        const int rows = min(p.group, tiles_m - gi * p.group);
        u -= gi * grouped;
        tm = gi * p.group + u % rows;
        tn = u / rows;
    }
    t.row0 = tm * BM;
    t.col0 = tn * BN;
    const int kblocks = ceil_div(p.dyn == 2 ? live : p.K, BK);
    const int each_k = ceil_div(kblocks, p.splits);
    t.kb0 = min(t.split * each_k, kblocks);
    t.kb1 = min(t.kb0 + each_k, kblocks);
    return t;
}

// Instruction descriptor of kind::f16 without its N: FP32 accumulator, M = 256, operand types
// FP16 (0) or bfloat16 (1), and the operands' major indices.
inline unsigned instruction(bool bf16, bool a_mn, bool b_mn) {
    const unsigned type = bf16 ? 1u : 0u;
    return (1u << 4) | (type << 7) | (type << 10) | (unsigned(a_mn) << 15) |
           (unsigned(b_mn) << 16) | (unsigned(BM >> 4) << 24);
}

// ---- shared memory --------------------------------------------------------------------
// The same offsets in both CTAs. full, acc_empty, slot_empty, drain: used in the first CTA.
struct Smem {
    uint32_t ring, bar0, slots;
    uint8_t* staging;
    volatile int* slot_ptr;
    uint32_t* tmem_slot;
    volatile int* abort_flag;
    __device__ uint32_t at(int i) const { return bar0 + 8u * i; }
    __device__ uint32_t full(int s) const { return at(s); }
    __device__ uint32_t empty(int s) const { return at(MAX_STAGES + s); }
    __device__ uint32_t acc_full(int b) const { return at(2 * MAX_STAGES + b); }
    __device__ uint32_t acc_empty(int b) const { return at(2 * MAX_STAGES + 2 + b); }
    __device__ uint32_t slot_full(int i) const { return at(2 * MAX_STAGES + 4 + i); }
    __device__ uint32_t slot_empty(int i) const { return at(2 * MAX_STAGES + 4 + SLOTS + i); }
    __device__ uint32_t drain() const { return at(2 * MAX_STAGES + 4 + 2 * SLOTS); }
    __device__ uint32_t claim() const { return at(2 * MAX_STAGES + 5 + 2 * SLOTS); }
    __device__ uint32_t loaded(int i) const { return at(2 * MAX_STAGES + 6 + 2 * SLOTS + i); }
};

template <class R>
__device__ __forceinline__ Smem carve(uint8_t* raw) {
    uint8_t* base =
        reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    Smem s;
    s.ring = ptx::smem_u32(base);
    s.staging = base + R::STAGES * R::STAGE_BYTES;
    uint64_t* bars = reinterpret_cast<uint64_t*>(s.staging + R::BLOCKS * EPI_WARPS * STAGING);
    s.bar0 = ptx::smem_u32(bars);
    int* words = reinterpret_cast<int*>(bars + NUM_BARS);
    s.slots = ptx::smem_u32(words);
    s.slot_ptr = words;
    s.tmem_slot = reinterpret_cast<uint32_t*>(words + SLOTS);
    s.abort_flag = words + SLOTS + 1;
    return s;
}

__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, const Smem& sm, int* err) {
    return wait_phase(bar, parity, sm.abort_flag, err);
}

// ---- operands in shared memory ----------------------------------------------------------
// k contiguous: rows of 128 bytes (64 k), 8-row groups 1024 bytes apart; 16 k are 32 bytes.
// Other index contiguous: chunks of 64 of it, 8192 bytes apart (the leading offset), each with
// one 128-byte row for every k, 8 k 1024 bytes apart; 16 k are 2048 bytes. Both 128-byte
// swizzled, as TMA writes them.
struct OperandDesc {
    uint32_t lo, hi;  // of the operand in stage 0
    uint32_t step;    // of `lo` to the next 16 k
    __device__ __forceinline__ OperandDesc(uint32_t saddr, bool mn) {
        lo = ((saddr >> 4) & 0x3FFFu) | uint32_t(mn ? CHUNK_BYTES >> 4 : 1) << 16;
        hi = (1024u >> 4) | 1u << 14 | 2u << 29;
        step = mn ? 2048u >> 4 : 32u >> 4;
    }
};

// ---- staging ------------------------------------------------------------------------------
// A staging block holds 32 rows of 128 bytes, 16-byte piece c of row r at c ^ (r % 8), which is
// TMA's 128-byte swizzle: both a lane's own row and four whole rows at a time are free of bank
// conflicts.
__device__ __forceinline__ uint4* staged(uint8_t* block, int row, int piece) {
    return reinterpret_cast<uint4*>(block + row * 128 + ((piece ^ (row & 7)) << 4));
}

// An epilogue warp's staging blocks (one or two) and its TMA traffic through them, which its first
// lane issues. A block is written again once the store that last used it has read it.
template <int BLOCKS>
struct WarpIo {
    uint8_t* blocks;
    uint32_t bar;  // of block 0's loads; block 1's is 8 bytes on
    // the block of the n-th use
    static __device__ __forceinline__ int of(int n) { return n & (BLOCKS - 1); }
    volatile int* abort_flag;
    int* err;
    uint32_t parity = 0;  // bit i: of block i's next load
    int last = 0;         // block of the latest store
    bool first;           // this lane issues
    __device__ __forceinline__ uint8_t* block(int i) const { return blocks + i * STAGING; }
    __device__ __forceinline__ void acquire(int i) {
        if (first) {
            if (BLOCKS == 1 || last == i)
                ptx::bulk_wait_read0();
            else
                ptx::bulk_wait_read<1>();
        }
        __syncwarp();
    }
    // The block's 4096 bytes from a map whose boxes have as many.
    __device__ __forceinline__ void load(int i, const CUtensorMap* map, int x, int y, int z) {
        acquire(i);
        if (first) {
            ptx::mbar_arrive_expect_tx(bar + 8u * i, STAGING);
            ptx::tma_load_3d(ptx::smem_u32(block(i)), map, bar + 8u * i, x, y, z);
        }
    }
    __device__ __forceinline__ void wait_load(int i) {
        wait_phase(bar + 8u * i, parity >> i & 1u, abort_flag, err);
        parity ^= 1u << i;
        __syncwarp();
    }
    // What the lanes wrote to the block goes out.
    __device__ __forceinline__ void store(int i, const CUtensorMap* map, int x, int y, int z) {
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (first) {
            ptx::tma_store_3d(map, ptx::smem_u32(block(i)), x, y, z);
            ptx::bulk_commit();
        }
        last = i;
    }
    __device__ __forceinline__ void finish() {
        if (first) ptx::bulk_wait0();
    }
};

// A lane's row of a staging block from 32 registers.
template <int C, int N>
__device__ __forceinline__ void stage_words(uint8_t* block, const float (&s)[N]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        *staged(block, lane, j) =
            make_uint4(__float_as_uint(s[C + 4 * j]), __float_as_uint(s[C + 4 * j + 1]),
                       __float_as_uint(s[C + 4 * j + 2]), __float_as_uint(s[C + 4 * j + 3]));
}

// Where a block's rows go. The code that follows is kept short: an epilogue passes through it once
// a unit, and instructions that are fetched for one use cost more than they compute.
struct Rows {
    char* base;        // of row 0's first byte
    long long pitch;   // bytes
    int count;         // rows from here on are not written
    int bytes;         // of a row, at most 128
    bool wide;         // 16-byte aligned rows of whole 16-byte pieces; else element by element
};

// Writes the staged block to global memory, 16 bytes a lane and four rows at a time. MAPPED: lane
// l's `index` is the row that row l goes to. SIZE: bytes of an element.
template <int SIZE, bool MAPPED = false>
__device__ __forceinline__ void store_block(uint8_t* block, const Rows& to, int index = 0) {
    const int lane = threadIdx.x & 31;
    __syncwarp();
    if (to.wide) {
        const int piece = lane & 7, r0 = lane >> 3;
        const bool here = piece * 16 < to.bytes;
        char* at = to.base + piece * 16;
        if (!MAPPED) at += r0 * to.pitch;
        const long long step = 4 * to.pitch;
#pragma unroll
        for (int i0 = 0; i0 < 8; i0 += 4) {
            uint4 v[4];  // read before the first store, which the compiler cannot tell apart
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = *staged(block, (i0 + i) * 4 + r0, piece);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = (i0 + i) * 4 + r0;
                char* p = at;
                if (MAPPED) p += __shfl_sync(~0u, index, r) * to.pitch;
                if (here && r < to.count) *reinterpret_cast<uint4*>(p) = v[i];
                if (!MAPPED) at += step;
            }
        }
    } else {
        // four rows in flight, 32 consecutive elements a store
        constexpr int PER = 16 / SIZE, TURNS = SIZE == 4 ? 1 : 2;
        const int elements = to.bytes / SIZE;
#pragma unroll 1
        for (int r0 = 0; r0 < 32 && r0 < to.count; r0 += 4) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = r0 + i, row = MAPPED ? __shfl_sync(~0u, index, r) : r;
                char* p = to.base + row * to.pitch;
#pragma unroll
                for (int j = 0; j < TURNS; ++j) {
                    const int e = lane + 32 * j;
                    const uint4* q = staged(block, r, e / PER);
                    const bool here = e < elements && r < to.count;
                    if (SIZE == 4) {
                        const uint32_t v = reinterpret_cast<const uint32_t*>(q)[e % PER];
                        if (here) reinterpret_cast<uint32_t*>(p)[e] = v;
                    } else {
                        const unsigned short v = reinterpret_cast<const unsigned short*>(q)[e % PER];
                        if (here) reinterpret_cast<unsigned short*>(p)[e] = v;
                    }
                }
            }
        }
    }
    __syncwarp();
}

// Two values as one word of bfloat16 or FP16, rounded to nearest.
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if constexpr (BF16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&v);
    } else {
        const __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
}

// ---- the kernel -----------------------------------------------------------------------------
// EPI::BN, EPI::Params, and EPI(params, live, warp's io) with
//   bool reads(const Unit&): whether start reads what the phase before wrote (a chain's alone)
//   void start(const Unit&, int row, int col)
//   void unit(const Unit&, int row, int col, float (&acc)[BN / 2])
// called by each epilogue warp at the beginning of a unit (to load what it will need) and with its
// sums: lane l holds row `row` + l, columns col .. col + BN / 2.
// EPI::PROBLEMS: of the launch at most. EPI::PLANES: staged together (see Ring); with two, every unit has
// some of the reduction. EPI::CHAIN: units are claimed in order, and one waits until all units of the phase
// before that belong to the same product have been stored. Every earlier unit was claimed by a CTA that runs,
// and waits for still earlier ones only, so that all waits end however many CTAs the GPU runs at a time.
template <class EPI>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    half_gemm_kernel(const __grid_constant__ Args<EPI::PROBLEMS> g,
                     const __grid_constant__ typename EPI::Params ep) {
    constexpr int BN = EPI::BN;
    constexpr bool CHAIN = EPI::CHAIN;
    constexpr int COLS = BN / 2;  // columns of an epilogue warp
    using R = Ring<EPI>;
    constexpr int STAGES = R::STAGES;
    extern __shared__ uint8_t smem_raw[];
    const Smem sm = carve<R>(smem_raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = ptx::cluster_ctarank();

    if (threadIdx.x == 0) {
        for (int s = 0; s < 2 * MAX_STAGES; ++s) ptx::mbar_init(sm.at(s), 1);  // full, empty
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(sm.acc_full(b), 1);
            ptx::mbar_init(sm.acc_empty(b), 2 * EPI_WARPS);
        }
        for (int i = 0; i < SLOTS; ++i) {
            ptx::mbar_init(sm.slot_full(i), 1);
            // the first CTA's MMA warp, the TMA and the epilogue warps of both
            ptx::mbar_init(sm.slot_empty(i), 5 + 2 * EPI_WARPS);
        }
        ptx::mbar_init(sm.drain(), 1);
        ptx::mbar_init(sm.claim(), 1);
        for (int i = 0; i < 2 * EPI_WARPS; ++i) ptx::mbar_init(sm.loaded(i), 1);
        *sm.abort_flag = 0;
        ptx::fence_mbar_init();
        for (int i = 0; i < g.problems; ++i) {
            ptx::prefetch_tensormap(&g.a[i]);
            ptx::prefetch_tensormap(&g.b[i]);
        }
    }
    if (warp == 1) {
        ptx::tmem_alloc_pair(ptx::smem_u32(sm.tmem_slot), R::TMEM_COLUMNS);
        ptx::tmem_relinquish_pair();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::cluster_sync();
    ptx::tc_fence_after();
    const uint32_t tmem = *sm.tmem_slot;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    int live = 0;
    if (g.live) live = min(max(*g.live - g.live0, 0), g.live_max);
    const Units n_units = Units::of<BN, CHAIN>(g, live);
    // chain: what the phase before this unit's computes of its product has been stored, for TMA to
    // read
    int ready_phase = 0, ready_batch = -1;  // that this warp has found complete
    auto wait_before = [&](const Unit& t) {
        if (t.phase == 0 || (t.phase == ready_phase && t.batch == ready_batch)) return true;
        const int type = (t.phase - 1) % 3, batch = g.p[0].batch;
        const int units =
            type == 0 ? n_units.first : type == 1 ? n_units.second : n_units.third;
        bool ok = true;
        if (lane == 0)
            ok = wait_count(g.done + (t.phase - 1) * batch + t.batch, 2 * EPI_WARPS * (units / batch),
                            sm.abort_flag, g.err);
        ok = __all_sync(~0u, ok) != 0;
        ptx::fence_proxy_async_global();
        ready_phase = t.phase;
        ready_batch = t.batch;
        return ok;
    };
    // the unit in slot i, or -1 at the end or when a wait ran out
    auto take = [&](int i) {
        const int s = i % SLOTS;
        // the slot is written by the first CTA's thread: the only data that ordinary stores hand
        // to another CTA
        const bool there = wait_phase(sm.slot_full(s), (i / SLOTS) & 1, sm.abort_flag, g.err,
                                      WAIT_LIMIT_NS, true);
        return __all_sync(~0u, there) ? sm.slot_ptr[s] : -1;
    };
    // a whole warp's wait, with the same answer for all lanes
    auto wait_all = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(~0u, wait(bar, parity, sm, g.err)) != 0;
    };
    auto taken = [&](int i) {
        ptx::mbar_arrive_remote(ptx::mapa_shared(sm.slot_empty(i % SLOTS), 0));
    };

    if (warp < EPI_WARP0) {
        ptx::regs_give_up<REGS_FEW>();
        if (warp == 0 || warp == 2) {
            // all lanes go through the loop with equal values, one of them issues
            const bool is_a = warp == 0;
            const uint32_t full0 = sm.full(0), empty0 = sm.empty(0);
            const uint32_t signal0 = ptx::mapa_shared(full0, 0);  // the first CTA's barriers
            const bool expects = is_a && rank == 0;
            const uint32_t ring = sm.ring + (is_a ? 0 : R::B_AT);
            const uint32_t plane_bytes = is_a ? A_BYTES : B_BYTES<BN>;
            const bool tells = is_a && rank == 0 && lane == 0;  // that the next unit may be claimed
            int s = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int i = 0; ok; ++i) {
                const int u = take(i);
                __syncwarp();
                if (u < 0) break;
                if (lane == 0) taken(i);
                if (tells) ptx::mbar_arrive(sm.claim());
                const Unit t = unit_at<BN, CHAIN>(g, n_units, u, live);
                const Problem& p = g.p[t.problem];
                const CUtensorMap* map = is_a ? &g.a[t.problem] : &g.b[t.problem];
                const bool mn = is_a ? p.a_mn : p.b_mn;
                const unsigned char* planes = is_a ? p.pa : p.pb;
                const int z0 = t.batch * (is_a ? p.planes_a : p.planes_b);
                const int products = p.products;
                unsigned order = 0;  // the products' planes, four bits each
                for (int q = 0; q < products; ++q) order |= unsigned(planes[q]) << (4 * q);
                // coordinates of the first box, and how they move on
                const int o = is_a ? t.row0 + int(rank) * HALF_M : t.col0 + int(rank) * (BN / 2);
                const int k0 = t.kb0 * BK, first = is_a ? p.a_row : p.b_row;
                int x = mn ? o : k0, y = first + (mn ? k0 : o);
                const int dx = mn ? 0 : BK, dy = mn ? BK : 0;
                const bool two = mn && (is_a || BN == 256);
                ok = !CHAIN || wait_before(t);
                for (int kb = t.kb0; ok && kb < t.kb1; ++kb) {
                    unsigned planes_left = order;
                    for (int q = 0; q < products; ++q) {
                        const int z = z0 + int(planes_left & 15u);
                        planes_left >>= 4;
                        ok = wait_all(empty0 + 8u * s, ph ^ 1u);
                        if (!ok) break;
                        const uint32_t bar = signal0 + 8u * s;
                        uint32_t st = ring + uint32_t(s) * R::STAGE_BYTES;
                        // the bytes of both CTAs; some may have arrived already
                        if (expects)
                            ptx::mbar_arrive_expect_tx_elect(full0 + 8u * s, 2 * R::STAGE_BYTES);
#pragma unroll
                        for (int i = 0; i < R::PLANES; ++i) {
                            const int zi = R::PLANES == 1 ? z : z0 + i;
                            ptx::tma_load_3d_pair(st, map, bar, x, y, zi);
                            if (two)
                                ptx::tma_load_3d_pair(st + CHUNK_BYTES, map, bar, x + 64, y, zi);
                            st += plane_bytes;
                        }
                        if (++s == STAGES) {
                            s = 0;
                            ph ^= 1u;
                        }
                    }
                    x += dx;
                    y += dy;
                }
            }
            if (*sm.abort_flag) {  // copies in flight arrive before shared memory is given up
                const unsigned long long t0 = ptx::globaltimer_ns();
                while (ptx::globaltimer_ns() - t0 < 10000000ull) {
                }
            }
        } else if (warp == 3 && rank == 0) {
            // the first units are given out by the pairs' numbers, in a chain claimed like all
            // others: a pair may not be running yet
            const int pairs = CHAIN ? 0 : gridDim.x >> 1;
            if (lane == 0) {
                int next = CHAIN ? atomicAdd(g.counter, 1) : blockIdx.x >> 1;
                for (int i = 0;; ++i) {
                    const int slot = i % SLOTS;
                    int u = next < n_units.all ? next : -1;
                    if (!wait(sm.slot_empty(slot), ((i / SLOTS) & 1) ^ 1, sm, g.err)) u = -1;
                    sm.slot_ptr[slot] = u;
                    ptx::st_shared_cluster_f32(ptx::mapa_shared(sm.slots + 4u * slot, 1),
                                               __int_as_float(u));
                    ptx::mbar_arrive_cluster(ptx::mapa_shared(sm.slot_full(slot), 0));
                    ptx::mbar_arrive_cluster(ptx::mapa_shared(sm.slot_full(slot), 1));
                    if (u < 0) break;
                    // when the unit's loads begin; earlier, other pairs would run out of units
                    const bool go = wait(sm.claim(), i & 1, sm, g.err);
                    next = go ? pairs + atomicAdd(g.counter, 1) : n_units.all;
                }
            }
        } else if (warp == 1 && rank == 0) {
            int s = 0, seg = 0;
            uint32_t ph = 0;
            bool ok = true, issued = false;
            for (int i = 0; ok; ++i) {
                const int u = take(i);
                __syncwarp();
                if (u < 0) break;
                if (lane == 0) taken(i);
                const Unit t = unit_at<BN, CHAIN>(g, n_units, u, live);
                const Problem& p = g.p[t.problem];
                const uint32_t idesc = p.idesc | (uint32_t(BN >> 3) << 17);
                const OperandDesc a(sm.ring, p.a_mn), b(sm.ring + R::B_AT, p.b_mn);
                // Two planes: the unit's sum of the products that have a second one. The unit before the
                // last had this accumulator, and its last segment, read with it, was waited for at the
                // latest with this unit's first: the unit between has one at least.
                const uint32_t d_low = tmem + uint32_t(2 * BN + (i & 1) * BN);
                uint32_t started = 0;
                int left = (t.kb1 - t.kb0) * p.products;
                for (; ok && left > 0; left -= g.seg_steps, ++seg) {
                    const int half = seg & 1;
                    ok = wait_all(sm.acc_empty(half), ((seg >> 1) & 1) ^ 1);
                    if (!ok) break;
                    ptx::tc_fence_after();
                    const uint32_t d = tmem + uint32_t(half * BN);
                    const int steps = min(left, g.seg_steps);
                    for (int j = 0; j < steps; ++j) {
                        ok = wait_all(sm.full(s), ph);
                        if (!ok) break;
                        ptx::tc_fence_after();
                        const uint32_t at = uint32_t(s) * (R::STAGE_BYTES >> 4);
                        if constexpr (R::PLANES == 1) {
                            ptx::mma_pair_x4(d, a.lo + at, a.hi, a.step, b.lo + at, b.hi, b.step,
                                             idesc, j);
                        } else {
                            constexpr uint32_t A1 = A_BYTES >> 4, B1 = B_BYTES<BN> >> 4;
                            ptx::mma_pair_x4(d_low, a.lo + at + A1, a.hi, a.step, b.lo + at, b.hi,
                                             b.step, idesc, started);
                            started = 1;
                            ptx::mma_pair_x4(d_low, a.lo + at, a.hi, a.step, b.lo + at + B1, b.hi,
                                             b.step, idesc, 1);
                            ptx::mma_pair_x4(d, a.lo + at, a.hi, a.step, b.lo + at, b.hi, b.step,
                                             idesc, j);
                        }
                        issued = true;
                        ptx::mma_commit_pair_elect(sm.empty(s), 0x3);
                        if (++s == STAGES) {
                            s = 0;
                            ph ^= 1u;
                        }
                    }
                    if (!ok) break;
                    ptx::mma_commit_pair_elect(sm.acc_full(half), 0x3);
                }
            }
            if (__any_sync(~0u, *sm.abort_flag != 0) && issued) {
                // MMAs in flight end before TMEM is freed
                ptx::mma_commit_pair_elect(sm.drain(), 0x1);
                const unsigned long long t0 = ptx::globaltimer_ns();
                while (!ptx::mbar_try_wait(sm.drain(), 0) &&
                       ptx::globaltimer_ns() - t0 < WAIT_LIMIT_NS) {
                }
            }
        }
    } else {
        ptx::regs_take<REGS_MANY>();
        // warp w reads TMEM lanes [32 (w % 4), +32) and the first or second half of the columns
        const int q = warp & 3, h = (warp - EPI_WARP0) >> 2;
        WarpIo<R::BLOCKS> io;
        io.blocks = sm.staging + R::BLOCKS * (warp - EPI_WARP0) * STAGING;
        io.bar = sm.loaded(2 * (warp - EPI_WARP0));
        io.abort_flag = sm.abort_flag;
        io.err = g.err;
        io.first = lane == 0;
        EPI epi(ep, live, io);
        float acc[COLS];
        int seg = 0;
        bool ok = true;
        for (int i = 0; ok; ++i) {
            const int u = take(i);
            __syncwarp();  // all lanes have read the slot
            if (u < 0) break;
            if (lane == 0) taken(i);
            const Unit t = unit_at<BN, CHAIN>(g, n_units, u, live);
            const int steps = (t.kb1 - t.kb0) * g.p[t.problem].products;
            const int segs = (steps + g.seg_steps - 1) / g.seg_steps;
            const int row = t.row0 + int(rank) * HALF_M + q * 32, col = t.col0 + h * COLS;
            if constexpr (CHAIN) {
                if (epi.reads(t) && !wait_before(t)) break;
            }
            epi.start(t, row, col);
            for (int sg = 0; sg < segs; ++sg, ++seg) {
                const int b = seg & 1;
                ok = wait_all(sm.acc_full(b), (seg >> 1) & 1);
                if (!ok) break;
                ptx::tc_fence_after();
                const uint32_t at = tmem + (uint32_t(q * 32) << 16) + uint32_t(b * BN + h * COLS);
                if (sg == 0) {
#pragma unroll
                    for (int c = 0; c < COLS; c += 64) {
                        uint32_t r[64];
                        __syncwarp();
                        ptx::tmem_ld_64(at + c, r);
#pragma unroll
                        for (int j = 0; j < 64; ++j) acc[c + j] = __uint_as_float(r[j]);
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < COLS; c += 16) {
                        uint32_t r[16];
                        __syncwarp();
                        ptx::tmem_ld_16(at + c, r);
#pragma unroll
                        for (int j = 0; j < 16; ++j) acc[c + j] += __uint_as_float(r[j]);
                    }
                }
                if constexpr (R::PLANES == 2) {
                    if (sg == segs - 1) {
                        const uint32_t low =
                            tmem + (uint32_t(q * 32) << 16) + uint32_t((2 + (i & 1)) * BN + h * COLS);
#pragma unroll
                        for (int c = 0; c < COLS; c += 16) {
                            uint32_t r[16];
                            __syncwarp();
                            ptx::tmem_ld_16(low + c, r);
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                acc[c + j] = fmaf(__uint_as_float(r[j]), SECOND_DOWN, acc[c + j]);
                        }
                    }
                }
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive_remote(ptx::mapa_shared(sm.acc_empty(b), 0));
            }
            if (!ok) break;
            if (segs == 0) {
#pragma unroll
                for (int j = 0; j < COLS; ++j) acc[j] = 0.f;
            }
            epi.unit(t, row, col, acc);
            if constexpr (CHAIN) {
                __syncwarp();
                if (lane == 0) {
                    ptx::bulk_wait0();  // its stores are in global memory
                    ptx::fence_proxy_async_global();
                    ptx::red_release_gpu_add(g.done + t.phase * g.p[0].batch + t.batch, 1);
                }
            }
        }
        io.finish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::cluster_sync();
    if (warp == 1) {
        __syncwarp();
        ptx::tc_fence_after();
        ptx::tmem_dealloc_pair(tmem, R::TMEM_COLUMNS);
    }
}

// ---- host -------------------------------------------------------------------------------------
// A 3-D map over 16-bit elements: `inner` contiguous elements, `rows` of pitch `ld` elements (a
// multiple of 8), `slabs` of `slab` elements apart; boxes of 64 x box_rows. Zeros are read outside.
bool encode_operand(CUtensorMap* map, const void* base, bool bf16, long long inner, long long rows,
                    long long ld, long long slabs, long long slab, int box_rows);

// The same for the epilogue's blocks: elements of `size` bytes (2, FP16; 4, FP32), boxes of box_cols
// x box_rows, 128-byte swizzled where a row has 128 bytes. Nothing is written outside.
bool encode_block(CUtensorMap* map, const void* base, int size, long long cols, long long rows,
                  long long ld, long long slabs, long long slab, int box_cols, int box_rows);

// Launches `kernel`, allowed to start while the kernel before it on the stream ends (it waits
// for that one by griddepcontrol.wait).
template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kernel)(KArgs...), unsigned grid, unsigned block, size_t smem,
                   cudaStream_t stream, const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    count_launch();
    return e;
}

// Regions of one allocation, each 256-byte aligned.
struct Layout {
    size_t total = 0;
    size_t add(size_t bytes) {
        const size_t at = total;
        total += (bytes + 255) & ~size_t(255);
        return at;
    }
};

// Box rows of an operand: 64 k of a chunk, or its rows in a CTA.
inline int box_rows(bool mn, int rows_of_cta) { return mn ? BK : rows_of_cta; }

// Raises the kernel's shared-memory limit, once per device, and makes sure that its threads start
// with the registers that its warpgroups share out among themselves: with fewer, the second of them
// would wait for registers that nobody gives up.
template <class EPI>
cudaError_t prepare_gemm() {
    const cudaError_t e = set_smem_limit_once<half_gemm_kernel<EPI>>(Ring<EPI>::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    static const cudaError_t enough = [] {
        cudaFuncAttributes attr;
        const cudaError_t f = cudaFuncGetAttributes(&attr, half_gemm_kernel<EPI>);
        if (f != cudaSuccess) return f;
        return 3 * attr.numRegs < REGS_FEW + 2 * REGS_MANY ? cudaErrorLaunchOutOfResources
                                                           : cudaSuccess;
    }();
    return enough;
}

template <class EPI>
cudaError_t launch_gemm(const Args<EPI::PROBLEMS>& g, const typename EPI::Params& ep, int sm_count,
                        cudaStream_t stream) {
    const cudaError_t e = prepare_gemm<EPI>();
    if (e != cudaSuccess) return e;
    // pairs for all units, in a chain for those of its largest phase
    int units = 0;
    for (int i = 0; i < g.problems; ++i) {
        const int n = unit_count<EPI::BN>(g.p[i], g.live_max);
        units = !EPI::CHAIN ? units + n : units > n ? units : n;
    }
    if (units == 0) return cudaSuccess;
    const int pairs = sm_count / 2 > 0 ? sm_count / 2 : 1;
    return launch(half_gemm_kernel<EPI>, 2u * unsigned(units < pairs ? units : pairs), THREADS,
                  Ring<EPI>::SMEM_BYTES, stream, g, ep);
}

}  // namespace hg
}  // namespace sgemm
