// Few-row products with 4-bit weights: C[M x K] = A[M x N] . B, B in the packed format of
// q4.cuh. The bytes of B are the cost, so the kernel is built to keep HBM busy and to spend few
// instructions on a weight.
//
// One CTA an SM works on tiles of 128 columns of C. Per unit (128 columns x 128 n, about 8.5 KB):
//  * a producer lane copies it into a ring of shared-memory slots with one bulk copy, many
//    units ahead;
//  * one of two warpgroups (they take turns) turns its codes into operand words, a thread a
//    column, and stores them to its lane of tensor memory: 80 logic instructions for 128
//    weights;
//  * the MMA warp multiplies them with the CTA's columns of A^T (tcgen05, 128 x 16 from tensor
//    memory by 16 x 16 or 16 x 32 from shared memory; a "column" is a bfloat16 piece of a row of
//    A), a group of n at a time into an accumulator of its own;
//  * the warpgroup reads each group's sums, scales them in FP32 and adds them to its totals in
//    registers. With two units of each warpgroup in flight the round trip through tensor
//    memory (about 700 cycles) is hidden.
// The columns are staged in shared memory once for all the tiles of a CTA. Where the tiles alone
// would not fill the GPU, or the columns not fit, the CTAs of a cluster split n. Each CTA then
// owns a part of the tile's columns of C; its output warps fetch all CTAs' totals of that part
// through distributed shared memory, add them in a fixed order and write C: one launch, no
// workspace, no atomics.
//
// What bounds it: the instructions of a unit in two warpgroups, some 600 cycles an SM against the
// 365 that its bytes take at HBM's rate. 16 x 8192 by 65536 columns, group 128: 74 us (3.7 TB/s);
// 16 x 8192 by 6144, group 64: 18.0 us; 64 x 8192 by 65536 (two launches' worth of rows in one
// grid, each reading the weights): 215 us. Four warpgroups with one unit each in flight measured
// 91, 26 and 216 us, short of registers.
#include <atomic>
#include <type_traits>

#include "q4_stage.cuh"
#include "wait.cuh"

namespace sgemm {
namespace {

// two MMA warps, eight of the warpgroups, four output warps
constexpr int WARP_PRODUCER = 0, WARP_MMA = 1, WARP_SIGNAL = 3, WARP_GROUPS = 4, WARP_OUTPUT = 12;
constexpr int WARPS = 16, THREADS = WARPS * 32;
constexpr int OUTPUT_WARPS = WARPS - WARP_OUTPUT, OUTPUT_THREADS = OUTPUT_WARPS * 32;
constexpr int MAX_RING = 20;
constexpr int SMEM_LIMIT = 227 * 1024;
constexpr int TMEM_COLUMNS = 512;  // two warpgroups' pairs of operand and accumulator buffers
constexpr int TMEM_SLOT = 64;      // columns of one of them

struct Plan {
    int cluster;   // CTAs that split n
    int units;     // of a CTA's n range
    int clusters;  // launched; cluster i takes tiles i, i + clusters, ...
    int ring;      // slots
    int smem;
};

// Columns that a CTA multiplies (COLUMNS of them have their sums read), as the MMA takes them:
// its N, and the rows of 16 bytes that hold them in shared memory (N = 16 with 8 such rows reads
// these twice).
template <int COLUMNS>
struct Shape {
    static constexpr int N = COLUMNS < 16 ? 16 : COLUMNS;
    static constexpr int ROWS = COLUMNS <= 8 ? 8 : COLUMNS;
    // bytes from 8 n to the next; 16 more than the rows take, so that staging meets few bank
    // conflicts
    static constexpr int STRIDE = ROWS * 16 + 16;
};

// Where a CTA's shared memory holds what, in bytes.
struct Offsets {
    int ring, xsum, send, bars, end;
};
template <int COLUMNS, int GROUP>
__host__ __device__ constexpr Offsets offsets(int units, int ring, int unit_bytes) {
    Offsets o{};
    o.ring = units * (kQ4UnitN / 8) * Shape<COLUMNS>::STRIDE;
    o.xsum = o.ring + ring * unit_bytes;
    o.send = o.xsum + units * (kQ4UnitN / GROUP) * COLUMNS * 4;
    o.bars = o.send + 2 * 2 * kQ4UnitK * COLUMNS * 4;
    o.end = o.bars + 8 * (2 * MAX_RING + 20);
    return o;
}

// Shared-memory matrix descriptor of 16 n of the columns, no swizzle: blocks of 8 columns x 16
// bytes (8 n) are contiguous; lbo from one 8 n to the next, sbo from 8 columns to the next.
__device__ __forceinline__ uint64_t column_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    return uint64_t((saddr >> 4) & 0x3FFFu) | uint64_t(lbo >> 4) << 16 | uint64_t(sbo >> 4) << 32 |
           uint64_t(1) << 46;
}
// kind::f16 with bfloat16 operands, FP32 accumulator, M = 128.
__host__ __device__ constexpr uint32_t idesc_bf16(int n) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(n >> 3) << 17) | (8u << 24);
}

// Spins until the phase is over or the limit has passed, whatever the abort flag says.
__device__ __noinline__ void wait_drained(uint32_t bar, uint32_t parity) {
    const unsigned long long t0 = ptx::globaltimer_ns();
    while (!ptx::mbar_try_wait(bar, parity) && ptx::globaltimer_ns() - t0 < WAIT_LIMIT_NS) {
    }
}

template <int COLUMNS, int GROUP, bool ZEROS>
__global__ void __launch_bounds__(THREADS, 1) q4_matmul_kernel(const Q4Product args, const Plan plan) {
    extern __shared__ __align__(128) uint8_t smem[];
    using S = Shape<COLUMNS>;
    constexpr int GROUPS = kQ4UnitN / GROUP;
    // groups that share an accumulator slot, and slots' worth of groups of a unit
    constexpr int GROUPS_SLOT = GROUPS < TMEM_SLOT / S::N ? GROUPS : TMEM_SLOT / S::N;
    constexpr int STEPS = GROUPS / GROUPS_SLOT;
    __shared__ uint32_t tmem_base_s;
    __shared__ volatile int abort_s;

    const Q4Geom& geom = args.geom;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = plan.cluster > 1 ? int(ptx::cluster_ctarank()) : 0;
    const int first_tile = blockIdx.x / plan.cluster;
    const int tiles = (geom.tiles - first_tile + plan.clusters - 1) / plan.clusters;
    const int unit0 = rank * plan.units;
    const int units = max(0, min(plan.units, geom.units - unit0));  // of a tile, here
    const int total_units = tiles * units;
    const int row_columns = args.row_columns, most_rows = COLUMNS / row_columns;
    const int row0 = blockIdx.y * most_rows;
    const int rows = min(most_rows, args.M - row0);
    const int quads = (rows * row_columns + 3) / 4;  // of columns

    const Offsets at = offsets<COLUMNS, GROUP>(plan.units, plan.ring, geom.unit_bytes);
    uint8_t* ring = smem + at.ring;
    float* xsum = reinterpret_cast<float*>(smem + at.xsum);
    const uint32_t bar0 = ptx::smem_u32(smem + at.bars);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (MAX_RING + s); };
    auto a_full = [&](int wg, int b) { return bar0 + 8u * (2 * MAX_RING + 2 * wg + b); };
    auto d_full = [&](int wg, int b) { return bar0 + 8u * (2 * MAX_RING + 4 + 2 * wg + b); };
    auto d_empty = [&](int wg, int b) { return bar0 + 8u * (2 * MAX_RING + 8 + 2 * wg + b); };
    auto send_full = [&](int b) { return bar0 + 8u * (2 * MAX_RING + 12 + b); };
    auto peers_full = [&](int b) { return bar0 + 8u * (2 * MAX_RING + 18 + b); };
    auto credit = [&](int b) { return bar0 + 8u * (2 * MAX_RING + 14 + b); };
    auto drained = [&](int wg) { return bar0 + 8u * (2 * MAX_RING + 16 + wg); };
    // Bounded. When a wait gives up, the abort flag makes all later ones return at once: every
    // role then runs through to its end on whatever memory holds (its addresses do not depend
    // on what it reads), and the producer stops fetching.
    auto wait = [&](uint32_t bar, int use, bool cluster = false) {
        wait_phase(bar, use & 1, &abort_s, args.err, WAIT_LIMIT_NS, cluster);
    };

    // rows of a tile that each CTA of the cluster adds up
    const int slice = kQ4UnitK / plan.cluster;
    if (threadIdx.x == 0) {
        for (int s = 0; s < plan.ring; ++s) {
            ptx::mbar_init(full(s), 1);
            ptx::mbar_init(empty(s), 4);
        }
        for (int wg = 0; wg < 2; ++wg)
            for (int b = 0; b < 2; ++b) {
                ptx::mbar_init(a_full(wg, b), 4);
                ptx::mbar_init(d_full(wg, b), 1);
                ptx::mbar_init(d_empty(wg, b), 4);
            }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(send_full(b), 8);  // the warps of the warpgroups
            ptx::mbar_init(peers_full(b), plan.cluster);
            ptx::mbar_init(credit(b), plan.cluster * OUTPUT_WARPS);
        }
        for (int wg = 0; wg < 2; ++wg) ptx::mbar_init(drained(wg), 1);
        abort_s = 0;
        ptx::fence_mbar_init();
    }
    if (warp == WARP_MMA) {
        ptx::tmem_alloc(ptx::smem_u32(&tmem_base_s), TMEM_COLUMNS);
        ptx::tmem_relinquish();
    }
    // Nothing in global memory is touched before the kernels ahead in the stream are done; the
    // next one may take its place on SMs as they come free.
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    ptx::tc_fence_before();
    __syncthreads();
    if (plan.cluster > 1) ptx::cluster_sync();  // the peers' barriers are there too
    ptx::tc_fence_after();
    const uint32_t tmem = tmem_base_s;

    // the producer's state: the next unit to fetch
    int f_unit = 0, f_slot = 0, f_use = 0, f_in_tile = 0;
    const uint8_t* f_from = args.data + size_t(first_tile) * geom.tile_bytes() +
                            size_t(unit0) * geom.unit_bytes;
    const size_t f_wrap = size_t(plan.clusters) * geom.tile_bytes() - size_t(units) * geom.unit_bytes;
    auto fetch = [&]() {
        ptx::mbar_arrive_expect_tx(full(f_slot), geom.unit_bytes);
        ptx::bulk_load(ptx::smem_u32(ring + f_slot * geom.unit_bytes), f_from, geom.unit_bytes,
                       full(f_slot));
        f_from += geom.unit_bytes;
        if (++f_in_tile == units) {
            f_in_tile = 0;
            f_from += f_wrap;
        }
        ++f_unit;
        if (++f_slot == plan.ring) {
            f_slot = 0;
            ++f_use;
        }
    };
    if (threadIdx.x == WARP_PRODUCER * 32)
        for (int i = min(plan.ring, total_units); i > 0; --i) fetch();

    Staging st;
    st.A = static_cast<const uint8_t*>(args.A) + row0 * args.lda * dtype_bytes(args.dtype);
    st.lda = args.lda;
    st.dtype = args.dtype;
    st.rows = rows;
    st.n0 = unit0 * kQ4UnitN;
    st.N = geom.N;
    st.octets = units * (kQ4UnitN / 8);
    st.threads = THREADS;
    st.octet_stride = S::STRIDE;
    st.column_stride = 16;
    st.vec = args.vec;
    st.xs = smem;
    st.xsum = xsum;
    st.sum_pitch = COLUMNS;
    st.log_octets = GROUP == 32 ? 2 : GROUP == 64 ? 3 : 4;
    st.factor = ZEROS ? -1.0f : -8.0f;
    st.turn = first_tile;
    st.turns = plan.clusters;
    const bool special = stage_columns(st);

    if (warp == WARP_PRODUCER) {
        if (lane == 0)
            while (f_unit < total_units) {
                wait(empty(f_slot), f_use + 1);
                if (abort_s) break;
                fetch();
            }
        __syncwarp();
    } else if (warp < WARP_SIGNAL) {
        constexpr uint32_t idesc = idesc_bf16(S::N);
        const uint32_t xs = ptx::smem_u32(smem);
        const int wg = warp - WARP_MMA;
        int in_tile = wg % units, k = 0;
        for (int s = wg; s < total_units; s += 2, ++k) {
            wait(a_full(wg, k & 1), k >> 1);
            // the broadcasts tell the compiler that the operands are uniform
            const uint32_t a =
                __shfl_sync(0xffffffffu, tmem + uint32_t(wg * 2 + (k & 1)) * TMEM_SLOT, 0);
            const uint64_t b = column_desc(
                __shfl_sync(0xffffffffu, xs + in_tile * (kQ4UnitN / 8) * S::STRIDE, 0), S::STRIDE,
                S::ROWS > 8 ? 128 : 0);
#pragma unroll
            for (int step = 0; step < STEPS; ++step) {
                const int use = k * STEPS + step;
                // with one step, the unit's operand words came after the slot was read
                if (STEPS > 1) wait(d_empty(wg, use & 1), (use >> 1) + 1);
                ptx::tc_fence_after();
                const uint32_t d =
                    __shfl_sync(0xffffffffu, tmem + uint32_t(4 + wg * 2 + (use & 1)) * TMEM_SLOT, 0);
#pragma unroll
                for (int g = 0; g < GROUPS_SLOT; ++g)
#pragma unroll
                    for (int i = 0; i < GROUP / 16; ++i) {
                        const int at16 = (step * GROUPS_SLOT + g) * (GROUP / 16) + i;
                        ptx::mma_ts(d + g * S::N, a + at16 * 8, b + at16 * 2 * (S::STRIDE / 16), idesc,
                                    i > 0);
                    }
                ptx::mma_commit(d_full(wg, use & 1));
            }
            for (in_tile += 2; in_tile >= units;) in_tile -= units;
        }
        if (abort_s) {  // MMAs may still be in flight
            ptx::mma_commit(drained(wg));
            wait_drained(drained(wg), 0);
        }
    } else if (warp == WARP_SIGNAL) {
        // Tells the owners that this CTA's totals are there. An arrival on another CTA's barrier
        // that releases what was written here takes some 1500 cycles, which the warpgroups would
        // otherwise spend on each tile.
        if (plan.cluster > 1)
            for (int i = 0; i < tiles; ++i) {
                wait(send_full(i & 1), i >> 1);
                if (lane < plan.cluster)
                    ptx::mbar_arrive_cluster(ptx::mapa_shared(peers_full(i & 1), lane));
            }
        __syncwarp();
    } else if (warp < WARP_OUTPUT) {
        auto work = [&](auto centred) {
            constexpr bool CENTRED = decltype(centred)::value;
            const int wg = (warp - WARP_GROUPS) >> 2;
            const int row = (warp & 3) * 32 + lane;  // of the tile, and lane of tensor memory
            const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
            float scale0[GROUPS], scale1[GROUPS];  // of the unit in buffer 0 and 1
            float zero0[GROUPS], zero1[GROUPS];
#pragma unroll
            for (int g = 0; g < GROUPS; ++g) scale0[g] = scale1[g] = zero0[g] = zero1[g] = 1.0f;

            // Unit number k of this warpgroup's (sequence number wg + 2 k): read() takes its codes,
            // scales and zero points into registers, operand() turns them into operand words.
            int q_slot = wg, q_use = 0;
            uint4 w[4];
            float scale[GROUPS], zero[GROUPS];
            uint32_t base[GROUPS];
            auto read = [&](int k) {
                if (wg + 2 * k >= total_units) return;
                wait(full(q_slot), q_use);
                const uint8_t* unit = ring + q_slot * geom.unit_bytes;
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    w[b] = reinterpret_cast<const uint4*>(unit)[b * kQ4UnitK + row];
#pragma unroll
                for (int g = 0; g < GROUPS; ++g) {
                    scale[g] = q4_scale(
                        reinterpret_cast<const uint16_t*>(unit + kQ4CodeBytes)[g * kQ4UnitK + row],
                        geom.fp16);
                    uint32_t z = 8;
                    if constexpr (ZEROS)
                        z = unit[kQ4CodeBytes + GROUPS * kQ4UnitK * 2 + g * kQ4UnitK + row];
                    base[g] = 0x43004300u | z * 0x00010001u;
                    zero[g] = __uint_as_float(base[g] & 0xffff0000u) - 128.0f;
                }
                __syncwarp();  // all lanes have read
                if (lane == 0) ptx::mbar_arrive(empty(q_slot));
                q_slot += 2;
                if (q_slot >= plan.ring) {
                    q_slot -= plan.ring;
                    ++q_use;
                }
            };
            auto operand = [&](int k) {
                if (wg + 2 * k >= total_units) return;
                const uint32_t a = tmem + lanes + uint32_t(wg * 2 + (k & 1)) * TMEM_SLOT;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const uint32_t word[4] = {w[b].x, w[b].y, w[b].z, w[b].w};
                    uint32_t r[16];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t o[4];
                        if constexpr (CENTRED)
                            q4_centred(word[i], base[b * 32 / GROUP], o);
                        else
                            q4_plain(word[i], o);
#pragma unroll
                        for (int j = 0; j < 4; ++j) r[4 * i + j] = o[j];
                    }
                    ptx::tmem_st_16(a + b * 16, r);
                }
#pragma unroll
                for (int g = 0; g < GROUPS; ++g) {
                    scale0[g] = k & 1 ? scale0[g] : scale[g];
                    scale1[g] = k & 1 ? scale[g] : scale1[g];
                    if constexpr (ZEROS) {
                        zero0[g] = k & 1 ? zero0[g] : zero[g];
                        zero1[g] = k & 1 ? zero[g] : zero1[g];
                    }
                }
                ptx::tmem_st_wait();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(a_full(wg, k & 1));
            };

            float total[COLUMNS];
            read(0);
            operand(0);
            read(1);
            operand(1);
            int k = 0;
            for (int i = 0; i < tiles; ++i) {
#pragma unroll
                for (int j = 0; j < COLUMNS; ++j) total[j] = 0.0f;
                for (int in_tile = wg ^ (i * units & 1); in_tile < units; in_tile += 2, ++k) {
                    read(k + 2);
#pragma unroll
                    for (int step = 0; step < STEPS; ++step) {
                        const int use = k * STEPS + step;
                        wait(d_full(wg, use & 1), use >> 1);
                        ptx::tc_fence_after();
                        const uint32_t d = tmem + lanes + uint32_t(4 + wg * 2 + (use & 1)) * TMEM_SLOT;
                        constexpr int READ = COLUMNS < 16 ? COLUMNS : 16;
#pragma unroll
                        for (int g = 0; g < GROUPS_SLOT; ++g) {
                            const int gg = step * GROUPS_SLOT + g;
                            const float s = k & 1 ? scale1[gg] : scale0[gg];
                            const float z = k & 1 ? zero1[gg] : zero0[gg];
                            const float4* xs4 = reinterpret_cast<const float4*>(
                                xsum + (in_tile * GROUPS + gg) * COLUMNS);
#pragma unroll
                            for (int c0 = 0; c0 < COLUMNS; c0 += READ) {
                                float acc[READ];
                                ptx::tmem_ld<READ>(d + g * S::N + c0, acc);
#pragma unroll
                                for (int c = 0; c < READ; c += 4) {
                                    const float4 x4 = xs4[(c0 + c) / 4];
                                    const float x[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
                                    for (int e = 0; e < 4; ++e) {
                                        float& sum = total[c0 + c + e];
                                        if constexpr (CENTRED)
                                            sum = add_centred(s, x[e], acc[c + e], sum);
                                        else
                                            sum = fmaf(s, fmaf(acc[c + e], kQ4Unscale,
                                                               ZEROS ? z * x[e] : x[e]), sum);
                                    }
                                }
                            }
                        }
                        ptx::tc_fence_before();
                        __syncwarp();
                        if (STEPS > 1 && lane == 0) ptx::mbar_arrive(d_empty(wg, use & 1));
                    }
                    operand(k + 2);
                }
                // the totals: [warpgroup][4 columns][row]; the owners of the rows fetch them
                const int buffer = i & 1;
                wait(credit(buffer), (i >> 1) + 1, plan.cluster > 1);
                float4* mine = reinterpret_cast<float4*>(smem + at.send) +
                               (buffer * 2 + wg) * (COLUMNS / 4) * kQ4UnitK + row;
#pragma unroll
                for (int q = 0; q < COLUMNS / 4; ++q)
                    if (q < quads)
                        mine[q * kQ4UnitK] = make_float4(total[4 * q], total[4 * q + 1],
                                                         total[4 * q + 2], total[4 * q + 3]);
                __syncwarp();  // the arrival below releases the whole warp's stores
                if (lane == 0) ptx::mbar_arrive(send_full(buffer));
            }
        };
        if (special)
            work(std::true_type());
        else
            work(std::false_type());
    } else {
        // output warps: the totals of this CTA's slice of each tile, in rank order
        const int id = threadIdx.x - WARP_OUTPUT * 32;
        const int slice_log = __ffs(slice) - 1;
        const bool alone = plan.cluster == 1;
        for (int i = 0; i < tiles; ++i) {
            const int buffer = i & 1;
            wait(alone ? send_full(buffer) : peers_full(buffer), i >> 1, !alone);
            const int k0 = (first_tile + i * plan.clusters) * kQ4UnitK + rank * slice;
            const uint32_t from = ptx::smem_u32(smem + at.send) +
                                  (buffer * 2 * (COLUMNS / 4) * kQ4UnitK + rank * slice) * 16;
            for (int cell = id; cell < quads << slice_log; cell += OUTPUT_THREADS) {
                const int q = cell >> slice_log, local = cell - (q << slice_log), k = k0 + local;
                float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
                for (int src = 0; src < plan.cluster; ++src) {
                    const uint32_t theirs = alone ? from : ptx::mapa_shared(from, src);
#pragma unroll
                    for (int wg = 0; wg < 2; ++wg) {
                        const uint32_t there =
                            theirs + ((wg * (COLUMNS / 4) + q) * kQ4UnitK + local) * 16;
                        const float4 x =
                            alone ? ptx::ld_shared_v4(there) : ptx::ld_shared_cluster_v4(there);
                        v.x += x.x;
                        v.y += x.y;
                        v.z += x.z;
                        v.w += x.w;
                    }
                }
                if (k >= geom.K) continue;
                size_t to = row0 * args.ldc + k;
                if (args.dtype == SGEMM_FLOAT32) {
                    store_from_float(args.C, SGEMM_FLOAT32, to + q * args.ldc, v.x + v.y + v.z);
                } else if (args.dtype == SGEMM_FLOAT16) {
                    to += 2 * q * args.ldc;
                    store_from_float(args.C, SGEMM_FLOAT16, to, v.x + v.y);
                    if (2 * q + 1 < rows)
                        store_from_float(args.C, SGEMM_FLOAT16, to + args.ldc, v.z + v.w);
                } else {
                    const float e[4] = {v.x, v.y, v.z, v.w};
                    to += 4 * q * args.ldc;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (4 * q + j < rows)
                            store_from_float(args.C, SGEMM_BFLOAT16, to + j * args.ldc, e[j]);
                }
            }
            __syncwarp();
            if (plan.cluster == 1) {
                if (lane == 0) ptx::mbar_arrive(credit(buffer));
            } else if (lane < plan.cluster) {
                ptx::mbar_arrive_cluster(ptx::mapa_shared(credit(buffer), lane));
            }
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (abort_s && threadIdx.x == WARP_PRODUCER * 32)  // copies may still be in flight
        for (int s = 0; s < plan.ring; ++s) {
            const int uses = f_use + (s < f_slot);  // of this slot so far
            if (uses > 0) wait_drained(full(s), (uses - 1) & 1);
        }
    if (warp == WARP_MMA) ptx::tmem_dealloc(tmem, TMEM_COLUMNS);
    // a CTA's shared memory is written by the others until here
    if (plan.cluster > 1) ptx::cluster_sync();
}

// Clusters of this size that the device holds at once, one CTA an SM.
template <auto KERNEL>
int resident_clusters(int cluster, int sm_count) {
    if (cluster == 1) return sm_count;
    constexpr int kDevices = 64;
    static std::atomic<int> known[kDevices][3];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) dev = 0;
    std::atomic<int>& slot = known[dev][cluster == 2 ? 0 : cluster == 4 ? 1 : 2];
    int n = slot.load(std::memory_order_relaxed);
    if (n > 0) return n;
    cudaLaunchConfig_t config = {};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    config.gridDim = dim3(sm_count / cluster * cluster);
    config.blockDim = dim3(THREADS);
    config.dynamicSmemBytes = SMEM_LIMIT - 1024;
    config.attrs = &attr;
    config.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, KERNEL, &config) != cudaSuccess || n < 1) {
        cudaGetLastError();
        n = sm_count / cluster > 0 ? sm_count / cluster : 1;
    }
    slot.store(n, std::memory_order_relaxed);
    return n;
}

// The split of the product: the cluster size whose slowest SM is done first. In cycles: a
// unit takes an SM 600, or what its bytes take of HBM's rate (3500 a cycle) when all that are
// busy share it; a cluster's exchange 1500 a tile; staging 28 a column and unit. Larger clusters
// stage less each but exchange more, and of 8 only 15 are resident: 16 rows of 4096 by 14336
// columns take 19.8, 17.6, 16.6 and 21.1 us with clusters of 1, 2, 4 and 8.
template <int COLUMNS, int GROUP, bool ZEROS>
bool make_plan(const Q4Geom& g, int sm_count, Plan* best) {
    constexpr int STATIC = 1024;  // statically allocated shared memory and the system's
    double best_cost = 1e30;
    for (int cluster = 1; cluster <= 8; cluster *= 2) {
        Plan p;
        p.cluster = cluster;
        p.units = (g.units + cluster - 1) / cluster;
        if (cluster > 1 && p.units * (cluster - 1) >= g.units) break;  // the last would be idle
        const int fixed = offsets<COLUMNS, GROUP>(p.units, 0, g.unit_bytes).end;
        p.ring = (SMEM_LIMIT - STATIC - fixed) / g.unit_bytes;
        if (fixed > SMEM_LIMIT - STATIC || p.ring < 4) continue;
        if (p.ring > MAX_RING) p.ring = MAX_RING;
        p.ring &= ~1;  // so that a slot's units are all one warpgroup's, which meets its phases in order
        p.smem = offsets<COLUMNS, GROUP>(p.units, p.ring, g.unit_bytes).end;
        const int slots = resident_clusters<q4_matmul_kernel<COLUMNS, GROUP, ZEROS>>(cluster, sm_count);
        p.clusters = g.tiles < slots ? g.tiles : slots;
        const int rounds = (g.tiles + p.clusters - 1) / p.clusters;
        const double shared = double(g.unit_bytes) * p.clusters * cluster / 3500.0;
        const double cost =
            rounds * (p.units * (shared > 600.0 ? shared : 600.0) + (cluster > 1 ? 1500.0 : 200.0)) +
            28.0 * COLUMNS * p.units;
        if (cost < best_cost) {
            best_cost = cost;
            *best = p;
        }
    }
    return best_cost < 1e30;
}

template <int COLUMNS, int GROUP, bool ZEROS>
cudaError_t launch_kernel(const Q4Product& args, int sm_count, cudaStream_t stream) {
    constexpr auto kernel = q4_matmul_kernel<COLUMNS, GROUP, ZEROS>;
    const cudaError_t err = set_smem_limit_once<kernel>(SMEM_LIMIT - 1024);
    if (err != cudaSuccess) return err;
    Plan plan;
    if (!make_plan<COLUMNS, GROUP, ZEROS>(args.geom, sm_count, &plan))
        return cudaErrorInvalidConfiguration;
    const int rows = COLUMNS / args.row_columns;
    cudaLaunchConfig_t config = {};
    config.gridDim = dim3(plan.clusters * plan.cluster, (args.M + rows - 1) / rows);
    config.blockDim = dim3(THREADS);
    config.dynamicSmemBytes = plan.smem;
    config.stream = stream;
    cudaLaunchAttribute attrs[2];
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = plan.cluster;
    attrs[1].val.clusterDim.y = 1;
    attrs[1].val.clusterDim.z = 1;
    config.attrs = attrs;
    config.numAttrs = plan.cluster > 1 ? 2 : 1;
    count_launch();
    return cudaLaunchKernelEx(&config, kernel, args, plan);
}

template <int COLUMNS>
cudaError_t launch(const Q4Product& args, int sm_count, cudaStream_t stream) {
    switch (args.geom.group + args.geom.zeros) {
        case 32: return launch_kernel<COLUMNS, 32, false>(args, sm_count, stream);
        case 33: return launch_kernel<COLUMNS, 32, true>(args, sm_count, stream);
        case 64: return launch_kernel<COLUMNS, 64, false>(args, sm_count, stream);
        case 65: return launch_kernel<COLUMNS, 64, true>(args, sm_count, stream);
        case 128: return launch_kernel<COLUMNS, 128, false>(args, sm_count, stream);
        default: return launch_kernel<COLUMNS, 128, true>(args, sm_count, stream);
    }
}

}  // namespace

cudaError_t launch_q4_tensor(const Q4Product& p, int most_columns, int sm_count, cudaStream_t stream) {
    if (most_columns >= 32) return launch<32>(p, sm_count, stream);
    if (most_columns >= 16) return launch<16>(p, sm_count, stream);
    return launch<8>(p, sm_count, stream);
}

}  // namespace sgemm
