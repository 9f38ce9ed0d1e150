// Few-row products with 4-bit weights for up to 8 columns (bfloat16 pieces of rows of A). The
// bytes of B are the cost, so the kernel is built to keep HBM busy from its first to its last
// instruction:
//  * A CTA stages the columns of its n range in shared memory once and keeps them for all its
//    strips of 16 columns of C.
//  * 8 warps are split WN ways over n and 8 / WN ways over strips; a warp takes MT strips at a
//    time, so that a column's words serve MT instructions. Each warp streams its chunks (a
//    strip's part of a unit) through a private ring of cp.async stages: no barrier stands between
//    a load and its use, and the ring runs on across strips while sums are exchanged.
//  * Sums of the n ranges are added in a fixed order, over warps in shared memory and, where
//    the strips alone would not fill the GPU (or the columns not fit), over a cluster's CTAs
//    through distributed shared memory: one launch, no workspace, no atomics.
//
// Measured, one row: 8192 x 65536 columns, bfloat16, group 128, 51 us (5.4 TB/s, 81 % of a copy);
// 8192 x 8192 10.9 us; 6144 x 4096 in float32 7.2; 512 x 512 3.1, which is a launch and two trips to
// memory. What bounds it between these: staging and the first loads' latency, some 3 us, and with
// 8 columns the instructions of a chunk (76 us at 65536 columns).
#include <atomic>

#include "q4_stage.cuh"
#include "q4_warp.cuh"

namespace sgemm {
namespace {

constexpr int COLUMNS = 8;
constexpr int WARPS = 8, THREADS = WARPS * 32;
constexpr int SMEM_LIMIT = 227 * 1024;  // of a CTA
constexpr int SMEM_SM = 228 * 1024;     // of an SM; 1 KB of each CTA's share is the system's
constexpr int MOST_RESIDENT = 2;        // CTAs of an SM: 128 registers a thread

// Stages of a warp's ring: with 16 warps on an SM 50 to 130 KB are in flight; 35 KB cover HBM's
// latency at its full rate.
template <int MT>
constexpr int depth() { return MT == 4 ? 3 : 4; }

struct Plan {
    int mt;        // strips that a warp takes at a time
    int cluster;   // CTAs that split n
    int wn;        // warps of a CTA that split n
    int units;     // of a CTA's n range
    int groups;    // of WARPS / wn * MT strips
    int clusters;  // launched
    int staged;    // columns that a CTA stages
    int smem;
};

// Bytes of a column of so many units in shared memory: 64 bytes more than a multiple of 256, so
// that the 8 lanes of a 16-byte load phase (4 words of two columns) meet no bank twice.
__host__ __device__ constexpr int column_pitch(int units) { return units * kQ4UnitN * 2 + 64; }

// Where a CTA's shared memory holds what, in bytes; `staged`: columns.
struct Offsets {
    int ring;  // [warp][stage]
    int red;   // sums of one group of strips: [wn][strip][column][16, padded to 17]
    int xsum;  // the columns' sums: [group of n][column]
    int part;  // this CTA's part of a group's sums, twice, only with a cluster: [row][column of C]
    int part_floats;
    int end;
};
template <int MT, int GROUP, bool ZEROS>
__host__ __device__ constexpr Offsets offsets(int staged, int units, bool cluster) {
    Offsets o{};
    o.ring = staged * column_pitch(units);
    o.red = o.ring + WARPS * depth<MT>() * MT * q4_chunk_bytes(GROUP, ZEROS);
    o.xsum = o.red + WARPS * MT * staged * 17 * 4;
    o.part = o.xsum + units * (kQ4UnitN / GROUP) * COLUMNS * 4;
    o.part_floats = WARPS * MT * kQ4StripK * staged;
    o.end = o.part + (cluster ? 2 * o.part_floats * 4 : 0);
    return o;
}

template <int MT, int GROUP, bool ZEROS>
__global__ void __launch_bounds__(THREADS, MOST_RESIDENT)
    q4_warp_kernel(const Q4Product args, const Plan plan) {
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr int DEPTH = depth<MT>();
    constexpr int CHUNK = q4_chunk_bytes(GROUP, ZEROS), STAGE = MT * CHUNK;
    constexpr int GROUPS = kQ4UnitN / GROUP;
    const Q4Geom& geom = args.geom;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = lane >> 2, c = lane & 3;
    const int wn = warp & (plan.wn - 1), wm = warp / plan.wn;
    const int strips_per_group = WARPS / plan.wn * MT;  // a power of two
    const int strips = (geom.K + kQ4StripK - 1) / kQ4StripK;
    const int rank = plan.cluster > 1 ? int(ptx::cluster_ctarank()) : 0;
    const int first_group = blockIdx.x / plan.cluster;
    const int unit0 = rank * plan.units;
    const int units = max(0, min(plan.units, geom.units - unit0));
    const int rows = args.M, columns = plan.staged;

    const int pitch = column_pitch(plan.units);
    const Offsets at = offsets<MT, GROUP, ZEROS>(plan.staged, plan.units, plan.cluster > 1);
    uint8_t* xs = smem;
    uint8_t* ring = smem + at.ring + warp * DEPTH * STAGE;
    float* red = reinterpret_cast<float*>(smem + at.red);
    float* xsum = reinterpret_cast<float*>(smem + at.xsum);
    float* part = reinterpret_cast<float*>(smem + at.part);

    // The warp's sequence: for each of the CTA's groups, units wn, wn + WN, ... of the range.
    // Strips past the last one are not fetched; what is computed for them is not used.
    const int my_units = wn < units ? (units - wn + plan.wn - 1) / plan.wn : 0;
    const Q4Side side = q4_side<GROUP, ZEROS>(lane);
    const size_t step = size_t(plan.wn) * geom.unit_bytes;
    const int strip_step = plan.clusters * strips_per_group;
    int fetch_strip = my_units > 0 ? first_group * strips_per_group + wm * MT : strips;
    const uint8_t* fetch_from = nullptr;
    int fetch_left = 0;
    const uint32_t ring_u32 = ptx::smem_u32(ring);
    uint32_t fetch_to = ring_u32;
    auto fetch = [&]() {
        if (fetch_strip < strips) {
            if (fetch_left == 0) {
                fetch_left = my_units;
                fetch_from = args.data + size_t(fetch_strip / kQ4StripsOfTile) * geom.tile_bytes() +
                             size_t(unit0 + wn) * geom.unit_bytes;
            }
            q4_fetch<MT>(fetch_to, CHUNK, fetch_from, fetch_strip % kQ4StripsOfTile,
                         strips - fetch_strip, lane, side);
            fetch_from += step;
            if (--fetch_left == 0) fetch_strip += strip_step;
        }
        ptx::cp_async_commit();
        fetch_to += STAGE;
        if (fetch_to == ring_u32 + DEPTH * STAGE) fetch_to = ring_u32;
    };
    // Nothing in global memory is touched before the kernels ahead in the stream are done; the
    // next one may take its place on SMs as they come free.
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
#pragma unroll 1
    for (int i = 0; i < DEPTH - 1; ++i) fetch();

    Staging st;
    st.A = args.A;
    st.lda = args.lda;
    st.dtype = args.dtype;
    st.rows = rows;
    st.n0 = unit0 * kQ4UnitN;
    st.N = geom.N;
    st.octets = units * (kQ4UnitN / 8);
    st.threads = THREADS;
    st.vec = args.vec;
    st.xs = xs;
    st.octet_stride = 16;
    st.column_stride = pitch;
    st.xsum = xsum;
    st.sum_pitch = COLUMNS;
    st.log_octets = GROUP == 32 ? 2 : GROUP == 64 ? 3 : 4;
    st.factor = ZEROS ? -1.0f : -8.0f;
    st.turn = first_group;
    st.turns = plan.clusters;
    const bool special = stage_columns(st);

    // a lane's words of column r in the warp's first unit; columns that do not exist repeat the
    // last one, and their sums are not used
    const int xcol = min(r, columns - 1) * pitch + c * 16 + wn * (kQ4UnitN * 2);
    const float* sums0 = xsum + wn * GROUPS * COLUMNS + 2 * c;

    const uint8_t* stage = ring;
    const uint8_t* const ring_end = ring + DEPTH * STAGE;
    const int width_log = __ffs(strips_per_group * kQ4StripK) - 1;
    const int cells = rows << width_log;
    int buffer = 0;
    for (int group = first_group; group < plan.groups; group += plan.clusters) {
        float total[MT][1][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) total[m][0][i] = 0.0f;
        const uint8_t* x = xs + xcol;
        const float* sums = sums0;
        auto next = [&]() {
            x += plan.wn * (kQ4UnitN * 2);
            sums += plan.wn * GROUPS * COLUMNS;
            stage += STAGE;
            if (stage == ring_end) stage = ring;
        };
        auto word = [&](int b) { return *reinterpret_cast<const uint4*>(x + b * 64); };
        auto sum = [&](int g) { return *reinterpret_cast<const float2*>(sums + g * COLUMNS); };
        if (special) {
#pragma unroll 1
            for (int i = 0; i < my_units; ++i, next()) {
                ptx::cp_async_wait<DEPTH - 2>();
                __syncwarp();
                fetch();
#pragma unroll
                for (int m = 0; m < MT; ++m)
                    q4_chunk_centred<GROUP, ZEROS>(stage + m * CHUNK, geom.fp16, lane, word,
                                                   sum, total[m][0]);
            }
        } else {
#pragma unroll 1
            for (int i = 0; i < my_units; ++i, next()) {
                ptx::cp_async_wait<DEPTH - 2>();
                __syncwarp();
                fetch();
                q4_chunk<MT, 1, GROUP, ZEROS>(
                    [&](int m) { return stage + m * CHUNK; }, geom.fp16, lane,
                    [&](int b, int) { return word(b); }, [&](int g, int) { return sum(g); },
                    total);
            }
        }
        // sums over the warps that split n, in their order
        if (group != first_group) __syncthreads();
        float* mine = red + (wn * strips_per_group + wm * MT) * columns * 17 + r;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (2 * c + i < columns) {
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    mine[(m * columns + 2 * c + i) * 17] = total[m][0][i];
                    mine[(m * columns + 2 * c + i) * 17 + 8] = total[m][0][i + 2];
                }
            }
        __syncthreads();
        const int k0 = group << width_log;
        const int wn_stride = strips_per_group * columns * 17;
        float* shared_sums = part + buffer * at.part_floats;
        auto put = [&](int i, float v) {
            const int row = i >> width_log, k = k0 + i - (row << width_log);
            if (k < geom.K) store_from_float(args.C, args.dtype, row * args.ldc + k, v);
        };
        const int pieces = args.row_columns == 4 ? 3 : args.row_columns;
        for (int i = threadIdx.x; i < cells; i += THREADS) {
            const int row = i >> width_log, col = i - (row << width_log);
            const float* from =
                red + ((col / kQ4StripK) * columns + row * args.row_columns) * 17 + col % kQ4StripK;
            float s = 0.0f;
            for (int p = 0; p < pieces; ++p, from += 17)
#pragma unroll 8
                for (int w = 0; w < plan.wn; ++w) s += from[w * wn_stride];
            if (plan.cluster > 1)
                shared_sums[i] = s;
            else
                put(i, s);
        }
        if (plan.cluster > 1) {
            // two buffers in turn: a CTA is back at one of them only after the barrier that
            // follows the others' reading of it
            ptx::cluster_sync();
            // each CTA adds the ranges' sums of its share of the cells, in rank order
            const int share = (cells + plan.cluster - 1) / plan.cluster;
            const uint32_t base = ptx::smem_u32(shared_sums);
            for (int i = rank * share + threadIdx.x; i < min(cells, (rank + 1) * share);
                 i += THREADS) {
                float s = 0.0f;
                for (int q = 0; q < plan.cluster; ++q)
                    s += ptx::ld_shared_cluster_f32(ptx::mapa_shared(base + i * 4, q));
                put(i, s);
            }
        }
        buffer ^= 1;
    }
    ptx::cp_async_wait<0>();
    // a CTA's shared memory is read by the others until here
    if (plan.cluster > 1) ptx::cluster_sync();
}

// Clusters of this size that the device holds at once, `resident` CTAs an SM.
template <auto KERNEL>
int resident_clusters(int cluster, int resident, int sm_count) {
    if (cluster == 1) return sm_count * resident;
    constexpr int kDevices = 64;
    static std::atomic<int> known[kDevices][3][MOST_RESIDENT];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) dev = 0;
    std::atomic<int>& slot = known[dev][cluster == 2 ? 0 : cluster == 4 ? 1 : 2][resident - 1];
    int n = slot.load(std::memory_order_relaxed);
    if (n > 0) return n;
    cudaLaunchConfig_t config = {};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    config.gridDim = dim3(sm_count / cluster * cluster * resident);
    config.blockDim = dim3(THREADS);
    config.dynamicSmemBytes = resident == 1 ? SMEM_LIMIT : SMEM_SM / resident - 1024;
    config.attrs = &attr;
    config.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, KERNEL, &config) != cudaSuccess || n < 1) {
        cudaGetLastError();
        n = sm_count * resident / cluster;
        if (n < 1) n = 1;
    }
    slot.store(n, std::memory_order_relaxed);
    return n;
}

// The split of the product for this MT: the cluster size and warp split whose slowest SM is done
// first. In cycles: a chunk takes an SM 46 with 16 warps on it and 72 with 8, a fifth more where
// a column's words serve one strip; staging and exchanging sums take some hundreds each.
template <int MT, int GROUP, bool ZEROS>
void make_plan(const Q4Geom& g, int columns, int sm_count, double* best_cost, Plan* best) {
    constexpr auto kernel = q4_warp_kernel<MT, GROUP, ZEROS>;
    if (set_smem_limit_once<kernel>(SMEM_LIMIT) != cudaSuccess) return;
    const int all_strips = (g.K + kQ4StripK - 1) / kQ4StripK;
    for (int cluster = 1; cluster <= 8; cluster *= 2) {
        if (cluster > 1 && g.units < 2 * cluster) break;
        for (int wn = WARPS; wn >= 1; wn /= 2) {
            Plan p;
            p.mt = MT;
            p.cluster = cluster;
            p.wn = wn;
            p.units = (g.units + cluster - 1) / cluster;
            if (wn > 1 && wn > p.units) continue;
            p.staged = columns;
            p.smem = offsets<MT, GROUP, ZEROS>(columns, p.units, cluster > 1).end;
            if (p.smem > SMEM_LIMIT) continue;
            int resident = 1;
            while (resident < MOST_RESIDENT && (p.smem + 1024) * (resident + 1) <= SMEM_SM) ++resident;
            const int strips = WARPS / wn * MT;
            p.groups = (all_strips + strips - 1) / strips;
            const int slots = resident_clusters<kernel>(cluster, resident, sm_count);
            p.clusters = p.groups < slots ? p.groups : slots;
            const int rounds = (p.groups + p.clusters - 1) / p.clusters;
            const int chunks = (p.units + wn - 1) / wn * MT;  // of a warp and group
            const int busy = (p.clusters * cluster + sm_count - 1) / sm_count;
            const double chunk = (busy > 1 ? 46.0 : 72.0) * (MT == 1 ? 1.2 : 1.0);
            const double cost = busy * 8.0 * columns * p.units + (cluster > 1 ? 1200.0 : 0.0) +
                                rounds * (busy * WARPS * chunks * chunk + 400.0 + (wn - 1) * MT * 30.0 +
                                          (cluster > 1 ? 500.0 : 0.0));
            if (cost < *best_cost) {
                *best_cost = cost;
                *best = p;
            }
        }
    }
}

template <int MT, int GROUP, bool ZEROS>
cudaError_t launch_kernel(const Q4Product& args, const Plan& plan, cudaStream_t stream) {
    cudaLaunchConfig_t config = {};
    config.gridDim = dim3(plan.clusters * plan.cluster);
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
    return cudaLaunchKernelEx(&config, q4_warp_kernel<MT, GROUP, ZEROS>, args, plan);
}

template <int GROUP, bool ZEROS>
cudaError_t launch_group(const Q4Product& args, int sm_count, cudaStream_t stream) {
    // A plan depends on sizes and the device alone, and looking for one costs some microseconds of
    // host time, as much as a small product: each thread keeps those of its latest sizes.
    struct Known {
        int N, K, columns, device;
        Plan plan;
    };
    constexpr int PLANS = 64;
    static thread_local Known known[PLANS];  // mt 0: none
    const int columns = args.M * args.row_columns;
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess) return cudaErrorInvalidDevice;
    Known& slot = known[(unsigned(args.geom.N) * 31u + unsigned(args.geom.K) * 7u + columns) % PLANS];
    if (slot.plan.mt == 0 || slot.N != args.geom.N || slot.K != args.geom.K ||
        slot.columns != columns || slot.device != device) {
        double cost = 1e30;
        Plan plan{};
        make_plan<1, GROUP, ZEROS>(args.geom, columns, sm_count, &cost, &plan);
        make_plan<2, GROUP, ZEROS>(args.geom, columns, sm_count, &cost, &plan);
        make_plan<4, GROUP, ZEROS>(args.geom, columns, sm_count, &cost, &plan);
        slot = Known{args.geom.N, args.geom.K, columns, device, plan};
    }
    const Plan& plan = slot.plan;
    if (plan.mt == 1) return launch_kernel<1, GROUP, ZEROS>(args, plan, stream);
    if (plan.mt == 2) return launch_kernel<2, GROUP, ZEROS>(args, plan, stream);
    if (plan.mt == 4) return launch_kernel<4, GROUP, ZEROS>(args, plan, stream);
    return cudaErrorInvalidConfiguration;
}

}  // namespace

cudaError_t launch_q4_warp(const Q4Product& args, int sm_count, cudaStream_t stream) {
    switch (args.geom.group + args.geom.zeros) {
        case 32: return launch_group<32, false>(args, sm_count, stream);
        case 33: return launch_group<32, true>(args, sm_count, stream);
        case 64: return launch_group<64, false>(args, sm_count, stream);
        case 65: return launch_group<64, true>(args, sm_count, stream);
        case 128: return launch_group<128, false>(args, sm_count, stream);
        default: return launch_group<128, true>(args, sm_count, stream);
    }
}

}  // namespace sgemm
