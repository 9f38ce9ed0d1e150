// Few-row products with 4-bit weights: C[M x K] = A[M x N] . B, B in the packed format of
// q4.cuh. The bytes of B are the cost, so the kernel is built to keep HBM busy from its first
// to its last instruction and to spend few instructions on a weight:
//  * A "column" is a bfloat16 piece of a row of A (1, 2 or 3 a row); the CTA stages the
//    columns of its n range in shared memory once and keeps them for all its strips.
//  * 8 warps are split WN ways over n and 8 / WN ways over strips; a warp takes MT strips at
//    a time, so that a column's words serve MT instructions. Each warp streams its chunks
//    through a private ring of cp.async stages: no barrier stands between a load and its use,
//    and the ring runs on across strips while sums are exchanged.
//  * Sums of the n ranges are added in a fixed order, over warps in shared memory and, where
//    the strips alone would not fill the GPU (or the columns not fit), over a cluster's CTAs
//    through distributed shared memory: one launch, no workspace, no atomics.
#include "internal.cuh"
#include "q4.cuh"

namespace sgemm {
namespace {

constexpr int SMEM_LIMIT = 227 * 1024;  // of a CTA
constexpr int SMEM_SM = 228 * 1024;     // of an SM; 1 KB of each CTA's share is the system's

// Warps of a CTA: 8, or 16 where the columns of one CTA leave no room for a second.
template <int NT>
constexpr int max_warps() { return NT == 1 ? 8 : 16; }

template <int NT>
constexpr int min_blocks() { return NT == 1 ? 2 : 1; }

// Stages of a warp's ring: with 16 warps on an SM about 70 KB are in flight, twice what
// covers HBM's latency at its full rate.
template <int MT>
constexpr int depth() { return MT == 4 ? 3 : 4; }

struct Plan {
    int mt;       // strips that a warp takes at a time
    int warps;    // of a CTA
    int cluster;  // CTAs that split n
    int wn;       // warps of a CTA that split n
    int chunks;   // of a CTA's n range
    int groups;   // of warps / wn * MT strips
    int clusters; // launched
    int staged;   // columns that a CTA stages
    int smem;
};

struct Args {
    const void* A;
    size_t lda;
    int M, dtype, pieces;
    const uint8_t* data;
    Q4Geom geom;
    void* C;
    size_t ldc;
    Plan plan;
    bool vec;  // rows of A start on 16-byte boundaries
};

// Bytes of a column of `chunks` chunks in shared memory: 64 bytes more than a multiple of
// 256, so that the 8 lanes of a 16-byte load phase (4 words of two columns) meet no bank twice.
__host__ __device__ constexpr int column_pitch(int chunks) { return chunks * kQ4ChunkN * 2 + 64; }
// Floats of the sums of one group: [wn][strip][column][16], a column's 16 padded to 17.
__host__ __device__ constexpr int red_floats(int warps, int mt, int columns) {
    return warps * mt * columns * 17;
}
// Floats of the staged columns' sums over each group of n.
__host__ __device__ constexpr int xsum_floats(int chunks, int group, int nt) {
    return chunks * (kQ4ChunkN / group) * nt * 8;
}
// Floats of a CTA's part of a group's sums when a cluster shares it: [row][column of C].
__host__ __device__ constexpr int part_floats(int warps, int mt, int columns) {
    return warps * mt * kQ4StripK * columns;
}

// What a CTA stages of the columns: rows of A, n from n0 on, `units` of 8 values (a multiple
// of 16), and factor times their sums over each group of 8 << log_units values.
struct Staging {
    const void* A;
    size_t lda;
    int dtype, rows, n0, N, units, threads, pitch;
    bool vec;
    uint8_t* xs;
    float* xsum;  // [group][column], sum_pitch floats a group
    int sum_pitch, log_units;
    float factor;
};

// Writes the pieces of the rows, times scale, to their columns, and their sums; true where
// the plain form cannot take one of the thread's values. A group's units lie in neighbouring
// lanes of a warp, so that shuffles add them.
template <int P, class T>
__device__ __noinline__ bool stage_rows(const Staging& s, float scale) {
    constexpr int AHEAD = 4;  // loads in flight
    const T* A = static_cast<const T*>(s.A);
    const int items = s.units * s.rows, threads = s.threads;
    const int group_mask = (1 << s.log_units) - 1;
    int row = 0, u = threadIdx.x;
    bool special = false;
    for (int i = threadIdx.x; i - int(threadIdx.x & 31) < items; i += AHEAD * threads) {
        Raw8<T> raw[AHEAD];
        int rows_[AHEAD], units_[AHEAD];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            rows_[j] = -1;
            if (i + j * threads < items) {
                while (u >= s.units) {
                    u -= s.units;
                    ++row;
                }
                rows_[j] = row;
                units_[j] = u;
                raw[j] = load_raw8(A + row * s.lda, s.n0 + u * 8, s.N, s.vec);
                u += threads;
            }
        }
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            float sum[P];
#pragma unroll
            for (int p = 0; p < P; ++p) sum[p] = 0.0f;
            if (rows_[j] >= 0) {
                uint4 piece[P];
                split_raw8<P>(raw[j], scale, special, piece, sum);
#pragma unroll
                for (int p = 0; p < P; ++p)
                    *reinterpret_cast<uint4*>(s.xs + (rows_[j] * P + p) * s.pitch + units_[j] * 16) =
                        piece[p];
            }
            if (i - int(threadIdx.x & 31) + j * threads >= items) continue;  // warp-uniform
#pragma unroll
            for (int p = 0; p < P; ++p) {
                for (int o = 1; o <= group_mask; o *= 2)
                    sum[p] += __shfl_xor_sync(0xffffffffu, sum[p], o);
                if (rows_[j] >= 0 && (units_[j] & group_mask) == 0)
                    s.xsum[(units_[j] >> s.log_units) * s.sum_pitch + rows_[j] * P + p] =
                        sum[p] * s.factor;
            }
        }
    }
    return special;
}

__device__ __forceinline__ bool stage_any(const Staging& s, float scale) {
    if (s.dtype == SGEMM_BFLOAT16) return stage_rows<1, __nv_bfloat16>(s, scale);
    if (s.dtype == SGEMM_FLOAT16) return stage_rows<2, __half>(s, scale);
    return stage_rows<3, float>(s, scale);
}

// Stages the columns, scaled for the plain form; true where that form cannot take one of the
// values, and then they are staged as they are.
__device__ __noinline__ bool stage_columns(const Staging& s) {
    if (!__syncthreads_or(stage_any(s, kQ4Scale))) return false;
    stage_any(s, 1.0f);
    __syncthreads();
    return true;
}

// Where a CTA's shared memory holds what, in bytes; `columns`: those that it stages.
struct Offsets {
    int ring, red, xsum, part, end;
};
__host__ __device__ constexpr Offsets offsets(int warps, int mt, int depth, int chunk_bytes,
                                              int columns, int chunks, int group, int nt,
                                              bool cluster) {
    Offsets o{};
    o.ring = columns * column_pitch(chunks);
    o.red = o.ring + warps * depth * mt * chunk_bytes;
    o.xsum = o.red + red_floats(warps, mt, columns) * 4;
    o.part = o.xsum + xsum_floats(chunks, group, nt) * 4;
    o.end = o.part + (cluster ? 2 * part_floats(warps, mt, columns) * 4 : 0);
    return o;
}

template <int MT, int NT, int GROUP, bool ZEROS>
__global__ void __launch_bounds__(max_warps<NT>() * 32, min_blocks<NT>())
    q4_matmul_kernel(const Args args) {
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr int DEPTH = depth<MT>();
    const Plan& plan = args.plan;
    const Q4Geom& geom = args.geom;
    const int threads = plan.warps * 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = lane >> 2, c = lane & 3;
    const int wn = warp & (plan.wn - 1), wm = warp / plan.wn;
    const int strips_per_group = plan.warps / plan.wn * MT;  // a power of two
    const int rank = plan.cluster > 1 ? int(ptx::cluster_ctarank()) : 0;
    const int first_group = blockIdx.x / plan.cluster;
    const int chunk0 = rank * plan.chunks;
    const int chunks = max(0, min(plan.chunks, geom.chunks - chunk0));
    const int pieces = args.pieces, most_rows = NT * 8 / pieces;
    const int row0 = blockIdx.y * most_rows;
    const int rows = min(most_rows, args.M - row0), columns = rows * pieces;

    const int pitch = column_pitch(plan.chunks);
    const int chunk_bytes = geom.chunk_bytes, stage_bytes = MT * chunk_bytes;
    uint8_t* xs = smem;
    const Offsets at = offsets(plan.warps, MT, DEPTH, chunk_bytes, plan.staged, plan.chunks, GROUP,
                               NT, plan.cluster > 1);
    uint8_t* ring = smem + at.ring + warp * DEPTH * stage_bytes;
    float* red = reinterpret_cast<float*>(smem + at.red);
    float* xsum = reinterpret_cast<float*>(smem + at.xsum);  // [group of n][column]
    float* part = reinterpret_cast<float*>(smem + at.part);  // only with a cluster

    // The warp's sequence: for each of the CTA's groups, chunks wn, wn + WN, ... of the range.
    // Strips past the last one are not fetched; what is computed for them is not used.
    const int my_chunks = wn < chunks ? (chunks - wn + plan.wn - 1) / plan.wn : 0;
    const bool tail = kQ4CodeBytes + lane * 16 < chunk_bytes;
    const uint32_t step = plan.wn * chunk_bytes;
    const int strip_step = plan.clusters * strips_per_group;
    const size_t wrap = size_t(strip_step) * geom.strip_bytes() - size_t(my_chunks) * step;
    int fetch_strip = my_chunks > 0 ? first_group * strips_per_group + wm * MT : geom.strips;
    const uint8_t* fetch_from = args.data + size_t(fetch_strip) * geom.strip_bytes() +
                                size_t(chunk0 + wn) * chunk_bytes + lane * 16;
    int fetch_left = my_chunks;
    uint32_t fetch_to = ptx::smem_u32(ring) + lane * 16;
    const uint32_t fetch_end = fetch_to + DEPTH * stage_bytes;
    auto fetch = [&]() {
        if (fetch_strip < geom.strips) {
            q4_fetch(fetch_to, fetch_from, tail);
#pragma unroll
            for (int m = 1; m < MT; ++m)
                if (fetch_strip + m < geom.strips)
                    q4_fetch(fetch_to + m * chunk_bytes, fetch_from + m * geom.strip_bytes(), tail);
            fetch_from += step;
            if (--fetch_left == 0) {
                fetch_left = my_chunks;
                fetch_from += wrap;
                fetch_strip += strip_step;
            }
        }
        ptx::cp_async_commit();
        fetch_to += stage_bytes;
        if (fetch_to == fetch_end) fetch_to -= DEPTH * stage_bytes;
    };
    // Nothing in global memory is touched before the kernels ahead in the stream are done; the
    // next one may take its place on SMs as they come free.
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
#pragma unroll
    for (int i = 0; i < DEPTH - 1; ++i) fetch();

    Staging st;
    st.A = static_cast<const uint8_t*>(args.A) + row0 * args.lda * dtype_bytes(args.dtype);
    st.lda = args.lda;
    st.dtype = args.dtype;
    st.rows = rows;
    st.n0 = chunk0 * kQ4ChunkN;
    st.N = geom.N;
    st.units = chunks * (kQ4ChunkN / 8);
    st.threads = threads;
    st.pitch = pitch;
    st.vec = args.vec;
    st.xs = xs;
    st.xsum = xsum;
    st.sum_pitch = NT * 8;
    st.log_units = GROUP == 32 ? 2 : GROUP == 64 ? 3 : 4;
    st.factor = ZEROS ? -1.0f : -8.0f;
    const bool special = stage_columns(st);

    // a lane's words of column 8 nt + r in the warp's first chunk; columns that do not exist
    // repeat the last one, and their sums are not used
    uint32_t xcol[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
        xcol[nt] = min(nt * 8 + r, columns - 1) * pitch + c * 16 + wn * (kQ4ChunkN * 2);
    const float* sums0 = xsum + wn * (kQ4ChunkN / GROUP) * (NT * 8) + 2 * c;

    const uint8_t* stage = ring;
    const uint8_t* const ring_end = ring + DEPTH * stage_bytes;
    const int width_log = __ffs(strips_per_group * kQ4StripK) - 1;
    const int cells = rows << width_log;
    int buffer = 0;
    for (int group = first_group; group < plan.groups; group += plan.clusters) {
        float total[MT][NT][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) total[m][nt][i] = 0.0f;
        const uint8_t* x = xs;
        const float* sums = sums0;
        auto next = [&]() {
            x += plan.wn * (kQ4ChunkN * 2);
            sums += plan.wn * (kQ4ChunkN / GROUP) * (NT * 8);
            stage += stage_bytes;
            if (stage == ring_end) stage = ring;
        };
        if (special) {
#pragma unroll 1
            for (int i = 0; i < my_chunks; ++i, next()) {
                ptx::cp_async_wait<DEPTH - 2>();
                __syncwarp();
                fetch();
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        q4_chunk_centred<GROUP, ZEROS>(stage + m * chunk_bytes, x + xcol[nt],
                                                       geom.fp16, lane, total[m][nt]);
            }
        } else {
#pragma unroll 1
            for (int i = 0; i < my_chunks; ++i, next()) {
                ptx::cp_async_wait<DEPTH - 2>();
                __syncwarp();
                fetch();
                q4_chunk<MT, NT, GROUP, ZEROS>(
                    [&](int m) { return stage + m * chunk_bytes; }, geom.fp16, lane,
                    [&](int b, int nt) {
                        return *reinterpret_cast<const uint4*>(x + xcol[nt] + b * 64);
                    },
                    [&](int g, int nt) {
                        return *reinterpret_cast<const float2*>(sums + g * (NT * 8) + nt * 8);
                    },
                    total);
            }
        }
        // Sums over the warps that split n, in their order
        if (group != first_group) __syncthreads();
        float* mine = red + (wn * strips_per_group + wm * MT) * columns * 17 + r;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int col = nt * 8 + 2 * c + i;
                if (col >= columns) continue;
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    mine[(m * columns + col) * 17] = total[m][nt][i];
                    mine[(m * columns + col) * 17 + 8] = total[m][nt][i + 2];
                }
            }
        __syncthreads();
        const int k0 = group << width_log;
        const int wn_stride = strips_per_group * columns * 17;
        float* shared_sums = part + buffer * part_floats(plan.warps, MT, plan.staged);
        auto put = [&](int i, float v) {
            const int row = i >> width_log, k = k0 + i - (row << width_log);
            if (k < geom.K) store_from_float(args.C, args.dtype, (row0 + row) * args.ldc + k, v);
        };
        for (int i = threadIdx.x; i < cells; i += threads) {
            const int row = i >> width_log, col = i - (row << width_log);
            const float* from =
                red + ((col / kQ4StripK) * columns + row * pieces) * 17 + col % kQ4StripK;
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
            ptx::cluster_sync();
            // each CTA adds the ranges' sums of its share of the cells, in rank order
            const int share = (cells + plan.cluster - 1) / plan.cluster;
            const uint32_t base = ptx::smem_u32(shared_sums);
            for (int i = rank * share + threadIdx.x; i < min(cells, (rank + 1) * share);
                 i += threads) {
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

constexpr double kNoPlan = 1e30;

// Clusters of this size that the device holds at once, `resident` CTAs an SM.
template <auto KERNEL>
int resident_clusters(int cluster, int resident, int threads, int sm_count) {
    if (cluster == 1) return sm_count * resident;
    constexpr int kDevices = 64;
    static std::atomic<int> known[kDevices][3][3];
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
    config.blockDim = dim3(threads);
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

// The split of an N x K product with this many columns: the warps, cluster size and warp split
// whose slowest SM is done first.
template <int MT, int NT, int GROUP, bool ZEROS>
void make_plan(const Q4Geom& g, int columns, int sm_count, double* best_cost, Plan* best) {
    constexpr int DEPTH = depth<MT>();
    if (set_smem_limit_once<q4_matmul_kernel<MT, NT, GROUP, ZEROS>>(SMEM_LIMIT) != cudaSuccess) return;
    for (int warps = 8; warps <= max_warps<NT>(); warps *= 2)
        for (int cluster = 1; cluster <= 8; cluster *= 2) {
            if (cluster > 1 && g.chunks < 2 * cluster) break;
            for (int wn = warps; wn >= 1; wn /= 2) {
                Plan p;
                p.mt = MT;
                p.warps = warps;
                p.cluster = cluster;
                p.wn = wn;
                p.chunks = (g.chunks + cluster - 1) / cluster;
                if (wn > 1 && wn > p.chunks) continue;
                p.staged = columns;
                p.smem = offsets(warps, MT, DEPTH, g.chunk_bytes, columns, p.chunks, GROUP, NT,
                                 cluster > 1)
                             .end;
                if (p.smem > SMEM_LIMIT) continue;
                int resident = 1;
                while (resident < (16 / warps) &&
                       (p.smem + 1024) * (resident + 1) <= SMEM_SM)
                    ++resident;
                const int strips = warps / wn * MT;
                p.groups = (g.strips + strips - 1) / strips;
                const int slots = resident_clusters<q4_matmul_kernel<MT, NT, GROUP, ZEROS>>(
                    cluster, resident, warps * 32, sm_count);
                p.clusters = p.groups < slots ? p.groups : slots;
                const int rounds = (p.groups + p.clusters - 1) / p.clusters;
                const int units = (p.chunks + wn - 1) / wn * MT;  // of a warp and group
                const int busy = (p.clusters * cluster + sm_count - 1) / sm_count;
                const double chunk_cost = busy * warps > 8 ? 45.0 : 70.0;
                const double stage = busy * 3.0 * columns * p.chunks + 1500.0;
                const double cost = stage + rounds * (busy * warps * units * chunk_cost + 300.0 +
                                              (wn - 1) * MT * 60.0 + (cluster > 1 ? 500.0 : 0.0));
                if (cost < *best_cost) {
                    *best_cost = cost;
                    *best = p;
                }
            }
        }
}

template <int MT, int NT, int GROUP, bool ZEROS>
cudaError_t launch_kernel(const Args& args, int launch_rows, cudaStream_t stream) {
    cudaLaunchConfig_t config = {};
    config.gridDim = dim3(args.plan.clusters * args.plan.cluster, launch_rows);
    config.blockDim = dim3(args.plan.warps * 32);
    config.dynamicSmemBytes = args.plan.smem;
    config.stream = stream;
    cudaLaunchAttribute attrs[2];
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = args.plan.cluster;
    attrs[1].val.clusterDim.y = 1;
    attrs[1].val.clusterDim.z = 1;
    config.attrs = attrs;
    config.numAttrs = args.plan.cluster > 1 ? 2 : 1;
    count_launch();
    return cudaLaunchKernelEx(&config, q4_matmul_kernel<MT, NT, GROUP, ZEROS>, args);
}

template <int NT, int GROUP, bool ZEROS>
cudaError_t launch_group(Args args, int sm_count, cudaStream_t stream) {
    const int most_rows = NT * 8 / args.pieces;
    const int launch_rows = (args.M + most_rows - 1) / most_rows;
    const int columns = (args.M < most_rows ? args.M : most_rows) * args.pieces;
    // one strip a warp only where a product is small: its columns' words serve once
    constexpr int LEAST = NT == 1 ? 1 : 2, MOST = NT == 4 ? 2 : 4;
    double cost = kNoPlan;
    args.plan = Plan{};
    if constexpr (LEAST <= 1) make_plan<1, NT, GROUP, ZEROS>(args.geom, columns, sm_count, &cost, &args.plan);
    make_plan<2, NT, GROUP, ZEROS>(args.geom, columns, sm_count, &cost, &args.plan);
    if constexpr (MOST >= 4) make_plan<4, NT, GROUP, ZEROS>(args.geom, columns, sm_count, &cost, &args.plan);
    if (cost >= kNoPlan) return cudaErrorInvalidConfiguration;
    if constexpr (LEAST <= 1)
        if (args.plan.mt == 1) return launch_kernel<1, NT, GROUP, ZEROS>(args, launch_rows, stream);
    if constexpr (MOST >= 4)
        if (args.plan.mt == 4) return launch_kernel<4, NT, GROUP, ZEROS>(args, launch_rows, stream);
    return launch_kernel<2, NT, GROUP, ZEROS>(args, launch_rows, stream);
}

template <int NT>
cudaError_t launch(const Args& args, int sm_count, cudaStream_t stream) {
    switch (args.geom.group + args.geom.zeros) {
        case 32: return launch_group<NT, 32, false>(args, sm_count, stream);
        case 33: return launch_group<NT, 32, true>(args, sm_count, stream);
        case 64: return launch_group<NT, 64, false>(args, sm_count, stream);
        case 65: return launch_group<NT, 64, true>(args, sm_count, stream);
        case 128: return launch_group<NT, 128, false>(args, sm_count, stream);
        default: return launch_group<NT, 128, true>(args, sm_count, stream);
    }
}

}  // namespace
}  // namespace sgemm

using namespace sgemm;

extern "C" int sgemm_q4_matmul(const void* A, int dtype, long long lda, int M, const sgemm_q4* w,
                               void* C, long long ldc, void* stream) {
    if (!q4_valid(w) || w->count != 1 || !w->data || !aligned16(w->data)) return SGEMM_ERR_ARG;
    if (!dtype_valid(dtype) || M < 0 || M > 65536 || lda < w->N || ldc < w->K) return SGEMM_ERR_ARG;
    if (lda > (1ll << 40) || ldc > (1ll << 40)) return SGEMM_ERR_ARG;
    if (M == 0) return SGEMM_OK;
    if (!A || !C) return SGEMM_ERR_ARG;
    const size_t size = dtype_bytes(dtype);
    if (reinterpret_cast<uintptr_t>(A) % size || reinterpret_cast<uintptr_t>(C) % size)
        return SGEMM_ERR_ARG;
    const size_t a_bytes = (size_t(M - 1) * lda + w->N) * size;
    const size_t c_bytes = (size_t(M - 1) * ldc + w->K) * size;
    if (ranges_overlap(C, c_bytes, A, a_bytes) ||
        ranges_overlap(C, c_bytes, w->data, q4_bytes(*w)))
        return SGEMM_ERR_OVERLAP;
    const DeviceInfo* info = current_device(nullptr);
    if (!info) return SGEMM_ERR_NO_DEVICE;
    Args args;
    args.A = A;
    args.lda = size_t(lda);
    args.M = M;
    args.dtype = dtype;
    args.pieces = pieces_of(dtype);
    args.data = static_cast<const uint8_t*>(w->data);
    args.geom = q4_geom(*w);
    args.C = C;
    args.ldc = size_t(ldc);
    args.vec = aligned16(A) && size_t(lda) * size % 16 == 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // few enough columns at a time that a cluster's shared memory holds them (8 always fit)
    const int columns = M * args.pieces;
    cudaError_t err = cudaErrorInvalidConfiguration;
    if (columns > 16) err = launch<4>(args, info->sm_count, s);
    if (columns > 8 && err == cudaErrorInvalidConfiguration) err = launch<2>(args, info->sm_count, s);
    if (err == cudaErrorInvalidConfiguration) err = launch<1>(args, info->sm_count, s);
    return err == cudaSuccess ? SGEMM_OK : SGEMM_ERR_CUDA;
}
