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

constexpr int WARPS = 8;
constexpr int THREADS = WARPS * 32;
constexpr int DEPTH = 6;         // stages of a warp's ring
constexpr int SMEM_LIMIT = 227 * 1024;
constexpr int SMEM_HALF = 113 * 1024;  // two CTAs on an SM

struct Plan {
    int cluster;       // CTAs that split n
    int wn;            // warps of a CTA that split n
    int chunks;        // of a CTA's n range
    int window;        // chunks whose columns are staged at a time (a multiple of wn, or all)
    int groups;        // of WARPS / wn * MT strips
    int clusters;      // launched
    int staged;        // columns that a CTA stages
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
    bool vec;          // rows of A start on 16-byte boundaries
};

// Bytes of a column of `chunks` chunks in shared memory: 64 bytes more than a multiple of
// 256, so that the 8 lanes of a 16-byte load phase (4 words of two columns) meet no bank twice.
__host__ __device__ constexpr int column_pitch(int chunks) { return chunks * kQ4ChunkN * 2 + 64; }
// Floats of a CTA's part of a group's sums when a cluster shares it: [row][column of C].
__host__ __device__ constexpr int part_floats(int mt, int nt) {
    return WARPS * mt * kQ4StripK * nt * 8;
}
// Floats of the sums of one group: [wn][strip][column][16], a column's 16 padded to 17.
__host__ __device__ constexpr int red_floats(int mt, int nt) { return WARPS * mt * nt * 8 * 17; }

template <int MT, int NT, int GROUP>
__global__ void __launch_bounds__(THREADS, 2) q4_matmul_kernel(const Args args) {
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr int STAGE = MT * kQ4MaxChunk;
    const Plan& plan = args.plan;
    const Q4Geom& geom = args.geom;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = lane >> 2, c = lane & 3;
    const int wn = warp % plan.wn, wm = warp / plan.wn;
    const int strips_per_group = WARPS / plan.wn * MT;
    const int rank = plan.cluster > 1 ? int(ptx::cluster_ctarank()) : 0;
    const int first_group = blockIdx.x / plan.cluster;
    const int chunk0 = rank * plan.chunks;
    const int chunks = max(0, min(plan.chunks, geom.chunks - chunk0));
    // this launch row's share of the rows of A
    const int pieces = args.pieces, most_rows = NT * 8 / pieces;
    const int row0 = blockIdx.y * most_rows;
    const int rows = min(most_rows, args.M - row0), columns = rows * pieces;

    const int pitch = column_pitch(plan.window);
    uint8_t* xs = smem;
    uint8_t* ring = xs + plan.staged * pitch + warp * DEPTH * STAGE;
    float* red = reinterpret_cast<float*>(xs + plan.staged * pitch + WARPS * DEPTH * STAGE);
    float* part = red + 2 * red_floats(MT, NT);  // only with a cluster
    const uint32_t ring_u32 = ptx::smem_u32(ring);

    // the warp's sequence: for each of the CTA's groups, chunks wn, wn + WN, ... of the range
    int fetch_group = first_group, fetch_chunk = wn;
    auto fetch = [&](int stage) {
        if (fetch_group < plan.groups && wn < chunks) {
            const uint8_t* src[MT];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                // past the last strip: the last one again, its sums are not used
                const int strip =
                    min(fetch_group * strips_per_group + wm * MT + m, geom.strips - 1);
                src[m] = args.data + strip * geom.strip_bytes() +
                         size_t(chunk0 + fetch_chunk) * geom.chunk_bytes;
            }
            q4_fetch<MT>(ring_u32 + stage * STAGE, src, geom.chunk_bytes, lane);
            fetch_chunk += plan.wn;
            if (fetch_chunk >= chunks) {
                fetch_chunk = wn;
                fetch_group += plan.clusters;
            }
        }
        ptx::cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < DEPTH - 1; ++i) fetch(i);

    auto stage_columns = [&](int from) {
        const int units = min(plan.window, chunks - from) * (kQ4ChunkN / 8);
        const int n0 = (chunk0 + from) * kQ4ChunkN;
        for (int i = threadIdx.x; i < units * rows; i += THREADS) {
            const int row = i / units, u = i - row * units;
            const size_t at = (row0 + row) * args.lda;
            uint8_t* dst = xs + row * pieces * pitch + u * 16;
            if (args.dtype == SGEMM_BFLOAT16) {
                uint4 piece[1];
                load_split8<1>(static_cast<const __nv_bfloat16*>(args.A) + at, n0 + u * 8, geom.N,
                               args.vec, piece);
                *reinterpret_cast<uint4*>(dst) = piece[0];
            } else if (args.dtype == SGEMM_FLOAT16) {
                uint4 piece[2];
                load_split8<2>(static_cast<const __half*>(args.A) + at, n0 + u * 8, geom.N,
                               args.vec, piece);
                *reinterpret_cast<uint4*>(dst) = piece[0];
                *reinterpret_cast<uint4*>(dst + pitch) = piece[1];
            } else {
                uint4 piece[3];
                load_split8<3>(static_cast<const float*>(args.A) + at, n0 + u * 8, geom.N, args.vec,
                               piece);
#pragma unroll
                for (int p = 0; p < 3; ++p)
                    *reinterpret_cast<uint4*>(dst + p * pitch) = piece[p];
            }
        }
    };
    const bool whole = plan.window >= plan.chunks;
    if (whole) {
        stage_columns(0);
        __syncthreads();
    }

    // a lane's words of column 8 nt + r; columns that do not exist repeat the last one, and
    // their sums are not used
    const uint8_t* xcol[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) xcol[nt] = xs + min(nt * 8 + r, columns - 1) * pitch + c * 16;

    int stage = 0, buffer = 0;
    for (int group = first_group; group < plan.groups; group += plan.clusters) {
        float total[MT][NT][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) total[m][nt][i] = 0.0f;
        for (int from = 0; from < chunks; from += plan.window) {
            if (!whole) {
                __syncthreads();
                stage_columns(from);
                __syncthreads();
            }
            const int to = min(chunks, from + plan.window);
            for (int ch = from + wn; ch < to; ch += plan.wn) {
                ptx::cp_async_wait<DEPTH - 2>();
                __syncwarp();
                fetch(stage == 0 ? DEPTH - 1 : stage - 1);
                const uint8_t* codes = ring + stage * STAGE;
                const int x_at = (ch - from) * kQ4ChunkN * 2;
                q4_chunk<MT, NT, GROUP>(
                    [&](int m) { return codes + m * kQ4MaxChunk; }, geom.zeros, geom.fp16, lane,
                    [&](int b, int nt) {
                        return *reinterpret_cast<const uint4*>(xcol[nt] + x_at + b * 64);
                    },
                    total);
                stage = stage == DEPTH - 1 ? 0 : stage + 1;
            }
        }
        // sums over the warps that split n, in their order
        float* mine = red + buffer * red_floats(MT, NT) + (wn * strips_per_group + wm * MT) * NT * 8 * 17;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    mine[((m * NT + nt) * 8 + 2 * c + (i & 1)) * 17 + r + 8 * (i >> 1)] =
                        total[m][nt][i];
        __syncthreads();
        const float* sums = red + buffer * red_floats(MT, NT);
        const int width = strips_per_group * kQ4StripK, cells = width * rows;
        const int k0 = group * width;
        for (int i = threadIdx.x; i < cells; i += THREADS) {
            const int row = i / width, col = i - row * width;
            const float* at = sums + ((col / kQ4StripK) * NT * 8 + row * pieces) * 17 + col % kQ4StripK;
            float s = 0.0f;
            for (int w = 0; w < plan.wn; ++w) {
                for (int p = 0; p < pieces; ++p) s += at[p * 17];
                at += strips_per_group * NT * 8 * 17;
            }
            if (plan.cluster > 1)
                part[buffer * part_floats(MT, NT) + i] = s;
            else if (k0 + col < geom.K)
                store_from_float(args.C, args.dtype, (row0 + row) * args.ldc + k0 + col, s);
        }
        if (plan.cluster > 1) {
            ptx::cluster_sync();
            // each CTA adds the ranges' sums of its share of the cells, in rank order
            const int share = (cells + plan.cluster - 1) / plan.cluster;
            const uint32_t base =
                ptx::smem_u32(part + buffer * part_floats(MT, NT));
            for (int i = rank * share + threadIdx.x; i < min(cells, (rank + 1) * share);
                 i += THREADS) {
                float s = 0.0f;
                for (int q = 0; q < plan.cluster; ++q)
                    s += ptx::ld_shared_cluster_f32(ptx::mapa_shared(base + i * 4, q));
                const int row = i / width, col = i - row * width;
                if (k0 + col < geom.K) store_from_float(args.C, args.dtype, (row0 + row) * args.ldc + k0 + col, s);
            }
        }
        buffer ^= 1;
    }
    ptx::cp_async_wait<0>();
    // a CTA's shared memory is read by the others until here
    if (plan.cluster > 1) ptx::cluster_sync();
}

// The split of an N x K product with this many columns on sm_count SMs, for kernels with MT
// and NT: the cluster size and warp split whose slowest SM is done first. A chunk costs an
// SM about 45 cycles at the HBM rate; exchanging sums some hundreds a group.
Plan make_plan(const Q4Geom& g, int columns, int mt, int nt, int sm_count, double* cost_out) {
    Plan best{};
    double best_cost = 1e30;
    for (int cluster = 1; cluster <= 4; cluster *= 2) {
        if (cluster > 1 && g.chunks < 2 * cluster) break;
        for (int wn = WARPS; wn >= 1; wn /= 2) {
            Plan p;
            p.cluster = cluster;
            p.wn = wn;
            p.chunks = (g.chunks + cluster - 1) / cluster;
            if (wn > 1 && wn > p.chunks) continue;
            const int fixed = WARPS * DEPTH * mt * kQ4MaxChunk + 2 * red_floats(mt, nt) * 4 +
                              (cluster > 1 ? 2 * part_floats(mt, nt) * 4 : 0);
            p.staged = columns;
            p.window = p.chunks;
            int smem = fixed + columns * column_pitch(p.window);
            if (smem > SMEM_LIMIT) {
                p.window = ((SMEM_LIMIT - fixed) / columns - 64) / (kQ4ChunkN * 2) / wn * wn;
                if (p.window < wn) continue;
                smem = fixed + columns * column_pitch(p.window);
            }
            p.smem = smem;
            const int resident = smem <= SMEM_HALF ? 2 : 1;
            const int strips = WARPS / wn * mt;
            p.groups = (g.strips + strips - 1) / strips;
            const int slots = sm_count * resident / cluster;
            p.clusters = p.groups < slots ? p.groups : slots;
            const int rounds = (p.groups + p.clusters - 1) / p.clusters;
            const int units = (p.chunks + wn - 1) / wn * mt;  // of a warp and group
            const int busy = (p.clusters * cluster + sm_count - 1) / sm_count;
            const double windows = double((p.chunks + p.window - 1) / p.window);
            const double cost = rounds * (busy * WARPS * units * 45.0 + 300.0 +
                                          (cluster > 1 ? 400.0 : 0.0) +
                                          (windows > 1 ? windows * 1500.0 : 0.0));
            if (cost < best_cost) {
                best_cost = cost;
                best = p;
            }
        }
    }
    *cost_out = best_cost;
    return best;
}

template <int MT, int NT, int GROUP>
cudaError_t launch_kernel(const Args& args, int launch_rows, cudaStream_t stream) {
    const cudaError_t err = set_smem_limit_once<q4_matmul_kernel<MT, NT, GROUP>>(SMEM_LIMIT);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t config = {};
    config.gridDim = dim3(args.plan.clusters * args.plan.cluster, launch_rows);
    config.blockDim = dim3(THREADS);
    config.dynamicSmemBytes = args.plan.smem;
    config.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = args.plan.cluster;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    config.attrs = &attr;
    config.numAttrs = args.plan.cluster > 1 ? 1 : 0;
    count_launch();
    return cudaLaunchKernelEx(&config, q4_matmul_kernel<MT, NT, GROUP>, args);
}

template <int NT>
cudaError_t launch(Args args, int sm_count, cudaStream_t stream) {
    const int most_rows = NT * 8 / args.pieces;
    const int launch_rows = (args.M + most_rows - 1) / most_rows;
    const int columns = (args.M < most_rows ? args.M : most_rows) * args.pieces;
    double one, two;
    const Plan p1 = make_plan(args.geom, columns, 1, NT, sm_count, &one);
    const Plan p2 = make_plan(args.geom, columns, 2, NT, sm_count, &two);
    const bool pair = two <= one;
    args.plan = pair ? p2 : p1;
    switch (args.geom.group * 2 + (pair ? 1 : 0)) {
        case 64: return launch_kernel<1, NT, 32>(args, launch_rows, stream);
        case 65: return launch_kernel<2, NT, 32>(args, launch_rows, stream);
        case 128: return launch_kernel<1, NT, 64>(args, launch_rows, stream);
        case 129: return launch_kernel<2, NT, 64>(args, launch_rows, stream);
        case 256: return launch_kernel<1, NT, 128>(args, launch_rows, stream);
        default: return launch_kernel<2, NT, 128>(args, launch_rows, stream);
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
    const int columns = M * args.pieces;
    const cudaError_t err = columns <= 8    ? launch<1>(args, info->sm_count, s)
                            : columns <= 16 ? launch<2>(args, info->sm_count, s)
                                            : launch<4>(args, info->sm_count, s);
    return err == cudaSuccess ? SGEMM_OK : SGEMM_ERR_CUDA;
}
