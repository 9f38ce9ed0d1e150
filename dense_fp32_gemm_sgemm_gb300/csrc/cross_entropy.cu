// Softmax cross entropy of an output head, x W^T, over a large vocabulary, with its gradients.
//
//     s[t][v] = x[t] . w[v],  lse[t] = log sum_v exp s[t][v],  loss[t] = lse[t] - s[t][y[t]],
//     g[t][v] = c[t] (exp(s[t][v] - lse[t]) - [v = y[t]]),  dx = g . W,  dW = g^T . x
//
// over the tokens that count (0 <= y < V). Three products of T V D multiply-adds, the least that
// the gradients take; the logits exist in the tensor core's accumulators only.
//
//  1. ce_plan lists the counted tokens in order, ce_gather packs their rows of x (ce_select does
//     both for few). Uncounted rows
//     are never read again: whatever they hold stays out of dW, and costs no products.
//  2. The first product's epilogue has a row's 64 or 128 columns in a thread: the target's logit (FP32)
//     is picked out, the maximum m and the sum of exp(s - m) (FP32) of the other columns go to `stats`,
//     and, for gradients, exp(s - m) is stored in 16 bits. That rounding (2^-9 of each value, bfloat16;
//     2^-12, FP16, which holds them times 2^15 so that small ones keep their bits) and the one
//     of g average out in the sums over tokens and vocabulary; s itself in 16 bits would be off
//     by 2^-9 |s| in the exponent.
//  3. ce_finish joins the stats of a row to the others' sum, `rest`, and with the target's exponential e
//     to lse, and turns the exponentials into g in place: times exp(m - lse) c / max c. The target's
//     loss and element are log1p(rest / e) and -rest / (e + rest): a confident token's, whose rest may
//     be below 2^-24 of e, keep their bits, which a sum of all exponentials has dropped. c is divided
//     by the largest |c|, which the last epilogue multiplies back: where all c are equal, nothing is
//     rounded by them.
//  4. A second product computes dx (reduction over V, in parts where it is long and tiles are
//     few) and dW (reduction over the tokens) in one launch, long units first.
//
// Tokens are worked through in chunks, so that the exponentials take CE_CHUNK_BYTES at most.
// float32 operands are three bfloat16 planes (24 bits), of which six products are taken; the
// logits are then kept in FP32 and g in three planes.
//
// Measured (8192 x 4096 by 65536, bfloat16): 8.0 to 8.3 ms, 1.59 to 1.65 PFLOP/s, where the power cap holds
// cuBLAS at 1.71 to 1.77; 2.3 + 0.37 + 4.4 ms for the three passes with the clock at 1.9 GHz.
#include <algorithm>
#include <cstring>

#include "half_gemm.cuh"
#include "sgemm.h"

namespace sgemm {
namespace {

constexpr long long CE_CHUNK_BYTES = 1ll << 31;
constexpr int FINISH_THREADS = 256;
constexpr int PLAN_THREADS = 1024;
constexpr int PLAN_ITEMS = 4;
// Up to which ce_select does the work of both, in which every CTA goes through all targets. Loss of T x 512
// by 1000 on the device: T = 64 22.7 us against 24.7 with two launches, 512 24.7 and 26.7, 1024 28 and 27,
// 2048 49 and 38, 8192 289 and 68.
constexpr int SELECT_TOKENS = 1024;
constexpr long long MAX_TMA_PITCH = 1ll << 37;  // elements; a map's pitch ends at 2^40 bytes
constexpr float LOG2E = 1.4426950408889634f;

// What ce_plan leaves on the device.
struct CeInfo {
    int count;     // counted tokens
    int finished;  // CTAs of ce_finish that are done
    float c_max;   // largest finite |c| of them (1 where that is 0)
    float c_mean;  // 1 / count
};

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ bool finite(float x) { return fabsf(x) <= 3.402823466e38f; }

// x as three bfloat16 pieces whose sum it is, rounded to nearest each; an infinity or NaN is in
// the first.
__device__ __forceinline__ void split3(float x, __nv_bfloat16 (&p)[3]) {
    p[0] = __float2bfloat16_rn(x);
    if (!finite(__bfloat162float(p[0]))) {
        if (!finite(x)) {
            p[1] = p[2] = __float2bfloat16_rn(0.f);
            return;
        }
        p[0] = __float2bfloat16_rz(x);
    }
    const float r = x - __bfloat162float(p[0]);
    p[1] = __float2bfloat16_rn(r);
    p[2] = __float2bfloat16_rn(r - __bfloat162float(p[1]));
}

// ---- the tokens that count ------------------------------------------------------------------
template <class TARGET>
__global__ void __launch_bounds__(PLAN_THREADS)
    ce_plan(const TARGET* __restrict__ target, const float* __restrict__ c, int T, int V,
            int* __restrict__ rows, int* __restrict__ label, CeInfo* info, int* counters,
            int n_counters) {
    __shared__ int warp_sum[32];
    __shared__ float warp_max[32];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i < n_counters; i += PLAN_THREADS) counters[i] = 0;
    int base = 0;
    float top = 0.f;
    for (int t0 = 0; t0 < T; t0 += PLAN_THREADS * PLAN_ITEMS) {
        const int first = t0 + tid * PLAN_ITEMS;
        int y[PLAN_ITEMS];
        int mine = 0;
#pragma unroll
        for (int j = 0; j < PLAN_ITEMS; ++j) {
            const long long v = first + j < T ? (long long)target[first + j] : -1;
            y[j] = v >= 0 && v < V ? int(v) : -1;
            if (y[j] >= 0) {
                ++mine;
                if (c) {
                    const float a = fabsf(c[first + j]);
                    if (finite(a)) top = fmaxf(top, a);
                }
            }
        }
        int scan = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(~0u, scan, o);
            if (lane >= o) scan += up;
        }
        __syncthreads();
        if (lane == 31) warp_sum[warp] = scan;
        __syncthreads();
        int before = 0, all = 0;
        {
            const int s = warp_sum[lane];
            int w = s;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(~0u, w, o);
                if (lane >= o) w += up;
            }
            all = __shfl_sync(~0u, w, 31);
            before = __shfl_sync(~0u, w - s, warp);
        }
        int at = base + before + scan - mine;
#pragma unroll
        for (int j = 0; j < PLAN_ITEMS; ++j) {
            if (y[j] < 0) continue;
            rows[at] = first + j;
            label[at] = y[j];
            ++at;
        }
        base += all;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    if (lane == 0) warp_max[warp] = top;
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < 32; ++w) top = fmaxf(top, warp_max[w]);
        info->count = base;
        info->finished = 0;
        info->c_mean = base > 0 ? 1.f / float(base) : 0.f;
        info->c_max = c ? (top > 0.f ? top : 1.f) : (base > 0 ? info->c_mean : 1.f);
    }
}

// One row of D elements as Dp elements, zeros behind D (all zeros where `from` is null): 16 bits as
// they are, float32 as three planes. Eight elements a thread and turn; `wide`: 16-byte aligned rows
// of a multiple of 8 elements.
template <class T_IN>
__device__ __forceinline__ void pack_row(const T_IN* from, int D, int Dp, long long plane, bool wide,
                                         unsigned short* to) {
    for (int d = threadIdx.x * 8; d < Dp; d += blockDim.x * 8) {
        if constexpr (sizeof(T_IN) == 4) {
            float v[8];
            if (from && wide && d < D) {
                const float4 a = *reinterpret_cast<const float4*>(from + d);
                const float4 b = *reinterpret_cast<const float4*>(from + d + 4);
                v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
                v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = from && d + j < D ? from[d + j] : 0.f;
            }
            __align__(16) __nv_bfloat16 p[3][8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                __nv_bfloat16 q[3];
                split3(v[j], q);
#pragma unroll
                for (int i = 0; i < 3; ++i) p[i][j] = q[i];
            }
#pragma unroll
            for (int i = 0; i < 3; ++i)
                *reinterpret_cast<uint4*>(to + i * plane + d) = *reinterpret_cast<const uint4*>(p[i]);
        } else {
            const unsigned short* f = reinterpret_cast<const unsigned short*>(from);
            uint4 w = make_uint4(0, 0, 0, 0);
            if (f && wide && d < D) {
                w = *reinterpret_cast<const uint4*>(f + d);
            } else if (f) {
                uint32_t h[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) h[j] = d + j < D ? f[d + j] : 0u;
                w = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16,
                               h[6] | h[7] << 16);
            }
            *reinterpret_cast<uint4*>(to + d) = w;
        }
    }
}

// Packs row rows[r] of x as row r of xc, zeros up to the next multiple of 64 rows (the reduction over
// tokens reads them); gives token r, where it does not count, its zeros. A CTA a row.
template <class T_IN>
__global__ void __launch_bounds__(128)
    ce_gather(const T_IN* __restrict__ x, long long ldx, int T, int D, int Dp, long long plane,
              const int* __restrict__ rows, const CeInfo* __restrict__ info,
              unsigned short* __restrict__ xc, const void* __restrict__ target, int target64, int V,
              float* __restrict__ losses, float* __restrict__ lse, T_IN* __restrict__ dx,
              long long lddx, int wide) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int r = blockIdx.x;
    const int n = info->count;
    if (r < ((n + 63) & ~63))
        pack_row(r < n ? x + (long long)rows[r] * ldx : nullptr, D, Dp, plane, wide,
                 xc + (long long)r * Dp);
    if (r < T) {
        const long long y = target64 ? reinterpret_cast<const long long*>(target)[r]
                                     : (long long)reinterpret_cast<const int*>(target)[r];
        if (y < 0 || y >= V) {
            if (threadIdx.x == 0) {
                losses[r] = 0.f;
                lse[r] = 0.f;
            }
            if (dx)
                for (int d = threadIdx.x; d < D; d += blockDim.x)
                    dx[(long long)r * lddx + d] = T_IN(0.f);
        }
    }
}

// ce_plan and ce_gather in one launch, for few tokens: every CTA goes through all targets itself to
// find the one that its row is for (1 x 512 by 4096, loss alone: 16.2 us of device time a call with two
// launches, 14.3 with one).
template <class T_IN>
__global__ void __launch_bounds__(128)
    ce_select(const T_IN* __restrict__ x, long long ldx, int T, int D, int Dp, long long plane,
              const void* __restrict__ target, int target64, int V, const float* __restrict__ c,
              int* __restrict__ rows, int* __restrict__ label, CeInfo* info, int* counters,
              int n_counters, unsigned short* __restrict__ xc, float* __restrict__ losses,
              float* __restrict__ lse, T_IN* __restrict__ dx, long long lddx, int wide) {
    __shared__ int warp_sum[4];
    __shared__ float warp_max[4];
    __shared__ int my_token;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = blockIdx.x;
    auto target_of = [&](int t) {
        const long long y = target64 ? reinterpret_cast<const long long*>(target)[t]
                                     : (long long)reinterpret_cast<const int*>(target)[t];
        return y >= 0 && y < V ? int(y) : -1;
    };
    const int each = (T + 127) / 128, t0 = tid * each, t1 = min(t0 + each, T);
    int mine = 0;
    float top = 0.f;
    for (int t = t0; t < t1; ++t) {
        if (target_of(t) < 0) continue;
        ++mine;
        if (c && r == 0) {
            const float a = fabsf(c[t]);
            if (finite(a)) top = fmaxf(top, a);
        }
    }
    int scan = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(~0u, scan, o);
        if (lane >= o) scan += up;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    if (lane == 31) warp_sum[warp] = scan;
    if (lane == 0) warp_max[warp] = top;
    __syncthreads();
    int first = scan - mine, n = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        if (w < warp) first += warp_sum[w];
        n += warp_sum[w];
    }
    if (r >= first && r < first + mine) {
        int at = first, t = t0;
        while (true) {
            const int y = target_of(t);
            if (y >= 0 && at++ == r) {
                my_token = t;
                rows[r] = t;
                label[r] = y;
                break;
            }
            ++t;
        }
    }
    if (r == 0) {
        for (int i = tid; i < n_counters; i += 128) counters[i] = 0;
        if (tid == 0) {
#pragma unroll
            for (int w = 1; w < 4; ++w) top = fmaxf(top, warp_max[w]);
            info->count = n;
            info->finished = 0;
            info->c_mean = n > 0 ? 1.f / float(n) : 0.f;
            info->c_max = c ? (top > 0.f ? top : 1.f) : (n > 0 ? info->c_mean : 1.f);
        }
    }
    __syncthreads();
    if (r < ((n + 63) & ~63))
        pack_row(r < n ? x + (long long)my_token * ldx : nullptr, D, Dp, plane, wide,
                 xc + (long long)r * Dp);
    if (r < T && target_of(r) < 0) {
        if (tid == 0) {
            losses[r] = 0.f;
            lse[r] = 0.f;
        }
        if (dx)
            for (int d = tid; d < D; d += 128) dx[(long long)r * lddx + d] = T_IN(0.f);
    }
}

// Weights that TMA cannot read as they are. A CTA a row.
template <class T_IN>
__global__ void __launch_bounds__(128)
    ce_weights(const T_IN* __restrict__ w, long long ldw, int D, int Dp, long long plane, int wide,
               unsigned short* __restrict__ wc) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    pack_row(w + (long long)blockIdx.x * ldw, D, Dp, plane, wide, wc + (long long)blockIdx.x * Dp);
}

// ---- the first product's epilogue -------------------------------------------------------------
// What is kept of the logits: nothing, their exponentials (bfloat16, or FP16 times 2^15), or
// themselves.
enum class Keep { none, bf16, fp16, logits };
constexpr int FP16_EXP_BITS = 15;   // exponentials of up to 1 are held times 2^15
constexpr int FP16_GRAD_BITS = 14;  // and g, of up to 1 in size, times 2^14

template <int BN_, Keep KEEP>
struct CeForward {
    static constexpr int BN = BN_;
    static constexpr int COLS = BN / 2;
    static constexpr int PROBLEMS = 1, PLANES = 1;
    static constexpr bool CHAIN = false;
    struct Params {
        float2* stats;   // [block of COLS columns][row of the chunk]: maximum, sum without the target
        float* picked;   // [row of the chunk]
        const int* label;  // of the chunk's rows
        CUtensorMap kept;  // blocks of 64 columns (16 bits) or 32 (logits)
        int stats_pitch;
        int V;
    };
    using Io = hg::WarpIo<hg::Ring<CeForward>::BLOCKS>;
    const Params& p;
    Io& io;
    int live;
    __device__ CeForward(const Params& p_, int live_, Io& io_)
        : p(p_), io(io_), live(live_) {}

    // `words` words of every lane, 32 at a time, to columns `col` on of `kept`, which a word has
    // 32 / `each` of. (Loops, as the code is fetched anew in every launch: see hg::Rows.)
    __device__ __forceinline__ void keep(float (&s)[COLS], int words, int each, int row, int col) {
        int block = 0;
#pragma unroll 1
        for (int at = 0; at < words; at += 32) {
            io.acquire(block);
            hg::stage_words<0>(io.block(block), s);
            io.store(block, &p.kept, col, row, 0);
            col += each;
            block = Io::of(block + 1);
#pragma unroll
            for (int j = 0; j + 32 < COLS; ++j) s[j] = s[j + 32];
        }
    }
    __device__ __forceinline__ void start(const hg::Unit&, int, int) {}
    __device__ __forceinline__ void unit(const hg::Unit&, int row, int col, float (&s)[COLS]) {
        const int lane = threadIdx.x & 31;
        const int cols = min(COLS, p.V - col);
        if (cols <= 0 || row >= live) return;
        if (cols < COLS) {
#pragma unroll
            for (int j = 0; j < COLS; ++j)
                if (j >= cols) s[j] = -INFINITY;
        }
        const int r = row + lane;
        const int y = r < live ? p.label[r] - col : -1;
        if (__any_sync(~0u, y >= 0 && y < cols)) {
            float v = 0.f;
#pragma unroll
            for (int j = 0; j < COLS; ++j) {
                v = y == j ? s[j] : v;
                s[j] = y == j ? -INFINITY : s[j];  // the statistics are of the others
            }
            if (y >= 0 && y < cols) p.picked[r] = v;
        }
        float m = s[0];
#pragma unroll
        for (int j = 1; j < COLS; ++j) m = fmaxf(m, s[j]);
        const float from = m == -INFINITY ? 0.f : m;
        float sum = 0.f;
        constexpr bool HALF = KEEP == Keep::bf16 || KEEP == Keep::fp16;
        constexpr float BIAS = KEEP == Keep::fp16 ? float(FP16_EXP_BITS) : 0.f;
#pragma unroll
        for (int j = 0; j < COLS; j += 2) {
            const float a = exp2_fast((s[j] - from) * LOG2E + BIAS);
            const float b = exp2_fast((s[j + 1] - from) * LOG2E + BIAS);
            sum += a + b;
            if constexpr (HALF)
                s[j / 2] = __uint_as_float(hg::pack2<KEEP == Keep::bf16>(a, b));
        }
        if constexpr (HALF) keep(s, COLS / 2, 64, row, col);
        if constexpr (KEEP == Keep::logits) keep(s, COLS, 32, row, col);
        if constexpr (KEEP == Keep::fp16) sum *= 1.f / float(1 << FP16_EXP_BITS);
        p.stats[(long long)(col / COLS) * p.stats_pitch + r] = make_float2(m, sum);
    }
};

// ---- lse, losses and g ---------------------------------------------------------------------------
struct FinishArgs {
    const float2* stats;
    int stats_pitch, blocks, cols;  // blocks of `cols` columns
    const float* picked;
    const int* rows;   // of the chunk
    const int* label;
    CeInfo* info;
    int live0, live_max;
    const float* c;    // by token, or null
    float* loss;       // or null
    float* losses;
    float* lse;
    void* kept;        // exponentials (16 bits, in place) or logits; null without gradients
    unsigned short* planes;  // of g for float32
    long long pitch, plane;
    int V, last_finished;  // CTAs of this kernel in the whole call
};

// ROWS rows a CTA, with the same columns of all of them in flight together; 8 columns a thread and
// turn. Bound by the memory it reads and writes: 8192 x 65536 of 16 bits, 4 rows a CTA, take 370 us
// (5.8 TB/s; 399 with the rows one after the other). Where few rows would leave SMs without a CTA, one
// row each (256 x 8192: 11.7 us against 22).
template <Keep KEEP, int ROWS>
__global__ void __launch_bounds__(FINISH_THREADS) ce_finish(const FinishArgs a) {
    __shared__ float2 part[FINISH_THREADS / 32][ROWS];
    __shared__ float row_from[ROWS], row_log[ROWS], row_scale[ROWS], row_label[ROWS];
    __shared__ int row_y[ROWS];
    __shared__ double sums[FINISH_THREADS / 32];
    __shared__ int is_last;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int count = a.info->count;
    const int live = min(max(count - a.live0, 0), a.live_max);
    const int r0 = blockIdx.x * ROWS;
    if (r0 < live) {
        float m[ROWS], l[ROWS];
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
        }
        auto join = [](float& m0, float& l0, float m1, float l1) {
            // a block of -inf alone (or NaN) has no maximum; its sum, 0 or NaN, counts as it is
            const float top = fmaxf(m0, m1);
            l0 = (m0 == -INFINITY ? l0 : l0 * expf(m0 - top)) +
                 (m1 == -INFINITY ? l1 : l1 * expf(m1 - top));
            m0 = top;
        };
        for (int b = tid; b < a.blocks; b += FINISH_THREADS) {
            const float2* at = a.stats + (long long)b * a.stats_pitch + r0;
            float2 v[ROWS];
#pragma unroll
            for (int i = 0; i < ROWS; ++i) v[i] = at[i];
#pragma unroll
            for (int i = 0; i < ROWS; ++i) join(m[i], l[i], v[i].x, v[i].y);
        }
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                const float m1 = __shfl_xor_sync(~0u, m[i], o), l1 = __shfl_xor_sync(~0u, l[i], o);
                // in the order of the lanes, so that both partners get the same bits
                if (lane & o) {
                    float ma = m1, la = l1;
                    join(ma, la, m[i], l[i]);
                    m[i] = ma;
                    l[i] = la;
                } else {
                    join(m[i], l[i], m1, l1);
                }
            }
            if (lane == 0) part[warp][i] = make_float2(m[i], l[i]);
        }
        __syncthreads();
    }
    if (tid < ROWS) {
        const int r = r0 + tid;
        float from = 0.f, logl = 0.f, scale = 0.f, at_label = 0.f;
        int y = -1;
        if (r < live) {
            float2 t = part[0][tid];
            for (int w = 1; w < FINISH_THREADS / 32; ++w) {
                const float2 u = part[w][tid];
                const float top = fmaxf(t.x, u.x);
                t.y = (t.x == -INFINITY ? t.y : t.y * expf(t.x - top)) +
                      (u.x == -INFINITY ? u.y : u.y * expf(u.x - top));
                t.x = top;
            }
            const int token = a.rows[r];
            y = a.label[r];
            const float picked = a.picked[r];
            from = fmaxf(t.x, picked);  // t: of all but the target
            const float rest = t.x == -INFINITY ? t.y : t.y * expf(t.x - from);
            const float e = picked == -INFINITY ? 0.f : expf(picked - from);
            const float total = e + rest;
            logl = logf(total);
            a.lse[token] = from + logl;
            a.losses[token] = rest <= e ? log1pf(rest / e) : (from - picked) + logl;
            const float c = a.c ? a.c[token] : a.info->c_mean;
            scale = c / a.info->c_max;
            at_label = -(rest / total) * scale;
        }
        row_from[tid] = from;
        row_log[tid] = logl;
        row_scale[tid] = scale;
        row_label[tid] = at_label;
        row_y[tid] = y;
    }
    __syncthreads();
    if constexpr (KEEP != Keep::none) {
        const int padded = (live + 63) & ~63;  // zeros up to here: the reduction over tokens reads them
        const int n = min(ROWS, padded - r0);
        if (n > 0) {
            for (int v0 = tid * 8; v0 < a.V; v0 += FINISH_THREADS * 8) {
                if constexpr (KEEP == Keep::logits) {
#pragma unroll 1
                    for (int i = 0; i < n; ++i) {
                        const int r = r0 + i, y = row_y[i];
                        const float* at =
                            static_cast<const float*>(a.kept) + (long long)r * a.pitch + v0;
                        float g[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) g[j] = 0.f;
                        if (r < live) {
                            const float4 u = *reinterpret_cast<const float4*>(at);
                            const float4 w = *reinterpret_cast<const float4*>(at + 4);
                            const float s[8] = {u.x, u.y, u.z, u.w, w.x, w.y, w.z, w.w};
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                g[j] = expf((s[j] - row_from[i]) - row_log[i]) * row_scale[i];
                        }
                        if (y >= v0 && y < v0 + 8) {
#pragma unroll
                            for (int j = 0; j < 8; ++j) g[j] = y == v0 + j ? row_label[i] : g[j];
                        }
                        uint32_t w[3][4];
#pragma unroll
                        for (int j = 0; j < 8; j += 2) {
                            __nv_bfloat16 p[3], q[3];
                            split3(g[j], p);
                            split3(g[j + 1], q);
#pragma unroll
                            for (int k = 0; k < 3; ++k)
                                w[k][j / 2] =
                                    uint32_t(*reinterpret_cast<unsigned short*>(&p[k])) |
                                    uint32_t(*reinterpret_cast<unsigned short*>(&q[k])) << 16;
                        }
#pragma unroll
                        for (int k = 0; k < 3; ++k)
                            *reinterpret_cast<uint4*>(a.planes + k * a.plane +
                                                      (long long)r * a.pitch + v0) =
                                make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]);
                    }
                } else {
                    constexpr bool BF = KEEP == Keep::bf16;
                    constexpr float GRAD_UP = BF ? 1.f : float(1 << FP16_GRAD_BITS);
                    constexpr float UNIT = BF ? 1.f : GRAD_UP / float(1 << FP16_EXP_BITS);
                    unsigned short* at =
                        static_cast<unsigned short*>(a.kept) + (long long)r0 * a.pitch + v0;
                    const float2* stats = a.stats + (long long)(v0 / a.cols) * a.stats_pitch + r0;
                    uint4 e[ROWS];
                    float top[ROWS];
#pragma unroll
                    for (int i = 0; i < ROWS; ++i) {
                        e[i] = make_uint4(0, 0, 0, 0);
                        top[i] = 0.f;
                        if (r0 + i < live) {
                            e[i] = *reinterpret_cast<const uint4*>(at + i * a.pitch);
                            top[i] = stats[i].x;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < ROWS; ++i) {
                        const float f = expf((top[i] - row_from[i]) - row_log[i]) * row_scale[i] * UNIT;
                        const uint32_t in[4] = {e[i].x, e[i].y, e[i].z, e[i].w};
                        float g[8];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            float2 v;
                            if constexpr (BF) {
                                v.x = __uint_as_float(in[j] << 16);
                                v.y = __uint_as_float(in[j] & 0xffff0000u);
                            } else {
                                v = __half22float2(*reinterpret_cast<const __half2*>(&in[j]));
                            }
                            g[2 * j] = v.x * f;
                            g[2 * j + 1] = v.y * f;
                        }
                        const int y = row_y[i];
                        if (y >= v0 && y < v0 + 8) {
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                g[j] = y == v0 + j ? row_label[i] * GRAD_UP : g[j];
                        }
                        uint4 out = make_uint4(hg::pack2<BF>(g[0], g[1]), hg::pack2<BF>(g[2], g[3]),
                                               hg::pack2<BF>(g[4], g[5]), hg::pack2<BF>(g[6], g[7]));
                        if (r0 + i >= live) out = make_uint4(0, 0, 0, 0);
                        if (i < n) *reinterpret_cast<uint4*>(at + i * a.pitch) = out;
                    }
                }
            }
        }
    }
    // the last CTA of the call sums up the losses, in a fixed order
    if (a.loss == nullptr) return;
    __threadfence();
    __syncthreads();
    if (tid == 0) is_last = atomicAdd(&a.info->finished, 1) == a.last_finished - 1;
    __syncthreads();
    if (!is_last) return;
    __threadfence();
    const int* all = a.rows - a.live0;
    double sum = 0.0;
    for (int r = tid; r < count; r += FINISH_THREADS) {
        const int token = all[r];
        const float c = a.c ? a.c[token] : a.info->c_mean;
        sum += double(c) * double(__ldcg(a.losses + token));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    if (lane == 0) sums[warp] = sum;
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < FINISH_THREADS / 32; ++w) sum += sums[w];
        *a.loss = float(sum);
    }
}

// ---- the second launch's epilogue ------------------------------------------------------------------
struct GradOut {
    CUtensorMap map;  // of the output (blocks of 128 bytes a row) or, FP32, of the parts
    void* out;
    long long ld;
    int dtype;        // SGEMM_FLOAT32, SGEMM_BFLOAT16 or SGEMM_FLOAT16
    int tma;          // stored through the map; else row by row
    int wide;         // rows are 16-byte aligned
    int rows_n, cols_n;
    const int* rows;  // output row of each row, or null
    float* sums;      // FP32 sums over chunks (pitch cols_n rounded up to 4), or null
    int first, last;  // chunk of those
    int part_rows;    // rows of a part of a split reduction, or 0
};

template <bool SUMS>
struct CeGrad {
    static constexpr int BN = 256;
    static constexpr int COLS = BN / 2;
    static constexpr int PROBLEMS = 2, PLANES = 1;
    static constexpr bool CHAIN = false;
    struct Params {
        GradOut out[2];
        const CeInfo* info;
        float down;  // 2^-FP16_GRAD_BITS or 1
    };
    using Io = hg::WarpIo<hg::Ring<CeGrad>::BLOCKS>;
    const Params& p;
    Io& io;
    int live;
    float scale;
    __device__ CeGrad(const Params& p_, int live_, Io& io_)
        : p(p_), io(io_), live(live_) {
        scale = p.info->c_max * p.down;
    }

    // the staged FP32 block added to the sums; with the last chunk the result goes out
    __device__ __forceinline__ void add_block(uint8_t* block, const GradOut& o, int row, int col) {
        const int lane = threadIdx.x & 31;
        const long long pitch = (o.cols_n + 3) & ~3;
        __syncwarp();
#pragma unroll 1
        for (int i = 0; i < 32; ++i) {
            const int r = row + i, c = col + lane;
            if (r >= o.rows_n) break;
            if (c < o.cols_n) {
                const uint32_t* words = reinterpret_cast<const uint32_t*>(
                    hg::staged(block, i, lane >> 2));
                float v = __uint_as_float(words[lane & 3]);
                float* sum = o.sums + r * pitch + c;
                if (!o.first) v += *sum;
                if (!o.last) {
                    *sum = v;
                } else if (o.dtype == SGEMM_FLOAT32) {
                    static_cast<float*>(o.out)[r * o.ld + c] = v;
                } else if (o.dtype == SGEMM_BFLOAT16) {
                    static_cast<__nv_bfloat16*>(o.out)[r * o.ld + c] = __float2bfloat16_rn(v);
                } else {
                    static_cast<__half*>(o.out)[r * o.ld + c] = __float2half_rn(v);
                }
            }
        }
        __syncwarp();
    }

    // The first 32 words of every lane through a staging block to columns `col` on.
    template <int SIZE>
    __device__ __forceinline__ void part(const hg::Unit& t, const GradOut& o, int b, int row, int col,
                                         int index, const float (&s)[COLS]) {
        io.acquire(b);
        hg::stage_words<0>(io.block(b), s);
        if (o.tma) {
            io.store(b, &o.map, col, t.split * o.part_rows + row, 0);
        } else if (SUMS && SIZE == 4 && o.sums) {
            add_block(io.block(b), o, row, col);
        } else {
            const int bytes = min(128, (o.cols_n - col) * SIZE);
            char* base = static_cast<char*>(o.out) + (long long)col * SIZE;
            if (!o.rows) base += row * (o.ld * SIZE);
            const hg::Rows to = {base, o.ld * SIZE, (o.rows ? live : o.rows_n) - row, bytes,
                                 o.wide && bytes % 16 == 0};
            if (o.rows)
                hg::store_block<SIZE, true>(io.block(b), to, index);
            else
                hg::store_block<SIZE>(io.block(b), to);
        }
    }

    __device__ __forceinline__ void start(const hg::Unit&, int, int) {}
    __device__ __forceinline__ void unit(const hg::Unit& t, int row, int col, float (&s)[COLS]) {
        const GradOut& o = p.out[t.problem];
        const int lane = threadIdx.x & 31;
        const int index = o.rows && row + lane < live ? o.rows[row + lane] : 0;
        if (!o.part_rows) {
#pragma unroll
            for (int j = 0; j < COLS; ++j) s[j] *= scale;
        }
        const bool wide = o.part_rows || (SUMS && o.sums) || o.dtype == SGEMM_FLOAT32;
        if (!wide) {
            const bool bf16 = o.dtype == SGEMM_BFLOAT16;
#pragma unroll
            for (int j = 0; j < COLS; j += 2)
                s[j / 2] = __uint_as_float(bf16 ? hg::pack2<true>(s[j], s[j + 1])
                                                : hg::pack2<false>(s[j], s[j + 1]));
        }
        const int each = wide ? 32 : 64, end = min(col + COLS, o.cols_n);
        int b = 0;
#pragma unroll 1
        for (int at = col; at < end; at += each) {
            if (wide)
                part<4>(t, o, b, row, at, index, s);
            else
                part<2>(t, o, b, row, at, index, s);
            b = Io::of(b + 1);
#pragma unroll
            for (int j = 0; j + 32 < COLS; ++j) s[j] = s[j + 32];
        }
    }
};

// dx from the parts of its reduction, added in order. A CTA a row.
template <class T_OUT>
__global__ void __launch_bounds__(256)
    ce_join(const float* __restrict__ parts, long long part, int splits, int D, int live0,
            int live_max, const int* __restrict__ rows, const CeInfo* __restrict__ info, float down,
            T_OUT* __restrict__ dx, long long lddx) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int r = blockIdx.x;
    if (r >= min(max(info->count - live0, 0), live_max)) return;
    const float scale = info->c_max * down;
    const float* from = parts + (long long)r * ((D + 3) & ~3);
    T_OUT* to = dx + rows[r] * lddx;
    for (int d = threadIdx.x; d < D; d += blockDim.x) {
        float v = from[d];
        for (int s = 1; s < splits; ++s) v += from[s * part + d];
        v *= scale;
        if constexpr (sizeof(T_OUT) == 4)
            to[d] = v;
        else
            to[d] = T_OUT(v);
    }
}

// ---- host ---------------------------------------------------------------------------------------------
int round_up(int n, int to) { return (n + to - 1) / to * to; }

struct Planes {
    int count;     // planes of an operand
    int products;
    unsigned char pa[hg::MAX_PRODUCTS], pb[hg::MAX_PRODUCTS];
};
constexpr Planes ONE = {1, 1, {0}, {0}};
constexpr Planes THREE = {3, 6, {1, 0, 2, 0, 1, 0}, {1, 2, 0, 1, 0, 0}};

void set_planes(hg::Problem& p, const Planes& k) {
    p.planes_a = p.planes_b = k.count;
    p.products = k.products;
    std::memcpy(p.pa, k.pa, sizeof p.pa);
    std::memcpy(p.pb, k.pb, sizeof p.pb);
}

int element_size(int dtype) { return dtype == SGEMM_FLOAT32 ? 4 : 2; }

// Bytes from the first to behind the last element of `rows` rows.
size_t extent(int rows, int cols, long long ld, int size) {
    return rows < 1 ? 0 : (size_t(rows - 1) * size_t(ld) + size_t(cols)) * size_t(size);
}

int check(const sgemm_ce& a) {
    if (a.dtype < SGEMM_FLOAT32 || a.dtype > SGEMM_FLOAT16) return SGEMM_ERR_ARG;
    if (a.T < 0 || a.T > (1 << 20) || a.D < 1 || a.D > 65536 || a.V < 1 || a.V > (1 << 20))
        return SGEMM_ERR_ARG;
    if (a.target_bits != 32 && a.target_bits != 64) return SGEMM_ERR_ARG;
    const int size = element_size(a.dtype);
    if (!a.weight || a.ldw < a.D || !aligned_to(a.weight, size)) return SGEMM_ERR_ARG;
    if (a.dweight && (a.lddw < a.D || !aligned_to(a.dweight, size))) return SGEMM_ERR_ARG;
    if (a.loss && !aligned_to(a.loss, 4)) return SGEMM_ERR_ARG;
    if (a.T > 0) {
        if (!a.x || a.ldx < a.D || !aligned_to(a.x, size)) return SGEMM_ERR_ARG;
        if (!a.target || !aligned_to(a.target, a.target_bits / 8)) return SGEMM_ERR_ARG;
        if (!a.losses || !a.lse || !aligned_to(a.losses, 4) || !aligned_to(a.lse, 4))
            return SGEMM_ERR_ARG;
        if (a.token_weights && !aligned_to(a.token_weights, 4)) return SGEMM_ERR_ARG;
        if (a.dx && (a.lddx < a.D || !aligned_to(a.dx, size))) return SGEMM_ERR_ARG;
    }
    struct Range {
        const void* p;
        size_t bytes;
    };
    const size_t t4 = size_t(a.T) * 4;
    const Range in[] = {{a.x, extent(a.T, a.D, a.ldx, size)},
                        {a.weight, extent(a.V, a.D, a.ldw, size)},
                        {a.target, size_t(a.T) * size_t(a.target_bits / 8)},
                        {a.token_weights, t4}};
    const Range out[] = {{a.loss, 4},
                         {a.losses, t4},
                         {a.lse, t4},
                         {a.dx, extent(a.T, a.D, a.lddx, size)},
                         {a.dweight, extent(a.V, a.D, a.lddw, size)}};
    for (size_t i = 0; i < 5; ++i) {
        if (!out[i].p || !out[i].bytes) continue;
        for (const Range& r : in)
            if (r.p && r.bytes && ranges_overlap(out[i].p, out[i].bytes, r.p, r.bytes))
                return SGEMM_ERR_OVERLAP;
        for (size_t j = 0; j < i; ++j)
            if (out[j].p && out[j].bytes &&
                ranges_overlap(out[i].p, out[i].bytes, out[j].p, out[j].bytes))
                return SGEMM_ERR_OVERLAP;
    }
    return SGEMM_OK;
}

template <int BN>
cudaError_t forward(Keep keep, const hg::Args<1>& g, float2* stats, float* picked, const int* label,
                    const CUtensorMap& kept, int stats_pitch, int V, int sm_count, cudaStream_t s) {
    switch (keep) {
        case Keep::none:
            return hg::launch_gemm<CeForward<BN, Keep::none>>(
                g, {stats, picked, label, kept, stats_pitch, V}, sm_count, s);
        case Keep::bf16:
            return hg::launch_gemm<CeForward<BN, Keep::bf16>>(
                g, {stats, picked, label, kept, stats_pitch, V}, sm_count, s);
        case Keep::fp16:
            return hg::launch_gemm<CeForward<BN, Keep::fp16>>(
                g, {stats, picked, label, kept, stats_pitch, V}, sm_count, s);
        default:
            return hg::launch_gemm<CeForward<BN, Keep::logits>>(
                g, {stats, picked, label, kept, stats_pitch, V}, sm_count, s);
    }
}

template <Keep KEEP>
cudaError_t finish(const FinishArgs& a, int rows, int ctas, cudaStream_t s) {
    return rows == 4 ? hg::launch(ce_finish<KEEP, 4>, ctas, FINISH_THREADS, 0, s, a)
                     : hg::launch(ce_finish<KEEP, 1>, ctas, FINISH_THREADS, 0, s, a);
}

// Parts of dx's reduction: a unit should take no more than half of a pair's share of the launch,
// so that the shares come out even.
int dx_splits(int tiles_dx, int kblocks_dx, int tiles_dw, int kblocks_dw, int pairs) {
    const long long all = (long long)tiles_dx * kblocks_dx + (long long)tiles_dw * kblocks_dw;
    const long long most = std::max(all / pairs / 2, 16ll);
    return int((kblocks_dx + most - 1) / most);
}

template <class T_IN>
cudaError_t run(const sgemm_ce& a, const DeviceInfo& info, int dev, cudaStream_t s) {
    const bool f32 = a.dtype == SGEMM_FLOAT32;
    const bool bf16 = a.dtype != SGEMM_FLOAT16;  // type of the operands
    const int size = element_size(a.dtype);
    const Planes& planes = f32 ? THREE : ONE;
    const bool grad = a.dx || a.dweight;
    const int Dp = round_up(a.D, 64);  // rows of whole 128-byte lines
    const long long pitch = round_up(a.V, 128);
    const int Tp = round_up(a.T, 256);
    // rows of a chunk: what is kept of their logits, and statistics of 64 columns at least
    const long long row_bytes = (grad ? pitch * (f32 ? 4 + 6 : 2) : 0) + pitch / 64 * 8;
    int chunk = Tp;
    if (Tp * row_bytes > CE_CHUNK_BYTES)
        chunk = int(std::max(CE_CHUNK_BYTES / row_bytes / 256 * 256, 256ll));
    const int chunks = (Tp + chunk - 1) / chunk;
    const int pairs = std::max(info.sm_count / 2, 1);
    // 128 columns a tile where 256 would leave pairs without one
    const bool narrow = chunk / 256 * ((a.V + 255) / 256) < pairs;
    const int cols = narrow ? 64 : 128;
    const int blocks = (a.V + cols - 1) / cols;
    const bool direct =
        !f32 && aligned16(a.weight) && a.ldw % 8 == 0 && a.ldw < MAX_TMA_PITCH;
    const int tiles_d = (a.D + 255) / 256;
    const int splits =
        a.dx ? dx_splits(chunk / 256 * tiles_d, (a.V + 63) / 64,
                         a.dweight ? (a.V + 255) / 256 * tiles_d : 0, chunk / 64, pairs)
             : 1;
    const bool sums = a.dweight && chunks > 1;

    hg::Layout lay;
    const size_t at_info = lay.add(sizeof(CeInfo));
    const size_t at_counters = lay.add(size_t(chunks) * 2 * sizeof(int));
    const size_t at_rows = lay.add(size_t(Tp) * 4);
    const size_t at_label = lay.add(size_t(Tp) * 4);
    const size_t x_plane = size_t(Tp) * Dp, w_plane = size_t(a.V) * Dp;
    const size_t at_x = lay.add(x_plane * 2 * planes.count);
    const size_t at_w = direct ? 0 : lay.add(w_plane * 2 * planes.count);
    const size_t at_stats = lay.add(size_t(blocks) * chunk * sizeof(float2));
    const size_t at_picked = lay.add(size_t(chunk) * 4);
    const size_t g_plane = size_t(chunk) * size_t(pitch);
    const size_t at_kept = grad ? lay.add(g_plane * (f32 ? 4 : 2)) : 0;
    const size_t at_planes = grad && f32 ? lay.add(g_plane * 6) : 0;
    const long long d4 = round_up(a.D, 4);
    const size_t part = size_t(chunk) * size_t(d4);
    const size_t at_parts = splits > 1 ? lay.add(part * 4 * size_t(splits)) : 0;
    const size_t at_sums = sums ? lay.add(size_t(a.V) * size_t(d4) * 4) : 0;
    Scratch scratch;
    cudaError_t e = scratch.alloc(dev, lay.total, s);
    if (e != cudaSuccess) return e;
    uint8_t* base = static_cast<uint8_t*>(scratch.ptr);
    CeInfo* ci = reinterpret_cast<CeInfo*>(base + at_info);
    int* counters = reinterpret_cast<int*>(base + at_counters);
    int* rows = reinterpret_cast<int*>(base + at_rows);
    int* label = reinterpret_cast<int*>(base + at_label);
    unsigned short* xc = reinterpret_cast<unsigned short*>(base + at_x);
    unsigned short* wc = reinterpret_cast<unsigned short*>(base + at_w);
    float2* stats = reinterpret_cast<float2*>(base + at_stats);
    float* picked = reinterpret_cast<float*>(base + at_picked);
    void* kept = grad ? base + at_kept : nullptr;
    unsigned short* g_planes = reinterpret_cast<unsigned short*>(base + at_planes);
    float* parts = reinterpret_cast<float*>(base + at_parts);
    float* sum = reinterpret_cast<float*>(base + at_sums);
    const void* w = direct ? a.weight : wc;
    const long long ldw = direct ? a.ldw : Dp;

    // operands as tensors
    const void* g_of = f32 ? static_cast<const void*>(g_planes) : kept;
    hg::Args<1> fwd;
    hg::Args<2> bwd;
    std::memset(&fwd, 0, sizeof fwd);
    std::memset(&bwd, 0, sizeof bwd);
    const int half = narrow ? 64 : 128;
    if (!hg::encode_operand(&fwd.a[0], xc, bf16, a.D, Tp, Dp, planes.count, x_plane, 128) ||
        !hg::encode_operand(&fwd.b[0], w, bf16, a.D, a.V, ldw, planes.count,
                            direct ? ldw : (long long)w_plane, half))
        return cudaErrorInvalidValue;
    fwd.problems = 1;
    hg::Problem& f = fwd.p[0];
    f.M = chunk;
    f.N = a.V;
    f.K = a.D;
    f.batch = f.splits = 1;
    f.dyn = 1;
    // tile rows worked through together: their rows of x, some 32 MB, stay in L2 while the
    // weights pass by once for each group
    f.group = std::max(1, int((32ll << 20) / ((long long)a.D * 512 * planes.count)));
    set_planes(f, planes);
    f.idesc = hg::instruction(bf16, false, false);
    fwd.live = bwd.live = &ci->count;
    fwd.live_max = bwd.live_max = chunk;
    fwd.err = bwd.err = info.error_word;
    // Losses are FP32 whatever the inputs, so segments are short (relative error of the losses, against
    // 64 bits): 16 stages 7 to 9e-7, 8 stages 3 to 5e-7, 4 stages 2 to 3e-7, 2 stages 1e-7. With several
    // rows of tiles the epilogue has only two segments' time: 8 stages take as long as 16 (2048 x 4096 by
    // 65536, bfloat16: 652 and 655 us; 4 stages 685, 2 stages 740). A single row of tiles waits for its
    // weights, and 4 stages cost nothing (256 x 4096 by 65536: 133.3 and 133.2 us with 16, float32 901 and
    // 897 with 8; 2 stages 139 and 961). Tiles of 128 columns, of which a pair has two at most: 2 stages.
    fwd.seg_steps = narrow ? 2 : chunk == 256 ? 4 : 8;
    // 128 MMAs cut off 2^-16 of a sum of one sign, which is far below a 16-bit gradient's rounding
    bwd.seg_steps = f32 ? 8 : 32;

    CUtensorMap kept_map;
    std::memset(&kept_map, 0, sizeof kept_map);
    if (grad && !hg::encode_block(&kept_map, kept, f32 ? 4 : 2, pitch, chunk, pitch, 1, pitch,
                                  f32 ? 32 : 64, 32))
        return cudaErrorInvalidValue;
    GradOut outs[2];
    std::memset(outs, 0, sizeof outs);
    int n = 0, dx_at = -1;
    if (a.dx) {
        hg::Problem& p = bwd.p[n];
        if (!hg::encode_operand(&bwd.a[n], g_of, bf16, a.V, chunk, pitch, planes.count, g_plane,
                                128) ||
            !hg::encode_operand(&bwd.b[n], w, bf16, a.D, a.V, ldw, planes.count,
                                direct ? ldw : (long long)w_plane, hg::BK))
            return cudaErrorInvalidValue;
        p.M = chunk;
        p.N = a.D;
        p.K = a.V;
        p.batch = 1;
        p.splits = splits;
        p.dyn = 1;
        // 8192 x 4096 by 65536 takes 7.0 ms with 8 tile rows together, 7.2 with 2, 7.7 with 32
        p.group = 8;
        p.b_mn = 1;
        set_planes(p, planes);
        p.idesc = hg::instruction(bf16, false, true);
        outs[n].out = a.dx;
        outs[n].ld = a.lddx;
        outs[n].dtype = a.dtype;
        outs[n].wide = aligned16(a.dx) && a.lddx * size % 16 == 0;
        outs[n].rows_n = chunk;
        outs[n].cols_n = a.D;
        if (splits > 1) {
            outs[n].tma = 1;
            outs[n].part_rows = chunk;
            if (!hg::encode_block(&outs[n].map, parts, 4, d4, (long long)splits * chunk, d4, 1, d4,
                                  32, 32))
                return cudaErrorInvalidValue;
        }
        dx_at = n++;
    }
    int dw_at = -1;
    if (a.dweight) {
        hg::Problem& p = bwd.p[n];
        if (!hg::encode_operand(&bwd.a[n], g_of, bf16, a.V, chunk, pitch, planes.count, g_plane,
                                hg::BK) ||
            !hg::encode_operand(&bwd.b[n], xc, bf16, a.D, Tp, Dp, planes.count, x_plane, hg::BK))
            return cudaErrorInvalidValue;
        p.M = a.V;
        p.N = a.D;
        p.K = chunk;
        p.batch = p.splits = 1;
        p.dyn = 2;
        // the same call takes 7.0 ms with 4, 7.3 with 1, 7.1 with 16
        p.group = 4;
        p.a_mn = p.b_mn = 1;
        set_planes(p, planes);
        p.idesc = hg::instruction(bf16, true, true);
        outs[n].out = a.dweight;
        outs[n].ld = a.lddw;
        outs[n].dtype = a.dtype;
        outs[n].wide = aligned16(a.dweight) && a.lddw * size % 16 == 0;
        outs[n].rows_n = a.V;
        outs[n].cols_n = a.D;
        outs[n].sums = sums ? sum : nullptr;
        outs[n].tma = !sums && outs[n].wide && a.lddw < MAX_TMA_PITCH;
        if (outs[n].tma && !hg::encode_block(&outs[n].map, a.dweight, size, a.D, a.V, a.lddw, 1,
                                             a.lddw, 128 / size, 32))
            return cudaErrorInvalidValue;
        dw_at = n++;
    }
    bwd.problems = n;
    const float down = a.dtype == SGEMM_FLOAT16 ? 1.f / float(1 << FP16_GRAD_BITS) : 1.f;

    // launches
    const int wide_x = aligned16(a.x) && a.ldx * size % 16 == 0 && a.D % 8 == 0;
    const int wide_w = aligned16(a.weight) && a.ldw * size % 16 == 0 && a.D % 8 == 0;
    const T_IN* x = static_cast<const T_IN*>(a.x);
    T_IN* dx = static_cast<T_IN*>(a.dx);
    const int packed_rows = round_up(a.T, 64), target64 = a.target_bits == 64;
    if (a.T <= SELECT_TOKENS) {
        e = hg::launch(ce_select<T_IN>, packed_rows, 128, 0, s, x, a.ldx, a.T, a.D, Dp,
                       (long long)x_plane, a.target, target64, a.V, a.token_weights, rows, label, ci,
                       counters, 2 * chunks, xc, a.losses, a.lse, dx, a.lddx, wide_x);
    } else {
        if (target64)
            e = hg::launch(ce_plan<long long>, 1, PLAN_THREADS, 0, s,
                           static_cast<const long long*>(a.target), a.token_weights, a.T, a.V, rows,
                           label, ci, counters, 2 * chunks);
        else
            e = hg::launch(ce_plan<int>, 1, PLAN_THREADS, 0, s, static_cast<const int*>(a.target),
                           a.token_weights, a.T, a.V, rows, label, ci, counters, 2 * chunks);
        if (e != cudaSuccess) return e;
        e = hg::launch(ce_gather<T_IN>, packed_rows, 128, 0, s, x, a.ldx, a.T, a.D, Dp,
                       (long long)x_plane, static_cast<const int*>(rows),
                       static_cast<const CeInfo*>(ci), xc, a.target, target64, a.V, a.losses, a.lse,
                       dx, a.lddx, wide_x);
    }
    if (e != cudaSuccess) return e;
    if (!direct) {
        e = hg::launch(ce_weights<T_IN>, a.V, 128, 0, s, static_cast<const T_IN*>(a.weight), a.ldw,
                       a.D, Dp, (long long)w_plane, wide_w, wc);
        if (e != cudaSuccess) return e;
    }
    // rows that ce_finish has something to do for: those of tokens, for gradients 64 at a time
    const int finish_n = std::min(chunk, grad ? round_up(a.T, 64) : a.T);
    const int finish_rows = finish_n >= 8 * info.sm_count ? 4 : 1;
    const int finish_ctas = (finish_n + finish_rows - 1) / finish_rows;
    for (int c = 0; c < chunks; ++c) {
        const int live0 = c * chunk;
        const Keep keep = !grad ? Keep::none : f32 ? Keep::logits : bf16 ? Keep::bf16 : Keep::fp16;
        fwd.live0 = bwd.live0 = live0;
        fwd.p[0].a_row = live0;
        fwd.counter = counters + 2 * c;
        const int stats_pitch = chunk;
        e = narrow ? forward<128>(keep, fwd, stats, picked, label + live0, kept_map, stats_pitch, a.V,
                                  info.sm_count, s)
                   : forward<256>(keep, fwd, stats, picked, label + live0, kept_map, stats_pitch, a.V,
                                  info.sm_count, s);
        if (e != cudaSuccess) return e;
        FinishArgs fa = {stats, stats_pitch, blocks, cols, picked, rows + live0, label + live0, ci,
                         live0, chunk, a.token_weights, a.loss, a.losses, a.lse, kept, g_planes,
                         pitch, (long long)g_plane, a.V, finish_ctas * chunks};
        e = keep == Keep::none   ? finish<Keep::none>(fa, finish_rows, finish_ctas, s)
            : keep == Keep::bf16 ? finish<Keep::bf16>(fa, finish_rows, finish_ctas, s)
            : keep == Keep::fp16 ? finish<Keep::fp16>(fa, finish_rows, finish_ctas, s)
                                 : finish<Keep::logits>(fa, finish_rows, finish_ctas, s);
        if (e != cudaSuccess) return e;
        if (!grad) continue;
        bwd.counter = counters + 2 * c + 1;
        if (dx_at >= 0) outs[dx_at].rows = rows + live0;
        if (dw_at >= 0) {
            bwd.p[dw_at].b_row = live0;
            outs[dw_at].first = c == 0;
            outs[dw_at].last = c == chunks - 1;
        }
        if (sums)
            e = hg::launch_gemm<CeGrad<true>>(bwd, {{outs[0], outs[1]}, ci, down}, info.sm_count, s);
        else
            e = hg::launch_gemm<CeGrad<false>>(bwd, {{outs[0], outs[1]}, ci, down}, info.sm_count,
                                               s);
        if (e != cudaSuccess) return e;
        if (splits > 1) {
            e = hg::launch(ce_join<T_IN>, chunk, 256, 0, s, static_cast<const float*>(parts),
                           (long long)part, splits, a.D, live0, chunk,
                           static_cast<const int*>(rows + live0), static_cast<const CeInfo*>(ci),
                           down, static_cast<T_IN*>(a.dx), a.lddx);
            if (e != cudaSuccess) return e;
        }
    }
    return cudaGetLastError();
}

}  // namespace
}  // namespace sgemm

using namespace sgemm;

extern "C" int sgemm_cross_entropy(const sgemm_ce* args, void* stream) {
    if (!args) return SGEMM_ERR_ARG;
    const sgemm_ce a = *args;
    const int rc = check(a);
    if (rc != SGEMM_OK) return rc;
    int dev = -1;
    const DeviceInfo* info = current_device(&dev);
    if (!info) return SGEMM_ERR_NO_DEVICE;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (a.T == 0) {  // nothing but zeros
        e = cudaSuccess;
        if (a.loss) e = cudaMemsetAsync(a.loss, 0, 4, s);
        if (e == cudaSuccess && a.dweight) {
            const size_t size = element_size(a.dtype);
            e = cudaMemset2DAsync(a.dweight, size_t(a.lddw) * size, 0, size_t(a.D) * size,
                                  size_t(a.V), s);
        }
    } else if (a.dtype == SGEMM_FLOAT32) {
        e = run<float>(a, *info, dev, s);
    } else if (a.dtype == SGEMM_BFLOAT16) {
        e = run<__nv_bfloat16>(a, *info, dev, s);
    } else {
        e = run<__half>(a, *info, dev, s);
    }
    if (e != cudaSuccess) {
        cudaGetLastError();
        return SGEMM_ERR_CUDA;
    }
    return SGEMM_OK;
}
