// Newton-Schulz products: X = a X + (b A + c A A) X with A = X X^T (or the same from the right
// for a tall X), some five times over, which drive the singular values of a normalised matrix
// towards one.
//
// Three products a step. A and A A are symmetric: only tiles that reach the diagonal or lie below
// it are computed and the others written from them, so that a step of r x q (r <= q) costs
// r r q + r r r + 2 r r q operations.
//
// Precision. The iteration multiplies small singular values by a (3.4) each step, and with them
// whatever rounding put there. So X itself is kept in two FP16 pieces, 22 bits, and only the factors
// of the products are rounded further: the term a X, which carries the small values, keeps its
// bits, and (b A + c A A) X adds little to them. With factors of one FP16 piece (11 bits) the
// result is off by 0.5 to 1.7e-3 of its RMS for normal, low-rank and graded matrices, about as much
// as by the rounding of a bfloat16 result (1.7e-3); bfloat16 factors give 0.5 to 1.3e-2, and 1 to
// 20e-2 where X is rounded to them too. float16 and float32 results take both pieces of each factor
// and three products: 0.3 to 6e-6, where FP32 arithmetic throughout gives 0.2 to 3e-6. (CPU
// simulations of 256 x 256 to 512 x 1024.) The pieces are of values times a power of two, so that
// small entries stay in FP16's normal range: 2^13 for X, 2^12 for A, 2^10 for the polynomial.
#include <algorithm>
#include <cstring>

#include "half_gemm.cuh"
#include "sgemm.h"

namespace sgemm {
namespace {

constexpr float UP_X = 0x1p13f, UP_A = 0x1p12f, UP_P = 0x1p10f;  // scales of the pieces
constexpr int NORM_THREADS = 256;
constexpr int MAX_NORM_CTAS = 304;      // for one matrix
constexpr int CONVERT_THREADS = 256;
constexpr int MAX_STEPS = 64;

__device__ __forceinline__ float load(const float* p) { return *p; }
__device__ __forceinline__ float load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float load(const __half* p) { return __half2float(*p); }

// ---- the norm ------------------------------------------------------------------------------
// Sums of squares of the rows that a CTA takes, one partial sum for each CTA. Eight elements are
// squared and added in FP32 where that neither overflows nor loses them (their largest between
// 2^-50 and 2^50, or all zero), else in FP64; a thread's sums are FP64.
template <class T_IN>
__global__ void __launch_bounds__(NORM_THREADS)
    ns_norm(const T_IN* __restrict__ g, long long ld, long long stride, int M, int N,
            double* __restrict__ partial, int* counters, int n_counters) {
    __shared__ double sums[NORM_THREADS / 32];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    if (blockIdx.x == 0 && blockIdx.y == 0)
        for (int i = threadIdx.x; i < n_counters; i += NORM_THREADS) counters[i] = 0;
    const T_IN* from = g + blockIdx.y * stride;
    const int groups = (N + 7) / 8;
    const long long all = (long long)M * groups;
    double sum = 0.0;
    for (long long i = (long long)blockIdx.x * NORM_THREADS + threadIdx.x; i < all;
         i += (long long)gridDim.x * NORM_THREADS) {
        const int row = int(i / groups), c0 = int(i - (long long)row * groups) * 8;
        const T_IN* p = from + row * ld + c0;
        float v[8], top = 0.f, s = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[j] = c0 + j < N ? load(p + j) : 0.f;
            top = fmaxf(top, fabsf(v[j]));
            s = fmaf(v[j], v[j], s);
        }
        if (top == 0.f || (top > 0x1p-50f && top < 0x1p50f)) {
            sum += double(s);  // NaN where one of them is
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) sum += double(v[j]) * double(v[j]);
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < NORM_THREADS / 32; ++w) sum += sums[w];
        partial[(long long)blockIdx.y * gridDim.x + blockIdx.x] = sum;
    }
}

// X = G / (norm + eps) in two pieces. Rows of Np elements, zeros behind N.
template <class T_IN>
__global__ void __launch_bounds__(CONVERT_THREADS)
    ns_convert(const T_IN* __restrict__ g, long long ld, long long stride, int M, int N, int Np,
               const double* __restrict__ partial, int partials, float eps,
               __half* __restrict__ x) {
    __shared__ double sums[CONVERT_THREADS / 32];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    double sum = 0.0;
    const double* mine = partial + (long long)blockIdx.y * partials;
    for (int i = threadIdx.x; i < partials; i += CONVERT_THREADS) sum += mine[i];
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = sum;
    __syncthreads();
    sum = 0.0;
    for (int w = 0; w < CONVERT_THREADS / 32; ++w) sum += sums[w];
    const double norm = sqrt(sum) + double(eps);
    const float by = float(norm);
    // a norm outside FP32's range is divided by in FP64
    const bool plain = by > 0x1p-100f && by < 0x1p100f;
    const T_IN* from = g + blockIdx.y * stride;
    const long long plane = (long long)M * Np;
    __half* to = x + blockIdx.y * 2 * plane;
    const int groups = Np / 8;
    const long long all = (long long)M * groups;
    for (long long i = (long long)blockIdx.x * CONVERT_THREADS + threadIdx.x; i < all;
         i += (long long)gridDim.x * CONVERT_THREADS) {
        const int row = int(i / groups), c0 = int(i - (long long)row * groups) * 8;
        const T_IN* p = from + row * ld + c0;
        __half2 high[4], low[4];
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            float v[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int c = c0 + j + k;
                v[k] = c < N ? load(p + j + k) : 0.f;
                // columns behind N stay zero, whatever the norm is
                if (c < N) v[k] = (plain ? v[k] / by : float(double(v[k]) / norm)) * UP_X;
            }
            high[j / 2] = __floats2half2_rn(v[0], v[1]);
            const float2 h = __half22float2(high[j / 2]);
            low[j / 2] = __floats2half2_rn(v[0] - h.x, v[1] - h.y);
        }
        __half* o = to + row * (long long)Np + c0;
        *reinterpret_cast<uint4*>(o) = *reinterpret_cast<const uint4*>(high);
        *reinterpret_cast<uint4*>(o + plane) = *reinterpret_cast<const uint4*>(low);
    }
}

// ---- epilogues ---------------------------------------------------------------------------------
// Turns a thread's values into factors in place: words 2 j and 2 j + 1 get the first and the second
// pieces of values 2 j and 2 j + 1. (A conversion instruction for each value and use would cost
// more than everything else here: they go at 16 a clock and SM.)
template <int PIECES, int N>
__device__ __forceinline__ void pack_factors(float (&s)[N]) {
#pragma unroll
    for (int j = 0; j < N; j += 2) {
        const __half2 high = __floats2half2_rn(s[j], s[j + 1]);
        if constexpr (PIECES == 2) {
            const float2 h = __half22float2(high);
            const __half2 low = __floats2half2_rn(s[j] - h.x, s[j + 1] - h.y);
            s[j + 1] = __uint_as_float(*reinterpret_cast<const uint32_t*>(&low));
        }
        s[j] = __uint_as_float(*reinterpret_cast<const uint32_t*>(&high));
    }
}

// Where factors go: blocks of 64 columns x 32 rows, and blocks turned over (32 x 64).
struct FactorMaps {
    CUtensorMap straight, turned;
};

// Piece K of 64 packed values from s[C] on, through block B, to `slab` at (row, col); with MIRROR
// and `mirror` also, turned over, through the other block, to (col, row).
template <int C, int K, int B, bool MIRROR, int N>
__device__ __forceinline__ void store_factor(hg::WarpIo& io, const FactorMaps& to,
                                             const float (&s)[N], int slab, int row, int col,
                                             int cols_n, bool mirror) {
    const int lane = threadIdx.x & 31;
    if (col >= cols_n) return;
    io.acquire(B);
    uint8_t* block = io.block(B);
#pragma unroll
    for (int j = 0; j < 8; ++j)
        *hg::staged(block, lane, j) = make_uint4(
            __float_as_uint(s[C + 8 * j + K]), __float_as_uint(s[C + 8 * j + 2 + K]),
            __float_as_uint(s[C + 8 * j + 4 + K]), __float_as_uint(s[C + 8 * j + 6 + K]));
    io.store(B, &to.straight, col, row, slab);
    if (MIRROR && mirror) {
        io.acquire(B ^ 1);
        // 64 rows of 32 values, 64 bytes each
        unsigned short* turned = reinterpret_cast<unsigned short*>(io.block(B ^ 1)) + lane;
#pragma unroll
        for (int j = 0; j < 64; j += 2) {
            const uint32_t w = __float_as_uint(s[C + j + K]);
            turned[j * 32] = (unsigned short)w;
            turned[j * 32 + 32] = (unsigned short)(w >> 16);
        }
        io.store(B ^ 1, &to.turned, row, col, slab);
    }
}

// All of a thread's values as factors (and so packed).
template <int PIECES, bool MIRROR, int N>
__device__ __forceinline__ void store_factors(hg::WarpIo& io, const FactorMaps& to, float (&s)[N],
                                              int batch, int row, int col, int cols_n, bool mirror) {
    pack_factors<PIECES>(s);
    const int slab = batch * PIECES;
    store_factor<0, 0, 0, MIRROR>(io, to, s, slab, row, col, cols_n, mirror);
    if constexpr (PIECES == 2)
        store_factor<0, 1, 1, MIRROR>(io, to, s, slab + 1, row, col, cols_n, mirror);
    if constexpr (N == 128) {
        store_factor<64, 0, PIECES == 1, MIRROR>(io, to, s, slab, row, col + 64, cols_n, mirror);
        if constexpr (PIECES == 2)
            store_factor<64, 1, 1, MIRROR>(io, to, s, slab + 1, row, col + 64, cols_n, mirror);
    }
}

// s = s + f * (the pieces' sum) over a thread's columns: PIECES pieces of a matrix in blocks of 64
// columns, through the two staging blocks in turn, the next two on their way.
template <int COLS, int PIECES>
struct Adder {
    static constexpr int BLOCKS = COLS / 64 * PIECES;
    // piece I % PIECES of columns I / PIECES * 64 on, into staging block I % 2
    template <int I>
    static __device__ __forceinline__ void load(hg::WarpIo& io, const CUtensorMap* from, int slab,
                                                int row, int col, int cols_n) {
        if constexpr (I < BLOCKS) {
            constexpr int C = I / PIECES * 64;
            if (col + C < cols_n) io.load(I % 2, from, col + C, row, slab + I % PIECES);
        }
    }
    static __device__ __forceinline__ void start(hg::WarpIo& io, const CUtensorMap* from, int slab,
                                                 int row, int col, int cols_n) {
        load<0>(io, from, slab, row, col, cols_n);
        load<1>(io, from, slab, row, col, cols_n);
    }
    template <int I>
    static __device__ __forceinline__ void add(hg::WarpIo& io, const CUtensorMap* from, int slab,
                                               int row, int col, int cols_n, float f,
                                               float (&s)[COLS]) {
        if constexpr (I < BLOCKS) {
            constexpr int C = I / PIECES * 64;
            if (col + C >= cols_n) return;
            const int lane = threadIdx.x & 31;
            io.wait_load(I % 2);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint4 v = *hg::staged(io.block(I % 2), lane, j);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
                    s[C + 8 * j + 2 * k] = fmaf(f, x.x, s[C + 8 * j + 2 * k]);
                    s[C + 8 * j + 2 * k + 1] = fmaf(f, x.y, s[C + 8 * j + 2 * k + 1]);
                }
            }
            __syncwarp();  // read by all lanes
            load<I + 2>(io, from, slab, row, col, cols_n);
        }
    }
    static __device__ __forceinline__ void run(hg::WarpIo& io, const CUtensorMap* from, int slab,
                                               int row, int col, int cols_n, float f,
                                               float (&s)[COLS]) {
        add<0>(io, from, slab, row, col, cols_n, f, s);
        add<1>(io, from, slab, row, col, cols_n, f, s);
        add<2>(io, from, slab, row, col, cols_n, f, s);
        add<3>(io, from, slab, row, col, cols_n, f, s);
    }
};

// A = X X^T: the factors of A, from the tiles at and below the diagonal.
template <int BN_, int PIECES>
struct NsGram {
    static constexpr int BN = BN_;
    static constexpr int COLS = BN / 2;
    struct Params {
        FactorMaps out;
        int r;
    };
    const Params& p;
    hg::WarpIo& io;
    __device__ NsGram(const Params& p_, hg::WarpIo& io_) : p(p_), io(io_) {}
    __device__ __forceinline__ void unit(const hg::Unit& t, int row, int col, float (&s)[COLS]) {
        if (row >= p.r) return;
#pragma unroll
        for (int j = 0; j < COLS; ++j) s[j] *= UP_A / (UP_X * UP_X);
        store_factors<PIECES, true>(io, p.out, s, t.batch, row, col, p.r, t.col0 + BN <= t.row0);
    }
};

// b A + c A A, from the tiles at and below the diagonal.
template <int BN_, int PIECES>
struct NsPoly {
    static constexpr int BN = BN_;
    static constexpr int COLS = BN / 2;
    using Add = Adder<COLS, PIECES>;
    struct Params {
        CUtensorMap gram;
        FactorMaps out;
        int r;
    };
    const Params& p;
    hg::WarpIo& io;
    __device__ NsPoly(const Params& p_, hg::WarpIo& io_) : p(p_), io(io_) {}
    __device__ __forceinline__ void start(const hg::Unit& t, int row, int col) {
        if (row < p.r) Add::start(io, &p.gram, t.batch * PIECES, row, col, p.r);
    }
    __device__ __forceinline__ void unit(const hg::Unit& t, int row, int col, float b, float c,
                                         float (&s)[COLS]) {
        if (row >= p.r) return;
        c *= UP_P / (UP_A * UP_A);
#pragma unroll
        for (int j = 0; j < COLS; ++j) s[j] *= c;
        Add::run(io, &p.gram, t.batch * PIECES, row, col, p.r, b * (UP_P / UP_A), s);
        store_factors<PIECES, true>(io, p.out, s, t.batch, row, col, p.r, t.col0 + BN <= t.row0);
    }
};

// X = a X + (product), in pieces for the next step or as the result. X always has two pieces.
template <int BN_>
struct NsUpdate {
    static constexpr int BN = BN_;
    static constexpr int COLS = BN / 2;
    using Add = Adder<COLS, 2>;
    struct Params {
        FactorMaps x[2];  // of X before a step and after it, by the step's parity
        int M, N;
        void* result;
        long long ldo, stride;
        int dtype, wide;
    };
    const Params& p;
    hg::WarpIo& io;
    __device__ NsUpdate(const Params& p_, hg::WarpIo& io_) : p(p_), io(io_) {}
    __device__ __forceinline__ void start(const hg::Unit& t, int row, int col, int odd) {
        if (row < p.M) Add::start(io, &p.x[odd].straight, t.batch * 2, row, col, p.N);
    }

    // 32 words from word C on, through block B, to the result's columns `col` on
    template <int C, int B, int SIZE>
    __device__ __forceinline__ void result(const hg::Unit& t, int row, int col,
                                           const float (&s)[COLS]) {
        if (col >= p.N) return;
        io.acquire(B);
        hg::stage_words<C>(io.block(B), s);
        const int bytes = min(128, (p.N - col) * SIZE);
        char* base = static_cast<char*>(p.result) + (t.batch * p.stride + row * p.ldo + col) * SIZE;
        hg::store_block<SIZE>(io.block(B),
                              {base, p.ldo * SIZE, p.M - row, bytes, p.wide && bytes % 16 == 0});
    }

    __device__ __forceinline__ void unit(const hg::Unit& t, int row, int col, int odd, float a,
                                         bool last, float (&s)[COLS]) {
        if (row >= p.M) return;
        const float down = last ? 1.f / (UP_P * UP_X) : 1.f / UP_P;
#pragma unroll
        for (int j = 0; j < COLS; ++j) s[j] *= down;
        Add::run(io, &p.x[odd].straight, t.batch * 2, row, col, p.N, last ? a / UP_X : a, s);
        if (!last) {
            store_factors<2, false>(io, p.x[odd ^ 1], s, t.batch, row, col, p.N, false);
            return;
        }
        if (p.dtype == SGEMM_FLOAT32) {
            result<0, 0, 4>(t, row, col, s);
            result<32, 1, 4>(t, row, col + 32, s);
            if constexpr (COLS == 128) {
                result<64, 0, 4>(t, row, col + 64, s);
                result<96, 1, 4>(t, row, col + 96, s);
            }
            return;
        }
        const bool bf16 = p.dtype == SGEMM_BFLOAT16;
#pragma unroll
        for (int j = 0; j < COLS; j += 2)
            s[j / 2] = __uint_as_float(bf16 ? hg::pack2<true>(s[j], s[j + 1])
                                            : hg::pack2<false>(s[j], s[j + 1]));
        result<0, 0, 2>(t, row, col, s);
        if constexpr (COLS == 128) result<32, 1, 2>(t, row, col + 64, s);
    }
};

// The whole iteration as a chain of phases: three for each step. Launching them one by one costs
// some 6 us each where they are small (a launch, barriers and TMEM set up, the code fetched anew).
template <int BN_, int PIECES>
struct NsChain {
    static constexpr int BN = BN_;
    static constexpr int COLS = BN / 2;
    static constexpr int PROBLEMS = 6;
    static constexpr bool CHAIN = true;
    using Gram = NsGram<BN, PIECES>;
    using Poly = NsPoly<BN, PIECES>;
    using Update = NsUpdate<BN>;
    struct Params {
        typename Gram::Params gram;
        typename Poly::Params poly;
        typename Update::Params update;
        int steps;
        float coefficients[3 * MAX_STEPS];
    };
    const Params& p;
    Gram gram;
    Poly poly;
    Update update;
    __device__ NsChain(const Params& p_, int, hg::WarpIo& io)
        : p(p_), gram(p_.gram, io), poly(p_.poly, io), update(p_.update, io) {}
    // (the update reads an X that was stored three phases before, but the phases between may not
    // have begun when a unit is handed out)
    __device__ __forceinline__ bool reads(const hg::Unit& t) const { return t.phase % 3 != 0; }
    __device__ __forceinline__ void start(const hg::Unit& t, int row, int col) {
        const int type = t.phase % 3;
        if (type == 1)
            poly.start(t, row, col);
        else if (type == 2)
            update.start(t, row, col, t.problem == 5);
    }
    __device__ __forceinline__ void unit(const hg::Unit& t, int row, int col, float (&s)[COLS]) {
        const int step = t.phase / 3, type = t.phase - 3 * step;
        const float* c = p.coefficients + 3 * step;
        if (type == 0)
            gram.unit(t, row, col, s);
        else if (type == 1)
            poly.unit(t, row, col, c[1], c[2], s);
        else
            update.unit(t, row, col, t.problem == 5, c[0], step == p.steps - 1, s);
    }
};

// ---- host -----------------------------------------------------------------------------------------
struct Call {
    const void* G;
    int dtype, count, M, N;
    long long ldg, stride_g;
    void* out;
    long long ldo, stride_o;
    int steps;
    const float* coefficients;
    float eps;
};

struct Layout {
    size_t total = 0;
    size_t add(size_t bytes) {
        const size_t at = total;
        total += (bytes + 255) & ~size_t(255);
        return at;
    }
};

// Products of one piece each, or of low.high, high.low and high.high pieces.
void set_products(hg::Problem& p, int pieces) {
    p.planes_a = p.planes_b = pieces;
    p.products = pieces == 1 ? 1 : 3;
    if (pieces == 2) p.pa[0] = p.pb[1] = 1;
}

// counters: of claimed units, then of each phase's finished ones
template <int BN, int PIECES>
cudaError_t iterate(const Call& a, const DeviceInfo& info, __half* (&x)[2], __half* gram,
                    __half* poly, int* counters, int Np, int rp, cudaStream_t s) {
    const bool tall = a.M > a.N;
    const int r = std::min(a.M, a.N), q = std::max(a.M, a.N);
    const long long x_plane = (long long)a.M * Np, r_plane = (long long)r * rp;
    const int slabs = a.count * PIECES;
    using Chain = NsChain<BN, PIECES>;
    hg::Args<6> g;
    std::memset(&g, 0, sizeof g);
    g.problems = 3;
    g.rounds = a.steps;
    g.counter = counters;
    g.done = counters + 1;
    g.err = info.error_word;
    // 16-bit results bear an accumulator that is cut off 4 * 256 times (2^-15 of a sum, at most)
    g.seg_steps = a.dtype == SGEMM_FLOAT32 ? 8 : 256;
    // operand maps: k contiguous, or the other index
    auto x_operand = [&](CUtensorMap& m, int i, bool mn, int rows_of_cta) {
        return hg::encode_operand(&m, x[i], false, a.N, a.M, Np, 2 * a.count, x_plane,
                                  hg::box_rows(mn, rows_of_cta));
    };
    auto r_operand = [&](CUtensorMap& m, const __half* base, int rows_of_cta) {
        return hg::encode_operand(&m, base, false, r, r, rp, slabs, r_plane, rows_of_cta);
    };
    for (int i = 0; i < 2; ++i) {
        hg::Problem* p = g.p + 3 * i;
        for (int j = 0; j < 3; ++j) {
            p[j].batch = a.count;
            p[j].splits = 1;
            p[j].group = 8;
            set_products(p[j], PIECES);
        }
        p[0].planes_a = p[0].planes_b = 2;
        (tall ? p[2].planes_a : p[2].planes_b) = 2;
        // A = X X^T: both operands along the columns; tall, X^T X: both along the rows
        p[0].M = p[0].N = r;
        p[0].K = q;
        p[0].symmetric = 1;
        p[0].a_mn = p[0].b_mn = tall;
        p[0].idesc = hg::instruction(false, tall, tall);
        // A A, symmetric both
        p[1].M = p[1].N = p[1].K = r;
        p[1].symmetric = 1;
        p[1].idesc = hg::instruction(false, false, false);
        // the polynomial P times X, whose columns are contiguous; tall: X times P
        p[2].M = a.M;
        p[2].N = a.N;
        p[2].K = r;
        p[2].b_mn = !tall;
        p[2].idesc = hg::instruction(false, false, !tall);
        CUtensorMap *ma = g.a + 3 * i, *mb = g.b + 3 * i;
        if (!x_operand(ma[0], i, tall, hg::HALF_M) || !x_operand(mb[0], i, tall, BN / 2) ||
            !r_operand(ma[1], gram, hg::HALF_M) || !r_operand(mb[1], gram, BN / 2))
            return cudaErrorInvalidValue;
        if (tall ? !x_operand(ma[2], i, false, hg::HALF_M) || !r_operand(mb[2], poly, BN / 2)
                 : !r_operand(ma[2], poly, hg::HALF_M) || !x_operand(mb[2], i, true, 0))
            return cudaErrorInvalidValue;
    }
    // the epilogues' blocks
    typename Chain::Params p;
    auto factor_maps = [&](FactorMaps& m, const __half* base, int cols, int rows, int ld, int n) {
        const long long plane = (long long)rows * ld;
        return hg::encode_block(&m.straight, base, 2, cols, rows, ld, n, plane, 64, 32) &&
               hg::encode_block(&m.turned, base, 2, cols, rows, ld, n, plane, 32, 64);
    };
    if (!factor_maps(p.gram.out, gram, r, r, rp, slabs) ||
        !factor_maps(p.poly.out, poly, r, r, rp, slabs) ||
        !factor_maps(p.update.x[0], x[0], a.N, a.M, Np, 2 * a.count) ||
        !factor_maps(p.update.x[1], x[1], a.N, a.M, Np, 2 * a.count))
        return cudaErrorInvalidValue;
    const int size = a.dtype == SGEMM_FLOAT32 ? 4 : 2;
    p.gram.r = p.poly.r = r;
    p.poly.gram = p.gram.out.straight;
    p.update.M = a.M;
    p.update.N = a.N;
    p.update.result = a.out;
    p.update.ldo = a.ldo;
    p.update.stride = a.stride_o;
    p.update.dtype = a.dtype;
    p.update.wide = aligned16(a.out) && a.ldo * size % 16 == 0 && a.stride_o * size % 16 == 0;
    p.steps = a.steps;
    std::memset(p.coefficients, 0, sizeof p.coefficients);
    std::memcpy(p.coefficients, a.coefficients, size_t(3) * a.steps * sizeof(float));
    return hg::launch_gemm<Chain>(g, p, info.sm_count, s);
}

template <class T_IN, int PIECES>
cudaError_t run(const Call& a, const DeviceInfo& info, int dev, cudaStream_t s) {
    const int r = std::min(a.M, a.N);
    const int Np = (a.N + 7) / 8 * 8, rp = (r + 7) / 8 * 8;
    const size_t x_plane = size_t(a.M) * Np, r_plane = size_t(r) * rp;
    const long long groups = (long long)a.M * ((a.N + 7) / 8);
    const int most = std::max(1, std::min(MAX_NORM_CTAS, 2048 / a.count + 1));
    const int ctas = int(std::min<long long>(most, (groups + NORM_THREADS - 1) / NORM_THREADS));
    Layout lay;
    const int n_counters = 1 + 3 * a.steps * a.count;
    const size_t at_counters = lay.add(size_t(n_counters) * sizeof(int));
    const size_t at_norm = lay.add(size_t(a.count) * ctas * sizeof(double));
    const size_t at_x0 = lay.add(x_plane * 4 * a.count);
    const size_t at_x1 = a.steps > 1 ? lay.add(x_plane * 4 * a.count) : at_x0;
    const size_t at_gram = lay.add(r_plane * 2 * PIECES * a.count);
    const size_t at_poly = lay.add(r_plane * 2 * PIECES * a.count);
    Scratch scratch;
    cudaError_t e = scratch.alloc(dev, lay.total, s);
    if (e != cudaSuccess) return e;
    uint8_t* base = static_cast<uint8_t*>(scratch.ptr);
    int* counters = reinterpret_cast<int*>(base + at_counters);
    double* partial = reinterpret_cast<double*>(base + at_norm);
    __half* x[2] = {reinterpret_cast<__half*>(base + at_x0),
                    reinterpret_cast<__half*>(base + at_x1)};
    __half* gram = reinterpret_cast<__half*>(base + at_gram);
    __half* poly = reinterpret_cast<__half*>(base + at_poly);
    const T_IN* G = static_cast<const T_IN*>(a.G);
    const dim3 grid(ctas, a.count);
    // both kernels have one grid row for each matrix
    auto launch2 = [&](auto kernel, unsigned threads, auto... args) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = grid;
        cfg.blockDim = dim3(threads);
        cfg.stream = s;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        count_launch();
        return cudaLaunchKernelEx(&cfg, kernel, args...);
    };
    e = launch2(ns_norm<T_IN>, NORM_THREADS, G, a.ldg, a.stride_g, a.M, a.N, partial, counters,
                n_counters);
    if (e != cudaSuccess) return e;
    e = launch2(ns_convert<T_IN>, CONVERT_THREADS, G, a.ldg, a.stride_g, a.M, a.N, Np,
                static_cast<const double*>(partial), ctas, a.eps, x[0]);
    if (e != cudaSuccess) return e;
    // 128 columns a tile where 256 would leave pairs without one
    const int tiles = ((a.M + 255) / 256) * ((a.N + 255) / 256) * a.count;
    return tiles < std::max(info.sm_count / 2, 1)
               ? iterate<128, PIECES>(a, info, x, gram, poly, counters, Np, rp, s)
               : iterate<256, PIECES>(a, info, x, gram, poly, counters, Np, rp, s);
}

// Bytes from the first to behind the last element.
size_t extent(const Call& a, long long ld, long long stride, int size) {
    return (size_t(a.count - 1) * size_t(stride) + size_t(a.M - 1) * size_t(ld) + size_t(a.N)) *
           size_t(size);
}

}  // namespace
}  // namespace sgemm

using namespace sgemm;

extern "C" int sgemm_orthogonalize(const void* G, int dtype, int count, int M, int N, long long ldg,
                                   long long stride_g, void* out, long long ldo,
                                   long long stride_o, int steps, const float* coefficients,
                                   float eps, void* stream) {
    if (dtype < SGEMM_FLOAT32 || dtype > SGEMM_FLOAT16) return SGEMM_ERR_ARG;
    if (count < 0 || count > 4096 || M < 1 || N < 1 || M > 32768 || N > 32768) return SGEMM_ERR_ARG;
    if (std::min(M, N) > 16384 || steps < 1 || steps > MAX_STEPS || !coefficients) return SGEMM_ERR_ARG;
    if (!(eps >= 0.f) || ldg < N || ldo < N) return SGEMM_ERR_ARG;
    if (count == 0) return SGEMM_OK;
    const int size = dtype == SGEMM_FLOAT32 ? 4 : 2;
    if (!G || !out || !aligned_to(G, size) || !aligned_to(out, size)) return SGEMM_ERR_ARG;
    if (count > 1 && (stride_g < (M - 1) * ldg + N || stride_o < (M - 1) * ldo + N))
        return SGEMM_ERR_ARG;
    Call a = {G, dtype, count, M, N, ldg, stride_g, out, ldo, stride_o, steps, coefficients, eps};
    if (count == 1) a.stride_g = a.stride_o = 0;
    const bool same = G == out && ldg == ldo && a.stride_g == a.stride_o;
    if (!same && ranges_overlap(G, extent(a, ldg, a.stride_g, size), out,
                                extent(a, ldo, a.stride_o, size)))
        return SGEMM_ERR_OVERLAP;
    int dev = -1;
    const DeviceInfo* info = current_device(&dev);
    if (!info) return SGEMM_ERR_NO_DEVICE;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == SGEMM_FLOAT32    ? run<float, 2>(a, *info, dev, s)
                          : dtype == SGEMM_BFLOAT16 ? run<__nv_bfloat16, 1>(a, *info, dev, s)
                                                    : run<__half, 2>(a, *info, dev, s);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return SGEMM_ERR_CUDA;
    }
    return SGEMM_OK;
}
