// Newton-Schulz products: X = a X + (b A + c A A) X with A = X X^T (or the same from the right
// for a tall X), some five times over, which drive the singular values of a normalised matrix
// towards one.
//
// Three products a step. A and A A are symmetric: only tiles that reach the diagonal or lie below
// it are computed and the others written from them, so that a step of r x q (r <= q) costs
// r r q + r r r + 2 r r q operations.
//
// Precision. The iteration multiplies small singular values by a (3.4) each step, and with them
// whatever rounding put there. So X itself is kept in FP32, and only the factors of the products
// are rounded: the term a X, which carries the small values, is exact, and (b A + c A A) X adds
// little to them. With the factors in FP16 (11 bits) the result is off by 0.5 to 1.7e-3 of its
// RMS for normal, low-rank and graded matrices, about as much as by the rounding of a bfloat16
// result (1.7e-3); factors in bfloat16 give 0.5 to 1.3e-2, and 1 to 20e-2 where X itself is rounded too.
// float16 and float32 results take two FP16 pieces of each factor (22 bits) and three products:
// 3e-7 to 4e-6, as much as FP32 arithmetic's. (CPU simulations of 256 x 256 to 512 x 1024.)
// Factors are held times 2^8, so that entries down to 2^-22 keep all their bits.
#include <algorithm>
#include <cstring>

#include "half_gemm.cuh"
#include "sgemm.h"

namespace sgemm {
namespace {

constexpr float UP = 256.f;             // scale of the factors
constexpr float DOWN = 1.f / UP;
constexpr float DOWN2 = DOWN * DOWN;    // of their products
constexpr int NORM_THREADS = 256;
constexpr int MAX_NORM_CTAS = 304;      // for one matrix
constexpr int CONVERT_THREADS = 256;

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

// One or two FP16 pieces of v.
template <int PIECES>
__device__ __forceinline__ void pieces_of(float v, __half (&p)[PIECES]) {
    p[0] = __float2half_rn(v);
    if constexpr (PIECES == 2) p[1] = __float2half_rn(v - __half2float(p[0]));
}

// X = G / (norm + eps), in FP32 and as factors. Rows of Np elements, zeros behind N.
template <class T_IN, int PIECES>
__global__ void __launch_bounds__(CONVERT_THREADS)
    ns_convert(const T_IN* __restrict__ g, long long ld, long long stride, int M, int N, int Np,
               const double* __restrict__ partial, int partials, float eps, float* __restrict__ x,
               __half* __restrict__ planes) {
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
    // a norm outside FP32's range is divided by in two steps
    const bool plain = by > 0x1p-100f && by < 0x1p100f;
    const T_IN* from = g + blockIdx.y * stride;
    const long long plane = (long long)M * Np;
    float* to = x + blockIdx.y * plane;
    __half* pl = planes + blockIdx.y * PIECES * plane;
    const int groups = Np / 8;
    const long long all = (long long)M * groups;
    for (long long i = (long long)blockIdx.x * CONVERT_THREADS + threadIdx.x; i < all;
         i += (long long)gridDim.x * CONVERT_THREADS) {
        const int row = int(i / groups), c0 = int(i - (long long)row * groups) * 8;
        const T_IN* p = from + row * ld + c0;
        float v[8];
        __half q[PIECES][8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[j] = c0 + j < N ? load(p + j) : 0.f;
            // columns behind N stay zero, whatever the norm is
            if (c0 + j < N) v[j] = plain ? v[j] / by : float(double(v[j]) / norm);
            __half w[PIECES];
            pieces_of<PIECES>(v[j] * UP, w);
#pragma unroll
            for (int k = 0; k < PIECES; ++k) q[k][j] = w[k];
        }
        float4* o = reinterpret_cast<float4*>(to + row * (long long)Np + c0);
        o[0] = make_float4(v[0], v[1], v[2], v[3]);
        o[1] = make_float4(v[4], v[5], v[6], v[7]);
#pragma unroll
        for (int k = 0; k < PIECES; ++k)
            *reinterpret_cast<uint4*>(pl + k * plane + row * (long long)Np + c0) =
                *reinterpret_cast<const uint4*>(q[k]);
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
    __device__ NsGram(const Params& p_, const hg::Args&, int, hg::WarpIo& io_) : p(p_), io(io_) {}
    __device__ __forceinline__ void start(const hg::Unit&, int, int) {}
    __device__ __forceinline__ void unit(const hg::Unit& t, int row, int col, float (&s)[COLS]) {
        if (row >= p.r) return;
#pragma unroll
        for (int j = 0; j < COLS; ++j) s[j] *= DOWN;
        store_factors<PIECES, true>(io, p.out, s, t.batch, row, col, p.r, t.col0 + BN <= t.row0);
    }
};

// b A + c A A, from the tiles at and below the diagonal.
template <int BN_, int PIECES>
struct NsPoly {
    static constexpr int BN = BN_;
    static constexpr int COLS = BN / 2;
    struct Params {
        CUtensorMap gram;  // blocks of 64 columns
        FactorMaps out;
        int r;
        float b, c;
    };
    const Params& p;
    hg::WarpIo& io;
    __device__ NsPoly(const Params& p_, const hg::Args&, int, hg::WarpIo& io_) : p(p_), io(io_) {}
    // piece I % PIECES of A at columns I / PIECES * 64 of the thread's, into block I % 2
    template <int I>
    __device__ __forceinline__ void load(const hg::Unit& t, int row, int col) {
        if constexpr (I < COLS / 64 * PIECES) {
            constexpr int C = I / PIECES * 64;
            if (col + C < p.r) io.load(I % 2, &p.gram, col + C, row, t.batch * PIECES + I % PIECES);
        }
    }
    __device__ __forceinline__ void start(const hg::Unit& t, int row, int col) {
        if (row >= p.r) return;
        load<0>(t, row, col);
        load<1>(t, row, col);
    }
    template <int I>
    __device__ __forceinline__ void add(const hg::Unit& t, int row, int col, float (&s)[COLS]) {
        if constexpr (I < COLS / 64 * PIECES) {
            constexpr int C = I / PIECES * 64;
            const int lane = threadIdx.x & 31;
            if (col + C >= p.r) return;
            io.wait_load(I % 2);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint4 v = *hg::staged(io.block(I % 2), lane, j);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
                    s[C + 8 * j + 2 * k] = fmaf(p.b, f.x, s[C + 8 * j + 2 * k]);
                    s[C + 8 * j + 2 * k + 1] = fmaf(p.b, f.y, s[C + 8 * j + 2 * k + 1]);
                }
            }
            __syncwarp();  // read by all lanes
            load<I + 2>(t, row, col);
        }
    }
    __device__ __forceinline__ void unit(const hg::Unit& t, int row, int col, float (&s)[COLS]) {
        if (row >= p.r) return;
        const float c = p.c * DOWN;
#pragma unroll
        for (int j = 0; j < COLS; ++j) s[j] *= c;
        add<0>(t, row, col, s);
        add<1>(t, row, col, s);
        add<2>(t, row, col, s);
        add<3>(t, row, col, s);
        store_factors<PIECES, true>(io, p.out, s, t.batch, row, col, p.r, t.col0 + BN <= t.row0);
    }
};

// X = a X + (product): in FP32 and as factors for the next step, or as the result.
template <int BN_, int PIECES>
struct NsUpdate {
    static constexpr int BN = BN_;
    static constexpr int COLS = BN / 2;
    struct Params {
        CUtensorMap x;      // FP32, in place: blocks of 32 columns
        FactorMaps out;
        int M, N;
        float a;
        int last;           // the result goes out instead
        void* result;
        long long ldo, stride;
        int dtype, wide;
    };
    const Params& p;
    hg::WarpIo& io;
    __device__ NsUpdate(const Params& p_, const hg::Args&, int, hg::WarpIo& io_) : p(p_), io(io_) {}

    __device__ __forceinline__ void start(const hg::Unit& t, int row, int col) {
        if (row >= p.M) return;
        if (col < p.N) io.load(0, &p.x, col, row, t.batch);
        if (col + 32 < p.N) io.load(1, &p.x, col + 32, row, t.batch);
    }

    template <int C>
    __device__ __forceinline__ void step32(const hg::Unit& t, int row, int col, float (&s)[COLS]) {
        constexpr int B = C / 32 % 2;
        const int lane = threadIdx.x & 31;
        if (col + C >= p.N) return;
        io.wait_load(B);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint4 v = *hg::staged(io.block(B), lane, j);
            s[C + 4 * j] = fmaf(p.a, __uint_as_float(v.x), s[C + 4 * j] * DOWN2);
            s[C + 4 * j + 1] = fmaf(p.a, __uint_as_float(v.y), s[C + 4 * j + 1] * DOWN2);
            s[C + 4 * j + 2] = fmaf(p.a, __uint_as_float(v.z), s[C + 4 * j + 2] * DOWN2);
            s[C + 4 * j + 3] = fmaf(p.a, __uint_as_float(v.w), s[C + 4 * j + 3] * DOWN2);
        }
        if (!p.last) {
            hg::stage_words<C>(io.block(B), s);  // over the values that this lane has just read
            io.store(B, &p.x, col + C, row, t.batch);
        } else {
            __syncwarp();  // read by all lanes
        }
        if constexpr (C + 64 < COLS)
            if (col + C + 64 < p.N) io.load(B, &p.x, col + C + 64, row, t.batch);
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

    __device__ __forceinline__ void unit(const hg::Unit& t, int row, int col, float (&s)[COLS]) {
        if (row >= p.M) return;
        step32<0>(t, row, col, s);
        step32<32>(t, row, col, s);
        if constexpr (COLS == 128) {
            step32<64>(t, row, col, s);
            step32<96>(t, row, col, s);
        }
        if (!p.last) {
#pragma unroll
            for (int j = 0; j < COLS; ++j) s[j] *= UP;
            store_factors<PIECES, false>(io, p.out, s, t.batch, row, col, p.N, false);
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

template <int PIECES>
void set_planes(hg::Problem& p) {
    p.planes_a = p.planes_b = PIECES;
    p.products = PIECES == 1 ? 1 : 3;
    if (PIECES == 2) {  // low.high, high.low, high.high
        p.pa[0] = 1;
        p.pb[1] = 1;
    }
}

template <int BN, int PIECES>
cudaError_t iterate(const Call& a, const DeviceInfo& info, float* x, __half* (&factors)[2],
                    __half* gram, __half* poly, int* counters, int Np, int rp, cudaStream_t s) {
    const bool tall = a.M > a.N;
    const int r = std::min(a.M, a.N), q = std::max(a.M, a.N);
    const long long x_plane = (long long)a.M * Np, r_plane = (long long)r * rp;
    const int slabs = a.count * PIECES;
    hg::Args base;
    std::memset(&base, 0, sizeof base);
    base.problems = 1;
    base.err = info.error_word;
    hg::Problem& p = base.p[0];
    p.batch = a.count;
    p.splits = 1;
    p.group = 8;
    set_planes<PIECES>(p);
    // maps of X with k and with the other index contiguous (wide: k is a column), of A and of the
    // polynomial, with k contiguous (they are symmetric)
    hg::Args gram_args[2] = {base, base}, poly_args = base, update_args[2] = {base, base};
    for (int i = 0; i < 2; ++i) {
        hg::Args& g = gram_args[i];
        // A = X X^T: both operands along the columns; tall, X^T X: both along the rows
        if (!hg::encode_operand(&g.a[0], factors[i], false, a.N, a.M, Np, slabs, x_plane,
                                hg::box_rows(tall, hg::HALF_M)) ||
            !hg::encode_operand(&g.b[0], factors[i], false, a.N, a.M, Np, slabs, x_plane,
                                hg::box_rows(tall, BN / 2)))
            return cudaErrorInvalidValue;
        hg::Problem& gp = g.p[0];
        gp.M = gp.N = r;
        gp.K = q;
        gp.symmetric = 1;
        gp.a_mn = gp.b_mn = tall;
        gp.idesc = hg::instruction(false, tall, tall);
        // wide: P (r x r) times X, whose columns are contiguous; tall: X times P
        hg::Args& u = update_args[i];
        hg::Problem& up = u.p[0];
        up.M = a.M;
        up.N = a.N;
        up.K = r;
        up.b_mn = !tall;
        up.idesc = hg::instruction(false, false, !tall);
        const bool ok =
            tall ? hg::encode_operand(&u.a[0], factors[i], false, a.N, a.M, Np, slabs, x_plane,
                                      hg::HALF_M) &&
                       hg::encode_operand(&u.b[0], poly, false, r, r, rp, slabs, r_plane, BN / 2)
                 : hg::encode_operand(&u.a[0], poly, false, r, r, rp, slabs, r_plane, hg::HALF_M) &&
                       hg::encode_operand(&u.b[0], factors[i], false, a.N, a.M, Np, slabs, x_plane,
                                          hg::BK);
        if (!ok) return cudaErrorInvalidValue;
    }
    if (!hg::encode_operand(&poly_args.a[0], gram, false, r, r, rp, slabs, r_plane, hg::HALF_M) ||
        !hg::encode_operand(&poly_args.b[0], gram, false, r, r, rp, slabs, r_plane, BN / 2))
        return cudaErrorInvalidValue;
    hg::Problem& pp = poly_args.p[0];
    pp.M = pp.N = pp.K = r;
    pp.symmetric = 1;
    pp.idesc = hg::instruction(false, false, false);
    // the epilogues' blocks
    auto factor_maps = [&](FactorMaps& m, const __half* base, int cols, int rows, int ld) {
        const long long plane = (long long)rows * ld;
        return hg::encode_block(&m.straight, base, 2, cols, rows, ld, slabs, plane, 64, 32) &&
               hg::encode_block(&m.turned, base, 2, cols, rows, ld, slabs, plane, 32, 64);
    };
    FactorMaps gram_out, poly_out, x_out[2];
    CUtensorMap x_map;
    if (!factor_maps(gram_out, gram, r, r, rp) || !factor_maps(poly_out, poly, r, r, rp) ||
        !factor_maps(x_out[0], factors[0], a.N, a.M, Np) ||
        !factor_maps(x_out[1], factors[1], a.N, a.M, Np) ||
        !hg::encode_block(&x_map, x, 4, a.N, a.M, Np, a.count, x_plane, 32, 32))
        return cudaErrorInvalidValue;
    const int size = a.dtype == SGEMM_FLOAT32 ? 4 : 2;
    const int wide = aligned16(a.out) && a.ldo * size % 16 == 0 && a.stride_o * size % 16 == 0;
    for (int i = 0; i < a.steps; ++i) {
        const float* c = a.coefficients + 3 * i;
        hg::Args g = gram_args[i & 1], u = update_args[i & 1];
        g.counter = counters + 3 * i;
        poly_args.counter = counters + 3 * i + 1;
        u.counter = counters + 3 * i + 2;
        cudaError_t e =
            hg::launch_gemm<NsGram<BN, PIECES>>(g, {gram_out, r}, info.sm_count, s);
        if (e != cudaSuccess) return e;
        e = hg::launch_gemm<NsPoly<BN, PIECES>>(
            poly_args, {gram_out.straight, poly_out, r, c[1], c[2]}, info.sm_count, s);
        if (e != cudaSuccess) return e;
        const bool last = i == a.steps - 1;
        e = hg::launch_gemm<NsUpdate<BN, PIECES>>(
            u, {x_map, x_out[(i + 1) & 1], a.M, a.N, c[0], last, a.out, a.ldo, a.stride_o, a.dtype,
                wide},
            info.sm_count, s);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
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
    const size_t at_counters = lay.add(size_t(3) * a.steps * sizeof(int));
    const size_t at_norm = lay.add(size_t(a.count) * ctas * sizeof(double));
    const size_t at_x = lay.add(x_plane * 4 * a.count);
    const size_t at_f0 = lay.add(x_plane * 2 * PIECES * a.count);
    const size_t at_f1 = lay.add(a.steps > 1 ? x_plane * 2 * PIECES * a.count : 0);
    const size_t at_gram = lay.add(r_plane * 2 * PIECES * a.count);
    const size_t at_poly = lay.add(r_plane * 2 * PIECES * a.count);
    Scratch scratch;
    cudaError_t e = scratch.alloc(dev, lay.total, s);
    if (e != cudaSuccess) return e;
    uint8_t* base = static_cast<uint8_t*>(scratch.ptr);
    int* counters = reinterpret_cast<int*>(base + at_counters);
    double* partial = reinterpret_cast<double*>(base + at_norm);
    float* x = reinterpret_cast<float*>(base + at_x);
    __half* factors[2] = {reinterpret_cast<__half*>(base + at_f0),
                          reinterpret_cast<__half*>(base + (a.steps > 1 ? at_f1 : at_f0))};
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
                3 * a.steps);
    if (e != cudaSuccess) return e;
    e = launch2(ns_convert<T_IN, PIECES>, CONVERT_THREADS, G, a.ldg, a.stride_g, a.M, a.N, Np,
                static_cast<const double*>(partial), ctas, a.eps, x, factors[0]);
    if (e != cudaSuccess) return e;
    // 128 columns a tile where 256 would leave pairs without one
    const int tiles = ((a.M + 255) / 256) * ((a.N + 255) / 256) * a.count;
    return tiles < std::max(info.sm_count / 2, 1)
               ? iterate<128, PIECES>(a, info, x, factors, gram, poly, counters, Np, rp, s)
               : iterate<256, PIECES>(a, info, x, factors, gram, poly, counters, Np, rp, s);
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
    if (std::min(M, N) > 16384 || steps < 1 || steps > 64 || !coefficients) return SGEMM_ERR_ARG;
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
