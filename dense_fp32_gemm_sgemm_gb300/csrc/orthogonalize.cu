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
// simulations of 256 x 256 to 512 x 1024.) The first pieces are of values times a power of two, so that
// small entries stay in FP16's normal range: 2^13 for X, 2^12 for A, 2^10 for the polynomial; the second
// of what they leave, times 2^11 more, so that a value has 22 bits down to 2^-27 (X), 2^-26 and 2^-24 and
// steps of 2^-48, 2^-47 and 2^-45 below. Rows of small entries keep their own precision: one 1e-5 times as
// large as the others of 256 x 256 or 256 x 1024 is good to 1 to 5e-7, 1e-7 to 3 to 5e-6 (without the 2^11
// 0.5 to 1e-4 and 0.4 to 1e-2; FP32 0.4 to 2e-6).
//
// With two pieces, E = A - I/2 is stored in A's place, and the polynomial is c E E + (b + c) E + (b/2 + c/4) I.
// Once singular values are near one, A's diagonal holds most of its size, and a sum of A A one product, its
// square, from which the accumulator cuts all others: 2^-22 of it, which the later steps multiply by up to 20
// (64 x 999 of normal entries: 3.4e-6, with E 1.7e-6; 71 x 6384 with strong directions 1.4 and 0.6e-6). One
// half is between the squares of 0 and 1.2; with zero or one 1.3 to 4 times the error in simulations.
//
// Measured: 6144 x 8192, bfloat16, 4.1 to 4.2 ms (1.4 PFLOP/s of what symmetric products cannot do without);
// 4096 x 4096 1.08 to 1.11 ms, where whole rounds of 76 units take 1.15 of the work (gram and polynomial 2 for
// 1.8, update 4 for 3.4), the update's second term and stores 11 % and the ends of 15 phases some 8 us
// each. A finer order, in which a unit waits for its own blocks of rows alone, brought nothing.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "half_gemm.cuh"
#include "sgemm.h"

namespace sgemm {
namespace {

constexpr float UP_X = 0x1p13f, UP_A = 0x1p12f, UP_P = 0x1p10f;  // scales of the pieces
constexpr int NORM_THREADS = 256;
constexpr int MAX_NORM_CTAS = 1216;     // for one matrix: eight an SM
constexpr int MAX_STEPS = 64;

// Eight elements of a row from column c on, zeros from N on. wide: 16-byte aligned rows.
template <class T_IN>
__device__ __forceinline__ void load8(const T_IN* p, int c, int N, bool wide, float (&v)[8]) {
    if (wide && c + 8 <= N) {
        if constexpr (sizeof(T_IN) == 4) {
            const float4 a = reinterpret_cast<const float4*>(p)[0];
            const float4 b = reinterpret_cast<const float4*>(p)[1];
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
            v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
            const uint4 a = *reinterpret_cast<const uint4*>(p);
            const T_IN* e = reinterpret_cast<const T_IN*>(&a);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = float(e[j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = c + j < N ? float(p[j]) : 0.f;
    }
}

// ---- the norm and the first X --------------------------------------------------------------
// FP32 sum with what its additions rounded off.
struct Compensated {
    float sum = 0.f, rest = 0.f;
    __device__ __forceinline__ void add(float s) {
        const float t = sum + s, u = t - sum;
        rest += (sum - (t - u)) + (s - u);
        sum = t;
    }
    // of all lanes' sums, in the first lane
    __device__ __forceinline__ double of_warp() {
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const float other = __shfl_down_sync(~0u, sum, o);
            rest += __shfl_down_sync(~0u, rest, o);
            add(other);
        }
        return (threadIdx.x & 31) == 0 ? double(sum) + double(rest) : 0.0;
    }
};

// The sum of a CTA's squares over groups of eight elements i0, i0 + step, ... of a matrix, in its
// first thread. Groups are squared and added in FP32, those whose largest element is not between
// 2^-50 and 2^50 after a power of two and for themselves; a warp's sums are compensated, and joined in
// FP64, of which an SM does two operations a clock.
template <int THREADS, class T_IN>
__device__ __forceinline__ double sum_squares(const T_IN* from, long long ld, int M, int N, bool wide,
                                              unsigned i0, unsigned step) {
    __shared__ double sums[THREADS / 32];
    const unsigned groups = (N + 7) / 8, all = M * groups;  // at most 2^27
    Compensated small, middle, large;
    for (unsigned i = i0; i < all; i += step) {
        const unsigned row = i / groups;
        const int c0 = int(i - row * groups) * 8;
        float v[8], top = 0.f;
        load8(from + row * ld + c0, c0, N, wide, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(v[j]));
        auto squares = [&](float f) {
            float s = 0.f;  // NaN where one of them is
#pragma unroll
            for (int j = 0; j < 8; ++j) s = fmaf(v[j] * f, v[j] * f, s);
            return s;
        };
        if (top >= 0x1p50f)
            large.add(squares(0x1p-78f));
        else if (top <= 0x1p-50f)
            small.add(squares(0x1p76f));
        else
            middle.add(squares(1.f));
    }
    double sum = middle.of_warp();
    if (__any_sync(~0u, small.sum != 0.f || large.sum != 0.f))
        sum += small.of_warp() * 0x1p-152 + large.of_warp() * 0x1p156;
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x == 0)
        for (int w = 1; w < THREADS / 32; ++w) sum += sums[w];
    return sum;
}

// 1 / (sqrt(sum) + eps) as a power of two, in two exact factors, times a number of (1/2, 1], rounded
// once for all elements. For one thread: FP64 arithmetic of a whole CTA takes microseconds.
__device__ __forceinline__ float4 divisor(double sum, float eps) {
    const double norm = sqrt(sum) + double(eps);
    if (!(norm > 0.0 && norm < 0x1p300))  // 0, infinity or NaN
        return make_float4(1.f, 1.f, float(1.0 / norm) * UP_X, 0.f);
    const int k = ilogb(norm);
    return make_float4(float(scalbn(1.0, -(k / 2))), float(scalbn(1.0, -(k - k / 2))),
                       float(1.0 / scalbn(norm, -k)) * UP_X, 0.f);
}

// X = G / norm in two pieces, the same groups. Rows of Np elements, zeros behind N.
template <class T_IN>
__device__ __forceinline__ void first_x(const T_IN* from, long long ld, int M, int N, int Np, bool wide,
                                        float4 by, __half* to, unsigned i0, unsigned step) {
    const float f0 = by.x, f1 = by.y, f2 = by.z;
    const long long plane = (long long)M * Np;
    const unsigned groups = Np / 8, all = M * groups;
    for (unsigned i = i0; i < all; i += step) {
        const unsigned row = i / groups;
        const int c0 = int(i - row * groups) * 8;
        float v[8];
        load8(from + row * ld + c0, c0, N, wide, v);
        __align__(16) __half2 high[4];
        __align__(16) __half2 low[4];
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            // columns behind N stay zero, whatever the norm is
            const float a = c0 + j < N ? ((v[j] * f0) * f1) * f2 : 0.f;
            const float b = c0 + j + 1 < N ? ((v[j + 1] * f0) * f1) * f2 : 0.f;
            high[j / 2] = __floats2half2_rn(a, b);
            const float2 h = __half22float2(high[j / 2]);
            low[j / 2] = __floats2half2_rn((a - h.x) * hg::SECOND_UP, (b - h.y) * hg::SECOND_UP);
        }
        __half* o = to + row * (long long)Np + c0;
        *reinterpret_cast<uint4*>(o) = *reinterpret_cast<const uint4*>(high);
        *reinterpret_cast<uint4*>(o + plane) = *reinterpret_cast<const uint4*>(low);
    }
}

// Partial sums of squares, one for each CTA of a matrix (grid row).
template <class T_IN>
__global__ void __launch_bounds__(NORM_THREADS)
    ns_norm(const T_IN* __restrict__ g, long long ld, long long stride, int M, int N, int wide,
            double* __restrict__ partial, int* counters, int n_counters) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int cta = blockIdx.y * gridDim.x + blockIdx.x;
    for (int i = cta * NORM_THREADS + threadIdx.x; i < n_counters;
         i += gridDim.x * gridDim.y * NORM_THREADS)
        counters[i] = 0;
    const double sum = sum_squares<NORM_THREADS>(
        g + blockIdx.y * stride, ld, M, N, wide,
        blockIdx.x * NORM_THREADS + threadIdx.x, gridDim.x * NORM_THREADS);
    if (threadIdx.x == 0) partial[cta] = sum;
}

template <class T_IN>
__global__ void __launch_bounds__(NORM_THREADS)
    ns_convert(const T_IN* __restrict__ g, long long ld, long long stride, int M, int N, int Np,
               int wide, const double* __restrict__ partial, int partials, float eps,
               __half* __restrict__ x) {
    __shared__ float4 by;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    if (threadIdx.x < 32) {
        double sum = 0.0;
        const double* mine = partial + (long long)blockIdx.y * partials;
        for (int i = threadIdx.x; i < partials; i += 32) sum += mine[i];
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
        if (threadIdx.x == 0) by = divisor(sum, eps);
    }
    __syncthreads();
    first_x(g + blockIdx.y * stride, ld, M, N, Np, wide, by,
            x + blockIdx.y * 2 * ((long long)M * Np),
            blockIdx.x * NORM_THREADS + threadIdx.x, gridDim.x * NORM_THREADS);
}

// ---- the epilogue -------------------------------------------------------------------------------
// Where factors go: blocks of 64 columns x 32 rows, and blocks turned over (32 x 64).
struct FactorMaps {
    CUtensorMap straight, turned;
};

// The whole iteration is a chain of phases, three for each step, in one launch (one by one they
// cost some 6 us each where they are small: a launch, barriers and TMEM set up). The phases share
// one epilogue:
//
//     s = f s + h (the pieces of a matrix at the tile's place), stored as pieces,
//
// for A without the second term, for the polynomial with that of A (the products of symmetric
// matrices from the tiles at and below the diagonal, the others as mirror images), for the new X
// with that of X. It is written as loops over 64 columns and over pieces with the values moved to
// where the next turn expects them: an SM fetches instructions for the first time at some 100 ns
// for each 128 bytes, and fully unrolled the three epilogues took 20 us each at their first use, a
// whole phase 5.
template <int BN_, int PIECES>
struct NsChain {
    static constexpr int BN = BN_;
    static constexpr int COLS = BN / 2;
    static constexpr int PROBLEMS = 6;
    static constexpr int PLANES = PIECES;
    static constexpr bool CHAIN = true;
    static constexpr float MIDDLE = PIECES == 2 ? 0.5f : 0.f;  // see above
    struct Params {
        FactorMaps gram, poly;
        FactorMaps x[2];  // X before a step and after it, by the step's parity; two pieces
        int r, M, N;
        void* result;     // of the last step
        long long ldo, stride;
        int dtype, wide;
        int steps;
        float coefficients[3 * MAX_STEPS];
    };
    using Io = hg::WarpIo<hg::Ring<NsChain>::BLOCKS>;
    static constexpr int AHEAD = hg::Ring<NsChain>::BLOCKS;  // blocks loaded ahead
    const Params& p;
    Io& io;
    __device__ NsChain(const Params& p_, int, Io& io_) : p(p_), io(io_) {}

    // The matrix of the second term.
    struct Second {
        const CUtensorMap* map;
        int pieces, slab, rows, cols;
    };
    __device__ __forceinline__ Second second(const hg::Unit& t, int type) const {
        if (type == 1) return {&p.gram.straight, PIECES, t.batch * PIECES, p.r, p.r};
        return {&p.x[t.problem == 5].straight, 2, t.batch * 2, p.M, p.N};
    }
    // Block n of the second term: 64 columns, piece by piece.
    __device__ __forceinline__ void load(const Second& m, int n, int row, int col) {
        const int c = m.pieces == 2 ? n >> 1 : n;
        if (c * 64 < COLS && col + c * 64 < m.cols)
            io.load(Io::of(n), m.map, col + c * 64, row, m.slab + (m.pieces == 2 ? n & 1 : 0));
    }
    __device__ __forceinline__ bool reads(const hg::Unit& t) const { return t.phase % 3 != 0; }
    __device__ __forceinline__ void start(const hg::Unit& t, int row, int col) {
        const int type = t.phase % 3;
        if (type == 0) return;
        const Second m = second(t, type);
        if (row >= m.rows) return;
        load(m, 0, row, col);
        if (AHEAD > 1) load(m, 1, row, col);
    }

    // The next 64 columns to the front.
    static __device__ __forceinline__ void turn(float (&s)[COLS]) {
        if constexpr (COLS == 128) {
#pragma unroll
            for (int j = 0; j < 64; ++j) {
                const float v = s[j];
                s[j] = s[j + 64];
                s[j + 64] = v;
            }
        }
    }

    // The first 32 words of every lane to columns `col` on of the result.
    template <int SIZE>
    __device__ __forceinline__ void store_result(const hg::Unit& t, int block, int row, int col,
                                                 const float (&s)[COLS]) {
        io.acquire(block);
        hg::stage_words<0>(io.block(block), s);
        const int bytes = min(128, (p.N - col) * SIZE);
        char* base = static_cast<char*>(p.result) + (t.batch * p.stride + row * p.ldo + col) * SIZE;
        hg::store_block<SIZE>(io.block(block),
                              {base, p.ldo * SIZE, p.M - row, bytes, p.wide && bytes % 16 == 0});
    }

    __device__ __forceinline__ void unit(const hg::Unit& t, int row, int col, float (&s)[COLS]) {
        const int lane = threadIdx.x & 31;
        const int step = t.phase / 3, type = t.phase - 3 * step;
        const float* c = p.coefficients + 3 * step;
        const bool last = type == 2 && step == p.steps - 1;
        const int rows_n = type == 2 ? p.M : p.r, cols_n = type == 2 ? p.N : p.r;
        if (row >= rows_n || col >= cols_n) return;
        float f, h = 0.f, unit = 0.f;  // unit: times the identity
        if (type == 0) {
            f = UP_A / (UP_X * UP_X);
            unit = -MIDDLE * UP_A;
        } else if (type == 1) {
            f = c[2] * (UP_P / (UP_A * UP_A));
            h = (c[1] + 2.f * MIDDLE * c[2]) * (UP_P / UP_A);
            unit = (c[1] + MIDDLE * c[2]) * MIDDLE * UP_P;
        } else {
            f = last ? 1.f / (UP_P * UP_X) : 1.f / UP_P;
            h = last ? c[0] / UP_X : c[0];
        }
#pragma unroll
        for (int j = 0; j < COLS; ++j) s[j] *= f;
        if (type != 0) {
            const Second m = second(t, type);
            int n = 0;
#pragma unroll 1
            for (int at = 0; at < COLS; at += 64) {
#pragma unroll 1
                for (int k = 0; k < m.pieces && col + at < cols_n; ++k, ++n) {
                    const float times = k == 0 ? h : h * hg::SECOND_DOWN;
                    io.wait_load(Io::of(n));
                    uint8_t* block = io.block(Io::of(n));
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint4 v = *hg::staged(block, lane, j);
                        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 x =
                                __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                            s[8 * j + 2 * i] = fmaf(times, x.x, s[8 * j + 2 * i]);
                            s[8 * j + 2 * i + 1] = fmaf(times, x.y, s[8 * j + 2 * i + 1]);
                        }
                    }
                    __syncwarp();  // read by all lanes
                    load(m, n + AHEAD, row, col);
                }
                turn(s);
            }
        }
        if (MIDDLE != 0.f && type != 2 && row + 32 > col && row < col + COLS) {
            const int diagonal = row + lane - col;
#pragma unroll
            for (int j = 0; j < COLS; ++j) s[j] = j == diagonal ? s[j] + unit : s[j];
        }
        if (!last)
            store_pieces(t, type, row, col, cols_n, s);
        else
            store_last(t, row, col, s);
    }

    // All values as pieces of the next factor. The words 2 j and 2 j + 1 get the first and second
    // pieces of values 2 j and 2 j + 1: one conversion for two values and each piece.
    __device__ __forceinline__ void store_pieces(const hg::Unit& t, int type, int row, int col,
                                                 int cols_n, float (&s)[COLS]) {
        const int lane = threadIdx.x & 31;
        const int pieces = type == 2 ? 2 : PIECES;
        const FactorMaps& to =
            type == 0 ? p.gram : type == 1 ? p.poly : p.x[t.problem != 5];
        const int slab = t.batch * pieces;
        const bool mirror = type != 2 && t.col0 + BN <= t.row0;
        int block = 0;
#pragma unroll 1
        for (int at = col; at < min(col + COLS, cols_n); at += 64) {
#pragma unroll
            for (int j = 0; j < 64; j += 2) {
                const __half2 high = __floats2half2_rn(s[j], s[j + 1]);
                const float2 v = __half22float2(high);
                const __half2 low = __floats2half2_rn((s[j] - v.x) * hg::SECOND_UP,
                                                      (s[j + 1] - v.y) * hg::SECOND_UP);
                s[j] = __uint_as_float(*reinterpret_cast<const uint32_t*>(&high));
                s[j + 1] = __uint_as_float(*reinterpret_cast<const uint32_t*>(&low));
            }
#pragma unroll 1
            for (int k = 0; k < pieces; ++k) {
                io.acquire(block);
                uint8_t* straight = io.block(block);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    *hg::staged(straight, lane, j) =
                        make_uint4(__float_as_uint(s[8 * j]), __float_as_uint(s[8 * j + 2]),
                                   __float_as_uint(s[8 * j + 4]), __float_as_uint(s[8 * j + 6]));
                io.store(block, &to.straight, at, row, slab + k);
                block = Io::of(block + 1);
                if (mirror) {
                    // turned over: 64 rows of 32 values, 64 bytes each
                    io.acquire(block);
                    unsigned short* turned =
                        reinterpret_cast<unsigned short*>(io.block(block)) + lane;
#pragma unroll
                    for (int j = 0; j < 64; j += 2) {
                        const uint32_t w = __float_as_uint(s[j]);
                        turned[j * 32] = (unsigned short)w;
                        turned[j * 32 + 32] = (unsigned short)(w >> 16);
                    }
                    io.store(block, &to.turned, row, at, slab + k);
                    block = Io::of(block + 1);
                }
#pragma unroll
                for (int j = 0; j < 64; j += 2) s[j] = s[j + 1];
            }
            turn(s);
        }
    }

    __device__ __forceinline__ void store_last(const hg::Unit& t, int row, int col,
                                               float (&s)[COLS]) {
        const bool f32 = p.dtype == SGEMM_FLOAT32;
        if (!f32) {
            const bool bf16 = p.dtype == SGEMM_BFLOAT16;
#pragma unroll
            for (int j = 0; j < COLS; j += 2)
                s[j / 2] = __uint_as_float(bf16 ? hg::pack2<true>(s[j], s[j + 1])
                                                : hg::pack2<false>(s[j], s[j + 1]));
        }
        const int each = f32 ? 32 : 64, end = min(col + COLS, p.N);
        int block = 0;
#pragma unroll 1
        for (int at = col; at < end; at += each) {
            if (f32)
                store_result<4>(t, block, row, at, s);
            else
                store_result<2>(t, block, row, at, s);
            block = Io::of(block + 1);
#pragma unroll
            for (int j = 0; j + 32 < COLS; ++j) s[j] = s[j + 32];
        }
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

// Factors of one piece each, or of two that a stage holds together (all but the product of the second ones).
void set_products(hg::Problem& p, int pieces) {
    p.planes_a = p.planes_b = pieces;
    p.products = 1;
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
    // 16-bit results: 128 MMAs at most between two additions in FP32, which cut off 2^-16 of a sum of one
    // sign.
    // float32 (MMAs of the first pieces): 8 where the smaller side is below 512 and FP32 arithmetic itself is
    // good to 1 to 2e-6 (150 x 1408: 1.2e-6, with 4 0.8, with 12 1.7, FP32 1.4; 64 x 20000 769 us, with 4 980);
    // 12 below 2048 (1210 x 5480: 1.5e-6, with 8 1.1, with 16 2.0, FP32 2.7; 550 us, 543 and 532); then 24
    // (2102 x 3552: 1.9e-6, with 12 1.1, FP32 2.5; 6144 x 8192 12.1 and 12.5 ms).
    g.seg_steps = a.dtype != SGEMM_FLOAT32 ? 32 : r < 512 ? 2 : r < 2048 ? 3 : 6;
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
            p[j].group = 8;  // 6144 x 8192, bfloat16: 3.50 ms, with 2 3.61, with 32 3.57
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
    // the epilogue's blocks
    typename Chain::Params p;
    auto factor_maps = [&](FactorMaps& m, const __half* base, int cols, int rows, int ld, int n) {
        const long long plane = (long long)rows * ld;
        return hg::encode_block(&m.straight, base, 2, cols, rows, ld, n, plane, 64, 32) &&
               hg::encode_block(&m.turned, base, 2, cols, rows, ld, n, plane, 32, 64);
    };
    if (!factor_maps(p.gram, gram, r, r, rp, slabs) || !factor_maps(p.poly, poly, r, r, rp, slabs) ||
        !factor_maps(p.x[0], x[0], a.N, a.M, Np, 2 * a.count) ||
        !factor_maps(p.x[1], x[1], a.N, a.M, Np, 2 * a.count))
        return cudaErrorInvalidValue;
    const int size = a.dtype == SGEMM_FLOAT32 ? 4 : 2;
    p.r = r;
    p.M = a.M;
    p.N = a.N;
    p.result = a.out;
    p.ldo = a.ldo;
    p.stride = a.stride_o;
    p.dtype = a.dtype;
    p.wide = aligned16(a.out) && a.ldo * size % 16 == 0 && a.stride_o * size % 16 == 0;
    p.steps = a.steps;
    std::memset(p.coefficients, 0, sizeof p.coefficients);
    std::memcpy(p.coefficients, a.coefficients, size_t(3) * a.steps * sizeof(float));
    return hg::launch_gemm<Chain>(g, p, info.sm_count, s);
}

// Columns of a tile with factors of one piece: whatever gives the shorter step by what was measured, 522
// cycles for a stage of 256 columns and 430 for one of 128, and what the last unit's epilogue adds to a
// phase, 6000 or 3000. A phase of one matrix takes whole rounds of units; the phases of several overlap.
// (Two pieces have 128: their second accumulators take the rest of the tensor memory.)
template <int BN>
double step_cycles(const Call& a, int pairs) {
    const int r = std::min(a.M, a.N), q = std::max(a.M, a.N);
    hg::Problem square = {}, whole = {};
    square.symmetric = 1;
    const int tiles_r = hg::ceil_div(r, hg::BM);
    const double units_r =
        double(a.count) * hg::tile_count<BN>(square, tiles_r, hg::ceil_div(r, BN));
    const double units_x = double(a.count) * hg::tile_count<BN>(whole, hg::ceil_div(a.M, hg::BM),
                                                                hg::ceil_div(a.N, BN));
    auto rounds = [&](double units) {
        const double n = units / pairs;
        return a.count == 1 ? std::ceil(n) : std::max(n, 1.);
    };
    const double k_q = hg::ceil_div(q, hg::BK), k_r = hg::ceil_div(r, hg::BK);
    return (rounds(units_r) * (k_q + k_r) + rounds(units_x) * k_r) * (BN == 256 ? 522. : 430.) +
           3 * (BN == 256 ? 6000. : 3000.);
}

template <class T_IN, int PIECES>
cudaError_t run(const Call& a, const DeviceInfo& info, int dev, cudaStream_t s) {
    const int r = std::min(a.M, a.N);
    // rows of whole 128-byte lines, so that TMA's boxes do not straddle them
    const int Np = (a.N + 63) / 64 * 64, rp = (r + 63) / 64 * 64;
    const size_t x_plane = size_t(a.M) * Np, r_plane = size_t(r) * rp;
    const long long groups = (long long)a.M * ((a.N + 7) / 8);
    const int most = std::max(1, std::min(MAX_NORM_CTAS, 4096 / a.count + 1));
    const int ctas = int(std::min<long long>(most, (groups + NORM_THREADS - 1) / NORM_THREADS));
    hg::Layout lay;
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
    const int size = sizeof(T_IN);
    const int wide = aligned16(G) && a.ldg * size % 16 == 0 && a.stride_g * size % 16 == 0;
    // both kernels have one grid row for each matrix
    auto launch2 = [&](auto kernel, auto... args) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(ctas, a.count);
        cfg.blockDim = dim3(NORM_THREADS);
        cfg.stream = s;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        count_launch();
        return cudaLaunchKernelEx(&cfg, kernel, args...);
    };
    e = launch2(ns_norm<T_IN>, G, a.ldg, a.stride_g, a.M, a.N, wide, partial, counters, n_counters);
    if (e != cudaSuccess) return e;
    e = launch2(ns_convert<T_IN>, G, a.ldg, a.stride_g, a.M, a.N, Np, wide,
                static_cast<const double*>(partial), ctas, a.eps, x[0]);
    if (e != cudaSuccess) return e;
    if constexpr (PIECES == 1) {
        const int pairs = std::max(info.sm_count / 2, 1);
        if (step_cycles<256>(a, pairs) <= step_cycles<128>(a, pairs))
            return iterate<256, 1>(a, info, x, gram, poly, counters, Np, rp, s);
    }
    return iterate<128, PIECES>(a, info, x, gram, poly, counters, Np, rp, s);
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
