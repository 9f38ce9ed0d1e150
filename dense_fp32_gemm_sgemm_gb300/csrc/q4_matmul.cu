// Few-row products with 4-bit weights: C[M x K] = A[M x N] . B, B in the packed format of
// q4.cuh.
//
// A CTA owns one strip (16 columns of C) and up to 8 NT columns of A^T, where a column is a
// bfloat16 piece of a row of A; its warps take the strip's chunks in turn and their sums
// are added in warp order.
#include "internal.cuh"
#include "q4.cuh"

namespace sgemm {
namespace {

constexpr int WARPS = 8;

// 8 consecutive bfloat16 from n on of piece p of a row of A; zeros past N.
__device__ __forceinline__ uint4 load_piece(const void* A, int dtype, size_t row_at, int n, int N,
                                            int p) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float x = n + i < N ? load_as_float(A, dtype, row_at + n + i) : 0.0f;
        float piece[3];
        split_pieces<3>(x, piece);
        v[i] = piece[p];
    }
    return make_uint4(pack_pieces(v[0], v[1]), pack_pieces(v[2], v[3]), pack_pieces(v[4], v[5]),
                      pack_pieces(v[6], v[7]));
}

template <int NT, int GROUP>
__global__ void __launch_bounds__(WARPS * 32)
    q4_matmul_kernel(const void* __restrict__ A, int dtype, size_t lda, int M, int pieces,
                     const uint8_t* __restrict__ data, Q4Geom geom, void* __restrict__ C,
                     size_t ldc) {
    __shared__ float red[WARPS][NT * 8][17];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = lane >> 2, c = lane & 3;
    const int strip = blockIdx.x;
    const int rows_per_cta = NT * 8 / pieces;
    const int row0 = blockIdx.y * rows_per_cta;
    const int rows = min(rows_per_cta, M - row0);
    float total[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) total[nt][i] = 0.0f;
    for (int ch = warp; ch < geom.chunks; ch += WARPS) {
        const uint8_t* chunk = data + strip * geom.strip_bytes() + size_t(ch) * geom.chunk_bytes;
        const uint4 w0 = __ldg(reinterpret_cast<const uint4*>(chunk) + lane);
        const uint4 w1 = __ldg(reinterpret_cast<const uint4*>(chunk + 512) + lane);
        const uint32_t words[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
        q4_chunk<NT, GROUP>(
            words, chunk + kQ4CodeBytes, geom.zeros, geom.fp16, lane,
            [&](int b, int nt) {
                const int col = nt * 8 + r, row = col / pieces;
                if (row >= rows) return make_uint4(0, 0, 0, 0);
                return load_piece(A, dtype, (row0 + row) * lda, ch * kQ4ChunkN + 32 * b + 8 * c,
                                  geom.N, col - row * pieces);
            },
            total);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) red[warp][nt * 8 + 2 * c + (i & 1)][r + 8 * (i >> 1)] = total[nt][i];
    __syncthreads();
    for (int i = threadIdx.x; i < rows * kQ4StripK; i += WARPS * 32) {
        const int row = i / kQ4StripK, col = i % kQ4StripK;
        const int k = strip * kQ4StripK + col;
        float s = 0.0f;
        for (int w = 0; w < WARPS; ++w)
            for (int p = 0; p < pieces; ++p) s += red[w][row * pieces + p][col];
        if (k < geom.K) store_from_float(C, dtype, (row0 + row) * ldc + k, s);
    }
}

template <int NT>
cudaError_t launch(const void* A, int dtype, size_t lda, int M, const sgemm_q4& w, void* C,
                   size_t ldc, cudaStream_t stream) {
    const Q4Geom g = q4_geom(w);
    const int pieces = pieces_of(dtype);
    const int rows_per_cta = NT * 8 / pieces;
    const dim3 grid(g.strips, (M + rows_per_cta - 1) / rows_per_cta);
    const uint8_t* data = static_cast<const uint8_t*>(w.data);
    auto kernel = g.group == 32   ? q4_matmul_kernel<NT, 32>
                  : g.group == 64 ? q4_matmul_kernel<NT, 64>
                                  : q4_matmul_kernel<NT, 128>;
    kernel<<<grid, WARPS * 32, 0, stream>>>(A, dtype, lda, M, pieces, data, g, C, ldc);
    count_launch();
    return cudaGetLastError();
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
    const size_t a_bytes = (size_t(M - 1) * lda + w->N) * size;
    const size_t c_bytes = (size_t(M - 1) * ldc + w->K) * size;
    if (ranges_overlap(C, c_bytes, A, a_bytes) ||
        ranges_overlap(C, c_bytes, w->data, q4_bytes(*w)))
        return SGEMM_ERR_OVERLAP;
    if (!current_device(nullptr)) return SGEMM_ERR_NO_DEVICE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int columns = M * pieces_of(dtype);
    const cudaError_t err = columns <= 8    ? launch<1>(A, dtype, lda, M, *w, C, ldc, s)
                            : columns <= 16 ? launch<2>(A, dtype, lda, M, *w, C, ldc, s)
                                            : launch<4>(A, dtype, lda, M, *w, C, ldc, s);
    return err == cudaSuccess ? SGEMM_OK : SGEMM_ERR_CUDA;
}
