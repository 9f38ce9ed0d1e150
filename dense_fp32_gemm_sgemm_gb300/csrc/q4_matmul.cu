// The few-row product with 4-bit weights: checks, and the choice of its kernel.
//
// Where a row wants the centred form of the weights (q4.cuh), the CTAs that meet its value stage
// their columns again and convert. One such value in a row, against none: 1 x 8192 by 8192, bfloat16,
// 19.7 us against 10.8; 1 x 6144 by 4096, float32, 11.4 against 7.4; 16 x 8192 by 6144, bfloat16, 26.4
// against 18.3; 64 x 8192 by 65536 274 against 217.
#include "q4_stage.cuh"

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
    if (!aligned_to(A, size) || !aligned_to(C, size)) return SGEMM_ERR_ARG;
    const DeviceInfo* info = current_device(nullptr);
    if (!info) return SGEMM_ERR_NO_DEVICE;
    Q4Product args;
    args.A = A;
    args.lda = size_t(lda);
    args.M = M;
    args.dtype = dtype;
    args.row_columns = dtype == SGEMM_FLOAT32 ? 4 : pieces_of(dtype);
    args.data = static_cast<const uint8_t*>(w->data);
    args.geom = q4_geom(*w);
    args.C = C;
    args.ldc = size_t(ldc);
    args.vec = aligned16(A) && size_t(lda) * size % 16 == 0;
    args.err = info->error_word;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // Up to 8 columns go to the warp kernel; more to the tensor kernel, as many at a time as a
    // cluster's shared memory holds (8 always fit).
    const int columns = M * args.row_columns;
    cudaError_t err = cudaErrorInvalidConfiguration;
    if (columns <= 8) {
        err = launch_q4_warp(args, info->sm_count, s);
    } else {
        for (int most = columns > 16 ? 32 : 16; most >= 8 && err == cudaErrorInvalidConfiguration;
             most /= 2)
            err = launch_q4_tensor(args, most, info->sm_count, s);
    }
    return err == cudaSuccess ? SGEMM_OK : SGEMM_ERR_CUDA;
}
