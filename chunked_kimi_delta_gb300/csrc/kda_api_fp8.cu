// kda_api_fp8.cu - C ABI of the 8-bit projection path (RMS norm, quantiser,
// matrix product): host-side argument checks, then one launcher each.
#include "kda_fp8.cuh"

using namespace kda;

namespace {

inline bool mis16(const void *p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
inline kda_status cuda_status(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }
inline bool bad_dtype(kda_dtype d) { return d != KDA_F32 && d != KDA_BF16; }
inline int64_t blocks(int64_t n) { return (n + FP8_BLOCK - 1) / FP8_BLOCK; }

__device__ __align__(256) unsigned char g_matmul_workspace[KDA_FP8_MATMUL_WORKSPACE_BYTES];

}  // namespace

extern "C" {

kda_status kda_rms_norm(const kda_rms_norm_args *a, kda_stream_t stream) {
  if (!a || a->rows < 0 || a->cols < 1 || bad_dtype(a->dtype)) return KDA_ERR_INVALID_ARG;
  if (a->rows > 0 && (!a->x || (!a->out && !a->fp8))) return KDA_ERR_INVALID_ARG;
  if (a->residual && (!a->residual_out || a->residual_out == a->out)) return KDA_ERR_INVALID_ARG;
  if (a->fp8 && (!a->fp8_scales || a->ld_fp8 < a->cols)) return KDA_ERR_INVALID_ARG;
  if (a->cols > KDA_RMS_NORM_MAX_COLS || a->rows > INT32_MAX) return KDA_ERR_UNSUPPORTED;
  if (mis16(a->x) || mis16(a->residual) || mis16(a->weight) || mis16(a->residual_out) || mis16(a->out) ||
      mis16(a->fp8) || mis16(a->fp8_scales) || (a->fp8 && a->ld_fp8 % 16 != 0))
    return KDA_ERR_ALIGNMENT;
  if (a->rows == 0) return KDA_OK;
  return cuda_status(launch_rms_norm(*a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t kda_rms_norm_bwd_workspace_size(int64_t rows, int32_t cols) {
  if (rows < 0 || cols < 1 || cols > KDA_RMS_NORM_MAX_COLS || rows > INT32_MAX) return 0;
  return rms_norm_bwd_workspace(rows, cols);
}

kda_status kda_rms_norm_bwd(const kda_rms_norm_bwd_args *a, kda_stream_t stream) {
  if (!a || a->rows < 0 || a->cols < 1 || bad_dtype(a->dtype)) return KDA_ERR_INVALID_ARG;
  if (a->rows > 0 && (!a->d_out || !a->h || !a->dx)) return KDA_ERR_INVALID_ARG;
  if (a->cols > KDA_RMS_NORM_MAX_COLS || a->rows > INT32_MAX) return KDA_ERR_UNSUPPORTED;
  if (mis16(a->d_out) || mis16(a->h) || mis16(a->weight) || mis16(a->d_residual) || mis16(a->dx) ||
      mis16(a->dweight))
    return KDA_ERR_ALIGNMENT;
  if (a->dweight && a->rows > 0) {
    if (!a->workspace || a->workspace_bytes < rms_norm_bwd_workspace(a->rows, a->cols))
      return KDA_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(a->workspace) & 255u) return KDA_ERR_ALIGNMENT;
  }
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (a->rows == 0)
    return a->dweight ? cuda_status(cudaMemsetAsync(a->dweight, 0, sizeof(float) * (size_t)a->cols, st)) : KDA_OK;
  return cuda_status(launch_rms_norm_bwd(*a, st));
}

kda_status kda_fp8_quantize(const kda_fp8_quantize_args *a, kda_stream_t stream) {
  if (!a || a->rows < 0 || a->cols < 0 || bad_dtype(a->dtype)) return KDA_ERR_INVALID_ARG;
  if (a->rows == 0 || a->cols == 0) return KDA_OK;
  if (!a->x || (!a->row && !a->col && !a->tile)) return KDA_ERR_INVALID_ARG;
  if ((a->row && !a->row_scales) || (a->col && !a->col_scales) || (a->tile && !a->tile_scales))
    return KDA_ERR_INVALID_ARG;
  if (a->ld < a->cols) return KDA_ERR_INVALID_ARG;
  // rows first: the product of any two 64-bit counts could wrap
  if (a->rows / FP8_BLOCK >= INT32_MAX / 2 || blocks(a->rows) * blocks(a->cols) > INT32_MAX / 2)
    return KDA_ERR_UNSUPPORTED;
  if (mis16(a->x) || mis16(a->row) || mis16(a->col) || mis16(a->tile) || mis16(a->row_scales) ||
      mis16(a->col_scales) || mis16(a->tile_scales) || a->ld % 16 != 0)
    return KDA_ERR_ALIGNMENT;
  return cuda_status(launch_fp8_quantize(*a, reinterpret_cast<cudaStream_t>(stream)));
}

kda_status kda_fp8_matmul(const kda_fp8_matmul_args *a, kda_stream_t stream) {
  if (!a || a->m < 0 || a->n < 0 || a->k < 0 || bad_dtype(a->out_dtype)) return KDA_ERR_INVALID_ARG;
  if (a->form != KDA_FP8_NT && a->form != KDA_FP8_NN && a->form != KDA_FP8_TN) return KDA_ERR_INVALID_ARG;
  if (a->flags & ~KDA_TEST_WAIT_TIMEOUT) return KDA_ERR_INVALID_ARG;
  if (a->m == 0 || a->n == 0) return KDA_OK;
  const int64_t es = a->out_dtype == KDA_F32 ? 4 : 2;
  if (!a->out || a->ldo < a->n) return KDA_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(a->out) % es != 0) return KDA_ERR_ALIGNMENT;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (a->k == 0)
    return cuda_status(cudaMemset2DAsync(a->out, (size_t)(a->ldo * es), 0, (size_t)(a->n * es), (size_t)a->m, st));
  if (!a->a || !a->b || !a->a_scales || !a->b_scales) return KDA_ERR_INVALID_ARG;
  if (a->lda < (a->form == KDA_FP8_TN ? a->m : a->k) || a->ldb < (a->form == KDA_FP8_NT ? a->k : a->n))
    return KDA_ERR_INVALID_ARG;
  // coordinates up to a tile past the edge stay 32-bit
  const int32_t most = INT32_MAX - 1024;
  if (a->m > most || a->n > most || a->k > most || a->lda > INT32_MAX || a->ldb > INT32_MAX ||
      blocks(a->m) * blocks(a->n) > INT32_MAX / 64)
    return KDA_ERR_UNSUPPORTED;
  if (mis16(a->a) || mis16(a->b) || mis16(a->a_scales) || mis16(a->b_scales) || a->lda % 16 != 0 ||
      a->ldb % 16 != 0)
    return KDA_ERR_ALIGNMENT;
  if (!a->workspace || a->workspace_bytes < KDA_FP8_MATMUL_WORKSPACE_BYTES) return KDA_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(a->workspace) & 255u) return KDA_ERR_ALIGNMENT;
  return cuda_status(launch_fp8_matmul(*a, st));
}

kda_status kda_fp8_matmul_shared_workspace(void **workspace) {
  if (!workspace) return KDA_ERR_INVALID_ARG;
  // The first question on a device loads the array: not an operation that a
  // capture of this thread's would record, so it need not refuse it.
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  if (cudaThreadExchangeStreamCaptureMode(&mode) != cudaSuccess) return KDA_ERR_CUDA;
  void *p = nullptr;
  const cudaError_t e = cudaGetSymbolAddress(&p, g_matmul_workspace);
  if (cudaThreadExchangeStreamCaptureMode(&mode) != cudaSuccess || e != cudaSuccess || !p) return KDA_ERR_CUDA;
  *workspace = p;
  return KDA_OK;
}

}  // extern "C"
