// kda_api_lora.cu - C ABI of the low-rank adapters: host-side argument checks,
// then the launches.
#include "kda_lora.cuh"

using namespace kda;

namespace {

inline bool mis16(const void *p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
inline kda_status cuda_status(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

// What the forward's and the backward's arguments have in common.
template <typename A> kda_status check(const A *a) {
  if (!a || a->rows < 0 || a->n_in < 1 || a->n_out < 1 || a->rank < 1 || a->adapters < 1) return KDA_ERR_INVALID_ARG;
  if (a->dtype != KDA_F32 && a->dtype != KDA_BF16) return KDA_ERR_INVALID_ARG;
  if (a->idx_dtype != KDA_I32 && a->idx_dtype != KDA_I64) return KDA_ERR_INVALID_ARG;
  if (a->num_requests < (a->rows > 0 ? 1 : 0)) return KDA_ERR_INVALID_ARG;
  if (!a->cu_seqlens && a->rows > 0 && a->rows % a->num_requests != 0) return KDA_ERR_INVALID_ARG;
  if (a->rows > 0 && (!a->x || !a->a || !a->b || !a->idx)) return KDA_ERR_INVALID_ARG;
  if (a->rank > KDA_LORA_MAX_RANK) return KDA_ERR_UNSUPPORTED;
  // rows are 32-bit, and so is eight CTAs for each tile of 16 or 64 of them
  if (a->rows > INT32_MAX || (a->rows / 16 + a->num_requests + 1) > INT32_MAX / 8 || a->n_in > INT32_MAX - 1024 ||
      a->n_out > INT32_MAX - 1024 || a->adapters > 65535)
    return KDA_ERR_UNSUPPORTED;
  if (mis16(a->x) || mis16(a->a) || mis16(a->b) || mis16(a->scale)) return KDA_ERR_ALIGNMENT;
  return KDA_OK;
}

kda_status check_bwd(const kda_lora_bwd_args *a) {
  const kda_status s = check(a);
  if (s != KDA_OK) return s;
  if (!a->d_x && !a->d_a && !a->d_b) return KDA_ERR_INVALID_ARG;
  // 32 x 32 elements of every matrix a block of the transposes
  if ((int64_t)a->adapters * 4 * ((int64_t)a->n_in / 32 + a->n_out / 32 + 3) > INT32_MAX) return KDA_ERR_UNSUPPORTED;
  if (a->rows > 0 && !a->d_out) return KDA_ERR_INVALID_ARG;
  if (a->rows > 0 && a->d_x && (a->d_x == a->d_out || a->d_x == a->x)) return KDA_ERR_INVALID_ARG;  // both are read after it
  return mis16(a->d_out) || mis16(a->d_x_in) || mis16(a->d_x) || mis16(a->d_a) || mis16(a->d_b) ? KDA_ERR_ALIGNMENT : KDA_OK;
}

// The row shares of the gradients go by the SMs of the device; a machine
// without one answers as for the GPU that the library is made for.
int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 152;
  return n;
}

}  // namespace

extern "C" {

kda_status kda_lora(const kda_lora_args *a, kda_stream_t stream) {
  const kda_status s = check(a);
  if (s != KDA_OK) return s;
  if (a->rows > 0 && (!a->y || !a->out || a->out == a->x)) return KDA_ERR_INVALID_ARG;  // x is read by others meanwhile
  if (mis16(a->y) || mis16(a->out)) return KDA_ERR_ALIGNMENT;
  if (a->rows == 0) return KDA_OK;
  return cuda_status(lora::launch_lora(*a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t kda_lora_bwd_workspace_size(const kda_lora_bwd_args *a) {
  if (check_bwd(a) != KDA_OK) return 0;
  return lora::bwd_plan(*a, sm_count()).total;
}

kda_status kda_lora_bwd(const kda_lora_bwd_args *a, kda_stream_t stream) {
  const kda_status s = check_bwd(a);
  if (s != KDA_OK) return s;
  const lora::BwdPlan p = lora::bwd_plan(*a, sm_count());
  if (!a->workspace || a->workspace_bytes < p.total) return KDA_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(a->workspace) & 255u) return KDA_ERR_ALIGNMENT;
  return cuda_status(lora::launch_lora_bwd(*a, p, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
