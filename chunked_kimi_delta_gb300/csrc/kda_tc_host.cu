// kda_tc_host.cu - host side of the tensor-core path: TMA descriptors for the
// inputs, encoded through the driver entry point (no link-time libcuda).
#include <cudaTypedefs.h>
#include <string.h>

#include "kda_tc.cuh"

namespace kda {
namespace tcp {

namespace {

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}

// One map.  The encoder is a driver call and wants a current context, which a
// host thread has only after a call of the runtime that needs one: a thread
// that has made none is given its device's context first.
bool encode(CUtensorMap *m, CUtensorMapDataType dt, cuuint32_t rank, const void *ptr, const cuuint64_t *dims,
            const cuuint64_t *strides, const cuuint32_t *box, CUtensorMapSwizzle sw, CUtensorMapL2promotion l2) {
  auto fn = encoder();
  if (!fn) return false;
  memset(m, 0, sizeof(*m));
  const cuuint32_t es[3] = {1, 1, 1};
  auto once = [&]() {
    return fn(m, dt, rank, const_cast<void *>(ptr), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, sw, l2,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  };
  CUresult r = once();
  if (r == CUDA_ERROR_INVALID_CONTEXT) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaSetDevice(dev) != cudaSuccess) return false;
    r = once();
  }
  return r == CUDA_SUCCESS;
}

// Token-major [T_tot, H, D] tensor seen as 3-D (D, H, T_tot); a box covers
// `box0` channels of one head over 64 tokens.
bool encode3(CUtensorMap *m, CUtensorMapDataType dt, uint32_t esize, const void *ptr, int D, int H,
             int64_t T, uint32_t box0, CUtensorMapSwizzle sw) {
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)T};
  cuuint64_t strides[2] = {(cuuint64_t)D * esize, (cuuint64_t)H * D * esize};
  cuuint32_t box[3] = {box0, 1, (cuuint32_t)BT};
  return encode(m, dt, 3, ptr, dims, strides, box, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

}  // namespace

bool make_input_maps(const void *q, const void *k, const void *v, const float *x, int64_t T_tot,
                     int dk, int dv, int H, int Hk, TcMaps &maps) {
  if (T_tot <= 0 || (dk != 64 && dk != 128) || (dv != 64 && dv != 128)) return false;
  return encode3(&maps.q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, q, dk, Hk, T_tot, (uint32_t)dk,
                 CU_TENSOR_MAP_SWIZZLE_NONE) &&
         encode3(&maps.k, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, k, dk, Hk, T_tot, (uint32_t)dk,
                 CU_TENSOR_MAP_SWIZZLE_NONE) &&
         encode3(&maps.v, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, v, dv, H, T_tot, 64,
                 CU_TENSOR_MAP_SWIZZLE_128B) &&
         encode3(&maps.x, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, x, dk, H, T_tot, (uint32_t)dk,
                 CU_TENSOR_MAP_SWIZZLE_NONE);
}

bool make_out_map(const void *o, int64_t T_tot, int H, int dv, CUtensorMap &map) {
  if (T_tot <= 0 || (dv != 64 && dv != 128)) return false;
  return encode3(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, o, dv, H, T_tot, 64, CU_TENSOR_MAP_SWIZZLE_128B);
}

bool make_value_map(const void *x, int64_t T_tot, int H, CUtensorMap &map) {
  if (T_tot <= 0) return false;
  return encode3(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, x, V, H, T_tot, 64,
                 CU_TENSOR_MAP_SWIZZLE_128B);
}

bool make_byte_map(const void *p, int64_t inner, int64_t outer, int64_t pitch, uint32_t box_outer,
                   CUtensorMap &map) {
  if (inner <= 0 || outer <= 0) return false;
  cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)outer};
  cuuint64_t strides[1] = {(cuuint64_t)pitch};
  cuuint32_t box[2] = {128, box_outer};
  return encode(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, p, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

bool make_out_tile_map(const void *p, bool f32, int64_t inner, int64_t outer, int64_t pitch, uint32_t box_inner,
                       uint32_t box_outer, CUtensorMap &map) {
  if (inner <= 0 || outer <= 0) return false;
  cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)outer};
  cuuint64_t strides[1] = {(cuuint64_t)pitch * (f32 ? 4 : 2)};
  cuuint32_t box[2] = {box_inner, box_outer};
  return encode(&map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p, dims, strides, box,
                f32 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE);
}

}  // namespace tcp
}  // namespace kda
