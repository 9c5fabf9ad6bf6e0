// kda_fp8.cuh - scaled 8-bit values: the block exponent, rounding to e4m3,
// eight-element loads and stores shared by the norm and the quantiser, and
// the launchers of the 8-bit projection path.
#pragma once

#include <cuda_fp8.h>

#include "kda_internal.cuh"

namespace kda {

constexpr int FP8_BLOCK = 128;          // columns or rows that share a scale
constexpr uint32_t FP8_SCALE_ONE = 127; // scale byte of 1.0

// Scale byte (e + 127) of a block whose largest finite magnitude is amax: the
// smallest e >= -127 with amax <= 448 * 2^e.  448 = 1.75 * 2^8, so with
// amax = 1.f * 2^(E - 127) the answer is E - 135, one more when 1.f > 1.75:
// exact, straight from the bits.
__device__ __forceinline__ uint32_t fp8_scale_byte(float amax) {
  const uint32_t u = __float_as_uint(amax);
  if (u == 0) return FP8_SCALE_ONE;
  const int b = (int)(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return (uint32_t)(b < 0 ? 0 : b);
}
// 2^-e of a scale byte below 248 (which fp8_scale_byte never exceeds).
__device__ __forceinline__ float fp8_inv_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// Four scaled values as e4m3 bytes, lowest first.  None is infinite
// (drop_infinities): the conversion would clamp it to 448.
__device__ __forceinline__ uint32_t fp8_pack4(float a, float b, float c, float d, float inv) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a * inv, b * inv), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c * inv, d * inv), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}

// Largest magnitude, NaN left out (fmaxf returns the other operand).
__device__ __forceinline__ float block_amax(const float (&y)[8]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(y[i]));
  return m;
}
// e4m3 has no infinity: they become NaN, and so leave block_amax alone.
__device__ __forceinline__ void drop_infinities(float (&y)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = fmaf(y[i], 0.f, y[i]);
}

// Eight consecutive elements of a row, zeros from element `n` on (n <= 0:
// none).  VEC: 16-byte accesses, n is 8 or none.
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T *p, int n, float (&v)[8]) {
  if (VEC) {
    if (n > 0) {
      if constexpr (sizeof(T) == 2) {
        const uint4 raw = *reinterpret_cast<const uint4 *>(p);
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // bf16 is the upper half of an fp32
          v[2 * i] = __uint_as_float(w[i] << 16);
          v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
      } else {
        const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? to_f32<T>(p[i]) : 0.f;
  }
}
template <typename T, bool VEC>
__device__ __forceinline__ void store8(T *p, int n, const float (&v)[8]) {
  if (VEC) {
    if (n <= 0) return;
    if constexpr (sizeof(T) == 2) {
      __nv_bfloat162 o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(o);
    } else {
      reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = from_f32<T>(v[i]);
  }
}
// Eight e4m3 bytes at an 8-byte aligned address, the first n of them.
__device__ __forceinline__ void store8_fp8(uint8_t *p, int n, uint32_t lo, uint32_t hi) {
  if (n >= 8) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(lo, hi);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = (uint8_t)((i < 4 ? lo >> (8 * i) : hi >> (8 * (i - 4))) & 0xFFu);
  }
}

// Host: launchers.
cudaError_t launch_rms_norm(const kda_rms_norm_args &a, cudaStream_t st);
cudaError_t launch_rms_norm_bwd(const kda_rms_norm_bwd_args &a, cudaStream_t st);
size_t rms_norm_bwd_workspace(int64_t rows, int32_t cols);
cudaError_t launch_fp8_quantize(const kda_fp8_quantize_args &a, cudaStream_t st);
cudaError_t launch_fp8_matmul(const kda_fp8_matmul_args &a, cudaStream_t st);

}  // namespace kda
