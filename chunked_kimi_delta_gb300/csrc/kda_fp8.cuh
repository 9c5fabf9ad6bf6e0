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

// Two fp32 operations in one instruction, each rounded as its scalar form.
__device__ __forceinline__ uint64_t f2_bits(float2 a) { return (uint64_t)__float_as_uint(a.y) << 32 | __float_as_uint(a.x); }
__device__ __forceinline__ float2 f2_of(uint64_t b) {
  return make_float2(__uint_as_float((uint32_t)b), __uint_as_float((uint32_t)(b >> 32)));
}
__device__ __forceinline__ float2 f2_mul(float2 a, float2 b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(f2_bits(a)), "l"(f2_bits(b)));
  return f2_of(d);
}
__device__ __forceinline__ float2 f2_fma(float2 a, float2 b, float2 c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(f2_bits(a)), "l"(f2_bits(b)), "l"(f2_bits(c)));
  return f2_of(d);
}
__device__ __forceinline__ float2 f2_add(float2 a, float2 b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(f2_bits(a)), "l"(f2_bits(b)));
  return f2_of(d);
}
__device__ __forceinline__ float2 f2_splat(float a) { return make_float2(a, a); }

// Four values times `inv` as e4m3 bytes, lowest first.  None is infinite
// (drop_infinities): the conversion would clamp it to 448.
__device__ __forceinline__ uint32_t fp8_pack4(float2 a, float2 b, float2 inv_a, float2 inv_b) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(f2_mul(a, inv_a), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(f2_mul(b, inv_b), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}
__device__ __forceinline__ uint32_t fp8_pack4(float2 a, float2 b, float2 inv) { return fp8_pack4(a, b, inv, inv); }

// Largest magnitude, NaN left out (fmaxf returns the other operand).
__device__ __forceinline__ float block_amax(const float2 (&y)[4]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = fmaxf(m, fmaxf(fabsf(y[i].x), fabsf(y[i].y)));
  return m;
}
// e4m3 has no infinity: they become NaN, and so leave block_amax alone.
__device__ __forceinline__ void drop_infinities(float2 (&y)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = make_float2(fmaf(y[i].x, 0.f, y[i].x), fmaf(y[i].y, 0.f, y[i].y));
}
__device__ __forceinline__ float half_warp_max(float m) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
  return m;
}

// Eight elements as they are stored: bf16 in pairs, or fp32.
template <typename T> struct Raw8;
template <> struct Raw8<float> {
  uint4 v[2];
  __device__ __forceinline__ void get(float2 (&f)[4]) const {
    f[0] = make_float2(__uint_as_float(v[0].x), __uint_as_float(v[0].y));
    f[1] = make_float2(__uint_as_float(v[0].z), __uint_as_float(v[0].w));
    f[2] = make_float2(__uint_as_float(v[1].x), __uint_as_float(v[1].y));
    f[3] = make_float2(__uint_as_float(v[1].z), __uint_as_float(v[1].w));
  }
  __device__ __forceinline__ void put(const float2 (&f)[4]) {
    v[0] = make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x), __float_as_uint(f[1].y));
    v[1] = make_uint4(__float_as_uint(f[2].x), __float_as_uint(f[2].y), __float_as_uint(f[3].x), __float_as_uint(f[3].y));
  }
};
template <> struct Raw8<__nv_bfloat16> {
  uint4 v[1];
  __device__ __forceinline__ void get(float2 (&f)[4]) const {
    const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
    for (int j = 0; j < 4; ++j)  // bf16 is the upper half of an fp32
      f[j] = make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
  }
  __device__ __forceinline__ void put(const float2 (&f)[4]) {  // rounds to nearest even
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(f[j].x, f[j].y);
      w[j] = *reinterpret_cast<const uint32_t *>(&p);
    }
    v[0] = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <typename T> __device__ __forceinline__ Raw8<T> raw_zero() {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < (int)(sizeof(r) / 16); ++i) r.v[i] = make_uint4(0, 0, 0, 0);
  return r;
}
template <typename T> __device__ __forceinline__ Raw8<T> raw_load(const T *p) {  // 16-byte aligned
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < (int)(sizeof(r) / 16); ++i) r.v[i] = reinterpret_cast<const uint4 *>(p)[i];
  return r;
}
template <typename T> __device__ __forceinline__ void raw_store(T *p, const Raw8<T> &r) {
#pragma unroll
  for (int i = 0; i < (int)(sizeof(r) / 16); ++i) reinterpret_cast<uint4 *>(p)[i] = r.v[i];
}
// The same one element at a time, `step` apart, the first n of eight (zeros
// beyond): rows that do not start on 16 bytes.
template <typename T> __device__ __forceinline__ Raw8<T> raw_gather(const T *p, int step, int n) {
  float2 f[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[j].x = 2 * j * step < n ? to_f32<T>(p[2 * j * step]) : 0.f;
    f[j].y = (2 * j + 1) * step < n ? to_f32<T>(p[(2 * j + 1) * step]) : 0.f;
  }
  Raw8<T> r;
  r.put(f);
  return r;
}
template <typename T> __device__ __forceinline__ void raw_scatter(T *p, int step, int n, const Raw8<T> &r) {
  float2 f[4];
  r.get(f);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (2 * j * step < n) p[2 * j * step] = from_f32<T>(f[j].x);
    if ((2 * j + 1) * step < n) p[(2 * j + 1) * step] = from_f32<T>(f[j].y);
  }
}
// a + b, rounded once to T.  The sum of two bf16 that fp32 could not hold
// exactly is nowhere near halfway between two bf16, so one rounding from the
// exact sum and two through fp32 agree.
__device__ __forceinline__ Raw8<float> raw_add(const Raw8<float> &a, const Raw8<float> &b) {
  float2 x[4], y[4];
  a.get(x);
  b.get(y);
#pragma unroll
  for (int j = 0; j < 4; ++j) x[j] = f2_add(x[j], y[j]);
  Raw8<float> r;
  r.put(x);
  return r;
}
__device__ __forceinline__ uint32_t bf2_add(uint32_t a, uint32_t b) {
  const __nv_bfloat162 s = __hadd2(*reinterpret_cast<const __nv_bfloat162 *>(&a), *reinterpret_cast<const __nv_bfloat162 *>(&b));
  return *reinterpret_cast<const uint32_t *>(&s);
}
__device__ __forceinline__ Raw8<__nv_bfloat16> raw_add(const Raw8<__nv_bfloat16> &a, const Raw8<__nv_bfloat16> &b) {
  Raw8<__nv_bfloat16> r;
  r.v[0] = make_uint4(bf2_add(a.v[0].x, b.v[0].x), bf2_add(a.v[0].y, b.v[0].y), bf2_add(a.v[0].z, b.v[0].z),
                      bf2_add(a.v[0].w, b.v[0].w));
  return r;
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

// The kernels of this path follow one another, most of them for tens of
// microseconds: each may be set up while the one before it in the stream
// ends.  grid_start() lets the next one come and then waits for the end of
// the one before (its writes are visible after it); no thread touches global
// memory ahead of it.
__device__ __forceinline__ void grid_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Dynamic shared memory that a kernel of this path may ask for: of a CTA's
// 227 KB, 1 KB is left to its static variables.
constexpr size_t MAX_DYNAMIC_SMEM = 226 * 1024;

// Host: launches a kernel that calls grid_start(), in clusters of `cluster`.
// The limit of a kernel is one value for all host threads: it is always set to
// the same, never to what this call needs, which another thread's call of
// another size could lower between the setting and the launch.
template <typename... P, typename... A>
cudaError_t launch_overlapped(void (*kern)(P...), unsigned grid, unsigned threads, size_t smem, unsigned cluster,
                              cudaStream_t st, A... args) {
  if (smem > 40 * 1024) {  // with the static part, past the 48 KB that need no leave
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)MAX_DYNAMIC_SMEM);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute at[2]{};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

// Host: SMs of the current device (152 on a whole GB300, fewer where a process
// is given a part of one).
inline int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 152;  // no device: the launch will say so
  return sms < 2 ? 2 : sms;
}

// Host: launchers.
cudaError_t launch_rms_norm(const kda_rms_norm_args &a, cudaStream_t st);
cudaError_t launch_rms_norm_bwd(const kda_rms_norm_bwd_args &a, cudaStream_t st);
size_t rms_norm_bwd_workspace(int64_t rows, int32_t cols);
cudaError_t launch_fp8_quantize(const kda_fp8_quantize_args &a, cudaStream_t st);
cudaError_t launch_fp8_matmul(const kda_fp8_matmul_args &a, cudaStream_t st);

}  // namespace kda
