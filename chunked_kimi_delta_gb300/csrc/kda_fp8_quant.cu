// kda_fp8_quant.cu - quantiser to scaled 8-bit values: one read of the matrix,
// any of the three kinds of scales.
#include "kda_fp8.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;

// Eight elements as loaded: fp32, or bf16 pairs (four registers).
template <typename T> struct Vec8;
template <> struct Vec8<float> {
  float f[8];
  __device__ __forceinline__ void get(float (&o)[8]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = f[j];
  }
  __device__ __forceinline__ void set(const float (&o)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = o[j];
  }
  __device__ __forceinline__ void raw(const uint4 *p) {
    const uint4 a = p[0], b = p[1];
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(w[j]);
  }
};
template <> struct Vec8<__nv_bfloat16> {
  uint32_t w[4];
  __device__ __forceinline__ void get(float (&o)[8]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      o[2 * j] = __uint_as_float(w[j] << 16);
      o[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  }
  __device__ __forceinline__ void set(const float (&o)[8]) {  // exact: the values are bf16 (or NaN)
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = __float_as_uint(o[2 * j]) >> 16 | (__float_as_uint(o[2 * j + 1]) & 0xFFFF0000u);
  }
  __device__ __forceinline__ void raw(const uint4 *p) {
    const uint4 a = *p;
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
  }
};

// The magnitudes' maxima: of one vector, and column by column.  bf16 works on
// pairs: a maximum is one of its operands, so nothing is rounded.
__device__ __forceinline__ float row_amax(const Vec8<float> &v) { return block_amax(v.f); }
__device__ __forceinline__ float row_amax(const Vec8<__nv_bfloat16> &v) {
  const __nv_bfloat162 *p = reinterpret_cast<const __nv_bfloat162 *>(v.w);
  const __nv_bfloat162 m = __hmax2(__hmax2(__habs2(p[0]), __habs2(p[1])), __hmax2(__habs2(p[2]), __habs2(p[3])));
  const float2 f = __bfloat1622float2(m);
  return fmaxf(fmaxf(f.x, f.y), 0.f);  // 0 when both are NaN
}
__device__ __forceinline__ void col_amax(Vec8<float> &m, const Vec8<float> &v) {
#pragma unroll
  for (int j = 0; j < 8; ++j) m.f[j] = fmaxf(m.f[j], fabsf(v.f[j]));
}
__device__ __forceinline__ void col_amax(Vec8<__nv_bfloat16> &m, const Vec8<__nv_bfloat16> &v) {
  __nv_bfloat162 *a = reinterpret_cast<__nv_bfloat162 *>(m.w);
  const __nv_bfloat162 *b = reinterpret_cast<const __nv_bfloat162 *>(v.w);
#pragma unroll
  for (int j = 0; j < 4; ++j) a[j] = __hmax2(a[j], __habs2(b[j]));
}

// How a block comes in: RING (bf16) copies the CTA's next block ahead into
// shared memory (cp.async; each thread its own elements, so no barrier),
// DIRECT loads 16 bytes at a time, ODD (rows not on 16 bytes) one element.
enum Mode { RING, DIRECT, ODD };

// Persistent CTAs over 128 x 128 blocks: thread t holds columns 8 (t % 16) ..
// + 7 of the rows t / 16 + 16 i, i < 8.  A row's maximum is that of 16
// neighbouring lanes; a column's is over i, the two half-warps and the eight
// warps; the block's is that of its columns.  Memory bounds it: every element
// is read once and written once for each kind.  The block stays in registers
// as it was loaded (32 of them for bf16), three CTAs to an SM.
template <typename T, Mode M>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 && M != ODD ? 3 : 2) fp8_quantize_kernel(kda_fp8_quantize_args a, int cblocks,
                                                                                       int tiles) {
  extern __shared__ uint4 ring[];  // RING: [2][8][kThreads]
  __shared__ float colmax[2][8][FP8_BLOCK];
  __shared__ float warpmax[2][8];
  const int lane16 = threadIdx.x & 15, warp = threadIdx.x >> 5;
  auto fetch = [&](int tile, int buf) {
    if (M != RING) return;
    if (tile < tiles) {
      const int c = (tile % cblocks) * FP8_BLOCK + 8 * lane16;
      const int64_t r0 = (int64_t)(tile / cblocks) * FP8_BLOCK + threadIdx.x / 16;
      const T *x = static_cast<const T *>(a.x) + r0 * a.cols + c;
      const uint32_t dst = (uint32_t)__cvta_generic_to_shared(ring + buf * 8 * kThreads + threadIdx.x);
#pragma unroll
      for (int i = 0; i < 8; ++i) {  // zeros outside
        const bool in = c < a.cols && r0 + 16 * i < a.rows;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                     :: "r"(dst + i * kThreads * 16), "l"(in ? (const void *)(x + (int64_t)(16 * i) * a.cols) : a.x), "r"(in ? 16 : 0)
                     : "memory");
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  fetch(blockIdx.x, 0);
  fetch(blockIdx.x + gridDim.x, 1);
  int par = 0;
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x, par ^= 1) {
    const int rb = tile / cblocks, cb = tile % cblocks;
    const int c = cb * FP8_BLOCK + 8 * lane16;      // first column of this thread
    const int n = a.cols - c;                       // columns it holds, at most 8
    const int64_t r0 = (int64_t)rb * FP8_BLOCK + threadIdx.x / 16;
    Vec8<T> v[8];
    if (M == RING) {
      asm volatile("cp.async.wait_group 1;" ::: "memory");
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i].raw(ring + (par * 8 + i) * kThreads + threadIdx.x);
    } else {
      const T *x = static_cast<const T *>(a.x) + r0 * a.cols + c;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float f[8];
        load8<T, M == DIRECT>(x + (int64_t)(16 * i) * a.cols, r0 + 16 * i < a.rows ? n : 0, f);
        v[i].set(f);
      }
    }
    Vec8<T> cmax = {};
#pragma unroll
    for (int i = 0; i < 8; ++i) col_amax(cmax, v[i]);
    float cm[8];
    cmax.get(cm);
    bool inf = false;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      cm[j] = fmaxf(cm[j], 0.f);
      inf |= isinf(cm[j]);
    }
    if (inf) {  // infinities count as NaN
      cmax = {};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float f[8];
        v[i].get(f);
        drop_infinities(f);
        v[i].set(f);
        col_amax(cmax, v[i]);
      }
      cmax.get(cm);
#pragma unroll
      for (int j = 0; j < 8; ++j) cm[j] = fmaxf(cm[j], 0.f);
    }
    if (a.row) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float m = row_amax(v[i]);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
        const uint32_t sb = fp8_scale_byte(m);
        const float inv = fp8_inv_scale(sb);
        const int64_t r = r0 + 16 * i;
        if (r >= a.rows) continue;
        float f[8];
        v[i].get(f);
        store8_fp8(static_cast<uint8_t *>(a.row) + r * a.ld + c, n, fp8_pack4(f[0], f[1], f[2], f[3], inv),
                   fp8_pack4(f[4], f[5], f[6], f[7], inv));
        if (lane16 == 0) {
          uint8_t *s = a.row_scales + ((int64_t)(cb >> 2) * a.rows + r) * 4;
          s[cb & 3] = (uint8_t)sb;
          if (cb == cblocks - 1)
            for (int p = (cb & 3) + 1; p < 4; ++p) s[p] = (uint8_t)FP8_SCALE_ONE;
        }
      }
    }
    if (a.col || a.tile) {
#pragma unroll
      for (int j = 0; j < 8; ++j) cm[j] = fmaxf(cm[j], __shfl_xor_sync(~0u, cm[j], 16));
      if ((threadIdx.x & 16) == 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) colmax[par][warp][8 * lane16 + j] = cm[j];
      }
      if (a.tile) {
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = fmaxf(m, cm[j]);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
        if ((threadIdx.x & 31) == 0) warpmax[par][warp] = m;
      }
      __syncthreads();  // the maxima alternate between two buffers, so one barrier a block is enough
    }
    // the maxima needed every value: this thread's slots are free
    fetch(tile + 2 * (int)gridDim.x, par);
    if (a.col) {
      float inv[8];
      uint32_t sb[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float m = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) m = fmaxf(m, colmax[par][w][8 * lane16 + j]);
        sb[j] = fp8_scale_byte(m);
        inv[j] = fp8_inv_scale(sb[j]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t r = r0 + 16 * i;
        if (r >= a.rows) continue;
        float s[8];
        v[i].get(s);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] *= inv[j];
        store8_fp8(static_cast<uint8_t *>(a.col) + r * a.ld + c, n, fp8_pack4(s[0], s[1], s[2], s[3], 1.f),
                   fp8_pack4(s[4], s[5], s[6], s[7], 1.f));
      }
      if (threadIdx.x < 16) {
        const int rblocks = (int)((a.rows + FP8_BLOCK - 1) / FP8_BLOCK);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < n) {
            uint8_t *s = a.col_scales + ((int64_t)(rb >> 2) * a.cols + c + j) * 4;
            s[rb & 3] = (uint8_t)sb[j];
            if (rb == rblocks - 1)
              for (int p = (rb & 3) + 1; p < 4; ++p) s[p] = (uint8_t)FP8_SCALE_ONE;
          }
      }
    }
    if (a.tile) {
      float m = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) m = fmaxf(m, warpmax[par][w]);
      const uint32_t sb = fp8_scale_byte(m);
      const float inv = fp8_inv_scale(sb);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t r = r0 + 16 * i;
        if (r >= a.rows) continue;
        float f[8];
        v[i].get(f);
        store8_fp8(static_cast<uint8_t *>(a.tile) + r * a.ld + c, n, fp8_pack4(f[0], f[1], f[2], f[3], inv),
                   fp8_pack4(f[4], f[5], f[6], f[7], inv));
      }
      if (threadIdx.x == 0) a.tile_scales[(int64_t)rb * cblocks + cb] = (uint8_t)sb;
    }
  }
}

template <typename T, Mode M> cudaError_t launch(const kda_fp8_quantize_args &a, int cblocks, int tiles, cudaStream_t st) {
  auto kern = fp8_quantize_kernel<T, M>;
  const int smem = M == RING ? 2 * 8 * kThreads * 16 : 0, most = 152 * (sizeof(T) == 2 && M != ODD ? 3 : 2);
  if (M == RING) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  kern<<<tiles < most ? tiles : most, kThreads, smem, st>>>(a, cblocks, tiles);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_fp8_quantize(const kda_fp8_quantize_args &a, cudaStream_t st) {
  const int cblocks = (a.cols + FP8_BLOCK - 1) / FP8_BLOCK;
  const int tiles = (int)((a.rows + FP8_BLOCK - 1) / FP8_BLOCK * cblocks);
  const bool vec = a.cols % 8 == 0;
  if (a.dtype == KDA_F32) return vec ? launch<float, DIRECT>(a, cblocks, tiles, st) : launch<float, ODD>(a, cblocks, tiles, st);
  return vec ? launch<__nv_bfloat16, RING>(a, cblocks, tiles, st) : launch<__nv_bfloat16, ODD>(a, cblocks, tiles, st);
}

}  // namespace kda
