// kda_fp8_quant.cu - quantiser to scaled 8-bit values: one read of the matrix,
// any of the three kinds of scales.
//
//   2^e = the smallest power of two with max |x| <= 448 2^e over the block
//   q = e4m3(x 2^-e), exact up to the one rounding
//
// Every element is read once and written once for each kind; what bounds it is
// instructions (24 an element for rows and columns together as first written,
// 17 now), so maxima are taken on bf16 pairs, products on fp32 pairs, and a
// column's scale is worked out by one thread and not by the sixteen that hold
// its rows.  32768 x 4096 bf16: row 64.5 us, col 61.2 us (97% of the copy
// rate), both at once 90.7 us (87%).
#include "kda_fp8.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;

// Magnitudes' maxima, element by element; NaN left out.
struct Max8f {
  float2 m[4];
  __device__ __forceinline__ void add(const Raw8<float> &v) {
    float2 f[4];
    v.get(f);
#pragma unroll
    for (int j = 0; j < 4; ++j) m[j] = make_float2(fmaxf(m[j].x, fabsf(f[j].x)), fmaxf(m[j].y, fabsf(f[j].y)));
  }
  __device__ __forceinline__ void get(float2 (&f)[4]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = m[j];
  }
};
// bf16 works on pairs: a maximum is one of its operands, so nothing is rounded.
__device__ __forceinline__ __nv_bfloat162 abs2(uint32_t w) {
  w &= 0x7FFF7FFFu;
  return *reinterpret_cast<const __nv_bfloat162 *>(&w);
}
struct Max8h {
  __nv_bfloat162 m[4];
  __device__ __forceinline__ void add(const Raw8<__nv_bfloat16> &v) {
    m[0] = __hmax2(m[0], abs2(v.v[0].x));
    m[1] = __hmax2(m[1], abs2(v.v[0].y));
    m[2] = __hmax2(m[2], abs2(v.v[0].z));
    m[3] = __hmax2(m[3], abs2(v.v[0].w));
  }
  __device__ __forceinline__ void get(float2 (&f)[4]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = __bfloat1622float2(m[j]);
  }
};
template <typename T> struct Max8;
template <> struct Max8<float> { using type = Max8f; };
template <> struct Max8<__nv_bfloat16> { using type = Max8h; };

__device__ __forceinline__ float row_max(const Raw8<float> &v) {
  float2 f[4];
  v.get(f);
  return block_amax(f);
}
__device__ __forceinline__ float row_max(const Raw8<__nv_bfloat16> &v) {
  const float2 f = __bfloat1622float2(__hmax2(__hmax2(abs2(v.v[0].x), abs2(v.v[0].y)), __hmax2(abs2(v.v[0].z), abs2(v.v[0].w))));
  return fmaxf(fmaxf(f.x, f.y), 0.f);  // 0 when both are NaN
}

// How a block comes in: RING (bf16) copies the CTA's next block ahead into
// shared memory (cp.async; each thread its own elements, so no barrier) once
// the last one is in registers, DIRECT loads 16 bytes at a time, ODD (rows not on 16 bytes) one element.
enum Mode { RING, DIRECT, ODD };

// Persistent CTAs over 128 x 128 blocks: thread t holds columns 8 (t % 16) ..
// + 7 of the rows t / 16 + 16 i, i < 8.  A row's maximum is that of 16
// neighbouring lanes; a column's is over i, the two half-warps and the eight
// warps; the block's is that of its columns.  The block stays in registers as
// it was loaded (32 of them for bf16), three CTAs to an SM (four: 108 us for
// rows and columns, against 92).
template <typename T, Mode M>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 && M != ODD ? 3 : 2)
fp8_quantize_kernel(kda_fp8_quantize_args a, int cblocks, int tiles) {
  extern __shared__ uint4 smem_raw[];
  Raw8<T> *ring = reinterpret_cast<Raw8<T> *>(smem_raw) + threadIdx.x;  // RING: [8][kThreads]
  __shared__ float colmax[8][FP8_BLOCK];
  __shared__ __align__(16) float colinv[FP8_BLOCK];
  __shared__ float warpmax[2][4];
  const int lane16 = threadIdx.x & 15, warp = threadIdx.x >> 5;
  const int64_t row_step = (int64_t)16 * a.cols;
  auto fetch = [&](int tile) {
    if (M != RING) return;
    if (tile < tiles) {
      const int c = (tile % cblocks) * FP8_BLOCK + 8 * lane16;
      const int64_t r0 = (int64_t)(tile / cblocks) * FP8_BLOCK + threadIdx.x / 16;
      const T *x = static_cast<const T *>(a.x) + r0 * a.cols + c;
      const uint32_t dst = (uint32_t)__cvta_generic_to_shared(ring);
      const int rows = c < a.cols ? (int)min(a.rows - r0, (int64_t)FP8_BLOCK) : 0;  // from r0 on
#pragma unroll
      for (int i = 0; i < 8; ++i, x += row_step) {  // zeros outside
        const bool in = 16 * i < rows;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                     :: "r"(dst + i * kThreads * 16), "l"(in ? (const void *)x : a.x), "r"(in ? 16 : 0) : "memory");
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  grid_start();
  fetch(blockIdx.x);
  int buf = 0;
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x, buf ^= 1) {
    const int rb = tile / cblocks, cb = tile % cblocks;
    const int c = cb * FP8_BLOCK + 8 * lane16;  // first column of this thread
    const int n = a.cols - c;                   // columns it holds, at most 8
    const int64_t r0 = (int64_t)rb * FP8_BLOCK + threadIdx.x / 16;
    const int rows = (int)min(a.rows - r0, (int64_t)FP8_BLOCK);  // from r0 on
    Raw8<T> v[8];
    if (M == RING) {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = ring[i * kThreads];
    } else {
      const T *x = static_cast<const T *>(a.x) + r0 * a.cols + c;
#pragma unroll
      for (int i = 0; i < 8; ++i, x += row_step) {
        if (M == ODD) v[i] = raw_gather<T>(x, 1, 16 * i < rows ? n : 0);
        else v[i] = 16 * i < rows && n > 0 ? raw_load<T>(x) : raw_zero<T>();
      }
    }
    typename Max8<T>::type max8 = {};
#pragma unroll
    for (int i = 0; i < 8; ++i) max8.add(v[i]);
    float2 cm[4];
    max8.get(cm);
    if (isinf(block_amax(cm))) {  // infinities count as NaN
      max8 = {};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float2 f[4];
        v[i].get(f);
        drop_infinities(f);
        v[i].put(f);
        max8.add(v[i]);
      }
      max8.get(cm);
    }
    // the test above needed every value: this thread's slots are free
    fetch(tile + (int)gridDim.x);
    if (a.row) {
      uint8_t *q = static_cast<uint8_t *>(a.row) + r0 * a.ld + c;
      uint8_t *s = a.row_scales + ((int64_t)(cb >> 2) * a.rows + r0) * 4 + (cb & 3);
#pragma unroll
      for (int i = 0; i < 8; ++i, q += 16 * a.ld) {
        const uint32_t sb = fp8_scale_byte(half_warp_max(row_max(v[i])));
        if (16 * i >= rows) continue;
        const float2 inv = f2_splat(fp8_inv_scale(sb));
        float2 f[4];
        v[i].get(f);
        store8_fp8(q, n, fp8_pack4(f[0], f[1], inv), fp8_pack4(f[2], f[3], inv));
        if (lane16 == 0) {
          s[64 * i] = (uint8_t)sb;
          if (cb == cblocks - 1)
            for (int p = (cb & 3) + 1; p < 4; ++p) s[64 * i + p - (cb & 3)] = (uint8_t)FP8_SCALE_ONE;
        }
      }
    }
    if (a.col || a.tile) {
      float *cf = reinterpret_cast<float *>(cm);
#pragma unroll
      for (int j = 0; j < 8; ++j) cf[j] = fmaxf(fmaxf(cf[j], __shfl_xor_sync(~0u, cf[j], 16)), 0.f);
      if ((threadIdx.x & 16) == 0) {
        float4 *d = reinterpret_cast<float4 *>(&colmax[warp][8 * lane16]);
        d[0] = make_float4(cf[0], cf[1], cf[2], cf[3]);
        d[1] = make_float4(cf[4], cf[5], cf[6], cf[7]);
      }
      __syncthreads();
      // a column's scale, by one thread of the first four warps
      if (threadIdx.x < FP8_BLOCK) {
        float m = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) m = fmaxf(m, colmax[w][threadIdx.x]);
        if (a.col) {
          const uint32_t sb = fp8_scale_byte(m);
          colinv[threadIdx.x] = fp8_inv_scale(sb);
          const int col = cb * FP8_BLOCK + threadIdx.x;
          if (col < a.cols) {
            uint8_t *s = a.col_scales + ((int64_t)(rb >> 2) * a.cols + col) * 4;
            s[rb & 3] = (uint8_t)sb;
            if ((int64_t)(rb + 1) * FP8_BLOCK >= a.rows)
              for (int p = (rb & 3) + 1; p < 4; ++p) s[p] = (uint8_t)FP8_SCALE_ONE;
          }
        }
        if (a.tile) {
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
          if ((threadIdx.x & 31) == 0) warpmax[buf][warp] = m;
        }
      }
      __syncthreads();
    }
    if (a.col) {
      float2 inv[4];
      const float4 lo = *reinterpret_cast<const float4 *>(&colinv[8 * lane16]);
      const float4 hi = *reinterpret_cast<const float4 *>(&colinv[8 * lane16 + 4]);
      inv[0] = make_float2(lo.x, lo.y);
      inv[1] = make_float2(lo.z, lo.w);
      inv[2] = make_float2(hi.x, hi.y);
      inv[3] = make_float2(hi.z, hi.w);
      uint8_t *q = static_cast<uint8_t *>(a.col) + r0 * a.ld + c;
#pragma unroll
      for (int i = 0; i < 8; ++i, q += 16 * a.ld) {
        if (16 * i >= rows) continue;
        float2 f[4];
        v[i].get(f);
        store8_fp8(q, n, fp8_pack4(f[0], f[1], inv[0], inv[1]), fp8_pack4(f[2], f[3], inv[2], inv[3]));
      }
    }
    if (a.tile) {
      const float m = fmaxf(fmaxf(warpmax[buf][0], warpmax[buf][1]), fmaxf(warpmax[buf][2], warpmax[buf][3]));
      const uint32_t sb = fp8_scale_byte(m);
      const float2 inv = f2_splat(fp8_inv_scale(sb));
      uint8_t *q = static_cast<uint8_t *>(a.tile) + r0 * a.ld + c;
#pragma unroll
      for (int i = 0; i < 8; ++i, q += 16 * a.ld) {
        if (16 * i >= rows) continue;
        float2 f[4];
        v[i].get(f);
        store8_fp8(q, n, fp8_pack4(f[0], f[1], inv), fp8_pack4(f[2], f[3], inv));
      }
      if (threadIdx.x == 0) a.tile_scales[(int64_t)rb * cblocks + cb] = (uint8_t)sb;
    }
  }
}

template <typename T, Mode M> cudaError_t launch(const kda_fp8_quantize_args &a, int cblocks, int tiles, cudaStream_t st) {
  // three CTAs in turn on each place: SMs are not equally fast (one: 92.1 us, three: 90.7, one per block: 101)
  const int most = 3 * sm_count() * (sizeof(T) == 2 && M != ODD ? 3 : 2);
  return launch_overlapped(fp8_quantize_kernel<T, M>, (unsigned)(tiles < most ? tiles : most), kThreads,
                           M == RING ? 8 * kThreads * 16 : 0, 1, st, a, cblocks, tiles);
}

}  // namespace

cudaError_t launch_fp8_quantize(const kda_fp8_quantize_args &a, cudaStream_t st) {
  const int cblocks = (int)(((int64_t)a.cols + FP8_BLOCK - 1) / FP8_BLOCK);
  const int tiles = (int)((a.rows + FP8_BLOCK - 1) / FP8_BLOCK * cblocks);
  const bool vec = a.cols % 8 == 0;
  if (a.dtype == KDA_F32) return vec ? launch<float, DIRECT>(a, cblocks, tiles, st) : launch<float, ODD>(a, cblocks, tiles, st);
  return vec ? launch<__nv_bfloat16, RING>(a, cblocks, tiles, st) : launch<__nv_bfloat16, ODD>(a, cblocks, tiles, st);
}

}  // namespace kda
