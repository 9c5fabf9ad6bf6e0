// kda_fp8_quant.cu - quantiser to scaled 8-bit values: one read of the matrix,
// any of the three kinds of scales.
#include "kda_fp8.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;

// One CTA per 128 x 128 block: thread t holds columns 8 (t % 16) .. + 7 of
// the rows t / 16 + 16 i, i < 8.  A row's maximum is that of 16 neighbouring
// lanes; a column's is over i, the two half-warps and the eight warps; the
// block's is that of its columns.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) fp8_quantize_kernel(kda_fp8_quantize_args a, int cblocks) {
  __shared__ float colmax[8][FP8_BLOCK];
  __shared__ float warpmax[8];
  const int rb = blockIdx.x / cblocks, cb = blockIdx.x % cblocks;
  const int lane16 = threadIdx.x & 15, warp = threadIdx.x >> 5;
  const int c = cb * FP8_BLOCK + 8 * lane16;      // first column of this thread
  const int n = a.cols - c;                       // columns it holds, at most 8
  const int64_t r0 = (int64_t)rb * FP8_BLOCK + threadIdx.x / 16;
  float v[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + 16 * i;
    load8<T, VEC>(static_cast<const T *>(a.x) + r * a.cols + c, r < a.rows ? n : 0, v[i]);
  }
  if (a.row) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float m = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = fmaxf(m, finite_abs(v[i][j]));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
      const uint32_t sb = fp8_scale_byte(m);
      const float inv = fp8_inv_scale(sb);
      const int64_t r = r0 + 16 * i;
      if (r >= a.rows) continue;
      store8_fp8(static_cast<uint8_t *>(a.row) + r * a.ld + c, n, fp8_pack4(v[i][0], v[i][1], v[i][2], v[i][3], inv),
                 fp8_pack4(v[i][4], v[i][5], v[i][6], v[i][7], inv));
      if (lane16 == 0) {
        uint8_t *s = a.row_scales + ((int64_t)(cb >> 2) * a.rows + r) * 4;
        s[cb & 3] = (uint8_t)sb;
        if (cb == cblocks - 1)
          for (int p = (cb & 3) + 1; p < 4; ++p) s[p] = (uint8_t)FP8_SCALE_ONE;
      }
    }
  }
  if (!a.col && !a.tile) return;
  float cm[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, finite_abs(v[i][j]));
    cm[j] = fmaxf(m, __shfl_xor_sync(~0u, m, 16));
  }
  if ((threadIdx.x & 16) == 0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) colmax[warp][8 * lane16 + j] = cm[j];
  }
  __syncthreads();
  if (a.col) {
    float inv[8];
    uint32_t sb[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float m = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) m = fmaxf(m, colmax[w][8 * lane16 + j]);
      sb[j] = fp8_scale_byte(m);
      inv[j] = fp8_inv_scale(sb[j]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t r = r0 + 16 * i;
      if (r >= a.rows) continue;
      float s[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] = v[i][j] * inv[j];
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
    for (int j = 0; j < 8; ++j) m = fmaxf(m, cm[j]);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
    if ((threadIdx.x & 31) == 0) warpmax[warp] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) m = fmaxf(m, warpmax[w]);
    const uint32_t sb = fp8_scale_byte(m);
    const float inv = fp8_inv_scale(sb);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t r = r0 + 16 * i;
      if (r >= a.rows) continue;
      store8_fp8(static_cast<uint8_t *>(a.tile) + r * a.ld + c, n, fp8_pack4(v[i][0], v[i][1], v[i][2], v[i][3], inv),
                 fp8_pack4(v[i][4], v[i][5], v[i][6], v[i][7], inv));
    }
    if (threadIdx.x == 0) a.tile_scales[(int64_t)rb * cblocks + cb] = (uint8_t)sb;
  }
}

}  // namespace

cudaError_t launch_fp8_quantize(const kda_fp8_quantize_args &a, cudaStream_t st) {
  const int cblocks = (a.cols + FP8_BLOCK - 1) / FP8_BLOCK;
  const int64_t rblocks = (a.rows + FP8_BLOCK - 1) / FP8_BLOCK;
  const unsigned grid = (unsigned)(rblocks * cblocks);
  const bool vec = a.cols % 8 == 0;
  if (a.dtype == KDA_F32) {
    if (vec) fp8_quantize_kernel<float, true><<<grid, kThreads, 0, st>>>(a, cblocks);
    else fp8_quantize_kernel<float, false><<<grid, kThreads, 0, st>>>(a, cblocks);
  } else {
    if (vec) fp8_quantize_kernel<__nv_bfloat16, true><<<grid, kThreads, 0, st>>>(a, cblocks);
    else fp8_quantize_kernel<__nv_bfloat16, false><<<grid, kThreads, 0, st>>>(a, cblocks);
  }
  return cudaGetLastError();
}

}  // namespace kda
