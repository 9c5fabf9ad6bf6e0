// kda_norm.cu - RMS norm with the residual's addition and an 8-bit result, and
// its backward.
#include "kda_fp8.cuh"

namespace kda {
namespace {

// Sum over the CTA's threads, the same value in all of them: shuffles inside
// a warp, then the warps' sums in order.  `red`: one float per warp.
__device__ __forceinline__ float cta_sum(float v, float *red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  const int warps = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
  for (int i = 0; i < warps; ++i) s += red[i];
  __syncthreads();
  return s;
}

// Largest finite magnitude of the 128 columns that 16 neighbouring lanes hold.
__device__ __forceinline__ float half_warp_amax(const float (&y)[8]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, finite_abs(y[i]));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
  return m;
}

// One CTA per row; the row stays in registers between the sum of squares and
// the result: thread t holds columns 8 (t + i blockDim) .. + 7 for i < VPT, so
// 16 neighbouring lanes hold the 128 columns of one scale.
template <typename T, bool VEC, int VPT>
__global__ void __launch_bounds__(VPT == 1 ? 512 : 1024) rms_norm_kernel(kda_rms_norm_args a) {
  __shared__ float red[32];
  const int64_t row = blockIdx.x;
  const int cols = a.cols;
  const T *x = static_cast<const T *>(a.x) + row * cols;
  const T *res = a.residual ? static_cast<const T *>(a.residual) + row * cols : nullptr;
  float h[VPT][8];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = 8 * (threadIdx.x + i * blockDim.x);
    load8<T, VEC>(x + c, cols - c, h[i]);
    if (res) {
      float r[8];
      load8<T, VEC>(res + c, cols - c, r);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] = to_f32<T>(from_f32<T>(h[i][j] + r[j]));
      store8<T, VEC>(static_cast<T *>(a.residual_out) + row * cols + c, cols - c, h[i]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(h[i][j], h[i][j], ss);
  }
  const float rstd = 1.f / sqrtf(cta_sum(ss, red) / (float)cols + a.eps);
  const int cb = (cols + FP8_BLOCK - 1) / FP8_BLOCK;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = 8 * (threadIdx.x + i * blockDim.x);
    float w[8], y[8];
    if (a.weight) {
      load8<float, VEC>(a.weight + c, cols - c, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = h[i][j] * rstd * w[j];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = h[i][j] * rstd;
    }
    if (a.out) store8<T, VEC>(static_cast<T *>(a.out) + row * cols + c, cols - c, y);
    if (a.fp8) {
      const uint32_t sb = fp8_scale_byte(half_warp_amax(y));
      const float inv = fp8_inv_scale(sb);
      store8_fp8(static_cast<uint8_t *>(a.fp8) + row * a.ld_fp8 + c, cols - c,
                 fp8_pack4(y[0], y[1], y[2], y[3], inv), fp8_pack4(y[4], y[5], y[6], y[7], inv));
      const int b = c / FP8_BLOCK;
      if ((threadIdx.x & 15) == 0 && b < ((cb + 3) & ~3))
        a.fp8_scales[((b >> 2) * a.rows + row) * 4 + (b & 3)] = (uint8_t)sb;  // 1.0 past the last block
    }
  }
}

template <typename T, bool VEC>
cudaError_t norm_typed(const kda_rms_norm_args &a, cudaStream_t st) {
  // whole groups of four blocks, so that the scales past the last block get written
  const int vecs = (a.cols + 511) / 512 * 64;
  const int vpt = vecs <= 512 ? 1 : vecs <= 2048 ? 2 : 4;
  const int threads = (vecs / vpt + 31) / 32 * 32;
  const dim3 grid((unsigned)a.rows);
  if (vpt == 1) rms_norm_kernel<T, VEC, 1><<<grid, threads, 0, st>>>(a);
  else if (vpt == 2) rms_norm_kernel<T, VEC, 2><<<grid, threads, 0, st>>>(a);
  else rms_norm_kernel<T, VEC, 4><<<grid, threads, 0, st>>>(a);
  return cudaGetLastError();
}

// ------------------------------------------------------------------ backward

constexpr int kBwdParts = 608;  // partial dweight rows: 4 CTAs on each of 152 SMs

// CTAs walk the rows with a stride of the grid; dweight of a CTA's rows is
// summed in its registers and left as one row of partial sums.
template <typename T, bool VEC, int VPT>
__global__ void __launch_bounds__(VPT == 1 ? 512 : 1024) rms_norm_bwd_kernel(kda_rms_norm_bwd_args a) {
  __shared__ float red[32];
  const int cols = a.cols;
  float dw[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.f;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    float h[VPT][8], g[VPT][8];
    float ss = 0.f, sg = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = 8 * (threadIdx.x + i * blockDim.x);
      load8<T, VEC>(static_cast<const T *>(a.h) + row * cols + c, cols - c, h[i]);
      load8<T, VEC>(static_cast<const T *>(a.d_out) + row * cols + c, cols - c, g[i]);
      float w[8];
      if (a.weight) load8<float, VEC>(a.weight + c, cols - c, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        ss = fmaf(h[i][j], h[i][j], ss);
        sg = fmaf(a.weight ? g[i][j] * w[j] : g[i][j], h[i][j], sg);
      }
    }
    ss = cta_sum(ss, red);
    sg = cta_sum(sg, red);
    const float rstd = 1.f / sqrtf(ss / (float)cols + a.eps);
    const float mean = sg * rstd / (float)cols;  // mean of weight * d_out * n
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = 8 * (threadIdx.x + i * blockDim.x);
      float w[8], r[8], dx[8];
      if (a.weight) load8<float, VEC>(a.weight + c, cols - c, w);
      if (a.d_residual) load8<T, VEC>(static_cast<const T *>(a.d_residual) + row * cols + c, cols - c, r);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float n = h[i][j] * rstd;
        dw[i][j] = fmaf(g[i][j], n, dw[i][j]);
        dx[j] = rstd * ((a.weight ? g[i][j] * w[j] : g[i][j]) - n * mean);
        if (a.d_residual) dx[j] += r[j];
      }
      store8<T, VEC>(static_cast<T *>(a.dx) + row * cols + c, cols - c, dx);
    }
  }
  if (a.dweight) {
    float *part = static_cast<float *>(a.workspace) + (int64_t)blockIdx.x * cols;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = 8 * (threadIdx.x + i * blockDim.x);
      store8<float, VEC>(part + c, cols - c, dw[i]);
    }
  }
}

// dweight[c] = the sum of the partial rows: 32 columns x 8 row lanes per CTA,
// each lane in row order, then the lanes in order.
__global__ void __launch_bounds__(256) dweight_kernel(const float *__restrict__ part, int parts, int cols,
                                                      float *__restrict__ dw) {
  __shared__ float s[8][33];
  const int lane = threadIdx.x & 31, r = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (c < cols)
    for (int p = r; p < parts; p += 8) v += part[(int64_t)p * cols + c];
  s[r][lane] = v;
  __syncthreads();
  if (r == 0 && c < cols) {
#pragma unroll
    for (int i = 1; i < 8; ++i) v += s[i][lane];
    dw[c] = v;
  }
}

template <typename T, bool VEC>
cudaError_t bwd_typed(const kda_rms_norm_bwd_args &a, cudaStream_t st) {
  const int vecs = (a.cols + 7) / 8;
  const int vpt = vecs <= 512 ? 1 : vecs <= 2048 ? 2 : 4;
  const int threads = ((vecs + vpt - 1) / vpt + 31) / 32 * 32;
  const int parts = (int)(a.rows < kBwdParts ? a.rows : kBwdParts);
  if (vpt == 1) rms_norm_bwd_kernel<T, VEC, 1><<<parts, threads, 0, st>>>(a);
  else if (vpt == 2) rms_norm_bwd_kernel<T, VEC, 2><<<parts, threads, 0, st>>>(a);
  else rms_norm_bwd_kernel<T, VEC, 4><<<parts, threads, 0, st>>>(a);
  if (a.dweight)
    dweight_kernel<<<(a.cols + 31) / 32, 256, 0, st>>>(static_cast<const float *>(a.workspace), parts, a.cols,
                                                       a.dweight);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rms_norm(const kda_rms_norm_args &a, cudaStream_t st) {
  const bool vec = a.cols % 8 == 0;  // rows then start on 16-byte boundaries
  if (a.dtype == KDA_F32) return vec ? norm_typed<float, true>(a, st) : norm_typed<float, false>(a, st);
  return vec ? norm_typed<__nv_bfloat16, true>(a, st) : norm_typed<__nv_bfloat16, false>(a, st);
}

size_t rms_norm_bwd_workspace(int64_t rows, int32_t cols) {
  return align256(sizeof(float) * (size_t)(rows < kBwdParts ? rows : kBwdParts) * (size_t)cols);
}

cudaError_t launch_rms_norm_bwd(const kda_rms_norm_bwd_args &a, cudaStream_t st) {
  const bool vec = a.cols % 8 == 0;
  if (a.dtype == KDA_F32) return vec ? bwd_typed<float, true>(a, st) : bwd_typed<float, false>(a, st);
  return vec ? bwd_typed<__nv_bfloat16, true>(a, st) : bwd_typed<__nv_bfloat16, false>(a, st);
}

}  // namespace kda
