// kda_fp8_matmul.cu - matrix product of scaled 8-bit matrices.
#include "kda_fp8.cuh"

namespace kda {
namespace {

// An operand seen as [rows of the output side, k]: element (i, k) at
// p[i * si + k * sk], its scale byte's place by the kind of scales.
struct Operand {
  const uint8_t *p, *s;
  int64_t si, sk;
  int rows;
  // TILE: byte (i / 128) * ti + (k / 128) * tk; ROW and COL: ti = 0, word layout
  int64_t ti, tk;
};

__device__ __forceinline__ float scale_of(const Operand &o, int i, int kb) {
  const uint32_t b = o.ti ? o.s[(i / FP8_BLOCK) * o.ti + kb * o.tk] : o.s[((int64_t)(kb >> 2) * o.rows + i) * 4 + (kb & 3)];
  return b ? __uint_as_float(b == 255 ? 0x7FFFFFFFu : b << 23) : __uint_as_float(0x00400000u);
}
__device__ __forceinline__ float e4m3(uint8_t b) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(b, __NV_E4M3);
  return __half2float(__half(h));
}

// 64 x 64 outputs per CTA, 4 x 4 per thread, 16 of k at a time; the sum of
// each block of 128 is scaled when the block ends.
template <typename T>
__global__ void __launch_bounds__(256) fp8_matmul_kernel(Operand A, Operand B, int m, int n, int k, T *out,
                                                         int64_t ldo) {
  __shared__ float sa[16][65], sb[16][65];
  const int tiles_n = (n + 63) / 64;
  const int i0 = (int)(blockIdx.x / tiles_n) * 64, j0 = (int)(blockIdx.x % tiles_n) * 64;
  const int ti = threadIdx.x / 16, tj = threadIdx.x % 16;
  float acc[4][4] = {}, part[4][4] = {};
  for (int k0 = 0; k0 < k; k0 += 16) {
    for (int e = threadIdx.x; e < 64 * 16; e += 256) {
      // neighbouring threads along the operand's contiguous dimension
      const int ia = A.sk == 1 ? e / 16 : e % 64, ka = A.sk == 1 ? e % 16 : e / 64;
      sa[ka][ia] = i0 + ia < m && k0 + ka < k ? e4m3(A.p[(i0 + ia) * A.si + (k0 + ka) * A.sk]) : 0.f;
      const int ib = B.sk == 1 ? e / 16 : e % 64, kb = B.sk == 1 ? e % 16 : e / 64;
      sb[kb][ib] = j0 + ib < n && k0 + kb < k ? e4m3(B.p[(j0 + ib) * B.si + (k0 + kb) * B.sk]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < 16; ++x)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) part[i][j] = fmaf(sa[x][ti + 16 * i], sb[x][tj + 16 * j], part[i][j]);
    __syncthreads();
    if (k0 + 16 >= k || (k0 + 16) % FP8_BLOCK == 0) {
      const int kb = k0 / FP8_BLOCK;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = i0 + ti + 16 * i;
        const float s = r < m ? scale_of(A, r, kb) : 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = j0 + tj + 16 * j;
          if (c < n) acc[i][j] = fmaf(part[i][j] * s, scale_of(B, c, kb), acc[i][j]);
          part[i][j] = 0.f;
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = i0 + ti + 16 * i, c = j0 + tj + 16 * j;
      if (r < m && c < n) out[r * ldo + c] = from_f32<T>(acc[i][j]);
    }
}

}  // namespace

cudaError_t launch_fp8_matmul(const kda_fp8_matmul_args &a, cudaStream_t st) {
  const bool tn = a.form == KDA_FP8_TN, nt = a.form == KDA_FP8_NT;
  const int64_t nb = (a.n + FP8_BLOCK - 1) / FP8_BLOCK, kb = (a.k + FP8_BLOCK - 1) / FP8_BLOCK;
  Operand A{static_cast<const uint8_t *>(a.a), a.a_scales, tn ? 1 : a.lda, tn ? a.lda : 1, a.m, 0, 0};
  Operand B{static_cast<const uint8_t *>(a.b), a.b_scales, nt ? a.ldb : 1, nt ? 1 : a.ldb, a.n, 0, 0};
  if (nt) { B.ti = kb; B.tk = 1; }
  else if (!tn) { B.ti = 1; B.tk = nb; }
  const unsigned grid = (unsigned)((int64_t)((a.m + 63) / 64) * ((a.n + 63) / 64));
  if (a.out_dtype == KDA_F32)
    fp8_matmul_kernel<float><<<grid, 256, 0, st>>>(A, B, a.m, a.n, a.k, static_cast<float *>(a.out), a.ldo);
  else
    fp8_matmul_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(A, B, a.m, a.n, a.k, static_cast<__nv_bfloat16 *>(a.out), a.ldo);
  return cudaGetLastError();
}

}  // namespace kda
