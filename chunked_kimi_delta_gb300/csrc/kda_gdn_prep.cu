// kda_gdn_prep.cu - what a chunk of the gated delta rule (one gate per head)
// needs before its state is known: the fp16 pieces of q and k, the numbers per
// token, A = (I + L)^-1 and P (kda_gdn.cuh).
//
// One CTA of four warps per (chunk, key head); the value heads of its group
// take turns on the products q k^T and k k^T, which are theirs in common.
// Warp w holds rows 16 w .. of both products in registers.  The inverse: the
// four diagonal blocks of 16 by substitution (a lane per column, fp32), then
// block column c by warp c alone, A_bc = -D_b (sum over m of L_bm A_mc), as
// three-term products of fp16 pieces.  A block is kept transposed in the
// half of L's array above the diagonal: the layout in which the next product
// reads it.
#include "kda_gdn.cuh"

namespace kda {
namespace gdn {
namespace {

constexpr int NT = 128;
constexpr int LP = 68;  // floats a row of L

// (hi, lo) + (h, l) with the rounding error of the sum kept
__device__ __forceinline__ void add2(float &hi, float &lo, float h, float l) {
  const float s = hi + h, v = s - hi;
  lo += l + ((hi - (s - v)) + (h - v));
  hi = s;
}

// Block (rows 16 b.., columns 16 m..) of L as the A operand, in pieces.
__device__ __forceinline__ void block_a(const float *M, int lane, float s, uint32_t (&hi)[4], uint32_t (&lo)[4]) {
  const int g = lane >> 2, t = (lane & 3) * 2;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = *reinterpret_cast<const float2 *>(M + (g + (i & 1) * 8) * LP + t + (i >> 1) * 8);
    split2(x.x * s, x.y * s, hi[i], lo[i]);
  }
}
// The same of a block that is kept transposed.
__device__ __forceinline__ void block_at(const float *M, int lane, float s, uint32_t (&hi)[4], uint32_t (&lo)[4]) {
  const int g = lane >> 2, t = (lane & 3) * 2;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float *x = M + (t + (i >> 1) * 8) * LP + g + (i & 1) * 8;
    split2(x[0] * s, x[LP] * s, hi[i], lo[i]);
  }
}
// Column tile nt of a transposed block as the B operand.
__device__ __forceinline__ void block_b(const float *M, int lane, int nt, float s, uint32_t (&hi)[2], uint32_t (&lo)[2]) {
  const int g = lane >> 2, t = (lane & 3) * 2;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 x = *reinterpret_cast<const float2 *>(M + (8 * nt + g) * LP + t + i * 8);
    split2(x.x * s, x.y * s, hi[i], lo[i]);
  }
}
__device__ __forceinline__ void mma3(float (&c)[4], const uint32_t (&ah)[4], const uint32_t (&al)[4], const uint32_t (&bh)[2],
                                     const uint32_t (&bl)[2]) {
  mma16(c, al, bh[0], bh[1]);
  mma16(c, ah, bl[0], bl[1]);
  mma16(c, ah, bh[0], bh[1]);
}
// Largest |x| of a 16 x 16 block over the warp.
__device__ __forceinline__ float block_max(const float *M, int lane) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(M[(lane >> 1) * LP + (lane & 1) * 8 + i]));
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
  return m;
}

template <typename T, int DK, bool BWD>
__global__ void __launch_bounds__(NT)
gdn_prep_kernel(Problem p, char *kq, char *ap, size_t kq_stride, size_t ap_stride) {
  constexpr int NI = pieces<T>(), U = DK / 8, NP = BWD ? 2 : NI;
  constexpr uint32_t TILE = C * DK * 2;
  extern __shared__ __align__(128) unsigned char smem[];
  float *Ls = reinterpret_cast<float *>(smem + 2 * NI * TILE);
  __shared__ float s_num[2][C], s_r[2][C], s_g[2][C], s_beta[C];  // 1 / norm of k and q, with and without the pieces' unit; G; beta
  __shared__ int s_max[2];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int hk = blockIdx.x % p.Hk;
  const int64_t c = blockIdx.x / p.Hk;
  int n, len;
  int64_t batch, tok;
  if (!chunk_at(p.s, c, n, batch, tok, len)) return;

  // ---- k and q: norms, pieces into shared memory and out
  char *kq_out = kq + (size_t)blockIdx.x * kq_stride;
  {
    constexpr int RW = 32 / U;  // rows a warp takes at once
    const int u = lane % U;
    for (int which = 0; which < 2; ++which) {
      const T *src = static_cast<const T *>(which ? p.q : p.k) + batch * p.qk.b + tok * p.qk.t + hk * p.qk.h;
#pragma unroll 4
      for (int r0 = warp * 16; r0 < warp * 16 + 16; r0 += RW) {
        const int r = r0 + lane / U;
        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (r < len) load8(src + r * p.qk.t + u * 8, x);
        float ss = 0.f, m = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          ss = fmaf(x[i], x[i], ss);
          m = fmaxf(m, fabsf(x[i]));
        }
#pragma unroll
        for (int o = U / 2; o; o >>= 1) {
          ss += __shfl_xor_sync(~0u, ss, o);
          m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
        }
        const float2 sc = piece_scale(m);
        uint4 hi, lo;
        split2(x[0] * sc.x, x[1] * sc.x, hi.x, lo.x);
        split2(x[2] * sc.x, x[3] * sc.x, hi.y, lo.y);
        split2(x[4] * sc.x, x[5] * sc.x, hi.z, lo.z);
        split2(x[6] * sc.x, x[7] * sc.x, hi.w, lo.w);
        const uint32_t at = which * NI * TILE + unit_at<U>(r, u);
        *reinterpret_cast<uint4 *>(smem + at) = hi;
        *reinterpret_cast<uint4 *>(kq_out + at) = hi;
        if constexpr (NI == 2) {
          *reinterpret_cast<uint4 *>(smem + at + TILE) = lo;
          *reinterpret_cast<uint4 *>(kq_out + at + TILE) = lo;
        }
        if (u == 0) {
          // x / norm = (unit / norm) (x / unit); rows past the end are zero
          const float f = (p.gp.flags & KDA_L2NORM_QK) ? 1.f / sqrtf(ss + p.gp.eps) : 1.f;
          s_num[which][r] = r < len ? f * sc.y : 0.f;
          s_r[which][r] = f;
        }
      }
    }
  }
  __syncthreads();

  // ---- k k^T and q k^T, rows 16 warp ..
  float kk[8][4], qk[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) kk[i][j] = qk[i][j] = 0.f;
  {
    const uint32_t K0 = smem_addr(smem), Q0 = K0 + NI * TILE;
    const int ra = 16 * warp + (lane & 15), ua = lane >> 4;                       // as the left operand
    const int rb = ((lane >> 4) << 3) + (lane & 7), ub = (lane >> 3) & 1;         // as the right one
#pragma unroll
    for (int ks = 0; ks < DK / 16; ++ks) {
      uint32_t ka[NI][4], qa[NI][4];
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        ldsm4(ka[i], K0 + i * TILE + unit_at<U>(ra, 2 * ks + ua));
        ldsm4(qa[i], Q0 + i * TILE + unit_at<U>(ra, 2 * ks + ua));
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (q > warp) continue;  // above the diagonal
        uint32_t b[NI][4];
#pragma unroll
        for (int i = 0; i < NI; ++i) ldsm4(b[i], K0 + i * TILE + unit_at<U>(16 * q + rb, 2 * ks + ub));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if constexpr (NI == 2) {
            mma16(kk[2 * q + h], ka[1], b[0][2 * h], b[0][2 * h + 1]);
            mma16(qk[2 * q + h], qa[1], b[0][2 * h], b[0][2 * h + 1]);
            mma16(kk[2 * q + h], ka[0], b[1][2 * h], b[1][2 * h + 1]);
            mma16(qk[2 * q + h], qa[0], b[1][2 * h], b[1][2 * h + 1]);
          }
          mma16(kk[2 * q + h], ka[0], b[0][2 * h], b[0][2 * h + 1]);
          mma16(qk[2 * q + h], qa[0], b[0][2 * h], b[0][2 * h + 1]);
        }
      }
    }
  }

  const int group = p.H / p.Hk;
  for (int hi_ = 0; hi_ < group; ++hi_) {
    const int h = hk * group + hi_;
    char *ap_out = ap + ((size_t)c * p.H + h) * ap_stride;
    float *num = reinterpret_cast<float *>(ap_out);
    if (hi_) __syncthreads();  // the last head's reads of shared memory are done
    if (tid < 2) s_max[tid] = 0;
    if (warp == 0) {
      // ---- the gate: two tokens a lane, running sum in two floats
      const float nea = (p.gp.flags & KDA_GATE_IN_KERNEL) ? -expf(p.gp.a_log[h]) : 0.f;
      const float bias = p.gp.dt_bias ? p.gp.dt_bias[h] : 0.f;
      const int64_t off = batch * p.gate.b + tok * p.gate.t + h * p.gate.h;
      float g[2], b[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 2 * lane + i;
        g[i] = r < len ? log_decay(p.g[off + r * p.gate.t], p.gp, nea, bias) : 0.f;
        b[i] = r < len ? p.beta[off + r * p.gate.t] : 0.f;
        if ((p.gp.flags & KDA_BETA_SIGMOID) && r < len) b[i] = 1.f / (1.f + expf(-b[i]));
      }
      float sh = g[0], sl = 0.f;
      add2(sh, sl, g[1], 0.f);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float h_ = __shfl_up_sync(~0u, sh, o), l_ = __shfl_up_sync(~0u, sl, o);
        if (lane >= o) add2(sh, sl, h_, l_);
      }
      float Gh[2] = {sh, sh}, Gl[2] = {sl, sl};
      add2(Gh[0], Gl[0], -g[1], 0.f);
      const float Ch = __shfl_sync(~0u, sh, 31), Cl = __shfl_sync(~0u, sl, 31);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 2 * lane + i;
        const float kn = s_num[0][r], qn = s_num[1][r];
        const float e = expf(Gh[i] + Gl[i]), f = expf((Ch - Gh[i]) + (Cl - Gl[i]));
        s_g[0][r] = Gh[i];
        s_g[1][r] = Gl[i];
        s_beta[r] = b[i];
        num[NUM_BETA + r] = b[i];
        num[NUM_EK + r] = e * kn;
        num[NUM_EQ + r] = e * qn * p.gp.scale;
        num[NUM_FK + r] = f * kn;
        num[NUM_K + r] = kn;
        num[NUM_Q + r] = qn;
        num[NUM_GH + r] = Gh[i];
        num[NUM_GL + r] = Gl[i];
        num[NUM_RK + r] = s_r[0][r];
        num[NUM_RQ + r] = s_r[1][r];
      }
      if (lane == 0) num[NUM_MISC] = expf(Ch + Cl);
    }
    __syncthreads();

    // ---- L into shared memory, P in registers
    const int g = lane >> 2, t = (lane & 3) * 2;
    float P[8][4];
    float pm = 0.f;
#pragma unroll
    for (int nt = 0; nt < 8; ++nt) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = 16 * warp + g + (e >> 1) * 8, j = 8 * nt + t + (e & 1);
        float lv = 0.f, pv = 0.f;
        if (j <= i) {
          const float y = expf((s_g[0][i] - s_g[0][j]) + (s_g[1][i] - s_g[1][j])) * s_num[0][j];
          pv = qk[nt][e] * s_num[1][i] * y * p.gp.scale;
          if (j < i) lv = kk[nt][e] * s_num[0][i] * y * s_beta[i];
        }
        P[nt][e] = pv;
        pm = fmaxf(pm, fabsf(pv));
        if (nt < 2 * warp + 2) Ls[i * LP + j] = lv;
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) pm = fmaxf(pm, __shfl_xor_sync(~0u, pm, o));
    if (lane == 0) atomicMax(&s_max[1], __float_as_int(pm));
    __syncwarp();

    // ---- D_w, transposed into its own place
    {
      float x[16];
      const float *Lw = Ls + 16 * warp * LP + 16 * warp;
      if (lane < 16) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float s = i == lane ? 1.f : 0.f;
#pragma unroll
          for (int l = 0; l < 16; ++l)
            if (l < i) s = fmaf(-Lw[i * LP + l], x[l], s);
          x[i] = s;
        }
      }
      __syncwarp();
      if (lane < 16) {
#pragma unroll
        for (int i = 0; i < 16; ++i) Ls[(16 * warp + lane) * LP + 16 * warp + i] = x[i];
      }
    }
    __syncthreads();

    // ---- block column `warp`
    float am = block_max(Ls + 16 * warp * (LP + 1), lane);
    for (int b = warp + 1; b < 4; ++b) {
      float acc[2][4] = {};
      // one unit for the products of this block row, from the largest of each side
      float lm = 0.f;
      for (int m = warp; m < b; ++m) lm = fmaxf(lm, block_max(Ls + 16 * b * LP + 16 * m, lane));
      const float2 sl = piece_scale(lm), sa = piece_scale(am);
      for (int m = warp; m < b; ++m) {
        uint32_t lh[4], ll[4];
        block_a(Ls + 16 * b * LP + 16 * m, lane, sl.x, lh, ll);
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          uint32_t bh[2], bl[2];
          block_b(Ls + 16 * warp * LP + 16 * m, lane, nt, sa.x, bh, bl);
          mma3(acc[nt], lh, ll, bh, bl);
        }
      }
      // M = sum over m, transposed to where A_bc will be, then A_bc = -D_b M
      float *At = Ls + 16 * warp * LP + 16 * b;
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) At[(8 * nt + t + (e & 1)) * LP + g + (e >> 1) * 8] = acc[nt][e] * sl.y * sa.y;
      __syncwarp();
      const float2 sm = piece_scale(block_max(At, lane)), sd = piece_scale(block_max(Ls + 16 * b * (LP + 1), lane));
      uint32_t dh[4], dl[4], mh[2][2], ml[2][2];
      block_at(Ls + 16 * b * (LP + 1), lane, -sd.x, dh, dl);
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        block_b(At, lane, nt, sm.x, mh[nt], ml[nt]);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[nt][e] = 0.f;
        mma3(acc[nt], dh, dl, mh[nt], ml[nt]);
      }
      __syncwarp();
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) At[(8 * nt + t + (e & 1)) * LP + g + (e >> 1) * 8] = acc[nt][e] * sd.y * sm.y;
      __syncwarp();
      am = fmaxf(am, block_max(At, lane));
    }
    if (lane == 0) atomicMax(&s_max[0], __float_as_int(am));
    __syncthreads();

    // ---- out: A (from its transposed blocks) and P
    const float2 sA = piece_scale(__int_as_float(s_max[0])), sP = piece_scale(__int_as_float(s_max[1]));
    char *A = ap_out + NUM_BYTES, *Pm = A + 2 * MAT_BYTES;
    if (tid == 0) {
      num[NUM_MISC + 1] = sA.y;
      num[NUM_MISC + 2] = sP.y;
    }
    for (int x = tid; x < C * 8; x += NT) {
      const int i = x & 63, u = x >> 6;
      if ((u >> 1) > (i >> 4)) continue;
      uint4 hi, lo;
      const float *col = Ls + 8 * u * LP + i;
      split2(col[0] * sA.x, col[LP] * sA.x, hi.x, lo.x);
      split2(col[2 * LP] * sA.x, col[3 * LP] * sA.x, hi.y, lo.y);
      split2(col[4 * LP] * sA.x, col[5 * LP] * sA.x, hi.z, lo.z);
      split2(col[6 * LP] * sA.x, col[7 * LP] * sA.x, hi.w, lo.w);
      *reinterpret_cast<uint4 *>(A + unit_at<8>(i, u)) = hi;
      *reinterpret_cast<uint4 *>(A + MAT_BYTES + unit_at<8>(i, u)) = lo;
    }
#pragma unroll
    for (int nt = 0; nt < 8; ++nt) {
      if (nt >= 2 * warp + 2) continue;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint32_t at = unit_at<8>(16 * warp + g + 8 * r, nt) + t * 2;
        uint32_t hi, lo;
        split2(P[nt][2 * r] * sP.x, P[nt][2 * r + 1] * sP.x, hi, lo);
        *reinterpret_cast<uint32_t *>(Pm + at) = hi;
        if constexpr (NP == 2) *reinterpret_cast<uint32_t *>(Pm + MAT_BYTES + at) = lo;
      }
    }
  }
}

}  // namespace

cudaError_t launch_gdn_prep(kda_dtype dt, bool bwd, const Problem &p, char *ws, const Plan &pl, cudaStream_t st) {
  if (p.nchunks == 0) return cudaSuccess;
  const size_t kqs = kq_bytes(dt, p.dk), aps = ap_bytes(dt, bwd);
  const int smem = (int)kqs + C * LP * 4;
  auto go = [&](auto kernel) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)(p.nchunks * (int64_t)p.Hk), NT, smem, st>>>(p, ws + pl.off_kq, ws + pl.off_ap, kqs, aps);
    return cudaGetLastError();
  };
  const bool w = p.dk == 128;
  if (dt == KDA_BF16) {
    if (bwd) return w ? go(gdn_prep_kernel<__nv_bfloat16, 128, true>) : go(gdn_prep_kernel<__nv_bfloat16, 64, true>);
    return w ? go(gdn_prep_kernel<__nv_bfloat16, 128, false>) : go(gdn_prep_kernel<__nv_bfloat16, 64, false>);
  }
  if (bwd) return w ? go(gdn_prep_kernel<float, 128, true>) : go(gdn_prep_kernel<float, 64, true>);
  return w ? go(gdn_prep_kernel<float, 128, false>) : go(gdn_prep_kernel<float, 64, false>);
}

}  // namespace gdn
}  // namespace kda
