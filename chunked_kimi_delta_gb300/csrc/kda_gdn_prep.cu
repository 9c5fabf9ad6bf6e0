// kda_gdn_prep.cu - what a chunk of the gated delta rule (one gate per head)
// needs before its state is known: the fp16 pieces of q and k, the numbers per
// token, A = (I + L)^-1 and P (kda_gdn.cuh).
//
// One CTA of four warps per (chunk, key head); the value heads of its group
// take turns on q k^T and k k^T, which are theirs in common and lie in shared
// memory where the pieces of q and k were.  The inverse: the four diagonal
// blocks of 16 by substitution (a lane per column, fp32), then two blocks of 16
// and one of 32 below them, A_21 = -A_22 (L_21 A_11), a warp to every eight
// columns: these never meet another warp's.  Their products take tf32 operands
// in two pieces (22 bits; tf32 has fp32's range, so no scaling has to be found).
// A is kept transposed in the half of L's array above the diagonal: the layout
// in which the next product reads it.
//
// 4 x 8192 tokens, 16 key heads of 128 with two value heads each, bf16: 292 us
// (8,192 CTAs, four an SM); its 0.97 GB would take 142.  What bounds it: 24 k
// instructions of a CTA at 46% of the issue slots, in dependent steps between
// barriers.  With the products in registers, and so three CTAs an SM and block
// column c of the inverse by warp c alone, 722 us.
#include <float.h>

#include "kda_gdn.cuh"

namespace kda {
namespace gdn {
namespace {

constexpr int NT = 128;
constexpr int LP = 68;  // floats a row of L
constexpr int HEADS = 4;  // value heads whose gates are computed at once, a warp each

// 8 values as they lie in memory
__device__ __forceinline__ void unpack8(const float4 (&r)[1], float (&x)[8]) {
  const uint32_t w[4] = {__float_as_uint(r[0].x), __float_as_uint(r[0].y), __float_as_uint(r[0].z), __float_as_uint(r[0].w)};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack8(const float4 (&r)[2], float (&x)[8]) {
  x[0] = r[0].x; x[1] = r[0].y; x[2] = r[0].z; x[3] = r[0].w;
  x[4] = r[1].x; x[5] = r[1].y; x[6] = r[1].z; x[7] = r[1].w;
}

// (hi, lo) + (h, l) with the rounding error of the sum kept
__device__ __forceinline__ void add2(float &hi, float &lo, float h, float l) {
  const float s = hi + h, v = s - hi;
  lo += l + ((hi - (s - v)) + (h - v));
  hi = s;
}

// A value's two tf32 pieces.
__device__ __forceinline__ void split_tf32(float x, uint32_t &hi, uint32_t &lo) {
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(hi) : "f"(x));
  const float r = x - __uint_as_float(hi);
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(lo) : "f"(r));
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// c[16 MT, 8] += M [16 MT, K] X [K, 8].  M: element (i, k) at M[i LP + k], or
// kept transposed at M[k LP + i]; where TRI its blocks above the diagonal, whose
// place holds L, are left out.  X: element (k, j) at X[j LP + k], from k = k0 on
// (likewise).
template <int MT, int K, bool TRANSPOSED, bool TRI>
__device__ __forceinline__ void block_product(float (&c)[MT][4], const float *M, const float *X, int lane, float sign, int k0 = 0) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int ks = 0; ks < K / 8; ++ks) {
    if (8 * ks < k0) continue;
    uint32_t bh[2], bl[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) split_tf32(X[g * LP + 8 * ks + t + 4 * i], bh[i], bl[i]);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (TRI && 8 * ks >= 16 * (m + 1)) continue;
      uint32_t ah[4], al[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 16 * m + g + 8 * (i & 1), k = 8 * ks + t + 4 * (i >> 1);
        split_tf32(sign * (TRANSPOSED ? M[k * LP + r] : M[r * LP + k]), ah[i], al[i]);
      }
      mma_tf32(c[m], al, bh[0], bh[1]);
      mma_tf32(c[m], ah, bl[0], bl[1]);
      mma_tf32(c[m], ah, bh[0], bh[1]);
    }
  }
}
// The accumulators to where X is read from, element (k, j) at X[j LP + k].
template <int MT> __device__ __forceinline__ void put_columns(const float (&c)[MT][4], float *X, int lane) {
  const int g = lane >> 2, t = (lane & 3) * 2;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int e = 0; e < 4; ++e) X[(t + (e & 1)) * LP + 16 * m + g + 8 * (e >> 1)] = c[m][e];
}

template <typename T, int DK> struct PrepShape {
  static constexpr uint32_t TILES = 2 * pieces<T>() * C * DK * 2, PRODUCTS = 2 * C * LP * 4;
  static constexpr uint32_t S_L = TILES > PRODUCTS ? TILES : PRODUCTS, BYTES = S_L + C * LP * 4;
};

template <typename T, int DK, bool BWD>
__global__ void __launch_bounds__(NT, 4)
gdn_prep_kernel(Problem p, char *kq, char *ap, size_t kq_stride, size_t ap_stride) {
  using Sh = PrepShape<T, DK>;
  constexpr int NI = pieces<T>(), U = DK / 8, NP = BWD ? 2 : NI;
  constexpr uint32_t TILE = C * DK * 2;
  extern __shared__ __align__(128) unsigned char smem[];
  // the pieces of k and q, and over them, once used, their products [64][LP]
  float *s_kk = reinterpret_cast<float *>(smem), *s_qk = s_kk + C * LP, *Ls = reinterpret_cast<float *>(smem + Sh::S_L);
  __shared__ __align__(16) float s_num[2][C], s_r[2][C];  // 1 / norm of k and q, with and without the pieces' unit
  __shared__ __align__(16) float s_g[HEADS][2][C], s_beta[HEADS][C], s_top[2][2];
  __shared__ int s_max;

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
    constexpr int K = 16 / RW;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const T *src = static_cast<const T *>(which ? p.q : p.k) + batch * p.qk.b + tok * p.qk.t + hk * p.qk.h;
      // all rows on their way before the first is used: no store to memory may come between, the compiler
      // could not tell it from what is read
      float4 raw[K][sizeof(T) / 2];
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int r = warp * 16 + k * RW + lane / U;
#pragma unroll
        for (int w = 0; w < (int)sizeof(T) / 2; ++w)
          raw[k][w] = r < len ? reinterpret_cast<const float4 *>(src + r * p.qk.t + u * 8)[w] : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      float ss[K], m[K];
#pragma unroll
      for (int k = 0; k < K; ++k) {
        float x[8];
        unpack8(raw[k], x);
        ss[k] = m[k] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          ss[k] = fmaf(x[i], x[i], ss[k]);
          m[k] = fmaxf(m[k], fabsf(x[i]));
        }
      }
#pragma unroll
      for (int o = U / 2; o; o >>= 1)
#pragma unroll
        for (int k = 0; k < K; ++k) {
          ss[k] += __shfl_xor_sync(~0u, ss[k], o);
          m[k] = fmaxf(m[k], __shfl_xor_sync(~0u, m[k], o));
        }
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int r = warp * 16 + k * RW + lane / U;
        const float2 sc = piece_scale(m[k]);
        float x[8];
        unpack8(raw[k], x);
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
          s_r[which][r] = ss[k];
          s_num[which][r] = r < len ? sc.y : 0.f;
        }
      }
    }
  }
  __syncthreads();
  {
    // a thread a row: x / norm = (unit / norm) (x / unit); rows past the end are zero
    const int which = tid / C, r = tid % C;
    const float ss = s_r[which][r];
    const bool l2 = (p.gp.flags & KDA_L2NORM_QK) != 0;
    const float f = r >= len ? 0.f : l2 ? 1.f / sqrtf(ss + p.gp.eps) : 1.f;  // eps may be zero
    const float unit = s_num[which][r] * f;
    s_r[which][r] = f;
    s_num[which][r] = unit;
    // the row's norm, from above; where its squares leave fp32's range by its largest value, below 2^14 units
    float top = ss > 1e-30f && ss < 1e30f ? sqrtf(ss) * f : fminf(sqrtf((float)DK) * 16384.f * unit, FLT_MAX);
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    if (lane == 0) s_top[which][warp & 1] = top;
  }

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

  __syncthreads();  // the pieces are used
  {
    const int g = lane >> 2, t = (lane & 3) * 2;
#pragma unroll
    for (int nt = 0; nt < 8; ++nt) {
      if (nt >= 2 * warp + 2) continue;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int at = (16 * warp + g + 8 * h) * LP + 8 * nt + t;
        *reinterpret_cast<float2 *>(s_kk + at) = make_float2(kk[nt][2 * h], kk[nt][2 * h + 1]);
        *reinterpret_cast<float2 *>(s_qk + at) = make_float2(qk[nt][2 * h], qk[nt][2 * h + 1]);
      }
    }
  }
  // |P| is at most the scale times the largest norms: a unit for its pieces
  // without looking at P itself
  const float bound = fminf(fabsf(p.gp.scale) * fmaxf(s_top[1][0], s_top[1][1]), FLT_MAX) * fmaxf(s_top[0][0], s_top[0][1]);
  const float2 sP = piece_scale(bound);

  const int group = p.H / p.Hk;
  for (int hv = 0; hv < group; ++hv) {
    const int h = hk * group + hv;
    if (hv % HEADS == 0) {
      __syncthreads();
      if (hv + warp < group) {
        // ---- the gate of head h + warp: two tokens a lane, running sum in two floats, to base 2
        const int hw = h + warp;
        float *num = reinterpret_cast<float *>(ap + ((size_t)c * p.H + hw) * ap_stride);
        const float nea = (p.gp.flags & KDA_GATE_IN_KERNEL) ? -expf(p.gp.a_log[hw]) : 0.f;
        const float bias = p.gp.dt_bias ? p.gp.dt_bias[hw] : 0.f;
        const int64_t off = batch * p.gate.b + tok * p.gate.t + hw * p.gate.h;
        float g[2], b[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = 2 * lane + i;
          g[i] = r < len ? LOG2E * log_decay(p.g[off + r * p.gate.t], p.gp, nea, bias) : 0.f;
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
          const float e = exp2f(Gh[i] + Gl[i]), f = exp2f((Ch - Gh[i]) + (Cl - Gl[i]));
          s_g[warp][0][r] = Gh[i];
          s_g[warp][1][r] = Gl[i];
          s_beta[warp][r] = b[i];
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
        if (lane == 0) {
          num[NUM_MISC] = exp2f(Ch + Cl);
          num[NUM_MISC + 2] = sP.y;
        }
      }
    }
    __syncthreads();  // the gates; the last head's A is out
    char *ap_out = ap + ((size_t)c * p.H + h) * ap_stride;
    char *A = ap_out + NUM_BYTES, *Pm = A + 2 * MAT_BYTES;
    const float *gh = s_g[hv % HEADS][0], *gl = s_g[hv % HEADS][1], *beta = s_beta[hv % HEADS];
    if (tid == 0) s_max = 0;

    // ---- L, and P on its way out: eight columns a thread, blocks of 16 down to the diagonal alone
    for (int x = tid; x < 320; x += NT) {
      // block row b has 2 (b + 1) units in each of its 16 rows: 32, 64, 96, 128 of them
      const int b = x < 32 ? 0 : x < 96 ? 1 : x < 192 ? 2 : 3, y = x - 16 * b * (b + 1);
      const int i = 16 * b + y % 16, u = y / 16;
      const float hi_i = gh[i], lo_i = gl[i], ki = s_num[0][i] * beta[i], qi = s_num[1][i] * p.gp.scale * sP.x;
      float pv[8], lv[8];
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const int j0 = 8 * u + 4 * w;
        const float4 kk4 = *reinterpret_cast<const float4 *>(s_kk + i * LP + j0), qk4 = *reinterpret_cast<const float4 *>(s_qk + i * LP + j0),
                     h4 = *reinterpret_cast<const float4 *>(gh + j0), l4 = *reinterpret_cast<const float4 *>(gl + j0),
                     n4 = *reinterpret_cast<const float4 *>(s_num[0] + j0);
        const float kkv[4] = {kk4.x, kk4.y, kk4.z, kk4.w}, qkv[4] = {qk4.x, qk4.y, qk4.z, qk4.w}, hv4[4] = {h4.x, h4.y, h4.z, h4.w},
                    lv4[4] = {l4.x, l4.y, l4.z, l4.w}, nv[4] = {n4.x, n4.y, n4.z, n4.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = j0 + e;
          const float gam = j <= i ? exp2_neg((hi_i - hv4[e]) + (lo_i - lv4[e])) * nv[e] : 0.f;
          pv[4 * w + e] = j <= i ? qkv[e] * gam * qi : 0.f;
          lv[4 * w + e] = j < i ? kkv[e] * gam * ki : 0.f;
        }
        *reinterpret_cast<float4 *>(Ls + i * LP + j0) = make_float4(lv[4 * w], lv[4 * w + 1], lv[4 * w + 2], lv[4 * w + 3]);
      }
      uint4 hi, lo;
      split2(pv[0], pv[1], hi.x, lo.x);
      split2(pv[2], pv[3], hi.y, lo.y);
      split2(pv[4], pv[5], hi.z, lo.z);
      split2(pv[6], pv[7], hi.w, lo.w);
      *reinterpret_cast<uint4 *>(Pm + unit_at<8>(i, u)) = hi;
      if constexpr (NP == 2) *reinterpret_cast<uint4 *>(Pm + MAT_BYTES + unit_at<8>(i, u)) = lo;
    }
    __syncthreads();

    // ---- diagonal blocks, transposed into their own places
    float top = 1.f;  // A's own diagonal
    {
      float x[16];
      const float *Lw = Ls + 16 * warp * (LP + 1);
      if (lane < 16) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float s[2] = {i == lane ? 1.f : 0.f, 0.f};
#pragma unroll
          for (int l = 0; l < 16; ++l)
            if (l < i) s[l & 1] = fmaf(-Lw[i * LP + l], x[l], s[l & 1]);
          x[i] = s[0] + s[1];
          top = fmaxf(top, fabsf(x[i]));
        }
      }
      __syncwarp();
      if (lane < 16) {
#pragma unroll
        for (int i = 0; i < 16; i += 4)
          *reinterpret_cast<float4 *>(Ls + (16 * warp + lane) * LP + 16 * warp + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
      }
    }
    __syncthreads();
    // ---- blocks (1, 0) and (3, 2): a pair of warps each, eight columns a warp
    {
      const int d = 32 * (warp >> 1), col = 8 * (warp & 1);
      float acc[1][4] = {};
      block_product<1, 16, false, false>(acc, Ls + (d + 16) * LP + d, Ls + (d + col) * LP + d, lane, 1.f);
      float *X = Ls + (d + col) * LP + d + 16;  // rows: columns of A; where block (1, 0) is kept
      put_columns(acc, X, lane);
      __syncwarp();
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[0][e] = 0.f;
      block_product<1, 16, true, false>(acc, Ls + (d + 16) * (LP + 1), X, lane, -1.f);
      __syncwarp();
      put_columns(acc, X, lane);
#pragma unroll
      for (int e = 0; e < 4; ++e) top = fmaxf(top, fabsf(acc[0][e]));
    }
    __syncthreads();
    // ---- the block of 32 below: eight columns a warp
    {
      float acc[2][4] = {};
      block_product<2, 32, false, false>(acc, Ls + 32 * LP, Ls + 8 * warp * LP, lane, 1.f, 16 * (warp >> 1));
      float *X = Ls + 8 * warp * LP + 32;
      put_columns(acc, X, lane);
      __syncwarp();
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[m][e] = 0.f;
      block_product<2, 32, true, true>(acc, Ls + 32 * (LP + 1), X, lane, -1.f);
      __syncwarp();
      put_columns(acc, X, lane);
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) top = fmaxf(top, fabsf(acc[m][e]));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    if (lane == 0) atomicMax(&s_max, __float_as_int(top));
    __syncthreads();

    // ---- A out, from its transpose
    const float2 sA = piece_scale(__int_as_float(s_max));
    if (tid == 0) reinterpret_cast<float *>(ap_out)[NUM_MISC + 1] = sA.y;
    for (int x = tid; x < 320; x += NT) {
      const int b = x < 32 ? 0 : x < 96 ? 1 : x < 192 ? 2 : 3, y = x - 16 * b * (b + 1);
      const int i = 16 * b + y % 16, u = y / 16;
      uint4 hi, lo;
      const float *col = Ls + 8 * u * LP + i;
      split2(col[0] * sA.x, col[LP] * sA.x, hi.x, lo.x);
      split2(col[2 * LP] * sA.x, col[3 * LP] * sA.x, hi.y, lo.y);
      split2(col[4 * LP] * sA.x, col[5 * LP] * sA.x, hi.z, lo.z);
      split2(col[6 * LP] * sA.x, col[7 * LP] * sA.x, hi.w, lo.w);
      *reinterpret_cast<uint4 *>(A + unit_at<8>(i, u)) = hi;
      *reinterpret_cast<uint4 *>(A + MAT_BYTES + unit_at<8>(i, u)) = lo;
    }
  }
}

// Zeros behind the last sequence, the blocks' share `block` of `blocks`.
__device__ void zero_behind(const SeqInfo &s, const Behind &z, int64_t block, int64_t blocks) {
  const int64_t end = s.bounds[s.N], tok = end < 0 ? 0 : end > s.T_tot ? s.T_tot : end, bytes = (s.T_tot - tok) * z.token;
  if (bytes == 0) return;
  const int64_t first = (block * ORDERED + threadIdx.x) * 16, step = blocks * ORDERED * 16;
  for (int64_t h = 0; h < z.heads; ++h) {
    char *to = static_cast<char *>(z.p) + h * z.pitch + tok * z.token;
    if (z.token % 16 == 0 && z.pitch % 16 == 0) {
      for (int64_t x = first; x < bytes; x += step) *reinterpret_cast<uint4 *>(to + x) = make_uint4(0, 0, 0, 0);
    } else {  // g's and beta's, one word a token and head
      for (int64_t x = first / 4; x < bytes; x += step / 4) *reinterpret_cast<uint32_t *>(to + x) = 0;
    }
  }
}

// The first block: a thread a sequence.
__global__ void __launch_bounds__(ORDERED) gdn_map_kernel(SeqInfo s, int32_t *chunk_off, int32_t *order, BehindAll z) {
  __shared__ int s_n[ORDERED], s_w[ORDERED / 32];
  const int with_map = order != nullptr;
  if ((int)blockIdx.x >= with_map) {
    for (int i = 0; i < z.n; ++i) zero_behind(s, z.a[i], blockIdx.x - with_map, gridDim.x - with_map);
    return;
  }
  const int n = threadIdx.x, lane = n & 31, warp = n >> 5;
  int chunks = 0;
  if (n < s.N) {
    int64_t t0, t1;
    seq_range(s, n, t0, t1);
    chunks = (int)((t1 - t0 + C - 1) / C);
  }
  s_n[n] = chunks;
  int sum = chunks;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(~0u, sum, o);
    if (lane >= o) sum += v;
  }
  if (lane == 31) s_w[warp] = sum;
  __syncthreads();
  if (n >= s.N) return;
  for (int w = 0; w < warp; ++w) sum += s_w[w];
  if (n == 0) chunk_off[0] = 0;
  chunk_off[n + 1] = sum;
  int rank = 0;
  for (int m = 0; m < s.N; ++m) rank += s_n[m] > chunks || (s_n[m] == chunks && m < n);
  order[rank] = n;
}

}  // namespace

cudaError_t launch_gdn_map(const SeqInfo &s, int32_t *chunk_off, int32_t *order, const BehindAll &z, cudaStream_t st) {
  gdn_map_kernel<<<(order ? 1 : 0) + (z.n ? 32 : 0), ORDERED, 0, st>>>(s, chunk_off, order, z);
  return cudaGetLastError();
}

cudaError_t launch_gdn_prep(kda_dtype dt, bool bwd, const Problem &p, char *ws, const Plan &pl, cudaStream_t st) {
  if (p.nchunks == 0) return cudaSuccess;
  const size_t kqs = kq_bytes(dt, p.dk), aps = ap_bytes(dt, bwd);
  auto go = [&](auto kernel, int smem) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)(p.nchunks * (int64_t)p.Hk), NT, smem, st>>>(p, ws + pl.off_kq, ws + pl.off_ap, kqs, aps);
    return cudaGetLastError();
  };
  const bool w = p.dk == 128;
  if (dt == KDA_BF16) {
    if (bwd) return w ? go(gdn_prep_kernel<__nv_bfloat16, 128, true>, PrepShape<__nv_bfloat16, 128>::BYTES) : go(gdn_prep_kernel<__nv_bfloat16, 64, true>, PrepShape<__nv_bfloat16, 64>::BYTES);
    return w ? go(gdn_prep_kernel<__nv_bfloat16, 128, false>, PrepShape<__nv_bfloat16, 128>::BYTES) : go(gdn_prep_kernel<__nv_bfloat16, 64, false>, PrepShape<__nv_bfloat16, 64>::BYTES);
  }
  if (bwd) return w ? go(gdn_prep_kernel<float, 128, true>, PrepShape<float, 128>::BYTES) : go(gdn_prep_kernel<float, 64, true>, PrepShape<float, 64>::BYTES);
  return w ? go(gdn_prep_kernel<float, 128, false>, PrepShape<float, 128>::BYTES) : go(gdn_prep_kernel<float, 64, false>, PrepShape<float, 64>::BYTES);
}

}  // namespace gdn
}  // namespace kda
