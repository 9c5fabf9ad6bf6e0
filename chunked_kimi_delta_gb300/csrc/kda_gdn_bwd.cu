// kda_gdn_bwd.cu - backward of the gated delta rule with one gate per head
// (kda_gdn.cuh).  With dS' the gradient of the state leaving a chunk:
//   dW = P^T dO + (e^{G_C - G} K) dS'        dY = A^T dW      dR = beta dY = dV
//   dS = e^{G_C} dS' + (scale e^G Q)^T dO - (e^G K)^T dR
//   dP = dO W^T (j <= i)                     dL = -dY W^T (j < i)
//   dQ = scale (e^G dO S^T + (dP e^{G_i - G_j}) K)
//   dK = -e^G dR S^T + e^{G_C - G} W dS'^T + (..dP..)^T scale Q + (M + M^T) K,   M_ij = beta_i e^{G_i - G_j} dL_ij
//   dbeta_i = dY_i.R_i + sum_j dL_ij L_ij / beta_i
// The gate at token r scales everything that crosses it, and only that:
//   dg_r = sum_{i >= r > j} (dP_ij P_ij + dL_ij L_ij) + sum_{i >= r} (scale e^G (q S).dO - e^G (k S).dR)_i
//          + sum_{j < r} (e^{G_C - G} W.(k dS'))_j + e^{G_C} <S, dS'>
// Summed like this nothing cancels that the result does not cancel itself (as
// differences of sums over q dq and k dk it loses 10^-4 under strong decay).
//
// Three kernels after the preparation: the forward's chain once more, which
// leaves each chunk's S and W; the chain backwards, warps as there, dS^T in
// registers (reverse_kernel); then all chunks at once for what meets over the
// value channels (intra_kernel).  4 x 8192 tokens of 32 heads on 16 key heads, d = 128,
// bf16: preparation 298 us, chain 641, reverse 1,089 (484 products a warp and
// chunk, 7.7 k of its 17 k cycles; beside them 250 KB of a chunk in and out),
// intra 2,513.  With one unit for a chunk's d_out instead of a token's 2,476.
#include "kda_gdn.cuh"

namespace kda {
namespace gdn {
namespace {

// ---------------------------------------------------------------- chain, backwards
template <typename T, int DK, int WARPS> struct RevShape {
  static constexpr int NI = pieces<T>();
  static constexpr uint32_t TILE = C * DK * 2, STRIP = C * 16 * sizeof(T);
  static constexpr uint32_t S_K = 0, S_Q = NI * TILE, S_NUM = 2 * NI * TILE, S_A = S_NUM + NUM_BYTES, S_P = S_A + 2 * MAT_BYTES,
                            S_DO = S_P + 2 * MAT_BYTES, S_V = S_DO + WARPS * STRIP, STAGE = (S_V + WARPS * STRIP + 127) / 128 * 128,
                            REST = (NI == 1 ? WARPS * STRIP : 0) + WARPS * DOT_FLOATS * 4;
  static constexpr int STAGES = 2 * STAGE + REST <= 232448 ? 2 : 1;
  static constexpr int THREADS = WARPS * 32 + (STAGES == 2 ? FILL : 0);
  static constexpr uint32_t S_OUT = STAGES * STAGE, S_DOTS = S_OUT + (NI == 1 ? WARPS * STRIP : 0),
                            BYTES = S_DOTS + WARPS * DOT_FLOATS * 4;
};

// A warp's strip [64 tokens][16 channels] transposed, as accumulators.
template <typename T> __device__ __forceinline__ void load_strip(const unsigned char *strip, int lane, float (&x)[8][4]) {
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t r[4];
      ldsm4t(r, smem_addr(strip) + (16 * q + ((lane >> 4) << 3) + (lane & 7)) * 32 + ((lane >> 3) & 1) * 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * q + (i >> 1)][2 * (i & 1)] = __uint_as_float(r[i] << 16);
        x[2 * q + (i >> 1)][2 * (i & 1) + 1] = __uint_as_float(r[i] & 0xffff0000u);
      }
    }
  } else {
    const float *f = reinterpret_cast<const float *>(strip);
    const int g = lane >> 2, t = (lane & 3) * 2;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[i][e] = f[(8 * i + t + (e & 1)) * 16 + g + (e >> 1) * 8];
  }
}

// Sums over a warp's 16 channels for all 64 tokens: x[2 tile + e] is this
// lane's part (two channels) for token 8 tile + 2 (lane % 4) + e.  The lanes
// share out the tiles as they add, so that 14 exchanges do.
__device__ __forceinline__ void channel_sums(float (&x)[16], int lane, float *to) {
#pragma unroll
  for (int n = 8; n >= 2; n >>= 1) {
    const int bit = 2 * n;  // lanes 16, 8, 4 apart
    const bool up = lane & bit;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float send = up ? x[i] : x[i + n], keep = up ? x[i + n] : x[i];
      x[i] = keep + __shfl_xor_sync(~0u, send, bit);
    }
  }
  const int tile = (lane >> 4 & 1) * 4 + (lane >> 3 & 1) * 2 + (lane >> 2 & 1);
  *reinterpret_cast<float2 *>(to + 8 * tile + 2 * (lane & 3)) = make_float2(x[0], x[1]);
}

template <typename T, int DK, int WARPS>
__global__ void __launch_bounds__(RevShape<T, DK, WARPS>::THREADS, 1)
gdn_reverse_kernel(Problem p, char *ws, Plan pl, size_t kq_stride, size_t ap_stride, GradOut io) {
  using Sh = RevShape<T, DK, WARPS>;
  constexpr int NI = Sh::NI, U = DK / 8, NK = DK / 8;
  extern __shared__ __align__(128) unsigned char smem[];
  const char *kq = ws + pl.off_kq, *ap = ws + pl.off_ap;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = (lane & 3) * 2;
  const int slices = p.dv / (16 * WARPS), slice = blockIdx.x % slices;
  const int h = (int)(blockIdx.x / slices % p.H), at = (int)(blockIdx.x / slices / p.H), n = p.order ? p.order[at] : at;
  const int hk = h / (p.H / p.Hk);
  const int v0 = (slice * WARPS + warp) * 16;
  int64_t t0, t1;
  seq_range(p.s, n, t0, t1);
  const int64_t c0 = seq_first_chunk(p.s, n);
  const int nc = (int)max((int64_t)0, min((t1 - t0 + C - 1) / C, p.nchunks - c0));
  const int64_t batch = p.s.bounds ? 0 : n, tok = p.s.bounds ? t0 : 0;
  const int64_t v_off = batch * p.v.b + tok * p.v.t + h * p.v.h + v0;
  const T *v = static_cast<const T *>(p.val) + v_off;
  const T *d_out = io.d_out ? static_cast<const T *>(io.d_out) + v_off : nullptr;
  T *dv = static_cast<T *>(io.dv) + v_off;
  float *s_dots = reinterpret_cast<float *>(smem + Sh::S_DOTS) + warp * DOT_FLOATS;

  const uint32_t base = smem_addr(smem);
  auto load = [&](int c, uint32_t stage, uint32_t first, uint32_t step) {
    const char *a = kq + ((size_t)(c0 + c) * p.Hk + hk) * kq_stride, *b = ap + ((size_t)(c0 + c) * p.H + h) * ap_stride;
#pragma unroll 4
    for (uint32_t x = first; x < Sh::S_NUM; x += step) cp16(stage + Sh::S_K + x, a + x);
#pragma unroll 4
    for (uint32_t x = first; x < Sh::S_DO - Sh::S_NUM; x += step) cp16(stage + Sh::S_NUM + x, b + x);
  };
  if constexpr (Sh::STAGES == 2) {
    if (warp >= WARPS) {
      registers_to_fill<WARPS>();
      const int first = tid - WARPS * 32;
      const T *vs = v - warp * 16, *os = d_out ? d_out - warp * 16 : vs;  // without d_out zeros, and nothing is read
      fill_buffers<WARPS / 4>(nc, [&](int i) {
        const int c = nc - 1 - i;
        const uint32_t stage = base + (i & 1) * Sh::STAGE;
        const int64_t r0 = (int64_t)c * C;
        load(c, stage, first * 16, FILL * 16);
        load_strips<WARPS>(stage + Sh::S_DO, os + r0 * p.v.t, p.v.t, d_out ? t1 - t0 - r0 : 0, first);
        load_strips<WARPS>(stage + Sh::S_V, vs + r0 * p.v.t, p.v.t, t1 - t0 - r0, first);
        // what this chunk's warps read themselves is on its way to L2 as well
        const int64_t unit = (c0 + c) * p.H + h;
        const size_t part = (unit * p.dv + slice * WARPS * 16) * (C * 4);
        const char *w = ws + pl.off_w + part, *e = ws + pl.off_e + part;
        for (int x = first * 128; x < WARPS * 16 * C * 4; x += FILL * 128) {
          asm volatile("prefetch.global.L2 [%0];" ::"l"(w + x));
          asm volatile("prefetch.global.L2 [%0];" ::"l"(e + x));
        }
      });
      return;
    }
    registers_to_compute<WARPS>();
  }
  const int group = warp >> 2;

  const int64_t s_off = ((int64_t)n * p.H + h) * DK * p.dv;
  const int64_t sk = p.v_first ? 1 : p.dv, sv = p.v_first ? DK : 1;
  float D[NK][4];
#pragma unroll
  for (int i = 0; i < NK; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      D[i][e] = io.d_final ? io.d_final[s_off + (8 * i + t + (e & 1)) * sk + (v0 + g + (e >> 1) * 8) * sv] : 0.f;

  const int rb = ((lane >> 4) << 3) + (lane & 7), ub = (lane >> 3) & 1;
  const int rt = (((lane >> 3) & 1) << 3) + (lane & 7), ut = lane >> 4;
  // The second group begins a chunk when the first has dW of it: left alone they fall in step or out of it as the code
  // around happens to be (1110 to 1180 us for 4 x 8192 tokens of 32 heads, bf16 128 x 128; so 1089, at the first chunk
  // alone 1079 to 1170; 64 x 128 800, so 793; 16 chunks 152, so 145).  Two barriers in turn: the first group comes to
  // the second chunk after this one only when the second has emptied this one's buffer.
  constexpr bool APART = Sh::STAGES == 2 && WARPS == 8;
  for (int c = nc - 1; c >= 0; --c) {
    const int stage = (nc - 1 - c) & 1;
    const uint32_t so = Sh::STAGES == 2 ? stage * Sh::STAGE : 0, st = base + so;
    if constexpr (Sh::STAGES == 2) {
      bar_sync(bar_full(stage, group), GROUP + FILL);
      if (APART && group == 1) bar_sync(BAR_START + stage, 2 * GROUP);
    } else {
      load(c, st, tid * 16, WARPS * 512);
#pragma unroll
      for (int x = lane; x < C * 4; x += 32) {
        const int64_t r = (int64_t)c * C + x / 4;
        const bool in = r < t1 - t0;
        const int64_t at = (in ? r * p.v.t : 0) + x % 4 * 4;
        cp16z(st + Sh::S_V + warp * Sh::STRIP + x * 16, v + at, in);
        cp16z(st + Sh::S_DO + warp * Sh::STRIP + x * 16, d_out ? d_out + at : v + at, in && d_out);
      }
      cp_commit();
      cp_wait<0>();
      __syncthreads();
    }
    const float *num = reinterpret_cast<const float *>(smem + so + Sh::S_NUM);
    const int64_t unit = (c0 + c) * p.H + h;
    float *maxes = reinterpret_cast<float *>(ws + pl.off_max) + unit * MAX_FLOATS + v0 / 16;
    auto tiles = [&](size_t off, int n_) { return reinterpret_cast<float4 *>(ws + off) + (unit * (p.dv / 16) + v0 / 16) * n_ * 32 + lane; };

    // ---- dS' out; X = e^{G_C - G} k dS' and its sums with W
    float4 *ds_to = tiles(pl.off_ds, NK);
#pragma unroll
    for (int i = 0; i < NK; ++i) ds_to[i * 32] = make_float4(D[i][0], D[i][1], D[i][2], D[i][3]);
    float2 z0, z1;
    {
      const float m = warp_max(D);
      if (lane == 0) maxes[MAX_DS] = m;
    }
    float4 wv[8];
    {
      const float4 *from = tiles(pl.off_w, 8);
#pragma unroll
      for (int i = 0; i < 8; ++i) wv[i] = from[i * 32];
    }
    row_scales(D, z0, z1);
    float X[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) X[i][e] = 0.f;
#pragma unroll
    for (int ks = 0; ks < DK / 16; ++ks) {
      uint32_t ah[4], al[4];
      as_left(D, ks, z0.x, z1.x, ah, al);
      uint32_t b[4][4];
#pragma unroll
      for (int q = 0; q < 4; ++q) ldsm4(b[q], st + Sh::S_K + unit_at<U>(16 * q + rb, 2 * ks + ub));
      mma_row(X, al, b);
      mma_row(X, ah, b);
      if constexpr (NI == 2) {
#pragma unroll
        for (int q = 0; q < 4; ++q) ldsm4(b[q], st + Sh::S_K + Sh::TILE + unit_at<U>(16 * q + rb, 2 * ks + ub));
        mma_row(X, ah, b);
      }
    }
    float dots[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 fk = *reinterpret_cast<const float2 *>(num + NUM_FK + 8 * i + t);
      X[i][0] = X[i][0] * fk.x * z0.y;
      X[i][1] = X[i][1] * fk.y * z0.y;
      X[i][2] = X[i][2] * fk.x * z1.y;
      X[i][3] = X[i][3] * fk.y * z1.y;
      dots[2 * i] = wv[i].x * X[i][0] + wv[i].z * X[i][2];
      dots[2 * i + 1] = wv[i].y * X[i][1] + wv[i].w * X[i][3];
    }
    channel_sums(dots, lane, s_dots + DOT_Y);

    // ---- dW = X + P^T dO
    float O[8][4], Y[8][4];
    load_strip<T>(smem + so + Sh::S_DO + warp * Sh::STRIP, lane, O);
    row_scales(O, z0, z1);
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) Y[i][e] = 0.f;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      uint32_t ah[4], al[4];
      as_left(O, ks, z0.x, z1.x, ah, al);
      uint32_t b[4][4];
#pragma unroll
      for (int q = 0; q <= ks; ++q) ldsm4t(b[q], st + Sh::S_P + MAT_BYTES + unit_at<8>(16 * ks + rt, 2 * q + ut));
      mma_row(Y, ah, b, 0, ks + 1);
#pragma unroll
      for (int q = 0; q <= ks; ++q) ldsm4t(b[q], st + Sh::S_P + unit_at<8>(16 * ks + rt, 2 * q + ut));
      if constexpr (NI == 2) mma_row(Y, al, b, 0, ks + 1);
      mma_row(Y, ah, b, 0, ks + 1);
    }
    {
      const float a = num[NUM_MISC + 2];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        X[i][0] += Y[i][0] * a * z0.y;
        X[i][1] += Y[i][1] * a * z0.y;
        X[i][2] += Y[i][2] * a * z1.y;
        X[i][3] += Y[i][3] * a * z1.y;
      }
    }
    float4 ev[8];
    {
      const float4 *from = tiles(pl.off_e, 8);
#pragma unroll
      for (int i = 0; i < 8; ++i) ev[i] = from[i * 32];
    }

    if (APART && group == 0) bar_arrive(BAR_START + stage, 2 * GROUP);

    // ---- dY = A^T dW
    row_scales(X, z0, z1);
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) Y[i][e] = 0.f;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      uint32_t ah[4], al[4];
      as_left(X, ks, z0.x, z1.x, ah, al);
      uint32_t b[4][4];
#pragma unroll
      for (int q = 0; q <= ks; ++q) ldsm4t(b[q], st + Sh::S_A + MAT_BYTES + unit_at<8>(16 * ks + rt, 2 * q + ut));
      mma_row(Y, ah, b, 0, ks + 1);
#pragma unroll
      for (int q = 0; q <= ks; ++q) ldsm4t(b[q], st + Sh::S_A + unit_at<8>(16 * ks + rt, 2 * q + ut));
      mma_row(Y, al, b, 0, ks + 1);
      mma_row(Y, ah, b, 0, ks + 1);
    }
    load_strip<T>(smem + so + Sh::S_V + warp * Sh::STRIP, lane, O);  // v, for R = v - e^G k S
    float4 *dy_to = tiles(pl.off_dy, 8);
    const float a = num[NUM_MISC + 1];
    float ym = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      Y[i][0] = Y[i][0] * a * z0.y;
      Y[i][1] = Y[i][1] * a * z0.y;
      Y[i][2] = Y[i][2] * a * z1.y;
      Y[i][3] = Y[i][3] * a * z1.y;
      ym = fmaxf(ym, fmaxf(fmaxf(fabsf(Y[i][0]), fabsf(Y[i][1])), fmaxf(fabsf(Y[i][2]), fabsf(Y[i][3]))));
      dy_to[i * 32] = make_float4(Y[i][0], Y[i][1], Y[i][2], Y[i][3]);
      dots[2 * i] = Y[i][0] * (O[i][0] - ev[i].x) + Y[i][2] * (O[i][2] - ev[i].z);
      dots[2 * i + 1] = Y[i][1] * (O[i][1] - ev[i].y) + Y[i][3] * (O[i][3] - ev[i].w);
    }
    channel_sums(dots, lane, s_dots + DOT_BETA);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 be = *reinterpret_cast<const float2 *>(num + NUM_BETA + 8 * i + t);
      Y[i][0] *= be.x;
      Y[i][1] *= be.y;
      Y[i][2] *= be.x;
      Y[i][3] *= be.y;
      dots[2 * i] = -(Y[i][0] * ev[i].x + Y[i][2] * ev[i].z);
      dots[2 * i + 1] = -(Y[i][1] * ev[i].y + Y[i][3] * ev[i].w);
    }
    channel_sums(dots, lane, s_dots + DOT_K);
#pragma unroll
    for (int o = 16; o; o >>= 1) ym = fmaxf(ym, __shfl_xor_sync(~0u, ym, o));
    if (lane == 0) maxes[MAX_DY] = ym;

    // ---- dV = dR
    const int64_t r0 = (int64_t)c * C;
    const int len = (int)(t1 - t0 - r0 < C ? t1 - t0 - r0 : C);
    if constexpr (NI == 1) {
      const uint32_t os = base + Sh::S_OUT + warp * Sh::STRIP;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __nv_bfloat162 x = __floats2bfloat162_rn(Y[2 * q + (i >> 1)][2 * (i & 1)], Y[2 * q + (i >> 1)][2 * (i & 1) + 1]);
          r[i] = *reinterpret_cast<const uint32_t *>(&x);
        }
        stsm4t(os + (16 * q + ((lane >> 4) << 3) + (lane & 7)) * 32 + ((lane >> 3) & 1) * 16, r[0], r[1], r[2], r[3]);
      }
      __syncwarp();
#pragma unroll
      for (int x = lane; x < C * 2; x += 32)
        if ((x >> 1) < len)
          *reinterpret_cast<uint4 *>(dv + (r0 + (x >> 1)) * p.v.t + (x & 1) * 8) =
              *reinterpret_cast<const uint4 *>(smem + Sh::S_OUT + warp * Sh::STRIP + x * 16);
      __syncwarp();
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = 8 * i + t + (e & 1);
          if (j < len) dv[(r0 + j) * p.v.t + g + (e >> 1) * 8] = Y[i][e];
        }
    }

    // ---- dS^T = e^{G_C} dS'^T + (scale e^G dO)^T q - (e^G dR)^T k
    const float ec = num[NUM_MISC];
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      if (which == 0) load_strip<T>(smem + so + Sh::S_DO + warp * Sh::STRIP, lane, O);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 f = *reinterpret_cast<const float2 *>(num + (which ? NUM_EK : NUM_EQ) + 8 * i + t);
        if (which) {
          O[i][0] = -Y[i][0] * f.x;
          O[i][1] = -Y[i][1] * f.y;
          O[i][2] = -Y[i][2] * f.x;
          O[i][3] = -Y[i][3] * f.y;
        } else {
          O[i][0] *= f.x;
          O[i][1] *= f.y;
          O[i][2] *= f.x;
          O[i][3] *= f.y;
        }
      }
      row_scales(O, z0, z1);
      uint32_t xh[4][4], xl[4][4];
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) as_left(O, ks, z0.x, z1.x, xh[ks], xl[ks]);
      const uint32_t right = st + (which ? Sh::S_K : Sh::S_Q);
#pragma unroll
      for (int q = 0; q < NK / 2; q += 2) {
        float acc[4][4] = {};
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          uint32_t b[2][4];
#pragma unroll
          for (int i = 0; i < 2; ++i) ldsm4t(b[i], right + unit_at<U>(16 * ks + rt, 2 * (q + i) + ut));
          mma_row(acc, xl[ks], b);
          mma_row(acc, xh[ks], b);
          if constexpr (NI == 2) {
#pragma unroll
            for (int i = 0; i < 2; ++i) ldsm4t(b[i], right + Sh::TILE + unit_at<U>(16 * ks + rt, 2 * (q + i) + ut));
            mma_row(acc, xh[ks], b);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float(&d)[4] = D[2 * q + i];
          const float f = which ? 1.f : ec;
          d[0] = f * d[0] + acc[i][0] * z0.y;
          d[1] = f * d[1] + acc[i][1] * z0.y;
          d[2] = f * d[2] + acc[i][2] * z1.y;
          d[3] = f * d[3] + acc[i][3] * z1.y;
        }
      }
    }
    // the buffer may be refilled; a group's four warps add their sums
    if constexpr (Sh::STAGES == 1) __syncthreads();
    else if (c >= 2) bar_arrive(bar_empty(stage, group), GROUP + FILL);
    bar_sync(BAR_GROUP + group, GROUP);
    float *to = reinterpret_cast<float *>(ws + pl.off_dots) + (unit * 2 + slice * (WARPS / 4) + group) * DOT_FLOATS;
    const float *from = reinterpret_cast<const float *>(smem + Sh::S_DOTS) + group * 4 * DOT_FLOATS;
    for (int x = tid & (GROUP - 1); x < DOT_FLOATS; x += GROUP)
      to[x] = (from[x] + from[DOT_FLOATS + x]) + (from[2 * DOT_FLOATS + x] + from[3 * DOT_FLOATS + x]);
    if constexpr (Sh::STAGES == 1) __syncthreads();
  }

  if (io.d_initial) {
#pragma unroll
    for (int i = 0; i < NK; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        io.d_initial[s_off + (8 * i + t + (e & 1)) * sk + (v0 + g + (e >> 1) * 8) * sv] = D[i][e];
  }
}

// ---------------------------------------------------------------- chunks by themselves
// Sixteen warps: warp w has rows 16 (w % 4) .. of every product and quarter
// w / 4 of its columns; of the two pairs of [64, 64] products, half of q k^T
// with dO W^T or of k k^T with dY W^T.  The value heads of a key head take turns, dQ and dK stay
// in registers meanwhile.  A head takes 43 k cycles of an SM: loads and their
// conversion to pieces 12 k, products 16 k, elementwise work 6 k, the coefficients'
// tiles 4 k, the rest barriers; its 208 KB of shared memory leave no room for a
// second CTA or a second buffer.  With eight warps 3.20 ms.
constexpr int NT = 512;  // of the intra kernel

template <typename T, int DK, int DV> struct IntraShape {
  static constexpr int NI = pieces<T>();
  static constexpr int DH = NI == 1 ? DK : 64;  // key channels of S and dS' held at once
  static constexpr uint32_t KT = C * DK * 2, VT = C * DV * 2, ST = DV * DH * 2;
  static constexpr uint32_t S_K = 0, S_Q = NI * KT, S_W = 2 * NI * KT, S_DY = S_W + 2 * VT, S_DO = S_DY + 2 * VT,
                            S_S = S_DO + NI * VT, S_DS = S_S + 2 * ST, END = S_DS + NI * ST;
  // over S and dS' once these are used: the coefficients of k and q, then the pairs of dg
  static constexpr uint32_t S_T = S_S, S_X = S_T + 3 * NI * MAT_BYTES, END2 = S_X + C * C * 4;
  static constexpr uint32_t S_NUM = END > END2 ? END : END2, BYTES = S_NUM + 11 * C * 4 + 192;
};

template <int N> __device__ __forceinline__ void zero(float (&x)[N][4]) {
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) x[i][e] = 0.f;
}
// c[2 q + e] += a b[q] over pieces, NA of a and NB of b with the smallest
// products left out, for tile pairs q below n: one pair of pieces on all tiles in
// a row, so that no product waits for the sum of the one before.
template <int NA, int NB, int N, int Q>
__device__ __forceinline__ void mma_tiles(float (&c)[N][4], const uint32_t (&a)[NA][4], const uint32_t (&b)[Q][NB][4], int n = Q) {
  constexpr int M = NA > NB ? NA : NB;
#pragma unroll
  for (int s = M - 1; s >= 0; --s)
#pragma unroll
    for (int i = 0; i < NA; ++i)
      if (s - i >= 0 && s - i < NB)
#pragma unroll
        for (int q = 0; q < Q; ++q)
          if (q < n) {
            mma16(c[2 * q], a[i], b[q][s - i][0], b[q][s - i][1]);
            mma16(c[2 * q + 1], a[i], b[q][s - i][2], b[q][s - i][3]);
          }
}

template <typename T, int DK, int DV>
__global__ void __launch_bounds__(NT, 1)
gdn_intra_kernel(Problem p, char *ws, Plan pl, size_t kq_stride, size_t ap_stride, GradOut io, int sms) {
  using Sh = IntraShape<T, DK, DV>;
  constexpr int NI = Sh::NI, DH = Sh::DH, PASSES = DK / DH, NW = DH / 32;  // n-tiles of a warp in a pass
  constexpr int UK = DK / 8, UV = DV / 8, US = DH / 8;
  extern __shared__ __align__(128) unsigned char smem[];
  float *s_beta = reinterpret_cast<float *>(smem + Sh::S_NUM), *s_kn = s_beta + C, *s_qn = s_kn + C, *s_gh = s_qn + C,
        *s_gl = s_gh + C, *s_e = s_gl + C, *s_f = s_e + C, *s_iq = s_f + C /* [4][C] */,
        *s_db = s_e;  // [2][C], once e^G is used
  int *s_max = reinterpret_cast<int *>(s_iq + 4 * C);  // [3]
  float *s_z = s_iq + 4 * C + 4;                       // [16]
  uint8_t *s_do = reinterpret_cast<uint8_t *>(s_z + 16);  // [C]: exponents of d_out's units, a token's each
  auto unit_of = [&](int i) { return __uint_as_float((uint32_t)s_do[i] << 23); };
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, quarter = warp >> 2, half = quarter >> 1, side = quarter & 1;
  const int mt = side ? 3 - (warp & 3) : warp & 3;  // later rows have more to do: each scheduler gets early and late ones
  const int g = lane >> 2, t = (lane & 3) * 2;
  const int hk = (int)(blockIdx.x % p.Hk);
  const int64_t c = blockIdx.x / p.Hk;
  int n, len;
  int64_t batch, tok;
  if (!chunk_at(p.s, c, n, batch, tok, len)) return;
  const uint32_t base = smem_addr(smem);
  {
    const char *a = ws + pl.off_kq + (size_t)blockIdx.x * kq_stride;
    for (uint32_t x = tid * 16; x < 2 * NI * Sh::KT; x += NT * 16) cp16(base + x, a + x);
    cp_commit();
    cp_wait<0>();
  }
  const float scale = p.gp.scale;
  const int group = p.H / p.Hk;
  const int row0 = 16 * mt + g;  // this thread's rows: row0, row0 + 8
  const int ra = 16 * mt + (lane & 15), ua = lane >> 4;                                                 // left, rows as they are
  const int rat = ((lane >> 4) << 3) + (lane & 7), uat = 2 * mt + ((lane >> 3) & 1);                    // left, transposed
  const int rb = ((lane >> 4) << 3) + (lane & 7), ub = (lane >> 3) & 1;                                 // right, rows are columns
  const int rt = (((lane >> 3) & 1) << 3) + (lane & 7), ut = lane >> 4;                                 // right, transposed
  float dq[PASSES][NW][4], dk[PASSES][NW][4];
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    zero(dq[i]);
    zero(dk[i]);
  }
  const float *num = nullptr;

  for (int hv = 0; hv < group; ++hv) {
    const int h = hk * group + hv;
    const int64_t unit = c * p.H + h;
    __syncthreads();
    // ---- numbers, W, dY, dO
    num = reinterpret_cast<const float *>(ws + pl.off_ap + (size_t)unit * ap_stride);
    if (tid < C) {
      const float gh = num[NUM_GH + tid], gl = num[NUM_GL + tid];
      s_beta[tid] = num[NUM_BETA + tid];
      s_kn[tid] = num[NUM_K + tid];
      s_qn[tid] = num[NUM_Q + tid];
      s_gh[tid] = gh;
      s_gl[tid] = gl;
      s_e[tid] = exp2f(gh + gl);
      s_f[tid] = exp2f((num[NUM_GH + C - 1] - gh) + (num[NUM_GL + C - 1] - gl));
    }
    if (tid < 3) s_max[tid] = 0;
    float2 sc[4];  // S, dS', W, dY: one unit of pieces for the whole of each, eight lanes to find its largest
    {
      const float *m = reinterpret_cast<const float *>(ws + pl.off_max) + unit * MAX_FLOATS;
      float a = (lane & 7) < DV / 16 ? m[lane] : 0.f;
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) a = fmaxf(a, __shfl_xor_sync(~0u, a, o));
#pragma unroll
      for (int i = 0; i < 4; ++i) sc[i] = piece_scale(__shfl_sync(~0u, a, 8 * i));
    }
    // the states' first share on its way before the rest is worked on
    constexpr int ROUNDS = DV / 16 * US * 32 / NT, EARLY = ROUNDS < 4 ? ROUNDS : 4;
    float4 sv[EARLY], dv_[EARLY];
#pragma unroll
    for (int e = 0; e < EARLY; ++e) {
      const int x = tid + e * NT, from = (((x >> 5) / US) * UK + (x >> 5) % US) * 32 + (x & 31);
      sv[e] = reinterpret_cast<const float4 *>(ws + pl.off_s)[unit * (DV / 16) * UK * 32 + from];
      dv_[e] = reinterpret_cast<const float4 *>(ws + pl.off_ds)[unit * (DV / 16) * UK * 32 + from];
    }
    const T *o = static_cast<const T *>(io.d_out) + batch * p.v.b + tok * p.v.t + h * p.v.h;
    // bf16 rows of d_out as well; fp32 ones would take too many registers
    constexpr int OR = C * UV / NT;
    uint4 raw[OR];
    if constexpr (NI == 1) {
#pragma unroll
      for (int k = 0; k < OR; ++k) {
        const int x = tid + k * NT, r = x / UV, u = x % UV;
        raw[k] = r < len && io.d_out ? *reinterpret_cast<const uint4 *>(o + r * p.v.t + u * 8) : make_uint4(0, 0, 0, 0);
      }
    }
    {
      const float4 *w = reinterpret_cast<const float4 *>(ws + pl.off_w) + unit * (DV / 16) * 8 * 32;
      const float4 *y = reinterpret_cast<const float4 *>(ws + pl.off_dy) + unit * (DV / 16) * 8 * 32;
#pragma unroll 4
      for (int x = tid; x < DV / 16 * 8 * 32; x += NT) {
        const int l = x & 31, nt = (x >> 5) & 7, r = (x >> 8) * 16 + (l >> 2);
        const uint32_t at = unit_at<8>(r, nt) + (l & 3) * 4, at8 = unit_at<8>(r + 8, nt) + (l & 3) * 4;
        uint32_t hi, lo;
        const float4 a = w[x], b = y[x];
        split2(a.x * sc[2].x, a.y * sc[2].x, hi, lo);
        *reinterpret_cast<uint32_t *>(smem + Sh::S_W + at) = hi;
        *reinterpret_cast<uint32_t *>(smem + Sh::S_W + Sh::VT + at) = lo;
        split2(a.z * sc[2].x, a.w * sc[2].x, hi, lo);
        *reinterpret_cast<uint32_t *>(smem + Sh::S_W + at8) = hi;
        *reinterpret_cast<uint32_t *>(smem + Sh::S_W + Sh::VT + at8) = lo;
        split2(b.x * sc[3].x, b.y * sc[3].x, hi, lo);
        *reinterpret_cast<uint32_t *>(smem + Sh::S_DY + at) = hi;
        *reinterpret_cast<uint32_t *>(smem + Sh::S_DY + Sh::VT + at) = lo;
        split2(b.z * sc[3].x, b.w * sc[3].x, hi, lo);
        *reinterpret_cast<uint32_t *>(smem + Sh::S_DY + at8) = hi;
        *reinterpret_cast<uint32_t *>(smem + Sh::S_DY + Sh::VT + at8) = lo;
      }
#pragma unroll
      for (int k = 0; k < OR; ++k) {
        const int x = tid + k * NT, r = x / UV, u = x % UV;
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if constexpr (NI == 1) {
          const uint32_t w8[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w8[i] << 16);
            v[2 * i + 1] = __uint_as_float(w8[i] & 0xffff0000u);
          }
        } else if (r < len && io.d_out) {
          load8(o + r * p.v.t + u * 8, v);
        }
        // a token's row in a unit of its own: what is its own alone, dq, keeps its bits beside larger ones
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
#pragma unroll
        for (int o = 1; o < UV; o <<= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
        const float2 so = piece_scale(m);
        if (u == 0) s_do[r] = (uint8_t)(__float_as_uint(so.y) >> 23);
        uint4 hi, lo;
        split2(v[0] * so.x, v[1] * so.x, hi.x, lo.x);
        split2(v[2] * so.x, v[3] * so.x, hi.y, lo.y);
        split2(v[4] * so.x, v[5] * so.x, hi.z, lo.z);
        split2(v[6] * so.x, v[7] * so.x, hi.w, lo.w);
        *reinterpret_cast<uint4 *>(smem + Sh::S_DO + unit_at<UV>(r, u)) = hi;
        if constexpr (NI == 2) *reinterpret_cast<uint4 *>(smem + Sh::S_DO + Sh::VT + unit_at<UV>(r, u)) = lo;
      }
    }

    // the next head's share of memory on its way to L2: of this CTA, or of the one
    // that will take its place
    {
      const int64_t after = (int64_t)blockIdx.x + sms;
      const int64_t next = hv + 1 < group ? unit + 1 : after < gridDim.x ? after / p.Hk * p.H + after % p.Hk * group : -1;
      if (next >= 0) {
        constexpr int SB = DK * DV * 4, WB = C * DV * 4;
        for (int x = tid * 128; x < 2 * SB + 2 * WB; x += NT * 128) {
          const char *at = x < SB ? ws + pl.off_s + next * SB + x
                         : x < 2 * SB ? ws + pl.off_ds + next * SB + (x - SB)
                         : x < 2 * SB + WB ? ws + pl.off_w + next * WB + (x - 2 * SB) : ws + pl.off_dy + next * WB + (x - 2 * SB - WB);
          asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
        }
      }
    }

    // ---- what meets the states
    float zsum = 0.f, iq[2] = {0.f, 0.f};
#pragma unroll
    for (int pass = 0; pass < PASSES; ++pass) {
      if (pass) __syncthreads();
      {
        const float4 *s = reinterpret_cast<const float4 *>(ws + pl.off_s) + unit * (DV / 16) * UK * 32;
        const float4 *d = reinterpret_cast<const float4 *>(ws + pl.off_ds) + unit * (DV / 16) * UK * 32;
#pragma unroll
        for (int k = 0; k < ROUNDS; ++k) {
          const int x = tid + k * NT, l = x & 31, nt = (x >> 5) % US, w = (x >> 5) / US, r = w * 16 + (l >> 2);
          if (k >= EARLY || pass > 0) {
            if ((k - (pass ? 0 : EARLY)) % EARLY == 0) {
#pragma unroll
              for (int e = 0; e < EARLY; ++e)
                if (k + e < ROUNDS) {
                  const int x2 = x + e * NT, from2 = (((x2 >> 5) / US) * UK + pass * US + (x2 >> 5) % US) * 32 + l;
                  sv[e] = s[from2];
                  dv_[e] = d[from2];
                }
            }
          }
          const uint32_t at = unit_at<US>(r, nt) + (l & 3) * 4, at8 = unit_at<US>(r + 8, nt) + (l & 3) * 4;
          uint32_t hi, lo;
          const float4 a = sv[k % EARLY], b = dv_[k % EARLY];
          zsum += (a.x * b.x + a.y * b.y) + (a.z * b.z + a.w * b.w);
          split2(a.x * sc[0].x, a.y * sc[0].x, hi, lo);
          *reinterpret_cast<uint32_t *>(smem + Sh::S_S + at) = hi;
          *reinterpret_cast<uint32_t *>(smem + Sh::S_S + Sh::ST + at) = lo;
          split2(a.z * sc[0].x, a.w * sc[0].x, hi, lo);
          *reinterpret_cast<uint32_t *>(smem + Sh::S_S + at8) = hi;
          *reinterpret_cast<uint32_t *>(smem + Sh::S_S + Sh::ST + at8) = lo;
          split2(b.x * sc[1].x, b.y * sc[1].x, hi, lo);
          *reinterpret_cast<uint32_t *>(smem + Sh::S_DS + at) = hi;
          if constexpr (NI == 2) *reinterpret_cast<uint32_t *>(smem + Sh::S_DS + Sh::ST + at) = lo;
          split2(b.z * sc[1].x, b.w * sc[1].x, hi, lo);
          *reinterpret_cast<uint32_t *>(smem + Sh::S_DS + at8) = hi;
          if constexpr (NI == 2) *reinterpret_cast<uint32_t *>(smem + Sh::S_DS + Sh::ST + at8) = lo;
        }
      }
      __syncthreads();
      float x[NW][4], y[NW][4];
      zero(x);
      zero(y);
#pragma unroll 2
      for (int ks = 0; ks < DV / 16; ++ks) {  // dO S, dY S
        uint32_t o[NI][4], r[NI][4];
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          ldsm4(o[i], base + Sh::S_DO + i * Sh::VT + unit_at<UV>(ra, 2 * ks + ua));
          ldsm4t(r[i], base + Sh::S_DY + i * Sh::VT + unit_at<8>(16 * ks + rat, uat));
        }
        uint32_t b[NW / 2][2][4];
#pragma unroll
        for (int q = 0; q < NW / 2; ++q)
#pragma unroll
          for (int i = 0; i < 2; ++i) ldsm4t(b[q][i], base + Sh::S_S + i * Sh::ST + unit_at<US>(16 * ks + rt, quarter * NW + 2 * q + ut));
        mma_tiles<NI, 2>(x, o, b);
        if constexpr (NI == 2) {
          mma_tiles<2, 2>(y, r, b);
        } else {
#pragma unroll
          for (int q = 0; q < NW / 2; ++q) {
            mma16(y[2 * q], r[0], b[q][0][0], b[q][0][1]);
            mma16(y[2 * q + 1], r[0], b[q][0][2], b[q][0][3]);
          }
        }
      }
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        const int i = row0 + 8 * rr;
        const float eq = s_e[i] * scale, ek = s_e[i] * s_beta[i], un = unit_of(i);
#pragma unroll
        for (int nt = 0; nt < NW; ++nt) {
          const uint32_t at = unit_at<UK>(i, pass * US + quarter * NW + nt) + t * 2;
          float2 q = __half22float2(*reinterpret_cast<const __half2 *>(smem + Sh::S_Q + at));
          if constexpr (NI == 2) {
            const float2 ql = __half22float2(*reinterpret_cast<const __half2 *>(smem + Sh::S_Q + Sh::KT + at));
            q.x += ql.x;
            q.y += ql.y;
          }
          const float a = x[nt][2 * rr] * un * sc[0].y, b = x[nt][2 * rr + 1] * un * sc[0].y;
          iq[rr] = fmaf(a, q.x, fmaf(b, q.y, iq[rr]));
          dq[pass][nt][2 * rr] = fmaf(eq, a, dq[pass][nt][2 * rr]);
          dq[pass][nt][2 * rr + 1] = fmaf(eq, b, dq[pass][nt][2 * rr + 1]);
          dk[pass][nt][2 * rr] -= ek * (y[nt][2 * rr] * sc[3].y * sc[0].y);
          dk[pass][nt][2 * rr + 1] -= ek * (y[nt][2 * rr + 1] * sc[3].y * sc[0].y);
        }
      }
      zero(x);
#pragma unroll 2
      for (int ks = 0; ks < DV / 16; ++ks) {  // W dS'
        uint32_t w[NI][4];
#pragma unroll
        for (int i = 0; i < NI; ++i) ldsm4t(w[i], base + Sh::S_W + i * Sh::VT + unit_at<8>(16 * ks + rat, uat));
        uint32_t b[NW / 2][NI][4];
#pragma unroll
        for (int q = 0; q < NW / 2; ++q)
#pragma unroll
          for (int i = 0; i < NI; ++i) ldsm4t(b[q][i], base + Sh::S_DS + i * Sh::ST + unit_at<US>(16 * ks + rt, quarter * NW + 2 * q + ut));
        mma_tiles<NI, NI>(x, w, b);
      }
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        const float f = s_f[row0 + 8 * rr];
#pragma unroll
        for (int nt = 0; nt < NW; ++nt) {
          dk[pass][nt][2 * rr] += f * (x[nt][2 * rr] * sc[2].y * sc[1].y);
          dk[pass][nt][2 * rr + 1] += f * (x[nt][2 * rr + 1] * sc[2].y * sc[1].y);
        }
      }
    }
#pragma unroll
    for (int rr = 0; rr < 2; ++rr) {
      iq[rr] += __shfl_xor_sync(~0u, iq[rr], 1);
      iq[rr] += __shfl_xor_sync(~0u, iq[rr], 2);
      if ((lane & 3) == 0) s_iq[quarter * C + row0 + 8 * rr] = iq[rr] * s_e[row0 + 8 * rr] * s_qn[row0 + 8 * rr] * scale;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) zsum += __shfl_xor_sync(~0u, zsum, o);
    if (lane == 0) s_z[warp] = zsum;

    // ---- inside the chunk: half 0 has q k^T and dP, half 1 k k^T and dL
    const int pairs = mt < side ? 0 : mt < side + 2 ? 1 : 2;  // down to the diagonal
    float x[4][4], m[4][4];  // tile pairs `side` and `side` + 2
    zero(x);
    zero(m);
#pragma unroll 2
    for (int ks = 0; ks < DK / 16; ++ks) {
      uint32_t a[NI][4];
#pragma unroll
      for (int i = 0; i < NI; ++i) ldsm4(a[i], base + (half ? Sh::S_K : Sh::S_Q) + i * Sh::KT + unit_at<UK>(ra, 2 * ks + ua));
      uint32_t b[2][NI][4];
#pragma unroll
      for (int qi = 0; qi < 2; ++qi)
        if (qi < pairs)
#pragma unroll
          for (int i = 0; i < NI; ++i) ldsm4(b[qi][i], base + Sh::S_K + i * Sh::KT + unit_at<UK>(16 * (side + 2 * qi) + rb, 2 * ks + ub));
      mma_tiles<NI, NI>(x, a, b, pairs);
    }
#pragma unroll 2
    for (int ks = 0; ks < DV / 16; ++ks) {
      uint32_t a[2][4];
      if (half) {
#pragma unroll
        for (int i = 0; i < 2; ++i) ldsm4t(a[i], base + Sh::S_DY + i * Sh::VT + unit_at<8>(16 * ks + rat, uat));
      } else {
#pragma unroll
        for (int i = 0; i < NI; ++i) ldsm4(a[i], base + Sh::S_DO + i * Sh::VT + unit_at<UV>(ra, 2 * ks + ua));
      }
      uint32_t b[2][2][4];
#pragma unroll
      for (int qi = 0; qi < 2; ++qi)
        if (qi < pairs)
#pragma unroll
          for (int i = 0; i < 2; ++i) ldsm4t(b[qi][i], base + Sh::S_W + i * Sh::VT + unit_at<8>(16 * ks + rt, 2 * (side + 2 * qi) + ut));
      if (NI == 2 || half) {
        mma_tiles<2, 2>(m, a, b, pairs);
      } else {
        const uint32_t one[1][4] = {{a[0][0], a[0][1], a[0][2], a[0][3]}};
        mma_tiles<1, 2>(m, one, b, pairs);
      }
    }
    auto col_of = [&](int nt) { return 16 * (side + (nt & 2)) + 8 * (nt & 1) + t; };
    float db[2] = {0.f, 0.f}, top0 = 0.f, top1 = 0.f;
    const float un[2] = {half ? -sc[3].y : unit_of(row0), half ? -sc[3].y : unit_of(row0 + 8)};
#pragma unroll
    for (int nt = 0; nt < 4; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = row0 + 8 * (e >> 1), j = col_of(nt) + (e & 1);
        float mv = 0.f, xv = 0.f;
        if (half ? j < i : j <= i) {
          const float gam = exp2_neg((s_gh[i] - s_gh[j]) + (s_gl[i] - s_gl[j]));
          mv = m[nt][e] * sc[2].y * gam;  // dP in d_out's units
          if (half) {
            mv *= un[e >> 1];
            const float kk = x[nt][e] * s_kn[i] * s_kn[j];
            db[e >> 1] = fmaf(mv, kk, db[e >> 1]);
            mv *= s_beta[i];
            xv = mv * kk;
            top0 = fmaxf(top0, fmaxf(fabsf(mv * s_kn[j]), fabsf(mv * s_kn[i])));
          } else {
            xv = mv * un[e >> 1] * (x[nt][e] * s_qn[i] * s_kn[j] * scale);
            top0 = fmaxf(top0, fabsf(mv * s_kn[j]));
            top1 = fmaxf(top1, fabsf(mv * un[e >> 1] * s_qn[i]));
          }
        }
        m[nt][e] = mv;
        x[nt][e] = xv;
      }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      top0 = fmaxf(top0, __shfl_xor_sync(~0u, top0, o));
      top1 = fmaxf(top1, __shfl_xor_sync(~0u, top1, o));
    }
    if (lane == 0) {
      atomicMax(&s_max[half ? 2 : 0], __float_as_int(top0));
      if (!half) atomicMax(&s_max[1], __float_as_int(top1));
    }
    __syncthreads();  // the states' place is free, the largest values are known
    if (half) {
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        db[rr] += __shfl_xor_sync(~0u, db[rr], 1);
        db[rr] += __shfl_xor_sync(~0u, db[rr], 2);
        if ((lane & 3) == 0) s_db[side * C + row0 + 8 * rr] = db[rr];
      }
    }
    const float2 s1 = piece_scale(__int_as_float(s_max[0])), s2 = piece_scale(__int_as_float(s_max[1])),
                 s3 = piece_scale(__int_as_float(s_max[2]));
    auto put = [&](int which, int i, int j, float v) {  // one element of a tile
      const __half hi = __float2half_rn(v);
      const uint32_t at = Sh::S_T + which * NI * MAT_BYTES + unit_at<8>(i, j >> 3) + (j & 7) * 2;
      *reinterpret_cast<__half *>(smem + at) = hi;
      if constexpr (NI == 2) *reinterpret_cast<__half *>(smem + at + MAT_BYTES) = __float2half_rn(v - __half2float(hi));
    };
    auto put2 = [&](int which, int i, int j, float v, float w) {  // two of a row, j even
      uint32_t hi, lo;
      split2(v, w, hi, lo);
      const uint32_t at = Sh::S_T + which * NI * MAT_BYTES + unit_at<8>(i, j >> 3) + (j & 7) * 2;
      *reinterpret_cast<uint32_t *>(smem + at) = hi;
      if constexpr (NI == 2) *reinterpret_cast<uint32_t *>(smem + at + MAT_BYTES) = lo;
    };
    float *Xs = reinterpret_cast<float *>(smem + Sh::S_X);
    auto x_at = [&](int i, int j) -> float & { return Xs[i * C + (j ^ (i & 31))]; };
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
      if (side + (nt & 2) > mt) continue;
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const int i = row0 + 4 * e, j = col_of(nt);
        const float mv = m[nt][e], mw = m[nt][e + 1];
        if (half) {
          // M + M^T times k's factors: its own pair in a block below the diagonal blocks, one by one in these
          const float kj = s_kn[j] * s3.x, kw = s_kn[j + 1] * s3.x, ki = s_kn[i] * s3.x;
          if (side + (nt & 2) < mt) {
            put2(2, i, j, mv * kj, mw * kw);
          } else {
            if (j <= i) put(2, i, j, mv * kj);  // zero on the diagonal
            if (j + 1 <= i) put(2, i, j + 1, mw * kw);
          }
          if (j < i) put(2, j, i, mv * ki);
          if (j + 1 < i) put(2, j + 1, i, mw * ki);
        } else {
          const float qi = s_qn[i] * s2.x, ui = un[e >> 1];
          put2(0, i, j, mv * (s_kn[j] * s1.x), mw * (s_kn[j + 1] * s1.x));
          put2(1, i, j, mv * ui * qi, mw * ui * qi);
          x_at(i, j) = x[nt][e];
          x_at(i, j + 1) = x[nt][e + 1];
        }
      }
    }
    __syncthreads();
    if (half) {
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
        if (side + (nt & 2) > mt) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) x_at(row0 + 8 * (e >> 1), col_of(nt) + (e & 1)) += x[nt][e];
      }
    }
    // dQ += dP.. k, dK += (dP..)^T q + (M + M^T) k
    const float ud[2] = {unit_of(row0), unit_of(row0 + 8)};
#pragma unroll
    for (int pass = 0; pass < PASSES; ++pass) {
      float a[NW][4], b[NW][4], d[NW][4];
      zero(a);
      zero(b);
      zero(d);
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        uint32_t l1[NI][4], l2[NI][4], l3[NI][4];
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          if (ks <= mt) ldsm4(l1[i], base + Sh::S_T + i * MAT_BYTES + unit_at<8>(ra, 2 * ks + ua));
          if (ks >= mt) ldsm4t(l2[i], base + Sh::S_T + (NI + i) * MAT_BYTES + unit_at<8>(16 * ks + rat, uat));
          ldsm4(l3[i], base + Sh::S_T + (2 * NI + i) * MAT_BYTES + unit_at<8>(ra, 2 * ks + ua));
        }
        uint32_t r[NW / 2][NI][4];
#pragma unroll
        for (int q = 0; q < NW / 2; ++q)
#pragma unroll
          for (int i = 0; i < NI; ++i)
            ldsm4t(r[q][i], base + Sh::S_K + i * Sh::KT + unit_at<UK>(16 * ks + rt, pass * US + quarter * NW + 2 * q + ut));
        if (ks <= mt) mma_tiles<NI, NI>(a, l1, r);
        mma_tiles<NI, NI>(d, l3, r);
        if (ks >= mt) {
#pragma unroll
          for (int q = 0; q < NW / 2; ++q)
#pragma unroll
            for (int i = 0; i < NI; ++i)
              ldsm4t(r[q][i], base + Sh::S_Q + i * Sh::KT + unit_at<UK>(16 * ks + rt, pass * US + quarter * NW + 2 * q + ut));
          mma_tiles<NI, NI>(b, l2, r);
        }
      }
#pragma unroll
      for (int nt = 0; nt < NW; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          dq[pass][nt][e] = fmaf(scale, a[nt][e] * s1.y * ud[e >> 1], dq[pass][nt][e]);
          dk[pass][nt][e] += scale * (b[nt][e] * s2.y) + d[nt][e] * s3.y;
        }
    }
    // what the last step wants from memory, on its way meanwhile
    float I[2], Y[2], B[2], xg[2], alog = 0.f, bias = 0.f, ec = 0.f;
    const int64_t g_off = batch * p.gate.b + tok * p.gate.t + h * p.gate.h;
    if (warp == 0) {
      const float *sums = reinterpret_cast<const float *>(ws + pl.off_dots) + unit * 2 * DOT_FLOATS;
      auto dots = [&](int at) { return DV == 128 ? sums[at] + sums[DOT_FLOATS + at] : sums[at]; };
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 2 * lane + i;
        I[i] = dots(DOT_K + r);
        Y[i] = dots(DOT_Y + r);
        B[i] = dots(DOT_BETA + r);
        xg[i] = r < len ? p.g[g_off + r * p.gate.t] : 0.f;
      }
      if (p.gp.flags & KDA_GATE_IN_KERNEL) alog = p.gp.a_log[h];
      if (p.gp.dt_bias) bias = p.gp.dt_bias[h];
      ec = num[NUM_MISC];
    }
    __syncthreads();
    // sums over i >= r of the pairs, in place: first within eight rows, a thread a column
    float *s_tot = reinterpret_cast<float *>(smem + Sh::S_T), *s_pairs = s_tot + NT;  // over the coefficients
    {
      const int j = tid & (C - 1), seg = tid / C;
      float sum = 0.f;
#pragma unroll
      for (int i = 8 * seg + 7; i >= 8 * seg; --i) {
        if (i > j) sum += x_at(i, j);
        x_at(i, j) = sum;
      }
      s_tot[tid] = sum;
    }
    __syncthreads();
    // then over j < r, eight lanes a row, with the totals of the later rows
    {
      const int r = tid >> 3;
      float sum = 0.f;
      for (int j = tid & 7; j < r; j += 8) {
        sum += x_at(r, j);
        for (int seg = r / 8 + 1; seg < 8; ++seg) sum += s_tot[seg * C + j];
      }
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(~0u, sum, o);
      if ((tid & 7) == 0) s_pairs[r] = sum;
    }
    __syncthreads();
    if (warp == 0) {
      float F[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 2 * lane + i;
        F[i] = s_pairs[r];
        I[i] += (s_iq[r] + s_iq[C + r]) + (s_iq[2 * C + r] + s_iq[3 * C + r]);
      }
      float si = I[0] + I[1], sy = Y[0] + Y[1];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float a = __shfl_down_sync(~0u, si, o), b = __shfl_up_sync(~0u, sy, o);
        if (lane + o < 32) si += a;
        if (lane >= o) sy += b;
      }
      float before = __shfl_up_sync(~0u, sy, 1), after = __shfl_down_sync(~0u, si, 1);
      if (lane == 0) before = 0.f;
      if (lane == 31) after = 0.f;
      float z = 0.f;
#pragma unroll
      for (int w = 0; w < NT / 32; ++w) z += s_z[w];
      z *= ec;
      const float dg[2] = {F[0] + si + before + z, F[1] + (I[1] + after) + (before + Y[0]) + z};
      const bool gate = (p.gp.flags & KDA_GATE_IN_KERNEL) != 0;
      const float ea = gate ? expf(alog) : 0.f;
      float da = 0.f, dt = 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 2 * lane + i;
        if (r < len) {
          const float be = s_beta[r];
          float dx = dg[i];
          if (gate) {
            da = fmaf(log_decay(xg[i], p.gp, -ea, bias), dg[i], da);
            dx = -ea * dg[i] / (1.f + expf(-(xg[i] + bias)));
            dt += dx;
          }
          io.dg[g_off + r * p.gate.t] = dx;
          float d = B[i] + (s_db[r] + s_db[C + r]);
          if (p.gp.flags & KDA_BETA_SIGMOID) d *= be * (1.f - be);
          io.dbeta[g_off + r * p.gate.t] = d;
        }
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        da += __shfl_xor_sync(~0u, da, o);
        dt += __shfl_xor_sync(~0u, dt, o);
      }
      if (lane == 0) reinterpret_cast<float2 *>(ws + pl.off_part)[unit] = make_float2(da, dt);
    }
  }

  // ---- through the norms: dx = r (dx^ - x^ (x^.dx^)), x^ = r x
  const bool l2 = (p.gp.flags & KDA_L2NORM_QK) != 0;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    auto &d = which ? dk : dq;
    const uint32_t tile = which ? Sh::S_K : Sh::S_Q;
    float dot[2] = {0.f, 0.f};
    auto hat = [&](int pass, int nt, int rr) {  // two values of x^, without the unit's factor
      const uint32_t at = unit_at<UK>(row0 + 8 * rr, pass * US + quarter * NW + nt) + t * 2;
      float2 v = __half22float2(*reinterpret_cast<const __half2 *>(smem + tile + at));
      if constexpr (NI == 2) {
        const float2 l = __half22float2(*reinterpret_cast<const __half2 *>(smem + tile + Sh::KT + at));
        v.x += l.x;
        v.y += l.y;
      }
      return v;
    };
    if (l2) {
#pragma unroll
      for (int pass = 0; pass < PASSES; ++pass)
#pragma unroll
        for (int nt = 0; nt < NW; ++nt)
#pragma unroll
          for (int rr = 0; rr < 2; ++rr) {
            const float2 v = hat(pass, nt, rr);
            dot[rr] = fmaf(v.x, d[pass][nt][2 * rr], fmaf(v.y, d[pass][nt][2 * rr + 1], dot[rr]));
          }
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        dot[rr] += __shfl_xor_sync(~0u, dot[rr], 1);
        dot[rr] += __shfl_xor_sync(~0u, dot[rr], 2);
      }
      __syncthreads();
      if ((lane & 3) == 0) {
        s_iq[quarter * C + row0] = dot[0];
        s_iq[quarter * C + row0 + 8] = dot[1];
      }
      __syncthreads();
    }
    T *out = static_cast<T *>(which ? io.dk : io.dq) + batch * p.qk.b + tok * p.qk.t + hk * p.qk.h;
#pragma unroll
    for (int rr = 0; rr < 2; ++rr) {
      const int i = row0 + 8 * rr;
      if (i >= len) continue;
      const float xn = which ? s_kn[i] : s_qn[i], r = num[(which ? NUM_RK : NUM_RQ) + i];
      const float full = l2 ? ((s_iq[i] + s_iq[C + i]) + (s_iq[2 * C + i] + s_iq[3 * C + i])) * xn * xn : 0.f;
#pragma unroll
      for (int pass = 0; pass < PASSES; ++pass)
#pragma unroll
        for (int nt = 0; nt < NW; ++nt) {
          float a = d[pass][nt][2 * rr], b = d[pass][nt][2 * rr + 1];
          if (l2) {
            const float2 v = hat(pass, nt, rr);
            a = r * (a - v.x * full);
            b = r * (b - v.y * full);
          }
          T *to = out + i * p.qk.t + pass * DH + quarter * NW * 8 + nt * 8 + t;
          if constexpr (NI == 1) *reinterpret_cast<__nv_bfloat162 *>(to) = __floats2bfloat162_rn(a, b);
          else *reinterpret_cast<float2 *>(to) = make_float2(a, b);
        }
    }
  }
}

// a_log's and dt_bias's gradients: the chunks' sums in a fixed order, a warp a head.
__global__ void __launch_bounds__(32) gdn_param_kernel(Problem p, const float2 *part, float *da_log, float *ddt_bias) {
  const int h = blockIdx.x, lane = threadIdx.x;
  const bool gate = (p.gp.flags & KDA_GATE_IN_KERNEL) != 0;
  const int64_t n = !gate ? 0 : p.s.bounds ? min((int64_t)p.s.chunk_off[p.s.N], (int64_t)p.nchunks) : p.nchunks;
  float a = 0.f, b = 0.f;
  for (int64_t c = lane; c < n; c += 32) {
    const float2 x = part[c * p.H + h];
    a += x.x;
    b += x.y;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    a += __shfl_xor_sync(~0u, a, o);
    b += __shfl_xor_sync(~0u, b, o);
  }
  if (lane == 0) {
    if (da_log) da_log[h] = a;
    if (ddt_bias) ddt_bias[h] = b;
  }
}

template <typename T, int DK, int WARPS>
cudaError_t go_reverse(const Problem &p, char *ws, const Plan &pl, const GradOut &io, cudaStream_t st) {
  const kda_dtype dt = sizeof(T) == 2 ? KDA_BF16 : KDA_F32;
  auto kernel = gdn_reverse_kernel<T, DK, WARPS>;
  constexpr int smem = RevShape<T, DK, WARPS>::BYTES;
  static_assert(smem <= 232448, "shared memory of a CTA");
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int64_t grid = (int64_t)p.s.N * p.H * (p.dv / (16 * WARPS));
  kernel<<<(unsigned)grid, RevShape<T, DK, WARPS>::THREADS, smem, st>>>(p, ws, pl, kq_bytes(dt, p.dk), ap_bytes(dt, true), io);
  return cudaGetLastError();
}

template <typename T, int DK, int DV> cudaError_t go(const Problem &p, char *ws, const Plan &pl, const GradOut &io, cudaStream_t st) {
  const kda_dtype dt = sizeof(T) == 2 ? KDA_BF16 : KDA_F32;
  const size_t kqs = kq_bytes(dt, p.dk), aps = ap_bytes(dt, true);
  auto intra = gdn_intra_kernel<T, DK, DV>;
  constexpr int in_smem = IntraShape<T, DK, DV>::BYTES;
  static_assert(in_smem <= 232448, "shared memory of a CTA");
  cudaError_t e = DV == 128 && !p.halves ? go_reverse<T, DK, 8>(p, ws, pl, io, st) : go_reverse<T, DK, 4>(p, ws, pl, io, st);
  if (e != cudaSuccess) return e;
  if ((e = cudaFuncSetAttribute(intra, cudaFuncAttributeMaxDynamicSharedMemorySize, in_smem)) != cudaSuccess) return e;
  if (p.nchunks > 0) {
    int dev = 0, sms = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess || (e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
      return e;
    intra<<<(unsigned)((int64_t)p.nchunks * p.Hk), NT, in_smem, st>>>(p, ws, pl, kqs, aps, io, sms);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if (io.da_log || io.ddt_bias)
    gdn_param_kernel<<<p.H, 32, 0, st>>>(p, reinterpret_cast<const float2 *>(ws + pl.off_part), io.da_log, io.ddt_bias);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gdn_bwd(kda_dtype dt, const Problem &p, char *ws, const Plan &pl, const GradOut &io, cudaStream_t st) {
  const bool w = p.dk == 128;
#define GDN_GO(T_)                                                                                              \
  if (p.dv == 128) return w ? go<T_, 128, 128>(p, ws, pl, io, st) : go<T_, 64, 128>(p, ws, pl, io, st);         \
  return w ? go<T_, 128, 64>(p, ws, pl, io, st) : go<T_, 64, 64>(p, ws, pl, io, st)
  if (dt == KDA_BF16) { GDN_GO(__nv_bfloat16); }
  GDN_GO(float);
#undef GDN_GO
}

}  // namespace gdn
}  // namespace kda
