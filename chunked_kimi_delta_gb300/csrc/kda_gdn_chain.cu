// kda_gdn_chain.cu - from chunk to chunk: the state, the corrected values and
// the outputs of the gated delta rule with one gate per head (kda_gdn.cuh).
//
// A value channel's column of the state never meets another one, so a warp
// takes 16 of them and walks the chunks alone: it holds S^T [16, dk] in the
// accumulator layout of the tensor-core instruction, which is at once (rounded
// to pieces) the layout of a left operand, and so do Y^T and W^T, its
// intermediates.  Nothing of the recurrence passes through shared memory; that
// holds only what the warps of a CTA read in common (k, q, A, P of the chunk),
// twice where it fits, filled by warps of their own.
//
// 4 x 8192 tokens of 32 heads on 16 key heads, d = 128, bf16: 668 us, 10.2 k cycles a
// chunk.  What bounds it: 400 tensor-core products a warp and chunk, two warps
// a scheduler at 8 cycles each, 6.4 k cycles, covered only in part by the other
// warp's elementwise work.  With the computing warps copying and a barrier for
// all after every chunk 774 us.  Half the value channels a CTA shorten a chunk
// where chains are few (130 tokens of 2 heads: 21.9 -> 13.9 us).
#include "kda_gdn.cuh"

namespace kda {
namespace gdn {
namespace {

template <typename T, int DK, int WARPS, bool STORE> struct Shape {
  static constexpr int NI = pieces<T>(), NP = STORE ? 2 : NI;
  static constexpr uint32_t TILE = C * DK * 2;
  static constexpr uint32_t S_K = 0, S_Q = NI * TILE, S_NUM = 2 * NI * TILE, S_A = S_NUM + NUM_BYTES,
                            S_P = S_A + 2 * MAT_BYTES, S_V = S_P + NP * MAT_BYTES;
  static constexpr uint32_t V_STRIP = C * 16 * sizeof(T);
  static constexpr uint32_t STAGE = (S_V + WARPS * V_STRIP + 127) / 128 * 128;
  static constexpr int STAGES = 2 * STAGE + (NI == 1 ? WARPS * V_STRIP : 0) <= 232448 ? 2 : 1;  // fp32 of 128 key channels: one
  static constexpr int THREADS = WARPS * 32 + (STAGES == 2 ? FILL : 0);
  static constexpr uint32_t S_OUT = STAGES * STAGE;  // a strip a warp, bf16 only
  static constexpr uint32_t BYTES = S_OUT + (NI == 1 && !STORE ? WARPS * V_STRIP : 0);
};

template <typename T, int DK, int WARPS, bool STORE>
__global__ void __launch_bounds__(Shape<T, DK, WARPS, STORE>::THREADS, 1)
gdn_chain_kernel(Problem p, char *ws, Plan pl, size_t kq_stride, size_t ap_stride, ChainOut io) {
  using Sh = Shape<T, DK, WARPS, STORE>;
  constexpr int NI = Sh::NI, U = DK / 8, NK = DK / 8;
  extern __shared__ __align__(128) unsigned char smem[];
  const char *kq = ws + pl.off_kq, *ap = ws + pl.off_ap;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = (lane & 3) * 2;
  const int slices = p.dv / (16 * WARPS);
  const int slice = blockIdx.x % slices;
  const int h = (int)(blockIdx.x / slices % p.H);
  const int at = (int)(blockIdx.x / slices / p.H), n = p.order ? p.order[at] : at;
  const int hk = h / (p.H / p.Hk);
  const int v0 = (slice * WARPS + warp) * 16;  // this warp's first value channel
  int64_t t0, t1;
  seq_range(p.s, n, t0, t1);
  const int64_t c0 = seq_first_chunk(p.s, n);
  // offsets that overlap (a broken cu_seqlens) could ask for more chunks than there are
  const int nc = (int)max((int64_t)0, min((t1 - t0 + C - 1) / C, p.nchunks - c0));
  const int64_t batch = p.s.bounds ? 0 : n, tok = p.s.bounds ? t0 : 0;
  const int64_t v_off = batch * p.v.b + tok * p.v.t + h * p.v.h + v0;
  const T *v = static_cast<const T *>(p.val) + v_off;
  T *out = STORE ? nullptr : static_cast<T *>(io.out) + v_off;

  const uint32_t base = smem_addr(smem);
  const uint32_t kq_part = STORE ? Sh::S_Q : Sh::S_NUM, ap_part = (STORE ? Sh::S_P : Sh::S_V) - Sh::S_NUM;  // q and P are for o alone
  auto load = [&](int c, uint32_t stage, uint32_t first, uint32_t step) {
    const char *a = kq + ((size_t)(c0 + c) * p.Hk + hk) * kq_stride, *b = ap + ((size_t)(c0 + c) * p.H + h) * ap_stride;
#pragma unroll 4
    for (uint32_t x = first; x < kq_part; x += step) cp16(stage + Sh::S_K + x, a + x);
#pragma unroll 4
    for (uint32_t x = first; x < ap_part; x += step) cp16(stage + Sh::S_NUM + x, b + x);
  };
  if constexpr (Sh::STAGES == 2) {
    if (warp >= WARPS) {
      registers_to_fill<WARPS>();
      const int first = tid - WARPS * 32;
      const T *vs = v - warp * 16;
      fill_buffers<WARPS / 4>(nc, [&](int c) {
        const uint32_t stage = base + (c & 1) * Sh::STAGE;
        load(c, stage, first * 16, FILL * 16);
        load_strips<WARPS>(stage + Sh::S_V, vs + (int64_t)c * C * p.v.t, p.v.t, t1 - t0 - (int64_t)c * C, first);
      });
      return;
    }
    registers_to_compute<WARPS>();
  }
  const int group = warp >> 2;

  // S^T: channel of k along the columns.  (row, column) of a state in memory
  const int64_t s_off = ((int64_t)n * p.H + h) * DK * p.dv;
  const int64_t sk = p.v_first ? 1 : p.dv, sv = p.v_first ? DK : 1;
  float S[NK][4];
#pragma unroll
  for (int i = 0; i < NK; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      S[i][e] = io.initial ? io.initial[s_off + (8 * i + t + (e & 1)) * sk + (v0 + g + (e >> 1) * 8) * sv] : 0.f;

  const int rb = ((lane >> 4) << 3) + (lane & 7), ub = (lane >> 3) & 1;  // right operand, rows are its columns
  const int rt = (((lane >> 3) & 1) << 3) + (lane & 7), ut = lane >> 4;  // right operand, transposed on the way
  // Started together the groups stay in step and then wait for the same unit at a time, so the second one starts when
  // the first has W of its first chunk (storing: Y), half (a quarter) of a chunk later.  Together / so / with the first
  // chunk done, whole calls on 4 sequences of 32 heads, us:
  //   forward,   128 chunks  bf16 128 x 128 1006 / 966 / 973   bf16 64 x 128 726 / 715 / 717   fp32 64 x 128 955 / 983 / 998
  //               16 chunks                  140 / 135 / 135                 103 / 99 / 101                  137 / 135 / 137
  //   gradients, 128 chunks                 4666 / 4541 / 4662              3296 / 3275 / 3307              4410 / 4329 / 4437
  //               16 chunks                  632 / 615 / 619                 448 / 442 / 451                 590 / 581 / 592
  // One chunk alone gains nothing from it.
  const bool apart = Sh::STAGES == 2 && WARPS == 8 && nc > 1;
  if (apart && group == 1) bar_sync(BAR_START, 2 * GROUP);
  auto start_second = [&](int c) {
    if (apart && group == 0 && c == 0) bar_arrive(BAR_START, 2 * GROUP);
  };
  for (int c = 0; c < nc; ++c) {
    const uint32_t st = base + (Sh::STAGES == 2 ? (c & 1) * Sh::STAGE : 0);
    if constexpr (Sh::STAGES == 2) {
      bar_sync(bar_full(c & 1, group), GROUP + FILL);
    } else {
      load(c, st, tid * 16, WARPS * 512);
      const uint32_t strip = st + Sh::S_V + warp * Sh::V_STRIP;
#pragma unroll
      for (int x = lane; x < C * 4; x += 32) {
        const int64_t r = (int64_t)c * C + x / 4;
        const bool in = r < t1 - t0;
        cp16z(strip + x * 16, v + (in ? r * p.v.t : 0) + x % 4 * 4, in);
      }
      cp_commit();
      cp_wait<0>();
      __syncthreads();
    }
    const float *num = reinterpret_cast<const float *>(smem + (st - base) + Sh::S_NUM);

    // ---- S^T k^T and S^T q^T
    float2 z0, z1;
    row_scales(S, z0, z1);
    const int64_t unit = (c0 + c) * p.H + h;  // of what the backward is handed
    auto keep = [&](size_t off, const auto &x, int n, float top, int which) {
      float4 *to = reinterpret_cast<float4 *>(ws + off) + (unit * (p.dv / 16) + v0 / 16) * n * 32 + lane;
#pragma unroll
      for (int i = 0; i < (int)(sizeof(x) / 16); ++i) to[i * 32] = make_float4(x[i][0], x[i][1], x[i][2], x[i][3]);
      if (which >= 0 && lane == 0) reinterpret_cast<float *>(ws + pl.off_max)[unit * MAX_FLOATS + which + v0 / 16] = top;
    };
    if constexpr (STORE) keep(pl.off_s, S, NK, warp_max(S), MAX_S);
    float Y[8][4], O[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) Y[i][e] = O[i][e] = 0.f;
#pragma unroll
    for (int ks = 0; ks < DK / 16; ++ks) {
      uint32_t ah[4], al[4];
      as_left(S, ks, z0.x, z1.x, ah, al);
      // eight products of one kind in a row: none waits for the sum of the one before
      uint32_t b[4][4];
#pragma unroll
      for (int q = 0; q < 4; ++q) ldsm4(b[q], st + Sh::S_K + unit_at<U>(16 * q + rb, 2 * ks + ub));
      mma_row(Y, al, b);
      mma_row(Y, ah, b);
      if constexpr (NI == 2) {
#pragma unroll
        for (int q = 0; q < 4; ++q) ldsm4(b[q], st + Sh::S_K + Sh::TILE + unit_at<U>(16 * q + rb, 2 * ks + ub));
        mma_row(Y, ah, b);
      }
      if constexpr (!STORE) {
#pragma unroll
      for (int q = 0; q < 4; ++q) ldsm4(b[q], st + Sh::S_Q + unit_at<U>(16 * q + rb, 2 * ks + ub));
      mma_row(O, ah, b);
      if constexpr (NI == 2) {
        mma_row(O, al, b);
#pragma unroll
        for (int q = 0; q < 4; ++q) ldsm4(b[q], st + Sh::S_Q + Sh::TILE + unit_at<U>(16 * q + rb, 2 * ks + ub));
        mma_row(O, ah, b);
      }
      }
    }

    // ---- Y = beta (v - e^G k S); the part of o that the state gives
    const unsigned char *strip = smem + (st - base) + Sh::S_V + warp * Sh::V_STRIP;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float x[2][4];
      if constexpr (NI == 1) {
        uint32_t r[4];
        ldsm4t(r, smem_addr(strip) + (16 * q + ((lane >> 4) << 3) + (lane & 7)) * 32 + ((lane >> 3) & 1) * 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[i >> 1][2 * (i & 1)] = __uint_as_float(r[i] << 16);
          x[i >> 1][2 * (i & 1) + 1] = __uint_as_float(r[i] & 0xffff0000u);
        }
      } else {
        const float *f = reinterpret_cast<const float *>(strip);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[i][e] = f[(16 * q + 8 * i + t + (e & 1)) * 16 + g + (e >> 1) * 8];
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int nt = 2 * q + i, j = 8 * nt + t;
        const float2 be = *reinterpret_cast<const float2 *>(num + NUM_BETA + j), ek = *reinterpret_cast<const float2 *>(num + NUM_EK + j),
                     eq = *reinterpret_cast<const float2 *>(num + NUM_EQ + j);
        Y[nt][0] = Y[nt][0] * ek.x * z0.y;
        Y[nt][1] = Y[nt][1] * ek.y * z0.y;
        Y[nt][2] = Y[nt][2] * ek.x * z1.y;
        Y[nt][3] = Y[nt][3] * ek.y * z1.y;
        if constexpr (STORE)
          reinterpret_cast<float4 *>(ws + pl.off_e)[((unit * (p.dv / 16) + v0 / 16) * 8 + nt) * 32 + lane] =
              make_float4(Y[nt][0], Y[nt][1], Y[nt][2], Y[nt][3]);
        Y[nt][0] = be.x * (x[i][0] - Y[nt][0]);
        Y[nt][1] = be.y * (x[i][1] - Y[nt][1]);
        Y[nt][2] = be.x * (x[i][2] - Y[nt][2]);
        Y[nt][3] = be.y * (x[i][3] - Y[nt][3]);
        if constexpr (STORE) continue;  // no outputs
        // factor by factor: the factors' product may be too small for fp32 where the result is not
        O[nt][0] = O[nt][0] * eq.x * z0.y;
        O[nt][1] = O[nt][1] * eq.y * z0.y;
        O[nt][2] = O[nt][2] * eq.x * z1.y;
        O[nt][3] = O[nt][3] * eq.y * z1.y;
      }
    }

    if constexpr (STORE) start_second(c);
    // ---- W^T = Y^T A^T
    float W[8][4];
    row_scales(Y, z0, z1);
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) W[i][e] = 0.f;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      uint32_t ah[4], al[4];
      as_left(Y, ks, z0.x, z1.x, ah, al);
      uint32_t b[4][4];
#pragma unroll
      for (int q = ks; q < 4; ++q) ldsm4(b[q], st + Sh::S_A + MAT_BYTES + unit_at<8>(16 * q + rb, 2 * ks + ub));
      mma_row(W, ah, b, ks);
#pragma unroll
      for (int q = ks; q < 4; ++q) ldsm4(b[q], st + Sh::S_A + unit_at<8>(16 * q + rb, 2 * ks + ub));
      mma_row(W, al, b, ks);
      mma_row(W, ah, b, ks);
    }
    {
      const float a = num[NUM_MISC + 1];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        W[i][0] = W[i][0] * a * z0.y;
        W[i][1] = W[i][1] * a * z0.y;
        W[i][2] = W[i][2] * a * z1.y;
        W[i][3] = W[i][3] * a * z1.y;
      }
    }

    if constexpr (STORE) {
      keep(pl.off_w, W, 8, warp_max(W), MAX_W);
    } else {
    start_second(c);
    // ---- o += P W
    row_scales(W, z0, z1);
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) Y[i][e] = 0.f;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      uint32_t ah[4], al[4];
      as_left(W, ks, z0.x, z1.x, ah, al);
      uint32_t b[4][4];
#pragma unroll
      for (int q = ks; q < 4; ++q) ldsm4(b[q], st + Sh::S_P + unit_at<8>(16 * q + rb, 2 * ks + ub));
      mma_row(Y, ah, b, ks);
      if constexpr (NI == 2) {
        mma_row(Y, al, b, ks);
#pragma unroll
        for (int q = ks; q < 4; ++q) ldsm4(b[q], st + Sh::S_P + MAT_BYTES + unit_at<8>(16 * q + rb, 2 * ks + ub));
        mma_row(Y, ah, b, ks);
      }
    }
    const int64_t r0 = (int64_t)c * C;
    const int len = (int)(t1 - t0 - r0 < C ? t1 - t0 - r0 : C);
    {
      const float a = num[NUM_MISC + 2];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        O[i][0] += Y[i][0] * a * z0.y;
        O[i][1] += Y[i][1] * a * z0.y;
        O[i][2] += Y[i][2] * a * z1.y;
        O[i][3] += Y[i][3] * a * z1.y;
      }
    }
    if constexpr (NI == 1) {
      const uint32_t os = base + Sh::S_OUT + warp * Sh::V_STRIP;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __nv_bfloat162 x = __floats2bfloat162_rn(O[2 * q + (i >> 1)][2 * (i & 1)], O[2 * q + (i >> 1)][2 * (i & 1) + 1]);
          r[i] = *reinterpret_cast<const uint32_t *>(&x);
        }
        stsm4t(os + (16 * q + ((lane >> 4) << 3) + (lane & 7)) * 32 + ((lane >> 3) & 1) * 16, r[0], r[1], r[2], r[3]);
      }
      __syncwarp();
#pragma unroll
      for (int x = lane; x < C * 2; x += 32)
        if ((x >> 1) < len)
          *reinterpret_cast<uint4 *>(out + (r0 + (x >> 1)) * p.v.t + (x & 1) * 8) =
              *reinterpret_cast<const uint4 *>(smem + Sh::S_OUT + warp * Sh::V_STRIP + x * 16);
      __syncwarp();
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = 8 * i + t + (e & 1);
          if (j < len) out[(r0 + j) * p.v.t + g + (e >> 1) * 8] = O[i][e];
        }
    }
    }

    // ---- S^T = e^{G_C} S^T + (e^{G_C - G} W)^T k
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 fk = *reinterpret_cast<const float2 *>(num + NUM_FK + 8 * i + t);
      W[i][0] *= fk.x;
      W[i][1] *= fk.y;
      W[i][2] *= fk.x;
      W[i][3] *= fk.y;
    }
    row_scales(W, z0, z1);
    uint32_t wh[4][4], wl[4][4];
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) as_left(W, ks, z0.x, z1.x, wh[ks], wl[ks]);
    const float ec = num[NUM_MISC];
#pragma unroll
    for (int q = 0; q < NK / 2; q += 2) {
      float acc[4][4] = {};
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        uint32_t b[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) ldsm4t(b[i], st + Sh::S_K + unit_at<U>(16 * ks + rt, 2 * (q + i) + ut));
        mma_row(acc, wl[ks], b);
        mma_row(acc, wh[ks], b);
        if constexpr (NI == 2) {
#pragma unroll
          for (int i = 0; i < 2; ++i) ldsm4t(b[i], st + Sh::S_K + Sh::TILE + unit_at<U>(16 * ks + rt, 2 * (q + i) + ut));
          mma_row(acc, wh[ks], b);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        S[2 * q + i][0] = ec * S[2 * q + i][0] + acc[i][0] * z0.y;
        S[2 * q + i][1] = ec * S[2 * q + i][1] + acc[i][1] * z0.y;
        S[2 * q + i][2] = ec * S[2 * q + i][2] + acc[i][2] * z1.y;
        S[2 * q + i][3] = ec * S[2 * q + i][3] + acc[i][3] * z1.y;
      }
    }
    // the buffer may be refilled
    if constexpr (Sh::STAGES == 1) __syncthreads();
    else if (c + 2 < nc) bar_arrive(bar_empty(c & 1, group), GROUP + FILL);
  }

  if (io.final_state) {
#pragma unroll
    for (int i = 0; i < NK; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        io.final_state[s_off + (8 * i + t + (e & 1)) * sk + (v0 + g + (e >> 1) * 8) * sv] = S[i][e];
  }
}

template <typename T, int DK, int WARPS, bool STORE>
cudaError_t go(const Problem &p, char *ws, const Plan &pl, const ChainOut &io, cudaStream_t st) {
  auto kernel = gdn_chain_kernel<T, DK, WARPS, STORE>;
  constexpr int smem = Shape<T, DK, WARPS, STORE>::BYTES;
  const kda_dtype dt = sizeof(T) == 2 ? KDA_BF16 : KDA_F32;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int64_t grid = (int64_t)p.s.N * p.H * (p.dv / (16 * WARPS));
  kernel<<<(unsigned)grid, Shape<T, DK, WARPS, STORE>::THREADS, smem, st>>>(p, ws, pl, kq_bytes(dt, p.dk), ap_bytes(dt, STORE), io);
  return cudaGetLastError();
}

template <typename T, bool STORE>
cudaError_t go_dims(const Problem &p, char *ws, const Plan &pl, const ChainOut &io, cudaStream_t st) {
  const bool w = p.dk == 128;
  if (p.dv == 128 && !p.halves) return w ? go<T, 128, 8, STORE>(p, ws, pl, io, st) : go<T, 64, 8, STORE>(p, ws, pl, io, st);
  return w ? go<T, 128, 4, STORE>(p, ws, pl, io, st) : go<T, 64, 4, STORE>(p, ws, pl, io, st);
}

}  // namespace

cudaError_t launch_gdn_chain(kda_dtype dt, bool bwd, const Problem &p, char *ws, const Plan &pl, const ChainOut &io, cudaStream_t st) {
  if (dt == KDA_BF16)
    return bwd ? go_dims<__nv_bfloat16, true>(p, ws, pl, io, st) : go_dims<__nv_bfloat16, false>(p, ws, pl, io, st);
  return bwd ? go_dims<float, true>(p, ws, pl, io, st) : go_dims<float, false>(p, ws, pl, io, st);
}

}  // namespace gdn
}  // namespace kda
