// kda_gdn.cuh - the gated delta rule with one gate per head: what its kernels
// share.
//
//   S_t = e^{g_t} (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T,   o_t = scale S_t^T q_t
//
// With G the running sum of g inside a chunk of 64 tokens and S the state
// entering it,
//   L_ij = beta_i e^{G_i - G_j} k_i.k_j (j < i),   A = (I + L)^-1
//   Y  = beta (V - e^G K S),   W = A Y             (the corrected values)
//   O  = scale e^G Q S + P W,  P_ij = scale e^{G_i - G_j} q_i.k_j (j <= i)
//   S' = e^{G_C} S + (e^{G_C - G} K)^T W
// A gate of one number per head commutes with every product over channels, so
// k and q enter the products as the caller gave them and the gates, norms and
// the scale are numbers per token, applied to sums.
//
// Arithmetic.  Products run on the tensor cores as fp16 pieces with fp32
// sums: a value x is s x = hi + lo, s a power of two that takes the largest that
// shares it to [2^13, 2^14), and a product of two such values is hi hi + hi lo +
// lo hi.  fp16's numbers end at 2^-24: x is off by at most 2^-23 of itself (22
// bits and more) down to 2^-15 of that largest one, below that by 2^-38 of it
// (hi alone: 2^-12 of itself, and from 2^-27 on 2^-38 of the largest).  What shares a unit: a
// token's k, q and, in the last kernel, d_out; a value channel's row of S, Y, W and
// their gradients over a chunk's 64 tokens; A and P of a chunk; in the last
// kernel S, dS', W, dY and the tiles of coefficients, each as a whole.  So
// tokens of very different size in a chunk cost the small ones bits, but not
// dq, which is a token's d_out's own (and out, with norms).  bf16
// inputs are one piece (8 bits fit fp16's 11), so the state, held in fp32,
// costs two products with them and keeps fp32's accuracy; bf16 pieces would
// lose 2^-17 of it at the same cost.  What only leads to a bf16 result (o, dq,
// dk) takes the first piece alone: 2^-12, an eighth of bf16's own rounding.
#pragma once

#include <cuda_fp16.h>

#include "kda_fill.cuh"
#include "kda_internal.cuh"

namespace kda {
namespace gdn {

constexpr int C = BT;

// Element strides of a [.., tokens, heads, channels] tensor.
struct Strides {
  int64_t b, t, h;
};

// One problem, as every kernel of the family takes it.
struct Problem {
  SeqInfo s;
  int H, Hk, dk, dv;
  int32_t nchunks;         // upper bound
  Strides qk, v, gate;     // q and k; v, out and their gradients; g and beta (no channels)
  const void *q, *k, *val;
  const float *g, *beta;
  GateParams gp;
  bool v_first;            // states are [dv, dk]
  bool halves;             // chains of 128 value channels as two CTAs: with few of them, each chunk is done sooner
  const int32_t *order;    // packed sequences from the longest to the shortest, or null: as they come
};

// Up to so many packed sequences are taken in the order of their lengths: the
// chains' time is their longest's, if that does not start last.
constexpr int ORDERED = 1024;

// Chunk c's first token: batch row and token inside it, as the strides want
// them, and the tokens it holds (false: none).
__device__ __forceinline__ bool chunk_at(const SeqInfo &s, int64_t c, int &n, int64_t &batch, int64_t &tok, int &len) {
  int64_t t0;
  if (!chunk_lookup(s, c, n, t0, len)) return false;
  batch = s.bounds ? 0 : n;
  tok = s.bounds ? t0 : t0 - (int64_t)n * s.T;
  return true;
}

// ---------------------------------------------------------------- workspace
// Per (chunk, key head): the fp16 pieces of k, then of q, each [64, dk] as the
// bytes of a shared-memory tile (16-byte units XOR-swizzled by row, so that
// eight rows' units of one column lie in different banks).
// Per (chunk, value head): numbers per token, then the pieces of A, then of P
// ([64, 64] tiles; blocks of 16 above the diagonal are not written).
// Numbers: beta; e^G, e^{G_C - G} with the norms' factors (and the scale, for q)
// in them; those factors alone, times what a unit of the pieces stands for (no
// scale) and by themselves; G to base 2 in two floats.  misc: 0 e^{G_C}, 1 what a unit of
// A's pieces stands for, 2 the same of P's.
constexpr int NUM_MISC = 0, NUM_BETA = 16, NUM_EK = 80, NUM_EQ = 144, NUM_FK = 208, NUM_K = 272, NUM_Q = 336, NUM_GH = 400,
              NUM_GL = 464, NUM_RK = 528, NUM_RQ = 592, NUM_FLOATS = 656;
constexpr int NUM_BYTES = NUM_FLOATS * 4;
constexpr int MAT_BYTES = C * C * 2;

template <typename T> constexpr int pieces() { return sizeof(T) == 2 ? 1 : 2; }

inline int in_pieces(kda_dtype d) { return d == KDA_BF16 ? 1 : 2; }
inline size_t kq_bytes(kda_dtype d, int dk) { return (size_t)2 * in_pieces(d) * C * dk * 2; }
// P in two pieces where the backward reads it (its products lead to fp32 results)
inline size_t ap_bytes(kda_dtype d, bool bwd) { return NUM_BYTES + (size_t)MAT_BYTES * (2 + (bwd ? 2 : in_pieces(d))); }

// What the backward's kernels hand on, per (chunk, value head), in fp32 and in
// the order in which a warp's lanes hold it ([16 value channels][8 columns]
// tiles, four values a lane): the state entering the chunk and the gradient of
// the one leaving it ([dv, dk]), W, e^G k S and dY ([dv, 64]); the largest of
// each of S, dS, W, dY in each warp's 16 channels; sums over each 64
// channels for each token; the sums of a_log's and dt_bias's gradients.
struct Plan {
  size_t off_chunks, off_kq, off_ap, off_s, off_ds, off_w, off_e, off_dy, off_max, off_dots, off_part, total;
};
constexpr int MAX_S = 0, MAX_DS = 8, MAX_W = 16, MAX_DY = 24, MAX_FLOATS = 32;
constexpr int DOT_BETA = 0, DOT_K = 64, DOT_Y = 128, DOT_FLOATS = 192;
inline Plan make_gdn_plan(kda_dtype d, int64_t nchunks, int N, int H, int Hk, int dk, int dv, bool bwd) {
  Plan p{};
  size_t o = 256;
  p.off_chunks = o; o = align256(o + sizeof(int32_t) * (2 * (size_t)N + 1));
  p.off_kq = o; o = align256(o + (size_t)nchunks * Hk * kq_bytes(d, dk));
  p.off_ap = o; o = align256(o + (size_t)nchunks * H * ap_bytes(d, bwd));
  if (bwd) {
    const size_t u = (size_t)nchunks * H;
    p.off_s = o; o = align256(o + u * dk * dv * 4);
    p.off_ds = o; o = align256(o + u * dk * dv * 4);
    p.off_w = o; o = align256(o + u * C * dv * 4);
    p.off_e = o; o = align256(o + u * C * dv * 4);
    p.off_dy = o; o = align256(o + u * C * dv * 4);
    p.off_max = o; o = align256(o + u * MAX_FLOATS * 4);
    p.off_dots = o; o = align256(o + u * 2 * DOT_FLOATS * 4);
    p.off_part = o; o = align256(o + u * 2 * 4);
  }
  p.total = o;
  return p;
}

// ---------------------------------------------------------------- primitives
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// c[2 q], c[2 q + 1] += a b[q] for a row of tiles, from tile pair q0 to q1.
template <int N, int M>
__device__ __forceinline__ void mma_row(float (&c)[N][4], const uint32_t (&a)[4], const uint32_t (&b)[M][4], int q0 = 0, int q1 = N / 2) {
#pragma unroll
  for (int q = 0; q < N / 2; ++q)
    if (q >= q0 && q < q1) {
      mma16(c[2 * q], a, b[q][0], b[q][1]);
      mma16(c[2 * q + 1], a, b[q][2], b[q][3]);
    }
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void stsm4t(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b),
               "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint32_t smem_addr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void cp16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// 16 bytes, or zeros (src is then not read)
__device__ __forceinline__ void cp16z(uint32_t dst, const void *src, bool fill) {
  const int n = fill ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
// [64 tokens][16 W channels] as W strips [64][16] (a warp's); rows from `rows` on
// are zero and not read.
template <int W, typename T> __device__ __forceinline__ void load_strips(uint32_t dst, const T *src, int64_t stride, int64_t rows, int first) {
  constexpr int U = sizeof(T);  // 16-byte units of a strip's row
#pragma unroll 4
  for (int x = first; x < C * U * W; x += FILL) {
    const int r = x / (U * W), u = x % (U * W);
    const bool in = r < rows;
    cp16z(dst + (u / U) * (C * U * 16) + (r * U + u % U) * 16, in ? src + r * stride + u * (16 / sizeof(T)) : src, in);
  }
}

// Byte offset of 16-byte unit u of row r, rows of U units (8 or 16).
template <int U> __device__ __forceinline__ uint32_t unit_at(int r, int u) { return (uint32_t)((r * U + (u ^ (r & 7))) * 16); }

__device__ __forceinline__ uint32_t pack_half(float a, float b) {
  __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<uint32_t *>(&h);
}
// hi and lo pieces of two values that are in range already
__device__ __forceinline__ void split2(float a, float b, uint32_t &hi, uint32_t &lo) {
  const __half2 h = __floats2half2_rn(a, b);
  const float2 f = __half22float2(h);
  hi = *reinterpret_cast<const uint32_t *>(&h);
  lo = pack_half(a - f.x, b - f.y);
}
// The power of two s that takes m (>= 0) to [2^13, 2^14), and 1 / s.  Both
// are normal numbers; a maximum below 2^-113 stays smaller, one of zero takes any.
__device__ __forceinline__ float2 piece_scale(float m) {
  int e = (int)(__float_as_uint(m) >> 23);
  int sb = 267 - e;
  sb = sb > 253 ? 253 : sb;
  return make_float2(__uint_as_float((uint32_t)sb << 23), __uint_as_float((uint32_t)(254 - sb) << 23));
}
// Largest of |c0|, |c1| (row lane / 4) and of |c2|, |c3| (row + 8) over a row's
// four lanes, as scales.
template <int N>
__device__ __forceinline__ void row_scales(const float (&x)[N][4], float2 &lo, float2 &hi) {
  float a = 0.f, b = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    a = fmaxf(a, fmaxf(fabsf(x[i][0]), fabsf(x[i][1])));
    b = fmaxf(b, fmaxf(fabsf(x[i][2]), fabsf(x[i][3])));
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    a = fmaxf(a, __shfl_xor_sync(~0u, a, o));
    b = fmaxf(b, __shfl_xor_sync(~0u, b, o));
  }
  lo = piece_scale(a);
  hi = piece_scale(b);
}

// Largest |x| of a warp's accumulators.
template <int N>
__device__ __forceinline__ float warp_max(const float (&x)[N][4]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) m = fmaxf(m, fmaxf(fmaxf(fabsf(x[i][0]), fabsf(x[i][1])), fmaxf(fabsf(x[i][2]), fabsf(x[i][3]))));
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
  return m;
}

// Columns 16 ks .. of an accumulator as the left operand, in pieces.
template <int N>
__device__ __forceinline__ void as_left(const float (&x)[N][4], int ks, float s0, float s1, uint32_t (&hi)[4], uint32_t (&lo)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    split2(x[2 * ks + i][0] * s0, x[2 * ks + i][1] * s0, hi[2 * i], lo[2 * i]);
    split2(x[2 * ks + i][2] * s1, x[2 * ks + i][3] * s1, hi[2 * i + 1], lo[2 * i + 1]);
  }
}

// 8 values of a row as fp32
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&x)[8]) {
  const uint4 r = *reinterpret_cast<const uint4 *>(p);
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const float *p, float (&x)[8]) {
  const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

constexpr float LOG2E = 1.4426950408889634f;

// 2^x, x <= 0, to 2^-22 of its size; below 2^-126 zero.
__device__ __forceinline__ float exp2_neg(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Log-decay of one token and head from what the caller gave.  From -256 on
// (e^-256 is zero in fp32) it is held there: -inf, a decay to nothing, would
// make NaN of the differences of running sums.
__device__ __forceinline__ float log_decay(float x, const GateParams &gp, float neg_exp_alog, float bias) {
  if (gp.flags & KDA_GATE_IN_KERNEL) {
    const float z = x + bias;
    x = neg_exp_alog * (fmaxf(z, 0.f) + log1pf(expf(-fabsf(z))));
  }
  return x < -256.f ? -256.f : x;
}

// ---------------------------------------------------------------- launchers
// A tensor whose tokens behind the last packed sequence are set to zero: `heads`
// runs of all tokens, `pitch` bytes apart, `token` bytes each.
struct Behind {
  void *p;
  int64_t heads, pitch, token;
};
struct BehindAll {
  Behind a[5];
  int n;
};
// Chunk offsets [N + 1] and order [N] of at most ORDERED packed sequences (order
// null: neither), and zeros behind the last one.
cudaError_t launch_gdn_map(const SeqInfo &s, int32_t *chunk_off, int32_t *order, const BehindAll &z, cudaStream_t st);
cudaError_t launch_gdn_prep(kda_dtype dt, bool bwd, const Problem &p, char *ws, const Plan &pl, cudaStream_t st);

// The forward's chain writes out and final_state; the backward's first one (out
// null) S, W, e^G k S and their largest values instead.
struct ChainOut {
  void *out;
  const float *initial;
  float *final_state;
};
cudaError_t launch_gdn_chain(kda_dtype dt, bool bwd, const Problem &p, char *ws, const Plan &pl, const ChainOut &io, cudaStream_t st);

struct GradOut {
  const void *d_out;        // or null: zeros
  const float *d_final;     // or null: zeros
  void *dq, *dk, *dv;
  float *dg, *dbeta, *da_log, *ddt_bias, *d_initial;
};
cudaError_t launch_gdn_bwd(kda_dtype dt, const Problem &p, char *ws, const Plan &pl, const GradOut &io, cudaStream_t st);

cudaError_t launch_gdn_step(const kda_decode_args &a, cudaStream_t st);

}  // namespace gdn
}  // namespace kda
