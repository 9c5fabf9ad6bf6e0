// kda_gdn_step.cu - the gated delta rule with one gate per head, token by
// token on states kept in a cache pool (decode):
//   S = e^g S;  d = beta (v - S^T k);  S = S + k d^T;  o = scale S^T q
// in fp32 throughout.
//
// A thread holds half a value channel's column of the state in registers: the
// two dot products of a token are its own sums and one exchange with the lane
// that holds the other half, k and q come from shared memory as broadcasts,
// and all loads of the state are in flight before the first is used.
// What bounds it is the state's way from and to memory.  64 x 32 states of 128 x 128,
// 32 heads on 16, us: fp32 55 (72% of the copy rate), bf16 37 (54%: as many loads, of two
// bytes); V-first, whose neighbouring lanes are 512 (256) bytes apart, 250 and 370; four
// tokens at once 96.  With d_k = 128 a thread's 64 values leave too few of its 128
// registers: 144 bytes are spilled.
#include "kda_gdn.cuh"

namespace kda {
namespace gdn {
namespace {

struct StepArgs {
  const void *q, *k, *v;
  const float *g, *beta;
  GateParams gp;
  void *out, *cache;
  int64_t num_rows, row_stride;
  const void *idx;
  const bool *init_flags;
  int T, H, Hk;
  bool idx64;
};

// A CTA has COLS of the dv value channels, two threads a channel.  Measured on
// 64 x 32 states of 128 x 128 fp32 (272 MB there and back, in a graph): 52.0 us with 64
// channels (5.2 TB/s, 77% of the copy rate), 58.5 with 128, 57.8 with 32; a
// thread a whole column (fewer threads, more registers) 57.6, four threads 67.9.
constexpr int COLS = 64;

template <typename T, typename Tc, int DK, int DV, bool VF>
__global__ void __launch_bounds__(2 * COLS, 4)
gdn_step_kernel(StepArgs a) {
  constexpr int R = DK / 2, WARPS = 2 * COLS / 32, PARTS = DV / COLS;
  __shared__ __align__(16) float s_k[DK], s_q[DK];
  __shared__ float s_sum[2][WARPS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int col = (int)(blockIdx.x % PARTS) * COLS + warp * 16 + (lane & 15), r0 = (lane >> 4) * R;
  const int n = (int)(blockIdx.x / PARTS / a.H), h = (int)(blockIdx.x / PARTS % a.H), hk = h / (a.H / a.Hk);
  const int64_t row = a.idx64 ? static_cast<const int64_t *>(a.idx)[n] : static_cast<const int32_t *>(a.idx)[n];
  const bool valid = row >= 0 && row < a.num_rows;
  Tc *state = static_cast<Tc *>(a.cache) + (valid ? row * a.row_stride : 0) + (int64_t)h * DK * DV + (VF ? col * DK + r0 : r0 * DV + col);
  constexpr int step = VF ? 1 : DV;
  float S[R];
  if (valid && (!a.init_flags || a.init_flags[n])) {
#pragma unroll
    for (int i = 0; i < R; ++i) S[i] = to_f32<Tc>(state[(int64_t)i * step]);
  } else {
#pragma unroll
    for (int i = 0; i < R; ++i) S[i] = 0.f;
  }
  const float nea = (a.gp.flags & KDA_GATE_IN_KERNEL) ? -expf(a.gp.a_log[h]) : 0.f;
  const float bias = a.gp.dt_bias ? a.gp.dt_bias[h] : 0.f;
  const T *q = static_cast<const T *>(a.q), *k = static_cast<const T *>(a.k), *v = static_cast<const T *>(a.v);
  T *out = static_cast<T *>(a.out);

  for (int t = 0; t < a.T; ++t) {
    const int64_t tk = ((int64_t)n * a.T + t) * a.Hk + hk, th = ((int64_t)n * a.T + t) * a.H + h;
    float kk = 0.f, qq = 0.f;
    for (int i = tid; i < DK; i += 2 * COLS) {
      const float x = to_f32<T>(k[tk * DK + i]), y = to_f32<T>(q[tk * DK + i]);
      s_k[i] = x;
      s_q[i] = y;
      kk = fmaf(x, x, kk);
      qq = fmaf(y, y, qq);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      kk += __shfl_xor_sync(~0u, kk, o);
      qq += __shfl_xor_sync(~0u, qq, o);
    }
    if (lane == 0) {
      s_sum[0][warp] = kk;
      s_sum[1][warp] = qq;
    }
    const float decay = expf(log_decay(a.g[th], a.gp, nea, bias));
    float b = a.beta[th];
    if (a.gp.flags & KDA_BETA_SIGMOID) b = 1.f / (1.f + expf(-b));
    const float vv = to_f32<T>(v[th * DV + col]);
    __syncthreads();
    float rk = 1.f, rq = a.gp.scale;
    if (a.gp.flags & KDA_L2NORM_QK) {
      kk = qq = 0.f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        kk += s_sum[0][w];
        qq += s_sum[1][w];
      }
      rk = 1.f / sqrtf(kk + a.gp.eps);
      rq = a.gp.scale / sqrtf(qq + a.gp.eps);
    }
    // four sums a dot product: shorter chains, and less rounding than one
    float p[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < R; i += 4) {
      const float4 x = *reinterpret_cast<const float4 *>(s_k + r0 + i);
      p[0] = fmaf(S[i], x.x, p[0]);
      p[1] = fmaf(S[i + 1], x.y, p[1]);
      p[2] = fmaf(S[i + 2], x.z, p[2]);
      p[3] = fmaf(S[i + 3], x.w, p[3]);
    }
    float sk = (p[0] + p[1]) + (p[2] + p[3]);
    sk += __shfl_xor_sync(~0u, sk, 16);
    const float d = b * rk * (vv - decay * rk * sk);
    p[0] = p[1] = p[2] = p[3] = 0.f;
#pragma unroll
    for (int i = 0; i < R; i += 4) {
      const float4 x = *reinterpret_cast<const float4 *>(s_k + r0 + i), y = *reinterpret_cast<const float4 *>(s_q + r0 + i);
      S[i] = fmaf(x.x, d, decay * S[i]);
      S[i + 1] = fmaf(x.y, d, decay * S[i + 1]);
      S[i + 2] = fmaf(x.z, d, decay * S[i + 2]);
      S[i + 3] = fmaf(x.w, d, decay * S[i + 3]);
      p[0] = fmaf(S[i], y.x, p[0]);
      p[1] = fmaf(S[i + 1], y.y, p[1]);
      p[2] = fmaf(S[i + 2], y.z, p[2]);
      p[3] = fmaf(S[i + 3], y.w, p[3]);
    }
    float sq = (p[0] + p[1]) + (p[2] + p[3]);
    sq += __shfl_xor_sync(~0u, sq, 16);
    if (lane < 16) out[th * DV + col] = from_f32<T>(rq * sq);
    __syncthreads();  // k and q are staged anew
  }
  if (valid) {
#pragma unroll
    for (int i = 0; i < R; ++i) state[(int64_t)i * step] = from_f32<Tc>(S[i]);
  }
}

template <typename T, typename Tc, bool VF> cudaError_t go(const kda_decode_args &x, const StepArgs &a, cudaStream_t st) {
  const unsigned grid = (unsigned)((int64_t)x.N * x.H * (x.dv / COLS));
  if (x.dv == 128) {
    if (x.dk == 128) gdn_step_kernel<T, Tc, 128, 128, VF><<<grid, 2 * COLS, 0, st>>>(a);
    else gdn_step_kernel<T, Tc, 64, 128, VF><<<grid, 2 * COLS, 0, st>>>(a);
  } else {
    if (x.dk == 128) gdn_step_kernel<T, Tc, 128, 64, VF><<<grid, 2 * COLS, 0, st>>>(a);
    else gdn_step_kernel<T, Tc, 64, 64, VF><<<grid, 2 * COLS, 0, st>>>(a);
  }
  return cudaGetLastError();
}
template <typename T, typename Tc> cudaError_t go_layout(const kda_decode_args &x, const StepArgs &a, cudaStream_t st) {
  return (x.flags & KDA_STATE_V_FIRST) ? go<T, Tc, true>(x, a, st) : go<T, Tc, false>(x, a, st);
}

}  // namespace

cudaError_t launch_gdn_step(const kda_decode_args &x, cudaStream_t st) {
  StepArgs a;
  a.q = x.q; a.k = x.k; a.v = x.v; a.g = x.g; a.beta = x.beta;
  a.gp.a_log = x.a_log;
  a.gp.dt_bias = x.dt_bias;
  a.gp.scale = x.scale;
  a.gp.eps = x.eps;
  a.gp.flags = x.flags;
  a.out = x.out; a.cache = x.cache; a.num_rows = x.num_rows; a.row_stride = x.row_stride_elems;
  a.idx = x.idx; a.init_flags = x.init_flags;
  a.T = x.T; a.H = x.H; a.Hk = x.Hk > 0 ? x.Hk : x.H;
  a.idx64 = x.idx_dtype == KDA_I64;
  const bool c = x.cache_dtype == KDA_BF16;
  if (x.qkv_dtype == KDA_BF16)
    return c ? go_layout<__nv_bfloat16, __nv_bfloat16>(x, a, st) : go_layout<__nv_bfloat16, float>(x, a, st);
  return c ? go_layout<float, __nv_bfloat16>(x, a, st) : go_layout<float, float>(x, a, st);
}

}  // namespace gdn
}  // namespace kda
