// kda_api_gdn.cu - C ABI of the gated delta rule with one gate per head:
// host-side argument checks, the workspace plan, then the launches.
#include "kda_gdn.cuh"

using namespace kda;

namespace {

inline bool mis16(const void *p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
inline kda_status cuda_status(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

constexpr uint32_t kFlags = KDA_L2NORM_QK | KDA_BETA_SIGMOID | KDA_GATE_IN_KERNEL | KDA_USE_EXP2 | KDA_STATE_V_FIRST |
                            KDA_LAYOUT_HEAD_MAJOR;
constexpr uint32_t kChunkFlags = kFlags | KDA_ZERO_BEHIND;
constexpr uint32_t kRefused = KDA_REUSE_PREP | KDA_SAFE_GATE | KDA_ALLOW_NEG_EIGVAL;

inline int key_heads(const kda_fwd_args *a) { return a->Hk > 0 ? a->Hk : a->H; }
inline int64_t tokens(const kda_fwd_args *a) { return (int64_t)a->B * a->T; }

kda_status check(const kda_fwd_args *a) {
  if (!a || a->B < 1 || a->T < 0 || a->H < 1) return KDA_ERR_INVALID_ARG;
  if (a->Hk < 0 || (a->Hk > 0 && a->H % a->Hk != 0)) return KDA_ERR_INVALID_ARG;
  if (a->flags & ~(kChunkFlags | kRefused)) return KDA_ERR_INVALID_ARG;
  if (a->qkv_dtype != KDA_F32 && a->qkv_dtype != KDA_BF16) return KDA_ERR_INVALID_ARG;
  if (tokens(a) > 0 && (!a->q || !a->k || !a->v || !a->g || !a->beta)) return KDA_ERR_INVALID_ARG;
  if ((a->flags & KDA_GATE_IN_KERNEL) && !a->a_log) return KDA_ERR_INVALID_ARG;
  if (a->cu_seqlens && (a->B != 1 || a->num_seqs < 1)) return KDA_ERR_INVALID_ARG;
  if ((a->dk != 64 && a->dk != 128) || (a->dv != 64 && a->dv != 128) || a->chunk != BT) return KDA_ERR_UNSUPPORTED;
  if ((a->flags & kRefused) || a->h_out || a->v_new_out) return KDA_ERR_UNSUPPORTED;
  if (tokens(a) > INT32_MAX) return KDA_ERR_UNSUPPORTED;  // token ids are 32-bit
  const int64_t n = a->cu_seqlens ? a->num_seqs : a->B;
  // one CTA per (chunk, head) and per (sequence, head)
  if ((tokens(a) / BT + n) * a->H > INT32_MAX) return KDA_ERR_UNSUPPORTED;
  if (mis16(a->q) || mis16(a->k) || mis16(a->v) || mis16(a->g) || mis16(a->beta) || mis16(a->a_log) || mis16(a->dt_bias) ||
      mis16(a->initial_state) || mis16(a->cu_seqlens))
    return KDA_ERR_ALIGNMENT;
  return KDA_OK;
}

kda_status check_fwd(const kda_fwd_args *a) {
  const kda_status s = check(a);
  if (s != KDA_OK) return s;
  if (!a->out && tokens(a) > 0) return KDA_ERR_INVALID_ARG;
  return mis16(a->out) || mis16(a->final_state) ? KDA_ERR_ALIGNMENT : KDA_OK;
}

gdn::Problem problem(const kda_fwd_args *a) {
  gdn::Problem p{};
  p.s.bounds = a->cu_seqlens;
  p.s.T_tot = tokens(a);
  p.s.T = a->T;
  p.s.N = a->cu_seqlens ? a->num_seqs : a->B;
  p.H = a->H;
  p.Hk = key_heads(a);
  p.dk = a->dk;
  p.dv = a->dv;
  p.nchunks = (int32_t)chunks_upper_bound(p.s.T_tot, p.s.N, a->cu_seqlens != nullptr, a->T);
  const bool hm = (a->flags & KDA_LAYOUT_HEAD_MAJOR) != 0;
  auto strides = [&](int64_t heads, int64_t d) {
    const int64_t T = a->T;
    return hm ? gdn::Strides{heads * T * d, d, T * d} : gdn::Strides{T * heads * d, heads * d, d};
  };
  p.qk = strides(p.Hk, a->dk);
  p.v = strides(a->H, a->dv);
  p.gate = strides(a->H, 1);
  p.q = a->q; p.k = a->k; p.val = a->v;
  p.g = a->g; p.beta = a->beta;
  p.gp.a_log = a->a_log;
  p.gp.dt_bias = a->dt_bias;
  p.gp.scale = a->scale;
  p.gp.eps = a->eps;
  p.gp.flags = a->flags;
  p.v_first = (a->flags & KDA_STATE_V_FIRST) != 0;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) == cudaSuccess && cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess)
    p.halves = p.dv == 128 && (int64_t)p.s.N * p.H * 2 <= sms;
  return p;
}

// What is set to zero behind the last packed sequence, if the caller wants it.
struct Written {
  void *p;
  int heads, d;  // d: channels, 0 for fp32 numbers without any
};
template <size_t N> gdn::BehindAll behind(const kda_fwd_args *a, const Written (&w)[N]) {
  static_assert(N <= sizeof(gdn::BehindAll::a) / sizeof(gdn::Behind), "");
  gdn::BehindAll z{};
  if (!a->cu_seqlens || !(a->flags & KDA_ZERO_BEHIND)) return z;
  const bool hm = (a->flags & KDA_LAYOUT_HEAD_MAJOR) != 0;
  for (const Written &x : w) {
    if (!x.p) continue;
    const int64_t one = x.d ? (int64_t)x.d * (a->qkv_dtype == KDA_BF16 ? 2 : 4) : 4;
    z.a[z.n++] = hm ? gdn::Behind{x.p, x.heads, a->T * one, one} : gdn::Behind{x.p, 1, 0, x.heads * one};
  }
  return z;
}

// Chunk offsets of packed sequences (p.s.chunk_off) and their order, then the preparation.
cudaError_t prepare(const kda_fwd_args *a, bool bwd, gdn::Problem &p, char *ws, const gdn::Plan &pl, const gdn::BehindAll &z,
                    cudaStream_t st) {
  int32_t *co = reinterpret_cast<int32_t *>(ws + pl.off_chunks);
  p.s.chunk_off = co;
  cudaError_t e = cudaSuccess;
  if (p.s.bounds && p.s.N <= gdn::ORDERED) {
    p.order = co + p.s.N + 1;
    e = gdn::launch_gdn_map(p.s, co, co + p.s.N + 1, z, st);
  } else if (p.s.bounds) {
    e = launch_chunk_map(p.s, co, st);
    if (e == cudaSuccess && z.n) e = gdn::launch_gdn_map(p.s, nullptr, nullptr, z, st);
  }
  if (e == cudaSuccess) e = gdn::launch_gdn_prep(a->qkv_dtype, bwd, p, ws, pl, st);
  return e;
}

}  // namespace

extern "C" {

size_t kda_gdn_chunk_fwd_workspace_size(const kda_fwd_args *a) {
  if (check_fwd(a) != KDA_OK) return 0;
  const gdn::Problem p = problem(a);
  return gdn::make_gdn_plan(a->qkv_dtype, p.nchunks, p.s.N, p.H, p.Hk, p.dk, p.dv, false).total;
}

kda_status kda_gdn_chunk_fwd(const kda_fwd_args *a, kda_stream_t stream) {
  const kda_status s = check_fwd(a);
  if (s != KDA_OK) return s;
  gdn::Problem p = problem(a);
  const gdn::Plan pl = gdn::make_gdn_plan(a->qkv_dtype, p.nchunks, p.s.N, p.H, p.Hk, p.dk, p.dv, false);
  if (!a->workspace || a->workspace_bytes < pl.total) return KDA_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(a->workspace) & 255u) return KDA_ERR_ALIGNMENT;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  char *ws = static_cast<char *>(a->workspace);
  cudaError_t e = prepare(a, false, p, ws, pl, behind(a, {Written{a->out, p.H, p.dv}}), st);
  if (e == cudaSuccess)
    e = gdn::launch_gdn_chain(a->qkv_dtype, false, p, ws, pl, gdn::ChainOut{a->out, a->initial_state, a->final_state}, st);
  return cuda_status(e);
}

static kda_status check_bwd(const kda_bwd_args *b) {
  if (!b) return KDA_ERR_INVALID_ARG;
  const kda_status s = check(&b->fwd);
  if (s != KDA_OK) return s;
  if (tokens(&b->fwd) > 0 && (!b->dq || !b->dk || !b->dv || !b->dg || !b->dbeta)) return KDA_ERR_INVALID_ARG;
  // d_out is read again after dv, and by chunks beside those whose dq and dk are written
  if (b->d_out && tokens(&b->fwd) > 0 && (b->d_out == b->dq || b->d_out == b->dk || b->d_out == b->dv)) return KDA_ERR_INVALID_ARG;
  if (mis16(b->d_out) || mis16(b->d_final_state) || mis16(b->dq) || mis16(b->dk) || mis16(b->dv) || mis16(b->dg) ||
      mis16(b->dbeta) || mis16(b->da_log) || mis16(b->ddt_bias) || mis16(b->d_initial_state))
    return KDA_ERR_ALIGNMENT;
  return KDA_OK;
}

size_t kda_gdn_chunk_bwd_workspace_size(const kda_bwd_args *b) {
  if (check_bwd(b) != KDA_OK) return 0;
  const gdn::Problem p = problem(&b->fwd);
  return gdn::make_gdn_plan(b->fwd.qkv_dtype, p.nchunks, p.s.N, p.H, p.Hk, p.dk, p.dv, true).total;
}

kda_status kda_gdn_chunk_bwd(const kda_bwd_args *b, kda_stream_t stream) {
  const kda_status s = check_bwd(b);
  if (s != KDA_OK) return s;
  const kda_fwd_args *a = &b->fwd;
  gdn::Problem p = problem(a);
  const gdn::Plan pl = gdn::make_gdn_plan(a->qkv_dtype, p.nchunks, p.s.N, p.H, p.Hk, p.dk, p.dv, true);
  if (!b->workspace || b->workspace_bytes < pl.total) return KDA_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(b->workspace) & 255u) return KDA_ERR_ALIGNMENT;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  char *ws = static_cast<char *>(b->workspace);
  cudaError_t e = prepare(a, true, p, ws, pl, behind(a, {Written{b->dq, p.Hk, p.dk}, Written{b->dk, p.Hk, p.dk}, Written{b->dv, p.H, p.dv},
                                                         Written{b->dg, p.H, 0}, Written{b->dbeta, p.H, 0}}), st);
  if (e == cudaSuccess) e = gdn::launch_gdn_chain(a->qkv_dtype, true, p, ws, pl, gdn::ChainOut{nullptr, a->initial_state, nullptr}, st);
  if (e == cudaSuccess)
    e = gdn::launch_gdn_bwd(a->qkv_dtype, p, ws, pl,
                            gdn::GradOut{b->d_out, b->d_final_state, b->dq, b->dk, b->dv, b->dg, b->dbeta, b->da_log,
                                         b->ddt_bias, b->d_initial_state}, st);
  return cuda_status(e);
}

kda_status kda_gdn_recurrent_step(const kda_decode_args *a, kda_stream_t stream) {
  if (!a || a->N < 0 || a->T < 1 || a->H < 1) return KDA_ERR_INVALID_ARG;
  if (a->Hk < 0 || (a->Hk > 0 && a->H % a->Hk != 0)) return KDA_ERR_INVALID_ARG;
  if (a->flags & ~(kFlags | kRefused)) return KDA_ERR_INVALID_ARG;
  if (a->flags & (kRefused | KDA_LAYOUT_HEAD_MAJOR)) return KDA_ERR_UNSUPPORTED;
  if ((a->dk != 64 && a->dk != 128) || (a->dv != 64 && a->dv != 128)) return KDA_ERR_UNSUPPORTED;
  if (a->qkv_dtype != KDA_F32 && a->qkv_dtype != KDA_BF16) return KDA_ERR_INVALID_ARG;
  if (a->cache_dtype != KDA_F32 && a->cache_dtype != KDA_BF16) return KDA_ERR_INVALID_ARG;
  if (a->idx_dtype != KDA_I32 && a->idx_dtype != KDA_I64) return KDA_ERR_INVALID_ARG;
  if (a->num_rows < 1 || a->row_stride_elems < (int64_t)a->H * a->dk * a->dv) return KDA_ERR_INVALID_ARG;
  if ((a->flags & KDA_GATE_IN_KERNEL) && !a->a_log) return KDA_ERR_INVALID_ARG;
  if (a->N == 0) return KDA_OK;
  if (!a->q || !a->k || !a->v || !a->g || !a->beta || !a->out || !a->cache || !a->idx) return KDA_ERR_INVALID_ARG;
  if (a->out == a->q || a->out == a->k) return KDA_ERR_INVALID_ARG;  // read by the other CTAs of a head, and of a group
  if ((int64_t)a->N * a->H > INT32_MAX / 2) return KDA_ERR_UNSUPPORTED;  // two CTAs a state
  return cuda_status(gdn::launch_gdn_step(*a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
