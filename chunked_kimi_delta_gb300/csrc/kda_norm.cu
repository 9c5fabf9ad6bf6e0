// kda_norm.cu - RMS norm with the residual's addition and an 8-bit result, and
// its backward.
//
//   h = x + r,  y = h rstd w,  rstd = (mean h^2 + eps)^-1/2
//   dx = rstd (w g - n mean(w g n)) + d,  dw = sum over rows of g n,  n = h rstd
//
// Both read every element once and write it once, so memory bounds them; what
// costs is the wait for a row's sum between its loads and its stores.  Teams
// of threads (a CTA, or a warp for rows of up to 1,024 columns) are
// persistent and walk the rows; each thread copies its own columns of the rows
// to come into shared memory (cp.async, kDepth rows ahead) and no thread reads
// another's copies, so the copies need no barrier and stay in flight while a
// row's sum is formed.
#include "kda_fp8.cuh"

namespace kda {
namespace {

constexpr int kDepth = 2;  // rows in flight per team

// How a row's columns are read and which thread holds them.
//   RING    cp.async into shared memory, kDepth rows ahead; thread t of a team
//           holds columns 8 (t + i team) .. + 7
//   DIRECT  16-byte loads straight to registers: rows too wide for the ring
//   ODD     rows that do not start on 16 bytes (cols % 8 != 0): one element at
//           a time, column 16 j + t % 16 of the group, so that 16 lanes read
//           neighbouring elements
// In all three, 16 neighbouring lanes hold the 128 columns of one scale.
enum Mode { RING, DIRECT, ODD };

// Eight elements of a row of `cols` for this thread's i-th place.
template <Mode M, bool WARP> __device__ __forceinline__ int first_col(int i) {
  const int t = WARP ? (threadIdx.x & 31) + i * 32 : threadIdx.x + i * blockDim.x;
  return M == ODD ? (t >> 4) * FP8_BLOCK + (t & 15) : 8 * t;
}
constexpr int kOddStep = 16;

template <typename T, Mode M> __device__ __forceinline__ Raw8<T> load(const T *row, int c, int cols) {
  if (M == ODD) return raw_gather<T>(row + c, kOddStep, cols - c);
  return c < cols ? raw_load<T>(row + c) : raw_zero<T>();
}
template <typename T, Mode M> __device__ __forceinline__ void store(T *row, int c, int cols, const Raw8<T> &r) {
  if (M == ODD) raw_scatter<T>(row + c, kOddStep, cols - c, r);
  else if (c < cols) raw_store<T>(row + c, r);
}
template <typename T, Mode M> __device__ __forceinline__ void store(T *row, int c, int cols, const float2 (&f)[4]) {
  Raw8<T> r;
  r.put(f);
  store<T, M>(row, c, cols, r);
}
// Products on pairs; the odd layout's scattered loads do not end up in
// register pairs, and moving them there costs more than it saves.
template <Mode M> __device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  return M == ODD ? make_float2(a.x * b.x, a.y * b.y) : f2_mul(a, b);
}
template <Mode M> __device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  return M == ODD ? make_float2(fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y)) : f2_fma(a, b, c);
}
template <Mode M> __device__ __forceinline__ void load_weight(const float *w, int c, int cols, float2 (&f)[4]) {
  if (w) {
    load<float, M>(w, c, cols).get(f);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = f2_splat(1.f);
  }
}

// The ring of one tensor: thread-private slots of eight elements.
template <typename T> __device__ __forceinline__ void copy_ahead(Raw8<T> *slot, const T *src) {
  const uint32_t d = (uint32_t)__cvta_generic_to_shared(slot);
#pragma unroll
  for (int i = 0; i < (int)(sizeof(Raw8<T>) / 16); ++i)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                 :: "r"(d + 16 * i), "l"(reinterpret_cast<const uint4 *>(src) + i) : "memory");
}
__device__ __forceinline__ void commit_ahead() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void wait_oldest() { asm volatile("cp.async.wait_group %0;" :: "n"(kDepth - 1) : "memory"); }

// Sums over the team's threads, the same values in all of them, pairwise: the
// lanes of a warp, then the warps.  `red` alternates between two
// buffers from call to call, so one barrier is enough.
template <bool WARP, int N> __device__ __forceinline__ void team_sums(float (&v)[N], float (*red)[32]) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(~0u, v[n], o);
  if (WARP) return;
  const int warps = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int n = 0; n < N; ++n) red[n][threadIdx.x >> 5] = v[n];
  __syncthreads();
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = lane < warps ? red[n][lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(~0u, v[n], o);
}

// 32768 x 4096 bf16 with a residual, to 8 bits: 139 us, 6.8 TB/s, the copy
// rate; 8192 x 2048: 23 us, 5.2 TB/s (7 rows a CTA: start and end show); rows
// that start anywhere 25 to 75% of the rate, by their element accesses.
template <typename T, Mode M, int VPT, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : M == RING || VPT == 1 ? 512 : 1024) rms_norm_kernel(kda_rms_norm_args a) {
  extern __shared__ uint4 smem_raw[];
  __shared__ float red[2][1][32];
  const int cols = a.cols, blocks = (cols + FP8_BLOCK - 1) / FP8_BLOCK;
  const float inv_cols = 1.f / (float)cols;
  const T *x = static_cast<const T *>(a.x), *res = static_cast<const T *>(a.residual);
  const int tensors = res ? 2 : 1;  // in the ring, as the launch sized it
  Raw8<T> *ring = reinterpret_cast<Raw8<T> *>(smem_raw) + threadIdx.x;
  auto slot = [&](int stage, int tensor, int i) { return ring + ((stage * tensors + tensor) * VPT + i) * blockDim.x; };
  auto fetch = [&](int64_t row, int stage) {
    if (M != RING) return;
    if (row < a.rows) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = first_col<M, WARP>(i);
        if (c >= cols) continue;
        copy_ahead(slot(stage, 0, i), x + row * cols + c);
        if (res) copy_ahead(slot(stage, 1, i), res + row * cols + c);
      }
    }
    commit_ahead();
  };
  const int teams = WARP ? blockDim.x >> 5 : 1;
  const int64_t row0 = WARP ? (int64_t)blockIdx.x * teams + (threadIdx.x >> 5) : blockIdx.x;
  const int64_t step = (int64_t)gridDim.x * teams;
  grid_start();
  for (int s = 0; s < kDepth; ++s) fetch(row0 + s * step, s);
  constexpr bool KEEP = VPT < 4 || M == RING;  // threads of few columns keep their weights
  float2 w[KEEP ? VPT : 1][4];
  if (KEEP) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) load_weight<M>(a.weight, first_col<M, WARP>(i), cols, w[i]);
  }
  int stage = 0, parity = 0;
  for (int64_t row = row0; row < a.rows; row += step) {
    Raw8<T> h[VPT];
    float2 ss = f2_splat(0.f);
    if (M == RING) wait_oldest();
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = first_col<M, WARP>(i);
      if (M == RING) {
        h[i] = c < cols ? *slot(stage, 0, i) : raw_zero<T>();
        if (res && c < cols) h[i] = raw_add(h[i], *slot(stage, 1, i));
      } else {
        h[i] = load<T, M>(x + row * cols, c, cols);
        if (res) h[i] = raw_add(h[i], load<T, M>(res + row * cols, c, cols));
      }
      if (res) store<T, M>(static_cast<T *>(a.residual_out) + row * cols, c, cols, h[i]);
      float2 f[4];
      h[i].get(f);
#pragma unroll
      for (int j = 0; j < 4; ++j) ss = fma2<M>(f[j], f[j], ss);
    }
    float sums[1] = {ss.x + ss.y};
    team_sums<WARP>(sums, red[parity]);
    parity ^= 1;
    // every thread of the team has used its slots: the sum needed them
    fetch(row + kDepth * step, stage);
    stage = stage == kDepth - 1 ? 0 : stage + 1;
    const float rstd = 1.f / sqrtf(fmaf(sums[0], inv_cols, a.eps));
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = first_col<M, WARP>(i);
      // (h rstd) w: h w may leave the range of fp32 where y does not
      float2 y[4];
      h[i].get(y);
      if (!KEEP) load_weight<M>(a.weight, c, cols, w[0]);
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = mul2<M>(mul2<M>(y[j], f2_splat(rstd)), w[KEEP ? i : 0][j]);
      if (a.out) store<T, M>(static_cast<T *>(a.out) + row * cols, c, cols, y);
      if (!a.fp8) continue;
      float m = half_warp_max(block_amax(y));
      if (__any_sync(~0u, isinf(m))) {  // infinities count as NaN
        drop_infinities(y);
        m = half_warp_max(block_amax(y));
      }
      const uint32_t sb = fp8_scale_byte(m);
      const float2 inv = f2_splat(fp8_inv_scale(sb));
      const uint32_t lo = fp8_pack4(y[0], y[1], inv), hi = fp8_pack4(y[2], y[3], inv);
      uint8_t *q = static_cast<uint8_t *>(a.fp8) + row * a.ld_fp8;
      if (M == ODD) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c + kOddStep * j < cols) q[c + kOddStep * j] = (uint8_t)((j < 4 ? lo : hi) >> (8 * (j & 3)));
      } else if (c < cols) {
        *reinterpret_cast<uint2 *>(q + c) = make_uint2(lo, hi);
      }
      const int b = c / FP8_BLOCK;
      if ((threadIdx.x & 15) == 0 && b < ((blocks + 3) & ~3))
        a.fp8_scales[((b >> 2) * a.rows + row) * 4 + (b & 3)] = (uint8_t)sb;  // 1.0 past the last block
    }
  }
}

// ------------------------------------------------------------------ backward

constexpr int kMaxParts = 1216;  // partial dweight rows, and CTAs, at most: eight on each of 152 SMs

// dweight of a team's rows is summed in its registers; a CTA leaves one row of
// partial sums.  32768 x 4096 bf16 with the residual's gradient: 162 us for
// this and the sum of the parts, 6.7 TB/s, 98% of the copy rate.
template <typename T, Mode M, int VPT, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : M == RING || VPT < 4 ? 512 : 1024, WARP && VPT == 2 ? (M == ODD ? 2 : 4) : M != RING && VPT == 1 ? 2 : 1)
rms_norm_bwd_kernel(kda_rms_norm_bwd_args a) {
  extern __shared__ uint4 smem_raw[];
  __shared__ float red[2][2][32];
  const int cols = a.cols;
  const float inv_cols = 1.f / (float)cols;
  const T *hp = static_cast<const T *>(a.h), *gp = static_cast<const T *>(a.d_out);
  const T *dp = static_cast<const T *>(a.d_residual);
  const int tensors = dp ? 3 : 2;  // in the ring, as the launch sized it
  Raw8<T> *ring = reinterpret_cast<Raw8<T> *>(smem_raw) + threadIdx.x;
  auto slot = [&](int stage, int tensor, int i) { return ring + ((stage * tensors + tensor) * VPT + i) * blockDim.x; };
  auto fetch = [&](int64_t row, int stage) {
    if (M != RING) return;
    if (row < a.rows) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = first_col<M, WARP>(i);
        if (c >= cols) continue;
        copy_ahead(slot(stage, 0, i), hp + row * cols + c);
        copy_ahead(slot(stage, 1, i), gp + row * cols + c);
        if (dp) copy_ahead(slot(stage, 2, i), dp + row * cols + c);
      }
    }
    commit_ahead();
  };
  float2 dw[VPT][4];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) dw[i][j] = f2_splat(0.f);
  const int teams = WARP ? blockDim.x >> 5 : 1;
  const int64_t row0 = WARP ? (int64_t)blockIdx.x * teams + (threadIdx.x >> 5) : blockIdx.x;
  const int64_t step = (int64_t)gridDim.x * teams;
  grid_start();
  for (int s = 0; s < kDepth; ++s) fetch(row0 + s * step, s);
  constexpr bool KEEP = VPT < 4 || M == RING;  // as above; outside the ring, the row's values too
  float2 w[KEEP ? VPT : 1][4];
  if (KEEP) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) load_weight<M>(a.weight, first_col<M, WARP>(i), cols, w[i]);
  }
  int stage = 0, parity = 0;
  for (int64_t row = row0; row < a.rows; row += step) {
    if (M == RING) wait_oldest();
    // In the ring, h and g are read again after the sum: kept in registers they
    // would leave room for fewer threads.
    Raw8<T> kept[KEEP && M != RING ? VPT : 1][3];
    if (KEEP && M != RING) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = first_col<M, WARP>(i);
        kept[i][0] = load<T, M>(hp + row * cols, c, cols);
        kept[i][1] = load<T, M>(gp + row * cols, c, cols);
        if (dp) kept[i][2] = load<T, M>(dp + row * cols, c, cols);
      }
    }
    auto get = [&](int tensor, const T *p, int i, int c) {
      if (KEEP && M != RING) return kept[i][tensor];
      if (M != RING) return load<T, M>(p + row * cols, c, cols);
      return c < cols ? *slot(stage, tensor, i) : raw_zero<T>();
    };
    float2 ss = f2_splat(0.f), sg = f2_splat(0.f);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = first_col<M, WARP>(i);
      float2 h[4], g[4];
      get(0, hp, i, c).get(h);
      get(1, gp, i, c).get(g);
      if (!KEEP) load_weight<M>(a.weight, c, cols, w[0]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        ss = fma2<M>(h[j], h[j], ss);
        sg = fma2<M>(mul2<M>(g[j], w[KEEP ? i : 0][j]), h[j], sg);
      }
    }
    float sums[2] = {ss.x + ss.y, sg.x + sg.y};
    team_sums<WARP>(sums, red[parity]);
    parity ^= 1;
    const float rstd = 1.f / sqrtf(fmaf(sums[0], inv_cols, a.eps));
    const float mean = sums[1] * rstd * inv_cols;  // mean of weight * d_out * n
    const float2 r2 = f2_splat(rstd), nm = f2_splat(-mean);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = first_col<M, WARP>(i);
      float2 h[4], g[4], d[4], dx[4];
      get(0, hp, i, c).get(h);
      get(1, gp, i, c).get(g);
      if (!KEEP) load_weight<M>(a.weight, c, cols, w[0]);
      if (dp) get(2, dp, i, c).get(d);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 n = mul2<M>(h[j], r2);  // rstd squared may leave the range of fp32
        dw[i][j] = fma2<M>(g[j], n, dw[i][j]);
        // rstd (w g - n mean) + d
        const float2 t = fma2<M>(n, nm, mul2<M>(g[j], w[KEEP ? i : 0][j]));
        dx[j] = dp ? fma2<M>(t, r2, d[j]) : mul2<M>(t, r2);
      }
      store<T, M>(static_cast<T *>(a.dx) + row * cols, c, cols, dx);
    }
    // this thread has used its slots: its stores needed them
    fetch(row + kDepth * step, stage);
    stage = stage == kDepth - 1 ? 0 : stage + 1;
  }
  if (!a.dweight) return;
  float *part = static_cast<float *>(a.workspace) + (int64_t)blockIdx.x * cols;
  if (!WARP) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) store<float, M>(part, first_col<M, WARP>(i), cols, dw[i]);
    return;
  }
  // the warps' sums, in their order, through shared memory
  float *sum = reinterpret_cast<float *>(smem_raw);
  for (int v = 0; v < teams; ++v) {
    __syncthreads();
    if ((int)(threadIdx.x >> 5) != v) continue;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = first_col<M, WARP>(i);
      float2 f[4];
      load<float, M>(sum, c, cols).get(f);
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = v ? f2_add(f[j], dw[i][j]) : dw[i][j];
      store<float, M>(sum, c, cols, f);
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < cols; c += blockDim.x) part[c] = sum[c];
}

// dweight[c] = the sum of the partial rows: 8 columns x 64 row lanes per CTA
// (a CTA of 32 columns leaves too few of them), each lane in row order, then
// the lanes of a warp pairwise, then the warps in order.
constexpr int kSumThreads = 512;
__global__ void __launch_bounds__(kSumThreads) dweight_kernel(const float *part, int parts, int cols, float *dw) {
  __shared__ float s[kSumThreads / 32][8];
  const int col = threadIdx.x & 7, c = blockIdx.x * 8 + col;
  float v = 0.f;
  grid_start();
  if (c < cols) {
#pragma unroll 4
    for (int p = threadIdx.x >> 3; p < parts; p += kSumThreads / 8) v += part[(int64_t)p * cols + c];
  }
  v += __shfl_xor_sync(~0u, v, 8);
  v += __shfl_xor_sync(~0u, v, 16);
  if ((threadIdx.x & 31) < 8) s[threadIdx.x >> 5][col] = v;
  __syncthreads();
  if (threadIdx.x < 8 && c < cols) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < kSumThreads / 32; ++i) v += s[i][col];
    dw[c] = v;
  }
}

// ------------------------------------------------------------------ launch

struct Shape {
  Mode mode;
  bool warp;
  int vpt, threads, grid;
  size_t smem;
};

// `vecs` groups of eight columns a row, of which `tensors` x `esize` bytes an
// element travel through the ring; a CTA's threads take two each from `wide`
// of them on (four from 1,025), else one; `per_sm_threads`: the threads an SM's registers hold.
//
// Warps take a row each up to 512 columns, and up to 1,024 in the ring
// (32768 rows of bf16, forward / backward: 512 columns 21.6 / 28.5 us with a
// warp a row, 24.1 / 35.1 with a CTA; 1,024 columns 38 / 50 and 42 / 59;
// odd rows of 903 columns 52 / 90 and 43 / 60).
Shape shape_for(int64_t rows, int cols, int vecs, int tensors, int esize, int wide, int per_sm_threads, int rounds) {
  Shape s{};
  s.mode = cols % 8 != 0 ? ODD : RING;
  s.warp = vecs <= (s.mode == ODD ? 64 : 128);
  auto cta = [&](int vpt) {
    s.vpt = vpt;
    s.threads = ((vecs + vpt - 1) / vpt + 31) / 32 * 32;
  };
  if (s.warp) {
    s.vpt = vecs <= 64 ? 2 : 4;
    s.threads = 256;
    if (s.vpt == 4) per_sm_threads = 512;
  } else {
    cta(vecs < wide ? 1 : vecs <= 1024 ? 2 : 4);
    if (s.vpt == 2 && tensors > 2) per_sm_threads = 512;  // the backward's: 88 registers
  }
  s.smem = (size_t)kDepth * tensors * s.vpt * s.threads * 8 * esize;
  // rows too wide for two of them in shared memory, or for 512 threads of four: straight from memory
  if (s.mode == RING && (s.threads > 512 || s.smem > 200 * 1024)) s.mode = DIRECT;
  int per_sm = per_sm_threads / s.threads;
  if (s.mode == RING) {
    const int fit = (int)(227 * 1024 / (s.smem + 2048));
    per_sm = fit < per_sm ? fit : per_sm;
  } else {
    s.smem = s.warp ? 4096 : 0;  // the backward's sums over warps
    if (!s.warp) cta(vecs <= 512 ? 1 : vecs <= 1024 ? 2 : 4);
    per_sm = 2048 / s.threads;
  }
  if (per_sm < 1) per_sm = 1;
  const int64_t teams = s.warp ? s.threads / 32 : 1, resident = sm_count() * (int64_t)per_sm;
  const int64_t need = (rows + teams - 1) / teams;
  // Up to `rounds` CTAs in turn on each place, of at least 8 rows: SMs are not
  // equally fast (32768 x 4096: 168 us in one round, 155 in two, 140 in six).
  // A CTA alone on its SM has no neighbour to cover its start: one round.
  int64_t most = per_sm > 1 ? need / (8 * resident) : 1;
  most = resident * (most < 1 ? 1 : most > rounds ? rounds : most);
  s.grid = (int)(need < most ? need : most);
  return s;
}

template <typename A> cudaError_t launch_rows(void (*kern)(A), const Shape &s, const A &a, cudaStream_t st) {
  return launch_overlapped(kern, (unsigned)s.grid, (unsigned)s.threads, s.smem, 1, st, a);
}

template <typename T> cudaError_t norm_typed(const kda_rms_norm_args &a, cudaStream_t st) {
  // whole groups of four blocks, so that the scales past the last block get written
  const Shape s = shape_for(a.rows, a.cols, (a.cols + 511) / 512 * 64, a.residual ? 2 : 1, sizeof(T), 0, 1024, 6);
#define KDA_NORM(M_, V_, W_) return launch_rows(rms_norm_kernel<T, M_, V_, W_>, s, a, st)
  if (s.warp) {
    if (s.mode == RING) { if (s.vpt == 2) KDA_NORM(RING, 2, true); else KDA_NORM(RING, 4, true); }
    KDA_NORM(ODD, 2, true);
  }
  if (s.mode == RING) { if (s.vpt == 2) KDA_NORM(RING, 2, false); else KDA_NORM(RING, 4, false); }
  if (s.mode == DIRECT) KDA_NORM(DIRECT, 4, false);
  if (s.vpt == 1) KDA_NORM(ODD, 1, false); else if (s.vpt == 2) KDA_NORM(ODD, 2, false); else KDA_NORM(ODD, 4, false);
#undef KDA_NORM
}

template <typename T> cudaError_t bwd_typed(const kda_rms_norm_bwd_args &a, cudaStream_t st) {
  // whole groups of 16 threads: the odd layout spreads a block over them
  Shape s = shape_for(a.rows, a.cols, (a.cols + 127) / 128 * 16, a.d_residual ? 3 : 2, sizeof(T), 257, 768, 1);
  if (s.grid > kMaxParts) s.grid = kMaxParts;
  cudaError_t e;
#define KDA_BWD(M_, V_, W_) e = launch_rows(rms_norm_bwd_kernel<T, M_, V_, W_>, s, a, st)
  if (s.warp) {
    if (s.mode == RING) { if (s.vpt == 2) KDA_BWD(RING, 2, true); else KDA_BWD(RING, 4, true); }
    else KDA_BWD(ODD, 2, true);
  }
  else if (s.mode == RING) {
    if (s.vpt == 1) KDA_BWD(RING, 1, false);
    else if (s.vpt == 2) KDA_BWD(RING, 2, false);
    else KDA_BWD(RING, 4, false);
  }
  else if (s.mode == DIRECT) KDA_BWD(DIRECT, 4, false);
  else if (s.vpt == 1) KDA_BWD(ODD, 1, false);
  else if (s.vpt == 2) KDA_BWD(ODD, 2, false);
  else KDA_BWD(ODD, 4, false);
#undef KDA_BWD
  if (e != cudaSuccess || !a.dweight) return e;
  return launch_overlapped(dweight_kernel, (unsigned)((a.cols + 7) / 8), kSumThreads, 0, 1, st,
                           static_cast<const float *>(a.workspace), s.grid, a.cols, a.dweight);
}

}  // namespace

cudaError_t launch_rms_norm(const kda_rms_norm_args &a, cudaStream_t st) {
  return a.dtype == KDA_F32 ? norm_typed<float>(a, st) : norm_typed<__nv_bfloat16>(a, st);
}

size_t rms_norm_bwd_workspace(int64_t rows, int32_t cols) {
  return align256(sizeof(float) * (size_t)(rows < kMaxParts ? rows : kMaxParts) * (size_t)cols);
}

cudaError_t launch_rms_norm_bwd(const kda_rms_norm_bwd_args &a, cudaStream_t st) {
  return a.dtype == KDA_F32 ? bwd_typed<float>(a, st) : bwd_typed<__nv_bfloat16>(a, st);
}

}  // namespace kda
