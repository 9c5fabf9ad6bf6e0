// kda_lora_bwd.cu - gradients of the low-rank adapters (kda_lora.cu):
//   du = scale dY B,  dX += du A,  dA = sum over rows of du^T x,  dB = sum over rows of scale dY^T (x A^T)
// du and dX are the forward's kernel with the matrices' roles changed (both
// transposed once), u = x A^T is it again in the same launch.  dA and dB share a
// launch too: tiles of 64 rows of one adapter, [columns, ranks] in registers,
// narrow operands in three pieces (24 bits).  32,768 rows, 4,096 and 4,096 wide, rank 64:
// du, dX and u 305 us, dA and dB 276 (their tensor-core products alone 170).
#include "kda_fill.cuh"
#include "kda_lora_kernel.cuh"

namespace kda {
namespace lora {
namespace {

// One launch for what the others want first: the row tiles of 64 of every
// adapter, in the order of the requests (a warp an adapter, requests looked at
// 1,024 at a time, a lane to a tile), and both matrices of every adapter
// transposed (32 x 32 elements a block).
struct Transpose {  // dst[l][c][r] = src[l][r][c], rows of src R; dst's row pitch ld >= R (zeros behind R)
  const void *src;
  void *dst;
  int R, C, ld;
  __host__ __device__ int64_t blocks(int L) const { return src ? (int64_t)L * ((C + 31) / 32) * ((ld + 31) / 32) : 0; }
};

// A block does one of the two.
template <typename T> union BeforeShared {
  struct {
    int l[1024], r0[1024], r1[1024];  // adapter and rows of the requests looked at
  } requests;
  T tile[32][33];
};

template <typename T>
__global__ void __launch_bounds__(256)
before_kernel(Args a, int32_t *count, int2 *list, int64_t cap, int64_t list_blocks, Transpose t0, Transpose t1) {
  __shared__ BeforeShared<T> sh;
  auto &s_l = sh.requests.l, &s_r0 = sh.requests.r0, &s_r1 = sh.requests.r1;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (blockIdx.x >= list_blocks) {
    auto &tile = sh.tile;
    int64_t b = blockIdx.x - list_blocks;
    const bool second = b >= t0.blocks(a.adapters);
    if (second) b -= t0.blocks(a.adapters);
    const Transpose &t = second ? t1 : t0;
    const int cb = (t.C + 31) / 32, rb = (t.ld + 31) / 32;
    const int c0 = (int)(b % cb) * 32, r0 = (int)(b / cb % rb) * 32;
    const int64_t l = b / cb / rb;
    const T *src = static_cast<const T *>(t.src);
    T *dst = static_cast<T *>(t.dst);
    for (int y = warp; y < 32; y += 8) {
      const int r = r0 + y, c = c0 + lane;
      tile[y][lane] = r < t.R && c < t.C ? src[(l * t.R + r) * t.C + c] : from_f32<T>(0.f);
    }
    __syncthreads();
    for (int y = warp; y < 32; y += 8) {
      const int c = c0 + y, r = r0 + lane;
      if (c < t.C && r < t.ld) dst[(l * t.C + c) * t.ld + r] = tile[lane][y];
    }
    return;
  }
  const int l = blockIdx.x * 8 + warp;
  int64_t n = 0;
  for (int n0 = 0; n0 < a.requests; n0 += 1024) {
    __syncthreads();
    const int here = min(1024, a.requests - n0);
    for (int i = threadIdx.x; i < here; i += 256) {
      int64_t r0, r1;
      rows_of(a, n0 + i, r0, r1);
      s_l[i] = adapter_of(a, n0 + i);
      s_r0[i] = (int)r0;
      s_r1[i] = (int)r1;
    }
    __syncthreads();
    if (l >= a.adapters) continue;
    for (int i0 = 0; i0 < here; i0 += 32) {
      uint32_t mine = __ballot_sync(~0u, i0 + lane < here && s_l[min(i0 + lane, 1023)] == l);
      while (mine) {
        const int i = i0 + __ffs(mine) - 1;
        mine &= mine - 1;
        const int r0 = s_r0[i], r1 = s_r1[i], tiles = (r1 - r0 + TM - 1) / TM;
        for (int k = lane; k < tiles && n + k < cap; k += 32)
          list[l * cap + n + k] = make_int2(r0 + k * TM, min(TM, r1 - r0 - k * TM));
        n = min(n + tiles, cap);
      }
    }
  }
  if (l < a.adapters && lane == 0) count[l] = (int32_t)n;
}

// Sum over an adapter's rows of wide[row, col] narrow[row, r] (narrow in three
// pieces) -> grad[l]: [col, r] (dB) or [r, col] (dA).  CTA: 8 warps, W columns
// each; share s of the tiles.
template <typename T, int RP> struct GradShape {
  static constexpr int NI = Type<T>::IN, MT = RP == 128 ? 1 : 2, W = 16 * MT, COLS = 8 * W;
  static constexpr int WP = COLS + 8, NP = 3 * RP + 8;  // row pitches in elements: eight rows' 16 bytes in different banks
  static constexpr size_t WIDE = (size_t)NI * TM * WP * 2, NARROW = (size_t)TM * NP * 2, STAGE = WIDE + NARROW;
  static constexpr int STAGES = NI == 1 ? 2 : 1;
  static constexpr size_t BYTES = STAGES * STAGE;
  static constexpr int THREADS = NT + (STAGES == 2 ? FILL : 0);
};

// One of the two gradients a launch makes.
struct Grad {
  const void *wide;
  const uint16_t *narrow;
  int n, cols;       // width, column blocks
  bool rank_rows;    // [rank, n] or [n, rank]
  float *grad;       // the shares' sums follow one another, `share` elements apart
  int64_t share;
};

template <typename T, int RP, int V>
__global__ void __launch_bounds__(GradShape<T, RP>::THREADS, 1)
grad_kernel(Grad g0, Grad g1, const int32_t *count, const int2 *list, int64_t cap, int shares, int rank) {
  using Sh = GradShape<T, RP>;
  constexpr int NI = Sh::NI, MT = Sh::MT, RT = RP / 8;
  extern __shared__ __align__(128) unsigned char smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int l = blockIdx.y;
  const bool second = (int)blockIdx.x >= g0.cols * shares;
  const Grad &gr = second ? g1 : g0;
  const int b = second ? blockIdx.x - g0.cols * shares : blockIdx.x;
  const int share = b / gr.cols, col0 = b % gr.cols * Sh::COLS, n = gr.n;
  const T *wide = static_cast<const T *>(gr.wide);
  const uint16_t *narrow = gr.narrow;
  const int tiles = count[l];
  const int i0 = (int)((int64_t)tiles * share / shares), i1 = (int)((int64_t)tiles * (share + 1) / shares);

  auto load = [&](int2 rl, unsigned char *st, int first, int step) {
    constexpr int UW = Sh::COLS / 8, UN = 3 * RP / 8;
#pragma unroll 4
    for (int x = first; x < TM * UW; x += step) {
      const int r = x / UW, u = x % UW;
      const T *from = wide + ((int64_t)rl.x + (r < rl.y ? r : 0)) * n + col0 + u * 8;
      stage8<T, V>(st + (r * Sh::WP + u * 8) * 2, TM * Sh::WP * 2, from, r < rl.y ? (int64_t)n - col0 - u * 8 : 0, wide);
    }
#pragma unroll 4
    for (int x = first; x < TM * UN; x += step) {
      const int r = x / UN, u = x % UN;
      const int bytes = r < rl.y ? 16 : 0;
      const uint16_t *from = narrow + ((int64_t)rl.x + (r < rl.y ? r : 0)) * 3 * RP + u * 8;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                       (uint32_t)__cvta_generic_to_shared(st + Sh::WIDE + (r * Sh::NP + u * 8) * 2)),
                   "l"(from), "r"(bytes) : "memory");
    }
  };
  if constexpr (Sh::STAGES == 2) {
    if (warp >= 8) {
      registers_to_fill<8>();
      int2 next = i0 < i1 ? list[l * cap + i0] : make_int2(0, 0);  // a tile's place in memory is read one tile ahead
      fill_buffers<2>(i1 - i0, [&](int i) {
        const int2 rl = next;
        if (i0 + i + 1 < i1) next = list[l * cap + i0 + i + 1];
        load(rl, smem + (i & 1) * Sh::STAGE, tid - NT, FILL);
      });
      return;
    }
    registers_to_compute<8>();
  }

  float sum[MT][RT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[m][i][e] = 0.f;
  // transposed on the way: left operand [columns, rows], right operand [rows, ranks]
  const int ra = ((lane >> 4) << 3) + (lane & 7), ua = (lane >> 3) & 1;
  const int rb = (((lane >> 3) & 1) << 3) + (lane & 7), ub = lane >> 4;
  for (int i = i0; i < i1; ++i) {
    const int stage = Sh::STAGES == 2 ? (i - i0) & 1 : 0;
    unsigned char *st = smem + stage * Sh::STAGE;
    if constexpr (Sh::STAGES == 2) {
      bar_sync(bar_full(stage, warp >> 2), GROUP + FILL);
    } else {
      load(list[l * cap + i], st, tid, NT);
      cp_commit();
      cp_wait<0>();
      __syncthreads();
    }
    const uint32_t w0 = (uint32_t)__cvta_generic_to_shared(st), n0 = w0 + (uint32_t)Sh::WIDE;
    float acc[MT][RT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < RT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[m][j][e] = 0.f;
#pragma unroll 2
    for (int ks = 0; ks < TM / 16; ++ks) {
      uint32_t f[MT][NI][4];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < NI; ++j)
          ldsm4t(f[m][j], w0 + ((j * TM + 16 * ks + ra) * Sh::WP + warp * Sh::W + 16 * m + 8 * ua) * 2);
      // products of one pair of pieces on all tiles in a row: none waits for the sum of the one before
      constexpr int Q = RT == 2 ? 1 : 2;
#pragma unroll
      for (int q0 = 0; q0 < RT / 2; q0 += Q) {
        uint32_t b[Q][3][4];
#pragma unroll
        for (int q = 0; q < Q; ++q)
#pragma unroll
          for (int j = 0; j < 3; ++j) ldsm4t(b[q][j], n0 + ((16 * ks + rb) * Sh::NP + j * RP + 16 * (q0 + q) + 8 * ub) * 2);
#pragma unroll
        for (int s = 2; s >= 0; --s)
#pragma unroll
          for (int i = 0; i < NI && i <= s; ++i)
#pragma unroll
            for (int q = 0; q < Q; ++q)
#pragma unroll
              for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int m = 0; m < MT; ++m) mma(acc[m][2 * (q0 + q) + e], f[m][i], b[q][s - i][2 * e], b[q][s - i][2 * e + 1]);
      }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < RT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[m][j][e] += acc[m][j][e];
    if constexpr (Sh::STAGES == 1) __syncthreads();
    else if (i + 2 < i1) bar_arrive(bar_empty(stage, warp >> 2), GROUP + FILL);
  }
  float *to = gr.grad + share * gr.share + (int64_t)l * n * rank;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = col0 + warp * Sh::W + 16 * m + g + 8 * (e >> 1), r = 8 * i + 2 * t + (e & 1);
        if (c < n && r < rank) to[gr.rank_rows ? (int64_t)r * n + c : (int64_t)c * rank + r] = sum[m][i][e];
      }
}

// The shares' sums in order, of both gradients.
__global__ void __launch_bounds__(256) shares_kernel(Grad g0, Grad g1, int shares, float *out0, float *out1) {
  const int64_t n0 = g0.share, n = n0 + g1.share;
  for (int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x; x < n; x += (int64_t)gridDim.x * 256) {
    const bool second = x >= n0;
    const float *part = second ? g1.grad : g0.grad;
    const int64_t i = second ? x - n0 : x, step = second ? g1.share : n0;
    float s = part[i];
    for (int k = 1; k < shares; ++k) s += part[k * step + i];
    (second ? out1 : out0)[i] = s;
  }
}

template <typename T, int RP, int V>
cudaError_t grad_go(Grad g0, Grad g1, const int32_t *count, const int2 *list, int64_t cap, int L, int shares, int rank, cudaStream_t st) {
  using Sh = GradShape<T, RP>;
  auto kernel = grad_kernel<T, RP, V>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Sh::BYTES);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)((g0.cols + g1.cols) * shares), (unsigned)L);
  kernel<<<grid, Sh::THREADS, Sh::BYTES, st>>>(g0, g1, count, list, cap, shares, rank);
  return cudaGetLastError();
}
template <typename T, int RP>
cudaError_t grad_vec(Grad g0, Grad g1, const int32_t *count, const int2 *list, int64_t cap, int L, int shares, int rank, cudaStream_t st) {
  const int v = min_vec<T>(g0.n, g1.n);
  if constexpr (sizeof(T) == 2)
    if (v == 8) return grad_go<T, RP, 8>(g0, g1, count, list, cap, L, shares, rank, st);
  return v == 4 ? grad_go<T, RP, 4>(g0, g1, count, list, cap, L, shares, rank, st)
                : grad_go<T, RP, 1>(g0, g1, count, list, cap, L, shares, rank, st);
}
template <typename T>
cudaError_t grad_rank(int rp, Grad g0, Grad g1, const int32_t *count, const int2 *list, int64_t cap, int L, int shares, int rank, cudaStream_t st) {
  switch (rp) {
    case 16: return grad_vec<T, 16>(g0, g1, count, list, cap, L, shares, rank, st);
    case 32: return grad_vec<T, 32>(g0, g1, count, list, cap, L, shares, rank, st);
    case 64: return grad_vec<T, 64>(g0, g1, count, list, cap, L, shares, rank, st);
    default: return grad_vec<T, 128>(g0, g1, count, list, cap, L, shares, rank, st);
  }
}

inline int grad_cols(int n, int rp) { return (n + (rp == 128 ? 127 : 255)) / (rp == 128 ? 128 : 256); }

// Shares of the rows, at least 512 in each: of up to eight the number that
// leaves the fewest SMs idle in its last round, the smaller of two alike.
int shares_of(int64_t ctas, int64_t rows, int sms) {
  int best = 1;
  double most = 0;
  for (int s = 1; s <= 8 && (s == 1 || rows >= 512 * (int64_t)s); ++s) {
    const int64_t rounds = (ctas * s + sms - 1) / sms;
    const double busy = (double)(ctas * s) / (double)(rounds * sms);
    if (busy > most * 1.02) {
      most = busy;
      best = s;
    }
  }
  return best;
}

}  // namespace

BwdPlan bwd_plan(const kda_lora_bwd_args &a, int sms) {
  BwdPlan p{};
  const size_t e = a.dtype == KDA_BF16 ? 2 : 4, L = a.adapters, rp = padded(a.rank);
  p.tiles = a.rows / TM + a.num_requests;
  const int64_t ctas = ((a.d_a ? grad_cols(a.n_in, (int)rp) : 0) + (a.d_b ? grad_cols(a.n_out, (int)rp) : 0)) * (int64_t)L;
  p.shares = ctas ? shares_of(ctas, a.rows, sms) : 1;
  const size_t one = L * a.rank * ((a.d_a ? (size_t)a.n_in : 0) + (a.d_b ? (size_t)a.n_out : 0)) * 4;
  size_t o = 256;
  p.off_at = o; o = align256(o + L * a.n_in * rp * e);
  p.off_bt = o; o = align256(o + L * a.rank * a.n_out * e);
  p.off_u = o; o = align256(o + (size_t)a.rows * 3 * rp * 2);
  p.off_du = o; o = align256(o + (size_t)a.rows * 3 * rp * 2);
  p.off_count = o; o = align256(o + L * 4);
  p.off_list = o; o = align256(o + L * p.tiles * 8);
  p.off_part = o; o = align256(o + (p.shares > 1 ? p.shares * one : 0));
  p.total = o;
  return p;
}

cudaError_t launch_lora_bwd(const kda_lora_bwd_args &x, const BwdPlan &p, cudaStream_t st) {
  char *ws = static_cast<char *>(x.workspace);
  const int rp = padded(x.rank), L = x.adapters;
  const bool bf = x.dtype == KDA_BF16;
  const bool rows = x.rows > 0, du = rows && (x.d_x || x.d_a), u = rows && x.d_b;
  Args a{};
  a.rows = x.rows;
  a.rank = x.rank; a.adapters = L;
  a.idx = x.idx;
  a.idx64 = x.idx_dtype == KDA_I64;
  a.b_vec = true;
  a.requests = x.num_requests;
  a.cu = x.cu_seqlens;
  a.scale = x.scale;
  Pair both{};
  int calls = 0;
  if (du) {  // du = dY B, then dX = dX + du A: the forward with the matrices' roles changed
    Args &c = both.a[calls++] = a;
    c.n_in = x.n_out; c.n_out = x.n_in;
    c.a_ld = x.n_out; c.b_ld = rp;
    c.a_adapter = (int64_t)x.rank * x.n_out;
    c.b_adapter = (int64_t)x.n_in * rp;
    c.x = x.d_out; c.a = ws + p.off_bt; c.b = ws + p.off_at; c.y = x.d_x_in; c.out = x.d_x;
    c.u_out = x.d_a ? reinterpret_cast<uint16_t *>(ws + p.off_du) : nullptr;
  }
  if (u) {  // u = x A^T alone
    Args &c = both.a[calls++] = a;
    c.n_in = x.n_in; c.n_out = x.n_out;
    c.a_ld = x.n_in;
    c.a_adapter = (int64_t)x.rank * x.n_in;
    c.x = x.x; c.a = x.a;
    c.u_out = reinterpret_cast<uint16_t *>(ws + p.off_u);
  }
  int32_t *count = reinterpret_cast<int32_t *>(ws + p.off_count);
  int2 *list = reinterpret_cast<int2 *>(ws + p.off_list);
  const bool grads = x.d_a || x.d_b;
  Transpose t0{}, t1{};
  if (du) t0 = Transpose{x.b, ws + p.off_bt, x.n_out, x.rank, x.n_out};
  if (du && x.d_x) t1 = Transpose{x.a, ws + p.off_at, x.rank, x.n_in, rp};
  const int64_t list_blocks = grads ? (L + 7) / 8 : 0, before = list_blocks + t0.blocks(L) + t1.blocks(L);
  if (before > INT32_MAX) return cudaErrorInvalidValue;
  cudaError_t e = cudaSuccess;
  if (before > 0) {
    if (bf) before_kernel<__nv_bfloat16><<<(unsigned)before, 256, 0, st>>>(a, count, list, p.tiles, list_blocks, t0, t1);
    else before_kernel<float><<<(unsigned)before, 256, 0, st>>>(a, count, list, p.tiles, list_blocks, t0, t1);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess && calls) e = run<true>(x.dtype, both, calls, st);
  if (e != cudaSuccess || !grads) return e;
  float *part = reinterpret_cast<float *>(ws + p.off_part);
  const bool shared = p.shares > 1;
  Grad ga{}, gb{};
  ga.n = gb.n = x.d_a ? x.n_in : x.n_out;
  if (x.d_a) {
    ga = Grad{x.x, reinterpret_cast<const uint16_t *>(ws + p.off_du), x.n_in, grad_cols(x.n_in, rp), true, shared ? part : x.d_a,
              (int64_t)L * x.n_in * x.rank};
    part += p.shares * ga.share;
  }
  if (x.d_b)
    gb = Grad{x.d_out, reinterpret_cast<const uint16_t *>(ws + p.off_u), x.n_out, grad_cols(x.n_out, rp), false, shared ? part : x.d_b,
              (int64_t)L * x.n_out * x.rank};
  e = bf ? grad_rank<__nv_bfloat16>(rp, ga, gb, count, list, p.tiles, L, p.shares, x.rank, st)
         : grad_rank<float>(rp, ga, gb, count, list, p.tiles, L, p.shares, x.rank, st);
  if (e != cudaSuccess || !shared) return e;
  const int64_t blocks = (ga.share + gb.share + 1023) / 1024;
  shares_kernel<<<(unsigned)(blocks < 2048 ? blocks : 2048), 256, 0, st>>>(ga, gb, p.shares, x.d_a, x.d_b);
  return cudaGetLastError();
}

}  // namespace lora
}  // namespace kda
