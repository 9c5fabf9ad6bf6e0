// kda_lora_kernel.cuh - the kernel of the low-rank adapters, for the forward and
// the backward alike, with what its launch needs.
#pragma once

#include "kda_lora.cuh"

#include <cuda_bf16.h>

namespace kda {
namespace lora {
namespace {

constexpr int NT = 256;

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&x);
}
__device__ __forceinline__ float2 unpack2(uint32_t w) { return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); }

// Pairs of values in N bf16 pieces, the largest first (infinite ones in one).
template <int N> __device__ __forceinline__ void split(float a, float b, uint32_t (&p)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    p[i] = pack2(a, b);
    const float2 f = unpack2(p[i]);
    a = isinf(f.x) ? 0.f : a - f.x;
    b = isinf(f.y) ? 0.f : b - f.y;
  }
}

template <typename T> struct Type;
template <> struct Type<__nv_bfloat16> { static constexpr int IN = 1, U = 2; };
template <> struct Type<float> { static constexpr int IN = 3, U = 3; };

// Eight neighbouring values (of which `left` exist), vectors of V elements, as
// pairs in pieces: x[piece][pair].
template <typename T, int V> struct Eight {
  uint32_t x[Type<T>::IN][4];
  __device__ __forceinline__ void load(const T *p, int64_t left) {
    if constexpr (sizeof(T) == 2) {
      if constexpr (V == 8) {
        const uint4 r = left > 0 ? *reinterpret_cast<const uint4 *>(p) : make_uint4(0, 0, 0, 0);
        x[0][0] = r.x; x[0][1] = r.y; x[0][2] = r.z; x[0][3] = r.w;
      } else if constexpr (V == 4) {
        const uint2 r = left > 0 ? *reinterpret_cast<const uint2 *>(p) : make_uint2(0, 0);
        const uint2 s = left > 4 ? *reinterpret_cast<const uint2 *>(p + 4) : make_uint2(0, 0);
        x[0][0] = r.x; x[0][1] = r.y; x[0][2] = s.x; x[0][3] = s.y;
      } else {
        const unsigned short *q = reinterpret_cast<const unsigned short *>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[0][i] = (uint32_t)(left > 2 * i ? q[2 * i] : 0) | (uint32_t)(left > 2 * i + 1 ? q[2 * i + 1] : 0) << 16;
      }
    } else {
      float f[8];
      load_f32(p, left, f);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t s[Type<T>::IN];
        split<Type<T>::IN>(f[2 * i], f[2 * i + 1], s);
#pragma unroll
        for (int j = 0; j < Type<T>::IN; ++j) x[j][i] = s[j];
      }
    }
  }
  static __device__ __forceinline__ void load_f32(const float *p, int64_t left, float (&f)[8]) {
    if constexpr (V >= 4) {
      const float4 a = left > 0 ? *reinterpret_cast<const float4 *>(p) : make_float4(0.f, 0.f, 0.f, 0.f);
      const float4 b = left > 4 ? *reinterpret_cast<const float4 *>(p + 4) : make_float4(0.f, 0.f, 0.f, 0.f);
      f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
      f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = left > i ? p[i] : 0.f;
    }
  }
  static __device__ __forceinline__ void store(T *p, int64_t left, const float (&f)[8]) {
    if constexpr (sizeof(T) == 2) {
      const uint32_t w[4] = {pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7])};
      if constexpr (V == 8) {
        if (left > 0) *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
      } else if constexpr (V == 4) {
        if (left > 0) *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
        if (left > 4) *reinterpret_cast<uint2 *>(p + 4) = make_uint2(w[2], w[3]);
      } else {
        unsigned short *q = reinterpret_cast<unsigned short *>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (left > i) q[i] = (unsigned short)(w[i >> 1] >> (16 * (i & 1)));
      }
    } else if constexpr (V >= 4) {
      if (left > 0) *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
      if (left > 4) *reinterpret_cast<float4 *>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (left > i) p[i] = f[i];
    }
  }
};

// Eight neighbouring values as they are stored.
template <typename T, int V> struct Raw {
  uint32_t w[2 * sizeof(T)];
  __device__ __forceinline__ void load(const T *p, int64_t left) {
    if constexpr (sizeof(T) == 2) {
      Eight<T, V> e;
      e.load(p, left);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = e.x[0][i];
    } else {
      float f[8];
      Eight<T, V>::load_f32(p, left, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(f[i]);
    }
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 v = unpack2(w[i]);
        f[2 * i] = v.x;
        f[2 * i + 1] = v.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
    }
  }
};

// c += a b over pieces; products below 2^-24 of the largest are left out.
template <int NA, int NB>
__device__ __forceinline__ void mma_pieces(float (&c)[4], const uint32_t (&a)[NA][4], const uint32_t (&b0)[NB], const uint32_t (&b1)[NB]) {
  constexpr int N = NA > NB ? NA : NB;
#pragma unroll
  for (int s = N - 1; s >= 0; --s)
#pragma unroll
    for (int i = 0; i < NA; ++i)
      if (s - i >= 0 && s - i < NB) mma(c, a[i], b0[s - i], b1[s - i]);
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ float remote_f32(uint32_t addr, uint32_t rank) {
  uint32_t a;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}

struct Args {
  int64_t rows;
  int n_in, n_out, rank, adapters;
  int64_t a_ld, b_ld;      // row pitches of A [.., rank, n_in] and B [.., n_out, rank]
  int64_t a_adapter, b_adapter;
  const void *x, *a, *b, *y;
  void *out;               // null: u alone
  const void *idx;
  bool idx64, b_vec;       // b_vec: B's rows can be read four values at a time
  int requests;
  const int32_t *cu;       // or null: rows / requests rows each
  const float *scale;
  uint16_t *u_out;         // [rows, 3, RP] pieces of scale u, or null
};

// Calls that one launch takes (blockIdx.y): same rows, requests, type and rank.
struct Pair {
  Args a[2];
};

// The adapter of request n, -1 where it has none.
__device__ __forceinline__ int adapter_of(const Args &a, int n) {
  const int64_t l = a.idx64 ? static_cast<const int64_t *>(a.idx)[n] : (int64_t) static_cast<const int32_t *>(a.idx)[n];
  return l >= 0 && l < a.adapters ? (int)l : -1;
}
// Rows [r0, r1) of request n; request `requests` are the rows behind the last one.
__device__ __forceinline__ void rows_of(const Args &a, int n, int64_t &r0, int64_t &r1) {
  if (a.cu) {
    r0 = a.cu[n];
    r1 = n < a.requests ? (int64_t)a.cu[n + 1] : a.rows;
    r0 = r0 < 0 ? 0 : r0 > a.rows ? a.rows : r0;
    r1 = r1 < r0 ? r0 : r1 > a.rows ? a.rows : r1;
  } else {
    const int64_t per = a.rows / a.requests;
    r0 = n * per;
    r1 = n < a.requests ? r0 + per : a.rows;
  }
}

// Tile -> first row, rows and adapter; a warp's 32 lanes look at 32 requests at once.
// With offsets every CTA walks them: nothing for hundreds of requests, but 4,096 single rows of
// 1,024 -> 1,024 take 383 us so and 88 as rows / requests rows each.
template <int M> __device__ __forceinline__ void find_tile(const Args &a, int64_t tile, int lane, int64_t &row0, int &len, int &l) {
  len = 0;
  if (!a.cu) {
    const int64_t per = a.rows / a.requests, tp = (per + M - 1) / M;
    const int n = (int)(tile / tp);
    if (n >= a.requests) return;
    const int64_t off = tile % tp * M;
    row0 = n * per + off;
    len = (int)(per - off < M ? per - off : M);
    l = adapter_of(a, n);
    return;
  }
  int64_t before = 0;
  for (int n0 = 0; n0 <= a.requests; n0 += 32) {
    const int n = n0 + lane;
    int64_t r0 = 0, r1 = 0;
    if (n <= a.requests) rows_of(a, n, r0, r1);
    const int mine = (int)((r1 - r0 + M - 1) / M);
    int sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(~0u, sum, o);
      if (lane >= o) sum += v;
    }
    const bool here = tile >= before + sum - mine && tile < before + sum;
    const uint32_t who = __ballot_sync(~0u, here);
    if (who) {
      const int src = __ffs(who) - 1;
      const int64_t off = (tile - (before + sum - mine)) * M;
      row0 = __shfl_sync(~0u, r0 + off, src);
      len = __shfl_sync(~0u, (int)(r1 - r0 - off < M ? r1 - r0 - off : M), src);
      l = n0 + src < a.requests ? adapter_of(a, n0 + src) : -1;
      return;
    }
    before += __shfl_sync(~0u, sum, 31);
  }
}

// M rows a tile, RP ranks.  x and A pass through a ring in shared memory, KC
// columns at a time; a warp has 16 rows and KS of the steps of 16 columns (the
// warps share these KW ways).
template <typename T, int M, int RP> struct Shape {
  static constexpr int NI = Type<T>::IN;
  static constexpr int MG = M / 16, KW = 8 / MG, KC = M == 16 ? 128 : 64, UX = KC / 8, KS = KC / 16 / KW;
  static constexpr int STAGES = NI == 1 ? 4 : 2;
  static constexpr uint32_t X = M * KC * 2, A = RP * KC * 2, STAGE = NI * (X + A);
  static constexpr int PITCH = RP + 8;  // elements a row of u's pieces
  static constexpr size_t U = (size_t)M * RP * 4, RING = (size_t)STAGES * STAGE, PART = (size_t)KW * M * RP * 4,
                          PIECES = (size_t)3 * M * PITCH * 2, OVER = RING > PART ? RING : PART;
  static constexpr size_t BYTES = U + (OVER > PIECES ? OVER : PIECES);
};

// Byte offset of 16-byte unit u of row r in rows of U units, eight rows' units
// of a column in different banks.
template <int U> __device__ __forceinline__ uint32_t unit_at(int r, int u) { return (uint32_t)((r * U + (u ^ (r & 7))) * 16); }

// Eight neighbouring values, of which `left` exist, to shared memory (zeros for
// the others): asynchronously where they can be read 8 or 16 bytes at a time.
template <typename T, int V>
__device__ __forceinline__ void stage8(unsigned char *to, uint32_t piece, const T *from, int64_t left, const void *any) {
  if constexpr (sizeof(T) == 2 && V == 8) {
    const int n = left > 0 ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(to)),
                 "l"(n ? (const void *)from : any), "r"(n) : "memory");
  } else if constexpr (sizeof(T) == 2 && V == 4) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int n = left > 4 * i ? 8 : 0;
      asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(to + 8 * i)),
                   "l"(n ? (const void *)(from + 4 * i) : any), "r"(n) : "memory");
    }
  } else {
    Eight<T, V> e;
    e.load(from, left);
#pragma unroll
    for (int j = 0; j < Type<T>::IN; ++j) *reinterpret_cast<uint4 *>(to + j * piece) = make_uint4(e.x[j][0], e.x[j][1], e.x[j][2], e.x[j][3]);
  }
}

// TWO: the backward's products of one launch (blockIdx.y); u's pieces are kept.
template <typename T, int M, int RP, int V, bool TWO>
__global__ void __launch_bounds__(NT, sizeof(T) == 2 && RP <= 64 ? 2 : 1) lora_kernel(const __grid_constant__ Pair both) {
  const Args &a = both.a[TWO ? blockIdx.y : 0];
  using Sh = Shape<T, M, RP>;
  constexpr int KW = Sh::KW, NI = Type<T>::IN, NU = Type<T>::U, RT = RP / 8, PITCH = Sh::PITCH;
  extern __shared__ __align__(128) unsigned char smem[];
  float *u_s = reinterpret_cast<float *>(smem), *part = u_s + M * RP;  // the ring, then the warps' parts, then u's pieces
  unsigned char *ring = reinterpret_cast<unsigned char *>(part);
  uint16_t *pieces = reinterpret_cast<uint16_t *>(part);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const uint32_t rank = cluster_rank(), size = cluster_size();
  int64_t row0 = 0;
  int len = 0, l = -1;
  find_tile<M>(a, blockIdx.x / size, lane, row0, len, l);
  if (len == 0) return;  // the whole cluster

  if (l >= 0) {
    // ---- u = x A^T over this CTA's and warp's part of n_in
    const int mg = warp / KW, kw = warp % KW;
    const T *A = static_cast<const T *>(a.a) + l * a.a_adapter, *X = static_cast<const T *>(a.x) + row0 * a.n_in;
    const int chunks = (a.n_in + Sh::KC - 1) / Sh::KC;
    const int c0 = (int)((int64_t)chunks * rank / size), nc = (int)((int64_t)chunks * (rank + 1) / size) - c0;
    auto load = [&](int c) {
      unsigned char *st = ring + (c % Sh::STAGES) * Sh::STAGE;
      const int k0 = (c0 + c) * Sh::KC;
#pragma unroll
      for (int i = 0; i < ((M + RP) * Sh::UX + NT - 1) / NT; ++i) {
        const int x = tid + i * NT, r = x / Sh::UX, u = x % Sh::UX, k = k0 + u * 8;
        if (r >= M + RP) break;
        if (r < M) {  // rows past the end: nothing, their u is not used
          if (r < len) stage8<T, V>(st + unit_at<Sh::UX>(r, u), Sh::X, X + (int64_t)r * a.n_in + k, a.n_in - k, a.x);
        } else {
          const int q = r - M;
          stage8<T, V>(st + NI * Sh::X + unit_at<Sh::UX>(q, u), Sh::A, A + (q < a.rank ? q * a.a_ld : 0) + k, q < a.rank ? a.n_in - k : 0, a.a);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    float sum[RT][4], acc[RT][4];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[i][e] = acc[i][e] = 0.f;
    const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(ring);
    const int ra = 16 * mg + (lane & 15), ua = lane >> 4, rb = ((lane >> 4) << 3) + (lane & 7), ub = (lane >> 3) & 1;
#pragma unroll
    for (int c = 0; c < Sh::STAGES - 1; ++c) {
      if (c < nc) load(c);
      else asm volatile("cp.async.commit_group;" ::: "memory");
    }
    for (int c = 0; c < nc; ++c) {
      asm volatile("cp.async.wait_group %0;" ::"n"(Sh::STAGES - 2) : "memory");
      __syncthreads();  // chunk c is there; every warp is done with chunk c - 1, whose place is next
      if (c + Sh::STAGES - 1 < nc) load(c + Sh::STAGES - 1);
      else asm volatile("cp.async.commit_group;" ::: "memory");
      const uint32_t x_at = ring_at + (c % Sh::STAGES) * Sh::STAGE, a_at = x_at + NI * Sh::X;
#pragma unroll
      for (int ks = 0; ks < Sh::KS; ++ks) {
        const int u0 = 2 * (kw * Sh::KS + ks);
        uint32_t f[NI][4];
#pragma unroll
        for (int j = 0; j < NI; ++j) ldsm4(f[j], x_at + j * Sh::X + unit_at<Sh::UX>(ra, u0 + ua));
#pragma unroll
        for (int q = 0; q < RT / 2; ++q) {
          uint32_t b[NI][4];
#pragma unroll
          for (int j = 0; j < NI; ++j) ldsm4(b[j], a_at + j * Sh::A + unit_at<Sh::UX>(16 * q + rb, u0 + ub));
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint32_t b0[NI], b1[NI];
#pragma unroll
            for (int j = 0; j < NI; ++j) {
              b0[j] = b[j][2 * e];
              b1[j] = b[j][2 * e + 1];
            }
            mma_pieces<NI, NI>(acc[2 * q + e], f, b0, b1);
          }
        }
      }
      if ((c + 1) % (8 / Sh::KS) == 0) {
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            sum[i][e] += acc[i][e];
            acc[i][e] = 0.f;
          }
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<float2 *>(part + ((size_t)kw * M + mg * 16 + g + 8 * h) * RP + 8 * i + 2 * t) =
            make_float2(sum[i][2 * h] + acc[i][2 * h], sum[i][2 * h + 1] + acc[i][2 * h + 1]);
    __syncthreads();
    for (int i = tid; i < M * RP; i += NT) {
      float s = part[i];
#pragma unroll
      for (int w = 1; w < KW; ++w) s += part[w * M * RP + i];
      u_s[i] = s;
    }
    if (size > 1) cluster_sync();
    else __syncthreads();
    // ---- the CTAs' parts in order, times the scale, in pieces
    const float scale = a.scale ? a.scale[l] : 1.f;
    const uint32_t u_at = (uint32_t)__cvta_generic_to_shared(u_s);
    for (int i = tid * 2; i < M * RP; i += NT * 2) {
      const int r = i / RP, k = i % RP;
      float s0 = u_s[i], s1 = u_s[i + 1];
      if (size > 1) {
        s0 = remote_f32(u_at + i * 4, 0);
        s1 = remote_f32(u_at + i * 4 + 4, 0);
        for (uint32_t c = 1; c < size; ++c) {
          s0 += remote_f32(u_at + i * 4, c);
          s1 += remote_f32(u_at + i * 4 + 4, c);
        }
      }
      uint32_t p[3];
      split<3>(s0 * scale, s1 * scale, p);
#pragma unroll
      for (int j = 0; j < 3; ++j) {
        *reinterpret_cast<uint32_t *>(pieces + (j * M + r) * PITCH + k) = p[j];
        if (TWO && a.u_out && rank == 0 && r < len) *reinterpret_cast<uint32_t *>(a.u_out + ((row0 + r) * 3 + j) * RP + k) = p[j];
      }
    }
    if (size > 1) cluster_sync();  // no CTA leaves while another still reads its part
    else __syncthreads();
  }
  if (!a.out || (l < 0 && a.out == a.y)) return;

  // ---- out = y + u B^T, 32 columns a warp at a time
  const T *B = static_cast<const T *>(a.b) + (l < 0 ? 0 : l * a.b_adapter);
  const T *y = a.y ? static_cast<const T *>(a.y) + row0 * a.n_out : nullptr;
  T *out = static_cast<T *>(a.out) + row0 * a.n_out;
  const int groups = (a.n_out + COLS - 1) / COLS;
  const int g0 = (int)((int64_t)groups * rank / size), g1 = (int)((int64_t)groups * (rank + 1) / size);
  for (int cg = g0 + warp; cg < g1; cg += 8) {
    const int col = cg * COLS + 8 * t;  // this lane's eight columns
    const int64_t left = a.n_out - col;
    // B's rows: tile j, column 2 t' + e of the product is column 8 t' + 2 j + e here
    uint32_t b[4][RP / 16][NI][2];
    if (l >= 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = cg * COLS + 8 * (g >> 1) + 2 * j + (g & 1);
        const T *p = B + (c < a.n_out ? c * a.b_ld : 0);
#pragma unroll
        for (int s = 0; s < RP / 16; ++s) {
          const int r = 16 * s + 4 * t;
          const int have = c < a.n_out ? a.rank - r : 0;
          if constexpr (sizeof(T) == 2) {
            if (a.b_vec) {
              const uint2 w = have > 0 ? *reinterpret_cast<const uint2 *>(p + r) : make_uint2(0, 0);
              b[j][s][0][0] = w.x;
              b[j][s][0][1] = w.y;
            } else {
              const unsigned short *q = reinterpret_cast<const unsigned short *>(p + r);
              b[j][s][0][0] = (uint32_t)(have > 0 ? q[0] : 0) | (uint32_t)(have > 1 ? q[1] : 0) << 16;
              b[j][s][0][1] = (uint32_t)(have > 2 ? q[2] : 0) | (uint32_t)(have > 3 ? q[3] : 0) << 16;
            }
          } else {
            float f[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = have > i ? p[r + i] : 0.f;
            uint32_t q0[NI], q1[NI];
            split<NI>(f[0], f[1], q0);
            split<NI>(f[2], f[3], q1);
#pragma unroll
            for (int i = 0; i < NI; ++i) {
              b[j][s][i][0] = q0[i];
              b[j][s][i][1] = q1[i];
            }
          }
        }
      }
    }
    // y of all rows on its way before the first product
    Raw<T, V> yr[M / 16][2];
    if (y) {
#pragma unroll
      for (int m = 0; m < M / 16; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = m * 16 + g + 8 * h;
          yr[m][h].load(y + (int64_t)r * a.n_out + col, r < len ? left : 0);
        }
    }
#pragma unroll
    for (int m = 0; m < M / 16; ++m) {
      if (m * 16 >= len) break;
      float v[2][8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (y) yr[m][h].get(v[h]);
        else
#pragma unroll
          for (int i = 0; i < 8; ++i) v[h][i] = 0.f;
      }
      if (l >= 0) {
        float c[4][4] = {};
#pragma unroll
        for (int s = 0; s < RP / 16; ++s) {
          uint32_t f[NU][4];
#pragma unroll
          for (int j = 0; j < NU; ++j) {
            const uint2 lo = *reinterpret_cast<const uint2 *>(pieces + (j * M + m * 16 + g) * PITCH + 16 * s + 4 * t);
            const uint2 hi = *reinterpret_cast<const uint2 *>(pieces + (j * M + m * 16 + g + 8) * PITCH + 16 * s + 4 * t);
            f[j][0] = lo.x;
            f[j][1] = hi.x;
            f[j][2] = lo.y;
            f[j][3] = hi.y;
          }
          constexpr int N = NU > NI ? NU : NI;
#pragma unroll
          for (int w = N - 1; w >= 0; --w)
#pragma unroll
            for (int i = 0; i < NU; ++i)
              if (w - i >= 0 && w - i < NI)
#pragma unroll
                for (int j = 0; j < 4; ++j) mma(c[j], f[i], b[j][s][w - i][0], b[j][s][w - i][1]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e >> 1][2 * j + (e & 1)] += c[j][e];
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = m * 16 + g + 8 * h;
        if (r < len) Eight<T, V>::store(out + (int64_t)r * a.n_out + col, left, v[h]);
      }
    }
  }
}

// Elements of a row of n that can be read at once (up to 16 bytes).
template <typename T> int vec_of(int64_t n) { return sizeof(T) == 2 && n % 8 == 0 ? 8 : n % 4 == 0 ? 4 : 1; }

template <typename T> int min_vec(int64_t a, int64_t b) { return vec_of<T>(a) < vec_of<T>(b) ? vec_of<T>(a) : vec_of<T>(b); }

template <typename T, int M, int RP, int V, bool TWO>
cudaError_t go(const Pair &a, int n, int64_t tiles, int size, cudaStream_t st) {
  auto kernel = lora_kernel<T, M, RP, V, TWO>;
  constexpr size_t smem = Shape<T, M, RP>::BYTES;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(tiles * size), (unsigned)n);
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)size;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}
template <typename T, int M, int RP, bool TWO> cudaError_t go_vec(const Pair &a, int n, int64_t tiles, int size, cudaStream_t st) {
  const int v = min_vec<T>(a.a[0].n_in, a.a[0].n_out);  // the second's widths are these as well
  if constexpr (sizeof(T) == 2)
    if (v == 8) return go<T, M, RP, 8, TWO>(a, n, tiles, size, st);
  return v == 4 ? go<T, M, RP, 4, TWO>(a, n, tiles, size, st) : go<T, M, RP, 1, TWO>(a, n, tiles, size, st);
}
template <typename T, int M, bool TWO> cudaError_t go_rank(const Pair &a, int n, int64_t tiles, int size, cudaStream_t st) {
  switch (padded(a.a[0].rank)) {
    case 16: return go_vec<T, M, 16, TWO>(a, n, tiles, size, st);
    case 32: return go_vec<T, M, 32, TWO>(a, n, tiles, size, st);
    case 64: return go_vec<T, M, 64, TWO>(a, n, tiles, size, st);
    default: return go_vec<T, M, 128, TWO>(a, n, tiles, size, st);
  }
}

template <bool TWO> cudaError_t run(kda_dtype dt, const Pair &both, int n, cudaStream_t st) {
  const Args &a = both.a[0];
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int64_t per = a.rows / a.requests;
  auto tiles_of = [&](int m) { return a.cu ? a.rows / m + a.requests + 1 : a.requests * ((per + m - 1) / m); };
  // Rows a tile.  Where requests have up to 16 rows in the mean, and where all tiles of 16 run at once, 16: two a SM,
  // one for fp32 above rank 16.  64 x n rows, 4,096 -> 4,096, tiles of 16 / of 64, us: bf16 rank 16 n = 32 16 / 30,
  // n = 64 33 / 37, n = 96 (384 tiles) 62 / 47; rank 128 n = 64 107 / 177, n = 96 157 / 156; fp32 rank 16 n = 64 92 / 150,
  // rank 64 n = 32 158 / 214, n = 48 (192 tiles) 306 / 241.  Rows in all, not the mean, decide above 16: 64 single rows
  // beside 2,048 22.6 / 32.3, beside 4,096 51.5 / 40.7; 512 x 32 124 / 113.  Eight times 64 at rank 128 would want 64
  // (47 / 37).
  const int64_t at_once = (dt == KDA_BF16 || a.rank <= 16 ? 2 : 1) * (int64_t)sms;
  const int m = per <= 16 || n * tiles_of(16) <= at_once ? 16 : 64;
  const int64_t tiles = tiles_of(m);
  // CTAs a tile.  Tiles of 64 rows: until every SM has its two (115 tiles of 2,048 -> 4,196: 48.5 us with 4 of
  // them, 51.4 with 2; 512 tiles of 4,096 -> 4,096, enough by themselves: 230 us with 1, 277 with 4, which fill the
  // last round better but add their parts).  Tiles of 16, a few rows each, are the start and end of a CTA more
  // than anything: as many as run at once (64 tiles of 4,096 -> 4,096: 12.5 us with 4, 17.8 with 8).
  int size = 1;
  while (size < 8 && (m == 64 ? n * tiles * size < 2 * sms : n * tiles * size * 2 <= 2 * sms)) size *= 2;
  if (dt == KDA_BF16)
    return m == 16 ? go_rank<__nv_bfloat16, 16, TWO>(both, n, tiles, size, st) : go_rank<__nv_bfloat16, 64, TWO>(both, n, tiles, size, st);
  return m == 16 ? go_rank<float, 16, TWO>(both, n, tiles, size, st) : go_rank<float, 64, TWO>(both, n, tiles, size, st);
}

}  // namespace
}  // namespace lora
}  // namespace kda
