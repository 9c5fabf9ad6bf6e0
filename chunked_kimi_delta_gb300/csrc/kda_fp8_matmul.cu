// kda_fp8_matmul.cu - matrix product of scaled 8-bit matrices on the tensor
// cores: out[m, n] = sum over blocks b of 128 of 2^(ea + eb) sum_k a b.
//
// The scales are powers of two, so the block-scaled MMA (kind::mxf8f6f4, one
// UE8M0 byte for 32 of k, the same byte for the four steps of a block)
// applies them inside the tensor core: products are exact, the running sum is
// fp32 in tensor memory, and no CUDA core touches it before the end.
//
// Tiles.  The 128 lanes of an accumulator are 128 columns n of the output
// (operand b, "lane side"), its columns are rows m of the output (operand a,
// "column side", `width` of them).  Few rows m then cost a narrow tile and
// not a padded one, and a warp of the epilogue writes 32 neighbouring columns
// n of a row with one instruction whatever the alignment of `out`.
// Both operands come in by TMA as 128-byte-wide swizzled boxes of one block
// of k: K-major where k is contiguous, MN-major where it is not, so no form
// needs a transposed copy.  Edges are zeros from TMA.
//
// Scales.  Stored words (four blocks of k of one row) are what a column of
// tensor memory holds: word of row r at lane r % 32, column r / 32, the same
// in all four lane quarters.  Four warps load them from global memory and
// store them to tensor memory (tcgen05.st), each its lane quarter, a ring of
// words ahead of the MMAs.
#include <cuda_bf16.h>

#include "kda_fp8.cuh"
#include "kda_tc.cuh"

namespace kda {
namespace {

using tcp::globaltimer;

constexpr int SF_COLS = 16;       // tensor-memory columns of one ring entry: 4 lane side, 8 column side
constexpr int SF_RING = 4;
constexpr int MAX_STAGES = 8;
constexpr uint32_t LANE_BYTES = 16384;  // lane-side box: 128 x 128 bytes

struct MmArgs {
  const uint8_t *lane_scales, *col_scales;
  int64_t tile_i, tile_k;  // lane-side TILE scales: strides of the block of n and of k; tile_i = 0: words
  int lanes, cols, kblocks;  // n, m, ceil(k / 128)
  int width;                 // columns of a tile (rows m)
  int stages;
  uint32_t stage_bytes, col_box_bytes;
  uint32_t idesc;
  uint32_t lane_step, col_step;  // descriptor units per 32 of k
  bool lane_mn, col_mn;          // MN-major operands
  int lane_tiles, tiles, splits;
  void *out;
  int64_t ldo;
  uint32_t *err;
  bool test_wait;
};

struct Bars {
  uint64_t full[MAX_STAGES], empty[MAX_STAGES];
  uint64_t sf_full[SF_RING], sf_empty[SF_RING];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t never;
  uint32_t tmem;
  volatile uint32_t abort;
};

// ---- cluster helpers
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer_addr(const volatile void *p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(tc::smem_u32(const_cast<const void *>(p))), "r"(rank));
  return a;
}
__device__ __forceinline__ void arrive_remote(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" :: "r"(bar) : "memory");
}
__device__ __forceinline__ bool try_wait_cluster(uint64_t *bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok) : "r"(tc::smem_u32(bar)), "r"(parity) : "memory");
  return ok != 0;
}

// Bounded wait.  The first wait of a cluster that runs out records the
// timeout and tells every CTA of the cluster, whose waits then end too.
__device__ bool mm_wait_slow(uint64_t *bar, uint32_t parity, Bars *b, uint32_t *err, uint32_t cluster_ctas,
                             unsigned long long limit_ns) {
  const unsigned long long t0 = globaltimer();
  while (true) {
    for (int i = 0; i < 64; ++i)
      if (try_wait_cluster(bar, parity)) return true;
    if (b->abort) return false;
    if (globaltimer() - t0 > limit_ns) {
      atomicOr(err, DEV_ERR_TIMEOUT);
      for (uint32_t r = 0; r < cluster_ctas; ++r)
        asm volatile("st.shared::cluster.u32 [%0], %1;" :: "r"(peer_addr(&b->abort, r)), "r"(1u) : "memory");
      return false;
    }
  }
}
__device__ __forceinline__ bool mm_wait(uint64_t *bar, uint32_t parity, Bars *b, uint32_t *err, uint32_t cluster_ctas) {
  return try_wait_cluster(bar, parity) || mm_wait_slow(bar, parity, b, err, cluster_ctas, tcp::WAIT_LIMIT_NS);
}

// ---- tensor memory and MMA, for one CTA or a pair
template <bool PAIR> __device__ __forceinline__ void mm_alloc(uint32_t *dst, uint32_t cols) {
  if (PAIR)
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                 :: "r"(tc::smem_u32(dst)), "r"(cols) : "memory");
  else
    tc::tmem_alloc(dst, cols);
  if (PAIR) asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  else tc::tmem_relinquish();
}
template <bool PAIR> __device__ __forceinline__ void mm_dealloc(uint32_t addr, uint32_t cols) {
  if (PAIR)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" :: "r"(addr), "r"(cols) : "memory");
  else
    tc::tmem_dealloc(addr, cols);
}
template <bool PAIR>
__device__ __forceinline__ void mma_scaled(uint32_t d, uint64_t lane_desc, uint64_t col_desc, uint32_t idesc,
                                           uint32_t sf_lane, uint32_t sf_col, bool accumulate) {
  if (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        :: "r"(d), "l"(lane_desc), "l"(col_desc), "r"(idesc), "r"(sf_lane), "r"(sf_col), "r"(accumulate ? 1u : 0u)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        :: "r"(d), "l"(lane_desc), "l"(col_desc), "r"(idesc), "r"(sf_lane), "r"(sf_col), "r"(accumulate ? 1u : 0u)
        : "memory");
}
// Arrival (in both CTAs of a pair) when this thread's MMAs so far have completed.
template <bool PAIR> __device__ __forceinline__ void mm_commit(uint64_t *bar) {
  if (PAIR)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
        :: "r"(tc::smem_u32(bar)), "h"((uint16_t)3) : "memory");
  else
    tc::mma_commit(bar);
}
// TMA box into this CTA's shared memory, its bytes counted on a barrier of
// the pair's first CTA.
__device__ __forceinline__ void tma_load_pair(void *dst, const CUtensorMap *map, uint32_t bar, int32_t x, int32_t y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];"
      :: "r"(tc::smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint32_t (&r)[4]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};"
               :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
               :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// ---- scales
constexpr uint32_t WORD_ONE = FP8_SCALE_ONE * 0x01010101u;

__device__ __forceinline__ uint32_t scale_word(const uint8_t *s, int64_t rows, int64_t row, int w) {
  return row < rows ? __ldg(reinterpret_cast<const uint32_t *>(s) + w * rows + row) : WORD_ONE;
}
// The four blocks of k of word w for the 128 lane-side rows from l0 on.
__device__ __forceinline__ uint32_t tile_word(const MmArgs &a, int l0, int w) {
  uint32_t word = WORD_ONE;
  if (l0 < a.lanes) {
    word = 0;
    const uint8_t *p = a.lane_scales + (l0 / FP8_BLOCK) * a.tile_i;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int kb = 4 * w + j;
      word |= (kb < a.kblocks ? (uint32_t)__ldg(p + kb * a.tile_k) : FP8_SCALE_ONE) << (8 * j);
    }
  }
  return word;
}
// One ring entry into this warp's lane quarter.
__device__ __forceinline__ void load_scales(const MmArgs &a, int l0, int c0, int w, int lane, uint32_t (&ls)[4],
                                            uint32_t (&cs)[8]) {
  if (a.tile_i) {
    ls[0] = ls[1] = ls[2] = ls[3] = tile_word(a, l0, w);
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c) ls[c] = scale_word(a.lane_scales, a.lanes, (int64_t)l0 + 32 * c + lane, w);
  }
#pragma unroll
  for (int c = 0; c < 8; ++c)
    cs[c] = 32 * c < a.width ? scale_word(a.col_scales, a.cols, (int64_t)c0 + 32 * c + lane, w) : WORD_ONE;
}
__device__ __forceinline__ void store_scales(uint32_t tmem_sf, int quarter, const uint32_t (&ls)[4], const uint32_t (&cs)[8]) {
  const uint32_t t = tmem_sf + ((uint32_t)(32 * quarter) << 16);
  tmem_st4(t, ls);
  tmem_st8(t + 4, cs);
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
  tc::tc_fence_before();
}

// The four MMAs of one block of k.
template <bool PAIR>
__device__ __forceinline__ void mma_block(const MmArgs &a, uint32_t acc, uint32_t stage_addr, uint32_t sf, int kb,
                                          bool first) {
  const uint64_t ld = a.lane_mn ? tc::smem_desc_sw128(stage_addr, 16384, 1024) : tc::smem_desc_sw128(stage_addr, 16, 1024);
  const uint64_t cd = a.col_mn ? tc::smem_desc_sw128(stage_addr + LANE_BYTES, 16384, 1024)
                               : tc::smem_desc_sw128(stage_addr + LANE_BYTES, 16, 1024);
  const uint32_t idesc = a.idesc | (uint32_t)(kb & 3) << 4 | (uint32_t)(kb & 3) << 29;  // byte of the scale words
#pragma unroll
  for (int j = 0; j < 4; ++j)
    mma_scaled<PAIR>(acc, ld + (uint64_t)(j * a.lane_step), cd + (uint64_t)(j * a.col_step), idesc, sf, sf + 4,
                     !(first && j == 0));
}

// 32 accumulator columns (rows m from m0 on, below `end`) of this warp's lanes (columns n).
template <typename T>
__device__ __forceinline__ void store_columns(const MmArgs &a, const uint32_t (&r)[32], int n, int m0, int end) {
  if (n >= a.lanes) return;
  T *p = static_cast<T *>(a.out) + (int64_t)m0 * a.ldo + n;
#pragma unroll
  for (int c = 0; c < 32; ++c)
    if (m0 + c < end) p[c * a.ldo] = from_f32<T>(__uint_as_float(r[c]));
}

// The last arrivals of MMA commits on a ring of `size` barriers used `count`
// times: a CTA leaves only when none is still to come.
__device__ __forceinline__ void ring_drain(uint64_t *ring, int size, int count, Bars *b, uint32_t *err,
                                           uint32_t cluster_ctas) {
  for (int i = count > size ? count - size : 0; i < count; ++i)
    if (!mm_wait(ring + i % size, (i / size) & 1, b, err, cluster_ctas)) return;
}

__device__ __forceinline__ uint8_t *align1024(uint8_t *p) {
  return reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}

// After a timeout: copies and MMAs in flight end by themselves within
// microseconds; give them a millisecond before memory is released.
__device__ __forceinline__ void settle() {
  const unsigned long long t0 = globaltimer();
  while (globaltimer() - t0 < 1000000ull) {
  }
}

// ------------------------------------------------------------ many tiles
// Persistent CTA pairs: 256 columns n x width rows m per tile, one pair-wide
// MMA (cta_group::2) on each CTA's 128 lanes and half of the column side.
// Two accumulators: the epilogue of a tile runs under the next one's MMAs.
// Warps 0-3 scales, 4-11 epilogue, 12 TMA, 13 MMA (first CTA of the pair).
constexpr int PAIR_THREADS = 448;
constexpr int PAIR_MAX_WIDTH = 224;  // two accumulators and the scale ring fill the 512 columns
constexpr uint32_t PAIR_SF = 2 * PAIR_MAX_WIDTH;

template <typename T>
__global__ void __launch_bounds__(PAIR_THREADS, 1) fp8_matmul_pair_kernel(const __grid_constant__ CUtensorMap lane_map,
                                                                          const __grid_constant__ CUtensorMap col_map,
                                                                          const __grid_constant__ MmArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Bars b;
  uint8_t *sm = align1024(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int i = 0; i < a.stages; ++i) {
      tc::mbar_init(b.full + i, 1);
      tc::mbar_init(b.empty + i, 1);
    }
    for (int i = 0; i < SF_RING; ++i) {
      tc::mbar_init(b.sf_full + i, 8);   // four warps of each CTA
      tc::mbar_init(b.sf_empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(b.acc_full + i, 1);
      tc::mbar_init(b.acc_empty + i, 16);  // eight warps of each CTA
    }
    tc::mbar_init(&b.never, 1);
    b.abort = 0;
    tc::mbar_fence_init();
  }
  if (warp == 0) mm_alloc<true>(&b.tmem, 512);
  __syncthreads();
  tc::tc_fence_before();
  cluster_sync();
  tc::tc_fence_after();
  const uint32_t tmem = b.tmem;

  auto lane0_of = [&](int t) { return (t % a.lane_tiles) * 256 + (int)rank * 128; };  // this CTA's first n
  auto col0_of = [&](int t) { return (t / a.lane_tiles) * a.width; };                 // the tile's first m

  if (warp < 4) {  // scales
    int it = 0;
    bool ok = true;
    for (int t = pair; t < a.tiles && ok; t += pairs) {
      for (int w = 0; w < (a.kblocks + 3) / 4; ++w, ++it) {
        uint32_t ls[4], cs[8];
        load_scales(a, lane0_of(t), col0_of(t), w, lane, ls, cs);
        const int e = it % SF_RING;
        ok = __all_sync(~0u, mm_wait(b.sf_empty + e, ((it / SF_RING) & 1) ^ 1, &b, a.err, 2));
        if (!ok) break;
        store_scales(tmem + PAIR_SF + e * SF_COLS, warp, ls, cs);
        if (lane == 0) arrive_remote(peer_addr(b.sf_full + e, 0));
      }
    }
    if (ok) ring_drain(b.sf_empty, SF_RING, it, &b, a.err, 2);
    __syncwarp();
  } else if (warp < 12) {  // epilogue
    int it = 0;
    for (int t = pair; t < a.tiles; t += pairs, ++it) {
      const int buf = it & 1;
      if (!__all_sync(~0u, mm_wait(b.acc_full + buf, (it >> 1) & 1, &b, a.err, 2))) break;
      tc::tc_fence_after();
      const int n = lane0_of(t) + 32 * (warp & 3) + lane;
      const uint32_t acc = tmem + buf * PAIR_MAX_WIDTH + ((uint32_t)(32 * (warp & 3)) << 16);
      const int chunks = a.width / 32;
      for (int ch = (warp - 4) >> 2; ch < chunks; ch += 2) {
        uint32_t r[32];
        tmem_ld32(acc + 32 * ch, r);
        tc::tmem_ld_wait();
        store_columns<T>(a, r, n, col0_of(t) + 32 * ch, min(a.cols, col0_of(t) + a.width));
      }
      tc::tc_fence_before();
      if (lane == 0) arrive_remote(peer_addr(b.acc_empty + buf, 0));
      __syncwarp();
    }
  } else if (warp == 12) {  // TMA
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int t = pair; t < a.tiles && ok; t += pairs) {
        const int l0 = lane0_of(t), c0 = col0_of(t) + (int)rank * (a.width / 2);
        for (int kb = 0; kb < a.kblocks; ++kb, ++it) {
          const int s = it % a.stages;
          ok = mm_wait(b.empty + s, ((it / a.stages) & 1) ^ 1, &b, a.err, 2);
          if (!ok) break;
          if (rank == 0) tc::mbar_arrive_expect_tx(b.full + s, 2 * (LANE_BYTES + a.col_box_bytes));
          const uint32_t bar = peer_addr(b.full + s, 0);
          uint8_t *dst = sm + s * a.stage_bytes;
          const int k0 = kb * FP8_BLOCK;
          tma_load_pair(dst, &lane_map, bar, a.lane_mn ? l0 : k0, a.lane_mn ? k0 : l0);
          tma_load_pair(dst + LANE_BYTES, &col_map, bar, a.col_mn ? c0 : k0, a.col_mn ? k0 : c0);
        }
      }
      if (ok) ring_drain(b.empty, a.stages, it, &b, a.err, 2);
    }
    __syncwarp();
  } else if (rank == 0) {  // MMA
    if (lane == 0) {
      bool ok = !a.test_wait || mm_wait_slow(&b.never, 0, &b, a.err, 2, 1000000ull);
      int it = 0, is = 0, ia = 0;
      for (int t = pair; t < a.tiles && ok; t += pairs, ++ia) {
        const int buf = ia & 1;
        ok = mm_wait(b.acc_empty + buf, ((ia >> 1) & 1) ^ 1, &b, a.err, 2);
        if (!ok) break;
        tc::tc_fence_after();
        for (int kb = 0; kb < a.kblocks; ++kb, ++it) {
          const int e = is % SF_RING, s = it % a.stages;
          if ((kb & 3) == 0) {
            ok = mm_wait(b.sf_full + e, (is / SF_RING) & 1, &b, a.err, 2);
            if (!ok) break;
          }
          ok = mm_wait(b.full + s, (it / a.stages) & 1, &b, a.err, 2);
          if (!ok) break;
          tc::tc_fence_after();
          mma_block<true>(a, tmem + buf * PAIR_MAX_WIDTH, tc::smem_u32(sm + s * a.stage_bytes),
                          tmem + PAIR_SF + e * SF_COLS, kb, kb == 0);
          mm_commit<true>(b.empty + s);
          if ((kb & 3) == 3 || kb == a.kblocks - 1) {
            mm_commit<true>(b.sf_empty + e);
            ++is;
          }
        }
        if (ok) mm_commit<true>(b.acc_full + buf);
      }
    }
    __syncwarp();
  }
  __syncthreads();
  if (b.abort) settle();
  tc::tc_fence_before();
  cluster_sync();
  tc::tc_fence_after();
  if (warp == 0) mm_dealloc<true>(tmem, 512);
}

// ------------------------------------------------------------ few tiles
// One tile of 128 columns n x width rows m for a cluster of `splits` CTAs,
// each with its own range of k; the partial sums meet through distributed
// shared memory and are added in the order of k.
// Warps 0-3 scales, then epilogue; 4 TMA, 5 MMA.
constexpr int SPLIT_THREADS = 192;
constexpr int SPLIT_MAX_WIDTH = 128;
constexpr uint32_t SPLIT_TMEM = 256;  // two CTAs fit an SM

template <typename T>
__global__ void __launch_bounds__(SPLIT_THREADS, 2) fp8_matmul_split_kernel(const __grid_constant__ CUtensorMap lane_map,
                                                                            const __grid_constant__ CUtensorMap col_map,
                                                                            const __grid_constant__ MmArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Bars b;
  uint8_t *sm = align1024(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank(), splits = a.splits;
  const int tile = blockIdx.x / splits;
  const int l0 = (tile % a.lane_tiles) * 128, c0 = (tile / a.lane_tiles) * a.width;
  const int kb0 = (int)((int64_t)a.kblocks * rank / splits), kb1 = (int)((int64_t)a.kblocks * (rank + 1) / splits);

  if (threadIdx.x == 0) {
    for (int i = 0; i < a.stages; ++i) {
      tc::mbar_init(b.full + i, 1);
      tc::mbar_init(b.empty + i, 1);
    }
    for (int i = 0; i < SF_RING; ++i) {
      tc::mbar_init(b.sf_full + i, 4);
      tc::mbar_init(b.sf_empty + i, 1);
    }
    tc::mbar_init(b.acc_full, 1);
    tc::mbar_init(&b.never, 1);
    b.abort = 0;
    tc::mbar_fence_init();
  }
  if (warp == 0) mm_alloc<false>(&b.tmem, SPLIT_TMEM);
  tc::tc_fence_before();
  __syncthreads();
  if (splits > 1) cluster_sync();  // `abort` of every CTA is set before a peer may write it
  tc::tc_fence_after();
  const uint32_t tmem = b.tmem, tmem_sf = tmem + SPLIT_MAX_WIDTH;

  if (warp < 4) {
    bool ok = true;
    int it = 0;
    for (int w = kb0 >> 2; 4 * w < kb1; ++w, ++it) {
      uint32_t ls[4], cs[8];
      load_scales(a, l0, c0, w, lane, ls, cs);
      const int e = it % SF_RING;
      ok = __all_sync(~0u, mm_wait(b.sf_empty + e, ((it / SF_RING) & 1) ^ 1, &b, a.err, splits));
      if (!ok) break;
      store_scales(tmem_sf + e * SF_COLS, warp, ls, cs);
      if (lane == 0) tc::mbar_arrive(b.sf_full + e);
    }
    if (ok) ring_drain(b.sf_empty, SF_RING, it, &b, a.err, splits);
    __syncwarp();
    ok = ok && __all_sync(~0u, mm_wait(b.acc_full, 0, &b, a.err, splits));
    tc::tc_fence_after();
    const int n = l0 + 32 * warp + lane;
    float *part = reinterpret_cast<float *>(sm);  // [columns][128]: the stages are free now
    const int valid = min(a.width, a.cols - c0);
    if (ok)
      for (int ch = 0; 32 * ch < valid; ++ch) {
        uint32_t r[32];
        tmem_ld32(tmem + 32 * ch + ((uint32_t)(32 * warp) << 16), r);
        tc::tmem_ld_wait();
        if (splits == 1) {
          store_columns<T>(a, r, n, c0 + 32 * ch, c0 + valid);
        } else {
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (32 * ch + c < valid) part[(32 * ch + c) * 128 + 32 * warp + lane] = __uint_as_float(r[c]);
        }
      }
    tc::tc_fence_before();
  } else if (warp == 4) {
    if (lane == 0) {
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb) {
        const int it = kb - kb0, s = it % a.stages;
        ok = mm_wait(b.empty + s, ((it / a.stages) & 1) ^ 1, &b, a.err, splits);
        if (!ok) break;
        tc::mbar_arrive_expect_tx(b.full + s, LANE_BYTES + a.col_box_bytes);
        uint8_t *dst = sm + s * a.stage_bytes;
        const int k0 = kb * FP8_BLOCK;
        tc::tma_load_2d(dst, &lane_map, b.full + s, a.lane_mn ? l0 : k0, a.lane_mn ? k0 : l0);
        tc::tma_load_2d(dst + LANE_BYTES, &col_map, b.full + s, a.col_mn ? c0 : k0, a.col_mn ? k0 : c0);
      }
      if (ok) ring_drain(b.empty, a.stages, kb1 - kb0, &b, a.err, splits);
    }
    __syncwarp();
  } else {
    if (lane == 0) {
      bool ok = !a.test_wait || mm_wait_slow(&b.never, 0, &b, a.err, splits, 1000000ull);
      int is = 0;
      for (int kb = kb0; kb < kb1 && ok; ++kb) {
        const int it = kb - kb0, s = it % a.stages, e = is % SF_RING;
        if (kb == kb0 || (kb & 3) == 0) {
          ok = mm_wait(b.sf_full + e, (is / SF_RING) & 1, &b, a.err, splits);
          if (!ok) break;
        }
        ok = mm_wait(b.full + s, (it / a.stages) & 1, &b, a.err, splits);
        if (!ok) break;
        tc::tc_fence_after();
        mma_block<false>(a, tmem, tc::smem_u32(sm + s * a.stage_bytes), tmem_sf + e * SF_COLS, kb, kb == kb0);
        mm_commit<false>(b.empty + s);
        if ((kb & 3) == 3 || kb == kb1 - 1) {
          mm_commit<false>(b.sf_empty + e);
          ++is;
        }
      }
      if (ok) mm_commit<false>(b.acc_full);
    }
    __syncwarp();
  }
  __syncthreads();
  if (b.abort) settle();
  if (warp == 0) mm_dealloc<false>(tmem, SPLIT_TMEM);
  if (splits == 1) return;
  cluster_sync();
  if (warp < 4 && !b.abort) {
    // element e of the tile (column e / 128, lane e % 128): CTA (e / 128) % splits
    const int n = l0 + (int)threadIdx.x;
    const int valid = min(a.width, a.cols - c0);
    for (int c = rank; c < valid; c += splits) {
      const float *p = reinterpret_cast<const float *>(sm) + c * 128 + threadIdx.x;
      float v[8], s = 0.f;
#pragma unroll
      for (uint32_t r = 0; r < 8; ++r)
        if (r < splits) asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v[r]) : "r"(peer_addr(p, r)));
#pragma unroll
      for (uint32_t r = 0; r < 8; ++r)
        if (r < splits) s += v[r];
      if (n < a.lanes) static_cast<T *>(a.out)[(int64_t)(c0 + c) * a.ldo + n] = from_f32<T>(s);
    }
  }
  __syncwarp();
  cluster_sync();  // no CTA leaves while a peer reads its sums
}

// ------------------------------------------------------------ host

// kind::mxf8f6f4 instruction descriptor: e4m3 x e4m3, UE8M0 scales, fp32 sums.
uint32_t idesc_scaled(int M, int N, bool lane_mn, bool col_mn) {
  return (lane_mn ? 1u << 15 : 0u) | (col_mn ? 1u << 16 : 0u) | (uint32_t)(N >> 3) << 17 | 1u << 23 |
         (uint32_t)(M >> 4) << 24;
}

constexpr uint32_t SMEM_LIMIT = 227 * 1024 - 1024 - sizeof(Bars);  // dynamic, after alignment

template <typename T>
cudaError_t launch_pair(const CUtensorMap &lm, const CUtensorMap &cm, const MmArgs &a, cudaStream_t st) {
  auto kern = fp8_matmul_pair_kernel<T>;
  const int smem = (int)(a.stages * a.stage_bytes + 1024);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(2 * (a.tiles < 76 ? a.tiles : 76)));
  cfg.blockDim = dim3(PAIR_THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = 2;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, lm, cm, a);
}

template <typename T>
cudaError_t launch_split(const CUtensorMap &lm, const CUtensorMap &cm, const MmArgs &a, cudaStream_t st) {
  auto kern = fp8_matmul_split_kernel<T>;
  int smem = (int)(a.stages * a.stage_bytes + 1024);
  if (smem < 80 * 1024) smem = 80 * 1024;  // two CTAs an SM at most: that is what tensor memory holds
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(a.tiles * a.splits));
  cfg.blockDim = dim3(SPLIT_THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = (unsigned)a.splits;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, lm, cm, a);
}

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

}  // namespace

cudaError_t launch_fp8_matmul(const kda_fp8_matmul_args &p, cudaStream_t st) {
  const bool nt = p.form == KDA_FP8_NT, tn = p.form == KDA_FP8_TN;
  MmArgs a{};
  a.lane_scales = p.b_scales;
  a.col_scales = p.a_scales;
  a.lanes = p.n;
  a.cols = p.m;
  a.kblocks = ceil_div(p.k, FP8_BLOCK);
  if (nt) { a.tile_i = a.kblocks; a.tile_k = 1; }
  else if (!tn) { a.tile_i = 1; a.tile_k = ceil_div(p.n, FP8_BLOCK); }
  a.lane_mn = !nt;
  a.col_mn = tn;
  a.lane_step = a.lane_mn ? 256 : 2;  // 32 of k: four 8-row groups, or 32 bytes of a row
  a.col_step = a.col_mn ? 256 : 2;
  a.out = p.out;
  a.ldo = p.ldo;
  a.err = static_cast<uint32_t *>(p.workspace);
  a.test_wait = (p.flags & KDA_TEST_WAIT_TIMEOUT) != 0;

  // Pairs when they have tiles for half of the GPU's 76 pairs, clusters that split k otherwise.
  const int64_t pair_tiles = (int64_t)ceil_div(p.n, 256) * ceil_div(p.m, PAIR_MAX_WIDTH);
  const bool pair = pair_tiles >= 38;
  if (pair) {
    a.width = PAIR_MAX_WIDTH;
    a.lane_tiles = ceil_div(p.n, 256);
    a.splits = 1;
  } else {
    a.width = p.m <= 16 ? 16 : p.m <= 32 ? 32 : p.m <= 64 ? 64 : SPLIT_MAX_WIDTH;
    a.lane_tiles = ceil_div(p.n, 128);
  }
  const int box_rows = pair ? a.width / 2 : a.width;  // column-side rows of one CTA
  a.tiles = a.lane_tiles * ceil_div(p.m, a.width);
  a.col_box_bytes = a.col_mn ? 16384 : (uint32_t)box_rows * 128;
  a.stage_bytes = LANE_BYTES + ((a.col_box_bytes + 1023) & ~1023u);
  if (!pair) {
    a.splits = 1;
    while (a.splits < 8 && a.splits * 2 <= a.kblocks && (int64_t)a.tiles * a.splits * 2 <= 304) a.splits *= 2;
  }
  const int per_cta = ceil_div(a.kblocks, a.splits);
  // pairs have the SM to themselves; split CTAs share it two by two
  const uint32_t budget = pair ? SMEM_LIMIT : (SMEM_LIMIT - 1024 - (uint32_t)sizeof(Bars)) / 2 - 1024;
  a.stages = (int)(budget / a.stage_bytes);
  if (a.stages > MAX_STAGES) a.stages = MAX_STAGES;
  if (!pair && a.stages > per_cta) a.stages = per_cta;
  if (!pair && a.stages * a.stage_bytes < (uint32_t)a.width * 512) a.stages = ceil_div(a.width * 512, a.stage_bytes);
  a.idesc = idesc_scaled(pair ? 256 : 128, a.width, a.lane_mn, a.col_mn);

  CUtensorMap lm, cm;
  const bool ok = (a.lane_mn ? tcp::make_byte_map(p.b, p.n, p.k, p.ldb, 128, lm)
                             : tcp::make_byte_map(p.b, p.k, p.n, p.ldb, 128, lm)) &&
                  (a.col_mn ? tcp::make_byte_map(p.a, p.m, p.k, p.lda, 128, cm)
                            : tcp::make_byte_map(p.a, p.k, p.m, p.lda, (uint32_t)box_rows, cm));
  if (!ok) return cudaErrorInvalidValue;
  if (pair)
    return p.out_dtype == KDA_F32 ? launch_pair<float>(lm, cm, a, st) : launch_pair<__nv_bfloat16>(lm, cm, a, st);
  return p.out_dtype == KDA_F32 ? launch_split<float>(lm, cm, a, st) : launch_split<__nv_bfloat16>(lm, cm, a, st);
}

}  // namespace kda
