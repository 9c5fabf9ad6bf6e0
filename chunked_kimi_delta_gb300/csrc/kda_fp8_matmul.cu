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
// Scales.  A stored word (four blocks of k of one row) is what a lane and
// column of tensor memory hold: the word of row r at lane r % 32, column
// r / 32, the same in all four lane quarters.  One warp brings the words into
// a ring in shared memory as [32 lanes][4 columns] (cp.async, four bytes a
// lane: rows need no alignment), and the thread that issues the MMAs copies
// an entry to tensor memory ahead of them (tcgen05.cp, which orders itself
// before the MMAs and repeats the entry for the four quarters).  Storing the
// words to tensor memory from registers instead (tcgen05.st by four warps)
// took 2,400 cycles a word against the 1,800 of its MMAs: 2.9 PFLOP/s from rest
// at 32768 x 4096 x 4096 where this reaches 3.5 (3.0 in a stream of calls under
// the power cap).
#include <cuda_bf16.h>

#include "kda_fp8.cuh"
#include "kda_tc.cuh"

namespace kda {
namespace {

using tcp::globaltimer;

constexpr int SF_COLS = 16;       // tensor-memory columns of one ring entry: 4 lane side, 8 column side
constexpr int SF_RING = 4;
constexpr uint32_t SF_ENTRY = 1536;  // bytes of an entry in shared memory: 512 lane side, 2 x 512 column side
constexpr uint32_t SF_BYTES = SF_RING * SF_ENTRY;
static_assert(SF_BYTES % 1024 == 0, "what follows the ring is aligned like a tile");
// Blocks of k that tensor memory sums before the epilogue takes the sum into
// registers.  A step of the MMA (32 of k) drops up to 2^-23 of the running sum,
// always towards zero (measured on positive terms: 1.1e-8 a step); their
// number in a span, not the size of k, then bounds the error.  fp32 results:
// relative 3.7e-7 at k = 8200 in spans of 32 blocks, 1.7e-7 in 16, 1.3e-7 in
// 12, where one fp32 sum on the CUDA cores has 1.6e-7.  Shorter ones hold the
// MMAs up (32768 x 4096 x 4096 "nt": 328 us in spans of 32 blocks,
// 335 in 16, 350 in 12, 380 in 8; "tn" 4096 x 2048 x 8200: 59, 60, 59, 63).
// bf16 results round by up to 2^-8; 4,096 steps, 5e-5 on positive terms, stay
// an eightieth of that, and what fits one span (k up to 131,072) has a kernel
// without the sums in registers (777 x 1111 x 2064: 8.6 us, with them 9.5).
constexpr int SPAN_F32 = 12, SPAN_BF16 = 1024;
static_assert(SPAN_F32 % 4 == 0 && SPAN_BF16 % 4 == 0, "a span starts with a word of scales");
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
  int span;                  // blocks of k that one accumulator sums
  void *out;
  int64_t ldo;
  bool out_tma;              // the output takes TMA stores (rows start and end on 16 bytes)
  uint32_t *err;
  bool test_wait;
};

struct Bars {
  uint64_t full[MAX_STAGES], empty[MAX_STAGES];
  uint64_t sf_full[SF_RING], sf_empty[SF_RING];
  uint64_t sf_peer[SF_RING];  // pairs, first CTA: the entry is in the second CTA's shared memory too
  uint64_t acc_full[2], acc_empty[2];
  uint64_t never;
  uint32_t tmem;
  volatile uint32_t abort;
};

// Position in a ring of barriers, without divisions: the threads that feed the
// tensor core go round it every few hundred cycles.
struct Ring {
  int size, s = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ explicit Ring(int n) : size(n) {}
  __device__ __forceinline__ void next() {
    if (++s == size) {
      s = 0;
      phase ^= 1;
    }
  }
};
// One thread of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
  return ok != 0;
}

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

__device__ __forceinline__ float4 load_peer(const float *p, uint32_t rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(peer_addr(p, rank)));
  return v;
}

// Bounded wait.  The first wait that runs out records the timeout and tells
// the CTA, and with pairs (cluster_ctas 2) the other one: their waits then
// end too.
__device__ bool mm_wait_slow(uint64_t *bar, uint32_t parity, Bars *b, uint32_t *err, uint32_t cluster_ctas,
                             unsigned long long limit_ns) {
  const unsigned long long t0 = globaltimer();
  while (true) {
    for (int i = 0; i < 8; ++i)  // a try may be held by the hardware for milliseconds
      if (try_wait_cluster(bar, parity)) return true;
    if (b->abort) return false;
    if (globaltimer() - t0 > limit_ns) {
      atomicOr(err, DEV_ERR_TIMEOUT);
      b->abort = 1;
      for (uint32_t r = 0; cluster_ctas > 1 && r < cluster_ctas; ++r)
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
// ---- scales
// Rows past the edge take the last row's scale: it only reaches outputs that
// are not stored.
__device__ __forceinline__ void copy_word(uint32_t smem, const uint8_t *s, int rows, int row, int w) {
  const uint32_t *p = reinterpret_cast<const uint32_t *>(s) + ((int64_t)w * rows + min(row, rows - 1));
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" :: "r"(smem), "l"(p) : "memory");
}
// TILE scales of the lane side, one byte for all 128 lanes: lane i holds the
// byte of block 32 g + i, loaded one group of eight words ahead of its use.
__device__ __forceinline__ uint32_t tile_bytes(const MmArgs &a, int l0, int g, int lane) {
  return *(a.lane_scales + (min(l0, a.lanes - 1) / FP8_BLOCK) * a.tile_i +
               min(32 * g + lane, a.kblocks - 1) * a.tile_k);
}
// One ring entry, by a full warp: word w of the tile at (l0, c0).  Its
// barrier counts every lane twice: when its copies have landed, and when its
// own stores are done.
__device__ __forceinline__ void fill_scales(const MmArgs &a, uint8_t *entry, uint64_t *bar, int l0, int c0, int w,
                                            uint32_t bytes, int lane) {
  const uint32_t dst = tc::smem_u32(entry) + 16 * lane;
  if (a.tile_i) {
    uint32_t v = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) v |= __shfl_sync(~0u, bytes, 4 * (w & 7) + j) << (8 * j);
    *reinterpret_cast<uint4 *>(entry + 16 * lane) = make_uint4(v, v, v, v);
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c) copy_word(dst + 4 * c, a.lane_scales, a.lanes, l0 + 32 * c + lane, w);
  }
#pragma unroll
  for (int c = 0; c < 8; ++c)
    if (32 * c < a.width) copy_word(dst + 512 + 512 * (c >> 2) + 4 * (c & 3), a.col_scales, a.cols, c0 + 32 * c + lane, w);
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" :: "r"(tc::smem_u32(bar)) : "memory");
  tc::mbar_arrive(bar);
}
// An entry from shared to tensor memory (in both CTAs of a pair, each from
// its own), by the thread that issues the MMAs.  No swizzle, groups of eight
// 16-byte rows 128 bytes apart.
template <bool PAIR> __device__ __forceinline__ void copy_scales(uint32_t tmem_sf, uint32_t entry, int width) {
  const uint64_t desc = (uint64_t)((entry & 0x3FFFFu) >> 4) | (uint64_t)(128 >> 4) << 32 | (uint64_t)1 << 46;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    if (i == 2 && width <= 128) break;
    if (PAIR)
      asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" :: "r"(tmem_sf + 4 * i), "l"(desc + 32 * i) : "memory");
    else
      asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" :: "r"(tmem_sf + 4 * i), "l"(desc + 32 * i) : "memory");
  }
}

// The MMAs of a block of k: descriptors of stage 0, and what a stage and 32
// of k add to them.
struct MmaIssue {
  uint64_t lane0, col0;
  uint32_t lane_step, col_step, stage_step, idesc;
  __device__ __forceinline__ MmaIssue(const MmArgs &a, const uint8_t *sm)
      : lane_step(a.lane_step), col_step(a.col_step), stage_step(a.stage_bytes >> 4), idesc(a.idesc) {
    const uint32_t s = tc::smem_u32(sm);
    lane0 = tc::smem_desc_sw128(s, a.lane_mn ? 16384 : 16, 1024);
    col0 = tc::smem_desc_sw128(s + LANE_BYTES, a.col_mn ? 16384 : 16, 1024);
  }
  // `byte`: the block's byte of the scale words; `first`: overwrites the accumulator
  template <bool PAIR>
  __device__ __forceinline__ void block(uint32_t acc, int stage, uint32_t sf, int byte, bool first) const {
    const uint64_t l = lane0 + (uint64_t)(stage * stage_step), c = col0 + (uint64_t)(stage * stage_step);
    const uint32_t id = idesc | (uint32_t)byte << 4 | (uint32_t)byte << 29;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      mma_scaled<PAIR>(acc, l + (uint64_t)(j * lane_step), c + (uint64_t)(j * col_step), id, sf, sf + 4,
                       j != 0 || !first);
  }
};

// 16 accumulator columns (rows m from m0 on, below `end`) of this warp's lanes (columns n).
template <typename T>
__device__ __forceinline__ void store_columns(const MmArgs &a, const float (&v)[16], int n, int m0, int end) {
  if (n >= a.lanes) return;
  T *p = static_cast<T *>(a.out) + (int64_t)m0 * a.ldo + n;
#pragma unroll
  for (int c = 0; c < 16; ++c)
    if (m0 + c < end) p[c * a.ldo] = from_f32<T>(v[c]);
}
// The same columns of one span of k: added to `sum`, which ends up in v.
__device__ __forceinline__ void add_span(float (&sum)[16], float (&v)[16], bool first) {
#pragma unroll
  for (int c = 0; c < 16; ++c) v[c] = sum[c] = (first ? 0.f : sum[c]) + v[c];
}

// ---- bf16 results of a pair's tile through shared memory
// 16 lanes x 32 columns of tensor memory as matrix fragments: register
// 4 c + 2 h + i is lane 8 h + t / 4, column 8 c + 2 (t % 4) + i of thread t.
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
constexpr uint32_t OUT_BUF = 2048;                // a warp's 32 rows m x 32 columns n of bf16, or 16 of fp32
constexpr uint32_t OUT_BYTES = 8 * 2 * OUT_BUF;   // two for each warp of the epilogue
// A warp's 32 lanes of 32 rows m into its staging tile: fragments are stored
// transposed, so that a row m of shared memory holds neighbouring n.
__device__ __forceinline__ void stage_chunk(uint32_t acc, uint8_t *buf, int lane) {
  uint32_t f[2][16];
  tmem_ld_frag(acc, f[0]);
  tmem_ld_frag(acc + (16u << 16), f[1]);
  tc::tmem_ld_wait();
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int n8 = 0; n8 < 2; ++n8) {
      uint32_t v[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(__uint_as_float(f[h][4 * c + 2 * n8]), __uint_as_float(f[h][4 * c + 2 * n8 + 1]));
        v[c] = *reinterpret_cast<const uint32_t *>(&p);
      }
      // lane t gives the address of row m = t: 16 bytes of n, in the 64-byte swizzle that the TMA store reads
      const uint32_t addr = tc::smem_u32(buf) + lane * 64 + (((2 * h + n8) ^ ((lane >> 1) & 3)) << 4);
      asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};"
                   :: "r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
    }
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, const void *src, int32_t x, int32_t y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];"
               :: "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(tc::smem_u32(src)) : "memory");
}

// The last arrivals of MMA commits on a ring: a CTA leaves only when none is
// still to come.  Every slot's latest use, oldest first; a slot never used
// (fewer uses than slots) answers at once, as in a producer's first round.
__device__ __forceinline__ void ring_drain(uint64_t *bars, Ring r, Bars *b, uint32_t *err, uint32_t cluster_ctas) {
  for (int i = 0; i < r.size; ++i, r.next())
    if (!mm_wait(bars + r.s, r.phase ^ 1, b, err, cluster_ctas)) return;
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
// What bounds it is the way of the operands: a block of k brings 30.7 KB to
// an SM, 480 cycles at 64 bytes a cycle from L2 (and again 480 for shared
// memory to take them in and give them to the MMAs at 128), against 448
// cycles of MMAs; measured about 560 at 32768 x 4096 x 4096 (354 to 363 us,
// 3.0 to 3.1 PFLOP/s, back to back under the power cap at 1,395 to 1,460 MHz;
// 315 us over the first 30 calls after a rest; tensor pipe 79% busy).  Half of
// the MMAs left out changed little (314 to 300 us), 26% less read from L2 by
// multicast of the lane side to a second pair nothing at all.
// Warps 0-7 epilogue, 8 scales, 9 TMA, 10 MMA (first CTA of the pair).
constexpr int PAIR_THREADS = 352;
constexpr int PAIR_MAX_WIDTH = 224;  // two accumulators and the scale ring fill the 512 columns
constexpr uint32_t PAIR_SF = 2 * PAIR_MAX_WIDTH;

// SPANS: a tile's sum may take more than one span of k.
template <typename T, bool SPANS>
__global__ void __launch_bounds__(PAIR_THREADS, 1) fp8_matmul_pair_kernel(const __grid_constant__ CUtensorMap lane_map,
                                                                          const __grid_constant__ CUtensorMap col_map,
                                                                          const __grid_constant__ CUtensorMap out_map,
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
      tc::mbar_init(b.sf_full + i, 64);
      tc::mbar_init(b.sf_peer + i, 1);
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
  grid_start();
  const uint32_t tmem = b.tmem;

  auto lane0_of = [&](int t) { return (t % a.lane_tiles) * 256 + (int)rank * 128; };  // this CTA's first n
  auto col0_of = [&](int t) { return (t / a.lane_tiles) * a.width; };                 // the tile's first m

  uint8_t *sf_ring = sm + a.stages * a.stage_bytes;
  if (warp == 8) {  // scales
    Ring f(SF_RING);
    bool ok = true;
    const int words = (a.kblocks + 3) / 4;
    uint32_t next = a.tile_i && pair < a.tiles ? tile_bytes(a, lane0_of(pair), 0, lane) : 0, bytes = 0;
    for (int t = pair; t < a.tiles && ok; t += pairs) {
      const int l0 = lane0_of(t), c0 = col0_of(t);
      for (int w = 0; w < words; ++w, f.next()) {
        if (a.tile_i && (w & 7) == 0) {
          bytes = next;
          if (w + 8 < words) next = tile_bytes(a, l0, (w >> 3) + 1, lane);
          else if (t + pairs < a.tiles) next = tile_bytes(a, lane0_of(t + pairs), 0, lane);
        }
        ok = __all_sync(~0u, mm_wait(b.sf_empty + f.s, f.phase ^ 1, &b, a.err, 2));
        if (!ok) break;
        fill_scales(a, sf_ring + f.s * SF_ENTRY, b.sf_full + f.s, l0, c0, w, bytes, lane);
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (ok) ring_drain(b.sf_empty, f, &b, a.err, 2);
    __syncwarp();
  } else if (warp < 8) {  // epilogue
    const int quarter = warp & 3, half = warp >> 2;
    // Full columns leave through this warp's two staging tiles and TMA stores:
    // whole sectors whatever the order of the lanes, and nothing to wait for.
    uint8_t *stage = sm + a.stages * a.stage_bytes + SF_BYTES + warp * 2 * OUT_BUF;
    int buf = 0;
    auto stage_begin = [&]() {
      if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
      __syncwarp();  // the tile's last store has been read
      return stage + buf * OUT_BUF;
    };
    auto stage_end = [&](int n0, int m0, bool any) {
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (any) tma_store_2d(&out_map, stage + buf * OUT_BUF, n0, m0);
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      }
      buf ^= 1;
    };
    Ring full(2);
    float sum[8][16];  // this thread's outputs over the spans of k, when there is more than one
    for (int t = pair, kb = 0; t < a.tiles; full.next()) {
      if (!__all_sync(~0u, mm_wait(b.acc_full + full.s, full.phase, &b, a.err, 2))) break;
      tc::tc_fence_after();
      const int n0 = lane0_of(t) + 32 * quarter, c0 = col0_of(t);
      const uint32_t acc = tmem + full.s * PAIR_MAX_WIDTH + ((uint32_t)(32 * quarter) << 16);
      const int end = min(a.width, a.cols - c0);
      const bool first = kb == 0, last = kb + a.span >= a.kblocks;
      auto free_accumulator = [&]() {
        tc::tc_fence_before();
        if (lane == 0) arrive_remote(peer_addr(b.acc_empty + full.s, 0));
        __syncwarp();
      };
      if (SPANS) {  // into registers, and the accumulator is free before the stores
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = 32 * half + 64 * i;
          if (c >= a.width) break;
          float v[2][16];
          tc::tmem_ld16(acc + c, v[0]);
          tc::tmem_ld16(acc + c + 16, v[1]);
          tc::tmem_ld_wait();
          add_span(sum[2 * i], v[0], first);
          add_span(sum[2 * i + 1], v[1], first);
        }
        free_accumulator();
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = 32 * half + 64 * i;
        if (c >= a.width || (SPANS && !last)) break;
        if (sizeof(T) == 2 && !SPANS && a.out_tma) {
          stage_chunk(acc + c, stage_begin(), lane);
          stage_end(n0, c0 + c, c < end && n0 < a.lanes);
          continue;
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float v[16];
          if (!SPANS) {
            tc::tmem_ld16(acc + c + 16 * u, v);
            tc::tmem_ld_wait();
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = sum[2 * i + u][j];
          }
          if (sizeof(T) == 4 && a.out_tma) {  // 128 bytes a row, as they are
            float *dst = reinterpret_cast<float *>(stage_begin());
#pragma unroll
            for (int j = 0; j < 16; ++j) dst[32 * j + lane] = v[j];
            stage_end(n0, c0 + c + 16 * u, c + 16 * u < end && n0 < a.lanes);
          } else {
            store_columns<T>(a, v, n0 + lane, c0 + c + 16 * u, c0 + end);
          }
        }
      }
      if (!SPANS) free_accumulator();
      kb += a.span;
      if (last) {
        kb = 0;
        t += pairs;
      }
    }
    if (a.out_tma && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
  } else if (warp == 9) {  // TMA
    if (elect_one()) {
      Ring r(a.stages);
      bool ok = true;
      const uint32_t full0 = peer_addr(b.full, 0);
      const uint32_t bytes = 2 * (LANE_BYTES + a.col_box_bytes);
      for (int t = pair; t < a.tiles && ok; t += pairs) {
        const int l0 = lane0_of(t), c0 = col0_of(t) + (int)rank * (a.width / 2);
        for (int k0 = 0; k0 < a.kblocks * FP8_BLOCK; k0 += FP8_BLOCK) {
          ok = mm_wait(b.empty + r.s, r.phase ^ 1, &b, a.err, 2);
          if (!ok) break;
          if (rank == 0) tc::mbar_arrive_expect_tx(b.full + r.s, bytes);
          const uint32_t bar = full0 + 8 * r.s;
          uint8_t *dst = sm + r.s * a.stage_bytes;
          tma_load_pair(dst, &lane_map, bar, a.lane_mn ? l0 : k0, a.lane_mn ? k0 : l0);
          tma_load_pair(dst + LANE_BYTES, &col_map, bar, a.col_mn ? c0 : k0, a.col_mn ? k0 : c0);
          r.next();
        }
      }
      if (ok) ring_drain(b.empty, r, &b, a.err, 2);
    }
    __syncwarp();
  } else if (rank == 0) {  // MMA
    if (elect_one()) {
      bool ok = !a.test_wait || mm_wait_slow(&b.never, 0, &b, a.err, 2, 1000000ull);
      const MmaIssue mma(a, sm);
      Ring r(a.stages), f(SF_RING), acc(2);
      int kb = 0;  // a tile is one span of k after another, an accumulator each
      for (int t = pair; t < a.tiles && ok; kb = kb < a.kblocks ? kb : (t += pairs, 0), acc.next()) {
        ok = mm_wait(b.acc_empty + acc.s, acc.phase ^ 1, &b, a.err, 2);
        if (!ok) break;
        tc::tc_fence_after();
        const int span0 = kb, span1 = min(kb + a.span, a.kblocks);
        for (; kb < span1; kb += 4) {
          ok = mm_wait(b.sf_full + f.s, f.phase, &b, a.err, 2) && mm_wait(b.sf_peer + f.s, f.phase, &b, a.err, 2);
          if (!ok) break;
          tc::fence_proxy_async_smem();
          copy_scales<true>(tmem + PAIR_SF + f.s * SF_COLS, tc::smem_u32(sf_ring) + f.s * SF_ENTRY, a.width);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (kb + i >= span1) break;
            ok = mm_wait(b.full + r.s, r.phase, &b, a.err, 2);
            if (!ok) break;
            tc::tc_fence_after();
            mma.block<true>(tmem + acc.s * PAIR_MAX_WIDTH, r.s, tmem + PAIR_SF + f.s * SF_COLS, i, kb + i == span0);
            mm_commit<true>(b.empty + r.s);
            r.next();
          }
          if (!ok) break;
          mm_commit<true>(b.sf_empty + f.s);
          f.next();
        }
        if (ok) mm_commit<true>(b.acc_full + acc.s);
      }
    }
    __syncwarp();
  } else {  // tells the first CTA which entries of scales have landed here
    if (elect_one()) {
      Ring f(SF_RING);
      bool ok = true;
      for (int t = pair; t < a.tiles && ok; t += pairs)
        for (int w = 0; w < (a.kblocks + 3) / 4; ++w, f.next()) {
          ok = mm_wait(b.sf_full + f.s, f.phase, &b, a.err, 2);
          if (!ok) break;
          tc::fence_proxy_async_smem();
          arrive_remote(peer_addr(b.sf_peer + f.s, 0));
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
// What bounds it is latency, from the launch over one pass of loads and MMAs
// to the meeting of the sums: 1 x 4096 x 4096 takes 6.6 us where the weight's
// bytes take 2.5.
// Warps 0-3 epilogue, 4 scales, 5 TMA, 6 MMA.
constexpr int SPLIT_THREADS = 224;
constexpr int SPLIT_MAX_WIDTH = 64;
constexpr uint32_t SPLIT_TMEM = 256;  // two CTAs fit an SM

template <typename T, bool SPANS>
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

  // The CTAs of a cluster work by themselves until their sums meet: a wait
  // that runs out ends this CTA's waits only.
  auto issue_load = [&](int kb, int s) {
    tc::mbar_arrive_expect_tx(b.full + s, LANE_BYTES + a.col_box_bytes);
    uint8_t *dst = sm + s * a.stage_bytes;
    const int k0 = kb * FP8_BLOCK;
    tc::tma_load_2d(dst, &lane_map, b.full + s, a.lane_mn ? l0 : k0, a.lane_mn ? k0 : l0);
    tc::tma_load_2d(dst + LANE_BYTES, &col_map, b.full + s, a.col_mn ? c0 : k0, a.col_mn ? k0 : c0);
  };
  if (threadIdx.x == 160) {  // the TMA warp fills the stages while the others set up
    tc::tma_prefetch_desc(&lane_map);
    tc::tma_prefetch_desc(&col_map);
    for (int i = 0; i < a.stages; ++i) {
      tc::mbar_init(b.full + i, 1);
      tc::mbar_init(b.empty + i, 1);
    }
    for (int i = 0; i < SF_RING; ++i) {
      tc::mbar_init(b.sf_full + i, 64);
      tc::mbar_init(b.sf_empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(b.acc_full + i, 1);
      tc::mbar_init(b.acc_empty + i, 4);  // the four epilogue warps
    }
    tc::mbar_init(&b.never, 1);
    b.abort = 0;
    tc::mbar_fence_init();
    grid_start();
    for (int kb = kb0; kb < kb1 && kb - kb0 < a.stages; ++kb) issue_load(kb, kb - kb0);
  }
  if (warp == 0) mm_alloc<false>(&b.tmem, SPLIT_TMEM);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  grid_start();
  const uint32_t tmem = b.tmem, tmem_sf = tmem + 2 * SPLIT_MAX_WIDTH;

  uint8_t *sf_ring = sm + a.stages * a.stage_bytes;
  if (warp < 4) {
    const int n = l0 + 32 * warp + lane;
    float *part = reinterpret_cast<float *>(sm);  // [columns][128]: the stages are free after the last MMA
    const int valid = min(a.width, a.cols - c0);
    float sum[SPLIT_MAX_WIDTH / 16][16];  // this thread's sums over the spans of k, when there is more than one
    Ring full(2);
    for (int kb = kb0; kb < kb1; kb += a.span, full.next()) {
      if (!__all_sync(~0u, mm_wait(b.acc_full + full.s, full.phase, &b, a.err, 1))) break;
      tc::tc_fence_after();
      const bool first = kb == kb0, last = kb + a.span >= kb1;
#pragma unroll
      for (int i = 0; i < SPLIT_MAX_WIDTH / 16; ++i) {
        if (16 * i >= valid) break;
        float v[16];
        tc::tmem_ld16(tmem + full.s * SPLIT_MAX_WIDTH + 16 * i + ((uint32_t)(32 * warp) << 16), v);
        tc::tmem_ld_wait();
        if (SPANS && !(first && last)) add_span(sum[i], v, first);
        if (!last) continue;
        if (splits == 1) {
          store_columns<T>(a, v, n, c0 + 16 * i, c0 + valid);
        } else {
#pragma unroll
          for (int c = 0; c < 16; ++c)
            if (16 * i + c < valid) part[(16 * i + c) * 128 + 32 * warp + lane] = v[c];
        }
      }
      tc::tc_fence_before();
      if (lane == 0) tc::mbar_arrive(b.acc_empty + full.s);
      __syncwarp();
    }
  } else if (warp == 4) {
    Ring f(SF_RING);
    bool ok = true;
    uint32_t bytes = 0;
    for (int w = kb0 >> 2; 4 * w < kb1; ++w, f.next()) {
      if (a.tile_i && ((w & 7) == 0 || w == kb0 >> 2)) bytes = tile_bytes(a, l0, w >> 3, lane);
      ok = __all_sync(~0u, mm_wait(b.sf_empty + f.s, f.phase ^ 1, &b, a.err, 1));
      if (!ok) break;
      fill_scales(a, sf_ring + f.s * SF_ENTRY, b.sf_full + f.s, l0, c0, w, bytes, lane);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (ok) ring_drain(b.sf_empty, f, &b, a.err, 1);
    __syncwarp();
  } else if (warp == 5) {
    if (elect_one()) {
      Ring r(a.stages);
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb, r.next()) {
        if (kb - kb0 < a.stages) continue;  // on its way
        ok = mm_wait(b.empty + r.s, r.phase ^ 1, &b, a.err, 1);
        if (!ok) break;
        issue_load(kb, r.s);
      }
      if (ok) ring_drain(b.empty, r, &b, a.err, 1);
    }
    __syncwarp();
  } else {
    if (elect_one()) {
      bool ok = !a.test_wait || mm_wait_slow(&b.never, 0, &b, a.err, 1, 1000000ull);
      const MmaIssue mma(a, sm);
      Ring r(a.stages), f(SF_RING), acc(2);
      int in_span = 0;
      for (int kb = kb0; kb < kb1 && ok; ++kb, r.next()) {
        if (in_span == 0) {
          ok = mm_wait(b.acc_empty + acc.s, acc.phase ^ 1, &b, a.err, 1);
          if (!ok) break;
        }
        if (kb == kb0 || (kb & 3) == 0) {
          ok = mm_wait(b.sf_full + f.s, f.phase, &b, a.err, 1);
          if (!ok) break;
          tc::fence_proxy_async_smem();
          copy_scales<false>(tmem_sf + f.s * SF_COLS, tc::smem_u32(sf_ring) + f.s * SF_ENTRY, a.width);
        }
        ok = mm_wait(b.full + r.s, r.phase, &b, a.err, 1);
        if (!ok) break;
        tc::tc_fence_after();
        mma.block<false>(tmem + acc.s * SPLIT_MAX_WIDTH, r.s, tmem_sf + f.s * SF_COLS, kb & 3, in_span == 0);
        mm_commit<false>(b.empty + r.s);
        if ((kb & 3) == 3 || kb == kb1 - 1) {
          mm_commit<false>(b.sf_empty + f.s);
          f.next();
        }
        if (++in_span == a.span || kb == kb1 - 1) {
          mm_commit<false>(b.acc_full + acc.s);
          acc.next();
          in_span = 0;
        }
      }
    }
    __syncwarp();
  }
  __syncthreads();
  if (b.abort) settle();
  if (warp == 0) mm_dealloc<false>(tmem, SPLIT_TMEM);
  if (splits == 1) return;
  cluster_sync();
  if (warp < 4 && !b.abort) {
    // Four columns at a time per CTA, a warp each, four lanes of the tile per
    // thread; two of these in flight, since a load from a peer takes long.
    const int valid = min(a.width, a.cols - c0), step = 4 * (int)splits;
    const float *part = reinterpret_cast<const float *>(sm) + 4 * lane;
    for (int c = 4 * (int)rank + warp; c < valid; c += 2 * step) {
      float4 v[2][8];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (uint32_t r = 0; r < 8; ++r)
          if (r < splits && c + u * step < valid) v[u][r] = load_peer(part + (c + u * step) * 128, r);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (c + u * step >= valid) break;
        float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (uint32_t r = 0; r < 8; ++r)
          if (r < splits) {
            s[0] += v[u][r].x;
            s[1] += v[u][r].y;
            s[2] += v[u][r].z;
            s[3] += v[u][r].w;
          }
        T *p = static_cast<T *>(a.out) + (int64_t)(c0 + c + u * step) * a.ldo + l0 + 4 * lane;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (l0 + 4 * lane + q < a.lanes) p[q] = from_f32<T>(s[q]);
      }
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

constexpr uint32_t SMEM_LIMIT = MAX_DYNAMIC_SMEM - 1024;  // after alignment
static_assert(sizeof(Bars) <= 227 * 1024 - MAX_DYNAMIC_SMEM, "static shared memory");

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

struct Plan {
  bool pair;
  int width, splits;
};

// Pairs of CTAs take the work when there is a 256 x 224 tile for each pair of
// the `sms` SMs (all figures here: 152 of them), in tiles as wide as makes
// their turns shortest: a turn costs about its width and 120 columns more (3000
// x 2048 x 2048, two turns at any width from 160 to 224: 14.3, 14.5, 14.9 us;
// 2000 x 8192 x 2048, four turns of 224 or five of 192: 24.8 and 27.6).  Fewer
// tiles leave pairs idle, and 128 x 64 ones for single CTAs, two to an SM, are
// then as fast or faster (us, pairs at their best width against single CTAs:
// 777 x 1111 x 2064 10.8 / 9.8, 512 x 4096 x 4096 13.9 / 14.8, 300 x 1024 x
// 1024 7.5 / 6.8).  So they are up to 64 rows: a lane-side box then serves one
// tile whichever kernel reads it, and two CTAs an SM keep more of them in
// flight (1 x 32768 x 4096 37.6 / 23.3, 64 x 32768 x 4096 31.4 / 24.5, 64 x
// 100000 x 2048 42.0 / 38.3; but 100 x 32768 x 4096, each box read twice, 32.0
// / 42.1).  Where single CTAs do not fill the SMs, k is split while a part
// keeps at least four blocks: a smaller part costs more in the meeting of the
// sums than it saves.  Up to one CTA an SM; up to two where few rows make the
// sums short (with one / two: 1 x 4096 x 4096 7.4 / 6.3 us, 1 x 8192 x 4096 9.4
// / 8.4, 1 x 4096 x 16384 15.0 / 13.6, but 777 x 1111 x 2064 8.3 / 10.5).
Plan choose_plan(int m, int n, int kblocks, int sms) {
  const int64_t lane_tiles = ceil_div(n, 256), pairs = sms / 2;
  if (m > SPLIT_MAX_WIDTH && lane_tiles * ceil_div(m, PAIR_MAX_WIDTH) >= pairs) {
    Plan best{true, PAIR_MAX_WIDTH, 1};
    int64_t least = INT64_MAX;
    for (int width = PAIR_MAX_WIDTH; width >= 128; width -= 32) {
      const int64_t cost = (int64_t)ceil_div(lane_tiles * ceil_div(m, width), pairs) * (width + 120);
      if (cost < least) {
        least = cost;
        best.width = width;
      }
    }
    return best;
  }
  Plan p{false, m <= 16 ? 16 : m <= 32 ? 32 : SPLIT_MAX_WIDTH, 1};
  const int64_t tiles = (int64_t)ceil_div(n, 128) * ceil_div(m, p.width);
  while (p.splits < 8 && 8 * p.splits <= kblocks && tiles * p.splits * 2 <= (p.width <= 32 ? 2 * sms : sms)) p.splits *= 2;
  return p;
}

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

  const int sms = sm_count();
  const Plan plan = choose_plan(p.m, p.n, a.kblocks, sms);
  const bool pair = plan.pair;
  a.width = plan.width;
  a.splits = plan.splits;
  a.span = p.out_dtype == KDA_F32 ? SPAN_F32 : SPAN_BF16;
  a.lane_tiles = ceil_div(p.n, pair ? 256 : 128);
  a.tiles = a.lane_tiles * ceil_div(p.m, a.width);
  const int box_rows = pair ? a.width / 2 : a.width;  // column-side rows of one CTA
  a.col_box_bytes = a.col_mn ? 16384 : (uint32_t)box_rows * 128;
  a.stage_bytes = LANE_BYTES + ((a.col_box_bytes + 1023) & ~1023u);
  const bool f32 = p.out_dtype == KDA_F32;
  const bool spans = f32 || a.kblocks > a.span;  // kernels that add up spans of k
  // TMA stores clip a row at 16 bytes, not at elements: rows that end inside of
  // 16 leave by plain stores, or they would reach into what lies beside them.
  // So do sums of spans in bf16: over so long a k that costs nothing.
  const int64_t es = f32 ? 4 : 2;
  a.out_tma = pair && f32 == spans && p.n * es % 16 == 0 && p.ldo * es % 16 == 0 && p.ldo <= INT32_MAX &&
              reinterpret_cast<uintptr_t>(p.out) % 16 == 0;
  // A pair has its SMs to itself, and so do split CTAs when all of them fit that
  // way; else two share one.  A cluster stays within a group of SMs, whose number
  // is no multiple of it: of 152 SMs fours fill 144, eights surely 64 (1 x 2048 x
  // 8192, 16 clusters of eight: 12.5 us alone, in two turns, 6.8 sharing).
  const int64_t fit = a.splits == 8 ? sms * 64 / 152 : a.splits == 4 ? sms * 144 / 152 : sms;
  const bool alone = pair || (int64_t)a.tiles * a.splits <= fit;
  uint32_t budget = SMEM_LIMIT - SF_BYTES - (a.out_tma ? OUT_BYTES : 0);
  if (!alone) budget = (SMEM_LIMIT - 1024 - (uint32_t)sizeof(Bars)) / 2 - 1024 - SF_BYTES;
  a.stages = (int)(budget / a.stage_bytes);
  if (a.stages > MAX_STAGES) a.stages = MAX_STAGES;
  if (!pair) {
    const int per_cta = ceil_div(a.kblocks, a.splits);
    if (a.stages > per_cta) a.stages = per_cta;
    if (a.stages * a.stage_bytes < (uint32_t)a.width * 512) a.stages = ceil_div(a.width * 512, a.stage_bytes);
  }
  a.idesc = idesc_scaled(pair ? 256 : 128, a.width, a.lane_mn, a.col_mn);

  CUtensorMap lm, cm, om{};
  const bool ok = (a.lane_mn ? tcp::make_byte_map(p.b, p.n, p.k, p.ldb, 128, lm)
                             : tcp::make_byte_map(p.b, p.k, p.n, p.ldb, 128, lm)) &&
                  (a.col_mn ? tcp::make_byte_map(p.a, p.m, p.k, p.lda, 128, cm)
                            : tcp::make_byte_map(p.a, p.k, p.m, p.lda, (uint32_t)box_rows, cm)) &&
                  (!a.out_tma || tcp::make_out_tile_map(p.out, f32, p.n, p.m, p.ldo, 32, f32 ? 16 : 32, om));
  if (!ok) return cudaErrorInvalidValue;
  uint32_t smem = a.stages * a.stage_bytes + SF_BYTES + 1024;
  if (pair) {
    smem += a.out_tma ? OUT_BYTES : 0;
    const unsigned grid = 2u * (unsigned)(a.tiles < sms / 2 ? a.tiles : sms / 2);
    return launch_overlapped(f32     ? fp8_matmul_pair_kernel<float, true>
                             : spans ? fp8_matmul_pair_kernel<__nv_bfloat16, true>
                                     : fp8_matmul_pair_kernel<__nv_bfloat16, false>,
                             grid, PAIR_THREADS, smem, 2, st, lm, cm, om, a);
  }
  if (smem < 80 * 1024) smem = 80 * 1024;  // two CTAs an SM at most: that is what tensor memory holds
  const unsigned grid = (unsigned)(a.tiles * a.splits), cluster = (unsigned)a.splits;
  return launch_overlapped(f32     ? fp8_matmul_split_kernel<float, true>
                           : spans ? fp8_matmul_split_kernel<__nv_bfloat16, true>
                                   : fp8_matmul_split_kernel<__nv_bfloat16, false>,
                           grid, SPLIT_THREADS, smem, cluster, st, lm, cm, a);
}

}  // namespace kda
