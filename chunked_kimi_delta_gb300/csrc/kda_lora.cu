// kda_lora.cu - low-rank adapters of many requests beside a shared projection:
//   out = y + scale[l] (x A[l]^T) B[l]^T      for the rows of a request with adapter l
// and the gradients.  A row tile (up to 64 rows of one request; 16 where
// requests have few) is one cluster's: its CTAs share the sum over n_in, add
// their parts of u = x A^T through distributed shared memory, and share the
// columns of the result.  So u never leaves the chip, one launch does it all,
// and a decode batch of single rows still uses every SM.
//
// x and A pass through a ring in shared memory (read straight into registers,
// two steps ahead, u of 32,768 x 4,096 took 150 us and more: too few bytes in
// flight).  B and y go to registers directly: a sum does not care for the order
// of its terms, so a lane takes four neighbouring ranks as its share of a step
// of 16, on both sides alike; and the columns of a result tile are dealt so that
// a lane ends up with eight neighbouring ones of y.
//
// bf16 values are exact operands; u is carried in two of them (16 bits; three
// where an fp32 gradient comes of it), fp32 inputs in three (24 bits, six
// products).  Sums over many steps are taken into fp32 registers every eight
// steps: the tensor core cuts what does not fit off its running sum, always
// towards zero.
//
// 6,731 packed rows of 2,048 -> 4,196, rank 24: 51 us (floor 21: bytes at the copy rate);
// 64 single rows of 4,096 -> 4,096, rank 16: 10.3 us, rank 128 43 (floors 2.1 and 15); du with dX of 32,768 rows of
// 4,096 -> 4,096, rank 64: 230 us (floor 119).  What bounds it is the latency of loads
// that its phases do not cover: about half the copy rate in both of them.
#include "kda_lora_kernel.cuh"

namespace kda {
namespace lora {

cudaError_t launch_lora(const kda_lora_args &x, cudaStream_t st) {
  Args a{};
  a.rows = x.rows;
  a.n_in = x.n_in; a.n_out = x.n_out; a.rank = x.rank; a.adapters = x.adapters;
  a.a_ld = x.n_in; a.b_ld = x.rank;
  a.a_adapter = (int64_t)x.rank * x.n_in;
  a.b_adapter = (int64_t)x.rank * x.n_out;
  a.x = x.x; a.a = x.a; a.b = x.b; a.y = x.y; a.out = x.out;
  a.idx = x.idx;
  a.idx64 = x.idx_dtype == KDA_I64;
  a.b_vec = x.rank % 4 == 0;
  a.requests = x.num_requests;
  a.cu = x.cu_seqlens;
  a.scale = x.scale;
  return run<false>(x.dtype, Pair{{a, a}}, 1, st);
}

}  // namespace lora
}  // namespace kda
