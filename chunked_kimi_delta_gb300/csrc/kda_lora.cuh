// kda_lora.cuh - low-rank adapters of many requests: launchers and workspace.
#pragma once

#include "kda_internal.cuh"

namespace kda {
namespace lora {

constexpr int TM = 64;     // rows of a tile
constexpr int COLS = 32;   // wide columns a warp takes at once

// The rank as the kernels hold it.
inline int padded(int rank) { return rank <= 16 ? 16 : rank <= 32 ? 32 : rank <= 64 ? 64 : 128; }

// Workspace of the backward: both matrices of every adapter transposed, u and
// du in three bf16 pieces, the row tiles of each adapter, and, where the rows
// are shared out, each share's sums.
struct BwdPlan {
  size_t off_at, off_bt, off_u, off_du, off_count, off_list, off_part, total;
  int64_t tiles;  // at most so many row tiles
  int shares;     // of the rows, for the gradients' sums
};
BwdPlan bwd_plan(const kda_lora_bwd_args &a, int sms);

cudaError_t launch_lora(const kda_lora_args &a, cudaStream_t st);
cudaError_t launch_lora_bwd(const kda_lora_bwd_args &a, const BwdPlan &p, cudaStream_t st);

}  // namespace lora
}  // namespace kda
