// norm.cuh -- how the layer norm kernels divide rows: a group of `warps` warps holds one row at
// a time, 512 columns a warp and 16 values a lane, and walks the rows grid-wide.  A block holds as
// many groups as its warps allow (24 forward, 16 backward: what fits an SM's registers).
// The next rows of each group are on their way into shared memory by asynchronous copies
// (every thread copies the bytes it will read itself, so no barrier guards them).
#pragma once
#include "internal.h"
#include "rowops.cuh"

namespace fp8q {

constexpr int kNormWarpCols = 512;
constexpr int kNormWarpsMost = 32;    // of a row: 16384 columns
constexpr int kNormStages = 4;        // most rows in flight a group
constexpr int kNormSmem = 200 * 1024; // shared memory for them

// How a launch divides its rows (host side).
struct NormPlan {
  int warps;        // warps a row
  int groups;       // rows a block has at a time
  int stages;       // rows in flight a group
  int blocks;
  bool wide;        // rows of more warps than a block of the usual kernel has
  size_t smem;
};
// block_warps: warps of a block of the usual kernel; stage_bytes: shared memory of one warp's
// piece of one row
inline NormPlan norm_plan(int64_t rows, int64_t cols, int block_warps, int stage_bytes, int num_sms) {
  NormPlan n{};
  n.warps = static_cast<int>((cols + kNormWarpCols - 1) / kNormWarpCols);
  n.wide = n.warps > block_warps;
  n.groups = n.wide ? 1 : block_warps / n.warps;
  if (n.warps > 1 && n.groups > 15) n.groups = 15;   // a named barrier a group, 1..15
  // few rows: spread over the SMs first
  const int64_t per_sm = (rows + num_sms - 1) / num_sms;
  if (n.groups > per_sm) n.groups = static_cast<int>(per_sm);
  const int64_t stage = static_cast<int64_t>(stage_bytes) * n.warps * n.groups;
  int64_t s = stage > 0 ? kNormSmem / stage : 1;
  n.stages = static_cast<int>(s < 1 ? 1 : (s > kNormStages ? kNormStages : s));
  const int64_t want = (rows + n.groups - 1) / n.groups;
  n.blocks = static_cast<int>(want < num_sms ? want : num_sms);
  n.smem = static_cast<size_t>(stage * n.stages);
  return n;
}

// Barrier of one group's warps (nothing for a group of one warp).
__device__ __forceinline__ void group_sync(int group, int warps) {
  if (warps == 1)
    __syncwarp();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(warps * 32) : "memory");
}

template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? BYTES : 0;   // 0: the destination is filled with zeros
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// until at most `stages` - 1 of the committed copies are outstanding
__device__ __forceinline__ void cp_async_wait_oldest(int stages) {
  if (stages == 4)
    asm volatile("cp.async.wait_group 3;" ::: "memory");
  else if (stages == 3)
    asm volatile("cp.async.wait_group 2;" ::: "memory");
  else if (stages == 2)
    asm volatile("cp.async.wait_group 1;" ::: "memory");
  else
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

}  // namespace fp8q
