// rms.cuh -- how the RMS norm kernels divide rows: as the layer norm's (norm.cuh), a group of warps a row and
// a block an SM, but with fewer rows at a time.  Three or four matrices move at once here, and what counts is
// the bytes that an SM has on their way: few enough that the streams of all SMs stay near each other in memory.
#pragma once
#include "norm.cuh"

namespace fp8q {

// warp_cols: columns of a warp; block_warps: most warps of a block; stage_bytes: shared memory of one warp's part
// of one row.  A block's rows fill at most `most` bytes (or are one row), its stages at most `in_flight` (or are
// `least_stages`).  A plan
// whose single row does not fit has smem above kNormSmem.
inline NormPlan rms_plan(int64_t rows, int64_t cols, int warp_cols, int block_warps, int64_t stage_bytes, int64_t most,
                         int64_t in_flight, int least_stages, int num_sms) {
  NormPlan n{};
  n.warps = static_cast<int>((cols + warp_cols - 1) / warp_cols);
  const int64_t row = stage_bytes * n.warps;
  n.groups = n.warps < block_warps ? block_warps / n.warps : 1;
  if (n.warps > 1 && n.groups > 15) n.groups = 15;   // a named barrier a group, 1..15
  if (n.groups * row > most) n.groups = most > row ? static_cast<int>(most / row) : 1;
  // few rows: spread over the SMs first
  const int64_t per_sm = (rows + num_sms - 1) / num_sms;
  if (n.groups > per_sm) n.groups = static_cast<int>(per_sm);
  n.ring = n.warps * warp_cols * 4;
  const int64_t room = kNormSmem - n.ring, stage = row * n.groups;
  const int64_t want = in_flight / stage;
  if (n.groups == 1 && least_stages < 2) least_stages = 2;   // a lone row would leave the SM waiting for the next
  n.stages = static_cast<int>(want < least_stages ? least_stages : (want > kNormStages ? kNormStages : want));
  if (n.stages * stage > room) n.stages = static_cast<int>(room / stage > 1 ? room / stage : 1);
  const int64_t blocks = (rows + n.groups - 1) / n.groups;
  n.blocks = static_cast<int>(blocks < num_sms ? blocks : num_sms);
  n.smem = static_cast<size_t>(n.ring + stage * n.stages);
  return n;
}

}  // namespace fp8q
