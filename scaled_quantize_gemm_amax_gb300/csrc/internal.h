// internal.h -- launchers shared between the C-ABI layer and the kernel files.
#pragma once
#include <atomic>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace fp8q {

enum Recipe : int { kTensor = 0, kBlock1x128 = 1, kBlock128x128 = 2, kMx = 3 };

constexpr int kMaxDevices = 64;

// Raise a kernel's dynamic shared-memory limit once per device (the setting is
// per function and device); `done` is the caller's per-kernel flag array (atomic:
// any host thread may launch; setting the attribute twice is harmless).
template <typename Kernel>
inline cudaError_t ensure_smem_limit(Kernel* fn, int bytes, std::atomic<bool> (&done)[kMaxDevices]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done[dev].store(true, std::memory_order_release);
  return e;
}

// The same for a kernel whose clusters may have 16 blocks.
template <typename Kernel>
inline cudaError_t ensure_wide_cluster(Kernel* fn, std::atomic<bool> (&done)[kMaxDevices]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) done[dev].store(true, std::memory_order_release);
  return e;
}

// Launch with programmatic stream serialization: the kernel may be scheduled while the
// kernel before it in the stream drains.  Every kernel of this library executes
// griddepcontrol.wait (pdl_wait) before its first global-memory access, which returns
// once the preceding kernel has completed and its writes are visible, so stream order
// holds for all data; only launch latency and set-up (barriers, TMEM, tensor-map
// prefetch) overlap.  cluster_x > 1 adds a cluster dimension.
template <class... KArgs, class... Args>
inline cudaError_t launch_pdl(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, int cluster_x,
                              Args... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  unsigned n = 0;
  attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[n].val.programmaticStreamSerializationAllowed = 1;
  ++n;
  if (cluster_x > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = static_cast<unsigned>(cluster_x);
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// ---- amax / scale / history (amax.cu)
cudaError_t launch_reciprocal(const float* in, float* out, cudaStream_t s);
// p[0 .. n) = 0 as a (programmatically launched) kernel, ahead of an atomicMax reduction
cudaError_t launch_zero_f32(float* p, int n, cudaStream_t s);
// The amax kernels, and the casts when amax_out is set, must be launched right after
// launch_zero_f32 of their amax: they read their inputs before griddepcontrol.wait (the
// zeroing kernel waited for every earlier kernel before letting them start) and wait
// only before the atomic.
cudaError_t launch_amax(const void* x, int64_t n, float* amax, int num_sms, cudaStream_t s);
cudaError_t launch_amax_f32(const float* x, int64_t n, float* amax, int num_sms, cudaStream_t s);
cudaError_t launch_compute_scale(const float* amax, bool e5m2, float* scale, float* scale_inv, cudaStream_t s);
cudaError_t launch_history_update(float* hist, int32_t len, int32_t* pos, const float* amax, bool e5m2, float* scale,
                                  float* scale_inv, uint32_t* err, cudaStream_t s);

// ---- quantize / cast-transpose (quantize.cu)
struct CastParams {
  int64_t R, C;          // input rows / columns (bf16, row-major)
  int recipe;
  int e5m2;
  int mx_tiled;          // MX scales in the GEMM-ready tiled layout
  int mx_floor;          // MX exponent by the floor rule (else the ceil rule)
  int do_row, do_col;
  const float* scale;    // per-tensor scale (device)
  float* amax_out;       // optional (device, zeroed by the kernel launched just before)
  uint8_t* q_row;        // [R, C] (generic path only; the tiled path stores through tensor maps)
  uint8_t* q_col;        // [C, R]
  void* s_row;
  void* s_col;
  uint32_t* err;
  int tiles_r, tiles_c;
  int col_from_row;      // set by the launcher: the column copy as the byte transpose of the row copy
  int keep_col_scales;   // set by the launcher: 1x128 column scales stored with the L2 evict-last policy
  int one_division;      // set by the launcher: a 1x128 tile's row and column scales from one division a lane
};
// Tiled TMA path; requires C % 16 == 0 and (when do_col) R % 16 == 0.
cudaError_t launch_cast_transpose_tiled(const CastParams& p, const CUtensorMap& tm_x, const CUtensorMap& tm_qrow,
                                        const CUtensorMap& tm_qcol, int num_sms, cudaStream_t s);
// Plain path for the per-tensor recipe at any shape.
cudaError_t launch_cast_generic(const CastParams& p, const void* x, cudaStream_t s);
// The same two paths for a binary32 input (quantize_f32.cu); the tiled path's tensor map
// holds the input as 32-column boxes of 128 rows.
cudaError_t launch_cast_transpose_tiled_f32(const CastParams& p, const CUtensorMap& tm_x, const CUtensorMap& tm_qrow,
                                            const CUtensorMap& tm_qcol, int num_sms, cudaStream_t s);
cudaError_t launch_cast_generic_f32(const CastParams& p, const void* x, cudaStream_t s);
// Several tiled casts in one launch: job j owns tiles [tile_start[j], tile_start[j+1]).
constexpr int kMaxCastJobs = 4;
struct CastJobMaps {
  CUtensorMap x, qrow, qcol;
};
struct CastJobs {
  CastJobMaps m[kMaxCastJobs];
  CastParams p[kMaxCastJobs];
  int tile_start[kMaxCastJobs + 1];
  int n;
};
cudaError_t launch_cast_jobs(const CastJobs& jobs, int num_sms, cudaStream_t s);

// ---- dequantize (dequantize.cu): y bf16 [R, C] = RN_bf16(decode(q) * multiplier)
cudaError_t launch_dequantize(const uint8_t* q, int64_t R, int64_t C, int recipe, bool mx_tiled, bool e5m2,
                              const void* s, void* y, int num_sms, cudaStream_t stream);

// ---- FP8 gradient all-reduce of k ranks held as rows of g [k, n] (allreduce.cu);
// *amax must hold the global amax when the kernel runs
cudaError_t launch_allreduce(const void* g, int k, int64_t n, const float* amax, bool e5m2, uint8_t* q,
                             float* scale_inv, float* out, int num_sms, cudaStream_t s);

// ---- the all-reduce with its amax in library-owned scratch (noalloc.cu)
int noalloc_max_ranks();
cudaError_t launch_allreduce_noalloc(const void* g, int k, int64_t n, bool e5m2, uint8_t* q, float* scale_inv,
                                     float* out, cudaStream_t s);

// ---- layer norm (norm.cu, norm_backward.cu); strides (ld*) in elements, f32: binary32 data, else bf16
struct NormParams {
  const void* x;
  int64_t rows, cols, ldx;
  int f32;
  const void* w;         // weight and bias [cols], null: 1 and 0
  const void* b;
  int w_f32;
  float eps;
  void* y;
  int64_t ldy;
  float* mean;           // [rows], null: not stored
  float* rstd;
  int e5m2;
  uint8_t* q;            // [rows, cols] codes of the normalised rows, null: none
  int64_t ldq;
  float* s;              // [rows, ceil(cols / 128)] their multipliers
};
struct NormBwdParams {
  const void* dy;
  int64_t rows, cols, lddy;
  int f32;
  const void* x;         // the input and its rows' means; null: q and s
  int64_t ldx;
  const float* mean;
  const float* rstd;
  int e5m2;
  const uint8_t* q;
  int64_t ldq;
  const float* s;
  const void* w;
  int w_f32;
  void* dx;
  int64_t lddx;
  void* dw;              // [cols], each nullable
  void* db;
  float* partial;        // [norm_partials(rows)][2][cols]
};
constexpr int kMaxNormPartials = 304;   // most blocks of the backward pass
int norm_partials(int64_t rows);
cudaError_t launch_norm(const NormParams& p, int num_sms, cudaStream_t s);
cudaError_t launch_norm_backward(const NormBwdParams& p, int num_sms, cudaStream_t s);

// ---- gated and plain activations (act.cu)
enum Act : int { kActSilu = 0, kActGelu = 1, kActGeluTanh = 2 };
struct ActParams {
  const void* a;
  int64_t rows, cols, lda;
  int f32, act;
  const void* b;         // null: not gated
  int64_t ldb;
  void* y;
  int64_t ldy;
  int e5m2;
  uint8_t* qa;           // [rows, cols] codes and multipliers of a and b, null: none
  uint8_t* qb;
  int64_t ldq;
  float* sa;
  float* sb;
};
struct ActBwdParams {
  const void* dy;
  int64_t rows, cols, lddy;
  int f32, act;
  const void* a;         // a and b, or their codes
  const void* b;
  int64_t lda, ldb;
  int e5m2;
  const uint8_t* qa;
  const uint8_t* qb;
  int64_t ldq;
  const float* sa;
  const float* sb;
  void* da;
  void* db;              // null: not gated
  int64_t ldda, lddb;
};
cudaError_t launch_act(const ActParams& p, int num_sms, cudaStream_t s);
cudaError_t launch_act_backward(const ActBwdParams& p, int num_sms, cudaStream_t s);

// ---- expert routing (moe.cu)
constexpr int kMaxExperts = 1024;
struct RouteParams {
  const void* experts;   // [n] int32 or int64
  int ids64;
  int64_t n;
  int n_experts;
  int align;
  int64_t capacity;
  int* offsets;          // [n_experts + 1]
  int* pos;              // [n]
  int* src;              // [capacity]
  int64_t per_block;     // choices of a block and of a warp, set by the launcher
  int64_t per_warp;
};
cudaError_t launch_route(RouteParams p, cudaStream_t s);
struct ScatterParams {
  const void* in;        // [tokens, cols]
  int64_t tokens, cols, ldin;
  int k, f32;
  const int* pos;        // [tokens, k]
  const int* src;        // [capacity]
  int64_t capacity;
  const float* weights;  // [tokens, k], null: 1
  void* out;             // [capacity, cols]
  int64_t ldout;
  const void* other;     // [capacity, cols], read for the dots only
  int64_t ldother;
  float* dots;           // [tokens, k], null: none
  uint32_t* err;
};
cudaError_t launch_scatter(const ScatterParams& p, int num_sms, cudaStream_t s);
struct CombineParams {
  const void* ys;        // [capacity, cols]
  int64_t capacity, ldys;
  int64_t tokens, cols;
  int k, f32;
  const int* pos;
  const float* weights;  // null: 1
  void* y;               // [tokens, cols]
  int64_t ldy;
  uint32_t* err;
};
cudaError_t launch_combine(const CombineParams& p, int num_sms, cudaStream_t s);

// ---- scaled GEMM (gemm.cu)
struct GemmParams {
  int64_t M, N, K;
  int kind;              // kTensor, kBlock1x128 (A 1x128), kMx
  int b_1x128;           // blockwise: B scales per (row, 128-K) instead of per (128 rows, 128-K)
  int e5m2_a, e5m2_b;
  int out_fp32;
  const void* sa;        // per-tensor: float[1]; blockwise: float[M, K/128]; MX: tiled E8M0
  const void* sb;        // per-tensor: float[1]; blockwise: float[N/128, K/128] or [N, K/128]; MX: tiled E8M0
  void* c;               // [M, N] row-major, bf16 or fp32; null: not stored
  // fused output quantization (all null: off).  y = the value stored in c (bf16-rounded
  // for bf16 output): c_amax = max |y|, cq = encode_sat(y * c_scale), c_scale_inv = 1 / c_scale
  float* c_amax;         // float[1], zeroed by the caller's stream before the launch
  const float* c_scale;  // float[1]
  uint8_t* cq;           // [M, N] row-major FP8 (format e5m2_c)
  float* c_scale_inv;    // float[1]
  int e5m2_c;
  uint32_t* err;
  // Split of the last, partial wave (per-tensor and MX on CTA pairs): the tiles from
  // tail0 on are cut into `split` K ranges computed by otherwise idle pairs; range c > 0
  // leaves its raw FP32 accumulators in ws slot (c - 1) * (tiles - tail0) + j and counts
  // its warps on ws_flags[slot]; the pair with range 0 adds the ranges in order and
  // resets the count.  split = 1: off (tail0 = the tile count).
  int split;
  int tail0;
  // Balanced division instead (streamk = 1, same kernels and workspace): the tiles' K
  // blocks in order, cut into one contiguous share per pair; a tile cut between pairs u
  // and u + 1 has its later part left in slot u + 1 by pair u + 1 (its first work) and
  // added by pair u (its last work).
  int streamk;
  float* ws;             // [slots][256][256] fp32
  int* ws_flags;         // [slots], 0 between launches
  int64_t ws_len;        // floats in ws, and
  int ws_nflags;         // counters in ws_flags (index checks of debug builds)
  // Blockwise 1x128 x 128x128 on 256 x 160 pair tiles (set by gemm_select_wide)
  int wide160;
};
// Whether the blockwise 1x128 x 128x128 GEMM these parameters describe runs on 256 x 160
// pair tiles with 128-deep stages (BF16 out, no fused output cast, M % 256 == 0, K / 128
// odd); the caller stores the answer in p.wide160 before asking for the tile shape and
// building the tensor maps.
bool gemm_select_wide(const GemmParams& p, int num_sms);
// Width (N) of one output tile of the GEMM variant these parameters select.
int gemm_block_n(const GemmParams& p);
// Whether the GEMM runs on 2-CTA pairs (256-row tiles) for these parameters.
bool gemm_uses_pair(const GemmParams& p);
// Rows of B one TMA box carries (the tile width, or half of it for a pair).
int gemm_b_box_rows(const GemmParams& p);
// Columns of C one TMA store box carries: 16 (BF16, unswizzled) for the 160-wide tiles,
// else 0: the usual 128-byte box (64 BF16 or 32 FP32 columns, 128-byte swizzle).
int gemm_c_box_cols(const GemmParams& p);
// The division of a CTA-pair launch's tiles (host logic only): whole tiles, stream-K
// shares of the tiles from tail0 on (streamk = 1), or the last wave cut into `split` K
// ranges; `launched` pairs.  Per-tensor and MX only (other kinds: whole tiles).  Both cuts
// also need the stream's workspace; without it a launch runs whole tiles.
struct PairDivision {
  int streamk;
  int split;
  int tail0;
  int64_t launched;
};
PairDivision pair_division(int kind, int64_t ntiles, int64_t pairs, int64_t k);
// What a GEMM with these parameters launches (host logic only, p.wide160 already chosen):
// kernel variant (kTensor, kBlock1x128, kMx, or the blockwise variants 4 = per-row B on
// one CTA, 5 = 256-deep stages, 6 = per-row B on pairs, 7 = 256 x 160 pair tiles), CTA
// pairs or not, tile width, tile count, and the division above.
struct GemmPlan {
  int pair;
  int variant;
  int block_n;
  int64_t ntiles;
  PairDivision div;
};
GemmPlan gemm_plan(const GemmParams& p, int num_sms, int resident_pairs);
// tm_sfa / tm_sfb: MX only (the tiled E8M0 buffers as [atoms * 2, 256] bytes, box 2 x 256).
cudaError_t launch_gemm(const GemmParams& p, const CUtensorMap& tm_a, const CUtensorMap& tm_b, const CUtensorMap& tm_sfa,
                        const CUtensorMap& tm_sfb, const CUtensorMap& tm_c, int num_sms, cudaStream_t s);

// ---- RMS norm (rms.cu, rms_backward.cu); strides (ld*) in elements, f32: binary32 data, else bf16
struct RmsParams {
  const void* x;
  int64_t rows, cols, ldx;
  int f32;
  const void* res;       // [rows, cols] added to x, null: none
  int64_t ldr;
  const void* w;         // [cols], null: 1
  int w_f32;
  float eps;
  void* h;               // [rows, cols] x + res as rounded, null: not stored
  int64_t ldh;
  void* y;               // [rows, cols], null: not stored
  int64_t ldy;
  float* rstd;           // [rows], null: not stored
  int recipe;            // of q: kTensor, kBlock1x128 or kMx
  int mx_tiled, mx_floor;
  int e5m2;
  const float* scale;    // kTensor: float[1]
  float* amax;           // float[1], zeroed by the kernel launched just before; null: none
  uint8_t* q;            // [rows, cols] codes of y, null: none
  int64_t ldq;
  void* s;               // kTensor: float[1]; kBlock1x128: float[rows, ceil(cols / 128)]; kMx: E8M0 bytes
};
struct RmsBwdParams {
  const void* dy;
  int64_t rows, cols, lddy;
  int f32;
  const void* h;
  int64_t ldh;
  const float* rstd;
  const void* dh;        // added to dx, null: none
  int64_t lddh;
  const void* w;
  int w_f32;
  void* dx;
  int64_t lddx;
  void* dw;              // [cols], null: none
  float* partial;        // [norm_partials(rows)][cols]
};
cudaError_t launch_rms(const RmsParams& p, int num_sms, cudaStream_t s);
cudaError_t launch_rms_backward(const RmsBwdParams& p, int num_sms, cudaStream_t s);

// ---- the gradients' norm and clipping (clip.cu)
struct ClipTensor {
  const void* in;
  void* out;
  int64_t n;             // elements
  int f32;
};
// doubles of partial sums that n_tensors need (clip.cu's workspace)
int64_t clip_partials(int64_t n_tensors);
// *norm = 2-norm over all tensors; with `clip`, out = in * min(1, max_norm / (*norm + 1e-6)) too
cudaError_t launch_clip(const ClipTensor* t, int64_t n, bool clip, float max_norm, double* partial, float* norm, int num_sms,
                        cudaStream_t s);

// ---- products grouped by expert (grouped.cu)
struct GroupedParams {
  int kind;              // kTensor or kMx
  int depth;             // 0: C [capacity, N], an expert's rows; 1: C [n_experts][M, N], summed over an expert's rows
  int n_experts;
  const int* offsets;    // [n_experts + 1], multiples of 128
  int64_t capacity;      // rows that the segments lie in
  int M, N, K;           // M: depth only; K: rows only
  int b_cols;            // rows: the experts' B are side by side, [N, n_experts * K], not [n_experts * N, K]
  int a_rows, a_cols;    // A's matrix, and B's (where its scale atoms are)
  int b_cols_all, b_rows_all;
  int e5m2_a, e5m2_b, out_fp32;
  const float* sa;       // kTensor: float[1]
  const float* sb;       // kTensor: float[1] or (sb_step 1) one an expert
  int sb_step;
  void* c;
  int zero_tail;         // rows: 1: rows behind the last segment are set to 0, 2: those in front of the first too
  int loads;             // whether there is anything to multiply (the tensor maps of A and B are valid)
  uint32_t* err;
};
struct GroupedMaps {
  CUtensorMap a, b, sfa, sfb, c;
};
// How a call is divided.  Boxes have 128 rows of A; 128 of B for pairs, else the width; of C 32 rows of
// 128 bytes, or of 64 with bf16 and no pairs, swizzled as wide.  Pairs with per-tensor scales have A by boxes of 64 rows in sfa.
struct GroupedPlan {
  int width;             // columns of a CTA's tile of 128 rows, 0 for CTA pairs and tiles of 256 x 256
  int stages;            // of the ring (without pairs of B's)
  int accumulators;      // in TMEM
};
GroupedPlan grouped_plan(const GroupedParams& p, int num_sms);
cudaError_t launch_grouped(const GroupedParams& p, const GroupedMaps& m, const GroupedPlan& g, int num_sms, cudaStream_t s);

// Bounded-wait self test: one CTA waits on an mbarrier nothing arrives on.
cudaError_t launch_wait_selftest(uint32_t* err, cudaStream_t s);
// Index-check self test: one thread checks `index` against `extent` the way the kernels
// check their accesses (no memory is touched); only debug builds report.
cudaError_t launch_index_selftest(int64_t index, int64_t extent, uint32_t* err, cudaStream_t s);

}  // namespace fp8q
