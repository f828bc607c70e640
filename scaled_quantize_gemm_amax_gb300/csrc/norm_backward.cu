// norm_backward.cu -- layer norm, backward.
//
//   g = dy w,  c1 = sum g / H,  c2 = sum g xh / H,  dx = r (g - c1 - xh c2)
//   dw = sum over rows of dy xh,  db = sum over rows of dy
// with xh = (x - m) r, or the values of its 8-bit copy.  All sums are binary32, in an order
// that depends on the shape alone.
//
// Bound by HBM: dy and x (or the codes) once in, dx once out.  A thread owns the same columns
// for all the rows of its group, so the column sums stay in registers over the whole walk; they
// leave as one partial sum a block, added up by a second, small launch.
// 8192x4096 bf16 from codes 36.9 us (4.6 TB/s, 0.68 of what a copy reaches), 2048x12288 from x 36.6
// (0.61), 65536x4096 from codes 0.94; binary32 from x 8192x4096 66 us (0.90), 2048x16384, one row in flight a
// block, 78 (0.76); unaligned bf16 8192x4099 77 from x and 82 from codes (0.38, 0.31).  What is left at the short sizes does not grow with the rows:
// every SM reads the same weights at the start (1.7 to 3 us at 4096 columns, 5 at 12288), and the
// partial sums are written and added up at the end (4.4 and 8 us, the second launch included).
#include "norm.cuh"

namespace fp8q {

namespace {

constexpr int kMostCols = 16384;   // of a row held in registers
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Sums over the block; the result is valid in every thread.  `red` holds 2 * kWarps floats
// and is free again after the block's next barrier.
__device__ __forceinline__ float2 block_sum(float a, float b, float* red) {
  a = warp_sum(a);
  b = warp_sum(b);
  const int w = threadIdx.x >> 5;
  __syncthreads();
  if ((threadIdx.x & 31) == 0) {
    red[w] = a;
    red[kWarps + w] = b;
  }
  __syncthreads();
  float2 r = {0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    r.x += red[i];
    r.y += red[kWarps + i];
  }
  return r;
}

// xh of one element, from x or from the codes
template <typename T>
__device__ __forceinline__ float normalised(const NormBwdParams& p, int64_t row, int64_t c, int64_t groups, float mean,
                                            float rstd) {
  if (p.q == nullptr) return (ld_elem(static_cast<const T*>(p.x) + row * p.ldx + c) - mean) * rstd;
  float v, unused;
  decode_pair(p.q[row * p.ldq + c], p.e5m2, v, unused);
  return v * p.s[row * groups + c / 128];
}

// dx of rows of any width: one block per row, two passes.  Rows of more than kMostCols columns, with the
// column pass below: 2048x20480 bf16 from x 290 us (0.13), binary32 346 (0.22).
template <typename T>
__global__ void __launch_bounds__(kThreads) k_norm_dx_any(const NormBwdParams p) {
  __shared__ float red[2 * kWarps];
  const int64_t groups = (p.cols + 127) / 128;
  const float inv_n = 1.0f / static_cast<float>(p.cols);
  pdl_wait();
  pdl_launch_dependents();
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* dy = static_cast<const T*>(p.dy) + row * p.lddy;
    T* dx = static_cast<T*>(p.dx) + row * p.lddx;
    const float mean = p.q == nullptr ? p.mean[row] : 0.0f, rstd = p.rstd[row];
    float s1 = 0.0f, s2 = 0.0f;
    for (int64_t c = threadIdx.x; c < p.cols; c += kThreads) {
      const float g = ld_elem(dy + c) * (p.w != nullptr ? ld_param(p.w, p.w_f32, c) : 1.0f);
      s1 += g;
      s2 = fmaf(g, normalised<T>(p, row, c, groups, mean, rstd), s2);
    }
    const float2 s = block_sum(s1, s2, red);
    const float c1 = s.x * inv_n, c2 = s.y * inv_n;
    for (int64_t c = threadIdx.x; c < p.cols; c += kThreads) {
      const float g = ld_elem(dy + c) * (p.w != nullptr ? ld_param(p.w, p.w_f32, c) : 1.0f);
      st_elem(dx + c, rstd * (g - c1 - normalised<T>(p, row, c, groups, mean, rstd) * c2));
    }
  }
}

// Partial sums of dw and db: block (x, y) sums 256 columns over the rows of slab y, one
// thread per column; partial [slab][dw, db][cols].
template <typename T>
__global__ void __launch_bounds__(kThreads) k_norm_partial_any(const NormBwdParams p, int slabs) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (c >= p.cols) return;
  const int64_t groups = (p.cols + 127) / 128;
  const int64_t r0 = p.rows * blockIdx.y / slabs, r1 = p.rows * (blockIdx.y + 1) / slabs;
  float dw = 0.0f, db = 0.0f;
  for (int64_t row = r0; row < r1; ++row) {
    const float dy = ld_elem(static_cast<const T*>(p.dy) + row * p.lddy + c);
    const float xh = normalised<T>(p, row, c, groups, p.q == nullptr ? p.mean[row] : 0.0f, p.rstd[row]);
    dw = fmaf(dy, xh, dw);
    db += dy;
  }
  float* out = p.partial + static_cast<int64_t>(blockIdx.y) * 2 * p.cols;
  out[c] = dw;
  out[p.cols + c] = db;
}

// Shared memory of one warp's part of one row: dy, x or the codes, and 12 floats: the part's
// multipliers, rstd and mean.
template <typename T, bool VECTOR, bool CODES, int V>
struct NormBackwardStage {
  using P = Piece<T, VECTOR>;
  static constexpr int kIn = RowPart<P, 32 * V, VECTOR, T>::kBytes;   // where x or the codes start
  static constexpr int kScalars = kIn + (CODES ? RowPart<P, 32 * V, VECTOR, uint8_t>::kBytes : RowPart<P, 32 * V, VECTOR, T>::kBytes);
  static constexpr int kBytes = (kScalars + 48 + 127) / 128 * 128;
};

// Rows of up to kMostCols columns, V values a lane.  The column sums take 2 V of a thread's
// registers and g V; xh is read from shared memory twice, before and after the row's sums are
// known.
template <typename T, bool VECTOR, bool CODES, int V, int BLOCK_WARPS>
__global__ void __launch_bounds__(BLOCK_WARPS * 32)
    k_norm_backward(const NormBwdParams p, const int warps, const int stages, const int ring) {
  using P = Piece<T, VECTOR>;
  constexpr int E = P::E, J = V / E, H = E / 2, kGroups = V / 4;   // kGroups: of 128 columns in a warp's part
  using PartDy = RowPart<P, 32 * V, VECTOR, T>;
  using PartQ = RowPart<P, 32 * V, VECTOR, uint8_t>;
  using Stage = NormBackwardStage<T, VECTOR, CODES, V>;
  constexpr int kStage = Stage::kBytes, kIn = Stage::kIn, kScalars = Stage::kScalars;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float red[2][2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = warp / warps, w_in = warp - group * warps;
  const int n_groups = (blockDim.x >> 5) / warps, step = gridDim.x * n_groups;
  const int rows = static_cast<int>(p.rows), cols = static_cast<int>(p.cols), groups8 = (cols + 127) / 128;
  const int lddy = static_cast<int>(p.lddy), ldx = static_cast<int>(p.ldx), ldq = static_cast<int>(p.ldq),
            lddx = static_cast<int>(p.lddx);
  // this lane's first column and the columns from there to the row's end
  const int base = w_in * 32 * V, c = base + P::first(lane), left = cols - c;
  const float inv_n = 1.0f / static_cast<float>(cols);
  uint8_t* const mine = smem + ring + warp * stages * kStage;
  float* const ws = reinterpret_cast<float*>(smem);

  // row `row` into stage s: the warp's part of dy and x / codes; the first lanes the warp's
  // multipliers, rstd and mean
  auto issue = [&](int row, int s) {
    if (row < rows) {
      uint8_t* const to = mine + s * kStage;
      const int64_t r = row;
      PartDy::start(to, static_cast<const T*>(p.dy) + r * lddy, r * lddy, base, cols, lane);
      if constexpr (CODES)
        PartQ::start(to + kIn, p.q + r * ldq, r * ldq, base, cols, lane);
      else
        PartDy::start(to + kIn, static_cast<const T*>(p.x) + r * ldx, r * ldx, base, cols, lane);
      const float* scalar = (lane == kGroups ? p.rstd : p.mean) + row;
      bool want = lane == kGroups || (lane == kGroups + 1 && !CODES);
      if (CODES && lane < kGroups) {
        const int g = w_in * kGroups + lane;
        want = g < groups8;
        scalar = p.s + r * groups8 + (want ? g : 0);
      }
      if (want) cp_async<4>(smem_u32(to) + kScalars + lane * 4, scalar, true);
    }
    cp_async_commit();
  };
  // What piece j of the row in stage s holds beside dy: the codes' values and their multiplier, or
  // x - mean and rstd; xh is their product.  Past the row's end dy is 0 and xh must be finite, which
  // -mean rstd need not be (a row of one value, 2^120): aligned rows take 0 for rstd there, others 0 for
  // x - mean in rows whose product overflows (`far`; 1 to 2 % slower, for all rows 2 to 8 %).
  auto fetch = [&](int s, int m, int j, float rstd, float mean, bool far, float (&h)[E]) -> float {
    const uint8_t* const at = mine + s * kStage + kIn;
    if constexpr (CODES) {
      P::decode(PartQ::read_codes(at, m, lane, j), p.e5m2, h);
      // past the row's end the codes are 0, and the multiplier was not copied
      return left > j * P::WC ? reinterpret_cast<const float*>(mine + s * kStage + kScalars)[(j * P::WC + P::first(lane)) / 128] : 0.0f;
    } else {
      PartDy::read(at, m, lane, j, h);
#pragma unroll
      for (int i = 0; i < E; i += 2) {
        const float2 d = add2(make_float2(h[i], h[i + 1]), both(-mean));
        h[i] = d.x;
        h[i + 1] = d.y;
      }
      if (VECTOR) return left > j * P::WC ? rstd : 0.0f;
      if (far) {
#pragma unroll
        for (int i = 0; i < E; ++i) h[i] = P::has(left - j * P::WC, i) ? h[i] : 0.0f;
      }
      return rstd;
    }
  };

  pdl_wait();
  pdl_launch_dependents();
  float2 dw[J][H], db[J][H];
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int i = 0; i < H; ++i) dw[j][i] = db[j][i] = make_float2(0.0f, 0.0f);
  int row = blockIdx.x * n_groups + group;
  start_param<P, V>(p.w, p.w_f32, cols, warps, 1.0f, ws);
  cp_async_commit();
  for (int s = 0; s < stages; ++s) issue(row + s * step, s);
  cp_async_wait_oldest(stages + 1);
  settle_param<P, V>(p.w, p.w_f32, warps, ws);
  __syncthreads();
  for (int s = 0, buf = 0; row < rows; row += step, buf ^= 1) {
    cp_async_wait_oldest(stages);
    __syncwarp();   // the row's scalars, and unaligned a lane's last elements, were copied by other lanes
    const float* const scalars = reinterpret_cast<const float*>(mine + s * kStage + kScalars);
    const float rstd = scalars[kGroups], mean = CODES ? 0.0f : scalars[kGroups + 1];
    // elements between granules and values, of dy and of x or the codes
    const int m_dy = PartDy::past(static_cast<const T*>(p.dy) + static_cast<int64_t>(row) * lddy + base);
    const int m_in = CODES ? PartQ::past(p.q + static_cast<int64_t>(row) * ldq + base)
                           : PartDy::past(static_cast<const T*>(p.x) + static_cast<int64_t>(row) * ldx + base);
    const bool far = !VECTOR && !CODES && is_inf_or_nan(mean * rstd);
    float2 g[J][H], s1 = {0.0f, 0.0f}, s2 = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < J; ++j) {
      float d[E], h[E], w[E];
      PartDy::read(mine + s * kStage, m_dy, lane, j, d);
      const float2 m = both(fetch(s, m_in, j, rstd, mean, far, h));
      read_param<P, V>(ws, w_in, j, lane, w);
#pragma unroll
      for (int i = 0; i < H; ++i) {
        const float2 dy = {d[2 * i], d[2 * i + 1]}, xh = mul2(make_float2(h[2 * i], h[2 * i + 1]), m);
        g[j][i] = mul2(dy, make_float2(w[2 * i], w[2 * i + 1]));
        dw[j][i] = fma2(dy, xh, dw[j][i]);
        db[j][i] = add2(db[j][i], dy);
        s1 = add2(s1, g[j][i]);
        s2 = fma2(g[j][i], xh, s2);
      }
    }
    // both sums over the warp: the lower half of its lanes takes c1 and the upper half c2
    const float a = s1.x + s1.y, b = s2.x + s2.y;
    float v = (lane < 16 ? a : b) + __shfl_xor_sync(0xFFFFFFFFu, lane < 16 ? b : a, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (warps > 1) {
      if ((lane & 15) == 0) red[buf][lane >> 4][warp] = v;
      group_sync(group, warps);
      // lane l of a half joins warps l and l + 16 (the other buffer is written before this one is reused)
      const int l = lane & 15;
      const float* part = red[buf][lane >> 4] + group * warps;
      v = l < warps ? part[l] : 0.0f;
      if (BLOCK_WARPS > 16 && l + 16 < warps) v += part[l + 16];
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    }
    const float c1 = __shfl_sync(0xFFFFFFFFu, v, 0) * inv_n, c2 = __shfl_sync(0xFFFFFFFFu, v, 16) * inv_n;
    // dx = r g - r c1 - (r c2) xh
    const float2 r = both(rstd), k1 = both(-rstd * c1);
    const float k2 = -rstd * c2;
    T* const dx0 = static_cast<T*>(p.dx) + static_cast<int64_t>(row) * lddx + c;
    constexpr int N = VECTOR ? 1 : J;   // pieces stored together: unaligned, the fewer ends the better
#pragma unroll
    for (int j0 = 0; j0 < J; j0 += N) {
      uint4 packed[N];
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int j = j0 + k;
        float h[E], out[E];
        const float2 m = both(k2 * fetch(s, m_in, j, rstd, mean, false, h));   // past the end nothing is stored
#pragma unroll
        for (int i = 0; i < H; ++i) {
          const float2 o = fma2(make_float2(h[2 * i], h[2 * i + 1]), m, fma2(g[j][i], r, k1));
          out[2 * i] = o.x;
          out[2 * i + 1] = o.y;
        }
        packed[k] = P::pack(out);
      }
      P::store_raw(dx0 + j0 * P::WC, left - j0 * P::WC, packed);
    }
    __syncwarp();   // all lanes have read what this one copied
    issue(row + stages * step, s);
    s = s + 1 == stages ? 0 : s + 1;
  }
  if (p.dw == nullptr && p.db == nullptr) return;
  // the block's groups joined pairwise in shared memory (the ring is free: every copy was waited for)
  __syncthreads();
  float2* join = reinterpret_cast<float2*>(smem + ring);
  for (int n = n_groups; n > 1;) {
    const int half = (n + 1) / 2;
    if (group >= half && group < n) {
      float2* out = join + ((group - half) * warps + w_in) * 32 * V + lane;
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < H; ++i) {
          out[(j * H + i) * 32] = dw[j][i];
          out[(j * H + i) * 32 + 16 * V] = db[j][i];
        }
    }
    __syncthreads();
    if (group < n - half) {
      const float2* in = join + (group * warps + w_in) * 32 * V + lane;
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < H; ++i) {
          dw[j][i] = add2(dw[j][i], in[(j * H + i) * 32]);
          db[j][i] = add2(db[j][i], in[(j * H + i) * 32 + 16 * V]);
        }
    }
    __syncthreads();
    n = half;
  }
  if (group != 0) return;
  if (gridDim.x > 1) {   // partial sums
    float* part = p.partial + static_cast<int64_t>(blockIdx.x) * 2 * cols + c;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      float* out = part + j * P::WC;
      if constexpr (VECTOR) {   // cols is a multiple of 4, the workspace 16-byte aligned
        if (left <= j * P::WC) continue;
#pragma unroll
        for (int i = 0; i < H; i += 2) {
          reinterpret_cast<float4*>(out)[i / 2] = make_float4(dw[j][i].x, dw[j][i].y, dw[j][i + 1].x, dw[j][i + 1].y);
          reinterpret_cast<float4*>(out + cols)[i / 2] = make_float4(db[j][i].x, db[j][i].y, db[j][i + 1].x, db[j][i + 1].y);
        }
      } else {
#pragma unroll
        for (int i = 0; i < E; ++i) {
          if (!P::has(left - j * P::WC, i)) continue;
          out[P::at(i)] = i % 2 ? dw[j][i / 2].y : dw[j][i / 2].x;
          out[cols + P::at(i)] = i % 2 ? db[j][i / 2].y : db[j][i / 2].x;
        }
      }
    }
    return;
  }
  // one block's sums are the result
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int i = 0; i < E; ++i) {
      if (!P::has(left - j * P::WC, i)) continue;
      const int at = c + j * P::WC + P::at(i);
      if (p.dw != nullptr) st_param(p.dw, p.w_f32, at, i % 2 ? dw[j][i / 2].y : dw[j][i / 2].x);
      if (p.db != nullptr) st_param(p.db, p.w_f32, at, i % 2 ? db[j][i / 2].y : db[j][i / 2].x);
    }
}

// The 2 * cols sums of the partial sums: a block takes 32 lanes' worth of them (four a lane where
// cols % 4 == 0), warp k the partials k, k + 32, ...; then the 32 warps' sums in order.
constexpr int kParamWarps = 32;
template <int N>
__global__ void __launch_bounds__(kParamWarps * 32) k_norm_params(const float* partial, int n, int cols, bool f32, void* dw, void* db) {
  __shared__ float part[kParamWarps][32 * N];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (static_cast<int64_t>(blockIdx.x) * 32 + lane) * N, total = 2 * static_cast<int64_t>(cols);
  pdl_wait();
  pdl_launch_dependents();
  float v[N] = {};
  if (c < total) {
#pragma unroll 5
    for (int k = warp; k < n; k += kParamWarps) {
      const float* from = partial + k * total + c;
      if constexpr (N == 4) {
        const float4 u = *reinterpret_cast<const float4*>(from);
        v[0] += u.x, v[1] += u.y, v[2] += u.z, v[3] += u.w;
      } else {
        v[0] += *from;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) part[warp][i * 32 + lane] = v[i];
  __syncthreads();
  if (warp >= N) return;
  // warp i of the first N: value i of every lane
  const int64_t at = c + warp;
  if (c >= total) return;
  float sum = 0.0f;
#pragma unroll
  for (int k = 0; k < kParamWarps; ++k) sum += part[k][warp * 32 + lane];
  void* out = at < cols ? dw : db;
  if (out != nullptr) st_param(out, f32, at < cols ? at : at - cols, sum);
}

// *partials: number of partial sums left in p.partial (0: none)
template <typename T, bool VECTOR, bool CODES, int V, int BLOCK_WARPS>
cudaError_t run_norm_backward(const NormBwdParams& p, int num_sms, cudaStream_t s, int* partials) {
  const int stage = NormBackwardStage<T, VECTOR, CODES, V>::kBytes;
  NormPlan n = norm_plan(p.rows, p.cols, 32 * V, BLOCK_WARPS, 1, stage, num_sms < kMaxNormPartials ? num_sms : kMaxNormPartials);
  const size_t join = n.ring + static_cast<size_t>(n.groups / 2) * n.warps * 64 * V * sizeof(float);
  if (n.smem < join) n.smem = join;
  static std::atomic<bool> done[kMaxDevices];
  auto kernel = k_norm_backward<T, VECTOR, CODES, V, BLOCK_WARPS>;
  const cudaError_t e = ensure_smem_limit(kernel, kNormSmem, done);
  if (e != cudaSuccess) return e;
  *partials = n.blocks > 1 ? n.blocks : 0;
  return launch_pdl(kernel, dim3(n.blocks), dim3(static_cast<unsigned>(n.warps * n.groups * 32)), n.smem, s, 1, p, n.warps,
                    n.stages, n.ring);
}

// Values a lane and warps of a block.  32 values halve what a row costs besides its values, and 12
// warps leave a thread the 168 registers that they and the column sums take (8192x4096 from codes
// and 2048x12288 from x, when chosen: 39.3 and 42.7 us; 24 warps of 16 values 41.5 and 52.4; 16
// warps of 32 values in 128 registers 41.0 and 58.2, needed above 12288 columns).  24 warps of 16 values and 16
// of 32 spill 4 to 56 bytes a thread in 11 of their 16 forms.  Narrow rows take
// the fewest values that hold them: 131072x128 from x 34 us, with 16 values 49.
template <typename T, bool VECTOR, bool CODES>
cudaError_t run_norm_backward(const NormBwdParams& p, int num_sms, cudaStream_t s, int* partials) {
  if (p.cols <= 256) return run_norm_backward<T, VECTOR, CODES, 8, 24>(p, num_sms, s, partials);
  if (p.cols <= 512) return run_norm_backward<T, VECTOR, CODES, 16, 24>(p, num_sms, s, partials);
  // rows of 5, 7 or 8 warps leave 2 to 5 of 12 idle and at most 2 of 16: bf16 from codes 8192x8192 66
  // us with 16 warps, 77 with 12, 13107x5120 67 and 73; unaligned from x 16372x4099 140 and 155;
  // aligned from x 76 and 71 at 5120, binary32 60 and 52 at 4096x8192: these stay
  const int64_t warps = (p.cols + 1023) / 1024;
  const bool idle = warps <= 12 && 4 * (12 / warps) < 3 * (16 / warps);
  if (p.cols <= 12288 && !(idle && sizeof(T) == 2 && (CODES || !VECTOR)))
    return run_norm_backward<T, VECTOR, CODES, 32, 12>(p, num_sms, s, partials);
  return run_norm_backward<T, VECTOR, CODES, 32, 16>(p, num_sms, s, partials);
}

template <typename T, bool VECTOR>
cudaError_t run_norm_backward(const NormBwdParams& p, int num_sms, cudaStream_t s, int* partials) {
  return p.q != nullptr ? run_norm_backward<T, VECTOR, true>(p, num_sms, s, partials)
                        : run_norm_backward<T, VECTOR, false>(p, num_sms, s, partials);
}

template <typename T>
cudaError_t run_any(const NormBwdParams& p, int num_sms, cudaStream_t s, int* partials) {
  const int64_t cap = static_cast<int64_t>(num_sms) * 8;
  if (p.rows > 0) {
    const cudaError_t e = launch_pdl(k_norm_dx_any<T>, dim3(static_cast<unsigned>(p.rows < cap ? p.rows : cap)), dim3(kThreads),
                                     0, s, 1, p);
    if (e != cudaSuccess) return e;
  }
  if (p.dw == nullptr && p.db == nullptr) return cudaSuccess;
  *partials = norm_partials(p.rows);
  return launch_pdl(k_norm_partial_any<T>, dim3(static_cast<unsigned>((p.cols + kThreads - 1) / kThreads), *partials),
                    dim3(kThreads), 0, s, 1, p, *partials);
}

}  // namespace

int norm_partials(int64_t rows) { return static_cast<int>(rows < 1 ? 1 : (rows > kMaxNormPartials ? kMaxNormPartials : rows)); }

cudaError_t launch_norm_backward(const NormBwdParams& p, int num_sms, cudaStream_t s) {
  const int64_t size = p.f32 ? 4 : 2, e16 = 16 / size;
  int partials = 0;
  cudaError_t e;
  if (p.cols > kMostCols || p.rows == 0) {
    e = p.f32 ? run_any<float>(p, num_sms, s, &partials) : run_any<uint16_t>(p, num_sms, s, &partials);
  } else {
    const bool vec = takes(p.dy, p.lddy, p.cols, size, 16) && takes(p.x, p.ldx, p.cols, size, 16) &&
                     takes(p.dx, p.lddx, p.cols, size, 16) && takes(p.q, p.ldq, p.cols, 1, e16) && takes(p.w, 0, 0, 1, 16);
    if (p.f32)
      e = vec ? run_norm_backward<float, true>(p, num_sms, s, &partials) : run_norm_backward<float, false>(p, num_sms, s, &partials);
    else
      e = vec ? run_norm_backward<uint16_t, true>(p, num_sms, s, &partials)
              : run_norm_backward<uint16_t, false>(p, num_sms, s, &partials);
  }
  if (e != cudaSuccess || partials == 0 || (p.dw == nullptr && p.db == nullptr)) return e;
  const int quad = p.cols % 4 == 0 ? 4 : 1;
  return launch_pdl(quad == 4 ? k_norm_params<4> : k_norm_params<1>,
                    dim3(static_cast<unsigned>((2 * p.cols / quad + 31) / 32)), dim3(kParamWarps * 32), 0, s, 1,
                    static_cast<const float*>(p.partial), partials, static_cast<int>(p.cols), p.w_f32 != 0, p.dw, p.db);
}

}  // namespace fp8q
