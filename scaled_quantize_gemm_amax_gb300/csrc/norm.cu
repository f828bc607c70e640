// norm.cu -- layer norm, forward.
//
//   m = sum x / H,  v = sum (x - m)^2 / H,  r = 1 / sqrt(v + eps),  xh = (x - m) r
//   y = xh w + b
// The normalised rows xh may be kept as 8-bit codes with one multiplier per 128 columns, from
// which the backward pass needs neither x nor m.  All sums are binary32.
//
// Bound by HBM: x once in, y (and the codes) once out.  A row stays in registers between its
// statistics and its output.
#include "norm.cuh"

namespace fp8q {

namespace {

constexpr int kBlockWarps = 24;   // 80 registers a thread
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Sum over a block of kThreads; the result is valid in every thread.
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float r = 0.0f;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) r += red[i];
  return r;
}

// 1 / sqrt(v): the approximate reciprocal root and one Newton step (no step at 0 and infinity,
// where it would make a NaN)
__device__ __forceinline__ float inv_sqrt(float v) {
  const float r = rsqrtf(v);
  const float e = fmaf(-v * r, r, 1.0f);
  return v > 0.0f && !is_inf_or_nan(v) ? fmaf(0.5f * e, r, r) : r;
}

// Rows of any width: one block per row, three passes over it (sum, squared differences, output).
template <typename T>
__global__ void __launch_bounds__(kThreads) k_norm_any(const NormParams p) {
  __shared__ float red[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t groups = (p.cols + 127) / 128;
  const float inv_n = 1.0f / static_cast<float>(p.cols);
  pdl_wait();
  pdl_launch_dependents();
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    T* y = static_cast<T*>(p.y) + row * p.ldy;
    float sum = 0.0f;
    for (int64_t c = threadIdx.x; c < p.cols; c += kThreads) sum += ld_elem(x + c);
    const float mean = block_sum(sum, red) * inv_n;
    float sq = 0.0f;
    for (int64_t c = threadIdx.x; c < p.cols; c += kThreads) {
      const float d = ld_elem(x + c) - mean;
      sq = fmaf(d, d, sq);
    }
    const float var = block_sum(sq, red) * inv_n;
    const float rstd = inv_sqrt(var + p.eps);
    if (threadIdx.x == 0) {
      if (p.mean != nullptr) p.mean[row] = mean;
      if (p.rstd != nullptr) p.rstd[row] = rstd;
    }
    for (int g = warp; g < groups; g += kWarps) {
      float xh[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = Piece<T, false>::col(g * 128, lane, i);
        xh[i] = 0.0f;
        if (c < p.cols) {
          xh[i] = (ld_elem(x + c) - mean) * rstd;
          const float w = p.w != nullptr ? ld_param(p.w, p.w_f32, c) : 1.0f;
          const float b = p.b != nullptr ? ld_param(p.b, p.w_f32, c) : 0.0f;
          st_elem(y + c, fmaf(xh[i], w, b));
        }
      }
      if (p.q != nullptr) {
        const float v[1][4] = {{xh[0], xh[1], xh[2], xh[3]}};
        store_copies<Piece<T, false>, 1>({p.q + row * p.ldq}, {p.s + row * groups}, {g * 128}, lane, static_cast<int>(p.cols),
                                         p.e5m2, v);
      }
    }
  }
}

// Rows of up to 16384 columns.  Each warp takes the mean and the sum of squared differences of
// its own 512 columns in two passes over registers; the warps' (n, mean, M2) are then joined by
//   M2 = sum M2_w + n_w (mean_w - mean)^2
// so a row costs one barrier and loses no digits to a large mean.
template <typename T, bool VECTOR, bool WIDE>
__global__ void __launch_bounds__((WIDE ? kNormWarpsMost : kBlockWarps) * 32)
    k_norm(const NormParams p, const int warps, const int stages) {
  using P = Piece<T, VECTOR>;
  constexpr int E = P::E, J = 16 / E;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float2 red[2][kNormWarpsMost];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = warp / warps, w_in = warp - group * warps;
  const int n_groups = (blockDim.x >> 5) / warps;
  const int64_t step = static_cast<int64_t>(gridDim.x) * n_groups;
  const int cols = static_cast<int>(p.cols), base = w_in * kNormWarpCols;
  const int copies = (cols + 127) / 128;
  const float n_w = static_cast<float>(min(cols - base, kNormWarpCols));
  const float inv_nw = 1.0f / n_w, inv_n = 1.0f / static_cast<float>(cols);
  // this thread's 16 bytes of piece j in stage s: ring + slot + (s * J + j) * 512
  const uint32_t slot = smem_u32(ring) + warp * stages * J * 512 + lane * 16;

  auto issue = [&](int64_t row, int s) {
    if constexpr (VECTOR) {
      if (row < p.rows) {
        const T* x = static_cast<const T*>(p.x) + row * p.ldx;
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const int c = P::col(base + j * P::WC, lane, 0);
          cp_async<16>(slot + (s * J + j) * 512, x + (c < cols ? c : 0), c < cols);
        }
      }
      cp_async_commit();
    }
  };
  pdl_wait();
  pdl_launch_dependents();
  int64_t row = static_cast<int64_t>(blockIdx.x) * n_groups + group;
  for (int s = 0; s < stages; ++s) issue(row + s * step, s);
  // weight and bias of this thread's columns, kept for all its rows (rows of more than kBlockWarps warps
  // have 64 registers a thread and read them again each time)
  float w[WIDE ? 1 : J][E], b[WIDE ? 1 : J][E];
  if constexpr (!WIDE) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      load_param<P, VECTOR>(p.w, p.w_f32, base + j * P::WC, lane, cols, 1.0f, w[j]);
      load_param<P, VECTOR>(p.b, p.w_f32, base + j * P::WC, lane, cols, 0.0f, b[j]);
    }
  }
  for (int s = 0, buf = 0; row < p.rows; row += step, s = s + 1 == stages ? 0 : s + 1, buf ^= 1) {
    float x[J][E];
    if constexpr (VECTOR) {
      cp_async_wait_oldest(stages);
#pragma unroll
      for (int j = 0; j < J; ++j)
        P::unpack(*reinterpret_cast<const uint4*>(ring + (slot - smem_u32(ring)) + (s * J + j) * 512), x[j]);
    } else {
      const T* in = static_cast<const T*>(p.x) + row * p.ldx;
#pragma unroll
      for (int j = 0; j < J; ++j) P::load(in, base + j * P::WC, lane, cols, x[j]);
    }
    float2 acc = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int i = 0; i < E; i += 2) acc = add2(acc, make_float2(x[j][i], x[j][i + 1]));
    float mean = warp_sum(acc.x + acc.y) * inv_nw;
    acc = both(0.0f);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      float2 sq = both(0.0f);
#pragma unroll
      for (int i = 0; i < E; i += 2) {
        float2 d = add2(make_float2(x[j][i], x[j][i + 1]), both(-mean));
        if (!VECTOR) {
          if (!P::valid(base + j * P::WC, lane, cols, i)) d.x = 0.0f;
          if (!P::valid(base + j * P::WC, lane, cols, i + 1)) d.y = 0.0f;
        }
        sq = fma2(d, d, sq);
      }
      if (!VECTOR || P::valid(base + j * P::WC, lane, cols, 0)) acc = add2(acc, sq);
    }
    float m2 = warp_sum(acc.x + acc.y);
    if (warps > 1) {
      if (lane == 0) red[buf][warp] = make_float2(mean, m2);
      group_sync(group, warps);
      // lane l joins warp l's part of the row (the other buffer is written before this one is reused)
      const float2 v = lane < warps ? red[buf][group * warps + lane] : make_float2(0.0f, 0.0f);
      const float n_l = lane < warps ? static_cast<float>(min(cols - lane * kNormWarpCols, kNormWarpCols)) : 0.0f;
      mean = warp_sum(n_l * v.x) * inv_n;
      const float d = v.x - mean;
      m2 = warp_sum(lane < warps ? fmaf(n_l * d, d, v.y) : 0.0f);
    }
    const float rstd = inv_sqrt(fmaf(m2, inv_n, p.eps));
    if (w_in == 0 && lane == 0) {
      if (p.mean != nullptr) p.mean[row] = mean;
      if (p.rstd != nullptr) p.rstd[row] = rstd;
    }
    issue(row + stages * step, s);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c0 = base + j * P::WC;
      float y[E];
      if constexpr (WIDE) {
        load_param<P, VECTOR>(p.w, p.w_f32, c0, lane, cols, 1.0f, w[0]);
        load_param<P, VECTOR>(p.b, p.w_f32, c0, lane, cols, 0.0f, b[0]);
      }
      const int k = WIDE ? 0 : j;
#pragma unroll
      for (int i = 0; i < E; i += 2) {
        const float2 h = mul2(add2(make_float2(x[j][i], x[j][i + 1]), both(-mean)), both(rstd));
        const float2 v = fma2(h, make_float2(w[k][i], w[k][i + 1]), make_float2(b[k][i], b[k][i + 1]));
        x[j][i] = h.x;
        x[j][i + 1] = h.y;
        y[i] = v.x;
        y[i + 1] = v.y;
      }
      P::store(static_cast<T*>(p.y) + row * p.ldy, c0, lane, cols, y);
    }
    if (p.q != nullptr) {
      uint8_t* const q = p.q + row * p.ldq;
      float* const s_row = p.s + row * copies;
      if constexpr (J == 2)
        store_copies<P, 2>({q, q}, {s_row, s_row}, {base, base + P::WC}, lane, cols, p.e5m2, x);
      else
        store_copies<P, 4>({q, q, q, q}, {s_row, s_row, s_row, s_row}, {base, base + P::WC, base + 2 * P::WC, base + 3 * P::WC},
                           lane, cols, p.e5m2, x);
    }
  }
}

template <typename T, bool VECTOR>
cudaError_t run_norm(const NormParams& p, int num_sms, cudaStream_t s) {
  // copies of the rows in flight: 16 columns a lane
  const NormPlan n = norm_plan(p.rows, p.cols, kBlockWarps, VECTOR ? kNormWarpCols * static_cast<int>(sizeof(T)) : 0, num_sms);
  static std::atomic<bool> done[2][kMaxDevices];
  const dim3 block(static_cast<unsigned>(n.warps * n.groups * 32));
  auto kernel = n.wide ? k_norm<T, VECTOR, true> : k_norm<T, VECTOR, false>;
  const cudaError_t e = ensure_smem_limit(kernel, kNormSmem, done[n.wide]);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(n.blocks), block, n.smem, s, 1, p, n.warps, n.stages);
}

}  // namespace

cudaError_t launch_norm(const NormParams& p, int num_sms, cudaStream_t s) {
  const int64_t size = p.f32 ? 4 : 2;
  if (p.cols > kNormWarpsMost * kNormWarpCols) {
    const int64_t cap = static_cast<int64_t>(num_sms) * 8;
    const dim3 grid(static_cast<unsigned>(p.rows < cap ? p.rows : cap));
    return p.f32 ? launch_pdl(k_norm_any<float>, grid, dim3(kThreads), 0, s, 1, p)
                 : launch_pdl(k_norm_any<uint16_t>, grid, dim3(kThreads), 0, s, 1, p);
  }
  const bool vec = takes(p.x, p.ldx, p.cols, size, 16) && takes(p.y, p.ldy, p.cols, size, 16) &&
                   takes(p.q, p.ldq, p.cols, 1, 16 / size) && takes(p.w, 0, 0, 1, 16) && takes(p.b, 0, 0, 1, 16);
  if (p.f32) return vec ? run_norm<float, true>(p, num_sms, s) : run_norm<float, false>(p, num_sms, s);
  return vec ? run_norm<uint16_t, true>(p, num_sms, s) : run_norm<uint16_t, false>(p, num_sms, s);
}

}  // namespace fp8q
