// norm.cu -- layer norm, forward.
//
//   m = sum x / H,  v = sum (x - m)^2 / H,  r = 1 / sqrt(v + eps),  xh = (x - m) r
//   y = xh w + b
// The normalised rows xh may be kept as 8-bit codes with one multiplier per 128 columns, from
// which the backward pass needs neither x nor m.  All sums are binary32.
//
// Bound by HBM: x once in, y (and the codes) once out.  A row stays in registers between its
// statistics and its output; weight and bias stay in shared memory for the whole walk.
// 8192x4096 bf16 with codes 32.6 us (5.2 TB/s, 0.76 of what a copy reaches), 65536x4096 0.89,
// 16384x4096 without codes 0.87, one row of 4096 3.1 us; binary32 8192x4096 44.5 us (0.89), 2048x16384, one
// row in flight a block, 46.2 (0.86).  What is left at 8192x4096: launch, the
// first rows' way in and the last ones' way out (5 us), and SMs that finish at different times (the
// rows are dealt out beforehand: 26 to 32 us).  Rows handed out on demand by cluster launch control
// took a 25th warp a block and with it registers from the others: 36.4 us.
#include "norm.cuh"

namespace fp8q {

namespace {

// warps of a block at V values a lane: 80 registers a thread, 64 at 8 values
template <int V>
constexpr int kBlockWarps = V == 8 ? 32 : 24;
constexpr int kMostCols = 16384;  // of a row held in registers, its weight and bias in shared memory
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

// Rows of any width: one block per row, three passes over it (sum, squared differences, output), which a
// row of more than kMostCols columns takes: 2048x20480 bf16 125 us (0.20), binary32 90 (0.55).
template <typename T>
__global__ void __launch_bounds__(kThreads) k_norm_any(const NormParams p) {
  __shared__ float red[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int cols = static_cast<int>(p.cols), groups = (cols + 127) / 128;
  const float inv_n = 1.0f / static_cast<float>(cols);
  pdl_wait();
  pdl_launch_dependents();
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    T* y = static_cast<T*>(p.y) + row * p.ldy;
    float sum = 0.0f;
    for (int c = threadIdx.x; c < cols; c += kThreads) sum += ld_elem(x + c);
    const float mean = block_sum(sum, red) * inv_n;
    float sq = 0.0f;
    for (int c = threadIdx.x; c < cols; c += kThreads) {
      const float d = ld_elem(x + c) - mean;
      sq = fmaf(d, d, sq);
    }
    const float var = block_sum(sq, red) * inv_n;
    const float rstd = inv_sqrt(var + p.eps);
    if (threadIdx.x == 0) {
      if (p.mean != nullptr) p.mean[row] = mean;
      if (p.rstd != nullptr) p.rstd[row] = rstd;
    }
    using P = Piece<T, false>;
    for (int c0 = warp * P::WC; c0 < cols; c0 += kWarps * P::WC) {
      const int c = c0 + P::first(lane), left = cols - c;
      float v[1][P::E], w[P::E], b[P::E], xh[1][P::E];
      P::load(x + c, c, left, v);
      P::load_param(p.w, p.w_f32, c, left, 1.0f, w);
      P::load_param(p.b, p.w_f32, c, left, 0.0f, b);
#pragma unroll
      for (int i = 0; i < P::E; ++i) {
        xh[0][i] = (v[0][i] - mean) * rstd;
        v[0][i] = fmaf(xh[0][i], w[i], b[i]);
      }
      P::store(y + c, left, v);
      if (p.q != nullptr) store_copies<P, 1>(p.q + row * p.ldq + c, p.s + row * groups + c / 128, lane, left, p.e5m2, xh);
    }
  }
}

// Rows of up to kMostCols columns, V values a lane.  Each warp takes the mean and the
// sum of squared differences of its own columns in two passes over registers; the warps'
// (n, mean, M2) are then joined by
//   M2 = sum M2_w + n_w (mean_w - mean)^2
// so a row costs one barrier and loses no digits to a large mean.
template <typename T, bool VECTOR, int V>
__global__ void __launch_bounds__(kBlockWarps<V> * 32) k_norm(const NormParams p, const int warps, const int stages, const int ring) {
  using P = Piece<T, VECTOR>;
  constexpr int E = P::E, J = V / E, kCols = 32 * V;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float2 red[2][kBlockWarps<V>];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = warp / warps, w_in = warp - group * warps;
  const int n_groups = (blockDim.x >> 5) / warps, step = gridDim.x * n_groups;
  const int rows = static_cast<int>(p.rows), cols = static_cast<int>(p.cols), groups8 = (cols + 127) / 128;
  const int ldx = static_cast<int>(p.ldx), ldy = static_cast<int>(p.ldy), ldq = static_cast<int>(p.ldq);
  using Part = RowPart<P, kCols, VECTOR, T>;
  // this lane's first column and the columns from there to the row's end
  const int base = w_in * kCols, c = base + P::first(lane), left = cols - c;
  const float inv_nw = 1.0f / static_cast<float>(min(cols - w_in * kCols, kCols)), inv_n = 1.0f / static_cast<float>(cols);
  // columns of the warp that this lane joins below
  const float n_l = lane < warps ? static_cast<float>(min(cols - lane * kCols, kCols)) : 0.0f;
  uint8_t* const slots = smem + ring + warp * stages * Part::kBytes;   // the warp's part of its group's next rows
  float* const ws = reinterpret_cast<float*>(smem);
  float* const bs = ws + warps * kCols;

  auto issue = [&](int row, int s) {
    if (row < rows) {
      const int64_t before = static_cast<int64_t>(row) * ldx;
      Part::start(slots + s * Part::kBytes, static_cast<const T*>(p.x) + before, before, base, cols, lane);
    }
    cp_async_commit();
  };
  pdl_wait();
  pdl_launch_dependents();
  int row = blockIdx.x * n_groups + group;
  start_param<P, V>(p.w, p.w_f32, cols, warps, 1.0f, ws);
  start_param<P, V>(p.b, p.w_f32, cols, warps, 0.0f, bs);
  cp_async_commit();
  for (int s = 0; s < stages; ++s) issue(row + s * step, s);
  cp_async_wait_oldest(stages + 1);
  settle_param<P, V>(p.w, p.w_f32, warps, ws);
  settle_param<P, V>(p.b, p.w_f32, warps, bs);
  __syncthreads();
  for (int s = 0, buf = 0; row < rows; row += step, buf ^= 1) {
    float x[J][E];
    cp_async_wait_oldest(stages);
    if (!VECTOR) __syncwarp();   // other lanes copied some of this lane's elements
    Part::read(slots + s * Part::kBytes, Part::past(static_cast<const T*>(p.x) + static_cast<int64_t>(row) * ldx + base), lane, x);
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
          if (!P::has(left - j * P::WC, i)) d.x = 0.0f;
          if (!P::has(left - j * P::WC, i + 1)) d.y = 0.0f;
        }
        sq = fma2(d, d, sq);
      }
      if (!VECTOR || left > j * P::WC) acc = add2(acc, sq);
    }
    float m2 = warp_sum(acc.x + acc.y);
    if (warps > 1) {
      if (lane == 0) red[buf][warp] = make_float2(mean, m2);
      group_sync(group, warps);
      // lane l joins warp l's part of the row (the other buffer is written before this one is reused)
      const float2 v = lane < warps ? red[buf][group * warps + lane] : make_float2(0.0f, 0.0f);
      mean = warp_sum(n_l * v.x) * inv_n;
      const float d = v.x - mean;
      m2 = warp_sum(fmaf(n_l * d, d, v.y));
    }
    const float rstd = inv_sqrt(fmaf(m2, inv_n, p.eps));
    if (w_in == 0 && lane == 0) {
      if (p.mean != nullptr) p.mean[row] = mean;
      if (p.rstd != nullptr) p.rstd[row] = rstd;
    }
    if (!VECTOR) __syncwarp();   // other lanes have read this lane's granules
    issue(row + stages * step, s);
    s = s + 1 == stages ? 0 : s + 1;
    uint4 y[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      float v[E], w[E], b[E];
      read_param<P, V>(ws, w_in, j, lane, w);
      read_param<P, V>(bs, w_in, j, lane, b);
#pragma unroll
      for (int i = 0; i < E; i += 2) {
        const float2 h = mul2(add2(make_float2(x[j][i], x[j][i + 1]), both(-mean)), both(rstd));
        const float2 o = fma2(h, make_float2(w[i], w[i + 1]), make_float2(b[i], b[i + 1]));
        x[j][i] = h.x;
        x[j][i + 1] = h.y;
        v[i] = o.x;
        v[i + 1] = o.y;
      }
      y[j] = P::pack(v);
      if constexpr (VECTOR) {   // at once, without waiting in registers
        const uint4 one[1] = {y[j]};
        P::store_raw(static_cast<T*>(p.y) + static_cast<int64_t>(row) * ldy + c + j * P::WC, left - j * P::WC, one);
      }
    }
    if constexpr (!VECTOR) P::store_raw(static_cast<T*>(p.y) + static_cast<int64_t>(row) * ldy + c, left, y);
    if (p.q != nullptr) {
      constexpr int N = J < 4 ? J : 4;
      uint8_t* const q = p.q + static_cast<int64_t>(row) * ldq + c;
      float* const s8 = p.s + static_cast<int64_t>(row) * groups8 + c / 128;
#pragma unroll
      for (int j = 0; j < J; j += N) {
        float v[N][E];
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
          for (int i = 0; i < E; ++i) v[k][i] = x[j + k][i];
        store_copies<P, N>(q + j * P::WC, s8 + j * P::WC / 128, lane, left - j * P::WC, p.e5m2, v);
      }
    }
  }
}

template <typename T, bool VECTOR, int V>
cudaError_t run_norm(const NormParams& p, int num_sms, cudaStream_t s) {
  const NormPlan n = norm_plan(p.rows, p.cols, 32 * V, kBlockWarps<V>, 2,
                               RowPart<Piece<T, VECTOR>, 32 * V, VECTOR, T>::kBytes, num_sms);
  static std::atomic<bool> done[kMaxDevices];
  const cudaError_t e = ensure_smem_limit(k_norm<T, VECTOR, V>, kNormSmem, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_norm<T, VECTOR, V>, dim3(n.blocks), dim3(static_cast<unsigned>(n.warps * n.groups * 32)), n.smem, s, 1, p,
                    n.warps, n.stages, n.ring);
}

// 32 values a lane halve what a row costs besides its values (sums over lanes and warps,
// addresses); 16 where that would leave lanes empty (rows of up to 512 columns) or where a row's
// latency counts and there are warps to spare (no more rows than SMs); 8 where 16 would leave half
// of them empty (up to 256 columns: 131072x128 with codes 37 us, 53 with 16 values; 262144x256 73 and
// 106), and there 32 warps an SM, since a row is then mostly sums over lanes (24: 40 and 78 us).
// Unaligned bf16 at 32 values spills 32 bytes a thread at its 80 registers.
template <typename T, bool VECTOR>
cudaError_t run_norm(const NormParams& p, int num_sms, cudaStream_t s) {
  if (p.cols <= 256) return run_norm<T, VECTOR, 8>(p, num_sms, s);
  if (p.cols <= 512 || (p.rows <= num_sms && p.cols <= kBlockWarps<16> * 512)) return run_norm<T, VECTOR, 16>(p, num_sms, s);
  return run_norm<T, VECTOR, 32>(p, num_sms, s);
}

}  // namespace

cudaError_t launch_norm(const NormParams& p, int num_sms, cudaStream_t s) {
  const int64_t size = p.f32 ? 4 : 2;
  if (p.cols > kMostCols) {
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
