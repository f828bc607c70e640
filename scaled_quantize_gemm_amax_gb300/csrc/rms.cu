// rms.cu -- RMS norm, forward, with the residual's addition before it and an 8-bit output behind it.
//
//   h = x + residual (rounded to the data's type: the stream as it is kept),
//   r = 1 / sqrt(sum h^2 / H + eps),  y = h r w
// y leaves in the data's type, as codes with the scales of any row-wise recipe, or both.  The codes
// are taken from y's binary32 values.  All sums are binary32.
//
// Bound by HBM: x and the residual once in, h and y (or the codes) once out.  A row stays in
// registers between its sum and its output; the weight stays in shared memory for the whole walk.
// With a residual, bf16: 8192x4096 to tiled MXFP8 codes 39 us (6.0 TB/s, 0.89 of what a copy reaches), 65536x4096 to 1x128 codes
// 275 (1.01), 131072x256 38, 2048x16384 40; binary32 8192x4096 70 (0.92); without a residual 8192x4096 21 (0.70), 65536x4096 140
// (0.85); one row of 4096 3.  Unaligned, to y: bf16 8192x4099 64 (0.62), binary32 4096x4099 48 (0.83).  Rows of more than
// kMostCols columns are read twice: bf16 1x16512 9, 2048x16512 72 (0.49).
#include "rms.cuh"

namespace fp8q {

namespace {

// warps of a block at V values a lane: 80 registers a thread, 64 at 8 values; unaligned binary32 at 32 values, which
// only the widest rows take, spills at 80 and has 128
template <typename T, bool VECTOR, int V>
constexpr int kBlockWarps = V == 8 ? 32 : (V == 32 && !VECTOR && sizeof(T) == 4 ? 16 : 24);
// Bytes of a block's rows and of its stages (rms_plan).  With a residual, bf16 and 1x128 codes, 65536x4096: 64 KB 275 us,
// 96 KB 300, two stages of 96 KB 319; 8192x4096 39.7, 39.8 and 43.5.  Unaligned rows take 2.2 times the instructions, whose waits
// (issue slots 39 % busy, shared memory 44 %) more warps hide, as many as fit: 8192x4099 65 us with 96 KB, 73 with 64.
template <bool VECTOR>
constexpr int kMost = (VECTOR ? 64 : 96) * 1024;
constexpr int kInFlight = 64 * 1024;
constexpr int kMostCols = 16384;   // of a row held in registers, its weight in shared memory
constexpr int kThreads = 512;

// 1 / sqrt(v): the approximate reciprocal root and one Newton step (no step at 0 and infinity,
// where it would make a NaN)
__device__ __forceinline__ float inv_sqrt(float v) {
  const float r = rsqrtf(v);
  const float e = fmaf(-v * r, r, 1.0f);
  return v > 0.0f && !is_inf_or_nan(v) ? fmaf(0.5f * e, r, r) : r;
}

// Where a row's E8M0 byte of block b lies: row-major, or in the tiled layout's atoms of 128 rows x 4 blocks.
__device__ __forceinline__ int64_t mx_at(bool tiled, int64_t row, int64_t blocks, int64_t b) {
  return tiled ? ((row / 128 * (blocks / 4) + b / 4) * 512 + row % 32 * 16 + row % 128 / 32 * 4 + b % 4) : row * blocks + b;
}

// The codes of N consecutive pieces of a row by the MXFP8 rule, a block of 32 columns its
// power-of-two scale.  q: the lane's first code of the first piece; c0: that piece's first column
// in the row.  Each lane finds one piece's exponent (lane % N) and has the others' from its neighbours.
template <typename P, int N>
__device__ __forceinline__ void store_mx(const RmsParams& p, uint8_t* q, int64_t row, int c0, int lane, int left,
                                         const float (&v)[N][P::E]) {
  uint8_t* const s = static_cast<uint8_t*>(p.s);
  const int64_t blocks = (p.cols + 31) / 32;
  const bool e5m2 = p.e5m2;
  const int top = fmax_exp_of(e5m2);
  if constexpr (P::kStrided) {
    // value i of all lanes is one block
#pragma unroll
    for (int j = 0; j < N; ++j) {
      float sc = 1.0f;
      float by[P::E];
#pragma unroll
      for (int i = 0; i < P::E; ++i) {
        float a = P::has(left - j * P::WC, i) ? max_abs3(0.0f, v[j][i], 0.0f) : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
        const int e = p.mx_floor ? mx_exponent_floor(a, top) : mx_exponent(a, top);
        sc = pow2_neg(e);
        by[i] = __fmul_rn(v[j][i], sc);
        if (lane == 0 && P::has(left - j * P::WC, i))
          s[mx_at(p.mx_tiled, row, blocks, (c0 + j * P::WC + P::at(i)) / 32)] = static_cast<uint8_t>(e + 127);
      }
      if (e5m2) P::template encode<true>(q + j * P::WC, left - j * P::WC, by, 1.0f);
      else P::template encode<false>(q + j * P::WC, left - j * P::WC, by, 1.0f);
    }
  } else {
    constexpr int W = 32 / P::E;   // lanes of a block
    float a[N];
#pragma unroll
    for (int i = 0; i < N; ++i) a[i] = P::amax(v[i], left - i * P::WC);
    const float most = group_max<N, W>(a, lane);
    const int e = p.mx_floor ? mx_exponent_floor(most, top) : mx_exponent(most, top);
    // lanes i < N of the block's own write the byte of piece i
    const int i_mine = lane % N, c = c0 + P::first(lane) + i_mine * P::WC;
    if (lane % W < N && left > i_mine * P::WC) s[mx_at(p.mx_tiled, row, blocks, c / 32)] = static_cast<uint8_t>(e + 127);
    const float mine = pow2_neg(e);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float sc = N == 1 ? mine : __shfl_sync(0xFFFFFFFFu, mine, (lane & ~(N - 1)) | i);
      if (e5m2) P::template encode<true>(q + i * P::WC, left - i * P::WC, v[i], sc);
      else P::template encode<false>(q + i * P::WC, left - i * P::WC, v[i], sc);
    }
  }
}

// The codes of N consecutive pieces by the call's recipe; `amax` takes the per-tensor recipe's max |y|.
template <typename P, int N>
__device__ __forceinline__ void store_codes(const RmsParams& p, int64_t row, int c0, int lane, int left, float scale,
                                            const float (&v)[N][P::E], float& amax) {
  uint8_t* const q = p.q + row * p.ldq + c0 + P::first(lane);
  if (p.recipe == kMx) {
    store_mx<P, N>(p, q, row, c0, lane, left, v);
  } else if (p.recipe == kBlock1x128) {
    const int64_t groups = (p.cols + 127) / 128;
    store_copies<P, N>(q, static_cast<float*>(p.s) + row * groups + (c0 + P::first(lane)) / 128, lane, left, p.e5m2, v);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      amax = fmaxf(amax, P::amax(v[i], left - i * P::WC));
      if (p.e5m2) P::template encode<true>(q + i * P::WC, left - i * P::WC, v[i], scale);
      else P::template encode<false>(q + i * P::WC, left - i * P::WC, v[i], scale);
    }
  }
}

// max |y| of a warp's values into p.amax, on the non-negative float bits, which order like the values
__device__ __forceinline__ void join_amax(const RmsParams& p, float amax, int lane) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
  if (lane == 0 && amax > 0.0f) atomicMax(reinterpret_cast<unsigned int*>(p.amax), __float_as_uint(amax));
}

// the multiplier of the per-tensor recipe's codes
__device__ __forceinline__ void store_inverse(const RmsParams& p, float scale) {
  if (p.q != nullptr && p.recipe == kTensor && p.s != nullptr && blockIdx.x == 0 && threadIdx.x == 0)
    *static_cast<float*>(p.s) = recip_rn(scale);
}

// h of a piece: x + residual rounded to the data's type (packed too)
template <typename P>
__device__ __forceinline__ uint4 add_residual(float (&x)[P::E], const float (&r)[P::E]) {
#pragma unroll
  for (int i = 0; i < P::E; i += 2) {
    const float2 s = add2(make_float2(x[i], x[i + 1]), make_float2(r[i], r[i + 1]));
    x[i] = s.x;
    x[i + 1] = s.y;
  }
  const uint4 h = P::pack(x);
  P::unpack(h, x);
  return h;
}

// Rows of any width: one block per row, two passes over it.
template <typename T, bool VECTOR>
__global__ void __launch_bounds__(kThreads) k_rms_any(const RmsParams p) {
  using P = Piece<T, VECTOR>;
  __shared__ float red[kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, cols = static_cast<int>(p.cols);
  const float inv_n = 1.0f / static_cast<float>(cols);
  pdl_wait();
  pdl_launch_dependents();
  const float scale = p.q != nullptr && p.recipe == kTensor ? *p.scale : 1.0f;
  store_inverse(p, scale);
  float amax = 0.0f;
  // the lane's h of the piece at column c0 (0 past the row's end)
  auto piece = [&](int64_t row, int c0, float (&h)[1][P::E]) -> uint4 {
    const int c = c0 + P::first(lane), left = cols - c;
    P::load(static_cast<const T*>(p.x) + row * p.ldx + c, c, left, h);
    float r[1][P::E] = {};
    if (p.res != nullptr) P::load(static_cast<const T*>(p.res) + row * p.ldr + c, c, left, r);
    return add_residual<P>(h[0], r[0]);
  };
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    float sum = 0.0f;
    for (int c0 = warp * P::WC; c0 < cols; c0 += kThreads / 32 * P::WC) {
      float h[1][P::E];
      piece(row, c0, h);
#pragma unroll
      for (int i = 0; i < P::E; ++i)
        if (P::has(cols - c0 - P::first(lane), i)) sum = fmaf(h[0][i], h[0][i], sum);
    }
    sum = warp_sum(sum);
    __syncthreads();
    if (lane == 0) red[warp] = sum;
    __syncthreads();
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) sum += red[i];
    const float rstd = inv_sqrt(fmaf(sum, inv_n, p.eps));
    if (threadIdx.x == 0 && p.rstd != nullptr) p.rstd[row] = rstd;
    for (int c0 = warp * P::WC; c0 < cols; c0 += kThreads / 32 * P::WC) {
      const int c = c0 + P::first(lane), left = cols - c;
      float v[1][P::E], w[P::E];
      const uint4 h[1] = {piece(row, c0, v)};
      if (p.h != nullptr) P::store_raw(static_cast<T*>(p.h) + row * p.ldh + c, left, h);
      P::load_param(p.w, p.w_f32, c, left, 1.0f, w);
#pragma unroll
      for (int i = 0; i < P::E; ++i) v[0][i] = __fmul_rn(__fmul_rn(v[0][i], rstd), w[i]);
      if (p.y != nullptr) P::store(static_cast<T*>(p.y) + row * p.ldy + c, left, v);
      if (p.q != nullptr) store_codes<P, 1>(p, row, c0, lane, left, scale, v, amax);
    }
  }
  if (p.amax != nullptr) join_amax(p, amax, lane);
}

// Rows of up to kMostCols columns, V values a lane; a group of `warps` warps holds a row, and a row costs
// one barrier.
template <typename T, bool VECTOR, int V>
__global__ void __launch_bounds__(kBlockWarps<T, VECTOR, V> * 32) k_rms(const RmsParams p, const int warps, const int stages, const int ring) {
  using P = Piece<T, VECTOR>;
  constexpr int E = P::E, J = V / E, kCols = 32 * V;
  using Part = RowPart<P, kCols, VECTOR, T>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float red[2][kBlockWarps<T, VECTOR, V>];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = warp / warps, w_in = warp - group * warps;
  const int n_groups = (blockDim.x >> 5) / warps, step = gridDim.x * n_groups;
  const int rows = static_cast<int>(p.rows), cols = static_cast<int>(p.cols);
  const bool res = p.res != nullptr;
  const int stage_bytes = Part::kBytes * (res ? 2 : 1);
  // this lane's first column and the columns from there to the row's end
  const int base = w_in * kCols, c = base + P::first(lane), left = cols - c;
  const float inv_n = 1.0f / static_cast<float>(cols);
  uint8_t* const slots = smem + ring + warp * stages * stage_bytes;   // the warp's part of its group's next rows
  float* const ws = reinterpret_cast<float*>(smem);

  auto issue = [&](int row, int s) {
    if (row < rows) {
      uint8_t* const to = slots + s * stage_bytes;
      const int64_t bx = static_cast<int64_t>(row) * p.ldx, br = static_cast<int64_t>(row) * p.ldr;
      Part::start(to, static_cast<const T*>(p.x) + bx, bx, base, cols, lane);
      if (res) Part::start(to + Part::kBytes, static_cast<const T*>(p.res) + br, br, base, cols, lane);
    }
    cp_async_commit();
  };
  pdl_wait();
  pdl_launch_dependents();
  int row = blockIdx.x * n_groups + group;
  start_param<P, V>(p.w, p.w_f32, cols, warps, 1.0f, ws);
  cp_async_commit();
  for (int s = 0; s < stages; ++s) issue(row + s * step, s);
  const float scale = p.q != nullptr && p.recipe == kTensor ? *p.scale : 1.0f;
  store_inverse(p, scale);
  float amax = 0.0f;
  cp_async_wait_oldest(stages + 1);
  settle_param<P, V>(p.w, p.w_f32, warps, ws);
  __syncthreads();
  for (int s = 0, buf = 0; row < rows; row += step, buf ^= 1) {
    float x[J][E];
    cp_async_wait_oldest(stages);
    if (!VECTOR) __syncwarp();   // other lanes copied some of this lane's elements
    const uint8_t* const slot = slots + s * stage_bytes;
    const int64_t r64 = row;
    Part::read(slot, Part::past(static_cast<const T*>(p.x) + r64 * p.ldx + base), lane, x);
    if (res) {
      const int m = Part::past(static_cast<const T*>(p.res) + r64 * p.ldr + base);
      uint4 h[J];
#pragma unroll
      for (int j = 0; j < J; ++j) {
        float r[E];
        Part::read(slot + Part::kBytes, m, lane, j, r);
        h[j] = add_residual<P>(x[j], r);
        if constexpr (VECTOR) {   // at once, without waiting in registers
          const uint4 one[1] = {h[j]};
          if (p.h != nullptr) P::store_raw(static_cast<T*>(p.h) + r64 * p.ldh + c + j * P::WC, left - j * P::WC, one);
        }
      }
      if constexpr (!VECTOR)
        if (p.h != nullptr) P::store_raw(static_cast<T*>(p.h) + r64 * p.ldh + c, left, h);
    }
    float2 acc = both(0.0f);
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int i = 0; i < E; i += 2) {   // past the row's end lie zeros
        const float2 d = {x[j][i], x[j][i + 1]};
        acc = fma2(d, d, acc);
      }
    float sum = warp_sum(acc.x + acc.y);
    if (warps > 1) {
      if (lane == 0) red[buf][warp] = sum;
      group_sync(group, warps);
      // lane l joins warp l's part of the row (the other buffer is written before this one is reused)
      sum = warp_sum(lane < warps ? red[buf][group * warps + lane] : 0.0f);
    }
    const float rstd = inv_sqrt(fmaf(sum, inv_n, p.eps));
    if (w_in == 0 && lane == 0 && p.rstd != nullptr) p.rstd[row] = rstd;
    if (!VECTOR) __syncwarp();   // other lanes have read this lane's granules
    issue(row + stages * step, s);
    s = s + 1 == stages ? 0 : s + 1;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      float w[E];
      read_param<P, V>(ws, w_in, j, lane, w);
#pragma unroll
      for (int i = 0; i < E; i += 2) {
        const float2 o = mul2(mul2(make_float2(x[j][i], x[j][i + 1]), both(rstd)), make_float2(w[i], w[i + 1]));
        x[j][i] = o.x;
        x[j][i + 1] = o.y;
      }
    }
    if (p.y != nullptr) {
      uint4 y[J];
#pragma unroll
      for (int j = 0; j < J; ++j) y[j] = P::pack(x[j]);
      P::store_raw(static_cast<T*>(p.y) + r64 * p.ldy + c, left, y);
    }
    if (p.q != nullptr) {
      constexpr int N = J < 4 ? J : 4;
#pragma unroll
      for (int j = 0; j < J; j += N) {
        float v[N][E];
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
          for (int i = 0; i < E; ++i) v[k][i] = x[j + k][i];
        store_codes<P, N>(p, r64, base + j * P::WC, lane, left - j * P::WC, scale, v, amax);
      }
    }
  }
  if (p.amax != nullptr) join_amax(p, amax, lane);
}

template <typename T, bool VECTOR, int V>
cudaError_t run_rms(const RmsParams& p, int num_sms, cudaStream_t s) {
  const int part = RowPart<Piece<T, VECTOR>, 32 * V, VECTOR, T>::kBytes;
  const NormPlan n = rms_plan(p.rows, p.cols, 32 * V, kBlockWarps<T, VECTOR, V>, part * (p.res != nullptr ? 2 : 1), kMost<VECTOR>, kInFlight, 1,
                              num_sms);
  static std::atomic<bool> done[kMaxDevices];
  const cudaError_t e = ensure_smem_limit(k_rms<T, VECTOR, V>, kNormSmem, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_rms<T, VECTOR, V>, dim3(n.blocks), dim3(static_cast<unsigned>(n.warps * n.groups * 32)), n.smem, s, 1, p,
                    n.warps, n.stages, n.ring);
}

// Values a lane: 8 for rows of up to 256 columns; 32 halve what a row costs besides its values; 16 where that would leave
// lanes empty (up to 512 columns) or where a row's latency counts and there are warps to spare, and for unaligned rows,
// which wait for their own instructions, while a row's ends cost more than its middle: binary32 (4096x4099 with a residual 45
// us, 73 with 32 values; 2048x9001 50 and 77) and bf16 up to 3584 columns (16384x1003 42 and 52, 8192x3001 50 and 51; 8192x4099 74 and 65).
template <typename T, bool VECTOR>
cudaError_t run_rms(const RmsParams& p, int num_sms, cudaStream_t s) {
  constexpr int64_t kMost16 = kBlockWarps<T, VECTOR, 16> * 512, kMostUnaligned = sizeof(T) == 4 ? kMost16 : 7 * 512;
  if (p.cols <= 256) return run_rms<T, VECTOR, 8>(p, num_sms, s);
  if (p.cols <= 512 || (p.rows <= num_sms && p.cols <= kMost16) || (!VECTOR && p.cols <= kMostUnaligned))
    return run_rms<T, VECTOR, 16>(p, num_sms, s);
  return run_rms<T, VECTOR, 32>(p, num_sms, s);
}

}  // namespace

cudaError_t launch_rms(const RmsParams& p, int num_sms, cudaStream_t s) {
  const int64_t size = p.f32 ? 4 : 2;
  const bool vec = takes(p.x, p.ldx, p.cols, size, 16) && takes(p.res, p.ldr, p.cols, size, 16) &&
                   takes(p.h, p.ldh, p.cols, size, 16) && takes(p.y, p.ldy, p.cols, size, 16) &&
                   takes(p.q, p.ldq, p.cols, 1, 16 / size) && takes(p.w, 0, 0, 1, 16);
  if (p.cols > kMostCols) {
    const int64_t cap = static_cast<int64_t>(num_sms) * 8;
    const dim3 grid(static_cast<unsigned>(p.rows < cap ? p.rows : cap));
    if (p.f32) return launch_pdl(vec ? k_rms_any<float, true> : k_rms_any<float, false>, grid, dim3(kThreads), 0, s, 1, p);
    return launch_pdl(vec ? k_rms_any<uint16_t, true> : k_rms_any<uint16_t, false>, grid, dim3(kThreads), 0, s, 1, p);
  }
  if (p.f32) return vec ? run_rms<float, true>(p, num_sms, s) : run_rms<float, false>(p, num_sms, s);
  return vec ? run_rms<uint16_t, true>(p, num_sms, s) : run_rms<uint16_t, false>(p, num_sms, s);
}

}  // namespace fp8q
