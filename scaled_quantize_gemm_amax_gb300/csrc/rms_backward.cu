// rms_backward.cu -- RMS norm, backward.
//
//   g = dy w,  xh = h r,  c = sum g xh / H,  dx = r (g - xh c) + dh
//   dw = sum over rows of dy xh
// dh is the gradient that reaches h by the residual stream; dx is the gradient of both x and the
// residual.  All sums are binary32, in an order that depends on the shape alone.
//
// Bound by HBM: dy, h and dh once in, dx once out.  A thread owns the same columns for all the rows
// of its group, so the column sums stay in registers over the whole walk; they leave as one partial
// sum a block, added up by a second, small launch.  Few rows take one launch of another kind (k_rms_backward_few).
// bf16 with dh: 8192x4096 44 to 46 us (6.0 TB/s, 0.89 of what a copy reaches), 65536x4096 307 (1.03), 4096x8192 46; without
// dh 2048x12288 32 (0.69), 8192x12288 95 (0.94): what does not grow with the rows is the weights' way to every SM (1.8
// us) and the column sums (4.4 us, the second launch included).  binary32 8192x4096 81 to 92 (0.97 to 0.86, boxes differ);
// 2048x16384, whose dh does not fit beside dy and h and is read late, 123 (0.65).  Unaligned bf16 8192x4099 91 (0.44), binary32 4096x4099 67 (0.59).
// Rows of more than kMostCols columns are read three times, once for dw: bf16 2048x16512 90 (0.44).
#include "rms.cuh"

namespace fp8q {

namespace {

constexpr int kMostCols = 16384;   // of a row held in registers
// Bytes of a block's rows and of its stages (rms_plan): bf16 with dh, 8192x4096: 46.1 us, with twice as much 49.1; 65536x4096 308
// and 323.  Unaligned rows take 2.3 times the instructions, whose waits (issue slots 43 % busy, shared memory 54 %) more warps
// hide, as many as fit: 8192x4099 91 us, with 52 KB 168.
template <bool VECTOR>
constexpr int kMost = (VECTOR ? 56 : 96) * 1024;
constexpr int kInFlight = 104 * 1024;

// Few rows (no more than SMs; half as many if unaligned binary32), of any width: one launch for both results, which need only the
// rstd of the forward pass.  Block r < rows takes row r, in two passes; the blocks behind them sum dw over all rows, kFewCols columns
// each, warp w the rows w, w + kFewWarps, ...  Without the latter, dx of rows that registers cannot hold.  bf16 with dh, us, and by
// partial sums and a second launch: 1x4096 2.1 and 3.9, 16x12288 3.8 and 7.1, 64x4096 2.2 and 4.9, 152x8192 4.8 and 7.9; binary32
// 152x12288 9.8 and 10.8; unaligned binary32 64x5849 5.6 and 7.9, 128x5849 11.4 and 8.9.  Beyond as many rows as SMs a second round
// of blocks soon costs more than the second launch: of narrow rows 256x1024 are a little faster in one launch (4.0 and 4.6),
// 512x1024 are not (7.6 and 4.8).
constexpr int kFewThreads = 512, kFewWarps = kFewThreads / 32, kFewLane = 4, kFewCols = 32 * kFewLane;
__device__ __forceinline__ void load4(const float* m, float* v) {
  const float4 u = __ldg(reinterpret_cast<const float4*>(m));
  v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
}
__device__ __forceinline__ void load4(const uint16_t* m, float* v) {
  const uint2 u = __ldg(reinterpret_cast<const uint2*>(m));
  v[0] = __uint_as_float(u.x << 16), v[1] = __uint_as_float(u.x & 0xFFFF0000u);
  v[2] = __uint_as_float(u.y << 16), v[3] = __uint_as_float(u.y & 0xFFFF0000u);
}
// dw of the columns from c0 on over the rows [from, to); whether this thread has one of them, *col, and its sum.
template <typename T, bool VECTOR>
__device__ __forceinline__ bool sum_columns(const RmsBwdParams& p, int c0, int64_t from, int64_t to, float (&red)[kFewWarps][kFewCols],
                                            int* col, float* sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, cols = static_cast<int>(p.cols), c = c0 + kFewLane * lane;
  float dw[kFewLane] = {};
#pragma unroll 4
  for (int64_t row = from + warp; row < to; row += kFewWarps) {
    const T* const dy = static_cast<const T*>(p.dy) + row * p.lddy + c;
    const T* const h = static_cast<const T*>(p.h) + row * p.ldh + c;
    float a[kFewLane] = {}, b[kFewLane] = {};
    if (VECTOR) {   // cols is a multiple of kFewLane
      if (c < cols) {
        load4(dy, a);
        load4(h, b);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kFewLane; ++i)
        if (c + i < cols) a[i] = ld_elem(dy + i), b[i] = ld_elem(h + i);
    }
    const float rstd = p.rstd[row];
#pragma unroll
    for (int i = 0; i < kFewLane; ++i) dw[i] = fmaf(a[i], b[i] * rstd, dw[i]);
  }
#pragma unroll
  for (int i = 0; i < kFewLane; ++i) red[warp][i * 32 + lane] = dw[i];
  __syncthreads();
  *col = c0 + static_cast<int>(threadIdx.x);
  if (threadIdx.x >= kFewCols || *col >= cols) return false;
  *sum = 0.0f;
#pragma unroll
  for (int w = 0; w < kFewWarps; ++w) *sum += red[w][threadIdx.x % kFewLane * 32 + threadIdx.x / kFewLane];
  return true;
}

template <typename T, bool VECTOR>
__global__ void __launch_bounds__(kFewThreads) k_rms_backward_few(const RmsBwdParams p) {
  constexpr int E = VECTOR ? 16 / static_cast<int>(sizeof(T)) : 1;
  __shared__ float red[kFewWarps][kFewCols];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rows = static_cast<int>(p.rows), cols = static_cast<int>(p.cols);
  pdl_wait();
  pdl_launch_dependents();
  if (static_cast<int>(blockIdx.x) >= rows) {
    int c;
    float sum;
    if (sum_columns<T, VECTOR>(p, (static_cast<int>(blockIdx.x) - rows) * kFewCols, 0, rows, red, &c, &sum)) st_param(p.dw, p.w_f32, c, sum);
    return;
  }
  const int64_t row = blockIdx.x;
  const T* const dy = static_cast<const T*>(p.dy) + row * p.lddy;
  const T* const h = static_cast<const T*>(p.h) + row * p.ldh;
  const T* const dh = p.dh != nullptr ? static_cast<const T*>(p.dh) + row * p.lddh : nullptr;
  T* const dx = static_cast<T*>(p.dx) + row * p.lddx;
  const float rstd = p.rstd[row];
  // dy w and h of E elements at column c
  auto load = [&](int c, float (&g)[E], float (&x)[E]) {
    if constexpr (VECTOR) {
      float w[E];
      Piece<T, true>::unpack(__ldg(reinterpret_cast<const uint4*>(dy + c)), g);
      Piece<T, true>::unpack(__ldg(reinterpret_cast<const uint4*>(h + c)), x);
#pragma unroll
      for (int i = 0; i < E; i += 4) {
        if (p.w == nullptr) w[i] = w[i + 1] = w[i + 2] = w[i + 3] = 1.0f;
        else if (p.w_f32) load4(static_cast<const float*>(p.w) + c + i, w + i);
        else load4(static_cast<const uint16_t*>(p.w) + c + i, w + i);
      }
#pragma unroll
      for (int i = 0; i < E; ++i) g[i] *= w[i];
    } else {
      g[0] = ld_elem(dy + c) * (p.w != nullptr ? ld_param(p.w, p.w_f32, c) : 1.0f);
      x[0] = ld_elem(h + c);
    }
  };
  float sum = 0.0f;
#pragma unroll 4
  for (int c = static_cast<int>(threadIdx.x) * E; c < cols; c += kFewThreads * E) {
    float g[E], x[E];
    load(c, g, x);
#pragma unroll
    for (int i = 0; i < E; ++i) sum = fmaf(g[i], x[i] * rstd, sum);
  }
  sum = warp_sum(sum);
  if (lane == 0) red[0][warp] = sum;
  __syncthreads();
  sum = warp_sum(lane < kFewWarps ? red[0][lane] : 0.0f);
  const float k = -rstd * (sum / static_cast<float>(cols));
#pragma unroll 2
  for (int c = static_cast<int>(threadIdx.x) * E; c < cols; c += kFewThreads * E) {
    float g[E], x[E], a[E] = {};
    if (dh != nullptr) {
      if constexpr (VECTOR) Piece<T, true>::unpack(__ldg(reinterpret_cast<const uint4*>(dh + c)), a);
      else a[0] = ld_elem(dh + c);
    }
    load(c, g, x);
#pragma unroll
    for (int i = 0; i < E; ++i) a[i] = fmaf(x[i] * rstd, k, fmaf(g[i], rstd, a[i]));
    if constexpr (VECTOR) *reinterpret_cast<uint4*>(dx + c) = Piece<T, true>::pack(a);
    else st_elem(dx + c, a[0]);
  }
}

// Partial sums of dw, of rows that registers cannot hold: block (x, y) sums kFewCols columns over the rows of slab y.
template <typename T, bool VECTOR>
__global__ void __launch_bounds__(kFewThreads) k_rms_partial_any(const RmsBwdParams p) {
  __shared__ float red[kFewWarps][kFewCols];
  pdl_wait();
  pdl_launch_dependents();
  const int64_t slabs = gridDim.y, from = p.rows * blockIdx.y / slabs, to = p.rows * (blockIdx.y + 1) / slabs;
  int c;
  float sum;
  if (sum_columns<T, VECTOR>(p, static_cast<int>(blockIdx.x) * kFewCols, from, to, red, &c, &sum)) p.partial[blockIdx.y * p.cols + c] = sum;
}

// Rows of up to kMostCols columns, V values a lane.  A stage holds a warp's part of a row: dy, h, dh (`ahead`;
// otherwise dh is read when it is used) and the row's rstd.  The column sums and g take V of a thread's registers each; h and dh are read from
// shared memory when they are used.
template <typename T, bool VECTOR, int V, int BLOCK_WARPS>
__global__ void __launch_bounds__(BLOCK_WARPS * 32)
    k_rms_backward(const RmsBwdParams p, const int warps, const int stages, const int ring, const bool ahead) {
  using P = Piece<T, VECTOR>;
  constexpr int E = P::E, J = V / E, H = E / 2, kCols = 32 * V;
  using Part = RowPart<P, kCols, VECTOR, T>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float red[2][BLOCK_WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = warp / warps, w_in = warp - group * warps;
  const int n_groups = (blockDim.x >> 5) / warps, step = gridDim.x * n_groups;
  const int rows = static_cast<int>(p.rows), cols = static_cast<int>(p.cols);
  const bool add = p.dh != nullptr;
  const int scalar = Part::kBytes * (ahead ? 3 : 2), stage_bytes = scalar + 128;
  // this lane's first column and the columns from there to the row's end
  const int base = w_in * kCols, c = base + P::first(lane), left = cols - c;
  const float inv_n = 1.0f / static_cast<float>(cols);
  uint8_t* const mine = smem + ring + warp * stages * stage_bytes;
  float* const ws = reinterpret_cast<float*>(smem);

  auto issue = [&](int row, int s) {
    if (row < rows) {
      uint8_t* const to = mine + s * stage_bytes;
      const int64_t r = row;
      Part::start(to, static_cast<const T*>(p.dy) + r * p.lddy, r * p.lddy, base, cols, lane);
      Part::start(to + Part::kBytes, static_cast<const T*>(p.h) + r * p.ldh, r * p.ldh, base, cols, lane);
      if (ahead) Part::start(to + 2 * Part::kBytes, static_cast<const T*>(p.dh) + r * p.lddh, r * p.lddh, base, cols, lane);
      if (lane == 0) cp_async<4>(smem_u32(to) + scalar, p.rstd + row, true);
    }
    cp_async_commit();
  };
  // past the row's start, in elements of a granule
  auto past = [&](const void* m, int64_t ld, int row) {
    return Part::past(static_cast<const T*>(m) + static_cast<int64_t>(row) * ld + base);
  };

  pdl_wait();
  pdl_launch_dependents();
  float2 dw[J][H];
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int i = 0; i < H; ++i) dw[j][i] = both(0.0f);
  int row = blockIdx.x * n_groups + group;
  start_param<P, V>(p.w, p.w_f32, cols, warps, 1.0f, ws);
  cp_async_commit();
  for (int s = 0; s < stages; ++s) issue(row + s * step, s);
  cp_async_wait_oldest(stages + 1);
  settle_param<P, V>(p.w, p.w_f32, warps, ws);
  __syncthreads();
  for (int s = 0, buf = 0; row < rows; row += step, buf ^= 1) {
    cp_async_wait_oldest(stages);
    __syncwarp();   // the row's rstd, and unaligned a lane's last elements, were copied by other lanes
    const uint8_t* const at = mine + s * stage_bytes;
    const float rstd = *reinterpret_cast<const float*>(at + scalar);
    const int m_dy = past(p.dy, p.lddy, row), m_h = past(p.h, p.ldh, row);
    float2 g[J][H], acc = both(0.0f);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      float d[E], h[E], w[E];
      Part::read(at, m_dy, lane, j, d);
      Part::read(at + Part::kBytes, m_h, lane, j, h);
      read_param<P, V>(ws, w_in, j, lane, w);
#pragma unroll
      for (int i = 0; i < H; ++i) {
        const float2 dy = {d[2 * i], d[2 * i + 1]}, xh = mul2(make_float2(h[2 * i], h[2 * i + 1]), both(rstd));
        g[j][i] = mul2(dy, make_float2(w[2 * i], w[2 * i + 1]));
        dw[j][i] = fma2(dy, xh, dw[j][i]);
        acc = fma2(g[j][i], xh, acc);
      }
    }
    float sum = warp_sum(acc.x + acc.y);
    if (warps > 1) {
      if (lane == 0) red[buf][warp] = sum;
      group_sync(group, warps);
      // lane l joins warp l's part (the other buffer is written before this one is reused)
      sum = warp_sum(lane < warps ? red[buf][group * warps + lane] : 0.0f);
    }
    // dx = r g - (r c) xh + dh; r meets h first, since its square may leave binary32's range where r is in it (a row near 1e-20)
    const float2 r = both(rstd), k = both(-rstd * (sum * inv_n));
    const int m_dh = ahead ? past(p.dh, p.lddh, row) : 0;
    const T* const dh0 = static_cast<const T*>(p.dh) + static_cast<int64_t>(row) * p.lddh + c;
    T* const dx0 = static_cast<T*>(p.dx) + static_cast<int64_t>(row) * p.lddx + c;
    constexpr int N = VECTOR ? 1 : J;   // pieces stored together: unaligned, the fewer ends the better
#pragma unroll
    for (int j0 = 0; j0 < J; j0 += N) {
      uint4 packed[N];
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const int j = j0 + n;
        float h[E], a[E] = {};
        Part::read(at + Part::kBytes, m_h, lane, j, h);
        if (ahead) {
          Part::read(at + 2 * Part::kBytes, m_dh, lane, j, a);
        } else if (add) {
          float v[1][E];
          P::load(dh0 + j * P::WC, c + j * P::WC, left - j * P::WC, v);
#pragma unroll
          for (int i = 0; i < E; ++i) a[i] = v[0][i];
        }
#pragma unroll
        for (int i = 0; i < H; ++i) {
          const float2 xh = mul2(make_float2(h[2 * i], h[2 * i + 1]), r);
          const float2 o = fma2(xh, k, fma2(g[j][i], r, make_float2(a[2 * i], a[2 * i + 1])));
          a[2 * i] = o.x;
          a[2 * i + 1] = o.y;
        }
        packed[n] = P::pack(a);
      }
      P::store_raw(dx0 + j0 * P::WC, left - j0 * P::WC, packed);
    }
    __syncwarp();   // all lanes have read what this one copied
    issue(row + stages * step, s);
    s = s + 1 == stages ? 0 : s + 1;
  }
  if (p.dw == nullptr) return;
  // the block's groups joined pairwise in shared memory (the ring is free: every copy was waited for)
  __syncthreads();
  float2* join = reinterpret_cast<float2*>(smem + ring);
  for (int n = n_groups; n > 1;) {
    const int half = (n + 1) / 2;
    if (group >= half && group < n) {
      float2* out = join + ((group - half) * warps + w_in) * 16 * V + lane;
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < H; ++i) out[(j * H + i) * 32] = dw[j][i];
    }
    __syncthreads();
    if (group < n - half) {
      const float2* in = join + (group * warps + w_in) * 16 * V + lane;
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < H; ++i) dw[j][i] = add2(dw[j][i], in[(j * H + i) * 32]);
    }
    __syncthreads();
    n = half;
  }
  if (group != 0) return;
  float* const part = p.partial + static_cast<int64_t>(blockIdx.x) * cols;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    if (VECTOR) {   // cols is a multiple of 4, the workspace 16-byte aligned
      if (left <= j * P::WC) continue;
#pragma unroll
      for (int i = 0; i < H; i += 2)
        reinterpret_cast<float4*>(part + c + j * P::WC)[i / 2] = make_float4(dw[j][i].x, dw[j][i].y, dw[j][i + 1].x, dw[j][i + 1].y);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        if (!P::has(left - j * P::WC, i)) continue;
        part[c + j * P::WC + P::at(i)] = i % 2 ? dw[j][i / 2].y : dw[j][i / 2].x;
      }
    }
  }
}

// The cols sums of the n partial sums: a block takes 32 lanes' worth of them (N a lane), warp k the partials
// k, k + 32, ...; then the 32 warps' sums in order.
constexpr int kParamWarps = 32;
template <int N>
__global__ void __launch_bounds__(kParamWarps * 32) k_rms_params(const float* partial, int n, int cols, bool f32, void* dw) {
  __shared__ float part[kParamWarps][32 * N];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (static_cast<int64_t>(blockIdx.x) * 32 + lane) * N;
  pdl_wait();
  pdl_launch_dependents();
  float v[N] = {};
  if (c < cols) {
#pragma unroll 5
    for (int k = warp; k < n; k += kParamWarps) {
      const float* from = partial + static_cast<int64_t>(k) * cols + c;
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
  if (warp >= N || c >= cols) return;
  float sum = 0.0f;   // warp i of the first N: value i of every lane
#pragma unroll
  for (int k = 0; k < kParamWarps; ++k) sum += part[k][warp * 32 + lane];
  st_param(dw, f32, c + warp, sum);
}

// *partials: number of partial sums left in p.partial (0: the result stands)
template <typename T, bool VECTOR, int V, int BLOCK_WARPS>
cudaError_t run_rms_backward(const RmsBwdParams& p, int num_sms, cudaStream_t s, int* partials) {
  const int part = RowPart<Piece<T, VECTOR>, 32 * V, VECTOR, T>::kBytes;
  const int blocks = num_sms < kMaxNormPartials ? num_sms : kMaxNormPartials;
  bool ahead = p.dh != nullptr;
  NormPlan n = rms_plan(p.rows, p.cols, 32 * V, BLOCK_WARPS, part * (ahead ? 3 : 2) + 128, kMost<VECTOR>, kInFlight, 2, blocks);
  if (ahead && n.smem > kNormSmem) {   // binary32 rows of over 12288 columns: three parts of a row do not fit
    ahead = false;
    n = rms_plan(p.rows, p.cols, 32 * V, BLOCK_WARPS, part * 2 + 128, kMost<VECTOR>, kInFlight, 2, blocks);
  }
  const size_t join = n.ring + static_cast<size_t>(n.groups / 2) * n.warps * 32 * V * sizeof(float);
  if (n.smem < join) n.smem = join;
  static std::atomic<bool> done[kMaxDevices];
  auto kernel = k_rms_backward<T, VECTOR, V, BLOCK_WARPS>;
  const cudaError_t e = ensure_smem_limit(kernel, kNormSmem, done);
  if (e != cudaSuccess) return e;
  *partials = n.blocks;
  return launch_pdl(kernel, dim3(n.blocks), dim3(static_cast<unsigned>(n.warps * n.groups * 32)), n.smem, s, 1, p, n.warps,
                    n.stages, n.ring, ahead);
}

// Values a lane and warps of a block: as few as hold a narrow row; 16 values leave two warps for each of a row's 1024 columns
// (6000x5120 43.7 us, with 32 values 50.4; 8192x4096 46.1 and 46.3); 32 where 24 warps of 16 would hold one row and
// leave its registers short (2048x12288 33.3 us, 34.1) or not hold it.
template <typename T, bool VECTOR>
cudaError_t run_rms_backward(const RmsBwdParams& p, int num_sms, cudaStream_t s, int* partials) {
  if (p.cols <= 256) return run_rms_backward<T, VECTOR, 8, 24>(p, num_sms, s, partials);
  if (p.cols <= 8192) return run_rms_backward<T, VECTOR, 16, 24>(p, num_sms, s, partials);
  return run_rms_backward<T, VECTOR, 32, 16>(p, num_sms, s, partials);
}

template <typename T, bool VECTOR>
cudaError_t run_few(const RmsBwdParams& p, cudaStream_t s) {
  const int64_t blocks = p.rows + (p.dw != nullptr ? (p.cols + kFewCols - 1) / kFewCols : 0);
  return launch_pdl(k_rms_backward_few<T, VECTOR>, dim3(static_cast<unsigned>(blocks)), dim3(kFewThreads), 0, s, 1, p);
}

template <typename T, bool VECTOR>
cudaError_t run_any(const RmsBwdParams& p, int num_sms, cudaStream_t s, int* partials) {
  if (p.rows > 0) {
    RmsBwdParams q = p;
    q.dw = nullptr;
    const cudaError_t e = run_few<T, VECTOR>(q, s);
    if (e != cudaSuccess) return e;
  }
  if (p.dw == nullptr) return cudaSuccess;
  // as many slabs as keep the SMs busy
  const int64_t blocks = (p.cols + kFewCols - 1) / kFewCols, want = (3 * num_sms + blocks - 1) / blocks;
  *partials = static_cast<int>(want < norm_partials(p.rows) ? want : norm_partials(p.rows));
  return launch_pdl(k_rms_partial_any<T, VECTOR>, dim3(static_cast<unsigned>(blocks), *partials), dim3(kFewThreads), 0, s, 1, p);
}

template <typename T, bool VECTOR>
cudaError_t run(const RmsBwdParams& p, int num_sms, cudaStream_t s, int* partials) {
  const int few = sizeof(T) == 4 && !VECTOR ? num_sms / 2 : num_sms;
  if (p.rows > 0 && p.rows <= few) return run_few<T, VECTOR>(p, s);
  if (p.cols > kMostCols || p.rows == 0) return run_any<T, VECTOR>(p, num_sms, s, partials);
  return run_rms_backward<T, VECTOR>(p, num_sms, s, partials);
}

}  // namespace

cudaError_t launch_rms_backward(const RmsBwdParams& p, int num_sms, cudaStream_t s) {
  const int64_t size = p.f32 ? 4 : 2;
  int partials = 0;
  cudaError_t e;
  const bool vec = takes(p.dy, p.lddy, p.cols, size, 16) && takes(p.h, p.ldh, p.cols, size, 16) &&
                   takes(p.dh, p.lddh, p.cols, size, 16) && takes(p.dx, p.lddx, p.cols, size, 16) && takes(p.w, 0, 0, 1, 16);
  if (p.f32)
    e = vec ? run<float, true>(p, num_sms, s, &partials) : run<float, false>(p, num_sms, s, &partials);
  else
    e = vec ? run<uint16_t, true>(p, num_sms, s, &partials) : run<uint16_t, false>(p, num_sms, s, &partials);
  if (e != cudaSuccess || partials == 0 || p.dw == nullptr) return e;
  const int quad = p.cols % 4 == 0 ? 4 : 1;
  return launch_pdl(quad == 4 ? k_rms_params<4> : k_rms_params<1>, dim3(static_cast<unsigned>((p.cols / quad + 31) / 32)),
                    dim3(kParamWarps * 32), 0, s, 1, static_cast<const float*>(p.partial), partials, static_cast<int>(p.cols),
                    p.w_f32 != 0, p.dw);
}

}  // namespace fp8q
