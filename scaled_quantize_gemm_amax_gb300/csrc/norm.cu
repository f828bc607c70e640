// norm.cu -- layer norm, forward and backward.
//
//   m = sum x / H,  v = sum (x - m)^2 / H,  r = 1 / sqrt(v + eps),  xh = (x - m) r
//   y = xh w + b
//   g = dy w,  c1 = sum g / H,  c2 = sum g xh / H,  dx = r (g - c1 - xh c2)
//   dw = sum over rows of dy xh,  db = sum over rows of dy
// The normalised rows xh may be kept as 8-bit codes with one multiplier per 128 columns; the
// backward pass then needs neither x nor m.  All sums are binary32.
#include "internal.h"
#include "rowops.cuh"

namespace fp8q {

namespace {

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

// One block per row, three passes over it (sum, squared differences, output).
template <typename T>
__global__ void __launch_bounds__(kThreads) k_norm_any(const NormParams p) {
  __shared__ float red[2 * kWarps];
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
    const float mean = block_sum(sum, 0.0f, red).x * inv_n;
    float sq = 0.0f;
    for (int64_t c = threadIdx.x; c < p.cols; c += kThreads) {
      const float d = ld_elem(x + c) - mean;
      sq = fmaf(d, d, sq);
    }
    const float var = block_sum(sq, 0.0f, red).x * inv_n;
    const float rstd = 1.0f / sqrtf(var + p.eps);
    if (threadIdx.x == 0) {
      if (p.mean != nullptr) p.mean[row] = mean;
      if (p.rstd != nullptr) p.rstd[row] = rstd;
    }
    for (int64_t g = warp; g < groups; g += kWarps) {
      float xh[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t c = Piece<T, false>::col(g * 128, lane, i);
        xh[i] = 0.0f;
        if (c < p.cols) {
          xh[i] = (ld_elem(x + c) - mean) * rstd;
          const float w = p.w != nullptr ? ld_param(p.w, p.w_f32, c) : 1.0f;
          const float b = p.b != nullptr ? ld_param(p.b, p.w_f32, c) : 0.0f;
          st_elem(y + c, fmaf(xh[i], w, b));
        }
      }
      if (p.q != nullptr)
        Piece<T, false>::store_codes(p.q + row * p.ldq, p.s + row * groups, g * 128, lane, p.cols, p.e5m2, xh);
    }
  }
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

// dx: one block per row, two passes.
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

// dw, db = the partial sums added in slab order
__global__ void __launch_bounds__(kThreads) k_norm_params(const float* partial, int slabs, int64_t cols, bool f32, void* dw,
                                                          void* db) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (c >= cols) return;
  float a = 0.0f, b = 0.0f;
  for (int k = 0; k < slabs; ++k) {
    a += partial[static_cast<int64_t>(k) * 2 * cols + c];
    b += partial[static_cast<int64_t>(k) * 2 * cols + cols + c];
  }
  if (dw != nullptr) st_param(dw, f32, c, a);
  if (db != nullptr) st_param(db, f32, c, b);
}

int grid_of(int64_t want, int num_sms, int per_sm) {
  const int64_t cap = static_cast<int64_t>(num_sms) * per_sm;
  return static_cast<int>(want < 1 ? 1 : (want > cap ? cap : want));
}

}  // namespace

int norm_partials(int64_t rows) {
  const int64_t n = (rows + 31) / 32;
  return static_cast<int>(n < 1 ? 1 : (n > kMaxNormPartials ? kMaxNormPartials : n));
}

cudaError_t launch_norm(const NormParams& p, int num_sms, cudaStream_t s) {
  const dim3 grid(grid_of(p.rows, num_sms, 8));
  return p.f32 ? launch_pdl(k_norm_any<float>, grid, dim3(kThreads), 0, s, 1, p)
               : launch_pdl(k_norm_any<uint16_t>, grid, dim3(kThreads), 0, s, 1, p);
}

cudaError_t launch_norm_backward(const NormBwdParams& p, int num_sms, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  if (p.rows > 0) {
    const dim3 grid(grid_of(p.rows, num_sms, 8));
    e = p.f32 ? launch_pdl(k_norm_dx_any<float>, grid, dim3(kThreads), 0, s, 1, p)
              : launch_pdl(k_norm_dx_any<uint16_t>, grid, dim3(kThreads), 0, s, 1, p);
    if (e != cudaSuccess) return e;
  }
  if (p.dw == nullptr && p.db == nullptr) return e;
  const int slabs = norm_partials(p.rows);
  const unsigned blocks = static_cast<unsigned>((p.cols + kThreads - 1) / kThreads);
  e = p.f32 ? launch_pdl(k_norm_partial_any<float>, dim3(blocks, slabs), dim3(kThreads), 0, s, 1, p, slabs)
            : launch_pdl(k_norm_partial_any<uint16_t>, dim3(blocks, slabs), dim3(kThreads), 0, s, 1, p, slabs);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_norm_params, dim3(blocks), dim3(kThreads), 0, s, 1, static_cast<const float*>(p.partial), slabs, p.cols,
                    p.w_f32 != 0, p.dw, p.db);
}

}  // namespace fp8q
