// act.cu -- gated and plain activations, forward and backward.
//
//   y = f(a) b   (or f(a));   da = dy b f'(a),  db = dy f(a)
//   SiLU       f = x s,  f' = s (1 + x (1 - s)),  s = 1 / (1 + exp(-x))
//   GELU       f = x P,  f' = P + x exp(-x^2 / 2) / sqrt(2 pi),  P = (1 + erf(x / sqrt 2)) / 2
//   GELU tanh  f = x s,  f' = s + x s (1 - s) u',  u = 2 sqrt(2 / pi) (x + 0.044715 x^3),
//              s = 1 / (1 + exp(-u))      ((1 + tanh(u / 2)) / 2 = s)
// The inputs may be kept as 8-bit codes with one multiplier per 128 columns of a row; the
// backward pass then differentiates at the values the codes stand for.
#include "internal.h"
#include "rowops.cuh"

namespace fp8q {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

template <int ACT>
__device__ __forceinline__ float act_value(float x) {
  if (ACT == kActSilu) return x / (1.0f + expf(-x));
  if (ACT == kActGelu) return x * (0.5f + 0.5f * erff(x * 0.70710678f));
  const float u = 1.59576912f * fmaf(0.044715f * x * x, x, x);
  return x / (1.0f + expf(-u));
}

// f(x) in .x and f'(x) in .y
template <int ACT>
__device__ __forceinline__ float2 act_grad(float x) {
  if (ACT == kActGelu) {
    const float cdf = 0.5f + 0.5f * erff(x * 0.70710678f);
    return {x * cdf, fmaf(x, 0.39894228f * expf(-0.5f * x * x), cdf)};
  }
  // beyond +-128 s is 0 or 1 and the product with (1 - s) is 0: the clamp keeps it from being 0 * inf
  const float xc = fminf(fmaxf(x, -128.0f), 128.0f), x2 = xc * xc;
  const float u = ACT == kActSilu ? x : 1.59576912f * fmaf(0.044715f * x * x, x, x);
  const float du = ACT == kActSilu ? 1.0f : 1.59576912f * fmaf(0.134145f, x2, 1.0f);
  const float s = 1.0f / (1.0f + expf(-u));
  return {x * s, fmaf(xc * s * (1.0f - s), du, s)};
}

template <typename T, bool VECTOR, int ACT, bool GATED>
__global__ void __launch_bounds__(kThreads) k_act(const ActParams p) {
  using P = Piece<T, VECTOR>;
  const int lane = threadIdx.x & 31;
  const int64_t groups = (p.cols + 127) / 128;
  Walk at(static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5), static_cast<int64_t>(gridDim.x) * kWarps,
          (p.cols + P::WC - 1) / P::WC);
  pdl_wait();
  pdl_launch_dependents();
  for (; at.row < p.rows; at.next()) {
    const int64_t row = at.row;
    const int c0 = static_cast<int>(at.piece * P::WC), cols = static_cast<int>(p.cols);
    float a[P::E], b[P::E], y[P::E];
    P::load(static_cast<const T*>(p.a) + row * p.lda, c0, lane, cols, a);
    if (GATED) P::load(static_cast<const T*>(p.b) + row * p.ldb, c0, lane, cols, b);
#pragma unroll
    for (int i = 0; i < P::E; ++i) y[i] = GATED ? act_value<ACT>(a[i]) * b[i] : act_value<ACT>(a[i]);
    P::store(static_cast<T*>(p.y) + row * p.ldy, c0, lane, cols, y);
    if (p.qa != nullptr) P::store_codes(p.qa + row * p.ldq, p.sa + row * groups, c0, lane, cols, p.e5m2, a);
    if (GATED && p.qb != nullptr) P::store_codes(p.qb + row * p.ldq, p.sb + row * groups, c0, lane, cols, p.e5m2, b);
  }
}

template <typename T, bool VECTOR, int ACT, bool GATED, bool CODES>
__global__ void __launch_bounds__(kThreads) k_act_backward(const ActBwdParams p) {
  using P = Piece<T, VECTOR>;
  const int lane = threadIdx.x & 31;
  const int64_t groups = (p.cols + 127) / 128;
  Walk at(static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5), static_cast<int64_t>(gridDim.x) * kWarps,
          (p.cols + P::WC - 1) / P::WC);
  pdl_wait();
  pdl_launch_dependents();
  for (; at.row < p.rows; at.next()) {
    const int64_t row = at.row;
    const int c0 = static_cast<int>(at.piece * P::WC), cols = static_cast<int>(p.cols);
    float dy[P::E], a[P::E], b[P::E];
    P::load(static_cast<const T*>(p.dy) + row * p.lddy, c0, lane, cols, dy);
    if (CODES) {
      P::load_codes(p.qa + row * p.ldq, p.sa + row * groups, c0, lane, cols, p.e5m2, a);
      if (GATED) P::load_codes(p.qb + row * p.ldq, p.sb + row * groups, c0, lane, cols, p.e5m2, b);
    } else {
      P::load(static_cast<const T*>(p.a) + row * p.lda, c0, lane, cols, a);
      if (GATED) P::load(static_cast<const T*>(p.b) + row * p.ldb, c0, lane, cols, b);
    }
#pragma unroll
    for (int i = 0; i < P::E; ++i) {
      const float2 f = act_grad<ACT>(a[i]);
      a[i] = (GATED ? dy[i] * b[i] : dy[i]) * f.y;
      if (GATED) b[i] = dy[i] * f.x;
    }
    P::store(static_cast<T*>(p.da) + row * p.ldda, c0, lane, cols, a);
    if (GATED) P::store(static_cast<T*>(p.db) + row * p.lddb, c0, lane, cols, b);
  }
}

dim3 grid_of(int64_t rows, int64_t cols, int64_t wc, int num_sms) {
  const int64_t want = (rows * ((cols + wc - 1) / wc) + kWarps - 1) / kWarps, cap = static_cast<int64_t>(num_sms) * 8;
  return dim3(static_cast<unsigned>(want < cap ? want : cap));
}

template <typename T, bool VECTOR, int ACT>
cudaError_t run_act(const ActParams& p, int num_sms, cudaStream_t s) {
  const dim3 grid = grid_of(p.rows, p.cols, Piece<T, VECTOR>::WC, num_sms), block(kThreads);
  return p.b != nullptr ? launch_pdl(k_act<T, VECTOR, ACT, true>, grid, block, 0, s, 1, p)
                        : launch_pdl(k_act<T, VECTOR, ACT, false>, grid, block, 0, s, 1, p);
}

template <typename T, bool VECTOR, int ACT>
cudaError_t run_act_backward(const ActBwdParams& p, int num_sms, cudaStream_t s) {
  const dim3 grid = grid_of(p.rows, p.cols, Piece<T, VECTOR>::WC, num_sms), block(kThreads);
  if (p.qa != nullptr)
    return p.db != nullptr ? launch_pdl(k_act_backward<T, VECTOR, ACT, true, true>, grid, block, 0, s, 1, p)
                           : launch_pdl(k_act_backward<T, VECTOR, ACT, false, true>, grid, block, 0, s, 1, p);
  return p.db != nullptr ? launch_pdl(k_act_backward<T, VECTOR, ACT, true, false>, grid, block, 0, s, 1, p)
                         : launch_pdl(k_act_backward<T, VECTOR, ACT, false, false>, grid, block, 0, s, 1, p);
}

template <typename T, bool VECTOR>
cudaError_t of_kind(const ActParams& p, int n, cudaStream_t s) {
  return p.act == kActSilu ? run_act<T, VECTOR, kActSilu>(p, n, s)
         : p.act == kActGelu ? run_act<T, VECTOR, kActGelu>(p, n, s) : run_act<T, VECTOR, kActGeluTanh>(p, n, s);
}
template <typename T, bool VECTOR>
cudaError_t of_kind(const ActBwdParams& p, int n, cudaStream_t s) {
  return p.act == kActSilu ? run_act_backward<T, VECTOR, kActSilu>(p, n, s)
         : p.act == kActGelu ? run_act_backward<T, VECTOR, kActGelu>(p, n, s) : run_act_backward<T, VECTOR, kActGeluTanh>(p, n, s);
}

}  // namespace

cudaError_t launch_act(const ActParams& p, int num_sms, cudaStream_t s) {
  const int64_t size = p.f32 ? 4 : 2, e = 16 / size;
  const bool vec = takes(p.a, p.lda, p.cols, size, 16) && takes(p.b, p.ldb, p.cols, size, 16) &&
                   takes(p.y, p.ldy, p.cols, size, 16) && takes(p.qa, p.ldq, p.cols, 1, e) && takes(p.qb, p.ldq, p.cols, 1, e);
  if (p.f32) return vec ? of_kind<float, true>(p, num_sms, s) : of_kind<float, false>(p, num_sms, s);
  return vec ? of_kind<uint16_t, true>(p, num_sms, s) : of_kind<uint16_t, false>(p, num_sms, s);
}

cudaError_t launch_act_backward(const ActBwdParams& p, int num_sms, cudaStream_t s) {
  const int64_t size = p.f32 ? 4 : 2, e = 16 / size;
  const bool vec = takes(p.dy, p.lddy, p.cols, size, 16) && takes(p.a, p.lda, p.cols, size, 16) &&
                   takes(p.b, p.ldb, p.cols, size, 16) && takes(p.da, p.ldda, p.cols, size, 16) &&
                   takes(p.db, p.lddb, p.cols, size, 16) && takes(p.qa, p.ldq, p.cols, 1, e) &&
                   takes(p.qb, p.ldq, p.cols, 1, e);
  if (p.f32) return vec ? of_kind<float, true>(p, num_sms, s) : of_kind<float, false>(p, num_sms, s);
  return vec ? of_kind<uint16_t, true>(p, num_sms, s) : of_kind<uint16_t, false>(p, num_sms, s);
}

}  // namespace fp8q
