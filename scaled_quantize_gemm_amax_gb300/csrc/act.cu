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

// A warp per 128-column group.
template <typename T, int ACT>
__global__ void __launch_bounds__(kThreads) k_act(const ActParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t groups = (p.cols + 127) / 128, total = p.rows * groups;
  pdl_wait();
  pdl_launch_dependents();
  for (int64_t at = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); at < total;
       at += static_cast<int64_t>(gridDim.x) * kWarps) {
    const int64_t row = at / groups, g = at - row * groups;
    float a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t c = group_col(g, lane, i);
      a[i] = b[i] = 0.0f;
      if (c < p.cols) {
        a[i] = ld_elem(static_cast<const T*>(p.a) + row * p.lda + c);
        if (p.b != nullptr) b[i] = ld_elem(static_cast<const T*>(p.b) + row * p.ldb + c);
        const float f = act_value<ACT>(a[i]);
        st_elem(static_cast<T*>(p.y) + row * p.ldy + c, p.b != nullptr ? f * b[i] : f);
      }
    }
    if (p.qa != nullptr) store_group8(a, g, lane, p.cols, p.e5m2, p.qa + row * p.ldq, p.sa + row * groups);
    if (p.qb != nullptr) store_group8(b, g, lane, p.cols, p.e5m2, p.qb + row * p.ldq, p.sb + row * groups);
  }
}

template <typename T, int ACT>
__global__ void __launch_bounds__(kThreads) k_act_backward(const ActBwdParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t groups = (p.cols + 127) / 128, total = p.rows * groups;
  auto value = [&](const void* v, int64_t ld, const uint8_t* q, const float* s, int64_t row, int64_t c) {
    if (q == nullptr) return ld_elem(static_cast<const T*>(v) + row * ld + c);
    float x, unused;
    decode_pair(q[row * p.ldq + c], p.e5m2, x, unused);
    return x * s[row * groups + c / 128];
  };
  pdl_wait();
  pdl_launch_dependents();
  for (int64_t at = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); at < total;
       at += static_cast<int64_t>(gridDim.x) * kWarps) {
    const int64_t row = at / groups, g = at - row * groups;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t c = group_col(g, lane, i);
      if (c >= p.cols) continue;
      const float dy = ld_elem(static_cast<const T*>(p.dy) + row * p.lddy + c);
      const float2 f = act_grad<ACT>(value(p.a, p.lda, p.qa, p.sa, row, c));
      if (p.db == nullptr) {
        st_elem(static_cast<T*>(p.da) + row * p.ldda + c, dy * f.y);
      } else {
        st_elem(static_cast<T*>(p.da) + row * p.ldda + c, dy * value(p.b, p.ldb, p.qb, p.sb, row, c) * f.y);
        st_elem(static_cast<T*>(p.db) + row * p.lddb + c, dy * f.x);
      }
    }
  }
}

int grid_of(int64_t rows, int64_t cols, int num_sms) {
  const int64_t want = (rows * ((cols + 127) / 128) + kWarps - 1) / kWarps, cap = static_cast<int64_t>(num_sms) * 8;
  return static_cast<int>(want < 1 ? 1 : (want > cap ? cap : want));
}

}  // namespace

cudaError_t launch_act(const ActParams& p, int num_sms, cudaStream_t s) {
  const dim3 grid(grid_of(p.rows, p.cols, num_sms)), block(kThreads);
#define FP8Q_ACT(A) (p.f32 ? launch_pdl(k_act<float, A>, grid, block, 0, s, 1, p) : launch_pdl(k_act<uint16_t, A>, grid, block, 0, s, 1, p))
  return p.act == kActSilu ? FP8Q_ACT(kActSilu) : p.act == kActGelu ? FP8Q_ACT(kActGelu) : FP8Q_ACT(kActGeluTanh);
#undef FP8Q_ACT
}

cudaError_t launch_act_backward(const ActBwdParams& p, int num_sms, cudaStream_t s) {
  const dim3 grid(grid_of(p.rows, p.cols, num_sms)), block(kThreads);
#define FP8Q_ACT(A) \
  (p.f32 ? launch_pdl(k_act_backward<float, A>, grid, block, 0, s, 1, p) : launch_pdl(k_act_backward<uint16_t, A>, grid, block, 0, s, 1, p))
  return p.act == kActSilu ? FP8Q_ACT(kActSilu) : p.act == kActGelu ? FP8Q_ACT(kActGelu) : FP8Q_ACT(kActGeluTanh);
#undef FP8Q_ACT
}

}  // namespace fp8q
