// act.cu -- gated and plain activations, forward and backward.
//
//   y = f(a) b   (or f(a));   da = dy b f'(a),  db = dy f(a)
//   SiLU       f = x s,  f' = s (1 + x (1 - s)),  s = 1 / (1 + exp(-x))
//   GELU       f = x P,  f' = P + x exp(-x^2 / 2) / sqrt(2 pi),  P = (1 + erf(x / sqrt 2)) / 2
//   GELU tanh  f = x s,  f' = s + x s (1 - s) u',  u = 2 sqrt(2 / pi) (x + 0.044715 x^3),
//              s = 1 / (1 + exp(-u))      ((1 + tanh(u / 2)) / 2 = s)
// The inputs may be kept as 8-bit codes with one multiplier per 128 columns of a row; the
// backward pass then differentiates at the values the codes stand for.
//
// Bound by HBM: every element once in and once out, a warp two pieces of a row at a time, nothing
// shared between warps.  At 8192x11008 bf16, gated SiLU with codes 111.3 us (0.96 of what a copy
// reaches) and its gradient from the codes 105.5 (1.02); plain GELU's gradient at 8192x12288 88.3
// (1.01); 8192x9001, unaligned, forward 127 (0.69).  The arithmetic must not take the issue slots
// for that: one exponential and one reciprocal an element, divisions shared by lanes.
// Binary32 data have twice the bytes an element and take longer forms of f, right to the last places:
// 4096x8192 plain GELU 47.6 us (0.83), SiLU 43.1 (0.92), gated with codes 86.5 and 73.0 (0.81, 0.95), the
// gradients 57.5 to 96 (1.03).  With the shorter forms 40.5 to 72; with CUDA's normcdff, expf and an
// IEEE division GELU took 75, gated with codes 112.
#include "internal.h"
#include "rowops.cuh"

namespace fp8q {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kLog2e = 1.44269504f;

// s = e / (1 + e), e = exp(u) with u = x (SiLU) or GELU tanh's argument.  e is the square of its
// root, so that no subnormal passes through the approximate functions, which flush them; it is
// held to 2^60, where s is 1.  (1 / (1 + exp(-u)) is 2 instructions an element less, 109.3
// us instead of 111.3 above, and is 0 from u = -87 on.)
template <int ACT>
__device__ __forceinline__ float2 sigmoid2(float2 x, float2 x2) {
  float2 t;   // half the exponent
  if (ACT == kActSilu) {
    t = mul2(x, both(0.5f * kLog2e));   // off by 2 roundings, |x| 2^-23 of e: nothing in bf16
  } else {
    constexpr float kA = static_cast<float>(0.79788456080286536 * 1.44269504088896341);
    t = mul2(x, fma2(x2, both(0.044715f * kA), both(kA)));
  }
  const float2 h = make_float2(ex2(fminf(t.x, 30.0f)), ex2(fminf(t.y, 30.0f)));
  const float2 d = fma2(h, h, both(1.0f));
  return mul2(mul2(h, h), make_float2(rcp(d.x), rcp(d.y)));
}

// The normal distribution function P(x) = 1/2 + x R(x^2): R, smooth and even, by a polynomial of
// degree 14 in v = 2 x^2 / 5.25^2 - 1, fitted on |x| <= 5.25 (least squares on Chebyshev nodes,
// reweighted to an even error); beyond, R is held and P saturates to 0 and 1, off by at most
// 7.6e-8.  Error of P below 2^-23 in binary32.  No exponential and no branch: two values in
// 10 instructions each, where the library's erf took 25 and made GELU bound by issue slots.
__device__ __forceinline__ float2 normal_cdf2(float2 x, float2 x2) {
  constexpr float kR[15] = {0.13465935f,       -0.067126818f,    0.0496457852f,    -0.0397634134f,  0.0320314392f,
                            -0.0250419322f,    0.0185386483f,    -0.0127752507f,   0.00841787085f,  -0.00544851972f,
                            0.00289236126f,    -0.00103953469f,  0.000664732244f,  -0.000656583812f, 0.00023995011f};
  const float2 u = make_float2(fminf(x2.x, 27.5625f), fminf(x2.y, 27.5625f));
  const float2 v = fma2(u, both(2.0f / 27.5625f), both(-1.0f));
  float2 r = both(kR[14]);
#pragma unroll
  for (int i = 13; i >= 0; --i) r = fma2(r, v, both(kR[i]));
  return make_float2(__saturatef(fmaf(x.x, r.x, 0.5f)), __saturatef(fmaf(x.y, r.y, 0.5f)));
}

// ---- binary32 data: f and f' to a few units in the last place of the value itself, however small.
// (bf16 data take the shorter forms above: their error is absolute, below 2^-23 in P, so GELU loses
// bf16's own digits below x = -3.8, where P is under 1e-4.)

// exp(-(z + lo)) for 0 <= z <= 112, lo below half a unit in z's last place: the rounding of the
// base-2 exponent is made up for to first order.
__device__ __forceinline__ float2 exp_minus2(float2 z, float2 lo) {
  constexpr float kLo = static_cast<float>(1.44269504088896341 - static_cast<double>(kLog2e));
  const float2 a = mul2(z, both(kLog2e));
  float2 e = fma2(z, both(-kLog2e), a), r;
  e = fma2(z, both(-kLo), e);
  e = fma2(lo, both(-kLog2e), e);
  asm("ex2.approx.f32 %0, %1;" : "=f"(r.x) : "f"(-a.x));   // subnormal results kept
  asm("ex2.approx.f32 %0, %1;" : "=f"(r.y) : "f"(-a.y));
  return fma2(r, mul2(e, both(0.693147181f)), r);
}
__device__ __forceinline__ float2 where_not_negative(float2 x, float2 a, float2 b) {
  return make_float2(x.x >= 0.0f ? a.x : b.x, x.y >= 0.0f ? a.y : b.y);
}

// s and 1 - s at z from t = exp(-|z|), which neither overflows nor is subtracted from anything
__device__ __forceinline__ void exact_sigmoid2(float2 z, float2& s, float2& rest) {
  const float2 t = exp_minus2(make_float2(fminf(fabsf(z.x), 110.0f), fminf(fabsf(z.y), 110.0f)), both(0.0f));
  const float2 d = add2(t, both(1.0f)), inv = make_float2(rcp(d.x), rcp(d.y)), small = mul2(t, inv);
  s = where_not_negative(z, inv, small);
  rest = where_not_negative(z, small, inv);
}
__device__ __forceinline__ float2 gelu_tanh_arg2(float2 x, float2 x2) {
  return mul2(x, fma2(x2, both(static_cast<float>(2 * 0.79788456080286536 * 0.044715)), both(static_cast<float>(2 * 0.79788456080286536))));
}

// P and exp(-x^2 / 2).  With t = |x|, P(-t) = exp(-t^2 / 2) g(t), where g(t) (t + 3.5) varies by a
// third only: a polynomial of degree 9 in 1 / (t + 3.5), mapped to [-1, 1], fitted on t <= 14.5
// (least squares on Chebyshev nodes, reweighted to an even relative error, 2^-27); beyond, the
// exponential is 0.  P(t) = 1 - P(-t).
__device__ __forceinline__ void exact_normal_cdf2(float2 x, float2& cdf, float2& e) {
  constexpr float kG[10] = {0.867188275f,    0.565379858f,    0.250826538f,    0.0662314445f,   0.00398294767f,
                            -0.00327375275f, -0.000580223743f, 0.000220249422f, 4.04635721e-05f, -1.58110779e-05f};
  const float2 t = make_float2(fminf(fabsf(x.x), 15.0f), fminf(fabsf(x.y), 15.0f)), minus_half = mul2(t, both(-0.5f));
  const float2 square = mul2(t, minus_half), z = make_float2(-square.x, -square.y);   // z + lo = t^2 / 2
  const float2 lo = fma2(t, mul2(t, both(0.5f)), square);
  e = exp_minus2(z, lo);
  const float2 d = add2(t, both(3.5f)), minus_d = make_float2(-d.x, -d.y);
  float2 r = make_float2(rcp(d.x), rcp(d.y));
  r = fma2(r, fma2(minus_d, r, both(1.0f)), r);   // one Newton step: the polynomial's steep end multiplies r's error by 4
  // the offset one unit below its nearest value, which makes P(0) exactly 1/2
  const float2 u = fma2(r, both(static_cast<float>(2 / (1 / 3.5 - 1 / 18.0))), both(-1.48275876f));
  float2 g = both(kG[9]);
#pragma unroll
  for (int i = 8; i >= 0; --i) g = fma2(g, u, both(kG[i]));
  const float2 q = mul2(e, mul2(r, g));
  cdf = where_not_negative(x, fma2(q, both(-1.0f), both(1.0f)), q);
}

template <int ACT>
__device__ __forceinline__ void exact_act2(float2 x, float2& f, float2& df) {
  if (ACT == kActGelu) {
    float2 cdf, e;
    exact_normal_cdf2(x, cdf, e);
    f = mul2(x, cdf);
    df = fma2(mul2(x, both(0.39894228f)), e, cdf);
    return;
  }
  const float2 x2 = mul2(x, x);
  float2 s, rest;
  exact_sigmoid2(ACT == kActSilu ? x : gelu_tanh_arg2(x, x2), s, rest);
  f = mul2(x, s);
  rest = mul2(f, rest);
  if (ACT == kActGeluTanh) {   // u': x^2 is held below the overflow of its multiple, where 1 - s or f is 0 already
    const float2 c = make_float2(fminf(x2.x, 1e30f), fminf(x2.y, 1e30f));
    rest = mul2(rest, fma2(c, both(1.59576912f * 0.134145f), both(1.59576912f)));
  }
  df = add2(rest, s);
}

template <int ACT, bool EXACT>
__device__ __forceinline__ float2 act_value2(float2 x) {
  if (EXACT) {
    float2 f, unused;
    exact_act2<ACT>(x, f, unused);
    return f;
  }
  const float2 x2 = mul2(x, x);
  return mul2(x, ACT == kActGelu ? normal_cdf2(x, x2) : sigmoid2<ACT>(x, x2));
}

// f and f' at x
template <int ACT, bool EXACT>
__device__ __forceinline__ void act_grad2(float2 x, float2& f, float2& df) {
  if (EXACT) return exact_act2<ACT>(x, f, df);
  const float2 x2 = mul2(x, x);
  if (ACT == kActGelu) {
    const float2 cdf = normal_cdf2(x, x2), t = mul2(x2, both(-0.5f * kLog2e));
    f = mul2(x, cdf);
    df = fma2(mul2(x, both(0.39894228f)), make_float2(ex2(t.x), ex2(t.y)), cdf);
    return;
  }
  const float2 s = sigmoid2<ACT>(x, x2);
  f = mul2(x, s);
  float2 g = mul2(f, fma2(s, both(-1.0f), both(1.0f)));   // x s (1 - s)
  if (ACT == kActGeluTanh) {
    // u': x^2 is held below the overflow of its multiple, where g is 0 already
    const float2 c = make_float2(fminf(x2.x, 1e30f), fminf(x2.y, 1e30f));
    g = mul2(g, fma2(c, both(1.59576912f * 0.134145f), both(1.59576912f)));
  }
  df = add2(g, s);
}

// A warp takes kPieces pieces of a row at a time: enough loads in flight, and the 8-bit copies
// of all of them share the divisions.
constexpr int kPieces = 2;

template <typename T, bool VECTOR, int ACT, bool GATED>
__global__ void __launch_bounds__(kThreads, VECTOR ? 4 : 3) k_act(const ActParams p) {
  using P = Piece<T, VECTOR>;
  constexpr int E = P::E;
  const int lane = threadIdx.x & 31, cols = static_cast<int>(p.cols), groups = (cols + 127) / 128;
  Walk at(static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5), static_cast<int64_t>(gridDim.x) * kWarps,
          (cols + kPieces * P::WC - 1) / (kPieces * P::WC));
  pdl_wait();
  pdl_launch_dependents();
  for (; at.row < p.rows; at.next()) {
    const int64_t row = at.row;
    const int c = static_cast<int>(at.piece) * kPieces * P::WC + P::first(lane), left = cols - c;
    const T* pa = static_cast<const T*>(p.a) + row * p.lda + c;
    const T* pb = static_cast<const T*>(p.b) + row * p.ldb + c;
    T* py = static_cast<T*>(p.y) + row * p.ldy + c;
    typename P::template Run<kPieces> ra, rb;
    P::load_raw(pa, c, left, ra);
    if (GATED) P::load_raw(pb, c, left, rb);
    P::settle(ra);
    if (GATED) P::settle(rb);
    float a[kPieces][E], b[kPieces][E];
    uint4 y[kPieces];
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      P::unpack(ra.r[k], a[k]);
      if (GATED) P::unpack(rb.r[k], b[k]);
      float v[E];
#pragma unroll
      for (int i = 0; i < E; i += 2) {
        float2 f = act_value2<ACT, sizeof(T) == 4>(make_float2(a[k][i], a[k][i + 1]));
        if (GATED) f = mul2(f, make_float2(b[k][i], b[k][i + 1]));
        v[i] = f.x;
        v[i + 1] = f.y;
      }
      y[k] = P::pack(v);
    }
    P::store_raw(py, left, y);
    const int64_t q = row * p.ldq + c, s = row * groups + c / 128;
    if (p.qa != nullptr) store_copies<P, kPieces>(p.qa + q, p.sa + s, lane, left, p.e5m2, a);
    if (GATED && p.qb != nullptr) store_copies<P, kPieces>(p.qb + q, p.sb + s, lane, left, p.e5m2, b);
  }
}

template <typename T, bool VECTOR, int ACT, bool GATED, bool CODES>
__global__ void __launch_bounds__(kThreads, VECTOR ? 4 : 3) k_act_backward(const ActBwdParams p) {
  using P = Piece<T, VECTOR>;
  constexpr int E = P::E;
  const int lane = threadIdx.x & 31, cols = static_cast<int>(p.cols), groups = (cols + 127) / 128;
  Walk at(static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5), static_cast<int64_t>(gridDim.x) * kWarps,
          (cols + kPieces * P::WC - 1) / (kPieces * P::WC));
  pdl_wait();
  pdl_launch_dependents();
  for (; at.row < p.rows; at.next()) {
    const int64_t row = at.row;
    const int c = static_cast<int>(at.piece) * kPieces * P::WC + P::first(lane), left = cols - c;
    const int64_t q = row * p.ldq + c, s = row * groups + c / 128;
    typename P::template Run<kPieces> rdy, ra, rb;
    typename P::Codes ca[kPieces], cb[kPieces];
    float sa[kPieces], sb[kPieces];
    P::load_raw(static_cast<const T*>(p.dy) + row * p.lddy + c, c, left, rdy);
    if (CODES) {
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        const int off = k * P::WC, rest = left - off;
        ca[k] = P::load_codes(p.qa + q + off, c + off, rest);
        sa[k] = rest > 0 ? __ldg(p.sa + s + off / 128) : 0.0f;
        if (GATED) {
          cb[k] = P::load_codes(p.qb + q + off, c + off, rest);
          sb[k] = rest > 0 ? __ldg(p.sb + s + off / 128) : 0.0f;
        }
      }
    } else {
      P::load_raw(static_cast<const T*>(p.a) + row * p.lda + c, c, left, ra);
      if (GATED) P::load_raw(static_cast<const T*>(p.b) + row * p.ldb + c, c, left, rb);
      P::settle(ra);
      if (GATED) P::settle(rb);
    }
    P::settle(rdy);
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      float dy[E], a[E], b[E];
      P::unpack(rdy.r[k], dy);
      if (CODES) {
        P::decode(ca[k], sa[k], p.e5m2, a);
        if (GATED) P::decode(cb[k], sb[k], p.e5m2, b);
      } else {
        P::unpack(ra.r[k], a);
        if (GATED) P::unpack(rb.r[k], b);
      }
#pragma unroll
      for (int i = 0; i < E; i += 2) {
        const float2 d = make_float2(dy[i], dy[i + 1]);
        float2 f, df, da;
        act_grad2<ACT, sizeof(T) == 4>(make_float2(a[i], a[i + 1]), f, df);
        da = mul2(GATED ? mul2(d, make_float2(b[i], b[i + 1])) : d, df);
        a[i] = da.x;
        a[i + 1] = da.y;
        if (GATED) {
          f = mul2(d, f);
          b[i] = f.x;
          b[i + 1] = f.y;
        }
      }
      ra.r[k] = P::pack(a);
      if (GATED) rb.r[k] = P::pack(b);
    }
    P::store_raw(static_cast<T*>(p.da) + row * p.ldda + c, left, ra.r);
    if (GATED) P::store_raw(static_cast<T*>(p.db) + row * p.lddb + c, left, rb.r);
  }
}

// More blocks than the SMs hold at once (SMs that finish early take more), but not one an item:
// 8192x11008 gated SiLU forward / backward at 4 blocks an SM 112 / 122 us, 16: 112 / 109, 32:
// 111 / 106, one a group of 8 pieces 118 / 108.
dim3 grid_of(int64_t rows, int64_t cols, int64_t wc, int num_sms) {
  const int64_t want = (rows * ((cols + wc - 1) / wc) + kWarps - 1) / kWarps, cap = static_cast<int64_t>(num_sms) * 32;
  return dim3(static_cast<unsigned>(want < cap ? want : cap));
}

template <typename T, bool VECTOR, int ACT>
cudaError_t run_act(const ActParams& p, int num_sms, cudaStream_t s) {
  const dim3 grid = grid_of(p.rows, p.cols, kPieces * Piece<T, VECTOR>::WC, num_sms), block(kThreads);
  return p.b != nullptr ? launch_pdl(k_act<T, VECTOR, ACT, true>, grid, block, 0, s, 1, p)
                        : launch_pdl(k_act<T, VECTOR, ACT, false>, grid, block, 0, s, 1, p);
}

template <typename T, bool VECTOR, int ACT>
cudaError_t run_act_backward(const ActBwdParams& p, int num_sms, cudaStream_t s) {
  const dim3 grid = grid_of(p.rows, p.cols, kPieces * Piece<T, VECTOR>::WC, num_sms), block(kThreads);
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
