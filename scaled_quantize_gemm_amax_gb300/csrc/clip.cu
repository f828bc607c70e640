// clip.cu -- the 2-norm over many tensors, and the tensors scaled so that it stays below a limit.
//
//   norm = sqrt(sum over all elements of g^2),  out = g min(1, max_norm / (norm + 1e-6))
// The tensors' addresses and sizes travel in the launch's parameters, a table of up to kTable
// tensors; a launch takes its tensors in pieces of kPiece elements, piece i by block i mod grid.
// Squares are summed in binary32 over a thread's part of a piece (64 elements) and a warp, and in
// binary64 from there on; a warp whose sum leaves binary32's range takes its part again in
// binary64, so that no value is too large or too small.  Sums are taken in an order that depends on
// the sizes and alignments alone.
//
// Bound by HBM: the gradients once in for the norm, once in and once out for the clipping.
#include <cfloat>

#include "internal.h"
#include "rowops.cuh"

namespace fp8q {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kPiece = 16384;          // elements of a piece
constexpr int kTable = 896;            // tensors of a launch: 28 bytes each in at most 32764 bytes of parameters
constexpr int kMaxBlocks = 1216;       // partial sums of a launch (152 SMs, 8 blocks each)

struct Table {
  const void* in[kTable];
  void* out[kTable];
  int64_t n[kTable];       // elements, negative - 1 for binary32
  int first[kTable + 1];   // the tensors' first pieces
  int tensors;
};
static_assert(sizeof(Table) + 64 <= 32764, "kernel parameters");

// Tensor of piece i: the last whose first piece is not above it.
__device__ __forceinline__ int tensor_of(const Table& t, int i) {
  int lo = 0, hi = t.tensors;
  while (hi - lo > 1) {
    const int m = (lo + hi) / 2;
    if (t.first[m] <= i) lo = m;
    else hi = m;
  }
  return lo;
}

// The sum of a thread's squares of `len` elements at p, a block's threads sharing them: 16-byte accesses
// between the first and the last 16-byte boundary.  `f` sees the elements' values.
template <typename T, typename F>
__device__ __forceinline__ void each(const T* p, int len, F f) {
  constexpr int E = 16 / static_cast<int>(sizeof(T));
  using P = Piece<T, true>;
  const int head = min(len, static_cast<int>((16 - reinterpret_cast<uintptr_t>(p) % 16) % 16 / sizeof(T)));
  const int vecs = (len - head) / E, tail = head + vecs * E;
  const uint4* const v = reinterpret_cast<const uint4*>(p + head);
  constexpr int U = 4;   // loads in flight together
  for (int i = threadIdx.x; i < vecs; i += U * kThreads) {
    uint4 w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) w[u] = i + u * kThreads < vecs ? __ldg(v + i + u * kThreads) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float x[E];
      P::unpack(w[u], x);
#pragma unroll
      for (int k = 0; k < E; ++k) f(x[k]);
    }
  }
  if (static_cast<int>(threadIdx.x) < head) f(ld_elem(p + threadIdx.x));
  if (tail + static_cast<int>(threadIdx.x) < len) f(ld_elem(p + tail + threadIdx.x));
}

// Sum of squares of one piece over a warp's lanes, in binary64.
template <typename T>
__device__ __forceinline__ double squares(const T* p, int len) {
  float s = 0.0f;
  uint32_t any = 0;
  each(p, len, [&](float x) {
    s = fmaf(x, x, s);
    any |= __float_as_uint(x);
  });
  s = warp_sum(s);
  // below 2^-60 squares may have lost digits or vanished (a piece of zeros has not)
  const bool odd = !(s <= FLT_MAX) || (s < 0x1p-60f && __any_sync(0xFFFFFFFFu, (any & 0x7FFFFFFFu) != 0u));
  if (!odd) return s;
  double d = 0.0;
  each(p, len, [&](float x) { d = fma(static_cast<double>(x), static_cast<double>(x), d); });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xFFFFFFFFu, d, o);
  return d;
}

__global__ void __launch_bounds__(kThreads) k_squares(const __grid_constant__ Table t, double* partial) {
  __shared__ double part[kWarps];
  pdl_wait();
  pdl_launch_dependents();
  double sum = 0.0;
  const int pieces = t.first[t.tensors];
  for (int i = blockIdx.x; i < pieces; i += gridDim.x) {
    const int k = tensor_of(t, i);
    const int64_t from = static_cast<int64_t>(i - t.first[k]) * kPiece;
    const bool f32 = t.n[k] < 0;
    const int64_t left = (f32 ? -t.n[k] - 1 : t.n[k]) - from;
    const int len = static_cast<int>(left < kPiece ? left : kPiece);
    sum += f32 ? squares(static_cast<const float*>(t.in[k]) + from, len) : squares(static_cast<const uint16_t*>(t.in[k]) + from, len);
  }
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    double all = 0.0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) all += part[w];
    partial[blockIdx.x] = all;
  }
}

// the sum of n partial sums, in every thread of the block
__device__ __forceinline__ double join(const double* partial, int n) {
  __shared__ double part[kWarps];
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) s += partial[i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
  __syncthreads();
  s = 0.0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) s += part[w];
  return s;
}

__global__ void __launch_bounds__(kThreads) k_norm_of(const double* partial, int n, float* norm) {
  pdl_wait();
  pdl_launch_dependents();
  const double s = join(partial, n);
  if (threadIdx.x == 0) *norm = static_cast<float>(sqrt(s));
}

template <typename T>
__device__ __forceinline__ void scale_piece(const T* in, T* out, int len, float by) {
  constexpr int E = 16 / static_cast<int>(sizeof(T));
  using P = Piece<T, true>;
  int head = min(len, static_cast<int>((16 - reinterpret_cast<uintptr_t>(in) % 16) % 16 / sizeof(T)));
  // an output at another place of its 16 bytes is written element by element
  if ((reinterpret_cast<uintptr_t>(in) - reinterpret_cast<uintptr_t>(out)) % 16 != 0) head = len;
  const int vecs = (len - head) / E, tail = head + vecs * E;
  const uint4* const v = reinterpret_cast<const uint4*>(in + head);
  uint4* const o = reinterpret_cast<uint4*>(out + head);
  constexpr int U = 4;
  for (int i = threadIdx.x; i < vecs; i += U * kThreads) {
    uint4 w[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i + u * kThreads < vecs) w[u] = v[i + u * kThreads];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i + u * kThreads >= vecs) break;
      float x[E];
      P::unpack(w[u], x);
#pragma unroll
      for (int k = 0; k < E; ++k) x[k] = __fmul_rn(x[k], by);
      o[i + u * kThreads] = P::pack(x);
    }
  }
  for (int i = threadIdx.x; i < head; i += kThreads) st_elem(out + i, __fmul_rn(ld_elem(in + i), by));
  for (int i = tail + threadIdx.x; i < len; i += kThreads) st_elem(out + i, __fmul_rn(ld_elem(in + i), by));
}

__global__ void __launch_bounds__(kThreads) k_clip(const __grid_constant__ Table t, const double* partial, int n, float max_norm,
                                                   float* norm) {
  pdl_wait();
  pdl_launch_dependents();
  const float total = static_cast<float>(sqrt(join(partial, n)));
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = total;
  float by = __fdiv_rn(max_norm, total + 1e-6f);
  if (by > 1.0f) by = 1.0f;   // a NaN stays
  const int pieces = t.first[t.tensors];
  // from the last piece on: the norm's pass has left the last ones in L2
  for (int i = pieces - 1 - static_cast<int>(blockIdx.x); i >= 0; i -= gridDim.x) {
    const int k = tensor_of(t, i);
    if (by == 1.0f && t.in[k] == t.out[k]) continue;   // in place, nothing to scale
    const int64_t from = static_cast<int64_t>(i - t.first[k]) * kPiece;
    const bool f32 = t.n[k] < 0;
    const int64_t left = (f32 ? -t.n[k] - 1 : t.n[k]) - from;
    const int len = static_cast<int>(left < kPiece ? left : kPiece);
    if (f32)
      scale_piece(static_cast<const float*>(t.in[k]) + from, static_cast<float*>(t.out[k]) + from, len, by);
    else
      scale_piece(static_cast<const uint16_t*>(t.in[k]) + from, static_cast<uint16_t*>(t.out[k]) + from, len, by);
  }
}

int blocks_of(int64_t pieces, int num_sms) {
  int64_t most = static_cast<int64_t>(num_sms) * 8;
  if (most > kMaxBlocks) most = kMaxBlocks;
  return static_cast<int>(pieces < 1 ? 1 : (pieces < most ? pieces : most));
}

}  // namespace

int64_t clip_partials(int64_t n_tensors) { return ((n_tensors + kTable - 1) / kTable < 1 ? 1 : (n_tensors + kTable - 1) / kTable) * kMaxBlocks; }

cudaError_t launch_clip(const ClipTensor* tensors, int64_t n, bool clip, float max_norm, double* partial, float* norm, int num_sms,
                        cudaStream_t s) {
  Table t;
  int sums = 0;
  for (int pass = 0; pass < (clip ? 2 : 1); ++pass) {
    for (int64_t from = 0; from < n || from == 0; from += kTable) {
      t.tensors = static_cast<int>(n - from < kTable ? n - from : kTable);
      int64_t pieces = 0;
      for (int i = 0; i < t.tensors; ++i) {
        const ClipTensor& x = tensors[from + i];
        t.in[i] = x.in;
        t.out[i] = x.out;
        t.n[i] = x.f32 ? -x.n - 1 : x.n;
        t.first[i] = static_cast<int>(pieces);
        pieces += (x.n + kPiece - 1) / kPiece;
      }
      t.first[t.tensors] = static_cast<int>(pieces);
      const int blocks = blocks_of(pieces, num_sms);
      cudaError_t e;
      if (pass == 0) {
        e = launch_pdl(k_squares, dim3(blocks), dim3(kThreads), 0, s, 1, t, partial + sums);
        sums += blocks;
      } else {
        e = launch_pdl(k_clip, dim3(blocks), dim3(kThreads), 0, s, 1, t, static_cast<const double*>(partial), sums, max_norm, norm);
      }
      if (e != cudaSuccess) return e;
    }
  }
  if (clip) return cudaSuccess;
  return launch_pdl(k_norm_of, dim3(1), dim3(kThreads), 0, s, 1, static_cast<const double*>(partial), sums, norm);
}

}  // namespace fp8q
