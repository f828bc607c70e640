// moe.cu -- token choices sorted by expert, rows copied to their experts' segments, expert
// outputs combined, and the gradients of both.
//
// Choice i = t k + j of token t goes to expert e_i; a choice outside [0, E) is dropped.
//   n_e = choices of expert e,  off_0 = 0,  off_{e+1} = off_e + align ceil(n_e / align)
//   pos_i = off_{e_i} + #{i' < i : e_i' = e_i}   (a stable counting sort),  -1 when dropped
//   src_r = the choice placed at row r, -1 for a row that pads a segment
//   dispatch          xs_r = x_{src_r / k},  0 for padding
//   combine           y_t = sum_j w_{t,j} ys_{pos_{t,j}}  over the choices not dropped, in order of j
//   combine backward  dys_r = w_{src_r} dy_{src_r / k},  dw_{t,j} = <dy_t, ys_{pos_{t,j}}>
//   dispatch backward = combine with w = 1
#include "internal.h"
#include "rowops.cuh"

namespace fp8q {

namespace {

// ------------------------------------------------------------------ route
constexpr int kRouteThreads = 1024;
constexpr int kRouteWarps = kRouteThreads / 32;
constexpr int kRouteBlocks = 128;       // most blocks of a route: each adds up all blocks' counts
constexpr int kRouteSingle = 4096;      // most choices that one block sorts alone

__device__ __forceinline__ int expert_of(const RouteParams& p, int64_t i) {
  const int64_t e = p.ids64 ? static_cast<const int64_t*>(p.experts)[i] : static_cast<const int32_t*>(p.experts)[i];
  return e >= 0 && e < p.n_experts ? static_cast<int>(e) : -1;
}

// counts[block][expert] of the block's choices
__global__ void __launch_bounds__(kRouteThreads) k_route_count(const RouteParams p) {
  extern __shared__ int hist[];
  pdl_wait();
  pdl_launch_dependents();
  for (int e = threadIdx.x; e < p.n_experts; e += kRouteThreads) hist[e] = 0;
  __syncthreads();
  const int64_t i1 = min(p.n, (blockIdx.x + 1) * p.per_block);
  for (int64_t i = blockIdx.x * p.per_block + threadIdx.x; i < i1; i += kRouteThreads) {
    const int e = expert_of(p, i);
    if (e >= 0) atomicAdd(hist + e, 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.n_experts; e += kRouteThreads)
    p.counts[static_cast<int64_t>(blockIdx.x) * p.n_experts + e] = hist[e];
}

// Shared memory: next[E], the row of the expert's next choice (first its count, when one block
// sorts alone), and of[kRouteWarps][E], the warps' counts within 1024 choices.
__global__ void __launch_bounds__(kRouteThreads) k_route_place(const RouteParams p) {
  extern __shared__ int smem[];
  __shared__ int warp_total[kRouteWarps];
  const int E = p.n_experts, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int* next = smem;
  uint16_t* of = reinterpret_cast<uint16_t*>(smem + E);
  pdl_wait();
  pdl_launch_dependents();
  const int64_t i0 = blockIdx.x * p.per_block, i1 = min(p.n, i0 + p.per_block);
  // this expert's choices in all blocks, and in the blocks before this one
  int total = 0, before = 0;
  if (p.counts == nullptr) {
    if (tid < E) next[tid] = 0;
    __syncthreads();
    for (int64_t i = i0 + tid; i < i1; i += kRouteThreads) {
      const int e = expert_of(p, i);
      if (e >= 0) atomicAdd(next + e, 1);
    }
    __syncthreads();
    if (tid < E) total = next[tid];
  } else if (tid < E) {
    for (int b = 0; b < static_cast<int>(gridDim.x); ++b) {
      const int c = p.counts[static_cast<int64_t>(b) * E + tid];
      total += c;
      before += b < static_cast<int>(blockIdx.x) ? c : 0;
    }
  }
  // exclusive scan of the padded totals over the experts
  const int padded = static_cast<int>((static_cast<int64_t>(total) + p.align - 1) / p.align * p.align);
  int incl = padded;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_total[warp] = incl;
  __syncthreads();
  int off = incl - padded;
  for (int w = 0; w < warp; ++w) off += warp_total[w];
  if (tid < E) {
    next[tid] = off + before;
    if (blockIdx.x == 0) {
      p.offsets[tid] = off;
      if (tid == E - 1) p.offsets[E] = off + padded;
    }
  }
  // rows that pad this expert's segment, shared out over the blocks by expert; then the rows
  // past the last segment
  if (tid < E && tid % gridDim.x == blockIdx.x) {
    for (int r = off + total; r < off + padded; ++r) p.src[r] = -1;
  }
  int rows = 0;
  for (int w = 0; w < kRouteWarps; ++w) rows += warp_total[w];
  for (int64_t r = rows + static_cast<int64_t>(blockIdx.x) * kRouteThreads + tid; r < p.capacity;
       r += static_cast<int64_t>(gridDim.x) * kRouteThreads)
    p.src[r] = -1;
  // 1024 choices at a time: a choice's rank is the choices of its expert in the warps before,
  // then in the lanes before
  for (int64_t base = i0; base < i1; base += kRouteThreads) {
    for (int i = tid; i < E * kRouteWarps / 2; i += kRouteThreads) reinterpret_cast<uint32_t*>(of)[i] = 0;
    __syncthreads();
    const int64_t i = base + tid;
    const int e = i < i1 ? expert_of(p, i) : -1;
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
    const int rank = __popc(same & ((1u << lane) - 1u));
    if (e >= 0 && rank == 0) of[warp * E + e] = static_cast<uint16_t>(__popc(same));
    __syncthreads();
    int sum = 0;
    if (tid < E) {
      for (int w = 0; w < kRouteWarps; ++w) {
        const int c = of[w * E + tid];
        of[w * E + tid] = static_cast<uint16_t>(sum);
        sum += c;
      }
    }
    __syncthreads();
    if (i < i1) {
      const int row = e >= 0 ? next[e] + of[warp * E + e] + rank : -1;
      p.pos[i] = row;
      if (row >= 0) p.src[row] = static_cast<int>(i);
    }
    __syncthreads();
    if (tid < E) next[tid] += sum;
  }
}

// ------------------------------------------------------------------ rows
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// A row index read from device memory: valid, dropped (-1), or out of range, which is reported.
__device__ __forceinline__ bool valid_row(int pos, int64_t capacity, uint32_t* err) {
  if (pos >= 0 && pos < capacity) return true;
  if (pos != -1) atomicOr(err, kErrBadState);
  return false;
}

// Block per token: rows out[pos_j] = w_j in[t] and the dots <in[t], other[pos_j]>; after the
// tokens, a warp per row of `out` that no choice fills, set to zero.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_scatter(const ScatterParams p) {
  __shared__ float red[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_launch_dependents();
  const int64_t items = p.tokens + (p.capacity + kWarps - 1) / kWarps;
  for (int64_t t = blockIdx.x; t < items; t += gridDim.x) {
    if (t >= p.tokens) {
      const int64_t r = (t - p.tokens) * kWarps + warp;
      if (r < p.capacity && p.src[r] < 0) {
        T* out = static_cast<T*>(p.out) + r * p.ldout;
        for (int64_t c = lane; c < p.cols; c += 32) st_elem(out + c, 0.0f);
      }
      continue;
    }
    const T* in = static_cast<const T*>(p.in) + t * p.ldin;
    for (int j = 0; j < p.k; ++j) {
      const int pos = p.pos[t * p.k + j];
      const bool kept = valid_row(pos, p.capacity, p.err);
      float dot = 0.0f;
      if (kept) {
        T* out = static_cast<T*>(p.out) + pos * p.ldout;
        const float w = p.weights != nullptr ? p.weights[t * p.k + j] : 1.0f;
        const T* other = p.dots != nullptr ? static_cast<const T*>(p.other) + pos * p.ldother : nullptr;
        for (int64_t c = threadIdx.x; c < p.cols; c += kThreads) {
          const float v = ld_elem(in + c);
          st_elem(out + c, w * v);
          if (other != nullptr) dot = fmaf(v, ld_elem(other + c), dot);
        }
      }
      if (p.dots != nullptr) {
        dot = warp_sum(dot);
        __syncthreads();
        if (lane == 0) red[warp] = dot;
        __syncthreads();
        if (threadIdx.x == 0) {
          float d = 0.0f;
          for (int w = 0; w < kWarps; ++w) d += red[w];
          p.dots[t * p.k + j] = d;
        }
      }
    }
  }
}

// Block per token: y[t] = sum_j w_j ys[pos_j], the choices in order.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_combine(const CombineParams p) {
  pdl_wait();
  pdl_launch_dependents();
  for (int64_t t = blockIdx.x; t < p.tokens; t += gridDim.x) {
    for (int64_t c = threadIdx.x; c < p.cols; c += kThreads) {
      float acc = 0.0f;
      for (int j = 0; j < p.k; ++j) {
        const int pos = p.pos[t * p.k + j];
        if (!valid_row(pos, p.capacity, p.err)) continue;
        const float v = ld_elem(static_cast<const T*>(p.ys) + pos * p.ldys + c);
        acc = p.weights != nullptr ? fmaf(p.weights[t * p.k + j], v, acc) : acc + v;
      }
      st_elem(static_cast<T*>(p.y) + t * p.ldy + c, acc);
    }
  }
}

unsigned grid_of(int64_t want, int num_sms, int per_sm) {
  const int64_t cap = static_cast<int64_t>(num_sms) * per_sm;
  return static_cast<unsigned>(want < 1 ? 1 : (want > cap ? cap : want));
}

size_t place_smem(int experts) {
  return static_cast<size_t>(experts) * (sizeof(int) + kRouteWarps * sizeof(uint16_t));
}

}  // namespace

int route_blocks(int64_t n) {
  if (n <= kRouteSingle) return 1;
  const int64_t b = (n + kRouteThreads - 1) / kRouteThreads;
  return static_cast<int>(b < kRouteBlocks ? b : kRouteBlocks);
}

cudaError_t launch_route(RouteParams p, cudaStream_t s) {
  static std::atomic<bool> done[kMaxDevices];
  cudaError_t e = ensure_smem_limit(k_route_place, static_cast<int>(place_smem(kMaxExperts)), done);
  if (e != cudaSuccess) return e;
  const unsigned blocks = static_cast<unsigned>(route_blocks(p.n));
  // whole multiples of 1024 choices a block
  p.per_block = ((p.n + blocks - 1) / blocks + kRouteThreads - 1) / kRouteThreads * kRouteThreads;
  if (blocks == 1) {
    p.counts = nullptr;
  } else {
    e = launch_pdl(k_route_count, dim3(blocks), dim3(kRouteThreads), p.n_experts * sizeof(int), s, 1, p);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(k_route_place, dim3(blocks), dim3(kRouteThreads), place_smem(p.n_experts), s, 1, p);
}

cudaError_t launch_scatter(const ScatterParams& p, int num_sms, cudaStream_t s) {
  const dim3 grid(grid_of(p.tokens + (p.capacity + kWarps - 1) / kWarps, num_sms, 8));
  return p.f32 ? launch_pdl(k_scatter<float>, grid, dim3(kThreads), 0, s, 1, p)
               : launch_pdl(k_scatter<uint16_t>, grid, dim3(kThreads), 0, s, 1, p);
}

cudaError_t launch_combine(const CombineParams& p, int num_sms, cudaStream_t s) {
  const dim3 grid(grid_of(p.tokens, num_sms, 8));
  return p.f32 ? launch_pdl(k_combine<float>, grid, dim3(kThreads), 0, s, 1, p)
               : launch_pdl(k_combine<uint16_t>, grid, dim3(kThreads), 0, s, 1, p);
}

}  // namespace fp8q
