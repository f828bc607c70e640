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
//
// The rows are bound by HBM: 8192 tokens, 2 choices of 8 experts, 4096 wide in bf16, dispatch 33 us
// and combine 32 (0.93 of what a copy reaches); 2047 tokens, 8 choices of 64, combine backward 61
// and dispatch backward 25 (0.86).  In binary32 the two pairs 136 and 164 us (0.89, 0.91); 4099 wide,
// unaligned bf16, 115 and 182 (0.53, 0.41).  Routing is bound by latency (6.2 us there, 3.2 for a token).
#include "internal.h"
#include "rowops.cuh"

namespace fp8q {

namespace {

// ------------------------------------------------------------------ route
constexpr int kRouteThreads = 1024;
constexpr int kRouteWarps = kRouteThreads / 32;
constexpr int kRouteBlocks = 16;  // most blocks of the one cluster that sorts (8 is the portable limit)

__device__ __forceinline__ int expert_of(const RouteParams& p, int64_t i) {
  const int64_t e = p.ids64 ? static_cast<const int64_t*>(p.experts)[i] : static_cast<const int32_t*>(p.experts)[i];
  return e >= 0 && e < p.n_experts ? static_cast<int>(e) : -1;
}
// The lanes whose expert is this lane's, from one vote a bit of the number (a match instruction
// takes a turn for every different value: 131072 choices of 64 experts 34 us).
__device__ __forceinline__ uint32_t same_expert(int e, int bits) {
  uint32_t m = __ballot_sync(0xFFFFFFFFu, e >= 0);
  for (int b = 0; b < bits; ++b) {
    const bool set = (e >> b & 1) != 0;
    const uint32_t v = __ballot_sync(0xFFFFFFFFu, set);
    m &= set ? v : ~v;
  }
  return m;
}
__device__ __forceinline__ int ld_cluster(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// One cluster.  Every warp counts the choices of its contiguous part by expert, the block adds its
// warps' counts up, reads the other blocks' from their shared memory, and every warp then places
// its part in order: a choice's row is its expert's first, then the choices of the expert in the
// blocks before, in the warps before, and in the warp so far.  A warp's counts are its own, so
// neither walk needs a barrier.  One launch, no workspace: bound by latency.  8192 tokens with 2
// choices of 8 experts 6.3 us and 131072 choices 24 us when the blocks counted and ranked 1024
// choices at a time between barriers.
// Shared memory: total[E], this block's counts; used[E], the row past the expert's last choice;
// next[kRouteWarps][E], the warps' counts, then the rows of their next choices.
__global__ void __launch_bounds__(kRouteThreads) k_route(const RouteParams p) {
  extern __shared__ int smem[];
  __shared__ int warp_total[kRouteWarps];
  const int E = p.n_experts, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int blocks = gridDim.x, rank = blockIdx.x;
  int *total_of = smem, *used = smem + E, *mine = smem + 2 * E + warp * E;
  const int64_t first = rank * p.per_block + warp * p.per_warp;   // this warp's part
  const int64_t i0 = min(first, min(p.n, (rank + 1) * p.per_block)), i1 = min(first + p.per_warp, min(p.n, (rank + 1) * p.per_block));
  const int warps = p.n == 0 ? 0 : static_cast<int>((p.per_block + p.per_warp - 1) / p.per_warp);   // that have a part
  if (warp < warps)
    for (int e = lane; e < E; e += 32) mine[e] = 0;
  __syncwarp();
  pdl_wait();
  pdl_launch_dependents();
  const int bits = 32 - __clz(E - 1);   // of an expert's number
  int next = i0 + lane < i1 ? expert_of(p, i0 + lane) : -1;   // fetched ahead
  for (int64_t base = i0; base < i1; base += 32) {
    const int e = next;
    next = base + 32 + lane < i1 ? expert_of(p, base + 32 + lane) : -1;
    const uint32_t same = same_expert(e, bits);
    if (e >= 0 && (same & ((1u << lane) - 1u)) == 0) mine[e] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  // the warps' counts as sums over the warps before
  int total = 0, before = 0;
  if (tid < E) {
#pragma unroll 8
    for (int w = 0; w < warps; ++w) {
      const int c = smem[2 * E + w * E + tid];
      smem[2 * E + w * E + tid] = total;
      total += c;
    }
  }
  // this expert's choices in all blocks, and in the blocks before this one
  if (blocks > 1) {
    if (tid < E) total_of[tid] = total;
    cluster_sync();
    if (tid < E) {
      const uint32_t at = smem_u32(total_of + tid);
      total = 0;
      for (int b = 0; b < blocks; ++b) {
        const int c = ld_cluster(mapa_shared(at, b));
        total += c;
        before += b < rank ? c : 0;
      }
    }
    cluster_sync();   // no block leaves while another still reads its counts
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
  int off = incl - padded, rows = 0;
  for (int w = 0; w < kRouteWarps; ++w) {
    off += w < warp ? warp_total[w] : 0;
    rows += warp_total[w];
  }
  if (tid < E) {
    used[tid] = off + total;
#pragma unroll 8
    for (int w = 0; w < warps; ++w) smem[2 * E + w * E + tid] += off + before;
    if (rank == 0) {
      p.offsets[tid] = off;
      if (tid == E - 1) p.offsets[E] = rows;
    }
  }
  __syncthreads();
  next = i0 + lane < i1 ? expert_of(p, i0 + lane) : -1;
  for (int64_t base = i0; base < i1; base += 32) {
    const int64_t i = base + lane;
    const int e = next;
    next = i + 32 < i1 ? expert_of(p, i + 32) : -1;
    const uint32_t same = same_expert(e, bits);
    const int in_warp = __popc(same & ((1u << lane) - 1u));
    const int row = e >= 0 ? mine[e] + in_warp : -1;
    __syncwarp();
    if (e >= 0 && in_warp == 0) mine[e] += __popc(same);
    __syncwarp();
    if (i < i1) {
      p.pos[i] = row;
      if (row >= 0) p.src[row] = static_cast<int>(i);
    }
  }
  // rows that pad a segment, a warp an expert; then the rows past the last segment
  if (p.align > 1) {
    for (int e = rank * kRouteWarps + warp; e < E; e += blocks * kRouteWarps) {
      const int r0 = used[e], r1 = (r0 + p.align - 1) / p.align * p.align;   // segments start at multiples of align
      for (int r = r0 + lane; r < r1; r += 32) p.src[r] = -1;
    }
  }
  for (int64_t r = rows + static_cast<int64_t>(rank) * kRouteThreads + tid; r < p.capacity;
       r += static_cast<int64_t>(blocks) * kRouteThreads)
    p.src[r] = -1;
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

constexpr int kPieces = 2;   // pieces of a row a warp has in flight, of each of FLIGHT choices

// The choices j0 .. j0 + 31 of token t, one a lane: their rows and weights (-1 and 0 for those
// dropped, whose weights count for nothing).
struct Choices {
  int pos = -1;
  float w = 0.0f;
  __device__ Choices() {}
  __device__ Choices(const int* p_pos, const float* weights, int64_t t, int64_t tokens, int k, int j0, int lane) {
    if (t < tokens && j0 + lane < k) {
      const int64_t at = t * k + j0 + lane;
      pos = __ldg(p_pos + at);
      w = weights != nullptr ? __ldg(weights + at) : 1.0f;
    }
  }
  __device__ void check(int64_t capacity, uint32_t* err) {
    if (!valid_row(pos, capacity, err)) {
      pos = -1;
      w = 0.0f;
    }
  }
};

// `warps` warps per token (a block has one or more tokens at a time), each holding its pieces of
// the token's row: rows out[pos_j] = w_j in[t], and the dots <in[t], other[pos_j]>.  The token's
// row is read once for all its choices, and the next token's choices are fetched while this
// one's rows move.  After the tokens, a warp per `zero_rows` rows of `out` sets those that no
// choice fills to zero.
constexpr int kMostWarps = 11;   // of a token's row
constexpr int kZeroRows = 4;
template <typename T, bool VECTOR, bool DOTS, int FLIGHT>
__global__ void __maxnreg__(VECTOR ? (!DOTS ? 48 : FLIGHT > 2 ? 80 : 64) : (!DOTS ? 72 : 128))
    k_scatter(const ScatterParams p, const int warps, const int zero_rows) {
  using P = Piece<T, VECTOR>;
  __shared__ float part[2][kWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = warp / warps, w_in = warp - group * warps;
  const int cols = static_cast<int>(p.cols), block_cols = warps * kPieces * P::WC;
  const int64_t per_item = static_cast<int64_t>(warps) * zero_rows, items = p.tokens + (p.capacity + per_item - 1) / per_item;
  const int groups = static_cast<int>(blockDim.x >> 5) / warps;
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  int buf = 0;
  pdl_wait();
  pdl_launch_dependents();
  int64_t t = static_cast<int64_t>(blockIdx.x) * groups + group;
  Choices next(p.pos, p.weights, t, p.tokens, p.k, 0, lane);
  for (; t < items; t += step) {
    if (t >= p.tokens) {
      const int64_t r0 = ((t - p.tokens) * warps + w_in) * zero_rows, r = r0 + lane;
      uint32_t empty = __ballot_sync(0xFFFFFFFFu, lane < zero_rows && r < p.capacity && __ldg(p.src + r) < 0);
      const uint4 zero[1] = {make_uint4(0u, 0u, 0u, 0u)};
      for (; empty != 0; empty &= empty - 1) {
        T* out = static_cast<T*>(p.out) + (r0 + __ffs(empty) - 1) * p.ldout;
        for (int c0 = 0, c = P::first(lane); c0 < cols; c0 += P::WC, c += P::WC) P::store_raw(out + c, cols - c, zero);
      }
      continue;
    }
    const T* in = static_cast<const T*>(p.in) + t * p.ldin;
    Choices c = next;
    next = Choices(p.pos, p.weights, t + step, p.tokens, p.k, 0, lane);
    for (int j0 = 0; j0 < p.k; j0 += 32) {
      if (j0 > 0) c = Choices(p.pos, p.weights, t, p.tokens, p.k, j0, lane);
      c.check(p.capacity, p.err);
      const int n = min(32, p.k - j0);
      float my_dot = 0.0f;   // of choice j0 + lane
      for (int cb = w_in * kPieces * P::WC; cb < cols; cb += block_cols) {
        const int first = cb + P::first(lane), left = cols - first;
        typename P::template Run<kPieces> raw;
        P::load_raw(in + first, first, left, raw);
        if (!DOTS) P::settle(raw);
        for (int j = 0; j < n; j += FLIGHT) {
          typename P::template Run<kPieces> o[DOTS ? FLIGHT : 1];
          if constexpr (DOTS) {
#pragma unroll
            for (int u = 0; u < FLIGHT; ++u) {
              const int pos = __shfl_sync(0xFFFFFFFFu, c.pos, (j + u) & 31);
              const bool on = j + u < n && pos >= 0;
              const T* other = static_cast<const T*>(p.other) + (on ? pos : 0) * p.ldother + first;
              P::clear(o[u]);
              if (on) P::load_raw(other, first, left, o[u]);
            }
            if (j == 0) P::settle(raw);
          }
#pragma unroll
          for (int u = 0; u < FLIGHT; ++u) {
            if (j + u >= n) break;
            const int pos = __shfl_sync(0xFFFFFFFFu, c.pos, j + u);
            const float w = __shfl_sync(0xFFFFFFFFu, c.w, j + u);
            if (pos < 0) continue;
            T* out = static_cast<T*>(p.out) + pos * p.ldout + first;
            float2 dot = {0.0f, 0.0f};
            if constexpr (DOTS) P::settle(o[u]);
            uint4 moved[kPieces];
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
              float v[P::E], y[P::E];
              P::unpack(raw.r[i], v);
#pragma unroll
              for (int e = 0; e < P::E; e += 2) {
                const float2 m = mul2(both(w), make_float2(v[e], v[e + 1]));
                y[e] = m.x;
                y[e + 1] = m.y;
              }
              moved[i] = P::pack(y);
              if constexpr (DOTS) {
                P::unpack(o[u].r[i], y);
#pragma unroll
                for (int e = 0; e < P::E; e += 2) dot = fma2(make_float2(v[e], v[e + 1]), make_float2(y[e], y[e + 1]), dot);
              }
            }
            P::store_raw(out, left, moved);
            if constexpr (DOTS) {
              const float d = warp_sum(dot.x + dot.y);
              if (lane == j + u) my_dot += d;
            }
          }
        }
      }
      if constexpr (DOTS) {
        // the warps' parts in order (the buffer after next is written past another barrier)
        if (warps > 1) {
          part[buf][warp][lane] = my_dot;
          asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(warps * 32) : "memory");
          my_dot = 0.0f;
          for (int i = 0; i < warps; ++i) my_dot += part[buf][group * warps + i][lane];
          buf ^= 1;
        }
        if (w_in == 0 && lane < n) p.dots[t * p.k + j0 + lane] = my_dot;
      }
    }
  }
}

// A warp per kPieces pieces of a token's row: y[t] = sum_j w_j ys[pos_j], the choices in order.
template <typename T, bool VECTOR, int FLIGHT>
__global__ void __launch_bounds__(kThreads, VECTOR ? (FLIGHT > 2 ? 3 : 4) : 2) k_combine(const CombineParams p) {
  using P = Piece<T, VECTOR>;
  const int lane = threadIdx.x & 31, cols = static_cast<int>(p.cols);
  Walk at(static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5), static_cast<int64_t>(gridDim.x) * kWarps,
          (cols + kPieces * P::WC - 1) / (kPieces * P::WC));
  pdl_wait();
  pdl_launch_dependents();
  Choices next(p.pos, p.weights, at.row, p.tokens, p.k, 0, lane);
  while (at.row < p.tokens) {
    const int64_t t = at.row;
    const int first = static_cast<int>(at.piece) * kPieces * P::WC + P::first(lane), left = cols - first;
    Choices c = next;
    at.next();
    next = Choices(p.pos, p.weights, at.row, p.tokens, p.k, 0, lane);
    float acc[kPieces][P::E];
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
#pragma unroll
      for (int e = 0; e < P::E; ++e) acc[i][e] = 0.0f;
    for (int j0 = 0; j0 < p.k; j0 += 32) {
      if (j0 > 0) c = Choices(p.pos, p.weights, t, p.tokens, p.k, j0, lane);
      c.check(p.capacity, p.err);
      const int n = min(32, p.k - j0);
      for (int j = 0; j < n; j += FLIGHT) {
        typename P::template Run<kPieces> raw[FLIGHT];
        float w[FLIGHT];
#pragma unroll
        for (int u = 0; u < FLIGHT; ++u) {
          const int pos = __shfl_sync(0xFFFFFFFFu, c.pos, (j + u) & 31);
          w[u] = __shfl_sync(0xFFFFFFFFu, c.w, (j + u) & 31);
          const bool on = j + u < n && pos >= 0;
          const T* ys = static_cast<const T*>(p.ys) + (on ? pos : 0) * p.ldys + first;
          P::clear(raw[u]);
          if (on) P::load_raw(ys, first, left, raw[u]);
        }
#pragma unroll
        for (int u = 0; u < FLIGHT; ++u) {
          if (j + u >= n) break;
          P::settle(raw[u]);
#pragma unroll
          for (int i = 0; i < kPieces; ++i) {
            float v[P::E];
            P::unpack(raw[u].r[i], v);
#pragma unroll
            for (int e = 0; e < P::E; e += 2) {
              const float2 m = fma2(both(w[u]), make_float2(v[e], v[e + 1]), make_float2(acc[i][e], acc[i][e + 1]));
              acc[i][e] = m.x;
              acc[i][e + 1] = m.y;
            }
          }
        }
      }
    }
    T* y = static_cast<T*>(p.y) + t * p.ldy + first;
    P::store(y, left, acc);
  }
}

// Blocks of a launch over `want` blocks' worth of items: more than an SM holds, so that SMs that
// finish early take more, but each with several items, whose choices it fetches ahead.  8192
// tokens, 2 choices, 4096 wide (dispatch / combine / combine backward): 4 blocks an SM 39.5 / 34.2
// / 67.5 us, 8: 35.5 / 34.5 / 64.8, 16: 33.4 / 36.2 / 66.0, one block an item 42 / 41 / 73.
unsigned grid_of(int64_t want, int num_sms, int per_sm) {
  const int64_t cap = static_cast<int64_t>(num_sms) * per_sm;
  return static_cast<unsigned>(want < 1 ? 1 : (want > cap ? cap : want));
}

size_t route_smem(int experts) {
  return static_cast<size_t>(experts) * (2 + kRouteWarps) * sizeof(int);
}

}  // namespace

cudaError_t launch_route(RouteParams p, cudaStream_t s) {
  static std::atomic<bool> done[kMaxDevices];
  cudaError_t e = ensure_smem_limit(k_route, static_cast<int>(route_smem(kMaxExperts)), done);
  if (e != cudaSuccess) return e;
  int blocks = 1;
  while (blocks < kRouteBlocks && static_cast<int64_t>(blocks) * kRouteThreads < p.n) blocks *= 2;
  if (blocks > 8) {
    static std::atomic<bool> wide[kMaxDevices];
    e = ensure_wide_cluster(k_route, wide);
    if (e != cudaSuccess) return e;
  }
  // a warp's part: whole 32s, so that only the last is not
  p.per_warp = ((p.n + blocks - 1) / blocks + kRouteThreads - 1) / kRouteThreads * 32;
  p.per_block = (p.n + blocks - 1) / blocks;
  return launch_pdl(k_route, dim3(static_cast<unsigned>(blocks)), dim3(kRouteThreads), route_smem(p.n_experts), s, blocks, p);
}

namespace {

template <typename T, bool VECTOR>
cudaError_t run_scatter(const ScatterParams& p, int num_sms, cudaStream_t s) {
  // A warp for every kPieces pieces of a row, and blocks of as many tokens as 8 warps hold.  Past 8
  // warps' pieces the block grows a little before it goes round twice (dispatch, 4099 wide: 57 us with
  // 9 warps, 65 with 8; 12 warps, 6144 wide, are no gain and 16, 12288 wide, lose a quarter).  With
  // dots, whose warps wait for each other, a power of two up to 8 (both gradients, 2047 tokens, 8 of 64, 4099
  // wide: 9 warps 208 us, 8 180).
  const int64_t wc = Piece<T, VECTOR>::WC * kPieces, runs = (p.cols + wc - 1) / wc;
  int warps = 1;
  if (p.dots == nullptr && runs <= kMostWarps)
    warps = static_cast<int>(runs < 1 ? 1 : runs);
  else
    while (warps < kWarps && warps < runs) warps *= 2;
  const int groups = warps < kWarps ? kWarps / warps : 1;
  // rows a warp looks through for those to set to zero: few enough that every SM has some
  int64_t zero_rows = p.capacity / (static_cast<int64_t>(num_sms) * kWarps);
  zero_rows = zero_rows < 1 ? 1 : zero_rows > kZeroRows ? kZeroRows : zero_rows;
  const int64_t per_item = warps * zero_rows, items = p.tokens + (p.capacity + per_item - 1) / per_item;
  const bool few = p.k <= 2;
  const dim3 grid(grid_of((items + groups - 1) / groups, num_sms, p.dots == nullptr ? 16 : 8));
  auto kernel = p.dots == nullptr ? k_scatter<T, VECTOR, false, 2> : few ? k_scatter<T, VECTOR, true, 2> : k_scatter<T, VECTOR, true, 4>;
  return launch_pdl(kernel, grid, dim3(static_cast<unsigned>(warps * groups * 32)), 0, s, 1, p, warps, static_cast<int>(zero_rows));
}

template <typename T, bool VECTOR>
cudaError_t run_combine(const CombineParams& p, int num_sms, cudaStream_t s) {
  const int64_t wc = Piece<T, VECTOR>::WC * kPieces, items = p.tokens * ((p.cols + wc - 1) / wc);
  const bool few = p.k <= 2;
  return launch_pdl(few ? k_combine<T, VECTOR, 2> : k_combine<T, VECTOR, 4>,
                    dim3(grid_of((items + kWarps - 1) / kWarps, num_sms, 8)), dim3(kThreads), 0, s, 1, p);
}

}  // namespace

cudaError_t launch_scatter(const ScatterParams& p, int num_sms, cudaStream_t s) {
  const int64_t size = p.f32 ? 4 : 2;
  const bool vec = takes(p.in, p.ldin, p.cols, size, 16) && takes(p.out, p.ldout, p.cols, size, 16) &&
                   (p.dots == nullptr || takes(p.other, p.ldother, p.cols, size, 16));
  if (p.f32) return vec ? run_scatter<float, true>(p, num_sms, s) : run_scatter<float, false>(p, num_sms, s);
  return vec ? run_scatter<uint16_t, true>(p, num_sms, s) : run_scatter<uint16_t, false>(p, num_sms, s);
}

cudaError_t launch_combine(const CombineParams& p, int num_sms, cudaStream_t s) {
  const int64_t size = p.f32 ? 4 : 2;
  const bool vec = takes(p.ys, p.ldys, p.cols, size, 16) && takes(p.y, p.ldy, p.cols, size, 16);
  if (p.f32) return vec ? run_combine<float, true>(p, num_sms, s) : run_combine<float, false>(p, num_sms, s);
  return vec ? run_combine<uint16_t, true>(p, num_sms, s) : run_combine<uint16_t, false>(p, num_sms, s);
}

}  // namespace fp8q
