// clip.cu -- the 2-norm over many tensors, and the tensors scaled so that it stays below a limit.
//
//   norm = sqrt(sum over all elements of g^2),  out = g min(1, max_norm / (norm + 1e-6))
// The tensors' addresses and sizes travel in the launch's parameters, a table of up to kMostTensors.
// The tensors, one behind the other, are cut into pieces of a few KB, and every block takes a run of
// consecutive ones, so of most tensors a whole stretch; the host says at which tensor a run starts.  The
// second pass takes a run from its end, of which the first has left the most in L2.
// Squares are summed in binary32 over the 16 or 32 elements that a thread has in registers and in binary64
// from there on; where binary32's range ends, those elements are taken again in binary64, so that no value
// is too large or too small.  Sums are taken in an order that depends on the sizes and alignments alone.
//
// Bound by HBM: the gradients once in for the norm, once in and once out for the clipping: 810 million bf16 734 us (three
// passes of 1.6 GB take 718 at a copy's rate), 39.5 million 36 us (the second read from L2: two passes take 23, four to five us
// of launches and first loads in each).  Outputs that lie at another place of their 16 bytes than their gradients are written element
// by element, bound by those accesses: 134 million bf16 475 us instead of 126, half as many binary32 283.
#include <cfloat>

#include "internal.h"
#include "rowops.cuh"

namespace fp8q {

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kPerSm = 2, kMaxBlocks = 152 * kPerSm;
constexpr int kPiece = 4096;           // bytes of a piece, doubled until there are fewer than 2^30
constexpr int kLoads = 4;              // 16-byte loads of a thread in flight together
constexpr int kMostTensors = 960;      // of a launch

struct Entry {
  const void* in;
  void* out;
  int64_t n;       // elements, negative - 1 for binary32
  int64_t first;   // the tensor's first piece
};
// The parameters of a launch for up to N tensors; copying the largest costs the host 2 us a launch.
template <int N>
struct Table {
  uint16_t starts[kMaxBlocks];      // the tensors of the blocks' first pieces
  int pieces, shift;                // pieces are kPiece << shift bytes
  Entry of[N + 1];                  // the last: where the pieces end
};
static_assert(sizeof(Table<kMostTensors>) + 64 <= 32764, "kernel parameters");

// A block's run of pieces [lo, hi), and its stretch of one tensor.
struct Run {
  int lo, hi;
  template <int N>
  __device__ explicit Run(const Table<N>& t) {
    const int64_t n = t.pieces;
    lo = static_cast<int>(n * blockIdx.x / gridDim.x);
    hi = static_cast<int>(n * (blockIdx.x + 1) / gridDim.x);
  }
};
// A stretch of a tensor: elements, 16-byte vectors between its first and its last 16-byte boundary, and what lies
// in front of and behind them.
struct Stretch {
  const uint8_t* in;
  uint8_t* out;
  int64_t n;
  int head, vecs, size;   // elements in front, vectors, bytes of an element
  // e: the tensor; end: the first piece behind it
  __device__ Stretch(const Entry& e, int64_t end, const Run& r, int shift) {
    const int64_t all = e.n < 0 ? -e.n - 1 : e.n;
    size = e.n < 0 ? 4 : 2;
    const int64_t piece = static_cast<int64_t>(kPiece / size) << shift;   // in elements
    const int64_t from = (r.lo > e.first ? r.lo - e.first : 0) * piece, to = r.hi < end ? (r.hi - e.first) * piece : all;
    n = to - from;
    in = static_cast<const uint8_t*>(e.in) + from * size;
    out = static_cast<uint8_t*>(e.out) + from * size;
    const int front = static_cast<int>((16 - reinterpret_cast<uintptr_t>(in) % 16) % 16) / size;
    head = n < front ? static_cast<int>(n) : front;
    vecs = static_cast<int>((n - head) * size / 16);
  }
  __device__ int64_t tail() const { return head + static_cast<int64_t>(vecs) * (16 / size); }
  __device__ float at(int64_t i) const {
    return size == 4 ? ld_elem(reinterpret_cast<const float*>(in) + i) : ld_elem(reinterpret_cast<const uint16_t*>(in) + i);
  }
  __device__ void put(int64_t i, float v) const {
    if (size == 4) st_elem(reinterpret_cast<float*>(out) + i, v);
    else st_elem(reinterpret_cast<uint16_t*>(out) + i, v);
  }
};

// The threads that share a stretch: the block, or of a short one some warps of it, the others taking the next ones.
struct Team {
  int id, size;
};
constexpr int kTeam = 128, kShort = kTeam * kLoads * 16;   // threads, and bytes that they load at once
__device__ __forceinline__ bool team_of(const Stretch& x, int k, Team& team) {
  team = {static_cast<int>(threadIdx.x), kThreads};
  if (x.n * x.size > kShort) return true;
  team = {static_cast<int>(threadIdx.x % kTeam), kTeam};
  return static_cast<int>(threadIdx.x / kTeam) == k % (kThreads / kTeam);
}

// The sum of squares of 16 bytes, in binary64.
__device__ __forceinline__ double squares64(const uint4& w, int size) {
  float x[8];
  if (size == 4) {
    float y[4];
    Piece<float, true>::unpack(w, y);
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = y[k];
#pragma unroll
    for (int k = 4; k < 8; ++k) x[k] = 0.0f;
  } else {
    Piece<uint16_t, true>::unpack(w, x);
  }
  double d = 0.0;
#pragma unroll
  for (int k = 0; k < 8; ++k) d = fma(static_cast<double>(x[k]), static_cast<double>(x[k]), d);
  return d;
}
// of a thread's loads, where binary32 does not do: not inlined, for its registers
__device__ __noinline__ double squares64(uint4 a, uint4 b, uint4 c, uint4 d, int size) {
  return squares64(a, size) + squares64(b, size) + squares64(c, size) + squares64(d, size);
}
static_assert(kLoads == 4, "squares64 takes four");

// Sum of squares of a thread's loads.
template <typename T>
__device__ __forceinline__ double squares(const uint4 (&w)[kLoads]) {
  using P = Piece<T, true>;
  float2 s = both(0.0f);
  uint32_t any = 0;
#pragma unroll
  for (int u = 0; u < kLoads; ++u) {
    float x[P::E];
    P::unpack(w[u], x);
#pragma unroll
    for (int k = 0; k < P::E; k += 2) s = fma2(make_float2(x[k], x[k + 1]), make_float2(x[k], x[k + 1]), s);
    any |= w[u].x | w[u].y | w[u].z | w[u].w;
  }
  const float sum = s.x + s.y;
  // Squares below 2^-126 lose up to 2^-150 each, the smallest of them all they have, and so does a sum of them: 2^-145 for 32.
  // Of 2^-110 or more that is 2^-35, nothing; smaller sums are taken again, unless of zeros (of either sign).  Binary64 is slow
  // here, so what is not needed of it is left: 134 million bf16 near 1e-11 took 533 us with a border of 2^-60, 43 now (as of
  // ordinary values); near 1e-20 they still take 533.
  constexpr uint32_t kMagnitude = sizeof(T) == 2 ? 0x7FFF7FFFu : 0x7FFFFFFFu;
  if (sum <= FLT_MAX && (sum >= 0x1p-110f || (any & kMagnitude) == 0u)) return sum;
  return squares64(w[0], w[1], w[2], w[3], sizeof(T));
}

// This thread's share of the sum over a stretch.  The next loads are under way while one is summed.
__device__ __forceinline__ double squares(const Stretch& x, const Team team) {
  const uint4* const v = reinterpret_cast<const uint4*>(x.in + x.head * x.size);
  const double front = team.id < x.head ? x.at(team.id) : 0.0f, back = x.tail() + team.id < x.n ? x.at(x.tail() + team.id) : 0.0f;
  auto load = [&](int i, uint4 (&w)[kLoads]) {
#pragma unroll
    for (int u = 0; u < kLoads; ++u) w[u] = i + u * team.size < x.vecs ? __ldg(v + i + u * team.size) : make_uint4(0u, 0u, 0u, 0u);
  };
  double d = 0.0;
  uint4 w[kLoads];
  int i = team.id;
  load(i, w);
  while (i < x.vecs) {
    uint4 next[kLoads];
    i += kLoads * team.size;
    load(i, next);
    d += x.size == 4 ? squares<float>(w) : squares<uint16_t>(w);
#pragma unroll
    for (int u = 0; u < kLoads; ++u) w[u] = next[u];
  }
  return fma(front, front, fma(back, back, d));
}

template <typename T>
__device__ __forceinline__ uint4 scaled(const uint4& w, float by) {
  using P = Piece<T, true>;
  float x[P::E];
  P::unpack(w, x);
#pragma unroll
  for (int k = 0; k < P::E; k += 2) {
    const float2 m = mul2(make_float2(x[k], x[k + 1]), both(by));
    x[k] = m.x;
    x[k + 1] = m.y;
  }
  return P::pack(x);
}

// out = in by, from the stretch's end on
__device__ __forceinline__ void scale(const Stretch& x, float by, const Team team) {
  // an output at another place of its 16 bytes is written element by element
  const bool apart = (reinterpret_cast<uintptr_t>(x.in) - reinterpret_cast<uintptr_t>(x.out)) % 16 != 0;
  if (apart) {
    for (int64_t i = team.id; i < x.n; i += team.size) x.put(i, __fmul_rn(x.at(i), by));
    return;
  }
  const uint4* const v = reinterpret_cast<const uint4*>(x.in + x.head * x.size);
  uint4* const o = reinterpret_cast<uint4*>(x.out + x.head * x.size);
  if (x.tail() + team.id < x.n) x.put(x.tail() + team.id, __fmul_rn(x.at(x.tail() + team.id), by));
  if (team.id < x.head) x.put(team.id, __fmul_rn(x.at(team.id), by));
  // the last use of the input, and outputs that should not displace what is still to be read
  for (int i = x.vecs - 1 - team.id; i >= 0; i -= kLoads * team.size) {
    uint4 w[kLoads];
#pragma unroll
    for (int u = 0; u < kLoads; ++u)
      if (i >= u * team.size) w[u] = __ldcs(v + i - u * team.size);
#pragma unroll
    for (int u = 0; u < kLoads; ++u)
      if (i >= u * team.size) __stcs(o + i - u * team.size, x.size == 4 ? scaled<float>(w[u], by) : scaled<uint16_t>(w[u], by));
  }
}

// the sum over the block's threads, in its first warp
__device__ __forceinline__ double block_sum(double s) {
  __shared__ double part[kWarps];
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  if (lane == 0) part[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x >= 32) return 0.0;
  s = part[lane % kWarps];
#pragma unroll
  for (int o = kWarps / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  return s;
}

// The parameters are read through a cache that starts empty: the block's warps read its next tensors at once, where
// one after the other each would wait for its own.
template <int N>
__device__ __forceinline__ void read_ahead(const Table<N>& t, int k, int step) {
  const int at = k + step * 2 * static_cast<int>(threadIdx.x >> 5);
  if (at >= 0 && at <= N) asm volatile("" ::"l"(t.of[at].n));
}

// What a block's run starts with.
struct Start {
  Run run;
  int k;         // the tensor of its first piece
  Entry e, next; // that tensor and the one behind it
  template <int N>
  __device__ explicit Start(const Table<N>& t) : run(t), k(t.starts[blockIdx.x]), e(t.of[k]), next(t.of[k + 1]) {}
};

// This thread's share of the sum over a block's run.
template <int N>
__device__ __forceinline__ double squares(const Table<N>& t, Start s) {
  double sum = 0.0;
  while (s.run.lo < s.run.hi && s.k < N && s.e.first < s.run.hi) {
    const Stretch x(s.e, s.next.first, s.run, t.shift);
    Team team;
    const bool mine = team_of(x, s.k, team);
    ++s.k;
    s.e = s.next;
    if (s.next.first < s.run.hi) s.next = t.of[s.k + 1];
    if (mine) sum += squares(x, team);
  }
  return sum;
}

template <int N>
__global__ void __launch_bounds__(kThreads, kPerSm) k_squares(const __grid_constant__ Table<N> t, double* partial) {
  const Start start(t);
  read_ahead(t, start.k, 1);
  pdl_wait();
  pdl_launch_dependents();
  const double sum = block_sum(squares(t, start));
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

// sqrt(s), in binary32 where its range allows
__device__ __forceinline__ float root(double s) {
  return s >= 1e-30 && s <= 1e30 ? __fsqrt_rn(static_cast<float>(s)) : static_cast<float>(sqrt(s));
}

// the root of the sum of n partial sums, in every thread of the block
__device__ __forceinline__ float root_of(const double* partial, int n) {
  __shared__ float norm;
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) s += partial[i];
  s = block_sum(s);
  if (threadIdx.x == 0) norm = root(s);
  __syncthreads();
  return norm;
}

__global__ void __launch_bounds__(kThreads) k_norm_of(const double* partial, int n, float* norm) {
  pdl_wait();
  pdl_launch_dependents();
  const float r = root_of(partial, n);
  if (threadIdx.x == 0) *norm = r;
}

// The factor of the gradients; a NaN stays.
__device__ __forceinline__ float factor(float max_norm, float norm) {
  const float by = __fdiv_rn(max_norm, norm + 1e-6f);
  return by > 1.0f ? 1.0f : by;
}

// A block's run scaled, from its end: e is the tensor of its last piece, end the first piece behind it.
template <int N>
__device__ __forceinline__ void scale(const Table<N>& t, const Run& run, int k, Entry e, int64_t end, float by) {
  while (run.lo < run.hi) {
    const Stretch x(e, end, run, t.shift);
    Team team;
    const bool mine = team_of(x, k, team), last = e.first <= run.lo;
    end = e.first;
    if (!last) e = t.of[--k];
    if (mine && (by != 1.0f || x.in != x.out)) scale(x, by, team);   // else another's, or in place and nothing to scale
    if (last) break;
  }
}

template <int N>
__global__ void __launch_bounds__(kThreads, kPerSm) k_clip(const __grid_constant__ Table<N> t, const double* partial, int n,
                                                           float max_norm, float* norm) {
  const Run run(t);
  int k = t.starts[blockIdx.x];
  int64_t end = t.of[k + 1].first;
  while (end < run.hi) end = t.of[++k + 1].first;
  const Entry e = t.of[k];
  read_ahead(t, k, -1);
  pdl_wait();
  pdl_launch_dependents();
  const float total = root_of(partial, n);
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = total;
  scale(t, run, k, e, end, factor(max_norm, total));
}

// Both passes of small gradients by one cluster, whose blocks exchange their sums through distributed shared memory:
// one launch and no workspace.
// (seven tensors of 143 KB 7.3 us, 7.0 by two launches, which take the host 10 us instead of 7.5; 900 of 64 elements,
// which meet in few blocks, 95 and 17.)
constexpr int kCluster = 8, kMostSmallTensors = 64;
constexpr int64_t kMostSmall = 1 << 20;   // bytes
template <int N>
__global__ void __launch_bounds__(kThreads) k_clip_small(const __grid_constant__ Table<N> t, bool clip, float max_norm, float* norm) {
  __shared__ double mine;
  const Start start(t);
  read_ahead(t, start.k, 1);
  int k = start.k;
  int64_t end = start.next.first;
  while (end < start.run.hi) end = t.of[++k + 1].first;
  const Entry e = t.of[k];
  pdl_wait();
  pdl_launch_dependents();
  const double sum = block_sum(squares(t, start));
  if (threadIdx.x == 0) mine = sum;
  cluster_sync();
  double v[kCluster];
#pragma unroll
  for (uint32_t r = 0; r < kCluster; ++r)
    asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v[r]) : "r"(mapa_shared(smem_u32(&mine), r)));
#pragma unroll
  for (int n = kCluster / 2; n > 0; n /= 2)
#pragma unroll
    for (int r = 0; r < n; ++r) v[r] += v[r + n];
  const float total = root(v[0]);
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = total;
  if (clip) scale(t, start.run, k, e, end, factor(max_norm, total));
  cluster_sync();   // no block leaves while another may still read its sum
}

// Fills the table with the tensors from `from` on, for `least` to `most` blocks (as many as pieces, between them);
// returns their number.
template <int N>
int fill(Table<N>& t, const ClipTensor* tensors, int64_t from, int64_t n, int least, int most) {
  const int count = static_cast<int>(n - from < N ? n - from : N);
  int64_t pieces;
  t.shift = -1;
  do {
    const int64_t bytes = static_cast<int64_t>(kPiece) << ++t.shift;
    pieces = 0;
    for (int i = 0; i < count; ++i) {
      const ClipTensor& x = tensors[from + i];
      t.of[i] = {x.in, x.out, x.f32 ? -x.n - 1 : x.n, pieces};
      const int64_t each = bytes / (x.f32 ? 4 : 2);
      pieces += (x.n + each - 1) / each;
    }
  } while (pieces >= (int64_t{1} << 30));
  t.of[count] = {nullptr, nullptr, 0, pieces};
  if (count == 0) t.of[1] = t.of[0];   // a block reads its first tensor's entry and the next
  t.pieces = static_cast<int>(pieces);
  const int64_t blocks = pieces < least ? least : (pieces < most ? pieces : most);
  int k = 0;
  for (int64_t b = 0; b < blocks; ++b) {
    while (k + 1 < count && t.of[k + 1].first <= pieces * b / blocks) ++k;
    t.starts[b] = static_cast<uint16_t>(k);
  }
  return static_cast<int>(blocks);
}

template <int N>
cudaError_t run_clip(const ClipTensor* tensors, int64_t n, bool clip, float max_norm, double* partial, float* norm, int num_sms,
                     cudaStream_t s) {
  Table<N> t;
  if constexpr (N <= 100) {
    int64_t bytes = 0;
    for (int64_t i = 0; i < n; ++i) bytes += tensors[i].n * (tensors[i].f32 ? 4 : 2);
    if (n <= kMostSmallTensors && bytes <= kMostSmall) {
      fill(t, tensors, 0, n, kCluster, kCluster);
      return launch_pdl(k_clip_small<N>, dim3(kCluster), dim3(kThreads), 0, s, kCluster, t, clip, max_norm, norm);
    }
  }
  const int most = num_sms * kPerSm < kMaxBlocks ? num_sms * kPerSm : kMaxBlocks;
  int sums = 0, blocks = 0;
  for (int64_t from = 0; from < n; from += N) {
    blocks = fill(t, tensors, from, n, 1, most);
    const cudaError_t e = launch_pdl(k_squares<N>, dim3(blocks), dim3(kThreads), 0, s, 1, t, partial + sums);
    if (e != cudaSuccess) return e;
    sums += blocks;
  }
  if (!clip) return launch_pdl(k_norm_of, dim3(1), dim3(kThreads), 0, s, 1, static_cast<const double*>(partial), sums, norm);
  for (int64_t from = 0; from < n; from += N) {
    if (n > N) blocks = fill(t, tensors, from, n, 1, most);   // else the table is the one just used
    const cudaError_t e = launch_pdl(k_clip<N>, dim3(blocks), dim3(kThreads), 0, s, 1, t, static_cast<const double*>(partial), sums,
                                     max_norm, norm);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

int64_t clip_partials(int64_t n_tensors) {
  const int64_t tables = (n_tensors + kMostTensors - 1) / kMostTensors;
  return (tables < 1 ? 1 : tables) * kMaxBlocks;
}

cudaError_t launch_clip(const ClipTensor* tensors, int64_t n, bool clip, float max_norm, double* partial, float* norm, int num_sms,
                        cudaStream_t s) {
  if (n <= 12) return run_clip<12>(tensors, n, clip, max_norm, partial, norm, num_sms, s);
  if (n <= 100) return run_clip<100>(tensors, n, clip, max_norm, partial, norm, num_sms, s);
  if (n <= 400) return run_clip<400>(tensors, n, clip, max_norm, partial, norm, num_sms, s);
  return run_clip<kMostTensors>(tensors, n, clip, max_norm, partial, norm, num_sms, s);
}

}  // namespace fp8q
