// norm_backward.cu -- layer norm, backward.
//
//   g = dy w,  c1 = sum g / H,  c2 = sum g xh / H,  dx = r (g - c1 - xh c2)
//   dw = sum over rows of dy xh,  db = sum over rows of dy
// with xh = (x - m) r, or the values of its 8-bit copy.  All sums are binary32, in an order
// that depends on the shape alone.
//
// Bound by HBM: dy and x (or the codes) once in, dx once out.  A thread owns the same 16 columns
// for all the rows of its group, so the column sums stay in registers over the whole walk; they
// leave as one partial sum a block, added up by a second, small launch.
#include "norm.cuh"

namespace fp8q {

namespace {

constexpr int kBlockWarps = 16;   // 128 registers a thread
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

// xh of one element, from x or from the codes
template <typename T>
__device__ __forceinline__ float normalised(const NormBwdParams& p, int64_t row, int64_t c, int64_t groups, float mean,
                                            float rstd) {
  if (p.q == nullptr) return (ld_elem(static_cast<const T*>(p.x) + row * p.ldx + c) - mean) * rstd;
  float v, unused;
  decode_pair(p.q[row * p.ldq + c], p.e5m2, v, unused);
  return v * p.s[row * groups + c / 128];
}

// dx of rows of any width: one block per row, two passes.
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

// Rows of up to 16384 columns.  WIDE, rows of more than kBlockWarps warps: 64 registers a thread
// hold the column sums and little else, so dy, xh and w are fetched a second time for dx.
template <typename T, bool VECTOR, bool CODES, bool WIDE>
__global__ void __launch_bounds__((WIDE ? kNormWarpsMost : kBlockWarps) * 32)
    k_norm_backward(const NormBwdParams p, const int warps, const int stages) {
  using P = Piece<T, VECTOR>;
  constexpr int E = P::E, J = 16 / E, H = E / 2;
  constexpr int kIn = CODES ? E : 16;                    // a lane's bytes of x or the codes in one piece
  constexpr int kPiece = 32 * (16 + kIn);                // a warp's bytes of dy and x / codes in one piece
  constexpr int kStage = J * kPiece + 32;                // and in one row, with 4 multipliers, rstd and mean
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float2 red[2][kNormWarpsMost];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = warp / warps, w_in = warp - group * warps;
  const int n_groups = (blockDim.x >> 5) / warps;
  const int64_t step = static_cast<int64_t>(gridDim.x) * n_groups;
  const int cols = static_cast<int>(p.cols), base = w_in * kNormWarpCols, copies = (cols + 127) / 128;
  const float inv_n = 1.0f / static_cast<float>(cols);
  uint8_t* const mine = ring + warp * stages * kStage;

  // row `row` into stage s: every lane its own bytes of dy and x / codes; lanes 0..5 the warp's
  // multipliers, rstd and mean
  auto issue = [&](int64_t row, int s) {
    if constexpr (VECTOR) {
      if (row < p.rows) {
        const uint32_t at = smem_u32(mine + s * kStage);
        const T* dy = static_cast<const T*>(p.dy) + row * p.lddy;
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const int c = P::col(base + j * P::WC, lane, 0), c_in = c < cols ? c : 0;
          cp_async<16>(at + j * kPiece + lane * 16, dy + c_in, c < cols);
          if constexpr (CODES)
            cp_async<kIn>(at + j * kPiece + 512 + lane * kIn, p.q + row * p.ldq + c_in, c < cols);
          else
            cp_async<16>(at + j * kPiece + 512 + lane * 16, static_cast<const T*>(p.x) + row * p.ldx + c_in, c < cols);
        }
        const int g = base / 128 + lane;
        const float* scalar = lane == 4 ? p.rstd + row : p.mean + row;
        bool want = lane == 4 || (lane == 5 && !CODES);
        if (CODES && lane < 4) {
          scalar = p.s + row * copies + (g < copies ? g : 0);
          want = g < copies;
        }
        if (want) cp_async<4>(at + J * kPiece + lane * 4, scalar, true);
      }
      cp_async_commit();
    }
  };
  // dy and xh of piece j of the row in stage s (or, unaligned, of row `row` itself).  Past the
  // row's end dy is 0; xh is finite there unless the row's scalars are not.
  auto fetch = [&](int64_t row, int s, int j, float rstd, float mean, float (&dy)[E], float (&xh)[E]) {
    const int c0 = base + j * P::WC;
    if constexpr (VECTOR) {
      const uint8_t* at = mine + s * kStage + j * kPiece;
      P::unpack(*reinterpret_cast<const uint4*>(at + lane * 16), dy);
      if constexpr (CODES) {
        const float* mult = reinterpret_cast<const float*>(mine + s * kStage + J * kPiece);
        // the codes past the row's end are 0, and their multiplier may be anything
        const float m = P::valid(c0, lane, cols, 0) ? mult[(j * P::WC + lane * E) / 128] : 0.0f;
        P::decode(P::read_codes(at + 512 + lane * kIn), m, p.e5m2, xh);
      } else {
        P::unpack(*reinterpret_cast<const uint4*>(at + 512 + lane * 16), xh);
      }
    } else {
      P::load(static_cast<const T*>(p.dy) + row * p.lddy, c0, lane, cols, dy);
      if constexpr (CODES)
        P::decode(P::load_codes(p.q + row * p.ldq, c0, lane, cols), P::load_multiplier(p.s + row * copies, c0, lane, cols), p.e5m2, xh);
      else
        P::load(static_cast<const T*>(p.x) + row * p.ldx, c0, lane, cols, xh);
    }
    if constexpr (!CODES) {
#pragma unroll
      for (int i = 0; i < E; ++i) xh[i] = (xh[i] - mean) * rstd;
    }
  };

  pdl_wait();
  pdl_launch_dependents();
  float2 dw[J][H], db[J][H];
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int i = 0; i < H; ++i) dw[j][i] = db[j][i] = make_float2(0.0f, 0.0f);
  int64_t row = static_cast<int64_t>(blockIdx.x) * n_groups + group;
  for (int s = 0; s < stages; ++s) issue(row + s * step, s);
  float w[WIDE ? 1 : J][E];
  if constexpr (!WIDE) {
#pragma unroll
    for (int j = 0; j < J; ++j) load_param<P, VECTOR>(p.w, p.w_f32, base + j * P::WC, lane, cols, 1.0f, w[j]);
  }
  for (int s = 0, buf = 0; row < p.rows; row += step, s = s + 1 == stages ? 0 : s + 1, buf ^= 1) {
    float rstd, mean = 0.0f;
    if constexpr (VECTOR) {
      cp_async_wait_oldest(stages);
      __syncwarp();   // the row's scalars were copied by other lanes
      const float* scalars = reinterpret_cast<const float*>(mine + s * kStage + J * kPiece);
      rstd = scalars[4];
      if (!CODES) mean = scalars[5];
    } else {
      rstd = __ldg(p.rstd + row);
      if (!CODES) mean = __ldg(p.mean + row);
    }
    float dy[WIDE ? 1 : J][E], xh[WIDE ? 1 : J][E];
    float2 s1 = {0.0f, 0.0f}, s2 = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < J; ++j) {
      constexpr bool kOne = WIDE;
      const int k = kOne ? 0 : j;
      if constexpr (WIDE) load_param<P, VECTOR>(p.w, p.w_f32, base + j * P::WC, lane, cols, 1.0f, w[0]);
      fetch(row, s, j, rstd, mean, dy[k], xh[k]);
#pragma unroll
      for (int i = 0; i < H; ++i) {
        const float2 d = {dy[k][2 * i], dy[k][2 * i + 1]}, h = {xh[k][2 * i], xh[k][2 * i + 1]};
        const float2 g = mul2(d, make_float2(w[k][2 * i], w[k][2 * i + 1]));
        dw[j][i] = fma2(d, h, dw[j][i]);
        db[j][i] = add2(db[j][i], d);
        s1 = add2(s1, g);
        s2 = fma2(g, h, s2);
      }
    }
    float c1 = warp_sum(s1.x + s1.y), c2 = warp_sum(s2.x + s2.y);
    if (warps > 1) {
      if (lane == 0) red[buf][warp] = make_float2(c1, c2);
      group_sync(group, warps);
      // the other buffer is written before this one is reused
      const float2 v = lane < warps ? red[buf][group * warps + lane] : make_float2(0.0f, 0.0f);
      c1 = warp_sum(v.x);
      c2 = warp_sum(v.y);
    }
    const float2 m1 = both(-c1 * inv_n), m2 = both(-c2 * inv_n), r = both(rstd);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      constexpr bool kOne = WIDE;
      const int k = kOne ? 0 : j;
      if constexpr (WIDE) {
        load_param<P, VECTOR>(p.w, p.w_f32, base + j * P::WC, lane, cols, 1.0f, w[0]);
        fetch(row, s, j, rstd, mean, dy[0], xh[0]);
      }
      float out[E];
#pragma unroll
      for (int i = 0; i < H; ++i) {
        const float2 d = {dy[k][2 * i], dy[k][2 * i + 1]}, h = {xh[k][2 * i], xh[k][2 * i + 1]};
        const float2 v = mul2(r, fma2(h, m2, fma2(d, make_float2(w[k][2 * i], w[k][2 * i + 1]), m1)));
        out[2 * i] = v.x;
        out[2 * i + 1] = v.y;
      }
      P::store(static_cast<T*>(p.dx) + row * p.lddx, base + j * P::WC, lane, cols, out);
    }
    if constexpr (VECTOR) __syncwarp();   // all lanes have read the stage's scalars
    issue(row + stages * step, s);
  }
  if (p.dw == nullptr && p.db == nullptr) return;
  // the block's groups joined pairwise in shared memory (the ring is free: every copy was waited for)
  __syncthreads();
  float2* join = reinterpret_cast<float2*>(ring);
  for (int n = n_groups; n > 1;) {
    const int half = (n + 1) / 2;
    if (group >= half && group < n) {
      float2* out = join + ((group - half) * warps + w_in) * 512 + lane;
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < H; ++i) {
          out[(j * H + i) * 32] = dw[j][i];
          out[(j * H + i) * 32 + 256] = db[j][i];
        }
    }
    __syncthreads();
    if (group < n - half) {
      const float2* in = join + (group * warps + w_in) * 512 + lane;
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < H; ++i) {
          dw[j][i] = add2(dw[j][i], in[(j * H + i) * 32]);
          db[j][i] = add2(db[j][i], in[(j * H + i) * 32 + 256]);
        }
    }
    __syncthreads();
    n = half;
  }
  if (group != 0) return;
  // one block's sums are the result; several leave partial sums
  const bool last = gridDim.x == 1;
  float* part = p.partial + static_cast<int64_t>(blockIdx.x) * 2 * cols;
  void* to_dw = last ? p.dw : part;
  void* to_db = last ? p.db : part + cols;
  const bool f32 = !last || p.w_f32;
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int c = P::col(base + j * P::WC, lane, i);
      if (c >= cols) continue;
      if (to_dw != nullptr) st_param(to_dw, f32, c, i % 2 ? dw[j][i / 2].y : dw[j][i / 2].x);
      if (to_db != nullptr) st_param(to_db, f32, c, i % 2 ? db[j][i / 2].y : db[j][i / 2].x);
    }
}

// The 2 * cols sums of the partial sums: a block takes 32 of them, warp k the partials k, k + 8,
// ...; then the 8 warps' sums in order.
__global__ void __launch_bounds__(kThreads) k_norm_params(const float* partial, int n, int64_t cols, bool f32, void* dw,
                                                          void* db) {
  __shared__ float part[kWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  pdl_wait();
  pdl_launch_dependents();
  float v = 0.0f;
  if (c < 2 * cols)
    for (int k = warp; k < n; k += kWarps) v += partial[static_cast<int64_t>(k) * 2 * cols + c];
  part[warp][lane] = v;
  __syncthreads();
  if (warp != 0 || c >= 2 * cols) return;
  v = 0.0f;
#pragma unroll
  for (int k = 0; k < kWarps; ++k) v += part[k][lane];
  void* out = c < cols ? dw : db;
  if (out != nullptr) st_param(out, f32, c < cols ? c : c - cols, v);
}

// number of partial sums left in p.partial (0: none)
template <typename T, bool VECTOR, bool CODES>
cudaError_t run_norm_backward(const NormBwdParams& p, int num_sms, cudaStream_t s, int* partials) {
  using P = Piece<T, VECTOR>;
  const int stage = VECTOR ? 16 / P::E * 32 * (16 + (CODES ? P::E : 16)) + 32 : 0;
  NormPlan n = norm_plan(p.rows, p.cols, kBlockWarps, stage, num_sms < kMaxNormPartials ? num_sms : kMaxNormPartials);
  const size_t join = static_cast<size_t>(n.groups / 2) * n.warps * 1024 * sizeof(float);
  if (n.smem < join) n.smem = join;
  static std::atomic<bool> done[2][kMaxDevices];
  auto kernel = n.wide ? k_norm_backward<T, VECTOR, CODES, true> : k_norm_backward<T, VECTOR, CODES, false>;
  const cudaError_t e = ensure_smem_limit(kernel, kNormSmem, done[n.wide]);
  if (e != cudaSuccess) return e;
  *partials = n.blocks > 1 ? n.blocks : 0;
  return launch_pdl(kernel, dim3(n.blocks), dim3(static_cast<unsigned>(n.warps * n.groups * 32)), n.smem, s, 1, p, n.warps,
                    n.stages);
}

template <typename T>
cudaError_t run_any(const NormBwdParams& p, int num_sms, cudaStream_t s, int* partials) {
  const int64_t cap = static_cast<int64_t>(num_sms) * 8;
  if (p.rows > 0) {
    const cudaError_t e = launch_pdl(k_norm_dx_any<T>, dim3(static_cast<unsigned>(p.rows < cap ? p.rows : cap)), dim3(kThreads),
                                     0, s, 1, p);
    if (e != cudaSuccess) return e;
  }
  if (p.dw == nullptr && p.db == nullptr) return cudaSuccess;
  *partials = norm_partials(p.rows);
  return launch_pdl(k_norm_partial_any<T>, dim3(static_cast<unsigned>((p.cols + kThreads - 1) / kThreads), *partials),
                    dim3(kThreads), 0, s, 1, p, *partials);
}

}  // namespace

int norm_partials(int64_t rows) { return static_cast<int>(rows < 1 ? 1 : (rows > kMaxNormPartials ? kMaxNormPartials : rows)); }

cudaError_t launch_norm_backward(const NormBwdParams& p, int num_sms, cudaStream_t s) {
  const int64_t size = p.f32 ? 4 : 2, e16 = 16 / size;
  int partials = 0;
  cudaError_t e;
  if (p.cols > kNormWarpsMost * kNormWarpCols || p.rows == 0) {
    e = p.f32 ? run_any<float>(p, num_sms, s, &partials) : run_any<uint16_t>(p, num_sms, s, &partials);
  } else {
    const bool vec = takes(p.dy, p.lddy, p.cols, size, 16) && takes(p.x, p.ldx, p.cols, size, 16) &&
                     takes(p.dx, p.lddx, p.cols, size, 16) && takes(p.q, p.ldq, p.cols, 1, e16) && takes(p.w, 0, 0, 1, 16);
#define FP8Q_RUN(T, V) \
  (p.q != nullptr ? run_norm_backward<T, V, true>(p, num_sms, s, &partials) : run_norm_backward<T, V, false>(p, num_sms, s, &partials))
    e = p.f32 ? (vec ? FP8Q_RUN(float, true) : FP8Q_RUN(float, false))
              : (vec ? FP8Q_RUN(uint16_t, true) : FP8Q_RUN(uint16_t, false));
#undef FP8Q_RUN
  }
  if (e != cudaSuccess || partials == 0 || (p.dw == nullptr && p.db == nullptr)) return e;
  return launch_pdl(k_norm_params, dim3(static_cast<unsigned>((2 * p.cols + 31) / 32)), dim3(kThreads), 0, s, 1,
                    static_cast<const float*>(p.partial), partials, p.cols, p.w_f32 != 0, p.dw, p.db);
}

}  // namespace fp8q
