// norm.cuh -- how the layer norm kernels divide rows: a group of `warps` warps holds one row at
// a time, each warp a fixed number of its columns, and walks the rows grid-wide.  A block holds
// as many groups as its warps allow (what fits an SM's registers), and there is a block an SM.
// The next rows of each group are on their way into shared memory by asynchronous copies of 16
// bytes a lane.  Rows that are not 16-byte aligned are copied by their aligned 16-byte granules
// and read at their own offset; a warp reads what its own lanes copied, so no block barrier guards them.
#pragma once
#include "internal.h"
#include "rowops.cuh"

namespace fp8q {

constexpr int kNormStages = 4;        // most rows in flight a group
// Bytes in flight that a block aims at.  Fewer leave HBM waiting (backward from codes, 65536x4096:
// 72 KB 218 us, 108 KB 212); more lengthen the walk's end, where rows have arrived and wait for
// their turn (forward, 8192x4096: 96 KB 32.6 us, 192 KB 34.6; 32768x1024 20.8 and 25.1).
constexpr int kNormInFlight = 96 * 1024;
constexpr int kNormSmem = 220 * 1024; // dynamic shared memory of a block: those rows and the parameters

// How a launch divides its rows (host side).
struct NormPlan {
  int warps;        // warps a row
  int groups;       // rows a block has at a time
  int stages;       // rows in flight a group
  int blocks;
  int ring;         // where the rows in flight start in shared memory
  size_t smem;
};
// warp_cols: columns of a warp; block_warps: most warps of a block; params: parameter vectors kept
// in shared memory in binary32; stage_bytes: shared memory of one warp's part of one row
inline NormPlan norm_plan(int64_t rows, int64_t cols, int warp_cols, int block_warps, int params, int stage_bytes, int num_sms) {
  NormPlan n{};
  n.warps = static_cast<int>((cols + warp_cols - 1) / warp_cols);
  n.groups = n.warps < block_warps ? block_warps / n.warps : 1;
  if (n.warps > 1 && n.groups > 15) n.groups = 15;   // a named barrier a group, 1..15
  // few rows: spread over the SMs first
  const int64_t per_sm = (rows + num_sms - 1) / num_sms;
  if (n.groups > per_sm) n.groups = static_cast<int>(per_sm);
  n.ring = params * n.warps * warp_cols * 4;
  const int64_t room = kNormSmem - n.ring, stage = static_cast<int64_t>(stage_bytes) * n.warps * n.groups;
  const int64_t want_stages = (kNormInFlight + stage - 1) / stage;
  n.stages = static_cast<int>(want_stages < 2 ? 2 : (want_stages > kNormStages ? kNormStages : want_stages));
  if (n.stages * stage > room) n.stages = static_cast<int>(room / stage > 1 ? room / stage : 1);
  const int64_t want = (rows + n.groups - 1) / n.groups;
  n.blocks = static_cast<int>(want < num_sms ? want : num_sms);
  n.smem = static_cast<size_t>(n.ring + stage * n.stages);
  return n;
}

// the first n of BYTES bytes, and zeros
template <int BYTES>
__device__ __forceinline__ void cp_async_part(uint32_t dst, const void* src, int n) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(n) : "memory");
}
template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, bool valid) {
  cp_async_part<BYTES>(dst, src, valid ? BYTES : 0);
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// A parameter vector (`none` without one; past its end anything finite) in shared memory as
// binary32, in the order in which a warp's lanes read their pieces, four values a lane: a quad.
// The block starts the copies here, ahead of its first rows', and finishes them (of bf16: widens
// them) in settle_param once its own copies have arrived; a barrier follows.
template <typename P, int V>
__device__ __forceinline__ int quad_col(int i) {   // first column of quad i
  constexpr int Q = P::E / 4, J = V / P::E;
  const int l = i & 31, q = (i >> 5) % Q, j = (i >> 5) / Q % J, w = (i >> 5) / (Q * J);
  return w * 32 * V + j * P::WC + P::first(l) + P::at(q * 4);
}
template <typename P, int V>
__device__ __forceinline__ void start_param(const void* vec, bool f32, int cols, int warps, float none, float* to) {
  // every block reads the whole vector: each starts at another place of it
  const int n = warps * 8 * V, turn = static_cast<int>(blockIdx.x) * 97 % (n / 32) * 32;
  for (int k = threadIdx.x; k < n; k += blockDim.x) {
    const int i = k + turn < n ? k + turn : k + turn - n, c = quad_col<P, V>(i);
    if (vec == nullptr) {
      reinterpret_cast<float4*>(to)[i] = make_float4(none, none, none, none);
    } else if (P::kVector) {   // cols is a multiple of 4 and the vector 16-byte aligned
      const int from = c < cols ? c : 0;
      if (f32)
        cp_async<16>(smem_u32(to + 4 * i), static_cast<const float*>(vec) + from, c < cols);
      else
        cp_async<8>(smem_u32(to + 4 * i), static_cast<const uint16_t*>(vec) + from, c < cols);
    } else {
#pragma unroll
      for (int m = 0; m < 4; ++m) to[4 * i + m] = c + P::at(m) < cols ? ld_param(vec, f32, c + P::at(m)) : 0.0f;
    }
  }
}
template <typename P, int V>
__device__ __forceinline__ void settle_param(const void* vec, bool f32, int warps, float* at) {
  if (vec == nullptr || f32 || !P::kVector) return;
  const int n = warps * 8 * V, turn = static_cast<int>(blockIdx.x) * 97 % (n / 32) * 32;
  for (int k = threadIdx.x; k < n; k += blockDim.x) {
    const int i = k + turn < n ? k + turn : k + turn - n;
    const uint2 u = *reinterpret_cast<const uint2*>(at + 4 * i);
    reinterpret_cast<float4*>(at)[i] = make_float4(bf16lo(u.x), bf16hi(u.x), bf16lo(u.y), bf16hi(u.y));
  }
}
// the lane's values of piece j of warp w
template <typename P, int V>
__device__ __forceinline__ void read_param(const float* from, int w, int j, int lane, float (&v)[P::E]) {
#pragma unroll
  for (int q = 0; q < P::E / 4; ++q) {
    const float4 u = *reinterpret_cast<const float4*>(from + (w * 32 * V + j * 32 * P::E + q * 128 + lane * 4));
    v[4 * q] = u.x;
    v[4 * q + 1] = u.y;
    v[4 * q + 2] = u.z;
    v[4 * q + 3] = u.w;
  }
}

// Barrier of one group's warps (warps > 1).
__device__ __forceinline__ void group_sync(int group, int warps) {
  asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(warps * 32) : "memory");
}

// One warp's part of a row, SPAN columns from column `base` on, in shared memory: SPAN / E granules
// of E elements, unaligned one more.  VECTOR: granule k holds the elements from base + k E on; otherwise
// from base + k E - m on, where row + base - m is a multiple of E elements.
template <typename P, int SPAN, bool VECTOR, typename T>
struct RowPart {
  static constexpr int G = P::E * static_cast<int>(sizeof(T));   // bytes of a granule (T: the data's type, or one-byte codes)
  static constexpr int K = SPAN / P::E;
  // a multiple of 128: 32 lanes' 16 bytes then fill whole lines of shared memory (starting 16 bytes
  // off them, 8192x4096 forward took 36.8 us instead of 33.6)
  static constexpr int kBytes = VECTOR ? K * G : (K * G + G + 127) / 128 * 128;

  __device__ static __forceinline__ int past(const T* p) {
    return VECTOR ? 0 : static_cast<int>(reinterpret_cast<uintptr_t>(p) / sizeof(T) % P::E);
  }
  // Copies of granules lane, lane + 32, ... of the row that starts at `row`, `before` elements of
  // whose matrix lie in front of it; zeros past its end.  What a granule holds in front of the
  // row is never used.
  __device__ static __forceinline__ void start(uint8_t* to, const T* row, int64_t before, int base, int cols, int lane) {
    uint32_t at = smem_u32(to) + lane * G;
    if constexpr (VECTOR) {
      const int left = cols - base - lane * P::E;
      const T* const p = row + (left > 0 ? base + lane * P::E : 0);
#pragma unroll
      for (int j = 0; j < K / 32; ++j) cp_async<G>(at + j * 32 * G, left > j * P::WC ? p + j * P::WC : p, left > j * P::WC);
    } else {
      const int m = past(row + base), c0 = base + lane * P::E - m;
      const T* const p = row + c0;
      if (base >= P::E && cols - base >= SPAN + P::E) {   // every granule is the row's: the whole warp takes this way
#pragma unroll
        for (int j = 0; j < K / 32; ++j) cp_async<G>(at + j * 32 * G, p + j * P::WC, true);
        if (lane == 0 && m != 0) cp_async<G>(at + K * G, p + SPAN, true);
        return;
      }
#pragma unroll
      for (int k0 = 0; k0 <= K; k0 += 32) {
        const int c = c0 + k0 * P::E;
        if (k0 == K && (lane != 0 || m == 0)) continue;
        const int have = min(max(cols - c, 0), P::E);   // elements in front of the row's end
        if (have > 0 && before + c < 0) {               // a granule that starts in front of the matrix
          T* const out = reinterpret_cast<T*>(to + (k0 + lane) * G);
          for (int i = 0; i < P::E; ++i)
            if (c + i >= 0) out[i] = i < have ? row[c + i] : T(0);
        } else {
          cp_async_part<G>(at + k0 * G, have > 0 ? row + c : row + base - m, have * static_cast<int>(sizeof(T)));
        }
      }
    }
  }
  // The lane's values of piece j; m = past(row + base).
  __device__ static __forceinline__ void read(const uint8_t* from, int m, int lane, int j, float (&v)[P::E]) {
    if constexpr (P::kStrided) {
#pragma unroll
      for (int i = 0; i < P::E; ++i) v[i] = *reinterpret_cast<const T*>(from + (m + j * P::WC + lane + P::at(i)) * G / P::E);
    } else {
      const uint8_t* const at = from + (j * 32 + lane) * G;
      if (VECTOR || m == 0)
        P::unpack(*reinterpret_cast<const uint4*>(at), v);
      else
        P::unpack(P::words(reinterpret_cast<const uint32_t*>(at + (m & ~1) * static_cast<int>(sizeof(T))), (m & 1) != 0), v);
    }
  }
  template <int J>
  __device__ static __forceinline__ void read(const uint8_t* from, int m, int lane, float (&v)[J][P::E]) {
#pragma unroll
    for (int j = 0; j < J; ++j) read(from, m, lane, j, v[j]);
  }
  // the same of one-byte codes
  __device__ static __forceinline__ typename P::Codes read_codes(const uint8_t* from, int m, int lane, int j) {
    if constexpr (P::kStrided) {
      typename P::Codes c = {};
#pragma unroll
      for (int i = 0; i < P::E; ++i) c.u[0] |= static_cast<uint32_t>(from[m + j * P::WC + lane + P::at(i)]) << (8 * i);
      return c;
    } else {
      const uint8_t* const at = from + (j * 32 + lane) * G + m;
      return VECTOR || m == 0 ? P::read_codes(at) : P::code_words(at);
    }
  }
};
// until at most `stages` - 1 of the committed copies are outstanding
__device__ __forceinline__ void cp_async_wait_oldest(int stages) {
  if (stages == 5)
    asm volatile("cp.async.wait_group 4;" ::: "memory");
  else if (stages == 4)
    asm volatile("cp.async.wait_group 3;" ::: "memory");
  else if (stages == 3)
    asm volatile("cp.async.wait_group 2;" ::: "memory");
  else if (stages == 2)
    asm volatile("cp.async.wait_group 1;" ::: "memory");
  else
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

}  // namespace fp8q
