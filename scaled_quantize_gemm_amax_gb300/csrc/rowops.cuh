// rowops.cuh -- device helpers of the operators that work on rows of a matrix (layer norm,
// gated activation, expert dispatch): how a warp holds a piece of a row, and the 8-bit copy of
// 128 consecutive columns of a row.
//
// bf16 elements are held as their 16-bit patterns; all arithmetic is binary32.
#pragma once
#include <cstdint>

#include "ptx.cuh"
#include "recipes.cuh"

namespace fp8q {

__device__ __forceinline__ float ld_elem(const uint16_t* p) { return __uint_as_float(static_cast<uint32_t>(*p) << 16); }
__device__ __forceinline__ float ld_elem(const float* p) { return *p; }
// element i of a parameter vector (weight, bias) of either type
__device__ __forceinline__ float ld_param(const void* p, bool f32, int64_t i) {
  return f32 ? static_cast<const float*>(p)[i] : ld_elem(static_cast<const uint16_t*>(p) + i);
}

// two binary32 -> two bf16, nearest even, `lo` in the low half
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ void st_elem(uint16_t* p, float v) { *p = static_cast<uint16_t>(pack_bf16(v, 0.0f)); }
__device__ __forceinline__ void st_elem(float* p, float v) { *p = v; }
__device__ __forceinline__ void st_param(void* p, bool f32, int64_t i, float v) {
  if (f32)
    static_cast<float*>(p)[i] = v;
  else
    st_elem(static_cast<uint16_t*>(p) + i, v);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// Two binary32 operations in one instruction (sm_100 and later), each rounded to nearest.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// max(|a|, |b|, |c|), NaN ignored (all NaN: NaN)
__device__ __forceinline__ float max_abs3(float a, float b, float c) {
  float d;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// ------------------------------------------------------------------ a warp's piece of a row
// How a warp holds WC consecutive columns of a row, E = 16 bytes' worth a lane.
//   VECTOR           the row is 16-byte aligned and cols % E == 0 (a lane is all in or all out):
//                    lane l the E columns from l E on, one 16-byte access.
//   bf16 otherwise   the same columns, in 4-byte words: rows that start at an odd element are read
//                    a word more and shifted by half a word; what a lane stores begins with the
//                    lane before's last value, so that every word but the ends' is whole.  A run
//                    of pieces that touches the row's end goes element by element; no byte outside
//                    the row is touched.  (8192x9001 gated SiLU, when chosen, 124 us; element by element
//                    throughout 265; aligned 16-byte granules shifted over the lanes 157, 11 selections
//                    a lane and tensor; pairs 2 l and 2 l + 64, halves exchanged between lanes, 147.)
//   binary32 otherwise  lane l columns l, l + 32, l + 64, l + 96, element by element, which
//                    coalesces at any alignment (4096x9001 gated SiLU, when chosen, 84 us; granules 136).
// A lane works from its own first column `c` of the row: pointers point there, and `left` is the
// number of columns from there to the row's end (possibly none).  Every function is called by
// the whole warp, with the same values but for the lane's own c and left.
// 128-column groups (the 8-bit copy's) are kGroupLanes lanes.
template <typename T, bool VECTOR>
struct Piece {
  static constexpr bool kVector = VECTOR;
  static constexpr bool kStrided = !VECTOR && sizeof(T) == 4;
  static constexpr int E = 16 / static_cast<int>(sizeof(T));
  static constexpr int WC = 32 * E;
  static constexpr int kGroupLanes = 128 / E;
  static constexpr int kWords = E / 4;   // of codes

  __device__ static __forceinline__ int first(int lane) { return kStrided ? lane : lane * E; }
  // column of value i after the lane's first
  __device__ static __forceinline__ constexpr int at(int i) { return kStrided ? 32 * i : i; }
  __device__ static __forceinline__ bool has(int left, int i) { return left > (VECTOR ? 0 : at(i)); }
  __device__ static __forceinline__ uint32_t bits(const T* p) {
    if constexpr (sizeof(T) == 2)
      return *p;
    else
      return __float_as_uint(*p);
  }
  // whether p is at an odd element of a 4-byte word (bf16)
  __device__ static __forceinline__ bool odd(const T* p) { return (reinterpret_cast<uintptr_t>(p) & 2) != 0; }
  // 16 bytes from 4-byte words at w, or from two bytes on (shared memory)
  __device__ static __forceinline__ uint4 words(const uint32_t* w, bool half) {
    const uint32_t a = w[0], b = w[1], c = w[2], d = w[3];
    if (!half) return make_uint4(a, b, c, d);
    return make_uint4(__funnelshift_r(a, b, 16), __funnelshift_r(b, c, 16), __funnelshift_r(c, d, 16), __funnelshift_r(d, w[4], 16));
  }

  // The lane's values of N consecutive pieces as they lie in memory (0 past the row's end): what
  // waits in registers waits in this form.  Unaligned bf16 from an odd element is held as the words
  // around it until settle(), so that loads that nothing waits for yet stay in flight together.
  template <int N>
  struct Run {
    uint4 r[N];
    uint32_t past[N];   // the word after each piece's four
    bool half;
  };
  template <int N>
  __device__ static __forceinline__ void clear(Run<N>& x) {
#pragma unroll
    for (int j = 0; j < N; ++j) x.r[j] = make_uint4(0u, 0u, 0u, 0u);
    x.half = false;
  }
  template <int N>
  __device__ static __forceinline__ void settle(Run<N>& x) {
    if constexpr (!VECTOR && !kStrided) {
      if (!x.half) return;
#pragma unroll
      for (int j = 0; j < N; ++j)
        x.r[j] = make_uint4(__funnelshift_r(x.r[j].x, x.r[j].y, 16), __funnelshift_r(x.r[j].y, x.r[j].z, 16),
                            __funnelshift_r(x.r[j].z, x.r[j].w, 16), __funnelshift_r(x.r[j].w, x.past[j], 16));
    }
  }
  template <int N>
  __device__ static __forceinline__ void load_raw(const T* p, int c, int left, Run<N>& x) {
    uint4(&r)[N] = x.r;
    if constexpr (VECTOR) {
#pragma unroll
      for (int j = 0; j < N; ++j)
        r[j] = left > j * WC ? __ldg(reinterpret_cast<const uint4*>(p + j * WC)) : make_uint4(0u, 0u, 0u, 0u);
    } else if constexpr (kStrided) {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int rest = left - j * WC;
        const T* q = p + j * WC;
        r[j] = make_uint4(has(rest, 0) ? bits(q) : 0u, has(rest, 1) ? bits(q + at(1)) : 0u, has(rest, 2) ? bits(q + at(2)) : 0u,
                          has(rest, 3) ? bits(q + at(3)) : 0u);
      }
    } else {
      const int lane = threadIdx.x & 31, row_left = left + first(lane);
      const bool half = odd(p);
      // every word is the row's: the whole warp takes this way
      if ((c > first(lane) || !half) && row_left > N * WC) {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(p - (half ? 1 : 0));
        x.half = half;
#pragma unroll
        for (int j = 0; j < N; ++j) {
          r[j] = make_uint4(__ldg(w + j * WC / 2), __ldg(w + j * WC / 2 + 1), __ldg(w + j * WC / 2 + 2), __ldg(w + j * WC / 2 + 3));
          if (half) x.past[j] = __ldg(w + j * WC / 2 + 4);
        }
      } else {
        x.half = false;
#pragma unroll
        for (int j = 0; j < N; ++j) {
          uint32_t u[4] = {0u, 0u, 0u, 0u};
#pragma unroll
          for (int i = 0; i < E; ++i)
            if (left - j * WC > i) u[i / 2] |= bits(p + j * WC + i) << (i % 2 * 16);
          r[j] = make_uint4(u[0], u[1], u[2], u[3]);
        }
      }
    }
  }
  template <int N>
  __device__ static __forceinline__ void load(const T* p, int c, int left, float (&v)[N][E]) {
    Run<N> x;
    load_raw(p, c, left, x);
    settle(x);
#pragma unroll
    for (int j = 0; j < N; ++j) unpack(x.r[j], v[j]);
  }
  __device__ static __forceinline__ void unpack(const uint4& w, float (&v)[E]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 2) {
        v[2 * i] = bf16lo(u[i]);
        v[2 * i + 1] = bf16hi(u[i]);
      } else {
        v[i] = __uint_as_float(u[i]);
      }
    }
  }
  __device__ static __forceinline__ uint4 pack(const float (&v)[E]) {
    if constexpr (sizeof(T) == 2)
      return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
    else
      return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
  __device__ static __forceinline__ void store_bits(T* p, uint32_t b) {
    if constexpr (sizeof(T) == 2)
      *p = static_cast<uint16_t>(b);
    else
      *p = __uint_as_float(b);
  }
  // N consecutive pieces, packed
  template <int N>
  __device__ static __forceinline__ void store_raw(T* p, int left, const uint4 (&r)[N]) {
    if constexpr (VECTOR) {
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (left > j * WC) *reinterpret_cast<uint4*>(p + j * WC) = r[j];
    } else if constexpr (kStrided) {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const uint32_t u[4] = {r[j].x, r[j].y, r[j].z, r[j].w};
#pragma unroll
        for (int i = 0; i < E; ++i)
          if (has(left - j * WC, i)) store_bits(p + j * WC + at(i), u[i]);
      }
    } else {
      const int lane = threadIdx.x & 31;
      const bool half = odd(p);
      if (left + first(lane) < N * WC) {   // the row ends in the run: the whole warp takes this way
#pragma unroll
        for (int j = 0; j < N; ++j) {
          if (N > 2 && left + first(lane) <= j * WC) break;
          const uint32_t u[4] = {r[j].x, r[j].y, r[j].z, r[j].w};
#pragma unroll
          for (int i = 0; i < E; ++i)
            if (left - j * WC > i) store_bits(p + j * WC + i, u[i / 2] >> (i % 2 * 16));
        }
      } else if (!half) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
          uint32_t* w = reinterpret_cast<uint32_t*>(p + j * WC);
          w[0] = r[j].x, w[1] = r[j].y, w[2] = r[j].z, w[3] = r[j].w;
        }
      } else {
        // word k: the last value before, then value 2 k; the lane before lane 0 is lane 31 of the piece before
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const uint32_t give = lane == 31 && j > 0 ? r[j > 0 ? j - 1 : 0].w : r[j].w;
          const uint32_t before = __shfl_sync(0xFFFFFFFFu, give, (lane + 31) & 31);
          T* q = p + j * WC;
          uint32_t* w = reinterpret_cast<uint32_t*>(q - 1);
          if (lane > 0 || j > 0)
            w[0] = __funnelshift_r(before, r[j].x, 16);
          else
            store_bits(q, r[j].x);
          w[1] = __funnelshift_r(r[j].x, r[j].y, 16);
          w[2] = __funnelshift_r(r[j].y, r[j].z, 16);
          w[3] = __funnelshift_r(r[j].z, r[j].w, 16);
        }
        if (lane == 31) store_bits(p + (N - 1) * WC + E - 1, r[N - 1].w >> 16);
      }
    }
  }
  template <int N>
  __device__ static __forceinline__ void store(T* p, int left, const float (&v)[N][E]) {
    uint4 r[N];
#pragma unroll
    for (int j = 0; j < N; ++j) r[j] = pack(v[j]);
    store_raw(p, left, r);
  }
  // The lane's part of a parameter vector (`none` without one and past its end), element by element.
  __device__ static __forceinline__ void load_param(const void* vec, bool f32, int c, int left, float none, float (&v)[E]) {
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = vec != nullptr && has(left, i) ? ld_param(vec, f32, c + at(i)) : none;
  }

  // ---- the 8-bit copy
  // max |v| of the lane's columns (NaN ignored)
  __device__ static __forceinline__ float amax(const float (&v)[E], int left) {
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < E; i += 2) a = max_abs3(a, VECTOR || has(left, i) ? v[i] : 0.0f, VECTOR || has(left, i + 1) ? v[i + 1] : 0.0f);
    return left > 0 ? a : 0.0f;
  }
  // codes = satRNE(v sc)
  template <bool E5>
  __device__ static __forceinline__ void encode(uint8_t* q, int left, const float (&v)[E], float sc) {
    uint32_t u[E / 2], w[kWords];
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      const float2 m = mul2(make_float2(v[2 * i], v[2 * i + 1]), both(sc));
      u[i] = E5 ? cvt_pair_e5m2(m.x, m.y) : cvt_pair_e4m3(m.x, m.y);
    }
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = __byte_perm(u[2 * i], u[2 * i + 1], 0x5410);
    if (VECTOR ? left > 0 : !kStrided && left >= E && reinterpret_cast<uintptr_t>(q) % E == 0) {
      if constexpr (E == 8)
        *reinterpret_cast<uint2*>(q) = make_uint2(w[0], w[1]);
      else
        *reinterpret_cast<uint32_t*>(q) = w[0];
    } else if (!VECTOR) {
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (has(left, i)) q[at(i)] = static_cast<uint8_t>(w[i / 4] >> (8 * (i % 4)));
    }
  }
  // The codes of a lane's columns, value i in byte i % 4 of word i / 4 (0 past the row's end).
  struct Codes {
    uint32_t u[kWords];
  };
  __device__ static __forceinline__ Codes read_codes(const uint8_t* q) {   // E codes at q, a multiple of E
    Codes c;
    if constexpr (E == 8) {
      const uint2 w = *reinterpret_cast<const uint2*>(q);
      c.u[0] = w.x;
      c.u[1] = w.y;
    } else {
      c.u[0] = *reinterpret_cast<const uint32_t*>(q);
    }
    return c;
  }
  // E codes at any byte, all of whose 4-byte words may be read
  __device__ static __forceinline__ Codes code_words(const uint8_t* q) {
    const int m = static_cast<int>(reinterpret_cast<uintptr_t>(q) & 3);
    const uint32_t* w = reinterpret_cast<const uint32_t*>(q - m);
    Codes c;
#pragma unroll
    for (int i = 0; i < kWords; ++i) c.u[i] = __funnelshift_r(w[i], w[i + 1], m * 8);
    return c;
  }
  __device__ static __forceinline__ Codes load_codes(const uint8_t* q, int c, int left) {
    Codes r = {};
    if constexpr (VECTOR) {
      if (left > 0) r = read_codes(q);
    } else if constexpr (kStrided) {
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (has(left, i)) r.u[0] |= static_cast<uint32_t>(q[at(i)]) << (8 * i);
    } else {
      const int lane = threadIdx.x & 31;
      if (c > first(lane) && left + first(lane) >= WC + 4) {   // every word is the row's: the whole warp takes this way
        r = code_words(q);
      } else {
#pragma unroll
        for (int i = 0; i < E; ++i)
          if (left > i) r.u[i / 4] |= static_cast<uint32_t>(q[i]) << (8 * (i % 4));
      }
    }
    return r;
  }
  // the codes' own values
  __device__ static __forceinline__ void decode(const Codes& c, bool e5m2, float (&v)[E]) {
    if (e5m2) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        decode_pair(c.u[i] & 0xFFFFu, true, v[4 * i], v[4 * i + 1]);
        decode_pair(c.u[i] >> 16, true, v[4 * i + 2], v[4 * i + 3]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        decode_pair(c.u[i] & 0xFFFFu, false, v[4 * i], v[4 * i + 1]);
        decode_pair(c.u[i] >> 16, false, v[4 * i + 2], v[4 * i + 3]);
      }
    }
  }
  // the values the codes stand for, each product rounded to binary32
  __device__ static __forceinline__ void decode(const Codes& c, float s, bool e5m2, float (&v)[E]) {
    decode(c, e5m2, v);
#pragma unroll
    for (int i = 0; i < E; i += 2) {
      const float2 m = mul2(make_float2(v[i], v[i + 1]), both(s));
      v[i] = m.x;
      v[i + 1] = m.y;
    }
  }
};

// The maximum over each `W`-lane group of N values a lane (N = 1, 2 or 4): lane l gets value
// l % N's.  Each exchange halves the values a lane carries, so N maxima cost log2(W) + N - 1 -
// log2(N) exchanges instead of N log2(W).
template <int N, int W>
__device__ __forceinline__ float group_max(const float (&a)[N], int lane) {
  constexpr uint32_t kAll = 0xFFFFFFFFu;
  float m;
  if constexpr (N == 1) {
    m = a[0];
  } else {
    float k[N / 2];
#pragma unroll
    for (int h = 0; h < N / 2; ++h) {
      const float keep = lane & 1 ? a[2 * h + 1] : a[2 * h], give = lane & 1 ? a[2 * h] : a[2 * h + 1];
      k[h] = fmaxf(keep, __shfl_xor_sync(kAll, give, 1));
    }
    m = k[0];
    if constexpr (N == 4) m = fmaxf(lane & 2 ? k[1] : k[0], __shfl_xor_sync(kAll, lane & 2 ? k[0] : k[1], 2));
  }
#pragma unroll
  for (int o = N; o < W; o <<= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
  return m;
}

// The 8-bit copies of N consecutive pieces of a row by the blockwise recipe's rule, codes
// satRNE(v FMAX / amax) and multiplier 1 / (FMAX / amax) per 128 columns.  q: the lane's first
// code of the first piece; s: the multiplier of the lane's group there; left: as for that piece.
// Each lane makes the two divisions of one piece only (lane % N) and has the others' scales from
// its neighbours: the divisions would otherwise be a third of the copy's instructions.
template <typename P, int N>
__device__ __forceinline__ void store_copies(uint8_t* q, float* s, int lane, int left, bool e5m2, const float (&v)[N][P::E]) {
  float a[N];
#pragma unroll
  for (int i = 0; i < N; ++i) a[i] = P::amax(v[i], left - i * P::WC);
  const float mine = scale_from_amax(group_max<N, P::kGroupLanes>(a, lane), fmax_of(e5m2));
  const float inv = recip_rn(mine);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    // lane i of the group, if the group's first column is in the row
    if (lane % P::kGroupLanes == i && left + P::first(i) > i * P::WC) s[i * (P::WC / 128)] = inv;
    const float sc = N == 1 ? mine : __shfl_sync(0xFFFFFFFFu, mine, (lane & ~(N - 1)) | i);
    if (e5m2)
      P::template encode<true>(q + i * P::WC, left - i * P::WC, v[i], sc);
    else
      P::template encode<false>(q + i * P::WC, left - i * P::WC, v[i], sc);
  }
}

// Pieces (rows x pieces of a row) shared out over all warps: piece `at`, `at` + stride, ...
// advanced without a division a step.
struct Walk {
  int64_t row, piece, row_step, piece_step, per_row;
  __device__ Walk(int64_t at, int64_t stride, int64_t pieces) : per_row(pieces) {
    row = at / pieces;
    piece = at - row * pieces;
    row_step = stride / pieces;
    piece_step = stride - row_step * pieces;
  }
  __device__ void next() {
    row += row_step;
    piece += piece_step;
    if (piece >= per_row) {
      piece -= per_row;
      ++row;
    }
  }
};

// Whether a [rows, cols] matrix of `size`-byte elements, row stride ld, takes accesses of
// `bytes` bytes throughout (null matrices do).
inline bool takes(const void* p, int64_t ld, int64_t cols, int64_t size, int64_t bytes) {
  return p == nullptr || (reinterpret_cast<uintptr_t>(p) % bytes == 0 && ld * size % bytes == 0 && cols * size % bytes == 0);
}

}  // namespace fp8q
