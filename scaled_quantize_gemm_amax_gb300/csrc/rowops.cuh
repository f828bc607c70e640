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
// How a warp holds WC consecutive columns of a row, E values a lane.
//   VECTOR      lane l holds E = 16 bytes' worth of consecutive columns: one 16-byte access a
//               lane.  Needs a 16-byte aligned row and cols % E == 0 (a lane is all in or all out).
//   otherwise   lane l holds columns l, l + 32, l + 64, l + 96: consecutive lanes on consecutive
//               columns, so any element alignment coalesces.
// A lane works from its own first column, first(lane) after the piece's: pointers point there,
// and `left` is the number of columns from there to the row's end (possibly none).
// 128-column groups (the 8-bit copy's) never cross lanes' bounds: kGroupLanes lanes hold one.
template <typename T, bool VECTOR>
struct Piece {
  static constexpr bool kVector = VECTOR;
  static constexpr int E = VECTOR ? 16 / static_cast<int>(sizeof(T)) : 4;
  static constexpr int WC = 32 * E;
  static constexpr int kGroupLanes = 128 / E;
  static constexpr int kWords = E / 4;   // of codes

  __device__ static __forceinline__ int first(int lane) { return VECTOR ? lane * E : lane; }
  // column of value i after the lane's first
  __device__ static __forceinline__ constexpr int at(int i) { return VECTOR ? i : 32 * i; }
  __device__ static __forceinline__ bool has(int left, int i) { return left > (VECTOR ? 0 : 32 * i); }

  // The lane's values as loaded, four registers (0 past the row's end): what waits in registers
  // waits in this form.
  __device__ static __forceinline__ uint4 load_raw(const T* p, int left) {
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    if constexpr (VECTOR) {
      if (left > 0) w = __ldg(reinterpret_cast<const uint4*>(p));
    } else {
      if (has(left, 0)) w.x = __float_as_uint(ld_elem(p + at(0)));
      if (has(left, 1)) w.y = __float_as_uint(ld_elem(p + at(1)));
      if (has(left, 2)) w.z = __float_as_uint(ld_elem(p + at(2)));
      if (has(left, 3)) w.w = __float_as_uint(ld_elem(p + at(3)));
    }
    return w;
  }
  // v = the row's values, 0 past its end
  __device__ static __forceinline__ void load(const T* p, int left, float (&v)[E]) { unpack(load_raw(p, left), v); }
  __device__ static __forceinline__ void unpack(const uint4& w, float (&v)[E]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (VECTOR && sizeof(T) == 2) {
        v[2 * i] = bf16lo(u[i]);
        v[2 * i + 1] = bf16hi(u[i]);
      } else {
        v[i] = __uint_as_float(u[i]);
      }
    }
  }
  __device__ static __forceinline__ void store(T* p, int left, const float (&v)[E]) {
    if constexpr (VECTOR) {
      if (left <= 0) return;
      uint32_t u[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 2)
          u[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
        else
          u[i] = __float_as_uint(v[i]);
      }
      *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (has(left, i)) st_elem(p + at(i), v[i]);
    }
  }
  // The lane's part of a parameter vector (`none` without one and past its end); `c` is the
  // lane's first column, VECTOR: the vector is 16-byte aligned.
  __device__ static __forceinline__ void load_param(const void* vec, bool f32, int c, int left, float none, float (&v)[E]) {
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = none;
    if (vec == nullptr) return;
    if constexpr (VECTOR) {
      if (left <= 0) return;
      if (f32) {
#pragma unroll
        for (int i = 0; i < E / 4; ++i) {
          const float4 w = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(vec) + c) + i);
          v[4 * i] = w.x;
          v[4 * i + 1] = w.y;
          v[4 * i + 2] = w.z;
          v[4 * i + 3] = w.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < E / 4; ++i) {
          const uint2 w = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(vec) + c) + i);
          v[4 * i] = bf16lo(w.x);
          v[4 * i + 1] = bf16hi(w.x);
          v[4 * i + 2] = bf16lo(w.y);
          v[4 * i + 3] = bf16hi(w.y);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (has(left, i)) v[i] = ld_param(vec, f32, c + at(i));
    }
  }

  // ---- the 8-bit copy
  // max |v| of the lane's columns (NaN ignored)
  __device__ static __forceinline__ float amax(const float (&v)[E], int left) {
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < E; i += 2)
      a = max_abs3(a, VECTOR || has(left, i) ? v[i] : 0.0f, VECTOR || has(left, i + 1) ? v[i + 1] : 0.0f);
    return left > 0 ? a : 0.0f;
  }
  // codes = satRNE(v sc)
  template <bool E5>
  __device__ static __forceinline__ void encode(uint8_t* q, int left, const float (&v)[E], float sc) {
    uint32_t u[E / 2];
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      const float2 m = mul2(make_float2(v[2 * i], v[2 * i + 1]), both(sc));
      u[i] = E5 ? cvt_pair_e5m2(m.x, m.y) : cvt_pair_e4m3(m.x, m.y);
    }
    if constexpr (VECTOR) {
      if (left <= 0) return;
      if constexpr (E == 8)
        *reinterpret_cast<uint2*>(q) = make_uint2(__byte_perm(u[0], u[1], 0x5410), __byte_perm(u[2], u[3], 0x5410));
      else
        *reinterpret_cast<uint32_t*>(q) = __byte_perm(u[0], u[1], 0x5410);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (has(left, i)) q[at(i)] = static_cast<uint8_t>(u[i / 2] >> (8 * (i % 2)));
    }
  }
  // The codes of a lane's columns, value i in byte i % 4 of word i / 4 (0 past the row's end).
  struct Codes {
    uint32_t u[kWords];
  };
  __device__ static __forceinline__ Codes read_codes(const uint8_t* q) {   // E consecutive codes at q
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
  __device__ static __forceinline__ Codes load_codes(const uint8_t* q, int left) {
    Codes c = {};
    if constexpr (VECTOR) {
      if (left > 0) c = read_codes(q);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (has(left, i)) c.u[0] |= static_cast<uint32_t>(q[at(i)]) << (8 * i);
    }
    return c;
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
