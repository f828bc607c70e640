// rowops.cuh -- device helpers of the operators that work on rows of a matrix (layer norm,
// gated activation, expert dispatch): element loads and stores of either data type, block
// sums, and the 8-bit copy of 128 consecutive columns of a row.
//
// bf16 elements are held as their 16-bit patterns; all arithmetic is binary32.
#pragma once
#include <cstdint>

#include "ptx.cuh"
#include "recipes.cuh"

namespace fp8q {

__device__ __forceinline__ float ld_elem(const uint16_t* p) { return __uint_as_float(static_cast<uint32_t>(*p) << 16); }
__device__ __forceinline__ float ld_elem(const float* p) { return *p; }
// a parameter vector (weight, bias) of either type
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
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
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

// ------------------------------------------------------------------ a warp's piece of a row
// How a warp holds WC consecutive columns of a row, E values a lane.
//   VECTOR      lane l holds E = 16 bytes' worth of consecutive columns: one 16-byte access a
//               lane.  Needs a 16-byte aligned row and cols % E == 0 (a lane is all in or all out).
//   otherwise   lane l holds columns l, l + 32, l + 64, l + 96: consecutive lanes on consecutive
//               columns, so any element alignment coalesces.
// 128-column groups (the 8-bit copy's) never cross lanes' bounds: kGroupLanes lanes hold one.
template <typename T, bool VECTOR>
struct Piece {
  static constexpr int E = VECTOR ? 16 / static_cast<int>(sizeof(T)) : 4;
  static constexpr int WC = 32 * E;
  static constexpr int kGroupLanes = 128 / E;

  __device__ static __forceinline__ int col(int c0, int lane, int i) {
    return VECTOR ? c0 + lane * E + i : c0 + lane + 32 * i;
  }
  // v = the row's values, 0 past its end
  __device__ static __forceinline__ void load(const T* row, int c0, int lane, int cols, float (&v)[E]) {
    if constexpr (VECTOR) {
      uint4 w = make_uint4(0u, 0u, 0u, 0u);
      if (col(c0, lane, 0) < cols) w = __ldg(reinterpret_cast<const uint4*>(row + col(c0, lane, 0)));
      unpack(w, v);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) v[i] = col(c0, lane, i) < cols ? ld_elem(row + col(c0, lane, i)) : 0.0f;
    }
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
  __device__ static __forceinline__ void store(T* row, int c0, int lane, int cols, const float (&v)[E]) {
    if constexpr (VECTOR) {
      if (col(c0, lane, 0) >= cols) return;
      uint32_t u[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 2)
          u[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
        else
          u[i] = __float_as_uint(v[i]);
      }
      *reinterpret_cast<uint4*>(row + col(c0, lane, 0)) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (col(c0, lane, i) < cols) st_elem(row + col(c0, lane, i), v[i]);
    }
  }
  // The 8-bit copy of the piece by the blockwise recipe's rule: codes = satRNE(v FMAX / amax),
  // multiplier 1 / (FMAX / amax), per 128 columns.  v = 0 past the row's end.
  __device__ static __forceinline__ void store_codes(uint8_t* q_row, float* s_row, int c0, int lane, int cols, bool e5m2,
                                                     const float (&v)[E]) {
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) a = fmaxf(a, fabsf(v[i]));   // a NaN operand is ignored
#pragma unroll
    for (int o = kGroupLanes / 2; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
    const float sc = scale_from_amax(a, fmax_of(e5m2));
    if constexpr (VECTOR) {
      if (col(c0, lane, 0) >= cols) return;
      uint32_t u[E / 4];
#pragma unroll
      for (int i = 0; i < E / 4; ++i)
        u[i] = cvt_pair(__fmul_rn(v[4 * i], sc), __fmul_rn(v[4 * i + 1], sc), e5m2) |
               cvt_pair(__fmul_rn(v[4 * i + 2], sc), __fmul_rn(v[4 * i + 3], sc), e5m2) << 16;
      if constexpr (E == 8)
        *reinterpret_cast<uint2*>(q_row + col(c0, lane, 0)) = make_uint2(u[0], u[1]);
      else
        *reinterpret_cast<uint32_t*>(q_row + col(c0, lane, 0)) = u[0];
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (col(c0, lane, i) < cols)
          q_row[col(c0, lane, i)] = static_cast<uint8_t>(cvt_pair(__fmul_rn(v[i], sc), 0.0f, e5m2));
    }
    if (lane % kGroupLanes == 0 && col(c0, lane, 0) < cols) s_row[col(c0, lane, 0) / 128] = recip_rn(sc);
  }
  // E consecutive codes (aligned to E bytes, in global or shared memory) times s, 0 if not `valid`
  __device__ static __forceinline__ void decode(const uint8_t* q, float s, bool valid, bool e5m2, float (&v)[E]) {
    uint32_t u[E / 4];
    if constexpr (E == 8) {
      const uint2 w = *reinterpret_cast<const uint2*>(q);
      u[0] = w.x;
      u[1] = w.y;
    } else {
      u[0] = *reinterpret_cast<const uint32_t*>(q);
    }
#pragma unroll
    for (int i = 0; i < E / 4; ++i) {
      decode_pair(u[i] & 0xFFFFu, e5m2, v[4 * i], v[4 * i + 1]);
      decode_pair(u[i] >> 16, e5m2, v[4 * i + 2], v[4 * i + 3]);
    }
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = valid ? v[i] * s : 0.0f;
  }
  // The values the codes stand for (each product rounded to binary32), 0 past the row's end.
  __device__ static __forceinline__ void load_codes(const uint8_t* q_row, const float* s_row, int c0, int lane, int cols,
                                                    bool e5m2, float (&v)[E]) {
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = 0.0f;
    if (col(c0, lane, 0) >= cols) return;
    const float s = __ldg(s_row + col(c0, lane, 0) / 128);
    if constexpr (VECTOR) {
      decode(q_row + col(c0, lane, 0), s, true, e5m2, v);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        float x = 0.0f, unused;
        if (col(c0, lane, i) < cols) decode_pair(q_row[col(c0, lane, i)], e5m2, x, unused);
        v[i] = x * s;
      }
    }
  }
};

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

// A piece of a parameter vector (`none` without one and past its end); VECTOR: 16-byte aligned.
template <typename P, bool VECTOR>
__device__ __forceinline__ void load_param(const void* v, bool f32, int c0, int lane, int cols, float none, float (&out)[P::E]) {
#pragma unroll
  for (int i = 0; i < P::E; ++i) out[i] = none;
  if (v == nullptr) return;
  if constexpr (VECTOR) {
    const int c = P::col(c0, lane, 0);
    if (c >= cols) return;
    if (f32) {
#pragma unroll
      for (int i = 0; i < P::E / 4; ++i) {
        const float4 w = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(v) + c) + i);
        out[4 * i] = w.x;
        out[4 * i + 1] = w.y;
        out[4 * i + 2] = w.z;
        out[4 * i + 3] = w.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < P::E / 4; ++i) {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(v) + c) + i);
        out[4 * i] = bf16lo(w.x);
        out[4 * i + 1] = bf16hi(w.x);
        out[4 * i + 2] = bf16lo(w.y);
        out[4 * i + 3] = bf16hi(w.y);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < P::E; ++i)
      if (P::col(c0, lane, i) < cols) out[i] = ld_param(v, f32, P::col(c0, lane, i));
  }
}

// Whether a [rows, cols] matrix of `size`-byte elements, row stride ld, takes accesses of
// `bytes` bytes throughout (null matrices do).
inline bool takes(const void* p, int64_t ld, int64_t cols, int64_t size, int64_t bytes) {
  return p == nullptr || (reinterpret_cast<uintptr_t>(p) % bytes == 0 && ld * size % bytes == 0 && cols * size % bytes == 0);
}

}  // namespace fp8q
