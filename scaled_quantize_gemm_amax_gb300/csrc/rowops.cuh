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

// The columns of 128-column group `g` that lane `lane` of a warp holds, element i of 4:
// consecutive lanes on consecutive columns, so any element alignment coalesces.
__device__ __forceinline__ int64_t group_col(int64_t g, int lane, int i) { return g * 128 + lane + 32 * i; }

// The 8-bit copy of one group held by a warp as above: the blockwise recipe's rule,
// codes = satRNE(v * FMAX / amax), multiplier 1 / (FMAX / amax).  v = 0 past `cols`.
__device__ __forceinline__ void store_group8(const float (&v)[4], int64_t g, int lane, int64_t cols, bool e5m2, uint8_t* q_row,
                                             float* s_row) {
  float a = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) a = fmaxf(a, fabsf(v[i]));   // a NaN operand is ignored
  const float sc = scale_from_amax(warp_max(a), fmax_of(e5m2));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t c = group_col(g, lane, i);
    if (c < cols) q_row[c] = static_cast<uint8_t>(cvt_pair(__fmul_rn(v[i], sc), 0.0f, e5m2));
  }
  if (lane == 0) s_row[g] = recip_rn(sc);
}

}  // namespace fp8q
