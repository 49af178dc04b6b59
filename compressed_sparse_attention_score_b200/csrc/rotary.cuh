// Rotary positions: angles as 64-bit fractions of a turn.
#pragma once
#include "common.cuh"

namespace csa2 {

// Signed fraction of a turn, in 2^-64 turns, of pair step `step` at position p: the product wraps
// modulo 2^64, which is modulo one turn, so the angle is exact at every position.
__device__ __forceinline__ int64_t rotary_turn(uint64_t step, int64_t p) { return int64_t(step * uint64_t(p)); }

// cos and sin in fp32: the turn rounded to fp32 (an angle error of at most 2^-24 pi) for the rotation of
// bf16 and fp32 heads, whose own rounding is as coarse or coarser.
__device__ __forceinline__ float2 rotary_cs32(uint64_t step, int64_t p) {
  float c, s;
  sincospif(float(rotary_turn(step, p)) * 0x1p-63f, &s, &c);
  return make_float2(c, s);
}

// cos and sin in fp64, for values that are quantised next: an fp32 rotation would leave the codes of
// values next to a rounding border to the last bit of sin and cos.
__device__ __forceinline__ double2 rotary_cs64(uint64_t step, int64_t p) {
  double c, s;
  sincospi(double(rotary_turn(step, p)) * 0x1p-63, &s, &c);
  return make_double2(c, s);
}

// Dims (from the head's start) of pair i.
__device__ __forceinline__ int rotary_dim0(const csa2_rotary &r, int i) {
  return r.first + (r.layout == CSA2_ROTARY_HALF ? i : 2 * i);
}
__device__ __forceinline__ int rotary_dim1(const csa2_rotary &r, int i) {
  return r.first + (r.layout == CSA2_ROTARY_HALF ? i + r.rot_dim / 2 : 2 * i + 1);
}

}  // namespace csa2
