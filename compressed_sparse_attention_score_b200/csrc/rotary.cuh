// Rotary positions: angles as 64-bit fractions of a turn.
#pragma once
#include "common.cuh"

namespace csa2 {

// Signed fraction of a turn, in 2^-64 turns, of pair step `step` at position p: the product wraps
// modulo 2^64, which is modulo one turn, so the angle is exact at every position.
__device__ __forceinline__ int64_t rotary_turn(uint64_t step, int64_t p) { return int64_t(step * uint64_t(p)); }

// cos and sin in fp32, for the rotation of heads: the turn rounded to fp32, an angle error of at most 2^-24 pi.  That is
// far below the rounding of bf16 heads; fp32 heads are off by up to 2^-21 of their pair's size with it.
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

// (a.x + i a.y)(b.x + i b.y), each rounding named: the same bits in every kernel.
__device__ __forceinline__ double2 turned_by(double2 a, double2 b) {
  return make_double2(__fma_rn(a.x, b.x, -__dmul_rn(a.y, b.y)), __fma_rn(a.x, b.y, __dmul_rn(a.y, b.x)));
}

// cos and sin of entry n of a cache of ratio r (position n r): those of the first of its 32 entries, turned n % 32 times by one
// entry's angle.  A run of entries has them from one to the next, and yet they are a function of n alone, wherever a chunk
// begins or a warp's run does, and the same in the append.  The first and the angle are off by (pi + 2) 2^-53 at most (the turn
// rounded, sincospi's two units in the last place), a product by three roundings more: 2^-44 in all.
struct EntryAngle {
  double2 at, by;
  uint64_t step;
  int r;
  __device__ __forceinline__ EntryAngle(uint64_t step, int r) : by(rotary_cs64(step, r)), step(step), r(r) {}
  __device__ __forceinline__ void first(int64_t n) { at = rotary_cs64(step, (n & ~int64_t(31)) * r); }
  __device__ __forceinline__ void start(int64_t n) {
    first(n);
    for (int k = int(n & 31); k > 0; --k) at = turned_by(at, by);
  }
  // from entry n - 1 to n
  __device__ __forceinline__ void next(int64_t n) {
    if (n & 31) at = turned_by(at, by);
    else first(n);
  }
};

// Dims (from the head's start) of pair i.
__device__ __forceinline__ int rotary_dim0(const csa2_rotary &r, int i) {
  return r.first + (r.layout == CSA2_ROTARY_HALF ? i : 2 * i);
}
__device__ __forceinline__ int rotary_dim1(const csa2_rotary &r, int i) {
  return r.first + (r.layout == CSA2_ROTARY_HALF ? i + r.rot_dim / 2 : 2 * i + 1);
}

}  // namespace csa2
