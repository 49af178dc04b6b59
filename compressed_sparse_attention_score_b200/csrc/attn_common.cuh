// Pieces that the attention kernels share: operand layouts in shared memory, the query's prescale,
// reductions over lanes.
#pragma once
#include "common.cuh"

namespace csa2 {

// Offsets inside the swizzled operand layouts (bytes).
// K-major, 128-byte rows, 1 KB atoms of 8 rows: 16-byte unit u of row r.
__device__ __forceinline__ int kmaj128(int r, int u) { return (r >> 3) * 1024 + (r & 7) * 128 + ((u ^ (r & 7)) << 4); }
// MN-major, 128-byte swizzle: element block (m / 64) at LBO 8192, K-row k: unit u of 8 M-elements.
__device__ __forceinline__ int mnmaj128(int k, int mblk, int u) {
  return mblk * 8192 + (k >> 3) * 1024 + (k & 7) * 128 + ((u ^ (k & 7)) << 4);
}
// MN-major, 64-byte swizzle (P^T): K-row k (key), unit u of 8 heads.
__device__ __forceinline__ int mnmaj64(int k, int u) { return (k >> 3) * 512 + (k & 7) * 64 + ((u ^ ((k & 7) >> 1)) << 4); }

// Exponent s of the prescale of a head whose largest |bf16| bit pattern is mb (0 for an all-zero
// or non-finite head).  floor(log2 max) = E - 127 for the biased exponent E.
__device__ __forceinline__ int query_prescale_exp(uint32_t mb) {
  const int E = int(mb >> 7);
  if (mb == 0 || E >= 255) return 0;
  return min(126, 141 - max(E, 1));
}
// Max or sum over the 32 lanes of each of 32 per-lane values: afterwards lane l
// holds the reduction of value index l.  31 shuffles (reduce-scatter butterfly).
template <bool MAX>
__device__ __forceinline__ float reduce_scatter32(float (&v)[32]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int width = 16; width >= 1; width >>= 1) {
    const bool upper = lane & width;
#pragma unroll
    for (int i = 0; i < width; ++i) {
      // keep the half selected by this lane's bit, send the other half
      const float send = upper ? v[i] : v[i + width];
      const float keep = upper ? v[i + width] : v[i];
      const float got = __shfl_xor_sync(0xffffffffu, send, width);
      v[i] = MAX ? fmaxf(keep, got) : keep + got;
    }
  }
  return v[0];
}

}  // namespace csa2
