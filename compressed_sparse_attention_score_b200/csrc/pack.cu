// K1/K2: the compressor + packer of global KV entries and the SWA packer.
//
// Both are HBM streaming kernels: one warp per output entry (or SWA token),
// 16-byte vector loads, quantisation in registers, coalesced row stores.
#include <cuda_fp16.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.cuh"
#include "rotary.cuh"
#include "sm100.cuh"

namespace csa2 {

template <typename T>
__device__ __forceinline__ void load16(const T *p, float (&v)[16]);

template <>
__device__ __forceinline__ void load16<float>(const float *p, float (&v)[16]) {
  const float4 *q = reinterpret_cast<const float4 *>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float4 a = q[i];
    v[4 * i] = a.x, v[4 * i + 1] = a.y, v[4 * i + 2] = a.z, v[4 * i + 3] = a.w;
  }
}

template <>
__device__ __forceinline__ void load16<uint16_t>(const uint16_t *p, float (&v)[16]) {
  const uint4 *q = reinterpret_cast<const uint4 *>(p);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint4 a = q[i];
    uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
      v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  }
}

// Sixteen values as they lie in memory, and their fp32 values.
template <typename T>
struct Raw16 {
  uint4 w[sizeof(T)];  // 16 values: bf16 two words of 16 bytes, fp32 four
  uint32_t i[sizeof(T)];  // and four more
};
template <typename T>
__device__ __forceinline__ void load_raw(const T *main, const T *index, Raw16<T> &r) {
#pragma unroll
  for (int k = 0; k < int(sizeof(T)); ++k) r.w[k] = reinterpret_cast<const uint4 *>(main)[k];
  if constexpr (sizeof(T) == 2) {
    const uint2 u = *reinterpret_cast<const uint2 *>(index);
    r.i[0] = u.x, r.i[1] = u.y;
  } else {
    const uint4 u = *reinterpret_cast<const uint4 *>(index);
    r.i[0] = u.x, r.i[1] = u.y, r.i[2] = u.z, r.i[3] = u.w;
  }
}
template <typename T>
__device__ __forceinline__ float raw_value(const uint32_t *w, int k) {
  if constexpr (sizeof(T) == 4) return __uint_as_float(w[k]);
  return __uint_as_float((k & 1) ? w[k >> 1] & 0xFFFF0000u : w[k >> 1] << 16);
}
template <typename T>
__device__ __forceinline__ void raw_values(const Raw16<T> &r, float (&v)[16], float (&vi)[4]) {
#pragma unroll
  for (int k = 0; k < 16; ++k) v[k] = raw_value<T>(&r.w[0].x, k);
#pragma unroll
  for (int k = 0; k < 4; ++k) vi[k] = raw_value<T>(r.i, k);
}

template <typename T>
__device__ __forceinline__ void load4(const T *p, float (&v)[4]);
template <>
__device__ __forceinline__ void load4<float>(const float *p, float (&v)[4]) {
  float4 a = *reinterpret_cast<const float4 *>(p);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
}
template <>
__device__ __forceinline__ void load4<uint16_t>(const uint16_t *p, float (&v)[4]) {
  uint2 a = *reinterpret_cast<const uint2 *>(p);
  v[0] = __uint_as_float(a.x << 16), v[1] = __uint_as_float(a.x & 0xFFFF0000u);
  v[2] = __uint_as_float(a.y << 16), v[3] = __uint_as_float(a.y & 0xFFFF0000u);
}

// Two bf16 values of two e2m1 codes (one byte, low nibble first) times a scale: s16, an fp16 pair, and `after`, a power of
// two.  At most six significant bits, so exact in fp16 and in bf16.
__device__ __forceinline__ uint32_t hat2(uint32_t byte, uint32_t s16, float after) {
  const uint32_t h = sm100::hmul2_u32(sm100::cvt_e2m1x2_f16x2(byte), s16);
  const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
  return __byte_perm(__float_as_uint(f.x * after), __float_as_uint(f.y * after), 0x7632);
}
// Eight of them.  (For E4M3 scales the fp16 products are multiples of 2^-10 up to 2688.)
__device__ __forceinline__ uint4 hat8(uint32_t codes, uint32_t s16) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(codes));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t v = sm100::hmul2_u32(h[i], s16);
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&v));
    h[i] = __byte_perm(__float_as_uint(f.x), __float_as_uint(f.y), 0x7632);
  }
  return make_uint4(h[0], h[1], h[2], h[3]);
}

// x / s rounded to nearest, for r within an ulp of 1 / s and results and remainders in normal range: an estimate corrected
// by its exact remainder.  The corrected value is within 2^-21 ulp of the quotient before it is rounded; where s has few
// significant bits (E4M3: four; 6: two) no quotient is that close to the middle of two numbers (at least 1/30 ulp: the distance is a
// multiple of 1 / 2 s in units of the numbers' last places), so one correction is enough.  __fdiv_rn, which takes every
// case, is three times as long.
__device__ __forceinline__ float quotient(float x, float s, float r) {
  const float q = __fmul_rn(x, r);
  return __fmaf_rn(__fmaf_rn(-q, s, x), r, q);
}
// 1 / s within an ulp.
__device__ __forceinline__ float rcp_estimate(float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return r;
}
// Two quotients by packed operations, half the instructions.
__device__ __forceinline__ void quotient2(const float *x, float s, float r, float *q) {
  asm("{\n\t.reg .b64 x, r, s, q, e;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 r, {%4, %4};\n\tmov.b64 s, {%5, %5};\n\t"
      "mul.rn.f32x2 q, x, r;\n\tfma.rn.f32x2 e, q, s, x;\n\tfma.rn.f32x2 q, e, r, q;\n\t"
      "mov.b64 {%0, %1}, q;\n\t}"
      : "=f"(q[0]), "=f"(q[1])
      : "f"(x[0]), "f"(x[1]), "f"(r), "f"(-s));
}
// The same for any s: the second correction starts from an estimate within one ulp, from which q + r (x - s q) is the
// rounded quotient (Markstein, "Computation of elementary functions on the IBM RISC System/6000 processor", 1990).
__device__ __forceinline__ float quotient_any(float x, float s, float r) {
  const float q = quotient(x, s, r);
  return __fmaf_rn(__fmaf_rn(-q, s, x), r, q);
}

// e2m1 codes of eight values divided by s: a zero result is code 0 whatever its sign (the conversion keeps the sign).
// The values are finite.
__device__ __forceinline__ uint32_t codes8(const float *x, float s, float r) {
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; i += 2) quotient2(x + i, s, r, q + i);
  uint32_t w;  // (the conversion puts its first operand in the high nibble)
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(w)
      : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
  const uint32_t m = (w | (w >> 1) | (w >> 2)) & 0x11111111u;  // nibbles with a magnitude
  return w & (0x77777777u | (m << 3));
}

// max(|a|, |b|, |c|), NaN if one is.
__device__ __forceinline__ float max_abs_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Quantise the pooled entry a warp holds (lane l: main values [16l, 16l+16), one E4M3 block,
// and indexer values [4l, 4l+4), eight lanes per E8M0 block) and store it at `slot`.
// With kv_hat / ix_hat (rows of 512 and 128 bf16) the values that the codes stand for are stored too.
__device__ __forceinline__ void store_entry(const float (&x)[16], const float (&xi)[4], int64_t slot,
                                            const csa2_cache &c, int lane, uint16_t *kv_hat = nullptr,
                                            uint16_t *ix_hat = nullptr) {
  float amax = 0.f, am = 0.f;  // (NaN if a value is)
#pragma unroll
  for (int i = 0; i < 16; i += 2) amax = max_abs_nan(amax, x[i], x[i + 1]);
#pragma unroll
  for (int i = 0; i < 4; i += 2) am = max_abs_nan(am, xi[i], xi[i + 1]);
  // values that are not finite, or nearly not, take the general divisions
  const bool special = __any_sync(0xffffffffu, !(amax < 0x1p126f) || !(am < 0x1p126f));
  if (special) {
    amax = am = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(x[i]));
#pragma unroll
    for (int i = 0; i < 4; ++i) am = fmaxf(am, fabsf(xi[i]));
  }
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));

  // Main KV: E4M3 scale per 16 values, e2m1 codes; indexer key: E8M0 exponent per 32 values (8 lanes), e2m1 codes.
  uint32_t sc, s16, lo, hi, code4;
  int ex;
  auto scale = [&](float q) {
    sc = e4m3_code(q);
    s16 = sm100::cvt_e4m3x2_f16x2(sc * 0x101u);
    return __half2float(__ushort_as_half(uint16_t(s16)));
  };
  if (special) {
    const float s = scale(__fdiv_rn(amax, 6.0f));
    lo = hi = code4 = 0;
    if (s != 0.f) {
#pragma unroll
      for (int i = 0; i < 8; ++i) lo |= e2m1_code(__fdiv_rn(x[i], s)) << (4 * i);
#pragma unroll
      for (int i = 0; i < 8; ++i) hi |= e2m1_code(__fdiv_rn(x[8 + i], s)) << (4 * i);
    }
    ex = -127;
    if (am != 0.f) {
      ex = e8m0_ceil_exponent(__fdiv_rn(am, 6.0f));
      const float si = pow2f(ex);
#pragma unroll
      for (int i = 0; i < 4; ++i) code4 |= e2m1_code(__fdiv_rn(xi[i], si)) << (4 * i);
    }
  } else {
    // (below 2^-100 the estimate's last bits may be off, but the code is 0 either way)
    const float s = scale(quotient(amax, 6.0f, 1.0f / 6.0f));
    // (a quotient below 2^-126 is code 0 whatever its last bits; a scale of 0 leaves none)
    const float r = rcp_estimate(s);
    lo = codes8(x, s, r), hi = codes8(x + 8, s, r);
    if (s == 0.f) lo = hi = 0;
    // 2^ex >= am / 6 is 1.5 x 2^(ex + 2) >= am, which the bits of am tell, down to where the quotient would be subnormal
    ex = int((__float_as_uint(am) + 0x3FFFFFu) >> 23) - 129;
    if (am < 0x1p-120f) ex = e8m0_ceil_exponent(__fdiv_rn(am, 6.0f));  // (-127 for 0)
    const float by = pow2f(-ex);  // (a power of two: the product is the quotient)
    code4 = sm100::e2m1x2_code(xi[0] * by, xi[1] * by) | sm100::e2m1x2_code(xi[2] * by, xi[3] * by) << 8;
    code4 &= 0x7777u | ((code4 | (code4 >> 1) | (code4 >> 2)) & 0x1111u) << 3;
  }
  reinterpret_cast<uint2 *>(c.kv_codes + slot * CSA2_MAIN_CODE_BYTES)[lane] = make_uint2(lo, hi);
  c.kv_scales[slot * CSA2_MAIN_SCALE_BYTES + lane] = uint8_t(sc);
  reinterpret_cast<uint16_t *>(c.ix_codes + slot * CSA2_IX_CODE_BYTES)[lane] = uint16_t(code4);
  if ((lane & 7) == 0) c.ix_scales[slot * CSA2_IX_SCALE_BYTES + (lane >> 3)] = uint8_t(ex + 127);
  if (kv_hat) {
    reinterpret_cast<uint4 *>(kv_hat)[2 * lane] = hat8(lo, s16);
    reinterpret_cast<uint4 *>(kv_hat)[2 * lane + 1] = hat8(hi, s16);
  }
  if (ix_hat) {
    const float si = pow2f(ex);
    reinterpret_cast<uint2 *>(ix_hat)[lane] = make_uint2(hat2(code4 & 0xFF, 0x3C003C00u, si), hat2(code4 >> 8, 0x3C003C00u, si));
  }
}

// What the rotating writers add to the plain ones.
struct RotaryWrite {
  csa2_rotary kv, ix;  // rot_dim 0: not turned
  bool same;           // both use one table and turn as many dims: one sine and cosine serve both
  bool runs;           // at most 32 pairs of one table: pack_run_kernel's entries, whose angles are formed in groups
  uint16_t *kv_hat, *ix_hat;
};

// Main value d of the row that a warp keeps in shared memory to turn it: four floats of padding
// after every 16, so that the lanes' 16-value pieces start in different banks.
__device__ __forceinline__ int turn_at(int d) { return d + 4 * (d >> 4); }
constexpr int TURN_MAIN = D + 4 * (D / 16), TURN_ROW = TURN_MAIN + DI;

// Pair (a, b) turned in fp64 and rounded once to fp32.
__device__ __forceinline__ void turn_pair(float &a, float &b, double2 cs, float scale) {
  const double2 v = turned_by(make_double2(a, b), cs);
  a = float(__dmul_rn(v.x, scale));
  b = float(__dmul_rn(v.y, scale));
}

// Turn the values a warp holds (x: main, lane l 16l ..; xi: indexer, lane l 4l .., or none) through the warp's row `buf` of
// shared memory: turn_pairs(kv or ix, its part of the row) turns the pairs in place there.
template <bool IX, typename F>
__device__ __forceinline__ void turn_through(float (&x)[16], float (&xi)[4], bool main, bool index, float *buf, int lane,
                                             F &&turn_pairs) {
  __syncwarp();  // the row's previous use is over
  if (main) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<float4 *>(buf + turn_at(16 * lane) + 4 * i) =
          make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
  }
  if (IX && index) *reinterpret_cast<float4 *>(buf + TURN_MAIN + 4 * lane) = make_float4(xi[0], xi[1], xi[2], xi[3]);
  __syncwarp();
  turn_pairs();
  __syncwarp();
  if (main) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 v = *reinterpret_cast<const float4 *>(buf + turn_at(16 * lane) + 4 * i);
      x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
    }
  }
  if (IX && index) {
    const float4 v = *reinterpret_cast<const float4 *>(buf + TURN_MAIN + 4 * lane);
    xi[0] = v.x, xi[1] = v.y, xi[2] = v.z, xi[3] = v.w;
  }
}
__device__ __forceinline__ void turn_main(const csa2_rotary &kv, int i, double2 cs, float *buf) {
  turn_pair(buf[turn_at(rotary_dim0(kv, i))], buf[turn_at(rotary_dim1(kv, i))], cs, kv.scale);
}
__device__ __forceinline__ void turn_index(const csa2_rotary &ix, int i, double2 cs, float *buf) {
  turn_pair(buf[TURN_MAIN + rotary_dim0(ix, i)], buf[TURN_MAIN + rotary_dim1(ix, i)], cs, ix.scale);
}

// At position pos, one pair per lane and step.  `runs`: entry n of a cache of ratio r, with the angles of pack_run_kernel.
template <bool IX>
__device__ __forceinline__ void turn_values(float (&x)[16], float (&xi)[4], const csa2_rotary &kv, const csa2_rotary &ix,
                                            bool same, int64_t pos, float *buf, int lane, bool runs = false, int64_t n = 0,
                                            int r = 1) {
  turn_through<IX>(x, xi, kv.rot_dim != 0, ix.rot_dim != 0, buf, lane, [&]() {
    if (IX && runs) {
      if (lane >= max(kv.rot_dim, ix.rot_dim) / 2) return;
      const uint64_t step = (kv.rot_dim ? kv.step : ix.step)[lane];
      EntryAngle angle(step, r);
      angle.start(n);
      if (kv.rot_dim) turn_main(kv, lane, angle.at, buf);
      if (ix.rot_dim) turn_index(ix, lane, angle.at, buf);
      return;
    }
    for (int i = lane; i < kv.rot_dim / 2; i += 32) {
      const double2 cs = rotary_cs64(kv.step[i], pos);
      turn_main(kv, i, cs, buf);
      if (IX && same) turn_index(ix, i, cs, buf);
    }
    if (IX && !same)
      for (int i = lane; i < ix.rot_dim / 2; i += 32) turn_index(ix, i, rotary_cs64(ix.step[i], pos), buf);
  });
}

// exp(x) from a fixed sequence of fp32 operations (so that the gated compressor's weights,
// and through them the quantised codes, do not depend on a math library): t = x log2(e),
// n = rint(t), f = t - n, 2^f = e^(f ln 2) by its Taylor polynomial of degree 7 (Horner,
// each product and sum rounded), times 2^n; 0 below 2^-126, inf above 2^127.  The
// coefficients are (ln 2)^i / i! rounded to fp32.
__device__ __forceinline__ float exp_fixed(float x) {
  constexpr float c[8] = {0x1.0p+0f,      0x1.62e430p-1f,  0x1.ebfbe0p-3f,  0x1.c6b08ep-5f,
                          0x1.3b2ab6p-7f, 0x1.5d87fep-10f, 0x1.430912p-13f, 0x1.ffcbfcp-17f};
  const float t = __fmul_rn(x, 0x1.715476p+0f);
  const float n = rintf(t);
  const float f = __fsub_rn(t, n);
  float p = c[7];
#pragma unroll
  for (int i = 6; i >= 0; --i) p = __fadd_rn(__fmul_rn(p, f), c[i]);
  if (n < -126.f) return 0.f;
  if (n > 127.f) return INFINITY;
  return __fmul_rn(p, __int_as_float((int(n) + 127) << 23));
}

// One warp per new entry.  Lane l owns main values [16l, 16l+16) (one E4M3 block)
// and indexer values [4l, 4l+4) (eight lanes per E8M0 block).  Pooling: pool_w per token
// (or fp32(1/r)), or with gate_kv / gate_ix the gated sum: per channel the softmax over the
// entry's r tokens of the gate logits (max subtracted, exp_fixed, sum left to right, fp32
// division) weights the tokens, summed left to right.
// ROT: the entry is turned at its first token's position between pooling and quantisation.  GATED: a kernel of its own,
// since its registers would halve the others' occupancy.
template <typename T, bool ROT, bool GATED>
__global__ void __launch_bounds__(256) pack_kv_kernel(const T *__restrict__ lat_kv,
                                                      const T *__restrict__ lat_ix,
                                                      const float *__restrict__ pool_w,
                                                      const float *__restrict__ gate_kv,
                                                      const float *__restrict__ gate_ix, int B, int T_,
                                                      const int32_t *__restrict__ first_entry,
                                                      csa2_cache c, RotaryWrite rw, int32_t *err) {
  const int lane = threadIdx.x & 31;
  __shared__ __align__(16) float turn_buf[ROT ? 8 : 1][ROT ? TURN_ROW : 1];
  const int n_new = T_ / c.ratio;
  const int64_t e = int64_t(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (e >= int64_t(B) * n_new) return;
  const int b = int(e / n_new), j = int(e % n_new);
  const int64_t n = int64_t(first_entry[b]) + j, slot = cache_slot<false>(c, b, n);
  if (slot < 0) {
    if (lane == 0) report(err, CSA2_ERR_INDEX);
    return;
  }
  float x[16], xi[4];
  const int64_t tok0 = int64_t(b) * T_ + int64_t(j) * c.ratio;
  auto finish = [&]() {
    if constexpr (ROT) {
      turn_values<true>(x, xi, rw.kv, rw.ix, rw.same, n * c.ratio, turn_buf[threadIdx.x >> 5], lane);
      store_entry(x, xi, slot, c, lane, rw.kv_hat ? rw.kv_hat + e * D : nullptr,
                  rw.ix_hat ? rw.ix_hat + e * DI : nullptr);
    } else {
      store_entry(x, xi, slot, c, lane);
    }
  };

  if constexpr (GATED) {
    // ---- gated sum: three passes over the group (max, normaliser, weighted sum)
    float m[16], mi[4], den[16], deni[4];
    for (int t = 0; t < c.ratio; ++t) {
      float g[16], gi[4];
      load16<float>(gate_kv + (tok0 + t) * D + 16 * lane, g);
      load4<float>(gate_ix + (tok0 + t) * DI + 4 * lane, gi);
#pragma unroll
      for (int i = 0; i < 16; ++i) m[i] = t == 0 ? g[i] : fmaxf(m[i], g[i]);
#pragma unroll
      for (int i = 0; i < 4; ++i) mi[i] = t == 0 ? gi[i] : fmaxf(mi[i], gi[i]);
    }
    for (int t = 0; t < c.ratio; ++t) {
      float g[16], gi[4];
      load16<float>(gate_kv + (tok0 + t) * D + 16 * lane, g);
      load4<float>(gate_ix + (tok0 + t) * DI + 4 * lane, gi);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float ev = exp_fixed(__fsub_rn(g[i], m[i]));
        den[i] = t == 0 ? ev : __fadd_rn(den[i], ev);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float ev = exp_fixed(__fsub_rn(gi[i], mi[i]));
        deni[i] = t == 0 ? ev : __fadd_rn(deni[i], ev);
      }
    }
    for (int t = 0; t < c.ratio; ++t) {
      float g[16], gi[4], v[16], vi[4];
      load16<float>(gate_kv + (tok0 + t) * D + 16 * lane, g);
      load4<float>(gate_ix + (tok0 + t) * DI + 4 * lane, gi);
      load16<T>(lat_kv + (tok0 + t) * D + 16 * lane, v);
      load4<T>(lat_ix + (tok0 + t) * DI + 4 * lane, vi);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float term = __fmul_rn(__fdiv_rn(exp_fixed(__fsub_rn(g[i], m[i])), den[i]), v[i]);
        x[i] = t == 0 ? term : __fadd_rn(x[i], term);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float term = __fmul_rn(__fdiv_rn(exp_fixed(__fsub_rn(gi[i], mi[i])), deni[i]), vi[i]);
        xi[i] = t == 0 ? term : __fadd_rn(xi[i], term);
      }
    }
  } else {
    // ---- pool the tokens of this entry (fp32, left to right, no fused multiply-add)
    const float w_default = __fdiv_rn(1.0f, float(c.ratio));
    for (int t = 0; t < c.ratio; ++t) {
      const float wt = pool_w ? pool_w[tok0 + t] : w_default;
      float v[16], vi[4];
      load16<T>(lat_kv + (tok0 + t) * D + 16 * lane, v);
      load4<T>(lat_ix + (tok0 + t) * DI + 4 * lane, vi);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = t == 0 ? __fmul_rn(wt, v[i]) : __fadd_rn(x[i], __fmul_rn(wt, v[i]));
#pragma unroll
      for (int i = 0; i < 4; ++i) xi[i] = t == 0 ? __fmul_rn(wt, vi[i]) : __fadd_rn(xi[i], __fmul_rn(wt, vi[i]));
    }
  }
  finish();
}

// The rotating pack of a chunk whose main and indexer values share one table of at most 32 pairs: a warp takes `run`
// consecutive entries (lanes as in pack_kv_kernel; lane l turns pair l), so that a sine and cosine in fp64 serve 32 of them
// (EntryAngle), and asks for the next entry's first token before it quantises this one.  Bound by its 442 instructions a warp and
// entry, which fill 68 % of the issue slots, and by the latencies that 24 warps an SM leave uncovered (fixed ones, and the
// turned values' way through shared memory): 131288 bf16 tokens, r = 1, with the values stored, 80 us (73 % of the copy
// rate); 64000 fp32 tokens 50 us.  Other rotations (two tables, even of equal content, or more than 64 dims) are
// pack_kv_kernel's: with two tables 136 us, with 128 turned dims 143, gated 426.  Blocks are as many as leave
// registers enough: with 64 a thread, 32 warps an SM, a few spilled values made it 99 us (fp32, 80 a thread: 65 us).
constexpr int64_t PACK_RUN = 64;  // entries that a warp takes at most
template <typename T>
constexpr int PACK_WARPS = sizeof(T) == 2 ? 8 : 4;  // of a block
template <typename T>
constexpr int PACK_BLOCKS = sizeof(T) == 2 ? 3 : 5;  // on an SM
template <typename T>
__global__ void __launch_bounds__(32 * PACK_WARPS<T>, PACK_BLOCKS<T>)
    pack_run_kernel(const T *__restrict__ lat_kv, const T *__restrict__ lat_ix, const float *__restrict__ pool_w, int T_,
                    int n_new, int64_t all, int run, const int32_t *__restrict__ first_entry, csa2_cache c, RotaryWrite rw,
                    int32_t *err) {
  __shared__ __align__(16) float turn_buf[PACK_WARPS<T>][TURN_ROW];
  const int lane = threadIdx.x & 31, r = c.ratio;
  float *buf = turn_buf[threadIdx.x >> 5];
  int64_t e = (int64_t(blockIdx.x) * PACK_WARPS<T> + (threadIdx.x >> 5)) * run;
  int left = int(min(int64_t(run), all - e));
  if (left <= 0) return;
  int b = int(e / n_new), j = int(e % n_new);
  const bool turns = lane < max(rw.kv.rot_dim, rw.ix.rot_dim) / 2;
  const uint64_t step = turns ? (rw.kv.rot_dim ? rw.kv.step : rw.ix.step)[lane] : 0;
  const bool one = r == 1 && !pool_w;  // the entry is its token
  const float w_default = __fdiv_rn(1.0f, float(r));
  Raw16<T> raw;
  auto load = [&](int64_t tok) { load_raw(lat_kv + tok * D + 16 * lane, lat_ix + tok * DI + 4 * lane, raw); };
  load(int64_t(b) * T_ + int64_t(j) * r);
  int64_t first = first_entry[b];
  EntryAngle angle(step, r);
  bool fresh = true;
  for (; left > 0; --left, ++e) {
    const int64_t n = first + j, slot = cache_slot<false>(c, b, n);
    float x[16], xi[4];
    raw_values(raw, x, xi);
    if (!one) {
      const int64_t tok0 = int64_t(b) * T_ + int64_t(j) * r;
      const float w0 = pool_w ? pool_w[tok0] : w_default;
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = __fmul_rn(w0, x[i]);
#pragma unroll
      for (int i = 0; i < 4; ++i) xi[i] = __fmul_rn(w0, xi[i]);
      for (int t = 1; t < r; ++t) {
        const float wt = pool_w ? pool_w[tok0 + t] : w_default;
        load(tok0 + t);
        float v[16], vi[4];
        raw_values(raw, v, vi);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = __fadd_rn(x[i], __fmul_rn(wt, v[i]));
#pragma unroll
        for (int i = 0; i < 4; ++i) xi[i] = __fadd_rn(xi[i], __fmul_rn(wt, vi[i]));
      }
    }
    // this entry's angle; then on to the next one
    if (fresh) angle.start(n);
    else angle.next(n);
    fresh = false;
    if (++j == n_new) {
      j = 0, ++b;
      fresh = true;
    }
    if (left > 1) {
      load(int64_t(b) * T_ + int64_t(j) * r);
      if (fresh) first = first_entry[b];
    }
    turn_through<true>(x, xi, rw.kv.rot_dim != 0, rw.ix.rot_dim != 0, buf, lane, [&]() {
      if (turns) {
        if (rw.kv.rot_dim) turn_main(rw.kv, lane, angle.at, buf);
        if (rw.ix.rot_dim) turn_index(rw.ix, lane, angle.at, buf);
      }
    });
    if (slot < 0) {
      if (lane == 0) report(err, CSA2_ERR_INDEX);
    } else {
      store_entry(x, xi, slot, c, lane, rw.kv_hat ? rw.kv_hat + e * D : nullptr, rw.ix_hat ? rw.ix_hat + e * DI : nullptr);
    }
  }
}

// Decode-time append, one warp per sequence (lanes as in pack_kv_kernel).  The token at
// position pos[b] goes to the sequence's staging row pos % r (fp32: exactly the input); when
// it completes a group of r tokens, the group is pooled like pack_kv_kernel does (fp32, left to
// right, weight fp32(1/r)) into entry pos / r, which is quantised and stored, and
// num_entries[b] is raised to pos / r + 1.  Staging row t of sequence b (512 main then 128
// indexer values) starts at stage + b * stage_stride + t * 640; stage may be NULL when r = 1.
// ROT: a completed entry is turned at its first token's position before it is quantised.
template <typename T, bool ROT>
__global__ void __launch_bounds__(256) append_kv_kernel(const T *__restrict__ lat_kv, const T *__restrict__ lat_ix,
                                                        int B, const int32_t *__restrict__ pos, float *stage,
                                                        int64_t stage_stride, csa2_cache c, int32_t *num_entries,
                                                        RotaryWrite rw, int32_t *err) {
  const int lane = threadIdx.x & 31;
  __shared__ __align__(16) float turn_buf[ROT ? 8 : 1][ROT ? TURN_ROW : 1];
  const int b = int(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (b >= B) return;
  const int p = pos[b];
  if (p < 0) return;  // padding row
  const int r = c.ratio, cur = p % r;
  float v[16], vi[4];
  load16<T>(lat_kv + int64_t(b) * D + 16 * lane, v);
  load4<T>(lat_ix + int64_t(b) * DI + 4 * lane, vi);
  float *srow = stage ? stage + int64_t(b) * stage_stride : nullptr;
  if (srow && r > 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      reinterpret_cast<float4 *>(srow + cur * (D + DI) + 16 * lane)[i] =
          make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    *reinterpret_cast<float4 *>(srow + cur * (D + DI) + D + 4 * lane) = make_float4(vi[0], vi[1], vi[2], vi[3]);
  }
  if (cur != r - 1) return;  // the group is not complete yet
  const int j = p / r;
  const int64_t slot = cache_slot<!ROT>(c, b, j);
  if (slot < 0) {
    if (lane == 0) report(err, CSA2_ERR_INDEX);
    return;
  }
  if (r > 1 && !srow) {
    if (lane == 0) report(err, CSA2_ERR_SHAPE);
    return;
  }
  const float wt = __fdiv_rn(1.0f, float(r));
  float x[16], xi[4];
  for (int t = 0; t < r; ++t) {
    float u[16], ui[4];
    if (t == cur) {
#pragma unroll
      for (int i = 0; i < 16; ++i) u[i] = v[i];
#pragma unroll
      for (int i = 0; i < 4; ++i) ui[i] = vi[i];
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 f = reinterpret_cast<const float4 *>(srow + t * (D + DI) + 16 * lane)[i];
        u[4 * i] = f.x, u[4 * i + 1] = f.y, u[4 * i + 2] = f.z, u[4 * i + 3] = f.w;
      }
      const float4 f = *reinterpret_cast<const float4 *>(srow + t * (D + DI) + D + 4 * lane);
      ui[0] = f.x, ui[1] = f.y, ui[2] = f.z, ui[3] = f.w;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = t == 0 ? __fmul_rn(wt, u[i]) : __fadd_rn(x[i], __fmul_rn(wt, u[i]));
#pragma unroll
    for (int i = 0; i < 4; ++i) xi[i] = t == 0 ? __fmul_rn(wt, ui[i]) : __fadd_rn(xi[i], __fmul_rn(wt, ui[i]));
  }
  if constexpr (ROT) {
    turn_values<true>(x, xi, rw.kv, rw.ix, rw.same, int64_t(j) * r, turn_buf[threadIdx.x >> 5], lane, rw.runs, j, r);
    store_entry(x, xi, slot, c, lane, rw.kv_hat ? rw.kv_hat + int64_t(b) * D : nullptr,
                rw.ix_hat ? rw.ix_hat + int64_t(b) * DI : nullptr);
  } else {
    store_entry(x, xi, slot, c, lane);
  }
  if (lane == 0 && num_entries) atomicMax(&num_entries[b], j + 1);
}

// One warp per SWA token; lane l owns values [16l, 16l+16).  Only the last R
// tokens of a call are stored (earlier ones would be overwritten in the ring).  Ring b
// takes its positions from row b % pos_rows of pos (several layers' rings of the same
// sequences in one launch).
// ROT: the token is turned at its own position first.
template <typename T, bool ROT>
__global__ void __launch_bounds__(256) pack_swa_kernel(const T *__restrict__ x, int B, int T_,
                                                       const int32_t *__restrict__ pos, int pos_rows,
                                                       uint8_t *__restrict__ codes,
                                                       float *__restrict__ scale, int R, csa2_rotary rot,
                                                       int32_t *err) {
  const int lane = threadIdx.x & 31;
  __shared__ __align__(16) float turn_buf[ROT ? 8 : 1][ROT ? TURN_MAIN : 1];
  const int64_t e = int64_t(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (e >= int64_t(B) * T_) return;
  const int b = int(e / T_), t = int(e % T_);
  if (t < T_ - R) return;
  const int p = pos[int64_t(b % pos_rows) * T_ + t];
  if (p < 0) return;  // padding token of a ragged batch
  const int64_t slot = int64_t(b) * R + (p % R);
  float v[16];
  load16<T>(x + e * D + 16 * lane, v);
  if constexpr (ROT) {
    float none[4];
    turn_values<false>(v, none, rot, rot, false, p, turn_buf[threadIdx.x >> 5], lane);
  }
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(v[i]));
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const float s = __fdiv_rn(amax, 448.0f);
  uint32_t w[4] = {0, 0, 0, 0};
  if (s > 0x1p-60f && s < 0x1p60f) {  // (NaN values stay NaN)
    const float r = __frcp_rn(s);
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      const float2 q = make_float2(quotient_any(v[i], s, r), quotient_any(v[i + 1], s, r));
      w[i >> 2] |= uint32_t(__nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3)) << (8 * (i & 3));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)  // a zero result is code 0 whatever its sign
      w[i] &= 0x7F7F7F7Fu | (((w[i] & 0x7F7F7F7Fu) + 0x7F7F7F7Fu) & 0x80808080u);
  } else if (s != 0.f) {
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i >> 2] |= e4m3_code(__fdiv_rn(v[i], s)) << (8 * (i & 3));
  }
  reinterpret_cast<uint4 *>(codes + slot * CSA2_SWA_DIM)[lane] = make_uint4(w[0], w[1], w[2], w[3]);
  if (lane == 0) scale[slot] = s;
}

// What the rotating writers are given, as the kernels take it.
static RotaryWrite rotary_write(const csa2_rotary *kv, const csa2_rotary *ix, uint16_t *kv_hat, uint16_t *ix_hat) {
  RotaryWrite w{};
  if (kv) w.kv = *kv;
  if (ix) w.ix = *ix;
  w.same = kv && ix && kv->step == ix->step && kv->rot_dim == ix->rot_dim;
  w.runs = (w.same || !w.kv.rot_dim || !w.ix.rot_dim) && w.kv.rot_dim <= 64 && w.ix.rot_dim <= 64;
  w.kv_hat = kv_hat, w.ix_hat = ix_hat;
  return w;
}

template <typename T, bool ROT>
static void pack_kv(const void *lat_kv, const void *lat_ix, const float *pool_w, const float *gate_kv,
                    const float *gate_ix, int B, int T_, const int32_t *first_entry, const csa2_cache &c,
                    const RotaryWrite &rw, int32_t *err, cudaStream_t st) {
  const int64_t n = int64_t(B) * (T_ / c.ratio);
  if (n == 0) return;
  if (ROT && !gate_kv && rw.runs) {
    // runs of up to PACK_RUN entries, of a length that fills the device a whole number of times
    const int64_t fit = int64_t(sm_count()) * PACK_WARPS<T> * PACK_BLOCKS<T>;  // warps at once
    const int64_t rounds = (n + PACK_RUN * fit - 1) / (PACK_RUN * fit);
    const int run = int((n + rounds * fit - 1) / (rounds * fit));
    pack_run_kernel<T><<<unsigned((n + PACK_WARPS<T> * run - 1) / (PACK_WARPS<T> * run)), 32 * PACK_WARPS<T>, 0, st>>>(
        static_cast<const T *>(lat_kv), static_cast<const T *>(lat_ix), pool_w, T_, T_ / c.ratio, n, run, first_entry, c, rw, err);
    return;
  }
  const auto kernel = gate_kv ? pack_kv_kernel<T, ROT, true> : pack_kv_kernel<T, ROT, false>;
  kernel<<<unsigned((n + 7) / 8), 256, 0, st>>>(static_cast<const T *>(lat_kv), static_cast<const T *>(lat_ix), pool_w,
                                                gate_kv, gate_ix, B, T_, first_entry, c, rw, err);
}

void launch_pack_kv(const void *lat_kv, const void *lat_ix, csa2_dtype dtype, const float *pool_w,
                    const float *gate_kv, const float *gate_ix, int B, int T, const int32_t *first_entry,
                    const csa2_cache &c, int32_t *err, cudaStream_t st) {
  const auto f = dtype == CSA2_F32 ? pack_kv<float, false> : pack_kv<uint16_t, false>;
  f(lat_kv, lat_ix, pool_w, gate_kv, gate_ix, B, T, first_entry, c, RotaryWrite{}, err, st);
}

void launch_pack_kv_rotary(const void *lat_kv, const void *lat_ix, csa2_dtype dtype, const float *pool_w,
                           const float *gate_kv, const float *gate_ix, int B, int T, const int32_t *first_entry,
                           const csa2_rotary *rot_kv, const csa2_rotary *rot_ix, const csa2_cache &c, uint16_t *kv_hat,
                           uint16_t *ix_hat, int32_t *err, cudaStream_t st) {
  const auto f = dtype == CSA2_F32 ? pack_kv<float, true> : pack_kv<uint16_t, true>;
  f(lat_kv, lat_ix, pool_w, gate_kv, gate_ix, B, T, first_entry, c, rotary_write(rot_kv, rot_ix, kv_hat, ix_hat), err,
    st);
}

template <typename T, bool ROT>
static void pack_swa(const void *x, int B, int T_, const int32_t *pos, int pos_rows, uint8_t *codes, float *scale,
                     int R, const csa2_rotary &rot, int32_t *err, cudaStream_t st) {
  const int64_t n = int64_t(B) * T_;
  if (n == 0) return;
  pack_swa_kernel<T, ROT><<<unsigned((n + 7) / 8), 256, 0, st>>>(static_cast<const T *>(x), B, T_, pos, pos_rows, codes,
                                                                 scale, R, rot, err);
}

void launch_pack_swa(const void *x, csa2_dtype dtype, int B, int T, const int32_t *pos, int pos_rows,
                     uint8_t *codes, float *scale, int R, int32_t *err, cudaStream_t st) {
  const auto f = dtype == CSA2_F32 ? pack_swa<float, false> : pack_swa<uint16_t, false>;
  f(x, B, T, pos, pos_rows, codes, scale, R, csa2_rotary{}, err, st);
}

void launch_pack_swa_rotary(const void *x, csa2_dtype dtype, int B, int T, const int32_t *pos, const csa2_rotary &rot,
                            uint8_t *codes, float *scale, int R, int32_t *err, cudaStream_t st) {
  const auto f = dtype == CSA2_F32 ? pack_swa<float, true> : pack_swa<uint16_t, true>;
  f(x, B, T, pos, B, codes, scale, R, rot, err, st);
}

template <typename T, bool ROT>
static void append_kv(const void *lat_kv, const void *lat_ix, int B, const int32_t *pos, float *stage,
                      int64_t stage_stride, const csa2_cache &c, int32_t *num_entries, const RotaryWrite &rw,
                      int32_t *err, cudaStream_t st) {
  if (B == 0) return;
  append_kv_kernel<T, ROT><<<(B + 7) / 8, 256, 0, st>>>(static_cast<const T *>(lat_kv), static_cast<const T *>(lat_ix),
                                                        B, pos, stage, stage_stride, ROT ? c : divisible_pages(c), num_entries, rw, err);
}

void launch_append_kv(const void *lat_kv, const void *lat_ix, csa2_dtype dtype, int B, const int32_t *pos,
                      float *stage, int64_t stage_stride, const csa2_cache &c, int32_t *num_entries, int32_t *err,
                      cudaStream_t st) {
  const auto f = dtype == CSA2_F32 ? append_kv<float, false> : append_kv<uint16_t, false>;
  f(lat_kv, lat_ix, B, pos, stage, stage_stride, c, num_entries, RotaryWrite{}, err, st);
}

void launch_append_kv_rotary(const void *lat_kv, const void *lat_ix, csa2_dtype dtype, int B, const int32_t *pos,
                             float *stage, int64_t stage_stride, const csa2_rotary *rot_kv, const csa2_rotary *rot_ix,
                             const csa2_cache &c, int32_t *num_entries, uint16_t *kv_hat, uint16_t *ix_hat, int32_t *err,
                             cudaStream_t st) {
  const auto f = dtype == CSA2_F32 ? append_kv<float, true> : append_kv<uint16_t, true>;
  f(lat_kv, lat_ix, B, pos, stage, stage_stride, c, num_entries, rotary_write(rot_kv, rot_ix, kv_hat, ix_hat), err, st);
}

}  // namespace csa2
