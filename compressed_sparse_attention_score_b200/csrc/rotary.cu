// Rotary positions of heads (csa2_rotate) and the host-side table of frequencies.
#include <cmath>

#include "kernels.cuh"
#include "rotary.cuh"

namespace csa2 {
namespace {

struct RotateArgs {
  const void *x;
  void *out;
  int64_t xt, xh, ot, oh;  // strides in elements: tokens, heads
  int heads, dim;
  const int32_t *pos;
  csa2_rotary rot;
  bool inverse, in_place;
};

__device__ __forceinline__ float load1(const float *p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t *p) { return bf16_to_f32(*p); }
__device__ __forceinline__ void store1(float *p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t *p, float v) { *p = __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

// Any shape: one block per token and group of heads, one thread per dim or pair.  One value a thread and load, so far from the
// memory's rate: 8192 x 64 heads of 510 bf16, 62 turned, 752 us (1.4 TB/s in and out), 1021 x 64 x 510 fp32 105 us, 8 x 64 x
// 510 bf16 4 us.
template <typename TX, typename TO>
__global__ void __launch_bounds__(256) rotate_kernel(RotateArgs a) {
  const int64_t t = blockIdx.x;
  const int p = a.pos[t];
  if (p < 0) return;
  const int pairs = a.rot.rot_dim / 2, rest = a.in_place ? 0 : a.dim - a.rot.rot_dim;
  const TX *x = static_cast<const TX *>(a.x) + t * a.xt;
  TO *o = static_cast<TO *>(a.out) + t * a.ot;
  for (int u = threadIdx.x; u < pairs + rest; u += 256) {
    if (u < pairs) {
      float2 cs = rotary_cs32(a.rot.step[u], p);
      if (a.inverse) cs.y = -cs.y;
      const int i = rotary_dim0(a.rot, u), j = rotary_dim1(a.rot, u);
      for (int h = blockIdx.y; h < a.heads; h += gridDim.y) {
        const float v = load1(x + h * a.xh + i), w = load1(x + h * a.xh + j);
        store1(o + h * a.oh + i, (v * cs.x - w * cs.y) * a.rot.scale);
        store1(o + h * a.oh + j, (v * cs.y + w * cs.x) * a.rot.scale);
      }
    } else {
      const int d = u - pairs, i = d < a.rot.first ? d : d + a.rot.rot_dim;
      for (int h = blockIdx.y; h < a.heads; h += gridDim.y) store1(o + h * a.oh + i, load1(x + h * a.xh + i));
    }
  }
}

// Eight values of a head: bf16 in one 16-byte word, fp32 in two.
template <typename T>
struct Eight {
  uint4 w[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Eight<T> load8(const T *p) {
  Eight<T> v;
#pragma unroll
  for (int i = 0; i < int(sizeof(T) / 2); ++i) v.w[i] = reinterpret_cast<const uint4 *>(p)[i];
  return v;
}
template <typename T>
__device__ __forceinline__ void store8(T *p, const Eight<T> &v) {
#pragma unroll
  for (int i = 0; i < int(sizeof(T) / 2); ++i) reinterpret_cast<uint4 *>(p)[i] = v.w[i];
}
__device__ __forceinline__ void values8(const Eight<float> &v, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = __uint_as_float((&v.w[i >> 2].x)[i & 3]);
}
__device__ __forceinline__ void values8(const Eight<uint16_t> &v, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t w = (&v.w[0].x)[i >> 1];
    f[i] = __uint_as_float((i & 1) ? w & 0xFFFF0000u : w << 16);
  }
}
__device__ __forceinline__ void pack8(const float (&f)[8], Eight<float> &v) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    v.w[i] = make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]), __float_as_uint(f[4 * i + 2]),
                        __float_as_uint(f[4 * i + 3]));
}
__device__ __forceinline__ void pack8(const float (&f)[8], Eight<uint16_t> &v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&h);
  }
  v.w[0] = make_uint4(w[0], w[1], w[2], w[3]);
}

// Heads in units of eight values, 16-byte aligned: one block per token and `hpb` heads.  A unit is eight
// neighbouring dims, or (HALF, turned dims) eight and the eight that they are paired with.  The token's cosines and
// sines are formed once per block, in shared memory, while the first units' loads are under way; four units
// are in flight per thread.  Bound by memory: every value once in, once out (8192 x 64 heads of 512 bf16, 64 turned:
// 168 us, 98 % of the copy rate; one value a thread 752 us; 1021 x 64 x 512 fp32 to bf16 37 us, 83 %).
template <typename TX, typename TO, bool HALF>
__global__ void __launch_bounds__(256) rotate8_kernel(RotateArgs a, int hpb, int units, uint32_t magic) {
  extern __shared__ float2 table[];
  constexpr int U = sizeof(TX) == 2 && !HALF ? 4 : 2;
  const int64_t t = blockIdx.x;
  const int p = a.pos[t], h0 = blockIdx.y * hpb, all = min(hpb, a.heads - h0) * units;
  if (p < 0) return;
  const TX *x = static_cast<const TX *>(a.x) + t * a.xt + h0 * a.xh;
  TO *o = static_cast<TO *>(a.out) + t * a.ot + h0 * a.oh;
  const int pairs = a.rot.rot_dim / 2, turned = HALF ? pairs / 8 : pairs / 4;  // units that turn; the others copy
  Eight<TX> v[U], w[HALF ? U : 1];
  int64_t xo[U], oo[U];
  int un[U];
  auto load = [&](int b) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int u = b + 256 * i;
      un[i] = -1;
      if (u >= all) continue;
      const int h = magic ? int(__umulhi(uint32_t(u), magic)) : u, r = u - h * units;  // r: turned units first, then the others
      const int d = r < turned ? a.rot.first + 8 * r : (8 * (r - turned) < a.rot.first ? 8 * (r - turned) : 8 * (r - turned) + a.rot.rot_dim);
      un[i] = r;
      xo[i] = h * a.xh + d, oo[i] = h * a.oh + d;
      v[i] = load8(x + xo[i]);
      if (HALF && r < turned) w[HALF ? i : 0] = load8(x + xo[i] + pairs);
    }
  };
  load(threadIdx.x);
  for (int i = threadIdx.x; i < pairs; i += 256) {
    float2 cs = rotary_cs32(a.rot.step[i], p);
    cs.x *= a.rot.scale, cs.y *= a.inverse ? -a.rot.scale : a.rot.scale;
    table[i] = cs;
  }
  __syncthreads();
  for (int b = threadIdx.x; b < all;) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int r = un[i];
      if (r < 0) continue;
      float f[8], g[8];
      values8(v[i], f);
      Eight<TO> y;
      if (r >= turned) {
        if constexpr (sizeof(TX) == sizeof(TO)) {
#pragma unroll
          for (int k = 0; k < int(sizeof(TO) / 2); ++k) y.w[k] = v[i].w[k];
        } else {
          pack8(f, y);
        }
        store8(o + oo[i], y);
      } else if (HALF) {
        values8(w[HALF ? i : 0], g);
        float c[8], d[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float2 cs = table[8 * r + k];
          c[k] = f[k] * cs.x - g[k] * cs.y;
          d[k] = f[k] * cs.y + g[k] * cs.x;
        }
        pack8(c, y);
        store8(o + oo[i], y);
        pack8(d, y);
        store8(o + oo[i] + pairs, y);
      } else {
        float c[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 cs = table[4 * r + k];
          c[2 * k] = f[2 * k] * cs.x - f[2 * k + 1] * cs.y;
          c[2 * k + 1] = f[2 * k] * cs.y + f[2 * k + 1] * cs.x;
        }
        pack8(c, y);
        store8(o + oo[i], y);
      }
    }
    b += 256 * U;
    if (b < all) load(b);
  }
}

template <typename TX, typename TO>
void launch(const RotateArgs &a, int tokens, cudaStream_t st) {
  // 16-byte words of eight values everywhere, and a table that fits
  const bool half = a.rot.layout == CSA2_ROTARY_HALF;
  const int units = (a.in_place ? 0 : (a.dim - a.rot.rot_dim) / 8) + a.rot.rot_dim / (half ? 16 : 8);
  const int64_t strides = a.xt | a.xh | a.ot | a.oh;
  const bool words = ((a.dim | a.rot.first | a.rot.rot_dim) & 7) == 0 && (!half || (a.rot.rot_dim & 15) == 0) &&
                     (strides & 7) == 0 && ((reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.out)) & 15) == 0;
  int hpb = a.heads;  // heads per block: all, or fewer while the blocks would not fill the device
  while (hpb > 1 && int64_t(hpb) * units > 256 && int64_t(tokens) * ((a.heads + hpb - 1) / hpb) < 16 * sm_count()) hpb = (hpb + 1) / 2;
  if (words && a.rot.rot_dim <= 4096 && int64_t(hpb) * units * units < (int64_t(1) << 32) && (a.heads + hpb - 1) / hpb <= 65535) {
    // u / units as a multiplication, exact for u units < 2^32 (one unit a head: no division)
    const uint32_t magic = units == 1 ? 0u : uint32_t(((uint64_t(1) << 32) + units - 1) / units);
    const dim3 grid(tokens, (a.heads + hpb - 1) / hpb);
    const size_t smem = size_t(a.rot.rot_dim / 2) * sizeof(float2);
    if (half) rotate8_kernel<TX, TO, true><<<grid, 256, smem, st>>>(a, hpb, units, magic);
    else rotate8_kernel<TX, TO, false><<<grid, 256, smem, st>>>(a, hpb, units, magic);
    return;
  }
  rotate_kernel<TX, TO><<<dim3(tokens, a.heads < 64 ? a.heads : 64), 256, 0, st>>>(a);
}

}  // namespace

void launch_rotate(const void *x, csa2_dtype xd, int64_t xt, int64_t xh, void *out, csa2_dtype od, int64_t ot,
                   int64_t oh, int tokens, int heads, int dim, const int32_t *pos, const csa2_rotary &rot, bool inverse,
                   cudaStream_t st) {
  const RotateArgs a{x, out, xt, xh, ot, oh, heads, dim, pos, rot, inverse, x == out};
  if (xd == CSA2_F32) {
    if (od == CSA2_F32) launch<float, float>(a, tokens, st);
    else launch<float, uint16_t>(a, tokens, st);
  } else {
    if (od == CSA2_F32) launch<uint16_t, float>(a, tokens, st);
    else launch<uint16_t, uint16_t>(a, tokens, st);
  }
}

// Pair index (as a real number) whose frequency turns `turns` times over len positions.
static long double pair_of(long double turns, int len, int rot_dim, long double log_base) {
  return rot_dim * logl(len / (2.0L * acosl(-1.0L) * turns)) / (2.0L * log_base);
}

// Steps in 2^-64 turns: frequency / 2 pi times 2^64 in the host's extended precision.
void rotary_table(int rot_dim, double base, csa2_rotary_scaling scaling, double factor, int original_len,
                  double beta_fast, double beta_slow, uint64_t *step, float *scale) {
  const long double two_pi = 2.0L * acosl(-1.0L), lb = logl(base), s = factor;
  const long double nb = scaling == CSA2_ROTARY_NTK ? lb + logl(s) * rot_dim / (rot_dim - 2) : lb;
  long double lo = 0.0L, hi = 0.0L;
  if (scaling == CSA2_ROTARY_YARN) {
    lo = fmaxl(floorl(pair_of(beta_fast, original_len, rot_dim, lb)), 0.0L);
    hi = fminl(ceill(pair_of(beta_slow, original_len, rot_dim, lb)), rot_dim - 1.0L);
    if (hi <= lo) hi = lo + 0.001L;
  }
  for (int i = 0; i < rot_dim / 2; ++i) {
    long double f = expl(-nb * 2 * i / rot_dim);
    if (scaling == CSA2_ROTARY_LINEAR) f /= s;
    if (scaling == CSA2_ROTARY_YARN) {
      const long double ramp = fminl(1.0L, fmaxl(0.0L, (i - lo) / (hi - lo)));
      f = f / s * ramp + f * (1.0L - ramp);
    }
    const long double turns = f / two_pi;  // below one sixth of a turn, so the rounded step fits
    step[i] = uint64_t(rintl(turns * 18446744073709551616.0L));
  }
  if (scale) *scale = scaling == CSA2_ROTARY_YARN && factor > 1.0 ? float(0.1L * logl(s) + 1.0L) : 1.0f;
}

}  // namespace csa2
