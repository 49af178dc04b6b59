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

// Any shape: one block per token and group of heads, one thread per dim or pair.
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

template <typename TX, typename TO>
void launch(const RotateArgs &a, int tokens, cudaStream_t st) {
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
