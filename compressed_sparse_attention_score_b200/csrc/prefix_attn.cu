// Dense attention of a batch whose sequences share their first entries (csa2_prefix_attn).
//
// For a query token's 64 heads q_h and its keys v_j (512-d main entries, used as key and value, then
// window tokens): x_hj = tau q_h . v_j, o_h = sum_j e^(x_hj - m_h) v_j / sum_j e^(x_hj - m_h), in one pass
// over the keys with a running reference m_h.  Entries below `prefix` are read through sequence 0's slots
// by every sequence, so the batch's blocks read one copy of them, from L2 after the first.
//
// A persistent block per SM takes an equal share of the batch's 128-key tiles, in row order; a row whose
// tiles lie in several blocks is left as partial (O, m, l) in the workspace and joined by combine_kernel.
// Within a block, per tile:
//   8 producer warps   dequantise the tile once (e2m1 x E4M3 to fp16: exact) into 128 KB of shared memory,
//                      8 blocks of 64 dims, 128-byte swizzle: the K-major A operand of S^T = K Q^T and, the
//                      same bytes, the MN-major A operand of O^T += V^T P^T;
//   1 issuing thread   32 + 32 tcgen05.mma of 128 x 64 x 16 (M = keys or dims, N = the 64 heads); O^T stays in
//                      TMEM (4 x 64 columns) over all tiles of a row;
//   8 softmax warps    read S^T (a lane is a key, a register a head), exponentiate and write P^T in fp16.
// The reference m_h moves only when a logit exceeds it by 2^LAG, so O^T is rarely rescaled; weights are held
// as 2^(x - m + BIAS), which keeps weights down to 2^-29 of the largest in fp16 while 2^(LAG + BIAS) stays far
// below its maximum.  The sums are fp32 of the unrounded weights.
#include <cuda_fp16.h>

#include "attn_common.cuh"
#include "common.cuh"
#include "kernels.cuh"
#include "sm100.cuh"

namespace csa2 {
using namespace sm100;

namespace {
constexpr int PX_TILE = 128;                 // keys per tile
constexpr int PX_PROD = 256, PX_SOFT = 256;  // producer and softmax threads (warps 0-7, 8-15)
constexpr int PX_THREADS = PX_PROD + PX_SOFT + 128;  // the issuer's warpgroup has one working thread
// Registers per thread after launch (96 x 640): 256 x 96 + 256 x 120 + 128 x 48 = 61440.
constexpr int PX_REG_PROD = 96, PX_REG_SOFT = 120, PX_REG_ISSUE = 48;
static_assert(PX_PROD * PX_REG_PROD + PX_SOFT * PX_REG_SOFT + 128 * PX_REG_ISSUE <= 96 * PX_THREADS,
              "the warpgroups' registers exceed the block's");
constexpr int PX_MAX_CTAS = 160;             // workspace is sized for at most this many blocks
constexpr float PX_LAG = 5.f, PX_BIAS = 5.f;
constexpr uint64_t PX_WAIT_NS = 2000000000ull;
constexpr uint32_t PX_TMEM_S = 256, PX_TMEM_COLS = 512;  // O^T in columns 0-255, S^T behind

constexpr int PX_K = 0;                           // key tile: 8 x 16 KB
constexpr int PX_Q = PX_K + 8 * 16384;            // query heads in fp16: 8 chunks of 64 dims x 64 heads
constexpr int PX_P = PX_Q + 8 * 8192;             // P^T: 128 keys x 64 heads fp16
constexpr int PX_MUL = PX_P + 16384;              // [2][128] logit and weight multipliers of the tile's keys
constexpr int PX_HEAD = PX_MUL + 2 * 128 * 8;     // [2][64] 2^-s and, [64], the references
constexpr int PX_RED = PX_HEAD + 3 * 64 * 4;      // [8 warps][32]
constexpr int PX_QMX = PX_RED + 8 * 32 * 4;       // [8 warps][16] query maxima
constexpr int PX_SCAN = PX_QMX + 8 * 16 * 4;      // 40 ints
constexpr int PX_BAR = PX_SCAN + 40 * 4;
constexpr int PX_SMEM = PX_BAR + 16 * 8 + 1024;
static_assert(PX_SMEM <= 227 * 1024, "prefix attention exceeds the shared memory of a block");

constexpr int PX_PART = H * D;               // floats of a partial O; then 64 references and 64 sums
constexpr int PX_SLOT = PX_PART + 2 * H;

struct PrefixArgs {
  const uint16_t *q;
  const int32_t *q_pos;
  int rows, Q;
  float tau2;  // tau log2(e)
  int prefix, n_bound, page_shift;
  csa2_cache c;
  const uint8_t *codes;
  const float *scale;
  int R, window;
  void *o;
  int o_bf16;
  float *lse;
  int32_t *plan;  // [0] tiles per block; from [16]: first tile of each row, and the number of tiles
  float *parts;   // two slots of PX_SLOT floats per block
  int32_t *err;
};

// The keys of a row: entries 0 .. nks - 1, then window tokens lo .. pos.
struct RowKeys {
  int b, nks, lo, nk, tiles;
};
__device__ __forceinline__ RowKeys row_keys(const PrefixArgs &p, int row) {
  RowKeys k;
  k.b = row / p.Q;
  const int pos = p.q_pos[row];
  k.nks = max(0, min(visible_entries(p.c, k.b, pos), p.n_bound));
  k.lo = 0;
  int nkw = 0;
  if (p.codes && pos >= 0) {
    k.lo = max(0, pos - p.window + 1);
    nkw = pos - k.lo + 1;
  }
  k.nk = k.nks + nkw;
  k.tiles = (k.nks + nkw + PX_TILE - 1) / PX_TILE;
  return k;
}

// A block's tiles in order: tile `tile` of row `row`, `left` tiles to go with it.
struct Work {
  int row, tile, left;
  RowKeys k;
  __device__ __forceinline__ void next(const PrefixArgs &p) {
    ++tile;
    if (--left == 0) return;
    while (tile == k.tiles && row + 1 < p.rows) {
      k = row_keys(p, ++row);
      tile = 0;
    }
  }
  __device__ __forceinline__ bool ends_piece() const { return left == 1 || tile + 1 == k.tiles; }
};

__device__ __forceinline__ int64_t entry_slot(const PrefixArgs &p, int b, int n) {
  int64_t s;
  if (p.c.page_table == nullptr) {
    if (n >= p.c.seq_stride) return -1;
    s = int64_t(b) * p.c.seq_stride + n;
  } else {
    const int page = n >> p.page_shift;
    if (page >= p.c.max_pages) return -1;
    const int32_t pid = p.c.page_table[int64_t(b) * p.c.max_pages + page];
    if (pid < 0) return -1;
    s = (int64_t(pid) << p.page_shift) + (n & (p.c.page_size - 1));
  }
  return s < p.c.num_slots ? s : -1;
}

// One key half (dims 256 half .. + 255) as the producer holds it between its loads and the tile.
struct KeyHalf {
  uint4 raw[9];  // an entry's 128 code bytes and 16 scale bytes
  const uint8_t *codes;  // a window token's 256 codes (NULL: an entry or nothing)
  uint32_t shift;        // 2^k in both halves: the token's power of two
  bool valid;
  float mu, pv;
};

__device__ __forceinline__ void load_key(const PrefixArgs &p, const Work &w, int key_in, int half, KeyHalf &r) {
  const int j = w.tile * PX_TILE + key_in;
  r.codes = nullptr;
  r.valid = false;
  r.mu = __int_as_float(0x7FFFFFFF);  // NaN: no key
  r.pv = 0.f;
  if (j < w.k.nks) {
    const int64_t s = entry_slot(p, j < p.prefix ? 0 : w.k.b, j);
    if (s < 0) {
      if (half == 0) report(p.err, CSA2_ERR_INDEX);
      return;
    }
    r.valid = true;
    r.mu = p.tau2;
    r.pv = 1.f;
    const uint4 *src = reinterpret_cast<const uint4 *>(p.c.kv_codes + s * CSA2_MAIN_CODE_BYTES + half * 128);
#pragma unroll
    for (int i = 0; i < 8; ++i) r.raw[i] = src[i];
    r.raw[8] = *reinterpret_cast<const uint4 *>(p.c.kv_scales + s * CSA2_MAIN_SCALE_BYTES + half * 16);
  } else if (j < w.k.nk) {
    const int64_t s = int64_t(w.k.b) * p.R + (w.k.lo + (j - w.k.nks)) % p.R;
    const float sc = p.scale[s];
    // the token's scale is 2^k f: 2^k goes into the fp16 value (exact for -15 <= k <= 7, codes being
    // multiples of 2^-9 up to 448), f into the logit and the weight
    const int k = max(-15, min(7, int((__float_as_uint(sc) >> 23) & 255) - 127));
    const float f = sc * pow2f(-k);
    r.valid = true;
    r.mu = p.tau2 * f;
    r.pv = f;
    const __half2 h = __float2half2_rn(pow2f(k));
    r.shift = *reinterpret_cast<const uint32_t *>(&h);
    r.codes = p.codes + s * CSA2_SWA_DIM + half * 256;
  }
}

// Block c (64 dims) of the half into row key_in of its tile block.
__device__ __forceinline__ void store_block(const KeyHalf &r, int c, int key_in, uint8_t *dst) {
#pragma unroll
  for (int q2 = 0; q2 < 2; ++q2) {
    uint32_t h16[16];
    if (r.codes) {
      const uint4 a = reinterpret_cast<const uint4 *>(r.codes)[4 * c + 2 * q2];
      const uint4 b = reinterpret_cast<const uint4 *>(r.codes)[4 * c + 2 * q2 + 1];
      const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 16; ++i)
        h16[i] = hmul2_u32(cvt_e4m3x2_f16x2((w[i >> 1] >> (16 * (i & 1))) & 0xFFFF), r.shift);
    } else if (r.valid) {
      const uint4 a = r.raw[2 * c + q2];
      const uint32_t sc = ((&r.raw[8].x)[c] >> (16 * q2)) & 0xFFFF;
      const uint32_t s0 = cvt_e4m3x2_f16x2((sc & 0xFF) * 0x101u), s1 = cvt_e4m3x2_f16x2((sc >> 8) * 0x101u);
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int i = 0; i < 16; ++i)
        h16[i] = hmul2_u32(cvt_e2m1x2_f16x2((w[i >> 2] >> (8 * (i & 3))) & 0xFF), i < 8 ? s0 : s1);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) h16[i] = 0u;
    }
#pragma unroll
    for (int v = 0; v < 4; ++v)
      *reinterpret_cast<uint4 *>(dst + kmaj128(key_in, 4 * q2 + v)) =
          make_uint4(h16[4 * v], h16[4 * v + 1], h16[4 * v + 2], h16[4 * v + 3]);
  }
}

// Barrier over the softmax threads; returns the OR of `pred` over them.
__device__ __forceinline__ bool soft_any(bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(uint32_t(pred))
      : "memory");
  return r != 0;
}

// This warpgroup's registers per thread (all of its warps call it).
template <int N>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void tc_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
      "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The query heads of `row` in fp16, scaled per head by a power of two (query_prescale_exp), into the Q
// operand; qinv[h] = 2^-s.  Called by the softmax threads (t of 256); contains two barriers of theirs.
__device__ __forceinline__ void load_query(const PrefixArgs &p, int row, uint8_t *smem, float *qinv, int t) {
  uint32_t *qmx = reinterpret_cast<uint32_t *>(smem + PX_QMX);
  const uint4 *src = reinterpret_cast<const uint4 *>(p.q + int64_t(row) * H * D);
  uint4 v[16];
#pragma unroll
  for (int u = 0; u < 16; ++u) v[u] = src[t + 256 * u];  // head t / 64 + 4 u, dims 8 (t % 64) ..
  const int warp = t >> 5;
#pragma unroll
  for (int u = 0; u < 16; ++u) {
    const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
    uint32_t mb = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) mb = max(mb, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
    mb = __reduce_max_sync(0xffffffffu, mb);
    if ((t & 31) == 0) qmx[warp * 16 + u] = mb;
  }
  soft_any(false);
  const int pair = warp & ~1;  // the two warps that hold the heads t / 64 + 4 u
#pragma unroll
  for (int u = 0; u < 16; ++u) {
    const float sc = pow2f(query_prescale_exp(max(qmx[pair * 16 + u], qmx[pair * 16 + 16 + u])));
    const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
    uint32_t o4[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 hv = __floats2half2_rn(__uint_as_float(w[i] << 16) * sc, __uint_as_float(w[i] & 0xFFFF0000u) * sc);
      o4[i] = *reinterpret_cast<const uint32_t *>(&hv);
    }
    const int h = (t >> 6) + 4 * u, u8 = t & 63;
    *reinterpret_cast<uint4 *>(smem + PX_Q + (u8 / 8) * 8192 + kmaj128(h, u8 % 8)) = make_uint4(o4[0], o4[1], o4[2], o4[3]);
  }
  if (t < H) {
    const int c = t & 3, u = t >> 2;
    qinv[t] = pow2f(-query_prescale_exp(max(qmx[2 * c * 16 + u], qmx[(2 * c + 1) * 16 + u])));
  }
  fence_proxy_async_smem();
  soft_any(false);
}

__global__ void __launch_bounds__(PX_THREADS, 1) prefix_attn_kernel(const __grid_constant__ PrefixArgs p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float2 *mul = reinterpret_cast<float2 *>(smem + PX_MUL);
  float *qinv = reinterpret_cast<float *>(smem + PX_HEAD);  // [2][64]
  float *mref = qinv + 2 * H;
  float *red = reinterpret_cast<float *>(smem + PX_RED);
  int *scan = reinterpret_cast<int *>(smem + PX_SCAN);
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + PX_BAR);  // [4] pair of blocks written (4 warps)
  uint64_t *freed = full + 4;                                    // [4] pair of blocks consumed
  uint64_t *s_full = freed + 4, *p_full = s_full + 1, *q_full = s_full + 2, *o_full = s_full + 3, *idle = s_full + 4;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(s_full + 5);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(s_full + 6);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // ---- the plan: all rows' tiles, the tiles per block, and where this block's begin
  int sum = 0;
  for (int row = tid; row < p.rows; row += PX_THREADS) {
    sum += row_keys(p, row).tiles;
    if (blockIdx.x == 0 && visible_entries(p.c, row / p.Q, p.q_pos[row]) > p.n_bound) report(p.err, CSA2_ERR_SHAPE);
  }
  int total = 0;
  block_exclusive_scan_1024(sum, scan, &total);
  const int per = max(1, (total + int(gridDim.x) - 1) / int(gridDim.x));
  const int t0 = blockIdx.x * per, t1 = min(total, t0 + per);
  if (blockIdx.x == 0 && tid == 0) {
    p.plan[0] = per;
    p.plan[16 + p.rows] = total;
  }
  if (t0 >= t1 && blockIdx.x != 0) return;
  int *first = scan + 36;
  for (int row0 = 0, base = 0; row0 < p.rows; row0 += PX_THREADS) {
    const int row = row0 + tid;
    const int n = row < p.rows ? row_keys(p, row).tiles : 0;
    int all = 0;
    const int off = base + block_exclusive_scan_1024(n, scan, &all);
    if (blockIdx.x == 0 && row < p.rows) p.plan[16 + row] = off;
    if (n > 0 && off <= t0 && t0 < off + n) {
      first[0] = row;
      first[1] = t0 - off;
    }
    base += all;
    if (blockIdx.x != 0 && t0 < base) break;
  }
  grid_dep_launch();
  if (t0 >= t1) return;
  if (warp == 16) {
    tmem_alloc(tmem_slot, PX_TMEM_COLS);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < 4; ++i) {
      mbar_init(&full[i], 4);
      mbar_init(&freed[i], 1);
    }
    mbar_init(s_full, 1);
    mbar_init(p_full, 8);
    mbar_init(q_full, 8);
    mbar_init(o_full, 1);
    mbar_init(idle, 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  Work w;
  w.row = first[0], w.tile = first[1], w.left = t1 - t0;
  w.k = row_keys(p, w.row);

  if (warp < 8) {
    // ------------------------------------------------------------ producers: key tid % 128, half tid / 128
    regs_down<PX_REG_PROD>();
    const int key_in = tid & 127, half = tid >> 7;
    KeyHalf r;
    load_key(p, w, key_in, half, r);
    for (int n = 0; w.left > 0; ++n) {
      bool ok = true;
#pragma unroll
      for (int c2 = 0; c2 < 2; ++c2) {
        const int d = 2 * half + c2;
        if (n > 0) ok = __all_sync(0xffffffffu, mbar_wait_bounded(&freed[d], (n - 1) & 1, abort_flag, PX_WAIT_NS));
        if (!ok) break;
        if (c2 == 0 && half == 0) mul[(n & 1) * 128 + key_in] = make_float2(r.mu, r.pv);
        store_block(r, 2 * c2, key_in, smem + PX_K + (2 * d) * 16384);
        store_block(r, 2 * c2 + 1, key_in, smem + PX_K + (2 * d + 1) * 16384);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[d]);
      }
      if (!ok) break;
      w.next(p);
      if (w.left > 0) load_key(p, w, key_in, half, r);
    }
  } else if (warp < 16) {
    // ------------------------------------------------------------ softmax
    regs_up<PX_REG_SOFT>();
    const int t = tid - PX_PROD, q4 = warp & 3, hb = 32 * ((warp - 8) >> 2), key = 32 * q4 + lane;
    const uint32_t lanes = tmem + (uint32_t(32 * q4) << 16);
    float sum_h[32];
    int piece = 0;
    bool begins = true, alive = true;
    load_query(p, w.row, smem, qinv, t);
    __syncwarp();
    if (lane == 0) mbar_arrive(q_full);
    for (int n = 0; w.left > 0; ++n) {
      const bool ok = mbar_wait_bounded(s_full, n & 1, abort_flag, PX_WAIT_NS);
      tc_fence_after();
      uint32_t s[32];
      __syncwarp();
      const float2 m2 = mul[(n & 1) * 128 + key];
      const bool valid = m2.x == m2.x;
      const float4 *qi4 = reinterpret_cast<const float4 *>(qinv + (piece & 1) * H + hb);
      float *mr = mref + hb;
      // the logits in units of log 2 into s; returns how far they exceed the references
      auto logits = [&]() {
        tc_ld_32x32b_x32(lanes + PX_TMEM_S + hb, s);
        tc_wait_ld();
        float over = -INFINITY;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 qi = qi4[i], m4 = reinterpret_cast<const float4 *>(mr)[i];
          const float qs[4] = {qi.x, qi.y, qi.z, qi.w}, ms[4] = {m4.x, m4.y, m4.z, m4.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x = valid ? (m2.x * __uint_as_float(s[4 * i + e])) * qs[e] : -INFINITY;
            s[4 * i + e] = __float_as_uint(x);
            over = fmaxf(over, x - ms[e]);
          }
        }
        return over;
      };
      const float over = logits();
      if (begins) {
#pragma unroll
        for (int h = 0; h < 32; ++h) sum_h[h] = 0.f;
      }
      if (soft_any(begins || !ok || over > PX_LAG)) {
        // new references: the maxima so far; O^T and the sums follow (O^T holds nothing yet where a piece begins)
        red[(warp - 8) * 32 + lane] = reduce_scatter32<true>(reinterpret_cast<float(&)[32]>(s));
        if (soft_any(!ok)) {
          alive = false;
          break;
        }
        const float *rg = red + (hb >> 5) * 128;
        const float top = fmaxf(fmaxf(rg[lane], rg[32 + lane]), fmaxf(rg[64 + lane], rg[96 + lane]));
        const float old = begins ? -INFINITY : mr[lane];
        const float now = fmaxf(old, top);
        const float alpha = old == -INFINITY ? 0.f : ex2(old - now);  // lane h: head hb + h
        soft_any(false);  // every warp has read the old references and the maxima
        if (q4 == 0) mr[lane] = now;
        if (!begins) {
#pragma unroll
          for (int h = 0; h < 32; ++h) sum_h[h] *= __shfl_sync(0xffffffffu, alpha, h);
          for (int d = 0; d < 4; ++d) {
            uint32_t r[32];
            tc_ld_32x32b_x32(lanes + d * 64 + hb, r);
            tc_wait_ld();
#pragma unroll
            for (int h = 0; h < 32; ++h) r[h] = __float_as_uint(__uint_as_float(r[h]) * __shfl_sync(0xffffffffu, alpha, h));
            tc_st_32x32b_x32(lanes + d * 64 + hb, r);
          }
          tc_wait_st();
        }
        soft_any(false);  // the new references are written
        logits();         // (the reduction above used the registers up)
      }
      begins = false;
      uint32_t ph[16];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 m4 = reinterpret_cast<const float4 *>(mr)[i];
        const float ms[4] = {m4.x, m4.y, m4.z, m4.w};
        float e[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          e[u] = valid ? ex2(__uint_as_float(s[4 * i + u]) - (ms[u] - PX_BIAS)) : 0.f;
          sum_h[4 * i + u] += e[u];
        }
        const __half2 h0 = __floats2half2_rn(e[0] * m2.y, e[1] * m2.y), h1 = __floats2half2_rn(e[2] * m2.y, e[3] * m2.y);
        ph[2 * i] = *reinterpret_cast<const uint32_t *>(&h0);
        ph[2 * i + 1] = *reinterpret_cast<const uint32_t *>(&h1);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        *reinterpret_cast<uint4 *>(smem + PX_P + kmaj128(key, hb / 8 + u)) =
            make_uint4(ph[4 * u], ph[4 * u + 1], ph[4 * u + 2], ph[4 * u + 3]);
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full);
      if (!w.ends_piece()) {
        w.next(p);
        continue;
      }
      // ---- the piece's tiles are done: the next piece's query goes out first, then O^T is read
      const int row = w.row;
      // whole, or a part: the row began in an earlier block (slot 0) or only goes on in a later one (slot 1)
      const bool from_start = piece > 0 || first[1] == 0;
      const bool whole = from_start && w.tile + 1 == w.k.tiles;
      w.next(p);
      if (w.left > 0) {
        load_query(p, w.row, smem, qinv + ((piece + 1) & 1) * H, t);
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);
      }
      const bool o_ok = mbar_wait_bounded(o_full, piece & 1, abort_flag, PX_WAIT_NS);
      tc_fence_after();
      red[(warp - 8) * 32 + lane] = reduce_scatter32<false>(sum_h);
      if (soft_any(!o_ok)) {
        alive = false;
        break;
      }
      const float *rg = red + (hb >> 5) * 128;
      const float total_h = (rg[lane] + rg[32 + lane]) + (rg[64 + lane] + rg[96 + lane]);
      const float m = mr[lane];
      float *part = p.parts + (int64_t(blockIdx.x) * 2 + (from_start ? 1 : 0)) * PX_SLOT;
      const float inv = whole ? (total_h > 0.f ? 1.f / total_h : (total_h == 0.f ? 0.f : total_h)) : 1.f;
      if (q4 == 0) {
        if (whole) {
          p.lse[int64_t(row) * H + hb + lane] =
              total_h == 0.f ? -INFINITY : (m - PX_BIAS + log2f(total_h)) * 0.69314718055994531f;
        } else {
          part[PX_PART + hb + lane] = m;
          part[PX_PART + H + hb + lane] = total_h;
        }
      }
      for (int d = 0; d < 4; ++d) {
        uint32_t r[32];
        tc_ld_32x32b_x32(lanes + d * 64 + hb, r);
        tc_wait_ld();
        const int dim = 128 * d + key;
        if (whole && p.o_bf16) {
          uint16_t *orow = static_cast<uint16_t *>(p.o) + (int64_t(row) * H + hb) * D + dim;
#pragma unroll
          for (int h = 0; h < 32; ++h)
            orow[h * D] = __bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float(r[h]) * __shfl_sync(0xffffffffu, inv, h)));
        } else {
          float *orow = whole ? static_cast<float *>(p.o) + (int64_t(row) * H + hb) * D + dim : part + hb * D + dim;
#pragma unroll
          for (int h = 0; h < 32; ++h) orow[h * D] = __uint_as_float(r[h]) * __shfl_sync(0xffffffffu, inv, h);
        }
      }
      tc_fence_before();
      soft_any(false);  // the sums and O^T have been read
      ++piece;
      begins = true;
    }
    if (!alive && t == 0) report(p.err, CSA2_ERR_TIMEOUT);
  } else {
    regs_down<PX_REG_ISSUE>();
  }
  if (tid == PX_PROD + PX_SOFT) {
    // ------------------------------------------------------------ the tensor core's issuer
    const uint32_t kt = smem_u32(smem + PX_K), qt = smem_u32(smem + PX_Q), pt = smem_u32(smem + PX_P);
    constexpr uint32_t id_s = idesc_f16(PX_TILE, H, false, false), id_o = idesc_f16(PX_TILE, H, true, true);
    bool begins = true, ok = true;
    int piece = 0;
    for (int n = 0; w.left > 0 && ok; ++n) {
      if (begins) {
        if (!(ok = mbar_wait_bounded(q_full, piece & 1, abort_flag, PX_WAIT_NS))) break;
        tc_fence_after();
      }
#pragma unroll 1
      for (int i = 0; i < 4; ++i) {
        const int d = (i & 1) * 2 + (i >> 1);  // the order in which the producers' halves write them
        if (!(ok = mbar_wait_bounded(&full[d], n & 1, abort_flag, PX_WAIT_NS))) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int k4 = 0; k4 < 4; ++k4)
            tc_mma_f16(tmem + PX_TMEM_S, smem_desc(kt + (2 * d + c) * 16384 + 32 * k4, 16, 1024, LAYOUT_SWIZZLE_128B),
                       smem_desc(qt + (2 * d + c) * 8192 + 32 * k4, 16, 1024, LAYOUT_SWIZZLE_128B), id_s,
                       i > 0 || c > 0 || k4 > 0);
      }
      if (!ok) break;
      tc_commit(s_full);
      if (!(ok = mbar_wait_bounded(p_full, n & 1, abort_flag, PX_WAIT_NS))) break;
      tc_fence_after();
#pragma unroll 1
      for (int i = 0; i < 4; ++i) {
        const int d = (i & 1) * 2 + (i >> 1);
#pragma unroll
        for (int jc = 0; jc < 2; ++jc)
#pragma unroll
          for (int k4 = 0; k4 < 4; ++k4)
            tc_mma_f16(tmem + d * 64,
                       smem_desc(kt + (2 * d) * 16384 + jc * 8192 + 2048 * k4, 16384, 1024, LAYOUT_SWIZZLE_128B),
                       smem_desc(pt + (8 * jc + 2 * k4) * 1024, 16, 1024, LAYOUT_SWIZZLE_128B), id_o,
                       !begins || jc > 0 || k4 > 0);
        tc_commit(&freed[d]);
      }
      begins = w.ends_piece();
      if (begins) {
        tc_commit(o_full);
        ++piece;
      }
      w.next(p);
    }
    tc_commit(idle);
    mbar_wait_bounded(idle, 0, abort_flag, PX_WAIT_NS);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 16) {
    tc_fence_after();
    tmem_dealloc(tmem, PX_TMEM_COLS);
  }
}

// Rows whose tiles lie in several blocks: o = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s over their
// partials, in block order; and rows without a key: o = 0, lse = -inf.  One block per row and 8 heads.
__global__ void __launch_bounds__(256) prefix_combine_kernel(const __grid_constant__ PrefixArgs p) {
  __shared__ float wts[PX_MAX_CTAS][8];
  __shared__ float inv[8];
  grid_dep_wait();
  const int row = blockIdx.x, h0 = 8 * blockIdx.y, t = threadIdx.x;
  const int a = p.plan[16 + row], b = p.plan[17 + row], per = p.plan[0];
  const int c0 = a / per, n = b > a ? (b - 1) / per - c0 + 1 : 0;
  if (n == 1) return;
  // the first block holds the row's start as its last piece (slot 1), the others as their first (slot 0)
  auto part = [&](int i) { return p.parts + (int64_t(c0 + i) * 2 + (i == 0 ? 1 : 0)) * PX_SLOT; };
  if (t < 8) {
    const int h = h0 + t;
    float M = -INFINITY, L = 0.f;
    for (int i = 0; i < n; ++i) M = fmaxf(M, part(i)[PX_PART + h]);
    for (int i = 0; i < n; ++i) {
      const float *s = part(i) + PX_PART;
      const float w = s[h] == -INFINITY ? 0.f : ex2(s[h] - M);
      wts[i][t] = w;
      L += w * s[H + h];
    }
    inv[t] = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
    p.lse[int64_t(row) * H + h] = L == 0.f ? -INFINITY : (M - PX_BIAS + log2f(L)) * 0.69314718055994531f;
  }
  __syncthreads();
  for (int it = t; it < 8 * D / 4; it += 256) {
    const int hl = it / (D / 4), d = 4 * (it % (D / 4));
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = 0; i < n; ++i) {
      const float w = wts[i][hl];
      const float4 x = *reinterpret_cast<const float4 *>(part(i) + (h0 + hl) * D + d);
      acc.x += w * x.x, acc.y += w * x.y, acc.z += w * x.z, acc.w += w * x.w;
    }
    const float s = inv[hl];
    const int64_t at = (int64_t(row) * H + h0 + hl) * D + d;
    if (p.o_bf16) {
      const __nv_bfloat162 u = __floats2bfloat162_rn(acc.x * s, acc.y * s), v = __floats2bfloat162_rn(acc.z * s, acc.w * s);
      *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.o) + at) =
          make_uint2(*reinterpret_cast<const uint32_t *>(&u), *reinterpret_cast<const uint32_t *>(&v));
    } else {
      *reinterpret_cast<float4 *>(static_cast<float *>(p.o) + at) = make_float4(acc.x * s, acc.y * s, acc.z * s, acc.w * s);
    }
  }
}

// Blocks of a call: no more than it can have tiles.
int prefix_blocks(int64_t rows, int max_entries, int most) {
  const int64_t tiles = rows * ((int64_t(max_entries) + 128 + PX_TILE - 1) / PX_TILE);
  return int(tiles < most ? tiles : most);
}
size_t plan_bytes(int64_t rows) { return (size_t(rows) * 4 + 68 + 255) & ~size_t(255); }
}  // namespace

size_t prefix_workspace(int64_t rows, int max_entries) {
  return plan_bytes(rows) + size_t(prefix_blocks(rows, max_entries, PX_MAX_CTAS)) * 2 * PX_SLOT * 4;
}

void launch_prefix_attn(const uint16_t *q, int B, int Q, const int32_t *q_pos, float tau, int prefix, int max_entries,
                        const csa2_cache &c, const uint8_t *codes, const float *scale, int R, int window, void *o,
                        bool o_bf16, float *lse, void *ws, int32_t *err, cudaStream_t st) {
  PrefixArgs a{};
  const int rows = B * Q;
  a.q = q, a.q_pos = q_pos, a.rows = rows, a.Q = Q, a.tau2 = tau * 1.4426950408889634f;
  a.prefix = prefix, a.n_bound = max_entries, a.c = c;
  for (a.page_shift = 0; c.page_table && (1 << a.page_shift) < c.page_size;) ++a.page_shift;
  a.codes = codes, a.scale = scale, a.R = R, a.window = window;
  a.o = o, a.o_bf16 = o_bf16, a.lse = lse, a.err = err;
  a.plan = static_cast<int32_t *>(ws);
  a.parts = reinterpret_cast<float *>(static_cast<char *>(ws) + plan_bytes(rows));
  set_smem_limit(prefix_attn_kernel, PX_SMEM);
  const int sms = sm_count();
  prefix_attn_kernel<<<prefix_blocks(rows, max_entries, sms < PX_MAX_CTAS ? sms : PX_MAX_CTAS), PX_THREADS, PX_SMEM, st>>>(a);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(rows, H / 8);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, prefix_combine_kernel, a);
}

}  // namespace csa2
