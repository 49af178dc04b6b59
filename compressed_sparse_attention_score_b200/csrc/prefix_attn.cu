// Dense attention of a batch whose sequences share their first entries (csa2_prefix_attn).
//
// For a query token's 64 heads q_h and its keys v_j (512-d main entries, used as key and value, then
// window tokens): x_hj = tau q_h . v_j, o_h = sum_j e^(x_hj - m_h) v_j / sum_j e^(x_hj - m_h), in one pass
// over the keys with a running reference m_h.
//
// Shared entries are dequantised once for the whole batch: expand_kernel writes them to the workspace in fp16
// (e2m1 x E4M3 has at most six significant bits: exact; held as 2^-7 of the value), and every row's tiles of them
// are TMA copies from L2.  Own entries, window tokens and the prefix's last, incomplete tile are dequantised
// in the attention kernel, as is the whole prefix where too few rows share it.
//
// A persistent block per SM takes an equal share of the batch's 128-key tiles, in row order; a row whose
// tiles lie in several blocks is left as partial (O, m, l) in the workspace and joined by combine_kernel.
// Within a block, per tile:
//   the key tile       128 KB of shared memory, 8 blocks of 64 dims, 128-byte swizzle: the K-major A operand of
//                      S^T = K Q^T and, the same bytes, the MN-major A operand of O^T += V^T P^T; written by
//   1 loading warp     (shared tiles, TMA) or by
//   8 producer warps   (the others), a pair of blocks as soon as the previous tile's products have read it;
//   1 issuing warp     32 + 32 tcgen05.mma of 128 x 64 x 16 (M = keys or dims, N = the 64 heads); O^T stays in
//                      TMEM (4 x 64 columns) over all tiles of a row;
//   8 softmax warps    read S^T (a lane is a key, a register a head), exponentiate and write P^T in fp16.
// The reference m_h moves only when a logit exceeds it by 2^LAG, so O^T is rarely rescaled; weights are held
// as 2^(x - m + BIAS), which keeps weights down to 2^-29 of the largest in fp16 while 2^(LAG + BIAS) stays far
// below its maximum.  The sums are fp32 of the unrounded weights.
//
// What bounds it: a product of 128 x 64 x 16 reads 6 KB of shared memory (48.8 clocks; the tensor core would take 32), a
// tile has 64 of them, and its 128 KB are written there too: 4150 clocks a tile, 4700 to 5000 measured where it is copied
// (2.6 to 2.7 us at the 1.80 GHz that the SMs average in this kernel) and 9500 to 10000 where it is dequantised in the block
// (5.4 us).  The rest is the softmax between a tile's products; TMEM and shared memory hold one row's tile, so nothing else
// can run meanwhile.
// Measured (whole call): 32 rows over 8192 shared entries 68 us, 96 over 4096 96 us, 16 over 65536 200 us (692
// TFLOP/s), 13 over 2999 33 us, 2 over 96 21 us.
#include <cuda_fp16.h>
#include <string.h>

#include "attn_common.cuh"
#include "common.cuh"
#include "kernels.cuh"
#include "sm100.cuh"

namespace csa2 {
using namespace sm100;

namespace {
constexpr int PX_TILE = 128;                 // keys per tile
constexpr int PX_PROD = 256, PX_SOFT = 256;  // producer and softmax threads (warps 0-7, 8-15)
constexpr int PX_ISSUE_WARP = 16, PX_LOAD_WARP = 17;
constexpr int PX_THREADS = PX_PROD + PX_SOFT + 128;  // (the last warpgroup has two working warps)
// Registers per thread after launch (96 x 640): 256 x 96 + 256 x 128 + 128 x 32 = 61440.  (Softmax warps with 120
// spill more: 16 rows over 65536 shared entries 217 against 211 us.)
constexpr int PX_REG_SOFT = 128, PX_REG_ISSUE = 32;
static_assert(PX_PROD * 96 + PX_SOFT * PX_REG_SOFT + 128 * PX_REG_ISSUE <= 96 * PX_THREADS,
              "the warpgroups' registers exceed the block's");
// A shared prefix is dequantised ahead where at least this many rows have at least this many tiles of it in all (2.7 tiles a
// block).  Measured, ahead against by every row (up to 100 own entries and a window of 128): 16 rows over 8192 entries
// 43 / 60 us, 8 over 8192 39 / 43, 4 over 32768 60 / 66; 6 over 8192 38 / 39, 16 over 2048 31 / 29, 4 over 8192 35 / 33,
// 2 over 32768 67 / 64.
constexpr int PX_MIN_ROWS = 4, PX_MIN_SHARED = 400;
constexpr int PX_MAX_CTAS = 160;             // workspace is sized for at most this many blocks
constexpr float PX_LAG = 5.f, PX_BIAS = 5.f;
constexpr uint64_t PX_WAIT_NS = 2000000000ull;
constexpr uint32_t PX_TMEM_S = 256, PX_TMEM_COLS = 512;  // O^T in columns 0-255, S^T behind

constexpr int PX_K = 0;                           // key tile: 8 x 16 KB
constexpr int PX_Q = PX_K + 8 * 16384;            // query heads in fp16: 8 chunks of 64 dims x 64 heads
constexpr int PX_P = PX_Q + 8 * 8192;             // P^T: 128 keys x 64 heads fp16
constexpr int PX_MUL = PX_P + 16384;              // [2][128] logit and weight multipliers of the tile's keys
constexpr int PX_QMU = PX_MUL + 2 * 128 * 8;      // [64] logit factor of each head
// What each lane quarter's softmax warps keep for themselves, [4][64] each: the references m, BIAS - m, and the factors of a
// finished row.
constexpr int PX_MREF = PX_QMU + 64 * 4;
constexpr int PX_NREF = PX_MREF + 4 * 64 * 4;
constexpr int PX_INV = PX_NREF + 4 * 64 * 4;
constexpr int PX_RED = PX_INV + 4 * 64 * 4;       // [8 warps][32] maxima
constexpr int PX_SUM = PX_RED + 8 * 32 * 4;       // [8 warps][32] sums
constexpr int PX_SCAN = PX_SUM + 8 * 32 * 4;      // 48 ints
constexpr int PX_BAR = PX_SCAN + 48 * 4;
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
  int32_t *plan;  // [0] tiles per block, or [1] blocks per row; from [16]: first tile of each row, and the number of tiles
  int shared;     // tiles of the prefix that are dequantised ahead (0: none),
  uint16_t *rows16;  // their entries in fp16, 512 each,
  int32_t *bad;      // and for each 32 of them whether one is outside the cache
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

// A row of n tiles in at most `parts` parts: no part of fewer than two tiles (joining a partial row costs about what
// a tile does); and the first tile of part i.
__device__ __forceinline__ int part_count(int n, int parts) { return min((n + 1) / 2, parts); }
// Dequantising a tile in the block costs twice what copying it does (see above); parts are equal with 7 : 4 for it, as all
// the measured calls were split (2 : 1 was not tried).  The row's first `shared` tiles are copied.
__device__ __forceinline__ int part_start(int n, int shared, int i, int parts) {
  const int m = part_count(n, parts);
  if (i >= m) return n;
  const int64_t cost = (4 * int64_t(shared) + 7 * int64_t(n - shared)) * i / m;
  return cost <= 4 * int64_t(shared) ? int(cost / 4) : shared + int((cost - 4 * int64_t(shared)) / 7);
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
  // every key of the tile is among the first `limit` entries
  __device__ __forceinline__ bool within(int limit) const { return (tile + 1) * PX_TILE <= min(limit, k.nks); }
};

// Slot of entry j of sequence b, given its page table's entry for it (-1: none); NO_SLOT if outside the cache.
// (A slot's bytes are in memory, so its number fits 32 bits.)
constexpr uint32_t NO_SLOT = 0xFFFFFFFFu;
__device__ __forceinline__ int32_t entry_page(const PrefixArgs &p, int b, int j) {
  const int n = j >> p.page_shift;
  return p.c.page_table && n < p.c.max_pages ? p.c.page_table[int64_t(b) * p.c.max_pages + n] : -1;
}
__device__ __forceinline__ uint32_t entry_slot(const PrefixArgs &p, int b, int j, int32_t page) {
  int64_t s = -1;
  if (p.c.page_table) {
    if (page >= 0) s = (int64_t(page) << p.page_shift) + (j & (p.c.page_size - 1));
  } else if (j < p.c.seq_stride) {
    s = int64_t(b) * p.c.seq_stride + j;
  }
  return s >= 0 && s < p.c.num_slots ? uint32_t(s) : NO_SLOT;
}

// Eight 4-bit codes times 2^-7 s (s128: 2^7 s in both halves) in fp16: o[e] holds elements e and e + 4, the order that a
// word unpacks to pairwise (the query and the output use the same order of dims).  A code's three magnitude bits,
// moved to bits 9 - 11 of an fp16 number, are 2^-14 of its value (subnormal for 0.5, as in e2m1): four codes at a time to
// the high bytes of such numbers, then a byte permutation each.
__device__ __forceinline__ void unpack8(uint32_t w, uint32_t s128, uint32_t *o) {
  const uint32_t even = ((w << 4) & 0x80808080u) | ((w << 1) & 0x0E0E0E0Eu), odd = (w & 0x80808080u) | ((w >> 3) & 0x0E0E0E0Eu);
  o[0] = hmul2_u32(__byte_perm(even, 0u, 0x2404), s128);
  o[1] = hmul2_u32(__byte_perm(odd, 0u, 0x2404), s128);
  o[2] = hmul2_u32(__byte_perm(even, 0u, 0x3414), s128);
  o[3] = hmul2_u32(__byte_perm(odd, 0u, 0x3414), s128);
}
// 2^7 times an E4M3 scale, in both halves (at most 57344).
__device__ __forceinline__ uint32_t scale128(uint32_t byte) { return hmul2_u32(cvt_e4m3x2_f16x2(byte * 0x101u), 0x58005800u); }

// The prefix's complete tiles in fp16, 32 entries a block, four a warp; lane l holds dims 8 l .. and 256 + 8 l .., so that every
// load and store of a warp is one contiguous piece.  Memory bound: 288 bytes read and 1 KB written an entry
// (65536 entries: 15 us).
constexpr int EXPAND = 32;
__global__ void __launch_bounds__(256) prefix_expand_kernel(const __grid_constant__ PrefixArgs p) {
  grid_dep_wait();    // (the table and the planes may be the previous kernel's work)
  grid_dep_launch();  // from here on the attention kernel may start, and read what was written before this call
  const int lane = threadIdx.x & 31, j0 = blockIdx.x * EXPAND + 4 * (threadIdx.x >> 5);
  int32_t page[4];
  uint32_t slot[4], sc[4][2], codes[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i) page[i] = entry_page(p, 0, j0 + i);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    slot[i] = entry_slot(p, 0, j0 + i, page[i]);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      codes[i][u] = sc[i][u] = 0u;
      if (slot[i] != NO_SLOT) {
        codes[i][u] = reinterpret_cast<const uint32_t *>(p.c.kv_codes + int64_t(slot[i]) * CSA2_MAIN_CODE_BYTES)[32 * u + lane];
        sc[i][u] = p.c.kv_scales[int64_t(slot[i]) * CSA2_MAIN_SCALE_BYTES + 16 * u + (lane >> 1)];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      uint32_t h[4];
      unpack8(codes[i][u], scale128(sc[i][u]), h);
      reinterpret_cast<uint4 *>(p.rows16 + int64_t(j0 + i) * D)[32 * u + lane] = make_uint4(h[0], h[1], h[2], h[3]);
    }
  const int any = __syncthreads_or(slot[0] == NO_SLOT || slot[1] == NO_SLOT || slot[2] == NO_SLOT || slot[3] == NO_SLOT);
  if (threadIdx.x == 0) p.bad[blockIdx.x] = any;
}

// A window token's scale as 2^k f: 2^(k - 7) goes into the fp16 values, f into the logit and the weight.  Codes
// are multiples of 2^-9 up to 448, so that is exact for -8 <= k <= 14; for smaller scales down to k = -16 it is
// off by 2^-10 of the token's largest value at most, its E4M3 codes by 2^-5.
__device__ __forceinline__ int window_exponent(float scale) {
  return max(-16, min(14, int((__float_as_uint(scale) >> 23) & 255) - 127));
}

// A producer thread's part of a tile: 32 dims of each pair of blocks, of two keys 8 apart.  A warp's load of 16 bytes
// a thread covers 64 bytes of each of eight keys, and its 16-byte stores fall into all banks.
struct KeyPart {
  uint32_t slot[2];  // cache slot of an entry, ring slot of a window token; NO_SLOT: no key
  int entries;       // keys of the tile below this are entries
  float scale[2];    // a window token's scale
};
struct KeyBytes {
  uint4 raw[2][2];  // in one pair of blocks, an entry's 32 codes [0] and two scales [1].x, or a token's 32 codes
};
struct KeyPlace {
  int key0;   // the first of its keys
  int piece;  // which 32 dims of the pair
};

// The slots of the tile's keys.
__device__ __forceinline__ void find_keys(const PrefixArgs &p, const Work &w, const KeyPlace &at, KeyPart &r) {
  r.entries = w.k.nks - w.tile * PX_TILE;
  int32_t page[2];  // (the two table entries are fetched together)
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int j = w.tile * PX_TILE + at.key0 + 8 * i;
    page[i] = j < w.k.nks ? entry_page(p, j < p.prefix ? 0 : w.k.b, j) : -1;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int j = w.tile * PX_TILE + at.key0 + 8 * i;
    r.slot[i] = j < w.k.nks ? entry_slot(p, j < p.prefix ? 0 : w.k.b, j, page[i]) : NO_SLOT;
    if (j >= w.k.nks && j < w.k.nk) {
      r.slot[i] = uint32_t(w.k.b) * p.R + (w.k.lo + (j - w.k.nks)) % p.R;
      r.scale[i] = p.scale[r.slot[i]];
    }
  }
  if (at.piece == 0) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (r.slot[i] == NO_SLOT && at.key0 + 8 * i < r.entries) report(p.err, CSA2_ERR_INDEX);
  }
}

// The keys' bytes of pair d.
__device__ __forceinline__ void load_keys(const PrefixArgs &p, const KeyPlace &at, int d, const KeyPart &r, KeyBytes &x) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (r.slot[i] == NO_SLOT) continue;
    if (at.key0 + 8 * i < r.entries) {
      x.raw[i][0] = *reinterpret_cast<const uint4 *>(p.c.kv_codes + int64_t(r.slot[i]) * CSA2_MAIN_CODE_BYTES + 64 * d + at.piece * 16);
      x.raw[i][1].x = *reinterpret_cast<const uint16_t *>(p.c.kv_scales + int64_t(r.slot[i]) * CSA2_MAIN_SCALE_BYTES + 8 * d + at.piece * 2);
    } else {
      const uint4 *src = reinterpret_cast<const uint4 *>(p.codes + int64_t(r.slot[i]) * CSA2_SWA_DIM + 128 * d + 32 * at.piece);
      x.raw[i][0] = src[0];
      x.raw[i][1] = src[1];
    }
  }
}

// The factors of the logits and weights of the tile's keys (NaN and 0: no key; a window token's scale may be NaN itself, in both).
__device__ __forceinline__ void store_factors(const KeyPlace &at, const KeyPart &r, float2 *mul) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float f = __int_as_float(0x7FFFFFFF);
    if (r.slot[i] != NO_SLOT)
      f = at.key0 + 8 * i < r.entries ? 1.f : r.scale[i] * pow2f(-window_exponent(r.scale[i]));
    mul[at.key0 + 8 * i] = make_float2(f, r.slot[i] != NO_SLOT ? f : 0.f);
  }
}

// Key i's 32 dims in fp16, times 2^-7, in the order of unpack8.
__device__ __forceinline__ void dequant_key(const KeyPlace &at, const KeyPart &r, const KeyBytes &x, int i, uint32_t (&h)[16]) {
  const uint4 a = x.raw[i][0], b = x.raw[i][1];
  if (r.slot[i] == NO_SLOT) {
#pragma unroll
    for (int e = 0; e < 16; ++e) h[e] = 0u;
  } else if (at.key0 + 8 * i < r.entries) {
    const uint32_t s0 = scale128(b.x & 0xFFu), s1 = scale128(b.x >> 8);
    unpack8(a.x, s0, h);
    unpack8(a.y, s0, h + 4);
    unpack8(a.z, s1, h + 8);
    unpack8(a.w, s1, h + 12);
  } else {
    const __half2 two = __float2half2_rn(pow2f(window_exponent(r.scale[i]) - 7));
    const uint32_t s = *reinterpret_cast<const uint32_t *>(&two);
    const uint32_t w8[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int v = 0; v < 4; ++v)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        h[4 * v + e] = hmul2_u32(cvt_e4m3x2_f16x2(__byte_perm(w8[2 * v], w8[2 * v + 1], e | ((4 + e) << 4)) & 0xFFFF), s);
  }
}

// Those values into the pair of blocks at dst.
__device__ __forceinline__ void store_key(const uint32_t (&h)[16], const KeyPlace &at, int i, uint8_t *dst) {
#pragma unroll
  for (int v = 0; v < 4; ++v)
    *reinterpret_cast<uint4 *>(dst + (at.piece >> 1) * 16384 + kmaj128(at.key0 + 8 * i, 4 * (at.piece & 1) + v)) =
        make_uint4(h[4 * v], h[4 * v + 1], h[4 * v + 2], h[4 * v + 3]);
}

// One block of 64 dims of the prefix's tile `tile` into shared memory, completing on `bar`.
__device__ __forceinline__ void tma_block(uint32_t dst, const CUtensorMap *map, int block, int tile, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(64 * block), "r"(tile * PX_TILE), "r"(smem_u32(bar))
      : "memory");
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

// D (+)= A B^T with operands `da` and `db` 16-byte units behind the descriptors whose low words are a and b (the high
// words are the same for all: 1 KB between 8-row groups, 128-byte swizzle), issued by the lane with `leader`.  The
// whole warp runs it, so that the descriptors stay in uniform registers: in a branch of one lane a product took
// 90 clocks to issue, twice its execution.
constexpr uint32_t DESC_HIGH = (1024 >> 4) | (1u << 14) | (uint32_t(LAYOUT_SWIZZLE_128B) << 29);
__device__ __forceinline__ uint32_t desc_low(uint32_t saddr, uint32_t lbo_bytes) { return (saddr >> 4) | ((lbo_bytes >> 4) << 16); }
__device__ __forceinline__ void mma_at(uint32_t leader, uint32_t d_tmem, uint32_t a, uint32_t da, uint32_t b, uint32_t db,
                                       uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, l;\n\t.reg .b64 x, y;\n\t"
      "mov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 l, %6, 0;\n\t"
      "@l tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a + da), "r"(b + db), "r"(idesc), "r"(uint32_t(accumulate)), "n"(DESC_HIGH), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void commit_to(uint32_t leader, uint64_t *bar) {
  asm volatile(
      "{\n\t.reg .pred l;\n\tsetp.ne.b32 l, %1, 0;\n\t"
      "@l tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(leader)
      : "memory");
}
// This warpgroup's registers per thread (all of its warps call it).
template <int N>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

// One lane of a converged warp (the same one every time).
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}

// Four heads' logit factors and negated references.  Volatile: kept where they are used, or all heads' would take the
// registers at once.
__device__ __forceinline__ void lds_pair(float4 &q, float4 &r, uint32_t q_at, uint32_t r_at) {
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%8];\n\tld.shared.v4.f32 {%4, %5, %6, %7}, [%9];"
               : "=f"(q.x), "=f"(q.y), "=f"(q.z), "=f"(q.w), "=f"(r.x), "=f"(r.y), "=f"(r.z), "=f"(r.w)
               : "r"(q_at), "r"(r_at)
               : "memory");
}
__device__ __forceinline__ float redux_max(float x) {
  float m;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x));
  return m;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// a += x, b += y, and a *= x, b *= y (one packed operation, each result rounded to nearest).
__device__ __forceinline__ void add2(float &a, float &b, float x, float y) {
  asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\tadd.rn.f32x2 p, p, q;\n\t"
      "mov.b64 {%0, %1}, p;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(x), "f"(y));
}

__device__ __forceinline__ void mul2(float &a, float &b, float x, float y) {
  asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\tmul.rn.f32x2 p, p, q;\n\t"
      "mov.b64 {%0, %1}, p;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(x), "f"(y));
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
// operand; qmu[h] = 2^7 tau log2(e) 2^-s (the tile holds 2^-7 of the keys).  A softmax warp takes the heads 8 w ..; nothing
// waits: every warp has read the previous row's factors, and the tensor core its query, when one gets here.
__device__ __forceinline__ void load_query(const PrefixArgs &p, int row, uint8_t *smem, float *qmu, int w, int lane) {
  const uint4 *src = reinterpret_cast<const uint4 *>(p.q + (int64_t(row) * H + 8 * w) * D) + lane;
  uint4 v[16];  // head 8 w + u / 2, dims 8 lane + 256 (u % 2) ..
#pragma unroll
  for (int u = 0; u < 16; ++u) v[u] = src[32 * u];
#pragma unroll
  for (int hh = 0; hh < 8; ++hh) {
    uint32_t mb = 0;
#pragma unroll
    for (int u = 2 * hh; u < 2 * hh + 2; ++u) {
      const uint32_t x[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) mb = max(mb, max(x[i] & 0x7FFFu, (x[i] >> 16) & 0x7FFFu));
    }
    const int e = query_prescale_exp(__reduce_max_sync(0xffffffffu, mb)), h = 8 * w + hh;
    const float sc = pow2f(e);
#pragma unroll
    for (int u = 2 * hh; u < 2 * hh + 2; ++u) {
      const uint32_t x[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
      uint32_t o4[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // dims i and i + 4 of the eight
        const uint32_t lo = x[i >> 1], hi = x[2 + (i >> 1)];
        const __half2 hv = __floats2half2_rn(__uint_as_float((i & 1) ? lo & 0xFFFF0000u : lo << 16) * sc,
                                             __uint_as_float((i & 1) ? hi & 0xFFFF0000u : hi << 16) * sc);
        o4[i] = *reinterpret_cast<const uint32_t *>(&hv);
      }
      const int u8 = lane + 32 * (u & 1);
      *reinterpret_cast<uint4 *>(smem + PX_Q + (u8 / 8) * 8192 + kmaj128(h, u8 % 8)) = make_uint4(o4[0], o4[1], o4[2], o4[3]);
    }
    if (lane == 0) qmu[h] = 128.f * p.tau2 * pow2f(-e);
  }
  fence_proxy_async_smem();
  __syncwarp();
}

__global__ void __launch_bounds__(PX_THREADS, 1) prefix_attn_kernel(const __grid_constant__ CUtensorMap map,
                                                                     const __grid_constant__ PrefixArgs p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float2 *mul = reinterpret_cast<float2 *>(smem + PX_MUL);
  float *qmu = reinterpret_cast<float *>(smem + PX_QMU);
  float *red = reinterpret_cast<float *>(smem + PX_RED), *sums = reinterpret_cast<float *>(smem + PX_SUM);
  int *scan = reinterpret_cast<int *>(smem + PX_SCAN);
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + PX_BAR);  // [4] pair of blocks written
  uint64_t *freed = full + 4;                                    // [4] pair of blocks consumed
  uint64_t *s_full = freed + 4, *o_full = s_full + 1, *p_full = s_full + 2, *q_full = s_full + 3, *idle = s_full + 4;
  uint64_t *p_again = s_full + 5;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(s_full + 6);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(s_full + 7), *moving = abort_flag + 1;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

  if (p.shared == 0) grid_dep_wait();  // (the inputs may be the previous kernel's work)
  // ---- the plan: the tiles of all rows and of the longest, and this block's share
  int *first = scan + 36;  // this block's first row, first tile of it, shared tiles, longest row, its tiles (2), the row's keys (5)
  auto first_row = [&](int row, int tile, const RowKeys &k) {
    first[0] = row, first[1] = tile;
    first[6] = k.b, first[7] = k.nks, first[8] = k.lo, first[9] = k.nk, first[10] = k.tiles;
  };
  RowKeys mine{};  // (read for up to 32 rows, a lane's own)
  int sum = 0, most = 0;
  for (int row = tid; row < p.rows; row += PX_THREADS) {
    mine = row_keys(p, row);
    sum += mine.tiles;
    most = max(most, mine.tiles);
    if (blockIdx.x == 0 && visible_entries(p.c, row / p.Q, p.q_pos[row]) > p.n_bound) report(p.err, CSA2_ERR_SHAPE);
  }
  // Up to 32 rows are counted by the first warp alone, which saves the block's barriers.
  const bool few = p.rows <= 32;
  int total = 0;
  if (!few) {
    if (tid == 0) first[3] = 0;
    block_exclusive_scan_1024(sum, scan, &total);
    const int m = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) atomicMax(&first[3], m);
    __syncthreads();
    most = first[3];
  } else if (warp == 0) {
    total = __reduce_add_sync(0xffffffffu, sum);
    most = __reduce_max_sync(0xffffffffu, most);
  }
  // Equal shares of all tiles in row order; or, where that makes no block's share more than two tiles longer (what going
  // over to another row costs, and a little less), each row in as many equal parts as there are blocks for it.  Rows of
  // equal length then pass over the prefix side by side, and what one of them has read is still in L2 for the others.
  const int parts = int(gridDim.x) / p.rows;
  int per = 0, by_row = 0, t0 = 0, t1 = 0;
  auto share = [&]() {
    per = max(1, (total + int(gridDim.x) - 1) / int(gridDim.x));
    by_row = parts > 0 && (most + parts - 1) / max(parts, 1) <= per + 2 ? parts : 0;
    t0 = blockIdx.x * per, t1 = min(total, t0 + per);
  };
  if (few) {
    if (warp == 0) {
      share();
      int off = sum;  // lane i: the first tile of row i
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, off, o);
        if (lane >= o) off += y;
      }
      off -= sum;
      if (blockIdx.x == 0 && lane < p.rows) p.plan[16 + lane] = off;
      int row = by_row ? int(blockIdx.x) / parts : 0;
      if (by_row) {
        const int n = __shfl_sync(0xffffffffu, sum, row & 31), i = blockIdx.x % parts;
        const int copied = __shfl_sync(0xffffffffu, min(p.shared, mine.nks / PX_TILE), row & 31);
        t0 = row < p.rows ? part_start(n, copied, i, parts) : 0, t1 = row < p.rows ? part_start(n, copied, i + 1, parts) : 0;
        if (lane == row) first_row(row, t0, mine);
      } else if (sum > 0 && off <= t0 && t0 < off + sum) {
        first_row(lane, t0 - off, mine);
      }
      if (lane == 0) first[4] = t0, first[5] = t1;
    }
    __syncthreads();
    t0 = first[4], t1 = first[5];
  } else {
    share();
    if (by_row) {
      const int row = blockIdx.x / parts, i = blockIdx.x % parts;
      RowKeys k{};
      if (row < p.rows) k = row_keys(p, row);
      const int copied = min(p.shared, k.nks / PX_TILE);
      t0 = part_start(k.tiles, copied, i, parts), t1 = part_start(k.tiles, copied, i + 1, parts);
      if (tid == 0) first_row(row, t0, k);
    }
    if (!by_row || blockIdx.x == 0)
      for (int row0 = 0, base = 0; row0 < p.rows; row0 += PX_THREADS) {
        const int row = row0 + tid;
        RowKeys k{};
        if (row < p.rows) k = row_keys(p, row);
        const int n = k.tiles;
        int all = 0;
        const int off = base + block_exclusive_scan_1024(n, scan, &all);
        if (blockIdx.x == 0 && row < p.rows) p.plan[16 + row] = off;
        if (!by_row && n > 0 && off <= t0 && t0 < off + n) first_row(row, t0 - off, k);
        base += all;
        if (blockIdx.x != 0 && t0 < base) break;
      }
  }
  if (blockIdx.x == 0 && tid == 0) {
    p.plan[0] = per;
    p.plan[1] = by_row;
    p.plan[16 + p.rows] = total;
  }
  grid_dep_launch();
  if (t0 >= t1) {
    grid_dep_wait();  // (so that this kernel's end implies the expansion's)
    return;
  }
  if (!few) __syncthreads();  // the first row is written
  if (tid < 512)  // the first query row on its way into L2 while the block is set up
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p.q + int64_t(first[0]) * H * D + 64 * tid));
  // entries below `limit` are read from the workspace: the shared tiles before the first bad one
  int *limit_at = first + 2;
  if (tid == 0) *limit_at = p.shared;
  grid_dep_wait();
  __syncthreads();
  for (int i = tid; i < p.shared * (PX_TILE / EXPAND); i += PX_THREADS)
    if (p.bad[i]) atomicMin(limit_at, i / (PX_TILE / EXPAND));
  if (warp == 0) {
    tmem_alloc(tmem_slot, PX_TMEM_COLS);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < 4; ++i) {
      mbar_init(&full[i], i == 0 ? 9 : 8);  // the producer warps; the first pair's also the loader, whoever writes the tile
      mbar_init(&freed[i], 1);
    }
    mbar_init(s_full, 1);
    mbar_init(o_full, 1);
    mbar_init(p_full, 8);
    mbar_init(p_again, 8);
    mbar_init(q_full, 8);
    mbar_init(idle, 1);
    *abort_flag = 0;
    *moving = 0;
    mbar_init_fence();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  Work w;
  w.row = first[0], w.tile = first[1], w.left = t1 - t0;
  w.k = RowKeys{first[6], first[7], first[8], first[9], first[10]};
  const int limit = *limit_at * PX_TILE;

  if (warp < 8) {
    // ------------------------------------------------------------ producers: warp w keys 16 w .. + 15
    // The next pair's bytes are asked for before a pair is dequantised, and its first key waits in registers for the pair's
    // blocks to be free.
    const KeyPlace at{16 * warp + (lane & 3) + 4 * ((lane >> 3) & 1), ((lane >> 2) & 1) + 2 * (lane >> 4)};
    KeyPart r;
    KeyBytes x, ahead;
    uint32_t h[16];
    bool ok = true;
    auto wait = [&](int d, int n) {
      return __all_sync(0xffffffffu, mbar_wait_bounded(&freed[d], n & 1, abort_flag, PX_WAIT_NS));
    };
    for (int n = 0; w.left > 0 && ok; ++n, w.next(p)) {
      if (w.within(limit)) {
        // The loader's tile.  It counts these warps all the same: a barrier's parity tells only its last two phases apart, and
        // as no tile's products begin before every writer has seen the tile before it freed, `freed` cannot run ahead of a
        // writer that is late.  (Given up, the arrival still ends the phase that the loader's copies belong to.)
        if (n > 0) ok = wait(0, n - 1);
        if (lane == 0) mbar_arrive(&full[0]);
        continue;
      }
      find_keys(p, w, at, r);
      load_keys(p, at, 0, r, x);
#pragma unroll 1
      for (int d = 0; d < 4; ++d) {
        if (d < 3) load_keys(p, at, d + 1, r, ahead);
        dequant_key(at, r, x, 0, h);
        if (n > 0) ok = wait(d, n - 1);
        if (!ok) break;
        if (d == 0 && at.piece == 0) store_factors(at, r, mul + (n & 1) * 128);
        uint8_t *dst = smem + PX_K + d * 2 * 16384;
        store_key(h, at, 0, dst);
        dequant_key(at, r, x, 1, h);
        store_key(h, at, 1, dst);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[d]);
        x = ahead;
      }
    }
  } else if (warp >= PX_ISSUE_WARP) {
    regs_down<PX_REG_ISSUE>();
    if (warp == PX_LOAD_WARP) {
      // ---------------------------------------------------------- the loader of shared tiles
      const uint32_t kt = smem_u32(smem + PX_K);
      if (p.shared > 0) asm volatile("fence.proxy.async;" ::: "memory");  // (the expansion's stores were generic ones)
      bool ok = true;
      int last[4] = {-1, -1, -1, -1}, never = 0;
      auto wait = [&](int d, int n) {
        return __all_sync(0xffffffffu, mbar_wait_bounded(&freed[d], n & 1, abort_flag, PX_WAIT_NS));
      };
      for (int n = 0; w.left > 0 && ok; ++n, w.next(p)) {
        if (!w.within(limit)) {  // the producers' tile (see there)
          if (n > 0) ok = wait(0, n - 1);
          if (lane == 0) mbar_arrive(&full[0]);
          continue;
        }
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          if (ok && n > 0) ok = wait(d, n - 1);
          if (ok) last[d] = n;
          if (ok && lane == 0) {
            mbar_arrive_expect_tx(&full[d], 2 * 16384);
            tma_block(kt + (2 * d) * 16384, &map, 2 * d, w.tile, &full[d]);
            tma_block(kt + (2 * d + 1) * 16384, &map, 2 * d + 1, w.tile, &full[d]);
          } else if (ok && d > 0 && lane < 8) {
            mbar_arrive(&full[d]);  // (the barrier counts the eight producer warps)
          }
          __syncwarp();
        }
      }
      if (!ok)  // given up: the copies under way still have to land before the block ends
        for (int d = 0; d < 4; ++d)
          if (last[d] >= 0) mbar_wait_bounded(&full[d], last[d] & 1, &never, PX_WAIT_NS);
    }
    // ------------------------------------------------------------ the tensor core's issuer
    // O^T += V^T P^T, 128 dims (a pair of blocks) at a time, then S^T of the next tile over each pair as soon as it is
    // written, four steps behind its last use.
    if (warp == PX_ISSUE_WARP) {
      const uint32_t kt = smem_u32(smem + PX_K), qt = smem_u32(smem + PX_Q), pt = smem_u32(smem + PX_P);
      const uint32_t leader = elect_one();
      constexpr uint32_t id_s = idesc_f16(PX_TILE, H, false, false), id_o = idesc_f16(PX_TILE, H, true, true);
      auto wait = [&](uint64_t *bar, int phase) {
        const bool ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar, phase & 1, abort_flag, PX_WAIT_NS));
        tc_fence_after();
        return ok;
      };
      auto step_s = [&](int n, int d, bool opens) {
        if (!wait(&full[d], n)) return false;
        const uint32_t a = desc_low(kt, 16) + 2048 * d, b = desc_low(qt, 16) + 1024 * d;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int k4 = 0; k4 < 4; ++k4)
            mma_at(leader, tmem + PX_TMEM_S, a, 1024 * c + 2 * k4, b, 512 * c + 2 * k4, id_s, !opens || c > 0 || k4 > 0);
        return true;
      };
      auto step_o = [&](int d, bool opens) {
        const uint32_t a = desc_low(kt, 16384) + 2048 * d, b = desc_low(pt, 16);
#pragma unroll
        for (int jc = 0; jc < 2; ++jc)
#pragma unroll
          for (int k4 = 0; k4 < 4; ++k4)
            mma_at(leader, tmem + d * 64, a, 512 * jc + 128 * k4, b, 512 * jc + 128 * k4, id_o, !opens || jc > 0 || k4 > 0);
        commit_to(leader, &freed[d]);
      };
      bool begins = true, more = true;
      for (int n = 0, piece = 0, moved = 0; more; ++n) {
        if (begins) {  // S^T of a piece's first tile
          if (!wait(q_full, piece)) break;
          if (!step_s(n, 0, true) || !step_s(n, 1, false) || !step_s(n, 2, false) || !step_s(n, 3, false)) break;
          commit_to(leader, s_full);
        }
        const bool ends = w.ends_piece();
        // P^T counts once all warps have written it, unless one of them has found that a reference has to move: then once
        // they have all written it again (which has a barrier of its own: on one, the second writing could end before this
        // warp has seen the first, and parity would not tell)
        if (!wait(p_full, n)) break;
        if (*moving) {
          if (!wait(p_again, moved++)) break;
          *moving = 0;
          __syncwarp();
        }
#pragma unroll
        for (int d = 0; d < 4; ++d) step_o(d, begins);
        if (ends) {
          commit_to(leader, o_full);
          ++piece;
        } else {
          if (!step_s(n + 1, 0, true) || !step_s(n + 1, 1, false) || !step_s(n + 1, 2, false) || !step_s(n + 1, 3, false)) break;
          commit_to(leader, s_full);
        }
        w.next(p);
        more = w.left > 0;
        begins = ends;
      }
      if (more) {  // given up: the products under way still have to end before the block does
        int never = 0;
        commit_to(leader, idle);
        mbar_wait_bounded(idle, 0, &never, PX_WAIT_NS);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    regs_up<PX_REG_SOFT>();
    const int t = tid - PX_PROD, q4 = warp & 3, hb = 32 * ((warp - 8) >> 2), key = 32 * q4 + lane;
    const uint32_t lanes = tmem + (uint32_t(32 * q4) << 16);
    float *mref = reinterpret_cast<float *>(smem + PX_MREF) + 64 * q4 + hb, *nref = reinterpret_cast<float *>(smem + PX_NREF) + 64 * q4 + hb;
    float *oinv = reinterpret_cast<float *>(smem + PX_INV) + 64 * q4 + hb;
    const uint32_t q_at = smem_u32(qmu + hb), r_at = smem_u32(nref);
    float sum_h[32];
#pragma unroll
    for (int h = 0; h < 32; ++h) sum_h[h] = 0.f;
    int piece = 0;
    bool begins = true, alive = true;
    load_query(p, w.row, smem, qmu, warp - 8, lane);
    if (lane == 0) mbar_arrive(q_full);
    for (int n = 0; w.left > 0; ++n) {
      const bool ok = mbar_wait_bounded(s_full, n & 1, abort_flag, PX_WAIT_NS);
      tc_fence_after();
      __syncwarp();
      const bool shared = w.within(limit);
      const float2 m2 = shared ? make_float2(1.f, 1.f) : mul[(n & 1) * 128 + key];
      const bool valid = m2.x == m2.x || m2.y != 0.f;
      const bool plain = shared || __all_sync(0xffffffffu, m2.x == 1.f);  // this warp's keys are all entries
      float s[32];
      // The weights 2^(logit - reference + BIAS) into s and, times the keys' factors, in fp16 into P^T;
      // returns the largest exponent.
      auto weights = [&]() {
        float top = -INFINITY;
#pragma unroll
        for (int g = 0; g < 2; ++g) {  // 16 heads at a time
          tc_ld_32x32b_x16(lanes + PX_TMEM_S + hb + 16 * g, reinterpret_cast<uint32_t(&)[16]>(s[16 * g]));
          tc_wait_ld();
#pragma unroll
          for (int i = 4 * g; i < 4 * g + 4; ++i) {
            float4 q, r;
            lds_pair(q, r, q_at + 16 * i, r_at + 16 * i);
            float x[4] = {s[4 * i], s[4 * i + 1], s[4 * i + 2], s[4 * i + 3]};
            if (!plain) {
#pragma unroll
              for (int e = 0; e < 4; ++e) x[e] *= m2.x;
            }
            // (product and difference rounded one after the other, as the references are formed: a fused one would
            // differ from them by more than the lag where logits are very large)
            mul2(x[0], x[1], q.x, q.y);
            mul2(x[2], x[3], q.z, q.w);
            add2(x[0], x[1], r.x, r.y);
            add2(x[2], x[3], r.z, r.w);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (!plain) x[e] = valid ? x[e] : -INFINITY;
              top = fmaxf(top, x[e]);
              s[4 * i + e] = ex2(x[e]);
            }
          }
          uint32_t ph[8];
#pragma unroll
          for (int h = 0; h < 16; h += 2) {
            const float e0 = s[16 * g + h], e1 = s[16 * g + h + 1];
            const __half2 hp = plain ? __floats2half2_rn(e0, e1) : __floats2half2_rn(e0 * m2.y, e1 * m2.y);
            ph[h >> 1] = *reinterpret_cast<const uint32_t *>(&hp);
          }
#pragma unroll
          for (int u = 0; u < 2; ++u)
            *reinterpret_cast<uint4 *>(smem + PX_P + kmaj128(key, hb / 8 + 2 * g + u)) =
                make_uint4(ph[4 * u], ph[4 * u + 1], ph[4 * u + 2], ph[4 * u + 3]);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        return top;
      };
      // P^T is written before it is known whether a reference has to move; it seldom has, except where a piece
      // begins.  (Once moved the references are the maxima so far: there is no third round.)
      for (int round = begins ? 0 : 1;; ++round) {
        if (round > 0) {
          const float top = weights();
          const bool moves = __any_sync(0xffffffffu, round == 1 && top > PX_LAG + PX_BIAS);
          __syncwarp();  // (the lanes' parts of P^T stand before the arrival)
          if (lane == 0) {  // (the vote below is off the tensor core's path)
            if (moves) *moving = 1;
            mbar_arrive(begins || round == 1 ? p_full : p_again);
          }
          if (!soft_any(!ok || moves)) break;
        }
        // new references; O^T and the sums follow (O^T holds nothing yet where a piece begins)
        tc_ld_32x32b_x32(lanes + PX_TMEM_S + hb, reinterpret_cast<uint32_t(&)[32]>(s));
        tc_wait_ld();
        float most = -INFINITY;  // lane h: the warp's maximum of head hb + h
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float4 q, r;
          lds_pair(q, r, q_at + 16 * i, r_at + 16 * i);
          const float qs[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float m = redux_max(valid ? (s[4 * i + e] * m2.x) * qs[e] : -INFINITY);
            if (lane == 4 * i + e) most = m;
          }
        }
        red[(warp - 8) * 32 + lane] = most;
        if (soft_any(!ok)) {
          alive = false;
          break;
        }
        const float *rg = red + (hb >> 5) * 128;
        most = fmaxf(fmaxf(rg[lane], rg[32 + lane]), fmaxf(rg[64 + lane], rg[96 + lane]));
        const float old = round == 0 ? -INFINITY : mref[lane];
        const float now = fmaxf(old, most);
        const float alpha = old == -INFINITY ? 0.f : ex2(old - now);  // lane h: head hb + h
        mref[lane] = now;  // (every quarter's warps find the same)
        nref[lane] = PX_BIAS - now;
        __syncwarp();
        if (round > 0) {
#pragma unroll
          for (int h = 0; h < 32; ++h) sum_h[h] *= __shfl_sync(0xffffffffu, alpha, h);
#pragma unroll 1
          for (int d = 0; d < 4; ++d) {
            uint32_t r[32];
            tc_ld_32x32b_x32(lanes + d * 64 + hb, r);
            tc_wait_ld();
#pragma unroll
            for (int h = 0; h < 32; ++h) r[h] = __float_as_uint(__uint_as_float(r[h]) * __shfl_sync(0xffffffffu, alpha, h));
            tc_st_32x32b_x32(lanes + d * 64 + hb, r);
          }
          tc_wait_st();
          tc_fence_before();
        }
        round = 1;
      }
      if (!alive) break;
      const bool ends = w.ends_piece();
#pragma unroll
      for (int h = 0; h < 32; h += 2) add2(sum_h[h], sum_h[h + 1], s[h], s[h + 1]);
      begins = ends;
      if (!ends) {
        w.next(p);
        continue;
      }
      // ---- the piece's tiles are done: the next piece begins on the tensor core, then O^T is read
      const int row = w.row;
      // whole, or a part: the row began in an earlier block (slot 0) or only goes on in a later one (slot 1)
      const bool from_start = piece > 0 || first[1] == 0;
      const bool whole = from_start && w.tile + 1 == w.k.tiles;
      sums[(warp - 8) * 32 + lane] = reduce_scatter32<false>(sum_h);
      w.next(p);
      if (w.left > 0) {
        load_query(p, w.row, smem, qmu, warp - 8, lane);
        if (lane == 0) mbar_arrive(q_full);
      }
      const bool o_ok = mbar_wait_bounded(o_full, piece & 1, abort_flag, PX_WAIT_NS);
      tc_fence_after();
      if (soft_any(!o_ok)) {
        alive = false;
        break;
      }
      const float *sg = sums + (hb >> 5) * 128;
      const float total_h = (sg[lane] + sg[32 + lane]) + (sg[64 + lane] + sg[96 + lane]);  // lane h: head hb + h
      float *part = p.parts + (int64_t(blockIdx.x) * 2 + (from_start ? 1 : 0)) * PX_SLOT;
      // 2^7: the tile's values are 2^-7 of the keys'; over the sum where it is whole (0 for no key; NaN stays)
      oinv[lane] = !whole ? 128.f : total_h > 0.f ? 128.f / total_h : total_h;
      __syncwarp();
      const int dim = (key & ~7) + ((key & 7) >> 1) + 4 * (key & 1);  // of this lane's O^T row (see unpack8)
      float ahead[16];
      if (q4 == 0) {
        const float m = mref[lane];
        if (whole) {
          p.lse[int64_t(row) * H + hb + lane] =
              total_h == 0.f ? -INFINITY : (m - PX_BIAS + log2f(total_h)) * 0.69314718055994531f;
        } else {
          part[PX_PART + hb + lane] = m;
          part[PX_PART + H + hb + lane] = total_h;
        }
      }
#pragma unroll 1
      for (int g = 0; g < 8; ++g) {  // 128 dims of 16 heads at a time, the next ones on their way
        const int d = g >> 1, h0 = 16 * (g & 1);
        float r[16];
        if (g == 0) tc_ld_32x32b_x16(lanes + hb, reinterpret_cast<uint32_t(&)[16]>(ahead));
        tc_wait_ld();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 f = reinterpret_cast<const float4 *>(oinv + h0)[i];
          r[4 * i] = ahead[4 * i] * f.x, r[4 * i + 1] = ahead[4 * i + 1] * f.y;
          r[4 * i + 2] = ahead[4 * i + 2] * f.z, r[4 * i + 3] = ahead[4 * i + 3] * f.w;
        }
        if (g < 7)
          tc_ld_32x32b_x16(lanes + ((g + 1) >> 1) * 64 + 16 * ((g + 1) & 1) + hb, reinterpret_cast<uint32_t(&)[16]>(ahead));
        if (whole && p.o_bf16) {
          // lanes l and l ^ 2 hold neighbouring dims: of two heads the first lane stores the one, the second the other
          const bool second = lane & 2;
          uint32_t *orow = reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p.o) +
                                                        (int64_t(row) * H + hb + h0 + (second ? 1 : 0)) * D + 128 * d + (dim & ~1));
#pragma unroll
          for (int h = 0; h < 16; h += 2) {
            const float got = __shfl_xor_sync(0xffffffffu, second ? r[h] : r[h + 1], 2);
            const __nv_bfloat162 v = second ? __floats2bfloat162_rn(got, r[h + 1]) : __floats2bfloat162_rn(r[h], got);
            orow[h * (D / 2)] = *reinterpret_cast<const uint32_t *>(&v);
          }
        } else {
          float *orow = (whole ? static_cast<float *>(p.o) + (int64_t(row) * H + hb + h0) * D : part + (hb + h0) * D) + 128 * d + dim;
#pragma unroll
          for (int h = 0; h < 16; ++h) orow[h * D] = r[h];
        }
      }
      // (the next products into O^T, and the next sums, stand behind the softmax threads' next barrier)
      tc_fence_before();
#pragma unroll
      for (int h = 0; h < 32; ++h) sum_h[h] = 0.f;
      ++piece;
    }
    if (!alive && t == 0) report(p.err, CSA2_ERR_TIMEOUT);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, PX_TMEM_COLS);
  }
}

// Rows whose tiles lie in several blocks: o = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s over their
// partials, in block order; and rows without a key: o = 0, lse = -inf.  One warp per row and head; lane l holds
// dims 4 l + 128 i ..
__global__ void __launch_bounds__(256) prefix_combine_kernel(const __grid_constant__ PrefixArgs p) {
  grid_dep_wait();
  const int row = blockIdx.x, lane = threadIdx.x & 31, h = 8 * blockIdx.y + (threadIdx.x >> 5);
  const int a = p.plan[16 + row], b = p.plan[17 + row], per = p.plan[0], by_row = p.plan[1];
  // the blocks that hold a part of the row: c0 .. c0 + n - 1
  const int c0 = by_row ? row * by_row : a / per;
  const int n = by_row ? part_count(b - a, by_row) : (b > a ? (b - 1) / per - c0 + 1 : 0);
  if (n == 1) return;
  // the first block holds the row's start as its last piece (slot 1), the others as their first (slot 0)
  auto part = [&](int i) { return p.parts + (int64_t(c0 + i) * 2 + (i == 0 ? 1 : 0)) * PX_SLOT; };
  // the statistics of the first 32 parts, and the values of the first four, asked for together
  float m = -INFINITY, l = 0.f;
  if (lane < n) m = part(lane)[PX_PART + h], l = part(lane)[PX_PART + H + h];
  float4 x[4][4];
  auto load = [&](int i0) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i0 + i < n) {
        const float4 *src = reinterpret_cast<const float4 *>(part(i0 + i) + h * D) + lane;
#pragma unroll
        for (int u = 0; u < 4; ++u) x[i][u] = src[32 * u];
      }
  };
  load(0);
  float M = m, L = 0.f;
  for (int i = lane + 32; i < n; i += 32) M = fmaxf(M, part(i)[PX_PART + h]);
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float4 acc[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) acc[u] = make_float4(0.f, 0.f, 0.f, 0.f);
  float w = 0.f;  // lane i: the weight of part i0 + i, and (l) its weighted sum
  for (int i0 = 0; i0 < n; i0 += 4) {
    if ((i0 & 31) == 0) {
      if (i0 > 0) {
        m = -INFINITY, l = 0.f;
        if (i0 + lane < n) m = part(i0 + lane)[PX_PART + h], l = part(i0 + lane)[PX_PART + H + h];
      }
      w = m == -INFINITY ? 0.f : ex2(m - M);
      l = l == 0.f ? 0.f : w * l;  // (a sum that is NaN stays, also under a reference of -inf: all its logits are NaN)
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i0 + i >= n) break;
      const float wi = __shfl_sync(0xffffffffu, w, (i0 + i) & 31);
      L += __shfl_sync(0xffffffffu, l, (i0 + i) & 31);
#pragma unroll
      for (int u = 0; u < 4; ++u)
        acc[u].x += wi * x[i][u].x, acc[u].y += wi * x[i][u].y, acc[u].z += wi * x[i][u].z, acc[u].w += wi * x[i][u].w;
    }
    if (i0 + 4 < n) load(i0 + 4);
  }
  const float s = L > 0.f ? 1.f / L : L;  // (0 for no key; NaN stays)
  if (lane == 0) p.lse[int64_t(row) * H + h] = L == 0.f ? -INFINITY : (M - PX_BIAS + log2f(L)) * 0.69314718055994531f;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int64_t at = (int64_t(row) * H + h) * D + 4 * lane + 128 * u;
    if (p.o_bf16) {
      const __nv_bfloat162 x = __floats2bfloat162_rn(acc[u].x * s, acc[u].y * s), y = __floats2bfloat162_rn(acc[u].z * s, acc[u].w * s);
      *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.o) + at) =
          make_uint2(*reinterpret_cast<const uint32_t *>(&x), *reinterpret_cast<const uint32_t *>(&y));
    } else {
      *reinterpret_cast<float4 *>(static_cast<float *>(p.o) + at) = make_float4(acc[u].x * s, acc[u].y * s, acc[u].z * s, acc[u].w * s);
    }
  }
}

// Blocks of a call: no more than it can have tiles.
int prefix_blocks(int64_t rows, int max_entries, int most) {
  const int64_t tiles = rows * ((int64_t(max_entries) + 128 + PX_TILE - 1) / PX_TILE);
  return int(tiles < most ? tiles : most);
}
size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

// The workspace: the plan, the shared tiles' flags, the partial rows, the shared tiles in fp16.
struct Layout {
  int shared;
  size_t bad, parts, rows16, bytes;
  Layout(int64_t rows, int entries, int blocks) {
    shared = entries / PX_TILE;
    if (rows < PX_MIN_ROWS || rows * shared < PX_MIN_SHARED) shared = 0;
    bad = round256(size_t(rows + 17) * 4);
    parts = bad + round256(size_t(shared) * (PX_TILE / EXPAND) * 4);
    rows16 = parts + round256(size_t(blocks) * 2 * PX_SLOT * 4);
    bytes = rows16 + size_t(shared) * PX_TILE * D * 2;
  }
};
}  // namespace

size_t prefix_workspace(int64_t rows, int max_entries, int prefix) {
  return Layout(rows, prefix < max_entries ? prefix : max_entries, prefix_blocks(rows, max_entries, PX_MAX_CTAS)).bytes;
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
  const int sms = sm_count(), blocks = prefix_blocks(rows, max_entries, sms < PX_MAX_CTAS ? sms : PX_MAX_CTAS);
  const Layout at(rows, prefix < max_entries ? prefix : max_entries, blocks);
  char *w = static_cast<char *>(ws);
  a.plan = reinterpret_cast<int32_t *>(w);
  a.bad = reinterpret_cast<int32_t *>(w + at.bad);
  a.parts = reinterpret_cast<float *>(w + at.parts);
  a.rows16 = reinterpret_cast<uint16_t *>(w + at.rows16);
  CUtensorMap map;
  memset(&map, 0, sizeof(map));
  if (at.shared > 0 && make_half_rows_map(&map, a.rows16, int64_t(at.shared) * PX_TILE)) a.shared = at.shared;
  set_smem_limit(prefix_attn_kernel, PX_SMEM);
  // Every kernel may be launched while the one before it ends: each waits for it before it reads or writes anything.
  cudaLaunchAttribute dependent[1];
  dependent[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  dependent[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = st;
  cfg.attrs = dependent;
  cfg.numAttrs = 1;
  cfg.blockDim = dim3(256);
  if (a.shared > 0) {
    cfg.gridDim = dim3(a.shared * (PX_TILE / EXPAND));
    cudaLaunchKernelEx(&cfg, prefix_expand_kernel, a);
  }
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(PX_THREADS);
  cfg.dynamicSmemBytes = PX_SMEM;
  cudaLaunchKernelEx(&cfg, prefix_attn_kernel, map, a);
  cfg.gridDim = dim3(rows, H / 8);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  cudaLaunchKernelEx(&cfg, prefix_combine_kernel, a);
}

}  // namespace csa2
