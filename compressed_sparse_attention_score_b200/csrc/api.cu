// The C ABI of the CSA2 library: argument checks, workspace carving, launches.
#include <cuda_runtime.h>

#include <cstdio>
#include <string>

#include "../../include/csa2.h"
#include "kernels.cuh"

#define CSA2_EXPORT extern "C" __attribute__((visibility("default")))

namespace {

thread_local std::string g_last_error;

csa2_status fail(csa2_status s, const char *msg) {
  g_last_error = msg;
  return s;
}

csa2_status launched(const char *what) {
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    g_last_error = std::string(what) + ": " + cudaGetErrorString(e);
    return CSA2_ERR_CUDA;
  }
  g_last_error.clear();
  return CSA2_OK;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

csa2_status check_cache(const csa2_cache *c, int B) {
  if (!c) return fail(CSA2_ERR_INVALID_ARG, "cache is NULL");
  if (!c->kv_codes || !c->kv_scales || !c->ix_codes || !c->ix_scales || !c->num_entries)
    return fail(CSA2_ERR_INVALID_ARG, "cache plane or num_entries is NULL");
  if (!aligned16(c->kv_codes) || !aligned16(c->ix_codes) || !aligned16(c->kv_scales) || (reinterpret_cast<uintptr_t>(c->ix_scales) & 3))
    return fail(CSA2_ERR_INVALID_ARG, "cache planes must be 16-byte aligned (ix_scales 4-byte)");
  if (c->ratio < 1) return fail(CSA2_ERR_INVALID_ARG, "cache ratio must be >= 1");
  if (c->num_slots < 0 || c->batch < 0) return fail(CSA2_ERR_INVALID_ARG, "negative cache size");
  if (B > c->batch) return fail(CSA2_ERR_SHAPE, "B exceeds cache batch");
  if (c->page_table) {
    if (c->page_size <= 0 || (c->page_size & (c->page_size - 1)) || c->max_pages <= 0)
      return fail(CSA2_ERR_INVALID_ARG, "paged cache needs a power-of-two page_size and max_pages > 0");
  } else if (c->seq_stride <= 0) {
    return fail(CSA2_ERR_INVALID_ARG, "contiguous cache needs seq_stride > 0");
  }
  return CSA2_OK;
}

size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

// Dense attention runs over segments of csa2::attn_dense_segment() entries (8192, or 4096 on a
// device that cannot hold a 16-CTA cluster); the workspace is sized for the smaller.
constexpr int kDenseMinSegment = 4096;

// Full mode with this many query rows or more (a prefill chunk) and no pool selects with the
// fused prefill indexer: each CTA serves 3 query tokens over every key tile they see, so there
// must be enough of them to fill the device; the scores are never materialised.
constexpr int64_t kFusedPrefillRows = 1024;
bool fused_prefill(int64_t rows, int32_t pool_k) { return rows >= kFusedPrefillRows && pool_k == 0; }

}  // namespace

namespace csa2 {
// Lets other translation units of the library set the thread's error text.
void set_last_error(const char *msg) { g_last_error = msg; }
}  // namespace csa2

CSA2_EXPORT int csa2_version(void) { return 100; }

CSA2_EXPORT const char *csa2_last_error_string(void) { return g_last_error.c_str(); }

CSA2_EXPORT csa2_status csa2_check(const int32_t *err, csa2_stream_t stream) {
  if (!err) return fail(CSA2_ERR_INVALID_ARG, "err is NULL");
  int32_t h = 0;
  cudaError_t e = cudaMemcpyAsync(&h, err, sizeof(h), cudaMemcpyDeviceToHost, stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess) {
    g_last_error = std::string("csa2_check: ") + cudaGetErrorString(e);
    return CSA2_ERR_CUDA;
  }
  return csa2_status(h);
}

CSA2_EXPORT size_t csa2_workspace_size(csa2_mode mode, int32_t B, int32_t Q, int32_t max_entries, int32_t k,
                                       int32_t pool_k) {
  if (B < 0 || Q < 0 || max_entries < 0 || k < 0 || pool_k < 0) return 0;
  const size_t rows = size_t(B) * Q;
  switch (mode) {
    case CSA2_MODE_FULL:
      return (fused_prefill(int64_t(rows), pool_k) ? 0 : round256(rows * max_entries * 4)) + round256(rows * k * 4);
    case CSA2_MODE_REINDEX:  // pools of at most REINDEX_SELECT_MAX: scores never leave the chip
      return (pool_k <= csa2::REINDEX_SELECT_MAX ? 0 : round256(rows * pool_k * 4)) + round256(rows * k * 4);
    case CSA2_MODE_DENSE:  // partial (o, lse) of one key segment beyond the first
      return max_entries > kDenseMinSegment ? round256(rows * CSA2_HEADS * CSA2_MAIN_DIM * 4) +
                                                  round256(rows * CSA2_HEADS * 4)
                                            : 0;
    default: return 0;
  }
}

CSA2_EXPORT csa2_status csa2_pack_kv(const void *lat_kv, const void *lat_ix, csa2_dtype dtype, const float *pool_w,
                                     int32_t B, int32_t T, const int32_t *first_entry, const csa2_cache *cache,
                                     int32_t *err, csa2_stream_t stream) {
  if (B < 0 || T < 0) return fail(CSA2_ERR_INVALID_ARG, "negative size");
  if (B == 0 || T == 0) return CSA2_OK;
  if (csa2_status s = check_cache(cache, B)) return s;
  if (!lat_kv || !lat_ix || !first_entry) return fail(CSA2_ERR_INVALID_ARG, "NULL input");
  if (dtype != CSA2_F32 && dtype != CSA2_BF16) return fail(CSA2_ERR_INVALID_ARG, "bad dtype");
  if (!aligned16(lat_kv) || (reinterpret_cast<uintptr_t>(lat_ix) & 7)) return fail(CSA2_ERR_INVALID_ARG, "latents misaligned");
  csa2::launch_pack_kv(lat_kv, lat_ix, dtype, pool_w, nullptr, nullptr, B, T, first_entry, *cache, err, stream);
  return launched("csa2_pack_kv");
}

CSA2_EXPORT csa2_status csa2_pack_kv_gated(const void *lat_kv, const void *lat_ix, csa2_dtype dtype,
                                           const float *gate_kv, const float *gate_ix, int32_t B, int32_t T,
                                           const int32_t *first_entry, const csa2_cache *cache, int32_t *err,
                                           csa2_stream_t stream) {
  if (B < 0 || T < 0) return fail(CSA2_ERR_INVALID_ARG, "negative size");
  if (B == 0 || T == 0) return CSA2_OK;
  if (csa2_status s = check_cache(cache, B)) return s;
  if (!lat_kv || !lat_ix || !gate_kv || !gate_ix || !first_entry) return fail(CSA2_ERR_INVALID_ARG, "NULL input");
  if (dtype != CSA2_F32 && dtype != CSA2_BF16) return fail(CSA2_ERR_INVALID_ARG, "bad dtype");
  if (!aligned16(lat_kv) || (reinterpret_cast<uintptr_t>(lat_ix) & 7) || !aligned16(gate_kv) || !aligned16(gate_ix))
    return fail(CSA2_ERR_INVALID_ARG, "latents or gates misaligned");
  csa2::launch_pack_kv(lat_kv, lat_ix, dtype, nullptr, gate_kv, gate_ix, B, T, first_entry, *cache, err, stream);
  return launched("csa2_pack_kv_gated");
}

CSA2_EXPORT csa2_status csa2_pack_swa(const void *x, csa2_dtype dtype, int32_t B, int32_t T, const int32_t *pos,
                                      uint8_t *swa_codes, float *swa_scale, int32_t R, int32_t *err,
                                      csa2_stream_t stream) {
  if (B < 0 || T < 0 || R < 1) return fail(CSA2_ERR_INVALID_ARG, "bad size");
  if (B == 0 || T == 0) return CSA2_OK;
  if (!x || !pos || !swa_codes || !swa_scale) return fail(CSA2_ERR_INVALID_ARG, "NULL input");
  if (dtype != CSA2_F32 && dtype != CSA2_BF16) return fail(CSA2_ERR_INVALID_ARG, "bad dtype");
  if (!aligned16(x) || !aligned16(swa_codes)) return fail(CSA2_ERR_INVALID_ARG, "x / swa_codes misaligned");
  csa2::launch_pack_swa(x, dtype, B, T, pos, B, swa_codes, swa_scale, R, err, stream);
  return launched("csa2_pack_swa");
}

CSA2_EXPORT csa2_status csa2_index_score(const uint16_t *q_ix, const uint16_t *w, int32_t B, int32_t Q,
                                         const int32_t *q_pos, const int32_t *cand, int32_t P, int32_t max_entries,
                                         const csa2_cache *cache, float *scores, int32_t *err,
                                         csa2_stream_t stream) {
  if (B < 0 || Q < 0 || max_entries < 0 || (cand && P <= 0)) return fail(CSA2_ERR_INVALID_ARG, "bad size");
  if (B == 0 || Q == 0) return CSA2_OK;
  if (csa2_status s = check_cache(cache, B)) return s;
  if (!q_ix || !w || !q_pos || !scores) return fail(CSA2_ERR_INVALID_ARG, "NULL input");
  if (!aligned16(q_ix)) return fail(CSA2_ERR_INVALID_ARG, "q_ix misaligned");
  const int n_out = cand ? P : max_entries;
  if (size_t(B) * Q > 65535) return fail(CSA2_ERR_UNSUPPORTED, "more than 65535 query rows per call");
  csa2::launch_index_score_mma(q_ix, w, B, Q, q_pos, cand, P, n_out, *cache, scores, err, stream);
  return launched("csa2_index_score");
}

CSA2_EXPORT csa2_status csa2_index_topk(const uint16_t *q_ix, const uint16_t *w, int32_t B, int32_t Q,
                                        const int32_t *q_pos, int32_t k, int32_t max_entries,
                                        const csa2_cache *cache, int32_t *idx, int32_t *err, csa2_stream_t stream) {
  if (B < 0 || Q < 0 || max_entries < 0 || k < 1) return fail(CSA2_ERR_INVALID_ARG, "bad size");
  if (B == 0 || Q == 0) return CSA2_OK;
  if (csa2_status s = check_cache(cache, B)) return s;
  if (!q_ix || !w || !q_pos || !idx) return fail(CSA2_ERR_INVALID_ARG, "NULL input");
  if (k > 512) return fail(CSA2_ERR_UNSUPPORTED, "k > 512");
  if (!aligned16(q_ix)) return fail(CSA2_ERR_INVALID_ARG, "q_ix misaligned");
  if (B > 65535) return fail(CSA2_ERR_UNSUPPORTED, "more than 65535 sequences per call");
  csa2::launch_prefill_index(q_ix, w, B, Q, q_pos, k, max_entries, *cache, idx, err, stream);
  return launched("csa2_index_topk");
}

CSA2_EXPORT csa2_status csa2_topk(const float *scores, const int32_t *n_valid, int32_t R, int32_t N, int32_t k,
                                  int32_t *idx, float *val, int32_t k2, int32_t *idx2, float *val2,
                                  csa2_stream_t stream) {
  if (R < 0 || N < 0 || k < 1 || k2 < 0) return fail(CSA2_ERR_INVALID_ARG, "bad size");
  if (R == 0) return CSA2_OK;
  if (!scores || !idx) return fail(CSA2_ERR_INVALID_ARG, "NULL input");
  if (k2 > 0 && !idx2) return fail(CSA2_ERR_INVALID_ARG, "k2 > 0 needs idx2");
  if (int64_t(R) * 16 > INT32_MAX) return fail(CSA2_ERR_UNSUPPORTED, "too many rows");
  csa2::launch_topk_cluster(scores, n_valid, R, N, k, idx, val, k2, k2 > 0 ? idx2 : nullptr, val2, nullptr, stream);
  return launched("csa2_topk");
}

CSA2_EXPORT csa2_status csa2_sparse_attn(csa2_mode mode, const uint16_t *q, int32_t B, int32_t Q,
                                         const int32_t *q_pos, float softmax_scale, const uint16_t *q_ix,
                                         const uint16_t *w, int32_t k, int32_t pool_k, int32_t *pool_io,
                                         const int32_t *idx_in, int32_t *idx_out, int32_t max_entries,
                                         const csa2_cache *cache, const uint8_t *swa_codes, const float *swa_scale,
                                         int32_t R, int32_t window, const uint16_t *swa_new, float *o, float *lse,
                                         void *ws, size_t ws_bytes, int32_t *err, csa2_stream_t stream) {
  if (B < 0 || Q < 0 || k < 1 || pool_k < 0 || max_entries < 0) return fail(CSA2_ERR_INVALID_ARG, "bad size");
  if (B == 0 || Q == 0) return CSA2_OK;
  if (csa2_status s = check_cache(cache, B)) return s;
  if (!q || !q_pos || !o || !lse) return fail(CSA2_ERR_INVALID_ARG, "NULL input");
  if (k > 512 && mode != CSA2_MODE_DENSE) return fail(CSA2_ERR_UNSUPPORTED, "k > 512");
  if (!aligned16(q)) return fail(CSA2_ERR_INVALID_ARG, "q misaligned");
  if (swa_codes) {
    if (!swa_scale || window < 1 || window > 128 || R < window) return fail(CSA2_ERR_INVALID_ARG, "need 1 <= window <= 128, window <= R");
    if (!aligned16(swa_codes)) return fail(CSA2_ERR_INVALID_ARG, "swa_codes misaligned");
  }
  if (swa_new) {
    if (!swa_codes || Q != 1) return fail(CSA2_ERR_INVALID_ARG, "swa_new needs the window branch and Q == 1");
    if (reinterpret_cast<uintptr_t>(swa_new) & 7) return fail(CSA2_ERR_INVALID_ARG, "swa_new misaligned");
  }
  if (int64_t(B) * Q > 65535 * 16) return fail(CSA2_ERR_UNSUPPORTED, "too many query rows per call");
  const int rows = B * Q;
  const int32_t *idx = nullptr;
  if (mode == CSA2_MODE_DENSE) {
    // every visible entry, in segments of at most `seg` entries; the partials of the segments
    // after the first go through the workspace and are merged into o / lse in place
    const int seg = csa2::attn_dense_segment();
    if (max_entries > seg) {
      if (!ws || ws_bytes < csa2_workspace_size(mode, B, Q, max_entries, k, pool_k))
        return fail(CSA2_ERR_INVALID_ARG, "workspace too small");
    }
    float *po = static_cast<float *>(ws);
    float *pl = reinterpret_cast<float *>(static_cast<char *>(ws) + round256(size_t(rows) * CSA2_HEADS * CSA2_MAIN_DIM * 4));
    for (int s = 0, e0 = 0; s == 0 || e0 < max_entries; ++s, e0 += seg) {
      const int e1 = e0 + seg < max_entries ? e0 + seg : max_entries;
      csa2::launch_attn_mma(q, B, Q, q_pos, softmax_scale, nullptr, 0, true, e0, e1, max_entries, cache,
                            s == 0 ? swa_codes : nullptr, s == 0 && swa_codes ? swa_scale : nullptr, R, window,
                            s == 0 ? o : po, s == 0 ? lse : pl, err, stream, s == 0 ? swa_new : nullptr);
      if (s > 0) csa2::launch_merge(o, lse, po, pl, int64_t(rows) * CSA2_HEADS, CSA2_MAIN_DIM, o, lse, stream);
    }
    return launched("csa2_sparse_attn");
  }
  if (mode == CSA2_MODE_REUSE) {
    if (!idx_in) return fail(CSA2_ERR_INVALID_ARG, "REUSE needs idx_in");
    idx = idx_in;
  } else if (mode == CSA2_MODE_FULL || mode == CSA2_MODE_REINDEX) {
    if (!q_ix || !w) return fail(CSA2_ERR_INVALID_ARG, "FULL/REINDEX need q_ix and w");
    if (!aligned16(q_ix)) return fail(CSA2_ERR_INVALID_ARG, "q_ix misaligned");
    if (mode == CSA2_MODE_REINDEX && (!pool_io || pool_k < 1)) return fail(CSA2_ERR_INVALID_ARG, "REINDEX needs pool_io and pool_k");
    if (mode == CSA2_MODE_FULL && pool_k > 0 && !pool_io) return fail(CSA2_ERR_INVALID_ARG, "pool_k > 0 needs pool_io");
    const size_t need = csa2_workspace_size(mode, B, Q, max_entries, k, pool_k);
    if (!ws || ws_bytes < need) return fail(CSA2_ERR_INVALID_ARG, "workspace too small");
    if (mode == CSA2_MODE_FULL && fused_prefill(rows, pool_k)) {
      // a prefill chunk: fused indexer + causal top-k, no score matrix
      int32_t *sel = idx_out ? idx_out : static_cast<int32_t *>(ws);
      csa2::launch_prefill_index(q_ix, w, B, Q, q_pos, k, max_entries, *cache, sel, err, stream);
      csa2::launch_attn_mma(q, B, Q, q_pos, softmax_scale, sel, k, false, 0, 0, 0, cache, swa_codes,
                            swa_codes ? swa_scale : nullptr, R, window, o, lse, err, stream, swa_new);
      return launched("csa2_sparse_attn");
    }
    const int n_out = mode == CSA2_MODE_FULL ? max_entries : pool_k;
    if (rows > 65535) return fail(CSA2_ERR_UNSUPPORTED, "more than 65535 query rows per call");
    const bool fused_select = mode == CSA2_MODE_REINDEX && pool_k <= csa2::REINDEX_SELECT_MAX;
    float *scores = static_cast<float *>(ws);
    int32_t *sel = reinterpret_cast<int32_t *>(static_cast<char *>(ws) +
                                               (fused_select ? 0 : round256(size_t(rows) * n_out * 4)));
    if (idx_out) sel = idx_out;
    if (mode == CSA2_MODE_FULL) {
      csa2::launch_index_score_mma(q_ix, w, B, Q, q_pos, nullptr, 0, max_entries, *cache, scores, err, stream);
      csa2::launch_topk_cluster(scores, nullptr, rows, max_entries, k, sel, nullptr, pool_k,
                                pool_k > 0 ? pool_io : nullptr, nullptr, nullptr, stream);
    } else if (fused_select) {
      csa2::launch_reindex_select(q_ix, w, B, Q, q_pos, pool_io, pool_k, k, *cache, sel, err, stream);
    } else {
      csa2::launch_index_score_mma(q_ix, w, B, Q, q_pos, pool_io, pool_k, pool_k, *cache, scores, err, stream);
      csa2::launch_topk_cluster(scores, nullptr, rows, pool_k, k, sel, nullptr, 0, nullptr, nullptr, pool_io, stream);
    }
    idx = sel;
  } else {
    return fail(CSA2_ERR_INVALID_ARG, "bad mode");
  }
  // (a programmatic dependent launch after the selection measured no faster here: 0.390 against
  // 0.389 ms on the hier1m step, 62 against 53 us on one-query Full decode)
  csa2::launch_attn_mma(q, B, Q, q_pos, softmax_scale, idx, k, false, 0, 0, 0, cache, swa_codes,
                        swa_codes ? swa_scale : nullptr, R, window, o, lse, err, stream, swa_new);
  return launched("csa2_sparse_attn");
}

CSA2_EXPORT csa2_status csa2_swa_attn(const uint16_t *q, int32_t B, int32_t Q, const int32_t *q_pos,
                                      const uint8_t *swa_codes, const float *swa_scale, int32_t R, int32_t window,
                                      float softmax_scale, float *o, float *lse, int32_t *err, csa2_stream_t stream) {
  if (B < 0 || Q < 0 || window < 1 || R < window) return fail(CSA2_ERR_INVALID_ARG, "need 1 <= window <= R");
  if (B == 0 || Q == 0) return CSA2_OK;
  if (!q || !q_pos || !swa_codes || !swa_scale || !o || !lse) return fail(CSA2_ERR_INVALID_ARG, "NULL input");
  if (window > 128) return fail(CSA2_ERR_UNSUPPORTED, "window > 128");
  if (!aligned16(swa_codes) || !aligned16(q)) return fail(CSA2_ERR_INVALID_ARG, "swa_codes / q misaligned");
  if (int64_t(B) * Q > 65535 * 16) return fail(CSA2_ERR_UNSUPPORTED, "too many query rows per call");
  csa2::launch_attn_mma(q, B, Q, q_pos, softmax_scale, nullptr, 0, false, 0, 0, 0, nullptr, swa_codes, swa_scale, R,
                        window, o, lse, err, stream);
  return launched("csa2_swa_attn");
}

CSA2_EXPORT csa2_status csa2_merge(const float *o1, const float *l1, const float *o2, const float *l2, int64_t rows,
                                   int32_t D, float *o, float *lse, csa2_stream_t stream) {
  if (rows < 0 || D < 4 || (D & 3)) return fail(CSA2_ERR_INVALID_ARG, "D must be a positive multiple of 4");
  if (rows == 0) return CSA2_OK;
  if (!o1 || !l1 || !o2 || !l2 || !o || !lse) return fail(CSA2_ERR_INVALID_ARG, "NULL input");
  if (!aligned16(o1) || !aligned16(o2) || !aligned16(o)) return fail(CSA2_ERR_INVALID_ARG, "o misaligned");
  csa2::launch_merge(o1, l1, o2, l2, rows, D, o, lse, stream);
  return launched("csa2_merge");
}

// ---------------------------------------------------------------- rotary positions
namespace {

bool aligned8(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 7) == 0; }
bool is_dtype(csa2_dtype t) { return t == CSA2_F32 || t == CSA2_BF16; }

// A rotation of heads (or values) of `dim` dims.
csa2_status check_rotary(const csa2_rotary *r, int dim) {
  if (!r->step || !aligned8(r->step)) return fail(CSA2_ERR_INVALID_ARG, "rotary step is NULL or misaligned");
  if (r->layout != CSA2_ROTARY_INTERLEAVED && r->layout != CSA2_ROTARY_HALF)
    return fail(CSA2_ERR_INVALID_ARG, "bad rotary layout");
  if (r->rot_dim < 2 || (r->rot_dim & 1)) return fail(CSA2_ERR_INVALID_ARG, "rot_dim must be even and at least 2");
  if (r->first < 0 || r->rot_dim > dim || r->first > dim - r->rot_dim)
    return fail(CSA2_ERR_SHAPE, "rotated dims outside the head");
  if (!(r->scale - r->scale == 0.f)) return fail(CSA2_ERR_INVALID_ARG, "rotary scale must be finite");
  return CSA2_OK;
}

csa2_status check_rotary_write(const csa2_rotary *kv, const csa2_rotary *ix, const void *kv_hat, const void *ix_hat) {
  if (kv)
    if (csa2_status s = check_rotary(kv, CSA2_MAIN_DIM)) return s;
  if (ix)
    if (csa2_status s = check_rotary(ix, CSA2_IX_DIM)) return s;
  if (!aligned16(kv_hat) || !aligned8(ix_hat)) return fail(CSA2_ERR_INVALID_ARG, "kv_hat / ix_hat misaligned");
  return CSA2_OK;
}

// Whether the heads of `out` lie apart from one another, tokens outermost or heads outermost.
bool heads_apart(int64_t ts, int64_t hs, int64_t tokens, int64_t heads, int64_t dim) {
  const bool by_token = (heads == 1 || hs >= dim) && (tokens == 1 || ts >= (heads - 1) * hs + dim);
  const bool by_head = (tokens == 1 || ts >= dim) && (heads == 1 || hs >= (tokens - 1) * ts + dim);
  return by_token || by_head;
}

}  // namespace

CSA2_EXPORT csa2_status csa2_rotary_table(int32_t rot_dim, double base, csa2_rotary_scaling scaling, double factor,
                                          int32_t original_len, double beta_fast, double beta_slow, uint64_t *step,
                                          float *scale) {
  if (!step) return fail(CSA2_ERR_INVALID_ARG, "step is NULL");
  if (rot_dim < 2 || (rot_dim & 1)) return fail(CSA2_ERR_INVALID_ARG, "rot_dim must be even and at least 2");
  if (scaling < CSA2_ROTARY_NONE || scaling > CSA2_ROTARY_YARN) return fail(CSA2_ERR_INVALID_ARG, "bad rotary scaling");
  const double most = 1.7976931348623157e308;
  if (!(base > 1.0 && base <= most) || !(factor >= 1.0 && factor <= most))
    return fail(CSA2_ERR_INVALID_ARG, "need base > 1 and factor >= 1");
  if (scaling == CSA2_ROTARY_NTK && rot_dim == 2) return fail(CSA2_ERR_INVALID_ARG, "NTK scaling needs rot_dim > 2");
  if (scaling == CSA2_ROTARY_YARN && !(original_len > 0 && beta_slow > 0.0 && beta_fast > beta_slow && beta_fast <= most))
    return fail(CSA2_ERR_INVALID_ARG, "YaRN needs original_len > 0 and beta_fast > beta_slow > 0");
  csa2::rotary_table(rot_dim, base, scaling, factor, original_len, beta_fast, beta_slow, step, scale);
  return CSA2_OK;
}

CSA2_EXPORT csa2_status csa2_rotate(const void *x, csa2_dtype x_dtype, int64_t x_token_stride, int64_t x_head_stride,
                                    void *out, csa2_dtype out_dtype, int64_t out_token_stride, int64_t out_head_stride,
                                    int32_t tokens, int32_t heads, int32_t dim, const int32_t *pos,
                                    const csa2_rotary *rot, int32_t inverse, csa2_stream_t stream) {
  if (tokens < 0 || heads < 0 || dim < 1) return fail(CSA2_ERR_INVALID_ARG, "bad size");
  if (tokens == 0 || heads == 0) return CSA2_OK;
  if (!x || !out || !pos || !rot) return fail(CSA2_ERR_INVALID_ARG, "NULL input");
  if (!is_dtype(x_dtype) || !is_dtype(out_dtype)) return fail(CSA2_ERR_INVALID_ARG, "bad dtype");
  if (csa2_status s = check_rotary(rot, dim)) return s;
  if ((reinterpret_cast<uintptr_t>(x) & (x_dtype == CSA2_F32 ? 3 : 1)) ||
      (reinterpret_cast<uintptr_t>(out) & (out_dtype == CSA2_F32 ? 3 : 1)))
    return fail(CSA2_ERR_INVALID_ARG, "x / out misaligned");
  if (x_token_stride < 0 || x_head_stride < 0 || out_token_stride < 0 || out_head_stride < 0)
    return fail(CSA2_ERR_INVALID_ARG, "negative stride");
  if (!heads_apart(out_token_stride, out_head_stride, tokens, heads, dim))
    return fail(CSA2_ERR_SHAPE, "the heads of out overlap");
  if (x == out && (x_dtype != out_dtype || x_token_stride != out_token_stride || x_head_stride != out_head_stride))
    return fail(CSA2_ERR_INVALID_ARG, "in place needs the same type and strides");
  csa2::launch_rotate(x, x_dtype, x_token_stride, x_head_stride, out, out_dtype, out_token_stride, out_head_stride,
                      tokens, heads, dim, pos, *rot, inverse != 0, stream);
  return launched("csa2_rotate");
}

CSA2_EXPORT csa2_status csa2_pack_kv_rotary(const void *lat_kv, const void *lat_ix, csa2_dtype dtype,
                                            const float *pool_w, const float *gate_kv, const float *gate_ix, int32_t B,
                                            int32_t T, const int32_t *first_entry, const csa2_rotary *rot_kv,
                                            const csa2_rotary *rot_ix, const csa2_cache *cache, uint16_t *kv_hat,
                                            uint16_t *ix_hat, int32_t *err, csa2_stream_t stream) {
  if (B < 0 || T < 0) return fail(CSA2_ERR_INVALID_ARG, "negative size");
  if (B == 0 || T == 0) return CSA2_OK;
  if (csa2_status s = check_cache(cache, B)) return s;
  if (!lat_kv || !lat_ix || !first_entry) return fail(CSA2_ERR_INVALID_ARG, "NULL input");
  if (!is_dtype(dtype)) return fail(CSA2_ERR_INVALID_ARG, "bad dtype");
  if ((gate_kv != nullptr) != (gate_ix != nullptr) || (gate_kv && pool_w))
    return fail(CSA2_ERR_INVALID_ARG, "give gate_kv and gate_ix together, and no pool_w with them");
  if (!aligned16(lat_kv) || (dtype == CSA2_F32 ? !aligned16(lat_ix) : !aligned8(lat_ix)) || !aligned16(gate_kv) ||
      !aligned16(gate_ix))
    return fail(CSA2_ERR_INVALID_ARG, "latents or gates misaligned");
  if (csa2_status s = check_rotary_write(rot_kv, rot_ix, kv_hat, ix_hat)) return s;
  if (int64_t(B) * (T / cache->ratio) > int64_t(INT32_MAX) * 8) return fail(CSA2_ERR_UNSUPPORTED, "too many entries per call");
  csa2::launch_pack_kv_rotary(lat_kv, lat_ix, dtype, pool_w, gate_kv, gate_ix, B, T, first_entry, rot_kv, rot_ix,
                              *cache, kv_hat, ix_hat, err, stream);
  return launched("csa2_pack_kv_rotary");
}

CSA2_EXPORT csa2_status csa2_append_kv_rotary(const void *lat_kv, const void *lat_ix, csa2_dtype dtype, int32_t B,
                                              const int32_t *pos, float *stage, const csa2_rotary *rot_kv,
                                              const csa2_rotary *rot_ix, const csa2_cache *cache, uint16_t *kv_hat,
                                              uint16_t *ix_hat, int32_t *err, csa2_stream_t stream) {
  if (B < 0) return fail(CSA2_ERR_INVALID_ARG, "negative size");
  if (B == 0) return CSA2_OK;
  if (csa2_status s = check_cache(cache, B)) return s;
  if (!lat_kv || !lat_ix || !pos) return fail(CSA2_ERR_INVALID_ARG, "NULL input");
  if (!is_dtype(dtype)) return fail(CSA2_ERR_INVALID_ARG, "bad dtype");
  if (!aligned16(lat_kv) || (dtype == CSA2_F32 ? !aligned16(lat_ix) : !aligned8(lat_ix)))
    return fail(CSA2_ERR_INVALID_ARG, "latents misaligned");
  if (cache->ratio > 1 && (!stage || !aligned16(stage)))
    return fail(CSA2_ERR_INVALID_ARG, "ratio > 1 needs a 16-byte aligned staging buffer");
  if (csa2_status s = check_rotary_write(rot_kv, rot_ix, kv_hat, ix_hat)) return s;
  csa2::launch_append_kv_rotary(lat_kv, lat_ix, dtype, B, pos, stage,
                                int64_t(cache->ratio) * (CSA2_MAIN_DIM + CSA2_IX_DIM), rot_kv, rot_ix, *cache,
                                const_cast<int32_t *>(cache->num_entries), kv_hat, ix_hat, err, stream);
  return launched("csa2_append_kv_rotary");
}

CSA2_EXPORT csa2_status csa2_pack_swa_rotary(const void *x, csa2_dtype dtype, int32_t B, int32_t T, const int32_t *pos,
                                             const csa2_rotary *rot, uint8_t *swa_codes, float *swa_scale, int32_t R,
                                             int32_t *err, csa2_stream_t stream) {
  if (B < 0 || T < 0 || R < 1) return fail(CSA2_ERR_INVALID_ARG, "bad size");
  if (B == 0 || T == 0) return CSA2_OK;
  if (!x || !pos || !rot || !swa_codes || !swa_scale) return fail(CSA2_ERR_INVALID_ARG, "NULL input");
  if (!is_dtype(dtype)) return fail(CSA2_ERR_INVALID_ARG, "bad dtype");
  if (!aligned16(x) || !aligned16(swa_codes)) return fail(CSA2_ERR_INVALID_ARG, "x / swa_codes misaligned");
  if (csa2_status s = check_rotary(rot, CSA2_SWA_DIM)) return s;
  if (int64_t(B) * T > int64_t(INT32_MAX) * 8) return fail(CSA2_ERR_UNSUPPORTED, "too many tokens per call");
  csa2::launch_pack_swa_rotary(x, dtype, B, T, pos, *rot, swa_codes, swa_scale, R, err, stream);
  return launched("csa2_pack_swa_rotary");
}

// ---------------------------------------------------------------- attention over a shared prefix
CSA2_EXPORT size_t csa2_prefix_workspace_size(int32_t B, int32_t Q, int32_t max_entries) {
  if (B <= 0 || Q <= 0 || max_entries < 0) return 0;
  return csa2::prefix_workspace(int64_t(B) * Q, max_entries, max_entries);
}

CSA2_EXPORT size_t csa2_prefix_workspace_bytes(int32_t B, int32_t Q, int32_t max_entries, int32_t prefix_entries) {
  if (B <= 0 || Q <= 0 || max_entries < 0 || prefix_entries < 0) return 0;
  return csa2::prefix_workspace(int64_t(B) * Q, max_entries, prefix_entries);
}

CSA2_EXPORT csa2_status csa2_prefix_attn(const uint16_t *q, int32_t B, int32_t Q, const int32_t *q_pos,
                                         float softmax_scale, int32_t prefix_entries, int32_t max_entries,
                                         const csa2_cache *cache, const uint8_t *swa_codes, const float *swa_scale,
                                         int32_t R, int32_t window, void *o, csa2_dtype o_dtype, float *lse, void *ws,
                                         size_t ws_bytes, int32_t *err, csa2_stream_t stream) {
  if (B < 0 || Q < 0 || prefix_entries < 0 || max_entries < 0) return fail(CSA2_ERR_INVALID_ARG, "negative size");
  if (B == 0 || Q == 0) return CSA2_OK;
  if (csa2_status s = check_cache(cache, B)) return s;
  if (!q || !q_pos || !o || !lse) return fail(CSA2_ERR_INVALID_ARG, "NULL input");
  if (!is_dtype(o_dtype)) return fail(CSA2_ERR_INVALID_ARG, "bad dtype");
  if (!aligned16(q) || !aligned16(o)) return fail(CSA2_ERR_INVALID_ARG, "q / o misaligned");
  if (swa_codes) {
    if (!swa_scale || window < 1 || window > 128 || R < window)
      return fail(CSA2_ERR_INVALID_ARG, "need 1 <= window <= 128, window <= R");
    if (!aligned16(swa_codes)) return fail(CSA2_ERR_INVALID_ARG, "swa_codes misaligned");
  }
  if (!(softmax_scale - softmax_scale == 0.f)) return fail(CSA2_ERR_INVALID_ARG, "softmax_scale must be finite");
  // (key tiles are counted in 32 bits)
  if (int64_t(B) * Q > 65535 * 16 || int64_t(B) * Q * ((int64_t(max_entries) + 255) / 128) > INT32_MAX / 2)
    return fail(CSA2_ERR_UNSUPPORTED, "too many query rows per call");
  if (!ws || !aligned16(ws) || ws_bytes < csa2_prefix_workspace_bytes(B, Q, max_entries, prefix_entries))
    return fail(CSA2_ERR_INVALID_ARG, "workspace too small or misaligned");
  csa2::launch_prefix_attn(q, B, Q, q_pos, softmax_scale, prefix_entries, max_entries, *cache, swa_codes, swa_scale, R,
                           window, o, o_dtype == CSA2_BF16, lse, ws, err, stream);
  return launched("csa2_prefix_attn");
}
