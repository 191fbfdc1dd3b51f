// The C ABI of the KV cache: argument checks and dispatch.  Every exported
// function is declared in include/attn25.h.
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include <cuda.h>
#include <cuda_runtime.h>

#include "api_common.h"
#include "attn25.h"
#include "cache.h"

namespace attn25 {

namespace {

bool strides_ok(const attn_strides& s) {
  return s.b >= 8 && s.h >= 8 && s.s >= 8 && s.b % 8 == 0 && s.h % 8 == 0 && s.s % 8 == 0;
}

// Sizes, page table and lengths of a cache (the pools only where they are used).
int check_cache(const attn_cache* c, bool pools) {
  if (c == nullptr || c->lens == nullptr) return ATTN_ERR_ARG;
  if (c->B < 1 || c->Hkv < 1 || c->num_pages < 1 || c->page_size < 1 || c->max_pages < 1) return ATTN_ERR_ARG;
  if (c->D != 64 && c->D != 128) return ATTN_ERR_UNSUPPORTED;
  if (!page_size_ok(c->page_size)) return ATTN_ERR_UNSUPPORTED;
  if (static_cast<long long>(c->max_pages) * c->page_size > kMaxCapacity) return ATTN_ERR_UNSUPPORTED;
  if (c->B > 65535 || c->Hkv > 65535 || static_cast<long long>(c->B) * c->Hkv > 65535) return ATTN_ERR_UNSUPPORTED;
  if (!aligned4(c->lens) || !aligned4(c->page_table)) return ATTN_ERR_ALIGN;
  if (pools) {
    if (c->k == nullptr || c->v == nullptr) return ATTN_ERR_ARG;
    if (!aligned16(c->k) || !aligned16(c->v)) return ATTN_ERR_ALIGN;
    if (!strides_ok(c->k_strides) || !strides_ok(c->v_strides)) return ATTN_ERR_ALIGN;
  }
  return ATTN_OK;
}

CacheIndex index_of(const attn_cache* c) {
  return CacheIndex{c->page_table, c->lens, c->B, c->Hkv, c->num_pages, c->page_size, c->max_pages,
                    c->max_pages * c->page_size};
}

CacheDev cache_dev(const attn_cache* c, const DeviceInfo* d) {
  CacheDev r{};
  r.k = reinterpret_cast<__nv_bfloat16*>(c->k);
  r.v = reinterpret_cast<__nv_bfloat16*>(c->v);
  r.k_st = Strides{c->k_strides.b, c->k_strides.h, c->k_strides.s};
  r.v_st = Strides{c->v_strides.b, c->v_strides.h, c->v_strides.s};
  r.ix = index_of(c);
  r.D = c->D;
  r.status = d->status;
  return r;
}

// Query heads, scale and mod of a call that scores against a cache: no mod, or softcap.
int check_scores(const attn_cache* c, int Hq, float scale, int mod_kind, const attn_mod_params* mp, float& softcap) {
  if (Hq < 1 || Hq % c->Hkv != 0) return ATTN_ERR_ARG;
  if (static_cast<long long>(c->B) * Hq > (1 << 24)) return ATTN_ERR_UNSUPPORTED;
  if (!(scale > 0.f) || !std::isfinite(scale)) return ATTN_ERR_ARG;
  ModSpec ms;
  if (!split_mod(mod_kind, ms)) return ATTN_ERR_ARG;
  if (ms.mask != 0 || (ms.score != MOD_NONE && ms.score != MOD_SOFTCAP)) return ATTN_ERR_UNSUPPORTED;
  softcap = 0.f;
  if (ms.score == MOD_SOFTCAP) {
    if (mp == nullptr || !(mp->softcap > 0.f) || !std::isfinite(mp->softcap)) return ATTN_ERR_ARG;
    softcap = mp->softcap;
  }
  return ATTN_OK;
}

// q as (D, head, token, row), one query tile to a box
bool encode_query_tiles(CUtensorMap* m, const void* q, const attn_cache* c, int Hq, int T, const Strides& st) {
  const RowTiles rt = row_tiles(Hq / c->Hkv, T);
  return encode_bf16_dims(m, q, {c->D, Hq, T, c->B}, {st.h, st.s, st.b}, rt.head_tile, rt.tok_tile);
}

// a pool as (D, row of the page, head, page), min(page_size, 128) rows to a box
bool encode_pool(CUtensorMap* m, const void* pool, const attn_cache* c, const Strides& st) {
  return encode_bf16_4d(m, pool, c->D, c->page_size, c->Hkv, c->num_pages, st, c->page_size < TILE ? c->page_size : TILE);
}

// Do two int32 arrays of n entries share memory?
bool rows_meet(const int32_t* x, const int32_t* y, int n) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(y);
  return (a < b ? b - a : a - b) < static_cast<uintptr_t>(n) * sizeof(int32_t);
}

int launched(cudaError_t e) { return e == cudaSuccess ? ATTN_OK : ATTN_ERR_LAUNCH; }

}  // namespace

}  // namespace attn25

using namespace attn25;

extern "C" {

int attn_cache_append(const attn_cache* cache, const attn_bf16* k_new, const attn_bf16* v_new, int32_t* lens_out,
                      const int32_t* path, const int32_t* counts, int T, const attn_layouts* layouts,
                      int32_t* positions, const int32_t* seen, attn_stream_t stream) {
  int rc = check_cache(cache, true);
  if (rc != ATTN_OK) return rc;
  if (k_new == nullptr || v_new == nullptr || T < 1) return ATTN_ERR_ARG;
  if (T > kMaxCapacity) return ATTN_ERR_UNSUPPORTED;
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned4(lens_out) || !aligned4(path) || !aligned4(counts) ||
      !aligned4(positions) || !aligned4(seen))
    return ATTN_ERR_ALIGN;
  if (lens_out == nullptr) lens_out = cache->lens;
  bool late = false;
  for (const int32_t* read : {static_cast<const int32_t*>(cache->lens), counts, seen}) {
    late = late || lens_out == read;
    if (read != nullptr && lens_out != read && rows_meet(lens_out, read, cache->B)) return ATTN_ERR_ARG;
  }
  AppendArgs a{};
  if (!layout_of(layouts ? &layouts->k : nullptr, cache->Hkv, T, cache->D, a.kn_st) ||
      !layout_of(layouts ? &layouts->v : nullptr, cache->Hkv, T, cache->D, a.vn_st))
    return ATTN_ERR_ALIGN;
  DeviceInfo* d = nullptr;
  rc = current_device(&d);
  if (rc != ATTN_OK) return rc;
  a.c = cache_dev(cache, d);
  a.k_new = reinterpret_cast<const __nv_bfloat16*>(k_new);
  a.v_new = reinterpret_cast<const __nv_bfloat16*>(v_new);
  a.path = path;
  a.counts = counts;
  a.seen = seen;
  a.positions = positions;
  a.lens_out = lens_out;
  a.late = late;
  a.T = T;
  return launched(launch_cache_append(a, d->sms, reinterpret_cast<cudaStream_t>(stream)));
}

size_t attn_tree_workspace_size(int Hq, int Hkv, int T, int D) {
  if (Hkv < 1 || Hq < 1 || Hq % Hkv != 0 || T < 1 || T > kMaxTreeTokens || (D != 64 && D != 128)) return 0;
  return tree_workspace_bytes(Hq / Hkv, T, D);
}

int attn_tree_fwd(const attn_bf16* q, const attn_bf16* k_new, const attn_bf16* v_new, const attn_cache* cache,
                  attn_bf16* out, float* lse, void* workspace, size_t workspace_bytes, const int32_t* parents,
                  const int32_t* counts, int Hq, int T, float scale, int mod_kind, const attn_mod_params* mod_params,
                  const attn_layouts* layouts, attn_stream_t stream) {
  int rc = check_cache(cache, true);
  if (rc != ATTN_OK) return rc;
  if (q == nullptr || out == nullptr || workspace == nullptr || T < 1) return ATTN_ERR_ARG;
  if ((k_new == nullptr) != (v_new == nullptr) || (k_new == nullptr && parents != nullptr)) return ATTN_ERR_ARG;
  if (T > kMaxTreeTokens) return ATTN_ERR_UNSUPPORTED;
  TreeArgs a{};
  rc = check_scores(cache, Hq, scale, mod_kind, mod_params, a.softcap);
  if (rc != ATTN_OK) return rc;
  if (!aligned16(q) || !aligned16(k_new) || !aligned16(v_new) || !aligned16(out) || !aligned4(lse) ||
      !aligned4(parents) || !aligned4(counts) || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return ATTN_ERR_ALIGN;
  if (!layout_of(layouts ? &layouts->q : nullptr, Hq, T, cache->D, a.q_st) ||
      !layout_of(layouts ? &layouts->out : nullptr, Hq, T, cache->D, a.o_st) ||
      !layout_of(layouts && k_new ? &layouts->k : nullptr, cache->Hkv, T, cache->D, a.kn_st) ||
      !layout_of(layouts && k_new ? &layouts->v : nullptr, cache->Hkv, T, cache->D, a.vn_st))
    return ATTN_ERR_ALIGN;
  if (workspace_bytes < attn_tree_workspace_size(Hq, cache->Hkv, T, cache->D)) return ATTN_ERR_WORKSPACE;
  DeviceInfo* d = nullptr;
  rc = current_device(&d);
  if (rc != ATTN_OK) return rc;
  a.c = cache_dev(cache, d);
  a.q = reinterpret_cast<const __nv_bfloat16*>(q);
  a.k_new = reinterpret_cast<const __nv_bfloat16*>(k_new);
  a.v_new = reinterpret_cast<const __nv_bfloat16*>(v_new);
  a.out = reinterpret_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.parents = parents;
  a.counts = counts;
  a.Hq = Hq;
  a.G = Hq / cache->Hkv;
  a.T = T;
  a.scale = scale;
  TreeMaps m{};
  if (!encode_query_tiles(&m.q, q, cache, Hq, T, a.q_st) || !encode_pool(&m.k, cache->k, cache, a.c.k_st) ||
      !encode_pool(&m.v, cache->v, cache, a.c.v_st))
    return ATTN_ERR_ARG;
  if (k_new != nullptr && (!encode_bf16_4d(&m.kn, k_new, cache->D, T, cache->Hkv, cache->B, a.kn_st, TILE) ||
                           !encode_bf16_4d(&m.vn, v_new, cache->D, T, cache->Hkv, cache->B, a.vn_st, TILE)))
    return ATTN_ERR_ARG;
  return launched(launch_tree(m, a, workspace, wait_ns(), reinterpret_cast<cudaStream_t>(stream)));
}

int attn_cache_weights(const attn_bf16* q, const float* lse, const attn_cache* cache, const float* weights_in,
                       float* weights_out, const int32_t* path, const int32_t* counts, int Hq, int T, float scale,
                       int mod_kind, const attn_mod_params* mod_params, const attn_layouts* layouts,
                       attn_stream_t stream) {
  int rc = check_cache(cache, true);
  if (rc != ATTN_OK) return rc;
  if (q == nullptr || lse == nullptr || weights_out == nullptr || T < 1) return ATTN_ERR_ARG;
  if (T > 262144) return ATTN_ERR_UNSUPPORTED;
  WeightsArgs a{};
  rc = check_scores(cache, Hq, scale, mod_kind, mod_params, a.softcap);
  if (rc != ATTN_OK) return rc;
  if (!aligned16(q) || !aligned4(lse) || !aligned4(weights_in) || !aligned4(weights_out) || !aligned4(path) ||
      !aligned4(counts))
    return ATTN_ERR_ALIGN;
  if (!layout_of(layouts ? &layouts->q : nullptr, Hq, T, cache->D, a.q_st)) return ATTN_ERR_ALIGN;
  DeviceInfo* d = nullptr;
  rc = current_device(&d);
  if (rc != ATTN_OK) return rc;
  a.c = cache_dev(cache, d);
  a.q = reinterpret_cast<const __nv_bfloat16*>(q);
  a.lse = lse;
  a.w_in = weights_in;
  a.w_out = weights_out;
  a.path = path;
  a.counts = counts;
  a.Hq = Hq;
  a.G = Hq / cache->Hkv;
  a.T = T;
  a.scale = scale;
  CUtensorMap tq, tk;
  if (!encode_query_tiles(&tq, q, cache, Hq, T, a.q_st) || !encode_pool(&tk, cache->k, cache, a.c.k_st)) return ATTN_ERR_ARG;
  return launched(launch_cache_weights(tq, tk, a, wait_ns(), d->sms, reinterpret_cast<cudaStream_t>(stream)));
}

int attn_evict_plan(const attn_cache* cache, const float* weights, const int32_t* positions, const int32_t* seen,
                    int32_t* moves, int32_t* n_moves, int budget, int first, int recent, attn_stream_t stream) {
  int rc = check_cache(cache, false);
  if (rc != ATTN_OK) return rc;
  if (weights == nullptr || positions == nullptr || seen == nullptr || moves == nullptr || n_moves == nullptr)
    return ATTN_ERR_ARG;
  if (budget < 1 || first < 0 || recent < 0 || first > budget || recent > budget - first) return ATTN_ERR_ARG;
  if (budget > kMaxCapacity) return ATTN_ERR_UNSUPPORTED;
  if (!aligned4(weights) || !aligned4(positions) || !aligned4(seen) || !aligned4(n_moves) ||
      (reinterpret_cast<uintptr_t>(moves) & 7u))
    return ATTN_ERR_ALIGN;
  DeviceInfo* d = nullptr;
  rc = current_device(&d);
  if (rc != ATTN_OK) return rc;
  PlanArgs a{index_of(cache), weights, positions, seen, moves, n_moves, budget, first, recent, d->status, 0, false};
  return launched(launch_evict_plan(a, d->sms, reinterpret_cast<cudaStream_t>(stream)));
}

int attn_cache_compact(const attn_cache* cache, const int32_t* moves, const int32_t* n_moves, int budget,
                       float* weights, int32_t* positions, attn_stream_t stream) {
  int rc = check_cache(cache, true);
  if (rc != ATTN_OK) return rc;
  if (moves == nullptr || n_moves == nullptr || budget < 1) return ATTN_ERR_ARG;
  if (budget > kMaxCapacity) return ATTN_ERR_UNSUPPORTED;
  if (!aligned4(n_moves) || !aligned4(weights) || !aligned4(positions) || (reinterpret_cast<uintptr_t>(moves) & 7u))
    return ATTN_ERR_ALIGN;
  DeviceInfo* d = nullptr;
  rc = current_device(&d);
  if (rc != ATTN_OK) return rc;
  CompactArgs a{cache_dev(cache, d), moves, n_moves, weights, positions, cache->lens, budget};
  return launched(launch_cache_compact(a, d->sms, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
