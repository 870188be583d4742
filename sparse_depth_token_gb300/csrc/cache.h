// What the key/value cache's entry points share: argument checks, and the cache as the
// kernels see it.
#pragma once

#include "internal.h"

namespace xmod {

inline bool ptr16(const void* p) { return p && ((uintptr_t)p & 15u) == 0; }
inline bool ptr16_or_null(const void* p) { return ((uintptr_t)p & 15u) == 0; }
// Row indices and status words: 4-byte arrays, of which callers pass slices.
inline bool ptr4_or_null(const void* p) { return ((uintptr_t)p & 3u) == 0; }

// XMOD_OK, or why the dims and the cache cannot be used together.
inline int cache_status(const xmod_dims* dm, const xmod_kv_cache* c) {
  if (!dims_ok(dm) || !c) return XMOD_ERR_INVALID_ARG;
  if (!head_dim_supported(dm->head_dim)) return XMOD_ERR_UNSUPPORTED;
  if (c->n_pages <= 0 || c->n_seqs <= 0 || c->max_pages <= 0 || c->page_size <= 0 ||
      c->page_size % 16 || (int64_t)c->max_pages * c->page_size > INT32_MAX)
    return XMOD_ERR_INVALID_ARG;
  if (!ptr16(c->k) || !ptr16(c->v) || !c->table || !ptr4_or_null(c->table))
    return XMOD_ERR_INVALID_ARG;
  if (c->format == XMOD_CACHE_E4M3) {
    if (!ptr16(c->k_scale) || !ptr16(c->v_scale)) return XMOD_ERR_INVALID_ARG;
    if (dm->dtype != XMOD_BF16) return XMOD_ERR_UNSUPPORTED;
  } else if (c->format != XMOD_CACHE_NATIVE || c->k_scale || c->v_scale) {
    return XMOD_ERR_INVALID_ARG;
  }
  // slots of one KV head over all pages: the row coordinate of a TMA tile
  if ((int64_t)c->n_pages * dm->n_kv_heads * c->page_size > INT32_MAX)
    return XMOD_ERR_UNSUPPORTED;
  return XMOD_OK;
}

}  // namespace xmod
