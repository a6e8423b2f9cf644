// cfr_cells.cuh -- places in a writable paged cache: resolving (sequence, token)
// to its page and row, and the host checks of the entry points that write or
// read back whole rows.
#pragma once

#include <climits>

#include "cfr_codec.cuh"

namespace cfr {

// The cache as the writing and reading kernels see it.
struct CacheView {
  uint8_t *k_pool[kFmtCount], *v_pool[kFmtCount];
  float *scales[kFmtCount];
  long long pool_pages[kFmtCount];
  const int32_t *page_table;
  const uint8_t *page_fmt;
  uint32_t *err;
  int uniform_fmt, max_pages, batch, Hkv, D, P;
};

// Format and slot of logical page lp of sequence b (both inside the table).
// False, with the error word set, when its format is unknown or not one of `formats` (bit f:
// format f), it has no pool, or its slot is outside the pool.
__device__ __forceinline__ bool resolve_page(const CacheView &c, int b, int lp, uint32_t formats,
                                             int &fmt, long long &slot) {
  const long long cell = static_cast<long long>(b) * c.max_pages + lp;
  slot = c.page_table[cell];
  fmt = c.page_fmt ? static_cast<int>(c.page_fmt[cell]) : c.uniform_fmt;
  if (fmt >= kFmtCount || !((formats >> fmt) & 1u)) {
    set_err(c.err, CFR_DEVERR_PAGE_FMT);
    return false;
  }
  if (!c.k_pool[fmt]) {
    // an entry point for some formats only counts a missing pool among the wrong formats
    set_err(c.err, formats == (1u << kFmtCount) - 1u ? CFR_DEVERR_POOL : CFR_DEVERR_PAGE_FMT);
    return false;
  }
  if (slot < 0 || slot >= c.pool_pages[fmt]) {
    set_err(c.err, CFR_DEVERR_PAGE_ID);
    return false;
  }
  return true;
}

// byte offset of row `tin` of (slot, kv head g) in a pool of `fmt`
__device__ __forceinline__ long long row_at(const CacheView &c, int fmt, long long slot, int g, int tin) {
  return ((slot * c.Hkv + g) * c.P + tin) * row_bytes(fmt, c.D);
}

// ---- host ------------------------------------------------------------------

inline bool ptr_aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Checks the pool description and the table's sizes, and fills the view with the
// pools of `formats` (others are left out).
inline cfr_status make_view(const cfr_kv_pool *kv, const int32_t *page_table, int32_t max_pages,
                            const uint8_t *page_fmt, int32_t uniform_fmt, int32_t batch,
                            uint32_t formats, uint32_t *err, CacheView *c) {
  if (!kv || !page_table) return CFR_ERR_INVALID_ARG;
  if (kv->num_kv_heads <= 0 || kv->head_dim <= 0 || kv->page_tokens <= 0) return CFR_ERR_INVALID_ARG;
  if (batch <= 0 || max_pages <= 0) return CFR_ERR_INVALID_ARG;
  if (kv->head_dim != 64 && kv->head_dim != 128) return CFR_ERR_UNSUPPORTED;
  if (kv->page_tokens < 8 || kv->num_kv_heads > kMaxQHeads) return CFR_ERR_UNSUPPORTED;
  if (static_cast<long long>(max_pages) * kv->page_tokens > INT_MAX ||
      static_cast<long long>(batch) * max_pages > INT_MAX)
    return CFR_ERR_OVERFLOW;
  bool any = false;
  for (int f = 0; f < kFmtCount; ++f) {
    const bool use = (formats >> f) & 1u;
    c->k_pool[f] = use ? static_cast<uint8_t *>(const_cast<void *>(kv->k_pool[f])) : nullptr;
    c->v_pool[f] = use ? static_cast<uint8_t *>(const_cast<void *>(kv->v_pool[f])) : nullptr;
    c->scales[f] = use ? const_cast<float *>(kv->scales[f]) : nullptr;
    c->pool_pages[f] = c->k_pool[f] ? kv->pool_pages[f] : 0;
    if (!c->k_pool[f] != !c->v_pool[f]) return CFR_ERR_INVALID_ARG;
    if (!c->k_pool[f]) continue;
    if (!ptr_aligned(c->k_pool[f], 16) || !ptr_aligned(c->v_pool[f], 16) || c->pool_pages[f] < 0)
      return CFR_ERR_INVALID_ARG;
    if (is_quantised(f) && c->pool_pages[f] > 0 && (!c->scales[f] || !ptr_aligned(c->scales[f], 8)))
      return CFR_ERR_INVALID_ARG;
    const long long per = static_cast<long long>(kv->num_kv_heads) * kv->page_tokens *
                          row_bytes(f, kv->head_dim);
    if (c->pool_pages[f] > 0 && per > LLONG_MAX / c->pool_pages[f]) return CFR_ERR_OVERFLOW;
    any = true;
  }
  if (!any) return CFR_ERR_INVALID_ARG;
  if (!page_fmt && (uniform_fmt < 0 || uniform_fmt >= kFmtCount || !c->k_pool[uniform_fmt]))
    return CFR_ERR_INVALID_ARG;
  c->page_table = page_table;
  c->page_fmt = page_fmt;
  c->err = err;
  c->uniform_fmt = uniform_fmt;
  c->max_pages = max_pages;
  c->batch = batch;
  c->Hkv = kv->num_kv_heads;
  c->D = kv->head_dim;
  c->P = kv->page_tokens;
  return CFR_OK;
}

// a [rows][heads][head_dim] argument of F32 or BF16 rows `stride` values apart
inline bool rows_ok(const void *p, int64_t stride, int64_t heads, int d, int fmt) {
  const int eb = fmt == CFR_FMT_F32 ? 4 : 2;
  return p && ptr_aligned(p, 16) && stride >= heads * d && stride <= LLONG_MAX / 4 / INT_MAX &&
         (stride * eb) % 16 == 0;
}

constexpr uint32_t kHotFormats = (1u << CFR_FMT_F32) | (1u << CFR_FMT_BF16);
constexpr uint32_t kAllFormats = (1u << kFmtCount) - 1u;

}  // namespace cfr
