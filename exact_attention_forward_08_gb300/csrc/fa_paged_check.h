// Argument checks that the C entry points on the paged cache share.
#pragma once
#include <cstddef>
#include <cstdint>

#include "fa.h"
#include "fa_host.h"

namespace fa {

constexpr int kMaxBatch = 16384;

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

inline bool dims_supported(int d_qk, int d_v) {
  return (d_qk == 64 && d_v == 64) || ((d_qk == 128 || d_qk == 192) && (d_v == 64 || d_v == 128));
}

// strides in bytes {page, head, token} of a cache of rows of d codes
inline bool strides_ok(const int64_t* s, int pages, int heads, int d) {
  const int64_t most = int64_t(1) << 40;
  for (int i = 0; i < 3; ++i)
    if (s[i] < 0 || s[i] % 16 != 0 || s[i] >= most) return false;
  if (s[2] < d || s[2] >= int64_t(1) << 24) return false;  // offsets inside a page are counted in 32 bits
  return (heads == 1 || s[1] >= d) && (pages == 1 || s[0] >= d);
}

inline int check_cache(const fa_kv_cache* c) {
  if (c == nullptr) return FA_ERR_INVALID_ARG;
  if (c->heads_kv < 1 || c->num_pages < 1 || c->max_pages < 1 || c->table_stride < c->max_pages) return FA_ERR_INVALID_ARG;
  if (!dims_supported(c->d_qk, c->d_v)) return FA_ERR_UNSUPPORTED;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128) return FA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(c->max_pages) * c->page_size > (int64_t(1) << 30)) return FA_ERR_INVALID_ARG;
  if (!strides_ok(c->k_stride, c->num_pages, c->heads_kv, c->d_qk) ||
      !strides_ok(c->v_stride, c->num_pages, c->heads_kv, c->d_v))
    return FA_ERR_INVALID_ARG;
  return FA_OK;
}

inline int check_cache_pointers(const fa_kv_cache* c) {
  if (c->k == nullptr || c->v == nullptr || c->k_scale == nullptr || c->v_scale == nullptr ||
      c->block_table == nullptr || c->seqlens_k == nullptr)
    return FA_ERR_INVALID_ARG;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->block_table, 4) || !aligned(c->seqlens_k, 4))
    return FA_ERR_INVALID_ARG;
  return FA_OK;
}

inline bool cache_on_device(const fa_kv_cache* c, int dev) {
  return fa::host_is_device_ptr(c->k, dev) && fa::host_is_device_ptr(c->v, dev) &&
         fa::host_is_device_ptr(c->k_scale, dev) && fa::host_is_device_ptr(c->v_scale, dev) &&
         fa::host_is_device_ptr(c->block_table, dev) && fa::host_is_device_ptr(c->seqlens_k, dev);
}

inline int page_shift(int page_size) { return page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : 7; }

inline size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

}  // namespace fa
