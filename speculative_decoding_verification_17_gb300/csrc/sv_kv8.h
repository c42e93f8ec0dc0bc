// sv_kv8.h — argument checks of the calls on a cache in 8 bits.
#pragma once

#include "specverify_kv8.h"
#include "sv_kv.h"

namespace sv {

constexpr int kMaxBlock = 128;  // slots that share a scale

inline sv_status check_pool8(const sv_kv_pool* p) {
  if (!p || !p->data || !aligned_to(p->data, 16)) return SV_ERR_INVALID_ARG;
  for (int64_t st : {p->page_stride, p->token_stride, p->head_stride})
    if (st <= 0 || st % 16 != 0 || st >= (1ll << 40)) return SV_ERR_INVALID_ARG;
  return SV_OK;
}

// Whether heads of a pool that is written lie apart, as far as each stride by itself tells.
inline bool heads_apart(const sv_kv_shape* s, const sv_kv_pool* p) {
  return (s->num_pages < 2 || p->page_stride >= s->D) && p->token_stride >= s->D &&
         (s->Hkv < 2 || p->head_stride >= s->D);
}

// Slots that share a scale: a power of two that divides a page, and a tile of 128 keys.
inline sv_status check_block(const sv_kv_shape* s, int block) {
  if (block < 1 || (block & (block - 1)) != 0 || block > s->page_size) return SV_ERR_INVALID_ARG;
  return block > kMaxBlock ? SV_ERR_UNSUPPORTED : SV_OK;
}

}  // namespace sv
