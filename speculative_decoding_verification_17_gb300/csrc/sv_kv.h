// sv_kv.h — what the key-value calls share: their argument checks and the device view of a
// paged pool.
#pragma once

#include <cmath>
#include <cstdint>

#include "specverify_kv.h"
#include "sv_host.h"

namespace sv {

constexpr int kMaxGroup = 64;      // query heads per kv head
constexpr int kMaxKvHeads = 1024;
constexpr int kMaxPageSize = 1024;

inline sv_status check_kv_shape(const sv_kv_shape* s, bool queries) {
  if (!s) return SV_ERR_INVALID_ARG;
  if (s->dtype != SV_KV_BF16 && s->dtype != SV_KV_F16) return SV_ERR_INVALID_ARG;
  if (s->B < 0 || s->Hkv < 1 || s->D < 1 || s->page_size < 1 || s->num_pages < 0 ||
      s->max_pages < 1)
    return SV_ERR_INVALID_ARG;
  if (queries && (s->P < 1 || s->Hq < 1 || s->Hq % s->Hkv != 0)) return SV_ERR_INVALID_ARG;
  if ((int64_t)s->max_pages * s->page_size >= (1ll << 30)) return SV_ERR_UNSUPPORTED;
  if (s->D != 64 && s->D != 128 && s->D != 256) return SV_ERR_UNSUPPORTED;
  if (s->Hkv > kMaxKvHeads || s->page_size < 8 || s->page_size > kMaxPageSize ||
      (s->page_size & (s->page_size - 1)) != 0)
    return SV_ERR_UNSUPPORTED;
  if (queries && (s->P > SV_MAX_K + 1 || s->Hq / s->Hkv > kMaxGroup)) return SV_ERR_UNSUPPORTED;
  if ((int64_t)s->B * s->Hkv >= (1ll << 24)) return SV_ERR_UNSUPPORTED;
  return SV_OK;
}

inline sv_status check_pool(const sv_kv_pool* p) {
  if (!p || !p->data || !aligned_to(p->data, 16)) return SV_ERR_INVALID_ARG;
  for (int64_t st : {p->page_stride, p->token_stride, p->head_stride})
    if (st <= 0 || st % 8 != 0 || st >= (1ll << 39)) return SV_ERR_INVALID_ARG;
  return SV_OK;
}

inline sv_status check_rule(const sv_score_rule* r) {
  if (!r || !std::isfinite(r->scale) || !std::isfinite(r->softcap) ||
      (r->softcap != 0.0f && r->softcap < 1e-6f) || r->window < 0 || !aligned_to(r->slopes, 4))
    return SV_ERR_INVALID_ARG;
  return SV_OK;
}

inline int log2_of(int x) {
  int l = 0;
  while ((1 << l) < x) ++l;
  return l;
}

// The rule as the kernels take it.
struct ScoreRule {
  float scale, softcap;
  int window;  // 2^30 (past every position) for none
  const float* slopes;
};
inline ScoreRule score_rule(const sv_score_rule* r) {
  return {r->scale, r->softcap, r->window > 0 && r->window < (1 << 30) ? r->window : 1 << 30, r->slopes};
}

}  // namespace sv
