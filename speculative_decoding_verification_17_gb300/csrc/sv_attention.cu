// sv_attention.cu — attention of a verify step's new positions over a paged cache, and the
// weight each cached key received.
//
// The plain form: one warp per query row walks the row's keys with a running maximum and sum
// (attention), or one warp per key walks the rows that see it (weights). All sums are fp32.
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "specverify_kv.h"
#include "sv_device.cuh"
#include "sv_host.h"
#include "sv_kv.h"

namespace sv {
namespace {

constexpr int kWarpsPerCta = 4;

struct AttnArgs {
  const void *q, *k, *v;
  int64_t q_req, q_row, q_head, kp, kt, kh, vp, vt, vh;
  const int32_t *table, *seq_len, *num_draft, *accept_len;
  void* out;
  float* out_lse;
  const float *lse, *prior;
  float* weights;
  int64_t stride, lse_req, lse_row, lse_head;
  ScoreRule rule;
  int B, P, Hq, Hkv, D, log_page, num_pages, max_pages;
};

__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_f(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_f(__half* p, float x) { *p = __float2half_rn(x); }

__device__ __forceinline__ float score(float qk, const ScoreRule& r, float slope, int away) {
  float s = qk * r.scale;
  if (r.softcap > 0.0f) s = r.softcap * tanhf(s / r.softcap);
  return s - slope * (float)away;
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

template <typename T>
__global__ void attend_rows(const AttnArgs A) {
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * kWarpsPerCta + (threadIdx.x >> 5);
  if (row >= (int64_t)A.B * A.P * A.Hq) return;
  const int head = row % A.Hq, i = row / A.Hq % A.P, b = row / A.Hq / A.P;
  const int h = head / (A.Hq / A.Hkv);
  const int n = __ldg(A.seq_len + b), nd = A.num_draft ? __ldg(A.num_draft + b) : A.P - 1;
  T* o = static_cast<T*>(A.out) + row * A.D;
  const int cols = A.D / 32;
  bool bad = n < 0 || n > (A.max_pages << A.log_page) || nd < 0 || nd >= A.P;
  if (!bad && i > nd) return;
  const T* q = static_cast<const T*>(A.q) + b * A.q_req + i * A.q_row + head * A.q_head;
  const T* k = static_cast<const T*>(A.k) + h * A.kh;
  const T* v = static_cast<const T*>(A.v) + h * A.vh;
  const float slope = A.rule.slopes ? __ldg(A.rule.slopes + head) : 0.0f;
  const int mask = (1 << A.log_page) - 1;
  float qf[8], acc[8], top = -INFINITY, sum = 0.0f;
  for (int c = 0; c < cols; ++c) {
    qf[c] = bad ? 0.0f : to_f(q[c * 32 + lane]);
    acc[c] = 0.0f;
  }
  const int pos = n - 1 - nd + i;
  const int first = pos - A.rule.window + 1 > 0 ? pos - A.rule.window + 1 : 0;
  // the pages of every live row are checked by each of them
  const int all0 = n - 1 - nd - A.rule.window + 1 > 0 ? n - 1 - nd - A.rule.window + 1 : 0;
  if (!bad)
    for (int t = (all0 >> A.log_page) + lane; t <= (n - 1) >> A.log_page && n > 0; t += 32) {
      const int p = __ldg(A.table + (int64_t)b * A.max_pages + t);
      bad |= p < 0 || p >= A.num_pages;
    }
  bad = __any_sync(0xffffffffu, bad);
  if (!bad)
    for (int j = first; j <= pos; ++j) {
      const int64_t p = __ldg(A.table + (int64_t)b * A.max_pages + (j >> A.log_page));
      const T* kj = k + p * A.kp + (j & mask) * A.kt;
      const T* vj = v + p * A.vp + (j & mask) * A.vt;
      float s = 0.0f;
      for (int c = 0; c < cols; ++c) s += qf[c] * to_f(kj[c * 32 + lane]);
      s = score(warp_sum(s), A.rule, slope, pos - j);
      const float m = fmaxf(top, s);
      const float a = m == -INFINITY ? 1.0f : expf(top - m);
      const float e = m == -INFINITY ? 0.0f : expf(s - m);
      sum = sum * a + e;
      for (int c = 0; c < cols; ++c) acc[c] = acc[c] * a + e * to_f(vj[c * 32 + lane]);
      top = m;
    }
  const float nan = __uint_as_float(0x7fc00000u);
  for (int c = 0; c < cols; ++c)
    from_f(o + c * 32 + lane, bad ? nan : sum == 0.0f ? 0.0f : acc[c] / sum);
  if (A.out_lse && lane == 0) A.out_lse[row] = bad ? nan : top + logf(sum);
}

template <typename T>
__global__ void weigh_keys(const AttnArgs A) {
  const int lane = threadIdx.x & 31;
  const int bh = blockIdx.y, b = bh / A.Hkv, h = bh % A.Hkv, G = A.Hq / A.Hkv;
  const int n = __ldg(A.seq_len + b), nd = A.num_draft ? __ldg(A.num_draft + b) : A.P - 1;
  const int a = A.accept_len ? __ldg(A.accept_len + b) : nd;
  float* w = A.weights + (int64_t)bh * A.stride;
  const float* prior = A.prior ? A.prior + (int64_t)bh * A.stride : nullptr;
  const float nan = __uint_as_float(0x7fc00000u);
  if (n < 0 || n > (A.max_pages << A.log_page) || n > A.stride || nd < 0 || nd >= A.P ||
      a < -1 || a > nd) {
    if (blockIdx.x == 0 && threadIdx.x == 0) w[0] = nan;
    return;
  }
  const int mask = (1 << A.log_page) - 1;
  for (int j = blockIdx.x * kWarpsPerCta + (threadIdx.x >> 5); j < n;
       j += gridDim.x * kWarpsPerCta) {
    const int p = __ldg(A.table + (int64_t)b * A.max_pages + (j >> A.log_page));
    float total = 0.0f;
    const bool bad = p < 0 || p >= A.num_pages;
    const T* k = static_cast<const T*>(A.k) + (int64_t)p * A.kp + (j & mask) * A.kt + h * A.kh;
    for (int i = 0; i <= a && !bad; ++i) {
      const int pos = n - 1 - nd + i;
      if (j > pos || pos - j >= A.rule.window) continue;
      for (int g = 0; g < G; ++g) {
        const int head = h * G + g;
        const T* q = static_cast<const T*>(A.q) + b * A.q_req + i * A.q_row + head * A.q_head;
        float s = 0.0f;
        for (int c = lane; c < A.D; c += 32) s += to_f(q[c]) * to_f(k[c]);
        const float lse = A.lse[b * A.lse_req + i * A.lse_row + head * A.lse_head];
        s = score(warp_sum(s), A.rule, A.rule.slopes ? A.rule.slopes[head] : 0.0f, pos - j);
        if (lse != -INFINITY) total += expf(s - lse);
      }
    }
    if (lane == 0) w[j] = bad ? nan : (prior ? prior[j] : 0.0f) + total;
  }
}

sv_status fill_args(AttnArgs& A, const sv_kv_shape* s, const sv_score_rule* rule, const void* q,
                    int64_t q_req, int64_t q_row, int64_t q_head, const sv_kv_pool* k,
                    const int32_t* page_table, const int32_t* seq_len,
                    const int32_t* num_draft) {
  const sv_status ok = check_kv_shape(s, true);
  if (ok != SV_OK) return ok;
  const sv_status okr = check_rule(rule);
  if (okr != SV_OK) return okr;
  if (s->B == 0) return SV_OK;
  const sv_status okp = check_pool(k);
  if (okp != SV_OK) return okp;
  if (!q || !page_table || !seq_len || !aligned_to(q, 16) || !aligned_to(page_table, 4) ||
      !aligned_to(seq_len, 4) || !aligned_to(num_draft, 4))
    return SV_ERR_INVALID_ARG;
  if (q_req < 0 || q_row < 0 || q_head < 0 || q_req % 8 || q_row % 8 || q_head % 8)
    return SV_ERR_INVALID_ARG;
  A = AttnArgs{};
  A.q = q;
  A.k = k->data;
  A.q_req = q_req;
  A.q_row = q_row;
  A.q_head = q_head;
  A.kp = k->page_stride;
  A.kt = k->token_stride;
  A.kh = k->head_stride;
  A.table = page_table;
  A.seq_len = seq_len;
  A.num_draft = num_draft;
  A.rule = score_rule(rule);
  A.B = s->B;
  A.P = s->P;
  A.Hq = s->Hq;
  A.Hkv = s->Hkv;
  A.D = s->D;
  A.log_page = log2_of(s->page_size);
  A.num_pages = s->num_pages;
  A.max_pages = s->max_pages;
  return SV_OK;
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" size_t paged_attention_workspace(const sv_kv_shape* shape) {
  if (check_kv_shape(shape, true) != SV_OK) return 0;
  return 256;
}

extern "C" sv_status paged_attention(const sv_kv_shape* shape, const sv_score_rule* rule,
                                     const void* q, int64_t q_req, int64_t q_row,
                                     int64_t q_head, const sv_kv_pool* k, const sv_kv_pool* v,
                                     const int32_t* page_table, const int32_t* seq_len,
                                     const int32_t* num_draft, void* out, float* out_lse,
                                     void* workspace, size_t workspace_bytes,
                                     sv_stream_t stream) {
  AttnArgs A;
  const sv_status ok = fill_args(A, shape, rule, q, q_req, q_row, q_head, k, page_table,
                                 seq_len, num_draft);
  if (ok != SV_OK) return ok;
  if (shape->B == 0) return SV_OK;
  const sv_status okv = check_pool(v);
  if (okv != SV_OK) return okv;
  if (!out || !aligned_to(out, 16) || !aligned_to(out_lse, 4)) return SV_ERR_INVALID_ARG;
  if (!workspace || !aligned_to(workspace, 256) ||
      workspace_bytes < paged_attention_workspace(shape))
    return SV_ERR_WORKSPACE;
  A.v = v->data;
  A.vp = v->page_stride;
  A.vt = v->token_stride;
  A.vh = v->head_stride;
  A.out = out;
  A.out_lse = out_lse;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int64_t rows = (int64_t)A.B * A.P * A.Hq;
  const unsigned grid = (unsigned)((rows + kWarpsPerCta - 1) / kWarpsPerCta);
  if (shape->dtype == SV_KV_BF16)
    attend_rows<__nv_bfloat16><<<grid, 32 * kWarpsPerCta, 0, st>>>(A);
  else
    attend_rows<__half><<<grid, 32 * kWarpsPerCta, 0, st>>>(A);
  return launch_status();
}

extern "C" sv_status attention_weight_sum(const sv_kv_shape* shape, const sv_score_rule* rule,
                                          const void* q, int64_t q_req, int64_t q_row,
                                          int64_t q_head, const sv_kv_pool* k,
                                          const int32_t* page_table, const int32_t* seq_len,
                                          const int32_t* num_draft, const float* lse,
                                          int64_t lse_req, int64_t lse_row, int64_t lse_head,
                                          const int32_t* accept_len, const float* prior,
                                          float* out, int64_t stride, sv_stream_t stream) {
  AttnArgs A;
  const sv_status ok = fill_args(A, shape, rule, q, q_req, q_row, q_head, k, page_table,
                                 seq_len, num_draft);
  if (ok != SV_OK) return ok;
  if (stride < 1 || lse_req < 0 || lse_row < 0 || lse_head < 0) return SV_ERR_INVALID_ARG;
  if (shape->B == 0) return SV_OK;
  if (!lse || !out || !aligned_to(lse, 4) || !aligned_to(out, 4) || !aligned_to(prior, 4) ||
      !aligned_to(accept_len, 4))
    return SV_ERR_INVALID_ARG;
  if (shape->B * shape->Hkv > 65535) return SV_ERR_UNSUPPORTED;
  A.lse = lse;
  A.lse_req = lse_req;
  A.lse_row = lse_row;
  A.lse_head = lse_head;
  A.accept_len = accept_len;
  A.prior = prior;
  A.weights = out;
  A.stride = stride;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const dim3 grid(64, (unsigned)(shape->B * shape->Hkv));
  if (shape->dtype == SV_KV_BF16)
    weigh_keys<__nv_bfloat16><<<grid, 32 * kWarpsPerCta, 0, st>>>(A);
  else
    weigh_keys<__half><<<grid, 32 * kWarpsPerCta, 0, st>>>(A);
  return launch_status();
}
