// sv_evict.cu — eviction from a paged cache: the most recent and the heaviest keys are kept.
//
// Two launches. select_kernel, one CTA per (request, kv head), finds the (budget - recent)-th
// largest weight among the keys that are not recent by a radix select (three histogram passes
// over 11, 11 and 10 bits of an order-preserving integer map of the weights), then walks the
// keys once more in ascending order and gives each kept one its slot by a running count; of
// the keys that equal the threshold the lowest are taken, so the result is unique. move_kernel
// copies the kept keys and values to the new pages, 16 bytes per lane.
#include <cstdint>

#include "specverify_kv.h"
#include "sv_device.cuh"
#include "sv_host.h"
#include "sv_kv.h"

namespace sv {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;

struct SelectArgs {
  const int32_t *table, *seq_len, *new_table;
  const float* weights;
  int64_t stride;
  int32_t *out_len, *out_index;
  float* out_weights;
  int Hkv, budget, recent, log_page, num_pages, max_pages, new_num_pages, new_max_pages;
};

// Order-preserving map of a weight onto uint32: NaN as -inf, -0 as 0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) w = __uint_as_float(0xff800000u);
  const uint32_t u = __float_as_uint(w + 0.0f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelectArgs A) {
  __shared__ uint32_t hist[kBins];
  __shared__ uint32_t warp_sum[2][kSelWarps];
  __shared__ uint32_t s_digit, s_above;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / A.Hkv, h = blockIdx.x % A.Hkv;
  const int n = __ldg(A.seq_len + b);
  const int64_t row = (int64_t)b * A.Hkv + h;
  int32_t* index = A.out_index + row * A.budget;
  float* kept_w = A.out_weights ? A.out_weights + row * A.budget : nullptr;
  const int m = n < A.budget ? n : A.budget;

  // every page that is read or written must exist
  bool bad = n < 0 || n > (A.max_pages << A.log_page) || n > A.stride;
  if (!bad) {
    const int page = 1 << A.log_page;
    const int old_pages = (n + page - 1) >> A.log_page, new_pages = (m + page - 1) >> A.log_page;
    for (int i = tid; i < old_pages; i += kSelThreads) {
      const int p = __ldg(A.table + (int64_t)b * A.max_pages + i);
      bad |= p < 0 || p >= A.num_pages;
    }
    for (int i = tid; i < new_pages; i += kSelThreads) {
      const int p = __ldg(A.new_table + (int64_t)b * A.new_max_pages + i);
      bad |= p < 0 || p >= A.new_num_pages;
    }
  }
  bad = __syncthreads_or(bad);
  if (tid == 0 && h == 0) A.out_len[b] = bad ? -1 : m;
  for (int j = (bad ? 0 : m) + tid; j < A.budget; j += kSelThreads) {
    index[j] = -1;
    if (kept_w) kept_w[j] = 0.0f;
  }
  if (bad) return;
  const float* w = A.weights + row * A.stride;
  if (n <= A.budget) {
    for (int j = tid; j < m; j += kSelThreads) {
      index[j] = j;
      if (kept_w) kept_w[j] = w[j];
    }
    return;
  }

  // the threshold: the `want`-th largest key of the n - recent older ones
  const int old = n - A.recent, want = A.budget - A.recent;
  uint32_t prefix = 0, known = 0;  // the threshold's bits found so far, and which they are
  uint32_t left = want;            // how many are still to take among keys with this prefix
  if (want > 0) {
    for (int shift = 21; shift >= 0; shift = shift == 21 ? 10 : shift == 10 ? 0 : -1) {
      const uint32_t bins = shift == 0 ? 1024u : 2048u;
      for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (int j = tid; j < old; j += kSelThreads) {
        const uint32_t key = weight_key(__ldg(w + j));
        if ((key & known) == prefix) atomicAdd(&hist[(key >> shift) & (bins - 1)], 1u);
      }
      __syncthreads();
      // suffix counts from the largest digit down: thread t holds the bins 2t and 2t + 1 from
      // the top
      const uint32_t top = bins - 1 - 2 * tid;
      const bool mine = 2 * tid < (int)bins;
      const uint32_t a = mine ? hist[top] : 0, c = mine ? hist[top - 1] : 0;
      uint32_t s = a + c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
      }
      if (lane == 31) warp_sum[0][warp] = s;
      __syncthreads();
      uint32_t before = 0;
      for (int q = 0; q < warp; ++q) before += warp_sum[0][q];
      const uint32_t incl = before + s, excl = incl - a - c;  // keys above this pair: excl
      if (mine && excl < left && left <= incl) {
        const bool first = left <= excl + a;
        s_digit = first ? top : top - 1;
        s_above = first ? excl : excl + a;
      }
      __syncthreads();
      prefix |= s_digit << shift;
      known |= (bins - 1) << shift;
      left -= s_above;
    }
  }
  // keys above the threshold are kept, and the first `left` of those that equal it
  uint32_t slot = 0, ties = 0;
  for (int j0 = 0; j0 < n; j0 += kSelThreads) {
    const int j = j0 + tid;
    float x = 0.0f;
    bool above = false, tie = false;
    if (j < n) {
      x = __ldg(w + j);
      const uint32_t key = weight_key(x);
      above = j >= old || (want > 0 && key > prefix);
      tie = j < old && want > 0 && key == prefix;
    }
    const uint32_t ba = __ballot_sync(0xffffffffu, above), bt = __ballot_sync(0xffffffffu, tie);
    if (lane == 0) {
      warp_sum[0][warp] = __popc(ba);
      warp_sum[1][warp] = __popc(bt);
    }
    __syncthreads();
    uint32_t na = 0, nt = 0, all_a = 0, all_t = 0;
    for (int q = 0; q < kSelWarps; ++q) {
      const uint32_t va = warp_sum[0][q], vt = warp_sum[1][q];
      if (q < warp) {
        na += va;
        nt += vt;
      }
      all_a += va;
      all_t += vt;
    }
    const uint32_t lt = (1u << lane) - 1u;
    const uint32_t ties_before = ties + nt + __popc(bt & lt);
    // ties taken before this key: the first `left` of all
    const uint32_t taken = ties_before < left ? ties_before : left;
    const uint32_t at = slot + na + __popc(ba & lt) + taken;
    if (above || (tie && ties_before < left)) {
      index[at] = j;
      if (kept_w) kept_w[at] = x;
    }
    slot += all_a;
    ties += all_t;
    __syncthreads();
  }
}

struct MoveArgs {
  const char *k, *v;
  char *nk, *nv;
  int64_t kp, kt, kh, vp, vt, vh, nkp, nkt, nkh, nvp, nvt, nvh;  // strides in bytes
  const int32_t *table, *new_table, *out_len, *index;
  int Hkv, budget, log_page, max_pages, new_max_pages;
  int log_lanes;  // lanes per key: D * 2 / 16
};

constexpr int kMoveThreads = 256;
constexpr int kMoveKeys = 128;  // kept slots per CTA

__global__ void __launch_bounds__(kMoveThreads) move_kernel(const MoveArgs A) {
  const int tid = threadIdx.x;
  const int bh = blockIdx.y, b = bh / A.Hkv, h = bh % A.Hkv;
  const int m = __ldg(A.out_len + b);
  const int lanes = 1 << A.log_lanes, mask = (1 << A.log_page) - 1;
  const int64_t x = (int64_t)(tid & (lanes - 1)) * 16;
  const int end = (int)(blockIdx.x + 1) * kMoveKeys < m ? (int)(blockIdx.x + 1) * kMoveKeys : m;
  for (int j = blockIdx.x * kMoveKeys + (tid >> A.log_lanes); j < end;
       j += kMoveThreads >> A.log_lanes) {
    const int s = __ldg(A.index + (int64_t)bh * A.budget + j);
    const int64_t p = __ldg(A.table + (int64_t)b * A.max_pages + (s >> A.log_page));
    const int64_t q = __ldg(A.new_table + (int64_t)b * A.new_max_pages + (j >> A.log_page));
    const uint4 kv = *reinterpret_cast<const uint4*>(A.k + p * A.kp + (s & mask) * A.kt +
                                                     h * A.kh + x);
    const uint4 vv = *reinterpret_cast<const uint4*>(A.v + p * A.vp + (s & mask) * A.vt +
                                                     h * A.vh + x);
    *reinterpret_cast<uint4*>(A.nk + q * A.nkp + (j & mask) * A.nkt + h * A.nkh + x) = kv;
    *reinterpret_cast<uint4*>(A.nv + q * A.nvp + (j & mask) * A.nvt + h * A.nvh + x) = vv;
  }
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" sv_status kv_cache_evict(const sv_kv_shape* shape, const sv_kv_pool* k,
                                    const sv_kv_pool* v, const int32_t* page_table,
                                    const int32_t* seq_len, const float* weights,
                                    int64_t stride, int budget, int recent,
                                    const sv_kv_pool* new_k, const sv_kv_pool* new_v,
                                    int new_num_pages, const int32_t* new_table,
                                    int new_max_pages, int32_t* out_len, int32_t* out_index,
                                    float* out_weights, sv_stream_t stream) {
  const sv_status ok = check_kv_shape(shape, false);
  if (ok != SV_OK) return ok;
  if (budget < 1 || recent < 0 || recent > budget || stride < 1 || new_num_pages < 0 ||
      new_max_pages < 1)
    return SV_ERR_INVALID_ARG;
  if ((int64_t)new_max_pages * shape->page_size >= (1ll << 30)) return SV_ERR_UNSUPPORTED;
  if (budget > new_max_pages * shape->page_size) return SV_ERR_INVALID_ARG;
  if (shape->B == 0) return SV_OK;
  for (const sv_kv_pool* p : {k, v, new_k, new_v}) {
    const sv_status s = check_pool(p);
    if (s != SV_OK) return s;
  }
  if (!page_table || !seq_len || !weights || !new_table || !out_len || !out_index)
    return SV_ERR_INVALID_ARG;
  if (!aligned_to(page_table, 4) || !aligned_to(seq_len, 4) || !aligned_to(weights, 4) ||
      !aligned_to(new_table, 4) || !aligned_to(out_len, 4) || !aligned_to(out_index, 4) ||
      !aligned_to(out_weights, 4))
    return SV_ERR_INVALID_ARG;
  const int rows = shape->B * shape->Hkv;
  if (rows > 65535) return SV_ERR_UNSUPPORTED;
  const int lp = log2_of(shape->page_size);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  SelectArgs S{page_table, seq_len, new_table, weights, stride, out_len, out_index, out_weights,
               shape->Hkv, budget, recent, lp, shape->num_pages, shape->max_pages,
               new_num_pages, new_max_pages};
  select_kernel<<<(unsigned)rows, kSelThreads, 0, st>>>(S);
  const sv_status s1 = launch_status();
  if (s1 != SV_OK) return s1;
  MoveArgs M{static_cast<const char*>(k->data), static_cast<const char*>(v->data),
             static_cast<char*>(new_k->data), static_cast<char*>(new_v->data),
             2 * k->page_stride, 2 * k->token_stride, 2 * k->head_stride,
             2 * v->page_stride, 2 * v->token_stride, 2 * v->head_stride,
             2 * new_k->page_stride, 2 * new_k->token_stride, 2 * new_k->head_stride,
             2 * new_v->page_stride, 2 * new_v->token_stride, 2 * new_v->head_stride,
             page_table, new_table, out_len, out_index, shape->Hkv, budget, lp,
             shape->max_pages, new_max_pages, log2_of(shape->D / 8)};
  const dim3 grid((unsigned)((budget + kMoveKeys - 1) / kMoveKeys), (unsigned)rows);
  move_kernel<<<grid, kMoveThreads, 0, st>>>(M);
  return launch_status();
}
