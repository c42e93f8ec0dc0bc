// sv_evict.cu — eviction from a paged cache: the most recent and the heaviest keys are kept.
//
// One CTA per (request, kv head) finds the (budget - recent)-th largest weight among the keys
// that are not recent by a radix select: three histogram passes over 11, 11 and 10 bits of an
// order-preserving integer map of the weights, which stay in shared memory up to kHeld of them.
// Then each warp takes a contiguous share of the keys, counts what it keeps, and, with the counts
// of the warps before it, gives each kept key its slot; of the keys that equal the threshold the
// lowest are taken, so the result is unique.
//
// The kept keys and values are copied 16 bytes per lane, several keys per thread in flight. With
// enough (request, head) pairs to fill the SMs the selecting CTA copies its own, so that one CTA's
// selection (latency: about ten CTA barriers) passes under another's copies (bandwidth); with
// fewer a second launch spreads the copies over all SMs. Bound: the copies. Measured in graph
// replays: 64 requests x 8 heads of 128, 1000 .. 16384 keys cut to 2048, 169 us (1005 MB, 88 % of
// the 6782 GB/s a copy reaches); one request of 5003 keys cut to 1024, 13.4 us.
#include <cstdint>

#include "specverify_kv.h"
#include "sv_device.cuh"
#include "sv_host.h"
#include "sv_kv.h"

namespace sv {

int device_sm_count();

namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kHeld = 16384;   // weights in shared memory (64 KiB)
constexpr int kMoveBatch = 2;  // keys per thread in flight
// CTAs of an SM that select and copy: with two (32 registers a thread) one's selection passes under
// the other's copies. 64 requests x 8 heads of up to 16384 keys: 169 us; with one CTA and two or
// four keys a thread 188 and 186 us; with two CTAs of 512 threads 216 and 190 us.
constexpr int kBothCtas = 2;

struct MoveArgs {
  const char *k, *v;
  char *nk, *nv;
  int64_t kp, kt, kh, vp, vt, vh, nkp, nkt, nkh, nvp, nvt, nvh;  // strides in bytes
  const int32_t *table, *new_table, *out_len, *index;
  int Hkv, budget, log_page, max_pages, new_max_pages;
  int log_lanes;  // lanes per key: D * 2 / 16
};

// Copies the kept slots [first, last) of a (request, head) by `threads` threads.
__device__ __forceinline__ void move_keys(const MoveArgs& A, int bh, int first, int last, int tid,
                                          int threads) {
  const int b = bh / A.Hkv, h = bh % A.Hkv;
  const int lanes = 1 << A.log_lanes, mask = (1 << A.log_page) - 1, step = threads >> A.log_lanes;
  const int64_t x = (int64_t)(tid & (lanes - 1)) * 16;
  const int32_t* index = A.index + (int64_t)bh * A.budget;
#pragma unroll 1
  for (int j0 = first + (tid >> A.log_lanes); j0 < last; j0 += kMoveBatch * step) {
    uint4 kv[kMoveBatch], vv[kMoveBatch];
#pragma unroll
    for (int u = 0; u < kMoveBatch; ++u) {
      const int j = j0 + u * step;
      if (j < last) {
        const int s = index[j];
        const int64_t p = __ldg(A.table + (int64_t)b * A.max_pages + (s >> A.log_page));
        kv[u] = *reinterpret_cast<const uint4*>(A.k + p * A.kp + (s & mask) * A.kt + h * A.kh + x);
        vv[u] = *reinterpret_cast<const uint4*>(A.v + p * A.vp + (s & mask) * A.vt + h * A.vh + x);
      }
    }
#pragma unroll
    for (int u = 0; u < kMoveBatch; ++u) {
      const int j = j0 + u * step;
      if (j < last) {
        const int64_t q = __ldg(A.new_table + (int64_t)b * A.new_max_pages + (j >> A.log_page));
        *reinterpret_cast<uint4*>(A.nk + q * A.nkp + (j & mask) * A.nkt + h * A.nkh + x) = kv[u];
        *reinterpret_cast<uint4*>(A.nv + q * A.nvp + (j & mask) * A.nvt + h * A.nvh + x) = vv[u];
      }
    }
  }
}

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

// The kept slots of one (request, head): index, weights and (h = 0) the length. Returns how many
// are to be copied (0 for a data error).
__device__ __forceinline__ int select_keys(const SelectArgs& A, int b, int h, float* held_w) {
  __shared__ uint32_t hist[kBins];
  __shared__ uint32_t warp_sum[2][kSelWarps];
  __shared__ uint32_t s_digit, s_above;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = __ldg(A.seq_len + b);
  const int64_t row = (int64_t)b * A.Hkv + h;
  int32_t* index = A.out_index + row * A.budget;
  float* kept_w = A.out_weights ? A.out_weights + row * A.budget : nullptr;
  const int m = n < A.budget ? n : A.budget;
  const float* w = A.weights + row * A.stride;

  // every page that is read or written must exist
  bool bad = n < 0 || n > (A.max_pages << A.log_page) || n > A.stride;
  const bool held = !bad && n <= kHeld, evicts = !bad && n > A.budget;
  if (held && evicts) {
#pragma unroll 8
    for (int j = tid; j < n; j += kSelThreads) held_w[j] = __ldg(w + j);
  }
  if (!bad) {
    const int page = 1 << A.log_page;
    const int old_pages = (n + page - 1) >> A.log_page, new_pages = (m + page - 1) >> A.log_page;
#pragma unroll 1
    for (int i = tid; i < old_pages; i += kSelThreads) {
      const int p = __ldg(A.table + (int64_t)b * A.max_pages + i);
      bad |= p < 0 || p >= A.num_pages;
    }
#pragma unroll 1
    for (int i = tid; i < new_pages; i += kSelThreads) {
      const int p = __ldg(A.new_table + (int64_t)b * A.new_max_pages + i);
      bad |= p < 0 || p >= A.new_num_pages;
    }
  }
  bad = __syncthreads_or(bad);
  if (tid == 0 && h == 0) A.out_len[b] = bad ? -1 : m;
#pragma unroll 1
  for (int j = (bad ? 0 : m) + tid; j < A.budget; j += kSelThreads) {
    index[j] = -1;
    if (kept_w) kept_w[j] = 0.0f;
  }
  if (bad) return 0;
  if (!evicts) {
#pragma unroll 1
    for (int j = tid; j < m; j += kSelThreads) {
      index[j] = j;
      if (kept_w) kept_w[j] = __ldg(w + j);
    }
    return m;
  }
  auto weight = [&](int j) { return held ? held_w[j] : __ldg(w + j); };

  // the threshold: the `want`-th largest key of the n - recent older ones
  const int old = n - A.recent, want = A.budget - A.recent;
  uint32_t prefix = 0, known = 0;  // the threshold's bits found so far, and which they are
  uint32_t left = want;            // how many are still to take among keys with this prefix
  if (want > 0) {
#pragma unroll 1
    for (int shift = 21; shift >= 0; shift = shift == 21 ? 10 : shift == 10 ? 0 : -1) {
      const uint32_t bins = shift == 0 ? 1024u : 2048u;
#pragma unroll
      for (int i = 0; i < kBins / kSelThreads; ++i) hist[i * kSelThreads + tid] = 0;
      __syncthreads();
#pragma unroll 4
      for (int j0 = 0; j0 < old; j0 += kSelThreads) {
        const int j = j0 + tid;
        const float x = j < old ? weight(j) : 0.0f;
        const uint32_t key = weight_key(x), bin = (key >> shift) & (bins - 1);
        const bool mine = j < old && (key & known) == prefix;
        // keys that nothing ever looked at all weigh 0: a warp counts those together
        const uint32_t zeros = __ballot_sync(0xffffffffu, mine && x == 0.0f);
        if (mine && (x != 0.0f || __ffs(zeros) - 1 == lane))
          atomicAdd(&hist[bin], x != 0.0f ? 1u : (uint32_t)__popc(zeros));
      }
      __syncthreads();
      // suffix counts from the largest digit down: thread t holds kEach bins from bin
      // kEach * t from the top on
      constexpr int kEach = kBins / kSelThreads;
      const int from_top = kEach * tid;
      uint32_t c[kEach], s = 0;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        c[i] = from_top + i < (int)bins ? hist[bins - 1 - from_top - i] : 0u;
        s += c[i];
      }
      const uint32_t mine = s;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
      }
      if (lane == 31) warp_sum[0][warp] = s;
      __syncthreads();
      // the sum of the warps before, by a lane each
      uint32_t above = __reduce_add_sync(0xffffffffu, lane < warp ? warp_sum[0][lane] : 0u) + s -
                       mine;  // keys above this thread's bins
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        if (above < left && left <= above + c[i]) {
          s_digit = bins - 1 - from_top - i;
          s_above = above;
        }
        above += c[i];
      }
      __syncthreads();
      prefix |= s_digit << shift;
      known |= (bins - 1) << shift;
      left -= s_above;
    }
  }
  // keys above the threshold are kept, and the first `left` of those that equal it; warp i takes
  // the i-th contiguous share of the keys
  const int share = ((n + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
  const int j_lo = warp * share, j_hi = j_lo + share < n ? j_lo + share : n;
  auto kind = [&](int j, bool& above, bool& tie) {
    above = tie = false;
    if (j >= j_hi) return 0.0f;
    const float x = weight(j);
    const uint32_t key = weight_key(x);
    above = j >= old || (want > 0 && key > prefix);
    tie = j < old && want > 0 && key == prefix;
    return x;
  };
  uint32_t na = 0, nt = 0;
#pragma unroll 4
  for (int j0 = j_lo; j0 < j_hi; j0 += 32) {
    bool above, tie;
    kind(j0 + lane, above, tie);
    na += __popc(__ballot_sync(0xffffffffu, above));
    nt += __popc(__ballot_sync(0xffffffffu, tie));
  }
  if (lane == 0) {
    warp_sum[0][warp] = na;
    warp_sum[1][warp] = nt;
  }
  __syncthreads();
  uint32_t slot = __reduce_add_sync(0xffffffffu, lane < warp ? warp_sum[0][lane] : 0u);
  uint32_t ties = __reduce_add_sync(0xffffffffu, lane < warp ? warp_sum[1][lane] : 0u);
  const uint32_t lt = (1u << lane) - 1u;
#pragma unroll 2
  for (int j0 = j_lo; j0 < j_hi; j0 += 32) {
    bool above, tie;
    const float x = kind(j0 + lane, above, tie);
    const uint32_t ba = __ballot_sync(0xffffffffu, above), bt = __ballot_sync(0xffffffffu, tie);
    // ties taken before this key: the first `left` of all
    const uint32_t ties_before = ties + __popc(bt & lt);
    const uint32_t at = slot + __popc(ba & lt) + (ties_before < left ? ties_before : left);
    if (above || (tie && ties_before < left)) {
      index[at] = j0 + lane;
      if (kept_w) kept_w[at] = x;
    }
    slot += __popc(ba);
    ties += __popc(bt);
  }
  return m;
}

template <bool kMoves>
__global__ void __launch_bounds__(kSelThreads, kMoves ? kBothCtas : 1)
    select_kernel(const SelectArgs A, const __grid_constant__ MoveArgs M) {
  extern __shared__ float held_w[];
  if (!kMoves) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int m = select_keys(A, blockIdx.x / A.Hkv, blockIdx.x % A.Hkv, held_w);
  if (kMoves) {
    __syncthreads();
    move_keys(M, blockIdx.x, 0, m, threadIdx.x, kSelThreads);
  }
}

// Whether two ranges of bytes share one (no range: NULL).
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + nb && y < x + na;
}

constexpr int kMoveThreads = 256;

__global__ void __launch_bounds__(kMoveThreads)
    move_kernel(const __grid_constant__ MoveArgs A) {
  const int share = kMoveBatch * (kMoveThreads >> A.log_lanes), first = (int)blockIdx.x * share;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int m = A.out_len[blockIdx.y / A.Hkv];
  move_keys(A, blockIdx.y, first, first + share < m ? first + share : m, threadIdx.x,
            kMoveThreads);
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
  // one head's CTA writes a request's length while another may still read it, and rows of weights
  // move
  if (overlap(out_len, 4 * (size_t)shape->B, seq_len, 4 * (size_t)shape->B) ||
      overlap(out_weights, 4 * (size_t)rows * budget, weights, 4 * (size_t)rows * stride))
    return SV_ERR_INVALID_ARG;
  if (rows > 65535) return SV_ERR_UNSUPPORTED;
  const int lp = log2_of(shape->page_size);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  SelectArgs S{page_table, seq_len, new_table, weights, stride, out_len, out_index, out_weights,
               shape->Hkv, budget, recent, lp, shape->num_pages, shape->max_pages,
               new_num_pages, new_max_pages};
  MoveArgs M{static_cast<const char*>(k->data), static_cast<const char*>(v->data),
             static_cast<char*>(new_k->data), static_cast<char*>(new_v->data),
             2 * k->page_stride, 2 * k->token_stride, 2 * k->head_stride,
             2 * v->page_stride, 2 * v->token_stride, 2 * v->head_stride,
             2 * new_k->page_stride, 2 * new_k->token_stride, 2 * new_k->head_stride,
             2 * new_v->page_stride, 2 * new_v->token_stride, 2 * new_v->head_stride,
             page_table, new_table, out_len, out_index, shape->Hkv, budget, lp,
             shape->max_pages, new_max_pages, log2_of(shape->D / 8)};
  // (64 requests x 8 heads of up to 16384 keys, one CTA per SM: 187 us fused, 204 us in two
  // launches; 8 rows of 5003 keys: 13 us in two launches, of which the copies take 6)
  const bool fused = rows >= device_sm_count();
  auto select = fused ? select_kernel<true> : select_kernel<false>;
  cudaError_t e = cudaFuncSetAttribute(select, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kHeld * (int)sizeof(float));
  if (e != cudaSuccess) return cuda_fail(e);
  // as much as the longest cache needs, if that stays in shared memory
  const int64_t most = (int64_t)shape->max_pages * shape->page_size;
  const size_t smem = sizeof(float) * (size_t)(most < kHeld ? most : kHeld);
  select<<<(unsigned)rows, kSelThreads, smem, st>>>(S, M);
  const sv_status s1 = launch_status();
  if (s1 != SV_OK || fused) return s1;
  // the copies' CTAs take their places while the selection ends, and wait for it
  const int per_cta = kMoveBatch * (kMoveThreads >> M.log_lanes);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((budget + per_cta - 1) / per_cta), (unsigned)rows);
  cfg.blockDim = dim3(kMoveThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, move_kernel, M);
  return e == cudaSuccess ? launch_status() : cuda_fail(e);
}
