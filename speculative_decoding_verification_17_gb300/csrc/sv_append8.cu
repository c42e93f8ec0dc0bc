// sv_append8.cu — new keys and values into a paged cache of 8 bits, with a scale for each block of
// tokens and kv head.
//
// Mathematics: scale = the smallest power of two that brings the block's largest magnitude within
// 448, or the block's scale so far where earlier tokens hold it up; code = x / scale, rounded to e4m3.
// A power of two is read off the bits of the largest magnitude, divides exactly, and re-rounds
// earlier codes exactly but for those that become subnormal.
//
// Work: rows of one block stand side by side, so the first of them (its predecessor is in another
// block) finds the others. A warp takes one such run for one head of keys or values: it reads the
// run's rows once for the largest magnitude and codes them from registers, or again from L2 where
// there are more than sixteen loads of them. No two warps share a block.
//
// Bound: 3 bytes an element (2 read, 1 written). Measured, in graph replays (bytes at 6801 GB/s first):
// one token of 64 requests 0.06 us, 3.9 us; prompts of 64 requests, 48600 rows of 8 heads of 128 44.0 us,
// 54.5 us, 81 % of a copy's bandwidth.
#include <cstdint>

#include <cuda_fp8.h>

#include "specverify_kv8.h"
#include "sv_kv8.h"
#include "sv_kv_tiles.cuh"

namespace sv {
namespace {

// Small CTAs, as many as registers for a run's loads leave room for: 640 threads of an SM hold 160 KB on
// its way (prompts of 48600 rows of 8 heads of 128, in graph replays: 5 CTAs of 128 threads 54.5 us, 4 of
// them 56.8, 2 of 256 60.7, 10 of 64 58.4; 6 of 128, whose loads spill, 61.2; half the loads kept and the
// rest read again 70).
constexpr int kAppThreads = 128, kAppCtas = 5, kAppWarps = kAppThreads / 32;

struct AppendArgs {
  const uint16_t* x[2];  // keys, values
  int64_t row[2], head[2];
  unsigned char* pool[2];
  int64_t page[2], token[2], pool_head[2];
  float* scale[2];
  const int64_t* slots;
  int64_t num_slots;  // of the pools
  int rows, Hkv, log_page, log_block;
};

// Eight numbers as e4m3 codes. With a plain scale (a power of two, and no number of the run past the
// limit) a product; else a quotient, and what is not finite, or too large for any scale, becomes NaN.
template <bool kBf16, bool kPlain>
__device__ __forceinline__ uint2 code8(const uint4& v, float scale, uint32_t limit) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t b[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float2 f = unpack16<kBf16>(w[k]);
    if (kPlain) {  // (scale is the reciprocal)
      f = split(two_mul(two(f.x, f.y), two(scale, scale)));
    } else {
      f.x = (w[k] & 0x7fffu) > limit ? __uint_as_float(0x7fc00000u) : __fdiv_rn(f.x, scale);
      f.y = (w[k] >> 16 & 0x7fffu) > limit ? __uint_as_float(0x7fc00000u) : __fdiv_rn(f.y, scale);
    }
    b[k] = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(__byte_perm(b[0], b[1], 0x5410), __byte_perm(b[2], b[3], 0x5410));
}

// The rows of a chunk of 32 and of those after it that its last run may reach (a run from the chunk's
// last row on has at most 128, and one too many, so 31 + 1 + 128 rows): a bit each for rows that go on
// with the block of the row ahead of them, and for those of them whose slot is higher.
struct Rows {
  static constexpr int kWindows = 1 + kMaxBlock / 32;
  uint32_t same[kWindows], higher[kWindows];
};

template <int D, bool kBf16>
__global__ void __launch_bounds__(kAppThreads, kAppCtas) append_kernel(const __grid_constant__ AppendArgs A) {
  constexpr int kLanes = D / 8, kPer = 32 / kLanes;  // lanes of a row, rows at a time
  constexpr int kKeep = 16;                          // loads of a run kept in registers
  // the largest finite magnitude that a scale reaches (448 * 2^40 in bf16)
  constexpr uint32_t kLimit = kBf16 ? 0x57e0u : 0x7bffu;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int block = 1 << A.log_block, windows = 1 + (block + 31) / 32;  // (of 32 rows)
  const int t0 = blockIdx.x * 32;
  // a row's slot, -1 for a row that is left out
  auto slot_of = [&](int t) {
    const int64_t s = t >= 0 && t < A.rows ? __ldg(A.slots + t) : -1;
    return s < A.num_slots ? s : -1;
  };
  __shared__ Rows R;
  __shared__ int64_t slots[32];
  __shared__ uint32_t first_rows;
  for (int w = warp; w < windows; w += kAppWarps) {
    const int64_t s = slot_of(t0 + 32 * w + lane), p = slot_of(t0 + 32 * w + lane - 1);
    const bool same = s >= 0 && p >= 0 && s >> A.log_block == p >> A.log_block;
    const uint32_t same_mask = __ballot_sync(0xffffffffu, same);
    const uint32_t higher = __ballot_sync(0xffffffffu, same && s > p);
    const uint32_t starting = __ballot_sync(0xffffffffu, s >= 0 && !same);
    if (w == 0) slots[lane] = s;
    if (lane == 0) {
      R.same[w] = same_mask;
      R.higher[w] = higher;
      if (w == 0) first_rows = starting;
    }
  }
  __syncthreads();
  uint32_t starts = first_rows;
  const int units = __popc(starts) * A.Hkv * 2;
  int at_run = 0;  // the run that is the lowest bit of `starts`
#pragma unroll 1
  for (int u = blockIdx.y * kAppWarps + warp; u < units; u += gridDim.y * kAppWarps) {
    const int run = u / (2 * A.Hkv), h = (u - run * 2 * A.Hkv) >> 1, which = u & 1;
    for (; at_run < run; ++at_run) starts &= starts - 1;
    const int cur = __ffs(starts) - 1;
    const int64_t first = slots[cur];
    const uint16_t* x =
        A.x[which] + (int64_t)(t0 + cur) * A.row[which] + h * A.head[which] + lane % kLanes * 8;
    const int mine = lane / kLanes;  // the lane's row of a load
    // the run's rows, and whether their slots ascend
    int n = 1;
    bool ordered = true, open = true;
#pragma unroll 1
    for (int w = 0; w < windows && open; ++w) {
      const int from = w == 0 ? cur + 1 : 0;
      const uint32_t rest = from < 32 ? R.same[w] >> from : 0u;
      const int more = ~rest ? __ffs(~rest) - 1 : 32;  // rows that go on
      const uint32_t mask = more == 32 ? 0xffffffffu : (1u << more) - 1;
      ordered = ordered && !(mask & ~(from < 32 ? R.higher[w] >> from : 0u));
      open = from + more == 32;
      n += more;
    }
    ordered = ordered && n <= block;
    const int64_t page = first >> A.log_page;
    const int at = (int)(first & ((1 << A.log_page) - 1));
    float* scale_at = A.scale[which] + (page * (1 << (A.log_page - A.log_block)) + (at >> A.log_block)) * A.Hkv + h;
    if (!ordered) {
      if (lane == 0) *scale_at = __uint_as_float(0x7fc00000u);
      continue;
    }
    const int earlier = at & (block - 1);  // slots of the block below the first new one
    auto load = [&](int i) {
      return i < n ? ld_stream16(x + i * A.row[which]) : make_uint4(0u, 0u, 0u, 0u);
    };
    uint4 keep[kKeep];
#pragma unroll
    for (int s = 0; s < kKeep; ++s) keep[s] = load(s * kPer + mine);
    const float old = earlier ? *scale_at : 0.0f;
    // the largest magnitude by its bits, two numbers in a word
    uint32_t most = 0;
    auto raise = [&](const uint4& v) {
      most = __vmaxu2(most, __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                     __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
    };
#pragma unroll
    for (int s = 0; s < kKeep; ++s)
      if (s * kPer < n) raise(keep[s]);
#pragma unroll 1
    for (int s0 = kKeep; s0 * kPer < n; s0 += 4) {
      uint4 v[4];
#pragma unroll
      for (int s = 0; s < 4; ++s) v[s] = load((s0 + s) * kPer + mine);
#pragma unroll
      for (int s = 0; s < 4; ++s) raise(v[s]);
    }
    uint32_t top = __reduce_max_sync(0xffffffffu, max(most & 0xffffu, most >> 16));
    const bool odd = top > kLimit;
    if (__builtin_expect(odd, 0)) {  // numbers past the limit do not count
      most = 0;
#pragma unroll 1
      for (int s = 0; s * kPer < n; ++s) {
        const uint4 v = load(s * kPer + mine);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
          const uint32_t lo = w[k] & 0x7fffu, hi = w[k] >> 16 & 0x7fffu;
          most = max(most, max(lo > kLimit ? 0u : lo, hi > kLimit ? 0u : hi));
        }
      }
      top = __reduce_max_sync(0xffffffffu, most);
    }
    // 448 = 1.75 * 2^8
    const uint32_t bits = __float_as_uint(unpack16<kBf16>(top).x);
    const int e = max(-40, (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u));
    float scale = __uint_as_float((uint32_t)(127 + e) << 23);
    unsigned char* pool = A.pool[which] + page * A.page[which] + h * A.pool_head[which];
    const int64_t token = A.token[which];
    if (earlier) {
      if (!(old >= 0.0f && old <= 1099511627776.0f)) {
        scale = __uint_as_float(0x7fc00000u);
      } else if (old >= scale) {
        scale = old;
      } else {
        // earlier codes, four at a time (those of a scale of 0 stand for 0, and become 0)
        const float ratio = old / scale;
        unsigned char* p = pool + (int64_t)(at - earlier) * token;
#pragma unroll 2
        for (int q = lane; q < earlier * (D / 4); q += 32) {
          uint32_t* w = reinterpret_cast<uint32_t*>(p + (int64_t)(q / (D / 4)) * token + q % (D / 4) * 4);
          const uint32_t v = *w;
          uint32_t out = 0;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(v >> 16 * k), __NV_E4M3);
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r));
            out |= (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(f.x * ratio, f.y * ratio),
                                                      __NV_SATFINITE, __NV_E4M3) << 16 * k;
          }
          *w = out;
        }
      }
    }
    if (lane == 0) *scale_at = scale;
    const bool plain = !odd && (__float_as_uint(scale) & 0x7fffffu) == 0;
    unsigned char* const column = pool + lane % kLanes * 8;
    // slots ascend, but need not be neighbours
    const bool close = n == 1 || __ldg(A.slots + t0 + cur + n - 1) - first == n - 1;
    if (__builtin_expect(plain && close, 1)) {
      const float inverse = 1.0f / scale;
      unsigned char* to = column + (at + mine) * token;
#pragma unroll
      for (int s = 0; s < kKeep; ++s, to += kPer * token)
        if (s * kPer < n && s * kPer + mine < n)
          *reinterpret_cast<uint2*>(to) = code8<kBf16, true>(keep[s], inverse, kLimit);
#pragma unroll 1
      for (int s0 = kKeep; s0 * kPer < n; s0 += 4, to += 4 * kPer * token) {
        uint4 v[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) v[s] = load((s0 + s) * kPer + mine);
#pragma unroll
        for (int s = 0; s < 4; ++s)
          if ((s0 + s) * kPer + mine < n)
            *reinterpret_cast<uint2*>(to + s * kPer * token) = code8<kBf16, true>(v[s], inverse, kLimit);
      }
    } else {
      // (kept short, as rare as it is: beside the loop above it pushed that out of the instruction cache)
#pragma unroll 1
      for (int i = mine; i < n; i += kPer) {
        const int s = (int)(__ldg(A.slots + t0 + cur + i) & ((1 << A.log_page) - 1));
        *reinterpret_cast<uint2*>(column + s * token) = code8<kBf16, false>(load(i), scale, kLimit);
      }
    }
  }
}

template <int D, bool kBf16>
sv_status launch_append(const AppendArgs& A, cudaStream_t st) {
  const int64_t chunks = (A.rows + 31) / 32;
  // enough CTAs for the SMs and a warp for each unit of one run, up to one for each unit of 32 runs (more
  // CTAs than a chunk's units only look at its slots again)
  int64_t split = (32 * (int64_t)device_sm_count() + chunks - 1) / chunks;
  const int64_t most = (64 * (int64_t)A.Hkv + kAppWarps - 1) / kAppWarps;
  const int64_t least = (2 * (int64_t)A.Hkv + kAppWarps - 1) / kAppWarps;
  split = split > most ? most : split < least ? least : split;
  append_kernel<D, kBf16><<<dim3((unsigned)chunks, (unsigned)split), kAppThreads, 0, st>>>(A);
  return launch_status();
}

template <bool kBf16>
sv_status launch_append_width(int D, const AppendArgs& A, cudaStream_t st) {
  switch (D) {
    case 64: return launch_append<64, kBf16>(A, st);
    case 128: return launch_append<128, kBf16>(A, st);
  }
  return launch_append<256, kBf16>(A, st);
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" sv_status kv_cache_append_q8(const sv_kv_shape* shape, int rows, const void* k,
                                        int64_t k_row, int64_t k_head, const void* v, int64_t v_row,
                                        int64_t v_head, const int64_t* slots,
                                        const sv_kv_pool* k_pool, const sv_kv_pool* v_pool,
                                        float* k_scale, float* v_scale, int block,
                                        sv_stream_t stream) {
  sv_status s = check_kv_shape(shape, false);
  if (s == SV_OK) s = check_block(shape, block);
  if (s != SV_OK) return s;
  if (rows < 0) return SV_ERR_INVALID_ARG;
  if (rows > 1 << 30) return SV_ERR_UNSUPPORTED;
  if (rows == 0) return SV_OK;
  if (check_pool8(k_pool) != SV_OK || check_pool8(v_pool) != SV_OK) return SV_ERR_INVALID_ARG;
  if (!k || !v || !slots || !k_scale || !v_scale || !aligned_to(k, 16) || !aligned_to(v, 16) ||
      !aligned_to(slots, 8) || !aligned_to(k_scale, 4) || !aligned_to(v_scale, 4))
    return SV_ERR_INVALID_ARG;
  for (int64_t st : {k_row, k_head, v_row, v_head})
    if (st < 0 || st % 8 != 0 || st >= (1ll << 39)) return SV_ERR_INVALID_ARG;
  // no two warps may write one block's codes or scale
  if (k_pool->data == v_pool->data || !heads_apart(shape, k_pool) || !heads_apart(shape, v_pool))
    return SV_ERR_INVALID_ARG;
  const uint64_t scales = (uint64_t)shape->num_pages * (shape->page_size / block) * shape->Hkv * sizeof(float);
  const uintptr_t ka = reinterpret_cast<uintptr_t>(k_scale), va = reinterpret_cast<uintptr_t>(v_scale);
  if ((ka < va ? va - ka : ka - va) < scales) return SV_ERR_INVALID_ARG;
  const AppendArgs A{{static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v)},
                     {k_row, v_row},
                     {k_head, v_head},
                     {static_cast<unsigned char*>(k_pool->data), static_cast<unsigned char*>(v_pool->data)},
                     {k_pool->page_stride, v_pool->page_stride},
                     {k_pool->token_stride, v_pool->token_stride},
                     {k_pool->head_stride, v_pool->head_stride},
                     {k_scale, v_scale},
                     slots,
                     (int64_t)shape->num_pages * shape->page_size,
                     rows,
                     shape->Hkv,
                     log2_of(shape->page_size),
                     log2_of(block)};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return shape->dtype == SV_KV_BF16 ? launch_append_width<true>(shape->D, A, st)
                                    : launch_append_width<false>(shape->D, A, st);
}
