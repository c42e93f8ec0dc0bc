// sv_logits.cu — penalties, biases and an allowed-token mask over the logit rows of a verify.
//
// One CTA takes one chunk of the vocabulary of one request, for all the request's rows. It
// first builds in shared memory what is the same for every row of the chunk:
//   add[v]   = bias(v) - f * c(v) - pi * [c(v) > 0]  with c over the history's output part
//   seen bits (v occurs in the history), touched bits (seen, biased or drafted), draft bits
// by scanning the request's whole history (a few tens of KiB out of L2) and keeping the tokens
// that fall into the chunk. The counts are integers until they are final, and the biases are
// entered in order by one warp, so the result does not depend on the order of atomics. A token
// drafted in this step (at most 16 per request) takes its count at a row's position from the
// drafts themselves, so no row waits for another one.
//
// The rows themselves never pass through registers as a whole: a ring of row pieces is copied
// in and out of shared memory by bulk copies, and the threads only visit the 16-byte vectors
// that the mask or a touched token changes, in place. Bound: reading and writing the rows. (A
// first form that streamed every vector through registers, with the penalties inlined for all
// its elements, ran at 46 % of the copy rate: its code did not fit the instruction cache.)
// Rows whose V or addresses do not allow 16-byte copies take a second kernel, element by element.
//
// Measured in graph replays, of the 6782 GB/s a copy reaches: 512 requests x 9 rows of 128256 bf16
// with histories of 8192, 64 biases and masks 377 us (2098 MB, 82 %; the scan of the histories,
// which each of a request's 32 chunks repeats, is about 50 us of it, but shared by clusters of 2, 4
// or 8 CTAs, over distributed shared memory, the call took 467, 578 and 607 us); 64 x 6 rows of 32000 bf16 with masks
// 14.2 us (46 MB); one request of 5 rows of 50257 fp32 5.3 us.

#include <cstdint>

#include <cuda_bf16.h>

#include "specverify_logits.h"
#include "sv_device.cuh"
#include "sv_host.h"

namespace sv {

constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s: far past any legitimate wait

int device_sm_count();

namespace {

constexpr int kAdjThreads = 256;
constexpr int kMaxDraft = SV_MAX_K;

struct AdjustArgs {
  const void* in;
  void* out;
  int64_t in_req, in_row, out_req, out_row;
  const int32_t *history, *hist_len, *prompt_len, *draft, *num_draft;
  const float *rep, *pres, *freq;
  const int32_t* bias_tok;
  const float* bias_val;
  const uint32_t* allowed;
  int L_max, n_bias, B, P, V, W;
  int log_chunk;  // tokens per chunk, 1024 to 4096, a power of two
  uint64_t wait_ns;          // the limit of a wait
  unsigned int more_arrivals;  // (self-test) the last stage's barrier waits for as many more
};

// E elements of a row as floats, and back (one rounding).
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int E = 4;
  __device__ static __forceinline__ float get(const uint4& v, int l) {
    return F32::get(v, l);
  }
  __device__ static __forceinline__ uint4 pack(const float (&y)[4]) {
    return make_uint4(__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]),
                      __float_as_uint(y[3]));
  }
  __device__ static __forceinline__ float load1(const float* p) { return *p; }
  __device__ static __forceinline__ void store1(float* p, float y) { *p = y; }
  // v with the elements whose bit of `ok` is clear set to -inf
  __device__ static __forceinline__ uint4 mask(uint4 v, uint32_t ok) {
    v.x = (ok & 1u) ? v.x : F32::kNegInfBits;
    v.y = (ok & 2u) ? v.y : F32::kNegInfBits;
    v.z = (ok & 4u) ? v.z : F32::kNegInfBits;
    v.w = (ok & 8u) ? v.w : F32::kNegInfBits;
    return v;
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int E = 8;
  __device__ static __forceinline__ float get(const uint4& v, int l) {
    return BF16::get(v, l);
  }
  __device__ static __forceinline__ uint32_t two(float a, float b) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&p);
  }
  __device__ static __forceinline__ uint4 pack(const float (&y)[8]) {
    return make_uint4(two(y[0], y[1]), two(y[2], y[3]), two(y[4], y[5]), two(y[6], y[7]));
  }
  __device__ static __forceinline__ float load1(const __nv_bfloat16* p) {
    return __bfloat162float(*p);
  }
  __device__ static __forceinline__ void store1(__nv_bfloat16* p, float y) {
    *p = __float2bfloat16_rn(y);
  }
  // Two words of four elements under four bits: the bits go to the signs of four bytes, and a
  // byte permutation that replicates signs widens each to an element.
  __device__ static __forceinline__ void mask4(uint32_t& a, uint32_t& b, uint32_t ok) {
    const uint32_t signs = ((ok & 15u) * 0x10204080u) & 0x80808080u;
    uint32_t ka, kb;
    asm("prmt.b32 %0, %1, 0, 0x9988;" : "=r"(ka) : "r"(signs));
    asm("prmt.b32 %0, %1, 0, 0xbbaa;" : "=r"(kb) : "r"(signs));
    a = (a & ka) | (0xff80ff80u & ~ka);
    b = (b & kb) | (0xff80ff80u & ~kb);
  }
  __device__ static __forceinline__ uint4 mask(uint4 v, uint32_t ok) {
    mask4(v.x, v.y, ok);
    mask4(v.z, v.w, ok >> 4);
    return v;
  }
};

// The chunk's tables in shared memory.
struct Tables {
  float* add;
  uint32_t *seen, *touched, *drafted, *listed;  // one bit per token of the chunk
};

struct RowRule {
  float rho, inv, pi, f;
  const int32_t* x;       // the request's drafted tokens, relative to the chunk (shared)
  const int32_t* x_said;  // whether the history's output part already holds x_t (shared)
};

// The adjusted value of token t (relative to the chunk) with logit z at position i.
__device__ __forceinline__ float adjusted(const Tables& T, const RowRule& r, int t, float z,
                                          int i) {
  bool seen = (T.seen[t >> 5] >> (t & 31)) & 1u;
  float a = T.add[t];
  if ((T.drafted[t >> 5] >> (t & 31)) & 1u) {
    int m = 0;
    bool said = false;
    for (int s = 0; s < i; ++s)
      if (r.x[s] == t) {
        ++m;
        said = r.x_said[s] != 0;
      }
    if (m > 0) {
      seen = true;
      a -= r.f * (float)m + (said ? 0.0f : r.pi);
    }
  }
  const float y = seen ? (z > 0.0f ? z * r.inv : z * r.rho) : z;
  return y + a;
}

// Row pieces in flight, of 8 KiB: five CTAs fit an SM with three, four with four (512 requests x 9
// rows of 128256 bf16: 374 and 395 us; with two 455).
constexpr int kAdjStages = 3;
// A chunk with up to kListed touched tokens lists them, and its threads share the list out; in one
// with more each thread visits its own vectors. (Of text that repeats, the chunk of the most
// frequent tokens is nearly full, the others hold a few percent: with the vectors alone a warp
// walked some hit in almost every 32 of them.)
constexpr int kListed = 1024;

// What every thread of a CTA knows of its request and chunk.
struct Chunk {
  int b, c0, c1, n, prompt, nd;
  bool bad;
};
__device__ __forceinline__ Chunk chunk_of(const AdjustArgs& A) {
  Chunk c;
  c.b = blockIdx.x % A.B;  // (the chunks of the lowest, most frequent tokens first)
  c.c0 = (int)(blockIdx.x / A.B) << A.log_chunk;
  c.c1 = c.c0 + (1 << A.log_chunk) < A.V ? c.c0 + (1 << A.log_chunk) : A.V;
  c.n = A.hist_len ? __ldg(A.hist_len + c.b) : 0;
  c.prompt = A.prompt_len ? __ldg(A.prompt_len + c.b) : 0;
  c.nd = A.num_draft ? __ldg(A.num_draft + c.b) : A.P - 1;
  c.bad = c.n < 0 || c.n > A.L_max || c.prompt < 0 || c.prompt > c.n || c.nd < 0 ||
          c.nd > A.P - 1;
  return c;
}

struct DraftShared {
  int32_t x[kMaxDraft], said[kMaxDraft];
};

// Builds the chunk's tables (all threads; ends with a CTA barrier).
__device__ __forceinline__ void build_tables(const AdjustArgs& A, const Chunk& c,
                                             unsigned char* smem, int my_draft,
                                             DraftShared& D, Tables& S, RowRule& r) {
  const int C = 1 << A.log_chunk, tid = threadIdx.x, lane = tid & 31, b = c.b;
  S.add = reinterpret_cast<float*>(smem);
  S.seen = reinterpret_cast<uint32_t*>(smem + 4 * (size_t)C);
  S.touched = S.seen + C / 32;
  S.drafted = S.touched + C / 32;
  S.listed = S.drafted + C / 32;
  uint32_t* cnt = reinterpret_cast<uint32_t*>(S.add);
  r.rho = A.rep ? __ldg(A.rep + b) : 1.0f;
  r.inv = 1.0f / r.rho;
  r.pi = A.pres ? __ldg(A.pres + b) : 0.0f;
  r.f = A.freq ? __ldg(A.freq + b) : 0.0f;
  r.x = D.x;
  r.x_said = D.said;
  const int ndraft = A.draft ? c.nd : 0;
  {
    uint4* z = reinterpret_cast<uint4*>(smem);
    const int n16 = (C * 4 + 4 * (C / 32) * 4) / 16;
#pragma unroll 4
    for (int q = tid; q < n16; q += kAdjThreads) z[q] = make_uint4(0u, 0u, 0u, 0u);
  }
  __syncthreads();
  if (A.history) {
    const int32_t* h = A.history + (int64_t)b * A.L_max;
    const int here = c.c1 - c.c0;
    auto enter = [&](int q, int t) {
      const int v = t - c.c0;
      if ((unsigned)v < (unsigned)here && q < c.n) {
        atomicOr(&S.seen[v >> 5], 1u << (v & 31));
        if (q >= c.prompt) atomicAdd(&cnt[v], 1u);
      }
    };
    constexpr int U = 8;
    // four tokens a load where the row allows (rows are L_max long, a multiple of 4)
    if (A.L_max % 4 == 0 && (reinterpret_cast<uintptr_t>(h) & 15) == 0) {
#pragma unroll 1
      for (int q0 = 4 * tid; q0 < c.n; q0 += 4 * U * kAdjThreads) {
        int4 t[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int q = q0 + 4 * u * kAdjThreads;
          t[u] = q < c.n ? __ldg(reinterpret_cast<const int4*>(h + q)) : make_int4(-1, -1, -1, -1);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int q = q0 + 4 * u * kAdjThreads;
          if (q >= c.n) break;
          enter(q, t[u].x);
          enter(q + 1, t[u].y);
          enter(q + 2, t[u].z);
          enter(q + 3, t[u].w);
        }
      }
    } else {
#pragma unroll 1
      for (int q0 = tid; q0 < c.n; q0 += U * kAdjThreads) {
        int t[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int q = q0 + u * kAdjThreads;
          t[u] = q < c.n ? __ldg(h + q) : -1;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) enter(q0 + u * kAdjThreads, t[u]);
      }
    }
  }
  __syncthreads();
  if (tid < ndraft) {
    const int v = my_draft - c.c0;
    const bool here = (unsigned)v < (unsigned)(c.c1 - c.c0);
    D.x[tid] = here ? v : -1;
    D.said[tid] = here && cnt[v] > 0;
    if (here) atomicOr(&S.drafted[v >> 5], 1u << (v & 31));
  }
  __syncthreads();
#pragma unroll 1
  for (int w = tid; w < C / 32; w += kAdjThreads) {
    uint32_t m = S.seen[w];
    S.touched[w] = m | S.drafted[w];
#pragma unroll 1
    for (; m; m &= m - 1) {
      const int v = 32 * w + __ffs(m) - 1;
      const uint32_t k = cnt[v];
      S.add[v] = k ? -(r.f * (float)k) - r.pi : 0.0f;
    }
  }
  if (A.n_bias > 0) {
    __syncthreads();
    if (tid < 32) {
      const int32_t* bt = A.bias_tok + (int64_t)b * A.n_bias;
      const float* bv = A.bias_val + (int64_t)b * A.n_bias;
      // entries in order, 32 at a time: a token's first entry counts (listed bits)
#pragma unroll 1
      for (int q0 = 0; q0 < A.n_bias; q0 += 32) {
        const int q = q0 + lane;
        const int v = (q < A.n_bias ? __ldg(bt + q) : -1) - c.c0;
        const bool here = q < A.n_bias && (unsigned)v < (unsigned)(c.c1 - c.c0);
        if (!__any_sync(0xffffffffu, here)) continue;
        const uint32_t same = __match_any_sync(0xffffffffu, here ? v : -1 - lane);
        const bool first = here && (__ffs(same) - 1) == lane &&
                           !((S.listed[v >> 5] >> (v & 31)) & 1u);
        __syncwarp();
        if (first) {
          S.add[v] += __ldg(bv + q);
          atomicOr(&S.touched[v >> 5], 1u << (v & 31));
          atomicOr(&S.listed[v >> 5], 1u << (v & 31));
        }
        __syncwarp();
      }
    }
  }
  __syncthreads();
}

// Bulk copy of shared memory to global memory (both 16-byte aligned, a multiple of 16 bytes).
__device__ __forceinline__ void bulk_s2g(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst),
               "r"(smem_u32(src)), "r"(bytes)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
template <int kPending>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kPending) : "memory");
}

// The rest of a wait for row i's copy.
__device__ __noinline__ void wait_row(uint64_t* bar, uint32_t phase, uint64_t limit_ns, int* lost_row,
                                      int i) {
  if (!mbar_wait(bar, phase, limit_ns)) atomicMin(lost_row, i);
}

// The copy of row i never came: that row and those after it are NaN, once no copy is in flight any
// more. All threads.
template <typename T>
__device__ __noinline__ void give_up(const AdjustArgs& A, uint64_t* full, int i, int rows, int nvec,
                                     T* out) {
  using X = Vec<T>;
  if (threadIdx.x == 0) {
    for (int r = i; r < kAdjStages + i && r < rows; ++r)
      mbar_wait(&full[r % kAdjStages], (uint32_t)(r / kAdjStages) & 1u, A.wait_ns);
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // (row i is on its way out)
  }
  __syncthreads();
  const float nan[8] = {NAN, NAN, NAN, NAN, NAN, NAN, NAN, NAN};
  const uint4 v = X::pack(reinterpret_cast<const float(&)[X::E]>(nan));
#pragma unroll 1
  for (int r = i; r < rows; ++r)
#pragma unroll 1
    for (int q = threadIdx.x; q < nvec; q += kAdjThreads)
      *reinterpret_cast<uint4*>(out + r * A.out_row + q * X::E) = v;
}

// Rows in 16-byte vectors.
template <typename T>
__global__ void __launch_bounds__(kAdjThreads) adjust_kernel(const AdjustArgs A) {
  using X = Vec<T>;
  constexpr int E = X::E;
  constexpr uint32_t kFull = (1u << E) - 1u;
  extern __shared__ __align__(128) unsigned char adj_smem[];
  __shared__ DraftShared D;
  __shared__ __align__(8) uint64_t full[kAdjStages];
  __shared__ uint16_t list[kListed];
  __shared__ int warp_count[kAdjThreads / 32];
  __shared__ int lost_row;  // the first whose copy never came
  const int tid = threadIdx.x;
  const int b0 = blockIdx.x % A.B;
  const int my_draft =
      A.draft && threadIdx.x < A.P - 1 ? __ldg(A.draft + (int64_t)b0 * (A.P - 1) + threadIdx.x) : -1;
  const Chunk c = chunk_of(A);
  const T* in = static_cast<const T*>(A.in) + c.b * A.in_req + c.c0;
  T* out = static_cast<T*>(A.out) + c.b * A.out_req + c.c0;
  const int rows = c.bad ? A.P : c.nd + 1, nvec = (c.c1 - c.c0) / E;
  const uint32_t bytes = (uint32_t)nvec * 16u;
  unsigned char* ring = adj_smem;
  const int stage = (int)sizeof(T) << A.log_chunk;
  if (c.bad) {
    const float nan[8] = {NAN, NAN, NAN, NAN, NAN, NAN, NAN, NAN};
    const uint4 v = X::pack(reinterpret_cast<const float(&)[E]>(nan));
    for (int i = 0; i < rows; ++i)
      for (int q = tid; q < nvec; q += kAdjThreads)
        *reinterpret_cast<uint4*>(out + i * A.out_row + q * E) = v;
    return;
  }
  if (tid == 0) {
    lost_row = INT32_MAX;
    for (int s = 0; s < kAdjStages; ++s)
      mbar_init(&full[s], s == kAdjStages - 1 ? 1 + A.more_arrivals : 1);
    fence_barrier_init();
    for (int i = 0; i < kAdjStages && i < rows; ++i) {
      mbar_arrive_expect_tx(&full[i], bytes);
      bulk_g2s(ring + i * stage, in + i * A.in_row, bytes, &full[i]);
    }
  }
  // A thread's vectors are q = tid + u * kAdjThreads; kVecs of them cover the largest chunk. Their
  // touched bits stay in registers, their masks are loaded a row ahead.
  constexpr int kVecs = 2;
  const uint8_t* const allowed =
      A.allowed ? reinterpret_cast<const uint8_t*>(A.allowed + (int64_t)c.b * A.P * A.W) + c.c0 / 8
                : nullptr;
  uint32_t touch[kVecs], next_ok[kVecs];
  auto load_ok = [&](int i) {
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      const int q = tid + u * kAdjThreads, at = E == 8 ? q : q >> 1;
      next_ok[u] = 0xffu;
      if (allowed && i < rows && q < nvec) next_ok[u] = __ldg(allowed + (int64_t)i * A.W * 4 + at);
    }
  };
  load_ok(0);
  Tables S;
  RowRule r;
  build_tables(A, c, adj_smem + kAdjStages * stage, my_draft, D, S, r);
  const uint8_t* touched = reinterpret_cast<const uint8_t*>(S.touched);

  // The touched tokens in ascending order, a word of their bits per thread.
  int count = 0;
  {
    const int lane = tid & 31, warp = tid >> 5;
    uint32_t m = tid < (1 << A.log_chunk) / 32 ? S.touched[tid] : 0u;
    int at = __popc(m);
    const int mine = at;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, at, o);
      if (lane >= o) at += y;
    }
    if (lane == 31) warp_count[warp] = at;
    __syncthreads();
    at -= mine;
#pragma unroll
    for (int q = 0; q < kAdjThreads / 32; ++q) {
      if (q < warp) at += warp_count[q];
      count += warp_count[q];
    }
    if (count <= kListed)
#pragma unroll 1
      for (; m; m &= m - 1) list[at++] = (uint16_t)(32 * tid + __ffs(m) - 1);
    __syncthreads();
  }
  const bool listed = count <= kListed;

#pragma unroll
  for (int u = 0; u < kVecs; ++u) {
    const int q = tid + u * kAdjThreads, at = E == 8 ? q : q >> 1;
    touch[u] = q < nvec ? (uint32_t)(touched[at] >> (E == 8 ? 0 : 4 * (q & 1))) & kFull : 0u;
  }
  auto bits_of = [&](const uint32_t* bits, int q) {
    const uint8_t byte = reinterpret_cast<const uint8_t*>(bits)[E == 8 ? q : q >> 1];
    return (uint32_t)(byte >> (E == 8 ? 0 : 4 * (q & 1))) & kFull;
  };
  auto drafted_of = [&](int q) { return bits_of(S.drafted, q); };
  auto seen_of = [&](int q) { return bits_of(S.seen, q); };
  int s = 0;
  uint32_t phase = 0;
#pragma unroll 1
  for (int i = 0; i < rows; ++i) {
    unsigned char* buf = ring + s * stage;
    uint32_t ok[kVecs];
#pragma unroll
    for (int u = 0; u < kVecs; ++u)
      ok[u] = (next_ok[u] >> (E == 8 ? 0 : 4 * ((tid + u * kAdjThreads) & 1))) & kFull;
    load_ok(i + 1);
    if (!mbar_try_wait(&full[s], phase)) wait_row(&full[s], phase, A.wait_ns, &lost_row, i);
    if (listed && count > 0) {
#pragma unroll 1
      for (int e = tid; e < count; e += kAdjThreads) {
        T* z = reinterpret_cast<T*>(buf) + list[e];
        X::store1(z, adjusted(S, r, list[e], X::load1(z), i));
      }
      if (allowed) __syncthreads();  // the masks, by vectors, come last
    }
#pragma unroll 1
    for (int u = 0; u < kVecs; ++u) {
      const int q = tid + u * kAdjThreads;
      if (q >= nvec) break;
      uint4* v = reinterpret_cast<uint4*>(buf) + q;
      const uint32_t may = u == 0 ? ok[0] : ok[1];
      if (!listed) {
        const uint32_t hit = u == 0 ? touch[0] : touch[1];
        if (hit & may) {
          const uint32_t drafts = drafted_of(q);
          uint4 w = *v;
          float y[E];
#pragma unroll
          for (int l = 0; l < E; ++l) y[l] = X::get(w, l);
          if (__builtin_expect(drafts != 0, 0)) {
#pragma unroll
            for (int l = 0; l < E; ++l)
              if ((hit >> l) & 1u) y[l] = adjusted(S, r, q * E + l, y[l], i);
          } else {
            const uint32_t seen = seen_of(q);
#pragma unroll
            for (int l = 0; l < E; ++l) {
              const float z = y[l];
              y[l] = ((seen >> l) & 1u ? (z > 0.0f ? z * r.inv : z * r.rho) : z) +
                     S.add[q * E + l];
            }
          }
          *v = X::pack(y);
        }
      }
      if (may != kFull) *v = X::mask(may ? *v : make_uint4(0u, 0u, 0u, 0u), may);
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
    const int lost = *(volatile int*)&lost_row;
    if (tid == 0) {
      bulk_s2g(out + i * A.out_row, buf, bytes);
      // the piece before this one has left its buffer: the next row into it
      const int next = i - 1 + kAdjStages;
      if (i > 0 && next < rows) {
        bulk_wait_read<1>();
        const int sb = s == 0 ? kAdjStages - 1 : s - 1;
        mbar_arrive_expect_tx(&full[sb], bytes);
        bulk_g2s(ring + sb * stage, in + next * A.in_row, bytes, &full[sb]);
      }
    }
    // (a thread ahead may have lost a later row: that one's barrier tells all)
    if (__builtin_expect(lost <= i, 0)) {
      give_up<T>(A, full, i, rows, nvec, out);
      return;
    }
    if (++s == kAdjStages) {
      s = 0;
      phase ^= 1u;
    }
  }
  if (tid == 0) bulk_wait_read<0>();
}

// Rows that 16-byte vectors do not divide: element by element.
template <typename T>
__global__ void __launch_bounds__(kAdjThreads) adjust_any_kernel(const AdjustArgs A) {
  using X = Vec<T>;
  extern __shared__ __align__(128) unsigned char adj_smem[];
  __shared__ DraftShared D;
  const int b0 = blockIdx.x % A.B;
  const int my_draft =
      A.draft && threadIdx.x < A.P - 1 ? __ldg(A.draft + (int64_t)b0 * (A.P - 1) + threadIdx.x) : -1;
  const Chunk c = chunk_of(A);
  const T* in = static_cast<const T*>(A.in) + c.b * A.in_req;
  T* out = static_cast<T*>(A.out) + c.b * A.out_req;
  if (c.bad) {
    for (int i = 0; i < A.P; ++i)
      for (int j = c.c0 + threadIdx.x; j < c.c1; j += kAdjThreads)
        X::store1(out + i * A.out_row + j, NAN);
    return;
  }
  Tables S;
  RowRule r;
  build_tables(A, c, adj_smem, my_draft, D, S, r);
  const uint32_t* allowed = A.allowed ? A.allowed + (int64_t)c.b * A.P * A.W : nullptr;
#pragma unroll 1
  for (int i = 0; i <= c.nd; ++i) {
    const uint32_t* ok = allowed ? allowed + (int64_t)i * A.W : nullptr;
    constexpr int U = 4;
#pragma unroll 1
    for (int j0 = c.c0 + threadIdx.x; j0 < c.c1; j0 += U * kAdjThreads) {
      float z[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j = j0 + u * kAdjThreads;
        z[u] = 0.0f;
        if (j < c.c1)
          z[u] = ok && !((__ldg(ok + (j >> 5)) >> (j & 31)) & 1u)
                     ? __uint_as_float(F32::kNegInfBits)
                     : X::load1(in + i * A.in_row + j);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j = j0 + u * kAdjThreads, t = j - c.c0;
        if (j >= c.c1) break;
        const bool masked = ok && !((__ldg(ok + (j >> 5)) >> (j & 31)) & 1u);
        if (!masked && ((S.touched[t >> 5] >> (t & 31)) & 1u)) z[u] = adjusted(S, r, t, z[u], i);
        X::store1(out + i * A.out_row + j, z[u]);
      }
    }
  }
}

template <typename T>
sv_status launch_adjust(AdjustArgs A, bool aligned, cudaStream_t st) {
  // Chunks of 4096 bf16 or 2048 fp32 logits, or half of that (each scans the history) while they
  // would leave SMs without work. (512 requests of 9 rows of 128256 bf16, four pieces in flight:
  // 405 us in chunks of 4096, 478 us of 2048, 472 us of 8192, whose tables leave room for fewer
  // CTAs.)
  const int64_t wanted = 2 * (int64_t)device_sm_count();
  constexpr int least = sizeof(T) == 4 ? 10 : 11;
  A.log_chunk = least + 1;
  while (A.log_chunk > least && (((int64_t)A.V - 1) / (1 << A.log_chunk) + 1) * A.B < wanted)
    --A.log_chunk;
  const int64_t chunks = ((int64_t)A.V + (1 << A.log_chunk) - 1) >> A.log_chunk;
  const int64_t grid = chunks * A.B;
  if (grid >= (1ll << 31)) return SV_ERR_UNSUPPORTED;
  const size_t tables = ((size_t)4 << A.log_chunk) + 4 * (((size_t)1 << A.log_chunk) / 8);
  const size_t smem = tables + (aligned ? kAdjStages * (sizeof(T) << A.log_chunk) : 0);
  // The largest chunk's tables and ring and the static shared memory stay within what every launch
  // may have: no limit is raised (one raised per call could be lowered under another thread's launch).
  constexpr int kMost = least + 1;
  constexpr size_t kStatic = sizeof(DraftShared) + 8 * kAdjStages + 2 * kListed + kAdjThreads / 8;
  static_assert((4u << kMost) + (1u << kMost) / 2 + kAdjStages * (sizeof(T) << kMost) + kStatic + 64 <=
                    48 * 1024,
                "shared memory");
  auto kernel = aligned ? adjust_kernel<T> : adjust_any_kernel<T>;
  kernel<<<(unsigned)grid, kAdjThreads, smem, st>>>(A);
  return launch_status();
}

sv_status adjust(const void* logits, int64_t in_req_stride, int64_t in_row_stride, sv_dtype dtype,
                 const int32_t* history, const int32_t* hist_len, const int32_t* prompt_len,
                 int L_max, const int32_t* draft_tokens, const int32_t* num_draft,
                 const float* repetition, const float* presence, const float* frequency,
                 const int32_t* bias_tokens, const float* bias_values, int n_bias,
                 const uint32_t* allowed, int B, int P, int V, void* out,
                 int64_t out_req_stride, int64_t out_row_stride,
                 uint64_t wait_ns, unsigned int more_arrivals, sv_stream_t stream) {
  if (B < 0 || P < 1 || V < 1 || L_max < 0 || n_bias < 0) return SV_ERR_INVALID_ARG;
  if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_INVALID_ARG;
  if (P > SV_MAX_K + 1 || L_max >= (1 << 30)) return SV_ERR_UNSUPPORTED;
  if (B == 0) return SV_OK;
  if (!logits || !out) return SV_ERR_INVALID_ARG;
  if (history ? (!hist_len || L_max < 1) : (hist_len || prompt_len || L_max != 0))
    return SV_ERR_INVALID_ARG;
  if (n_bias > 0 ? (!bias_tokens || !bias_values) : (bias_tokens || bias_values))
    return SV_ERR_INVALID_ARG;
  if (in_row_stride < (P > 1 ? V : 0) || out_row_stride < (P > 1 ? V : 0) ||
      in_req_stride < 0 || out_req_stride < 0)
    return SV_ERR_INVALID_ARG;
  if (B > 1 && (in_req_stride < (P - 1) * in_row_stride + V ||
                out_req_stride < (P - 1) * out_row_stride + V))
    return SV_ERR_INVALID_ARG;
  const size_t eb = (size_t)elem_bytes(dtype);
  if (!aligned_to(logits, eb) || !aligned_to(out, eb) || !aligned_to(history, 4) ||
      !aligned_to(hist_len, 4) || !aligned_to(prompt_len, 4) || !aligned_to(draft_tokens, 4) ||
      !aligned_to(num_draft, 4) || !aligned_to(repetition, 4) || !aligned_to(presence, 4) ||
      !aligned_to(frequency, 4) || !aligned_to(bias_tokens, 4) || !aligned_to(bias_values, 4) ||
      !aligned_to(allowed, 4))
    return SV_ERR_INVALID_ARG;
  if (logits == out && (in_req_stride != out_req_stride || in_row_stride != out_row_stride))
    return SV_ERR_INVALID_ARG;
  AdjustArgs A{logits, out, in_req_stride, in_row_stride, out_req_stride, out_row_stride,
               history, hist_len, prompt_len, draft_tokens, num_draft, repetition, presence,
               frequency, bias_tokens, bias_values, allowed, L_max, n_bias, B, P, V,
               (V + 31) / 32, 13, wait_ns, more_arrivals};
  const int E = 16 / (int)eb;
  const bool aligned = aligned_to(logits, 16) && aligned_to(out, 16) && V % E == 0 &&
                       (P == 1 || (in_row_stride % E == 0 && out_row_stride % E == 0)) &&
                       (B == 1 || (in_req_stride % E == 0 && out_req_stride % E == 0));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return dtype == SV_F32 ? launch_adjust<float>(A, aligned, st)
                         : launch_adjust<__nv_bfloat16>(A, aligned, st);
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" sv_status logit_adjust(const void* logits, int64_t in_req_stride,
                                  int64_t in_row_stride, sv_dtype dtype,
                                  const int32_t* history, const int32_t* hist_len,
                                  const int32_t* prompt_len, int L_max,
                                  const int32_t* draft_tokens, const int32_t* num_draft,
                                  const float* repetition, const float* presence,
                                  const float* frequency, const int32_t* bias_tokens,
                                  const float* bias_values, int n_bias,
                                  const uint32_t* allowed, int B, int P, int V, void* out,
                                  int64_t out_req_stride, int64_t out_row_stride,
                                  sv_stream_t stream) {
  return adjust(logits, in_req_stride, in_row_stride, dtype, history, hist_len, prompt_len, L_max,
                draft_tokens, num_draft, repetition, presence, frequency, bias_tokens,
                bias_values, n_bias, allowed, B, P, V, out, out_req_stride, out_row_stride,
                kWaitLimitNs, 0u, stream);
}

extern "C" sv_status logit_adjust_wait_selftest(
    const void* logits, int64_t in_req_stride, int64_t in_row_stride, sv_dtype dtype,
    const int32_t* history, const int32_t* hist_len, const int32_t* prompt_len,
    int L_max, const int32_t* draft_tokens, const int32_t* num_draft,
    const float* repetition, const float* presence, const float* frequency,
    const int32_t* bias_tokens, const float* bias_values, int n_bias,
    const uint32_t* allowed, int B, int P, int V, void* out,
    int64_t out_req_stride, int64_t out_row_stride, unsigned int wait_us,
    sv_stream_t stream) {
  if (wait_us < 1000 || wait_us > 100000) return SV_ERR_INVALID_ARG;
  return adjust(logits, in_req_stride, in_row_stride, dtype, history, hist_len, prompt_len, L_max,
                draft_tokens, num_draft, repetition, presence, frequency, bias_tokens,
                bias_values, n_bias, allowed, B, P, V, out, out_req_stride, out_row_stride,
                (uint64_t)wait_us * 1000ull, 1u, stream);
}
