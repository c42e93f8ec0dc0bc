// sv_logits.cu — penalties, biases and an allowed-token mask over the logit rows of a verify.
//
// One CTA takes one chunk of the vocabulary of one request, for all the request's rows. It
// first builds in shared memory what is the same for every row of the chunk:
//   add[v]   = bias(v) - f * c(v) - pi * [c(v) > 0]  with c over the history's output part
//   seen bits (v occurs in the history), touched bits (seen, biased or drafted), draft bits
// by scanning the request's whole history (a few tens of KiB out of L2) and keeping the tokens
// that fall into the chunk. The rows then stream through registers once, 16 bytes at a time:
//   - a vector with no touched token is copied as it is, or set to -inf under the mask,
//     without being read where the mask allows none of it;
//   - one with touched tokens takes y = (seen ? (z > 0 ? z / rho : z * rho) : z) + add;
//   - a token drafted in this step (at most 16 per request) takes its count at this row's
//     position from the drafts themselves, so no row waits for another one.
// The counts are integers until they are final, and the biases are entered in order by one
// warp, so the result does not depend on the order of atomics.
#include <cstdint>

#include <cuda_bf16.h>

#include "specverify_logits.h"
#include "sv_device.cuh"
#include "sv_host.h"

namespace sv {

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
  int log_chunk;  // tokens per chunk, a power of two >= 1024
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
  __device__ static __forceinline__ uint32_t mask2(uint32_t w, uint32_t ok) {
    const uint32_t keep = ((ok & 1u) ? 0xffffu : 0u) | ((ok & 2u) ? 0xffff0000u : 0u);
    return (w & keep) | (0xff80ff80u & ~keep);
  }
  __device__ static __forceinline__ uint4 mask(uint4 v, uint32_t ok) {
    return make_uint4(mask2(v.x, ok), mask2(v.y, ok >> 2), mask2(v.z, ok >> 4),
                      mask2(v.w, ok >> 6));
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

template <typename T, bool kAligned>
__global__ void __launch_bounds__(kAdjThreads) adjust_kernel(const AdjustArgs A) {
  using X = Vec<T>;
  constexpr int E = X::E;
  extern __shared__ __align__(16) unsigned char adj_smem[];
  __shared__ int32_t s_draft[kMaxDraft], s_said[kMaxDraft];
  const int C = 1 << A.log_chunk;
  const int tid = threadIdx.x, lane = tid & 31;
  const int b = blockIdx.x % A.B, c0 = (blockIdx.x / A.B) << A.log_chunk;
  const int c1 = c0 + C < A.V ? c0 + C : A.V;

  const int n = A.hist_len ? __ldg(A.hist_len + b) : 0;
  const int prompt = A.prompt_len ? __ldg(A.prompt_len + b) : 0;
  const int nd = A.num_draft ? __ldg(A.num_draft + b) : A.P - 1;
  const T* in = static_cast<const T*>(A.in) + b * A.in_req;
  T* out = static_cast<T*>(A.out) + b * A.out_req;
  if (n < 0 || n > A.L_max || prompt < 0 || prompt > n || nd < 0 || nd > A.P - 1) {
    for (int i = 0; i < A.P; ++i)
      for (int j = c0 + tid; j < c1; j += kAdjThreads)
        X::store1(out + i * A.out_row + j, __uint_as_float(0x7fc00000u));
    return;
  }

  // ---- the chunk's tables
  Tables S;
  S.add = reinterpret_cast<float*>(adj_smem);
  S.seen = reinterpret_cast<uint32_t*>(adj_smem + 4 * (size_t)C);
  S.touched = S.seen + C / 32;
  S.drafted = S.touched + C / 32;
  S.listed = S.drafted + C / 32;
  uint32_t* cnt = reinterpret_cast<uint32_t*>(S.add);
  RowRule r;
  r.rho = A.rep ? __ldg(A.rep + b) : 1.0f;
  r.inv = 1.0f / r.rho;
  r.pi = A.pres ? __ldg(A.pres + b) : 0.0f;
  r.f = A.freq ? __ldg(A.freq + b) : 0.0f;
  r.x = s_draft;
  r.x_said = s_said;
  const int ndraft = A.draft ? nd : 0;
  {
    uint4* z = reinterpret_cast<uint4*>(adj_smem);
    const int n16 = (C * 4 + 4 * (C / 32) * 4) / 16;
    for (int q = tid; q < n16; q += kAdjThreads) z[q] = make_uint4(0u, 0u, 0u, 0u);
  }
  __syncthreads();
  if (A.history) {
    const int32_t* h = A.history + (int64_t)b * A.L_max;
    constexpr int U = 4;
    for (int q0 = 0; q0 < n; q0 += U * kAdjThreads) {
      int t[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int q = q0 + u * kAdjThreads + tid;
        t[u] = q < n ? __ldg(h + q) : -1;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int q = q0 + u * kAdjThreads + tid;
        if (t[u] >= c0 && t[u] < c1) {
          const int v = t[u] - c0;
          atomicOr(&S.seen[v >> 5], 1u << (v & 31));
          if (q >= prompt) atomicAdd(&cnt[v], 1u);
        }
      }
    }
  }
  __syncthreads();
  if (tid < ndraft) {
    const int t = __ldg(A.draft + (int64_t)b * (A.P - 1) + tid);
    const bool here = t >= c0 && t < c1;
    s_draft[tid] = here ? t - c0 : -1;
    s_said[tid] = here && cnt[t - c0] > 0;
    if (here) atomicOr(&S.drafted[(t - c0) >> 5], 1u << ((t - c0) & 31));
  }
  __syncthreads();
  for (int w = tid; w < C / 32; w += kAdjThreads) {
    uint32_t m = S.seen[w];
    S.touched[w] = m | S.drafted[w];
    while (m) {
      const int v = 32 * w + __ffs(m) - 1;
      m &= m - 1;
      const uint32_t c = cnt[v];
      S.add[v] = c ? -(r.f * (float)c) - r.pi : 0.0f;
    }
  }
  if (A.n_bias > 0) {
    __syncthreads();
    if (tid < 32) {
      const int32_t* bt = A.bias_tok + (int64_t)b * A.n_bias;
      const float* bv = A.bias_val + (int64_t)b * A.n_bias;
      // entries in order, 32 at a time: a token's first entry counts (listed bits)
      for (int q0 = 0; q0 < A.n_bias; q0 += 32) {
        const int q = q0 + lane;
        const int t = q < A.n_bias ? __ldg(bt + q) : -1;
        const bool here = t >= c0 && t < c1;
        if (!__any_sync(0xffffffffu, here)) continue;
        const uint32_t same = __match_any_sync(0xffffffffu, here ? t : -1 - lane);
        const bool first = here && (__ffs(same) - 1) == lane &&
                           !((S.listed[(t - c0) >> 5] >> ((t - c0) & 31)) & 1u);
        __syncwarp();
        if (first) {
          const int v = t - c0;
          S.add[v] += __ldg(bv + q);
          atomicOr(&S.touched[v >> 5], 1u << (v & 31));
          atomicOr(&S.listed[v >> 5], 1u << (v & 31));
        }
        __syncwarp();
      }
    }
  }
  __syncthreads();

  // ---- the rows
  const uint32_t full = (1u << E) - 1u;
  const uint32_t* allowed = A.allowed ? A.allowed + (int64_t)b * A.P * A.W : nullptr;
  if (kAligned) {
    // vectors of the chunk, counted through all rows: 4 in flight per thread
    constexpr int U = 4;
    const int lv = A.log_chunk - (E == 8 ? 3 : 2);
    const int items = (nd + 1) << lv;
    for (int it0 = tid; it0 < items; it0 += U * kAdjThreads) {
      uint32_t ok[U];
      uint4 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int it = it0 + u * kAdjThreads;
        const int i = it >> lv, j = c0 + (it & ((1 << lv) - 1)) * E;
        ok[u] = 0;
        if (it < items && j < A.V) {
          ok[u] = full;
          if (allowed) {
            const uint8_t byte =
                __ldg(reinterpret_cast<const uint8_t*>(allowed + (int64_t)i * A.W) + (j >> 3));
            ok[u] = (E == 8 ? byte : byte >> (j & 4)) & full;
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int it = it0 + u * kAdjThreads;
        const int i = it >> lv, j = c0 + (it & ((1 << lv) - 1)) * E;
        v[u] = X::mask(make_uint4(0u, 0u, 0u, 0u), 0u);
        if (ok[u]) v[u] = *reinterpret_cast<const uint4*>(in + i * A.in_row + j);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int it = it0 + u * kAdjThreads;
        const int i = it >> lv, t = (it & ((1 << lv) - 1)) * E, j = c0 + t;
        if (it >= items || j >= A.V) continue;
        const uint32_t hit = (S.touched[t >> 5] >> (t & 31)) & full & ok[u];
        if (hit) {
          float y[E];
#pragma unroll
          for (int l = 0; l < E; ++l) {
            y[l] = X::get(v[u], l);
            if ((hit >> l) & 1u) y[l] = adjusted(S, r, t + l, y[l], i);
          }
          v[u] = X::pack(y);
        }
        if (ok[u] != full) v[u] = X::mask(v[u], ok[u]);
        *reinterpret_cast<uint4*>(out + i * A.out_row + j) = v[u];
      }
    }
  } else {
    for (int i = 0; i <= nd; ++i) {
      const T* zi = in + i * A.in_row;
      T* yi = out + i * A.out_row;
      const uint32_t* al = allowed ? allowed + (int64_t)i * A.W : nullptr;
      for (int j = c0 + tid; j < c1; j += kAdjThreads) {
        const int t = j - c0;
        if (al && !((__ldg(al + (j >> 5)) >> (j & 31)) & 1u)) {
          X::store1(yi + j, __uint_as_float(F32::kNegInfBits));
          continue;
        }
        float z = X::load1(zi + j);
        if ((S.touched[t >> 5] >> (t & 31)) & 1u) z = adjusted(S, r, t, z, i);
        X::store1(yi + j, z);
      }
    }
  }
}

template <typename T>
sv_status launch_adjust(const AdjustArgs& A, bool aligned, cudaStream_t st) {
  const int64_t chunks = ((int64_t)A.V + (1 << A.log_chunk) - 1) >> A.log_chunk;
  const int64_t grid = chunks * A.B;
  if (grid >= (1ll << 31)) return SV_ERR_UNSUPPORTED;
  const size_t smem = ((size_t)4 << A.log_chunk) + 4 * (((size_t)1 << A.log_chunk) / 8);
  auto kernel = aligned ? adjust_kernel<T, true> : adjust_kernel<T, false>;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return cuda_fail(e);
  kernel<<<(unsigned)grid, kAdjThreads, smem, st>>>(A);
  return launch_status();
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
  if (B < 0 || P < 1 || V < 1 || L_max < 0 || n_bias < 0) return SV_ERR_INVALID_ARG;
  if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_INVALID_ARG;
  if (P > SV_MAX_K + 1) return SV_ERR_UNSUPPORTED;
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
               (V + 31) / 32, 13};
  const int E = 16 / (int)eb;
  const bool aligned = aligned_to(logits, 16) && aligned_to(out, 16) && V % E == 0 &&
                       (P == 1 || (in_row_stride % E == 0 && out_row_stride % E == 0)) &&
                       (B == 1 || (in_req_stride % E == 0 && out_req_stride % E == 0));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return dtype == SV_F32 ? launch_adjust<float>(A, aligned, st)
                         : launch_adjust<__nv_bfloat16>(A, aligned, st);
}
