// sv_rotary.cu — the norm of every query and key head and its rotation by the row's position, in one
// pass.
//
// Mathematics: y = x / sqrt(mean x^2 + eps) * w, then (a, b) -> (a cos t - b sin t, a sin t + b cos t)
// with t = position * inv_freq. Weights, cosines and sines of a row are the same for all its heads, so
// a warp folds them into two factors per element, out = r * (x * c + partner * s), and keeps those
// over the heads it takes; r is the head's own 1 / sqrt.
//
// Angles. A position times a frequency has more digits than fp32 keeps: at position 131072 the product
// is off by 0.004 of a radian. Frequencies are held as 64-bit fractions of a turn instead, so that the
// product modulo one turn is an integer product modulo 2^64, off by 2^-65 of a turn per position; what
// is left is rounded to fp32 once (2^-25 of a half turn).
//
// Bound: reading and writing every row once. A head of D = 128 is 16 lanes of 16 bytes, a warp takes
// two at a time, and loads those it takes next before it works on the ones at hand.
#include <cstdint>

#include "specverify_step.h"
#include "sv_host.h"
#include "sv_kv.h"
#include "sv_kv_tiles.cuh"

namespace sv {
namespace {

#ifndef ROT_CTAS
#define ROT_CTAS 3
#endif
#ifndef ROT_AHEAD
#define ROT_AHEAD 4
#endif
constexpr int kRotThreads = 256, kRotWarps = kRotThreads / 32;

struct HeadRows {
  const uint16_t* in;
  uint16_t* out;
  int64_t req, row, head, out_req, out_row, out_head;
  int heads;
  const void* weight;
};
struct RotArgs {
  HeadRows x[2];  // queries, keys
  const int32_t* positions;
  const void* inv_freq;
  int64_t rows;
  int P, R, weight_f32, freq_f64, norm, interleaved;
  float eps;
};

template <bool kBf16>
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 p = unpack16<kBf16>(w[k]);
    f[2 * k] = p.x;
    f[2 * k + 1] = p.y;
  }
}

// (Not through the read-only path: outputs may be the inputs.)
__device__ __forceinline__ uint4 load16(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// kSplit warps share a row (one token's heads). Nothing is shared between warps but the frequencies
// and the weights, so no warp waits for another one's rows: with a table of cosines per CTA and
// barriers around it prompts of 24576 rows took 145 us.
template <int D, bool kBf16, int kSplit>
__global__ void __launch_bounds__(kRotThreads, ROT_CTAS) rotate_kernel(const __grid_constant__ RotArgs A) {
  constexpr int kLanes = D / 8, kPer = 32 / kLanes;  // lanes of a head, heads at a time
  constexpr int kAhead = ROT_AHEAD;                          // groups of heads in flight
  __shared__ uint64_t turn[D / 2];                   // frequencies in 2^-64 of a turn
  __shared__ float odd[D / 2];                       // NaN where one is not finite, else 0
  __shared__ float weight[2][D];
  __shared__ float2 table[kRotWarps][D / 2];  // cosines and sines of each warp's row
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int half = A.R / 2;
  for (int i = tid; i < half; i += kRotThreads) {
    const double f = A.freq_f64 ? static_cast<const double*>(A.inv_freq)[i]
                                : (double)static_cast<const float*>(A.inv_freq)[i];
    const double t = f * 0.15915494309189533577;  // 1 / (2 pi)
    turn[i] = __double2ull_rn((t - floor(t)) * 18446744073709551616.0);
    odd[i] = isfinite(f) ? 0.0f : __uint_as_float(0x7fc00000u);
  }
  for (int e = tid; e < 2 * D; e += kRotThreads) {
    const void* w = A.x[e / D].weight;
    weight[e / D][e % D] = !w            ? 1.0f
                           : A.weight_f32 ? static_cast<const float*>(w)[e % D]
                                          : unpack16<kBf16>(static_cast<const uint16_t*>(w)[e % D]).x;
  }
  __syncthreads();
  const int sub = warp % kSplit, d0 = lane % kLanes * 8;
  const int mate = A.interleaved ? 0 : d0 < half ? half : -half;
  const int from = A.interleaved || d0 >= A.R ? lane : lane + mate / 8;  // the partners' lane
  const bool turned = d0 < A.R;
  constexpr int64_t kRows = kRotWarps / kSplit;
#pragma unroll 1
  for (int64_t row = blockIdx.x * kRows + warp / kSplit; row < A.rows; row += gridDim.x * kRows) {
    const int p = __ldg(A.positions + row);
    if (p < 0) continue;
    const int64_t req = row / A.P, at = row - req * A.P;
    __syncwarp();  // the last row's table has been read
    for (int i = lane; i < half; i += 32) {
      // the signed fraction of a turn, in half turns
      const float t = (float)(int32_t)((turn[i] * (uint64_t)(int64_t)p) >> 32) * 4.656612873077393e-10f;
      float s, c;
      sincospif(t, &s, &c);
      table[warp][i] = make_float2(c + odd[i], s + odd[i]);
    }
    __syncwarp();
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
      const HeadRows& X = A.x[which];
      // what multiplies the element and its partner
      float c[8], s[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int d = d0 + e;
        float2 cs = make_float2(1.0f, 0.0f);
        int other = d;
        if (turned) {
          cs = table[warp][A.interleaved ? d >> 1 : d < half ? d : d - half];
          other = A.interleaved ? d ^ 1 : d + mate;
          if (A.interleaved ? !(d & 1) : d < half) cs.y = -cs.y;
        }
        c[e] = weight[which][d] * cs.x;
        s[e] = weight[which][other] * cs.y;
      }
      const uint16_t* in = X.in + req * X.req + at * X.row + d0;
      uint16_t* out = X.out + req * X.out_req + at * X.out_row + d0;
      constexpr int kStep = kSplit * kPer;
      const int first = sub * kPer + lane / kLanes;
#pragma unroll 1
      for (int h0 = 0; h0 < X.heads; h0 += kAhead * kStep) {
        uint4 raw[kAhead];
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
          const int h = h0 + first + a * kStep;
          raw[a] = make_uint4(0u, 0u, 0u, 0u);
          if (h < X.heads) raw[a] = load16(in + h * X.head);
        }
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
          const int h = h0 + first + a * kStep;
          if (h0 + a * kStep >= X.heads) break;  // (whole warps)
          float x[8], y[8];
          unpack8<kBf16>(raw[a], x);
          float r = 1.0f;
          if (A.norm) {
            float sum = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) sum = fmaf(x[e], x[e], sum);
#pragma unroll
            for (int o = kLanes / 2; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            r = rsqrtf(sum * (1.0f / D) + A.eps);
          }
          if (A.interleaved) {
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = x[e ^ 1];
          } else {
            uint4 v;
            v.x = __shfl_sync(0xffffffffu, raw[a].x, from);
            v.y = __shfl_sync(0xffffffffu, raw[a].y, from);
            v.z = __shfl_sync(0xffffffffu, raw[a].z, from);
            v.w = __shfl_sync(0xffffffffu, raw[a].w, from);
            unpack8<kBf16>(v, y);
          }
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int e = 2 * k;
            // (components past R have no partner: what lies there may be infinite)
            const float p0 = turned ? fmaf(y[e], s[e], x[e] * c[e]) : x[e] * c[e];
            const float p1 = turned ? fmaf(y[e + 1], s[e + 1], x[e + 1] * c[e + 1]) : x[e + 1] * c[e + 1];
            w[k] = pack16<kBf16>(r * p0, r * p1);
          }
          if (h < X.heads)
            *reinterpret_cast<uint4*>(out + h * X.out_head) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
  }
}

template <int D, bool kBf16>
sv_status launch_rotate(const RotArgs& A, cudaStream_t st) {
  // a CTA per row while there are few, so that a row's heads are loaded at once; a warp per row once
  // those fill the SMs
  const int64_t sms = device_sm_count();
  if (A.rows <= 8 * sms) {
    rotate_kernel<D, kBf16, 8><<<(unsigned)A.rows, kRotThreads, 0, st>>>(A);
  } else {
    const int64_t want = (A.rows + kRotWarps - 1) / kRotWarps, ctas = want < ROT_CTAS * sms ? want : ROT_CTAS * sms;
    rotate_kernel<D, kBf16, 1><<<(unsigned)ctas, kRotThreads, 0, st>>>(A);
  }
  return launch_status();
}

template <bool kBf16>
sv_status launch_rotate_width(int D, const RotArgs& A, cudaStream_t st) {
  switch (D) {
    case 64: return launch_rotate<64, kBf16>(A, st);
    case 128: return launch_rotate<128, kBf16>(A, st);
  }
  return launch_rotate<256, kBf16>(A, st);
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" sv_status qk_norm_rotate(sv_kv_dtype dtype, int B, int P, int D, int R,
                                    const sv_head_rows* q, const sv_head_rows* k, int weight_f32,
                                    const int32_t* positions, const void* inv_freq, int freq_f64,
                                    int norm, float eps, int interleaved, sv_stream_t stream) {
  if ((dtype != SV_KV_BF16 && dtype != SV_KV_F16) || B < 0 || P < 0 || D < 1 || R < 0 || !q || !k ||
      !(eps >= 0.0f) || q->heads < 0 || k->heads < 0)
    return SV_ERR_INVALID_ARG;
  if ((D != 64 && D != 128 && D != 256) || R > D || R % 16 != 0) return SV_ERR_UNSUPPORTED;
  if ((int64_t)B * P >= (1ll << 31)) return SV_ERR_UNSUPPORTED;
  if (B == 0 || P == 0) return SV_OK;
  RotArgs A{};
  int i = 0;
  for (const sv_head_rows* x : {q, k}) {
    if (x->heads > 0 && (!x->data || !x->out || !aligned_to(x->data, 16) || !aligned_to(x->out, 16) ||
                         !aligned_to(x->weight, weight_f32 ? 4 : 2)))
      return SV_ERR_INVALID_ARG;
    for (int64_t s : {x->req, x->row, x->head, x->out_req, x->out_row, x->out_head})
      if (x->heads > 0 && (s < 0 || s % 8 != 0 || s >= (1ll << 39))) return SV_ERR_INVALID_ARG;
    // rows of the output lie apart
    if (x->heads > 0 && ((B > 1 && x->out_req == 0) || (P > 1 && x->out_row == 0) ||
                         (x->heads > 1 && x->out_head == 0)))
      return SV_ERR_INVALID_ARG;
    A.x[i++] = {static_cast<const uint16_t*>(x->data), static_cast<uint16_t*>(x->out), x->req, x->row,
                x->head, x->out_req, x->out_row, x->out_head, x->heads, x->weight};
  }
  if (!positions || !aligned_to(positions, 4) ||
      (R > 0 && (!inv_freq || !aligned_to(inv_freq, freq_f64 ? 8 : 4))))
    return SV_ERR_INVALID_ARG;
  A.positions = positions;
  A.inv_freq = inv_freq;
  A.rows = (int64_t)B * P;
  A.P = P;
  A.R = R;
  A.weight_f32 = weight_f32;
  A.freq_f64 = freq_f64;
  A.norm = norm;
  A.interleaved = interleaved;
  A.eps = eps;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return dtype == SV_KV_BF16 ? launch_rotate_width<true>(D, A, st) : launch_rotate_width<false>(D, A, st);
}
