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
// product modulo one turn is an integer product modulo 2^64, off by what the fraction is: f / 2 pi is a
// product of doubles, so 2^-52 of it per position (at f = 1 2^-37 of a turn at position 131072); what is
// left is rounded to fp32 once (2^-25 of a half turn).
//
// Bound: reading and writing every row once. A head of D = 128 is 16 lanes of 16 bytes; a warp takes
// two at a time and has eight of them loaded while the eight before them are turned. Measured, in graph
// replays (bytes at 6801 GB/s first): one row of 40 heads of 128 0.003 us, 4.4 us; 384 rows of 72 heads
// 1.9 us, 6.1 us; 24576 rows of 40 heads 74.0 us, 83.8 us, 88 % of a copy's bandwidth.
#include <cstdint>

#include "specverify_step.h"
#include "sv_host.h"
#include "sv_kv.h"
#include "sv_kv_tiles.cuh"

namespace sv {
namespace {

// Three CTAs per SM: registers for the next heads' loads (four CTAs spill, 101 us, two 88; four without
// those loads 86.5).
constexpr int kRotThreads = 256, kRotWarps = kRotThreads / 32, kRotCtas = 3;

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

// (Not through the read-only path: outputs may be the inputs.)
__device__ __forceinline__ uint2 load8(const void* p) {
  uint2 v;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];"
               : "=r"(v.x), "=r"(v.y)
               : "l"(p)
               : "memory");
  return v;
}

// Squares of bf16 numbers pass the range of fp32 (fp16's do not): above where one is 2^60 or more, and
// below they lose bits to subnormal numbers or vanish. Heads whose mean square with eps is outside
// [2^-96, 2^128) are scaled by a power of two, which bf16 numbers take without loss: those with all
// components below 2^-44 (2^-48 times the root of 256) by 2^100, and those with one of 2^60 or more by
// 2^-70, which brings the largest below 2^58 and its square below 2^116 (and what lies below 2^-79, and
// becomes subnormal, comes out below 2^-133, the smallest bf16 number). Zeros, infinities and NaN come out
// as the formula has them. (Four flags and one rolled loop at the end of four heads: 83.5 us for prompts
// of 24576 rows beside 83.0 without; the scaling unrolled beside each head's sum 84.8, in a function 86.1.)
constexpr float kSmallMean = 1.262177448e-29f, kLargeMean = 3.402823466e38f;  // 2^-96, the largest number
constexpr float kRaise = 1.267650600e30f, kLower = 8.470329473e-22f;          // 2^100, 2^-70

// kSplit warps share a row (one token's heads). Nothing is shared between warps but the frequencies
// and the weights, so no warp waits for another one's rows: with a table of cosines per CTA and
// barriers around it prompts of 24576 rows took 145 us.
// A lane holds eight components of a head: four pairs (a, b). Of halves those are four of the first
// and four of the second, in two loads of 8 bytes, so that no component has to come from another
// lane (with 16 consecutive bytes per lane and shuffles, 157 instructions a step, 107 us).
template <int D, bool kBf16, bool kInterleaved, int kSplit>
__global__ void __launch_bounds__(kRotThreads, kRotCtas) rotate_kernel(const __grid_constant__ RotArgs A) {
  constexpr int kLanes = D / 8, kPer = 32 / kLanes;  // lanes of a head, heads at a time
  constexpr int kAhead = 4;                          // groups of heads in flight
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
  const int place = lane % kLanes, sub = warp % kSplit;
  // where the lane's two groups of four components start, and those of its k-th pair
  const bool turned = place * 8 < A.R;
  const int da = kInterleaved || !turned ? place * 8 : place * 4;
  const int db = kInterleaved || !turned ? place * 8 + 4 : half + place * 4;
  auto component = [&](int k, int which) {  // of the pair's first or second
    return kInterleaved ? da + 2 * k + which : which ? db + k : da + k;
  };
  constexpr int64_t kRows = kRotWarps / kSplit;
  static_assert(kRows >= 1 && kRotWarps % kSplit == 0, "whole rows to a CTA");
  constexpr int kStep = kSplit * kPer;
  const int first = sub * kPer + lane / kLanes;
#pragma unroll 1
  for (int64_t row = blockIdx.x * kRows + warp / kSplit; row < A.rows; row += gridDim.x * kRows) {
    const int p = __ldg(A.positions + row);
    if (p < 0) continue;
    const int64_t req = row / A.P, at = row - req * A.P;
    // the lane's share of kAhead groups of heads; the next ones are loaded while these are turned
    uint2 na[kAhead], nb[kAhead];
    auto fetch = [&](int which, int h0) {
      const HeadRows& X = A.x[which];
      const uint16_t* from = X.in + req * X.req + at * X.row + (int64_t)(h0 + first) * X.head;
#pragma unroll
      for (int g = 0; g < kAhead; ++g, from += kStep * X.head) {
        na[g] = nb[g] = make_uint2(0u, 0u);
        if (h0 + first + g * kStep < X.heads) {
          na[g] = load8(from + da);
          nb[g] = load8(from + db);
        }
      }
    };
    fetch(A.x[0].heads > 0 ? 0 : 1, 0);
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
      // out a = a * aa + b * ab, out b = a * ba + b * bb (times the head's own factor)
      Two aa[2], ab[2], ba[2], bb[2];
#pragma unroll
      for (int k = 0; k < 4; k += 2) {
        float f[2][4];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const float wa = weight[which][component(k + q, 0)], wb = weight[which][component(k + q, 1)];
          const float2 cs = turned ? table[warp][place * 4 + k + q] : make_float2(1.0f, 0.0f);
          f[q][0] = wa * cs.x;
          f[q][1] = -wb * cs.y;
          f[q][2] = wa * cs.y;
          f[q][3] = wb * cs.x;
        }
        aa[k / 2] = two(f[0][0], f[1][0]);
        ab[k / 2] = two(f[0][1], f[1][1]);
        ba[k / 2] = two(f[0][2], f[1][2]);
        bb[k / 2] = two(f[0][3], f[1][3]);
      }
      uint16_t* out = X.out + req * X.out_req + at * X.out_row;
#pragma unroll 1
      for (int h0 = 0; h0 < X.heads; h0 += kAhead * kStep) {
        uint16_t* to = out + (int64_t)(h0 + first) * X.out_head;
        uint2 va[kAhead], vb[kAhead];
#pragma unroll
        for (int g = 0; g < kAhead; ++g) va[g] = na[g], vb[g] = nb[g];
        if (h0 + kAhead * kStep < X.heads)
          fetch(which, h0 + kAhead * kStep);
        else if (which == 0 && A.x[1].heads > 0)
          fetch(1, 0);
        // (the lane's share of a head, as pairs; the head's mean square with eps; and what it becomes)
        auto pairs = [&](const uint2& va, const uint2& vb, Two (&a)[2], Two (&b)[2]) {
          const uint32_t w[4] = {va.x, va.y, vb.x, vb.y};
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float2 u = unpack16<kBf16>(w[kInterleaved ? 2 * k : k]);
            const float2 v = unpack16<kBf16>(w[kInterleaved ? 2 * k + 1 : k + 2]);
            a[k] = kInterleaved ? two(u.x, v.x) : two(u.x, u.y);
            b[k] = kInterleaved ? two(u.y, v.y) : two(v.x, v.y);
          }
        };
        auto mean_of = [&](const Two (&a)[2], const Two (&b)[2], float eps, uint32_t lanes) {
          const float2 q = split(two_fma(a[0], a[0], two_fma(a[1], a[1], two_fma(b[0], b[0], two_mul(b[1], b[1])))));
          float sum = q.x + q.y;
#pragma unroll
          for (int o = kLanes / 2; o >= 1; o >>= 1) sum += __shfl_xor_sync(lanes, sum, o);
          return sum * (1.0f / D) + eps;
        };
        auto give = [&](const Two (&a)[2], const Two (&b)[2], float r, bool there, uint16_t* to) {
          const Two rr = two(r, r);
          float2 x[2], y[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            // (components past R have no partner: what lies there may be infinite)
            Two u = two_mul(a[k], aa[k]), v = two_mul(b[k], bb[k]);
            if (turned) {
              u = two_fma(b[k], ab[k], u);
              v = two_fma(a[k], ba[k], v);
            }
            x[k] = split(two_mul(u, rr));
            y[k] = split(two_mul(v, rr));
          }
          if (there) {
            if (kInterleaved) {
              *reinterpret_cast<uint2*>(to + da) =
                  make_uint2(pack16<kBf16>(x[0].x, y[0].x), pack16<kBf16>(x[0].y, y[0].y));
              *reinterpret_cast<uint2*>(to + db) =
                  make_uint2(pack16<kBf16>(x[1].x, y[1].x), pack16<kBf16>(x[1].y, y[1].y));
            } else {
              *reinterpret_cast<uint2*>(to + da) =
                  make_uint2(pack16<kBf16>(x[0].x, x[0].y), pack16<kBf16>(x[1].x, x[1].y));
              *reinterpret_cast<uint2*>(to + db) =
                  make_uint2(pack16<kBf16>(y[0].x, y[0].y), pack16<kBf16>(y[1].x, y[1].y));
            }
          }
        };
        bool held[kAhead];  // in range
#pragma unroll
        for (int g = 0; g < kAhead; ++g) held[g] = true;
#pragma unroll
        for (int g = 0; g < kAhead; ++g, to += kStep * X.out_head) {
          if (h0 + g * kStep >= X.heads) break;  // (whole warps)
          Two a[2], b[2];
          pairs(va[g], vb[g], a, b);
          float r = 1.0f;
          if (A.norm) {
            const float mean = mean_of(a, b, A.eps, 0xffffffffu);
            r = rsqrtf(mean);
            if (kBf16) held[g] = mean >= kSmallMean && mean <= kLargeMean;
          }
          give(a, b, r, h0 + first + g * kStep < X.heads && held[g], to);
        }
        // heads out of range once more, scaled (they have not been written, should that be in place)
        if (kBf16 && __builtin_expect(!(held[0] && held[1] && held[2] && held[3]), 0)) {
          static_assert(kAhead == 4, "heads at a time");
          uint32_t again = 0;
#pragma unroll
          for (int g = 0; g < kAhead; ++g) again |= held[g] ? 0u : 1u << g;
          const uint32_t lanes = kLanes == 32 ? 0xffffffffu : ((1u << kLanes % 32) - 1) << lane / kLanes * kLanes;
#pragma unroll 1
          for (int64_t h = h0 + first; again && h < X.heads; h += kStep, again >>= 1) {
            if (!(again & 1u)) continue;
            const uint16_t* x = X.in + req * X.req + at * X.row + h * X.head;
            Two a[2], b[2];
            pairs(load8(x + da), load8(x + db), a, b);
            const float scale = mean_of(a, b, A.eps, lanes) < kSmallMean ? kRaise : kLower;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              a[k] = two_mul(a[k], two(scale, scale));
              b[k] = two_mul(b[k], two(scale, scale));
            }
            give(a, b, rsqrtf(mean_of(a, b, A.eps * scale * scale, lanes)), true, out + h * X.out_head);
          }
        }
      }
    }
  }
}

template <int D, bool kBf16, bool kInterleaved>
sv_status launch_rotate(const RotArgs& A, cudaStream_t st) {
  // a CTA per row while there are few, so that a row's heads are loaded at once; a warp per row once
  // those fill the SMs
  const int64_t sms = device_sm_count();
  if (A.rows <= 8 * sms) {
    rotate_kernel<D, kBf16, kInterleaved, 8><<<(unsigned)A.rows, kRotThreads, 0, st>>>(A);
  } else {
    const int64_t want = (A.rows + kRotWarps - 1) / kRotWarps, most = kRotCtas * sms;
    rotate_kernel<D, kBf16, kInterleaved, 1>
        <<<(unsigned)(want < most ? want : most), kRotThreads, 0, st>>>(A);
  }
  return launch_status();
}

template <int D, bool kBf16>
sv_status launch_rotate_kind(const RotArgs& A, cudaStream_t st) {
  return A.interleaved ? launch_rotate<D, kBf16, true>(A, st) : launch_rotate<D, kBf16, false>(A, st);
}

template <bool kBf16>
sv_status launch_rotate_width(int D, const RotArgs& A, cudaStream_t st) {
  switch (D) {
    case 64: return launch_rotate_kind<64, kBf16>(A, st);
    case 128: return launch_rotate_kind<128, kBf16>(A, st);
  }
  return launch_rotate_kind<256, kBf16>(A, st);
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
    // heads of the output lie apart, as far as each stride by itself tells
    if (x->heads > 0 && ((B > 1 && x->out_req < D) || (P > 1 && x->out_row < D) ||
                         (x->heads > 1 && x->out_head < D)))
      return SV_ERR_INVALID_ARG;
    // in place, each head goes where it came from
    if (x->heads > 0 && x->out == x->data &&
        ((B > 1 && x->out_req != x->req) || (P > 1 && x->out_row != x->row) ||
         (x->heads > 1 && x->out_head != x->head)))
      return SV_ERR_INVALID_ARG;
    A.x[i++] = {static_cast<const uint16_t*>(x->data), static_cast<uint16_t*>(x->out), x->req, x->row,
                x->head, x->out_req, x->out_row, x->out_head, x->heads, x->weight};
  }
  // no output starts where the other's rows do
  if (q->heads > 0 && k->heads > 0 && (q->out == k->out || q->out == k->data || k->out == q->data))
    return SV_ERR_INVALID_ARG;
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
