// sv_pages.cu — the pages and slots of a step's new positions, from the requests' lengths.
//
// Mathematics: three prefix sums over the requests (rows, pages taken, pages given back), then every
// row, every new table entry and every ring place is found by a search in them. Each CTA forms the
// sums itself in shared memory (12 bytes per request from L2), so one launch does it all and no CTA
// waits for another: what one reads (kept entries, the ring's front) none writes (new entries, the
// ring's end).
//
// Bound: latency for a step (three dependent loads and two scans); for packed prompts the 12 bytes of
// a row. A thread takes four rows, which share a search and leave in 16-byte stores.
#include <cstdint>

#include "specverify_step.h"
#include "sv_host.h"
#include "sv_kv.h"

namespace sv {

int device_sm_count();

namespace {

constexpr int kMapThreads = 512;
constexpr int kRowsPer = 4;
constexpr int kMaxRequests = 8192;

struct MapArgs {
  int B, log_page, num_pages, max_pages, ring_size, P, rows;
  int32_t* table;
  const int32_t *old_len, *seq_len, *num_new;
  int32_t* ring;
  const int32_t* state;
  int64_t* slots;
  int32_t *positions, *out_len, *out_first, *out_state;
};

// Exclusive prefix of x over the block's threads, and the total (two CTA barriers).
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t* scratch, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) scratch[warp] = incl;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kMapThreads / 32; ++w) {
    const int64_t s = scratch[w];
    if (w < warp) before += s;
    all += s;
  }
  __syncthreads();
  *total = all;
  return before + incl - x;
}

__device__ __forceinline__ int capped(int64_t x) { return x < INT32_MAX ? (int)x : INT32_MAX; }

// The last of the n + 1 ascending values at[] that is at most x, below n.
__device__ __forceinline__ int find(const int* at, int n, int x) {
  int lo = 0, hi = n;  // at[lo] <= x < at[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (at[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

struct Request {
  int old_len, n, add, have, need;
  bool valid;  // its lengths (not whether its rows fit)
};
__device__ __forceinline__ Request load_request(const MapArgs& A, int b) {
  Request r;
  r.old_len = __ldg(A.old_len + b);
  r.n = __ldg(A.seq_len + b);
  r.add = __ldg(A.num_new + b);
  const int most = A.max_pages << A.log_page, up = (1 << A.log_page) - 1;
  r.valid = r.old_len >= 0 && r.old_len <= most && r.n >= 0 && r.n <= most && r.add >= 0 &&
            r.add <= r.n && (A.P == 0 || r.add <= A.P);
  r.have = r.valid ? (r.old_len + up) >> A.log_page : 0;
  r.need = r.valid ? (r.n + up) >> A.log_page : 0;
  if (!r.valid) r.add = 0;
  return r;
}

__global__ void __launch_bounds__(kMapThreads) map_kernel(const MapArgs A) {
  extern __shared__ int map_smem[];
  __shared__ int64_t scratch[kMapThreads / 32];
  int* first = map_smem;            // [B + 1] rows before each request (packed rows)
  int* taken = first + A.B + 1;     // [B + 1] growth before each request
  int* given = taken + A.B + 1;     // [B + 1] pages given back before each request
  const int tid = threadIdx.x;
  const int head = __ldg(A.state), count = __ldg(A.state + 1);
  const int each = (A.B + kMapThreads - 1) / kMapThreads;
  const int b0 = min(tid * each, A.B), b1 = min(b0 + each, A.B);

  int64_t rows = 0, total;
  for (int b = b0; b < b1; ++b) rows += load_request(A, b).add;
  int64_t at = block_scan(rows, scratch, &total);
  if (tid == 0) first[A.B] = capped(total);
  int64_t grow = 0, drop = 0;
  for (int b = b0; b < b1; ++b) {
    const Request r = load_request(A, b);
    first[b] = capped(at);
    at += r.add;
    if (A.P == 0 && at > A.rows) continue;  // its rows do not fit
    grow += max(r.need - r.have, 0);
    drop += max(r.have - r.need, 0);
  }
  int64_t all_grow, all_drop;
  int64_t g = block_scan(grow, scratch, &all_grow), d = block_scan(drop, scratch, &all_drop);
  if (tid == 0) {
    taken[A.B] = capped(all_grow);
    given[A.B] = capped(all_drop);
  }
  for (int b = b0; b < b1; ++b) {
    const Request r = load_request(A, b);
    taken[b] = capped(g);
    given[b] = capped(d);
    if (A.P == 0 && (int64_t)first[b] + r.add > A.rows) continue;
    g += max(r.need - r.have, 0);
    d += max(r.have - r.need, 0);
  }
  __syncthreads();

  const bool ring_ok = head >= 0 && head < A.ring_size && count >= 0 && count <= A.ring_size &&
                       all_drop <= (int64_t)A.ring_size - count;
  // requests find pages as long as the sum of the growth up to them is at most count
  // (a sum that was capped is more than any count)
  auto enough = [&](int sum) { return sum <= count && sum != INT32_MAX; };
  auto fits = [&](const Request& r, int b) { return r.need <= r.have || enough(taken[b + 1]); };
  auto lost = [&](const Request& r, int b) {  // a data error of the request
    return !r.valid || (A.P == 0 && (int64_t)first[b] + r.add > A.rows);
  };
  auto place = [&](unsigned x) { return x < (unsigned)A.ring_size ? x : x - A.ring_size; };
  int most = 0;  // pages taken: the largest sum that fits
  {
    int lo = 0, hi = A.B + 1;  // taken[lo] is enough, taken[hi] not
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (enough(taken[mid]))
        lo = mid;
      else
        hi = mid;
    }
    most = taken[lo];
  }
  const int stride = gridDim.x * kMapThreads, me = blockIdx.x * kMapThreads + tid;

  // rows
  for (int64_t row0 = (int64_t)me * kRowsPer; row0 < A.rows; row0 += (int64_t)stride * kRowsPer) {
    int64_t slot[kRowsPer];
    int pos[kRowsPer];
    int b = -1, end = 0, start = 0;
    Request r{};
    bool live = false;
#pragma unroll
    for (int k = 0; k < kRowsPer; ++k) {
      const int64_t row = row0 + k;
      slot[k] = pos[k] = -1;
      if (row >= A.rows || !ring_ok) continue;
      if (b < 0 || row >= end) {
        if (A.P > 0) {
          b = (int)(row / A.P);
          start = b * A.P;
          end = start + A.P;
        } else {
          if (row >= first[A.B]) continue;
          b = find(first, A.B, (int)row);
          start = first[b];
          end = first[b + 1];
        }
        r = load_request(A, b);
        live = !lost(r, b) && fits(r, b);
      }
      const int i = (int)row - start;
      if (!live || i >= r.add) continue;
      const int p = r.n - r.add + i, t = p >> A.log_page;
      const int page = t < r.have
                           ? __ldg(A.table + (int64_t)b * A.max_pages + t)
                           : __ldg(A.ring + place((unsigned)head + taken[b] + (t - r.have)));
      pos[k] = p;
      if (page >= 0 && page < A.num_pages)
        slot[k] = ((int64_t)page << A.log_page) + (p & ((1 << A.log_page) - 1));
    }
    if (row0 + kRowsPer <= A.rows && ((uintptr_t)A.slots & 15) == 0 &&
        ((uintptr_t)A.positions & 15) == 0) {
      longlong2* s = reinterpret_cast<longlong2*>(A.slots + row0);
      s[0] = make_longlong2(slot[0], slot[1]);
      s[1] = make_longlong2(slot[2], slot[3]);
      *reinterpret_cast<int4*>(A.positions + row0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
#pragma unroll
      for (int k = 0; k < kRowsPer; ++k)
        if (row0 + k < A.rows) {
          A.slots[row0 + k] = slot[k];
          A.positions[row0 + k] = pos[k];
        }
    }
  }
  if (ring_ok) {
    // table entries of new pages
    for (int x = me; x < most; x += stride) {
      const int b = find(taken, A.B, x);
      A.table[(int64_t)b * A.max_pages + load_request(A, b).have + (x - taken[b])] =
          __ldg(A.ring + place((unsigned)head + x));
    }
    // pages that go back
    for (int x = me; x < (int)all_drop; x += stride) {
      const int b = find(given, A.B, x);
      A.ring[place(place((unsigned)head + count) + (unsigned)x)] =
          __ldg(A.table + (int64_t)b * A.max_pages + load_request(A, b).need + (x - given[b]));
    }
  }
  for (int b = me; b < A.B; b += stride) {
    const Request r = load_request(A, b);
    A.out_len[b] = !ring_ok || lost(r, b) ? -1 : fits(r, b) ? r.n : r.old_len;
  }
  for (int b = me; b <= A.B; b += stride) A.out_first[b] = A.P > 0 ? b * A.P : first[b];
  if (me == 0) {
    A.out_state[0] = ring_ok ? (int)place((unsigned)head + most) : -1;
    A.out_state[1] = ring_ok ? count - most + (int)all_drop : -1;
  }
}

bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  const char *p = static_cast<const char*>(a), *q = static_cast<const char*>(b);
  return p < q + nb && q < p + na;
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" sv_status kv_page_map(int B, int page_size, int num_pages, int32_t* page_table,
                                 int max_pages, const int32_t* old_len, const int32_t* seq_len,
                                 const int32_t* num_new, int32_t* ring, int ring_size,
                                 const int32_t* ring_state, int P, int rows, int64_t* out_slots,
                                 int32_t* out_positions, int32_t* out_len, int32_t* out_first,
                                 int32_t* out_state, sv_stream_t stream) {
  if (B < 0 || page_size < 1 || num_pages < 0 || max_pages < 1 || ring_size < 1 || P < 0 || rows < 0)
    return SV_ERR_INVALID_ARG;
  if (page_size < 8 || page_size > kMaxPageSize || (page_size & (page_size - 1)) != 0 ||
      (int64_t)max_pages * page_size >= (1ll << 30) || B > kMaxRequests)
    return SV_ERR_UNSUPPORTED;
  if (P > 0 && (int64_t)B * P != rows) return SV_ERR_INVALID_ARG;
  if (B == 0) return SV_OK;
  if (!page_table || !old_len || !seq_len || !num_new || !ring || !ring_state || !out_len ||
      !out_first || !out_state || (rows > 0 && (!out_slots || !out_positions)) ||
      !aligned_to(out_slots, 8))
    return SV_ERR_INVALID_ARG;
  for (const void* p : {(const void*)page_table, (const void*)old_len, (const void*)seq_len,
                        (const void*)num_new, (const void*)ring, (const void*)ring_state,
                        (const void*)out_positions, (const void*)out_len, (const void*)out_first,
                        (const void*)out_state})
    if (!aligned_to(p, 4)) return SV_ERR_INVALID_ARG;
  const int64_t n = 4 * (int64_t)B;
  for (const int32_t* in : {old_len, seq_len, num_new})
    if (overlap(in, n, out_len, n) || overlap(in, n, out_first, n + 4) || overlap(in, n, out_state, 8))
      return SV_ERR_INVALID_ARG;
  if (overlap(ring_state, 8, out_len, n) || overlap(ring_state, 8, out_first, n + 4) ||
      overlap(ring_state, 8, out_state, 8))
    return SV_ERR_INVALID_ARG;
  const MapArgs A{B,      log2_of(page_size), num_pages,  max_pages,     ring_size, P,         rows,
                  page_table, old_len,        seq_len,    num_new,       ring,      ring_state,
                  out_slots,  out_positions,  out_len,    out_first,     out_state};
  const size_t smem = 3 * (size_t)(B + 1) * sizeof(int);
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(
        map_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 3 * (kMaxRequests + 1) * sizeof(int));
    if (e != cudaSuccess) return cuda_fail(e);
  }
  // a CTA per 2048 rows and per 512 requests, at most two per SM
  const int64_t wanted = (rows + kMapThreads * kRowsPer - 1ll) / (kMapThreads * kRowsPer);
  const int64_t other = (B + kMapThreads - 1) / kMapThreads;
  int64_t ctas = wanted > other ? wanted : other;
  if (ctas > 2 * device_sm_count()) ctas = 2 * device_sm_count();
  map_kernel<<<(unsigned)ctas, kMapThreads, smem, reinterpret_cast<cudaStream_t>(stream)>>>(A);
  return launch_status();
}
