// sv_pages.cu — the pages and slots of a step's new positions, from the requests' lengths.
//
// Mathematics: three prefix sums over the requests (rows, pages taken, pages given back), then every
// row, every new table entry and every ring place is found by a search in them. Each CTA forms the
// sums itself in shared memory (12 bytes per request from L2), so one launch does it all and no CTA
// waits for another: what one reads (kept entries, the ring's front) none writes (new entries, the
// ring's end).
//
// Bound: latency for a step (three dependent loads and two scans); for packed prompts the 12 bytes of
// a row, written. There a thread takes eight rows, whose pages are looked up at once and which mostly
// share a search. Measured, in graph replays (bytes at 6801 GB/s first): a step of 512 requests of 9
// rows 0.02 us, 4.4 us; 1024 prompts of 16 .. 16384 tokens packed in 2.4 million rows 4.4 us, 15.5 us
// (16.5 with a search wherever a request ends).
#include <cstdint>

#include "specverify_step.h"
#include "sv_host.h"
#include "sv_kv.h"

namespace sv {

int device_sm_count();

namespace {

constexpr int kMapThreads = 512;
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

// Exclusive prefixes of kCount numbers over the block's threads, and their totals (two CTA barriers).
template <int kCount>
__device__ __forceinline__ void block_scan(int64_t (&x)[kCount], int64_t (*scratch)[kMapThreads / 32],
                                           int64_t (&total)[kCount]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t incl[kCount];
#pragma unroll
  for (int k = 0; k < kCount; ++k) incl[k] = x[k];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
    for (int k = 0; k < kCount; ++k) {
      const int64_t y = __shfl_up_sync(0xffffffffu, incl[k], o);
      if (lane >= o) incl[k] += y;
    }
  }
  constexpr int kWarps = kMapThreads / 32;
  if (lane == 31) {
#pragma unroll
    for (int k = 0; k < kCount; ++k) scratch[k][warp] = incl[k];
  }
  __syncthreads();
  // every warp sums the warps' totals
#pragma unroll
  for (int k = 0; k < kCount; ++k) {
    int64_t sum = lane < kWarps ? scratch[k][lane] : 0;
#pragma unroll
    for (int o = 1; o < kWarps; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    const int64_t before = __shfl_sync(0xffffffffu, sum, (warp + 31) & 31);
    total[k] = __shfl_sync(0xffffffffu, sum, kWarps - 1);
    x[k] = (warp == 0 ? 0 : before) + incl[k] - x[k];
  }
  __syncthreads();
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

// kRowsPer rows to a thread: one where rows are few, so that every load is on its way at once.
template <int kRowsPer>
__global__ void __launch_bounds__(kMapThreads, kRowsPer == 1 ? 2 : 3) map_kernel(const MapArgs A) {
  extern __shared__ int map_smem[];
  __shared__ int64_t scratch[2][kMapThreads / 32];
  int* first = map_smem;         // [B + 1] rows before each request (packed rows)
  int* taken = first + A.B + 1;  // [B + 1] growth before each request
  int* given = taken + A.B + 1;  // [B + 1] pages given back before each request
  int* have = given + A.B + 1;   // [B] pages held
  int* rows_of = have + A.B;     // [B] new rows, 0 where the request gets none
  int* begin = rows_of + A.B;    // [B] the first new row's position
  int* length = begin + A.B;     // [B] the length it comes out with
  const int tid = threadIdx.x;
  const int head = __ldg(A.state), count = __ldg(A.state + 1);
  const int each = (A.B + kMapThreads - 1) / kMapThreads;
  const int b0 = min(tid * each, A.B), b1 = min(b0 + each, A.B);

  int64_t total[1] = {0}, at[1] = {0};
  if (A.P == 0) {
    for (int b = b0; b < b1; ++b) at[0] += load_request(A, b).add;
    block_scan<1>(at, scratch, total);
  }
  auto lost = [&](const Request& r, int64_t row) {  // a data error of the request, its first row given
    return !r.valid || (A.P == 0 && row + r.add > A.rows);
  };
  int64_t moved[2] = {0, 0}, all[2], row = at[0];  // taken, given back
  for (int b = b0; b < b1; ++b) {
    const Request r = load_request(A, b);
    if (!lost(r, row)) {
      moved[0] += max(r.need - r.have, 0);
      moved[1] += max(r.have - r.need, 0);
    }
    row += r.add;
  }
  block_scan<2>(moved, scratch, all);
  const bool ring_ok = head >= 0 && head < A.ring_size && count >= 0 && count <= A.ring_size &&
                       all[1] <= (int64_t)A.ring_size - count;
  // requests find pages as long as the sum of the growth up to them is at most count (a sum that was
  // capped is more than any count)
  auto enough = [&](int sum) { return sum <= count && sum != INT32_MAX; };
  auto place = [&](unsigned x) { return x < (unsigned)A.ring_size ? x : x - A.ring_size; };
  row = at[0];
  for (int b = b0; b < b1; ++b) {
    const Request r = load_request(A, b);
    first[b] = A.P > 0 ? b * A.P : capped(row);
    taken[b] = capped(moved[0]);
    given[b] = capped(moved[1]);
    const bool bad = lost(r, row);
    if (!bad) {
      moved[0] += max(r.need - r.have, 0);
      moved[1] += max(r.have - r.need, 0);
    }
    row += r.add;
    const bool fits = r.need <= r.have || enough(capped(moved[0]));
    have[b] = r.have;
    begin[b] = r.n - r.add;
    rows_of[b] = ring_ok && !bad && fits ? r.add : 0;
    length[b] = !ring_ok || bad ? -1 : fits ? r.n : r.old_len;
  }
  if (tid == 0) {
    first[A.B] = A.P > 0 ? A.B * A.P : capped(total[0]);
    taken[A.B] = capped(all[0]);
    given[A.B] = capped(all[1]);
  }
  __syncthreads();
  // pages taken: the largest sum that fits
  int most = 0;
  if (ring_ok) {
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
  const int drops = ring_ok ? (int)all[1] : 0;

  // one range of work: groups of rows, new table entries, pages that go back, requests
  const int64_t groups = ((int64_t)A.rows + 32 * kRowsPer - 1) / (32 * kRowsPer) * 32;
  const int64_t work = groups + most + drops + A.B + 1;
#pragma unroll 1
  for (int64_t x = (int64_t)blockIdx.x * kMapThreads + tid; x < work;
       x += (int64_t)gridDim.x * kMapThreads) {
    if (x >= groups) {
      if (x - groups < most) {  // (this part is sums and counts of 31 bits, not their sum)
        const int y = (int)(x - groups), b = find(taken, A.B, y);
        A.table[(int64_t)b * A.max_pages + have[b] + (y - taken[b])] =
            __ldg(A.ring + place((unsigned)head + (unsigned)y));
        continue;
      }
      int64_t y = x - groups - most;
      if (y < drops) {
        // (its entries from the new length's page on)
        const int b = find(given, A.B, (int)y), left = have[b] - (given[b + 1] - given[b]);
        A.ring[place(place((unsigned)head + count) + (unsigned)y)] =
            __ldg(A.table + (int64_t)b * A.max_pages + left + (y - given[b]));
        continue;
      }
      y -= drops;
      A.out_first[y] = first[y];
      if (y < A.B) {
        A.out_len[y] = length[y];
      } else {
        A.out_state[0] = ring_ok ? (int)place((unsigned)head + most) : -1;
        A.out_state[1] = ring_ok ? count - most + drops : -1;
      }
      continue;
    }
    // (a warp's threads take its rows in turn: their stores lie side by side)
    const uint32_t row0 = (uint32_t)x / 32 * (32 * kRowsPer) + (x & 31), rows = A.rows;
    int pos[kRowsPer], page[kRowsPer];
    int b = -1, end = 0, start = 0;
#pragma unroll
    for (int k = 0; k < kRowsPer; ++k) {
      pos[k] = page[k] = -1;
      if (row0 + 32 * k >= rows) continue;
      const int row = (int)(row0 + 32 * k);
      if (b < 0 || row >= end) {
        if (A.P > 0) {
          b = row / A.P;
        } else {
          if (row >= first[A.B]) continue;
          // (past a request's last row it is mostly the next one's)
          b = b >= 0 && row < first[min(b + 2, A.B)] ? b + 1 : find(first, A.B, row);
        }
        start = first[b];
        end = first[b + 1];
      }
      const int i = row - start;
      if (i >= rows_of[b]) continue;
      pos[k] = begin[b] + i;
      const int t = pos[k] >> A.log_page, held = have[b];
      page[k] = __ldg(t < held ? A.table + (int64_t)b * A.max_pages + t
                               : A.ring + place((unsigned)head + taken[b] + (t - held)));
    }
#pragma unroll
    for (int k = 0; k < kRowsPer; ++k) {
      const uint32_t row = row0 + 32 * k;
      if (row >= rows) break;
      const bool there = page[k] >= 0 && page[k] < A.num_pages;
      A.slots[row] = there ? ((int64_t)page[k] << A.log_page) + (pos[k] & ((1 << A.log_page) - 1)) : -1;
      A.positions[row] = pos[k];
    }
  }
}

// Whether p is memory that CUDA knows. (Asked of an empty batch alone, whose caller may have no arrays.)
bool on_device(const void* p) {
  cudaPointerAttributes a{};
  const bool known = p && cudaPointerGetAttributes(&a, p) == cudaSuccess;
  if (!known) cudaGetLastError();
  return known && a.type != cudaMemoryTypeUnregistered;
}

bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  const char *p = static_cast<const char*>(a), *q = static_cast<const char*>(b);
  return na > 0 && nb > 0 && p < q + nb && q < p + na;
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
  // an empty batch has a ring's state to hand on and rows to mark all the same
  if (B == 0 && !on_device(out_state)) return SV_OK;
  if ((B > 0 && (!page_table || !old_len || !seq_len || !num_new || !ring || !out_len)) || !ring_state ||
      !out_first || !out_state || (rows > 0 && (!out_slots || !out_positions)) ||
      !aligned_to(out_slots, 8))
    return SV_ERR_INVALID_ARG;
  for (const void* p : {(const void*)page_table, (const void*)old_len, (const void*)seq_len,
                        (const void*)num_new, (const void*)ring, (const void*)ring_state,
                        (const void*)out_positions, (const void*)out_len, (const void*)out_first,
                        (const void*)out_state})
    if (!aligned_to(p, 4)) return SV_ERR_INVALID_ARG;
  // what is only read may be one array; nothing that is written may share bytes with another
  const int64_t n = 4 * (int64_t)B, r = 4 * (int64_t)rows;
  const struct { const void* p; int64_t bytes; } all[] = {
      {old_len, n},        {seq_len, n},           {num_new, n},       {ring_state, 8},
      {page_table, n * max_pages}, {ring, 4 * (int64_t)ring_size}, {out_slots, 2 * r},
      {out_positions, r},  {out_len, n},           {out_first, n + 4}, {out_state, 8}};
  for (int i = 4; i < 11; ++i)
    for (int j = 0; j < i; ++j)
      if (overlap(all[i].p, all[i].bytes, all[j].p, all[j].bytes)) return SV_ERR_INVALID_ARG;
  const MapArgs A{B,      log2_of(page_size), num_pages,  max_pages,     ring_size, P,         rows,
                  page_table, old_len,        seq_len,    num_new,       ring,      ring_state,
                  out_slots,  out_positions,  out_len,    out_first,     out_state};
  // a thread per row up to two CTAs per SM of them, then eight rows to a thread
  const int64_t sms = device_sm_count(), few = 2 * sms * kMapThreads;
  const int per = rows <= few ? 1 : 8;
  auto kernel = per == 1 ? map_kernel<1> : map_kernel<8>;
  const size_t smem = 7 * (size_t)(B + 1) * sizeof(int);
  if (smem > 47 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               7 * (kMaxRequests + 1) * (int)sizeof(int));
    if (e != cudaSuccess) return cuda_fail(e);
  }
  int64_t ctas = (rows / per + 2ll * B + kMapThreads - 1) / kMapThreads;
  const int64_t most = 2 * sms;
  ctas = ctas > most ? most : ctas < 1 ? 1 : ctas;
  kernel<<<(unsigned)ctas, kMapThreads, smem, reinterpret_cast<cudaStream_t>(stream)>>>(A);
  return launch_status();
}
