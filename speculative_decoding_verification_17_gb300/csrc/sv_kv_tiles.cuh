// sv_kv_tiles.cuh — the tensor-core kernel behind paged_attention and attention_weight_sum.
//
// Mathematics. With the N query rows of one request and kv head as columns (its G query heads
// times its positions), a tile of 128 keys gives
//   S^T [128 keys, N] = K [128, D] * Q^T [D, N]        one matrix instruction per 16 of D
//   P^T = 2^(S^T * scale * log2(e) - m)                a thread per key, N columns in registers
//   O^T [D, N] += V^T [D, 128] * P^T [128, N]          accumulated in tensor memory
// The keys are the 128 rows of the instruction and the query rows its columns: a step reads a
// few query rows against very many keys, so no row of the tensor core idles when N is 16, and
// the softmax of a tile is spread over 128 threads instead of the few that own a query row.
//
// Bound: reading K and V once. 64 KiB per tile of D = 128 at this card's bandwidth is 2800
// clocks of one SM; the instructions of a tile take 256 + 512 clocks (the operand read from
// shared memory bounds a narrow instruction), the softmax about 1000.
//
// Running maximum. m[c] only moves when a score passes it by 2^8: the products of a tile are
// at most 2^8, far inside fp32 and the 16-bit types, and the accumulators are rescaled only in
// the first tiles of a row instead of in every tile.
//
// Rounding. The weights P are given to the tensor core as two 16-bit numbers, p = hi + lo, and
// V^T is multiplied by both: 16 bits of the weight instead of 8 (bf16), so the output carries
// no error but its own rounding. The second product costs tensor time that the memory hides.
//
// Work. All tiles of all (request, kv head, row block) items are one flat range, cut evenly
// over one CTA per SM: ragged lengths balance by construction. A CTA walks its range piece by
// piece (a piece = its part of one item). A piece that is a whole item is written out; others
// leave (O, m, l) in the workspace, and the CTA whose arrival completes an item joins its
// pieces in order, so the result does not depend on the order of arrival. No CTA waits for
// another one.
//
// Roles. One warp looks up pages and starts the tiled copies (a ring of 16 KiB units, 64
// columns of 128 keys each, in the order K0 K1 V0 K2 V1 ...), one thread issues the matrix
// instructions in the same order, 4 or 8 warps do the softmax and the outputs. S is double
// buffered: the scores of tile t+1 are computed while tile t is in the softmax.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sv_device.cuh"
#include "sv_host.h"
#include "sv_kv.h"
#include "sv_tcgen05.cuh"

namespace sv {

constexpr int kTileKeys = 128;
constexpr int kUnitBytes = kTileKeys * 128;  // 64 columns of a tile
constexpr int kUnitSmemMax = 232448 - 8192;  // dynamic shared memory for operands
constexpr float kNoMax = -3.402823466e38f;   // a maximum below every finite score
constexpr float kLog2e = 1.4426950408889634f;

struct TileArgs {
  const int32_t *table, *seq_len, *num_draft, *accept_len;
  int B, P, Hq, Hkv, G, log_page, num_pages, max_pages;
  int pos_block, blocks;  // positions per row block, row blocks per request
  int box;                // slots per copy
  int bf16;
  ScoreRule rule;
  // attention
  void* out;
  float *out_lse, *part;
  unsigned int* counters;
  // key weights
  const float *lse, *prior;
  float* weights;
  int64_t stride, lse_req, lse_row, lse_head;
};

template <int kD, int kN, bool kWeigh>
struct TileShape {
  static constexpr int D = kD, N = kN;
  static constexpr bool Weigh = kWeigh;
  static constexpr int U = D / 64;  // units of a key or value tile
  // softmax warps: groups of four (one per quarter of the tile's keys). In the attention two
  // groups share the columns of a wide tile; in the key weights each takes every other tile.
  static constexpr int Groups = kWeigh ? 2 : (N >= 64 ? 2 : 1);
  static constexpr int SoftWarps = 4 * Groups;
  static constexpr int SoftThreads = 32 * SoftWarps;
  static constexpr int Threads = SoftThreads + 64;
  static constexpr int NC = kWeigh ? N : N / Groups;  // columns per softmax thread
  static constexpr int QBytes = N * D * 2;
  static constexpr int NQ = N * D <= 64 * 128 ? 2 : 1;  // query buffers
  static constexpr int PBytes = kWeigh ? 0 : 2 * kTileKeys * N * 2;
  static constexpr int Room = (kUnitSmemMax - 1024 - NQ * QBytes - PBytes) / kUnitBytes;
  static constexpr int NU = (Room > 12 ? 12 : Room) / 2 * 2;  // ring units, an even number
  static constexpr int Smem = 1024 + NQ * QBytes + PBytes + NU * kUnitBytes;
  static constexpr int MBlocks = kWeigh ? 0 : (D + 127) / 128;  // accumulators of 128 of D
  static constexpr int TmemNeed = (2 + MBlocks) * N;
  static constexpr int TmemCols = TmemNeed <= 32 ? 32 : TmemNeed <= 64 ? 64 : TmemNeed <= 128 ? 128
                                  : TmemNeed <= 256 ? 256 : 512;
  // the last value tile lies one (unused) key tile past the last key tile: its place must not
  // have been that key tile's
  static_assert(kWeigh || NU >= 2 * U, "ring");
  static_assert(TmemNeed <= 512 && NU >= U && Smem <= kUnitSmemMax, "tile shape");
};

// ---- the work list ----------------------------------------------------------------------------
// One (request, row block): which rows it has, the keys they see and the tiles of those.
struct Item {
  int n, nd, acc;
  bool bad;
  int i0, live;     // live positions [i0, i0 + live)
  int pos0;         // cache position of row i0
  int first, last;  // the keys any live row sees; last < first: none
  int t0, tiles;    // tiles to walk (0: nothing to write)
};

template <bool kWeigh>
__device__ __forceinline__ Item item_of(const TileArgs& A, int n, int nd, int acc, int rb) {
  Item it;
  it.n = n;
  it.nd = nd;
  it.acc = acc;
  it.bad = n < 0 || n > (A.max_pages << A.log_page) || nd < 0 || nd >= A.P ||
           (kWeigh && (n > A.stride || acc < -1 || acc > nd));
  it.i0 = rb * A.pos_block;
  const int rows = it.bad ? A.P : kWeigh ? acc + 1 : nd + 1;
  it.live = rows - it.i0 < A.pos_block ? rows - it.i0 : A.pos_block;
  it.pos0 = it.first = it.last = it.t0 = it.tiles = 0;
  if (it.live <= 0 && !(kWeigh && rb == 0)) return it;
  if (it.live < 0) it.live = 0;
  if (it.bad) {
    it.last = -1;
    it.tiles = 1;
    return it;
  }
  it.pos0 = n - 1 - nd + it.i0;
  it.first = it.pos0 - A.rule.window + 1 > 0 ? it.pos0 - A.rule.window + 1 : 0;
  it.last = it.pos0 + it.live - 1;
  if (it.live == 0) it.last = it.first - 1;
  if (kWeigh) {
    it.tiles = (n + kTileKeys - 1) / kTileKeys;
  } else if (it.last < 0) {
    it.tiles = 1;
  } else {
    it.t0 = it.first / kTileKeys;
    it.tiles = it.last / kTileKeys - it.t0 + 1;
  }
  return it;
}

__device__ __forceinline__ int load_n(const TileArgs& A, int b) { return __ldg(A.seq_len + b); }
__device__ __forceinline__ int load_nd(const TileArgs& A, int b) {
  return A.num_draft ? __ldg(A.num_draft + b) : A.P - 1;
}
__device__ __forceinline__ int load_acc(const TileArgs& A, int b, int nd) {
  return A.accept_len ? __ldg(A.accept_len + b) : nd;
}

// Tiles of a request per kv head, over its row blocks (in the key weights a tile is walked once
// per block, so all blocks count as one item).
template <bool kWeigh>
__device__ __forceinline__ int request_tiles(const TileArgs& A, int b) {
  const int n = load_n(A, b), nd = load_nd(A, b), acc = kWeigh ? load_acc(A, b, nd) : 0;
  if (kWeigh) return item_of<true>(A, n, nd, acc, 0).tiles;
  int t = 0;
  for (int rb = 0; rb < A.blocks; ++rb) t += item_of<false>(A, n, nd, acc, rb).tiles;
  return t;
}

// Where a CTA's range starts (shared memory).
struct Start {
  int64_t flat, left, per;
  int b, h, rb, off;
};

// A CTA's part of one item: tiles [ta, tb) of the item, of which [ma, mb) go through the tensor
// cores (none: filled or copied without them).
struct Piece {
  int b, h, rb;
  Item it;
  int ta, tb, ma, mb;
  bool starts, ends;  // whether it holds the item's first and last tile
  int64_t item0;      // flat index of the item's first tile
};

// The tiles of a piece that some key of [first, last] falls into.
__device__ __forceinline__ void mma_range(Piece& p) {
  p.ma = p.mb = 0;
  if (p.it.bad || p.it.last < p.it.first || p.it.last < 0) return;
  const int lo = p.it.first / kTileKeys, hi = p.it.last / kTileKeys + 1;
  p.ma = p.ta > lo ? p.ta : lo;
  p.mb = p.tb < hi ? p.tb : hi;
  if (p.mb < p.ma) p.mb = p.ma;
}

// The key weights walk a piece once per row block: turns p into its pass rb; false past the last.
__device__ __forceinline__ bool weigh_pass(const TileArgs& A, Piece& p, int rb) {
  if (rb == 0) return true;
  if (rb >= A.blocks || p.it.bad) return false;
  p.it = item_of<true>(A, p.it.n, p.it.nd, p.it.acc, rb);
  p.rb = rb;
  mma_range(p);
  return p.it.live > 0;
}

template <bool kWeigh>
struct Walk {
  const TileArgs& A;
  int b, h, rb, off, n, nd, acc;
  int64_t flat, left;
  Item it;
  __device__ __forceinline__ Walk(const TileArgs& a, const Start& s)
      : A(a), b(s.b), h(s.h), rb(s.rb), off(s.off), flat(s.flat), left(s.left) {
    load();
  }
  __device__ __forceinline__ void load() {
    n = load_n(A, b);
    nd = load_nd(A, b);
    acc = kWeigh ? load_acc(A, b, nd) : 0;
    it = item_of<kWeigh>(A, n, nd, acc, rb);
  }
  __device__ __forceinline__ bool next(Piece& p) {
    if (left <= 0) return false;
    while (it.tiles == 0) advance();
    const int64_t rest = it.tiles - off, take = rest < left ? rest : left;
    p.b = b;
    p.h = h;
    p.rb = rb;
    p.it = it;
    p.ta = it.t0 + off;
    p.tb = p.ta + (int)take;
    p.starts = off == 0;
    p.ends = take == rest;
    p.item0 = flat - off;
    mma_range(p);
    flat += take;
    left -= take;
    off += (int)take;
    if (off == it.tiles && left > 0) advance();
    return true;
  }
  __device__ __forceinline__ void advance() {
    off = 0;
    if (!kWeigh && ++rb < A.blocks) {
      it = item_of<kWeigh>(A, n, nd, acc, rb);
      return;
    }
    rb = 0;
    if (++h == A.Hkv) {
      h = 0;
      ++b;
      load();
    } else if (!kWeigh) {
      it = item_of<kWeigh>(A, n, nd, acc, rb);
    }
  }
};

// The CTA's share of the flat range (all threads; ends with a CTA barrier).
template <class S>
__device__ __forceinline__ void find_start(const TileArgs& A, Start* s, int64_t* scratch) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kW = S::Threads / 32;
  const int each = (A.B + S::Threads - 1) / S::Threads;
  const int b0 = tid * each, b1 = b0 + each < A.B ? b0 + each : A.B;
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) mine += (int64_t)request_tiles<S::Weigh>(A, b) * A.Hkv;
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) scratch[warp] = incl;
  __syncthreads();
  int64_t before = 0, total = 0;
  for (int q = 0; q < kW; ++q) {
    if (q < warp) before += scratch[q];
    total += scratch[q];
  }
  incl += before;
  const int64_t per = (total + gridDim.x - 1) / gridDim.x;
  const int64_t from = per * blockIdx.x;
  if (tid == 0) {
    s->flat = from;
    s->per = per;
    s->left = from >= total ? 0 : (total - from < per ? total - from : per);
  }
  if (from < total && incl - mine <= from && from < incl) {
    int64_t at = incl - mine;
    int b = b0;
    int64_t t = (int64_t)request_tiles<S::Weigh>(A, b) * A.Hkv;
    while (at + t <= from) {
      at += t;
      ++b;
      t = (int64_t)request_tiles<S::Weigh>(A, b) * A.Hkv;
    }
    const int64_t per_head = t / A.Hkv;
    s->b = b;
    s->h = (int)((from - at) / per_head);
    int off = (int)((from - at) % per_head);
    int rb = 0;
    if (!S::Weigh) {
      const int n = load_n(A, b), nd = load_nd(A, b);
      int tiles = item_of<false>(A, n, nd, 0, 0).tiles;
      while (off >= tiles) {
        off -= tiles;
        tiles = item_of<false>(A, n, nd, 0, ++rb).tiles;
      }
    }
    s->rb = rb;
    s->off = off;
  }
  __syncthreads();
}

// ---- shared memory ------------------------------------------------------------------------------
template <class S>
struct TileShared {
  uint64_t full[S::NU], empty[S::NU];
  uint64_t q_full[S::NQ], q_empty[S::NQ];
  uint64_t s_full[2], s_empty[2];
  uint64_t p_full, pv_done;
  uint32_t tmem;
  int dead;
  int bad_piece[4];  // 1 + the ordinal of a piece with a page outside the pool, by ordinal % 4
  int issued[S::NU]; // passes whose copies into the unit were started
  int q_issued[S::NQ];
  uint64_t drain;
  int last_arrival;
  int64_t scratch[16];
  Start start;
  alignas(16) float m[S::N];       // running maximum; in the key weights the row's lse (log2)
  alignas(16) float slope[S::N];   // log2(e) * slope
  alignas(16) float ahead[S::N];   // the column's position less the block's first
  alignas(16) float alpha[S::N];
  alignas(16) float red[4][S::N];  // per-warp maxima or sums
  int hi[S::N], lo[S::N];          // the column sees keys j with lo < j <= hi
  int row[S::N];                   // output row of the column, from the item's first
  unsigned int odd_keys;           // partly visible keys whose values are not finite
  int odd_first;
};

// Position of tensor `idx` (in ring order) in the ring.
template <class S>
__device__ __forceinline__ int unit_slot(int unit) {
  return unit % S::NU;
}
template <class S>
__device__ __forceinline__ uint32_t unit_pass(int unit) {
  return (uint32_t)(unit / S::NU);
}
// First unit of the key tile and of the value tile of the x-th tile the CTA walks.
template <class S>
__device__ __forceinline__ int k_unit(int x) {
  return S::Weigh ? x * S::U : (x == 0 ? 0 : (2 * x - 1) * S::U);
}
template <class S>
__device__ __forceinline__ int v_unit(int x) {
  return (2 * x + 2) * S::U;
}

// ---- the copying warp -----------------------------------------------------------------------
template <class S>
struct Loader {
  const TileArgs& A;
  TileShared<S>& sh;
  unsigned char* ring;
  int lane;

  // Page of the lane's group of `box` keys in a tile, or -1 where no key of it is seen, -2 for
  // a page that does not exist.
  __device__ __forceinline__ int page_of(const Piece& p, int tile) const {
    const int j = tile * kTileKeys + lane * A.box;
    if (lane * A.box >= kTileKeys || j > p.it.last || j + A.box - 1 < p.it.first) return -1;
    const int id = __ldg(A.table + (int64_t)p.b * A.max_pages + (j >> A.log_page));
    return id < 0 || id >= A.num_pages ? -2 : id;
  }
  __device__ __forceinline__ void load(const CUtensorMap* map, const Piece& p, int tile, int page,
                                       int unit0) const {
    const bool mine = page >= 0;
    const uint32_t bytes =
        (uint32_t)(__popc(__ballot_sync(0xffffffffu, mine)) * A.box) * 128u;
    const int slot_in_page = (tile * kTileKeys + lane * A.box) & ((1 << A.log_page) - 1);
#pragma unroll
    for (int c = 0; c < S::U; ++c) {
      const int s = unit_slot<S>(unit0 + c);
      const uint32_t pass = unit_pass<S>(unit0 + c);
      if (pass > 0) wait_phase(&sh.empty[s], (pass - 1) & 1u, &sh.dead);
      __syncwarp();
      const bool dead = __any_sync(0xffffffffu, *(volatile int*)&sh.dead);
      if (dead) continue;
      if (lane == 0) {
        sh.issued[s] = (int)pass + 1;
        mbar_arrive_expect_tx(&sh.full[s], bytes);
      }
      __syncwarp();
      if (mine)
        tile_g2s(ring + s * kUnitBytes + lane * A.box * 128, map, &sh.full[s], c * 64,
                 slot_in_page, p.h, page);
    }
  }
};

template <class S>
__device__ __forceinline__ void copy_role(const TileArgs& A, TileShared<S>& sh,
                                          unsigned char* qbuf, unsigned char* ring,
                                          const CUtensorMap* mq, const CUtensorMap* mk,
                                          const CUtensorMap* mv) {
  const int lane = threadIdx.x & 31;
  Loader<S> L{A, sh, ring, lane};
  Walk<S::Weigh> w(A, sh.start);
  Piece p, prev{};
  int x = 0, ordinal = 0, prev_tile = 0, prev_page = 0;
  while (w.next(p)) {
    for (int rb = 0; S::Weigh ? weigh_pass(A, p, rb) : rb == 0; ++rb) {
      if (p.mb <= p.ma) continue;
      const int qs = ordinal % S::NQ, qp = ordinal / S::NQ;
      if (qp > 0) wait_phase(&sh.q_empty[qs], (uint32_t)(qp - 1) & 1u, &sh.dead);
      __syncwarp();
      if (lane == 0 && !*(volatile int*)&sh.dead) {
        sh.q_issued[qs] = qp + 1;
        mbar_arrive_expect_tx(&sh.q_full[qs], (uint32_t)(A.G * A.pos_block * S::D * 2));
        for (int c = 0; c < S::U; ++c)
          tile_g2s(qbuf + qs * S::QBytes + c * S::N * 128, mq, &sh.q_full[qs], c * 64, p.h * A.G,
                   p.it.i0, p.b);
      }
      __syncwarp();
      int page = L.page_of(p, p.ma);
      for (int t = p.ma; t < p.mb; ++t) {
        const int next_page = t + 1 < p.mb ? L.page_of(p, t + 1) : -1;
        if (__any_sync(0xffffffffu, page == -2) && lane == 0)
          *(volatile int*)&sh.bad_piece[ordinal & 3] = ordinal + 1;
        __syncwarp();
        L.load(mk, p, t, page, k_unit<S>(x));
        if (!S::Weigh) {
          if (x > 0) L.load(mv, prev, prev_tile, prev_page, v_unit<S>(x - 1));
          prev = p;
          prev_tile = t;
          prev_page = page;
        }
        page = next_page;
        ++x;
      }
      ++ordinal;
    }
  }
  if (!S::Weigh && x > 0) L.load(mv, prev, prev_tile, prev_page, v_unit<S>(x - 1));
  if (*(volatile int*)&sh.dead && lane == 0) {
    // given up: no copy may outlive the CTA
    for (int s = 0; s < S::NU; ++s)
      if (sh.issued[s] > 0) mbar_wait(&sh.full[s], (uint32_t)(sh.issued[s] - 1) & 1u, kTileWaitNs);
    for (int s = 0; s < S::NQ; ++s)
      if (sh.q_issued[s] > 0)
        mbar_wait(&sh.q_full[s], (uint32_t)(sh.q_issued[s] - 1) & 1u, kTileWaitNs);
  }
  __syncwarp();
}

// ---- the thread that issues the matrix instructions -----------------------------------------
template <class S>
struct Issuer {
  const TileArgs& A;
  TileShared<S>& sh;
  uint32_t q_addr, p_addr, ring_addr, tmem;
  uint32_t qk_desc, pv_desc;

  __device__ __forceinline__ bool dead() const { return *(volatile int*)&sh.dead != 0; }

  // S^T of the tile whose keys start at ring unit `unit`, into S buffer `buf`.
  __device__ __forceinline__ void scores(int unit, int qs, int buf) const {
#pragma unroll
    for (int c = 0; c < S::U; ++c) {
      const int s = unit_slot<S>(unit + c);
      wait_phase(&sh.full[s], unit_pass<S>(unit + c) & 1u, &sh.dead);
      tc_fence_after();
      if (dead()) continue;
      const uint32_t a0 = ring_addr + s * kUnitBytes;
      const uint32_t b0 = q_addr + qs * S::QBytes + c * S::N * 128;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        mma_f16(tmem + buf * S::N, smem_desc(a0 + 32 * k, 16, 1024, kSwizzle128),
                smem_desc(b0 + 32 * k, 16, 1024, kSwizzle128), qk_desc, c > 0 || k > 0);
      mma_commit(&sh.empty[s]);
    }
    if (!dead()) mma_commit(&sh.s_full[buf]);
  }
  // O^T (+)= V^T P^T of the y-th tile.
  __device__ __forceinline__ void values(int y, bool first) const {
    wait_phase(&sh.p_full, (uint32_t)y & 1u, &sh.dead);
    tc_fence_after();
    constexpr int kPer = S::U >= 2 ? 2 : 1;  // units per accumulator
#pragma unroll
    for (int m = 0; m < S::MBlocks; ++m) {
      const int unit = v_unit<S>(y) + m * kPer;
      const int s = unit_slot<S>(unit);
#pragma unroll
      for (int c = 0; c < kPer; ++c) {
        wait_phase(&sh.full[unit_slot<S>(unit + c)], unit_pass<S>(unit + c) & 1u, &sh.dead);
      }
      tc_fence_after();
      if (dead()) continue;
      const uint32_t a0 = ring_addr + s * kUnitBytes;
#pragma unroll
      for (int part = 0; part < 2; ++part)  // the weights' high and low halves
#pragma unroll
        for (int k = 0; k < kTileKeys / 16; ++k)
          // values of 64 columns lie 128 bytes per key; with D = 64 both halves of the
          // instruction's rows read the same columns, and the upper half is not used
          mma_f16(tmem + (2 + m) * S::N,
                  smem_desc(a0 + k * 2048, kPer == 2 ? kUnitBytes : 0, 1024, kSwizzle128),
                  smem_desc(p_addr + part * (kTileKeys * S::N * 2) + k * 512, kTileKeys * 32, 256,
                            kSwizzle32),
                  pv_desc, !(first && part == 0 && k == 0));
#pragma unroll
      for (int c = 0; c < kPer; ++c) mma_commit(&sh.empty[unit_slot<S>(unit + c)]);
    }
    if (!dead()) mma_commit(&sh.pv_done);
  }
};

template <class S>
__device__ __forceinline__ void issue_role(const TileArgs& A, TileShared<S>& sh,
                                           unsigned char* qbuf, unsigned char* pbuf,
                                           unsigned char* ring) {
  Issuer<S> I{A, sh, smem_u32(qbuf), smem_u32(pbuf), smem_u32(ring), sh.tmem,
              mma_desc(A.bf16, false, false, 128, S::N), mma_desc(A.bf16, true, true, 128, S::N)};
  Walk<S::Weigh> w(A, sh.start);
  Piece p;
  int x = 0, ordinal = 0, used[2] = {0, 0};
  bool prev_first = false;
  while (w.next(p)) {
    for (int rb = 0; S::Weigh ? weigh_pass(A, p, rb) : rb == 0; ++rb) {
      if (p.mb <= p.ma) continue;
      const int qs = ordinal % S::NQ;
      wait_phase(&sh.q_full[qs], (uint32_t)(ordinal / S::NQ) & 1u, &sh.dead);
      for (int t = p.ma; t < p.mb; ++t) {
        const int buf = (S::Weigh ? t : x) & 1;
        const int c = buf ? used[1]++ : used[0]++;
        if (c > 0) wait_phase(&sh.s_empty[buf], (uint32_t)(c - 1) & 1u, &sh.dead);
        tc_fence_after();
        I.scores(k_unit<S>(x), qs, buf);
        if (t + 1 == p.mb && !I.dead()) mma_commit(&sh.q_empty[qs]);
        if (!S::Weigh) {
          if (x > 0) I.values(x - 1, prev_first);
          prev_first = t == p.ma;
        }
        ++x;
      }
      ++ordinal;
    }
  }
  if (!S::Weigh && x > 0) I.values(x - 1, prev_first);
  if (I.dead()) {  // given up: no instruction may outlive the tensor memory
    mma_commit(&sh.drain);
    mbar_wait(&sh.drain, 0, kTileWaitNs);
  }
}

// ---- the softmax threads ------------------------------------------------------------------------
__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ bool bar_or(int id, int threads, bool pred) {
  uint32_t r;
  asm volatile(
      "{ .reg .pred p, q;\n"
      "  setp.ne.u32 p, %1, 0;\n"
      "  bar.red.or.pred q, %2, %3, p;\n"
      "  selp.u32 %0, 1, 0, q; }"
      : "=r"(r)
      : "r"((uint32_t)pred), "r"(id), "r"(threads)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Column-wise reduction over a warp's lanes of kC values per lane (16 or a multiple of 32):
// halves the columns a lane carries at every step, so 31 exchanges serve 32 columns. Lane l
// ends with column 32 * g + l of each group g (16 columns: lanes l and l + 16 share column l).
template <int kC, bool kMax>
__device__ __forceinline__ void column_reduce(const float (&v)[kC], float* out, int lane) {
  auto op = [](float a, float b) { return kMax ? fmaxf(a, b) : a + b; };
  constexpr int kW = kC < 32 ? kC : 32;
#pragma unroll
  for (int g = 0; g < kC; g += kW) {
    float r[kW];
#pragma unroll
    for (int c = 0; c < kW; ++c) r[c] = v[g + c];
#pragma unroll
    for (int o = kW / 2; o >= 1; o >>= 1) {
      const bool up = lane & o;
#pragma unroll
      for (int c = 0; c < o; ++c) {
        const float give = up ? r[c] : r[c + o], keep = up ? r[c + o] : r[c];
        r[c] = op(keep, __shfl_xor_sync(0xffffffffu, give, o));
      }
    }
    if (kW == 16) r[0] = op(r[0], __shfl_xor_sync(0xffffffffu, r[0], 16));
    if (lane < kW) out[g + lane] = r[0];
  }
}

// Scores of a thread's key from the products q.k, in units of log2: scale, cap, distance.
template <int kC>
__device__ __forceinline__ void apply_rule(float (&s)[kC], const ScoreRule& r, float away,
                                           const float* slope, const float* ahead) {
  const float scale2 = r.scale * kLog2e;
  if (r.softcap > 0.0f) {
    // c tanh(y) = c - 2 c / (1 + 2^(2 log2(e) y))
    const float in = 2.0f * scale2 / r.softcap, c2 = r.softcap * kLog2e;
#pragma unroll
    for (int c = 0; c < kC; ++c) s[c] = fmaf(-2.0f * c2, rcp_fast(1.0f + ex2(s[c] * in)), c2);
  } else {
#pragma unroll
    for (int c = 0; c < kC; ++c) s[c] *= scale2;
  }
  if (r.slopes) {
#pragma unroll
    for (int c = 0; c < kC; ++c) s[c] = fmaf(-slope[c], away + ahead[c], s[c]);
  }
}

// The tables of a piece's columns (all softmax threads; barriers around it are the caller's).
template <class S>
__device__ __forceinline__ void set_columns(const TileArgs& A, TileShared<S>& sh, const Piece& p) {
  for (int c = threadIdx.x; c < S::N; c += S::SoftThreads) {
    const int i = c / A.G, g = c - i * A.G;
    const bool live = i < p.it.live;
    const int pos = p.it.pos0 + i;
    sh.slope[c] = live && A.rule.slopes ? __ldg(A.rule.slopes + p.h * A.G + g) * kLog2e : 0.0f;
    sh.ahead[c] = (float)i;
    sh.hi[c] = live ? pos : -1;
    sh.lo[c] = pos - A.rule.window;
    sh.row[c] = i * A.Hq + g;
    if (S::Weigh) {
      // a row that does not count, or one of no weight, gets none from any key
      float l = INFINITY;
      if (live) {
        const float v = __ldg(A.lse + p.b * A.lse_req + (p.it.i0 + i) * A.lse_row +
                              (p.h * A.G + g) * A.lse_head);
        if (v != -INFINITY) l = v * kLog2e;
      }
      sh.m[c] = l;
    } else {
      sh.m[c] = kNoMax;
    }
  }
}

__device__ __forceinline__ uint32_t pack16(bool bf16, float a, float b) {
  if (bf16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float2 unpack16(bool bf16, uint32_t w) {
  if (bf16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ void store16(void* base, int64_t at, bool bf16, float x) {
  if (bf16)
    static_cast<__nv_bfloat16*>(base)[at] = __float2bfloat16_rn(x);
  else
    static_cast<__half*>(base)[at] = __float2half_rn(x);
}
__device__ __forceinline__ bool not_finite16(bool bf16, uint32_t x) {
  const uint32_t m = bf16 ? 0x7f80u : 0x7c00u;
  return (x & m) == m;
}

constexpr int kAllBar = 3;  // named barriers: 1 and 2 for the groups, 3 for all softmax threads

// ---- attention --------------------------------------------------------------------------------
// What one softmax thread does for the attention: its key of every tile, its share of O.
template <class S>
struct Attend {
  const TileArgs& A;
  TileShared<S>& sh;
  unsigned char *pbuf, *ring;
  int lane, quarter, group, key;
  uint32_t lane_base;  // tensor-memory address of the thread's lanes
  int col0;            // the group's first column

  __device__ __forceinline__ void group_sync() const { bar_sync(1 + group, 128); }

  // Raise the columns' maxima to those of this tile's scores s, and scale what they hold.
  __device__ __forceinline__ void raise(const float (&s)[S::NC], float (&l)[S::NC], bool first) {
    column_reduce<S::NC, true>(s, &sh.red[quarter][col0], lane);
    group_sync();
    if (quarter == 0) {
      for (int c = col0 + lane; c < col0 + S::NC; c += 32) {
        const float was = sh.m[c];
        const float m = fmaxf(fmaxf(fmaxf(sh.red[0][c], sh.red[1][c]),
                                    fmaxf(sh.red[2][c], sh.red[3][c])), was);
        sh.alpha[c] = ex2(was - m);
        sh.m[c] = m;
      }
    }
    group_sync();
#pragma unroll
    for (int c = 0; c < S::NC; ++c) l[c] *= sh.alpha[col0 + c];
    if (first) return;
    tc_fence_after();
#pragma unroll
    for (int m = 0; m < S::MBlocks; ++m)
#pragma unroll
      for (int q = 0; q < S::NC; q += 16) {
        float o[16];
        const uint32_t at = lane_base + (2 + m) * S::N + col0 + q;
        tmem_ld16(at, o);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 16; ++c) o[c] *= sh.alpha[col0 + q + c];
        tmem_st16(at, o);
      }
    tmem_wait_st();
  }

  // Values of keys that some row of a tile does not see: what no row sees becomes 0; of a key
  // that only some rows see, the values that are not finite become 0 and are added to the rows
  // that see it at the end (0 times infinity would reach the others).
  __device__ __forceinline__ void clean_values(const Piece& p, int x, int j, int first_full) {
    const int unit = v_unit<S>(x);
#pragma unroll
    for (int c = 0; c < S::U; ++c)
      wait_phase(&sh.full[unit_slot<S>(unit + c)], unit_pass<S>(unit + c) & 1u, &sh.dead);
    const bool none = j > p.it.last || j < p.it.first;
    const bool some = !none && (j > p.it.pos0 || j < first_full);
    if (!none && !some) return;
    bool odd = false;
#pragma unroll
    for (int c = 0; c < S::U; ++c) {
      uint4* row = reinterpret_cast<uint4*>(ring + unit_slot<S>(unit + c) * kUnitBytes + key * 128);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        if (none) {
          row[q] = make_uint4(0u, 0u, 0u, 0u);
          continue;
        }
        uint4 v = row[q];
        uint32_t* w = reinterpret_cast<uint32_t*>(&v);
        bool hit = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (not_finite16(A.bf16, w[e] & 0xffffu)) {
            w[e] &= 0xffff0000u;
            hit = true;
          }
          if (not_finite16(A.bf16, w[e] >> 16)) {
            w[e] &= 0xffffu;
            hit = true;
          }
        }
        if (hit) row[q] = v;
        odd |= hit;
      }
    }
    if (odd) atomicOr(&sh.odd_keys, 1u << (j > p.it.pos0 ? j - p.it.pos0 - 1 : 16 + j - p.it.first));
  }

  // One tile: the scores of x, their weights into shared memory.
  __device__ __forceinline__ void tile(const Piece& p, int t, int x, int first_full,
                                       float (&l)[S::NC]) {
    const int buf = x & 1, j = t * kTileKeys + key;
    const bool first = t == p.ma;
    float s[S::NC];
    wait_phase(&sh.s_full[buf], (uint32_t)(x >> 1) & 1u, &sh.dead);
    tc_fence_after();
#pragma unroll
    for (int q = 0; q < S::NC; q += 16)
      tmem_ld16(lane_base + buf * S::N + col0 + q, reinterpret_cast<float(&)[16]>(s[q]));
    tmem_wait_ld();
    tc_fence_before();
    mbar_arrive(&sh.s_empty[buf]);
    apply_rule<S::NC>(s, A.rule, (float)(p.it.pos0 - j), &sh.slope[col0], &sh.ahead[col0]);
    const bool edge = t * kTileKeys < first_full || t * kTileKeys + kTileKeys - 1 > p.it.pos0;
    if (edge) {
#pragma unroll
      for (int c = 0; c < S::NC; ++c)
        if (j > sh.hi[col0 + c] || j <= sh.lo[col0 + c]) s[c] = -INFINITY;
    }
    float top = -INFINITY;
#pragma unroll
    for (int c = 0; c < S::NC; ++c) top = fmaxf(top, s[c] - sh.m[col0 + c]);
    bool waited = first;  // the previous product of this piece has read P and written O
    if (bar_or(1 + group, 128, top > 8.0f)) {
      if (!waited) wait_phase(&sh.pv_done, (uint32_t)(x - 1) & 1u, &sh.dead);
      waited = true;
      raise(s, l, first);
    }
    if (!waited) wait_phase(&sh.pv_done, (uint32_t)(x - 1) & 1u, &sh.dead);
#pragma unroll
    for (int q = 0; q < S::NC; q += 16) {
      uint32_t hi[8], lo[8];
#pragma unroll
      for (int c = 0; c < 16; c += 2) {
        const float a = ex2(s[q + c] - sh.m[col0 + q + c]);
        const float b = ex2(s[q + c + 1] - sh.m[col0 + q + c + 1]);
        l[q + c] += a;
        l[q + c + 1] += b;
        hi[c / 2] = pack16(A.bf16, a, b);
        const float2 h = unpack16(A.bf16, hi[c / 2]);
        lo[c / 2] = pack16(A.bf16, a - h.x, b - h.y);
      }
      // 16 columns of a key: 32 bytes, their 16-byte halves swapped in every other 4 keys
      unsigned char* at = pbuf + (col0 + q) / 16 * (kTileKeys * 32) + key * 32;
      const int sw = ((key >> 2) & 1) * 16;
      *reinterpret_cast<uint4*>(at + sw) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      *reinterpret_cast<uint4*>(at + (16 - sw)) = make_uint4(hi[4], hi[5], hi[6], hi[7]);
      at += kTileKeys * S::N * 2;
      *reinterpret_cast<uint4*>(at + sw) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      *reinterpret_cast<uint4*>(at + (16 - sw)) = make_uint4(lo[4], lo[5], lo[6], lo[7]);
    }
    if (edge && group == 0) clean_values(p, x, j, first_full);
    fence_proxy_async();
    tc_fence_before();
    mbar_arrive(&sh.p_full);
  }

  // Rows without a visible key, or of a request with bad counts.
  __device__ __forceinline__ void fill(const Piece& p) const {
    const int64_t row0 = ((int64_t)p.b * A.P + p.it.i0) * A.Hq + p.h * A.G;
    const float v = p.it.bad ? __uint_as_float(0x7fc00000u) : 0.0f;
    const int rows = p.it.live * A.G;
    for (int e = threadIdx.x; e < rows * S::D; e += S::SoftThreads)
      store16(A.out, (row0 + sh.row[e / S::D]) * S::D + e % S::D, A.bf16, v);
    if (A.out_lse)
      for (int c = threadIdx.x; c < rows; c += S::SoftThreads)
        A.out_lse[row0 + sh.row[c]] = p.it.bad ? v : -INFINITY;
  }

  __device__ __forceinline__ float* slot(int64_t i) const {
    return A.part + i * (S::N * (S::D + 2));
  }

  // The end of a piece: O and the sums leave for the output or for the workspace.
  __device__ __forceinline__ void finish(const Piece& p, int x, int ordinal, float (&l)[S::NC]) {
    wait_phase(&sh.pv_done, (uint32_t)x & 1u, &sh.dead);
    tc_fence_after();
    column_reduce<S::NC, false>(l, &sh.red[quarter][col0], lane);
    group_sync();
    const bool poison = *(volatile int*)&sh.dead ||
                        *(volatile int*)&sh.bad_piece[ordinal & 3] == ordinal + 1;
    const bool whole = p.starts && p.ends;
    const int rows = p.it.live * A.G;
    const int64_t row0 = ((int64_t)p.b * A.P + p.it.i0) * A.Hq + p.h * A.G;
    float* part = slot(2 * (int64_t)blockIdx.x + (p.starts ? 1 : 0));
    if (quarter == 0) {
      for (int c = col0 + lane; c < col0 + S::NC; c += 32) {
        float sum = (sh.red[0][c] + sh.red[1][c]) + (sh.red[2][c] + sh.red[3][c]);
        if (poison) sum = __uint_as_float(0x7fc00000u);
        const float m = sh.m[c];
        if (c < rows) {
          if (whole) {
            if (A.out_lse)
              A.out_lse[row0 + sh.row[c]] =
                  sum == 0.0f ? -INFINITY : (m + log2f(sum)) * (1.0f / kLog2e);
          } else {
            *reinterpret_cast<float2*>(part + S::N * S::D + 2 * c) = make_float2(m, sum);
          }
        }
        sh.alpha[c] = sum == 0.0f ? 0.0f : 1.0f / sum;
      }
    }
    group_sync();
    const unsigned int odd = *(volatile unsigned int*)&sh.odd_keys;
    if (S::D >= 128 || quarter < 2) {
#pragma unroll
      for (int m = 0; m < S::MBlocks; ++m) {
        const int d = m * 128 + quarter * 32 + lane;
#pragma unroll
        for (int q = 0; q < S::NC; q += 16) {
          float o[16];
          tmem_ld16(lane_base + (2 + m) * S::N + col0 + q, o);
          tmem_wait_ld();
          if (odd) add_odd(p, odd, d, col0 + q, o);
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const int n = col0 + q + c;
            if (n < rows) {
              if (whole)
                store16(A.out, (row0 + sh.row[n]) * S::D + d, A.bf16, o[c] * sh.alpha[n]);
              else
                part[n * S::D + d] = o[c];
            }
          }
        }
      }
    }
    tc_fence_before();
    if (!whole) join(p, rows, row0);
  }

  __device__ __forceinline__ void add_odd(const Piece& p, unsigned int odd, int d, int n0,
                                          float (&o)[16]) const {
    while (odd) {
      const int bit = __ffs(odd) - 1;
      odd &= odd - 1;
      const int j = bit < 16 ? p.it.pos0 + 1 + bit : p.it.first + bit - 16;
      const float v = odd_value(p, j, d);
      if (isfinite(v)) continue;
#pragma unroll
      for (int c = 0; c < 16; ++c)
        if (j <= sh.hi[n0 + c] && j > sh.lo[n0 + c]) o[c] += v;
    }
  }
  const void* v_data;
  int64_t vp, vt, vh;
  __device__ __forceinline__ float odd_value(const Piece& p, int j, int d) const {
    const int page = __ldg(A.table + (int64_t)p.b * A.max_pages + (j >> A.log_page));
    if (page < 0 || page >= A.num_pages) return 0.0f;
    const int64_t at = page * vp + (j & ((1 << A.log_page) - 1)) * vt + p.h * vh + d;
    return A.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(v_data)[at])
                  : __half2float(static_cast<const __half*>(v_data)[at]);
  }

  // Count this piece in; the CTA that brings an item's last piece joins them, in order.
  __device__ __forceinline__ void join(const Piece& p, int rows, int64_t row0) {
    const int64_t per = sh.start.per;
    const int64_t c0 = p.item0 / per, c1 = (p.item0 + p.it.tiles - 1) / per;
    __threadfence();
    bar_sync(kAllBar, S::SoftThreads);
    if (threadIdx.x == 0) {
      // the counters are cleared by the launch ahead of this one
      asm volatile("griddepcontrol.wait;" ::: "memory");
      sh.last_arrival = arrive_last(A.counters + c0, (unsigned int)(c1 - c0 + 1));
    }
    bar_sync(kAllBar, S::SoftThreads);
    if (!sh.last_arrival) return;
    __threadfence();
    const int np = (int)(c1 - c0 + 1);
    auto slot_of = [&](int i) { return slot(i == 0 ? 2 * c0 + 1 : 2 * (c0 + i)); };
    constexpr int kV = S::D / 32;  // of D per lane
    for (int n = threadIdx.x >> 5; n < rows; n += S::SoftWarps) {
      float m = kNoMax;
      for (int i = lane; i < np; i += 32)
        m = fmaxf(m, __ldcg(slot_of(i) + S::N * S::D + 2 * n));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      float sum = 0.0f;
      for (int i = lane; i < np; i += 32) {
        const float2 ml = __ldcg(reinterpret_cast<const float2*>(slot_of(i) + S::N * S::D + 2 * n));
        sum += ex2(ml.x - m) * ml.y;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      float acc[kV];
#pragma unroll
      for (int e = 0; e < kV; ++e) acc[e] = 0.0f;
#pragma unroll 4
      for (int i = 0; i < np; ++i) {
        const float* s = slot_of(i);
        const float w = ex2(__ldcg(s + S::N * S::D + 2 * n) - m);
#pragma unroll
        for (int e = 0; e < kV; e += 2) {
          const float2 v = __ldcg(reinterpret_cast<const float2*>(s + n * S::D + e * 32 + 2 * lane));
          acc[e] = fmaf(w, v.x, acc[e]);
          acc[e + 1] = fmaf(w, v.y, acc[e + 1]);
        }
      }
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      const int64_t at = (row0 + sh.row[n]) * S::D;
#pragma unroll
      for (int e = 0; e < kV; e += 2)
        *reinterpret_cast<uint32_t*>(static_cast<char*>(A.out) + 2 * (at + e * 32 + 2 * lane)) =
            pack16(A.bf16, acc[e] * inv, acc[e + 1] * inv);
      if (A.out_lse && lane == 0)
        A.out_lse[row0 + sh.row[n]] = sum == 0.0f ? -INFINITY : (m + log2f(sum)) * (1.0f / kLog2e);
    }
  }

  __device__ __forceinline__ void run() {
    Walk<false> w(A, sh.start);
    Piece p;
    int x = 0, ordinal = 0;
    while (w.next(p)) {
      bar_sync(kAllBar, S::SoftThreads);  // the last piece's tables have been read
      set_columns<S>(A, sh, p);
      if (threadIdx.x == 0) sh.odd_keys = 0;
      bar_sync(kAllBar, S::SoftThreads);
      if (p.mb <= p.ma) {
        fill(p);
        continue;
      }
      float l[S::NC];
#pragma unroll
      for (int c = 0; c < S::NC; ++c) l[c] = 0.0f;
      // keys from here on are inside every row's window
      const int first_full = p.it.last - A.rule.window + 1;
      for (int t = p.ma; t < p.mb; ++t) tile(p, t, x++, first_full, l);
      finish(p, x - 1, ordinal++, l);
    }
  }
};

// ---- key weights ------------------------------------------------------------------------------
template <class S>
__device__ __forceinline__ void weigh_role(const TileArgs& A, TileShared<S>& sh) {
  const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3, group = threadIdx.x >> 7;
  const int key = quarter * 32 + lane;
  const uint32_t lane_base = sh.tmem + ((uint32_t)(quarter * 32) << 16);
  const float nan = __uint_as_float(0x7fc00000u);
  Walk<true> w(A, sh.start);
  Piece p;
  int used = 0;  // tiles this group has taken from its S buffer
  while (w.next(p)) {
    const int64_t row = ((int64_t)p.b * A.Hkv + p.h) * A.stride;
    float* out = A.weights + row;
    const float* prior = A.prior ? A.prior + row : nullptr;
    if (p.it.bad) {
      if (threadIdx.x == 0) out[0] = nan;
      continue;
    }
    for (int rb = 0; weigh_pass(A, p, rb); ++rb) {
      bar_sync(kAllBar, S::SoftThreads);
      set_columns<S>(A, sh, p);
      bar_sync(kAllBar, S::SoftThreads);
      const int first_full = p.it.last - A.rule.window + 1;
      const int ta = rb == 0 ? p.ta : p.ma, tb = rb == 0 ? p.tb : p.mb;
      for (int t = ta; t < tb; ++t) {
        if ((t & 1) != group) continue;
        const int j = t * kTileKeys + key;
        const bool inside = j < p.it.n;
        float total = 0.0f, before = 0.0f;
        if (inside) before = rb > 0 ? out[j] : prior ? prior[j] : 0.0f;
        if (t >= p.ma && t < p.mb) {
          bool bad = false;
          if (j >= p.it.first && j <= p.it.last) {
            const int page = __ldg(A.table + (int64_t)p.b * A.max_pages + (j >> A.log_page));
            bad = page < 0 || page >= A.num_pages;
          }
          const bool edge =
              t * kTileKeys < first_full || t * kTileKeys + kTileKeys - 1 > p.it.pos0;
          wait_phase(&sh.s_full[group], (uint32_t)used & 1u, &sh.dead);
          ++used;
          tc_fence_after();
#pragma unroll
          for (int q = 0; q < S::N; q += 16) {
            float s[16];
            tmem_ld16(lane_base + group * S::N + q, s);
            tmem_wait_ld();
            apply_rule<16>(s, A.rule, (float)(p.it.pos0 - j), &sh.slope[q], &sh.ahead[q]);
            float part = 0.0f;
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              float e = ex2(s[c] - sh.m[q + c]);
              if (edge && (j > sh.hi[q + c] || j <= sh.lo[q + c])) e = 0.0f;
              part += e;
            }
            total += part;
          }
          tc_fence_before();
          mbar_arrive(&sh.s_empty[group]);
          if (bad || *(volatile int*)&sh.dead) total = nan;
        }
        if (inside) out[j] = before + total;
      }
    }
  }
}

// ---- the kernel ---------------------------------------------------------------------------------
struct ValuePool {
  const void* data;
  int64_t page, token, head;
};

template <class S>
__global__ void __launch_bounds__(S::Threads, 1)
    tile_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                const __grid_constant__ CUtensorMap mv, const __grid_constant__ TileArgs A,
                const __grid_constant__ ValuePool vpool) {
  extern __shared__ unsigned char tile_smem[];
  __shared__ TileShared<S> sh;
  // operand tiles start on 1024-byte boundaries (the swizzle pattern's period)
  unsigned char* base = tile_smem + ((1024u - (smem_u32(tile_smem) & 1023u)) & 1023u);
  unsigned char* qbuf = base;
  unsigned char* pbuf = qbuf + S::NQ * S::QBytes;
  unsigned char* ring = pbuf + S::PBytes;
  const int tid = threadIdx.x, warp = tid >> 5;

  find_start<S>(A, &sh.start, sh.scratch);
  if (sh.start.left <= 0) return;
  if (tid == 0) {
    for (int s = 0; s < S::NU; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], 1);
      sh.issued[s] = 0;
    }
    for (int s = 0; s < S::NQ; ++s) {
      mbar_init(&sh.q_full[s], 1);
      mbar_init(&sh.q_empty[s], 1);
      sh.q_issued[s] = 0;
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sh.s_full[s], 1);
      mbar_init(&sh.s_empty[s], S::Weigh ? 128 : S::SoftThreads);
    }
    mbar_init(&sh.p_full, S::SoftThreads);
    mbar_init(&sh.pv_done, 1);
    mbar_init(&sh.drain, 1);
    sh.dead = 0;
    for (int i = 0; i < 4; ++i) sh.bad_piece[i] = 0;
    fence_barrier_init();
  }
  if (warp == 0) tmem_alloc(&sh.tmem, S::TmemCols);
  // columns past the query rows multiply zeros: the copies never write them
  {
    const int rows = A.G * A.pos_block;
    for (int q = 0; q < S::NQ; ++q)
      for (int c = 0; c < S::U; ++c) {
        uint4* z = reinterpret_cast<uint4*>(qbuf + q * S::QBytes + c * S::N * 128);
        for (int e = rows * 8 + tid; e < S::N * 8; e += S::Threads)
          z[e] = make_uint4(0u, 0u, 0u, 0u);
      }
    fence_proxy_async();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  if (warp == S::SoftWarps) {
    copy_role<S>(A, sh, qbuf, ring, &mq, &mk, &mv);
  } else if (warp == S::SoftWarps + 1) {
    if ((tid & 31) == 0) issue_role<S>(A, sh, qbuf, pbuf, ring);
    __syncwarp();
  } else if constexpr (S::Weigh) {
    weigh_role<S>(A, sh);
  } else {
    const int lane = tid & 31, quarter = warp & 3, group = warp >> 2;
    Attend<S> R{A, sh, pbuf, ring, lane, quarter, group, quarter * 32 + lane,
                sh.tmem + ((uint32_t)(quarter * 32) << 16), group * S::NC,
                vpool.data, vpool.page, vpool.token, vpool.head};
    R.run();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_free(sh.tmem, S::TmemCols);
}

// ---- the host side ------------------------------------------------------------------------------
int device_sm_count();

// A 4-D tensor map of 16-bit elements, 64 wide boxes of 128-byte swizzled rows.
sv_status encode_map(CUtensorMap* map, const void* data, bool bf16, const uint64_t (&dims)[4],
                     const int64_t (&strides)[3], const uint32_t (&box)[4]);

// Arguments common to both calls, checked; fills the shared part of TileArgs and the q map's
// and key map's inputs. SV_OK with B == 0 means there is nothing to do.
sv_status check_tile_call(const sv_kv_shape* s, const sv_score_rule* rule, const void* q,
                          int64_t q_req, int64_t q_row, int64_t q_head, const sv_kv_pool* k,
                          const int32_t* page_table, const int32_t* seq_len,
                          const int32_t* num_draft);
sv_status fill_tile_args(TileArgs& A, CUtensorMap* mq, CUtensorMap* mk, const sv_kv_shape* s,
                         const sv_score_rule* rule, const void* q, int64_t q_req, int64_t q_row,
                         int64_t q_head, const sv_kv_pool* k, const int32_t* page_table,
                         const int32_t* seq_len, const int32_t* num_draft, bool weigh);
sv_status encode_pool(CUtensorMap* map, const sv_kv_shape* s, const sv_kv_pool* pool);

// Query rows per pass: as many whole positions as 128 columns hold (64 in an attention of
// D = 256, where the weights of more columns would leave no room for two tiles), evenly over
// the passes.
inline void row_blocks(const sv_kv_shape* s, bool weigh, int* pos_block, int* blocks,
                       int* columns) {
  const int G = s->Hq / s->Hkv, most = (s->D == 256 && !weigh ? 64 : 128) / G;
  *blocks = (s->P + most - 1) / most;
  *pos_block = (s->P + *blocks - 1) / *blocks;
  const int rows = G * *pos_block;
  *columns = rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
}

}  // namespace sv
