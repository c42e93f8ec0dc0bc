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
// shared memory bounds a narrow instruction), the softmax about 1000. Measured, in graph
// replays, of the 6782 GB/s a copy reaches (D = 128, 16-bit; boxes differ by 3 %):
//   1 token of 64 requests, 200 .. 8192 keys, 32 / 8 heads   567 MB   95.1 us  5959 GB/s  88 %
//   6 positions of 32, 500 .. 16384 keys, 64 / 8 heads       570 MB  104.3 us  5465 GB/s  81 %
//   9 positions of 2, 100001 .. 131072 keys, 32 / 8 heads   1052 MB  167.7 us  6275 GB/s  93 %
//   5 positions of 16, window 4096, 16 / 8 heads of 256      214 MB   47.3 us  4520 GB/s  67 %
//   1 token of 1 request of 777 keys                         3.2 MB   13.0 us  (latency)
//   key weights, 6 positions of 64, 1000 .. 8192 keys        463 MB   85.4 us  5420 GB/s  80 %
//   key weights, 1 request of 1501 keys                      3.2 MB    8.2 us  (latency)
// About 10 us of a call do not depend on its size: the launch, the work list's sums (2.5 us) and
// the join (4 us). Pages of 16 slots, copied in eight pieces per unit, reach 82 % where pages of
// 64 reach 88 %, pages of 8 reach 69 %.
//
// Running maximum. m[c] only moves when a score passes it by 2^8: the accumulators are rescaled only
// in the first tiles of a row instead of in every tile. The weights are 2^(s - m + lift), with a lift
// of 7 for fp16, whose numbers end at 2^-24: a weight is at most 2^15, and 2^-32 of the largest score's
// still counts (without the lift 2^-25: 131072 keys of that weight, 0.4 % of a row, came to 0).
//
// Rounding. The weights P are given to the tensor core as a sum of 16-bit numbers, each the rest that
// those before it leave, and V^T is multiplied by all. Every rounding leaves at most half a step of what
// it rounds. fp16 takes two: a weight is off by 2^-22 of it (or by 2^-32 of the largest). bf16 takes
// three up to 32 columns, 2^-24, as fp32 itself, at next to no cost (1 token of 64 requests 97.4 us
// with two, 97.3 with three, D = 256 in a window 49.4 and 49.1, 24 rows 100.6 and 101.8), and two
// above, 2^-16 (the output's own rounding is 2^-8), where the softmax and its buffers bound and a
// third cost 2 to 17 % (9 positions over long caches 166 -> 172 us, 64 rows 109 -> 119).
//
// Work. All tiles of all (request, kv head, row block) items are one flat range, cut into equal
// costs over one CTA per SM: ragged lengths balance by construction. A CTA walks its range piece
// by piece (a piece = its part of one item), the newest keys of an item first, as their scores
// are most often the largest. A piece that is a whole item is written out; others leave (O, m, l)
// in the workspace, and a second launch, already resident while the tiles are walked, joins the
// pieces of each item in order. No CTA waits for another one, and equal calls give equal bits.
//
// Roles. Keys and values have a ring each of 16 KiB units (64 columns of 128 keys), a warp each
// that looks up the pages and starts the tiled copies, and a thread each that issues the matrix
// instructions; 8 warps do the softmax and the outputs. S is double buffered: the scores of tile
// t+1 are computed while tile t is in the softmax. The key copies' warp alone walks the work list
// and hands the pieces with tiles to the others through a queue (write_rest does the rest at the
// end). The roles' loops are kept rolled and their
// rare parts out of line: all five run at once, and at 139 KB of code (79 KB now) their loops
// pushed one another out of the instruction cache, which cost 20 to 30 % of every case.
//
// Waits. Every wait on a barrier is bounded (sv_tcgen05.cuh): one that runs out marks the CTA
// dead, after which no wait blocks, a role whose wait failed starts no copy and no instruction any
// more, and all leave their loops at the end of the piece at hand. The CTA then waits for its copies and instructions in flight, walks its range
// once more and writes NaN to everything in it: rows, key weights, its parts of split items. A
// barrier's phase is one bit, so each ring has a single consumer that takes every phase in order:
// a reader that skipped phases could take a later one for its own.
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
constexpr int kSmemMax = 232448;             // shared memory of a CTA
constexpr float kNoMax = -3.402823466e38f;   // a maximum below every finite score
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct JoinItem;

struct TileArgs {
  const int32_t *table, *seq_len, *num_draft, *accept_len;
  int B, P, Hq, Hkv, G, log_page, num_pages, max_pages;
  int pos_block, blocks;  // positions per row block, row blocks per request
  int box;                // slots per copy
  int bf16;
  ScoreRule rule;
  uint64_t wait_ns;  // the limit of a wait
  // attention
  void* out;
  float *out_lse, *part;
  struct JoinItem* joins;
  // key weights
  const float *lse, *prior;
  float* weights;
  int64_t stride, lse_req, lse_row, lse_head;
};

// An item split over several CTAs, as its first CTA leaves it for the joining kernel.
struct JoinItem {
  int rows, pieces;  // rows = 0: none
  int64_t row0;      // output row of its first column
};

template <int kD, int kN, bool kWeigh, bool kBf16 = false>
struct TileShape {
  static constexpr int D = kD, N = kN;
  static constexpr bool Bf16 = kBf16;  // (attention) the type is bf16, else fp16
  static constexpr bool Weigh = kWeigh;
  static constexpr float Lift = kBf16 ? 0.0f : 7.0f;  // (attention) of the weights' exponents
  static constexpr int U = D / 64;  // units of a key or value tile
  // Softmax warps: two groups of four (one warp per quarter of the tile's keys). In the
  // attention of 16 columns the groups are two teams that take the pieces in turn, each
  // with its own score, weight and output buffers, so one team's end of a piece (its last
  // product, its output, the next piece's tables) passes under the other's tiles; of wider
  // tiles each group takes half of the columns and there is one team (6 positions of 64 requests,
  // 24 of 32 columns: 98 us with one team, 111 us with two, whose buffers shorten the rings). In
  // the key weights each group takes every other tile.
  static constexpr int Teams = !kWeigh && N == 16 ? 2 : 1;
  static constexpr int SoftWarps = 8;
  static constexpr int SoftThreads = 32 * SoftWarps;
  static constexpr int Threads = SoftThreads + (kWeigh ? 64 : 128);
  // the warps after the softmax: key (and query) copies, scores, value copies, values
  static constexpr int KeyWarp = SoftWarps, ScoreWarp = KeyWarp + 1, CopyVWarp = KeyWarp + 2,
                       ValueWarp = KeyWarp + 3;
  static constexpr int TeamThreads = SoftThreads / Teams;
  static constexpr int NC = kWeigh || Teams == 2 ? N : N / 2;  // columns per softmax thread
  static constexpr int CH = NC < 32 ? NC : 32;                 // of which at a time
  static constexpr int QBytes = N * D * 2;
  static constexpr int NQ = N * D <= 64 * 128 ? 2 : 1;  // query buffers
  static constexpr int Parts = kBf16 && N <= 32 ? 3 : 2;  // 16-bit numbers a weight is given in
  static constexpr int PBytes = kWeigh ? 0 : Parts * kTileKeys * N * 2;
  // two buffers of weights per team where the ring keeps three tensors (of D = 256 two tiles, or ten
  // units beside weights of three parts: in a window 49.1 us with one buffer, 51.0 with two)
  static constexpr int kTables = 96 * N + 1792;  // (the size of TileShared, at most)
  static constexpr int kLeft = kSmemMax - kTables - 1024 - NQ * QBytes;
  static constexpr int NP =
      kWeigh ? 1 : (kLeft - 2 * Teams * PBytes) / kUnitBytes >= (U == 4 ? 2 * Parts + 4 : 6) ? 2 : 1;
  static constexpr int Room = (kLeft - Teams * NP * PBytes) / kUnitBytes;
  // Ring units: one ring for keys, one for values, as each has its own consumer. (A consumer
  // that skipped some phases of a unit's barrier could not tell a phase from the one after next.)
  static constexpr int NU = Room > 12 ? 12 : Room;
  static constexpr int NV = kWeigh ? 0 : U == 1 ? NU / 2 : (NU + 2) / 4 * 2;  // (pairs)
  static constexpr int NK = NU - NV;
  static constexpr int Smem = 1024 + NQ * QBytes + Teams * NP * PBytes + NU * kUnitBytes;
  static constexpr int MBlocks = kWeigh ? 0 : (D + 127) / 128;  // accumulators of 128 of D
  // Two score buffers per team, two outputs. Where tensor memory has room, the products with the
  // parts of the weights are one instruction of as many times the columns (the values, whose read
  // from shared memory bounds a narrow instruction, are read once) and are added at the end; else
  // they accumulate onto one another. (9 positions over long caches, 64 columns:
  // 163 us wide, 179 us in two; 16 columns: 94 and 96 us.)
  static constexpr bool Wide = !kWeigh && 2 * (Teams + Parts * MBlocks) * N <= 512;
  static constexpr int ON = Wide ? Parts * N : N;  // columns of an accumulator
  static constexpr int TmemNeed = 2 * (Teams * N + MBlocks * ON);
  static constexpr int TmemCols = TmemNeed <= 32 ? 32 : TmemNeed <= 64 ? 64 : TmemNeed <= 128 ? 128
                                  : TmemNeed <= 256 ? 256 : 512;
  // The cost of a tile and of starting a piece, in the units the work is divided by: a quarter
  // of the time a tile's bytes take (about 350 clocks per 64 columns; half that for the keys
  // alone).
  static constexpr int TileCost = 4;
  static constexpr int PieceCost = (kWeigh ? 20 : Teams == 2 ? 8 : 16) / U + 1;
  static_assert(TmemNeed <= 512 && NK >= 2 && Smem + kTables <= kSmemMax, "tile shape");
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
  template <class S>
  __device__ __forceinline__ int cost() const {
    return tiles == 0 ? 0 : S::PieceCost + tiles * S::TileCost;
  }
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

// Cost of a request per kv head, over its row blocks (in the key weights a tile is walked once
// per block, so all blocks count as one item).
template <class S>
__device__ __noinline__ int64_t request_cost(const TileArgs& A, int b) {
  const int n = load_n(A, b), nd = load_nd(A, b), acc = S::Weigh ? load_acc(A, b, nd) : 0;
  int64_t c = 0;
#pragma unroll 1
  for (int rb = 0; rb < (S::Weigh ? 1 : A.blocks); ++rb)
    c += item_of<S::Weigh>(A, n, nd, acc, rb).template cost<S>();
  return c;
}

// A CTA's range (shared memory): `left` units of `per`, which the other CTAs have too, from unit
// `off` of item (b, h, rb) on.
struct Start {
  int left, per, off;
  int b, h, rb;
};

// A CTA's part of one item (in the key weights: one pass over it, for one row block), as the warp
// that walks the work list hands it to the other roles.
struct Piece {
  int b, h, i0, live, pos0, first, last;  // of the item
  int n;                                  // tokens of the request
  int ta, tb;                             // its tiles
  int ma, mb;                             // those that go through the tensor cores
  int turn;    // pieces before it with such tiles
  int x0;      // such tiles before it
  int pieces;  // CTAs that hold a part of the item
  int flags;
};
// kFresh: (key weights) no earlier pass over its tiles took any through the tensor cores; kHollow:
// nor does this one, the last of them.
enum { kStarts = 1, kEnds = 2, kBad = 4, kEndOfList = 8, kFresh = 16, kHollow = 32 };

// Walks a range of the flat work list, in which an item takes PieceCost + tiles * TileCost
// units; tile k belongs to the range that holds the item's unit PieceCost + k * TileCost.
template <class S>
struct Walk {
  const TileArgs& A;
  int b, h, rb, n = 0, nd = 0, acc = 0;
  int off, left, per;
  Item it;
  int turns = 0, x = 0;
  int pass = 0;  // (key weights) the pass last given out
  bool more_passes = false, had = false;
  enum { kLoad, kStay, kAdvance } step = kLoad;
  __device__ __forceinline__ Walk(const TileArgs& a, const Start& s)
      : A(a), b(s.b), h(s.h), rb(s.rb), off(s.off), left(s.left), per(s.per) {}
  // The first tile at or past unit u of the item.
  __device__ __forceinline__ int tile_from(int u) const {
    return u <= S::PieceCost ? 0 : (u - S::PieceCost + S::TileCost - 1) / S::TileCost;
  }
  __device__ __forceinline__ bool has_pass(int k) const {
    return k < A.blocks && k * A.pos_block < acc + 1;
  }
  __device__ __forceinline__ bool next(Piece& p) {
    bool found = S::Weigh && more_passes;  // the same tiles for the next row block
    if (found) it = item_of<S::Weigh>(A, n, nd, acc, ++pass);
#pragma unroll 1
    while (!found) {
      if (left <= 0) return false;
      if (step != kStay) {
        bool load = step == kLoad;
        if (step == kAdvance) {
          off = 0;
          if (S::Weigh || ++rb == A.blocks) {
            rb = 0;
            if (++h == A.Hkv) {
              h = 0;
              ++b;
              load = true;
            }
          }
        }
        if (load) {
          n = load_n(A, b);
          nd = load_nd(A, b);
          acc = S::Weigh ? load_acc(A, b, nd) : 0;
        }
        it = item_of<S::Weigh>(A, n, nd, acc, rb);
      }
      const int rest = it.template cost<S>() - off, take = rest < left ? rest : left;
      const int ka = tile_from(off), kb = tile_from(off + take);
      step = take == rest ? kAdvance : kStay;
      if (kb > ka) {
        found = true;
        p.b = b;
        p.h = h;
        p.n = n;
        p.ta = it.t0 + ka;
        p.tb = it.t0 + kb;
        pass = 0;
        had = false;
        p.flags = (ka == 0 ? kStarts : 0) | (kb == it.tiles ? kEnds : 0) | (it.bad ? kBad : 0);
        // of an item that goes on in other CTAs: how many of the ranges, from this one on, hold
        // its tiles (the first lies at unit PieceCost of it)
        p.pieces = 1 + (per - left + S::PieceCost - off + (it.tiles - 1) * S::TileCost) / per;
      }
      off += take;
      left -= take;
    }
    p.i0 = it.i0;
    p.live = it.live;
    p.pos0 = it.pos0;
    p.first = it.first;
    p.last = it.last;
    p.ma = p.mb = 0;
    if (!it.bad && it.last >= it.first && it.last >= 0) {
      const int lo = it.first / kTileKeys, hi = it.last / kTileKeys + 1;
      p.ma = p.ta > lo ? p.ta : lo;
      p.mb = p.tb < hi ? p.tb : hi;
      if (p.mb < p.ma) p.mb = p.ma;
    }
    p.turn = turns;
    p.x0 = x;
    x += p.mb - p.ma;
    if (S::Weigh) {
      more_passes = !it.bad && has_pass(pass + 1);
      // (the next piece starts from the item of the first pass)
      if (!more_passes && pass > 0 && step == kStay) step = kLoad;
    }
    const bool busy = p.mb > p.ma;
    p.flags = (p.flags & ~(kFresh | kHollow)) | (had ? 0 : kFresh) |
              (busy || had || more_passes ? 0 : kHollow);
    turns += busy;
    had |= busy;
    return true;
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
#pragma unroll 1
  for (int b = b0; b < b1; ++b) mine += request_cost<S>(A, b) * A.Hkv;
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) scratch[warp] = incl;
  __syncthreads();
  int64_t before = 0, total = 0;
#pragma unroll 1
  for (int q = 0; q < kW; ++q) {
    if (q < warp) before += scratch[q];
    total += scratch[q];
  }
  incl += before;
  // (a range of TileCost units or more holds a tile of any item that spans it)
  const int wanted = total >> 31 ? (int)((total + gridDim.x - 1) / gridDim.x)
                                 : (int)(((unsigned)total + gridDim.x - 1) / gridDim.x);
  const int per = wanted < S::TileCost ? S::TileCost : wanted;
  const int64_t from = (int64_t)per * blockIdx.x;
  if (tid == 0) {
    s->per = per;
    s->left = from >= total ? 0 : (int)(total - from < per ? total - from : per);
  }
  if (from < total && incl - mine <= from && from < incl) {
    int64_t at = from - (incl - mine);
    int b = b0;
    int64_t t = 0;
#pragma unroll 1
    for (;; ++b, at -= t) {
      t = request_cost<S>(A, b) * A.Hkv;
      if (at < t) break;
    }
    const int n = load_n(A, b), nd = load_nd(A, b), acc = S::Weigh ? load_acc(A, b, nd) : 0;
    // the head, then the row block
    const int per_head = (int)(t / A.Hkv);
    s->b = b;
    s->h = (int)(at / per_head);
    int off = (int)(at - (int64_t)s->h * per_head), rb = 0;
#pragma unroll 1
    for (; !S::Weigh; ++rb) {
      const int cost = item_of<S::Weigh>(A, n, nd, acc, rb).template cost<S>();
      if (off < cost) break;
      off -= cost;
    }
    s->rb = rb;
    s->off = off;
  }
  __syncthreads();
}

// Pieces handed out and not yet taken by every role. Only pieces with tiles for the tensor cores are
// handed out, so the queue cannot stop the walk: the warp that copies the keys takes the next piece
// before it copies the last tile of the one at hand, X, and all it then waits for is that every role
// has taken the piece kPieceQueue - 1 before X, which needs no tile later than those of the piece
// ahead of X. (Any number of pieces without tiles may follow X: in the queue they would fill it while
// the other roles wait for X's last tile.)
constexpr int kPieceQueue = 8;

// ---- shared memory ------------------------------------------------------------------------------
template <class S>
struct TileShared {
  uint64_t full[S::NU], empty[S::NU];
  uint64_t q_full[S::NQ], q_empty[S::NQ];
  uint64_t s_full[S::Teams][2], s_empty[S::Teams][2];
  uint64_t p_full[S::Teams][S::NP], pv_done[S::Teams][S::NP];
  uint64_t v_ready[S::Teams];  // the values of a tile that some rows see in part have landed
  uint64_t o_done[2];  // a piece has its last product, by ordinal % 2
  uint32_t tmem;
  Waits waits;
  int hollow;  // the range holds pieces without tiles for the tensor cores
  int bad_piece[8];  // 1 + the ordinal of a piece with a page outside the pool, by ordinal % 8
  uint64_t drain[2];
  // the pieces, from the warp that walks the work list to the other roles
  Piece piece[kPieceQueue];
  uint64_t piece_full[kPieceQueue], piece_empty[kPieceQueue];
  int64_t scratch[16];
  Start start;
  struct Table {
    alignas(16) float m[S::N];       // lift - the running maximum, or minus the row's lse (log2)
    alignas(16) float slope[S::N];   // log2(e) * slope
    alignas(16) float ahead[S::N];   // the column's position less the block's first
    alignas(16) float alpha[S::N];
    alignas(16) float red[4][S::N];  // per-warp maxima or sums
    int hi[S::N], lo[S::N];          // the column sees keys j with lo < j <= hi
    int row[S::N];                   // output row of the column, from the item's first
    Piece piece;                     // whose columns these are (its end reads it from here)
    int odd;                         // a partly visible key has values that are not finite
  } table[2];                        // by ordinal % 2 (with two teams: one each)
  JoinItem join;
};

// A place in a ring of n units whose barriers start at full[base], and the parity of its use.
struct RingPos {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int n) {
    if (++slot == n) {
      slot = 0;
      phase ^= 1u;
    }
  }
};
// Where the c-th unit of the values of the CTA's x-th tile lies.
template <class S>
__device__ __forceinline__ int value_slot(int x, int c) {
  return S::NK + (x * S::U + c) % S::NV;
}

// The i-th tile a piece walks: the attention goes from the newest keys to the oldest, so that
// a bias by distance (or plain recency) puts the maximum into the first tile.
template <class S>
__device__ __forceinline__ int tile_at(const Piece& p, int i) {
  return S::Weigh ? p.ma + i : p.mb - 1 - i;
}

// Keys from here on are inside the window of every row of a piece.
__device__ __forceinline__ int first_full(const Piece& p, int window) {
  return p.last - window + 1;
}
// Whether some row of the piece does not see some key of tile t.
__device__ __forceinline__ bool edge_tile(const Piece& p, int window, int t) {
  return t * kTileKeys < first_full(p, window) || t * kTileKeys + kTileKeys - 1 > p.pos0;
}

// How the other roles take the pieces: every one in turn, none left out (a reader that skipped
// some could not tell a phase of a barrier from the one after next).
template <class S>
struct Reader {
  TileShared<S>& sh;
  RingPos at;
  __device__ __forceinline__ explicit Reader(TileShared<S>& s) : sh(s) {}
  __device__ __forceinline__ const Piece& wait() {
    wait_phase(&sh.piece_full[at.slot], at.phase, &sh.waits);
    return sh.piece[at.slot];
  }
  // One thread of each role (of the softmax, of each warp) gives the place back.
  __device__ __forceinline__ void release(bool mine) {
    if (mine) mbar_arrive(&sh.piece_empty[at.slot]);
    at.next(kPieceQueue);
  }
  // Takes the next piece, by one thread or (kWarp) by a whole warp; false at the end of the list
  // or when the CTA has given up.
  template <bool kWarp>
  __device__ __forceinline__ bool next(Piece& p) {
    p = wait();
    bool end = *(volatile int*)&sh.waits.dead || (p.flags & kEndOfList);
    if (kWarp) end = __any_sync(0xffffffffu, end);  // (and every lane has read the piece)
    if (end) return false;
    release(!kWarp || (threadIdx.x & 31) == 0);
    return true;
  }
};

// ---- the copying warps ------------------------------------------------------------------------
// Whether some row sees a key of the lane's group of `box` keys in a tile, and that group's page
// (not looked at here: the load is a tile ahead of its use).
__device__ __forceinline__ bool group_seen(const TileArgs& A, const Piece& p, int tile, int lane) {
  const int j = tile * kTileKeys + lane * A.box;
  return lane * A.box < kTileKeys && j <= p.last && j + A.box - 1 >= p.first;
}
__device__ __forceinline__ int group_page(const TileArgs& A, const Piece& p, int tile, int lane) {
  const int j = tile * kTileKeys + lane * A.box;
  return __ldg(A.table + (int64_t)p.b * A.max_pages + (j >> A.log_page));
}

// One warp walks the work list, hands out the pieces and copies the keys (and the queries) of
// their tiles; another copies the values. Each lane starts the copies of its group of keys; the
// pages of the next tile are looked up a tile ahead. (All roles' loops are kept short and rolled:
// together they have to stay in the instruction cache, whose misses are latency of every tile.)
template <class S, bool kValues>
__device__ __forceinline__ void copy_role(const TileArgs& A, TileShared<S>& sh,
                                          unsigned char* qbuf, unsigned char* ring,
                                          const CUtensorMap* mq, const CUtensorMap* map) {
  constexpr int kBase = kValues ? S::NK : 0, kUnits = kValues ? S::NV + S::Weigh : S::NK;
  const int lane = threadIdx.x & 31;
  unsigned char* dst = ring + kBase * kUnitBytes + lane * A.box * 128;
  Walk<S> walk(A, sh.start);
  Reader<S> reader(sh);
  // the next piece with tiles for the tensor cores; all lanes
  bool hollow = false;
  auto take = [&](Piece& p) -> bool {
    if (kValues) return reader.template next<true>(p);
    bool more;
#pragma unroll 1
    while ((more = walk.next(p)) && p.mb == p.ma) hollow |= (p.flags & kHollow) != 0;
    if (!more) p.flags = kEndOfList;
    bool ok = wait_phase(&sh.piece_empty[reader.at.slot], reader.at.phase ^ 1u, &sh.waits);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) return false;
    if (lane == 0) {
      sh.hollow = hollow;
      sh.piece[reader.at.slot] = p;
      mbar_arrive(&sh.piece_full[reader.at.slot]);
    }
    reader.at.next(kPieceQueue);
    return more;
  };
  Piece p;
  bool more = take(p);
  int i = 0;
  bool seen = more && group_seen(A, p, tile_at<S>(p, 0), lane);
  int page = seen ? group_page(A, p, tile_at<S>(p, 0), lane) : 0;
  RingPos at;
  int issued = 0, q_issued = 0;
#pragma unroll 1
  while (more) {
    const int head = p.h, turn = p.turn;
    const int slot = (tile_at<S>(p, i) * kTileKeys + lane * A.box) & ((1 << A.log_page) - 1);
    if (!kValues && i == 0) {
      const int qs = turn % S::NQ;
      if (!__all_sync(0xffffffffu, wait_phase(&sh.q_empty[qs], ((uint32_t)(turn / S::NQ) & 1u) ^ 1u,
                                              &sh.waits)))
        goto end;
      if (lane == 0) {
        mbar_arrive_expect_tx(&sh.q_full[qs], (uint32_t)(A.G * A.pos_block * S::D * 2));
#pragma unroll 1
        for (int c = 0; c < S::U; ++c)
          tile_g2s(qbuf + qs * S::QBytes + c * S::N * 128, mq, &sh.q_full[qs], c * 64,
                   head * A.G, p.i0, p.b);
      }
      ++q_issued;
      __syncwarp();
    }
    if (__builtin_expect(++i == p.mb - p.ma, 0)) {
      more = take(p);
      i = 0;
    }
    const bool next_seen = more && group_seen(A, p, tile_at<S>(p, i), lane);
    const int next_page = next_seen ? group_page(A, p, tile_at<S>(p, i), lane) : 0;
    const bool mine = seen && page >= 0 && page < A.num_pages;
    if (!kValues) {
      if (__builtin_expect(__any_sync(0xffffffffu, seen && !mine), 0) && lane == 0)
        *(volatile int*)&sh.bad_piece[turn & 7] = turn + 1;
    }
    const uint32_t bytes =
        (uint32_t)(__popc(__ballot_sync(0xffffffffu, mine)) * A.box) * 128u;
#pragma unroll 1
    for (int c = 0; c < S::U; ++c) {
      uint64_t* full = &sh.full[kBase + at.slot];
      if (!__all_sync(0xffffffffu, wait_phase(&sh.empty[kBase + at.slot], at.phase ^ 1u, &sh.waits)))
        goto end;
      if (lane == 0) mbar_arrive_expect_tx(full, bytes);
      ++issued;
      __syncwarp();
      if (mine) tile_g2s(dst + at.slot * kUnitBytes, map, full, c * 64, slot, head, page);
      at.next(kUnits);
    }
    page = next_page;
    seen = next_seen;
  }
end:
  if (lane == 0) {
    // no copy may outlive the CTA, should the others give up before they have seen it land
#pragma unroll 1
    for (int u = issued > kUnits ? issued - kUnits : 0; u < issued; ++u)
      mbar_wait(&sh.full[kBase + u % kUnits], (uint32_t)(u / kUnits) & 1u, kTileWaitNs);
#pragma unroll 1
    for (int u = q_issued > S::NQ ? q_issued - S::NQ : 0; u < q_issued; ++u)
      mbar_wait(&sh.q_full[u % S::NQ], (uint32_t)(u / S::NQ) & 1u, kTileWaitNs);
  }
  __syncwarp();
}

// ---- the threads that issue the matrix instructions -------------------------------------------
// One issues the scores, as far ahead as their buffers allow, one the products with the values.
// One whose wait failed issues nothing any more (what it then waits for is not what its loop is at).
// At the end each waits for its own: no instruction may outlive the tensor memory, should the others
// give up before they have seen it finish.
template <class S>
__device__ __forceinline__ void drain(TileShared<S>& sh, int which) {
  mma_commit(&sh.drain[which]);
  mbar_wait(&sh.drain[which], 0, kTileWaitNs);
}

// S^T = K Q^T of every tile.
template <class S>
__device__ __forceinline__ void score_role(const TileArgs& A, TileShared<S>& sh,
                                           unsigned char* qbuf, unsigned char* ring) {
  const uint32_t idesc = mma_desc(A.bf16, false, false, 128, S::N);
  const uint64_t rows = smem_desc(0, 16, 1024, kSwizzle128);
  const uint64_t a0 = rows + (smem_u32(ring) >> 4), b0 = rows + (smem_u32(qbuf) >> 4);
  Reader<S> reader(sh);
  RingPos at;
  int used[2] = {0, 0};  // tiles so far per team (attention) or per score buffer (key weights)
  Piece p;
#pragma unroll 1
  while (reader.template next<false>(p)) {
    const int qs = p.turn % S::NQ, team = p.turn % S::Teams, tiles = p.mb - p.ma;
    if (!wait_phase(&sh.q_full[qs], (uint32_t)(p.turn / S::NQ) & 1u, &sh.waits)) goto end;
#pragma unroll 1
    for (int i = 0; i < tiles; ++i) {
      const int of = S::Weigh ? tile_at<S>(p, i) & 1 : team;
      const int y = of ? used[1]++ : used[0]++;
      const int buf = S::Weigh ? of : y & 1, turn = S::Weigh ? y : y >> 1;
      if (!wait_phase(&sh.s_empty[team][buf], ((uint32_t)turn & 1u) ^ 1u, &sh.waits)) goto end;
      tc_fence_after();
      const uint32_t d = sh.tmem + (2 * team + buf) * S::N;
      uint64_t b = b0 + qs * (S::QBytes >> 4);
#pragma unroll 1
      for (int c = 0; c < S::U; ++c, b += S::N * 8) {
        if (!wait_phase(&sh.full[at.slot], at.phase, &sh.waits)) goto end;
        tc_fence_after();
        const uint64_t a = a0 + at.slot * (kUnitBytes >> 4);
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_f16(d, a + 2 * k, b + 2 * k, idesc, c > 0 || k > 0);
        mma_commit(&sh.empty[at.slot]);
        at.next(S::NK);
      }
      mma_commit(&sh.s_full[team][buf]);
    }
    mma_commit(&sh.q_empty[qs]);
  }
end:
  drain<S>(sh, 0);
}

// O^T (+)= V^T P^T of every tile. Of an edge tile the softmax threads clean the values once they
// have landed, before they pass on the weights.
template <class S>
__device__ __forceinline__ void value_role(const TileArgs& A, TileShared<S>& sh,
                                           unsigned char* pbuf, unsigned char* ring) {
  constexpr int kPer = S::U >= 2 ? 2 : 1;  // units per accumulator
  const uint32_t idesc = mma_desc(A.bf16, true, true, 128, S::ON);
  // values of 64 columns lie 128 bytes per key; with D = 64 both halves of the instruction's rows
  // read the same columns, and the upper half is not used
  const uint64_t a0 = smem_desc(0, kPer == 2 ? kUnitBytes : 0, 1024, kSwizzle128) +
                      ((smem_u32(ring) + S::NK * kUnitBytes) >> 4);
  const uint64_t b0 = smem_desc(0, kTileKeys * 32, 256, kSwizzle32) + (smem_u32(pbuf) >> 4);
  Reader<S> reader(sh);
  RingPos at;
  int used[2] = {0, 0};
  Piece p;
#pragma unroll 1
  while (reader.template next<false>(p)) {
    const int team = p.turn % S::Teams, tiles = p.mb - p.ma;
    const uint32_t o = sh.tmem + 2 * S::Teams * S::N + (p.turn & 1) * S::MBlocks * S::ON;
#pragma unroll 1
    for (int i = 0; i < tiles; ++i) {
      const int y = team ? used[1]++ : used[0]++, pb = y % S::NP;
      if (__builtin_expect(edge_tile(p, A.rule.window, tile_at<S>(p, i)), 0)) {
        RingPos look = at;
#pragma unroll 1
        for (int c = 0; c < S::U; ++c) {
          if (!wait_phase(&sh.full[S::NK + look.slot], look.phase, &sh.waits)) goto end;
          look.next(S::NV);
        }
        mbar_arrive(&sh.v_ready[team]);
      }
      if (!wait_phase(&sh.p_full[team][pb], (uint32_t)(y / S::NP) & 1u, &sh.waits)) goto end;
      const uint64_t b = b0 + (team * S::NP + pb) * (S::PBytes >> 4);
      uint32_t d = o;
#pragma unroll 1
      for (int m = 0; m < S::MBlocks; ++m, d += S::ON) {
        const uint64_t a = a0 + at.slot * (kUnitBytes >> 4);
        uint64_t* empty = &sh.empty[S::NK + at.slot];
#pragma unroll 1
        for (int c = 0; c < kPer; ++c) {
          if (!wait_phase(&sh.full[S::NK + at.slot], at.phase, &sh.waits)) goto end;
          at.next(S::NV);
        }
        tc_fence_after();
#pragma unroll 1
        for (int part = 0; part < (S::Wide ? 1 : S::Parts); ++part)  // the weights' parts
#pragma unroll 4
          for (int k = 0; k < kTileKeys / 16; ++k)
            mma_f16(d, a + k * 128, b + part * (kTileKeys * S::N * 2 >> 4) + k * 32, idesc,
                    !(i == 0 && part == 0 && k == 0));
#pragma unroll
        for (int c = 0; c < kPer; ++c) mma_commit(empty + c);  // (a pair lies side by side)
      }
      mma_commit(&sh.pv_done[team][pb]);
    }
    mma_commit(&sh.o_done[p.turn & 1]);
  }
end:
  drain<S>(sh, 1);
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
// Two floats in one 64-bit register: one instruction for both.
using Two = unsigned long long;
__device__ __forceinline__ Two two(float a, float b) {
  Two v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
  return v;
}
__device__ __forceinline__ float2 split(Two v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ Two two_fma(Two a, Two b, Two c) {
  Two v;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
  return v;
}
__device__ __forceinline__ Two two_add(Two a, Two b) {
  Two v;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
  return v;
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
  if (__builtin_expect(r.softcap > 0.0f, 0)) {
    // c tanh(y) = c - 2 c / (1 + 2^(2 log2(e) y)); below |y| = 1/8, where that cancels, the series
    // y (1 - y^2/3 + 2 y^4/15), off by y^6 / 18 (2^-22)
    const float in = scale2 / r.softcap * kLn2, c2 = r.softcap * kLog2e;
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      const float y = s[c] * in, y2 = y * y;
      const float far = fmaf(-2.0f * c2, rcp_fast(1.0f + ex2(y * (2.0f * kLog2e))), c2);
      const float near = s[c] * scale2 * fmaf(y2, fmaf(y2, 2.0f / 15.0f, -1.0f / 3.0f), 1.0f);
      s[c] = y2 < 1.0f / 64.0f ? near : far;
    }
  } else {
#pragma unroll
    for (int c = 0; c < kC; ++c) s[c] *= scale2;
  }
  if (__builtin_expect(r.slopes != nullptr, 0)) {
#pragma unroll
    for (int c = 0; c < kC; ++c) s[c] = fmaf(-slope[c], away + ahead[c], s[c]);
  }
}

// The tables of a piece's columns, by thread `me` of `all` (barriers around it are the caller's).
template <class S>
__device__ __forceinline__ void set_columns(const TileArgs& A, typename TileShared<S>::Table& T,
                                            const Piece& p, int me, int all) {
#pragma unroll 1
  for (int c = me; c < S::N; c += all) {
    const int i = c / A.G, g = c - i * A.G;
    const bool live = i < p.live;
    const int pos = p.pos0 + i;
    T.slope[c] = live && A.rule.slopes ? __ldg(A.rule.slopes + p.h * A.G + g) * kLog2e : 0.0f;
    T.ahead[c] = (float)i;
    T.hi[c] = live ? pos : -1;
    T.lo[c] = pos - A.rule.window;
    T.row[c] = i * A.Hq + g;
    if (S::Weigh) {
      // a row that does not count, or one of no weight, gets none from any key
      float l = INFINITY;
      if (live) {
        const float v = __ldg(A.lse + p.b * A.lse_req + (p.i0 + i) * A.lse_row +
                              (p.h * A.G + g) * A.lse_head);
        if (v != -INFINITY) l = v * kLog2e;
      }
      T.m[c] = -l;
    } else {
      T.m[c] = live ? -kNoMax : kNoMax;  // (a column without a row never rises)
    }
  }
}

template <bool kBf16>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  if (kBf16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <bool kBf16>
__device__ __forceinline__ float2 unpack16(uint32_t w) {
  if (kBf16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <bool kBf16>
__device__ __forceinline__ void store16(void* base, int64_t at, float x) {
  static_cast<uint16_t*>(base)[at] = (uint16_t)pack16<kBf16>(x, 0.0f);
}
// Nonzero where one of two 16-bit values is infinite or NaN: its exponent field carries into
// the sign's place.
template <bool kBf16>
__device__ __forceinline__ uint32_t not_finite2(uint32_t w) {
  return kBf16 ? ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u
               : ((w & 0x7c007c00u) + 0x04000400u) & 0x80008000u;
}

// Named barriers: 1 and 2 for the two groups of softmax warps, 3 for all of them.
constexpr int kAllBar = 3;

// The log-sum-exp of a row from m (its maximum less the lift) and its lifted sum.
template <bool kBf16>
__device__ __forceinline__ float row_lse(float m, float sum) {
  constexpr float kLift = TileShape<64, 16, false, kBf16>::Lift;
  if (sum == 0.0f) return -INFINITY;
  return (m + kLift + log2f(kBf16 ? sum : sum * 0.0078125f)) * (1.0f / kLog2e);
}

struct ValuePool {
  const void* data;
  int64_t page, token, head;
};

// The outputs of a piece that values make infinite or NaN. In the tensor cores such a value meets
// weights of 0: the low half of an exact weight, or a weight that is too small for its type. So the
// values of the piece's keys that are not finite are summed here, for one thread's share of D: those
// of the keys that all rows see, and for each row of its columns those of the others it sees. What
// comes out not finite is the row's output (times a positive weight, and plus finite numbers, it is
// the same); a row whose values are finite keeps what it has.
template <class S>
__device__ __noinline__ void special_values(const TileArgs& A, const ValuePool& vpool,
                                            const typename TileShared<S>::Table& T, int b, int h,
                                            int pos0, int first, int last, int ma, int mb, int col0,
                                            int rows, int d0, float* part, int64_t row0) {
  const int j0 = first > ma * kTileKeys ? first : ma * kTileKeys;
  const int j1 = last < mb * kTileKeys - 1 ? last : mb * kTileKeys - 1;
  // keys [f0, f1] are seen by all rows; where there are none, [j0, j1] are all looked at row by row
  int f0 = last - A.rule.window + 1 > j0 ? last - A.rule.window + 1 : j0, f1 = pos0 < j1 ? pos0 : j1;
  if (f0 > f1) f0 = j1 + 1, f1 = j1;
#pragma unroll 1
  for (int d = d0; d < S::D; d += 128) {
    auto odd_part = [&](int j) {  // the value if it is not finite, else 0
      const int page = __ldg(A.table + (int64_t)b * A.max_pages + (j >> A.log_page));
      if (page < 0 || page >= A.num_pages) return 0.0f;
      const int64_t at = page * vpool.page + (j & ((1 << A.log_page) - 1)) * vpool.token +
                         h * vpool.head + d;
      const float v = unpack16<S::Bf16>(__ldg(static_cast<const unsigned short*>(vpool.data) + at)).x;
      return isfinite(v) ? 0.0f : v;
    };
    float all = 0.0f;
#pragma unroll 8
    for (int j = f0; j <= f1; ++j) all += odd_part(j);
#pragma unroll 1
    for (int n = col0; n < col0 + S::NC && n < rows; ++n) {
      if (T.red[0][n] == 0.0f) continue;
      float sum = all;
#pragma unroll 1
      for (int j = j0; j <= j1; ++j) {
        if (j == f0) j = f1 + 1;
        if (j <= j1 && j <= T.hi[n] && j > T.lo[n]) sum += odd_part(j);
      }
      if (isfinite(sum)) continue;
      if (part)
        part[n * S::D + d] = sum;
      else
        store16<S::Bf16>(A.out, (row0 + T.row[n]) * S::D + d, sum);
    }
  }
}

// ---- attention --------------------------------------------------------------------------------
// What one softmax thread does for the attention: its key of every tile, its share of O.
template <class S>
struct Attend {
  using Table = typename TileShared<S>::Table;
  const TileArgs& A;
  const ValuePool& vpool;
  TileShared<S>& sh;
  unsigned char *pbuf, *ring;
  int lane, quarter, group, key;
  uint32_t lane_base;  // tensor-memory address of the thread's lanes
  int team, me;        // the team, the thread's index in it
  int col0;            // the group's first column
  int edges = 0;       // edge tiles so far

  // Wait until the products of the team's tile y have read P and are in O.
  __device__ __forceinline__ void wait_values(int y) const {
    wait_phase(&sh.pv_done[team][y % S::NP], (uint32_t)(y / S::NP) & 1u, &sh.waits);
  }
  __device__ __forceinline__ void group_sync() const { bar_sync(1 + group, 128); }
  __device__ __forceinline__ void team_sync() const {
    bar_sync(S::Teams == 2 ? 1 + group : kAllBar, S::TeamThreads);
  }
  // The accumulator of a piece, the group's first column.
  __device__ __forceinline__ uint32_t output(int turn) const {
    return lane_base + 2 * S::Teams * S::N + (turn & 1) * S::MBlocks * S::ON + col0;
  }

  // Raise the maxima of the CH columns from c0 to those of this tile's scores s, and scale what
  // those columns hold.
  __device__ __forceinline__ void raise(Table& T, const float (&s)[S::CH], Two (&l)[S::NC / 2],
                                        int k, bool first, uint32_t o_base) {
    const int c0 = col0 + k;
    column_reduce<S::CH, true>(s, &T.red[quarter][c0], lane);
    group_sync();
    if (quarter == 0 && lane < S::CH) {
      const int c = c0 + lane;
      const float was = -T.m[c];
      const float top = fmaxf(fmaxf(T.red[0][c], T.red[1][c]), fmaxf(T.red[2][c], T.red[3][c]));
      const float m = fmaxf(top - S::Lift, was);
      T.alpha[c] = ex2(was - m);
      T.m[c] = -m;
    }
    group_sync();
    if (first) return;
#pragma unroll
    for (int c = 0; c < S::CH; c += 2) {
      const float2 v = split(l[(k + c) / 2]);
      l[(k + c) / 2] = two(v.x * T.alpha[c0 + c], v.y * T.alpha[c0 + c + 1]);
    }
    tc_fence_after();
#pragma unroll 1
    for (int m = 0; m < S::MBlocks * (S::Wide ? S::Parts : 1); ++m)  // (wide: a product per part)
#pragma unroll 1
      for (int q = 0; q < S::CH; q += 16) {
        float o[16];
        const uint32_t at = o_base + m * S::N + k + q;
        tmem_ld16(at, o);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 16; ++c) o[c] *= T.alpha[c0 + q + c];
        tmem_st16(at, o);
      }
    tmem_wait_st();
  }

  // Values of keys that some row of a tile does not see: what no row sees becomes 0; of a key
  // that only some rows see, the values that are not finite become 0 (times a weight of 0 they would
  // reach the others) and special_values adds them at the end to the rows that see it.
  __device__ __forceinline__ void clean_values(Table& T, const Piece& p, int x, int j) {
    const bool none = j > p.last || j < p.first;
    const bool some = !none && (j > p.pos0 || j < first_full(p, A.rule.window));
    if (!__any_sync(0xffffffffu, none || some)) return;
    uint32_t odd = 0;
#pragma unroll 1
    for (int c = 0; c < S::U; ++c) {
      uint4* row = reinterpret_cast<uint4*>(ring + value_slot<S>(x, c) * kUnitBytes + key * 128);
      // (each lane starts with another 16 bytes of its row: no bank conflicts)
      if (none) {
#pragma unroll
        for (int q = 0; q < 8; ++q) row[(q + lane) & 7] = make_uint4(0u, 0u, 0u, 0u);
      } else if (some) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const uint4 v = row[(q + lane) & 7];
          odd |= not_finite2<S::Bf16>(v.x) | not_finite2<S::Bf16>(v.y) |
                 not_finite2<S::Bf16>(v.z) | not_finite2<S::Bf16>(v.w);
        }
      }
    }
    if (odd) {
      *(volatile int*)&T.odd = 1;
#pragma unroll 1
      for (int c = 0; c < S::U; ++c) {
        uint32_t* w = reinterpret_cast<uint32_t*>(ring + value_slot<S>(x, c) * kUnitBytes +
                                                  key * 128);
#pragma unroll 1
        for (int e = 0; e < 32; ++e) {
          const uint32_t bad = not_finite2<S::Bf16>(w[e]);
          if (bad) w[e] &= ~((bad >> 15) * 0xffffu);
        }
      }
    }
  }

  // One tile, the CTA's x-th and the team's y-th: its scores, their weights into shared memory.
  // (What most tiles do is kept short: it has to stay in the instruction cache beside the other
  // roles' loops.)
  __device__ __forceinline__ void tile(Table& T, const Piece& p, int t, bool first, int x, int y,
                                       Two (&l)[S::NC / 2]) {
    const int buf = y & 1, j = t * kTileKeys + key;
    const bool edge = edge_tile(p, A.rule.window, t);
    unsigned char* const pb =
        pbuf + (team * S::NP + y % S::NP) * S::PBytes + col0 / 16 * (kTileKeys * 32) + key * 32;
    wait_phase(&sh.s_full[team][buf], (uint32_t)(y >> 1) & 1u, &sh.waits);
    tc_fence_after();
#pragma unroll
    for (int k = 0; k < S::NC; k += S::CH) {
      const int c0 = col0 + k;
      float s[S::CH];
      float scale = A.rule.scale * kLog2e;  // to what the thread holds in s
#pragma unroll
      for (int q = 0; q < S::CH; q += 16)
        tmem_ld16(lane_base + (2 * team + buf) * S::N + c0 + q,
                  reinterpret_cast<float(&)[16]>(s[q]));
      tmem_wait_ld();
      if (k + S::CH == S::NC) {
        tc_fence_before();
        mbar_arrive(&sh.s_empty[team][buf]);
      }
      if (__builtin_expect(edge || A.rule.softcap > 0.0f || A.rule.slopes, 0)) {
        apply_rule<S::CH>(s, A.rule, (float)(p.pos0 - j), &T.slope[c0], &T.ahead[c0]);
        scale = 1.0f;
        if (edge) {
#pragma unroll
          for (int c = 0; c < S::CH; ++c)
            if (j > T.hi[c0 + c] || j <= T.lo[c0 + c]) s[c] = -INFINITY;
        }
      }
      Two e[S::CH / 2];
      auto exponents = [&]() {
        const Two sc = two(scale, scale);
#pragma unroll
        for (int c = 0; c < S::CH; c += 4) {
          const float4 m = *reinterpret_cast<const float4*>(&T.m[c0 + c]);
          e[c / 2] = two_fma(two(s[c], s[c + 1]), sc, two(m.x, m.y));
          e[c / 2 + 1] = two_fma(two(s[c + 2], s[c + 3]), sc, two(m.z, m.w));
        }
      };
      exponents();
      float top = -INFINITY;
#pragma unroll
      for (int c = 0; c < S::CH / 2; ++c) {
        const float2 v = split(e[c]);
        top = fmaxf(top, fmaxf(v.x, v.y));
      }
      if (__builtin_expect(bar_or(1 + group, 128, top > 8.0f + S::Lift), 0)) {
        if (!first) wait_values(y - 1);
#pragma unroll
        for (int c = 0; c < S::CH; ++c) s[c] *= scale;
        scale = 1.0f;
        raise(T, s, l, k, first, output(p.turn));
        exponents();
      }
      uint32_t w16[S::Parts][S::CH / 2];
#pragma unroll
      for (int c = 0; c < S::CH / 2; ++c) {
        const float2 v = split(e[c]);
        const float a = ex2(v.x), b = ex2(v.y);
        Two w = two(a, b);  // what the parts so far leave of the weights
        l[k / 2 + c] = two_add(l[k / 2 + c], w);
#pragma unroll
        for (int part = 0; part < S::Parts; ++part) {
          const float2 r = split(w);
          w16[part][c] = pack16<S::Bf16>(r.x, r.y);
          const float2 h = unpack16<S::Bf16>(w16[part][c]);
          if (part + 1 < S::Parts) w = two_fma(two(h.x, h.y), two(-1.0f, -1.0f), w);
        }
      }
      // the product that last read this buffer
      if (k == 0 && y >= S::NP) wait_values(y - S::NP);
#pragma unroll
      for (int q = 0; q < S::CH; q += 16) {
        // 16 columns of a key: 32 bytes, their 16-byte halves swapped in every other 4 keys
        unsigned char* at = pb + (k + q) / 16 * (kTileKeys * 32);
        const int sw = ((key >> 2) & 1) * 16, w = q / 2;
#pragma unroll
        for (int part = 0; part < S::Parts; ++part, at += kTileKeys * S::N * 2) {
          const uint32_t* v = &w16[part][w];
          *reinterpret_cast<uint4*>(at + sw) = make_uint4(v[0], v[1], v[2], v[3]);
          *reinterpret_cast<uint4*>(at + (16 - sw)) = make_uint4(v[4], v[5], v[6], v[7]);
        }
      }
    }
    if (__builtin_expect(edge, 0)) {
      wait_phase(&sh.v_ready[team], (uint32_t)(edges++) & 1u, &sh.waits);
      if (S::Teams == 2 || group == 0) clean_values(T, p, x, j);
    }
    fence_proxy_async();
    tc_fence_before();
    mbar_arrive(&sh.p_full[team][y % S::NP]);
  }

  // Output row of a piece's first column.
  __device__ __forceinline__ int64_t first_row(const Piece& p) const {
    return ((int64_t)p.b * A.P + p.i0) * A.Hq + p.h * A.G;
  }

  // The end of a piece (its sums' warp parts are in T.red): O and the sums leave for the output
  // or for the workspace.
  __device__ __forceinline__ void finish(Table& T) {
    const Piece& p = T.piece;
    group_sync();
    const bool poison = *(volatile int*)&sh.bad_piece[p.turn & 7] == p.turn + 1;
    const bool starts = p.flags & kStarts, whole = starts && (p.flags & kEnds);
    const int rows = p.live * A.G;
    const int64_t row0 = first_row(p);
    float* part =
        A.part + (2 * (int64_t)blockIdx.x + (starts ? 1 : 0)) * (S::N * (S::D + 2));
    if (quarter == 0) {
#pragma unroll 1
      for (int c = col0 + lane; c < col0 + S::NC; c += 32) {
        float sum = (T.red[0][c] + T.red[1][c]) + (T.red[2][c] + T.red[3][c]);
        if (poison) sum = __uint_as_float(0x7fc00000u);
        const float m = -T.m[c];
        if (c < rows) {
          if (!whole)
            *reinterpret_cast<float2*>(part + S::N * S::D + 2 * c) = make_float2(m, sum);
          else if (A.out_lse)
            A.out_lse[row0 + T.row[c]] =
                row_lse<S::Bf16>(m, sum);
        }
        T.alpha[c] = !whole ? 1.0f : sum == 0.0f ? 0.0f : rcp_fast(sum);
        T.red[0][c] = c < rows && sum == sum ? 1.0f : 0.0f;  // its output is a number unless a value is not
      }
    }
    if (me == 0 && starts && !whole) {
      sh.join.pieces = p.pieces;
      sh.join.row0 = row0;
      sh.join.rows = rows;
    }
    group_sync();
    wait_phase(&sh.o_done[p.turn & 1], (uint32_t)(p.turn >> 1) & 1u, &sh.waits);
    tc_fence_after();
    if (S::D >= 128 || quarter < 2) {
      int d = quarter * 32 + lane;
      float odd = *(volatile int*)&T.odd ? __uint_as_float(0x7fc00000u) : 0.0f;
#pragma unroll 1
      for (int m = 0; m < S::MBlocks; ++m, d += 128)
#pragma unroll 1
        for (int q = 0; q < S::NC && col0 + q < rows; q += 16) {
          float o[16];
          tmem_ld16(output(p.turn) + m * S::ON + q, o);
          tmem_wait_ld();
          if (S::Wide) {
#pragma unroll 1
            for (int part = 1; part < S::Parts; ++part) {
              float low[16];
              tmem_ld16(output(p.turn) + m * S::ON + part * S::N + q, low);
              tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < 16; ++c) o[c] += low[c];
            }
          }
          const int n0 = col0 + q;
          float all = 0.0f;
#pragma unroll
          for (int c = 0; c < 16; ++c) all = fmaf(o[c], T.red[0][n0 + c], all);
          odd = fmaf(all, 0.0f, odd);  // (NaN from here on if one of them is not finite)
          if (whole) {
            uint16_t* out = static_cast<uint16_t*>(A.out) + row0 * S::D + d;
#pragma unroll
            for (int c = 0; c < 16; c += 2) {
              const uint32_t w =
                  pack16<S::Bf16>(o[c] * T.alpha[n0 + c], o[c + 1] * T.alpha[n0 + c + 1]);
              if (n0 + c < rows) out[T.row[n0 + c] * S::D] = (uint16_t)w;
              if (n0 + c + 1 < rows) out[T.row[n0 + c + 1] * S::D] = (uint16_t)(w >> 16);
            }
          } else {
#pragma unroll
            for (int c = 0; c < 16; ++c)
              if (n0 + c < rows) part[(n0 + c) * S::D + d] = o[c];
          }
        }
      if (__builtin_expect(odd != odd && !poison, 0))
        special_values<S>(A, vpool, T, p.b, p.h, p.pos0, p.first, p.last, p.ma, p.mb, col0, rows,
                          quarter * 32 + lane, whole ? nullptr : part, row0);
    }
    tc_fence_before();
  }

  // The pieces in turn. With one team the end of a piece waits until the first tile of the next
  // one is in the tensor cores' hands, so that its last product, and its output, pass under that
  // tile; with two the other team's tiles cover it.
  __device__ __forceinline__ void run() {
    Reader<S> reader(sh);
    Piece p{};
    int y = 0, i = 0, ended = 0;
    bool pending = false;
    Two l[S::NC / 2];
    auto table = [&](int turn) -> Table& { return sh.table[S::Teams == 2 ? team : turn & 1]; };
#pragma unroll 1
    for (;;) {
      const bool flush = S::Teams == 2 && pending;  // the end first
      bool more = true;
      if (!flush) {
        if (__builtin_expect(i == p.mb - p.ma, 0)) {
#pragma unroll 1
          for (;;) {
            p = reader.wait();
            more = !(p.flags & kEndOfList) && !*(volatile int*)&sh.waits.dead;
            more = !bar_or(1 + group, 128, !more);
            if (S::Teams == 1) more = !bar_or(kAllBar, S::SoftThreads, !more);
            if (!more) break;
            reader.release(lane == 0);
            if (p.turn % S::Teams == team) break;
          }
          if (more) {
            Table& T = table(p.turn);
            team_sync();  // the last piece with this table is out of it
            set_columns<S>(A, T, p, me, S::TeamThreads);
            if (me == 0) T.piece = p, T.odd = 0;
            team_sync();
            i = 0;
          }
#pragma unroll
          for (int c = 0; c < S::NC / 2; ++c) l[c] = 0ull;
        }
        if (more) {
          tile(table(p.turn), p, tile_at<S>(p, i), i == 0, p.x0 + i, y, l);
          ++i;
          ++y;
        }
      }
      if (pending) {
        finish(table(ended));
        pending = false;
      }
      if (!more) break;
      if (!flush && i == p.mb - p.ma) {
        float sums[S::NC];
#pragma unroll
        for (int c = 0; c < S::NC; c += 2) {
          const float2 v = split(l[c / 2]);
          sums[c] = v.x;
          sums[c + 1] = v.y;
        }
        column_reduce<S::NC, false>(sums, &table(p.turn).red[quarter][col0], lane);
        ended = p.turn;
        pending = true;
      }
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
  auto& T = sh.table[0];
  Reader<S> reader(sh);
  Piece p;
  int used = 0;  // tiles this group has taken from its S buffer
#pragma unroll 1
  for (;;) {
    p = reader.wait();
    bool more = !(p.flags & kEndOfList) && !*(volatile int*)&sh.waits.dead;
    more = !bar_or(kAllBar, S::SoftThreads, !more);  // (the last piece's tables have been read)
    if (!more) return;
    reader.release(lane == 0);
    const int64_t row = ((int64_t)p.b * A.Hkv + p.h) * A.stride;
    float* out = A.weights + row;
    const float* prior = A.prior ? A.prior + row : nullptr;
    // the first pass that has tiles here writes every tile of the piece, later ones add to theirs
    const bool fresh = p.flags & kFresh;
    {
      set_columns<S>(A, T, p, threadIdx.x, S::SoftThreads);
      bar_sync(kAllBar, S::SoftThreads);
      const int ta = fresh ? p.ta : p.ma, tb = fresh ? p.tb : p.mb;
      // the columns from here on are of rows that do not count, or of none: their products may be
      // anything (a zero query times an infinite key is NaN)
      const int dead = p.live * A.G;
      // what a key's slot holds already and its page, loaded a tile ahead
      auto held = [&](int t) {
        const int j = t * kTileKeys + key;
        return t < tb && j < p.n ? (!fresh ? out[j] : prior ? prior[j] : 0.0f) : 0.0f;
      };
      auto page_of = [&](int t) {
        const int j = t * kTileKeys + key;
        return t < p.mb && j >= p.first && j <= p.last
                   ? __ldg(A.table + (int64_t)p.b * A.max_pages + (j >> A.log_page))
                   : 0;
      };
      int t = ta + ((ta ^ group) & 1);
      float before = held(t);
      int page = page_of(t);
#pragma unroll 1
      for (; t < tb; t += 2) {
        const float next_before = held(t + 2);
        const int next_page = page_of(t + 2);
        const int j = t * kTileKeys + key;
        float total = 0.0f;
        if (t >= p.ma && t < p.mb) {
          const bool edge = edge_tile(p, A.rule.window, t);
          wait_phase(&sh.s_full[0][group], (uint32_t)used & 1u, &sh.waits);
          ++used;
          tc_fence_after();
#pragma unroll 2
          for (int q = 0; q < S::N; q += 16) {
            if (q >= dead) break;
            float s[16];
            tmem_ld16(lane_base + group * S::N + q, s);
            tmem_wait_ld();
            if (__builtin_expect(q + 16 > dead, 0)) {
#pragma unroll
              for (int c = 0; c < 16; ++c)
                if (q + c >= dead) s[c] = 0.0f;
            }
            float scale = A.rule.scale * kLog2e;
            if (__builtin_expect(edge || A.rule.softcap > 0.0f || A.rule.slopes, 0)) {
              apply_rule<16>(s, A.rule, (float)(p.pos0 - j), &T.slope[q], &T.ahead[q]);
              scale = 1.0f;
              if (edge) {
#pragma unroll
                for (int c = 0; c < 16; ++c)
                  if (j > T.hi[q + c] || j <= T.lo[q + c]) s[c] = -INFINITY;
              }
            }
            const Two sc = two(scale, scale);
            Two part = 0ull;
#pragma unroll
            for (int c = 0; c < 16; c += 2) {
              const float2 m = *reinterpret_cast<const float2*>(&T.m[q + c]);
              const float2 e = split(two_fma(two(s[c], s[c + 1]), sc, two(m.x, m.y)));
              part = two_add(part, two(ex2(e.x), ex2(e.y)));
            }
            total += split(part).x + split(part).y;
          }
          tc_fence_before();
          mbar_arrive(&sh.s_empty[0][group]);
          if (page < 0 || page >= A.num_pages) total = nan;
        }
        if (j < p.n) out[j] = before + total;
        before = next_before;
        page = next_page;
      }
    }
  }
}

// ---- what the roles leave ------------------------------------------------------------------------
// Pieces without tiles for the tensor cores: rows that see no key get 0 and a log-sum-exp of -inf,
// keys that no counted row sees keep what they held, requests with bad counts get NaN. Of a CTA that
// gave up, all pieces: NaN in rows, key weights and the parts of split items, whose join then gives
// NaN as well. All threads, once the roles are done.
template <class S>
__device__ __noinline__ void write_rest(const TileArgs& A, const TileShared<S>& sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float nan = __uint_as_float(0x7fc00000u);
  const bool dead = sh.waits.dead;
  Walk<S> walk(A, sh.start);
  Piece p;
  JoinItem join{};
  int at = 0;
#pragma unroll 1
  while (walk.next(p)) {
    if (!dead && !(p.flags & kHollow)) continue;
    const bool bad = dead || (p.flags & kBad);
    if constexpr (S::Weigh) {
      const int64_t row = ((int64_t)p.b * A.Hkv + p.h) * A.stride;
      if (p.flags & kBad) {
        if (threadIdx.x == 0) A.weights[row] = nan;
        continue;
      }
      const int end = p.tb * kTileKeys < p.n ? p.tb * kTileKeys : p.n;
#pragma unroll 4
      for (int j = p.ta * kTileKeys + (int)threadIdx.x; j < end; j += S::Threads)
        A.weights[row + j] = dead ? nan : A.prior ? A.prior[row + j] : 0.0f;
    } else {
      const int64_t row0 = ((int64_t)p.b * A.P + p.i0) * A.Hq + p.h * A.G;
      const int rows = p.live * A.G;
      const bool starts = p.flags & kStarts, whole = starts && (p.flags & kEnds);
      if (starts && !whole) join = JoinItem{rows, p.pieces, row0};
      if (at++ % (S::Threads / 32) != warp) continue;  // (a warp per piece)
      if (!whole) {
        float* part = A.part + (2 * (int64_t)blockIdx.x + (starts ? 1 : 0)) * (S::N * (S::D + 2));
#pragma unroll 1
        for (int c = lane; c < rows; c += 32)
          *reinterpret_cast<float2*>(part + S::N * S::D + 2 * c) = make_float2(0.0f, nan);
        continue;
      }
      const uint32_t w = pack16<S::Bf16>(bad ? nan : 0.0f, bad ? nan : 0.0f);
      constexpr int kVecs = S::D / 8;
#pragma unroll 1
      for (int e = lane; e < rows * kVecs; e += 32) {
        const int c = e / kVecs;
        const int64_t r = row0 + c / A.G * A.Hq + c % A.G;
        reinterpret_cast<uint4*>(A.out)[r * kVecs + e % kVecs] = make_uint4(w, w, w, w);
      }
      if (A.out_lse)
#pragma unroll 1
        for (int c = lane; c < rows; c += 32)
          A.out_lse[row0 + c / A.G * A.Hq + c % A.G] = bad ? nan : -INFINITY;
    }
  }
  if (!S::Weigh && dead && threadIdx.x == 0) A.joins[blockIdx.x] = join;
}

// ---- the kernel ---------------------------------------------------------------------------------
template <class S>
__global__ void __launch_bounds__(S::Threads, 1)
    tile_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                const __grid_constant__ CUtensorMap mv, const __grid_constant__ TileArgs A,
                const __grid_constant__ ValuePool vpool) {
  extern __shared__ unsigned char tile_smem[];
  __shared__ TileShared<S> sh;
  static_assert(sizeof(TileShared<S>) <= S::kTables, "shared memory");
  // operand tiles start on 1024-byte boundaries (the swizzle pattern's period)
  unsigned char* base = tile_smem + ((1024u - (smem_u32(tile_smem) & 1023u)) & 1023u);
  unsigned char* qbuf = base;
  unsigned char* pbuf = qbuf + S::NQ * S::QBytes;
  unsigned char* ring = pbuf + S::Teams * S::NP * S::PBytes;
  const int tid = threadIdx.x, warp = tid >> 5;

  if (tid == 0) {
#pragma unroll 1
    for (int s = 0; s < S::NU; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], 1);
    }
    for (int s = 0; s < S::NQ; ++s) {
      mbar_init(&sh.q_full[s], 1);
      mbar_init(&sh.q_empty[s], 1);
    }
    for (int t = 0; t < S::Teams; ++t) {
      for (int s = 0; s < 2; ++s) {
        mbar_init(&sh.s_full[t][s], 1);
        mbar_init(&sh.s_empty[t][s], S::Weigh ? 128 : S::TeamThreads);
      }
      for (int s = 0; s < S::NP; ++s) {
        mbar_init(&sh.p_full[t][s], S::TeamThreads);
        mbar_init(&sh.pv_done[t][s], 1);
      }
    }
    for (int t = 0; t < S::Teams; ++t) mbar_init(&sh.v_ready[t], 1);
    mbar_init(&sh.o_done[0], 1);
    mbar_init(&sh.o_done[1], 1);
    for (int s = 0; s < kPieceQueue; ++s) {
      mbar_init(&sh.piece_full[s], 1);
      // taken by the softmax warps, the issuing threads and the value copies
      mbar_init(&sh.piece_empty[s], S::SoftWarps + (S::Weigh ? 1 : 3));
    }
    mbar_init(&sh.drain[0], 1);
    mbar_init(&sh.drain[1], 1);
    sh.waits.dead = sh.hollow = 0;
    sh.waits.limit_ns = A.wait_ns;
    sh.join.rows = 0;
    for (int i = 0; i < 8; ++i) sh.bad_piece[i] = 0;
    fence_barrier_init();
  }
  if (tid == 32) {
    prefetch_map(&mq);
    prefetch_map(&mk);
    if (!S::Weigh) prefetch_map(&mv);
  }
  if (warp == S::ScoreWarp) tmem_alloc(&sh.tmem, S::TmemCols);
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
  find_start<S>(A, &sh.start, sh.scratch);
  tc_fence_after();
  if (!S::Weigh) {
    // the joining kernel may take its place beside this one; it waits for this one's end
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  }
  if (sh.start.left <= 0) {
    if (!S::Weigh && tid == 0) A.joins[blockIdx.x] = JoinItem{};
    if (warp == S::ScoreWarp) tmem_free(sh.tmem, S::TmemCols);
    return;
  }

  if (warp == S::KeyWarp) {
    copy_role<S, false>(A, sh, qbuf, ring, &mq, &mk);
  } else if (warp == S::ScoreWarp) {
    if ((tid & 31) == 0) score_role<S>(A, sh, qbuf, ring);
    __syncwarp();
  } else if (!S::Weigh && warp == S::CopyVWarp) {
    copy_role<S, true>(A, sh, qbuf, ring, &mq, &mv);
  } else if (!S::Weigh && warp == S::ValueWarp) {
    if ((tid & 31) == 0) value_role<S>(A, sh, pbuf, ring);
    __syncwarp();
  } else if constexpr (S::Weigh) {
    weigh_role<S>(A, sh);
  } else {
    const int lane = tid & 31, quarter = warp & 3, group = warp >> 2;
    const int team = S::Teams == 2 ? group : 0;
    Attend<S> R{A, vpool, sh, pbuf, ring, lane, quarter, group, quarter * 32 + lane,
                sh.tmem + ((uint32_t)(quarter * 32) << 16), team,
                S::Teams == 2 ? tid & 127 : tid, S::Teams == 2 ? 0 : group * S::NC};
    R.run();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (!S::Weigh && tid == 0) A.joins[blockIdx.x] = sh.join;
  if (warp == S::ScoreWarp) tmem_free(sh.tmem, S::TmemCols);
  if (sh.hollow || sh.waits.dead) write_rest<S>(A, sh);
}

// ---- joining the pieces of split items --------------------------------------------------------
// Thread: four of D of one row, over all its pieces: those of an item are the second slot of the
// CTA that began it and the first slots of the CTAs after it, joined in that order, eight in
// flight.
constexpr int kJoinThreads = 128;
template <int kD, int kN>
constexpr int kJoinShares = kN * (kD / 4) / kJoinThreads;

template <int kD, int kN, bool kBf16>
__global__ void __launch_bounds__(kJoinThreads)
    join_kernel(const JoinItem* joins, const float* part, int G, int Hq, void* out, float* out_lse) {
  constexpr int64_t kSlot = kN * (kD + 2);
  constexpr int kBatch = 8;
  const int c = blockIdx.x, e = blockIdx.y * kJoinThreads + threadIdx.x;
  const int n = e / (kD / 4), d = e % (kD / 4) * 4;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const JoinItem J = joins[c];
  if (n >= J.rows) return;
  const float* s0 = part + (2 * c + 1) * kSlot;  // the first piece; the i-th is at s1 + 2 i slots
  const float* s1 = part + 2 * c * kSlot;
  float m = kNoMax, sum = 0.0f;
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
  for (int i0 = 0; i0 < J.pieces; i0 += kBatch) {
    float2 ml[kBatch];
    float4 v[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      ml[i] = make_float2(kNoMax, 0.0f);
      v[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (i0 + i < J.pieces) {
        const float* s = i0 + i == 0 ? s0 : s1 + 2 * (i0 + i) * kSlot;
        ml[i] = *reinterpret_cast<const float2*>(s + kN * kD + 2 * n);
        v[i] = *reinterpret_cast<const float4*>(s + n * kD + d);
      }
    }
    float top = m;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) top = fmaxf(top, ml[i].x);
    const float a = ex2(m - top);
    m = top;
    sum *= a;
    acc.x *= a;
    acc.y *= a;
    acc.z *= a;
    acc.w *= a;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      // (never 0: a part that an infinite value made infinite stays so)
      const float w = fmaxf(ex2(ml[i].x - m), 1.17549435e-38f);
      sum += w * ml[i].y;
      acc.x = fmaf(w, v[i].x, acc.x);
      acc.y = fmaf(w, v[i].y, acc.y);
      acc.z = fmaf(w, v[i].z, acc.z);
      acc.w = fmaf(w, v[i].w, acc.w);
    }
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  const int64_t row = J.row0 + n / G * Hq + n % G;
  *reinterpret_cast<uint2*>(static_cast<char*>(out) + 2 * (row * kD + d)) =
      make_uint2(pack16<kBf16>(acc.x * inv, acc.y * inv), pack16<kBf16>(acc.z * inv, acc.w * inv));
  if (out_lse && d == 0)
    out_lse[row] = row_lse<kBf16>(m, sum);
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

// Whether a CTA's share of the longest work list these sizes allow stays in 32 bits.
inline bool ranges_fit(const sv_kv_shape* s, int blocks) {
  const double tiles = (double)s->max_pages * s->page_size / kTileKeys + 1;
  return (double)s->B * s->Hkv * blocks * (tiles * 4 + 32) < 1e9 * device_sm_count();
}

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
