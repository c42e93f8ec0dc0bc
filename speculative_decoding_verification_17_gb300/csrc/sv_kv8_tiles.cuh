// sv_kv8_tiles.cuh — what the tile kernel (sv_kv_tiles.cuh) does otherwise over a cache in 8 bits.
//
// Mathematics. Keys and values are e4m3 codes with a scale for each block of tokens and kv head.
// With ks_j and vs_j the scales of key j's block, and codes k, v,
//   s_j = scale * ks_j * (q . k_j)                    a thread per key: one factor more
//   w_j = 2^(s_j - m) * vs_j,  O = sum w_j v_j        the values' scale goes into the weight
//   l   = sum 2^(s_j - m)                             the softmax's sum does not have it
// so the codes go to the tensor cores as they lie in the cache (kind::f8f6f4, 32 deep), and no tile
// is ever widened: 32 KiB per 128 keys of D = 128 instead of 64.
//
// Rounding. Both operands of the instruction are 8 bits wide, so queries and weights are given to it
// as sums of such numbers.
// - A query row is scaled by a power of two to a largest magnitude in [128, 256) and split into two
//   e4m3 numbers (bf16) or three (fp16): its 8 or 11 bits exactly, or for an element below 2^-9 (bf16)
//   or 2^-6 (fp16) of the row's largest, to 2^-17 of that at worst.
// - A weight is rounded to fp16, to nearest: by 2^-11 of it at worst, as the output of fp16 itself and
//   an eighth of bf16's. The upper byte of an fp16 number is an e5m2 number (cut, not rounded), what
//   that leaves has three bits less, and four such cuts take all 11. Below 2^-16, the last step of
//   e5m2, nothing is left to cut: the weight is rounded to that step first, to nearest, so that the cuts
//   lose nothing: 2^-17 more, which is 2^-27 (bf16) or 2^-28 (fp16) of the row's largest weight, 2^Lift or
//   more. (Half the step added ahead of the cuts was a one-sided error of as much in every weight, for 89.1
//   us instead of 87.4 for five drafts; half a step of the last cut's own, added to its bits, rounds the
//   middle up, which numbers of fp16 below 2^-6 hit often: 87.8.)
// The four products are one instruction of four times the columns and are added at the end of a piece.
// The instruction adds up in fp32, cut: measured 2^-20.7 of sum |a b| over 128 products, and sums that
// fp32 holds exactly come out exact.
// Weights as four e4m3 numbers, each 16 times finer than the one before, keep 2^-16 of a weight; the
// conversions took 9 % (one token of 64 requests 97 -> 94 us, five drafts 207 -> 196).
//
// Running maximum. Of s_j + log2 vs_j, as that is what bounds a weight: m is the maximum less Lift when
// it moves, which it does when a weight passes 2^15.875 (fp16 ends at 2^16). log2 vs_j counts as
// -40 .. 40; a scale above 2^40, negative or not a number makes what sees the key NaN.
//
// Bound: reading the codes once, until the softmax takes longer. A tile of D = 128 is 1400 clocks of
// one SM's share of the bandwidth; its softmax at 48 columns is a chain of about 2000 (loads from
// tensor memory, two exponents, cuts, stores to shared memory, the hand-over), of which 12 warps hide
// half, and four instructions of 128 x 4N x 32 take 400 up to 128 columns, 520 at 256. Measured, in
// graph replays (the bytes read and written once at 6801 GB/s first):
//   1 token of 64 requests, 200 .. 8192 keys, 32 / 8 heads   41.8 us   54.8 us   76 %
//   6 positions of 32, 500 .. 16384 keys, 64 / 8 heads       42.4 us   89.2 us   48 %
//   9 positions of 2, 100001 .. 131072 keys, 32 / 8 heads    77.4 us  122.3 us   63 %
//   5 positions of 16, window 4096, 16 / 8 heads of 256      15.8 us   35.0 us   45 %
//   1 token of 1 request of 777 keys                          0.2 us   10.5 us  (latency)
// and by query rows per kv head (64 requests of 200 .. 8192 keys, 8 kv heads, D = 128, floor 42 to 44
// us; over 16 bits in brackets): 4 57 (98), 12 62 (100), 24 83 (103), 32 85 (104), 48 104 (116), 64 129
// (116), 72 173 (200). Above 48 rows the softmax bounds and half the bytes gain nothing.
#pragma once

#include <cuda_fp8.h>

#include "sv_kv_tiles.cuh"

namespace sv {

constexpr float kMaxScale = 1099511627776.0f;  // 2^40

template <int kD, int kN, bool kBf16>
struct TileShape8 {
  static constexpr int D = kD, N = kN;
  static constexpr bool Bf16 = kBf16, Weigh = false, Quant = true;  // (the queries' and outputs' type)
  // log2 of the largest weight when the maximum moves, and at most
  static constexpr float Lift = kBf16 ? 10.0f : 11.0f, Top = 15.875f;
  static constexpr int UnitCols = D < 128 ? D : 128, RowBytes = UnitCols, UnitBytes = kTileKeys * RowBytes;
  static constexpr int U = D / UnitCols;
  // Softmax threads take a key and 16 columns (8 where there are no more): a group of four warps for
  // each 16. Two CTAs share an SM up to 16 columns, so that one's chain of dependent steps passes under
  // the other's (at 32 columns their 88 registers are too few: 24 rows 108 us, 82 with one).
  static constexpr int Teams = 1, Groups = N == 8 ? 1 : N / 16, SoftWarps = 4 * Groups;
  static constexpr int CtasPerSm = N <= 16 ? 2 : 1;
  static constexpr int SoftThreads = 32 * SoftWarps;
  // the softmax, then a warp each: copies, scores, values
  static constexpr int KeyWarp = SoftWarps, ScoreWarp = KeyWarp + 1, ValueWarp = KeyWarp + 2,
                       CopyVWarp = -1;
  static constexpr int Threads = SoftThreads + 96;
  static constexpr int TeamThreads = SoftThreads;
  static constexpr int NC = N == 8 ? 8 : 16, CH = NC;  // columns per softmax thread
  // e4m3 numbers of a query element, and how many of them are columns of the score instruction (whose
  // columns are a multiple of 16): a third is added in a pass of its own, or beside a row of zeros
  static constexpr int QParts = kBf16 ? 2 : 3, QWide = N == 8 && !kBf16 ? 4 : 2;
  static constexpr int QRows = QParts > QWide ? QParts : QWide;  // parts in the buffer
  static constexpr int QBytes = QRows * N * D;
  static constexpr int NQ = 1;
  static constexpr int Parts = 4;  // of a weight
  // Tiles of a pass. Two hide the chain of one CTA on an SM (24 rows of 64 requests: 83 us, one at a
  // time 89; 48 rows: 102, 110). One leaves 64 columns, and two CTAs, enough registers (64 rows: 131
  // us, two at a time 145; 12 rows: 62, 74; 4 rows of 128 dimensions 57 either way, 2 of 256: 54, 56).
  static constexpr int Pair = N == 64 || CtasPerSm > 1 ? 1 : 2;
  static constexpr int PTile = Parts * kTileKeys * N, PBytes = Pair * PTile, NP = 1;
  static constexpr int kTables = 104 * N + 1920;
  static constexpr int kRoom = kSmemMax / CtasPerSm - (CtasPerSm == 2 ? 512 : 0) - kTables - 1024 -
                               NQ * QBytes - PBytes;
  static constexpr int NU = kRoom / UnitBytes > 16 ? 16 : kRoom / UnitBytes;
  static constexpr int NV = NU / 2, NK = NU - NV;
  static constexpr int Smem = 1024 + NQ * QBytes + PBytes + NU * UnitBytes;
  static constexpr int MBlocks = (D + 127) / 128;
  static constexpr bool Wide = true;
  static constexpr int ON = Parts * N;
  // a score buffer of two tiles, read into registers before the next ones need it (or two of one)
  static constexpr int SN = QWide * N, OBase = 2 * SN, SBufs = 2 / Pair;
  static constexpr int Outs = 1;  // (a piece's output leaves while the next one's first scores are made)
  static constexpr int TmemNeed = OBase + Outs * MBlocks * ON;
  static constexpr int TmemCols = TmemNeed <= 128 ? 128 : TmemNeed <= 256 ? 256 : 512;
  // The cost of a tile and of a piece's start and end, which only other CTAs of the SM can cover; with
  // two tiles a pass a tile counts for less, so a piece for more. Measured, us, the figure that was taken
  // third:  5 drafts, 48 columns      108 with 13    97 with 24    88 with 26   91 with 40
  //         20 rows, D = 256          83 with 6      69 with 14    62 with 20   67 with 32
  //         64 rows, 64 columns       159 with 6     137 with 10   125 with 16  132 with 26
  //         12 rows, 16 columns       67 with 8      62 with 12    61 with 16   63 with 24
  //         4 rows, 8 columns         60 with 3      58 with 8     57 with 12   59 with 24
  //         window, D = 256           40 with 3      36 with 6     35 with 9    36 with 24
  static constexpr int TileCost = 4;
  static constexpr int PieceCost = Pair == 2 ? (D == 256 ? 20 : 26) : D == 256 ? 9 : N == 8 ? 12 : 16;
  static_assert(CtasPerSm * TmemCols <= 512 && NV >= U && NK >= U &&
                CtasPerSm * (Smem + kTables) <= kSmemMax, "tile shape");
};

// The tiles [lo, hi) of a piece whose keys every row sees. Those go two at a time, others (and the
// last of an odd number) alone.
struct WholeTiles {
  int lo, hi;
  __device__ __forceinline__ WholeTiles(const Piece& p, int window)
      : lo((first_full(p, window) + kTileKeys - 1) >> 7), hi((p.pos0 + 1) >> 7) {}
  __device__ __forceinline__ bool edge(int t) const { return t < lo || t >= hi; }
  // How many go together from tile t (of left tiles, newest first) on.
  template <class S>
  __device__ __forceinline__ int at(int t, int left) const {
    return S::Pair == 2 && left > 1 && t < hi && t > lo ? 2 : 1;
  }
};

__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       bool accumulate) {
  asm volatile(
      "{ .reg .pred p;\n"
      "  setp.ne.b32 p, %4, 0;\n"
      "  tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p; }" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}
// The instruction descriptor: fp32 accumulator, A of e4m3, B of e4m3 or e5m2.
__device__ __forceinline__ uint32_t mma_desc8(bool mn, bool b_e5m2, int M, int N) {
  return 1u << 4 | (b_e5m2 ? 1u << 10 : 0u) | (mn ? 3u << 15 : 0u) | (uint32_t)(N >> 3) << 17 |
         (uint32_t)(M >> 4) << 24;
}
constexpr uint32_t kSwizzle64 = 4;
// Operand rows of RowBytes bytes: their swizzle, and the bytes of eight of them.
template <class S>
constexpr uint32_t kRowSwizzle = S::RowBytes == 128 ? kSwizzle128 : kSwizzle64;
template <class S>
constexpr uint32_t kRows8 = 8 * S::RowBytes;

// ---- the copies ----------------------------------------------------------------------------------
// One warp walks the work list, hands out the pieces and copies the keys and values of their tiles,
// each lane those of its group of keys; the pages of the next tile are looked up a tile ahead. The
// values go kLag tiles behind the keys: a pass's scores need its keys alone, and keys that waited
// behind values, whose ring is freed last, held up the next pass's scores (five drafts 96.9 -> 91.6 us,
// long caches 127.5 -> 120.5, heads of 256 in a window 47.5 -> 40.9).
template <class S>
__device__ __forceinline__ void copy_role8(const TileArgs& A, TileShared<S>& sh, unsigned char* ring,
                                           const CUtensorMap* mk, const CUtensorMap* mv) {
  const int lane = threadIdx.x & 31;
  Walk<S> walk(A, sh.start);
  RingPos queue;
  bool hollow = false;
  // the next piece with tiles for the tensor cores; all lanes
  auto take = [&](Piece& p) -> bool {
    bool more;
#pragma unroll 1
    while ((more = walk.next(p)) && p.mb == p.ma) hollow |= (p.flags & kHollow) != 0;
    if (!more) p.flags = kEndOfList;
    if (!__all_sync(0xffffffffu, wait_phase(&sh.piece_empty[queue.slot], queue.phase ^ 1u, &sh.waits)))
      return false;
    if (lane == 0) {
      sh.hollow = hollow;
      sh.piece[queue.slot] = p;
      mbar_arrive(&sh.piece_full[queue.slot]);
    }
    queue.next(kPieceQueue);
    return more;
  };
  // a tile as the lane copies it: its page (-1: not), the bytes of all lanes, where its keys lie
  struct Group {
    uint32_t bytes;
    int slot, head, page;
  };
  // the units of a tile of keys or values into their ring; false when a wait failed
  auto copy = [&](const CUtensorMap* map, RingPos& at, int base, int units, int& issued,
                  const Group& g) -> bool {
#pragma unroll 1
    for (int c = 0; c < S::U; ++c) {
      uint64_t* full = &sh.full[base + at.slot];
      if (!__all_sync(0xffffffffu, wait_phase(&sh.empty[base + at.slot], at.phase ^ 1u, &sh.waits)))
        return false;
      if (lane == 0) mbar_arrive_expect_tx(full, g.bytes);
      ++issued;
      __syncwarp();
      if (g.page >= 0)
        tile_g2s(ring + (base + at.slot) * S::UnitBytes + lane * A.box * S::RowBytes, map, full,
                 c * S::UnitCols, g.slot, g.head, g.page);
      at.next(units);
    }
    return true;
  };
  // (a pass whose values have to be cleaned waits for them before its keys' successors are read: the
  // key ring has to hold the tiles of the lag without any of them being freed)
  constexpr int kLag = S::NK / S::U >= 2 ? 2 : 1;
  Group behind[kLag];
  int held = 0;  // tiles whose values are still to be copied, the oldest first
  Piece p;
  bool more = take(p);
  int i = 0, keys = 0, values = 0;
  bool seen = more && group_seen(A, p, tile_at<S>(p, 0), lane);
  int page = seen ? group_page(A, p, tile_at<S>(p, 0), lane) : 0;
  RingPos at_k, at_v;
#pragma unroll 1
  while (more || held > 0) {
    Group g;
    const bool key = more;
    if (key) {
      const int turn = p.turn;
      const bool mine = seen && (unsigned)page < (unsigned)A.num_pages;
      g.page = mine ? page : -1;
      g.head = p.h;
      g.slot = (tile_at<S>(p, i) * kTileKeys + lane * A.box) & ((1 << A.log_page) - 1);
      if (__builtin_expect(__any_sync(0xffffffffu, seen && !mine), 0) && lane == 0)
        *(volatile int*)&sh.bad_piece[turn & (kMarks - 1)] = turn + 1;
      g.bytes = (uint32_t)(__popc(__ballot_sync(0xffffffffu, mine)) * A.box) * (uint32_t)S::RowBytes;
      if (__builtin_expect(++i == p.mb - p.ma, 0)) {
        more = take(p);
        i = 0;
      }
      seen = more && group_seen(A, p, tile_at<S>(p, i), lane);
      page = seen ? group_page(A, p, tile_at<S>(p, i), lane) : 0;
      if (!copy(mk, at_k, 0, S::NK, keys, g)) break;
    }
    if (held == kLag || !key) {
      if (!copy(mv, at_v, S::NK, S::NV, values, behind[0])) break;
#pragma unroll
      for (int k = 0; k + 1 < kLag; ++k) behind[k] = behind[k + 1];
      --held;
    }
    if (key) {
#pragma unroll
      for (int k = 0; k < kLag; ++k)
        if (k == held) behind[k] = g;
      ++held;
    }
  }
  if (lane == 0) {
    // no copy may outlive the CTA, should the others give up before they have seen it land
#pragma unroll 1
    for (int u = keys > S::NK ? keys - S::NK : 0; u < keys; ++u)
      mbar_wait(&sh.full[u % S::NK], (uint32_t)(u / S::NK) & 1u, kTileWaitNs);
#pragma unroll 1
    for (int u = values > S::NV ? values - S::NV : 0; u < values; ++u)
      mbar_wait(&sh.full[S::NK + u % S::NV], (uint32_t)(u / S::NV) & 1u, kTileWaitNs);
  }
  __syncwarp();
}

// ---- the queries ---------------------------------------------------------------------------------
// The softmax threads read a piece's query rows, 8 elements at a time, and leave them as e4m3 numbers,
// part by part (per unit of the row's columns), in the layout of the instruction's operand: rows of
// RowBytes, 16-byte pieces swapped by the row. (One warp of its own took 5 us for 48 rows, which a
// piece's first scores waited for.)
template <class S>
struct Queries8 {
  static constexpr int kLanes = S::D / 8;  // threads of a row
  static constexpr int kTurns = (S::N * kLanes + S::SoftThreads - 1) / S::SoftThreads;
  uint4 x[kTurns];
  __device__ __forceinline__ int row(int me, int s) const { return (s * S::SoftThreads + me) / kLanes; }
  __device__ __forceinline__ void load(const TileArgs& A, const Piece& p, int me) {
    const uint16_t* q = static_cast<const uint16_t*>(A.q) + p.b * A.q_req + p.i0 * A.q_row +
                        (int64_t)p.h * A.G * A.q_head + me % kLanes * 8;
    const int rows = p.live * A.G;
#pragma unroll
    for (int s = 0; s < kTurns; ++s) {
      const int c = row(me, s), i = c / A.G;
      x[s] = make_uint4(0u, 0u, 0u, 0u);
      if (c < rows) x[s] = *reinterpret_cast<const uint4*>(q + i * A.q_row + (c - i * A.G) * A.q_head);
    }
  }
  __device__ __forceinline__ void give(int me, unsigned char* qbuf, float* column_scale) const {
    const int col = me % kLanes * 8;
    unsigned char* buf = qbuf + col / S::UnitCols * (S::QRows * S::N * S::RowBytes);
#pragma unroll
    for (int s = 0; s < kTurns; ++s) {
      const int c = row(me, s);
      if (c >= S::N) break;  // (whole warps)
      const uint32_t w[4] = {x[s].x, x[s].y, x[s].z, x[s].w};
      // the row's largest magnitude, by its bits (those of what is not finite are the largest)
      uint32_t top = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) top = max(top, max(w[e] & 0x7fffu, w[e] >> 16 & 0x7fffu));
#pragma unroll
      for (int o = kLanes / 2; o >= 1; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      const bool odd = top >= (S::Bf16 ? 0x7f80u : 0x7c00u);
      // 2^e <= top < 2^(e+1), e at least -100 (what is smaller counts as 0)
      const int e =
          top == 0 ? 0 : max(-100, (int)(__float_as_uint(unpack16<S::Bf16>(top).x) >> 23) - 127);
      const float up = odd ? 1.0f : __uint_as_float((uint32_t)(127 + 7 - e) << 23);
      float f[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 v = unpack16<S::Bf16>(w[k]);
        f[2 * k] = v.x * up;
        f[2 * k + 1] = v.y * up;
      }
      const uint32_t at0 = c * S::RowBytes + col % S::UnitCols;
      const uint32_t at = at0 ^ ((at0 >> 7 & (S::RowBytes == 128 ? 7u : 3u)) << 4);
#pragma unroll
      for (int part = 0; part < S::QRows; ++part) {
        uint32_t out[2] = {0u, 0u};
        if (part < S::QParts) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const __nv_fp8x2_storage_t b =
                __nv_cvt_float2_to_fp8x2(make_float2(f[2 * k], f[2 * k + 1]), __NV_SATFINITE, __NV_E4M3);
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(b, __NV_E4M3);
            const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&h));
            f[2 * k] -= back.x;
            f[2 * k + 1] -= back.y;
            out[k / 2] |= (uint32_t)b << 16 * (k & 1);
          }
          if (odd) out[0] = out[1] = 0x7f7f7f7fu;  // NaN
        }
        *reinterpret_cast<uint2*>(buf + part * (S::N * S::RowBytes) + at) = make_uint2(out[0], out[1]);
      }
      if (me % kLanes == 0)
        column_scale[c] = __uint_as_float((uint32_t)(127 - 7 + (odd ? 7 : e)) << 23);
    }
  }
};

// ---- the threads that issue the matrix instructions -------------------------------------------
// S^T = K Q^T of every tile, the queries' parts side by side as columns.
template <class S>
__device__ __forceinline__ void score_role8(const TileArgs& A, TileShared<S>& sh,
                                            unsigned char* qbuf, unsigned char* ring) {
  const uint32_t idesc = mma_desc8(false, false, 128, S::SN);
  const uint64_t rows = smem_desc(0, 16, kRows8<S>, kRowSwizzle<S>);
  const uint64_t a0 = rows + (smem_u32(ring) >> 4), b0 = rows + (smem_u32(qbuf) >> 4);
  Reader<S> reader(sh);
  RingPos at;
  uint32_t y = 0;  // turns of the score buffer
  Piece p;
#pragma unroll 1
  while (reader.template next<false>(p)) {
    const int tiles = p.mb - p.ma;
    if (!wait_phase(&sh.q_full[0], (uint32_t)p.turn & 1u, &sh.waits)) goto end;
    const WholeTiles whole(p, A.rule.window);
    int i = 0;
#pragma unroll 1
    while (i < tiles) {
      const int last = i + whole.template at<S>(tile_at<S>(p, i), tiles - i);
      const uint32_t buf = y % S::SBufs;
      if (!wait_phase(&sh.s_empty[0][buf], (y / S::SBufs & 1u) ^ 1u, &sh.waits)) goto end;
      tc_fence_after();
      uint32_t d = sh.tmem + buf * S::SN;
#pragma unroll 1
      for (; i < last; ++i, d += S::SN) {
        uint64_t b = b0;
#pragma unroll 1
        for (int c = 0; c < S::U; ++c, b += S::QRows * S::N * S::RowBytes >> 4) {
          if (!wait_phase(&sh.full[at.slot], at.phase, &sh.waits)) goto end;
          tc_fence_after();
          const uint64_t a = a0 + at.slot * (S::UnitBytes >> 4);
#pragma unroll
          for (int k = 0; k < S::RowBytes / 32; ++k)
            mma_f8(d, a + 2 * k, b + 2 * k, idesc, c > 0 || k > 0);
          if (S::QParts > S::QWide) {  // (onto the first part's)
            const uint32_t third = mma_desc8(false, false, 128, S::N);
#pragma unroll
            for (int k = 0; k < S::RowBytes / 32; ++k)
              mma_f8(d, a + 2 * k, b + (S::QWide * S::N * S::RowBytes >> 4) + 2 * k, third, true);
          }
          mma_commit(&sh.empty[at.slot]);
          at.next(S::NK);
        }
      }
      mma_commit(&sh.s_full[0][buf]);
      ++y;
    }
  }
end:
  drain<S>(sh, 0);
}

// O^T (+)= V^T P^T of every tile, the weights' parts side by side as columns.
template <class S>
__device__ __forceinline__ void value_role8(const TileArgs& A, TileShared<S>& sh,
                                            unsigned char* pbuf, unsigned char* ring) {
  const uint32_t idesc = mma_desc8(true, true, 128, S::ON);
  // (with D = 64 both halves of the instruction's rows read the same columns, and the upper half is
  // not used)
  const uint64_t a0 = smem_desc(0, 0, kRows8<S>, kRowSwizzle<S>) +
                      ((smem_u32(ring) + S::NK * S::UnitBytes) >> 4);
  const uint64_t b0 = smem_desc(0, kTileKeys * 32, 256, kSwizzle32) + (smem_u32(pbuf) >> 4);
  Reader<S> reader(sh);
  RingPos at;
  uint32_t y = 0;
  Piece p;
#pragma unroll 1
  while (reader.template next<false>(p)) {
    const int tiles = p.mb - p.ma;
    const uint32_t o = sh.tmem + S::OBase + (p.turn & (S::Outs - 1)) * S::MBlocks * S::ON;
    const WholeTiles whole(p, A.rule.window);
    int i = 0;
#pragma unroll 1
    while (i < tiles) {
      const int last = i + whole.template at<S>(tile_at<S>(p, i), tiles - i);
      if (__builtin_expect(whole.edge(tile_at<S>(p, i)), 0)) {
        RingPos look = at;
#pragma unroll 1
        for (int c = 0; c < S::U; ++c) {
          if (!wait_phase(&sh.full[S::NK + look.slot], look.phase, &sh.waits)) goto end;
          look.next(S::NV);
        }
        mbar_arrive(&sh.v_ready[0]);
      }
      if (!wait_phase(&sh.p_full[0][0], y & 1u, &sh.waits)) goto end;
      uint64_t b = b0;
#pragma unroll 1
      for (; i < last; ++i, b += S::PTile >> 4) {
        uint32_t d = o;
#pragma unroll 1
        for (int m = 0; m < S::MBlocks; ++m, d += S::ON) {
          if (!wait_phase(&sh.full[S::NK + at.slot], at.phase, &sh.waits)) goto end;
          tc_fence_after();
          const uint64_t a = a0 + at.slot * (S::UnitBytes >> 4);
#pragma unroll
          for (int k = 0; k < kTileKeys / 32; ++k)
            mma_f8(d, a + k * (4 * kRows8<S> >> 4), b + k * 64, idesc, !(i == 0 && k == 0));
          mma_commit(&sh.empty[S::NK + at.slot]);
          at.next(S::NV);
        }
      }
      mma_commit(&sh.pv_done[0][0]);
      ++y;
    }
    mma_commit(&sh.o_done[p.turn & 1]);
  }
end:
  drain<S>(sh, 1);
}

// ---- the softmax threads ------------------------------------------------------------------------
// The scales of the thread's keys in the two tiles at hand, and the pages of its keys in the tiles
// from the second of them on: each loaded a pass before it is looked at.
template <class S>
struct KeyScales<S, true> {
  float k[2], v[2];
  int page[3];
};

// The page of the thread's key in the i-th tile of a piece, -1 where no row sees it.
template <class S>
__device__ __forceinline__ int key_page(const Attend<S>& me, const Piece& p, int i) {
  const int j = tile_at<S>(p, i) * kTileKeys + me.key;
  return i < p.mb - p.ma && j >= p.first && j <= p.last
             ? __ldg(me.A.table + (int64_t)p.b * me.A.max_pages + (j >> me.A.log_page))
             : -1;
}
// Its scales (0 without a page: what no row sees is masked, and a bad page makes the piece NaN).
template <class S>
__device__ __forceinline__ void load_scales(Attend<S>& me, const Piece& p, int which, int i, int page) {
  const TileArgs& A = me.A;
  me.scales.k[which] = me.scales.v[which] = 0.0f;
  if ((unsigned)page < (unsigned)A.num_pages) {
    const int j = tile_at<S>(p, i) * kTileKeys + me.key;
    const int64_t at = scale_at(A, page, j & ((1 << A.log_page) - 1), p.h);
    me.scales.k[which] = __ldg(A.k_scale + at);
    me.scales.v[which] = __ldg(A.v_scale + at);
  }
}

__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// One arrival per warp (of each thread made no difference that could be measured).
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// The scores of a thread's key under the rule, in place (out of line: few calls have one).
template <class S>
__device__ __noinline__ void apply_rule8(float* s, const ScoreRule& r, float away, const float* slope,
                                         const float* ahead) {
  apply_rule<S::CH>(*reinterpret_cast<float(*)[S::CH]>(s), r, away, slope, ahead);
}

// Raise the maxima of the thread's columns to those of these scores, and scale what the columns hold,
// the product of the y-th turn among it.
template <class S>
__device__ __forceinline__ void raise8(Attend<S>& me, typename TileShared<S>::Table& T,
                                       const float (&s)[S::NC], Two (&l)[S::NC / 2], bool first, int y,
                                       uint32_t o_base) {
  const int c0 = me.col0, lane = me.lane;
  column_max<S::NC>(s, &T.red[me.quarter][c0], lane);
  me.group_sync();
  if (me.quarter == 0 && lane < S::NC) {
    const int c = c0 + lane;
    const float was = -T.m[c];
    const float top = fmaxf(fmaxf(T.red[0][c], T.red[1][c]), fmaxf(T.red[2][c], T.red[3][c]));
    const float m = fmaxf(top - S::Lift, was);
    T.alpha[c] = ex2(was - m);
    T.m[c] = -m;
  }
  me.group_sync();
  if (first) return;
#pragma unroll
  for (int c = 0; c < S::NC; c += 2) {
    const float2 v = split(l[c / 2]);
    l[c / 2] = two(v.x * T.alpha[c0 + c], v.y * T.alpha[c0 + c + 1]);
  }
  me.wait_values(y);
  tc_fence_after();
#pragma unroll 1
  for (int m = 0; m < S::MBlocks * S::Parts; m += S::NC < 16 ? 2 : 1) {
    float o[16];
    const uint32_t at = o_base + m * S::N;
    tmem_ld16(at, o);
    tmem_wait_ld();
#pragma unroll
    for (int c = 0; c < 16; ++c) o[c] *= T.alpha[c0 + c % S::NC];
    tmem_st16(at, o);
  }
  tmem_wait_st();
}

// One pass: one or two of the piece's tiles from the i-th on, the y-th turn of the score buffer. Returns how many.
template <class S>
__device__ __forceinline__ int quant_tiles(Attend<S>& me, typename TileShared<S>::Table& T,
                                           const Piece& p, const WholeTiles& whole, int i, int y,
                                           Two (&l)[S::NC / 2]) {
  constexpr int kC = S::NC;
  const TileArgs& A = me.A;
  auto& sh = me.sh;
  const int t = tile_at<S>(p, i), j = t * kTileKeys + me.key;
  const int both = whole.template at<S>(t, p.mb - p.ma - i);
  const bool edge = both == 1 && whole.edge(t);
  const float* columns = sh.column_scale[p.turn & 1];
  const int c0 = me.col0;
  float ks[S::Pair], vs[S::Pair], lv[S::Pair];
#pragma unroll
  for (int q = 0; q < S::Pair; ++q) {
    ks[q] = me.scales.k[q];
    vs[q] = me.scales.v[q];
    if (!(vs[q] >= 0.0f && vs[q] <= kMaxScale && fabsf(ks[q]) < INFINITY)) {
      ks[q] = __uint_as_float(0x7fc00000u);
      vs[q] = 1.0f;
    }
    lv[q] = fmaxf(lg2(vs[q]), -40.0f);
  }
  load_scales(me, p, 0, i + both, both == 2 ? me.scales.page[1] : me.scales.page[0]);
  load_scales(me, p, 1, i + both + 1, both == 2 ? me.scales.page[2] : me.scales.page[1]);
  me.scales.page[0] = both == 2 ? me.scales.page[2] : me.scales.page[1];
  me.scales.page[1] = key_page(me, p, i + both + 2);
  me.scales.page[2] = key_page(me, p, i + both + 3);
  const uint32_t buf = (uint32_t)y % S::SBufs;
  wait_phase(&sh.s_full[0][buf], (uint32_t)y / S::SBufs & 1u, &sh.waits);
  tc_fence_after();
  float s[S::Pair][kC];
#pragma unroll
  for (int q = 0; q < S::Pair; ++q) {
    const uint32_t at = me.lane_base + (buf + q) * S::SN;
    float a[16], b[16];
    tmem_ld16(at + c0, a);
    if (kC == 16 || S::QWide == 4) tmem_ld16(kC == 16 ? at + S::N + c0 : at + 16, b);
    tmem_wait_ld();
#pragma unroll
    for (int c = 0; c < kC; c += 4) {
      const float4 f = *reinterpret_cast<const float4*>(&columns[c0 + c]);
#pragma unroll
      for (int k = c; k < c + 4; k += 2) {
        Two sum = kC == 16 ? two_add(two(a[k], a[k + 1]), two(b[k], b[k + 1]))
                           : two_add(two(a[k], a[k + 1]), two(a[8 + k], a[9 + k]));
        if (kC == 8 && S::QWide == 4) sum = two_add(sum, two(b[k], b[k + 1]));
        const float2 v = split(two_mul(sum, k == c ? two(f.x, f.y) : two(f.z, f.w)));
        s[q][k] = v.x;
        s[q][k + 1] = v.y;
      }
    }
  }
  warp_arrive(&sh.s_empty[0][buf], me.lane);
  float scale[S::Pair];
#pragma unroll
  for (int q = 0; q < S::Pair; ++q) scale[q] = A.rule.scale * kLog2e * ks[q];
  if (__builtin_expect(edge || A.rule.softcap > 0.0f || A.rule.slopes, 0)) {
#pragma unroll
    for (int q = 0; q < S::Pair; ++q) {
      if (q < both && (A.rule.softcap > 0.0f || A.rule.slopes)) {
        float held[kC];
#pragma unroll
        for (int c = 0; c < kC; ++c) held[c] = s[q][c] * ks[q];
        apply_rule8<S>(held, A.rule, (float)(p.pos0 - j + q * kTileKeys), &T.slope[c0], &T.ahead[c0]);
#pragma unroll
        for (int c = 0; c < kC; ++c) s[q][c] = held[c];
        scale[q] = 1.0f;
      }
    }
    if (edge) {
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        s[0][c] *= scale[0];
        if (j > T.hi[c0 + c] || j <= T.lo[c0 + c]) s[0][c] = -INFINITY;
      }
      scale[0] = 1.0f;
    }
  }
  float top = -INFINITY;
  auto exponents = [&](int q, Two (&e)[kC / 2]) {
    const Two sc = two(scale[q], scale[q]);
#pragma unroll
    for (int c = 0; c < kC; c += 4) {
      const float4 m = *reinterpret_cast<const float4*>(&T.m[c0 + c]);
      e[c / 2] = two_fma(two(s[q][c], s[q][c + 1]), sc, two(m.x, m.y));
      e[c / 2 + 1] = two_fma(two(s[q][c + 2], s[q][c + 3]), sc, two(m.z, m.w));
    }
  };
#pragma unroll
  for (int q = 0; q < S::Pair; ++q) {
    if (q == 1 && both == 1) break;
    Two e[kC / 2];
    exponents(q, e);
    float most = -INFINITY;
#pragma unroll
    for (int c = 0; c < kC / 2; ++c) {
      const float2 v = split(e[c]);
      most = fmaxf(most, fmaxf(v.x, v.y));
    }
    top = fmaxf(top, most + lv[q]);
  }
  if (__builtin_expect(bar_or(1 + me.group, 128, top > S::Top), 0)) {
    float most[kC];
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      most[c] = fmaf(s[0][c], scale[0], lv[0]);
      if (S::Pair == 2 && both == 2)
        most[c] = fmaxf(most[c], fmaf(s[S::Pair - 1][c], scale[S::Pair - 1], lv[S::Pair - 1]));
    }
    raise8<S>(me, T, most, l, i == 0, y - 1, me.output(p.turn));
  }
  // the product that last read the weights' buffer
  if (y > 0) me.wait_values(y - 1);
  // (beside 1.5 * 2^7 a number is rounded to the last cut's step, 2^-16)
  const Two beside = two(192.0f, 192.0f), away = two(-192.0f, -192.0f);
#pragma unroll
  for (int q = 0; q < S::Pair; ++q) {
    if (q == 1 && both == 1) break;
    Two e[kC / 2];
    exponents(q, e);
    uint32_t part[S::Parts][kC / 2];
    const Two size = two(vs[q], vs[q]);
#pragma unroll
    for (int c = 0; c < kC / 2; ++c) {
      const float2 v = split(e[c]);
      const Two w = two(ex2(v.x), ex2(v.y));
      l[c] = two_add(l[c], w);
      const float2 y2 = split(two_add(two_fma(w, size, beside), away));
      __half2 r = __floats2half2_rn(y2.x, y2.y);
#pragma unroll
      for (int k = 0; k < S::Parts; ++k) {
        // the upper byte of an fp16 number is an e5m2 number: what is left has three bits less
        const uint32_t bits = *reinterpret_cast<const uint32_t*>(&r), top3 = bits & 0xff00ff00u;
        part[k][c] = bits;
        if (k + 1 < S::Parts) r = __hsub2(r, *reinterpret_cast<const __half2*>(&top3));
      }
    }
    // 32 columns of a key are 32 bytes, their 16-byte halves swapped in every other 4 keys
    unsigned char* const pb = me.pbuf + q * S::PTile + me.key * 32;
    auto bytes4 = [&](int k, int c) { return __byte_perm(part[k][c], part[k][c + 1], 0x7531); };
    if (kC == 8) {
#pragma unroll
      for (int k = 0; k < S::Parts; k += 2)
        *reinterpret_cast<uint4*>(pb + ((k / 2 ^ me.key >> 2) & 1) * 16) =
            make_uint4(bytes4(k, 0), bytes4(k, 2), bytes4(k + 1, 0), bytes4(k + 1, 2));
    } else {
#pragma unroll
      for (int k = 0; k < S::Parts; ++k) {
        const int n = k * S::N + c0;
        *reinterpret_cast<uint4*>(pb + n / 32 * (kTileKeys * 32) + ((n / 16 ^ me.key >> 2) & 1) * 16) =
            make_uint4(bytes4(k, 0), bytes4(k, 2), bytes4(k, 4), bytes4(k, 6));
      }
    }
  }
  if (__builtin_expect(edge, 0)) {
    wait_phase(&sh.v_ready[0], (uint32_t)(me.edges++) & 1u, &sh.waits);
    if (me.group == 0) me.clean_values(T, p, p.x0 + i, j);
  }
  fence_proxy_async();
  warp_arrive(&sh.p_full[0][0], me.lane);
  return both;
}

// The pieces in turn. A piece's queries are given before the output of the one before it leaves, so
// that its first scores are made meanwhile. (The last scores of the piece before have been read, so
// its queries are done with.)
template <class S>
__device__ __forceinline__ void run8(Attend<S>& me, unsigned char* qbuf) {
  auto& sh = me.sh;
  const TileArgs& A = me.A;
  Reader<S> reader(sh);
  int y = 0, ended = -1;
#pragma unroll 1
  for (;;) {
    const Piece p = reader.wait();
    bool more = !(p.flags & kEndOfList) && !*(volatile int*)&sh.waits.dead;
    more = !bar_or(kAllBar<S>, S::SoftThreads, !more);
    auto& T = sh.table[p.turn & 1];
    if (more) {
      reader.release(me.lane == 0);
      Queries8<S> q;
      q.load(A, p, me.me);
      const int page = key_page(me, p, 0);
#pragma unroll
      for (int k = 0; k < 3; ++k) me.scales.page[k] = key_page(me, p, k + 1);
      set_columns<S>(A, T, p, me.me, S::TeamThreads);
      if (me.me == 0) T.piece = p, T.odd = 0;
      q.give(me.me, qbuf, sh.column_scale[p.turn & 1]);
      fence_proxy_async();
      warp_arrive(&sh.q_full[0], me.lane);
      load_scales(me, p, 0, 0, page);
      load_scales(me, p, 1, 1, me.scales.page[0]);
    }
    if (ended >= 0) me.finish(sh.table[ended & 1]);
    if (!more) break;
    bar_sync(kAllBar<S>, S::SoftThreads);
    const WholeTiles whole(p, A.rule.window);
    Two l[S::NC / 2];
#pragma unroll
    for (int c = 0; c < S::NC / 2; ++c) l[c] = 0ull;
#pragma unroll 1
    for (int i = 0; i < p.mb - p.ma; ++y) i += quant_tiles<S>(me, T, p, whole, i, y, l);
    float sums[S::NC];
#pragma unroll
    for (int c = 0; c < S::NC; c += 2) {
      const float2 v = split(l[c / 2]);
      sums[c] = v.x;
      sums[c + 1] = v.y;
    }
    column_reduce<S::NC, false>(sums, &T.red[me.quarter][me.col0], me.lane);
    ended = p.turn;
  }
}

// The outputs that NaN codes among the values of partly visible keys make NaN (those codes went to
// the tensor cores as 0): of the keys that some rows of the piece see and others do not.
template <class S>
__device__ __noinline__ void special_values8(const TileArgs& A, const ValuePool& vpool,
                                             const typename TileShared<S>::Table& T,
                                             const Piece& p, int col0, int rows, int d0,
                                             float* part, int64_t row0) {
  const int j0 = p.first > p.ma * kTileKeys ? p.first : p.ma * kTileKeys;
  const int j1 = p.last < p.mb * kTileKeys - 1 ? p.last : p.mb * kTileKeys - 1;
  // keys [f0, f1] are seen by all rows
  int f0 = first_full(p, A.rule.window) > j0 ? first_full(p, A.rule.window) : j0;
  int f1 = p.pos0 < j1 ? p.pos0 : j1;
  if (f0 > f1) f0 = j1 + 1, f1 = j1;
  const float nan = __uint_as_float(0x7fc00000u);
#pragma unroll 1
  for (int d = d0; d < S::D; d += 128) {
#pragma unroll 1
    for (int j = j0; j <= j1; ++j) {
      if (j == f0) j = f1 + 1;
      if (j > j1) break;
      const int page = __ldg(A.table + (int64_t)p.b * A.max_pages + (j >> A.log_page));
      if (page < 0 || page >= A.num_pages) continue;
      const int64_t at = page * vpool.page + (j & ((1 << A.log_page) - 1)) * vpool.token +
                         p.h * vpool.head + d;
      if ((__ldg(static_cast<const unsigned char*>(vpool.data) + at) & 0x7f) != 0x7f) continue;
#pragma unroll 1
      for (int n = col0; n < col0 + S::NC && n < rows; ++n) {
        if (j > T.hi[n] || j <= T.lo[n]) continue;
        if (part)
          part[n * S::D + d] = nan;
        else
          store16<S::Bf16>(A.out, (row0 + T.row[n]) * S::D + d, nan);
      }
    }
  }
}

}  // namespace sv
