// attn_prefill_paged.cu — attention of packed new tokens over the paged cache, bf16 or
// e4m3: prompts, pieces of them, a few drafted tokens and single ones in one call, over
// all keys before them or a window and the first few.
//
// For query row r (token and query head) at position p, which sees the keys j <= p with
// j > p - window or j < sinks (all j <= p without a window):
//     s_rj = scale q_r.k_j,   o_r = sum_j 2^(t_rj - m_r) v_j / l_r,
//     t_rj = s_rj log2(e),    l_r = sum_j 2^(t_rj - m_r)
// over 128-key tiles with a running reference m_r, on CTA pairs with tcgen05, as the
// attention of packed prompts does it (attn_prefill.cu explains the pair's tile, its TMEM
// and shared memory, the softmax and the care for values that are not finite).  Weights are
// rounded to bf16 for the product with V, as there (2^-8 of sum w |v| at most; their sum l and O
// stay in fp32): pairs would double that product, half of a piece's time.  What is
// different here:
//
// Work.  (m, l, O) of disjoint sets of keys join by rescaling to the larger m.  So a pair's
// share is not tiles of queries but an equal part of all keys that tiles of queries go
// through, in (sequence, KV head, tile) order: single tokens over long caches and long
// prompts fill the GPU alike, and the last wave of tiles costs nothing (2,048 tokens on
// 16,000 keys 254 to 264 us, where whole tiles take 260 to 272; 2 tokens on 16,000 keys 22
// us for 139).  The counts before a tile
// are sums of max(0, x + i n) over its number i, which has a closed form, so each pair finds
// its share by itself.  A tile of queries that several pairs go through is joined by a
// second kernel, from (m, l, O) in the workspace, in the order of the pairs.
//
// Keys.  With a window a piece of work goes through the key tiles of the first keys, then
// those from the window's first one on.  Tiles of which some row does not see some key are
// edge tiles (masks; V looked through).  A position without a page is masked like them: a
// warp that brings K or V notes which eights of a tile's keys have no page.  Pages of which no
// query sees a key (before the window's first one, a tile starts at a multiple of 128) are not
// looked up: they may be gone.
//
// bf16 rows come by TMA, up to 64 keys of a page at a time.  Pages of 16 keys cost 1 to 2 %,
// of 8 keys 20 %: the copies are asked for one by one, and K and V have a warp each for it
// (with one warp for both 2,000 tokens on 11,011, heads of 128, pages of 16, took 324 us
// for 229).
//
// e4m3 rows are widened to bf16 (exact: a row's unit is a power of two), once for all tiles
// of queries of a sequence, by a kernel before this one, where the sequence has kWideTiles or
// more and the workspace has room; else by two warps for K and two for V, from codes that
// they copy for themselves into the swizzled tiles that the products read.  Bound by those
// warps: 58 instructions for 16 codes of a lane at one warp a scheduler, and by where they come
// from (see there): a key tile takes 1.3 us at D = 128 and 2.1 at 256, its products 0.7 and 1.4.
//
// Measured, calls back to back (both kernels; "floor" is the larger of bytes at a plain
// copy's rate and flops at a plain product's burst rate).  bf16: 2,048 tokens on 16,000
// keys, 16 heads of 256 on 2, 254 to 290 us by the board's power, floor 261; 4,000 on 20,000
// in a window of 4,096 188 to 200 us, floor 140 (a tile's window spans 34 or 35 key tiles for
// 32 of keys, three of them edge tiles, and a tile of queries costs 12 us beside its key tiles);
// 512 on 6,000 beside 24 single tokens, 32 heads of 128 on 8, 101 us, floor 53 (products of
// 256 rows for the single tokens' four, as long as their rows take to come, and neither under
// the other); 32 tokens on 131,072 69 us, floor 41; five on a million 315 us, 6.5 TB/s; 28
// tokens of eight sequences on up to 4,090 keys 19 us (latency: 7 us from the start to
// the first scores, 4 of the join).  e4m3: 2,000 on 11,011, 32 heads of 128 on 8, 243 us,
// floor 171 (409 widened by each tile of queries); 8 on 131,072 and 60,001 99 us, floor 29; 64
// single tokens in a window of 2,048 83 us, floor 19 (over bf16 rows 61 us).
#include <cuda.h>
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "attn_common.cuh"
#include "attn_params.h"
#include "attn_tc.cuh"
#include "params.h"
#include "per_device.h"
#include "rows.cuh"

namespace gdn {
namespace {

constexpr int kKeys = 128;          // keys a tile
constexpr int kRows = 128;          // rows a CTA
constexpr int kSoftmaxThreads = 256, kEpilogueWarp = 8, kTmaWarp = 12, kMmaWarp = 13, kScheduleWarp = 14, kEdgeWarp = 15;
constexpr int kThreads = 512;
constexpr uint32_t kBarSoftmax = 1;  // named barrier of the softmax warps
constexpr int kWideners = 2;         // warps of a CTA that write its half of K of an e4m3 tile, or of V
constexpr int kNoted = 8;            // key tiles whose missing pages are noted

// Work, in keys: a tile of queries counts the keys that its rows see, and kTileCost for
// taking it up (Q in, the first scores, O out): 512 tokens on 6,000 beside 24 single ones took
// 128 us with 128, 116 with 256, 106 with 384, 107 with 640.  A share is at least kMinShare: 28
// tokens on up to 4,090 keys took 22.8 us with 384, 24.1 with 768, 29.3 with 1,536.
constexpr int kTileCost = 384, kMinShare = 384;
// Over e4m3 rows a key counts more in tiles of queries that widen it for themselves (at times
// the time: 1.3 us a key tile of 128 at D = 128, 2.1 at 256) than in those that find it widened
// (0.8, 1.2): 512 tokens on 6,000 beside 24 single ones 156 us, all alike 177.
constexpr int kNarrowWeight = 7, kWideWeight = 4;
// e4m3 rows of a sequence with at least so many tiles of queries are widened once, into the
// workspace, where there is room (it writes and reads back four bytes a code, and is a kernel
// more).  Once, or by each tile: tiles of 64 tokens on 11,011 rows of 8 heads of
// 128: three 52, 57 us, four 60, 70, thirty-two 242, 410; of 32 tokens on 16,000 rows of 2 heads of
// 256: three 47, 43, four 47, 48, five 51, 54; three on 1,500 rows of 8 heads of 128 28, 23.
constexpr int kWideTiles = 4;

template <int D, bool kFp8>
struct Cfg {
  // Softmax warps, score tiles and slots as in the attention of packed prompts
  // (attn_prefill.cu): at D = 256 all eight on one key tile, at D = 128 two groups in turn.
  static constexpr int kGroups = D == 256 ? 1 : 2, kHalves = D == 256 ? 2 : 1;
  static constexpr int kCols = kKeys / kHalves;  // scores a thread
  static constexpr int kS = D == 256 ? 2 : 3;
  static constexpr int kLag = kS - 1;  // key tiles that the scores are ahead of P V
  static constexpr int kPWarps = 4 * kHalves;  // warps that write P of a key tile
  static constexpr int kArrivals = kFp8 ? kWideners : 1;  // that make K or V of a key tile full, beside bytes
  // and V of an edge tile, in the even CTA: for the odd CTA's warps its edge warp arrives
  static constexpr int kEdgeArrivals = kFp8 ? kWideners + 1 : 1;
  // Registers of a thread of the four warpgroups: softmax (two), epilogue, and the rest;
  // together the 65,536 that the CTA starts with, of which a thread has 128.  What widens e4m3
  // rows spills with fewer than all of those (64 tokens on 9,000 positions each, 112 212 us, 128
  // 204), the softmax with fewer than 152 at D = 128 (2,000 tokens on 11,011: 144 248 us, 152 242).
  static constexpr int kSoftmaxRegs = !kFp8 ? 168 : D == 256 ? 144 : 152, kEpilogueRegs = kFp8 ? 128 : 88;
  static constexpr int kOtherRegs = 512 - 2 * kSoftmaxRegs - kEpilogueRegs;
  static_assert(kSoftmaxRegs >= 128 && kEpilogueRegs <= 128 && kOtherRegs <= 128, "more, and fewer");
  static constexpr int kOut = 32;  // columns of O that the epilogue holds
  static constexpr uint32_t kQBytes = kRows * D * 2;
  static constexpr uint32_t kEntry = 64 * D * 2;  // half of K (64 keys) or of V (D / 2 dims)
  static constexpr int kSlots = D == 256 ? 2 : 4;  // key tiles of K, and of V, in shared memory
  static constexpr uint32_t kK = kQBytes, kV = kK + kSlots * kEntry;
  // Groups of e4m3 codes (2 KB) that a warp which widens them has under way.  D = 256, 5 tokens
  // on 131,072 positions: one 140 us, two 114, three (all that fits) 107; D = 128: two 165, four
  // 169.
  static constexpr int kDeep = D == 256 ? 3 : 2;
  // a warp's: 64 columns of o on their way out, and those codes
  static constexpr uint32_t kStageWarp = kFp8 ? kDeep * 2048 : 32 * 128;
  static_assert(kStageWarp >= 32 * 128, "64 columns of o");
  static constexpr uint32_t kStage = kV + kSlots * kEntry;
  static constexpr uint32_t kShared = kStage + 4 * kStageWarp;  // the barriers and the rest
  static constexpr int kSteps = D / 16;
  static constexpr uint32_t kTmemO = kS * kKeys;
  static constexpr uint32_t kTmemCols = 512;
  static_assert(kTmemO + D <= kTmemCols, "TMEM");
};

// ------------------------------------------------------------------ work
// a table's entry, or another value; without a branch, behind which it would be waited for
__device__ __forceinline__ int load_if(const int32_t* src, bool valid, int other) {
  int x;
  asm("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\tmov.b32 %0, %3;\n\t@p ld.global.nc.b32 %0, [%1];\n\t}"
               : "=&r"(x)
               : "l"(src), "r"((int)valid), "r"(other));
  return x;
}
// One sequence's queries and keys (bad ones have no queries; recorded once).
struct Seq {
  int q0, a, off, tiles;  // first row of q, queries, keys before the first of them, tiles of queries
};
// One piece of a pair's work: keys of a tile of queries; count < 0 ends the schedule
struct Piece {
  int32_t token, left;  // first row of q of the pair's; queries of the sequence from there
  int32_t pos;          // its position (may be < 0)
  int32_t seq, kvh;
  int32_t sight;       // keys that the last row sees (its position + 1)
  int32_t firsts, w0;  // key tiles that hold the first keys; number of the window's first one
  int32_t v0, count;   // key tiles to go through, of both in this order
  int32_t part;        // where its partial result goes (0, 1), or -1: all of the tile's keys
  int32_t wide;        // row of the widened copy that holds position 0, or -1
};

template <bool kFp8>
struct Work {
  int64_t window, reach;  // reach = window + sinks
  int sinks;
  Divisor tokens;  // of a pair
  __device__ __forceinline__ explicit Work(const PagedPrefillArgs& p)
      : window(p.window), reach((int64_t)p.window + p.sinks), sinks(p.window ? p.sinks : 0),
        tokens(p.tile, p.tile_inv) {}

  __device__ __forceinline__ Seq sequence(const PagedPrefillArgs& p, int n, bool report) const {
    Seq s{0, 0, 0, 0};
    const bool valid = n < p.num_seqs;
    const int q0 = load_if(p.cu_q + n, valid, 0), q1 = load_if(p.cu_q + n + 1, valid, 0);
    int len = load_if(p.cache_len + n, valid, 0);
    const bool bad = q0 < 0 || q1 < q0 || q1 > p.total_q;
    const bool open = (n == 0 && q0 != 0) || (n == p.num_seqs - 1 && q1 != p.total_q);
    const bool beyond = len < 0 || (int64_t)len > ((int64_t)p.cache.max_pages << p.cache.page_shift);
    if (report && (bad || open)) raise_error(p.err, kErrBadCuSeqlens);
    if (report && beyond) raise_error(p.err, kErrBadCacheLen);
    if (bad) return s;
    if (beyond) len = 0;
    s.q0 = q0;
    s.a = q1 - q0;
    s.off = len - s.a;
    s.tiles = s.a > 0 ? tokens.divide(s.a - 1) + 1 : 0;
    return s;
  }
  // of a sequence's keys (whether there is room to widen them or not, so that the same shares
  // and results come out), and of kMinShare's
  __device__ __forceinline__ int weight(const Seq& s) const {
    return !kFp8 ? 1 : s.tiles >= kWideTiles ? kWideWeight : kNarrowWeight;
  }
  __device__ __forceinline__ int unit() const { return kFp8 ? kNarrowWeight : 1; }
  // sum over i < m of max(0, x + i tokens)
  __device__ __forceinline__ int64_t ramp(int64_t x, int m) const {
    if (m <= 0 || x + (int64_t)(m - 1) * tokens.d <= 0) return 0;
    // (-x < m tokens, which a sequence's queries bound)
    const int k = x >= 0 ? 0 : (int)tokens.divide((uint32_t)(-x + tokens.d - 1));
    const int64_t n = m - k;
    return n * (x + (int64_t)k * tokens.d) + tokens.d * (n * (n - 1) / 2);
  }
  // of the first m tiles of a sequence, for one KV head
  __device__ __forceinline__ int64_t before(const Seq& s, int m) const {
    int64_t x = ramp((int64_t)s.off + tokens.d, m);
    if (m > 0 && m == s.tiles)
      x -= max((int64_t)0, s.off + (int64_t)m * tokens.d) - max((int64_t)0, (int64_t)s.off + s.a);
    if (window) x -= ramp((int64_t)s.off + 1 - reach, m);
    return weight(s) * (x + (int64_t)m * kTileCost);
  }
  // keys that tile i counts
  __device__ __forceinline__ int64_t keys(const Seq& s, int i) const {
    const int64_t first = (int64_t)i * tokens.d, last = min((int64_t)s.a, first + tokens.d);
    const int64_t x = max((int64_t)0, s.off + last);
    return window ? x - max((int64_t)0, s.off + first + 1 - reach) : x;
  }
  __device__ __forceinline__ Piece piece(const Seq& s, int seq, int kvh, int i) const {
    Piece t;
    const int first = i * tokens.d;
    t.token = s.q0 + first;
    t.left = s.a - first;
    t.pos = s.off + first;
    t.seq = seq;
    t.kvh = kvh;
    t.sight = max(0, t.pos + min(t.left, tokens.d));
    const int lo = window ? (int)max((int64_t)0, t.pos + 1 - window) : 0;
    t.w0 = lo / kKeys;
    t.firsts = (int)min((int64_t)t.w0, ((int64_t)sinks + kKeys - 1) / kKeys);
    t.v0 = 0;
    t.count = t.firsts + (t.sight + kKeys - 1) / kKeys - t.w0;
    t.part = t.wide = -1;
    return t;
  }
  // rows of the widened copy that a sequence takes
  __device__ __forceinline__ int64_t wide(const PagedPrefillArgs& p, const Seq& s) const {
    return p.wide_rows > 0 && s.tiles >= kWideTiles ? (int64_t)s.off + s.a : 0;
  }
  // how many of a tile's `count` key tiles lie before work r of it, at `weight` a key
  __device__ __forceinline__ int visits(int64_t r, int64_t keys, int weight, int count) const {
    r -= weight * kTileCost;
    keys *= weight;
    return r <= 0 ? 0 : r >= keys ? count : (int)quotient(r * count, keys);
  }
};
// What a pair leaves for the joining pass: which of its parts there are, and the tile of
// queries that it has started and not finished (rows 0: none), whose keys pairs up to `last`
// go through.
struct alignas(16) Join {
  int32_t there[2];
  int32_t last, rows;
  int32_t token, head;  // the tile's first row of q, and query head
  int32_t unused[2];
};
// what the sequences come to, and where a share starts
struct Found {
  int64_t total, base;  // all work, that before sequence seq
  int64_t wide;         // rows of the widened copy that the sequences before it take
  int64_t work;         // of it, all heads
  int seq;
  Seq s;
};

// A place in the work: tile i of KV head kvh of sequence n, which starts at `start`.
struct Place {
  Seq s;
  int n, kvh, i;
  int64_t start, end;           // (end: -1 before it is known)
  int64_t u0, u, u_end, total;  // of a share: where it starts, is and ends; all work
  int64_t wide;                 // rows of the widened copy before the sequence's
  int there;                    // which of its two parts there are, as bits
  template <class W>
  __device__ __forceinline__ void find(const PagedPrefillArgs& p, const W& w, const Found& f, int64_t u, int lane) {
    n = f.seq;
    wide = f.wide;
    s = f.s;
    const int64_t head = quotient(f.work, p.cache.h_kv);
    kvh = (int)quotient(u - f.base, head);
    const int64_t at = f.base + kvh * head;
    // the last tile that starts at u or before: 32 probes a step
    int lo = 0, hi = s.tiles;
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32, m = lo + lane * step;
      const unsigned below = __ballot_sync(kFullMask, m < hi && w.before(s, m) <= u - at);
      lo += (__popc(below) - 1) * step;
      hi = min(hi, lo + step);
    }
    i = lo;
    start = at + (i > 0 ? w.before(s, i) : 0);
  }
  template <class W>
  __device__ __forceinline__ void next(const PagedPrefillArgs& p, const W& w, int lane) {
    start = end;
    if (++i < s.tiles) return;
    i = 0;
    if (++kvh < p.cache.h_kv) return;
    kvh = 0;
    wide += w.wide(p, s);
    for (++n; n < p.num_seqs; n += 32) {  // the next one with queries, 32 at a time
      const Seq mine = w.sequence(p, n + lane, false);
      const unsigned some = __ballot_sync(kFullMask, mine.tiles > 0);
      if (some == 0) continue;
      const int src = __ffs(some) - 1;
      n += src;
      s.q0 = __shfl_sync(kFullMask, mine.q0, src);
      s.a = __shfl_sync(kFullMask, mine.a, src);
      s.off = __shfl_sync(kFullMask, mine.off, src);
      s.tiles = __shfl_sync(kFullMask, mine.tiles, src);
      return;
    }
  }
};

// The share of pair c: false when there is none.  Up to kFew sequences are counted by the
// schedule's warp alone (64 of them: 2 us; by the block, which meets twice, 6.6), more by the
// whole block.
constexpr int kFew = 256;
template <class W>
__device__ __forceinline__ int sharers(const W& w, int64_t total, int pairs) {
  return (int)min((int64_t)pairs, max((int64_t)1, quotient(total, w.unit() * kMinShare)));
}
__device__ __forceinline__ int64_t scan_up(int64_t x, int lane) {
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t y = __shfl_up_sync(kFullMask, x, off);
    if (lane >= off) x += y;
  }
  return x;
}
// total, and the sequence that holds work u of share c (its first piece of work)
template <class W>
__device__ __forceinline__ bool find_few(const PagedPrefillArgs& p, const W& w, int c, bool report, int lane, Found* f) {
  const int per = (p.num_seqs + 31) / 32;  // sequences a lane counts
  int n = lane * per;
  auto work_of = [&](const Seq& s) { return s.tiles > 0 ? p.cache.h_kv * w.before(s, s.tiles) : 0; };
  Seq s = w.sequence(p, n, report);  // of the lane's, the first
  int64_t x = work_of(s);
  int64_t mine = x, rows = w.wide(p, s);
  for (int i = 1; i < per; ++i) {
    const Seq more = w.sequence(p, n + i, report);
    mine += work_of(more);
    rows += w.wide(p, more);
  }
  const int64_t incl = scan_up(mine, lane);
  f->total = __shfl_sync(kFullMask, incl, 31);
  const int sharing = sharers(w, f->total, p.pairs);
  if (f->total == 0 || c >= sharing) return false;
  const int64_t u = Shares(f->total, sharing).start(c);
  int64_t base = incl - mine, wide = p.wide_rows > 0 ? scan_up(rows, lane) - rows : 0;
  const int src = __ffs(__ballot_sync(kFullMask, incl > u)) - 1;
  if (lane == src) {
    while (u >= base + x) {  // (it is one of the lane's)
      base += x;
      wide += w.wide(p, s);
      s = w.sequence(p, ++n, false);
      x = work_of(s);
    }
  }
  f->seq = __shfl_sync(kFullMask, n, src);
  f->base = __shfl_sync(kFullMask, base, src);
  f->wide = __shfl_sync(kFullMask, wide, src);
  f->work = __shfl_sync(kFullMask, x, src);
  f->s.q0 = __shfl_sync(kFullMask, s.q0, src);
  f->s.a = __shfl_sync(kFullMask, s.a, src);
  f->s.off = __shfl_sync(kFullMask, s.off, src);
  f->s.tiles = __shfl_sync(kFullMask, s.tiles, src);
  return true;
}
struct Sums {  // the block's, for this
  int64_t of[16], rows[16];
  Found found;
};
template <int kT, class W>
__device__ __noinline__ bool find_many(const PagedPrefillArgs& p, const W& w, int c, bool report, Sums& sh, Found* f) {
  static_assert(kT <= 512, "sums");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.num_seqs - 1) / kT + 1;  // sequences a thread counts
  const int lo = (int)min((int64_t)p.num_seqs, (int64_t)tid * per), hi = (int)min((int64_t)p.num_seqs, (int64_t)lo + per);
  int64_t mine = 0, rows = 0;
  for (int n = lo; n < hi; ++n) {
    const Seq s = w.sequence(p, n, report);
    if (s.tiles > 0) mine += p.cache.h_kv * w.before(s, s.tiles);
    rows += w.wide(p, s);
  }
  const int64_t incl = scan_up(mine, lane), rows_incl = scan_up(rows, lane);
  if (lane == 31) {
    sh.of[warp] = incl;
    sh.rows[warp] = rows_incl;
  }
  __syncthreads();
  int64_t before = incl - mine, total = 0, wide = rows_incl - rows;
#pragma unroll
  for (int k = 0; k < kT / 32; ++k) {
    if (k < warp) {
      before += sh.of[k];
      wide += sh.rows[k];
    }
    total += sh.of[k];
  }
  const int sharing = sharers(w, total, p.pairs);
  if (total == 0 || c >= sharing) return false;  // (for all threads alike)
  const int64_t u = Shares(total, sharing).start(c);
  if (before <= u && u < before + mine) {
    for (int n = lo; n < hi; ++n) {
      const Seq s = w.sequence(p, n, false);
      const int64_t x = s.tiles > 0 ? p.cache.h_kv * w.before(s, s.tiles) : 0;
      if (u < before + x) {
        sh.found.seq = n;
        sh.found.base = before;
        sh.found.wide = wide;
        sh.found.work = x;
        sh.found.s = s;
        break;
      }
      before += x;
      wide += w.wide(p, s);
    }
  }
  __syncthreads();
  *f = sh.found;
  f->total = total;
  return true;
}

__device__ __forceinline__ Join* joins(const PagedPrefillArgs& p) {  // of the pairs, behind the parts
  return reinterpret_cast<Join*>(p.partial + (int64_t)kPagedPrefillMaxPairs * 2 * (2 * kRows * (p.cache.head_dim + 2)));
}

// Key tile j of a piece: its first key, how many of its keys some row may see, and whether
// some row does not see some of those (or the tile ends behind them).
struct Keys {
  int first, rows;
  bool edge;
};
__device__ __forceinline__ Keys key_tile_of(const Piece& t, int j, int window, int sinks) {
  Keys k;
  const int v = t.v0 + j;
  const bool firsts = v < t.firsts;
  k.first = (firsts ? v : t.w0 + v - t.firsts) * kKeys;
  k.rows = min(kKeys, (firsts ? sinks : t.sight) - k.first);
  const int whole = t.pos + 1;  // keys that every row sees, but for the window
  const int low = window ? max(0, t.sight - window) : 0;  // first key of the last row's window
  k.edge = k.first + kKeys > whole || max(k.first, sinks) < min(k.first + kKeys, low);
  return k;
}
// Which rows of an edge tile's V may need care (the others, every row of queries sees): those
// before the window of the last one, and those after the position of the first, in sixteens.
struct Care {
  int before, from;
};
__device__ __forceinline__ Care care_of(const Piece& t, const Keys& k, int window, int sinks) {
  const int low = window ? max(0, t.sight - window) : 0;
  Care c;
  c.before = max(k.first, sinks) < min(k.first + kKeys, low) ? low - k.first : 0;
  c.from = max(0, t.pos + 1 - k.first) & ~15;
  return c;
}
// how many of a piece's key tiles are edge tiles, for a warp that does not go through them
__device__ __forceinline__ int edges_of(const Piece& t, int window, int sinks, int lane) {
  int n = 0;
  for (int j = lane; j < t.count; j += 32) n += key_tile_of(t, j, window, sinks).edge;
  return __reduce_add_sync(kFullMask, n);
}
__device__ __forceinline__ uint32_t lowest(int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1; }

template <int D, bool kFp8>
struct Shared {  // beside the tiles
  using C = Cfg<D, kFp8>;
  // by key tile h: K, V of h % kSlots are there; the scores of h, the product with V
  // of h are done (h % kSlots; this frees their slots too); P of h is in TMEM (h % kS)
  uint64_t k_full[C::kSlots], v_full[C::kSlots], s_done[C::kSlots], o_done[C::kSlots], p_ready[C::kS];
  uint64_t q_full, q_empty, o_free;
  uint64_t m_ready[2][4];  // two groups: a key tile's references are in m, by quarters of the rows
  // edge tiles, counted through (% kSlots): V is there in both CTAs; is finite there
  uint64_t v_edge[C::kSlots], v_clean[C::kSlots];
  uint64_t sums_in[2];     // the rows' sums of two pieces are there, for the epilogue
  uint64_t noted[kNoted];  // groups of key tile h (% kNoted) are there
  // What was found in V in the edge tiles of a piece (by number & 3): the number + 1 where
  // that was a non-finite value; that this has been told.
  uint64_t flags_in[4];
  uint32_t poison[4];
  uint64_t tile_full[2], tile_empty[2], drained;
  uint64_t copy_v[2];  // e4m3: V of a piece (by number & 1) may be copied
  Piece tile[2], late[4];
  uint32_t tmem, failed;
  Sums work;
  Place place;
  uint32_t groups[kNoted];  // which eights of a key tile's keys have a page
  // halves: the row maxima of a key tile's halves, two key tiles; groups: the
  // references of two key tiles
  float red[2][2][128];
  float sums[2][2][128];  // row sums of two pieces, in two parts
  float refs[2][128];     // and the references that they go by
  // e4m3: what a warp of the odd CTA copies to say that its rows of a key tile are there (by
  // slots: the tile's number + 1), and in the even CTA what it has copied last
  alignas(16) uint32_t said[4][C::kSlots][4];
  uint32_t said_last[4][C::kSlots];
  alignas(16) uint8_t bytes[4][2][64];  // e4m3: exponent bytes of a warp's eights, two key tiles
};

// 16 bytes of this CTA's shared memory to the same place in the even CTA's, counted on a
// barrier there
__device__ __forceinline__ void tell(const void* what, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], 16, [%2];" ::"r"(
                   tc2::in_cta(what, 0)),
               "r"(tc::smem_u32(what)), "r"(tc2::in_cta(bar, 0))
               : "memory");
}
// 8 bytes from global to shared memory; zeros when !valid (nothing is read)
__device__ __forceinline__ void copy8(const void* dst, const void* src, bool valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(tc::smem_u32(dst)), "l"(src), "r"(valid ? 8 : 0)
               : "memory");
}
__device__ __forceinline__ void copy16(const void* dst, const void* src, bool valid) {  // the same of 16
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(dst)), "l"(src), "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// bytes 0 and 1 (kUpper: 2 and 3) of a word as two 16-bit integers, with their signs
template <bool kUpper>
__device__ __forceinline__ uint32_t signed_halves(uint32_t w) {
  uint32_t y;
  asm("prmt.b32 %0, %1, 0, %2;" : "=r"(y) : "r"(w), "n"(kUpper ? 0xb3a2 : 0x9180));
  return y;
}
// Sixteen e4m3 codes of a row, times its unit (up to 2^7 of it), as bf16 (exact).  A NaN code
// comes out as 480 units and raises the top bit of a byte of `odd`: see mend.
__device__ __forceinline__ void widen16(const uint4& x, uint32_t unit, uint4& lo, uint4& hi, uint32_t& odd) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t y[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    odd |= (w[i] & 0x7f7f7f7fu) + 0x01010101u;
    // two codes with their signs above them, shifted into place
    y[2 * i] = times((signed_halves<false>(w[i]) << 4) & (kMagnitude | kSigns), unit);
    y[2 * i + 1] = times((signed_halves<true>(w[i]) << 4) & (kMagnitude | kSigns), unit);
  }
  lo = make_uint4(y[0], y[1], y[2], y[3]);
  hi = make_uint4(y[4], y[5], y[6], y[7]);
}
// Eight of those where a NaN code or a unit above 2^7 has been seen: NaN for 480 units, and
// the rest of the unit.
__device__ __forceinline__ uint4 mend(const uint4& x, uint32_t byte) {
  const uint32_t nan = times(kMagnitude, value_units(byte, byte));
  uint32_t rest = byte > kUnitTop ? (byte - kUnitTop + 127) << 7 : 127u << 7;
  rest |= rest << 16;
  auto two = [&](uint32_t y) { return times(y, rest) | (__vcmpeq2(y & ~kSigns, nan) & 0x7fc07fc0u); };
  return make_uint4(two(x.x), two(x.y), two(x.z), two(x.w));
}

template <int D, bool kFp8>
__global__ void __launch_bounds__(kThreads, 1)
    attn_prefill_paged_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                              const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PagedPrefillArgs p) {
  using C = Cfg<D, kFp8>;
  extern __shared__ __align__(1024) uint8_t smem[];
  Shared<D, kFp8>& sh = *reinterpret_cast<Shared<D, kFp8>*>(smem + C::kShared);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = tc::cluster_rank();
  const int G = p.group;
  const int tok_cta = kRows / G;  // tokens a CTA
  const int window = p.window, sinks = window ? p.sinks : 0;
  if (warp == 0) {
    tc2::tmem_alloc(&sh.tmem, C::kTmemCols);
    tc2::tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < C::kSlots; ++i) {
      tc::mbar_init(&sh.k_full[i], C::kArrivals);
      tc::mbar_init(&sh.v_full[i], C::kArrivals);
      tc::mbar_init(&sh.s_done[i], 1);
      tc::mbar_init(&sh.o_done[i], 1);
    }
    tc::mbar_init(&sh.q_full, 1);
    tc::mbar_init(&sh.q_empty, 1);
    for (int i = 0; i < C::kS; ++i) tc::mbar_init(&sh.p_ready[i], 2 * C::kPWarps);
    for (int i = 0; i < 2; ++i) {
      for (int k = 0; k < 4; ++k) tc::mbar_init(&sh.m_ready[i][k], 1);
      tc::mbar_init(&sh.tile_full[i], 1);
      tc::mbar_init(&sh.copy_v[i], 1);
      tc::mbar_init(&sh.sums_in[i], 8);
      // readers: the softmax, epilogue and TMA warps, in the even CTA the products' and the edge
      // warp, in the odd one the edge warp over e4m3 rows
      tc::mbar_init(&sh.tile_empty[i], 13 + (rank == 0 ? 2 : kFp8 ? 1 : 0));
    }
    for (int i = 0; i < 4; ++i) {
      tc::mbar_init(&sh.flags_in[i], 1);
      sh.poison[i] = 0;
    }
    for (int i = 0; i < kNoted; ++i) tc::mbar_init(&sh.noted[i], 1);
    for (int i = 0; i < C::kSlots; ++i) {
      tc::mbar_init(&sh.v_edge[i], rank == 0 ? C::kEdgeArrivals : kWideners);
      tc::mbar_init(&sh.v_clean[i], 1);
    }
    tc::mbar_init(&sh.o_free, 2 * 4);
    tc::mbar_init(&sh.drained, 1);
    sh.failed = 0;
    tc::fence_mbar_init();
  }
  if (kFp8 && tid < 4 * C::kSlots) {
    sh.said[tid / C::kSlots][tid % C::kSlots][0] = 0;
    sh.said_last[tid / C::kSlots][tid % C::kSlots] = 0;
  }
  if (lane == 0 && warp == kTmaWarp) {
    tc::prefetch_tmap(&tm_q);
    tc::prefetch_tmap(&tm_k);
    tc::prefetch_tmap(&tm_v);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::cluster_sync();
  tc::fence_after_sync();
  const uint32_t tmem = sh.tmem;
  const uint32_t sbase = tc::smem_u32(smem);
  bool ok = true;
  tc::wait_prerequisites();  // q, the cache, its table, the offsets and lengths come from earlier kernels
  tc::allow_dependents();

  // ---- this pair's share, and its pieces one after the other (for the schedule warp)
  const Work<kFp8> work(p);
  const int me = blockIdx.x / 2;
  Found found{};
  bool any = false;
  if (p.num_seqs > kFew) any = find_many<kThreads>(p, work, me, blockIdx.x == 0, sh.work, &found);
  else if (warp == kScheduleWarp) any = find_few(p, work, me, blockIdx.x == 0, lane, &found);
  // (the schedule warp keeps its place in shared memory: between two pieces it copies V)
  auto next_piece = [&](Piece* t) {
    Place at = sh.place;
    __syncwarp();
    bool found_one = false;
    while (at.u < at.u_end && !found_one) {
      if (at.u == at.end) at.next(p, work, lane);
      const int64_t keys = work.keys(at.s, at.i), r0 = at.u - at.start;
      const int weight = work.weight(at.s);
      at.end = at.start + weight * (kTileCost + keys);
      at.u = min(at.end, at.u_end);
      *t = work.piece(at.s, at.n, at.kvh, at.i);
      const int64_t rows = kFp8 ? work.wide(p, at.s) : 0;
      t->wide = rows > 0 && at.wide + rows <= p.wide_rows ? (int32_t)at.wide : -1;
      const int all = t->count, v0 = work.visits(r0, keys, weight, all), v1 = work.visits(at.u - at.start, keys, weight, all);
      t->v0 = v0;
      t->count = v1 - v0;
      if (t->count < all) t->part = r0 > 0 ? 0 : 1;
      if (t->part >= 0 && t->count > 0) at.there |= 1 << t->part;
      found_one = t->count > 0 || (all == 0 && r0 == 0);
    }
    if (!found_one) t->count = -1;
    if (lane == 0) sh.place = at;
    __syncwarp();
    return found_one;
  };
  if (warp == kScheduleWarp) {
    Place at;
    at.u = at.u_end = 0;
    at.end = -1;
    at.there = 0;
    if (any) {
      const Shares shares(found.total, sharers(work, found.total, p.pairs));
      at.total = found.total;
      at.u0 = at.u = shares.start(me);
      at.u_end = shares.start(me + 1);
      at.find(p, work, found, at.u, lane);
    }
    if (lane == 0) sh.place = at;
    __syncwarp();
    Piece t;
    next_piece(&t);
    if (lane == 0) {
      sh.tile[0] = t;
      tc::mbar_arrive(&sh.tile_full[0]);
    }
    __syncwarp();
  }

  // wait for what a barrier by key tile says of key tile h
  auto of_tile = [&](uint64_t* bars, int h) { return tc::mbar_wait(&bars[h % C::kSlots], (h / C::kSlots) & 1); };

  // The warp's next piece (pass counts them); false at the end or when a wait expired.
  auto next_tile = [&](int pass, Piece* t) {
    const bool w = __all_sync(kFullMask, tc::mbar_wait(&sh.tile_full[pass & 1], (pass >> 1) & 1));
    if (!w) {
      ok = false;
      return false;
    }
    *t = sh.tile[pass & 1];
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&sh.tile_empty[pass & 1]);
    return t->count >= 0;
  };
  // Whether key `key` of a tile that starts before the window of the first row, or of the first
  // keys, is in a page of which some row sees a key: a page that nobody sees need not be there.
  const int shift = p.cache.page_shift;
  auto seen_page = [&](const Piece& t, int key) {
    const int low = window && t.pos >= window ? t.pos + 1 - window : 0;  // first key of the window
    return (key | ((1 << shift) - 1)) >= low || key >> shift << shift < sinks;
  };
  // Whether the warp's lanes look key `first` + `eight` of key tile k up.
  auto wanted = [&](const Piece& t, const Keys& k, int eight) {
    return eight < k.rows && seen_page(t, k.first + eight);
  };
  // The page table's entry for key `key` (-1 where there is none), and the key's cached row (~0
  // without a page).
  auto entry_of = [&](const Piece& t, int key, bool wanted) {
    return load_if(p.cache.table + (int64_t)t.seq * p.cache.max_pages + (key >> shift),
                   wanted && (key >> shift) < p.cache.max_pages, -1);
  };
  auto row_of = [&](const Piece& t, int key, int page) {
    return page >= 0 && page < p.cache.num_pages
               ? (((uint32_t)page * p.cache.h_kv + t.kvh) << shift) + (key & ((1 << shift) - 1))
               : ~0u;
  };

  // For the warp that brings K of key tile h, or over e4m3 rows V (which has less to do): which
  // eights of its keys have no page.  (It has waited for the scores of h - kSlots, or the product
  // with V, before which the softmax was through with h - kNoted.)
  auto note = [&](int h, bool missing) {
    const uint32_t gone = __ballot_sync(kFullMask, missing) & 0xffffu;
    if (lane == 0) {
      if (gone && rank == 0) raise_error(p.err, kErrBadPage);
      sh.groups[h % kNoted] = 0xffffu & ~gone;
      tc::mbar_arrive(&sh.noted[h % kNoted]);
    }
  };

  if (warp < kEpilogueWarp) {
    tc2::more_registers<C::kSoftmaxRegs>();
    // ------------------------------------------------------------ softmax
    Piece t;
    int used = 0, g = 0;
    const int part = warp >> 2, row = (warp & 3) * 32 + lane;
    const int grp = C::kGroups > 1 ? part : 0, half = C::kHalves > 1 ? part : 0;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    // (scale 0: all scores alike, by the smallest factor that keeps a masked score infinite:
    // 2^-149, with which the largest product is 2^-21)
    const float c = p.scale == 0.f ? __uint_as_float(1) : p.scale * kLog2e;
    const bool down = c < 0.f;  // the largest score is then the smallest product
    const uint32_t r_p = tc2::in_cta(sh.p_ready, 0);
    bool carried = true;  // no wait expired since the last barrier of these warps
    for (int pass = 0;; ++pass) {
      // all softmax warps go on or none: they meet at barriers without a limit
      const bool more = next_tile(pass, &t);
      if (!(ok = tc::named_sync_and(kBarSoftmax, kSoftmaxThreads, ok && carried)) || !more) break;
      const int tok = (int)rank * tok_cta + row / G;
      const bool real = row < tok_cta * G && tok < t.left;
      const int lim = real ? max(0, t.pos + tok + 1) : 0;   // keys this row sees,
      const int low = window ? max(0, lim - window) : 0;  // from this one, and the first ones
      const bool idle = !__any_sync(kFullMask, real);  // no queries: their P may be anything
      float m = -INFINITY, l = 0.f;
      // with two groups, this one takes every other key tile (g counts them through)
      auto key_tile = [&](int j) {
        const int h = g + j, sb = h % C::kS;
        const Keys keys = key_tile_of(t, j, window, sinks);
        const int key0 = keys.first;
        // (there before the scores: what follows from the tile alone is done in their shadow)
        bool w = carried && tc::mbar_wait(&sh.noted[h % kNoted], (h / kNoted) & 1);
        const uint32_t paged = sh.groups[h % kNoted];
        const bool masked = (keys.edge || paged != 0xffffu) && !idle;
        w = w && of_tile(sh.s_done, h);
        tc::fence_after_sync();
        w = __all_sync(kFullMask, w);
        const float none = down ? INFINITY : -INFINITY;
        const uint32_t scores = tmem + lanes + sb * kKeys + C::kCols * half;
        // the upper 64 of 128 columns only if some row sees them, as the product with V
        // takes no more
        const bool upper = C::kCols > 64 && keys.rows > 64;
        const int cols = upper ? C::kCols : 64;
        if (masked) {
          // The scores that a row does not see are overwritten, in one short loop before code
          // that all tiles share.
          const int left = lim - key0 - C::kCols * half;  // columns of this thread up to the row's last,
          const int from = low - key0 - C::kCols * half;  // from the window's first,
          const int first = sinks - key0 - C::kCols * half;  // and up to the first keys' last
          const bool all = paged == 0xffffu && __all_sync(kFullMask, from <= 0 || !real);  // no other bound
          const int skip = all ? max(0, __reduce_min_sync(kFullMask, left)) & ~31 : 0;
#pragma unroll 1
          for (int k = skip; k < cols; k += 32) {
            uint32_t see = lowest(left - k) & (~lowest(from - k) | lowest(first - k));
            if (paged != 0xffffu) {
              const uint32_t eights = paged >> ((k + C::kCols * half) >> 3);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (!((eights >> i) & 1)) see &= ~(0xffu << (8 * i));
            }
            float x[32];
            tc::tmem_ld32(scores + k, x);
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = (see >> i) & 1 ? x[i] : none;
            tc::tmem_st32(scores + k, x);
          }
        }
        float s[64];  // 64 of the thread's scores
        auto fetch = [&](int k) { tc2::tmem_ld(scores + k, s); };
        float x = none;
        if (!idle) {
          if (upper) {
            fetch(64);
            x = down ? least(s) : largest(s);
          }
          fetch(0);
          const float x0 = down ? least(s) : largest(s);
          x = C::kCols > 64 ? (down ? fminf(x, x0) : fmaxf(x, x0)) : x0;
        }
        float now = m;  // the row's reference, which O and the tiles before go by
        if (C::kHalves > 1) {
          float(&red)[2][128] = sh.red[h & 1];
          red[half][row] = x;
          tc::fence_before_sync();
          if (!(ok = tc::named_sync_and(kBarSoftmax, kSoftmaxThreads, w))) return;
          tc::fence_after_sync();
          const float y = red[half ^ 1][row];
          x = down ? fminf(x, y) : fmaxf(x, y);
        } else {
          carried = w;
          if (j > 0) {
            carried = __all_sync(kFullMask, carried && tc::mbar_wait(&sh.m_ready[(h - 1) & 1][warp & 3], ((h - 1) >> 1) & 1));
            now = sh.red[(h - 1) & 1][0][row];
          }
        }
        // Rows that are no queries hold other rows' q or what was there before: they never
        // move a reference, and neither does one that is NaN already
        const bool any = real && x != (down ? INFINITY : -INFINITY);
        const float top = any ? x * c : -INFINITY;
        const float next = top > now + kSlack || now == -INFINITY ? top : now;
        const bool grow = next != now && now == now;
        if (C::kGroups > 1) {
          sh.red[h & 1][0][row] = next;
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&sh.m_ready[h & 1][warp & 3]);
        }
        if (j > 0 && __any_sync(kFullMask, grow)) {  // O holds the tiles before: rescale it
          const bool v = __all_sync(kFullMask, of_tile(sh.o_done, h - 1));
          tc::fence_after_sync();
          const float f = now == -INFINITY ? 0.f : ex2(now - next);
          if (v) {
#pragma unroll
            for (int i = 0; i < D / 32 / C::kHalves; ++i) {
              float ov[32];
              const uint32_t at = tmem + lanes + C::kTmemO + half * (D / 2) + 32 * i;
              tc::tmem_ld32(at, ov);
              if (grow) {
#pragma unroll
                for (int k = 0; k < 32; ++k) ov[k] *= f;
              }
              tc::tmem_st32(at, ov);
            }
          }
          carried = carried && v;
        }
        if (next != m) {
          l *= m == -INFINITY ? 0.f : ex2(m - next);
          m = next;
        }
        if (!idle) {
          const float ref = m == -INFINITY ? 0.f : m;
          const float2 c2 = make_float2(c, c), r2 = make_float2(-ref, -ref);
          float2 l0 = make_float2(0.f, 0.f), l1 = l0;
#pragma unroll
          for (int k = 0; k < C::kCols; k += 64) {
            if (k > 0) {
              if (!upper) break;
              fetch(k);
            }
            uint32_t pk[32];
#pragma unroll
            for (int i = 0; i < 64; i += 4) {
              float2 p0 = tc2::fma2(make_float2(s[i], s[i + 1]), c2, r2);
              float2 p1 = tc2::fma2(make_float2(s[i + 2], s[i + 3]), c2, r2);
              p0 = make_float2(ex2(p0.x), ex2(p0.y));
              p1 = make_float2(ex2(p1.x), ex2(p1.y));
              l0 = tc2::add2(l0, p0);
              l1 = tc2::add2(l1, p1);
              pk[i / 2] = pack_bf16(p0.x, p0.y);
              pk[i / 2 + 1] = pack_bf16(p1.x, p1.y);
            }
            tc2::tmem_st(scores + k, pk);  // over scores that are done with
          }
          l0 = tc2::add2(l0, l1);
          l += l0.x + l0.y;
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc2::arrive_remote_relaxed(r_p + sb * 8);
      };
      for (int j = C::kGroups > 1 ? (g ^ grp) & 1 : 0; j < t.count && ok; j += C::kGroups) key_tile(j);
      // ---- the pair's rows are through their keys: their sums go to the epilogue
      if (t.count > 0) {
        if (C::kGroups > 1) {
          const int h = g + t.count - 1;
          carried = carried && tc::mbar_wait(&sh.m_ready[h & 1][warp & 3], (h >> 1) & 1);
          const float last = sh.red[h & 1][0][row];  // of the last tile, which O goes by
          if (m != last) l *= m == -INFINITY ? 0.f : ex2(m - last);
          m = last;
        }
        sh.sums[used & 1][part][row] = l;
        if (part == 0) sh.refs[used & 1][row] = m;
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sh.sums_in[used & 1]);
        g += t.count;
        ++used;
      }
    }
  } else if (warp < kTmaWarp) {
    tc2::fewer_registers<C::kEpilogueRegs>();
    // ------------------------------------------------------------ epilogue, and widening of e4m3 rows
    const int wq = warp & 3, row = wq * 32 + lane;
    const uint32_t lanes = (uint32_t)(wq * 32) << 16;
    const uint32_t r_free = tc2::in_cta(&sh.o_free, 0);
    // 32 rows of 128 bytes for each warp, 16-byte pieces c of row r at c ^ (r & 7)
    uint8_t* stage = smem + C::kStage + wq * C::kStageWarp;
    // O of piece t, the used'th with keys, whose last key tile is h
    auto epilogue = [&](const Piece t, int used, int h) {
      const int tok0 = (int)rank * tok_cta;
      const int rows = min(tok_cta, t.left - tok0) * G - wq * 32;  // that are there, of the warp's
      const bool real = lane < rows;
      const int lim = real ? max(0, t.pos + tok0 + row / G + 1) : 0;  // keys this row sees
      const int low = window ? max(0, lim - window) : 0;
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.o) +
                           (((int64_t)t.token + tok0) * p.h_q + (int64_t)t.kvh * G) * D + (lane & 7) * 8;
      int32_t to[8];  // which row of o rows 4 i + lane / 8 of the warp's are, from the first one
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = wq * 32 + 4 * i + (lane >> 3);
        to[i] = r / G * p.h_q + r % G;
      }
      float inv = 0.f, total = 0.f, ref = 0.f;
      bool dirty = false;
      if (t.count > 0) {
        bool w = tc::mbar_wait(&sh.sums_in[used & 1], (used >> 1) & 1) &&
                 tc2::wait(&sh.flags_in[used & 3], (used >> 2) & 1);
        total = sh.sums[used & 1][0][row] + sh.sums[used & 1][1][row];
        ref = sh.refs[used & 1][row];
        inv = total == 0.f ? 0.f : 1.f / total;
        dirty = sh.poison[used & 3] == (uint32_t)used + 1;
        w = w && of_tile(sh.o_done, h);
        tc::fence_after_sync();
        if (!(ok = __all_sync(kFullMask, w) != 0)) return;
      }
      float* part = nullptr;  // of a part of the keys: O as it is, four columns of all rows side by side
      if (t.part >= 0) {
        part = p.partial + (int64_t)(2 * me + t.part) * (2 * kRows * (D + 2));
        if (real) {
          part[2 * kRows * D + rank * kRows + row] = ref;
          part[2 * kRows * (D + 1) + rank * kRows + row] = total;
        }
        part += (int)rank * kRows * D + row * 4;
        inv = 1.f;
      }
      // kOut columns at a time (a thread has a row), through shared memory: stored from
      // there in rows of 128 bytes
#pragma unroll 1
      for (int i = 0; i < D; i += C::kOut) {
        float ov[C::kOut];
        if (t.count > 0) {
          tc2::tmem_ld(tmem + lanes + C::kTmemO + i, ov);
          if (i == D - C::kOut) {
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc2::arrive_remote_relaxed(r_free);  // O may be overwritten
          }
        } else {
#pragma unroll
          for (int k = 0; k < C::kOut; ++k) ov[k] = 0.f;
        }
        const float2 inv2 = make_float2(inv, inv);
#pragma unroll
        for (int k = 0; k < C::kOut; k += 2) {
          const float2 y = tc2::mul2(make_float2(ov[k], ov[k + 1]), inv2);
          ov[k] = y.x;
          ov[k + 1] = y.y;
        }
        if (dirty && real) {  // non-finite values that the edge warp took out, for the rows that see them
#pragma unroll 1
          for (int j = 0; j < t.count; ++j) {
            const Keys keys = key_tile_of(t, j, window, sinks);
            if (!keys.edge) continue;
            const Care care = care_of(t, keys, window, sinks);
#pragma unroll 1
            for (int x = care.before > 0 ? 0 : care.from; x < keys.rows; ++x) {
              const int key = keys.first + x;
              const uint32_t r = row_of(t, key, entry_of(t, key, true));
              if (key >= lim || (key < low && key >= sinks) || r == ~0u) continue;
              if (kFp8) {
                const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.cache.v_pages) + (int64_t)r * D + i);
                const uint32_t byte = __ldg(p.cache.v_exp + r);
#pragma unroll
                for (int k = 0; k < C::kOut; k += 16) {
                  uint4 y[2];
                  uint32_t odd = 0;
                  widen16(__ldg(src + k / 16), value_units(byte, byte), y[0], y[1], odd);
#pragma unroll
                  for (int n = 0; n < 2; ++n) {
                    const uint4 z = mend(y[n], byte);
                    const uint32_t two[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                      ov[k + 8 * n + 2 * e] += poison_of(two[e] & 0xffffu);
                      ov[k + 8 * n + 2 * e + 1] += poison_of(two[e] >> 16);
                    }
                  }
                }
              } else {
                const uint32_t* src = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(p.cache.v_pages) + (int64_t)r * D + i);
#pragma unroll
                for (int k = 0; k < C::kOut / 2; ++k) {
                  const uint32_t two = __ldg(src + k);
                  ov[2 * k] += poison_of(two & 0xffffu);
                  ov[2 * k + 1] += poison_of(two >> 16);
                }
              }
            }
          }
        }
        if (part) {
          if (real) {
#pragma unroll
            for (int k = 0; k < C::kOut; k += 4)
              *reinterpret_cast<float4*>(part + (i + k) * kRows) = make_float4(ov[k], ov[k + 1], ov[k + 2], ov[k + 3]);
          }
          continue;
        }
#pragma unroll
        for (int k = 0; k < C::kOut; k += 8) {
          const uint4 x = make_uint4(pack_bf16(ov[k], ov[k + 1]), pack_bf16(ov[k + 2], ov[k + 3]),
                                     pack_bf16(ov[k + 4], ov[k + 5]), pack_bf16(ov[k + 6], ov[k + 7]));
          *reinterpret_cast<uint4*>(stage + lane * 128 + (((((i + k) >> 3) & 7) ^ (lane & 7)) << 4)) = x;
        }
        if (((i + C::kOut) & 63) == 0) {
          __syncwarp();
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            const int r = 4 * x + (lane >> 3);
            const uint4 y = *reinterpret_cast<const uint4*>(stage + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
            if (r < rows) *reinterpret_cast<uint4*>(out + (int64_t)to[x] * D + i + C::kOut - 64) = y;
          }
          __syncwarp();
        }
      }
    };
    Piece t;
    int used = 0, g = 0;
    if (!kFp8) {
      for (int pass = 0; next_tile(pass, &t); ++pass) {
        epilogue(t, used, g + t.count - 1);
        if (!ok) break;
        if (t.count > 0) {
          g += t.count;
          ++used;
        }
      }
    } else {
      // Two warps of each CTA widen its half of K, two that of V: an eight of keys x 64 dims
      // at a time, which is a whole swizzle atom, the next ones' codes on their way meanwhile.
      // The epilogue of a piece follows the first tiles of the next one.
      const bool is_v = wq >= 2;
      const int w2 = wq & 1;
      const int eight = 8 * (lane & 15);
      // within an atom: row, and which 16 of its 64 codes, such that eight lanes' stores
      // fall into different banks
      const int r8 = ((lane >> 1) & 1) | ((lane >> 2) & 2) | (lane & 4), c4 = (lane & 1) | ((lane >> 3) & 2);
      const uint32_t put = r8 * 128 + (((2 * c4) ^ r8) << 4), put2 = r8 * 128 + (((2 * c4 + 1) ^ r8) << 4);
      // A warp's part of a key tile is D / 64 groups of four atoms: of K (64 keys, D dims) every
      // second eight, a block of 64 dims a group; of V (128 keys, D / 2 dims) every second eight
      // too, four of those and a block a group.  A group's code is all there is to loop over:
      // with eight atoms in it, and their codes in registers, instructions came from L2 (64 KB
      // of code in the SM's way; 446 us for 2,000 tokens on 11,011).
      constexpr int kGroupsOf = D / 64, kBlocks = D / 128;
      const uint8_t* codes = static_cast<const uint8_t*>(is_v ? p.cache.v_pages : p.cache.k_pages) + r8 * D + 16 * c4 +
                             (is_v ? rank * (D / 2) : 0);
      const uint8_t* exps = is_v ? p.cache.v_exp : p.cache.k_exp;
      const int eight0 = (is_v ? 0 : 8 * (int)rank) + w2;
      uint8_t* const to_warp = smem + (is_v ? C::kV : C::kK) + w2 * 1024;
      uint64_t* const free_bar = is_v ? sh.o_done : sh.s_done;
      uint64_t* const full_bar = is_v ? sh.v_full : sh.k_full;
      uint8_t(*bytes)[64] = sh.bytes[wq];  // exponent bytes of the warp's eights
      uint8_t* const codes_in = stage + lane * 16;  // groups' codes, which a lane brings for itself
      int slot = 0;  // of those: the oldest group's
      // group q of a key tile: number of its first eight among the warp's, its block
      auto eights_of = [&](int q) { return is_v ? 4 * (q / kBlocks) : 0; };
      auto block_of = [&](int q) { return is_v ? q % kBlocks : q; };
      // (groups of the same eights follow each other: their rows are kept, and their units)
      auto first_of_eights = [&](int q) { return is_v ? q % kBlocks == 0 : q == 0; };
      uint32_t from[4], unit[4], high = 0;
      auto bring = [&](uint32_t rows, int q) {  // (always a group of copies, whether there are any)
        if (first_of_eights(q)) {
          const int first = eight0 + 2 * eights_of(q);
#pragma unroll
          for (int e = 0; e < 4; ++e) from[e] = __shfl_sync(kFullMask, rows, first + 2 * e);
        }
        const uint8_t* src = codes + 64 * block_of(q);
#pragma unroll
        for (int e = 0; e < 4; ++e) copy16(codes_in + (slot * 4 + e) * 512, src + (int64_t)from[e] * D, from[e] != ~0u);
        copy_commit();
        if (++slot == C::kDeep) slot = 0;
      };
      auto bring_bytes = [&](uint32_t rows, int b) {  // (with the group that follows)
        const uint32_t mine = __shfl_sync(kFullMask, rows, (eight0 + 2 * lane) & 15);
        if (lane < (is_v ? 8 : 4)) copy8(&bytes[b][8 * lane], exps + (int64_t)mine, mine != ~0u);
      };
      int late_used = 0, late_h = 0, parity = 0;
      int ve = 0;  // edge tiles so far; in the odd CTA without those of copied pieces
      auto start = [&](uint32_t rows) {
        bring_bytes(rows, parity);
#pragma unroll
        for (int q = 0; q < C::kDeep; ++q) bring(rows, q);
      };
      bool due = false, late_wide = false;
      for (int pass = 0; ok; ++pass) {
        const bool more = next_tile(pass, &t);
        if (!ok) break;
        const int tiles = more ? t.count : 0, count = tiles > 0 && t.wide < 0 ? tiles : 0;  // all, to widen
        // the page of the lane's eight of key tile j, and their cached rows
        auto look = [&](int j) {
          const Keys k = key_tile_of(t, j, window, sinks);
          return entry_of(t, k.first + eight, j < count && wanted(t, k, eight));
        };
        auto rows_of = [&](int j, int page) { return row_of(t, key_tile_of(t, j, window, sinks).first + eight, page); };
        uint32_t rows = rows_of(0, look(0));
        int page = look(1);
        copy_wait<0>();  // (the last ones, of no row, into the same places)
        start(rows);
        // After a piece that was copied, whose key tiles these warps have not waited for one by
        // one, its epilogue comes first: by then all its products are done, and the waits for
        // free slots are for the barriers' present phases.
        const int when = late_wide ? -1 : min(C::kLag, max(0, count - 1));
        for (int j = min(when, 0); ok; ++j) {
          const int h = g + j, s = h % C::kSlots;
          if (j >= 0 && j < count) {
            const uint32_t ahead = rows_of(j + 1, page);
            page = look(j + 2);
            const Keys keys = key_tile_of(t, j, window, sinks);
            if (h >= C::kSlots && !(ok = __all_sync(kFullMask, of_tile(free_bar, h - C::kSlots)) != 0)) break;
            if (wq == 2) note(h, wanted(t, keys, eight) && rows == ~0u);
            if (rank == 1) sh.said[wq][s][0] = (uint32_t)h + 1;  // (long before the fence, which waits for it)
            uint8_t* const to_tile = to_warp + s * C::kEntry;
            bring_bytes(ahead, parity ^ 1);
#pragma unroll 1
            for (int q = 0; q < kGroupsOf; ++q) {
              copy_wait<C::kDeep - 1>();
              const uint8_t* byte_of = &bytes[parity][8 * eights_of(q) + r8];
              if (first_of_eights(q)) {
                __syncwarp();  // (the bytes are other lanes')
                high = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const uint32_t byte = byte_of[8 * e];
                  unit[e] = value_units(byte, byte);
                  high |= byte > kUnitTop ? 0x80u : 0u;
                }
              }
              uint8_t* to = to_tile + eights_of(q) * 2048 + block_of(q) * (is_v ? 16384 : 8192);
              uint4 x[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) x[e] = *reinterpret_cast<const uint4*>(codes_in + (slot * 4 + e) * 512);
              // into the place of these codes, which have been read, before they are worked on
              bring(q + C::kDeep < kGroupsOf ? rows : ahead, (q + C::kDeep) % kGroupsOf);
              uint32_t odd = high;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                uint4 lo, hi;
                widen16(x[e], unit[e], lo, hi, odd);
                *reinterpret_cast<uint4*>(to + e * 2048 + put) = lo;
                *reinterpret_cast<uint4*>(to + e * 2048 + put2) = hi;
              }
              if (odd & 0x80808080u) {  // in a loop of its own, as it hardly ever runs
#pragma unroll 1
                for (int e = 0; e < 4; ++e) {
                  uint8_t* atom = to + e * 2048;
                  *reinterpret_cast<uint4*>(atom + put) = mend(*reinterpret_cast<const uint4*>(atom + put), byte_of[8 * e]);
                  *reinterpret_cast<uint4*>(atom + put2) = mend(*reinterpret_cast<const uint4*>(atom + put2), byte_of[8 * e]);
                }
              }
            }
            parity ^= 1;
            tc::fence_proxy_async();  // the rows -> this CTA's tensor cores
            __syncwarp();
            // The even CTA's tensor cores hear of the odd one's rows by 16 bytes copied there: the
            // fence has ordered the copy behind the rows, it is in the tensor cores' proxy, and
            // its arrival on the barrier is a release in the cluster; its thread need not wait
            // (an arrival there with a release of its own waits for all that the thread has under
            // way: 800 of 4,300 cycles a key tile, and from a warp of its own still 506 us where
            // this takes 400).  The edge warp reads the rows with ordinary loads, for which a copy
            // says nothing of other threads' ordinary stores: V of an edge tile, of which there
            // are few, is handed on by the odd CTA's edge warp (by such arrivals from here 8 tokens
            // on 131,072 positions took 85 us, by its edge warp 75).
            const bool edge = is_v && keys.edge;
            if (lane == 0) {
              if (edge) tc::mbar_arrive(&sh.v_edge[ve % C::kSlots]);
              if (rank == 1) tell(sh.said[wq][s], &full_bar[s]);
              else if (w2 == 0) tc::mbar_arrive_expect_tx(&full_bar[s], kWideners * 16);
              else tc::mbar_arrive(&full_bar[s]);
            }
            ve += edge;
            rows = ahead;
          }
          if (due && j == when) {
            copy_wait<0>();
            __syncwarp();
            epilogue(sh.late[wq], late_used, late_h);
            due = false;
            // (what was under way went where the epilogue keeps o)
            start(rows);
          }
          if (j + 1 >= count) break;
        }
        if (!ok || !more) break;
        if (lane == 0) sh.late[wq] = t;  // whose epilogue is due
        __syncwarp();
        late_used = used;
        late_h = g + tiles - 1;
        late_wide = count < tiles;
        due = true;
        if (tiles > 0) {
          if (is_v && rank == 0 && count == 0) ve += edges_of(t, window, sinks, lane);
          g += tiles;
          ++used;
        }
      }
      copy_wait<0>();
      __syncwarp();
      if (rank == 1 && lane < C::kSlots) tc2::store_remote(tc2::in_cta(&sh.said_last[wq][lane], 0), sh.said[wq][lane][0]);
    }
  } else {
    tc2::fewer_registers<C::kOtherRegs>();
    // For copies of K and V: a lane looks up the page of eight keys of a tile.  Keys that lie
    // side by side in a page are copied together, up to 64 (a box); the first lane of a box asks
    // for it, at 80 to 100 cycles a box and block of dims, which pages of few keys make many
    // (so K and V have a warp each).
    // A widened copy's rows, [row][KV head][D], lie side by side.
    const int eight = 8 * (lane & 15), box = kFp8 ? 64 : min(1 << shift, 64);
    const bool lead = lane < 16 && (eight & (box - 1)) == 0;
    const int none = max(1, p.cache.num_pages * p.cache.h_kv);  // past the pages: reads as zeros
    auto look = [&](const Piece& t, int j) {
      const Keys k = key_tile_of(t, j, window, sinks);
      return entry_of(t, k.first + eight, j < t.count && wanted(t, k, eight));
    };
    struct Where {  // of the lane's eight keys of a tile
      uint32_t row;  // in the cache (~0: no page)
      int y, z;      // in the tensor maps
    };
    auto where = [&](const Piece& t, const Keys& k, int page) {
      Where w;
      w.row = row_of(t, k.first + eight, page);
      w.y = w.row == ~0u ? 0 : w.row & ((1 << shift) - 1);
      w.z = w.row == ~0u ? none : (int)(w.row >> shift);
      if (kFp8) {
        w.y = t.kvh;
        w.z = t.wide + k.first + eight;
      }
      return w;
    };
    if (warp == kScheduleWarp) {
      // ------------------------------------------------------------ schedule, copies of V
      Piece t = sh.tile[0];
      int g = 0, vc = 0, ve = 0;  // key tiles; up to which V was asked for; edge tiles
      bool last_copied = false;
      const uint32_t r_v = tc2::in_cta(sh.v_full, 0), r_ve = tc2::in_cta(sh.v_edge, 0);
      for (int pass = 1; t.count >= 0 && ok; ++pass) {
        Piece next;
        next_piece(&next);
        if (pass >= 2 && !__all_sync(kFullMask, tc::mbar_wait(&sh.tile_empty[pass & 1], ((pass >> 1) - 1) & 1))) {
          ok = false;
          break;
        }
        if (lane == 0) {
          sh.tile[pass & 1] = next;
          tc::mbar_arrive(&sh.tile_full[pass & 1]);
        }
        // Before a copied piece there may be ones that were widened, whose key tiles this warp has
        // not waited for one by one: it goes on when their scores are done (and so all products
        // with V up to kSlots key tiles before this piece's first), which the other copying warp
        // tells for each piece in turn; of those, it is never two ahead, as this warp hands the
        // pieces out.
        if (kFp8 && !(ok = __all_sync(kFullMask, tc::mbar_wait(&sh.copy_v[(pass - 1) & 1], ((pass - 1) >> 1) & 1)) != 0)) break;
        const bool copied = !kFp8 || t.wide >= 0;  // (not widened by warps of their own)
        if (!copied) ve += edges_of(t, window, sinks, lane);
        if (t.count > 0) last_copied = copied;
        int page = kFp8 ? -1 : look(t, 0);
        for (int j = 0; copied && j < t.count; ++j) {
          const int h = g + j, s = h % C::kSlots, e = ve % C::kSlots;
          const Keys k = key_tile_of(t, j, window, sinks);
          const Where at = where(t, k, page);
          if (!kFp8) page = look(t, j + 1);
          const bool mine = lead && eight < k.rows;
          uint8_t* to = smem + C::kV + s * C::kEntry + eight * 128;
          const uint32_t bytes = ((k.rows + box - 1) & -box) * D * 2, bar = k.edge ? r_ve + e * 8 : r_v + s * 8;
          if (h >= C::kSlots && !(ok = __all_sync(kFullMask, of_tile(sh.o_done, h - C::kSlots)) != 0)) break;
          // The bytes of both CTAs count on the even CTA's barrier, in an edge tile on one of
          // its own that the edge warp can count through; v_full keeps step.
          if (rank == 0 && lane == 0) {
            tc::mbar_arrive_expect_tx(k.edge ? &sh.v_edge[e] : &sh.v_full[s], bytes);
            for (int i = 1; i < (k.edge ? C::kEdgeArrivals : C::kArrivals); ++i)
              tc::mbar_arrive(k.edge ? &sh.v_edge[e] : &sh.v_full[s]);
          }
          if (mine) {
#pragma unroll
            for (int kb = 0; kb < D / 128; ++kb)
              tc2::tma_load_3d(to + kb * 16384, &tm_v, (int)rank * (D / 2) + 64 * kb, at.y, at.z, bar);
          }
          __syncwarp();
          if (k.edge && rank == 0 && lane == 0)
            for (int i = 0; i < C::kArrivals; ++i) tc::mbar_arrive(&sh.v_full[s]);
          vc = h + 1;
          ve += k.edge;
        }
        g += t.count;
        t = next;
      }
      if (rank == 0 && lane == 0) {
        const Place& at = sh.place;
        Join join{};
        join.there[0] = at.there & 1;
        join.there[1] = at.there >> 1;
        if (at.u < at.end && at.start >= at.u0) {  // its last tile, which it has started
          const int first = at.i * work.tokens.d;
          join.last = Shares(at.total, sharers(work, at.total, p.pairs)).owner(at.end - 1);
          join.rows = min(work.tokens.d, at.s.a - first) * G;
          join.token = at.s.q0 + first;
          join.head = at.kvh * G;
        }
        joins(p)[me] = join;
      }
      // Copies still in flight land before the CTA ends: after an expired wait, the
      // even CTA's barriers tell of both CTAs' copies.
      if (lane == 0 && rank == 0 && last_copied) {
        for (int h = max(0, vc - C::kSlots); h < vc; ++h) ok = of_tile(sh.v_full, h) && ok;
        for (int e = max(0, ve - C::kSlots); e < ve; ++e) ok = of_tile(sh.v_edge, e) && ok;
      }
    } else if (warp == kTmaWarp) {
      // ------------------------------------------------------------ copies of Q and K
      Piece t;
      int g = 0, used = 0;  // key tiles, pieces with Q so far
      int kc = 0;           // key tiles up to which K was asked for
      bool last_copied = false;
      const uint32_t r_k = tc2::in_cta(sh.k_full, 0), r_q = tc2::in_cta(&sh.q_full, 0);
      for (int pass = 0; next_tile(pass, &t); ++pass) {
        if (t.count == 0) {
          if (kFp8 && lane == 0) tc::mbar_arrive(&sh.copy_v[pass & 1]);
          continue;
        }
        int page = look(t, 0);
        if (used > 0) ok = __all_sync(kFullMask, tc::mbar_wait(&sh.q_empty, (used - 1) & 1)) != 0;
        if (!ok) break;
        if (lane == 0) {
          if (kFp8) tc::mbar_arrive(&sh.copy_v[pass & 1]);
          if (rank == 0) tc::mbar_arrive_expect_tx(&sh.q_full, 2u * (uint32_t)(tok_cta * G) * D * 2);
          for (int kb = 0; kb < D / 64; ++kb)
            tc2::tma_load_3d(smem + kb * 16384, &tm_q, 64 * kb, t.kvh * G, t.token + (int)rank * tok_cta, r_q);
        }
        __syncwarp();
        ++used;
        last_copied = !kFp8 || t.wide >= 0;
        for (int j = 0; last_copied && j < t.count && ok; ++j) {
          const int h = g + j, s = h % C::kSlots;
          const Keys k = key_tile_of(t, j, window, sinks);
          const Where at = where(t, k, page);
          page = look(t, j + 1);
          const bool mine = lead && eight < k.rows && (lane >> 3) == (int)rank;
          uint8_t* to = smem + C::kK + s * C::kEntry + (lane & 7) * 1024;
          const uint32_t bytes = ((k.rows + box - 1) & -box) * D * 2;
          if (h >= C::kSlots && !(ok = __all_sync(kFullMask, of_tile(sh.s_done, h - C::kSlots)) != 0)) break;
          // the bytes of both CTAs count on the even CTA's barrier
          if (rank == 0 && lane == 0) {
            tc::mbar_arrive_expect_tx(&sh.k_full[s], bytes);
            for (int i = 1; i < C::kArrivals; ++i) tc::mbar_arrive(&sh.k_full[s]);
          }
          if (mine) {
#pragma unroll
            for (int kb = 0; kb < D / 64; ++kb) tc2::tma_load_3d(to + kb * 8192, &tm_k, 64 * kb, at.y, at.z, r_k + s * 8);
          }
          __syncwarp();
          note(h, wanted(t, k, eight) && at.row == ~0u);
          kc = h + 1;
        }
        g += t.count;
        if (!ok) break;
      }
      if (lane == 0 && rank == 0) {  // (as for V)
        for (int h = max(0, kc - C::kSlots); last_copied && h < kc; ++h) ok = of_tile(sh.k_full, h) && ok;
        if (used > 0 && !tc::mbar_wait(&sh.q_full, (used - 1) & 1)) ok = false;
      }
    } else if (warp == kMmaWarp) {
      // ------------------------------------------------------------ products
      Piece t;
      int used = 0;  // pieces with Q so far
      // slots of K and V, score tiles to write and to read, and their barriers' phases
      // (counted, not divided: the issue of a product waits for all of this)
      uint32_t ks = 0, k_ph = 0, vs = 0, v_ph = 0, sw = 0, sr = 0, sr_ph = 0;
      const uint32_t idesc_s = tc::idesc_bf16_f32(256, kKeys, false, false);
      const uint32_t idesc_o = tc::idesc_bf16_f32(256, D, false, true);
      const uint64_t dq = tc::smem_desc(sbase, 16, 1024, tc::kLayoutSw128);
      const uint64_t dk = tc::smem_desc(sbase + C::kK, 16, 1024, tc::kLayoutSw128);
      const uint64_t dv = tc::smem_desc(sbase + C::kV, 16384, 1024, tc::kLayoutSw128);
      const bool leader = tc::elect_one();
      auto step = [](uint32_t& i, uint32_t& ph, uint32_t n) {
        if (++i == n) {
          i = 0;
          ph ^= 1;
        }
      };
      int edges = 0;  // edge tiles so far
      // the even CTA's warp issues for the pair
      for (int pass = 0; rank == 0 && next_tile(pass, &t); ++pass) {
        if (t.count == 0) continue;
        const bool in = tc::mbar_wait(&sh.q_full, used & 1);
        tc::fence_after_sync();
        ok = __all_sync(kFullMask, in) != 0;
        for (int j = 0; j < t.count + C::kLag && ok; ++j) {
          if (j < t.count) {  // S = Q K^T of key tile j
            const bool w = tc::mbar_wait(&sh.k_full[ks], k_ph);
            tc::fence_after_sync();
            if (!(ok = __all_sync(kFullMask, w) != 0)) break;
            if (leader) {
              const uint64_t kd = dk + ((ks * C::kEntry) >> 4);
#pragma unroll
              for (int kk = 0; kk < C::kSteps; ++kk)
                tc2::mma_ss(tmem + sw * kKeys, dq + (((kk >> 2) * 16384 + (kk & 3) * 32) >> 4),
                            kd + (((kk >> 2) * 8192 + (kk & 3) * 32) >> 4), idesc_s, kk > 0);
              tc2::commit(&sh.s_done[ks]);
              if (j == t.count - 1) tc2::commit(&sh.q_empty);
            }
            __syncwarp();
            if (++sw == C::kS) sw = 0;
            step(ks, k_ph, C::kSlots);
          }
          const int i = j - C::kLag;
          if (i >= 0) {  // O += P V of key tile i
            const Keys k = key_tile_of(t, i, window, sinks);
            bool w = tc::mbar_wait(&sh.v_full[vs], v_ph);
            if (k.edge) {  // V may have been edited in both CTAs (ordinary writes): acquire those
              w = w && of_tile(sh.v_edge, edges) && tc2::wait(&sh.v_clean[edges % C::kSlots], (edges / C::kSlots) & 1);
              ++edges;
            }
            w = w && tc::mbar_wait(&sh.p_ready[sr], sr_ph);
            if (i == 0 && used > 0) w = w && tc::mbar_wait(&sh.o_free, (used - 1) & 1);
            tc::fence_after_sync();
            if (!(ok = __all_sync(kFullMask, w) != 0)) break;
            if (leader) {
              const uint64_t vd = dv + ((vs * C::kEntry) >> 4);
#pragma unroll
              for (int kk = 0; kk < kKeys / 16; ++kk)
                if (16 * kk < k.rows)  // no weight beyond
                  tc2::mma_ts(tmem + C::kTmemO, tmem + sr * kKeys + 64 * (kk >> 2) + 8 * (kk & 3), vd + ((kk * 2048) >> 4),
                              idesc_o, (i > 0) || (kk > 0));
              tc2::commit(&sh.o_done[vs]);
            }
            __syncwarp();
            step(sr, sr_ph, C::kS);
            step(vs, v_ph, C::kSlots);
          }
        }
        if (!ok) break;
        ++used;
      }
      // every product issued has completed before either CTA leaves the barrier at the end
      if (rank == 0) {
        if (leader) tc2::commit(&sh.drained);
        __syncwarp();
        if (!__all_sync(kFullMask, tc::mbar_wait(&sh.drained, 0))) ok = false;
      }
    } else if (warp == kEdgeWarp && rank == 0) {
      // ------------------------------------------------------------ edge tiles
      // V of both CTAs: a value that is not finite, in a row that some query of the pair does
      // not see, becomes zero (the epilogue adds it where it is seen).
      Piece t;
      int g = 0, used = 0, edges = 0;
      const uint32_t r_flags = tc2::in_cta(sh.flags_in, 1), r_poison = tc2::in_cta(sh.poison, 1);
      const uint32_t v_even = tc2::in_cta(smem + C::kV, 0) + lane * 16, v_odd = tc2::in_cta(smem + C::kV, 1) + lane * 16;
      for (int pass = 0; next_tile(pass, &t); ++pass) {
        if (t.count == 0) continue;
        bool told = false;  // a non-finite value that a row sees
        for (int j = 0; j < t.count && ok; ++j) {
          const Keys keys = key_tile_of(t, j, window, sinks);
          if (!keys.edge) continue;
          const int h = g + j, rows = keys.rows;  // rows of V that some query sees
          const Care care = care_of(t, keys, window, sinks);
          const int row0 = care.before > 0 ? 0 : care.from;
          if (!(ok = __all_sync(kFullMask, tc2::wait(&sh.v_edge[edges % C::kSlots], (edges / C::kSlots) & 1)))) break;
          const uint32_t slot = h % C::kSlots * C::kEntry;
          // the largest of the magnitudes, as 16-bit integers (a non-finite one is 0x7f80 or
          // more); in a short loop, as it runs once a tile of queries and not from a cache
          uint32_t most = 0;
#pragma unroll 1
          for (int r = row0; r < rows; r += 16) {
            if (r >= care.before && r < care.from) {
              r = care.from - 16;
              continue;
            }
            // eight loads in flight: both halves' rows at D = 128, a half's at 256
#pragma unroll
            for (int c = 0; c < D / 16; c += 8) {
              uint4 y[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const int k = (c + i) % (D / 32);
                const uint32_t at = slot + (k >> 2) * 16384 + r * 128 + (k & 3) * 512;
                y[i] = c + i < D / 32 ? tc2::load_remote(v_odd + at)
                                      : *reinterpret_cast<const uint4*>(smem + C::kV + at + lane * 16);
              }
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                most = __vimax3_u16x2(most, y[i].x & 0x7fff7fffu, y[i].y & 0x7fff7fffu);
                most = __vimax3_u16x2(most, y[i].z & 0x7fff7fffu, y[i].w & 0x7fff7fffu);
              }
            }
          }
          bool seen = false;
          const bool edited = __any_sync(kFullMask, (most & 0xffffu) >= 0x7f80u || most >= 0x7f800000u);
          if (edited) {
#pragma unroll 1
            for (int i = 0; i < 2 * (int)C::kEntry / 512; ++i) {  // four rows at a time
              const int k = i % ((int)C::kEntry / 512), r = 4 * (k & 31);
              if (r < row0) continue;
              const uint32_t at = (i == k ? v_even : v_odd) + slot + k * 512;
              auto finite = [](uint32_t x) { return x & ~__vcmpeq2(x & 0x7f807f80u, 0x7f807f80u); };
              const uint4 y = tc2::load_remote(at), z = make_uint4(finite(y.x), finite(y.y), finite(y.z), finite(y.w));
              if (z.x != y.x || z.y != y.y || z.z != y.z || z.w != y.w) {
                tc2::store_remote(at, z);
                seen = seen || r + (lane >> 3) < rows;
              }
            }
          }
          if (__any_sync(kFullMask, seen)) told = true;
          if (edited) tc2::fence_proxy_async();  // the edited V rows -> the tensor cores of both CTAs
          __syncwarp();
          if (lane == 0) {
            if (edited) tc2::arrive_remote(tc2::in_cta(&sh.v_clean[edges % C::kSlots], 0));
            else tc::mbar_arrive(&sh.v_clean[edges % C::kSlots]);
          }
          ++edges;
        }
        if (!ok) break;
        if (lane == 0) {
          if (told) {
            sh.poison[used & 3] = (uint32_t)used + 1;
            tc2::store_remote(r_poison + (used & 3) * 4, (uint32_t)used + 1);
          }
          tc::mbar_arrive(&sh.flags_in[used & 3]);
          if (told) tc2::arrive_remote(r_flags + (used & 3) * 8);
          else tc2::arrive_remote_relaxed(r_flags + (used & 3) * 8);
        }
        g += t.count;
        ++used;
      }
    } else if (kFp8 && warp == kEdgeWarp) {
      // ------------------------------------------------------------ edge tiles of the odd CTA
      // V that this CTA's warps have widened, handed to the even CTA's edge warp.
      Piece t;
      int edges = 0, own = 0;  // edge tiles, as that warp counts them; of those, the ones widened here
      const uint32_t r_edge = tc2::in_cta(sh.v_edge, 0);
      for (int pass = 0; ok && next_tile(pass, &t); ++pass) {
        const int n = edges_of(t, window, sinks, lane);
        for (int i = 0; i < n && t.wide < 0; ++i) {
          if (!(ok = __all_sync(kFullMask, of_tile(sh.v_edge, own)) != 0)) break;
          if (lane == 0) tc2::arrive_remote(r_edge + (edges + i) % C::kSlots * 8);
          ++own;
        }
        edges += n;
      }
    }
  }
  if (!ok) {
    raise_error(p.err, kErrDeviceTimeout);
    if (kFp8) sh.failed = 1;
  }
  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  tc::cluster_sync();  // neither CTA's memory is in use by the other any more
  // (but for what the odd CTA has told and the even one, which gave up, has not waited for: 16
  // bytes a copy, of which it knows what they will be)
  if (kFp8 && rank == 0 && sh.failed && tid < 4 * C::kSlots) {
    const volatile uint32_t* there = sh.said[tid / C::kSlots][tid % C::kSlots];
    const uint64_t t0 = tc::globaltimer_ns();
    while (*there != sh.said_last[tid / C::kSlots][tid % C::kSlots] && tc::globaltimer_ns() - t0 < 1000000000ull)
      __nanosleep(100);
  }
  tc::fence_after_sync();
  if (warp == 0) tc2::tmem_dealloc(tmem, C::kTmemCols);
}

// The rows of e4m3 sequences with many tiles of queries, widened once: a warp a row of all
// heads, for a block's rows (some 16 KB of codes) after the sequences have been counted as find_many does.
// (At 8 heads of 128 16 rows a block took 104 us with 600 tokens' attention on 11,011 rows, 32
// 109; at 2 of 256 for 96 on 16,000 16 rows 47.3, 32 46.1.)
constexpr int kWidenThreads = 256;
inline __host__ __device__ int widen_rows_of_block(int h_kv, int D) {
  const int rows = 16384 / (h_kv * D);
  return rows < 8 ? 8 : rows > 32 ? 32 : rows;
}
template <int D>
__global__ void __launch_bounds__(kWidenThreads) widen_rows_kernel(const __grid_constant__ PagedPrefillArgs p) {
  constexpr int kLanes = D / 8, kHeads = 32 / kLanes;
  __shared__ int64_t sums[kWidenThreads / 32];
  __shared__ int64_t found_base;
  __shared__ int found_seq;
  tc::allow_dependents();
  tc::wait_prerequisites();
  const Work<true> work(p);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, block_rows = widen_rows_of_block(p.cache.h_kv, D);
  const int per = (p.num_seqs - 1) / kWidenThreads + 1;  // sequences a thread counts
  const int lo = (int)min((int64_t)p.num_seqs, (int64_t)tid * per), hi = (int)min((int64_t)p.num_seqs, (int64_t)lo + per);
  int64_t mine = 0;
  for (int n = lo; n < hi; ++n) mine += work.wide(p, work.sequence(p, n, false));
  const int64_t incl = scan_up(mine, lane);
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  int64_t before = incl - mine, total = 0;
  for (int k = 0; k < kWidenThreads / 32; ++k) {
    if (k < warp) before += sums[k];
    total += sums[k];
  }
  total = min(total, p.wide_rows);  // (the rows of a sequence that ends beyond are not used)
  for (int64_t first = (int64_t)blockIdx.x * block_rows; first < total; first += (int64_t)gridDim.x * block_rows) {
    __syncthreads();
    if (before <= first && first < before + mine) {
      int64_t base = before;
      for (int n = lo; n < hi; ++n) {
        const int64_t rows = work.wide(p, work.sequence(p, n, false));
        if (first < base + rows) {
          found_seq = n;
          found_base = base;
          break;
        }
        base += rows;
      }
    }
    __syncthreads();
    int n = found_seq;
    int64_t base = found_base, rows = work.wide(p, work.sequence(p, n, false));
    for (int64_t row = first + warp; row < min(total, first + block_rows); row += kWidenThreads / 32) {
      while (row >= base + rows) {  // (there is one: row < total)
        base += rows;
        rows = work.wide(p, work.sequence(p, ++n, false));
      }
      const int pos = (int)(row - base), entry = pos >> p.cache.page_shift;
      const int page = entry < p.cache.max_pages ? __ldg(p.cache.table + (int64_t)n * p.cache.max_pages + entry) : -1;
      const bool there = page >= 0 && page < p.cache.num_pages;
      const int64_t at = (((int64_t)(there ? page : 0) * p.cache.h_kv) << p.cache.page_shift) + (pos & ((1 << p.cache.page_shift) - 1));
#pragma unroll 2
      for (int h = lane / kLanes; h < p.cache.h_kv; h += kHeads) {
        const int64_t r = at + ((int64_t)h << p.cache.page_shift);
        const int64_t to = (row * p.cache.h_kv + h) * D + 8 * (lane % kLanes);
        uint2 kc = make_uint2(0, 0), vc = kc;
        uint32_t kb = 127, vb = 127;
        if (there) {
          kc = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.cache.k_pages) + r * D) + lane % kLanes);
          vc = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.cache.v_pages) + r * D) + lane % kLanes);
          kb = __ldg(p.cache.k_exp + r);
          vb = __ldg(p.cache.v_exp + r);
        }
        auto wide = [&](uint2 c, uint32_t byte) {
          uint4 x, unused;
          uint32_t odd = byte > kUnitTop ? 0x80u : 0u;
          widen16(make_uint4(c.x, c.y, 0, 0), value_units(byte, byte), x, unused, odd);
          return odd & 0x80808080u ? mend(x, byte) : x;
        };
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.wide_k) + to) = wide(kc, kb);
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.wide_v) + to) = wide(vc, vb);
      }
    }
  }
}

// Tiles of queries whose keys several pairs went through: block (c, y, z) joins rows 32 y ..
// and columns 64 z .. of the tile that pair c has started and others finished, if there
// is one.  A lane has a row, a warp eight columns of all parts: they are two at most with
// many tiles and some tens with few, whose loads then go out eight and four at a time.
// (Eight warps that shared the parts and met in shared memory took 30 us for two parts of
// 75 tiles of 256 rows.)
constexpr int kJoinWarps = 8, kJoinColumns = 64;
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) attn_prefill_paged_join_kernel(const __grid_constant__ PagedPrefillArgs p) {
  constexpr int kMasks = (kPagedPrefillMaxPairs + 31) / 32;
  tc::allow_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x;
  tc::wait_prerequisites();  // the parts
  // (what there is to know is read at once, of the pairs that may have parts: kMasks times 32)
  const Join* js = joins(p);
  const int4 facts = __ldg(reinterpret_cast<const int4*>(&js[c]));  // there, last, rows
  const int2 place = __ldg(reinterpret_cast<const int2*>(&js[c].token));
  int other[kMasks];
#pragma unroll
  for (int i = 0; i < kMasks; ++i) {
    const int k = 32 * i + lane;
    other[i] = __ldg(&js[min(c + k, p.pairs - 1)].there[k == 0]);
  }
  const int last = facts.z, rows = facts.w, token = place.x, head = place.y, x = 32 * blockIdx.y + lane;
  if (32 * (int)blockIdx.y >= rows) return;
  const int G = p.group, even = min(kRows / G * G, rows);  // rows of the even CTA
  const bool real = x < rows;
  const int cta = x >= even, row = real ? x - cta * even : 0;
  // which parts there are: k of the tile is in slot 1 of pair c, in slot 0 of the pairs after it
  uint32_t there[kMasks], any = 0;
#pragma unroll
  for (int i = 0; i < kMasks; ++i) {
    there[i] = __ballot_sync(kFullMask, c + 32 * i + lane <= last && other[i]);
    any |= there[i];
  }
  if (any == 0) return;  // all keys were one pair's, which has written o
  const int parts = last - c + 1;
  auto is_there = [&](int k) {
    uint32_t m = there[0];
#pragma unroll
    for (int i = 1; i < kMasks; ++i) m = k >= 32 * i ? there[i] : m;
    return ((m >> (k & 31)) & 1) != 0;
  };
  const int at_row = cta * kRows + row, column = kJoinColumns * blockIdx.z + 8 * warp;
  float top = -INFINITY, sum = 0.f;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
  auto scale = [](float4 x, float f) { return make_float4(x.x * f, x.y * f, x.z * f, x.w * f); };
  auto join = [&](auto batch) {
    constexpr int N = decltype(batch)::value;  // parts whose loads go out together
    for (int k0 = 0; k0 < parts; k0 += N) {
      float m[N], l[N], most = top;
      float4 v[N], w[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int k = min(k0 + i, parts - 1);
        const float* part = p.partial + (int64_t)(2 * (c + k) + (k == 0)) * (2 * kRows * (D + 2));
        m[i] = part[2 * kRows * D + at_row];
        l[i] = part[2 * kRows * (D + 1) + at_row];
        v[i] = *reinterpret_cast<const float4*>(part + cta * kRows * D + column * kRows + row * 4);
        w[i] = *reinterpret_cast<const float4*>(part + cta * kRows * D + (column + 4) * kRows + row * 4);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        // not there, or the row sees none of its keys
        if (k0 + i >= parts || !is_there(k0 + i)) m[i] = -INFINITY;
        most = fmaxf(most, m[i]);
      }
      if (top != most && top != -INFINITY) {
        const float f = ex2(top - most);
        sum *= f;
        a = scale(a, f);
        b = scale(b, f);
      }
      top = most;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (m[i] == -INFINITY) continue;
        const float f = ex2(m[i] - top);
        sum = fmaf(f, l[i], sum);
        a = make_float4(fmaf(f, v[i].x, a.x), fmaf(f, v[i].y, a.y), fmaf(f, v[i].z, a.z), fmaf(f, v[i].w, a.w));
        b = make_float4(fmaf(f, w[i].x, b.x), fmaf(f, w[i].y, b.y), fmaf(f, w[i].z, b.z), fmaf(f, w[i].w, b.w));
      }
    }
  };
  if (parts <= 2) join(std::integral_constant<int, 2>{});
  else join(std::integral_constant<int, 4>{});
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  if (real) {
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.o) + ((int64_t)(token + x / G) * p.h_q + head + x % G) * D + column;
    *reinterpret_cast<uint4*>(out) = make_uint4(pack_bf16(a.x * inv, a.y * inv), pack_bf16(a.z * inv, a.w * inv),
                                                pack_bf16(b.x * inv, b.y * inv), pack_bf16(b.z * inv, b.w * inv));
  }
}

// A pool of pages as [pages x h_kv][page_size][D] bf16: boxes of 64 dimensions x `rows` rows
bool encode_pages(CUtensorMap* map, const void* base, const PagedCache& c, int rows) {
  auto enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t row = (cuuint64_t)c.head_dim * 2;
  const cuuint64_t dims[3] = {(cuuint64_t)c.head_dim, (cuuint64_t)1 << c.page_shift, (cuuint64_t)c.num_pages * c.h_kv};
  const cuuint64_t strides[2] = {row, row << c.page_shift};
  const cuuint32_t box[3] = {64, (cuuint32_t)rows, 1}, estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool kFp8>
cudaError_t launch(const PagedPrefillArgs& a, cudaStream_t stream) {
  using C = Cfg<D, kFp8>;
  const int G = a.h_q / a.cache.h_kv, rows = a.cache.page_shift >= 6 ? 64 : 1 << a.cache.page_shift;
  CUtensorMap mq, mk, mv;
  if (!encode(&mq, a.q, D, a.h_q, a.total_q, a.q_stride, G, kRows / G)) return cudaErrorInvalidValue;
  if (!kFp8) {
    PagedCache c = a.cache;
    if (c.num_pages == 0) {  // no page is ever there: the kernel asks for what lies past this one
      c.num_pages = c.h_kv = 1;
      c.k_pages = c.v_pages = const_cast<void*>(a.q);
    }
    if (!encode_pages(&mk, c.k_pages, c, rows) || !encode_pages(&mv, c.v_pages, c, rows)) return cudaErrorInvalidValue;
  } else if (a.wide_rows > 0) {
    const int64_t stride = (int64_t)a.cache.h_kv * D;
    if (!encode(&mk, a.wide_k, D, a.cache.h_kv, a.wide_rows, stride, 1, 64) ||
        !encode(&mv, a.wide_v, D, a.cache.h_kv, a.wide_rows, stride, 1, 64))
      return cudaErrorInvalidValue;
  } else {
    mk = mv = mq;  // (not copied)
  }
  const int smem = (int)(C::kShared + sizeof(Shared<D, kFp8>));
  static_assert(C::kShared + sizeof(Shared<D, kFp8>) <= 227 * 1024, "shared memory");
  static PerDeviceOnce attrs;
  cudaError_t e = attrs.run([&] {
    return cudaFuncSetAttribute(attn_prefill_paged_kernel<D, kFp8>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  });
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (a.wide_rows > 0) {
    cfg.numAttrs = 1;
    const int rows_of_block = widen_rows_of_block(a.cache.h_kv, D);
    cfg.gridDim = dim3((unsigned)min((int64_t)16 * a.pairs, (a.wide_rows + rows_of_block - 1) / rows_of_block));
    cfg.blockDim = dim3(kWidenThreads);
    e = cudaLaunchKernelEx(&cfg, widen_rows_kernel<D>, a);
    if (e != cudaSuccess) return e;
    cfg.numAttrs = 2;
  }
  cfg.gridDim = dim3((unsigned)(2 * a.pairs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  e = cudaLaunchKernelEx(&cfg, attn_prefill_paged_kernel<D, kFp8>, mq, mk, mv, a);
  if (e != cudaSuccess || a.pairs == 1) return e;
  cfg.numAttrs = 1;
  const int64_t most = min((int64_t)2 * (kRows / G), a.total_q) * G;  // rows of a tile
  cfg.gridDim = dim3((unsigned)(a.pairs - 1), (unsigned)((most + 31) / 32), D / kJoinColumns);
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, attn_prefill_paged_join_kernel<D>, a);
}

}  // namespace

// A call whose queries may make kWideTiles tiles of a sequence, over e4m3 rows
bool paged_prefill_widens(int64_t total_q, int32_t group, int dtype) {
  return dtype == kCacheE4M3 && total_q > (int64_t)(kWideTiles - 1) * 2 * (kRows / group);
}

size_t paged_prefill_workspace_bytes(int32_t head_dim) {
  return (size_t)kPagedPrefillMaxPairs * (2 * 2 * kRows * (head_dim + 2) * sizeof(float) + sizeof(Join));
}

cudaError_t launch_attn_prefill_paged(const PagedPrefillArgs& in, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  PagedPrefillArgs a = in;
  a.group = a.h_q / a.cache.h_kv;
  a.tile = 2 * (kRows / a.group);
  a.tile_inv = 0xffffffffu / (uint32_t)a.tile + 1u;
  a.pairs = sms / 2 < kPagedPrefillMaxPairs ? sms / 2 : kPagedPrefillMaxPairs;
  const bool fp8 = a.cache.dtype == kCacheE4M3;
  if (a.cache.head_dim == 256) return fp8 ? launch<256, true>(a, stream) : launch<256, false>(a, stream);
  return fp8 ? launch<128, true>(a, stream) : launch<128, false>(a, stream);
}

}  // namespace gdn
