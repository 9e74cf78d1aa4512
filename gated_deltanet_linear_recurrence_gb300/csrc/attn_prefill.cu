// attn_prefill.cu — causal grouped-query attention over packed prompts, on
// tcgen05 with a pair of CTAs for each tile of queries.
//
// For query row r (token and query head) that sees the keys 0 .. lim_r - 1:
//     s_rj = scale q_r.k_j,   o_r = sum_j 2^(t_rj - m_r) v_j / sum_j 2^(t_rj - m_r),
//     t_rj = s_rj log2(e)
// over 128-key tiles with a running reference m_r: as long as a tile's maximum
// exceeds m_r by at most 8 (weights up to 2^8) m_r stays, so O is seldom rescaled.
//
// Tile.  A CTA pair takes 256 rows: 2 floor(128 / G) consecutive tokens of one
// sequence with the G query heads of a KV head, rows (token, head) in that order,
// which is the order in which q holds them (one TMA box fetches them).  Sharing
// the rows of a KV head keeps the causal edge short (G tokens' rows end at the
// same key) and fills tiles of short sequences.
//
// Bound by the tensor pipe at D = 256: a pair's products take 8 D cycles a key tile
// (4 D flops a row and key), its softmax about 1,450.  With one CTA the operands
// would not fit the shared-memory bandwidth: Q and K tiles read at 128 bytes a cycle
// and K and V written at 64.  cta_group::2 lets each CTA hold half of K (keys) and of
// V (dimensions), and P stays in TMEM, which leaves
//     Q 4 KB + K 2 KB a 64-cycle step; V 4 KB a 128-cycle step (D = 256)
// to read and half of the writes.  At D = 128 the products take half as long (1,024
// cycles) and the softmax of a tile still 1,800, so two groups of warps take the
// tiles in turn: about 1,150 cycles a tile.  Between two tiles of queries the tensor
// pipe pauses 2,500 cycles (the last P, its product, O read out, the next product),
// which is what short sequences pay.
//
// Measured, calls back to back for a second (in brackets runs of some milliseconds,
// before the board's power limit sets in); flops of the visible keys only: 16,384 tokens
// with 16 query heads of 256 on 2 KV heads 1.20 ms, 1.83 PFLOP/s (1.16, 1.90), the rate of
// a plain library product; 4,096 tokens 87 us, 1.58 (78.5, 1.75); 2,048 new tokens on
// 16,000 keys 291 us, 1.73 (280, 1.79).  At D = 128, seven prompts of 1 to 4,096 tokens
// with 32 query heads on 8, 200 us, 1.37 (189, 1.45); 8,192 tokens with 16 on 2 (168,
// 1.64); 600 prompts of 64 tokens with 32 on 8 (174 us).  Seven prompts of 1 to 200 tokens
// (D = 256) 9.7 us (launch and latency).
//
// TMEM (512 columns): S of two or three key tiles (128 fp32 columns each, of whose
// two halves P then takes 32 columns of bf16 pairs), O (D columns).  Shared memory:
// Q (64 KB at D = 256), K and V halves of two or four key tiles, 64 columns of O.
// The scores of the next key tiles are computed while the softmax warps work
// on one, and the products with V follow one or two key tiles behind.
//
// Roles (16 warps): 0-7 softmax, 8-11 epilogue (O to o while the next tile's scores
// are under way), 12 TMA, 13 products (the even CTA's issues them for the pair), 14
// the schedule, 15 V of edge tiles (the even CTA's, of both).  The pairs are persistent.
//
// Rounding: P is rounded to bf16 for the second product (by at most 2^-8 of a weight,
// as the output is; the sums l stay fp32 over unrounded weights).  Weights as bf16
// pairs would double the second product, which is half of all the work.
//
// What a query does not see must not reach it even as NaN: its scores are masked,
// and in a tile that some row sees in part (an edge tile), warp 15 replaces non-finite
// values of V by zero in shared memory; the epilogue adds them back to the rows that do
// see them (from global memory, only in tiles where any was found).
#include <cuda.h>
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>

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

struct Tile {  // one unit of work of a pair; tiles < 0 ends the schedule
  int32_t q0, k0;     // packed rows where the sequence's queries and keys start
  int32_t a, off;     // queries of the sequence; keys before its first query (may be < 0)
  int32_t tok0, kvh;  // first token of the pair's rows; KV head
  int32_t tiles;      // key tiles to go through
  int32_t sight;      // keys that the last row sees
};

template <int D>
struct Cfg {
  // Eight softmax warps.  At D = 256 a tile's products take as long as its softmax,
  // and O leaves room for two score tiles: all warps work on one key tile, two
  // threads a row.  At D = 128 the products take half as long and there is room for
  // three: two groups of four warps take the key tiles in turn, a thread a row, each
  // with two tiles' time for one.
  static constexpr int kGroups = D == 256 ? 1 : 2, kHalves = D == 256 ? 2 : 1;
  static constexpr int kCols = kKeys / kHalves;  // scores a thread
  static constexpr int kS = D == 256 ? 2 : 3;
  static constexpr int kLag = kS - 1;  // key tiles that the scores are ahead of P V
  static constexpr int kPWarps = 4 * kHalves;  // warps that write P of a key tile
  // Registers of a thread of the four warpgroups: softmax (two), epilogue, and 64 for the
  // rest; together the 65,536 that the CTA starts with (setmaxnreg takes them from there).
  // At D = 128 a softmax thread's 128 scores want more than 168 (198 against 222 us for
  // seven packed prompts, when that was tried), and the epilogue reads fewer columns at once.
  static constexpr int kSoftmaxRegs = D == 256 ? 168 : 184, kEpilogueRegs = D == 256 ? 112 : 80;
  static constexpr int kOut = D == 256 ? 64 : 32;  // columns of O that the epilogue holds
  static_assert(2 * kSoftmaxRegs + kEpilogueRegs + 64 == 512, "registers");
  static constexpr uint32_t kQBytes = kRows * D * 2;
  static constexpr uint32_t kEntry = 64 * D * 2;  // half of K (64 keys) or of V (D / 2 dims)
  static constexpr int kSlots = D == 256 ? 2 : 4;  // key tiles of K, and of V, in shared memory
  static constexpr uint32_t kK = kQBytes, kV = kK + kSlots * kEntry;
  static constexpr uint32_t kStage = kV + kSlots * kEntry;  // 64 columns of o on their way out
  static constexpr uint32_t kShared = kStage + kRows * 128;  // the barriers and the rest
  static constexpr int kSteps = D / 16;
  static constexpr uint32_t kTmemO = kS * kKeys;
  static constexpr uint32_t kTmemCols = 512;
  static_assert(kTmemO + D <= kTmemCols, "TMEM");
};

template <int D>
struct Shared {  // beside the tiles
  using C = Cfg<D>;
  // by key tile h: K, V of h % kSlots have landed; the scores of h, the product with V
  // of h are done (h % kSlots; this frees their slots too); P of h is in TMEM (h % kS)
  uint64_t k_full[C::kSlots], v_full[C::kSlots], s_done[C::kSlots], o_done[C::kSlots], p_ready[C::kS];
  uint64_t q_full, q_empty, o_free;
  uint64_t m_ready[2][4];  // two groups: a key tile's references are in m, by quarters of the rows
  // edge tiles, counted through (% kSlots): V has landed in both CTAs; is finite there
  uint64_t v_edge[C::kSlots], v_clean[C::kSlots];
  uint64_t sums_in[2];          // the rows' sums of two tiles are there, for the epilogue
  // What was found in V in the edge tiles of a tile (by number & 3: the schedule's two
  // tiles bound how far this runs ahead of the epilogue): the number + 1 where that was
  // a non-finite value; that this has been told.
  uint64_t flags_in[4];
  uint32_t poison[4];
  uint64_t tile_full[2], tile_empty[2], drained;
  Tile tile[2];
  uint32_t tmem;
  // halves: the row maxima of a key tile's halves, two key tiles; groups: the
  // references of two key tiles
  float red[2][2][128];
  float sums[2][2][128];  // row sums of two tiles, in two parts
};

// ------------------------------------------------------------------ schedule
// One sequence's ranges (bad ones count no tiles; recorded once).
struct Seq {
  int q0, k0, a, b, tiles;
};
__device__ __forceinline__ Seq sequence(const AttnPrefillArgs& p, int n, Divisor tokens, bool report) {
  Seq s{0, 0, 0, 0, 0};
  if (n >= p.num_seqs) return s;
  const int q0 = __ldg(p.cu_q + n), q1 = __ldg(p.cu_q + n + 1);
  const int k0 = __ldg(p.cu_k + n), k1 = __ldg(p.cu_k + n + 1);
  const bool bad = q0 < 0 || q1 < q0 || q1 > p.total_q || k0 < 0 || k1 < k0 || k1 > p.total_k;
  const bool open = (n == 0 && (q0 != 0 || k0 != 0)) ||
                    (n == p.num_seqs - 1 && (q1 != p.total_q || k1 != p.total_k));
  if (report && (bad || open)) raise_error(p.err, kErrBadCuSeqlens);
  if (bad) return s;
  s.q0 = q0;
  s.k0 = k0;
  s.a = q1 - q0;
  s.b = k1 - k0;
  s.tiles = s.a > 0 ? tokens.divide(s.a - 1) + 1 : 0;
  return s;
}
// Tiles of s that see at least x >= 1 keys (its later tiles see more); all of them for x <= 0.
__device__ __forceinline__ int tiles_from(const Seq& s, int x, Divisor tokens) {
  if (x <= 0) return s.tiles;
  if (x > s.b || s.tiles == 0) return 0;
  const int need = x - (s.b - s.a);  // tokens up to the first one that sees x keys
  const int skip = need <= 0 ? 0 : tokens.divide(need - 1);
  return s.tiles - min(skip, s.tiles);
}
__device__ __forceinline__ Tile make_tile(const Seq& s, int i, int kvh, int tokens) {
  Tile t;
  t.q0 = s.q0;
  t.k0 = s.k0;
  t.a = s.a;
  t.off = s.b - s.a;
  t.tok0 = i * tokens;
  t.kvh = kvh;
  t.sight = max(0, t.off + min(s.a, t.tok0 + tokens));
  t.tiles = (t.sight + kKeys - 1) / kKeys;
  return t;
}
__device__ __forceinline__ Seq pick(const Seq& s, int lane) {
  Seq r;
  r.q0 = __shfl_sync(kFullMask, s.q0, lane);
  r.k0 = __shfl_sync(kFullMask, s.k0, lane);
  r.a = __shfl_sync(kFullMask, s.a, lane);
  r.b = __shfl_sync(kFullMask, s.b, lane);
  r.tiles = __shfl_sync(kFullMask, s.tiles, lane);
  return r;
}
__device__ __forceinline__ int prefix(int x, int lane) {  // of the lanes before
  int y = x;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int z = __shfl_up_sync(kFullMask, y, off);
    if (lane >= off) y += z;
  }
  return y - x;
}

// Tiles in the order of the schedule, for one warp.  Either by how many keys they see,
// most first, which makes the pairs' shares even; or sequence by sequence, last tile
// first, so that pairs at work at the same time share keys and values.  The latter for
// more than 32 sequences (their number evens the shares out too) and where the launch
// asks for it.
struct Schedule {
  Seq s;       // this lane's sequence of the current 32
  int base;    // first sequence of the current 32
  int before;  // tiles of the sequences before them
  int lane;
  Divisor tokens;
  __device__ __forceinline__ Schedule(const AttnPrefillArgs& p, int toks, int ln, bool report)
      : base(0), before(0), lane(ln), tokens(toks) {
    s = sequence(p, lane, tokens, report);
    if (report)  // the other sequences' checks
      for (int n = 32 + lane; n < p.num_seqs; n += 32) sequence(p, n, tokens, true);
  }
  // tile number r (asked in increasing order) of KV head kvh; false past the end
  __device__ __forceinline__ bool get(const AttnPrefillArgs& p, int r, int kvh, Tile* t) {
    if (p.num_seqs == 1) {  // one sequence: its last tile sees most
      const Seq q = pick(s, 0);
      if (r >= q.tiles) return false;
      *t = make_tile(q, q.tiles - 1 - r, kvh, tokens.d);
      return true;
    }
    if (p.num_seqs <= 32 && !p.by_sequence) {
      if (r >= __reduce_add_sync(kFullMask, s.tiles)) return false;
      int lo = 0, hi = __reduce_max_sync(kFullMask, s.b) + 1;  // tiles_from(lo) > r >= tiles_from(hi)
      while (hi - lo > 1) {
        const int mid = lo + (hi - lo) / 2;
        if (__reduce_add_sync(kFullMask, tiles_from(s, mid, tokens)) > r) lo = mid;
        else hi = mid;
      }
      const int at = tiles_from(s, lo, tokens), above = tiles_from(s, lo + 1, tokens);
      const int k = r - __reduce_add_sync(kFullMask, above);  // among the tiles that see lo keys
      const int pre = prefix(at - above, lane);
      const unsigned hit = __ballot_sync(kFullMask, k >= pre && k < pre + at - above);
      const int src = __ffs(hit) - 1;
      const Seq q = pick(s, src);
      *t = make_tile(q, q.tiles - __shfl_sync(kFullMask, at, src) + k - __shfl_sync(kFullMask, pre, src),
                     kvh, tokens.d);
      return true;
    }
    for (;;) {
      const int n = __reduce_add_sync(kFullMask, s.tiles);
      if (r < before + n) break;
      before += n;
      base += 32;
      if (base >= p.num_seqs) return false;
      s = sequence(p, base + lane, tokens, false);
    }
    const int pre = before + prefix(s.tiles, lane);
    const unsigned hit = __ballot_sync(kFullMask, r >= pre && r < pre + s.tiles);
    const int src = __ffs(hit) - 1;
    const Seq q = pick(s, src);
    *t = make_tile(q, q.tiles - 1 - (r - __shfl_sync(kFullMask, pre, src)), kvh, tokens.d);
    return true;
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_prefill_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const AttnPrefillArgs p) {
  using C = Cfg<D>;
  // (the tiles' swizzle needs this alignment; there is no other shared memory, and the
  // barriers and the rest, 4.5 KB, follow the tiles)
  extern __shared__ __align__(1024) uint8_t smem[];
  Shared<D>& sh = *reinterpret_cast<Shared<D>*>(smem + C::kShared);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = tc::cluster_rank();
  const int G = p.h_q / p.h_kv;
  const int tok_cta = kRows / G, tokens = 2 * tok_cta;  // tokens a CTA, a pair
  if (warp == 0) {
    tc2::tmem_alloc(&sh.tmem, C::kTmemCols);
    tc2::tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < C::kSlots; ++i) {
      tc::mbar_init(&sh.k_full[i], 1);
      tc::mbar_init(&sh.v_full[i], 1);
      tc::mbar_init(&sh.s_done[i], 1);
      tc::mbar_init(&sh.o_done[i], 1);
    }
    tc::mbar_init(&sh.q_full, 1);
    tc::mbar_init(&sh.q_empty, 1);
    for (int i = 0; i < C::kS; ++i) tc::mbar_init(&sh.p_ready[i], 2 * C::kPWarps);
    for (int i = 0; i < 2; ++i) {
      for (int k = 0; k < 4; ++k) tc::mbar_init(&sh.m_ready[i][k], 1);
      tc::mbar_init(&sh.tile_full[i], 1);
      tc::mbar_init(&sh.sums_in[i], 8);
      // readers: the softmax, epilogue and TMA warps, and in the even CTA the products' and edge warps
      tc::mbar_init(&sh.tile_empty[i], 12 + (rank == 0 ? 3 : 1));
    }
    for (int i = 0; i < 4; ++i) {
      tc::mbar_init(&sh.flags_in[i], 1);
      sh.poison[i] = 0;
    }
    for (int i = 0; i < C::kSlots; ++i) {
      tc::mbar_init(&sh.v_edge[i], 1);
      tc::mbar_init(&sh.v_clean[i], 1);
    }
    tc::mbar_init(&sh.o_free, 2 * 4);
    tc::mbar_init(&sh.drained, 1);
    tc::fence_mbar_init();
  }
  if (warp == kScheduleWarp) {  // the first tile, while the pair gets ready
    tc::wait_prerequisites();
    Tile t;
    if (!Schedule(p, tokens, lane, blockIdx.x == 0).get(p, (int)(blockIdx.x / 2) / p.h_kv, (int)(blockIdx.x / 2) % p.h_kv, &t))
      t.tiles = -1;
    if (lane == 0) sh.tile[0] = t;
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::cluster_sync();
  tc::fence_after_sync();
  const uint32_t tmem = sh.tmem;
  const uint32_t sbase = tc::smem_u32(smem);
  bool ok = true;
  tc::wait_prerequisites();  // q, k, v and the offsets come from earlier kernels
  tc::allow_dependents();

  // wait for what a barrier by key tile says of key tile h
  auto of_tile = [&](uint64_t* bars, int h) { return tc::mbar_wait(&bars[h % C::kSlots], (h / C::kSlots) & 1); };

  // The warp's next tile (pass counts tiles); false at the end or when a wait expired.
  auto next_tile = [&](int pass, Tile* t) {
    // (the first is there from the start; of tile_full's phases it takes none)
    const bool w = pass == 0 || __all_sync(kFullMask, tc::mbar_wait(&sh.tile_full[pass & 1], ((pass - 1) >> 1) & 1));
    if (!w) {
      ok = false;
      return false;
    }
    *t = sh.tile[pass & 1];
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&sh.tile_empty[pass & 1]);
    return t->tiles >= 0;
  };

  if (warp < kEpilogueWarp) {
    tc2::more_registers<C::kSoftmaxRegs>();
    // ------------------------------------------------------------ softmax
    Tile t;
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
      const int tok = t.tok0 + (int)rank * tok_cta + row / G;
      const bool real = row < tok_cta * G && tok < t.a;
      const int lim = real ? max(0, t.off + tok + 1) : 0;  // keys this row sees
      const int whole = t.off + t.tok0 + 1;                // keys that every row of the pair sees
      float m = -INFINITY, l = 0.f;
      // with two groups, this one takes every other key tile (g counts them through)
      auto key_tile = [&](int j) {
        const int h = g + j, key0 = j * kKeys, sb = h % C::kS;
        bool w = carried && of_tile(sh.s_done, h);
        tc::fence_after_sync();
        w = __all_sync(kFullMask, w);
        const float none = down ? INFINITY : -INFINITY;
        const uint32_t scores = tmem + lanes + sb * kKeys + C::kCols * half;
        // the upper 64 of 128 columns only if some row sees them, as the product with V
        // takes no more (packed prompts 180 -> 177 us, 600 prompts of 64 tokens 221 -> 190,
        // when that was tried)
        const bool upper = C::kCols > 64 && t.sight - key0 > 64;
        const int cols = upper ? C::kCols : 64;
        if (key0 + kKeys > whole) {
          // An edge tile: the scores that a row does not see are overwritten.  One short
          // loop before code that all tiles share: with the masks inside an unrolled copy
          // of that code, its instructions (run once a tile of queries, so never near)
          // took 4,500 cycles where a tile without an edge takes 1,800 (seven packed
          // prompts 196 us, then 184; with this loop an edge tile takes 2,400).
          const int left = lim - key0 - C::kCols * half;  // columns of this thread that the row sees
          const int all = __reduce_min_sync(kFullMask, left);
#pragma unroll 1
          for (int k = max(0, all) & ~31; k < cols; k += 32) {
            float x[32];
            tc::tmem_ld32(scores + k, x);
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = i < left - k ? x[i] : none;
            tc::tmem_st32(scores + k, x);
          }
        }
        float s[64];  // 64 of the thread's scores
        auto fetch = [&](int k) { tc2::tmem_ld(scores + k, s); };
        float x = none;
        if (upper) {
          fetch(64);
          x = down ? least(s) : largest(s);
        }
        fetch(0);
        const float x0 = down ? least(s) : largest(s);
        x = C::kCols > 64 ? (down ? fminf(x, x0) : fmaxf(x, x0)) : x0;
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
        // Rows that are no queries (past the sequence's end, or the tile's) hold other rows' q
        // or what was there before: they never move a reference, and neither does one that is
        // NaN already (two queries on 16,000 keys, D = 128, beside rows of NaN: 154 -> 78 us)
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
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc2::arrive_remote_relaxed(r_p + sb * 8);
      };
      for (int j = C::kGroups > 1 ? (g ^ grp) & 1 : 0; j < t.tiles && ok; j += C::kGroups) key_tile(j);
      // ---- the pair's rows are through their keys: their sums go to the epilogue
      if (t.tiles > 0) {
        if (C::kGroups > 1) {
          const int h = g + t.tiles - 1;
          carried = carried && tc::mbar_wait(&sh.m_ready[h & 1][warp & 3], (h >> 1) & 1);
          const float last = sh.red[h & 1][0][row];  // of the last tile, which O goes by
          if (m != last) l *= m == -INFINITY ? 0.f : ex2(m - last);
        }
        sh.sums[used & 1][part][row] = l;
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sh.sums_in[used & 1]);
        g += t.tiles;
        ++used;
      }
    }
  } else if (warp < kTmaWarp) {
    tc2::fewer_registers<C::kEpilogueRegs>();
    // ------------------------------------------------------------ epilogue
    Tile t;
    int used = 0, g = 0;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t r_free = tc2::in_cta(&sh.o_free, 0);
    // 32 rows of 128 bytes for each warp, 16-byte pieces c of row r at c ^ (r & 7)
    uint8_t* stage = smem + C::kStage + (warp & 3) * 4096;
    int32_t to[8];  // which row of o rows 4 i + lane / 8 of the warp's are, from the first one
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = (warp & 3) * 32 + 4 * i + (lane >> 3);
      to[i] = r / G * p.h_q + r % G;
    }
    for (int pass = 0; next_tile(pass, &t); ++pass) {
      const int tok0 = t.tok0 + (int)rank * tok_cta;
      const int rows = min(tok_cta, t.a - tok0) * G - (warp & 3) * 32;  // that are there, of the warp's
      const bool real = lane < rows;
      const int lim = real ? max(0, t.off + tok0 + row / G + 1) : 0;  // keys this row sees
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.o) +
                           (((int64_t)t.q0 + tok0) * p.h_q + (int64_t)t.kvh * G) * D + (lane & 7) * 8;
      float inv = 0.f;
      bool dirty = false;
      if (t.tiles > 0) {
        const int h = g + t.tiles - 1;
        bool w = tc::mbar_wait(&sh.sums_in[used & 1], (used >> 1) & 1) &&
                 tc2::wait(&sh.flags_in[used & 3], (used >> 2) & 1);
        const float total = sh.sums[used & 1][0][row] + sh.sums[used & 1][1][row];
        inv = total == 0.f ? 0.f : 1.f / total;
        dirty = sh.poison[used & 3] == (uint32_t)used + 1;
        w = w && of_tile(sh.o_done, h);
        tc::fence_after_sync();
        if (!(ok = __all_sync(kFullMask, w) != 0)) break;
      }
      // kOut columns at a time (a thread has a row), through shared memory: stored from
      // there in rows of 128 bytes.  (With 32 bytes a row, as the threads hold them, 64
      // KB took 3,900 cycles, in which the softmax warps' next tile took 3,400 for 1,450.)
#pragma unroll 1
      for (int i = 0; i < D; i += C::kOut) {
        float ov[C::kOut];
        if (t.tiles > 0) {
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
        if (dirty && real) {
          const int whole = t.off + t.tok0 + 1;
          const int first = max(0, whole) & ~15;  // first key of those that were edited
          const __nv_bfloat16* vr = static_cast<const __nv_bfloat16*>(p.v) + (int64_t)t.kvh * D + i;
          for (int key = first; key < lim; ++key) {
            const uint32_t* src = reinterpret_cast<const uint32_t*>(vr + ((int64_t)t.k0 + key) * p.v_stride);
#pragma unroll
            for (int k = 0; k < C::kOut / 2; ++k) {
              const uint32_t two = __ldg(src + k);
              ov[2 * k] += poison_of(two & 0xffffu);
              ov[2 * k + 1] += poison_of(two >> 16);
            }
          }
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
      if (t.tiles > 0) {
        g += t.tiles;
        ++used;
      }
    }
  } else {
    tc2::fewer_registers<64>();
    if (warp == kScheduleWarp) {
      // ------------------------------------------------------------ schedule
      const int pairs = gridDim.x / 2, me = blockIdx.x / 2;
      Schedule sc(p, tokens, lane, false);
      bool more = sh.tile[0].tiles >= 0;
      for (int pass = 1; more; ++pass) {
        // pass by pass in alternating direction, so that the pairs' sums come out alike
        const int64_t i = (int64_t)pass * pairs + ((pass & 1) ? pairs - 1 - me : me);
        const int r = i <= INT32_MAX ? (int)i / p.h_kv : (int)(i / p.h_kv);
        Tile t;
        more = sc.get(p, r, (int)(i - (int64_t)r * p.h_kv), &t);
        if (!more) t.tiles = -1;
        if (pass >= 2 && !__all_sync(kFullMask, tc::mbar_wait(&sh.tile_empty[pass & 1], ((pass >> 1) - 1) & 1))) {
          ok = false;
          break;
        }
        if (lane == 0) {
          sh.tile[pass & 1] = t;
          tc::mbar_arrive(&sh.tile_full[pass & 1]);
        }
      }
    } else if (warp == kTmaWarp) {
      // ------------------------------------------------------------ copies
      Tile t;
      int g = 0, used = 0;  // key tiles, tiles with Q so far
      int kc = 0, vc = 0;   // key tiles whose K, V were asked for
      int ve = 0;           // edge tiles among the latter
      const uint32_t r_k = tc2::in_cta(sh.k_full, 0), r_v = tc2::in_cta(sh.v_full, 0);
      const uint32_t r_ve = tc2::in_cta(sh.v_edge, 0), r_q = tc2::in_cta(&sh.q_full, 0);
      if (lane == 0) {
        tc::prefetch_tmap(&tm_q);
        tc::prefetch_tmap(&tm_k);
        tc::prefetch_tmap(&tm_v);
      }
      for (int pass = 0; next_tile(pass, &t); ++pass) {
        if (t.tiles == 0) continue;
        if (lane == 0) {
          const int whole = t.off + t.tok0 + 1;
          if (used > 0) ok = tc::mbar_wait(&sh.q_empty, (used - 1) & 1);
          if (ok) {
            if (rank == 0) tc::mbar_arrive_expect_tx(&sh.q_full, 2u * (uint32_t)(tok_cta * G) * D * 2);
            for (int kb = 0; kb < D / 64; ++kb)
              tc2::tma_load_3d(smem + kb * 16384, &tm_q, 64 * kb, t.kvh * G,
                               t.q0 + t.tok0 + (int)rank * tok_cta, r_q);
          }
          for (int j = 0; j < t.tiles + C::kLag && ok; ++j) {
            if (j < t.tiles) {
              const int h = g + j, s = h % C::kSlots;
              if (h >= C::kSlots && !(ok = of_tile(sh.s_done, h - C::kSlots))) break;
              // the bytes of both CTAs count on the even CTA's barrier
              if (rank == 0) tc::mbar_arrive_expect_tx(&sh.k_full[s], 2 * C::kEntry);
#pragma unroll
              for (int kb = 0; kb < D / 64; ++kb)
                tc2::tma_load_3d(smem + C::kK + s * C::kEntry + kb * 8192, &tm_k, 64 * kb, t.kvh,
                                 t.k0 + j * kKeys + (int)rank * 64, r_k + s * 8);
              kc = h + 1;
            }
            const int i = j - C::kLag;
            if (i >= 0) {
              const int h = g + i, s = h % C::kSlots;
              if (h >= C::kSlots && !(ok = of_tile(sh.o_done, h - C::kSlots))) break;
              // So do those of V, in an edge tile on a barrier of its own that the edge warp can
              // count through; v_full keeps step.
              const bool edge = (i + 1) * kKeys > whole;
              const int e = ve % C::kSlots;
              if (rank == 0) {
                tc::mbar_arrive_expect_tx(edge ? &sh.v_edge[e] : &sh.v_full[s], 2 * C::kEntry);
                if (edge) tc::mbar_arrive(&sh.v_full[s]);
              }
#pragma unroll
              for (int kb = 0; kb < D / 128; ++kb)
                tc2::tma_load_3d(smem + C::kV + s * C::kEntry + kb * 16384, &tm_v, (int)rank * (D / 2) + 64 * kb, t.kvh,
                                 t.k0 + i * kKeys, edge ? r_ve + e * 8 : r_v + s * 8);
              vc = h + 1;
              ve += edge;
            }
          }
        }
        g += t.tiles;
        ++used;
        ok = __all_sync(kFullMask, ok);
        if (!ok) break;
      }
      // Copies still in flight land before the CTA ends: after an expired wait, the
      // even CTA's barriers tell of both CTAs' copies.
      if (lane == 0 && rank == 0) {
        for (int h = max(0, kc - C::kSlots); h < kc; ++h) ok = of_tile(sh.k_full, h) && ok;
        for (int h = max(0, vc - C::kSlots); h < vc; ++h) ok = of_tile(sh.v_full, h) && ok;
        for (int e = max(0, ve - C::kSlots); e < ve; ++e) ok = of_tile(sh.v_edge, e) && ok;
        if (used > 0 && !tc::mbar_wait(&sh.q_full, (used - 1) & 1)) ok = false;
      }
    } else if (warp == kMmaWarp) {
      // ------------------------------------------------------------ products
      Tile t;
      int used = 0;  // tiles with Q so far
      // slots of K and V, score tiles to write and to read, and their barriers' phases
      // (counted, not divided: the issue of a product waits for all of this)
      uint32_t ks = 0, k_ph = 0, vs = 0, v_ph = 0, sw = 0, sr = 0, sr_ph = 0;
      const uint32_t idesc_s = tc::idesc_bf16_f32(256, kKeys, false, false);
      const uint32_t idesc_o = tc::idesc_bf16_f32(256, D, false, true);
      const uint64_t dq = tc::smem_desc(sbase, 16, 1024, tc::kLayoutSw128);
      const uint64_t dk = tc::smem_desc(sbase + C::kK, 16, 1024, tc::kLayoutSw128);
      const uint64_t dv = tc::smem_desc(sbase + C::kV, 16384, 1024, tc::kLayoutSw128);
      const bool leader = tc::elect_one();
      auto warp_wait = [&](uint64_t* bar, uint32_t parity) {
        const bool w = tc::mbar_wait(bar, parity);
        tc::fence_after_sync();
        return __all_sync(kFullMask, w) != 0;
      };
      auto step = [](uint32_t& i, uint32_t& ph, uint32_t n) {
        if (++i == n) {
          i = 0;
          ph ^= 1;
        }
      };
      int edges = 0;  // edge tiles so far
      // the even CTA's warp issues for the pair
      for (int pass = 0; rank == 0 && next_tile(pass, &t); ++pass) {
        if (t.tiles == 0) continue;
        ok = warp_wait(&sh.q_full, used & 1);
        const int whole = t.off + t.tok0 + 1;
        for (int j = 0; j < t.tiles + C::kLag && ok; ++j) {
          if (j < t.tiles) {  // S = Q K^T of key tile j
            if (!(ok = warp_wait(&sh.k_full[ks], k_ph))) break;
            if (leader) {
              const uint64_t kd = dk + ((ks * C::kEntry) >> 4);
#pragma unroll
              for (int kk = 0; kk < C::kSteps; ++kk)
                tc2::mma_ss(tmem + sw * kKeys, dq + (((kk >> 2) * 16384 + (kk & 3) * 32) >> 4),
                            kd + (((kk >> 2) * 8192 + (kk & 3) * 32) >> 4), idesc_s, kk > 0);
              tc2::commit(&sh.s_done[ks]);
              if (j == t.tiles - 1) tc2::commit(&sh.q_empty);
            }
            __syncwarp();
            if (++sw == C::kS) sw = 0;
            step(ks, k_ph, C::kSlots);
          }
          const int i = j - C::kLag;
          if (i >= 0) {  // O += P V of key tile i
            bool w = tc::mbar_wait(&sh.v_full[vs], v_ph);
            if ((i + 1) * kKeys > whole) {  // V may have been edited in both CTAs (ordinary writes): acquire those
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
                if (16 * kk < t.sight - i * kKeys)  // no weight beyond
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
        if (!warp_wait(&sh.drained, 0)) ok = false;
      }
    } else if (warp == kEdgeWarp && rank == 0) {
      // ------------------------------------------------------------ edge tiles
      // V of both CTAs, whose bytes all count on this CTA's barriers: see the note at the top.
      // (With a warp for each half, the odd CTA's has to hand over that V has landed there, with
      // a release: 600 prompts of 64 tokens 193 us at D = 128, so 174, though 16 prompts of
      // 1,024 tokens with 8 KV heads of 256 take 218 for 212.)
      Tile t;
      int g = 0, used = 0, edges = 0;
      const uint32_t r_flags = tc2::in_cta(sh.flags_in, 1), r_poison = tc2::in_cta(sh.poison, 1);
      const uint32_t v_even = tc2::in_cta(smem + C::kV, 0) + lane * 16, v_odd = tc2::in_cta(smem + C::kV, 1) + lane * 16;
      for (int pass = 0; next_tile(pass, &t); ++pass) {
        if (t.tiles == 0) continue;
        bool told = false;  // a non-finite value that a row sees
        for (int j = max(0, t.off + t.tok0 + 1) / kKeys; j < t.tiles && ok; ++j) {
          const int h = g + j, rows = t.sight - j * kKeys;  // rows of V that some query sees
          // the first that some does not (rounded down); those before need no care
          const int row0 = max(0, t.off + t.tok0 + 1 - j * kKeys) & ~15;
          if (!(ok = __all_sync(kFullMask, tc2::wait(&sh.v_edge[edges % C::kSlots], (edges / C::kSlots) & 1)))) break;
          const uint32_t slot = h % C::kSlots * C::kEntry;
          // the largest of the magnitudes, as 16-bit integers (a non-finite one is 0x7f80 or
          // more); in a short loop, as it runs once a tile of queries and not from a cache
          // (600 prompts of 64 tokens, D = 128: 188 us unrolled, 169 so, when that was tried)
          uint32_t most = 0;
#pragma unroll 1
          for (int r = row0; r < min(rows, kKeys); r += 16) {
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
        g += t.tiles;
        ++used;
      }
    }
  }
  if (!ok) raise_error(p.err, kErrDeviceTimeout);
  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  tc::cluster_sync();  // neither CTA's memory is in use by the other any more
  tc::fence_after_sync();
  if (warp == 0) tc2::tmem_dealloc(tmem, C::kTmemCols);
}

template <int D>
cudaError_t launch(const AttnPrefillArgs& a, int sms, cudaStream_t stream) {
  using C = Cfg<D>;
  const int G = a.h_q / a.h_kv, tok_cta = kRows / G;
  // with no keys no tile of K or V is ever copied; the maps then describe q
  const bool keys = a.total_k > 0;
  CUtensorMap mq, mk, mv;
  if (!encode(&mq, a.q, D, a.h_q, a.total_q, a.q_stride, G, tok_cta) ||
      !encode(&mk, keys ? a.k : a.q, D, keys ? a.h_kv : 1, keys ? a.total_k : 1, keys ? a.k_stride : a.q_stride,
              1, 64) ||
      !encode(&mv, keys ? a.v : a.q, D, keys ? a.h_kv : 1, keys ? a.total_k : 1, keys ? a.v_stride : a.q_stride,
              1, kKeys))
    return cudaErrorInvalidValue;
  const int smem = (int)(C::kShared + sizeof(Shared<D>));
  static_assert(C::kShared + sizeof(Shared<D>) <= 227 * 1024, "shared memory");
  static PerDeviceOnce attrs;
  cudaError_t e = attrs.run([&] {
    return cudaFuncSetAttribute(attn_prefill_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  });
  if (e != cudaSuccess) return e;
  int64_t pairs = (a.total_q / (2 * tok_cta) + a.num_seqs) * a.h_kv;  // at least as many as tiles
  AttnPrefillArgs args = a;
  // Sequence by sequence where no pair has two tiles (their order does not matter then;
  // seven short prompts 10.8 us by sight, 9.8 so), and where keys and values exceed half of
  // L2, as they would be read from DRAM by tile after tile (16 prompts of 1,024 tokens, 32
  // heads of 256 on 8: 242 us by sight, 224 so; 16 pieces of 576 tokens on 1,024 keys 192
  // and 167; 8 on 4,096 keys, heads of 128, 210 and 181; 28 ragged prompts 858 and 740).
  // Below that even shares are worth more (seven prompts of 1 to 4,096 tokens, 46 MB: 176
  // by sight, 187 by sequence).
  args.by_sequence = pairs <= sms / 2 || a.total_k * a.h_kv * D * 4 > (int64_t)64 << 20;
  if (pairs > sms / 2) pairs = sms / 2;
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
  cfg.gridDim = dim3((unsigned)(2 * pairs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  return cudaLaunchKernelEx(&cfg, attn_prefill_kernel<D>, mq, mk, mv, args);
}

}  // namespace

cudaError_t launch_attn_prefill(const AttnPrefillArgs& a, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  return a.head_dim == 256 ? launch<256>(a, sms, stream) : launch<128>(a, sms, stream);
}

}  // namespace gdn
