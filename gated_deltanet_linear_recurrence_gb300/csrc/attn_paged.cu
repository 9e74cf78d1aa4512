// attn_paged.cu — decode attention over the paged cache: one new query of each
// sequence over the sequence's cached rows, bf16 or e4m3.
//
// For sequence b, query head h on KV head j, over the L_b cached rows
//     s_i = scale q.k_i,   o = sum_i 2^(t_i - m) v_i / sum_i 2^(t_i - m),
//     t_i = s_i log2(e),   m = max_i t_i
// evaluated online: a warp keeps (m, l, O) of the up to eight query heads of a
// KV head and rescales them when m grows.  (m, l, O) of disjoint sets of rows
// join by rescaling to the larger m, which is how warps, and then CTAs, meet.
//
// Bound by HBM: every cached row is read once (8 flops per value and head).
// What the layout is for:
//   * A CTA's share of the batch is a range of units of 64 rows (e4m3: 128) in
//     (sequence, KV head, row) order, as much work for every CTA whatever the lengths
//     are: ragged batches and single long sequences fill the GPU alike.  The shares
//     follow from the device's lengths alone, so each CTA (and the joining pass)
//     works them out for itself, and the workspace is two partial results a CTA.
//   * A warp owns its tiles of 16 rows (e4m3: 32) end to end: a ring of its own in shared
//     memory (24 KB at D = 256 and two CTAs an SM, 12 KB at D = 128 and four, with e4m3
//     three) filled by 16-byte asynchronous copies, warp-level matrix products (m16n8k16:
//     16 rows x 8 query heads), no CTA barrier before the end of a (sequence, KV head).
//     Rows are addressed by eights through the page table, so a page may be smaller than a
//     tile or end anywhere inside it.
//   * The products are S^T = K Q^T and O^T = V^T P^T, whose N = 8 is the number
//     of query heads on a KV head, so no multiply is padding at eight heads; one
//     8x8 register transpose turns S^T's layout into P^T's.
// Rounding: the weights P go to the matrix unit as bf16 pairs hi + lo (16
// significant bits; the second product is free next to the memory time).  Scores,
// maxima, sums and O are fp32.
// With an e4m3 cache a key's unit 2^ke scales its score; the codes widen exactly to f16,
// and q is scaled into f16 by a power of two for each head: exact down to 2^-31 of the
// head's largest, to within 2^-39 of it below, which moves no score that fp32 sums would
// resolve unless the keys are zero where q is large.  A value's code times its unit 2^ve
// is widened exactly to the bf16 that reading the row back gives (above 2^7 the weight
// takes the rest of the unit), so that both caches share one second product with fp32's
// range of exponents.  (Weights in f16, units included, lost rows beside one with a far larger unit, a row of zeros beside small
// values among them.  They took 29.8 us for 131,072 keys, where these take 31.3, and 90
// for 608 sequences of 396 keys, where these take 113: 350,000 instructions an SM then,
// 475,000 now, with latency to match; long batches are as fast.)
// (Products of e4m3 operands themselves, with q and P as sums of e4m3 parts,
// measured slower: at warp level they run as f16 products after a widening.)
//
// Measured (calls back to back, both kernels).  bf16: 64 sequences of 8,192 keys, 16 query
// heads of 256 on 2, 161 us = 6.7 TB/s, 98 % of a plain copy's rate; 48 heads of 128 on 8,
// 40 ragged sequences 154 us = 6.4; 32 on 8, 64 of 4,096 keys 166 us = 6.5, one of 32,768
// 30 us, one of 4,096 10 us (heads of 256 on 2: 9 us).  e4m3: 16 heads of 256 on 2, one
// sequence of 131,072 keys 31 us = 4.3 TB/s, one eight times as long 170 us = 6.3; 48
// heads of 128 on 8, 40 ragged sequences 86 us = 5.8, 20 of 12,040 keys 84 us = 5.9, 152
// of 1,584 keys 91 us = 5.5, 304 of 792 keys 97 us = 5.1, 608 of 396 keys 113 us = 4.4.
// So rows of long sequences stream at 6.5 to 6.9 TB/s, and a call costs about 10 us beside
// that: lengths, table and first rows one after the other (3 us), the last rows' weights,
// the warps' join, and the joining pass (4 to 5 us).  Short sequences of e4m3 rows also
// show a piece's whole tiles: four warps with 13 tiles of 32 rows wait for the one with 4.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math.h>
#include <stdint.h>

#include "attn_common.cuh"
#include "attn_params.h"
#include "params.h"
#include "per_device.h"
#include "rows.cuh"
#include "tc.cuh"

namespace gdn {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kHeads = 8;  // query heads of a KV head, padded (N of the products)
constexpr int kSlots = 2;  // tiles whose row counts and units are kept: one at work, one on its way

// CTAs on an SM, as registers allow (O and Q of a warp: 12 KB at D = 256, 6 at 128; with
// e4m3 at 128 a fourth CTA leaves 128 registers, and 40 ragged sequences take 90 for 86 us,
// though 608 of 396 keys 112 for 113), bytes of a warp's ring, and rows of its tile.
__host__ __device__ constexpr int ctas_per_sm(int D, bool fp8) { return D == 128 ? (fp8 ? 3 : 4) : 2; }
__host__ __device__ constexpr uint32_t ring_bytes(int D) { return D == 128 ? 12288 : 24576; }
__host__ __device__ constexpr int tile_rows(bool fp8) { return fp8 ? 32 : 16; }
// Rows of a unit of work: a tile for each warp.
__host__ __device__ constexpr int unit_rows(bool fp8) { return kWarps * tile_rows(fp8); }

struct TileInfo {     // of a tile on its way through a warp's ring
  uint32_t rows;      // rows to use in each group of eight, a byte a group
  uint32_t pad;
  uint8_t k_unit[32], v_unit[32];  // exponent bytes
};

__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

// 16 bytes from global to shared memory; zeros when !valid (nothing is read)
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// four e4m3 codes widened to two pairs of f16 (exact)
__device__ __forceinline__ void widen(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// an exponent byte's unit in two factors of half its exponent
__device__ __forceinline__ float2 half_units(uint32_t byte) {
  return make_float2(__uint_as_float((byte / 2 + 64) << 23), __uint_as_float((byte - byte / 2 + 63) << 23));
}
// (the weight's part of a row's unit: see value_units)
__device__ __forceinline__ float weight_unit(uint32_t byte) {
  return __uint_as_float((max(byte, kUnitTop) - (kUnitTop - 127)) << 23);
}
__device__ __forceinline__ float lo_part(uint32_t packed, float x) {
  return x - __uint_as_float(packed << 16);
}
__device__ __forceinline__ float hi_part(uint32_t packed, float x) {
  return x - __uint_as_float(packed & 0xffff0000u);
}

// Cached rows of sequence b; 0 for a length outside the table's reach.
__device__ __forceinline__ int length_of(const PagedAttnArgs& p, int b) {
  const int len = __ldg(p.cache_len + b);
  return (len < 0 || (int64_t)len > ((int64_t)p.cache.max_pages << p.cache.page_shift)) ? 0 : len;
}
// Work of one (sequence, KV head): its units, and kPieceCost units more for taking it up
// (q and the first rows arrive, the warps join), so that a CTA with many short
// sequences is not given more than it can do in the same time (40 ragged sequences on 8
// KV heads of 128: 86.0 us with one unit, 86.2 with two, 87.6 with three; without any, a
// sixth more when that was tried).
constexpr int kPieceCost = 1;
template <int kUnit>
__device__ __forceinline__ int64_t span_of(int len) {
  return len > 0 ? kPieceCost + (uint32_t)(len + kUnit - 1) / kUnit : 0;
}

// Sums and largest values over a block's warps, on every thread (two barriers apart
// from each other's use of `at`, one value a warp).
template <int kT>
__device__ __forceinline__ float block_max(float x, float* at) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) x = fmaxf(x, __shfl_xor_sync(kFullMask, x, off));
  if (lane == 0) at[threadIdx.x >> 5] = x;
  __syncthreads();
  x = lane < kT / 32 ? at[lane] : -INFINITY;
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) x = fmaxf(x, __shfl_xor_sync(kFullMask, x, off));
  return x;
}
template <int kT>
__device__ __forceinline__ float block_sum(float x, float* at) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) x += __shfl_xor_sync(kFullMask, x, off);
  if (lane == 0) at[threadIdx.x >> 5] = x;
  __syncthreads();
  x = lane < kT / 32 ? at[lane] : 0.f;
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) x += __shfl_xor_sync(kFullMask, x, off);
  return x;
}

// For up to 32 sequences: all work, and on each lane that before the lane's sequence.
template <int kUnit>
__device__ __forceinline__ int64_t count_work(const PagedAttnArgs& p, int lane, int64_t& total, int64_t& before) {
  const int64_t mine = lane < p.batch ? p.cache.h_kv * span_of<kUnit>(length_of(p, lane)) : 0;
  int64_t incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t y = __shfl_up_sync(kFullMask, incl, off);
    if (lane >= off) incl += y;
  }
  total = __shfl_sync(kFullMask, incl, 31);
  before = incl - mine;
  return incl;
}
// For a whole block: all work, where that of CTA c starts, the sequence b that it falls
// into and the work before that one.  False when there is none for c.
template <int kT, int kUnit>
__device__ __forceinline__ bool find_work(const PagedAttnArgs& p, int c, bool report, int64_t& total, int64_t& u,
                                          int& b, int64_t& base) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (p.batch <= 32) {  // a lane counts a sequence, each warp for itself
    if (report && lane < p.batch && length_of(p, lane) != __ldg(p.cache_len + lane)) raise_error(p.err, kErrBadCacheLen);
    int64_t before;
    const int64_t incl = count_work<kUnit>(p, lane, total, before);
    u = Shares(total, p.ctas).start(c);
    if (u >= total) return false;
    b = __ffs(__ballot_sync(kFullMask, incl > u)) - 1;
    base = __shfl_sync(kFullMask, before, b);
    return true;
  }
  const int per = (p.batch + kT - 1) / kT;  // sequences a thread counts
  const int lo = min(p.batch, tid * per), hi = min(p.batch, lo + per);
  int64_t mine = 0;
  for (int i = lo; i < hi; ++i) {
    const int len = length_of(p, i);
    if (report && len != __ldg(p.cache_len + i)) raise_error(p.err, kErrBadCacheLen);
    mine += p.cache.h_kv * span_of<kUnit>(len);
  }
  int64_t incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t y = __shfl_up_sync(kFullMask, incl, off);
    if (lane >= off) incl += y;
  }
  __shared__ int64_t scan[kT / 32], found_work;
  __shared__ int found;
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  int64_t before = incl - mine;
  total = 0;
#pragma unroll
  for (int w = 0; w < kT / 32; ++w) {
    if (w < warp) before += scan[w];
    total += scan[w];
  }
  u = Shares(total, p.ctas).start(c);
  if (u >= total) return false;
  if (before <= u && u < before + mine) {
    int i = lo;
    for (;; ++i) {
      const int64_t n = p.cache.h_kv * span_of<kUnit>(length_of(p, i));
      if (u < before + n) break;
      before += n;
    }
    found = i;
    found_work = before;
  }
  __syncthreads();
  b = found;
  base = found_work;
  return true;
}

template <int D, bool kFp8>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(D, kFp8)) attn_paged_kernel(const PagedAttnArgs p) {
  constexpr int kRowBytes = kFp8 ? D : 2 * D;
  constexpr uint32_t kRing = ring_bytes(D);
  constexpr int kRows = tile_rows(kFp8), kUnit = unit_rows(kFp8);
  constexpr int kM = kRows / 16;              // row blocks of the products
  constexpr int kGroups = kRows / 8;          // groups of rows within a page
  constexpr uint32_t kEntry = kRows * kRowBytes;  // K or V of a tile
  constexpr int kEntries = 3;  // of the ring: K, V and the next K, or V, K and the next V
  constexpr int kRowLanes = kRowBytes / 16;   // lanes copying a row
  constexpr int kRowsAtOnce = 32 / kRowLanes;
  constexpr int kQ = D / 16;                  // k-steps of S
  constexpr int kChunk = D / 4, kPad = kChunk + 4;  // dims the warps join at once
  static_assert(kEntries * kEntry == kRing, "ring");
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) TileInfo infos[kWarps][kSlots];
  __shared__ float wm[kWarps][kHeads], wl[kWarps][kHeads];
  __shared__ __align__(16) float joined[kWarps][kHeads][kPad];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  tc::wait_prerequisites();  // q, the cache, its table and lengths come from earlier kernels
  tc::allow_dependents();    // the joining pass may be scheduled; it reads only the lengths early

  // ---- this CTA's share
  const int G = p.h_q / p.cache.h_kv;
  int64_t total, u, base;  // all work, this CTA's, and that before its first sequence
  int b;                   // its first sequence
  if (!find_work<kThreads, kUnit>(p, blockIdx.x, blockIdx.x == 0, total, u, b, base)) return;
  const int64_t u_end = Shares(total, p.ctas).start(blockIdx.x + 1);

  const uint32_t ring = tc::smem_u32(smem) + warp * kRing;
  const int quad = lane >> 2, pair = lane & 3;  // fragment row, and column pair
  const uint32_t swz = lane & 7;
  const float score_unit = p.scale * kLog2e;

  // ---- pieces: this CTA's part of one (sequence, KV head) after the other
  int len = length_of(p, b);
  int j = 0, k_lo = 0, k_hi = 0;
  bool from_start = false, whole = false;  // has the first unit; has all of them
  int seq = 0;
  auto next_piece = [&]() {
    while (u < u_end) {
      const int64_t span = span_of<kUnit>(len);
      if (u >= base + p.cache.h_kv * span) {
        base += p.cache.h_kv * span;
        len = length_of(p, ++b);
        continue;
      }
      j = (int)quotient(u - base, span);
      const int64_t r0 = u - base - j * span, r1 = min(span, r0 + (u_end - u));
      u += r1 - r0;
      if (r1 <= kPieceCost) continue;
      const int64_t c0 = max((int64_t)0, r0 - kPieceCost), c1 = r1 - kPieceCost;
      k_lo = (int)(c0 * kUnit);
      k_hi = (int)min((int64_t)len, c1 * kUnit);
      from_start = c0 == 0;
      whole = from_start && r1 == span;
      seq = b;
      return true;
    }
    return false;
  };

  // ---- the warp's tiles: rows k_lo + kRows (warp + kWarps i) ..
  // Tiles start at multiples of 16 rows, so eight rows lie side by side in a page:
  // lane x looks up and keeps group x of the tile being copied.
  int count = 0, first_key = 0;
  const int32_t* table = nullptr;
  TileInfo* info = infos[warp];
  auto page_of = [&](int i) {
    const int key = first_key + kRows * kWarps * i;
    return (i < count && key < k_hi) ? __ldg(table + (key >> p.cache.page_shift)) : -1;
  };
  int next_page = -1;
  uint32_t row = 0;  // first cached row of the lane's group
  int valid = 0;     // rows of the group that hold keys
  uint2 ku = make_uint2(0, 0), vu = ku;  // its exponent bytes, on their way to info
  uint32_t put = 0;  // ring entry to fill
  auto copy = [&](const void* pages) {
    const uint32_t dst = ring + put * kEntry + (lane / kRowLanes) * kRowBytes;
    const int c = lane % kRowLanes, sub = lane / kRowLanes;
    const uint8_t* base = static_cast<const uint8_t*>(pages) + 16 * c + sub * kRowBytes;
#pragma unroll
    for (int x = 0; x < kGroups; ++x) {
      const uint32_t from = __shfl_sync(kFullMask, row, x);
      const int n = __shfl_sync(kFullMask, valid, x);
      const uint8_t* src = base + (size_t)from * kRowBytes;
#pragma unroll
      for (int s = 0; s < 8 / kRowsAtOnce; ++s) {
        const int r = s * kRowsAtOnce + sub;  // row of the group
        copy16(dst + (8 * x + s * kRowsAtOnce) * kRowBytes + ((c ^ r) << 4), src + s * kRowsAtOnce * kRowBytes,
               r < n);
      }
    }
  };
  auto issue_k = [&](int i) {  // a commit group even when no tile is left
    if (kFp8 && i > 0 && i <= count && lane < kGroups) {
      TileInfo& t = info[(i - 1) % kSlots];
      *reinterpret_cast<uint2*>(t.k_unit + 8 * lane) = ku;
      *reinterpret_cast<uint2*>(t.v_unit + 8 * lane) = vu;
    }
    if (i < count) {
      const int key = first_key + kRows * kWarps * i;
      const int page = next_page;
      const bool ok = page >= 0 && page < p.cache.num_pages;
      valid = min(8, max(0, k_hi - key));
      if (valid > 0 && !ok) {
        raise_error(p.err, kErrBadPage);
        valid = 0;
      }
      row = valid > 0 ? (((uint32_t)page * p.cache.h_kv + j) << p.cache.page_shift) +
                            (key & ((1 << p.cache.page_shift) - 1))
                      : 0u;
      if (lane < kGroups) reinterpret_cast<uint8_t*>(&info[i % kSlots].rows)[lane] = (uint8_t)valid;
      if (kFp8 && valid > 0 && lane < kGroups) {
        ku = __ldg(reinterpret_cast<const uint2*>(p.cache.k_exp + row));
        vu = __ldg(reinterpret_cast<const uint2*>(p.cache.v_exp + row));
      }
      next_page = page_of(i + 1);
      copy(p.cache.k_pages);
      if (++put == kEntries) put = 0;
    }
    copy_commit();
  };
  auto issue_v = [&](int i) {
    if (i < count) {
      copy(p.cache.v_pages);
      if (++put == kEntries) put = 0;
    }
    copy_commit();
  };
  auto open = [&]() {  // the piece's first copies
    const int n_tiles = (k_hi - k_lo + kRows - 1) / kRows;
    count = n_tiles > warp ? (n_tiles - warp + kWarps - 1) / kWarps : 0;
    first_key = k_lo + kRows * warp + 8 * (lane & (kGroups - 1));
    table = p.cache.table + (int64_t)seq * p.cache.max_pages;
    next_page = page_of(0);
    issue_k(0);
    issue_v(0);
  };

  // The piece's q, as it is: pairs of dims in the order in which a row's arrive
  // (bf16 2 pair, + 1, 2 pair + 8, + 9 of sixteen; e4m3 4 pair .. + 3).
  uint32_t qf[kQ][2];
  auto load_q = [&]() {
    const __nv_bfloat16* qrow = static_cast<const __nv_bfloat16*>(p.q) + (int64_t)seq * p.q_stride +
                                ((int64_t)j * G + quad) * D;
#pragma unroll
    for (int kk = 0; kk < kQ; ++kk) {
      uint2 x = make_uint2(0, 0);
      if (quad < G) {
        if (kFp8) {
          x = __ldg(reinterpret_cast<const uint2*>(qrow + 16 * kk + 4 * pair));
        } else {
          x.x = __ldg(reinterpret_cast<const uint32_t*>(qrow + 16 * kk + 2 * pair));
          x.y = __ldg(reinterpret_cast<const uint32_t*>(qrow + 16 * kk + 2 * pair + 8));
        }
      }
      qf[kk][0] = x.x;
      qf[kk][1] = x.y;
    }
  };

  uint32_t get = 0;  // ring entry to use
  bool more = next_piece();
  if (more) {
    load_q();  // ahead of the copies: behind every CTA's first ones it took 2 us
    open();
  }
  while (more) {
    const int64_t head0 = (int64_t)seq * p.h_q + (int64_t)j * G;
    // ---- Q^T as the products' B operand: head `quad`, zeros past G
    float unit0 = score_unit, unit1 = score_unit;  // of heads 2 pair, 2 pair + 1
    float rest0 = 1.f, rest1 = 1.f;                // (e4m3: half of q's exponent apart)
    if (kFp8) {
      // scaled by a power of two per head so that f16 holds what bf16 held (see the top)
      float top = 0.f;
#pragma unroll
      for (int kk = 0; kk < kQ; ++kk)
#pragma unroll
        for (int r = 0; r < 2; ++r)
          top = fmaxf(top, fmaxf(fabsf(__uint_as_float(qf[kk][r] << 16)), fabsf(__uint_as_float(qf[kk][r] & 0xffff0000u))));
      top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 1));
      top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 2));
      const int e = min(max((int)(__float_as_uint(top) >> 23), 16), 254) - 127 - 14;
      const float inv = pow2(-e);
#pragma unroll
      for (int kk = 0; kk < kQ; ++kk)
#pragma unroll
        for (int r = 0; r < 2; ++r)
          qf[kk][r] = pack_f16(__uint_as_float(qf[kk][r] << 16) * inv,
                               __uint_as_float(qf[kk][r] & 0xffff0000u) * inv);
      const int e0 = __shfl_sync(kFullMask, e, 8 * pair), e1 = __shfl_sync(kFullMask, e, 8 * pair + 4);
      unit0 *= pow2(e0 / 2);
      unit1 *= pow2(e1 / 2);
      rest0 = pow2(e0 - e0 / 2);
      rest1 = pow2(e1 - e1 / 2);
    }

    float o[kQ][4];
#pragma unroll
    for (int t = 0; t < kQ; ++t)
#pragma unroll
      for (int c = 0; c < 4; ++c) o[t][c] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY;  // references of heads 2 pair, 2 pair + 1
    float l0 = 0.f, l1 = 0.f;              // this lane's rows only

    for (int i = 0; i < count; ++i) {
      // ---- S^T = K Q^T: rows quad and quad + 8 of each block, heads 2 pair, 2 pair + 1
      copy_wait<1>();
      __syncwarp();
      issue_k(i + 1);
      __syncwarp();
      float s[kM][4];
      {
        float acc[2][kM][4];
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int m = 0; m < kM; ++m)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[x][m][c] = 0.f;
        const uint32_t tile = ring + get * kEntry + ((lane & 7) + 8 * ((lane >> 3) & 1)) * kRowBytes;
#pragma unroll
        for (int kk = 0; kk < kRowBytes / 32; ++kk)  // 32 bytes of each row
#pragma unroll
          for (int m = 0; m < kM; ++m) {
            uint32_t r[4];
            ldsm4(tile + 16 * m * kRowBytes + (((2 * kk + (lane >> 4)) ^ swz) << 4), r);
            if (!kFp8) {
              mma_bf16(acc[kk & 1][m], r, qf[kk][0], qf[kk][1]);
            } else {
              uint32_t a[4];
              widen(r[0], a[0], a[2]);
              widen(r[1], a[1], a[3]);
              mma_f16(acc[0][m], a, qf[2 * kk][0], qf[2 * kk][1]);
              widen(r[2], a[0], a[2]);
              widen(r[3], a[1], a[3]);
              mma_f16(acc[1][m], a, qf[2 * kk + 1][0], qf[2 * kk + 1][1]);
            }
          }
#pragma unroll
        for (int m = 0; m < kM; ++m)
#pragma unroll
          for (int c = 0; c < 4; ++c) s[m][c] = acc[0][m][c] + acc[1][m][c];
      }
      if (++get == kEntries) get = 0;
      const TileInfo& ti = info[i % kSlots];
      const uint32_t rows = ti.rows;
      uint32_t vu2[kM][2];  // units of V's rows 2 pair, 2 pair + 1 (and + 8) of each block
#pragma unroll
      for (int m = 0; m < kM; ++m) {
        if (kFp8) {
          // the key's unit and the head's are multiplied in by halves of their exponents, in
          // turn: a large one and a small one whose product is ordinary leave the range nowhere
          const float2 f0 = half_units(ti.k_unit[16 * m + quad]), f1 = half_units(ti.k_unit[16 * m + 8 + quad]);
          s[m][0] = s[m][0] * f0.x * unit0 * f0.y * rest0;
          s[m][1] = s[m][1] * f0.x * unit1 * f0.y * rest1;
          s[m][2] = s[m][2] * f1.x * unit0 * f1.y * rest0;
          s[m][3] = s[m][3] * f1.x * unit1 * f1.y * rest1;
#pragma unroll
          for (int x = 0; x < 2; ++x)
            vu2[m][x] = value_units(ti.v_unit[16 * m + 8 * x + 2 * pair], ti.v_unit[16 * m + 8 * x + 2 * pair + 1]);
        }
        const bool ok0 = quad < (int)((rows >> (16 * m)) & 0xff), ok1 = quad < (int)((rows >> (16 * m + 8)) & 0xff);
        if (!kFp8) {
          s[m][0] *= unit0;
          s[m][1] *= unit1;
          s[m][2] *= unit0;
          s[m][3] *= unit1;
        }
        s[m][0] = ok0 ? s[m][0] : -INFINITY;
        s[m][1] = ok0 ? s[m][1] : -INFINITY;
        s[m][2] = ok1 ? s[m][2] : -INFINITY;
        s[m][3] = ok1 ? s[m][3] : -INFINITY;
      }
      // ---- online softmax; a reference moves when it is exceeded by more than kSlack
      auto col_max = [&](float x) {
#pragma unroll
        for (int off = 4; off <= 16; off <<= 1) x = fmaxf(x, __shfl_xor_sync(kFullMask, x, off));
        return x;
      };
      auto moved = [&](float ref, float top) { return top > ref + kSlack || ref == -INFINITY ? top : ref; };
      float t0 = fmaxf(s[0][0], s[0][2]), t1 = fmaxf(s[0][1], s[0][3]);
#pragma unroll
      for (int m = 1; m < kM; ++m) {
        t0 = fmaxf(t0, fmaxf(s[m][0], s[m][2]));
        t1 = fmaxf(t1, fmaxf(s[m][1], s[m][3]));
      }
      const float n0 = moved(m0, col_max(t0)), n1 = moved(m1, col_max(t1));
      float g0 = n0 == -INFINITY ? 0.f : n0, g1 = n1 == -INFINITY ? 0.f : n1;
      float a0 = 1.f, a1 = 1.f;
      if (__any_sync(kFullMask, n0 != m0 || n1 != m1)) {
        a0 = ex2(m0 - g0);
        a1 = ex2(m1 - g1);
        l0 *= a0;
        l1 *= a1;
      }
      m0 = n0;
      m1 = n1;
      float w[kM][4];
#pragma unroll
      for (int m = 0; m < kM; ++m) {
        w[m][0] = ex2(s[m][0] - g0);
        w[m][1] = ex2(s[m][1] - g1);
        w[m][2] = ex2(s[m][2] - g0);
        w[m][3] = ex2(s[m][3] - g1);
        l0 += w[m][0] + w[m][2];
        l1 += w[m][1] + w[m][3];
      }
      if (kFp8) {
#pragma unroll
        for (int m = 0; m < kM; ++m) {
          const float e0 = weight_unit(ti.v_unit[16 * m + quad]), e1 = weight_unit(ti.v_unit[16 * m + 8 + quad]);
          w[m][0] *= e0;
          w[m][1] *= e0;
          w[m][2] *= e1;
          w[m][3] *= e1;
        }
      }
      if (__any_sync(kFullMask, a0 != 1.f || a1 != 1.f)) {
#pragma unroll
        for (int t = 0; t < kQ; ++t) {
          o[t][0] *= a0;
          o[t][1] *= a1;
          o[t][2] *= a0;
          o[t][3] *= a1;
        }
      }
      // ---- P^T as the B operand
      uint32_t ph[kM][2], pl[kM][2];
#pragma unroll
      for (int m = 0; m < kM; ++m) {
        const uint32_t x = pack_bf16(w[m][0], w[m][1]), y = pack_bf16(w[m][2], w[m][3]);
        ph[m][0] = transpose8x8(x);
        ph[m][1] = transpose8x8(y);
        pl[m][0] = transpose8x8(pack_bf16(lo_part(x, w[m][0]), hi_part(x, w[m][1])));
        pl[m][1] = transpose8x8(pack_bf16(lo_part(y, w[m][2]), hi_part(y, w[m][3])));
      }
      // ---- O^T += V^T P^T
      copy_wait<1>();
      __syncwarp();
      issue_v(i + 1);
      const uint32_t vt = ring + get * kEntry;
      if (++get == kEntries) get = 0;
      if (!kFp8) {
        const uint32_t tile = vt + ((lane & 7) + 8 * (lane >> 4)) * kRowBytes;
#pragma unroll
        for (int t = 0; t < kQ; ++t)
#pragma unroll
          for (int m = 0; m < kM; ++m) {
            uint32_t r[4];
            ldsm4t(tile + 16 * m * kRowBytes + (((2 * t + ((lane >> 3) & 1)) ^ swz) << 4), r);
            mma_bf16(o[t], r, ph[m][0], ph[m][1]);
            mma_bf16(o[t], r, pl[m][0], pl[m][1]);
          }
      } else {
        const uint32_t tile = vt + ((lane & 7) + 8 * ((lane >> 3) & 1)) * kRowBytes;
        // (row blocks outside: the products of one accumulator far apart; the other way
        // round 131,072 keys took 32.7 for 31.3 us)
        uint32_t most = 0;
#pragma unroll
        for (int m = 0; m < kM; ++m)
#pragma unroll
          for (int t = 0; t < kQ; t += 2) {
            uint32_t r[4];  // chunks t (r0: rows 0-7, r1: 8-15) and t + 1 (r2, r3)
            ldsm4t(tile + 16 * m * kRowBytes + (((t + (lane >> 4)) ^ swz) << 4), r);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              // bytes (row 2 pair: dims 2 quad, 2 quad + 1; row 2 pair + 1: the same)
              uint32_t a[4];
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const uint32_t c = r[2 * h + x];
                const uint32_t even = even_magnitudes(c), odd = odd_magnitudes(c);
                most = __vimax3_u16x2(most, even, odd);
                a[2 * x] = times(even | ((c << 8) & kSigns), vu2[m][x]);
                a[2 * x + 1] = times(odd | (c & kSigns), vu2[m][x]);
              }
              mma_bf16(o[t + h], a, ph[m][0], ph[m][1]);
              mma_bf16(o[t + h], a, pl[m][0], pl[m][1]);
            }
          }
        // a value that is not finite makes its dimension of every head so
        if (__any_sync(kFullMask, nan_code(most))) {
#pragma unroll
          for (int t = 0; t < kQ; t += 2)
#pragma unroll 1
            for (int m = 0; m < kM; ++m) {
              uint32_t r[4];
              ldsm4t(tile + 16 * m * kRowBytes + (((t + (lane >> 4)) ^ swz) << 4), r);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t a[4] = {
                    nan_where(even_magnitudes(r[2 * h])), nan_where(odd_magnitudes(r[2 * h])),
                    nan_where(even_magnitudes(r[2 * h + 1])), nan_where(odd_magnitudes(r[2 * h + 1]))};
                mma_bf16(o[t + h], a, 0x3f803f80u, 0x3f803f80u);
              }
            }
        }
      }
    }
    copy_wait<0>();
    __syncwarp();

    // ---- join the warps, a quarter of the dimensions at a time; the next piece's
    // first copies are on their way meanwhile
#pragma unroll
    for (int off = 4; off <= 16; off <<= 1) {
      l0 += __shfl_xor_sync(kFullMask, l0, off);
      l1 += __shfl_xor_sync(kFullMask, l1, off);
    }
    if (quad == 0) {
      wm[warp][2 * pair] = m0;
      wm[warp][2 * pair + 1] = m1;
      wl[warp][2 * pair] = l0;
      wl[warp][2 * pair + 1] = l1;
    }
    const bool to_o = whole;
    const int64_t part = ((int64_t)blockIdx.x * 2 + (from_start ? 1 : 0)) * G;
    more = next_piece();
    if (more) open();
    __syncthreads();
    float t0 = wm[0][2 * pair], t1 = wm[0][2 * pair + 1];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
      t0 = fmaxf(t0, wm[w][2 * pair]);
      t1 = fmaxf(t1, wm[w][2 * pair + 1]);
    }
    const float f0 = m0 == -INFINITY ? 0.f : ex2(m0 - t0), f1 = m1 == -INFINITY ? 0.f : ex2(m1 - t1);
    // the head and the four dims that this thread finishes
    const int h = tid / (kChunk / 4), d4 = tid % (kChunk / 4);
    float M = -INFINITY, l = 0.f, r = 0.f;
    if (h < G) {
      M = wm[0][h];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) M = fmaxf(M, wm[w][h]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) l += wm[w][h] == -INFINITY ? 0.f : wl[w][h] * ex2(wm[w][h] - M);
      // l > 0 whenever a row was seen; NaN stays NaN
      r = l == 0.f ? 0.f : 1.f / l;
      if (!to_o && d4 == 0)
        reinterpret_cast<float2*>(p.partial + (int64_t)p.ctas * 2 * G * D)[part + h] = make_float2(M, l);
    }
#pragma unroll
    for (int x = 0; x < D / kChunk; ++x) {
#pragma unroll
      for (int y = 0; y < kQ / 4; ++y) {
        const int t = x * (kQ / 4) + y;
        // e4m3: rows of V^T interleave two dims (see the products above)
        const int d0 = 16 * y + (kFp8 ? 2 * quad : quad), d1 = kFp8 ? d0 + 1 : d0 + 8;
        joined[warp][2 * pair][d0] = o[t][0] * f0;
        joined[warp][2 * pair + 1][d0] = o[t][1] * f1;
        joined[warp][2 * pair][d1] = o[t][2] * f0;
        joined[warp][2 * pair + 1][d1] = o[t][3] * f1;
      }
      __syncthreads();
      if (h < G) {
        float4 a = *reinterpret_cast<const float4*>(&joined[0][h][4 * d4]);
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
          const float4 y = *reinterpret_cast<const float4*>(&joined[w][h][4 * d4]);
          a.x += y.x;
          a.y += y.y;
          a.z += y.z;
          a.w += y.w;
        }
        a = make_float4(a.x * r, a.y * r, a.z * r, a.w * r);
        const int d = x * kChunk + 4 * d4;
        if (to_o)
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + (head0 + h) * D + d) =
              make_uint2(pack_bf16(a.x, a.y), pack_bf16(a.z, a.w));
        else
          *reinterpret_cast<float4*>(p.partial + (part + h) * D + d) = a;
      }
      __syncthreads();
    }
    if (more) load_q();
  }
}

// The results of a (sequence, KV head) whose units went to several CTAs:
//     o = sum_s w_s o_s / sum_s w_s,   w_s = 2^(m_s - M) l_s,   M = max_s m_s
// with each CTA's o_s already divided by its l_s.  Also writes the zeros of sequences
// without cached rows.  With up to kFew splits of an item (a sequence's KV head) one
// block does all query heads, a warp each; with more, several share out the heads and
// kSlices parts of their dims, a lane four values of a row, the splits dealt to the
// groups of lanes, eight loads in flight in each.
// Few rows of o (kByItem): a block for every item, head and part.  Else a block for
// every boundary between two CTAs' shares: what the boundaries that fall into an item
// show is all that there is to join, and they are its blocks.  (A block for every item
// and head, most of them with nothing to join, took 110 of 187 us for 608 sequences
// with 8 KV heads, when that was tried; these take 9.)
// Few splits, measured (bf16, 16 heads of 256 on 2): 16 sequences of 4,096 keys, 10 splits
// an item, 29.9 us with a limit of 16, 27.6 with 8; one of 2,048 keys, 32 splits, 15.0 us
// with a limit of 32, 7.9 with 8.
constexpr int kFew = 8;
template <int D, int kUnit, int kJoinThreads, int kSlices>
__global__ void __launch_bounds__(kJoinThreads) attn_paged_join_kernel(const PagedAttnArgs p) {
  constexpr int kRow = D / 4, kLanes = kRow / kSlices, kGroups = kJoinThreads / kLanes;
  constexpr bool kByItem = kSlices > 1;
  __shared__ float w_sm[kPagedMaxCtas];
  __shared__ float red[2][kJoinThreads / 32];
  __shared__ float4 sum_sm[kGroups][kLanes];
  // (The next call's kernel is not let in early: with its CTAs taking their places
  // between these blocks, 40 sequences with 8 KV heads took 105 for 89 us, when tried.)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h_kv = p.cache.h_kv, G = p.h_q / h_kv;
  int64_t total = 0, u, base;
  int b = 0, j = 0, c_lo = 0, n = 1;  // the block's item; its first CTA, its splits
  int mine = 0, blocks = G * kSlices;  // the block's number among the item's
  if (kByItem) {  // at most 32 sequences
    mine = blockIdx.x % blocks;
    j = blockIdx.x / blocks % h_kv;
    b = blockIdx.x / blocks / h_kv;
    count_work<kUnit>(p, lane, total, base);
    base = __shfl_sync(kFullMask, base, b);
  } else if (blockIdx.x + 1 >= p.ctas || !find_work<kJoinThreads, kUnit>(p, blockIdx.x + 1, false, total, u, b, base)) {
    total = 0;
  }
  const int64_t span = total > 0 ? span_of<kUnit>(length_of(p, b)) : 0;
  if (span > 0) {
    if (!kByItem) j = (int)quotient(u - base, span);
    const int64_t first = base + (int64_t)j * span + kPieceCost, end = base + (int64_t)(j + 1) * span;
    const Shares sh(total, p.ctas);
    c_lo = sh.owner(first);
    n = sh.owner(end - 1) - c_lo + 1;
    if (!kByItem) {
      mine = (int)blockIdx.x - c_lo;
      blocks = n - 1;
      if (mine < 0) n = 1;  // not inside the item's units
    }
  }
  int empty = blockIdx.x;  // a sequence without cached rows
  while (empty < p.batch && length_of(p, empty) > 0) empty += gridDim.x;
  // every block waits: the kernel after this one takes its end for that of both
  tc::wait_prerequisites();
  for (; empty < p.batch; empty += gridDim.x)
    if (length_of(p, empty) == 0)
      for (int d = tid; d < p.h_q * D / 8; d += kJoinThreads)
        reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o) + (int64_t)empty * p.h_q * D)[d] = make_uint4(0, 0, 0, 0);
  if (n == 1) return;  // written by its CTA
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.o) + ((int64_t)b * p.h_q + (int64_t)j * G) * D;
  // the CTA with the first unit wrote slot 1, those that start inside it slot 0
  auto part = [&](int s, int h) { return ((int64_t)(c_lo + s) * 2 + (s == 0)) * G + h; };
  const float4* acc_in = reinterpret_cast<const float4*>(p.partial);
  const float2* ml_in = reinterpret_cast<const float2*>(p.partial + (int64_t)p.ctas * 2 * G * D);
  auto add = [](float4& a, float f, const float4& v) {
    if (f != 0.f) {
      a.x = fmaf(f, v.x, a.x);
      a.y = fmaf(f, v.y, a.y);
      a.z = fmaf(f, v.z, a.z);
      a.w = fmaf(f, v.w, a.w);
    }
  };
  auto store = [&](int h, int d4, const float4& a, float den) {
    const float r = den == 0.f ? 0.f : 1.f / den;
    *reinterpret_cast<uint2*>(o + (int64_t)h * D + 4 * d4) =
        make_uint2(pack_bf16(a.x * r, a.y * r), pack_bf16(a.z * r, a.w * r));
  };
  if (n <= kFew) {
    const int h = warp;
    if (mine > 0 || h >= G) return;
    float2 ml = lane < n ? ml_in[part(lane, h)] : make_float2(-INFINITY, 0.f);
    float4 a[D / 128];
#pragma unroll
    for (int k = 0; k < D / 128; ++k) a[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    float mx = ml.x;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFullMask, mx, off));
    const float w = ml.x == -INFINITY ? 0.f : ex2(ml.x - mx) * ml.y;
    float den = w;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) den += __shfl_xor_sync(kFullMask, den, off);
#pragma unroll 4
    for (int s = 0; s < n; ++s) {
      const float f = __shfl_sync(kFullMask, w, s);
#pragma unroll
      for (int k = 0; k < D / 128; ++k) add(a[k], f, acc_in[part(s, h) * kRow + 32 * k + lane]);
    }
#pragma unroll
    for (int k = 0; k < D / 128; ++k) store(h, 32 * k + lane, a[k], den);
    return;
  }
  for (int x = mine; x < G * kSlices; x += blocks) {  // query head, part of its dims
    const int h = x % G, grp = tid / kLanes, d4 = tid % kLanes + x / G * kLanes;
    float4 in[8];  // the first loads go out before the weights are known
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int s = grp + k * kGroups;
      in[k] = s < n ? acc_in[part(s, h) * kRow + d4] : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    constexpr int kMine = (kPagedMaxCtas + kJoinThreads - 1) / kJoinThreads;  // splits a thread
    float2 ml[kMine];
    float mx = -INFINITY;
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
      const int s = tid + k * kJoinThreads;
      ml[k] = s < n ? ml_in[part(s, h)] : make_float2(-INFINITY, 0.f);
      mx = fmaxf(mx, ml[k].x);
    }
    mx = block_max<kJoinThreads>(mx, red[0]);
    float den = 0.f;
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
      const float w = ml[k].x == -INFINITY ? 0.f : ex2(ml[k].x - mx) * ml[k].y;
      if (tid + k * kJoinThreads < n) w_sm[tid + k * kJoinThreads] = w;
      den += w;
    }
    den = block_sum<kJoinThreads>(den, red[1]);  // and every thread's weights are in w_sm
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (grp + k * kGroups < n) add(a, w_sm[grp + k * kGroups], in[k]);
#pragma unroll 8
    for (int s = grp + 8 * kGroups; s < n; s += kGroups) add(a, w_sm[s], acc_in[part(s, h) * kRow + d4]);
    sum_sm[grp][tid % kLanes] = a;
    __syncthreads();
    if (grp == 0) {
#pragma unroll
      for (int g = 1; g < kGroups; ++g) {
        const float4 y = sum_sm[g][tid % kLanes];
        a.x += y.x;
        a.y += y.y;
        a.z += y.z;
        a.w += y.w;
      }
      store(h, d4, a, den);
    }
    __syncthreads();
  }
}

template <int D, bool kFp8>
cudaError_t launch_paged(const PagedAttnArgs& args, cudaStream_t stream) {
  static PerDeviceOnce attrs;
  const size_t smem = kWarps * ring_bytes(D);
  cudaError_t e = attrs.run([&] {
    return cudaFuncSetAttribute(attn_paged_kernel<D, kFp8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)smem);
  });
  if (e != cudaSuccess) return e;
  // both kernels launch while the kernel before them drains, and wait for its
  // results before they read them
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3((unsigned)args.ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  e = cudaLaunchKernelEx(&cfg, attn_paged_kernel<D, kFp8>, args);
  if (e != cudaSuccess) return e;
  cfg.dynamicSmemBytes = 0;
  // Few rows of o, with many splits each: by item.  Measured: 16 heads of 256 on 2, bf16, one
  // sequence of 32,768 keys 13.5 us by item and 16.2 by boundary, four of 16,384 28.7 and
  // 29.1; past 64 rows the other way, 32 heads of 128 on 8, e4m3, four of 16,384 keys 36.1
  // and 31.3.
  if ((int64_t)args.batch * args.h_q <= 64 && args.batch <= 32) {
    cfg.gridDim = dim3((unsigned)(args.batch * args.h_q * 4));
    cfg.blockDim = dim3(512);
    return cudaLaunchKernelEx(&cfg, attn_paged_join_kernel<D, unit_rows(kFp8), 512, 4>, args);
  }
  cfg.gridDim = dim3((unsigned)(args.ctas > 1 ? args.ctas - 1 : 1));
  cfg.blockDim = dim3(256);
  return cudaLaunchKernelEx(&cfg, attn_paged_join_kernel<D, unit_rows(kFp8), 256, 1>, args);
}

}  // namespace

size_t paged_attn_workspace_bytes(int32_t h_q, int32_t h_kv, int32_t head_dim) {
  return (size_t)kPagedMaxCtas * 2 * (h_q / h_kv) * (head_dim + 2) * sizeof(float);
}

cudaError_t launch_attn_decode_paged(const PagedAttnArgs& a, cudaStream_t stream) {
  if (a.batch == 0) return cudaSuccess;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  PagedAttnArgs args = a;
  // As many CTAs as are resident at once, but no more than units the table can reach.
  const bool fp8 = a.cache.dtype == kCacheE4M3;
  const int unit = unit_rows(fp8);
  const int64_t reach = ((int64_t)a.cache.max_pages << a.cache.page_shift) + unit - 1;
  const int64_t units = (int64_t)a.batch * a.cache.h_kv * (reach / unit);
  int64_t ctas = (int64_t)ctas_per_sm(a.cache.head_dim, fp8) * sms;
  if (ctas > kPagedMaxCtas) ctas = kPagedMaxCtas;
  if (ctas > units) ctas = units > 0 ? units : 1;
  args.ctas = (int32_t)ctas;
  if (a.cache.head_dim == 256)
    return fp8 ? launch_paged<256, true>(args, stream) : launch_paged<256, false>(args, stream);
  return fp8 ? launch_paged<128, true>(args, stream) : launch_paged<128, false>(args, stream);
}

}  // namespace gdn
