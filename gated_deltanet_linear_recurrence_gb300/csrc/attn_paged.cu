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
//   * A CTA's share of the batch is a range of 64-row units in (sequence, KV
//     head, row) order, the same number for every CTA whatever the lengths are:
//     ragged batches and single long sequences fill the GPU alike.  The shares
//     follow from the device's lengths alone, so each CTA (and the joining pass)
//     works them out for itself, and the workspace is two partial results a CTA.
//   * A warp owns its 16-row tiles end to end: a ring of its own in shared
//     memory filled by 16-byte asynchronous copies, warp-level matrix products
//     (m16n8k16: 16 rows x 8 query heads), no CTA barrier before the end of a
//     (sequence, KV head).  Rows are addressed one by one through the page table,
//     so a page may be smaller than a tile or end anywhere inside it.
//   * The products are S^T = K Q^T and O^T = V^T P^T, whose N = 8 is the number
//     of query heads on a KV head, so no multiply is padding at eight heads; one
//     8x8 register transpose turns S^T's layout into P^T's.
// Rounding: the weights P go to the matrix unit as bf16 pairs hi + lo (16
// significant bits; the second product is free next to the memory time), or with
// an e4m3 cache as f16, to which e4m3 values widen exactly.  Scores, maxima, sums
// and O are fp32.
// With an e4m3 cache a key's unit 2^ke scales its score, and a value's unit 2^ve
// joins the exponent, 2^(t_i + ve_i - m') with m' = max_i (t_i + ve_i), so that
// the f16 weights use their range whatever the units are; l keeps its own m.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math.h>
#include <stdint.h>

#include "attn_params.h"
#include "params.h"
#include "per_device.h"
#include "rows.cuh"
#include "tc.cuh"

namespace gdn {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kUnit = 64;  // rows in a unit of work: one 16-row tile for each warp
constexpr int kTileRows = 16;
constexpr int kHeads = 8;  // query heads of a KV head, padded (N of the products)
constexpr uint32_t kRing = 24576;  // bytes of a warp's ring: two CTAs fit on an SM
constexpr int kTileSlots = 8;      // tiles whose row validity and units are kept
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
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
template <bool kF16>
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                      uint32_t a3, uint32_t b0, uint32_t b1) {
  if (kF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// two e4m3 codes (the low 16 bits) widened to f16
__device__ __forceinline__ uint32_t widen(uint32_t codes) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(codes & 0xffffu), __NV_E4M3);
  return (uint32_t)h.x | ((uint32_t)h.y << 16);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
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
__device__ __forceinline__ int64_t units_of(const PagedAttnArgs& p, int len) {
  return (int64_t)p.cache.h_kv * ((len + (int64_t)kUnit - 1) / kUnit);
}

// Units of the sequences before `upto`, and of the whole batch, on every thread.
template <int kT>
__device__ __forceinline__ void count_units(const PagedAttnArgs& p, int upto, int64_t* before,
                                            int64_t* total) {
  __shared__ int64_t sums[2][kT / 32];
  int64_t s = 0, all = 0;
  for (int b = threadIdx.x; b < p.batch; b += kT) {
    const int64_t u = units_of(p, length_of(p, b));
    all += u;
    if (b < upto) s += u;
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) {
    s += __shfl_xor_sync(kFullMask, s, off);
    all += __shfl_xor_sync(kFullMask, all, off);
  }
  if ((threadIdx.x & 31) == 0) {
    sums[0][threadIdx.x >> 5] = s;
    sums[1][threadIdx.x >> 5] = all;
  }
  __syncthreads();
  s = all = 0;
#pragma unroll
  for (int w = 0; w < kT / 32; ++w) {
    s += sums[0][w];
    all += sums[1][w];
  }
  *before = s;
  *total = all;
}

// The units of CTA c: the first `more` CTAs have size + 1 of them, the others size
// (CTAs beyond the number of units none).
struct Shares {
  int64_t size, more, split;
  __device__ __forceinline__ Shares(int64_t total, int ctas) {
    size = total / ctas;
    more = total - size * ctas;
    split = more * (size + 1);
  }
  __device__ __forceinline__ int64_t start(int c) const { return c * size + min((int64_t)c, more); }
  __device__ __forceinline__ int owner(int64_t u) const {
    return u < split ? (int)(u / (size + 1)) : (int)(more + (u - split) / size);
  }
};

template <int D, bool kFp8>
__global__ void __launch_bounds__(kThreads, 2) attn_paged_kernel(const PagedAttnArgs p) {
  constexpr int kRowBytes = kFp8 ? D : 2 * D;
  constexpr uint32_t kEntry = kTileRows * kRowBytes;  // K or V of a tile
  constexpr int kEntries = kRing / kEntry;
  constexpr int kRowLanes = kRowBytes / 16;   // lanes copying a row
  constexpr int kRowsAtOnce = 32 / kRowLanes;
  constexpr int kQ = D / 16;                  // k-steps of S
  constexpr int kPad = D + 4;                 // floats between heads in the warps' join
  static_assert(kEntries >= 3 && kEntries / 2 + 1 < kTileSlots, "ring");
  static_assert(kHeads * kPad * 4 <= kRing, "join buffer");
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint8_t row_unit[kWarps][kTileSlots][32];  // exponent bytes: 16 keys, 16 values
  __shared__ uint32_t row_ok[kWarps][kTileSlots];       // rows of a tile that hold a key
  __shared__ float wm[kWarps][kHeads], wv[kWarps][kHeads], wl[kWarps][kHeads];
  __shared__ int64_t at_units;
  __shared__ int at_seq;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  tc::wait_prerequisites();  // q, the cache, its table and lengths come from earlier kernels
  tc::allow_dependents();    // the joining pass may be scheduled; it reads only the lengths early

  // ---- this CTA's units
  const int G = p.h_q / p.cache.h_kv;
  const int per = (p.batch + kThreads - 1) / kThreads;  // sequences a thread counts
  const int b_lo = min(p.batch, tid * per), b_hi = min(p.batch, b_lo + per);
  int64_t mine = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    const int len = length_of(p, b);
    if (blockIdx.x == 0 && len != __ldg(p.cache_len + b)) raise_error(p.err, kErrBadCacheLen);
    mine += units_of(p, len);
  }
  __shared__ int64_t scan[kWarps];
  int64_t incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t y = __shfl_up_sync(kFullMask, incl, off);
    if (lane >= off) incl += y;
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  int64_t total = 0, before = incl - mine;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += scan[w];
    total += scan[w];
  }
  const Shares sh(total, gridDim.x);
  const int64_t u_start = sh.start(blockIdx.x), u_end = sh.start(blockIdx.x + 1);
  if (u_start == u_end) return;
  int64_t u = u_start;
  if (before <= u && u < before + mine) {
    int b = b_lo;
    for (;; ++b) {
      const int64_t n = units_of(p, length_of(p, b));
      if (u < before + n) break;
      before += n;
    }
    at_seq = b;
    at_units = before;
  }
  __syncthreads();
  int b = at_seq;
  int64_t base = at_units;

  const uint32_t ring = tc::smem_u32(smem) + warp * kRing;
  const int quad = lane >> 2, pair = lane & 3;  // fragment row, and column pair
  const uint32_t swz_k = lane & 7, swz_v = lane & 7;
  const float score_unit = p.scale * kLog2e;

  while (u < u_end) {
    int len = length_of(p, b);
    while (u >= base + units_of(p, len)) {
      base += units_of(p, len);
      len = length_of(p, ++b);
    }
    const int64_t tiles = (len + kUnit - 1) / kUnit;  // units of one KV head
    const int j = (int)((u - base) / tiles);
    const int64_t c0 = (u - base) % tiles;
    const int64_t c1 = min(tiles, c0 + (u_end - u));
    const int k_lo = (int)(c0 * kUnit), k_hi = (int)min((int64_t)len, c1 * kUnit);
    const int64_t head0 = (int64_t)b * p.h_q + (int64_t)j * G;
    const int32_t* table = p.cache.table + (int64_t)b * p.cache.max_pages;

    // ---- Q^T as the products' B operand: head `quad`, zeros past G
    uint32_t qf[kQ][2];
    float unit0 = score_unit, unit1 = score_unit;  // of heads 2 pair, 2 pair + 1
    {
      const __nv_bfloat16* qrow = static_cast<const __nv_bfloat16*>(p.q) + (int64_t)b * p.q_stride +
                                  ((int64_t)j * G + quad) * D;
      if (!kFp8) {
#pragma unroll
        for (int kk = 0; kk < kQ; ++kk) {
          const uint32_t* s = reinterpret_cast<const uint32_t*>(qrow + 16 * kk + 2 * pair);
          qf[kk][0] = quad < G ? __ldg(s) : 0u;
          qf[kk][1] = quad < G ? __ldg(s + 4) : 0u;
        }
      } else {
        // dims 16 kk + 4 pair .. + 3 in two registers, the order in which the
        // widened codes of a row arrive; scaled by a power of two per head so
        // that f16 holds what bf16 held (down to 2^-38 of the head's largest)
        float top = 0.f;
#pragma unroll
        for (int kk = 0; kk < kQ; ++kk) {
          uint2 x = make_uint2(0, 0);
          if (quad < G) x = __ldg(reinterpret_cast<const uint2*>(qrow + 16 * kk + 4 * pair));
          qf[kk][0] = x.x;
          qf[kk][1] = x.y;
          top = fmaxf(top, fmaxf(fmaxf(fabsf(__uint_as_float(x.x << 16)), fabsf(__uint_as_float(x.x & 0xffff0000u))),
                                 fmaxf(fabsf(__uint_as_float(x.y << 16)), fabsf(__uint_as_float(x.y & 0xffff0000u)))));
        }
        top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 1));
        top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 2));
        const int e = min(max((int)((__float_as_uint(top) >> 23) & 0xff), 16), 240) - 127 - 14;
        const float inv = pow2(-e);
#pragma unroll
        for (int kk = 0; kk < kQ; ++kk)
#pragma unroll
          for (int r = 0; r < 2; ++r)
            qf[kk][r] = pack_f16(__uint_as_float(qf[kk][r] << 16) * inv,
                                 __uint_as_float(qf[kk][r] & 0xffff0000u) * inv);
        unit0 *= __shfl_sync(kFullMask, pow2(e), 8 * pair);
        unit1 *= __shfl_sync(kFullMask, pow2(e), 8 * pair + 4);
      }
    }

    // ---- the warp's tiles: rows k_lo + 16 (warp + kWarps i) ..
    const int n_tiles = (k_hi - k_lo + kTileRows - 1) / kTileRows;
    const int count = n_tiles > warp ? (n_tiles - warp + kWarps - 1) / kWarps : 0;
    const int last = count * 2;  // ring entries: K, V, K, V, ...
    const int my_row = lane & 15;
    auto page_of = [&](int i) {  // page of this lane's row of tile i; -1: no row
      const int key = k_lo + kTileRows * (warp + kWarps * i) + my_row;
      return (i < count && key < k_hi) ? __ldg(table + (key >> p.cache.page_shift)) : -1;
    };
    int next_page = page_of(0);
    uint32_t row = 0;         // this lane's cached row of the tile being copied
    bool row_valid = false;
    uint32_t unit_byte = 0;   // exponent byte on its way to row_unit
    auto issue = [&](int e) {  // copy entry e (a commit group even when there is none left)
      const int i = e >> 1;
      if ((e & 1) == 0) {
        if (kFp8 && i > 0 && i <= count) row_unit[warp][(i - 1) % kTileSlots][lane] = (uint8_t)unit_byte;
        if (i < count) {
          const int key = k_lo + kTileRows * (warp + kWarps * i) + my_row;
          const int page = next_page;
          row_valid = key < k_hi && page >= 0 && page < p.cache.num_pages;
          if (key < k_hi && !row_valid) raise_error(p.err, kErrBadPage);
          row = row_valid ? (((uint32_t)page * p.cache.h_kv + j) << p.cache.page_shift) +
                                (key & ((1 << p.cache.page_shift) - 1))
                          : 0u;
          const unsigned ok = __ballot_sync(kFullMask, row_valid);
          if (lane == 0) row_ok[warp][i % kTileSlots] = ok & 0xffffu;
          if (kFp8) unit_byte = row_valid ? (lane < 16 ? p.cache.k_exp[row] : p.cache.v_exp[row]) : 127u;
          next_page = page_of(i + 1);
        }
      }
      if (e < last) {
        const uint8_t* src = static_cast<const uint8_t*>((e & 1) ? p.cache.v_pages : p.cache.k_pages);
        const uint32_t dst = ring + (uint32_t)(e % kEntries) * kEntry;
        const int c = lane % kRowLanes;
#pragma unroll
        for (int s = 0; s < kTileRows / kRowsAtOnce; ++s) {
          const int r = s * kRowsAtOnce + lane / kRowLanes;
          const uint32_t from = __shfl_sync(kFullMask, row, r);
          const bool ok = __shfl_sync(kFullMask, (int)row_valid, r) != 0;
          copy16(dst + r * kRowBytes + ((c ^ (r & 7)) << 4), src + (size_t)from * kRowBytes + 16 * c, ok);
        }
      }
      copy_commit();
    };
#pragma unroll
    for (int e = 0; e < kEntries - 1; ++e) issue(e);

    float o[kQ][4];
#pragma unroll
    for (int t = 0; t < kQ; ++t)
#pragma unroll
      for (int c = 0; c < 4; ++c) o[t][c] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY;  // of heads 2 pair, 2 pair + 1
    float v0 = -INFINITY, v1 = -INFINITY;  // maxima with the values' units (e4m3)
    float l0 = 0.f, l1 = 0.f;              // this lane's rows only

    for (int i = 0; i < count; ++i) {
      // ---- S^T = K Q^T: rows quad and quad + 8, heads 2 pair and 2 pair + 1
      copy_wait<kEntries - 2>();
      __syncwarp();
      issue(2 * i + kEntries - 1);
      float s[4];
      {
        float acc[4][4];
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[x][c] = 0.f;
        const uint32_t tile = ring + (uint32_t)((2 * i) % kEntries) * kEntry +
                              ((lane & 7) + 8 * ((lane >> 3) & 1)) * kRowBytes;
#pragma unroll
        for (int kk = 0; kk < (kFp8 ? kQ / 2 : kQ); ++kk) {
          uint32_t r[4];
          ldsm4(tile + (((2 * kk + (lane >> 4)) ^ swz_k) << 4), r);
          if (!kFp8) {
            mma16<false>(acc[kk & 3], r[0], r[1], r[2], r[3], qf[kk][0], qf[kk][1]);
          } else {
            mma16<true>(acc[(2 * kk) & 3], widen(r[0]), widen(r[1]), widen(r[0] >> 16), widen(r[1] >> 16),
                        qf[2 * kk][0], qf[2 * kk][1]);
            mma16<true>(acc[(2 * kk + 1) & 3], widen(r[2]), widen(r[3]), widen(r[2] >> 16),
                        widen(r[3] >> 16), qf[2 * kk + 1][0], qf[2 * kk + 1][1]);
          }
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) s[c] = (acc[0][c] + acc[1][c]) + (acc[2][c] + acc[3][c]);
      }
      const uint32_t ok = row_ok[warp][i % kTileSlots];
      const bool ok0 = (ok >> quad) & 1, ok1 = (ok >> (quad + 8)) & 1;
      float ve0 = 0.f, ve1 = 0.f;
      if (kFp8) {
        const uint8_t* ub = row_unit[warp][i % kTileSlots];
        const float k0 = pow2((int)ub[quad] - 127), k1 = pow2((int)ub[quad + 8] - 127);
        ve0 = (float)((int)ub[16 + quad] - 127);
        ve1 = (float)((int)ub[24 + quad] - 127);
        s[0] *= k0;
        s[1] *= k0;
        s[2] *= k1;
        s[3] *= k1;
      }
      s[0] = ok0 ? s[0] * unit0 : -INFINITY;
      s[1] = ok0 ? s[1] * unit1 : -INFINITY;
      s[2] = ok1 ? s[2] * unit0 : -INFINITY;
      s[3] = ok1 ? s[3] * unit1 : -INFINITY;
      // ---- online softmax
      auto col_max = [&](float x) {
#pragma unroll
        for (int off = 4; off <= 16; off <<= 1) x = fmaxf(x, __shfl_xor_sync(kFullMask, x, off));
        return x;
      };
      const float n0 = fmaxf(m0, col_max(fmaxf(s[0], s[2])));
      const float n1 = fmaxf(m1, col_max(fmaxf(s[1], s[3])));
      const float g0 = n0 == -INFINITY ? 0.f : n0, g1 = n1 == -INFINITY ? 0.f : n1;
      float e0 = ex2(s[0] - g0), e1 = ex2(s[1] - g1), e2 = ex2(s[2] - g0), e3 = ex2(s[3] - g1);
      float a0 = ex2(m0 - g0), a1 = ex2(m1 - g1);
      l0 = fmaf(l0, a0, e0 + e2);
      l1 = fmaf(l1, a1, e1 + e3);
      m0 = n0;
      m1 = n1;
      if (kFp8) {
        const float x0 = fmaxf(v0, col_max(fmaxf(s[0] + ve0, s[2] + ve1)));
        const float x1 = fmaxf(v1, col_max(fmaxf(s[1] + ve0, s[3] + ve1)));
        const float h0 = x0 == -INFINITY ? 0.f : x0, h1 = x1 == -INFINITY ? 0.f : x1;
        e0 = ex2(s[0] + ve0 - h0);
        e1 = ex2(s[1] + ve0 - h1);
        e2 = ex2(s[2] + ve1 - h0);
        e3 = ex2(s[3] + ve1 - h1);
        a0 = ex2(v0 - h0);
        a1 = ex2(v1 - h1);
        v0 = x0;
        v1 = x1;
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
      uint32_t b0, b1, c0 = 0, c1 = 0;
      if (kFp8) {
        b0 = transpose8x8(pack_f16(e0, e1));
        b1 = transpose8x8(pack_f16(e2, e3));
      } else {
        const uint32_t x = pack_bf16(e0, e1), y = pack_bf16(e2, e3);
        b0 = transpose8x8(x);
        b1 = transpose8x8(y);
        c0 = transpose8x8(pack_bf16(lo_part(x, e0), hi_part(x, e1)));
        c1 = transpose8x8(pack_bf16(lo_part(y, e2), hi_part(y, e3)));
      }
      // ---- O^T += V^T P^T
      copy_wait<kEntries - 2>();
      __syncwarp();
      issue(2 * i + kEntries);
      const uint32_t vt = ring + (uint32_t)((2 * i + 1) % kEntries) * kEntry;
      if (!kFp8) {
        const uint32_t tile = vt + ((lane & 7) + 8 * (lane >> 4)) * kRowBytes;
#pragma unroll
        for (int t = 0; t < kQ; ++t) {
          uint32_t r[4];
          ldsm4t(tile + (((2 * t + ((lane >> 3) & 1)) ^ swz_v) << 4), r);
          mma16<false>(o[t], r[0], r[1], r[2], r[3], b0, b1);
          mma16<false>(o[t], r[0], r[1], r[2], r[3], c0, c1);
        }
      } else {
        const uint32_t tile = vt + ((lane & 7) + 8 * ((lane >> 3) & 1)) * kRowBytes;
#pragma unroll
        for (int t = 0; t < kQ; t += 2) {
          uint32_t r[4];  // chunks t (r0: rows 0-7, r1: 8-15) and t + 1 (r2, r3)
          ldsm4t(tile + (((t + (lane >> 4)) ^ swz_v) << 4), r);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            // bytes (row 2 pair: dims 2 quad, 2 quad + 1; row 2 pair + 1: the same)
            const uint32_t x = __byte_perm(r[2 * h], 0, 0x3120), y = __byte_perm(r[2 * h + 1], 0, 0x3120);
            mma16<true>(o[t + h], widen(x), widen(x >> 16), widen(y), widen(y >> 16), b0, b1);
          }
        }
      }
    }
    copy_wait<0>();
    __syncwarp();

    // ---- join the warps
#pragma unroll
    for (int off = 4; off <= 16; off <<= 1) {
      l0 += __shfl_xor_sync(kFullMask, l0, off);
      l1 += __shfl_xor_sync(kFullMask, l1, off);
    }
    if (!kFp8) {
      v0 = m0;
      v1 = m1;
    }
    if (quad == 0) {
      wm[warp][2 * pair] = m0;
      wm[warp][2 * pair + 1] = m1;
      wv[warp][2 * pair] = v0;
      wv[warp][2 * pair + 1] = v1;
      wl[warp][2 * pair] = l0;
      wl[warp][2 * pair + 1] = l1;
    }
    __syncthreads();
    {
      float t0 = wv[0][2 * pair], t1 = wv[0][2 * pair + 1];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) {
        t0 = fmaxf(t0, wv[w][2 * pair]);
        t1 = fmaxf(t1, wv[w][2 * pair + 1]);
      }
      const float f0 = v0 == -INFINITY ? 0.f : ex2(v0 - t0), f1 = v1 == -INFINITY ? 0.f : ex2(v1 - t1);
      float* buf = reinterpret_cast<float*>(smem + warp * kRing);
#pragma unroll
      for (int t = 0; t < kQ; ++t) {
        // e4m3: rows of V^T interleave two dims (see the products above)
        const int d0 = 16 * t + (kFp8 ? 2 * quad : quad), d1 = kFp8 ? d0 + 1 : d0 + 8;
        buf[(2 * pair) * kPad + d0] = o[t][0] * f0;
        buf[(2 * pair + 1) * kPad + d0] = o[t][1] * f1;
        buf[(2 * pair) * kPad + d1] = o[t][2] * f0;
        buf[(2 * pair + 1) * kPad + d1] = o[t][3] * f1;
      }
    }
    __syncthreads();
    const bool whole = c0 == 0 && c1 == tiles;
    const int slot = u_start > base + (int64_t)j * tiles ? 0 : 1;
    float* part = p.partial + ((int64_t)blockIdx.x * 2 + slot) * G * (D + 2);
    for (int x = tid; x < G * D; x += kThreads) {
      const int h = x / D, d = x % D;
      float M = wm[0][h], T = wv[0][h];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) {
        M = fmaxf(M, wm[w][h]);
        T = fmaxf(T, wv[w][h]);
      }
      float l = 0.f, acc = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        l += wm[w][h] == -INFINITY ? 0.f : wl[w][h] * ex2(wm[w][h] - M);
        acc += reinterpret_cast<const float*>(smem + w * kRing)[h * kPad + d];
      }
      // l > 0 whenever a row was seen; NaN stays NaN
      const float r = l == 0.f ? 0.f : acc * (kFp8 ? ex2(T - M) : 1.f) / l;
      if (whole) {
        static_cast<__nv_bfloat16*>(p.o)[(head0 + h) * D + d] = __float2bfloat16_rn(r);
      } else {
        part[h * (D + 2) + d] = r;
        if (d == 0) {
          part[h * (D + 2) + D] = M;
          part[h * (D + 2) + D + 1] = l;
        }
      }
    }
    __syncthreads();  // the buffers are refilled by the next (sequence, KV head)
    u += c1 - c0;
  }
}

// The results of a (sequence, KV head) whose units went to several CTAs:
//     o = sum_s w_s o_s / sum_s w_s,   w_s = 2^(m_s - M) l_s,   M = max_s m_s
// with each CTA's o_s already divided by its l_s.  Also writes the zeros of a
// sequence without cached rows.  One block per (sequence, KV head, query head).
constexpr int kJoinThreads = 256;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) attn_paged_join_kernel(const PagedAttnArgs p) {
  __shared__ float w_sm[kPagedMaxCtas];
  __shared__ float red[kJoinThreads / 32];
  __shared__ float sum_sm[kJoinThreads];
  tc::allow_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h_kv = p.cache.h_kv, G = p.h_q / h_kv;
  const int b = blockIdx.x / h_kv, j = blockIdx.x % h_kv, h = blockIdx.y;
  int64_t base, total;
  count_units<kJoinThreads>(p, b, &base, &total);
  const int64_t tiles = (length_of(p, b) + (int64_t)kUnit - 1) / kUnit;
  const int64_t first = base + (int64_t)j * tiles, end = first + tiles;
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.o) + ((int64_t)b * p.h_q + (int64_t)j * G + h) * D;
  tc::wait_prerequisites();
  if (tiles == 0) {
    for (int d = tid; d < D; d += kJoinThreads) o[d] = __float2bfloat16_rn(0.f);
    return;
  }
  const Shares sh(total, p.ctas);
  const int c_lo = sh.owner(first), c_hi = sh.owner(end - 1);
  if (c_lo == c_hi) return;  // written by its CTA
  const int n = c_hi - c_lo + 1;
  // the CTA with the first unit wrote slot 1, those that start inside it slot 0
  auto part = [&](int s) {
    return p.partial + (((int64_t)(c_lo + s) * 2 + (s == 0)) * G + h) * (D + 2);
  };
  float mx = -INFINITY;
  for (int s = tid; s < n; s += kJoinThreads) {
    const float m = part(s)[D];
    w_sm[s] = m;
    mx = fmaxf(mx, m);
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFullMask, mx, off));
  if (lane == 0) red[warp] = mx;
  __syncthreads();
  mx = red[0];
#pragma unroll
  for (int w = 1; w < kJoinThreads / 32; ++w) mx = fmaxf(mx, red[w]);
  __syncthreads();
  float den = 0.f;
  for (int s = tid; s < n; s += kJoinThreads) {
    const float m = w_sm[s];
    const float w = m == -INFINITY ? 0.f : ex2(m - mx) * part(s)[D + 1];
    w_sm[s] = w;
    den += w;
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) den += __shfl_xor_sync(kFullMask, den, off);
  if (lane == 0) red[warp] = den;
  __syncthreads();
  den = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinThreads / 32; ++w) den += red[w];
  constexpr int kGroups = kJoinThreads / D;
  const int d = tid % D, grp = tid / D;
  float acc = 0.f;
#pragma unroll 8
  for (int s = grp; s < n; s += kGroups) {
    const float w = w_sm[s];
    acc += w == 0.f ? 0.f : w * part(s)[d];
  }
  if (kGroups > 1) {
    sum_sm[tid] = acc;
    __syncthreads();
    if (grp > 0) return;
#pragma unroll
    for (int g = 1; g < kGroups; ++g) acc += sum_sm[g * D + d];
  }
  o[d] = __float2bfloat16_rn(den == 0.f ? 0.f : acc / den);
}

template <int D, bool kFp8>
cudaError_t launch_paged(const PagedAttnArgs& args, cudaStream_t stream) {
  static PerDeviceOnce attrs;
  const size_t smem = kWarps * kRing;
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
  cfg.gridDim = dim3((unsigned)(args.batch * args.cache.h_kv), (unsigned)(args.h_q / args.cache.h_kv));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, attn_paged_join_kernel<D>, args);
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
  // Two CTAs are resident on an SM; no more CTAs than units the table can reach.
  const int64_t reach = ((int64_t)a.cache.max_pages << a.cache.page_shift) + kUnit - 1;
  const int64_t units = (int64_t)a.batch * a.cache.h_kv * (reach / kUnit);
  int64_t ctas = 2 * (int64_t)sms;
  if (ctas > kPagedMaxCtas) ctas = kPagedMaxCtas;
  if (ctas > units) ctas = units > 0 ? units : 1;
  args.ctas = (int32_t)ctas;
  const bool fp8 = a.cache.dtype == kCacheE4M3;
  if (a.cache.head_dim == 256)
    return fp8 ? launch_paged<256, true>(args, stream) : launch_paged<256, false>(args, stream);
  return fp8 ? launch_paged<128, true>(args, stream) : launch_paged<128, false>(args, stream);
}

}  // namespace gdn
