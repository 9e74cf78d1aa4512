// kv_rows.cuh — where packed tokens lie in the paged cache, and a row's 8-bit form: shared
// by the kernels that write the cache and read it back.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "attn_params.h"
#include "params.h"
#include "rows.cuh"

namespace gdn {

// Largest n in [0, N) with cu[n] <= t, for the whole warp (32 probes a step).
// Entries out of order only make the answer wrong, which the caller checks (and then
// looks through all sequences).
__device__ __forceinline__ int find_sequence(const int32_t* cu, int N, int t, int lane) {
  int lo = 0, hi = N;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + lane * step;
    const unsigned below = __ballot_sync(kFullMask, i < hi && __ldg(cu + i) <= t);
    const int c = __popc(below);
    if (c == 0) return lo;
    lo += (c - 1) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// The first sequence whose range holds token t, by looking at each; -1 when none does.
// For offsets out of order, among which the search by halves loses its way.
static __device__ __noinline__ int look_for_sequence(const KvRowsArgs& a, int t, int lane) {
  for (int base = 0; base < a.num_seqs; base += 32) {
    const int n = base + lane;
    bool holds = false;
    if (n < a.num_seqs) {
      const int c0 = __ldg(a.cu_seqlens + n), c1 = __ldg(a.cu_seqlens + n + 1);
      holds = c0 >= 0 && c0 <= t && t < c1 && c1 <= a.total_tokens;
    }
    const unsigned hit = __ballot_sync(kFullMask, holds);
    if (hit) return base + __ffs(hit) - 1;
  }
  return -1;
}

// The sequence n that token t belongs to and its position there; false when no range
// holds it (offsets out of order are recorded).
__device__ __forceinline__ bool token_position(const KvRowsArgs& a, int t, int lane, int& n, int64_t& pos) {
  n = find_sequence(a.cu_seqlens, a.num_seqs, t, lane);
  int c0 = __ldg(a.cu_seqlens + n), c1 = __ldg(a.cu_seqlens + n + 1);
  if (c0 < 0 || t < c0 || t >= c1) {
    if (lane == 0) raise_error(a.err, kErrBadCuSeqlens);
    n = look_for_sequence(a, t, lane);
    if (n < 0) return false;
    c0 = __ldg(a.cu_seqlens + n);
  }
  pos = (int64_t)__ldg(a.start + n) + (t - c0);
  return true;
}

// Index of the cached row of (position pos of sequence n, head 0), or -1 (with the error
// recorded).  Rows of the other heads follow page_size apart.
__device__ __forceinline__ int64_t position_row(const KvRowsArgs& a, int n, int64_t pos, int lane) {
  const int64_t pi = pos >> a.cache.page_shift;
  int page = -1;
  if (pos >= 0 && pi < a.cache.max_pages)
    page = __ldg(a.cache.table + (int64_t)n * a.cache.max_pages + pi);
  if (page < 0 || page >= a.cache.num_pages) {
    if (lane == 0) raise_error(a.err, kErrBadPage);
    return -1;
  }
  const int slot = (int)(pos & ((1 << a.cache.page_shift) - 1));
  return (((int64_t)page * a.cache.h_kv) << a.cache.page_shift) + slot;
}

// The same of (token t, head 0).
__device__ __forceinline__ int64_t token_row(const KvRowsArgs& a, int t, int lane) {
  int n;
  int64_t pos;
  return token_position(a, t, lane, n, pos) ? position_row(a, n, pos, lane) : -1;
}

// The packing itself: cu[0] = 0, no range decreases, cu[N] = T.  The warps share the
// sequences out, 32 at a time: one that owns no token has no warp of its own to look.
__device__ __forceinline__ void check_packing(const KvRowsArgs& a, int t, int lane) {
  for (int64_t n = (int64_t)t * 32 + lane; n < a.num_seqs; n += a.total_tokens * 32) {
    const int c0 = __ldg(a.cu_seqlens + n), c1 = __ldg(a.cu_seqlens + n + 1);
    if (c1 < c0 || (n == 0 && c0 != 0) || (n == a.num_seqs - 1 && c1 != a.total_tokens))
      raise_error(a.err, kErrBadCuSeqlens);
  }
}

__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

// Exponent of a row's unit from the bits of its largest finite |x| (a bf16).
// 448 = 1.75 * 2^8, and |x| = (1 + m / 128) 2^(b - 127).
__device__ __forceinline__ int unit_exponent(uint32_t bits) {
  if (bits == 0) return 0;
  const int b = (int)(bits >> 7);
  return max(-126, b - 127 - ((bits & 0x7f) <= 96 ? 8 : 7));
}

// 8 bf16 values of a row spread over kLanes lanes -> 8 e4m3 codes, and the row's
// exponent byte (on every lane).
template <int kLanes>
__device__ __forceinline__ uint2 quantise_row(uint4 x, int lane, uint32_t* byte) {
  uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t top = 0;  // largest |x| of the lane, per 16-bit half, as bits
#pragma unroll
  for (int i = 0; i < 4; ++i) top = __vmaxu2(top, w[i] & 0x7fff7fffu);
  top = max(top & 0xffffu, top >> 16);
  auto row_max = [&](uint32_t v) {
#pragma unroll
    for (int off = kLanes / 2; off >= 1; off >>= 1) v = max(v, __shfl_xor_sync(kFullMask, v, off));
    return v;
  };
  top = row_max(top);
  if (__any_sync(kFullMask, top >= 0x7f80u)) {  // inf or NaN in a row of the warp
    uint32_t fin = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = w[i] & 0x7fffu, hi = (w[i] >> 16) & 0x7fffu;
      fin = max(fin, lo < 0x7f80u ? lo : 0u);
      fin = max(fin, hi < 0x7f80u ? hi : 0u);
      if (lo >= 0x7f80u) w[i] = (w[i] & 0xffff0000u) | 0x7fc0u;
      if (hi >= 0x7f80u) w[i] = (w[i] & 0x0000ffffu) | 0x7fc00000u;
    }
    top = row_max(fin);
  }
  const int e = unit_exponent(top);
  const float inv = pow2(-e);
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 f;
    f.x = __uint_as_float(w[i] << 16) * inv;
    f.y = __uint_as_float(w[i] & 0xffff0000u) * inv;
    c[i] = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
  }
  *byte = (uint32_t)(e + 127);
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

}  // namespace gdn
