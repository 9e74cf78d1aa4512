// rope.cu — what stands between an attention layer's projections and its attention: the
// RMS norms of the heads of q and k, their rotation by the token's position, and k with v
// on into the paged cache.
//
// A head's row x of D values, with a weight w, and pairs (x_a, x_b) of its first R dims
// (a, b = i, i + R / 2, or 2 i, 2 i + 1) turned by the angle p f_i of frequency i:
//     y = w x / sqrt(sum x^2 / D + eps)
//     y_a' = y_a cos(p f_i) - y_b sin(p f_i),   y_b' = y_b cos(p f_i) + y_a sin(p f_i)
// all in fp32 and rounded once, to bf16 (an e4m3 row is quantised from that, so that it is
// the row which the dense form followed by gdn_kv_append would leave).
//
// Angles.  p f_i of far positions loses its fraction of a turn in 32 bits.  Here a
// frequency is the 64-bit fraction F = f_i / 2 pi mod 1 in units of 2^-64 turns (an integer
// product with the first 128 bits of 1 / 2 pi), and p F mod 2^64 is the angle's fraction of
// a turn to within 2^-33 for any 32-bit p: one integer product, and sincospif takes it.
//
// Bound by HBM: each row in once, out once.  A warp takes a token, or some of its rows
// where there are few tokens, and works the angles out once for all of them.  A lane has
// eight values of a row, such that a pair's two are its own and no lane asks another for
// its half: of the dims that turn as i and i + R / 2 four and their four partners (two
// 8-byte accesses), else eight in a row.
//
// Measured (calls back to back in a graph): 32,768 tokens of 32 + 8 heads of 128 in 107 us, 6.27
// TB/s, 92 % of a plain copy's rate; a ragged batch of 27,878 into bf16 pages, with v, 104 us,
// 97 %; 9,001 tokens of 16 + 4 heads of 128 on three axes 20 us, floor 13.6 (1.9 waves of
// warps); a step of 64 tokens 3.9 us, of 256 into e4m3 pages 6.3 (latency).  Choices, for the
// first two of those: blocks of four warps with 64 registers 107 and 105 us, of eight with 80
// 119 and 111, nine blocks an SM (56 registers) 112 and 109; four rows under way 107, two 126,
// eight 116.  A token's rows are shared out only while that many warps fit at once, as each
// works the angles out again: with twice as many 9,001 tokens take 28 us for 20.
#include <cuda_bf16.h>

#include "attn_params.h"
#include "kv_rows.cuh"
#include "params.h"
#include "rows.cuh"
#include "tc.cuh"

namespace gdn {
namespace {

constexpr int kWarps = 4;
constexpr int kAhead = 4;  // rows (D = 256; pairs of rows at 128) whose loads a warp has under way

enum class To { kDense, kBF16, kE4M3 };

// f / 2 pi mod 1 in units of 2^-64, for finite f.  f = m 2^e with integer m, and P = m C
// with C = floor(2^128 / 2 pi) is the product in units of 2^(e - 128).
__device__ __forceinline__ uint64_t turns(float f) {
  constexpr uint64_t kC1 = 0x28be60db9391054aull, kC0 = 0x7f09d5f47d4d3770ull;
  const uint32_t bits = __float_as_uint(f);
  const int ex = (int)((bits >> 23) & 0xff);
  const uint64_t m = (bits & 0x7fffffu) | (ex ? 0x800000u : 0u);
  const int s = 64 - (max(ex, 1) - 150);  // P >> s counts units of 2^-64
  const uint64_t p0 = m * kC0;
  uint64_t p1 = m * kC1, p2 = __umul64hi(m, kC1);
  const uint64_t c = __umul64hi(m, kC0);
  p1 += c;
  p2 += p1 < c;
  uint64_t r;
  if (s >= 128) r = s < 192 ? p2 >> (s - 128) : 0;
  else if (s > 64) r = (p1 >> (s - 64)) | (p2 << (128 - s));
  else if (s == 64) r = p1;
  else if (s > 0) r = (p0 >> s) | (p1 << (64 - s));
  else r = p0 << -s;  // (|f| of 2^41 and more: the last bits are not there)
  return (bits >> 31) ? 0 - r : r;
}

__device__ __forceinline__ float4 widen4(uint2 x) {
  return make_float4(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u), __uint_as_float(x.y << 16),
                     __uint_as_float(x.y & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// What a lane knows for all rows of its token: where its eight values lie, and the
// rotation of its four pairs.
struct Turn {
  int da, db;  // first of its four dims, and of the other four
  bool turns;
  float c[4], s[4];
};

// 1 / sqrt(mean of squares + eps).  Squares of values beyond 2^63 overflow and of values
// below 2^-63 vanish, where that matters beside eps: the row is scaled by a power of two
// then (a and b with it).
template <int D, int kLanes>
__device__ __forceinline__ float norm_factor(float4& a, float4& b, float eps) {
  float ss = group_sum<kLanes>(dot4(b, b, dot4(a, a, 0.f)));
  const bool large = !(ss < 0x1p100f), small = ss < 0x1p-100f && eps < 0x1p-80f;
  if (__any_sync(kFullMask, large || small)) {
    const float f = large ? 0x1p-100f : small ? 0x1p100f : 1.f;
    a = make_float4(a.x * f, a.y * f, a.z * f, a.w * f);
    b = make_float4(b.x * f, b.y * f, b.z * f, b.w * f);
    ss = group_sum<kLanes>(dot4(b, b, dot4(a, a, 0.f)));
    eps = eps * f * f;
  }
  return rsqrtf(fmaf(ss, 1.f / D, eps));
}

template <int D, bool kPairs, To kTo>
__global__ void __launch_bounds__(kWarps * 32, 8) rope_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int kLanes = D / 8;        // lanes per row
  constexpr int kHeads = 32 / kLanes;  // rows a warp holds at once
  tc::allow_dependents();
  tc::wait_prerequisites();
  const int lane = threadIdx.x & 31;
  const int l = lane % kLanes, sub = lane / kLanes;
  const int q_groups = (a.h_q + kHeads - 1) / kHeads, k_groups = (a.h_kv + kHeads - 1) / kHeads;
  const int all = q_groups + (kTo == To::kDense ? 1 : 2) * k_groups;
  const int parts = (all + a.groups - 1) / a.groups;  // warps that share a token
  const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int64_t tt = parts == 1 ? w : w / parts;
  if (tt >= a.rows.total_tokens) return;
  const int t = (int)tt;
  const int g0 = (int)(w - tt * parts) * a.groups, g1 = min(all, g0 + a.groups);

  Turn u;
  const int turning = a.rotary / 8;  // lanes of a row that hold dims which turn
  u.turns = l < turning;
  if (kPairs) {
    u.da = 8 * l;
    u.db = u.da + 4;
  } else {
    u.da = u.turns ? 4 * l : 8 * l;
    u.db = u.turns ? a.rotary / 2 + 4 * l : 8 * l + 4;
  }

  // rows of one of q, k and v: groups [from, to) of kHeads heads, loaded kAhead at a time
  // (the first ones before anything else)
  uint2 xa[kAhead], xb[kAhead];
  auto load = [&](const void* base, int64_t stride, int heads, int from, int to) {
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(base) + t * stride;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int h = (from + i) * kHeads + sub;
      xa[i] = xb[i] = make_uint2(0, 0);
      if (from + i < to && h < heads) {
        xa[i] = *reinterpret_cast<const uint2*>(src + (int64_t)h * D + u.da);
        xb[i] = *reinterpret_cast<const uint2*>(src + (int64_t)h * D + u.db);
      }
    }
  };
  // the sections' groups that are this warp's
  const int q_from = g0, q_to = min(g1, q_groups);
  const int k_from = max(g0, q_groups) - q_groups, k_to = min(g1, q_groups + k_groups) - q_groups;
  const int v_from = max(g0, q_groups + k_groups) - q_groups - k_groups, v_to = g1 - q_groups - k_groups;
  if (q_from < q_to) load(a.q, a.q_stride, a.h_q, q_from, q_to);
  else if (k_from < k_to) load(a.rows.k, a.rows.k_stride, a.h_kv, k_from, k_to);
  else if (kTo != To::kDense) load(a.rows.v, a.rows.v_stride, a.h_kv, v_from, v_to);

  // ---- where the token is
  int64_t pos = 0, row0 = 0;
  bool placed = true;
  if (kTo != To::kDense) {
    int n = t;
    // (one token of each sequence, as a decoding step has: no search, 8.9 us for 256 with it)
    const bool step = t < a.rows.num_seqs && __ldg(a.rows.cu_seqlens + t) == t && __ldg(a.rows.cu_seqlens + t + 1) == t + 1;
    if (step) pos = __ldg(a.rows.start + t);
    else placed = token_position(a.rows, t, lane, n, pos);
    if (g0 == 0) check_packing(a.rows, t, lane);
    if (!placed) return;
    row0 = g1 > q_groups ? position_row(a.rows, n, pos, lane) : -1;
  }
  // ---- the rotation of the lane's pairs: frequencies 4 l ..
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    u.c[i] = 1.f;
    u.s[i] = 0.f;
  }
  if (u.turns && g0 < q_groups + k_groups) {
    const float4 f4 = make_float4(__ldg(a.inv_freq + 4 * l), __ldg(a.inv_freq + 4 * l + 1),
                                  __ldg(a.inv_freq + 4 * l + 2), __ldg(a.inv_freq + 4 * l + 3));
    const float f[4] = {f4.x, f4.y, f4.z, f4.w};
    int64_t p[4] = {pos, pos, pos, pos};
    if (a.positions) {
      const int64_t T = a.rows.total_tokens;
      p[0] = p[1] = p[2] = p[3] = __ldg(a.positions + t);
      if (a.axes > 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = __ldg(a.positions + a.axis_of[4 * l + i] * T + t);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t part = (uint64_t)p[i] * turns(f[i]);
      // half turns from -1 to 1
      const float x = (float)(int32_t)(part >> 32) * 0x1p-31f;
      sincospif(isfinite(f[i]) ? x : f[i] * 0.f, &u.s[i], &u.c[i]);
    }
  }

  // ---- the rows
  auto section = [&](const void* base, int64_t stride, int heads, int from, int to, bool loaded, const float* weight,
                     bool normed, bool turned, auto&& store) {
    float4 wa = make_float4(1.f, 1.f, 1.f, 1.f), wb = wa;
    if (normed && weight) {
      wa = __ldg(reinterpret_cast<const float4*>(weight + u.da));
      wb = __ldg(reinterpret_cast<const float4*>(weight + u.db));
    }
    for (int g = from; g < to; g += kAhead) {
      if (!loaded) load(base, stride, heads, g, to);
      loaded = false;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (g + i >= to) break;
        const int h = (g + i) * kHeads + sub;
        uint2 ya = xa[i], yb = xb[i];
        if (normed || turned) {
          float4 x = widen4(xa[i]), y = widen4(xb[i]);
          if (normed) {
            const float r = norm_factor<D, kLanes>(x, y, a.eps);
            x = make_float4(x.x * r * wa.x, x.y * r * wa.y, x.z * r * wa.z, x.w * r * wa.w);
            y = make_float4(y.x * r * wb.x, y.y * r * wb.y, y.z * r * wb.z, y.w * r * wb.w);
          }
          if (turned && u.turns) {
            auto turn = [&](float& p, float& q, int k) {
              const float p0 = p;
              p = fmaf(p0, u.c[k], -(q * u.s[k]));
              q = fmaf(q, u.c[k], p0 * u.s[k]);
            };
            if (kPairs) {
              turn(x.x, x.y, 0);
              turn(x.z, x.w, 1);
              turn(y.x, y.y, 2);
              turn(y.z, y.w, 3);
            } else {
              turn(x.x, y.x, 0);
              turn(x.y, y.y, 1);
              turn(x.z, y.z, 2);
              turn(x.w, y.w, 3);
            }
          }
          ya = make_uint2(pack(x.x, x.y), pack(x.z, x.w));
          yb = make_uint2(pack(y.x, y.y), pack(y.z, y.w));
        }
        store(h, h < heads, ya, yb);
      }
    }
  };
  auto dense = [&](void* base, int64_t stride) {
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(base) + t * stride;
    return [=](int h, bool mine, uint2 ya, uint2 yb) {
      if (!mine) return;
      *reinterpret_cast<uint2*>(dst + (int64_t)h * D + u.da) = ya;
      *reinterpret_cast<uint2*>(dst + (int64_t)h * D + u.db) = yb;
    };
  };
  auto paged = [&](void* pages, uint8_t* exps) {
    return [=](int h, bool mine, uint2 ya, uint2 yb) {
      const int64_t row = row0 + ((int64_t)h << a.rows.cache.page_shift);
      if (kTo == To::kE4M3) {
        uint32_t byte;
        const uint2 c = quantise_row<kLanes>(make_uint4(ya.x, ya.y, yb.x, yb.y), lane, &byte);
        if (!mine) return;
        uint8_t* dst = static_cast<uint8_t*>(pages) + row * D;
        *reinterpret_cast<uint32_t*>(dst + u.da) = c.x;
        *reinterpret_cast<uint32_t*>(dst + u.db) = c.y;
        if (l == 0) exps[row] = (uint8_t)byte;
      } else if (mine) {
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(pages) + row * D;
        *reinterpret_cast<uint2*>(dst + u.da) = ya;
        *reinterpret_cast<uint2*>(dst + u.db) = yb;
      }
    };
  };
  const bool q_first = q_from < q_to, k_first = !q_first && k_from < k_to;
  section(a.q, a.q_stride, a.h_q, q_from, q_to, q_first, a.q_weight, a.norm, true, dense(a.q_out, a.q_out_stride));
  if (kTo == To::kDense) {
    section(a.rows.k, a.rows.k_stride, a.h_kv, k_from, k_to, k_first, a.k_weight, a.norm, true,
            dense(a.k_out, a.k_out_stride));
  } else if (row0 >= 0) {
    section(a.rows.k, a.rows.k_stride, a.h_kv, k_from, k_to, k_first, a.k_weight, a.norm, true,
            paged(a.rows.cache.k_pages, a.rows.cache.k_exp));
    section(a.rows.v, a.rows.v_stride, a.h_kv, v_from, v_to, !q_first && !k_first, nullptr, false, false,
            paged(a.rows.cache.v_pages, a.rows.cache.v_exp));
  }
}

template <int D, bool kPairs, To kTo>
cudaError_t launch(const RopeArgs& in, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  RopeArgs a = in;
  constexpr int kHeads = 256 / D;
  const int k_groups = (a.h_kv + kHeads - 1) / kHeads;
  const int64_t all = (a.h_q + kHeads - 1) / kHeads + (kTo == To::kDense ? 1 : 2) * (int64_t)k_groups;
  // a token's rows are shared out while there are fewer warps than the GPU holds at once
  const int64_t per = a.rows.total_tokens * all / ((int64_t)sms * 32);
  a.groups = (int32_t)(per < 1 ? 1 : per > all ? all : per);
  const int64_t parts = (all + a.groups - 1) / a.groups;
  const int64_t blocks = (a.rows.total_tokens * parts + kWarps - 1) / kWarps;
  // programmatic stream serialization, as for the cache's other kernels
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kWarps * 32);
  return cudaLaunchKernelEx(&cfg, rope_kernel<D, kPairs, kTo>, a);
}

template <To kTo>
cudaError_t launch_to(const RopeArgs& a, cudaStream_t stream) {
  if (a.head_dim == 256) return a.pairs ? launch<256, true, kTo>(a, stream) : launch<256, false, kTo>(a, stream);
  return a.pairs ? launch<128, true, kTo>(a, stream) : launch<128, false, kTo>(a, stream);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeArgs& a, cudaStream_t stream) {
  if (a.rows.total_tokens == 0) return cudaSuccess;
  return launch_to<To::kDense>(a, stream);
}

cudaError_t launch_kv_append_rope(const RopeArgs& a, cudaStream_t stream) {
  if (a.rows.total_tokens == 0) return cudaSuccess;
  return a.rows.cache.dtype == kCacheE4M3 ? launch_to<To::kE4M3>(a, stream) : launch_to<To::kBF16>(a, stream);
}

}  // namespace gdn
