// kv_cache.cu — rows of keys and values written into the paged cache as they
// are produced, and read back as packed bf16 rows.
//
// A cached row is one (token, KV head)'s D values.  In an e4m3 cache the row's
// unit is the power of two 2^e with e the smallest integer for which its largest
// finite |x| is at most 448 * 2^e (448 is the largest e4m3 value):
//     code_i = e4m3(x_i / 2^e), round to nearest even;   byte = e + 127
// Dividing by a power of two is exact, so the only rounding is the code's own
// (half a unit in the fourth significant bit, relative 2^-4; below 2^-6 units,
// half of 2^-9 units), and code_i * 2^e has four significant bits, so reading
// back into bf16 rounds nothing.  A non-finite x_i is stored as the NaN code.
//
// Both passes are bound by HBM (each row in once, out once).  One warp takes a
// token: it finds the token's sequence and page once for all its heads, after
// the loads of the first rows have been issued.  A lane holds 16 bytes of a bf16
// row (8 values), so a row is 32 lanes at D = 256 and 16 at D = 128.
//
// Measured, append and gather together, calls back to back: 48,262 rows of 8 e4m3
// heads of 128 in ragged batches 96 us for 595 MB = 6.2 TB/s, 91 % of a plain copy's
// rate (the append also issues in three quarters of its cycles: 13 instructions a
// value for maximum, scaling and rounding); 4,096 rows of 2 bf16 heads of 256 9 to 10 us
// (8.6 in a graph) and one row of each of 256 sequences 9 us (5.5), which is two launches.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "attn_params.h"
#include "kv_rows.cuh"
#include "params.h"
#include "rows.cuh"
#include "tc.cuh"

namespace gdn {
namespace {

constexpr int kKvWarps = 8;

__device__ __forceinline__ uint32_t two_values(uint32_t codes, float unit) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(codes & 0xffffu), __NV_E4M3);
  const float2 f = __half22float2(__half2(h));
  const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * unit, f.y * unit);
  return *reinterpret_cast<const uint32_t*>(&b);
}

template <int D, bool kFp8>
__global__ void __launch_bounds__(kKvWarps * 32) kv_append_kernel(const KvRowsArgs a) {
  constexpr int kLanes = D / 8;        // lanes per row
  constexpr int kHeads = 32 / kLanes;  // rows a warp holds at once
  tc::allow_dependents();
  tc::wait_prerequisites();
  const int lane = threadIdx.x & 31;
  const int64_t tt = (int64_t)blockIdx.x * kKvWarps + (threadIdx.x >> 5);
  if (tt >= a.total_tokens) return;
  const int t = (int)tt;
  const int part = lane % kLanes, sub = lane / kLanes;
  const uint4* ks = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.k) + t * a.k_stride);
  const uint4* vs = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.v) + t * a.v_stride);
  const int h_kv = a.cache.h_kv;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  uint4 kx = zero, vx = zero;
  if (sub < h_kv) {
    kx = __ldg(ks + lane);
    vx = __ldg(vs + lane);
  }
  const int64_t row0 = token_row(a, t, lane);
  check_packing(a, t, lane);
  if (row0 < 0) return;
  for (int j0 = 0; j0 < h_kv; j0 += kHeads) {
    const int j = j0 + sub;
    const bool mine = j < h_kv;
    uint4 kn = zero, vn = zero;  // the next heads' rows
    if (j + kHeads < h_kv) {
      kn = __ldg(ks + (j0 + kHeads) * kLanes + lane);
      vn = __ldg(vs + (j0 + kHeads) * kLanes + lane);
    }
    const int64_t row = row0 + ((int64_t)j << a.cache.page_shift);
    if (kFp8) {
      uint32_t kb, vb;
      const uint2 kc = quantise_row<kLanes>(kx, lane, &kb);
      const uint2 vc = quantise_row<kLanes>(vx, lane, &vb);
      if (mine) {
        static_cast<uint2*>(a.cache.k_pages)[row * kLanes + part] = kc;
        static_cast<uint2*>(a.cache.v_pages)[row * kLanes + part] = vc;
        if (part == 0) {
          a.cache.k_exp[row] = (uint8_t)kb;
          a.cache.v_exp[row] = (uint8_t)vb;
        }
      }
    } else if (mine) {
      static_cast<uint4*>(a.cache.k_pages)[row * kLanes + part] = kx;
      static_cast<uint4*>(a.cache.v_pages)[row * kLanes + part] = vx;
    }
    kx = kn;
    vx = vn;
  }
}

template <int D, bool kFp8>
__global__ void __launch_bounds__(kKvWarps * 32) kv_gather_kernel(const KvRowsArgs a) {
  constexpr int kLanes = D / 8;
  constexpr int kHeads = 32 / kLanes;
  tc::allow_dependents();
  tc::wait_prerequisites();
  const int lane = threadIdx.x & 31;
  const int64_t tt = (int64_t)blockIdx.x * kKvWarps + (threadIdx.x >> 5);
  if (tt >= a.total_tokens) return;
  const int t = (int)tt;
  const int part = lane % kLanes, sub = lane / kLanes;
  uint4* ks = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.k) + t * a.k_stride);
  uint4* vs = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.v) + t * a.v_stride);
  const int64_t row0 = token_row(a, t, lane);
  check_packing(a, t, lane);
#pragma unroll 4
  for (int j = sub; j < a.cache.h_kv; j += kHeads) {
    uint4 kx = make_uint4(0, 0, 0, 0), vx = kx;  // a row without a page reads as zeros
    if (row0 >= 0) {
      const int64_t row = row0 + ((int64_t)j << a.cache.page_shift);
      if (kFp8) {
        const uint2 kc = static_cast<const uint2*>(a.cache.k_pages)[row * kLanes + part];
        const uint2 vc = static_cast<const uint2*>(a.cache.v_pages)[row * kLanes + part];
        const float ku = pow2((int)a.cache.k_exp[row] - 127), vu = pow2((int)a.cache.v_exp[row] - 127);
        kx = make_uint4(two_values(kc.x, ku), two_values(kc.x >> 16, ku), two_values(kc.y, ku),
                        two_values(kc.y >> 16, ku));
        vx = make_uint4(two_values(vc.x, vu), two_values(vc.x >> 16, vu), two_values(vc.y, vu),
                        two_values(vc.y >> 16, vu));
      } else {
        kx = static_cast<const uint4*>(a.cache.k_pages)[row * kLanes + part];
        vx = static_cast<const uint4*>(a.cache.v_pages)[row * kLanes + part];
      }
    }
    ks[j * kLanes + part] = kx;
    vs[j * kLanes + part] = vx;
  }
}

template <typename Kernel>
cudaError_t launch_rows(Kernel kernel, const KvRowsArgs& a, cudaStream_t stream) {
  // programmatic stream serialization: the launch overlaps the end of the kernel
  // before it, whose results the kernel waits for before its first load
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3((unsigned)((a.total_tokens + kKvWarps - 1) / kKvWarps));
  cfg.blockDim = dim3(kKvWarps * 32);
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

cudaError_t launch_kv_append(const KvRowsArgs& a, cudaStream_t stream) {
  if (a.total_tokens == 0) return cudaSuccess;
  const bool fp8 = a.cache.dtype == kCacheE4M3;
  if (a.cache.head_dim == 256)
    return fp8 ? launch_rows(kv_append_kernel<256, true>, a, stream)
               : launch_rows(kv_append_kernel<256, false>, a, stream);
  return fp8 ? launch_rows(kv_append_kernel<128, true>, a, stream)
             : launch_rows(kv_append_kernel<128, false>, a, stream);
}

cudaError_t launch_kv_gather(const KvRowsArgs& a, cudaStream_t stream) {
  if (a.total_tokens == 0) return cudaSuccess;
  const bool fp8 = a.cache.dtype == kCacheE4M3;
  if (a.cache.head_dim == 256)
    return fp8 ? launch_rows(kv_gather_kernel<256, true>, a, stream)
               : launch_rows(kv_gather_kernel<256, false>, a, stream);
  return fp8 ? launch_rows(kv_gather_kernel<128, true>, a, stream)
             : launch_rows(kv_gather_kernel<128, false>, a, stream);
}

}  // namespace gdn
