// attn_common.cuh — what the attention layers' kernels share: softmax arithmetic, e4m3
// codes as bf16, even shares of work, tensor maps.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cudaTypedefs.h>
#include <math.h>
#include <stdint.h>

#include <mutex>

#include "attn_tc.cuh"

namespace gdn {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.f;  // log2 of the largest weight before a reference moves

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float poison_of(uint32_t bits16) {  // the value if it is not finite
  return (bits16 & 0x7f80u) == 0x7f80u ? __uint_as_float(bits16 << 16) : 0.f;
}

template <int N>
__device__ __forceinline__ float largest(const float (&s)[N]) {
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = fmaxf(s[i], s[8 + i]);
#pragma unroll
  for (int k = 16; k < N; k += 16)
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = tc2::max3(x[i], s[k + i], s[k + 8 + i]);
  return tc2::max3(tc2::max3(x[0], x[1], x[2]), tc2::max3(x[3], x[4], x[5]), fmaxf(x[6], x[7]));
}
template <int N>
__device__ __forceinline__ float least(const float (&s)[N]) {
  float x = s[0];
#pragma unroll
  for (int i = 1; i < N; ++i) x = fminf(x, s[i]);
  return x;
}

// The unit of a row of V in two factors: 2^120 times the part up to 2^7 for the codes
// below (of two rows, as bf16), the rest for the weight (1 for bytes up to 134).
constexpr uint32_t kUnitTop = 134;
__device__ __forceinline__ uint32_t value_units(uint32_t byte0, uint32_t byte1) {
  return ((min(byte0, kUnitTop) + 120) << 7) | ((min(byte1, kUnitTop) + 120) << 23);
}
// An e4m3 code's sign, exponent and significand bits put where bf16 has them are 2^-120
// of its value, subnormal codes included: the magnitudes of the even and of the odd bytes
// of a word (a NaN code as 480), and two such values times their units (exact).
constexpr uint32_t kMagnitude = 0x07f007f0u, kSigns = 0x80008000u;
__device__ __forceinline__ uint32_t even_magnitudes(uint32_t codes) { return (codes << 4) & kMagnitude; }
__device__ __forceinline__ uint32_t odd_magnitudes(uint32_t codes) { return (codes >> 4) & kMagnitude; }
__device__ __forceinline__ uint32_t times(uint32_t two, uint32_t units) {
  uint32_t y;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(two), "r"(units));
  return y;
}
// of the largest magnitudes seen, by halves
__device__ __forceinline__ bool nan_code(uint32_t most) { return most >= 0x07f00000u || (most & 0xffffu) >= 0x07f0u; }
// bf16 NaN where a magnitude is that of a NaN code, else zero
__device__ __forceinline__ uint32_t nan_where(uint32_t magnitudes) {
  return __vcmpeq2(magnitudes, kMagnitude) & 0x7fc07fc0u;
}

// Division of non-negative numbers by the tokens of a tile (at least 2):
// x floor(2^32 / d + 1) / 2^32 is at most one more than x / d.
struct Divisor {
  int d;
  uint32_t inv;
  __device__ __forceinline__ explicit Divisor(int by) : d(by), inv(0xffffffffu / (uint32_t)by + 1u) {}
  __device__ __forceinline__ Divisor(int by, uint32_t inverse) : d(by), inv(inverse) {}  // (as above)
  __device__ __forceinline__ uint32_t divide(uint32_t x) const {
    const uint32_t q = __umulhi(x, inv);
    return (uint64_t)q * (uint32_t)d > x ? q - 1 : q;
  }
};

// Quotient of non-negative numbers (those of 32 bits, nearly all, take the short way).
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// The work of CTA c: the first `more` CTAs have size + 1 of it, the others size.
struct Shares {
  int64_t size, more, split;
  __device__ __forceinline__ Shares(int64_t total, int ctas) {
    size = quotient(total, ctas);
    more = total - size * ctas;
    split = more * (size + 1);
  }
  __device__ __forceinline__ int64_t start(int c) const { return c * size + min((int64_t)c, more); }
  __device__ __forceinline__ int owner(int64_t u) const {
    return u < split ? (int)quotient(u, size + 1) : (int)(more + quotient(u - split, size));
  }
};

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

// [rows][heads][D] bf16, `stride` elements between rows; boxes of 64 dimensions
// x box_heads x box_rows with the 128-byte swizzle
inline bool encode(CUtensorMap* map, const void* base, int D, int64_t heads, int64_t rows, int64_t stride,
            int box_heads, int box_rows) {
  auto enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace gdn
