// rq_fp8.h -- device helpers of the block-scaled FP8 kernels: scales, and a
// block of 128 values quantized by the lanes that hold it.
#pragma once

#include "rq_common.h"

namespace rq {

// The value of an E8M0 scale: 2^(b - 127), NaN for 255.
__device__ __forceinline__ float e8m0_value(u32 b) {
  const u32 bits = b == 0 ? 0x00400000u : (b == 255 ? 0x7FC00000u : b << 23);
  return __builtin_bit_cast(float, bits);
}

// Largest over the LPR consecutive lanes of a group (a power of two <= 64).
template <int CTRL>
__device__ __forceinline__ u32 dpp_mov_u32(u32 v) {
  return (u32)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}
template <int LPR>
__device__ __forceinline__ u32 group_max(u32 v) {
  if constexpr (LPR >= 2) v = max(v, dpp_mov_u32<0xB1>(v));   // lane ^ 1
  if constexpr (LPR >= 4) v = max(v, dpp_mov_u32<0x4E>(v));   // lane ^ 2
  if constexpr (LPR >= 8) v = max(v, dpp_mov_u32<0x141>(v));  // i <-> 7 - i
  if constexpr (LPR >= 16) v = max(v, dpp_mov_u32<0x140>(v)); // i <-> 15 - i
  if constexpr (LPR >= 32) v = max(v, (u32)__shfl_xor((int)v, 16, 64));
  if constexpr (LPR >= 64) v = max(v, (u32)__shfl_xor((int)v, 32, 64));
  return v;
}

__device__ __forceinline__ u32 abs_bits(float v) {
  return __builtin_bit_cast(u32, v) & 0x7FFFFFFFu;
}
constexpr u32 INF_BITS = 0x7F800000u;

// Biased exponent of the smallest power of two s >= 2^-126 with a <= 448 s, from
// the bits of a finite a >= 0: 448 = 1.75 * 2^8, and adding what lies between
// 1.75 and 2 carries into the exponent exactly where the fraction is above 1.75.
__device__ __forceinline__ u32 scale_exponent(u32 a) {
  return (u32)max(1, (int)((a + 0x001FFFFFu) >> 23) - 8);
}
__device__ __forceinline__ float pow2_bits(u32 biased) {
  return __builtin_bit_cast(float, biased << 23);
}

// Four values times 1/s (a power of two: exact) as E4M3, to the nearest, ties to
// even; what is not finite becomes NaN.
__device__ __forceinline__ u32 e4m3x4(float a, float b, float c, float d, float inv) {
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, 0, false);
  return (u32)__builtin_amdgcn_cvt_pk_fp8_f32(c * inv, d * inv, r, true);
}

// The largest finite |v| (as bits) of a group of LPR lanes with N values each.
// What is not finite is rare, so one branch looks for it.
template <int LPR, int N>
__device__ __forceinline__ u32 block_amax(const float* v) {
  u32 a = 0;
#pragma unroll
  for (int i = 0; i < N; i++) a = max(a, abs_bits(v[i]));
  a = group_max<LPR>(a);
  if (__builtin_expect(__any(a >= INF_BITS), 0)) {
    u32 f = 0;
#pragma unroll
    for (int i = 0; i < N; i++) f = max(f, abs_bits(v[i]) < INF_BITS ? abs_bits(v[i]) : 0u);
    a = group_max<LPR>(f);
  }
  return a;
}

// max(z, 0)^2; NaN stays NaN
__device__ __forceinline__ float relu2(float z) {
  const float a = z < 0.0f ? 0.0f : z;
  return a * a;
}

// Stores the scale of a biased exponent as scale i.
__device__ __forceinline__ void store_scale(void* scales, size_t i, u32 biased, bool e8m0) {
  if (e8m0)
    reinterpret_cast<uint8_t*>(scales)[i] = (uint8_t)biased;
  else
    reinterpret_cast<float*>(scales)[i] = pow2_bits(biased);
}

}  // namespace rq
