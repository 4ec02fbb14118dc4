// rq_groupnorm.hip -- the norm between the state recurrence and the output
// projection: per token and group (head) of G channels
//   z = (y - mean) / sqrt(mean((y - mean)^2) + eps) * weight + bias + sum(r k r_k) v,
//   out = z * act(gate).
//
// A lane holds four channels, so a group is G/4 lanes and all of its sums stay in
// a wave (DPP).  y is read once: the variance is that of the centred values in
// registers, which a group far from zero needs (E[y^2] - E[y]^2 in binary32 loses
// it).  Tokens lie one after another over the lanes, so no width leaves lanes empty.
// E4M3 outputs are those of the binary16 value, whose block of 128 is 32 lanes.
//
// Bound by memory: up to five arrays read and one written.  4001 tokens of 64 heads
// of 64 with bonus and gate, binary32, to E4M3: 60.5 us on one MI355X (344 MB: 5.7
// TB/s, where a copy does 5.07), one token a launch.
#include "rq_common.h"
#include "rq_fp8.h"
#include "rq_internal.h"

namespace rq {
namespace {

__device__ __forceinline__ f4 load4(const float* p, size_t i) {
  return *reinterpret_cast<const f4*>(p + i);
}
template <bool HALF>
__device__ __forceinline__ f4 load4(const void* p, size_t i) {
  if constexpr (HALF) {
    const h4 h = *reinterpret_cast<const h4*>(static_cast<const _Float16*>(p) + i);
    return f4{(float)h[0], (float)h[1], (float)h[2], (float)h[3]};
  } else {
    return load4(static_cast<const float*>(p), i);
  }
}

// g / (1 + e^-g) from e^-|g|, which does not overflow: e^-g would be infinite, and
// the result zero, from -89 down, where the result is a normal number still.
__device__ __forceinline__ float silu(float g) {
  const float e = expf(-fabsf(g));
  return (g < 0.0f ? g * e : g) / (1.0f + e);
}

template <int LPR, bool HALF>
__global__ void __launch_bounds__(256)
k_groupnorm(const GroupnormArgs a) {
  // the lane's four channels; lanes without any are whole groups and blocks
  const size_t i = (((size_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x) * 4;
  if (i >= (size_t)a.T * a.C) return;
  const int c = (u32)(i / 4) % (u32)(a.C / 4) * 4;
  constexpr float inv_g = 1.0f / (4 * LPR);
  f4 y = load4(a.y, i);
  f4 z = {0, 0, 0, 0};
  const float mean = group_sum<LPR>(y[0] + y[1] + y[2] + y[3]) * inv_g;
  float sq = 0.0f;
#pragma unroll
  for (int e = 0; e < 4; e++) y[e] -= mean, sq += y[e] * y[e];
  const float rstd = 1.0f / sqrtf(group_sum<LPR>(sq) * inv_g + a.eps);
  const f4 one = {1, 1, 1, 1};
  const f4 w = a.weight ? load4(a.weight, c) : one;
  const f4 b = a.bias ? load4(a.bias, c) : z;
#pragma unroll
  for (int e = 0; e < 4; e++) z[e] = y[e] * rstd * w[e] + b[e];
  if (a.r) {
    const f4 r = load4<HALF>(a.r, i), k = load4<HALF>(a.k, i), rk = load4(a.r_k, c);
    const f4 v = load4<HALF>(a.v, i);
    const float dot =
        group_sum<LPR>(r[0] * k[0] * rk[0] + r[1] * k[1] * rk[1] + r[2] * k[2] * rk[2] +
                       r[3] * k[3] * rk[3]);
#pragma unroll
    for (int e = 0; e < 4; e++) z[e] += dot * v[e];
  }
  if (a.gate) {
    const f4 g = load4<HALF>(a.gate, i);
#pragma unroll
    for (int e = 0; e < 4; e++) z[e] *= a.silu ? silu(g[e]) : g[e];
  }
  if (a.out_type == 0) {
    *reinterpret_cast<f4*>(static_cast<float*>(a.out) + i) = z;
    return;
  }
  const h4 h = {(_Float16)z[0], (_Float16)z[1], (_Float16)z[2], (_Float16)z[3]};
  if (a.out_type == 1) {
    *reinterpret_cast<h4*>(static_cast<_Float16*>(a.out) + i) = h;
    return;
  }
  // the binary16 output's block of 128: 32 lanes
  const float q[4] = {(float)h[0], (float)h[1], (float)h[2], (float)h[3]};
  const u32 se = scale_exponent(block_amax<32, 4>(q));
  reinterpret_cast<u32*>(a.out)[i / 4] = e4m3x4(q[0], q[1], q[2], q[3], pow2_bits(254 - se));
  if (c % 128 == 0) store_scale(a.out_scales, i / 128, se, a.e8m0);
}

template <int LPR>
void launch_lpr(const GroupnormArgs& a, hipStream_t s) {
  // a launch has fewer than 2^32 work-items along an axis, so the largest calls take
  // a second one
  const size_t n = ((size_t)a.T * (a.C / 4) + 255) / 256, rows = n > 1 << 23 ? 2 : 1;
  const dim3 grid((unsigned)((n + rows - 1) / rows), (unsigned)rows);
  if (a.half)
    hipLaunchKernelGGL((k_groupnorm<LPR, true>), grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((k_groupnorm<LPR, false>), grid, dim3(256), 0, s, a);
}

}  // namespace

hipError_t launch_groupnorm(const GroupnormArgs& a, hipStream_t s) {
  switch (a.C / a.groups) {
    case 32: launch_lpr<8>(a, s); break;
    case 64: launch_lpr<16>(a, s); break;
    case 128: launch_lpr<32>(a, s); break;
    default: launch_lpr<64>(a, s); break;
  }
  return hipGetLastError();
}

}  // namespace rq
