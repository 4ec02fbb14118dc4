// rq_quant.hip -- rows quantized to E4M3 in blocks of 128 values with a
// power-of-two scale each:
//   s = min 2^e >= 2^-126 with |a| <= 448 s,  q = e4m3(a / s),  a = x or max(x, 0)^2.
//
// Rows are whole blocks, so the array is one list of blocks and the scales one
// list beside it.  Sixteen lanes take a block, eight values each: a maximum over
// the lanes by DPP, then exact products with 1/s and the conversion.  Eight values
// are one load of binary16 (two of binary32) and one store of 8 bytes, and sixteen
// lanes are what DPP reaches without LDS.
//
// Bound by memory: 2 or 4 bytes read and 1 written per value.  2047 x 16384 binary32
// values, squared above zero, take 29.7 us on one MI355X (168 MB: 5.6 TB/s, where a
// copy does 5.07), 4593 x 2560 binary16 ones 6.8 us (35.6 MB: 5.2), one row a launch.
#include "rq_common.h"
#include "rq_fp8.h"
#include "rq_internal.h"

namespace rq {
namespace {

constexpr int PER = 8;               // values of a lane
constexpr int LANES = 128 / PER;     // lanes of a block

template <bool HALF, bool RELU2>
__global__ void __launch_bounds__(256)
k_quant(const void* x, u32x2* q, void* scales, size_t blocks, int e8m0) {
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;  // the lane's 8 values
  const size_t block = i / LANES;
  const bool active = block < blocks;
  const size_t j = active ? i : 0;
  float a[PER];
  if constexpr (HALF) {
    const h8 h = reinterpret_cast<const h8*>(x)[j];
#pragma unroll
    for (int e = 0; e < PER; e++) a[e] = (float)h[e];
  } else {
    const f4 lo = reinterpret_cast<const f4*>(x)[2 * j], hi = reinterpret_cast<const f4*>(x)[2 * j + 1];
#pragma unroll
    for (int e = 0; e < 4; e++) a[e] = lo[e], a[e + 4] = hi[e];
  }
  if constexpr (RELU2) {
#pragma unroll
    for (int e = 0; e < PER; e++) a[e] = relu2(a[e]);
  }
  const u32 se = scale_exponent(block_amax<LANES, PER>(a));
  const float inv = pow2_bits(254 - se);
  if (!active) return;
  q[i] = u32x2{e4m3x4(a[0], a[1], a[2], a[3], inv), e4m3x4(a[4], a[5], a[6], a[7], inv)};
  if (i % LANES == 0) store_scale(scales, block, se, e8m0);
}

}  // namespace

hipError_t launch_quant(const QuantArgs& a, hipStream_t s) {
  const size_t blocks = (size_t)a.M * (a.K / 128);
  const dim3 grid((unsigned)((blocks * LANES + 255) / 256)), block(256);
  u32x2* q = static_cast<u32x2*>(a.q);
  if (a.half && a.relu2)
    hipLaunchKernelGGL((k_quant<true, true>), grid, block, 0, s, a.x, q, a.scales, blocks, a.e8m0);
  else if (a.half)
    hipLaunchKernelGGL((k_quant<true, false>), grid, block, 0, s, a.x, q, a.scales, blocks, a.e8m0);
  else if (a.relu2)
    hipLaunchKernelGGL((k_quant<false, true>), grid, block, 0, s, a.x, q, a.scales, blocks, a.e8m0);
  else
    hipLaunchKernelGGL((k_quant<false, false>), grid, block, 0, s, a.x, q, a.scales, blocks, a.e8m0);
  return hipGetLastError();
}

}  // namespace rq
