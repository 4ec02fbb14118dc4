// rq_gemm_fp8.hip -- products of block-scaled E4M3 operands:
//   y[m][n] = y_in[m][n] + sum_b xs[m][b] ws[n/128][b] sum_{k in b} x[m][k] w[n][k].
//
// Inside a block of 128 the E4M3 numbers are widened to binary16 (exact) and meet
// in the binary16 matrix instructions, whose sums are binary32; the block's sum
// then enters the binary32 total with one multiply-add by the two scales.
#include "rq_common.h"
#include "rq_fp8.h"
#include "rq_internal.h"

namespace rq {
namespace {

constexpr int NT = 8;  // 16-row tiles of w of a wave: one block of outputs

// The 16 E4M3 numbers of a 16-byte piece as two operands of 8.
__device__ __forceinline__ void widen(u32x4 v, h8 (&o)[2]) {
  union {
    h2 p[8];
    h8 o[2];
  } u;
#pragma unroll
  for (int i = 0; i < 4; i++) unpack_fp8(v[i], &u.p[2 * i]);
  o[0] = u.o[0];
  o[1] = u.o[1];
}

template <bool E8M0>
__device__ __forceinline__ float scale_value(const void* s, size_t i) {
  if constexpr (E8M0)
    return e8m0_value(static_cast<const uint8_t*>(s)[i]);
  else
    return static_cast<const float*>(s)[i];
}

// Lane l of a 16 x 16 tile holds row m = l % 16 and columns n = 4 * (l / 16) + i.
template <bool E8M0>
__global__ void __launch_bounds__(64) k_fp8(const Fp8Args a) {
  const Fp8Problem& p = a.p[blockIdx.y];
  const int lane = threadIdx.x, r = lane & 15, h = lane >> 4;
  const u32 mt = (a.M + 15) / 16, nb = blockIdx.x / mt;  // block of outputs
  const int n0 = nb * 16 * NT;
  const size_t m = (size_t)(blockIdx.x % mt) * 16 + r;
  if (n0 >= p.N) return;
  const size_t mc = min(m, (size_t)a.M - 1);  // rows past the end repeat the last one
  const int kb = p.K / 128;
  const uint8_t* xp = p.x + mc * p.K + 16 * h;
  f4 acc[NT];
#pragma unroll
  for (int t = 0; t < NT; t++) acc[t] = f4{0, 0, 0, 0};
  for (int b = 0; b < kb; b++) {
    h8 x[2][2];
#pragma unroll
    for (int q = 0; q < 2; q++)
      widen(*reinterpret_cast<const u32x4*>(xp + b * 128 + 64 * q), x[q]);
    const float s = scale_value<E8M0>(p.xs, mc * kb + b) *
                    scale_value<E8M0>(p.ws, (size_t)nb * kb + b);
#pragma unroll
    for (int t = 0; t < NT; t++) {
      const int n = min(n0 + 16 * t + r, p.N - 1);
      const uint8_t* wp = p.w + (size_t)n * p.K + 16 * h + b * 128;
      f4 d = {0, 0, 0, 0};
#pragma unroll
      for (int q = 0; q < 2; q++) {
        h8 w[2];
        widen(*reinterpret_cast<const u32x4*>(wp + 64 * q), w);
        d = __builtin_amdgcn_mfma_f32_16x16x32_f16(w[0], x[q][0], d, 0, 0, 0);
        d = __builtin_amdgcn_mfma_f32_16x16x32_f16(w[1], x[q][1], d, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < 4; i++) acc[t][i] = __builtin_fmaf(d[i], s, acc[t][i]);
    }
  }
  if (a.out == OUT_E4M3) {
    // the block's largest of a row is spread over the four lanes of the row
    float v[NT * 4];
#pragma unroll
    for (int t = 0; t < NT; t++)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const float z = (float)(_Float16)acc[t][i];
        v[4 * t + i] = a.relu2 ? relu2(z) : z;
      }
    u32 top = 0;
#pragma unroll
    for (int i = 0; i < NT * 4; i++) top = max(top, abs_bits(v[i]) < INF_BITS ? abs_bits(v[i]) : 0u);
    top = max(top, (u32)__shfl_xor((int)top, 16, 64));
    top = max(top, (u32)__shfl_xor((int)top, 32, 64));
    const u32 se = scale_exponent(top);
    const float inv = pow2_bits(254 - se);
    if (m >= (size_t)a.M) return;
#pragma unroll
    for (int t = 0; t < NT; t++)
      *reinterpret_cast<u32*>(static_cast<uint8_t*>(p.y) + m * p.N + n0 + 16 * t + 4 * h) =
          e4m3x4(v[4 * t], v[4 * t + 1], v[4 * t + 2], v[4 * t + 3], inv);
    if (h == 0) store_scale(p.ys, m * (p.N / 128) + nb, se, E8M0);
    return;
  }
  if (m >= (size_t)a.M) return;
#pragma unroll
  for (int t = 0; t < NT; t++)
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int n = n0 + 16 * t + 4 * h + i;
      if (n >= p.N) continue;
      const size_t at = m * p.N + n;
      if (a.out == OUT_F32)
        static_cast<float*>(p.y)[at] = p.y_in ? p.y_in[at] + acc[t][i] : acc[t][i];
      else
        static_cast<_Float16*>(p.y)[at] = (_Float16)acc[t][i];
    }
}

}  // namespace

size_t fp8_workspace_bytes(const Fp8Args&) { return 0; }

hipError_t launch_fp8(const Fp8Args& a, void*, hipStream_t s) {
  int n = 0;
  for (int i = 0; i < a.count; i++) n = a.p[i].N > n ? a.p[i].N : n;
  const dim3 grid((a.M + 15) / 16 * ((n + 16 * NT - 1) / (16 * NT)), a.count);
  if (a.e8m0)
    hipLaunchKernelGGL((k_fp8<true>), grid, dim3(64), 0, s, a);
  else
    hipLaunchKernelGGL((k_fp8<false>), grid, dim3(64), 0, s, a);
  return hipGetLastError();
}

}  // namespace rq
