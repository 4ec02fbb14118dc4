// rq_wkv.hip -- the RWKV-7 state recurrence.  Per head, with S[i][j] (value
// row i, key column j, 64 x 64, binary32) and per token
//   d_j = exp(-e^{-1/2} sigmoid(w_j)),
//   S <- S diag(d) - (S kappa) (eta o kappa)^T + v k^T,   y = S r.
#include "rq_common.h"
#include "rq_internal.h"

namespace rq {
namespace {

constexpr int HD = WKV_HEAD;

// exp(-e^{-1/2} sigmoid(w)) = 2^{-C / (1 + 2^{-w log2 e})}, C = e^{-1/2} log2 e:
// two v_exp_f32 and a v_rcp_f32, each within one unit in the last place.  The
// error of the inner exponential is damped by sigmoid's slope, so the decay,
// which lies in [0.545, 1], stays within about two units.
__device__ __forceinline__ float decay_of(float w) {
  const float e = __builtin_amdgcn_exp2f(w * -1.44269504088896341f);
  return __builtin_amdgcn_exp2f(-0.87503877f * __builtin_amdgcn_rcpf(1.0f + e));
}

template <typename T>
__device__ __forceinline__ f4 load4(const T* p) {
  if constexpr (sizeof(T) == 4) {
    return *reinterpret_cast<const f4*>(p);
  } else {
    const h4 h = *reinterpret_cast<const h4*>(p);
    return f4{(float)h.x, (float)h.y, (float)h.z, (float)h.w};
  }
}

// One token after another.  A wave holds 16 rows of S, four at a time across
// its lanes: lane l has columns 4 (l mod 16) .. + 3 of rows 4 q + l / 16,
// q = 0..3, so a state row is one coalesced 256-byte access and the sums over
// a row stay inside 16 lanes (four DPP steps).
//
// Bound by the state's traffic where sequences are single tokens (32 KiB per
// head and token against 36864 flops), by the latency of the two row sums
// where they are long.
template <typename T>
__global__ void __launch_bounds__(256)
k_wkv_seq(const WkvArgs a) {
  const int q = blockIdx.x, h = blockIdx.y;
  const int lo = max(a.offsets[q], 0), hi = min(a.offsets[q + 1], a.T);
  if (lo >= hi) return;
  const int slot = a.slots ? a.slots[q] : q;
  const bool stored = slot >= 0 && slot < a.nslots;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = 4 * (lane & 15);
  const int row0 = 16 * wave + (lane >> 4);
  float* st = a.state + ((size_t)(stored ? slot : 0) * a.H + h) * HD * HD;
  f4 S[4];
#pragma unroll
  for (int p = 0; p < 4; p++) {
    S[p] = f4{0, 0, 0, 0};
    if (stored) S[p] = *reinterpret_cast<const f4*>(st + (row0 + 4 * p) * HD + col);
  }
  const size_t ld = (size_t)a.H * HD;
  const size_t base = (size_t)h * HD;
  for (int t = lo; t < hi; t++) {
    const size_t at = (size_t)t * ld + base;
    const f4 w = load4(static_cast<const T*>(a.w) + at + col);
    const f4 k = load4(static_cast<const T*>(a.k) + at + col);
    const f4 kap = load4(static_cast<const T*>(a.kappa) + at + col);
    const f4 eta = load4(static_cast<const T*>(a.eta) + at + col);
    const f4 r = load4(static_cast<const T*>(a.r) + at + col);
    float v[4];
#pragma unroll
    for (int p = 0; p < 4; p++) v[p] = (float)static_cast<const T*>(a.v)[at + row0 + 4 * p];
    f4 d, ek;
#pragma unroll
    for (int c = 0; c < 4; c++) {
      d[c] = decay_of(w[c]);
      ek[c] = eta[c] * kap[c];
    }
    float y[4];
#pragma unroll
    for (int p = 0; p < 4; p++) {
      float sk = 0.0f;
#pragma unroll
      for (int c = 0; c < 4; c++) sk += S[p][c] * kap[c];
      sk = group_sum<16>(sk);
      float o = 0.0f;
#pragma unroll
      for (int c = 0; c < 4; c++) {
        S[p][c] = S[p][c] * d[c] - sk * ek[c] + v[p] * k[c];
        o += S[p][c] * r[c];
      }
      y[p] = group_sum<16>(o);
    }
    if ((lane & 15) == 0) {
#pragma unroll
      for (int p = 0; p < 4; p++) a.y[at + row0 + 4 * p] = y[p];
    }
  }
  if (stored) {
#pragma unroll
    for (int p = 0; p < 4; p++) *reinterpret_cast<f4*>(st + (row0 + 4 * p) * HD + col) = S[p];
  }
}

}  // namespace

hipError_t launch_wkv(const WkvArgs& a, hipStream_t s) {
  const dim3 grid(a.sequences, a.H);
  if (a.half)
    hipLaunchKernelGGL((k_wkv_seq<_Float16>), grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((k_wkv_seq<float>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace rq
