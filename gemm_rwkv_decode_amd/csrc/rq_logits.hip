// rq_logits.hip -- penalties for repeated tokens, biases and grammar masks on
// a row of logits, and the greatest of the result.  For token i of a row, with
// c its occurrences in the generated part of the row's history and "seen" in
// any part:
//   z = x;  seen: z > 0 ? z / rep : z * rep;  z = z - freq c;  c > 0: z - pres;
//   z + bias (of the last entry of i);  not allowed by the row's mask: -inf.
// Each step is one binary32 operation, rounded on its own, in this order.
//
// Bound by the logits' traffic (8 bytes a value).  A workgroup takes a slice
// of SL tokens of one row: it issues the loads of its logits, counts the
// history's tokens that fall into the slice in LDS (integer atomics, whose
// order does not matter), and applies all steps on the way out.  No counts
// table goes through memory, and nothing is sorted; the price is that every
// slice reads the row's whole history (from L2).
//
// The greatest: the values' order as an integer in the upper half, the
// complement of the token's number in the lower half, so the maximum is the
// greatest value's lowest token whatever the order of the slices.  Slices join through one
// device-scope atomic maximum and an arrival counter per row; the last one
// writes the token and leaves both zero.  No workgroup waits for another.
#include "rq_common.h"
#include "rq_internal.h"

namespace rq {
namespace {

typedef float f4u __attribute__((ext_vector_type(4), aligned(4)));
typedef unsigned long long u64;

constexpr int THREADS = 256;
constexpr u32 SEEN = 0x80000000u;  // in the history at all; low bits: count generated

struct Range {
  int lo, hi;
};
// entries of a row's ragged list, whatever the offsets hold
__device__ __forceinline__ Range list_range(const int* off, int m, int total) {
  const int lo = min(max(off[m], 0), total);
  return Range{lo, min(max(off[m + 1], lo), total)};
}

// Position of z in the order of the values, 0 for what is never chosen (-inf
// and NaN); -0 counts as +0.
__device__ __forceinline__ u32 order_of(float z) {
  if (!(z > -__builtin_inff())) return 0;
  const u32 b = __builtin_bit_cast(u32, z + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// Contraction is off: freq * n and the subtraction round on their own.
__device__ __forceinline__ float apply_one(float z, u32 c, float rep, float freq, float pres) {
#pragma clang fp contract(off)
  if (c == 0) return z;
  z = z > 0.0f ? z / rep : z * rep;
  const u32 n = c & ~SEEN;
  z = z - freq * (float)n;
  return n ? z - pres : z;
}

template <int SL>
__global__ void __launch_bounds__(THREADS)
k_logits(const LogitsArgs a, u64* best, u32* arrived) {
  extern __shared__ u32 lds[];  // counts [SL], then the bias entries [SL]
  __shared__ u64 wave_best[THREADS / 64];
  constexpr int Q = SL / (4 * THREADS);
  u32* cnt = lds;
  u32* ent = lds + (a.history ? SL : 0);
  const int tid = threadIdx.x;
  const int m = blockIdx.y;
  const int v0 = blockIdx.x * SL;
  const int n = min(SL, a.V - v0);  // tokens of this slice
  const float* x = a.logits + (size_t)m * a.V + v0;
  float* out = a.out + (size_t)m * a.V + v0;
  const int mid = a.masks ? a.mask_ids[m] : -1;
  const bool masked = mid >= 0 && mid < a.nmasks;
  const u32* mrow = a.masks + (masked ? (size_t)mid * ((a.V + 31) / 32) + v0 / 32 : 0);

  f4 z[Q];
  u32 word[Q];
#pragma unroll
  for (int q = 0; q < Q; q++) {
    const int e = (q * THREADS + tid) * 4;
    z[q] = f4{0, 0, 0, 0};
    word[q] = ~0u;
    if (e + 4 <= n) {
      z[q] = *reinterpret_cast<const f4u*>(x + e);
    } else {
#pragma unroll
      for (int c = 0; c < 3; c++)
        if (e + c < n) z[q][c] = x[e + c];
    }
    if (masked && e < n) word[q] = mrow[e / 32] >> (e % 32);
  }

  if (a.history || a.bias_ids) {
    const int words = (a.history ? SL : 0) + (a.bias_ids ? SL : 0);
    for (int i = tid * 4; i < words; i += THREADS * 4)
      *reinterpret_cast<u32x4*>(lds + i) = u32x4{0, 0, 0, 0};
    __syncthreads();
    if (a.history) {
      const Range r = list_range(a.history_offsets, m, a.history_len);
      const int own = r.lo + (a.prompt ? max(a.prompt[m], 0) : 0);
      for (int i = r.lo + tid; i < r.hi; i += THREADS) {
        const u32 t = (u32)a.history[i] - (u32)v0;
        if (t < (u32)n) {
          if (i < own) atomicOr(&cnt[t], SEEN);
          else atomicAdd(&cnt[t], 1u);
        }
      }
    }
    if (a.bias_ids) {
      const Range r = list_range(a.bias_offsets, m, a.bias_len);
      for (int i = r.lo + tid; i < r.hi; i += THREADS) {
        const u32 t = (u32)a.bias_ids[i] - (u32)v0;
        if (t < (u32)n) atomicMax(&ent[t], (u32)i + 1u);
      }
    }
    __syncthreads();
  }

  const float rep = a.repetition ? a.repetition[m] : 1.0f;
  const float freq = a.frequency ? a.frequency[m] : 0.0f;
  const float pres = a.presence ? a.presence[m] : 0.0f;
  u64 top = 0;
#pragma unroll
  for (int q = 0; q < Q; q++) {
    const int e = (q * THREADS + tid) * 4;
    if (a.history) {
      const u32x4 c = *reinterpret_cast<const u32x4*>(cnt + e);
#pragma unroll
      for (int i = 0; i < 4; i++) z[q][i] = apply_one(z[q][i], c[i], rep, freq, pres);
    }
    if (a.bias_ids) {
      const u32x4 b = *reinterpret_cast<const u32x4*>(ent + e);
#pragma unroll
      for (int i = 0; i < 4; i++)
        if (b[i]) z[q][i] += a.bias[b[i] - 1];
    }
#pragma unroll
    for (int i = 0; i < 4; i++)
      if (!((word[q] >> i) & 1u)) z[q][i] = -__builtin_inff();
    if (e + 4 <= n) {
      *reinterpret_cast<f4u*>(out + e) = z[q];
    } else {
#pragma unroll
      for (int c = 0; c < 3; c++)
        if (e + c < n) out[e + c] = z[q][c];
    }
    if (a.tokens) {
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const u32 o = e + i < n ? order_of(z[q][i]) : 0u;
        const u64 key = o ? ((u64)o << 32) | (u32)~(u32)(v0 + e + i) : 0;
        top = key > top ? key : top;
      }
    }
  }
  if (!a.tokens) return;

#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const u64 o = __shfl_xor(top, d, 64);
    top = o > top ? o : top;
  }
  if ((tid & 63) == 0) wave_best[tid >> 6] = top;
  __syncthreads();
  if (tid != 0) return;
#pragma unroll
  for (int w = 1; w < THREADS / 64; w++) top = wave_best[w] > top ? wave_best[w] : top;
  if (gridDim.x > 1) {
    __hip_atomic_fetch_max(&best[m], top, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    // the maximum has been taken before the arrival is counted
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_waitcnt(0);
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    const u32 before =
        __hip_atomic_fetch_add(&arrived[m], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (before != gridDim.x - 1) return;
    top = __hip_atomic_exchange(&best[m], (u64)0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __hip_atomic_store(&arrived[m], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  a.tokens[m] = top ? (int)~(u32)top : -1;
}

constexpr int SLICE = 4096;

}  // namespace

int logits_slices(int V) { return (V + SLICE - 1) / SLICE; }

hipError_t launch_logits(const LogitsArgs& a, void* ws, hipStream_t s) {
  u64* best = static_cast<u64*>(ws);
  u32* arrived = reinterpret_cast<u32*>(best + LOGITS_MAX_M);
  const size_t lds = ((a.history ? SLICE : 0) + (a.bias_ids ? SLICE : 0)) * sizeof(u32);
  hipLaunchKernelGGL(k_logits<SLICE>, dim3(logits_slices(a.V), a.M), dim3(THREADS), lds, s, a,
                     best, arrived);
  return hipGetLastError();
}

}  // namespace rq
