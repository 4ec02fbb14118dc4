// rq_logits.hip -- penalties for repeated tokens, biases and grammar masks on
// a row of logits, and the greatest of the result.  For token i of a row, with
// c its occurrences in the generated part of the row's history and "seen" in
// any part:
//   z = x;  seen: z > 0 ? z / rep : z * rep;  z = z - freq c;  c > 0: z - pres;
//   z + bias (of the last entry of i);  not allowed by the row's mask: -inf.
// Each step is one binary32 operation, rounded on its own, in this order.
//
// Bound by the logits' traffic (8 bytes a value) where rows are many, by the
// chain of dependent loads and atomics (offsets, history, logits, maximum,
// arrival) where they are few.  A workgroup takes slices of one row: it issues
// the loads of a slice's logits, counts the history's tokens that fall into
// the slice in LDS (integer atomics, whose order does not matter), and applies
// all steps on the way out.  No table of counts goes through memory, and nothing
// is sorted; the price is that every slice reads the row's whole history (from
// L2).  An entry of the bias list is remembered the same way, by its place, so
// that of several the last holds.
//
// The greatest: the values' order as an integer in the upper half, the
// complement of the token's number in the lower half, so the maximum is the
// greatest value's lowest token whatever the order of the slices.  A row's
// workgroups join through one device-scope atomic maximum and an arrival
// counter; the last one writes the token and leaves both zero.  No workgroup
// waits for another.
#include "rq_common.h"
#include "rq_internal.h"

namespace rq {
namespace {

typedef float f4u __attribute__((ext_vector_type(4), aligned(4)));
typedef unsigned long long u64;

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

// f(place, token) for the entries of a list, dealt out over the threads, AHEAD
// loads in flight per thread.  t holds the thread's first batch, which the
// caller loads (list_batch) before anything else; -1 past the end.
constexpr int AHEAD = 8;
template <int NT>
__device__ __forceinline__ void list_batch(const int* list, int i, int hi, int* t) {
  if (i - (int)threadIdx.x + AHEAD * NT <= hi) {  // the same for all threads
#pragma unroll
    for (int k = 0; k < AHEAD; k++) t[k] = list[i + k * NT];
  } else {
#pragma unroll
    for (int k = 0; k < AHEAD; k++) {
      t[k] = -1;
      if (i + k * NT < hi) t[k] = list[i + k * NT];
    }
  }
}
template <int NT, typename F>
__device__ __forceinline__ void for_list(const int* list, int lo, int hi, int* t, F f) {
  for (int i0 = lo; i0 < hi; i0 += AHEAD * NT) {
    const int i = i0 + (int)threadIdx.x;
    int now[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; k++) now[k] = t[k];
    if (i0 + AHEAD * NT < hi) list_batch<NT>(list, i + AHEAD * NT, hi, t);
#pragma unroll
    for (int k = 0; k < AHEAD; k++) f(i + k * NT, now[k]);
  }
}

// A workgroup takes `per` slices of 4 Q NT tokens of one row, one after another.
template <int NT, int Q>
__global__ void __launch_bounds__(NT)
k_logits(const LogitsArgs a, u64* records, int stride, int per) {
  constexpr int SL = 4 * NT * Q;
  extern __shared__ u32 lds[];  // counts [SL], then the bias entries [SL]
  __shared__ u64 wave_best[NT / 64];
  u32* cnt = lds;
  u32* ent = lds + (a.history ? SL : 0);
  const int tid = threadIdx.x;
  const int m = blockIdx.y;
  const int first = blockIdx.x * per * SL, last = min(first + per * SL, a.V);
  const float* x = a.logits + (size_t)m * a.V;
  float* out = a.out + (size_t)m * a.V;
  // what the loads below wait for, asked for together
  const int mid = a.masks ? a.mask_ids[m] : -1;
  const Range hr = a.history ? list_range(a.history_offsets, m, a.history_len) : Range{0, 0};
  const Range br = a.bias_ids ? list_range(a.bias_offsets, m, a.bias_len) : Range{0, 0};
  const int given = a.history && a.prompt ? a.prompt[m] : 0;
  const float rep = a.repetition ? a.repetition[m] : 1.0f;
  const float freq = a.frequency ? a.frequency[m] : 0.0f;
  const float pres = a.presence ? a.presence[m] : 0.0f;
  const int own = hr.lo + max(given, 0);
  const bool masked = mid >= 0 && mid < a.nmasks;
  const u32* mrow = a.masks + (masked ? (size_t)mid * ((a.V + 31) / 32) : 0);

  f4 next[Q];
  u32 next_word[Q];
  const auto fetch = [&](int v0) {
#pragma unroll
    for (int q = 0; q < Q; q++) {
      const int e = v0 + (q * NT + tid) * 4;
      next[q] = f4{0, 0, 0, 0};
      next_word[q] = ~0u;
      if (e + 4 <= last) {
        next[q] = *reinterpret_cast<const f4u*>(x + e);
      } else {
#pragma unroll
        for (int c = 0; c < 3; c++)
          if (e + c < last) next[q][c] = x[e + c];
      }
      if (masked && e < last) next_word[q] = mrow[e / 32];
    }
  };
  int ht[AHEAD], bt[AHEAD];
  fetch(first);
  list_batch<NT>(a.history, hr.lo + tid, hr.hi, ht);
  list_batch<NT>(a.bias_ids, br.lo + tid, br.hi, bt);
  u64 top = 0;
  for (int v0 = first; v0 < last; v0 += SL) {
    const int n = min(SL, last - v0);
    if (a.history || a.bias_ids) {
      const int words = (a.history ? SL : 0) + (a.bias_ids ? SL : 0);
      for (int i = tid * 4; i < words; i += NT * 4)
        *reinterpret_cast<u32x4*>(lds + i) = u32x4{0, 0, 0, 0};
      __syncthreads();
      if (a.history) {
        if (v0 > first) list_batch<NT>(a.history, hr.lo + tid, hr.hi, ht);
        for_list<NT>(a.history, hr.lo, hr.hi, ht, [&](int i, int token) {
          const u32 t = (u32)token - (u32)v0;
          if (t < (u32)n) {
            if (i < own) atomicOr(&cnt[t], SEEN);
            else atomicAdd(&cnt[t], 1u);
          }
        });
      }
      if (a.bias_ids) {
        if (v0 > first) list_batch<NT>(a.bias_ids, br.lo + tid, br.hi, bt);
        for_list<NT>(a.bias_ids, br.lo, br.hi, bt, [&](int i, int token) {
          const u32 t = (u32)token - (u32)v0;
          if (t < (u32)n) atomicMax(&ent[t], (u32)i + 1u);
        });
      }
      __syncthreads();
    }
    f4 z[Q];
    u32 word[Q];
#pragma unroll
    for (int q = 0; q < Q; q++) {
      z[q] = next[q];
      word[q] = next_word[q];
    }
    if (v0 + SL < last) fetch(v0 + SL);
#pragma unroll
    for (int q = 0; q < Q; q++) {
      const int e = (q * NT + tid) * 4;
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
        if (!((word[q] >> (e % 32 + i)) & 1u)) z[q][i] = -__builtin_inff();
      if (a.tokens) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const u32 o = e + i < n ? order_of(z[q][i]) : 0u;
          const u64 key = o ? ((u64)o << 32) | (u32)~(u32)(v0 + e + i) : 0;
          top = key > top ? key : top;
        }
      }
      if (e + 4 <= n) {
        *reinterpret_cast<f4u*>(out + v0 + e) = z[q];
      } else {
#pragma unroll
        for (int c = 0; c < 3; c++)
          if (e + c < n) out[v0 + e + c] = z[q][c];
      }
    }
    if ((a.history || a.bias_ids) && v0 + SL < last) __syncthreads();  // before the next clearing
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
  for (int w = 1; w < NT / 64; w++) top = wave_best[w] > top ? wave_best[w] : top;
  if (gridDim.x > 1) {
    u64* const best = records + (size_t)m * stride;
    u32* const arrived = reinterpret_cast<u32*>(best + 1);
    __hip_atomic_fetch_max(best, top, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    // the maximum has been taken before the arrival is counted
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_waitcnt(0);
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    const u32 before =
        __hip_atomic_fetch_add(arrived, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (before != gridDim.x - 1) return;
    top = __hip_atomic_exchange(best, (u64)0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __hip_atomic_store(arrived, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  a.tokens[m] = top ? (int)~(u32)top : -1;
}

template <int NT, int Q>
void launch_slices(const LogitsArgs& a, u64* records, int stride, int per, hipStream_t s) {
  constexpr int SL = 4 * NT * Q;
  const size_t lds = ((a.history ? SL : 0) + (a.bias_ids ? SL : 0)) * sizeof(u32);
  hipLaunchKernelGGL((k_logits<NT, Q>), dim3((a.V + per * SL - 1) / (per * SL), a.M), dim3(NT), lds,
                     s, a, records, stride, per);
}

}  // namespace

hipError_t launch_logits(const LogitsArgs& a, void* ws, hipStream_t s) {
  u64* records = static_cast<u64*>(ws);
  // a record per row, as far apart as the workspace allows: rows that share a
  // memory channel's line take their turns there (64 rows x 65536 in slices
  // of 1024, records 16 bytes apart 41 us, 1 KiB apart 12.4 us)
  int stride = 2 * LOGITS_MAX_M;  // in 8 bytes
  for (int m = 1; m < a.M; m *= 2) stride /= 2;
  // Up to 2^20 values: slices of 2048, a workgroup each, for the most
  // workgroups (1 x 65536 5.3 us, slices of 8192 7.0 us; 16 x 65536 7.9 and
  // 9.1 us).  Above: slices of 8192, so that the history is read by fewer of
  // them, and one workgroup per CU that takes several with the next slice's
  // loads in flight (64 x 65536 with histories of 1000 14.2 us, slices of 2048
  // 23 us; 200 x 65529 with histories of 12000 45.6 and 86 us).
  if ((long long)a.M * a.V <= 1 << 20) {
    launch_slices<512, 1>(a, records, stride, 1, s);
  } else {
    const int slices = (a.V + 8191) / 8192, workgroups = a.M < 256 ? 256 / a.M : 1;  // of a row
    launch_slices<1024, 2>(a, records, stride, (slices + workgroups - 1) / workgroups, s);
  }
  return hipGetLastError();
}

}  // namespace rq
