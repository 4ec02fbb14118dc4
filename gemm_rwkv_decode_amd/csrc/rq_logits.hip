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
// arrival) where they are few.  A workgroup takes a range of one row's tokens:
// it asks for its first logits, counts the history's tokens that fall into the
// range in LDS (integer atomics, whose order does not matter; 16 bits a token,
// so that a row of 65536 is one range), and applies all steps as the logits
// stream through.  No table of counts goes through memory, and nothing is
// sorted; the price is that every range reads the row's whole history (from L2).
// An entry of the bias list is remembered the same way, by its place, so that
// of several the last holds.  200 x 65529 with histories of 9000 to 12000: 29 us,
// 3.9 TB/s (in slices of 8192 tokens with 32-bit counts 47 us).
//
// The greatest: the values' order as an integer in the upper half, the
// complement of the token's number in the lower half, so the maximum is the
// greatest value's lowest token whatever the order of the slices.  A row's
// workgroups join through one device-scope atomic maximum and an arrival
// counter; the last one writes the token and leaves both zero.  No workgroup
// waits for another.
#include <type_traits>

#include "rq_common.h"
#include "rq_internal.h"

namespace rq {
namespace {

typedef float f4u __attribute__((ext_vector_type(4), aligned(4)));
typedef unsigned long long u64;

constexpr u32 SEEN = 0x80000000u;  // in the history at all; low bits: count generated
constexpr u32 SEEN_HALF = 0x8000u;  // the same of a 16-bit count
constexpr int MAX_HALF = 0x7FFF;

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

// Occurrences of a slice's tokens, 16 bits a token, or 32 where a row has more
// generated tokens than 15 bits hold (`big`).
__device__ __forceinline__ void count_token(u32* cnt, u32 t, bool generated, bool big) {
  const int sh = big ? 0 : 16 * (t & 1);
  const u32 seen = big ? SEEN : SEEN_HALF;
  u32* const word = cnt + (big ? t : t / 2);
  if (generated) atomicAdd(word, 1u << sh);
  else atomicOr(word, seen << sh);
}
// of the four tokens from t on
__device__ __forceinline__ u32x4 counts_of(const u32* cnt, u32 t, bool big) {
  if (big) return *reinterpret_cast<const u32x4*>(cnt + t);
  const u32x2 w = *reinterpret_cast<const u32x2*>(cnt + t / 2);
  u32x4 c;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const u32 h = (w[i / 2] >> (16 * (i & 1))) & 0xFFFFu;
    c[i] = (h & (u32)MAX_HALF) | ((h & SEEN_HALF) << 16);
  }
  return c;
}

// A workgroup takes `per` tokens of one row, in slices of `sl` tokens (half as
// many where the counts need 32 bits), and a slice in steps of 4 NT.
template <int NT, bool TOKENS>
__global__ void __launch_bounds__(NT)
k_logits(const LogitsArgs a, u64* records, int stride, int per, int sl) {
  constexpr int STEP = 4 * NT;
  extern __shared__ __attribute__((aligned(16))) u32 lds[];  // counts, then bias entries [sl]
  __shared__ u64 wave_best[NT / 64];
  u32* cnt = lds;
  u32* ent = lds + (a.history ? sl / 2 : 0);
  const int tid = threadIdx.x;
  const int m = blockIdx.y;
  const int first = blockIdx.x * per, last = min(first + per, a.V);
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
  const int own = hr.lo + min(max(given, 0), hr.hi - hr.lo);
  const bool big = hr.hi - own > MAX_HALF;
  const int span = big ? sl / 2 : sl;
  const bool masked = mid >= 0 && mid < a.nmasks;
  const u32* mrow = a.masks + (masked ? (size_t)mid * ((a.V + 31) / 32) : 0);

  f4 next;
  u32 next_word = ~0u;
  // Of the step at u0, which may pass the end of its slice and of the row: no
  // load depends on a branch, or the compiler would wait for stores with them.
  // What lies past the row's end is some other value of it.
  const auto fetch = [&](int u0) {
    if (a.V < 4) return;
    const int e = u0 + tid * 4;
    next = *reinterpret_cast<const f4u*>(x + min(e, a.V - 4));
    if (masked) next_word = mrow[min(e, a.V - 1) / 32];
  };
  int ht[AHEAD], bt[AHEAD];
  fetch(first);
  list_batch<NT>(a.history, hr.lo + tid, hr.hi, ht);
  list_batch<NT>(a.bias_ids, br.lo + tid, br.hi, bt);
  u64 top = 0;
  for (int v0 = first; v0 < last; v0 += span) {
    const int n = min(span, last - v0);
    if (a.history || a.bias_ids) {
      const int words = (a.history ? sl / 2 : 0) + (a.bias_ids ? sl : 0);
      for (int i = tid * 4; i < words; i += NT * 4)
        *reinterpret_cast<u32x4*>(lds + i) = u32x4{0, 0, 0, 0};
      __syncthreads();
      if (a.history) {
        if (v0 > first) list_batch<NT>(a.history, hr.lo + tid, hr.hi, ht);
        for_list<NT>(a.history, hr.lo, hr.hi, ht, [&](int i, int token) {
          const u32 t = (u32)token - (u32)v0;
          if (t < (u32)n) count_token(cnt, t, i >= own, big);
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
    const auto step = [&](int u0, auto whole) {
      f4 z = next;
      u32 word = next_word;
      fetch(u0 + STEP < n ? v0 + u0 + STEP : v0 + span);
      const int e = u0 + tid * 4;
      const bool all = whole() || e + 4 <= n;
      if (!whole() && e >= n) return;
      if (!all) {
#pragma unroll
        for (int c = 0; c < 3; c++)
          if (e + c < n) z[c] = x[v0 + e + c];
        if (masked) word = mrow[(v0 + e) / 32];
      }
      if (a.history) {
        const u32x4 c = counts_of(cnt, e, big);
#pragma unroll
        for (int i = 0; i < 4; i++) z[i] = apply_one(z[i], c[i], rep, freq, pres);
      }
      if (a.bias_ids) {
        const u32x4 b = *reinterpret_cast<const u32x4*>(ent + e);
#pragma unroll
        for (int i = 0; i < 4; i++)
          if (b[i]) z[i] += a.bias[b[i] - 1];
      }
#pragma unroll
      for (int i = 0; i < 4; i++)
        if (!((word >> ((v0 + e) % 32 + i)) & 1u)) z[i] = -__builtin_inff();
      if constexpr (TOKENS) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const u32 o = all || e + i < n ? order_of(z[i]) : 0u;
          const u64 key = o ? ((u64)o << 32) | (u32)~(u32)(v0 + e + i) : 0;
          top = key > top ? key : top;
        }
      }
      if (all) {
        // Past the caches where the tokens are chosen here, as nobody has to read the
        // outputs then (200 x 65529 with histories of 12000, batches in turn 32.0 ->
        // 28.5 us, 64 x 65536 13.8 -> 13.2).  Without tokens the caller reads them
        // next: with a softmax behind the call 64 x 65536 take 34.8 us through the
        // caches, 42.5 past them.
        if constexpr (TOKENS)
          __builtin_nontemporal_store((f4u)z, reinterpret_cast<f4u*>(out + v0 + e));
        else
          *reinterpret_cast<f4u*>(out + v0 + e) = (f4u)z;
      } else {
#pragma unroll
        for (int c = 0; c < 3; c++)
          if (e + c < n) out[v0 + e + c] = z[c];
      }
    };
    int u0 = 0;
    for (; u0 + STEP <= n; u0 += STEP) step(u0, std::true_type());
    if (u0 < n) step(u0, std::false_type());
    if ((a.history || a.bias_ids) && v0 + span < last) __syncthreads();  // before the clearing
  }
  if constexpr (!TOKENS) return;
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

// `workgroups` of a row, each in as few slices as its LDS allows.
constexpr size_t LOGITS_LDS = 152 << 10;
template <int NT, bool TOKENS>
hipError_t launch_slices(const LogitsArgs& a, u64* records, int stride, int workgroups,
                         hipStream_t s) {
  constexpr int STEP = 4 * NT;
  const int steps = (a.V + STEP - 1) / STEP;
  const int own = (steps + workgroups - 1) / workgroups;  // of a workgroup
  const size_t token = (a.history ? 2 : 0) + (a.bias_ids ? 4 : 0);  // bytes
  const int most = token ? (int)(LOGITS_LDS / (token * STEP)) : own;
  const int slices = (own + most - 1) / most;
  const int sl = (own + slices - 1) / slices * STEP;
  const size_t lds = token * sl;
  constexpr size_t fixed = NT / 64 * sizeof(u64);  // wave_best
  if (lds + fixed > (64 << 10)) {
    static LdsLimit limit;
    const hipError_t e = limit.raise(reinterpret_cast<const void*>(k_logits<NT, TOKENS>), LOGITS_LDS);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((k_logits<NT, TOKENS>), dim3((steps + own - 1) / own, a.M), dim3(NT), lds, s, a,
                     records, stride, own * STEP, sl);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_logits(const LogitsArgs& a, void* ws, hipStream_t s) {
  u64* records = static_cast<u64*>(ws);
  // a record per row, as far apart as the workspace allows: rows that share a
  // memory channel's line take their turns there (64 rows x 65536 in slices
  // of 1024, records 16 bytes apart 41 us, 1 KiB apart 12.4 us)
  int stride = 2 * LOGITS_MAX_M;  // in 8 bytes
  for (int m = 1; m < a.M; m *= 2) stride /= 2;
  // Workgroups of 512 threads and 2048 tokens while that makes no more than one
  // for each compute unit, or where a row has no more tokens; else 1024 threads, and
  // as many workgroups as compute units or rows, so that the history is read by few.
  // Both ways, tokens wanted: histories of 257 1 x 65536 5.9 / 6.8 us, 8 x 65536 6.3 /
  // 7.2, 16 x 65536 7.4 / 7.5, 200 x 4096 7.3 / 6.4; of 1000 64 x 65536 24 / 12, of 4000
  // 28 / 13; of 100 4000 x 2000 37 / 70.
  const int small = (a.V + 2047) / 2048;
  const bool few = (long long)a.M * small <= 256 || small == 1;
  const int workgroups = few ? small : a.M < 256 ? 256 / a.M : 1;
  if (a.tokens)
    return few ? launch_slices<512, true>(a, records, stride, workgroups, s)
               : launch_slices<1024, true>(a, records, stride, workgroups, s);
  return few ? launch_slices<512, false>(a, records, stride, workgroups, s)
             : launch_slices<1024, false>(a, records, stride, workgroups, s);
}

}  // namespace rq
