// rq_shift.hip -- the token shift: every output row is a channel-wise mix of a
// token's row and the row before it in its sequence,
//   out[i][t] = x[t] + (prev[t] - x[t]) * mu[i],
// prev[t] = x[t-1], or the sequence's stored row for its first token; the
// stored row becomes the sequence's last row.
//
// Bound by memory: (1 + n) * T * D binary16 values moved for 3 n T D flops.
// A thread owns 8 channels (16 bytes) of TB = 2 consecutive tokens: a row of x is
// read once or twice (the second time from L2), a mix vector once per two
// tokens, however many mixes are made from them, and all of a thread's loads
// are asked for together.  The outputs stay in the caches for the products that
// read them next: stored past them, a call whose batches take turns in more memory
// than the last-level cache is faster by itself (4001 tokens of width 2560, six
// mixes, three batches in turn 25.8 against 31.6 us; one batch 25.0 against 23.8),
// but with the receptance, key and value products behind it the chain is slower
// (1308 against 1126 us; 512 tokens of width 4096 146 against 141 us), and so are
// whole layers (1000 tokens of width 2560, four layers 6.24 against 5.97 ms).
//
// Which tokens begin a sequence is found by all threads together: each looks
// at some sequences and, where one begins inside this workgroup's tokens,
// notes it in LDS.  This is one pass over the offsets and no search.  The
// thread that handles a sequence's first token reads the stored row and then
// overwrites it with the sequence's last row; nobody else touches that row.
//
// The mix is computed in binary32 and rounded once to binary16, the type the
// products of this library take.
#include "rq_common.h"
#include "rq_internal.h"

namespace rq {
namespace {

constexpr int TB = 2;           // tokens of a thread
constexpr int SHIFT_NONE = -2;  // no sequence begins at this token

union Row8 {
  u32x4 v;
  _Float16 h[8];
};

__global__ void __launch_bounds__(256)
k_shift(const ShiftArgs a) {
  __shared__ int begin_slot[TB];  // slot of the sequence that begins here, -1: none stored
  __shared__ int begin_last[TB];  // its last token
  const int tid = threadIdx.x, nthr = blockDim.x;
  const int t0 = blockIdx.x * TB;
  const int nt = min(TB, a.T - t0);
  const int c8 = blockIdx.y * nthr + tid;  // the thread's 8 channels
  const bool active = c8 * 8 < a.D;
  const size_t D = a.D;
  const _Float16* xp = a.x + (size_t)t0 * D + (size_t)c8 * 8;
  Row8 x[TB], prev, mus[SHIFT_MAX_MIXES];
  prev.v = u32x4{0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < TB; j++) {
    x[j].v = u32x4{0, 0, 0, 0};
    if (active && j < nt) x[j].v = *reinterpret_cast<const u32x4*>(xp + j * D);
  }
  if (active && t0 > 0) prev.v = *reinterpret_cast<const u32x4*>(xp - D);
#pragma unroll
  for (int i = 0; i < SHIFT_MAX_MIXES; i++)
    if (active && i < a.n)
      mus[i].v = *reinterpret_cast<const u32x4*>(a.mu + (size_t)i * D + (size_t)c8 * 8);
  if (tid < TB) begin_slot[tid] = SHIFT_NONE;
  __syncthreads();
  for (int q = tid; q < a.sequences; q += nthr) {
    const int lo = a.offsets[q], hi = a.offsets[q + 1];
    if (lo >= t0 && lo < t0 + nt && hi > lo && hi <= a.T) {
      const int slot = a.slots ? a.slots[q] : q;
      begin_slot[lo - t0] = (slot >= 0 && slot < a.nslots) ? slot : -1;
      begin_last[lo - t0] = hi - 1;
    }
  }
  __syncthreads();
  if (!active) return;
  // prev of every token, in binary32 differences
  Row8 before[TB];
#pragma unroll
  for (int j = 0; j < TB; j++) {
    before[j].v = j == 0 ? prev.v : x[j - 1].v;
    if (j < nt) {
      const int slot = begin_slot[j];
      if (slot != SHIFT_NONE) {
        before[j].v = u32x4{0, 0, 0, 0};
        if (slot >= 0) {
          u32x4* st = reinterpret_cast<u32x4*>(a.state + (size_t)slot * D + (size_t)c8 * 8);
          before[j].v = *st;
          *st = *reinterpret_cast<const u32x4*>(a.x + (size_t)begin_last[j] * D + (size_t)c8 * 8);
        }
      }
    }
  }
  const size_t plane = (size_t)a.T * D;
  _Float16* op = a.out + (size_t)t0 * D + (size_t)c8 * 8;
#pragma unroll
  for (int i = 0; i < SHIFT_MAX_MIXES; i++) {
    if (i >= a.n) break;
    const Row8 mu = mus[i];
#pragma unroll
    for (int j = 0; j < TB; j++) {
      if (j < nt) {
        Row8 o;
#pragma unroll
        for (int e = 0; e < 8; e++) {
          const float xe = (float)x[j].h[e];
          o.h[e] = (_Float16)(xe + ((float)before[j].h[e] - xe) * (float)mu.h[e]);
        }
        *reinterpret_cast<u32x4*>(op + i * plane + j * D) = o.v;
      }
    }
  }
}

}  // namespace

hipError_t launch_shift(const ShiftArgs& a, hipStream_t s) {
  // workgroups of at most 256 threads, the channels split evenly over them
  const int lanes = a.D / 8;
  const int parts = (lanes + 255) / 256;
  const int threads = ((lanes + parts - 1) / parts + 63) / 64 * 64;
  const int by = (lanes + threads - 1) / threads;
  hipLaunchKernelGGL(k_shift, dim3((a.T + TB - 1) / TB, by), dim3(threads), 0, s, a);
  return hipGetLastError();
}

}  // namespace rq
