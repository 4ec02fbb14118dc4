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
  const int q = blockIdx.x / a.H, h = blockIdx.x % a.H;
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

// ---------------------------------------------------------------------------
// Sixteen tokens at a time.  With P_t = d_1 ... d_t (per key column, from the
// chunk's start) and S0 the state before the chunk, the recurrence is
//   u_t  = S0 (kappa_t o P_{t-1}) + sum_{s<t} (Mb[t][s] u_s + Mk[t][s] v_s)
//   y_t  = S0 (r_t o P_t)         + sum_{s<=t} (Nb[t][s] u_s + Nk[t][s] v_s)
//   S16  = S0 diag(P_16) + sum_s (u_s bc_s^T + v_s kc_s^T)
// where u_t = S_{t-1} kappa_t, and with b_s = -(eta o kappa)_s / P_s, k^_s = k_s / P_s
//   Mb[t][s] = (kappa_t o P_{t-1}) . b_s    Mk[t][s] = (kappa_t o P_{t-1}) . k^_s
//   Nb[t][s] = (r_t o P_t) . b_s            Nk[t][s] = (r_t o P_t) . k^_s
//   bc_s = b_s o P_16,  kc_s = k^_s o P_16.
// Mb is strictly lower triangular, so U = X (S0 part + Mk V), X = (I - Mb)^-1.
// Everything is a product of small matrices on the binary32 matrix cores
// (v_mfma_f32_16x16x4_f32): 80 of them per chunk and 16 state rows where the
// token loop needs 36 vector instructions, and one dependent pass per 16
// tokens.  Every decay is at least 0.545, so 1 / P stays below 2^14 and
// nothing is lost to the factoring; a chunk is 16 tokens for that reason and
// because it is the matrix instruction's tile.
//
// The contraction order is free, so operands are laid out for the accumulator:
// a lane's accumulator f4 covers rows 4 (l / 16) .. + 3 of column l mod 16, and
// as a right operand of four MFMAs it is the contraction index 4 (l / 16) + v.
// The state S^T [keys][values], U and V are therefore used as they come, with
// no exchange between lanes, and the state never leaves its registers.
//
// A workgroup has NR state waves, 16 value rows each, and three producer waves
// that prepare what depends on the inputs alone (decays, the four 16x16
// matrices, the triangular inverse), one chunk each, in three segments one
// barrier apart; chunk c's operands go through LDS, two buffers in turn.
// ---------------------------------------------------------------------------
constexpr int CH = 16;      // tokens of a chunk
constexpr int LDR = 68;     // floats between rows of a [16][64] operand (bank order)
constexpr int LDT = 20;     // floats between rows of a [64][16] or [16][16] operand
constexpr int PRODUCERS = 3;

// What a chunk's state waves read.  With one state wave per workgroup the
// producers also make the products with V, which leaves the state wave with
// what depends on the state.
template <int NR>
struct alignas(16) ChunkOps {
  float ah[CH * LDR];   // kappa_t o P_{t-1}
  float rh[CH * LDR];   // r_t o P_t
  float bcT[HD * LDT];  // [key][token]
  float x[CH * LDT];    // (I - Mb)^-1
  float nb[CH * LDT];
  float pc[HD];         // P_16
  // NR > 1: kcT and the matrices that multiply V; NR = 1: the products
  // themselves, as accumulators [j][lane] of kc^T V, then Mk V and Nk V
  float v[NR == 1 ? 6 * 256 : HD * LDT + 2 * CH * LDT];
  int bad;              // a value that is not finite: token by token
  __device__ __forceinline__ float* kcT() { return v; }
  __device__ __forceinline__ float* mk() { return v + HD * LDT; }
  __device__ __forceinline__ float* nk() { return v + HD * LDT + CH * LDT; }
};

// product over the lanes of a row of 16 up to this one, for four values: a
// lane without a left neighbour at the distance keeps its value (a DPP read
// needs two wait states after its register was written: the s_nops, and between
// the steps the other three values)
__device__ __forceinline__ void row_scan4(f4& p) {
  float a = p[0], b = p[1], c = p[2], d = p[3];
#define RQ_SCAN_STEP(n)                                              \
  "v_mul_f32_dpp %0, %0, %0 row_shr:" #n " row_mask:0xf bank_mask:0xf\n" \
  "v_mul_f32_dpp %1, %1, %1 row_shr:" #n " row_mask:0xf bank_mask:0xf\n" \
  "v_mul_f32_dpp %2, %2, %2 row_shr:" #n " row_mask:0xf bank_mask:0xf\n" \
  "v_mul_f32_dpp %3, %3, %3 row_shr:" #n " row_mask:0xf bank_mask:0xf\n"
  asm("s_nop 1\n" RQ_SCAN_STEP(1) RQ_SCAN_STEP(2) RQ_SCAN_STEP(4) RQ_SCAN_STEP(8) "s_nop 1\n"
      : "+v"(a), "+v"(b), "+v"(c), "+v"(d));
#undef RQ_SCAN_STEP
  p = f4{a, b, c, d};
}
// the left neighbour's value, 1 in a row's first lane
__device__ __forceinline__ float left_or_one(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
                                       0x3f800000, __builtin_bit_cast(int, v), 0x111, 0xF, 0xF,
                                       false));
}

__device__ __forceinline__ f4 mma4(const f4& a, const f4& b, f4 c) {
#pragma unroll
  for (int v = 0; v < 4; v++) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[v], b[v], c, 0, 0, 0);
  return c;
}

// Barrier that waits for this wave's LDS accesses only: loads of later chunks
// and stores of outputs stay in flight across it (s_waitcnt with lgkmcnt 0,
// the other counters at their maxima).  Nothing is scheduled across it: what
// the compiler moved over a barrier to fill one wave's gaps made another wave's
// step longer.
__device__ __forceinline__ void step_barrier() {
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (0 << 8) | (3 << 14));
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// Inputs of one chunk as a producer lane holds them: token lane mod 16, keys
// 16 jt + 4 (lane / 16) .. + 3.  They stay as they were loaded until they are
// used: a conversion here would wait for them.
template <typename T>
struct Vec4;
template <>
struct Vec4<float> {
  typedef f4 type;
};
template <>
struct Vec4<_Float16> {
  typedef h4 type;
};
template <typename T>
struct ChunkIn {
  typedef typename Vec4<T>::type vec;
  vec w[4], k[4], kap[4], eta[4], r[4];
  __device__ __forceinline__ void load(const WkvArgs& a, size_t at) {
#pragma unroll
    for (int j = 0; j < 4; j++) {
      w[j] = *reinterpret_cast<const vec*>(static_cast<const T*>(a.w) + at + 16 * j);
      k[j] = *reinterpret_cast<const vec*>(static_cast<const T*>(a.k) + at + 16 * j);
      kap[j] = *reinterpret_cast<const vec*>(static_cast<const T*>(a.kappa) + at + 16 * j);
      eta[j] = *reinterpret_cast<const vec*>(static_cast<const T*>(a.eta) + at + 16 * j);
      r[j] = *reinterpret_cast<const vec*>(static_cast<const T*>(a.r) + at + 16 * j);
    }
  }
};

// z = kc^T V, from kcT [key][token] in LDS
__device__ __forceinline__ void keys_times_v(const float* kcT, const f4& V, f4* z) {
  const int lane = threadIdx.x & 63;
  f4 k[4];
#pragma unroll
  for (int j = 0; j < 4; j++) {
    k[j] = *reinterpret_cast<const f4*>(&kcT[(16 * j + (lane & 15)) * LDT + 4 * (lane >> 4)]);
    z[j] = f4{0, 0, 0, 0};
  }
  // four independent sums, so no MFMA waits for the one before it
#pragma unroll
  for (int v = 0; v < 4; v++)
#pragma unroll
    for (int j = 0; j < 4; j++)
      z[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(k[j][v], V[v], z[j], 0, 0, 0);
}
// mv = Mk V, nv = Nk V
__device__ __forceinline__ void tokens_times_v(const float* mk, const float* nk, const f4& V,
                                               f4* mv, f4* nv) {
  const int lane = threadIdx.x & 63, at = (lane & 15) * LDT + 4 * (lane >> 4);
  const f4 m = *reinterpret_cast<const f4*>(&mk[at]);
  const f4 n = *reinterpret_cast<const f4*>(&nk[at]);
  *mv = *nv = f4{0, 0, 0, 0};
#pragma unroll
  for (int v = 0; v < 4; v++) {
    *mv = __builtin_amdgcn_mfma_f32_16x16x4f32(m[v], V[v], *mv, 0, 0, 0);
    *nv = __builtin_amdgcn_mfma_f32_16x16x4f32(n[v], V[v], *nv, 0, 0, 0);
  }
}

// V of a chunk as a right operand: tokens 4 g + v of the lane's value row, as
// loaded; tokens past the end repeat the last one until they are used.
template <typename T>
struct ChunkV {
  T v[4];
  __device__ __forceinline__ void load(const T* col, size_t ld, int t0, int hi) {
    const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int i = 0; i < 4; i++) v[i] = col[(size_t)min(t0 + 4 * g + i, hi - 1) * ld];
  }
  __device__ __forceinline__ f4 get(int t0, int hi) const {
    const int g = (threadIdx.x & 63) >> 4;
    f4 r;
#pragma unroll
    for (int i = 0; i < 4; i++) r[i] = t0 + 4 * g + i < hi ? (float)v[i] : 0.0f;
    return r;
  }
};

// The value that lanes 16 G .. 16 G + 15 hold, in every row of 16 lanes.
template <int G>
__device__ __forceinline__ float row_of(float v) {
  const u32 u = __builtin_bit_cast(u32, v);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);  // rows 0 0 2 2, 1 1 3 3
  const u32 w = a[G & 1];
  const auto b = __builtin_amdgcn_permlane32_swap(w, w, false, false);
  const u32 r = b[G >> 1];
  return __builtin_bit_cast(float, r);
}
// Rows after S of x += column S of the strictly lower triangular m times row
// S of x (accumulator layout: rows 4 g + v, columns lane mod 16), then the
// rows after S + 1, and so on.
template <int S>
__device__ __forceinline__ void eliminate(const f4& m, f4& x) {
  if constexpr (S < CH - 1) {
    const float xs = row_of<S / 4>(x[S % 4]);
#pragma unroll
    for (int v = 0; v < 4; v++) {
      const float mv = m[v];
      x[v] = __builtin_fmaf(dpp_mov<0x150 + S>(mv), xs, x[v]);  // lane S of the row
    }
    eliminate<S + 1>(m, x);
  }
}

template <typename T, int NR>
__device__ __forceinline__ void produce(const WkvArgs& a, ChunkOps<NR>* ops, float* scratch,
                                        int p, int lo, int hi, size_t base, size_t ld, int row) {
  const int lane = threadIdx.x & 63, l16 = lane & 15, g = lane >> 4;
  const int n = (hi - lo + CH - 1) / CH;
  const T* vp = static_cast<const T*>(a.v) + base + row;
  ChunkIn<T> in;
  ChunkV<T> vin;
  auto fetch = [&](int c) {
    const int t0 = lo + c * CH;
    in.load(a, (size_t)min(t0 + l16, hi - 1) * ld + base + 4 * g);
    if constexpr (NR == 1) vin.load(vp, ld, t0, hi);
  };
  if (p < n) fetch(p);
  int steps = p;
  for (int i = 0; i < p; i++) step_barrier();
  for (int c = p; c < n; c += PRODUCERS) {
    const int t0 = lo + c * CH;
    // segment 1: decays and the scaled operands
    f4 ah[4], rh[4], bh[4], kh[4], pc[4], V = {0, 0, 0, 0};
    const bool live = t0 + l16 < hi;
    if (t0 + CH > hi && !live) {  // past the end: nothing decays, nothing is added
#pragma unroll
      for (int j = 0; j < 4; j++) {
        in.k[j] = in.kap[j] = in.eta[j] = in.r[j] = T(0);
        in.w[j] = T(-INFINITY);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; j++) {
      f4 P;
#pragma unroll
      for (int v = 0; v < 4; v++) P[v] = decay_of((float)in.w[j][v]);
      row_scan4(P);
#pragma unroll
      for (int v = 0; v < 4; v++) {
        const float kap = (float)in.kap[j][v];
        const float inv = __builtin_amdgcn_rcpf(P[v]);
        pc[j][v] = dpp_mov<0x15F>(P[v]);  // lane 15 of the row
        ah[j][v] = kap * left_or_one(P[v]);
        rh[j][v] = (float)in.r[j][v] * P[v];
        bh[j][v] = -((float)in.eta[j][v] * kap) * inv;
        kh[j][v] = (float)in.k[j][v] * inv;
      }
    }
    if constexpr (NR == 1) V = vin.get(t0, hi);
    if (c + PRODUCERS < n) fetch(c + PRODUCERS);  // two steps ahead of its use
    float* const kcT = NR == 1 ? scratch : ops[c & 1].kcT();
    f4 z[4];
    if constexpr (NR == 1) {
#pragma unroll
      for (int j = 0; j < 4; j++)
#pragma unroll
        for (int v = 0; v < 4; v++)
          kcT[(16 * j + 4 * g + v) * LDT + l16] = kh[j][v] * pc[j][v];
      // this wave's own writes, read back transposed (LDS keeps a wave's order)
      __atomic_signal_fence(__ATOMIC_SEQ_CST);
      keys_times_v(kcT, V, z);
    }
    step_barrier();
    // segment 2: the four products, rows t = 4 g + v, columns s = lane mod 16
    // (kept on this side of the barrier: the segments are of about one length)
#pragma unroll
    for (int j = 0; j < 4; j++) asm volatile("" : "+v"(ah[j]), "+v"(rh[j]));
    f4 mb = {0, 0, 0, 0}, mk = mb, nb = mb, nk = mb;
#pragma unroll
    for (int j = 0; j < 4; j++) {
#pragma unroll
      for (int v = 0; v < 4; v++) {
        mb = __builtin_amdgcn_mfma_f32_16x16x4f32(ah[j][v], bh[j][v], mb, 0, 0, 0);
        mk = __builtin_amdgcn_mfma_f32_16x16x4f32(ah[j][v], kh[j][v], mk, 0, 0, 0);
        nb = __builtin_amdgcn_mfma_f32_16x16x4f32(rh[j][v], bh[j][v], nb, 0, 0, 0);
        nk = __builtin_amdgcn_mfma_f32_16x16x4f32(rh[j][v], kh[j][v], nk, 0, 0, 0);
      }
    }
    // a value that is not finite leaves none of its row's or column's sums finite
    float zero = 0.0f;
    float* const mks = kcT + HD * LDT;
    float* const nks = mks + CH * LDT;
#pragma unroll
    for (int v = 0; v < 4; v++) {
      const int t = 4 * g + v;
      zero = __builtin_fmaf(mb[v], 0.0f, __builtin_fmaf(mk[v], 0.0f, zero));
      zero = __builtin_fmaf(nb[v], 0.0f, __builtin_fmaf(nk[v], 0.0f, zero));
      if (l16 >= t) mb[v] = mk[v] = 0.0f;
      if (l16 > t) nb[v] = nk[v] = 0.0f;
    }
    f4 mv, nv;
    if constexpr (NR == 1) {
#pragma unroll
      for (int v = 0; v < 4; v++) {
        mks[(4 * g + v) * LDT + l16] = mk[v];
        nks[(4 * g + v) * LDT + l16] = nk[v];
      }
      __atomic_signal_fence(__ATOMIC_SEQ_CST);  // as above
      tokens_times_v(mks, nks, V, &mv, &nv);
    }
    step_barrier();
    // segment 3: the rest, into the chunk's buffer
    ChunkOps<NR>& o = ops[c & 1];
#pragma unroll
    for (int j = 0; j < 4; j++) {
#pragma unroll
      for (int v = 0; v < 4; v++) {
        const int key = 16 * j + 4 * g + v;
        if constexpr (NR > 1) kcT[key * LDT + l16] = kh[j][v] * pc[j][v];
        o.bcT[key * LDT + l16] = bh[j][v] * pc[j][v];
      }
      *reinterpret_cast<f4*>(&o.ah[l16 * LDR + 16 * j + 4 * g]) = ah[j];
      *reinterpret_cast<f4*>(&o.rh[l16 * LDR + 16 * j + 4 * g]) = rh[j];
      if (l16 == 0) *reinterpret_cast<f4*>(&o.pc[16 * j + 4 * g]) = pc[j];
    }
#pragma unroll
    for (int v = 0; v < 4; v++) {
      const int at = (4 * g + v) * LDT + l16;
      if constexpr (NR > 1) {
        mks[at] = mk[v];
        nks[at] = nk[v];
      }
      o.nb[at] = nb[v];
    }
    if constexpr (NR == 1) {
      f4* dst = reinterpret_cast<f4*>(o.v) + lane;
#pragma unroll
      for (int j = 0; j < 4; j++) dst[64 * j] = z[j];
      dst[256] = mv;
      dst[320] = nv;
#pragma unroll
      for (int v = 0; v < 4; v++) zero = __builtin_fmaf(z[0][v], 0.0f, zero);
    }
    // X by forward substitution: row s is final once the rows before it have
    // been taken off; it goes to all lanes, and every row takes its share
    f4 x;
#pragma unroll
    for (int v = 0; v < 4; v++) x[v] = l16 == 4 * g + v ? 1.0f : 0.0f;
    eliminate<0>(mb, x);
#pragma unroll
    for (int v = 0; v < 4; v++) o.x[(4 * g + v) * LDT + l16] = x[v];
    const bool bad = __ballot(!(zero == 0.0f)) != 0;
    if (lane == 0) o.bad = bad;
    step_barrier();
    steps += 3;
  }
  for (; steps < n + 3; steps++) step_barrier();
}

template <typename T, int NR>
__global__ void __launch_bounds__(64 * (NR + PRODUCERS))
k_wkv_chunk(const WkvArgs a) {
  __shared__ __align__(16) ChunkOps<NR> ops[2];
  // the producers' own copies of kcT, mk and nk
  __shared__ __align__(16) float scratch[NR == 1 ? PRODUCERS : 1][NR == 1 ? (2 * CH + HD) * LDT : 1];
  // heads are the fast index: a sequence's workgroups go to all XCDs
  constexpr int TILES = 4 / NR;
  const int q = blockIdx.x / (a.H * TILES), h = blockIdx.x % (a.H * TILES) / TILES;
  const int lo = max(a.offsets[q], 0), hi = min(a.offsets[q + 1], a.T);
  if (lo >= hi) return;
  const int n = (hi - lo + CH - 1) / CH;
  const size_t ld = (size_t)a.H * HD, base = (size_t)h * HD;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, l16 = lane & 15, g = lane >> 4;
  const int i = 16 * (blockIdx.x % TILES * NR + wave % NR) + l16;  // the lane's value row
  if (wave >= NR) {
    produce<T, NR>(a, ops, scratch[NR == 1 ? wave - NR : 0], wave - NR, lo, hi, base, ld, i);
    return;
  }
  const int slot = a.slots ? a.slots[q] : q;
  const bool stored = slot >= 0 && slot < a.nslots;
  float* st = a.state + (((size_t)(stored ? slot : 0) * a.H + h) * HD + i) * HD + 4 * g;
  f4 S[4];  // keys 16 j + 4 g + v
#pragma unroll
  for (int j = 0; j < 4; j++) {
    S[j] = f4{0, 0, 0, 0};
    if (stored) S[j] = *reinterpret_cast<const f4*>(st + 16 * j);
  }
  const T* vp = static_cast<const T*>(a.v) + base + i;
  float* yp = a.y + base + i;
  ChunkV<T> vin;
  if constexpr (NR > 1) vin.load(vp, ld, lo, hi);
  for (int s = 0; s < 3; s++) step_barrier();
  // the state has arrived before the loop, so that no wait inside it stands
  // for these loads (and with them for the stores of y)
#pragma unroll
  for (int j = 0; j < 4; j++) asm volatile("" : "+v"(S[j]));
  for (int c = 0; c < n; c++) {
    ChunkOps<NR>& o = ops[c & 1];
    const int t0 = lo + c * CH;
    const int at = l16 * LDT + 4 * g;
    f4 u, y, z[4], ah[4], rh[4], bc[4], pc[4];
    // all of the chunk's operands are asked for at once
#pragma unroll
    for (int j = 0; j < 4; j++) {
      ah[j] = *reinterpret_cast<const f4*>(&o.ah[l16 * LDR + 16 * j + 4 * g]);
      rh[j] = *reinterpret_cast<const f4*>(&o.rh[l16 * LDR + 16 * j + 4 * g]);
    }
    const int bad = o.bad;
    const f4 x = *reinterpret_cast<const f4*>(&o.x[at]);
    const f4 nb = *reinterpret_cast<const f4*>(&o.nb[at]);
#pragma unroll
    for (int j = 0; j < 4; j++) {
      bc[j] = *reinterpret_cast<const f4*>(&o.bcT[16 * j * LDT + at]);
      pc[j] = *reinterpret_cast<const f4*>(&o.pc[16 * j + 4 * g]);
    }
    float zero = 0.0f;  // NaN where a state is not finite
#pragma unroll
    for (int j = 0; j < 4; j++)
#pragma unroll
      for (int v = 0; v < 4; v++) zero = __builtin_fmaf(S[j][v], 0.0f, zero);
    if constexpr (NR > 1) {
      const f4 V = vin.get(t0, hi);
      if (c + 1 < n) vin.load(vp, ld, t0 + CH, hi);
#pragma unroll
      for (int v = 0; v < 4; v++) zero = __builtin_fmaf(V[v], 0.0f, zero);
      keys_times_v(o.kcT(), V, z);
      tokens_times_v(o.mk(), o.nk(), V, &u, &y);
    } else {
      const f4* src = reinterpret_cast<const f4*>(o.v) + lane;
#pragma unroll
      for (int j = 0; j < 4; j++) z[j] = src[64 * j];
      u = src[256];
      y = src[320];
    }
#pragma unroll
    for (int j = 0; j < 4; j++) {
#pragma unroll
      for (int v = 0; v < 4; v++) {
        u = __builtin_amdgcn_mfma_f32_16x16x4f32(ah[j][v], S[j][v], u, 0, 0, 0);
        y = __builtin_amdgcn_mfma_f32_16x16x4f32(rh[j][v], S[j][v], y, 0, 0, 0);
      }
    }
    if (!bad && __ballot(!(zero == 0.0f)) == 0) {
      const f4 U = mma4(x, u, f4{0, 0, 0, 0});
#pragma unroll
      for (int j = 0; j < 4; j++)
#pragma unroll
        for (int v = 0; v < 4; v++) S[j][v] = __builtin_fmaf(S[j][v], pc[j][v], z[j][v]);
#pragma unroll
      for (int v = 0; v < 4; v++) {
#pragma unroll
        for (int j = 0; j < 4; j++)
          S[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(bc[j][v], U[v], S[j], 0, 0, 0);
        y = __builtin_amdgcn_mfma_f32_16x16x4f32(nb[v], U[v], y, 0, 0, 0);
      }
      float* yt = yp + (size_t)(t0 + 4 * g) * ld;
      if (t0 + CH <= hi) {
#pragma unroll
        for (int v = 0; v < 4; v++) yt[v * ld] = y[v];
      } else {
#pragma unroll
        for (int v = 0; v < 4; v++)
          if (t0 + 4 * g + v < hi) yt[v * ld] = y[v];
      }
    } else {
      // a value that is not finite must not reach earlier tokens through
      // products with the zeros of the triangular matrices
      for (int t = t0; t < min(t0 + CH, hi); t++) {
        const size_t at = (size_t)t * ld + base + 4 * g;
        const float vt = (float)vp[(size_t)t * ld];
        f4 kap[4];
        float sk = 0.0f, yt = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; j++) {
          kap[j] = load4(static_cast<const T*>(a.kappa) + at + 16 * j);
#pragma unroll
          for (int v = 0; v < 4; v++) sk += S[j][v] * kap[j][v];
        }
        sk += __shfl_xor(sk, 16, 64);
        sk += __shfl_xor(sk, 32, 64);
#pragma unroll
        for (int j = 0; j < 4; j++) {
          const f4 w = load4(static_cast<const T*>(a.w) + at + 16 * j);
          const f4 k = load4(static_cast<const T*>(a.k) + at + 16 * j);
          const f4 eta = load4(static_cast<const T*>(a.eta) + at + 16 * j);
          const f4 r = load4(static_cast<const T*>(a.r) + at + 16 * j);
#pragma unroll
          for (int v = 0; v < 4; v++) {
            S[j][v] = S[j][v] * decay_of(w[v]) - sk * (eta[v] * kap[j][v]) + vt * k[v];
            yt += S[j][v] * r[v];
          }
        }
        yt += __shfl_xor(yt, 16, 64);
        yt += __shfl_xor(yt, 32, 64);
        if (g == 0) yp[(size_t)t * ld] = yt;
      }
    }
    step_barrier();
  }
  if (stored) {
#pragma unroll
    for (int j = 0; j < 4; j++) *reinterpret_cast<f4*>(st + 16 * j) = S[j];
  }
}

template <typename T, int NR>
void launch_chunks(const WkvArgs& a, unsigned heads, hipStream_t s) {
  hipLaunchKernelGGL((k_wkv_chunk<T, NR>), dim3(heads * (4 / NR)), dim3(64 * (NR + PRODUCERS)), 0,
                     s, a);
}

template <typename T>
void launch(const WkvArgs& a, hipStream_t s) {
  const unsigned heads = (unsigned)a.sequences * a.H;
  if (a.T - a.sequences < 32)
    hipLaunchKernelGGL((k_wkv_seq<T>), dim3(heads), dim3(256), 0, s, a);
  else if (heads <= 80)
    launch_chunks<T, 1>(a, heads, s);
  else if (heads < 256)
    launch_chunks<T, 2>(a, heads, s);
  else
    launch_chunks<T, 4>(a, heads, s);
}

}  // namespace

hipError_t launch_wkv(const WkvArgs& a, hipStream_t s) {
  if (a.half) launch<_Float16>(a, s);
  else launch<float>(a, s);
  return hipGetLastError();
}

}  // namespace rq
