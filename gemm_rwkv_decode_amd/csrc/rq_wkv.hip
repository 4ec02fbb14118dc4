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
// chunk's start), Q = P_8 and S0 the state before the chunk, the recurrence is
//   u_t = (S0 o Q) (kappa_t o P_{t-1} / Q) + sum_{s<t}  (Mb[t][s] u_s + Mk[t][s] v_s)
//   y_t = (S0 o Q) (r_t o P_t / Q)         + sum_{s<=t} (Nb[t][s] u_s + Nk[t][s] v_s)
//   S16 = S0 diag(P_16) + sum_s (u_s bc_s^T + v_s kc_s^T)
// where u_t = S_{t-1} kappa_t and, with a_t = kappa_t o P_{t-1} / Q, q_t = r_t o
// P_t / Q, b_s = -(eta o kappa)_s o Q / P_s, k_s standing for k_s o Q / P_s,
//   Mb[t][s] = a_t . b_s   Mk[t][s] = a_t . k_s   Nb[t][s] = q_t . b_s   Nk[t][s] = q_t . k_s
//   bc_s = b_s o P_16 / Q,   kc_s = k_s o P_16 / Q.
// Mb is strictly lower triangular, so U = X (S0 part + Mk V), X = (I - Mb)^-1.
// Every decay is at least 0.545, so the factors P / Q lie between 2^-7 and
// 2^7 whatever w is; a chunk is 16 tokens for that reason and because it is
// the matrix instructions' tile.
//
// Products run on the binary16 matrix cores with binary32 sums, every operand
// in two parts, x = hi + 2^-11 lo, both binary16: hi hi' goes to one sum, hi lo'
// + lo hi' to a second that joins with 2^-11.  What is left out or rounded is
// below 2^-22 of an operand (2^-36 in absolute terms for values under 2^-14),
// so a product is as good as a binary32 one, at three binary16 MFMAs for eight
// binary32 ones of twice the length.  The state itself, the decays, the
// triangular inverse and everything added up stay binary32.
// A chunk in which a value does not fit this (not finite, 2^15 or more, or
// nothing as large as 2^-12 in k, r, or the state and v together) is done token
// by token in binary32 instead.
//
// The contraction order is free, so operands are laid out for the accumulator:
// a lane's accumulator f4 covers rows 4 (l / 16) .. + 3 of column l mod 16, and
// as a right operand it is the contraction index 4 (l / 16) + v (of two tiles,
// for the 32-deep instruction).  The state S^T [keys][values], U and V are
// therefore used as they come, with no exchange between lanes, and the state
// never leaves its registers.  The left operands Mk, Nb, Nk and X are made as
// their transposes, whose accumulators are the operands; kc and bc are turned
// by products with the identity.
//
// A workgroup has NR state waves, 16 value rows each, and three producer waves
// that prepare what depends on the inputs alone (decays, the four 16x16
// matrices, the triangular inverse), one chunk each, in three segments one
// barrier apart; chunk c's operands go through LDS, two buffers in turn.
// ---------------------------------------------------------------------------
constexpr int CH = 16;  // tokens of a chunk
constexpr int PRODUCERS = 3;
constexpr float UP = 2048.0f, DOWN = 1.0f / 2048.0f;  // the low part's scale
constexpr float TINY = 1.0f / 4096.0f, HUGE_ = 32768.0f;

// Two-part operands: 4 deep (one accumulator tile) and 8 deep (two).
struct P4 {
  h4 hi, lo;
};
struct P8 {
  h8 hi, lo;
};
__device__ __forceinline__ P4 split(const f4& x) {
  P4 p;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    // x as rounded to binary32: the compiler would else round the product
    // behind x to binary16 in one step in one place and in two in another, and
    // hi and lo would not belong together
    float v = x[i];
    asm("" : "+v"(v));
    p.hi[i] = (_Float16)v;
    p.lo[i] = (_Float16)__builtin_fmaf(-UP, (float)p.hi[i], UP * v);
  }
  return p;
}
__device__ __forceinline__ P8 join(const P4& a, const P4& b) {
  return P8{__builtin_shufflevector(a.hi, b.hi, 0, 1, 2, 3, 4, 5, 6, 7),
            __builtin_shufflevector(a.lo, b.lo, 0, 1, 2, 3, 4, 5, 6, 7)};
}
// A product's two sums.
struct Sum {
  f4 main, cross;
  __device__ __forceinline__ f4 value() const {
    f4 r;
#pragma unroll
    for (int i = 0; i < 4; i++) r[i] = __builtin_fmaf(DOWN, cross[i], main[i]);
    return r;
  }
};
__device__ __forceinline__ Sum none() { return Sum{f4{0, 0, 0, 0}, f4{0, 0, 0, 0}}; }
__device__ __forceinline__ void mma(const P4& a, const P4& b, Sum& c) {
  c.main = __builtin_amdgcn_mfma_f32_16x16x16f16(a.hi, b.hi, c.main, 0, 0, 0);
  c.cross = __builtin_amdgcn_mfma_f32_16x16x16f16(a.hi, b.lo, c.cross, 0, 0, 0);
  c.cross = __builtin_amdgcn_mfma_f32_16x16x16f16(a.lo, b.hi, c.cross, 0, 0, 0);
}
__device__ __forceinline__ void mma(const P8& a, const P8& b, Sum& c) {
  c.main = __builtin_amdgcn_mfma_f32_16x16x32_f16(a.hi, b.hi, c.main, 0, 0, 0);
  c.cross = __builtin_amdgcn_mfma_f32_16x16x32_f16(a.hi, b.lo, c.cross, 0, 0, 0);
  c.cross = __builtin_amdgcn_mfma_f32_16x16x32_f16(a.lo, b.hi, c.cross, 0, 0, 0);
}

// What a chunk's state waves read: left operands by lane, decays by key.
struct alignas(16) ChunkOps {
  h8 a[2][2][64];   // [part][two key tiles][lane]: a_t
  h8 q[2][2][64];   // q_t
  h8 kb[2][4][64];  // [part][key tile][lane]: kc, then bc, of tokens 4 g + v
  h4 x[2][64], nb[2][64], mk[2][64], nk[2][64];
  int slow;         // token by token
};
// Q and P_16 of a chunk.  Written two steps before the other operands, so four
// of them in turn.
struct alignas(16) ChunkDecays {
  float mid[HD], end[HD];
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
// X^T = I + Mb^T X^T by substitution from the last row: row T is final once the
// rows after it have been taken off; it goes to all lanes, and every row s takes
// Mb^T[s][T] of it (accumulator layout: rows 4 g + v, columns lane mod 16).
template <int T>
__device__ __forceinline__ void eliminate(const f4& m, f4& x) {
  if constexpr (T > 0) {
    const float xs = row_of<T / 4>(x[T % 4]);
#pragma unroll
    for (int v = 0; v < 4; v++) {
      const float mv = m[v];
      x[v] = __builtin_fmaf(dpp_mov<0x150 + T>(mv), xs, x[v]);  // lane T of the row
    }
    eliminate<T - 1>(m, x);
  }
}

__device__ __forceinline__ float larger(float m, const f4& x) {
#pragma unroll
  for (int i = 0; i < 4; i++) m = fmaxf(m, fabsf(x[i]));
  return m;
}
// Whether the wave's largest magnitude (m over the lanes) is too small for
// two-part operands: under 2^-12 and not zero.
__device__ __forceinline__ bool too_small(float m) {
  return __ballot(m >= TINY) == 0 && __ballot(m > 0.0f) != 0;
}

template <typename T>
__device__ __forceinline__ void produce(const WkvArgs& a, ChunkOps* ops, ChunkDecays* decays,
                                        int p, int lo, int hi, size_t base, size_t ld) {
  const int lane = threadIdx.x & 63, l16 = lane & 15, g = lane >> 4;
  const int n = (hi - lo + CH - 1) / CH;
  ChunkIn<T> in;
  auto fetch = [&](int c) {
    in.load(a, (size_t)min(lo + c * CH + l16, hi - 1) * ld + base + 4 * g);
  };
  h4 identity;
#pragma unroll
  for (int v = 0; v < 4; v++) identity[v] = l16 == 4 * g + v ? (_Float16)1.0f : (_Float16)0.0f;
  if (p < n) fetch(p);
  int steps = p;
  for (int i = 0; i < p; i++) step_barrier();
  for (int c = p; c < n; c += PRODUCERS) {
    const int t0 = lo + c * CH;
    // segment 1: decays and the scaled operands
    f4 av[4], qv[4], bv[4], kv[4], rest[4];  // rest: P_16 / Q
    const bool live = t0 + l16 < hi;
    if (t0 + CH > hi && !live) {  // past the end: nothing decays, nothing is added
#pragma unroll
      for (int j = 0; j < 4; j++) {
        in.k[j] = in.kap[j] = in.eta[j] = in.r[j] = T(0);
        in.w[j] = T(-INFINITY);
      }
    }
    float big_k = 0.0f, big_r = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; j++) {
      f4 P, mid, end;
#pragma unroll
      for (int v = 0; v < 4; v++) P[v] = decay_of((float)in.w[j][v]);
      row_scan4(P);
#pragma unroll
      for (int v = 0; v < 4; v++) {
        const float kap = (float)in.kap[j][v], k = (float)in.k[j][v], r = (float)in.r[j][v];
        const float inv = __builtin_amdgcn_rcpf(P[v]);
        mid[v] = dpp_mov<0x157>(P[v]);           // lane 7 of the row: Q
        const float over = dpp_mov<0x157>(inv);  // 1 / Q
        end[v] = dpp_mov<0x15F>(P[v]);           // lane 15: P_16
        rest[j][v] = end[v] * over;
        const float up = inv * mid[v];
        av[j][v] = kap * (left_or_one(P[v]) * over);
        qv[j][v] = r * (P[v] * over);
        bv[j][v] = -((float)in.eta[j][v] * kap) * up;
        kv[j][v] = k * up;
        big_k = fmaxf(big_k, fabsf(k));
        big_r = fmaxf(big_r, fabsf(r));
      }
      if (l16 == 0) {
        *reinterpret_cast<f4*>(&decays[c & 3].mid[16 * j + 4 * g]) = mid;
        *reinterpret_cast<f4*>(&decays[c & 3].end[16 * j + 4 * g]) = end;
      }
    }
    if (c + PRODUCERS < n) fetch(c + PRODUCERS);  // two steps ahead of its use
    bool slow = too_small(big_k) || too_small(big_r);
    step_barrier();
    // segment 2: the four products' transposes, rows s = 4 g + v, columns t =
    // lane mod 16, and kc and bc turned from tokens x keys to keys x tokens by
    // products with the identity, which are exact
    P8 ap[2], qp[2], kb[4];
    Sum mb = none(), mk = mb, nb = mb, nk = mb;
#pragma unroll
    for (int q = 0; q < 2; q++) {
      ap[q] = join(split(av[2 * q]), split(av[2 * q + 1]));
      qp[q] = join(split(qv[2 * q]), split(qv[2 * q + 1]));
      const P8 bp = join(split(bv[2 * q]), split(bv[2 * q + 1]));
      const P8 kp = join(split(kv[2 * q]), split(kv[2 * q + 1]));
      mma(bp, ap[q], mb);
      mma(kp, ap[q], mk);
      mma(bp, qp[q], nb);
      mma(kp, qp[q], nk);
    }
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const P4 kp = split(kv[j] * rest[j]), bp = split(bv[j] * rest[j]);
      const f4 z = {0, 0, 0, 0};
      const f4 kh = __builtin_amdgcn_mfma_f32_16x16x16f16(kp.hi, identity, z, 0, 0, 0);
      const f4 bh = __builtin_amdgcn_mfma_f32_16x16x16f16(bp.hi, identity, z, 0, 0, 0);
      const f4 kl = __builtin_amdgcn_mfma_f32_16x16x16f16(kp.lo, identity, z, 0, 0, 0);
      const f4 bl = __builtin_amdgcn_mfma_f32_16x16x16f16(bp.lo, identity, z, 0, 0, 0);
#pragma unroll
      for (int v = 0; v < 4; v++) {
        kb[j].hi[v] = (_Float16)kh[v];
        kb[j].hi[4 + v] = (_Float16)bh[v];
        kb[j].lo[v] = (_Float16)kl[v];
        kb[j].lo[4 + v] = (_Float16)bl[v];
      }
    }
    f4 mbv = mb.value(), mkv = mk.value(), nbv = nb.value(), nkv = nk.value();
    step_barrier();
    // segment 3: the triangular inverse, and everything to the chunk's buffer
    ChunkOps& o = ops[c & 1];
#pragma unroll
    for (int q = 0; q < 2; q++) {
      o.a[0][q][lane] = ap[q].hi;
      o.a[1][q][lane] = ap[q].lo;
      o.q[0][q][lane] = qp[q].hi;
      o.q[1][q][lane] = qp[q].lo;
    }
#pragma unroll
    for (int j = 0; j < 4; j++) {
      o.kb[0][j][lane] = kb[j].hi;
      o.kb[1][j][lane] = kb[j].lo;
    }
    // a value that is not finite, or too large for an operand, leaves none of
    // its row's or column's sums finite
    float zero = 0.0f;
#pragma unroll
    for (int v = 0; v < 4; v++) {
      zero = __builtin_fmaf(mbv[v], 0.0f, __builtin_fmaf(mkv[v], 0.0f, zero));
      zero = __builtin_fmaf(nbv[v], 0.0f, __builtin_fmaf(nkv[v], 0.0f, zero));
      if (4 * g + v >= l16) mbv[v] = mkv[v] = 0.0f;
      if (4 * g + v > l16) nbv[v] = nkv[v] = 0.0f;
    }
    f4 x;
#pragma unroll
    for (int v = 0; v < 4; v++) x[v] = l16 == 4 * g + v ? 1.0f : 0.0f;
    eliminate<CH - 1>(mbv, x);
    const float big = larger(larger(larger(larger(0.0f, x), mkv), nbv), nkv);
    slow = slow || __ballot(!(zero == 0.0f) || !(big < HUGE_)) != 0;
    const P4 xp = split(x), mkp = split(mkv), nbp = split(nbv), nkp = split(nkv);
    o.x[0][lane] = xp.hi;
    o.x[1][lane] = xp.lo;
    o.mk[0][lane] = mkp.hi;
    o.mk[1][lane] = mkp.lo;
    o.nb[0][lane] = nbp.hi;
    o.nb[1][lane] = nbp.lo;
    o.nk[0][lane] = nkp.hi;
    o.nk[1][lane] = nkp.lo;
    if (lane == 0) o.slow = slow;
    step_barrier();
    steps += 3;
  }
  for (; steps < n + 3; steps++) step_barrier();
}

template <typename T, int NR>
__global__ void __launch_bounds__(64 * (NR + PRODUCERS))
k_wkv_chunk(const WkvArgs a) {
  __shared__ ChunkOps ops[2];
  __shared__ ChunkDecays decays[4];
  // heads are the fast index: a sequence's workgroups go to all XCDs
  constexpr int TILES = 4 / NR;
  const int sq = blockIdx.x / (a.H * TILES), h = blockIdx.x % (a.H * TILES) / TILES;
  const int lo = max(a.offsets[sq], 0), hi = min(a.offsets[sq + 1], a.T);
  if (lo >= hi) return;
  const int n = (hi - lo + CH - 1) / CH;
  const size_t ld = (size_t)a.H * HD, base = (size_t)h * HD;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (wave >= NR) {
    produce<T>(a, ops, decays, wave - NR, lo, hi, base, ld);
    return;
  }
  const int lane = threadIdx.x & 63, l16 = lane & 15, g = lane >> 4;
  const int i = 16 * (blockIdx.x % TILES * NR + wave % NR) + l16;  // the lane's value row
  const int slot = a.slots ? a.slots[sq] : sq;
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
  vin.load(vp, ld, lo, hi);
  for (int s = 0; s < 3; s++) step_barrier();
  // the state has arrived before the loop, so that no wait inside it stands
  // for these loads (and with them for the stores of y)
#pragma unroll
  for (int j = 0; j < 4; j++) asm volatile("" : "+v"(S[j]));
  for (int c = 0; c < n; c++) {
    const ChunkOps& o = ops[c & 1];
    const int t0 = lo + c * CH;
    P8 ap[2], qp[2], kb[4];
#pragma unroll
    for (int q = 0; q < 2; q++) {
      ap[q] = P8{o.a[0][q][lane], o.a[1][q][lane]};
      qp[q] = P8{o.q[0][q][lane], o.q[1][q][lane]};
    }
    const P4 mk{o.mk[0][lane], o.mk[1][lane]}, nk{o.nk[0][lane], o.nk[1][lane]};
    const P4 xp{o.x[0][lane], o.x[1][lane]}, nb{o.nb[0][lane], o.nb[1][lane]};
#pragma unroll
    for (int j = 0; j < 4; j++) kb[j] = P8{o.kb[0][j][lane], o.kb[1][j][lane]};
    bool slow = o.slow;
    const f4 V = vin.get(t0, hi);
    if (c + 1 < n) vin.load(vp, ld, t0 + CH, hi);
    f4 Sq[4];
    float big = larger(0.0f, V);
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const f4 mid = *reinterpret_cast<const f4*>(&decays[c & 3].mid[16 * j + 4 * g]);
#pragma unroll
      for (int v = 0; v < 4; v++) Sq[j][v] = S[j][v] * mid[v];
      big = larger(big, Sq[j]);
    }
    slow = slow || too_small(big);
    const P4 vs = split(V);
    Sum u = none(), y = u;
    mma(mk, vs, u);
    mma(nk, vs, y);
#pragma unroll
    for (int q = 0; q < 2; q++) {
      const P8 sp = join(split(Sq[2 * q]), split(Sq[2 * q + 1]));
      mma(ap[q], sp, u);
      mma(qp[q], sp, y);
    }
    Sum us = none();
    mma(xp, split(u.value()), us);
    const f4 U = us.value();
    // what is not finite, or too large for an operand, in V, S or U
    slow = slow || __ballot(!(fabsf(U[0]) + fabsf(U[1]) + fabsf(U[2]) + fabsf(U[3]) < HUGE_)) != 0;
    if (!slow) {
      const P4 up = split(U);
      const P8 vu = join(vs, up);
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const f4 end = *reinterpret_cast<const f4*>(&decays[c & 3].end[16 * j + 4 * g]);
        Sum s = none();
#pragma unroll
        for (int v = 0; v < 4; v++) s.main[v] = S[j][v] * end[v];
        mma(kb[j], vu, s);
        S[j] = s.value();
      }
      mma(nb, up, y);
      const f4 yv = y.value();
      float* yt = yp + (size_t)(t0 + 4 * g) * ld;
      if (t0 + CH <= hi) {
#pragma unroll
        for (int v = 0; v < 4; v++) yt[v * ld] = yv[v];
      } else {
#pragma unroll
        for (int v = 0; v < 4; v++)
          if (t0 + 4 * g + v < hi) yt[v * ld] = yv[v];
      }
    } else {
      // token by token (a value that is not finite must not reach earlier
      // tokens through products with the zeros of the triangular matrices)
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
