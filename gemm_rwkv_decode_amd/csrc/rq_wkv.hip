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

struct ChunkOps {
  float ah[CH * LDR];     // kappa_t o P_{t-1}
  float rh[CH * LDR];     // r_t o P_t
  float bcT[HD * LDT];    // [key][token]
  float kcT[HD * LDT];
  float x[CH * LDT];      // (I - Mb)^-1
  float mk[CH * LDT], nb[CH * LDT], nk[CH * LDT];
  float pc[HD];           // P_16
  int bad;                // a value that is not finite: token by token
};

// product over the lanes of a row of 16 up to this one
template <int CTRL>
__device__ __forceinline__ float dpp_or_one(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
                                       0x3f800000, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF,
                                       false));
}
__device__ __forceinline__ float row_scan(float v) {
  v *= dpp_or_one<0x111>(v);  // row_shr:1
  v *= dpp_or_one<0x112>(v);
  v *= dpp_or_one<0x114>(v);
  v *= dpp_or_one<0x118>(v);
  return v;
}

__device__ __forceinline__ f4 mma4(const f4& a, const f4& b, f4 c) {
#pragma unroll
  for (int v = 0; v < 4; v++) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[v], b[v], c, 0, 0, 0);
  return c;
}

__device__ __forceinline__ void step_barrier() { __syncthreads(); }

// Inputs of one chunk as a producer lane holds them: token lane mod 16, keys
// 16 jt + 4 (lane / 16) .. + 3.
template <typename T>
struct ChunkIn {
  f4 w[4], k[4], kap[4], eta[4], r[4];
  __device__ __forceinline__ void load(const WkvArgs& a, size_t at, bool in) {
#pragma unroll
    for (int j = 0; j < 4; j++) {
      w[j] = load4(static_cast<const T*>(a.w) + at + 16 * j);
      k[j] = load4(static_cast<const T*>(a.k) + at + 16 * j);
      kap[j] = load4(static_cast<const T*>(a.kappa) + at + 16 * j);
      eta[j] = load4(static_cast<const T*>(a.eta) + at + 16 * j);
      r[j] = load4(static_cast<const T*>(a.r) + at + 16 * j);
    }
    // tokens past the sequence's end: nothing decays, nothing is added
    if (!in) {
#pragma unroll
      for (int j = 0; j < 4; j++) {
        k[j] = kap[j] = eta[j] = r[j] = f4{0, 0, 0, 0};
        w[j] = f4{-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      }
    }
  }
};

template <typename T>
__device__ __forceinline__ void produce(const WkvArgs& a, ChunkOps* ops, float* scratch, int p,
                                        int lo, int hi, size_t base, size_t ld) {
  const int lane = threadIdx.x & 63, l16 = lane & 15, g = lane >> 4;
  const int n = (hi - lo + CH - 1) / CH;
  ChunkIn<T> in;
  auto fetch = [&](int c) {
    const int t = lo + c * CH + l16;
    in.load(a, (size_t)min(t, hi - 1) * ld + base + 4 * g, t < hi);
  };
  if (p < n) fetch(p);
  int steps = p;
  for (int i = 0; i < p; i++) step_barrier();
  for (int c = p; c < n; c += PRODUCERS) {
    // segment 1: decays and the scaled operands
    f4 ah[4], rh[4], bh[4], kh[4], pc[4];
    float zero = 0.0f;  // NaN as soon as anything is not finite
#pragma unroll
    for (int j = 0; j < 4; j++) {
#pragma unroll
      for (int v = 0; v < 4; v++) {
        const float P = row_scan(decay_of(in.w[j][v]));
        const float before = dpp_or_one<0x111>(P);
        const float inv = __builtin_amdgcn_rcpf(P);
        pc[j][v] = dpp_mov<0x15F>(P);  // lane 15 of the row
        ah[j][v] = in.kap[j][v] * before;
        rh[j][v] = in.r[j][v] * P;
        bh[j][v] = -(in.eta[j][v] * in.kap[j][v]) * inv;
        kh[j][v] = in.k[j][v] * inv;
        zero = __builtin_fmaf(ah[j][v], 0.0f, zero);
        zero = __builtin_fmaf(rh[j][v], 0.0f, zero);
        zero = __builtin_fmaf(bh[j][v], 0.0f, zero);
        zero = __builtin_fmaf(kh[j][v], 0.0f, zero);
      }
    }
    const bool bad = __ballot(!(zero == 0.0f)) != 0;
    step_barrier();
    // segment 2: the four products, rows t = 4 g + v, columns s = lane mod 16
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
#pragma unroll
    for (int v = 0; v < 4; v++) {
      const int t = 4 * g + v;
      if (l16 >= t) mb[v] = mk[v] = 0.0f;
      if (l16 > t) nb[v] = nk[v] = 0.0f;
      scratch[t * LDT + l16] = mb[v];
    }
    step_barrier();
    // segment 3: column l16 of X by forward substitution, then everything to
    // the chunk's buffer
    ChunkOps& o = ops[c & 1];
    float x[CH];
#pragma unroll
    for (int t = 0; t < CH; t++) {
      x[t] = l16 == t ? 1.0f : 0.0f;
#pragma unroll
      for (int s4 = 0; s4 < t; s4 += 4) {
        const f4 m = *reinterpret_cast<const f4*>(&scratch[t * LDT + s4]);
#pragma unroll
        for (int s = s4; s < s4 + 4 && s < t; s++) x[t] = __builtin_fmaf(m[s - s4], x[s], x[t]);
      }
      o.x[t * LDT + l16] = x[t];
    }
#pragma unroll
    for (int j = 0; j < 4; j++) {
      *reinterpret_cast<f4*>(&o.ah[l16 * LDR + 16 * j + 4 * g]) = ah[j];
      *reinterpret_cast<f4*>(&o.rh[l16 * LDR + 16 * j + 4 * g]) = rh[j];
      if (l16 == 0) *reinterpret_cast<f4*>(&o.pc[16 * j + 4 * g]) = pc[j];
#pragma unroll
      for (int v = 0; v < 4; v++) {
        const int key = 16 * j + 4 * g + v;
        o.bcT[key * LDT + l16] = bh[j][v] * pc[j][v];
        o.kcT[key * LDT + l16] = kh[j][v] * pc[j][v];
      }
    }
#pragma unroll
    for (int v = 0; v < 4; v++) {
      const int at = (4 * g + v) * LDT + l16;
      o.mk[at] = mk[v];
      o.nb[at] = nb[v];
      o.nk[at] = nk[v];
    }
    if (lane == 0) o.bad = bad;
    if (c + PRODUCERS < n) fetch(c + PRODUCERS);
    step_barrier();
    steps += 3;
  }
  for (; steps < n + 3; steps++) step_barrier();
}

template <typename T, int NR>
__global__ void __launch_bounds__(64 * (NR + PRODUCERS))
k_wkv_chunk(const WkvArgs a) {
  __shared__ __align__(16) ChunkOps ops[2];
  __shared__ __align__(16) float scratch[PRODUCERS][CH * LDT];
  const int q = blockIdx.x, h = blockIdx.y / (4 / NR);
  const int lo = max(a.offsets[q], 0), hi = min(a.offsets[q + 1], a.T);
  if (lo >= hi) return;
  const int n = (hi - lo + CH - 1) / CH;
  const size_t ld = (size_t)a.H * HD, base = (size_t)h * HD;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (wave >= NR) {
    produce<T>(a, ops, scratch[wave - NR], wave - NR, lo, hi, base, ld);
    return;
  }
  const int lane = threadIdx.x & 63, l16 = lane & 15, g = lane >> 4;
  const int i = 16 * (NR == 4 ? wave : blockIdx.y % 4) + l16;  // the lane's value row
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
  f4 V;  // tokens 4 g + v of the next chunk
  auto fetch_v = [&](int c) {
#pragma unroll
    for (int v = 0; v < 4; v++) {
      const int t = lo + c * CH + 4 * g + v;
      V[v] = t < hi ? (float)vp[(size_t)t * ld] : 0.0f;
    }
  };
  fetch_v(0);
  for (int s = 0; s < 3; s++) step_barrier();
  for (int c = 0; c < n; c++) {
    const ChunkOps& o = ops[c & 1];
    const int t0 = lo + c * CH;
    const f4 Vc = V;
    float zero = 0.0f;
#pragma unroll
    for (int v = 0; v < 4; v++) {
      zero = __builtin_fmaf(Vc[v], 0.0f, zero);
#pragma unroll
      for (int j = 0; j < 4; j++) zero = __builtin_fmaf(S[j][v], 0.0f, zero);
    }
    if (c + 1 < n) fetch_v(c + 1);
    if (!o.bad && __ballot(!(zero == 0.0f)) == 0) {
      f4 u = {0, 0, 0, 0}, y = u;
      const int at = l16 * LDT + 4 * g;
      u = mma4(*reinterpret_cast<const f4*>(&o.mk[at]), Vc, u);
      y = mma4(*reinterpret_cast<const f4*>(&o.nk[at]), Vc, y);
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const f4 ah = *reinterpret_cast<const f4*>(&o.ah[l16 * LDR + 16 * j + 4 * g]);
        const f4 rh = *reinterpret_cast<const f4*>(&o.rh[l16 * LDR + 16 * j + 4 * g]);
#pragma unroll
        for (int v = 0; v < 4; v++) {
          u = __builtin_amdgcn_mfma_f32_16x16x4f32(ah[v], S[j][v], u, 0, 0, 0);
          y = __builtin_amdgcn_mfma_f32_16x16x4f32(rh[v], S[j][v], y, 0, 0, 0);
        }
      }
      const f4 zeros = {0, 0, 0, 0};
      const f4 U = mma4(*reinterpret_cast<const f4*>(&o.x[at]), u, zeros);
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const f4 pc = *reinterpret_cast<const f4*>(&o.pc[16 * j + 4 * g]);
#pragma unroll
        for (int v = 0; v < 4; v++) S[j][v] *= pc[v];
        const int key = (16 * j + l16) * LDT + 4 * g;
        S[j] = mma4(*reinterpret_cast<const f4*>(&o.kcT[key]), Vc, S[j]);
        S[j] = mma4(*reinterpret_cast<const f4*>(&o.bcT[key]), U, S[j]);
      }
      y = mma4(*reinterpret_cast<const f4*>(&o.nb[at]), U, y);
#pragma unroll
      for (int v = 0; v < 4; v++) {
        const int t = t0 + 4 * g + v;
        if (t < hi) yp[(size_t)t * ld] = y[v];
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

template <typename T>
void launch(const WkvArgs& a, hipStream_t s) {
  if (a.T - a.sequences < 32) {
    hipLaunchKernelGGL((k_wkv_seq<T>), dim3(a.sequences, a.H), dim3(256), 0, s, a);
  } else if ((long long)a.sequences * a.H >= 256) {
    hipLaunchKernelGGL((k_wkv_chunk<T, 4>), dim3(a.sequences, a.H), dim3(64 * 7), 0, s, a);
  } else {
    hipLaunchKernelGGL((k_wkv_chunk<T, 1>), dim3(a.sequences, a.H * 4), dim3(64 * 4), 0, s, a);
  }
}

}  // namespace

hipError_t launch_wkv(const WkvArgs& a, hipStream_t s) {
  if (a.half) launch<_Float16>(a, s);
  else launch<float>(a, s);
  return hipGetLastError();
}

}  // namespace rq
