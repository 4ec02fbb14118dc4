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
// head and token against 36864 flops; 64 requests, 64 heads: 142 MB in 22 us,
// part of it from the last-level cache), by the latency of the two row sums
// where they are long (4096 tokens, 64 heads: 3025 us, 1770 cycles a token).
template <typename T>
__global__ void __launch_bounds__(256)
k_wkv_seq(const WkvArgs a, int below) {
  const int q = blockIdx.x / a.H, h = blockIdx.x % a.H;
  const int lo = max(a.offsets[q], 0), hi = min(a.offsets[q + 1], a.T);
  if (lo >= hi || hi - lo >= below) return;
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
// below 2^-22 of an operand, or 2^-36 where the operand is under 2^-14, and three
// binary16 instructions stand for eight binary32 ones (over 32 terms; measured
// against those: 64 heads of 4096 tokens in 16 sequences 241 -> 184 us).  The
// state itself, the decays, the triangular inverse and everything added up stay
// binary32.
//
// So that 2^-36 is small beside what a result is made of, operands have powers of
// two of their own: r and k per token, their largest key to [8, 16) (before the
// decays: W below is then as even over the tokens as v and k are, and the products
// of a q and an earlier k stay within 2^14), and S, W and U per value row (the
// recurrence is linear in a row; the k's power goes to v, W_s = 2^e_s v_s, the r's
// and the row's to y).  A key of r or k counts to 2^-32 of the token's largest, a
// state entry to 2^-26 of its row's largest or better; a and b need none while b is at most 256, as what they add to the
// state is a multiple of the state.  That leaves a value row whose state is small
// beside its W.  It is sound as long as the chunk's first W in the row is not (every
// y and the state then contain it), or every W that is not zero is at least 2^-14.
// A chunk with any other such row, a larger b, a value that is not finite or an
// operand of 2^15 or more is done token by token in binary32, and the rows'
// powers are set anew from the state: its largest to [2^7, 2^8), so that it may
// grow 2^7 and shrink 2^17 times until the next chunk of this kind (12 us).  (The
// powers cost 32 multiplications in a producer and 8 in a state wave a chunk, with
// the checks 132 -> 136 us for 4096 tokens in 16 sequences, 64 heads.)
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
// barrier apart; chunk c's operands go through LDS, two buffers in turn.  Six
// producers cut the segments in two.
//
// Bound by the chain of chunks where heads are few: a step is as long as a
// producer's longest segment or the state's chain of five dependent products,
// most of which are instructions issued and the rest their latencies.  One prompt
// of 4096 tokens, 64 heads: 243 us, 2280 cycles a chunk, 472 MB at 1.9 TB/s.  Bound
// by the SIMDs' instruction rate where heads are many (4096 tokens in 16 sequences,
// 64 heads: 136 us).
// ---------------------------------------------------------------------------
constexpr int CH = 16;  // tokens of a chunk
constexpr float UP = 2048.0f, DOWN = 1.0f / 2048.0f;  // the low part's scale
constexpr float HUGE_ = 32768.0f, LARGE_B = 256.0f;
// a row's state and a W are small below these
constexpr float SMALL_ROW = 1.0f / 1024.0f, SMALL_W = 1.0f / 16384.0f;

// Two-part operands: 4 deep (one accumulator tile) and 8 deep (two).
struct P4 {
  h4 hi, lo;
};
struct P8 {
  h8 hi, lo;
};
typedef float f2 __attribute__((ext_vector_type(2)));
typedef int i4 __attribute__((ext_vector_type(4)));
// Two values in two parts.
__device__ __forceinline__ void split2(float x, float y, h2* hi, h2* lo) {
  *hi = __builtin_convertvector(f2{x, y}, h2);
  const f2 back = __builtin_convertvector(*hi, f2);
  *lo = __builtin_convertvector(
      f2{__builtin_fmaf(-UP, back.x, UP * x), __builtin_fmaf(-UP, back.y, UP * y)}, h2);
}
// Of values that are no longer visible as products (pinned, or passed through
// rounded()): the compiler would else round the product behind x to binary16 in
// one step in one place and in two in another, and hi and lo would not belong
// together.
__device__ __forceinline__ P4 split(const f4& x) {
  h2 h0, h1, l0, l1;
  split2(x[0], x[1], &h0, &l0);
  split2(x[2], x[3], &h1, &l1);
  return P4{__builtin_shufflevector(h0, h1, 0, 1, 2, 3),
            __builtin_shufflevector(l0, l1, 0, 1, 2, 3)};
}
__device__ __forceinline__ f4 rounded(f4 x) {
  asm("" : "+v"(x));
  return x;
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
  int exps[2 * CH];  // 2^exps[t] q_t and 2^exps[16 + s] k_s are meant
  int slow;          // token by token
};
// Q and then P_16 of a chunk.  Written in its first segment, as many steps before
// they are read as there are producers, while that many later chunks write theirs:
// a ring of more places than that.
struct alignas(16) ChunkDecays {
  float at[2][HD];
};
constexpr int RING = 8;

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
// the left neighbour's value, `first` in a row's first lane
__device__ __forceinline__ float left_or(float v, float first) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
                                       __builtin_bit_cast(int, first), __builtin_bit_cast(int, v),
                                       0x111, 0xF, 0xF, false));
}
// lane N of the row of 16
template <int N>
__device__ __forceinline__ float row_bcast(float v) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x150 + N, 0xF, 0xF, true));
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

// The value is made here: left alone, the compiler moves work over a barrier to
// where its result is used, into another segment.
template <typename V>
__device__ __forceinline__ void pin(V& v) {
  asm volatile("" : "+v"(v));
}

// A head's rows of a chunk from token t0 on, as a buffer that ends with the
// sequence: reads past the end give zeros (nothing is added), writes there are
// dropped, and the addresses are made on the scalar unit.
template <typename T>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t chunk_rows(const void* x, size_t base, size_t ld,
                                                             int t0, int hi) {
  const int n = min(hi - t0, CH);
  const T* p = static_cast<const T*>(x) + ((size_t)t0 * ld + base);
  const size_t bytes = n > 0 ? ((n - 1) * ld + HD) * sizeof(T) : 0;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(p), 0, (u32)bytes, 0x00020000);
}
template <typename T>
struct Vec4;
template <>
struct Vec4<float> {
  typedef f4 type;
  static __device__ __forceinline__ f4 load(__amdgpu_buffer_rsrc_t r, u32 at) {
    return __builtin_bit_cast(f4, __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0));
  }
  static __device__ __forceinline__ float load1(__amdgpu_buffer_rsrc_t r, u32 at) {
    return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(r, at, 0, 0));
  }
};
template <>
struct Vec4<_Float16> {
  typedef h4 type;
  static __device__ __forceinline__ h4 load(__amdgpu_buffer_rsrc_t r, u32 at) {
    return __builtin_bit_cast(h4, __builtin_amdgcn_raw_buffer_load_b64(r, at, 0, 0));
  }
  static __device__ __forceinline__ _Float16 load1(__amdgpu_buffer_rsrc_t r, u32 at) {
    return __builtin_bit_cast(_Float16, __builtin_amdgcn_raw_buffer_load_b16(r, at, 0, 0));
  }
};

// Inputs of one chunk as a producer lane holds them: token lane mod 16, keys
// 16 jt + 4 (lane / 16) .. + 3.  They stay as they were loaded until they are
// used: a conversion here would wait for them.
template <typename T>
struct ChunkIn {
  typedef typename Vec4<T>::type vec;
  vec w[4], k[4], kap[4], eta[4], r[4];
  __device__ __forceinline__ void load(const WkvArgs& a, size_t base, size_t ld, int t0, int hi,
                                       u32 at) {
    const __amdgpu_buffer_rsrc_t rw = chunk_rows<T>(a.w, base, ld, t0, hi);
    const __amdgpu_buffer_rsrc_t rk = chunk_rows<T>(a.k, base, ld, t0, hi);
    const __amdgpu_buffer_rsrc_t rkap = chunk_rows<T>(a.kappa, base, ld, t0, hi);
    const __amdgpu_buffer_rsrc_t reta = chunk_rows<T>(a.eta, base, ld, t0, hi);
    const __amdgpu_buffer_rsrc_t rr = chunk_rows<T>(a.r, base, ld, t0, hi);
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const u32 to = at + 16 * j * (u32)sizeof(T);
      w[j] = Vec4<T>::load(rw, to);
      k[j] = Vec4<T>::load(rk, to);
      kap[j] = Vec4<T>::load(rkap, to);
      eta[j] = Vec4<T>::load(reta, to);
      r[j] = Vec4<T>::load(rr, to);
    }
  }
  // P of key tile j: the decays' products up to the lane's token (a token past
  // the end does not decay)
  __device__ __forceinline__ f4 decays(int j, bool live) const {
    f4 P;
#pragma unroll
    for (int v = 0; v < 4; v++) P[v] = live ? decay_of((float)w[j][v]) : 1.0f;
    row_scan4(P);
    return P;
  }
};

// V of a chunk as a right operand: tokens 4 g + v of the lane's value row, as
// loaded.
template <typename T>
struct ChunkV {
  T v[4];
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t rows, const u32* at) {
#pragma unroll
    for (int i = 0; i < 4; i++) v[i] = Vec4<T>::load1(rows, at[i]);
  }
  // v[i] 2^e[i], into registers of its own (an operation the compiler does not
  // see through): the next load takes these, or it would move them at the loop's
  // end, and wait
  __device__ __forceinline__ f4 get(const i4& e) const {
    f4 r;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const float x = (float)v[i];
      const int ei = e[i];
      float y;
      asm volatile("v_ldexp_f32 %0, %1, %2" : "=v"(y) : "v"(x), "v"(ei));
      r[i] = y;
    }
    return r;
  }
};

// X = I + Mb X by forward substitution, with row t of X in lane t of every row
// of 16 lanes (columns 4 g + v): row T is final once the rows before it have
// been taken off, and one DPP multiply-add per column hands every later row its
// share, mt[T] = Mb[t][T] of the lane's row t (zero for t <= T).  A register is
// read by DPP three instructions after it was written, one more than it has to be.
__device__ __forceinline__ void substitute(const float* mt, f4& x) {
  float a = x[0], b = x[1], c = x[2], d = x[3];
#define RQ_TAKE_OFF(T, m)                                                      \
  "v_fmac_f32_dpp %0, %0, " m " row_newbcast:" #T " row_mask:0xf bank_mask:0xf\n" \
  "v_fmac_f32_dpp %1, %1, " m " row_newbcast:" #T " row_mask:0xf bank_mask:0xf\n" \
  "v_fmac_f32_dpp %2, %2, " m " row_newbcast:" #T " row_mask:0xf bank_mask:0xf\n" \
  "v_fmac_f32_dpp %3, %3, " m " row_newbcast:" #T " row_mask:0xf bank_mask:0xf\n"
  asm("s_nop 1\n" RQ_TAKE_OFF(0, "%4") RQ_TAKE_OFF(1, "%5") RQ_TAKE_OFF(2, "%6")
      RQ_TAKE_OFF(3, "%7") RQ_TAKE_OFF(4, "%8") RQ_TAKE_OFF(5, "%9") RQ_TAKE_OFF(6, "%10")
      RQ_TAKE_OFF(7, "%11") RQ_TAKE_OFF(8, "%12") RQ_TAKE_OFF(9, "%13") RQ_TAKE_OFF(10, "%14")
      RQ_TAKE_OFF(11, "%15") RQ_TAKE_OFF(12, "%16") RQ_TAKE_OFF(13, "%17")
      RQ_TAKE_OFF(14, "%18") "s_nop 1\n"
      : "+v"(a), "+v"(b), "+v"(c), "+v"(d)
      : "v"(mt[0]), "v"(mt[1]), "v"(mt[2]), "v"(mt[3]), "v"(mt[4]), "v"(mt[5]), "v"(mt[6]),
        "v"(mt[7]), "v"(mt[8]), "v"(mt[9]), "v"(mt[10]), "v"(mt[11]), "v"(mt[12]), "v"(mt[13]),
        "v"(mt[14]));
#undef RQ_TAKE_OFF
  x = f4{a, b, c, d};
}
// m: Mb transposed, as an accumulator (rows s = 4 g + v, columns t = lane mod
// 16).  Returns X, row t in lane t, columns 4 g + v.
__device__ __forceinline__ f4 inverse(const f4& m) {
  const int lane = threadIdx.x & 63, l16 = lane & 15, g = lane >> 4;
  float mt[CH];  // Mb[t][T] for all T: the other lane rows' values
#pragma unroll
  for (int v = 0; v < 4; v++) {
    const float mv = m[v];
    const u32 u = __builtin_bit_cast(u32, mv);
    const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);  // rows 0 0 2 2, 1 1 3 3
    const u32 a0 = a[0], a1 = a[1];
    const auto b = __builtin_amdgcn_permlane32_swap(a0, a0, false, false);  // row 0, row 2
    const auto c = __builtin_amdgcn_permlane32_swap(a1, a1, false, false);  // row 1, row 3
    const u32 b0 = b[0], b1 = b[1], c0 = c[0], c1 = c[1];
    mt[v] = __builtin_bit_cast(float, b0);
    mt[4 + v] = __builtin_bit_cast(float, c0);
    mt[8 + v] = __builtin_bit_cast(float, b1);
    mt[12 + v] = __builtin_bit_cast(float, c1);
  }
  f4 x;
#pragma unroll
  for (int v = 0; v < 4; v++) x[v] = l16 == 4 * g + v ? 1.0f : 0.0f;
  substitute(mt, x);
  return x;
}

__device__ __forceinline__ float larger(float m, const f4& x) {
#pragma unroll
  for (int i = 0; i < 4; i++) m = fmaxf(m, fabsf(x[i]));
  return m;
}
__device__ __forceinline__ float largest(const f4* x) {
  return larger(larger(larger(larger(0.0f, x[0]), x[1]), x[2]), x[3]);
}
// The largest of the four lanes 16 apart, of values that are not negative (a
// NaN is the largest).
__device__ __forceinline__ float over_groups(float m) {
  const u32 u = __builtin_bit_cast(u32, m);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const u32 a0 = a[0], a1 = a[1], b = max(a0, a1);
  const auto c = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  const u32 c0 = c[0], c1 = c[1];
  return __builtin_bit_cast(float, max(c0, c1));
}
// What the lane's row of 16 lanes holds in the first one of the four.
__device__ __forceinline__ float of_first_group(float m) {
  const u32 u = __builtin_bit_cast(u32, m);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const u32 a0 = a[0];
  const auto c = __builtin_amdgcn_permlane32_swap(a0, a0, false, false);
  const u32 c0 = c[0];
  return __builtin_bit_cast(float, c0);
}
// m = max(m, |x|, |y|), of values as loaded (which fmaxf would quieten first)
__device__ __forceinline__ void take_larger(float& m, float x, float y) {
  asm("v_max3_f32 %0, %0, |%1|, |%2|" : "+v"(m) : "v"(x), "v"(y));
}
// The exponent that brings a magnitude to [2^(e-1), 2^e) (any for zero,
// infinities and NaN).
__device__ __forceinline__ int exponent_to(int e, float m) {
  return e - __builtin_amdgcn_frexp_expf(m);
}
__device__ __forceinline__ f4 scaled(const f4& x, int e) {
  return f4{ldexpf(x[0], e), ldexpf(x[1], e), ldexpf(x[2], e), ldexpf(x[3], e)};
}
// Position of |x| in the order of the magnitudes that are not zero; zero is last.
__device__ __forceinline__ u32 order_not_zero(float x) {
  return (__builtin_bit_cast(u32, x) << 1) - 1u;
}

// SCALE_LATE: the scaling of q and k goes to segment 2, as segment 1 is else the
// longest of three (1531 ragged tokens, 40 heads, binary16 62.8 -> 59.9 us; 256
// tokens, 64 heads, binary32 23.5 -> 22.7).  With four state waves on the same
// SIMDs only conversions make it so (in binary32 63.0 -> 63.7 us; 4096 tokens of 16
// sequences, 64 heads 135.8 -> 138.4).
template <typename T, int PRODUCERS, bool SCALE_LATE>
__device__ __forceinline__ void produce(const WkvArgs& a, ChunkOps* ops, ChunkDecays* decays,
                                        int p, int lo, int hi, size_t base, size_t ld) {
  const int lane = threadIdx.x & 63, l16 = lane & 15, g = lane >> 4;
  const int n = (hi - lo + CH - 1) / CH;
  ChunkIn<T> in;
  const auto live = [&](int c) { return lo + c * CH + l16 < hi; };
  const u32 at = (u32)((l16 * ld + 4 * g) * sizeof(T));
  const auto fetch = [&](int c) { in.load(a, base, ld, lo + c * CH, hi, at); };
  h4 identity;
#pragma unroll
  for (int v = 0; v < 4; v++) identity[v] = l16 == 4 * g + v ? (_Float16)1.0f : (_Float16)0.0f;
  const auto half_barrier = [] {
    if constexpr (PRODUCERS == 6) step_barrier();
  };
  f4 P[4];
  fetch(p);
  P[0] = in.decays(0, live(p));
  P[1] = in.decays(1, live(p));
  int steps = p;
  for (int i = 0; i < p; i++) step_barrier();
  for (int c = p; c < n; c += PRODUCERS) {
    // segment 1: decays (half of them were made in the last segment of the
    // chunk before, so that the segments are of about one length) and the scaled
    // operands
    f4 av[4], qv[4], bv[4], kv[4], rest[4];  // rest: P_16 / Q
    P[2] = in.decays(2, live(c));
    P[3] = in.decays(3, live(c));
    float big_r = 0.0f, big_k = 0.0f;
    const auto scale = [&](int j) {
      take_larger(big_r, (float)in.r[j][0], (float)in.r[j][1]);
      take_larger(big_r, (float)in.r[j][2], (float)in.r[j][3]);
      take_larger(big_k, (float)in.k[j][0], (float)in.k[j][1]);
      take_larger(big_k, (float)in.k[j][2], (float)in.k[j][3]);
#pragma unroll
      for (int v = 0; v < 4; v++) {
        const float kap = (float)in.kap[j][v], k = (float)in.k[j][v], r = (float)in.r[j][v];
        const float pv = P[j][v];
        const float inv = __builtin_amdgcn_rcpf(pv);
        const float over = row_bcast<7>(inv);  // 1 / Q
        const float rel = pv * over, up = inv * row_bcast<7>(pv);
        rest[j][v] = row_bcast<15>(rel);
        av[j][v] = kap * left_or(rel, over);
        qv[j][v] = r * rel;
        bv[j][v] = -((float)in.eta[j][v] * kap) * up;
        kv[j][v] = k * up;
      }
      // Q is token 7's P, P_16 token 15's
      if ((l16 & 7) == 7)
        *reinterpret_cast<f4*>(&decays[c & (RING - 1)].at[l16 >> 3][16 * j + 4 * g]) = P[j];
    };
    // a token's largest r and k to [8, 16)
    int up_r, up_k;
    bool slow;
    const auto even_out = [&] {
      up_r = exponent_to(4, over_groups(big_r));
      up_k = exponent_to(4, over_groups(big_k));
#pragma unroll
      for (int j = 0; j < 4; j++) {
        qv[j] = scaled(qv[j], up_r);
        kv[j] = scaled(kv[j], up_k);
        pin(qv[j]), pin(kv[j]);
      }
      slow = __ballot(largest(bv) > LARGE_B) != 0;
    };
#pragma unroll
    for (int j = 0; j < 4; j++) {
      scale(j);
      pin(av[j]), pin(qv[j]), pin(bv[j]), pin(kv[j]), pin(rest[j]);
      if (j == 1) half_barrier();
    }
    if constexpr (!SCALE_LATE) even_out();
    // two steps ahead of their use, into the registers that are free by now
    // (the operands are made before, not after; past the end too, as a branch here
    // would make the compiler wait for the loads to move them)
    __builtin_amdgcn_sched_barrier(0);
    fetch(c + PRODUCERS);
    step_barrier();
    // segment 2: the four products' transposes, rows s = 4 g + v, columns t =
    // lane mod 16, and kc and bc turned from tokens x keys to keys x tokens by
    // products with the identity, which are exact
    if constexpr (SCALE_LATE) even_out();
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
    f4 mbv = mb.value(), mkv = mk.value(), nbv = nb.value(), nkv = nk.value();
    pin(mbv), pin(mkv), pin(nbv), pin(nkv);
    half_barrier();
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const P4 kp = split(rounded(kv[j] * rest[j])), bp = split(rounded(bv[j] * rest[j]));
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
#pragma unroll
    for (int j = 0; j < 4; j++) pin(kb[j].hi), pin(kb[j].lo);
    step_barrier();
    // segment 3: the triangular inverse, and everything to the chunk's buffer
    ChunkOps& o = ops[c & 1];
    const auto put = [&] {
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
    };
    if constexpr (PRODUCERS == 3) put();
    // a value that is not finite, or too large for an operand, leaves none of
    // its row's or column's sums finite
    float zero = 0.0f;
    f4 mbt, mkt, nbt, nkt;
#pragma unroll
    for (int v = 0; v < 4; v++) {
      zero = __builtin_fmaf(mbv[v], 0.0f, __builtin_fmaf(mkv[v], 0.0f, zero));
      zero = __builtin_fmaf(nbv[v], 0.0f, __builtin_fmaf(nkv[v], 0.0f, zero));
      const bool before = 4 * g + v < l16, upto = 4 * g + v <= l16;
      mbt[v] = before ? mbv[v] : 0.0f;
      mkt[v] = before ? mkv[v] : 0.0f;
      nbt[v] = upto ? nbv[v] : 0.0f;
      nkt[v] = upto ? nkv[v] : 0.0f;
    }
    f4 x = inverse(mbt);
    if constexpr (PRODUCERS == 6) {
      pin(x), pin(mkt), pin(nbt), pin(nkt);
      step_barrier();
      put();
    }
    const float big = larger(larger(larger(larger(0.0f, x), mkt), nbt), nkt);
    slow = slow || __ballot(!(zero == 0.0f) || !(big < HUGE_)) != 0;
    const P4 xp = split(x), mkp = split(mkt), nbp = split(nbt), nkp = split(nkt);
    o.x[0][lane] = xp.hi;
    o.x[1][lane] = xp.lo;
    o.mk[0][lane] = mkp.hi;
    o.mk[1][lane] = mkp.lo;
    o.nb[0][lane] = nbp.hi;
    o.nb[1][lane] = nbp.lo;
    o.nk[0][lane] = nkp.hi;
    o.nk[1][lane] = nkp.lo;
    if (lane < 2 * CH) o.exps[lane] = g == 0 ? -up_r : -up_k;
    if (lane == 0) o.slow = slow;
#pragma unroll
    for (int j = 0; j < 2; j++) {
      P[j] = in.decays(j, live(c + PRODUCERS));
      pin(P[j]);
    }
    step_barrier();
    steps += PRODUCERS;
  }
  for (; steps < n + PRODUCERS; steps++) step_barrier();
}

template <typename T, int NR, int PRODUCERS>
__global__ void __launch_bounds__(64 * (NR + PRODUCERS), 2)
k_wkv_chunk(const WkvArgs a, int from) {
  __shared__ ChunkOps ops[2];
  __shared__ ChunkDecays decays[RING];
  static_assert(RING > PRODUCERS && (RING & (RING - 1)) == 0, "chunks c % RING in turn");
  // heads are the fast index: a sequence's workgroups go to all XCDs, a head's
  // (they read the same inputs) to one
  constexpr int TILES = 4 / NR;
  const int b = blockIdx.x, hd = b / (8 * TILES) * 8 + b % 8, tile = b / 8 % TILES;
  if (hd >= a.sequences * a.H) return;
  const int sq = hd / a.H, h = hd % a.H;
  const int lo = max(a.offsets[sq], 0), hi = min(a.offsets[sq + 1], a.T);
  if (lo >= hi || hi - lo < from) return;
  const int n = (hi - lo + CH - 1) / CH;
  const size_t ld = (size_t)a.H * HD, base = (size_t)h * HD;
  // Waves go to the four SIMDs in turn.  Six producers take three of them, two
  // waves each, the state waves the fourth.
  const int nth = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool producer = PRODUCERS == 6 ? nth % 4 != 3 : nth >= NR;
  if (producer) {
    // where a producer shares a SIMD with a state wave, it is the later one (1531
    // ragged tokens, 40 heads: 64 -> 60 us)
    if (PRODUCERS == 3) __builtin_amdgcn_s_setprio(1);
    constexpr bool LATE = PRODUCERS == 3 && (sizeof(T) == 2 || NR < 4);
    produce<T, PRODUCERS, LATE>(a, ops, decays, PRODUCERS == 6 ? nth - nth / 4 : nth - NR, lo, hi,
                                base, ld);
    return;
  }
  const int wave = PRODUCERS == 6 ? nth / 4 : nth;
  const int lane = threadIdx.x & 63, l16 = lane & 15, g = lane >> 4;
  const int i = 16 * (tile * NR + wave % NR) + l16;  // the lane's value row
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
  u32 vat[4], yat[4];  // of tokens 4 g + v in a chunk's rows
#pragma unroll
  for (int v = 0; v < 4; v++) {
    vat[v] = (u32)(((4 * g + v) * ld + i) * sizeof(T));
    yat[v] = (u32)(((4 * g + v) * ld + i) * sizeof(float));
  }
  // V of the even and the odd chunks, two chunks ahead
  ChunkV<T> even, odd;
  even.load(chunk_rows<T>(a.v, base, ld, lo, hi), vat);
  odd.load(chunk_rows<T>(a.v, base, ld, lo + CH, hi), vat);
  for (int s = 0; s < PRODUCERS; s++) step_barrier();
  // the state has arrived before the loop, so that no wait inside it stands
  // for these loads (and with them for the stores of y)
#pragma unroll
  for (int j = 0; j < 4; j++) pin(S[j]);
  // S, W and U of a value row are held times 2^lift, the row's own
  int lift;
  const auto center = [&](float m) {
    lift = exponent_to(8, over_groups(m));
#pragma unroll
    for (int j = 0; j < 4; j++) S[j] = scaled(S[j], lift);
  };
  {
    const i4 ke = *reinterpret_cast<const i4*>(&ops[0].exps[CH + 4 * g]) + 4;
    center(larger(largest(S), even.get(ke)));  // 16 W beside S: k's keys reach 16
  }
  const auto chunk = [&](int c, ChunkV<T>& vin) {
    const ChunkOps& o = ops[c & 1];
    const int t0 = lo + c * CH;
    // operands in the order of their use (LDS answers in order)
    bool slow = o.slow;
    const i4 re = *reinterpret_cast<const i4*>(&o.exps[4 * g]);
    const i4 ke = *reinterpret_cast<const i4*>(&o.exps[CH + 4 * g]);
    f4 mid[4], end[4];
#pragma unroll
    for (int j = 0; j < 4; j++)
      mid[j] = *reinterpret_cast<const f4*>(&decays[c & (RING - 1)].at[0][16 * j + 4 * g]);
    const P4 mk{o.mk[0][lane], o.mk[1][lane]}, nk{o.nk[0][lane], o.nk[1][lane]};
    P8 ap[2], qp[2], kb[4];
#pragma unroll
    for (int q = 0; q < 2; q++) {
      ap[q] = P8{o.a[0][q][lane], o.a[1][q][lane]};
      qp[q] = P8{o.q[0][q][lane], o.q[1][q][lane]};
    }
    const P4 xp{o.x[0][lane], o.x[1][lane]};
#pragma unroll
    for (int j = 0; j < 4; j++) {
      end[j] = *reinterpret_cast<const f4*>(&decays[c & (RING - 1)].at[1][16 * j + 4 * g]);
      kb[j] = P8{o.kb[0][j][lane], o.kb[1][j][lane]};
    }
    const P4 nb{o.nb[0][lane], o.nb[1][lane]};
    const f4 W = vin.get(ke + lift);
    vin.load(chunk_rows<T>(a.v, base, ld, t0 + 2 * CH, hi), vat);
    f4 Sq[4];
#pragma unroll
    for (int j = 0; j < 4; j++) Sq[j] = rounded(S[j] * mid[j]);
    const float row = over_groups(largest(Sq)), lead = of_first_group(W[0]);
    const u32 least = min(min(order_not_zero(W[0]), order_not_zero(W[1])),
                          min(order_not_zero(W[2]), order_not_zero(W[3])));
    const bool small = row < SMALL_ROW && fabsf(lead) < SMALL_W &&
                       (row > 0.0f || least < order_not_zero(SMALL_W));
    slow = slow || __ballot(small) != 0;
    const P4 vs = split(W);
    // (32 deep beside zeros: a 16-deep instruction's sum is not carried on by a
    // 32-deep one, which, right behind it, took half of the sum for zero)
    const h4 no = {0, 0, 0, 0};
    Sum u = none(), y = u;
    mma(join(mk, P4{no, no}), join(vs, vs), u);
#pragma unroll
    for (int q = 0; q < 2; q++) {
      const P8 sp = join(split(Sq[2 * q]), split(Sq[2 * q + 1]));
      mma(ap[q], sp, u);
      mma(qp[q], sp, y);
    }
    Sum us = none();
    mma(xp, split(rounded(u.value())), us);
    const f4 U = rounded(us.value());
    // what is not finite, or too large for an operand, in W, S or U
    slow = slow || __ballot(!(fabsf(U[0]) + fabsf(U[1]) + fabsf(U[2]) + fabsf(U[3]) < HUGE_)) != 0;
    if (!slow) {
      const P4 up = split(U);
      const P8 vu = join(vs, up);
#pragma unroll
      for (int j = 0; j < 4; j++) {
        Sum s{S[j] * end[j], f4{0, 0, 0, 0}};
        mma(kb[j], vu, s);
        S[j] = s.value();
      }
      mma(join(nk, nb), vu, y);
      const f4 yv = y.value();
      const __amdgpu_buffer_rsrc_t ry = chunk_rows<float>(a.y, base, ld, t0, hi);
#pragma unroll
      for (int v = 0; v < 4; v++) {
        const float yt = ldexpf(yv[v], re[v] - lift);
        __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(u32, yt), ry, yat[v], 0, 0);
      }
    } else {
      // token by token (a value that is not finite must not reach earlier
      // tokens through products with the zeros of the triangular matrices)
#pragma unroll
      for (int j = 0; j < 4; j++) S[j] = scaled(S[j], -lift);
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
      center(largest(S));
    }
    step_barrier();
  };
  // (no way out between the two: on it, the compiler would see the even chunk's
  // loads as the newest ones at the loop's head, and wait for all)
  int c = 0;
  for (; c + 2 <= n; c += 2) {
    chunk(c, even);
    chunk(c + 1, odd);
  }
  if (c < n) chunk(c, even);
  if (stored) {
#pragma unroll
    for (int j = 0; j < 4; j++) *reinterpret_cast<f4*>(st + 16 * j) = scaled(S[j], -lift);
  }
}

template <typename T, int NR, int PRODUCERS>
void launch_chunks(const WkvArgs& a, unsigned heads, int from, hipStream_t s) {
  hipLaunchKernelGGL((k_wkv_chunk<T, NR, PRODUCERS>), dim3((heads + 7) / 8 * 8 * (4 / NR)),
                     dim3(64 * (NR + PRODUCERS)), 0, s, a, from);
}

// Sequences go token by token below a length, in chunks from it on.  Few heads:
// 8 tokens (token by token / chunks: 64 heads, one sequence of 4 tokens 4.5 / 6.6
// us, 8 6.4 / 6.6, 12 8.3 / 6.6); many: 16 (1024 heads, sequences of 8 tokens
// 18 / 26 us, 16 28 / 27; 2048 heads 28 / 48 and 53 / 52 us).
//
// The lengths are on the device.  Where no sequence reaches that length, as all of
// them have a token, or all together have not as many, all go token by token
// (fewer tokens than sequences mean empty ones, and any of the others may be long:
// 255 tokens in one of 256 slots, 64 heads 151 -> 43 us; a second launch for every batch
// of single tokens would cost it 2 to 6 us).  Where sequences have on average more
// than 12 tokens beyond their first, all go in chunks; between the two each kind
// has a launch of its own, which passes over the other's sequences (chunks only /
// both: 64 heads, 31 single tokens before one sequence of 48 52 / 26 us, of 500 93 /
// 70 but behind it 61 / 67; 16 sequences of 8 26 / 20, of 16 27 / 29).
//
// A workgroup of the chunk kernel takes 16, 32 or 64 of a head's value rows.
// Fewer rows make a chunk's step shorter (a state wave then has a SIMD to
// itself), but the producers' work is done again by each of a head's
// workgroups, which pays while there is a compute unit for each of these 4 or 2
// workgroups.  Binary32, 16 / 32 / 64 rows on one card: one prompt of 4096 tokens, 64
// heads 267 / 342 / 365 us, of 256 23.1 / 27.4 / 29.5; of 1000 tokens, 72 heads 134 /
// 90 / 96, 128 heads 135 / 92 / 96, 160 heads 200 / 177 / 102; 4096 tokens in 16
// sequences, 64 heads 354 / 210 / 130.
//
// At 16 rows a SIMD's second wave is free, and six producers keep up with the
// state better than three, but its chain starts three steps later: binary32 inputs
// take six past 512 tokens (64 heads, three / six: 128 tokens 15.5 / 17.0 us, 512
// 40.0 / 40.0, 1024 72.8 / 71.0, 4096 256 / 246).  With binary16 inputs three have
// conversions to do as well, and six always pay.
template <typename T>
void launch(const WkvArgs& a, hipStream_t s) {
  const unsigned heads = (unsigned)a.sequences * a.H;
  const int from = heads <= 128 ? 8 : 16;
  const int extra = a.T - a.sequences;
  const bool all_short = a.T < from || (extra >= 0 && extra + 1 < from);
  const bool all_long = !all_short && (a.sequences == 1 || extra / 12 >= a.sequences);
  if (!all_long)
    hipLaunchKernelGGL((k_wkv_seq<T>), dim3(heads), dim3(256), 0, s, a,
                       all_short ? a.T + 1 : from);
  if (all_short) return;
  const int least = all_long ? 0 : from;
  if (heads <= 64 && (sizeof(T) == 2 || a.T > 512))
    launch_chunks<T, 1, 6>(a, heads, least, s);
  else if (heads <= 64)
    launch_chunks<T, 1, 3>(a, heads, least, s);
  else if (heads <= 128)
    launch_chunks<T, 2, 3>(a, heads, least, s);
  else
    launch_chunks<T, 4, 3>(a, heads, least, s);
}

}  // namespace

hipError_t launch_wkv(const WkvArgs& a, hipStream_t s) {
  if (a.half) launch<_Float16>(a, s);
  else launch<float>(a, s);
  return hipGetLastError();
}

}  // namespace rq
