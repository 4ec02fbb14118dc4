// rq_gemm_fp8.hip -- products of block-scaled E4M3 operands:
//   y[m][n] = y_in[m][n] + sum_b xs[m][b] ws[n/128][b] sum_{k in b} x[m][k] w[n][k].
//
// Few rows are bound by w, a byte a weight from memory; many by the matrix units.
// Times below are of one MI355X, whose memory copies at 5.07 TB/s and whose library
// products reach 3077 TFLOP/s in FP8 and 1434 in binary16.
//
//   k_rows  up to 16 rows: operands from memory straight to registers.  Three
//           products of 4096 x 4096 and one row 9.8 us (50.4 MB: 5.2 TB/s).
//   k_ring  some rows: each wave takes every eighth block of K through LDS of its
//           own.  32 rows, 4096 x 16384: 17.2 us; 203 rows, 2560 x 10240: 22.7.
//   k_tile  many rows: tiles of a workgroup staged through LDS.  61 rows of 65529 x
//           2048, binary32: 32.5 us; 2047 rows of 16384 x 4096, binary32: 262 us.
//   k_big   256 x 256 tiles for binary16 and E4M3 outputs.  2047 rows of 16384 x 4096
//           to E4M3 124 us (2220 TFLOP/s); 4001 rows of 4096 x 4096 59 us (2280 TFLOP/s).
#include "rq_common.h"
#include "rq_fp8.h"
#include "rq_internal.h"

#include <type_traits>
#include <utility>

namespace rq {
namespace {

typedef int i8v __attribute__((ext_vector_type(8)));

// How a block of 128 meets:
//   WIDE   widened to binary16 (exact), binary16 matrix instructions, one
//          multiply-add by the scales for each block's sum;
//   FP8S   the FP8 matrix instruction of depth 128, the same multiply-add;
//   FP8E   the FP8 matrix instruction with the power of two as its own scale.
// The FP8 instructions align the products of eight neighbouring k to the largest and
// drop what is 2^-13 of it or less: measured, an error of 1.3e-5 to 4e-5 of the
// 2-norm of y for normal values, with and without a few large channels, and of 5e-5
// for all codes alike.  That is far inside the rounding of binary16 or E4M3 outputs
// (2e-4 and 2.6e-2 of the 2-norm), so those take them, and not inside that of binary32
// outputs, which are WIDE: 1e-8 to 8e-8, at half the rate and a conversion for each
// pair of codes.  A caller chooses between them by the type of its outputs.
enum Mode { WIDE, FP8S, FP8E };

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

// The product of two scales: its binary32 value, or (FP8E) the exponent byte.
template <Mode MODE>
__device__ __forceinline__ u32 joint_scale(u32 a, u32 b, bool e8m0) {
  if constexpr (MODE == FP8E) {
    const int e = (int)a + (int)b - 127;
    return a == 255 || b == 255 ? 255u : (u32)min(max(e, 0), 254);
  } else {
    const float fa = e8m0 ? e8m0_value(a) : __builtin_bit_cast(float, a);
    const float fb = e8m0 ? e8m0_value(b) : __builtin_bit_cast(float, b);
    return __builtin_bit_cast(u32, fa * fb);
  }
}
__device__ __forceinline__ u32 load_scale(const void* s, size_t i, bool e8m0) {
  return e8m0 ? (u32) static_cast<const uint8_t*>(s)[i] : static_cast<const u32*>(s)[i];
}

template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}

__device__ __forceinline__ void lds_copy16(__amdgpu_buffer_rsrc_t r, void* dst, u32 voff, u32 soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)dst, 16,
                                           voff, soff, 0, 0);
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* p) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, -1, 0x00020000);
}

// Work of a launch: tiles of all problems one after another, m fastest, each in
// `splits` ranges of K.
struct Launch {
  int tile0[FP8_BATCH + 1];  // first tile of each problem
  int mt;                    // tiles of M
  int splits;
  unsigned* counters;        // one per wave of a tile, zero between launches
  float* partial;            // [tile][split][outputs of a tile, as the lanes hold them]
};

// WN x WM waves, each 16 TN outputs of 16 TM rows; ST stages of 128 columns.  w is
// the instruction's first operand, so that a lane has four consecutive outputs of a
// row.
template <int WN_, int WM_, int TN_, int TM_, int ST_>
struct Tile {
  static constexpr int WN = WN_, WM = WM_, TN = TN_, TM = TM_, ST = ST_;
  static constexpr int W = WN * WM, THREADS = 64 * W;
  static constexpr int BN = 16 * TN * WN, BM = 16 * TM * WM, NB = BN / 128;
  static constexpr int STAGE = (BN + BM) * 128;
  static constexpr int COPIES = (BN + BM) / 8 / W;  // of a wave for a stage
  static constexpr int WCOPIES = BN / 8 / W;        // of these, rows of w
  static constexpr int SC = 4;                      // blocks of K whose scales are staged together
  static constexpr int SCALES = SC * NB * BM;       // dwords of a buffer of scales
  static constexpr int LDS = ST * STAGE + 2 * SCALES * 4;
  static_assert(BN % 128 == 0 && (BN + BM) / 8 % W == 0 && BN / 8 % W == 0, "whole copies");
  static_assert(LDS <= 160 * 1024, "LDS");
  static constexpr int ROWS = THREADS / BM > 0 ? THREADS / BM : 1;  // blocks staged at once
  static constexpr int PER = SC > ROWS ? SC / ROWS : 1;             // scales of x of a thread
  static_assert(THREADS % BM == 0 && (SC % ROWS == 0 || ROWS % SC == 0), "scales");
};

union Op {
  u32x4 q[2];
  i8v v;
};

// acc += (a block's products of TN x TM tiles of widened operands) * f, the chains
// of several tiles side by side: a product waits for the one before it in its chain.
template <int TN, int TM>
__device__ __forceinline__ void multiply_wide(const h8 (&w)[TN][2][2], const h8 (&x)[TM][2][2],
                                              const float (&f)[TM], f4 (&acc)[TN][TM]) {
  f4 v[TN][TM];
#pragma unroll
  for (int t = 0; t < TN; t++)
#pragma unroll
    for (int j = 0; j < TM; j++) v[t][j] = f4{0, 0, 0, 0};
#pragma unroll
  for (int q = 0; q < 2; q++)
#pragma unroll
    for (int e = 0; e < 2; e++)
#pragma unroll
      for (int t = 0; t < TN; t++)
#pragma unroll
        for (int j = 0; j < TM; j++)
          v[t][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w[t][q][e], x[j][q][e], v[t][j], 0, 0, 0);
#pragma unroll
  for (int t = 0; t < TN; t++)
#pragma unroll
    for (int j = 0; j < TM; j++)
#pragma unroll
      for (int i = 0; i < 4; i++) acc[t][j][i] = __builtin_fmaf(v[t][j][i], f[j], acc[t][j][i]);
}

// The same for TN tiles of w in LDS from `w` on, G at once.
template <int TN, int TM>
__device__ __forceinline__ void multiply_wide(const char* wl, int o0, int o1,
                                              const h8 (&x)[TM][2][2], const float (&f)[TM],
                                              f4 (&acc)[TN][TM]) {
  constexpr int G = TM >= 4 || TN < 2 ? 1 : 2;
#pragma unroll
  for (int t = 0; t < TN; t += G) {
    h8 w[G][2][2];
    f4 part[G][TM];
#pragma unroll
    for (int g = 0; g < G; g++) {
      widen(*reinterpret_cast<const u32x4*>(wl + (t + g) * 2048 + o0), w[g][0]);
      widen(*reinterpret_cast<const u32x4*>(wl + (t + g) * 2048 + o1), w[g][1]);
#pragma unroll
      for (int j = 0; j < TM; j++) part[g][j] = acc[t + g][j];
    }
    multiply_wide<G, TM>(w, x, f, part);
#pragma unroll
    for (int g = 0; g < G; g++)
#pragma unroll
      for (int j = 0; j < TM; j++) acc[t + g][j] = part[g][j];
  }
}

// The products of one block of K from a stage in LDS.
template <typename T, Mode MODE>
__device__ __forceinline__ void multiply(const char* stage, const u32* scales, int wn, int wm,
                                         f4 (&acc)[T::TN][T::TM]) {
  constexpr int TN = T::TN, TM = T::TM;
  const int lane = threadIdx.x & 63, r = lane & 15, h = lane >> 4;
  // chunk 4 p + h of a row, in the slot its row's last bits exchange it to
  const int o0 = r * 128 + ((h ^ (r & 7)) << 4), o1 = r * 128 + (((4 + h) ^ (r & 7)) << 4);
  const char* wp = stage + wn * TN * 16 * 128;
  const char* xp = stage + T::BN * 128 + wm * TM * 16 * 128;
  u32 s[TM];
#pragma unroll
  for (int j = 0; j < TM; j++)
    s[j] = scales[wn * TN / 8 * T::BM + (wm * TM + j) * 16 + r];
  if constexpr (MODE == WIDE) {
    h8 x[TM][2][2];
#pragma unroll
    for (int j = 0; j < TM; j++) {
      widen(*reinterpret_cast<const u32x4*>(xp + j * 2048 + o0), x[j][0]);
      widen(*reinterpret_cast<const u32x4*>(xp + j * 2048 + o1), x[j][1]);
    }
    float f[TM];
#pragma unroll
    for (int j = 0; j < TM; j++) f[j] = __builtin_bit_cast(float, s[j]);
    multiply_wide<TN, TM>(wp, o0, o1, x, f, acc);
  } else {
    Op x[TM];
#pragma unroll
    for (int j = 0; j < TM; j++) {
      x[j].q[0] = *reinterpret_cast<const u32x4*>(xp + j * 2048 + o0);
      x[j].q[1] = *reinterpret_cast<const u32x4*>(xp + j * 2048 + o1);
    }
#pragma unroll
    for (int t = 0; t < TN; t++) {
      Op w;
      w.q[0] = *reinterpret_cast<const u32x4*>(wp + t * 2048 + o0);
      w.q[1] = *reinterpret_cast<const u32x4*>(wp + t * 2048 + o1);
#pragma unroll
      for (int j = 0; j < TM; j++) {
        if constexpr (MODE == FP8E) {
          acc[t][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              w.v, x[j].v, acc[t][j], 0, 0, 0, 127, 0, (int)s[j]);
        } else {
          const f4 z = {0, 0, 0, 0};
          const f4 d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w.v, x[j].v, z, 0, 0, 0, 127,
                                                                       0, 127);
          const float f = __builtin_bit_cast(float, s[j]);
#pragma unroll
          for (int i = 0; i < 4; i++) acc[t][j][i] = __builtin_fmaf(d[i], f, acc[t][j][i]);
        }
      }
    }
  }
}

// Four consecutive outputs of row m.  Rows of any N are whole numbers of dwords in
// binary32, and of even N in binary16, and a store of several dwords needs the
// alignment of one.  (61 rows of 65529 outputs: 33.9 us, a dword at a time 38.9.)
typedef float f4_dword __attribute__((ext_vector_type(4), aligned(4)));
typedef _Float16 h4_dword __attribute__((ext_vector_type(4), aligned(4)));
__device__ __forceinline__ void store4(const Fp8Problem& p, int out, size_t m, int n, f4 v) {
  const size_t at = m * p.N + n;
  if (out == OUT_F32) {
    float* y = static_cast<float*>(p.y) + at;
    if (n + 4 <= p.N) {
      if (p.y_in) v = *reinterpret_cast<const f4_dword*>(p.y_in + at) + v;
      *reinterpret_cast<f4_dword*>(y) = v;
    } else {
#pragma unroll
      for (int i = 0; i < 4; i++)
        if (n + i < p.N) y[i] = p.y_in ? p.y_in[at + i] + v[i] : v[i];
    }
  } else {
    _Float16* y = static_cast<_Float16*>(p.y) + at;
    const h4 o = {(_Float16)v[0], (_Float16)v[1], (_Float16)v[2], (_Float16)v[3]};
    if (p.N % 2 == 0 && n + 4 <= p.N) {
      *reinterpret_cast<h4_dword*>(y) = o;
    } else {
#pragma unroll
      for (int i = 0; i < 4; i++)
        if (n + i < p.N) y[i] = o[i];
    }
  }
}

// f(0), f(1), ... with constants.
template <typename F, int... I>
__device__ __forceinline__ void each_of(F f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void each(F f) {
  each_of(f, std::make_integer_sequence<int, N>{});
}

// Dword i of quarter h of the wave <-> dword h of quarter i.
__device__ __forceinline__ void transpose4(u32 (&v)[4]) { span_fix<4>(v); }

// The largest over the four quarters of the wave.
__device__ __forceinline__ float quarters_max(float v) {
  u32 a = __builtin_bit_cast(u32, v), b = a;
  lane_swap16(a, b);
  v = fmaxf(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b));
  a = b = __builtin_bit_cast(u32, v);
  lane_swap32(a, b);
  return fmaxf(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b));
}

// C rows' blocks of 128 outputs, each spread over four lanes (outputs 16 t + 4 h +
// i), as E4M3 codes of their binary16 values: c[j][t] is tile t's dword of row j,
// se[j] the biased exponent of its scale.  All rows together, so that a lone wave
// has independent work.
constexpr int TB = 8;  // tiles of a block of outputs
template <int C>
__device__ __forceinline__ void quantize_rows(const f4 (&acc)[TB][C], bool square, u32 (&c)[C][TB],
                                              u32 (&se)[C]) {
  h2 z[C][2 * TB];
  const h2 zero = {0, 0};
  h2 odd = zero;  // NaN once a value is not finite
  float top[C];
#pragma unroll
  for (int j = 0; j < C; j++) {
    h2 most = zero;
#pragma unroll
    for (int t = 0; t < TB; t++)
#pragma unroll
      for (int q = 0; q < 2; q++) {
        const h2 v = {(_Float16)acc[t][j][2 * q], (_Float16)acc[t][j][2 * q + 1]};
        odd = __builtin_elementwise_fma(v, zero, odd);
        z[j][2 * t + q] = square ? __builtin_elementwise_max(v, zero) : v;
        most = __builtin_elementwise_max(most, square ? z[j][2 * t + q] : as_h2(as_u32(v) & 0x7FFF7FFFu));
      }
    top[j] = quarters_max(fmaxf((float)most[0], (float)most[1]));
    // squares grow with what is squared, so the largest is the largest one's
    if (square) top[j] *= top[j];
  }
  if (__builtin_expect(__any(odd[0] != odd[0] || odd[1] != odd[1]), 0)) {
    // the largest finite one, and NaN as it is
#pragma unroll
    for (int j = 0; j < C; j++) {
      u32 most = 0;
#pragma unroll
      for (int t = 0; t < TB; t++)
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const _Float16 v = (_Float16)acc[t][j][i];
          z[j][2 * t + i / 2][i & 1] = square && v < (_Float16)0 ? (_Float16)0 : v;
          const float f = square ? relu2((float)v) : (float)v;
          most = max(most, abs_bits(f) < INF_BITS ? abs_bits(f) : 0u);
        }
      top[j] = quarters_max(__builtin_bit_cast(float, most));
    }
  }
#pragma unroll
  for (int j = 0; j < C; j++) {
    se[j] = scale_exponent(__builtin_bit_cast(u32, top[j]) & 0x7FFFFFFFu);
    const float inv = pow2_bits(254 - se[j]);
#pragma unroll
    for (int t = 0; t < TB; t++) {
      float f[4];
#pragma unroll
      for (int i = 0; i < 4; i++) {
        f[i] = (float)z[j][2 * t + i / 2][i & 1];
        if (square) f[i] *= f[i];
      }
      c[j][t] = e4m3x4(f[0], f[1], f[2], f[3], inv);
    }
  }
}

// A wave's 128 outputs of its rows.  Lane l holds rows 16 j + l % 16 and outputs
// 16 t + 4 (l / 16) + i; exchanges between the quarters of the wave make whole
// 16-byte stores of binary16 and E4M3 outputs.
template <int TM>
__device__ __forceinline__ void store_tile(const Fp8Args& a, const Fp8Problem& p, int n0, size_t m0,
                                           const f4 (&acc)[TB][TM]) {
  const int lane = threadIdx.x & 63, r = lane & 15, h = lane >> 4;
  if (a.out == OUT_E4M3) {
    constexpr int C = TM < 2 ? TM : 2;
    each<TM / C>([&](auto part) {
      constexpr int j0 = decltype(part)::value * C;
      f4 rows[TB][C];
      u32 c[C][TB], se[C];
#pragma unroll
      for (int t = 0; t < TB; t++)
#pragma unroll
        for (int j = 0; j < C; j++) rows[t][j] = acc[t][j0 + j];
      quantize_rows<C>(rows, a.relu2, c, se);
#pragma unroll
      for (int j = 0; j < C; j++) {
        const size_t m = m0 + 16 * (j0 + j) + r;
        const bool in = m < (size_t)a.M && n0 < p.N;
#pragma unroll
        for (int g = 0; g < TB / 4; g++) {
          u32 v[4] = {c[j][4 * g], c[j][4 * g + 1], c[j][4 * g + 2], c[j][4 * g + 3]};
          transpose4(v);
          if (in)
            *reinterpret_cast<u32x4*>(static_cast<uint8_t*>(p.y) + m * p.N + n0 + 64 * g + 16 * h) =
                u32x4{v[0], v[1], v[2], v[3]};
        }
        if (in && h == 0) store_scale(p.ys, m * (p.N / 128) + n0 / 128, se[j], a.e8m0);
      }
    });
    return;
  }
  each<TM>([&](auto column) {
    constexpr int j = decltype(column)::value;
    const size_t m = m0 + 16 * j + r;
    const bool in = m < (size_t)a.M && n0 < p.N;
    if (a.out == OUT_F16 && p.N % 8 == 0) {
#pragma unroll
      for (int g = 0; g < TB / 4; g++) {
        u32 v[2][4];
#pragma unroll
        for (int t = 0; t < 4; t++)
#pragma unroll
          for (int q = 0; q < 2; q++) {
            const f4 d = acc[4 * g + t][j];
            v[q][t] = as_u32(h2{(_Float16)d[2 * q], (_Float16)d[2 * q + 1]});
          }
        transpose4(v[0]);
        transpose4(v[1]);
        const int n = n0 + 64 * g + 16 * h;
        u32x4* y = reinterpret_cast<u32x4*>(static_cast<_Float16*>(p.y) + m * p.N + n);
        if (in && n < p.N) y[0] = u32x4{v[0][0], v[1][0], v[0][1], v[1][1]};
        if (in && n + 8 < p.N) y[1] = u32x4{v[0][2], v[1][2], v[0][3], v[1][3]};
      }
    } else if (in) {
#pragma unroll
      for (int t = 0; t < TB; t++) store4(p, a.out, m, n0 + 16 * t + 4 * h, acc[t][j]);
    }
  });
}

// A workgroup's tile and range of K.
struct Where {
  int problem, tile, split, n0, b0, steps;
  size_t m0;
};
__device__ __forceinline__ Where where(const Fp8Args& a, const Launch& l, int bn, int bm) {
  // every XCD (workgroups go to them in turn) takes a run of neighbouring tiles,
  // which share rows of x and w in its L2
  const u32 total = gridDim.x, xcd = blockIdx.x & 7, each = total >> 3, more = total & 7;
  const u32 id = xcd * each + min(xcd, more) + (blockIdx.x >> 3);
  Where o;
  o.split = id % l.splits;
  o.tile = id / l.splits;
  o.problem = 0;
  while (o.problem + 1 < a.count && o.tile >= l.tile0[o.problem + 1]) o.problem++;
  const int at = o.tile - l.tile0[o.problem], KB = a.p[o.problem].K / 128;
  o.n0 = at / l.mt * bn;
  o.m0 = (size_t)(at % l.mt) * bm;
  o.b0 = (int)((long long)KB * o.split / l.splits);
  o.steps = (int)((long long)KB * (o.split + 1) / l.splits) - o.b0;
  return o;
}

template <typename V>
__device__ __forceinline__ void pin(V& v) {
  asm volatile("" : "+v"(v));
}

// End of a phase or step (loads of later ones stay in flight): this wave's LDS
// accesses are done, then everybody's.
__device__ __forceinline__ void phase_end() {
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (0 << 8) | (3 << 14));
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// Many rows: a ring of ST stages that all waves copy into (memory to LDS, nothing
// through registers) and read; one barrier a step.  The scales of SC blocks are
// multiplied together once for a row and 128 outputs and wait in LDS too.  Two
// workgroups share a compute unit, so one multiplies while the other is at its
// barrier or its outputs: a tile twice as wide, alone on its compute unit, gains 2%
// at K = 16384 and loses 5 to 40% at K = 4096 and below.
template <typename T, Mode MODE, bool E8>
__global__ void __launch_bounds__(T::THREADS, T::W / 2)
k_tile(const Fp8Args a, const Launch l) {
  constexpr int W = T::W, TN = T::TN, TM = T::TM, ST = T::ST, SC = T::SC;
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  u32* const scales = reinterpret_cast<u32*>(lds + ST * T::STAGE);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave / T::WM, wm = wave % T::WM;

  const Where o = where(a, l, T::BN, T::BM);
  const Fp8Problem& p = a.p[o.problem];
  const int n0 = o.n0, b0 = o.b0, steps = o.steps, split = o.split, tile = o.tile;
  const size_t m0 = o.m0;
  const int KB = p.K / 128, nb = (p.N + 127) / 128;

  // copies of this wave: eight rows of 128 bytes each; slot s of row q holds
  // chunk s ^ (q % 8), so that the reads of 16 rows' equal chunks spread over all
  // banks.  Rows past the end repeat the last one.
  const __amdgpu_buffer_rsrc_t wr = buffer(p.w + (size_t)n0 * p.K + (size_t)b0 * 128);
  const __amdgpu_buffer_rsrc_t xr = buffer(p.x + m0 * p.K + (size_t)b0 * 128);
  const int w_last = p.N - 1 - n0, x_last = (int)min((size_t)a.M - 1 - m0, (size_t)T::BM);
  u32 off[T::COPIES];
#pragma unroll
  for (int c = 0; c < T::COPIES; c++) {
    const int row = (c * W + wave) * 8 + (lane >> 3);
    const int q = c < T::WCOPIES ? min(row, w_last) : min(row - T::BN, x_last);
    off[c] = (u32)q * p.K + (((lane & 7) ^ (lane >> 3)) << 4);
  }
  auto copy = [&](int step) {
    char* dst = lds + step % ST * T::STAGE + wave * 1024;
#pragma unroll
    for (int c = 0; c < T::COPIES; c++)
      lds_copy16(c < T::WCOPIES ? wr : xr, dst + c * W * 1024, off[c], step * 128);
  };

  // scales of SC blocks: thread -> row of x and blocks
  const int srow = tid % T::BM, sblock = tid / T::BM;
  const size_t xs_row = (m0 + min(srow, x_last)) * KB + b0;
  u32 sx[T::PER], sw[T::NB][T::PER];
  auto load_scales = [&](int first) {
#pragma unroll
    for (int i = 0; i < T::PER; i++) {
      const int b = min(first + sblock + i * T::ROWS, steps - 1);
      sx[i] = load_scale(p.xs, xs_row + b, E8);
#pragma unroll
      for (int n = 0; n < T::NB; n++)
        sw[n][i] = load_scale(p.ws, (size_t)min(n0 / 128 + n, nb - 1) * KB + b0 + b, E8);
    }
  };
  auto keep_scales = [&](int buf) {
#pragma unroll
    for (int i = 0; i < T::PER; i++) {
      const int b = sblock + i * T::ROWS;
#pragma unroll
      for (int n = 0; n < T::NB; n++)
        if (b < SC)
          scales[buf * T::SCALES + (b * T::NB + n) * T::BM + srow] =
              joint_scale<MODE>(sx[i], sw[n][i], E8);
    }
  };

  f4 acc[TN][TM];
#pragma unroll
  for (int t = 0; t < TN; t++)
#pragma unroll
    for (int j = 0; j < TM; j++) acc[t][j] = f4{0, 0, 0, 0};

  load_scales(0);
#pragma unroll
  for (int s = 0; s < ST - 1; s++)
    if (s < steps) copy(s);
  keep_scales(0);
  for (int s = 0; s < steps; s++) {
    // the stage has arrived (this wave's copies, then everybody's), and everybody
    // has left the stage that the next copies go to
    if (s + ST - 2 < steps)
      wait_vm<(ST - 2) * T::COPIES>();
    else
      wait_vm<0>();
    phase_end();
    if (s + ST - 1 < steps) copy(s + ST - 1);
    if (s % SC == 0 && s + SC < steps) load_scales(s + SC);
    multiply<T, MODE>(lds + s % ST * T::STAGE,
                      scales + (s / SC & 1) * T::SCALES + s % SC * T::NB * T::BM, wn, wm, acc);
    if (s % SC == SC / 2 && s - s % SC + SC < steps) keep_scales((s / SC & 1) ^ 1);
  }

  const int wave_n0 = n0 + wn * TN * 16;
  const size_t wave_m0 = m0 + wm * TM * 16;
  if (MODE != WIDE && l.splits > 1) {
    // This range's sums, as the lanes hold them, past the caches that other XCDs do
    // not see; then the wave's arrival at its part of the tile.  The last of the
    // ranges' waves to arrive adds them in order, the sums of several ranges asked
    // for together.
    constexpr int PART = T::BN * T::BM, AGENT = 16;  // scope bit of the buffer instructions
    const __amdgpu_buffer_rsrc_t pr = buffer(l.partial + (size_t)tile * l.splits * PART);
    const u32 lane_at = (wave * 256 + lane * 4) * 4;
#pragma unroll
    for (int t = 0; t < TN; t++)
#pragma unroll
      for (int j = 0; j < TM; j++)
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, acc[t][j]), pr,
                                               lane_at + (split * PART + (t * TM + j) * W * 256) * 4, 0,
                                               AGENT);
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    wait_vm<0>();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    unsigned* const counter = l.counters + tile * W + wave;
    unsigned before = 0;
    if (lane == 0)
      before = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (__builtin_amdgcn_readfirstlane(before) != (unsigned)(l.splits - 1)) return;
    if (lane == 0) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
    for (int t = 0; t < TN; t++)
#pragma unroll
      for (int j = 0; j < TM; j++) acc[t][j] = f4{0, 0, 0, 0};
    constexpr int SB = 2;
    for (int q0 = 0; q0 < l.splits; q0 += SB) {
      u32x4 v[SB][TN][TM];
#pragma unroll
      for (int q = 0; q < SB; q++)
#pragma unroll
        for (int t = 0; t < TN; t++)
#pragma unroll
          for (int j = 0; j < TM; j++)
            v[q][t][j] = __builtin_amdgcn_raw_buffer_load_b128(
                pr, lane_at + (min(q0 + q, l.splits - 1) * PART + (t * TM + j) * W * 256) * 4, 0, AGENT);
#pragma unroll
      for (int q = 0; q < SB; q++) {
        if (q0 + q >= l.splits) break;
#pragma unroll
        for (int t = 0; t < TN; t++)
#pragma unroll
          for (int j = 0; j < TM; j++) acc[t][j] += __builtin_bit_cast(f4, v[q][t][j]);
      }
    }
  }
  if constexpr (MODE != WIDE) {
    store_tile<TM>(a, p, wave_n0, wave_m0, acc);
  } else {
    const int r = lane & 15, h = lane >> 4;
#pragma unroll
    for (int j = 0; j < TM; j++) {
      const size_t m = wave_m0 + 16 * j + r;
      if (m < (size_t)a.M) {
#pragma unroll
        for (int t = 0; t < TN; t++) store4(p, OUT_F32, m, wave_n0 + 16 * t + 4 * h, acc[t][j]);
      }
    }
  }
}

// Large tiles: eight waves in two groups that take turns, one reading operands
// from LDS while the other multiplies.  A step (128 columns) is four phases:
// read x and half of w, multiply, read the other half, multiply; the second group
// is one phase behind, so that the matrix units of a SIMD, which has a wave of
// each group, always have work.  (4001 rows of three 2560 x 2560 to binary16: 121 us
// with 128 x 128 tiles and a barrier a step, 89 so.)  256 x 256 because
// a step's 1 us of matrix instructions then hides its 64 KB of copies (137 B/ns) and
// 192 KB of LDS reads (436 B/ns).  A step takes 1.5 us: the 16 products of a phase are
// 244 ns, but the other group's reads of a phase, their latency and the barrier up to
// 370.  The start and end of a tile are 5 and up to 9 us of 60.  Waves that read the
// next operands between their products and meet twice a step, without turns, took 150
// us where this takes 124.
template <typename T, Mode MODE>
__global__ void __launch_bounds__(T::THREADS, 2) k_big(const Fp8Args a, const Launch l) {
  constexpr int W = T::W, TN = T::TN, TM = T::TM, SC = T::SC;
  static_assert(W == 8 && TN == 8 && T::ST == 2 && MODE != WIDE, "two groups of four waves");
  constexpr bool E8 = MODE == FP8E;
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  u32* const scales = reinterpret_cast<u32*>(lds + 2 * T::STAGE);
  const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, h = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave / T::WM, wm = wave % T::WM;
  const Where o = where(a, l, T::BN, T::BM);
  const Fp8Problem& p = a.p[o.problem];
  const int n0 = o.n0, steps = o.steps;
  const size_t m0 = o.m0;
  const int KB = p.K / 128, nb = (p.N + 127) / 128;

  const __amdgpu_buffer_rsrc_t wr = buffer(p.w + (size_t)n0 * p.K + (size_t)o.b0 * 128);
  const __amdgpu_buffer_rsrc_t xr = buffer(p.x + m0 * p.K + (size_t)o.b0 * 128);
  const int w_last = p.N - 1 - n0, x_last = (int)min((size_t)a.M - 1 - m0, (size_t)T::BM);
  u32 off[T::COPIES];
#pragma unroll
  for (int c = 0; c < T::COPIES; c++) {
    const int row = (c * W + wave) * 8 + (lane >> 3);
    const int q = c < T::WCOPIES ? min(row, w_last) : min(row - T::BN, x_last);
    off[c] = (u32)q * p.K + (((lane & 7) ^ (lane >> 3)) << 4);
  }
  auto copy = [&](int step) {
    if (step >= steps) return;
    char* dst = lds + (step & 1) * T::STAGE + wave * 1024;
#pragma unroll
    for (int c = 0; c < T::COPIES; c++)
      lds_copy16(c < T::WCOPIES ? wr : xr, dst + c * W * 1024, off[c], step * 128);
  };
  constexpr int PER = T::PER, SPAN = T::ROWS;
  const int srow = tid % T::BM;
  const size_t xs_row = (m0 + min(srow, x_last)) * KB + o.b0;
  u32 sx[PER], sw[T::NB][PER];
  auto load_scales = [&](int first) {
#pragma unroll
    for (int i = 0; i < PER; i++) {
      const int b = min(first + tid / T::BM + i * SPAN, steps - 1);
      sx[i] = load_scale(p.xs, xs_row + b, E8);
#pragma unroll
      for (int n = 0; n < T::NB; n++)
        sw[n][i] = load_scale(p.ws, (size_t)min(n0 / 128 + n, nb - 1) * KB + o.b0 + b, E8);
    }
  };
  auto keep_scales = [&](int buf) {
#pragma unroll
    for (int i = 0; i < PER; i++)
#pragma unroll
      for (int n = 0; n < T::NB; n++)
        scales[buf * T::SCALES + ((tid / T::BM + i * SPAN) * T::NB + n) * T::BM + srow] =
            joint_scale<MODE>(sx[i], sw[n][i], E8);
  };

  f4 acc[TN][TM];
#pragma unroll
  for (int t = 0; t < TN; t++)
#pragma unroll
    for (int j = 0; j < TM; j++) acc[t][j] = f4{0, 0, 0, 0};
  // chunk 4 q + h of a row, in the slot its row's last bits exchange it to
  const int o0 = r * 128 + ((h ^ (r & 7)) << 4), o1 = r * 128 + (((4 + h) ^ (r & 7)) << 4);
  const char* const wl = lds + wn * 128 * 128;
  const char* const xl = lds + T::BN * 128 + wm * TM * 16 * 128;
  Op x[TM], w[TN / 2];
  u32 s[TM];
  auto read_w = [&](int step, int half) {
    const char* b = wl + (step & 1) * T::STAGE + half * (TN / 2) * 2048;
#pragma unroll
    for (int t = 0; t < TN / 2; t++) {
      w[t].q[0] = *reinterpret_cast<const u32x4*>(b + t * 2048 + o0);
      w[t].q[1] = *reinterpret_cast<const u32x4*>(b + t * 2048 + o1);
    }
  };
  auto read_x = [&](int step) {
    const char* b = xl + (step & 1) * T::STAGE;
#pragma unroll
    for (int j = 0; j < TM; j++) {
      x[j].q[0] = *reinterpret_cast<const u32x4*>(b + j * 2048 + o0);
      x[j].q[1] = *reinterpret_cast<const u32x4*>(b + j * 2048 + o1);
    }
    const u32* sp = scales + (step / SC & 1) * T::SCALES + (step % SC * T::NB + wn) * T::BM +
                    wm * TM * 16 + r;
#pragma unroll
    for (int j = 0; j < TM; j++) s[j] = sp[16 * j];
  };
  auto multiply_half = [&](auto half) {
    constexpr int T0 = decltype(half)::value * (TN / 2);
    __builtin_amdgcn_s_setprio(1);
    if constexpr (E8) {
#pragma unroll
      for (int t = 0; t < TN / 2; t++)
#pragma unroll
        for (int j = 0; j < TM; j++)
          acc[T0 + t][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              w[t].v, x[j].v, acc[T0 + t][j], 0, 0, 0, 127, 0, (int)s[j]);
    } else {
      // a product's multiply-adds come two products later, when it is there
      constexpr int L = 2, N = TN / 2 * TM;
      f4 d[L + 1];
#pragma unroll
      for (int i = 0; i < N + L; i++) {
        if (i < N) {
          const f4 z = {0, 0, 0, 0};
          d[i % (L + 1)] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              w[i / TM].v, x[i % TM].v, z, 0, 0, 0, 127, 0, 127);
        }
        if (i >= L) {
          const int q = i - L;
#pragma unroll
          for (int e = 0; e < 4; e++)
            acc[T0 + q / TM][q % TM][e] = __builtin_fmaf(d[q % (L + 1)][e], __builtin_bit_cast(float, s[q % TM]),
                                                         acc[T0 + q / TM][q % TM][e]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    // made here: left alone, the compiler moves products over a barrier into
    // another phase
#pragma unroll
    for (int t = 0; t < TN / 2; t++)
#pragma unroll
      for (int j = 0; j < TM; j++) pin(acc[T0 + t][j]);
    __builtin_amdgcn_s_setprio(0);
  };
  load_scales(0);
  copy(0);
  wait_vm<0>();
  keep_scales(0);
  phase_end();
  // Phase g of the workgroup is phase g % 4 of step g / 4 in the first group and
  // phase g - 1 in the second.  A stage is last read in phase 4 step + 3 (the
  // second group's third), so copies into it are allowed from phase 4 (step + 1)
  // on, which is where both groups begin; the next step is first read one phase
  // after the second group's third, where both have waited.
  if (wave >= 4) phase_end();
  for (int step = 0; step < steps; step++) {
    if (step % SC == 0 && step + SC < steps) load_scales(step + SC);
    read_x(step);
    read_w(step, 0);
    __builtin_amdgcn_sched_barrier(0);
    copy(step + 1);
    phase_end();
    multiply_half(std::integral_constant<int, 0>{});
    phase_end();
    read_w(step, 1);
    wait_vm<0>();
    if (step % SC == SC - 2 && step + 2 < steps) keep_scales((step / SC & 1) ^ 1);
    phase_end();
    multiply_half(std::integral_constant<int, 1>{});
    phase_end();
  }
  if (wave < 4) phase_end();
  store_tile<TM>(a, p, n0 + wn * 128, m0 + wm * TM * 16, acc);
}

// Up to 16 rows: a workgroup takes 16 TW outputs and its eight waves every eighth
// block of K, from memory straight to the operands, D blocks asked for ahead; the
// eight sums meet in LDS.  No wave waits for another before that, and no sums go
// through memory (K split over workgroups instead took 17.1 us where this takes 9.8).
constexpr int SW = 8;
template <int TW>
struct Block {
  u32x4 w[TW][2], x[2];
  u32 sx, sw;
};

template <int TW, int D, bool E8>
__global__ void __launch_bounds__(64 * SW, 2) k_rows(const Fp8Args a, const Launch l) {
  __shared__ f4 sums[SW][TW][64];
  const int lane = threadIdx.x & 63, r = lane & 15, h = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // neighbouring tiles to one XCD
  const u32 xcd = blockIdx.x & 7, each = gridDim.x >> 3, more = gridDim.x & 7;
  const int tile = xcd * each + min(xcd, more) + (blockIdx.x >> 3);
  int pi = 0;
  while (pi + 1 < a.count && tile >= l.tile0[pi + 1]) pi++;
  const Fp8Problem& p = a.p[pi];
  const int n0 = (tile - l.tile0[pi]) * 16 * TW, KB = p.K / 128;
  const uint8_t* wp[TW];
#pragma unroll
  for (int t = 0; t < TW; t++) wp[t] = p.w + (size_t)min(n0 + 16 * t + r, p.N - 1) * p.K + 16 * h;
  const size_t m = min(r, a.M - 1);  // rows past the end repeat the last one
  const uint8_t* xp = p.x + m * p.K + 16 * h;
  // of lanes, not of the wave: a scale in a scalar register is waited for at once
  int lane0 = 0;
  pin(lane0);
  const size_t xs = m * KB, ws = (size_t)(n0 / 128) * KB + lane0;
  Block<TW> ring[D];
  auto load = [&](Block<TW>& v, int b) {
    const size_t at = (size_t)b * 128;
#pragma unroll
    for (int t = 0; t < TW; t++)
#pragma unroll
      for (int q = 0; q < 2; q++)
        v.w[t][q] = *reinterpret_cast<const u32x4*>(wp[t] + at + 64 * q);
#pragma unroll
    for (int q = 0; q < 2; q++) v.x[q] = *reinterpret_cast<const u32x4*>(xp + at + 64 * q);
    v.sx = load_scale(p.xs, xs + b, E8);
    v.sw = load_scale(p.ws, ws + b, E8);
  };
  f4 acc[TW][1];
#pragma unroll
  for (int t = 0; t < TW; t++) acc[t][0] = f4{0, 0, 0, 0};
  auto multiply_block = [&](const Block<TW>& v) {
    h8 w[TW][2][2], x[1][2][2];
#pragma unroll
    for (int q = 0; q < 2; q++) {
#pragma unroll
      for (int t = 0; t < TW; t++) widen(v.w[t][q], w[t][q]);
      widen(v.x[q], x[0][q]);
    }
    const float f[1] = {__builtin_bit_cast(float, joint_scale<WIDE>(v.sx, v.sw, E8))};
    multiply_wide<TW, 1>(w, x, f, acc);
  };
  // Rounds whose next blocks are all there, and the rest: with a condition at every
  // load the compiler waits for all loads where the ways meet (3 rows, 65536 x 2048:
  // 30.5 us, and 28.7 so; 8 rows, 16384 x 4096 12.8 and 12.2).
  int b = wave;
  if (b + (2 * D - 1) * SW < KB) {
#pragma unroll
    for (int d = 0; d < D; d++) {
      load(ring[d], b + d * SW);
      __builtin_amdgcn_sched_barrier(0);
    }
    do {
#pragma unroll
      for (int d = 0; d < D; d++) {
        multiply_block(ring[d]);
        __builtin_amdgcn_sched_barrier(0);
        load(ring[d], b + (d + D) * SW);
        __builtin_amdgcn_sched_barrier(0);
      }
      b += D * SW;
    } while (b + (2 * D - 1) * SW < KB);
  } else {
#pragma unroll
    for (int d = 0; d < D; d++)
      if (b + d * SW < KB) load(ring[d], b + d * SW);
  }
#pragma unroll
  for (int d = 0; d < D; d++) {
    if (b + d * SW < KB) multiply_block(ring[d]);
    if (b + (d + D) * SW < KB) load(ring[d], b + (d + D) * SW);
  }
#pragma unroll
  for (int d = 0; d < D - 1; d++)
    if (b + (d + D) * SW < KB) multiply_block(ring[d]);
#pragma unroll
  for (int t = 0; t < TW; t++) sums[wave][t][lane] = acc[t][0];
  __syncthreads();
  for (int t = wave; t < TW; t += SW) {
    f4 v = sums[0][t][lane];
#pragma unroll
    for (int w = 1; w < SW; w++) v += sums[w][t][lane];
    const int n = n0 + 16 * t + 4 * h;
    if (r < a.M && n < p.N) store4(p, a.out, r, n, v);
  }
}

template <int TW, int D>
hipError_t launch_rows(const Fp8Args& a, const Launch& l, int tiles, hipStream_t s) {
  if (a.e8m0)
    hipLaunchKernelGGL((k_rows<TW, D, true>), dim3(tiles), dim3(64 * SW), 0, s, a, l);
  else
    hipLaunchKernelGGL((k_rows<TW, D, false>), dim3(tiles), dim3(64 * SW), 0, s, a, l);
  return hipGetLastError();
}

// Some rows: a workgroup takes 16 TN outputs of 16 TM rows, and each of its eight
// waves every eighth block of K through a ring of ST stages in LDS of its own; the
// eight sums meet at the end.  No wave waits for another before that, and no sums go
// through memory (32 rows, 4096 x 16384: 26.4 us with K split over workgroups of
// k_tile, 17.2 so).  Through LDS because its copies take whole lines of eight rows;
// the operands' own layout is 64 bytes of sixteen, and loads of that straight to
// registers are slower from two row tiles on (203 rows, 2560 x 10240: 44.9 us).
// Bound by the copies (with one stage a wave asks for the next block when it has
// multiplied the last, and the other seven waves hide it) and, from three row tiles
// on, by widening both operands in every wave.
template <int TN, int TM, int ST, bool E8>
__global__ void __launch_bounds__(64 * SW, 2) k_ring(const Fp8Args a, const Launch l) {
  constexpr int W = SW;
  constexpr int STAGE = (TN + TM) * 2048, COPIES = 2 * (TN + TM);
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, h = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const Where o = where(a, l, 16 * TN, 16 * TM);
  const Fp8Problem& p = a.p[o.problem];
  const int n0 = o.n0, KB = p.K / 128;
  const size_t m0 = o.m0;
  char* const ring = lds + wave * ST * STAGE;
  const __amdgpu_buffer_rsrc_t wr = buffer(p.w + (size_t)n0 * p.K);
  const __amdgpu_buffer_rsrc_t xr = buffer(p.x + m0 * p.K);
  const int w_last = p.N - 1 - n0, x_last = (int)min((size_t)a.M - 1 - m0, (size_t)16 * TM);
  u32 off[COPIES];
#pragma unroll
  for (int c = 0; c < COPIES; c++) {
    const int row = c * 8 + (lane >> 3);
    const int q = c < 2 * TN ? min(row, w_last) : min(row - 16 * TN, x_last);
    off[c] = (u32)q * p.K + (((lane & 7) ^ (lane >> 3)) << 4);
  }
  size_t xs[TM];
#pragma unroll
  for (int j = 0; j < TM; j++) xs[j] = (m0 + min(16 * j + r, x_last)) * KB;
  int lane0 = 0;
  // of lanes, not of the wave: a scale in a scalar register would be waited for before
  // the copies behind it
  if constexpr (ST > 1) pin(lane0);
  const size_t ws = (size_t)(n0 / 128) * KB + lane0;
  u32 sx[ST][TM], sw[ST];
  auto ask_scales = [&](int b, int d) {
#pragma unroll
    for (int j = 0; j < TM; j++) sx[d][j] = load_scale(p.xs, xs[j] + b, E8);
    sw[d] = load_scale(p.ws, ws + b, E8);
    __builtin_amdgcn_sched_barrier(0);
  };
  // The wave's step i in slot d; past its last one, the last block again, so that
  // every step has the same loads behind it.  With several stages the scales come
  // first: whether they are vector or scalar loads, a slot's copies then have at least
  // the copies of the later slots behind them, which is what the waits count on.  One
  // stage waits for all it asked for, and its copies are the longer way (203 rows,
  // 2560 x 10240: 22.8 us, scales first 24.2).
  auto ask = [&](int i, int d) {
    const int b = min(wave + i * W, KB - 1);
    if constexpr (ST > 1) ask_scales(b, d);
#pragma unroll
    for (int c = 0; c < COPIES; c++)
      lds_copy16(c < 2 * TN ? wr : xr, ring + d * STAGE + c * 1024, off[c], b * 128);
    if constexpr (ST == 1) ask_scales(b, d);
    __builtin_amdgcn_sched_barrier(0);
  };
  f4 acc[TN][TM];
#pragma unroll
  for (int t = 0; t < TN; t++)
#pragma unroll
    for (int j = 0; j < TM; j++) acc[t][j] = f4{0, 0, 0, 0};
  const int o0 = r * 128 + ((h ^ (r & 7)) << 4), o1 = r * 128 + (((4 + h) ^ (r & 7)) << 4);
  const int n = (KB - wave + W - 1) / W;
  auto multiply_step = [&](int d) {
    __builtin_amdgcn_sched_barrier(0);
    wait_vm<(ST - 1) * COPIES>();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    const char* const st = ring + d * STAGE;
    h8 x[TM][2][2];
#pragma unroll
    for (int j = 0; j < TM; j++) {
      widen(*reinterpret_cast<const u32x4*>(st + (TN + j) * 2048 + o0), x[j][0]);
      widen(*reinterpret_cast<const u32x4*>(st + (TN + j) * 2048 + o1), x[j][1]);
    }
    float f[TM];
#pragma unroll
    for (int j = 0; j < TM; j++)
      f[j] = __builtin_bit_cast(float, joint_scale<WIDE>(sx[d][j], sw[d], E8));
    multiply_wide<TN, TM>(st, o0, o1, x, f, acc);
    // the slot has been read
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (0 << 8) | (3 << 14));
    __builtin_amdgcn_sched_barrier(0);
  };
#pragma unroll
  for (int d = 0; d < ST; d++) ask(d, d);
  // whole rounds of the slots, and the rest: a way out of the middle of a round makes
  // the compiler wait for every load where the ways meet
  int i = 0;
  for (; i + ST <= n; i += ST) {
#pragma unroll
    for (int d = 0; d < ST; d++) {
      multiply_step(d);
      ask(i + d + ST, d);
    }
  }
  static_assert(ST <= 2, "at most one step is left, with the next one's copies behind its own");
  if (i < n) multiply_step(0);
  wait_vm<0>();
  __syncthreads();
  f4* const sums = reinterpret_cast<f4*>(lds);
#pragma unroll
  for (int t = 0; t < TN; t++)
#pragma unroll
    for (int j = 0; j < TM; j++) sums[((t * TM + j) * W + wave) * 64 + lane] = acc[t][j];
  __syncthreads();
  if constexpr (TN == 8) {  // whole blocks of outputs, to be quantized
    for (int j = wave; j < TM; j += W) {
      f4 rows[TB][1];
#pragma unroll
      for (int t = 0; t < TB; t++) {
        rows[t][0] = sums[(t * TM + j) * W * 64 + lane];
#pragma unroll
        for (int w = 1; w < W; w++) rows[t][0] += sums[((t * TM + j) * W + w) * 64 + lane];
      }
      store_tile<1>(a, p, n0, m0 + 16 * j, rows);
    }
    return;
  }
  for (int c = wave; c < TN * TM; c += W) {
    f4 v = sums[c * W * 64 + lane];
#pragma unroll
    for (int w = 1; w < W; w++) v += sums[(c * W + w) * 64 + lane];
    const size_t m = m0 + 16 * (c % TM) + r;
    const int at = n0 + 16 * (c / TM) + 4 * h;
    if (m < (size_t)a.M && at < p.N) store4(p, a.out, m, at, v);
  }
}

template <int TN, int TM, int ST>
hipError_t launch_ring(const Fp8Args& a, const Launch& l, int tiles, hipStream_t s) {
  constexpr int BYTES = SW * ST * (TN + TM) * 2048;
  static_assert(BYTES <= 160 * 1024 && SW * TN * TM * 1024 <= BYTES, "LDS");
  static LdsLimit limits[2];
  const auto kernel = a.e8m0 ? k_ring<TN, TM, ST, true> : k_ring<TN, TM, ST, false>;
  const hipError_t e = limits[a.e8m0 != 0].raise(reinterpret_cast<const void*>(kernel), BYTES);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kernel, dim3(tiles), dim3(64 * SW), BYTES, s, a, l);
  return hipGetLastError();
}

// FP8 operands: 128 outputs a wave, so that a row's block is one wave's
typedef Tile<2, 4, 8, 4, 2> T256;  // 256 outputs x 256 rows
typedef Tile<1, 4, 8, 2, 2> T128;  // 128 x 128
typedef Tile<1, 4, 8, 1, 2> T64;   // 128 x 64
// binary16 operands, widened by every wave that reads them: as square as they go
// (2047 rows of 16384 x 4096: 262 us, by eight waves of 64 x 32 280; both with the
// inputs in turn)
typedef Tile<2, 2, 4, 4, 2> W128;  // 128 x 128
// (61 rows of 65529 x 2048: 32.5 us; with one set of inputs over and over, half of it in
// the last-level cache, 28.1, and by eight waves of 32 x 32 30.6)
typedef Tile<2, 2, 4, 2, 2> W64;   // 128 x 64

// What a call runs: a kernel with its tile, and the ranges of K.
enum Kind {
  ROWS16, ROWS64, RING1X2, RING2X2, RING4X2, RING4X3, RING4X4, RING8X1, RING8X2, WIDE64, WIDE128, FP128,
  FP256, FP64
};
struct Shape {
  int bn, bm;
};
constexpr Shape SHAPES[] = {{16, 16},  {64, 16},  {16, 32},  {32, 32},  {64, 32},   {64, 48},  {64, 64},
                            {128, 16}, {128, 32}, {128, 64}, {128, 128}, {128, 128}, {256, 256}, {128, 64}};
struct Plan {
  Kind kind;
  int splits;
};
constexpr int CUS = 256;

long long tiles_of(const Fp8Args& a, Kind kind) {
  const Shape& s = SHAPES[kind];
  long long n = 0;
  for (int i = 0; i < a.count; i++)
    n += (long long)((a.M + s.bm - 1) / s.bm) * ((a.p[i].N + s.bn - 1) / s.bn);
  return n;
}

constexpr int COUNTERS = 16384;  // dwords at the front of a workspace, of which tiles count in a few

size_t plan_bytes(const Fp8Args& a, const Plan& c) {
  if (c.splits <= 1) return 0;
  const Shape& s = SHAPES[c.kind];
  return COUNTERS * 4 + (size_t)tiles_of(a, c.kind) * c.splits * s.bn * s.bm * 4;
}

// Products in binary16 instructions.  Rows and rings add in one order whatever their
// tile, each wave's blocks and then the waves, which quantized outputs count on.
Kind choose_wide(const Fp8Args& a) {
  // Tiles of 16 rows while they all run at once (32 rows, us: 4096 outputs of K =
  // 16384 29.5 and in tiles of 32 rows 38.9; 16384 of 4096 17.1 and 18.8), of 32
  // where they do not, which read w half as often (96 rows, 8192 outputs of K = 2048:
  // 11.1, and in tiles of 16 rows 16.0).
  if (a.out == OUT_E4M3) return a.M <= 16 || tiles_of(a, RING8X1) <= CUS ? RING8X1 : RING8X2;
  int kb = 0;
  for (int i = 0; i < a.count; i++) kb = a.p[i].K / 128 > kb ? a.p[i].K / 128 : kb;
  // Rows straight to registers, us beside the best of the tiles below:
  //   rows x outputs x K       64 outputs  16 outputs  tiles
  //   1 x 16384 x 4096            12.1        12.9      13.3
  //   1 x 4096 x 4096, three      10.5         9.8      11.1
  //   8 x 16384 x 4096            12.3        16.1      13.4
  //   16 x 65536 x 2048           30.6        43.5      28.5
  //   16 x 768 x 768               4.2         3.5       3.7
  //   16 x 4096 x 4096, three     12.5        15.9      11.5
  //   4 x 4096 x 16384            34.7        15.0      13.4
  //   16 x 4096 x 16384           40.3        20.3      14.5
  if (a.M <= 16) {
    const long long n = tiles_of(a, ROWS64);
    if (n >= CUS && (a.M <= 4 || n < 4 * CUS || a.out != OUT_F32)) return ROWS64;
    if (a.M <= 4 || (tiles_of(a, ROWS16) <= CUS && kb <= 32)) return ROWS16;
  }
  // What a compute unit takes for as many tiles as it has at once (`most`, or fewer):
  // their start and end, and a block of K, in us, fitted to about 50 sizes.  It puts,
  // say, 61 rows x 32768 x 2048 in tiles of 64 rows (18.0 us; rings 21.8, 128 rows
  // 23.4), 600 x 4096 x 4096 too (38.5; 37.6, 41.8), 256 x 4096 x 4096 in rings (14.4;
  // 26.9, 40.4), 1500 x 4096 x 4096 in tiles of 64 (55.2; 79.7, 62.4), 2047 x 4096 x
  // 4096 in tiles of 128 (65.7; 64 rows 73.2).
  const struct {
    Kind kind;
    int most;
    double us[3][2];
  } tiles[] = {{RING1X2, 1, {{3.4, 0.11}}},
               {RING2X2, 2, {{3.2, 0.12}, {3.2, 0.24}}},
               {RING4X2, 1, {{4.3, 0.155}}},
               {RING4X3, 1, {{5.0, 0.2}}},
               {RING4X4, 1, {{5.4, 0.25}}},
               {WIDE64, 3, {{3.0, 0.8}, {4.0, 1.1}, {4.5, 1.6}}},
               {WIDE128, 2, {{4.5, 1.15}, {5.8, 1.85}}}};
  Kind best = RING4X4;
  double least = 1e30;
  for (const auto& q : tiles) {
    if ((q.kind == WIDE64 || q.kind == WIDE128) && a.out != OUT_F32) continue;
    const long long n = (tiles_of(a, q.kind) + CUS - 1) / CUS;  // of a compute unit
    auto us = [&](long long at_once) {
      return at_once ? q.us[at_once - 1][0] + kb * q.us[at_once - 1][1] : 0.0;
    };
    const double t = (double)(n / q.most) * us(q.most) + us(n % q.most);
    if (t < least) least = t, best = q.kind;
  }
  return best;
}

// Rows and rings for all binary32 outputs, and for the others while tiles of 128 x
// 128 would leave three quarters of the card empty (half, of up to 64 rows, which fill
// half a tile).  Measured, binary16 outputs, us (rings; tiles of 128 rows with K split
// through a workspace; tiles of 64 rows):
//   rows x outputs x K         tiles   rings  split  64 rows
//   203 x 4096 x 4096            64     14.2   17.8    21.0
//   256 x 4096 x 16384           64     43.0   35.4    70.2
//   100 x 4096 x 4096, three     96     26.3   22.5    22.8
//   512 x 4096 x 4096           128     26.6   21.9    22.7
//   203 x 4096 x 4096, three    192     38.4     -     24.7
//   64 x 16384 x 4096           128     17.3   24.9    24.7
//   48 x 20480 x 4096           160     26.2     -     28.5
//   17 x 65536 x 2048           512     34.5     -     26.6
//   64 x 65536 x 2048           512     47.8     -     28.7
// The rule goes by tiles alone.  At its borders K and rows matter too: the second and
// the seventh of these sizes take the kernel that is 21% and 9% slower.
bool few(const Fp8Args& a) {
  const long long tiles = tiles_of(a, FP128);
  return a.out == OUT_F32 || a.M <= 16 || tiles <= CUS / 4 || (a.M <= 64 && tiles <= CUS / 2);
}

// K is split, with a workspace, where compute units would have no tile of 128 x 128,
// in ranges of 16 blocks at least (binary16, us, split and in whole tiles of 64 rows:
// 512 x 4096 x 4096 21.9 and 22.7, 400 x 4096 x 16384 53.4 and 71.8; with ranges of
// eight 1000 x 2048 x 2048 15.8 and 13.0, 300 x 4096 x 2048 14.6 and 12.4).
Plan choose(const Fp8Args& a, bool split) {
  if (few(a)) return Plan{choose_wide(a), 1};
  // A round of tiles of 256 x 256, one to a compute unit, takes 1.2 times as long as
  // one of 128 x 128, two to a compute unit, of half as much; the smaller ones do
  // not wait for each other's round.  (4096 outputs of K = 4096, us, 256 and 128:
  // 2048 rows 48.8 and 36.8, 2500 48.8 and 56.7, 4001 59.0 and 77.7, 4352 97.6 and 93.8.)
  const long long large = (tiles_of(a, FP256) + CUS - 1) / CUS, small = tiles_of(a, FP128);
  if (12 * large * 2 * CUS < 10 * (small < 2 * CUS ? 2 * CUS : small)) return Plan{FP256, 1};
  // Where every tile of 128 x 128 has a compute unit to itself, or half its rows would
  // be past the end, tiles of 64 rows share one and fill each other's waits (binary16,
  // us, 64 and 128 rows: 1024 x 4096 x 4096 26.9 and 29.0, 203 rows of three 4096 x
  // 4096 24.7 and 26.9, 64 x 65536 x 2048 28.7 and 30.4; 1300 x 4096 x 4096, which has
  // more tiles, 33.8 and 32.6).
  const Plan whole{small <= CUS || a.M <= 64 ? FP64 : FP128, 1};
  if (!split) return whole;
  int kb = 1 << 30;
  for (int i = 0; i < a.count; i++) kb = a.p[i].K / 128 < kb ? a.p[i].K / 128 : kb;
  const long long want = CUS / small;  // 3 at most: `few` has the rest
  const int splits = (int)(want < kb / 16 ? want : kb / 16);
  return splits > 1 ? Plan{FP128, splits} : whole;
}

template <typename T, Mode MODE, bool E8>
hipError_t launch_tile(const Fp8Args& a, const Launch& l, int tiles, hipStream_t s) {
  static LdsLimit limit;
  void (*kernel)(const Fp8Args, const Launch);
  if constexpr (T::BM == 256)
    kernel = k_big<T, MODE>;
  else
    kernel = k_tile<T, MODE, E8>;
  const hipError_t e = limit.raise(reinterpret_cast<const void*>(kernel), T::LDS);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kernel, dim3((unsigned)tiles * l.splits), dim3(T::THREADS), T::LDS, s, a, l);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_wide(const Fp8Args& a, const Launch& l, int tiles, hipStream_t s) {
  return a.e8m0 ? launch_tile<T, WIDE, true>(a, l, tiles, s)
                : launch_tile<T, WIDE, false>(a, l, tiles, s);
}
template <typename T>
hipError_t launch_fp8_tile(const Fp8Args& a, const Launch& l, int tiles, hipStream_t s) {
  return a.e8m0 ? launch_tile<T, FP8E, true>(a, l, tiles, s)
                : launch_tile<T, FP8S, false>(a, l, tiles, s);
}

}  // namespace

size_t fp8_workspace_bytes(const Fp8Args& a) { return plan_bytes(a, choose(a, true)); }

hipError_t launch_fp8(const Fp8Args& a, void* ws, hipStream_t s) {
  const Plan c = choose(a, ws != nullptr);
  const Shape& t = SHAPES[c.kind];
  Launch l{};
  l.mt = (a.M + t.bm - 1) / t.bm;
  l.splits = c.splits;
  if (c.splits > 1) {
    l.counters = static_cast<unsigned*>(ws);
    l.partial = static_cast<float*>(ws) + COUNTERS;
  }
  for (int i = 0; i < a.count; i++)
    l.tile0[i + 1] = l.tile0[i] + l.mt * ((a.p[i].N + t.bn - 1) / t.bn);
  const int tiles = l.tile0[a.count];
  switch (c.kind) {
    case ROWS16: return launch_rows<1, 2>(a, l, tiles, s);
    case ROWS64: return launch_rows<4, 1>(a, l, tiles, s);
    case RING1X2: return launch_ring<1, 2, 2>(a, l, tiles, s);
    case RING2X2: return launch_ring<2, 2, 1>(a, l, tiles, s);
    case RING4X2: return launch_ring<4, 2, 1>(a, l, tiles, s);
    case RING4X3: return launch_ring<4, 3, 1>(a, l, tiles, s);
    case RING4X4: return launch_ring<4, 4, 1>(a, l, tiles, s);
    case RING8X1: return launch_ring<8, 1, 1>(a, l, tiles, s);
    case RING8X2: return launch_ring<8, 2, 1>(a, l, tiles, s);
    case WIDE64: return launch_wide<W64>(a, l, tiles, s);
    case WIDE128: return launch_wide<W128>(a, l, tiles, s);
    case FP128: return launch_fp8_tile<T128>(a, l, tiles, s);
    case FP64: return launch_fp8_tile<T64>(a, l, tiles, s);
    default: return launch_fp8_tile<T256>(a, l, tiles, s);
  }
}

}  // namespace rq
