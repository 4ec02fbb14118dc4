// rq_gemm_fp8.hip -- products of block-scaled E4M3 operands:
//   y[m][n] = y_in[m][n] + sum_b xs[m][b] ws[n/128][b] sum_{k in b} x[m][k] w[n][k].
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
  unsigned* counters;        // one per tile, zero between launches
  float* partial;            // [tile][split][outputs of a tile, as the lanes hold them]
};

constexpr int TN = 8;  // 16-row tiles of w of a wave: one block of outputs

// WN x WM waves, each 128 outputs of 16 * TM rows; ST stages of 128 columns.
template <int WN_, int WM_, int TM_, int ST_>
struct Tile {
  static constexpr int WN = WN_, WM = WM_, TM = TM_, ST = ST_;
  static constexpr int W = WN * WM, THREADS = 64 * W;
  static constexpr int BN = 128 * WN, BM = 16 * TM * WM;
  static constexpr int STAGE = (BN + BM) * 128;
  static constexpr int COPIES = (BN + BM) / 8 / W;  // of a wave for a stage
  static constexpr int WCOPIES = BN / 8 / W;        // of these, rows of w
  static constexpr int SC = 4;                      // blocks of K whose scales are staged together
  static constexpr int SCALES = SC * WN * BM;       // dwords of a buffer of scales
  static constexpr int LDS = ST * STAGE + 2 * SCALES * 4;
  static_assert((BN + BM) / 8 % W == 0 && BN / 8 % W == 0, "whole copies");
  static_assert(LDS <= 160 * 1024, "LDS");
  static constexpr int PER = SC * BM / THREADS;  // scales of x that a thread stages
  static_assert(SC * BM % THREADS == 0 || SC * BM < THREADS, "scales");
};

// The products of one block of K from a stage in LDS.
template <typename T, Mode MODE>
__device__ __forceinline__ void multiply(const char* stage, const u32* scales, int wn, int wm,
                                         f4 (&acc)[TN][T::TM]) {
  constexpr int TM = T::TM;
  const int lane = threadIdx.x & 63, r = lane & 15, h = lane >> 4;
  // chunk 4 p + h of a row, in the slot its row's last bits exchange it to
  const int o0 = r * 128 + ((h ^ (r & 7)) << 4), o1 = r * 128 + (((4 + h) ^ (r & 7)) << 4);
  const char* wp = stage + wn * 128 * 128;
  const char* xp = stage + T::BN * 128 + wm * TM * 16 * 128;
  u32 s[TM];
#pragma unroll
  for (int j = 0; j < TM; j++) s[j] = scales[wn * T::BM + (wm * TM + j) * 16 + r];
  if constexpr (MODE == WIDE) {
    h8 x[TM][2][2];
#pragma unroll
    for (int j = 0; j < TM; j++) {
      widen(*reinterpret_cast<const u32x4*>(xp + j * 2048 + o0), x[j][0]);
      widen(*reinterpret_cast<const u32x4*>(xp + j * 2048 + o1), x[j][1]);
    }
#pragma unroll
    for (int t = 0; t < TN; t++) {
      h8 w[2][2];
      widen(*reinterpret_cast<const u32x4*>(wp + t * 2048 + o0), w[0]);
      widen(*reinterpret_cast<const u32x4*>(wp + t * 2048 + o1), w[1]);
#pragma unroll
      for (int j = 0; j < TM; j++) {
        f4 d = {0, 0, 0, 0};
#pragma unroll
        for (int q = 0; q < 2; q++)
#pragma unroll
          for (int e = 0; e < 2; e++)
            d = __builtin_amdgcn_mfma_f32_16x16x32_f16(w[q][e], x[j][q][e], d, 0, 0, 0);
        const float f = __builtin_bit_cast(float, s[j]);
#pragma unroll
        for (int i = 0; i < 4; i++) acc[t][j][i] = __builtin_fmaf(d[i], f, acc[t][j][i]);
      }
    }
  } else {
    union Op {
      u32x4 q[2];
      i8v v;
    };
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

// Four consecutive outputs of row m.
__device__ __forceinline__ void store4(const Fp8Problem& p, int out, size_t m, int n, f4 v) {
  const size_t at = m * p.N + n;
  const bool whole = p.N % 4 == 0 && n < p.N;
  if (out == OUT_F32) {
    float* y = static_cast<float*>(p.y) + at;
    if (whole) {
      if (p.y_in) v = *reinterpret_cast<const f4*>(p.y_in + at) + v;
      *reinterpret_cast<f4*>(y) = v;
    } else {
#pragma unroll
      for (int i = 0; i < 4; i++)
        if (n + i < p.N) y[i] = p.y_in ? p.y_in[at + i] + v[i] : v[i];
    }
  } else {
    _Float16* y = static_cast<_Float16*>(p.y) + at;
    const h4 o = {(_Float16)v[0], (_Float16)v[1], (_Float16)v[2], (_Float16)v[3]};
    if (whole) {
      *reinterpret_cast<h4*>(y) = o;
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
template <int C>
__device__ __forceinline__ void quantize_rows(const f4 (&acc)[TN][C], bool square, u32 (&c)[C][TN],
                                              u32 (&se)[C]) {
  h2 z[C][2 * TN];
  const h2 zero = {0, 0};
  h2 odd = zero;  // NaN once a value is not finite
  float top[C];
#pragma unroll
  for (int j = 0; j < C; j++) {
    h2 most = zero;
#pragma unroll
    for (int t = 0; t < TN; t++)
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
      for (int t = 0; t < TN; t++)
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
    for (int t = 0; t < TN; t++) {
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
                                           const f4 (&acc)[TN][TM]) {
  const int lane = threadIdx.x & 63, r = lane & 15, h = lane >> 4;
  if (a.out == OUT_E4M3) {
    constexpr int C = TM < 2 ? TM : 2;
    each<TM / C>([&](auto part) {
      constexpr int j0 = decltype(part)::value * C;
      f4 rows[TN][C];
      u32 c[C][TN], se[C];
#pragma unroll
      for (int t = 0; t < TN; t++)
#pragma unroll
        for (int j = 0; j < C; j++) rows[t][j] = acc[t][j0 + j];
      quantize_rows<C>(rows, a.relu2, c, se);
#pragma unroll
      for (int j = 0; j < C; j++) {
        const size_t m = m0 + 16 * (j0 + j) + r;
        const bool in = m < (size_t)a.M && n0 < p.N;
#pragma unroll
        for (int g = 0; g < TN / 4; g++) {
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
      for (int g = 0; g < TN / 4; g++) {
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
      for (int t = 0; t < TN; t++) store4(p, a.out, m, n0 + 16 * t + 4 * h, acc[t][j]);
    }
  });
}

// A workgroup's tile and range of K.
struct Where {
  int problem, tile, split, n0, b0, steps;
  size_t m0;
};
template <typename T>
__device__ __forceinline__ Where where(const Fp8Args& a, const Launch& l) {
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
  o.n0 = at / l.mt * T::BN;
  o.m0 = (size_t)(at % l.mt) * T::BM;
  o.b0 = (int)((long long)KB * o.split / l.splits);
  o.steps = (int)((long long)KB * (o.split + 1) / l.splits) - o.b0;
  return o;
}

template <typename T, Mode MODE>
__global__ void __launch_bounds__(T::THREADS, T::W / 4 > 0 ? T::W / 4 : 1)
k_tile(const Fp8Args a, const Launch l) {
  constexpr int W = T::W, TM = T::TM, ST = T::ST, SC = T::SC;
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  u32* const scales = reinterpret_cast<u32*>(lds + ST * T::STAGE);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave / T::WM, wm = wave % T::WM;

  const Where o = where<T>(a, l);
  const Fp8Problem& p = a.p[o.problem];
  const int n0 = o.n0, b0 = o.b0, steps = o.steps, split = o.split, tile = o.tile;
  const size_t m0 = o.m0;
  const int KB = p.K / 128, nb = (p.N + 127) / 128;
  const bool e8m0 = a.e8m0;

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
  constexpr int PER = T::PER > 0 ? T::PER : 1;
  const int srow = tid % T::BM;
  const bool stager = T::PER > 0 || tid < SC * T::BM;
  const size_t xs_row = (m0 + min(srow, x_last)) * KB + b0;
  u32 sx[PER], sw[T::WN][PER];
  auto load_scales = [&](int first) {
#pragma unroll
    for (int i = 0; i < PER; i++) {
      const int b = min(first + tid / T::BM + i * (T::THREADS / T::BM > 0 ? T::THREADS / T::BM : 1),
                        steps - 1);
      sx[i] = load_scale(p.xs, xs_row + b, e8m0);
#pragma unroll
      for (int n = 0; n < T::WN; n++)
        sw[n][i] = load_scale(p.ws, (size_t)min(n0 / 128 + n, nb - 1) * KB + b0 + b, e8m0);
    }
  };
  auto keep_scales = [&](int buf) {
#pragma unroll
    for (int i = 0; i < PER; i++) {
      const int b = tid / T::BM + i * (T::THREADS / T::BM > 0 ? T::THREADS / T::BM : 1);
#pragma unroll
      for (int n = 0; n < T::WN; n++)
        if (stager)
          scales[buf * T::SCALES + (b * T::WN + n) * T::BM + srow] =
              joint_scale<MODE>(sx[i], sw[n][i], e8m0);
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
    __syncthreads();
    if (s + ST - 1 < steps) copy(s + ST - 1);
    if (s % SC == 0 && s + SC < steps) load_scales(s + SC);
    multiply<T, MODE>(lds + s % ST * T::STAGE,
                      scales + (s / SC & 1) * T::SCALES + s % SC * T::WN * T::BM, wn, wm, acc);
    if (s % SC == SC / 2 && s - s % SC + SC < steps) keep_scales((s / SC & 1) ^ 1);
  }

  const int wave_n0 = n0 + wn * 128;
  const size_t wave_m0 = m0 + wm * TM * 16;
  if (l.splits > 1) {
    // this range's sums, as the lanes hold them, past the caches that other XCDs
    // do not see; then the arrival.  The last to arrive adds the ranges in order.
    constexpr int PART = T::BN * T::BM;
    float* mine = l.partial + ((size_t)tile * l.splits) * PART;
    const __amdgpu_buffer_rsrc_t pr = buffer(mine);
    constexpr int AGENT = 16;  // scope bit of the buffer instructions
#pragma unroll
    for (int t = 0; t < TN; t++)
#pragma unroll
      for (int j = 0; j < TM; j++)
        __builtin_amdgcn_raw_buffer_store_b128(
            __builtin_bit_cast(u32x4, acc[t][j]), pr,
            (split * PART + ((t * TM + j) * W + wave) * 256 + lane * 4) * 4, 0, AGENT);
    wait_vm<0>();
    __syncthreads();
    unsigned* const flag = reinterpret_cast<unsigned*>(lds);
    if (tid == 0)
      *flag = __hip_atomic_fetch_add(l.counters + tile, 1u, __ATOMIC_RELAXED,
                                     __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (*flag != (unsigned)(l.splits - 1)) return;
    if (tid == 0)
      __hip_atomic_store(l.counters + tile, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
    for (int t = 0; t < TN; t++)
#pragma unroll
      for (int j = 0; j < TM; j++) acc[t][j] = f4{0, 0, 0, 0};
    for (int q = 0; q < l.splits; q++) {
#pragma unroll
      for (int t = 0; t < TN; t++)
#pragma unroll
        for (int j = 0; j < TM; j++)
          acc[t][j] += __builtin_bit_cast(
              f4, __builtin_amdgcn_raw_buffer_load_b128(
                      pr, (q * PART + ((t * TM + j) * W + wave) * 256 + lane * 4) * 4, 0, AGENT));
    }
  }
  store_tile<TM>(a, p, wave_n0, wave_m0, acc);
}

// Large tiles: eight waves in two groups that take turns, one reading operands
// from LDS while the other multiplies.  A step (128 columns) is four phases:
// read x and half of w, multiply, read the other half, multiply; the second group
// is one phase behind, so that the matrix units of a SIMD, which has a wave of
// each group, always have work.
union Op {
  u32x4 q[2];
  i8v v;
};

template <typename V>
__device__ __forceinline__ void pin(V& v) {
  asm volatile("" : "+v"(v));
}

// End of a phase: this wave's LDS accesses are done, then everybody's.
__device__ __forceinline__ void phase_end() {
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (0 << 8) | (3 << 14));
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

template <typename T, Mode MODE>
__global__ void __launch_bounds__(T::THREADS, 2) k_big(const Fp8Args a, const Launch l) {
  constexpr int W = T::W, TM = T::TM, SC = T::SC;
  static_assert(W == 8 && T::ST == 2 && MODE != WIDE, "two groups of four waves");
  constexpr bool E8 = MODE == FP8E;
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  u32* const scales = reinterpret_cast<u32*>(lds + 2 * T::STAGE);
  const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, h = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave / T::WM, wm = wave % T::WM;
  const Where o = where<T>(a, l);
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
  constexpr int PER = T::PER, SPAN = T::THREADS / T::BM;
  const int srow = tid % T::BM;
  const size_t xs_row = (m0 + min(srow, x_last)) * KB + o.b0;
  u32 sx[PER], sw[T::WN][PER];
  auto load_scales = [&](int first) {
#pragma unroll
    for (int i = 0; i < PER; i++) {
      const int b = min(first + tid / T::BM + i * SPAN, steps - 1);
      sx[i] = load_scale(p.xs, xs_row + b, E8);
#pragma unroll
      for (int n = 0; n < T::WN; n++)
        sw[n][i] = load_scale(p.ws, (size_t)min(n0 / 128 + n, nb - 1) * KB + o.b0 + b, E8);
    }
  };
  auto keep_scales = [&](int buf) {
#pragma unroll
    for (int i = 0; i < PER; i++)
#pragma unroll
      for (int n = 0; n < T::WN; n++)
        scales[buf * T::SCALES + ((tid / T::BM + i * SPAN) * T::WN + n) * T::BM + srow] =
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
    const u32* sp = scales + (step / SC & 1) * T::SCALES + (step % SC * T::WN + wn) * T::BM +
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

// One row tile, few rows: every wave takes 16 outputs and every 8th block of K,
// straight from memory to the operands; the eight sums meet in LDS.
constexpr int SW = 8;
template <int U>
__global__ void __launch_bounds__(64 * SW, 2) k_rows(const Fp8Args a, const Launch l) {
  __shared__ f4 sums[SW][64];
  const int lane = threadIdx.x & 63, r = lane & 15, h = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tile = blockIdx.x;
  int pi = 0;
  while (pi + 1 < a.count && tile >= l.tile0[pi + 1]) pi++;
  const Fp8Problem& p = a.p[pi];
  const int n0 = (tile - l.tile0[pi]) * 16, KB = p.K / 128;
  const bool e8m0 = a.e8m0;
  const uint8_t* wp = p.w + (size_t)min(n0 + r, p.N - 1) * p.K + 16 * h;
  const int mc = min(r, a.M - 1);
  const uint8_t* xp = p.x + (size_t)mc * p.K + 16 * h;
  f4 acc = {0, 0, 0, 0};
  for (int b = wave; b < KB; b += SW * U) {
    u32x4 w[U][2], x[U][2];
    u32 sx[U], sw[U];
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int bu = min(b + u * SW, KB - 1);
#pragma unroll
      for (int q = 0; q < 2; q++)
        w[u][q] = load_stream16(wp + (size_t)bu * 128 + 64 * q);
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int bu = min(b + u * SW, KB - 1);
#pragma unroll
      for (int q = 0; q < 2; q++)
        x[u][q] = *reinterpret_cast<const u32x4*>(xp + (size_t)bu * 128 + 64 * q);
      sx[u] = load_scale(p.xs, (size_t)mc * KB + bu, e8m0);
      sw[u] = load_scale(p.ws, (size_t)(n0 / 128) * KB + bu, e8m0);
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
      if (b + u * SW >= KB) break;
      f4 d = {0, 0, 0, 0};
#pragma unroll
      for (int q = 0; q < 2; q++) {
        h8 wh[2], xh[2];
        widen(w[u][q], wh);
        widen(x[u][q], xh);
        d = __builtin_amdgcn_mfma_f32_16x16x32_f16(wh[0], xh[0], d, 0, 0, 0);
        d = __builtin_amdgcn_mfma_f32_16x16x32_f16(wh[1], xh[1], d, 0, 0, 0);
      }
      const float f = __builtin_bit_cast(float, joint_scale<WIDE>(sx[u], sw[u], e8m0));
#pragma unroll
      for (int i = 0; i < 4; i++) acc[i] = __builtin_fmaf(d[i], f, acc[i]);
    }
  }
  sums[wave][lane] = acc;
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int w = 1; w < SW; w++) acc += sums[w][lane];
  if (r < a.M && n0 + 4 * h < p.N) store4(p, a.out, r, n0 + 4 * h, acc);
}

typedef Tile<2, 4, 4, 2> T256;  // 256 x 256
typedef Tile<1, 4, 2, 2> T128;  // 128 outputs x 128 rows
typedef Tile<1, 4, 1, 3> T64;   // 128 x 64
typedef Tile<1, 2, 1, 4> T32;   // 128 x 32

struct Plan {
  int kind;  // 0 k_rows, 1 T32, 2 T64, 3 T128, 4 T256
  int splits;
};
constexpr int BNS[] = {16, 128, 128, 128, 256}, BMS[] = {16, 32, 64, 128, 256};

int tiles_of(const Fp8Args& a, int kind) {
  long long n = 0;
  for (int i = 0; i < a.count; i++)
    n += (long long)((a.M + BMS[kind] - 1) / BMS[kind]) * ((a.p[i].N + BNS[kind] - 1) / BNS[kind]);
  return n > (1 << 30) ? 1 << 30 : (int)n;
}

constexpr int COUNTERS = 16384;  // arrival counters at the front of a workspace
constexpr size_t WS_MAX = (size_t)64 << 20;

size_t plan_bytes(const Fp8Args& a, const Plan& c) {
  if (c.splits <= 1) return 0;
  return COUNTERS * 4 + (size_t)tiles_of(a, c.kind) * c.splits * BNS[c.kind] * BMS[c.kind] * 4;
}

Plan choose(const Fp8Args& a, bool split) {
  Plan c{0, 1};
  if (a.M <= 16 && a.out == OUT_F32) return c;
  if (a.M <= 32)
    c.kind = 1;
  else if (a.M <= 64)
    c.kind = 2;
  else
    c.kind = tiles_of(a, 4) >= 192 ? 4 : 3;
  const int tiles = tiles_of(a, c.kind);
  int kb = 1 << 30;
  for (int i = 0; i < a.count; i++) kb = a.p[i].K / 128 < kb ? a.p[i].K / 128 : kb;
  if (split && c.kind < 4 && tiles <= COUNTERS) {
    int want = 256 / tiles;
    if (want > kb / 4) want = kb / 4;
    if (want > 16) want = 16;
    for (; want > 1; want--) {
      c.splits = want;
      if (plan_bytes(a, c) <= WS_MAX) break;
    }
    c.splits = want > 1 ? want : 1;
  }
  return c;
}

template <typename T, Mode MODE>
hipError_t launch_tile(const Fp8Args& a, const Launch& l, int tiles, hipStream_t s) {
  static LdsLimit limit;
  constexpr bool big = T::W == 8 && MODE != WIDE;
  void (*kernel)(const Fp8Args, const Launch);
  if constexpr (big)
    kernel = k_big<T, MODE>;
  else
    kernel = k_tile<T, MODE>;
  const hipError_t e = limit.raise(reinterpret_cast<const void*>(kernel), T::LDS);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kernel, dim3((unsigned)tiles * l.splits), dim3(T::THREADS), T::LDS, s, a, l);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_mode(const Fp8Args& a, const Launch& l, int tiles, hipStream_t s) {
  if (a.out == OUT_F32) return launch_tile<T, WIDE>(a, l, tiles, s);
  return a.e8m0 ? launch_tile<T, FP8E>(a, l, tiles, s) : launch_tile<T, FP8S>(a, l, tiles, s);
}

}  // namespace

size_t fp8_workspace_bytes(const Fp8Args& a) { return plan_bytes(a, choose(a, true)); }

hipError_t launch_fp8(const Fp8Args& a, void* ws, hipStream_t s) {
  const Plan c = choose(a, ws != nullptr);
  Launch l{};
  l.mt = (a.M + BMS[c.kind] - 1) / BMS[c.kind];
  l.splits = c.splits;
  l.counters = static_cast<unsigned*>(ws);
  l.partial = static_cast<float*>(ws) + COUNTERS;
  for (int i = 0; i < a.count; i++)
    l.tile0[i + 1] = l.tile0[i] + l.mt * ((a.p[i].N + BNS[c.kind] - 1) / BNS[c.kind]);
  const int tiles = l.tile0[a.count];
  switch (c.kind) {
    case 0:
      hipLaunchKernelGGL((k_rows<4>), dim3(tiles), dim3(64 * SW), 0, s, a, l);
      return hipGetLastError();
    case 1: return launch_mode<T32>(a, l, tiles, s);
    case 2: return launch_mode<T64>(a, l, tiles, s);
    case 3: return launch_mode<T128>(a, l, tiles, s);
    default: return launch_mode<T256>(a, l, tiles, s);
  }
}

}  // namespace rq
