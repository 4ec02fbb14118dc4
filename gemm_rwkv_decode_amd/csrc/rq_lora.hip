// rq_lora.hip -- low-rank adapters of many requests beside a shared
// projection: row m with adapter i = ids[m] of rank r gets
//   y[m] = y_in[m] + s_i B_i (A_i x[m]),   A_i [r][K], B_i [N][r] binary16.
//
// Two launches: k_lora_down makes t = A_i x[m] for every row (K split over
// workgroups), k_lora_up adds the K ranges' sums in a fixed order and
// multiplies by B_i.  Bound by memory where every request has an adapter of
// its own (2 r (K + N) bytes each), by y's traffic (8 M N bytes) for prompts.
//
// Rows are taken in blocks of 64, one lane a row.  In a block the rows with
// the same adapter are found with one ballot per bit of the adapter's number,
// and a workgroup serves all of them, so an adapter's matrices are read once
// per block however its rows lie.  A row without an adapter costs nothing in
// the first launch and a copy of y_in (where y is another array) in the second.
//
// Both products run on the matrix cores.  x and A are binary16, so the first
// is exact up to its binary32 sums.  t is binary32 and is not rounded to
// binary16: it is split into two binary16 parts, t = 2^e (hi + lo), with e the
// row's own power of two, so B t loses nothing above 2^-22 of the row's largest
// t and cannot overflow for a large x.
//
// A y of many rows goes past the caches both ways, a smaller one stays there for
// its reader (below).  2047 rows of 16384 outputs, rank 64: 75 us, 291 MB at 3.9
// TB/s.  32 requests of 24 adapters of rank 64 on three
// 4096x4096 projections: 25 us, 56 MB (traced apart, the two launches take 11 and
// 14), a third of each the chain ids, offsets, first loads.
#include <algorithm>

#include "rq_common.h"
#include "rq_internal.h"

namespace rq {
namespace {

constexpr int ROWS = 64;  // rows of a block: one per lane
constexpr long long LORA_WORKGROUPS = 1024;

typedef unsigned long long u64;

// The lanes' rows that share the g-th distinct adapter of a block.
struct Group {
  u64 rows;    // 0: the block has no g-th adapter
  int id;      // a.adapters: no adapter
  int off, r;  // its first A row and its rank (0: no adapter)
};

struct Rows {
  int id;       // of the lane's row; a.adapters: none
  int offsets;  // offsets[lane] where all of them fit in a wave
  u64 same;     // the rows with the lane's id
  u64 leaders;  // the first row of every id
};

__device__ __forceinline__ Rows load_rows(const LoraArgs& a, int base) {
  const int lane = threadIdx.x & 63;
  const bool in = base + lane < a.M;
  Rows q;
  q.id = in ? a.ids[base + lane] : 0;
  // asked for beside the ids, not after them
  q.offsets = a.adapters < 64 ? a.offsets[min(lane, a.adapters)] : 0;
  if (q.id < 0 || q.id > a.adapters) q.id = a.adapters;
  q.same = __ballot(in);
  for (int b = 0; (a.adapters >> b) != 0; b++) {
    const u64 set = __ballot((q.id >> b) & 1);
    q.same &= ((q.id >> b) & 1) ? set : ~set;
  }
  q.leaders = __ballot(in && (q.same & ((1ull << lane) - 1)) == 0);
  return q;
}

// The g-th distinct adapter of the block.
__device__ __forceinline__ Group find_group(const LoraArgs& a, const Rows& w, int g) {
  u64 leaders = w.leaders;
  for (int i = 0; i < g; i++) leaders &= leaders - 1;
  Group q{0, 0, 0, 0};
  if (!leaders) return q;
  const int lead = __builtin_amdgcn_readfirstlane(__builtin_ctzll(leaders));
  q.id = __builtin_amdgcn_readlane(w.id, lead);
  q.rows = (u64)(u32)__builtin_amdgcn_readlane((int)(u32)w.same, lead) |
           (u64)(u32)__builtin_amdgcn_readlane((int)(u32)(w.same >> 32), lead) << 32;
  if (q.id < a.adapters) {
    int o, e;
    if (a.adapters < 64) {
      o = __builtin_amdgcn_readlane(w.offsets, q.id);
      e = __builtin_amdgcn_readlane(w.offsets, q.id + 1);
    } else {
      o = a.offsets[q.id];
      e = a.offsets[q.id + 1];
    }
    // anything but a whole rank inside the pool counts as no adapter
    if (o >= 0 && e > o && e <= a.total_rank && e - o <= a.max_rank && o % 8 == 0 &&
        (e - o) % 8 == 0) {
      q.off = o;
      q.r = e - o;
    }
  }
  return q;
}

// list[j] = the block row of the group's j-th row (all waves write the same)
__device__ __forceinline__ int list_rows(u64 rows, unsigned char* list) {
  const int lane = threadIdx.x & 63;
  if ((rows >> lane) & 1) list[__popcll(rows & ((1ull << lane) - 1))] = (unsigned char)lane;
  return __popcll(rows);
}

// Products of 16 A rows with TILES tiles of 16 activation rows over a wave's
// share of K: rounds of 128 columns, every `stride`-th one.  MFMA: A operand =
// adapter rows, B operand = activation rows, so a lane ends with four
// consecutive rank entries of one row.  The 16-byte loads of U rounds are asked
// for before their first product.  (Rounds are dealt out in turn because rows are
// a power of two apart: waves that walk ranges of their own would all ask the
// same memory channel.)
template <int TILES, int U>
__device__ __forceinline__ void down_rounds(const _Float16* ap, const _Float16* const* xp, int K,
                                            int first, int stride, f4* acc) {
  const int h = (threadIdx.x & 63) >> 4;
  const int rounds = (K + 127) / 128;
  for (int q = first; q < rounds; q += U * stride) {
    h8 av[U][4], xv[U][4][TILES];
#pragma unroll
    for (int u = 0; u < U; u++) {
#pragma unroll
      for (int s = 0; s < 4; s++) {
        const int k = (q + u * stride) * 128 + s * 32;
        const bool in = k + 8 * h < K;  // K is a multiple of 8
        av[u][s] = h8{0, 0, 0, 0, 0, 0, 0, 0};
        if (in) av[u][s] = *reinterpret_cast<const h8*>(ap + k);
#pragma unroll
        for (int i = 0; i < TILES; i++) {
          xv[u][s][i] = h8{0, 0, 0, 0, 0, 0, 0, 0};
          if (in) xv[u][s][i] = *reinterpret_cast<const h8*>(xp[i] + k);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; u++)
#pragma unroll
      for (int s = 0; s < 4; s++)
#pragma unroll
        for (int i = 0; i < TILES; i++)
          acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(av[u][s], xv[u][s][i], acc[i], 0, 0, 0);
  }
}

// t of one rank tile (16 A rows) for a group's rows, over one share of K, TB
// tiles of 16 rows at a time.  The four waves' sums are added in wave order
// through LDS.
template <int TB>
__global__ void __launch_bounds__(256, TB == 1 ? 4 : 3)
k_lora_down(const LoraBatch bt, const LoraArgs a) {
  __shared__ unsigned char list[ROWS];
  __shared__ f4 part[4][TB][64];
  const int blocks = (a.M + ROWS - 1) / ROWS;
  const int pi = blockIdx.y / blocks;
  const LoraProblem& p = bt.p[pi];
  const int base = (blockIdx.y % blocks) * ROWS;
  const int rt = blockIdx.x / a.splits, sp = blockIdx.x % a.splits;
  const Rows rows = load_rows(a, base);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l16 = lane & 15, h = lane >> 4;
  for (int gi = blockIdx.z;; gi += gridDim.z) {
    const Group g = find_group(a, rows, gi);
    if (!g.rows) return;
    if (rt * 16 >= g.r) continue;
    const int cnt = list_rows(g.rows, list);
    __syncthreads();
    const int K = p.K;
    // rows past the rank or the group repeat a valid one; their results are not stored
    const _Float16* ap = p.a + (size_t)(g.off + min(rt * 16 + l16, g.r - 1)) * K + 8 * h;
    for (int c0 = 0; c0 < cnt; c0 += 16 * TB) {
      const int tiles = min((cnt - c0 + 15) / 16, TB);
      const _Float16* xp[TB];
#pragma unroll
      for (int i = 0; i < TB; i++)
        xp[i] = p.x + (size_t)(base + list[min(c0 + i * 16 + l16, cnt - 1)]) * K + 8 * h;
      f4 acc[TB];
#pragma unroll
      for (int i = 0; i < TB; i++) acc[i] = f4{0, 0, 0, 0};
      const int first = sp * 4 + wave, stride = 4 * a.splits;
      if constexpr (TB == 1) {
        down_rounds<1, 2>(ap, xp, K, first, stride, acc);
      } else {
        if (tiles == 1) down_rounds<1, 2>(ap, xp, K, first, stride, acc);
        else if (tiles == 2) down_rounds<2, 1>(ap, xp, K, first, stride, acc);
        else down_rounds<4, 1>(ap, xp, K, first, stride, acc);
      }
#pragma unroll
      for (int i = 0; i < TB; i++)
        if (i < tiles) part[wave][i][lane] = acc[i];
      __syncthreads();
      // wave i finishes row tile i
      if (wave < tiles) {
        f4 sum = part[0][wave][lane];
#pragma unroll
        for (int w = 1; w < 4; w++) sum += part[w][wave][lane];
        const int j = c0 + wave * 16 + l16;
        if (j < cnt) {
          const size_t row = ((size_t)pi * a.splits + sp) * a.M + base + list[j];
          *reinterpret_cast<f4*>(a.ws + row * a.rank_ld + rt * 16 + 4 * h) = sum;
        }
      }
      __syncthreads();  // before the next sums, or the next group's list
    }
  }
}

// The group's rows times B, TB tiles of 16 rows at a time; a wave has UT tiles
// of 16 outputs, a workgroup eight times that.  A tile of rows goes through LDS
// on its way out, so that a wave reads and writes y in whole rows of 1 KiB: as
// the products lie in its lanes, an access would take 64 bytes of each of 16
// rows.
constexpr int UP_WAVES = 8;
constexpr int UP_ROWS = 16 / UP_WAVES;  // rows of a tile a wave takes out
typedef float f4u __attribute__((ext_vector_type(4), aligned(4)));

template <int UT>
struct Up {
  static constexpr int N = UP_WAVES * UT * 16;  // outputs of a workgroup
  static constexpr int Q = N / 256;             // 16-byte accesses of a lane to a row
  static constexpr int LD = N + 4;              // floats between rows of a tile in LDS
};

template <int KS, int TB, int UT>  // k steps of 32: the rank is at most 32 KS
struct UpShared {
  static constexpr int LD = 32 * KS + 8;  // halves; rows start 16 bytes apart in bank order
  float out[16 * Up<UT>::LD];
  _Float16 hi[16 * TB * LD], lo[16 * TB * LD];
  float back[16 * TB];  // 2^x s_i
  unsigned char list[ROWS];
};

template <int KS, int TB, int UT, bool PAST>  // PAST: y goes past the caches
__device__ __forceinline__ void up_body(const LoraProblem& p, const LoraArgs& a, const Group& g,
                                        int pi, int base, int n0, int cnt, UpShared<KS, TB, UT>& sh) {
  constexpr int LD = UpShared<KS, TB, UT>::LD, Q = Up<UT>::Q;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int l16 = lane & 15, h = lane >> 4;
  const int N = p.N;
  const int nw = n0 + wave * (UT * 16);
  const _Float16* bblock = p.b + (size_t)g.off * N;  // [N][r]
  const int n = n0 + 4 * lane;  // this lane's outputs of a whole row, and 256 on
  for (int c0 = 0; c0 < cnt; c0 += 16 * TB) {
    const int rows = min(cnt - c0, 16 * TB), tiles = (rows + 15) / 16;
    // t of all rows, asked for first: loads come back in order, and t is needed
    // before the others.  LT lanes a row, four entries a lane
    constexpr int LT = 8 * KS, PASS = 64 * UP_WAVES / LT, PASSES = (16 * TB + PASS - 1) / PASS;
    const int e = 4 * (tid % LT);
    f4 t[PASSES];
    const float* src[PASSES];
#pragma unroll
    for (int i = 0; i < PASSES; i++) {
      t[i] = f4{0, 0, 0, 0};
      const int j = min(c0 + i * PASS + tid / LT, cnt - 1);
      src[i] = a.ws + ((size_t)pi * a.splits * a.M + base + sh.list[j]) * a.rank_ld + e;
    }
    const size_t plane = (size_t)a.M * a.rank_ld;
    if (e < g.r) {  // ranks are multiples of 8; the shares of K in a fixed order
      constexpr int AHEAD = PASSES == 1 ? 4 : 2;  // shares asked for together
      for (int s = 0; s < a.splits; s += AHEAD) {
        f4 v[AHEAD][PASSES];
#pragma unroll
        for (int u = 0; u < AHEAD; u++)
#pragma unroll
          for (int i = 0; i < PASSES; i++) {
            v[u][i] = f4{0, 0, 0, 0};
            if (s + u < a.splits && i * PASS < rows)
              v[u][i] = *reinterpret_cast<const f4*>(src[i] + (s + u) * plane);
          }
#pragma unroll
        for (int u = 0; u < AHEAD; u++)
#pragma unroll
          for (int i = 0; i < PASSES; i++) t[i] += v[u][i];
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    h8 bv[UT][KS];
#pragma unroll
    for (int nt = 0; nt < UT; nt++) {
      const _Float16* bp = bblock + (size_t)min(nw + nt * 16 + l16, N - 1) * g.r + 8 * h;
#pragma unroll
      for (int k = 0; k < KS; k++) {
        bv[nt][k] = h8{0, 0, 0, 0, 0, 0, 0, 0};
        if (32 * k + 8 * h < g.r) bv[nt][k] = *reinterpret_cast<const h8*>(bp + 32 * k);
      }
    }
    // rows c0 + i * 16 + wave * UP_ROWS + q of the group
    f4 y[TB][UP_ROWS][Q];
#pragma unroll
    for (int i = 0; i < TB; i++) {
#pragma unroll
      for (int q = 0; q < UP_ROWS; q++) {
        const int j = c0 + i * 16 + wave * UP_ROWS + q;
        const float* src = p.y_in + (size_t)(base + sh.list[min(j, cnt - 1)]) * N;
#pragma unroll
        for (int w = 0; w < Q; w++) {
          const int nw = n + 256 * w;
          y[i][q][w] = f4{0, 0, 0, 0};
          if (!p.y_in || j >= cnt) continue;
          if (nw + 4 <= N) {
            const f4u* const at = reinterpret_cast<const f4u*>(src + nw);
            if constexpr (PAST) y[i][q][w] = __builtin_nontemporal_load(at);
            else y[i][q][w] = *at;
          } else {
#pragma unroll
            for (int c = 0; c < 3; c++)
              if (nw + c < N) y[i][q][w][c] = src[nw + c];
          }
        }
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    const float scale = a.scales ? a.scales[g.id] : 1.0f;
#pragma unroll
    for (int i = 0; i < PASSES; i++) {
      if (i * PASS >= rows) break;
      float big = fmaxf(fmaxf(fabsf(t[i][0]), fabsf(t[i][1])), fmaxf(fabsf(t[i][2]), fabsf(t[i][3])));
#pragma unroll
      for (int d = LT / 2; d > 0; d >>= 1) big = fmaxf(big, __shfl_xor(big, d, 64));
      // 2^x with big / 2^x in [0.5, 1); 1 where big is zero; beside an infinity no
      // finite entry may become one (their difference would be NaN)
      int x = 128;
      if (big < __builtin_inff()) x = __builtin_amdgcn_frexp_expf(big);
      const int j = i * PASS + tid / LT;
      h4 vh, vl;
#pragma unroll
      for (int c = 0; c < 4; c++) {
        const float u = ldexpf(t[i][c], 8 - x);  // [2^7, 2^8): lo stays a normal binary16 longer
        vh[c] = (_Float16)u;
        vl[c] = __builtin_isinf(u) ? (_Float16)0.0f : (_Float16)(u - (float)vh[c]);
      }
      if (j < rows) {  // past the rank t is zero
        *reinterpret_cast<h4*>(&sh.hi[j * LD + e]) = vh;
        *reinterpret_cast<h4*>(&sh.lo[j * LD + e]) = vl;
        if (e == 0) sh.back[j] = ldexpf(scale, x - 8);
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TB; i++) {
      if (i >= tiles) break;
      const int j = min(i * 16 + l16, rows - 1);
      f4 acc[UT];
#pragma unroll
      for (int nt = 0; nt < UT; nt++) acc[nt] = f4{0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < KS; k++) {
        const h8 tl = *reinterpret_cast<const h8*>(&sh.lo[j * LD + 32 * k + 8 * h]);
        const h8 th = *reinterpret_cast<const h8*>(&sh.hi[j * LD + 32 * k + 8 * h]);
#pragma unroll
        for (int nt = 0; nt < UT; nt++) {
          acc[nt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(bv[nt][k], tl, acc[nt], 0, 0, 0);
          acc[nt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(bv[nt][k], th, acc[nt], 0, 0, 0);
        }
      }
      const float f = sh.back[j];
#pragma unroll
      for (int nt = 0; nt < UT; nt++)
        *reinterpret_cast<f4*>(&sh.out[l16 * Up<UT>::LD + wave * (UT * 16) + nt * 16 + 4 * h]) =
            acc[nt] * f;
      __syncthreads();
#pragma unroll
      for (int q = 0; q < UP_ROWS; q++) {
        const int jr = wave * UP_ROWS + q;
        if (i * 16 + jr >= rows) continue;
        float* dst = p.y + (size_t)(base + sh.list[c0 + i * 16 + jr]) * N;
#pragma unroll
        for (int w = 0; w < Q; w++) {
          const int nw = n + 256 * w;
          const f4 v = y[i][q][w] +
                       *reinterpret_cast<const f4*>(&sh.out[jr * Up<UT>::LD + 256 * w + 4 * lane]);
          if (nw + 4 <= N) {
            f4u* const at = reinterpret_cast<f4u*>(dst + nw);
            if constexpr (PAST) __builtin_nontemporal_store((f4u)v, at);
            else *at = (f4u)v;
          } else {
#pragma unroll
            for (int c = 0; c < 3; c++)
              if (nw + c < N) dst[nw + c] = v[c];
          }
        }
      }
      if (i + 1 < tiles) __syncthreads();  // before the next tile is put in place
    }
    __syncthreads();  // before the next rows
  }
}

template <int KS, int TB, int UT, bool PAST>  // KS: enough for the call's largest rank
__global__ void __launch_bounds__(64 * UP_WAVES)
k_lora_up(const LoraBatch bt, const LoraArgs a) {
  __shared__ __align__(16) UpShared<KS, TB, UT> sh;
  const int blocks = (a.M + ROWS - 1) / ROWS;
  const int pi = blockIdx.y / blocks;
  const LoraProblem& p = bt.p[pi];
  const int base = (blockIdx.y % blocks) * ROWS;
  const int N = p.N, n0 = blockIdx.x * Up<UT>::N;
  if (n0 >= N) return;  // problems of a call may differ in N
  const Rows rows = load_rows(a, base);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int gi = blockIdx.z;; gi += gridDim.z) {
    const Group g = find_group(a, rows, gi);
    if (!g.rows) return;
    const int cnt = list_rows(g.rows, sh.list);
    __syncthreads();
    if (g.r != 0) {
      up_body<KS, TB, UT, PAST>(p, a, g, pi, base, n0, cnt, sh);
    } else if (p.y_in != p.y) {  // no adapter: y = y_in
      const int nn = min(Up<UT>::N, N - n0);
      for (int j = wave; j < cnt; j += UP_WAVES) {
        const size_t at = (size_t)(base + sh.list[j]) * N + n0;
        for (int n = lane; n < nn; n += 64) p.y[at + n] = p.y_in ? p.y_in[at + n] : 0.0f;
      }
    }
    __syncthreads();  // before the next group's list and rows
  }
}

}  // namespace

// Shares of K over workgroups: about LORA_WORKGROUPS workgroups in all, with
// two rounds of 128 columns for each of their four waves (one batch of loads;
// smaller shares cost the second launch more than they save here).  Of several
// blocks of rows, most are taken to have one adapter, as prompts do (1800 rows
// of 24 adapters of rank 32, three projections 4096x4096: 69 us; as for a block
// of requests, one adapter a row, 83 us).
int lora_splits(int count, int M, int K, int adapters, int max_rank) {
  const int each = M > ROWS ? 1 : M < adapters ? M : adapters;  // adapters of a block
  const long long wgs =
      (long long)count * ((M + ROWS - 1) / ROWS) * ((max_rank + 15) / 16) * each;
  long long s = LORA_WORKGROUPS / (wgs > 0 ? wgs : 1);
  if (s > (K + 1023) / 1024) s = (K + 1023) / 1024;
  if (s > LORA_MAX_SPLITS) s = LORA_MAX_SPLITS;
  return s < 1 ? 1 : (int)s;
}

hipError_t launch_lora(const LoraBatch& bt, const LoraArgs& a, hipStream_t s) {
  const int blocks = (a.M + ROWS - 1) / ROWS;
  int groups = a.M < ROWS ? a.M : ROWS;
  if (groups - 1 > a.adapters) groups = a.adapters + 1;
  // the more blocks of rows, the fewer workgroups for a block's groups: each
  // then takes several, where there are several, instead of most finding none
  // (prompts: a block's rows mostly share an adapter or two)
  if (blocks > 1) groups = std::min(groups, std::max(2, 128 / blocks));
  int n = 0;
  for (int i = 0; i < bt.count; i++) n = bt.p[i].N > n ? bt.p[i].N : n;
  // Groups are the slow index: where most blocks have one or two, the
  // workgroups that find rows are neighbours and spread over all CUs.
  const dim3 down(a.splits * (a.rank_ld / 16), bt.count * blocks, groups);
  // Few rows an adapter (16 at a time, more workgroups per CU) or many (64).
  // With few, a wave takes four tiles of 16 outputs for more of B in flight (64
  // rows, 48 adapters of rank 32 or 16, 4096x4096: 22.1 -> 16.6 us), two where
  // that would leave CUs without work (one row, 768x768: 7.2 against 7.7 us).
  const bool few = blocks == 1 && (a.M <= 16 || a.adapters >= (a.M + 7) / 8);
  const bool wide = few && (long long)n * bt.count * groups >= 256 * Up<4>::N;
  const int per = wide ? Up<4>::N : Up<2>::N;
  const dim3 up((n + per - 1) / per, bt.count * blocks, groups);
  // The next call reads y, so it stays in the caches unless it is much of the
  // last level's 256 MB (past the caches / through them, 32 requests on r/k/v with
  // rq_wkv7 as y's reader 39.7 / 37.4 us, 64 52.2 / 48.2; 16384 outputs with a
  // squared ReLU as the reader: 128 rows 30.3 / 28.9 us, 512 57.6 / 56.5, 1024 94.6
  // / 95.4, 1400 129 / 133, 2047 190 / 198).
  size_t y_bytes = 0;
  for (int i = 0; i < bt.count; i++) y_bytes += (size_t)a.M * bt.p[i].N * sizeof(float);
  const bool past = y_bytes > (64u << 20);
#define RQ_LORA_UP(KS)                                                                          \
  do {                                                                                          \
    const dim3 th(64 * UP_WAVES);                                                               \
    if (wide) hipLaunchKernelGGL((k_lora_up<KS, 1, 4, false>), up, th, 0, s, bt, a);            \
    else if (few) hipLaunchKernelGGL((k_lora_up<KS, 1, 2, false>), up, th, 0, s, bt, a);        \
    else if (past) hipLaunchKernelGGL((k_lora_up<KS, 4, 2, true>), up, th, 0, s, bt, a);        \
    else hipLaunchKernelGGL((k_lora_up<KS, 4, 2, false>), up, th, 0, s, bt, a);                 \
  } while (0)
  if (few) hipLaunchKernelGGL(k_lora_down<1>, down, dim3(256), 0, s, bt, a);
  else hipLaunchKernelGGL(k_lora_down<4>, down, dim3(256), 0, s, bt, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (a.max_rank <= 32) RQ_LORA_UP(1);
  else if (a.max_rank <= 64) RQ_LORA_UP(2);
  else RQ_LORA_UP(4);
#undef RQ_LORA_UP
  return hipGetLastError();
}

}  // namespace rq
