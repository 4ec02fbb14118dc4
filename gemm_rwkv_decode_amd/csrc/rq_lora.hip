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
#include "rq_common.h"
#include "rq_internal.h"

namespace rq {
namespace {

constexpr int ROWS = 64;  // rows of a block: one per lane
constexpr int UP_N = 256; // outputs of a workgroup of k_lora_up

typedef unsigned long long u64;

// The lanes' rows that share the g-th distinct adapter of a block.
struct Group {
  u64 rows;    // 0: the block has no g-th adapter
  int id;      // a.adapters: no adapter
  int off, r;  // its first A row and its rank (0: no adapter)
};

__device__ __forceinline__ Group find_group(const LoraArgs& a, int base, int g) {
  const int lane = threadIdx.x & 63;
  const bool in = base + lane < a.M;
  int id = in ? a.ids[base + lane] : 0;
  if (id < 0 || id > a.adapters) id = a.adapters;
  u64 same = __ballot(in);
  const u64 all = same;
  for (int b = 0; (a.adapters >> b) != 0; b++) {
    const u64 set = __ballot((id >> b) & 1);
    same &= ((id >> b) & 1) ? set : ~set;
  }
  u64 leaders = __ballot(in && (same & ((1ull << lane) - 1)) == 0) & all;
  for (int i = 0; i < g; i++) leaders &= leaders - 1;
  Group q{0, 0, 0, 0};
  if (!leaders) return q;
  const int lead = __builtin_amdgcn_readfirstlane(__builtin_ctzll(leaders));
  q.id = __builtin_amdgcn_readlane(id, lead);
  q.rows = __ballot(in && id == q.id);
  if (q.id < a.adapters) {
    const int o = a.offsets[q.id], e = a.offsets[q.id + 1];
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

// t of one rank tile (16 A rows) for a group's rows, over one K range.  The
// four waves split the range; their sums are added in wave order through LDS.
// MFMA: A operand = adapter rows, B operand = activation rows, so a lane ends
// with four consecutive rank entries of one row.
__global__ void __launch_bounds__(256)
k_lora_down(const LoraBatch bt, const LoraArgs a) {
  __shared__ unsigned char list[ROWS];
  __shared__ f4 part[4][4][64];
  const int blocks = (a.M + ROWS - 1) / ROWS;
  const LoraProblem& p = bt.p[blockIdx.z / blocks];
  const int base = (blockIdx.z % blocks) * ROWS;
  const int rt = blockIdx.x / a.splits, sp = blockIdx.x % a.splits;
  const Group g = find_group(a, base, blockIdx.y);
  if (rt * 16 >= g.r) return;
  const int cnt = list_rows(g.rows, list);
  __syncthreads();
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l16 = lane & 15, h = lane >> 4;
  const int tiles = (cnt + 15) / 16;
  const int K = p.K;
  const int steps = (K + 31) / 32;
  const int ranges = 4 * a.splits, mine = sp * 4 + wave;
  const int s0 = (int)((long long)steps * mine / ranges);
  const int s1 = (int)((long long)steps * (mine + 1) / ranges);
  // rows past the rank or the group repeat a valid one; their results are not stored
  const _Float16* ap = p.a + (size_t)(g.off + min(rt * 16 + l16, g.r - 1)) * K + 8 * h;
  const _Float16* xp[4];
#pragma unroll
  for (int i = 0; i < 4; i++)
    xp[i] = p.x + (size_t)(base + list[min(i * 16 + l16, cnt - 1)]) * K + 8 * h;
  f4 acc[4];
#pragma unroll
  for (int i = 0; i < 4; i++) acc[i] = f4{0, 0, 0, 0};
  for (int s = s0; s < s1; s++) {
    const int k = s * 32;
    const bool in = k + 8 * h < K;  // K is a multiple of 8
    h8 av = {0, 0, 0, 0, 0, 0, 0, 0};
    if (in) av = *reinterpret_cast<const h8*>(ap + k);
#pragma unroll
    for (int i = 0; i < 4; i++) {
      if (i < tiles) {
        h8 xv = {0, 0, 0, 0, 0, 0, 0, 0};
        if (in) xv = *reinterpret_cast<const h8*>(xp[i] + k);
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(av, xv, acc[i], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; i++)
    if (i < tiles) part[wave][i][lane] = acc[i];
  __syncthreads();
  // wave i finishes row tile i
  if (wave >= tiles) return;
  f4 sum = part[0][wave][lane];
#pragma unroll
  for (int w = 1; w < 4; w++) sum += part[w][wave][lane];
  const int j = wave * 16 + l16;
  if (j < cnt) {
    const size_t row = ((size_t)(blockIdx.z / blocks) * a.splits + sp) * a.M + base + list[j];
    *reinterpret_cast<f4*>(a.ws + row * a.rank_ld + rt * 16 + 4 * h) = sum;
  }
}

// The group's rows times B: 256 outputs a workgroup, 64 a wave.
__global__ void __launch_bounds__(256)
k_lora_up(const LoraBatch bt, const LoraArgs a) {
  constexpr int LD = LORA_MAX_RANK + 8;  // halves; rows start 16 bytes apart in bank order
  __shared__ unsigned char list[ROWS];
  __shared__ __align__(16) _Float16 hi[ROWS][LD], lo[ROWS][LD];
  __shared__ float back[ROWS];  // 2^e s_i
  const int blocks = (a.M + ROWS - 1) / ROWS;
  const int pi = blockIdx.z / blocks;
  const LoraProblem& p = bt.p[pi];
  const int base = (blockIdx.z % blocks) * ROWS;
  const int N = p.N, n0 = blockIdx.x * UP_N;
  if (n0 >= N) return;  // problems of a call may differ in N
  const Group g = find_group(a, base, blockIdx.y);
  if (!g.rows) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int cnt = list_rows(g.rows, list);
  __syncthreads();
  if (g.r == 0) {  // no adapter: y = y_in
    if (p.y_in == p.y) return;
    const int nn = min(UP_N, N - n0);
    for (int j = wave; j < cnt; j += 4) {
      const size_t at = (size_t)(base + list[j]) * N + n0;
      for (int n = lane; n < nn; n += 64) p.y[at + n] = p.y_in ? p.y_in[at + n] : 0.0f;
    }
    return;
  }
  const float scale = a.scales ? a.scales[g.id] : 1.0f;
  const int rpad = (g.r + 31) / 32 * 32;  // the k steps of the MFMAs
  // a wave per row: add the K ranges, find the row's power of two, split
  for (int j = wave; j < cnt; j += 4) {
    const float* t0 = a.ws + ((size_t)pi * a.splits * a.M + base + list[j]) * a.rank_ld;
    float t[LORA_MAX_RANK / 64];
    float big = 0.0f;
#pragma unroll
    for (int i = 0; i < LORA_MAX_RANK / 64; i++) {
      const int e = i * 64 + lane;
      float sum = 0.0f;
      if (e < g.r)
        for (int s = 0; s < a.splits; s++) sum += t0[(size_t)s * a.M * a.rank_ld + e];
      t[i] = sum;
      big = fmaxf(big, fabsf(sum));
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) big = fmaxf(big, __shfl_xor(big, d, 64));
    // 2^e with big / 2^e in [0.5, 1); 1 where big is zero or not finite
    int e = 0;
    if (big > 0.0f && big < __builtin_inff()) e = __builtin_amdgcn_frexp_expf(big);
#pragma unroll
    for (int i = 0; i < LORA_MAX_RANK / 64; i++) {
      const int c = i * 64 + lane;
      if (c < rpad) {
        const float u = ldexpf(t[i], 8 - e);  // [2^7, 2^8): lo stays a normal binary16 longer
        const _Float16 uh = (_Float16)u;
        hi[j][c] = uh;
        lo[j][c] = __builtin_isinf(u) ? (_Float16)0.0f : (_Float16)(u - (float)uh);
      }
    }
    if (lane == 0) back[j] = ldexpf(scale, e - 8);
  }
  __syncthreads();
  const int l16 = lane & 15, h = lane >> 4;
  const int tiles = (cnt + 15) / 16;
  const _Float16* bblock = p.b + (size_t)g.off * N;  // [N][r]
  for (int nt = 0; nt < UP_N / 64; nt++) {
    const int n16 = n0 + wave * (UP_N / 4) + nt * 16;
    if (n16 >= N) break;
    const _Float16* bp = bblock + (size_t)min(n16 + l16, N - 1) * g.r + 8 * h;
    f4 acc[4];
#pragma unroll
    for (int i = 0; i < 4; i++) acc[i] = f4{0, 0, 0, 0};
    for (int k = 0; k < g.r; k += 32) {
      h8 bv = {0, 0, 0, 0, 0, 0, 0, 0};
      if (k + 8 * h < g.r) bv = *reinterpret_cast<const h8*>(bp + k);
#pragma unroll
      for (int i = 0; i < 4; i++) {
        if (i < tiles) {
          const int j = min(i * 16 + l16, cnt - 1);
          const h8 tl = *reinterpret_cast<const h8*>(&lo[j][k + 8 * h]);
          const h8 th = *reinterpret_cast<const h8*>(&hi[j][k + 8 * h]);
          acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(bv, tl, acc[i], 0, 0, 0);
          acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(bv, th, acc[i], 0, 0, 0);
        }
      }
    }
    // lane: row i*16 + l16, outputs n16 + 4 h .. + 3
    const int n = n16 + 4 * h;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int j = i * 16 + l16;
      if (i < tiles && j < cnt && n < N) {
        const size_t at = (size_t)(base + list[j]) * N + n;
        const float f = back[j];
        if (N % 4 == 0) {
          f4 v = f4{0, 0, 0, 0};
          if (p.y_in) v = *reinterpret_cast<const f4*>(p.y_in + at);
#pragma unroll
          for (int c = 0; c < 4; c++) v[c] += f * acc[i][c];
          *reinterpret_cast<f4*>(p.y + at) = v;
        } else {
#pragma unroll
          for (int c = 0; c < 4; c++)
            if (n + c < N) p.y[at + c] = (p.y_in ? p.y_in[at + c] : 0.0f) + f * acc[i][c];
        }
      }
    }
  }
}

}  // namespace

// K ranges over workgroups: about 512 workgroups in all, at least 256 columns
// of K each (2 steps a wave).
int lora_splits(int count, int M, int K, int adapters, int max_rank) {
  const int rows = M < ROWS ? M : ROWS;
  const long long wgs = (long long)count * ((M + ROWS - 1) / ROWS) * ((max_rank + 15) / 16) *
                        (rows < adapters ? rows : adapters);
  long long s = 512 / (wgs > 0 ? wgs : 1);
  if (s > K / 256) s = K / 256;
  if (s > LORA_MAX_SPLITS) s = LORA_MAX_SPLITS;
  return s < 1 ? 1 : (int)s;
}

hipError_t launch_lora(const LoraBatch& bt, const LoraArgs& a, hipStream_t s) {
  const int blocks = (a.M + ROWS - 1) / ROWS;
  int groups = a.M < ROWS ? a.M : ROWS;
  if (groups > a.adapters + 1) groups = a.adapters + 1;
  int n = 0;
  for (int i = 0; i < bt.count; i++) n = bt.p[i].N > n ? bt.p[i].N : n;
  hipLaunchKernelGGL(k_lora_down, dim3(a.splits * (a.rank_ld / 16), groups, bt.count * blocks),
                     dim3(256), 0, s, bt, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_lora_up, dim3((n + UP_N - 1) / UP_N, groups, bt.count * blocks), dim3(256),
                     0, s, bt, a);
  return hipGetLastError();
}

}  // namespace rq
