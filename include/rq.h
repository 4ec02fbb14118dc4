/*
 * rq.h -- C interface of librq: group-wise low-bit weight dequantization and
 * dequantize-and-multiply (GEMV / small-M GEMM) on AMD Instinct MI355X (gfx950).
 *
 * The operation.  A weight matrix W with N rows (outputs) and K columns
 * (inputs) is stored as packed integer codes q[n][k] plus per-group scale
 * material; rows are [out][in], as the FFN key (16384x4096) and FFN value
 * (4096x16384) of a width-4096 RWKV-7 model are listed on the package page
 * "RWKV-7 FP8 Quantized Inference" (section "Operator Optimization Details").
 * Five storage formats are supported:
 *
 *   RQ_LAYOUT_SYM, bits = 4, group in {32, 64, 128}
 *       The 4-bit symmetric format with one scale per group of consecutive
 *       weights of a row; group 64 is the format of the model card
 *       "RWKV-7 G1 1.5B -- int4 GPTQ for rwkv-sglang" (opening paragraph,
 *       section "Format & loading").  qweight: uint8 [N][K/2], two codes per
 *       byte, the even k in bits 0-3, each code a 4-bit two's complement
 *       integer (-8..7).  scales: IEEE binary16 [N][K/group].  w = s * q.
 *   RQ_LAYOUT_SYM, bits = 8, group in {16, 32, 64}
 *       The 8-bit symmetric projection format of the REDUCTION preset (group
 *       16) in the news article "rwkv-quant: keeping one matrix in bf16 ..."
 *       (section "Two presets and six sizes").  qweight: int8 [N][K] two's
 *       complement.  scales: binary16 [N][K/group].  w = s * q.
 *   RQ_LAYOUT_ASYM_SB, bits = 4, group = 32
 *       The 4-bit asymmetric superblock projection format of the COMPRESSION
 *       preset (same article and section): each 32-wide group has its own
 *       scale and shift.  qweight: uint8 [N][K/2], unsigned codes 0..15, even
 *       k in bits 0-3.  A superblock is 256 consecutive k of one row (eight
 *       groups).  scales: [N][K/256] records of 8 bytes: binary16 d in bytes
 *       0-1 (little endian), then eight 6-bit unsigned sub-scales sc_j packed
 *       LSB-first in the 48-bit little-endian field of bytes 2-7 (sc_j at bits
 *       6j..6j+5).  zeros: records of the same shape holding m and the
 *       sub-mins mn_j.  With j = (k mod 256)/32:
 *       w = (d * sc_j) * q - (m * mn_j).
 *   RQ_LAYOUT_ASYM_SB, bits = 5 or 6, group = 32
 *       The same superblock layout with 5- or 6-bit unsigned codes (0..31,
 *       0..63): the FFN key and head in 5 bits (COMPRESSION) and the FFN in
 *       6 bits (REDUCTION), same article and section; the pages give the
 *       widths only, the storage below is ours.  qweight holds two planes: the
 *       low 4 bits of every code exactly as the 4-bit layout stores them
 *       ([N][K/2]), then the high bits, [N][K*(bits-4)/8] bytes: per row, per
 *       32-code chunk, 1 (5-bit) or 2 (6-bit) little-endian dwords.  Code
 *       8i + j of a chunk (i = 0..3, j = 0..7), with base = (j >= 4 ? 16 : 0)
 *       + (j even ? 4 : 8) and g = (j mod 4)/2, keeps bit 4 at bit
 *       base + (g == 0 ? i - 4 : i + 4) of the dword (5-bit), or bits 4 and 5
 *       at bits base + s and base + 1 + s of dword i/2 with s = -4, -2, 4, 6
 *       for (i mod 2, g) = (0,0), (0,1), (1,0), (1,1) (6-bit).
 *   RQ_LAYOUT_FP8_TENSOR, bits = 8, group = 0
 *       FP8 E4M3 weights with one binary32 scale for the whole matrix, the
 *       format of the package page "RWKV-7 FP8 Quantized Inference" (sections
 *       "Core Approach: Full FP8, No Residuals" and "Quantization Principle";
 *       the scale is fp32 per section "Quantization Metadata Format"), used
 *       here as weight-only quantization (binary16 activations).  qweight:
 *       uint8 [N][K], each byte an OCP E4M3 value (bias 7, 3 fraction bits,
 *       subnormals, no infinities, S.1111.111 = NaN, largest finite 448).
 *       scales: one float (binary32).  zeros: NULL.  w = fp8 * scale.
 *
 * Every dequantized weight is the binary32 value nearest (ties to even) the
 * exact value of its formula; for these formats that value is the same however
 * the products are grouped, so there is exactly one right answer.
 *
 * Pointers.  Every pointer is device memory owned by the caller and must be
 * 16-byte aligned.  Each operand (packed codes, scales, x, y) must be smaller
 * than 2 GiB (RQ_ERR_SHAPE otherwise).  The library never allocates or frees
 * device memory, does not retain caller memory between calls (a workspace
 * is passed in: rq_gemm_smallm_ws), never copies to the host and never
 * synchronizes: work is
 * enqueued on `stream`
 * (a hipStream_t; NULL means the null stream) and the call returns after the
 * enqueue.  Outputs must not overlap any input.
 *
 * Errors.  Arguments are validated on the host before any HIP call, so a call
 * that returns an error other than RQ_ERR_LAUNCH or RQ_ERR_DEVICE has
 * enqueued nothing.  A kernel fault is reported by the caller's next
 * synchronization, as for any asynchronous HIP work.  No exception crosses
 * this interface and nothing is printed.
 */
#ifndef RQ_H
#define RQ_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    RQ_OK = 0,
    RQ_ERR_NULL = 1,        /* a required pointer is NULL                       */
    RQ_ERR_SHAPE = 2,       /* M, N, K or group violate the shape rules         */
    RQ_ERR_UNSUPPORTED = 3, /* (layout, bits, group, out_kind) not supported    */
    RQ_ERR_ALIGN = 4,       /* a pointer is not 16-byte aligned                 */
    RQ_ERR_LAUNCH = 5,      /* the kernel launch was rejected by the runtime    */
    RQ_ERR_ALIAS = 6,       /* an output range overlaps an input range          */
    RQ_ERR_DEVICE = 7,      /* no usable gfx950 device                           */
    RQ_ERR_SCRATCH = 8      /* the split-K partial sums would not fit the
                               caller's workspace (rq_gemm_smallm_ws) or the
                               fixed array (rq_gemm_smallm_noalloc)              */
} rq_status;

typedef enum { RQ_LAYOUT_SYM = 0, RQ_LAYOUT_ASYM_SB = 1, RQ_LAYOUT_FP8_TENSOR = 2 } rq_layout;

typedef enum {
    RQ_OUT_F32 = 0,     /* binary32 weights [N][K]                               */
    RQ_OUT_CODES_I8 = 1 /* the integer codes as int8 [N][K]: -8..7 (4-bit sym),
                           -128..127 (8-bit), 0..15 (asymmetric)                 */
} rq_out_kind;

/* Largest M accepted by rq_gemv, rq_gemv_batched and rq_gemm_smallm. */
#define RQ_MAX_M 64

/* Largest number of problems in one rq_gemv_batched call. */
#define RQ_MAX_BATCH 64

/* One product y = x W^T of rq_gemv_batched (pointers as for rq_gemv). */
typedef struct {
    const void* qweight;
    const void* scales;
    const void* zeros;
    const void* x; /* binary16 [M][K] */
    float* y;      /* float [M][N], overwritten */
    int N;
    int K;
} rq_problem;

/*
 * rq_dequant -- unpack the codes of W, or dequantize W to binary32.
 * Defines the dequantization of the formats above (the model card's accuracy
 * paragraph reports that the serving kernel reproduces the offline dequant bit
 * for bit; this call is that offline dequant).
 *   out: RQ_OUT_F32 -> float [N][K]; RQ_OUT_CODES_I8 -> int8 [N][K] (not for
 *   RQ_LAYOUT_FP8_TENSOR, whose codes are not integers: RQ_ERR_UNSUPPORTED).
 *   zeros: NULL for RQ_LAYOUT_SYM and RQ_LAYOUT_FP8_TENSOR, required for
 *   RQ_LAYOUT_ASYM_SB.
 * Shape rules: N >= 1, K >= 1, K % group == 0 (group > 0), K*bits/8 % 16 == 0,
 * and for the asymmetric layout K % 256 == 0.
 */
rq_status rq_dequant(const void* qweight, const void* scales, const void* zeros,
                     void* out, int N, int K, int bits, int group, int layout,
                     int out_kind, void* stream);

/*
 * rq_gemv -- y[m][n] = sum_k x[m][k] * w[n][k] for 1 <= M <= RQ_MAX_M, where w
 * is the dequantized weight above (the weight-only decode product whose speed
 * the model card reports against fp16, section "Speed").
 *   x: binary16 [M][K] row-major.  y: float [M][N] row-major, overwritten.
 * Each output is within 1e-3 * sum_k |x[m][k] * w[n][k]| of the exact value
 * (fp32 accumulation).  The kernel is chosen per M, format and shape:
 * vector units at M <= 2 (a matrix-core kernel where K is too long for their
 * tuned launch shapes); from M = 3 on the small-batch matrix-core kernel of
 * rq_gemm_smallm (4 or 8 activation rows staged for M <= 4 or 8, else M
 * padded to a multiple of 16), or the matrix-core decode kernel where the
 * former does not take K and for one measured RWKV-7 shape at M = 3..4
 * (4-bit asymmetric 10240x2560); the vector units, in passes of up to 8
 * rows, wherever K suits neither and for one measured shape at M = 3..4
 * (int4 g64 2048x8192).  The small-batch kernel runs here with K whole:
 * this entry point never allocates or synchronizes.
 * Shape rules as for rq_dequant, plus 1 <= M <= RQ_MAX_M.
 */
rq_status rq_gemv(const void* qweight, const void* scales, const void* zeros,
                  const void* x, float* y, int M, int N, int K, int bits,
                  int group, int layout, void* stream);

/*
 * rq_gemv_batched -- `count` independent products, issued as few kernel
 * launches as possible: problems with the same K share one launch (up to 16
 * per launch on the vector-unit and decode kernels, up to 8 on the
 * small-batch matrix-core kernel).  Each group takes the kernel rq_gemv
 * would take for M, its K and its total row count; K is never split.
 * This is the grouped
 * form of the decode step's independent projections -- the package page
 * "RWKV-7 FP8 Quantized Inference" (section "Operator Optimization Details")
 * computes the receptance, key and value projections of a layer in a single
 * kernel.  All problems share M, bits, group and layout; N, K and the
 * pointers are per problem.  `problems` is a host array the call reads before
 * it returns.  No output may overlap another output or any input.
 * Errors as for rq_gemv; a failed call enqueues nothing.
 */
rq_status rq_gemv_batched(const rq_problem* problems, int count, int M, int bits,
                          int group, int layout, void* stream);

/*
 * rq_gemm_smallm -- the same product and contract as rq_gemv, computed on the
 * matrix cores (fp16 MFMA on exact integer or FP8 codes, fp32 per-group
 * scaling; FP8 sums are scaled once by the matrix scale).  This is the
 * batched-decode member of the kernel family the model card "RWKV-7 G1 1.5B --
 * int4 GPTQ for rwkv-sglang" names in its "Speed" line (a small-M GEMM next
 * to the GEMV, credited with beating fp16 at every batch up to 32).  Every
 * layout and code width, 5- and 6-bit codes included.
 * Tuned for 16 <= M <= 64 (batched decode); for M <= 4 or 8 only 4 or 8
 * activation rows are staged per round, otherwise M is padded to a multiple
 * of 16; it beats the vector units from M = 3 on.
 * This entry point keeps K whole: it has no workspace, and the library never
 * allocates, frees or synchronizes.  rq_gemm_smallm_ws below is the same call
 * with a caller-owned workspace, through which K may be split.
 */
rq_status rq_gemm_smallm(const void* qweight, const void* scales, const void* zeros,
                         const void* x, float* y, int M, int N, int K, int bits,
                         int group, int layout, void* stream);

/* The most workspace rq_gemm_smallm_ws ever uses (split-K arrival counters
 * and partial sums); a workspace of this size suits every call. */
#define RQ_GEMM_WORKSPACE_MAX_BYTES (64 << 20)

/*
 * rq_gemm_smallm_workspace_size -- *bytes = the workspace rq_gemm_smallm_ws
 * uses at these arguments: 0 where K is kept whole, at most
 * RQ_GEMM_WORKSPACE_MAX_BYTES.  Host-only (no device call); shape rules and
 * errors as for rq_gemm_smallm.
 */
rq_status rq_gemm_smallm_workspace_size(int M, int N, int K, int bits, int group,
                                        int layout, size_t* bytes);

/*
 * rq_gemm_smallm_ws -- rq_gemm_smallm with a workspace owned by the caller.
 * For long rows at small row counts the kernel splits K across workgroups
 * (more rows share each staged copy of x); the partial sums then go through
 * `workspace`, and the last workgroup to finish a 16-row tile adds them in a
 * fixed order, so results are deterministic.
 *   workspace: device memory, 16-byte aligned, of workspace_bytes bytes; the
 *   bytes the call uses (the size rq_gemm_smallm_workspace_size reports) must
 *   overlap no input and not y (RQ_ERR_ALIAS).  Its first 64 KiB (the arrival counters)
 *   must be zero before its first use; every call leaves them zero again, and
 *   the rest needs no clearing.  NULL keeps K whole (then workspace_bytes is
 *   ignored).
 * Errors as for rq_gemm_smallm, plus RQ_ERR_SCRATCH when a non-NULL workspace
 * is smaller than rq_gemm_smallm_workspace_size reports (nothing enqueued).
 * Calls that share one workspace must not overlap in time (calls on one
 * stream are ordered; graphs holding the same workspace must not be replayed
 * concurrently).  The library never allocates, frees or synchronizes.
 */
rq_status rq_gemm_smallm_ws(const void* qweight, const void* scales, const void* zeros,
                            const void* x, float* y, int M, int N, int K, int bits,
                            int group, int layout, void* workspace, size_t workspace_bytes,
                            void* stream);

/* Bytes of the fixed device array behind rq_gemm_smallm_noalloc. */
#define RQ_NOALLOC_SCRATCH_BYTES ((8 << 20) + (64 << 10))

/*
 * rq_gemm_smallm_noalloc -- rq_gemm_smallm for callers that cannot allocate
 * device memory (code under graph capture, tight serving loops, harnesses
 * that forbid allocation): the arguments of rq_gemm_smallm and the kernels,
 * arrangement, K split and results (bit for bit) of rq_gemm_smallm_ws with an
 * ample workspace, but the split-K arrival counters and
 * partial sums go to a fixed device array of RQ_NOALLOC_SCRATCH_BYTES that
 * the library holds on each GPU it runs on until the process ends.  The call
 * never allocates, frees or synchronizes.  The array covers every split the
 * automatic choice makes; a call whose partial sums would exceed it (only
 * with a forced split count) returns RQ_ERR_SCRATCH and enqueues nothing.
 * Every partial sum is written before it is read and every launch leaves the
 * counters at zero, so nothing needs clearing between calls, but all calls
 * on one GPU share the array: calls that may overlap in time on one GPU (on
 * different streams, or graphs replayed concurrently) race on it.
 */
rq_status rq_gemm_smallm_noalloc(const void* qweight, const void* scales, const void* zeros,
                                 const void* x, float* y, int M, int N, int K, int bits,
                                 int group, int layout, void* stream);

/*
 * Around the products.  The calls below do what a serving step needs next to
 * the packed projections: per-request adapters, the token shift, the state
 * recurrence and the treatment of the head's logits.  They keep the rules
 * above (caller-owned 16-byte-aligned device memory, host-side checks before
 * any HIP call, work enqueued on `stream`, no allocation, no
 * synchronization), with two differences: operands may exceed 2 GiB, and index
 * arrays (ids, offsets, slots, ...) are device memory of int32 with 4-byte
 * alignment.  Their contents are read on the device only, so they may change between
 * replays of a captured graph; every index read from them is checked there
 * against the sizes of the call, and what lies outside is treated as said at
 * each call, so no content makes a kernel leave its operands.
 *
 * A batch of sequences is described by offsets[sequences + 1]: sequence q is
 * the rows offsets[q] .. offsets[q+1] - 1 of the token arrays (0 <= offsets[0]
 * <= ... <= offsets[sequences] <= T); a sequence may be empty, one token, or a
 * prompt.  slots[q] is its row in a pool of nslots stored states, in which it
 * starts and to which it returns (slots NULL: slot q); a slot outside
 * 0 .. nslots-1 means a zero start and nothing stored.  Two sequences of a
 * call must not share a slot unless one is empty.
 */

/* Largest number of sequences in a call of rq_shift or rq_wkv7. */
#define RQ_MAX_SEQUENCES 65536

/* Largest T of rq_shift and rq_wkv7. */
#define RQ_MAX_TOKENS (1 << 24)

/* Largest n of rq_shift. */
#define RQ_SHIFT_MAX_MIXES 8

/*
 * rq_shift -- the token shift that makes the inputs of a layer's projections:
 *   out[i][t] = x[t] + (prev[t] - x[t]) * mu[i],   i < n,
 * prev[t] = x[t-1], or the stored row state[slot] for a sequence's first
 * token; then state[slot] = the sequence's last row.  A causal convolution of
 * two taps, n of them over one input (RWKV-7's time mix takes six).
 *   x: binary16 [T][D].  mu: binary16 [n][D].  state: binary16 [nslots][D].
 *   out: binary16 [n][T][D], computed in binary32 and rounded once.
 * Rows of x that no sequence covers leave unspecified rows in out.  A sequence
 * whose offsets leave 0 .. T does not begin: its slot is neither read nor written,
 * and its rows are mixed with the row before them in x (row 0 with zeros).
 * Shape rules: 1 <= T <= RQ_MAX_TOKENS, 8 <= D <= 1 << 24, D % 8 == 0, 1 <= n <=
 * RQ_SHIFT_MAX_MIXES, 1 <= sequences <= RQ_MAX_SEQUENCES, nslots >= 0 (at least `sequences` when slots is NULL; state
 * may be NULL when nslots is 0, which needs slots).
 */
rq_status rq_shift(const void* x, const void* mu, void* state, void* out, const int* offsets,
                   const int* slots, int T, int D, int n, int sequences, int nslots,
                   void* stream);

/* Channels of a head of rq_wkv7. */
#define RQ_WKV_HEAD 64

/* Types of values: rq_wkv7's inputs are of the first two. */
typedef enum { RQ_TYPE_F32 = 0, RQ_TYPE_F16 = 1, RQ_TYPE_E4M3 = 2 } rq_type;

/*
 * rq_wkv7 -- the RWKV-7 state recurrence between the receptance/key/value
 * projections and the output projection.  Per head, S binary32 [64 values i]
 * [64 keys j], and per token t of a sequence, in order:
 *   d_j = exp(-exp(-1/2) * sigmoid(w_j))           (between 0.545 and 1)
 *   S   = S diag(d) - (S kappa) (eta * kappa)^T + v k^T
 *   y_i = sum_j S_ij r_j
 *   r, w, k, v, kappa, eta: [T][H*64], all of input_type.  w is the decay
 *   before its two activations, kappa the removal key, eta its learning rate.
 *   state: float [nslots][H][64][64], read and overwritten for every
 *   sequence that has a token.  y: float [T][H*64]; rows that no sequence
 *   covers are not written.  A sequence whose offsets leave 0 .. T is cut to it.
 * All sums and the state are binary32.  Tokens go one by one or, in longer
 * sequences, sixteen at a time; then factors are held to 22 bits, and the error
 * of y[t][i] is about 2^-20 or less beside |r_t| times the largest 2-norm that
 * row i of the state had up to t, whatever the sizes at other tokens and rows.
 * Which of the two forms a sequence takes follows from H and from the number and
 * lengths of all sequences of the call, so the low bits of its results may change
 * with the batch around it.  (A call with as many tokens as sequences, or up to
 * 14 more, is taken to have no empty sequence: a long one in it, which only empty
 * ones make possible, goes token by token.)  Non-finite inputs reach the outputs of their own
 * token and later ones only.
 * Shape rules: T, sequences and nslots as for rq_shift, 1 <= H <= 4096,
 * sequences * H <= 1 << 22.
 */
rq_status rq_wkv7(const void* r, const void* w, const void* k, const void* v, const void* kappa,
                  const void* eta, int input_type, float* state, float* y, const int* offsets,
                  const int* slots, int T, int H, int sequences, int nslots, void* stream);

/* Limits of rq_lora. */
#define RQ_LORA_MAX_M 8192
#define RQ_LORA_MAX_RANK 128
#define RQ_LORA_MAX_BATCH 8

/* One projection of rq_lora.  Adapter i has rank r_i = offsets[i+1] -
 * offsets[i], the A rows offsets[i] .. offsets[i+1] - 1, and the block of B
 * [N][r_i] that starts at value offsets[i] * N. */
typedef struct {
    const void* a;     /* binary16 [total_rank][K]: the A rows of all adapters */
    const void* b;     /* binary16, total_rank * N values: the B blocks         */
    const void* x;     /* binary16 [M][K]                                       */
    const float* y_in; /* float [M][N], NULL for zero; y itself, or disjoint    */
    float* y;          /* float [M][N]                                          */
    int N;
    int K;
} rq_lora_problem;

/*
 * rq_lora -- adapters of many requests beside a shared projection: with
 * i = ids[m],
 *   y[m] = y_in[m] + scales[i] * B_i (A_i x[m]),
 * for `count` projections (receptance, key and value, say) in two launches.
 * y_in is the shared projection's output, y usually the same array.  A row
 * whose id lies outside 0 .. adapters-1, or whose adapter has rank 0, gets
 * y[m] = y_in[m].  So does one whose rank is not a multiple of 8, exceeds
 * max_rank or leaves 0 .. total_rank.  A_i x is kept in binary32 and meets B_i in
 * 22 bits of its largest entry; infinities and NaN in A_i x reach y as in the
 * formula, an infinite value of B_i as NaN.
 *   ids: [M].  offsets: [adapters + 1], multiples of 8.  scales: float
 *   [adapters], NULL for 1.  workspace: device memory of at least
 *   rq_lora_workspace_size bytes, 16-byte aligned, that overlaps nothing else; it needs
 *   no clearing and holds nothing between calls.
 * Results do not depend on which other rows share the call's blocks of rows,
 * beyond the split of K, which follows the call's sizes.
 * Shape rules: 1 <= count <= RQ_LORA_MAX_BATCH, 1 <= M <= RQ_LORA_MAX_M, 1 <=
 * N <= 1 << 24, 8 <= K <= 1 << 24, K % 8 == 0, adapters >= 1, total_rank >= 0, 8
 * <= max_rank <= RQ_LORA_MAX_RANK, max_rank % 8 == 0.  RQ_ERR_SCRATCH: the
 * workspace is NULL or too small.  `problems` is a host array the call reads
 * before it returns.
 */
rq_status rq_lora(const rq_lora_problem* problems, int count, int M, const int* ids,
                  const int* offsets, const float* scales, int adapters, int total_rank,
                  int max_rank, void* workspace, size_t workspace_bytes, void* stream);

/* The workspace rq_lora uses at these arguments (N, K of `problems` only).
 * Host-only. */
rq_status rq_lora_workspace_size(const rq_lora_problem* problems, int count, int M, int adapters,
                                 int max_rank, size_t* bytes);

/* Limits and workspace of rq_logits. */
#define RQ_LOGITS_MAX_M 4096
#define RQ_LOGITS_WORKSPACE_BYTES (64 << 10)

/* Arguments of rq_logits; a NULL first pointer of a group leaves the group's
 * step out. */
typedef struct {
    const float* logits; /* [M][V]                                                */
    float* out;          /* [M][V]; logits itself, or disjoint                    */
    int* tokens;         /* [M], the greatest entry of each row; NULL: not wanted */
    int M;
    int V;
    /* tokens so far: row m's are history[history_offsets[m] .. [m+1] - 1], the
     * first prompt[m] of them given, the others generated */
    const int* history;
    const int* history_offsets; /* [M + 1]                                        */
    const int* prompt;          /* [M], NULL for none                             */
    int history_len;            /* entries of history                             */
    const float* repetition;    /* [M], > 0, NULL for 1; only with a history      */
    const float* presence;      /* [M], NULL for 0                                */
    const float* frequency;     /* [M], NULL for 0                                */
    /* additions: row m's are entries bias_offsets[m] .. [m+1] - 1 */
    const int* bias_ids;
    const float* bias;
    const int* bias_offsets; /* [M + 1]                                           */
    int bias_len;
    /* allowed tokens: bit v % 32 of masks[mask_ids[m]][v / 32] */
    const unsigned* masks; /* [nmasks][(V + 31) / 32]                             */
    const int* mask_ids;   /* [M]; outside 0 .. nmasks-1: every token allowed     */
    int nmasks;
} rq_logits_args;

/*
 * rq_logits -- penalties, biases and masks on the head's logits, and the
 * greatest.  For every value z of row m, token v, with c its occurrences in
 * the generated part of the row's history:
 *   v anywhere in the history:  z = z > 0 ? z / repetition : z * repetition,
 *                               z = z - frequency * c,  c > 0: z = z - presence;
 *   v among the row's biases:   z = z + bias, of its last entry;
 *   v not allowed:              z = -infinity, whatever it was.
 * Each operation is rounded to binary32 on its own, in this order.  tokens[m]
 * is the lowest v of the greatest z; NaN is never chosen, and a row with
 * nothing above -infinity gives -1.  History and bias entries outside 0 ..
 * V-1 are ignored.
 *   workspace: needed when tokens is not NULL; RQ_LOGITS_WORKSPACE_BYTES of
 *   device memory, 16-byte aligned, overlapping nothing else, zero before its first
 *   use; every call leaves it zero (the first 64 KiB of a workspace of
 *   rq_gemm_smallm_ws will do).  Calls that share it must not overlap in time.
 *   RQ_ERR_SCRATCH: NULL or too small.
 * Shape rules: 1 <= M <= RQ_LOGITS_MAX_M, 1 <= V <= 1 << 30, history_len and
 * bias_len from 0 to 1 << 30, nmasks >= 1 with masks.
 */
rq_status rq_logits(const rq_logits_args* args, void* workspace, size_t workspace_bytes,
                    void* stream);

/*
 * Block-scaled FP8.  Both operands of a product are OCP E4M3 numbers with a
 * scale for each block of 128: activations one for 128 consecutive values of a
 * row, weights one for 128 x 128.  Scales are binary32, or E8M0: one byte b that
 * stands for 2^(b - 127), 255 for NaN.  These calls keep the rules of the calls
 * around the products; scales need the alignment of their type only.
 */
#define RQ_FP8_BLOCK 128

/* Types of scales (a call's weights, activations and outputs share one). */
typedef enum { RQ_SCALE_F32 = 0, RQ_SCALE_E8M0 = 1 } rq_scale_type;

typedef enum {
    RQ_ACT_NONE = 0,
    RQ_ACT_RELU2 = 1, /* max(z, 0)^2     */
    RQ_ACT_SILU = 2   /* z / (1 + e^-z)  */
} rq_act;

/* Limits of the block-scaled calls. */
#define RQ_FP8_MAX_K (1 << 22)
#define RQ_FP8_MAX_BATCH 8
#define RQ_FP8_MAX_VALUES (1ll << 34)

/*
 * rq_quant_fp8 -- rows quantized in blocks of 128 values:
 *   a = act(x) (RQ_ACT_NONE or RQ_ACT_RELU2; the square is rounded to binary32),
 *   s = the smallest power of two, 2^-126 at least, with |a| <= 448 s for every
 *       finite a of the block,
 *   q = the E4M3 number nearest a / s, ties to even; NaN where a is not finite.
 * The scale is a power of two in either type, so a / s is exact and there is one
 * right answer.  A block of zeros has the scale 2^-126.
 *   x: binary32 or binary16 (input_type) [M][K].  q: E4M3 [M][K].  scales: of
 *   scale_type, [M][K/128].
 * Shape rules: 1 <= M <= RQ_MAX_TOKENS, 128 <= K <= RQ_FP8_MAX_K, K % 128 == 0, at
 * most RQ_FP8_MAX_VALUES values.
 */
rq_status rq_quant_fp8(const void* x, int input_type, int act, void* q, void* scales,
                       int scale_type, int M, int K, void* stream);

/* One product of rq_gemm_fp8. */
typedef struct {
    const void* w;        /* E4M3 [N][K]                                           */
    const void* w_scales; /* [(N + 127) / 128][K / 128]                            */
    const void* x;        /* E4M3 [M][K]                                           */
    const void* x_scales; /* [M][K / 128]                                          */
    const float* y_in;    /* float [M][N], NULL for zero; y itself, or disjoint    */
    void* y;              /* [M][N] of out_type                                    */
    void* y_scales;       /* [M][N / 128] with RQ_TYPE_E4M3, else not used         */
    int N;
    int K;
} rq_fp8_problem;

/*
 * rq_gemm_fp8 -- y = y_in + x W^T of block-scaled operands, for `count`
 * independent products with M rows each (receptance, key and value, say) in one
 * launch:
 *   y[m][n] = y_in[m][n] + sum_b xs[m][b] ws[n/128][b] sum_{k in block b} x[m][k] w[n][k].
 *   out_type RQ_TYPE_F32: binary32.  Every sum is held in binary32: errors are
 *     about 2^-23 of the sum of the products' magnitudes.
 *   RQ_TYPE_F16: rounded to binary16 (past 65504 infinite); no y_in.
 *   RQ_TYPE_E4M3: what rq_quant_fp8 with `act` makes of the RQ_TYPE_F16 output (of
 *     a call that has a workspace too, or none too), to the bit, without that output
 *     in memory, and so with its range: NaN past 65504, steps of 2^-24 near zero; no
 *     y_in, N % 128 == 0.
 *     For these two, calls of more than 16 rows whose outputs make more than 64 tiles
 *     of 128 x 128 over all products (more than 128 with up to 64 rows) take the FP8
 *     matrix instructions, others binary32 sums as for RQ_TYPE_F32.  The FP8
 *     instructions drop what lies 2^-13 or more below the largest of eight products:
 *     within 2^-10 of the sum of the products' magnitudes, about 2^-15 of an ordinary
 *     output.  A caller that wants binary32 sums at every size, or the range of
 *     binary32 in a quantized output, takes RQ_TYPE_F32 (with rq_quant_fp8 behind it).
 *   act: RQ_ACT_NONE, or RQ_ACT_RELU2 with RQ_TYPE_E4M3.
 * NaN in an operand or a scale reaches its outputs.  The product of an x scale and
 * a w scale has to be a normal binary32 number (or zero); what a smaller or larger
 * one gives is not specified, but for a smaller one of a block whose values of x or
 * w are all zero, which adds zero.  Rows are independent: what is in row m of x does
 * not change another row's results.
 *   workspace: device memory, 16-byte aligned, overlapping nothing else, whose first
 *   64 KiB are zero before its first use; every call leaves them zero (a workspace of
 *   rq_gemm_smallm_ws will do).  Calls that share it must not overlap in time, in
 *   graphs neither.  Only RQ_TYPE_F16 and RQ_TYPE_E4M3 outputs that make more than 64
 *   and at most 128 tiles of 128 x 128, of K = 4096 or more, use one, to split K; NULL
 *   keeps K whole there too, which takes 5 to 20 % longer.  RQ_ERR_SCRATCH: smaller
 *   than rq_gemm_fp8_workspace_size reports.
 * Results are deterministic; which sums are taken together follows from the sizes
 * of the call (and from whether it has a workspace).
 * Shape rules: 1 <= count <= RQ_FP8_MAX_BATCH, 1 <= M <= RQ_MAX_TOKENS, 1 <= N <=
 * 1 << 24, 128 <= K <= RQ_FP8_MAX_K, K % 128 == 0, at most RQ_FP8_MAX_VALUES outputs
 * of a product.
 * `problems` is a host array the call reads before it returns.
 */
rq_status rq_gemm_fp8(const rq_fp8_problem* problems, int count, int M, int scale_type,
                      int out_type, int act, void* workspace, size_t workspace_bytes,
                      void* stream);

/* The workspace rq_gemm_fp8 uses at these arguments (N, K of `problems` only), at
 * most RQ_GEMM_WORKSPACE_MAX_BYTES.  Host-only. */
rq_status rq_gemm_fp8_workspace_size(const rq_fp8_problem* problems, int count, int M,
                                     int scale_type, int out_type, size_t* bytes);

/* Arguments of rq_groupnorm. */
typedef struct {
    const float* y;      /* [T][C]                                                 */
    const float* weight; /* [C], NULL for 1                                        */
    const float* bias;   /* [C], NULL for 0                                        */
    const void* r;       /* [T][C] of input_type, NULL for no bonus; with it:      */
    const void* k;       /*   [T][C] of input_type                                 */
    const float* r_k;    /*   [C]                                                  */
    const void* v;       /*   [T][C] of input_type                                 */
    const void* gate;    /* [T][C] of input_type, NULL for 1                       */
    void* out;           /* [T][C] of out_type; y itself with RQ_TYPE_F32, or disjoint */
    void* out_scales;    /* [T][C / 128] with RQ_TYPE_E4M3, else not used          */
    int input_type;      /* RQ_TYPE_F32 or RQ_TYPE_F16                             */
    int act;             /* of the gate: RQ_ACT_NONE or RQ_ACT_SILU                */
    int out_type;
    int scale_type;      /* of out_scales                                          */
    int T;
    int C;
    int groups;
    float eps;
} rq_groupnorm_args;

/*
 * rq_groupnorm -- the norm between the state recurrence and the output
 * projection: every token's channels in groups of C / groups (the heads), and
 * per group
 *   z   = (y - mean(y)) / sqrt(mean((y - mean(y))^2) + eps) * weight + bias
 *         + sum(r * k * r_k) * v,
 *   out = z * act(gate),
 * in binary32, the variance from the centred values.  RQ_TYPE_F16 is rounded
 * once; RQ_TYPE_E4M3 is what rq_quant_fp8 makes of the RQ_TYPE_F16 output, to the
 * bit.  A group's non-finite inputs stay in that group, but for the E4M3 outputs of
 * their own block, whose scale is that of its finite values.
 * Shape rules: 1 <= T <= RQ_MAX_TOKENS, C / groups 32, 64, 128 or 256, C <= 1 <<
 * 20, at most RQ_FP8_MAX_VALUES values, C % 128 == 0 with RQ_TYPE_E4M3, eps >= 0 and
 * finite.
 */
rq_status rq_groupnorm(const rq_groupnorm_args* args, void* stream);

/* A static, NUL-terminated English description of a status value. */
const char* rq_status_string(int status);

/* Interface version: (major << 16) | minor. */
int rq_version(void);

#ifdef __cplusplus
}
#endif

#endif /* RQ_H */
