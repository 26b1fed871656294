/*
 * aggemm.h -- C ABI of libaggemm: chunked AllGather fused with a bf16 GEMM, TGATHER, and a language
 * model's operators around the gathered product (the products, the norms before them, the updates
 * after them), on one AMD Instinct MI355X (gfx950).
 *
 * Pages this library implements:
 *   [AGMM]  "Triton第四课：基于对称内存融合 AllGather 与 MatMul，提速1.56倍" (the fused
 *           AllGather + MatMul pipeline: comm blocks, progress flags, rotated tile order)
 *   [TGATH] "CANN PTO-ISA TGATHER 指令深度解析：跨 Rank 行拼接 Gather 的实现原理与开发指南"
 *           (the root-side row-concatenating gather with 2D sliding tiles)
 *
 * On one GPU the N "ranks" are N separate device buffers ("shards"); the AllGather is an
 * HBM-to-HBM copy of their rows into one aggregate buffer.
 *
 * Conventions for every entry point:
 *   - All tensors are caller-owned DEVICE memory on the current HIP device, row-major and
 *     contiguous.  `shards` itself is a HOST array of N device pointers, read during the call only.
 *   - bf16 is IEEE binary32 truncated to its upper 16 bits (the layout of torch.bfloat16).
 *   - `stream` is a hipStream_t (NULL = the null stream).  Calls are enqueued on it and return
 *     before the GPU work finishes; results are valid once the stream has reached that point.
 *   - Arguments are validated before anything is enqueued; on a negative return nothing was
 *     enqueued.  Outputs must not overlap inputs.
 *   - The library keeps a per-device workspace (aggregate A buffer, progress flags, counters, a
 *     status word) that grows on demand and is released by ag_finalize().  Calls that use it are
 *     ordered with one another through an event, so at most one AG-GEMM uses it at a time.
 */
#ifndef AGGEMM_H
#define AGGEMM_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Return codes. */
#define AG_OK            0
#define AG_EINVAL       -1   /* an argument was rejected; nothing was enqueued */
#define AG_ENOMEM       -2   /* the workspace could not grow */
#define AG_EHIP         -3   /* the HIP runtime reported an error (message: ag_last_error()) */
#define AG_ETIMEOUT     -4   /* (ag_check) a tile gave up waiting on a chunk flag */
#define AG_EUNSUPPORTED -5   /* shape outside the library's limits (see each entry point) */

/* Schedules of ag_gemm_ex. */
#define AG_MODE_FUSED      0  /* chunked copy and GEMM overlapped, per-chunk flags */
#define AG_MODE_UNFUSED    1  /* full gather (tgather kernel), then the GEMM: the serial schedule */
#define AG_MODE_GEMM_ONLY  2  /* the fused GEMM with every flag already raised and no copy */
#define AG_MODE_PLAIN_GEMM 3  /* the GEMM of the serial schedule alone, on a_out (no flags at all) */

/* Who copies the chunks in AG_MODE_FUSED ([AGMM] 融合后的流水线 has the copy beside the MatMul). */
#define AG_PRODUCER_SIDE_STREAM  0  /* a copy kernel on a second stream (its first-wave part runs
                                       before the GEMM), waiting tiles help (default) */
#define AG_PRODUCER_IN_KERNEL    1  /* the GEMM's workgroups: tiles that would wait copy at once, and
                                       every running wave copies a little per K step */
#define AG_PRODUCER_COPY_ENGINE  2  /* per chunk, a device-to-device copy that uses no compute units
                                       (hipMemcpyDeviceToDeviceNoCU) then a stream write of the flag
                                       ([AGMM] 数据搬运与细粒度同步: copy, then stream_write_value32);
                                       the GEMM only waits */

/* Element type of C (ag_options.out_dtype). */
#define AG_OUT_BF16      0    /* bf16, round to nearest even (default) */
#define AG_OUT_FP8_E4M3  1    /* FP8 E4M3 "fn" (OCP; torch.float8_e4m3fn), one byte per element:
                                 C = e4m3fn(acc * out_scale), the fp32 sum times the fp32 scale,
                                 rounded to nearest even; NaN where that lands beyond +-448
                                 ([AGMM] MatMul 按需等待: the MatMul's FP8_OUTPUT variant) */

/* Element type of the shards, B and the gathered A (ag_options.in_dtype). */
#define AG_IN_BF16       0    /* bf16 (default) */
#define AG_IN_FP8_E4M3   1    /* FP8 E4M3 "fn" codes, one byte per element (K % 16 == 0).  Every
                                 product of two such values is exact in fp32 and the sums run in
                                 fp32, as for bf16; per-tensor scales of A and B fold into
                                 out_scale.  An extension of [AGMM]'s FP8 variant (there only the
                                 output is FP8) onto gfx950's FP8 matrix instructions. */

typedef struct ag_options {
    int32_t mode;          /* AG_MODE_* */
    int32_t local_rank;    /* shard whose rows the rotated tile walk starts at, 0..N-1 */
    void *a_out;           /* NULL, or an (M, K) device buffer (of the input element type) that
                              receives the gathered A.
                              Required for AG_MODE_GEMM_ONLY and AG_MODE_PLAIN_GEMM, where it must
                              already hold it. */
    int64_t timeout_us;    /* give-up time of one flag wait, microseconds (<= 0: 10 s) */
    int32_t reverse_order; /* test aid: the copy claims chunks in reverse ready order */
    int32_t skip_producer; /* test aid (AG_MODE_FUSED): copy nothing and leave the flags stale, so
                              every non-local tile's wait ends through timeout_us; ag_check then
                              reports AG_ETIMEOUT.  C is meaningless after such a call; later calls
                              are unaffected (every call starts from fresh counters, and a give-up
                              only short-cuts the waits of the call that gave up). */
    int32_t producer;      /* AG_PRODUCER_* (AG_MODE_FUSED only) */
    void *gemm_events[2];  /* measurement aid: NULL, or two hipEvent_t the call records on the GEMM
                              kernel's stream right before and right after launching it */
    int32_t out_dtype;     /* AG_OUT_*; with AG_OUT_FP8_E4M3, C is an (M, Nc) byte array */
    float out_scale;       /* AG_OUT_FP8_E4M3: factor applied to the fp32 sums before the
                              conversion; 0 means 1 (must be finite) */
    void *wait_stats;      /* measurement aid (AG_MODE_FUSED): NULL, or a device array of 4 uint64 the
                              GEMM adds to: 100 MHz clock ticks its workgroups spent waiting on chunk
                              flags (summed over workgroups), waits, pieces copied by waiting
                              workgroups, tiles that skipped their wait (flags read in advance) */
    int32_t in_dtype;      /* AG_IN_*; with AG_IN_FP8_E4M3 the shards, B and a_out hold one byte per
                              element, and C = out_scale * (A B^T) in bf16 or (out_dtype) FP8 --
                              out_scale then applies to bf16 output too (0 means 1) */
} ag_options;

/*
 * C = gather(shards) * B^T with the fused schedule ([AGMM] 融合后的流水线, MatMul 按需等待).
 *   shards[r]        (H, K) bf16, H = M / N; shard r holds rows [r*H, (r+1)*H) of A
 *   N                number of shards, 1..64
 *   M, K             rows of the gathered A and the reduction length; M % N == 0, K % 8 == 0,
 *                    K <= 2^21
 *   B                (Nc, K) bf16 (the weight stored row-major by output column)
 *   C                (M, Nc) bf16 output, written with round-to-nearest-even from fp32 sums
 *   comm_block_rows  rows per comm block (chunk) inside each shard, >= 1; the last chunk of a
 *                    shard may be shorter.  Chunk r*S + s (S = ceil(H / comm_block_rows)) has
 *                    its own uint32 progress flag ([AGMM] 数据搬运与细粒度同步).
 * Device pointers must be 16-byte aligned.  M == 0 or Nc == 0 enqueues nothing; K == 0 writes
 * zeros (shards and B may then be NULL).  The local shard is shard 0 (ag_gemm_ex chooses
 * another).
 */
int ag_gemm(const void *const *shards, int32_t N, int64_t M, int64_t K, const void *B,
            int64_t Nc, void *C, int64_t comm_block_rows, void *stream);

/* Same arguments; the serial schedule ([AGMM] 为什么要融合 AllGather 与 MatMul): the whole
 * gather into the workspace first, then the GEMM.  Bitwise equal to ag_gemm's C. */
int ag_gemm_unfused(const void *const *shards, int32_t N, int64_t M, int64_t K, const void *B,
                    int64_t Nc, void *C, int64_t comm_block_rows, void *stream);

/* ag_gemm with options (NULL = defaults: fused, side-stream producer, local_rank 0, internal buffer,
 * 10 s). */
int ag_gemm_ex(const void *const *shards, int32_t N, int64_t M, int64_t K, const void *B,
               int64_t Nc, void *C, int64_t comm_block_rows, void *stream,
               const ag_options *opt);

/*
 * TGATHER ([TGATH] 二 数学语义): dst[d0,d1,d2, r*H + i, j] = shards[r][d0,d1,d2, i, j].
 *   shards[r]            (D0, D1, D2, H, W) tensor of elem_size-byte elements, r < N (1..64)
 *   dst                  (D0, D1, D2, N*H, W) tensor
 *   valid_rows/cols      extent of the staging tile that slides over each rank's (H, W) plane
 *                        ([TGATH] 6.1, 7.4): >= 1; the last row / column tile is ragged when they
 *                        do not divide H / W; values above H / W mean one tile spans the plane.
 *                        The result does not depend on them (a copy is exact); the work split does.
 *   elem_size            1, 2, 4 or 8 bytes.
 * Any extent of 0 enqueues nothing ([TGATH] 7.4).  16-byte aligned pointers with
 * W * elem_size % 16 == 0 take the 16-byte vector path; anything else a slower element path.
 */
int tgather(const void *const *shards, int32_t N, void *dst, int64_t D0, int64_t D1, int64_t D2,
            int64_t H, int64_t W, int64_t valid_rows, int64_t valid_cols, int32_t elem_size,
            void *stream);

/* tgather into a taller dst of shape (D0, D1, D2, dst_rows, W), dst_rows >= N*H; rows at or
 * beyond N*H of every plane are left untouched ([TGATH] 7.2 内存约束).  root, 0..N-1, is the rank
 * whose buffer dst is ([TGATH] RunGatherWithRoot): on one GPU every shard is already addressable
 * from it, so it selects nothing and is only validated. */
int tgather_ex(const void *const *shards, int32_t N, void *dst, int64_t D0, int64_t D1,
               int64_t D2, int64_t H, int64_t W, int64_t dst_rows, int64_t valid_rows,
               int64_t valid_cols, int32_t elem_size, int32_t root, void *stream);

/*
 * GEMM + ReduceScatter, one rank's share ([AGMM] 从集合通信理解数据流: ReduceScatter leaves rank r
 * with the reduction, over all ranks, of block r; the mirror of the AllGather feeding the MatMul).
 * In the row-parallel form every rank multiplies its K slice, P = A * B^T, and the ranks reduce P
 * over row blocks of H = M / N rows.  On one GPU the other ranks' partials for this rank's rows
 * arrive as input buffers.
 *   A                 (M, K) bf16: this rank's K slice of the activations
 *   B                 (Nc, K) bf16: this rank's K slice of the weight
 *   recv              host array of N device pointers; recv[j], j != local_rank, is rank j's
 *                     (H, Nc) bf16 partial for rows [local_rank*H, (local_rank+1)*H);
 *                     recv[local_rank] is ignored (may be NULL)
 *   P                 (M, Nc) bf16 output: this rank's partial product, bf16 (nearest even) of the
 *                     fp32 sums -- every row block, the others being what the peers would receive
 *   out               (H, Nc) bf16 output: bf16 (nearest even) of the fp32 sum over j = 0..N-1, in
 *                     that order, of the partials (this rank's own rows of P in slot local_rank)
 *   mode              AG_RS_FUSED: a reducing kernel on a second stream starts on each GEMM tile
 *                     row of the block as soon as that row's tiles are written; AG_RS_UNFUSED: the
 *                     GEMM, then the reduction.  Both give bitwise the same P and out.
 * M % N == 0, K % 8 == 0, Nc % 8 == 0; 16-byte aligned pointers.  K > 2^21 or Nc > 2^26 returns
 * AG_EUNSUPPORTED.  A wait that gave up (10 s) is reported by ag_check.
 */
#define AG_RS_FUSED    0
#define AG_RS_UNFUSED  1
int gemm_rs(const void *A, const void *B, int32_t N, int32_t local_rank, int64_t M, int64_t Nc,
            int64_t K, const void *const *recv, void *P, void *out, int32_t mode, void *stream);

/* For callers that cannot allocate device memory: code under HIP graph capture, tight serving
 * loops, harnesses that forbid hipMalloc.  The same product as ag_gemm (C, and the gathered A in
 * a_out), by the fused schedule with the in-kernel producer on `stream` alone.  It allocates
 * nothing and creates no stream or event: its control words (one progress flag and one piece
 * count per chunk, two piece counters, a status block) live in a fixed array inside the library,
 * one per GPU, held until the process ends.
 *   a_out        (M, K) bf16 device buffer that receives the gathered A; required when K > 0
 *   local_rank   as in ag_options, 0..N-1
 *   other arguments as for ag_gemm.
 * Returns AG_EUNSUPPORTED when N * ceil((M/N) / comm_block_rows) > AG_NOALLOC_MAX_CHUNKS.
 * Every call on one GPU uses that GPU's one array: calls that overlap on one GPU (on two streams,
 * or from two host threads without ordering) race, and the caller must order them.  A flag wait
 * that gave up is reported by ag_check, as for the other entry points. */
#define AG_NOALLOC_MAX_CHUNKS 32768
int ag_gemm_noalloc(const void *const *shards, int32_t N, int64_t M, int64_t K, const void *B,
                    int64_t Nc, void *C, int64_t comm_block_rows, void *a_out, int32_t local_rank,
                    void *stream);

/* ------------------------------------------------------------------ language-model operators
 *
 * The products of a language model's block and head around the gathered A, with what follows them
 * fused in, the norm in front of them, their gradients, and what an optimiser makes of those.  All
 * matrices are bf16 (newton_schulz takes fp32 too), every sum and statistic fp32, outputs rounded once
 * (nearest even).  The conventions above hold, with two additions:
 *   - They keep nothing in the library.  A call that needs scratch memory takes `work`, a 16-byte
 *     aligned device buffer of at least `work_bytes`, what the matching ..._workspace() returns for
 *     the same extents (0: `work` may be NULL).  Calls on different streams with different workspaces
 *     are independent, and a call may be captured into a graph.
 *   - Extents of 0 are valid everywhere but V: what remains of the formula is written (K == 0: the
 *     products are zero; a gradient summed over no rows is zero).
 * K % 8 == 0; matrices and bias 16-byte aligned (rows of Nc or V elements may have any length).  K, Nc
 * or V > 2^21, rows > 2^30 or more than 2^28 tiles of 128 x 128 in an output return AG_EUNSUPPORTED. */

/* Activations. */
#define AG_ACT_NONE       0
#define AG_ACT_RELU       1
#define AG_ACT_SILU       2   /* x / (1 + exp(-x)) */
#define AG_ACT_GELU       3   /* x (1 + erf(x / sqrt 2)) / 2 */
#define AG_ACT_GELU_TANH  4   /* x (1 + tanh(sqrt(2/pi) (x + 0.044715 x^3))) / 2 */

/*
 * C = act(A B^T + bias) + residual.
 *   A (M, K), B (Nc, K), C (M, Nc); bias (Nc) or NULL; residual (M, Nc) or NULL; act AG_ACT_*;
 *   pre: NULL, or (M, Nc) that receives A B^T + bias in bf16 for gemm_bias_act_bwd.  (C itself uses
 *   the unrounded sums.)  residual may be the same buffer as C.
 */
int64_t gemm_bias_act_workspace(int64_t M, int64_t Nc, int64_t K);
int gemm_bias_act(const void *A, const void *B, const void *bias, const void *residual, int64_t M,
                  int64_t Nc, int64_t K, int32_t act, void *C, void *pre, void *work,
                  int64_t work_bytes, void *stream);

/*
 * Its gradients, with d = dC * act'(pre):  dA = d B (M, K), dB = d^T A (Nc, K), dbias = column sums of
 * d (Nc).  The residual's gradient is dC itself.  Each output may be NULL: it is then not computed (and
 * A, which only dB needs, or B, which only dA needs, may be NULL too).  pre: as gemm_bias_act stored
 * it; NULL with AG_ACT_NONE.  The products take d rounded to bf16; dbias sums it unrounded.  relu'(0) = 0.
 */
int64_t gemm_bias_act_bwd_workspace(int64_t M, int64_t Nc, int64_t K, int32_t act);
int gemm_bias_act_bwd(const void *dC, const void *A, const void *B, const void *pre, int64_t M,
                      int64_t Nc, int64_t K, int32_t act, void *dA, void *dB, void *dbias, void *work,
                      int64_t work_bytes, void *stream);

/*
 * Products grouped by expert: rows [ends[e-1], ends[e]) of C are the same rows of A times B[e]^T
 * (ends[-1] = 0); rows at or past ends[E-1] of C are zero.
 *   A (M, K), B (E, Nc, K), C (M, Nc); ends: E int32 on the DEVICE, the running sums of the experts'
 *   row counts.  The library never reads them on the host, so a router's output needs no
 *   synchronisation; an entry below its predecessor or beyond M counts as that bound.
 * Nc % 8 == 0; E > 1024 returns AG_EUNSUPPORTED.
 */
int gemm_grouped(const void *A, const void *B, const int32_t *ends, int32_t E, int64_t M, int64_t Nc,
                 int64_t K, void *C, void *stream);

/* Its gradients: rows of expert e: dA = dC B[e]; dB[e] = dC_e^T A_e over the expert's rows (zero for an
 * expert without rows).  Rows of dA past the last end are zero.  dA or dB may be NULL. */
int gemm_grouped_bwd(const void *dC, const void *A, const void *B, const int32_t *ends, int32_t E,
                     int64_t M, int64_t Nc, int64_t K, void *dA, void *dB, void *stream);

/*
 * Softmax cross entropy of the logits A B^T, which are never stored:
 *   lse[t] = log sum_v exp(a_t . b_v),  loss[t] = lse[t] - a_t . b_y,  y = targets[t].
 *   A (T, K), B (V, K), targets (T) int64 on the device, loss and lse (T) fp32.
 * A target outside [0, V) (such as -100) marks a row without one: its loss is 0 and it contributes no
 * gradient.  V >= 1.
 */
int64_t gemm_xent_workspace(int64_t T, int64_t V, int64_t K);
int gemm_xent(const void *A, const void *B, const int64_t *targets, int64_t T, int64_t V, int64_t K,
              float *loss, float *lse, void *work, int64_t work_bytes, void *stream);

/*
 * Its gradients for dloss (T) fp32 and the lse that gemm_xent wrote: with
 * D[t,v] = dloss[t] (exp(a_t . b_v - lse[t]) - [v = y]),  dA = D B (T, K),  dB = D^T A (V, K).
 * D is formed a piece of the vocabulary at a time, rounded to bf16 in units of one of dloss's values, by
 * which the sums are multiplied: a dloss common to all rows is not rounded with it.
 * gemm_xent_bwd_workspace() asks for pieces of up to 512 MiB, and a smaller workspace, down to 256
 * columns a piece, only makes more of them.  dA or dB may be NULL.
 */
int64_t gemm_xent_bwd_workspace(int64_t T, int64_t V, int64_t K);
int gemm_xent_bwd(const float *dloss, const void *A, const void *B, const int64_t *targets,
                  const float *lse, int64_t T, int64_t V, int64_t K, void *dA, void *dB, void *work,
                  int64_t work_bytes, void *stream);

/*
 * Layer norm of each row, with the residual stream added in front:
 *   h = x + residual (rounded to bf16; x itself without a residual),  m = mean(h),
 *   r = 1 / sqrt(mean((h - m)^2) + eps),  y = (h - m) r weight + bias.
 *   x, residual, y, h (rows, width); weight, bias (width); mean, rstd (rows) fp32: m and r.
 * residual, weight (then 1), bias (then 0), h, mean and rstd may be NULL; h needs a residual and may be the same buffer as
 * x or residual.  eps >= 0.  width > 2^21 or rows > 2^30 return AG_EUNSUPPORTED.  Rows may have any length (those of fewer than 8
 * columns take over a hundred times as long as longer ones would, those of more than 16384 half as long again); nothing is written
 * for rows of none.  Sums are fp32: a row whose values add up to more than that holds gives NaN, one whose squared differences do
 * an r of 0.
 */
int layer_norm(const void *x, const void *residual, const void *weight, const void *bias, int64_t rows, int64_t width,
               float eps, void *y, void *h, float *mean, float *rstd, void *stream);

/*
 * Its gradients, with xh = (h - mean) rstd and g = dy weight:
 *   dx = rstd (g - mean(g) - xh mean(g xh)) + dh   (for x and residual alike),
 *   dweight = sum over rows of dy xh,  dbias = sum over rows of dy.
 *   dy, h, dh, dx (rows, width); mean, rstd as layer_norm wrote them; dh: NULL, or the gradient that reaches h on its other
 *   way; dx may be the same buffer as dh.
 * Each output may be NULL: it is then not computed.  `work` serves the sums over rows: without dweight and dbias it may
 * be NULL.
 */
int64_t layer_norm_bwd_workspace(int64_t rows, int64_t width);
int layer_norm_bwd(const void *dy, const void *h, const float *mean, const float *rstd, const void *weight, const void *dh,
                   int64_t rows, int64_t width, void *dx, void *dweight, void *dbias, void *work, int64_t work_bytes,
                   void *stream);

/*
 * Newton-Schulz orthogonalisation of each matrix of a stack, as an optimiser does with a weight's update:
 *   X = G / (|G| + eps), |G| the Frobenius norm; for each step's (a, b, c):
 *   X = a X + (b A + c A A) X with A = X X^T  (X^T X from the right, if R > C: the same result).
 *   G (E, R, C) in g_type; out (E, R, C) bf16, may be G's buffer where that is bf16; coefficients: steps x 3 floats on the
 *   HOST, read during the call.
 * Every singular value s of X becomes s (a + b s^2 + c s^4), step by step.  The products take fp16 of X, A and
 * a I + b A + c A A, with fp32 sums, and what X loses by that is kept beside it where later steps would enlarge it: the result
 * is off by about 2e-3 of its norm, of which 1.7e-3 is its own rounding to bf16, for an fp32 G as for a bf16 one; by more, up to
 * 8e-3 measured, where a step's terms cancel (ten of the default steps, sets that start at a = 8).
 * Coefficients under which X could have a singular value above 3.5 on the way, could have none above 2^-6, or
 * |a + b t + c t^2| (t: the squares) could exceed 28, return AG_EUNSUPPORTED, as do those whose a's vanish, so that what is left
 * of R singular values of one size falls where fp16 has no bits ((0, 1, 0) twice is taken for up to 227 rows), R or C > 2^20,
 * E > 65535, and more than 2^21 tiles of 128 x 128 in a matrix or 2^26 in all.  Where |G| is far below eps, a step whose a is 0
 * gives zeros, and steps whose a's are far below the largest |a + b t + c t^2| leave X fewer bits.  A matrix with an infinity or NaN
 * gives NaN throughout, one of zeros (with eps > 0) zeros.
 */
#define AG_TYPE_BF16  0
#define AG_TYPE_F32   1
int64_t newton_schulz_workspace(int64_t E, int64_t R, int64_t C);
int newton_schulz(const void *G, int32_t g_type, int64_t E, int64_t R, int64_t C, const float *coefficients, int32_t steps,
                  float eps, void *out, void *work, int64_t work_bytes, void *stream);

/* Waits for `stream`, then reads and clears the current device's status words (the workspace's,
 * then ag_gemm_noalloc's).  Returns AG_OK, or AG_ETIMEOUT with info = {code, chunk, tile, epoch}
 * for the first flag wait that gave up since the last ag_check (epoch: the failing call's flag
 * value). */
int ag_check(void *stream, int64_t info[4]);

/* Static text for a return code. */
const char *ag_status_str(int status);

/* Text of the last HIP error seen by the library on this thread's calls ("" if none). */
const char *ag_last_error(void);

/* Waits for all devices the library used and frees every workspace.  Safe to call repeatedly. */
void ag_finalize(void);

#ifdef __cplusplus
}
#endif
#endif /* AGGEMM_H */
