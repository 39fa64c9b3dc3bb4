/*
 * dgemm.h -- dense GEMM C = A*B on AMD MI355X (gfx950), C ABI.
 *
 * The operation (both pages' kernels and the nine-levels tutorial's naive
 * kernel compute exactly this; see the sgemm tf32 page "[CUDA 优化实战] sgemm
 * tf32 - 超越 cuBLAS" section 2, the hgemm page "[CUDA 优化实战] hgemm - 超越
 * cuBLAS" section 1, and "CUDA GEMM优化九重天" section 2.1):
 *
 *     C[i][j] = sum_{k<K} A[i][k] * B[k][j],   0 <= i < M, 0 <= j < N
 *
 * A is row-major M x K with row pitch lda elements, B is row-major K x N with
 * row pitch ldb, C is row-major M x N with row pitch ldc.  Products are
 * accumulated in fp32 (the pages' matrix instructions all accumulate in fp32).
 * C is overwritten (gemm_ex adds alpha, beta, bias and ReLU).  Elements of C outside the M x N
 * window (the ldc - N gap of each row) are never written.
 *
 * Ownership: A, B and C (and gemm_ex's bias and workspace) are DEVICE pointers
 * owned by the caller, all in the memory of the calling thread's current HIP
 * device, and `stream` belongs to that device; the library launches there and
 * does not check where a pointer lives (a pointer into another GPU's memory is
 * the caller's error and faults like any bad address).  The library allocates
 * no device memory and keeps no pointer after a call returns.
 *
 * Execution: each call validates its arguments, enqueues its kernels (one,
 * or two for a split-K plan of gemm_ex) on `stream` (a hipStream_t; NULL
 * means the default stream) and returns without waiting.  Results are visible
 * once the stream has synchronised.  Calls from different host threads on
 * different streams are independent.
 *
 * Errors: a non-zero status is returned and NOTHING is enqueued when the
 * arguments are invalid; C is left untouched.  The library never aborts and
 * keeps no error state beyond the return value.
 *
 * Preconditions (the tutorial's advice in section 6.5 on 16-byte aligned,
 * row-major operands, which this library makes a rule):
 *   - A, B and C are 16-byte aligned, and every row pitch in bytes
 *     (lda*esize_in, ldb*esize_in, ldc*esize_out) is a multiple of 16;
 *   - lda >= max(1, K), ldb >= max(1, N), ldc >= max(1, N);
 *   - 256 rows of A, 64 rows of 16-bit B (32 of fp32 B) and 256 rows of C,
 *     at their row pitches, each span less than 2 GiB (the kernels address
 *     them with 32-bit buffer offsets): DGEMM_ERR_TOO_LARGE otherwise;
 *   - C's bytes overlap neither A's nor B's.  An operand's bytes are its rows
 *     (row i: row-length elements from base + i * pitch), not the gaps
 *     between them.  Operands with the same row pitch in bytes are compared
 *     row by row, so disjoint column windows of one buffer are accepted;
 *     with different pitches the library compares each operand's first to
 *     last byte, so rows that interleave without sharing a byte are still
 *     reported as DGEMM_ERR_ALIAS.
 * Edge semantics: M == 0 or N == 0 is a no-op; K == 0 writes C = 0 (the empty
 * sum).  Any M, N, K >= 0 is accepted; tiles at the matrix edges read zeros
 * beyond K and never store beyond M or N.
 */
#ifndef DGEMM_H
#define DGEMM_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    DGEMM_OK = 0,
    DGEMM_ERR_INVALID_VALUE = 1, /* negative M/N/K, NULL pointer with nonzero extent, bad enum   */
    DGEMM_ERR_LEADING_DIM = 2,   /* lda < max(1,K), ldb < max(1,N) or ldc < max(1,N)           */
    DGEMM_ERR_MISALIGNED = 3,    /* a base pointer or a row pitch in bytes not a multiple of 16
                                    (bias: of 4)                                               */
    DGEMM_ERR_ALIAS = 4,         /* C overlaps A, B or the bias; the workspace overlaps any of them */
    DGEMM_ERR_TOO_LARGE = 5,     /* 256*lda*esize, 128*ldb or 256*ldc*esize_out bytes reach 2 GiB */
    DGEMM_ERR_DEVICE = 6,        /* no current device, or it is not a gfx950                     */
    DGEMM_ERR_LAUNCH = 7,        /* the kernel launch reported an error                          */
    DGEMM_ERR_SCRATCH_SIZE = 8,  /* gemm_ex_static: scratch_bytes > DGEMM_STATIC_SCRATCH_BYTES   */
    DGEMM_ERR_WORKSPACE = 9      /* a backward pass: the workspace is smaller than the call needs */
} dgemm_status;

/* Format of C for the 16-bit entry points. */
typedef enum {
    DGEMM_OUT_F32 = 0,  /* C is fp32: the accumulator itself                          */
    DGEMM_OUT_SAME = 1  /* C has the input format, rounded once, to nearest even       */
} dgemm_out;

/*
 * fp32 inputs, fp32 C.  gfx950 has no reduced-precision (xf32) matrix
 * instruction, so products use the full-fp32 matrix instruction
 * v_mfma_f32_32x32x2_f32: the sgemm tf32 page's workload (section 0, M = N =
 * K = 4096 fp32) without its tf32 input truncation.  Outputs of at most 144
 * tiles of 128 x 128 (e.g. 1536 x 1536) run slice-K: 32 x 32 or 64 x 64 tiles
 * whose K is split across the 4 or 8 waves of one workgroup and summed in LDS
 * in wave order, so small products fill the GPU with no workspace; results
 * are deterministic for a given shape.
 */
int gemm_f32(int M, int N, int K,
             const float* A, int lda,
             const float* B, int ldb,
             float* C, int ldc,
             void* stream);

/*
 * fp32 inputs, fp32 C, computed with bf16 matrix instructions: each input is
 * split as x = hi + lo (+ e) with hi = bf16(x), lo = bf16(x - hi), |e| <=
 * 2^-16 |x|, and a*b is taken as hi*hi + hi*lo + lo*hi, accumulated in fp32
 * (three v_mfma_f32_32x32x16_bf16 per product, at 8x the fp32 matrix rate).
 * Per product the relative error is at most about 3 * 2^-16; results stay
 * within 1e-4 * sum_k |a_ik * b_kj| of the exact product.  This is the
 * MI355X counterpart of the sgemm tf32 page's approach (fp32 data on
 * reduced-precision tensor units), more accurate than TF32's 10-bit inputs.
 * Non-finite inputs: a NaN propagates as in gemm_f32, but an infinite x has
 * lo = inf - inf = NaN, so the outputs it reaches are NaN, not infinite (as
 * are those of finite inputs too large for bf16, |x| >= (2 - 2^-8) * 2^127).
 * Outputs of at most 64 tiles of 128 x 128 run slice-K as in gemm_f32.
 * Arguments, layout, errors and execution as gemm_f32.
 */
int gemm_f32_3xbf16(int M, int N, int K,
                    const float* A, int lda,
                    const float* B, int ldb,
                    float* C, int ldc,
                    void* stream);

/*
 * bf16 inputs (raw 16-bit storage), fp32 accumulation, C fp32 (out =
 * DGEMM_OUT_F32) or bf16 (out = DGEMM_OUT_SAME).  The hgemm page's workload
 * (section 0, M = N = K = 4096, bf16 in and out).  Outputs of at most 64
 * tiles of 128 x 128 run slice-K as in gemm_f32 (K split across the waves of
 * one workgroup, summed in LDS in wave order; no workspace).
 */
int gemm_bf16(int M, int N, int K,
              const void* A, int lda,
              const void* B, int ldb,
              void* C, int ldc,
              int out,
              void* stream);

/* fp16 inputs; otherwise as gemm_bf16 (the hgemm page covers both formats). */
int gemm_f16(int M, int N, int K,
             const void* A, int lda,
             const void* B, int ldb,
             void* C, int ldc,
             int out,
             void* stream);

/* Input format codes of gemm_ex, gemm_ex_plan and dgemm_tile_map. */
typedef enum {
    DGEMM_IN_F32 = 0,        /* fp32, full-fp32 matrix instruction (as gemm_f32)     */
    DGEMM_IN_BF16 = 1,       /* bf16 storage (as gemm_bf16)                           */
    DGEMM_IN_F16 = 2,        /* fp16 storage (as gemm_f16)                            */
    DGEMM_IN_F32_3XBF16 = 3  /* fp32 through the 3 x bf16 split (as gemm_f32_3xbf16) */
} dgemm_in;

/* Activations.  gemm_ex takes the first two; gemm_act, gemm_act_bwd and gemm_f8
   take all, as do gemm_f8_block, gemm_gated and gemm_gated_bwd.  Phi is the normal
   distribution's integral. */
typedef enum {
    DGEMM_ACT_NONE = 0,
    DGEMM_ACT_RELU = 1,       /* x < 0 -> 0; NaN passes through                              */
    DGEMM_ACT_GELU = 2,       /* x Phi(x) = x (1 + erf(x / sqrt 2)) / 2                      */
    DGEMM_ACT_GELU_TANH = 3,  /* x (1 + tanh(sqrt(2 / pi) (x + 0.044715 x^3))) / 2           */
    DGEMM_ACT_SILU = 4        /* x / (1 + exp(-x))                                           */
} dgemm_act;

/*
 * The general entry point: GEMM with a fused epilogue and an optional split-K
 * plan (or slice-K, Stream-K; see below).
 *
 *     C[i][j] := act(alpha * sum_k A[i][k] * B[k][j] + beta * C[i][j] + bias[j])
 *
 * The epilogue is evaluated in fp32 on the fp32 sum and rounded once (to
 * nearest even) to C's format; the old C is read in C's format and only when
 * beta != 0 (so C may hold NaN when beta == 0, as in BLAS).  bias is NULL or
 * a device array of N fp32 values (4-byte aligned).  With alpha = 1, beta = 0,
 * bias = NULL and act = DGEMM_ACT_NONE this is exactly the plain entry point
 * for `in`.  The hgemm page's closing discussion names the library kernel it
 * measures against, a bf16 GEMM with a fused ReLU epilogue; bias and
 * alpha/beta are the usual companions of that epilogue.
 *
 * Split-K (the nine-levels tutorial, section 2.9: K divided into pieces that
 * separate workgroups reduce, joined by a second reduction pass): when the
 * grid of output tiles cannot fill the GPU's 256 CUs (few or thin tiles, deep
 * K), a plan may split K into s pieces.  The GEMM kernel then writes s fp32
 * partial products into `workspace` and a second kernel sums them in a fixed
 * order (ascending piece), applies the epilogue and writes C; results are
 * deterministic for a given (shape, workspace_bytes) and differ from the
 * unsplit plan's only in fp32 summation order.  A split plan is used only if
 * the caller's workspace (device memory, 16-byte aligned, at least
 * workspace_bytes long, not overlapping A, B, C or bias) holds it; with
 * workspace = NULL / workspace_bytes = 0 the call never splits.  The
 * workspace is scratch: its contents before and after the call are
 * unspecified, and calls that share one workspace must be ordered (same
 * stream).  gemm_ex_plan reports the plan and the bytes it uses.
 *
 * Slice-K: small outputs (at most 144 tiles of 128 x 128 for fp32, 64 for the
 * other input formats) run by default on 32 x 32 or 64 x 64 tiles whose K is
 * split across the waves of one workgroup and summed in LDS in wave order:
 * no workspace and no second kernel, deterministic for a given shape.  Offered
 * a workspace, the planner compares this plan with the split plans by their
 * estimated times and takes a split plan only when it is estimated at least
 * 10 % faster: deep K on few tiles and, for bf16 / fp16, outputs that fill the
 * CUs with 64 x 64 tiles at K of about 4096 and more.
 *
 * Stream-K (the nine-levels tutorial, section 2.9: the refinement of Split-K
 * that gives every thread block the same amount of work): for bf16 / fp16
 * inputs with at most 256 tiles of 256 x 256, a plan may instead run one
 * persistent workgroup per CU, each taking an equal run of K steps across
 * tile boundaries; the workgroups that share a tile then reduce it together,
 * each adding up its share of the tile's outputs over their fp32 partial sums
 * (in the workspace) in k order: results are deterministic for a given
 * (shape, workspace_bytes) and differ from the other plans' only in fp32
 * summation order.  It needs 2 x 256 x 256 KiB + 2 KiB of workspace
 * (128 MiB), and is never used on a stream that is being captured into a
 * graph (hipStreamIsCapturing).  A workgroup waits a bounded time for a
 * partial and otherwise computes it itself, so the result does not depend on
 * how the grid is scheduled.  On MI355X it measured slower than the other
 * plans on every shape tried, so the cost model does not pick it; it runs when
 * forced with dgemm_set_plan_override.
 *
 * in:  a dgemm_in code.  out: DGEMM_OUT_F32, or DGEMM_OUT_SAME for C in the
 * input format (for fp32 inputs both mean fp32).  Other arguments,
 * preconditions and errors as the plain entry points.
 */
int gemm_ex(int in, int out, int M, int N, int K,
            const void* A, int lda,
            const void* B, int ldb,
            void* C, int ldc,
            float alpha, float beta, const float* bias, int act,
            void* workspace, size_t workspace_bytes,
            void* stream);

/* Bytes of the static device array that gemm_ex_static uses as its workspace. */
#define DGEMM_STATIC_SCRATCH_BYTES ((size_t)32 << 20)

/*
 * gemm_ex for callers that cannot allocate device memory: code being captured
 * into a HIP graph, tight serving loops, harnesses that forbid hipMalloc.  It
 * computes exactly what gemm_ex computes with a workspace of scratch_bytes,
 * and the split-K partials go to a static device array of
 * DGEMM_STATIC_SCRATCH_BYTES (32 MiB) that the library holds on every GPU it
 * runs on until the process ends.  The call allocates nothing; the caller
 * passes A, B, C and bias as for gemm_ex.  scratch_bytes (0 ..
 * DGEMM_STATIC_SCRATCH_BYTES) bounds the plan as gemm_ex's workspace_bytes
 * does: gemm_ex_plan(..., scratch_bytes, ...) reports the plan, and 0 never
 * splits.  A larger value returns DGEMM_ERR_SCRATCH_SIZE before anything is
 * enqueued.  Every call on one GPU shares that GPU's array, and no part of it
 * needs to start at zero (every partial is written before it is read): calls
 * whose kernels overlap in time on one GPU (different streams, or different
 * host threads without ordering) race on it and must be ordered by the
 * caller, e.g. by issuing them on one stream.  The array's address is looked
 * up on a device's first call.
 */
int gemm_ex_static(int in, int out, int M, int N, int K,
                   const void* A, int lda,
                   const void* B, int ldb,
                   void* C, int ldc,
                   float alpha, float beta, const float* bias, int act,
                   size_t scratch_bytes,
                   void* stream);

/*
 * Host-side query of the plan gemm_ex would use with `workspace_bytes`
 * available (no GPU needed): macro-tile shape, split count (1 = unsplit,
 * 0 = a Stream-K plan) and the workspace bytes that plan uses (0 when
 * unsplit).  gemm_ex never takes a Stream-K plan on a stream that is being
 * captured into a graph; this query assumes no capture.  Any output pointer
 * may be NULL.  Returns DGEMM_OK, or DGEMM_ERR_INVALID_VALUE for negative
 * sizes or a bad `in` / `out`.
 */
int gemm_ex_plan(int in, int out, int M, int N, int K, size_t workspace_bytes,
                 int* tile_rows, int* tile_cols, int* splits, size_t* workspace_used);

/*
 * A linear layer: the product with bias, activation and residual in its
 * epilogue, and its gradients.
 *
 *     Z[i][j] := sum_k A[i][k] * B[k][j] + bias[j]
 *     C[i][j] := act(Z[i][j]) + R[i][j]
 *
 * Evaluated in fp32 on the fp32 sum and rounded once (to nearest even) to C's
 * format; the activation takes the unrounded Z.  bias: NULL or N fp32 values
 * (4-byte aligned).  R: NULL or an M x N matrix in C's format, row pitch ldr;
 * it may be C itself (same pointer and pitch: C := act(..) + C), and overlaps C
 * in no other way.  Z: NULL, or where to keep the pre-activations for
 * gemm_act_bwd, in C's format, row pitch ldz.  R and Z obey C's rules of
 * alignment, pitch and panel size; ldr and ldz are not looked at where the
 * pointer is NULL.  Any dgemm_act.  in, out, sizes and the other arguments,
 * errors and execution as gemm_ex; a workspace allows split plans as in gemm_ex
 * (gemm_act_plan tells the bytes), never a Stream-K plan.
 *
 * At most 16 rows of bf16, fp16 and fp32 run a kernel of their own that streams
 * B through registers (tokens being generated: bound by reading B once).
 */
int gemm_act(int in, int out, int M, int N, int K,
             const void* A, int lda,
             const void* B, int ldb,
             void* C, int ldc,
             const float* bias, int act,
             const void* R, int ldr,
             void* Z, int ldz,
             void* workspace, size_t workspace_bytes,
             void* stream);

/* As gemm_ex_plan, for gemm_act (a 16-row tile: the kernel for few rows). */
int gemm_act_plan(int in, int out, int M, int N, int K, size_t workspace_bytes,
                  int* tile_rows, int* tile_cols, int* splits, size_t* workspace_used);

/*
 * gemm_act's backward pass.  Given dC, the gradient of C (M x N in C's format,
 * which `out` names as in gemm_act), and Z as gemm_act stored it:
 *
 *     dZ = dC o act'(Z)        dA := dZ * B^T       (M x K, input format)
 *     dbias := column sums of dZ (fp32)
 *                              dB := A^T * dZ       (K x N, input format)
 *
 * The residual's gradient is dC itself.  dA, dB and dbias may each be NULL
 * (not wanted); A is read only for dB, B only for dA, and with act =
 * DGEMM_ACT_NONE Z is not read.  relu'(0) = 0.  dZ is rounded once to the input
 * format for the products (unless it is dC itself), in fp16 to infinity beyond 65504
 * and to zero below 2^-25; dbias sums unrounded fp32
 * values, in an order that depends on the shape only.  Results are
 * deterministic; the products' order of sums follows the plan, which depends on
 * the sizes, formats, workspace and which of dA and dB are wanted (small
 * DGEMM_IN_F32_3XBF16 layers run in fp32 arithmetic).  Empty sums are zero: M == 0
 * writes dB = 0 and dbias = 0, N == 0 writes dA = 0.  Outputs overlap no input and no
 * other output.  dB of fp32 inputs takes M <= 2^21 - 4 (DGEMM_ERR_TOO_LARGE above: the
 * rows of A's transpose are that long).
 *
 * The workspace (16-byte aligned) holds dZ, partial column sums, transposes
 * (fp32) and split plans' partial products; its contents before and after are
 * unspecified.  DGEMM_ERR_WORKSPACE if it is smaller than `required` bytes of
 * gemm_act_bwd_workspace; with `best` bytes the products take their fastest
 * plans.  Both figures are those of a call that wants all three gradients.
 */
int gemm_act_bwd(int in, int out, int M, int N, int K,
                 const void* A, int lda,
                 const void* B, int ldb,
                 const void* dC, int lddc,
                 const void* Z, int ldz, int act,
                 void* dA, int ldda,
                 void* dB, int lddb,
                 float* dbias,
                 void* workspace, size_t workspace_bytes,
                 void* stream);

int gemm_act_bwd_workspace(int in, int out, int M, int N, int K, int act,
                           size_t* required, size_t* best);

/*
 * The product of 8-bit operands (OCP e4m3: 448 the largest value, no
 * infinities) with a scale per row of A and per row of B:
 *
 *     C[i][j] := act(scale_a[i] * scale_b[j] * sum_k A[i][k] * B[j][k] + bias[j])
 *                + R[i][j]
 *
 * A: M x K, B: N x K, both K-contiguous (a weight is stored per output, as
 * quant_f8 with transpose = 1 makes it from a K x N matrix); bases 16-byte
 * aligned, lda and ldb multiples of 16.  scale_a: M, scale_b: N fp32 values.
 * out: C's format (and R's) by its dgemm_in code DGEMM_IN_F32, _BF16 or _F16.
 * fp32 accumulation: exactly that for fp32 C and for at most 16 rows (a kernel
 * that streams B through registers); for 16-bit C the 8-bit matrix instruction,
 * which drops bits below 2^-13 of the largest of neighbouring products (in all
 * 1.5e-5 to 5e-5 of the result's 2-norm, below C's rounding).  bias, act, R,
 * workspace, errors and execution as gemm_act.
 */
int gemm_f8(int out, int M, int N, int K,
            const void* A, int lda,
            const void* B, int ldb,
            void* C, int ldc,
            const float* scale_a, const float* scale_b,
            const float* bias, int act,
            const void* R, int ldr,
            void* workspace, size_t workspace_bytes,
            void* stream);

/* As gemm_ex_plan, for gemm_f8. */
int gemm_f8_plan(int out, int M, int N, int K, size_t workspace_bytes,
                 int* tile_rows, int* tile_cols, int* splits, size_t* workspace_used);

/* Columns (along K) that share a scale in gemm_f8_block's operands. */
#define DGEMM_F8_BLOCK 128

/*
 * The product of 8-bit operands (e4m3) with a scale per block of 128 along K, in
 * fp32 between the blocks:
 *
 *     C[i][j] := act(sum over blocks b of sa(i, b) * sb(j, b)
 *                    * sum_{128 b <= k < 128 (b + 1)} A[i][k] * B[j][k] + bias[j]) + R[i][j]
 *
 *     sa(i, b) = scale_a[i * sa_row + b * sa_block]
 *     sb(j, b) = scale_b[(j / rows_b) * sb_row + b * sb_block],   rows_b = 128 or 1
 *
 * rows_b = 128: a weight, with a scale per 128 x 128 (quant_f8_block); with A's rows quantized
 * along K this is a layer's forward product, and with dZ's along N and the weight's 8-bit
 * transpose (whose scales are the transposed ones) the gradient of its input.  rows_b = 1: a
 * scale per row and block on both sides, the gradient of a weight from A and dZ quantized
 * along the batch.  A: M x K, B: N x K, both K-contiguous, as in gemm_f8; the last block may be
 * short.  Strides of the scales are in elements, >= 0; scales of neighbouring rows next to
 * each other (sa_row = 1) load fastest.  256 rows' scales span less than 2 GiB.
 *
 * Sums between blocks are fp32.  Within a block: exactly fp32 for fp32 C and for at most 16
 * rows; for 16-bit C of more rows the 8-bit matrix instruction, which drops bits below 2^-13 of the
 * largest of neighbouring products (against 64 bits no more than C's rounding shows).  out, bias,
 * act, R, workspace, errors and execution as gemm_f8.
 */
int gemm_f8_block(int out, int rows_b, int M, int N, int K,
                  const void* A, int lda,
                  const void* B, int ldb,
                  void* C, int ldc,
                  const float* scale_a, int sa_row, int sa_block,
                  const float* scale_b, int sb_row, int sb_block,
                  const float* bias, int act,
                  const void* R, int ldr,
                  void* workspace, size_t workspace_bytes,
                  void* stream);

/* As gemm_ex_plan, for gemm_f8_block. */
int gemm_f8_block_plan(int out, int rows_b, int M, int N, int K, size_t workspace_bytes,
                       int* tile_rows, int* tile_cols, int* splits, size_t* workspace_used);

/*
 * An M x N matrix to 8 bits with a scale per block of `rows` x 128 of the result Q, which is
 * X (transpose = 0) or X transposed (transpose = 1, Q is N x M):
 *
 *     s = max(max over the block |x| / 448, 2^-100)      scale[(i / rows) * scale_row + b * scale_block] := s
 *     Q[i][j] := e4m3(x / s), the exact quotient rounded once, to nearest even
 *
 * rows = 1 (gemm_f8_block's A; with transpose, both operands of a weight's gradient) or 128 (its
 * B: transpose = 1 for a K x N weight, 0 for its N x K transpose).  s is fp32 and the quotient
 * by that value (exact rounding for s above 2^-84).  A block holding an infinity or a NaN gets
 * scale NaN.  in: X's format (DGEMM_IN_F32, _BF16 or _F16).  The scales' strides, in elements, keep
 * them apart from each other (DGEMM_ERR_LEADING_DIM otherwise).  With rows = 128 or transpose
 * fewer than 2^23 blocks of 128 x 128 (DGEMM_ERR_TOO_LARGE).  M == 0 or N == 0 is a no-op.
 */
int quant_f8_block(int in, int rows, int transpose, int M, int N,
                   const void* X, int ldx,
                   void* Q, int ldq,
                   float* scale, int scale_row, int scale_block,
                   void* stream);

/* Output of rmsnorm and layernorm: X's format; gemm_f8's 8-bit rows and a scale per row;
   gemm_f8_block's, a scale per row and block of 128 columns. */
typedef enum { DGEMM_ROWS_SAME = 0, DGEMM_ROWS_F8 = 1, DGEMM_ROWS_F8_BLOCK = 2 } dgemm_rows;

/*
 * Root-mean-square norm of rows, with the residual's addition and an output in
 * 8 bits for gemm_f8 or gemm_f8_block:
 *
 *     s = X[i] + R[i]                    S[i] := s
 *     rstd[i] := (mean_j s_j^2 + eps)^-1/2
 *     y = s * rstd[i] * weight           Y[i] := y,  or in 8 bits
 *     scale[i] := max(max_j |y_j| / 448, 2^-100),  Y[i] := e4m3(y / scale[i])
 *
 * in: the format of X, R, S and a DGEMM_ROWS_SAME Y (DGEMM_IN_F32, _BF16 or
 * _F16).  R (NULL: none), S and rstd (NULL: not wanted) are optional; scale is
 * given with the 8-bit outputs and only with them: M values with DGEMM_ROWS_F8;
 * with DGEMM_ROWS_F8_BLOCK M * ceil(N / 128) of them, row i's for columns
 * 128 b .. 128 b + 127 at scale[b * M + i], by the largest of those columns alone
 * and with the quotient rounded once, as quant_f8_block's.  weight: N fp32 values,
 * 16-byte aligned.  All arithmetic is fp32 on the unrounded sum, each output rounded
 * once.  S and Y may each be X or R itself (same pointer, pitch and format).
 * A row holding an infinity or a NaN gets scale NaN in 8 bits.  1 <= N <= 32768
 * (DGEMM_ERR_TOO_LARGE above); M == 0 or N == 0 is a no-op; eps >= 0.  Rows obey
 * C's rules of alignment, pitch and panel size; errors and execution as gemm_ex.
 */
int rmsnorm(int in, int out, int M, int N,
            const void* X, int ldx,
            const void* R, int ldr,
            void* S, int lds,
            const float* weight, float eps,
            void* Y, int ldy,
            float* scale, float* rstd,
            void* stream);

/*
 * rmsnorm's backward pass.  Given dY, the gradient of Y, dS (or NULL), the
 * gradient that reaches S by other ways, S (X where there was no residual) and
 * rstd as rmsnorm stored them:
 *
 *     h = S[i] * rstd[i],  g = dY[i] * weight
 *     dX[i] := rstd[i] * (g - h * mean_j(g_j h_j)) + dS[i]   (R's gradient too)
 *     dweight := sum_i dY[i] * h                              (fp32)
 *
 * dX may be dY or dS itself.  dweight may be NULL; if not, a workspace of
 * rmsnorm_bwd_workspace's bytes (16-byte aligned) holds its partial sums, added
 * in a fixed order.  N <= 16384 (DGEMM_ERR_TOO_LARGE above); M == 0 writes
 * dweight = 0.  Otherwise as rmsnorm.
 */
int rmsnorm_bwd(int in, int M, int N,
                const void* dY, int lddy,
                const void* S, int lds,
                const float* weight, const float* rstd,
                const void* dS, int ldds,
                void* dX, int lddx,
                float* dweight,
                void* workspace, size_t workspace_bytes,
                void* stream);

int rmsnorm_bwd_workspace(int M, int N, size_t* required);

/*
 * Layer norm of rows, with the residual's addition and an output in 8 bits:
 *
 *     s = X[i] + R[i]                                S[i] := s
 *     mean[i] := mean_j s_j,  rstd[i] := (mean_j (s_j - mean[i])^2 + eps)^-1/2
 *     y = (s - mean[i]) * rstd[i] * weight + bias    Y[i] := y,  or in 8 bits as rmsnorm
 *
 * bias: NULL (none) or N fp32 values, 16-byte aligned.  mean, rstd (NULL: not wanted): M fp32
 * values each.  The deviations are taken from registers and centred once more before they are
 * squared: Y and rstd are off by half steps of the deviations, not of a mean far from zero
 * (s, the fp32 sum with R, and mean[i] are each rounded to fp32).  DGEMM_ROWS_F8: scale[i] per row
 * (its strides are not looked at); DGEMM_ROWS_F8_BLOCK: block b of row i at scale[i * scale_row +
 * b * scale_block], kept apart from each other (DGEMM_ERR_LEADING_DIM otherwise).  The order of a
 * row's sums depends on N and on whether M exceeds 256 (the same holds for rmsnorm with
 * DGEMM_ROWS_F8_BLOCK): a row's last bits may differ between batches on either side.  Otherwise as
 * rmsnorm.
 */
int layernorm(int in, int out, int M, int N,
              const void* X, int ldx,
              const void* R, int ldr,
              void* S, int lds,
              const float* weight, const float* bias, float eps,
              void* Y, int ldy,
              float* scale, int scale_row, int scale_block,
              float* mean, float* rstd,
              void* stream);

/*
 * layernorm's backward pass.  Given dY, dS (or NULL), S (X where there was no residual), mean
 * and rstd as for rmsnorm_bwd:
 *
 *     h = (S[i] - mean[i]) * rstd[i],  g = dY[i] * weight
 *     dX[i] := rstd[i] * (g - mean_j g_j - h * mean_j(g_j h_j)) + dS[i]   (R's gradient too)
 *     dweight := sum_i dY[i] * h,  dbias := sum_i dY[i]                    (fp32)
 *
 * dX may be dY or dS itself.  dweight and dbias may each be NULL; with either, a workspace of
 * layernorm_bwd_workspace's bytes holds partial sums, added in a fixed order.  N <= 16384
 * (DGEMM_ERR_TOO_LARGE above); M == 0 writes zeros to them.  Otherwise as rmsnorm.
 */
int layernorm_bwd(int in, int M, int N,
                  const void* dY, int lddy,
                  const void* S, int lds,
                  const float* weight, const float* mean, const float* rstd,
                  const void* dS, int ldds,
                  void* dX, int lddx,
                  float* dweight, float* dbias,
                  void* workspace, size_t workspace_bytes,
                  void* stream);

int layernorm_bwd_workspace(int M, int N, size_t* required);

/*
 * Rows to 8 bits: scale[i] := max(max_j |X[i][j]| / 448, 2^-100), Q[i][j] :=
 * e4m3(X[i][j] / scale[i]): the quotient is rounded to fp32 and then to e4m3, both to
 * nearest even (one that fp32 rounds to a tie of e4m3 goes to the even code).  With
 * transpose = 1 by columns: scale[j] from column j, Q (N x M, row pitch ldq)
 * [j][i] := e4m3(X[i][j] / scale[j]): a K x N weight becomes gemm_f8's N x K
 * operand.  A row (column) holding an infinity or a NaN gets scale NaN, one without
 * elements 2^-100.  in: X's format (DGEMM_IN_F32, _BF16 or _F16).  Without transpose
 * N <= 32768.
 */
int quant_f8(int in, int transpose, int M, int N,
             const void* X, int ldx,
             void* Q, int ldq,
             float* scale,
             void* stream);

/*
 * Gated projections, both products, the activation and the product of the two in one kernel:
 *
 *     G[i][j] := sum_k A[i][k] * Bg[k][j] + bias_g[j]
 *     U[i][j] := sum_k A[i][k] * Bu[k][j] + bias_u[j]
 *     C[i][j] := act(G[i][j]) * U[i][j]
 *
 * Evaluated in fp32 on the fp32 sums, each output rounded once (to nearest even) to C's format;
 * C takes the unrounded G and U.  in: DGEMM_IN_F32, _BF16 or _F16; out as gemm_act.  Bg and Bu: K x
 * N with row pitches of their own (two halves of one K x 2 N matrix, for instance).  bias_g,
 * bias_u: NULL or N fp32 values (4-byte aligned).  G, U: NULL, or where to keep them for
 * gemm_gated_bwd, in C's format (either may be asked for alone; the pitch is not looked at where
 * the pointer is NULL).  C, G and U overlap no input and not each other.  Any dgemm_act
 * (DGEMM_ACT_NONE: the plain product of both).  Alignment, pitches, panel size, errors and execution
 * as gemm_ex; a workspace allows split plans, whose results differ in the order of fp32 sums only
 * (gemm_gated_plan tells the bytes).  At most 16 rows run a kernel of their own that streams both
 * weights through registers.
 */
int gemm_gated(int in, int out, int M, int N, int K,
               const void* A, int lda,
               const void* Bg, int ldbg,
               const void* Bu, int ldbu,
               void* C, int ldc,
               const float* bias_g, const float* bias_u, int act,
               void* G, int ldg,
               void* U, int ldu,
               void* workspace, size_t workspace_bytes,
               void* stream);

/* As gemm_ex_plan, for gemm_gated: tile_cols columns of G and the same of U. */
int gemm_gated_plan(int in, int out, int M, int N, int K, size_t workspace_bytes,
                    int* tile_rows, int* tile_cols, int* splits, size_t* workspace_used);

/*
 * gemm_gated's backward pass.  Given dC, the gradient of C (in C's format, which `out` names), and
 * G and U as gemm_gated stored them:
 *
 *     dG = dC o U o act'(G),  dU = dC o act(G)
 *     dA := dG * Bg^T + dU * Bu^T                        (M x K, input format)
 *     dBg := A^T * dG,  dBu := A^T * dU                  (K x N, input format)
 *     dbias_g, dbias_u := column sums of dG and dU        (fp32)
 *
 * Each output may be NULL (not wanted); A is read only for dBg and dBu, Bg and Bu only for dA.
 * relu'(0) = 0.  dG and dU are rounded once to the input format for the products (of 16-bit layers:
 * the matrix instructions take them so; in fp16 values beyond 65504 become infinite, and dA and the
 * weights' gradients with them, and values below 2^-25 zero: scale dC for that range); dA's two products
 * are one fp32 sum; the biases' sums take unrounded fp32 values.  Results are deterministic; the order
 * of sums follows the plan, as for gemm_act_bwd, and so do empty sums, aliasing, limits of M for
 * fp32 weights' gradients, and the workspace (`required` bytes of gemm_gated_bwd_workspace hold dG,
 * dU, partial sums and an fp32 operand's transpose; with `best` the products take their fastest plans).
 */
int gemm_gated_bwd(int in, int out, int M, int N, int K,
                   const void* A, int lda,
                   const void* Bg, int ldbg,
                   const void* Bu, int ldbu,
                   const void* dC, int lddc,
                   const void* G, int ldg,
                   const void* U, int ldu, int act,
                   void* dA, int ldda,
                   void* dBg, int lddbg,
                   void* dBu, int lddbu,
                   float* dbias_g, float* dbias_u,
                   void* workspace, size_t workspace_bytes,
                   void* stream);

int gemm_gated_bwd_workspace(int in, int out, int M, int N, int K, size_t* required, size_t* best);

/* Plan kinds of dgemm_set_plan_override. */
typedef enum {
    DGEMM_PLAN_AUTO = 0,      /* the cost model's choice (the default)                */
    DGEMM_PLAN_GRID = 1,      /* one workgroup per tile and K split, as given         */
    DGEMM_PLAN_STREAM_K = 2,  /* Stream-K (16-bit inputs; 256 x 256 tiles)            */
    DGEMM_PLAN_NO_STREAM_K = 3 /* the cost model's choice among the other plans       */
} dgemm_plan_kind;

/*
 * Process-wide plan override for gemm_ex, gemm_ex_static and gemm_ex_plan,
 * for tests and for tuning the cost model (the plain entry points ignore it).
 * DGEMM_PLAN_GRID forces the macro-tile tile_rows x tile_cols (a shape the
 * input format's kernel has: 256 x 256, 192 x 256 or 128 x 128 for 16-bit
 * inputs, 128 x 128 for fp32, 256 x 256 or 128 x 128 for 3 x bf16) and
 * `splits` K pieces (>= 1; reduced to the number of K steps); it also forces
 * the slice-K tiles, 32 x 32 or 64 x 64 at any M and N in every input format,
 * where `splits` gives the waves per workgroup instead (4 or 8 for 32 x 32, 4
 * for 64 x 64, 1 for the planner's count; a slice-K plan has no K pieces);
 * DGEMM_PLAN_STREAM_K forces a Stream-K plan, DGEMM_PLAN_NO_STREAM_K rules it
 * out (tile and split arguments ignored by both).  A forced plan the call cannot take (tile shape the kernel lacks,
 * workspace too small, Stream-K for fp32 inputs or under graph capture) falls
 * back to the cost model's choice, which gemm_ex_plan then reports.
 * gemm_act, gemm_act_bwd and gemm_f8 follow DGEMM_PLAN_GRID too: gemm_act the
 * tiles above and, for at most 16 rows, 16 x 32, 16 x 64 and (16-bit inputs)
 * 16 x 128; the other two's 16-bit and 8-bit products 256 x 256, 128 x 128 and
 * the slice-K tiles (more than 16 rows).  gemm_f8_block follows it as gemm_f8
 * does (256 x 256 for 16-bit C only, its slice-K tiles with 8 and 4 waves
 * whatever `splits`); gemm_gated takes 256 x 256 (16-bit inputs), 128 x 128 and
 * 64 x 64 (its columns of G and U counted together; 64 x 64 is a slice-K tile),
 * 32 x 32 (32 columns of each) and the 16-row strips of 32 and 64 columns;
 * gemm_gated_bwd 256 x 256 and 128 x 128 (16-bit inputs; dA's K steps and the
 * weights' rows in `splits` runs) and the slice-K tiles.
 * DGEMM_PLAN_AUTO clears the override.  Not synchronised with calls running
 * on other host threads.  Returns DGEMM_OK, or DGEMM_ERR_INVALID_VALUE for a
 * bad kind or splits < 1 with DGEMM_PLAN_GRID.
 */
int dgemm_set_plan_override(int kind, int tile_rows, int tile_cols, int splits);

/*
 * Process-wide bound on how long a Stream-K workgroup waits for another's
 * partial sums before computing them itself, in microseconds; us < 0 restores
 * the default (twice the plan's estimated time plus 100 us), and 0 makes every
 * workgroup take only what is already there (a test of the fallback path,
 * whose results are bit for bit those of the waiting path).  Returns DGEMM_OK,
 * or DGEMM_ERR_INVALID_VALUE for NaN.
 */
int dgemm_set_stream_k_wait_us(double us);

/* Item roles reported by dgemm_stream_k_schedule. */
typedef enum {
    DGEMM_SK_PIECE = 0,      /* the workgroup's own k range of a tile, summed into `slot`   */
    DGEMM_SK_RECOMPUTE = 1,  /* another contributor's missing piece, into that one's slot  */
    DGEMM_SK_REDUCE = 2      /* blocks [lo, hi) of the tile: contributors first .. last
                                summed in that order, epilogue, stored to C             */
} dgemm_sk_role;

/*
 * Host-side query of the Stream-K schedule (no GPU needed; for tests and
 * tuning): the items workgroup `wg` (0 <= wg < 256; XCD x = wg % 8, rank
 * wg / 8) of a Stream-K launch runs for an M x N x K GEMM with 16-bit inputs
 * (`in` = DGEMM_IN_BF16 or DGEMM_IN_F16), in the order it runs them, with
 * every other contributor's piece already published (partials_present != 0)
 * or every one missing (0: the workgroup computes each itself).  Each item is
 * 10 ints in `items`: role (dgemm_sk_role), the tile's row and column index
 * (256 x 256 tiles), k_begin and k_end (elements of K; PIECE and RECOMPUTE),
 * the slot (0 .. 511; slots 2 wg and 2 wg + 1 hold workgroup wg's pieces;
 * -1 for REDUCE), the tile's first and last contributor (ranks of XCD x), and
 * lo and hi (REDUCE: the tile's 32 x 32 output blocks [lo, hi) of 64, block
 * q at rows 128 (q / 32) + 32 ((q / 4) % 4), columns 128 ((q / 16) % 2) +
 * 32 (q % 4) of the tile; 0 otherwise).  *n_items receives the count; only
 * the first max_items are written.  Returns DGEMM_OK, or
 * DGEMM_ERR_INVALID_VALUE for a shape Stream-K does not run (other than 16-bit
 * inputs with at most 256 tiles and at least 32 steps of 64 k per XCD that has
 * a tile), a bad argument, or max_items below the count.
 */
int dgemm_stream_k_schedule(int in, int M, int N, int K, int wg, int partials_present, int* items,
                            int max_items, int* n_items);

/* A static, NUL-terminated description of a status code (never NULL). */
const char* dgemm_status_string(int status);

/*
 * Host-side query of the kernel's work distribution, for tests and tuning; it
 * launches nothing and needs no GPU.  For a problem of M x N outputs and input
 * format `in` (a dgemm_in code), as the plain entry points launch it (no
 * split), writes the macro-tile shape and
 * the number of workgroups, and, when wg is in [0, *num_wg), the output tile
 * (row block *tile_m, column block *tile_n) that workgroup `wg` computes.  The
 * mapping is a bijection from workgroups to tiles: it first gives each of the
 * 8 XCDs a contiguous run of tiles (workgroups are dispatched to XCDs in turn),
 * then walks each run in column strips a few tile rows high so that
 * neighbouring workgroups share A and B panels in L2 (the sgemm tf32 page's
 * "Grid Swizzling", section 4).  Any output pointer may be NULL.
 * Returns DGEMM_OK, or DGEMM_ERR_INVALID_VALUE for negative sizes or a bad `in`.
 */
int dgemm_tile_map(int M, int N, int in, int wg,
                   int* tile_rows, int* tile_cols, int* num_wg,
                   int* tile_m, int* tile_n);

#ifdef __cplusplus
}
#endif

#endif /* DGEMM_H */
