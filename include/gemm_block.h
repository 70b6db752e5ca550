/*
 * gemm_block.h -- operators around the GEMMs of a transformer's feed-forward
 * block, in the same library and under the same conventions as gemm.h:
 *
 *   - MXFP4 operands: quantisation along either dimension, and a linear layer
 *     y = x W^T on quantised operands with its backward pass;
 *   - a whole mixture-of-experts layer for a few tokens;
 *   - the norms before and after a block, fused with the block's gate and
 *     residual scale, forward and backward.
 *
 * Every call validates its arguments before anything is enqueued, enqueues on
 * `stream` and returns; errors are a gemm_status and gemm_last_error().
 * Buffers are device memory and stay the caller's; any pointer alignment that
 * holds the element type is accepted. No call allocates device memory but
 * through a plan's own workspace (see gemm_mx4_linear). A size of zero is
 * valid everywhere and leaves outputs of no elements alone.
 */
#ifndef MI355_GEMM_BLOCK_H
#define MI355_GEMM_BLOCK_H

#include "gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- MXFP4 operands ---------------------------------------------------------
 *
 * An MXFP4 matrix of `rows` rows of k elements is stored as
 *   codes  [rows][kp / 2]   e2m1 codes, two per byte, element 2t in the low
 *                           nibble of byte t
 *   scales [rows][kp / 32]  E8M0 bytes e, one per 32 elements: 2^(e - 127)
 * with kp = gemm_mx4_padded(k), k rounded up to 256 (what the MXFP4 tile
 * kernels of gemm_plan_run_mx take), the padding holding code 0 and scale
 * byte 127. Codes are 16-byte, scales 8-byte aligned. */
int64_t gemm_mx4_padded(int64_t k);

/* Quantise x[rows][cols] (F32, F16 or BF16, rows `ld` elements apart).
 * Of each block of 32 elements (the last one of a row may be short) with
 * largest magnitude a:
 *   scale byte = clamp(floor(log2 a) - 2 + 127, 0, 254), 127 where a = 0,
 *   code = x / 2^(byte - 127) rounded to nearest even on 0, 1/2, 1, 3/2, 2,
 *   3, 4, 6 and saturated at 6;
 * a block that holds a NaN or an infinity gets scale byte 255 (NaN) and
 * codes 0. row_codes / row_scales: blocks along the columns, an MXFP4 matrix
 * of `rows` rows of cols elements. col_codes / col_scales: blocks along the
 * rows, the transposed matrix of `cols` rows of rows elements. Either pair
 * may be NULL (both NULL is GEMM_INVALID_ARG); x is read once for both. */
gemm_status gemm_mx4_quantize(const void *x, gemm_dtype x_type, int64_t rows, int64_t cols,
                              int64_t ld, uint8_t *row_codes, uint8_t *row_scales,
                              uint8_t *col_codes, uint8_t *col_scales, void *stream);

/* The values an MXFP4 matrix stands for, rounded once to out_type (F32, F16
 * or BF16); out is [rows][k] with rows `ld` elements apart. Scale byte 255
 * gives NaN. */
gemm_status gemm_mx4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows,
                                int64_t k, void *out, gemm_dtype out_type, int64_t ld,
                                void *stream);

/* y[M][N] = act(Q(x) W^T + bias), BF16: x[M][K] (x_type F32, F16 or BF16, rows
 * ldx elements apart) is quantised along K as above, W is an MXFP4 matrix of
 * N rows of K elements, bias (N elements, BF16) may be NULL, act is the
 * plan's epilogue. `plan`: an F4_E2M1 plan with A RowMajor, B ColumnMajor and
 * C RowMajor; its stream-K workspace is used, so one plan does not run on two
 * streams at once, and its first run of a shape allocates.
 * Up to eight rows of x are quantised inside the product's kernel, more by a
 * launch of their own into `workspace` (16-byte aligned, at least
 * gemm_mx4_linear_workspace(M, K) bytes, which is 0 where none is needed). Up
 * to 64 rows take a kernel that streams W once, more take the tile GEMM of
 * gemm_plan_run_mx; only that one uses the plan's schedule and workspace.
 * K == 0 gives act(bias). */
int64_t gemm_mx4_linear_workspace(int64_t M, int64_t K);
gemm_status gemm_mx4_linear(gemm_plan_t plan, const void *x, gemm_dtype x_type, int64_t ldx,
                            const uint8_t *w_codes, const uint8_t *w_scales, const void *bias,
                            void *y, int64_t M, int64_t N, int64_t K, void *workspace,
                            int64_t workspace_bytes, void *stream);

/* Gradients of gemm_mx4_linear with a LINEAR plan, each product on operands
 * quantised along the dimension that it sums over (the quantiser's rounding
 * is passed straight through):
 *   dx[M][K] = Qn(dy) Wn      Wn: MXFP4 matrix of K rows of N elements (the
 *                             weight quantised along N, gemm_mx4_quantize's
 *                             column form)
 *   dw[N][K] = Qm(dy)^T Qm(x)
 * dy[M][N] and x[M][K] have the type `type` (F32, F16 or BF16), dx and dw are
 * packed BF16. dx or dw may be NULL to leave it out; then wt_codes and
 * wt_scales, or x, may be NULL too. dy is read once for both, and one launch
 * quantises it and x.
 * M == 0 gives dw = 0, N == 0 gives dx = 0. */
int64_t gemm_mx4_linear_backward_workspace(int64_t M, int64_t N, int64_t K);
gemm_status gemm_mx4_linear_backward(gemm_plan_t plan, const void *dy, int64_t ld_dy,
                                     const void *x, int64_t ldx, gemm_dtype type,
                                     const uint8_t *wt_codes, const uint8_t *wt_scales, void *dx,
                                     void *dw, int64_t M, int64_t N, int64_t K, void *workspace,
                                     int64_t workspace_bytes, void *stream);

/* ---- mixture-of-experts layer for a few tokens ------------------------------
 *
 *   l = x router^T                         [tokens][experts]
 *   the top_k largest l of each token (equal ones by the lower index; a NaN
 *   comes after every number)
 *   p = softmax of l over all experts, or over the chosen ones (renormalize)
 *   [g; u] = up[e] x,  h = g / (1 + exp(-g)) * u,  out = sum_chosen p down[e] h
 *
 * Router sums are in 64 bits (a choice hangs on them), all others in fp32. h is
 * not rounded to the type, and may pass its range: with BF16 it keeps its 24
 * bits, with F16 22 bits from 2^-14 up and 2^-36 below (times the power of two
 * that brings a token's largest h below 2^15, if it is not). out is rounded
 * once. Weights are finite (an infinite one of down gives NaN). */
#define GEMM_MOE_MAX_TOKENS 64
#define GEMM_MOE_MAX_EXPERTS 512
#define GEMM_MOE_MAX_TOP_K 16
#define GEMM_MOE_MAX_SIZE (1 << 18)   /* hidden, inner */

typedef struct {
    int64_t hidden, inner;
    int32_t experts, top_k, renormalize;
    gemm_dtype type;          /* of x, router and out: F16 or BF16 */
    gemm_dtype weight_type;   /* `type`, or F4_E2M1 with BF16 */
    const void *router;       /* [experts][hidden] */
    const void *up;           /* [experts][2 * inner][hidden], the gate's rows first;
                                 F4_E2M1: codes of an MXFP4 matrix of those rows */
    const uint8_t *up_scales;     /* F4_E2M1 only */
    const void *down;             /* [experts][hidden][inner] */
    const uint8_t *down_scales;   /* F4_E2M1 only */
} gemm_moe_desc;

/* x[tokens][hidden] and out[tokens][hidden] with rows ldx / ld_out elements
 * apart. row_mask (one byte per token, or NULL): a token whose byte is 0 is
 * routed nowhere; its output is 0 and its x is not used. ids / probs
 * [tokens][top_k] (either may be NULL) receive each token's experts in
 * decreasing order of l and their weights, -1 and 0 for masked tokens.
 * tokens <= GEMM_MOE_MAX_TOKENS, experts, top_k, hidden and inner up to their
 * maxima and x spanning less than 2^31 bytes, else GEMM_UNSUPPORTED. More
 * tokens are calls of their own (the others of a call change nothing of a
 * token's result but the order of its sums), each of which reads its experts'
 * weights; many more on 16-bit experts are grouped_gemm_run's case, which
 * takes no F4_E2M1.
 * `workspace`: 16-byte aligned, gemm_moe_workspace(desc, tokens) bytes
 * (negative for a bad descriptor; more tokens never need less). Its first
 * gemm_moe_state_bytes(desc) bytes hold counters that must be zero before the
 * first call and that every call leaves zero; so one workspace does not serve
 * two streams at once. out may not overlap x. */
int64_t gemm_moe_state_bytes(const gemm_moe_desc *desc);
int64_t gemm_moe_workspace(const gemm_moe_desc *desc, int64_t tokens);
gemm_status gemm_moe_forward(const gemm_moe_desc *desc, const void *x, int64_t ldx,
                             const uint8_t *row_mask, void *out, int64_t ld_out, int32_t *ids,
                             float *probs, int64_t tokens, void *workspace,
                             int64_t workspace_bytes, void *stream);

/* ---- norms before and after a block, with its gate and residual scale -------
 *
 *   y    = block * rstd_post * w_post        (block, where w_post is NULL)
 *   out  = residual + scale * act(gate) * y  rounded to the type
 *   next = out * rstd_next * w_next
 *   rstd = 1 / sqrt(mean(v^2) + eps) of the row v of block / of out
 *
 * in fp32, each result rounded once. scale NULL is 1. gate [gate_rows][cols]
 * holds one row for every rows / gate_rows consecutive rows (gate_rows
 * divides rows), NULL is 1; gate_act is LINEAR or SIGMOID. block NULL: out is
 * the residual itself, not written (the norm before a first block). w_next
 * NULL: no next. Vectors are [cols]; all tensors have one type (F32, F16 or
 * BF16). cols <= GEMM_NORM_MAX_COLS. rstd_post / rstd_next [rows] fp32
 * receive what the backward pass needs (NULL: not kept). out may be residual
 * or block, next may be block (same leading dimension); any other overlap is
 * undefined. */
#define GEMM_NORM_MAX_COLS 16384

typedef struct {
    gemm_dtype type;
    gemm_epilogue gate_act;
    int64_t rows, cols, gate_rows;
    float eps;
    const void *block, *residual, *gate;
    int64_t ld_block, ld_residual, ld_gate;
    const void *w_post, *scale, *w_next;
    void *out, *next;
    int64_t ld_out, ld_next;
    float *rstd_post, *rstd_next;
} gemm_norm_args;

gemm_status gemm_norm_residual(const gemm_norm_args *args, void *stream);

/* The gradients, from d_out (of out) and d_next (of next; either may be NULL
 * for zero, d_next must be where w_next is). `out`, rstd_post and rstd_next
 * are what the forward pass left. d_block, d_gate, d_scale, d_w_post and
 * d_w_next may be NULL to leave them out (d_block is required where block is
 * given); the gradients of the vectors and of the gate (summed over the rows
 * that share it) have the tensors' type, are summed in fp32 in a fixed order
 * and are packed. With block NULL, `out` is the residual. d_residual may be
 * d_out, d_block may be d_next or block (same leading dimension).
 * workspace: 16-byte aligned, gemm_norm_backward_workspace(args) bytes. */
typedef struct {
    gemm_dtype type;
    gemm_epilogue gate_act;
    int64_t rows, cols, gate_rows;
    const void *d_out, *d_next, *block, *out, *gate;
    int64_t ld_d_out, ld_d_next, ld_block, ld_out, ld_gate;
    const void *w_post, *scale, *w_next;
    const float *rstd_post, *rstd_next;
    void *d_block, *d_residual;
    int64_t ld_d_block, ld_d_residual;
    void *d_gate, *d_scale, *d_w_post, *d_w_next;
    void *workspace;
    int64_t workspace_bytes;
} gemm_norm_backward_args;

int64_t gemm_norm_backward_workspace(const gemm_norm_backward_args *args);
gemm_status gemm_norm_residual_backward(const gemm_norm_backward_args *args, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MI355_GEMM_BLOCK_H */
