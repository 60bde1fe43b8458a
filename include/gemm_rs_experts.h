/*
 * gemm_rs_experts.h -- C ABI of the router, the experts' products and the 8-bit
 * floating-point product beside the row-parallel layer of gemm_rs.h, for AMD
 * Instinct MI355X (gfx950); in libgemm_rs_layer.so with gemm_rs_layer.h's calls.
 *
 *   8-bit product     gemm_rs_fp8_quant / _pack, gemm_rs_fp8_linear: operands in
 *                     e4m3 with a power-of-two scale for each block of 128 inputs.
 *   router            gemm_rs_route and its backward pass: the choice of k experts
 *                     for each token, their weights, and the plan (gemm_rs_expert_plan):
 *                     the tokens of every expert.
 *   experts           gemm_rs_experts_linear, gemm_rs_experts_wgrad: the 8-bit
 *                     product of every row with its expert's weights, and the
 *                     weights' gradients; gemm_rs_combine and its backward pass:
 *                     a token's rows back into one.
 *
 * Conventions are gemm_rs_layer.h's: error codes; arguments checked before
 * anything is enqueued; no allocation, no state, no waiting; the same bits on
 * every run; workspaces and buffers are the caller's, and calls may overlap on
 * different streams with a workspace each and be captured.  The number of rows of
 * an expert stays on the device: nothing here needs it on the host.
 * Message for an error code: gemm_rs_layer_strerror.
 */
#ifndef GEMM_RS_EXPERTS_H
#define GEMM_RS_EXPERTS_H

#include "gemm_rs_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- matrices in 8 bits ---------------------------------------------------- */

/* A matrix [rows][cols] in e4m3 with scales 2^e (E8M0 bytes, e + 127):
 *   q       [rows][Kp], Kp = cols rounded up to 128; the columns past cols are 0 (NaN in
 *           a block that stands for NaN)
 *   scales  [Kp / 128][Rp], Rp = rows + 3 rounded up to 4: byte [b][r] is the scale of
 *           columns 128 b .. 128 b + 127 of row r, 1 .. 254; the Rp - rows bytes behind
 *           a block's last row are not used, but the products read them: they take the
 *           scales of four neighbouring rows as a word, from any row on
 * both contiguous and 16-byte aligned; of E matrices, E times GEMM_RS_FP8_Q_BYTES and
 * E times GEMM_RS_FP8_SCALE_BYTES, one after the other.  A block holds
 *   e = the smallest integer >= -126 with max |x| <= 448 2^e (0 where all are zeros or one
 *   is no number),  q = e4m3(x 2^-e)
 * rounded to nearest even, and stands for q 2^e (2^128, past FP32's range, from
 * |x| = 1.9375 2^127 on); a block with an infinity or a NaN stands for NaN.  The calls
 * below make blocks of one row (activations, gradients) or of 128 rows that share a
 * scale (weights, which may then be transposed). */
#define GEMM_RS_FP8_BLOCK 128
#define GEMM_RS_FP8_BLOCKS(cols) (((int64_t)(cols) + 127) / 128)              /* Kp / 128 */
#define GEMM_RS_FP8_SCALE_ROWS(rows) (((int64_t)(rows) + 6) / 4 * 4)          /* Rp       */
#define GEMM_RS_FP8_Q_BYTES(rows, cols) ((int64_t)(rows) * GEMM_RS_FP8_BLOCKS(cols) * 128)
#define GEMM_RS_FP8_SCALE_BYTES(rows, cols) (GEMM_RS_FP8_SCALE_ROWS(rows) * GEMM_RS_FP8_BLOCKS(cols))
#define GEMM_RS_DTYPE_FP8 3 /* of an operand of gemm_rs_fp8_linear given so */

/* x [M][K] (BF16, F16 or F32) in blocks of one row. */
int gemm_rs_fp8_quant(int32_t dtype, int64_t M, int64_t K, const void *x, int64_t x_stride, void *q,
                      void *scales, void *stream);
/* x^T [K][M] in blocks of one row: 128 rows of x and one of its columns. */
int gemm_rs_fp8_quant_transposed(int32_t dtype, int64_t M, int64_t K, const void *x, int64_t x_stride,
                                 void *q, void *scales, void *stream);
/* E matrices w [N][K] (contiguous, one after the other) in blocks of 128 x 128, as
 * [N][K] or (transpose) as [K][N]: E q's and E scales of the layout above. */
int gemm_rs_fp8_pack(int32_t dtype, int64_t E, int64_t N, int64_t K, int32_t transpose, const void *w,
                     void *q, void *scales, void *stream);

/* ---- the products ----------------------------------------------------------- */

/* out[m][n] = add[m][n] + sum_k x^[m][k] w^[n][k], FP32 accumulation, one rounding.
 * Before it, an F32 result is within (K + 2) 2^-24 sum |x^| |w^|.  For BF16 and F16
 * results the products of eight neighbouring inputs are lined up with the largest of
 * them, and what lies below 2^-13 of that is dropped from each: to the bound comes
 * 2^-10 of the largest product of every eight inputs, summed over K (which is up to two
 * half steps of F16, or a quarter of BF16's, also where nothing cancels).
 * gemm_rs_fp8_linear: E, offsets and tokens are 0 and x_rows is M.
 * gemm_rs_experts_linear: rows offsets[e] .. offsets[e + 1] - 1 take the weights of
 * expert e; row m's input is row m of x, or row tokens[m] where tokens are given (zeros
 * for a token outside 0 .. x_rows - 1, as in gemm_rs_experts_wgrad).
 * Rows of out from offsets[E] on stay as they were.  M bounds offsets[E].
 * Sizes: N and K up to 2^22, E up to GEMM_RS_ROUTE_MAX_EXPERTS, scales of an operand
 * and x's q where it is gathered less than 2 GiB. */
typedef struct gemm_rs_fp8_args {
    int32_t x_dtype;         /* BF16, F16, F32: quantised by the call in blocks of a row; FP8 */
    int32_t out_dtype;       /* BF16, F16 or F32                                     */
    int64_t M, N, K;
    int64_t x_rows;          /* rows of x: 1 or more, but with M = 0                  */
    int64_t E;
    const void *x;           /* [x_rows][K], or q of an FP8 matrix                   */
    int64_t x_stride;        /* not of FP8                                           */
    const void *x_scales;    /* of FP8                                               */
    const void *w, *w_scales; /* [N][K] in FP8; E of them                            */
    const int32_t *offsets;  /* [E + 1], ascending from 0                            */
    const int32_t *tokens;   /* [M] or NULL                                          */
    const float *add;        /* [M][N] or NULL; with an F32 out, and may be it (of
                                the same stride)                                     */
    int64_t add_stride;
    void *out;               /* [M][N] */
    int64_t out_stride;
} gemm_rs_fp8_args;

/* How a product of these arguments runs (their sizes, types and whether tokens are given;
 * host only). */
typedef struct gemm_rs_fp8_info {
    int32_t tile;       /* edge of a workgroup's tile of results: 256 or 128; 16 or 32: the
                           kernel for few rows, of so many by 16 columns (0: M is 0)  */
    int32_t stages;     /* of inputs in LDS: 2 or 4; 0: few rows                      */
    int32_t quantises;  /* 1: the product's own kernel quantises x                    */
    int32_t tiles;      /* of the results; with experts' rows, at most               */
    int32_t workgroups; /* of the product's kernel; with tiles of 256 at most 256, which
                           take several where there are more                          */
} gemm_rs_fp8_info;

int gemm_rs_fp8_plan(const gemm_rs_fp8_args *args, gemm_rs_fp8_info *info);

/* Bytes of workspace (16-byte aligned; its contents need not be set). */
size_t gemm_rs_fp8_workspace(const gemm_rs_fp8_args *args);
int gemm_rs_fp8_linear(const gemm_rs_fp8_args *args, void *workspace, size_t workspace_bytes, void *stream);
int gemm_rs_experts_linear(const gemm_rs_fp8_args *args, void *workspace, size_t workspace_bytes,
                           void *stream);

/* dw[e][n][k] = add[e][n][k] + sum_{m of expert e} dy^[m][n] x^[tokens[m]][k], both in
 * blocks of 128 rows of the expert, counted from its first one, and one column.
 * An expert without rows has dw = add, or zero. */
typedef struct gemm_rs_experts_wgrad_args {
    int32_t dtype;          /* of dy and x: BF16, F16 or F32 */
    int32_t out_dtype;      /* F32 or dtype                  */
    int64_t M, N, K, E;     /* M: rows of dy                 */
    int64_t x_rows;
    const void *dy;         /* [M][N]      */
    int64_t dy_stride;
    const void *x;          /* [x_rows][K] */
    int64_t x_stride;
    const int32_t *offsets; /* [E + 1]     */
    const int32_t *tokens;  /* [M] or NULL: row m of x */
    const float *add;       /* [E][N][K] contiguous or NULL; with an F32 dw, and may be it */
    void *dw;               /* [E][N][K] contiguous */
} gemm_rs_experts_wgrad_args;

int gemm_rs_experts_wgrad_plan(const gemm_rs_experts_wgrad_args *args, gemm_rs_fp8_info *info);
size_t gemm_rs_experts_wgrad_workspace(const gemm_rs_experts_wgrad_args *args);
int gemm_rs_experts_wgrad(const gemm_rs_experts_wgrad_args *args, void *workspace, size_t workspace_bytes,
                          void *stream);

/* ---- router ------------------------------------------------------------------ */

#define GEMM_RS_SCORE_SOFTMAX 0
#define GEMM_RS_SCORE_SIGMOID 1
#define GEMM_RS_ROUTE_MAX_EXPERTS 1024
#define GEMM_RS_ROUTE_MAX_CHOICES 64

/* For each token: s = softmax or sigmoid of its logits, c = s + bias.  An expert is on
 * where its logit is not -inf.  With groups > 1 (E / groups neighbouring experts each)
 * the keep_groups groups with the largest sum of their two largest c stay.  The k
 * experts with the largest c, largest first, ties to the lowest index, are chosen:
 *   weights[t][j] = scale s_j  (renormalise: scale s_j / (sum_i s_i + 1e-20))
 * and -1 with weight 0 where fewer than k are on.  c is compared in 64 bits; without
 * a bias and groups the logits are compared.  A NaN counts as the lowest of those on.
 * Weights are of scores in FP32, which are 0 where it does not hold them. */
typedef struct gemm_rs_route_config {
    int32_t dtype;       /* of the logits: BF16, F16 or F32                */
    int32_t E;           /* 1 .. GEMM_RS_ROUTE_MAX_EXPERTS                 */
    int32_t k;           /* 1 .. min(E, GEMM_RS_ROUTE_MAX_CHOICES)         */
    int32_t score;       /* GEMM_RS_SCORE_*                                */
    int32_t renormalise; /* 0 or 1                                         */
    int32_t groups;      /* divides E, at most 64                          */
    int32_t keep_groups; /* 1 .. groups                                    */
    float scale;         /* finite                                         */
} gemm_rs_route_config;

/* The plan of T tokens' choices: rows in the order of the experts, and inside an
 * expert in the order of (token, j); -1 (any index outside 0 .. E - 1) takes no row. */
typedef struct gemm_rs_expert_plan_args {
    int32_t *offsets; /* [E + 1]: the experts' first rows, and the number of rows       */
    int32_t *tokens;  /* [T k]: the rows' tokens, -1 from row offsets[E] on             */
    int32_t *slots;   /* [T][k]: the choices' rows, or -1                               */
} gemm_rs_expert_plan_args;

int gemm_rs_route_validate(const gemm_rs_route_config *cfg);
/* Bytes of workspace of gemm_rs_route and gemm_rs_expert_plan (4-byte aligned). */
size_t gemm_rs_expert_plan_workspace(int64_t T, int32_t E, int32_t k);
/* bias: [E] FP32 or NULL.  weights [T][k] FP32, experts [T][k], contiguous. */
int gemm_rs_route(const gemm_rs_route_config *cfg, int64_t T, const void *logits, int64_t logits_stride,
                  const float *bias, float *weights, int32_t *experts, const gemm_rs_expert_plan_args *plan,
                  void *workspace, size_t workspace_bytes, void *stream);
int gemm_rs_expert_plan(int64_t T, int32_t E, int32_t k, const int32_t *experts, const gemm_rs_expert_plan_args *plan,
                 void *workspace, size_t workspace_bytes, void *stream);
/* dlogits [T][E] of the logits' type from dweights [T][k] FP32, for the experts that
 * were chosen (bias and groups choose only, and have no gradient). */
int gemm_rs_route_backward(const gemm_rs_route_config *cfg, int64_t T, const void *logits,
                           int64_t logits_stride, const int32_t *experts, const float *dweights,
                           void *dlogits, int64_t dlogits_stride, void *stream);

/* ---- rows back to tokens ------------------------------------------------------- */

/* out[t] = sum_j weights[t][j] y[slots[t][j]] over the choices with a row, in FP32, j
 * ascending, one rounding.  weights [T][k] FP32, or NULL: ones. */
int gemm_rs_combine(int32_t dtype, int64_t T, int64_t R, int64_t N, int32_t k, const void *y,
                    int64_t y_stride, const int32_t *slots, const float *weights, void *out,
                    int64_t out_stride, void *stream);
/* dy[slots[t][j]] = weights[t][j] dout[t], dweights[t][j] = <dout[t], y[slots[t][j]]> (0
 * without a row).  y and dweights are NULL together, as weights may be (ones).  Rows of
 * dy that no choice has stay as they were. */
int gemm_rs_combine_backward(int32_t dtype, int64_t T, int64_t R, int64_t N, int32_t k, const void *dout,
                             int64_t dout_stride, const void *y, int64_t y_stride, const int32_t *slots,
                             const float *weights, void *dy, int64_t dy_stride, float *dweights,
                             void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_RS_EXPERTS_H */
