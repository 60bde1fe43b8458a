/*
 * gemm_rs_layer.h -- C ABI of the operators around the row-parallel layer of
 * gemm_rs.h, for AMD Instinct MI355X (gfx950): libgemm_rs_layer.so.
 *
 *   4-bit weights     gemm_rs_w4_pack, gemm_rs_w4_linear: the layer's product
 *                     for a few tokens (decode), weights in 4 bits with a scale
 *                     (and optionally a zero point) per group of inputs.
 *   block norm        gemm_rs_block_norm and its backward pass: the sum of the
 *                     ranks' partials, a norm of the block's output, its gate
 *                     and scale, the residual, and the next block's norm, in
 *                     one pass over each row.
 *   8-bit checkpoint  gemm_rs_ckpt_pack / _unpack, gemm_rs_ckpt_wgrad: the
 *                     layer's input kept in 8 bits for the backward pass, and
 *                     the weight gradient computed from it.
 *
 * Conventions.
 *   - Error codes are gemm_rs.h's.  Arguments are checked before anything is
 *     enqueued; nothing aborts or throws across the ABI.
 *   - Calls enqueue kernels on `stream` (a hipStream_t, NULL = the null stream)
 *     and return without waiting.  They allocate nothing, keep no state and use
 *     no atomics: results are the same bits on every run, calls may overlap on
 *     different streams (with a workspace each) and may be captured into a HIP
 *     graph.  The caller owns every buffer until the stream work is done.
 *   - Pointers are device pointers, aligned to their element unless stated;
 *     16-byte alignment of pointers and row strides gives the fast loads.
 *   - Row strides are in elements, at least the row's width.  Buffers may be
 *     larger than 4 GiB: offsets are 64-bit.
 *   - Outputs must not overlap inputs unless stated.
 *   - Sizes past the limits given give GEMM_RS_ERR_UNSUPPORTED_SHAPE: N and K up
 *     to 2^22 each (4-bit weights: N K up to 2^37), M of the 4-bit product up to
 *     2^20, rows of a norm up to 2^22 - 1, M K of a checkpoint up to 2^36.
 *   - A call with no rows returns GEMM_RS_OK and enqueues nothing, except where
 *     a sum over rows is an output: that is then zero.
 */
#ifndef GEMM_RS_LAYER_H
#define GEMM_RS_LAYER_H

#include <stddef.h>
#include <stdint.h>

#include "gemm_rs.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- element types ------------------------------------------------------- */
#define GEMM_RS_DTYPE_BF16 0
#define GEMM_RS_DTYPE_F16 1
#define GEMM_RS_DTYPE_F32 2

/* Message for an error code (static storage; for GEMM_RS_ERR_HIP the last HIP
 * error this library saw on this thread). */
const char *gemm_rs_layer_strerror(int code);

/* ---- 4-bit weights -------------------------------------------------------- */

/* y[m][n] = sum_k x[m][k] w[n][k],  w[n][k] = s[n][k / group] (q[n][k] - z[n][k / group]) */
typedef struct gemm_rs_w4_config {
    int32_t N;           /* output features                                      */
    int32_t K;           /* inputs; even                                         */
    int32_t group;       /* inputs that share a scale: a multiple of 32, or K
                            itself; the last group may be short                  */
    int32_t dtype;       /* of x, y and the scales: BF16 or F16                  */
    int32_t zero_points; /* 0: z = 8 everywhere; 1: zero points are given        */
} gemm_rs_w4_config;

/* Checks a configuration (host only): GEMM_RS_OK, INVALID_ARG or UNSUPPORTED_SHAPE. */
int gemm_rs_w4_validate(const gemm_rs_w4_config *cfg);

/* Bytes of the packed weights (0 for an invalid configuration). */
size_t gemm_rs_w4_packed_bytes(const gemm_rs_w4_config *cfg);

/* Lays weights out for gemm_rs_w4_linear, once.
 *   q       [N][K/2] bytes: input k of row n in byte k/2, even k in the low half.
 *   scales  [N][ceil(K/group)] of cfg->dtype.
 *   zeros   [N][ceil(K/group)] bytes, 0..15 each (the low four bits are used);
 *           NULL exactly when zero_points is 0.
 *   packed  gemm_rs_w4_packed_bytes bytes, 16-byte aligned. */
int gemm_rs_w4_pack(const gemm_rs_w4_config *cfg, const void *q, const void *scales, const void *zeros,
                    void *packed, void *stream);

/* The product, M >= 0 rows.  FP32 accumulation, one rounding to cfg->dtype.
 * Inputs are multiplied by 16 + q, and (16 + z) times their sum taken off again:
 *   - before its rounding a result is within (2 ceil(K / 32) + 40) 2^-24 of
 *     sum_k |x| |s| (32 + q + z), not of sum_k |x| |s| |q - z|;
 *   - finite inputs of any size give the formula's result, an infinity only where
 *     that is past the type's range;
 *   - an infinity in a row of x gives NaN in all of that row of y, since it meets
 *     itself with the other sign. */
int gemm_rs_w4_linear(const gemm_rs_w4_config *cfg, const void *packed, int64_t M, const void *x,
                      int64_t x_stride, void *y, int64_t y_stride, void *stream);

/* ---- block norm ----------------------------------------------------------- */

#define GEMM_RS_GATE_NONE 0
#define GEMM_RS_GATE_CHANNEL 1 /* [width]: one factor per column, for every row */
#define GEMM_RS_GATE_TOKEN 2   /* [rows]: one factor per row                    */
#define GEMM_RS_GATE_FULL 3    /* [rows][width]                                 */

#define GEMM_RS_NORM_MAX_PARTS 8
#define GEMM_RS_NORM_MAX_WIDTH 32768

/* For each row, in FP32 with one rounding per output:
 *   y = parts[0] + ... + parts[parts-1]           (FP32, in that order)
 *   u = y r_y post_weight, r_y = 1 / sqrt(mean(y^2) + eps)   with post_norm
 *   u = y, r_y = 1                                           without
 *   h = residual_scale residual + block_scale gate u
 *   z = h r_h pre_weight,  r_h = 1 / sqrt(mean(h^2) + eps)   with pre_norm
 * post_norm closes the block whose output is y; pre_norm opens the next one.
 * The squares are FP32's too: a row whose mean square is past its range (values of
 * some 2^64) has r = 0, a norm of 0, and changes no other row. */
typedef struct gemm_rs_norm_config {
    int32_t width;          /* 1 .. GEMM_RS_NORM_MAX_WIDTH                       */
    int32_t dtype;          /* of parts, weights, gate, y, z: BF16, F16 or F32   */
    int32_t residual_dtype; /* of residual and h: dtype or F32                   */
    int32_t parts;          /* 1 .. GEMM_RS_NORM_MAX_PARTS (forward)             */
    int32_t gate;           /* GEMM_RS_GATE_*                                    */
    int32_t post_norm;      /* 0 or 1                                            */
    int32_t pre_norm;       /* 0 or 1                                            */
    float eps;              /* >= 0 and finite                                   */
    float block_scale, residual_scale; /* finite                                 */
} gemm_rs_norm_config;

typedef struct gemm_rs_norm_args {
    const void *parts[GEMM_RS_NORM_MAX_PARTS]; /* [rows][width] each             */
    int64_t part_stride;
    const void *residual;    /* [rows][width]; NULL: none (h = block_scale gate u) */
    int64_t residual_stride;
    const void *post_weight; /* [width]; with post_norm                          */
    const void *gate;        /* unless GATE_NONE                                 */
    int64_t gate_stride;     /* row stride of a FULL gate                        */
    const void *pre_weight;  /* [width]; with pre_norm                           */
    void *h;                 /* [rows][width] out; may be `residual` (same type and
                                stride): updated in place                        */
    int64_t h_stride;
    void *z;                 /* [rows][width] out; with pre_norm                 */
    int64_t z_stride;
    void *y;                 /* [rows][width] out or NULL: y for the backward pass;
                                may be parts[0] when parts is 1 and strides agree */
    int64_t y_stride;
    float *rstd;             /* [2][rows] out or NULL: r_y then r_h (r_h only
                                with pre_norm, else 0) for the backward pass     */
} gemm_rs_norm_args;

int gemm_rs_norm_validate(const gemm_rs_norm_config *cfg);
int gemm_rs_block_norm(const gemm_rs_norm_config *cfg, int64_t rows, const gemm_rs_norm_args *args,
                       void *stream);

/* The gradients of gemm_rs_block_norm's inputs from those of z and h.  Every
 * part has the gradient dy.  Sums over rows are FP32 and in a fixed order. */
typedef struct gemm_rs_norm_grad_args {
    const void *dz;       /* [rows][width] of dtype; with pre_norm                */
    int64_t dz_stride;
    const void *dh;       /* [rows][width] of residual_dtype, or NULL: zero       */
    int64_t dh_stride;
    const void *h;        /* as the forward pass wrote it; with pre_norm          */
    int64_t h_stride;
    const void *y;        /* as the forward pass wrote it; with post_norm or a gate */
    int64_t y_stride;
    const float *rstd;    /* [2][rows] as the forward pass wrote it               */
    const void *post_weight, *gate, *pre_weight; /* the forward pass's            */
    int64_t gate_stride;
    void *dresidual;      /* [rows][width] of residual_dtype, or NULL; may be dh  */
    int64_t dresidual_stride;
    void *dy;             /* [rows][width] of dtype; may be dz                    */
    int64_t dy_stride;
    float *dpre_weight;   /* [width]; with pre_norm                               */
    float *dpost_weight;  /* [width]; with post_norm                              */
    void *dgate;          /* CHANNEL: float [width]; TOKEN: dtype [rows];
                             FULL: dtype [rows][width]                            */
    int64_t dgate_stride;
} gemm_rs_norm_grad_args;

/* Bytes of workspace the backward pass needs (16-byte aligned; its contents
 * need not be set): a row of FP32 sums for each of pre_norm, post_norm and a
 * CHANNEL gate, per workgroup of rows; at most 96 MiB, 24 MiB up to 8192 columns. */
size_t gemm_rs_block_norm_workspace(const gemm_rs_norm_config *cfg, int64_t rows);
int gemm_rs_block_norm_backward(const gemm_rs_norm_config *cfg, int64_t rows,
                                const gemm_rs_norm_grad_args *args, void *workspace,
                                size_t workspace_bytes, void *stream);

/* ---- 8-bit checkpoints ------------------------------------------------------ */

/* A row of x is cut into blocks of 32 columns.  A block holds
 *   e = max(floor(log2(max |x|)) - 6, -126)   (-126 for a block of zeros)
 *   q = round-to-nearest-even(x 2^-e), limited to -127 .. 127
 * and stands for q 2^e, which BF16 represents exactly (and F16 for an F16 x).
 * A block with an infinity or a NaN has e = 127 and stands for NaN.
 *   q       [M][Kp] int8, Kp = K rounded up to 32; the columns past K are 0
 *   exps    [M][Kp / 32] int8
 * both contiguous, q 16-byte aligned. */
#define GEMM_RS_CKPT_BLOCK 32
#define GEMM_RS_CKPT_NAN 127

int gemm_rs_ckpt_pack(int32_t dtype, int64_t M, int64_t K, const void *x, int64_t x_stride, void *q,
                      void *exps, void *stream);
int gemm_rs_ckpt_unpack(int32_t dtype, int64_t M, int64_t K, const void *q, const void *exps, void *x,
                        int64_t x_stride, void *stream);

/* The weight gradient of a linear layer from its input's checkpoint:
 *   dw[n][k] = add[n][k] + sum_m dy[m][n] x^[m][k]
 * dy is BF16 or F16 (F16: the checkpoint of an F16 x); FP32 accumulation in a
 * fixed order, one rounding to out_dtype (F32 or dy's).
 *   add   [N][K] FP32 or NULL; may be dw when out_dtype is F32 and the strides
 *         agree (gradient accumulation in place).
 * M may be 0 (dw = add, or zero). */
typedef struct gemm_rs_wgrad_args {
    int32_t dtype, out_dtype;
    int64_t M, N, K;
    const void *dy;      /* [M][N] */
    int64_t dy_stride;
    const void *q;       /* [M][Kp], 16-byte aligned */
    const void *exps;    /* [M][Kp / 32] */
    const float *add;
    int64_t add_stride;
    void *dw;            /* [N][K] */
    int64_t dw_stride;
} gemm_rs_wgrad_args;

/* How gemm_rs_ckpt_wgrad splits the work of these arguments (their sizes, strides
 * and alignment; host only).  Tiles are squares of dw; those that do not fill the
 * device a last time may be cut along the tokens into equal shares, whose partial
 * tiles a second kernel joins. */
typedef struct gemm_rs_wgrad_info {
    int32_t words;      /* dy is read in 4-byte words: even N and row stride, aligned to 4;
                           else by elements, every tile whole                        */
    int32_t tile;       /* edge of a tile: 128 or 256                                */
    int32_t whole, cut; /* tiles computed by one workgroup each; tiles cut           */
    int32_t shares;     /* the cut tiles' shares of tokens (0: none are cut)         */
    int32_t workgroups; /* of the first kernel                                       */
    int32_t dealt;      /* 1: neighbouring shares run on different XCDs              */
    int32_t join_waves; /* waves per workgroup of the join (0: there is none)        */
} gemm_rs_wgrad_info;

int gemm_rs_ckpt_wgrad_plan(const gemm_rs_wgrad_args *args, gemm_rs_wgrad_info *info);

/* Bytes of workspace (16-byte aligned; its contents need not be set): a 64 or
 * 256 KiB partial tile for every share and every tile that is cut into shares;
 * less than 64 MiB with tiles of 128 x 128, 128 MiB with tiles of 256 x 256. */
size_t gemm_rs_ckpt_wgrad_workspace(const gemm_rs_wgrad_args *args);
int gemm_rs_ckpt_wgrad(const gemm_rs_wgrad_args *args, void *workspace, size_t workspace_bytes,
                       void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_RS_LAYER_H */
