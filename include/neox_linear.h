/*
 * neox_linear.h -- C ABI of a linear layer's operators around the ZeRO-1 step: products with
 * the half-precision weights the step writes, and the gradients it reads.  Part of
 * libneox_zero1.so.
 *
 *   neox_linear            y = r + D(act(x W^T + b)) in one pass over the result
 *   neox_linear_backward   its gradients: of x, W and b
 *   neox_dropout           y = r + D(x + b), and neox_dropout_backward
 *   neox_mxfp4_linear      neox_linear on two MXFP4 copies (neox_matrix.h)
 *
 * D is dropout with a mask that is never stored: it is computed from a counter wherever it is
 * needed, so the backward calls take the forward call's neox_drop again.
 *
 * Conventions are those of neox_zero1.h and neox_matrix.h: device pointers, hip_stream a
 * hipStream_t passed as void*, NEOX_OK or a negative NEOX_E* code with
 * neox_zero1_last_error(), arguments validated before any work is enqueued, nothing thrown
 * across the ABI.  The device current at the call must be the one the arrays and the stream
 * belong to.  Every call only enqueues work and may be recorded into a HIP graph; no call
 * keeps anything about its inputs.  A matrix is given by its first element and `ld`, the
 * elements from one row to the next (at least its columns; of no meaning for a single row).
 * Work that may run at the same time needs workspaces of its own, replays of graphs included.
 *
 * "half" is the call's dtype, NEOX_F16 or NEOX_BF16.  Products and sums are FP32, and what is
 * stored is rounded once, to the nearest, from FP32.  Results depend on the arguments' values,
 * sizes and types only, not on addresses, strides or what else runs.  Infinities and NaN
 * spread as in the formulas, except that a dropped element is zero whatever it was.
 */
#ifndef NEOX_LINEAR_H
#define NEOX_LINEAR_H

#include "neox_matrix.h"

#ifdef __cplusplus
extern "C" {
#endif

/* act(v); -inf gives 0 in all but NONE.                                                  */
#define NEOX_ACT_NONE      0       /* v                                                  */
#define NEOX_ACT_RELU      1       /* max(v, 0)                                          */
#define NEOX_ACT_GELU      2       /* v Phi(v), Phi the normal distribution's integral    */
#define NEOX_ACT_GELU_TANH 3       /* v / 2 (1 + tanh(sqrt(2 / pi) (v + 0.044715 v^3)))   */
#define NEOX_ACT_SILU      4       /* v / (1 + exp(-v))                                  */

/* Dropout of a rows x cols matrix.  With T = p 65536 rounded to the nearest integer (ties to
 * even), element (row, col) is zero if its 16 random bits, as a number, are below T, else it is
 * multiplied by 65536 / (65536 - T) (FP32).  T = 0 leaves everything, T = 65536 nothing.
 *
 * The bits: Philox-4x32 in ten rounds (Salmon, Moraes, Dror and Shaw, "Parallel random
 * numbers: as easy as 1, 2, 3", SC 2011) with the key {seed low, seed high} and the counter
 * {col / 8, row, o low, o high} (32-bit words), o = offset + *counter modulo 2^64; the element
 * takes half col % 8 of the 128 bits, the low half of the first word being the first.  So a
 * mask does not depend on a matrix's strides or size, and matrices with different offsets (or
 * seeds) have independent ones. */
typedef struct neox_drop {
    double   p;                    /* 0 to 1; 0 for none (the other fields are not looked at) */
    uint64_t seed;
    uint64_t offset;
    const uint64_t* counter;       /* NULL, or device memory (8-byte aligned) that is read when
                                      the work runs: a captured graph draws another mask in
                                      each replay if its counter moves on in between         */
} neox_drop;

/* What a product does to its result v = (the sum over k) + bias, before it is stored:
 * pre = v rounded to half; y = residual + D(act(v)). */
typedef struct neox_epilogue {
    int32_t     dtype;             /* half: the type of bias and pre                        */
    int32_t     act;               /* NEOX_ACT_*                                            */
    const void* bias;              /* NULL, or n elements                                   */
    const void* residual;          /* NULL, or m x n of y's type; y itself is allowed        */
    uint64_t    residual_ld;
    void*       pre;               /* NULL, or m x n: what the backward pass needs of an act */
    uint64_t    pre_ld;
    neox_drop   drop;
} neox_epilogue;

/* ------------------------------------------------------------------------------------
 * The layer: y = residual + D(act(x W^T + bias)) for x m x k and W n x k of half, y m x n of
 * half or NEOX_F32.
 *
 * Sizes: n and k 1 to 2^22, m 0 to 2^24 (0: nothing is done, and arrays with m rows may be
 * NULL), at most 2^23 tiles of 64 x 64 elements in any of the results.  y, pre and the inputs
 * must be apart from one another and from the workspace, but two matrices may lie side by
 * side in rows of one ld, and residual may be y.  Every address is aligned to its element;
 * operands whose address or ld is not a multiple of 16 bytes, or whose rows hold no multiple
 * of 8 elements, are first copied to the workspace.
 * ------------------------------------------------------------------------------------ */
typedef struct neox_linear_args {
    const void* x;
    const void* w;
    void*       y;
    uint64_t    x_ld, w_ld, y_ld;
    uint64_t    m, n, k;
    int32_t     y_dtype;           /* epi.dtype (of x and W too) or NEOX_F32                */
    int32_t     reserved;          /* 0                                                     */
    neox_epilogue epi;
} neox_linear_args;

/* Bytes of workspace that this call needs (0 for many): by sizes, lds, types and the addresses'
 * alignment; other addresses of the same alignment need as much.  Host only.  Errors: as
 * neox_linear. */
int neox_linear_workspace(const neox_linear_args* a, uint64_t* bytes);

/* Errors: NEOX_EINVAL (null, misaligned, a size outside the limits, an ld smaller than the
 * columns or above 2^40 or (rows - 1) ld above 2^60, unknown type or act, y_dtype neither half
 * nor NEOX_F32, reserved not 0, p outside [0, 1], arrays meeting, workspace too small or not
 * 256-byte aligned), NEOX_EHIP. */
int neox_linear(const neox_linear_args* a, void* workspace, uint64_t workspace_bytes, void* hip_stream);

/* The gradients of the same, from dy (m x n): with d = M(dy) act'(pre), M dropout's mask without
 * its factor f = 65536 / (65536 - T) (1 without dropout, 0 for T = 65536),
 *     dx = f d W,    dw = f d^T x,    dbias = f times the sum over the rows of d
 * (the residual's gradient is dy itself).  With an act, d is rounded to half for dx and dw (not
 * for dbias), as an operand of their products; f is applied to the sums, in FP32.  accumulate:
 * dw and dbias are added to in FP32 and rounded once; dx is always overwritten.  act' is 0 at
 * -inf, and of RELU 0 at 0.
 * All of half; dx m x k, dw n x k, dbias n; each may be NULL, not all.  x is needed for dw, W
 * for dx, pre for an act.  m = 0: dw and dbias are zeros, or with accumulate as they were.
 * Sizes, alignment and overlap as above; the outputs are apart from everything else. */
typedef struct neox_linear_grads {
    const void* dy;
    const void* pre;               /* as the forward call wrote it; not looked at for NONE  */
    const void* x;
    const void* w;
    void*       dx;
    void*       dw;
    void*       dbias;
    uint64_t    dy_ld, pre_ld, x_ld, w_ld, dx_ld, dw_ld;
    uint64_t    m, n, k;
    int32_t     dtype;             /* NEOX_F16 or NEOX_BF16                                 */
    int32_t     act;
    int32_t     accumulate;        /* 0 or 1                                                */
    int32_t     reserved;          /* 0                                                     */
    neox_drop   drop;
} neox_linear_grads;

int neox_linear_backward_workspace(const neox_linear_grads* a, uint64_t* bytes);
int neox_linear_backward(const neox_linear_grads* a, void* workspace, uint64_t workspace_bytes, void* hip_stream);

/* neox_linear for an m x k copy a and an n x k copy b in MXFP4: c = residual + D(act(a b^T +
 * bias)), dtype the type of c and of the residual (epi->dtype or NEOX_F32), epi->dtype that of
 * bias and pre.  Sums, sizes, alignment and errors as neox_mxfp4_product, and NEOX_EINVAL for
 * an epilogue that neox_linear refuses or whose arrays meet the others.  No workspace. */
int neox_mxfp4_linear(const void* a_codes, const void* a_scales, uint64_t m, const void* b_codes,
                      const void* b_scales, uint64_t n, uint64_t k, void* c, int32_t dtype,
                      uint64_t ldc, const neox_epilogue* epi, void* hip_stream);

/* ------------------------------------------------------------------------------------
 * Dropout by itself: y = residual + D(x + bias) for rows x cols matrices of one type
 * (NEOX_F16, NEOX_BF16 or NEOX_F32; sums in FP32, one rounding) and a bias of cols elements;
 * bias and residual may be NULL, and y may be x or residual.  drop may be NULL: no dropout.
 * rows 0 to 2^31 - 1, cols 1 to 2^31 - 1.
 * Errors: NEOX_EINVAL (null, misaligned to its element, a size outside the limits, an ld
 * smaller than cols or above 2^40 or (rows - 1) ld above 2^60, unknown type, p outside [0, 1],
 * y meeting an input otherwise), NEOX_EHIP. */
int neox_dropout(const void* x, uint64_t x_ld, const void* bias, const void* residual, uint64_t residual_ld,
                 void* y, uint64_t y_ld, uint64_t rows, uint64_t cols, int32_t dtype, const neox_drop* drop,
                 void* hip_stream);

/* Its gradients: dx = D(dy), and dbias = the sum over its rows, in FP32, of what D gives before
 * rounding (accumulate: added to dbias, rounded once).  Either may be NULL, not both; dx may be
 * dy.  rows = 0: dbias is zeros, or with accumulate as it was.  Only dbias needs a workspace.
 * Errors: as neox_dropout, and NEOX_EINVAL for accumulate not 0 or 1, or a workspace too small,
 * not 256-byte aligned or meeting an array. */
int neox_dropout_backward_workspace(uint64_t rows, uint64_t cols, uint64_t* bytes);
int neox_dropout_backward(const void* dy, uint64_t dy_ld, void* dx, uint64_t dx_ld, void* dbias,
                          int32_t accumulate, uint64_t rows, uint64_t cols, int32_t dtype, const neox_drop* drop,
                          void* workspace, uint64_t workspace_bytes, void* hip_stream);

#ifdef __cplusplus
}
#endif
#endif
