/*
 * neox_matrix.h -- C ABI of the matrix operators beside the ZeRO-1 step: operators that
 * see a weight as a matrix instead of a run of elements.  Part of libneox_zero1.so.
 *
 *   neox_orthogonalize   X (X^T X)^(-1/2), approximately, by Newton-Schulz products
 *   neox_muon_*          the optimizer step whose update is an orthogonalised momentum,
 *                        with the scaler, skip, clip, decay and half write-back of
 *                        neox_zero1_step
 *   neox_mxfp4_*         the model copy in 4-bit microscaled floating point: quantise (also
 *                        the transpose), dequantise, and the product of two such copies
 *
 * Conventions are those of neox_zero1.h: device pointers, hip_stream a hipStream_t passed
 * as void*, NEOX_OK or a negative NEOX_E* code with neox_zero1_last_error(), arguments
 * validated before any work is enqueued, nothing thrown across the ABI.  The device
 * current at the call must be the one the arrays and the stream belong to.  Every call
 * except neox_muon_create, neox_muon_state and neox_muon_destroy only enqueues work and
 * may be recorded into a HIP graph.  No call keeps anything about its inputs.
 */
#ifndef NEOX_MATRIX_H
#define NEOX_MATRIX_H

#include "neox_zero1.h"

#ifdef __cplusplus
extern "C" {
#endif

#define NEOX_F32 3              /* IEEE-754 binary32, beside NEOX_F16 and NEOX_BF16 */

/* ------------------------------------------------------------------------------------
 * Orthogonalisation.
 *
 * For a rows x cols matrix G: X0 = G / (||G||_F + eps); then, for each step's (a, b, c),
 *     A = X X^T,   X <- a X + (b A + c A A) X
 * (on the transpose when rows > cols, so A has the smaller side); the result is
 * scale * X.  With the default coefficients five steps bring every singular value that is
 * not tiny into about [0.7, 1.2].  A zero matrix gives zeros (eps > 0).  A matrix holding
 * an inf or NaN gives NaN throughout; the other matrices of a batch are not affected.
 *
 * Arithmetic: products of FP16 operands summed in FP32.  The iterate is carried as a pair
 * of FP16 numbers (22 bits) of which only the product terms see the first alone, and the
 * diagonals of A and of b A + c A A are kept in FP32.  With the default steps the result
 * differs from the polynomial in exact arithmetic, besides the rounding to the output type, by
 *   1e-3 of its norm as a rule, where G's elements vary freely; up to 3e-3, with a smaller side
 *       below 16 up to 8e-3, whether the singular values are alike or decay;
 *   more in small matrices of low rank, up to 0.2 / sqrt(smaller side) of the norm (at rank 1;
 *       half of it at rank 4) with a smaller side of up to 256, above that 3e-3 again;
 *   2e-3 as a rule and up to 3e-2 where many elements are equal (a constant matrix, blocks of
 *       ones).  With a smaller side above 512 and a larger one of at least twice that, where
 *       two steps are taken at a time, 4e-3 as a rule and up to 5e-2.
 * (In the last two roundings of one sign add up instead of averaging out.)  Where the norm of
 * G is below about 1e-7 eps, X0 falls below FP16's range and the error grows tenfold with each
 * tenth of the norm.
 * The order of all sums depends on the shape and the coefficients only, not on the batch nor
 * on where and how its matrices lie: each matrix gets the same bits as alone.
 * ------------------------------------------------------------------------------------ */
#define NEOX_NS_MAX_STEPS 16
typedef struct neox_ns_config {
    int32_t steps;              /* 1 .. NEOX_NS_MAX_STEPS                               */
    int32_t reserved;           /* 0                                                    */
    double  eps;                /* > 0 (also in FP32), added to the Frobenius norm      */
    double  coef[NEOX_NS_MAX_STEPS][3];   /* a, b, c of each step                       */
} neox_ns_config;

/* 5 steps of (3.4445, -4.7750, 2.0315), eps 1e-7.  Host only. */
int neox_ns_default_config(neox_ns_config* cfg);

/* Bytes of device workspace neox_orthogonalize needs for `count` rows x cols matrices, for
 * any coefficients: 8 per element and 4 per element of a smaller-side square (6 where the
 * larger side is at least twice the smaller one and that is above 512), each side rounded
 * up to a multiple of 64 or 128, and the partial sums: 2 KB a matrix, with a smaller side of
 * up to 512 and a larger one of 2,048 or more up to 3 MB.  A matrix of up to 128 x 128, or 64 x 256 or 256 x 64,
 * is one block's work: the size for those goes by the same formula, but nothing is written to
 * that memory.  Host only. */
int neox_orthogonalize_workspace(uint64_t count, uint64_t rows, uint64_t cols, uint64_t* bytes);

/* Orthogonalise `count` rows x cols matrices.  Matrix i starts at element i * src_stride
 * of src and i * dst_stride of dst; element (r, c) of it is r * ld + c further.  Types are
 * NEOX_F16, NEOX_BF16 or NEOX_F32.  The matrices may lie one behind the other or side by
 * side in rows of ld (src's may also overlap, or be one matrix with stride 0).  dst may be
 * src (same type, ld and stride); otherwise the memory from its first to its last element
 * must not meet src's, nor either the workspace.  The workspace (256-byte aligned, at least
 * the size above) holds nothing between calls; two calls that may run at the same time,
 * replays of graphs that hold them too, need two.
 * Errors: NEOX_EINVAL (null or misaligned pointer, a size of 0 or above 2^20 rows or cols,
 * count above 2^24, ld < cols, an ld or stride that passes 2^60 elements in all, matrices
 * of dst that overlap, memory that meets where it must not, unknown type, non-finite scale,
 * workspace too small, steps or eps out of range, coefficients that are not finite in FP32,
 * make |b| t^2 + |c| t^4 larger than 30000 for the largest singular value t a step can
 * meet, or take a singular value in (0, 1] above 8 in magnitude on the way), NEOX_EHIP. */
int neox_orthogonalize(const neox_ns_config* cfg, const void* src, int32_t src_dtype,
                       uint64_t src_ld, uint64_t src_stride, void* dst, int32_t dst_dtype,
                       uint64_t dst_ld, uint64_t dst_stride, uint64_t count, uint64_t rows,
                       uint64_t cols, double scale, void* workspace, uint64_t workspace_bytes,
                       void* hip_stream);

/* ------------------------------------------------------------------------------------
 * The Muon step over whole weight matrices.
 *
 *     g = grad * unscale * clip
 *     M <- beta1 M + g
 *     U = g + beta1 M (nesterov) or M
 *     W <- W - lr (s NS(U) + wd W)          (wd on matrices with NEOX_SEG_DECAY)
 *     half = W rounded, MXFP4 copies = W quantised
 * (NS: neox_orthogonalize's polynomial of U) with the loss scaling, skip on inf/NaN, pre-divide, clipping, counters and resume fields
 * of neox_zero1_step, taken from the same configuration struct, and s by scale_mode.  A
 * skipped step writes nothing but the state.
 * ------------------------------------------------------------------------------------ */
#define NEOX_MUON_SCALE_SHAPE 0    /* s = sqrt(max(1, rows / cols))                     */
#define NEOX_MUON_SCALE_RMS   1    /* s = 0.2 sqrt(max(rows, cols)): an update of about the
                                      size of AdamW's, for a shared lr and decay        */

typedef struct neox_muon_config {
    neox_ns_config ns;
    int32_t  nesterov;             /* 0 or 1                                            */
    int32_t  scale_mode;           /* NEOX_MUON_SCALE_*                                 */
    uint64_t workspace_bytes;      /* most device memory for the products, 0 = 4 GiB.  A
                                      matrix that needs more by itself gets what it needs;
                                      matrices of one shape share a launch as far as this
                                      lets them.  Matrices of up to 128 x 128, 64 x 256 or
                                      256 x 64 need none.  Results do not depend on it. */
} neox_muon_config;

/* One rows x cols weight: dense row-major arrays of rows * cols elements, types and
 * alignment as in neox_segment (momentum in the place of exp_avg). */
typedef struct neox_muon_matrix {
    const void* grad;
    void*       half;
    float*      master;
    float*      momentum;
    uint64_t    rows, cols;
    uint32_t    flags;             /* NEOX_SEG_DECAY                                    */
    uint32_t    reserved;          /* 0                                                 */
    /* Optional MXFP4 copies of the new weights (both or neither pointer of a pair): of the
     * matrix, and of its transpose, each laid out as neox_mxfp4_layout says for its shape. */
    void*       mx_codes;
    void*       mx_scales;
    void*       mx_codes_t;
    void*       mx_scales_t;
} neox_muon_matrix;

typedef struct neox_muon neox_muon;

/* The default neox_ns_config, nesterov 1, NEOX_MUON_SCALE_RMS, 4 GiB.  Host only. */
int neox_muon_default_config(neox_muon_config* cfg);

/* Create a step handle.  cfg's beta1 is the momentum; its beta2, eps, optimizer,
 * norm_blocks and chunked_update are checked as neox_zero1_create does and otherwise unused
 * (chunk_elems shapes the norm pass only); segment_norms must be 0.  Arrays stay the caller's; the rules of
 * neox_zero1_create on overlap and lifetime hold, for the MXFP4 copies too.  The handle
 * owns its workspace, so one handle's steps, replays of graphs that captured them among
 * them, must not run at the same time as one another.
 * Waits for hip_stream.
 * Errors: as neox_zero1_create and neox_orthogonalize; NEOX_EINVAL for half a pair of
 * MXFP4 pointers or a misaligned one (codes 16 bytes, scales 4). */
int neox_muon_create(const neox_zero1_config* cfg, const neox_muon_config* mcfg,
                     const neox_muon_matrix* mats, uint64_t n, void* hip_stream, neox_muon** out);

/* One step, enqueued on hip_stream.  Errors: NEOX_EINVAL (null handle, non-finite lr),
 * NEOX_EHIP. */
int neox_muon_step(neox_muon* h, float lr, void* hip_stream);

/* The step in two halves around an exchange of squared norms, exactly as
 * neox_zero1_step_local / neox_zero1_step_apply: over data-parallel ranks, or over the
 * handles of one rank (its matrices here, its other parameters in a neox_zero1 handle), or
 * both.  Handles with the same configuration that are given the same values in the same
 * order skip together and clip alike.  As there, the step's scaler state is the one its
 * step_local started from: give every step_apply its own step_local, and call
 * neox_muon_scaler_set between steps. */
int neox_muon_step_local(neox_muon* h, double* local_sumsq, void* hip_stream);
int neox_muon_step_apply(neox_muon* h, const double* rank_sumsq, uint32_t nranks, float lr,
                         void* hip_stream);

/* As neox_scaler_state / neox_scaler_set. */
int neox_muon_state(neox_muon* h, neox_scaler_state_t* out);
int neox_muon_scaler_set(neox_muon* h, const neox_scaler_state_t* st, void* hip_stream);

/* Wait for outstanding work and free the library's scratch.  NULL is a no-op. */
int neox_muon_destroy(neox_muon* h);

/* ------------------------------------------------------------------------------------
 * MXFP4: 4-bit elements (E2M1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) in blocks
 * of 32 consecutive elements of a row, each block with one 8-bit power-of-two scale
 * (E8M0: byte s stands for 2^(s - 127), 255 for NaN), as the OCP Microscaling Formats
 * specification 1.0 defines them.
 *
 * Layout of a rows x cols copy, K = cols rounded up to a multiple of 128: codes
 * [rows][K / 2] bytes, element 2j of a row in the low half of byte j; scales [rows][K / 32]
 * bytes.  Elements from cols to K are zeros, in blocks of their own with scale byte 0.
 *
 * Quantisation of a block: scale 2^(floor(log2 max|v|) - 2), at least 2^-127 (a block of
 * zeros has byte 0); elements v / scale rounded to the nearest E2M1 value, ties to the
 * even code, magnitudes above 6 to 6.  The sign of a zero is kept.  A block that holds an
 * inf or NaN gets scale byte 255 and codes 0: all of it reads as NaN.  A block at the end
 * of a row consists of the row's last cols % 32 elements and zeros.
 * ------------------------------------------------------------------------------------ */

/* Bytes of the codes and the scales of a rows x cols copy.  Host only.  Errors: NEOX_EINVAL
 * (null, a size of 0 or above 2^31 - 1, codes of more than 2^40 bytes). */
int neox_mxfp4_layout(uint64_t rows, uint64_t cols, uint64_t* code_bytes, uint64_t* scale_bytes);

/* Quantise the rows x cols matrix src (element (r, c) at r * ld + c), or with transpose = 1
 * its transpose: then the copy is cols x rows, with blocks along src's columns.
 * codes 16-byte aligned, scales 4-byte aligned.
 * Errors: NEOX_EINVAL (null, misaligned, a size of 0 or above 2^31 - 1, codes of more than
 * 2^40 bytes, ld < cols or above 2^60 / rows, unknown type, transpose not 0 or 1, codes,
 * scales and the memory from src's first to its last element not apart), NEOX_EHIP. */
int neox_mxfp4_quantize(const void* src, int32_t dtype, uint64_t rows, uint64_t cols, uint64_t ld,
                        int32_t transpose, void* codes, void* scales, void* hip_stream);

/* The values of a rows x cols copy, rounded to dtype, to dst (element (r, c) at r * ld + c).
 * Values above the type's range become infinite.  Errors: as neox_mxfp4_quantize. */
int neox_mxfp4_dequantize(const void* codes, const void* scales, uint64_t rows, uint64_t cols,
                          void* dst, int32_t dtype, uint64_t ld, void* hip_stream);

/* c[i][j] = sum over k of a[i][k] b[j][k] for an m x k copy a and an n x k copy b, summed in
 * FP32 in an order that depends on the sizes only, rounded to dtype (NEOX_F16, NEOX_BF16,
 * NEOX_F32) and written to c[i * ldc + j].  Elements between k and the next multiple of 128
 * are read: zeros, as quantisation writes them, in copies made elsewhere too.  A block that
 * reads as NaN makes its row's or column's results NaN.  With W of shape (out, in): y = x W^T is
 * (x, W); dx = dy W is (dy, transpose copy of W); dW = dy^T x is (transpose copies of dy
 * and x).  Errors: NEOX_EINVAL (null, misaligned, a size of 0 or above 2^31 - 1, k above
 * 2^24, codes of more than 2^40 bytes, 2^23 or more 128 x 128 tiles of c, ldc < n, unknown
 * type, c meeting an operand), NEOX_EHIP. */
int neox_mxfp4_product(const void* a_codes, const void* a_scales, uint64_t m, const void* b_codes,
                       const void* b_scales, uint64_t n, uint64_t k, void* c, int32_t dtype,
                       uint64_t ldc, void* hip_stream);

#ifdef __cplusplus
}
#endif
#endif
