// matrix_internal.h -- types shared by the host side and the gfx950 kernels of the matrix
// operators (include/neox_matrix.h).  Not part of the public ABI.
#pragma once

#include "neox_matrix.h"
#include "zero1_internal.h"

namespace nz1 {

// ------------------------------------------------------------------------------------
// Newton-Schulz products.  The matrices work on "the wide form": m x n with m <= n, the
// source transposed when it is tall.  Both sides are padded with zeros to whole tiles
// (mp, np), which the products leave zeros.
// ------------------------------------------------------------------------------------
constexpr uint32_t kNsParts = 256;       // most blocks (partial sums) of one matrix's norm

// Device memory of a batch, all arrays of matrix z at z times their size.
struct NsBuf {
    uint16_t* xh;      // [mp][np] FP16: the iterate, times S, first 11 bits
    uint16_t* xt[2];   // [np][mp] FP16: its transpose (read / written in turn)
    uint16_t* lt;      // [np][mp] FP16: what xh leaves, times 2^11, transposed
    uint16_t* sym[3];  // [mp][mp] FP16: X X^T and polynomials of it, without their diagonals
    float* diag[3];    // [mp] the diagonals (the third pair with `pairs` only)
    double* part;      // [kNsParts] partial squared norms of the source
    float* sums;       // [split][lower 64 x 64 tiles][4096] shares of X X^T (split > 1 only)
};

struct NsShape {
    uint32_t rows, cols;   // of the source
    uint32_t m, n;         // of the wide form
    uint32_t mp, np;       // padded
    uint32_t parts;        // partial sums per matrix
    bool tall;             // the wide form is the source's transpose
    bool small;            // one block does it all, without the buffers
    uint32_t split;        // shares of X X^T's sums
    bool pairs;            // the iterate is updated once for two steps
    float s;               // S, a power of two: the iterate is stored times S
};
// pairs: whether the coefficients allow two steps at a time (FP16 range).
NsShape ns_shape(uint64_t rows, uint64_t cols, bool pairs);
// Bytes of the buffers of `count` matrices, and their placement at base.
uint64_t ns_bytes(const NsShape& s, uint64_t count);
NsBuf ns_place(const NsShape& s, uint64_t count, void* base);

// Where the matrices come from and go to.
struct OrthIO {
    const void* src;
    void* dst;
    uint64_t src_ld, src_stride, dst_ld, dst_stride;
    int32_t src_dtype, dst_dtype;
    float scale;
    bool vec;              // dst can be written four elements at a time
    bool vec_src;          // src read so
    double eps;
};
struct MuonMat {           // device table entry
    const uint16_t* grad;
    uint16_t* half;
    float* master;
    float* mom;
    uint32_t decay;
    uint32_t vec;          // grad and half 8-byte, master and mom 16-byte aligned
    uint64_t pad_;
};
struct MuonIO {
    const MuonMat* mats;   // first matrix of the launch
    const DevState* st;
    int32_t dtype, nesterov;
    float mu, lr, wd, scale;
    double eps;
};

struct NsCoef {
    float a, b, c;
};
// Everything one batch launches, on stream: norm, conversion, steps, and the last step's
// epilogue (store, or weight update).
hipError_t enqueue_orth(const NsShape& s, const NsBuf& w, uint32_t count, const OrthIO& io,
                        const NsCoef* coef, int steps, hipStream_t stream);
hipError_t enqueue_muon(const NsShape& s, const NsBuf& w, uint32_t count, const MuonIO& io,
                        const NsCoef* coef, int steps, hipStream_t stream);

// ------------------------------------------------------------------------------------
// MXFP4
// ------------------------------------------------------------------------------------
struct MxShape {
    uint64_t code_pitch, scale_pitch;   // bytes per row
};
inline MxShape mx_shape(uint64_t cols) {
    const uint64_t k = (cols + 127) / 128;
    return MxShape{k * 64, k * 4};
}
// st: null, or a step state whose skip flag keeps the copy as it is.
hipError_t launch_mx_quantize(const void* src, int dtype, uint64_t rows, uint64_t cols, uint64_t ld,
                              bool transpose, void* codes, void* scales, const DevState* st,
                              hipStream_t stream);
hipError_t launch_mx_dequantize(const void* codes, const void* scales, uint64_t rows, uint64_t cols,
                                void* dst, int dtype, uint64_t ld, hipStream_t stream);
hipError_t launch_mx_product(const void* a_codes, const void* a_scales, uint64_t m,
                             const void* b_codes, const void* b_scales, uint64_t n, uint64_t k,
                             void* c, int dtype, uint64_t ldc, hipStream_t stream);
// Which kernel launch_mx_product takes for an m x n result (the choice does not depend on k).
enum MxKernel : int32_t {
    kMxTiles64, kMxTiles128, kMxTiles256,
    kMxStream1x4, kMxStream1x16, kMxStream2x16, kMxStream4x16,   // 16 rows of a each, waves
};
MxKernel mx_product_kernel(uint64_t m, uint64_t n);

}  // namespace nz1
