// linear_internal.h -- types shared by the host side and the gfx950 kernels of the linear
// layer's operators (include/neox_linear.h).  Not part of the public ABI.
#pragma once

#include "matrix_internal.h"
#include "neox_linear.h"

namespace nz1 {

// neox_drop as the kernels take it.
struct Drop {
    uint32_t limit;            // T: draws below it are dropped (0: no dropout)
    float scale;               // 65536 / (65536 - T); 0 for T = 65536
    uint32_t seed[2];
    uint64_t offset;
    const uint64_t* counter;
};
struct Epilogue {
    const uint16_t* bias;      // of the half type
    const void* residual;      // of the result's type
    uint16_t* pre;             // of the half type
    uint64_t residual_ld, pre_ld;
    int32_t act;
    Drop drop;
};

// One operand of a product: `side` rows or columns of the result, over K.  Rows of K
// consecutive elements, or (strided) K rows of `side` consecutive elements.
struct Operand {
    const uint16_t* at;
    uint64_t ld;
    bool strided;
    bool padded;               // its rows may be read up to a multiple of 8 elements: zeros
};
// out[j][i] = scale times the sum over k of p(i, k) q(j, k): I columns, J rows.
struct Product {
    Operand p, q;
    uint32_t I, J;
    uint64_t K;
    int32_t dtype;             // of the operands
    int32_t out_dtype;
    void* out;
    uint64_t out_ld;
    float scale;               // 1 but for gradients behind dropout
    Epilogue epi;              // (of nothing: all zero)
};
// Which kernel a product takes, and into how many shares of how many slabs (64 elements) its sums
// over K are split: by the sizes alone.  Deep: four slabs of K in LDS instead of two, for launches
// that leave a CU one block, whose loads are then all that is under way.
enum ProductKernel : int32_t { kTiles64, kTiles128, kTiles128Deep, kTiles256 };
struct ProductPlan {
    ProductKernel kernel;
    uint32_t shares;
    uint64_t slabs;
    double cost;               // us
};
ProductPlan product_plan(uint64_t I, uint64_t J, uint64_t K);
// Whether two products are worth one launch, and on which tiles.
bool pair_plan(uint64_t Ix, uint64_t Jx, const ProductPlan& x, uint64_t Iw, uint64_t Jw, const ProductPlan& w,
               ProductKernel* kernel);
// d = D(dy) act'(pre), and the sums of its columns times `scale`.  A linear layer's d lacks dropout's
// factor: drop.scale is 1 there, and `scale`, which its products take too, is the factor.  So d, which
// is rounded to half, overflows only where dy act'(pre) does, and is not rounded at all without an act.
struct Backward {
    const void* dy;
    const uint16_t* pre;       // null: no act
    void* d;                   // or null
    void* dbias;               // or null
    uint64_t dy_ld, pre_ld, d_ld;
    uint64_t rows, cols;
    int32_t dtype, act;
    bool accumulate;
    bool padded;               // rows of d are filled with zeros up to a multiple of 8 elements
    float scale;
    Drop drop;
};
// The sums of blocks that share the rows, [parts][cols] in FP32 in the workspace, are joined by
// launch_join, or by a kernel that follows anyway; 0 parts: dbias is written at once.
uint32_t backward_parts(uint64_t rows, uint64_t cols);
uint64_t backward_workspace(uint64_t rows, uint64_t cols);
hipError_t launch_backward(const Backward& b, void* workspace, bool join_here, hipStream_t stream);
hipError_t launch_join(const Backward& b, const void* workspace, hipStream_t stream);

// One product, or two (dx and dw, whose q is one matrix, read both ways) that may run side by side;
// either may be null.  join: null, or sums of a launch_backward, in `sums`, that are joined too.
uint64_t products_workspace(const Product* x, const Product* w);
hipError_t launch_products(const Product* x, const Product* w, const Backward* join, const void* sums, void* workspace,
                           hipStream_t stream);

hipError_t launch_dropout(const void* x, uint64_t x_ld, const void* bias, const void* residual, uint64_t residual_ld,
                          void* y, uint64_t y_ld, uint64_t rows, uint64_t cols, int32_t dtype, const Drop& drop,
                          hipStream_t stream);

// the MXFP4 product with an epilogue (mxfp4_kernels.hip)
hipError_t launch_mx_linear(const void* a_codes, const void* a_scales, uint64_t m, const void* b_codes,
                            const void* b_scales, uint64_t n, uint64_t k, void* c, int32_t dtype, uint64_t ldc,
                            int32_t half, const Epilogue& epi, hipStream_t stream);

}  // namespace nz1
