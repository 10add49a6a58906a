// column_sums.h -- the last step of a bias's gradient: joining the columns' sums of the blocks that
// shared the rows.  Device code of the element-wise passes and of the gradients' products.
#pragma once

#include "linear_internal.h"
#include "tile_core.h"

namespace nz1 {

template <int DT>
__device__ __forceinline__ void put_bias(const Backward& b, uint32_t c, float v) {
    if (b.accumulate) v += load_elem(b.dbias, DT, c);
    store_elem(b.dbias, DT, c, opaque(v));
}

// Adds up the `count` sums of 64 columns, eight loads a thread under way, in an order that does not
// depend on the block's threads: 16 shares of every 16th sum, joined in turn.  lds: 16 x 64.
template <int DT>
__device__ __forceinline__ void join_columns(const Backward& b, const float* part, uint32_t count, uint32_t block, float* lds) {
    const uint32_t c = block * 64 + (threadIdx.x & 63), waves = blockDim.x >> 6, wave = threadIdx.x >> 6;
    for (uint32_t share = wave; share < 16; share += waves) {
        float s = 0.0f;
        if (c < b.cols)
            for (uint32_t r = share; r < count; r += 16 * 8) {
                float t[8];
#pragma unroll
                for (uint32_t k = 0; k < 8; ++k) t[k] = r + 16 * k < count ? part[(uint64_t)(r + 16 * k) * b.cols + c] : 0.0f;
#pragma unroll
                for (uint32_t k = 0; k < 8; ++k) s += t[k];
            }
        lds[share * 64 + (threadIdx.x & 63)] = s;
    }
    __syncthreads();
    if (wave || c >= b.cols) return;
    float s = lds[threadIdx.x];
    for (int k = 1; k < 16; ++k) s += lds[k * 64 + threadIdx.x];
    put_bias<DT>(b, c, s);
}

}  // namespace nz1
