// linear_kernels.hip -- products of half-precision matrices with an epilogue on gfx950.
#include "epilogue.h"

namespace nz1 {

namespace {

// The value of element (row, col) of a result, from its sum.
template <class F>
__device__ __forceinline__ float finish(const Epilogue& e, int half, int out_dtype, uint64_t off, uint32_t row,
                                        uint32_t col, float v, F act) {
    if (e.bias) v += half_to_float(half, e.bias[col]);
    v = opaque(v);
    if (e.pre) e.pre[row * e.pre_ld + col] = float_to_half(half, v);
    v = activate<decltype(act)::value>(v);
    if (e.drop.limit) {
        const Bits b = philox(e.drop.seed, off, row, col / 8);
        const uint32_t k = col % 8;
        v = dropped(e.drop, k < 2 ? b.w[0] : k < 4 ? b.w[1] : k < 6 ? b.w[2] : b.w[3], k & 1, v);
    }
    if (e.residual) v += load_elem(e.residual, out_dtype, row * e.residual_ld + col);
    return v;
}

// 64 x 64 elements of the result by 256 threads, 4 x 4 each.
__global__ __launch_bounds__(256) void product_kernel(Product a) {
    __shared__ float sp[16][65], sq[16][65];
    const uint32_t across = (a.I + 63) / 64;
    const uint32_t i0 = blockIdx.x % across * 64, j0 = blockIdx.x / across * 64;
    const uint32_t tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float acc[4][4] = {};
    for (uint64_t k0 = 0; k0 < a.K; k0 += 16) {
        for (uint32_t t = threadIdx.x; t < 1024; t += 256) {
            const uint32_t kp = a.p.strided ? t / 64 : t % 16, ip = a.p.strided ? t % 64 : t / 16;
            const uint64_t k = k0 + kp;
            sp[kp][ip] = k < a.K && i0 + ip < a.I
                ? half_to_float(a.dtype, a.p.at[a.p.strided ? k * a.p.ld + i0 + ip : (i0 + ip) * a.p.ld + k]) : 0.0f;
            const uint32_t kq = a.q.strided ? t / 64 : t % 16, jq = a.q.strided ? t % 64 : t / 16;
            const uint64_t l = k0 + kq;
            sq[kq][jq] = l < a.K && j0 + jq < a.J
                ? half_to_float(a.dtype, a.q.at[a.q.strided ? l * a.q.ld + j0 + jq : (j0 + jq) * a.q.ld + l]) : 0.0f;
        }
        __syncthreads();
        for (int k = 0; k < 16; ++k)
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    acc[r][c] = __builtin_fmaf(sq[k][ty + 16 * r], sp[k][tx + 16 * c], acc[r][c]);
        __syncthreads();
    }
    const uint64_t off = drop_offset(a.epi.drop);
    with_act(a.epi.act, [&](auto act) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint32_t j = j0 + ty + 16 * r, i = i0 + tx + 16 * c;
                if (j >= a.J || i >= a.I) continue;
                float v = finish(a.epi, a.dtype, a.out_dtype, off, j, i, acc[r][c], act);
                if (a.accumulate) v += load_elem(a.out, a.out_dtype, j * a.out_ld + i);
                store_elem(a.out, a.out_dtype, j * a.out_ld + i, v);
            }
    });
}

}  // namespace

uint64_t product_workspace(const Product&) { return 0; }

hipError_t launch_product(const Product& p, void*, hipStream_t stream) {
    const uint32_t blocks = ((p.I + 63) / 64) * ((p.J + 63) / 64);
    product_kernel<<<blocks, 256, 0, stream>>>(p);
    return hipGetLastError();
}

}  // namespace nz1
