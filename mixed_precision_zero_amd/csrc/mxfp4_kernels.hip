// mxfp4_kernels.hip -- MXFP4 quantise, dequantise and product on gfx950 (layout and
// rounding as include/neox_matrix.h states them).
#include "matrix_internal.h"
#include "tile_core.h"

namespace nz1 {

namespace {

// E8M0 byte of a block from the FP32 bits of its largest magnitude: floor(log2) - 2, biased
// by 127, is the exponent field less 2 (subnormals fall to byte 0 as well); inf and NaN 255.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
    const uint32_t e = amax_bits >> 23;
    return e == 255u ? 255u : e > 2u ? e - 2u : 0u;
}

// E2M1 code of x (already divided by its block's scale, |x| < 8): ties to the even code.
// In each binade the step is a power of two, so rint() of x over it is the rounding.
__device__ __forceinline__ uint32_t e2m1(float x) {
    const float a = __builtin_fabsf(x);
    float c = a < 2.0f ? __builtin_rintf(a * 2.0f)
            : a < 4.0f ? __builtin_rintf(a) + 2.0f : __builtin_rintf(a * 0.5f) + 4.0f;
    c = c > 7.0f ? 7.0f : c;
    return (uint32_t)c | (__float_as_uint(x) >> 28 & 8u);
}

// a block of 32 elements by one thread: 16 bytes of codes and the scale byte
__device__ __forceinline__ uint32_t quantize32(const float (&v)[32], uint32_t (&w)[4]) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const uint32_t b = __float_as_uint(v[i]) & 0x7FFFFFFFu;
        top = b > top ? b : top;
    }
    const uint32_t s = scale_byte(top);
    const float inv = __uint_as_float((254u - (s == 255u ? 127u : s)) << 23);   // 2^(127 - s)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t u = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) u |= e2m1(v[8 * j + i] * inv) << (4 * i);
        w[j] = s == 255u ? 0u : u;
    }
    return s;
}

// one thread per block of 32; the copy is R x C (the source's transpose with T)
template <bool T>
__global__ __launch_bounds__(256) void quantize_kernel(const void* __restrict__ src, int dtype,
                                                       uint64_t R, uint64_t C, uint64_t ld,
                                                       uint8_t* __restrict__ codes,
                                                       uint8_t* __restrict__ scales,
                                                       MxShape sh, const DevState* __restrict__ st) {
    if (st && st->skip) return;
    const uint64_t per = sh.scale_pitch;
    const uint64_t id = (uint64_t)blockIdx.x * 256 + threadIdx.x;
    uint64_t r, b;
    if (T) { b = id / R; r = id % R; } else { r = id / per; b = id % per; }
    if (r >= R || b >= per) return;
    float v[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const uint64_t c = b * 32 + i;
        v[i] = c < C ? load_elem(src, dtype, T ? c * ld + r : r * ld + c) : 0.0f;
    }
    uint32_t w[4];
    const uint32_t s = quantize32(v, w);
    *(uint4*)(codes + r * sh.code_pitch + b * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    scales[r * sh.scale_pitch + b] = (uint8_t)s;
}

__device__ __forceinline__ float e2m1_value(uint32_t c) {
    const uint32_t m = c & 7u;
    // codes 2..7: exponent field m / 2 over bias 1, one mantissa bit; 0 and 1: 0 and 0.5
    const float a = m < 2u ? 0.5f * (float)m : __uint_as_float(((126u + (m >> 1)) << 23) | ((m & 1u) << 22));
    return c & 8u ? -a : a;
}

__global__ __launch_bounds__(256) void dequantize_kernel(const uint8_t* __restrict__ codes,
                                                         const uint8_t* __restrict__ scales,
                                                         uint64_t R, uint64_t C, MxShape sh,
                                                         void* __restrict__ dst, int dtype, uint64_t ld) {
    const uint64_t blocks = (C + 31) / 32;
    const uint64_t id = (uint64_t)blockIdx.x * 256 + threadIdx.x;
    const uint64_t r = id / blocks, b = id % blocks;
    if (r >= R) return;
    const uint32_t s = scales[r * sh.scale_pitch + b];
    const uint4 q = *(const uint4*)(codes + r * sh.code_pitch + b * 16);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    const float f = s == 255u ? __builtin_nanf("") : s == 0u ? 0x1p-127f : __uint_as_float(s << 23);
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const uint64_t c = b * 32 + i;
        if (c < C) store_elem(dst, dtype, r * ld + c, e2m1_value(w[i >> 3] >> (4 * (i & 7))) * f);
    }
}

// D = P Q^T with P the copy b (so that a lane's four results are consecutive columns of c)
template <class Core>
__global__ __launch_bounds__(Core::NT) void product_kernel(const uint8_t* a_codes, const uint8_t* a_scales,
                                                           uint32_t m, const uint8_t* b_codes,
                                                           const uint8_t* b_scales, uint32_t n, MxShape sh,
                                                           void* c, int dtype, uint64_t ldc) {
    __shared__ __attribute__((aligned(16))) uint8_t lds[Core::kLds];
    const uint32_t tn = (n + Core::BP - 1) / Core::BP;
    const uint32_t p0 = blockIdx.x % tn * Core::BP, q0 = blockIdx.x / tn * Core::BQ;
    const TileRows p{b_codes + (uint64_t)p0 * sh.code_pitch, b_scales + (uint64_t)p0 * sh.scale_pitch,
                     min((uint32_t)Core::BP, n - p0), (uint32_t)sh.code_pitch, (uint32_t)sh.scale_pitch};
    const TileRows q{a_codes + (uint64_t)q0 * sh.code_pitch, a_scales + (uint64_t)q0 * sh.scale_pitch,
                     min((uint32_t)Core::BQ, m - q0), (uint32_t)sh.code_pitch, (uint32_t)sh.scale_pitch};
    Core t;
    t.run(p, q, (uint32_t)sh.code_pitch, lds);
    const uint32_t lane = threadIdx.x & 63;
    const uint32_t jb = p0 + Core::wave_p() + (lane >> 4) * 4;
    const uint32_t ib = q0 + Core::wave_q() + (lane & 15);
#pragma unroll
    for (int u = 0; u < Core::TP; ++u)
#pragma unroll
        for (int v = 0; v < Core::TQ; ++v)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t i = ib + 16 * v, j = jb + 16 * u + e;
                if (i < m && j < n) store_elem(c, dtype, i * ldc + j, t.acc[u][v][e]);
            }
}

}  // namespace

hipError_t launch_mx_quantize(const void* src, int dtype, uint64_t rows, uint64_t cols, uint64_t ld,
                              bool transpose, void* codes, void* scales, const DevState* st,
                              hipStream_t stream) {
    const uint64_t R = transpose ? cols : rows, C = transpose ? rows : cols;
    const MxShape sh = mx_shape(C);
    const uint64_t blocks = (R * sh.scale_pitch + 255) / 256;
    if (transpose)
        quantize_kernel<true><<<(uint32_t)blocks, 256, 0, stream>>>(src, dtype, R, C, ld, (uint8_t*)codes,
                                                                    (uint8_t*)scales, sh, st);
    else
        quantize_kernel<false><<<(uint32_t)blocks, 256, 0, stream>>>(src, dtype, R, C, ld, (uint8_t*)codes,
                                                                     (uint8_t*)scales, sh, st);
    return hipGetLastError();
}

hipError_t launch_mx_dequantize(const void* codes, const void* scales, uint64_t rows, uint64_t cols,
                                void* dst, int dtype, uint64_t ld, hipStream_t stream) {
    const uint64_t blocks = (rows * ((cols + 31) / 32) + 255) / 256;
    dequantize_kernel<<<(uint32_t)blocks, 256, 0, stream>>>((const uint8_t*)codes, (const uint8_t*)scales,
                                                            rows, cols, mx_shape(cols), dst, dtype, ld);
    return hipGetLastError();
}

hipError_t launch_mx_product(const void* a_codes, const void* a_scales, uint64_t m, const void* b_codes,
                             const void* b_scales, uint64_t n, uint64_t k, void* c, int dtype,
                             uint64_t ldc, hipStream_t stream) {
    using Core = TileCore<128, 128, 2, 2, true>;
    const uint64_t blocks = ((m + Core::BQ - 1) / Core::BQ) * ((n + Core::BP - 1) / Core::BP);
    product_kernel<Core><<<(uint32_t)blocks, Core::NT, 0, stream>>>(
        (const uint8_t*)a_codes, (const uint8_t*)a_scales, (uint32_t)m, (const uint8_t*)b_codes,
        (const uint8_t*)b_scales, (uint32_t)n, mx_shape(k), c, dtype, ldc);
    return hipGetLastError();
}

}  // namespace nz1
