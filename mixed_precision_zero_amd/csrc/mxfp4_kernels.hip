// mxfp4_kernels.hip -- MXFP4 quantise, dequantise and product on gfx950 (layout and
// rounding as include/neox_matrix.h states them).
#include "matrix_internal.h"
#include "tile_core.h"

#include <algorithm>
#include <type_traits>

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

// How the rows of an array are spread over blocks of 256 threads, a thread taking eight
// elements: `wide` threads side by side (a power of two) on 256 / wide rows.
struct Spread {
    uint32_t shift;        // log2(wide)
    uint32_t across;       // blocks across a row
    uint64_t blocks;
};
Spread spread(uint64_t rows, uint64_t units) {
    Spread s{};
    while (s.shift < 8 && (1ull << s.shift) < units) ++s.shift;
    s.across = (uint32_t)((units + (1ull << s.shift) - 1) >> s.shift);
    const uint64_t per = 256u >> s.shift;
    s.blocks = (rows + per - 1) / per * s.across;
    return s;
}
struct Unit {
    uint64_t row;
    uint32_t unit;         // eight elements each
    __device__ explicit Unit(const Spread& s) {
        const uint32_t down = blockIdx.x / s.across;
        row = (uint64_t)down * (256u >> s.shift) + (threadIdx.x >> s.shift);
        unit = ((blockIdx.x - down * s.across) << s.shift) + (threadIdx.x & ((1u << s.shift) - 1));
    }
};

__device__ __forceinline__ float decode(int dtype, uint32_t w, int k) {
    return half_to_float(dtype, (uint16_t)(w >> (16 * k)));
}

// Memory-bound.  Four neighbouring threads hold a block of 32, eight elements each (16 or 32
// bytes), find its largest magnitude with two exchanges, and write four bytes of codes each.
template <int DT>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const void* __restrict__ src, uint64_t R, uint64_t C,
                                                            uint64_t ld, bool vec, uint8_t* __restrict__ codes,
                                                            uint8_t* __restrict__ scales, MxShape sh, Spread sp,
                                                            const DevState* __restrict__ st) {
    if (st && st->skip) return;
    const Unit u(sp);
    // whole groups of four threads leave together (16 units fill 128 elements)
    if (u.row >= R || u.unit * 4ull >= sh.code_pitch) return;
    const uint64_t c = u.unit * 8ull, at = u.row * ld + c;
    float v[8];
    if (vec && c + 8 <= C) {
        if constexpr (DT == NEOX_F32) {
            const tf32x4 a = *(const tf32x4*)((const float*)src + at), b = *(const tf32x4*)((const float*)src + at + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = a[i];
                v[4 + i] = b[i];
            }
        } else {
            const tu32x4 a = *(const tu32x4*)((const uint16_t*)src + at);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = decode(DT, a[i / 2], i & 1);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = c + i < C ? load_elem(src, DT, at + i) : 0.0f;
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    top = max(top, (uint32_t)__shfl_xor((int)top, 1, 64));
    top = max(top, (uint32_t)__shfl_xor((int)top, 2, 64));
    const uint32_t s = scale_byte(top);
    const float inv = __uint_as_float((254u - (s == 255u ? 127u : s)) << 23);   // 2^(127 - s)
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) w |= e2m1(v[i] * inv) << (4 * i);
    *(uint32_t*)(codes + u.row * sh.code_pitch + u.unit * 4ull) = s == 255u ? 0u : w;
    if ((u.unit & 3) == 0) scales[u.row * sh.scale_pitch + u.unit / 4] = (uint8_t)s;
}

// The transpose: a thread takes 32 rows of one column of src, a wave 64 neighbouring columns.
template <int DT>
__global__ __launch_bounds__(256) void quantize_cols_kernel(const void* __restrict__ src, uint64_t R, uint64_t C,
                                                            uint64_t ld, uint8_t* __restrict__ codes,
                                                            uint8_t* __restrict__ scales, MxShape sh,
                                                            uint32_t across, uint32_t b0,
                                                            const DevState* __restrict__ st) {
    if (st && st->skip) return;
    // R, C: the copy's; its row r is src's column r.  b: block of 32 along it
    const uint32_t down = blockIdx.x / across, b = b0 + down;
    const uint64_t r = (uint64_t)(blockIdx.x - down * across) * 256 + threadIdx.x;
    if (r >= R) return;
    float v[32];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const uint64_t c = b * 32ull + i;
        v[i] = c < C ? load_elem(src, DT, c * ld + r) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 32; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    const uint32_t s = scale_byte(top);
    const float inv = __uint_as_float((254u - (s == 255u ? 127u : s)) << 23);
    tu32x4 w = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 32; ++i) w[i / 8] |= e2m1(v[i] * inv) << (4 * (i % 8));
    if (s == 255u) w = tu32x4{0, 0, 0, 0};
    *(tu32x4*)(codes + r * sh.code_pitch + b * 16ull) = w;
    scales[r * sh.scale_pitch + b] = (uint8_t)s;
}

__device__ __forceinline__ float e2m1_value(uint32_t c) {
    const uint32_t m = c & 7u;
    // codes 2..7: exponent field m / 2 over bias 1, one mantissa bit; 0 and 1: 0 and 0.5
    const float a = m < 2u ? 0.5f * (float)m : __uint_as_float(((126u + (m >> 1)) << 23) | ((m & 1u) << 22));
    return c & 8u ? -a : a;
}

template <int DT>
__global__ __launch_bounds__(256) void dequantize_kernel(const uint8_t* __restrict__ codes,
                                                         const uint8_t* __restrict__ scales, uint64_t R,
                                                         uint64_t C, MxShape sh, void* __restrict__ dst,
                                                         uint64_t ld, bool vec, Spread sp) {
    const Unit u(sp);
    const uint64_t c = u.unit * 8ull, at = u.row * ld + c;
    if (u.row >= R || c >= C) return;
    const uint32_t s = scales[u.row * sh.scale_pitch + u.unit / 4];
    const uint32_t w = *(const uint32_t*)(codes + u.row * sh.code_pitch + u.unit * 4ull);
    const float f = s == 255u ? __builtin_nanf("") : s == 0u ? 0x1p-127f : __uint_as_float(s << 23);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = e2m1_value(w >> (4 * i)) * f;
    if (vec && c + 8 <= C) {
        if constexpr (DT == NEOX_F32) {
            *(tf32x4*)((float*)dst + at) = tf32x4{v[0], v[1], v[2], v[3]};
            *(tf32x4*)((float*)dst + at + 4) = tf32x4{v[4], v[5], v[6], v[7]};
        } else {
            tu32x4 q;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                q[i] = float_to_half(DT, v[2 * i]) | (uint32_t)float_to_half(DT, v[2 * i + 1]) << 16;
            *(tu32x4*)((uint16_t*)dst + at) = q;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < C) store_elem(dst, DT, at + i, v[i]);
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

// Blocks of one launch: a grid has fewer than 2^32 threads.
constexpr uint64_t kGrid = 1ull << 23;

// Launches f(first row, rows, their spread) for as many rows at a time as a grid takes.
template <class F>
static void rows_in_grids(uint64_t rows, uint64_t units, F f) {
    const Spread one = spread(256, units);              // blocks for 256 rows
    const uint64_t most = std::max<uint64_t>(1, kGrid / one.blocks) * 256;
    for (uint64_t r = 0; r < rows; r += most) {
        const uint64_t n = std::min(most, rows - r);
        f(r, n, spread(n, units));
    }
}

// whether rows of eight elements can be moved 16 bytes at a time
static bool eights(const void* p, int dtype, uint64_t ld) {
    return (uintptr_t)p % 16 == 0 && ld * (dtype == NEOX_F32 ? 4 : 2) % 16 == 0;
}

hipError_t launch_mx_quantize(const void* src, int dtype, uint64_t rows, uint64_t cols, uint64_t ld,
                              bool transpose, void* codes, void* scales, const DevState* st,
                              hipStream_t stream) {
    const uint64_t R = transpose ? cols : rows, C = transpose ? rows : cols;
    const MxShape sh = mx_shape(C);
    auto run = [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        if (transpose) {
            const uint32_t across = (uint32_t)((R + 255) / 256);
            const uint64_t most = std::max<uint64_t>(1, kGrid / across);
            for (uint64_t b = 0; b < sh.scale_pitch; b += most)
                quantize_cols_kernel<DT><<<(uint32_t)(across * std::min(most, sh.scale_pitch - b)), 256, 0, stream>>>(
                    src, R, C, ld, (uint8_t*)codes, (uint8_t*)scales, sh, across, (uint32_t)b, st);
        } else {
            rows_in_grids(R, sh.code_pitch / 4, [&](uint64_t r, uint64_t n, const Spread& sp) {
                quantize_rows_kernel<DT><<<(uint32_t)sp.blocks, 256, 0, stream>>>(
                    (const uint8_t*)src + r * ld * (DT == NEOX_F32 ? 4 : 2), n, C, ld, eights(src, dtype, ld),
                    (uint8_t*)codes + r * sh.code_pitch, (uint8_t*)scales + r * sh.scale_pitch, sh, sp, st);
            });
        }
    };
    if (dtype == NEOX_F32) run(std::integral_constant<int, NEOX_F32>{});
    else if (dtype == NEOX_F16) run(std::integral_constant<int, NEOX_F16>{});
    else run(std::integral_constant<int, NEOX_BF16>{});
    return hipGetLastError();
}

hipError_t launch_mx_dequantize(const void* codes, const void* scales, uint64_t rows, uint64_t cols,
                                void* dst, int dtype, uint64_t ld, hipStream_t stream) {
    const MxShape sh = mx_shape(cols);
    auto run = [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        rows_in_grids(rows, (cols + 7) / 8, [&](uint64_t r, uint64_t n, const Spread& sp) {
            dequantize_kernel<DT><<<(uint32_t)sp.blocks, 256, 0, stream>>>(
                (const uint8_t*)codes + r * sh.code_pitch, (const uint8_t*)scales + r * sh.scale_pitch, n, cols, sh,
                (uint8_t*)dst + r * ld * (DT == NEOX_F32 ? 4 : 2), ld, eights(dst, dtype, ld), sp);
        });
    };
    if (dtype == NEOX_F32) run(std::integral_constant<int, NEOX_F32>{});
    else if (dtype == NEOX_F16) run(std::integral_constant<int, NEOX_F16>{});
    else run(std::integral_constant<int, NEOX_BF16>{});
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
