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

// Eight elements' codes at scale byte s, the first in the lowest bits.  The conversion rounds to
// the nearest value, ties to the even code, and takes what lies above 6 to 6; it divides by the
// power of two that the scale operand's exponent field names, 0 meaning 2^-127, as here.
__device__ __forceinline__ uint32_t codes8(const float* v, uint32_t s) {
    const float f = __uint_as_float(s << 23);
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], f, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], f, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], f, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], f, 3);
    return s == 255u ? 0u : w;
}

// How the rows of an array are spread over blocks of 256 threads, a thread taking eight
// elements of each of `deep` rows: `wide` threads side by side (a power of two) on 256 / wide
// rows, `deep` times.
struct Spread {
    uint32_t shift;        // log2(wide)
    uint32_t across;       // blocks across a row
    uint64_t blocks;
};
Spread spread(uint64_t rows, uint64_t units, uint32_t deep) {
    Spread s{};
    while (s.shift < 8 && (1ull << s.shift) < units) ++s.shift;
    s.across = (uint32_t)((units + (1ull << s.shift) - 1) >> s.shift);
    const uint64_t per = (256u >> s.shift) * deep;
    s.blocks = (rows + per - 1) / per * s.across;
    return s;
}
struct Unit {
    uint64_t row;          // the first; the others `step` further each
    uint32_t unit;         // eight elements each
    uint32_t step;
    __device__ Unit(const Spread& s, uint32_t deep) {
        const uint32_t down = blockIdx.x / s.across;
        step = 256u >> s.shift;
        row = (uint64_t)down * (step * deep) + (threadIdx.x >> s.shift);
        unit = ((blockIdx.x - down * s.across) << s.shift) + (threadIdx.x & ((1u << s.shift) - 1));
    }
};

__device__ __forceinline__ float decode(int dtype, uint32_t w, int k) {
    return half_to_float(dtype, (uint16_t)(w >> (16 * k)));
}

// Rows a thread has in flight, measured (us, 24576 x 6144 at 1 / 2 / 4): quantise FP32 114 /
// 130 / 134, BF16 117 / 104 / 104; dequantise to BF16 108 / 96 / 77.
template <int DT>
constexpr uint32_t kDeepRows = DT == NEOX_F32 ? 1 : 2;
constexpr uint32_t kDeepBack = 4;

template <int DT>
__device__ __forceinline__ void load_eight(const void* src, uint64_t at, uint64_t c, uint64_t C, bool vec, float (&v)[8]) {
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
}

// Memory-bound.  Four neighbouring threads hold a block of 32, eight elements each (16 or 32
// bytes), find its largest magnitude with two exchanges, and write four bytes of codes each.
// Measured: FP32 24576 x 6144 136 us, 5.0 TB/s; BF16 8192 x 6144 25 us (5.1).
template <int DT>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const void* __restrict__ src, uint64_t R, uint64_t C,
                                                            uint64_t ld, bool vec, uint8_t* __restrict__ codes,
                                                            uint8_t* __restrict__ scales, MxShape sh, Spread sp,
                                                            const DevState* __restrict__ st) {
    if (st && st->skip) return;
    constexpr uint32_t kDeep = kDeepRows<DT>;
    const Unit u(sp, kDeep);
    // whole groups of four threads leave together (16 units fill 128 elements)
    if (u.unit * 4ull >= sh.code_pitch) return;
    const uint64_t c = u.unit * 8ull;
    float v[kDeep][8];
#pragma unroll
    for (uint32_t k = 0; k < kDeep; ++k) {
        const uint64_t row = u.row + k * u.step, at = row * ld + c;
        if (row < R) load_eight<DT>(src, at, c, C, vec, v[k]);
    }
#pragma unroll
    for (uint32_t k = 0; k < kDeep; ++k) {
        const uint64_t row = u.row + k * u.step;
        if (row >= R) break;
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[k][i]) & 0x7FFFFFFFu);
        top = max(top, (uint32_t)__shfl_xor((int)top, 1, 64));
        top = max(top, (uint32_t)__shfl_xor((int)top, 2, 64));
        const uint32_t s = scale_byte(top);
        *(uint32_t*)(codes + row * sh.code_pitch + u.unit * 4ull) = codes8(v[k], s);
        if ((u.unit & 3) == 0) scales[row * sh.scale_pitch + u.unit / 4] = (uint8_t)s;
    }
}

// The transpose: a thread takes 32 rows of one column of src (of two, as one dword, where src
// has 16-bit elements and lies for it), a wave 64 or 128 neighbouring columns, and the block's
// four waves four blocks of 32 of each: together 64 bytes of codes and four scales of each row
// of the copy, so that the L2 gets whole sectors from one CU.  Memory-bound: FP32 24576 x 6144
// 180 us, 3.8 TB/s (rows of 256 bytes read by a wave, 16 bytes written by a lane).
template <int DT, int N>
__global__ __launch_bounds__(256) void quantize_cols_kernel(const void* __restrict__ src, uint64_t R, uint64_t C,
                                                            uint64_t ld, uint8_t* __restrict__ codes,
                                                            uint8_t* __restrict__ scales, MxShape sh,
                                                            uint32_t across, uint64_t b0,
                                                            const DevState* __restrict__ st) {
    if (st && st->skip) return;
    // R, C: the copy's; its row r is src's column r.  b: block of 32 along it
    const uint32_t down = blockIdx.x / across;
    const uint64_t b = (b0 + down) * 4 + (threadIdx.x >> 6);
    const uint64_t r = ((uint64_t)(blockIdx.x - down * across) * 64 + (threadIdx.x & 63)) * N;
    if (r >= R) return;
    float v[N][32];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const uint64_t c = b * 32 + i;
        if constexpr (N == 1) {
            v[0][i] = c < C ? load_elem(src, DT, c * ld + r) : 0.0f;
        } else {
            const uint32_t q = c < C ? *(const uint32_t*)((const uint16_t*)src + c * ld + r) : 0u;
            v[0][i] = decode(DT, q, 0);
            v[1][i] = decode(DT, q, 1);
        }
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) top = max(top, __float_as_uint(v[n][i]) & 0x7FFFFFFFu);
        const uint32_t s = scale_byte(top);
        tu32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = codes8(v[n] + 8 * i, s);
        *(tu32x4*)(codes + (r + n) * sh.code_pitch + b * 16) = w;
        scales[(r + n) * sh.scale_pitch + b] = (uint8_t)s;
    }
}

__device__ __forceinline__ float e2m1_value(uint32_t c) {
    const uint32_t m = c & 7u;
    // codes 2..7: exponent field m / 2 over bias 1, one mantissa bit; 0 and 1: 0 and 0.5
    const float a = m < 2u ? 0.5f * (float)m : __uint_as_float(((126u + (m >> 1)) << 23) | ((m & 1u) << 22));
    return c & 8u ? -a : a;
}

// Memory-bound: BF16 24576 x 6144 73 us, 5.2 TB/s.
template <int DT>
__global__ __launch_bounds__(256) void dequantize_kernel(const uint8_t* __restrict__ codes,
                                                         const uint8_t* __restrict__ scales, uint64_t R,
                                                         uint64_t C, MxShape sh, void* __restrict__ dst,
                                                         uint64_t ld, bool vec, Spread sp) {
    constexpr uint32_t kDeep = kDeepBack;
    const Unit u(sp, kDeep);
    const uint64_t c = u.unit * 8ull;
    if (c >= C) return;
    uint32_t scale[kDeep], code[kDeep];
#pragma unroll
    for (uint32_t k = 0; k < kDeep; ++k) {
        const uint64_t row = u.row + k * u.step;
        if (row < R) {
            scale[k] = scales[row * sh.scale_pitch + u.unit / 4];
            code[k] = *(const uint32_t*)(codes + row * sh.code_pitch + u.unit * 4ull);
        }
    }
#pragma unroll
    for (uint32_t k = 0; k < kDeep; ++k) {
        const uint64_t row = u.row + k * u.step, at = row * ld + c;
        if (row >= R) break;
        const uint32_t s = scale[k], w = code[k];
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
}

// ------------------------------------------------------------------------------------
// product: D = P Q^T with P the copy b (its rows are columns of c), Q the copy a, so that a
// lane's four results are consecutive columns of c
//
// Large results are bound by the matrix units and LDS together: 8192 x 24576 x 6144 582 us,
// 4.25 PFLOP/s.  A slab takes 1.95 us on a CU; its products alone, from registers, 1.1 (7.9
// PFLOP/s on all CUs), its LDS traffic 0.9, and the scales' share of that is 10% of the time.
// Smaller ones take 128 x 128 or 64 x 64 tiles: 333 x 4096 x 1024 6.3 us, launch and latency
// mostly.
// ------------------------------------------------------------------------------------
struct ProductArgs {
    const uint8_t *a_codes, *a_scales, *b_codes, *b_scales;
    void* c;
    uint64_t ldc;
    uint32_t m, n;
    uint32_t pitch, spitch;    // bytes per row of the codes and the scales
    int32_t dtype;
    bool vec;                  // rows of c can be written 16 bytes at a time
};

__device__ __forceinline__ void store_four(const ProductArgs& a, uint32_t i, uint32_t j, tf32x4 x) {
    if (i >= a.m) return;
    const uint64_t at = i * a.ldc + j;
    if (a.vec && j + 4 <= a.n) {
        if (a.dtype == NEOX_F32) *(tf32x4*)((float*)a.c + at) = x;
        else *(ushort4*)((uint16_t*)a.c + at) = make_ushort4(float_to_half(a.dtype, x[0]), float_to_half(a.dtype, x[1]),
                                                             float_to_half(a.dtype, x[2]), float_to_half(a.dtype, x[3]));
    } else {
#pragma unroll
        for (uint32_t e = 0; e < 4; ++e)
            if (j + e < a.n) store_elem(a.c, a.dtype, at + e, x[e]);
    }
}

// One tile of c: rows at.j .., columns at.i ..
template <class Core>
__device__ __forceinline__ void product_tile(const ProductArgs& a, const TileAt& at, uint8_t* lds) {
    const TileRows p{a.b_codes + (uint64_t)at.i * a.pitch, a.b_scales + (uint64_t)at.i * a.spitch,
                     min((uint32_t)Core::BP, a.n - at.i), a.pitch, a.spitch};
    const TileRows q{a.a_codes + (uint64_t)at.j * a.pitch, a.a_scales + (uint64_t)at.j * a.spitch,
                     min((uint32_t)Core::BQ, a.m - at.j), a.pitch, a.spitch};
    Core t;
    t.run(p, q, a.pitch, lds);
    using P = Piece<Core>;
#pragma unroll
    for (int u0 = 0; u0 < Core::TP; u0 += P::kU) {
        const P pc(at, u0, lds);
        if (a.dtype != NEOX_F32 && a.vec && pc.i + 16 * P::kU <= a.n) {
            // 16-bit results: whole rows through LDS
#pragma unroll
            for (int u = 0; u < P::kU; ++u)
#pragma unroll
                for (int v = 0; v < P::kV; ++v) {
                    const tf32x4 x = t.acc[u0 + u][v];
                    const ushort4 h = make_ushort4(float_to_half(a.dtype, x[0]), float_to_half(a.dtype, x[1]),
                                                   float_to_half(a.dtype, x[2]), float_to_half(a.dtype, x[3]));
                    *(ushort4*)pc.down(pc.l0, u, v) = h;
                }
            const uint32_t left = pc.j < a.m ? a.m - pc.j : 0u;
            P::Down::store(pc.l0, (uint16_t*)a.c + (uint64_t)pc.j * a.ldc + pc.i, a.ldc, left);
        } else {
#pragma unroll
            for (int u = 0; u < P::kU; ++u)
#pragma unroll
                for (int v = 0; v < P::kV; ++v)
                    store_four(a, pc.j + 16 * v + pc.lj, pc.i + 16 * u + pc.li, t.acc[u0 + u][v]);
        }
    }
}

using Mx256 = TileCore<256, 256, 2, 4, true>;
using Mx128 = TileCore<128, 128, 2, 4, true>;        // by the same 512 threads: its quarters too
using Mx64 = TileCore<64, 64, 2, 2, true>;

__global__ __launch_bounds__(512, 2) void product_mixed_kernel(ProductArgs a, TileMap m) {
    __shared__ __attribute__((aligned(16))) uint8_t lds[Mx256::kLds];
    const TileAt at = place<false>(m);
    if (at.full) product_tile<Mx256>(a, at, lds);
    else if (!at.none) product_tile<Mx128>(a, at, lds);
}
// Two blocks share a CU, and so a SIMD's registers four waves.  Eight waves a tile instead of
// four: 700 x 5000 x 4096 18.6 -> 14.5 us, 512 x 6144 x 6144 23.1 -> 19.4.
template <class Core>
__global__ __launch_bounds__(Core::NT, 4) void product_even_kernel(ProductArgs a) {
    __shared__ __attribute__((aligned(16))) uint8_t lds[Core::kLds];
    const uint32_t p = (a.n + Core::BP - 1) / Core::BP;
    TileAt at{};
    at.i = blockIdx.x % p * Core::BP;
    at.j = blockIdx.x / p * Core::BQ;
    product_tile<Core>(a, at, lds);
}

// Few rows of a (up to 16 MT): bound by reading b once.  A block takes 16 rows of b; its WK
// waves share K in steps of 512 elements and add their results at the end in wave order.  No
// LDS on the way: per step a lane reads 64 bytes of its row (four blocks of 128 elements, a
// group of lanes each 32 of them) and their four scale bytes as one dword, so each of the four
// products of a step picks its scale by byte.  Measured: one row by 24576 x 6144 (80 MB) 16.0
// us, 5.0 TB/s.
template <int MT, int WK>
__global__ __launch_bounds__(WK * 64) void product_thin_kernel(ProductArgs a) {
    static_assert(WK >= MT, "");
    __shared__ tf32x4 part[WK][MT][64];
    const uint32_t lane = threadIdx.x & 63, l16 = lane & 15, g = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t n0 = blockIdx.x * 16;
    const uint32_t rows = min(16u, a.n - n0);
    const rsrc_t pb = raw_buffer(a.b_codes + (uint64_t)n0 * a.pitch, rows * a.pitch);
    const rsrc_t ps = raw_buffer(a.b_scales + (uint64_t)n0 * a.spitch, rows * a.spitch);
    const rsrc_t qb = raw_buffer(a.a_codes, a.m * a.pitch), qs = raw_buffer(a.a_scales, a.m * a.spitch);
    const uint32_t steps = (a.pitch + 255) / 256;
    tf32x4 acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = tf32x4{0, 0, 0, 0};
    // behind the end of a row: zeros (and scale byte 0)
    auto code = [&](const rsrc_t& r, uint32_t row, uint32_t s, int k) {
        const uint32_t at = s * 256 + g * 64 + k * 16;
        return __builtin_amdgcn_raw_buffer_load_b128(r, at < a.pitch ? row * a.pitch + at : kNowhere, 0, 0);
    };
    auto scale = [&](const rsrc_t& r, uint32_t row, uint32_t s) {
        const uint32_t at = s * 16 + g * 4;
        return __builtin_amdgcn_raw_buffer_load_b32(r, at < a.spitch ? row * a.spitch + at : kNowhere, 0, 0);
    };
    auto wide = [](tu32x4 f) { return ti32x8{(int)f.x, (int)f.y, (int)f.z, (int)f.w, 0, 0, 0, 0}; };
#pragma unroll 2
    for (uint32_t s = wave; s < steps; s += WK) {
        tu32x4 p[4], q[MT][4];
        uint32_t sp, sq[MT];
#pragma unroll
        for (int k = 0; k < 4; ++k) p[k] = __builtin_bit_cast(tu32x4, code(pb, l16, s, k));
        sp = scale(ps, l16, s);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
#pragma unroll
            for (int k = 0; k < 4; ++k) q[t][k] = __builtin_bit_cast(tu32x4, code(qb, 16 * t + l16, s, k));
            sq[t] = scale(qs, 16 * t + l16, s);
        }
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(p[0]), wide(q[t][0]), acc[t], 4, 4, 0, (int)sp, 0, (int)sq[t]);
            acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(p[1]), wide(q[t][1]), acc[t], 4, 4, 1, (int)sp, 1, (int)sq[t]);
            acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(p[2]), wide(q[t][2]), acc[t], 4, 4, 2, (int)sp, 2, (int)sq[t]);
            acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(p[3]), wide(q[t][3]), acc[t], 4, 4, 3, (int)sp, 3, (int)sq[t]);
        }
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) part[wave][t][lane] = acc[t];
    __syncthreads();
    if (wave < MT) {
        // wave t finishes result tile t
        tf32x4 x = part[0][wave][lane];
#pragma unroll
        for (int w = 1; w < WK; ++w) x = x + part[w][wave][lane];
        store_four(a, 16 * wave + l16, n0 + 4 * g, x);
    }
}

}  // namespace

// Blocks of one launch: a grid has fewer than 2^32 threads.
constexpr uint64_t kGrid = 1ull << 23;
// Rows of a transposed copy that a launch takes.
constexpr uint64_t kMostRows = 1ull << 22;

// Launches f(first row, rows, their spread) for as many rows at a time as a grid takes.
template <class F>
static void rows_in_grids(uint64_t rows, uint64_t units, uint32_t deep, F f) {
    const Spread one = spread(1, units, deep);          // (at most 2^20 blocks across)
    const uint64_t most = kGrid / one.across * ((256u >> one.shift) * deep);
    for (uint64_t r = 0; r < rows; r += most) {
        const uint64_t n = std::min(most, rows - r);
        f(r, n, spread(n, units, deep));
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
            auto cols = [&](auto nn) {
                constexpr int N = decltype(nn)::value;
                for (uint64_t r = 0; r < R; r += kMostRows) {
                    const uint64_t n = std::min(kMostRows, R - r);
                    const uint32_t across = (uint32_t)((n + 64 * N - 1) / (64 * N));
                    const uint64_t down = sh.scale_pitch / 4, most = kGrid / across;
                    for (uint64_t d = 0; d < down; d += most)
                        quantize_cols_kernel<DT, N><<<(uint32_t)(across * std::min(most, down - d)), 256, 0, stream>>>(
                            (const uint8_t*)src + r * (DT == NEOX_F32 ? 4 : 2), n, C, ld,
                            (uint8_t*)codes + r * sh.code_pitch, (uint8_t*)scales + r * sh.scale_pitch, sh, across, d, st);
                }
            };
            if (DT != NEOX_F32 && R % 2 == 0 && ld % 2 == 0 && (uintptr_t)src % 4 == 0)
                cols(std::integral_constant<int, DT == NEOX_F32 ? 1 : 2>{});
            else
                cols(std::integral_constant<int, 1>{});
        } else {
            rows_in_grids(R, sh.code_pitch / 4, kDeepRows<DT>, [&](uint64_t r, uint64_t n, const Spread& sp) {
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
        rows_in_grids(rows, (cols + 7) / 8, kDeepBack, [&](uint64_t r, uint64_t n, const Spread& sp) {
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

// The launch of 256 x 256 tiles, and its cost.
static TileMap mx_tiles256(uint64_t m, uint64_t n, double* cost, uint64_t* blocks) {
    return plan_tiles(256, false, (uint32_t)n, (uint32_t)m, 1, 2.0, 1.0, cost, blocks);
}
static uint64_t tiles(uint64_t m, uint64_t n, uint64_t unit) { return ((m + unit - 1) / unit) * ((n + unit - 1) / unit); }

MxKernel mx_product_kernel(uint64_t m, uint64_t n) {
    // us per slab of 256 elements of K, measured on the full chip: a round of 256 x 256 tiles
    // 2.0, of quarters in the same kernel 1.0, of 128 x 128 tiles 0.6 with one block a CU and
    // 1.25 with two, of 64 x 64 tiles 0.28 (65 x 6144 x 8192 12 us, by 128 x 128 ones 20; 65 x 1024
    // x 16384 20.5 and 35)
    double c256 = 0.0;
    uint64_t blocks = 0;
    mx_tiles256(m, n, &c256, &blocks);
    const uint64_t n128 = tiles(m, n, 128), n64 = tiles(m, n, 64);
    const double c128 = n128 <= kCUs ? 0.6 : 1.25 * (double)((n128 + 2 * kCUs - 1) / (2 * kCUs));
    const double c64 = n64 <= kGrid ? 0.28 * (double)((n64 + kCUs - 1) / kCUs) : 1e300;
    // Up to 64 rows the streaming kernel where it takes less by its own cost, for each 256 blocks
    // 0.07 a slab and 0.09 for 16 rows of a.  Streaming and tiles, us: 16 rows by 24576 x 6144 23.7
    // and 15.1 (1 row streaming 15.6, the same for tiles as 16), 64 rows 57 and 16.3; 16 rows by
    // 6144 x 8192 11.3 and 11.6, 64 rows 27.0 and 12.2; 64 rows by 1024 x 16384 24.0 and 20.3.
    // (Above 2^29 rows of b a grid holds no 64 x 64 tiles any more, and 128 x 128 ones cost what
    // streaming does: they take those, in one launch.)
    const double thin = (0.07 + 0.09 * (double)m / 16) * std::max(1.0, (double)n / (16 * kCUs));
    if (m <= 64 && n64 <= kGrid && thin <= std::min(c64, c128)) {
        // enough waves for the chip: more of them share K where there are few rows of b (from 13
        // rows of a on, 64 x 64 tiles take over before b has that many)
        if (m > 16) return m <= 32 ? kMxStream2x16 : kMxStream4x16;
        return n > 16 * (4 * kCUs - 1) ? kMxStream1x4 : kMxStream1x16;
    }
    if (c64 < c128 && c64 < c256) return kMxTiles64;
    return c256 < c128 ? kMxTiles256 : kMxTiles128;
}

hipError_t launch_mx_product(const void* a_codes, const void* a_scales, uint64_t m, const void* b_codes,
                             const void* b_scales, uint64_t n, uint64_t k, void* c, int dtype,
                             uint64_t ldc, hipStream_t stream) {
    const MxShape sh = mx_shape(k);
    const uint64_t es = dtype == NEOX_F32 ? 4 : 2;
    const ProductArgs a{(const uint8_t*)a_codes, (const uint8_t*)a_scales, (const uint8_t*)b_codes,
                        (const uint8_t*)b_scales, c, ldc, (uint32_t)m, (uint32_t)n, (uint32_t)sh.code_pitch,
                        (uint32_t)sh.scale_pitch, dtype, (uintptr_t)c % 16 == 0 && ldc * es % 16 == 0};
    const uint32_t stripes = (uint32_t)((n + 15) / 16);
    switch (mx_product_kernel(m, n)) {
    case kMxStream1x4: product_thin_kernel<1, 4><<<stripes, 256, 0, stream>>>(a); break;
    case kMxStream1x16: product_thin_kernel<1, 16><<<stripes, 1024, 0, stream>>>(a); break;
    case kMxStream2x16: product_thin_kernel<2, 16><<<stripes, 1024, 0, stream>>>(a); break;
    case kMxStream4x16: product_thin_kernel<4, 16><<<stripes, 1024, 0, stream>>>(a); break;
    case kMxTiles64: product_even_kernel<Mx64><<<(uint32_t)tiles(m, n, 64), Mx64::NT, 0, stream>>>(a); break;
    case kMxTiles128: product_even_kernel<Mx128><<<(uint32_t)tiles(m, n, 128), Mx128::NT, 0, stream>>>(a); break;
    case kMxTiles256: {
        double cost = 0.0;
        uint64_t blocks = 0;
        const TileMap map = mx_tiles256(m, n, &cost, &blocks);
        product_mixed_kernel<<<(uint32_t)blocks, 512, 0, stream>>>(a, map);
    }
    }
    return hipGetLastError();
}

}  // namespace nz1
