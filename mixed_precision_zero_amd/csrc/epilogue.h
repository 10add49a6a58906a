// epilogue.h -- device code that the linear layer's kernels and the MXFP4 product share: the
// random bits of dropout, activations and their slopes (include/neox_linear.h).
#pragma once

#include "linear_internal.h"
#include "tile_core.h"

#include <type_traits>

namespace nz1 {

// ------------------------------------------------------------------------------------
// dropout
// ------------------------------------------------------------------------------------
// The bits of elements (row, 8 unit) to (row, 8 unit + 7): Philox-4x32, ten rounds, written from
// its publication (Salmon et al., SC 2011): a round multiplies two words by constants and mixes
// the products' halves with the other two words and the round's key.  16 bits an element instead
// of 32: the 20 wide multiplications of a call, at a quarter of the rate of other instructions,
// are most of what dropout computes, and probabilities in steps of 2^-16 are fine enough.
struct Bits {
    uint32_t w[4];
};
// one instruction (0x96: the truth table of a ^ b ^ c)
__device__ __forceinline__ uint32_t xor3(uint32_t a, uint32_t b, uint32_t c) { return __builtin_amdgcn_bitop3_b32(a, b, c, 0x96); }
__device__ __forceinline__ Bits philox(const uint32_t (&seed)[2], uint64_t offset, uint32_t row, uint32_t unit) {
    uint32_t a = unit, b = row, c = (uint32_t)offset, d = (uint32_t)(offset >> 32);
    uint32_t k0 = seed[0], k1 = seed[1];
    // (the keys of all rounds would be kept, and crowd out a product's results)
    asm volatile("" : "+s"(k0), "+s"(k1));
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t x = (uint64_t)0xD2511F53u * a, y = (uint64_t)0xCD9E8D57u * c;
        a = xor3((uint32_t)(y >> 32), b, k0);
        b = (uint32_t)y;
        c = xor3((uint32_t)(x >> 32), d, k1);
        d = (uint32_t)x;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return Bits{{a, b, c, d}};
}
// o of the header: read once, when the work runs
__device__ __forceinline__ uint64_t drop_offset(const Drop& d) {
    return d.offset + (d.limit && d.counter ? *d.counter : 0ull);
}
// A dropped element is zero whatever v is.
__device__ __forceinline__ float dropped(const Drop& d, uint32_t word, int odd, float v) {
    const uint32_t bits = odd ? word >> 16 : word & 0xFFFFu;
    return bits >= d.limit ? v * d.scale : 0.0f;
}

// ------------------------------------------------------------------------------------
// activations, by the hardware's exp2 and reciprocal (1 ulp each)
// ------------------------------------------------------------------------------------
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float rcp_fast(float x) { return __builtin_amdgcn_rcpf(x); }

// The normal distribution's tail behind |x|, times exp(x^2 / 2): with t = 1 / (1 + 0.3 |x|) a
// polynomial of t, fitted on [0, 15] to 7.1e-8 relative (and FP32's roundings on top).
__device__ __forceinline__ float tail_scaled(float ax) {
    const float t = rcp_fast(__builtin_fmaf(0.3f, ax, 1.0f));
    float r = 0.03842540085315704f;
    r = __builtin_fmaf(r, t, -0.16939479112625122f);
    r = __builtin_fmaf(r, t, 0.22913166880607605f);
    r = __builtin_fmaf(r, t, -0.07704470306634903f);
    r = __builtin_fmaf(r, t, 0.1429063081741333f);
    r = __builtin_fmaf(r, t, 0.09452608972787857f);
    r = __builtin_fmaf(r, t, 0.12196046113967896f);
    r = __builtin_fmaf(r, t, 0.11948209255933762f);
    return __builtin_fmaf(r, t, 7.495441877836129e-06f);
}
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kTanhC = 0.7978845608028654f;          // sqrt(2 / pi)

// Below -kFar an act or slope is less than 3e-36 and taken as zero: near there the formulas'
// exponentials overflow, and at -inf they would give inf * 0.  Above kFar a slope is 1.  A NaN
// passes the comparisons.
template <int ACT>
constexpr float kFar = ACT == NEOX_ACT_GELU ? 15.0f : ACT == NEOX_ACT_GELU_TANH ? 10.0f : 88.0f;

template <int ACT>
__device__ __forceinline__ float activate(float x) {
    if constexpr (ACT == NEOX_ACT_NONE) return x;
    if constexpr (ACT == NEOX_ACT_RELU) return x <= 0.0f ? 0.0f : x;
    if constexpr (ACT == NEOX_ACT_GELU) {
        const float q = tail_scaled(__builtin_fabsf(x)) * exp2_fast(x * x * (-0.5f * kLog2e));
        // (1 - q) from the tail itself: x (1 - q) for x > 0
        const float y = x > 0.0f ? __builtin_fmaf(-x, q, x) : x * q;
        return x < -kFar<ACT> ? 0.0f : x > kFar<ACT> ? x : y;
    }
    if constexpr (ACT == NEOX_ACT_GELU_TANH) {
        // (1 + tanh u) / 2 = 1 / (1 + exp(-2 u))
        const float u = x * __builtin_fmaf(x * x, -2.0f * kLog2e * kTanhC * 0.044715f, -2.0f * kLog2e * kTanhC);
        const float y = x * rcp_fast(1.0f + exp2_fast(u));
        return x < -kFar<ACT> ? 0.0f : y;
    }
    if constexpr (ACT == NEOX_ACT_SILU) {
        const float y = x * rcp_fast(1.0f + exp2_fast(x * -kLog2e));
        return x < -kFar<ACT> ? 0.0f : y;
    }
}

template <int ACT>
__device__ __forceinline__ float slope(float x) {
    if constexpr (ACT == NEOX_ACT_NONE) return 1.0f;
    if constexpr (ACT == NEOX_ACT_RELU) return x <= 0.0f ? 0.0f : x > 0.0f ? 1.0f : x;
    if constexpr (ACT == NEOX_ACT_GELU) {
        const float e = exp2_fast(x * x * (-0.5f * kLog2e));
        const float q = tail_scaled(__builtin_fabsf(x)) * e;
        const float y = __builtin_fmaf(x * 0.3989422804014327f, e, x > 0.0f ? 1.0f - q : q);
        return x < -kFar<ACT> ? 0.0f : x > kFar<ACT> ? 1.0f : y;
    }
    if constexpr (ACT == NEOX_ACT_GELU_TANH) {
        const float xx = x * x;
        const float e = exp2_fast(x * __builtin_fmaf(xx, -2.0f * kLog2e * kTanhC * 0.044715f, -2.0f * kLog2e * kTanhC));
        const float s = rcp_fast(1.0f + e);
        // s + x s (1 - s) 2 u', 1 - s = e s
        const float du = __builtin_fmaf(xx, 6.0f * kTanhC * 0.044715f, 2.0f * kTanhC);
        const float y = __builtin_fmaf(x * s * (e * s), du, s);
        return x < -kFar<ACT> ? 0.0f : x > kFar<ACT> ? 1.0f : y;
    }
    if constexpr (ACT == NEOX_ACT_SILU) {
        const float e = exp2_fast(x * -kLog2e), s = rcp_fast(1.0f + e);
        const float y = __builtin_fmaf(x * s, e * s, s);
        return x < -kFar<ACT> ? 0.0f : x > kFar<ACT> ? 1.0f : y;
    }
}
template <class F>
__host__ __device__ __forceinline__ void with_act(int32_t act, F f) {
    switch (act) {
    case NEOX_ACT_RELU: f(std::integral_constant<int, NEOX_ACT_RELU>{}); break;
    case NEOX_ACT_GELU: f(std::integral_constant<int, NEOX_ACT_GELU>{}); break;
    case NEOX_ACT_GELU_TANH: f(std::integral_constant<int, NEOX_ACT_GELU_TANH>{}); break;
    case NEOX_ACT_SILU: f(std::integral_constant<int, NEOX_ACT_SILU>{}); break;
    default: f(std::integral_constant<int, NEOX_ACT_NONE>{});
    }
}

// ------------------------------------------------------------------------------------
// eight neighbouring elements of a row
// ------------------------------------------------------------------------------------
// Vectors at any element's address: gfx950 serves unaligned vector accesses of global memory, at
// full rate within a cache line, so rows that begin anywhere take one access each.
typedef tu32x4 __attribute__((aligned(2))) loose_u32x4;
typedef tf32x4 __attribute__((aligned(4))) loose_f32x4;

// NT: non-temporal, for what passes through once and is larger than the caches.
template <bool NT, class T>
__device__ __forceinline__ T get(const T* p) {
    if constexpr (NT) return __builtin_nontemporal_load(p);
    else return *p;
}
template <bool NT, class T>
__device__ __forceinline__ void put(T* p, T v) {
    if constexpr (NT) __builtin_nontemporal_store(v, p);
    else *p = v;
}
// Eight elements as they lie in memory, n of them (zeros for the others).
template <int DT>
struct Raw8 {
    tu32x4 q[DT == NEOX_F32 ? 2 : 1];
};
template <int DT, bool NT = false>
__device__ __forceinline__ Raw8<DT> raw8(const void* p, uint64_t at, uint32_t n) {
    Raw8<DT> r;
    if (n >= 8) {
        if constexpr (DT == NEOX_F32) {
            r.q[0] = __builtin_bit_cast(tu32x4, get<NT>((const loose_f32x4*)((const float*)p + at)));
            r.q[1] = __builtin_bit_cast(tu32x4, get<NT>((const loose_f32x4*)((const float*)p + at + 4)));
        } else {
            r.q[0] = get<NT>((const loose_u32x4*)((const uint16_t*)p + at));
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if constexpr (DT == NEOX_F32) {
                r.q[e / 4][e % 4] = e < (int)n ? ((const uint32_t*)p)[at + e] : 0u;
            } else {
                const uint32_t h = e < (int)n ? ((const uint16_t*)p)[at + e] : 0u;
                r.q[0][e / 2] = e & 1 ? r.q[0][e / 2] | h << 16 : h;
            }
        }
    }
    return r;
}
template <int DT>
__device__ __forceinline__ float element(const Raw8<DT>& r, int e) {
    if constexpr (DT == NEOX_F32) return __uint_as_float(r.q[e / 4][e % 4]);
    else return half_to_float(DT, (uint16_t)(r.q[0][e / 2] >> (16 * (e & 1))));
}
template <int DT, bool NT = false>
__device__ __forceinline__ void load8(const void* p, uint64_t at, uint32_t n, float (&v)[8]) {
    const Raw8<DT> r = raw8<DT, NT>(p, at, n);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = element(r, e);
}
template <int DT, bool NT = false>
__device__ __forceinline__ void store8(void* p, uint64_t at, uint32_t n, const float (&v)[8]) {
    if (n >= 8) {
        if constexpr (DT == NEOX_F32) {
            put<NT>((loose_f32x4*)((float*)p + at), (loose_f32x4)tf32x4{v[0], v[1], v[2], v[3]});
            put<NT>((loose_f32x4*)((float*)p + at + 4), (loose_f32x4)tf32x4{v[4], v[5], v[6], v[7]});
        } else {
            tu32x4 q;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                q[e] = float_to_half(DT, v[2 * e]) | (uint32_t)float_to_half(DT, v[2 * e + 1]) << 16;
            put<NT>((loose_u32x4*)((uint16_t*)p + at), (loose_u32x4)q);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < (int)n) store_elem(p, DT, at + e, v[e]);
    }
}
__device__ __forceinline__ void drop8(const Drop& d, uint64_t off, uint32_t row, uint32_t unit, float (&v)[8]) {
    const Bits b = philox(d.seed, off, row, unit);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = dropped(d, b.w[e / 2], e & 1, v[e]);
}

// ------------------------------------------------------------------------------------
// results of a product
// ------------------------------------------------------------------------------------
struct Result {
    void* out;
    uint64_t ld;
    uint32_t I, J;             // columns, rows
    int32_t dtype;             // of out
    bool beyond;               // out is larger than the caches
    float scale;               // of the sums; looked at where there is nothing but a residual
    Epilogue e;                // (of nothing: all zero)
};
constexpr uint64_t kBeyond = 1ull << 28;
// 16-bit results are written past the caches, whose room the operands need: 8192 x 24576 x 6144
// 1945 -> 1845 us, with an activation and pre 2116 -> 1935, 2048 x 4096 x 1024 22.2 -> 19.5.  A
// residual is read, and FP32 written, past them only where they could not hold it: 1968 -> 1914
// and 2044 -> 1925 us there, but 20.0 -> 24.3 and 23.6 -> 29.4 at 2048 x 4096 x 1024.
// What follows finds less in the caches: two BF16 layers in a row, 1024 wide with 4096 between them and
// pre stored, past the caches against left there where out is not larger than they: 35.4 us against
// 33.1 with 1024 tokens, 53.4 against 52.7 with 2048, 81.8 against 78.2 with 4096, 24.7 both with 333;
// with their gradients behind them 96.1 against 95.8, 151.5 against 153.5, 245.6 against 244.0, 67.7
// against 66.7; 6144 wide with 24576 between and 2048 tokens 3150 against 3162.  So it goes either way.
// Takes the sums of elements (row, col) to (row, col + 7), col a multiple of 8, to memory; bias and
// residual: what lies there (looked at where there are such).  LAYER: whether there may be anything
// but a residual; if not, the sums are those of a gradient, times r.scale.
template <int DT, int HT, bool LAYER>
__device__ __forceinline__ void emit8(const Result& r, uint64_t off, uint32_t row, uint32_t col, float (&v)[8],
                                      const Raw8<HT>& bias, const Raw8<DT>& residual) {
    const uint32_t n = r.I - col;
    if constexpr (LAYER) {
        if (r.e.bias) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += element(bias, e);
        }
        if (r.e.pre) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = opaque(v[e]);
            store8<HT, true>(r.e.pre, row * r.e.pre_ld + col, n, v);
        }
        with_act(r.e.act, [&](auto act) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = activate<decltype(act)::value>(v[e]);
        });
        if (r.e.drop.limit) drop8(r.e.drop, off, row, col / 8, v);
    }
    if (r.e.residual) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = LAYER ? v[e] + element(residual, e) : __builtin_fmaf(v[e], r.scale, element(residual, e));
    } else if constexpr (!LAYER) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= r.scale;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = opaque(v[e]);
    if (DT == NEOX_F32 && !r.beyond) store8<DT>(r.out, row * r.ld + col, n, v);
    else store8<DT, true>(r.out, row * r.ld + col, n, v);
}
template <int HT>
__device__ __forceinline__ Raw8<HT> bias8(const Result& r, uint32_t col) {
    return r.e.bias ? raw8<HT>(r.e.bias, col, r.I - col) : Raw8<HT>{};
}
template <int DT>
__device__ __forceinline__ Raw8<DT> residual8(const Result& r, uint32_t row, uint32_t col) {
    if (!r.e.residual) return Raw8<DT>{};
    const uint64_t at = row * r.e.residual_ld + col;
    return r.beyond ? raw8<DT, true>(r.e.residual, at, r.I - col) : raw8<DT>(r.e.residual, at, r.I - col);
}
// The same of elements that come one by one; out of type HT or FP32.
template <int HT>
__device__ __forceinline__ void emit8_any(const Result& r, uint64_t off, uint32_t row, uint32_t col, float (&v)[8]) {
    const Raw8<HT> bias = bias8<HT>(r, col);
    if (r.dtype == NEOX_F32) emit8<NEOX_F32, HT, true>(r, off, row, col, v, bias, residual8<NEOX_F32>(r, row, col));
    else emit8<HT, HT, true>(r, off, row, col, v, bias, residual8<HT>(r, row, col));
}

// The results of a wave's part of a block tile, through the wave's own part of LDS in FP32: there
// a lane's four elements of 16 rows become eight neighbouring ones of a row, so that what the
// epilogue reads and writes moves 16 bytes a lane, dropout takes all 128 bits of a call, and the
// epilogue's code is one loop and not one copy for each register.  Rows are padded by 16 bytes
// (they fall on different banks).  at.i, at.j: the block tile's first column and row.
template <class Core>
struct Rows {
    static constexpr int kWaves = Core::NT / 64;
    static constexpr int kU = Core::TP < 4 ? Core::TP : 4, kCols = 16 * kU, kPitch = kCols * 4 + 16;
    static constexpr int kV = Core::TQ >= 2 && 32 * kPitch * kWaves <= Core::kLds ? 2 : 1;
    static constexpr int kRows = 16 * kV, kBytes = kRows * kPitch;
    static_assert(kBytes * kWaves <= Core::kLds, "");
    static_assert(Core::TP % kU == 0 && Core::TQ % kV == 0, "");
};
template <int HT, bool LAYER = true, class Core>
__device__ __forceinline__ void emit_tile(const Result& r, const Core& t, uint32_t i0, uint32_t j0, uint8_t* lds) {
    using R = Rows<Core>;
    const uint32_t lane = threadIdx.x & 63, l16 = lane & 15, g = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    uint8_t* l = lds + wave * R::kBytes;
    const uint32_t wi = __builtin_amdgcn_readfirstlane(i0 + Core::wave_p()), wj = __builtin_amdgcn_readfirstlane(j0 + Core::wave_q());
    const uint64_t off = drop_offset(r.e.drop);
    constexpr uint32_t kLanes = R::kCols / 8, kStep = 64 / kLanes;      // lanes a row, rows a pass
    constexpr int kAcross = Core::TP / R::kU, kPieces = kAcross * (Core::TQ / R::kV);
    auto pass = [&](auto dt) {
        // (a loop over pieces that picks their registers by comparison made the compiler keep the
        // results in scratch memory)
#pragma unroll
        for (int piece = 0; piece < kPieces; ++piece) {
            const uint32_t bi = wi + piece % kAcross * R::kCols, bj = wj + piece / kAcross * R::kRows;
            if (bi >= r.I || bj >= r.J) continue;
#pragma unroll
            for (int u = 0; u < R::kU; ++u)
#pragma unroll
                for (int v = 0; v < R::kV; ++v)
                    *(tf32x4*)(l + (16 * v + l16) * R::kPitch + (16 * u + 4 * g) * 4) =
                        t.acc[piece % kAcross * R::kU + u][piece / kAcross * R::kV + v];
            // A wave's LDS operations execute in order; the compiler must keep them so too.
            asm volatile("" ::: "memory");
            constexpr int DT = decltype(dt)::value;
            const uint32_t c = bi + lane % kLanes * 8;
            uint32_t k = lane / kLanes;
            const uint32_t rows = c < r.I ? min((uint32_t)R::kRows, r.J - bj) : 0u;
            if (k < rows) {
                // the next row's residual is under way while this one is worked on
                const Raw8<HT> bias = LAYER ? bias8<HT>(r, c) : Raw8<HT>{};
                Raw8<DT> residual = residual8<DT>(r, bj + k, c);
#pragma unroll 1
                for (; k < rows; k += kStep) {
                    const tf32x4* s = (const tf32x4*)(l + k * R::kPitch + lane % kLanes * 32);
                    const tf32x4 a = s[0], b = s[1];
                    float x[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
                    const Raw8<DT> now = residual;
                    if (k + kStep < rows) residual = residual8<DT>(r, bj + k + kStep, c);
                    emit8<DT, HT, LAYER>(r, off, bj + k, c, x, bias, now);
                }
            }
            asm volatile("" ::: "memory");
        }
    };
    if (r.dtype == NEOX_F32) pass(std::integral_constant<int, NEOX_F32>{});
    else pass(std::integral_constant<int, HT>{});
}

}  // namespace nz1
