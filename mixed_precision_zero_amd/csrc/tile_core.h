// tile_core.h -- the block-tile product both matrix operators use: D = P Q^T for two
// operands stored as rows of consecutive K bytes, on gfx950's matrix cores.
//
// FP16 (v_mfma_f32_16x16x32_f16) and MXFP4 (v_mfma_scale_f32_16x16x128_f8f6f4) take the
// same bytes per lane: 16 bytes of row (lane % 16), lane group (lane / 16) of four covering
// 64 bytes of K.  So everything up to the matrix instruction is one code over bytes: a slab
// of 128 bytes of K (64 FP16 or 256 FP4 elements) per operand row goes from global memory
// straight to LDS (global_load_lds, 16 bytes a lane), double buffered, and each wave reads
// its rows back as 16-byte fragments.
//
// LDS layout: row r's eight 16-byte chunks sit at chunk position c ^ (r & 7), so that the
// eight rows which eight consecutive lanes read at one chunk fall on different banks.  The
// load writes LDS in lane order, so the swizzle is applied to the global address instead.
// Which K elements meet in which instruction is free as long as both operands agree: the
// lane group g takes chunks 2g and 2g + 1 of a slab, so its two MXFP4 scales are adjacent.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nz1 {

typedef float tf32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 tf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t tu32x4 __attribute__((ext_vector_type(4)));
typedef int32_t ti32x8 __attribute__((ext_vector_type(8)));

constexpr uint32_t kSlab = 128;       // bytes of K per row and stage

// One operand of a block: `rows` valid rows from base, row r at r * pitch bytes.  Rows past
// the last valid one read that one again (their results are not stored).
struct TileRows {
    const uint8_t* base;
    const uint8_t* scales;            // MXFP4: row r's at r * spitch
    uint32_t rows, pitch, spitch;
};

static __device__ __attribute__((aligned(16))) const uint32_t g_zero_chunk[4] = {0, 0, 0, 0};

__device__ __forceinline__ void load_lds16(const void* g, void* l) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)g,
                                     (__attribute__((address_space(3))) void*)l, 16, 0, 0);
}

template <int BP_, int BQ_, int WP_, int WQ_, bool FP4_>
struct TileCore {
    static constexpr int BP = BP_, BQ = BQ_, WP = WP_, WQ = WQ_;
    static constexpr bool FP4 = FP4_;
    static constexpr int NT = WP * WQ * 64;
    static constexpr int TP = BP / WP / 16, TQ = BQ / WQ / 16;      // 16x16 tiles per wave
    static constexpr int LP = BP * 8 / NT, LQ = BQ * 8 / NT;        // 16-byte loads per thread
    static constexpr int kStage = (BP + BQ) * kSlab;
    static_assert(LP >= 1 && LQ >= 1 && BP * 8 % NT == 0 && BQ * 8 % NT == 0, "whole loads");

    // acc[i][j]: 16x16 tile (i, j) of this wave; element e of a lane is D row
    // 16 i + 4 (lane / 16) + e, column 16 j + lane % 16 of the wave's part.
    tf32x4 acc[TP][TQ];

    static __device__ __forceinline__ int wave_p() { return (int)(threadIdx.x >> 6) / WQ * (BP / WP); }
    static __device__ __forceinline__ int wave_q() { return (int)(threadIdx.x >> 6) % WQ * (BQ / WQ); }

    template <int L>
    static __device__ __forceinline__ void offsets(const TileRows& t, uint32_t (&off)[L]) {
        const uint32_t tid = threadIdx.x;
        const uint32_t c = (tid & 7) ^ ((tid >> 3) & 7);
#pragma unroll
        for (int i = 0; i < L; ++i) {
            uint32_t r = (tid >> 3) + i * (NT / 8);
            r = r < t.rows ? r : t.rows - 1;
            off[i] = r * t.pitch + c * 16;
        }
    }
    template <int L>
    static __device__ __forceinline__ void issue(const uint8_t* base, const uint32_t (&off)[L],
                                                 uint8_t* lds, bool dead) {
        uint8_t* w = lds + (threadIdx.x & ~63u) * 16;               // wave-uniform
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const uint8_t* g = base + off[i];
            if (dead) g = (const uint8_t*)g_zero_chunk;
            load_lds16(g, w + i * NT * 16);
        }
    }
    static __device__ __forceinline__ tu32x4 frag(const uint8_t* rows, int row, int chunk) {
        return *(const tu32x4*)(rows + row * kSlab + ((chunk ^ (row & 7)) << 4));
    }

    // lds: 2 * kStage bytes.  kbytes: bytes of K, a multiple of 128 (FP16) or 64 (MXFP4).
    __device__ __forceinline__ void run(const TileRows& p, const TileRows& q, uint32_t kbytes,
                                        uint8_t* lds) {
        const uint32_t lane = threadIdx.x & 63, l16 = lane & 15, g = lane >> 4;
        uint32_t po[LP], qo[LQ];
        offsets(p, po);
        offsets(q, qo);
        const uint32_t slabs = (kbytes + kSlab - 1) / kSlab;
        // MXFP4: the last slab may be half a slab; its second half is read as zeros
        const bool upper = ((threadIdx.x & 7) ^ ((threadIdx.x >> 3) & 7)) >= 4;
        const bool half_tail = FP4 && (kbytes & 64u);
        const int rp = wave_p() + (int)l16, rq = wave_q() + (int)l16;
        uint32_t sp[TP], sq[TQ], spn[TP], sqn[TQ];
        auto scales = [&](uint32_t s) {
            if constexpr (FP4) {
                const uint32_t at = s * 8 + 2 * g;
                const bool in = at < p.spitch;
#pragma unroll
                for (int i = 0; i < TP; ++i) {
                    uint32_t r = (uint32_t)(rp + 16 * i);
                    r = r < p.rows ? r : p.rows - 1;
                    spn[i] = in ? *(const uint16_t*)(p.scales + (size_t)r * p.spitch + at) : 0x7F7Fu;
                }
#pragma unroll
                for (int j = 0; j < TQ; ++j) {
                    uint32_t r = (uint32_t)(rq + 16 * j);
                    r = r < q.rows ? r : q.rows - 1;
                    sqn[j] = in ? *(const uint16_t*)(q.scales + (size_t)r * q.spitch + at) : 0x7F7Fu;
                }
            }
        };
        auto stage = [&](uint32_t s, uint8_t* buf) {
            const bool dead = half_tail && s == slabs - 1 && upper;
            issue<LP>(p.base + (size_t)s * kSlab, po, buf, dead);
            issue<LQ>(q.base + (size_t)s * kSlab, qo, buf + BP * kSlab, dead);
            scales(s);
        };
#pragma unroll
        for (int i = 0; i < TP; ++i)
#pragma unroll
            for (int j = 0; j < TQ; ++j) acc[i][j] = tf32x4{0, 0, 0, 0};
        stage(0, lds);
        for (uint32_t s = 0; s < slabs; ++s) {
            const uint8_t* cur = lds + (s & 1) * kStage;
            if constexpr (FP4) {
#pragma unroll
                for (int i = 0; i < TP; ++i) sp[i] = spn[i];
#pragma unroll
                for (int j = 0; j < TQ; ++j) sq[j] = sqn[j];
            }
            // this thread's loads have landed; after the barrier everybody's have, and
            // everybody is done reading the other buffer
            __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0)
            __syncthreads();
            if (s + 1 < slabs) stage(s + 1, lds + ((s + 1) & 1) * kStage);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                tu32x4 fp[TP], fq[TQ];
#pragma unroll
                for (int i = 0; i < TP; ++i) fp[i] = frag(cur, rp + 16 * i, 2 * (int)g + h);
#pragma unroll
                for (int j = 0; j < TQ; ++j) fq[j] = frag(cur + BP * kSlab, rq + 16 * j, 2 * (int)g + h);
#pragma unroll
                for (int i = 0; i < TP; ++i)
#pragma unroll
                    for (int j = 0; j < TQ; ++j) {
                        if constexpr (FP4) {
                            const ti32x8 x = {(int)fp[i].x, (int)fp[i].y, (int)fp[i].z, (int)fp[i].w, 0, 0, 0, 0};
                            const ti32x8 y = {(int)fq[j].x, (int)fq[j].y, (int)fq[j].z, (int)fq[j].w, 0, 0, 0, 0};
                            acc[i][j] = h == 0
                                ? __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                                      x, y, acc[i][j], 4, 4, 0, (int)sp[i], 0, (int)sq[j])
                                : __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                                      x, y, acc[i][j], 4, 4, 1, (int)sp[i], 1, (int)sq[j]);
                        } else {
                            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                                __builtin_bit_cast(tf16x8, fp[i]), __builtin_bit_cast(tf16x8, fq[j]),
                                acc[i][j], 0, 0, 0);
                        }
                    }
            }
        }
    }
};

// ------------------------------------------------------------------------------------
// element types
// ------------------------------------------------------------------------------------
__device__ __forceinline__ float opaque(float x) {
    // an FP32 value that is stored and also rounded to a half must be rounded to FP32
    // first: without this the multiply-add before it may be rounded to the half directly
    asm("" : "+v"(x));
    return x;
}
__device__ __forceinline__ float half_to_float(int dtype, uint16_t v) {
    return dtype == NEOX_F16 ? (float)__builtin_bit_cast(_Float16, v)
                             : __uint_as_float((uint32_t)v << 16);
}
__device__ __forceinline__ uint16_t float_to_half(int dtype, float x) {
    return dtype == NEOX_F16 ? __builtin_bit_cast(uint16_t, (_Float16)x)
                             : __builtin_bit_cast(uint16_t, (__bf16)x);
}
__device__ __forceinline__ float load_elem(const void* p, int dtype, uint64_t i) {
    return dtype == NEOX_F32 ? ((const float*)p)[i] : half_to_float(dtype, ((const uint16_t*)p)[i]);
}
__device__ __forceinline__ void store_elem(void* p, int dtype, uint64_t i, float x) {
    if (dtype == NEOX_F32) ((float*)p)[i] = x;
    else ((uint16_t*)p)[i] = float_to_half(dtype, x);
}

}  // namespace nz1
