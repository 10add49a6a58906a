// tile_core.h -- the block-tile product both matrix operators use: D = P Q^T for two
// operands stored as rows of consecutive K bytes, on gfx950's matrix cores.
//
// FP16 (v_mfma_f32_16x16x32_f16) and MXFP4 (v_mfma_scale_f32_16x16x128_f8f6f4) take the
// same bytes per lane: 16 bytes of row (lane % 16), lane group (lane / 16) of four covering
// 64 bytes of K.  So everything up to the matrix instruction is one code over bytes: a slab
// of 128 bytes of K (64 FP16 or 256 FP4 elements) per operand row goes from global memory
// straight to LDS (buffer_load ... lds, 16 bytes a lane) and each wave reads
// its rows back as 16-byte fragments.
//
// LDS layout: row r's eight 16-byte chunks sit at chunk position c ^ (r & 7), so that the
// eight rows which eight consecutive lanes read at one chunk fall on different banks.  The
// load writes LDS in lane order, so the swizzle is applied to the global address instead.
// Which K elements meet in which instruction is free as long as both operands agree: the
// lane group g takes chunks 2g and 2g + 1 of a slab, so its two MXFP4 scales are adjacent.
//
// Measured, all tiles whole: FP16 8192 x 8192 x 4096 on 256 x 256 tiles 1.28 to 1.38 PFLOP/s
// (a library product of 8192^3 reaches 1.43, products from registers alone 2.13), on 128 x 128
// ones 1.1; MXFP4 8192 x 8192 x 16384 4.2 to 4.4 and 3.5.  The matrix units are busy 64% of the
// time in FP16; LDS, from which each wave reads 8 + 4 fragments for 32 products and into which
// the loads write, is busy nearly as long, and the two do not overlap in full.
#pragma once

#include "neox_matrix.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nz1 {

typedef float tf32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 tf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t tu32x4 __attribute__((ext_vector_type(4)));
typedef int32_t ti32x8 __attribute__((ext_vector_type(8)));

constexpr uint32_t kSlab = 128;       // bytes of K per row and stage

// One operand of a block: `rows` rows of `pitch` bytes from base.  Rows past the last one read
// as zeros (the loads carry the operand's length, and the hardware returns 0 behind it).
struct TileRows {
    const uint8_t* base;
    const uint8_t* scales;            // MXFP4: row r's at r * spitch
    uint32_t rows, pitch, spitch;
};

typedef __amdgpu_buffer_rsrc_t rsrc_t;
// A raw buffer of n bytes: what lies at or behind n reads 0.  Flags: the 32-bit data format word
// of gfx9's untyped buffers.  The loads below rely on two things that the hardware's range check
// does with a lane's offset v and the scalar offset s (measured on gfx950 for loads of 4 and 16
// bytes to LDS): it is made on v + s, not on v alone, and it holds where s by itself lies behind n
// (n = 64, v = 0, s = 2^20 reads 0, n = 2^23 with s = 3 * 2^29 too) and where v = 2^31 (s up to 3 *
// 2^29 + 2^23, n up to 2^31).  Edge tiles of MXFP4 operands need that: whole rows are in s, also
// rows that the operand does not have; of 256 rows of 2^23 bytes, the longest ones, s reaches 3 *
// 2^29 + 2^23 + 384.
__device__ __forceinline__ rsrc_t raw_buffer(const void* p, uint32_t n) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, n, 0x00027000);
}
constexpr uint32_t kNowhere = 0x80000000u;      // an offset behind every operand (at most 2^31 bytes);
                                                // with the largest s it stays below 2^32

// BP x BQ output tile by WP x WQ waves, FP16 or MXFP4, NS slabs of K in LDS.
//
// A slab is worked on in two halves (64 bytes of K each).  While the products of one half run,
// the fragments of the next are read: after the products of tile row i, its P fragment is
// overwritten by the next half's, and the Q fragments alternate between two sets.  The reads of
// slab s + 1 need it to have landed, so the block's one barrier per slab sits in the second
// half of slab s, behind the first row of products (which covers the latency of slab s's last
// reads; behind the second or third row it measured 2-3% slower).  Behind it slab s's buffer is
// free, and the load of slab s + NS goes there.  Row by row the order is pinned: left to itself
// the compiler reads all fragments at once and spills.  256 x 256 tiles take 8 waves of 236 to
// 256 registers; 4 waves of twice the part would keep results in the accumulation registers
// and copy them at each product (10 times slower).  Tried as well, of no use: slabs of 64 bytes
// in four stages (equal, 128 x 128 tiles 20% slower), more stages, the Q fragments a row
// earlier, waves 4 x 2, a higher wave priority in the products.
template <int BP_, int BQ_, int WP_, int WQ_, bool FP4_, int NS_ = 2>
struct TileCore {
    static constexpr int BP = BP_, BQ = BQ_, WP = WP_, WQ = WQ_, NS = NS_;
    static constexpr bool FP4 = FP4_;
    static constexpr int NT = WP * WQ * 64;
    static constexpr int TP = BP / WP / 16, TQ = BQ / WQ / 16;      // 16x16 tiles per wave
    static constexpr int LP = BP * 8 / NT, LQ = BQ * 8 / NT;        // 16-byte loads per thread and slab
    static constexpr int kStage = (BP + BQ) * kSlab;
    // MXFP4: the scales of four slabs, 32 bytes a row, double buffered
    static constexpr int kGroup = (BP + BQ) * 32;
    static constexpr int SP = BP * 8 / NT, SQ = BQ * 8 / NT;        // 4-byte loads per thread and group
    static constexpr int kLds = NS * kStage + (FP4 ? 2 * kGroup : 0);
    static_assert(LP >= 1 && LQ >= 1 && BP * 8 % NT == 0 && BQ * 8 % NT == 0, "whole loads");
    static_assert(NS >= 2 && (!FP4 || NS == 2), "");
    static_assert(kLds <= 160 * 1024, "LDS of a CU");

    // acc[i][j]: 16x16 tile (i, j) of this wave; element e of a lane is D row
    // 16 i + 4 (lane / 16) + e, column 16 j + lane % 16 of the wave's part.
    tf32x4 acc[TP][TQ];

    static __device__ __forceinline__ int wave_p() { return (int)(threadIdx.x >> 6) / WQ * (BP / WP); }
    static __device__ __forceinline__ int wave_q() { return (int)(threadIdx.x >> 6) % WQ * (BQ / WQ); }

    static __device__ __forceinline__ tu32x4 frag(const uint8_t* rows, int row, int chunk) {
        return *(const tu32x4*)(rows + row * kSlab + ((chunk ^ (row & 7)) << 4));
    }
    // Waits until at most n of this wave's loads are under way and its LDS reads are done,
    // then for everybody.  (A fence would wait for all loads.)
    template <int n>
    static __device__ __forceinline__ void wait_barrier() {
        static_assert(n < 64, "vmcnt has six bits");
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt((n & 15) | (n >> 4) << 14 | 0x0070);   // vmcnt(n) lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    }

    // lds: kLds bytes.  kbytes: bytes of K, a multiple of 128 (FP16) or 64 (MXFP4).
    __device__ __forceinline__ void run(const TileRows& p, const TileRows& q, uint32_t kbytes,
                                        uint8_t* lds) {
        const uint32_t tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, g = lane >> 4;
        const uint32_t slabs = (kbytes + kSlab - 1) / kSlab;
        const rsrc_t pb = raw_buffer(p.base, p.rows * p.pitch), qb = raw_buffer(q.base, q.rows * q.pitch);
        // this thread's chunk of its first row; the others are NT / 8 rows further each
        const uint32_t chunk = (tid & 7) ^ ((tid >> 3) & 7);
        const uint32_t pv = (tid >> 3) * p.pitch + chunk * 16, qv = (tid >> 3) * q.pitch + chunk * 16;
        const uint32_t pstep = NT / 8 * p.pitch, qstep = NT / 8 * q.pitch;
        // MXFP4: the last slab may be half a slab; its second half is read as zeros
        const bool half_tail = FP4 && (kbytes & 64u);
        const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        const int rp = wave_p() + (int)l16, rq = wave_q() + (int)l16;
        uint8_t* sl = lds + NS * kStage;

        typedef __attribute__((address_space(3))) void* lptr;
        // Load n (of LP + LQ) of slab s.  Slabs behind the last one are loaded from nowhere: the
        // loop has no branches, and the number of loads under way at each wait is known.
        auto stage = [&](int n, uint32_t s, uint8_t* buf) {
            const bool live = s < slabs - (half_tail && chunk >= 4 ? 1 : 0);
            if (n < LP)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(pb, (lptr)(buf + wave * 1024 + n * NT * 16), 16,
                                                         live ? pv : kNowhere, s * kSlab + n * pstep, 0, 0);
            else
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    qb, (lptr)(buf + BP * kSlab + wave * 1024 + (n - LP) * NT * 16), 16, live ? qv : kNowhere,
                    s * kSlab + (n - LP) * qstep, 0, 0);
        };
        // Quarter k of the scales of slabs 4u .. 4u + 3: a group is loaded over the four slabs
        // before it, so that these loads need no branch either.
        rsrc_t psb = pb, qsb = qb;
        uint32_t psv = 0, qsv = 0;
        // dword of a row's 32 bytes; rows 8 to 15 of 16 swap halves, to use the banks rows 0 to 7
        // leave
        const uint32_t sdw = (tid & 7) ^ (tid >> 4 & 4);
        if constexpr (FP4) {
            psb = raw_buffer(p.scales, p.rows * p.spitch);
            qsb = raw_buffer(q.scales, q.rows * q.spitch);
            psv = (tid >> 3) * p.spitch + sdw * 4;
            qsv = (tid >> 3) * q.spitch + sdw * 4;
        }
        auto group = [&](uint32_t u, uint32_t k) {
            if constexpr (FP4) {
                static_assert(SP == SQ && SP % 2 == 0, "whole quarters");
                const bool in = u * 32 + sdw * 4 < p.spitch;
                const uint32_t v = in ? (k < 2 ? psv : qsv) : kNowhere;
                const uint32_t step = NT / 8 * p.spitch;             // both operands have one K
                uint8_t* w = sl + (u & 1) * kGroup + wave * 256;
#pragma unroll
                for (int i = 0; i < SP / 2; ++i)
                    __builtin_amdgcn_raw_ptr_buffer_load_lds(k < 2 ? psb : qsb,
                                                             (lptr)(w + (k * (SP / 2) + i) * NT * 4), 4, v,
                                                             u * 32 + ((k & 1) * (SP / 2) + i) * step, 0, 0);
            }
        };
        tu32x4 fp[TP], fq[2][TQ];
        uint32_t sp[TP], sq[2][TQ];                  // MXFP4: two scale bytes each
        auto row = [&](int i, int h, int set) {
#pragma unroll
            for (int j = 0; j < TQ; ++j) {
                if constexpr (FP4) {
                    const ti32x8 x = {(int)fp[i].x, (int)fp[i].y, (int)fp[i].z, (int)fp[i].w, 0, 0, 0, 0};
                    const tu32x4 f = fq[h][j];
                    const ti32x8 y = {(int)f.x, (int)f.y, (int)f.z, (int)f.w, 0, 0, 0, 0};
                    acc[i][j] = h == 0
                        ? __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, acc[i][j], 4, 4, 0, (int)sp[i],
                                                                           0, (int)sq[set][j])
                        : __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, acc[i][j], 4, 4, 1, (int)sp[i],
                                                                           1, (int)sq[set][j]);
                } else {
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(tf16x8, fp[i]),
                                                                       __builtin_bit_cast(tf16x8, fq[h][j]),
                                                                       acc[i][j], 0, 0, 0);
                }
            }
        };
        auto read_p = [&](int i, const uint8_t* c, int h) { fp[i] = frag(c, rp + 16 * i, 2 * (int)g + h); };
        auto read_q = [&](int j, const uint8_t* c, int h) {
            fq[h][j] = frag(c + BP * kSlab, rq + 16 * j, 2 * (int)g + h);
        };
        const uint32_t sswap = (l16 & 8) << 1;
        auto scale_p = [&](int i, uint32_t s) {
            if constexpr (FP4)
                sp[i] = *(const uint16_t*)(sl + ((s >> 2) & 1) * kGroup + (rp + 16 * i) * 32 + (((s & 3) * 8 + 2 * g) ^ sswap));
        };
        auto scale_q = [&](int j, uint32_t s, int set) {
            if constexpr (FP4)
                sq[set][j] = *(const uint16_t*)(sl + ((s >> 2) & 1) * kGroup + (BP + rq + 16 * j) * 32 +
                                                (((s & 3) * 8 + 2 * g) ^ sswap));
        };
#pragma unroll
        for (int i = 0; i < TP; ++i)
#pragma unroll
            for (int j = 0; j < TQ; ++j) acc[i][j] = tf32x4{0, 0, 0, 0};
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k) group(0, k);
        group(1, 0);
#pragma unroll
        for (int k = 0; k < NS; ++k) {
#pragma unroll
            for (int n = 0; n < LP + LQ; ++n) stage(n, k, lds + k * kStage);
        }
        wait_barrier<(NS - 1) * (LP + LQ)>();
#pragma unroll
        for (int i = 0; i < TP; ++i) {
            read_p(i, lds, 0);
            scale_p(i, 0);
        }
#pragma unroll
        for (int j = 0; j < TQ; ++j) {
            read_q(j, lds, 0);
            scale_q(j, 0, 0);
        }
        uint32_t at = 0;                             // buffer of slab s
        for (uint32_t s = 0; s < slabs; ++s) {
            uint8_t* cur = lds + at * kStage;
            at = at + 1 == NS ? 0 : at + 1;
            const uint8_t* nxt = lds + at * kStage;
            // first half: products of (s, 0), reads of (s, 1)
#pragma unroll
            for (int i = 0; i < TP; ++i) {
                row(i, 0, 0);
                read_p(i, cur, 1);
#pragma unroll
                for (int j = i * TQ / TP; j < (i + 1) * TQ / TP; ++j) read_q(j, cur, 1);
                __builtin_amdgcn_sched_barrier(0);
            }
            // second half: products of (s, 1), reads of (s + 1, 0); behind the last slab these
            // read a buffer that holds an older one, or nothing, and are not used
#pragma unroll
            for (int i = 0; i < TP; ++i) {
                row(i, 1, 0);
                if (i == 0) wait_barrier<(NS - 2) * (LP + LQ)>();
                // the loads of slab s + NS, spread over the rows: issued at once they queue up and
                // hold back the products behind them (6% slower)
#pragma unroll
                for (int t = i * (LP + LQ) / TP; t < (i + 1) * (LP + LQ) / TP; ++t) stage(t, s + NS, cur);
                if (i == TP - 1) group(((s + 1) >> 2) + 1, (s + 1) & 3);
                read_p(i, nxt, 0);
                scale_p(i, s + 1);
#pragma unroll
                for (int j = i * TQ / TP; j < (i + 1) * TQ / TP; ++j) {
                    read_q(j, nxt, 0);
                    scale_q(j, s + 1, 1);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            if constexpr (FP4) {
#pragma unroll
                for (int j = 0; j < TQ; ++j) sq[0][j] = sq[1][j];
            }
        }
        wait_barrier<0>();       // nothing writes to or reads from lds any more
    }
};

// ------------------------------------------------------------------------------------
// which tile a block works on
// ------------------------------------------------------------------------------------
// Blocks [0, nfull) take whole tiles of unit x unit (256 or 128); the others take quarters of
// what is left: the tiles that would start another, mostly empty round on the chip's 256 CUs,
// and those that the matrix's edge cuts.  Tiles of a symmetric product lie on and below the
// diagonal, those on it last (a quarter of them above it is left out).  Neighbouring tiles on
// one XCD: an X <- P X of 6144 x 6144 on 128 x 128 tiles took 602 us in plain order, 486 so.
struct TileMap {
    uint32_t nfull;        // blocks with whole tiles
    uint32_t inner;        // whole tiles per matrix
    uint32_t edges;        // cut tiles per matrix
    uint32_t count;        // matrices
    uint32_t pi, qi;       // whole tiles down and across
    uint32_t q;            // tiles across, a cut one counted
    uint32_t mp, np;       // sides
    uint32_t unit;
};

// (i, j), j <= i, number t in row order of a lower triangle
__device__ __forceinline__ void lower(uint32_t t, uint32_t& ti, uint32_t& tj) {
    uint32_t i = (uint32_t)((__builtin_sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
    while (i * (i + 1) / 2 > t) --i;
    while ((i + 1) * (i + 2) / 2 <= t) ++i;
    ti = i;
    tj = t - i * (i + 1) / 2;
}

struct TileAt {
    uint32_t z, i, j;      // matrix, first row and column
    bool full, none;
    // Into scalar registers: the same for the whole block, but computed with vector
    // instructions (a square root); operands addressed through vector registers would turn
    // every buffer load into a loop over the lanes.
    __device__ __forceinline__ void settle() {
        z = __builtin_amdgcn_readfirstlane(z);
        i = __builtin_amdgcn_readfirstlane(i);
        j = __builtin_amdgcn_readfirstlane(j);
    }
};

template <bool SYM>
__device__ __forceinline__ TileAt place(const TileMap& m) {
    TileAt r{};
    uint32_t k, quarter = 0;
    r.full = blockIdx.x < m.nfull;
    if (r.full) {
        // consecutive blocks go to the eight XCDs in turn: give each XCD, and so each L2, one
        // run of neighbouring tiles
        const uint32_t per = m.nfull / 8;
        k = m.nfull % 8 ? blockIdx.x : blockIdx.x % 8 * per + blockIdx.x / 8;
    } else {
        k = m.nfull + (blockIdx.x - m.nfull) / 4;
        quarter = (blockIdx.x - m.nfull) % 4;
    }
    const uint32_t total = m.inner * m.count;
    uint32_t ti, tj;
    if (k < total) {
        r.z = k / m.inner;
        k -= r.z * m.inner;
        if (SYM) {
            const uint32_t below = m.pi * (m.pi - 1) / 2;
            if (k < below) {
                lower(k, ti, tj);
                ++ti;
            } else {
                ti = tj = k - below;
            }
        } else {
            // runs of eight tile rows, column by column: 64 tiles in a row share 8 + 8 panels
            const uint32_t g = k / (8 * m.qi), rows = min(8u, m.pi - 8 * g), in = k - g * 8 * m.qi;
            ti = 8 * g + in % rows;
            tj = in / rows;
        }
    } else {
        k -= total;
        r.z = k / m.edges;
        k -= r.z * m.edges;
        if (SYM) {
            ti = m.pi;
            tj = k;
        } else {
            const uint32_t right = m.q > m.qi ? m.pi : 0;
            ti = k < right ? k : m.pi;
            tj = k < right ? m.qi : k - right;
        }
    }
    r.i = ti * m.unit + (quarter >> 1) * (m.unit / 2);
    r.j = tj * m.unit + (quarter & 1) * (m.unit / 2);
    r.settle();
    r.none = r.i >= m.mp || r.j >= m.np || (SYM && !r.full && r.j > r.i);
    return r;
}

// The launch of one product with `count` p x q results (p = q and sym for symmetric ones; a
// cut tile reads zeros behind its operands' rows), and its cost per slab of K: `full` for a
// round of whole tiles over the chip's CUs, `quarter` for a round of quarters.  Quarters that
// the edge or the diagonal leaves empty are counted: they fall on the XCDs unevenly, and a cost
// without them chose launches that took 15 to 24% longer (7 of 4096 x 1024, 6 of 1920 x 1920).
constexpr uint32_t kCUs = 256;
inline TileMap plan_tiles(uint32_t unit, bool sym, uint32_t p, uint32_t q, uint32_t count, double full, double quarter,
                          double* cost, uint64_t* blocks) {
    TileMap m{};
    m.count = count;
    m.unit = unit;
    m.pi = p / unit;
    m.qi = q / unit;
    m.q = (q + unit - 1) / unit;
    m.mp = p;
    m.np = q;
    const bool cut_p = p % unit != 0, cut_q = q % unit != 0;
    if (sym) {
        m.inner = m.pi * (m.pi + 1) / 2;
        m.edges = cut_p ? m.pi + 1 : 0;
    } else {
        m.inner = m.pi * m.qi;
        m.edges = (cut_q ? m.pi : 0) + (cut_p ? m.q : 0);
    }
    const uint64_t total = (uint64_t)m.inner * count, cut = (uint64_t)m.edges * count;
    auto takes = [&](uint64_t n) {
        const uint64_t quarters = 4 * (total - n + cut);
        return full * (double)((n + kCUs - 1) / kCUs) + quarter * (double)((quarters + kCUs - 1) / kCUs);
    };
    const uint64_t whole = total / kCUs * kCUs;
    const uint64_t n = takes(total) <= takes(whole) ? total : whole;
    m.nfull = (uint32_t)n;
    *cost = takes(n);
    *blocks = n + 4 * (total - n + cut);
    return m;
}

// ------------------------------------------------------------------------------------
// results on their way to memory
// ------------------------------------------------------------------------------------
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));

// ROWS x COLS FP16 elements of a row-major array in a wave's own part of LDS, on their way
// between its result tiles and memory: a lane's four elements are 8 bytes of 16 different rows
// an instruction, which memory serves at half the rate of whole rows, so rows of COLS elements
// (32 to 128 bytes) are moved 16 bytes a lane instead.  The 16-byte chunks of a row are
// permuted by its number so that 16 rows at one column fall on different banks.  Only the wave
// that owns the part uses it, and its LDS operations execute in order: no barrier is needed.
template <int ROWS, int COLS>
struct Patch {
    static constexpr int kRow = COLS * 2, kChunks = kRow / 16, kBytes = ROWS * kRow;
    static constexpr int kPass = (kBytes + 1023) / 1024; // 64 lanes of 16 bytes, or 32 of one pass
    static_assert(kRow >= 32 && kRow <= 128 && (kBytes % 1024 == 0 || kBytes == 512), "");
    static __device__ __forceinline__ uint32_t turn(uint32_t row) { return row * kRow / 256 & (kChunks - 1); }
    // four elements at (row, col), col a multiple of 4
    static __device__ __forceinline__ f16x4* at(uint8_t* l, uint32_t row, uint32_t col) {
        return (f16x4*)(l + row * kRow + (((col >> 3) ^ turn(row)) << 4) + (col & 4) * 2);
    }
    // A pass moves kBytes / kPass bytes: rows k * kStep + lane / kChunks.  The lane's part of an
    // address stays apart from the pass's, which is the same for all lanes (Ld: 32 bits where
    // kStep rows are less than 4 GB).
    static constexpr int kStep = 64 / kChunks;
    template <class Ld>
    static __device__ __forceinline__ Ld lane_part(int k, Ld ld) {
        const uint32_t lane = threadIdx.x & 63;
        const uint32_t row = lane / kChunks, c = (lane % kChunks) ^ turn(k * kStep + row);
        return row * ld + c * 8;
    }
    // starts loading from g (row r at r * ld); wave_wait() before it is used
    static __device__ __forceinline__ void load(uint8_t* l, const uint16_t* g, uint32_t ld) {
        if (kBytes < 1024 && (threadIdx.x & 63) * 16 >= kBytes) return;
#pragma unroll
        for (int k = 0; k < kPass; ++k)
            __builtin_amdgcn_global_load_lds(
                (const __attribute__((address_space(1))) void*)(g + (uint64_t)(k * kStep) * ld + lane_part<uint32_t>(k, ld)),
                (__attribute__((address_space(3))) void*)(l + k * 1024), 16, 0, 0);
    }
    // rows [0, left) to g
    template <class Ld>
    static __device__ __forceinline__ void store(const uint8_t* l, uint16_t* g, Ld ld, uint32_t left = ROWS) {
        const uint32_t lane = threadIdx.x & 63;
#pragma unroll
        for (int k = 0; k < kPass; ++k)
            if (k * kStep + lane / kChunks < left)
                *(tu32x4*)(g + (uint64_t)(k * kStep) * ld + lane_part<Ld>(k, ld)) =
                    *(const tu32x4*)(l + (k * 64 + lane) * 16);
    }
};
// All of this wave's memory operations so far are done.
__device__ __forceinline__ void wave_wait() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070);         // vmcnt(0) lgkmcnt(0)
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// A wave's results of a block tile, worked on in pieces of 16 kU x 16 TQ elements.
template <class Core>
struct Piece {
    static constexpr int kU = Core::TP < 4 ? Core::TP : 4, kV = Core::TQ;
    using Down = Patch<16 * kV, 16 * kU>;       // rows are D's columns: an array [j][i]
    using Across = Patch<16 * kU, 16 * kV>;     // rows are D's rows: [i][j]
    static constexpr int kBytes = Down::kBytes, kWaves = Core::NT / 64;
    // Small tiles' patches have LDS of their own behind the tile's, so that they can be loaded
    // before the products instead of after them.
    static constexpr bool kEarly = Core::BP <= 64 && !Core::FP4;
    static constexpr int kPart = kEarly ? 2 * kBytes : Core::kLds / kWaves;
    static_assert(kEarly || 2 * kBytes <= kPart, "two patches per wave");
    uint32_t i, j;         // first row and column in the matrix
    uint32_t li, lj;       // this lane's first row and its column within 16 x 16
    uint8_t *l0, *l1;      // LDS of two patches
    __device__ Piece(const TileAt& t, int u0, uint8_t* lds) {
        const uint32_t lane = threadIdx.x & 63;
        i = __builtin_amdgcn_readfirstlane(t.i + Core::wave_p() + 16 * u0);
        j = __builtin_amdgcn_readfirstlane(t.j + Core::wave_q());
        li = (lane >> 4) * 4;
        lj = lane & 15;
        // (scalar, so that the patches' places and what follows from them are)
        const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        l0 = lds + (kEarly ? Core::kLds : 0) + wave * kPart;
        l1 = l0 + kBytes;
    }
    // The places of tile (u, v)'s elements of this lane, and of their transposes, in a patch.
    __device__ __forceinline__ f16x4* down(uint8_t* l, int u, int v) const { return Down::at(l, 16 * v + lj, 16 * u + li); }
    __device__ __forceinline__ f16x4* across(uint8_t* l, int u, int v) const { return Across::at(l, 16 * u + lj, 16 * v + li); }
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

// LDS of a block that works on Core's tiles.
template <class Core>
constexpr int room() {
    return Core::kLds + (Piece<Core>::kEarly ? Piece<Core>::kWaves * Piece<Core>::kPart : 0);
}

}  // namespace nz1
