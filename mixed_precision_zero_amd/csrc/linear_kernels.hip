// linear_kernels.hip -- products of half-precision matrices with an epilogue on gfx950.
#include "epilogue.h"
#include "spread.h"

#include <algorithm>

namespace nz1 {

namespace {

// ------------------------------------------------------------------------------------
// block tiles
// ------------------------------------------------------------------------------------
// p and q as tiles take them: rows of 16-byte aligned pitch.  Launches of more than one share
// split K: share z takes `slabs` slabs of 64 elements from z * slabs on, and writes its sums to
// r.out + z J ld in FP32, for join_kernel.
struct TileArgs {
    const uint8_t *p, *q;
    uint32_t p_pitch, q_pitch;
    uint64_t K, slabs;
    uint32_t shares;
    Result r;
};

template <bool STRIDED>
__device__ __forceinline__ TileRows rows_of(const uint8_t* base, uint32_t pitch, uint32_t first, uint32_t side, uint64_t k0,
                                            uint32_t left) {
    // (a strided operand has as many rows as K has elements left)
    if constexpr (STRIDED) return TileRows{base + k0 * pitch + (uint64_t)first * 2, nullptr, side, pitch, left};
    else return TileRows{base + (uint64_t)first * pitch + k0 * 2, nullptr, side, pitch, 0};
}

template <class Core, int HT>
__device__ __forceinline__ void linear_tile(const TileArgs& a, const TileAt& at, uint32_t share, uint8_t* lds) {
    const uint64_t k0 = share * a.slabs * 64;
    const uint32_t left = (uint32_t)min(a.K - k0, a.slabs * 64);
    const TileRows p = rows_of<Core::Form::kStridedP>(a.p, a.p_pitch, at.i, min((uint32_t)Core::BP, a.r.I - at.i), k0, left);
    const TileRows q = rows_of<Core::Form::kStridedQ>(a.q, a.q_pitch, at.j, min((uint32_t)Core::BQ, a.r.J - at.j), k0, left);
    Core t;
    // rows of K are zeros up to a multiple of 8
    t.run(p, q, (left + 7) / 8 * 16, lds);
    if (a.shares > 1) {
        Result r = a.r;
        r.out = (float*)a.r.out + share * (uint64_t)a.r.J * a.r.ld;
        emit_tile<HT>(r, t, at.i, at.j, lds);
    } else {
        emit_tile<HT>(a.r, t, at.i, at.j, lds);
    }
}

template <class Form>
using Lin256 = TileCore<256, 256, 2, 4, false, 2, Form>;
template <class Form>
using Lin128 = TileCore<128, 128, 2, 4, false, 2, Form>;
template <class Form>
using Lin64 = TileCore<64, 64, 2, 2, false, 4, Form>;
template <class Form>
using Lin128d = TileCore<128, 128, 2, 4, false, 4, Form>;
template <class Form, int HT>
__global__ __launch_bounds__(512, 2) void linear_mixed_kernel(TileArgs a, TileMap m) {
    __shared__ __attribute__((aligned(16))) uint8_t lds[Lin256<Form>::kLds];
    const TileAt at = place<false>(m);
    if (at.full) linear_tile<Lin256<Form>, HT>(a, at, 0, lds);
    else if (!at.none) linear_tile<Lin128<Form>, HT>(a, at, 0, lds);
}
// Even tiles: `down` x `across` of them, for each share of K.  Consecutive blocks go to the eight
// XCDs in turn; each XCD, and so each L2, is given one run of neighbouring tiles, eight rows of
// them column by column.
struct EvenMap {
    uint32_t across, down, per, blocks;     // per: tiles of a share
};
template <class Core, int HT>
__global__ __launch_bounds__(Core::NT, Core::NT == 512 ? 4 : 2) void linear_even_kernel(TileArgs a, EvenMap m) {
    __shared__ __attribute__((aligned(16))) uint8_t lds[Core::kLds];
    const uint32_t x = blockIdx.x % 8, run = m.blocks / 8, more = m.blocks % 8;
    const uint32_t b = x * run + min(x, more) + blockIdx.x / 8;
    const uint32_t share = b / m.per, t = b - share * m.per;
    const uint32_t group = t / (8 * m.across), rows = min(8u, m.down - 8 * group), in = t - group * 8 * m.across;
    TileAt at{};
    at.i = in / rows * Core::BP;
    at.j = (8 * group + in % rows) * Core::BQ;
    linear_tile<Core, HT>(a, at, share, lds);
}

// Adds up the shares in order and takes the sums through the epilogue.
template <int HT>
__global__ __launch_bounds__(256) void join_kernel(const float* part, uint64_t ld, uint32_t shares, Result r, Spread sp) {
    const Unit u(sp, 1);
    const uint32_t c = u.unit * 8;
    if (c >= r.I || u.row >= r.J) return;
    float v[8], t[8];
    load8<NEOX_F32>(part, u.row * ld + c, 8, v);
    for (uint32_t s = 1; s < shares; ++s) {
        load8<NEOX_F32>(part, (s * (uint64_t)r.J + u.row) * ld + c, 8, t);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += t[e];
    }
    emit8_any<HT>(r, drop_offset(r.e.drop), (uint32_t)u.row, c, v);
}

// Copies rows of `cols` 16-bit elements into rows of `pitch` elements, zeros behind them; two
// operands in one launch, the first by the first `blocks` blocks.
struct Pack {
    const uint16_t* src;
    uint16_t* dst;
    uint64_t ld, rows;
    uint32_t cols, pitch;
    uint32_t blocks;
};
__global__ __launch_bounds__(256) void pack_kernel(Pack p, Pack q) {
    const bool first = blockIdx.x < p.blocks;
    const Pack& a = first ? p : q;
    const uint32_t units = a.pitch / 8, block = first ? blockIdx.x : blockIdx.x - p.blocks;
    const uint64_t all = a.rows * units, step = a.blocks * 256ull;
    for (uint64_t u = block * 256ull + threadIdx.x; u < all; u += step) {
        const uint64_t row = u / units;
        const uint32_t c = (uint32_t)(u - row * units) * 8;
        const uint16_t* s = a.src + row * a.ld + c;
        tu32x4 v = {0, 0, 0, 0};
        if (c + 8 <= a.cols) {
            v = *(const loose_u32x4*)s;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c + e < a.cols) v[e / 2] |= (uint32_t)s[e] << (16 * (e & 1));
        }
        *(tu32x4*)(a.dst + u * 8) = v;
    }
}

// ------------------------------------------------------------------------------------
// which launch
// ------------------------------------------------------------------------------------
uint64_t tiles(uint64_t a, uint64_t b, uint64_t unit) { return ((a + unit - 1) / unit) * ((b + unit - 1) / unit); }

// Whether tiles can be loaded from where the operand lies; if not, it is packed first.
bool direct(const Operand& o, uint64_t side, uint64_t K) {
    const uint64_t cols = o.strided ? side : K;
    return (uintptr_t)o.at % 16 == 0 && o.ld % 8 == 0 && o.ld <= (1u << 22) && (o.padded || cols % 8 == 0);
}
// (whole 128-byte lines: 8192 x 24576 x 6144 takes 1780 us with rows of K + 64 elements, 2260 with
// K + 8)
uint64_t packed_pitch(const Operand& o, uint64_t side, uint64_t K) { return ((o.strided ? side : K) + 63) / 64 * 64; }
uint64_t packed_bytes(const Operand& o, uint64_t side, uint64_t K) {
    return direct(o, side, K) ? 0 : ((o.strided ? K : side) * packed_pitch(o, side, K) * 2 + 255) / 256 * 256;
}
uint64_t part_ld(uint64_t I) { return (I + 7) / 8 * 8; }

// Copies what tiles cannot be loaded from; moves `work` behind the copies.
void pack(Operand& p, uint64_t I, Operand& q, uint64_t J, uint64_t K, uint8_t*& work, hipStream_t stream) {
    auto one = [&](Operand& o, uint64_t side) {
        if (direct(o, side, K)) return Pack{};
        const uint64_t rows = o.strided ? K : side, pitch = packed_pitch(o, side, K);
        const Pack r{o.at, (uint16_t*)work, o.ld, rows, (uint32_t)(o.strided ? side : K), (uint32_t)pitch,
                     (uint32_t)std::min<uint64_t>((rows * pitch / 8 + 255) / 256, 1u << 13)};
        work += packed_bytes(o, side, K);
        o.at = r.dst;
        o.ld = pitch;
        return r;
    };
    const Pack a = one(p, I), b = one(q, J);
    if (a.blocks + b.blocks) pack_kernel<<<a.blocks + b.blocks, 256, 0, stream>>>(a, b);
}

// The launch of 256 x 256 tiles, and its cost (see product_plan).
TileMap tiles256(uint32_t I, uint32_t J, uint64_t slabs, double* cost, uint64_t* blocks) {
    return plan_tiles(256, false, I, J, 1, 1.5 * (double)slabs + 7.3, 0.75 * (double)slabs + 1.8, cost, blocks);
}

template <class T>
struct Type {
    using type = T;
};
template <class Form, int HT>
void launch_tiles(TileArgs a, const ProductPlan& c, hipStream_t stream) {
    const uint32_t I = a.r.I, J = a.r.J;
    auto even = [&](auto core) {
        using Core = typename decltype(core)::type;
        EvenMap m{};
        m.across = (I + Core::BP - 1) / Core::BP;
        m.down = (J + Core::BQ - 1) / Core::BQ;
        m.per = m.across * m.down;
        m.blocks = m.per * c.shares;
        linear_even_kernel<Core, HT><<<m.blocks, Core::NT, 0, stream>>>(a, m);
    };
    switch (c.kernel) {
    case kTiles64: even(Type<Lin64<Form>>{}); break;
    case kTiles128: even(Type<Lin128<Form>>{}); break;
    case kTiles128Deep: even(Type<Lin128d<Form>>{}); break;
    case kTiles256: {
        double cost = 0.0;
        uint64_t blocks = 0;
        const TileMap map = tiles256(I, J, c.slabs, &cost, &blocks);
        linear_mixed_kernel<Form, HT><<<(uint32_t)blocks, 512, 0, stream>>>(a, map);
    }
    }
}

}  // namespace

// The launch that costs least.  In us, fitted to 78 sizes of the three products, each timed with 4
// kernels and 1 to 8 shares of K (the choice takes 1.6% longer than the fastest of them on
// average, 25% at most): per slab of 64 elements of K and round of blocks over the chip, with up
// to `few` blocks and with more, and per round for its start and epilogue
//     64 x 64       0.27 (256 blocks), 0.53    0.9
//     128 x 128     0.66 (256),        0.91    3.5
//     .. deep       0.42 (128),        0.50    3.2
//     256 x 256     1.5, its quarters 0.75     7.3, 1.8
// and for shares (few results, long sums) a launch and the sums' way through memory, the caches
// mostly.  Blocks beyond a round start as others end: a part of a round more.
ProductPlan product_plan(uint64_t I, uint64_t J, uint64_t K) {
    const uint64_t slabs = std::max<uint64_t>(1, (K + 63) / 64), n64 = tiles(I, J, 64), n128 = tiles(I, J, 128);
    ProductPlan best{kTiles256, 1, slabs};
    uint64_t blocks = 0;
    double least = 0.0;
    tiles256((uint32_t)I, (uint32_t)J, slabs, &least, &blocks);
    auto consider = [&](ProductKernel kernel, uint64_t shares, uint64_t per, uint64_t blocks, uint64_t fit, uint64_t few,
                        double c_few, double c, double round) {
        const double join = shares == 1 ? 0.0 : 3.7 + (double)(shares * I * J) * 8e-6 / 5.7;
        const double rounds = blocks <= fit ? 1.0 : (double)blocks / (double)fit + 0.42;
        const double cost = join + rounds * ((double)per * (blocks <= few ? c_few : c) + round);
        if (cost < least) {
            least = cost;
            best = ProductPlan{kernel, (uint32_t)shares, per};
        }
    };
    for (uint64_t want = 1; want <= 16 && want <= slabs; want *= 2) {
        const uint64_t per = (slabs + want - 1) / want, shares = (slabs + per - 1) / per;
        consider(kTiles64, shares, per, n64 * shares, 512, 256, 0.27, 0.53, 0.9);
        consider(kTiles128, shares, per, n128 * shares, 512, 256, 0.66, 0.91, 3.5);
        consider(kTiles128Deep, shares, per, n128 * shares, 256, 128, 0.42, 0.50, 3.2);
        if (n64 > 1024) break;                          // enough blocks without shares
    }
    return best;
}

uint64_t product_workspace(const Product& p) {
    const ProductPlan c = product_plan(p.I, p.J, p.K);
    uint64_t n = packed_bytes(p.p, p.I, p.K) + packed_bytes(p.q, p.J, p.K);
    if (c.shares > 1) n += (c.shares * (uint64_t)p.J * part_ld(p.I) * 4 + 255) / 256 * 256;
    return n;
}

hipError_t launch_product(const Product& p, void* workspace, hipStream_t stream) {
    const ProductPlan c = product_plan(p.I, p.J, p.K);
    uint8_t* work = (uint8_t*)workspace;
    Operand P = p.p, Q = p.q;
    pack(P, p.I, Q, p.J, p.K, work, stream);
    const bool beyond = (uint64_t)p.I * p.J * (p.out_dtype == NEOX_F32 ? 4 : 2) >= kBeyond;
    const Result r{p.out, p.out_ld, p.I, p.J, p.out_dtype, beyond, p.epi};
    TileArgs a{(const uint8_t*)P.at, (const uint8_t*)Q.at, (uint32_t)(P.ld * 2), (uint32_t)(Q.ld * 2), p.K, c.slabs,
               c.shares, r};
    if (c.shares > 1) {
        a.r = Result{work, part_ld(p.I), p.I, p.J, NEOX_F32, false, Epilogue{}};
    }
    auto run = [&](auto ht) {
        constexpr int HT = decltype(ht)::value;
        constexpr bool BF = HT == NEOX_BF16;
        if (p.q.strided) launch_tiles<HalfOperands<BF, true, true>, HT>(a, c, stream);
        else if (p.p.strided) launch_tiles<HalfOperands<BF, true, false>, HT>(a, c, stream);
        else launch_tiles<HalfOperands<BF, false, false>, HT>(a, c, stream);
        if (c.shares > 1) {
            // (few results: one grid)
            const Spread sp = spread(p.J, (p.I + 7) / 8, 1);
            join_kernel<HT><<<(uint32_t)sp.blocks, 256, 0, stream>>>((const float*)work, part_ld(p.I), c.shares, r, sp);
        }
    };
    if (p.dtype == NEOX_F16) run(std::integral_constant<int, NEOX_F16>{});
    else run(std::integral_constant<int, NEOX_BF16>{});
    return hipGetLastError();
}

}  // namespace nz1
