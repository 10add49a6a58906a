// linear_kernels.hip -- products of half-precision matrices with an epilogue on gfx950: a layer's
// forward product (rows of K by rows of K), dx (W's rows are K) and dw (both operands' are).
//
// Large ones are bound by the matrix units, which are busy most of the time at a clock that this load
// lowers (see tile_core.h): 8192 x 24576 x 6144 forward 1850 to 1900 us without an epilogue (1.30 to
// 1.34 PFLOP/s, matrix units busy 67% of the time), dx 1805 to 1850 (70%), dw 1790 to 1870 (73%); a
// library product of these 1690, 1810 and 2070.
// The forward product is slower than the other two where a row of K is a multiple of 4 KB: its loads
// take 128 bytes of each of 512 rows, which then lie in the same channels of the L2; rows of K + 64
// elements take 1780 us.  Few results over long sums are split into shares of K (see product_plan).
// Few tokens are bound by reading W: one by 24576 x 6144 (302 MB) 50.8 us, 47 of them the product's
// (6.4 TB/s), the rest the join of its shares.
#include "column_sums.h"
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

// (only the layer's own product has more of an epilogue than a residual)
template <class Core, int HT, bool LAYER = !Core::Form::kStridedP>
__device__ __forceinline__ void linear_tile(const TileArgs& a, const TileAt& at, uint32_t share, uint8_t* lds) {
    const uint64_t k0 = share * a.slabs * 64;
    const uint32_t left = (uint32_t)min(a.K - k0, a.slabs * 64);
    const TileRows p = rows_of<Core::Form::kStridedP>(a.p, a.p_pitch, at.i, min((uint32_t)Core::BP, a.r.I - at.i), k0, left);
    const TileRows q = rows_of<Core::Form::kStridedQ>(a.q, a.q_pitch, at.j, min((uint32_t)Core::BQ, a.r.J - at.j), k0, left);
    Core t;
    // rows of K are zeros up to a multiple of 8
    t.run(p, q, (left + 7) / 8 * 16, lds);
    Result r = a.r;
    if (a.shares > 1) r.out = (float*)a.r.out + share * (uint64_t)a.r.J * a.r.ld;
    emit_tile<HT, LAYER>(r, t, at.i, at.j, lds);
}

// Measured and not taken: 64 x 64 tiles by 16 waves, four groups of four on a quarter of K each, sums
// joined in LDS (333 x 1024 x 4096 17.8 us against 12.7 with two shares); 64 x 64 tiles with 6 or 8
// slabs in LDS (equal with one block a CU, slower with two); 128 x 128 with 5 (equal); 128 x 64 tiles;
// slabs begun at another K on each XCD (1 to 2% slower).
template <class Form>
using Lin256 = TileCore<256, 256, 2, 4, false, 2, Form>;
template <class Form>
using Lin128 = TileCore<128, 128, 2, 4, false, 2, Form>;
template <class Form>
using Lin64 = TileCore<64, 64, 2, 2, false, 4, Form>;
template <class Form>
using Lin128d = TileCore<128, 128, 2, 4, false, 4, Form>;

// Whole tiles of 256 x 256, the rest in quarters (see TileMap).
template <class Form, int HT>
__global__ __launch_bounds__(512, 2) void linear_mixed_kernel(TileArgs a, TileMap m) {
    __shared__ __attribute__((aligned(16))) uint8_t lds[Lin256<Form>::kLds];
    const TileAt at = place<false>(m);
    if (at.full) linear_tile<Lin256<Form>, HT>(a, at, 0, lds);
    else if (!at.none) linear_tile<Lin128<Form>, HT>(a, at, 0, lds);
}
// Even tiles: `down` x `across` of them, for each share of K.  Consecutive blocks go to the eight
// XCDs in turn; each XCD, and so each L2, is given one run of neighbouring tiles, eight rows of
// them column by column (dw of 8000 x 704 x 6000 on 64 x 64 tiles 290 us in plain order, 167 so).
struct EvenMap {
    uint32_t across, down, per, blocks;     // per: tiles of a share
};
template <class Core>
__device__ __forceinline__ TileAt even_tile(const EvenMap& m, uint32_t block, uint32_t& share) {
    const uint32_t x = block % 8, run = m.blocks / 8, more = m.blocks % 8;
    const uint32_t b = x * run + min(x, more) + block / 8;
    share = b / m.per;
    const uint32_t t = b - share * m.per;
    const uint32_t group = t / (8 * m.across), rows = min(8u, m.down - 8 * group), in = t - group * 8 * m.across;
    TileAt at{};
    at.i = in / rows * Core::BP;
    at.j = (8 * group + in % rows) * Core::BQ;
    return at;
}
template <class Core, int HT>
__global__ __launch_bounds__(Core::NT, Core::NT == 512 ? 4 : 2) void linear_even_kernel(TileArgs a, EvenMap m) {
    __shared__ __attribute__((aligned(16))) uint8_t lds[Core::kLds];
    uint32_t share;
    const TileAt at = even_tile<Core>(m, blockIdx.x, share);
    linear_tile<Core, HT>(a, at, share, lds);
}
// The joins of the bias's gradient (first: they wait for memory mostly), dx's tiles and dw's, side by
// side: neither product of a few thousand tokens fills the chip alone.
template <class CoreX, class CoreW, int HT>
__global__ __launch_bounds__(CoreX::NT, CoreX::NT == 512 ? 4 : 2) void linear_pair_kernel(TileArgs x, EvenMap mx, TileArgs w,
                                                                                          EvenMap mw, Backward b, const float* sums,
                                                                                          uint32_t parts, uint32_t joins) {
    static_assert(CoreX::kLds == CoreW::kLds && CoreX::NT == CoreW::NT, "");
    __shared__ __attribute__((aligned(16))) uint8_t lds[CoreX::kLds];
    uint32_t share;
    if (blockIdx.x < joins) {
        join_columns<HT>(b, sums, parts, blockIdx.x, (float*)lds);
        return;
    }
    const uint32_t block = blockIdx.x - joins;
    if (block < mx.blocks) {
        const TileAt at = even_tile<CoreX>(mx, block, share);
        linear_tile<CoreX, HT>(x, at, share, lds);
    } else {
        const TileAt at = even_tile<CoreW>(mw, block - mx.blocks, share);
        linear_tile<CoreW, HT>(w, at, share, lds);
    }
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
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = opaque(v[e] * r.scale);
    emit8_any<HT>(r, drop_offset(r.e.drop), (uint32_t)u.row, c, v);
}

// Copies rows of `cols` 16-bit elements into rows of `pitch` elements, zeros behind them; up to three
// operands in one launch.
struct Pack {
    const uint16_t* src;
    uint16_t* dst;
    uint64_t ld, rows;
    uint32_t cols, pitch;
    uint32_t blocks;
};
__global__ __launch_bounds__(256) void pack_kernel(Pack p, Pack q, Pack r) {
    uint32_t block = blockIdx.x;
    const Pack* a = &p;
    if (block >= p.blocks) {
        block -= p.blocks;
        a = &q;
        if (block >= q.blocks) {
            block -= q.blocks;
            a = &r;
        }
    }
    const uint32_t units = a->pitch / 8;
    const uint64_t all = a->rows * units, step = a->blocks * 256ull;
    for (uint64_t u = block * 256ull + threadIdx.x; u < all; u += step) {
        const uint64_t row = u / units;
        const uint32_t c = (uint32_t)(u - row * units) * 8;
        const uint16_t* s = a->src + row * a->ld + c;
        tu32x4 v = {0, 0, 0, 0};
        if (c + 8 <= a->cols) {
            v = *(const loose_u32x4*)s;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c + e < a->cols) v[e / 2] |= (uint32_t)s[e] << (16 * (e & 1));
        }
        *(tu32x4*)(a->dst + u * 8) = v;
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
uint64_t part_ld(uint64_t I) { return (I + 7) / 8 * 8; }

// The launch of 256 x 256 tiles, and its cost (see product_plan).
TileMap tiles256(uint32_t I, uint32_t J, uint64_t slabs, double* cost, uint64_t* blocks) {
    return plan_tiles(256, false, I, J, 1, 1.5 * (double)slabs + 7.3, 0.75 * (double)slabs + 1.8, cost, blocks);
}

template <class T>
struct Type {
    using type = T;
};
EvenMap even_map(const TileArgs& a, uint32_t unit) {
    EvenMap m{};
    m.across = (a.r.I + unit - 1) / unit;
    m.down = (a.r.J + unit - 1) / unit;
    m.per = m.across * m.down;
    m.blocks = m.per * a.shares;
    return m;
}
// From this many bytes on, an operand that one row of tiles reads is not kept in the caches: no other
// block asks for it, and a model's weights do not fit them.  One token by 24576 x 6144 56 -> 51 us, by
// 4096 x 4096 11.7 -> 10.5, by 4096 x 1024 (8 MB, kept by the caches from call to call) 6.0 -> 6.7.
constexpr uint64_t kOnce = 1ull << 25;

template <bool BF, bool PS, bool QS, int HT>
void launch_tiles(const TileArgs& a, const ProductPlan& c, hipStream_t stream) {
    using Form = HalfOperands<BF, PS, QS>;
    const uint32_t I = a.r.I, J = a.r.J;
    auto even = [&](auto core) {
        using Core = typename decltype(core)::type;
        const EvenMap m = even_map(a, Core::BP);
        linear_even_kernel<Core, HT><<<m.blocks, Core::NT, 0, stream>>>(a, m);
    };
    if constexpr (!QS) {
        using Once = HalfOperands<BF, PS, QS, true>;
        if (J <= 64 && I * a.K * 2 >= kOnce && c.kernel == kTiles64) return even(Type<Lin64<Once>>{});
        if (J <= 64 && I * a.K * 2 >= kOnce && c.kernel == kTiles128Deep) return even(Type<Lin128d<Once>>{});
    }
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

// Costs of a launch of even tiles, in us (see product_plan): of one block, and of them all.
struct EvenCost {
    uint64_t fit, few;
    double c_few, c, round;
};
constexpr EvenCost kCost[3] = {{512, 256, 0.27, 0.53, 0.9}, {512, 256, 0.66, 0.91, 3.5}, {256, 128, 0.42, 0.50, 3.2}};
double block_cost(const EvenCost& k, uint64_t blocks, uint64_t slabs) {
    return (double)slabs * (blocks <= k.few ? k.c_few : k.c) + k.round;
}
double even_cost(const EvenCost& k, uint64_t blocks, uint64_t slabs) {
    return (blocks <= k.fit ? 1.0 : (double)blocks / (double)k.fit + 0.42) * block_cost(k, blocks, slabs);
}
double join_cost(uint64_t shares, uint64_t I, uint64_t J) {
    return shares == 1 ? 0.0 : 3.7 + (double)(shares * I * J) * 8e-6 / 5.7;
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
// mostly.  Blocks beyond a round start as others end: a part of a round more.  No launch takes less
// than its operands at 6.8 TB/s (products of 1 to 128 tokens with weights from memory, 30 of them: 3.3%
// longer than the fastest on average).  At most 16 shares: few results of the longest sums leave CUs
// without a block (64 x 64 over K = 2^20: 16 blocks, 280 us by these costs where the bytes take 43), and
// a share's FP32 sums are as long as a sixteenth of K.
ProductPlan product_plan(uint64_t I, uint64_t J, uint64_t K) {
    const uint64_t slabs = std::max<uint64_t>(1, (K + 63) / 64), n64 = tiles(I, J, 64), n128 = tiles(I, J, 128);
    ProductPlan best{kTiles256, 1, slabs, 0.0};
    uint64_t blocks = 0;
    tiles256((uint32_t)I, (uint32_t)J, slabs, &best.cost, &blocks);
    for (uint64_t want = 1; want <= 16 && want <= slabs; want *= 2) {
        const uint64_t per = (slabs + want - 1) / want, shares = (slabs + per - 1) / per;
        for (int k = kTiles64; k <= kTiles128Deep; ++k) {
            const double work = even_cost(kCost[k], (k == kTiles64 ? n64 : n128) * shares, per);
            const double cost = join_cost(shares, I, J) + std::max(work, 1.9 + (double)((I + J) * K) * 2e-6 / 6.8);
            if (cost < best.cost) best = ProductPlan{(ProductKernel)k, (uint32_t)shares, per, cost};
        }
        if (n64 > 1024) break;                          // enough blocks without shares
    }
    return best;
}

// Each keeps its shares, so neither's results depend on the other.  A block of one lasts as long as its
// sums; together they fill rounds.  2048 x 4096 x 1024 43 us against 28.5 + 21.5, 1000 x 1000 x 1000 12.7
// against 7.7 + 8.
bool pair_plan(uint64_t Ix, uint64_t Jx, const ProductPlan& x, uint64_t Iw, uint64_t Jw, const ProductPlan& w,
               ProductKernel* kernel) {
    double least = x.cost + w.cost + 2.0;               // a launch more
    bool pair = false;
    for (int k = kTiles64; k <= kTiles128Deep; ++k) {
        const uint64_t unit = k == kTiles64 ? 64 : 128;
        const uint64_t bx = tiles(Ix, Jx, unit) * x.shares, bw = tiles(Iw, Jw, unit) * w.shares, all = bx + bw;
        const double cx = block_cost(kCost[k], all, x.slabs), cw = block_cost(kCost[k], all, w.slabs);
        const double longest = std::max(cx, cw), work = ((double)bx * cx + (double)bw * cw) / (double)kCost[k].fit;
        const double cost = join_cost(x.shares, Ix, Jx) + join_cost(w.shares, Iw, Jw) +
                            (all <= kCost[k].fit ? longest : std::max(longest, work + 0.42 * longest));
        if (all < 1ull << 22 && cost < least) {
            least = cost;
            *kernel = (ProductKernel)k;
            pair = true;
        }
    }
    return pair;
}

namespace {

// The products of one call, with their packed operands and shares in the workspace.
struct Placed {
    const Product* p = nullptr;
    Operand q{};               // where tiles load it from
    ProductPlan c{};
    TileArgs a{};
    Result r{};
    const float* part = nullptr;
};
struct Work {
    Pack packs[3] = {};
    Placed at[2];
    int n = 0, npacks = 0;
    uint64_t bytes = 0;

    // base: the workspace's address, 0 where only its size is asked for
    Work(const Product* x, const Product* w, uintptr_t base) {
        for (const Product* p : {x, w})
            if (p) at[n++].p = p;
        for (int i = 0; i < n; ++i) {
            Placed& t = at[i];
            const Product& p = *t.p;
            t.c = product_plan(p.I, p.J, p.K);
            const Operand P = operand(p.p, p.I, p.K, base);
            // d is an operand of both gradients' products and is copied once: its rows are the same,
            // whichever way it is read.  (By its role, not by its address: what a workspace needs does
            // not depend on where the operands lie.)
            t.q = i == 0 ? operand(p.q, p.J, p.K, base) : at[0].q;
            t.r = Result{p.out, p.out_ld, p.I, p.J, p.out_dtype, (uint64_t)p.I * p.J * (p.out_dtype == NEOX_F32 ? 4 : 2) >= kBeyond,
                         p.scale, p.epi};
            t.a = TileArgs{(const uint8_t*)P.at, (const uint8_t*)t.q.at, (uint32_t)(P.ld * 2), (uint32_t)(t.q.ld * 2), p.K, t.c.slabs,
                           t.c.shares, t.r};
            if (t.c.shares > 1) {
                t.part = (const float*)(base + bytes);
                t.a.r = Result{(void*)(base + bytes), part_ld(p.I), p.I, p.J, NEOX_F32, false, 1.0f, Epilogue{}};
                bytes += (t.c.shares * (uint64_t)p.J * part_ld(p.I) * 4 + 255) / 256 * 256;
            }
        }
    }
    // The operand itself where tiles can be loaded from it, or its copy.
    Operand operand(Operand o, uint64_t side, uint64_t K, uintptr_t base) {
        if (direct(o, side, K)) return o;
        const uint64_t rows = o.strided ? K : side, cols = o.strided ? side : K, pitch = packed_pitch(o, side, K);
        packs[npacks++] = Pack{o.at, (uint16_t*)(base + bytes), o.ld, rows, (uint32_t)cols, (uint32_t)pitch,
                               (uint32_t)std::min<uint64_t>((rows * pitch / 8 + 255) / 256, 1u << 13)};
        o.at = (const uint16_t*)(base + bytes);
        o.ld = pitch;
        bytes += (rows * pitch * 2 + 255) / 256 * 256;
        return o;
    }
};

template <int HT>
hipError_t launch_work(const Work& w, const Backward* join, const void* sums, hipStream_t stream) {
    constexpr bool BF = HT == NEOX_BF16;
    const uint32_t blocks = w.packs[0].blocks + w.packs[1].blocks + w.packs[2].blocks;
    if (blocks) pack_kernel<<<blocks, 256, 0, stream>>>(w.packs[0], w.packs[1], w.packs[2]);
    ProductKernel kernel;
    if (w.n == 2 && pair_plan(w.at[0].p->I, w.at[0].p->J, w.at[0].c, w.at[1].p->I, w.at[1].p->J, w.at[1].c, &kernel)) {
        const TileArgs &x = w.at[0].a, &d = w.at[1].a;
        const uint32_t parts = join ? backward_parts(join->rows, join->cols) : 0;
        const uint32_t joins = parts ? (uint32_t)((join->cols + 63) / 64) : 0;
        auto pair = [&](auto cx, auto cw) {
            using X = typename decltype(cx)::type;
            using W = typename decltype(cw)::type;
            const EvenMap mx = even_map(x, X::BP), mw = even_map(d, X::BP);
            linear_pair_kernel<X, W, HT><<<mx.blocks + mw.blocks + joins, X::NT, 0, stream>>>(
                x, mx, d, mw, join ? *join : Backward{}, (const float*)sums, parts, joins);
        };
        using FX = HalfOperands<BF, true, false>;
        using FW = HalfOperands<BF, true, true>;
        if (kernel == kTiles64) pair(Type<Lin64<FX>>{}, Type<Lin64<FW>>{});
        else if (kernel == kTiles128) pair(Type<Lin128<FX>>{}, Type<Lin128<FW>>{});
        else pair(Type<Lin128d<FX>>{}, Type<Lin128d<FW>>{});
    } else {
        if (join) {
            const hipError_t e = launch_join(*join, sums, stream);
            if (e != hipSuccess) return e;
        }
        for (int i = 0; i < w.n; ++i) {
            const Placed& t = w.at[i];
            if (t.p->q.strided) launch_tiles<BF, true, true, HT>(t.a, t.c, stream);
            else if (t.p->p.strided) launch_tiles<BF, true, false, HT>(t.a, t.c, stream);
            else launch_tiles<BF, false, false, HT>(t.a, t.c, stream);
        }
    }
    for (int i = 0; i < w.n; ++i) {
        const Placed& t = w.at[i];
        if (t.c.shares == 1) continue;
        // (few results: one grid)
        const Spread sp = spread(t.r.J, (t.r.I + 7) / 8, 1);
        join_kernel<HT><<<(uint32_t)sp.blocks, 256, 0, stream>>>(t.part, part_ld(t.r.I), t.c.shares, t.r, sp);
    }
    return hipGetLastError();
}

}  // namespace

uint64_t products_workspace(const Product* x, const Product* w) { return Work(x, w, 0).bytes; }

hipError_t launch_products(const Product* x, const Product* w, const Backward* join, const void* sums, void* workspace,
                           hipStream_t stream) {
    const Work work(x, w, (uintptr_t)workspace);
    return (x ? x : w)->dtype == NEOX_F16 ? launch_work<NEOX_F16>(work, join, sums, stream)
                                          : launch_work<NEOX_BF16>(work, join, sums, stream);
}

}  // namespace nz1
