// matrix_kernels.hip -- Newton-Schulz orthogonalisation and the Muon update on gfx950.
//
// For each step, with X m x n (m <= n):
//   gram   A = X X^T                       symmetric: tiles on and below the diagonal only
//   sym    P = a I + b A + c A A           symmetric, as A is (A A = A A^T)
//   apply  X <- P X
// All three are products of rows with rows once X is kept in both orientations, so they
// share one tile core.
//
// Two steps at a time.  The next A is P A P, without X; so with n >= 2 m two steps go into one
// X <- (P' P) X at the cost of three more m x m products (they commute and are symmetric: half
// their tiles): 8.5 units of m^3 instead of 13 at n = 4 m, and X is read and written half as
// often.  Not more than two: an error of FP16's size in the part of A that belongs to tiny
// singular values grows by a^2 (12) a step, harmless once (1e-3 of a), not twice.
//
// Precision.  Products read FP16.  Rounding the iterate itself to FP16 in each step would
// put noise into the directions whose singular values are still tiny, and a later step
// multiplies those by up to a (3.4 per step, ~500 in five): a rank-1 matrix came out 15%
// off.  So X is carried as two FP16 numbers (22 bits), and only the products P X and X X^T
// see the first alone: their error is filtered through P or X once more and stays at the
// FP16 level.  A and P have diagonals far larger than the rest (of similar size along the
// diagonal too, so that their roundings would add up in one direction): the diagonals are
// kept in FP32, apart, and FP16 holds the rest.  Simulated against 64 bits: matrices of 128
// rows and more with Gaussian, decaying and low-rank (Gaussian factors) spectra 2e-4 .. 2e-3 of
// the result's norm, 4e-3 at rank 1 below 256 rows.  That counts on roundings of either sign in
// many elements.  Fewer rows leave fewer to average over: at rank 1 up to 0.15 / sqrt(rows) (1e-2
// at 128 rows, 8e-2 at 4), half of it at rank 4, 1e-3 at full rank.  And equal elements of A are
// rounded alike: of 16 million matrices of 1 to 64 diagonal blocks of ones half were off by 2e-3,
// one in a thousand by 1.5e-2, the worst by 2.6e-2; with two steps at a time, of 8 million, 4e-3,
// 2.7e-2 and 4.4e-2.  (All roundings at their largest and of one sign give 8e-2 and 1.3e-1 to
// first order.)  A second half for A and P, as X has one, would take that away, for twice the
// products and more.
#include "matrix_internal.h"
#include "tile_core.h"

#include <algorithm>
#include <type_traits>

namespace nz1 {

namespace {

constexpr float kLo = 2048.0f;            // lt holds (x - hi) * kLo

// The step state whose skip flag the kernels heed (none: always run).
__host__ __device__ inline const DevState* state_of(const OrthIO&) { return nullptr; }
__host__ __device__ inline const DevState* state_of(const MuonIO& io) { return io.st; }
__device__ __forceinline__ bool skipped(const DevState* st) { return st && st->skip; }

template <int NT>
__device__ __forceinline__ double sum_block(double v) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
    __shared__ double ws[NT / 64];
    if ((threadIdx.x & 63) == 0) ws[threadIdx.x >> 6] = v;
    __syncthreads();
    double r = ws[0];
#pragma unroll
    for (int k = 1; k < NT / 64; ++k) r += ws[k];
    return r;
}

// Four consecutive elements, as one load of 16 bytes (8 for halves).
__device__ __forceinline__ tf32x4 halves4(int dtype, uint2 q) {
    return tf32x4{half_to_float(dtype, (uint16_t)q.x), half_to_float(dtype, (uint16_t)(q.x >> 16)),
                  half_to_float(dtype, (uint16_t)q.y), half_to_float(dtype, (uint16_t)(q.y >> 16))};
}
__device__ __forceinline__ tf32x4 vec4(const void* p, int dtype, uint64_t i) {
    if (dtype == NEOX_F32) return *(const tf32x4*)((const float*)p + i);
    return halves4(dtype, *(const uint2*)((const uint16_t*)p + i));
}

// ------------------------------------------------------------------------------------
// squared norm of each source matrix; for Muon also the momentum's own update
//
// Memory-bound: 1,024 threads a block and at most kNsParts blocks a matrix, so that one large
// matrix still has a block on every CU with two vectors in flight a thread.  Sums in 64 bits.
// Measured: the momentum of 24576 x 6144 (10 B an element) 263 us, 5.7 TB/s; the norm of 8 of
// 4096 x 1024 in BF16 20 us, of 6144 x 6144 35 us (2.1 TB/s, 0.8% of that call).
// Which elements a thread adds, and in which order, goes by the shape alone: where the arrays'
// alignment or strides keep four neighbours from one load they are loaded one by one, in the
// same places, so that a matrix's norm has the same bits wherever it lies.
// ------------------------------------------------------------------------------------
constexpr int kNormThreads = 1024;

__device__ __forceinline__ double square4(tf32x4 v, double s) {
#pragma unroll
    for (int e = 0; e < 4; ++e) s = __builtin_fma((double)v[e], (double)v[e], s);
    return s;
}

__global__ __launch_bounds__(kNormThreads) void orth_norm_kernel(OrthIO io, uint32_t rows, uint32_t cols,
                                                                 uint32_t parts, double* __restrict__ part) {
    const uint32_t z = blockIdx.x / parts, p = blockIdx.x % parts;
    const uint32_t per = (rows + parts - 1) / parts;
    const uint32_t r0 = p * per, r1 = min(rows, r0 + per);
    const uint64_t at = z * io.src_stride;
    double s = 0.0, t = 0.0;
    if (cols % 4 == 0) {
        // this block's rows as one run of fours, two in flight
        const uint32_t w = cols / 4;
        uint32_t r = r0 + threadIdx.x / w, c = threadIdx.x % w;
        const uint32_t dr = kNormThreads / w, dc = kNormThreads % w;
        auto next = [&]() {
            r += dr;
            c += dc;
            if (c >= w) {
                c -= w;
                ++r;
            }
        };
        auto four = [&]() {
            const uint64_t i = at + r * io.src_ld + 4 * c;
            if (io.vec_src) return vec4(io.src, io.src_dtype, i);
            tf32x4 x;
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = load_elem(io.src, io.src_dtype, i + e);
            return x;
        };
        while (r < r1) {
            const tf32x4 v = four();
            next();
            if (r < r1) {
                const tf32x4 q = four();
                t = square4(q, t);
            }
            s = square4(v, s);
            next();
        }
    } else {
        // element by element, eight rows in flight
        for (uint32_t r = r0; r < r1; r += 8)
            for (uint32_t c = threadIdx.x; c < cols; c += kNormThreads) {
                float x[8];
#pragma unroll
                for (uint32_t k = 0; k < 8; ++k)
                    x[k] = r + k < r1 ? load_elem(io.src, io.src_dtype, at + (r + k) * io.src_ld + c) : 0.0f;
#pragma unroll
                for (uint32_t k = 0; k < 8; ++k) s = __builtin_fma((double)x[k], (double)x[k], s);
            }
    }
    s = sum_block<kNormThreads>(s + t);
    if (threadIdx.x == 0) part[(uint64_t)z * kNsParts + p] = s;
}

__device__ __forceinline__ float direction(const MuonIO& io, float g, float m) {
    return io.nesterov ? __builtin_fmaf(io.mu, m, g) : m;
}

__global__ __launch_bounds__(kNormThreads) void muon_momentum_kernel(MuonIO io, uint64_t numel, uint32_t parts,
                                                                     double* __restrict__ part) {
    if (io.st->skip) return;
    const float gs = io.st->gscale;
    const uint32_t z = blockIdx.x / parts, p = blockIdx.x % parts;
    const MuonMat mat = io.mats[z];
    double s = 0.0;
    const uint64_t n4 = numel / 4, step = (uint64_t)parts * kNormThreads, first = (uint64_t)p * kNormThreads + threadIdx.x;
    auto fours = [&](auto vec) {
        auto load = [&](uint64_t i, tf32x4& g, tf32x4& m) {
            if constexpr (vec) {
                g = halves4(io.dtype, *(const uint2*)(mat.grad + i));
                m = *(const tf32x4*)(mat.mom + i);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    g[e] = half_to_float(io.dtype, mat.grad[i + e]);
                    m[e] = mat.mom[i + e];
                }
            }
        };
        for (uint64_t i = first; i < n4; i += 2 * step) {
            const uint64_t j = i + step < n4 ? i + step : i;        // the same again at the end
            tf32x4 g[2], m[2];
            load(4 * i, g[0], m[0]);
            load(4 * j, g[1], m[1]);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if (k == 1 && j == i) break;
                tf32x4 u;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float x = g[k][e] * gs;
                    m[k][e] = __builtin_fmaf(io.mu, m[k][e], x);
                    u[e] = direction(io, x, m[k][e]);
                }
                float* to = mat.mom + 4 * (k ? j : i);
                if constexpr (vec) {
                    *(tf32x4*)to = m[k];
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) to[e] = m[k][e];
                }
                s = square4(u, s);
            }
        }
    };
    if (mat.vec) fours(std::true_type{});
    else fours(std::false_type{});
    for (uint64_t i = 4 * n4 + first; i < numel; i += step) {
        const float g = half_to_float(io.dtype, mat.grad[i]) * gs;
        const float m = __builtin_fmaf(io.mu, mat.mom[i], g);
        mat.mom[i] = m;
        const double u = direction(io, g, m);
        s = __builtin_fma(u, u, s);
    }
    s = sum_block<kNormThreads>(s);
    if (threadIdx.x == 0) part[(uint64_t)z * kNsParts + p] = s;
}

// ------------------------------------------------------------------------------------
// X0 = source / (norm + eps), split in two, both orientations, zero padded
//
// Memory-bound: 64 x 64 elements a block through LDS, rows of 128 bytes written.  Measured:
// 24576 x 6144 for Muon (6 B read, 6 written an element) 395 us, 4.6 TB/s.
// ------------------------------------------------------------------------------------
struct OrthSrc {
    const OrthIO& io;
    uint64_t at;
    bool vec;
    __device__ OrthSrc(const OrthIO& i, const NsShape& s, uint32_t z)
        : io(i), at(z * i.src_stride), vec(i.vec_src && s.cols % 4 == 0) {}
    __device__ float load(uint32_t r, uint32_t c, uint32_t) const {
        return load_elem(io.src, io.src_dtype, at + r * io.src_ld + c);
    }
    __device__ tf32x4 load4(uint32_t r, uint32_t c, uint32_t) const {
        return vec4(io.src, io.src_dtype, at + r * io.src_ld + c);
    }
};
struct MuonSrc {
    const MuonIO& io;
    MuonMat mat;
    float gs;
    bool vec;
    __device__ MuonSrc(const MuonIO& i, const NsShape& s, uint32_t z)
        : io(i), mat(i.mats[z]), gs(i.st->gscale), vec(mat.vec && s.cols % 4 == 0) {}
    __device__ float load(uint32_t r, uint32_t c, uint32_t cols) const {
        const uint64_t i = (uint64_t)r * cols + c;
        return direction(io, half_to_float(io.dtype, mat.grad[i]) * gs, mat.mom[i]);
    }
    __device__ tf32x4 load4(uint32_t r, uint32_t c, uint32_t cols) const {
        const uint64_t i = (uint64_t)r * cols + c;
        const tf32x4 g = halves4(io.dtype, *(const uint2*)(mat.grad + i)), m = *(const tf32x4*)(mat.mom + i);
        tf32x4 u;
#pragma unroll
        for (int e = 0; e < 4; ++e) u[e] = direction(io, g[e] * gs, m[e]);
        return u;
    }
};

template <class Src, class IO>
__global__ __launch_bounds__(256) void ns_convert_kernel(IO io, NsShape s, NsBuf w) {
    if (skipped(state_of(io))) return;
    __shared__ float tile[64][65];
    const uint32_t ti = s.mp / 64, tj = s.np / 64;
    const uint32_t z = blockIdx.x / (ti * tj), t = blockIdx.x % (ti * tj);
    const uint32_t i0 = t / tj * 64, j0 = t % tj * 64;
    const double* part = w.part + (uint64_t)z * kNsParts;
    const Src src(io, s, z);
    // lane: four neighbours of one of sixteen rows
    const uint32_t q = (threadIdx.x & 15) * 4, k0 = threadIdx.x >> 4;
    // the tile as the source has it: rows r0.., columns c0..
    const uint32_t r0 = s.tall ? j0 : i0, c0 = s.tall ? i0 : j0;
    tf32x4 v[4];
#pragma unroll
    for (uint32_t k = 0; k < 4; ++k) {
        const uint32_t r = r0 + k0 + 16 * k, c = c0 + q;
        v[k] = tf32x4{0, 0, 0, 0};
        if (r < s.rows && c < s.cols) {
            if (src.vec) {
                v[k] = src.load4(r, c, s.cols);
            } else {
#pragma unroll
                for (uint32_t e = 0; e < 4; ++e)
                    if (c + e < s.cols) v[k][e] = src.load(r, c + e, s.cols);
            }
        }
    }
    const double sq = sum_block<256>(threadIdx.x < s.parts ? part[threadIdx.x] : 0.0);
    const double f = (double)s.s / (__builtin_sqrt(sq) + io.eps);
    // products in 64 bits: f overflows or vanishes in 32 where the source is tiny or huge
#pragma unroll
    for (uint32_t k = 0; k < 4; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) tile[k0 + 16 * k][q + e] = (float)((double)v[k][e] * f);
    __syncthreads();
    const uint64_t xz = (uint64_t)z * s.mp * s.np;
#pragma unroll
    for (uint32_t k = 0; k < 4; ++k) {
        // row `row` of the tile in the wide form, and column `row` of it
        const uint32_t row = k0 + 16 * k;
        f16x4 across, hi, lo;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float a = tile[row][q + e], b = tile[q + e][row];
            across[e] = (_Float16)(s.tall ? b : a);
            const float y = s.tall ? a : b;
            hi[e] = (_Float16)y;
            lo[e] = (_Float16)((y - (float)hi[e]) * kLo);
        }
        *(f16x4*)(w.xh + xz + (uint64_t)(i0 + row) * s.np + j0 + q) = across;
        const uint64_t at = xz + (uint64_t)(j0 + row) * s.mp + i0 + q;
        *(f16x4*)(w.xt[0] + at) = hi;
        *(f16x4*)(w.lt + at) = lo;
    }
}

// ------------------------------------------------------------------------------------
// the products
// ------------------------------------------------------------------------------------
// Kernels of one launch each, an operation's tile() on a block's tile.  Measured at 24576 x 6144
// (m = 6144, n = 24576): P X 1.61 ms (1.15 PFLOP/s), the last one with Muon's update 1.80 ms,
// products of m x m matrices 222 us (half their tiles: 1.05 PFLOP/s), X X^T of 6144 x 6144
// 226 us.  The main loop alone would run at 1.3 (see tile_core.h); the rest is the epilogue,
// where all CUs read and write memory at once for about 30 us a round of tiles: 10 bytes an
// element for P X, 14 to 18 for the update.
//
// The tile of a block, for launches of one tile size only (TileMap: of two).
template <class Core, bool SYM>
__device__ __forceinline__ TileAt place_even(uint32_t mp, uint32_t np) {
    const uint32_t p = mp / Core::BP, q = np / Core::BQ, tiles = SYM ? p * (p + 1) / 2 : p * q;
    TileAt r{};
    r.z = blockIdx.x / tiles;
    const uint32_t t = blockIdx.x % tiles;
    uint32_t ti, tj;
    if (SYM) {
        lower(t, ti, tj);
    } else {
        ti = t / q;
        tj = t % q;
    }
    r.i = ti * Core::BP;
    r.j = tj * Core::BQ;
    r.settle();
    return r;
}

__device__ __forceinline__ TileRows rows_of(const uint16_t* base, uint64_t row, uint32_t len, int block) {
    return TileRows{(const uint8_t*)(base + row * len), nullptr, (uint32_t)block, len * 2u, 0u};
}

// A symmetric matrix: FP16 without its diagonal, and the diagonal.
struct SymBuf {
    uint16_t* a;
    float* d;
};

// A lane of a 16 x 16 result tile holds four consecutive rows of one column.  These are the
// elements of the same tile that are four consecutive columns of one row (row lane % 16,
// columns 4 (lane / 16) + 0..3): the four FP16 values, taken as the left operand of a product
// with the identity, come out transposed and exact.
__device__ __forceinline__ tf32x4 transposed(f16x4 v) {
    const uint32_t lane = threadIdx.x & 63;
    f16x4 one;
#pragma unroll
    for (int e = 0; e < 4; ++e) one[e] = (lane >> 4) * 4 + e == (lane & 15) ? (_Float16)1.0f : (_Float16)0.0f;
    return __builtin_amdgcn_mfma_f32_16x16x16f16(v, one, tf32x4{0, 0, 0, 0}, 0, 0, 0);
}
__device__ __forceinline__ f16x4 pack4(tf32x4 v) {
    return f16x4{(_Float16)v[0], (_Float16)v[1], (_Float16)v[2], (_Float16)v[3]};
}

// An FP16 result on and below the diagonal, to both sides of it, without the diagonal; the
// diagonal, and more(i) added to it, to d.  What lies above the diagonal always is what lies
// below it, inside a tile too: L M and M L of commuting matrices are one matrix but not one sum
// of rounded products, so an element computed above the diagonal would depend on how far its
// tile reaches over it, and a matrix's bits on the launch's choice of tiles.
template <class Core, class More>
__device__ __forceinline__ void store_sym(const Piece<Core>& p, tf32x4 (&acc)[Core::TP][Core::TQ], int u0,
                                          uint16_t* out, uint32_t ld, float* d, More more) {
    using P = Piece<Core>;
    if (p.i >= p.j + 16 * P::kV) {
        // all of it below the diagonal
#pragma unroll
        for (int u = 0; u < P::kU; ++u)
#pragma unroll
            for (int v = 0; v < P::kV; ++v) {
                const f16x4 h = pack4(acc[u0 + u][v]);
                *p.down(p.l0, u, v) = h;
                *p.across(p.l1, u, v) = pack4(transposed(h));
            }
        P::Down::store(p.l0, out + (uint64_t)p.j * ld + p.i, ld);
        P::Across::store(p.l1, out + (uint64_t)p.i * ld + p.j, ld);
        return;
    }
    // a piece of a tile on the diagonal: 16 x 16 at a time, eight bytes a lane
#pragma unroll
    for (int u = 0; u < P::kU; ++u)
#pragma unroll
        for (int v = 0; v < P::kV; ++v) {
            const uint32_t i = p.i + 16 * u, j = p.j + 16 * v;
            if (i < j) continue;
            tf32x4 x = acc[u0 + u][v];
            if (i == j) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (p.li + e == p.lj) {
                        d[j + p.lj] = x[e] + more(j + p.lj);
                        x[e] = 0.0f;
                    }
            }
            const f16x4 h = pack4(x);
            f16x4 a = pack4(transposed(h));
            if (i == j) {
#pragma unroll
                for (int e = 0; e < 4; ++e) a[e] = p.li + e > p.lj ? h[e] : a[e];
            } else {
                *(f16x4*)(out + (uint64_t)(j + p.lj) * ld + i + p.li) = h;
            }
            *(f16x4*)(out + (uint64_t)(i + p.lj) * ld + j + p.li) = a;
        }
}

// A = X X^T
struct Gram {
    static constexpr bool SYM = true;
    const uint16_t* xh;
    SymBuf out;
    uint32_t mp, np;
    float inv_s2;
    template <class Core>
    __device__ __forceinline__ void tile(const TileAt& at, uint8_t* lds) const {
        using P = Piece<Core>;
        const uint16_t* x = xh + (uint64_t)at.z * mp * np;
        Core t;
        t.run(rows_of(x, at.i, np, Core::BP), rows_of(x, at.j, np, Core::BQ), np * 2, lds);
#pragma unroll
        for (int u0 = 0; u0 < Core::TP; u0 += P::kU) {
#pragma unroll
            for (int u = 0; u < P::kU; ++u)
#pragma unroll
                for (int v = 0; v < P::kV; ++v) t.acc[u0 + u][v] = t.acc[u0 + u][v] * inv_s2;
            store_sym<Core>(P(at, u0, lds), t.acc, u0, out.a + (uint64_t)at.z * mp * mp, mp,
                            out.d + (uint64_t)at.z * mp, [](uint32_t) { return 0.0f; });
        }
    }
};

// X X^T of a few rows and many columns, K split: block `part` of `parts` sums its share of the
// columns of one 64 x 64 tile, and a second launch adds the shares in order.  One after the
// other, the 64-column slabs of 64 x 8192 take 29 us on one CU; in 16 shares 2, and 4 to join.
struct GramSplit {
    const uint16_t* xh;
    SymBuf out;
    float* sums;               // [matrix][part][tile][64 * 64], in the order of the lanes
    uint32_t mp, np, parts;
    float inv_s2;
};
using Core64 = TileCore<64, 64, 2, 2, false, 4>;
__global__ __launch_bounds__(Core64::NT) void gram_part_kernel(GramSplit g, const DevState* st) {
    if (skipped(st)) return;
    __shared__ __attribute__((aligned(16))) uint8_t lds[room<Core64>()];
    const uint32_t side = g.mp / 64, tiles = side * (side + 1) / 2;
    const uint32_t t = blockIdx.x % tiles, zp = blockIdx.x / tiles, z = zp / g.parts, part = zp % g.parts;
    TileAt at{};
    lower(t, at.i, at.j);
    at.settle();
    // whole slabs of 64 columns
    const uint32_t slabs = g.np / 64, k0 = slabs * part / g.parts * 64, k1 = slabs * (part + 1) / g.parts * 64;
    const uint16_t* x = g.xh + (uint64_t)z * g.mp * g.np + k0;
    Core64 c;
    c.run(rows_of(x, at.i * 64, g.np, 64), rows_of(x, at.j * 64, g.np, 64), (k1 - k0) * 2, lds);
    tf32x4* o = (tf32x4*)(g.sums + ((uint64_t)zp * tiles + t) * 4096) + threadIdx.x;
#pragma unroll
    for (int u = 0; u < Core64::TP; ++u)
#pragma unroll
        for (int v = 0; v < Core64::TQ; ++v) o[(u * Core64::TQ + v) * Core64::NT] = c.acc[u][v];
}
__global__ __launch_bounds__(Core64::NT) void gram_join_kernel(GramSplit g, const DevState* st) {
    if (skipped(st)) return;
    __shared__ __attribute__((aligned(16))) uint8_t lds[room<Core64>()];
    const uint32_t side = g.mp / 64, tiles = side * (side + 1) / 2;
    const uint32_t t = blockIdx.x % tiles, z = blockIdx.x / tiles;
    TileAt at{};
    lower(t, at.i, at.j);
    at.i *= 64;
    at.j *= 64;
    at.settle();
    Core64 c;
#pragma unroll
    for (int u = 0; u < Core64::TP; ++u)
#pragma unroll
        for (int v = 0; v < Core64::TQ; ++v) c.acc[u][v] = tf32x4{0, 0, 0, 0};
    for (uint32_t part = 0; part < g.parts; ++part) {
        const tf32x4* o = (const tf32x4*)(g.sums + (((uint64_t)z * g.parts + part) * tiles + t) * 4096) + threadIdx.x;
#pragma unroll
        for (int u = 0; u < Core64::TP; ++u)
#pragma unroll
            for (int v = 0; v < Core64::TQ; ++v) c.acc[u][v] = c.acc[u][v] + o[(u * Core64::TQ + v) * Core64::NT];
    }
#pragma unroll
    for (int u = 0; u < Core64::TP; ++u)
#pragma unroll
        for (int v = 0; v < Core64::TQ; ++v) c.acc[u][v] = c.acc[u][v] * g.inv_s2;
    store_sym<Core64>(Piece<Core64>(at, 0, lds), c.acc, 0, g.out.a + (uint64_t)z * g.mp * g.mp, g.mp,
                      g.out.d + (uint64_t)z * g.mp, [](uint32_t) { return 0.0f; });
}

// Products of symmetric buffers: R = ka I + kb L + kc L L (SAME), or R = L M for L and M that
// commute.  With L = O + D, M = N + E (diagonals apart): L M = O N + D_i N_ij + O_ij E_j, and
// D_i E_i on the diagonal, where O and N are 0.
template <bool SAME>
struct Sym {
    static constexpr bool SYM = true;
    SymBuf l, m, r;
    uint32_t mp, np;
    float ka, kb, kc;
    template <class Core>
    __device__ __forceinline__ void tile(const TileAt& at, uint8_t* lds) const {
        using P = Piece<Core>;
        const uint64_t sz = (uint64_t)at.z * mp * mp, dz = (uint64_t)at.z * mp;
        const uint16_t *lo = l.a + sz, *mo = SAME ? lo : m.a + sz;
        const float *ld = l.d + dz, *md = SAME ? ld : m.d + dz;
        auto fetch = [&](const P& p) {
            P::Down::load(p.l0, lo + (uint64_t)p.j * mp + p.i, mp);
            if (!SAME) P::Down::load(p.l1, mo + (uint64_t)p.j * mp + p.i, mp);
        };
        Core t;
        if constexpr (P::kEarly) fetch(P(at, 0, lds));
        t.run(rows_of(lo, at.i, mp, Core::BP), rows_of(mo, at.j, mp, Core::BQ), mp * 2, lds);
#pragma unroll
        for (int u0 = 0; u0 < Core::TP; u0 += P::kU) {
            const P p(at, u0, lds);
            if constexpr (!P::kEarly) fetch(p);
            tf32x4 dd[P::kU];
            float ee[P::kV];
#pragma unroll
            for (int u = 0; u < P::kU; ++u) dd[u] = *(const tf32x4*)(ld + p.i + 16 * u + p.li);
#pragma unroll
            for (int v = 0; v < P::kV; ++v) ee[v] = md[p.j + 16 * v + p.lj];
            if constexpr (!P::kEarly) wave_wait();
#pragma unroll
            for (int u = 0; u < P::kU; ++u) {
                const tf32x4 di = dd[u];
#pragma unroll
                for (int v = 0; v < P::kV; ++v) {
                    const float ej = ee[v];
                    const f16x4 o = *p.down(p.l0, u, v);
                    tf32x4& y = t.acc[u0 + u][v];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float oe = (float)o[e];
                        y[e] = SAME ? __builtin_fmaf(kc, __builtin_fmaf(di[e] + ej, oe, y[e]), kb * oe)
                                    : __builtin_fmaf(ej, oe, y[e]);
                    }
                    if (!SAME) {
                        const f16x4 n = *p.down(p.l1, u, v);
#pragma unroll
                        for (int e = 0; e < 4; ++e) y[e] = __builtin_fmaf(di[e], (float)n[e], y[e]);
                    }
                }
            }
            store_sym<Core>(p, t.acc, u0, r.a + sz, mp, r.d + dz, [&](uint32_t i) {
                const float d = ld[i], dd = d * md[i];
                return SAME ? __builtin_fmaf(kc, dd, __builtin_fmaf(kb, d, ka)) : dd;
            });
            if (u0 + P::kU < Core::TP) wave_wait();      // the next load overwrites the patches
        }
    }
};

// X <- B X, B in a symmetric buffer, to the iterate's buffers of the next step.  B's diagonal
// meets both halves of X, the rest of it the first.
struct Apply {
    static constexpr bool SYM = false;
    SymBuf by;
    const uint16_t* xin;       // X^T before
    uint16_t *xout, *xrow, *rest;   // X^T after, X, X^T's second half
    uint32_t mp, np;
    template <class Core>
    __device__ __forceinline__ void tile(const TileAt& at, uint8_t* lds) const {
        using P = Piece<Core>;
        const uint64_t xz = (uint64_t)at.z * mp * np;
        const uint16_t* b = by.a + (uint64_t)at.z * mp * mp;
        const uint16_t* xt = xin + xz;
        auto fetch = [&](const P& p) {
            const uint64_t down = xz + (uint64_t)p.j * mp + p.i;
            P::Down::load(p.l0, xin + down, mp);
            P::Down::load(p.l1, rest + down, mp);
        };
        Core t;
        if constexpr (P::kEarly) fetch(P(at, 0, lds));
        t.run(rows_of(b, at.i, mp, Core::BP), rows_of(xt, at.j, mp, Core::BQ), mp * 2, lds);
        const float* db = by.d + (uint64_t)at.z * mp;
#pragma unroll
        for (int u0 = 0; u0 < Core::TP; u0 += P::kU) {
            const P p(at, u0, lds);
            const uint64_t down = xz + (uint64_t)p.j * mp + p.i;
            if constexpr (!P::kEarly) fetch(p);
            tf32x4 dd[P::kU];
#pragma unroll
            for (int u = 0; u < P::kU; ++u) dd[u] = *(const tf32x4*)(db + p.i + 16 * u + p.li);
            if constexpr (!P::kEarly) wave_wait();
#pragma unroll
            for (int u = 0; u < P::kU; ++u) {
                const tf32x4 d = dd[u];
#pragma unroll
                for (int v = 0; v < P::kV; ++v) {
                    f16x4 *ph = p.down(p.l0, u, v), *pl = p.down(p.l1, u, v);
                    const f16x4 h = *ph, o = *pl;
                    tf32x4& y = t.acc[u0 + u][v];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        y[e] = __builtin_fmaf(d[e], __builtin_fmaf((float)o[e], 1.0f / kLo, (float)h[e]), y[e]);
                    const f16x4 nh = pack4(y);
                    f16x4 nl;
#pragma unroll
                    for (int e = 0; e < 4; ++e) nl[e] = (_Float16)((y[e] - (float)nh[e]) * kLo);
                    *ph = nh;
                    *pl = nl;
                }
            }
            P::Down::store(p.l0, xout + down, mp);
            P::Down::store(p.l1, rest + down, mp);
#pragma unroll
            for (int u = 0; u < P::kU; ++u)
#pragma unroll
                for (int v = 0; v < P::kV; ++v) *p.across(p.l0, u, v) = pack4(transposed(pack4(t.acc[u0 + u][v])));
            P::Across::store(p.l0, xrow + xz + (uint64_t)p.i * np + p.j, np);
            if (u0 + P::kU < Core::TP) wave_wait();
        }
    }
};

// What the last step's result becomes: four consecutive elements of a row at (r, c), the first
// `n` of them inside the matrix.
struct OrthDst {
    const OrthIO& io;
    uint64_t at;
    float f;
    bool vec;
    __device__ OrthDst(const OrthIO& i, const NsShape&, uint32_t z, float inv_s)
        : io(i), at(z * i.dst_stride), f(i.scale * inv_s), vec(i.vec) {}
    __device__ __forceinline__ void store(uint32_t r, uint32_t c, uint32_t n, tf32x4 x) const {
        const uint64_t p = at + r * io.dst_ld + c;
        if (vec && n == 4) {
            x = x * f;
            if (io.dst_dtype == NEOX_F32) *(tf32x4*)((float*)io.dst + p) = x;
            else *(ushort4*)((uint16_t*)io.dst + p) =
                     make_ushort4(float_to_half(io.dst_dtype, x[0]), float_to_half(io.dst_dtype, x[1]),
                                  float_to_half(io.dst_dtype, x[2]), float_to_half(io.dst_dtype, x[3]));
        } else {
#pragma unroll
            for (uint32_t e = 0; e < 4; ++e)
                if (e < n) store_elem(io.dst, io.dst_dtype, p + e, x[e] * f);
        }
    }
};
struct MuonDst {
    const MuonIO& io;
    MuonMat mat;
    uint32_t cols;
    float f, wd;
    bool vec;
    __device__ MuonDst(const MuonIO& i, const NsShape& s, uint32_t z, float inv_s)
        : io(i), mat(i.mats[z]), cols(s.cols), f(i.scale * inv_s), wd(mat.decay ? i.wd : 0.0f),
          vec(mat.vec && s.cols % 4 == 0) {}
    __device__ __forceinline__ float step(float w, float x) const {
        return opaque(__builtin_fmaf(-io.lr, __builtin_fmaf(wd, w, x * f), w));
    }
    __device__ __forceinline__ void store(uint32_t r, uint32_t c, uint32_t n, tf32x4 x) const {
        const uint64_t p = (uint64_t)r * cols + c;
        if (vec && n == 4) {
            tf32x4 w = *(const tf32x4*)(mat.master + p);
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = step(w[e], x[e]);
            *(tf32x4*)(mat.master + p) = w;
            *(ushort4*)(mat.half + p) = make_ushort4(float_to_half(io.dtype, w[0]), float_to_half(io.dtype, w[1]),
                                                     float_to_half(io.dtype, w[2]), float_to_half(io.dtype, w[3]));
        } else {
#pragma unroll
            for (uint32_t e = 0; e < 4; ++e)
                if (e < n) {
                    const float w = step(mat.master[p + e], x[e]);
                    mat.master[p + e] = w;
                    mat.half[p + e] = float_to_half(io.dtype, w);
                }
        }
    }
};

// The last step.  The operands are exchanged where the source is not transposed, so that a
// lane's four elements always are neighbours in a row of the source (a column of D): there D's
// rows are j and its columns i, the iterate's first half comes from xh and its second,
// transposed, from lt.
template <class IO, class Dst, bool TALL>
struct Last {
    static constexpr bool SYM = false;
    IO io;
    SymBuf by;
    const uint16_t *xin, *xrow, *rest;
    NsShape s;
    float inv_s;
    template <class Core>
    __device__ __forceinline__ void tile(const TileAt& at, uint8_t* lds) const {
        const uint32_t mp = s.mp, np = s.np;
        const uint64_t xz = (uint64_t)at.z * mp * np;
        const uint16_t* b = by.a + (uint64_t)at.z * mp * mp;
        const uint16_t* xt = xin + xz;
        const uint16_t* xh = xrow + xz;
        const uint16_t* lt = rest + xz;
        const float* db = by.d + (uint64_t)at.z * mp;
        const TileRows br = rows_of(b, TALL ? at.i : at.j, mp, TALL ? Core::BP : Core::BQ);
        const TileRows xr = rows_of(xt, TALL ? at.j : at.i, mp, TALL ? Core::BQ : Core::BP);
        using P = Piece<Core>;
        auto fetch = [&](const P& p) {
            if constexpr (TALL) {
                // D rows are i: four i of one j
                P::Down::load(p.l0, xt + (uint64_t)p.j * mp + p.i, mp);
                P::Down::load(p.l1, lt + (uint64_t)p.j * mp + p.i, mp);
            } else {
                // D rows (p.i) are j and its columns (p.j) are i: four j of one i
                P::Down::load(p.l0, xh + (uint64_t)p.j * np + p.i, np);
                P::Across::load(p.l1, lt + (uint64_t)p.i * mp + p.j, mp);
            }
        };
        Core t;
        if constexpr (P::kEarly) fetch(P(at, 0, lds));
        t.run(TALL ? br : xr, TALL ? xr : br, mp * 2, lds);
        const Dst dst(io, s, at.z, inv_s);
#pragma unroll
        for (int u0 = 0; u0 < Core::TP; u0 += P::kU) {
            const P p(at, u0, lds);
            if constexpr (!P::kEarly) {
                fetch(p);
                wave_wait();
            }
#pragma unroll
            for (int u = 0; u < P::kU; ++u) {
                const uint32_t i = p.i + 16 * u + p.li;
                const tf32x4 di = TALL ? *(const tf32x4*)(db + i) : tf32x4{0, 0, 0, 0};
#pragma unroll
                for (int v = 0; v < P::kV; ++v) {
                    const f16x4 h = *p.down(p.l0, u, v);
                    tf32x4 o;
                    if constexpr (TALL) {
                        const f16x4 q = *p.down(p.l1, u, v);
                        o = tf32x4{(float)q[0], (float)q[1], (float)q[2], (float)q[3]};
                    } else {
                        o = transposed(*p.across(p.l1, u, v));
                    }
                    const float dj = TALL ? 0.0f : db[p.j + 16 * v + p.lj];
                    tf32x4& y = t.acc[u0 + u][v];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        y[e] = __builtin_fmaf(TALL ? di[e] : dj, __builtin_fmaf(o[e], 1.0f / kLo, (float)h[e]), y[e]);
                }
            }
            // the source's rows (D's columns) through LDS: 128 or 256 bytes of a row at a time
            // instead of 64 (four lanes)
            constexpr uint32_t kRow = 16 * P::kU * 4, kChunks = kRow / 16, kRows = 16 * P::kV;
            static_assert(kRows * kRow <= 2 * P::kBytes, "the two patches' place");
#pragma unroll
            for (int u = 0; u < P::kU; ++u)
#pragma unroll
                for (int v = 0; v < P::kV; ++v) {
                    const uint32_t row = 16 * v + p.lj, c = (16 * u + p.li) / 4;
                    *(tf32x4*)(p.l0 + row * kRow + ((c ^ (row % kChunks)) << 4)) = t.acc[u0 + u][v];
                }
            const uint32_t rows = TALL ? s.n : s.m, cols = TALL ? s.m : s.n, lane = threadIdx.x & 63;
#pragma unroll 4
            for (uint32_t k = lane; k < kRows * kChunks; k += 64) {
                const uint32_t row = k / kChunks, c = (k % kChunks) ^ (row % kChunks);
                const uint32_t r = p.j + row, q = p.i + 4 * c;
                const tf32x4 y = *(const tf32x4*)(p.l0 + k * 16);
                if (r < rows && q < cols) dst.store(r, q, min(4u, cols - q), y);
            }
            if (u0 + P::kU < Core::TP) wave_wait();
        }
    }
};

using Core256 = TileCore<256, 256, 2, 4, false>;
using Core128 = TileCore<128, 128, 2, 4, false>;       // (quarters are by the same 512 threads)
using Core64q = TileCore<64, 64, 4, 2, false, 4>;      // quarters of those
using Core32 = TileCore<32, 32, 2, 2, false, 4>;

// (two blocks of 128 x 128 tiles share a CU, and so a SIMD's registers four waves)
template <class Op, class Full, class Quarter>
__global__ __launch_bounds__(Full::NT, Full::BP == 256 ? 2 : 4) void ns_mixed_kernel(Op op, const DevState* st, TileMap m) {
    static_assert(Full::NT == Quarter::NT && Full::kLds >= Quarter::kLds && Full::BP == 2 * Quarter::BP, "");
    if (skipped(st)) return;
    __shared__ __attribute__((aligned(16))) uint8_t lds[room<Full>() > room<Quarter>() ? room<Full>() : room<Quarter>()];
    const TileAt at = place<Op::SYM>(m);
    if (at.full) op.template tile<Full>(at, lds);
    else if (!at.none) op.template tile<Quarter>(at, lds);
}
template <class Op, class Core>
__global__ __launch_bounds__(Core::NT) void ns_even_kernel(Op op, const DevState* st, uint32_t mp, uint32_t np) {
    if (skipped(st)) return;
    __shared__ __attribute__((aligned(16))) uint8_t lds[room<Core>()];
    op.template tile<Core>(place_even<Core, Op::SYM>(mp, np), lds);
}

// ------------------------------------------------------------------------------------
// Small matrices: everything in one launch, one block per matrix
//
// Up to 128 x 128 (or 64 x 256) the iterate in both orientations, A and B fit one CU's LDS and
// the iterate itself, in FP32, the block's registers.  The fifteen launches of the tiled form
// would each wait for the one before (66 us for 64 matrices of 64 x 64; here 11.7 in one
// launch).  Bound by latency and by how fast a wave issues: five steps of three products with
// a barrier behind each; up to 256 matrices take the same time.
// ------------------------------------------------------------------------------------
struct NsSteps {
    int32_t n;
    NsCoef c[NEOX_NS_MAX_STEPS];
};

// Rows of B bytes in LDS, their 16-byte chunks permuted by the row's number.
template <int B>
__device__ __forceinline__ uint8_t* chunk_at(uint8_t* base, uint32_t row, uint32_t chunk) {
    return base + row * B + ((chunk ^ (row & 7)) << 4);
}
// the place of elements (row, col .. col + 3)
template <int B>
__device__ __forceinline__ f16x4* quad_at(uint8_t* base, uint32_t row, uint32_t col) {
    return (f16x4*)(chunk_at<B>(base, row, col >> 3) + (col & 4) * 2);
}

// acc += P Q^T over rows of B bytes
template <int TP, int TQ, int B>
__device__ __forceinline__ void lds_product(tf32x4 (&acc)[TP][TQ], uint8_t* p, uint32_t prow, uint8_t* q, uint32_t qrow) {
    const uint32_t lane = threadIdx.x & 63, l16 = lane & 15, g = lane >> 4;
#pragma unroll
    for (int u = 0; u < TP; ++u)
#pragma unroll
        for (int v = 0; v < TQ; ++v) acc[u][v] = tf32x4{0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < B / 64; ++k) {
        tf16x8 a[TP], b[TQ];
#pragma unroll
        for (int u = 0; u < TP; ++u) a[u] = *(const tf16x8*)chunk_at<B>(p, prow + 16 * u + l16, 4 * k + g);
#pragma unroll
        for (int v = 0; v < TQ; ++v) b[v] = *(const tf16x8*)chunk_at<B>(q, qrow + 16 * v + l16, 4 * k + g);
#pragma unroll
        for (int u = 0; u < TP; ++u)
#pragma unroll
            for (int v = 0; v < TQ; ++v) acc[u][v] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[u], b[v], acc[u][v], 0, 0, 0);
    }
}

// The source's elements (r, c .. c + n - 1), n <= 4; Muon's momentum is updated on the way.
struct OrthIn {
    OrthSrc src;
    __device__ OrthIn(const OrthIO& io, const NsShape& s, uint32_t z) : src(io, s, z) {}
    __device__ tf32x4 get(uint32_t r, uint32_t c, uint32_t n, uint32_t cols) const {
        if (src.vec) return src.load4(r, c, cols);
        tf32x4 x = {0, 0, 0, 0};
#pragma unroll
        for (uint32_t e = 0; e < 4; ++e)
            if (e < n) x[e] = src.load(r, c + e, cols);
        return x;
    }
};
struct MuonIn {
    MuonSrc src;
    __device__ MuonIn(const MuonIO& io, const NsShape& s, uint32_t z) : src(io, s, z) {}
    __device__ tf32x4 get(uint32_t r, uint32_t c, uint32_t n, uint32_t cols) const {
        const uint64_t at = (uint64_t)r * cols + c;
        tf32x4 x = {0, 0, 0, 0};
        if (src.vec) {
            const tf32x4 g = halves4(src.io.dtype, *(const uint2*)(src.mat.grad + at));
            tf32x4 m = *(const tf32x4*)(src.mat.mom + at);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                m[e] = __builtin_fmaf(src.io.mu, m[e], g[e] * src.gs);
                x[e] = direction(src.io, g[e] * src.gs, m[e]);
            }
            *(tf32x4*)(src.mat.mom + at) = m;
        } else {
#pragma unroll
            for (uint32_t e = 0; e < 4; ++e)
                if (e < n) {
                    const float g = half_to_float(src.io.dtype, src.mat.grad[at + e]) * src.gs;
                    const float m = __builtin_fmaf(src.io.mu, src.mat.mom[at + e], g);
                    src.mat.mom[at + e] = m;
                    x[e] = direction(src.io, g, m);
                }
        }
        return x;
    }
};

// A 16 x 16 result tile on the diagonal: the diagonal to d[0 .. 15], zeros in its place.
__device__ __forceinline__ void take_diagonal(tf32x4& x, float* d) {
    const uint32_t lane = threadIdx.x & 63, l16 = lane & 15;
    if (l16 / 4 != lane >> 4) return;
#pragma unroll
    for (uint32_t e = 0; e < 4; ++e)
        if (l16 % 4 == e) {
            d[l16] = x[e];
            x[e] = 0.0f;
        }
}

template <class IO, class In, class Dst, int MP, int NP, int WP, int WQ>
__global__ __launch_bounds__(WP * WQ * 64) void ns_small_kernel(IO io, NsShape s, NsSteps steps) {
    if (skipped(state_of(io))) return;
    constexpr int NT = WP * WQ * 64;
    constexpr int XB = NP * 2, TB = MP * 2;            // bytes of a row of X, and of X^T, A and B
    constexpr int kX = MP * XB, kA = MP * TB;
    constexpr int PF = NP + 1;                         // floats of a row of the FP32 buffer
    constexpr int kF = MP * PF * 4 > 2 * kA ? MP * PF * 4 : 2 * kA;
    __shared__ __attribute__((aligned(16))) uint8_t lds[2 * kX + kF + 2 * MP * 4];
    uint8_t *xh = lds, *xt = lds + kX, *la = lds + 2 * kX, *lb = la + kA;
    float* f32 = (float*)la;                           // source and result, in A's and B's place
    float *da = (float*)(lds + 2 * kX + kF), *db = da + MP;
    const uint32_t z = blockIdx.x, tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, g = lane >> 4;

    // the source into LDS in its wide form, its norm on the way
    const In in(io, s, z);
    const uint32_t w4 = (s.cols + 3) / 4;
    double sq = 0.0;
    for (uint32_t k = tid; k < s.rows * w4; k += NT) {
        const uint32_t r = k / w4, c = (k - r * w4) * 4, n = min(4u, s.cols - c);
        const tf32x4 x = in.get(r, c, n, s.cols);
        sq = square4(x, sq);
#pragma unroll
        for (uint32_t e = 0; e < 4; ++e)
            if (e < n) f32[s.tall ? (c + e) * PF + r : r * PF + c + e] = x[e];
    }
    sq = sum_block<NT>(sq);                            // (a barrier)
    const double f = (double)s.s / (__builtin_sqrt(sq) + io.eps);

    // X: this wave's part, four rows of a column a lane as everywhere
    constexpr int TP = MP / WP / 16, TQ = NP / WQ / 16, SQ = MP / WQ / 16;
    const uint32_t wave = tid >> 6;
    const uint32_t pi = wave / WQ * (MP / WP), qj = wave % WQ * (NP / WQ), qs = wave % WQ * (MP / WQ);
    tf32x4 x[TP][TQ];
    auto spread_x = [&]() {
#pragma unroll
        for (int u = 0; u < TP; ++u)
#pragma unroll
            for (int v = 0; v < TQ; ++v) {
                const f16x4 h = pack4(x[u][v]);
                *quad_at<TB>(xt, qj + 16 * v + l16, pi + 16 * u + 4 * g) = h;
                *quad_at<XB>(xh, pi + 16 * u + l16, qj + 16 * v + 4 * g) = pack4(transposed(h));
            }
    };
#pragma unroll
    for (int u = 0; u < TP; ++u)
#pragma unroll
        for (int v = 0; v < TQ; ++v)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t i = pi + 16 * u + 4 * g + e, j = qj + 16 * v + l16;
                x[u][v][e] = i < s.m && j < s.n ? (float)((double)f32[i * PF + j] * f) : 0.0f;
            }
    spread_x();
    __syncthreads();

    const float inv_s2 = 1.0f / (s.s * s.s);
    for (int k = 0; k < steps.n; ++k) {
        // A = X X^T, whole: its rows are written from its columns, which are the same
        tf32x4 a[TP][SQ];
        f16x4 o[TP][SQ];
        lds_product<TP, SQ, XB>(a, xh, pi, xh, qs);
#pragma unroll
        for (int u = 0; u < TP; ++u)
#pragma unroll
            for (int v = 0; v < SQ; ++v) {
                const uint32_t i = pi + 16 * u + 4 * g, j = qs + 16 * v + l16;
                a[u][v] = a[u][v] * inv_s2;
                if (pi + 16 * u == qs + 16 * v) take_diagonal(a[u][v], da + qs + 16 * v);
                o[u][v] = pack4(a[u][v]);
                *quad_at<TB>(la, j, i) = o[u][v];
            }
        __syncthreads();
        // B = b A + c A A (see Sym)
        lds_product<TP, SQ, TB>(a, la, pi, la, qs);
#pragma unroll
        for (int u = 0; u < TP; ++u)
#pragma unroll
            for (int v = 0; v < SQ; ++v) {
                const uint32_t i = pi + 16 * u + 4 * g, j = qs + 16 * v + l16;
                const tf32x4 di = *(const tf32x4*)(da + i);
                const float dj = da[j];
                tf32x4 b;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float off = (float)o[u][v][e];
                    b[e] = __builtin_fmaf(steps.c[k].c, __builtin_fmaf(di[e] + dj, off, a[u][v][e]), steps.c[k].b * off);
                }
                if (pi + 16 * u == qs + 16 * v) {
                    // on the diagonal O is 0 and D_i^2, b D_i and a are to be added
                    take_diagonal(b, db + qs + 16 * v);
                    if (l16 / 4 == g) {
                        const float more = __builtin_fmaf(steps.c[k].c * dj, dj, steps.c[k].b * dj) + steps.c[k].a;
                        db[j] += more;
                    }
                }
                *quad_at<TB>(lb, j, i) = pack4(b);
            }
        __syncthreads();
        // X <- a X + B X
        tf32x4 y[TP][TQ];
        lds_product<TP, TQ, TB>(y, lb, pi, xt, qj);
#pragma unroll
        for (int u = 0; u < TP; ++u) {
            const tf32x4 d = *(const tf32x4*)(db + pi + 16 * u + 4 * g);
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int v = 0; v < TQ; ++v) x[u][v][e] = __builtin_fmaf(d[e], x[u][v][e], y[u][v][e]);
        }
        __syncthreads();                               // everybody has read B and X^T
        if (k + 1 < steps.n) {
            spread_x();
            __syncthreads();
        }
    }

    // the result through LDS, to rows of the source's shape
#pragma unroll
    for (int u = 0; u < TP; ++u)
#pragma unroll
        for (int v = 0; v < TQ; ++v)
#pragma unroll
            for (int e = 0; e < 4; ++e) f32[(pi + 16 * u + 4 * g + e) * PF + qj + 16 * v + l16] = x[u][v][e];
    __syncthreads();
    const Dst dst(io, s, z, 1.0f / s.s);
    for (uint32_t k = tid; k < s.rows * w4; k += NT) {
        const uint32_t r = k / w4, c = (k - r * w4) * 4, n = min(4u, s.cols - c);
        tf32x4 v = {0, 0, 0, 0};
#pragma unroll
        for (uint32_t e = 0; e < 4; ++e)
            if (e < n) v[e] = f32[s.tall ? (c + e) * PF + r : r * PF + c + e];
        dst.store(r, c, n, v);
    }
}

template <class IO, class In, class Dst>
hipError_t launch_small(const NsShape& s, uint32_t count, const IO& io, const NsCoef* coef, int steps,
                        hipStream_t stream) {
    NsSteps st{};
    st.n = steps;
    for (int k = 0; k < steps; ++k) st.c[k] = coef[k];
    // Threads, us for 64 and for 2,000 matrices: 64 x 64 with 256 15.1 and 48, 512 11.7 and 48,
    // 1,024 11.1 and 54; 64 x 128 with 256 20.6 and 96, 512 15.8 and 77, 1,024 14.6 and 107; 64 x
    // 256 with 512 23.9 and 199, 1,024 21.8 and 175; 128 x 128 with 512 33.8 and 281, 1,024 32.2
    // and 261.  (Not by the number of matrices: the order of the norm's sum goes with it.)
    if (s.m > 64) ns_small_kernel<IO, In, Dst, 128, 128, 4, 4><<<count, 1024, 0, stream>>>(io, s, st);
    else if (s.n > 128) ns_small_kernel<IO, In, Dst, 64, 256, 4, 4><<<count, 1024, 0, stream>>>(io, s, st);
    else if (s.n > 64) ns_small_kernel<IO, In, Dst, 64, 128, 2, 4><<<count, 512, 0, stream>>>(io, s, st);
    else ns_small_kernel<IO, In, Dst, 64, 64, 2, 4><<<count, 512, 0, stream>>>(io, s, st);
    return hipGetLastError();
}

// ------------------------------------------------------------------------------------
// launches
// ------------------------------------------------------------------------------------
// One product over `count` matrices with mp x np results (mp = np for the symmetric ones).
// The tiles are chosen by what the launch would take per 128 bytes of K, from times measured on
// the full chip (us per slab): a round of 256 x 256 tiles (one block a CU) 1.45, of 128 x 128
// ones 0.5 (two blocks on a CU take twice that; by 8 waves, 8 matrices of 4096 x 1024 are
// orthogonalised in 769 us, by 4 waves in 786), of quarters of those 0.24; 64 x 64 tiles 0.23
// where each CU has one, 0.2 a round otherwise.  Few tiles take a block's own time, which goes
// by the bytes it loads and the instructions a wave issues: 32 x 32 tiles of four waves while a
// CU has at most two of them (387 x 1001 orthogonalised in 91 us, 98 with one wave a tile, 106
// with 64 x 64 ones; with up to four a CU 1000 x 1000 takes 136 us instead of 118).  Results
// do not depend on the choice: every element's products are added in the same order, and
// store_sym mirrors what lies below the diagonal.
template <class Op>
hipError_t launch_product(const Op& op, const DevState* st, uint32_t mp, uint32_t np, uint32_t count,
                          hipStream_t stream) {
    const uint64_t p64 = mp / 64, q64 = np / 64;
    const uint64_t n64 = (Op::SYM ? p64 * (p64 + 1) / 2 : p64 * q64) * count;
    const double c64 = n64 <= kCUs ? 0.23 : 0.2 * (double)((n64 + kCUs - 1) / kCUs);
    double c128 = 0.0, c256 = 1e300;
    uint64_t b128 = 0, b256 = 0;
    TileMap m256{};
    const TileMap m128 = plan_tiles(128, Op::SYM, mp, np, count, 0.5, 0.24, &c128, &b128);
    // quarters of the large tile are not cut
    if (mp % 128 == 0 && np % 128 == 0)
        m256 = plan_tiles(256, Op::SYM, mp, np, count, 1.45, 0.5, &c256, &b256);
    const uint64_t p32 = mp / 32, q32 = np / 32, n32 = (Op::SYM ? p32 * (p32 + 1) / 2 : p32 * q32) * count;
    if (n32 <= 2 * kCUs)
        ns_even_kernel<Op, Core32><<<(uint32_t)n32, Core32::NT, 0, stream>>>(op, st, mp, np);
    else if (c64 <= c128 && c64 <= c256)
        ns_even_kernel<Op, Core64><<<(uint32_t)n64, Core64::NT, 0, stream>>>(op, st, mp, np);
    else if (c128 < c256)
        ns_mixed_kernel<Op, Core128, Core64q><<<(uint32_t)b128, Core128::NT, 0, stream>>>(op, st, m128);
    else
        ns_mixed_kernel<Op, Core256, Core128><<<(uint32_t)b256, Core256::NT, 0, stream>>>(op, st, m256);
    return hipGetLastError();
}

template <class IO, class Src, class Dst>
hipError_t enqueue_steps(const NsShape& s, const NsBuf& w, uint32_t count, const IO& io,
                         const NsCoef* coef, int steps, hipStream_t stream) {
    const uint32_t conv = s.mp / 64 * (s.np / 64) * count;
    ns_convert_kernel<Src><<<conv, 256, 0, stream>>>(io, s, w);
    hipError_t e = hipGetLastError();
    const DevState* st = state_of(io);
    const float inv_s2 = 1.0f / (s.s * s.s), inv_s = 1.0f / s.s;
    int from = 0;
    SymBuf y[3];
    for (int k = 0; k < 3; ++k) y[k] = SymBuf{w.sym[k], w.diag[k]};
    // the products of Sym, by buffer
    auto sym = [&](int l, int m, int r, float ka, float kb, float kc) {
        if (e != hipSuccess) return;
        e = l == m ? launch_product(Sym<true>{y[l], y[m], y[r], s.mp, s.np, ka, kb, kc}, st, s.mp, s.mp, count, stream)
                   : launch_product(Sym<false>{y[l], y[m], y[r], s.mp, s.np, ka, kb, kc}, st, s.mp, s.mp, count, stream);
    };
    for (int k = 0; k < steps && e == hipSuccess;) {
        if (s.split > 1) {
            const GramSplit g{w.xh, y[0], w.sums, s.mp, s.np, s.split, inv_s2};
            const uint32_t tiles = s.mp / 64 * (s.mp / 64 + 1) / 2 * count;
            gram_part_kernel<<<tiles * s.split, Core64::NT, 0, stream>>>(g, st);
            e = hipGetLastError();
            if (e == hipSuccess) {
                gram_join_kernel<<<tiles, Core64::NT, 0, stream>>>(g, st);
                e = hipGetLastError();
            }
        } else {
            e = launch_product(Gram{w.xh, y[0], s.mp, s.np, inv_s2}, st, s.mp, s.mp, count, stream);
        }
        int by = 1;
        sym(0, 0, 1, coef[k].a, coef[k].b, coef[k].c);             // P = a I + b A + c A A
        if (s.pairs && k + 1 < steps) {
            sym(1, 0, 2, 0.0f, 0.0f, 1.0f);                        // P A
            sym(2, 1, 0, 0.0f, 0.0f, 1.0f);                        // A of the next step: P A P
            sym(0, 0, 2, coef[k + 1].a, coef[k + 1].b, coef[k + 1].c);
            sym(2, 1, 0, 0.0f, 0.0f, 1.0f);                        // both steps' P
            by = 0;
            ++k;
        }
        ++k;
        if (e != hipSuccess) break;
        if (k < steps)
            e = launch_product(Apply{y[by], w.xt[from], w.xt[from ^ 1], w.xh, w.lt, s.mp, s.np}, st, s.mp, s.np, count, stream);
        else if (s.tall)
            e = launch_product(Last<IO, Dst, true>{io, y[by], w.xt[from], w.xh, w.lt, s, inv_s}, st, s.mp, s.np, count, stream);
        else
            e = launch_product(Last<IO, Dst, false>{io, y[by], w.xt[from], w.xh, w.lt, s, inv_s}, st, s.np, s.mp, count, stream);
        from ^= 1;
    }
    return e;
}

}  // namespace

hipError_t enqueue_orth(const NsShape& s, const NsBuf& w, uint32_t count, const OrthIO& io,
                        const NsCoef* coef, int steps, hipStream_t stream) {
    if (s.small) return launch_small<OrthIO, OrthIn, OrthDst>(s, count, io, coef, steps, stream);
    orth_norm_kernel<<<s.parts * count, kNormThreads, 0, stream>>>(io, s.rows, s.cols, s.parts, w.part);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    return enqueue_steps<OrthIO, OrthSrc, OrthDst>(s, w, count, io, coef, steps, stream);
}

hipError_t enqueue_muon(const NsShape& s, const NsBuf& w, uint32_t count, const MuonIO& io,
                        const NsCoef* coef, int steps, hipStream_t stream) {
    if (s.small) return launch_small<MuonIO, MuonIn, MuonDst>(s, count, io, coef, steps, stream);
    const uint64_t numel = (uint64_t)s.rows * s.cols;
    muon_momentum_kernel<<<s.parts * count, kNormThreads, 0, stream>>>(io, numel, s.parts, w.part);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    return enqueue_steps<MuonIO, MuonSrc, MuonDst>(s, w, count, io, coef, steps, stream);
}

// ------------------------------------------------------------------------------------
// shapes
// ------------------------------------------------------------------------------------
NsShape ns_shape(uint64_t rows, uint64_t cols, bool pairs) {
    NsShape s{};
    s.rows = (uint32_t)rows;
    s.cols = (uint32_t)cols;
    s.tall = rows > cols;
    s.m = s.tall ? s.cols : s.rows;
    s.n = s.tall ? s.rows : s.cols;
    // whole 64 x 64 tiles where the small side has few of them, else whole 128 x 128 ones
    const uint32_t t = s.m <= 512 ? 64 : 128;
    s.mp = (s.m + t - 1) / t * t;
    s.np = (s.n + t - 1) / t * t;
    s.small = (s.m <= 128 && s.n <= 128) || (s.m <= 64 && s.n <= 256);
    // Shares of X X^T's sums: enough blocks for the chip where there are few tiles, eight slabs
    // of 64 columns or more in each, and only where it saves more than the second launch takes
    // (by the shape alone: the order of the sums must not depend on the batch)
    const uint32_t tiles = s.mp / 64 * (s.mp / 64 + 1) / 2, slabs = s.np / 64;
    s.split = 1;
    if (s.m <= 512 && slabs >= 32) s.split = std::min(std::min(16u, slabs / 8), (96 + tiles - 1) / tiles);
    s.pairs = pairs && s.m > 512 && s.n >= 2 * s.m;
    // one partial sum for each 16K elements, at most one for each row
    const uint64_t want = (rows * cols + 16383) / 16384;
    s.parts = (uint32_t)(want < kNsParts ? want : kNsParts);
    if (s.parts > s.rows) s.parts = s.rows;
    // S = 2^round(log2(n) / 2): the rows of the result have norm ~1, so its elements are
    // ~1 / sqrt(n) and times S of order 1, far from FP16's ends
    uint32_t lg = 0;
    while ((1ull << (lg + 1)) <= s.n) ++lg;
    s.s = (float)(1u << ((lg + 1) / 2));
    return s;
}

static uint64_t up256(uint64_t x) { return (x + 255) & ~255ull; }
static uint64_t split_bytes(const NsShape& s) {
    return s.split > 1 ? 4096ull * 4 * (s.mp / 64) * (s.mp / 64 + 1) / 2 * s.split : 0;
}

NsBuf ns_place(const NsShape& s, uint64_t count, void* base) {
    uint8_t* p = (uint8_t*)base;
    auto take = [&](uint64_t bytes) {
        uint8_t* r = p;
        p += up256(bytes);
        return r;
    };
    const uint64_t x = 2ull * s.mp * s.np * count, a = 2ull * s.mp * s.mp * count;
    NsBuf w{};
    w.xh = (uint16_t*)take(x);
    w.xt[0] = (uint16_t*)take(x);
    w.xt[1] = (uint16_t*)take(x);
    w.lt = (uint16_t*)take(x);
    for (int k = 0; k < (s.pairs ? 3 : 2); ++k) {
        w.sym[k] = (uint16_t*)take(a);
        w.diag[k] = (float*)take(4ull * s.mp * count);
    }
    w.part = (double*)take(8ull * kNsParts * count);
    if (s.split > 1) w.sums = (float*)take(split_bytes(s) * count);
    return w;
}

uint64_t ns_bytes(const NsShape& s, uint64_t count) {
    const uint64_t x = 2ull * s.mp * s.np * count, a = 2ull * s.mp * s.mp * count;
    return 4 * up256(x) + (s.pairs ? 3 : 2) * (up256(a) + up256(4ull * s.mp * count)) + up256(8ull * kNsParts * count) +
           up256(split_bytes(s) * count);
}

}  // namespace nz1
