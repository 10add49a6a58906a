// matrix_kernels.hip -- Newton-Schulz orthogonalisation and the Muon update on gfx950.
//
// For each step, with X m x n (m <= n):
//   gram   A = X X^T                       symmetric: tiles on and below the diagonal only
//   poly   B = b A + c A A                 symmetric, as A is (A A = A A^T)
//   apply  X <- a X + B X
// All three are products of rows with rows once X is kept in both orientations, so they
// share one tile core.
//
// Precision.  Products read FP16.  Rounding the iterate itself to FP16 in each step would
// put noise into the directions whose singular values are still tiny, and a later step
// multiplies those by up to a (3.4 per step, ~500 in five): a rank-1 matrix came out 15%
// off.  So X is carried as two FP16 numbers (22 bits), and only the products B X and X X^T
// see the first alone: their error is filtered through B or X once more and stays at the
// FP16 level.  A and B have diagonals far larger than the rest (of similar size along the
// diagonal too, so that their roundings would add up in one direction): the diagonals are
// kept in FP32, apart, and FP16 holds the rest.  Simulated against 64 bits on Gaussian,
// decaying and low-rank spectra: 2e-4 .. 1e-3 of the result's norm.
#include "matrix_internal.h"
#include "tile_core.h"

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

// Four or eight consecutive elements, as one or two 16-byte loads (8 bytes for four halves).
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
// matrix still has a block on every CU with two vectors in flight a thread.
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
    if (io.vec_src && cols % 4 == 0) {
        // this block's rows as one run of vectors, two in flight
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
        while (r < r1) {
            const tf32x4 v = vec4(io.src, io.src_dtype, at + r * io.src_ld + 4 * c);
            next();
            if (r < r1) {
                const tf32x4 q = vec4(io.src, io.src_dtype, at + r * io.src_ld + 4 * c);
                t = square4(q, t);
            }
            s = square4(v, s);
            next();
        }
    } else {
        for (uint32_t r = r0; r < r1; ++r)
            for (uint32_t c = threadIdx.x; c < cols; c += kNormThreads) {
                const double x = load_elem(io.src, io.src_dtype, at + r * io.src_ld + c);
                s = __builtin_fma(x, x, s);
            }
    }
    s = sum_block<kNormThreads>(s + t);
    if (threadIdx.x == 0) part[(uint64_t)z * kNsParts + p] = s;
}

__device__ __forceinline__ float direction(const MuonIO& io, float g, float m) {
    return io.nesterov ? __builtin_fmaf(io.mu, m, g) : m;
}

__global__ __launch_bounds__(kNormThreads) void muon_momentum_kernel(MuonIO io, uint64_t numel,
                                                                     uint32_t parts, double* __restrict__ part) {
    if (io.st->skip) return;
    const float gs = io.st->gscale;
    const uint32_t z = blockIdx.x / parts, p = blockIdx.x % parts;
    const MuonMat mat = io.mats[z];
    double s = 0.0;
    uint64_t done = 0;
    if (mat.vec) {
        const uint64_t n4 = numel / 4, step = (uint64_t)parts * kNormThreads;
        done = n4 * 4;
        for (uint64_t i = (uint64_t)p * kNormThreads + threadIdx.x; i < n4; i += 2 * step) {
            const uint64_t j = i + step < n4 ? i + step : i;        // the same again at the end
            tf32x4 g[2], m[2];
            g[0] = halves4(io.dtype, *(const uint2*)(mat.grad + 4 * i));
            g[1] = halves4(io.dtype, *(const uint2*)(mat.grad + 4 * j));
            m[0] = *(const tf32x4*)(mat.mom + 4 * i);
            m[1] = *(const tf32x4*)(mat.mom + 4 * j);
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
                *(tf32x4*)(mat.mom + 4 * (k ? j : i)) = m[k];
                s = square4(u, s);
            }
        }
    }
    for (uint64_t i = done + (uint64_t)p * kNormThreads + threadIdx.x; i < numel; i += (uint64_t)parts * kNormThreads) {
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
// The same for launches of one tile size only, one block per tile.
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
    return r;
}

__device__ __forceinline__ TileRows rows_of(const uint16_t* base, uint64_t row, uint32_t len, int block) {
    return TileRows{(const uint8_t*)(base + row * len), nullptr, (uint32_t)block, len * 2u, 0u};
}

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
// diagonal to d.
template <class Core>
__device__ __forceinline__ void store_sym(const TileAt& t, const Piece<Core>& p, tf32x4 (&x)[Piece<Core>::kU][Core::TQ],
                                          uint16_t* out, uint32_t ld, float* d) {
    using P = Piece<Core>;
#pragma unroll
    for (int u = 0; u < P::kU; ++u)
#pragma unroll
        for (int v = 0; v < P::kV; ++v) {
            if (t.i == t.j) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (p.i + 16 * u + p.li + e == p.j + 16 * v + p.lj) {
                        d[p.j + 16 * v + p.lj] = x[u][v][e];
                        x[u][v][e] = 0.0f;
                    }
            }
            const f16x4 h = pack4(x[u][v]);
            *p.down(p.l0, u, v) = h;
            *p.across(p.l1, u, v) = pack4(transposed(h));
        }
    if (t.i != t.j) P::Down::store(p.l0, out + (uint64_t)p.j * ld + p.i, ld);
    P::Across::store(p.l1, out + (uint64_t)p.i * ld + p.j, ld);
}

// A = X X^T
struct Gram {
    static constexpr bool SYM = true;
    NsBuf w;
    uint32_t mp, np;
    float inv_s2;
    template <class Core>
    __device__ __forceinline__ void tile(const TileAt& at, uint8_t* lds) const {
        using P = Piece<Core>;
        const uint16_t* x = w.xh + (uint64_t)at.z * mp * np;
        Core t;
        t.run(rows_of(x, at.i, np, Core::BP), rows_of(x, at.j, np, Core::BQ), np * 2, lds);
        uint16_t* a = w.a + (uint64_t)at.z * mp * mp;
        float* da = w.da + (uint64_t)at.z * mp;
#pragma unroll
        for (int u0 = 0; u0 < Core::TP; u0 += P::kU) {
            tf32x4 x[P::kU][Core::TQ];
#pragma unroll
            for (int u = 0; u < P::kU; ++u)
#pragma unroll
                for (int v = 0; v < P::kV; ++v) x[u][v] = t.acc[u0 + u][v] * inv_s2;
            store_sym<Core>(at, P(at, u0, lds), x, a, mp, da);
        }
    }
};

// B = b A + c A A.  A = O + D: A A = O O + (D_i + D_j) O_ij, and D_i^2 on the diagonal, where
// O is 0.
struct Poly {
    static constexpr bool SYM = true;
    NsBuf w;
    uint32_t mp, np;
    float kb, kc;
    template <class Core>
    __device__ __forceinline__ void tile(const TileAt& at, uint8_t* lds) const {
        using P = Piece<Core>;
        const uint16_t* a = w.a + (uint64_t)at.z * mp * mp;
        const float* da = w.da + (uint64_t)at.z * mp;
        Core t;
        t.run(rows_of(a, at.i, mp, Core::BP), rows_of(a, at.j, mp, Core::BQ), mp * 2, lds);
        uint16_t* b = w.b + (uint64_t)at.z * mp * mp;
        float* db = w.db + (uint64_t)at.z * mp;
#pragma unroll
        for (int u0 = 0; u0 < Core::TP; u0 += P::kU) {
            const P p(at, u0, lds);
            P::Down::load(p.l0, a + (uint64_t)p.j * mp + p.i, mp);
            wave_wait();
            tf32x4 x[P::kU][Core::TQ];
#pragma unroll
            for (int u = 0; u < P::kU; ++u) {
                const tf32x4 di = *(const tf32x4*)(da + p.i + 16 * u + p.li);
#pragma unroll
                for (int v = 0; v < P::kV; ++v) {
                    const float dj = da[p.j + 16 * v + p.lj];
                    const f16x4 o = *p.down(p.l0, u, v);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const bool diag = p.i + 16 * u + p.li + e == p.j + 16 * v + p.lj;
                        const float off = (float)o[e];
                        float sq = __builtin_fmaf(di[e] + dj, off, t.acc[u0 + u][v][e]);
                        if (diag) sq = __builtin_fmaf(dj, dj, sq);
                        x[u][v][e] = __builtin_fmaf(kc, sq, kb * (diag ? dj : off));
                    }
                }
            }
            store_sym<Core>(at, p, x, b, mp, db);
            if (u0 + P::kU < Core::TP) wave_wait();      // the next load overwrites the patches
        }
    }
};

// X <- a X + B X, to the buffers of the next step
struct Apply {
    static constexpr bool SYM = false;
    NsBuf w;
    uint32_t mp, np;
    float ka;
    int from;
    template <class Core>
    __device__ __forceinline__ void tile(const TileAt& at, uint8_t* lds) const {
        using P = Piece<Core>;
        const uint64_t xz = (uint64_t)at.z * mp * np;
        const uint16_t* b = w.b + (uint64_t)at.z * mp * mp;
        const uint16_t* xt = w.xt[from] + xz;
        Core t;
        t.run(rows_of(b, at.i, mp, Core::BP), rows_of(xt, at.j, mp, Core::BQ), mp * 2, lds);
        const float* db = w.db + (uint64_t)at.z * mp;
#pragma unroll
        for (int u0 = 0; u0 < Core::TP; u0 += P::kU) {
            const P p(at, u0, lds);
            const uint64_t down = xz + (uint64_t)p.j * mp + p.i;
            P::Down::load(p.l0, w.xt[from] + down, mp);
            P::Down::load(p.l1, w.lt + down, mp);
            wave_wait();
#pragma unroll
            for (int u = 0; u < P::kU; ++u) {
                const tf32x4 d = *(const tf32x4*)(db + p.i + 16 * u + p.li);
#pragma unroll
                for (int v = 0; v < P::kV; ++v) {
                    f16x4 *ph = p.down(p.l0, u, v), *pl = p.down(p.l1, u, v);
                    const f16x4 h = *ph, o = *pl;
                    tf32x4& y = t.acc[u0 + u][v];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        y[e] = __builtin_fmaf(ka + d[e], __builtin_fmaf((float)o[e], 1.0f / kLo, (float)h[e]), y[e]);
                    const f16x4 nh = pack4(y);
                    f16x4 nl;
#pragma unroll
                    for (int e = 0; e < 4; ++e) nl[e] = (_Float16)((y[e] - (float)nh[e]) * kLo);
                    *ph = nh;
                    *pl = nl;
                }
            }
            P::Down::store(p.l0, w.xt[from ^ 1] + down, mp);
            P::Down::store(p.l1, w.lt + down, mp);
#pragma unroll
            for (int u = 0; u < P::kU; ++u)
#pragma unroll
                for (int v = 0; v < P::kV; ++v) *p.across(p.l0, u, v) = pack4(transposed(pack4(t.acc[u0 + u][v])));
            P::Across::store(p.l0, w.xh + xz + (uint64_t)p.i * np + p.j, np);
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
// lane's four elements always are neighbours in a row of the source: there D's rows are j and
// its columns i, the iterate's first half comes from xh and its second, transposed, from lt.
template <class IO, class Dst, bool TALL>
struct Last {
    static constexpr bool SYM = false;
    IO io;
    NsBuf w;
    NsShape s;
    float ka, inv_s;
    int from;
    template <class Core>
    __device__ __forceinline__ void tile(const TileAt& at, uint8_t* lds) const {
        const uint32_t mp = s.mp, np = s.np;
        const uint64_t xz = (uint64_t)at.z * mp * np;
        const uint16_t* b = w.b + (uint64_t)at.z * mp * mp;
        const uint16_t* xt = w.xt[from] + xz;
        const uint16_t* xh = w.xh + xz;
        const uint16_t* lt = w.lt + xz;
        const float* db = w.db + (uint64_t)at.z * mp;
        const TileRows br = rows_of(b, TALL ? at.i : at.j, mp, TALL ? Core::BP : Core::BQ);
        const TileRows xr = rows_of(xt, TALL ? at.j : at.i, mp, TALL ? Core::BQ : Core::BP);
        Core t;
        t.run(TALL ? br : xr, TALL ? xr : br, mp * 2, lds);
        const Dst dst(io, s, at.z, inv_s);
        using P = Piece<Core>;
#pragma unroll
        for (int u0 = 0; u0 < Core::TP; u0 += P::kU) {
            const P p(at, u0, lds);
            if constexpr (TALL) {
                // D rows are i: four i of one j
                P::Down::load(p.l0, xt + (uint64_t)p.j * mp + p.i, mp);
                P::Down::load(p.l1, lt + (uint64_t)p.j * mp + p.i, mp);
            } else {
                // D rows (p.i) are j and its columns (p.j) are i: four j of one i
                P::Down::load(p.l0, xh + (uint64_t)p.j * np + p.i, np);
                P::Across::load(p.l1, lt + (uint64_t)p.i * mp + p.j, mp);
            }
            wave_wait();
#pragma unroll
            for (int u = 0; u < P::kU; ++u) {
                const uint32_t i = p.i + 16 * u + p.li;
                const tf32x4 di = TALL ? *(const tf32x4*)(db + i) : tf32x4{0, 0, 0, 0};
#pragma unroll
                for (int v = 0; v < P::kV; ++v) {
                    const uint32_t j = p.j + 16 * v + p.lj;
                    const f16x4 h = *p.down(p.l0, u, v);
                    tf32x4 o;
                    if constexpr (TALL) {
                        const f16x4 q = *p.down(p.l1, u, v);
                        o = tf32x4{(float)q[0], (float)q[1], (float)q[2], (float)q[3]};
                    } else {
                        o = transposed(*p.across(p.l1, u, v));
                    }
                    const float dj = TALL ? 0.0f : db[j];
                    tf32x4 y;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        y[e] = __builtin_fmaf(ka + (TALL ? di[e] : dj), __builtin_fmaf(o[e], 1.0f / kLo, (float)h[e]),
                                              t.acc[u0 + u][v][e]);
                    const uint32_t rows = TALL ? s.n : s.m, cols = TALL ? s.m : s.n;
                    if (j < rows && i < cols) dst.store(j, i, min(4u, cols - i), y);
                }
            }
            if (u0 + P::kU < Core::TP) wave_wait();
        }
    }
};

using Core256 = TileCore<256, 256, 2, 4, false>;
using Core128w = TileCore<128, 128, 2, 4, false>;      // quarters, by the same 512 threads
using Core128 = TileCore<128, 128, 2, 2, false>;
using Core64 = TileCore<64, 64, 2, 2, false, 4>;

template <class Op>
__global__ __launch_bounds__(512, 2) void ns_mixed_kernel(Op op, const DevState* st, TileMap m) {
    if (skipped(st)) return;
    __shared__ __attribute__((aligned(16))) uint8_t lds[Core256::kLds];
    const TileAt at = place<Op::SYM>(m);
    if (at.full) op.template tile<Core256>(at, lds);
    else if (!at.none) op.template tile<Core128w>(at, lds);
}
template <class Op, class Core>
__global__ __launch_bounds__(Core::NT) void ns_even_kernel(Op op, const DevState* st, uint32_t mp, uint32_t np) {
    if (skipped(st)) return;
    __shared__ __attribute__((aligned(16))) uint8_t lds[Core::kLds];
    op.template tile<Core>(place_even<Core, Op::SYM>(mp, np), lds);
}

// ------------------------------------------------------------------------------------
// launches
// ------------------------------------------------------------------------------------
// One product over `count` matrices with mp x np results (mp = np for the symmetric ones).
// The tile is chosen by what the launch would take per 128 bytes of K, from times measured on
// the full chip (us per slab): a round of 256 x 256 tiles (one block per CU) 1.45; of quarters
// in the same kernel 0.55; of 128 x 128 tiles 0.52 with one block per CU and 1.03 with two; of
// 64 x 64 tiles 0.23 and 0.39.  Results do not depend on the choice: every element's products
// are added in the same order.
template <class Op>
hipError_t launch_product(const Op& op, const DevState* st, uint32_t mp, uint32_t np, uint32_t count,
                          hipStream_t stream) {
    auto rounds = [](uint64_t n, double one, double two) {
        return n <= kCUs ? one : two * (double)((n + 2 * kCUs - 1) / (2 * kCUs));
    };
    const uint64_t p64 = mp / 64, q64 = np / 64;
    const uint64_t n64 = (Op::SYM ? p64 * (p64 + 1) / 2 : p64 * q64) * count;
    const double c64 = rounds(n64, 0.23, 0.39);
    if (mp % 128 || np % 128) {
        ns_even_kernel<Op, Core64><<<(uint32_t)n64, Core64::NT, 0, stream>>>(op, st, mp, np);
        return hipGetLastError();
    }
    const uint64_t p128 = mp / 128, q128 = np / 128;
    const uint64_t n128 = (Op::SYM ? p128 * (p128 + 1) / 2 : p128 * q128) * count;
    const double c128 = rounds(n128, 0.52, 1.03);
    double c256 = 0.0;
    uint64_t blocks = 0;
    const TileMap m = plan_tiles(Op::SYM, mp, np, count, 1.45, 0.55, &c256, &blocks);
    if (c256 < c128 && c256 < c64) {
        ns_mixed_kernel<Op><<<(uint32_t)blocks, 512, 0, stream>>>(op, st, m);
    } else if (c128 < c64) {
        ns_even_kernel<Op, Core128><<<(uint32_t)n128, Core128::NT, 0, stream>>>(op, st, mp, np);
    } else {
        ns_even_kernel<Op, Core64><<<(uint32_t)n64, Core64::NT, 0, stream>>>(op, st, mp, np);
    }
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
    for (int k = 0; k < steps && e == hipSuccess; ++k) {
        e = launch_product(Gram{w, s.mp, s.np, inv_s2}, st, s.mp, s.mp, count, stream);
        if (e == hipSuccess) e = launch_product(Poly{w, s.mp, s.np, coef[k].b, coef[k].c}, st, s.mp, s.mp, count, stream);
        if (e != hipSuccess) break;
        if (k + 1 < steps)
            e = launch_product(Apply{w, s.mp, s.np, coef[k].a, k & 1}, st, s.mp, s.np, count, stream);
        else if (s.tall)
            e = launch_product(Last<IO, Dst, true>{io, w, s, coef[k].a, inv_s, k & 1}, st, s.mp, s.np, count, stream);
        else
            e = launch_product(Last<IO, Dst, false>{io, w, s, coef[k].a, inv_s, k & 1}, st, s.np, s.mp, count, stream);
    }
    return e;
}

}  // namespace

hipError_t enqueue_orth(const NsShape& s, const NsBuf& w, uint32_t count, const OrthIO& io,
                        const NsCoef* coef, int steps, hipStream_t stream) {
    orth_norm_kernel<<<s.parts * count, kNormThreads, 0, stream>>>(io, s.rows, s.cols, s.parts, w.part);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    return enqueue_steps<OrthIO, OrthSrc, OrthDst>(s, w, count, io, coef, steps, stream);
}

hipError_t enqueue_muon(const NsShape& s, const NsBuf& w, uint32_t count, const MuonIO& io,
                        const NsCoef* coef, int steps, hipStream_t stream) {
    muon_momentum_kernel<<<s.parts * count, kNormThreads, 0, stream>>>(io, (uint64_t)s.rows * s.cols, s.parts, w.part);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    return enqueue_steps<MuonIO, MuonSrc, MuonDst>(s, w, count, io, coef, steps, stream);
}

// ------------------------------------------------------------------------------------
// shapes
// ------------------------------------------------------------------------------------
NsShape ns_shape(uint64_t rows, uint64_t cols) {
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
    w.a = (uint16_t*)take(a);
    w.b = (uint16_t*)take(a);
    w.da = (float*)take(4ull * s.mp * count);
    w.db = (float*)take(4ull * s.mp * count);
    w.part = (double*)take(8ull * kNsParts * count);
    return w;
}

uint64_t ns_bytes(const NsShape& s, uint64_t count) {
    const uint64_t x = 2ull * s.mp * s.np * count, a = 2ull * s.mp * s.mp * count;
    return 4 * up256(x) + 2 * up256(a) + 2 * up256(4ull * s.mp * count) + up256(8ull * kNsParts * count);
}

}  // namespace nz1
