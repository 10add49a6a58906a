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

__device__ __forceinline__ float f16(uint16_t v) { return (float)__builtin_bit_cast(_Float16, v); }
__device__ __forceinline__ uint16_t to_f16(float x) { return __builtin_bit_cast(uint16_t, (_Float16)x); }

constexpr float kLo = 2048.0f;            // lt holds (x - hi) * kLo

// The step state whose skip flag the kernels heed (none: always run).
__host__ __device__ inline const DevState* state_of(const OrthIO&) { return nullptr; }
__host__ __device__ inline const DevState* state_of(const MuonIO& io) { return io.st; }
__device__ __forceinline__ bool skipped(const DevState* st) { return st && st->skip; }

// The destination of the iterate between steps: none.
struct NoIO {
    const DevState* st;
};
__host__ __device__ inline const DevState* state_of(const NoIO& io) { return io.st; }
struct NoDst {
    __device__ NoDst(const NoIO&, uint32_t, float) {}
    __device__ void store(uint32_t, uint32_t, uint32_t, float) const {}
};

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

// ------------------------------------------------------------------------------------
// squared norm of each source matrix; for Muon also the momentum's own update
// ------------------------------------------------------------------------------------
__global__ __launch_bounds__(256) void orth_norm_kernel(OrthIO io, uint32_t rows, uint32_t cols,
                                                        uint32_t parts, double* __restrict__ part) {
    const uint32_t z = blockIdx.x / parts, p = blockIdx.x % parts;
    const uint32_t per = (rows + parts - 1) / parts;
    const uint32_t r0 = p * per, r1 = min(rows, r0 + per);
    double s = 0.0;
    for (uint32_t r = r0; r < r1; ++r) {
        const uint64_t at = z * io.src_stride + r * io.src_ld;
        for (uint32_t c = threadIdx.x; c < cols; c += 256) {
            const double x = load_elem(io.src, io.src_dtype, at + c);
            s = __builtin_fma(x, x, s);
        }
    }
    s = sum_block<256>(s);
    if (threadIdx.x == 0) part[(uint64_t)z * kNsParts + p] = s;
}

__device__ __forceinline__ float direction(const MuonIO& io, float g, float m) {
    return io.nesterov ? __builtin_fmaf(io.mu, m, g) : m;
}

__global__ __launch_bounds__(256) void muon_momentum_kernel(MuonIO io, uint64_t numel,
                                                            uint32_t parts, double* __restrict__ part) {
    if (io.st->skip) return;
    const float gs = io.st->gscale;
    const uint32_t z = blockIdx.x / parts, p = blockIdx.x % parts;
    const MuonMat mat = io.mats[z];
    double s = 0.0;
    for (uint64_t i = (uint64_t)p * 256 + threadIdx.x; i < numel; i += (uint64_t)parts * 256) {
        const float g = half_to_float(io.dtype, mat.grad[i]) * gs;
        const float m = __builtin_fmaf(io.mu, mat.mom[i], g);
        mat.mom[i] = m;
        const double u = direction(io, g, m);
        s = __builtin_fma(u, u, s);
    }
    s = sum_block<256>(s);
    if (threadIdx.x == 0) part[(uint64_t)z * kNsParts + p] = s;
}

// ------------------------------------------------------------------------------------
// X0 = source / (norm + eps), split in two, both orientations, zero padded
// ------------------------------------------------------------------------------------
struct OrthSrc {
    const OrthIO& io;
    uint64_t at;
    __device__ OrthSrc(const OrthIO& i, uint32_t z) : io(i), at(z * i.src_stride) {}
    __device__ float load(uint32_t r, uint32_t c, uint32_t) const {
        return load_elem(io.src, io.src_dtype, at + r * io.src_ld + c);
    }
};
struct MuonSrc {
    const MuonIO& io;
    MuonMat mat;
    float gs;
    __device__ MuonSrc(const MuonIO& i, uint32_t z) : io(i), mat(i.mats[z]), gs(i.st->gscale) {}
    __device__ float load(uint32_t r, uint32_t c, uint32_t cols) const {
        const uint64_t i = (uint64_t)r * cols + c;
        return direction(io, half_to_float(io.dtype, mat.grad[i]) * gs, mat.mom[i]);
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
    const double sq = sum_block<256>(threadIdx.x < s.parts ? part[threadIdx.x] : 0.0);
    const double f = (double)s.s / (__builtin_sqrt(sq) + io.eps);
    const Src src(io, z);
    const uint32_t lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    // the tile as the source has it: rows r0.., columns c0..
    const uint32_t r0 = s.tall ? j0 : i0, c0 = s.tall ? i0 : j0;
#pragma unroll 4
    for (uint32_t k = wv; k < 64; k += 4) {
        const uint32_t r = r0 + k, c = c0 + lane;
        tile[k][lane] = r < s.rows && c < s.cols ? (float)((double)src.load(r, c, s.cols) * f) : 0.0f;
    }
    __syncthreads();
    const uint64_t xz = (uint64_t)z * s.mp * s.np;
#pragma unroll 4
    for (uint32_t k = wv; k < 64; k += 4) {
        // row k of the tile in the wide form, and column k of it
        const float x = s.tall ? tile[lane][k] : tile[k][lane];
        w.xh[xz + (uint64_t)(i0 + k) * s.np + j0 + lane] = to_f16(x);
        const float y = s.tall ? tile[k][lane] : tile[lane][k];
        const uint16_t hi = to_f16(y);
        const uint64_t at = xz + (uint64_t)(j0 + k) * s.mp + i0 + lane;
        w.xt[0][at] = hi;
        w.lt[at] = to_f16((y - f16(hi)) * kLo);
    }
}

// ------------------------------------------------------------------------------------
// the products
// ------------------------------------------------------------------------------------
// tile (ti, tj), tj <= ti, of number t in row order of the lower triangle
__device__ __forceinline__ void lower(uint32_t t, uint32_t& ti, uint32_t& tj) {
    uint32_t i = (uint32_t)((__builtin_sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
    while (i * (i + 1) / 2 > t) --i;
    while ((i + 1) * (i + 2) / 2 <= t) ++i;
    ti = i;
    tj = t - i * (i + 1) / 2;
}

template <class Core>
__device__ __forceinline__ TileRows rows_of(const uint16_t* base, uint64_t row, uint32_t len, int block) {
    return TileRows{(const uint8_t*)(base + row * len), nullptr, (uint32_t)block, len * 2u, 0u};
}

template <class Core>
__global__ __launch_bounds__(Core::NT) void ns_gram_kernel(const DevState* st, NsShape s, NsBuf w, float inv_s2) {
    if (skipped(st)) return;
    __shared__ __attribute__((aligned(16))) uint8_t lds[2 * Core::kStage];
    const uint32_t side = s.mp / Core::BP, tiles = side * (side + 1) / 2;
    const uint32_t z = blockIdx.x / tiles;
    uint32_t ti, tj;
    lower(blockIdx.x % tiles, ti, tj);
    const uint16_t* x = w.xh + (uint64_t)z * s.mp * s.np;
    Core t;
    t.run(rows_of<Core>(x, (uint64_t)ti * Core::BP, s.np, Core::BP),
          rows_of<Core>(x, (uint64_t)tj * Core::BQ, s.np, Core::BQ), s.np * 2, lds);
    uint16_t* a = w.a + (uint64_t)z * s.mp * s.mp;
    float* da = w.da + (uint64_t)z * s.mp;
    const uint32_t lane = threadIdx.x & 63;
    const uint32_t ib = ti * Core::BP + Core::wave_p() + (lane >> 4) * 4;
    const uint32_t jb = tj * Core::BQ + Core::wave_q() + (lane & 15);
#pragma unroll
    for (int u = 0; u < Core::TP; ++u)
#pragma unroll
        for (int v = 0; v < Core::TQ; ++v) {
            const uint32_t j = jb + 16 * v;
            uint16_t h[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t i = ib + 16 * u + e;
                const float x = t.acc[u][v][e] * inv_s2;
                if (i == j) da[i] = x;
                h[e] = i == j ? (uint16_t)0 : to_f16(x);
                a[(uint64_t)i * s.mp + j] = h[e];
            }
            if (ti != tj)
                *(ushort4*)(a + (uint64_t)j * s.mp + ib + 16 * u) = make_ushort4(h[0], h[1], h[2], h[3]);
        }
}

template <class Core>
__global__ __launch_bounds__(Core::NT) void ns_poly_kernel(const DevState* st, NsShape s, NsBuf w, NsCoef k) {
    if (skipped(st)) return;
    __shared__ __attribute__((aligned(16))) uint8_t lds[2 * Core::kStage];
    const uint32_t side = s.mp / Core::BP, tiles = side * (side + 1) / 2;
    const uint32_t z = blockIdx.x / tiles;
    uint32_t ti, tj;
    lower(blockIdx.x % tiles, ti, tj);
    const uint16_t* a = w.a + (uint64_t)z * s.mp * s.mp;
    Core t;
    t.run(rows_of<Core>(a, (uint64_t)ti * Core::BP, s.mp, Core::BP),
          rows_of<Core>(a, (uint64_t)tj * Core::BQ, s.mp, Core::BQ), s.mp * 2, lds);
    uint16_t* b = w.b + (uint64_t)z * s.mp * s.mp;
    const float* da = w.da + (uint64_t)z * s.mp;
    float* db = w.db + (uint64_t)z * s.mp;
    const uint32_t lane = threadIdx.x & 63;
    const uint32_t ib = ti * Core::BP + Core::wave_p() + (lane >> 4) * 4;
    const uint32_t jb = tj * Core::BQ + Core::wave_q() + (lane & 15);
#pragma unroll
    for (int u = 0; u < Core::TP; ++u)
#pragma unroll
        for (int v = 0; v < Core::TQ; ++v) {
            const uint32_t j = jb + 16 * v;
            // A = O + D: A A = O O + (D_i + D_j) O_ij + D_i^2 on the diagonal (O is 0 there)
            const ushort4 o4 = *(const ushort4*)(a + (uint64_t)j * s.mp + ib + 16 * u);
            const uint16_t o[4] = {o4.x, o4.y, o4.z, o4.w};
            uint16_t h[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t i = ib + 16 * u + e;
                const float di = da[i], off = f16(o[e]);
                float sq = __builtin_fmaf(di + da[j], off, t.acc[u][v][e]);
                float lin = off;
                if (i == j) {
                    sq = __builtin_fmaf(di, di, sq);
                    lin = di;
                }
                const float x = __builtin_fmaf(k.c, sq, k.b * lin);
                if (i == j) db[i] = x;
                h[e] = i == j ? (uint16_t)0 : to_f16(x);
                b[(uint64_t)i * s.mp + j] = h[e];
            }
            if (ti != tj)
                *(ushort4*)(b + (uint64_t)j * s.mp + ib + 16 * u) = make_ushort4(h[0], h[1], h[2], h[3]);
        }
}

// What the last step's result becomes.
struct OrthDst {
    const OrthIO& io;
    uint64_t at;
    float f;
    __device__ OrthDst(const OrthIO& i, uint32_t z, float inv_s)
        : io(i), at(z * i.dst_stride), f(i.scale * inv_s) {}
    __device__ void store(uint32_t r, uint32_t c, uint32_t, float x) const {
        store_elem(io.dst, io.dst_dtype, at + r * io.dst_ld + c, x * f);
    }
};
struct MuonDst {
    const MuonIO& io;
    MuonMat mat;
    float f, wd;
    __device__ MuonDst(const MuonIO& i, uint32_t z, float inv_s)
        : io(i), mat(i.mats[z]), f(i.scale * inv_s), wd(mat.decay ? i.wd : 0.0f) {}
    __device__ void store(uint32_t r, uint32_t c, uint32_t cols, float x) const {
        const uint64_t i = (uint64_t)r * cols + c;
        const float w = mat.master[i];
        const float n = opaque(__builtin_fmaf(-io.lr, __builtin_fmaf(wd, w, x * f), w));
        mat.master[i] = n;
        mat.half[i] = float_to_half(io.dtype, n);
    }
};

// LAST: the result goes to Dst instead of the buffers.
template <class Core, class IO, class Dst, bool LAST>
__global__ __launch_bounds__(Core::NT) void ns_apply_kernel(IO io, NsShape s, NsBuf w, float ka,
                                                            int from, float inv_s) {
    if (skipped(state_of(io))) return;
    __shared__ __attribute__((aligned(16))) uint8_t lds[2 * Core::kStage];
    const uint32_t np_t = s.np / Core::BQ, tiles = s.mp / Core::BP * np_t;
    const uint32_t z = blockIdx.x / tiles, tt = blockIdx.x % tiles;
    const uint32_t ti = tt / np_t, tj = tt % np_t;
    const uint64_t xz = (uint64_t)z * s.mp * s.np;
    const uint16_t* b = w.b + (uint64_t)z * s.mp * s.mp;
    const uint16_t* xt = w.xt[from] + xz;
    Core t;
    t.run(rows_of<Core>(b, (uint64_t)ti * Core::BP, s.mp, Core::BP),
          rows_of<Core>(xt, (uint64_t)tj * Core::BQ, s.mp, Core::BQ), s.mp * 2, lds);
    const float* db = w.db + (uint64_t)z * s.mp;
    uint16_t* lt = w.lt + xz;
    uint16_t* xo = w.xt[from ^ 1] + xz;
    uint16_t* xh = w.xh + xz;
    const Dst dst(io, z, inv_s);
    const uint32_t lane = threadIdx.x & 63;
    const uint32_t ib = ti * Core::BP + Core::wave_p() + (lane >> 4) * 4;
    const uint32_t jb = tj * Core::BQ + Core::wave_q() + (lane & 15);
#pragma unroll
    for (int u = 0; u < Core::TP; ++u)
#pragma unroll
        for (int v = 0; v < Core::TQ; ++v) {
            const uint32_t j = jb + 16 * v, i = ib + 16 * u;
            const uint64_t at = (uint64_t)j * s.mp + i;
            const ushort4 h4 = *(const ushort4*)(xt + at), l4 = *(const ushort4*)(lt + at);
            const uint16_t h[4] = {h4.x, h4.y, h4.z, h4.w}, l[4] = {l4.x, l4.y, l4.z, l4.w};
            uint16_t nh[4], nl[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float x = __builtin_fmaf(f16(l[e]), 1.0f / kLo, f16(h[e]));
                const float y = __builtin_fmaf(ka + db[i + e], x, t.acc[u][v][e]);
                if constexpr (LAST) {
                    if (i + e < s.m && j < s.n) {
                        if (s.tall) dst.store(j, i + e, s.cols, y);
                        else dst.store(i + e, j, s.cols, y);
                    }
                } else {
                    nh[e] = to_f16(y);
                    nl[e] = to_f16((y - f16(nh[e])) * kLo);
                    xh[(uint64_t)(i + e) * s.np + j] = nh[e];
                }
            }
            if constexpr (!LAST) {
                *(ushort4*)(xo + at) = make_ushort4(nh[0], nh[1], nh[2], nh[3]);
                *(ushort4*)(lt + at) = make_ushort4(nl[0], nl[1], nl[2], nl[3]);
            }
        }
}

// ------------------------------------------------------------------------------------
// launches
// ------------------------------------------------------------------------------------
template <class Core, class IO, class Src, class Dst>
hipError_t enqueue_steps(const NsShape& s, const NsBuf& w, uint32_t count, const IO& io,
                         const NsCoef* coef, int steps, hipStream_t stream) {
    const uint32_t conv = s.mp / 64 * (s.np / 64) * count;
    ns_convert_kernel<Src><<<conv, 256, 0, stream>>>(io, s, w);
    hipError_t e = hipGetLastError();
    const uint32_t side = s.mp / Core::BP;
    const uint32_t sym = side * (side + 1) / 2 * count, full = side * (s.np / Core::BQ) * count;
    const float inv_s2 = 1.0f / (s.s * s.s), inv_s = 1.0f / s.s;
    for (int k = 0; k < steps && e == hipSuccess; ++k) {
        ns_gram_kernel<Core><<<sym, Core::NT, 0, stream>>>(state_of(io), s, w, inv_s2);
        e = hipGetLastError();
        if (e != hipSuccess) break;
        ns_poly_kernel<Core><<<sym, Core::NT, 0, stream>>>(state_of(io), s, w, coef[k]);
        e = hipGetLastError();
        if (e != hipSuccess) break;
        if (k + 1 < steps)
            ns_apply_kernel<Core, NoIO, NoDst, false><<<full, Core::NT, 0, stream>>>(NoIO{state_of(io)}, s, w, coef[k].a, k & 1, inv_s);
        else
            ns_apply_kernel<Core, IO, Dst, true><<<full, Core::NT, 0, stream>>>(io, s, w, coef[k].a, k & 1, inv_s);
        e = hipGetLastError();
    }
    return e;
}

using Core128 = TileCore<128, 128, 2, 2, false>;

template <class IO, class Src, class Dst>
hipError_t enqueue_any(const NsShape& s, const NsBuf& w, uint32_t count, const IO& io,
                       const NsCoef* coef, int steps, hipStream_t stream) {
    return enqueue_steps<Core128, IO, Src, Dst>(s, w, count, io, coef, steps, stream);
}

}  // namespace

hipError_t enqueue_orth(const NsShape& s, const NsBuf& w, uint32_t count, const OrthIO& io,
                        const NsCoef* coef, int steps, hipStream_t stream) {
    orth_norm_kernel<<<s.parts * count, 256, 0, stream>>>(io, s.rows, s.cols, s.parts, w.part);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    return enqueue_any<OrthIO, OrthSrc, OrthDst>(s, w, count, io, coef, steps, stream);
}

hipError_t enqueue_muon(const NsShape& s, const NsBuf& w, uint32_t count, const MuonIO& io,
                        const NsCoef* coef, int steps, hipStream_t stream) {
    muon_momentum_kernel<<<s.parts * count, 256, 0, stream>>>(io, (uint64_t)s.rows * s.cols, s.parts, w.part);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    return enqueue_any<MuonIO, MuonSrc, MuonDst>(s, w, count, io, coef, steps, stream);
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
    s.tile = 128;
    s.mp = (s.m + s.tile - 1) / s.tile * s.tile;
    s.np = (s.n + s.tile - 1) / s.tile * s.tile;
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
