// dropout_kernels.hip -- the element-wise passes of the linear layer on gfx950: dropout with
// bias and residual, and the way back through dropout and activation with the columns' sums.
#include "column_sums.h"
#include "epilogue.h"
#include "spread.h"

#include <algorithm>

namespace nz1 {

namespace {

struct DropoutArgs {
    const void *x, *bias, *residual;
    void* y;
    uint64_t x_ld, r_ld, y_ld, rows, row0;
    uint32_t cols;
    Drop drop;
};

constexpr uint32_t kDeep = 2;              // rows a thread has in flight
constexpr uint64_t kStreaming = 1ull << 26; // bytes of a pass from which on its accesses are non-temporal

// Rows of `units` threads in a row of all threads, for lengths that blocks of whole rows or stripes
// would leave threads idle in: n / units as a multiplication (n < 2^31; none for a single unit).
struct Flat {
    uint32_t units, mul, shift;
    uint64_t all;              // units in all
};
Flat flat(uint64_t rows, uint32_t units) {
    Flat f{units, 0, 0, rows * units};
    while ((1ull << f.shift) < units) ++f.shift;
    // 2^(31 + shift) / units, rounded up: off by less than units / 2^(31 + shift) of itself, too
    // little to show in a quotient of n < 2^31
    if (units > 1) f.mul = (uint32_t)(((1ull << (31 + f.shift)) + units - 1) / units);
    return f;
}
__device__ __forceinline__ uint32_t row_of(const Flat& f, uint32_t n) { return f.mul ? __umulhi(n, f.mul) >> (f.shift - 1) : n; }

// Memory-bound: BF16 16384 x 6144 with bias and residual 92 us, 6.5 TB/s; the random bits hide behind
// the memory (90 us without).  Two rows a thread, non-temporal both ways, measured (us): one row 103,
// four 105; ordinary loads 103, ordinary stores as well 111.  Below kStreaming bytes, where the caches
// keep what is read, ordinary accesses are as fast (2048 x 1024 4.9) and leave the result there.
template <int DT, bool NT, bool FLAT>
__global__ __launch_bounds__(256) void dropout_kernel(DropoutArgs a, Spread sp, Flat f) {
    const Unit u(sp, kDeep);
    const uint64_t off = drop_offset(a.drop);
    uint64_t row[kDeep];
    uint32_t unit[kDeep];
    bool in[kDeep];
    float x[kDeep][8], r[kDeep][8], b[kDeep][8] = {};
#pragma unroll
    for (uint32_t k = 0; k < kDeep; ++k) {
        if constexpr (FLAT) {
            const uint32_t n = (blockIdx.x * kDeep + k) * 256 + threadIdx.x, q = row_of(f, n);
            row[k] = q;
            unit[k] = n - q * f.units;
            in[k] = n < f.all;
        } else {
            row[k] = u.row + k * u.step;
            unit[k] = u.unit;
            in[k] = row[k] < a.rows && u.unit * 8u < a.cols;
        }
        const uint32_t c = unit[k] * 8, left = a.cols - c;
        if (!in[k]) break;
        if (a.bias && (FLAT || k == 0)) load8<DT>(a.bias, c, left, b[k]);
        load8<DT, NT>(a.x, row[k] * a.x_ld + c, left, x[k]);
        if (a.residual) load8<DT, NT>(a.residual, row[k] * a.r_ld + c, left, r[k]);
    }
#pragma unroll
    for (uint32_t k = 0; k < kDeep; ++k) {
        if (!in[k]) break;
        const uint32_t c = unit[k] * 8, left = a.cols - c;
        if (a.bias) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[k][e] += b[FLAT ? k : 0][e];
        }
        if (a.drop.limit) drop8(a.drop, off, (uint32_t)(a.row0 + row[k]), unit[k], x[k]);
        if (a.residual) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[k][e] += r[k][e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) x[k][e] = opaque(x[k][e]);
        store8<DT, NT>(a.y, row[k] * a.y_ld + c, left, x[k]);
    }
}

// The way back.  A block takes a stripe of columns and every count-th row (of groups of 256 / wide
// of them), so that the blocks under way sweep over neighbouring rows together, and adds up what
// it makes of them column by column: eight sums a thread, joined in order over the threads of one
// column, then over the blocks by join_kernel.  The sums' order goes by the sizes alone.
//
// Memory-bound without an act: BF16 16384 x 6144 73 us, 5.5 TB/s, and 4.5 of the join (64 without
// sums, by dropout_kernel).  With the join, blocks that take runs of rows instead 97 (their rows lie
// far apart), 512 of them 119, 1024 80, two rows in flight 81.  With an act and dropout bound by
// their arithmetic, some 60 instructions an element: 8192 x 24576 GELU 205 us to read 805 MB, 160
// without dropout.
struct BackArgs {
    Backward b;
    float* part;               // [count][cols], or null: no sums, or one block that writes dbias
    uint32_t across, shift;    // as in Spread
    uint32_t count;            // blocks that share the rows
};
constexpr uint32_t kDeepBack = 4;

constexpr uint32_t kMostBlocks = 768;

template <int DT, int ACT, bool NT>
__global__ __launch_bounds__(256) void backward_kernel(BackArgs a) {
    __shared__ float sums[256 * 8];
    const Backward& b = a.b;
    const uint32_t wide = 1u << a.shift, step = 256u >> a.shift;
    const uint32_t down = blockIdx.x / a.across;
    const uint32_t unit = ((blockIdx.x - down * a.across) << a.shift) + (threadIdx.x & (wide - 1));
    const uint32_t c = unit * 8;
    const uint32_t cols = (uint32_t)b.cols, n = c < cols ? cols - c : 0;
    const uint64_t off = drop_offset(b.drop);
    float s[8] = {};
    if (n) {
        const uint64_t apart = (uint64_t)a.count * step;
        for (uint64_t row0 = down * step + (threadIdx.x >> a.shift); row0 < b.rows; row0 += kDeepBack * apart) {
            float d[kDeepBack][8], p[kDeepBack][8];
#pragma unroll
            for (uint32_t k = 0; k < kDeepBack; ++k) {
                const uint64_t row = row0 + k * apart;
                if (row >= b.rows) break;
                load8<DT, NT>(b.dy, row * b.dy_ld + c, n, d[k]);
                if constexpr (ACT != NEOX_ACT_NONE) load8<DT, NT>(b.pre, row * b.pre_ld + c, n, p[k]);
            }
#pragma unroll
            for (uint32_t k = 0; k < kDeepBack; ++k) {
                const uint64_t row = row0 + k * apart;
                if (row >= b.rows) break;
                if constexpr (ACT != NEOX_ACT_NONE) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) d[k][e] *= slope<ACT>(p[k][e]);
                }
                if (b.drop.limit) drop8(b.drop, off, (uint32_t)row, unit, d[k]);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    d[k][e] = opaque(d[k][e]);
                    s[e] = __builtin_fmaf(d[k][e], b.scale, s[e]);
                }
                if (b.d) store8<DT, NT>(b.d, row * b.d_ld + c, b.padded ? 8 : n, d[k]);
            }
        }
    }
    if (!b.dbias) return;
    if (step > 1) {
#pragma unroll
        for (int e = 0; e < 8; ++e) sums[e * 256 + threadIdx.x] = s[e];
        __syncthreads();
        if (threadIdx.x >= wide) return;
        for (uint32_t k = 1; k < step; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] += sums[e * 256 + k * wide + threadIdx.x];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < (int)n) {
            if (a.part) a.part[(uint64_t)down * cols + c + e] = s[e];
            else put_bias<DT>(b, c + e, s[e]);
        }
}

template <int DT>
__global__ __launch_bounds__(1024) void join_kernel(Backward b, const float* part, uint32_t count) {
    __shared__ float sums[16 * 64];
    join_columns<DT>(b, part, count, blockIdx.x, sums);
}

// dbias of no rows
template <int DT>
__global__ __launch_bounds__(256) void no_rows_kernel(Backward b) {
    const uint64_t c = blockIdx.x * 256ull + threadIdx.x;
    if (c < b.cols) put_bias<DT>(b, (uint32_t)c, 0.0f);
}

// Blocks of the way back: enough for the chip, but not so many that their sums weigh against the
// rows.
struct Blocks {
    uint32_t shift, across, count;
};
Blocks blocks_of(uint64_t rows, uint64_t cols) {
    const Spread s = spread_close(1, (cols + 7) / 8, 1);
    const uint64_t least = (256u >> s.shift) * kDeepBack;       // rows a block has in flight
    const uint64_t most = std::max<uint64_t>(1, kMostBlocks / s.across);
    return Blocks{s.shift, s.across, (uint32_t)std::min((rows + least - 1) / least, most)};
}

template <class F>
void with_dtype(int32_t dtype, F f) {
    if (dtype == NEOX_F32) f(std::integral_constant<int, NEOX_F32>{});
    else if (dtype == NEOX_F16) f(std::integral_constant<int, NEOX_F16>{});
    else f(std::integral_constant<int, NEOX_BF16>{});
}

}  // namespace

hipError_t launch_dropout(const void* x, uint64_t x_ld, const void* bias, const void* residual, uint64_t residual_ld,
                          void* y, uint64_t y_ld, uint64_t rows, uint64_t cols, int32_t dtype, const Drop& drop,
                          hipStream_t stream) {
    const uint64_t size = dtype == NEOX_F32 ? 4 : 2;
    const bool nt = rows * cols * size * (residual ? 3 : 2) >= kStreaming;
    const uint64_t units = (cols + 7) / 8;
    const Spread one = spread_close(1, units, kDeep);
    const bool even = units % (1ull << one.shift) == 0;
    // rows of a launch: of whole rows or stripes as many as a grid takes, in a row 2^31 units
    const uint64_t most = even ? kGrid / one.across * ((256u >> one.shift) * kDeep) : std::max<uint64_t>(1, ((1ull << 31) - 1024) / units);
    for (uint64_t row = 0; row < rows; row += most) {
        const uint64_t n = std::min(most, rows - row);
        const DropoutArgs a{(const uint8_t*)x + row * x_ld * size, bias,
                            residual ? (const uint8_t*)residual + row * residual_ld * size : nullptr,
                            (uint8_t*)y + row * y_ld * size, x_ld, residual_ld, y_ld, n, row, (uint32_t)cols, drop};
        const Spread sp = spread_close(n, units, kDeep);
        const Flat f = flat(n, (uint32_t)units);
        const uint32_t blocks = even ? (uint32_t)sp.blocks : (uint32_t)((f.all + 256 * kDeep - 1) / (256 * kDeep));
        with_dtype(dtype, [&](auto dt) {
            constexpr int DT = decltype(dt)::value;
            if (even && nt) dropout_kernel<DT, true, false><<<blocks, 256, 0, stream>>>(a, sp, f);
            else if (even) dropout_kernel<DT, false, false><<<blocks, 256, 0, stream>>>(a, sp, f);
            else if (nt) dropout_kernel<DT, true, true><<<blocks, 256, 0, stream>>>(a, sp, f);
            else dropout_kernel<DT, false, true><<<blocks, 256, 0, stream>>>(a, sp, f);
        });
    }
    return hipGetLastError();
}

uint32_t backward_parts(uint64_t rows, uint64_t cols) {
    const uint32_t n = blocks_of(rows, cols).count;
    return n > 1 ? n : 0;
}

uint64_t backward_workspace(uint64_t rows, uint64_t cols) {
    const Blocks r = blocks_of(rows, cols);
    return r.count > 1 ? (r.count * cols * 4 + 255) / 256 * 256 : 0;
}

hipError_t launch_backward(const Backward& b, void* workspace, bool join_here, hipStream_t stream) {
    // without an act and sums it is dropout of dy
    if (!b.dbias && !b.pre && !b.padded)
        return launch_dropout(b.dy, b.dy_ld, nullptr, nullptr, 0, b.d, b.d_ld, b.rows, b.cols, b.dtype, b.drop, stream);
    const Blocks r = blocks_of(b.rows, b.cols);
    const uint64_t arrays = 1 + (b.pre ? 1 : 0) + (b.d ? 1 : 0);
    const bool nt = b.rows * b.cols * (b.dtype == NEOX_F32 ? 4 : 2) * arrays >= kStreaming;
    with_dtype(b.dtype, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        if (b.rows == 0) {
            no_rows_kernel<DT><<<(uint32_t)((b.cols + 255) / 256), 256, 0, stream>>>(b);
            return;
        }
        const bool join = b.dbias && r.count > 1;
        const BackArgs a{b, join ? (float*)workspace : nullptr, r.across, r.shift, r.count};
        const uint32_t blocks = r.across * r.count;
        auto run = [&](auto act) {
            constexpr int ACT = decltype(act)::value;
            if (nt) backward_kernel<DT, ACT, true><<<blocks, 256, 0, stream>>>(a);
            else backward_kernel<DT, ACT, false><<<blocks, 256, 0, stream>>>(a);
        };
        // (only half types have an act)
        if constexpr (DT == NEOX_F32) run(std::integral_constant<int, NEOX_ACT_NONE>{});
        else with_act(b.act, run);
    });
    if (join_here) return launch_join(b, workspace, stream);
    return hipGetLastError();
}

hipError_t launch_join(const Backward& b, const void* workspace, hipStream_t stream) {
    const uint32_t parts = backward_parts(b.rows, b.cols);
    if (b.dbias && parts)
        with_dtype(b.dtype, [&](auto dt) {
            join_kernel<decltype(dt)::value><<<(uint32_t)((b.cols + 63) / 64), 1024, 0, stream>>>(b, (const float*)workspace, parts);
        });
    return hipGetLastError();
}

}  // namespace nz1
