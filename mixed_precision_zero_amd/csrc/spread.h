// spread.h -- how element-wise passes over a matrix's rows are laid over blocks.
#pragma once

#include <hip/hip_runtime.h>
#include <algorithm>
#include <stdint.h>

namespace nz1 {

// How the rows of an array are spread over blocks of 256 threads, a thread taking eight
// elements of each of `deep` rows: `wide` threads side by side (a power of two) on 256 / wide
// rows, `deep` times.
struct Spread {
    uint32_t shift;        // log2(wide)
    uint32_t across;       // blocks across a row
    uint64_t blocks;
};
inline Spread spread(uint64_t rows, uint64_t units, uint32_t deep) {
    Spread s{};
    while (s.shift < 8 && (1ull << s.shift) < units) ++s.shift;
    s.across = (uint32_t)((units + (1ull << s.shift) - 1) >> s.shift);
    const uint64_t per = (256u >> s.shift) * deep;
    s.blocks = (rows + per - 1) / per * s.across;
    return s;
}
// The same with as few idle threads as rows of 16 threads or more allow: the widest one that wastes
// less than a tenth, or else the one that wastes least.
inline Spread spread_close(uint64_t rows, uint64_t units, uint32_t deep) {
    uint32_t best = 8;
    double most = 0.0;
    for (uint32_t shift = 8; shift >= 4; --shift) {
        const double used = (double)units / (double)((units + (1ull << shift) - 1) >> shift << shift);
        if (used > most) {
            most = used;
            best = shift;
        }
        if (used > 0.9) break;
    }
    while (best > 0 && units <= (1ull << best) / 2) --best;
    Spread s{};
    s.shift = best;
    s.across = (uint32_t)((units + (1ull << best) - 1) >> best);
    const uint64_t per = (256u >> best) * deep;
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

// Blocks of one launch: a grid has fewer than 2^32 threads.
constexpr uint64_t kGrid = 1ull << 23;

// Launches f(first row, rows, their spread) for as many rows at a time as a grid takes.
template <class F>
void rows_in_grids(uint64_t rows, uint64_t units, uint32_t deep, F f) {
    const Spread one = spread(1, units, deep);          // (at most 2^20 blocks across)
    const uint64_t most = kGrid / one.across * ((256u >> one.shift) * deep);
    for (uint64_t r = 0; r < rows; r += most) {
        const uint64_t n = std::min(most, rows - r);
        f(r, n, spread(n, units, deep));
    }
}

}  // namespace nz1
