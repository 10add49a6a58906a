// matrix_api.hip -- host side of include/neox_matrix.h: argument validation, workspace
// layout, the Muon handle and its grouping of matrices, and the MXFP4 entry points.
#include "neox_matrix.h"
#include "matrix_internal.h"

#include <algorithm>
#include <cmath>
#include <cstring>
#include <map>
#include <new>
#include <vector>

using namespace nz1;

namespace {

constexpr uint64_t kMaxSide = 1ull << 20;       // rows or cols of an orthogonalised matrix
constexpr uint64_t kMaxCount = 1ull << 24;
constexpr uint64_t kMaxMx = (1ull << 31) - 1;   // rows or cols of an MXFP4 copy
constexpr uint64_t kMaxK = 1ull << 24;          // k of a product (32-bit offsets in a tile)
constexpr uint64_t kMaxBlocks = 1ull << 24;     // grid limit: 2^32 threads at 256 per block
constexpr uint64_t kMaxTiles = 1ull << 23;      // 128 x 128 tiles of a product: 512 threads each
constexpr uint64_t kDefaultWorkspace = 4ull << 30;

bool known_type(int32_t t) { return t == NEOX_F16 || t == NEOX_BF16 || t == NEOX_F32; }
uint64_t type_bytes(int32_t t) { return t == NEOX_F32 ? 4 : 2; }

// The largest magnitude p(x) = a x + b x^3 + c x^5 takes on [0, top]: at the end or where
// p' = a + 3 b y + 5 c y^2 = 0, y = x^2.
double poly_top(double a, double b, double c, double top) {
    auto p = [&](double x) { return std::fabs(x * (a + x * x * (b + x * x * c))); };
    double best = p(top);
    auto at = [&](double y) {
        if (y > 0.0 && y < top * top) best = std::max(best, p(std::sqrt(y)));
    };
    if (c != 0.0) {
        const double d = 9.0 * b * b - 20.0 * a * c;
        if (d >= 0.0) {
            at((-3.0 * b + std::sqrt(d)) / (10.0 * c));
            at((-3.0 * b - std::sqrt(d)) / (10.0 * c));
        }
    } else if (b != 0.0) {
        at(-a / (3.0 * b));
    }
    return best;
}

// Validates the steps and rounds the coefficients; fills coef[steps].  *pairs: the product of
// two consecutive steps' polynomials fits FP16 too.
int ns_coefs(const neox_ns_config* c, NsCoef* coef, bool* pairs) {
    if (!c) return set_error(NEOX_EINVAL, "the Newton-Schulz configuration is NULL");
    if (c->steps < 1 || c->steps > NEOX_NS_MAX_STEPS)
        return set_error(NEOX_EINVAL, "steps %d not in [1, %d]", c->steps, NEOX_NS_MAX_STEPS);
    if (c->reserved) return set_error(NEOX_EINVAL, "reserved field %d is not 0", c->reserved);
    if (!(std::isfinite(c->eps) && (float)c->eps > 0.0f && std::isfinite((float)c->eps)))
        return set_error(NEOX_EINVAL, "eps %g: must be > 0 in FP32", c->eps);
    double top = 1.0, before = 0.0;
    *pairs = true;
    for (int k = 0; k < c->steps; ++k) {
        const double a = c->coef[k][0], b = c->coef[k][1], d = c->coef[k][2];
        if (!std::isfinite((float)a) || !std::isfinite((float)b) || !std::isfinite((float)d))
            return set_error(NEOX_EINVAL, "step %d: coefficients are not finite", k);
        // what the FP16 copies hold: elements of A up to top^2, of b A + c A A up to this
        if (std::fabs(b) * top * top + std::fabs(d) * top * top * top * top > 30000.0)
            return set_error(NEOX_EINVAL, "step %d: coefficients (%g, %g, %g) too large", k, a, b, d);
        const double size = std::fabs(a) + std::fabs(b) * top * top + std::fabs(d) * top * top * top * top;
        if (size * std::max(before, 1.0) > 30000.0) *pairs = false;
        before = size;
        top = 1.01 * poly_top(a, b, d, top);
        if (top > 8.0)
            return set_error(NEOX_EINVAL, "step %d: singular values grow to %g", k, top);
        coef[k] = NsCoef{(float)a, (float)b, (float)d};
    }
    return NEOX_OK;
}

int check_sides(uint64_t rows, uint64_t cols) {
    if (rows == 0 || cols == 0) return set_error(NEOX_EINVAL, "a matrix of %llu x %llu",
                                                 (unsigned long long)rows, (unsigned long long)cols);
    if (rows > kMaxSide || cols > kMaxSide)
        return set_error(NEOX_EINVAL, "a matrix of %llu x %llu: at most 2^20 a side",
                         (unsigned long long)rows, (unsigned long long)cols);
    return NEOX_OK;
}

// Matrices one launch may take: thread counts stay below the grid limit (the largest grids are
// those of 64 x 64 tiles, the split products' at most twice as many, and the norm's, at most
// kNsParts blocks of 1,024 threads).
uint64_t launch_count(const NsShape& s) {
    const uint64_t per = std::max<uint64_t>((uint64_t)(s.mp / 64) * (s.np / 64) * 2, 4 * kNsParts);
    return std::max<uint64_t>(1, (kMaxBlocks - 1) / per);
}

}  // namespace

// ------------------------------------------------------------------------------------
// orthogonalisation
// ------------------------------------------------------------------------------------
extern "C" int neox_ns_default_config(neox_ns_config* cfg) {
    if (!cfg) return set_error(NEOX_EINVAL, "cfg is NULL");
    std::memset(cfg, 0, sizeof *cfg);
    cfg->steps = 5;
    cfg->eps = 1e-7;
    for (int k = 0; k < NEOX_NS_MAX_STEPS; ++k) {
        cfg->coef[k][0] = 3.4445;
        cfg->coef[k][1] = -4.7750;
        cfg->coef[k][2] = 2.0315;
    }
    return NEOX_OK;
}

extern "C" int neox_orthogonalize_workspace(uint64_t count, uint64_t rows, uint64_t cols, uint64_t* bytes) {
    if (!bytes) return set_error(NEOX_EINVAL, "bytes is NULL");
    const int rc = check_sides(rows, cols);
    if (rc) return rc;
    if (count == 0 || count > kMaxCount)
        return set_error(NEOX_EINVAL, "count %llu not in [1, 2^24]", (unsigned long long)count);
    // as with two steps at a time, which needs more, whatever the coefficients will be
    const NsShape s = ns_shape(rows, cols, true);
    *bytes = ns_bytes(s, std::min(count, launch_count(s)));
    return NEOX_OK;
}

extern "C" int neox_orthogonalize(const neox_ns_config* cfg, const void* src, int32_t src_dtype,
                                  uint64_t src_ld, uint64_t src_stride, void* dst, int32_t dst_dtype,
                                  uint64_t dst_ld, uint64_t dst_stride, uint64_t count, uint64_t rows,
                                  uint64_t cols, double scale, void* workspace, uint64_t workspace_bytes,
                                  void* hip_stream) {
    NsCoef coef[NEOX_NS_MAX_STEPS];
    bool pairs = false;
    int rc = ns_coefs(cfg, coef, &pairs);
    if (rc) return rc;
    uint64_t need = 0;
    rc = neox_orthogonalize_workspace(count, rows, cols, &need);
    if (rc) return rc;
    if (!src || !dst || !workspace) return set_error(NEOX_EINVAL, "null argument");
    if (!known_type(src_dtype) || !known_type(dst_dtype))
        return set_error(NEOX_EINVAL, "types %d, %d", src_dtype, dst_dtype);
    const uint64_t sb = type_bytes(src_dtype), db = type_bytes(dst_dtype);
    if ((uintptr_t)src % sb || (uintptr_t)dst % db) return set_error(NEOX_EINVAL, "src or dst misaligned");
    if ((uintptr_t)workspace & 255u) return set_error(NEOX_EINVAL, "workspace not 256-byte aligned");
    if (workspace_bytes < need)
        return set_error(NEOX_EINVAL, "workspace of %llu bytes, %llu needed",
                         (unsigned long long)workspace_bytes, (unsigned long long)need);
    if (src_ld < cols || dst_ld < cols) return set_error(NEOX_EINVAL, "ld smaller than cols");
    // last element's index must stay far from 64 bits (in bytes too)
    const uint64_t lim = 1ull << 60;
    if (src_ld > lim / rows || dst_ld > lim / rows || src_stride > lim / count || dst_stride > lim / count)
        return set_error(NEOX_EINVAL, "ld or stride too large");
    const uint64_t span = (rows - 1) * dst_ld + cols, sspan = (rows - 1) * src_ld + cols;
    // one behind the other, or side by side in rows of dst_ld
    const bool beside = dst_stride >= cols && (rows == 1 || dst_stride <= (dst_ld - cols) / (count > 1 ? count - 1 : 1));
    if (count > 1 && dst_stride < span && !beside) return set_error(NEOX_EINVAL, "matrices of dst overlap");
    const uint64_t slen = ((count - 1) * src_stride + sspan) * sb, dlen = ((count - 1) * dst_stride + span) * db;
    const uintptr_t s0 = (uintptr_t)src, d0 = (uintptr_t)dst, w0 = (uintptr_t)workspace;
    const bool same = s0 == d0 && src_dtype == dst_dtype && src_ld == dst_ld &&
                      (count == 1 || src_stride == dst_stride);
    if (!same && s0 < d0 + dlen && d0 < s0 + slen)
        return set_error(NEOX_EINVAL, "dst overlaps src and is not the same matrices");
    if ((s0 < w0 + need && w0 < s0 + slen) || (d0 < w0 + need && w0 < d0 + dlen))
        return set_error(NEOX_EINVAL, "the workspace overlaps src or dst");
    if (!std::isfinite(scale) || !std::isfinite((float)scale))
        return set_error(NEOX_EINVAL, "scale %g is not finite", scale);

    const NsShape s = ns_shape(rows, cols, pairs);
    const uint64_t most = std::min(count, launch_count(s));
    const NsBuf w = ns_place(s, most, workspace);
    for (uint64_t z = 0; z < count; z += most) {
        const uint64_t n = std::min(most, count - z);
        const OrthIO io{(const uint8_t*)src + z * src_stride * sb, (uint8_t*)dst + z * dst_stride * db,
                        src_ld, src_stride, dst_ld, dst_stride, src_dtype, dst_dtype, (float)scale,
                        d0 % (4 * db) == 0 && dst_ld % 4 == 0 && (count == 1 || dst_stride % 4 == 0),
                        s0 % (4 * sb) == 0 && src_ld % 4 == 0 && (count == 1 || src_stride % 4 == 0), cfg->eps};
        const hipError_t e = enqueue_orth(s, w, (uint32_t)n, io, coef, cfg->steps,
                                          static_cast<hipStream_t>(hip_stream));
        if (e != hipSuccess) return set_hip_error(e, "orthogonalize launch");
    }
    return NEOX_OK;
}

// ------------------------------------------------------------------------------------
// Muon
// ------------------------------------------------------------------------------------
namespace {

// Matrices of one shape that share the launches: entries [first, first + count) of the table.
struct Group {
    NsShape shape;
    uint32_t first = 0, count = 0;
    float scale = 0.0f;
};

}  // namespace

struct neox_muon {
    int device = 0;
    StepLaunch sl;                        // norm pass and finalize, as a neox_zero1 handle's
    double ns_eps = 0.0;
    int32_t steps = 0, nesterov = 0;
    NsCoef coef[NEOX_NS_MAX_STEPS];
    std::vector<Group> groups;
    std::vector<neox_muon_matrix> mats;   // in table order
    Chunk* d_norm_chunks = nullptr;
    double* d_partial = nullptr;
    DevState* d_state = nullptr;
    MuonMat* d_mats = nullptr;
    void* d_work = nullptr;
    hipStream_t last_stream = nullptr;
};

extern "C" int neox_muon_default_config(neox_muon_config* cfg) {
    if (!cfg) return set_error(NEOX_EINVAL, "cfg is NULL");
    std::memset(cfg, 0, sizeof *cfg);
    const int rc = neox_ns_default_config(&cfg->ns);
    if (rc) return rc;
    cfg->nesterov = 1;
    cfg->scale_mode = NEOX_MUON_SCALE_RMS;
    return NEOX_OK;
}

static void free_muon(neox_muon* h) {
    if (!h) return;
    if (h->d_norm_chunks) (void)hipFree(h->d_norm_chunks);
    if (h->d_partial) (void)hipFree(h->d_partial);
    if (h->d_state) (void)hipFree(h->d_state);
    if (h->d_mats) (void)hipFree(h->d_mats);
    if (h->d_work) (void)hipFree(h->d_work);
    delete h;
}

// MXFP4 pointers: pairs, alignment, and no overlap with any array of the step.
static int check_copies(const neox_muon_matrix* mats, uint64_t n, const std::vector<neox_segment>& segs) {
    struct Range { uintptr_t p; uint64_t bytes; uint64_t mat; bool copy; };
    std::vector<Range> r;
    try {
        r.reserve(8 * n);
    } catch (const std::exception&) {
        return set_error(NEOX_ENOMEM, "host allocation of the overlap check");
    }
    bool any = false;
    for (uint64_t i = 0; i < n; ++i) {
        const neox_muon_matrix& m = mats[i];
        const void* c[2] = {m.mx_codes, m.mx_codes_t};
        const void* s[2] = {m.mx_scales, m.mx_scales_t};
        for (int t = 0; t < 2; ++t) {
            if (!c[t] != !s[t]) return set_error(NEOX_EINVAL, "matrix %llu: half a pair of MXFP4 pointers",
                                                 (unsigned long long)i);
            if (!c[t]) continue;
            if (((uintptr_t)c[t] & 15u) || ((uintptr_t)s[t] & 3u))
                return set_error(NEOX_EINVAL, "matrix %llu: MXFP4 pointers misaligned", (unsigned long long)i);
            const uint64_t rows = t ? m.cols : m.rows;
            const MxShape sh = mx_shape(t ? m.rows : m.cols);
            r.push_back({(uintptr_t)c[t], rows * sh.code_pitch, i, true});
            r.push_back({(uintptr_t)s[t], rows * sh.scale_pitch, i, true});
            any = true;
        }
        const neox_segment& g = segs[i];
        r.push_back({(uintptr_t)g.half, 2 * g.numel, i, false});
        r.push_back({(uintptr_t)g.master, 4 * g.numel, i, false});
        r.push_back({(uintptr_t)g.exp_avg, 4 * g.numel, i, false});
        r.push_back({(uintptr_t)g.grad, 2 * g.numel, i, false});
    }
    if (!any) return NEOX_OK;
    // gradients may overlap one another, so an earlier range may end later than a later one
    std::sort(r.begin(), r.end(), [](const Range& a, const Range& b) { return a.p < b.p; });
    uintptr_t end = 0, copy_end = 0;
    for (const Range& x : r) {
        if (x.p < (x.copy ? end : copy_end))
            return set_error(NEOX_EINVAL, "matrix %llu: an MXFP4 copy overlaps another array",
                             (unsigned long long)x.mat);
        end = std::max(end, x.p + (uintptr_t)x.bytes);
        if (x.copy) copy_end = std::max(copy_end, x.p + (uintptr_t)x.bytes);
    }
    return NEOX_OK;
}

extern "C" int neox_muon_create(const neox_zero1_config* cfg, const neox_muon_config* mcfg,
                                const neox_muon_matrix* mats, uint64_t n, void* hip_stream, neox_muon** out) {
    if (!out) return set_error(NEOX_EINVAL, "out is NULL");
    *out = nullptr;
    if (!cfg || !mcfg || !mats) return set_error(NEOX_EINVAL, "null argument");
    if (n == 0 || n > (1u << 24)) return set_error(NEOX_EINVAL, "%llu matrices: 1 to 2^24", (unsigned long long)n);
    if (cfg->segment_norms) return set_error(NEOX_EINVAL, "segment_norms is not supported here");
    if (cfg->optimizer != NEOX_OPT_ADAMW && cfg->optimizer != NEOX_OPT_SGD)
        return set_error(NEOX_EINVAL, "optimizer %d", cfg->optimizer);
    if (mcfg->nesterov != 0 && mcfg->nesterov != 1) return set_error(NEOX_EINVAL, "nesterov %d", mcfg->nesterov);
    if (mcfg->scale_mode != NEOX_MUON_SCALE_SHAPE && mcfg->scale_mode != NEOX_MUON_SCALE_RMS)
        return set_error(NEOX_EINVAL, "scale_mode %d", mcfg->scale_mode);
    neox_muon* h = new (std::nothrow) neox_muon();
    if (!h) return set_error(NEOX_ENOMEM, "host allocation of the handle");
    struct Guard {
        neox_muon* h;
        ~Guard() { free_muon(h); }
    } guard{h};
    bool pairs = false;
    int rc = ns_coefs(&mcfg->ns, h->coef, &pairs);
    if (rc) return rc;

    Plan plan;
    std::vector<MuonMat> table;
    uint64_t work = 0;
    try {
        std::vector<neox_segment> segs(n);
        for (uint64_t i = 0; i < n; ++i) {
            const neox_muon_matrix& m = mats[i];
            rc = check_sides(m.rows, m.cols);
            if (rc) return rc;
            if (m.reserved) return set_error(NEOX_EINVAL, "matrix %llu: reserved field is not 0", (unsigned long long)i);
            segs[i] = neox_segment{m.grad, m.half, m.master, m.momentum, nullptr, m.rows * m.cols, m.flags, 0, 0};
        }
        // the norm pass, the scaler and the array checks are the momentum-SGD step's
        neox_zero1_config c = *cfg;
        c.optimizer = NEOX_OPT_SGD;
        rc = make_plan(&c, segs.data(), n, plan);
        if (rc) return rc;
        rc = check_copies(mats, n, segs);
        if (rc) return rc;

        // group by shape, in order of first appearance within a shape
        std::map<std::pair<uint64_t, uint64_t>, std::vector<uint64_t>> by;
        for (uint64_t i = 0; i < n; ++i) by[{mats[i].rows, mats[i].cols}].push_back(i);
        const uint64_t cap = mcfg->workspace_bytes ? mcfg->workspace_bytes : kDefaultWorkspace;
        for (const auto& kv : by) {
            const NsShape s = ns_shape(kv.first.first, kv.first.second, pairs);
            uint64_t most = std::min<uint64_t>(kv.second.size(), launch_count(s));
            if (!s.small) {
                most = std::max<uint64_t>(1, std::min<uint64_t>(most, cap / ns_bytes(s, 1)));
                while (most > 1 && ns_bytes(s, most) > cap) --most;
            }
            const double rows = (double)s.rows, cols = (double)s.cols;
            const double f = mcfg->scale_mode == NEOX_MUON_SCALE_RMS ? 0.2 * std::sqrt(std::max(rows, cols))
                                                                     : std::sqrt(std::max(1.0, rows / cols));
            for (uint64_t k = 0; k < kv.second.size(); k += most) {
                Group g;
                g.shape = s;
                g.first = (uint32_t)(table.size());
                g.count = (uint32_t)std::min<uint64_t>(most, kv.second.size() - k);
                g.scale = (float)f;
                for (uint32_t q = 0; q < g.count; ++q) {
                    const neox_muon_matrix& m = mats[kv.second[k + q]];
                    MuonMat t{};
                    t.grad = (const uint16_t*)m.grad;
                    t.half = (uint16_t*)m.half;
                    t.master = m.master;
                    t.mom = m.momentum;
                    t.decay = m.flags & NEOX_SEG_DECAY ? 1u : 0u;
                    t.vec = !(((uintptr_t)m.grad | (uintptr_t)m.half) & 7u) &&
                            !(((uintptr_t)m.master | (uintptr_t)m.momentum) & 15u);
                    table.push_back(t);
                    h->mats.push_back(m);
                }
                h->groups.push_back(g);
                if (!s.small) work = std::max(work, ns_bytes(s, g.count));
            }
        }
    } catch (const std::exception&) {
        return set_error(NEOX_ENOMEM, "host allocation of the matrix table");
    }

    hipError_t e = hipGetDevice(&h->device);
    if (e != hipSuccess) return set_hip_error(e, "hipGetDevice");
    StepLaunch& sl = h->sl;
    rc = lds_reserve(h->device, NEOX_OPT_SGD, 1, &sl.lds);
    if (rc) return rc;
    const uint32_t nnorm = (uint32_t)plan.norm_table.size();
    e = hipMalloc(&h->d_norm_chunks, nnorm * sizeof(Chunk));
    if (e == hipSuccess) e = hipMalloc(&h->d_partial, nnorm * sizeof(double));
    if (e == hipSuccess) e = hipMalloc(&h->d_state, sizeof(DevState));
    if (e == hipSuccess) e = hipMalloc(&h->d_mats, table.size() * sizeof(MuonMat));
    if (e == hipSuccess && work) e = hipMalloc(&h->d_work, work);
    if (e != hipSuccess)
        return e == hipErrorOutOfMemory ? set_error(NEOX_ENOMEM, "hipMalloc of library scratch (%llu bytes)",
                                                    (unsigned long long)work)
                                        : set_hip_error(e, "hipMalloc");
    const DevState st = initial_state(*cfg, (float)cfg->init_scale, cfg->init_good_steps, cfg->init_step,
                                      cfg->init_skipped, cfg->init_consecutive_overflows);
    hipStream_t stream = static_cast<hipStream_t>(hip_stream);
    e = hipMemcpyAsync(h->d_norm_chunks, plan.norm_table.data(), nnorm * sizeof(Chunk), hipMemcpyHostToDevice, stream);
    if (e == hipSuccess)
        e = hipMemcpyAsync(h->d_mats, table.data(), table.size() * sizeof(MuonMat), hipMemcpyHostToDevice, stream);
    if (e == hipSuccess) e = hipMemcpyAsync(h->d_state, &st, sizeof st, hipMemcpyHostToDevice, stream);
    const hipError_t es = hipStreamSynchronize(stream);
    if (e != hipSuccess || es != hipSuccess)
        return set_hip_error(e != hipSuccess ? e : es, "upload of the matrix table");

    sl.dtype = cfg->dtype;
    sl.optimizer = NEOX_OPT_SGD;
    sl.norm_nt = plan.numel > kNormCachedMax;
    sl.norm_big = plan.norm_big;
    sl.norm_chunks = h->d_norm_chunks;
    sl.nnorm = nnorm;
    sl.norm_blocks = nnorm;
    sl.partial = h->d_partial;
    sl.st = h->d_state;
    sl.fin = finalize_args(*cfg);
    sl.upd = update_args(*cfg);
    h->ns_eps = mcfg->ns.eps;
    h->steps = mcfg->ns.steps;
    h->nesterov = mcfg->nesterov;
    h->last_stream = stream;
    guard.h = nullptr;
    *out = h;
    return NEOX_OK;
}

static hipError_t muon_norm(neox_muon* h, hipStream_t stream) {
    const StepLaunch& s = h->sl;
    return launch_norm(s.dtype, s.norm_nt, s.norm_big, s.norm_chunks, s.nnorm, s.norm_blocks, s.st, s.partial,
                       nullptr, s.norm_big ? s.lds.norm_big : s.lds.norm, stream);
}

// Everything after the norm pass, from the squared norms of nparts blocks or ranks.
static hipError_t muon_apply(neox_muon* h, const double* sumsq, uint32_t nparts, float lr, hipStream_t stream) {
    hipError_t e = launch_finalize(sumsq, nparts, h->sl.st, h->sl.fin, stream);
    for (const Group& g : h->groups) {
        if (e != hipSuccess) return e;
        const NsBuf w = g.shape.small ? NsBuf{} : ns_place(g.shape, g.count, h->d_work);
        const MuonIO io{h->d_mats + g.first, h->sl.st, h->sl.dtype, h->nesterov, h->sl.upd.b1, lr,
                        h->sl.upd.wd, g.scale, h->ns_eps};
        e = enqueue_muon(g.shape, w, g.count, io, h->coef, h->steps, stream);
    }
    for (const neox_muon_matrix& m : h->mats) {
        for (int t = 0; t < 2 && e == hipSuccess; ++t) {
            void* codes = t ? m.mx_codes_t : m.mx_codes;
            if (codes)
                e = launch_mx_quantize(m.master, NEOX_F32, m.rows, m.cols, m.cols, t != 0, codes,
                                       t ? m.mx_scales_t : m.mx_scales, h->sl.st, stream);
        }
    }
    return e;
}

extern "C" int neox_muon_step(neox_muon* h, float lr, void* hip_stream) {
    if (!h) return set_error(NEOX_EINVAL, "handle is NULL");
    if (!std::isfinite(lr)) return set_error(NEOX_EINVAL, "lr %g is not finite", (double)lr);
    hipStream_t stream = static_cast<hipStream_t>(hip_stream);
    hipError_t e = muon_norm(h, stream);
    if (e == hipSuccess) e = muon_apply(h, h->sl.partial, h->sl.norm_blocks, lr, stream);
    h->last_stream = stream;
    if (e != hipSuccess) return set_hip_error(e, "muon step launch");
    return NEOX_OK;
}

extern "C" int neox_muon_step_local(neox_muon* h, double* local_sumsq, void* hip_stream) {
    if (!h || !local_sumsq) return set_error(NEOX_EINVAL, "null argument");
    if ((uintptr_t)local_sumsq & 7u) return set_error(NEOX_EINVAL, "local_sumsq not 8-byte aligned");
    hipStream_t stream = static_cast<hipStream_t>(hip_stream);
    hipError_t e = muon_norm(h, stream);
    if (e == hipSuccess) e = launch_reduce(h->sl.partial, h->sl.norm_blocks, local_sumsq, stream);
    h->last_stream = stream;
    if (e != hipSuccess) return set_hip_error(e, "muon step_local launch");
    return NEOX_OK;
}

extern "C" int neox_muon_step_apply(neox_muon* h, const double* rank_sumsq, uint32_t nranks, float lr,
                                    void* hip_stream) {
    if (!h || !rank_sumsq) return set_error(NEOX_EINVAL, "null argument");
    if (nranks == 0 || nranks > (1u << 24)) return set_error(NEOX_EINVAL, "nranks %u not in [1, 2^24]", nranks);
    if ((uintptr_t)rank_sumsq & 7u) return set_error(NEOX_EINVAL, "rank_sumsq not 8-byte aligned");
    if (!std::isfinite(lr)) return set_error(NEOX_EINVAL, "lr %g is not finite", (double)lr);
    hipStream_t stream = static_cast<hipStream_t>(hip_stream);
    const hipError_t e = muon_apply(h, rank_sumsq, nranks, lr, stream);
    h->last_stream = stream;
    if (e != hipSuccess) return set_hip_error(e, "muon step_apply launch");
    return NEOX_OK;
}

extern "C" int neox_muon_state(neox_muon* h, neox_scaler_state_t* out) {
    if (!h || !out) return set_error(NEOX_EINVAL, "null argument");
    hipError_t e = hipStreamSynchronize(h->last_stream);
    if (e != hipSuccess) return set_hip_error(e, "hipStreamSynchronize");
    DevState st;
    e = hipMemcpy(&st, h->d_state, sizeof st, hipMemcpyDeviceToHost);
    if (e != hipSuccess) return set_hip_error(e, "state readback");
    out->loss_scale = st.loss_scale;
    out->good_steps = st.good_steps;
    out->step = st.step;
    out->skipped_total = st.skipped_total;
    out->consecutive_overflows = st.consecutive_overflows;
    out->last_skipped = st.last_skipped;
    out->last_grad_norm = st.last_grad_norm;
    out->last_clip_coef = st.last_clip_coef;
    out->last_sumsq = st.last_sumsq;
    out->device_loss_scale = &h->d_state->loss_scale;
    return NEOX_OK;
}

extern "C" int neox_muon_scaler_set(neox_muon* h, const neox_scaler_state_t* st, void* hip_stream) {
    if (!h || !st) return set_error(NEOX_EINVAL, "null argument");
    if (!(std::isfinite(st->loss_scale) && st->loss_scale > 0.0f))
        return set_error(NEOX_EINVAL, "loss_scale %g", (double)st->loss_scale);
    if (st->good_steps < 0 || st->step < 0 || st->skipped_total < 0 || st->consecutive_overflows < 0)
        return set_error(NEOX_EINVAL, "negative counter");
    hipStream_t stream = static_cast<hipStream_t>(hip_stream);
    const hipError_t e = launch_set_state(h->d_state, st->loss_scale, st->good_steps, st->step,
                                          st->skipped_total, st->consecutive_overflows,
                                          h->sl.fin.predivide_factor, h->sl.fin.dp_world_size, stream);
    h->last_stream = stream;
    if (e != hipSuccess) return set_hip_error(e, "scaler_set launch");
    return NEOX_OK;
}

extern "C" int neox_muon_destroy(neox_muon* h) {
    if (!h) return NEOX_OK;
    const hipError_t e = hipStreamSynchronize(h->last_stream);
    free_muon(h);
    if (e != hipSuccess) return set_hip_error(e, "hipStreamSynchronize");
    return NEOX_OK;
}

// ------------------------------------------------------------------------------------
// MXFP4
// ------------------------------------------------------------------------------------
static int mx_sides(uint64_t rows, uint64_t cols) {
    if (rows == 0 || cols == 0 || rows > kMaxMx || cols > kMaxMx)
        return set_error(NEOX_EINVAL, "a copy of %llu x %llu: sides of 1 to 2^31 - 1",
                         (unsigned long long)rows, (unsigned long long)cols);
    // bytes of the codes and offsets in them stay far from 64 bits
    if (rows > (1ull << 40) / mx_shape(cols).code_pitch)
        return set_error(NEOX_EINVAL, "a copy of %llu x %llu is too large", (unsigned long long)rows,
                         (unsigned long long)cols);
    return NEOX_OK;
}

static int mx_dense(const void* p, int32_t dtype, uint64_t rows, uint64_t cols, uint64_t ld) {
    if (!known_type(dtype)) return set_error(NEOX_EINVAL, "type %d", dtype);
    if ((uintptr_t)p % type_bytes(dtype)) return set_error(NEOX_EINVAL, "matrix misaligned");
    if (ld < cols || ld > (1ull << 60) / rows) return set_error(NEOX_EINVAL, "ld %llu", (unsigned long long)ld);
    return NEOX_OK;
}

static int mx_pair(const void* codes, const void* scales) {
    if (!codes || !scales) return set_error(NEOX_EINVAL, "null argument");
    if (((uintptr_t)codes & 15u) || ((uintptr_t)scales & 3u))
        return set_error(NEOX_EINVAL, "codes not 16-byte or scales not 4-byte aligned");
    return NEOX_OK;
}

static bool meet(const void* a, uint64_t an, const void* b, uint64_t bn) {
    return (uintptr_t)a < (uintptr_t)b + bn && (uintptr_t)b < (uintptr_t)a + an;
}

extern "C" int neox_mxfp4_layout(uint64_t rows, uint64_t cols, uint64_t* code_bytes, uint64_t* scale_bytes) {
    if (!code_bytes || !scale_bytes) return set_error(NEOX_EINVAL, "null argument");
    const int rc = mx_sides(rows, cols);
    if (rc) return rc;
    const MxShape s = mx_shape(cols);
    *code_bytes = rows * s.code_pitch;
    *scale_bytes = rows * s.scale_pitch;
    return NEOX_OK;
}

extern "C" int neox_mxfp4_quantize(const void* src, int32_t dtype, uint64_t rows, uint64_t cols, uint64_t ld,
                                   int32_t transpose, void* codes, void* scales, void* hip_stream) {
    if (transpose != 0 && transpose != 1) return set_error(NEOX_EINVAL, "transpose %d", transpose);
    if (!src) return set_error(NEOX_EINVAL, "null argument");
    int rc = mx_pair(codes, scales);
    if (!rc) rc = transpose ? mx_sides(cols, rows) : mx_sides(rows, cols);
    if (!rc) rc = mx_dense(src, dtype, rows, cols, ld);
    if (rc) return rc;
    const uint64_t R = transpose ? cols : rows;
    const MxShape s = mx_shape(transpose ? rows : cols);
    const uint64_t span = ((rows - 1) * ld + cols) * type_bytes(dtype);
    if (meet(src, span, codes, R * s.code_pitch) || meet(src, span, scales, R * s.scale_pitch) ||
        meet(codes, R * s.code_pitch, scales, R * s.scale_pitch))
        return set_error(NEOX_EINVAL, "src, codes and scales overlap");
    const hipError_t e = launch_mx_quantize(src, dtype, rows, cols, ld, transpose != 0, codes, scales, nullptr,
                                            static_cast<hipStream_t>(hip_stream));
    if (e != hipSuccess) return set_hip_error(e, "mxfp4_quantize launch");
    return NEOX_OK;
}

extern "C" int neox_mxfp4_dequantize(const void* codes, const void* scales, uint64_t rows, uint64_t cols,
                                     void* dst, int32_t dtype, uint64_t ld, void* hip_stream) {
    if (!dst) return set_error(NEOX_EINVAL, "null argument");
    int rc = mx_pair(codes, scales);
    if (!rc) rc = mx_sides(rows, cols);
    if (!rc) rc = mx_dense(dst, dtype, rows, cols, ld);
    if (rc) return rc;
    const MxShape s = mx_shape(cols);
    const uint64_t span = ((rows - 1) * ld + cols) * type_bytes(dtype);
    if (meet(dst, span, codes, rows * s.code_pitch) || meet(dst, span, scales, rows * s.scale_pitch))
        return set_error(NEOX_EINVAL, "dst overlaps the copy");
    const hipError_t e = launch_mx_dequantize(codes, scales, rows, cols, dst, dtype, ld,
                                              static_cast<hipStream_t>(hip_stream));
    if (e != hipSuccess) return set_hip_error(e, "mxfp4_dequantize launch");
    return NEOX_OK;
}

extern "C" int neox_mxfp4_product(const void* a_codes, const void* a_scales, uint64_t m, const void* b_codes,
                                  const void* b_scales, uint64_t n, uint64_t k, void* c, int32_t dtype,
                                  uint64_t ldc, void* hip_stream) {
    if (!c) return set_error(NEOX_EINVAL, "null argument");
    int rc = mx_pair(a_codes, a_scales);
    if (!rc) rc = mx_pair(b_codes, b_scales);
    if (!rc) rc = mx_sides(m, k);
    if (!rc) rc = mx_sides(n, k);
    if (rc) return rc;
    if (k > kMaxK) return set_error(NEOX_EINVAL, "k %llu: at most 2^24", (unsigned long long)k);
    rc = mx_dense(c, dtype, m, n, ldc);
    if (rc) return rc;
    if (((m + 127) / 128) * ((n + 127) / 128) >= kMaxTiles)
        return set_error(NEOX_EINVAL, "a result of %llu x %llu is too large", (unsigned long long)m,
                         (unsigned long long)n);
    const MxShape s = mx_shape(k);
    const uint64_t span = ((m - 1) * ldc + n) * type_bytes(dtype);
    if (meet(c, span, a_codes, m * s.code_pitch) || meet(c, span, a_scales, m * s.scale_pitch) ||
        meet(c, span, b_codes, n * s.code_pitch) || meet(c, span, b_scales, n * s.scale_pitch))
        return set_error(NEOX_EINVAL, "c overlaps an operand");
    const hipError_t e = launch_mx_product(a_codes, a_scales, m, b_codes, b_scales, n, k, c, dtype, ldc,
                                           static_cast<hipStream_t>(hip_stream));
    if (e != hipSuccess) return set_hip_error(e, "mxfp4_product launch");
    return NEOX_OK;
}
