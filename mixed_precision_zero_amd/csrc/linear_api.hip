// linear_api.hip -- host side of include/neox_linear.h: argument validation and workspace
// layout.
#include "linear_internal.h"

#include <algorithm>
#include <cmath>

using namespace nz1;

namespace {

constexpr uint64_t kMaxSide = 1ull << 22;       // n, k: a tile's 256 rows of one are below 2^31 bytes
constexpr uint64_t kMaxTokens = 1ull << 24;
constexpr uint64_t kMaxTiles = 1ull << 23;      // 64 x 64 tiles of a result: blocks of one grid
constexpr uint64_t kMaxLd = 1ull << 40;
constexpr uint64_t kMaxMx = (1ull << 31) - 1;
constexpr uint64_t kMaxMxK = 1ull << 24;
constexpr uint64_t kMaxMxTiles = 1ull << 23;    // 128 x 128 tiles of an MXFP4 product

bool half_type(int32_t t) { return t == NEOX_F16 || t == NEOX_BF16; }
bool known_type(int32_t t) { return half_type(t) || t == NEOX_F32; }
uint64_t type_bytes(int32_t t) { return t == NEOX_F32 ? 4 : 2; }
uint64_t round_up(uint64_t v, uint64_t to) { return (v + to - 1) / to * to; }

// A matrix in memory, in bytes.
struct Area {
    const char* name;
    uintptr_t at;
    uint64_t rows, pitch, width;
    uint64_t span() const { return rows == 0 ? 0 : (rows - 1) * pitch + width; }
};
// Whether two matrices share no byte: one lies behind the other, or they lie side by side in
// rows of one pitch.
bool apart(const Area& a, const Area& b) {
    if (a.span() == 0 || b.span() == 0) return true;
    if (a.at + a.span() <= b.at || b.at + b.span() <= a.at) return true;
    // (of a single row only the width counts, so it can take the other's pitch)
    const uint64_t pitch = a.rows > 1 ? a.pitch : b.pitch;
    if ((a.rows > 1 && b.rows > 1 && a.pitch != b.pitch) || pitch == 0) return false;
    const uint64_t from_a = a.at <= b.at ? (b.at - a.at) % pitch : (pitch - (a.at - b.at) % pitch) % pitch;
    return from_a >= a.width && from_a + b.width <= pitch;
}

// Collects a call's arrays, checking each by itself, then against the ones that are written.
struct Arrays {
    Area in[8], out[8];
    int ins = 0, outs = 0;
    int rc = NEOX_OK;

    Area make(const char* name, const void* p, uint64_t rows, uint64_t cols, uint64_t ld, uint64_t size) {
        if (rc) return Area{};
        if (rows == 0) return Area{name, 0, 0, 0, 0};
        if (!p) {
            rc = set_error(NEOX_EINVAL, "%s is null", name);
        } else if ((uintptr_t)p % size) {
            rc = set_error(NEOX_EINVAL, "%s is misaligned", name);
        } else if (rows > 1 && ld < cols) {
            rc = set_error(NEOX_EINVAL, "%s: ld %llu smaller than its %llu columns", name, (unsigned long long)ld,
                           (unsigned long long)cols);
        } else if (rows > 1 && ld > kMaxLd) {
            rc = set_error(NEOX_EINVAL, "%s: ld %llu above 2^40", name, (unsigned long long)ld);
        } else if (rows > 1 && ld > (1ull << 60) / (rows - 1)) {
            rc = set_error(NEOX_EINVAL, "%s: ld %llu too large for %llu rows", name, (unsigned long long)ld,
                           (unsigned long long)rows);
        }
        return Area{name, (uintptr_t)p, rows, (rows > 1 ? ld : cols) * size, cols * size};
    }
    void reads(const char* name, const void* p, uint64_t rows, uint64_t cols, uint64_t ld, uint64_t size) {
        in[ins++] = make(name, p, rows, cols, ld, size);
    }
    void writes(const char* name, void* p, uint64_t rows, uint64_t cols, uint64_t ld, uint64_t size) {
        out[outs++] = make(name, p, rows, cols, ld, size);
    }
    // an input that may be output `o` itself
    void reads_or_is(int o, const char* name, const void* p, uint64_t rows, uint64_t cols, uint64_t ld, uint64_t size) {
        const Area a = make(name, p, rows, cols, ld, size);
        if (!rc && a.at == out[o].at && a.pitch == out[o].pitch && a.width == out[o].width) return;
        in[ins++] = a;
    }
    int check() {
        for (int o = 0; o < outs && !rc; ++o) {
            for (int i = 0; i < ins && !rc; ++i)
                if (!apart(out[o], in[i])) rc = set_error(NEOX_EINVAL, "%s meets %s", out[o].name, in[i].name);
            for (int i = 0; i < o && !rc; ++i)
                if (!apart(out[o], out[i])) rc = set_error(NEOX_EINVAL, "%s meets %s", out[o].name, out[i].name);
        }
        return rc;
    }
    int check_workspace(void* p, uint64_t bytes, uint64_t need) {
        if (rc || check() || need == 0) return rc;
        if (!p) return rc = set_error(NEOX_EINVAL, "the workspace is null, %llu bytes needed", (unsigned long long)need);
        if ((uintptr_t)p & 255u) return rc = set_error(NEOX_EINVAL, "workspace not 256-byte aligned");
        if (bytes < need)
            return rc = set_error(NEOX_EINVAL, "workspace of %llu bytes, %llu needed", (unsigned long long)bytes,
                                  (unsigned long long)need);
        const Area w{"the workspace", (uintptr_t)p, 1, need, need};
        for (int i = 0; i < ins && !rc; ++i)
            if (!apart(w, in[i])) rc = set_error(NEOX_EINVAL, "the workspace meets %s", in[i].name);
        for (int o = 0; o < outs && !rc; ++o)
            if (!apart(w, out[o])) rc = set_error(NEOX_EINVAL, "the workspace meets %s", out[o].name);
        return rc;
    }
};

int take_drop(const neox_drop* d, Drop& out) {
    out = Drop{};
    if (!d) return NEOX_OK;
    if (!(d->p >= 0.0 && d->p <= 1.0)) return set_error(NEOX_EINVAL, "p %g not in [0, 1]", d->p);
    out.limit = (uint32_t)std::nearbyint(d->p * 65536.0);
    if (out.limit == 0) return NEOX_OK;
    if ((uintptr_t)d->counter & 7u) return set_error(NEOX_EINVAL, "the counter is misaligned");
    out.scale = out.limit == 65536u ? 0.0f : (float)(65536.0 / (65536.0 - out.limit));
    out.seed[0] = (uint32_t)d->seed;
    out.seed[1] = (uint32_t)(d->seed >> 32);
    out.offset = d->offset;
    out.counter = d->counter;
    return NEOX_OK;
}

int check_act(int32_t act) {
    if (act < NEOX_ACT_NONE || act > NEOX_ACT_SILU) return set_error(NEOX_EINVAL, "act %d", act);
    return NEOX_OK;
}

// Takes the epilogue of an m x n result (output 0 of arr) of type y_dtype.
int take_epilogue(const neox_epilogue& e, uint64_t m, uint64_t n, int32_t y_dtype, Arrays& arr, Epilogue& out) {
    if (!half_type(e.dtype)) return set_error(NEOX_EINVAL, "type %d of the epilogue", e.dtype);
    int rc = check_act(e.act);
    if (rc) return rc;
    rc = take_drop(&e.drop, out.drop);
    if (rc) return rc;
    out.act = e.act;
    out.bias = (const uint16_t*)e.bias;
    out.residual = m ? e.residual : nullptr;
    out.residual_ld = e.residual_ld;
    out.pre = m ? (uint16_t*)e.pre : nullptr;
    out.pre_ld = e.pre_ld;
    if (e.bias) arr.reads("bias", e.bias, 1, n, n, 2);
    if (out.residual) arr.reads_or_is(0, "the residual", e.residual, m, n, e.residual_ld, type_bytes(y_dtype));
    if (out.pre) arr.writes("pre", e.pre, m, n, e.pre_ld, 2);
    if (out.drop.counter) arr.reads("the counter", out.drop.counter, 1, 1, 1, 8);
    return arr.rc;
}

uint64_t tiles(uint64_t a, uint64_t b) { return ((a + 63) / 64) * ((b + 63) / 64); }

int check_sizes(uint64_t m, uint64_t n, uint64_t k) {
    if (n < 1 || n > kMaxSide || k < 1 || k > kMaxSide)
        return set_error(NEOX_EINVAL, "n %llu, k %llu not in [1, 2^22]", (unsigned long long)n, (unsigned long long)k);
    if (m > kMaxTokens) return set_error(NEOX_EINVAL, "m %llu above 2^24", (unsigned long long)m);
    return NEOX_OK;
}
int check_tiles(const char* what, uint64_t rows, uint64_t cols) {
    if (tiles(rows, cols) > kMaxTiles)
        return set_error(NEOX_EINVAL, "%s of %llu x %llu: more than 2^23 tiles of 64 x 64", what,
                         (unsigned long long)rows, (unsigned long long)cols);
    return NEOX_OK;
}

int take_linear(const neox_linear_args* a, Arrays& arr, Product& p) {
    if (!a) return set_error(NEOX_EINVAL, "null argument");
    int rc = check_sizes(a->m, a->n, a->k);
    if (!rc) rc = check_tiles("y", a->m, a->n);
    if (rc) return rc;
    if (a->reserved) return set_error(NEOX_EINVAL, "reserved field %d is not 0", a->reserved);
    if (a->y_dtype != NEOX_F32 && a->y_dtype != a->epi.dtype)
        return set_error(NEOX_EINVAL, "y of type %d for operands of type %d", a->y_dtype, a->epi.dtype);
    p = Product{};
    arr.writes("y", a->y, a->m, a->n, a->y_ld, type_bytes(a->y_dtype));
    rc = take_epilogue(a->epi, a->m, a->n, a->y_dtype, arr, p.epi);
    if (rc) return rc;
    arr.reads("x", a->x, a->m, a->k, a->x_ld, 2);
    arr.reads("w", a->w, a->n, a->k, a->w_ld, 2);
    if (arr.check()) return arr.rc;
    p.p = Operand{(const uint16_t*)a->w, a->n > 1 ? a->w_ld : a->k, false, false};
    p.q = Operand{(const uint16_t*)a->x, a->m > 1 ? a->x_ld : a->k, false, false};
    p.I = (uint32_t)a->n;
    p.J = (uint32_t)a->m;
    p.K = a->k;
    p.dtype = a->epi.dtype;
    p.out_dtype = a->y_dtype;
    p.out = a->y;
    p.out_ld = a->y_ld;
    p.scale = 1.0f;
    return NEOX_OK;
}

// A backward call: what each launch takes and where it lies in the workspace.
struct Gradients {
    Backward d{};              // the element-wise pass
    bool pass = false;         // ... if there is one
    Product dx{}, dw{};
    bool has_dx = false, has_dw = false;
    uint64_t d_bytes = 0;      // d itself, if it is not dy
    uint64_t sums_bytes = 0;   // the parts of dbias
    uint64_t bytes = 0;        // in all
};

int take_gradients(const neox_linear_grads* a, Arrays& arr, Gradients& g) {
    if (!a) return set_error(NEOX_EINVAL, "null argument");
    int rc = check_sizes(a->m, a->n, a->k);
    if (!rc && a->dx) rc = check_tiles("dx", a->m, a->k);
    if (!rc && a->dw) rc = check_tiles("dw", a->n, a->k);
    if (!rc) rc = check_act(a->act);
    if (rc) return rc;
    if (!half_type(a->dtype)) return set_error(NEOX_EINVAL, "type %d", a->dtype);
    if (a->accumulate != 0 && a->accumulate != 1) return set_error(NEOX_EINVAL, "accumulate %d", a->accumulate);
    if (a->reserved) return set_error(NEOX_EINVAL, "reserved field %d is not 0", a->reserved);
    if (!a->dx && !a->dw && !a->dbias && a->m) return set_error(NEOX_EINVAL, "no gradient is asked for");
    const uint64_t m = a->m, n = a->n, k = a->k;
    Backward& b = g.d;
    rc = take_drop(&a->drop, b.drop);
    if (rc) return rc;
    const bool act = a->act != NEOX_ACT_NONE;
    if (a->dx) arr.writes("dx", a->dx, m, k, a->dx_ld, 2);
    if (a->dw) arr.writes("dw", a->dw, n, k, a->dw_ld, 2);
    if (a->dbias) arr.writes("dbias", a->dbias, 1, n, n, 2);
    arr.reads("dy", a->dy, m, n, a->dy_ld, 2);
    if (act) arr.reads("pre", a->pre, m, n, a->pre_ld, 2);
    if (a->dw) arr.reads("x", a->x, m, k, a->x_ld, 2);
    if (a->dx) arr.reads("w", a->w, n, k, a->w_ld, 2);
    if (b.drop.counter) arr.reads("the counter", b.drop.counter, 1, 1, 1, 8);
    if (arr.check()) return arr.rc;

    // (nothing is added to what is there: even a zero sum would turn a -0 into 0)
    const bool sums = m || !a->accumulate;
    g.has_dx = a->dx && m;
    g.has_dw = a->dw && sums;
    const bool made = (act || b.drop.limit) && (g.has_dx || g.has_dw) && m;
    g.pass = made || (a->dbias && sums);
    // rows of d are whole lines of 128 bytes
    const uint64_t d_ld = round_up(n, 64);
    g.d_bytes = made ? round_up(m * d_ld * 2, 256) : 0;
    b.dy = a->dy;
    b.pre = act ? (const uint16_t*)a->pre : nullptr;
    b.dbias = a->dbias;
    b.dy_ld = m > 1 ? a->dy_ld : n;
    b.pre_ld = m > 1 ? a->pre_ld : n;
    b.d_ld = d_ld;
    b.rows = m;
    b.cols = n;
    b.dtype = a->dtype;
    b.act = a->act;
    b.accumulate = a->accumulate != 0;
    b.padded = made;
    // (p = 1: nothing is kept, the factor is zero)
    const float scale = b.drop.limit ? b.drop.scale : 1.0f;
    b.scale = scale;
    b.drop.scale = 1.0f;

    auto product = [&](Operand p, Operand q, uint64_t I, uint64_t J, uint64_t K, void* out, uint64_t out_ld) {
        Product r{};
        r.p = p;
        r.q = q;
        r.I = (uint32_t)I;
        r.J = (uint32_t)J;
        r.K = K;
        r.dtype = r.out_dtype = a->dtype;
        r.out = out;
        r.out_ld = out_ld;
        r.scale = scale;
        return r;
    };
    // (d's place is filled in when the workspace is known; its alignment is the workspace's)
    const Operand dy{made ? nullptr : (const uint16_t*)a->dy, made ? d_ld : b.dy_ld, false, made};
    if (g.has_dx)
        g.dx = product(Operand{(const uint16_t*)a->w, n > 1 ? a->w_ld : k, true, false}, dy, k, m, n, a->dx,
                       m > 1 ? a->dx_ld : k);
    if (g.has_dw) {
        g.dw = product(Operand{(const uint16_t*)a->x, m > 1 ? a->x_ld : k, true, false}, Operand{dy.at, dy.ld, true, made}, k, n, m,
                       a->dw, n > 1 ? a->dw_ld : k);
        if (a->accumulate) {
            g.dw.epi.residual = a->dw;
            g.dw.epi.residual_ld = g.dw.out_ld;
        }
    }
    g.sums_bytes = a->dbias ? backward_workspace(m, n) : 0;
    g.bytes = g.d_bytes + g.sums_bytes + products_workspace(g.has_dx ? &g.dx : nullptr, g.has_dw ? &g.dw : nullptr);
    return NEOX_OK;
}

}  // namespace

extern "C" int neox_linear_workspace(const neox_linear_args* a, uint64_t* bytes) {
    if (!bytes) return set_error(NEOX_EINVAL, "bytes is NULL");
    Arrays arr;
    Product p;
    const int rc = take_linear(a, arr, p);
    if (rc) return rc;
    *bytes = p.J ? products_workspace(&p, nullptr) : 0;
    return NEOX_OK;
}

extern "C" int neox_linear(const neox_linear_args* a, void* workspace, uint64_t workspace_bytes, void* hip_stream) {
    Arrays arr;
    Product p;
    int rc = take_linear(a, arr, p);
    if (rc) return rc;
    if (p.J == 0) return NEOX_OK;
    rc = arr.check_workspace(workspace, workspace_bytes, products_workspace(&p, nullptr));
    if (rc) return rc;
    const hipError_t e = launch_products(&p, nullptr, nullptr, nullptr, workspace, static_cast<hipStream_t>(hip_stream));
    return e == hipSuccess ? NEOX_OK : set_hip_error(e, "linear launch");
}

extern "C" int neox_linear_backward_workspace(const neox_linear_grads* a, uint64_t* bytes) {
    if (!bytes) return set_error(NEOX_EINVAL, "bytes is NULL");
    Arrays arr;
    Gradients g;
    const int rc = take_gradients(a, arr, g);
    if (rc) return rc;
    *bytes = g.bytes;
    return NEOX_OK;
}

extern "C" int neox_linear_backward(const neox_linear_grads* a, void* workspace, uint64_t workspace_bytes,
                                    void* hip_stream) {
    Arrays arr;
    Gradients g;
    int rc = take_gradients(a, arr, g);
    if (rc) return rc;
    rc = arr.check_workspace(workspace, workspace_bytes, g.bytes);
    if (rc) return rc;
    const hipStream_t s = static_cast<hipStream_t>(hip_stream);
    uint8_t* sums = (uint8_t*)workspace + g.d_bytes;
    if (g.d_bytes) {
        g.d.d = workspace;
        g.dx.q.at = g.dw.q.at = (const uint16_t*)workspace;
    }
    const bool products = g.has_dx || g.has_dw;
    hipError_t e = hipSuccess;
    if (g.pass) e = launch_backward(g.d, sums, !products, s);
    if (e == hipSuccess && products)
        e = launch_products(g.has_dx ? &g.dx : nullptr, g.has_dw ? &g.dw : nullptr, g.sums_bytes ? &g.d : nullptr, sums,
                            sums + g.sums_bytes, s);
    return e == hipSuccess ? NEOX_OK : set_hip_error(e, "linear_backward launch");
}

extern "C" int neox_mxfp4_linear(const void* a_codes, const void* a_scales, uint64_t m, const void* b_codes,
                                 const void* b_scales, uint64_t n, uint64_t k, void* c, int32_t dtype, uint64_t ldc,
                                 const neox_epilogue* epi, void* hip_stream) {
    if (!a_codes || !a_scales || !b_codes || !b_scales || !c || !epi) return set_error(NEOX_EINVAL, "null argument");
    if (((uintptr_t)a_codes & 15u) || ((uintptr_t)a_scales & 3u) || ((uintptr_t)b_codes & 15u) ||
        ((uintptr_t)b_scales & 3u))
        return set_error(NEOX_EINVAL, "codes or scales misaligned");
    if (m < 1 || m > kMaxMx || n < 1 || n > kMaxMx || k < 1 || k > kMaxMxK)
        return set_error(NEOX_EINVAL, "a product of %llu x %llu over %llu", (unsigned long long)m, (unsigned long long)n,
                         (unsigned long long)k);
    if (dtype != NEOX_F32 && dtype != epi->dtype)
        return set_error(NEOX_EINVAL, "c of type %d with an epilogue of type %d", dtype, epi->dtype);
    const MxShape sh = mx_shape(k);
    if (std::max(m, n) > (1ull << 40) / sh.code_pitch) return set_error(NEOX_EINVAL, "codes of more than 2^40 bytes");
    if (((m + 127) / 128) * ((n + 127) / 128) >= kMaxMxTiles)
        return set_error(NEOX_EINVAL, "a result of %llu x %llu is too large", (unsigned long long)m,
                         (unsigned long long)n);
    Arrays arr;
    Epilogue e{};
    arr.writes("c", c, m, n, ldc, type_bytes(dtype));
    const int rc = take_epilogue(*epi, m, n, dtype, arr, e);
    if (rc) return rc;
    arr.reads("a's codes", a_codes, 1, m * sh.code_pitch, 0, 1);
    arr.reads("a's scales", a_scales, 1, m * sh.scale_pitch, 0, 1);
    arr.reads("b's codes", b_codes, 1, n * sh.code_pitch, 0, 1);
    arr.reads("b's scales", b_scales, 1, n * sh.scale_pitch, 0, 1);
    if (arr.check()) return arr.rc;
    const hipError_t err = launch_mx_linear(a_codes, a_scales, m, b_codes, b_scales, n, k, c, dtype, ldc, epi->dtype, e,
                                            static_cast<hipStream_t>(hip_stream));
    return err == hipSuccess ? NEOX_OK : set_hip_error(err, "mxfp4_linear launch");
}

namespace {

int check_rows(uint64_t rows, uint64_t cols, int32_t dtype) {
    if (rows > kMaxMx || cols < 1 || cols > kMaxMx)
        return set_error(NEOX_EINVAL, "a matrix of %llu x %llu", (unsigned long long)rows, (unsigned long long)cols);
    if (!known_type(dtype)) return set_error(NEOX_EINVAL, "type %d", dtype);
    return NEOX_OK;
}

}  // namespace

extern "C" int neox_dropout(const void* x, uint64_t x_ld, const void* bias, const void* residual, uint64_t residual_ld,
                            void* y, uint64_t y_ld, uint64_t rows, uint64_t cols, int32_t dtype, const neox_drop* drop,
                            void* hip_stream) {
    int rc = check_rows(rows, cols, dtype);
    Drop d;
    if (!rc) rc = take_drop(drop, d);
    if (rc || rows == 0) return rc;
    const uint64_t size = type_bytes(dtype);
    Arrays arr;
    arr.writes("y", y, rows, cols, y_ld, size);
    arr.reads_or_is(0, "x", x, rows, cols, x_ld, size);
    if (bias) arr.reads("bias", bias, 1, cols, cols, size);
    if (residual) arr.reads_or_is(0, "the residual", residual, rows, cols, residual_ld, size);
    if (d.counter) arr.reads("the counter", d.counter, 1, 1, 1, 8);
    if (arr.check()) return arr.rc;
    const hipError_t e = launch_dropout(x, x_ld, bias, residual, residual_ld, y, y_ld, rows, cols, dtype, d,
                                        static_cast<hipStream_t>(hip_stream));
    return e == hipSuccess ? NEOX_OK : set_hip_error(e, "dropout launch");
}

extern "C" int neox_dropout_backward_workspace(uint64_t rows, uint64_t cols, uint64_t* bytes) {
    if (!bytes) return set_error(NEOX_EINVAL, "bytes is NULL");
    const int rc = check_rows(rows, cols, NEOX_F32);
    if (rc) return rc;
    *bytes = backward_workspace(rows, cols);
    return NEOX_OK;
}

extern "C" int neox_dropout_backward(const void* dy, uint64_t dy_ld, void* dx, uint64_t dx_ld, void* dbias,
                                     int32_t accumulate, uint64_t rows, uint64_t cols, int32_t dtype,
                                     const neox_drop* drop, void* workspace, uint64_t workspace_bytes,
                                     void* hip_stream) {
    int rc = check_rows(rows, cols, dtype);
    Backward b{};
    if (!rc) rc = take_drop(drop, b.drop);
    if (rc) return rc;
    if (accumulate != 0 && accumulate != 1) return set_error(NEOX_EINVAL, "accumulate %d", accumulate);
    if (!dx && !dbias && rows) return set_error(NEOX_EINVAL, "no gradient is asked for");
    const uint64_t size = type_bytes(dtype);
    Arrays arr;
    if (dx) arr.writes("dx", dx, rows, cols, dx_ld, size);
    if (dx) arr.reads_or_is(0, "dy", dy, rows, cols, dy_ld, size);
    else arr.reads("dy", dy, rows, cols, dy_ld, size);
    if (dbias) arr.writes("dbias", dbias, 1, cols, cols, size);
    if (b.drop.counter) arr.reads("the counter", b.drop.counter, 1, 1, 1, 8);
    rc = arr.check();
    if (!rc) rc = arr.check_workspace(workspace, workspace_bytes, dbias ? backward_workspace(rows, cols) : 0);
    if (rc) return rc;
    if (rows == 0 && (!dbias || accumulate)) return NEOX_OK;        // as in take_gradients
    b.dy = dy;
    b.d = rows ? dx : nullptr;
    b.dbias = dbias;
    b.dy_ld = dy_ld;
    b.d_ld = dx_ld;
    b.rows = rows;
    b.cols = cols;
    b.dtype = dtype;
    b.accumulate = accumulate != 0;
    b.scale = 1.0f;                                   // (dx itself is D(dy))
    const hipError_t e = launch_backward(b, workspace, true, static_cast<hipStream_t>(hip_stream));
    return e == hipSuccess ? NEOX_OK : set_hip_error(e, "dropout_backward launch");
}
