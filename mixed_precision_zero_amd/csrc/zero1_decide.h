// zero1_decide.h -- a step's decisions (skip, clip coefficient, step count, bias corrections,
// loss scale) from its squared norm, on the device: what the finalize kernel and every kernel
// that decides for itself evaluate, with the same bits.
#pragma once

#include "zero1_internal.h"

namespace nz1 {

__device__ __forceinline__ bool f64_finite(double x) {
    return (__double_as_longlong(x) & 0x7FF0000000000000ll) != 0x7FF0000000000000ll;
}
__device__ __forceinline__ bool f32_finite(float x) {
    return (__float_as_uint(x) & 0x7F800000u) != 0x7F800000u;
}

// Block size of every fixed-order sum of the partials (the finalize and the split step's
// reduce), so both add in the same order.
constexpr int kFinalizeBlock = kBlock;

// b^t for an integer t >= 1 by binary exponentiation: at most ~2 log2(t) roundings
// (a few ulps), and a short dependent chain for the one thread that runs it.
__device__ __forceinline__ double ipow(double b, int64_t t) {
    double r = 1.0;
    while (t) {
        if (t & 1) r *= b;
        b *= b;
        t >>= 1;
    }
    return r;
}

// The scaler state a step starts from.
struct PreState {
    float scale;
    float inv;                   // unscale factor the norm pass used
    int32_t good;
    int32_t consecutive;
    int64_t step;
    int64_t skipped;
};
__device__ __forceinline__ PreState read_pre(const DevState* __restrict__ st) {
    return PreState{st->loss_scale, st->inv, st->good_steps, st->consecutive_overflows,
                    st->step, st->skipped_total};
}

// The step's decisions from its squared norm: skip, clip coefficient, step count, bias
// corrections and the loss-scale state machine.  A pure function of its inputs, so every
// thread that evaluates it gets the same bits.
struct Decision {
    DevState next;               // the state block after the step
};
__device__ __forceinline__ Decision decide(double sumsq, const PreState& p, const FinalizeArgs& a) {
    Decision d;
    DevState& n = d.next;
    float scale = p.scale;
    if (!f64_finite(sumsq)) {
        // overflow: skip, back off (not below the floor), restart the clean count
        n.skip = 1;
        n.gscale = 0.0f;
        n.rbc1 = 0.0f;
        n.rsbc2 = 0.0f;
        if (a.dynamic) {
            float s = (float)((double)scale * a.backoff_factor);
            scale = s < a.min_scale ? a.min_scale : s;
        }
        n.good_steps = 0;
        n.consecutive_overflows = p.consecutive + 1;
        n.skipped_total = p.skipped + 1;
        n.step = p.step;
        n.last_skipped = 1;
        n.last_sumsq = 0.0;
        n.last_grad_norm = __builtin_inff();
        n.last_clip_coef = 1.0f;
    } else {
        const double norm = __builtin_sqrt(sumsq);
        double coef = 1.0;
        if (a.clip_norm > 0.0 && norm > a.clip_norm) coef = a.clip_norm / norm;
        const int64_t t = p.step + 1;
        const double bc1 = 1.0 - ipow(a.beta1, t);
        const double bc2 = 1.0 - ipow(a.beta2, t);
        n.skip = 0;
        n.gscale = (float)((double)p.inv * coef);
        n.rbc1 = (float)(1.0 / bc1);
        n.rsbc2 = (float)(1.0 / __builtin_sqrt(bc2));
        n.step = t;
        int32_t good = p.good + 1;
        if (a.dynamic && good >= a.growth_interval) {
            const float s = (float)((double)scale * a.growth_factor);
            if (f32_finite(s)) scale = s;
            good = 0;
        }
        n.good_steps = good;
        n.consecutive_overflows = 0;
        n.skipped_total = p.skipped;
        n.last_skipped = 0;
        n.last_sumsq = sumsq;
        n.last_grad_norm = (float)norm;
        n.last_clip_coef = (float)coef;
    }
    n.loss_scale = scale;
    n.inv = unscale_factor(a.predivide_factor, a.dp_world_size, scale);
    n.pad_[0] = n.pad_[1] = n.pad_[2] = 0;
    return d;
}

__device__ __forceinline__ void write_state(DevState* __restrict__ st, const DevState& n) {
    st->loss_scale = n.loss_scale;
    st->good_steps = n.good_steps;
    st->step = n.step;
    st->skipped_total = n.skipped_total;
    st->consecutive_overflows = n.consecutive_overflows;
    st->last_skipped = n.last_skipped;
    st->last_sumsq = n.last_sumsq;
    st->last_grad_norm = n.last_grad_norm;
    st->last_clip_coef = n.last_clip_coef;
    st->inv = n.inv;
    st->skip = n.skip;
    st->gscale = n.gscale;
    st->rbc1 = n.rbc1;
    st->rsbc2 = n.rsbc2;
}
// For a norm pass of at most kFuseMaxParts blocks the update takes the step's decisions
// itself and the finalize launch is not made.  Every wave of every update block sums the
// partials exactly as sum_partials does with kFinalizeBlock threads: thread t < nparts
// holds 0 + partial[t], the others 0; each wave of the finalize adds its 64 values by the
// xor-butterfly, and the wave sums are added in wave order.  One wave here walks the
// finalize's waves in turn with the same butterfly, so the squared norm and every
// decision have the bits the finalize kernel would give.  The pre-step state comes from
// the norm pass's snapshot, and block 0 writes the state block.
static_assert(kFuseMaxParts == kFinalizeBlock && kFinalizeBlock % 64 == 0,
              "a fused update covers the finalize's whole first pass");
struct Fuse {
    const double* partial;       // null: the finalize kernel ran, read the state block
    uint32_t nparts;
    const DevState* snap;
    DevState* st;                // written by block 0
    FinalizeArgs fin;
};
// The loads of fused_decide, so that a caller can issue them ahead of its data loads and
// let the decision's arithmetic overlap the data's latency.
struct FusedIn {
    double p[kFinalizeBlock / 64];   // this lane's partial of each finalize wave (0 if none)
    PreState pre;
};
__device__ __forceinline__ FusedIn fused_load(const Fuse& f) {
    const uint32_t lane = threadIdx.x & 63;
    FusedIn in;
    // unconditional loads (a lane past the partials reads partial[0], which fused_finish
    // ignores), so they issue back to back without a wait between them
#pragma unroll
    for (int w = 0; w < kFinalizeBlock / 64; ++w) {
        const uint32_t i = w * 64 + lane;
        in.p[w] = f.partial[i < f.nparts ? i : 0];
    }
    in.pre = read_pre(f.snap);
    return in;
}
// Issued after a block's data loads: the decision's arithmetic cannot be scheduled above
// this point (it depends on the values passed through), and the data loads cannot sink
// below it, so the arithmetic overlaps the data's latency.  Register operands only.
__device__ __forceinline__ void after_data(FusedIn& in) {
    static_assert(kFinalizeBlock / 64 == 4, "four partial registers");
    asm volatile("" : "+v"(in.p[0]), "+v"(in.p[1]), "+v"(in.p[2]), "+v"(in.p[3]) : : "memory");
}
__device__ __forceinline__ Decision fused_finish(const FusedIn& in, const Fuse& f) {
    const uint32_t lane = threadIdx.x & 63;
    // finalize waves holding partials; the others sum to +0, which is added as such
    const uint32_t waves = (f.nparts + 63) / 64;
    double r = 0.0;
#pragma unroll
    for (uint32_t w = 0; w < kFinalizeBlock / 64; ++w) {
        double v = 0.0;
        if (w < waves) {
            if (w * 64 + lane < f.nparts) v = 0.0 + in.p[w];
#pragma unroll
            for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
        }
        r = w == 0 ? v : r + v;
    }
    return decide(r, in.pre, f.fin);
}
__device__ __forceinline__ Decision fused_decide(const Fuse& f) {
    return fused_finish(fused_load(f), f);
}

}  // namespace nz1
