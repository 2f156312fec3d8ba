// Device helpers of the state space kernels.
#pragma once

#include "gdr_device.h"
#include "ssm_params.h"

namespace sconv {

constexpr float kLog2e = 1.4426950408889634f;

// softplus(v), or v where the steps come without.  log1p(e) with e = e^-|v| is 2 atanh(q), q = e / (2 + e) <= 1/3: the series'
// next term is below 2^-26 of it.  The exponent goes in two parts (its product's rounding alone would move e by |v| 2^-24), up to
// 128, where e is 0.
// Roundings of 2^-24: 3 of e, 1 of 2 + e, 2 of its reciprocal, 1 of q, 2 of the series, 1 of the sum.
__device__ __forceinline__ float ssm_softplus(const SsmParams &p, float v) {
    if (!p.softplus) return v;
    constexpr float kLog2eLow = 1.4426950408889634 - double(kLog2e);
    const float a = fminf(fabsf(v), 128.0f), h = a * -kLog2e, l = fmaf(a, -kLog2eLow, fmaf(a, -kLog2e, -h)), e0 = __builtin_amdgcn_exp2f(h);
    const float e = fmaf(e0 * l, 0.6931471805599453f, e0), q = e * __builtin_amdgcn_rcpf(2.0f + e), w = q * q;
    float s = fmaf(w, 2.0f / 15, 2.0f / 13);
    s = fmaf(w, s, 2.0f / 11);
    s = fmaf(w, s, 2.0f / 9);
    s = fmaf(w, s, 2.0f / 7);
    s = fmaf(w, s, 2.0f / 5);
    s = fmaf(w, s, 2.0f / 3);
    s = fmaf(w, s, 2.0f);
    return fmaf(q, s, v < 0.0f ? 0.0f : v);            // (NaN stays)
}
__device__ __forceinline__ float ssm_clamp(const SsmParams &p, float d) {
    d = d < p.dt_min ? p.dt_min : d;   // (NaN stays)
    return d > p.dt_max ? p.dt_max : d;
}
// The step size of head h, channel c at element offset `at` of dt (channel included).
__device__ __forceinline__ float ssm_step(const SsmParams &p, int64_t at, float bias) {
    const float d = p.dt_fp32 ? static_cast<const float *>(p.dt)[at] : bf_one(static_cast<const uint16_t *>(p.dt)[at]);
    return ssm_clamp(p, ssm_softplus(p, d + bias));
}

// e^(d A), at most 1 (NaN stays), and 1 for a step of 0 whatever A is.  Three roundings reach the argument (the product's with A,
// log2(e)'s and the product's with it), which move the result by 3 |d A| e^(d A) 2^-24 at most, below 2^-23.8: what a state
// keeps is right to that share of the state, and to the exponential's own.
__device__ __forceinline__ float ssm_decay(float d, float A) {
    const float g = d == 0.0f ? 0.0f : d * A;
    return __builtin_amdgcn_exp2f((g > 0.0f ? 0.0f : g) * kLog2e);
}

// y silu(z).
__device__ __forceinline__ float ssm_gate(float y, float z) { return y * act<true>(z); }

// Sequence b's (or entry b's) rows and line; false when nothing is to be done for it.
struct SsmSpan { int64_t t0, n, line; bool init; };
__device__ __forceinline__ bool ssm_span(const SsmParams &p, int32_t b, SsmSpan &sp) {
    sp.t0 = 0;
    sp.n = p.seqlen;
    sp.line = b;
    sp.init = p.state != nullptr;
    if (p.qsl) {
        int64_t a = p.qsl[b], e = p.qsl[b + 1];
        a = a < 0 ? 0 : (a > p.total_T ? p.total_T : a);
        e = e < a ? a : (e > p.total_T ? p.total_T : e);
        sp.t0 = a;
        sp.n = e - a;
        sp.init = p.state && p.has_init && p.has_init[b] != 0;
    }
    if (sp.n == 0) return false;
    if (p.ci) {
        int32_t step = 0;
        if (p.accepted) {
            step = p.accepted[b] - 1;
            if (step < 0 || step >= p.ci_steps) return false;
        }
        sp.line = p.ci[b * p.ci_sb + step * p.ci_ss];
        if (sp.line == p.pad_slot_id) return false;
    }
    return !(p.state && (sp.line < 0 || sp.line >= p.num_lines));
}

}  // namespace sconv
