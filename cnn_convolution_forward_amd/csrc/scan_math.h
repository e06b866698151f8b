// scan_math.h -- the gates of the recurrence h = a h + sqrt(1 - a^2) s x, per
// token and channel: r = sigmoid(gate), s = sigmoid(inp), a = exp(-k r).
#pragma once

#include "seq_common.h"

namespace convfwd {

// k = scale * log(1 + exp(decay)); log(1 + e^d) = d + log(1 + e^-d) keeps a
// large d from overflowing.
__device__ __forceinline__ float scan_rate(float scale, float decay) {
    return scale * (fmaxf(decay, 0.f) + log1pf(expf(-fabsf(decay))));
}

// v = 1 - a^2 = 1 - exp(-w), w = 2 k r.  Near w = 0, where the difference
// cancels, the series w - w^2/2 + ... (its first dropped term is below 5.5e-8 of
// the sum for w < 1/4); beyond, the difference itself loses at most two bits.
__device__ __forceinline__ float one_minus_sq(float w, float a) {
    float p = fmaf(w, -1.f / 720.f, 1.f / 120.f);
    p = fmaf(w, p, -1.f / 24.f);
    p = fmaf(w, p, 1.f / 6.f);
    p = fmaf(w, p, -0.5f);
    p = fmaf(w, p, 1.f);
    return w < 0.25f ? w * p : fmaf(-a, a, 1.f);
}

// A channel's constants: -k log2(e), so that a = 2^(kl r), and w = k2 r.
struct ScanRate {
    float k, kl, k2;
    __device__ __forceinline__ void set(float rate) {
        k = rate;
        kl = -kLog2e * rate;
        k2 = rate + rate;
    }
};

// v = 0 (k r underflows, or the gate is -inf) leaves h as it is: m is 0 then,
// and the clamp keeps 1/m finite, as it stands beside factors of k r, or 0.
struct ScanGates {
    float r, s, a, m, im;     // m = sqrt(1 - a^2), im = 1/m
    __device__ __forceinline__ ScanGates(const ScanRate &c, float gate, float inp) {
        r = sigmoid(gate);
        s = sigmoid(inp);
        a = __builtin_amdgcn_exp2f(c.kl * r);
        const float v = one_minus_sq(c.k2 * r, a);
        im = __builtin_amdgcn_rsqf(fmaxf(v, 1.17549435e-38f));
        m = v * im;
    }
};

}  // namespace convfwd
