// gla_act.cuh — the activations of gates and normalised values, on pairs of f32.
#pragma once

#include "gla_pairs.cuh"

namespace gla {

enum Act { kNone = GLA_ACT_NONE, kSilu = GLA_ACT_SILU, kSigmoid = GLA_ACT_SIGMOID };

// q = 1 / (1 + e^-x) and rest = 1 - q, each to 2 + |x| units of 2^-24 (the rounding of e^-x's argument), and a NaN where x
// is one.  rest is e^-x q (1 - q would leave 2^-24 of one where q is near 1, which SiLU's slope multiplies by x).  Below
// x = -87 e^-x runs into infinity and q into 0, which is the limit; rest is 1 to the last bit from x = -20 on and is not
// taken from their product there.
__device__ __forceinline__ void sigmoid(Pair x, Pair &q, Pair &rest) {
    const float2 f = parts(x);
    const float2 t = parts(x * both(-1.4426950408889634f));
    float e0, e1, q0, q1;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(t.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(t.y));
    const Pair e = pair(e0, e1);
    const float2 d = parts(e + both(1.f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q0) : "f"(d.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q1) : "f"(d.y));
    q = pair(q0, q1);
    const float2 r = parts(e * q);
    rest = pair(f.x < -20.f ? 1.f : r.x, f.y < -20.f ? 1.f : r.y);
}

// act(x), a gate's factor, and its slope.  SiLU's slope takes 1 - q as it is: its error, 2^-24 times x, is no more than that
// of q, and below x = -87 both end in 0.
__device__ __forceinline__ Pair sigmoid(Pair x) {
    float e0, e1, q0, q1;
    const float2 t = parts(x * both(-1.4426950408889634f));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(t.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(t.y));
    const float2 d = parts(pair(e0, e1) + both(1.f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q0) : "f"(d.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q1) : "f"(d.y));
    return pair(q0, q1);
}
__device__ __forceinline__ Pair activation(Pair x, int act) {
    if (act == kNone) return x;
    const Pair q = sigmoid(x);
    return act == kSilu ? x * q : q;
}
__device__ __forceinline__ Pair activation(Pair x, int act, Pair &slope) {
    if (act == kNone) {
        slope = both(1.f);
        return x;
    }
    if (act == kSilu) {
        const Pair q = sigmoid(x);
        slope = q * fma(x, fma(q, both(-1.f), both(1.f)), both(1.f));
        return x * q;
    }
    Pair q, rest;
    sigmoid(x, q, rest);
    slope = q * rest;
    return q;
}

}  // namespace gla
