// gla_scan.cuh — what the kernels of the gated recurrence share.
//
//     h_t = a_t h_{t-1} + w_t x_t,   out_t = h_t act(gate_t)
//
// on one number a channel, with a_t = exp(g_t) or sigmoid(g_t) and w_t = 1 or 1 - a_t.
#pragma once

#include "gla_act.cuh"
#include "gla_seq.cuh"

namespace gla {
namespace scan {

constexpr int kChunk = 64;  // rows of a chunk
// Rows of a run.  The state before every run is what a forward keeps for the gradient: half a byte for each element, for which
// the gradient's kernel needs neither the states before a chunk nor a second walk through its rows.
constexpr int kRun = 8;

struct Shape {
    int nseq, T, D;
    int form, act;
    const int32_t *cu;
};
__host__ inline int64_t total_rows(const Shape &p) { return p.cu ? (int64_t)p.T : (int64_t)p.nseq * p.T; }
__host__ inline int64_t slots(const Shape &p) { return chunk_slots(total_rows(p), p.nseq, kChunk); }
__host__ inline int64_t states_bytes(const Shape &p) {
    return chunk_slots(total_rows(p), p.nseq, kRun) * p.D * (int64_t)sizeof(float);
}
// where the state before a sequence's rows t .. t + kRun - 1 is kept; start: the sequence's first row
__device__ __forceinline__ int64_t state_slot(int start, int seq, int t) { return (int64_t)(start / kRun) + seq + t / kRun; }

// ---- two neighbouring channels of one row ------------------------------------------------------------------------
template <typename T> struct Two;
template <> struct Two<__nv_bfloat16> {
    using Raw = uint32_t;
    static __device__ __forceinline__ Pair open(Raw w) {
        return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    static __device__ __forceinline__ Raw close(Pair x) {
        const float2 f = parts(x);
        const __nv_bfloat162 v = __floats2bfloat162_rn(f.x, f.y);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
};
template <> struct Two<float> {
    using Raw = float2;
    static __device__ __forceinline__ Pair open(Raw w) { return pair(w.x, w.y); }
    static __device__ __forceinline__ Raw close(Pair x) { return parts(x); }
};
template <typename T> __device__ __forceinline__ void store_two(T *p, Pair x) {
    *reinterpret_cast<typename Two<T>::Raw *>(p) = Two<T>::close(x);
}
template <typename T> __device__ __forceinline__ Pair load_two(const T *p) {
    return Two<T>::open(__ldg(reinterpret_cast<const typename Two<T>::Raw *>(p)));
}
// four of them, as they lie in memory
template <typename T> struct FourRaw;
template <> struct FourRaw<__nv_bfloat16> {
    uint2 w;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { w = __ldg(reinterpret_cast<const uint2 *>(p)); }
    __device__ __forceinline__ void open(Pair (&x)[2]) const { x[0] = Two<__nv_bfloat16>::open(w.x), x[1] = Two<__nv_bfloat16>::open(w.y); }
};
template <> struct FourRaw<float> {
    float4 w;
    __device__ __forceinline__ void load(const float *p) { w = __ldg(reinterpret_cast<const float4 *>(p)); }
    __device__ __forceinline__ void open(Pair (&x)[2]) const { x[0] = pair(w.x, w.y), x[1] = pair(w.z, w.w); }
};
template <typename T> __device__ __forceinline__ void load_four(const T *p, Pair (&x)[2]) {
    FourRaw<T> f;
    f.load(p);
    f.open(x);
}
__device__ __forceinline__ void store_four(__nv_bfloat16 *p, const Pair (&x)[2]) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(Two<__nv_bfloat16>::close(x[0]), Two<__nv_bfloat16>::close(x[1]));
}
__device__ __forceinline__ void store_four(float *p, const Pair (&x)[2]) {
    const float2 a = parts(x[0]), b = parts(x[1]);
    *reinterpret_cast<float4 *>(p) = make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ Pair load_state(const float *p) {
    const float2 f = *reinterpret_cast<const float2 *>(p);
    return pair(f.x, f.y);
}
__device__ __forceinline__ void store_state(float *p, Pair x) { *reinterpret_cast<float2 *>(p) = parts(x); }

// ---- the decay ---------------------------------------------------------------------------------------------------
//
// Long memories need 1 - a more than a: an a of 1 - 1e-4 that is rounded to 2^-25 has 3e-4 of its decay rounded away, and
// all tokens' alike where g is.  So a decay is held as c + k: c = a - 1, good to a few units of its own last place, and k = 1
// where a is near 1; c = a, so that a strong decay keeps its digits too, and k = 0 elsewhere.  (k h is a NaN where h is an
// infinity and k = 0; choosing h or 0 instead costs twice the instructions, of which the chunked kernels have few to spare.)
struct Decay {
    Pair c, k;
};

template <int kForm>
__device__ __forceinline__ Decay decay(Pair g) {
    const float2 f = parts(g);
    float c0, c1;
    bool lo, hi;
    if (kForm == GLA_SCAN_LOG || kForm == GLA_SCAN_LOG_LEAK) {
        const float2 t = parts(g * both(1.4426950408889634f));
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(c0) : "f"(t.x));
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(c1) : "f"(t.y));
        // e^g - 1 by its series: behind g^6 / 6! the next term is below 2^-24 of the sum for |g| < 0.25
        Pair s = fma(g, both(1.f / 720.f), both(1.f / 120.f));
        s = fma(g, s, both(1.f / 24.f));
        s = fma(g, s, both(1.f / 6.f));
        s = fma(g, s, both(0.5f));
        s = fma(g, s, both(1.f));
        const float2 m = parts(s * g);
        lo = fabsf(f.x) < 0.25f;
        hi = fabsf(f.y) < 0.25f;
        c0 = lo ? m.x : c0;
        c1 = hi ? m.y : c1;
    } else {
        // 1 / (1 + e^-g), and 1 less that as e^-g / (1 + e^-g), where e^-g is small
        float e0, e1;
        const float2 t = parts(g * both(-1.4426950408889634f));
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(t.x));
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(t.y));
        const Pair e = pair(e0, e1);
        const float2 d = parts(e + both(1.f));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(c0) : "f"(d.x));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(c1) : "f"(d.y));
        const float2 r = parts(e * pair(c0, c1));
        lo = f.x > 1.f;
        hi = f.y > 1.f;
        c0 = lo ? -r.x : c0;
        c1 = hi ? -r.y : c1;
    }
    return {pair(c0, c1), pair(lo ? 1.f : 0.f, hi ? 1.f : 0.f)};
}
__host__ __device__ constexpr bool leaks(int form) { return form == GLA_SCAN_LOG_LEAK || form == GLA_SCAN_SIGMOID_LEAK; }
__host__ __device__ constexpr bool is_log(int form) { return form == GLA_SCAN_LOG || form == GLA_SCAN_LOG_LEAK; }

// a h + b, a h, a and 1 - a
__device__ __forceinline__ Pair decayed(const Decay &d, Pair h, Pair b) { return fma(d.c, h, fma(d.k, h, b)); }
__device__ __forceinline__ Pair decayed(const Decay &d, Pair h) { return fma(d.c, h, d.k * h); }
__device__ __forceinline__ Pair whole(const Decay &d) { return d.c + d.k; }
__device__ __forceinline__ Pair rest(const Decay &d) { return fma(d.c, both(-1.f), fma(d.k, both(-1.f), both(1.f))); }
// the input's part of h
template <int kForm>
__device__ __forceinline__ Pair input(const Decay &d, Pair x) {
    return leaks(kForm) ? x * rest(d) : x;
}

// Calls RUN(T, TG, kForm, kGate) for a call's types, form and gate.
#define GLA_SCAN_BY_FORM(T, TG, G, RUN)                                   \
    switch (p.form) {                                                     \
        case GLA_SCAN_LOG: RUN(T, TG, GLA_SCAN_LOG, G); break;            \
        case GLA_SCAN_LOG_LEAK: RUN(T, TG, GLA_SCAN_LOG_LEAK, G); break;  \
        case GLA_SCAN_SIGMOID: RUN(T, TG, GLA_SCAN_SIGMOID, G); break;    \
        default: RUN(T, TG, GLA_SCAN_SIGMOID_LEAK, G); break;             \
    }
#define GLA_SCAN_DISPATCH(dtype, g_dtype, gated, RUN)                                                            \
    if (dtype == GLA_F32) {                                                                                      \
        if (gated) { GLA_SCAN_BY_FORM(float, float, true, RUN) }                                                 \
        else { GLA_SCAN_BY_FORM(float, float, false, RUN) }                                                      \
    } else if (g_dtype == GLA_F32) {                                                                             \
        if (gated) { GLA_SCAN_BY_FORM(__nv_bfloat16, float, true, RUN) }                                         \
        else { GLA_SCAN_BY_FORM(__nv_bfloat16, float, false, RUN) }                                              \
    } else {                                                                                                     \
        if (gated) { GLA_SCAN_BY_FORM(__nv_bfloat16, __nv_bfloat16, true, RUN) }                                 \
        else { GLA_SCAN_BY_FORM(__nv_bfloat16, __nv_bfloat16, false, RUN) }                                      \
    }

}  // namespace scan
}  // namespace gla
