// gla_resnorm_bwd.cuh — the residual norm's gradient.
#pragma once

#include "gla_resnorm.cuh"

namespace gla {
namespace resnorm {
namespace {

constexpr int kBwdVecs = 2, kBwdMost = 640;
constexpr int kBwdThreads = 640;  // of an SM, at 96 registers each

// kMode: which parts there are, for the kernels built for one kind of call; kAnyMode: all of that is asked for at run time.
// (16,435 x 2,552 bf16: 212 us with all parts and 104 of a plain sum, asked at run time 318 and 211.)  kRagged: some threads have
// vectors without channels.  (Whole rows of 2,560: 177 and 95.)  kParams: the parameters are in shared memory, all that the parts
// could ask for (ones and zeros for those that there are not).
enum Mode { kOut = 1, kY = 2, kPost = 4, kGated = 8, kGatedSigmoid = 16, kAnyMode = 32, kParams = 64, kRagged = 128 };
enum Param { kWeight, kScale, kPostWeight, kPostBias };
constexpr __host__ __device__ int params_of(int mode) { return mode & (kPost | kAnyMode) ? 4 : mode & kY ? 2 : 1; }
template <typename T, typename TS, int kVec, bool kWide, int kMode>
__global__ void __launch_bounds__(kBwdMost, 1)
bwd_kernel(const Inputs<5> in, Weights weights, int kind, int post_, int act, float eps, TS *__restrict__ dx, T *__restrict__ dy,
           T *__restrict__ dgate, float *__restrict__ part, int64_t rows, int D, int slice, int lanes, int params_at) {
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ Bars bars;
    __shared__ __align__(16) Meeting<kWide> meet;
    const Cluster<kWide> cl;
    const int c0 = cl.rank * slice, here = kWide ? min(slice, D - c0) : D;  // the block's first channel, and how many
    const Place<kVec> pl(here, lanes);
    const float inv = 1.f / (float)D;
    constexpr bool kAny = (kMode & kAnyMode) != 0;
    const bool has_dr = in.from[0] != nullptr, layer = kind == GLA_NORM_LAYER;
    const bool has_out = kAny ? in.from[1] != nullptr : (kMode & kOut) != 0, has_y = kAny ? in.from[3] != nullptr : (kMode & kY) != 0,
               has_gate = kAny ? in.from[4] != nullptr : (kMode & (kGated | kGatedSigmoid)) != 0, post = kAny ? post_ != 0 : (kMode & kPost) != 0;
    const bool meets = (kWide || lanes > 32) && (post || has_out);
    Pair sums[kSums][kVec][2];
#pragma unroll
    for (int i = 0; i < kSums; ++i)
#pragma unroll
        for (int j = 0; j < kVec; ++j) sums[i][j][0] = sums[i][j][1] = both(0.f);
    Rows<true, 5, kWide> it(in, cl, ring, bars, rows, lanes);
    meet.clear();
    constexpr bool kShared = (kMode & kParams) != 0;
    if (kShared)
        for (int i = 0; i < params_of(kMode); ++i) {
            const float *const from = i == kWeight ? weights.weight : i == kScale ? weights.scale : i == kPostWeight ? weights.post_weight : weights.post_bias;
            const float fill = i == kPostBias ? 0.f : 1.f;
            float4 *const to = reinterpret_cast<float4 *>(ring + params_at) + i * (slice / 4);
            for (int c = threadIdx.x; c < here / 4; c += blockDim.x)
                to[c] = from ? __ldg(reinterpret_cast<const float4 *>(from + c0) + c) : make_float4(fill, fill, fill, fill);
        }
    const Weights w = kShared ? weights : weights.from(c0 + pl.channel);
    const float *const params = reinterpret_cast<const float *>(ring + params_at) + pl.channel;
    cl.sync();
    int half = 0;
    auto row = [&](auto all) {
        using Vs = Vectors<kVec, all.value>;
        const bool there = all.value || it.row < rows;
        const Vs vs{there ? pl.count : 0};
        const int64_t at = it.row * D + c0 + pl.channel;
        const TS *const from_r = it.template at<TS>(2, D, pl.channel);
        const T *const from_out = it.template at<T>(1, D, pl.channel), *const from_y = it.template at<T>(3, D, pl.channel);
        // one vector of an array, or of parameters
        auto vec = [&](Pair (&v)[2], const auto *p, int j) {
            using E = std::remove_cv_t<std::remove_reference_t<decltype(*p)>>;
            typename Four<E>::Raw raw{};
            if (vs.has(j)) raw = *reinterpret_cast<const typename Four<E>::Raw *>(p + j * kStride);
            Four<E>::open(v, raw);
        };
        // vector j of a parameter; v as it is where there is none
        auto param = [&](Pair (&v)[2], Param which, int j) {
            const float *const p = which == kWeight ? w.weight : which == kScale ? w.scale : which == kPostWeight ? w.post_weight : w.post_bias;
            if (kShared) vec(v, params + which * slice, j);
            else if (p != nullptr) vec(v, p, j);
        };
        // n(r) = r' q + qm and n(y) = y' uq + uqm, of r' = r + near_r and y' = y + near_y
        typename Vs::V rc, yc;
        Pair q = both(1.f), qm = both(0.f), uq = both(1.f), uqm = both(0.f), m1 = both(0.f), m2 = both(0.f);
        float near_r = 0.f, near_y = 0.f;
        if (has_out || post) {
            if (layer) {
                if (has_out) near_r = near_mean(it.template head<TS>(2, D), D, lanes, there);
                if (post) near_y = near_mean(it.template head<T>(3, D), D, lanes, there);
            }
            Pair s[6];
#pragma unroll
            for (int i = 0; i < 6; ++i) s[i] = both(0.f);
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                if (has_out) {
                    Pair up[2], wt[2] = {both(1.f), both(1.f)};
                    vec(rc[j], from_r, j);
                    vec(up, from_out, j);
                    param(wt, kWeight, j);
                    const Pair by = both(vs.has(j) ? near_r : 0.f);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        if (layer) rc[j][e] = rc[j][e] + by;
                        up[e] = up[e] * wt[e];
                        s[0] = s[0] + rc[j][e];
                        s[1] = fma(rc[j][e], rc[j][e], s[1]);
                        s[2] = s[2] + up[e];
                        s[3] = fma(up[e], rc[j][e], s[3]);
                    }
                }
                if (post) {
                    vec(yc[j], from_y, j);
                    const Pair by = both(vs.has(j) ? near_y : 0.f);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        if (layer) yc[j][e] = yc[j][e] + by;
                        s[4] = s[4] + yc[j][e];
                        s[5] = fma(yc[j][e], yc[j][e], s[5]);
                    }
                }
            }
            float o[6];
#pragma unroll
            for (int i = 0; i < 6; ++i) o[i] = total(s[i]);
            row_sums<kBwdMost>(o, lanes, cl, meet, half);
            if (meets) it.refill();
            // (a variance below zero is rounding; a NaN stays)
            const float mr = layer ? o[0] * inv : 0.f, mu = layer ? o[4] * inv : 0.f;
            const float vr = fmaf(-mr, mr, o[1] * inv), vu = fmaf(-mu, mu, o[5] * inv);
            const float rr = rsqrtf((vr < 0.f ? 0.f : vr) + eps), ru = rsqrtf((vu < 0.f ? 0.f : vu) + eps);
            q = both(rr), qm = both(-mr * rr);
            if (post) uq = both(ru), uqm = both(-mu * ru);
            if (layer) m1 = both(-o[2] * inv);
            m2 = both(-fmaf(-mr, o[2], o[3]) * rr * inv);
        }
        typename Vs::V d;
        Pair s = both(0.f), t = both(0.f);
        // dx, and from there on through the scale and the gate, one vector after the other
        auto through = [&](auto kind_of_act) {
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                d[j][0] = d[j][1] = both(0.f);
                if (has_dr) vec(d[j], it.template at<TS>(0, D, pl.channel), j);
                if (has_out) {
                    Pair up[2], wt[2] = {both(1.f), both(1.f)};
                    vec(up, from_out, j);
                    param(wt, kWeight, j);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const Pair h = fma(rc[j][e], q, qm);
                        sums[2][j][e] = fma(up[e], h, sums[2][j][e]);
                        sums[3][j][e] = sums[3][j][e] + up[e];
                        d[j][e] = fma(fma(h, m2, fma(up[e], wt[e], m1)), q, d[j][e]);
                    }
                    if (!vs.has(j)) d[j][0] = d[j][1] = both(0.f);
                }
                if (vs.has(j)) put<TS>(dx + at + j * kStride, d[j]);
                if (!has_y) continue;
                Pair u[2], p[2];
                if (post) u[0] = fma(yc[j][0], uq, uqm), u[1] = fma(yc[j][1], uq, uqm);
                else vec(u, from_y, j);
                Pair sc[2] = {both(1.f), both(1.f)};
                param(sc, kScale, j);
                if (kind_of_act.value >= 0) {
                    Pair g[2], slope;
                    Pair z[2] = {u[0], u[1]};  // what the scale and the gate multiply
                    if (post) {
                        p[0] = p[1] = both(1.f);
                        param(p, kPostWeight, j);
                        z[0] = z[0] * p[0], z[1] = z[1] * p[1];
                        p[0] = p[1] = both(0.f);
                        param(p, kPostBias, j);
                        z[0] = z[0] + p[0], z[1] = z[1] + p[1];
                    }
                    vec(g, it.template at<T>(4, D, pl.channel), j);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const Pair f = activation(g[e], kind_of_act.value, slope);
                        g[e] = d[j][e] * sc[e] * z[e] * slope;
                        d[j][e] = d[j][e] * f;
                    }
                    if (vs.has(j)) put<T>(dgate + at + j * kStride, g);
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    sums[0][j][e] = fma(d[j][e], u[e], sums[0][j][e]);
                    if (post) sums[1][j][e] = sums[1][j][e] + d[j][e];
                    d[j][e] = d[j][e] * sc[e];
                }
                if (!post) {
                    if (vs.has(j)) put<T>(dy + at + j * kStride, d[j]);
                    continue;
                }
                p[0] = p[1] = both(1.f);
                param(p, kPostWeight, j);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    d[j][e] = d[j][e] * p[e];
                    s = s + d[j][e];
                    t = fma(d[j][e], u[e], t);
                }
            }
        };
        if (!kAny) through(std::integral_constant<int, (kMode & kGated) != 0 ? (int)kSilu : (kMode & kGatedSigmoid) != 0 ? (int)kSigmoid : -1>{});
        else if (!has_gate) through(std::integral_constant<int, -1>{});
        else if (act == kSilu) through(std::integral_constant<int, kSilu>{});
        else if (act == kSigmoid) through(std::integral_constant<int, kSigmoid>{});
        else through(std::integral_constant<int, kNone>{});
        if (post) {
            const float2 o = row_sum(layer ? total(s) : 0.f, total(t), lanes, cl, meet, half);
            m1 = both(-o.x * inv), m2 = both(-o.y * inv);
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                Pair y[2];
                vec(y, from_y, j);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (layer) y[e] = y[e] + both(near_y);
                    d[j][e] = fma(fma(y[e], uq, uqm), m2, d[j][e] + m1) * uq;
                }
                if (vs.has(j)) put<T>(dy + at + j * kStride, d[j]);
            }
        }
    };
    for (; it.begin(meets); it.next()) row(std::integral_constant<bool, (kMode & (kAnyMode | kRagged)) == 0>{});
    it.end();
    // the block's rows of one channel set meet in shared memory; one writer per channel
    float *to = part + (int64_t)(kWide ? blockIdx.x / cl.ranks : blockIdx.x) * kSums * D;
    const int at_once = blockDim.x / lanes, mine = threadIdx.x / lanes;
    float4 *const tops = reinterpret_cast<float4 *>(ring);  // the stages are read
#pragma unroll
    for (int i = 0; i < kSums; ++i)
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            float4 v = Four<float>::close(sums[i][j]);
            if (at_once > 1) {
                __syncthreads();
                tops[threadIdx.x] = v;
                __syncthreads();
                if (mine == 0)
                    for (int m = 1; m < at_once; ++m) {
                        const float4 o = tops[threadIdx.x + m * lanes];
                        v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
                    }
            }
            if (mine == 0 && j < pl.count)
                *reinterpret_cast<float4 *>(to + (int64_t)i * D + c0 + pl.channel + j * kStride) = v;
        }
}

// A call's kernel: by its parts where rows leave no thread without work.  Returns the number of parts of the sums, 0: failed.
template <typename T, typename TS>
int launch_bwd(const void *dr, const void *dout, const void *r, const void *y, const void *gate, const Weights &w, int kind,
                int post, int act, float eps, void *dx, void *dy, void *dgate, float *part, int64_t rows, int D, cudaStream_t st) {
    const Plan pl = make_plan(D, kBwdVecs, kWidest);
    int n = per_sm(pl, kBwdThreads);
    constexpr int e = sizeof(T), es = sizeof(TS);
    Inputs<5> in{};
    const void *const from[5] = {dr, dout, dout != nullptr ? r : nullptr, y, gate};
    for (int i = 0; i < 5; ++i) {
        const int size = i == 0 || i == 2 ? es : e;
        in.from[i] = from[i];
        in.row_bytes[i] = D * size;
        in.slice_bytes[i] = pl.slice * size;
        in.head_bytes[i] = kind == GLA_NORM_LAYER && (i == 2 || i == 3) ? (size == 2 ? 8 : kStride) * size : 0;
    }
    const int mode = (dout != nullptr ? kOut : 0) + (y != nullptr ? kY : 0) + (post ? kPost : 0) +
                     (gate == nullptr ? 0 : act == kSilu ? kGated : act == kSigmoid ? kGatedSigmoid : kAnyMode);
    const bool known = mode == kOut + kY || mode == kOut + kY + kPost || (mode & ~(kPost | kGated | kGatedSigmoid)) == kOut + kY;
    const bool even = D % pl.slice == 0 && pl.slice % (kStride * kBwdVecs) == 0;
    int params_at;
    const int params = params_of(known && pl.vecs == kBwdVecs ? mode : kAnyMode) * pl.slice * 4;
    int bytes = lay_out(in, pl, rows, n, units(pl, rows, n), params, params_at);
    while (in.stages < 2 && n > 1) {  // fewer blocks of an SM, with room for their stages (f32 rows of 512 channels or so)
        --n;
        bytes = lay_out(in, pl, rows, n, units(pl, rows, n), params, params_at);
    }
    if (in.stages < 2) return 0;
    const int nu = units(pl, rows, n);
    // kernels of a call's own parts: all but those of a row in several blocks that have no room for its parameters
    const bool whole = even && rows % ((int64_t)pl.rows * in.passes) == 0;
    const bool own = pl.vecs == kBwdVecs && (params_at >= 0 || pl.ranks == 1);
#define GLA_RUN(V, W, M)                                                                                                   \
    return launch<bwd_kernel<T, TS, V, W, M>>(nu, pl.ranks, pl.threads, bytes, st, in, w, kind, post, act, eps, \
                                              (TS *)dx, (T *)dy, (T *)dgate, part, rows, D, pl.slice, pl.lanes, params_at);
#define GLA_WHOLE(M)                                                                                                       \
    if (own && mode == (M)) {                                                                                              \
        if (pl.ranks > 1 && whole) GLA_RUN(kBwdVecs, true, (M) + kParams)                                                  \
        if (pl.ranks > 1) GLA_RUN(kBwdVecs, true, (M) + kParams + kRagged)                                                 \
        if (params_at < 0 && whole) GLA_RUN(kBwdVecs, false, M)                                                            \
        if (params_at < 0) GLA_RUN(kBwdVecs, false, (M) + kRagged)                                                         \
        if (whole) GLA_RUN(kBwdVecs, false, (M) + kParams)                                                                 \
        GLA_RUN(kBwdVecs, false, (M) + kParams + kRagged)                                                                  \
    }
    GLA_WHOLE(kOut + kY + kPost + kGated)
    GLA_WHOLE(kOut + kY + kPost + kGatedSigmoid)
    GLA_WHOLE(kOut + kY + kPost)
    GLA_WHOLE(kOut + kY + kGated)
    GLA_WHOLE(kOut + kY + kGatedSigmoid)
    GLA_WHOLE(kOut + kY)
    if (pl.vecs == 1) {
        if (params_at < 0) return 0;  // (parameters of so few channels always have room)
        GLA_RUN(1, false, kAnyMode + kParams)
    }
    if (pl.ranks > 1) {
        if (params_at >= 0) GLA_RUN(kBwdVecs, true, kAnyMode + kParams)
        GLA_RUN(kBwdVecs, true, kAnyMode)
    }
    if (params_at >= 0) GLA_RUN(kBwdVecs, false, kAnyMode + kParams)
    GLA_RUN(kBwdVecs, false, kAnyMode)
#undef GLA_WHOLE
#undef GLA_RUN
}

}  // namespace
}  // namespace resnorm
}  // namespace gla
