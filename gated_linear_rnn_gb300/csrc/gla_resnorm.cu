// gla_resnorm.cu — the residual sum between two blocks with the norms on both of its sides, and its gradient.
//
// On a token's D channels, with n(v) = (v - mean) / sqrt(variance + eps) (layer) or v / sqrt(mean square + eps) (RMS):
//     u = n(y) post_weight + post_bias, or y;   r = x + scale act(gate) u;   out = n(r) weight + bias
//
// Gradient at r, with h = n(r), q = 1 / its root, uh and uq those of y:
//     d = dout weight,   dx = dr + q (d - mean(d) - h mean(d h))        (mean(d) for the layer norm alone)
//     du = dx scale act(gate),   dgate = dx scale u act'(gate),   dscale = sum over tokens of dx act(gate) u
//     e = du post_weight,   dy = uq (e - mean(e) - uh mean(e uh)), or du
//     dweight = sum of dout h, dbias = sum of dout, dpost_weight = sum of du uh, dpost_bias = sum of du
#include "gla_common.cuh"

GLA_DEFINE_STATUS(resnorm)

#include "gla_resnorm.cuh"

namespace gla {
namespace resnorm {

int64_t bwd_units(int64_t rows, int D);
#define GLA_BWD(NAME)                                                                                                      \
    int NAME(const void *dr, const void *dout, const void *r, const void *y, const void *gate, const float *scale,        \
              const float *post_weight, const float *post_bias, const float *weight, int kind, int post, int act,          \
              float eps, void *dx, void *dy, void *dgate, float *part, int64_t rows, int D, cudaStream_t st)
GLA_BWD(bwd_bf16);
GLA_BWD(bwd_mixed);
GLA_BWD(bwd_f32);
#undef GLA_BWD

namespace {

constexpr int kFwdVecs = 4;
constexpr int kFwdThreads = 768;  // of an SM, at 85 registers each

// Statistics are taken in two steps, a mean and then centred squares.
template <typename T, typename TS, int kVec, bool kStage, int kMost>
__global__ void __launch_bounds__(kMost, kMost <= 256 ? 3 : 1)
fwd_kernel(const Inputs<3> in, Weights weights, int kind, int post, int act, float eps, TS *r, T *__restrict__ out,
           int64_t rows, int D, int lanes) {
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ Bars bars;
    __shared__ __align__(16) Meeting<false> meet;
    const Cluster<false> cl;
    const Place<kVec> pl(D, lanes);
    const float inv = 1.f / (float)D;
    const bool has_y = in.from[1] != nullptr, has_gate = in.from[2] != nullptr, meets = lanes > 32 && (post || out != nullptr);
    Rows<kStage, 3, false> it(in, cl, ring, bars, rows, lanes);
    meet.clear();
    const Weights w = weights.from(pl.channel);
    __syncthreads();
    int half = 0;
    auto row = [&](auto all) {
        using Vs = Vectors<kVec, all.value>;
        const Vs vs{it.row < rows ? pl.count : 0};
        const int64_t at = it.row * D + pl.channel;
        typename Vs::V v;
        // v becomes n(v)
        auto normalise = [&](typename Vs::V &x) {
            if (kind == GLA_NORM_LAYER) vs.shift(x, -row_sum(Vs::sum(x), 0.f, lanes, cl, meet, half).x * inv);
            vs.times(x, rsqrtf(fmaf(row_sum(Vs::squares(x), 0.f, lanes, cl, meet, half).x, inv, eps)));
            if (meets) it.refill();
        };
        if (has_y) {
            typename Vs::V u;
            vs.fetch(u, it.template at<T>(1, D, pl.channel));
            if (post) {
                normalise(u);
                vs.times(u, w.post_weight);
                vs.plus(u, w.post_bias);
            }
            if (has_gate) {
                typename Vs::V g;
                vs.fetch(g, it.template at<T>(2, D, pl.channel));
                if (act == kSilu) Vs::template gate<kSilu>(g);
                else if (act == kSigmoid) Vs::template gate<kSigmoid>(g);
#pragma unroll
                for (int j = 0; j < kVec; ++j) u[j][0] = u[j][0] * g[j][0], u[j][1] = u[j][1] * g[j][1];
            }
            vs.times(u, w.scale);
            vs.fetch(v, it.template at<TS>(0, D, pl.channel));
#pragma unroll
            for (int j = 0; j < kVec; ++j) v[j][0] = v[j][0] + u[j][0], v[j][1] = v[j][1] + u[j][1];
            vs.store(r + at, v);
            vs.clear(v);
        } else {
            vs.fetch(v, it.template at<TS>(0, D, pl.channel));
        }
        if (out != nullptr) {
            normalise(v);
            vs.times(v, w.weight);
            vs.plus(v, w.bias);
            vs.store(out + at, v);
        }
    };
    const bool full_rows = (lanes < 32 ? D == lanes * 4 : D % (kStride * kVec) == 0) && rows % it.step == 0;
    for (; it.begin(meets); it.next()) {
        if (full_rows) row(std::true_type{});
        else row(std::false_type{});
    }
    it.end();
}

// Two rows at a time, a block's threads on the same channels of both: parameters are read once for two rows, and the rows' sums
// meet together.
constexpr int kTwoVecs = 2, kTwoMost = 640;
template <typename T, typename TS>
__global__ void __launch_bounds__(kTwoMost, 1)
fwd_two_kernel(const Inputs<3> in, Weights weights, int kind, int post, int act, float eps, TS *r, T *__restrict__ out,
               int64_t rows, int D, int lanes) {
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ Bars bars;
    __shared__ __align__(16) Meeting<false> meet;
    const Cluster<false> cl;
    const Place<kTwoVecs> pl(D, lanes);
    const float inv = 1.f / (float)D;
    const bool has_y = in.from[1] != nullptr, has_gate = in.from[2] != nullptr, meets = post || out != nullptr;
    Rows<true, 3, false> it(in, cl, ring, bars, rows, lanes);
    meet.clear();
    const Weights w = weights.from(pl.channel);
    __syncthreads();
    int half = 0;
    auto two = [&](auto all) {
        using Vs = Vectors<kTwoVecs, all.value>;
        const Vs of[2] = {{pl.count}, {it.row + 1 < rows ? pl.count : 0}};
        const int64_t at = it.row * D + pl.channel;
        typename Vs::V v[2];
        auto times = [&](typename Vs::V (&x)[2], const float *p) {
            of[0].with(p, [&](int j, const Pair (&a)[2]) {
#pragma unroll
                for (int k = 0; k < 2; ++k) x[k][j][0] = x[k][j][0] * a[0], x[k][j][1] = x[k][j][1] * a[1];
            });
        };
        auto plus = [&](typename Vs::V (&x)[2], const float *p) {
            of[0].with(p, [&](int j, const Pair (&a)[2]) {
#pragma unroll
                for (int k = 0; k < 2; ++k) x[k][j][0] = x[k][j][0] + a[0], x[k][j][1] = x[k][j][1] + a[1];
            });
        };
        auto normalise = [&](typename Vs::V (&x)[2]) {
            if (kind == GLA_NORM_LAYER) {
                const float2 o = row_sum(Vs::sum(x[0]), Vs::sum(x[1]), lanes, cl, meet, half);
                of[0].shift(x[0], -o.x * inv), of[1].shift(x[1], -o.y * inv);
            }
            const float2 o = row_sum(Vs::squares(x[0]), Vs::squares(x[1]), lanes, cl, meet, half);
            if (meets) it.refill();
            of[0].times(x[0], rsqrtf(fmaf(o.x, inv, eps))), of[1].times(x[1], rsqrtf(fmaf(o.y, inv, eps)));
        };
        auto fetch = [&](typename Vs::V (&x)[2], const auto *from) {
            of[0].fetch(x[0], from), of[1].fetch(x[1], from + D);
        };
        if (has_y) {
            typename Vs::V u[2];
            fetch(u, it.template at<T>(1, D, pl.channel));
            if (post) {
                normalise(u);
                times(u, w.post_weight);
                plus(u, w.post_bias);
            }
            if (has_gate) {
                typename Vs::V g[2];
                fetch(g, it.template at<T>(2, D, pl.channel));
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    if (act == kSilu) Vs::template gate<kSilu>(g[k]);
                    else if (act == kSigmoid) Vs::template gate<kSigmoid>(g[k]);
#pragma unroll
                    for (int j = 0; j < kTwoVecs; ++j) u[k][j][0] = u[k][j][0] * g[k][j][0], u[k][j][1] = u[k][j][1] * g[k][j][1];
                }
            }
            times(u, w.scale);
            fetch(v, it.template at<TS>(0, D, pl.channel));
#pragma unroll
            for (int k = 0; k < 2; ++k) {
#pragma unroll
                for (int j = 0; j < kTwoVecs; ++j) v[k][j][0] = v[k][j][0] + u[k][j][0], v[k][j][1] = v[k][j][1] + u[k][j][1];
                of[k].store(r + at + k * D, v[k]);
                of[k].clear(v[k]);
            }
        } else {
            fetch(v, it.template at<TS>(0, D, pl.channel));
        }
        if (out != nullptr) {
            normalise(v);
            times(v, w.weight);
            plus(v, w.bias);
            of[0].store(out + at, v[0]), of[1].store(out + at + D, v[1]);
        }
    };
    for (; it.begin(meets); it.next(), it.next()) {
        if (D % (kStride * kTwoVecs) == 0 && it.row + 1 < rows) two(std::true_type{});
        else two(std::false_type{});
    }
    it.end();
}

struct Sums {
    float *dscale, *dpost_weight, *dpost_bias, *dweight, *dbias;
};

// The blocks' parts of two of the sums added up, 32 channels x 8 runs of blocks a block, in a fixed order.
__global__ void __launch_bounds__(256)
sum_kernel(const float *__restrict__ part, int nblocks, int D, bool post, Weights w, Sums to) {
    __shared__ float sm[2][8][33];
    if (blockIdx.y == 0 ? !to.dscale && !to.dpost_weight && !to.dpost_bias : !to.dweight && !to.dbias) return;
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), run = threadIdx.x >> 5;
    float s = 0.f, t = 0.f;
    if (c < D)
#pragma unroll 8
        for (int i = run; i < nblocks; i += 8) {
            const float *from = part + ((int64_t)i * kSums + blockIdx.y * 2) * D + c;
            s += __ldg(from), t += __ldg(from + D);
        }
    sm[0][run][threadIdx.x & 31] = s;
    sm[1][run][threadIdx.x & 31] = t;
    __syncthreads();
    if (run != 0 || c >= D) return;
    s = t = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += sm[0][i][threadIdx.x & 31], t += sm[1][i][threadIdx.x & 31];
    if (blockIdx.y == 1) {
        if (to.dweight) to.dweight[c] = s;
        if (to.dbias) to.dbias[c] = t;
        return;
    }
    const float scale = w.scale ? w.scale[c] : 1.f;
    if (to.dscale) to.dscale[c] = post ? fmaf(w.post_weight ? w.post_weight[c] : 1.f, s, w.post_bias ? w.post_bias[c] * t : 0.f) : s;
    if (to.dpost_weight) to.dpost_weight[c] = scale * s;
    if (to.dpost_bias) to.dpost_bias[c] = scale * t;
}

template <typename T, typename TS>
int launch_fwd(const void *x, const void *y, const void *gate, const Weights &w, int kind, int post, int act, float eps,
                void *r, void *out, int64_t rows, int D, cudaStream_t st) {
    const Plan pl = make_plan(D, kFwdVecs, 16384);
    constexpr int e = sizeof(T), es = sizeof(TS);
    Inputs<3> in{{x, y, gate}, {D * es, D * e, D * e}};
    const int n = per_sm(pl, kFwdThreads), nu = units(pl, rows, n);
    int params_at, bytes = lay_out(in, pl, rows, n, nu, 0, params_at);
    // Two blocks of a wide row each want the L1 for the parameters more than stages (8,192 x 5,120 bf16, one row at a time:
    // 123 us, 149 with stages; one block, 4,096 x 8,192: 125 and 107).
    if (n > 1 && pl.threads > 256) in.stages = bytes = 0;
    // Two rows at a time where that has as many rows on an SM, however many a call has, so that a row's result does not depend on
    // the others (all parts, bf16, two and one:
    // 16,435 x 2,552 104 and 123 us, 69,905 x 600 135 and 176, 8,192 x 5,120 104 and 123, 16,384 x 2,560 97 and 99; with fewer
    // rows on an SM, 10,240 x 4,096 118 and 92).  What stages leave of shared memory caches the parameters: 60 KB on an SM where
    // there is a choice of stages, less where two take more (f32 of all parts at 4,616 channels 1 KB: 4,543 rows 85 us; at 4,864, one
    // row at a time, 4,311 rows 91).
    const Plan p2 = make_plan(D, kTwoVecs, 16384);
    const int n2 = per_sm(p2, kTwoMost), room = kMostShared / n2 - (n2 == 1 ? 0 : 3328);
    Inputs<3> two{{x, y, gate}, {D * es, D * e, D * e}};
    two.passes = 2;
    for (int i = 0; i < 3; ++i) {
        two.at[i] = two.stage_bytes;
        if (two.from[i] != nullptr) two.stage_bytes += (2 * two.row_bytes[i] + 127) / 128 * 128;
    }
    two.stages = (room - 60 * 1024 / n2) / two.stage_bytes;
    two.stages = two.stages < 2 ? 2 : two.stages > kMaxStages ? kMaxStages : two.stages;
    if (p2.lanes > 32 && p2.threads <= kTwoMost && 2 * n2 >= n * pl.rows && 2 * two.stage_bytes <= room)
        return launch<fwd_two_kernel<T, TS>>(units(p2, (rows + 1) / 2, n2), 1, p2.threads, two.stages * two.stage_bytes, st, two, w, kind,
                                             post, act, eps, (TS *)r, (T *)out, rows, D, p2.lanes);
#define GLA_RUN(V, S, N)                                                                                                   \
    return launch<fwd_kernel<T, TS, V, S, N>>(nu, 1, pl.threads, bytes, st, in, w, kind, post, act, eps, (TS *)r, (T *)out, rows, D, pl.lanes);
    if (pl.vecs < kFwdVecs && in.stages < 2) return 0;  // (so few channels always have room)
    if (pl.vecs == 1) GLA_RUN(1, true, 256)
    if (pl.vecs == 2) GLA_RUN(2, true, 256)
    if (in.stages > 0) {
        if (pl.threads <= 256) GLA_RUN(kFwdVecs, true, 256)
        if (pl.threads <= 512) GLA_RUN(kFwdVecs, true, 512)
        GLA_RUN(kFwdVecs, true, 1024)
    }
    if (pl.threads <= 256) GLA_RUN(kFwdVecs, false, 256)
    if (pl.threads <= 512) GLA_RUN(kFwdVecs, false, 512)
    GLA_RUN(kFwdVecs, false, 1024)
#undef GLA_RUN
}

}  // namespace

int64_t workspace(int64_t rows, int D) { return bwd_units(rows < 1 ? 1 : rows, D) * kSums * D * (int64_t)sizeof(float); }

int fwd(const void *x, const void *y, const void *gate, const float *scale, const float *post_weight, const float *post_bias,
        const float *weight, const float *bias, int kind, int post, int act, float eps, void *r, void *out, int64_t rows, int D,
        int dtype, int stream_dtype, cudaStream_t st) {
    if (rows == 0) return GLA_OK;
    const Weights w{scale, post_weight, post_bias, weight, bias};
    const auto run = dtype == GLA_F32 ? launch_fwd<float, float> : stream_dtype == GLA_F32 ? launch_fwd<__nv_bfloat16, float>
                                                                                          : launch_fwd<__nv_bfloat16, __nv_bfloat16>;
    const bool ok = 0 < run(x, y, gate, w, kind, post, act, eps, r, out, rows, D, st);
    count_launches(1);
    return ok && cudaGetLastError() == cudaSuccess ? GLA_OK : GLA_ERR_LAUNCH;
}

int bwd(const void *dr, const void *dout, const void *r, const void *y, const void *gate, const float *scale,
        const float *post_weight, const float *post_bias, const float *weight, int kind, int post, int act, float eps, void *dx,
        void *dy, void *dgate, float *dscale, float *dpost_weight, float *dpost_bias, float *dweight, float *dbias, int64_t rows,
        int D, int dtype, int stream_dtype, void *ws, cudaStream_t st) {
    int parts = 0;
    bool ok = true;
    if (rows > 0) {
        const auto run = dtype == GLA_F32 ? bwd_f32 : stream_dtype == GLA_F32 ? bwd_mixed : bwd_bf16;
        parts = run(dr, dout, r, y, gate, scale, post_weight, post_bias, weight, kind, post, act, eps, dx, dy, dgate, (float *)ws, rows, D, st);
        ok = parts > 0;
        count_launches(1);
    }
    if (dscale || dpost_weight || dpost_bias || dweight || dbias) {
        sum_kernel<<<dim3((unsigned)((D + 31) / 32), kSums / 2), 256, 0, st>>>(
            (const float *)ws, parts, D, post != 0, {scale, post_weight, post_bias, weight, nullptr},
            {dscale, dpost_weight, dpost_bias, dweight, dbias});
        count_launches(1);
    }
    return ok && cudaGetLastError() == cudaSuccess ? GLA_OK : GLA_ERR_LAUNCH;
}

}  // namespace resnorm
}  // namespace gla
