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
//
// A row is one block's, or a part of a warp's where it is short; a thread keeps the same channels for all of its rows, so the
// sums over tokens stay in registers until its last row.
#include "gla_act.cuh"

namespace gla {
namespace resnorm {
namespace {

constexpr int kSums = 5;  // dscale, dpost_weight, dpost_bias, dweight, dbias

// Threads to a row (whole warps above 32) and vectors of four channels to a thread.
struct Plan {
    int lanes, vecs, rows, threads;  // rows: of a block at a time
};

Plan make_plan(int D) {
    const int nv = D / 4;
    Plan p{};
    p.vecs = nv <= 2048 ? (nv <= 32 ? 1 : 2) : 4;
    const int need = (nv + p.vecs - 1) / p.vecs;
    p.lanes = 1;
    if (need <= 32)
        while (p.lanes < need) p.lanes *= 2;
    else
        p.lanes = (need + 31) / 32 * 32;
    p.rows = p.lanes <= 32 ? 128 / p.lanes : 1;
    p.threads = p.lanes * p.rows;
    return p;
}

template <typename T> struct Four;  // four channels of one row
template <> struct Four<__nv_bfloat16> {
    using Raw = uint2;
    static __device__ __forceinline__ void open(Raw w, Pair (&x)[2]) {
        x[0] = pair(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u));
        x[1] = pair(__uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
    }
    static __device__ __forceinline__ Raw close(const Pair (&x)[2]) {
        const float2 f = parts(x[0]), g = parts(x[1]);
        const __nv_bfloat162 u = __floats2bfloat162_rn(f.x, f.y), v = __floats2bfloat162_rn(g.x, g.y);
        return make_uint2(*reinterpret_cast<const uint32_t *>(&u), *reinterpret_cast<const uint32_t *>(&v));
    }
};
template <> struct Four<float> {
    using Raw = float4;
    static __device__ __forceinline__ void open(Raw w, Pair (&x)[2]) {
        x[0] = pair(w.x, w.y);
        x[1] = pair(w.z, w.w);
    }
    static __device__ __forceinline__ Raw close(const Pair (&x)[2]) {
        const float2 f = parts(x[0]), g = parts(x[1]);
        return make_float4(f.x, f.y, g.x, g.y);
    }
};

// A thread's place: its row in the block, its first channel and how many of its vectors exist.
struct Place {
    int row, channel, count, stride;
    __device__ __forceinline__ Place(int D, int lanes) {
        const int lane = threadIdx.x % lanes, nv = D >> 2;
        row = threadIdx.x / lanes;
        channel = lane * 4;
        stride = lanes * 4;
        count = lane < nv ? (nv - lane + lanes - 1) / lanes : 0;
    }
};

template <typename T, int kVec>
__device__ __forceinline__ void fetch(Pair (&v)[kVec][2], const T *from, int64_t at, const Place &pl, bool has) {
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        if (has && j < pl.count)
            Four<T>::open(__ldcs(reinterpret_cast<const typename Four<T>::Raw *>(from + at + pl.channel + j * pl.stride)), v[j]);
        else v[j][0] = v[j][1] = both(0.f);
    }
}
template <typename T>
__device__ __forceinline__ void put(T *to, int64_t at, const Place &pl, int j, const Pair (&x)[2]) {
    __stcs(reinterpret_cast<typename Four<T>::Raw *>(to + at + pl.channel + j * pl.stride), Four<T>::close(x));
}
// four parameters of vector j, or a constant where there are none
__device__ __forceinline__ void param(Pair (&v)[2], const float *from, const Place &pl, int j, float otherwise) {
    float4 f = make_float4(otherwise, otherwise, otherwise, otherwise);
    if (from != nullptr && j < pl.count) f = __ldg(reinterpret_cast<const float4 *>(from + pl.channel + j * pl.stride));
    v[0] = pair(f.x, f.y);
    v[1] = pair(f.z, f.w);
}

// Two sums over a row's threads at once.  Rows of more than a warp meet in shared memory, in one half of it after the other,
// so that one barrier a sum is enough; every thread of the block calls this.
struct Meeting {
    float2 at[2][32];
};
__device__ __forceinline__ float2 row_sum(float2 s, int lanes, Meeting &m, int &half) {
    for (int d = min(lanes, 32) >> 1; d > 0; d >>= 1) {
        s.x += __shfl_xor_sync(0xffffffffu, s.x, d);
        s.y += __shfl_xor_sync(0xffffffffu, s.y, d);
    }
    if (lanes > 32) {
        if ((threadIdx.x & 31) == 0) m.at[half][threadIdx.x >> 5] = s;
        __syncthreads();
        s = make_float2(0.f, 0.f);
        for (int w = 0; w < lanes >> 5; ++w) {
            s.x += m.at[half][w].x;
            s.y += m.at[half][w].y;
        }
        half ^= 1;
    }
    return s;
}

// v becomes n(v) without its root; returns the root's reciprocal.  An absent vector stays zero.
template <int kVec>
__device__ __forceinline__ float centre(Pair (&v)[kVec][2], const Place &pl, int kind, float inv, float eps, int lanes,
                                        Meeting &m, int &half) {
    if (kind == GLA_NORM_LAYER) {
        Pair s = both(0.f);
#pragma unroll
        for (int j = 0; j < kVec; ++j) s = s + (v[j][0] + v[j][1]);
        const float mean = row_sum(make_float2(total(s), 0.f), lanes, m, half).x * inv;
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            const Pair less = both(j < pl.count ? -mean : 0.f);
            v[j][0] = v[j][0] + less;
            v[j][1] = v[j][1] + less;
        }
    }
    Pair s = both(0.f);
#pragma unroll
    for (int j = 0; j < kVec; ++j) s = fma(v[j][0], v[j][0], fma(v[j][1], v[j][1], s));
    return rsqrtf(fmaf(row_sum(make_float2(total(s), 0.f), lanes, m, half).x, inv, eps));
}

struct Weights {
    const float *scale, *post_weight, *post_bias, *weight, *bias;
};

template <typename T, typename TS, int kVec>
__global__ void __launch_bounds__(1024)
fwd_kernel(const TS *__restrict__ x, const T *__restrict__ y, const T *__restrict__ gate, Weights w, int kind, int post, int act,
           float eps, TS *__restrict__ r, T *__restrict__ out, int64_t rows, int D, int lanes) {
    __shared__ Meeting meet;
    int half = 0;
    const Place pl(D, lanes);
    const int step = blockDim.x / lanes;
    const float inv = 1.f / (float)D;
    for (int64_t r0 = (int64_t)blockIdx.x * step; r0 < rows; r0 += (int64_t)gridDim.x * step) {
        const int64_t row = r0 + pl.row, at = row * D;
        const bool on = row < rows;
        Pair v[kVec][2];
        fetch<TS, kVec>(v, x, at, pl, on);
        if (y != nullptr) {
            Pair u[kVec][2], g[kVec][2];
            fetch<T, kVec>(u, y, at, pl, on);
            if (gate != nullptr) fetch<T, kVec>(g, gate, at, pl, on);
            Pair q = both(1.f);
            if (post) q = both(centre<kVec>(u, pl, kind, inv, eps, lanes, meet, half));
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                Pair pw[2], pb[2], sc[2];
                param(pw, w.post_weight, pl, j, 1.f);
                param(pb, w.post_bias, pl, j, 0.f);
                param(sc, w.scale, pl, j, 1.f);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (post) u[j][e] = fma(u[j][e] * q, pw[e], pb[e]);
                    if (gate != nullptr) u[j][e] = u[j][e] * activation(g[j][e], act);
                    v[j][e] = w.scale != nullptr ? fma(u[j][e], sc[e], v[j][e]) : v[j][e] + u[j][e];
                }
                if (on && j < pl.count) put<TS>(r, at, pl, j, v[j]);
                if (j >= pl.count) v[j][0] = v[j][1] = both(0.f);
            }
        }
        if (out != nullptr) {
            const Pair q = both(centre<kVec>(v, pl, kind, inv, eps, lanes, meet, half));
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                Pair pw[2], pb[2];
                param(pw, w.weight, pl, j, 1.f);
                param(pb, w.bias, pl, j, 0.f);
#pragma unroll
                for (int e = 0; e < 2; ++e) v[j][e] = fma(v[j][e] * q, pw[e], pb[e]);
                if (on && j < pl.count) put<T>(out, at, pl, j, v[j]);
            }
        }
    }
}

template <typename T, typename TS, int kVec>
__global__ void __launch_bounds__(1024)
bwd_kernel(const TS *__restrict__ dr, const T *__restrict__ dout, const TS *__restrict__ r, const T *__restrict__ y,
           const T *__restrict__ gate, Weights w, int kind, int post, int act, float eps, TS *__restrict__ dx,
           T *__restrict__ dy, T *__restrict__ dgate, float *__restrict__ part, int64_t rows, int D, int lanes) {
    __shared__ Meeting meet;
    __shared__ float4 tops[128];
    int half = 0;
    const Place pl(D, lanes);
    const int step = blockDim.x / lanes;
    const float inv = 1.f / (float)D;
    Pair sums[kSums][kVec][2];
#pragma unroll
    for (int i = 0; i < kSums; ++i)
#pragma unroll
        for (int j = 0; j < kVec; ++j) sums[i][j][0] = sums[i][j][1] = both(0.f);
    for (int64_t r0 = (int64_t)blockIdx.x * step; r0 < rows; r0 += (int64_t)gridDim.x * step) {
        const int64_t row = r0 + pl.row, at = row * D;
        const bool on = row < rows;
        Pair d[kVec][2];
        fetch<TS, kVec>(d, dr, at, pl, on && dr != nullptr);
        if (dout != nullptr) {
            Pair h[kVec][2], up[kVec][2];
            fetch<TS, kVec>(h, r, at, pl, on);
            fetch<T, kVec>(up, dout, at, pl, on);
            const float q = centre<kVec>(h, pl, kind, inv, eps, lanes, meet, half);
            Pair s1 = both(0.f), s2 = both(0.f);
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                Pair pw[2];
                param(pw, w.weight, pl, j, 1.f);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    h[j][e] = h[j][e] * both(q);
                    sums[3][j][e] = fma(up[j][e], h[j][e], sums[3][j][e]);
                    sums[4][j][e] = sums[4][j][e] + up[j][e];
                    up[j][e] = up[j][e] * pw[e];
                    s1 = s1 + up[j][e];
                    s2 = fma(up[j][e], h[j][e], s2);
                }
            }
            const float2 s = row_sum(make_float2(total(s1), total(s2)), lanes, meet, half);
            const Pair m1 = both(kind == GLA_NORM_LAYER ? -s.x * inv : 0.f), m2 = both(-s.y * inv);
#pragma unroll
            for (int j = 0; j < kVec; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) d[j][e] = fma(fma(h[j][e], m2, up[j][e] + m1), both(q), d[j][e]);
        }
#pragma unroll
        for (int j = 0; j < kVec; ++j)
            if (on && j < pl.count) put<TS>(dx, at, pl, j, d[j]);
        if (y == nullptr) continue;
        Pair u[kVec][2], g[kVec][2];
        fetch<T, kVec>(u, y, at, pl, on);
        if (gate != nullptr) fetch<T, kVec>(g, gate, at, pl, on);
        float uq = 1.f;
        if (post) uq = centre<kVec>(u, pl, kind, inv, eps, lanes, meet, half);
        Pair s1 = both(0.f), s2 = both(0.f);
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            Pair pw[2], pb[2], sc[2];
            param(pw, w.post_weight, pl, j, 1.f);
            param(pb, w.post_bias, pl, j, 0.f);
            param(sc, w.scale, pl, j, 1.f);
            const bool has = on && j < pl.count;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (!has) d[j][e] = both(0.f);
                if (post) u[j][e] = u[j][e] * both(uq);
                const Pair z = post ? fma(u[j][e], pw[e], pb[e]) : u[j][e];
                Pair slope = both(0.f), f = both(1.f);
                if (gate != nullptr) f = activation(g[j][e], act, slope);
                const Pair df = d[j][e] * f;
                sums[0][j][e] = fma(df, z, sums[0][j][e]);
                if (gate != nullptr) g[j][e] = d[j][e] * sc[e] * z * slope;
                d[j][e] = df * sc[e];
                if (post) {
                    sums[1][j][e] = fma(d[j][e], u[j][e], sums[1][j][e]);
                    sums[2][j][e] = sums[2][j][e] + d[j][e];
                    d[j][e] = d[j][e] * pw[e];
                    s1 = s1 + d[j][e];
                    s2 = fma(d[j][e], u[j][e], s2);
                }
            }
            if (gate != nullptr && has) put<T>(dgate, at, pl, j, g[j]);
        }
        if (post) {
            const float2 s = row_sum(make_float2(total(s1), total(s2)), lanes, meet, half);
            const Pair m1 = both(kind == GLA_NORM_LAYER ? -s.x * inv : 0.f), m2 = both(-s.y * inv);
#pragma unroll
            for (int j = 0; j < kVec; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) d[j][e] = fma(u[j][e], m2, d[j][e] + m1) * both(uq);
        }
#pragma unroll
        for (int j = 0; j < kVec; ++j)
            if (on && j < pl.count) put<T>(dy, at, pl, j, d[j]);
    }
    // the block's rows of one channel set meet in shared memory; one writer per channel
    float *to = part + (int64_t)blockIdx.x * kSums * D;
#pragma unroll
    for (int i = 0; i < kSums; ++i)
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            float4 v = Four<float>::close(sums[i][j]);
            if (step > 1) {
                __syncthreads();
                tops[threadIdx.x] = v;
                __syncthreads();
                if (pl.row == 0)
                    for (int m = 1; m < step; ++m) {
                        const float4 o = tops[threadIdx.x + m * lanes];
                        v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
                    }
            }
            if (pl.row == 0 && j < pl.count)
                *reinterpret_cast<float4 *>(to + (int64_t)i * D + pl.channel + j * pl.stride) = v;
        }
}

struct Sums {
    float *to[kSums];
};

// The blocks' parts of every sum added up, 32 channels x 8 runs of blocks a block, in a fixed order.
__global__ void __launch_bounds__(256)
sum_kernel(const float *__restrict__ part, int nblocks, int D, Sums sums) {
    __shared__ float sm[8][33];
    float *to = sums.to[blockIdx.y];
    if (to == nullptr) return;
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), run = threadIdx.x >> 5;
    float s = 0.f;
    if (c < D)
#pragma unroll 8
        for (int i = run; i < nblocks; i += 8) s += __ldg(part + ((int64_t)i * kSums + blockIdx.y) * D + c);
    sm[run][threadIdx.x & 31] = s;
    __syncthreads();
    if (run == 0 && c < D) {
        s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += sm[i][threadIdx.x & 31];
        to[c] = s;
    }
}

int blocks(const Plan &pl, int64_t rows, int per_sm) {
    const int64_t need = (rows + pl.rows - 1) / pl.rows;
    int64_t most = (int64_t)device_info().sm_count * per_sm;
    if (most < 1) most = 1;
    return (int)(need < most ? need : most);
}
int fwd_per_sm(const Plan &pl) { return 2048 / pl.threads < 1 ? 1 : 2048 / pl.threads; }
int bwd_per_sm(const Plan &pl) { return 512 / pl.threads < 1 ? 1 : 512 / pl.threads; }

#define GLA_BY_VEC(RUN, T, TS)            \
    switch (pl.vecs) {                    \
        case 1: RUN(T, TS, 1); break;     \
        case 2: RUN(T, TS, 2); break;     \
        default: RUN(T, TS, 4); break;    \
    }
#define GLA_BY_TYPE(RUN)                                                                          \
    if (dtype == GLA_F32) { GLA_BY_VEC(RUN, float, float) }                                       \
    else if (stream_dtype == GLA_F32) { GLA_BY_VEC(RUN, __nv_bfloat16, float) }                   \
    else { GLA_BY_VEC(RUN, __nv_bfloat16, __nv_bfloat16) }

}  // namespace

int64_t workspace(int64_t rows, int D) {
    const Plan pl = make_plan(D);
    return (int64_t)blocks(pl, rows < 1 ? 1 : rows, bwd_per_sm(pl)) * kSums * D * (int64_t)sizeof(float);
}

int fwd(const void *x, const void *y, const void *gate, const float *scale, const float *post_weight, const float *post_bias,
        const float *weight, const float *bias, int kind, int post, int act, float eps, void *r, void *out, int64_t rows, int D,
        int dtype, int stream_dtype, cudaStream_t st) {
    if (rows == 0) return GLA_OK;
    const Plan pl = make_plan(D);
    const Weights w{scale, post_weight, post_bias, weight, bias};
    const unsigned grid = (unsigned)blocks(pl, rows, fwd_per_sm(pl));
#define GLA_RUN(T, TS, V)                                                                                             \
    fwd_kernel<T, TS, V><<<grid, pl.threads, 0, st>>>((const TS *)x, (const T *)y, (const T *)gate, w, kind, post,    \
                                                      act, eps, (TS *)r, (T *)out, rows, D, pl.lanes)
    GLA_BY_TYPE(GLA_RUN)
#undef GLA_RUN
    count_launches(1);
    return cudaGetLastError() == cudaSuccess ? GLA_OK : GLA_ERR_LAUNCH;
}

int bwd(const void *dr, const void *dout, const void *r, const void *y, const void *gate, const float *scale,
        const float *post_weight, const float *post_bias, const float *weight, int kind, int post, int act, float eps, void *dx,
        void *dy, void *dgate, float *dscale, float *dpost_weight, float *dpost_bias, float *dweight, float *dbias, int64_t rows,
        int D, int dtype, int stream_dtype, void *ws, cudaStream_t st) {
    const Plan pl = make_plan(D);
    const Weights w{scale, post_weight, post_bias, weight, nullptr};
    const int nb = rows > 0 ? blocks(pl, rows, bwd_per_sm(pl)) : 0;
    if (nb > 0) {
#define GLA_RUN(T, TS, V)                                                                                                   \
    bwd_kernel<T, TS, V><<<(unsigned)nb, pl.threads, 0, st>>>((const TS *)dr, (const T *)dout, (const TS *)r, (const T *)y, \
                                                              (const T *)gate, w, kind, post, act, eps, (TS *)dx, (T *)dy,  \
                                                              (T *)dgate, (float *)ws, rows, D, pl.lanes)
        GLA_BY_TYPE(GLA_RUN)
#undef GLA_RUN
        count_launches(1);
    }
    if (dscale || dpost_weight || dpost_bias || dweight || dbias) {
        const Sums sums{{dscale, dpost_weight, dpost_bias, dweight, dbias}};
        sum_kernel<<<dim3((unsigned)((D + 31) / 32), kSums), 256, 0, st>>>((const float *)ws, nb, D, sums);
        count_launches(1);
    }
    return cudaGetLastError() == cudaSuccess ? GLA_OK : GLA_ERR_LAUNCH;
}

}  // namespace resnorm
}  // namespace gla
