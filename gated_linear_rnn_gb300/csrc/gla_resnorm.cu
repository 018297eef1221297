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
// Both are bound by HBM.  A row is one block's, or a part of a warp's where it is short; a thread takes four neighbouring
// channels at a time and keeps the same ones for all of its rows, so the gradient's sums over tokens stay in registers until
// its last row.  Rows come into shared memory by bulk copies, some rows ahead, and are read from there by each step that needs
// them: what is in flight and what a later step needs costs no registers, of which the sums take most.  Rows that two stages
// have no room for are read from memory each time.
#include "gla_act.cuh"
#include "sm100_ptx.cuh"

GLA_DEFINE_STATUS(resnorm)

namespace gla {
namespace resnorm {
namespace {

constexpr int kSums = 5;  // dscale, dpost_weight, dpost_bias, dweight, dbias
constexpr int kMaxStages = 6;
constexpr int kRowsThreads = 256;  // of a block with several rows
constexpr uint64_t kWaitNs = 2000000000ull;

// Threads to a row (whole warps above 32), vectors of four channels to a thread, rows of a block at a time.
struct Plan {
    int lanes, vecs, rows, threads;
};

Plan make_plan(int D, int vecs) {
    const int nv = D / 4;
    Plan p{};
    p.vecs = (nv + vecs - 1) / vecs <= 1024 ? vecs : 4;
    const int need = (nv + p.vecs - 1) / p.vecs;
    p.lanes = 1;
    if (need <= 32)
        while (p.lanes < need) p.lanes *= 2;
    else
        p.lanes = (need + 31) / 32 * 32;
    p.rows = p.lanes <= 32 ? kRowsThreads / p.lanes : 1;
    p.threads = p.lanes * p.rows;
    return p;
}
constexpr int kFwdVecs = 4, kBwdVecs = 2;

template <typename T> struct Four;  // four channels of one row
template <> struct Four<__nv_bfloat16> {
    using Raw = uint2;
    static __device__ __forceinline__ void open(Pair (&x)[2], Raw w) {
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
    static __device__ __forceinline__ void open(Pair (&x)[2], Raw w) {
        x[0] = pair(w.x, w.y);
        x[1] = pair(w.z, w.w);
    }
    static __device__ __forceinline__ Raw close(const Pair (&x)[2]) {
        const float2 f = parts(x[0]), g = parts(x[1]);
        return make_float4(f.x, f.y, g.x, g.y);
    }
};
template <typename T> __device__ __forceinline__ void put(T *to, const Pair (&x)[2]) {
    __stcs(reinterpret_cast<typename Four<T>::Raw *>(to), Four<T>::close(x));
}

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

// Four parameters, or a constant where there are none.
__device__ __forceinline__ void param(Pair (&v)[2], const float *from, int channel, float otherwise) {
    if (from != nullptr) Four<float>::open(v, __ldg(reinterpret_cast<const float4 *>(from + channel)));
    else v[0] = v[1] = both(otherwise);
}

// Two sums over a row's threads at once.  Rows of more than a warp meet in shared memory, in one half of it after the other,
// so that one barrier a sum is enough; every thread of the block calls this.
struct Meeting {
    float2 at[2][32];
};
__device__ __forceinline__ float2 row_sum(float2 s, int lanes, Meeting &m, int &half) {
    if (lanes < 32) {
        for (int d = lanes >> 1; d > 0; d >>= 1) {
            s.x += __shfl_xor_sync(0xffffffffu, s.x, d);
            s.y += __shfl_xor_sync(0xffffffffu, s.y, d);
        }
        return s;
    }
    // one half of the warp adds the one sum up, the other half the other
    const bool upper = threadIdx.x & 16;
    float v = (upper ? s.y : s.x) + __shfl_xor_sync(0xffffffffu, upper ? s.x : s.y, 16);
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    if (lanes == 32) {
        const float o = __shfl_xor_sync(0xffffffffu, v, 16);
        return upper ? make_float2(o, v) : make_float2(v, o);
    }
    if ((threadIdx.x & 15) == 0) reinterpret_cast<float *>(&m.at[half][threadIdx.x >> 5])[upper] = v;
    __syncthreads();
    s = make_float2(0.f, 0.f);
    const int warps = lanes >> 5;
#pragma unroll 4
    for (int w = 0; w < warps; w += 2) {  // the one past an odd number is zero
        const float4 f = *reinterpret_cast<const float4 *>(&m.at[half][w]);
        s.x += f.x + f.z;
        s.y += f.y + f.w;
    }
    half ^= 1;
    return s;
}
__device__ __forceinline__ void clear(Meeting &m) {
    if (threadIdx.x < 32) m.at[0][threadIdx.x] = m.at[1][threadIdx.x] = make_float2(0.f, 0.f);
}

// Arrays whose rows come in, and the stages that they come into: a block's rows of each array at a time.
template <int kArrays> struct Inputs {
    const void *from[kArrays];  // null: absent
    int row_bytes[kArrays], at[kArrays];
    int stage_bytes, stages;
};

// The rows of a block, one item (its rows at a time) after the other.
template <bool kStage, int kArrays>
struct Rows {
    const Inputs<kArrays> &in;
    uint8_t *ring;
    uint64_t *full;
    int *failed;
    int64_t rows, items, item;
    int step, st;
    uint32_t phase;
    bool first;
    __device__ __forceinline__ Rows(const Inputs<kArrays> &in_, uint8_t *ring_, uint64_t *full_, int *failed_, int64_t rows_, int lanes)
        : in(in_), ring(ring_), full(full_), failed(failed_), rows(rows_), item(blockIdx.x), step(blockDim.x / lanes), st(0), phase(0),
          first(true) {
        items = (rows + step - 1) / step;
        if (!kStage) return;
        if (threadIdx.x == 0) {
            *failed = 0;
            for (int i = 0; i < in.stages; ++i) ptx::mbar_init(ptx::smem_u32(full + i), 1);
            ptx::fence_mbar_init();
            for (int i = 0; i < in.stages; ++i) order(i, item + i * (int64_t)gridDim.x);
        }
    }
    // by one thread
    __device__ __forceinline__ void order(int to_stage, int64_t k) const {
        if (k >= items) return;
        const uint32_t b = ptx::smem_u32(full + to_stage), to = ptx::smem_u32(ring) + (uint32_t)(to_stage * in.stage_bytes);
        const int n = (int)min((int64_t)step, rows - k * step);
        uint32_t bytes = 0;
#pragma unroll
        for (int i = 0; i < kArrays; ++i)
            if (in.from[i] != nullptr) bytes += (uint32_t)(n * in.row_bytes[i]);
        ptx::mbar_expect_tx(b, bytes);
#pragma unroll
        for (int i = 0; i < kArrays; ++i)
            if (in.from[i] != nullptr)
                ptx::bulk_load_g2s(to + (uint32_t)in.at[i], (const uint8_t *)in.from[i] + k * step * in.row_bytes[i],
                                   (uint32_t)(n * in.row_bytes[i]), b);
    }
    __device__ __forceinline__ bool more() const { return item < items; }
    __device__ __forceinline__ void arrive() const {
        if (kStage && !ptx::mbar_wait(ptx::smem_u32(full + st), phase, failed, kWaitNs)) *(volatile int *)failed = 1;
    }
    // All threads of the block are past the item before: its stage takes another one.
    __device__ __forceinline__ void refill() const {
        if (kStage && threadIdx.x == 0 && !first) order(st == 0 ? in.stages - 1 : st - 1, item + (in.stages - 1) * (int64_t)gridDim.x);
    }
    __device__ __forceinline__ void next() {
        first = false;
        item += gridDim.x;
        if (kStage && ++st == in.stages) {
            st = 0;
            phase ^= 1u;
        }
    }
    // what a block that gave up has ordered still comes in
    __device__ __forceinline__ void end() const {
        if (kStage && threadIdx.x == 0 && *(volatile int *)failed) {
            record_status(GLA_ERR_TIMEOUT);
            for (int i = 0; i < in.stages; ++i) ptx::mbar_wait(ptx::smem_u32(full + i), phase ^ (uint32_t)(i < st), nullptr, kWaitNs);
        }
    }
    // four channels of array i
    template <typename T> __device__ __forceinline__ void get(Pair (&v)[2], int i, int row_in_item, int D, int channel) const {
        using Raw = typename Four<T>::Raw;
        if (kStage)
            Four<T>::open(v, *reinterpret_cast<const Raw *>(ring + st * in.stage_bytes + in.at[i] +
                                                            (row_in_item * D + channel) * (int)sizeof(T)));
        else
            Four<T>::open(v, __ldg(reinterpret_cast<const Raw *>((const T *)in.from[i] + (item * step + row_in_item) * D + channel)));
    }
};

struct Weights {
    const float *scale, *post_weight, *post_bias, *weight, *bias;
};

// The mean (of a layer norm; else 0) and the reciprocal root of one or two arrays' rows: GET(0 or 1, j, v) reads vector j.
template <int kVec, class Get>
__device__ __forceinline__ void statistics(Get get, bool one, bool two, int count, int kind, float inv, float eps, int lanes, Meeting &m,
                                           int &half, float2 &mean, float2 &root) {
    mean = make_float2(0.f, 0.f);
    if (kind == GLA_NORM_LAYER) {
        Pair s = both(0.f), t = both(0.f), v[2];
#pragma unroll
        for (int j = 0; j < kVec; ++j)
            if (j < count) {
                if (one) get(0, j, v), s = s + (v[0] + v[1]);
                if (two) get(1, j, v), t = t + (v[0] + v[1]);
            }
        mean = row_sum(make_float2(total(s), total(t)), lanes, m, half);
        mean.x *= inv, mean.y *= inv;
    }
    Pair s = both(0.f), t = both(0.f), v[2];
    const Pair a = both(-mean.x), b = both(-mean.y);
#pragma unroll
    for (int j = 0; j < kVec; ++j)
        if (j < count) {
            if (one) {
                get(0, j, v);
                v[0] = v[0] + a, v[1] = v[1] + a;
                s = fma(v[0], v[0], fma(v[1], v[1], s));
            }
            if (two) {
                get(1, j, v);
                v[0] = v[0] + b, v[1] = v[1] + b;
                t = fma(v[0], v[0], fma(v[1], v[1], t));
            }
        }
    root = row_sum(make_float2(total(s), total(t)), lanes, m, half);
    root.x = rsqrtf(fmaf(root.x, inv, eps)), root.y = rsqrtf(fmaf(root.y, inv, eps));
}

template <typename T, typename TS, int kVec, bool kStage, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads <= 256 ? 3 : 1)
fwd_kernel(Inputs<3> in, Weights w, int kind, int post, int act, float eps, TS *__restrict__ r, T *__restrict__ out, int64_t rows,
           int D, int lanes) {
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ uint64_t full[kMaxStages];
    __shared__ int failed;
    __shared__ __align__(16) Meeting meet;
    int half = 0;
    const Place pl(D, lanes);
    const float inv = 1.f / (float)D;
    const bool has_y = in.from[1] != nullptr, has_gate = in.from[2] != nullptr;
    const bool meets = lanes > 32 && (post || out != nullptr);
    Rows<kStage, 3> it(in, ring, full, &failed, rows, lanes);
    clear(meet);
    __syncthreads();
    for (; it.more(); it.next()) {
        if (!meets) {
            __syncthreads();
            it.refill();
        }
        it.arrive();
        const int64_t row = it.item * it.step + pl.row, at = row * D + pl.channel;
        const int count = row < rows ? pl.count : 0;
        Pair q = both(1.f), m = both(0.f);
        if (post) {
            float2 mean, root;
            statistics<kVec>([&](int, int j, Pair (&v)[2]) { it.template get<T>(v, 1, pl.row, D, pl.channel + j * pl.stride); }, true,
                             false, count, kind, inv, eps, lanes, meet, half, mean, root);
            q = both(root.x), m = both(-mean.x);
            if (meets) it.refill();
        }
        Pair v[kVec][2];
        if (has_y) {
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                v[j][0] = v[j][1] = both(0.f);
                if (j < count) {
                    const int c = pl.channel + j * pl.stride;
                    Pair u[2], g[2], a[2], b[2];
                    it.template get<TS>(v[j], 0, pl.row, D, c);
                    it.template get<T>(u, 1, pl.row, D, c);
                    if (post) {
                        param(a, w.post_weight, c, 1.f);
                        param(b, w.post_bias, c, 0.f);
#pragma unroll
                        for (int e = 0; e < 2; ++e) u[e] = fma((u[e] + m) * q, a[e], b[e]);
                    }
                    if (has_gate) {
                        it.template get<T>(g, 2, pl.row, D, c);
#pragma unroll
                        for (int e = 0; e < 2; ++e) u[e] = u[e] * activation(g[e], act);
                    }
                    param(a, w.scale, c, 1.f);
#pragma unroll
                    for (int e = 0; e < 2; ++e) v[j][e] = fma(u[e], a[e], v[j][e]);
                    put<TS>(r + at + j * pl.stride, v[j]);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                v[j][0] = v[j][1] = both(0.f);
                if (j < count) it.template get<TS>(v[j], 0, pl.row, D, pl.channel + j * pl.stride);
            }
        }
        if (out != nullptr) {
            float2 mean, root;
            statistics<kVec>([&](int, int j, Pair (&x)[2]) { x[0] = v[j][0], x[1] = v[j][1]; }, true, false, count, kind, inv, eps,
                             lanes, meet, half, mean, root);
            if (meets && !post) it.refill();
            q = both(root.x), m = both(-mean.x);
#pragma unroll
            for (int j = 0; j < kVec; ++j)
                if (j < count) {
                    const int c = pl.channel + j * pl.stride;
                    Pair a[2], b[2];
                    param(a, w.weight, c, 1.f);
                    param(b, w.bias, c, 0.f);
#pragma unroll
                    for (int e = 0; e < 2; ++e) a[e] = fma((v[j][e] + m) * q, a[e], b[e]);
                    put<T>(out + at + j * pl.stride, a);
                }
        }
    }
    it.end();
}

template <typename T, typename TS, int kVec, bool kStage, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads <= 320 ? 640 / kThreads : 1)
bwd_kernel(Inputs<5> in, Weights w, int kind, int post, int act, float eps, TS *__restrict__ dx, T *__restrict__ dy,
           T *__restrict__ dgate, float *__restrict__ part, int64_t rows, int D, int lanes) {
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ uint64_t full[kMaxStages];
    __shared__ int failed;
    __shared__ __align__(16) Meeting meet;
    __shared__ float4 tops[kRowsThreads];
    int half = 0;
    const Place pl(D, lanes);
    const float inv = 1.f / (float)D;
    const bool has_dr = in.from[0] != nullptr, has_out = in.from[1] != nullptr, has_y = in.from[3] != nullptr,
               has_gate = in.from[4] != nullptr;
    const bool meets = lanes > 32 && (post || has_out);
    Pair sums[kSums][kVec][2];
#pragma unroll
    for (int i = 0; i < kSums; ++i)
#pragma unroll
        for (int j = 0; j < kVec; ++j) sums[i][j][0] = sums[i][j][1] = both(0.f);
    Rows<kStage, 5> it(in, ring, full, &failed, rows, lanes);
    clear(meet);
    __syncthreads();
    for (; it.more(); it.next()) {
        if (!meets) {
            __syncthreads();
            it.refill();
        }
        it.arrive();
        const int64_t row = it.item * it.step + pl.row, at = row * D + pl.channel;
        const int count = row < rows ? pl.count : 0;
        float2 mean, root;  // of r, and of y
        if (has_out || post) {
            statistics<kVec>(
                [&](int which, int j, Pair (&v)[2]) {
                    if (which == 0) it.template get<TS>(v, 2, pl.row, D, pl.channel + j * pl.stride);
                    else it.template get<T>(v, 3, pl.row, D, pl.channel + j * pl.stride);
                },
                has_out, post, count, kind, inv, eps, lanes, meet, half, mean, root);
            if (meets) it.refill();
        }
        const Pair q = both(root.x), m = both(-mean.x), uq = both(root.y), um = both(-mean.y);
        Pair m1 = both(0.f), m2 = both(0.f);
        if (has_out) {
            Pair s1 = both(0.f), s2 = both(0.f);
#pragma unroll
            for (int j = 0; j < kVec; ++j)
                if (j < count) {
                    const int c = pl.channel + j * pl.stride;
                    Pair up[2], h[2], wt[2];
                    it.template get<T>(up, 1, pl.row, D, c);
                    it.template get<TS>(h, 2, pl.row, D, c);
                    param(wt, w.weight, c, 1.f);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        h[e] = (h[e] + m) * q;
                        sums[3][j][e] = fma(up[e], h[e], sums[3][j][e]);
                        sums[4][j][e] = sums[4][j][e] + up[e];
                        const Pair t = up[e] * wt[e];
                        s1 = s1 + t;
                        s2 = fma(t, h[e], s2);
                    }
                }
            const float2 s = row_sum(make_float2(total(s1), total(s2)), lanes, meet, half);
            m1 = both(kind == GLA_NORM_LAYER ? -s.x * inv : 0.f), m2 = both(-s.y * inv);
        }
        Pair d[kVec][2], s1 = both(0.f), s2 = both(0.f);
#pragma unroll
        for (int j = 0; j < kVec; ++j)
            if (j < count) {
                const int c = pl.channel + j * pl.stride;
                d[j][0] = d[j][1] = both(0.f);
                if (has_dr) it.template get<TS>(d[j], 0, pl.row, D, c);
                if (has_out) {
                    Pair up[2], h[2], wt[2];
                    it.template get<T>(up, 1, pl.row, D, c);
                    it.template get<TS>(h, 2, pl.row, D, c);
                    param(wt, w.weight, c, 1.f);
#pragma unroll
                    for (int e = 0; e < 2; ++e) d[j][e] = fma(fma((h[e] + m) * q, m2, fma(up[e], wt[e], m1)), q, d[j][e]);
                }
                put<TS>(dx + at + j * pl.stride, d[j]);
                if (has_y) {
                    Pair u[2], g[2], pw[2], pb[2], sc[2];
                    it.template get<T>(u, 3, pl.row, D, c);
                    param(sc, w.scale, c, 1.f);
                    if (post) {
                        param(pw, w.post_weight, c, 1.f);
                        param(pb, w.post_bias, c, 0.f);
                    }
                    if (has_gate) it.template get<T>(g, 4, pl.row, D, c);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        Pair z = u[e], df = d[j][e];
                        if (post) {
                            u[e] = (u[e] + um) * uq;
                            z = fma(u[e], pw[e], pb[e]);
                        }
                        if (has_gate) {
                            Pair slope;
                            df = df * activation(g[e], act, slope);
                            g[e] = d[j][e] * sc[e] * z * slope;
                        }
                        sums[0][j][e] = fma(df, z, sums[0][j][e]);
                        df = df * sc[e];
                        if (post) {
                            sums[1][j][e] = fma(df, u[e], sums[1][j][e]);
                            sums[2][j][e] = sums[2][j][e] + df;
                            df = df * pw[e];
                            s1 = s1 + df;
                            s2 = fma(df, u[e], s2);
                        }
                        d[j][e] = df;
                    }
                    if (has_gate) put<T>(dgate + at + j * pl.stride, g);
                    if (!post) put<T>(dy + at + j * pl.stride, d[j]);
                }
            }
        if (post) {
            const float2 s = row_sum(make_float2(total(s1), total(s2)), lanes, meet, half);
            m1 = both(kind == GLA_NORM_LAYER ? -s.x * inv : 0.f), m2 = both(-s.y * inv);
#pragma unroll
            for (int j = 0; j < kVec; ++j)
                if (j < count) {
                    Pair u[2];
                    it.template get<T>(u, 3, pl.row, D, pl.channel + j * pl.stride);
#pragma unroll
                    for (int e = 0; e < 2; ++e) d[j][e] = fma((u[e] + um) * uq, m2, d[j][e] + m1) * uq;
                    put<T>(dy + at + j * pl.stride, d[j]);
                }
        }
    }
    it.end();
    // the block's rows of one channel set meet in shared memory; one writer per channel
    float *to = part + (int64_t)blockIdx.x * kSums * D;
    const int step = blockDim.x / lanes;
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
// Blocks of an SM: as many as the threads' registers allow, 85 a thread of the forward and 102 of the gradient.
int per_sm(const Plan &pl, int threads) {
    const int n = threads / pl.threads;
    return n < 1 ? 1 : n;
}
constexpr int kFwdThreads = 768, kBwdThreads = 640;

constexpr int kMostShared = 220 * 1024;

// The stages of a block: rows of each array one behind the other.
template <int kArrays> int lay_out(Inputs<kArrays> &in, const Plan &pl, int per_sm) {
    int at = 0;
    for (int i = 0; i < kArrays; ++i) {
        in.at[i] = at;
        if (in.from[i] != nullptr) at += (pl.rows * in.row_bytes[i] + 127) / 128 * 128;
    }
    in.stage_bytes = at;
    const int room = 190 * 1024 / per_sm - 6144;  // what is left caches the parameters
    in.stages = room / at;
    if (in.stages < 2 && per_sm == 1) in.stages = kMostShared / at;
    if (in.stages > kMaxStages) in.stages = kMaxStages;
    if (in.stages < 2) in.stages = 0;
    return in.stages * at;
}

// RUN(T, TS, kVec, kStage, kThreads) for a call's types and plan; kSmall: threads of the kernels that share an SM.
#define GLA_BY_STAGE(RUN, T, TS, V, N)                 \
    if (staged) { RUN(T, TS, V, true, N) }             \
    else { RUN(T, TS, V, false, N) }
#define GLA_BY_PLAN(RUN, T, TS)                                                     \
    if (pl.vecs == kVecs && pl.threads <= kSmall) { GLA_BY_STAGE(RUN, T, TS, kVecs, kSmall) } \
    else if (pl.vecs == kVecs && pl.threads <= 512) { GLA_BY_STAGE(RUN, T, TS, kVecs, 512) }  \
    else if (pl.vecs == kVecs) { GLA_BY_STAGE(RUN, T, TS, kVecs, 1024) }            \
    else { GLA_BY_STAGE(RUN, T, TS, 4, 1024) }
#define GLA_BY_TYPE(RUN)                                                                          \
    if (dtype == GLA_F32) { GLA_BY_PLAN(RUN, float, float) }                                      \
    else if (stream_dtype == GLA_F32) { GLA_BY_PLAN(RUN, __nv_bfloat16, float) }                  \
    else { GLA_BY_PLAN(RUN, __nv_bfloat16, __nv_bfloat16) }

// Lets a kernel use as much shared memory as any call may ask for; asked of the runtime once per kernel and device.
template <auto kKernel> bool allow_most() {
    constexpr int kDevices = 64;
    static std::atomic<bool> allowed[kDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    if (dev < kDevices && allowed[dev].load(std::memory_order_acquire)) return true;
    if (cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostShared) != cudaSuccess) return false;
    if (dev < kDevices) allowed[dev].store(true, std::memory_order_release);
    return true;
}

}  // namespace

int64_t workspace(int64_t rows, int D) {
    const Plan pl = make_plan(D, kBwdVecs);
    return (int64_t)blocks(pl, rows < 1 ? 1 : rows, per_sm(pl, kBwdThreads)) * kSums * D * (int64_t)sizeof(float);
}

int fwd(const void *x, const void *y, const void *gate, const float *scale, const float *post_weight, const float *post_bias,
        const float *weight, const float *bias, int kind, int post, int act, float eps, void *r, void *out, int64_t rows, int D,
        int dtype, int stream_dtype, cudaStream_t st) {
    if (rows == 0) return GLA_OK;
    constexpr int kVecs = kFwdVecs, kSmall = 256;
    const Plan pl = make_plan(D, kVecs);
    const Weights w{scale, post_weight, post_bias, weight, bias};
    const int e = dtype == GLA_F32 ? 4 : 2, es = stream_dtype == GLA_F32 ? 4 : 2, n = per_sm(pl, kFwdThreads);
    Inputs<3> in{{x, y, gate}, {D * es, D * e, D * e}, {}, 0, 0};
    const int bytes = lay_out(in, pl, n);
    const bool staged = in.stages > 0;
    const unsigned grid = (unsigned)blocks(pl, rows, n);
    bool ok = false;
#define GLA_RUN(T, TS, V, S, N)                                                                                            \
    {                                                                                                                      \
        constexpr auto kKernel = fwd_kernel<T, TS, V, S, N>;                                                               \
        ok = allow_most<kKernel>();                                                                                        \
        if (ok) kKernel<<<grid, pl.threads, bytes, st>>>(in, w, kind, post, act, eps, (TS *)r, (T *)out, rows, D, pl.lanes); \
    }
    GLA_BY_TYPE(GLA_RUN)
#undef GLA_RUN
    count_launches(1);
    return ok && cudaGetLastError() == cudaSuccess ? GLA_OK : GLA_ERR_LAUNCH;
}

int bwd(const void *dr, const void *dout, const void *r, const void *y, const void *gate, const float *scale,
        const float *post_weight, const float *post_bias, const float *weight, int kind, int post, int act, float eps, void *dx,
        void *dy, void *dgate, float *dscale, float *dpost_weight, float *dpost_bias, float *dweight, float *dbias, int64_t rows,
        int D, int dtype, int stream_dtype, void *ws, cudaStream_t st) {
    constexpr int kVecs = kBwdVecs, kSmall = 320;
    const Plan pl = make_plan(D, kVecs);
    const Weights w{scale, post_weight, post_bias, weight, nullptr};
    const int n = per_sm(pl, kBwdThreads), nb = rows > 0 ? blocks(pl, rows, n) : 0;
    bool ok = true;
    if (nb > 0) {
        const int e = dtype == GLA_F32 ? 4 : 2, es = stream_dtype == GLA_F32 ? 4 : 2;
        Inputs<5> in{{dr, dout, dout != nullptr ? r : nullptr, y, gate}, {D * es, D * e, D * es, D * e, D * e}, {}, 0, 0};
        const int bytes = lay_out(in, pl, n);
        const bool staged = in.stages > 0;
#define GLA_RUN(T, TS, V, S, N)                                                                                            \
        {                                                                                                                  \
            constexpr auto kKernel = bwd_kernel<T, TS, V, S, N>;                                                           \
            ok = allow_most<kKernel>();                                                                                    \
            if (ok)                                                                                                        \
                kKernel<<<(unsigned)nb, pl.threads, bytes, st>>>(in, w, kind, post, act, eps, (TS *)dx, (T *)dy,           \
                                                                 (T *)dgate, (float *)ws, rows, D, pl.lanes);              \
        }
        GLA_BY_TYPE(GLA_RUN)
#undef GLA_RUN
        count_launches(1);
    }
    if (dscale || dpost_weight || dpost_bias || dweight || dbias) {
        const Sums sums{{dscale, dpost_weight, dpost_bias, dweight, dbias}};
        sum_kernel<<<dim3((unsigned)((D + 31) / 32), kSums), 256, 0, st>>>((const float *)ws, nb, D, sums);
        count_launches(1);
    }
    return ok && cudaGetLastError() == cudaSuccess ? GLA_OK : GLA_ERR_LAUNCH;
}

}  // namespace resnorm
}  // namespace gla
