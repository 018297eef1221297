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
// its last row.  An SM has several blocks, so that one row's barriers wait beside another's work.  Rows come into shared memory
// by bulk copies, some rows ahead, and are read from there by each step: what is in flight costs no registers.  Rows that two
// stages have no room for are read from memory.  Statistics are taken in two steps, a mean and then centred squares.
#include <type_traits>

#include "gla_act.cuh"
#include "sm100_ptx.cuh"

GLA_DEFINE_STATUS(resnorm)

namespace gla {
namespace resnorm {
namespace {

// Sums over tokens, with f = act(gate): of dx f n(y) and dx f, of dout h and dout.  They give dpost_weight and dpost_bias by the
// factor scale, dscale = post_weight (the first) + post_bias (the second), dweight and dbias.  (Without the norm of y the
// first is of dx f y, and dscale itself.)
constexpr int kSums = 4;
constexpr int kMaxStages = 6;
constexpr int kThreads = 256;  // of a block with several rows
constexpr uint64_t kWaitNs = 2000000000ull;

// Threads to a row (whole warps above 32), rows of a block at a time.  A thread's vectors are kStride channels apart, so that
// those of a warp are neighbours and a vector's place is a constant away from the thread's first.
struct Plan {
    int lanes, vecs, rows, threads;
};
constexpr int kStride = 128;
constexpr int kFwdVecs = 4, kBwdVecs = 2, kWideVecs = 4;

Plan make_plan(int D, int vecs) {
    Plan p{};
    p.vecs = D <= kStride ? 1 : D <= 2 * kStride ? 2 : D <= 1024 * 4 * vecs ? vecs : kWideVecs;
    p.lanes = 1;
    if (D <= kStride)
        while (p.lanes < D / 4) p.lanes *= 2;
    else
        p.lanes = (D + kStride * p.vecs - 1) / (kStride * p.vecs) * 32;
    p.rows = p.lanes <= 32 ? kThreads / p.lanes : 1;
    p.threads = p.lanes * p.rows;
    return p;
}

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

// A thread's vectors: fetch reads them (zero where there are none), times and plus take parameters that may be absent, for all
// of them or none.  kAll: every thread has all of its vectors.
template <int kVec, bool kAll> struct Vectors {
    using V = Pair[kVec][2];
    int count;
    __device__ __forceinline__ bool has(int j) const { return kAll || j < count; }
    template <typename T> __device__ __forceinline__ void fetch(V &v, const T *p) const {
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            if (!kAll) v[j][0] = v[j][1] = both(0.f);
            if (has(j)) Four<T>::open(v[j], *reinterpret_cast<const typename Four<T>::Raw *>(p + j * kStride));
        }
    }
    template <typename T> __device__ __forceinline__ void store(T *p, const V &v) const {
#pragma unroll
        for (int j = 0; j < kVec; ++j)
            if (has(j)) put<T>(p + j * kStride, v[j]);
    }
    template <class F> __device__ __forceinline__ void with(const float *p, F f) const {  // f(j, parameters), where there are any
        if (p == nullptr) return;
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            Pair a[2] = {both(0.f), both(0.f)};
            if (has(j)) Four<float>::open(a, *reinterpret_cast<const float4 *>(p + j * kStride));
            f(j, a);
        }
    }
    __device__ __forceinline__ void times(V &v, const float *p) const {
        with(p, [&](int j, const Pair (&a)[2]) { v[j][0] = v[j][0] * a[0], v[j][1] = v[j][1] * a[1]; });
    }
    __device__ __forceinline__ void plus(V &v, const float *p) const {
        with(p, [&](int j, const Pair (&a)[2]) { v[j][0] = v[j][0] + a[0], v[j][1] = v[j][1] + a[1]; });
    }
    __device__ __forceinline__ void times(V &v, float by) const {
#pragma unroll
        for (int j = 0; j < kVec; ++j) v[j][0] = v[j][0] * both(by), v[j][1] = v[j][1] * both(by);
    }
    __device__ __forceinline__ void shift(V &v, float by) const {  // those that there are
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            const Pair b = both(has(j) ? by : 0.f);
            v[j][0] = v[j][0] + b, v[j][1] = v[j][1] + b;
        }
    }
    __device__ __forceinline__ void clear(V &v) const {  // those that there are not
        if (kAll) return;
#pragma unroll
        for (int j = 0; j < kVec; ++j)
            if (!has(j)) v[j][0] = v[j][1] = both(0.f);
    }
    static __device__ __forceinline__ float sum(const V &v) {
        Pair s = v[0][0] + v[0][1];
#pragma unroll
        for (int j = 1; j < kVec; ++j) s = s + (v[j][0] + v[j][1]);
        return total(s);
    }
    static __device__ __forceinline__ float squares(const V &v) {
        Pair s = v[0][0] * v[0][0];
        s = fma(v[0][1], v[0][1], s);
#pragma unroll
        for (int j = 1; j < kVec; ++j) s = fma(v[j][0], v[j][0], fma(v[j][1], v[j][1], s));
        return total(s);
    }
    static __device__ __forceinline__ float product(const V &v, const V &u) {
        Pair s = v[0][0] * u[0][0];
        s = fma(v[0][1], u[0][1], s);
#pragma unroll
        for (int j = 1; j < kVec; ++j) s = fma(v[j][0], u[j][0], fma(v[j][1], u[j][1], s));
        return total(s);
    }
    // g becomes act(g), and slope act's slope: one choice for all vectors
    template <int kAct> static __device__ __forceinline__ void gate(V &g) {
#pragma unroll
        for (int j = 0; j < kVec; ++j) g[j][0] = activation(g[j][0], kAct), g[j][1] = activation(g[j][1], kAct);
    }
    template <int kAct> static __device__ __forceinline__ void gate(V &g, V &slope) {
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            g[j][0] = activation(g[j][0], kAct, slope[j][0]);
            g[j][1] = activation(g[j][1], kAct, slope[j][1]);
        }
    }
};

// Minus a value near a row's mean (is there a row): the mean of its first 8 channels in bf16, which every thread reads, of its
// first 128 (all, where there are no more) in f32.  Sums of v + near and of its square then give the row's variance with a
// loss of (their mean)^2 over the variance, which is below D / 8 or D / 128: at worst those channels alone are off from all
// others.  That leaves 2^-13 and 2^-17 of the variance at 16,384 channels, and 2^-24 times a small number for common rows.
template <typename E> __device__ __forceinline__ float near_mean(const E *row, int D, int lanes, bool is) {
    if (sizeof(E) == 2) {
        if (!is) return 0.f;
        const uint4 w = *reinterpret_cast<const uint4 *>(row);
        Pair v[2], u[2];
        Four<__nv_bfloat16>::open(v, make_uint2(w.x, w.y));
        Four<__nv_bfloat16>::open(u, make_uint2(w.z, w.w));
        return total((v[0] + v[1]) + (u[0] + u[1])) * -0.125f;
    }
    const int n = min(D, kStride), c = (threadIdx.x % lanes & 31) * 4;
    float s = 0.f;
    if (is && c < n) {
        const float4 w = *reinterpret_cast<const float4 *>(row + c);
        s = (w.x + w.y) + (w.z + w.w);
    }
    for (int d = min(lanes, 32) >> 1; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    return s * (-1.f / (float)n);
}

// Two sums over a row's threads at once.  The warps of a row meet in shared memory, in one half of it after the other, so that
// one barrier a sum is enough; every thread of the block calls this.
struct Meeting {
    float at[2][2][32];  // the first sum's parts by warp, and the second's
};
__device__ __forceinline__ float2 row_sum(float a, float b, int lanes, Meeting &m, int &half) {
    if (lanes < 32) {
        for (int d = lanes >> 1; d > 0; d >>= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, d);
            b += __shfl_xor_sync(0xffffffffu, b, d);
        }
        return make_float2(a, b);
    }
    // one half of the warp adds the one sum up, the other half the other; then the warps' parts likewise
    const int lane = threadIdx.x & 31, upper = lane >> 4;
    float v = (upper ? b : a) + __shfl_xor_sync(0xffffffffu, upper ? a : b, 16);
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    if (lanes > 32) {
        float(&at)[2][32] = m.at[half];
        if ((lane & 15) == 0) at[upper][threadIdx.x >> 5] = v;
        __syncthreads();
        v = at[upper][lane & 15];
        if (lanes > 512) v += at[upper][16 + (lane & 15)];
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
        half ^= 1;
    }
    const float o = __shfl_xor_sync(0xffffffffu, v, 16);
    return upper ? make_float2(o, v) : make_float2(v, o);
}

// Six sums at once, each thread's parts given and the row's sums returned in v: three halvings leave a lane with one of them.
// kMost: the block's threads at most.
struct SixMeeting {
    float at[2][32][8];  // by warp
};
template <int kMost> __device__ __forceinline__ void row_sums(float (&v)[6], int lanes, SixMeeting &m, int &half) {
    if (lanes < 32) {
        for (int d = lanes >> 1; d > 0; d >>= 1)
#pragma unroll
            for (int i = 0; i < 6; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], d);
        return;
    }
    const int lane = threadIdx.x & 31;
    const bool b16 = (lane & 16) != 0, b8 = (lane & 8) != 0, b4 = (lane & 4) != 0;
    float w[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) w[i] = (b16 ? v[i + 3] : v[i]) + __shfl_xor_sync(0xffffffffu, b16 ? v[i] : v[i + 3], 16);
    float x = (b8 ? w[1] : w[0]) + __shfl_xor_sync(0xffffffffu, b8 ? w[0] : w[1], 8);
    const float y = w[2] + __shfl_xor_sync(0xffffffffu, w[2], 8);
    x = (b4 ? y : x) + __shfl_xor_sync(0xffffffffu, b4 ? x : y, 4);
    x += __shfl_xor_sync(0xffffffffu, x, 2);
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    // the sum that a lane has: 3 (bit 4 of it) + 2 where bit 2 is set, else bit 3
    if (lanes == 32) {
#pragma unroll
        for (int i = 0; i < 6; ++i) v[i] = __shfl_sync(0xffffffffu, x, i / 3 * 16 + (i % 3 == 2 ? 4 : i % 3 * 8));
        return;
    }
    float(&at)[32][8] = m.at[half];
    if ((lane & 3) == 0 && !(b4 && b8)) at[threadIdx.x >> 5][(b16 ? 3 : 0) + (b4 ? 2 : b8 ? 1 : 0)] = x;
    __syncthreads();
    x = at[lane >> 3][lane & 7];
#pragma unroll
    for (int i = 1; i < (kMost / 32 + 3) / 4; ++i) x += at[(lane >> 3) + 4 * i][lane & 7];
    x += __shfl_xor_sync(0xffffffffu, x, 16);
    x += __shfl_xor_sync(0xffffffffu, x, 8);
#pragma unroll
    for (int i = 0; i < 6; ++i) v[i] = __shfl_sync(0xffffffffu, x, i);
    half ^= 1;
}
template <class M> __device__ __forceinline__ void clear(M &m) {  // warps that there are not add nothing
    for (int i = threadIdx.x; i < (int)(sizeof(M) / sizeof(float)); i += blockDim.x) reinterpret_cast<float *>(&m)[i] = 0.f;
}

// Arrays whose rows come in, and the stages that they come into: the rows of an item, of each array.
template <int kArrays> struct Inputs {
    const void *from[kArrays];  // null: absent
    int row_bytes[kArrays], at[kArrays];
    int stage_bytes, stages, passes;
};

// The rows of a block, an item (`passes` rows for each of its threads) after the other.
struct Bars {
    uint64_t full[kMaxStages], read[kMaxStages];
    int failed;
};
template <bool kStage, int kArrays>
struct Rows {
    const Inputs<kArrays> &in;
    uint8_t *ring;
    Bars &bars;
    int64_t rows, row;               // row: the thread's
    int item, items, at_once, step, mine, st;  // rows at once and of an item; the thread's row in its item
    uint32_t phase;
    bool late;  // whether the stage of the item before is still to be refilled
    __device__ __forceinline__ Rows(const Inputs<kArrays> &in_, uint8_t *ring_, Bars &bars_, int64_t rows_, int lanes)
        : in(in_), ring(ring_), bars(bars_), rows(rows_), item(blockIdx.x), at_once(blockDim.x / lanes), st(0), phase(0), late(false) {
        step = at_once * in.passes;
        mine = threadIdx.x / lanes;
        items = (int)((rows + step - 1) / step);
        row = (int64_t)item * step + mine;
        if (!kStage) return;
        if (threadIdx.x == 0) {
            bars.failed = 0;
            for (int i = 0; i < in.stages; ++i) {
                ptx::mbar_init(ptx::smem_u32(bars.full + i), 1);
                ptx::mbar_init(ptx::smem_u32(bars.read + i), (blockDim.x + 31) / 32);
            }
            ptx::fence_mbar_init();
            for (int i = 0; i < in.stages; ++i) order(i, item + i * (int)gridDim.x);
        }
    }
    // by one thread
    __device__ __forceinline__ void order(int to_stage, int k) const {
        if (k >= items) return;
        const uint32_t b = ptx::smem_u32(bars.full + to_stage), to = ptx::smem_u32(ring) + (uint32_t)(to_stage * in.stage_bytes);
        const int64_t first = (int64_t)k * step;
        const int n = (int)min((int64_t)step, rows - first);
        uint32_t bytes = 0;
#pragma unroll
        for (int i = 0; i < kArrays; ++i)
            if (in.from[i] != nullptr) bytes += (uint32_t)(n * in.row_bytes[i]);
        ptx::mbar_expect_tx(b, bytes);
#pragma unroll
        for (int i = 0; i < kArrays; ++i)
            if (in.from[i] != nullptr)
                ptx::bulk_load_g2s(to + (uint32_t)in.at[i], (const uint8_t *)in.from[i] + first * in.row_bytes[i],
                                   (uint32_t)(n * in.row_bytes[i]), b);
    }
    __device__ __forceinline__ void wait(uint64_t *bar, uint32_t parity) const {
        if (!ptx::mbar_wait(ptx::smem_u32(bar), parity, &bars.failed, kWaitNs)) *(volatile int *)&bars.failed = 1;
    }
    // The thread's next row; false when the block has no more.  meets: a barrier of the row's sums is followed by refill().
    __device__ __forceinline__ bool begin(bool meets) {
        if (item >= items) return false;
        if (kStage && mine < at_once) {
            if (!meets) {
                if (threadIdx.x == 0 && late) wait(bars.read + (st == 0 ? in.stages - 1 : st - 1), st == 0 ? phase ^ 1u : phase);
                refill();
            }
            wait(bars.full + st, phase);
        }
        return true;
    }
    // All threads are past the item before: its stage takes another one.
    __device__ __forceinline__ void refill() {
        if (kStage && late && threadIdx.x == 0) order(st == 0 ? in.stages - 1 : st - 1, item + (in.stages - 1) * (int)gridDim.x);
        late = false;
        __syncwarp();
    }
    __device__ __forceinline__ void next() {
        mine += at_once;
        row += at_once;
        if (mine < step) return;
        mine -= step;
        row += ((int64_t)gridDim.x - 1) * step;
        if (kStage) {
            __syncwarp();
            if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(ptx::smem_u32(bars.read + st));
            late = true;
            if (++st == in.stages) {
                st = 0;
                phase ^= 1u;
            }
        }
        item += gridDim.x;
    }
    // what a block that gave up has ordered still comes in
    __device__ __forceinline__ void end() const {
        if (kStage && threadIdx.x == 0 && *(volatile int *)&bars.failed) {
            record_status(GLA_ERR_TIMEOUT);
            for (int i = 0; i < in.stages; ++i) ptx::mbar_wait(ptx::smem_u32(bars.full + i), phase ^ (uint32_t)(i < st), nullptr, kWaitNs);
        }
    }
    // a channel of the thread's row of array i, staged or in memory
    template <typename T> __device__ __forceinline__ const T *at(int i, int D, int channel) const {
        if (kStage) return reinterpret_cast<const T *>(ring + st * in.stage_bytes + in.at[i]) + mine * D + channel;
        return (const T *)in.from[i] + row * D + channel;
    }
};

// A thread's place: its first channel and how many of its vectors exist.
template <int kVec> struct Place {
    int channel, count;
    __device__ __forceinline__ Place(int D, int lanes) {
        const int lane = threadIdx.x % lanes;
        channel = lanes < 32 ? lane * 4 : (lane >> 5) * (kStride * kVec) + (lane & 31) * 4;
        count = channel >= D ? 0 : lanes < 32 ? 1 : min(kVec, (D - channel + kStride - 1) / kStride);
    }
};

struct Weights {
    const float *scale, *post_weight, *post_bias, *weight, *bias;
    __device__ __forceinline__ Weights from(int channel) const {
        auto at = [&](const float *p) { return p == nullptr ? nullptr : p + channel; };
        return {at(scale), at(post_weight), at(post_bias), at(weight), at(bias)};
    }
    // those that there are, in shared memory, by the whole block
    __device__ __forceinline__ Weights shared(float *to, int D) const {
        auto copy = [&](const float *p) -> const float * {
            if (p == nullptr) return nullptr;
            for (int i = threadIdx.x; i < D / 4; i += blockDim.x)
                reinterpret_cast<float4 *>(to)[i] = __ldg(reinterpret_cast<const float4 *>(p) + i);
            const float *const there = to;
            to += D;
            return there;
        };
        const float *const a = copy(scale), *const b = copy(post_weight), *const c = copy(post_bias), *const d = copy(weight);
        return {a, b, c, d, copy(bias)};
    }
};

template <typename T, typename TS, int kVec, bool kStage, int kMost>
__global__ void __launch_bounds__(kMost, kMost <= 256 ? 3 : 1)
fwd_kernel(const Inputs<3> in, Weights weights, int kind, int post, int act, float eps, TS *__restrict__ r, T *__restrict__ out,
           int64_t rows, int D, int lanes, int params_at) {
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ Bars bars;
    __shared__ __align__(16) Meeting meet;
    const Place<kVec> pl(D, lanes);
    const float inv = 1.f / (float)D;
    const bool has_y = in.from[1] != nullptr, has_gate = in.from[2] != nullptr, meets = lanes > 32 && (post || out != nullptr);
    Rows<kStage, 3> it(in, ring, bars, rows, lanes);
    clear(meet);
    const Weights w = (params_at >= 0 ? weights.shared(reinterpret_cast<float *>(ring + params_at), D) : weights).from(pl.channel);
    __syncthreads();
    int half = 0;
    auto row = [&](auto all) {
        using Vs = Vectors<kVec, all.value>;
        const Vs vs{it.row < rows ? pl.count : 0};
        const int64_t at = it.row * D + pl.channel;
        typename Vs::V v;
        // v becomes n(v)
        auto normalise = [&](typename Vs::V &x) {
            if (kind == GLA_NORM_LAYER) vs.shift(x, -row_sum(Vs::sum(x), 0.f, lanes, meet, half).x * inv);
            vs.times(x, rsqrtf(fmaf(row_sum(Vs::squares(x), 0.f, lanes, meet, half).x, inv, eps)));
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

// kMode: which parts there are, for the kernels built for one kind of call whose rows leave no thread without work; kAnyMode: all
// of that is asked for at run time.  (Of 16,384 x 2,560 with all parts the latter takes a quarter more time.)
// kParams: the parameters are in shared memory, all that the parts could ask for (ones and zeros for those that there are not).
enum Mode { kOut = 1, kY = 2, kPost = 4, kGated = 8, kGatedSigmoid = 16, kAnyMode = 32, kParams = 64 };
enum Param { kWeight, kScale, kPostWeight, kPostBias };
constexpr __host__ __device__ int params_of(int mode) { return mode & kPost ? 4 : mode & kY ? 2 : 1; }
template <typename T, typename TS, int kVec, bool kStage, int kMost, int kMode>
__global__ void __launch_bounds__(kMost, kMost <= 320 ? 2 : 1)
bwd_kernel(const Inputs<5> in, Weights weights, int kind, int post_, int act, float eps, TS *__restrict__ dx, T *__restrict__ dy,
           T *__restrict__ dgate, float *__restrict__ part, int64_t rows, int D, int lanes, int params_at) {
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ Bars bars;
    __shared__ __align__(16) Meeting meet;
    __shared__ __align__(16) SixMeeting six;
    const Place<kVec> pl(D, lanes);
    const float inv = 1.f / (float)D;
    constexpr bool kAny = (kMode & kAnyMode) != 0;
    const bool has_dr = in.from[0] != nullptr, layer = kind == GLA_NORM_LAYER;
    const bool has_out = kAny ? in.from[1] != nullptr : (kMode & kOut) != 0, has_y = kAny ? in.from[3] != nullptr : (kMode & kY) != 0,
               has_gate = kAny ? in.from[4] != nullptr : (kMode & (kGated | kGatedSigmoid)) != 0, post = kAny ? post_ != 0 : (kMode & kPost) != 0;
    const bool meets = lanes > 32 && (post || has_out);
    Pair sums[kSums][kVec][2];
#pragma unroll
    for (int i = 0; i < kSums; ++i)
#pragma unroll
        for (int j = 0; j < kVec; ++j) sums[i][j][0] = sums[i][j][1] = both(0.f);
    Rows<kStage, 5> it(in, ring, bars, rows, lanes);
    clear(meet);
    clear(six);
    constexpr bool kShared = (kMode & kParams) != 0;
    if (kShared)
        for (int i = 0; i < params_of(kMode); ++i) {
            const float *const from = i == kWeight ? weights.weight : i == kScale ? weights.scale : i == kPostWeight ? weights.post_weight : weights.post_bias;
            const float fill = i == kPostBias ? 0.f : 1.f;
            float4 *const to = reinterpret_cast<float4 *>(ring + params_at) + i * (D / 4);
            for (int c = threadIdx.x; c < D / 4; c += blockDim.x)
                to[c] = from ? __ldg(reinterpret_cast<const float4 *>(from) + c) : make_float4(fill, fill, fill, fill);
        }
    const Weights w = kShared ? weights : (params_at >= 0 ? weights.shared(reinterpret_cast<float *>(ring + params_at), D) : weights).from(pl.channel);
    const float *const params = reinterpret_cast<const float *>(ring + params_at) + pl.channel;
    __syncthreads();
    int half = 0;
    auto row = [&](auto all) {
        using Vs = Vectors<kVec, all.value>;
        const bool there = all.value || it.row < rows;
        const Vs vs{there ? pl.count : 0};
        const int64_t at = it.row * D + pl.channel;
        const TS *const from_r = it.template at<TS>(2, D, pl.channel);
        const T *const from_out = it.template at<T>(1, D, pl.channel), *const from_y = it.template at<T>(3, D, pl.channel);
        // one vector of an array, or of parameters
        auto vec = [&](Pair (&v)[2], const auto *p, int j) {
            using E = std::remove_cv_t<std::remove_reference_t<decltype(*p)>>;
            if (!all.value) v[0] = v[1] = both(0.f);
            if (vs.has(j)) Four<E>::open(v, *reinterpret_cast<const typename Four<E>::Raw *>(p + j * kStride));
        };
        // vector j of a parameter; v as it is where there is none
        auto param = [&](Pair (&v)[2], Param which, int j) {
            const float *const p = which == kWeight ? w.weight : which == kScale ? w.scale : which == kPostWeight ? w.post_weight : w.post_bias;
            if (kShared) vec(v, params + which * D, j);
            else if (p != nullptr) vec(v, p, j);
        };
        // n(r) = r' q + qm and n(y) = y' uq + uqm, of r' = r + near_r and y' = y + near_y
        typename Vs::V rc, yc;
        Pair q = both(1.f), qm = both(0.f), uq = both(1.f), uqm = both(0.f), m1 = both(0.f), m2 = both(0.f);
        float near_r = 0.f, near_y = 0.f;
        if (has_out || post) {
            if (layer) {
                if (has_out) near_r = near_mean(it.template at<TS>(2, D, 0), D, lanes, there);
                if (post) near_y = near_mean(it.template at<T>(3, D, 0), D, lanes, there);
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
            row_sums<kMost>(o, lanes, six, half);
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
            const float2 o = row_sum(layer ? total(s) : 0.f, total(t), lanes, meet, half);
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
    for (; it.begin(meets); it.next()) row(std::integral_constant<bool, !kAny>{});
    it.end();
    // the block's rows of one channel set meet in shared memory; one writer per channel
    float *to = part + (int64_t)blockIdx.x * kSums * D;
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
                *reinterpret_cast<float4 *>(to + (int64_t)i * D + pl.channel + j * kStride) = v;
        }
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

// Blocks of an SM: as many as the threads' registers allow, 85 a thread of the forward and 102 of the gradient.
constexpr int kFwdThreads = 768, kBwdThreads = 640;
int per_sm(const Plan &pl, int threads) { return threads < pl.threads ? 1 : threads / pl.threads; }
int blocks(const Plan &pl, int64_t rows, int per_sm) {
    const int64_t need = (rows + pl.rows - 1) / pl.rows;
    int64_t most = (int64_t)device_info().sm_count * per_sm;
    if (most < 1) most = 1;
    return (int)(need < most ? need : most);
}

constexpr int kMostShared = 218 * 1024;

// The stages of a block: an item's rows of each array one behind the other; behind them the parameters, `params` bytes, where
// there is room (else params_at is negative: they are read from memory, and what shared memory leaves caches them).  Short rows
// are taken some at a time, while there are enough for all blocks: an item's copies then serve several rows of a thread.
template <int kArrays> int lay_out(Inputs<kArrays> &in, const Plan &pl, int64_t rows, int per_sm, int nblocks, int params, int &params_at) {
    int row = 0, at = 0;
    for (int i = 0; i < kArrays; ++i)
        if (in.from[i] != nullptr) row += in.row_bytes[i];
    in.passes = 1;
    while (in.passes < 8 && 2 * in.passes * pl.rows * row <= 16 * 1024 && rows >= 4LL * in.passes * pl.rows * nblocks) in.passes *= 2;
    for (int i = 0; i < kArrays; ++i) {
        in.at[i] = at;
        if (in.from[i] != nullptr) at += (in.passes * pl.rows * in.row_bytes[i] + 127) / 128 * 128;
    }
    in.stage_bytes = at;
    const int room = kMostShared / per_sm - (per_sm > 1 ? 3328 : 0);
    const bool shared = params > 0 && 2 * at + params <= room;
    in.stages = shared ? (room - params) / at : (room - (per_sm > 1 ? 28 * 1024 / per_sm : 0)) / at;
    if (in.stages < 2 && 2 * at <= room) in.stages = 2;
    if (in.stages > kMaxStages) in.stages = kMaxStages;
    if (in.stages < 2) in.stages = 0;
    int bytes = in.stages * at;
    if (bytes < 16 * pl.threads) bytes = 16 * pl.threads;
    params_at = in.stages > 0 && shared ? bytes : -1;
    return bytes + (params_at >= 0 ? params : 0);
}

// RUN(T, TS, kVec, kStage, kMost) for a call's types and plan.
#define GLA_BY_STAGE(RUN, T, TS, V, N)                 \
    if (staged) { RUN(T, TS, V, true, N) }             \
    else { RUN(T, TS, V, false, N) }
#define GLA_BY_PLAN(RUN, T, TS)                                                                     \
    if (pl.threads <= kSmall && pl.vecs == 1) { GLA_BY_STAGE(RUN, T, TS, 1, kSmall) }               \
    else if (pl.threads <= kSmall && pl.vecs == 2) { GLA_BY_STAGE(RUN, T, TS, 2, kSmall) }          \
    else if (pl.threads <= kSmall && pl.vecs == kVecs) { GLA_BY_STAGE(RUN, T, TS, kVecs, kSmall) }  \
    else if (pl.threads <= 512 && pl.vecs == kVecs) { GLA_BY_STAGE(RUN, T, TS, kVecs, 512) }        \
    else if (pl.vecs == kVecs) { GLA_BY_STAGE(RUN, T, TS, kVecs, 1024) }                            \
    else { GLA_BY_STAGE(RUN, T, TS, kWideVecs, 1024) }
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
    const int e = dtype == GLA_F32 ? 4 : 2, es = stream_dtype == GLA_F32 ? 4 : 2;
    Inputs<3> in{{x, y, gate}, {D * es, D * e, D * e}, {}, 0, 0, 1};
    const int n = per_sm(pl, kFwdThreads);
    const unsigned grid = (unsigned)blocks(pl, rows, n);
    int params_at;
    const int bytes = lay_out(in, pl, rows, n, (int)grid, 0, params_at);
    const bool staged = in.stages > 0;
    bool ok = false;
#define GLA_RUN(T, TS, V, S, N)                                                                                            \
    {                                                                                                                      \
        constexpr auto kKernel = fwd_kernel<T, TS, V, S, N>;                                                               \
        ok = allow_most<kKernel>();                                                                                        \
        if (ok) kKernel<<<grid, pl.threads, bytes, st>>>(in, w, kind, post, act, eps, (TS *)r, (T *)out, rows, D, pl.lanes, params_at); \
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
        Inputs<5> in{{dr, dout, dout != nullptr ? r : nullptr, y, gate}, {D * es, D * e, D * es, D * e, D * e}, {}, 0, 0, 1};
        int params_at;
        int arrays = (scale != nullptr) + (post_weight != nullptr) + (post_bias != nullptr) + (weight != nullptr);
        const int mode = (dout != nullptr ? kOut : 0) + (y != nullptr ? kY : 0) + (post ? kPost : 0) +
                         (gate == nullptr ? 0 : act == kSilu ? kGated : act == kSigmoid ? kGatedSigmoid : kAnyMode);
        const bool even = pl.vecs == kVecs && pl.threads <= kSmall && D % (kStride * kVecs) == 0;
        if (even && arrays < params_of(mode)) arrays = params_of(mode);
        const int bytes = lay_out(in, pl, rows, n, nb, arrays * D * 4, params_at);
        const bool staged = in.stages > 0;
        const bool whole = staged && even && rows % ((int64_t)pl.rows * in.passes) == 0;
#define GLA_MODE(T, TS, V, S, N, M)                                                                                        \
        {                                                                                                                  \
            constexpr auto kKernel = bwd_kernel<T, TS, V, S, N, M>;                                                        \
            ok = allow_most<kKernel>();                                                                                    \
            if (ok)                                                                                                        \
                kKernel<<<(unsigned)nb, pl.threads, bytes, st>>>(in, w, kind, post, act, eps, (TS *)dx, (T *)dy,           \
                                                                 (T *)dgate, (float *)ws, rows, D, pl.lanes, params_at);   \
        }
#define GLA_RUN(T, TS, V, S, N) GLA_MODE(T, TS, V, S, N, kAnyMode)
#define GLA_WHOLE_MODE(T, TS, M)                                                                                           \
        if (mode == (M)) {                                                                                                 \
            found = true;                                                                                                  \
            if (params_at >= 0) GLA_MODE(T, TS, kVecs, true, kSmall, (M) + kParams)                                        \
            else GLA_MODE(T, TS, kVecs, true, kSmall, M)                                                                   \
        }
#define GLA_WHOLE(T, TS)                                                                                                   \
        GLA_WHOLE_MODE(T, TS, kOut + kY + kPost + kGated)                                                                  \
        GLA_WHOLE_MODE(T, TS, kOut + kY + kPost + kGatedSigmoid)                                                           \
        GLA_WHOLE_MODE(T, TS, kOut + kY + kPost)                                                                           \
        GLA_WHOLE_MODE(T, TS, kOut + kY + kGated)                                                                          \
        GLA_WHOLE_MODE(T, TS, kOut + kY + kGatedSigmoid)                                                                   \
        GLA_WHOLE_MODE(T, TS, kOut + kY)
        bool found = false;
        if (whole) {
            if (dtype == GLA_F32) { GLA_WHOLE(float, float) }
            else if (stream_dtype == GLA_F32) { GLA_WHOLE(__nv_bfloat16, float) }
            else { GLA_WHOLE(__nv_bfloat16, __nv_bfloat16) }
        }
        if (!found) { GLA_BY_TYPE(GLA_RUN) }
#undef GLA_WHOLE
#undef GLA_WHOLE_MODE
#undef GLA_MODE
#undef GLA_RUN
        count_launches(1);
    }
    if (dscale || dpost_weight || dpost_bias || dweight || dbias) {
        const Sums sums{dscale, dpost_weight, dpost_bias, dweight, dbias};
        sum_kernel<<<dim3((unsigned)((D + 31) / 32), kSums / 2), 256, 0, st>>>((const float *)ws, nb, D, post != 0, w, sums);
        count_launches(1);
    }
    return ok && cudaGetLastError() == cudaSuccess ? GLA_OK : GLA_ERR_LAUNCH;
}

}  // namespace resnorm
}  // namespace gla
