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

constexpr int kSums = 5;  // dscale, dpost_weight, dpost_bias, dweight, dbias
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
__device__ __forceinline__ void clear(Meeting &m) {  // warps that there are not add nothing
    for (int i = threadIdx.x; i < 128; i += blockDim.x) (&m.at[0][0][0])[i] = 0.f;
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
enum Mode { kOut = 1, kY = 2, kPost = 4, kGated = 8, kGatedSigmoid = 16, kAnyMode = 32 };
template <typename T, typename TS, int kVec, bool kStage, int kMost, int kMode>
__global__ void __launch_bounds__(kMost, kMost <= 320 ? 2 : 1)
bwd_kernel(const Inputs<5> in, Weights weights, int kind, int post_, int act, float eps, TS *__restrict__ dx, T *__restrict__ dy,
           T *__restrict__ dgate, float *__restrict__ part, int64_t rows, int D, int lanes, int params_at) {
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ Bars bars;
    __shared__ __align__(16) Meeting meet;
    const Place<kVec> pl(D, lanes);
    const float inv = 1.f / (float)D;
    constexpr bool kAny = kMode == kAnyMode;
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
    const Weights w = (params_at >= 0 ? weights.shared(reinterpret_cast<float *>(ring + params_at), D) : weights).from(pl.channel);
    __syncthreads();
    int half = 0;
    // every step reads what it needs again: registers are what the sums leave
    auto row = [&](auto all) {
        using Vs = Vectors<kVec, all.value>;
        const Vs vs{it.row < rows ? pl.count : 0};
        const int64_t at = it.row * D + pl.channel;
        const TS *const from_r = it.template at<TS>(2, D, pl.channel);
        const T *const from_out = it.template at<T>(1, D, pl.channel), *const from_y = it.template at<T>(3, D, pl.channel);
        // one vector of an array, or of parameters
        auto vec = [&](Pair (&v)[2], const auto *p, int j) {
            using E = std::remove_cv_t<std::remove_reference_t<decltype(*p)>>;
            if (!all.value) v[0] = v[1] = both(0.f);
            if (vs.has(j)) Four<E>::open(v, *reinterpret_cast<const typename Four<E>::Raw *>(p + j * kStride));
        };
        Pair q = both(1.f), qm = both(0.f), uq = both(1.f), uqm = both(0.f);  // n(v) is (v + qm) q
        if (has_out || post) {
            float mr = 0.f, mu = 0.f;
            Pair s = both(0.f), t = both(0.f), v[2];
            if (layer) {
#pragma unroll
                for (int j = 0; j < kVec; ++j) {
                    if (has_out) vec(v, from_r, j), s = s + (v[0] + v[1]);
                    if (post) vec(v, from_y, j), t = t + (v[0] + v[1]);
                }
                const float2 o = row_sum(total(s), total(t), lanes, meet, half);
                mr = -o.x * inv, mu = -o.y * inv;
                s = t = both(0.f);
            }
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                if (has_out) {
                    vec(v, from_r, j);
                    const Pair by = both(vs.has(j) ? mr : 0.f);
                    v[0] = v[0] + by, v[1] = v[1] + by;
                    s = fma(v[0], v[0], fma(v[1], v[1], s));
                }
                if (post) {
                    vec(v, from_y, j);
                    const Pair by = both(vs.has(j) ? mu : 0.f);
                    v[0] = v[0] + by, v[1] = v[1] + by;
                    t = fma(v[0], v[0], fma(v[1], v[1], t));
                }
            }
            const float2 o = row_sum(total(s), total(t), lanes, meet, half);
            if (meets) it.refill();
            const float rr = rsqrtf(fmaf(o.x, inv, eps)), ru = rsqrtf(fmaf(o.y, inv, eps));
            q = both(rr), qm = both(mr);
            if (post) uq = both(ru), uqm = both(mu);
        }
        Pair m1 = both(0.f), m2 = both(0.f);
        if (has_out) {
            Pair s = both(0.f), t = both(0.f);
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                Pair up[2], h[2], wt[2] = {both(1.f), both(1.f)};
                vec(up, from_out, j);
                vec(h, from_r, j);
                if (w.weight != nullptr) vec(wt, w.weight, j);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    h[e] = (h[e] + qm) * q;
                    sums[3][j][e] = fma(up[e], h[e], sums[3][j][e]);
                    sums[4][j][e] = sums[4][j][e] + up[e];
                    up[e] = up[e] * wt[e];
                    s = s + up[e];
                    t = fma(up[e], h[e], t);
                }
            }
            const float2 o = row_sum(layer ? total(s) : 0.f, total(t), lanes, meet, half);
            m1 = both(-o.x * inv), m2 = both(-o.y * inv);
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
                    Pair up[2], h[2], wt[2] = {both(1.f), both(1.f)};
                    vec(up, from_out, j);
                    vec(h, from_r, j);
                    if (w.weight != nullptr) vec(wt, w.weight, j);
#pragma unroll
                    for (int e = 0; e < 2; ++e) d[j][e] = fma(fma((h[e] + qm) * q, m2, fma(up[e], wt[e], m1)), q, d[j][e]);
                    if (!vs.has(j)) d[j][0] = d[j][1] = both(0.f);
                }
                if (vs.has(j)) put<TS>(dx + at + j * kStride, d[j]);
                if (!has_y) continue;
                Pair u[2], z[2], p[2];
                vec(u, from_y, j);
                if (post) u[0] = (u[0] + uqm) * uq, u[1] = (u[1] + uqm) * uq;
                z[0] = u[0], z[1] = u[1];  // what the scale and the gate multiply
                if (w.post_weight != nullptr) {
                    vec(p, w.post_weight, j);
                    z[0] = z[0] * p[0], z[1] = z[1] * p[1];
                }
                if (w.post_bias != nullptr) {
                    vec(p, w.post_bias, j);
                    z[0] = z[0] + p[0], z[1] = z[1] + p[1];
                }
                Pair sc[2] = {both(1.f), both(1.f)};
                if (w.scale != nullptr) vec(sc, w.scale, j);
                if (kind_of_act.value >= 0) {
                    Pair g[2], slope;
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
                    sums[0][j][e] = fma(d[j][e], z[e], sums[0][j][e]);
                    d[j][e] = d[j][e] * sc[e];
                }
                if (!post) {
                    if (vs.has(j)) put<T>(dy + at + j * kStride, d[j]);
                    continue;
                }
                if (w.post_weight != nullptr) vec(p, w.post_weight, j);
                else p[0] = p[1] = both(1.f);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    sums[1][j][e] = fma(d[j][e], u[e], sums[1][j][e]);
                    sums[2][j][e] = sums[2][j][e] + d[j][e];
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
                Pair u[2];
                vec(u, from_y, j);
#pragma unroll
                for (int e = 0; e < 2; ++e) d[j][e] = fma((u[e] + uqm) * uq, m2, d[j][e] + m1) * uq;
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
    const int room = kMostShared / per_sm - (per_sm > 1 ? 2048 : 0);
    const bool shared = params > 0 && 2 * at + params <= room;
    in.stages = shared ? (room - params) / at : (room - (per_sm > 1 ? 28 * 1024 / per_sm : 0)) / at;
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
        const int arrays = (scale != nullptr) + (post_weight != nullptr) + (post_bias != nullptr) + (weight != nullptr);
        const int bytes = lay_out(in, pl, rows, n, nb, arrays * D * 4, params_at);
        const bool staged = in.stages > 0;
        const int mode = (dout != nullptr ? kOut : 0) + (y != nullptr ? kY : 0) + (post ? kPost : 0) +
                         (gate == nullptr ? 0 : act == kSilu ? kGated : act == kSigmoid ? kGatedSigmoid : kAnyMode);
        const bool whole = staged && pl.vecs == kVecs && pl.threads <= kSmall && D % (kStride * kVecs) == 0 &&
                           rows % ((int64_t)pl.rows * in.passes) == 0;
#define GLA_MODE(T, TS, V, S, N, M)                                                                                        \
        {                                                                                                                  \
            constexpr auto kKernel = bwd_kernel<T, TS, V, S, N, M>;                                                        \
            ok = allow_most<kKernel>();                                                                                    \
            if (ok)                                                                                                        \
                kKernel<<<(unsigned)nb, pl.threads, bytes, st>>>(in, w, kind, post, act, eps, (TS *)dx, (T *)dy,           \
                                                                 (T *)dgate, (float *)ws, rows, D, pl.lanes, params_at);   \
        }
#define GLA_RUN(T, TS, V, S, N) GLA_MODE(T, TS, V, S, N, kAnyMode)
#define GLA_WHOLE(T, TS)                                                                                                   \
        if (mode == kOut + kY + kPost + kGated) GLA_MODE(T, TS, kVecs, true, kSmall, kOut + kY + kPost + kGated)           \
        else if (mode == kOut + kY + kPost + kGatedSigmoid) GLA_MODE(T, TS, kVecs, true, kSmall, kOut + kY + kPost + kGatedSigmoid) \
        else if (mode == kOut + kY + kPost) GLA_MODE(T, TS, kVecs, true, kSmall, kOut + kY + kPost)                        \
        else if (mode == kOut + kY + kGated) GLA_MODE(T, TS, kVecs, true, kSmall, kOut + kY + kGated)                      \
        else if (mode == kOut + kY + kGatedSigmoid) GLA_MODE(T, TS, kVecs, true, kSmall, kOut + kY + kGatedSigmoid)        \
        else if (mode == kOut + kY) GLA_MODE(T, TS, kVecs, true, kSmall, kOut + kY)                                        \
        else found = false;
        bool found = whole;
        if (whole) {
            if (dtype == GLA_F32) { GLA_WHOLE(float, float) }
            else if (stream_dtype == GLA_F32) { GLA_WHOLE(__nv_bfloat16, float) }
            else { GLA_WHOLE(__nv_bfloat16, __nv_bfloat16) }
        }
        if (!found) { GLA_BY_TYPE(GLA_RUN) }
#undef GLA_WHOLE
#undef GLA_MODE
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
