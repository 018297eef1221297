// gla_resnorm.cuh — what the residual norm and its gradient share.
//
// Both are bound by HBM.  A row is one block's, a part of a warp's where it is short, a cluster's where it is wide; a thread takes
// four neighbouring channels at a time and keeps the same ones for all of its rows, so the gradient's sums over tokens stay in
// registers until its last row.  An SM has several blocks where their threads allow, so that one row's barriers wait beside another's
// work; the gradient has one above 2,560 channels, of 352 to 640 threads.  Rows come into shared memory by bulk copies, some rows ahead, and are read from there by each step: what is in flight costs no registers.
// Rows of the forward that two stages have no room for are read from memory.
//
// Measured with all parts (layer norms before and behind, gate, scale; bf16): forward of 16,384 x 2,560 97 us (the bytes at the
// rate of a copy: 62), of an RMS norm alone behind the sum 55 (50); gradient 177 and 95 (99 and 74).  8,192 x 5,120: 105 and 187;
// f32 8,192 x 2,560: 79 and 166 (62 and 99).  The gradient between two sizes that fill 640 threads, for the same bytes: 2,568 323 and
// 152, 3,584 230 and 115, 4,096 200 and 104, 5,112 214 and 101.  What bounds the gradient is this code's instructions, about 90 a
// channel, and two meetings of a row's warps; the forward waits for its four meetings (for two rows) and for the parameters, which
// are as many bytes as the row.
//
// The file that includes this defines record_status before it.
#pragma once

#include <type_traits>

#include "gla_act.cuh"
#include "sm100_ptx.cuh"

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

// A row is one block's, or where it is wide a cluster's: `ranks` blocks take `slice` channels each (the last the rest) and meet
// in one another's shared memory.  So a block of the gradient has at most kWidest channels: its threads' sums then have the
// registers that they need.  (In the gradient, one meeting of four blocks costs 2 us, of two 0.7, within one 0.4.  8,192 x 5,120
// bf16: one block of 640 threads 186 us, two of 320 on different SMs 254.)
// Threads to a block's part of a row (whole warps above 32), rows of a block at a time.  A thread's vectors are kStride channels
// apart, so that those of a warp are neighbours and a vector's place is a constant away from the thread's first.
struct Plan {
    int ranks, slice, lanes, vecs, rows, threads;
};
constexpr int kStride = 128, kWidest = 5120, kMostRanks = 4;
static_assert(kMostRanks * kWidest >= 16384, "");

inline Plan make_plan(int D, int vecs, int widest) {  // widest: of a block
    Plan p{};
    p.ranks = 1;
    while (p.ranks * widest < D) p.ranks *= 2;
    p.slice = p.ranks == 1 ? D : (D + 8 * p.ranks - 1) / (8 * p.ranks) * 8;
    p.vecs = D <= kStride ? 1 : D <= 2 * kStride ? 2 : vecs;
    p.lanes = 1;
    if (D <= kStride)
        while (p.lanes < D / 4) p.lanes *= 2;
    else
        p.lanes = (p.slice + kStride * p.vecs - 1) / (kStride * p.vecs) * 32;
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
            typename Four<T>::Raw raw{};
            if (has(j)) raw = *reinterpret_cast<const typename Four<T>::Raw *>(p + j * kStride);
            Four<T>::open(v[j], raw);
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

// A block's place in its row's cluster.
template <bool kWide> struct Cluster {
    int rank = 0, ranks = 1;
    __device__ __forceinline__ Cluster() {
        if (!kWide) return;
        asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
        asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
    }
    __device__ __forceinline__ void sync() const {
        if (kWide) {
            asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
            asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        } else {
            __syncthreads();
        }
    }
    __device__ __forceinline__ void put(float *here, float v, int to) const {  // the same place in another block
        uint32_t at;
        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(ptx::smem_u32(here)), "r"(to));
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
    }
};

// Where a row's warps meet for two sums at once and for six, in one half and then in the other, so that one barrier a sum is
// enough.  The entries of warps that there are not stay zero.
template <bool kWide> struct Meeting {
    static constexpr int kWarps = kWide ? kMostRanks * kWidest / 256 : 32;
    float two[2][2][kWarps];  // the first sum's parts by warp, and the second's
    float six[2][kWarps][8];
    __device__ __forceinline__ void clear() {
        for (int i = threadIdx.x; i < (int)(sizeof(Meeting) / sizeof(float)); i += blockDim.x) reinterpret_cast<float *>(this)[i] = 0.f;
    }
};

// Two sums over a row's threads at once; every thread of the block calls this.
template <bool kWide>
__device__ __forceinline__ float2 row_sum(float a, float b, int lanes, const Cluster<kWide> &cl, Meeting<kWide> &m, int &half) {
    if (!kWide && lanes < 32) {
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
    if (kWide || lanes > 32) {
        float(&at)[2][Meeting<kWide>::kWarps] = m.two[half];
        const int warps = blockDim.x >> 5;
        float *const mine = &at[upper][cl.rank * warps + (threadIdx.x >> 5)];
        if (kWide) {
            if ((lane & 15) < cl.ranks) cl.put(mine, v, lane & 15);
        } else if ((lane & 15) == 0) {
            *mine = v;
        }
        cl.sync();
        v = at[upper][lane & 15];
        if (kWide) {
            for (int i = 16; i < cl.ranks * warps; i += 16) v += at[upper][i + (lane & 15)];
        } else if (lanes > 512) {
            v += at[upper][16 + (lane & 15)];
        }
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
        half ^= 1;
    }
    const float o = __shfl_xor_sync(0xffffffffu, v, 16);
    return upper ? make_float2(o, v) : make_float2(v, o);
}

// Six sums at once, each thread's parts given and the row's sums returned in v: three halvings leave a lane with one of them.
// kMost: the block's threads at most.
template <int kMost, bool kWide>
__device__ __forceinline__ void row_sums(float (&v)[6], int lanes, const Cluster<kWide> &cl, Meeting<kWide> &m, int &half) {
    if (!kWide && lanes < 32) {
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
    if (!kWide && lanes == 32) {
#pragma unroll
        for (int i = 0; i < 6; ++i) v[i] = __shfl_sync(0xffffffffu, x, i / 3 * 16 + (i % 3 == 2 ? 4 : i % 3 * 8));
        return;
    }
    const int warps = blockDim.x >> 5;
    float(&at)[Meeting<kWide>::kWarps][8] = m.six[half];
    float *const mine = &at[cl.rank * warps + (threadIdx.x >> 5)][(b16 ? 3 : 0) + (b4 ? 2 : b8 ? 1 : 0)];
    if (!(b4 && b8)) {
        if (kWide) {
            for (int to = lane & 3; to < cl.ranks; to += 4) cl.put(mine, x, to);
        } else if ((lane & 3) == 0) {
            *mine = x;
        }
    }
    cl.sync();
    x = at[lane >> 3][lane & 7];
    if (kWide) {
        for (int i = 4; i < cl.ranks * warps; i += 4) x += at[(lane >> 3) + i][lane & 7];
    } else {
#pragma unroll
        for (int i = 1; i < (kMost / 32 + 3) / 4; ++i) x += at[(lane >> 3) + 4 * i][lane & 7];
    }
    x += __shfl_xor_sync(0xffffffffu, x, 16);
    x += __shfl_xor_sync(0xffffffffu, x, 8);
#pragma unroll
    for (int i = 0; i < 6; ++i) v[i] = __shfl_sync(0xffffffffu, x, i);
    half ^= 1;
}

// Arrays whose rows come in, and the stages that they come into: the rows of an item, of each array; of a wide row a block's
// slice, and the row's first channels for near_mean().
template <int kArrays> struct Inputs {
    const void *from[kArrays];  // null: absent
    int row_bytes[kArrays], slice_bytes[kArrays], head_bytes[kArrays], at[kArrays], head_at[kArrays];
    int stage_bytes, stages, passes;
};

// The rows of a block, an item (`passes` rows for each of its threads) after the other.
struct Bars {
    uint64_t full[kMaxStages], read[kMaxStages];
    int failed;
};
template <bool kStage, int kArrays, bool kWide>
struct Rows {
    const Inputs<kArrays> &in;
    const Cluster<kWide> &cl;
    uint8_t *ring;
    Bars &bars;
    int64_t rows, row;               // row: the thread's
    int item, items, units, at_once, step, mine, st;  // rows at once and of an item; the thread's row in its item
    uint32_t phase;
    bool late;  // whether the stage of the item before is still to be refilled
    __device__ __forceinline__ Rows(const Inputs<kArrays> &in_, const Cluster<kWide> &cl_, uint8_t *ring_, Bars &bars_, int64_t rows_, int lanes)
        : in(in_), cl(cl_), ring(ring_), bars(bars_), rows(rows_), item(blockIdx.x), units(gridDim.x), at_once(blockDim.x / lanes), st(0), phase(0),
          late(false) {
        if (kWide) item /= cl.ranks, units /= cl.ranks;
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
            for (int i = 0; i < in.stages; ++i) order(i, item + i * units);
        }
    }
    // by one thread
    __device__ __forceinline__ void order(int to_stage, int k) const {
        if (k >= items) return;
        const uint32_t b = ptx::smem_u32(bars.full + to_stage), to = ptx::smem_u32(ring) + (uint32_t)(to_stage * in.stage_bytes);
        const int64_t first = (int64_t)k * step;
        const int n = (int)min((int64_t)step, rows - first);
        uint32_t bytes = 0;
        // a slice's bytes, or the rows'
        auto size = [&](int i) {
            return (uint32_t)(kWide ? min(in.slice_bytes[i], in.row_bytes[i] - cl.rank * in.slice_bytes[i]) : n * in.row_bytes[i]);
        };
#pragma unroll
        for (int i = 0; i < kArrays; ++i)
            if (in.from[i] != nullptr) bytes += size(i) + (kWide ? (uint32_t)in.head_bytes[i] : 0u);
        ptx::mbar_expect_tx(b, bytes);
#pragma unroll
        for (int i = 0; i < kArrays; ++i)
            if (in.from[i] != nullptr) {
                const uint8_t *const from = (const uint8_t *)in.from[i] + first * in.row_bytes[i];
                ptx::bulk_load_g2s(to + (uint32_t)in.at[i], from + (kWide ? cl.rank * in.slice_bytes[i] : 0), size(i), b);
                if (kWide && in.head_bytes[i] > 0) ptx::bulk_load_g2s(to + (uint32_t)in.head_at[i], from, (uint32_t)in.head_bytes[i], b);
            }
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
        if (kStage && late && threadIdx.x == 0) order(st == 0 ? in.stages - 1 : st - 1, item + (in.stages - 1) * units);
        late = false;
        __syncwarp();
    }
    __device__ __forceinline__ void next() {
        mine += at_once;
        row += at_once;
        if (mine < step) return;
        mine -= step;
        row += ((int64_t)units - 1) * step;
        if (kStage) {
            __syncwarp();
            if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(ptx::smem_u32(bars.read + st));
            late = true;
            if (++st == in.stages) {
                st = 0;
                phase ^= 1u;
            }
        }
        item += units;
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
    // the row's first channel
    template <typename T> __device__ __forceinline__ const T *head(int i, int D) const {
        if (kWide) return reinterpret_cast<const T *>(ring + st * in.stage_bytes + in.head_at[i]);
        return at<T>(i, D, 0);
    }
};

// A thread's place in its block's part of a row, D channels: its first channel and how many of its vectors exist.
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
};

// Blocks of an SM, and the rows at a time of all of them (a block's, or a cluster's).
inline int per_sm(const Plan &pl, int threads) { return threads < pl.threads ? 1 : threads / pl.threads; }
inline int units(const Plan &pl, int64_t rows, int per_sm) {
    const int64_t need = (rows + pl.rows - 1) / pl.rows;
    int64_t most = (int64_t)device_info().sm_count * per_sm / pl.ranks;
    if (most < 1) most = 1;
    return (int)(need < most ? need : most);
}

constexpr int kMostShared = 218 * 1024;

// The stages of a block: an item's rows of each array one behind the other; behind them the parameters, `params` bytes, where
// there is room (else params_at is negative: they are read from memory, and what shared memory leaves caches them).  Short rows
// are taken some at a time, while there are enough for all blocks: an item's copies then serve several rows of a thread.
template <int kArrays>
int lay_out(Inputs<kArrays> &in, const Plan &pl, int64_t rows, int per_sm, int nblocks, int params, int &params_at) {
    const bool wide = pl.ranks > 1;
    int row = 0, at = 0;
    for (int i = 0; i < kArrays; ++i)
        if (in.from[i] != nullptr) row += in.row_bytes[i];
    in.passes = 1;
    while (!wide && in.passes < 8 && 2 * in.passes * pl.rows * row <= 16 * 1024 && rows >= 4LL * in.passes * pl.rows * nblocks) in.passes *= 2;
    const int room = kMostShared / per_sm - (per_sm == 1 ? 0 : wide ? 6144 : 3328);
    auto place = [&](int bytes) {
        const int here = at;
        at += (bytes + 127) / 128 * 128;
        return here;
    };
    for (;; in.passes /= 2) {  // fewer, where that leaves the parameters their room
        at = 0;
        for (int i = 0; i < kArrays; ++i) {
            if (in.from[i] == nullptr) continue;
            in.at[i] = place(wide ? in.slice_bytes[i] : in.passes * pl.rows * in.row_bytes[i]);
            if (wide) in.head_at[i] = place(in.head_bytes[i]);
        }
        if (in.passes == 1 || 2 * at + params <= room) break;
    }
    in.stage_bytes = at;
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

// Launches a kernel of `units` blocks, or clusters of `ranks` blocks: of those no more than run at once, since the rest would
// start when the others have taken their whole share of the rows (of 4 and 8 blocks the device does not take as many as its SMs
// have room for: a cluster is one GPC's).  Returns their number, 0 for a failure.  The runtime is asked once for the same kernel,
// block and shared memory on a device; what it answered last is kept in one word.
template <auto kKernel, class... Args>
int launch(int units, int ranks, int threads, int bytes, cudaStream_t st, Args... args) {
    if (!allow_most<kKernel>()) return 0;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3((unsigned)(units * ranks));
    c.blockDim = dim3((unsigned)threads);
    c.dynamicSmemBytes = (size_t)bytes;
    c.stream = st;
    cudaLaunchAttribute a{};
    a.id = cudaLaunchAttributeClusterDimension;
    a.val.clusterDim.x = (unsigned)ranks, a.val.clusterDim.y = a.val.clusterDim.z = 1;
    c.attrs = &a;
    c.numAttrs = ranks > 1 ? 1 : 0;
    if (ranks > 1) {
        static std::atomic<uint64_t> last;  // device, ranks, threads, bytes; clusters
        int dev = 0, n = 0;
        if (cudaGetDevice(&dev) != cudaSuccess) return 0;
        const uint64_t key = ((((uint64_t)dev << 4 | (uint64_t)ranks) << 11 | (uint64_t)threads) << 18 | (uint64_t)bytes) << 16;
        const uint64_t known = last.load(std::memory_order_relaxed);
        if ((known & ~(uint64_t)0xffff) == key && known != 0) n = (int)(known & 0xffff);
        else {
            if (cudaOccupancyMaxActiveClusters(&n, kKernel, &c) != cudaSuccess || n < 1) return 0;
            last.store(key | (uint64_t)(n & 0xffff), std::memory_order_relaxed);
        }
        if (units > n) units = n;
        c.gridDim = dim3((unsigned)(units * ranks));
    }
    return cudaLaunchKernelEx(&c, kKernel, args...) == cudaSuccess ? units : 0;
}

}  // namespace
}  // namespace resnorm
}  // namespace gla
