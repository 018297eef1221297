// gla_norm.cu — group normalisation of a token's channels (channels last, one group to a head) with an
// activation, and its gradient.
//
// For a token's group x of `width` channels, mean m and variance s2 over the group, r = 1 / sqrt(s2 + eps):
//     h = (x - m) r,   z = weight h + bias,   out = z act(gate), or act(z) without a gate.
// A causal mixer may not mix statistics over time, so the normalised extent is one token's group.
//
// Gradient, with dz = dout act(gate) (or dout act'(z)), dh = dz weight:
//     dx = r (dh - mean(dh) - h mean(dh h)),  dgate = dout z act'(gate),
//     dweight = sum over tokens of dz h,      dbias = sum over tokens of dz.
//
// Both are bound by HBM: every array is read or written once.  A thread keeps the same channels for all of its
// tokens (kVec vectors of four), so weight and bias stay in registers, as do the sums of dweight and dbias; the
// statistics are taken from the registers in two steps (mean, then centred squares) by shuffles between the
// lanes of a group.  The next token's vectors are on their way while one is computed.  The gradient does some
// thirty operations an element, so arithmetic runs on pairs of f32 (fma.rn.f32x2 and
// the like).  The blocks' sums of dweight and dbias go to a workspace that a second kernel adds up in a fixed order.
//
// 16,384 tokens of 16 groups of 192, bf16 with a gate: 55 us (302 MB, 5.5 TB/s, 0.81 of a copy's rate); gradient
// 100 us (503 MB, 5.0 TB/s, 0.74), of which 9 are the second kernel.  Scalar arithmetic took 71 and 209; pairs with
// fewer blocks on an SM 66 and 103.
#include "gla_act.cuh"

namespace gla {
namespace norm {
namespace {

constexpr int kThreads = 256;

// Lanes per group (a power of two, whole warps above 32) and vectors of four channels per lane.
struct Plan {
    int lanes, vecs, slots, per_block, blocks_y, rows_per_block;
};

// The vectors per lane that the kernels are built for: more would not fit their registers.
#define GLA_BY_VEC(v, CALL)       \
    switch (v) {                  \
        case 1: CALL(1); break;   \
        case 2: CALL(2); break;   \
        case 3: CALL(3); break;   \
        default: CALL(4); break;  \
    }

#define GLA_BY_ACT(V, RUN)                              \
    if (gate) {                                         \
        if (act == kNone) RUN(V, true, kNone);          \
        else if (act == kSilu) RUN(V, true, kSilu);     \
        else RUN(V, true, kSigmoid);                    \
    } else {                                            \
        if (act == kNone) RUN(V, false, kNone);         \
        else if (act == kSilu) RUN(V, false, kSilu);    \
        else RUN(V, false, kSigmoid);                   \
    }

Plan make_plan(int groups, int width) {
    const int nv = width / 4;
    Plan best{};
    int cost = 1 << 30;
    for (int L = 1; L <= 128; L *= 2) {
        const int v = (nv + L - 1) / L;
        if (v > 4) continue;
        // fewest idle vectors, then the fewest shuffles but at least eight lanes (64 neighbouring bytes of bf16)
        const int c = (L * v - nv) * 64 + (L < 8 ? 8 / L : 0) + L / 4;
        if (c < cost) {
            cost = c;
            best.lanes = L;
            best.vecs = v;
        }
    }
    best.slots = groups * best.lanes;
    best.per_block = best.slots < kThreads ? best.slots : kThreads;
    best.blocks_y = (best.slots + best.per_block - 1) / best.per_block;
    best.rows_per_block = kThreads / best.per_block;
    return best;
}

template <typename T> struct Vec;  // four elements as they lie in memory
template <> struct Vec<__nv_bfloat16> {
    uint2 a;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { a = __ldcs(reinterpret_cast<const uint2 *>(p)); }
    __device__ __forceinline__ void clear() { a = make_uint2(0, 0); }
    __device__ __forceinline__ Pair get(int e) const {
        const uint32_t w = e ? a.y : a.x;
        return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    static __device__ __forceinline__ void put(__nv_bfloat16 *p, const Pair (&x)[2]) {
        const float2 f = parts(x[0]), g = parts(x[1]);
        const __nv_bfloat162 u = __floats2bfloat162_rn(f.x, f.y), v = __floats2bfloat162_rn(g.x, g.y);
        __stcs(reinterpret_cast<uint2 *>(p),
               make_uint2(*reinterpret_cast<const uint32_t *>(&u), *reinterpret_cast<const uint32_t *>(&v)));
    }
};
template <> struct Vec<float> {
    float4 a;
    __device__ __forceinline__ void load(const float *p) { a = __ldcs(reinterpret_cast<const float4 *>(p)); }
    __device__ __forceinline__ void clear() { a = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ Pair get(int e) const { return e ? pair(a.z, a.w) : pair(a.x, a.y); }
    static __device__ __forceinline__ void put(float *p, const Pair (&x)[2]) {
        const float2 f = parts(x[0]), g = parts(x[1]);
        __stcs(reinterpret_cast<float4 *>(p), make_float4(f.x, f.y, g.x, g.y));
    }
};
// four parameters of this thread's vector, or a constant where the array or the vector is absent
__device__ __forceinline__ void load_param(Pair (&to)[2], const float *from, int at, bool has, float otherwise) {
    float4 f = make_float4(otherwise, otherwise, otherwise, otherwise);
    if (has && from != nullptr) f = __ldg(reinterpret_cast<const float4 *>(from + at));
    to[0] = pair(f.x, f.y);
    to[1] = pair(f.z, f.w);
}

// The sum over a group's lanes.  Groups of more than a warp meet in `wide`; every thread of the block calls this.
__device__ __forceinline__ float group_sum(float x, int lanes, float *wide) {
    for (int m = min(lanes, 32) >> 1; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    if (lanes > 32) {
        const int warp = threadIdx.x >> 5, warps = lanes >> 5, first = warp / warps * warps;
        __syncthreads();
        if ((threadIdx.x & 31) == 0) wide[warp] = x;
        __syncthreads();
        x = 0.f;
        for (int m = 0; m < warps; ++m) x += wide[first + m];
    }
    return x;
}

// Where a thread stands: its row in the block, its first channel, and how many of its vectors exist.
struct Place {
    int row_in_block, channel, count, stride;
    __device__ __forceinline__ Place(int groups, int width, int lanes, int per_block) {
        const int slot = blockIdx.y * per_block + threadIdx.x % per_block;
        row_in_block = threadIdx.x / per_block;
        const int sub = slot % lanes, nv = width >> 2;
        channel = (slot / lanes) * width + sub * 4;
        stride = lanes * 4;
        count = slot < groups * lanes && row_in_block < kThreads / per_block && sub < nv ? (nv - sub + lanes - 1) / lanes : 0;
    }
};

// The centred values d of a lane's part of its group (an absent vector is zero and stays out of both sums) and 1 /
// sqrt(variance + eps).
template <typename T, int kVec>
__device__ __forceinline__ void centre(const Vec<T> (&x)[kVec], Pair (&d)[kVec][2], int count, int lanes, float inv_width,
                                       float eps, float *wide, float &r) {
    Pair s = both(0.f);
#pragma unroll
    for (int j = 0; j < kVec; ++j) s = s + (x[j].get(0) + x[j].get(1));
    const float mean = group_sum(total(s), lanes, wide) * inv_width;
    s = both(0.f);
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        const Pair m = both(j < count ? -mean : 0.f);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            d[j][e] = x[j].get(e) + m;
            s = fma(d[j][e], d[j][e], s);
        }
    }
    r = rsqrtf(fmaf(group_sum(total(s), lanes, wide), inv_width, eps));
}

template <typename T, int kVec>
__device__ __forceinline__ void fetch(Vec<T> (&v)[kVec], const T *from, int64_t at, int count, int stride) {
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        if (j < count) v[j].load(from + at + j * stride);
        else v[j].clear();
    }
}

// Blocks that an SM holds at once, by the registers that a thread's vectors take.
template <typename T> constexpr int fwd_per_sm(int vecs) { return vecs * (int)sizeof(T) <= 6 ? 3 : 2; }
template <typename T> constexpr int bwd_per_sm(int vecs) { return vecs * (int)sizeof(T) <= 6 ? 2 : 1; }

template <typename T, int kVec, bool kGate, int kAct>
__global__ void __launch_bounds__(kThreads, fwd_per_sm<T>(kVec))
norm_fwd_kernel(const T *__restrict__ x, const float *__restrict__ weight, const float *__restrict__ bias,
                const T *__restrict__ gate, float eps, T *__restrict__ out, int64_t rows, int groups, int width,
                int lanes, int per_block) {
    __shared__ float wide[kThreads / 32];
    const Place pl(groups, width, lanes, per_block);
    const int64_t C = (int64_t)groups * width;
    const int step = kThreads / per_block;
    const int64_t hop = (int64_t)gridDim.x * step;
    int64_t row = (int64_t)blockIdx.x * step + pl.row_in_block;
    Vec<T> nx[kVec], ng[kVec];
    fetch<T, kVec>(nx, x, row * C + pl.channel, row < rows ? pl.count : 0, pl.stride);
    if (kGate) fetch<T, kVec>(ng, gate, row * C + pl.channel, row < rows ? pl.count : 0, pl.stride);
    Pair w[kVec][2], b[kVec][2];
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        load_param(w[j], weight, pl.channel + j * pl.stride, j < pl.count, 1.f);
        load_param(b[j], bias, pl.channel + j * pl.stride, j < pl.count, 0.f);
    }
    const float inv_width = 1.f / (float)width;
    for (int64_t r0 = (int64_t)blockIdx.x * step; r0 < rows; r0 += hop, row += hop) {
        Vec<T> vx[kVec], vg[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            vx[j] = nx[j];
            if (kGate) vg[j] = ng[j];
        }
        const int count = row < rows ? pl.count : 0, next = row + hop < rows ? pl.count : 0;
        fetch<T, kVec>(nx, x, (row + hop) * C + pl.channel, next, pl.stride);
        if (kGate) fetch<T, kVec>(ng, gate, (row + hop) * C + pl.channel, next, pl.stride);
        float r;
        Pair d[kVec][2];
        centre<T, kVec>(vx, d, pl.count, lanes, inv_width, eps, wide, r);
        const Pair rr = both(r);
#pragma unroll
        for (int j = 0; j < kVec; ++j)
            if (j < count) {
                Pair y[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const Pair z = fma(d[j][e] * rr, w[j][e], b[j][e]);
                    const Pair t = kGate ? vg[j].get(e) : z;
                    Pair q, rest;
                    if (kAct != kNone) sigmoid(t, q, rest);
                    if (kAct == kNone) y[e] = kGate ? z * t : z;
                    else if (kAct == kSilu) y[e] = kGate ? z * (t * q) : z * q;  // t q first: z t may overflow where q is 0
                    else y[e] = kGate ? z * q : q;
                }
                Vec<T>::put(out + row * C + pl.channel + j * pl.stride, y);
            }
    }
}

template <typename T, int kVec, bool kGate, int kAct>
__global__ void __launch_bounds__(kThreads, bwd_per_sm<T>(kVec))
norm_bwd_kernel(const T *__restrict__ dout, const T *__restrict__ x, const float *__restrict__ weight,
                const float *__restrict__ bias, const T *__restrict__ gate, float eps, T *__restrict__ dx,
                T *__restrict__ dgate, float *__restrict__ part, int64_t rows, int groups, int width, int lanes,
                int per_block) {
    __shared__ float sums[kThreads][5], wide[kThreads / 32];
    const Place pl(groups, width, lanes, per_block);
    const int64_t C = (int64_t)groups * width;
    const int step = kThreads / per_block;
    const int64_t hop = (int64_t)gridDim.x * step;
    int64_t row = (int64_t)blockIdx.x * step + pl.row_in_block;
    Vec<T> nx[kVec], nd[kVec], ng[kVec];
    {
        const int count = row < rows ? pl.count : 0;
        fetch<T, kVec>(nx, x, row * C + pl.channel, count, pl.stride);
        fetch<T, kVec>(nd, dout, row * C + pl.channel, count, pl.stride);
        if (kGate) fetch<T, kVec>(ng, gate, row * C + pl.channel, count, pl.stride);
    }
    Pair w[kVec][2], b[kVec][2], dw[kVec][2], db[kVec][2];
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        load_param(w[j], weight, pl.channel + j * pl.stride, j < pl.count, 1.f);
        load_param(b[j], bias, pl.channel + j * pl.stride, j < pl.count, 0.f);
        dw[j][0] = dw[j][1] = db[j][0] = db[j][1] = both(0.f);
    }
    const float inv_width = 1.f / (float)width;
    for (int64_t r0 = (int64_t)blockIdx.x * step; r0 < rows; r0 += hop, row += hop) {
        Vec<T> vx[kVec], vd[kVec], vg[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            vx[j] = nx[j];
            vd[j] = nd[j];
            if (kGate) vg[j] = ng[j];
        }
        const int count = row < rows ? pl.count : 0, next = row + hop < rows ? pl.count : 0;
        fetch<T, kVec>(nx, x, (row + hop) * C + pl.channel, next, pl.stride);
        fetch<T, kVec>(nd, dout, (row + hop) * C + pl.channel, next, pl.stride);
        if (kGate) fetch<T, kVec>(ng, gate, (row + hop) * C + pl.channel, next, pl.stride);
        float r;
        Pair h[kVec][2], dh[kVec][2], s2 = both(0.f), sh2 = both(0.f);
        centre<T, kVec>(vx, h, pl.count, lanes, inv_width, eps, wide, r);
        const Pair rr = both(r);
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            if (j < count) {
                Pair dg[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    h[j][e] = h[j][e] * rr;
                    const Pair z = fma(h[j][e], w[j][e], b[j][e]), up = vd[j].get(e);
                    const Pair t = kGate ? vg[j].get(e) : z;
                    Pair q, rest, slope;
                    if (kAct != kNone) sigmoid(t, q, rest);
                    if (kAct == kSilu) slope = q * fma(t, rest, both(1.f));
                    if (kAct == kSigmoid) slope = q * rest;
                    Pair dz = kAct == kNone ? up : up * slope;  // through the activation's slope
                    if (kGate) {
                        dg[e] = dz * z;
                        dz = up * (kAct == kNone ? t : kAct == kSilu ? t * q : q);
                    }
                    dw[j][e] = fma(dz, h[j][e], dw[j][e]);
                    db[j][e] = db[j][e] + dz;
                    dh[j][e] = dz * w[j][e];
                    s2 = s2 + dh[j][e];
                    sh2 = fma(dh[j][e], h[j][e], sh2);
                }
                if (kGate) Vec<T>::put(dgate + row * C + pl.channel + j * pl.stride, dg);
            }
        }
        const Pair s = both(-group_sum(total(s2), lanes, wide) * inv_width),
                   sh = both(-group_sum(total(sh2), lanes, wide) * inv_width);
#pragma unroll
        for (int j = 0; j < kVec; ++j)
            if (j < count) {
                Pair y[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) y[e] = rr * fma(h[j][e], sh, dh[j][e] + s);
                Vec<T>::put(dx + row * C + pl.channel + j * pl.stride, y);
            }
    }
    // the block's rows of one channel set meet in shared memory; one writer per channel
    float *to = part + (int64_t)blockIdx.x * 2 * C;
#pragma unroll
    for (int j = 0; j < kVec; ++j)
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const float2 lo = parts(which ? db[j][0] : dw[j][0]), hi = parts(which ? db[j][1] : dw[j][1]);
            float v[4] = {lo.x, lo.y, hi.x, hi.y};
            if (step > 1) {
                __syncthreads();
#pragma unroll
                for (int e = 0; e < 4; ++e) sums[threadIdx.x][e] = v[e];
                __syncthreads();
            }
            if (pl.row_in_block == 0 && j < pl.count) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    for (int m = 1; m < step; ++m) v[e] += sums[threadIdx.x + m * per_block][e];
                *reinterpret_cast<float4 *>(to + which * C + pl.channel + j * pl.stride) = make_float4(v[0], v[1], v[2], v[3]);
            }
        }
}

// dweight[c], dbias[c] = the sum of the blocks' parts, 32 channels x 8 runs of blocks a block, in a fixed order.
__global__ void __launch_bounds__(256)
norm_param_kernel(const float *__restrict__ part, int nblocks, int64_t C, float *__restrict__ dweight,
                  float *__restrict__ dbias) {
    __shared__ float sm[8][33];
    const int64_t c = (int64_t)blockIdx.x * 32 + (threadIdx.x & 31);  // 0 .. 2C-1: dweight, then dbias
    const int run = threadIdx.x >> 5;
    float s = 0.f;
    if (c < 2 * C)
#pragma unroll 8
        for (int i = run; i < nblocks; i += 8) s += part[(int64_t)i * 2 * C + c];
    sm[run][threadIdx.x & 31] = s;
    __syncthreads();
    if (run == 0 && c < 2 * C) {
        s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += sm[i][threadIdx.x & 31];
        if (c < C) { if (dweight != nullptr) dweight[c] = s; }
        else if (dbias != nullptr) dbias[c - C] = s;
    }
}

int blocks_x(const Plan &pl, int64_t rows, int per_sm) {
    // blocks of one column set that run at once; more rows than that are walked over
    const int64_t need = (rows + pl.rows_per_block - 1) / pl.rows_per_block;
    int64_t most = (int64_t)device_info().sm_count * per_sm / pl.blocks_y;
    if (most < 1) most = 1;
    return (int)(need < most ? need : most);
}

template <typename T>
int fwd(const T *x, const float *weight, const float *bias, const T *gate, int act, float eps, T *out, int64_t rows,
        int groups, int width, cudaStream_t st) {
    if (rows == 0) return GLA_OK;
    const Plan pl = make_plan(groups, width);
    const dim3 grid((unsigned)blocks_x(pl, rows, fwd_per_sm<T>(pl.vecs)), (unsigned)pl.blocks_y);
#define GLA_RUN(V, G, A)                                                                                           \
    norm_fwd_kernel<T, V, G, A><<<grid, kThreads, 0, st>>>(x, weight, bias, gate, eps, out, rows, groups, width,    \
                                                           pl.lanes, pl.per_block)
#define GLA_CALL(V) GLA_BY_ACT(V, GLA_RUN)
    GLA_BY_VEC(pl.vecs, GLA_CALL)
#undef GLA_RUN
#undef GLA_CALL
    count_launches(1);
    return cudaGetLastError() == cudaSuccess ? GLA_OK : GLA_ERR_LAUNCH;
}

template <typename T>
int bwd(const T *dout, const T *x, const float *weight, const float *bias, const T *gate, int act, float eps, T *dx,
        float *dweight, float *dbias, T *dgate, float *ws, int64_t rows, int groups, int width, cudaStream_t st) {
    const Plan pl = make_plan(groups, width);
    const int64_t C = (int64_t)groups * width;
    int nb = 0;
    if (rows > 0) {
        nb = blocks_x(pl, rows, bwd_per_sm<T>(pl.vecs));
        const dim3 grid((unsigned)nb, (unsigned)pl.blocks_y);
#define GLA_RUN(V, G, A)                                                                                             \
    norm_bwd_kernel<T, V, G, A><<<grid, kThreads, 0, st>>>(dout, x, weight, bias, gate, eps, dx, dgate, ws, rows,     \
                                                           groups, width, pl.lanes, pl.per_block)
#define GLA_CALL(V) GLA_BY_ACT(V, GLA_RUN)
        GLA_BY_VEC(pl.vecs, GLA_CALL)
#undef GLA_RUN
#undef GLA_CALL
        count_launches(1);
    }
    if (dweight != nullptr || dbias != nullptr) {
        norm_param_kernel<<<(unsigned)((2 * C + 31) / 32), 256, 0, st>>>(ws, nb, C, dweight, dbias);
        count_launches(1);
    }
    return cudaGetLastError() == cudaSuccess ? GLA_OK : GLA_ERR_LAUNCH;
}

}  // namespace

// Bytes of the blocks' sums of dweight and dbias (bf16's blocks are never fewer than f32's).
size_t workspace(int64_t rows, int groups, int width) {
    const Plan pl = make_plan(groups, width);
    return (size_t)blocks_x(pl, rows < 1 ? 1 : rows, bwd_per_sm<__nv_bfloat16>(pl.vecs)) * 2 * groups * width * sizeof(float);
}

int group_norm(const void *x, const float *weight, const float *bias, const void *gate, int act, float eps, void *out,
               int64_t rows, int groups, int width, int dtype, cudaStream_t st) {
    using B = __nv_bfloat16;
    if (dtype == GLA_F32)
        return fwd<float>((const float *)x, weight, bias, (const float *)gate, act, eps, (float *)out, rows, groups,
                          width, st);
    return fwd<B>((const B *)x, weight, bias, (const B *)gate, act, eps, (B *)out, rows, groups, width, st);
}

int group_norm_bwd(const void *dout, const void *x, const float *weight, const float *bias, const void *gate, int act,
                   float eps, void *dx, float *dweight, float *dbias, void *dgate, void *ws, int64_t rows, int groups,
                   int width, int dtype, cudaStream_t st) {
    using B = __nv_bfloat16;
    if (dtype == GLA_F32)
        return bwd<float>((const float *)dout, (const float *)x, weight, bias, (const float *)gate, act, eps, (float *)dx,
                          dweight, dbias, (float *)dgate, (float *)ws, rows, groups, width, st);
    return bwd<B>((const B *)dout, (const B *)x, weight, bias, (const B *)gate, act, eps, (B *)dx, dweight, dbias,
                  (B *)dgate, (float *)ws, rows, groups, width, st);
}

}  // namespace norm
}  // namespace gla
