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
// tokens (kVec vectors of eight), so weight and bias stay in registers, as do the sums of dweight and dbias; the
// statistics are taken from the registers in two steps (mean, then centred squares) by shuffles between the
// lanes of a group.  The blocks' sums of dweight and dbias go to a workspace that a second kernel adds up in a
// fixed order.
#include "gla_common.cuh"

namespace gla {
namespace norm {
namespace {

constexpr int kThreads = 128;

enum Act { kNone = GLA_ACT_NONE, kSilu = GLA_ACT_SILU, kSigmoid = GLA_ACT_SIGMOID };

// 1 / (1 + e^-x); for x below about -87 the exponential overflows and the quotient is the limit 0.
__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

// Lanes per group (a power of two) and vectors of eight channels per lane.
struct Plan {
    int lanes, vecs, slots, per_block, blocks_y, rows_per_block;
};

Plan make_plan(int groups, int width) {
    const int nv = width / 8;
    Plan best{};
    int cost = 1 << 30;
    for (int L = 1; L <= 32; L *= 2) {  // fewest idle vectors, then the most lanes (longer contiguous reads)
        const int v = (nv + L - 1) / L;
        if (v > 8) continue;
        const int c = (L * v - nv) * 64 - L + (v > 4 ? 16 : 0);
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

template <typename T> struct Vec;  // eight elements as they lie in memory
template <> struct Vec<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { a = __ldcs(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void put(__nv_bfloat16 *p, const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 t = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&t);
        }
        __stcs(reinterpret_cast<uint4 *>(p), make_uint4(w[0], w[1], w[2], w[3]));
    }
};
template <> struct Vec<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = __ldcs(reinterpret_cast<const float4 *>(p));
        b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
    static __device__ __forceinline__ void put(float *p, const float (&x)[8]) {
        __stcs(reinterpret_cast<float4 *>(p), make_float4(x[0], x[1], x[2], x[3]));
        __stcs(reinterpret_cast<float4 *>(p) + 1, make_float4(x[4], x[5], x[6], x[7]));
    }
};

__device__ __forceinline__ float group_sum(float x, int lanes) {
    for (int m = lanes >> 1; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

// Where a thread stands: its first channel, and whether each of its vectors exists.
template <int kVec> struct Place {
    int row_in_block, channel, nv, sub, lanes;
    bool live;
    __device__ __forceinline__ Place(int groups, int width, int lanes_, int per_block) : lanes(lanes_) {
        const int slot = blockIdx.y * per_block + threadIdx.x % per_block;
        row_in_block = threadIdx.x / per_block;
        nv = width >> 3;
        sub = slot % lanes;
        channel = (slot / lanes) * width + sub * 8;
        live = slot < groups * lanes && row_in_block < kThreads / per_block;
    }
    __device__ __forceinline__ bool has(int j) const { return live && sub + j * lanes < nv; }
    __device__ __forceinline__ int at(int j) const { return channel + j * lanes * 8; }
};

// Mean and 1 / sqrt(variance + eps) of the group whose part x a lane holds (zeros where it has no vector).
template <int kVec>
__device__ __forceinline__ void statistics(const float (&x)[kVec][8], const Place<kVec> &pl, float inv_width, float eps,
                                           float &mean, float &r) {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < kVec; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) s += x[j][e];
    mean = group_sum(s, pl.lanes) * inv_width;
    s = 0.f;
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        if (pl.has(j)) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = x[j][e] - mean;
                s = fmaf(d, d, s);
            }
        }
    }
    r = rsqrtf(fmaf(group_sum(s, pl.lanes), inv_width, eps));
}

template <typename T, int kVec, bool kGate>
__global__ void __launch_bounds__(kThreads)
norm_fwd_kernel(const T *__restrict__ x, const float *__restrict__ weight, const float *__restrict__ bias,
                const T *__restrict__ gate, int act, float eps, T *__restrict__ out, int64_t rows, int groups, int width,
                int lanes, int per_block) {
    const Place<kVec> pl(groups, width, lanes, per_block);
    const int64_t C = (int64_t)groups * width;
    float w[kVec][8], b[kVec][8];
#pragma unroll
    for (int j = 0; j < kVec; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            w[j][e] = pl.has(j) && weight != nullptr ? __ldg(weight + pl.at(j) + e) : 1.f;
            b[j][e] = pl.has(j) && bias != nullptr ? __ldg(bias + pl.at(j) + e) : 0.f;
        }
    const int step = kThreads / per_block;
    const float inv_width = 1.f / (float)width;
    for (int64_t r0 = (int64_t)blockIdx.x * step; r0 < rows; r0 += (int64_t)gridDim.x * step) {
        const int64_t row = r0 + pl.row_in_block;
        const bool live = row < rows;
        Vec<T> vx[kVec], vg[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j)
            if (live && pl.has(j)) {
                vx[j].load(x + row * C + pl.at(j));
                if (kGate) vg[j].load(gate + row * C + pl.at(j));
            }
        float f[kVec][8], mean, r;
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            if (live && pl.has(j)) vx[j].get(f[j]);
            else
#pragma unroll
                for (int e = 0; e < 8; ++e) f[j][e] = 0.f;
        }
        statistics<kVec>(f, pl, inv_width, eps, mean, r);
#pragma unroll
        for (int j = 0; j < kVec; ++j)
            if (live && pl.has(j)) {
                float g[8], y[8];
                if (kGate) vg[j].get(g);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float z = fmaf((f[j][e] - mean) * r, w[j][e], b[j][e]);
                    const float t = kGate ? g[e] : z;
                    if (act == kNone) y[e] = kGate ? z * t : z;
                    else if (act == kSilu) y[e] = (kGate ? z * t : z) * sigmoid(t);
                    else y[e] = kGate ? z * sigmoid(t) : sigmoid(t);
                }
                Vec<T>::put(out + row * C + pl.at(j), y);
            }
    }
}

template <typename T, int kVec, bool kGate>
__global__ void __launch_bounds__(kThreads)
norm_bwd_kernel(const T *__restrict__ dout, const T *__restrict__ x, const float *__restrict__ weight,
                const float *__restrict__ bias, const T *__restrict__ gate, int act, float eps, T *__restrict__ dx,
                T *__restrict__ dgate, float *__restrict__ part, int64_t rows, int groups, int width, int lanes,
                int per_block) {
    __shared__ float sums[kThreads][9];
    const Place<kVec> pl(groups, width, lanes, per_block);
    const int64_t C = (int64_t)groups * width;
    float w[kVec][8], b[kVec][8], dw[kVec][8], db[kVec][8];
#pragma unroll
    for (int j = 0; j < kVec; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            w[j][e] = pl.has(j) && weight != nullptr ? __ldg(weight + pl.at(j) + e) : 1.f;
            b[j][e] = pl.has(j) && bias != nullptr ? __ldg(bias + pl.at(j) + e) : 0.f;
            dw[j][e] = db[j][e] = 0.f;
        }
    const int step = kThreads / per_block;
    const float inv_width = 1.f / (float)width;
    for (int64_t r0 = (int64_t)blockIdx.x * step; r0 < rows; r0 += (int64_t)gridDim.x * step) {
        const int64_t row = r0 + pl.row_in_block;
        const bool live = row < rows;
        Vec<T> vx[kVec], vg[kVec], vd[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j)
            if (live && pl.has(j)) {
                vx[j].load(x + row * C + pl.at(j));
                vd[j].load(dout + row * C + pl.at(j));
                if (kGate) vg[j].load(gate + row * C + pl.at(j));
            }
        float f[kVec][8], d[kVec][8], mean, r;
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            if (live && pl.has(j)) vx[j].get(f[j]);
            else
#pragma unroll
                for (int e = 0; e < 8; ++e) f[j][e] = 0.f;
        }
        statistics<kVec>(f, pl, inv_width, eps, mean, r);
        float s = 0.f, sh = 0.f;
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            if (live && pl.has(j)) {
                float g[8], dg[8];
                vd[j].get(d[j]);
                if (kGate) vg[j].get(g);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float h = (f[j][e] - mean) * r, z = fmaf(h, w[j][e], b[j][e]);
                    const float t = kGate ? g[e] : z, q = sigmoid(t);
                    const float slope = act == kNone ? 1.f : act == kSilu ? q * fmaf(t, 1.f - q, 1.f) : q * (1.f - q);
                    float dz;
                    if (kGate) {
                        const float up = d[j][e];
                        dz = up * (act == kNone ? t : act == kSilu ? t * q : q);
                        dg[e] = up * z * slope;
                    } else {
                        dz = d[j][e] * slope;
                    }
                    dw[j][e] = fmaf(dz, h, dw[j][e]);
                    db[j][e] += dz;
                    const float dh = dz * w[j][e];
                    s += dh;
                    sh = fmaf(dh, h, sh);
                    f[j][e] = h;
                    d[j][e] = dh;
                }
                if (kGate) Vec<T>::put(dgate + row * C + pl.at(j), dg);
            }
        }
        s = group_sum(s, pl.lanes) * inv_width;
        sh = group_sum(sh, pl.lanes) * inv_width;
#pragma unroll
        for (int j = 0; j < kVec; ++j)
            if (live && pl.has(j)) {
                float y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = r * (d[j][e] - s - f[j][e] * sh);
                Vec<T>::put(dx + row * C + pl.at(j), y);
            }
    }
    // the block's rows of one channel set meet in shared memory; one writer per channel
    float *to = part + (int64_t)blockIdx.x * 2 * C;
#pragma unroll
    for (int j = 0; j < kVec; ++j)
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < 8; ++e) sums[threadIdx.x][e] = which ? db[j][e] : dw[j][e];
            __syncthreads();
            if (pl.row_in_block == 0 && pl.has(j)) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float v = 0.f;
                    for (int m = 0; m < step; ++m) v += sums[threadIdx.x + m * per_block][e];
                    to[which * C + pl.at(j) + e] = v;
                }
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
    const int64_t need = (rows + pl.rows_per_block - 1) / pl.rows_per_block;
    int64_t most = (int64_t)device_info().sm_count * per_sm / pl.blocks_y;
    if (most < 1) most = 1;
    return (int)(need < most ? need : most);
}

constexpr int kBwdPerSm = 4;

#define GLA_BY_VEC(v, CALL)      \
    switch (v) {                 \
        case 1: CALL(1); break;  \
        case 2: CALL(2); break;  \
        case 3: CALL(3); break;  \
        case 4: CALL(4); break;  \
        case 5: CALL(5); break;  \
        case 6: CALL(6); break;  \
        case 7: CALL(7); break;  \
        default: CALL(8); break; \
    }

template <typename T>
int fwd(const T *x, const float *weight, const float *bias, const T *gate, int act, float eps, T *out, int64_t rows,
        int groups, int width, cudaStream_t st) {
    if (rows == 0) return GLA_OK;
    const Plan pl = make_plan(groups, width);
    const dim3 grid((unsigned)blocks_x(pl, rows, 16), (unsigned)pl.blocks_y);
#define GLA_CALL(V)                                                                                               \
    if (gate) norm_fwd_kernel<T, V, true><<<grid, kThreads, 0, st>>>(x, weight, bias, gate, act, eps, out, rows,   \
                                                                     groups, width, pl.lanes, pl.per_block);       \
    else norm_fwd_kernel<T, V, false><<<grid, kThreads, 0, st>>>(x, weight, bias, gate, act, eps, out, rows,       \
                                                                 groups, width, pl.lanes, pl.per_block)
    GLA_BY_VEC(pl.vecs, GLA_CALL)
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
        nb = blocks_x(pl, rows, kBwdPerSm);
        const dim3 grid((unsigned)nb, (unsigned)pl.blocks_y);
#define GLA_CALL(V)                                                                                                  \
    if (gate) norm_bwd_kernel<T, V, true><<<grid, kThreads, 0, st>>>(dout, x, weight, bias, gate, act, eps, dx,       \
                                                                     dgate, ws, rows, groups, width, pl.lanes,        \
                                                                     pl.per_block);                                   \
    else norm_bwd_kernel<T, V, false><<<grid, kThreads, 0, st>>>(dout, x, weight, bias, gate, act, eps, dx, dgate,    \
                                                                 ws, rows, groups, width, pl.lanes, pl.per_block)
        GLA_BY_VEC(pl.vecs, GLA_CALL)
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

// Bytes of the blocks' sums of dweight and dbias.
size_t workspace(int64_t rows, int groups, int width) {
    const Plan pl = make_plan(groups, width);
    return (size_t)blocks_x(pl, rows < 1 ? 1 : rows, kBwdPerSm) * 2 * groups * width * sizeof(float);
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
