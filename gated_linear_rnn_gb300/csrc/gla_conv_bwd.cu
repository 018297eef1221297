// gla_conv_bwd.cu — the gradient of the causal depthwise Conv1d of width 4 with SiLU.
//
// With z_t = bias + sum_k weight[k] x_{t-3+k}, y_t = z_t s(z_t) and s the sigmoid, for each channel of a sequence of L tokens
// (x_{-3} .. x_{-1} is the state before it, x_{L-3} .. x_{L-1} the state behind it):
//     dz_t = dy_t s(z_t) (1 + z_t (1 - s(z_t))) for 0 <= t < L, else 0
//     dx_v = sum_k weight[k] dz_{v+3-k}, plus the gradient of the state behind for v >= L - 3;   v = -3 .. -1: of the state before
//     dweight[k] = sum over tokens of dz_t x_{t-3+k},   dbias = sum over tokens of dz_t
//
// A warp takes 128 channels, four a lane, of a run of rows of one sequence: the last three inputs and the last three dz stay
// in registers, and the three dz behind the run, which its last rows need, are computed again by the next run.
#include "gla_act.cuh"
#include "gla_seq.cuh"

GLA_DEFINE_STATUS(conv_bwd)

namespace gla {
namespace convbwd {
namespace {

constexpr int kRun = 64;      // rows of a run
constexpr int kWarps = 8;     // of a block
constexpr int kSlab = 128;    // channels of a warp
constexpr int kSums = 5;      // dweight[0 .. 3], dbias

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const int32_t *__restrict__ cu, int nseq, int T, int2 *rows) {
    if (plan_rows(cu, nseq, T, rows)) record_status(GLA_ERR_DEVICE_ARG);
}

template <typename T>
__device__ __forceinline__ void load4(Pair (&x)[2], const T *p);
template <>
__device__ __forceinline__ void load4<float>(Pair (&x)[2], const float *p) {
    const float4 f = __ldg(reinterpret_cast<const float4 *>(p));
    x[0] = pair(f.x, f.y);
    x[1] = pair(f.z, f.w);
}
template <>
__device__ __forceinline__ void load4<__nv_bfloat16>(Pair (&x)[2], const __nv_bfloat16 *p) {
    const uint2 w = __ldg(reinterpret_cast<const uint2 *>(p));
    x[0] = pair(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u));
    x[1] = pair(__uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
}
__device__ __forceinline__ void store4(float *p, const Pair (&x)[2]) {
    const float2 f = parts(x[0]), g = parts(x[1]);
    *reinterpret_cast<float4 *>(p) = make_float4(f.x, f.y, g.x, g.y);
}
__device__ __forceinline__ void store4(__nv_bfloat16 *p, const Pair (&x)[2]) {
    const float2 f = parts(x[0]), g = parts(x[1]);
    const __nv_bfloat162 u = __floats2bfloat162_rn(f.x, f.y), v = __floats2bfloat162_rn(g.x, g.y);
    *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const uint32_t *>(&u), *reinterpret_cast<const uint32_t *>(&v));
}
// entry m of four channels' states [D, 3]
__device__ __forceinline__ void load_state(Pair (&x)[2], const float *p, int m) {
    x[0] = pair(__ldg(p + m), __ldg(p + 3 + m));
    x[1] = pair(__ldg(p + 6 + m), __ldg(p + 9 + m));
}
__device__ __forceinline__ void store_state(float *p, int m, const Pair (&x)[2]) {
    const float2 f = parts(x[0]), g = parts(x[1]);
    p[m] = f.x, p[3 + m] = f.y, p[6 + m] = g.x, p[9 + m] = g.y;
}

template <typename T>
__global__ void __launch_bounds__(kWarps * 32)
bwd_kernel(const T *__restrict__ dy, const T *__restrict__ x, const float *__restrict__ weight, const float *__restrict__ bias,
           const float *__restrict__ state, const float *__restrict__ dstate_out, T *__restrict__ dx,
           float *__restrict__ dstate, float *__restrict__ part, Sequences q, int D, int64_t nslots) {
    __shared__ float4 tops[kWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.y * kSlab + lane * 4;
    const bool on = c < D;
    Pair w[4][2], b[2], dw[4][2], db[2];
    for (int e = 0; e < 2; ++e) {
        float4 p = make_float4(0.f, 0.f, 0.f, 0.f), r = p;
        if (on) {
            p = __ldg(reinterpret_cast<const float4 *>(weight + (int64_t)(c + 2 * e) * 4));
            r = __ldg(reinterpret_cast<const float4 *>(weight + (int64_t)(c + 2 * e + 1) * 4));
        }
        w[0][e] = pair(p.x, r.x), w[1][e] = pair(p.y, r.y), w[2][e] = pair(p.z, r.z), w[3][e] = pair(p.w, r.w);
        b[e] = on && bias != nullptr ? pair(__ldg(bias + c + 2 * e), __ldg(bias + c + 2 * e + 1)) : both(0.f);
        db[e] = both(0.f);
        for (int k = 0; k < 4; ++k) dw[k][e] = both(0.f);
    }
    const int first = (int)blockIdx.x * kWarps + warp, hop = (int)gridDim.x * kWarps;
    if (on && dstate != nullptr)  // sequences without tokens pass the gradient of their state on
        for (int64_t s = first; s < q.nseq; s += hop)
            if (rows_of(q, (int)s).y == 0)
                for (int m = 0; m < 12; ++m)
                    dstate[(s * D + c) * 3 + m] = dstate_out != nullptr ? __ldg(dstate_out + (s * D + c) * 3 + m) : 0.f;
    for (int64_t slot = first; slot < nslots; slot += hop) {
        const int s = sequence_of_slot(q, slot, kRun);
        const int2 r = rows_of(q, s);
        const int64_t run = slot - ((int64_t)r.x / kRun + s);
        if (run < 0 || run * kRun >= r.y || !on) continue;
        const int L = r.y, t0 = (int)run * kRun, t1 = min(t0 + kRun, L);
        const int64_t at = (int64_t)r.x * D + c, own = ((int64_t)s * D + c) * 3;
        Pair xw[4][2], zw[4][2];  // x_{t-3} .. x_t and dz_{t-3} .. dz_t
        for (int m = 0; m < 3; ++m) {
            const int t = t0 - 3 + m;
            if (t >= 0) load4<T>(xw[m + 1], x + at + (int64_t)t * D);
            else if (state != nullptr) load_state(xw[m + 1], state + own, t + 3);
            else xw[m + 1][0] = xw[m + 1][1] = both(0.f);
            zw[m + 1][0] = zw[m + 1][1] = both(0.f);
        }
        for (int t = t0; t < t1 + 3; ++t) {
            for (int m = 0; m < 3; ++m)
                for (int e = 0; e < 2; ++e) {
                    xw[m][e] = xw[m + 1][e];
                    zw[m][e] = zw[m + 1][e];
                }
            zw[3][0] = zw[3][1] = both(0.f);
            if (t < L) {
                Pair up[2];
                load4<T>(xw[3], x + at + (int64_t)t * D);
                load4<T>(up, dy + at + (int64_t)t * D);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const Pair z = fma(w[3][e], xw[3][e], fma(w[2][e], xw[2][e], fma(w[1][e], xw[1][e], fma(w[0][e], xw[0][e], b[e]))));
                    Pair slope;
                    activation(z, kSilu, slope);
                    zw[3][e] = up[e] * slope;
                    if (t < t1) {
                        db[e] = db[e] + zw[3][e];
                        for (int k = 0; k < 4; ++k) dw[k][e] = fma(zw[3][e], xw[k][e], dw[k][e]);
                    }
                }
            }
            const int v = t - 3;  // the row whose gradient is now complete
            if (v < t0 && (v >= 0 || dstate == nullptr || t0 > 0)) continue;
            Pair d[2];
#pragma unroll
            for (int e = 0; e < 2; ++e)
                d[e] = fma(w[0][e], zw[3][e], fma(w[1][e], zw[2][e], fma(w[2][e], zw[1][e], w[3][e] * zw[0][e])));
            if (v >= L - 3 && dstate_out != nullptr) {
                Pair o[2];
                load_state(o, dstate_out + own, v - (L - 3));
                d[0] = d[0] + o[0];
                d[1] = d[1] + o[1];
            }
            if (v >= 0) store4(dx + at + (int64_t)v * D, d);
            else store_state(dstate + own, v + 3, d);
        }
    }
    // the block's warps meet in shared memory
    for (int i = 0; i < kSums; ++i) {
        const float2 f = parts(i < 4 ? dw[i][0] : db[0]), g = parts(i < 4 ? dw[i][1] : db[1]);
        __syncthreads();
        tops[warp][lane] = make_float4(f.x, f.y, g.x, g.y);
        __syncthreads();
        if (warp == 0 && on) {
            float4 v = tops[0][lane];
            for (int m = 1; m < kWarps; ++m) {
                const float4 o = tops[m][lane];
                v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
            }
            *reinterpret_cast<float4 *>(part + ((int64_t)blockIdx.x * kSums + i) * D + c) = v;
        }
    }
}

// The blocks' parts of every sum added up, 32 channels x 8 runs of blocks a block, in a fixed order.
__global__ void __launch_bounds__(256)
sum_kernel(const float *__restrict__ part, int nblocks, int D, float *__restrict__ dweight, float *__restrict__ dbias) {
    __shared__ float sm[8][33];
    const int i = blockIdx.y, c = blockIdx.x * 32 + (threadIdx.x & 31), run = threadIdx.x >> 5;
    if (i < 4 ? dweight == nullptr : dbias == nullptr) return;
    float s = 0.f;
    if (c < D)
#pragma unroll 8
        for (int n = run; n < nblocks; n += 8) s += __ldg(part + ((int64_t)n * kSums + i) * D + c);
    sm[run][threadIdx.x & 31] = s;
    __syncthreads();
    if (run == 0 && c < D) {
        s = 0.f;
#pragma unroll
        for (int m = 0; m < 8; ++m) s += sm[m][threadIdx.x & 31];
        if (i < 4) dweight[(int64_t)c * 4 + i] = s;
        else dbias[c] = s;
    }
}

int64_t run_slots(int B, int T, bool packed) {
    return chunk_slots(packed ? (int64_t)T : (int64_t)B * T, B, kRun);
}
// Blocks to a slab of channels: as many as the device holds four to an SM, or as there are runs.
int blocks_x(int B, int T, int D, bool packed) {
    const int64_t slabs = (D + kSlab - 1) / kSlab, need = (run_slots(B, T, packed) + kWarps - 1) / kWarps;
    int64_t most = (int64_t)device_info().sm_count * 4 / slabs;
    if (most < 1) most = 1;
    return (int)(need < most ? need : most);
}

}  // namespace

int64_t workspace(int B, int T, int D, bool packed) {
    return rows_bytes(B, packed) + (int64_t)blocks_x(B, T, D, packed) * kSums * D * (int64_t)sizeof(float);
}

int bwd(const void *dy, const void *x, const float *weight, const float *bias, const float *state, const float *dstate_out,
        void *dx, float *dweight, float *dbias, float *dstate, int B, int T, int D, int dtype, const int32_t *cu, void *ws,
        cudaStream_t st) {
    const bool packed = cu != nullptr;
    Sequences q{B, T, nullptr};
    if (packed) {
        plan_kernel<<<1, kPlanThreads, 0, st>>>(cu, B, T, (int2 *)ws);
        count_launches(1);
        q.rows = (const int2 *)ws;
    }
    float *part = reinterpret_cast<float *>((uint8_t *)ws + rows_bytes(B, packed));
    const int nb = blocks_x(B, T, D, packed);
    const dim3 grid((unsigned)nb, (unsigned)((D + kSlab - 1) / kSlab));
    const int64_t nslots = run_slots(B, T, packed);
    using H16 = __nv_bfloat16;
    if (dtype == GLA_F32)
        bwd_kernel<float><<<grid, kWarps * 32, 0, st>>>((const float *)dy, (const float *)x, weight, bias, state, dstate_out,
                                                        (float *)dx, dstate, part, q, D, nslots);
    else
        bwd_kernel<H16><<<grid, kWarps * 32, 0, st>>>((const H16 *)dy, (const H16 *)x, weight, bias, state, dstate_out,
                                                      (H16 *)dx, dstate, part, q, D, nslots);
    count_launches(1);
    if (dweight != nullptr || dbias != nullptr) {
        sum_kernel<<<dim3((unsigned)((D + 31) / 32), kSums), 256, 0, st>>>(part, nb, D, dweight, dbias);
        count_launches(1);
    }
    return cudaGetLastError() == cudaSuccess ? GLA_OK : GLA_ERR_LAUNCH;
}

}  // namespace convbwd
}  // namespace gla
