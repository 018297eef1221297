// gla_conv_bwd.cu — the gradient of the causal depthwise Conv1d of width 4 with SiLU.
//
// With z_t = bias + sum_k weight[k] x_{t-3+k}, y_t = z_t s(z_t) and s the sigmoid, for each channel of a sequence of L tokens
// (x_{-3} .. x_{-1} is the state before it, x_{L-3} .. x_{L-1} the state behind it):
//     dz_t = dy_t s(z_t) (1 + z_t (1 - s(z_t))) for 0 <= t < L, else 0
//     dx_v = sum_k weight[k] dz_{v+3-k}, plus the gradient of the state behind for v >= L - 3;   v = -3 .. -1: of the state before
//     dweight[k] = sum over tokens of dz_t x_{t-3+k},   dbias = sum over tokens of dz_t
//
// Bound by HBM: x and dy are read and dx is written once.  A warp takes 128 channels, four a lane, of a run of rows of one
// sequence: the last three inputs and the last three dz stay in registers, and the three dz behind the run, which its last rows
// need, are computed again by the next run.  Rows come four at a time, the next four while four are worked on.  Runs are as long as
// makes a few of them for each warp (128 rows for 8 x 2,048 x 4,608, two a warp), see cut().  The warps' sums over tokens stay in
// registers until their last run; the blocks' are added up by a second kernel in a fixed order.
//
// Measured, bf16: 8 x 2,048 x 4,608 102 us (the bytes at the rate of a copy: 67), 1 x 32,768 x 2,048 85 (60); f32 4 x 2,048 x 4,608
// 80 (67).  Nothing is saturated: in bf16 the f32 pipe is busy for 43% of the time, half of the issue slots are used, and HBM is at
// 53%.  What bounds it is how few rows are on their way: they wait in registers, which leave 16 warps of an SM.  Six or eight rows
// at a time, and three blocks of an SM in bf16, are no faster.
#include <type_traits>

#include "gla_act.cuh"
#include "gla_seq.cuh"

GLA_DEFINE_STATUS(conv_bwd)

namespace gla {
namespace convbwd {
namespace {

constexpr int kWarps = 4;     // of a block
constexpr int kSlab = 128;    // channels of a warp
constexpr int kSums = 5;      // dweight[0 .. 3], dbias
constexpr int kRows = 4;      // that come at a time

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const int32_t *__restrict__ cu, int nseq, int T, int2 *rows) {
    if (plan_rows(cu, nseq, T, rows)) record_status(GLA_ERR_DEVICE_ARG);
}

template <typename T> struct Four;  // four channels of one row
template <> struct Four<__nv_bfloat16> {
    using Raw = uint2;
    static constexpr int kPerSm = 4;  // blocks that the registers allow
    static __device__ __forceinline__ Raw none() { return make_uint2(0, 0); }
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
    static constexpr int kPerSm = 3;
    static __device__ __forceinline__ Raw none() { return make_float4(0.f, 0.f, 0.f, 0.f); }
    static __device__ __forceinline__ void open(Pair (&x)[2], Raw w) {
        x[0] = pair(w.x, w.y);
        x[1] = pair(w.z, w.w);
    }
    static __device__ __forceinline__ Raw close(const Pair (&x)[2]) {
        const float2 f = parts(x[0]), g = parts(x[1]);
        return make_float4(f.x, f.y, g.x, g.y);
    }
};
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
__global__ void __launch_bounds__(kWarps * 32, Four<T>::kPerSm)
bwd_kernel(const T *__restrict__ dy, const T *__restrict__ x, const float *__restrict__ weight, const float *__restrict__ bias,
           const float *__restrict__ state, const float *__restrict__ dstate_out, T *__restrict__ dx,
           float *__restrict__ dstate, float *__restrict__ part, Sequences q, int D, int64_t nslots, int run_rows, int per_seq) {
    using Raw = typename Four<T>::Raw;
    __shared__ float4 tops[kWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.y * kSlab + lane * 4;
    const bool on = c < D;
    Pair w[4][2], b[2], dw[4][2], db[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        float4 p = make_float4(0.f, 0.f, 0.f, 0.f), r = p;
        if (on) {
            p = __ldg(reinterpret_cast<const float4 *>(weight + (int64_t)(c + 2 * e) * 4));
            r = __ldg(reinterpret_cast<const float4 *>(weight + (int64_t)(c + 2 * e + 1) * 4));
        }
        w[0][e] = pair(p.x, r.x), w[1][e] = pair(p.y, r.y), w[2][e] = pair(p.z, r.z), w[3][e] = pair(p.w, r.w);
        b[e] = on && bias != nullptr ? pair(__ldg(bias + c + 2 * e), __ldg(bias + c + 2 * e + 1)) : both(0.f);
        db[e] = both(0.f);
#pragma unroll
        for (int k = 0; k < 4; ++k) dw[k][e] = both(0.f);
    }
    const int first = (int)blockIdx.x * kWarps + warp, hop = (int)gridDim.x * kWarps;
    if (on && dstate != nullptr)  // sequences without tokens pass the gradient of their state on
        for (int64_t s = first; s < q.nseq; s += hop)
            if (rows_of(q, (int)s).y == 0)
                for (int m = 0; m < 12; ++m)
                    dstate[(s * D + c) * 3 + m] = dstate_out != nullptr ? __ldg(dstate_out + (s * D + c) * 3 + m) : 0.f;
    for (int64_t slot = first; slot < nslots; slot += hop) {
        int s;
        int64_t run;
        int2 r;
        if (q.rows == nullptr) {
            s = (int)(slot / per_seq);
            run = slot % per_seq;
            r = rows_of(q, s);
        } else {
            s = sequence_of_slot(q, slot, run_rows);
            r = rows_of(q, s);
            run = slot - ((int64_t)r.x / run_rows + s);
        }
        if (run < 0 || run * run_rows >= r.y || !on) continue;
        const int L = r.y, t0 = (int)run * run_rows, t1 = min(t0 + run_rows, L), most = min(t1 + 3, L);
        const int64_t at = (int64_t)r.x * D + c, own = ((int64_t)s * D + c) * 3;
        Pair xw[3][2], zw[3][2];  // x and dz of the three rows before t
#pragma unroll
        for (int m = 0; m < 3; ++m) {
            const int t = t0 - 3 + m;
            xw[m][0] = xw[m][1] = zw[m][0] = zw[m][1] = both(0.f);
            if (t >= 0) Four<T>::open(xw[m], __ldg(reinterpret_cast<const Raw *>(x + at + (int64_t)t * D)));
            else if (state != nullptr) load_state(xw[m], state + own, t + 3);
        }
        Raw nx[kRows], nd[kRows];  // the rows from t on
        auto fetch = [&](int t) {
            const T *px = x + at + (int64_t)t * D, *pd = dy + at + (int64_t)t * D;
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                nx[i] = nd[i] = Four<T>::none();
                if (t + i < most) {
                    nx[i] = __ldg(reinterpret_cast<const Raw *>(px + (int64_t)i * D));
                    nd[i] = __ldg(reinterpret_cast<const Raw *>(pd + (int64_t)i * D));
                }
            }
        };
        // rows t .. t + 3, which complete the gradients of rows t - 3 .. t; inside: all of these are the run's, and none of its
        // sequence's last three
        auto work = [&](int t, auto inside) {
            Raw vx[kRows], vd[kRows];
#pragma unroll
            for (int i = 0; i < kRows; ++i) vx[i] = nx[i], vd[i] = nd[i];
            fetch(t + kRows);
            T *to = dx + at + (int64_t)(t - 3) * D;
#pragma unroll
            for (int i = 0; i < kRows; ++i, to += D) {
                Pair xt[2], dz[2], d[2];
                Four<T>::open(xt, vx[i]);
                Four<T>::open(dz, vd[i]);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const Pair z = fma(w[3][e], xt[e], fma(w[2][e], xw[2][e], fma(w[1][e], xw[1][e], fma(w[0][e], xw[0][e], b[e]))));
                    Pair slope;
                    activation(z, kSilu, slope);
                    dz[e] = dz[e] * slope;
                    if (!inside.value && t + i >= L) dz[e] = both(0.f);
                    if (inside.value || t + i < t1) {
                        db[e] = db[e] + dz[e];
                        dw[0][e] = fma(dz[e], xw[0][e], dw[0][e]);
                        dw[1][e] = fma(dz[e], xw[1][e], dw[1][e]);
                        dw[2][e] = fma(dz[e], xw[2][e], dw[2][e]);
                        dw[3][e] = fma(dz[e], xt[e], dw[3][e]);
                    }
                    d[e] = fma(w[0][e], dz[e], fma(w[1][e], zw[2][e], fma(w[2][e], zw[1][e], w[3][e] * zw[0][e])));
                    xw[0][e] = xw[1][e], xw[1][e] = xw[2][e], xw[2][e] = xt[e];
                    zw[0][e] = zw[1][e], zw[1][e] = zw[2][e], zw[2][e] = dz[e];
                }
                if (inside.value) {
                    *reinterpret_cast<Raw *>(to) = Four<T>::close(d);
                    continue;
                }
                const int v = t + i - 3;
                if (v >= t1 || (v < t0 && (t0 > 0 || dstate == nullptr))) continue;
                if (v >= L - 3 && dstate_out != nullptr) {
                    Pair o[2];
                    load_state(o, dstate_out + own, v - (L - 3));
                    d[0] = d[0] + o[0];
                    d[1] = d[1] + o[1];
                }
                if (v >= 0) *reinterpret_cast<Raw *>(to) = Four<T>::close(d);
                else store_state(dstate + own, v + 3, d);
            }
        };
        fetch(t0);
        for (int t = t0; t < t1 + 3; t += kRows) {
            if (t > t0 && t + kRows <= t1) work(t, std::true_type{});
            else work(t, std::false_type{});
        }
    }
    // the block's warps meet in shared memory
#pragma unroll
    for (int i = 0; i < kSums; ++i) {
        const float2 f = parts(i < 4 ? dw[i < 4 ? i : 0][0] : db[0]), g = parts(i < 4 ? dw[i < 4 ? i : 0][1] : db[1]);
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

// How the work is cut: blocks to a slab of channels, as many as the device holds at once (or there are runs of sixteen rows),
// and rows to a run, a multiple of four.  A packed batch's runs are as many as a few for every warp.  A dense batch's sequences are
// cut into so many alike, rounded down: with between half as many sequences as a slab's warps and as many, each is one run, however
// long, and up to half of the warps have none (bf16 33 x 496 x 4,608 182 us, 32 x 512 103).
struct Cut {
    int blocks, run_rows, per_seq;  // per_seq: runs of a sequence of a dense batch
    int64_t slots;                  // runs, or (packed) slots for them
};
Cut cut(int B, int T, int D, bool packed, int per_sm) {
    const int64_t rows = packed ? (int64_t)T : (int64_t)B * T, slabs = (D + kSlab - 1) / kSlab;
    int64_t most = (int64_t)device_info().sm_count * per_sm / slabs, need = (rows / 16 + B + kWarps - 1) / kWarps;
    if (most < 1) most = 1;
    Cut c{};
    c.blocks = (int)(need < most ? need : most);
    const int64_t warps = (int64_t)c.blocks * kWarps;
    // so many times all warps that 256 rows or fewer come to a run; a packed batch's sequence has a slot more than its rows make
    const int64_t least = rows / 256 + 1 + (packed ? B + 1 : 0), runs = (least + warps - 1) / warps * warps;
    if (packed) {
        c.run_rows = (int)((rows + runs - B - 2) / (runs - B - 1));
    } else {
        const int64_t per = runs / B > 1 ? runs / B : 1;
        c.run_rows = (int)((T + per - 1) / per);
    }
    c.run_rows = (c.run_rows + 3) / 4 * 4;
    if (c.run_rows < 16) c.run_rows = 16;
    c.per_seq = (T + c.run_rows - 1) / c.run_rows;
    c.slots = packed ? chunk_slots(rows, B, c.run_rows) : (int64_t)B * c.per_seq;
    return c;
}
int per_sm(int dtype) { return dtype == GLA_F32 ? Four<float>::kPerSm : Four<__nv_bfloat16>::kPerSm; }

}  // namespace

// bf16's blocks are never fewer than f32's
int64_t workspace(int B, int T, int D, bool packed) {
    return rows_bytes(B, packed) + (int64_t)cut(B, T, D, packed, per_sm(GLA_BF16)).blocks * kSums * D * (int64_t)sizeof(float);
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
    const Cut c = cut(B, T, D, packed, per_sm(dtype));
    const dim3 grid((unsigned)c.blocks, (unsigned)((D + kSlab - 1) / kSlab));
    using H16 = __nv_bfloat16;
    if (dtype == GLA_F32)
        bwd_kernel<float><<<grid, kWarps * 32, 0, st>>>((const float *)dy, (const float *)x, weight, bias, state, dstate_out,
                                                        (float *)dx, dstate, part, q, D, c.slots, c.run_rows, c.per_seq);
    else
        bwd_kernel<H16><<<grid, kWarps * 32, 0, st>>>((const H16 *)dy, (const H16 *)x, weight, bias, state, dstate_out,
                                                      (H16 *)dx, dstate, part, q, D, c.slots, c.run_rows, c.per_seq);
    count_launches(1);
    if (dweight != nullptr || dbias != nullptr) {
        sum_kernel<<<dim3((unsigned)((D + 31) / 32), kSums), 256, 0, st>>>(part, c.blocks, D, dweight, dbias);
        count_launches(1);
    }
    return cudaGetLastError() == cudaSuccess ? GLA_OK : GLA_ERR_LAUNCH;
}

}  // namespace convbwd
}  // namespace gla
