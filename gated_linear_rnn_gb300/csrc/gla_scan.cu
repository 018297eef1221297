// gla_scan.cu — the gated recurrence: forward, gradient and the step for single tokens.
//
//     h_t = a_t h_{t-1} + w_t x_t,   out_t = h_t act(gate_t);   a_t = exp(g_t) or sigmoid(g_t),   w_t = 1 or 1 - a_t
//
// Gradient, backwards in time with D_T = dhT:
//     dh_t = dout_t act(gate_t) + D_t,   D_{t-1} = a_t dh_t,   dh0 = D_0,   dx_t = w_t dh_t,
//     da_t = dh_t (h_{t-1} - x_t) where the input leaks, dh_t h_{t-1} elsewhere,   dg_t = da_t a_t, times 1 - a_t for a sigmoid,
//     dgate_t = dout_t h_t act'(gate_t)
#include "gla_scan_tiles.cuh"

GLA_DEFINE_STATUS(scan)

namespace gla {
namespace scan {

bool tiles_fwd(const Shape &, const Tiles &, const Chain &, const void *, const void *, const void *, const float *, void *, float *,
               float *, int, int, cudaStream_t);
bool tiles_bwd(const Shape &, const Tiles &, const Chain &, const void *, const void *, const void *, const void *, const float *,
               const float *, void *, void *, void *, float *, int, int, cudaStream_t);

namespace {

constexpr int kThreads = 128;  // four channels each
constexpr int kWalked = 8, kWalkedOfMany = 32;  // tokens of a sequence, see walks()

// What has to be there before the others start: the rows and the chunks of a packed batch's sequences of more than `walked`
// tokens, and the words of the chains unset.  32 sequences, a warp's, have their first chunks listed, then their second ones.
__global__ void __launch_bounds__(kPlanThreads)
prepare_kernel(const int32_t *__restrict__ cu, int nseq, int T, int walked, int2 *rows, int2 *tasks, int *ntasks, uint4 *unset, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * kPlanThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kPlanThreads)
        unset[i] = make_uint4(kUnset, kUnset, kUnset, kUnset);
    if (blockIdx.x != 0) return;
    if (plan_rows(cu, nseq, T, rows)) record_status(GLA_ERR_DEVICE_ARG);
    __shared__ int of_warp[kPlanThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int done = 0;  // tasks listed before
    for (int first = 0; first < nseq; first += kPlanThreads) {
        const int s = first + (int)threadIdx.x, len = s < nseq ? rows[s].y : 0;  // the thread's own from plan_rows
        const int chunks = len > walked ? (len + kChunk - 1) / kChunk : 0;
        const int mine = __reduce_add_sync(0xffffffffu, chunks);
        if (lane == 0) of_warp[warp] = mine;
        __syncthreads();
        int at = done;
        for (int w = 0; w < kPlanThreads / 32; ++w) {
            if (w < warp) at += of_warp[w];
            done += of_warp[w];
        }
        for (int c = 0;; ++c) {
            const unsigned have = __ballot_sync(0xffffffffu, chunks > c);
            if (have == 0) break;
            if ((have & (have - 1)) == 0) {  // the rest is one sequence's
                const int who = __ffs(have) - 1, all = __shfl_sync(0xffffffffu, chunks, who), which = first + warp * 32 + who;
                for (int i = c + lane; i < all; i += 32) tasks[at + i - c] = make_int2(which, i);
                break;
            }
            if (chunks > c) tasks[at + __popc(have & ((1u << lane) - 1u))] = make_int2(s, c);
            at += __popc(have);
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) *ntasks = done;
}

// A thread takes four channels of a sequence of `most` tokens at most from its first token to its last, a run's loads at once.
template <typename T, typename TG, int kForm, bool kGate>
__global__ void __launch_bounds__(kThreads)
walk_fwd_kernel(const T *__restrict__ x, const TG *__restrict__ g, const T *__restrict__ gate, const float *__restrict__ h0,
                T *__restrict__ out, float *__restrict__ hT, float *__restrict__ states, Sequences q, int most, int D, int act, int shift,
                unsigned parts_of_row) {
    const int64_t s = (int64_t)(blockIdx.x / parts_of_row) * (kThreads >> shift) + (threadIdx.x >> shift);
    const int d = (int)((blockIdx.x % parts_of_row) << shift | (threadIdx.x & ((1u << shift) - 1u))) * 4;
    if (s >= q.nseq || d >= D) return;
    const int2 r = rows_of(q, (int)s);
    if (r.y > most) return;
    Pair h[2] = {both(0.f), both(0.f)};
    if (h0 != nullptr) load_four(h0 + s * D + d, h);
    for (int t0 = 0; t0 < r.y; t0 += kRun) {
        if (states != nullptr) store_four(states + state_slot(r.x, (int)s, t0) * D + d, h);
        const int n = min(kRun, r.y - t0);
        const int64_t first = (int64_t)(r.x + t0) * D + d;
        FourRaw<T> xs[kRun], zs[kGate ? kRun : 1];
        FourRaw<TG> gs[kRun];
#pragma unroll
        for (int t = 0; t < kRun; ++t)
            if (t < n) {
                const int64_t at = first + (int64_t)t * D;
                gs[t].load(g + at), xs[t].load(x + at);
                if (kGate && out != nullptr) zs[t].load(gate + at);
            }
#pragma unroll
        for (int t = 0; t < kRun; ++t)
            if (t < n) {
                Pair v[2], a[2], z[2], y[2];
                xs[t].open(v), gs[t].open(a);
                if (kGate && out != nullptr) zs[t].open(z);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const Decay c = decay<kForm>(a[e]);
                    h[e] = decayed(c, h[e], input<kForm>(c, v[e]));
                    y[e] = kGate && out != nullptr ? h[e] * activation(z[e], act) : h[e];
                }
                if (out != nullptr) store_four(out + first + (int64_t)t * D, y);
            }
    }
    if (hT != nullptr) store_four(hT + s * D + d, h);
}

// The states of a run of rows from the one before it, then backwards through the run.
template <typename T, typename TG, int kForm, bool kGate>
__global__ void __launch_bounds__(kThreads)
walk_bwd_kernel(const T *__restrict__ x, const TG *__restrict__ g, const T *__restrict__ gate, const T *__restrict__ dout,
                const float *__restrict__ dhT, const float *__restrict__ states, T *__restrict__ dx, TG *__restrict__ dg,
                T *__restrict__ dgate, float *__restrict__ dh0, Sequences q, int most, int D, int act, int shift, unsigned parts_of_row) {
    const int64_t s = (int64_t)(blockIdx.x / parts_of_row) * (kThreads >> shift) + (threadIdx.x >> shift);
    const int d = (int)((blockIdx.x % parts_of_row) << shift | (threadIdx.x & ((1u << shift) - 1u))) * 4;
    if (s >= q.nseq || d >= D) return;
    const int2 r = rows_of(q, (int)s);
    if (r.y > most) return;
    Pair back[2] = {both(0.f), both(0.f)};
    if (dhT != nullptr) load_four(dhT + s * D + d, back);
    for (int c = (r.y + kRun - 1) / kRun - 1; c >= 0; --c) {
        const int n = min(kRun, r.y - c * kRun);
        const int64_t first = (int64_t)(r.x + c * kRun) * D + d;
        Pair h[2], before[kRun][2];
        FourRaw<T> xs[kRun], us[kRun], zs[kGate ? kRun : 1];
        FourRaw<TG> gs[kRun];
        load_four(states + state_slot(r.x, (int)s, c * kRun) * D + d, h);
#pragma unroll
        for (int t = 0; t < kRun; ++t)
            if (t < n) {
                const int64_t at = first + (int64_t)t * D;
                gs[t].load(g + at), xs[t].load(x + at);
            }
#pragma unroll
        for (int t = 0; t < kRun; ++t)
            if (t < n) {
                const int64_t at = first + (int64_t)t * D;
                us[t].load(dout + at);
                if (kGate) zs[t].load(gate + at);
            }
#pragma unroll
        for (int t = 0; t < kRun; ++t)
            if (t < n) {
                Pair v[2], a[2];
                xs[t].open(v), gs[t].open(a);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    before[t][e] = h[e];
                    const Decay k = decay<kForm>(a[e]);
                    h[e] = decayed(k, h[e], input<kForm>(k, v[e]));
                }
            }
#pragma unroll
        for (int t = kRun - 1; t >= 0; --t)
            if (t < n) {
                const int64_t at = first + (int64_t)t * D;
                Pair v[2], a[2], up[2], z[2];
                xs[t].open(v), gs[t].open(a), us[t].open(up);
                if (kGate) zs[t].open(z);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const Decay k = decay<kForm>(a[e]);
                    Pair dh = up[e];
                    if (kGate) {
                        Pair slope;
                        dh = up[e] * activation(z[e], act, slope);
                        z[e] = up[e] * slope * decayed(k, before[t][e], input<kForm>(k, v[e]));
                    }
                    dh = dh + back[e];
                    Pair da = leaks(kForm) ? fma(v[e], both(-1.f), before[t][e]) : before[t][e];
                    da = dh * (da * whole(k));
                    if (!is_log(kForm)) da = da * rest(k);
                    a[e] = da;
                    v[e] = input<kForm>(k, dh);
                    back[e] = decayed(k, dh);
                }
                if (kGate) store_four(dgate + at, z);
                store_four(dg + at, a);
                store_four(dx + at, v);
            }
    }
    if (dh0 != nullptr) store_four(dh0 + s * D + d, back);
}

// One token of N sequences, four channels a thread, 1 << shift threads to a row; a block has a part of 256 >> shift rows.
constexpr int kStepThreads = 256;
template <typename T, typename TG, int kForm, bool kGate>
__global__ void __launch_bounds__(kStepThreads)
step_kernel(const T *__restrict__ x, const TG *__restrict__ g, const T *__restrict__ gate, float *__restrict__ state,
            const int32_t *__restrict__ slots, int nslots, T *__restrict__ out, int N, int D, int shift, unsigned parts, int act) {
    const int64_t n = (int64_t)(blockIdx.x / parts) * (kStepThreads >> shift) + (threadIdx.x >> shift);
    const int c = (int)((blockIdx.x % parts) << shift | (threadIdx.x & ((1u << shift) - 1u))) * 4;
    if (n >= N || c >= D) return;
    int64_t page = n;
    if (slots != nullptr) {
        page = __ldg(slots + n);
        if (page >= nslots) {
            record_status(GLA_ERR_DEVICE_ARG);
            page = -1;
        }
    }
    const int64_t at = n * D + c;
    Pair v[2], d[2], z[2], y[2] = {both(0.f), both(0.f)};
    if (page >= 0) {
        load_four(x + at, v);
        load_four(g + at, d);
        if (kGate) load_four(gate + at, z);
        float4 *const to = reinterpret_cast<float4 *>(state + page * D + c);
        const float4 s = *to;
        const Pair h[2] = {pair(s.x, s.y), pair(s.z, s.w)};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const Decay a = decay<kForm>(d[e]);
            y[e] = decayed(a, h[e], input<kForm>(a, v[e]));
        }
        const float2 p = gla::parts(y[0]), q = gla::parts(y[1]);
        *to = make_float4(p.x, p.y, q.x, q.y);
#pragma unroll
        for (int e = 0; e < 2; ++e)
            if (kGate) y[e] = y[e] * activation(z[e], act);
    }
    store_four(out + at, y);
}

int status() { return cudaGetLastError() == cudaSuccess ? GLA_OK : GLA_ERR_LAUNCH; }

int most_walked(const Shape &p) { return p.cu != nullptr ? kChunk : p.T; }

// How rows of D channels go to blocks of so many threads, four channels each: 1 << shift threads to a row's part.
struct Split {
    int shift;
    int64_t parts, blocks;
};
Split split(int64_t rows, int D, int threads) {
    Split w{};
    while ((1 << w.shift) < threads && (4 << w.shift) < D) ++w.shift;
    const int64_t at_once = threads >> w.shift;
    w.parts = (D + (4 << w.shift) - 1) >> (w.shift + 2);
    w.blocks = (rows + at_once - 1) / at_once * w.parts;
    return w;
}

void walk_fwd(const Shape &p, const void *x, const void *g, const void *gate, const float *h0, void *out, float *hT,
              float *states, int dtype, int g_dtype, const Sequences &q, cudaStream_t st) {
    const Split w = split(p.nseq, p.D, kThreads);
#define GLA_RUN(T, TG, F, G)                                                                                                \
    walk_fwd_kernel<T, TG, F, G><<<(unsigned)w.blocks, kThreads, 0, st>>>(                                                  \
        (const T *)x, (const TG *)g, (const T *)gate, h0, (T *)out, hT, states, q, most_walked(p), p.D, p.act, w.shift,     \
        (unsigned)w.parts)
    GLA_SCAN_DISPATCH(dtype, g_dtype, gate != nullptr, GLA_RUN)
#undef GLA_RUN
    count_launches(1);
}

void walk_bwd(const Shape &p, const void *x, const void *g, const void *gate, const void *dout, const float *dhT,
              const float *states, void *dx, void *dg, void *dgate, float *dh0, int dtype, int g_dtype, const Sequences &q,
              cudaStream_t st) {
    const Split w = split(p.nseq, p.D, kThreads);
#define GLA_RUN(T, TG, F, G)                                                                                                \
    walk_bwd_kernel<T, TG, F, G><<<(unsigned)w.blocks, kThreads, 0, st>>>(                                                  \
        (const T *)x, (const TG *)g, (const T *)gate, (const T *)dout, dhT, states, (T *)dx, (TG *)dg, (T *)dgate, dh0, q,  \
        most_walked(p), p.D, p.act, w.shift, (unsigned)w.parts)
    GLA_SCAN_DISPATCH(dtype, g_dtype, gate != nullptr, GLA_RUN)
#undef GLA_RUN
    count_launches(1);
}

// A call's workspace: the rows of a packed batch's sequences, a counter and a chain for each direction, and (of a gradient that
// is not given them) the states.
struct Layout {
    int64_t tasks, ntasks, counters, chains, states, total;  // (the rows are first)
};
constexpr int64_t kCounterBytes = 256;
bool chained(const Shape &p) { return p.cu != nullptr || p.T > kChunk; }
Layout layout(int op, const Shape &p) {
    Layout l{};
    const int64_t chain = chained(p) ? (chain_floats(p) * (int64_t)sizeof(float) + 255) / 256 * 256 : 0;
    const int dirs = op == GLA_OP_BACKWARD ? 2 : 1;
    l.tasks = rows_bytes(p.nseq, p.cu != nullptr);
    l.ntasks = l.tasks + (p.cu != nullptr ? (slots(p) * (int64_t)sizeof(int2) + 255) / 256 * 256 : 0);
    l.counters = l.ntasks + (p.cu != nullptr ? kCounterBytes : 0);
    l.chains = l.counters + (chain > 0 ? dirs * kCounterBytes : 0);
    l.states = l.chains + dirs * chain;
    l.total = l.states + (op == GLA_OP_BACKWARD ? states_bytes(p) : 0);
    return l;
}
Chain chain_at(const Layout &l, const Shape &p, void *ws, int dir) {
    uint8_t *b = (uint8_t *)ws;
    Chain c;
    c.next = (unsigned *)(b + l.counters + dir * kCounterBytes);
    c.effect = (float *)(b + l.chains + dir * ((chain_floats(p) * (int64_t)sizeof(float) + 255) / 256 * 256));
    c.result = c.effect + places(p) * p.D * 2;
    return c;
}

// A tile has 64 rows, used or not, and its meetings; a walk takes 0.25 us a token (0.4 the gradient's) and no less.  So sequences are
// walked that have kWalked tokens and fewer on average, or kWalkedOfMany where there are tiles for several rounds of the blocks;
// of a packed batch those of up to a tile's rows, and the tiles then take the others, if there are any (a decode step with a
// prompt in it).  Forward and gradient of 16,384 x 2,560 bf16 in us, walked and by tiles: sequences of 17 tokens 63, 134 and 152,
// 260; of 32 61, 126 and 98, 164; of 64 63, 129 and 66, 110; 8 sequences of 32 8, 13 and 4, 5; f32 256 x 32 52, 162 and 92, 146.
// (One rule for both: from 33 to 64 tokens the forward alone would still gain by walking, 5 to 20%, and the gradient lose as much.)
bool walks(const Shape &p) {
    const int64_t rows = total_rows(p), tiles = (int64_t)p.nseq * ((p.D + kSlab - 1) / kSlab);
    return rows <= (int64_t)kWalked * p.nseq ||
           (rows <= (int64_t)kWalkedOfMany * p.nseq && tiles >= 16 * (int64_t)device_info().sm_count);
}

// dirs: how many of the chains are used
Sequences prepare(const Shape &p, const Layout &l, void *ws, int dirs, cudaStream_t st) {
    if (!chained(p)) return {p.nseq, p.T, nullptr};
    uint8_t *b = (uint8_t *)ws;
    const int64_t bytes = l.chains - l.counters + dirs * ((chain_floats(p) * (int64_t)sizeof(float) + 255) / 256 * 256);
    if (p.cu == nullptr) {
        cudaMemsetAsync(b + l.counters, 0xff, (size_t)bytes, st);
        return {p.nseq, p.T, nullptr};
    }
    const int64_t n = bytes / 16, need = (n + 4 * kPlanThreads - 1) / (4 * kPlanThreads);
    const int64_t most = 2 * (int64_t)device_info().sm_count;
    prepare_kernel<<<(unsigned)(need < most ? need : most), kPlanThreads, 0, st>>>(
        p.cu, p.nseq, p.T, walks(p) ? kChunk : 0, (int2 *)ws, (int2 *)(b + l.tasks), (int *)(b + l.ntasks), (uint4 *)(b + l.counters), n);
    count_launches(1);
    return {p.nseq, p.T, (const int2 *)ws};
}

Tiles tiles_of(const Shape &p, const Sequences &q, const Layout &l, void *ws) {
    Tiles t = make_tiles(p, q);
    if (p.cu == nullptr) return t;
    t.walked = walks(p);
    t.tasks = (const int2 *)((uint8_t *)ws + l.tasks);
    t.ntasks = (const int *)((uint8_t *)ws + l.ntasks);
    return t;
}

}  // namespace

int64_t workspace(int op, const Shape &p) { return layout(op, p).total; }

int fwd(const Shape &p, const void *x, const void *g, const void *gate, const float *h0, void *out, float *hT, float *states,
        int dtype, int g_dtype, void *ws, cudaStream_t st) {
    const Layout l = layout(GLA_OP_FORWARD, p);
    const Sequences q = prepare(p, l, ws, 1, st);
    if (walks(p)) {
        walk_fwd(p, x, g, gate, h0, out, hT, states, dtype, g_dtype, q, st);
        if (p.cu == nullptr || p.T <= kChunk) return status();
    }
    if (!tiles_fwd(p, tiles_of(p, q, l, ws), chain_at(l, p, ws, 0), x, g, gate, h0, out, hT, states, dtype, g_dtype, st))
        return GLA_ERR_LAUNCH;
    return status();
}

int bwd(const Shape &p, const void *x, const void *g, const void *gate, const void *dout, const float *h0, const float *dhT,
        const float *states, void *dx, void *dg, void *dgate, float *dh0, int dtype, int g_dtype, void *ws, cudaStream_t st) {
    const Layout l = layout(GLA_OP_BACKWARD, p);
    const Sequences q = prepare(p, l, ws, states == nullptr ? 2 : 1, st);
    float *own = reinterpret_cast<float *>((uint8_t *)ws + l.states);
    const Tiles t = tiles_of(p, q, l, ws);
    if (walks(p)) {
        if (states == nullptr) walk_fwd(p, x, g, nullptr, h0, nullptr, nullptr, own, dtype, g_dtype, q, st);
        walk_bwd(p, x, g, gate, dout, dhT, states != nullptr ? states : own, dx, dg, dgate, dh0, dtype, g_dtype, q, st);
        if (p.cu == nullptr || p.T <= kChunk) return status();
    }
    if (states == nullptr &&
        !tiles_fwd(p, t, chain_at(l, p, ws, 1), x, g, nullptr, h0, nullptr, nullptr, own, dtype, g_dtype, st))
        return GLA_ERR_LAUNCH;
    if (!tiles_bwd(p, t, chain_at(l, p, ws, 0), x, g, gate, dout, dhT, states != nullptr ? states : own, dx, dg, dgate, dh0,
                   dtype, g_dtype, st))
        return GLA_ERR_LAUNCH;
    return status();
}

int step(const void *x, const void *g, const void *gate, float *state, const int32_t *slots, int nslots, void *out, int N,
         int D, int form, int act, int dtype, int g_dtype, cudaStream_t st) {
    const Split w = split(N, D, kStepThreads);
    if (w.blocks > 0x7fffffff) return GLA_ERR_UNSUPPORTED;
    const Shape p{N, 1, D, form, act, nullptr};
#define GLA_RUN(T, TG, F, G)                                                                                                \
    step_kernel<T, TG, F, G><<<(unsigned)w.blocks, kStepThreads, 0, st>>>((const T *)x, (const TG *)g, (const T *)gate, state, \
                                                                       slots, nslots, (T *)out, N, D, w.shift,              \
                                                                       (unsigned)w.parts, act)
    GLA_SCAN_DISPATCH(dtype, g_dtype, gate != nullptr, GLA_RUN)
#undef GLA_RUN
    count_launches(1);
    return status();
}

}  // namespace scan
}  // namespace gla
