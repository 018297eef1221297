// gla_delta.cu — the gated delta rule: decode step, and the token-by-token kernels that take every type and
// size of its forward and its gradient in f32 arithmetic.
//
// Per chain (sequence, value head), see gla_delta.cuh:
//     u = beta (v - a k S),   S <- a S + k^T u,   o = q S.
// Every column of S (one of the dv) obeys this map by itself: only k, q, a and beta are shared.  So the
// columns of a chain are split over threads, warps and blocks without any exchange between them.
#include <type_traits>

#include "gla_delta.cuh"
#include "gla_pairs.cuh"

GLA_DEFINE_STATUS(delta)

namespace gla {
namespace delta {
namespace {

// ---- decode step ---------------------------------------------------------------------------------------------
//
// Bound by HBM: 8 bytes per state element (read once, written once) against 7 FLOP.  u needs the sum over dk of
// k S before any element can be written, so a block holds its whole slice of the state in registers between the
// two: 8 row groups x up to 16 groups of four columns, kRows rows of 16 bytes a thread.  Both sums (k S and
// q S) are formed from that one read; o = a q S + (q k) u needs no second pass over the new state.
// 1,280 sequences of 16 heads of 96/192 (2.96 GB): 462 us, 6.4 TB/s, 0.94 of a copy's rate.  With sixteen rows a
// thread, and so four blocks to an SM, 484 us; with fewer blocks and their sums through shared memory 540.
constexpr int kStepGroups = 8;    // row groups per block

template <typename T> __device__ __forceinline__ void load4(const T *p, float (&x)[4]);
template <> __device__ __forceinline__ void load4<float>(const float *p, float (&x)[4]) {
    const float4 t = __ldg(reinterpret_cast<const float4 *>(p));
    x[0] = t.x; x[1] = t.y; x[2] = t.z; x[3] = t.w;
}
template <> __device__ __forceinline__ void load4<__nv_bfloat16>(const __nv_bfloat16 *p, float (&x)[4]) {
    const uint2 t = __ldg(reinterpret_cast<const uint2 *>(p));
    x[0] = __uint_as_float(t.x << 16); x[1] = __uint_as_float(t.x & 0xffff0000u);
    x[2] = __uint_as_float(t.y << 16); x[3] = __uint_as_float(t.y & 0xffff0000u);
}
template <typename T> __device__ __forceinline__ void store4(T *p, const float (&x)[4]);
template <> __device__ __forceinline__ void store4<float>(float *p, const float (&x)[4]) {
    *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
template <> __device__ __forceinline__ void store4<__nv_bfloat16>(__nv_bfloat16 *p, const float (&x)[4]) {
    __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
    uint2 t;
    t.x = *reinterpret_cast<uint32_t *>(&a);
    t.y = *reinterpret_cast<uint32_t *>(&b);
    *reinterpret_cast<uint2 *>(p) = t;
}

// Blocks per SM: the more of them, the more bytes in flight (five hold 123 KB of a 96 x 192 state); the registers of
// kRows rows set the number.
constexpr int step_per_sm(int rows) { return rows <= 8 ? 7 : rows <= 12 ? 5 : rows <= 16 ? 4 : 2; }

template <typename T, int kRows>
__global__ void __launch_bounds__(kStepGroups * 16, step_per_sm(kRows))
delta_step_kernel(const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v, const void *__restrict__ g,
                  const void *__restrict__ beta, int gate_f32, float *__restrict__ state,
                  const int32_t *__restrict__ slots, int nslots, T *__restrict__ out, int H, int Hk, int dk, int dv,
                  int ncg, int nslices) {
    extern __shared__ __align__(16) float sm[];
    float *red = sm;                                 // [2][kStepGroups][4 ncg], read and written by float4: first
    float *redqk = red + 2 * kStepGroups * 4 * ncg;  // [kStepGroups]
    float *ks = redqk + kStepGroups, *qs = ks + dk;  // [dk] each
    const unsigned chain32 = blockIdx.x / (unsigned)nslices;  // n * H + h
    const int slice = (int)(blockIdx.x % (unsigned)nslices);
    const int64_t chain = chain32, n = chain32 / (unsigned)H;
    const int h = (int)(chain32 % (unsigned)H);
    const int64_t kchain = n * Hk + h / (H / Hk);
    const int tid = threadIdx.x, cg = tid % ncg, rg = tid / ncg;
    const int col = (slice * ncg + cg) * 4;
    const bool live = col < dv;
    int64_t page = chain;
    if (slots != nullptr) {
        const int slot = __ldg(slots + n);
        if (slot < 0 || slot >= nslots) {  // padding row (or a bad slot, reported): zero output, no page
            if (slot >= nslots && tid == 0) record_status(GLA_ERR_DEVICE_ARG);
            const float zero[4] = {0.f, 0.f, 0.f, 0.f};
            if (rg == 0 && live) store4(out + chain * dv + col, zero);
            return;
        }
        page = (int64_t)slot * H + h;
    }
    float4 *S = reinterpret_cast<float4 *>(state + page * dk * dv + col);
    const int rowf4 = dv >> 2;
    float4 s[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int r = rg + i * kStepGroups;
        s[i] = r < dk && live ? __ldcs(S + (int64_t)r * rowf4) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int i = tid; i < dk; i += blockDim.x) {
        ks[i] = to_f32(k[kchain * dk + i]);
        qs[i] = to_f32(q[kchain * dk + i]);
    }
    const float a = expf(load_gate<T>(g, chain, gate_f32)), be = load_gate<T>(beta, chain, gate_f32);
    float vv[4] = {0.f, 0.f, 0.f, 0.f};
    if (live) load4<T>(v + chain * dv + col, vv);
    __syncthreads();
    float pk[4] = {0.f, 0.f, 0.f, 0.f}, pq[4] = {0.f, 0.f, 0.f, 0.f}, pqk = 0.f;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int r = rg + i * kStepGroups;
        if (r < dk) {
            const float kr = ks[r], qr = qs[r];
            pk[0] = fmaf(kr, s[i].x, pk[0]); pk[1] = fmaf(kr, s[i].y, pk[1]);
            pk[2] = fmaf(kr, s[i].z, pk[2]); pk[3] = fmaf(kr, s[i].w, pk[3]);
            pq[0] = fmaf(qr, s[i].x, pq[0]); pq[1] = fmaf(qr, s[i].y, pq[1]);
            pq[2] = fmaf(qr, s[i].z, pq[2]); pq[3] = fmaf(qr, s[i].w, pq[3]);
            pqk = fmaf(kr, qr, pqk);
        }
    }
    const int wide = 4 * ncg;
    // with 16 column groups a warp holds two row groups: they meet by shuffle, and half as many sums in shared memory
    int np = kStepGroups, at = rg;
    if (ncg == 16) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            pk[c] += __shfl_xor_sync(0xffffffffu, pk[c], 16);
            pq[c] += __shfl_xor_sync(0xffffffffu, pq[c], 16);
        }
        pqk += __shfl_xor_sync(0xffffffffu, pqk, 16);
        np = kStepGroups / 2;
        at = rg >> 1;
    }
    if (ncg != 16 || (rg & 1) == 0) {
        *reinterpret_cast<float4 *>(red + at * wide + cg * 4) = make_float4(pk[0], pk[1], pk[2], pk[3]);
        *reinterpret_cast<float4 *>(red + (kStepGroups + at) * wide + cg * 4) = make_float4(pq[0], pq[1], pq[2], pq[3]);
        if (cg == 0) redqk[at] = pqk;
    }
    __syncthreads();
    float u[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int j = 0; j < np; ++j) {
        const float4 t = *reinterpret_cast<const float4 *>(red + j * wide + cg * 4);
        u[0] += t.x; u[1] += t.y; u[2] += t.z; u[3] += t.w;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) u[c] = be * (vv[c] - a * u[c]);
    if (!live) return;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int r = rg + i * kStepGroups;
        if (r < dk) {
            const float kr = ks[r];
            __stcs(S + (int64_t)r * rowf4, make_float4(fmaf(a, s[i].x, kr * u[0]), fmaf(a, s[i].y, kr * u[1]),
                                                       fmaf(a, s[i].z, kr * u[2]), fmaf(a, s[i].w, kr * u[3])));
        }
    }
    if (rg == 0) {
        float o[4] = {0.f, 0.f, 0.f, 0.f}, qk = 0.f;
#pragma unroll 4
        for (int j = 0; j < np; ++j) {
            const float4 t = *reinterpret_cast<const float4 *>(red + (kStepGroups + j) * wide + cg * 4);
            o[0] += t.x; o[1] += t.y; o[2] += t.z; o[3] += t.w;
            qk += redqk[j];
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) o[c] = fmaf(a, o[c], qk * u[c]);
        store4(out + chain * dv + col, o);
    }
}

template <typename T>
int launch_step(const T *q, const T *k, const T *v, const void *g, const void *beta, int gate_f32, float *state,
                const int32_t *slots, int nslots, T *out, int N, int H, int Hk, int dk, int dv, cudaStream_t st) {
    // slices of at most 64 columns, as even as they come
    const int nslices = (dv / 4 + 15) / 16, ncg = (dv / 4 + nslices - 1) / nslices;
    const long long blocks = (long long)N * H * nslices;
    if (blocks > 0x7fffffffLL) return GLA_ERR_UNSUPPORTED;
    const size_t bytes = (size_t)(2 * dk + 2 * kStepGroups * 4 * ncg + kStepGroups) * sizeof(float);
    const int rows = (dk + kStepGroups - 1) / kStepGroups;
#define GLA_STEP(R)                                                                                                 \
    delta_step_kernel<T, R><<<(unsigned)blocks, ncg * kStepGroups, bytes, st>>>(q, k, v, g, beta, gate_f32, state,   \
                                                                                slots, nslots, out, H, Hk, dk, dv,  \
                                                                                ncg, nslices)
    if (rows <= 8) GLA_STEP(8);
    else if (rows <= 12) GLA_STEP(12);
    else if (rows <= 16) GLA_STEP(16);
    else GLA_STEP(32);
#undef GLA_STEP
    count_launches(1);
    return cudaGetLastError() == cudaSuccess ? GLA_OK : GLA_ERR_LAUNCH;
}

// ---- token-by-token recurrences -------------------------------------------------------------------------------
//
// A warp owns eight columns, four lanes to a column, and each lane kRpl of its dk rows in registers (rows past dk
// are zero and stay so).  A token costs 3 dk multiply-adds a column and two sums over four lanes, of which the
// chain from token to token is a quarter of dk multiply-adds and one sum: some 100 clocks, which bounds few chains
// (47 us for 256 tokens of two heads of 64/64 in f32); many are bound by the multiply-adds.
// Blocks of tokens of q, k, v and the gates are staged in shared memory in f32, the next block while one is
// computed.  Tokens past a sequence's end are staged as k = q = v = 0, beta = 0, decay 1, which leaves the state as
// it is, so every block runs whole.
constexpr int kCols = 32;     // columns per block of four warps

template <int kRpl> struct Staged {  // one block of tokens
    static constexpr int kTok = kRpl > 32 ? 8 : 16;
    static constexpr int kRow = 4 * (kRpl + 4);  // [4][kRpl + 4]: the lanes' reads meet no bank twice
    float k[kTok][kRow], q[kTok][kRow], v[kTok][kCols], a[kTok], beta[kTok];
};

__device__ __forceinline__ void copy4(float *dst, const float *src, bool has) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                 ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src), "r"(has ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(float *dst, const __nv_bfloat16 *src, bool has) {
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    if (has) load4<__nv_bfloat16>(src, x);
    *reinterpret_cast<float4 *>(dst) = make_float4(x[0], x[1], x[2], x[3]);
}
// rows of [.., dk] of n tokens, zero past dk and past n
template <typename T, int kRpl>
__device__ __forceinline__ void stage_rows(float (*dst)[Staged<kRpl>::kRow], const T *src, int64_t row, int64_t stride, int n,
                                           int dk) {
#pragma unroll
    for (int i = threadIdx.x; i < Staged<kRpl>::kTok * kRpl; i += 128) {
        const int t = i / kRpl, r = i % kRpl * 4;
        const bool has = t < n && r < dk;
        copy4(&dst[t][r / kRpl * (kRpl + 4) + r % kRpl], has ? src + (row + t) * stride + r : src, has);
    }
}
template <typename T, int kRpl>
__device__ __forceinline__ void stage(Staged<kRpl> &to, const Shape &p, const T *q, const T *k, const T *v, int64_t row, int n,
                                      int h, int hk, int col0) {
    stage_rows<T, kRpl>(to.k, k + (int64_t)hk * p.dk, row, (int64_t)p.Hk * p.dk, n, p.dk);
    if (q != nullptr) stage_rows<T, kRpl>(to.q, q + (int64_t)hk * p.dk, row, (int64_t)p.Hk * p.dk, n, p.dk);
    const T *vr = v + (int64_t)h * p.dv + col0;
#pragma unroll
    for (int i = threadIdx.x; i < Staged<kRpl>::kTok * kCols / 4; i += 128) {
        const int t = i / (kCols / 4), c = i % (kCols / 4) * 4;
        const bool has = t < n && col0 + c < p.dv;
        copy4(&to.v[t][c], has ? vr + (row + t) * p.H * p.dv + c : v, has);
    }
}
// the gates of a block's tokens: their loads before a block is computed, their place in shared memory after
struct Gates {
    float a, beta;
    template <typename T>
    __device__ __forceinline__ void load(const Shape &p, const void *g, const void *b, int64_t row, int n, int h) {
        a = 1.f;
        beta = 0.f;
        if ((int)threadIdx.x < n) {
            a = load_gate<T>(g, (row + threadIdx.x) * p.H + h, p.gate_f32);
            beta = load_gate<T>(b, (row + threadIdx.x) * p.H + h, p.gate_f32);
        }
    }
    template <int kRpl> __device__ __forceinline__ void put(Staged<kRpl> &to, int n) const {
        if (threadIdx.x < Staged<kRpl>::kTok) {
            to.a[threadIdx.x] = (int)threadIdx.x < n ? expf(a) : 1.f;
            to.beta[threadIdx.x] = beta;
        }
    }
};
__device__ __forceinline__ float sum4(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    return x + __shfl_xor_sync(0xffffffffu, x, 2);
}
// Four lanes with four parts each (one to a token): lane sub gets the sum of part sub.
__device__ __forceinline__ float sum4_of(const float (&x)[4], int sub) {
    const bool odd = sub & 1, high = sub & 2;
    const float a = (odd ? x[1] : x[0]) + __shfl_xor_sync(0xffffffffu, odd ? x[0] : x[1], 1);
    const float b = (odd ? x[3] : x[2]) + __shfl_xor_sync(0xffffffffu, odd ? x[2] : x[3], 1);
    return (high ? b : a) + __shfl_xor_sync(0xffffffffu, high ? a : b, 2);
}
// two pairs of a staged row
struct Pairs2 { Pair a, b; };
__device__ __forceinline__ Pairs2 pairs_at(const float4 *row, int i) {
    const ulonglong2 t = reinterpret_cast<const ulonglong2 *>(row)[i];
    return {{t.x}, {t.y}};
}
// this lane's part of a row times its part of the state
template <int kRpl> __device__ __forceinline__ float dot(const float4 *row, const Pair (&S)[kRpl / 2]) {
    Pair x = both(0.f), y = both(0.f);
#pragma unroll
    for (int i = 0; i < kRpl / 4; ++i) {
        const Pairs2 r = pairs_at(row, i);
        x = fma(r.a, S[2 * i], x);
        y = fma(r.b, S[2 * i + 1], y);
    }
    return total(x + y);
}
// S = a S + u row
template <int kRpl> __device__ __forceinline__ void update(Pair (&S)[kRpl / 2], Pair a, Pair u, const float4 *row) {
#pragma unroll
    for (int i = 0; i < kRpl / 4; ++i) {
        const Pairs2 r = pairs_at(row, i);
        S[2 * i] = fma(a, S[2 * i], r.a * u);
        S[2 * i + 1] = fma(a, S[2 * i + 1], r.b * u);
    }
}
// S = S + u row
template <int kRpl> __device__ __forceinline__ void add(Pair (&S)[kRpl / 2], Pair u, const float4 *row) {
#pragma unroll
    for (int i = 0; i < kRpl / 4; ++i) {
        const Pairs2 r = pairs_at(row, i);
        S[2 * i] = fma(r.a, u, S[2 * i]);
        S[2 * i + 1] = fma(r.b, u, S[2 * i + 1]);
    }
}

// Who a thread is, and its part of a state [dk][dv].
template <int kRpl> struct Lane {
    int s, h, hk, col0, sub, c;
    bool live;
    int64_t chain;
    __device__ __forceinline__ Lane(const Shape &p) {
        s = blockIdx.x / p.H;
        h = blockIdx.x % p.H;
        hk = h / p.group();
        col0 = blockIdx.y * kCols;
        const int lane = threadIdx.x & 31;
        sub = lane & 3;
        c = (threadIdx.x >> 5) * 8 + (lane >> 2);
        live = col0 + c < p.dv;
        chain = ((int64_t)s * p.H + h) * p.dk * p.dv + col0 + c;
    }
    __device__ __forceinline__ void load(Pair (&S)[kRpl / 2], const float *from, const Shape &p) const {
#pragma unroll
        for (int i = 0; i < kRpl / 2; ++i) {
            const int row = sub * kRpl + 2 * i;  // dk is even: a pair is whole or absent
            const bool has = from != nullptr && live && row < p.dk;
            S[i] = has ? pair(from[chain + (int64_t)row * p.dv], from[chain + (int64_t)(row + 1) * p.dv]) : both(0.f);
        }
    }
    __device__ __forceinline__ void store(float *to, const Pair (&S)[kRpl / 2], const Shape &p) const {
#pragma unroll
        for (int i = 0; i < kRpl / 2; ++i) {
            const int row = sub * kRpl + 2 * i;
            if (live && row < p.dk) {
                const float2 f = parts(S[i]);
                to[(int64_t)row * p.dv] = f.x;
                to[(int64_t)(row + 1) * p.dv] = f.y;
            }
        }
    }
};

// Forward: out (or, for the gradient, the residuals r = v - a k S in f32 and the state before every 64th token).
template <typename T, int kRpl, bool kResid>
__global__ void __launch_bounds__(128)
delta_rec_fwd_kernel(Shape p, const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v,
                     const void *__restrict__ g, const void *__restrict__ beta, const float *__restrict__ h0,
                     T *__restrict__ out, float *__restrict__ hT, float *__restrict__ resid, float *__restrict__ states) {
    using St = Staged<kRpl>;
    constexpr int kTok = St::kTok;
    __shared__ __align__(16) St sm[2];
    const Lane<kRpl> ln(p);
    SeqRange r;
    const bool good = good_sequence(p, ln.s, r);
    if (!good) {
        r.start = r.len = 0;
        if (threadIdx.x == 0) record_status(GLA_ERR_DEVICE_ARG);
    }
    if (p.rows != nullptr && ln.h == 0 && blockIdx.y == 0 && threadIdx.x < 32) {  // no later kernel asks for the span
        const int start = good ? (int)r.start : end_before(p, ln.s);
        if (threadIdx.x == 0) p.rows[ln.s] = make_int2(start, (int)r.len);
    }
    Pair S[kRpl / 2];
    ln.load(S, h0, p);
    const int64_t slot0 = r.start / 64 + ln.s;
    const auto count = [&](int64_t t0) { return (int)(r.len - t0 < kTok ? max(r.len - t0, (int64_t)0) : kTok); };
    Gates gates;
    const T *qq = kResid ? nullptr : q;
    if (r.len > 0) {
        gates.load<T>(p, g, beta, r.start, count(0), ln.h);
        stage<T, kRpl>(sm[0], p, qq, k, v, r.start, count(0), ln.h, ln.hk, ln.col0);
        gates.put(sm[0], count(0));
    }
    for (int64_t t0 = 0; t0 < r.len; t0 += kTok) {
        const St &cur = sm[(t0 / kTok) & 1];
        St &next = sm[(t0 / kTok + 1) & 1];
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
        const int ahead = count(t0 + kTok);
        const int64_t row = r.start + t0;
        if (ahead > 0) {
            gates.load<T>(p, g, beta, row + kTok, ahead, ln.h);
            stage<T, kRpl>(next, p, qq, k, v, row + kTok, ahead, ln.h, ln.hk, ln.col0);
        }
        if (kResid && (t0 & 63) == 0)
            ln.store(states + ((slot0 + t0 / 64) * p.H + ln.h) * p.dk * p.dv + ln.col0 + ln.c, S, p);
#pragma unroll 1
        for (int t = 0; t < kTok; t += 4) {
            float x[4];  // q S, summed over the lanes once for the four tokens: off the chain from token to token
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float4 *kt = reinterpret_cast<const float4 *>(cur.k[t + u] + ln.sub * (kRpl + 4));
                const float a = cur.a[t + u];
                const float res = cur.v[t + u][ln.c] - a * sum4(dot<kRpl>(kt, S));
                update<kRpl>(S, both(a), both(cur.beta[t + u] * res), kt);
                x[u] = kResid ? res : dot<kRpl>(reinterpret_cast<const float4 *>(cur.q[t + u] + ln.sub * (kRpl + 4)), S);
            }
            // this lane writes token t + sub of its column
            const float keep = kResid ? (ln.sub & 2 ? (ln.sub & 1 ? x[3] : x[2]) : (ln.sub & 1 ? x[1] : x[0])) : sum4_of(x, ln.sub);
            const int64_t tok = t0 + t + ln.sub;
            if (tok < r.len && ln.live) {
                const int64_t at = ((r.start + tok) * p.H + ln.h) * p.dv + ln.col0 + ln.c;
                if (kResid) resid[at] = keep;
                else out[at] = from_f32<T>(keep);
            }
        }
        if (ahead > 0) gates.put(next, ahead);
    }
    if (hT != nullptr) ln.store(hT + ln.chain, S, p);
}

// Backward in time.  dS is the gradient with respect to the state after token t:
//     dS += q^T do,  y = k dS,  dv = beta y,  dS <- a (dS - k^T dv).
// Writes dv, y (f32) and dS at the end of every 64 tokens of a sequence, before the token's own q^T do.
template <typename T, int kRpl>
__global__ void __launch_bounds__(128)
delta_rec_bwd_kernel(Shape p, const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ dout,
                     const void *__restrict__ g, const void *__restrict__ beta, const float *__restrict__ dhT,
                     T *__restrict__ dv, float *__restrict__ ys, float *__restrict__ states, float *__restrict__ dh0) {
    using St = Staged<kRpl>;
    constexpr int kTok = St::kTok;
    __shared__ __align__(16) St sm[2];
    const Lane<kRpl> ln(p);
    const SeqRange r = rows_of(p, ln.s);
    Pair S[kRpl / 2];
    ln.load(S, dhT, p);
    const int64_t slot0 = r.start / 64 + ln.s, last = r.len > 0 ? (r.len - 1) / kTok * kTok : -1;
    Gates gates;
    if (last >= 0) {
        const int n = (int)(r.len - last);
        gates.load<T>(p, g, beta, r.start + last, n, ln.h);
        stage<T, kRpl>(sm[(last / kTok) & 1], p, q, k, dout, r.start + last, n, ln.h, ln.hk, ln.col0);
        gates.put(sm[(last / kTok) & 1], n);
    }
    for (int64_t t0 = last; t0 >= 0; t0 -= kTok) {
        const St &cur = sm[(t0 / kTok) & 1];
        St &next = sm[(t0 / kTok + 1) & 1];
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
        const int64_t row = r.start + t0;
        if (t0 > 0) {  // every block before the last is whole
            gates.load<T>(p, g, beta, row - kTok, kTok, ln.h);
            stage<T, kRpl>(next, p, q, k, dout, row - kTok, kTok, ln.h, ln.hk, ln.col0);
        }
        if (((t0 + kTok) & 63) == 0 || t0 == last)
            ln.store(states + ((slot0 + t0 / 64) * p.H + ln.h) * p.dk * p.dv + ln.col0 + ln.c, S, p);
#pragma unroll 1
        for (int t = kTok - 4; t >= 0; t -= 4) {
            float keep = 0.f, b = 0.f;
#pragma unroll
            for (int u = 3; u >= 0; --u) {
                const float4 *kt = reinterpret_cast<const float4 *>(cur.k[t + u] + ln.sub * (kRpl + 4));
                const float a = cur.a[t + u], be = cur.beta[t + u];
                add<kRpl>(S, both(cur.v[t + u][ln.c]), reinterpret_cast<const float4 *>(cur.q[t + u] + ln.sub * (kRpl + 4)));
                const float y = sum4(dot<kRpl>(kt, S));
                update<kRpl>(S, both(a), both(-a * (be * y)), kt);
                if (ln.sub == u) {
                    keep = y;
                    b = be;
                }
            }
            const int64_t tok = t0 + t + ln.sub;
            if (tok < r.len && ln.live) {
                const int64_t at = ((r.start + tok) * p.H + ln.h) * p.dv + ln.col0 + ln.c;
                ys[at] = keep;
                dv[at] = from_f32<T>(b * keep);
            }
        }
        if (t0 > 0) gates.put(next, kTok);
    }
    if (dh0 != nullptr) ln.store(dh0 + ln.chain, S, p);
}

// ---- gradient of the shared inputs ------------------------------------------------------------------------------
//
// Given the residuals r, the y of the backward recurrence and, for a chunk of 64 tokens, the state S0 before it
// and the gradient dS1 after it, everything else is local to the chunk.  With D_ij the decay from token j to i,
// c_i from the chunk's start to i, d_j from j to its end and kappa = K K^T:
//     R_ij = beta_j D_ij (do_i . r_j), j <= i        N_ij = -beta_i beta_j D_ij (y_i . r_j), j < i
//     dq_i = c_i do_i S0^T + sum_j R_ij k_j
//     dk_i = d_i beta_i r_i dS1^T - c_i beta_i y_i S0^T + sum_j (R_ji q_j + (N_ij + N_ji) k_j)
//     dbeta_i = y_i . r_i
//     dg_l = sum_{j < l <= i} (R_ij q_i.k_j + N_ij kappa_ij) + sum_{i >= l} w_i + sum_{j < l} x_j + c_63 <S0, dS1>
// where w_i = q_i . (c_i do_i S0^T) - k_i . (c_i beta_i y_i S0^T) and x_j = k_j . (d_j beta_j r_j dS1^T): each term of
// the loss crosses the decay of token l if it starts before l and is read at or after it.
constexpr int kG = 64;        // chunk of the gradient
constexpr int kGP = kG + 1;

struct Tiles {
    float (*a)[kG + 4];
    float (*b)[kG + 4];
};

// f(i, n, sum_k fa(i, k) fb(k, n)) for i < 64 and n < N, 4 x 4 a thread; 256 threads, all of them call f for
// whole micro-tiles (n >= N included, with a zero sum).
template <class FA, class FB, class F>
__device__ __forceinline__ void tile_product(Tiles sm, int N, int K, FA fa, FB fb, F f) {
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int n0 = 0; n0 < N; n0 += kG) {
        float acc[4][4] = {};
        for (int k0 = 0; k0 < K; k0 += 16) {
            __syncthreads();
            for (int e = threadIdx.x; e < 16 * kG; e += 256) {
                const int i = e >> 4, kk = e & 15;
                sm.a[kk][i] = k0 + kk < K ? fa(i, k0 + kk) : 0.f;
            }
            for (int e = threadIdx.x; e < 16 * kG; e += 256) {
                const int kk = e >> 6, n = e & 63;
                sm.b[kk][n] = k0 + kk < K && n0 + n < N ? fb(k0 + kk, n0 + n) : 0.f;
            }
            __syncthreads();
#pragma unroll
            for (int kk = 0; kk < 16; ++kk) {
                const float4 x = *reinterpret_cast<const float4 *>(&sm.a[kk][ty * 4]);
                const float4 y = *reinterpret_cast<const float4 *>(&sm.b[kk][tx * 4]);
                const float xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(xs[i], ys[j], acc[i][j]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) f(ty * 4 + i, n0 + tx * 4 + j, i, acc[i][j]);
    }
    __syncthreads();
}

// to[i] = the sum over the 16 threads of a row of part[i]: one writer a row, a fixed order.
__device__ __forceinline__ void row_sums(float *to, float (&part)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float x = part[i];
        for (int m = 8; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
        if ((threadIdx.x & 15) == 0) to[(threadIdx.x >> 4) * 4 + i] += x;
        part[i] = 0.f;
    }
}

template <typename T>
__global__ void __launch_bounds__(256)
delta_grad_simt_kernel(Shape p, const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ dout,
                       const void *__restrict__ g, const void *__restrict__ beta, const float *__restrict__ resid,
                       const float *__restrict__ ys, const float *__restrict__ s0, const float *__restrict__ ds1,
                       T *__restrict__ dq, T *__restrict__ dk, void *__restrict__ dg, void *__restrict__ dbeta) {
    extern __shared__ __align__(16) float sm[];
    const int slot = (int)(blockIdx.x / (unsigned)p.Hk), hk = (int)(blockIdx.x % (unsigned)p.Hk);
    ChunkAt at;
    if (!chunk_of_slot<kG>(slot, p, at)) return;
    const int L = at.len, dkk = p.dk, dvv = p.dv, tid = threadIdx.x;
    float *kap = sm, *qk = kap + kG * kGP, *R = qk + kG * kGP, *Nm = R + kG * kGP;  // [64][65] each
    float *aq = Nm + kG * kGP, *ak = aq + kG * dkk;                                 // [64][dk] each
    float *al = ak + kG * dkk, *be = al + kG, *c = be + kG, *d = c + kG, *w = d + kG, *x = w + kG, *rs = x + kG,
          *cs = rs + kG, *part = cs + kG;                                            // [64] each, part [8]
    Tiles tl{reinterpret_cast<float(*)[kG + 4]>(part + 8), reinterpret_cast<float(*)[kG + 4]>(part + 8 + 16 * (kG + 4))};
    const T *kr = k + (at.row * p.Hk + hk) * dkk, *qr = q + (at.row * p.Hk + hk) * dkk;
    const int64_t kst = (int64_t)p.Hk * dkk, vst = (int64_t)p.H * dvv;
    auto K = [&](int i, int n) { return i < L ? to_f32(kr[i * kst + n]) : 0.f; };
    auto Q = [&](int i, int n) { return i < L ? to_f32(qr[i * kst + n]) : 0.f; };
    for (int i = tid; i < 2 * kG * dkk; i += 256) aq[i] = 0.f;  // aq and ak
    tile_product(tl, kG, dkk, K, [&](int kk, int n) { return K(n, kk); },
                 [&](int i, int n, int, float s) { kap[i * kGP + n] = s; });
    tile_product(tl, kG, dkk, Q, [&](int kk, int n) { return K(n, kk); },
                 [&](int i, int n, int, float s) { qk[i * kGP + n] = s; });
    for (int h = hk * p.group(); h < (hk + 1) * p.group(); ++h) {
        const int64_t vat = (at.row * p.H + h) * dvv, sat = ((int64_t)slot * p.H + h) * dkk * dvv;
        const T *dor = dout + vat;
        const float *rr = resid + vat, *yr = ys + vat, *S0 = s0 + sat, *S1 = ds1 + sat;
        auto DO = [&](int i, int n) { return i < L ? to_f32(dor[i * vst + n]) : 0.f; };
        auto RR = [&](int i, int n) { return i < L ? rr[i * vst + n] : 0.f; };
        auto Y = [&](int i, int n) { return i < L ? yr[i * vst + n] : 0.f; };
        __syncthreads();
        if (tid < kG) {
            al[tid] = tid < L ? expf(load_gate<T>(g, (at.row + tid) * p.H + h, p.gate_f32)) : 1.f;
            be[tid] = tid < L ? load_gate<T>(beta, (at.row + tid) * p.H + h, p.gate_f32) : 0.f;
            w[tid] = x[tid] = 0.f;
        }
        __syncthreads();
        if (tid < kG) {  // column tid of D as running products of the decays: no difference of logarithms
            float f = 0.f;
            for (int i = 0; i < kG; ++i) {
                f = i == tid ? 1.f : f * al[i];
                R[i * kGP + tid] = Nm[i * kGP + tid] = f;
            }
            d[tid] = f;
        } else if (tid == kG) {
            float f = 1.f;
            for (int i = 0; i < kG; ++i) c[i] = f *= al[i];
        }
        float rp[4] = {};
        tile_product(tl, kG, dvv, DO, [&](int kk, int n) { return RR(n, kk); }, [&](int i, int n, int, float s) {
            R[i * kGP + n] = n <= i ? R[i * kGP + n] * be[n] * s : 0.f;
        });
        tile_product(tl, kG, dvv, Y, [&](int kk, int n) { return RR(n, kk); }, [&](int i, int n, int, float s) {
            Nm[i * kGP + n] = n < i ? -(Nm[i * kGP + n] * be[n] * be[i]) * s : 0.f;
            if (n == i && i < L) store_gate<T>(dbeta, (at.row + i) * p.H + h, p.gate_f32, s);
        });
        auto S0T = [&](int kk, int n) { return S0[(int64_t)n * dvv + kk]; };
        tile_product(tl, dkk, dvv, DO, S0T, [&](int i, int n, int m, float s) {
            if (n < dkk) {
                s *= c[i];
                aq[i * dkk + n] += s;
                rp[m] = fmaf(Q(i, n), s, rp[m]);
            }
        });
        tile_product(tl, dkk, dvv, Y, S0T, [&](int i, int n, int m, float s) {
            if (n < dkk) {
                s *= -c[i] * be[i];
                ak[i * dkk + n] += s;
                rp[m] = fmaf(K(i, n), s, rp[m]);
            }
        });
        row_sums(w, rp);
        tile_product(tl, dkk, dvv, RR, [&](int kk, int n) { return S1[(int64_t)n * dvv + kk]; },
                     [&](int i, int n, int m, float s) {
                         if (n < dkk) {
                             s *= d[i] * be[i];
                             ak[i * dkk + n] += s;
                             rp[m] = fmaf(K(i, n), s, rp[m]);
                         }
                     });
        row_sums(x, rp);
        tile_product(tl, dkk, kG, [&](int i, int kk) { return R[i * kGP + kk]; }, K,
                     [&](int i, int n, int, float s) { if (n < dkk) aq[i * dkk + n] += s; });
        tile_product(tl, dkk, kG, [&](int i, int kk) { return R[kk * kGP + i]; }, Q,
                     [&](int i, int n, int, float s) { if (n < dkk) ak[i * dkk + n] += s; });
        tile_product(tl, dkk, kG, [&](int i, int kk) { return Nm[i * kGP + kk] + Nm[kk * kGP + i]; }, K,
                     [&](int i, int n, int, float s) { if (n < dkk) ak[i * dkk + n] += s; });
        float inner = 0.f;
        for (int i = tid; i < dkk * dvv; i += 256) inner = fmaf(S0[i], S1[i], inner);
        for (int m = 16; m > 0; m >>= 1) inner += __shfl_xor_sync(0xffffffffu, inner, m);
        if ((tid & 31) == 0) part[tid >> 5] = inner;
        if (tid < kG) {  // row and column sums of z_ij = R_ij q_i.k_j + N_ij kappa_ij over j < i
            float a = 0.f, b = 0.f;
            for (int j = 0; j < kG; ++j) {
                if (j < tid) a += R[tid * kGP + j] * qk[tid * kGP + j] + Nm[tid * kGP + j] * kap[tid * kGP + j];
                if (j > tid) b += R[j * kGP + tid] * qk[j * kGP + tid] + Nm[j * kGP + tid] * kap[j * kGP + tid];
            }
            rs[tid] = a;
            cs[tid] = b;
        }
        __syncthreads();
        if (tid < L) {
            float f = 0.f;
            for (int m = 0; m < 8; ++m) f += part[m];
            f *= c[kG - 1];
            for (int m = 0; m < tid; ++m) f += (cs[m] - rs[m]) + x[m];
            for (int m = tid; m < kG; ++m) f += w[m];
            store_gate<T>(dg, (at.row + tid) * p.H + h, p.gate_f32, f);
        }
    }
    __syncthreads();
    for (int i = tid; i < L * dkk; i += 256) {
        const int t = i / dkk, n = i % dkk;
        dq[(at.row + t) * kst + (int64_t)hk * dkk + n] = from_f32<T>(aq[i]);
        dk[(at.row + t) * kst + (int64_t)hk * dkk + n] = from_f32<T>(ak[i]);
    }
}

size_t grad_simt_smem(int dk) {
    return (size_t)(4 * kG * kGP + 2 * kG * dk + 8 * kG + 8 + 2 * 16 * (kG + 4)) * sizeof(float);
}

int check_launch(int n) {
    count_launches(n);
    return cudaGetLastError() == cudaSuccess ? GLA_OK : GLA_ERR_LAUNCH;
}

// rows of the state a lane holds: a quarter of dk, rounded up to what the kernels are built for; bf16 comes here with dk
// above 128 alone
#define GLA_BY_ROWS(T, dk, CALL)                                     \
    do {                                                             \
        if constexpr (!std::is_same<T, float>::value) { CALL(64); }  \
        else if (dk <= 32) { CALL(8); }                              \
        else if (dk <= 64) { CALL(16); }                             \
        else if (dk <= 96) { CALL(24); }                             \
        else if (dk <= 128) { CALL(32); }                            \
        else { CALL(64); }                                           \
    } while (0)

// out null: the residuals and states instead
template <typename T>
int rec_fwd(const Shape &p, const T *q, const T *k, const T *v, const void *g, const void *beta, const float *h0,
            T *out, float *hT, float *resid, float *states, cudaStream_t st) {
    const dim3 grid((unsigned)((long long)p.nseq * p.H), (unsigned)((p.dv + kCols - 1) / kCols));
#define GLA_CALL(R)                                                                                                \
    if (states == nullptr)                                                                                         \
        delta_rec_fwd_kernel<T, R, false><<<grid, 128, 0, st>>>(p, q, k, v, g, beta, h0, out, hT, resid, states);   \
    else                                                                                                           \
        delta_rec_fwd_kernel<T, R, true><<<grid, 128, 0, st>>>(p, q, k, v, g, beta, h0, out, hT, resid, states)
    GLA_BY_ROWS(T, p.dk, GLA_CALL);
#undef GLA_CALL
    return check_launch(1);
}

}  // namespace

size_t simt_bwd_workspace(const Shape &p) {
    const size_t rows = (size_t)total_rows(p) * p.H * p.dv;
    const size_t state = (size_t)chunk_slots(total_rows(p), p.nseq, kG) * p.H * p.dk * p.dv;
    return rows_bytes(p) + 2 * (rows + state) * sizeof(float);
}

template <typename T>
int simt_fwd(const Shape &p, const T *q, const T *k, const T *v, const void *g, const void *beta, const float *h0,
             T *out, float *hT, cudaStream_t st) {
    return rec_fwd<T>(p, q, k, v, g, beta, h0, out, hT, nullptr, nullptr, st);
}

template <typename T>
int simt_bwd(Shape p, const T *q, const T *k, const T *v, const void *g, const void *beta, const T *dout,
             const float *h0, const float *dhT, T *dq, T *dk, T *dv, void *dg, void *dbeta, float *dh0, void *ws,
             cudaStream_t st) {
    const long long rows = total_rows(p), slots = chunk_slots(rows, p.nseq, kG);
    if (slots * p.Hk > 0x7fffffffLL) return GLA_ERR_UNSUPPORTED;
    const size_t state = (size_t)slots * p.H * p.dk * p.dv;
    p.rows = p.cu ? (int2 *)ws : nullptr;
    float *s0 = (float *)((char *)ws + rows_bytes(p)), *ds1 = s0 + state, *resid = ds1 + state, *ys = resid + (size_t)rows * p.H * p.dv;
    int rc = rec_fwd<T>(p, q, k, v, g, beta, h0, nullptr, nullptr, resid, s0, st);
    if (rc != GLA_OK) return rc;
    const dim3 grid((unsigned)((long long)p.nseq * p.H), (unsigned)((p.dv + kCols - 1) / kCols));
#define GLA_CALL(R) \
    delta_rec_bwd_kernel<T, R><<<grid, 128, 0, st>>>(p, q, k, dout, g, beta, dhT, dv, ys, ds1, dh0)
    GLA_BY_ROWS(T, p.dk, GLA_CALL);
#undef GLA_CALL
    rc = check_launch(1);
    if (rc != GLA_OK || rows == 0) return rc;
    const size_t bytes = grad_simt_smem(p.dk);
    if (!allow_smem<delta_grad_simt_kernel<T>>()) return GLA_ERR_LAUNCH;
    delta_grad_simt_kernel<T><<<(unsigned)(slots * p.Hk), 256, bytes, st>>>(p, q, k, dout, g, beta, resid, ys, s0, ds1,
                                                                            dq, dk, dg, dbeta);
    return check_launch(1);
}

template int simt_fwd<float>(const Shape &, const float *, const float *, const float *, const void *, const void *,
                             const float *, float *, float *, cudaStream_t);
template int simt_fwd<__nv_bfloat16>(const Shape &, const __nv_bfloat16 *, const __nv_bfloat16 *, const __nv_bfloat16 *,
                                     const void *, const void *, const float *, __nv_bfloat16 *, float *, cudaStream_t);
template int simt_bwd<float>(Shape, const float *, const float *, const float *, const void *, const void *,
                             const float *, const float *, const float *, float *, float *, float *, void *, void *,
                             float *, void *, cudaStream_t);
template int simt_bwd<__nv_bfloat16>(Shape, const __nv_bfloat16 *, const __nv_bfloat16 *,
                                     const __nv_bfloat16 *, const void *, const void *, const __nv_bfloat16 *,
                                     const float *, const float *, __nv_bfloat16 *, __nv_bfloat16 *, __nv_bfloat16 *,
                                     void *, void *, float *, void *, cudaStream_t);

int decode_step(const void *q, const void *k, const void *v, const void *g, const void *beta, float *state,
                const int32_t *slots, int nslots, void *out, int N, int H, int Hk, int dk, int dv, int dtype,
                int gate_dtype, cudaStream_t st) {
    using B = __nv_bfloat16;
    const int gf = gate_dtype == GLA_F32;
    if (dtype == GLA_F32)
        return launch_step<float>((const float *)q, (const float *)k, (const float *)v, g, beta, gf, state, slots,
                                  nslots, (float *)out, N, H, Hk, dk, dv, st);
    return launch_step<B>((const B *)q, (const B *)k, (const B *)v, g, beta, gf, state, slots, nslots, (B *)out, N, H,
                          Hk, dk, dv, st);
}

}  // namespace delta
}  // namespace gla
