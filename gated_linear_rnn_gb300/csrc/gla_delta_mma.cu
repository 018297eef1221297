// gla_delta_mma.cu — the gated delta rule over whole sequences on the tensor cores (bf16 inputs).
//
// A chunk of C = 32 tokens with D_ij the decay from token j to token i (1 for i = j), c_i the decay from the
// chunk's start to token i, d_j from token j to its end, kappa_ij = k_i . k_j and L_ij = D_ij kappa_ij (j < i):
//     X = V - diag(c) K S0                       what the chunk's tokens would write into S0 alone
//     R = (I + L diag(beta))^-1 X                the residuals v_t - a_t k_t S_{t-1}
//     O = diag(c) Q S0 + (D o Q K^T) diag(beta) R
//     S1 = c_31 S0 + K^T diag(d beta) R
//
// Two kernels.  delta_prep_kernel forms, for every chunk and head at once, what does not depend on the state:
// M = (I + L diag(beta))^-1 by substitution in f32, P = D o Q K^T diag(beta), c and d beta.  delta_fwd_kernel
// then walks each chain.  All of its products leave the columns of S (the dv dimension) apart, so a warp owns 16
// columns for the whole walk and meets no other warp: it keeps S^T in registers as the f32 accumulators of
// mma.sync m16n8k16, whose layout is also that of the A operand, and every product has the form
// (16 columns x n) = (16 columns x k)(k x n) with the B operand from shared memory:
//     Y = S^T K^T,  X^T = V^T - Y diag(c),  R^T = X^T M^T,  O^T = S^T Q^T diag(c) + R^T P^T,
//     S^T = c_31 S^T + (R^T diag(d beta)) K.
// A step of a chain is three products long, without a barrier or a trip through memory between them; that, and
// not the rate of the tensor cores, is what a walk over a long sequence is made of.  mma.sync runs at 1,020 multiply-adds
// a clock and SM (measured), a quarter of tcgen05's rate.  A walk on tcgen05 could keep S^T, X^T and R^T as A operands in
// TMEM, through the registers between any two products for their scaling and splitting; it has not been built.
//
// Precision: q, k and v are bf16 and so exact as operands.  S, X, M and R are f32 values; where a product with
// them reaches the state, each is taken as two bf16 parts, hi + lo, whose sum holds 16 bits of it (2^-17 relative);
// M X takes three products, the others two.  hT is within 6e-6 of its norm, where f32 arithmetic alone would leave 2e-7.
// O, itself rounded to bf16, takes the hi parts alone: 3e-3 of its norm, where its own rounding leaves 1.7e-3.
//
// A warpgroup of its own, four threads to a row, fetches the rows of K, Q and V by 16-byte asynchronous copies (zero
// past a sequence's end, so a short chunk is computed like a whole one) and the chunk's M, P, c and d beta by one
// bulk copy into a ring of stages; a row's stride is an odd number of 16-byte units, so that ldmatrix meets no bank
// twice.  (One warp in its place was what the walk waited for: 360 us against 246 at the sizes below.)
//
// Eight sequences of 2,048 tokens, 16 heads of 96/192: 212 us, preparation 45 and walk 161.  That is 1.5 TB/s of the
// inputs and outputs: the walk keeps mma.sync's pipe 71% busy with one block of 128 registers a thread on an SM, and
// a quarter of its warps; HBM would need 46 us.
//
// A third and a fourth kernel serve few long chains, cut into segments (segment_tokens): a walk over each segment's
// map S -> M S + N, delta_join_kernel over the maps, then the walk of every segment from its own state.  32,768
// tokens of 16 heads: 865 us (preparation 80, maps 447, join 47, walk 281), against 1,416 as whole chains.
#include "gla_delta_mma.cuh"

GLA_DEFINE_STATUS(delta_mma)

namespace gla {
namespace delta {
namespace {

// ---- what does not depend on the state -----------------------------------------------------------------------
//
// One warp per chunk and value head.  K K^T and Q K^T by mma.sync (their inputs are exact, their sums f32).  Lane j
// then owns column j: first of D, as a running product of the decays (no difference of logarithms, so a decay of zero is
// as exact as any), which meets both products where their accumulators lie; then of the inverse by substitution,
// t_i = [i = j] - sum_{l < i} L_il beta_l t_l, with L's rows broadcast from shared memory and two l to an instruction.
// P's accumulators are the B operand of the walk as they are; the inverse goes through shared memory once more.
// The kernel is bound by issued instructions: 2,500 a chunk with Q K^T and D kept in shared memory as well.
constexpr int kPrepWarps = 4;
constexpr int kLd = 36;  // f32 row stride of the 32 x 32 tiles: rows 16-byte aligned, columns on different banks

template <int KT> constexpr int prep_warp_bytes() {
    const int tiles = 2 * kC * row_bytes<KT>(), mats = 2 * kC * kLd * 4;
    return tiles > mats ? tiles : mats;
}

// rows of 32 tokens of a head into shared memory, zero past len and past dk; asynchronous
template <int KT>
__device__ __forceinline__ void fetch_rows(uint32_t dst, const bf16 *src, int64_t stride, int len, int dk, int lane) {
#pragma unroll
    for (int i = 0; i < KT * 2; ++i) {
        const int e = i * 32 + lane, t = e / (KT * 2), u = e % (KT * 2);
        const bool has = t < len && u * 8 < dk;
        cp_async16(dst + t * row_bytes<KT>() + u * 16, src + (has ? t * stride + u * 8 : 0), has);
    }
}

// Column `lane` of (I + L diag(beta))^-1 (kLeft: of (I + diag(beta) L)^-1) in t.  L holds anything finite on its
// diagonal: what it multiplies there is still zero.
template <bool kLeft>
__device__ __forceinline__ void invert(const float *L, float be, int lane, float (&t)[kC]) {
    Pair s[kC / 2];  // t, or beta t
#pragma unroll
    for (int i = 0; i < kC / 2; ++i) s[i] = both(0.f);
#pragma unroll
    for (int i = 0; i < kC; ++i) {
        Pair x = both(0.f), y = both(0.f);
#pragma unroll
        for (int l = 0; l < i; l += 4) {
            const ulonglong2 row = *reinterpret_cast<const ulonglong2 *>(L + i * kLd + l);
            x = fma(Pair{row.x}, s[l / 2], x);
            y = fma(Pair{row.y}, s[l / 2 + 1], y);
        }
        const float own = i == lane ? 1.f : 0.f, b = __shfl_sync(0xffffffffu, be, i), sum = total(x + y);
        t[i] = kLeft ? fmaf(-b, sum, own) : own - sum;
        const float v = kLeft ? t[i] : b * t[i];
        const float2 f = parts(s[i / 2]);
        s[i / 2] = i & 1 ? pair(f.x, v) : pair(v, 0.f);
    }
}

template <int KT, bool kGrad>
__global__ void __launch_bounds__(kPrepWarps * 32)
delta_prep_kernel(Shape p, unsigned units, const bf16 *__restrict__ q, const bf16 *__restrict__ k,
                  const void *__restrict__ g, const void *__restrict__ beta, FwdRecord *__restrict__ records,
                  AgainRecord *__restrict__ again, BwdRecord *__restrict__ back) {
    extern __shared__ __align__(128) char sm_raw[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned unit = blockIdx.x * kPrepWarps + warp;  // slot * H + h
    if (unit >= units) return;
    const int h = (int)(unit % (unsigned)p.H), hk = h / p.group();
    const int slot = (int)(unit / (unsigned)p.H);
    ChunkAt at;
    bool has;
    if (p.cu == nullptr) {
        has = chunk_of_slot<kC>(slot, p, at);
    } else {
        // what the kernels that follow need of every sequence, by the last units: they have the fewest chunks
        const unsigned seq = units - 1 - unit;
        if (p.order != nullptr && seq < (unsigned)p.nseq) {
            const int turn = rank_of(p, (int)seq, lane);
            if (lane == 0) p.order[turn] = (int)seq;
        }
        if (p.planned) {
            has = chunk_of_slot<kC>(slot, p, at);
        } else {
            const bool in_order = offsets_in_order(p);
            if (seq < (unsigned)p.nseq) {
                SeqRange r;
                const bool good = checked_rows(p, in_order, (int)seq, r);
                if (lane == 0) {
                    p.rows[seq] = make_int2((int)r.start, (int)r.len);
                    if (seq == 0) p.rows[p.nseq] = span_of(p, in_order);
                    if (!good) record_status(GLA_ERR_DEVICE_ARG);
                }
            }
            has = checked_chunk_of_slot<kC>(slot, p, in_order, at);
        }
    }
    if (!has) return;
    char *ks = sm_raw + warp * prep_warp_bytes<KT>(), *qs = ks + kC * row_bytes<KT>();
    float *L = reinterpret_cast<float *>(ks), *D = L + kC * kLd;  // in the rows' place once these are read
    const uint32_t ka = ptx::smem_u32(ks), qa = ptx::smem_u32(qs);
    fetch_rows<KT>(ka, k + (at.row * p.Hk + hk) * p.dk, (int64_t)p.Hk * p.dk, at.len, p.dk, lane);
    fetch_rows<KT>(qa, q + (at.row * p.Hk + hk) * p.dk, (int64_t)p.Hk * p.dk, at.len, p.dk, lane);
    float a = 1.f, be = 0.f;
    if (lane < at.len) {
        a = expf(load_gate<bf16>(g, (at.row + lane) * p.H + h, p.gate_f32));
        be = load_gate<bf16>(beta, (at.row + lane) * p.H + h, p.gate_f32);
    }
    cp_async_wait_all();
    __syncwarp();
    const int m8 = lane >> 3, r8 = lane & 7;
    float kk[2][4][4] = {}, qq[2][4][4] = {};  // tiles on and below the diagonal
#pragma unroll
    for (int s = 0; s < KT; ++s) {
        uint32_t b[2][4], ak[2][4], aq[2][4];
#pragma unroll
        for (int t = 0; t < 2; ++t) {  // tokens 16 t ..: as columns (B) and as rows (A)
            ldsm4(b[t], ka + (t * 16 + (m8 >> 1) * 8 + r8) * row_bytes<KT>() + s * 32 + (m8 & 1) * 16);
            const uint32_t off = (t * 16 + (m8 & 1) * 8 + r8) * row_bytes<KT>() + s * 32 + (m8 >> 1) * 16;
            ldsm4(ak[t], ka + off);
            ldsm4(aq[t], qa + off);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int t = 0; t <= i; ++t) {
                mma(kk[i][2 * t], ak[i], b[t][0], b[t][1]);
                mma(kk[i][2 * t + 1], ak[i], b[t][2], b[t][3]);
                mma(qq[i][2 * t], aq[i], b[t][0], b[t][1]);
                mma(qq[i][2 * t + 1], aq[i], b[t][2], b[t][3]);
            }
    }
    __syncwarp();
    const int gr = lane >> 2, tg = lane & 3;
    float f = 0.f, run = 1.f, c = 1.f;
#pragma unroll
    for (int i = 0; i < kC; ++i) {
        const float ai = __shfl_sync(0xffffffffu, a, i);
        run *= ai;
        if (i == lane) c = run;
        f = i == lane ? 1.f : f * ai;
        D[i * kLd + lane] = f;
    }
    __syncwarp();
    // L = D o K K^T to shared memory (anything on the diagonal); P = D o Q K^T (diag(beta)) stays where it is
    uint32_t pp[4][4];  // [tile of 8 rows][tile of 8 columns]
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            if (t > n) {
                pp[n][t] = 0;
                if (t <= (n | 1)) *reinterpret_cast<float2 *>(L + (n * 8 + gr) * kLd + t * 8 + 2 * tg) = make_float2(0.f, 0.f);
                continue;
            }
            const int at0 = (n * 8 + gr) * kLd + t * 8 + 2 * tg, i = n >> 1, e = (n & 1) * 2;
            const float2 d = *reinterpret_cast<const float2 *>(D + at0);
            *reinterpret_cast<float2 *>(L + at0) = make_float2(d.x * kk[i][t][e], d.y * kk[i][t][e + 1]);
            float x = d.x * qq[i][t][e], y = d.y * qq[i][t][e + 1];
            if (!kGrad) {
                x *= __shfl_sync(0xffffffffu, be, t * 8 + 2 * tg);
                y *= __shfl_sync(0xffffffffu, be, t * 8 + 2 * tg + 1);
            }
            pp[n][t] = pack(x, y);
        }
    __syncwarp();
    float t[kC];
    if (kGrad) {
        BwdRecord *rec = back + unit;
        float left[kC];
        invert<true>(L, be, lane, left);
#pragma unroll
        for (int i = 0; i < kC; ++i) D[i * kLd + lane] = left[i];
        __syncwarp();
#pragma unroll
        for (int n = 0; n < 4; ++n) {  // as B operands over the rows (k = i, n = j)
            uint32_t mm[4], pt[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int at0 = (e * 8 + 2 * tg) * kLd + n * 8 + gr;
                mm[e] = e >= n ? pack(D[at0], D[at0 + kLd]) : 0;
                pt[e] = e >= n ? transpose8(pp[e][n]) : 0;
            }
            rec->m[n][lane] = make_uint4(mm[0], mm[1], mm[2], mm[3]);
            rec->p[n][lane] = make_uint4(pt[0], pt[1], pt[2], pt[3]);
        }
        rec->c[lane] = c;
        rec->d[lane] = f;
        rec->b[lane] = be;
        __syncwarp();
    }
    invert<false>(L, be, lane, t);
#pragma unroll
    for (int i = 0; i < kC; ++i) D[i * kLd + lane] = t[i];
    __syncwarp();
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        uint32_t hi[4] = {}, lo[4] = {};
#pragma unroll
        for (int e = 0; e <= n; ++e) {
            const float2 m = *reinterpret_cast<const float2 *>(D + (n * 8 + gr) * kLd + e * 8 + 2 * tg);
            split(m.x, m.y, hi[e], lo[e]);
        }
        if (kGrad) {
            again[unit].mhi[n][lane] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        } else {
            records[unit].mhi[n][lane] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            records[unit].mlo[n][lane] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            records[unit].p[n][lane] = make_uint4(pp[n][0], pp[n][1], pp[n][2], pp[n][3]);
        }
    }
    (kGrad ? again[unit].c : records[unit].c)[lane] = c;
    (kGrad ? again[unit].db : records[unit].db)[lane] = f * be;
}

// ---- the walk ---------------------------------------------------------------------------------------------------

// kSegment: a segment's part of the map S -> M S + N alone, from zero: its first tiles carry N (the state that v leaves,
// from a zero state), the others M (from the identity, with v = 0: a column past dv is staged as zero).
struct FwdArgs {
    const bf16 *q, *k, *v;
    const FwdRecord *records;
    const float *h0;       // [nseq, H, dk, dv] or null
    const float *starts;   // with segments: the state before each, [slots, H, dk, dv]
    bf16 *out;
    float *hT;
    float *N, *M;          // [slots, H, dk, dv], [slots, H, dk, dk]
};

template <int KT, bool kSegment>
__global__ void __launch_bounds__(kMaxThreads, 1)
delta_fwd_kernel(Shape p, Walk w, FwdArgs a) {
    extern __shared__ __align__(128) char sm_raw[];
    constexpr int kRow = row_bytes<KT>(), kTile = kC * kRow, kV = (kSegment ? 1 : 2) * kTile;
    const Frame f(p, w, blockIdx.x, sm_raw);
    if (!f.exists || (kSegment && f.last)) return;  // nothing starts where a sequence ends
    if (f.warp >= w.groups * 4) {
        give_registers();
        fetch<KT, !kSegment, false, kSegment ? 0 : 1>(p, w, f, a.q, a.k, a.v, a.records, a.out, nullptr);
        return;
    }
    take_registers();
    if (f.warp >= w.warps) return;
    const int lane = f.lane, tg = lane & 3, m8 = lane >> 3, r8 = lane & 7;
    const int col = f.col0 + f.warp * 16;
    const int mcol = col - (p.dv + 15) / 16 * 16;  // kSegment: column of M, or negative
    float S[2 * KT][4];
    if (kSegment) {
#pragma unroll
        for (int n = 0; n < 2 * KT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                S[n][e] = mcol >= 0 && n * 8 + 2 * tg + (e & 1) == mcol + (lane >> 2) + (e >> 1) * 8 ? 1.f : 0.f;
    } else if (w.segment) {
        load_state<KT>(S, a.starts, f.walk, p.dk, p.dv, col, lane);
    } else {
        load_state<KT>(S, a.h0, f.walk, p.dk, p.dv, col, lane);
    }
    for (int c = 0; c < f.nch; ++c) {
        const int sg = c % w.stages;
        if (!warp_wait(f.full + 8 * sg, (c / w.stages) & 1, f.abort_flag)) {
            if (lane == 0) {
                *f.abort_flag = 1;
                record_status(GLA_ERR_TIMEOUT);
            }
            return;
        }
        const uint32_t ks = f.ring + sg * w.stage_bytes, qs = ks + kTile, vs = ks + kV + f.warp * 32,
                       rec = ks + kV + kC * w.vrow;
        const uint32_t vec = rec + (uint32_t)offsetof(FwdRecord, c) + 8 * tg;
        // Y = S^T K^T
        float Y[4][4];
        const uint32_t row_off = ((m8 >> 1) * 8 + r8) * kRow + (m8 & 1) * 16;
#pragma unroll
        for (int i = 0; i < KT; ++i) {
            uint32_t ah[4], al[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                split(S[2 * i + (e >> 1)][(e & 1) * 2], S[2 * i + (e >> 1)][(e & 1) * 2 + 1], ah[e], al[e]);
            // four independent sums in turn: an accumulator is ready again 21 clocks after its product began
            uint32_t b0[4], b1[4];
            ldsm4(b0, ks + row_off + i * 32);
            ldsm4(b1, ks + row_off + 16 * kRow + i * 32);
            if (i == 0) {
                mma0(Y[0], ah, b0[0], b0[1]);
                mma0(Y[1], ah, b0[2], b0[3]);
                mma0(Y[2], ah, b1[0], b1[1]);
                mma0(Y[3], ah, b1[2], b1[3]);
            } else {
                mma(Y[0], ah, b0[0], b0[1]);
                mma(Y[1], ah, b0[2], b0[3]);
                mma(Y[2], ah, b1[0], b1[1]);
                mma(Y[3], ah, b1[2], b1[3]);
            }
            mma(Y[0], al, b0[0], b0[1]);
            mma(Y[1], al, b0[2], b0[3]);
            mma(Y[2], al, b1[0], b1[1]);
            mma(Y[3], al, b1[2], b1[3]);
        }
        // X^T = V^T - Y diag(c), as hi and lo parts
        uint32_t xh[2][4], xl[2][4];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            uint32_t b[4];
            ldsm4t(b, vs + (t * 16 + (m8 >> 1) * 8 + r8) * w.vrow + (m8 & 1) * 16);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int n = 2 * t + u;
                const float2 cc = lds_f2(vec + n * 32);
                split(fmaf(-cc.x, Y[n][0], lo_f(b[2 * u])), fmaf(-cc.y, Y[n][1], hi_f(b[2 * u])), xh[t][2 * u], xl[t][2 * u]);
                split(fmaf(-cc.x, Y[n][2], lo_f(b[2 * u + 1])), fmaf(-cc.y, Y[n][3], hi_f(b[2 * u + 1])),
                      xh[t][2 * u + 1], xl[t][2 * u + 1]);
            }
        }
        // R^T = X^T M^T: M is lower triangular, so the first 16 rows meet the first 16 columns only
        float R[4][4];
        {
            uint4 m[4];
#pragma unroll
            for (int n = 0; n < 4; ++n) m[n] = lds128(rec + n * 512 + lane * 16);
#pragma unroll
            for (int n = 0; n < 4; ++n) mma0(R[n], xh[0], m[n].x, m[n].y);
#pragma unroll
            for (int n = 0; n < 4; ++n) mma(R[n], xl[0], m[n].x, m[n].y);
            mma(R[2], xh[1], m[2].z, m[2].w);
            mma(R[3], xh[1], m[3].z, m[3].w);
            mma(R[2], xl[1], m[2].z, m[2].w);
            mma(R[3], xl[1], m[3].z, m[3].w);
#pragma unroll
            for (int n = 0; n < 4; ++n) m[n] = lds128(rec + 2048 + n * 512 + lane * 16);
#pragma unroll
            for (int n = 0; n < 4; ++n) mma(R[n], xh[0], m[n].x, m[n].y);
            mma(R[2], xh[1], m[2].z, m[2].w);
            mma(R[3], xh[1], m[3].z, m[3].w);
        }
        // O = S^T Q^T diag(c) + R^T P^T with S and R rounded to bf16; U = R diag(d beta) as hi and lo parts
        uint32_t rh[2][4], uh[2][4], ul[2][4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int t = n >> 1, u = (n & 1) * 2;
            const float2 db = lds_f2(vec + 4 * kC + n * 32);
            rh[t][u] = pack(R[n][0], R[n][1]);
            rh[t][u + 1] = pack(R[n][2], R[n][3]);
            split(R[n][0] * db.x, R[n][1] * db.y, uh[t][u], ul[t][u]);
            split(R[n][2] * db.x, R[n][3] * db.y, uh[t][u + 1], ul[t][u + 1]);
        }
        float O[4][4];
        if (!kSegment) {
#pragma unroll
        for (int i = 0; i < KT; ++i) {
            uint32_t a[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) a[e] = pack(S[2 * i + (e >> 1)][(e & 1) * 2], S[2 * i + (e >> 1)][(e & 1) * 2 + 1]);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                uint32_t b[4];
                ldsm4(b, qs + row_off + t * 16 * kRow + i * 32);
                if (i == 0) {
                    mma0(O[2 * t], a, b[0], b[1]);
                    mma0(O[2 * t + 1], a, b[2], b[3]);
                } else {
                    mma(O[2 * t], a, b[0], b[1]);
                    mma(O[2 * t + 1], a, b[2], b[3]);
                }
            }
        }
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const float2 cc = lds_f2(vec + n * 32);
            scale(O[n], pair(cc.x, cc.y));
            const uint4 pp = lds128(rec + 4096 + n * 512 + lane * 16);
            mma(O[n], rh[0], pp.x, pp.y);
            if (n >= 2) mma(O[n], rh[1], pp.z, pp.w);
        }
        }
        // S^T = c_31 S^T + U K
        const float last = lds_f2(rec + (uint32_t)offsetof(FwdRecord, c) + 8 * 15).y;
#pragma unroll
        for (int n = 0; n < 2 * KT; n += 4) {
            uint32_t b[4][4];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                ldsm4t(b[m], ks + lane * kRow + (n + m) * 16);
                scale(S[n + m], both(last));
            }
#pragma unroll
            for (int m = 0; m < 4; ++m) mma(S[n + m], uh[0], b[m][0], b[m][1]);
#pragma unroll
            for (int m = 0; m < 4; ++m) mma(S[n + m], uh[1], b[m][2], b[m][3]);
#pragma unroll
            for (int m = 0; m < 4; ++m) mma(S[n + m], ul[0], b[m][0], b[m][1]);
#pragma unroll
            for (int m = 0; m < 4; ++m) mma(S[n + m], ul[1], b[m][2], b[m][3]);
        }
        if (!kSegment) put_tile(O, vs, w.vrow, lane);  // in the place of this warp's columns of V
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(f.empty + 8 * sg);
    }
    if (kSegment) {
        if (mcol < 0) store_state<KT>(a.N, S, f.walk, p.dk, p.dv, col, lane);
        else store_state<KT>(a.M, S, f.walk, p.dk, p.dk, mcol, lane);
    } else if (a.hT != nullptr && f.last) {
        store_state<KT>(a.hT, S, (int64_t)f.s * p.H + f.h, p.dk, p.dv, col, lane);
    }
}

// The state before every segment of a chain, S_{i+1} = M_i S_i + N_i from h0, for 32 columns of a head: 256 threads, a
// column and every eighth row each.  The state and M (the next segment's while one is used) lie in shared memory; an
// element of S read there serves all of a thread's rows.  A sequence without tokens (or with bad offsets) has no
// segments: its final state is written here.
constexpr int kJoinCols = 32;
inline int join_bytes(int dk) { return (2 * dk * dk + dk * kJoinCols) * (int)sizeof(float); }  // >= (KT * 16 + dk) dk

template <int KT>
__global__ void __launch_bounds__(256)
delta_join_kernel(Shape p, int segment, const float *__restrict__ M, const float *__restrict__ N,
                  const float *__restrict__ h0, float *__restrict__ starts, float *__restrict__ hT) {
    extern __shared__ __align__(128) char sm_raw[];
    const int dk = p.dk, c = threadIdx.x & 31, part = threadIdx.x >> 5;
    float *m = reinterpret_cast<float *>(sm_raw), *S = m + 2 * dk * dk;  // [2][dk][dk], [dk][32]
    const int s = blockIdx.x / p.H, h = blockIdx.x % p.H, col = blockIdx.y * kJoinCols + c;
    const bool live = col < p.dv;
    const SeqRange r = rows_of(p, s);
    const int64_t slot0 = r.start / segment + s;
    const int n = (int)((r.len + segment - 1) / segment);
    const int64_t h_at = ((int64_t)s * p.H + h) * dk * p.dv + col;
    if (n == 0) {
        if (hT != nullptr && live)
            for (int i = part; i < dk; i += 8) hT[h_at + (int64_t)i * p.dv] = h0 != nullptr ? h0[h_at + (int64_t)i * p.dv] : 0.f;
        return;
    }
    const auto fetch_m = [&](int g) {
        const float *from = M + ((slot0 + g) * p.H + h) * dk * dk;
        const uint32_t to = ptx::smem_u32(m + (g & 1) * dk * dk);
        for (int i = threadIdx.x; i < dk * dk / 4; i += 256) cp_async16(to + i * 16, from + i * 4, true);
    };
    if (n > 1) fetch_m(0);
    for (int i = part; i < dk; i += 8) S[i * kJoinCols + c] = live && h0 != nullptr ? h0[h_at + (int64_t)i * p.dv] : 0.f;
    for (int g = 0; g < n; ++g) {
        const int64_t at = ((slot0 + g) * p.H + h) * dk * p.dv + col;
        float next[2 * KT];  // rows part, part + 8, ...
        cp_async_wait_all();
        __syncthreads();
        const bool go_on = g + 1 < n;
#pragma unroll
        for (int x = 0; x < 2 * KT; ++x) {
            const int i = x * 8 + part;
            const bool has = i < dk && live;
            if (has) starts[at + (int64_t)i * p.dv] = S[i * kJoinCols + c];
            next[x] = has && go_on ? __ldg(N + at + (int64_t)i * p.dv) : 0.f;
        }
        if (!go_on) break;
        if (g + 2 < n) fetch_m(g + 1);
        const float *mg = m + (g & 1) * dk * dk + part * dk;  // rows past dk read what lies behind, for no one
        for (int j = 0; j < dk; j += 4) {
            const float s0 = S[j * kJoinCols + c], s1 = S[(j + 1) * kJoinCols + c], s2 = S[(j + 2) * kJoinCols + c],
                        s3 = S[(j + 3) * kJoinCols + c];
#pragma unroll
            for (int x = 0; x < 2 * KT; ++x) {
                const float4 t = *reinterpret_cast<const float4 *>(mg + x * 8 * dk + j);
                next[x] = fmaf(t.x, s0, fmaf(t.y, s1, fmaf(t.z, s2, fmaf(t.w, s3, next[x]))));
            }
        }
        __syncthreads();
#pragma unroll
        for (int x = 0; x < 2 * KT; ++x)
            if (x * 8 < dk) S[(x * 8 + part) * kJoinCols + c] = next[x];
    }
}

// Tokens per segment, or 0 for whole chains.  A walk is one product after another, so few chains leave most of the GPU
// idle: B1 T32768 H16 dk96 dv192 takes 1,416 us as 16 chains and 865 cut.  Chains are cut into as many segments as fill
// the GPU (12 column tiles to an SM), none shorter than 256 tokens, where that is the cheaper way.  Counted in steps of a
// walk (a chunk of a chain, some 0.16 us times KT), with n segments to a sequence,
//     saved  the steps of n - 1 segments
//     paid   0.375 for each chunk that has to give a map, head and column tile of it (dv / 16 + KT) per SM, 4 for each
//            segment in the join's row (3 where dk <= 64), and 6 for two more launches
// At 248 sizes with both ways measured (1 to 32 heads of 24/40 to 128/256, 1 to 4 sequences of 256 to 32,768 tokens) this
// loses 0.4% against the better one, 11% at most.  Whole and cut, us: 4 x 2,048, 8 heads of 128/128 102 and 179; 1 x 4,096, 16
// heads of 96/192 146 and 163; 1 x 8,192 288 and 266; 1 x 2,048, 4 heads of 64/64 59 and 44.
// Of several packed sequences only the device knows the lengths, and the longest one decides: 1 of 5,200 and 5 of 100
// tokens, 6 heads of 24/40, 122 whole and 46 cut; 6 of 1,300, 24 heads of 32/32, 56 and 88.  They are cut where a sixth
// of the GPU's tiles would do for all chains, and where there are four segments in all; over 60 such batches that loses
// 5% on equal lengths and 1% on uneven ones.
int segment_tokens(const Shape &p) {
    const long long rows = total_rows(p), tiles = (p.dv + 15) / 16, sms = device_info().sm_count;
    if (rows == 0 || sms == 0) return 0;
    const long long segments = max(1LL, sms * kMaxWarps / (p.H * tiles));
    const long long tokens = (max(256LL, (rows + segments - 1) / segments) + kC - 1) / kC * kC;
    if (p.cu && p.nseq > 1)
        return (long long)p.nseq * p.H * tiles * 6 <= sms * kMaxWarps && rows >= 4 * tokens ? (int)tokens : 0;
    if (p.T <= tokens) return 0;
    const int kt = p.dk <= 32 ? 2 : p.dk <= 64 ? 4 : p.dk <= 96 ? 6 : 8;
    const double n = (double)p.T / (double)tokens, kept = 1.0 - 1.0 / n;
    const double maps = 0.375 * (double)rows / kC * kept * (double)(p.H * (tiles + kt)) / (double)sms;
    return (double)p.T / kC * kept > maps + (p.dk <= 64 ? 3.0 : 4.0) * n + 6.0 ? (int)tokens : 0;
}
struct Segments {
    int tokens;
    size_t slots, M, N, starts, total;  // offsets in bytes
};
Segments plan_segments(const Shape &p) {
    Segments g{};
    g.tokens = segment_tokens(p);
    if (g.tokens == 0) return g;
    g.slots = (size_t)chunk_slots(total_rows(p), p.nseq, g.tokens);
    const size_t n = g.slots * p.H * p.dk * sizeof(float);
    g.M = 0;
    g.N = (n * p.dk + 255) / 256 * 256;
    g.starts = g.N + (n * p.dv + 255) / 256 * 256;
    g.total = g.starts + n * p.dv;
    return g;
}

// The rows of every sequence of a batch of more than kMostChecked, by one block.
constexpr int kPlanThreads = 1024;
__global__ void __launch_bounds__(kPlanThreads) delta_plan_kernel(Shape p) {
    __shared__ int ends[kPlanThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int end = 0;  // of the sequences so far
    bool all_good = true;
    for (int64_t s0 = 0; s0 < p.nseq; s0 += kPlanThreads) {
        const int64_t s = s0 + threadIdx.x;
        SeqRange r{0, 0};
        const bool own = s < p.nseq && seq_range((int)s, p.T, p.cu, r);
        int upto = own ? (int)(r.start + r.len) : 0;  // the largest end of this warp's sequences up to this one
        for (int m = 1; m < 32; m <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, upto, m);
            if (lane >= m) upto = max(upto, x);
        }
        if (lane == 31) ends[warp] = upto;
        __syncthreads();
        int before = __shfl_up_sync(0xffffffffu, upto, 1);
        before = max(end, lane > 0 ? before : 0);
        for (int i = 0; i < kPlanThreads / 32; ++i) {
            if (i < warp) before = max(before, ends[i]);
            end = max(end, ends[i]);
        }
        if (s < p.nseq) {
            const bool good = own && r.start >= before;
            p.rows[s] = good ? make_int2((int)r.start, (int)r.len) : make_int2(before, 0);
            if (!good) record_status(GLA_ERR_DEVICE_ARG);
            all_good = all_good && good;
        }
        __syncthreads();
    }
    if (!__syncthreads_and(all_good)) all_good = false;
    if (threadIdx.x == 0) p.rows[p.nseq] = span_of(p, all_good);
}

template <int KT, bool kGrad>
int launch_prep(const Shape &p, const bf16 *q, const bf16 *k, const void *g, const void *beta, FwdRecord *records,
                AgainRecord *again, BwdRecord *back, cudaStream_t st) {
    const unsigned units = (unsigned)(chunk_slots(total_rows(p), p.nseq, kC) * p.H);
    const int bytes = kPrepWarps * prep_warp_bytes<KT>();
    if (!allow_smem<delta_prep_kernel<KT, kGrad>>()) return GLA_ERR_LAUNCH;
    if (p.planned) {
        delta_plan_kernel<<<1, kPlanThreads, 0, st>>>(p);
        count_launches(1);
    }
    delta_prep_kernel<KT, kGrad><<<(units + kPrepWarps - 1) / kPrepWarps, kPrepWarps * 32, bytes, st>>>(
        p, units, q, k, g, beta, records, again, back);
    count_launches(1);
    return cudaGetLastError() == cudaSuccess ? GLA_OK : GLA_ERR_LAUNCH;
}

// The workspace: the sequences' rows, the records, and the segments' maps and states.
size_t record_bytes(const Shape &p) {
    return ((size_t)chunk_slots(total_rows(p), p.nseq, kC) * p.H * sizeof(FwdRecord) + 255) / 256 * 256;
}

template <int KT>
int fwd_kt(Shape p, const bf16 *q, const bf16 *k, const bf16 *v, const void *g, const void *beta,
           const float *h0, bf16 *out, float *hT, char *ws, cudaStream_t st) {
    const Segments sg = plan_segments(p);
    const int tiles = (p.dv + 15) / 16;
    const long long walks = sg.tokens ? (long long)sg.slots * p.H : (long long)p.nseq * p.H;
    Walk w = make_walk<KT, FwdRecord>(walks, tiles, true, 1), ws_ = make_walk<KT, FwdRecord>(walks, tiles + KT, false, 0);
    w.segment = ws_.segment = sg.tokens;
    if (walks * max(w.splits, ws_.splits) > 0x7fffffffLL) return GLA_ERR_UNSUPPORTED;
    if (!allow_smem<delta_fwd_kernel<KT, false>>() || !allow_smem<delta_fwd_kernel<KT, true>>() ||
        !allow_smem<delta_join_kernel<KT>>())
        return GLA_ERR_LAUNCH;
    place_rows(p, ws, sg.tokens ? 0 : walks * w.splits);
    ws += rows_bytes(p);
    FwdRecord *records = (FwdRecord *)ws;
    int rc = launch_prep<KT, false>(p, q, k, g, beta, records, nullptr, nullptr, st);
    if (rc != GLA_OK) return rc;
    char *seg = ws + record_bytes(p);
    const FwdArgs a{q, k, v, records, h0, (float *)(seg + sg.starts), out, hT, (float *)(seg + sg.N), (float *)(seg + sg.M)};
    if (sg.tokens) {
        delta_fwd_kernel<KT, true><<<(unsigned)(walks * ws_.splits), (ws_.groups + 1) * 128, walk_bytes(ws_), st>>>(p, ws_, a);
        const dim3 grid((unsigned)(p.nseq * p.H), (unsigned)((p.dv + kJoinCols - 1) / kJoinCols));
        delta_join_kernel<KT><<<grid, 256, join_bytes(p.dk), st>>>(p, sg.tokens, a.M, a.N, h0, (float *)(seg + sg.starts), hT);
        count_launches(2);
    }
    delta_fwd_kernel<KT, false><<<(unsigned)(walks * w.splits), (w.groups + 1) * 128, walk_bytes(w), st>>>(p, w, a);
    count_launches(1);
    return cudaGetLastError() == cudaSuccess ? GLA_OK : GLA_ERR_LAUNCH;
}

}  // namespace

// bf16 with dk <= 128: a warp's share of the state fits its registers.
bool mma_supported(int dk) { return dk <= 128; }

size_t mma_fwd_workspace(const Shape &p) { return rows_bytes(p) + record_bytes(p) + plan_segments(p).total; }

int mma_fwd(const Shape &p, const void *q, const void *k, const void *v, const void *g, const void *beta,
            const float *h0, void *out, float *hT, void *ws, cudaStream_t st) {
#define GLA_CALL(KT) \
    return fwd_kt<KT>(p, (const bf16 *)q, (const bf16 *)k, (const bf16 *)v, g, beta, h0, (bf16 *)out, hT, (char *)ws, st)
    GLA_BY_KT(p.dk, GLA_CALL);
#undef GLA_CALL
}

// The gradient's records (gla_delta_bwd.cu).
int mma_prep_grad(const Shape &p, const void *q, const void *k, const void *g, const void *beta, void *again, void *back,
                  cudaStream_t st) {
#define GLA_CALL(KT)                                                                                               \
    return launch_prep<KT, true>(p, (const bf16 *)q, (const bf16 *)k, g, beta, nullptr, (AgainRecord *)again,      \
                                 (BwdRecord *)back, st)
    GLA_BY_KT(p.dk, GLA_CALL);
#undef GLA_CALL
}

}  // namespace delta
}  // namespace gla
