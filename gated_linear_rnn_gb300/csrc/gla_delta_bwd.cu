// gla_delta_bwd.cu — the gradient of the gated delta rule on the tensor cores (bf16 inputs).
//
// Three kernels, with the notation of gla_delta_mma.cu (dS1: the gradient after a chunk, dS0: before it):
//   delta_prep_kernel  for every chunk of 32 tokens and head: what does not depend on the states.
//   delta_walks_kernel walks each chain forwards as the forward does, without its output: the residuals R, and the
//                      state before every 64th token; and backwards: with dU = P^T dO + diag(d) K dS1 the gradient
//                      that reaches a token's write from outside the chunk and from its reads inside,
//                          Y = (I + diag(beta) L)^-T dU,  dV = diag(beta) Y,
//                          dS0 = c_31 dS1 + Q^T diag(c) dO - K^T diag(c) dV,
//                      and writes Y, dV and the gradient after every 64 tokens.
//   delta_grad_kernel  the rest is local to 64 tokens given S0, dS1, R, Y and dO (the residuals and Y belong to
//                      their tokens, not to a chunk's length): dq, dk, dg and dbeta.
// Both walks keep S^T (dS^T) in registers, 16 columns to a warp, as the forward does.  The gradients are rounded
// to bf16 at the end, so most of their products take operands rounded to bf16, without the lo parts that the
// forward's state needs; states and all sums are f32.  One rounding to bf16 is 1.7e-3 of a vector's norm, and
// they add in squares: X and dU, which every residual and every Y are made of, keep their lo parts (six products of
// 16 x 8 x 16 a chunk each), which takes dbeta, a product of both, from 4.7e-3 to 4e-3.
#include "gla_delta_mma.cuh"

GLA_DEFINE_STATUS(delta_bwd)

namespace gla {
namespace delta {

int mma_prep_grad(const Shape &p, const void *q, const void *k, const void *g, const void *beta, void *again, void *back,
                  cudaStream_t st);

namespace {

constexpr int kG = 64;  // tokens of a chunk of the gradient kernel: two chunks of a walk

// S^T's 16 columns rounded to bf16, as 8 x 8 matrices (rows: columns of S) of 128 bytes each, [KT][4] of them for each
// column tile: rows 0-7 and 8-15 of dk's columns 16 i .., then of 16 i + 8 ...  Read with ldmatrix (transposed) they are
// B operands (k = the 16 columns, n = dk).
template <int KT>
__device__ __forceinline__ void write_image(uint4 *image, const float (&S)[2 * KT][4], int lane) {
    uint32_t *to = reinterpret_cast<uint32_t *>(image) + lane;
#pragma unroll
    for (int n = 0; n < 2 * KT; ++n) {
        to[n * 64] = pack(S[n][0], S[n][1]);
        to[n * 64 + 32] = pack(S[n][2], S[n][3]);
    }
}
// the image of column tile `tile` of the state of (slot of 64 tokens, head)
template <int KT>
__device__ __forceinline__ int64_t image_at(const Shape &p, int64_t slot, int h, int tile) {
    return ((slot * p.H + h) * ((p.dv + 15) / 16) + tile) * KT * 32;
}

// acc[t] = S^T K^T over the chunk's 32 tokens (t: tiles of 8 tokens), S rounded to bf16
template <int KT>
__device__ __forceinline__ void state_times_rows(float (&acc)[4][4], const float (&S)[2 * KT][4], uint32_t rows, int lane) {
    const uint32_t off = (((lane >> 3) >> 1) * 8 + (lane & 7)) * row_bytes<KT>() + ((lane >> 3) & 1) * 16;
#pragma unroll
    for (int i = 0; i < KT; ++i) {
        uint32_t a[4], b0[4], b1[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) a[e] = pack(S[2 * i + (e >> 1)][(e & 1) * 2], S[2 * i + (e >> 1)][(e & 1) * 2 + 1]);
        ldsm4(b0, rows + off + i * 32);
        ldsm4(b1, rows + off + 16 * row_bytes<KT>() + i * 32);
        if (i == 0) {
            mma0(acc[0], a, b0[0], b0[1]);
            mma0(acc[1], a, b0[2], b0[3]);
            mma0(acc[2], a, b1[0], b1[1]);
            mma0(acc[3], a, b1[2], b1[3]);
        } else {
            mma(acc[0], a, b0[0], b0[1]);
            mma(acc[1], a, b0[2], b0[3]);
            mma(acc[2], a, b1[0], b1[1]);
            mma(acc[3], a, b1[2], b1[3]);
        }
    }
}
// S^T += U rows for U (16 columns x 32 tokens) as A operands
template <int KT>
__device__ __forceinline__ void add_outer(float (&S)[2 * KT][4], const uint32_t (&u)[2][4], uint32_t rows, int lane) {
#pragma unroll
    for (int n = 0; n < 2 * KT; n += 4) {
        uint32_t b[4][4];
#pragma unroll
        for (int m = 0; m < 4; ++m) ldsm4t(b[m], rows + lane * row_bytes<KT>() + (n + m) * 16);
#pragma unroll
        for (int m = 0; m < 4; ++m) mma(S[n + m], u[0], b[m][0], b[m][1]);
#pragma unroll
        for (int m = 0; m < 4; ++m) mma(S[n + m], u[1], b[m][2], b[m][3]);
    }
}

// Forwards, without an output.
template <int KT>
__device__ __forceinline__ void walk_again(const Shape &p, const Walk &w, unsigned block, char *sm_raw,
                                           const bf16 *__restrict__ k, const bf16 *__restrict__ v,
                                           const AgainRecord *__restrict__ records, const float *__restrict__ h0,
                                           bf16 *__restrict__ resid, uint4 *__restrict__ images) {
    constexpr int kTile = kC * row_bytes<KT>();
    const Frame f(p, w, block, sm_raw);
    if (f.bad && threadIdx.x == 0) record_status(GLA_ERR_DEVICE_ARG);
    if (f.warp >= w.groups * 4) {
        give_registers();
        fetch<KT, false, false, 1>(p, w, f, k, k, v, records, resid, nullptr);
        return;
    }
    take_registers();
    if (f.warp >= w.warps) return;
    const int lane = f.lane, tg = lane & 3, m8 = lane >> 3, r8 = lane & 7;
    const int col = f.col0 + f.warp * 16;
    const int64_t slot64 = f.r.start / kG + f.s;
    const bool live = col < p.dv;
    float S[2 * KT][4];
    load_state<KT>(S, h0, f.walk, p.dk, p.dv, col, lane);
    for (int c = 0; c < f.nch; ++c) {
        const int sg = c % w.stages;
        if (!warp_wait(f.full + 8 * sg, (c / w.stages) & 1, f.abort_flag)) {
            if (lane == 0) {
                *f.abort_flag = 1;
                record_status(GLA_ERR_TIMEOUT);
            }
            return;
        }
        if ((c & 1) == 0 && live) write_image<KT>(images + image_at<KT>(p, slot64 + c / 2, f.h, col / 16), S, lane);
        const uint32_t ks = f.ring + sg * w.stage_bytes, vs = ks + kTile + f.warp * 32, rec = ks + kTile + kC * w.vrow;
        const uint32_t vec = rec + (uint32_t)offsetof(AgainRecord, c) + 8 * tg;
        float Y[4][4];
        state_times_rows<KT>(Y, S, ks, lane);
        uint32_t x[2][4], xl[2][4];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            uint32_t b[4];
            ldsm4t(b, vs + (t * 16 + (m8 >> 1) * 8 + r8) * w.vrow + (m8 & 1) * 16);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int n = 2 * t + u;
                const float2 cc = lds_f2(vec + n * 32);
                split(fmaf(-cc.x, Y[n][0], lo_f(b[2 * u])), fmaf(-cc.y, Y[n][1], hi_f(b[2 * u])), x[t][2 * u], xl[t][2 * u]);
                split(fmaf(-cc.x, Y[n][2], lo_f(b[2 * u + 1])), fmaf(-cc.y, Y[n][3], hi_f(b[2 * u + 1])),
                      x[t][2 * u + 1], xl[t][2 * u + 1]);
            }
        }
        float R[4][4];
        uint4 m[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) m[n] = lds128(rec + n * 512 + lane * 16);
#pragma unroll
        for (int n = 0; n < 4; ++n) mma0(R[n], x[0], m[n].x, m[n].y);
#pragma unroll
        for (int n = 0; n < 4; ++n) mma(R[n], xl[0], m[n].x, m[n].y);
        mma(R[2], x[1], m[2].z, m[2].w);
        mma(R[3], x[1], m[3].z, m[3].w);
        mma(R[2], xl[1], m[2].z, m[2].w);
        mma(R[3], xl[1], m[3].z, m[3].w);
        uint32_t u[2][4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const float2 db = lds_f2(vec + 4 * kC + n * 32);
            u[n >> 1][(n & 1) * 2] = pack(R[n][0] * db.x, R[n][1] * db.y);
            u[n >> 1][(n & 1) * 2 + 1] = pack(R[n][2] * db.x, R[n][3] * db.y);
        }
        const float last = lds_f2(rec + (uint32_t)offsetof(AgainRecord, c) + 8 * 15).y;
#pragma unroll
        for (int n = 0; n < 2 * KT; ++n) scale(S[n], both(last));
        add_outer<KT>(S, u, ks, lane);
        put_tile(R, vs, w.vrow, lane);  // in the place of this warp's columns of V
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(f.empty + 8 * sg);
    }
}

// Backwards.
template <int KT>
__device__ __forceinline__ void walk_back(const Shape &p, const Walk &w, unsigned block, char *sm_raw,
                                          const bf16 *__restrict__ q, const bf16 *__restrict__ k,
                                          const bf16 *__restrict__ dout, const BwdRecord *__restrict__ records,
                                          const float *__restrict__ dhT, bf16 *__restrict__ ys, bf16 *__restrict__ dv,
                                          uint4 *__restrict__ images, float *__restrict__ dh0) {
    constexpr int kTile = kC * row_bytes<KT>();
    const Frame f(p, w, block, sm_raw);
    if (f.bad && threadIdx.x == 0) record_status(GLA_ERR_DEVICE_ARG);
    if (f.warp >= w.groups * 4) {
        give_registers();
        fetch<KT, true, true, 2>(p, w, f, q, k, dout, records, ys, dv);
        return;
    }
    take_registers();
    if (f.warp >= w.warps) return;
    const int lane = f.lane, tg = lane & 3, m8 = lane >> 3, r8 = lane & 7;
    const int col = f.col0 + f.warp * 16;
    const int64_t slot64 = f.r.start / kG + f.s;
    const bool live = col < p.dv;
    float S[2 * KT][4];
    load_state<KT>(S, dhT, f.walk, p.dk, p.dv, col, lane);
    for (int i = 0; i < f.nch; ++i) {
        const int c = f.nch - 1 - i, sg = i % w.stages;
        if (!warp_wait(f.full + 8 * sg, (i / w.stages) & 1, f.abort_flag)) {
            if (lane == 0) {
                *f.abort_flag = 1;
                record_status(GLA_ERR_TIMEOUT);
            }
            return;
        }
        if (((c & 1) == 1 || i == 0) && live)
            write_image<KT>(images + image_at<KT>(p, slot64 + c / 2, f.h, col / 16), S, lane);
        const uint32_t ks = f.ring + sg * w.stage_bytes, qs = ks + kTile, vs = qs + kTile + f.warp * 32,
                       rec = qs + kTile + kC * w.vrow;
        const uint32_t vec = rec + (uint32_t)offsetof(BwdRecord, c) + 8 * tg;  // c, then d and beta 4 kC bytes on
        // dO^T as it lies in the stage is an A operand
        uint32_t a[2][4];
#pragma unroll
        for (int t = 0; t < 2; ++t) ldsm4t(a[t], vs + (t * 16 + (m8 >> 1) * 8 + r8) * w.vrow + (m8 & 1) * 16);
        // dU^T = dS^T K^T diag(d) + dO^T P: P is lower triangular, its first 16 rows reach the first 16 columns only
        float U[4][4];
        state_times_rows<KT>(U, S, ks, lane);
        uint4 m[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const float2 d = lds_f2(vec + 4 * kC + n * 32);
            scale(U[n], pair(d.x, d.y));
            m[n] = lds128(rec + n * 512 + lane * 16);
        }
#pragma unroll
        for (int n = 0; n < 4; ++n) mma(U[n], a[1], m[n].z, m[n].w);
        mma(U[0], a[0], m[0].x, m[0].y);
        mma(U[1], a[0], m[1].x, m[1].y);
        uint32_t u[2][4], ul[2][4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            split(U[n][0], U[n][1], u[n >> 1][(n & 1) * 2], ul[n >> 1][(n & 1) * 2]);
            split(U[n][2], U[n][3], u[n >> 1][(n & 1) * 2 + 1], ul[n >> 1][(n & 1) * 2 + 1]);
            m[n] = lds128(rec + 2048 + n * 512 + lane * 16);
        }
        float Y[4][4];
#pragma unroll
        for (int n = 0; n < 4; ++n) mma0(Y[n], u[1], m[n].z, m[n].w);
#pragma unroll
        for (int n = 0; n < 4; ++n) mma(Y[n], ul[1], m[n].z, m[n].w);
        mma(Y[0], u[0], m[0].x, m[0].y);
        mma(Y[1], u[0], m[1].x, m[1].y);
        mma(Y[0], ul[0], m[0].x, m[0].y);
        mma(Y[1], ul[0], m[1].x, m[1].y);
        // dS^T = c_31 dS^T + dO^T diag(c) Q - dV^T diag(c) K
        float D[4][4];
        uint32_t e[2][4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const float2 cc = lds_f2(vec + n * 32), b = lds_f2(vec + 8 * kC + n * 32);
            D[n][0] = Y[n][0] * b.x; D[n][1] = Y[n][1] * b.y; D[n][2] = Y[n][2] * b.x; D[n][3] = Y[n][3] * b.y;
            e[n >> 1][(n & 1) * 2] = pack(-cc.x * D[n][0], -cc.y * D[n][1]);
            e[n >> 1][(n & 1) * 2 + 1] = pack(-cc.x * D[n][2], -cc.y * D[n][3]);
            uint32_t &a0 = a[n >> 1][(n & 1) * 2], &a1 = a[n >> 1][(n & 1) * 2 + 1];
            a0 = pack(cc.x * lo_f(a0), cc.y * hi_f(a0));
            a1 = pack(cc.x * lo_f(a1), cc.y * hi_f(a1));
        }
        const float last = lds_f2(rec + (uint32_t)offsetof(BwdRecord, c) + 8 * 15).y;
#pragma unroll
        for (int n = 0; n < 2 * KT; ++n) scale(S[n], both(last));
        add_outer<KT>(S, a, qs, lane);
        add_outer<KT>(S, e, ks, lane);
        put_tile(Y, vs, w.vrow, lane);  // in the place of this warp's columns of dO
        put_tile(D, rec + (uint32_t)sizeof(BwdRecord) + f.warp * 32, w.vrow, lane);
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(f.empty + 8 * sg);
    }
    if (dh0 != nullptr) store_state<KT>(dh0, S, f.walk, p.dk, p.dv, col, lane);
}

struct WalkArgs {
    const bf16 *q, *k, *v, *dout;
    const AgainRecord *again;
    const BwdRecord *back;
    const float *h0, *dhT;
    bf16 *resid, *ys, *dv;
    uint4 *s_images, *ds_images;
    float *dh0;
};

// Both walks in one launch, since neither needs the other: the blocks of the longer one, backwards, come first.
template <int KT>
__global__ void __launch_bounds__(kMaxThreads, 1)
delta_walks_kernel(Shape p, Walk again, Walk back, unsigned blocks, WalkArgs a) {
    extern __shared__ __align__(128) char sm_raw[];
    if (blockIdx.x < blocks)
        walk_back<KT>(p, back, blockIdx.x, sm_raw, a.q, a.k, a.dout, a.back, a.dhT, a.ys, a.dv, a.ds_images, a.dh0);
    else
        walk_again<KT>(p, again, blockIdx.x - blocks, sm_raw, a.k, a.v, a.again, a.h0, a.resid, a.s_images);
}

// ---- dq, dk, dg, dbeta -----------------------------------------------------------------------------------------
//
// A unit is 64 tokens of a value head.  With D_ij, c_i and d_j over the 64 tokens,
//     R'_ij = beta_j D_ij (do_i . r_j), j <= i             N_ij = -beta_i beta_j D_ij (y_i . r_j), j < i
//     dq = diag(c) dO S0^T + R' K
//     dk = diag(d beta) R dS1^T - diag(c beta) Y S0^T + R'^T Q + N^T K + N K
//     dbeta_i = y_i . r_i
// and for dg_l, whose decay every product of a token before l with one at or after l crosses:
//     dg_l = sum_{i >= l} w_i + sum_{j < l} (x_j + m_j) + c_63 <S0, dS1>,
//     w = rows of q . (diag(c) dO S0^T) - k . (diag(c beta) Y S0^T),  x = rows of k . (diag(d beta) R dS1^T),
//     m = rows of k . (R'^T Q + N^T K - N K) - q . (R' K):
// the crossing products in the chunk, summed from the left (a token's reads leave, its writes enter), so that both
// ends of a product carry the same rounding and cancel to f32.
// D_ij comes from products of decays alone (a decay of zero is as good as any).
//
// All products run on tcgen05 with accumulators in TMEM, 128 rows at a time: rows 0-63 are the query's side of the
// unit's tokens, rows 64-127 the key's, so that everything that meets in one row of dq or dk lies in one TMEM lane
// and one thread:
//     D1 = [dO; Y] S0^T,  D2 = [Y; R] dS1^T,  D3 = [dO; Y] R^T,  D4 = [R'; N] K,  D5 = [.; R'^T Q + N^T K]
// One block per SM walks over units with four kinds of warps: four fetch (slabs of 32 columns of dO, Y, R and of both
// states through a ring; K, Q and the decays of a unit), one thread issues the products, three warps form
// <S0, dS1> from the slabs, and two warpgroups take turns as epilogues: D3 becomes R' and N (a thread's row of D is a
// running product along the row) in shared memory for D4 and D5, the others are scaled, summed and written.  D4 and D5
// take the columns of D1 and D2 once these are in registers; with two sets of columns (dk <= 96) the products of
// one unit run under the epilogue of the other.  As mma.sync with its operands through ldmatrix (every state
// element loaded by four warps) the kernel took 308 us on the layer's gradient, bound by shared memory and by the
// sequence of its phases.
//
// Operand tiles are without swizzle: 16-byte units [unit][row], whose 8 x 16-byte blocks are core matrices either way (rows
// as M or N with K along the units, or rows as K).
constexpr int kGradThreads = 512;      // 2 epilogue warpgroups, 1 fetching, 1 with the issuer and the inner products
constexpr int kInnerWarps = 3;
constexpr uint32_t kTmemCols = 512;
static_assert(2 * 200 + 2 * 56 == 4 * 128, "the epilogues take what the others give back");

struct Decays {                        // of one unit
    float alpha[kG + 4], beta[kG], c[kG], d[kG];  // alpha[64] = 1 stands behind the last
};
struct Sums {                          // per token
    float wq[kG], wk[kG], x[kG], mq[kG], mk[kG];
};
template <int KT> struct GradPlan {
    static constexpr int kN = KT * 16;
    static constexpr int kTile = kG * kN * 2;                                      // K or Q: [2 KT units][64 rows] x 16 bytes
    static constexpr int kHead = 2 * kTile + (int)sizeof(Decays);                  // K | Q | decays, two of them
    static constexpr int kRows = 3 * kG * 64;                                      // dO | Y | R: [4 units][192 rows] x 16 bytes
    static constexpr int kImage = 2 * KT * 512;                                    // two column tiles of a state
    static constexpr int kSlab = kRows + 2 * kImage;                               // rows | S0 | dS1
    static constexpr int kStages = KT <= 6 ? 5 : 4;
    static constexpr int kOwn = 2 * kG * 128;                                      // [R'; N]: [8 units][128 rows] x 16 bytes
    static constexpr int kFlip = 3 * kG * 128;                                     // N | R' | N: [24 units][64 rows] x 16 bytes
    static constexpr int kOffHead = 256, kOffSlab = kOffHead + 2 * kHead, kOffT = kOffSlab + kStages * kSlab,
                         kOffSums = kOffT + kOwn + kFlip, kOffInner = kOffSums + 4 * (int)sizeof(Sums),
                         kTotal = kOffInner + 2 * 16;
    static constexpr int kSets = KT <= 6 ? 2 : 1;                                  // of accumulators
    static constexpr uint32_t kSetCols = 2 * kN + kG;                              // D1 (D4) | D2 (D5) | D3
    static_assert(kTotal <= 227 * 1024, "shared memory of a block");
    static_assert(kSets * kSetCols <= kTmemCols, "TMEM");
    static_assert(kHead % 16 == 0 && kSlab % 16 == 0 && kOffInner % 16 == 0 && sizeof(Decays) % 16 == 0, "16-byte copies");
    // barriers
    static constexpr int kHFull = 0, kHEmpty = 16, kFull = 32, kEmpty = kFull + 8 * kStages, kAccFull = kEmpty + 8 * kStages,
                         kAccFree = kAccFull + 16, kReady = kAccFree + 16, kInFull = kReady + 16, kInner = kInFull + 16,
                         kAbort = kInner + 16, kTmem = kAbort + 4;
    static_assert(kTmem + 4 <= kOffHead, "barriers");
};

struct GradArgs {
    const bf16 *q, *k, *dout;
    const void *g, *beta;
    const bf16 *resid, *ys;
    const uint4 *s_images, *ds_images;
    bf16 *dq, *dk;          // written when each key head has one value head
    float *dq_part, *dk_part;  // else [rows, H, dk] each, summed by delta_heads_kernel
    void *dg, *dbeta;
    unsigned units;         // slots * H
};

// The units that a block walks over, in the same order for all of its warps.
struct Units {
    unsigned unit;
    int slot, h, n;  // n: how many came before
    ChunkAt at;
    __device__ __forceinline__ Units() : unit(blockIdx.x), n(-1) {}
    __device__ __forceinline__ bool next(const Shape &p, unsigned units) {
        if (n >= 0) unit += gridDim.x;
        for (; unit < units; unit += gridDim.x) {
            slot = (int)(unit / (unsigned)p.H);
            h = (int)(unit % (unsigned)p.H);
            if (chunk_of_slot<kG>(slot, p, at)) {
                ++n;
                return true;
            }
        }
        return false;
    }
};

// Slabs of a unit, then its K and Q: the products over the states need the slabs alone, so they run ahead of the
// epilogue that frees K's and Q's place.
template <int KT>
__device__ __forceinline__ void grad_fetch(const Shape &p, const GradArgs &a, char *sm) {
    using P = GradPlan<KT>;
    const uint32_t base = ptx::smem_u32(sm);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + P::kAbort);
    const int id = threadIdx.x & 127;
    const int tiles = (p.dv + 15) / 16, slabs = (tiles + 1) / 2;
    const int64_t vst = (int64_t)p.H * p.dv;
    // Up to four groups of copies (a slab, or K and Q) are on their way at a time, some 90 KB: what a latency of two
    // microseconds takes at this SM's share of the bandwidth.  Groups become known in order, once they have landed.
    constexpr int kAhead = 4;
    int ns = 0, out = 0, groups = 0;  // slabs issued and made known, groups on their way
    uint32_t kinds = 0;               // 2 bits for each, the newest lowest: 0 a slab, else 1 + the head's place
    const auto publish = [&]() {      // the oldest group's copies, which have landed, to the tensor cores
        const uint32_t head = (kinds >> (2 * --groups)) & 3;
        ptx::fence_async_shared();
        ptx::mbar_arrive(base + (head ? P::kHFull + 8 * (head - 1) : P::kFull + 8 * (out++ % P::kStages)));
    };
    const auto issued = [&](uint32_t kind) {
        asm volatile("cp.async.commit_group;" ::: "memory");
        kinds = kinds << 2 | kind;
        if (++groups > kAhead) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kAhead) : "memory");
            publish();
        }
    };
    // before a wait, everything asked for becomes known: the others may need it to come to what is waited for
    const auto wait = [&](uint32_t bar, uint32_t parity) {
        if (!__all_sync(0xffffffffu, ptx::mbar_try_wait(bar, parity))) {
            cp_async_wait_all();
            while (groups > 0) publish();
        }
        return warp_wait(bar, parity, abort_flag);
    };
    bool ok = true;
    for (Units u; ok && u.next(p, a.units);) {
        const uint4 *s0 = a.s_images + image_at<KT>(p, u.slot, u.h, 0), *s1 = a.ds_images + image_at<KT>(p, u.slot, u.h, 0);
        const bf16 *rows[2];  // four threads to a row of 64 bytes, eight rows to a warp's copy
#pragma unroll
        for (int x = 0; x < 2; ++x)
            rows[x] = a.dout + (u.at.row + x * 32 + (id >> 2)) * vst + (int64_t)u.h * p.dv + (id & 3) * 8;
        const int64_t y_off = a.ys - a.dout, r_off = a.resid - a.dout;
        for (int s = 0; s < slabs; ++s, ++ns) {
            const int sg = ns % P::kStages;
            if (ns >= P::kStages && !(ok = wait(base + P::kEmpty + 8 * sg, (ns / P::kStages + 1) & 1))) break;
            const uint32_t to = base + P::kOffSlab + sg * P::kSlab;
            const int here = min(2, tiles - 2 * s) * KT * 512;
            if (id == 0) {
                ptx::mbar_expect_tx(base + P::kFull + 8 * sg, 2 * here);
                ptx::bulk_load_g2s(to + P::kRows, s0 + s * 2 * KT * 32, here, base + P::kFull + 8 * sg);
                ptx::bulk_load_g2s(to + P::kRows + P::kImage, s1 + s * 2 * KT * 32, here, base + P::kFull + 8 * sg);
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int t = x * 32 + (id >> 2), w = id & 3;
                const bool has = t < u.at.len && s * 32 + w * 8 < p.dv;
                const bf16 *from = has ? rows[x] + s * 32 : a.dout;
                const uint32_t dst = to + w * 3 * kG * 16 + t * 16;
                cp_async16(dst, from, has);
                cp_async16(dst + kG * 16, has ? from + y_off : a.ys, has);
                cp_async16(dst + 2 * kG * 16, has ? from + r_off : a.resid, has);
            }
            issued(0);
        }
        if (!ok) break;
        const int hb = u.n & 1, hk = u.h / p.group();
        if (u.n >= 2 && !(ok = wait(base + P::kHEmpty + 8 * hb, (u.n / 2 + 1) & 1))) break;
        const uint32_t ka = base + P::kOffHead + hb * P::kHead;
        const int t = id & 63;  // two threads to a row, neighbouring rows in a warp
        const bf16 *kr = a.k + ((u.at.row + t) * p.Hk + hk) * p.dk, *qr = a.q + ((u.at.row + t) * p.Hk + hk) * p.dk;
        for (int x = id >> 6; x < KT * 2; x += 2) {
            const bool has = t < u.at.len && x * 8 < p.dk;
            cp_async16(ka + x * kG * 16 + t * 16, has ? kr + x * 8 : a.k, has);
            cp_async16(ka + P::kTile + x * kG * 16 + t * 16, has ? qr + x * 8 : a.q, has);
        }
        issued(1 + hb);
    }
    cp_async_wait_all();
    while (ok && groups > 0) publish();
    if (!ok) {  // nothing may be in flight into a block that ends early
        *abort_flag = 1;
        for (int i = 0; i < P::kStages; ++i)
            for (int par = 0; par < 2; ++par) ptx::mbar_wait(base + P::kFull + 8 * i, par, nullptr, kWaitNs / 1000);
    }
}

// One thread: the products of the slabs into D1, D2 and D3, and of R' and N into D4 and D5 as soon as an epilogue has
// them ready.
template <int KT>
__device__ __forceinline__ bool grad_issue(const Shape &p, const GradArgs &a, char *sm, uint32_t tmem) {
    using P = GradPlan<KT>;
    const uint32_t base = ptx::smem_u32(sm);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + P::kAbort);
    const int tiles = (p.dv + 15) / 16, slabs = (tiles + 1) / 2;
    constexpr uint32_t i_state = ptx::idesc_bf16(128, P::kN, 0, 1), i_rows = ptx::idesc_bf16(128, kG, 0, 0),
                       i_flip = ptx::idesc_bf16(128, P::kN, 1, 1);
    const auto inside = [&](int n) {  // D4 and D5 of unit n
        ptx::tc_fence_after();
        const uint32_t d = tmem + (n % P::kSets) * P::kSetCols, head = base + P::kOffHead + (n & 1) * P::kHead;
        const uint32_t own = base + P::kOffT, flip = own + P::kOwn;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const uint64_t kd = ptx::smem_desc(head + s * 256, 128, kG * 16, ptx::kSwizzleNone),
                           qd = ptx::smem_desc(head + P::kTile + s * 256, 128, kG * 16, ptx::kSwizzleNone);
            ptx::mma_ss(d, ptx::smem_desc(own + s * 2 * 2 * kG * 16, 2 * kG * 16, 128, ptx::kSwizzleNone), kd, i_state, s > 0);
            ptx::mma_ss(d + P::kN, ptx::smem_desc(flip + s * 256, 128, kG * 16, ptx::kSwizzleNone), qd, i_flip, s > 0);
            ptx::mma_ss(d + P::kN, ptx::smem_desc(flip + 8 * kG * 16 + s * 256, 128, kG * 16, ptx::kSwizzleNone), kd, i_flip, 1);
        }
        ptx::mma_commit(base + P::kInFull + 8 * (n & 1));
    };
    int ns = 0, waiting = -1;  // a unit whose R' and N are still to come
    const auto ready = [&](int n) { return base + P::kReady + 8 * (n & 1); };
    for (Units u; u.next(p, a.units);) {
        const int set = u.n % P::kSets;
        if (u.n >= P::kSets &&
            !ptx::mbar_wait(base + P::kAccFree + 8 * set, (u.n / P::kSets + 1) & 1, abort_flag, kWaitNs))
            return false;
        const uint32_t d = tmem + set * P::kSetCols;
        for (int s = 0; s < slabs; ++s, ++ns) {
            const int sg = ns % P::kStages;
            // Until the slab is there, R' and N of the unit before may become ready; they do not wait for it, since the
            // slab may be waiting for them (a head is free once its epilogue is done).
            const uint64_t t0 = ptx::globaltimer();
            while (!ptx::mbar_try_wait(base + P::kFull + 8 * sg, (ns / P::kStages) & 1)) {
                if (waiting >= 0 && ptx::mbar_try_wait(ready(waiting), (waiting / 2) & 1)) {
                    inside(waiting);
                    waiting = -1;
                }
                if (*abort_flag || ptx::globaltimer() - t0 > kWaitNs) return false;
            }
            ptx::tc_fence_after();
            const uint32_t rows = base + P::kOffSlab + sg * P::kSlab, image = rows + P::kRows;
            for (int x = 0; x < min(2, tiles - 2 * s); ++x) {
                constexpr uint32_t kUnit = 3 * kG * 16;
                const uint32_t r = rows + x * 2 * kUnit, i = image + x * KT * 512;
                const uint32_t more = s > 0 || x > 0;
                const uint64_t top = ptx::smem_desc(r, kUnit, 128, ptx::kSwizzleNone);
                ptx::mma_ss(d, top, ptx::smem_desc(i, 128, 256, ptx::kSwizzleNone), i_state, more);
                ptx::mma_ss(d + P::kN, ptx::smem_desc(r + kG * 16, kUnit, 128, ptx::kSwizzleNone),
                            ptx::smem_desc(i + P::kImage, 128, 256, ptx::kSwizzleNone), i_state, more);
                ptx::mma_ss(d + 2 * P::kN, top, ptx::smem_desc(r + 2 * kG * 16, kUnit, 128, ptx::kSwizzleNone), i_rows, more);
            }
            ptx::mma_commit(base + P::kEmpty + 8 * sg);
            if (waiting >= 0 && ptx::mbar_try_wait(ready(waiting), (waiting / 2) & 1)) {
                inside(waiting);
                waiting = -1;
            }
        }
        ptx::mma_commit(base + P::kAccFull + 8 * set);
        if (waiting >= 0) {
            if (!ptx::mbar_wait(ready(waiting), (waiting / 2) & 1, abort_flag, kWaitNs)) return false;
            inside(waiting);
        }
        waiting = u.n;
        if (P::kSets == 1) {  // the next unit's products need this one's accumulators
            if (!ptx::mbar_wait(ready(waiting), (waiting / 2) & 1, abort_flag, kWaitNs)) return false;
            inside(waiting);
            waiting = -1;
        }
    }
    if (waiting >= 0) {
        if (!ptx::mbar_wait(ready(waiting), (waiting / 2) & 1, abort_flag, kWaitNs)) return false;
        inside(waiting);
    }
    return true;
}

// Three warps: <S0, dS1> of each unit, as the slabs come by; the first also the products of the unit's decays.
template <int KT>
__device__ __forceinline__ bool grad_inner(const Shape &p, const GradArgs &a, char *sm, int warp, int lane) {
    using P = GradPlan<KT>;
    const uint32_t base = ptx::smem_u32(sm);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + P::kAbort);
    const int tiles = (p.dv + 15) / 16, slabs = (tiles + 1) / 2;
    int ns = 0;
    for (Units u; u.next(p, a.units);) {
        float al[2] = {1.f, 1.f}, be[2] = {0.f, 0.f};  // lane owns tokens lane and 32 + lane
        if (warp == 0)
#pragma unroll
            for (int m = 0; m < 2; ++m)
                if (m * 32 + lane < u.at.len) {
                    al[m] = load_gate<bf16>(a.g, (u.at.row + m * 32 + lane) * p.H + u.h, p.gate_f32);
                    be[m] = load_gate<bf16>(a.beta, (u.at.row + m * 32 + lane) * p.H + u.h, p.gate_f32);
                }
        float inner = 0.f;
        for (int s = 0; s < slabs; ++s, ++ns) {
            const int sg = ns % P::kStages;
            if (!warp_wait(base + P::kFull + 8 * sg, (ns / P::kStages) & 1, abort_flag)) return false;
            const uint32_t image = base + P::kOffSlab + sg * P::kSlab + P::kRows;
            for (int i = warp * 32 + lane; i < min(2, tiles - 2 * s) * KT * 32; i += kInnerWarps * 32) {
                const uint4 x = lds128(image + i * 16), y = lds128(image + P::kImage + i * 16);
                const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) inner = fmaf(lo_f(xw[e]), lo_f(yw[e]), fmaf(hi_f(xw[e]), hi_f(yw[e]), inner));
            }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(base + P::kEmpty + 8 * sg);
        }
        for (int m = 16; m > 0; m >>= 1) inner += __shfl_xor_sync(0xffffffffu, inner, m);
        // the epilogue of two units before has read its sums and decays
        const int hb = u.n & 1;
        if (u.n >= 2 && !warp_wait(base + P::kHEmpty + 8 * hb, (u.n / 2 + 1) & 1, abort_flag)) return false;
        if (lane == 0) reinterpret_cast<float *>(sm + P::kOffInner)[hb * 4 + warp] = inner;
        if (warp == 0) {
            Decays &dc = *reinterpret_cast<Decays *>(sm + P::kOffHead + hb * P::kHead + 2 * P::kTile);
            float up[2], down[2];
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const int tok = m * 32 + lane;
                al[m] = tok < u.at.len ? expf(al[m]) : 1.f;
                dc.alpha[tok] = al[m];
                dc.beta[tok] = be[m];
                up[m] = al[m];
                const float behind = __shfl_down_sync(0xffffffffu, al[m], 1);
                down[m] = lane < 31 ? behind : 1.f;  // the product of the next ones, from this one's neighbour on
#pragma unroll
                for (int w = 1; w < 32; w <<= 1) {
                    const float x = __shfl_up_sync(0xffffffffu, up[m], w), y = __shfl_down_sync(0xffffffffu, down[m], w);
                    if (lane >= w) up[m] *= x;
                    if (lane + w < 32) down[m] *= y;
                }
            }
            dc.alpha[kG + (lane & 3)] = 1.f;
            const float first = __shfl_sync(0xffffffffu, up[0], 31), second = __shfl_sync(0xffffffffu, up[1], 31);
            dc.c[lane] = up[0];
            dc.c[32 + lane] = first * up[1];
            dc.d[lane] = down[0] * second;
            dc.d[32 + lane] = down[1];
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(base + P::kInner + 8 * hb);
    }
    return true;
}

// a row of the unit's K or Q tile, eight elements at a time
__device__ __forceinline__ void row8(uint32_t tile, int row, int unit, float (&x)[8]) {
    const uint4 t = lds128(tile + unit * kG * 16 + row * 16);
    const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        x[2 * e] = lo_f(w[e]);
        x[2 * e + 1] = hi_f(w[e]);
    }
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// A warpgroup: every second unit; thread = row of 128 (token row % 64 on the query's or the key's side).
template <int KT>
__device__ __forceinline__ bool grad_epilogue(const Shape &p, const GradArgs &a, char *sm, uint32_t tmem, int group) {
    using P = GradPlan<KT>;
    const uint32_t base = ptx::smem_u32(sm);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + P::kAbort);
    const int id = threadIdx.x & 127, warp = id >> 5, lane = id & 31, i = id & 63;
    const bool key = id >= kG;
    const uint32_t lanes = (uint32_t)(warp * 32) << 16;  // this warp's TMEM lanes
    int turn = 0;
    for (Units u; u.next(p, a.units);) {
        if ((u.n & 1) != group) continue;
        const int set = u.n % P::kSets;
        Sums &sums = reinterpret_cast<Sums *>(sm + P::kOffSums)[group * 2 + (turn++ & 1)];
        const uint32_t head = base + P::kOffHead + group * P::kHead, mine = head + (key ? 0 : P::kTile);
        const Decays &dc = *reinterpret_cast<const Decays *>(sm + P::kOffHead + group * P::kHead + 2 * P::kTile);
        const uint32_t d = tmem + set * P::kSetCols + lanes;
        bool ok = warp_wait(base + P::kAccFull + 8 * set, (u.n / P::kSets) & 1, abort_flag) &&
                  warp_wait(base + P::kInner + 8 * group, (u.n / 2) & 1, abort_flag) &&
                  warp_wait(base + P::kHFull + 8 * group, (u.n / 2) & 1, abort_flag);
        float A[P::kN], w = 0.f, x = 0.f;
        if (ok) {
            ptx::tc_fence_after();
            const float be = dc.beta[i], f1 = key ? -dc.c[i] * be : dc.c[i], f2 = dc.d[i] * be;
#pragma unroll
            for (int b = 0; b < P::kN; b += 32) {
                uint32_t r[32];
                ptx::tmem_ld32(d + b, r);
                ptx::tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) A[b + e] = f1 * __uint_as_float(r[e]);
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    float m[8];
                    row8(mine, i, (b + e) / 8, m);
#pragma unroll
                    for (int y = 0; y < 8; ++y) w = fmaf(m[y], A[b + e + y], w);
                }
                if (key) {
                    ptx::tmem_ld32(d + P::kN + b, r);
                    ptx::tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        float m[8];
                        row8(mine, i, (b + e) / 8, m);
#pragma unroll
                        for (int y = 0; y < 8; ++y) {
                            const float v = f2 * __uint_as_float(r[e + y]);
                            x = fmaf(m[y], v, x);
                            A[b + e + y] += v;
                        }
                    }
                }
            }
            (key ? sums.wk : sums.wq)[i] = w;
            if (key) sums.x[i] = x;
            // R' (query) or N (key), from the row's end: f = D_ij, zero for j > i
            const uint32_t own = base + P::kOffT, flip = own + P::kOwn;
            const float g = key ? -be : 1.f;
            // the products of the unit before have read their R' and N
            if (u.n > 0) ok = warp_wait(base + P::kInFull + 8 * (1 - group), ((u.n - 1) / 2) & 1, abort_flag);
            float f = 0.f;
#pragma unroll
            for (int b = 32; b >= 0; b -= 32) {
                uint32_t r[32];
                ptx::tmem_ld32(d + 2 * P::kN + b, r);
                ptx::tmem_wait_ld();
                if (key && i >= b && i < b + 32) {
                    float own_beta = 0.f;
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (b + e == i) own_beta = __uint_as_float(r[e]);
                    if (i < u.at.len) store_gate<bf16>(a.dbeta, (u.at.row + i) * p.H + u.h, p.gate_f32, own_beta);
                }
#pragma unroll
                for (int e0 = 24; e0 >= 0; e0 -= 8) {
                    float v[8];
#pragma unroll
                    for (int e = 7; e >= 0; --e) {
                        const int j = b + e0 + e;
                        f = j == i ? 1.f : f * dc.alpha[j + 1];
                        const float z = f * dc.beta[j] * g * __uint_as_float(r[e0 + e]);
                        v[e] = key && j == i ? 0.f : z;
                    }
                    const uint32_t q0 = pack(v[0], v[1]), q1 = pack(v[2], v[3]), q2 = pack(v[4], v[5]), q3 = pack(v[6], v[7]);
                    const uint32_t unit = (b + e0) / 8;
                    sts128(own + unit * 2 * kG * 16 + id * 16, q0, q1, q2, q3);
                    if (key) {
                        sts128(flip + unit * kG * 16 + i * 16, q0, q1, q2, q3);
                        sts128(flip + (16 + unit) * kG * 16 + i * 16, q0, q1, q2, q3);
                    } else {
                        sts128(flip + (8 + unit) * kG * 16 + i * 16, q0, q1, q2, q3);
                    }
                }
            }
            ptx::fence_async_shared();
            ptx::tc_fence_before();
        }
        ptx::mbar_arrive(base + P::kReady + 8 * group);
        ok = ok && warp_wait(base + P::kInFull + 8 * group, (u.n / 2) & 1, abort_flag);
        if (ok) {
            ptx::tc_fence_after();
            float m = 0.f;
#pragma unroll
            for (int b = 0; b < P::kN; b += 32) {
                uint32_t r[32], t[32];
                ptx::tmem_ld32(d + b, r);
                if (key) ptx::tmem_ld32(d + P::kN + b, t);
                ptx::tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    float v[8];
                    row8(mine, i, (b + e) / 8, v);
#pragma unroll
                    for (int y = 0; y < 8; ++y) {
                        const float n = __uint_as_float(r[e + y]), o = key ? __uint_as_float(t[e + y]) : 0.f;
                        m = fmaf(v[y], o - n, m);
                        A[b + e + y] += n + o;
                    }
                }
            }
            ptx::tc_fence_before();
            (key ? sums.mk : sums.mq)[i] = m;
        }
        ptx::mbar_arrive(base + P::kAccFree + 8 * set);
        if (ok && i < u.at.len) {
            const int64_t to = ((u.at.row + i) * p.H + u.h) * p.dk;
            if (a.dq_part == nullptr) {
                uint4 *out = reinterpret_cast<uint4 *>((key ? a.dk : a.dq) + to);
#pragma unroll
                for (int e = 0; e < P::kN; e += 8)
                    if (e < p.dk)
                        out[e / 8] = make_uint4(pack(A[e], A[e + 1]), pack(A[e + 2], A[e + 3]), pack(A[e + 4], A[e + 5]),
                                                pack(A[e + 6], A[e + 7]));
            } else {
                float4 *out = reinterpret_cast<float4 *>((key ? a.dk_part : a.dq_part) + to);
#pragma unroll
                for (int e = 0; e < P::kN; e += 4)
                    if (e < p.dk) out[e / 4] = make_float4(A[e], A[e + 1], A[e + 2], A[e + 3]);
            }
        }
        // all sums of the unit are there
        if (group == 0 ? any_of<1, 128>(!ok) : any_of<2, 128>(!ok)) return false;
        if (warp == 0) {  // dg: lane owns tokens 2 lane and 2 lane + 1
            const float *in = reinterpret_cast<const float *>(sm + P::kOffInner) + (u.n & 1) * 4;
            const float f = ((in[0] + in[1]) + in[2]) * dc.c[kG - 1];
            const int j = 2 * lane;
            const float w0 = sums.wq[j] + sums.wk[j], w1 = sums.wq[j + 1] + sums.wk[j + 1];
            const float x0 = sums.x[j] + (sums.mq[j] + sums.mk[j]), x1 = sums.x[j + 1] + (sums.mq[j + 1] + sums.mk[j + 1]);
            float pre = x0 + x1, suf = w0 + w1;
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const float y = __shfl_up_sync(0xffffffffu, pre, m), z = __shfl_down_sync(0xffffffffu, suf, m);
                if (lane >= m) pre += y;
                if (lane + m < 32) suf += z;
            }
            const float left = pre - (x0 + x1);  // tokens before 2 lane
            if (j < u.at.len) store_gate<bf16>(a.dg, (u.at.row + j) * p.H + u.h, p.gate_f32, f + left + suf);
            if (j + 1 < u.at.len) store_gate<bf16>(a.dg, (u.at.row + j + 1) * p.H + u.h, p.gate_f32, f + left + x0 + (suf - w0));
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(base + P::kHEmpty + 8 * group);
    }
    return true;
}

template <int KT>
__global__ void __launch_bounds__(kGradThreads, 1)
delta_grad_kernel(Shape p, GradArgs a) {
    using P = GradPlan<KT>;
    extern __shared__ __align__(128) char sm_raw[];
    const uint32_t base = ptx::smem_u32(sm_raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(base + P::kHFull + 8 * i, 128);
            ptx::mbar_init(base + P::kHEmpty + 8 * i, 4);
            ptx::mbar_init(base + P::kAccFull + 8 * i, 1);
            ptx::mbar_init(base + P::kAccFree + 8 * i, 128);
            ptx::mbar_init(base + P::kReady + 8 * i, 128);
            ptx::mbar_init(base + P::kInFull + 8 * i, 1);
            ptx::mbar_init(base + P::kInner + 8 * i, kInnerWarps);
        }
        for (int i = 0; i < P::kStages; ++i) {
            ptx::mbar_init(base + P::kFull + 8 * i, 129);   // the fetching threads, and the states' bytes
            ptx::mbar_init(base + P::kEmpty + 8 * i, 1 + kInnerWarps);
        }
        *reinterpret_cast<volatile int *>(sm_raw + P::kAbort) = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 12) ptx::tmem_alloc(base + P::kTmem, kTmemCols);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(sm_raw + P::kTmem);
    bool ok = true;
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        ok = grad_epilogue<KT>(p, a, sm_raw, tmem, warp >> 2);
    } else {
        give_registers();
        if (warp < 12) grad_fetch<KT>(p, a, sm_raw);
        else if (warp == 12) { if (lane == 0) ok = grad_issue<KT>(p, a, sm_raw, tmem); }
        else ok = grad_inner<KT>(p, a, sm_raw, warp - 13, lane);
    }
    if (!ok) {
        *reinterpret_cast<volatile int *>(sm_raw + P::kAbort) = 1;
        record_status(GLA_ERR_TIMEOUT);
    }
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();  // every wait above is bounded, so all warps come here
    if (warp == 12) {
        ptx::tmem_relinquish();
        ptx::tmem_dealloc(tmem, kTmemCols);
    }
}

// dq and dk of a key head: the sum over its value heads' parts, four elements a thread, in a fixed order.
__global__ void __launch_bounds__(256)
delta_heads_kernel(const float *__restrict__ dq_part, const float *__restrict__ dk_part, bf16 *__restrict__ dq,
                   bf16 *__restrict__ dk_out, int64_t n, int dk, int group) {
    const float *part = blockIdx.y ? dk_part : dq_part;
    bf16 *out = blockIdx.y ? dk_out : dq;
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;  // element of [rows, Hk, dk]
    if (i >= n) return;
    const float *from = part + (i / dk) * group * dk + i % dk;
    float4 s = *reinterpret_cast<const float4 *>(from);
    for (int m = 1; m < group; ++m) {
        const float4 x = *reinterpret_cast<const float4 *>(from + (int64_t)m * dk);
        s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
    }
    *reinterpret_cast<uint2 *>(out + i) = make_uint2(pack(s.x, s.y), pack(s.z, s.w));
}

struct Workspace {
    size_t again, back, s_images, ds_images, resid, ys, dq_part, dk_part, total;
};
template <int KT> Workspace workspace_kt(const Shape &p) {
    const long long rows = total_rows(p);
    const size_t units = (size_t)chunk_slots(rows, p.nseq, kC) * p.H;
    const size_t image = (size_t)chunk_slots(rows, p.nseq, kG) * p.H * ((p.dv + 15) / 16) * KT * 512;
    const size_t vecs = ((size_t)rows * p.H * p.dv * sizeof(bf16) + 255) / 256 * 256;
    Workspace w{};
    size_t at = 0;
    const auto take = [&at](size_t n) { const size_t x = at; at += (n + 255) / 256 * 256; return x; };
    w.again = take(units * sizeof(AgainRecord));
    w.back = take(units * sizeof(BwdRecord));
    w.s_images = take(image);
    w.ds_images = take(image);
    w.resid = take(vecs);
    w.ys = take(vecs);
    const size_t parts = p.H == p.Hk ? 0 : (size_t)rows * p.H * p.dk * sizeof(float);
    w.dq_part = take(parts);
    w.dk_part = take(parts);
    w.total = at;
    return w;
}

template <int KT>
int bwd_kt(const Shape &p, const bf16 *q, const bf16 *k, const bf16 *v, const void *g, const void *beta,
           const bf16 *dout, const float *h0, const float *dhT, bf16 *dq, bf16 *dk, bf16 *dv, void *dg, void *dbeta,
           float *dh0, char *ws, cudaStream_t st) {
    const Workspace at = workspace_kt<KT>(p);
    const long long rows = total_rows(p), slots = chunk_slots(rows, p.nseq, kG);
    const long long chains = (long long)p.nseq * p.H;
    const int tiles = (p.dv + 15) / 16;
    const Walk wa = make_walk<KT, AgainRecord>(chains, tiles, false, 1),
               wb = make_walk<KT, BwdRecord>(chains, tiles, true, 2);
    const int grad_bytes = GradPlan<KT>::kTotal;
    const long long blocks = chains * wa.splits;
    if (2 * blocks > 0x7fffffffLL || slots * p.H > 0x7fffffffLL) return GLA_ERR_UNSUPPORTED;
    const int walks_bytes = max(walk_bytes(wa), walk_bytes(wb));
    if (!allow_smem<delta_walks_kernel<KT>>() || !allow_smem<delta_grad_kernel<KT>>())
        return GLA_ERR_LAUNCH;
    int rc = mma_prep_grad(p, q, k, g, beta, ws + at.again, ws + at.back, st);
    if (rc != GLA_OK) return rc;
    bf16 *resid = (bf16 *)(ws + at.resid), *ys = (bf16 *)(ws + at.ys);
    uint4 *s_img = (uint4 *)(ws + at.s_images), *ds_img = (uint4 *)(ws + at.ds_images);
    const WalkArgs wargs{q, k, v, dout, (const AgainRecord *)(ws + at.again), (const BwdRecord *)(ws + at.back), h0, dhT,
                         resid, ys, dv, s_img, ds_img, dh0};
    delta_walks_kernel<KT><<<(unsigned)(2 * blocks), (wb.groups + 1) * 128, walks_bytes, st>>>(p, wa, wb, (unsigned)blocks,
                                                                                          wargs);
    count_launches(1);
    if (rows > 0) {
        const bool single = p.H == p.Hk;
        GradArgs a{q, k, dout, g, beta, resid, ys, s_img, ds_img, dq, dk, single ? nullptr : (float *)(ws + at.dq_part),
                   single ? nullptr : (float *)(ws + at.dk_part), dg, dbeta, (unsigned)(slots * p.H)};
        const unsigned sms = (unsigned)device_info().sm_count;
        delta_grad_kernel<KT><<<a.units < sms ? a.units : sms, kGradThreads, grad_bytes, st>>>(p, a);
        count_launches(1);
        if (!single) {
            const int64_t n = (int64_t)rows * p.Hk * p.dk;
            const dim3 grid((unsigned)((n / 4 + 255) / 256), 2);
            delta_heads_kernel<<<grid, 256, 0, st>>>(a.dq_part, a.dk_part, dq, dk, n, p.dk, p.group());
            count_launches(1);
        }
    }
    return cudaGetLastError() == cudaSuccess ? GLA_OK : GLA_ERR_LAUNCH;
}

}  // namespace

// bf16 with dk <= 128: a warp's share of the state fits its registers.
bool mma_bwd_supported(int dk) { return dk <= 128; }

size_t mma_bwd_workspace(const Shape &p) {
#define GLA_CALL(KT) return workspace_kt<KT>(p).total
    GLA_BY_KT(p.dk, GLA_CALL);
#undef GLA_CALL
}

int mma_bwd(const Shape &p, const void *q, const void *k, const void *v, const void *g, const void *beta,
            const void *dout, const float *h0, const float *dhT, void *dq, void *dk, void *dv, void *dg, void *dbeta,
            float *dh0, void *ws, cudaStream_t st) {
#define GLA_CALL(KT)                                                                                                 \
    return bwd_kt<KT>(p, (const bf16 *)q, (const bf16 *)k, (const bf16 *)v, g, beta, (const bf16 *)dout, h0, dhT,    \
                      (bf16 *)dq, (bf16 *)dk, (bf16 *)dv, dg, dbeta, dh0, (char *)ws, st)
    GLA_BY_KT(p.dk, GLA_CALL);
#undef GLA_CALL
}

}  // namespace delta
}  // namespace gla
