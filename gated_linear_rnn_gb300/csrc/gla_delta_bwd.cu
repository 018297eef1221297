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
//
// Eight sequences of 2,048 tokens, 16 heads of 96/192: 550 us: preparation 54, both walks 223 (260 before the fetching
// warps gave registers to the computing ones), gradient kernel 269.  The walks run in one launch since neither fills
// the GPU alone on a small batch; on a large one shared
// memory's pipe (70% busy) and mma.sync's (54%) bound them.
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
// D_ij comes from products of decays alone (a decay of zero is as good as any): within 16 tokens as a table, across
// them as (from the tile's start to i)(whole tiles between)(from j to its tile's end).
//
// One block per SM walks over units.  Twelve warps compute, in three roles of four (16 tokens each): dO's side (T = dO
// R^T, dO S0^T, R' K -> dq), Y's (Y R^T, Y S0^T, N K) and R's (R dS1^T, R'^T Q + N^T K); the last two meet in
// shared memory -> dk.  A fourth warpgroup fetches ahead: K, Q and the decay products of the next unit, and
// slabs of 64 columns (32 for dk > 96) of dO, Y, R and of both states through a ring.
// On the layer's gradient (4,096 units of 64 x 96 x 192, 790 MB): 266 us, of which the slabs' products are about 115,
// T with R' and N 70 and the products inside the unit 50: the phases of a unit follow one another, and shared memory
// carries every state element to four warps.  One block per unit with its states read from L2 between products
// took 489 us, slabs of 32 columns 275, and the same unit with all products on tcgen05 (128 rows of TMEM, one thread
// per row of dq and dk, two epilogues in turn) 281: its products took no time, but its unit waited through more
// hands, each of a microsecond, than its two sets of accumulators could cover.
constexpr int kGradWarps = 12;
constexpr int kGradThreads = (kGradWarps + 4) * 32;
constexpr int kMRow = kG * 2 + 16;  // bytes of a row of R' and N

struct Decays {                     // of one unit
    float diag[4][256];             // D within a tile of 16 tokens
    float pre[kG], suf[kG], c[kG], d[kG], beta[kG], whole[4], pad[4];
};
struct Sums {                       // per token
    float wq[kG], wk[kG], x[kG], mq[kG], my[kG], mr[kG], inner[kGradWarps], pad[4];
};
template <int KT> struct GradPlan {
    static constexpr int kTile = kG * row_bytes<KT>();
    static constexpr int kHead = 2 * kTile + (int)sizeof(Decays);                  // K | Q | decays, two of them
    static constexpr int kTiles = KT <= 6 ? 4 : 2;                                 // column tiles of 16 in a slab
    static constexpr int kSlabRow = kTiles * 32 + 16;                              // an odd number of 16-byte units
    static constexpr int kImage = kTiles * KT * 512;                               // its column tiles of a state
    static constexpr int kSlab = 3 * kG * kSlabRow + 2 * kImage;                   // dO | Y | R | S0 | dS1
    static constexpr int kStages = 2;
    static constexpr int kXRow = KT * 16 + 4;                                      // f32 row of the exchange tile
    static constexpr int kOffHead = 128, kOffSlab = kOffHead + 2 * kHead, kOffM = kOffSlab + kStages * kSlab,
                         kOffX = kOffM + 2 * kG * kMRow, kOffSums = kOffX + kG * kXRow * 4,
                         kTotal = kOffSums + 2 * (int)sizeof(Sums);
    static_assert(kTotal <= 227 * 1024, "shared memory of a block");
    static_assert(kTile % 16 == 0 && kHead % 16 == 0 && kSlab % 16 == 0 && kOffX % 16 == 0, "16-byte copies");
};

__device__ __forceinline__ void compute_sync() { ptx::named_bar_sync(1, kGradWarps * 32); }
// acc (16 rows x KT * 16) += A (16 x 16) times 16 rows of a tile
template <int KT>
__device__ __forceinline__ void add_rows(float (&acc)[2 * KT][4], const uint32_t (&a)[4], uint32_t rows, int lane) {
    const uint32_t at = rows + (((lane >> 3) & 1) * 8 + (lane & 7)) * row_bytes<KT>() + ((lane >> 3) >> 1) * 16;
#pragma unroll
    for (int i = 0; i < KT; ++i) {
        uint32_t b[4];
        ldsm4t(b, at + i * 32);
        mma(acc[2 * i], a, b[0], b[1]);
        mma(acc[2 * i + 1], a, b[2], b[3]);
    }
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
    uint32_t x;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(x) : "r"(addr) : "memory");
    return x;
}
// sums over dk of acc's two rows of this lane with the rows of a tile: lo for row gr, hi for row gr + 8
template <int KT>
__device__ __forceinline__ void row_dots(const float (&acc)[2 * KT][4], uint32_t rows, int lane, float &lo, float &hi) {
    const uint32_t at = rows + (lane >> 2) * row_bytes<KT>() + (lane & 3) * 4;
    lo = hi = 0.f;
#pragma unroll
    for (int n = 0; n < 2 * KT; ++n) {
        const uint32_t x = lds32(at + n * 16), y = lds32(at + 8 * row_bytes<KT>() + n * 16);
        lo = fmaf(acc[n][0], lo_f(x), fmaf(acc[n][1], hi_f(x), lo));
        hi = fmaf(acc[n][2], lo_f(y), fmaf(acc[n][3], hi_f(y), hi));
    }
    lo += __shfl_xor_sync(0xffffffffu, lo, 1);
    hi += __shfl_xor_sync(0xffffffffu, hi, 1);
    lo += __shfl_xor_sync(0xffffffffu, lo, 2);
    hi += __shfl_xor_sync(0xffffffffu, hi, 2);
}

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

template <int KT>
__device__ __forceinline__ void grad_fetch(const Shape &p, const GradArgs &a, char *sm) {
    using P = GradPlan<KT>;
    const uint32_t base = ptx::smem_u32(sm);
    const uint32_t hfull = base, hempty = base + 16, full = base + 32, empty = full + 8 * P::kStages;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + 120);
    const int id = threadIdx.x - kGradWarps * 32;
    const int tiles = (p.dv + 15) / 16, slabs = (tiles + P::kTiles - 1) / P::kTiles;
    int n = 0, ns = 0;  // units and slabs so far
    bool ok = true;
    for (unsigned unit = blockIdx.x; ok && unit < a.units; unit += gridDim.x) {
        const int slot = (int)(unit / (unsigned)p.H), h = (int)(unit % (unsigned)p.H), hk = h / p.group();
        ChunkAt at;
        if (!chunk_of_slot<kG>(slot, p, at)) continue;
        const int hb = n & 1;
        if (n >= 2 && !(ok = warp_wait(hempty + 8 * hb, (n / 2 + 1) & 1, abort_flag))) break;
        ++n;
        char *head = sm + P::kOffHead + hb * P::kHead;
        const uint32_t ka = base + P::kOffHead + hb * P::kHead;
        {
            const int t = id >> 1;  // two threads to a row
            const bf16 *kr = a.k + ((at.row + t) * p.Hk + hk) * p.dk, *qr = a.q + ((at.row + t) * p.Hk + hk) * p.dk;
            for (int u = id & 1; u < KT * 2; u += 2) {
                const bool has = t < at.len && u * 8 < p.dk;
                cp_async16(ka + t * row_bytes<KT>() + u * 16, has ? kr + u * 8 : a.k, has);
                cp_async16(ka + P::kTile + t * row_bytes<KT>() + u * 16, has ? qr + u * 8 : a.q, has);
            }
            cp_async_arrive(hfull + 8 * hb);
        }
        // the decays: thread j < 64 is column j of its tile of 16; both warps take all 64 tokens' decays
        Decays &dc = *reinterpret_cast<Decays *>(head + 2 * P::kTile);
        if (id < kG) {
            const int lane = id & 31, b = id >> 4, j = id & 15;
            float al[2];
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const int tok = m * 32 + lane;
                al[m] = tok < at.len ? expf(load_gate<bf16>(a.g, (at.row + tok) * p.H + h, p.gate_f32)) : 1.f;
            }
            dc.beta[id] = id < at.len ? load_gate<bf16>(a.beta, (at.row + id) * p.H + h, p.gate_f32) : 0.f;
            const float mine = id < 32 ? al[0] : al[1];
            float f = 0.f, run = 1.f, pre = 1.f, whole0 = 1.f, whole1 = 1.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float y = __shfl_sync(0xffffffffu, mine, i, 16);
                run *= y;
                if (i == j) pre = run;
                f = i == j ? 1.f : f * y;
                dc.diag[b][i * 16 + j] = f;
                whole0 *= __shfl_sync(0xffffffffu, al[0], i, 16);
                whole1 *= __shfl_sync(0xffffffffu, al[1], i, 16);
            }
            float before = 1.f, after = 1.f;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const float x = __shfl_sync(0xffffffffu, t < 2 ? whole0 : whole1, (t & 1) * 16);
                if (t < b) before *= x;
                if (t > b) after *= x;
                if (id == 0) dc.whole[t] = x;
            }
            dc.pre[id] = pre;
            dc.suf[id] = f;
            dc.c[id] = before * pre;
            dc.d[id] = f * after;
        }
        ptx::mbar_arrive(hfull + 8 * hb);
        const int64_t vst = (int64_t)p.H * p.dv;
        // neighbouring threads to neighbouring units of a row: 2 kTiles of them
        constexpr int kUnits = 2 * P::kTiles, kStep = 128 / kUnits;
        const int t0 = id / kUnits, u0 = id % kUnits;
        const int64_t vat = (at.row + t0) * vst + (int64_t)h * p.dv + u0 * 8;
        const uint4 *s0 = a.s_images + image_at<KT>(p, slot, h, 0), *s1 = a.ds_images + image_at<KT>(p, slot, h, 0);
        for (int s = 0; s < slabs; ++s, ++ns) {
            const int sg = ns % P::kStages;
            if (ns >= P::kStages && !(ok = warp_wait(empty + 8 * sg, (ns / P::kStages + 1) & 1, abort_flag))) break;
            const uint32_t to = base + P::kOffSlab + sg * P::kSlab;
            const int here = min(P::kTiles, tiles - P::kTiles * s) * KT * 512;
            if (id == 0) {
                ptx::mbar_expect_tx(full + 8 * sg, 2 * here);
                ptx::bulk_load_g2s(to + 3 * kG * P::kSlabRow, s0 + s * P::kTiles * KT * 32, here, full + 8 * sg);
                ptx::bulk_load_g2s(to + 3 * kG * P::kSlabRow + P::kImage, s1 + s * P::kTiles * KT * 32, here, full + 8 * sg);
            }
#pragma unroll 4
            for (int t = t0; t < kG; t += kStep) {
                const bool has = t < at.len && s * P::kTiles * 16 + u0 * 8 < p.dv;
                const int64_t off = has ? vat + (t - t0) * vst + s * P::kTiles * 16 : 0;
                const uint32_t dst = to + t * P::kSlabRow + u0 * 16;
                cp_async16(dst, a.dout + off, has);
                cp_async16(dst + kG * P::kSlabRow, a.ys + off, has);
                cp_async16(dst + 2 * kG * P::kSlabRow, a.resid + off, has);
            }
            cp_async_arrive(full + 8 * sg);
        }
    }
    // nothing may be in flight into a block that ends early; a whole walk over units has waited for every stage
    cp_async_wait_all();
    if (!ok) {
        *abort_flag = 1;
        for (int i = 0; i < P::kStages; ++i)
            for (int par = 0; par < 2; ++par) ptx::mbar_wait(full + 8 * i, par, nullptr, kWaitNs / 1000);
    }
}

template <int KT>
__global__ void __launch_bounds__(kGradThreads, 1)
delta_grad_kernel(Shape p, GradArgs a) {
    using P = GradPlan<KT>;
    extern __shared__ __align__(128) char sm_raw[];
    const uint32_t base = ptx::smem_u32(sm_raw);
    const uint32_t hfull = base, hempty = base + 16, full = base + 32, empty = full + 8 * P::kStages;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm_raw + 120);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(hfull + 8 * i, 256);  // the fetching threads' copies, and their decays
            ptx::mbar_init(hempty + 8 * i, kGradWarps);
        }
        for (int i = 0; i < P::kStages; ++i) {
            ptx::mbar_init(full + 8 * i, 129);
            ptx::mbar_init(empty + 8 * i, kGradWarps);
        }
        *abort_flag = 0;
        ptx::fence_mbar_init();
    }
    __syncthreads();
    if (warp >= kGradWarps) {
        give_registers();
        grad_fetch<KT>(p, a, sm_raw);
        return;
    }
    take_registers();
    // A tile of 16 tokens costs the more the further down it lies (T, R', N are triangular); the four SM quarters
    // take warps in turn, so Y's tiles run against dO's.
    const int role = warp >> 2, rt = role == 1 ? 3 - (warp & 3) : warp & 3;
    const int gr = lane >> 2, tg = lane & 3, m8 = lane >> 3, r8 = lane & 7;
    const int row0 = rt * 16 + gr;  // this lane's rows: row0 and row0 + 8
    const int tiles = (p.dv + 15) / 16, slabs = (tiles + P::kTiles - 1) / P::kTiles;
    const uint32_t mt = base + P::kOffM, nt = mt + kG * kMRow;
    float *exchange = reinterpret_cast<float *>(sm_raw + P::kOffX);
    int n = 0, ns = 0;
    for (unsigned unit = blockIdx.x; unit < a.units; unit += gridDim.x) {
        const int slot = (int)(unit / (unsigned)p.H), h = (int)(unit % (unsigned)p.H);
        ChunkAt at;
        if (!chunk_of_slot<kG>(slot, p, at)) continue;
        const int hb = n & 1;
        // a warp whose wait runs out goes on to the next barrier, where all learn of it and leave together
        bool ok = warp_wait(hfull + 8 * hb, (n / 2) & 1, abort_flag);
        Sums &sums = *reinterpret_cast<Sums *>(sm_raw + P::kOffSums + hb * sizeof(Sums));
        ++n;
        const uint32_t ks = base + P::kOffHead + hb * P::kHead, qs = ks + P::kTile;
        const Decays &dc = *reinterpret_cast<const Decays *>(sm_raw + P::kOffHead + hb * P::kHead + 2 * P::kTile);
        // T = do_i . r_j (or y_i . r_j) on and below the diagonal; A: this role's product with a state
        float T[8][4] = {}, A[2 * KT][4] = {}, inner = 0.f;
        for (int s = 0; s < slabs; ++s, ++ns) {
            const int sg = ns % P::kStages;
            ok = ok && warp_wait(full + 8 * sg, (ns / P::kStages) & 1, abort_flag);
            if (!ok) break;
            const uint32_t slab = base + P::kOffSlab + sg * P::kSlab;
            const uint32_t a_at = slab + (role * kG + rt * 16 + (m8 & 1) * 8 + r8) * P::kSlabRow + (m8 >> 1) * 16;
            const uint32_t b_at = slab + (2 * kG + (m8 >> 1) * 8 + r8) * P::kSlabRow + (m8 & 1) * 16;
            const uint32_t image = slab + 3 * kG * P::kSlabRow + (role == 2 ? P::kImage : 0) + lane * 16;  // matrix lane / 8, row lane % 8
            const int here = min(P::kTiles, tiles - P::kTiles * s);
#pragma unroll
            for (int x = 0; x < P::kTiles; ++x) {
                if (x >= here) break;
                uint32_t f[4];
                ldsm4(f, a_at + x * 32);
#pragma unroll
                for (int i = 0; i < KT; ++i) {
                    uint32_t b[4];
                    ldsm4t(b, image + (x * KT + i) * 512);
                    mma(A[2 * i], f, b[0], b[1]);
                    mma(A[2 * i + 1], f, b[2], b[3]);
                }
                if (role < 2) {
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        if (t <= rt) {
                            uint32_t b[4];
                            ldsm4(b, b_at + t * 16 * P::kSlabRow + x * 32);
                            mma(T[2 * t], f, b[0], b[1]);
                            mma(T[2 * t + 1], f, b[2], b[3]);
                        }
                }
            }
            for (int i = tid; i < here * KT * 32; i += kGradWarps * 32) {  // <S0, dS1>
                const uint4 x = lds128(slab + 3 * kG * P::kSlabRow + i * 16),
                            y = lds128(slab + 3 * kG * P::kSlabRow + P::kImage + i * 16);
                const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) inner = fmaf(lo_f(xw[e]), lo_f(yw[e]), fmaf(hi_f(xw[e]), hi_f(yw[e]), inner));
            }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(empty + 8 * sg);
        }
        if (!ok && lane == 0) {
            *abort_flag = 1;
            record_status(GLA_ERR_TIMEOUT);
        }
        for (int m = 16; m > 0; m >>= 1) inner += __shfl_xor_sync(0xffffffffu, inner, m);
        if (lane == 0) sums.inner[warp] = inner;
        float lo, hi;
        // the state's part of dq and dk, and its share of dg
        {
            const float *v = role == 2 ? dc.d : dc.c;
            float f0 = v[row0], f1 = v[row0 + 8];
            if (role > 0) {
                f0 *= role == 1 ? -dc.beta[row0] : dc.beta[row0];
                f1 *= role == 1 ? -dc.beta[row0 + 8] : dc.beta[row0 + 8];
            }
#pragma unroll
            for (int i = 0; i < 2 * KT; ++i) {
                A[i][0] *= f0; A[i][1] *= f0; A[i][2] *= f1; A[i][3] *= f1;
            }
            row_dots<KT>(A, (role ? ks : qs) + rt * 16 * row_bytes<KT>(), lane, lo, hi);
            float *to = role == 0 ? sums.wq : role == 1 ? sums.wk : sums.x;
            if (tg == 0) {
                to[row0] = lo;
                to[row0 + 8] = hi;
            }
        }
        if (role < 2) {  // R' or N
            float between[4];  // whole tiles strictly between tile t and this warp's
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                float f = 1.f;
                for (int m = t + 1; m < rt; ++m) f *= dc.whole[m];
                between[t] = f;
            }
            float own0 = 0.f, own1 = 0.f;  // the diagonal's two elements, where tg == gr / 2
            const float p0 = dc.pre[row0], p1 = dc.pre[row0 + 8];
            const float g0 = role ? -dc.beta[row0] : 1.f, g1 = role ? -dc.beta[row0 + 8] : 1.f;
#pragma unroll
            for (int t = 0; t < 8; ++t)
                if (t <= 2 * rt + 1) {
                    const int j = t * 8 + 2 * tg;
                    const float b0 = dc.beta[j], b1 = dc.beta[j + 1];
                    float x[4];
                    if ((t >> 1) == rt) {
                        const float *D = dc.diag[rt] + gr * 16 + (j & 15);
                        const float2 u = *reinterpret_cast<const float2 *>(D), v = *reinterpret_cast<const float2 *>(D + 128);
                        const int i0 = row0, i1 = row0 + 8, off = role;  // N leaves the diagonal out
                        if (t == 2 * rt) own0 = gr & 1 ? T[t][1] : T[t][0];
                        else own1 = gr & 1 ? T[t][3] : T[t][2];
                        x[0] = j + off <= i0 ? g0 * b0 * u.x * T[t][0] : 0.f;
                        x[1] = j + 1 + off <= i0 ? g0 * b1 * u.y * T[t][1] : 0.f;
                        x[2] = j + off <= i1 ? g1 * b0 * v.x * T[t][2] : 0.f;
                        x[3] = j + 1 + off <= i1 ? g1 * b1 * v.y * T[t][3] : 0.f;
                    } else {
                        const float m = between[t >> 1], s0 = m * dc.suf[j] * b0, s1 = m * dc.suf[j + 1] * b1;
                        x[0] = g0 * p0 * s0 * T[t][0];
                        x[1] = g0 * p0 * s1 * T[t][1];
                        x[2] = g1 * p1 * s0 * T[t][2];
                        x[3] = g1 * p1 * s1 * T[t][3];
                    }
                    char *to = sm_raw + P::kOffM + (role * kG + row0) * kMRow + j * 2;
                    *reinterpret_cast<uint32_t *>(to) = pack(x[0], x[1]);
                    *reinterpret_cast<uint32_t *>(to + 8 * kMRow) = pack(x[2], x[3]);
                }
            if (role && tg == gr >> 1) {
                if (row0 < at.len) store_gate<bf16>(a.dbeta, (at.row + row0) * p.H + h, p.gate_f32, own0);
                if (row0 + 8 < at.len) store_gate<bf16>(a.dbeta, (at.row + row0 + 8) * p.H + h, p.gate_f32, own1);
            }
        }
        if (any_of<1, kGradWarps * 32>(!ok)) return;  // R' and N are whole
        {
            float acc[2 * KT][4] = {};
            if (role < 2) {  // R' K or N K
                const uint32_t own = (role ? nt : mt) + (rt * 16 + (m8 & 1) * 8 + r8) * kMRow + (m8 >> 1) * 16;
                for (int t = 0; t <= rt; ++t) {
                    uint32_t f[4];
                    ldsm4(f, own + t * 32);
                    add_rows<KT>(acc, f, ks + t * 16 * row_bytes<KT>(), lane);
                }
            } else {  // R'^T Q + N^T K
                const uint32_t flip = ((m8 >> 1) * 8 + r8) * kMRow + rt * 32 + (m8 & 1) * 16;
                for (int t = rt; t < 4; ++t) {
                    uint32_t f[4];
                    ldsm4t(f, mt + flip + t * 16 * kMRow);
                    add_rows<KT>(acc, f, qs + t * 16 * row_bytes<KT>(), lane);
                    ldsm4t(f, nt + flip + t * 16 * kMRow);
                    add_rows<KT>(acc, f, ks + t * 16 * row_bytes<KT>(), lane);
                }
            }
            row_dots<KT>(acc, (role ? ks : qs) + rt * 16 * row_bytes<KT>(), lane, lo, hi);
            float *to = role == 0 ? sums.mq : role == 1 ? sums.my : sums.mr;
            if (tg == 0) {
                to[row0] = role == 2 ? lo : -lo;
                to[row0 + 8] = role == 2 ? hi : -hi;
            }
#pragma unroll
            for (int i = 0; i < 2 * KT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) A[i][e] += acc[i][e];
        }
        if (role == 2) {
#pragma unroll
            for (int i = 0; i < 2 * KT; ++i) {
                *reinterpret_cast<float2 *>(exchange + row0 * P::kXRow + i * 8 + 2 * tg) = make_float2(A[i][0], A[i][1]);
                *reinterpret_cast<float2 *>(exchange + (row0 + 8) * P::kXRow + i * 8 + 2 * tg) = make_float2(A[i][2], A[i][3]);
            }
        }
        compute_sync();  // R's part of dk and all sums are there; K, Q and the decays are read
        if (role == 1) {
#pragma unroll
            for (int i = 0; i < 2 * KT; ++i) {
                const float2 u = *reinterpret_cast<const float2 *>(exchange + row0 * P::kXRow + i * 8 + 2 * tg);
                const float2 v = *reinterpret_cast<const float2 *>(exchange + (row0 + 8) * P::kXRow + i * 8 + 2 * tg);
                A[i][0] += u.x; A[i][1] += u.y; A[i][2] += v.x; A[i][3] += v.y;
            }
        }
        if (role < 2 && a.dq_part == nullptr) {
            // 64 columns at a time through this warp's own 16 rows of R' or N, which the barrier has left free
            const uint32_t tile = (role ? nt : mt) + rt * 16 * kMRow;
            bf16 *to = (role ? a.dk : a.dq) + ((at.row + rt * 16) * p.H + h) * p.dk;
#pragma unroll
            for (int i0 = 0; i0 < 2 * KT; i0 += 8) {
                __syncwarp();
#pragma unroll
                for (int i = i0; i < (i0 + 8 < 2 * KT ? i0 + 8 : 2 * KT); i += 2)
                    stsm4(tile + ((m8 & 1) * 8 + r8) * kMRow + (i - i0 + (m8 >> 1)) * 16, pack(A[i][0], A[i][1]),
                          pack(A[i][2], A[i][3]), pack(A[i + 1][0], A[i + 1][1]), pack(A[i + 1][2], A[i + 1][3]));
                __syncwarp();
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int row = x * 4 + (lane >> 3), u = i0 + (lane & 7);
                    if (rt * 16 + row < at.len && u * 8 < p.dk)
                        *reinterpret_cast<uint4 *>(to + (int64_t)row * p.H * p.dk + u * 8) =
                            lds128(tile + row * kMRow + (lane & 7) * 16);
                }
            }
            __syncwarp();
        } else if (role < 2) {
            float *to = (role ? a.dk_part : a.dq_part) + ((at.row + row0) * p.H + h) * p.dk + 2 * tg;
            const int64_t far = (int64_t)8 * p.H * p.dk;
#pragma unroll
            for (int i = 0; i < 2 * KT; ++i)
                if (i * 8 < p.dk) {
                    if (row0 < at.len) *reinterpret_cast<float2 *>(to + i * 8) = make_float2(A[i][0], A[i][1]);
                    if (row0 + 8 < at.len) *reinterpret_cast<float2 *>(to + far + i * 8) = make_float2(A[i][2], A[i][3]);
                }
        }
        if (warp == 8) {  // dg: lane owns tokens 2 lane and 2 lane + 1
            float f = 0.f;
#pragma unroll
            for (int m = 0; m < kGradWarps; ++m) f += sums.inner[m];
            f *= dc.c[kG - 1];
            const int i = 2 * lane;
            const float w0 = sums.wq[i] + sums.wk[i], w1 = sums.wq[i + 1] + sums.wk[i + 1];
            const float x0 = sums.x[i] + (sums.mq[i] + sums.my[i] + sums.mr[i]),
                        x1 = sums.x[i + 1] + (sums.mq[i + 1] + sums.my[i + 1] + sums.mr[i + 1]);
            float pre = x0 + x1, suf = w0 + w1;
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const float u = __shfl_up_sync(0xffffffffu, pre, m), v = __shfl_down_sync(0xffffffffu, suf, m);
                if (lane >= m) pre += u;
                if (lane + m < 32) suf += v;
            }
            const float left = pre - (x0 + x1);  // tokens before 2 lane
            if (i < at.len) store_gate<bf16>(a.dg, (at.row + i) * p.H + h, p.gate_f32, f + left + suf);
            if (i + 1 < at.len) store_gate<bf16>(a.dg, (at.row + i + 1) * p.H + h, p.gate_f32, f + left + x0 + (suf - w0));
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(hempty + 8 * hb);
    }
}

// dq and dk of a key head: the sum over its value heads' parts, four elements a thread, in a fixed order.  Rows of a
// packed batch that are no sequence's have no parts, and stay as they are.
__global__ void __launch_bounds__(256)
delta_heads_kernel(Shape p, const float *__restrict__ dq_part, const float *__restrict__ dk_part, bf16 *__restrict__ dq,
                   bf16 *__restrict__ dk_out, int64_t n) {
    const int dk = p.dk, group = p.group();
    const float *part = blockIdx.y ? dk_part : dq_part;
    bf16 *out = blockIdx.y ? dk_out : dq;
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;  // element of [rows, Hk, dk]
    if (i >= n) return;
    const int2 span = __ldg(p.cu != nullptr ? p.rows + p.nseq : reinterpret_cast<const int2 *>(part));  // on its way with the parts
    const float *from = part + (i / dk) * group * dk + i % dk;
    float4 s = *reinterpret_cast<const float4 *>(from);
    for (int m = 1; m < group; ++m) {
        const float4 x = *reinterpret_cast<const float4 *>(from + (int64_t)m * dk);
        s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
    }
    if (p.cu != nullptr && !in_some_sequence(p, span, i, (int64_t)p.Hk * dk)) return;
    *reinterpret_cast<uint2 *>(out + i) = make_uint2(pack(s.x, s.y), pack(s.z, s.w));
}

struct Workspace {
    size_t again, back, s_images, ds_images, resid, ys, dq_part, dk_part, rows, total;
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
    w.rows = take(rows_bytes(p));
    w.total = at;
    return w;
}

template <int KT>
int bwd_kt(Shape p, const bf16 *q, const bf16 *k, const bf16 *v, const void *g, const void *beta,
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
    place_rows(p, ws + at.rows, 2 * blocks);
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
            delta_heads_kernel<<<grid, 256, 0, st>>>(p, a.dq_part, a.dk_part, dq, dk, n);
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
