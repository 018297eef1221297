// gla_delta_bwd.cu — the gradient of the gated delta rule on the tensor cores (bf16 inputs).
//
// Four kernels, with the notation of gla_delta_mma.cu (dS1: the gradient after a chunk, dS0: before it):
//   delta_prep_kernel  for every chunk of 32 tokens and head: what does not depend on the states.
//   delta_again_kernel walks each chain forwards as the forward does, without its output: the residuals R, and the
//                      state before every 64th token.
//   delta_back_kernel  walks each chain backwards. With dU = P^T dO + diag(d) K dS1 the gradient that reaches a
//                      token's write from outside the chunk and from its reads inside,
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

// S^T's 16 columns as bf16 B operands (k = the 16 columns, n = dk): [KT][32 lanes] x 16 bytes for each column tile,
// so that a warp of the gradient kernel reads 512 neighbouring bytes at a time.
template <int KT>
__device__ __forceinline__ void write_image(uint4 *to, const float (&S)[2 * KT][4], int lane) {
#pragma unroll
    for (int i = 0; i < KT; ++i)
        to[i * 32 + lane] = make_uint4(transpose8(pack(S[2 * i][0], S[2 * i][1])), transpose8(pack(S[2 * i][2], S[2 * i][3])),
                                       transpose8(pack(S[2 * i + 1][0], S[2 * i + 1][1])),
                                       transpose8(pack(S[2 * i + 1][2], S[2 * i + 1][3])));
}
// the image of column tile `tile` of the state of (slot of 64 tokens, head)
template <int KT>
__device__ __forceinline__ int64_t image_at(const Shape &p, int64_t slot, int h, int tile) {
    return ((slot * p.H + h) * ((p.dv + 15) / 16) + tile) * KT * 32;
}

// acc[t] += S^T K^T over the chunk's 32 tokens (t: tiles of 8 tokens), S rounded to bf16
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
        mma(acc[0], a, b0[0], b0[1]);
        mma(acc[1], a, b0[2], b0[3]);
        mma(acc[2], a, b1[0], b1[1]);
        mma(acc[3], a, b1[2], b1[3]);
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

template <int KT>
__global__ void __launch_bounds__(kMaxThreads)
delta_again_kernel(Shape p, Walk w, const bf16 *__restrict__ k, const bf16 *__restrict__ v,
                   const AgainRecord *__restrict__ records, const float *__restrict__ h0, bf16 *__restrict__ resid,
                   uint4 *__restrict__ images) {
    extern __shared__ __align__(128) char sm_raw[];
    constexpr int kTile = kC * row_bytes<KT>();
    const Frame f(p, w, sm_raw);
    if (f.bad && threadIdx.x == 0) record_status(GLA_ERR_DEVICE_ARG);
    if (f.warp >= w.groups * 4) {
        give_registers();
        fetch<KT, false, false>(p, w, f, k, k, v, records);
        return;
    }
    take_registers();
    if (f.warp >= w.warps) return;
    const int lane = f.lane, tg = lane & 3, m8 = lane >> 3, r8 = lane & 7;
    const int col = f.col0 + f.warp * 16;
    const uint32_t tile = f.outs + f.warp * kC * kOutRow;
    const int64_t slot64 = f.r.start / kG + f.s;
    const bool live = col < p.dv;
    float S[2 * KT][4];
    load_state<KT>(S, h0, p, f.chain, col, lane);
    for (int c = 0; c < f.nch; ++c) {
        const int sg = c % w.stages;
        if (!ptx::mbar_wait(f.full + 8 * sg, (c / w.stages) & 1, f.abort_flag, kWaitNs)) {
            if (lane == 0) {
                *f.abort_flag = 1;
                record_status(GLA_ERR_TIMEOUT);
            }
            return;
        }
        if ((c & 1) == 0 && live) write_image<KT>(images + image_at<KT>(p, slot64 + c / 2, f.h, col / 16), S, lane);
        const uint32_t ks = f.ring + sg * w.stage_bytes, vs = ks + kTile + f.warp * 32, rec = ks + kTile + kC * w.vrow;
        const uint32_t vec = rec + (uint32_t)offsetof(AgainRecord, c) + 8 * tg;
        float Y[4][4] = {};
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
        float R[4][4] = {};
        uint4 m[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) m[n] = lds128(rec + n * 512 + lane * 16);
#pragma unroll
        for (int n = 0; n < 4; ++n) mma(R[n], x[0], m[n].x, m[n].y);
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
        for (int n = 0; n < 2 * KT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) S[n][e] *= last;
        add_outer<KT>(S, u, ks, lane);
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(f.empty + 8 * sg);
        write_tile(resid, R, p, f, c, col, tile);
    }
}

template <int KT>
__global__ void __launch_bounds__(kMaxThreads)
delta_back_kernel(Shape p, Walk w, const bf16 *__restrict__ q, const bf16 *__restrict__ k, const bf16 *__restrict__ dout,
                  const BwdRecord *__restrict__ records, const float *__restrict__ dhT, bf16 *__restrict__ ys,
                  bf16 *__restrict__ dv, uint4 *__restrict__ images, float *__restrict__ dh0) {
    extern __shared__ __align__(128) char sm_raw[];
    constexpr int kTile = kC * row_bytes<KT>();
    const Frame f(p, w, sm_raw);
    if (f.bad && threadIdx.x == 0) record_status(GLA_ERR_DEVICE_ARG);
    if (f.warp >= w.groups * 4) {
        give_registers();
        fetch<KT, true, true>(p, w, f, q, k, dout, records);
        return;
    }
    take_registers();
    if (f.warp >= w.warps) return;
    const int lane = f.lane, tg = lane & 3, m8 = lane >> 3, r8 = lane & 7;
    const int col = f.col0 + f.warp * 16;
    const uint32_t tile = f.outs + f.warp * kC * kOutRow;
    const int64_t slot64 = f.r.start / kG + f.s;
    const bool live = col < p.dv;
    float S[2 * KT][4];
    load_state<KT>(S, dhT, p, f.chain, col, lane);
    for (int i = 0; i < f.nch; ++i) {
        const int c = f.nch - 1 - i, sg = i % w.stages;
        if (!ptx::mbar_wait(f.full + 8 * sg, (i / w.stages) & 1, f.abort_flag, kWaitNs)) {
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
        float U[4][4] = {};
        state_times_rows<KT>(U, S, ks, lane);
        uint4 m[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const float2 d = lds_f2(vec + 4 * kC + n * 32);
            U[n][0] *= d.x; U[n][1] *= d.y; U[n][2] *= d.x; U[n][3] *= d.y;
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
        float Y[4][4] = {};
#pragma unroll
        for (int n = 0; n < 4; ++n) mma(Y[n], u[1], m[n].z, m[n].w);
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
        for (int n = 0; n < 2 * KT; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x) S[n][x] *= last;
        add_outer<KT>(S, a, qs, lane);
        add_outer<KT>(S, e, ks, lane);
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(f.empty + 8 * sg);
        write_tile(ys, Y, p, f, c, col, tile);
        write_tile(dv, D, p, f, c, col, tile);
    }
    if (dh0 != nullptr) store_state<KT>(dh0, S, p, f.chain, col, lane);
}

// ---- dq, dk, dg, dbeta -----------------------------------------------------------------------------------------
//
// One block per 64 tokens and key head, eight warps: warps 0-3 own 16 tokens each of the query's side, warps 4-7
// of the key's.  With D_ij, c_i and d_j over the 64 tokens,
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
constexpr int kGradThreads = 256;
constexpr int kMRow = kG * 2 + 16;  // bytes of a row of R' and N

struct GradPlan {
    int vrow;                                 // bytes of a row of dO, Y, R
    int off_q, off_do, off_y, off_r, off_m, off_n, off_f, total;
};
template <int KT>
__host__ __device__ inline GradPlan grad_plan(int dv) {
    GradPlan g{};
    g.vrow = ((dv + 15) / 16 * 2 | 1) * 16;
    g.off_q = kG * row_bytes<KT>();
    g.off_do = 2 * g.off_q;
    g.off_y = g.off_do + kG * g.vrow;
    g.off_r = g.off_y + kG * g.vrow;
    g.off_m = g.off_r + kG * g.vrow;
    g.off_n = g.off_m + kG * kMRow;
    g.off_f = g.off_n + kG * kMRow;
    g.total = g.off_f + (4 * 256 + 11 * kG + 16) * 4;
    return g;
}

// rows of 64 tokens into shared memory, zero past len and past n; asynchronous
__device__ __forceinline__ void fetch_tile(uint32_t dst, int row_bytes_, int units, const bf16 *src, int64_t stride, int len,
                                           int n) {
    for (int e = threadIdx.x; e < kG * 4; e += kGradThreads) {
        const int t = e >> 2;
        for (int u = e & 3; u < units; u += 4) {
            const bool has = t < len && u * 8 < n;
            cp_async16(dst + t * row_bytes_ + u * 16, has ? src + t * stride + u * 8 : src, has);
        }
    }
}

// acc (16 rows x KT * 16) += rows (16 x dv, from shared memory) times an image (dv x dk, from global memory)
template <int KT>
__device__ __forceinline__ void rows_times_image(float (&acc)[2 * KT][4], uint32_t rows, int vrow, const uint4 *image,
                                                 int tiles, int lane) {
    const uint32_t at = rows + (((lane >> 3) & 1) * 8 + (lane & 7)) * vrow + ((lane >> 3) >> 1) * 16;
    for (int s = 0; s < tiles; ++s) {
        uint32_t a[4];
        uint4 b[KT];
#pragma unroll
        for (int i = 0; i < KT; ++i) b[i] = __ldg(image + (s * KT + i) * 32 + lane);
        ldsm4(a, at + s * 32);
#pragma unroll
        for (int i = 0; i < KT; ++i) {
            mma(acc[2 * i], a, b[i].x, b[i].y);
            mma(acc[2 * i + 1], a, b[i].z, b[i].w);
        }
    }
}
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
// sums over dk of acc's two rows of this lane with the rows of a tile: lo for row gr, hi for row gr + 8
template <int KT>
__device__ __forceinline__ void row_dots(const float (&acc)[2 * KT][4], uint32_t rows, int lane, float &lo, float &hi) {
    const uint32_t at = rows + (lane >> 2) * row_bytes<KT>() + (lane & 3) * 4;
    lo = hi = 0.f;
#pragma unroll
    for (int n = 0; n < 2 * KT; ++n) {
        uint32_t x, y;
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(x) : "r"(at + n * 16) : "memory");
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(y) : "r"(at + 8 * row_bytes<KT>() + n * 16) : "memory");
        lo = fmaf(acc[n][0], lo_f(x), fmaf(acc[n][1], hi_f(x), lo));
        hi = fmaf(acc[n][2], lo_f(y), fmaf(acc[n][3], hi_f(y), hi));
    }
    lo += __shfl_xor_sync(0xffffffffu, lo, 1);
    hi += __shfl_xor_sync(0xffffffffu, hi, 1);
    lo += __shfl_xor_sync(0xffffffffu, lo, 2);
    hi += __shfl_xor_sync(0xffffffffu, hi, 2);
}

template <int KT>
__global__ void __launch_bounds__(kGradThreads)
delta_grad_kernel(Shape p, const bf16 *__restrict__ q, const bf16 *__restrict__ k, const bf16 *__restrict__ dout,
                  const void *__restrict__ g, const void *__restrict__ beta, const bf16 *__restrict__ resid,
                  const bf16 *__restrict__ ys, const uint4 *__restrict__ s_images, const uint4 *__restrict__ ds_images,
                  bf16 *__restrict__ dq, bf16 *__restrict__ dk, void *__restrict__ dg, void *__restrict__ dbeta) {
    extern __shared__ __align__(128) char sm_raw[];
    const GradPlan pl = grad_plan<KT>(p.dv);
    const int slot = (int)(blockIdx.x / (unsigned)p.Hk), hk = (int)(blockIdx.x % (unsigned)p.Hk);
    ChunkAt at;
    if (!chunk_of_slot<kG>(slot, p, at)) return;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rt = warp & 3, gr = lane >> 2, tg = lane & 3;
    const bool key = warp >= 4;
    const int m8 = lane >> 3, r8 = lane & 7;
    const uint32_t base = ptx::smem_u32(sm_raw), ks = base, qs = base + pl.off_q, dos = base + pl.off_do,
                   yss = base + pl.off_y, rss = base + pl.off_r;
    char *Mt = sm_raw + pl.off_m, *Nt = sm_raw + pl.off_n;
    float *diag = reinterpret_cast<float *>(sm_raw + pl.off_f);  // [4][16][16]: D within a tile of 16 tokens
    float *pre = diag + 4 * 256, *suf = pre + kG, *cc = suf + kG, *dd = cc + kG, *be = dd + kG, *al = be + kG,
          *wq = al + kG, *wk = wq + kG, *xs = wk + kG, *mq = xs + kG, *mk = mq + kG, *part = mk + kG, *whole = part + 8;
    const int row0 = rt * 16 + gr;  // this lane's rows: row0 and row0 + 8
    const int tiles = (p.dv + 15) / 16;
    fetch_tile(ks, row_bytes<KT>(), KT * 2, k + (at.row * p.Hk + hk) * p.dk, (int64_t)p.Hk * p.dk, at.len, p.dk);
    fetch_tile(qs, row_bytes<KT>(), KT * 2, q + (at.row * p.Hk + hk) * p.dk, (int64_t)p.Hk * p.dk, at.len, p.dk);
    float total[2 * KT][4] = {};  // dq's or dk's rows, over the value heads of this key head
    for (int h = hk * p.group(); h < (hk + 1) * p.group(); ++h) {
        const int64_t vat = (at.row * p.H + h) * p.dv, vst = (int64_t)p.H * p.dv;
        fetch_tile(dos, pl.vrow, tiles * 2, dout + vat, vst, at.len, p.dv);
        fetch_tile(yss, pl.vrow, tiles * 2, ys + vat, vst, at.len, p.dv);
        fetch_tile(rss, pl.vrow, tiles * 2, resid + vat, vst, at.len, p.dv);
        const uint4 *s0 = s_images + image_at<KT>(p, slot, h, 0), *ds1 = ds_images + image_at<KT>(p, slot, h, 0);
        if (tid < kG) {
            al[tid] = tid < at.len ? expf(load_gate<bf16>(g, (at.row + tid) * p.H + h, p.gate_f32)) : 1.f;
            be[tid] = tid < at.len ? load_gate<bf16>(beta, (at.row + tid) * p.H + h, p.gate_f32) : 0.f;
        }
        __syncthreads();
        if (tid < kG) {  // column tid of its tile's D, and the products from the tile's start and to its end
            const int b = tid >> 4, j = tid & 15;
            float f = 0.f, run = 1.f;
            for (int i = 0; i < 16; ++i) {
                const float a = al[b * 16 + i];
                run *= a;
                if (i == j) pre[tid] = run;
                f = i == j ? 1.f : f * a;
                diag[b * 256 + i * 16 + j] = f;
            }
            suf[tid] = f;
            if (j == 0) whole[b] = run;
        }
        float inner = 0.f;  // <S0, dS1>
        for (int i = tid; i < tiles * KT * 32; i += kGradThreads) {
            const uint4 x = __ldg(s0 + i), y = __ldg(ds1 + i);
            const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) inner = fmaf(lo_f(xw[e]), lo_f(yw[e]), fmaf(hi_f(xw[e]), hi_f(yw[e]), inner));
        }
        for (int m = 16; m > 0; m >>= 1) inner += __shfl_xor_sync(0xffffffffu, inner, m);
        if (lane == 0) part[warp] = inner;
        cp_async_wait_all();
        __syncthreads();
        if (tid < kG) {
            const int b = tid >> 4;
            float before = 1.f, after = 1.f;
            for (int t = 0; t < 4; ++t) {
                if (t < b) before *= whole[t];
                if (t > b) after *= whole[t];
            }
            cc[tid] = before * pre[tid];
            dd[tid] = suf[tid] * after;
        }
        // do_i . r_j (or y_i . r_j) on and below the diagonal
        float T[8][4] = {};
        {
            const uint32_t a_at = (key ? yss : dos) + (rt * 16 + (m8 & 1) * 8 + r8) * pl.vrow + (m8 >> 1) * 16;
            const uint32_t b_at = rss + ((m8 >> 1) * 8 + r8) * pl.vrow + (m8 & 1) * 16;
            for (int s = 0; s < tiles; ++s) {
                uint32_t a[4];
                ldsm4(a, a_at + s * 32);
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    if (t <= rt) {
                        uint32_t b[4];
                        ldsm4(b, b_at + t * 16 * pl.vrow + s * 32);
                        mma(T[2 * t], a, b[0], b[1]);
                        mma(T[2 * t + 1], a, b[2], b[3]);
                    }
            }
        }
        __syncthreads();  // cc and dd; part, diag and whole have been read by those who write them next
        float between[4];  // whole tiles strictly between tile t and this warp's
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            float f = 1.f;
            for (int m = t + 1; m < rt; ++m) f *= whole[m];
            between[t] = f;
        }
#pragma unroll
        for (int t = 0; t < 8; ++t)
            if (t <= 2 * rt + 1) {
                float x[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = row0 + (e >> 1) * 8, j = t * 8 + 2 * tg + (e & 1);
                    const float D = (t >> 1) == rt ? diag[rt * 256 + (i & 15) * 16 + (j & 15)]
                                                   : pre[i] * between[t >> 1] * suf[j];
                    if (key) {
                        if (i == j && i < at.len) store_gate<bf16>(dbeta, (at.row + i) * p.H + h, p.gate_f32, T[t][e]);
                        x[e] = j < i ? -(be[i] * be[j]) * D * T[t][e] : 0.f;
                    } else {
                        x[e] = j <= i ? be[j] * D * T[t][e] : 0.f;
                    }
                }
                char *to = (key ? Nt : Mt) + row0 * kMRow + (t * 8 + 2 * tg) * 2;
                *reinterpret_cast<uint32_t *>(to) = pack(x[0], x[1]);
                *reinterpret_cast<uint32_t *>(to + 8 * kMRow) = pack(x[2], x[3]);
            }
        // products with the states
        {
            float acc[2 * KT][4] = {};
            rows_times_image<KT>(acc, (key ? yss : dos) + rt * 16 * pl.vrow, pl.vrow, s0, tiles, lane);
            const float f0 = key ? -cc[row0] * be[row0] : cc[row0], f1 = key ? -cc[row0 + 8] * be[row0 + 8] : cc[row0 + 8];
#pragma unroll
            for (int n = 0; n < 2 * KT; ++n) {
                acc[n][0] *= f0; acc[n][1] *= f0; acc[n][2] *= f1; acc[n][3] *= f1;
#pragma unroll
                for (int e = 0; e < 4; ++e) total[n][e] += acc[n][e];
            }
            float lo, hi;
            row_dots<KT>(acc, (key ? ks : qs) + rt * 16 * row_bytes<KT>(), lane, lo, hi);
            if (tg == 0) {
                (key ? wk : wq)[row0] = lo;
                (key ? wk : wq)[row0 + 8] = hi;
            }
        }
        if (key) {
            float acc[2 * KT][4] = {};
            rows_times_image<KT>(acc, rss + rt * 16 * pl.vrow, pl.vrow, ds1, tiles, lane);
            const float f0 = dd[row0] * be[row0], f1 = dd[row0 + 8] * be[row0 + 8];
#pragma unroll
            for (int n = 0; n < 2 * KT; ++n) {
                acc[n][0] *= f0; acc[n][1] *= f0; acc[n][2] *= f1; acc[n][3] *= f1;
#pragma unroll
                for (int e = 0; e < 4; ++e) total[n][e] += acc[n][e];
            }
            float lo, hi;
            row_dots<KT>(acc, ks + rt * 16 * row_bytes<KT>(), lane, lo, hi);
            if (tg == 0) {
                xs[row0] = lo;
                xs[row0 + 8] = hi;
            }
        }
        __syncthreads();  // R' and N are whole
        // products inside the chunk
        {
            const uint32_t mt = base + pl.off_m, nt = base + pl.off_n;
            const uint32_t own = (rt * 16 + (m8 & 1) * 8 + r8) * kMRow + (m8 >> 1) * 16;   // A = rows of this warp
            const uint32_t flip = ((m8 >> 1) * 8 + r8) * kMRow + rt * 32 + (m8 & 1) * 16;  // A = columns of this warp
            float acc[2 * KT][4] = {};
            float lo, hi;
            for (int t = 0; t <= rt; ++t) {  // R' K (query) or N K (key)
                uint32_t a[4];
                ldsm4(a, (key ? nt : mt) + own + t * 32);
                add_rows<KT>(acc, a, ks + t * 16 * row_bytes<KT>(), lane);
            }
            row_dots<KT>(acc, (key ? ks : qs) + rt * 16 * row_bytes<KT>(), lane, lo, hi);
#pragma unroll
            for (int n = 0; n < 2 * KT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) total[n][e] += acc[n][e];
            float sum0 = -lo, sum1 = -hi;
            if (key) {
#pragma unroll
                for (int n = 0; n < 2 * KT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
                for (int t = rt; t < 4; ++t) {  // R'^T Q + N^T K
                    uint32_t a[4];
                    ldsm4t(a, mt + flip + t * 16 * kMRow);
                    add_rows<KT>(acc, a, qs + t * 16 * row_bytes<KT>(), lane);
                    ldsm4t(a, nt + flip + t * 16 * kMRow);
                    add_rows<KT>(acc, a, ks + t * 16 * row_bytes<KT>(), lane);
                }
                row_dots<KT>(acc, ks + rt * 16 * row_bytes<KT>(), lane, lo, hi);
                sum0 += lo;
                sum1 += hi;
#pragma unroll
                for (int n = 0; n < 2 * KT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) total[n][e] += acc[n][e];
            }
            if (tg == 0) {
                (key ? mk : mq)[row0] = sum0;
                (key ? mk : mq)[row0 + 8] = sum1;
            }
        }
        __syncthreads();
        if (tid < at.len) {
            float f = 0.f;
            for (int m = 0; m < 8; ++m) f += part[m];
            f *= cc[kG - 1];
            for (int m = 0; m < kG; ++m) f += m < tid ? xs[m] + (mq[m] + mk[m]) : wq[m] + wk[m];
            store_gate<bf16>(dg, (at.row + tid) * p.H + h, p.gate_f32, f);
        }
        __syncthreads();  // the next head's tiles and sums may come
    }
    bf16 *to = (key ? dk : dq) + ((at.row + row0) * p.Hk + hk) * p.dk + 2 * tg;
#pragma unroll
    for (int n = 0; n < 2 * KT; ++n)
        if (n * 8 < p.dk) {
            if (row0 < at.len) *reinterpret_cast<uint32_t *>(to + n * 8) = pack(total[n][0], total[n][1]);
            if (row0 + 8 < at.len)
                *reinterpret_cast<uint32_t *>(to + (int64_t)8 * p.Hk * p.dk + n * 8) = pack(total[n][2], total[n][3]);
        }
}

struct Workspace {
    size_t again, back, s_images, ds_images, resid, ys, total;
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
    w.total = at;
    return w;
}

template <int KT>
int bwd_kt(const Shape &p, const bf16 *q, const bf16 *k, const bf16 *v, const void *g, const void *beta,
           const bf16 *dout, const float *h0, const float *dhT, bf16 *dq, bf16 *dk, bf16 *dv, void *dg, void *dbeta,
           float *dh0, char *ws, cudaStream_t st) {
    const Workspace at = workspace_kt<KT>(p);
    const long long rows = total_rows(p), slots = chunk_slots(rows, p.nseq, kG);
    const Walk wa = make_walk<KT, AgainRecord>(p, false), wb = make_walk<KT, BwdRecord>(p, true);
    const int grad_bytes = grad_plan<KT>(p.dv).total;
    const long long blocks = (long long)p.nseq * p.H * wa.splits;
    if (blocks > 0x7fffffffLL || slots * p.Hk > 0x7fffffffLL) return GLA_ERR_UNSUPPORTED;
    if (cudaFuncSetAttribute(delta_again_kernel<KT>, cudaFuncAttributeMaxDynamicSharedMemorySize, walk_bytes(wa)) !=
            cudaSuccess ||
        cudaFuncSetAttribute(delta_back_kernel<KT>, cudaFuncAttributeMaxDynamicSharedMemorySize, walk_bytes(wb)) !=
            cudaSuccess ||
        cudaFuncSetAttribute(delta_grad_kernel<KT>, cudaFuncAttributeMaxDynamicSharedMemorySize, grad_bytes) !=
            cudaSuccess)
        return GLA_ERR_LAUNCH;
    int rc = mma_prep_grad(p, q, k, g, beta, ws + at.again, ws + at.back, st);
    if (rc != GLA_OK) return rc;
    bf16 *resid = (bf16 *)(ws + at.resid), *ys = (bf16 *)(ws + at.ys);
    uint4 *s_img = (uint4 *)(ws + at.s_images), *ds_img = (uint4 *)(ws + at.ds_images);
    delta_again_kernel<KT><<<(unsigned)blocks, (wa.groups + 1) * 128, walk_bytes(wa), st>>>(
        p, wa, k, v, (const AgainRecord *)(ws + at.again), h0, resid, s_img);
    delta_back_kernel<KT><<<(unsigned)blocks, (wb.groups + 1) * 128, walk_bytes(wb), st>>>(
        p, wb, q, k, dout, (const BwdRecord *)(ws + at.back), dhT, ys, dv, ds_img, dh0);
    count_launches(2);
    if (rows > 0) {
        delta_grad_kernel<KT><<<(unsigned)(slots * p.Hk), kGradThreads, grad_bytes, st>>>(
            p, q, k, dout, g, beta, resid, ys, s_img, ds_img, dq, dk, dg, dbeta);
        count_launches(1);
    }
    return cudaGetLastError() == cudaSuccess ? GLA_OK : GLA_ERR_LAUNCH;
}

}  // namespace

// bf16 with dk <= 128 (a warp's share of the state fits its registers) and dv <= 256 (the gradient kernel's three
// tiles of 64 x dv fit in shared memory).
bool mma_bwd_supported(int dk, int dv) { return dk <= 128 && dv <= 256; }

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
