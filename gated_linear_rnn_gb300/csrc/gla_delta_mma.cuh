// gla_delta_mma.cuh — what the tensor-core kernels of the gated delta rule share: chunk records, mma.sync
// fragments, and the frame of a walk over a chain (fetching warpgroup, stages, state and output tiles).
#pragma once

#include "gla_delta.cuh"
#include "gla_pairs.cuh"
#include "sm100_ptx.cuh"

namespace gla {
namespace delta {
namespace {

using bf16 = __nv_bfloat16;
constexpr int kC = 32;                  // tokens per chunk of a walk
constexpr int kMaxWarps = 12;           // column tiles of 16 per block
constexpr uint64_t kWaitNs = 2000000000ull;

// Per chunk and value head, in the order of the B operands: [4 tiles of 8 columns][32 lanes] x 16 bytes
// (k 0..15 then 16..31).
struct FwdRecord {
    uint4 mhi[4][32], mlo[4][32], p[4][32];
    float c[kC], db[kC];  // c_i and d_j beta_j
};
// For the gradient: the walk that recomputes the residuals takes M alone; the walk backwards takes P without beta
// and (I + diag(beta) L)^-1, both as B operands of products over the token that reads (k = i, n = j).
struct AgainRecord {
    uint4 mhi[4][32];
    float c[kC], db[kC];
};
struct BwdRecord {
    uint4 p[4][32], m[4][32];
    float c[kC], d[kC], b[kC];
};
static_assert(sizeof(FwdRecord) % 16 == 0 && sizeof(AgainRecord) % 16 == 0 && sizeof(BwdRecord) % 16 == 0,
              "bulk copies take multiples of 16 bytes");

// ---- fragments -----------------------------------------------------------------------------------------------
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// the same from zero
__device__ __forceinline__ void mma0(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void scale(float (&d)[4], Pair by) {
    const float2 x = parts(pair(d[0], d[1]) * by), y = parts(pair(d[2], d[3]) * by);
    d[0] = x.x; d[1] = x.y; d[2] = y.x; d[3] = y.y;
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void stsm4t(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};"
                 ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void stsm4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};"
                 ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 t;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(t.x), "=r"(t.y), "=r"(t.z), "=r"(t.w) : "r"(addr) : "memory");
    return t;
}
__device__ __forceinline__ float2 lds_f2(uint32_t addr) {
    float2 t;
    asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];" : "=f"(t.x), "=f"(t.y) : "r"(addr) : "memory");
    return t;
}
// 16 bytes from global to shared memory, or 16 zero bytes
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool has) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(has ? 16 : 0) : "memory");
}
// this thread's arrival on `bar` once all of its copies so far have landed
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// two f32 to two bf16 (x in the low half), round to nearest
__device__ __forceinline__ uint32_t pack(float x, float y) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
    return r;
}
__device__ __forceinline__ float lo_f(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float hi_f(uint32_t p) { return __uint_as_float(p & 0xffff0000u); }
// x, y as hi + lo parts of 8 bits each
__device__ __forceinline__ void split(float x, float y, uint32_t &hi, uint32_t &lo) {
    hi = pack(x, y);
    const float2 rest = parts(fma(pair(lo_f(hi), hi_f(hi)), both(-1.f), pair(x, y)));  // exact
    lo = pack(rest.x, rest.y);
}

// 8 x 8 b16 values, a row's pair in each lane, transposed within the warp
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

template <int KT> constexpr int row_bytes() { return KT * 32 + 16; }  // KT * 16 bf16 and an odd number of 16-byte units

// ---- the frame of a walk -----------------------------------------------------------------------------------------

struct Walk {           // one block's share of a chain
    int warps, splits;  // column tiles per block, blocks per chain
    int groups;         // warpgroups that hold those tiles; one more fetches
    int vrow;           // bytes of a staged row of V, an odd number of 16-byte units
    int stages, stage_bytes;
    int segment;        // tokens per segment of a chain (a multiple of kC), or 0: a block walks the whole chain
};

// A block is launched with 128 registers a thread; the fetching warpgroup gives back 72 of them and each of the
// others takes 24 more: g 152 + 56 <= (g + 1) 128 for up to three.
constexpr int kMaxThreads = (kMaxWarps / 4 + 1) * 128;
static_assert(kMaxWarps == 12, "three warpgroups of column tiles: 3 * 152 + 56 = 4 * 128");
__device__ __forceinline__ void give_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 56;"); }
__device__ __forceinline__ void take_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 152;"); }

// Blocks per chain: one where the chains fill the GPU (the fewest reads of K and Q), else as many as fill it.
// B8 T2048 H16 dk96 dv192 (128 chains, 152 SMs) runs one block of 12 column tiles to a chain.
// walks: chains, or segments of them; tiles: column tiles of 16 of one; outputs: tiles of 32 x its columns that leave a
// stage, the first in V's place
template <int KT, class Rec>
Walk make_walk(long long walks, int tiles, bool with_q, int outputs) {
    Walk w{};
    const int sms = device_info().sm_count;
    int splits = (tiles + kMaxWarps - 1) / kMaxWarps;
    if (walks * splits < sms) splits = (int)min((long long)tiles, sms / walks);
    w.warps = (tiles + splits - 1) / splits;
    w.splits = (tiles + w.warps - 1) / w.warps;
    w.groups = (w.warps + 3) / 4;
    w.vrow = (w.warps * 2 | 1) * 16;
    w.stage_bytes = (with_q ? 2 : 1) * kC * row_bytes<KT>() + kC * w.vrow * (outputs > 1 ? outputs : 1) + (int)sizeof(Rec);
    w.stages = 4 * w.stage_bytes + 128 <= device_info().max_smem_optin ? 4 : 3;
    return w;
}
inline int walk_bytes(const Walk &w) { return 128 + w.stages * w.stage_bytes; }

// A bounded wait of a whole warp: all lanes learn the same.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const volatile int *abort_flag) {
    return __all_sync(0xffffffffu, ptx::mbar_wait(bar, parity, abort_flag, kWaitNs));
}

// A barrier of some of the block's warps that tells all of them whether any brings a failure, so that all of them leave
// together or none.
template <int kBarrier, int kThreads> __device__ __forceinline__ bool any_of(bool failed) {
    uint32_t any;
    asm volatile("{\n\t.reg .pred p, r;\n\t"
                 "setp.ne.u32 p, %1, 0;\n\t"
                 "barrier.cta.red.or.pred r, %2, %3, p;\n\t"
                 "selp.u32 %0, 1, 0, r;\n\t}"
                 : "=r"(any) : "r"((uint32_t)failed), "n"(kBarrier), "n"(kThreads) : "memory");
    return any != 0;
}

// The walks over a packed batch start in the order of their lengths, the longest first, so that the last ones to end are
// short, where their blocks run in more than one and at most eight waves.  The preparation finds each sequence's rank, by a warp that looks
// at all lengths.  16 heads of 96/192, in this order and in the batch's own: 24 sequences of 0..256 tokens 52 and 58 us,
// of 0..1,024 148 and 160, 64 of 0..1,024 381 and 416; of 64 equal lengths 58 and 56.  In one wave all start at once, and
// in many the order is nothing but its cost: 8 of 0..1,024 77 and 75 us, 128 of 0..256 262 and 262, 256 of them 513 and 498.
constexpr int kRankedWaves = 8;
// rows_bytes at `at`; blocks: of the launch whose blocks walk over whole chains, or 0
inline void place_rows(Shape &p, char *at, long long blocks) {
    const long long sms = device_info().sm_count;
    p.rows = reinterpret_cast<int2 *>(at);
    p.planned = p.cu != nullptr && p.nseq > kMostChecked;
    p.order = p.cu != nullptr && blocks > sms && blocks <= kRankedWaves * sms ? reinterpret_cast<int *>(p.rows + p.nseq + 1) : nullptr;
}
// How many sequences start before s: the longer ones, and of equals the first.  (A bad one's length is only an order here.)
__device__ __forceinline__ int rank_of(const Shape &p, int s, int lane) {
    SeqRange own, r;
    seq_range(s, p.T, p.cu, own);
    int before = 0;
    for (int i = lane; i < p.nseq; i += 32) {
        seq_range(i, p.T, p.cu, r);
        before += r.len > own.len || (r.len == own.len && i < s);
    }
    return __reduce_add_sync(0xffffffffu, before);
}

// Who a block and a thread are, and the shared memory: barriers, the stages (K | Q | V | record | a second output).
struct Frame {
    int lane, warp, s, h, hk, col0, width, nch;
    int walk;       // (sequence or segment's slot) * H + head
    bool exists;    // whether a segment has this slot
    bool last;      // of its sequence's segments
    SeqRange r;     // the rows that this block walks over
    int64_t slot0;  // slot of its first chunk
    uint32_t full, empty, ring;
    volatile int *abort_flag;

    __device__ __forceinline__ Frame(const Shape &p, const Walk &w, unsigned block, char *sm) {
        lane = threadIdx.x & 31;
        warp = threadIdx.x >> 5;
        walk = (int)(block / (unsigned)w.splits);
        s = walk / p.H;
        h = walk % p.H;
        hk = h / p.group();
        col0 = (int)(block % (unsigned)w.splits) * w.warps * 16;  // first column of the block
        width = min(w.warps * 16, p.dv - col0);                   // its columns of v, a multiple of 8 (none: <= 0)
        exists = last = true;
        if (w.segment == 0) {
            if (p.order != nullptr) {
                // through shared memory: the walk is 163 us for 160.5 at 8 x 2,048 tokens where each thread loads it
                volatile int *turn = reinterpret_cast<volatile int *>(sm + 16 * w.stages + 4);
                if (threadIdx.x == 0) *turn = __ldg(p.order + s);
                __syncthreads();
                s = *turn;
                walk = s * p.H + h;
            }
            r = rows_of(p, s);
            slot0 = r.start / kC + s;
        } else {
            // segment i of sequence s has the slot start_s / segment + s + i
            const int slot = s;
            s = bisect_slots(p, slot, w.segment, [&](int i) { return __ldg(p.rows + i).x; });
            r = rows_of(p, s);
            const int i = slot - ((int)r.start / w.segment + s);
            exists = i >= 0 && (int64_t)i * w.segment < r.len;  // a sequence without rows has none: delta_join_kernel's
            last = (int64_t)(i + 1) * w.segment >= r.len;
            slot0 = r.start / kC + s + (int64_t)i * (w.segment / kC);
            r.start += (int64_t)i * w.segment;
            r.len = min((int64_t)w.segment, r.len - (int64_t)i * w.segment);
        }
        nch = (int)((r.len + kC - 1) / kC);
        full = ptx::smem_u32(sm);
        empty = full + 8 * w.stages;
        abort_flag = reinterpret_cast<volatile int *>(sm + 16 * w.stages);
        ring = full + 128;
        if (threadIdx.x == 0) {
            for (int i = 0; i < w.stages; ++i) {
                ptx::mbar_init(full + 8 * i, 129);  // the fetching threads, and the record
                ptx::mbar_init(empty + 8 * i, w.warps);
            }
            *abort_flag = 0;
            ptx::fence_mbar_init();
        }
        __syncthreads();
    }
};

// The outputs of a stage, rows of the block's columns as the other warps left them, to rows of `out` and `out2` [rows, H,
// dv]; neighbouring threads write neighbouring bytes.
template <int kOut>
__device__ __forceinline__ void write_rows(const Shape &p, const Walk &w, const Frame &f, int c, uint32_t v, uint32_t second,
                                           bf16 *out, bf16 *out2) {
    const int units = f.width / 8, id = threadIdx.x - w.groups * 128;
    const int rows = (int)min((int64_t)kC, f.r.len - (int64_t)c * kC);
    const unsigned inv = (65536 + units - 1) / units;  // e / units for e < 32 * 24 by a product
    const int64_t at = ((f.r.start + (int64_t)c * kC) * p.H + f.h) * p.dv + f.col0;
    for (int e = id; e < rows * units; e += 128) {
        const int t = (int)(((unsigned)e * inv) >> 16), u = e - t * units;
        const int64_t to = at + (int64_t)t * p.H * p.dv + u * 8;
        *reinterpret_cast<uint4 *>(out + to) = lds128(v + t * w.vrow + u * 16);
        if (kOut > 1) *reinterpret_cast<uint4 *>(out2 + to) = lds128(second + t * w.vrow + u * 16);
    }
}

// The fetching warpgroup: four threads to a token's row.  kBack walks the chunks from the last to the first.  A stage
// that comes back holds its chunk's outputs (kOut of them), which go out before it is filled again: the
// other warps neither store to global memory nor wait for it.
template <int KT, bool kQ, bool kBack, int kOut, class Rec>
__device__ __forceinline__ void fetch(const Shape &p, const Walk &w, const Frame &f, const bf16 *q, const bf16 *k,
                                      const bf16 *v, const Rec *records, bf16 *out, bf16 *out2) {
    constexpr int kRow = row_bytes<KT>(), kTile = kC * kRow, kV = (kQ ? 2 : 1) * kTile;
    const int id = threadIdx.x - w.groups * 128, t = id >> 2, u0 = id & 3;
    const int vunits = w.warps * 2, vlive = f.width / 8, kunits = p.dk / 8;
    const int64_t kstride = (int64_t)p.Hk * p.dk, vstride = (int64_t)p.H * p.dv;
    const int64_t row0 = f.r.start + t + (kBack ? (int64_t)(f.nch - 1) * kC : 0);
    const bf16 *kr = k + row0 * kstride + f.hk * p.dk + u0 * 8, *qr = q + row0 * kstride + f.hk * p.dk + u0 * 8,
               *vr = v + row0 * vstride + (int64_t)f.h * p.dv + f.col0 + u0 * 8;
    const uint32_t kdst = f.ring + t * kRow + u0 * 16, vdst = f.ring + kV + t * w.vrow + u0 * 16;
    bool ok = true;
    for (int i = 0; i < f.nch + w.stages; ++i) {
        const int sg = i % w.stages;
        const uint32_t at = sg * w.stage_bytes;
        if (i >= w.stages) {
            if (i >= f.nch && kOut == 0) break;  // nothing is left to bring in or out
            ok = warp_wait(f.empty + 8 * sg, (i / w.stages + 1) & 1, f.abort_flag);
            if (kOut > 0) {
                const int done = i - w.stages;
                const uint32_t from = f.ring + at + kV;
                if (ok)
                    write_rows<kOut>(p, w, f, kBack ? f.nch - 1 - done : done, from,
                                     from + kC * w.vrow + (uint32_t)sizeof(Rec), out, out2);
                ok = !any_of<3, 128>(!ok);  // the rows are read before any thread's copies may land on them
            }
            if (!ok) break;
        }
        if (i >= f.nch) continue;
        const int c = kBack ? f.nch - 1 - i : i;
        const bool row = c * kC + t < f.r.len;  // a short chunk's missing rows are zero, and not read
        if (id == 0) {
            ptx::mbar_expect_tx(f.full + 8 * sg, (uint32_t)sizeof(Rec));
            ptx::bulk_load_g2s(f.ring + at + kV + kC * w.vrow, records + (f.slot0 + c) * p.H + f.h, sizeof(Rec),
                               f.full + 8 * sg);
        }
#pragma unroll
        for (int u = 0; u < KT * 2; u += 4) {
            const bool has = row && u0 + u < kunits;
            cp_async16(kdst + at + u * 16, has ? kr + u * 8 : k, has);
            if (kQ) cp_async16(kdst + at + kTile + u * 16, has ? qr + u * 8 : q, has);
        }
#pragma unroll 2
        for (int u = 0; u < vunits - u0; u += 4) {
            const bool has = row && u0 + u < vlive;
            cp_async16(vdst + at + u * 16, has ? vr + u * 8 : v, has);
        }
        cp_async_arrive(f.full + 8 * sg);
        kr += (kBack ? -kC : kC) * kstride;
        qr += (kBack ? -kC : kC) * kstride;
        vr += (kBack ? -kC : kC) * vstride;
    }
    // nothing may be in flight into a block that ends early; a whole walk has waited for every stage
    cp_async_wait_all();
    if (!ok) {
        *f.abort_flag = 1;
        for (int i = 0; i < w.stages; ++i)  // the records' bulk copies, bounded like every wait
            for (int par = 0; par < 2; ++par) ptx::mbar_wait(f.full + 8 * i, par, nullptr, kWaitNs / 1000);
    }
}

// A warp's 16 columns of a state [dk][cols] in f32 as the accumulators of S^T (16 x dk).
template <int KT>
__device__ __forceinline__ void load_state(float (&S)[2 * KT][4], const float *from, int64_t state, int dk, int cols, int col,
                                           int lane) {
    const int64_t at = state * dk * cols + col + (lane >> 2);
#pragma unroll
    for (int n = 0; n < 2 * KT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int row = n * 8 + 2 * (lane & 3) + (e & 1);
            const bool has = from != nullptr && row < dk && col + (e >> 1) * 8 < cols;
            S[n][e] = has ? from[at + (int64_t)row * cols + (e >> 1) * 8] : 0.f;
        }
}
template <int KT>
__device__ __forceinline__ void store_state(float *to, const float (&S)[2 * KT][4], int64_t state, int dk, int cols, int col,
                                            int lane) {
    const int64_t at = state * dk * cols + col + (lane >> 2);
#pragma unroll
    for (int n = 0; n < 2 * KT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int row = n * 8 + 2 * (lane & 3) + (e & 1);
            if (row < dk && col + (e >> 1) * 8 < cols) to[at + (int64_t)row * cols + (e >> 1) * 8] = S[n][e];
        }
}

// O^T (16 columns x 32 tokens) rounded to bf16 into the warp's columns of a stage's rows.
__device__ __forceinline__ void put_tile(const float (&O)[4][4], uint32_t cols, int vrow, int lane) {
    const uint32_t to = cols + ((lane >> 4) * 8 + (lane & 7)) * vrow + ((lane >> 3) & 1) * 16;
#pragma unroll
    for (int t = 0; t < 2; ++t)
        stsm4t(to + t * 16 * vrow, pack(O[2 * t][0], O[2 * t][1]), pack(O[2 * t][2], O[2 * t][3]),
               pack(O[2 * t + 1][0], O[2 * t + 1][1]), pack(O[2 * t + 1][2], O[2 * t + 1][3]));
}

}  // namespace
}  // namespace delta
}  // namespace gla

// the kernels' width of a state's rows, in units of 16
#define GLA_BY_KT(dk, CALL)        \
    do {                           \
        if (dk <= 32) { CALL(2); } \
        else if (dk <= 64) { CALL(4); } \
        else if (dk <= 96) { CALL(6); } \
        else { CALL(8); }          \
    } while (0)
