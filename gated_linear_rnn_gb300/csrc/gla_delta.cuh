// gla_delta.cuh — what the translation units of the gated delta rule share.
//
// Per (sequence, value head) chain with a dk x dv matrix state S (row vectors k, q, v, u, o):
//     u_t = beta_t (v_t - a_t k_t S_{t-1}),   S_t = a_t S_{t-1} + k_t^T u_t,   o_t = q_t S_t,   a_t = exp(g_t)
// Value head h reads the query and key head h / (H / Hk).
#pragma once

#include "gla_common.cuh"

namespace gla {
namespace delta {

// Sizes of one call.  q, k: [rows, Hk, dk]; v, out: [rows, H, dv]; g, beta: [rows, H] (f32 when gate_f32,
// else the type of q).  nseq sequences of T rows each (cu null) or packed with offsets cu.
struct Shape {
    int nseq, T, H, Hk, dk, dv;
    int gate_f32;
    const int32_t *cu;
    // packed, [nseq + 1], which the first kernel of a call writes: the first row and the number of rows of each sequence,
    // then the rows that all of them have together, or a negative number of them where the batch is not in order
    int2 *rows;
    int *order;  // [nseq], likewise: the sequences, the longest first; null where the walks take them as they come
    int planned;  // whether a kernel of its own has written rows, ahead of the preparation
    __host__ __device__ int group() const { return H / Hk; }
};

__host__ inline long long total_rows(const Shape &s) { return s.cu ? (long long)s.T : (long long)s.nseq * s.T; }

// Chunks of C tokens restart at every sequence start.  Chunk c of sequence s has the slot
// start_s / C + s + c; slots of different chunks differ, and all are below slots(rows, nseq, C).
__host__ inline long long chunk_slots(long long rows, int nseq, int C) { return rows / C + nseq + 1; }
__host__ inline size_t rows_bytes(const Shape &s) {
    return s.cu ? (((size_t)s.nseq + 1) * sizeof(int2) + (size_t)s.nseq * sizeof(int) + 255) / 256 * 256 : 0;
}

// ---- packed batches: offsets as they come ------------------------------------------------------------------------
//
// A batch is in order where its offsets lie in 0 .. T and never fall.  Elsewhere the sequences that have such an offset
// are bad, and so is one that starts before the end of an earlier one, whose rows and slots it would share; all others
// are what they are alone.  A call's first kernel looks at the offsets and leaves the rows of every sequence to the
// others: a bad one has none, at the end of those before it, so that the starts rise and can be bisected.

// Up to so many sequences, every warp that asks for a chunk by the offsets looks at all of them; more are planned by a
// kernel ahead.  Sequences of 8 tokens, 4 heads of 96/192, forward, us, checked and planned: 24 of them 13.9 and 15.8, 1,024
// 198 and 201, 4,096 790 and 774, 16,384 3,462 and 3,066.
constexpr int kMostChecked = 1024;

// By a whole warp.
__device__ __forceinline__ bool offsets_in_order(const Shape &p) {
    bool ok = true;
    for (int i = threadIdx.x & 31; i < p.nseq; i += 32) {
        const int32_t a = __ldg(p.cu + i), b = __ldg(p.cu + i + 1);
        ok = ok && a >= 0 && a <= b && b <= p.T;
    }
    return __all_sync(0xffffffffu, ok);
}

// Whether sequence s is good, by all threads of a block: what a kernel that takes sequences, not chunks, has to know.
__device__ __forceinline__ bool good_sequence(const Shape &p, int s, SeqRange &r) {
    const bool own = seq_range(s, p.T, p.cu, r);
    if (p.cu == nullptr) return true;
    bool shared = false;  // rows of an earlier one
    for (int j = threadIdx.x; j < s; j += blockDim.x) {
        SeqRange o;
        if (seq_range(j, p.T, p.cu, o) && o.start + o.len > r.start) shared = true;
    }
    return !__syncthreads_or(shared) && own;
}

// The largest end of the sequences before s, by a whole warp.
__device__ __forceinline__ int end_before(const Shape &p, int s) {
    int end = 0;
    for (int j = threadIdx.x & 31; j < s; j += 32) {
        SeqRange r;
        if (seq_range(j, p.T, p.cu, r)) end = max(end, (int)(r.start + r.len));
    }
    return __reduce_max_sync(0xffffffffu, end);
}

// The rows of sequence s, by a whole warp; false for a bad one.
__device__ __forceinline__ bool checked_rows(const Shape &p, bool in_order, int s, SeqRange &r) {
    bool good = seq_range(s, p.T, p.cu, r);
    if (!in_order) {
        const int end = end_before(p, s);
        if (r.start < end) good = false;
        if (!good) {
            r.start = end;
            r.len = 0;
        }
    }
    return good;
}

__device__ __forceinline__ int2 span_of(const Shape &p, bool in_order) {
    const int first = __ldg(p.cu);
    return in_order ? make_int2(first, __ldg(p.cu + p.nseq) - first) : make_int2(0, -1);
}

// ---- sequences and chunks ------------------------------------------------------------------------------------------

__device__ __forceinline__ SeqRange rows_of(const Shape &p, int s) {
    if (p.cu == nullptr) return {(int64_t)s * p.T, p.T};
    const int2 t = __ldg(p.rows + s);
    return {t.x, t.y};
}

// The largest s with start_s / C + s <= slot, whose chunk of C tokens it is if it is any sequence's.  Slots and rows are
// below 2^31 (the entry points see to it).
template <class F>
__device__ __forceinline__ int bisect_slots(const Shape &p, int slot, int C, F packed_start) {
    int lo = 0, hi = p.nseq - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        const int start = p.cu == nullptr ? mid * p.T : packed_start(mid);
        if (start / C + mid <= slot) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// Whether element i of rows of `width` elements lies in any sequence's row: where the batch is in order, all rows from
// the first sequence's to the last one's are; else the last that starts at or before a row is the only one that can have
// it.  span: rows[nseq], which the caller may load ahead.
__device__ __forceinline__ bool in_some_sequence(const Shape &p, int2 span, int64_t i, int64_t width) {
    if (span.y >= 0) return i >= span.x * width && i < (span.x + (int64_t)span.y) * width;
    const int row = (int)(i / width);
    int lo = 0, hi = p.nseq - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (__ldg(p.rows + mid).x <= row) lo = mid; else hi = mid - 1;
    }
    const int2 t = __ldg(p.rows + lo);
    return row >= t.x && row - t.x < t.y;
}

struct ChunkAt {
    int64_t row;   // first row of the chunk
    int len;       // its tokens, 1 .. C
};
// Chunk of sequence s in this slot; false if it has none there.
template <int C>
__device__ __forceinline__ bool chunk_at(int slot, int s, const SeqRange &r, ChunkAt &at) {
    const int start = (int)r.start, len = (int)r.len, c = slot - (start / C + s);
    if (c < 0 || c >= (len + C - 1) / C) return false;
    at.row = start + c * C;
    at.len = min(len - c * C, C);
    return true;
}

// The chunk that owns a slot; false for slots that no chunk has.
template <int C>
__device__ __forceinline__ bool chunk_of_slot(int slot, const Shape &p, ChunkAt &at) {
    const int s = bisect_slots(p, slot, C, [&](int i) { return __ldg(p.rows + i).x; });
    return chunk_at<C>(slot, s, rows_of(p, s), at);
}
// The same by the offsets themselves.
template <int C>
__device__ __forceinline__ bool checked_chunk_of_slot(int slot, const Shape &p, bool in_order, ChunkAt &at) {
    SeqRange r;
    if (in_order) {
        const int s = bisect_slots(p, slot, C, [&](int i) { return __ldg(p.cu + i); });
        return seq_range(s, p.T, p.cu, r) && chunk_at<C>(slot, s, r, at);
    }
    int64_t end = 0;
    for (int s = 0; s < p.nseq; ++s) {
        if (!seq_range(s, p.T, p.cu, r)) continue;
        if (r.start >= end && chunk_at<C>(slot, s, r, at)) return true;
        end = max(end, r.start + r.len);
    }
    return false;
}

// g and beta come in f32 or in the type of q.
template <typename T>
__device__ __forceinline__ float load_gate(const void *p, int64_t i, int f32) {
    return f32 ? __ldg(reinterpret_cast<const float *>(p) + i) : to_f32(reinterpret_cast<const T *>(p)[i]);
}
template <typename T>
__device__ __forceinline__ void store_gate(void *p, int64_t i, int f32, float x) {
    if (f32) reinterpret_cast<float *>(p)[i] = x;
    else reinterpret_cast<T *>(p)[i] = from_f32<T>(x);
}

}  // namespace delta
}  // namespace gla
