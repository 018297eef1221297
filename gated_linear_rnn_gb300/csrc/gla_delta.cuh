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
    __host__ __device__ int group() const { return H / Hk; }
};

__host__ inline long long total_rows(const Shape &s) { return s.cu ? (long long)s.T : (long long)s.nseq * s.T; }

// Chunks of C tokens restart at every sequence start.  Chunk c of sequence s has the slot
// start_s / C + s + c; slots of different chunks differ, and all are below slots(rows, nseq, C).
__host__ inline long long chunk_slots(long long rows, int nseq, int C) { return rows / C + nseq + 1; }

struct ChunkAt {
    int64_t row;   // first row of the chunk
    int len;       // its tokens, 1 .. C
    int seq;
    bool first, last;  // first / last chunk of its sequence
};

// The chunk that owns a slot; false for slots that no chunk has (and for sequences with bad offsets).  Slots and
// rows are below 2^31 (the entry points see to it).
template <int C>
__device__ __forceinline__ bool chunk_of_slot(int slot, const Shape &p, ChunkAt &at) {
    int lo = 0, hi = p.nseq - 1;  // the largest s with start_s / C + s <= slot
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        const int start = p.cu == nullptr ? mid * p.T : __ldg(p.cu + mid);
        if (start / C + mid <= slot) lo = mid; else hi = mid - 1;
    }
    SeqRange r;
    if (!seq_range(lo, p.T, p.cu, r)) return false;
    const int start = (int)r.start, len = (int)r.len;
    const int c = slot - (start / C + lo);
    if (c < 0 || c >= (len + C - 1) / C) return false;
    at.row = start + c * C;
    at.len = min(len - c * C, C);
    at.seq = lo;
    at.first = c == 0;
    at.last = c == (len + C - 1) / C - 1;
    return true;
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
