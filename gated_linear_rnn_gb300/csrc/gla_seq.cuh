// gla_seq.cuh — sequences of a dense or packed batch, as the kernels that work through rows in chunks see them.
//
// The offsets of a packed batch come from the device and may be bad.  A sequence is good where its offsets lie in 0 .. T,
// do not fall, and start at or behind the end of every earlier one with such offsets; a call's first kernel leaves (first
// row, rows) of every sequence to the others, and a bad one has no rows, at the end of those before it, so that the first
// rows rise and can be bisected.
#pragma once

#include "gla_common.cuh"

namespace gla {

// nseq sequences of T rows each (rows null) or the packed ones that plan_rows_kernel wrote.
struct Sequences {
    int nseq, T;
    const int2 *rows;
};

__host__ __device__ inline int64_t rows_bytes(int nseq, bool packed) {
    return packed ? ((int64_t)nseq * (int64_t)sizeof(int2) + 255) / 256 * 256 : 0;
}

__device__ __forceinline__ int2 rows_of(const Sequences &q, int s) {
    return q.rows == nullptr ? make_int2(s * q.T, q.T) : __ldg(q.rows + s);
}

// Chunks of C rows restart at every sequence's start: chunk c of sequence s has the slot start / C + s + c.  Slots of
// different chunks differ, and all are below chunk_slots; some belong to no chunk.
__host__ __device__ inline int64_t chunk_slots(int64_t rows, int nseq, int C) { return rows / C + nseq + 1; }

// The sequence whose chunk a slot is, if it is any's: the last with start / C + s <= slot.
__device__ __forceinline__ int sequence_of_slot(const Sequences &q, int64_t slot, int C) {
    int lo = 0, hi = q.nseq - 1;
    while (lo < hi) {
        const int mid = lo + (hi - lo + 1) / 2;
        if ((int64_t)rows_of(q, mid).x / C + mid <= slot) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// One block.  The ends of the sequences before each one are a running maximum, taken 1,024 sequences at a time; `bad`
// tells whether any sequence was.
constexpr int kPlanThreads = 1024;
__device__ __forceinline__ bool plan_rows(const int32_t *cu, int nseq, int T, int2 *rows) {
    __shared__ int tops[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int end = 0;
    bool bad = false;
    for (int first = 0; first < nseq; first += kPlanThreads) {
        const int s = first + (int)threadIdx.x;
        const int a = s < nseq ? __ldg(cu + s) : 0, b = s < nseq ? __ldg(cu + s + 1) : 0;
        const bool own = s < nseq && a >= 0 && a <= b && b <= T;
        int top = own ? b : 0;  // the largest end up to this one, then up to the one before it
        for (int d = 1; d < 32; d *= 2) {
            const int t = __shfl_up_sync(0xffffffffu, top, d);
            if (lane >= d) top = max(top, t);
        }
        if (lane == 31) tops[warp] = top;
        top = __shfl_up_sync(0xffffffffu, top, 1);
        if (lane == 0) top = 0;
        __syncthreads();
        int before = end;
        for (int w = 0; w < kPlanThreads / 32; ++w) {
            if (w < warp) before = max(before, tops[w]);
            end = max(end, tops[w]);
        }
        top = max(top, before);
        if (s < nseq) {
            const bool good = own && a >= top;
            rows[s] = good ? make_int2(a, b - a) : make_int2(top, 0);
            bad |= !good;
        }
        __syncthreads();
    }
    return bad;
}

}  // namespace gla
