// gla_scan_tiles.cuh — what the chunked forward and gradient of the gated recurrence share.
//
// A block works on tiles of 64 channels of a chunk of kChunk rows of one sequence: a warp takes eight rows, a lane two
// channels.  A tile's effect on a state is h -> A h + H.  Its warps find their rows' effects from a zero state, meet in shared
// memory, and the tile's effect is published; the state that enters it is then found by looking back over the effects of the
// tiles before it, to the nearest one whose own result is published.  The look back folds from that result on, one tile after
// the other, which is the same arithmetic wherever it starts: the results do not depend on who was first.
//
// What is published is its own flag: a word that holds kUnset has not been written yet.
//
// Log decays may be above 0.  A tile's product of decays, or its result from a zero state, can then leave f32 where the states do
// not: zeros, small states, those behind a reset.  A channel whose effect did so is apart: its effect and result stay unset, so that
// nobody folds them, and once the state that enters the tile is known its warps go through their rows one after the other from
// there, and the last one publishes the result: 18 us a tile in the forward, which has its rows to load again, 2 in the gradient.
// (Where no channel is apart, that it could be costs 0 to 2%.  A sigmoid is at most 1, and its kernels have none of it.)
//
// Tiles are handed out by a counter in an order in which a tile comes after all that it waits for, so that a waiting block
// waits only for blocks that run.  Rows come in by TMA, some tiles ahead.
//
// Each input is read once and each output written once.  Measured (bf16, sigmoid with a leak, gate): 8 x 2,048 x 2,560 forward
// 79 us, gradient 127 (the bytes at the rate of a copy: 50 and 87); 256 x 64, without chains, 67 and 110.  What bounds it there
// is the instructions of the decays and gates beside the wait for a tile's meeting.  Few long sequences (1 x 32,768 x 2,048 f32 log
// decays 153 and 214, for 79 and 139) take 4.2 us a tile and block where a batch without chains takes 3: some 14 tiles of a chain
// are in flight, and the look back is less than half of what they take beyond their bytes.  Tiles of 64 x 64 were measured
// against 128 x 32 (long 143 and 218, short sequences twice the time), clusters that hand the state on in shared memory (8 x 2,048:
// 137) and a warp that only follows the chain (gradient 116, of long sequences 236).
#pragma once

#include <cuda.h>

#include "gla_scan.cuh"
#include "sm100_ptx.cuh"

namespace gla {
bool make_map_2d(CUtensorMap *m, CUtensorMapDataType dtype, uint32_t elem_bytes, const void *base, uint64_t cols,
                 uint64_t rows, uint32_t box_cols, uint32_t box_rows, CUtensorMapSwizzle sw);
namespace scan {

constexpr int kLane = kRun;                  // rows of a warp
constexpr int kWarps = kChunk / kLane;
constexpr int kTileThreads = kWarps * 32;
constexpr int kSlab = 64;                    // channels of a tile
constexpr uint32_t kUnset = 0xffffffffu;     // a NaN that no result is: one that would be is stored as another
constexpr uint64_t kWaitNs = 2000000000ull;  // 2 s a wait
constexpr int kBack = 2 * kWarps;            // tiles that a look back reads at once, at most
constexpr float kMostF32 = 3.40282347e38f;

// The chunks' effects and results, for one direction.
struct Chain {
    float *effect;   // [places, D, 2]: A, H
    float *result;   // [places, D]
    unsigned *next;  // the counter of tiles, and behind it whether a wait gave up
};
// A chunk's place among them is start / kChunk + c in the forward and one less in the gradient.  A sequence of n chunks publishes
// for n - 1 of them, the forward for all but its last and the gradient for all but its first, so no two share a place: the next
// sequence starts at start / kChunk + n - 1 or behind.
__host__ inline int64_t places(const Shape &p) { return total_rows(p) / kChunk + 1; }
__host__ inline int64_t chain_floats(const Shape &p) { return places(p) * p.D * 3; }

struct Tiles {
    Sequences q;
    int D, slabs, nslots, per_seq;  // per_seq: chunks of a sequence of a dense batch
    unsigned total;
    int chained;                    // whether any sequence may have more than one chunk
    int window;                     // tiles that a look back reads at once
    bool walked;                    // short sequences are walked by other kernels
    const int2 *tasks;              // of a packed batch: sequence and chunk, in the forward's order
    const int *ntasks;
};
__device__ __forceinline__ unsigned tiles_of(const Tiles &t) {
    return t.tasks == nullptr ? t.total : (unsigned)__ldg(t.ntasks) * (unsigned)t.slabs;
}
__host__ inline Tiles make_tiles(const Shape &p, const Sequences &q) {
    Tiles t{q, p.D, (p.D + kSlab - 1) / kSlab, (int)slots(p), (p.T + kChunk - 1) / kChunk, 0, 1, 1, false, nullptr, nullptr};
    t.total = p.cu ? (unsigned)t.nslots * (unsigned)t.slabs : (unsigned)t.per_seq * (unsigned)p.nseq * (unsigned)t.slabs;
    t.chained = p.cu != nullptr || p.T > kChunk;
    return t;
}

struct Tile {
    int row, len, chunk, behind, seq, slot, col;  // behind: its sequence's chunks after it; col: its first channel
    __device__ int start() const { return row - chunk * kChunk; }  // its sequence's first row
};

// Tile k in the order of a direction, of n.  A dense batch goes through all sequences' first chunks, then their second ones and
// so on: what a tile waits for is then mostly done.  A packed one does so with 32 sequences after the other.
template <bool kForth>
__device__ __forceinline__ void tile_at(const Tiles &t, unsigned k, unsigned n, Tile &o) {
    o.col = (int)(k % (unsigned)t.slabs) * kSlab;
    unsigned r = k / (unsigned)t.slabs;
    int2 rows;
    if (t.q.rows == nullptr) {
        o.seq = (int)(r % (unsigned)t.q.nseq);
        o.chunk = (int)(r / (unsigned)t.q.nseq);
        if (!kForth) o.chunk = t.per_seq - 1 - o.chunk;
        rows = rows_of(t.q, o.seq);
    } else {
        const int2 task = __ldg(t.tasks + (kForth ? r : n / (unsigned)t.slabs - 1 - r));
        o.seq = task.x;
        o.chunk = task.y;
        rows = rows_of(t.q, o.seq);
    }
    o.slot = rows.x / kChunk + o.chunk - (kForth ? 0 : 1);
    o.row = rows.x + o.chunk * kChunk;
    o.len = min(kChunk, rows.y - o.chunk * kChunk);
    o.behind = (rows.y - 1) / kChunk - o.chunk;
}

// A block's tiles, by one thread.  The number of the tile after the next one is asked for ahead: the counter takes as long to
// answer as memory does.
template <bool kForth>
struct Turns {
    unsigned ahead, total;
    __device__ __forceinline__ void take(const Tiles &t, const Chain &c) {
        if (t.chained) ahead = atomicAdd(c.next, 1u) + 1u;  // the counter starts at kUnset
        else ahead += gridDim.x;
    }
    __device__ __forceinline__ void start(const Tiles &t, const Chain &c) {
        ahead = blockIdx.x;
        total = tiles_of(t);
        if (t.chained) take(t, c);
    }
    // the next tile; row < 0 when there are no more
    __device__ __forceinline__ Tile next(const Tiles &t, const Chain &c) {
        Tile o;
        const unsigned k = ahead;
        o.row = -1;
        if (k >= total) return o;
        take(t, c);
        tile_at<kForth>(t, k, total, o);
        return o;
    }
};

// two channels of a staged tile
template <typename T> __device__ __forceinline__ Pair staged(const uint8_t *tile, int at) {
    return Two<T>::open(*reinterpret_cast<const typename Two<T>::Raw *>(tile + at * (int)sizeof(T)));
}
template <typename T> constexpr int tile_bytes() { return kChunk * kSlab * (int)sizeof(T); }

// ---- what is published -----------------------------------------------------------------------------------------------
__device__ __forceinline__ float settled(float x) { return __float_as_uint(x) == kUnset ? __uint_as_float(0x7fffffffu) : x; }
// What is stored of x; of kernels whose effects may leave f32, those that did stay unset.
template <bool kFinite> __device__ __forceinline__ float told(float x) {
    return kFinite ? (fabsf(x) <= kMostF32 ? x : __uint_as_float(kUnset)) : settled(x);
}
__device__ __forceinline__ bool is_set(float x) { return __float_as_uint(x) != kUnset; }

template <bool kFinite>
__device__ __forceinline__ void publish_effect(const Chain &c, int64_t at, Pair A, Pair H) {
    const float2 a = parts(A), h = parts(H);
    asm volatile("st.relaxed.gpu.global.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(c.effect + at * 2), "f"(told<kFinite>(a.x)),
                 "f"(told<kFinite>(h.x)), "f"(told<kFinite>(a.y)), "f"(told<kFinite>(h.y))
                 : "memory");
}
template <bool kFinite>
__device__ __forceinline__ void publish_result(const Chain &c, int64_t at, Pair S) {
    const float2 s = parts(S);
    asm volatile("st.relaxed.gpu.global.v2.f32 [%0], {%1, %2};" ::"l"(c.result + at), "f"(told<kFinite>(s.x)), "f"(told<kFinite>(s.y))
                 : "memory");
}
__device__ __forceinline__ float4 read_effect(const Chain &c, int64_t at) {
    float4 f;
    asm volatile("ld.relaxed.gpu.global.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(f.x), "=f"(f.y), "=f"(f.z), "=f"(f.w)
                 : "l"(c.effect + at * 2)
                 : "memory");
    return f;
}
__device__ __forceinline__ float2 read_result(const Chain &c, int64_t at) {
    float2 f;
    asm volatile("ld.relaxed.gpu.global.v2.f32 {%0, %1}, [%2];" : "=f"(f.x), "=f"(f.y) : "l"(c.result + at) : "memory");
    return f;
}

// The state that enters a tile from the `n` tiles that are looked back over, by the whole block; kStep is how far a
// neighbour's slot lies off.  Each warp reads two of them at most, so that one trip to memory serves all.  Warp kWho has the
// state; a channel past the last has nothing to wait for.  False, for all threads, when the wait gave up: the state is then a NaN, so
// that what the tile tells others is none either.
struct Window {
    float4 effect[kBack][32];
    float2 result[kBack][32];
    int ready[kBack];  // 1: the result, 2: the effect
    int gave_up;
};
template <int kStep, int kWho>
__device__ __forceinline__ bool look_back(const Chain &c, Window &win, int64_t slot, int D, int d, int n, Pair &S) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint64_t since = 0;
    for (unsigned tries = 0;; ++tries) {
        float2 res[2] = {};
        float4 eff[2] = {};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int j = warp + i * kWarps;
            if (j < n && d < D) {
                const int64_t at = (slot + (int64_t)kStep * (j + 1)) * D + d;
                res[i] = read_result(c, at);
                if (j + 1 < n) eff[i] = read_effect(c, at);
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int j = warp + i * kWarps;
            if (j < n) {
                win.result[j][lane] = res[i];
                win.effect[j][lane] = eff[i];
                const bool r = __all_sync(0xffffffffu, is_set(res[i].x) && is_set(res[i].y));
                const bool e = __all_sync(0xffffffffu, is_set(eff[i].x) && is_set(eff[i].y) && is_set(eff[i].z) && is_set(eff[i].w));
                if (lane == 0) win.ready[j] = (r ? 1 : 0) + (e ? 2 : 0);
            }
        }
        __syncthreads();
        // the nearest tile whose result is there, and whether the effects of those between are
        const int word = lane < n ? win.ready[lane] : 0;
        const unsigned r = __ballot_sync(0xffffffffu, word & 1), e = __ballot_sync(0xffffffffu, word & 2);
        const unsigned between = (r & (0u - r)) - 1u;
        if (r != 0 && (e & between) == between) {
            if (warp == kWho) {
                int j = __ffs(r) - 1;
                const float2 f = win.result[j][lane];
                S = pair(f.x, f.y);
                for (--j; j >= 0; --j) {
                    const float4 t = win.effect[j][lane];
                    S = fma(pair(t.x, t.z), S, pair(t.y, t.w));
                }
            }
            return true;
        }
        if (threadIdx.x == 0 && (tries & 63u) == 63u) {
            unsigned gave_up;
            asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(gave_up) : "l"(c.next + 1) : "memory");
            const uint64_t now = ptx::globaltimer();
            if (since == 0) since = now;
            if (gave_up != kUnset || now - since > kWaitNs) {
                atomicExch(c.next + 1, 1u);
                win.gave_up = 1;
            }
        }
        __syncthreads();
        if (win.gave_up) {
            S = both(__uint_as_float(0x7fffffffu));
            return false;
        }
    }
}

// The channels of a tile that are apart: whether there are any, two bits a lane, what the fold gave as their and their neighbours'
// result, and the tile.
struct Apart {
    int any;
    int of[32];
    float2 folded[32];
    Tile tile;
};
// By the warp that tells a tile's result, which stayed unset where it is not finite: such a channel is apart if it is the tile's
// effect that left f32; else an infinity or a NaN enters the tile, and its result is told here.
__device__ __forceinline__ void find_apart(Apart &apart, const Chain &c, int64_t at, const Tile &o, bool tells, Pair A, Pair H, Pair end) {
    const float2 e = parts(end);
    const bool odd = !(fabsf(e.x) <= kMostF32 && fabsf(e.y) <= kMostF32);
    if (!__any_sync(0xffffffffu, odd)) return;
    const float2 f = parts(fma(H, both(0.f), A * both(0.f)));  // a NaN where either is none or infinite
    const int lane = threadIdx.x & 31, bits = (f.x == 0.f ? 0 : 1) | (f.y == 0.f ? 0 : 2);
    apart.of[lane] = bits;
    apart.folded[lane] = e;
    if (lane == 0) apart.tile = o;
    if (odd && bits == 0 && tells) publish_result<false>(c, at, end);
    if (bits != 0) apart.any = 1;
}
__device__ __forceinline__ Pair choose(int bits, Pair x, Pair rest) {
    const float2 f = parts(x), g = parts(rest);
    return pair(bits & 1 ? f.x : g.x, bits & 2 ? f.y : g.y);
}
template <typename T> __device__ __forceinline__ void store_some(T *p, Pair x, int bits) {
    const typename Two<T>::Raw raw = Two<T>::close(x);
    const T *const f = reinterpret_cast<const T *>(&raw);
    if (bits & 1) p[0] = f[0];
    if (bits & 2) p[1] = f[1];
}

// ---- launches --------------------------------------------------------------------------------------------------------

// Blocks of an SM and stages of a block: as many blocks as the threads' registers allow and two stages each leave room for.  That is
// three in the forward, but two of bf16 with f32 decays and a gate and of f32 without a gate, and one of f32 with it; two in the
// gradient, but one of f32.
struct Room {
    int per_sm, stages;
};
constexpr int kMaxStages = 4;
constexpr Room room_for(int stage_bytes, int most) {
    const int room = 225 * 1024, fixed = (int)sizeof(Window) + kWarps * 1536 + 2048;  // beside the stages
    int per_sm = room / (2 * stage_bytes + fixed);
    per_sm = per_sm > most ? most : per_sm;
    int stages = (room / per_sm - fixed) / stage_bytes;
    return {per_sm, stages > kMaxStages ? kMaxStages : stages};
}

// The map of an array [rows, D] for boxes of a tile.
template <typename T> bool tile_map(CUtensorMap *m, const T *at, const Shape &p) {
    return make_map_2d(m, sizeof(T) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                       (uint32_t)sizeof(T), at, (uint64_t)p.D, (uint64_t)total_rows(p), kSlab, kChunk,
                       CU_TENSOR_MAP_SWIZZLE_NONE);
}

// Tiles that a look back reads at once: about those of its chain that are worked on at the same time.
inline int window_for(const Tiles &t, int64_t grid) {
    const int64_t chains = t.q.rows == nullptr ? (int64_t)t.q.nseq * t.slabs : t.slabs, w = grid / chains + 2;
    return (int)(w < kBack ? w : kBack);
}

// Lets a kernel use so many bytes of dynamic shared memory; asked of the runtime once per kernel and device.
template <auto kKernel> bool allow_dynamic(int bytes) {
    constexpr int kDevices = 64;
    static std::atomic<bool> allowed[kDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    if (dev < kDevices && allowed[dev].load(std::memory_order_acquire)) return true;
    if (cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
    if (dev < kDevices) allowed[dev].store(true, std::memory_order_release);
    return true;
}

}  // namespace scan
}  // namespace gla
