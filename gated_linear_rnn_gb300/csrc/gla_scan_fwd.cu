// gla_scan_fwd.cu — the gated recurrence over chunks (see gla_scan_tiles.cuh): one pass over x, g and gate.
#include <type_traits>

#include "gla_scan_tiles.cuh"

GLA_DEFINE_STATUS(scan_fwd)

namespace gla {
namespace scan {
namespace {

constexpr int kPerSm = 768 / kTileThreads;  // blocks that the registers allow

template <typename T, typename TG, bool kGate> struct Ring {
    static constexpr int x = 0, g = tile_bytes<T>(), z = g + tile_bytes<TG>();
    static constexpr int bytes = z + (kGate ? tile_bytes<T>() : 0);
};

// The rows of a tile's channels that are apart, one warp after the other from the state that enters the tile; by all threads, after
// a barrier behind the writes of enters and apart.  x and g come from memory, since their stage has been refilled, for all warps at
// once, and wait in local memory: the kernel's registers are taken.
template <typename T, typename TG, int kForm, bool kGate>
__device__ __forceinline__ void again(const T *x, const TG *g, const T *gate, T *out, float *hT, float *states, Chain chain, int D,
                                      int act, const Apart &apart, float2 (&enters)[32]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, bits = apart.of[lane];
    const Tile o = apart.tile;
    const int d = o.col + 2 * lane, n = min(kLane, o.len - warp * kLane);
    const int64_t first = (int64_t)(o.row + warp * kLane) * D + d;
    Decay a[kLane];
    Pair v[kLane];
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        if (bits == 0) break;
        a[i] = decay<kForm>(load_two(g + first + (int64_t)i * D));
        v[i] = input<kForm>(a[i], load_two(x + first + (int64_t)i * D));
    }
    __syncthreads();  // all warps have read what enters the tile
    for (int w = 0; w < kWarps; ++w) {
        if (w == warp && bits != 0 && n > 0) {
            const float2 e = enters[lane];
            Pair S = pair(e.x, e.y);
            if (states != nullptr)
                store_some(states + state_slot(o.start(), o.seq, o.chunk * kChunk + warp * kLane) * D + d, S, bits);
#pragma unroll 1
            for (int i = 0; i < n; ++i) v[i] = S = decayed(a[i], S, v[i]);
            enters[lane] = parts(S);
        }
        __syncthreads();
    }
    if (warp == kWarps - 1 && bits != 0) {
        const float2 e = enters[lane], f = apart.folded[lane];
        const Pair end = choose(bits, pair(e.x, e.y), pair(f.x, f.y));
        if (o.behind > 0) publish_result<false>(chain, (int64_t)o.slot * D + d, end);
        else if (hT != nullptr) store_state(hT + (int64_t)o.seq * D + d, end);
    }
    if (out == nullptr || bits == 0) return;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        const int64_t at = first + (int64_t)i * D;
        store_some(out + at, kGate ? v[i] * activation(load_two(gate + at), act) : v[i], bits);
    }
}

template <typename T, typename TG, int kForm, bool kGate>
__global__ void __launch_bounds__(kTileThreads, kPerSm)
tiles_fwd_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mg,
                 const __grid_constant__ CUtensorMap mz, const T *x, const TG *g, const T *gate,
                 const float *__restrict__ h0, T *__restrict__ out, float *__restrict__ hT, float *__restrict__ states, Tiles t,
                 Chain chain, int act, int stages) {
    using namespace ptx;
    using R = Ring<T, TG, kGate>;
    if (tiles_of(t) == 0 && t.walked) return;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ float4 both_effects[2][kWarps][32];  // of this tile and the one before
    __shared__ float2 enters[32];
    __shared__ Window win;
    __shared__ Apart apart;
    __shared__ Tile tiles[kMaxStages];
    __shared__ __align__(8) uint64_t full[kMaxStages];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, D = t.D;
    const uint32_t base = smem_u32(ring), bar = smem_u32(full);
    Turns<true> turns;

    // by one thread: the next tile into a stage; its gate, which a tile's last part reads, later than the rest
    auto order = [&](int st) {
        tiles[st] = turns.next(t, chain);
        const Tile &o = tiles[st];
        if (o.row < 0) return;
        const uint32_t to = base + (uint32_t)(st * R::bytes), b = bar + 8u * (uint32_t)st;
        mbar_expect_tx(b, R::z);
        tma_load_2d(to + R::g, &mg, o.col, o.row, b);
        tma_load_2d(to + R::x, &mx, o.col, o.row, b);
    };
    auto order_gate = [&](int st) {
        const Tile &o = tiles[st];
        if (!kGate || o.row < 0) return;
        const uint32_t b = bar + 8u * (uint32_t)st;
        mbar_expect_tx(b, R::bytes - R::z);
        tma_load_2d(base + (uint32_t)(st * R::bytes + R::z), &mz, o.col, o.row, b);
    };
    if (threadIdx.x == 0) {
        win.gave_up = 0;
        if (is_log(kForm)) apart.any = 0;
        turns.start(t, chain);
        for (int st = 0; st < stages; ++st) mbar_init(bar + 8u * (uint32_t)st, kGate ? 2 : 1);
        fence_mbar_init();
        for (int st = 0; st < stages; ++st) {
            order(st);
            order_gate(st);
        }
    }
    // sequences without tokens pass their state on
    if (hT != nullptr && !t.walked)
        for (int s = blockIdx.x; s < t.q.nseq; s += gridDim.x)
            if (rows_of(t.q, s).y == 0)
                for (int d = threadIdx.x; d < D; d += kTileThreads)
                    hT[(int64_t)s * D + d] = h0 != nullptr ? __ldg(h0 + (int64_t)s * D + d) : 0.f;
    __syncthreads();

    int st = 0, half = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (bool first = true;; first = false, half ^= 1) {
        const Tile o = tiles[st];
        if (o.row < 0) break;
        const uint8_t *stage = ring + st * R::bytes + (warp * kLane * kSlab + 2 * lane) * (int)sizeof(T);
        uint8_t *stage_g = ring + st * R::bytes + R::g + (warp * kLane * kSlab + 2 * lane) * (int)sizeof(TG);
        if (!mbar_wait(bar + 8u * (uint32_t)st, phase, nullptr, kWaitNs)) {
            win.gave_up = 1;
            // the thread's first row has a decay of NaN then, and so has all that is told of the tile
            store_two(reinterpret_cast<TG *>(stage_g), both(__uint_as_float(0x7fffffffu)));
        }
        const int d = o.col + 2 * lane, n = min(kLane, o.len - warp * kLane);  // the warp's rows, none or fewer where n < 8
        auto &effects = both_effects[half];
        // the warp's rows from a zero state: h, and the product of the decays up to each
        Pair h[kLane], P[kLane];
        auto local = [&](auto whole_run) {
            Pair hh = both(0.f), PP = both(1.f);
#pragma unroll
            for (int i = 0; i < kLane; ++i) {
                if (whole_run.value || i < n) {
                    const Decay a = decay<kForm>(staged<TG>(stage_g, i * kSlab));
                    const Pair b = input<kForm>(a, staged<T>(stage + R::x, i * kSlab));
                    hh = i == 0 ? b : decayed(a, hh, b);
                    PP = i == 0 ? whole(a) : decayed(a, PP);
                }
                h[i] = hh;
                P[i] = PP;
            }
        };
        if (n == kLane) local(std::true_type{});
        else local(std::false_type{});
        {
            const float2 a = parts(P[kLane - 1]), b = parts(h[kLane - 1]);
            effects[warp][lane] = make_float4(a.x, a.y, b.x, b.y);
        }
        __syncthreads();
        // x and g are read, and the tile of the round before is done
        if (threadIdx.x == 0) {
            order(st);
            if (!first) order_gate(st == 0 ? stages - 1 : st - 1);
        }
        const int64_t at = (int64_t)o.slot * D + d;
        constexpr int kWho = kWarps - 1;
        Pair A = both(1.f), H = both(0.f), S = both(0.f);  // the effect of the warps before this one, and what enters the tile
        for (int w = 0; w < warp; ++w) {
            const float4 f = effects[w][lane];
            H = fma(pair(f.x, f.y), H, pair(f.z, f.w));
            A = A * pair(f.x, f.y);
        }
        const Pair tA = A * P[kLane - 1], tH = fma(P[kLane - 1], H, h[kLane - 1]);
        if (warp == kWho && d < D) {  // tA and tH are the tile's effect
            if (o.chunk > 0 && o.behind > 0) publish_effect<is_log(kForm)>(chain, at, tA, tH);
            if (o.chunk == 0 && h0 != nullptr) S = load_state(h0 + (int64_t)o.seq * D + d);
        }
        if (o.chunk > 0) ok = look_back<-1, kWho>(chain, win, o.slot, D, d, min(o.chunk, t.window), S);
        if (warp == kWho) {
            const Pair end = fma(tA, S, tH);
            if (d < D) {
                if (o.behind > 0) publish_result<is_log(kForm)>(chain, at, end);
                else if (hT != nullptr) store_state(hT + (int64_t)o.seq * D + d, end);
            }
            enters[lane] = parts(S);
            if (is_log(kForm)) find_apart(apart, chain, at, o, d < D && o.behind > 0, tA, tH, end);
        }
        __syncthreads();
        ok = ok && !win.gave_up;
        if (!ok) break;
        if (d < D && n > 0) {
            const float2 e = enters[lane];
            S = fma(A, pair(e.x, e.y), H);
            if (states != nullptr)
                store_state(states + state_slot(o.start(), o.seq, o.chunk * kChunk + warp * kLane) * D + d, S);
            T *to = out + (int64_t)(o.row + warp * kLane) * D + d;
            auto emit = [&](auto whole_run, int kind) {
#pragma unroll
                for (int i = 0; i < kLane; ++i)
                    if (whole_run.value || i < n) {
                        Pair y = fma(P[i], S, h[i]);
                        if (kGate) y = y * activation(staged<T>(stage + R::z, i * kSlab), kind);
                        store_two(to, y);
                        to += D;
                    }
            };
            if (out == nullptr) {
            } else if (n < kLane) emit(std::false_type{}, act);
            else if (!kGate || act == kSilu) emit(std::true_type{}, kSilu);
            else if (act == kSigmoid) emit(std::true_type{}, kSigmoid);
            else emit(std::true_type{}, kNone);
        }
        if (is_log(kForm) && apart.any) {
            again<T, TG, kForm, kGate>(x, g, gate, out, hT, states, chain, D, act, apart, enters);
            apart.any = 0;
        }
        if (++st == stages) {
            st = 0;
            phase ^= 1;
        }
    }
    // a block that gave up waits for what it has ordered
    if (!ok && threadIdx.x == 0) {
        record_status(GLA_ERR_TIMEOUT);
        if (t.chained) atomicExch(chain.next + 1, 1u);  // who waits for its tiles need not wait longer
        order_gate(st);
        for (int i = 0; i < stages; ++i) {
            if (++st == stages) {
                st = 0;
                phase ^= 1;
            }
            if (tiles[st].row >= 0) mbar_wait(bar + 8u * (uint32_t)st, phase, nullptr, kWaitNs);
        }
    }
}

template <typename T, typename TG, int kForm, bool kGate>
bool launch(const Shape &p, Tiles t, const Chain &chain, const T *x, const TG *g, const T *gate, const float *h0, T *out,
            float *hT, float *states, cudaStream_t st) {
    using R = Ring<T, TG, kGate>;
    constexpr Room room = room_for(R::bytes, kPerSm);
    constexpr int bytes = room.stages * R::bytes;
    static_assert(room.stages >= 2, "a tile is worked on while the next one comes in");
    constexpr auto kKernel = tiles_fwd_kernel<T, TG, kForm, kGate>;
    CUtensorMap mx, mg, mz;
    if (!tile_map(&mx, x, p) || !tile_map(&mg, g, p) || !tile_map(&mz, kGate ? gate : x, p)) return false;
    if (!allow_dynamic<kKernel>(bytes)) return false;
    int64_t grid = (int64_t)device_info().sm_count * room.per_sm;
    if (grid > (int64_t)t.total) grid = t.total;
    if (grid < 1) grid = 1;
    t.window = window_for(t, grid);
    kKernel<<<(unsigned)grid, kTileThreads, bytes, st>>>(mx, mg, mz, x, g, gate, h0, out, hT, states, t, chain, p.act, room.stages);
    count_launches(1);
    return true;
}

}  // namespace

bool tiles_fwd(const Shape &p, const Tiles &t, const Chain &chain, const void *x, const void *g, const void *gate,
               const float *h0, void *out, float *hT, float *states, int dtype, int g_dtype, cudaStream_t st) {
    bool ok = false;
#define GLA_RUN(T, TG, F, G)                                                                                              \
    ok = launch<T, TG, F, G>(p, t, chain, (const T *)x, (const TG *)g, (const T *)gate, h0, (T *)out, hT, states, st)
    GLA_SCAN_DISPATCH(dtype, g_dtype, gate != nullptr, GLA_RUN)
#undef GLA_RUN
    return ok;
}

}  // namespace scan
}  // namespace gla
