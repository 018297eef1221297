// gla_scan_bwd.cu — the gradient of the gated recurrence over chunks (see gla_scan_tiles.cuh), from the states before runs.
//
// A warp's states h come from the one before its rows, and dh from what is behind them: dh_t = up_t + D_t with up_t =
// dout_t act(gate_t) and D_{t-1} = a_t dh_t, an effect D -> A D + C of a row, a warp's rows and a tile like the forward's.
// Everything but dh is found on the way there, so that little is left for the rows once it is known.
#include <type_traits>

#include "gla_scan_tiles.cuh"

GLA_DEFINE_STATUS(scan_bwd)

namespace gla {
namespace scan {
namespace {

constexpr int kPerSm = 512 / kTileThreads;  // blocks that the registers allow

template <typename T, typename TG, bool kGate> struct Ring {
    static constexpr int x = 0, g = tile_bytes<T>(), u = g + tile_bytes<TG>(), z = u + tile_bytes<T>();
    static constexpr int bytes = z + (kGate ? tile_bytes<T>() : 0);
};

template <typename T, typename TG, int kForm, bool kGate>
__global__ void __launch_bounds__(kTileThreads, kPerSm)
tiles_bwd_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mg,
                 const __grid_constant__ CUtensorMap mu, const __grid_constant__ CUtensorMap mz,
                 const float *__restrict__ dhT, const float *__restrict__ states, T *__restrict__ dx, TG *__restrict__ dg,
                 T *__restrict__ dgate, float *__restrict__ dh0, Tiles t, Chain chain, int act, int stages) {
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
    Turns<false> turns;

    auto order = [&](int st) {  // by one thread
        tiles[st] = turns.next(t, chain);
        const Tile &o = tiles[st];
        if (o.row < 0) return;
        const uint32_t to = base + (uint32_t)(st * R::bytes), b = bar + 8u * (uint32_t)st;
        mbar_expect_tx(b, R::bytes);
        tma_load_2d(to + R::g, &mg, o.col, o.row, b);
        tma_load_2d(to + R::x, &mx, o.col, o.row, b);
        tma_load_2d(to + R::u, &mu, o.col, o.row, b);
        if (kGate) tma_load_2d(to + R::z, &mz, o.col, o.row, b);
    };
    const bool orders = threadIdx.x == kTileThreads - 32;  // not of the warp that folds what is looked back over
    if (orders) {
        win.gave_up = 0;
        if (is_log(kForm)) apart.any = 0;
        turns.start(t, chain);
        for (int st = 0; st < stages; ++st) mbar_init(bar + 8u * (uint32_t)st, 1);
        fence_mbar_init();
        for (int st = 0; st < stages; ++st) order(st);
    }
    // sequences without tokens pass the gradient of their state on
    if (dh0 != nullptr && !t.walked)
        for (int s = blockIdx.x; s < t.q.nseq; s += gridDim.x)
            if (rows_of(t.q, s).y == 0)
                for (int d = threadIdx.x; d < D; d += kTileThreads)
                    dh0[(int64_t)s * D + d] = dhT != nullptr ? __ldg(dhT + (int64_t)s * D + d) : 0.f;
    __syncthreads();

    // the state before the warp's rows of a tile, asked for a tile ahead
    auto state_of = [&](const Tile &o) {
        const int d = o.col + 2 * lane, t = warp * kLane;
        if (o.row < 0 || d >= D || t >= o.len) return both(0.f);
        return load_state(states + state_slot(o.start(), o.seq, o.chunk * kChunk + t) * D + d);
    };
    int st = 0, half = 0;
    uint32_t phase = 0;
    bool ok = true;
    Pair next = state_of(tiles[0]);
    for (;; half ^= 1) {
        const Tile o = tiles[st];
        if (o.row < 0) break;
        const int d = o.col + 2 * lane, n = min(kLane, o.len - warp * kLane);
        const bool on = d < D;
        const int64_t at = (int64_t)o.slot * D + d, out_at = (int64_t)(o.row + warp * kLane) * D + d;
        Pair h = next;
        const uint8_t *stage = ring + st * R::bytes + (warp * kLane * kSlab + 2 * lane) * (int)sizeof(T);
        uint8_t *stage_g = ring + st * R::bytes + R::g + (warp * kLane * kSlab + 2 * lane) * (int)sizeof(TG);
        if (!mbar_wait(bar + 8u * (uint32_t)st, phase, nullptr, kWaitNs)) {
            win.gave_up = 1;
            // the thread's first row has a decay of NaN then, and so has all that is told of the tile
            store_two(reinterpret_cast<TG *>(stage_g), both(__uint_as_float(0x7fffffffu)));
        }
        auto &effects = both_effects[half];
        // the warp's rows: their decays, dout times the gate's factor, dg without dh, and the rows' effect
        Decay a[kLane];
        Pair up[kLane], da[kLane];
        auto local = [&](auto whole_run, int kind) {
            T *to = kGate ? dgate + out_at : nullptr;
            Pair A = both(1.f), C = both(0.f);
#pragma unroll
            for (int i = 0; i < kLane; ++i)
                if (whole_run.value || i < n) {
                    a[i] = decay<kForm>(staged<TG>(stage_g, i * kSlab));
                    const Pair x = staged<T>(stage + R::x, i * kSlab), w = rest(a[i]);
                    A = i == 0 ? whole(a[i]) : decayed(a[i], A);
                    da[i] = whole(a[i]) * (leaks(kForm) ? fma(x, both(-1.f), h) : h);
                    if (!is_log(kForm)) da[i] = da[i] * w;
                    h = decayed(a[i], h, leaks(kForm) ? w * x : x);
                    up[i] = staged<T>(stage + R::u, i * kSlab);
                    if (kGate) {
                        Pair slope;
                        const Pair f = activation(staged<T>(stage + R::z, i * kSlab), kind, slope);
                        if (on) store_two(to, up[i] * slope * h);
                        up[i] = up[i] * f;
                        to += D;
                    }
                }
#pragma unroll
            for (int i = kLane - 1; i >= 0; --i)
                if (whole_run.value || i < n) C = decayed(a[i], up[i] + C);
            const float2 p = parts(A), q = parts(C);
            effects[warp][lane] = make_float4(p.x, p.y, q.x, q.y);
        };
        if (n < kLane) local(std::false_type{}, act);
        else if (!kGate || act == kSilu) local(std::true_type{}, kSilu);
        else if (act == kSigmoid) local(std::true_type{}, kSigmoid);
        else local(std::true_type{}, kNone);
        __syncthreads();
        if (orders) order(st);  // all of the stage is read
        constexpr int kWho = 0;
        Pair bA = both(1.f), bC = both(0.f), S = both(0.f);  // the effect of the warps behind this one, and what enters the tile
#pragma unroll
        for (int w = kWarps - 1; w > 0; --w)
            if (w > warp) {
                const float4 f = effects[w][lane];
                bC = fma(pair(f.x, f.y), bC, pair(f.z, f.w));
                bA = bA * pair(f.x, f.y);
            }
        Pair tA, tC;
        if (warp == kWho) {  // the tile's effect
            const float4 f = effects[kWho][lane];
            tC = fma(pair(f.x, f.y), bC, pair(f.z, f.w));
            tA = bA * pair(f.x, f.y);
            if (on && o.behind > 0 && o.chunk > 0) publish_effect<is_log(kForm)>(chain, at, tA, tC);
            if (on && o.behind == 0 && dhT != nullptr) S = load_state(dhT + (int64_t)o.seq * D + d);
        }
        if (o.behind > 0) ok = look_back<1, kWho>(chain, win, o.slot, D, d, min(o.behind, t.window), S);
        if (warp == kWho) {
            const Pair end = fma(tA, S, tC);
            if (on) {
                if (o.chunk > 0) publish_result<is_log(kForm)>(chain, at, end);
                else if (dh0 != nullptr) store_state(dh0 + (int64_t)o.seq * D + d, end);
            }
            enters[lane] = parts(S);
            if (is_log(kForm)) find_apart(apart, chain, at, o, on && o.chunk > 0, tA, tC, end);
        }
        __syncthreads();
        ok = ok && !win.gave_up;
        if (!ok) break;
        const float2 e = enters[lane];
        Pair K = fma(bA, pair(e.x, e.y), bC);
        next = state_of(tiles[st + 1 == stages ? 0 : st + 1]);
        if (is_log(kForm) && apart.any) {  // channels that are apart: what is behind a warp's rows from one warp after the other
            const int bits = apart.of[lane];
            __syncthreads();  // all warps have read what is behind the tile
            for (int w = kWarps - 1; w >= 0; --w) {
                if (w == warp) {
                    const float2 f = enters[lane];
                    Pair L = pair(f.x, f.y);
                    K = choose(bits, L, K);
#pragma unroll
                    for (int i = kLane - 1; i >= 0; --i)
                        if (i < n) L = decayed(a[i], up[i] + L);
                    enters[lane] = parts(L);
                }
                __syncthreads();
            }
            if (warp == kWho && bits != 0) {
                const float2 f = enters[lane], l = apart.folded[lane];
                const Pair end = choose(bits, pair(f.x, f.y), pair(l.x, l.y));
                if (o.chunk > 0) publish_result<false>(chain, at, end);
                else if (dh0 != nullptr) store_state(dh0 + (int64_t)o.seq * D + d, end);
            }
            apart.any = 0;
        }
        auto backwards = [&](auto whole_run) {
            T *to = dx + out_at + (int64_t)(kLane - 1) * D;
            TG *to_g = dg + out_at + (int64_t)(kLane - 1) * D;
#pragma unroll
            for (int i = kLane - 1; i >= 0; --i) {
                if (whole_run.value || i < n) {
                    const Pair dh = up[i] + K;
                    store_two(to_g, dh * da[i]);
                    store_two(to, input<kForm>(a[i], dh));
                    if (i > 0) K = decayed(a[i], dh);
                }
                to -= D;
                to_g -= D;
            }
        };
        if (on && n == kLane) backwards(std::true_type{});
        else if (on && n > 0) backwards(std::false_type{});
        if (++st == stages) {
            st = 0;
            phase ^= 1;
        }
    }
    // a block that gave up waits for what it has ordered
    if (!ok && threadIdx.x == 0) {
        record_status(GLA_ERR_TIMEOUT);
        if (t.chained) atomicExch(chain.next + 1, 1u);  // who waits for its tiles need not wait longer
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
bool launch(const Shape &p, Tiles t, const Chain &chain, const T *x, const TG *g, const T *gate, const T *dout,
            const float *dhT, const float *states, T *dx, TG *dg, T *dgate, float *dh0, cudaStream_t st) {
    using R = Ring<T, TG, kGate>;
    constexpr Room room = room_for(R::bytes, kPerSm);
    constexpr int bytes = room.stages * R::bytes;
    static_assert(room.stages >= 2, "a tile is worked on while the next one comes in");
    constexpr auto kKernel = tiles_bwd_kernel<T, TG, kForm, kGate>;
    CUtensorMap mx, mg, mu, mz;
    if (!tile_map(&mx, x, p) || !tile_map(&mg, g, p) || !tile_map(&mu, dout, p) || !tile_map(&mz, kGate ? gate : x, p)) return false;
    if (!allow_dynamic<kKernel>(bytes)) return false;
    int64_t grid = (int64_t)device_info().sm_count * room.per_sm;
    if (grid > (int64_t)t.total) grid = t.total;
    if (grid < 1) grid = 1;
    t.window = window_for(t, grid);
    kKernel<<<(unsigned)grid, kTileThreads, bytes, st>>>(mx, mg, mu, mz, dhT, states, dx, dg, dgate, dh0, t, chain, p.act,
                                                         room.stages);
    count_launches(1);
    return true;
}

}  // namespace

bool tiles_bwd(const Shape &p, const Tiles &t, const Chain &chain, const void *x, const void *g, const void *gate,
               const void *dout, const float *dhT, const float *states, void *dx, void *dg, void *dgate, float *dh0, int dtype,
               int g_dtype, cudaStream_t st) {
    bool ok = false;
#define GLA_RUN(T, TG, F, G)                                                                                                \
    ok = launch<T, TG, F, G>(p, t, chain, (const T *)x, (const TG *)g, (const T *)gate, (const T *)dout, dhT, states,       \
                             (T *)dx, (TG *)dg, (T *)dgate, dh0, st)
    GLA_SCAN_DISPATCH(dtype, g_dtype, gate != nullptr, GLA_RUN)
#undef GLA_RUN
    return ok;
}

}  // namespace scan
}  // namespace gla
