// hla_gated.cu -- gated linear recurrence over [B][n][d], elementwise per channel:
//   h_t = a_t h_{t-1} + b_t,   y_t = h_t,
//   HLA_GATE_GIVEN:   a = g,                  b = x
//   HLA_GATE_SIGMOID: a = sigma(g),           b = (1 - a) x
//   HLA_GATE_RATE:    a = exp(-r sigma(g)),   b = sqrt(1 - a^2) x
// its backward pass and its single-token step.
//
// A stretch of tokens is the map h -> A h + B (A the product of its a_t); stretches
// compose by (A1,B1) then (A2,B2) = (A2 A1, A2 B1 + B2).  The backward pass is the same
// scan in the other direction, of c_t = a_t gh_t (the gradient that token t hands to
// token t-1): gh_t = dy_t + c_{t+1}, c_t = a_t c_{t+1} + a_t dy_t.
//
// Every input element is read once and every output element written once (x, g -> y; g, y,
// dy[, x] -> dx, dg), with a few fp32 operations on each.  One CTA takes a tile of 8 warps x
// kTS tokens by 32 lanes x VEC channels, holds it in registers, and gets the state before its
// tile from the tiles before it while its own loads are the only traffic: each tile publishes
// its map (A, B) as soon as it has it, then looks back over the published maps to the nearest
// published state, folds forward from there, and publishes its own state.  The fold always runs
// state -> later tiles in order with the same fmaf, so a state has the same bits wherever the
// look-back found its start: results do not depend on timing.  Reading the inputs a second time
// instead (maps, scan, states) would move 5/3 of the forward's bytes.
//
// Measured: forward 3 x 5,003 x 1,001 fp32 (ragged) 52 us, 2.4 TB/s; 16,384 x 1,024 bf16 with
// rates 47 us, 2.1 TB/s; backward 4 x 2,048 x 512 bf16 25 us, 2.0 TB/s.  What bounds it is the
// path of one CTA, loads -> gates -> look-back -> stores, and how many CTAs are on it at once.
#include "hla_gated.cuh"
#include "hla_look_back.h"

namespace hla {
namespace gated {
namespace {

constexpr int WARPS = 8;
constexpr int kThreads = WARPS * 32;
// CTAs per SM, and tokens of one thread: about as many as leave what it holds of them in
// registers (the backward's four inputs take twice the room; single channels spill 8 to 44 bytes,
// pairs none).  A CTA mostly waits, for its loads and for the tiles before it: single channels gain
// from four per SM (3 x 5,003 x 1,001 fp32 forward 66 -> 52 us), pairs have room for two (three
// spill: 4 x 2,048 x 512 backward 26 -> 29 us).
enum Dir { FWD, BWD };
template <int VEC>
constexpr int kCtas = VEC == 1 ? 4 : 2;
template <typename T, Dir DIR, int VEC>
constexpr int kTS = DIR == FWD ? 16 : 8;
template <typename T, Dir DIR, int VEC>
constexpr int kTileT = WARPS * kTS<T, DIR, VEC>;  // tokens of one tile
constexpr int kTileLeast = WARPS * 8;
constexpr int BACK = 8;               // windows of WARPS earlier tiles kept by one look-back

// `tag` of a record: 4 * (number of the call) + kind (hla_look_back.h); anything else is left
// over from another call.

// Workspace: header, then one record per channel slot of every tile, then (backward with
// HLA_GATE_RATE) one partial sum per channel slot of every tile, in records with tag 0.
constexpr size_t kHeaderBytes = 256;

// ------------------------------------------------------------ look-back
__device__ __forceinline__ void publish(Record *p, float a, float b, unsigned long long tag) {
    const unsigned long long ab = (unsigned long long)__float_as_uint(a) | ((unsigned long long)__float_as_uint(b) << 32);
    asm volatile("{\n .reg .b128 r;\n mov.b128 r, {%1, %2};\n st.relaxed.gpu.global.b128 [%0], r;\n}\n" ::"l"(p), "l"(ab),
                 "l"(tag)
                 : "memory");
}
__device__ __forceinline__ Record peek(const Record *p) {
    unsigned long long ab, tag;
    asm volatile("{\n .reg .b128 r;\n ld.relaxed.gpu.global.b128 r, [%2];\n mov.b128 {%0, %1}, r;\n}\n"
                 : "=l"(ab), "=l"(tag)
                 : "l"(p)
                 : "memory");
    Record x;
    x.a = __uint_as_float((unsigned)ab);
    x.b = __uint_as_float((unsigned)(ab >> 32));
    x.tag = tag;
    return x;
}
// Wait, bounded, until the record belongs to call `call` and is at least a map (at least
// a state with `need_state`).  False: the limit passed and the sticky status is raised.
__device__ __forceinline__ bool await_record(const Record *p, unsigned long long call, bool need_state, Record &x, unsigned *err) {
    const unsigned long long state = 4 * call + REC_STATE, map = 4 * call + REC_MAP;
    x = peek(p);
    if (x.tag == state || (x.tag == map && !need_state)) return true;
    const uint64_t t0 = globaltimer_ns();
    do {
        __nanosleep(40);
        x = peek(p);
        if (x.tag == state || (x.tag == map && !need_state)) return true;
    } while (globaltimer_ns() - t0 < (uint64_t)kWaitLimitUs * 1000u);
    atomicOr(err, DEV_TIMEOUT);
    return false;
}

template <int VEC>
struct Shared {
    float2 agg[WARPS][32 * VEC];           // the warps' maps
    float2 back[BACK * WARPS][32 * VEC];   // maps of earlier tiles, nearest first
    int kind[WARPS][32 * VEC];             // of the newest window: REC_MAP, REC_STATE, 0 (none)
    float carry[32 * VEC];                 // state before the tile
    unsigned long long ticket, call;
};

// The state before tile `pos` of chain `chain` (positions count along the scan's
// direction, `first` is the chain's first active position) into sh.carry, and this tile's
// own state published.  `init` is the state before the chain.  Every thread of the CTA
// calls this once sh.agg is complete; false: a wait expired.
template <int VEC>
__device__ __forceinline__ bool look_back(Shared<VEC> &sh, const Args &a, size_t chain, int pos, int first,
                                          const float *init, int c0, float *out_state) {
    constexpr int C = 32 * VEC;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    Record *rec = a.rec + (chain * a.tiles) * C;
    const unsigned long long call = sh.call;
    float A = 1.f, Bv = 0.f;  // the tile's map, one channel per thread below C
    if (tid < C) {
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            const float2 m = sh.agg[w][tid];
            Bv = fmaf(m.x, Bv, m.y);
            A *= m.x;
        }
    }
    float h = 0.f;
    bool ok = true;
    if (pos == first) {
        if (tid < C && init && c0 + tid < a.d) h = init[c0 + tid];
    } else {
        if (tid < C) publish(rec + (size_t)pos * C + tid, A, Bv, 4 * call + REC_MAP);
        using Start = FoldStart<BACK, WARPS>;  // index in sh.back of the state this channel starts from
        Start start;
        for (int r = 0;; ++r) {
            const int slot = Start::slot(r);
            const int prev = pos - 1 - (slot * WARPS + warp);
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const int c = lane * VEC + v;
                Record x{};
                int kind = 0;
                if (prev >= first) {
                    // past the kept windows: wait for the states of the last one
                    ok = await_record(rec + (size_t)prev * C + c, call, Start::states_only(r), x, a.err) && ok;
                    kind = (int)(x.tag & 3);
                }
                sh.back[slot * WARPS + warp][c] = make_float2(x.a, x.b);
                sh.kind[warp][c] = kind;
            }
            if (!__syncthreads_and(ok)) {  // a state all the same, so that no later tile waits as long again
                if (tid < C) publish(rec + (size_t)pos * C + tid, 1.f, __int_as_float(0x7fc00000), 4 * call + REC_STATE);
                return false;
            }
            if (tid < C) start.look(r, [&](int w) { return sh.kind[w][tid]; });
            if (__syncthreads_and(tid >= C || start.found >= 0)) break;
        }
        if (tid < C)
            h = start.fold([&](int i) { return sh.back[i][tid].y; },
                           [&](int i, float x) { return fmaf(sh.back[i][tid].x, x, sh.back[i][tid].y); });
    }
    if (tid < C) {
        sh.carry[tid] = h;
        const float after = fmaf(A, h, Bv);
        if (a.hdr) publish(rec + (size_t)pos * C + tid, A, after, 4 * call + REC_STATE);
        if (out_state && c0 + tid < a.d) out_state[c0 + tid] = after;
    }
    __syncthreads();
    return true;
}

// This CTA's place: tiles of one position across all chains come before those of the
// next, in the order in which CTAs begin, so every tile that one waits for has begun.  False
// when there is no such tile (the header was not zeroed, or belongs to a call that still runs):
// the status word is raised, and the CTA has nothing to do.
template <int VEC>
__device__ __forceinline__ bool take_place(Shared<VEC> &sh, const Args &a) {
    if (threadIdx.x == 0) {
        if (a.hdr) {
            volatile unsigned long long *base = &a.hdr->base;
            const unsigned long long b0 = *base;  // stands until the last ticket is out
            __threadfence();
            const unsigned long long t = atomicAdd(&a.hdr->tickets, 1ull);
            sh.ticket = t - b0;
            sh.call = b0 + 1;
            if (sh.ticket == gridDim.x - 1) {  // every CTA of this call has read base
                __threadfence();
                *base = t + 1;
            }
            if (sh.ticket >= gridDim.x) atomicOr(a.err, DEV_WORKSPACE);
        } else {
            sh.ticket = blockIdx.x;
            sh.call = 0;
        }
    }
    __syncthreads();
    return sh.ticket < gridDim.x;
}

// ------------------------------------------------------------ forward
// The state before this warp's tokens: the tile's, taken through the maps of the warps before.
template <class V, int VEC>
HLA_DEVICE V before_warp(const Shared<VEC> &sh, int warp, int lane) {
    V h;
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        h.v[v] = sh.carry[lane * VEC + v];
        for (int w = 0; w < warp; ++w) {
            const float2 mp = sh.agg[w][lane * VEC + v];
            h.v[v] = fmaf(mp.x, h.v[v], mp.y);
        }
    }
    return h;
}

// One tile: loads, gates, the warps' maps, the state before the tile, outputs.  FULL: every
// thread of the CTA has all its TS tokens, so nothing is predicated.
template <typename T, int GATE, int VEC, bool FULL>
HLA_DEVICE void fwd_tile(Shared<VEC> &sh, const Args &a, size_t chain, int pos, int b, int c0, int t0, int m, int len) {
    constexpr int TS = kTS<T, FWD, VEC>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, ch = c0 + lane * VEC;
    const size_t so = (size_t)b * a.d;
    raw_t<T, VEC> xr[TS] = {}, gr[TS] = {};
    const Slice<T, VEC> xs(a.x, b, c0, t0, lane), gs(a.g, b, c0, t0, lane), ys(a.o1, b, c0, t0, lane);
#pragma unroll
    for (int i = 0; i < TS; ++i)
        if (FULL || i < m) gr[i] = gs.load(i);
#pragma unroll
    for (int i = 0; i < TS; ++i)
        if (FULL || i < m) xr[i] = xs.load(i);
    const Num<T, VEC> r = rate_of<GATE, Num<T, VEC>>(a, ch);
    Num<T, VEC> ea[TS], eb[TS], A = splat<Num<T, VEC>>(1.f), Bv = splat<Num<T, VEC>>(0.f);
#pragma unroll
    for (int i = 0; i < TS; ++i) {
        Num<T, VEC> x, g;
        unpack(xr[i], x.v);
        unpack(gr[i], g.v);
        gate_fwd<GATE>(g, r, x, ea[i], eb[i]);
        if (!FULL && i >= m) {
            ea[i] = splat<Num<T, VEC>>(1.f);
            eb[i] = splat<Num<T, VEC>>(0.f);
        }
        Bv = fma_(ea[i], Bv, eb[i]);
        A = mul_(A, ea[i]);
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) sh.agg[warp][lane * VEC + v] = make_float2(A.v[v], Bv.v[v]);
    __syncthreads();
    const bool last = pos == (len - 1) / kTileT<T, FWD, VEC>;
    if (!look_back<VEC>(sh, a, chain, pos, 0, a.state_in ? a.state_in + so : nullptr, c0,
                        last && a.out_state ? a.out_state + so : nullptr))
        return;
    Num<T, VEC> h = before_warp<Num<T, VEC>>(sh, warp, lane);
#pragma unroll
    for (int i = 0; i < TS; ++i) {
        h = fma_(ea[i], h, eb[i]);
        if (FULL || i < m) ys.store(i, h.v);
    }
}

template <typename T, int GATE, int VEC>
__global__ void __launch_bounds__(kThreads, kCtas<VEC>) gated_fwd_kernel(const Args a) {
    constexpr int TS = kTS<T, FWD, VEC>, TILE_T = kTileT<T, FWD, VEC>;
    constexpr int C = 32 * VEC;
    __shared__ Shared<VEC> sh;
    if (!take_place(sh, a)) return;
    const unsigned chains = (unsigned)a.B * a.slices, ticket = __shfl_sync(0xffffffffu, (unsigned)sh.ticket, 0);
    const int pos = (int)(ticket / chains);
    const unsigned chain = ticket % chains;
    const int b = (int)(chain / a.slices), c0 = (int)(chain % a.slices) * C;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, ch = c0 + lane * VEC;
    const int len = length_of(a, b);
    const size_t so = (size_t)b * a.d;
    if (len == 0 && pos == 0 && a.out_state) {  // no tokens: the state passes through
        for (int c = threadIdx.x; c < C; c += kThreads)
            if (c0 + c < a.d) a.out_state[so + c0 + c] = a.state_in ? a.state_in[so + c0 + c] : 0.f;
    }
    if (pos * TILE_T >= len) return;
    const int t0 = pos * TILE_T + __shfl_sync(0xffffffffu, warp, 0) * TS;  // the warp's, in uniform registers
    const int m = ch < a.d ? min(TS, len - t0) : 0;  // tokens of this thread (may be <= 0)
    if ((pos + 1) * TILE_T <= len && c0 + C <= a.d)  // the same for the whole CTA
        fwd_tile<T, GATE, VEC, true>(sh, a, chain, pos, b, c0, t0, m, len);
    else
        fwd_tile<T, GATE, VEC, false>(sh, a, chain, pos, b, c0, t0, m, len);
}

// ------------------------------------------------------------ backward
template <typename T, int GATE, int VEC, bool FULL>
HLA_DEVICE void bwd_tile(Shared<VEC> &sh, const Args &a, size_t chain, int pos, int tile, int b, int c0, int t0, int m,
                         int len) {
    constexpr int TS = kTS<T, BWD, VEC>;
    constexpr int C = 32 * VEC;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, ch = c0 + lane * VEC;
    const size_t so = (size_t)b * a.d;
    raw_t<T, VEC> gr[TS] = {}, dr[TS] = {}, yr[TS] = {}, xr[TS] = {};
    const Slice<T, VEC> gs(a.g, b, c0, t0, lane), ds(a.dy, b, c0, t0, lane), xs(a.x, b, c0, t0, lane),
        ys(a.y, b, c0, t0 - 1, lane),  // y one token earlier: h_{t-1}; the token before the first is state_in
        os(a.o1, b, c0, t0, lane), qs(a.o2, b, c0, t0, lane);
#pragma unroll
    for (int i = 0; i < TS; ++i) {
        if (FULL || i < m) {
            gr[i] = gs.load(i);
            dr[i] = ds.load(i);
        }
    }
#pragma unroll
    for (int i = 0; i < TS; ++i) {
        if (FULL || i < m) {
            if (i > 0 || t0 > 0) yr[i] = ys.load(i);
            if constexpr (GATE != HLA_GATE_GIVEN) xr[i] = xs.load(i);
        }
    }
    const Num<T, VEC> r = rate_of<GATE, Num<T, VEC>>(a, ch);
    Num<T, VEC> h0 = splat<Num<T, VEC>>(0.f), kept[TS], A = splat<Num<T, VEC>>(1.f), Bv = splat<Num<T, VEC>>(0.f);
    if (t0 == 0 && a.state_in) {
#pragma unroll
        for (int v = 0; v < VEC; ++v)
            if (ch + v < a.d) h0.v[v] = a.state_in[so + ch + v];
    }
#pragma unroll
    for (int i = TS - 1; i >= 0; --i) {
        Num<T, VEC> g, dy;
        unpack(gr[i], g.v);
        unpack(dr[i], dy.v);
        Num<T, VEC> at;
        kept[i] = gate_keep<GATE>(g, r, at);
        if (!FULL && i >= m) {
            kept[i] = splat<Num<T, VEC>>(kKeptOff<GATE>);
            at = splat<Num<T, VEC>>(1.f);
        }
        Bv = mul_(at, add_(dy, Bv));
        A = mul_(A, at);
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) sh.agg[warp][lane * VEC + v] = make_float2(A.v[v], Bv.v[v]);
    __syncthreads();
    const int first = a.tiles - 1 - (len - 1) / kTileT<T, BWD, VEC>;
    if (!look_back<VEC>(sh, a, chain, pos, first, a.d_state_out ? a.d_state_out + so : nullptr, c0,
                        tile == 0 && a.out_state ? a.out_state + so : nullptr))
        return;
    Num<T, VEC> c = before_warp<Num<T, VEC>>(sh, warp, lane), sum = splat<Num<T, VEC>>(0.f);
#pragma unroll
    for (int i = TS - 1; i >= 0; --i) {
        Num<T, VEC> g, dy, x = splat<Num<T, VEC>>(0.f), y, dx, dg, drv, at;
        unpack(gr[i], g.v);
        unpack(dr[i], dy.v);
        unpack(yr[i], y.v);
        if (i == 0 && t0 == 0) y = h0;
        if constexpr (GATE != HLA_GATE_GIVEN) unpack(xr[i], x.v);
        const Num<T, VEC> gh = add_(dy, c);
        gate_bwd<GATE>(g, r, x, y, gh, kept[i], dx, dg, drv, at);
        c = mul_(at, gh);
        if (FULL || i < m) {
            if constexpr (GATE == HLA_GATE_RATE) sum = add_(sum, drv);
            os.store(i, dx.v);
            qs.store(i, dg.v);
        }
    }
    if constexpr (GATE == HLA_GATE_RATE) {
        if (a.part) {  // the tile's sum of every channel, warps in order
            __syncthreads();
#pragma unroll
            for (int v = 0; v < VEC; ++v) sh.agg[warp][lane * VEC + v].x = sum.v[v];
            __syncthreads();
            if (threadIdx.x < C) {
                float s = 0.f;
#pragma unroll
                for (int w = 0; w < WARPS; ++w) s += sh.agg[w][threadIdx.x].x;
                Record *p = a.part + (chain * a.tiles + tile) * C + threadIdx.x;
                *reinterpret_cast<float4 *>(p) = make_float4(s, 0.f, 0.f, 0.f);
            }
        }
    }
}

template <typename T, int GATE, int VEC>
__global__ void __launch_bounds__(kThreads, kCtas<VEC>) gated_bwd_kernel(const Args a) {
    constexpr int TS = kTS<T, BWD, VEC>, TILE_T = kTileT<T, BWD, VEC>;
    constexpr int C = 32 * VEC;
    __shared__ Shared<VEC> sh;
    if (!take_place(sh, a)) return;
    const unsigned chains = (unsigned)a.B * a.slices, ticket = __shfl_sync(0xffffffffu, (unsigned)sh.ticket, 0);
    const int pos = (int)(ticket / chains);  // counts from the last tile
    const unsigned chain = ticket % chains;
    const int b = (int)(chain / a.slices), c0 = (int)(chain % a.slices) * C;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, ch = c0 + lane * VEC;
    const int len = length_of(a, b), tile = a.tiles - 1 - pos;
    const size_t so = (size_t)b * a.d;
    if (len == 0 && tile == 0 && a.out_state) {
        for (int c = threadIdx.x; c < C; c += kThreads)
            if (c0 + c < a.d) a.out_state[so + c0 + c] = a.d_state_out ? a.d_state_out[so + c0 + c] : 0.f;
    }
    if (tile * TILE_T >= len) return;
    // warp 0 takes the tile's last tokens: the warps follow the scan's direction
    const int t0 = tile * TILE_T + (WARPS - 1 - __shfl_sync(0xffffffffu, warp, 0)) * TS;
    const int m = ch < a.d ? min(TS, len - t0) : 0;

    if ((tile + 1) * TILE_T <= len && c0 + C <= a.d)
        bwd_tile<T, GATE, VEC, true>(sh, a, chain, pos, tile, b, c0, t0, m, len);
    else
        bwd_tile<T, GATE, VEC, false>(sh, a, chain, pos, tile, b, c0, t0, m, len);
}

// d_rate[c] = sum of the tiles' partial sums, in an order fixed by the sizes: warp w of a
// channel group takes tiles w, w + 8, ... of sequence 0, 1, ..., then the warps are added.
template <int VEC>
__global__ void __launch_bounds__(kThreads) gated_rate_kernel(const Args a, int tile_t, float *d_rate) {
    constexpr int C = 32 * VEC;
    __shared__ float red[WARPS][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < a.d) {
        for (int b = 0; b < a.B; ++b) {
            const int used = (int)(((long long)length_of(a, b) + tile_t - 1) / tile_t);
            const Record *p = a.part + (((size_t)b * a.slices + c / C) * a.tiles) * C + c % C;
            for (int t = warp; t < used; t += WARPS) s += __ldg(&p[(size_t)t * C].a);
        }
    }
    red[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < a.d) {
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) t += red[w][lane];
        d_rate[c] = t;
    }
}

// ------------------------------------------------------------ one token
template <typename T, int GATE, int VEC>
__global__ void __launch_bounds__(kThreads) gated_step_kernel(const Args a) {
    const size_t cols = (a.d + VEC - 1) / VEC, e = (size_t)blockIdx.x * kThreads + threadIdx.x;
    if (e >= cols * a.B) return;
    const int b = (int)(e / cols), ch = (int)(e % cols) * VEC;
    if (a.lengths && a.lengths[b] <= 0) return;
    Num<T, VEC> x, g, h, ea, eb;
    unpack(load<T, VEC>(a.x, (size_t)b * a.x.sb + ch), x.v);
    unpack(load<T, VEC>(a.g, (size_t)b * a.g.sb + ch), g.v);
    const size_t so = (size_t)b * a.d + ch;
#pragma unroll
    for (int v = 0; v < VEC; ++v) h.v[v] = a.state_in[so + v];
    gate_fwd<GATE>(g, rate_of<GATE, Num<T, VEC>>(a, ch), x, ea, eb);
    h = fma_(ea, h, eb);
#pragma unroll
    for (int v = 0; v < VEC; ++v) a.out_state[so + v] = h.v[v];
    store<T, VEC>(a.o1, (size_t)b * a.o1.sb + ch, h.v);
}

// ------------------------------------------------------------ host
template <int VEC>
int slices_of(int d) { return (d + 32 * VEC - 1) / (32 * VEC); }
int tiles_of(long long n, int tile) { return (int)((n + tile - 1) / tile); }
int most_tiles(const hla_gated_params *p) { return tiles_of(p->n, kTileLeast); }

// Two channels per lane when every row of every tensor starts on a two-channel boundary
// and rows hold a whole number of them: a row segment is then 128 bytes (bf16) per warp
// and load.  One channel per lane otherwise (odd widths or strides, offset pointers).
bool pairable(const hla_tensor *t, const hla_gated_params *p) {
    const size_t el = p->in_dtype == HLA_F32 ? 4 : 2;
    return !t || !t->p || ((reinterpret_cast<uintptr_t>(t->p) % (2 * el)) == 0 && (p->B == 1 || t->sb % 2 == 0) &&
                           (p->n == 1 || t->st % 2 == 0));
}

hla_status check(const hla_gated_params *p) {
    if (!p) return report(HLA_ERR_ARG, "params is NULL");
    if (p->B < 1 || p->d < 1 || p->n < 0) return report(HLA_ERR_ARG, "need B >= 1, d >= 1, n >= 0");
    if (p->in_dtype != HLA_F32 && p->in_dtype != HLA_BF16) return report(HLA_ERR_ARG, "unknown in_dtype");
    if (p->gate != HLA_GATE_GIVEN && p->gate != HLA_GATE_SIGMOID && p->gate != HLA_GATE_RATE)
        return report(HLA_ERR_ARG, "unknown gate");
    if (p->gate == HLA_GATE_RATE && !p->rate) return report(HLA_ERR_ARG, "HLA_GATE_RATE needs rate");
    if (p->n > 2147483647 - 1024) return report(HLA_ERR_ARG, "problem too large");  // token counters pass n by up to two tiles
    const double tiles = most_tiles(p), slices = (double)((p->d + 31LL) / 32);
    if ((double)p->B * (tiles < 1 ? 1 : tiles) * slices > 2147483647.0 || (double)p->B * p->d > 1099511627776.0)
        return report(HLA_ERR_ARG, "problem too large");
    return HLA_OK;
}

// in: null when not used by this gate; n rows of d channels per sequence.
hla_status check_in(const hla_tensor *t, const hla_gated_params *p, const char *what) {
    if (!t || !t->p) return report(HLA_ERR_ARG, what);
    const size_t el = p->in_dtype == HLA_F32 ? 4 : 2;
    if (reinterpret_cast<uintptr_t>(t->p) % el) return report(HLA_ERR_ARG, "a tensor is not aligned to its elements");
    if (t->sb < 0 || t->st < 0) return report(HLA_ERR_ARG, "strides must not be negative");
    if ((double)t->sb * (p->B - 1) + (double)t->st * (p->n > 0 ? p->n - 1 : 0) + p->d > 4e18)
        return report(HLA_ERR_ARG, "a tensor is too large");
    return HLA_OK;
}
// An output's rows must not share memory.
hla_status check_out(const hla_tensor *t, const hla_gated_params *p, const char *what) {
    hla_status s = check_in(t, p, what);
    if (s != HLA_OK) return s;
    const long long n = p->n, B = p->B, d = p->d;
    const bool tokens_inside = (n <= 1 || t->st >= d) && (B <= 1 || t->sb >= (n > 0 ? (n - 1) * t->st : 0) + d);
    const bool seqs_inside = (B <= 1 || t->sb >= d) && (n <= 1 || t->st >= (B - 1) * t->sb + d);
    if (!tokens_inside && !seqs_inside) return report(HLA_ERR_ARG, "rows of an output overlap");
    return HLA_OK;
}

Tensor view(const hla_tensor *t) {
    Tensor r{nullptr, 0, 0};
    if (t) r = Tensor{t->p, t->sb, t->st};
    return r;
}

// Records of a call: the channel slots of all tiles, for the wider of the two layouts.
size_t record_count(const hla_gated_params *p) {
    const size_t tiles = most_tiles(p);
    const size_t s1 = (size_t)slices_of<1>(p->d) * 32, s2 = (size_t)slices_of<2>(p->d) * 64;
    return (size_t)p->B * tiles * (s1 > s2 ? s1 : s2);
}
size_t workspace_bytes_of(const hla_gated_params *p) {
    // one tile per sequence and no rates' gradient needs none, but one size serves every call
    return p->n == 0 ? 0 : kHeaderBytes + 2 * record_count(p) * sizeof(Record);
}

enum Which { W_FWD, W_BWD, W_STEP };

// The forward takes fp32 channels one per lane always: a row is 128 bytes per warp even so, and
// twice the CTAs fit an SM (16,384 x 1,024 fp32 78 -> 52 us; the backward 102 us in pairs, 106 singly).
template <typename T, int VEC>
constexpr bool kFwdTakes = VEC * sizeof(T) <= 4;

template <typename T, int GATE, int VEC>
cudaError_t launch(Which w, Args a, float *d_rate, cudaStream_t st) {
    a.slices = slices_of<VEC>(a.d);
    a.tiles = w == W_BWD ? tiles_of(a.n, kTileT<T, BWD, VEC>) : tiles_of(a.n, kTileT<T, FWD, VEC>);
    if (w == W_STEP) {
        const size_t total = (size_t)a.B * ((a.d + VEC - 1) / VEC);
        gated_step_kernel<T, GATE, VEC><<<(unsigned)((total + kThreads - 1) / kThreads), kThreads, 0, st>>>(a);
        return cudaGetLastError();
    }
    const unsigned grid = (unsigned)((size_t)a.B * a.slices * a.tiles);
    if (a.tiles <= 1) a.hdr = nullptr;  // no tile waits for another
    if constexpr (kFwdTakes<T, VEC>) {
        if (w == W_FWD) {
            gated_fwd_kernel<T, GATE, VEC><<<grid, kThreads, 0, st>>>(a);
            return cudaGetLastError();
        }
    }
    gated_bwd_kernel<T, GATE, VEC><<<grid, kThreads, 0, st>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess && a.part && GATE == HLA_GATE_RATE) {
        gated_rate_kernel<VEC><<<(a.d + 31) / 32, kThreads, 0, st>>>(a, kTileT<T, BWD, VEC>, d_rate);
        e = cudaGetLastError();
    }
    return e;
}
template <typename T, int VEC>
cudaError_t by_gate(int gate, Which w, const Args &a, float *d_rate, cudaStream_t st) {
    if (gate == HLA_GATE_GIVEN) return launch<T, HLA_GATE_GIVEN, VEC>(w, a, d_rate, st);
    if (gate == HLA_GATE_SIGMOID) return launch<T, HLA_GATE_SIGMOID, VEC>(w, a, d_rate, st);
    return launch<T, HLA_GATE_RATE, VEC>(w, a, d_rate, st);
}
hla_status dispatch(const hla_gated_params *p, Which w, Args &a, bool pairs, float *d_rate, cudaStream_t st) {
    a.B = p->B; a.n = p->n; a.d = p->d;
    a.rate = p->rate;
    a.lengths = p->lengths;
    int dev = 0, sms = 0;
    cudaError_t e = dev_status_ptr(&a.err);
    if (e == cudaSuccess) e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) {
        if (w != W_STEP && pairs && stream_takes(a, p->in_dtype, w == W_BWD, sms))
            e = w == W_FWD ? stream_forward(a, p->in_dtype, p->gate, st)
                           : stream_backward(a, p->in_dtype, p->gate, d_rate, st);
        else if (p->in_dtype == HLA_F32)
            e = pairs && (w != W_FWD || kFwdTakes<float, 2>) ? by_gate<float, 2>(p->gate, w, a, d_rate, st) : by_gate<float, 1>(p->gate, w, a, d_rate, st);
        else
            e = pairs ? by_gate<__nv_bfloat16, 2>(p->gate, w, a, d_rate, st)
                      : by_gate<__nv_bfloat16, 1>(p->gate, w, a, d_rate, st);
    }
    if (e != cudaSuccess) return report(HLA_ERR_CUDA, cudaGetErrorString(e));
    return HLA_OK;
}

// Splits the caller's workspace; the header is needed from two tiles on.
hla_status take_workspace(const hla_gated_params *p, void *ws, size_t bytes, bool partials, Args &a) {
    const size_t need = workspace_bytes_of(p);
    if (!ws && most_tiles(p) <= 1 && !partials) return HLA_OK;
    if (!ws || bytes < need) return report(HLA_ERR_ARG, "workspace too small (hla_gated_workspace_size)");
    if (reinterpret_cast<uintptr_t>(ws) & 255u) return report(HLA_ERR_ARG, "workspace must be 256-byte aligned");
    a.hdr = static_cast<Header *>(ws);
    a.rec = reinterpret_cast<Record *>(static_cast<uint8_t *>(ws) + kHeaderBytes);
    if (partials) a.part = a.rec + record_count(p);
    return HLA_OK;
}

bool even_state(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace
}  // namespace gated
}  // namespace hla

using namespace hla;
using namespace hla::gated;

extern "C" {

size_t hla_gated_workspace_size(const hla_gated_params *p) {
    if (check(p) != HLA_OK) return 0;
    return workspace_bytes_of(p);
}

hla_status hla_gated_forward(const hla_gated_params *p, const hla_tensor *x, const hla_tensor *g, const hla_tensor *y,
                             const float *state_in, float *state_out, void *workspace, size_t workspace_bytes,
                             void *stream) {
    hla_status s = check(p);
    if (s != HLA_OK) return s;
    if (!even_state(state_in) || !even_state(state_out)) return report(HLA_ERR_ARG, "a state is not aligned to its elements");
    if (state_in && state_in == state_out) return report(HLA_ERR_ARG, "state_out may not alias state_in");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (p->n == 0) {
        if (!state_out) return HLA_OK;
        const size_t bytes = (size_t)p->B * p->d * 4;
        const cudaError_t e = state_in ? cudaMemcpyAsync(state_out, state_in, bytes, cudaMemcpyDeviceToDevice, st)
                                       : cudaMemsetAsync(state_out, 0, bytes, st);
        return e == cudaSuccess ? HLA_OK : report(HLA_ERR_CUDA, cudaGetErrorString(e));
    }
    if ((s = check_in(x, p, "x must be set")) != HLA_OK || (s = check_in(g, p, "g must be set")) != HLA_OK ||
        (s = check_out(y, p, "y must be set")) != HLA_OK)
        return s;
    if (y->p == x->p || y->p == g->p) return report(HLA_ERR_ARG, "y may not be x or g");
    Args a{};
    if ((s = take_workspace(p, workspace, workspace_bytes, false, a)) != HLA_OK) return s;
    a.x = view(x); a.g = view(g); a.o1 = view(y);
    a.state_in = state_in;
    a.out_state = state_out;
    return dispatch(p, W_FWD, a, p->d % 2 == 0 && pairable(x, p) && pairable(g, p) && pairable(y, p), nullptr, st);
}

hla_status hla_gated_backward(const hla_gated_params *p, const hla_tensor *x, const hla_tensor *g, const hla_tensor *y,
                              const hla_tensor *dy, const float *state_in, const float *d_state_out,
                              const hla_tensor *dx, const hla_tensor *dg, float *d_rate, float *d_state_in,
                              void *workspace, size_t workspace_bytes, void *stream) {
    hla_status s = check(p);
    if (s != HLA_OK) return s;
    if (!even_state(state_in) || !even_state(d_state_out) || !even_state(d_state_in) || !even_state(d_rate))
        return report(HLA_ERR_ARG, "a state is not aligned to its elements");
    if (d_state_out && d_state_out == d_state_in) return report(HLA_ERR_ARG, "d_state_in may not alias d_state_out");
    if (d_rate && p->gate != HLA_GATE_RATE) return report(HLA_ERR_ARG, "d_rate belongs to HLA_GATE_RATE");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (p->n == 0) {
        cudaError_t e = cudaSuccess;
        const size_t bytes = (size_t)p->B * p->d * 4;
        if (d_rate) e = cudaMemsetAsync(d_rate, 0, (size_t)p->d * 4, st);
        if (e == cudaSuccess && d_state_in)
            e = d_state_out ? cudaMemcpyAsync(d_state_in, d_state_out, bytes, cudaMemcpyDeviceToDevice, st)
                            : cudaMemsetAsync(d_state_in, 0, bytes, st);
        return e == cudaSuccess ? HLA_OK : report(HLA_ERR_CUDA, cudaGetErrorString(e));
    }
    const bool given = p->gate == HLA_GATE_GIVEN;
    if ((!given && (s = check_in(x, p, "x must be set")) != HLA_OK) || (s = check_in(g, p, "g must be set")) != HLA_OK ||
        (s = check_in(y, p, "y must be set")) != HLA_OK || (s = check_in(dy, p, "dy must be set")) != HLA_OK ||
        (s = check_out(dx, p, "dx must be set")) != HLA_OK || (s = check_out(dg, p, "dg must be set")) != HLA_OK)
        return s;
    const hla_tensor *ins[4] = {given ? nullptr : x, g, y, dy};
    for (const hla_tensor *i : ins)
        if (i && (dx->p == i->p || dg->p == i->p)) return report(HLA_ERR_ARG, "dx and dg may not be inputs");
    if (dx->p == dg->p) return report(HLA_ERR_ARG, "dx may not be dg");
    Args a{};
    if ((s = take_workspace(p, workspace, workspace_bytes, d_rate != nullptr, a)) != HLA_OK) return s;
    a.x = given ? Tensor{nullptr, 0, 0} : view(x);
    a.g = view(g); a.y = view(y); a.dy = view(dy); a.o1 = view(dx); a.o2 = view(dg);
    a.state_in = state_in;
    a.d_state_out = d_state_out;
    a.out_state = d_state_in;
    bool pairs = p->d % 2 == 0 && pairable(dx, p) && pairable(dg, p);
    for (const hla_tensor *i : ins) pairs = pairs && pairable(i, p);
    return dispatch(p, W_BWD, a, pairs, d_rate, st);
}

hla_status hla_gated_step(const hla_gated_params *p, const hla_tensor *x, const hla_tensor *g, const hla_tensor *y,
                          const float *state, float *state_out, void *stream) {
    hla_status s = check(p);
    if (s != HLA_OK) return s;
    if (p->n != 1) return report(HLA_ERR_ARG, "a step takes one token: n must be 1");
    if (!state || !state_out) return report(HLA_ERR_ARG, "state and state_out must be set");
    if (!even_state(state) || !even_state(state_out)) return report(HLA_ERR_ARG, "a state is not aligned to its elements");
    if ((s = check_in(x, p, "x must be set")) != HLA_OK || (s = check_in(g, p, "g must be set")) != HLA_OK ||
        (s = check_out(y, p, "y must be set")) != HLA_OK)
        return s;
    if (y->p == x->p || y->p == g->p) return report(HLA_ERR_ARG, "y may not be x or g");
    Args a{};
    a.x = view(x); a.g = view(g); a.o1 = view(y);
    a.state_in = state;
    a.out_state = state_out;
    return dispatch(p, W_STEP, a, p->d % 2 == 0 && pairable(x, p) && pairable(g, p) && pairable(y, p), nullptr,
                    static_cast<cudaStream_t>(stream));
}

}  // extern "C"
