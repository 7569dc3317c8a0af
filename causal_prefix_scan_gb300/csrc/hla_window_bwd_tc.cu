// hla_window_bwd_tc.cu -- backward of windowed attention for bf16 on the tensor cores.
//
// With P = exp(scale S - lse), S = Q K^T, dP = dO V^T, D = rowsum(dO o):
//   dS = P (dP - D),   dQ = scale dS K,   dK = scale dS^T Q,   dV = P^T dO.
// Two kernels, neither of which adds to memory that another CTA adds to, so every sum has a
// fixed order: dq over tiles of 128 queries (walking the keys they see; also forms D) and dkv
// over tiles of 128 keys (walking the queries that see them, all heads of the group).  S and
// dP are formed in both: 7 products per pair of tiles instead of 5, in exchange for no
// atomics and no fp32 buffer of dQ the size of Q.
//
// Roles (10 warps): 0-3 and 4-7 the elementwise part, one row per thread, columns [0,64) and
// [64,128) of each tile; 8 MMA; 9 TMA.  The MMA order is chosen so that the tensor cores
// always have the next product while the elementwise part works on the one before:
//   dq:   S(j+1) | dQ(j) | dP(j+1)            dkv:  dV(j) | S(j+1) | dK(j) | dP(j+1)
// P and dS are rounded to bf16 (half a step 2^-8 of each) and stay in TMEM over the columns
// of S and dP that they were made from, as the first operand of the next product; sums are
// fp32.  The scale is applied to the finished sums.
//
// Measured: B2 H16 Hkv4 n8192 d128 w1024 508 us (dq 223, dkv 283, join 5), 640 TFLOP/s counted
// with 5 products, 900 with the 7 that run; B3 H6 Hkv2 n1501 d64 w301 45 us (13.5, 27.5, 4).  Bound
// by the chain S -> P -> dS -> product of one tile pair per CTA: TMEM's 512 columns hold one.
#include "hla_window_tc.cuh"

namespace hla {
namespace win {
namespace {

using namespace tcw;

constexpr int kThreads = 320, kWarpMma = 8, kWarpTma = 9;
constexpr float kLog2e = 1.4426950408889634f;

struct Params {
    Args a;
    CUtensorMap mq, mk, mv, mg, mo;
};

HLA_DEVICE void elem_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// D (+)= A B over the 128 rows of B: A in TMEM as two blocks of 64 contraction rows (32 packed
// columns each) 64 columns apart.
HLA_DEVICE void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
    mma_ts32(d, a, b, idesc, acc);
    mma_ts32(d, a + 16, b + 256, idesc, true);
    mma_ts32(d, a + 64, b + 512, idesc, true);
    mma_ts32(d, a + 80, b + 768, idesc, true);
}

// Common set-up and end of both kernels.
template <int NB>
struct Cta {
    uint8_t *base;
    Waits ws;
    uint32_t tb;
    int warp;
    HLA_DEVICE Cta(uint8_t *b, int off_bar, unsigned *err, int eight_a, int eight_b, int eight_c) : base(b) {
        ws.bars = reinterpret_cast<uint64_t *>(b + off_bar);
        uint32_t *misc = reinterpret_cast<uint32_t *>(b + off_bar + NB * 8);
        ws.abort_p = reinterpret_cast<volatile int *>(misc + 1);
        ws.err = err;
        warp = threadIdx.x >> 5;
        if (threadIdx.x == 0) {
            misc[1] = 0u;
            for (int i = 0; i < NB; ++i) mbar_init(ws.bar(i), i == eight_a || i == eight_b || i == eight_c ? 8 : 1);
            fence_mbar_init();
        }
        if (warp == kWarpMma) {
            tmem_alloc(misc, 512);
            tmem_relinquish();
        }
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        tb = misc[0];
    }
    HLA_DEVICE void finish() {
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (warp == kWarpMma) tmem_dealloc(tb, 512);
    }
};

// ------------------------------------------------------------ dq
template <int DP>
struct LayQ {
    static constexpr int TILE = T * DP * 2;
    static constexpr int NS = DP == 64 ? 8 : 4;  // ring slots, K and V tiles in turn
    static constexpr int OFF_Q = 0, OFF_G = TILE, OFF_O = 2 * TILE, OFF_RING = 3 * TILE, OFF_BAR = OFF_RING + NS * TILE;
    static_assert(3 * TILE >= 8 * 4096, "the results leave through the inputs' tiles");
    static constexpr int B_Q = 0, B_GO = 1, B_FULL = 2, B_EMPTY = B_FULL + NS, B_S = B_EMPTY + NS, B_SF = B_S + 1, B_DP = B_SF + 1,
                         B_DS = B_DP + 1, B_O = B_DS + 1, B_FIN = B_O + 1, B_RAW = B_FIN + 1, NB = B_RAW + 1;
    static constexpr int SMEM = OFF_BAR + NB * 8 + 16;
    static constexpr uint32_t S = 0, DPC = T, DQ = 2 * T;  // TMEM columns
};

template <int DP>
__device__ __forceinline__ void dq_elem(const Params &p, const Waits &ws, uint8_t *base, uint32_t tb, const KeyTiles &kt,
                                        int b, int h, int i0, int rows) {
    using L = LayQ<DP>;
    const Args &a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, half = warp >> 2;
    const int r = i0 + (warp & 3) * 32 + lane, pos = a.p0 + r;
    const bool live = r < rows;
    const uint32_t quad = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t sa = tb + quad + L::S + half * 64, da = tb + quad + L::DPC + half * 64;
    const size_t row = ((size_t)b * a.H + h) * a.n + r;
    const float c = a.scale * kLog2e, lse = live ? a.lse[row] * kLog2e : 0.f;
    // D = rowsum(dO o) of the thread's row, also for the dkv kernel
    if (!ws.wait(L::B_GO, 0u)) return;
    float D = 0.f;
    for (int k = 0; k < ((a.dv + 7) & ~7); k += 8) {
        float x[8], y[8];
        tile_load_row8(base + L::OFF_G, T, (warp & 3) * 32 + lane, k, x);
        tile_load_row8(base + L::OFF_O, T, (warp & 3) * 32 + lane, k, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) D = fmaf(x[e], y[e], D);
    }
    if (live && half == 0) a.delta[row] = D;
    bool ok = true;
    uint32_t ph = 0;
    for (int it = 0; it < kt.total; ++it, ph ^= 1u) {
        const int j0 = kt[it] * T;
        const bool masked = !(j0 + T - 1 <= a.p0 + i0 && (a.p0 + i0 + T - 1 - j0 < a.window || j0 + T <= a.sinks));
        const int hi = pos - j0 + 1 - half * 64, sk = a.sinks - j0 - half * 64;
        const int lo = (pos >= a.window ? pos - a.window + 1 - j0 : 0) - half * 64;
        const uint32_t bits[2] = {visible_bits(0, lo, hi, sk), visible_bits(32, lo, hi, sk)};
        if (!(ok = ws.wait(L::B_S, ph))) break;
        tc_fence_after();
        float P[2][32];
        tmem_ld32(sa, P[0]);
        tmem_ld32(sa + 32, P[1]);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(ws.bar(L::B_SF));
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int e = 0; e < 32; ++e) P[k][e] = ex2_approx(fmaf(P[k][e], c, -lse));
        if (masked) {
#pragma unroll
            for (int k = 0; k < 2; ++k) mask32(P[k], bits[k], 0.f);
        }
        if (!(ok = ws.wait(L::B_DP, ph))) break;
        tc_fence_after();
        float v[2][32];
        tmem_ld32(da, v[0]);
        tmem_ld32(da + 32, v[1]);
        tmem_wait_ld();
        if (masked) {  // behind the sequence dP may be anything
#pragma unroll
            for (int k = 0; k < 2; ++k) mask32(v[k], bits[k], 0.f);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                pk[e] = __uint_as_float(pack_bf16(P[k][2 * e] * (v[k][2 * e] - D), P[k][2 * e + 1] * (v[k][2 * e + 1] - D)));
            }
            tmem_st16(da + 16 * k, pk);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(ws.bar(L::B_DS));
    }
    if (!ok || !ws.wait(L::B_O, 0u)) return;
    tc_fence_after();
    const int r0 = i0 + (warp & 3) * 32;  // every product is done: the inputs' tiles are free
    __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.dq.p) + (size_t)b * a.dq.sb + (size_t)h * a.dq.sh + (size_t)r0 * a.dq.st;
    store_rows<DP / 2>(base + warp * 4096, tb + quad + L::DQ + DP / 2 * half, a.scale, o, a.dq.st, rows - r0, DP / 2 * half, a.d);
}

template <int DP>
__device__ __forceinline__ void dq_mma(const Params &p, const Waits &ws, uint8_t *base, uint32_t tb, int N) {
    using L = LayQ<DP>;
    const Args &a = p.a;
    const uint32_t id_s = make_idesc(T, T, false, false), id_q = make_idesc(T, (a.d + 15) & ~15, false, true);
    const bool qk = a.d > 64, gv = a.dv > 64;
    const uint64_t q = kmajor(base + L::OFF_Q), g = kmajor(base + L::OFF_G), ring_k = kmajor(base + L::OFF_RING),
                   ring_m = mnmajor(base + L::OFF_RING);
    constexpr uint32_t STEP = L::TILE >> 4;
    Ring<L::NS> ring;  // the next tile: keys and values in turn
    uint32_t k_slot = 0;
    auto do_s = [&]() {
        if (!ws.wait(L::B_FULL + ring.slot, ring.phase)) return false;
        k_slot = ring.slot;
        mma_kk<DP>(tb + L::S, q, ring_k + ring.slot * STEP, id_s, qk);
        umma_commit_warp(ws.bar(L::B_S));
        ring.next();
        return true;
    };
    auto do_dp = [&]() {
        if (!ws.wait(L::B_FULL + ring.slot, ring.phase)) return false;
        mma_kk<DP>(tb + L::DPC, g, ring_k + ring.slot * STEP, id_s, gv);
        umma_commit_warp(ws.bar(L::B_DP));
        umma_commit_warp(ws.bar(L::B_EMPTY + ring.slot));
        ring.next();
        return true;
    };
    bool ok = ws.wait(L::B_Q, 0u) && do_s() && ws.wait(L::B_GO, 0u) && do_dp();
    for (int j = 0; j < N && ok; ++j) {
        const uint32_t ph = (uint32_t)j & 1u, slot = k_slot;
        if (j + 1 < N) {
            if (!(ok = ws.wait(L::B_SF, ph))) break;
            tc_fence_after();
            if (!(ok = do_s())) break;
        }
        if (!(ok = ws.wait(L::B_DS, ph))) break;
        tc_fence_after();
        mma_ts(tb + L::DQ, tb + L::DPC, ring_m + slot * STEP, id_q, j > 0);
        umma_commit_warp(ws.bar(L::B_EMPTY + slot));
        if (j + 1 < N) ok = do_dp();
    }
    if (ok) umma_commit_warp(ws.bar(L::B_O));
    umma_commit_warp(ws.bar(L::B_FIN));  // every MMA issued completes before TMEM is released
    mbar_wait(ws.bar(L::B_FIN), 0u, ws.err);
    __syncwarp();
}

template <int DP>
__device__ __forceinline__ void dq_tma(const Params &p, const Waits &ws, uint8_t *base, const KeyTiles &kt, int b, int h,
                                       int i0, int len) {
    using L = LayQ<DP>;
    const Args &a = p.a;
    const int lane = threadIdx.x & 31, hk = h / a.G;
    if (lane == 0) {
        mbar_expect_tx(ws.bar(L::B_Q), L::TILE);
        load_tile<DP>(base + L::OFF_Q, &p.mq, a.q, ws.bar(L::B_Q), i0, h, b);
        mbar_expect_tx(ws.bar(L::B_GO), 2 * L::TILE);
        load_tile<DP>(base + L::OFF_G, &p.mg, a.go, ws.bar(L::B_GO), i0, h, b);
        load_tile<DP>(base + L::OFF_O, &p.mo, a.o, ws.bar(L::B_GO), i0, h, b);
    }
    Ring<L::NS> ring;
    uint32_t raw = 0;
    int idx = 0;
    for (; idx < 2 * kt.total; ++idx) {
        const uint32_t s = ring.slot;
        if (idx >= L::NS && !ws.wait(L::B_EMPTY + s, ring.phase ^ 1u)) break;
        const bool key = (idx & 1) == 0;
        const int j0 = kt[idx >> 1] * T;
        const bool clean = key && len - j0 < T;  // dS K contracts over the keys: zeros behind the sequence
        const int full = clean ? L::B_RAW : L::B_FULL + (int)s;
        if (lane == 0) {
            mbar_expect_tx(ws.bar(full), L::TILE);
            load_tile<DP>(base + L::OFF_RING + s * L::TILE, key ? &p.mk : &p.mv, key ? a.k : a.v, ws.bar(full), j0, hk, b);
        }
        __syncwarp();
        if (clean) {
            if (!ws.wait(L::B_RAW, raw)) break;
            raw ^= 1u;
            zero_rows<DP>(base + L::OFF_RING + s * L::TILE, len - j0, lane);
            if (lane == 0) mbar_arrive(ws.bar(L::B_FULL + s));
        }
        ring.next();
    }
    // nothing may land after the CTA has ended (only an aborted CTA still has copies in flight)
    mbar_wait(ws.bar(L::B_Q), 0u, ws.err);
    mbar_wait(ws.bar(L::B_GO), 0u, ws.err);
    for (int k = max(0, idx - L::NS); k < idx; ++k)
        mbar_wait(ws.bar(L::B_FULL + k % L::NS), (uint32_t)(k / L::NS) & 1u, ws.err);
    __syncwarp();
}

template <int DP>
__global__ void __launch_bounds__(kThreads, 1) window_dq_kernel(const __grid_constant__ Params p) {
    using L = LayQ<DP>;
    extern __shared__ __align__(1024) uint8_t base[];
    const Args &a = p.a;
    const int tiles = (a.n + T - 1) / T, u = blockIdx.x % (a.B * a.H), h = u % a.H, b = u / a.H;
    const int i0 = (tiles - 1 - (int)(blockIdx.x / (a.B * a.H))) * T;  // long rows first
    const int len = length_of(a, b), rows = min(a.n, len - a.p0);
    if (i0 >= rows) return;
    const KeyTiles kt(a, a.p0 + i0, a.p0 + min(i0 + T, rows) - 1, T);
    Cta<L::NB> c(base, L::OFF_BAR, a.err, L::B_SF, L::B_DS, -1);
    if (c.warp == kWarpTma) {
        dq_tma<DP>(p, c.ws, base, kt, b, h, i0, len);
    } else if (c.warp == kWarpMma) {
        dq_mma<DP>(p, c.ws, base, uniform(c.tb), (int)uniform(kt.total));
    } else {
        dq_elem<DP>(p, c.ws, base, c.tb, kt, b, h, i0, rows);
    }
    c.finish();
}

// ------------------------------------------------------------ dk, dv
template <int DP>
struct LayK {
    static constexpr int TILE = T * DP * 2;
    static constexpr int NS = DP == 64 ? 4 : 2;  // stages of one Q and one dO tile
    static constexpr int OFF_K = 0, OFF_V = TILE, OFF_RING = 2 * TILE, OFF_ROW = OFF_RING + 2 * NS * TILE;
    static constexpr int OFF_BAR = OFF_ROW + 2 * 2 * T * 4;  // lse and D of the queries, two stages
    static constexpr int B_K = 0, B_FQ = 1, B_FG = B_FQ + NS, B_EMPTY = B_FG + NS, B_S = B_EMPTY + NS, B_P = B_S + 1,
                         B_DP = B_P + 1, B_DS = B_DP + 1, B_O = B_DS + 1, B_FIN = B_O + 1, B_RAW = B_FIN + 1, NB = B_RAW + 1;
    static constexpr int SMEM = OFF_BAR + NB * 8 + 16;
    static constexpr uint32_t S = 0, DPC = T, DV = 2 * T, DK = 2 * T + DP;  // TMEM columns
};

// The (head, query tile) pairs of one key tile: query tiles [q_lo, q_lo + each) of every head.
struct Walk {
    int q_lo, each, total;
    HLA_DEVICE int head(int i) const { return i / each; }
    HLA_DEVICE int tile(int i) const { return q_lo + i % each; }
};

template <int DP>
__device__ __forceinline__ void dkv_elem(const Params &p, const Waits &ws, uint8_t *smem, uint32_t tb, const Walk &w, int b,
                                         int hk, int j0, int len, int rows, int share, bool split) {
    using L = LayK<DP>;
    const Args &a = p.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, half = warp >> 2;
    const int j = j0 + (warp & 3) * 32 + lane;
    const uint32_t quad = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t sa = tb + quad + L::S + half * 64, da = tb + quad + L::DPC + half * 64;
    float *rowv = reinterpret_cast<float *>(smem + L::OFF_ROW);  // [2 stages][-lse * log2e, -D][128]
    const float c = a.scale * kLog2e;
    bool ok = true;
    uint32_t ph = 0;
    auto fetch = [&](int it) {  // threads 0-127 lse, 128-255 D
        const int r = w.tile(it) * T + (tid & 127);
        const size_t at = ((size_t)b * a.H + hk * a.G + w.head(it)) * a.n + r;
        return r < rows ? (tid < 128 ? a.lse[at] * -kLog2e : -a.delta[at]) : 0.f;
    };
    float next = w.total > 0 ? fetch(0) : 0.f;
    for (int it = 0; it < w.total; ++it, ph ^= 1u) {
        float *cur = rowv + (it & 1) * 2 * T;
        cur[tid] = next;
        elem_sync();
        if (it + 1 < w.total) next = fetch(it + 1);
        const int i0 = w.tile(it) * T, p_lo = a.p0 + i0;
        const bool masked = !(j0 + T - 1 <= p_lo && (p_lo + T - 1 - j0 < a.window || j0 + T <= a.sinks) && i0 + T <= rows);
        // visible queries of key j: columns [lo, hi)
        const int lo = j - p_lo - half * 64;
        const int hi = (j < a.sinks ? rows - i0 : (int)min((long long)rows - i0, (long long)j - p_lo + a.window)) - half * 64;
        const uint32_t bits[2] = {visible_bits(0, lo, hi, 0), visible_bits(32, lo, hi, 0)};
        // after an expired wait the loop goes on, so that the barrier above stays matched
        if (!ok || !(ok = ws.wait(L::B_S, ph))) continue;
        tc_fence_after();
        float P[2][32];
        tmem_ld32(sa, P[0]);
        tmem_ld32(sa + 32, P[1]);
        tmem_wait_ld();
        const float *lse = cur + half * 64, *D = cur + T + half * 64;  // both negated
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
                const float4 x = *reinterpret_cast<const float4 *>(lse + 32 * k + e);
                P[k][e] = ex2_approx(fmaf(P[k][e], c, x.x));
                P[k][e + 1] = ex2_approx(fmaf(P[k][e + 1], c, x.y));
                P[k][e + 2] = ex2_approx(fmaf(P[k][e + 2], c, x.z));
                P[k][e + 3] = ex2_approx(fmaf(P[k][e + 3], c, x.w));
            }
        if (masked) {
#pragma unroll
            for (int k = 0; k < 2; ++k) mask32(P[k], bits[k], 0.f);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) pk[e] = __uint_as_float(pack_bf16(P[k][2 * e], P[k][2 * e + 1]));
            tmem_st16(sa + 16 * k, pk);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(ws.bar(L::B_P));
        if (!(ok = ws.wait(L::B_DP, ph))) continue;
        tc_fence_after();
        float v[2][32];
        tmem_ld32(da, v[0]);
        tmem_ld32(da + 32, v[1]);
        tmem_wait_ld();
        if (masked) {  // queries behind the sequence: nothing, whatever dP is
#pragma unroll
            for (int k = 0; k < 2; ++k) mask32(v[k], bits[k], 0.f);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float pk[16];
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
                const float4 x = *reinterpret_cast<const float4 *>(D + 32 * k + 2 * e);
                pk[e] = __uint_as_float(pack_bf16(P[k][2 * e] * (v[k][2 * e] + x.x), P[k][2 * e + 1] * (v[k][2 * e + 1] + x.y)));
                pk[e + 1] = __uint_as_float(
                    pack_bf16(P[k][2 * e + 2] * (v[k][2 * e + 2] + x.z), P[k][2 * e + 3] * (v[k][2 * e + 3] + x.w)));
            }
            tmem_st16(da + 16 * k, pk);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(ws.bar(L::B_DS));
    }
    if (!ok) return;
    if (w.total > 0) {
        if (!ws.wait(L::B_O, 0u)) return;
        tc_fence_after();
    }
    // threads 0-127 dv, 128-255 dk of one key each
    const bool key = half == 1;
    const int width = key ? a.d : a.dv;
    const float f = key ? a.scale : 1.f;
    const View &out = key ? a.dk : a.dv_;
    const bool live = j < len;
    const uint32_t acc = tb + quad + (key ? L::DK : L::DV);
    if (split) {
        float *part = a.part + (((size_t)share * a.B * a.Hkv + (size_t)b * a.Hkv + hk) * a.far_keys + j) * (a.d + a.dv) + (key ? 0 : a.d);
        for (int k = 0; k < ((width + 15) & ~15); k += 16) {
            float x[16];
            tmem_ld16(acc + k, x);
            tmem_wait_ld();
            if (live) {
#pragma unroll
                for (int e = 0; e < 16; e += 4)
                    if (k + e < width)
                        *reinterpret_cast<float4 *>(part + k + e) =
                            w.total > 0 ? make_float4(x[e] * f, x[e + 1] * f, x[e + 2] * f, x[e + 3] * f) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            __syncwarp();
        }
        return;
    }
    const int r0 = j0 + (warp & 3) * 32;
    __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(out.p) + (size_t)b * out.sb + (size_t)hk * out.sh + (size_t)r0 * out.st;
    if (w.total > 0) {  // every product is done: the keys' and values' tiles are free
        for (int c0 = 0; c0 < width; c0 += 64) store_rows<64>(smem + warp * 4096, acc + c0, f, o, out.st, len - r0, c0, width);
    } else {  // no query sees these keys
        for (int e = lane; e < 32 * (width / 8); e += 32) {
            const int row = e / (width / 8), col = e % (width / 8) * 8;
            if (r0 + row < len) *reinterpret_cast<uint4 *>(o + (size_t)row * out.st + col) = make_uint4(0, 0, 0, 0);
        }
    }
}

template <int DP>
__device__ __forceinline__ void dkv_mma(const Params &p, const Waits &ws, uint8_t *base, uint32_t tb, int N) {
    using L = LayK<DP>;
    const Args &a = p.a;
    const uint32_t id_s = make_idesc(T, T, false, false);
    const uint32_t id_v = make_idesc(T, (a.dv + 15) & ~15, false, true), id_k = make_idesc(T, (a.d + 15) & ~15, false, true);
    const bool qk = a.d > 64, gv = a.dv > 64;
    const uint64_t kd = kmajor(base + L::OFF_K), vd = kmajor(base + L::OFF_V), ring_k = kmajor(base + L::OFF_RING),
                   ring_m = mnmajor(base + L::OFF_RING);
    constexpr uint32_t STEP = L::TILE >> 4;  // a stage is Q and dO: two steps
    Ring<L::NS> qs, gs;  // the stage that Q and dO are next taken from
    auto do_s = [&]() {
        if (!ws.wait(L::B_FQ + qs.slot, qs.phase)) return false;
        mma_kk<DP>(tb + L::S, kd, ring_k + 2 * qs.slot * STEP, id_s, qk);
        umma_commit_warp(ws.bar(L::B_S));
        qs.next();
        return true;
    };
    auto do_dp = [&]() {
        if (!ws.wait(L::B_FG + gs.slot, gs.phase)) return false;
        mma_kk<DP>(tb + L::DPC, vd, ring_k + (2 * gs.slot + 1) * STEP, id_s, gv);
        umma_commit_warp(ws.bar(L::B_DP));
        gs.next();
        return true;
    };
    bool ok = N == 0 || (ws.wait(L::B_K, 0u) && do_s() && do_dp());
    uint32_t stage = 0;
    for (int i = 0; i < N && ok; ++i) {
        const uint32_t ph = (uint32_t)i & 1u;
        if (!(ok = ws.wait(L::B_P, ph))) break;
        tc_fence_after();
        mma_ts(tb + L::DV, tb + L::S, ring_m + (2 * stage + 1) * STEP, id_v, i > 0);
        if (i + 1 < N && !(ok = do_s())) break;
        if (!(ok = ws.wait(L::B_DS, ph))) break;
        tc_fence_after();
        mma_ts(tb + L::DK, tb + L::DPC, ring_m + 2 * stage * STEP, id_k, i > 0);
        umma_commit_warp(ws.bar(L::B_EMPTY + stage));
        if (i + 1 < N) ok = do_dp();
        stage = stage + 1 == L::NS ? 0 : stage + 1;
    }
    if (ok) umma_commit_warp(ws.bar(L::B_O));
    umma_commit_warp(ws.bar(L::B_FIN));
    mbar_wait(ws.bar(L::B_FIN), 0u, ws.err);
    __syncwarp();
}

template <int DP>
__device__ __forceinline__ void dkv_tma(const Params &p, const Waits &ws, uint8_t *base, const Walk &w, int b, int hk, int j0,
                                        int rows) {
    using L = LayK<DP>;
    const Args &a = p.a;
    const int lane = threadIdx.x & 31;
    if (w.total == 0) return;
    if (lane == 0) {
        mbar_expect_tx(ws.bar(L::B_K), 2 * L::TILE);
        load_tile<DP>(base + L::OFF_K, &p.mk, a.k, ws.bar(L::B_K), j0, hk, b);
        load_tile<DP>(base + L::OFF_V, &p.mv, a.v, ws.bar(L::B_K), j0, hk, b);
    }
    Ring<L::NS> ring;
    uint32_t raw = 0;
    int i = 0;
    for (; i < w.total; ++i) {
        const uint32_t s = ring.slot;
        const int h = hk * a.G + w.head(i), i0 = w.tile(i) * T;
        if (i >= L::NS && !ws.wait(L::B_EMPTY + s, ring.phase ^ 1u)) break;
        uint8_t *d = base + L::OFF_RING + s * 2 * L::TILE;
        const bool clean = rows - i0 < T;  // dS^T Q and P^T dO contract over the queries: zeros behind the sequence
        const int fq = clean ? L::B_RAW : L::B_FQ + (int)s, fg = clean ? L::B_RAW : L::B_FG + (int)s;
        if (lane == 0) {
            if (clean) {
                mbar_expect_tx(ws.bar(L::B_RAW), 2 * L::TILE);
            } else {
                mbar_expect_tx(ws.bar(fq), L::TILE);
                mbar_expect_tx(ws.bar(fg), L::TILE);
            }
            load_tile<DP>(d, &p.mq, a.q, ws.bar(fq), i0, h, b);
            load_tile<DP>(d + L::TILE, &p.mg, a.go, ws.bar(fg), i0, h, b);
        }
        __syncwarp();
        if (clean) {
            if (!ws.wait(L::B_RAW, raw)) break;
            raw ^= 1u;
            zero_rows<DP>(d, rows - i0, lane);
            zero_rows<DP>(d + L::TILE, rows - i0, lane);
            if (lane == 0) {
                mbar_arrive(ws.bar(L::B_FQ + s));
                mbar_arrive(ws.bar(L::B_FG + s));
            }
        }
        ring.next();
    }
    mbar_wait(ws.bar(L::B_K), 0u, ws.err);
    for (int k = max(0, i - L::NS); k < i; ++k) {
        mbar_wait(ws.bar(L::B_FQ + k % L::NS), (uint32_t)(k / L::NS) & 1u, ws.err);
        mbar_wait(ws.bar(L::B_FG + k % L::NS), (uint32_t)(k / L::NS) & 1u, ws.err);
    }
    __syncwarp();
}

template <int DP>
__global__ void __launch_bounds__(kThreads, 1) window_dkv_kernel(const __grid_constant__ Params p) {
    using L = LayK<DP>;
    extern __shared__ __align__(1024) uint8_t base[];
    const Args &a = p.a;
    const int share = blockIdx.y, pairs = a.B * a.Hkv, bk = blockIdx.x % pairs, hk = bk % a.Hkv, b = bk / a.Hkv;
    const int j0 = (int)(blockIdx.x / pairs) * T;
    const int len = length_of(a, b), rows = max(min(a.n, len - a.p0), 0);
    const bool first = j0 < a.far_keys;  // holds first tokens whose sums are split
    if ((share > 0 && !first) || j0 >= len) return;
    // query tiles of the window, then the far ones (see the CUDA-core kernel)
    const int r_lo = max(0, j0 - a.p0), r_win = (int)max(0LL, min((long long)rows, (long long)j0 + T - 1 + a.window - a.p0));
    const int q_mid = max((r_win + T - 1) / T, r_lo / T);
    int q_lo = r_lo / T, q_hi = q_mid;
    const int end = (rows + T - 1) / T;
    if (share > 0) {
        const int all = max(end - q_mid, 0), each = (all + a.far - 1) / a.far;
        q_lo = min(q_mid + (share - 1) * each, end);
        q_hi = min(q_lo + each, end);
    }
    q_hi = min(q_hi, end);
    Walk w;
    w.q_lo = q_lo;
    w.each = max(q_hi - q_lo, 0);
    w.total = w.each * a.G;
    Cta<L::NB> c(base, L::OFF_BAR, a.err, L::B_P, L::B_DS, -1);
    if (c.warp == kWarpTma) {
        dkv_tma<DP>(p, c.ws, base, w, b, hk, j0, rows);
    } else if (c.warp == kWarpMma) {
        dkv_mma<DP>(p, c.ws, base, uniform(c.tb), (int)uniform(w.total));
    } else {
        dkv_elem<DP>(p, c.ws, base, c.tb, w, b, hk, j0, len, rows, share, first && a.far > 0);
    }
    c.finish();
}

template <int DP>
cudaError_t launch(Params &p, cudaStream_t st) {
    using Q = LayQ<DP>;
    using K = LayK<DP>;
    static_assert(Q::SMEM <= 227 * 1024 && K::SMEM <= 227 * 1024, "shared memory");
    const Args &a = p.a;
    if (!encode(&p.mq, a.q, a.d, a.n, a.H, a.B, T) || !encode(&p.mk, a.k, a.d, a.nk, a.Hkv, a.B, T) ||
        !encode(&p.mv, a.v, a.dv, a.nk, a.Hkv, a.B, T) || !encode(&p.mg, a.go, a.dv, a.n, a.H, a.B, T) ||
        !encode(&p.mo, a.o, a.dv, a.n, a.H, a.B, T))
        return cudaErrorNotSupported;
    cudaError_t e = cudaFuncSetAttribute(window_dq_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, Q::SMEM);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(window_dkv_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, K::SMEM);
    if (e != cudaSuccess) return e;
    window_dq_kernel<DP><<<(unsigned)((size_t)a.B * a.H * ((a.n + T - 1) / T)), kThreads, Q::SMEM, st>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    window_dkv_kernel<DP><<<dim3((unsigned)((size_t)a.B * a.Hkv * ((a.nk + T - 1) / T)), a.far + 1), kThreads, K::SMEM, st>>>(p);
    return cudaGetLastError();
}

bool rows16(const View &v) {
    return (reinterpret_cast<uintptr_t>(v.p) & 15u) == 0 && v.sb % 8 == 0 && v.sh % 8 == 0 && v.st % 8 == 0;
}

}  // namespace

bool bwd_tc_takes(const Args &a) {
    return a.d % 8 == 0 && a.dv % 8 == 0 && mappable(a.q) && mappable(a.k) && mappable(a.v) && mappable(a.go) && mappable(a.o) &&
           rows16(a.dq) && rows16(a.dk) && rows16(a.dv_);
}

cudaError_t bwd_tc(const Args &a, cudaStream_t st) {
    Params p;
    memset(&p, 0, sizeof p);
    p.a = a;
    return a.d <= 64 && a.dv <= 64 ? launch<64>(p, st) : launch<128>(p, st);
}

}  // namespace win
}  // namespace hla
