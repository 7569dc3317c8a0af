// hla_ssm_bwd_tc.cu -- backward of the selective state space scan for bf16 on the tensor cores
// (formulas in hla_ssm.h).
//
// states_kernel walks the pieces of hla_ssm_carry.cuh forward and then back and leaves, for every
// chunk and head, the state before it and the gradient behind it as bf16 tile images, and in fp32
// what they make of the tokens' own rows and of each other: w', v' and <g, h>, which the gradients of
// dt, A and dt_bias need.
// grad_kernel then takes a chunk of one group: B, C and C B^T (in registers) stay, the heads pass by
// 64 columns at a time.  Per head, rows j and columns t:
//   X dY^T                      -> M^T, S^T (bf16, with dt_j), sums of E = M o (dY X^T) in fp32
//   B g, M^T dY                 -> dX
//   S^T C, S B, (e dY) h^T, (w X) g^T: dB and dC, accumulated in TMEM over the heads
// so that dB and dC leave once per CTA.  A chunk's heads are shared by several CTAs only where
// chunks alone are too few; their parts are then added by a kernel of its own.  finish_kernel puts
// the sums together.
// Roundings: M, S and the images once, since dx, dB and dC are stored in bf16 anyway and a second part of any
// would double its products; the weighted rows that meet h and g in two parts, which GB's free columns
// hold (dB, dC 2.6e-3 -> 2.3e-3 off).  What the gradients of dt, A and dt_bias take is never rounded.
// Roles of grad_kernel (20 warps): 0-15 elementwise, 16 MMA, 17 loads of X, dY and weights, 18 of B, C
// and the images, 19 stores dX and the sums.
#include <cstring>

#include "hla_ssm_carry.cuh"

namespace hla {
namespace ssm {
namespace {

using namespace tcs;

// ------------------------------------------------------------ states of the chunks
// A piece forward and then back: on the way forward the state before each chunk, on the way back the
// gradient behind it, both as bf16 tile images, and in fp32 what they make of every token's own rows:
// w' = 2^s dY.(C h), v' = 2^(s_end - s) X.(B g).  The state meets C (or B) in three bf16 parts, like the
// rows that enter it.  Each thread lays its part of the state aside on the way forward and forms its
// share of <g, h> with it on the way back.  (With <g, h> followed from chunk to chunk by what w' and
// v' add up to, its error runs through all tokens behind it: dA came out 3e-5 off.)
// b2 n8192 h32 p64 s128: 170 us, 128 CTAs of 64 visits, 670 MB to and from memory (half of what could
// move in the time); a visit's 4,800 cycles are the elementwise warps': 2,300 issue slots of each
// scheduler, and latency.
// Roles (20 warps): 0-15 elementwise, 16 MMA, 17 loads of the rows that enter, 18 of those that meet
// the state and the images' stores, 19 loads of B and C.
constexpr int kStatesThreads = 20 * 32;
template <int NB>
struct LayStates {
    static constexpr int NX = 2, ND = 4;           // stages of the rows that enter, of the weights
    static constexpr int HB = NB * kHalf / 2;      // one part of a state
    static constexpr int OFF_X = 0, OFF_Y = NX * kHalf, OFF_P = OFF_Y + kHalf, OFF_Q = OFF_P + NB * kHalf, OFF_W = OFF_Q + NB * kHalf,
                         OFF_H = OFF_W + 3 * kHalf, OFF_DEC = OFF_H + 3 * HB, OFF_BAR = OFF_DEC + ND * kDecBytes;
    static constexpr int B_X = 0, B_XE = B_X + NX, B_Y = B_XE + NX, B_YE = B_Y + 1, B_P = B_YE + 1, B_PE = B_P + 1, B_Q = B_PE + 1, B_QE = B_Q + 1,
                         B_W = B_QE + 1, B_H = B_W + 1, B_D = B_H + 1, B_Z = B_D + 1, B_SE = B_Z + 1, B_FIN = B_SE + 1, B_RAWX = B_FIN + 1, B_RAWY = B_RAWX + 1,
                         B_RAWB = B_RAWY + 1, NBAR = B_RAWB + 1;
    static constexpr int SMEM = OFF_BAR + NBAR * 8 + 16;
    static constexpr uint32_t D = 0, Z = 192;  // TMEM columns
    HLA_DEVICE static int arrivals(int i) { return (i >= B_XE && i < B_Y) || i == B_YE || i == B_W || i == B_H ? kElemWarps : 1; }
};
struct StatesParams {
    Params p;
    uint8_t *image[2];  // [B][H][PT][chunks][64 NB rows][64]
    float *inter;       // [dir][PT][4][B][H][chunks * T]: w', v' by quarters of the columns
    float4 *aside;      // [B][H][PT][chunks][4][512]: states, by the threads that formed them
    float *dots;        // [B][H][chunks][PT][16]: <g, h> by warps
};
struct Walk {  // 2 K visits to the chunks of a piece
    Piece w;
    int K;
    HLA_DEVICE int dir(int k) const { return k >= K; }
    HLA_DEVICE int chunk(int k) const { return k < K ? w.lo + k : w.hi - 1 - (k - K); }
};

HLA_DEVICE float dot16(const float2 (&x)[8], const float2 (&y)[8]) {
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fma2(x[i], y[i], s);
    return s.x + s.y;
}
HLA_DEVICE float lanes_sum(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
HLA_DEVICE void load_row16(const uint8_t *tile, int rows, int r, int c0, float2 (&v)[8]) {
    unpack8(*reinterpret_cast<const uint4 *>(tile + tile_off(rows, r, c0)), v);
    unpack8(*reinterpret_cast<const uint4 *>(tile + tile_off(rows, r, c0 + 8)), v + 4);
}

template <int NB>
__device__ __forceinline__ void states_elem(const StatesParams &sp, const Waits &ws, uint8_t *base, uint32_t tb, const Walk &z) {
    using L = LayStates<NB>;
    const Params &p = sp.p;
    const Args &a = p.a;
    const Piece &w = z.w;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = warp & 3, cq = warp >> 2, row = 32 * q + lane, c0 = 16 * cq;
    const uint32_t lanes = tb + ((uint32_t)(32 * q) << 16);
    const int col = 64 * w.pt + c0, visits = 2 * z.K;
    const bool holds = q < 2 * NB;  // rows of the state
    const size_t unit = (size_t)w.b * a.H + w.h, NP = (size_t)a.N * a.P, plane = (size_t)a.B * a.H * a.nc * T;
    float2 carry[8];
    auto begin = [&](int dir) {
        const float *init = dir ? a.d_state_out : a.state_in;
        load_state(a, p.plan.pieces > 1 && w.used > 0 ? piece_state(p, dir, w) : init ? init + unit * NP : nullptr, row, col, carry);
    };
    auto dec = [&](int k) -> const Dec & { return *reinterpret_cast<const Dec *>(base + L::OFF_DEC + k % L::ND * kDecBytes); };
    auto aside = [&](int c) { return sp.aside + ((unit * p.plan.PT + w.pt) * a.nc + c) * 2048 + threadIdx.x; };
    // The rows that enter do not depend on the state: they are scaled a visit ahead, while the state meets
    // Q, and their product runs while the next state is split.
    auto scale = [&](int k) {
        if (!ws.wait(L::B_X + (k & 1), ring_phase<2>(k))) return false;
        const Dec &d = dec(k);
        scale_split16(base + L::OFF_X + (k & 1) * kHalf, base + L::OFF_W, row, c0, z.dir(k) ? d.to[row] : d.w[row]);
        fence_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(ws.bar(L::B_W));
            mbar_arrive(ws.bar(L::B_XE + (k & 1)));  // (every warp is also through with visit k - 2, whose weights leave next)
        }
        return true;
    };
    begin(0);
    bool ok = visits == 0 || scale(0);
#pragma unroll 1
    for (int k = 0; k < visits && ok; ++k) {
        const uint32_t ph = (uint32_t)k & 1u;
        const int c = z.chunk(k), dir = z.dir(k);
        const Dec &d = dec(k);
        // the state before (the gradient behind) the chunk
        if (k == z.K) begin(1);
        float4 h[4];
        if (k > 0 && !(ok = ws.wait(L::B_SE, ph ^ 1u))) break;
        if (holds) {
            if (dir) {
#pragma unroll
                for (int i = 0; i < 4; ++i) h[i] = aside(c)[512 * i];
            }
            store_split8<true>(base + L::OFF_H, L::HB, 64 * NB, row, c0, carry);
            store_split8<true>(base + L::OFF_H, L::HB, 64 * NB, row, c0 + 8, carry + 4);
        }
        fence_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(ws.bar(L::B_H));
        if (dir) {
            float s = 0.f;
            if (holds) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s = fmaf(h[i].x, carry[2 * i].x, s);
                    s = fmaf(h[i].y, carry[2 * i].y, s);
                    s = fmaf(h[i].z, carry[2 * i + 1].x, s);
                    s = fmaf(h[i].w, carry[2 * i + 1].y, s);
                }
            }
            s = lanes_sum(s);
            if (lane == 0) sp.dots[((unit * a.nc + c) * p.plan.PT + w.pt) * 16 + warp] = s;
        } else if (holds) {
#pragma unroll
            for (int i = 0; i < 4; ++i) aside(c)[512 * i] = make_float4(carry[2 * i].x, carry[2 * i].y, carry[2 * i + 1].x, carry[2 * i + 1].y);
        }
        if (!(ok = ws.wait(L::B_D, ph))) break;
        tc_fence_after();
        float2 v[8];
        if (holds) {
            load_parts16(lanes + L::D + c0, v);
            const float end = d.end;
#pragma unroll
            for (int i = 0; i < 8; ++i) carry[i] = fma2(both(end), carry[i], v[i]);
        }
        if (k + 1 >= z.K && k + 1 < visits && holds) {  // laid aside long ago
#pragma unroll
            for (int i = 0; i < 4; ++i) prefetch_l2(aside(z.chunk(k + 1)) + 512 * i);
        }
        if (k + 1 < visits && !(ok = scale(k + 1))) break;
        if (!(ok = ws.wait(L::B_Y, ph) && ws.wait(L::B_Z, ph))) break;
        tc_fence_after();
        load_parts16(lanes + L::Z + c0, v);
        {
            float2 y[8];
            load_row16(base + L::OFF_Y, T, row, c0, y);
            const float f = dir ? factor(d.s[T - 1], d.s[row]) : d.to[row];
            sp.inter[((size_t)(dir * p.plan.PT + w.pt) * 4 + cq) * plane + (unit * a.nc + c) * T + row] = f * dot16(v, y);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(ws.bar(L::B_YE));
    }
    if (visits == 0) begin(1);  // (no tokens: the gradient passes as it is)
    if (ok && w.piece == 0 && a.d_state_in && holds) store_state(a, a.d_state_in + unit * NP, row, col, carry);
}

template <int NB>
__device__ __forceinline__ void states_mma(const Waits &ws, uint8_t *base, uint32_t tb, int K) {
    using L = LayStates<NB>;
    constexpr uint32_t id = make_idesc(T, 192, false, true);
    const uint64_t H = make_sdesc(smem_u32(base + L::OFF_H), L::HB, 1024u), W = mnmajor(base + L::OFF_W);
    const uint64_t P = mnmajor(base + L::OFF_P), Q = kmajor(base + L::OFF_Q);
#pragma unroll 1
    for (int k = 0; k < K; ++k) {
        const uint32_t ph = (uint32_t)k & 1u;
        if (!ws.wait(L::B_W, ph) || !ws.wait(L::B_P, ph)) break;
        tc_fence_after();
        mma_state(tb + L::D, P, W, false);
        umma_commit_warp(ws.bar(L::B_D));
        umma_commit_warp(ws.bar(L::B_PE));
        if (!ws.wait(L::B_H, ph) || !ws.wait(L::B_Q, ph)) break;
        tc_fence_after();
        mma_km64(tb + L::Z, Q, H, id, false);
        if (NB > 1) mma_km64(tb + L::Z, Q + kBlock, H + kRows64, id, true);
        umma_commit_warp(ws.bar(L::B_Z));
        umma_commit_warp(ws.bar(L::B_QE));
    }
    umma_commit_warp(ws.bar(L::B_FIN));  // every MMA issued completes before TMEM is released
    mbar_wait(ws.bar(L::B_FIN), 0u, ws.err);
    __syncwarp();
}

// One warp's stream of tiles through SLOTS slots, with barriers for landed, free and raw.
template <int BLOCKS, int SLOTS, class First, class Issue>
HLA_DEVICE void stream(const Waits &ws, int K, int full, int empty, int rawb, uint8_t *tiles, int len, First first, Issue issue) {
    uint32_t raw = 0;
    int k = 0;
    bool ok = true;
#pragma unroll 1
    for (; k < K && ok; ++k) {
        const int s = k % SLOTS, t0 = first(k);
        if (k >= SLOTS && !(ok = ws.wait(empty + s, ring_phase<SLOTS>(k) ^ 1u))) break;
        const bool clear = len - t0 < T;
        uint8_t *t = tiles + s * BLOCKS * kHalf;
        if ((threadIdx.x & 31) == 0) issue(k, t, ws.bar(clear ? rawb : full + s));
        __syncwarp();
        if (clear) ok = clear_landed(ws, rawb, raw, full + s, t, BLOCKS, len - t0);
    }
    wait_landed<SLOTS>(ws, full, k);
}

template <int NB>
__device__ __forceinline__ void states_load(const StatesParams &sp, const Waits &ws, uint8_t *base, const Walk &z, int warp) {
    using L = LayStates<NB>;
    const Params &p = sp.p;
    const Args &a = p.a;
    const Piece &w = z.w;
    const int g = w.h / a.R, lane = threadIdx.x & 31, visits = 2 * z.K;
    auto first = [&](int k) { return z.chunk(k) * T; };
    uint32_t raw = 0;
    bool ok = true;
    if (warp == kWarpTma) {
        stream<1, L::NX>(ws, visits, L::B_X, L::B_XE, L::B_RAWX, base + L::OFF_X, w.len, first, [&](int k, uint8_t *t, uint64_t *bar) {
            mbar_expect_tx(bar, kHalf + kDecBytes);
            bulk_load(base + L::OFF_DEC + k % L::ND * kDecBytes, dec_of(a, p.dec, w.b, w.h, z.chunk(k)), kDecBytes, bar);
            load_tile<1>(t, &p.mx[z.dir(k)], p.vx[z.dir(k)], bar, 64 * w.pt, first(k), w.h, w.b);
        });
    } else if (warp == kWarpTmaX) {  // the rows that meet the state; the state's image leaves in between
        int k = 0;
#pragma unroll 1
        for (; k < visits && ok; ++k) {
            const int t0 = first(k), d = 1 - z.dir(k);
            const bool clear = w.len - t0 < T;
            if (k > 0 && !(ok = ws.wait(L::B_YE, ((uint32_t)k & 1u) ^ 1u))) break;
            if (lane == 0) {
                uint64_t *bar = ws.bar(clear ? L::B_RAWY : L::B_Y);
                mbar_expect_tx(bar, kHalf);
                load_tile<1>(base + L::OFF_Y, &p.mx[d], p.vx[d], bar, 64 * w.pt, t0, w.h, w.b);
            }
            __syncwarp();
            if (clear) ok = clear_landed(ws, L::B_RAWY, raw, L::B_Y, base + L::OFF_Y, 1, w.len - t0);
            if (!ok || !(ok = ws.wait(L::B_H, (uint32_t)k & 1u))) {
                ++k;
                break;
            }
            if (lane == 0) {
                const size_t at = (((size_t)w.b * a.H + w.h) * p.plan.PT + w.pt) * a.nc + z.chunk(k);
                bulk_store(sp.image[z.dir(k)] + at * L::HB, base + L::OFF_H, L::HB);
                bulk_commit();
                bulk_wait_read();
                mbar_arrive(ws.bar(L::B_SE));
            }
            __syncwarp();
        }
        wait_landed<1>(ws, L::B_Y, k);
        if (lane == 0) bulk_wait_all();
        __syncwarp();
    } else {  // the two tiles of a chunk in turn
        int r = 0;
#pragma unroll 1
        for (; r < 2 * visits && ok; ++r) {
            const int second = r & 1, k = r >> 1, t0 = first(k), d = second ? 1 - z.dir(k) : z.dir(k), full = second ? L::B_Q : L::B_P;
            const bool clear = w.len - t0 < T;
            if (k > 0 && !(ok = ws.wait(second ? L::B_QE : L::B_PE, ((uint32_t)k & 1u) ^ 1u))) break;
            uint8_t *t = base + (second ? L::OFF_Q : L::OFF_P);
            if (lane == 0) {
                uint64_t *bar = ws.bar(clear ? L::B_RAWB : full);
                mbar_expect_tx(bar, NB * kHalf);
                load_tile<NB>(t, &p.mb[d], p.vb[d], bar, 0, t0, g, w.b);
            }
            __syncwarp();
            if (clear) ok = clear_landed(ws, L::B_RAWB, raw, full, t, NB, w.len - t0);
        }
        wait_landed<1>(ws, L::B_P, (r + 1) / 2);
        wait_landed<1>(ws, L::B_Q, r / 2);
    }
}

template <int NB>
__global__ void __launch_bounds__(kStatesThreads, 1) ssm_states_kernel(const __grid_constant__ StatesParams sp) {
    using L = LayStates<NB>;
    extern __shared__ __align__(1024) uint8_t base[];
    Walk z;
    z.w = piece_of(sp.p.a, sp.p.plan, blockIdx.x);
    if (z.w.piece >= max(z.w.used, 1)) return;
    z.K = z.w.hi - z.w.lo;
    Cta<L::NBAR> cta(base, L::OFF_BAR, sp.p.a.err, [](int i) { return L::arrivals(i); });
    if (cta.warp < kElemWarps)
        states_elem<NB>(sp, cta.ws, base, cta.tb, z);
    else if (cta.warp == kWarpMma)
        states_mma<NB>(cta.ws, base, uniform(cta.tb), (int)uniform(2 * z.K));
    else
        states_load<NB>(sp, cta.ws, base, z, cta.warp);
    cta.finish();
}

// ------------------------------------------------------------ gradients of a chunk
// b2 n8192 h32 p64 s128: 147 us, 128 CTAs of 32 heads, 8,300 cycles a head.  Half of it are M, S and the
// sums of E, of which the triangle leaves four warps' worth to one scheduler and one to another (rows
// belong to schedulers: TMEM lanes), then the weighted rows and dX; a head's products and tiles keep
// shared memory busy for 3,400.
constexpr int kGradThreads = 20 * 32;

struct GradParams {
    Args a;
    int PT, splits;
    View vx, vdy, vb, vc;
    CUtensorMap mx, mdy, mb, mc, mdx;
    const Dec *dec;
    const uint8_t *h, *g;  // images
    float *own;            // [w, vE, diagonal][B][H][chunks * T]: sums of E
    float *dd;             // [B][H][chunks]: dY.X
};

template <int NB>
struct LayGrad {
    static constexpr int HB = NB * kHalf / 2, NS = 4;  // dY and X of the heads in turn through four slots
    static constexpr int OFF_B = 0, OFF_C = NB * kHalf, OFF_S = 2 * NB * kHalf, OFF_XD = OFF_S + 2 * kHalf, OFF_H = OFF_XD + NS * kHalf,
                         OFF_G = OFF_H + HB;
    static constexpr int OFF_DEC = OFF_G + HB, OFF_SUM = OFF_DEC + 2 * (int)sizeof(Dec);
    static constexpr int SUM_FLOATS = 13 * T;  // [w by rows' quadrant][4][128], [vE by columns' quarter][4][128], [dY.X by columns' quarter][4][128], C.B [128]
    static constexpr int OFF_BAR = OFF_SUM + SUM_FLOATS * 4;
    static constexpr int B_XD = 0, B_XDE = B_XD + NS, B_DEC = B_XDE + NS, B_DECE = B_DEC + 2, B_H = B_DECE + 2, B_HE = B_H + 1,
                         B_G = B_HE + 1, B_LO = B_G + 1, B_LE = B_LO + 1, B_BC = B_LE + 1, B_CB = B_BC + 1, B_DYX = B_CB + 1, B_DE = B_DYX + 1,
                         B_GB = B_DE + 1, B_MS = B_GB + 1, B_XM = B_MS + 1, B_SE = B_XM + 1, B_YT = B_SE + 1, B_Y = B_YT + 1,
                         B_SUM = B_Y + 2, B_SUME = B_SUM + 1, B_FIN = B_SUME + 1, B_RAW = B_FIN + 1, B_RAW2 = B_RAW + 1, NBAR = B_RAW2 + 1;
    static constexpr int SMEM = OFF_BAR + NBAR * 8 + 16;
    static constexpr uint32_t DC = 0, DB = T, DYX = 2 * T, M = 2 * T, XM = 2 * T + 64, YT = 3 * T, XT = YT + 32, GB = 3 * T + 64;
    HLA_DEVICE static int arrivals(int i) {
        return (i >= B_XDE && i < B_DEC) || i == B_DECE || i == B_DECE + 1                                 ? kElemWarps + 1
               : i == B_DE || i == B_MS || i == B_YT || i == B_LO || i == B_Y || i == B_Y + 1 || i == B_SUM ? kElemWarps
                                                                                               : 1;
    }
};

struct Job {  // one chunk of a group, the heads [h0, h1), U = heads x column tiles
    int b, g, c, len, t0, live, split, h0, U;
};
HLA_DEVICE int head_of(const GradParams &p, const Job &j, int u) { return j.h0 + u / p.PT; }

// Sums over the warp's lanes of 16 columns: lane l < 16 (and l + 16) ends with column l.
HLA_DEVICE float lane_sums16(float (&v)[16]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int c = 8; c > 0; c >>= 1) {
        const bool up = lane & c;
#pragma unroll
        for (int i = 0; i < c; ++i) {
            const float send = up ? v[i] : v[i + c], keep = up ? v[i + c] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, c);
        }
    }
    return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 16);
}
template <int NB>
__device__ __forceinline__ void grad_elem(const GradParams &p, const Waits &ws, uint8_t *base, uint32_t tb, const Job &job) {
    using L = LayGrad<NB>;
    const Args &a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = warp & 3, cq = warp >> 2, row = 32 * q + lane, c0 = 16 * cq;
    const uint32_t lanes = tb + ((uint32_t)(32 * q) << 16);
    float *sums = reinterpret_cast<float *>(base + L::OFF_SUM);
    float *sum_w = sums + q * T + 32 * cq, *sum_ve = sums + 4 * T + cq * T;
    const bool active = cq >= q;  // tokens t of this warp's columns at or behind its rows j
    float2 cb[16];
    bool ok = ws.wait(L::B_CB, 0u);
    tc_fence_after();
    if (active && ok) {
        tmem_pairs16(lanes + L::DYX + 32 * cq, reinterpret_cast<float2(&)[8]>(cb[0]));
        tmem_pairs16(lanes + L::DYX + 32 * cq + 16, reinterpret_cast<float2(&)[8]>(cb[8]));
        tmem_wait_ld();
    }
    tc_fence_before();
    if (cq == q) {  // this row's own
        float c = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) c = lane == 2 * i ? cb[i].x : lane == 2 * i + 1 ? cb[i].y : c;
        sums[12 * T + row] = c;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(ws.bar(L::B_DE));  // the products' columns are free
    uint8_t *S = base + L::OFF_S;
#pragma unroll 1
    for (int u = 0; u < job.U; ++u) {
        const uint32_t ph = (uint32_t)u & 1u;
        const int h = head_of(p, job, u), sy = (2 * u) % L::NS, sx = (2 * u + 1) % L::NS;
        const uint8_t *dy = base + L::OFF_XD + sy * kHalf;
        uint8_t *x = base + L::OFF_XD + sx * kHalf;
        const Dec &d = *reinterpret_cast<const Dec *>(base + L::OFF_DEC + (u & 1) * sizeof(Dec));
        // M^T, S^T and the sums of E over this thread's 32 columns
        ok = ok && ws.wait(L::B_DEC + (u & 1), ring_phase<2>(u)) && ws.wait(L::B_DYX, ph);
        if (u > 0) ok = ok && ws.wait(L::B_SE, ph ^ 1u) && ws.wait(L::B_SUME, ph ^ 1u);
        tc_fence_after();
        const Decay s = d.s[row];
        const float dt = d.dt[row];
        uint32_t pk[16];
        float ve = 0.f;
        if (active && ok) {
            const Decay first = d.s[32 * cq];
            const bool plain = cq > q || first.hi - d.s[32 * cq + 31].hi <= kBlockRange;
            const float2 f0 = both(plain ? factor(first, s) : 1.f);
            const uint32_t bits = cq > q ? 0xffffffffu : ~low_bits(lane), past = cq > q ? 0xffffffffu : ~low_bits(lane + 1);  // t >= j, t > j
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                float2 v[8];
                tmem_pairs16(lanes + L::DYX + 32 * cq + 16 * g, v);
                tmem_wait_ld();
                float e[16];
                uint32_t sp[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int t = 32 * cq + 16 * g + 2 * i;
                    float2 f;
                    if (plain) {
                        f = mul2(f0, *reinterpret_cast<const float2 *>(d.fw + t));
                    } else {
                        const float4 st = *reinterpret_cast<const float4 *>(d.s + t);
                        f = make_float2(factor({st.x, st.y}, s), factor({st.z, st.w}, s));
                    }
                    f.x = bits & (1u << (16 * g + 2 * i)) ? f.x : 0.f;  // (above the diagonal a factor may be anything)
                    f.y = bits & (2u << (16 * g + 2 * i)) ? f.y : 0.f;
                    const float2 m = mul2(cb[8 * g + i], f), sv = mul2(v[i], f), ee = mul2(m, v[i]);
                    // E's diagonal, C.B dY.X of one token, is formed apart: it cancels in the gradient of the
                    // decays, which differences of these sums give, and where decays are steep it is most of
                    // them (within the sums: dA 2.0e-6 off, dt_bias 8.5e-6, b2 n8192; apart 4.7e-7, 1.2e-6)
                    const float ex = past & (1u << (16 * g + 2 * i)) ? ee.x : 0.f, ey = past & (2u << (16 * g + 2 * i)) ? ee.y : 0.f;
                    ve += ex + ey;
                    e[2 * i] = ex * dt;
                    e[2 * i + 1] = ey * dt;
                    pk[8 * g + i] = pack2(mul2(m, both(dt)));
                    sp[i] = pack2(mul2(sv, both(dt)));
                }
                *reinterpret_cast<uint4 *>(S + tile_off(T, row, 32 * cq + 16 * g)) = make_uint4(sp[0], sp[1], sp[2], sp[3]);
                *reinterpret_cast<uint4 *>(S + tile_off(T, row, 32 * cq + 16 * g + 8)) = make_uint4(sp[4], sp[5], sp[6], sp[7]);
                const float w = lane_sums16(e);
                if (lane < 16) sum_w[16 * g + lane] = w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) pk[i] = 0u;
#pragma unroll
            for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4 *>(S + tile_off(T, row, 32 * cq + 8 * i)) = make_uint4(0, 0, 0, 0);
            sum_w[lane] = 0.f;
        }
        sum_ve[row] = ve;
        quad_sync(q);  // every warp of these rows has read its columns of the product that M^T overwrites
        tc_fence_after();
        tmem_st16(lanes + L::M + 16 * cq, reinterpret_cast<float(&)[16]>(pk));
        tmem_wait_st();
        fence_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(ws.bar(L::B_MS));
        // the weighted rows of dY and X, for the states' shares of dC and dB
        ok = ok && ws.wait(L::B_XD + sy, ring_phase<L::NS>(2 * u)) && ws.wait(L::B_XD + sx, ring_phase<L::NS>(2 * u + 1));
        if (u > 0) ok = ok && ws.wait(L::B_HE, ph ^ 1u);  // the last head's have been used
        float2 yr[8], xr[8];
        load_row16(dy, T, row, c0, yr);
        load_row16(x, T, row, c0, xr);
        const float2 to = both(d.to[row]), w = both(d.w[row]), D = both(a.D ? a.D[h] : 0.f);
        float ly[8], lx[8];  // what rounding leaves of them
        {
            float ty[8], tx[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 fy = mul2(yr[i], to), fx = mul2(xr[i], w);
                const uint32_t hy = pack2(fy), hx = pack2(fx);
                ty[i] = __uint_as_float(hy);
                tx[i] = __uint_as_float(hx);
                ly[i] = __uint_as_float(pack2(less(fy, hy)));
                lx[i] = __uint_as_float(pack2(less(fx, hx)));
            }
            tc_fence_after();
            tmem_st8(lanes + L::YT + 8 * cq, ty);
            tmem_st8(lanes + L::XT + 8 * cq, tx);
        }
        sums[(8 + cq) * T + row] = dot16(xr, yr);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(ws.bar(L::B_YT));
            mbar_arrive(ws.bar(L::B_XDE + sy));
            mbar_arrive(ws.bar(L::B_SUM));
            mbar_arrive(ws.bar(L::B_DECE + (u & 1)));
        }
        // dX = M^T dY (with dt) + w B g + D dY, over X
        ok = ok && ws.wait(L::B_GB, ph);
        tc_fence_after();
        float2 v[8];
        tmem_pairs16(lanes + L::GB + c0, v);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 8; ++i) yr[i] = fma2(D, yr[i], mul2(w, v[i]));
        tmem_st8(lanes + L::GB + c0, ly);  // in the columns that this warp has just read
        tmem_st8(lanes + L::GB + c0 + 8, lx);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(ws.bar(L::B_LO));
        ok = ok && ws.wait(L::B_XM, ph);
        tc_fence_after();
        tmem_pairs16(lanes + L::XM + c0, v);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = add2(v[i], yr[i]);
        store_row8(x, T, row, c0, v);
        store_row8(x, T, row, c0 + 8, v + 4);
        fence_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(ws.bar(L::B_DE));
            mbar_arrive(ws.bar(L::B_Y + (u & 1)));
            mbar_arrive(ws.bar(L::B_XDE + sx));
        }
    }
    // dC and dB of the chunk: rows t (or j), this warp's quarter of the columns
    if (!ok || !ws.wait(L::B_FIN, 0u)) return;
    tc_fence_after();
    constexpr int CW = 16 * NB;
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {
        const View &o = k ? a.db : a.dc;
#pragma unroll 1
        for (int g = 0; g < CW; g += 16) {
            float2 v[8];
            const int col = CW * cq + g;
            tmem_pairs16(lanes + (k ? L::DB : L::DC) + col, v);
            tmem_wait_ld();
            if (row < job.live) {
                if (p.splits == 1) {
                    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(o.p) + (size_t)job.b * o.sb + (size_t)job.g * o.sh + (size_t)(job.t0 + row) * o.st + col;
#pragma unroll
                    for (int i = 0; i < 8; i += 4)
                        if (col + 2 * i < a.N)
                            *reinterpret_cast<uint4 *>(out + 2 * i) = make_uint4(pack2(v[i]), pack2(v[i + 1]), pack2(v[i + 2]), pack2(v[i + 3]));
                } else {
                    const size_t half = (size_t)a.B * a.G * a.n * a.N;
                    float *out = a.dbc + ((size_t)2 * job.split + (k ? 0 : 1)) * half + (((size_t)job.b * a.G + job.g) * a.n + job.t0 + row) * a.N + col;
#pragma unroll
                    for (int i = 0; i < 8; i += 2)
                        if (col + 2 * i < a.N) *reinterpret_cast<float4 *>(out + 2 * i) = make_float4(v[i].x, v[i].y, v[i + 1].x, v[i + 1].y);
                }
            }
            __syncwarp();
        }
    }
}

template <int NB>
__device__ __forceinline__ void grad_mma(const Waits &ws, uint8_t *base, uint32_t tb, int U) {
    using L = LayGrad<NB>;
    constexpr uint32_t id_tt = make_idesc(T, T, false, false), id_y = make_idesc(T, 64, false, true), id_n = make_idesc(T, 64 * NB, false, true),
                       id_nn = make_idesc(T, 64 * NB, true, true), id_k = make_idesc(T, 64 * NB, false, false);
    const uint64_t Bk = kmajor(base + L::OFF_B), Ck = kmajor(base + L::OFF_C), Bm = mnmajor(base + L::OFF_B), Cm = mnmajor(base + L::OFF_C);
    const uint64_t Sk = kmajor(base + L::OFF_S), Sm = mnmajor(base + L::OFF_S);
    const uint64_t Gm = make_sdesc(smem_u32(base + L::OFF_G), L::HB, 1024u), Hk = kmajor(base + L::OFF_H), Gk = kmajor(base + L::OFF_G);
    bool ok = ws.wait(L::B_BC, 0u);
    if (ok) {
        mma_ss64(tb + L::DYX, Bk, Ck, id_tt, false);
        if (NB > 1) mma_ss64(tb + L::DYX, Bk + kBlock, Ck + kBlock, id_tt, true);
        umma_commit_warp(ws.bar(L::B_CB));
    }
    auto rest = [&](int u) {  // the weighted rows' second parts
        if (!ws.wait(L::B_LO, (uint32_t)u & 1u)) return false;
        tc_fence_after();
        mma_tk64<16>(tb + L::DC, tb + L::GB, Hk, id_k);
        mma_tk64<16>(tb + L::DB, tb + L::GB + 8, Gk, id_k);
        umma_commit_warp(ws.bar(L::B_LE));
        return true;
    };
#pragma unroll 1
    for (int u = 0; u < U && ok; ++u) {
        const uint32_t ph = (uint32_t)u & 1u;
        const int sy = (2 * u) % L::NS, sx = (2 * u + 1) % L::NS;
        const uint8_t *dy = base + L::OFF_XD + sy * kHalf, *x = base + L::OFF_XD + sx * kHalf;
        if (!(ok = ws.wait(L::B_XD + sy, ring_phase<L::NS>(2 * u)) && ws.wait(L::B_XD + sx, ring_phase<L::NS>(2 * u + 1)) && ws.wait(L::B_DE, ph))) break;
        tc_fence_after();
        mma_ss64(tb + L::DYX, kmajor(x), kmajor(dy), id_tt, false);
        umma_commit_warp(ws.bar(L::B_DYX));
        if (u > 0 && !(ok = rest(u - 1))) break;
        if (!(ok = ws.wait(L::B_G, ph))) break;  // (its load waits for rest's products, which read GB's columns)
        mma_km64(tb + L::GB, Bk, Gm, id_y, false);
        if (NB > 1) mma_km64(tb + L::GB, Bk + kBlock, Gm + kRows64, id_y, true);
        umma_commit_warp(ws.bar(L::B_GB));
        if (!(ok = ws.wait(L::B_MS, ph))) break;
        tc_fence_after();
        mma_ts128(tb + L::XM, tb + L::M, mnmajor(dy), id_y);
        umma_commit_warp(ws.bar(L::B_XM));
        mma_mm64(tb + L::DC, Sm, Bm, id_nn, u > 0);  // S B: the tile's rows are j
        mma_mm64(tb + L::DC, Sm + kRows64, Bm + kRows64, id_nn, true);
        mma_km64(tb + L::DB, Sk, Cm, id_n, u > 0);   // S^T C
        mma_km64(tb + L::DB, Sk + kBlock, Cm + kRows64, id_n, true);
        umma_commit_warp(ws.bar(L::B_SE));
        if (!(ok = ws.wait(L::B_YT, ph) && ws.wait(L::B_H, ph))) break;
        tc_fence_after();
        mma_tk64<8>(tb + L::DC, tb + L::YT, Hk, id_k);
        mma_tk64<8>(tb + L::DB, tb + L::XT, Gk, id_k);
        umma_commit_warp(ws.bar(L::B_HE));
        umma_commit_warp(ws.bar(L::B_XDE + sy));
    }
    if (ok && U > 0) rest(U - 1);
    umma_commit_warp(ws.bar(L::B_FIN));  // every MMA issued completes before TMEM is released
    mbar_wait(ws.bar(L::B_FIN), 0u, ws.err);
    __syncwarp();
}

template <int NB>
__device__ __forceinline__ void grad_load_xd(const GradParams &p, const Waits &ws, uint8_t *base, const Job &job) {
    using L = LayGrad<NB>;
    const int lane = threadIdx.x & 31;
    const bool clear = job.live < T;
    uint32_t raw = 0;
    int i = 0, weights = 0;  // copies issued
    bool ok = true;
#pragma unroll 1
    for (; i < 2 * job.U && ok; ++i) {
        const int u = i >> 1, s = i % L::NS, h = head_of(p, job, u), col = 64 * (u % p.PT);
        const bool is_x = i & 1;
        if (!is_x) {
            if (u >= 2 && !(ok = ws.wait(L::B_DECE + (u & 1), ring_phase<2>(u) ^ 1u))) break;
            if (lane == 0) {
                mbar_expect_tx(ws.bar(L::B_DEC + (u & 1)), sizeof(Dec));
                bulk_load(base + L::OFF_DEC + (u & 1) * sizeof(Dec), dec_of(p.a, p.dec, job.b, h, job.c), sizeof(Dec), ws.bar(L::B_DEC + (u & 1)));
            }
            ++weights;
        }
        if (i >= L::NS && !(ok = ws.wait(L::B_XDE + s, ring_phase<L::NS>(i) ^ 1u))) break;
        uint8_t *t = base + L::OFF_XD + s * kHalf;
        if (lane == 0) {
            uint64_t *bar = ws.bar(clear ? L::B_RAW : L::B_XD + s);
            mbar_expect_tx(bar, kHalf);
            if (is_x)
                load_tile<1>(t, &p.mx, p.vx, bar, col, job.t0, h, job.b);
            else
                load_tile<1>(t, &p.mdy, p.vdy, bar, col, job.t0, h, job.b);
        }
        __syncwarp();
        if (clear) ok = clear_landed(ws, L::B_RAW, raw, L::B_XD + s, t, 1, job.live);
    }
    wait_landed<L::NS>(ws, L::B_XD, i);
    wait_landed<2>(ws, L::B_DEC, weights);
}

template <int NB>
__device__ __forceinline__ void grad_load_state(const GradParams &p, const Waits &ws, uint8_t *base, const Job &job) {
    using L = LayGrad<NB>;
    const int lane = threadIdx.x & 31;
    const bool clear = job.live < T;
    if (lane == 0) {
        uint64_t *bar = ws.bar(clear ? L::B_RAW2 : L::B_BC);
        mbar_expect_tx(bar, 2 * NB * kHalf);
        load_tile<NB>(base + L::OFF_B, &p.mb, p.vb, bar, 0, job.t0, job.g, job.b);
        load_tile<NB>(base + L::OFF_C, &p.mc, p.vc, bar, 0, job.t0, job.g, job.b);
    }
    __syncwarp();
    uint32_t raw = 0;
    bool ok = !clear || clear_landed(ws, L::B_RAW2, raw, L::B_BC, base + L::OFF_B, 2 * NB, job.live);
    int u = 0;
#pragma unroll 1
    for (; u < job.U && ok; ++u) {
        const uint32_t ph = (uint32_t)u & 1u;
        const size_t at = (((size_t)job.b * p.a.H + head_of(p, job, u)) * p.PT + u % p.PT) * p.a.nc + job.c;
        if (u > 0 && !(ok = ws.wait(L::B_LE, ph ^ 1u))) break;
        if (lane == 0) {
            mbar_expect_tx(ws.bar(L::B_H), L::HB);
            bulk_load(base + L::OFF_H, p.h + at * L::HB, L::HB, ws.bar(L::B_H));
        }
        __syncwarp();
        if (lane == 0) {
            mbar_expect_tx(ws.bar(L::B_G), L::HB);
            bulk_load(base + L::OFF_G, p.g + at * L::HB, L::HB, ws.bar(L::B_G));
        }
        __syncwarp();
    }
    wait_landed<1>(ws, L::B_BC, 1);
    wait_landed<1>(ws, L::B_H, u);
    wait_landed<1>(ws, L::B_G, u);
}

// dX of each head's columns to memory; after a head's last columns the sums of E, four adjacent
// tokens a lane.
template <int NB>
__device__ __forceinline__ void grad_sums(const GradParams &p, const Waits &ws, uint8_t *base, const Job &job) {
    using L = LayGrad<NB>;
    const Args &a = p.a;
    const int lane = threadIdx.x & 31;
    const float *sums = reinterpret_cast<const float *>(base + L::OFF_SUM);
    float4 w, ve, dg;
    float dd = 0.f;
#pragma unroll 1
    for (int u = 0; u < job.U; ++u) {
        const uint32_t ph = (uint32_t)u & 1u;
        const int h = head_of(p, job, u), pt = u % p.PT, sx = (2 * u + 1) % L::NS;
        if (!ws.wait(L::B_DEC + (u & 1), ring_phase<2>(u)) || !ws.wait(L::B_SUM, ph)) break;
        if (pt == 0) {
            w = ve = dg = make_float4(0.f, 0.f, 0.f, 0.f);
            dd = 0.f;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float4 x = *reinterpret_cast<const float4 *>(sums + k * T + 4 * lane), y = *reinterpret_cast<const float4 *>(sums + (4 + k) * T + 4 * lane);
            w.x += x.x; w.y += x.y; w.z += x.z; w.w += x.w;
            ve.x += y.x; ve.y += y.y; ve.z += y.z; ve.w += y.w;
        }
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 8; k < 12; ++k) {
            const float4 x = *reinterpret_cast<const float4 *>(sums + k * T + 4 * lane);
            s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
        }
        const float4 x = *reinterpret_cast<const float4 *>(sums + 12 * T + 4 * lane);
        dg.x = fmaf(x.x, s.x, dg.x); dg.y = fmaf(x.y, s.y, dg.y); dg.z = fmaf(x.z, s.z, dg.z); dg.w = fmaf(x.w, s.w, dg.w);
        dd += (s.x + s.y) + (s.z + s.w);
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(ws.bar(L::B_SUME));
            mbar_arrive(ws.bar(L::B_DECE + (u & 1)));
        }
        if (pt == p.PT - 1) {
            const size_t at = ((size_t)job.b * a.H + h) * a.nc + job.c, plane = (size_t)a.B * a.H * a.nc * T;
            reinterpret_cast<float4 *>(p.own + at * T)[lane] = w;
            reinterpret_cast<float4 *>(p.own + plane + at * T)[lane] = ve;
            reinterpret_cast<float4 *>(p.own + 2 * plane + at * T)[lane] = dg;
            dd = lanes_sum(dd);
            if (lane == 0) p.dd[at] = dd;
        }
        if (!ws.wait(L::B_Y + (u & 1), ring_phase<2>(u))) break;
        store_tile(base + L::OFF_XD + sx * kHalf, &p.mdx, a.dx, pt, job.t0, job.live, h, job.b, a.P);
        if (lane == 0) mbar_arrive(ws.bar(L::B_XDE + sx));
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
}

template <int NB>
__global__ void __launch_bounds__(kGradThreads, 1) ssm_grad_tc_kernel(const __grid_constant__ GradParams p) {
    using L = LayGrad<NB>;
    extern __shared__ __align__(1024) uint8_t base[];
    const Args &a = p.a;
    Job j;
    j.split = blockIdx.x % p.splits;
    j.g = blockIdx.x / p.splits % a.G;
    j.c = blockIdx.x / p.splits / a.G % a.nc;
    j.b = blockIdx.x / p.splits / a.G / a.nc;
    j.len = clamp_length(a.lengths, j.b, a.n);
    j.t0 = j.c * T;
    j.live = min(T, j.len - j.t0);
    j.h0 = j.g * a.R + (int)((long long)a.R * j.split / p.splits);
    const int h1 = j.g * a.R + (int)((long long)a.R * (j.split + 1) / p.splits);
    j.U = (h1 - j.h0) * p.PT;
    if (j.live <= 0) return;
    Cta<L::NBAR> cta(base, L::OFF_BAR, a.err, [](int i) { return L::arrivals(i); });
    if (cta.warp < kElemWarps)
        grad_elem<NB>(p, cta.ws, base, cta.tb, j);
    else if (cta.warp == kWarpMma)
        grad_mma<NB>(cta.ws, base, uniform(cta.tb), (int)uniform(j.U));
    else if (cta.warp == kWarpTma)
        grad_load_xd<NB>(p, cta.ws, base, j);
    else if (cta.warp == kWarpTmaX)
        grad_load_state<NB>(p, cta.ws, base, j);
    else
        grad_sums<NB>(p, cta.ws, base, j);
    cta.finish();
}

// ------------------------------------------------------------ gradients of the steps
// A warp for a chunk of a head; a CTA's chunks are those of one piece.
constexpr int kFinishWarps = 16;
__global__ void __launch_bounds__(kFinishWarps * 32, 1) ssm_finish_kernel(const __grid_constant__ StatesParams sp, const float *own, const float *dd) {
    __shared__ float part[3][kFinishWarps];
    const Params &p = sp.p;
    const Args &a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int piece = blockIdx.x % p.plan.pieces, h = blockIdx.x / p.plan.pieces % a.H, b = blockIdx.x / p.plan.pieces / a.H;
    const int len = clamp_length(a.lengths, b, a.n), chunks = (len + T - 1) / T, PT = p.plan.PT;
    const int lo = min(piece * p.plan.per, chunks), hi = min(lo + p.plan.per, chunks);
    const size_t unit = (size_t)b * a.H + h, plane = (size_t)a.B * a.H * a.nc * T;
    float sA = 0.f, sD = 0.f, sb = 0.f;
    const float A = a.A[h];
#pragma unroll 1
    for (int c = lo + warp; c < hi; c += kFinishWarps) {
        const Dec &d = *dec_of(a, p.dec, b, h, c);
        const size_t at = unit * a.nc + c;
        float w[4], vi[4], vo[4], dg[4], dt[4], sl[4];  // four adjacent tokens
        auto read = [&](const float *q, float (&v)[4]) {
            const float4 x = reinterpret_cast<const float4 *>(q)[lane];
            v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
        };
        read(own + at * T, w);
        read(own + plane + at * T, vo);
        read(own + 2 * plane + at * T, dg);
        read(d.dt, dt);
        read(d.slope, sl);
#pragma unroll
        for (int i = 0; i < 4; ++i) vi[i] = 0.f;
        float th = 0.f;
#pragma unroll 1
        for (int k = 0; k < PT; ++k) {
            if (lane < 16) th += sp.dots[(at * PT + k) * 16 + lane];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float x[4], y[4];
                read(sp.inter + (size_t)(k * 4 + j) * plane + at * T, x);
                read(sp.inter + (size_t)((PT + k) * 4 + j) * plane + at * T, y);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    w[i] += x[i];
                    vi[i] += y[i];
                }
            }
        }
        th = lanes_sum(th) * d.end;
        float suf[4], pre[4], s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 3; i >= 0; --i) {
            s1 += fmaf(-dt[i], vo[i], w[i]);
            suf[i] = s1;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            pre[i] = s2;
            s2 = fmaf(dt[i], vi[i], s2);
        }
        float xs = s1, xp = s2;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float us = __shfl_down_sync(0xffffffffu, xs, o), up = __shfl_up_sync(0xffffffffu, xp, o);
            if (lane + o < 32) xs += us;
            if (lane >= o) xp += up;
        }
        xs = __shfl_down_sync(0xffffffffu, xs, 1);  // of the lanes behind, in front
        xp = __shfl_up_sync(0xffffffffu, xp, 1);
        if (lane == 31) xs = 0.f;
        if (lane == 0) xp = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = c * T + 4 * lane + i;
            const float da = th + (suf[i] + xs) + (pre[i] + xp), g = fmaf(A, da, (vo[i] + dg[i]) + vi[i]) * sl[i];
            if (t < len) {
                static_cast<__nv_bfloat16 *>(a.ddt.p)[(size_t)b * a.ddt.sb + (size_t)h * a.ddt.sh + (size_t)t * a.ddt.st] = __float2bfloat16_rn(g);
                sA = fmaf(da, dt[i], sA);
                sb += g;
            }
        }
        if (lane == 0) sD += dd[at];
    }
    sA = lanes_sum(sA);
    sb = lanes_sum(sb);
    if (lane == 0) {
        part[0][warp] = sA;
        part[1][warp] = sD;
        part[2][warp] = sb;
    }
    __syncthreads();
    if (threadIdx.x < 3) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kFinishWarps; ++i) s += part[threadIdx.x][i];
        a.sums[((size_t)b * p.plan.pieces + piece) * 3 * a.H + threadIdx.x * a.H + h] = s;
    }
}

template <int NB>
cudaError_t launch(const StatesParams &sp, const GradParams &g, cudaStream_t st) {
    using S = LayStates<NB>;
    using L = LayGrad<NB>;
    static_assert(S::SMEM <= 227 * 1024 && L::SMEM <= 227 * 1024, "shared memory");
    const Args &a = sp.p.a;
    cudaError_t e = starts<NB>(sp.p, 2, st);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(ssm_states_kernel<NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(ssm_grad_tc_kernel<NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM);
    if (e != cudaSuccess) return e;
    ssm_states_kernel<NB><<<(unsigned)((size_t)a.B * a.H * sp.p.plan.PT * sp.p.plan.pieces), kStatesThreads, S::SMEM, st>>>(sp);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    ssm_grad_tc_kernel<NB><<<(unsigned)((size_t)a.B * a.nc * a.G * g.splits), kGradThreads, L::SMEM, st>>>(g);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    ssm_finish_kernel<<<(unsigned)((size_t)a.B * a.H * sp.p.plan.pieces), kFinishWarps * 32, 0, st>>>(sp, g.own, g.dd);
    return cudaGetLastError();
}

}  // namespace

// CTAs that share a group's heads: as few as fill the device, in rounds of SMs as short as can be.
int tc_splits(const Args &a) {
    const long long ctas = (long long)a.B * a.G * a.nc;
    const int PT = (a.P + 63) / 64;
    long long best = -1;
    int splits = 1;
    for (int s = 1; s <= a.R && s <= 16; ++s) {
        const long long rounds = (ctas * s + kSms - 1) / kSms, cost = rounds * ((long long)(a.R + s - 1) / s * PT + 3);
        if (best < 0 || cost < best) {
            best = cost;
            splits = s;
        }
    }
    return splits;
}

cudaError_t tc_backward(const Args &a, cudaStream_t st) {
    StatesParams sp;
    GradParams g;
    memset(&sp, 0, sizeof sp);
    memset(&g, 0, sizeof g);
    Params &p = sp.p;
    p.a = a;
    cudaError_t e = dev_status_ptr(&p.a.err);
    if (e != cudaSuccess) return e;
    p.plan = plan_of(a, true);
    p.vx[0] = a.x; p.vx[1] = a.dy;
    p.vb[0] = a.b; p.vb[1] = a.c;
    p.pieces[0] = a.h; p.pieces[1] = a.g;
    p.factor = a.factor;
    p.dec = static_cast<const Dec *>(a.dec);
    sp.image[0] = a.image[0]; sp.image[1] = a.image[1];
    sp.inter = a.inter;
    sp.aside = reinterpret_cast<float4 *>(a.aside);
    sp.dots = a.dots;
    g.a = p.a;
    g.PT = p.plan.PT;
    g.splits = a.splits;
    g.vx = a.x; g.vdy = a.dy; g.vb = a.b; g.vc = a.c;
    g.dec = p.dec;
    g.h = a.image[0]; g.g = a.image[1];
    g.own = a.own;
    g.dd = a.dd;
    if (!encode(&p.mx[0], a.x, a.P, a.n, a.H, a.B, T) || !encode(&p.mx[1], a.dy, a.P, a.n, a.H, a.B, T) ||
        !encode(&p.mb[0], a.b, a.N, a.n, a.G, a.B, T) || !encode(&p.mb[1], a.c, a.N, a.n, a.G, a.B, T) ||
        !encode(&g.mdx, a.dx, a.P, a.n, a.H, a.B, T))
        return cudaErrorNotSupported;
    g.mx = p.mx[0]; g.mdy = p.mx[1]; g.mb = p.mb[0]; g.mc = p.mb[1];
    e = a.N <= 64 ? launch<1>(sp, g, st) : launch<2>(sp, g, st);
    if (e == cudaSuccess && a.splits > 1) e = join_parts(a, HLA_BF16, st);
    return e == cudaSuccess ? join_sums(a, a.B * p.plan.pieces, st) : e;
}

}  // namespace ssm
}  // namespace hla
