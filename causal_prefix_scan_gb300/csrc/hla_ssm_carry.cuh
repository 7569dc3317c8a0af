// hla_ssm_carry.cuh -- tensor-core kernels that carry a state along a head's chunks.
//
// A head's chunks are cut into pieces.  sum_kernel forms what a piece, or a part of one, adds to the
// state (one accumulator in TMEM over all its chunks: every token weighs by its decay to their end, so
// nothing is rescaled), scan_kernel turns the sums into the states at their starts, and
// carry_kernel walks each piece's chunks from its start: state' = 2^s_end state + B^T (w X).  Tokens
// are read twice, states only at the pieces' ends, and no CTA waits for another.  Backward the sums
// also run from the last chunk to the first on C and dY.
//
// The weighted rows w X enter as three bf16 parts whose sum is the fp32 product (with two, states
// were 2.4e-6 off): one operand of 192 columns, so that each row of B is read once for all; the
// parts' sums are added when they are read.
//
// Roles of a CTA: 16 elementwise warps, in which a thread has one row (a token, or a row of the
// state) and a quarter of its columns; one MMA warp; TMA warps, one for each stream of tiles.
#pragma once
#include "hla_ssm_tc.cuh"

namespace hla {
namespace ssm {
namespace tcs {

struct Params {
    Args a;
    Plan plan;
    View vx[2], vb[2];        // x and b; backward dy and c
    CUtensorMap mx[2], mb[2], mc, my;
    float *pieces[2];         // [B][H][parts][N][P]: sums, then start states
    float *factor;            // [B][H][parts]: decay over a part
    const Dec *dec;           // [B][H][chunks]
};

HLA_DEVICE float *part_state(const Params &p, int dir, const Piece &w, int part) {
    return p.pieces[dir] + (((size_t)w.b * p.a.H + w.h) * p.plan.pieces * p.plan.cuts + part) * p.a.N * p.a.P;
}
// What a piece starts from: the state before its first part, or the gradient behind its last one.
HLA_DEVICE float *piece_state(const Params &p, int dir, const Piece &w) {
    return part_state(p, dir, w, dir ? (w.hi - 1) / p.plan.part : w.piece * p.plan.cuts);
}
// This thread's 16 columns of row n of an fp32 [N][P] state (which may lie on any float).
HLA_DEVICE void load_state(const Args &a, const float *s, int n, int c0, float2 (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // (widths are multiples of 8)
        const float *q = s + (size_t)n * a.P + c0 + 2 * i;
        v[i] = s && n < a.N && c0 + 2 * i < a.P ? make_float2(q[0], q[1]) : make_float2(0.f, 0.f);
    }
}
HLA_DEVICE void store_state(const Args &a, float *s, int n, int c0, const float2 (&v)[8]) {
    if (n >= a.N) return;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (c0 + 2 * i < a.P) {
            s[(size_t)n * a.P + c0 + 2 * i] = v[i].x;
            s[(size_t)n * a.P + c0 + 2 * i + 1] = v[i].y;
        }
}
// Columns [c, c + 16) of the three parts' sums, added.
HLA_DEVICE void load_parts16(uint32_t taddr, float2 (&v)[8]) {
    float2 m[8], l[8];
    tmem_pairs16(taddr, v);
    tmem_pairs16(taddr + 64, m);
    tmem_pairs16(taddr + 128, l);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = add2(v[i], add2(m[i], l[i]));
}
// D [128 x 192] (+)= B^T (parts) over a chunk's 128 tokens.
HLA_DEVICE void mma_state(uint32_t d, uint64_t b, uint64_t w, bool acc) {
    constexpr uint32_t id = make_idesc(T, 192, true, true);
    mma_mm64(d, b, w, id, acc);
    mma_mm64(d, b + kRows64, w + kRows64, id, true);
}

// Phase of use i of a ring of NS slots.
template <int NS>
HLA_DEVICE uint32_t ring_phase(int i) { return (uint32_t)(i / NS) & 1u; }
// A tile that ends behind the sequence comes by way of barrier `raw` and is cleared there; in an aborted
// CTA too, so that `bar` is all that its last wait for copies in flight has to ask.
HLA_DEVICE bool clear_landed(const Waits &ws, int raw, uint32_t &phase, int bar, uint8_t *tile, int blocks, int rows) {
    const bool ok = ws.wait(raw, phase);
    if (!ok) mbar_wait(ws.bar(raw), phase, ws.err);
    phase ^= 1u;
    clear_rows(tile, blocks, rows);
    if ((threadIdx.x & 31) == 0) mbar_arrive(ws.bar(bar));
    return ok;
}
// The end of a warp that has issued `uses` copies into a ring of NS slots: nothing may land after the
// CTA has ended (only an aborted CTA still has copies in flight).
template <int NS>
HLA_DEVICE void wait_landed(const Waits &ws, int full, int uses) {
    for (int i = max(0, uses - NS); i < uses; ++i) mbar_wait(ws.bar(full + i % NS), ring_phase<NS>(i), ws.err);
    __syncwarp();
}

// ------------------------------------------------------------ sums of pieces
// Shared memory bounds the kernel: a chunk's tiles, weighted parts and products' operands are 190 KB
// in and out of it, 1,500 of the 1,900 cycles that a chunk takes.  (Two heads of a group through one
// CTA share B's tiles, but leave half as many CTAs: n16384 h64 p64 s128 82 us against 74, b2 n8192 h32
// both ways 60 against 39.)
constexpr int kSumThreads = 19 * 32;
template <int NB>
struct LaySum {
    static constexpr int NX = 3, NR = 2;  // stages of X and its weights, of B
    static constexpr int OFF_X = 0, OFF_R = NX * kHalf, OFF_W = OFF_R + NR * NB * kHalf, OFF_DEC = OFF_W + 2 * 3 * kHalf;
    static constexpr int OFF_BAR = OFF_DEC + NX * kDecBytes;
    static constexpr int B_X = 0, B_XE = B_X + NX, B_R = B_XE + NX, B_RE = B_R + NR, B_W = B_RE + NR, B_WE = B_W + 2, B_OUT = B_WE + 2,
                         B_FIN = B_OUT + 1, B_RAW = B_FIN + 1, B_RAWX = B_RAW + 1, NBAR = B_RAWX + 1;
    static constexpr int SMEM = OFF_BAR + NBAR * 8 + 16;
};

template <int NB>
__global__ void __launch_bounds__(kSumThreads, 1) ssm_sum_kernel(const __grid_constant__ Params p) {
    using L = LaySum<NB>;
    extern __shared__ __align__(1024) uint8_t base[];
    const Args &a = p.a;
    const int dir = gridDim.y == 2 ? blockIdx.y : 0;
    const Piece w = piece_of(a, p.plan.parts(), blockIdx.x);
    const int of = w.piece / p.plan.cuts, pieces = (w.used + p.plan.cuts - 1) / p.plan.cuts;
    if (dir ? of == 0 || w.piece >= w.used : of + 1 >= pieces) return;  // no piece starts from it
    const int K = w.hi - w.lo;
    auto chunk = [&](int k) { return dir ? w.lo + k : w.hi - 1 - k; };  // towards larger decays
    Cta<L::NBAR> cta(base, L::OFF_BAR, a.err, [](int i) {
        return (i >= L::B_W && i < L::B_WE) || (i >= L::B_XE && i < L::B_R) ? kElemWarps : 1;
    });
    const Waits &ws = cta.ws;
    const int warp = cta.warp, lane = threadIdx.x & 31;
    if (warp == kWarpTma || warp == kWarpTmaX) {  // B; X and its weights: neither waits for the other's slots
        const bool is_x = warp == kWarpTmaX;
        const int NS = is_x ? L::NX : L::NR, full = is_x ? L::B_X : L::B_R, empty = is_x ? L::B_XE : L::B_RE;
        uint32_t raw = 0;
        int i = 0;
        bool ok = true;
#pragma unroll 1
        for (; i < K && ok; ++i) {
            const int s = i % NS, c = chunk(i), t0 = c * T;
            const bool clear = w.len - t0 < T;
            if (i >= NS && !(ok = ws.wait(empty + s, ((uint32_t)(i / NS) & 1u) ^ 1u))) break;
            uint8_t *t = base + (is_x ? L::OFF_X + s * kHalf : L::OFF_R + s * NB * kHalf);
            if (lane == 0) {
                uint64_t *bar = ws.bar(!clear ? full + s : is_x ? L::B_RAWX : L::B_RAW);
                if (is_x) {
                    mbar_expect_tx(bar, kHalf + kDecBytes);
                    bulk_load(base + L::OFF_DEC + s * kDecBytes, dec_of(a, p.dec, w.b, w.h, c), kDecBytes, bar);
                    load_tile<1>(t, &p.mx[dir], p.vx[dir], bar, 64 * w.pt, t0, w.h, w.b);
                } else {
                    mbar_expect_tx(bar, NB * kHalf);
                    load_tile<NB>(t, &p.mb[dir], p.vb[dir], bar, 0, t0, w.h / a.R, w.b);
                }
            }
            __syncwarp();
            if (clear) ok = clear_landed(ws, is_x ? L::B_RAWX : L::B_RAW, raw, full + s, t, is_x ? 1 : NB, w.len - t0);
        }
        is_x ? wait_landed<L::NX>(ws, full, i) : wait_landed<L::NR>(ws, full, i);
    } else if (warp == kWarpMma) {
        const uint32_t tb = uniform(cta.tb);
        bool ok = true;
        for (int i = 0; i < K && ok; ++i) {
            const int rs = i % L::NR;
            if (!(ok = ws.wait(L::B_R + rs, ring_phase<L::NR>(i)) && ws.wait(L::B_W + (i & 1), (uint32_t)(i >> 1) & 1u))) break;
            tc_fence_after();
            mma_state(tb, mnmajor(base + L::OFF_R + rs * NB * kHalf), mnmajor(base + L::OFF_W + (i & 1) * 3 * kHalf), i > 0);
            umma_commit_warp(ws.bar(L::B_WE + (i & 1)));
            umma_commit_warp(ws.bar(L::B_RE + rs));
        }
        if (ok) umma_commit_warp(ws.bar(L::B_OUT));
        umma_commit_warp(ws.bar(L::B_FIN));  // every MMA issued completes before TMEM is released
        mbar_wait(ws.bar(L::B_FIN), 0u, a.err);
        __syncwarp();
    } else {
        const int q = warp & 3, cq = warp >> 2, row = 32 * q + lane;
        float off = 1.f;  // decay between the chunk and the piece's end (backward its start)
        bool ok = true;
#pragma unroll 1
        for (int i = 0; i < K; ++i) {
            const int s = i % L::NX, e = i & 1;
            if (!(ok = ws.wait(L::B_X + s, ring_phase<L::NX>(i)))) break;
            if (i >= 2 && !(ok = ws.wait(L::B_WE + e, (uint32_t)((i >> 1) & 1) ^ 1u))) break;
            const Dec &d = *reinterpret_cast<const Dec *>(base + L::OFF_DEC + s * kDecBytes);
            const float f = off * (dir ? d.to[row] : d.w[row]);
            off *= d.end;
            scale_split16(base + L::OFF_X + s * kHalf, base + L::OFF_W + e * 3 * kHalf, row, 16 * cq, f);
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(ws.bar(L::B_W + e));
                mbar_arrive(ws.bar(L::B_XE + s));
            }
        }
        // (backward the parts that the forward sums leave out)
        if (ok && threadIdx.x == 0 && w.pt == 0 && (dir == 0 || of + 1 == pieces)) p.factor[((size_t)w.b * a.H + w.h) * p.plan.pieces * p.plan.cuts + w.piece] = off;
        if (ok && ws.wait(L::B_OUT, 0u)) {
            tc_fence_after();
            if (q < 2 * NB) {
                float2 v[8];
                load_parts16(cta.tb + ((uint32_t)(32 * q) << 16) + 16 * cq, v);
                store_state(a, part_state(p, dir, w, w.piece), row, 64 * w.pt + 16 * cq, v);
            }
        }
    }
    cta.finish();
}

// Sums to the states that parts start from, in place, four elements a thread: blockIdx.y 0 from the
// first part on to the last piece's start, 1 from the last one back to the first piece's end.
static __global__ void __launch_bounds__(256) ssm_piece_scan_kernel(const __grid_constant__ Params p) {
    const Args &a = p.a;
    const int NP = a.N * a.P, blocks = (NP + 1023) / 1024, e = blockIdx.x % blocks * 1024 + 4 * threadIdx.x, u = blockIdx.x / blocks;
    if (e >= NP) return;  // (N and P are multiples of 8)
    const int dir = blockIdx.y, chunks = (clamp_length(a.lengths, u / a.H, a.n) + T - 1) / T;
    const int parts = (chunks + p.plan.part - 1) / p.plan.part, cuts = p.plan.cuts, last = (parts + cuts - 1) / cuts * cuts - cuts;
    const int used = chunks == 0 ? 0 : dir ? max(parts - cuts, 0) + 1 : last + 1;
    const float *init = dir ? a.d_state_out : a.state_in;
    float4 *s = reinterpret_cast<float4 *>(p.pieces[dir] + (size_t)u * p.plan.pieces * cuts * NP + e), h = make_float4(0.f, 0.f, 0.f, 0.f);
    if (init) {  // (on any float)
        init += (size_t)u * NP + e;
        h = make_float4(init[0], init[1], init[2], init[3]);
    }
    const float *f = p.factor + (size_t)u * p.plan.pieces * cuts;
    constexpr int U = 8;
    for (int i = 0; i < used; i += U) {
        float4 v[U];
        float g[U];
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (i + k + 1 < used) {  // the last part of the walk hands on nothing
                const int c = dir ? parts - 1 - i - k : i + k;
                v[k] = s[(size_t)c * (NP / 4)];
                g[k] = f[c];
            }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (i + k >= used) break;
            s[(size_t)(dir ? parts - 1 - i - k : i + k) * (NP / 4)] = h;
            if (i + k + 1 < used) h = make_float4(fmaf(g[k], h.x, v[k].x), fmaf(g[k], h.y, v[k].y), fmaf(g[k], h.z, v[k].z), fmaf(g[k], h.w, v[k].w));
        }
    }
}

// ------------------------------------------------------------ walk along a piece
// The outputs of the forward.  The elementwise warps take a chunk's steps in an order that leaves
// the tensor cores a step's time for each product: M of chunk k; state behind k, and its bf16 rows;
// weighted rows of k + 1; y of k, which leaves by TMA from x's own tile.
// M and the rows of the state that meet C are rounded to bf16 once, since y is (2.0e-3 to 2.3e-3 off, its own
// rounding 1.7e-3): a second part of the state would be another product of 64 columns and 8 NB KB a chunk
// through shared memory, which bounds the walk.  The state itself stays in fp32.
// n16384 h64 p64 s128: 145 us, 128 CTAs.  A chunk moves 400 KB through shared memory (operands of the
// products 208, tiles in and out 96, weighted parts and rows 96), 3,200 of its 4,300 cycles.
constexpr int kCarryThreads = 20 * 32;
// A factor 2^(s_t - s_j) goes in two halves by way of a token r.  With r between j and t neither leaves fp32's
// range while y_t stays in it; inside a block of 32 tokens r lies beyond both: the halves are taken where
// the block's decay is not below 2^-60 and, forward, where none grows (gradients ask for decays in range between
// all tokens, so that the halves are).
constexpr float kBlockRange = 60.f;
template <int NB>
struct LayCarry {
    static constexpr int NX = 3, NR = 3;       // stages of X, ring of C and B tiles in turn
    static constexpr int HB = NB * kHalf / 2;  // a state's bf16 rows: 64 NB of them
    static constexpr int OFF_X = 0, OFF_R = NX * kHalf, OFF_W = OFF_R + NR * NB * kHalf, OFF_H = OFF_W + 3 * kHalf, OFF_DEC = OFF_H + HB;
    static constexpr int OFF_BAR = OFF_DEC + NX * kDecBytes;
    static constexpr int B_X = 0, B_XE = B_X + NX, B_R = B_XE + NX, B_RE = B_R + NR, B_W = B_RE + NR, B_D = B_W + 1, B_A2 = B_D + 1,
                         B_Y = B_A2 + 1, B_CB = B_Y + NX, B_M = B_CB + 1, B_A1 = B_M + 1, B_FIN = B_A1 + 1, B_RAW = B_FIN + 1,
                         B_RAWX = B_RAW + 1, NBAR = B_RAWX + 1;
    static constexpr int SMEM = OFF_BAR + NBAR * 8 + 16;
    static constexpr uint32_t CB = 0, M = 0, A1 = T, A2 = T + 64, D = 2 * T + 64;  // TMEM columns (M over C B^T; A2 twice)
    HLA_DEVICE static int arrivals(int i) { return i == B_W || (i >= B_Y && i < B_CB) || i == B_M ? kElemWarps : 1; }
};

template <int NB>
__device__ __forceinline__ void carry_elem(const Params &p, const Waits &ws, uint8_t *base, uint32_t tb, const Piece &w, int K) {
    using L = LayCarry<NB>;
    const Args &a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = warp & 3, cq = warp >> 2, row = 32 * q + lane, c0 = 16 * cq;
    const uint32_t lanes = tb + ((uint32_t)(32 * q) << 16);
    const int col = 64 * w.pt + c0;
    const bool holds = q < 2 * NB;  // rows of the state
    const float skip = a.D ? a.D[w.h] : 0.f;
    float2 carry[8];
    load_state(a, p.plan.pieces > 1 && w.used > 0 ? piece_state(p, 0, w)
                  : a.state_in                    ? a.state_in + ((size_t)w.b * a.H + w.h) * a.N * a.P
                                                  : nullptr, row, col, carry);
    auto dec = [&](int k) -> const Dec & { return *reinterpret_cast<const Dec *>(base + L::OFF_DEC + k % L::NX * kDecBytes); };
    auto show = [&](int bar) {  // what this warp wrote, to the tensor cores and TMA
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(ws.bar(bar));
    };
    float ahead = 1.f;  // decay over the chunk whose rows were weighted last
    auto prepare = [&](int k) {  // the state before chunk k and its weighted rows
        const int s = k % L::NX;
        if (holds) {
            store_row8(base + L::OFF_H, 64 * NB, row, c0, carry);
            store_row8(base + L::OFF_H, 64 * NB, row, c0 + 8, carry + 4);
        }
        if (!ws.wait(L::B_X + s, ring_phase<L::NX>(k))) return false;
        const Dec &d = dec(k);
        scale_split16(base + L::OFF_X + s * kHalf, base + L::OFF_W, row, c0, d.w[row]);
        ahead = d.end;
        show(L::B_W);
        return true;
    };
    bool ok = K == 0 || prepare(0);
#pragma unroll 1
    for (int k = 0; k < K; ++k) {  // (after an expired wait the loop goes on, so that the quads' barrier stays matched)
        const uint32_t ph = (uint32_t)k & 1u;
        const float end = ahead;
        // M = (C B^T) o L diag(dt), bf16: this thread's 32 columns, nothing above the diagonal
        ok = ok && ws.wait(L::B_CB, ph);
        tc_fence_after();
        float pk[16];
        if (cq <= q && ok) {
            const Dec &d = dec(k);
            const Decay s = d.s[row], last = d.s[32 * cq + 31];
            const bool plain = cq < q || d.range[cq] <= kBlockRange;
            const float2 u = both(plain ? factor(s, last) : 1.f);
            const uint32_t bits = cq < q ? 0xffffffffu : low_bits(lane + 1);  // (behind the diagonal a factor may be anything)
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const int c = 32 * cq + 16 * g;
                float2 v[8];
                tmem_pairs16(lanes + L::CB + c, v);
                tmem_wait_ld();
                if (plain) {  // 2^(s_t - s_j) as 2^(s_t - s_r) 2^(s_r - s_j), r the last token of the columns
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 f = *reinterpret_cast<const float4 *>(d.v + c + 4 * i);
                        v[2 * i] = mul2(v[2 * i], mul2(u, make_float2(f.x, f.y)));
                        v[2 * i + 1] = mul2(v[2 * i + 1], mul2(u, make_float2(f.z, f.w)));
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 sj = *reinterpret_cast<const float4 *>(d.s + c + 2 * i);
                        const float2 dt = *reinterpret_cast<const float2 *>(d.dt + c + 2 * i);
                        v[i] = mul2(v[i], mul2(make_float2(factor(s, {sj.x, sj.y}), factor(s, {sj.z, sj.w})), dt));
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t m = bits >> (16 * g + 2 * i);
                    pk[8 * g + i] = __uint_as_float(pack_bf16(m & 1u ? v[i].x : 0.f, m & 2u ? v[i].y : 0.f));
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) pk[i] = 0.f;
        }
        quad_sync(q);  // every warp of these rows has read what M overwrites
        tc_fence_after();
        tmem_st16(lanes + L::M + 16 * cq, pk);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(ws.bar(L::B_M));
        // the state behind the chunk
        ok = ok && ws.wait(L::B_D, ph);
        tc_fence_after();
        if (holds && ok) {
            float2 x[8];
            load_parts16(lanes + L::D + c0, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) carry[i] = fma2(both(end), carry[i], x[i]);
        }
        tc_fence_before();
        ok = ok && ws.wait(L::B_A2, ph);
        if (k + 1 < K) ok = ok && prepare(k + 1);
        // y = M x + 2^s C h + D x, over x: its weighted rows and M x are done
        ok = ok && ws.wait(L::B_A1, ph);
        tc_fence_after();
        if (ok) {
            const float to = dec(k).to[row];
            uint8_t *x = base + L::OFF_X + k % L::NX * kHalf;
            float2 y[8], c[8], f[8];
            tmem_pairs16(lanes + L::A1 + c0, y);
            tmem_pairs16(lanes + L::A2 + 64 * (k & 1) + c0, c);
            unpack8(*reinterpret_cast<const uint4 *>(x + tile_off(T, row, c0)), f);
            unpack8(*reinterpret_cast<const uint4 *>(x + tile_off(T, row, c0 + 8)), f + 4);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = fma2(both(skip), f[i], fma2(both(to), c[i], y[i]));
            store_row8(x, T, row, c0, y);
            store_row8(x, T, row, c0 + 8, y + 4);
        }
        tc_fence_before();
        show(L::B_Y + k % L::NX);
    }
    if (ok && a.state_out && w.piece == max(w.used - 1, 0) && holds)
        store_state(a, a.state_out + ((size_t)w.b * a.H + w.h) * a.N * a.P, row, col, carry);
}

// In the order in which the elementwise warps ask for them: M x of chunk k and C B^T of k + 1, 2^s C h
// of k + 1, the state's sums over k + 1.
template <int NB>
__device__ __forceinline__ void carry_mma(const Waits &ws, uint8_t *base, uint32_t tb, int K) {
    using L = LayCarry<NB>;
    constexpr uint32_t id_y = make_idesc(T, 64, false, true), id_cb = make_idesc(T, T, false, false);
    const uint64_t H = make_sdesc(smem_u32(base + L::OFF_H), L::HB, 1024u), W = mnmajor(base + L::OFF_W);
    auto full = [&](int i) { return ws.wait(L::B_R + i % L::NR, ring_phase<L::NR>(i)); };
    auto tile = [&](int i) { return base + L::OFF_R + (i % L::NR) * NB * kHalf; };
    auto do_cb = [&](int k) {
        if (!full(2 * k) || !full(2 * k + 1)) return false;
        const uint64_t c = kmajor(tile(2 * k)), b = kmajor(tile(2 * k + 1));
        mma_ss64(tb + L::CB, c, b, id_cb, false);
        if (NB > 1) mma_ss64(tb + L::CB, c + kBlock, b + kBlock, id_cb, true);
        umma_commit_warp(ws.bar(L::B_CB));
        return true;
    };
    bool ok = K == 0 || do_cb(0);
#pragma unroll 1
    for (int k = 0; k < K && ok; ++k) {
        if (!(ok = ws.wait(L::B_W, (uint32_t)k & 1u))) break;
        tc_fence_after();
        const uint64_t c = kmajor(tile(2 * k));
        const uint32_t A2 = tb + L::A2 + 64 * (k & 1);
        mma_km64(A2, c, H, id_y, false);
        if (NB > 1) mma_km64(A2, c + kBlock, H + kRows64, id_y, true);
        umma_commit_warp(ws.bar(L::B_A2));
        umma_commit_warp(ws.bar(L::B_RE + 2 * k % L::NR));
        mma_state(tb + L::D, mnmajor(tile(2 * k + 1)), W, false);
        umma_commit_warp(ws.bar(L::B_D));
        umma_commit_warp(ws.bar(L::B_RE + (2 * k + 1) % L::NR));
        if (!(ok = ws.wait(L::B_X + k % L::NX, ring_phase<L::NX>(k)) && ws.wait(L::B_M, (uint32_t)k & 1u))) break;
        tc_fence_after();
        mma_ts128(tb + L::A1, tb + L::M, mnmajor(base + L::OFF_X + k % L::NX * kHalf), id_y);
        umma_commit_warp(ws.bar(L::B_A1));
        if (k + 1 < K) ok = do_cb(k + 1);
    }
    umma_commit_warp(ws.bar(L::B_FIN));  // every MMA issued completes before TMEM is released
    mbar_wait(ws.bar(L::B_FIN), 0u, ws.err);
    __syncwarp();
}

template <int NB>
__device__ __forceinline__ void carry_load(const Params &p, const Waits &ws, uint8_t *base, const Piece &w, int K) {
    using L = LayCarry<NB>;
    const Args &a = p.a;
    const int lane = threadIdx.x & 31;
    uint32_t raw = 0;
    int r = 0;
    bool ok = true;
#pragma unroll 1
    for (; r < 2 * K && ok; ++r) {
        const int s = r % L::NR, t0 = (w.lo + r / 2) * T;
        const bool is_c = r % 2 == 0, clear = w.len - t0 < T && !is_c;  // rows of C reach their own tokens only
        if (r >= L::NR && !(ok = ws.wait(L::B_RE + s, ring_phase<L::NR>(r) ^ 1u))) break;
        uint8_t *t = base + L::OFF_R + s * NB * kHalf;
        if (lane == 0) {
            uint64_t *bar = ws.bar(clear ? L::B_RAW : L::B_R + s);
            mbar_expect_tx(bar, NB * kHalf);
            load_tile<NB>(t, is_c ? &p.mc : &p.mb[0], is_c ? a.c : p.vb[0], bar, 0, t0, w.h / a.R, w.b);
        }
        __syncwarp();
        if (clear) ok = clear_landed(ws, L::B_RAW, raw, L::B_R + s, t, NB, w.len - t0);
    }
    wait_landed<L::NR>(ws, L::B_R, r);
}

template <int NB>
__device__ __forceinline__ void carry_load_x(const Params &p, const Waits &ws, uint8_t *base, const Piece &w, int K) {
    using L = LayCarry<NB>;
    const Args &a = p.a;
    const int lane = threadIdx.x & 31;
    uint32_t raw = 0;
    int k = 0;
    bool ok = true;
#pragma unroll 1
    for (; k < K && ok; ++k) {
        const int s = k % L::NX, t0 = (w.lo + k) * T;
        const bool clear = w.len - t0 < T;
        if (k >= L::NX && !(ok = ws.wait(L::B_XE + s, ring_phase<L::NX>(k) ^ 1u))) break;
        uint8_t *x = base + L::OFF_X + s * kHalf;
        if (lane == 0) {
            uint64_t *bar = ws.bar(clear ? L::B_RAWX : L::B_X + s);
            mbar_expect_tx(bar, kHalf + kDecBytes);
            bulk_load(base + L::OFF_DEC + s * kDecBytes, dec_of(a, p.dec, w.b, w.h, w.lo + k), kDecBytes, bar);
            load_tile<1>(x, &p.mx[0], p.vx[0], bar, 64 * w.pt, t0, w.h, w.b);
        }
        __syncwarp();
        if (clear) ok = clear_landed(ws, L::B_RAWX, raw, L::B_X + s, x, 1, w.len - t0);
    }
    wait_landed<L::NX>(ws, L::B_X, k);
}

// 128 rows of 64 columns of a head, from a tile in shared memory, by one warp: whole chunks by TMA;
// rows behind the sequence stay as they are.  Returns once the tile may be overwritten.
HLA_DEVICE void store_tile(const uint8_t *tile, const CUtensorMap *m, const View &v, int pt, int t0, int live, int h, int b, int P) {
    const int lane = threadIdx.x & 31;
    if (live >= T) {
        if (lane == 0) {
            tma_store_4d(tile, m, 64 * pt, t0, v.sh ? h : 0, v.sb ? b : 0);
            bulk_commit();
            bulk_wait_read();
        }
    } else {
        __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(v.p) + (size_t)b * v.sb + (size_t)h * v.sh + (size_t)t0 * v.st;
        for (int i = lane; i < live * 8; i += 32) {
            const int r = i >> 3, c = 64 * pt + 8 * (i & 7);
            if (c < P) *reinterpret_cast<uint4 *>(out + (size_t)r * v.st + c) = *reinterpret_cast<const uint4 *>(tile + tile_off(T, r, 8 * (i & 7)));
        }
    }
    __syncwarp();
}

template <int NB>
__device__ __forceinline__ void carry_store(const Params &p, const Waits &ws, uint8_t *base, const Piece &w, int K) {
    using L = LayCarry<NB>;
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int k = 0; k < K; ++k) {
        const int s = k % L::NX, t0 = (w.lo + k) * T;
        if (!ws.wait(L::B_Y + s, ring_phase<L::NX>(k))) break;
        store_tile(base + L::OFF_X + s * kHalf, &p.my, p.a.y, w.pt, t0, w.len - t0, w.h, w.b, p.a.P);
        if (lane == 0) mbar_arrive(ws.bar(L::B_XE + s));
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
}

template <int NB>
__global__ void __launch_bounds__(kCarryThreads, 1) ssm_carry_kernel(const __grid_constant__ Params p) {
    using L = LayCarry<NB>;
    extern __shared__ __align__(1024) uint8_t base[];
    const Piece w = piece_of(p.a, p.plan, blockIdx.x);
    if (w.piece >= max(w.used, 1)) return;
    const int K = w.hi - w.lo;
    Cta<L::NBAR> cta(base, L::OFF_BAR, p.a.err, [](int i) { return L::arrivals(i); });
    if (cta.warp < kElemWarps)
        carry_elem<NB>(p, cta.ws, base, cta.tb, w, K);
    else if (cta.warp == kWarpMma)
        carry_mma<NB>(cta.ws, base, uniform(cta.tb), (int)uniform(K));
    else if (cta.warp == kWarpTma)
        carry_load<NB>(p, cta.ws, base, w, K);
    else if (cta.warp == kWarpTmaX)
        carry_load_x<NB>(p, cta.ws, base, w, K);
    else
        carry_store<NB>(p, cta.ws, base, w, K);
    cta.finish();
}

// The weights of all chunks, then the states that pieces start from (dirs 2: and their gradients).
template <int NB>
cudaError_t starts(const Params &p, int dirs, cudaStream_t st) {
    const Args &a = p.a;
    cudaError_t e = weights(a, const_cast<Dec *>(p.dec), st);
    if (e != cudaSuccess || p.plan.pieces == 1) return e;
    using S = LaySum<NB>;
    static_assert(S::SMEM <= 227 * 1024, "shared memory");
    if ((e = cudaFuncSetAttribute(ssm_sum_kernel<NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM)) != cudaSuccess) return e;
    ssm_sum_kernel<NB><<<dim3((unsigned)((size_t)a.B * a.H * p.plan.PT * p.plan.pieces * p.plan.cuts), dirs), kSumThreads, S::SMEM, st>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    ssm_piece_scan_kernel<<<dim3((unsigned)((size_t)a.B * a.H * ((a.N * a.P + 1023) / 1024)), dirs), 256, 0, st>>>(p);
    return cudaGetLastError();
}
}  // namespace tcs
}  // namespace ssm
}  // namespace hla
