// hla_ssm_carry.cuh -- tensor-core kernels that carry a state along a head's chunks.
//
// A head's chunks are cut into pieces.  sum_kernel forms what a piece adds to the state (one
// accumulator in TMEM over the whole piece: every token weighs by its decay to the piece's end, so
// nothing is rescaled), scan_kernel turns the sums into the states at the pieces' starts, and
// carry_kernel walks each piece's chunks from its start: state' = 2^s_end state + B^T (w X), the
// weighted rows w X in two bf16 parts, so that the state carries fp32 (2^-17 of each term).  Tokens
// are then read twice, states only at the pieces' ends, and no CTA waits for another.
//   Backward the same kernels run from the last chunk to the first on C and dY.
//
// Roles of a CTA (19 warps): 0-15 elementwise, a thread has one row (a token, or a row of the
// state) and a quarter of its columns; 16 MMA; 17 TMA; 18 the chunk's weights.
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
    float *pieces[2];         // [B][H][pieces][N][P]: sums, then start states
    float *factor;            // [B][H][pieces]: decay over a piece
    uint8_t *image[2];        // STATES: [B][H][PT][chunks][hi, lo][NB * 64 rows][64] tile images
};

HLA_DEVICE float *piece_state(const Params &p, int dir, const Piece &w) {
    return p.pieces[dir] + (((size_t)w.b * p.a.H + w.h) * p.plan.pieces + w.piece) * p.a.N * p.a.P;
}
// This thread's 16 columns of row n of an fp32 [N][P] state.
HLA_DEVICE void load_state16(const Args &a, const float *s, int n, int c0, float (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (s && n < a.N && c0 + i < a.P) {
            const float *q = s + (size_t)n * a.P + c0 + i;
            x = make_float4(q[0], q[1], q[2], q[3]);  // (a caller's state may lie on any float)
        }
        v[i] = x.x; v[i + 1] = x.y; v[i + 2] = x.z; v[i + 3] = x.w;
    }
}
HLA_DEVICE void store_state16(const Args &a, float *s, int n, int c0, const float (&v)[16]) {
    if (n >= a.N) return;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (c0 + i < a.P) s[(size_t)n * a.P + c0 + i] = v[i];
}

// ------------------------------------------------------------ sums of pieces
template <int NB>
struct LaySum {
    static constexpr int NS = 3;
    static constexpr int STAGE = kHalf + NB * kHalf;  // X, then B
    static constexpr int OFF_X = 0, OFF_W = NS * STAGE, OFF_DEC = OFF_W + 2 * 2 * kHalf;  // weighted rows: two of (hi, lo)
    static constexpr int OFF_BAR = OFF_DEC + 2 * (int)sizeof(Dec);
    static constexpr int B_FULL = 0, B_EMPTY = B_FULL + NS, B_DF = B_EMPTY + NS, B_DE = B_DF + 2, B_W = B_DE + 2, B_WE = B_W + 2,
                         B_OUT = B_WE + 2, B_FIN = B_OUT + 1, B_RAW = B_FIN + 1, NBAR = B_RAW + 1;
    static constexpr int SMEM = OFF_BAR + NBAR * 8 + 16;
};

template <int NB>
__global__ void __launch_bounds__(kThreads, 1) ssm_sum_kernel(const __grid_constant__ Params p) {
    using L = LaySum<NB>;
    extern __shared__ __align__(1024) uint8_t base[];
    const Args &a = p.a;
    const int dir = gridDim.y == 2 ? blockIdx.y : 0;
    const Piece w = piece_of(a, p.plan, blockIdx.x);
    if (dir ? w.piece == 0 || w.piece >= w.used : w.piece + 1 >= w.used) return;  // no piece starts from it
    const int K = w.hi - w.lo;
    auto chunk = [&](int k) { return dir ? w.lo + k : w.hi - 1 - k; };  // towards larger decays
    Cta<L::NBAR> cta(base, L::OFF_BAR, a.err, [](int i) {
        return (i >= L::B_W && i < L::B_WE) || (i >= L::B_DE && i < L::B_W) ? kElemWarps : i >= L::B_EMPTY && i < L::B_DF ? kElemWarps + 1 : 1;
    });
    const Waits &ws = cta.ws;
    const int warp = cta.warp, lane = threadIdx.x & 31;
    Dec *dec = reinterpret_cast<Dec *>(base + L::OFF_DEC);
    if (warp == kWarpDec) {
        Decay off{0.f, 0.f};
        for (int k = 0; k < K; ++k) {
            Dec &d = dec[k & 1];
            if (k >= 2 && !ws.wait(L::B_DE + (k & 1), (uint32_t)((k >> 1) & 1) ^ 1u)) break;
            fill_dec(a, d, w.b, w.h, chunk(k) * T, w.len, dir == 1, off);
            const Decay end = d.s[T - 1];
            const float lo = off.lo + end.lo, r = rintf(lo);
            off = {off.hi + end.hi + r, lo - r};
            if (lane == 0) mbar_arrive(ws.bar(L::B_DF + (k & 1)));
        }
        if (w.pt == 0 && dir == 0 && lane == 0) p.factor[((size_t)w.b * a.H + w.h) * p.plan.pieces + w.piece] = factor(off);
        if (w.pt == 0 && dir == 1 && lane == 0 && w.piece + 1 == w.used)  // the forward direction leaves this one out
            p.factor[((size_t)w.b * a.H + w.h) * p.plan.pieces + w.piece] = factor(off);
    } else if (warp == kWarpTma) {
        uint32_t raw = 0;
        int k = 0;
        for (; k < K; ++k) {
            const int s = k % L::NS;
            if (k >= L::NS && !ws.wait(L::B_EMPTY + s, (uint32_t)((k / L::NS) & 1) ^ 1u)) break;
            const int t0 = chunk(k) * T;
            const bool clean = w.len - t0 < T;
            const int full = clean ? L::B_RAW : L::B_FULL + s;
            uint8_t *x = base + s * L::STAGE;
            if (lane == 0) {
                mbar_expect_tx(ws.bar(full), L::STAGE);
                load_tile<1>(x, &p.mx[dir], p.vx[dir], ws.bar(full), 64 * w.pt, t0, w.h, w.b);
                load_tile<NB>(x + kHalf, &p.mb[dir], p.vb[dir], ws.bar(full), 0, t0, w.h / a.R, w.b);
            }
            __syncwarp();
            if (clean) {
                if (!ws.wait(L::B_RAW, raw)) break;
                raw ^= 1u;
                clear_rows<1 + NB>(x, w.len - t0);
                if (lane == 0) mbar_arrive(ws.bar(L::B_FULL + s));
            }
        }
        for (int i = max(0, k - L::NS); i < k; ++i) mbar_wait(ws.bar(L::B_FULL + i % L::NS), (uint32_t)(i / L::NS) & 1u, a.err);
        __syncwarp();
    } else if (warp == kWarpMma) {
        const uint32_t tb = uniform(cta.tb), id = make_idesc(T, 64, true, true);
        bool ok = true;
        for (int k = 0; k < K && ok; ++k) {
            const int s = k % L::NS;
            if (!(ok = ws.wait(L::B_FULL + s, (uint32_t)(k / L::NS) & 1u) && ws.wait(L::B_W + (k & 1), (uint32_t)(k >> 1) & 1u))) break;
            tc_fence_after();
            const uint64_t A = mnmajor(base + s * L::STAGE + kHalf), W = mnmajor(base + L::OFF_W + (k & 1) * 2 * kHalf);
            mma_mm64(tb, A, W, id, k > 0);
            mma_mm64(tb, A + kRows64, W + kRows64, id, true);
            mma_mm64(tb, A, W + kBlock, id, true);
            mma_mm64(tb, A + kRows64, W + kBlock + kRows64, id, true);
            umma_commit_warp(ws.bar(L::B_WE + (k & 1)));
            umma_commit_warp(ws.bar(L::B_EMPTY + s));
        }
        if (ok) umma_commit_warp(ws.bar(L::B_OUT));
        umma_commit_warp(ws.bar(L::B_FIN));
        mbar_wait(ws.bar(L::B_FIN), 0u, a.err);
        __syncwarp();
    } else {
        const int q = warp & 3, cq = warp >> 2, row = 32 * q + lane;
        bool ok = true;
        for (int k = 0; k < K; ++k) {
            const int s = k % L::NS, e = k & 1;
            if (!(ok = ws.wait(L::B_DF + e, (uint32_t)(k >> 1) & 1u) && ws.wait(L::B_FULL + s, (uint32_t)(k / L::NS) & 1u))) break;
            if (k >= 2 && !(ok = ws.wait(L::B_WE + e, (uint32_t)((k >> 1) & 1) ^ 1u))) break;
            uint8_t *hi = base + L::OFF_W + e * 2 * kHalf;
            scale_split16(base + s * L::STAGE, hi, hi + kHalf, row, 16 * cq, dec[e].w[row]);
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(ws.bar(L::B_W + e));
                mbar_arrive(ws.bar(L::B_DE + e));
                mbar_arrive(ws.bar(L::B_EMPTY + s));
            }
        }
        if (ok && ws.wait(L::B_OUT, 0u)) {
            tc_fence_after();
            if (q < 2 * NB) {
                float v[16];
                tmem_ld16(cta.tb + ((uint32_t)(32 * q) << 16) + 16 * cq, v);
                tmem_wait_ld();
                store_state16(a, piece_state(p, dir, w), row, 64 * w.pt + 16 * cq, v);
            }
        }
    }
    cta.finish();
}

// Sums to the states that pieces start from, in place: blockIdx.y 0 from the first piece on, 1 from
// the last one back.
static __global__ void __launch_bounds__(256) ssm_piece_scan_kernel(const __grid_constant__ Params p) {
    const Args &a = p.a;
    const int NP = a.N * a.P, blocks = (NP + 255) / 256, e = blockIdx.x % blocks * 256 + threadIdx.x, u = blockIdx.x / blocks;
    if (e >= NP) return;
    const int dir = blockIdx.y, chunks = (clamp_length(a.lengths, u / a.H, a.n) + T - 1) / T;
    const int used = (chunks + p.plan.per - 1) / p.plan.per;
    const float *init = dir ? a.d_state_out : a.state_in;
    float *s = p.pieces[dir] + (size_t)u * p.plan.pieces * NP + e, h = init ? init[(size_t)u * NP + e] : 0.f;
    const float *f = p.factor + (size_t)u * p.plan.pieces;
    constexpr int U = 8;
    for (int i = 0; i < used; i += U) {
        float v[U], g[U];
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (i + k + 1 < used) {  // the last piece of the walk hands on nothing
                const int c = dir ? used - 1 - i - k : i + k;
                v[k] = s[(size_t)c * NP];
                g[k] = f[c];
            }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (i + k >= used) break;
            s[(size_t)(dir ? used - 1 - i - k : i + k) * NP] = h;
            if (i + k + 1 < used) h = fmaf(g[k], h, v[k]);
        }
    }
}

// ------------------------------------------------------------ walk along a piece
template <int NB, bool OUT>
struct LayCarry {
    static constexpr int NR = OUT ? 3 : 2;  // ring of B and C tiles in turn (STATES: one tile a chunk)
    static constexpr int OFF_X = 0, OFF_R = 2 * kHalf, OFF_W = OFF_R + NR * NB * kHalf, OFF_H = OFF_W + 2 * kHalf;
    static constexpr int HB = NB * kHalf / 2;                      // a state's bf16 rows: 64 NB of them
    static constexpr int OFF_Y = OFF_H + (OUT ? NB * kHalf / 2 : 0);  // OUT: y on its way out; STATES: the state's two parts
    static constexpr int OFF_DEC = OFF_Y + (OUT ? kHalf : 2 * HB);
    static constexpr int OFF_BAR = OFF_DEC + 2 * (int)sizeof(Dec);
    static constexpr int B_X = 0, B_XE = 2, B_R = 4, B_RE = B_R + NR, B_DF = B_RE + NR, B_DE = B_DF + 2, B_W = B_DE + 2, B_D = B_W + 1,
                         B_CB = B_D + 1, B_M = B_CB + 1, B_A1 = B_M + 1, B_A2 = B_A1 + 1, B_H = B_A2 + 1, B_FIN = B_H + 1,
                         B_RAW = B_FIN + 1, NBAR = B_RAW + 1;
    static constexpr int SMEM = OFF_BAR + NBAR * 8 + 16;
    static constexpr uint32_t CB = 0, M = T, D = T + 64, A1 = 2 * T, A2 = 2 * T + 64;  // TMEM columns (A2 twice)
};

template <int NB, bool OUT>
__device__ __forceinline__ void carry_elem(const Params &p, const Waits &ws, uint8_t *base, uint32_t tb, const Piece &w, int dir, int K) {
    using L = LayCarry<NB, OUT>;
    const Args &a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = warp & 3, cq = warp >> 2, row = 32 * q + lane;
    const uint32_t lanes = tb + ((uint32_t)(32 * q) << 16);
    const Dec *dec = reinterpret_cast<const Dec *>(base + L::OFF_DEC);
    const int col = 64 * w.pt + 16 * cq;
    const bool holds = q < 2 * NB;  // rows of the state
    float carry[16];
    {
        const size_t unit = ((size_t)w.b * a.H + w.h) * a.N * a.P;
        const float *init = dir ? a.d_state_out : a.state_in;
        load_state16(a, p.plan.pieces > 1 && w.used > 0 ? piece_state(p, dir, w) : init ? init + unit : nullptr, row, col, carry);
    }
    auto put_state = [&]() {  // OUT: the state, for C h
        if (holds) tile_store_row16(base + L::OFF_H, 64 * NB, row, 16 * cq, carry);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(ws.bar(L::B_H));
    };
    const float skip = OUT && a.D ? a.D[w.h] : 0.f;
    bool ok = true;
    if (OUT && K > 0) put_state();
    for (int k = 0; k < K; ++k) {
        const int e = k & 1, c = dir ? w.hi - 1 - k : w.lo + k;
        const uint32_t ph = (uint32_t)k & 1u, ph2 = (uint32_t)(k >> 1) & 1u;
        const Dec &d = dec[e];
        if constexpr (!OUT) {  // the state before (the gradient behind) this chunk
            if (threadIdx.x == 0) bulk_wait_read();
            elem_sync();
            if (holds) {
                uint8_t *im = base + L::OFF_Y;
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    uint4 h, l;
                    split2(carry[8 * g], carry[8 * g + 1], h.x, l.x);
                    split2(carry[8 * g + 2], carry[8 * g + 3], h.y, l.y);
                    split2(carry[8 * g + 4], carry[8 * g + 5], h.z, l.z);
                    split2(carry[8 * g + 6], carry[8 * g + 7], h.w, l.w);
                    const uint32_t off = tile_off(64 * NB, row, 16 * cq + 8 * g);
                    *reinterpret_cast<uint4 *>(im + off) = h;
                    *reinterpret_cast<uint4 *>(im + L::HB + off) = l;
                }
            }
            fence_async_smem();
            elem_sync();
            if (threadIdx.x == 0) {
                const size_t at = (((size_t)w.b * a.H + w.h) * p.plan.PT + w.pt) * a.nc + c;
                bulk_store(p.image[dir] + at * 2 * L::HB, base + L::OFF_Y, 2 * L::HB);
                bulk_commit();
            }
        }
        // after an expired wait the loop goes on, so that the barriers above and below stay matched
        ok = ok && ws.wait(L::B_DF + e, ph2) && ws.wait(L::B_X + e, ph2);
        const uint8_t *x = base + L::OFF_X + e * kHalf;
        if (ok) scale_split16(x, base + L::OFF_W, base + L::OFF_W + kHalf, row, 16 * cq, d.w[row]);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(ws.bar(L::B_W));
        if constexpr (OUT) {  // M = (C B^T) o L diag(dt), bf16, over 32 columns
            ok = ok && ws.wait(L::B_CB, ph);
            tc_fence_after();
            float pk[16];
            if (cq > q || !ok) {
#pragma unroll
                for (int i = 0; i < 16; ++i) pk[i] = 0.f;
            } else {
                float v[32];
                tmem_ld32(lanes + L::CB + 32 * cq, v);
                const Decay s = d.s[row];
                if (cq < q) {
                    const float u = factor(s, d.s[32 * cq + 31]);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        const float4 f = *reinterpret_cast<const float4 *>(d.v + 32 * cq + i);
                        pk[i / 2] = __uint_as_float(pack_bf16(v[i] * (u * f.x), v[i + 1] * (u * f.y)));
                        pk[i / 2 + 1] = __uint_as_float(pack_bf16(v[i + 2] * (u * f.z), v[i + 3] * (u * f.w)));
                    }
                } else {
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const float f = v[i] * (factor(s, d.s[32 * cq + i]) * d.dt[32 * cq + i]);
                        v[i] = i <= lane ? f : 0.f;
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) pk[i] = __uint_as_float(pack_bf16(v[2 * i], v[2 * i + 1]));
                }
            }
            tmem_st16(lanes + L::M + 16 * cq, pk);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(ws.bar(L::B_M));
        }
        // the state behind the chunk
        ok = ok && ws.wait(L::B_D, ph);
        tc_fence_after();
        if (holds && ok) {
            float v[16];
            tmem_ld16(lanes + L::D + 16 * cq, v);
            tmem_wait_ld();
            const float f = d.end;
#pragma unroll
            for (int i = 0; i < 16; ++i) carry[i] = fmaf(f, carry[i], v[i]);
        }
        if constexpr (OUT) {
            ok = ok && ws.wait(L::B_A2, ph);
            if (k + 1 < K) put_state();
            ok = ok && ws.wait(L::B_A1, ph);
            tc_fence_after();
            float y[16], z[16], xr[16];
            tmem_ld16(lanes + L::A1 + 16 * cq, y);
            tmem_ld16(lanes + L::A2 + 64 * e + 16 * cq, z);
            unpack8(*reinterpret_cast<const uint4 *>(x + tile_off(T, row, 16 * cq)), xr);
            unpack8(*reinterpret_cast<const uint4 *>(x + tile_off(T, row, 16 * cq + 8)), xr + 8);
            tmem_wait_ld();
            const float to = d.to[row];
#pragma unroll
            for (int i = 0; i < 16; ++i) y[i] = fmaf(skip, xr[i], fmaf(to, z[i], y[i]));
            const int t0 = c * T;
            if (threadIdx.x == 0) bulk_wait_read();
            elem_sync();
            tile_store_row16(base + L::OFF_Y, T, row, 16 * cq, y);
            fence_async_smem();
            elem_sync();
            if (ok && w.len - t0 >= T) {
                if (threadIdx.x == 0) {
                    tma_store_4d(base + L::OFF_Y, &p.my, 64 * w.pt, t0, a.y.sh ? w.h : 0, a.y.sb ? w.b : 0);
                    bulk_commit();
                }
            } else if (ok) {  // rows behind the sequence stay as they are
                __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.y.p) + (size_t)w.b * a.y.sb + (size_t)w.h * a.y.sh;
                for (int i = threadIdx.x; i < T * 8; i += kElemWarps * 32) {
                    const int r = i >> 3, cc = 64 * w.pt + 8 * (i & 7);
                    if (t0 + r < w.len && cc < a.P)
                        *reinterpret_cast<uint4 *>(out + (size_t)(t0 + r) * a.y.st + cc) =
                            *reinterpret_cast<const uint4 *>(base + L::OFF_Y + tile_off(T, r, 8 * (i & 7)));
                }
            }
            tc_fence_before();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(ws.bar(L::B_XE + e));
            mbar_arrive(ws.bar(L::B_DE + e));
        }
    }
    const int last = dir ? 0 : max(w.used - 1, 0);
    float *fin = dir ? a.d_state_in : a.state_out;
    if (ok && fin && w.piece == last && holds) store_state16(a, fin + ((size_t)w.b * a.H + w.h) * a.N * a.P, row, col, carry);
    if (threadIdx.x == 0) bulk_wait_all();
}

template <int NB, bool OUT>
__device__ __forceinline__ void carry_mma(const Params &p, const Waits &ws, uint8_t *base, uint32_t tb, int K) {
    using L = LayCarry<NB, OUT>;
    const uint32_t id_d = make_idesc(T, 64, true, true), id_cb = make_idesc(T, T, false, false), id_y = make_idesc(T, 64, false, true);
    const uint64_t W = mnmajor(base + L::OFF_W), H = make_sdesc(smem_u32(base + L::OFF_H), 64 * NB * 128u, 1024u);
    constexpr int EACH = OUT ? 2 : 1;  // ring tiles of a chunk
    auto slot = [](int i) { return i % L::NR; };
    auto full = [&](int i) { return ws.wait(L::B_R + slot(i), (uint32_t)(i / L::NR) & 1u); };
    auto tile = [&](int i) { return base + L::OFF_R + slot(i) * NB * kHalf; };
    auto do_cb = [&](int k) {
        if (!full(2 * k) || !full(2 * k + 1)) return false;
        const uint64_t b = kmajor(tile(2 * k)), c = kmajor(tile(2 * k + 1));
        mma_ss64(tb + L::CB, c, b, id_cb, false);
        if (NB > 1) mma_ss64(tb + L::CB, c + kBlock, b + kBlock, id_cb, true);
        umma_commit_warp(ws.bar(L::B_CB));
        return true;
    };
    bool ok = !OUT || K == 0 || do_cb(0);
    for (int k = 0; k < K && ok; ++k) {
        const int e = k & 1;
        const uint32_t ph = (uint32_t)k & 1u;
        if constexpr (OUT) {
            if (!(ok = ws.wait(L::B_H, ph))) break;
            tc_fence_after();
            const uint64_t c = kmajor(tile(2 * k + 1));
            mma_km64(tb + L::A2 + 64 * e, c, H, id_y, false);
            if (NB > 1) mma_km64(tb + L::A2 + 64 * e, c + kBlock, H + kRows64, id_y, true);
            umma_commit_warp(ws.bar(L::B_A2));
            umma_commit_warp(ws.bar(L::B_RE + slot(2 * k + 1)));
        }
        if (!(ok = full(EACH * k) && ws.wait(L::B_W, ph))) break;
        tc_fence_after();
        const uint64_t b = mnmajor(tile(EACH * k));
        mma_mm64(tb + L::D, b, W, id_d, false);
        mma_mm64(tb + L::D, b + kRows64, W + kRows64, id_d, true);
        mma_mm64(tb + L::D, b, W + kBlock, id_d, true);
        mma_mm64(tb + L::D, b + kRows64, W + kBlock + kRows64, id_d, true);
        umma_commit_warp(ws.bar(L::B_D));
        umma_commit_warp(ws.bar(L::B_RE + slot(EACH * k)));
        if constexpr (OUT) {
            if (!(ok = ws.wait(L::B_X + e, (uint32_t)(k >> 1) & 1u) && ws.wait(L::B_M, ph))) break;
            tc_fence_after();
            mma_ts128(tb + L::A1, tb + L::M, mnmajor(base + L::OFF_X + e * kHalf), id_y);
            umma_commit_warp(ws.bar(L::B_A1));
            umma_commit_warp(ws.bar(L::B_XE + e));
            if (k + 1 < K) ok = do_cb(k + 1);
        }
    }
    umma_commit_warp(ws.bar(L::B_FIN));  // every MMA issued completes before TMEM is released
    mbar_wait(ws.bar(L::B_FIN), 0u, ws.err);
    __syncwarp();
}

template <int NB, bool OUT>
__device__ __forceinline__ void carry_tma(const Params &p, const Waits &ws, uint8_t *base, const Piece &w, int dir, int K) {
    using L = LayCarry<NB, OUT>;
    const Args &a = p.a;
    const int lane = threadIdx.x & 31;
    constexpr int EACH = OUT ? 2 : 1;
    uint32_t raw = 0;
    int k = 0, issued = 0;  // ring tiles
    bool ok = true;
    for (; k < K; ++k) {
        const int e = k & 1, t0 = (dir ? w.hi - 1 - k : w.lo + k) * T;
        const bool clean = w.len - t0 < T;
        if (k >= 2 && !ws.wait(L::B_XE + e, (uint32_t)((k >> 1) & 1) ^ 1u)) break;
        uint8_t *x = base + L::OFF_X + e * kHalf;
        auto load = [&](uint8_t *dst, int bar, bool clear, uint32_t bytes, auto issue) {
            const int full = clear ? L::B_RAW : bar;
            if (lane == 0) {
                mbar_expect_tx(ws.bar(full), bytes);
                issue(full);
            }
            __syncwarp();
            if (!clear) return true;
            if (!ws.wait(L::B_RAW, raw)) return false;
            raw ^= 1u;
            if (bytes == kHalf)
                clear_rows<1>(dst, w.len - t0);
            else
                clear_rows<NB>(dst, w.len - t0);
            if (lane == 0) mbar_arrive(ws.bar(bar));
            return true;
        };
        if (!(ok = load(x, L::B_X + e, clean, kHalf, [&](int f) { load_tile<1>(x, &p.mx[dir], p.vx[dir], ws.bar(f), 64 * w.pt, t0, w.h, w.b); }))) {
            ++k;
            break;
        }
        for (int i = 0; i < EACH && ok; ++i) {
            const int s = issued % L::NR;
            if (issued >= L::NR && !(ok = ws.wait(L::B_RE + s, (uint32_t)((issued / L::NR) & 1) ^ 1u))) break;
            uint8_t *r = base + L::OFF_R + s * NB * kHalf;
            ++issued;
            ok = load(r, L::B_R + s, clean && i == 0, NB * kHalf, [&](int f) {
                load_tile<NB>(r, i ? &p.mc : &p.mb[dir], i ? a.c : p.vb[dir], ws.bar(f), 0, t0, w.h / a.R, w.b);
            });
        }
        if (!ok) {
            ++k;
            break;
        }
    }
    // nothing may land after the CTA has ended (only an aborted CTA still has copies in flight)
    if (ok) {
        for (int i = max(0, k - 2); i < k; ++i) mbar_wait(ws.bar(L::B_X + (i & 1)), (uint32_t)(i >> 1) & 1u, a.err);
        for (int i = max(0, issued - L::NR); i < issued; ++i) mbar_wait(ws.bar(L::B_R + i % L::NR), (uint32_t)(i / L::NR) & 1u, a.err);
    }
    __syncwarp();
}

template <int NB, bool OUT>
__global__ void __launch_bounds__(kThreads, 1) ssm_carry_kernel(const __grid_constant__ Params p) {
    using L = LayCarry<NB, OUT>;
    extern __shared__ __align__(1024) uint8_t base[];
    const Args &a = p.a;
    const int dir = OUT ? 0 : blockIdx.y;
    const Piece w = piece_of(a, p.plan, blockIdx.x);
    if (w.piece >= max(w.used, 1)) return;
    const int K = w.hi - w.lo;
    Cta<L::NBAR> cta(base, L::OFF_BAR, a.err, [](int i) {
        return (i >= L::B_DE && i <= L::B_W) || i == L::B_M || i == L::B_H ? kElemWarps
               : i == L::B_XE || i == L::B_XE + 1                           ? kElemWarps + (OUT ? 1 : 0)
                                                                            : 1;
    });
    if (cta.warp == kWarpDec) {
        Dec *dec = reinterpret_cast<Dec *>(base + L::OFF_DEC);
        for (int k = 0; k < K; ++k) {
            if (k >= 2 && !cta.ws.wait(L::B_DE + (k & 1), (uint32_t)((k >> 1) & 1) ^ 1u)) break;
            fill_dec(a, dec[k & 1], w.b, w.h, (dir ? w.hi - 1 - k : w.lo + k) * T, w.len, dir == 1, {0.f, 0.f});
            if ((threadIdx.x & 31) == 0) mbar_arrive(cta.ws.bar(L::B_DF + (k & 1)));
        }
    } else if (cta.warp == kWarpTma) {
        carry_tma<NB, OUT>(p, cta.ws, base, w, dir, K);
    } else if (cta.warp == kWarpMma) {
        carry_mma<NB, OUT>(p, cta.ws, base, uniform(cta.tb), K);
    } else {
        carry_elem<NB, OUT>(p, cta.ws, base, cta.tb, w, dir, K);
    }
    cta.finish();
}

}  // namespace tcs
}  // namespace ssm
}  // namespace hla
