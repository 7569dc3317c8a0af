// hla_ssm_tc.cuh -- what the tensor-core kernels of the selective state space scan share (bf16,
// chunks of 128 tokens, 64 columns of a head at a time; formulas in hla_ssm.h).
#pragma once
#include "hla_ssm.h"
#include "hla_window_tc.cuh"

namespace hla {
namespace ssm {
namespace tcs {

using win::tcw::encode;
using win::tcw::kmajor;
using win::tcw::mappable;
using win::tcw::mbar_arrive;
using win::tcw::mma_ss64;
using win::tcw::mma_ts32;
using win::tcw::mnmajor;
using win::tcw::tma_load_4d;
using win::tcw::tmem_ld32;
using win::tcw::uniform;
using win::tcw::Waits;

constexpr int kSms = 152;            // pieces are cut for these (results then do not depend on the device)
constexpr int T = 128;               // tokens of a chunk
constexpr int kHalf = T * 128;       // bytes of 128 rows of 64 bf16 columns
constexpr int kElemWarps = 16, kWarpMma = 16, kWarpTma = 17, kWarpDec = 18, kThreads = 19 * 32;

// D [128 x N] (+)= A B over 64 rows of both (MN-major tiles).
HLA_DEVICE void mma_mm64(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n .reg .pred p, e, t;\n .reg .b64 a1, a2, a3, b1, b2, b3;\n"
        " elect.sync _|e, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n setp.eq.b32 t, 0, 0;\n"
        " add.s64 a1, %1, 128;\n add.s64 b1, %2, 128;\n add.s64 a2, %1, 256;\n add.s64 b2, %2, 256;\n"
        " add.s64 a3, %1, 384;\n add.s64 b3, %2, 384;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, t;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, t;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u)
        : "memory");
}
// D [128 x N] (+)= A B over 64 columns of A (K-major) and 64 rows of B (MN-major).
HLA_DEVICE void mma_km64(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n .reg .pred p, e, t;\n .reg .b64 a1, a2, a3, b1, b2, b3;\n"
        " elect.sync _|e, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n setp.eq.b32 t, 0, 0;\n"
        " add.s64 a1, %1, 2;\n add.s64 b1, %2, 128;\n add.s64 a2, %1, 4;\n add.s64 b2, %2, 256;\n"
        " add.s64 a3, %1, 6;\n add.s64 b3, %2, 384;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, t;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, t;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u)
        : "memory");
}
// D (+)= A B over 128 rows of B, A packed bf16 in 64 columns of TMEM.
HLA_DEVICE void mma_ts128(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc) {
    mma_ts32(d, a, b, idesc, false);
    mma_ts32(d, a + 16, b + 256, idesc, true);
    mma_ts32(d, a + 32, b + 512, idesc, true);
    mma_ts32(d, a + 48, b + 768, idesc, true);
}
constexpr uint32_t kBlock = kHalf >> 4, kRows64 = 64 * 128 >> 4;  // descriptor steps: 64 columns, 64 rows

HLA_DEVICE void tma_store_4d(const void *src, const void *tmap, int c0, int c1, int c2, int c3) {
    asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(tmap),
                 "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
                 : "memory");
}
HLA_DEVICE void bulk_store(void *dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes) : "memory");
}
HLA_DEVICE void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}
HLA_DEVICE void elem_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kElemWarps * 32) : "memory"); }

// BLOCKS x 64 columns from column c0 on, rows t0 .. t0 + 127 of head h.
template <int BLOCKS>
HLA_DEVICE void load_tile(uint8_t *dst, const CUtensorMap *m, const View &v, uint64_t *bar, int c0, int t0, int h, int b) {
#pragma unroll
    for (int c = 0; c < BLOCKS; ++c) tma_load_4d(dst + c * kHalf, m, bar, c0 + 64 * c, t0, v.sh ? h : 0, v.sb ? b : 0);
}
// Zeroes rows [r0, T) of a tile (one warp): rows behind a sequence may be anything, and 0 times
// that is not 0 where they are contracted over.
template <int BLOCKS>
HLA_DEVICE void clear_rows(uint8_t *tile, int r0) {
#pragma unroll
    for (int c = 0; c < BLOCKS; ++c)
        for (int e = (r0 << 3) + (int)(threadIdx.x & 31); e < T * 8; e += 32)
            reinterpret_cast<uint4 *>(tile + c * kHalf)[e] = make_uint4(0, 0, 0, 0);
    fence_async_smem();
    __syncwarp();
}
HLA_DEVICE void unpack8(const uint4 u, float *v) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
// v as two bf16 parts: hi + lo is v within 2^-17.
HLA_DEVICE void split2(float a, float b, uint32_t &hi, uint32_t &lo) {
    hi = pack_bf16(a, b);
    lo = pack_bf16(a - __uint_as_float(hi << 16), b - __uint_as_float(hi & 0xFFFF0000u));
}
// 16 columns (c0 a multiple of 16) of row r of a 64-column tile, in two parts.
HLA_DEVICE void store_split16(uint8_t *hi, uint8_t *lo, int r, int c0, const float (&v)[16]) {
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        uint4 h, l;
        split2(v[8 * g], v[8 * g + 1], h.x, l.x);
        split2(v[8 * g + 2], v[8 * g + 3], h.y, l.y);
        split2(v[8 * g + 4], v[8 * g + 5], h.z, l.z);
        split2(v[8 * g + 6], v[8 * g + 7], h.w, l.w);
        const uint32_t off = tile_off(T, r, c0 + 8 * g);
        *reinterpret_cast<uint4 *>(hi + off) = h;
        *reinterpret_cast<uint4 *>(lo + off) = l;
    }
}
// The same row of a bf16 tile times f, in two parts.
HLA_DEVICE void scale_split16(const uint8_t *tile, uint8_t *hi, uint8_t *lo, int r, int c0, float f) {
    float v[16];
    unpack8(*reinterpret_cast<const uint4 *>(tile + tile_off(T, r, c0)), v);
    unpack8(*reinterpret_cast<const uint4 *>(tile + tile_off(T, r, c0 + 8)), v + 8);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] *= f;
    store_split16(hi, lo, r, c0, v);
}

// What a chunk's tokens weigh, in shared memory.
struct Dec {
    Decay s[T];
    float dt[T];
    float to[T];     // 2^s_t: from the chunk's start
    float w[T];      // weight of the token's row in the state: dt 2^(s_end - s), or 2^s backward
    float v[T];      // dt 2^(s_r - s), r the last token of its block of 32: M = CB v 2^(s_t - s_r) behind the block
    float end;       // 2^s_end
    float pad[3];
};

// Work of one CTA: columns [64 pt, 64 pt + 64) of a head's state over the chunks [lo, hi) of one piece.
struct Piece {
    int b, h, pt, piece, len, used, lo, hi;  // used: pieces below the length
};
struct Plan {
    int pieces, per, PT;  // chunks of a piece, column tiles of a head
};
HLA_DEVICE Piece piece_of(const Args &a, const Plan &p, unsigned u) {
    Piece r;
    r.pt = u % p.PT;
    r.h = u / p.PT % a.H;
    r.piece = u / p.PT / a.H % p.pieces;
    r.b = u / p.PT / a.H / p.pieces;
    r.len = clamp_length(a.lengths, r.b, a.n);
    const int chunks = (r.len + T - 1) / T;
    r.used = (chunks + p.per - 1) / p.per;
    r.lo = min(r.piece * p.per, chunks);
    r.hi = min(r.lo + p.per, chunks);
    return r;
}
// Pieces so that the rounds of CTAs over the SMs, each as long as a piece, are as few chunks in all
// as can be: more pieces than fill the device once only where they fill it better.
inline Plan plan_of(const Args &a, int sms) {
    Plan p;
    p.PT = (a.P + 63) / 64;
    const long long units = (long long)a.B * a.H * p.PT;
    const int chunks = (int)(((long long)a.n + T - 1) / T);
    long long best = -1;
    p.pieces = 1;
    p.per = chunks;
    for (int k = 1; k <= 64 && k <= chunks; ++k) {
        const int per = (chunks + k - 1) / k, real = (chunks + per - 1) / per;
        const long long rounds = (units * real + sms - 1) / sms;
        const long long cost = rounds * (per + 2) + (real > 1 ? rounds * per / 2 + 4 : 0);  // sums of pieces cost half a chunk each
        if (best < 0 || cost < best) {
            best = cost;
            p.pieces = real;
            p.per = per;
        }
    }
    return p;
}

// Common set-up and end of the kernels: barriers, TMEM, roles.
template <int NB>
struct Cta {
    Waits ws;
    uint32_t tb;
    int warp;
    template <class Count>
    HLA_DEVICE Cta(uint8_t *base, int off_bar, unsigned *err, Count count) {
        ws.bars = reinterpret_cast<uint64_t *>(base + off_bar);
        uint32_t *misc = reinterpret_cast<uint32_t *>(base + off_bar + NB * 8);
        ws.abort_p = reinterpret_cast<volatile int *>(misc + 1);
        ws.err = err;
        warp = threadIdx.x >> 5;
        if (threadIdx.x == 0) {
            misc[1] = 0u;
            for (int i = 0; i < NB; ++i) mbar_init(ws.bar(i), count(i));
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

// The decay warp: one chunk's weights.  `back`: rows weigh by 2^s (towards the chunk's start);
// `off`: decay from the chunk's end to the piece's end (or from the piece's start to the chunk's).
HLA_DEVICE void fill_dec(const Args &a, Dec &d, int b, int h, int t0, int len, bool back, Decay off) {
    const int lane = threadIdx.x & 31;
    chunk_decays<__nv_bfloat16, T / 32>(a, b, h, t0, len, d.dt, d.s, nullptr);
    __syncwarp();
    const Decay end = d.s[T - 1];
#pragma unroll
    for (int i = 0; i < T / 32; ++i) {
        const int t = lane + 32 * i;
        const Decay s = d.s[t];
        const float dt = d.dt[t];
        d.to[t] = factor(s);
        d.w[t] = back ? ex2_approx((s.hi + off.hi) + (s.lo + off.lo))
                      : dt * ex2_approx((end.hi - s.hi + off.hi) + (end.lo - s.lo + off.lo));
        d.v[t] = dt * factor(d.s[32 * i + 31], s);
    }
    if (lane == 0) d.end = factor(end);
    __syncwarp();
}

}  // namespace tcs

}  // namespace ssm
}  // namespace hla
