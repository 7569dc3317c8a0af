// hla_ssm_tc.cuh -- what the tensor-core kernels of the selective state space scan share (bf16,
// chunks of 128 tokens, 64 columns of a head at a time; formulas in hla_ssm.h).
#pragma once
#include <cstddef>

#include "hla_ssm.h"
#include "hla_window_tc.cuh"

namespace hla {
namespace ssm {
namespace tcs {

using win::tcw::encode;
using win::tcw::kmajor;
using win::tcw::low_bits;
using win::tcw::mappable;
using win::tcw::mbar_arrive;
using win::tcw::mma_ss64;
using win::tcw::mma_ts32;
using win::tcw::mnmajor;
using win::tcw::tma_load_4d;
using win::tcw::uniform;

constexpr int kSms = 152;            // pieces are cut for these (results then do not depend on the device)
constexpr int T = 128;               // tokens of a chunk
constexpr int kHalf = T * 128;       // bytes of 128 rows of 64 bf16 columns
constexpr int kElemWarps = 16, kWarpMma = 16, kWarpTma = 17, kWarpTmaX = 18;

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
// D += A B over 64 columns, A packed bf16 in four times 8 columns of TMEM, STEP apart, B K-major.
template <int STEP>
HLA_DEVICE void mma_tk64(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc) {
    asm volatile(
        "{\n .reg .pred e, t;\n .reg .b64 b1, b2, b3;\n .reg .b32 a1, a2, a3;\n elect.sync _|e, 0xffffffff;\n"
        " setp.eq.b32 t, 0, 0;\n add.s64 b1, %2, 2;\n add.s64 b2, %2, 4;\n add.s64 b3, %2, 6;\n"
        " add.u32 a1, %1, %4;\n add.u32 a2, %1, %5;\n add.u32 a3, %1, %6;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, t;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, t;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, t;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "n"(STEP), "n"(2 * STEP), "n"(3 * STEP)
        : "memory");
}
HLA_DEVICE void quad_sync(int q) { asm volatile("bar.sync %0, 128;" ::"r"(1 + q) : "memory"); }  // the four warps of 32 rows
constexpr uint32_t kBlock = kHalf >> 4, kRows64 = 64 * 128 >> 4;  // descriptor steps: 64 columns, 64 rows

HLA_DEVICE void tmem_st8(uint32_t taddr, const float (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(__float_as_uint(v[0])),
                 "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])),
                 "r"(__float_as_uint(v[5])), "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7]))
                 : "memory");
}
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
// Bounded, warp-uniform waits as win::tcw::Waits, what follows a first poll out of line: these
// kernels' roles go through long code once per chunk, and what does not fit the instruction cache
// stalls every warp (101 KB of it: 4,500 to 7,000 cycles a chunk).
static __device__ __noinline__ bool wait_on(uint64_t *bar, uint32_t parity, volatile int *abort_p, unsigned *err) {
    for (int polls = 0; !*abort_p; ++polls) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        if (polls == 2000) {
            atomicOr(err, DEV_TIMEOUT);
            *abort_p = 1;
        }
        __syncwarp();
    }
    return false;
}
struct Waits {
    uint64_t *bars;
    volatile int *abort_p;
    unsigned *err;
    HLA_DEVICE uint64_t *bar(int i) const { return bars + i; }
    HLA_DEVICE bool wait(int b, uint32_t parity) const {
        return __all_sync(0xffffffffu, mbar_try_wait(bars + b, parity)) || wait_on(bars + b, parity, abort_p, err);
    }
};

// BLOCKS x 64 columns from column c0 on, rows t0 .. t0 + 127 of head h.
template <int BLOCKS>
HLA_DEVICE void load_tile(uint8_t *dst, const CUtensorMap *m, const View &v, uint64_t *bar, int c0, int t0, int h, int b) {
#pragma unroll
    for (int c = 0; c < BLOCKS; ++c) tma_load_4d(dst + c * kHalf, m, bar, c0 + 64 * c, t0, v.sh ? h : 0, v.sb ? b : 0);
}
// Zeroes rows [r0, T) of a tile (one warp): rows behind a sequence may be anything, and 0 times
// that is not 0 where they are contracted over.
HLA_DEVICE void clear_rows(uint8_t *tile, int blocks, int r0) {
#pragma unroll 1
    for (int c = 0; c < blocks; ++c)
#pragma unroll 1
        for (int e = (r0 << 3) + (int)(threadIdx.x & 31); e < T * 8; e += 32)
            reinterpret_cast<uint4 *>(tile + c * kHalf)[e] = make_uint4(0, 0, 0, 0);
    fence_async_smem();
    __syncwarp();
}
HLA_DEVICE uint32_t pack2(float2 v) { return pack_bf16(v.x, v.y); }
HLA_DEVICE float2 unpack2(uint32_t w) { return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)); }
HLA_DEVICE void unpack8(const uint4 u, float2 *v) {
    v[0] = unpack2(u.x); v[1] = unpack2(u.y); v[2] = unpack2(u.z); v[3] = unpack2(u.w);
}
// v as three bf16 parts, whose sum is v to the last bit (above 2^-110): the first one rounded where
// it is of use alone, each other cut off, which is a byte permutation where rounding converts.
HLA_DEVICE uint32_t cut2(float2 v) { return __byte_perm(__float_as_uint(v.x), __float_as_uint(v.y), 0x7632); }
HLA_DEVICE float2 less(float2 v, uint32_t part) { return fma2(unpack2(part), both(-1.f), v); }
template <bool ROUND>
HLA_DEVICE void split3(float2 v, uint32_t &hi, uint32_t &mid, uint32_t &lo) {
    hi = ROUND ? pack2(v) : cut2(v);
    v = less(v, hi);
    mid = cut2(v);
    lo = cut2(less(v, mid));
}
// 8 columns (c0 a multiple of 8) of row r of a 64-column tile with `rows` rows, its parts `step` bytes apart.
template <bool ROUND>
HLA_DEVICE void store_split8(uint8_t *tile, int step, int rows, int r, int c0, const float2 *v) {
    uint4 h, m, l;
    split3<ROUND>(v[0], h.x, m.x, l.x);
    split3<ROUND>(v[1], h.y, m.y, l.y);
    split3<ROUND>(v[2], h.z, m.z, l.z);
    split3<ROUND>(v[3], h.w, m.w, l.w);
    uint8_t *at = tile + tile_off(rows, r, c0);
    *reinterpret_cast<uint4 *>(at) = h;
    *reinterpret_cast<uint4 *>(at + step) = m;
    *reinterpret_cast<uint4 *>(at + 2 * step) = l;
}
HLA_DEVICE void store_row8(uint8_t *tile, int rows, int r, int c0, const float2 *v) {
    *reinterpret_cast<uint4 *>(tile + tile_off(rows, r, c0)) = make_uint4(pack2(v[0]), pack2(v[1]), pack2(v[2]), pack2(v[3]));
}
// 16 columns of row r of a bf16 tile times f, in three parts kHalf bytes apart.
HLA_DEVICE void scale_split16(const uint8_t *tile, uint8_t *to, int r, int c0, float f) {
    const uint4 u0 = *reinterpret_cast<const uint4 *>(tile + tile_off(T, r, c0));
    const uint4 u1 = *reinterpret_cast<const uint4 *>(tile + tile_off(T, r, c0 + 8));
    float2 v[8];
    unpack8(u0, v);
    unpack8(u1, v + 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = mul2(v[i], both(f));
    store_split8<false>(to, kHalf, T, r, c0, v);
    store_split8<false>(to, kHalf, T, r, c0 + 8, v + 4);
}
// 16 columns of an accumulator in TMEM, as pairs.
HLA_DEVICE void tmem_pairs16(uint32_t taddr, float2 (&v)[8]) { tmem_ld16(taddr, reinterpret_cast<float(&)[16]>(v)); }

// What a chunk's tokens weigh, [B][H][chunks] in the workspace: formed once by weights_kernel (a
// warp's chain of loads, softplus and scan takes longer than the rest of a chunk's work: with a
// warp of each CTA for it, n16384 h64 p64 s128 took 457 us), copied by the TMA unit.
struct Dec {
    Decay s[T];
    float dt[T];
    float to[T];     // 2^s_t: from the chunk's start
    float w[T];      // dt 2^(s_end - s): the token's weight in the state
    float v[T];      // dt 2^(s_r - s), r the last token of its block of 32: M = CB v 2^(s_t - s_r) behind the block
    float end;       // 2^s_end
    float pad[3];
    float range[4];  // log2 of the decay over each block of 32, infinity where some decay of the chunk grows
    // for the gradients only:
    float slope[T];  // of dt over its raw value
    float fw[T];     // 2^(s - s_b), b the first token of its block of 32: L = 2^(s_b - s_j) fw in front of the block
};
constexpr int kDecBytes = offsetof(Dec, slope);  // what the walks take
HLA_DEVICE const Dec *dec_of(const Args &a, const Dec *dec, int b, int h, int c) { return dec + ((size_t)b * a.H + h) * a.nc + c; }

// One CTA for 8 heads of a chunk: their steps through shared memory, whichever of heads and tokens
// lie side by side; then a warp for each head, four adjacent tokens a lane.
constexpr int kWeightHeads = 8;
static __global__ void __launch_bounds__(kWeightHeads * 32, 8) ssm_weights_kernel(const Args a, Dec *dec) {
    constexpr int W = kWeightHeads;
    __shared__ float raw[T][W + 1];
    const int groups = (a.H + W - 1) / W, h0 = blockIdx.x % groups * W, c = blockIdx.x / groups % a.nc, b = blockIdx.x / groups / a.nc;
    const int len = clamp_length(a.lengths, b, a.n), t0 = c * T, heads = min(W, a.H - h0), live = min(T, len - t0);
    if (live <= 0) return;
    const bool by_head = a.dt.sh < a.dt.st;
#pragma unroll
    for (int e = threadIdx.x; e < T * W; e += W * 32) {
        const int t = by_head ? e / W : e & (T - 1), h = by_head ? e % W : e >> 7;
        if (t < live && h < heads) raw[t][h] = raw_step<__nv_bfloat16>(a, b, h0 + h, t0 + t);
    }
    __syncthreads();
    const int lane = threadIdx.x & 31;
    const int i = threadIdx.x >> 5;
    if (i < heads) {
        const int h = h0 + i;
        const float bias = a.softplus && a.dt_bias ? a.dt_bias[h] : 0.f;
        float d[4], sl[4];
        Decay s[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            sl[k] = 0.f;
            d[k] = 4 * lane + k < live ? step_from(a, raw[4 * lane + k][i], bias, sl[k]) : 0.f;
        }
        const float A2 = a.A[h] * kLog2e;
        scan_decays(d, A2, s);
        Dec *o = dec + ((size_t)b * a.H + h) * a.nc + c;
        auto from = [&](int l) { return Decay{__shfl_sync(0xffffffffu, s[3].hi, l), __shfl_sync(0xffffffffu, s[3].lo, l)}; };
        const Decay end = from(31), block = from(lane | 7);
        const Decay first{__shfl_sync(0xffffffffu, s[0].hi, lane & ~7), __shfl_sync(0xffffffffu, s[0].lo, lane & ~7)};
        float4 *q = reinterpret_cast<float4 *>(o->s + 4 * lane);
        q[0] = make_float4(s[0].hi, s[0].lo, s[1].hi, s[1].lo);
        q[1] = make_float4(s[2].hi, s[2].lo, s[3].hi, s[3].lo);
        auto put = [&](float *p, auto f) { *reinterpret_cast<float4 *>(p + 4 * lane) = make_float4(f(0), f(1), f(2), f(3)); };
        put(o->dt, [&](int k) { return d[k]; });
        put(o->to, [&](int k) { return factor(s[k]); });
        put(o->w, [&](int k) { return d[k] * factor(end, s[k]); });
        put(o->v, [&](int k) { return d[k] * factor(block, s[k]); });
        put(o->slope, [&](int k) { return sl[k]; });
        put(o->fw, [&](int k) { return factor(s[k], first); });
        const bool grows = __any_sync(0xffffffffu, fmaxf(fmaxf(d[0] * A2, d[1] * A2), fmaxf(d[2] * A2, d[3] * A2)) > 0.f);
        if (lane % 8 == 0) o->range[lane / 8] = grows ? INFINITY : first.hi - block.hi;
        if (lane == 0) o->end = factor(end);
    }
}
inline cudaError_t weights(const Args &a, Dec *dec, cudaStream_t st) {
    ssm_weights_kernel<<<(unsigned)((size_t)a.B * a.nc * ((a.H + kWeightHeads - 1) / kWeightHeads)), kWeightHeads * 32, 0, st>>>(a, dec);
    return cudaGetLastError();
}

// Work of one CTA: columns [64 pt, 64 pt + 64) of a head's state over the chunks [lo, hi) of one piece.
struct Piece {
    int b, h, pt, piece, len, used, lo, hi;  // used: pieces below the length
};
struct Plan {
    int pieces, per, PT;  // chunks of a piece, column tiles of a head
    int cuts, part;       // parts that a piece's sum is formed in, chunks of one: per = cuts part
    HLA_DEVICE Plan parts() const { return {pieces * cuts, part, PT, 1, part}; }
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
// Pieces, and parts of their sums, so that the rounds of CTAs over the SMs, each as long as a piece,
// are as few chunks in all as can be.  A chunk costs a sum half of what it costs the forward walk (1.3
// against 2.5 us, n16384 h64 p64 s128) and, both directions taken, a quarter of the backward's; a CTA's
// start and end cost it two.  (With sums of whole pieces seven pieces were best there, 239 us.)
inline Plan plan_of(const Args &a, bool backward) {
    Plan p{};
    p.PT = (a.P + 63) / 64;
    const unsigned units = (unsigned)a.B * a.H * p.PT, chunks = ((unsigned)a.n + T - 1) / T;  // (launches of units x chunks fit a grid)
    auto rounds = [](unsigned ctas) { return (ctas + kSms - 1) / kSms; };
    unsigned long long best = ~0ull;
    for (unsigned k = 1; k <= 64 && k <= chunks; ++k)
        for (unsigned cuts = 1; cuts <= 8; ++cuts) {
            const unsigned part = ((chunks + k - 1) / k + cuts - 1) / cuts, per = cuts * part, real = (chunks + per - 1) / per;
            unsigned long long cost = 4ull * rounds(units * real) * (per + 2);
            if (cost >= best) break;  // (more cuts make pieces no shorter)
            if (real > 1) cost += (unsigned long long)rounds(units * (real - 1) * cuts * (backward ? 2 : 1)) * (part + 2) * (backward ? 1 : 2) + 16;
            if (cost < best) {
                best = cost;
                p.pieces = (int)real;
                p.per = (int)per;
                p.cuts = (int)cuts;
                p.part = (int)part;
            }
            if (real == 1) break;  // nothing to sum
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

}  // namespace tcs

}  // namespace ssm
}  // namespace hla
