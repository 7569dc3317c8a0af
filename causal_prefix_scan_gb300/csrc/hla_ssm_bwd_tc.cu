// hla_ssm_bwd_tc.cu -- backward of the selective state space scan for bf16 on the tensor cores
// (formulas in hla_ssm.h).
//
// The walks of hla_ssm_carry.cuh leave, for every chunk and head, the state before it and the
// gradient behind it as pairs of bf16 tile images.  grad_kernel then takes a chunk of one group:
// B, C and C B^T (in registers) stay, the heads pass by 64 columns at a time.  Per head, rows j and
// columns t:
//   X dY^T                       -> M^T, S^T (bf16, with dt_j), sums of E = M o (dY X^T) in fp32
//   Z = C h, B g (both parts)    -> w, v: what enters the gradients of dt, A and dt_bias is fp32
//   M^T dY, S^T C, S B, (e dY) h^T, (w X) g^T: dX per head, dB and dC accumulated in TMEM
// so that dB and dC leave once per CTA.  A chunk's heads are shared by several CTAs only where
// chunks alone are too few; their parts are then added by a kernel of its own.
// Roles (20 warps): 0-15 elementwise, 16 MMA, 17 loads of X, dY and weights, 18 of B, C and the
// images, 19 stores dX and turns the sums into d_dt, dA, dD and dt_bias' gradient.
#include <cstring>

#include "hla_ssm_carry.cuh"

namespace hla {
namespace ssm {
namespace {

using namespace tcs;

constexpr int kGradThreads = 20 * 32;

struct GradParams {
    Args a;
    int PT, splits;
    View vx, vdy, vb, vc;
    CUtensorMap mx, mdy, mb, mc, mdx;
    const Dec *dec;
    const uint8_t *h, *g;  // images
};

template <int NB>
struct LayGrad {
    static constexpr int HB = NB * kHalf / 2, NS = 3;  // dY and X of the heads in turn through three slots
    static constexpr int OFF_B = 0, OFF_C = NB * kHalf, OFF_S = 2 * NB * kHalf, OFF_XD = OFF_S + 2 * kHalf, OFF_H = OFF_XD + NS * kHalf,
                         OFF_G = OFF_H + 2 * HB;
    static constexpr int OFF_DEC = OFF_G + 2 * HB, OFF_SUM = OFF_DEC + 2 * (int)sizeof(Dec);
    static constexpr int SUM_FLOATS = 16 * T + 32;  // [w by quadrant, vE, wz, vg][4][128], through [16], dD [16]
    static constexpr int OFF_BAR = OFF_SUM + SUM_FLOATS * 4;
    static constexpr int B_XD = 0, B_XDE = B_XD + NS, B_DEC = B_XDE + NS, B_DECE = B_DEC + 2, B_H = B_DECE + 2, B_HE = B_H + 1,
                         B_G = B_HE + 1, B_GE = B_G + 1, B_BC = B_GE + 1, B_CB = B_BC + 1, B_DYX = B_CB + 1, B_DE = B_DYX + 1,
                         B_Z = B_DE + 1, B_GB = B_Z + 1, B_MS = B_GB + 1, B_XM = B_MS + 1, B_SE = B_XM + 1, B_YT = B_SE + 1,
                         B_Y = B_YT + 1, B_SUM = B_Y + 2, B_SUME = B_SUM + 1, B_FIN = B_SUME + 1, B_RAW = B_FIN + 1, B_RAW2 = B_RAW + 1,
                         NBAR = B_RAW2 + 1;
    static constexpr int SMEM = OFF_BAR + NBAR * 8 + 16;
    static constexpr uint32_t DC = 0, DB = T, DYX = 2 * T, M = 2 * T, XM = 2 * T + 64, Z = 3 * T, GB = 3 * T + 64, YT = Z, XT = Z + 32;
    HLA_DEVICE static int arrivals(int i) {
        return (i >= B_XDE && i < B_DEC) || i == B_DECE || i == B_DECE + 1 || i == B_HE || i == B_GE ? kElemWarps + 1
               : i == B_DE || i == B_MS || i == B_YT || i == B_Y || i == B_Y + 1 || i == B_SUM                    ? kElemWarps
                                                                                                   : 1;
    }
};

struct Job {  // one chunk of a group, the heads [h0, h1), U = heads x column tiles
    int b, g, c, len, t0, live, split, h0, U;
};
HLA_DEVICE int head_of(const GradParams &p, const Job &j, int u) { return j.h0 + u / p.PT; }

HLA_DEVICE void quad_sync(int q) { asm volatile("bar.sync %0, 128;" ::"r"(1 + q) : "memory"); }

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
HLA_DEVICE float dot16(const float2 (&x)[8], const float2 (&y)[8]) {
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fma2(x[i], y[i], s);
    return s.x + s.y;
}
HLA_DEVICE void load_row16(const uint8_t *tile, int rows, int r, int c0, float2 (&v)[8]) {
    unpack8(*reinterpret_cast<const uint4 *>(tile + tile_off(rows, r, c0)), v);
    unpack8(*reinterpret_cast<const uint4 *>(tile + tile_off(rows, r, c0 + 8)), v + 4);
}

template <int NB>
__device__ __forceinline__ void grad_elem(const GradParams &p, const Waits &ws, uint8_t *base, uint32_t tb, const Job &job) {
    using L = LayGrad<NB>;
    const Args &a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = warp & 3, cq = warp >> 2, row = 32 * q + lane, c0 = 16 * cq;
    const uint32_t lanes = tb + ((uint32_t)(32 * q) << 16);
    float *sums = reinterpret_cast<float *>(base + L::OFF_SUM);
    float *sum_w = sums + q * T + 32 * cq, *sum_ve = sums + 4 * T + cq * T, *sum_wz = sums + 8 * T + cq * T, *sum_vg = sums + 12 * T + cq * T;
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
            const uint32_t bits = cq > q ? 0xffffffffu : ~low_bits(lane);  // t >= j
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
                    ve += ee.x + ee.y;
                    e[2 * i] = ee.x * dt;
                    e[2 * i + 1] = ee.y * dt;
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
        // w from the state before the chunk; <g, h>
        ok = ok && ws.wait(L::B_XD + sy, ring_phase<L::NS>(2 * u)) && ws.wait(L::B_XD + sx, ring_phase<L::NS>(2 * u + 1)) &&
             ws.wait(L::B_H, ph) && ws.wait(L::B_G, ph);
        float2 yr[8], xr[8];
        load_row16(dy, T, row, c0, yr);
        load_row16(x, T, row, c0, xr);
        float through = 0.f;
        if (q < 2 * NB) {
            float2 h1[8], h2[8], g1[8], g2[8];
            load_row16(base + L::OFF_H, 64 * NB, row, c0, h1);
            load_row16(base + L::OFF_H + L::HB, 64 * NB, row, c0, h2);
            load_row16(base + L::OFF_G, 64 * NB, row, c0, g1);
            load_row16(base + L::OFF_G + L::HB, 64 * NB, row, c0, g2);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                h1[i] = add2(h1[i], h2[i]);
                g1[i] = add2(g1[i], g2[i]);
            }
            through = dot16(h1, g1);
        }
        float dd = dot16(xr, yr);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            through += __shfl_xor_sync(0xffffffffu, through, o);
            dd += __shfl_xor_sync(0xffffffffu, dd, o);
        }
        if (lane == 0) {
            sums[16 * T + warp] = through;
            sums[16 * T + 16 + warp] = dd;
            mbar_arrive(ws.bar(L::B_HE));
            mbar_arrive(ws.bar(L::B_GE));
        }
        ok = ok && ws.wait(L::B_Z, ph);
        tc_fence_after();
        float2 v[8];
        tmem_pairs16(lanes + L::Z + c0, v);
        tmem_wait_ld();
        sum_wz[row] = dot16(v, yr);
        quad_sync(q);  // the weighted rows go over Z
        tc_fence_after();
        {
            const float2 to = both(d.to[row]), w = both(d.w[row]);
            float ty[8], tx[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                ty[i] = __uint_as_float(pack2(mul2(yr[i], to)));
                tx[i] = __uint_as_float(pack2(mul2(xr[i], w)));
            }
            tmem_st8(lanes + L::YT + 8 * cq, ty);
            tmem_st8(lanes + L::XT + 8 * cq, tx);
            tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(ws.bar(L::B_YT));
            mbar_arrive(ws.bar(L::B_XDE + sy));
        }
        // v from the gradient behind the chunk; dX
        ok = ok && ws.wait(L::B_GB, ph);
        tc_fence_after();
        tmem_pairs16(lanes + L::GB + c0, v);
        tmem_wait_ld();
        sum_vg[row] = dot16(v, xr);
        {
            const float2 D = both(a.D ? a.D[h] : 0.f), w = both(d.w[row]);
#pragma unroll
            for (int i = 0; i < 8; ++i) yr[i] = fma2(D, yr[i], mul2(w, v[i]));
        }
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(ws.bar(L::B_SUM));
            mbar_arrive(ws.bar(L::B_DECE + (u & 1)));
        }
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
    // both parts of an image: rows n by columns p, contracted over rows or over columns
    const uint64_t Hm = make_sdesc(smem_u32(base + L::OFF_H), 64 * NB * 128u, 1024u), Gm = make_sdesc(smem_u32(base + L::OFF_G), 64 * NB * 128u, 1024u);
    const uint64_t Hk = kmajor(base + L::OFF_H), Gk = kmajor(base + L::OFF_G);
    auto by_state = [&](uint32_t d, uint64_t rows, uint64_t image) {  // [128 x 64] = rows (hi + lo)
        mma_km64(d, rows, image, id_y, false);
        if (NB > 1) mma_km64(d, rows + kBlock, image + kRows64, id_y, true);
        mma_km64(d, rows, image + (L::HB >> 4), id_y, true);
        if (NB > 1) mma_km64(d, rows + kBlock, image + (L::HB >> 4) + kRows64, id_y, true);
    };
    bool ok = ws.wait(L::B_BC, 0u);
    if (ok) {
        mma_ss64(tb + L::DYX, Bk, Ck, id_tt, false);
        if (NB > 1) mma_ss64(tb + L::DYX, Bk + kBlock, Ck + kBlock, id_tt, true);
        umma_commit_warp(ws.bar(L::B_CB));
    }
#pragma unroll 1
    for (int u = 0; u < U && ok; ++u) {
        const uint32_t ph = (uint32_t)u & 1u;
        const int sy = (2 * u) % L::NS, sx = (2 * u + 1) % L::NS;
        const uint8_t *dy = base + L::OFF_XD + sy * kHalf, *x = base + L::OFF_XD + sx * kHalf;
        if (!(ok = ws.wait(L::B_XD + sy, ring_phase<L::NS>(2 * u)) && ws.wait(L::B_XD + sx, ring_phase<L::NS>(2 * u + 1)) && ws.wait(L::B_DE, ph))) break;
        tc_fence_after();
        mma_ss64(tb + L::DYX, kmajor(x), kmajor(dy), id_tt, false);
        umma_commit_warp(ws.bar(L::B_DYX));
        if (!(ok = ws.wait(L::B_H, ph))) break;
        by_state(tb + L::Z, Ck, Hm);
        umma_commit_warp(ws.bar(L::B_Z));
        if (!(ok = ws.wait(L::B_G, ph))) break;
        by_state(tb + L::GB, Bk, Gm);
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
        if (!(ok = ws.wait(L::B_YT, ph))) break;
        tc_fence_after();
        mma_tk64(tb + L::DC, tb + L::YT, Hk, id_k);  // both parts: the weighted rows are then the only rounding
        mma_tk64(tb + L::DC, tb + L::YT, Hk + (L::HB >> 4), id_k);
        mma_tk64(tb + L::DB, tb + L::XT, Gk, id_k);
        mma_tk64(tb + L::DB, tb + L::XT, Gk + (L::HB >> 4), id_k);
        umma_commit_warp(ws.bar(L::B_HE));
        umma_commit_warp(ws.bar(L::B_GE));
        umma_commit_warp(ws.bar(L::B_XDE + sy));
    }
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
    int i = 0;
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
    // nothing may land after the CTA has ended (only an aborted CTA still has copies in flight)
    if (ok) {
        for (int k = max(0, i - L::NS); k < i; ++k) mbar_wait(ws.bar(L::B_XD + k % L::NS), ring_phase<L::NS>(k), ws.err);
        for (int k = max(0, job.U - 2); k < job.U; ++k) mbar_wait(ws.bar(L::B_DEC + (k & 1)), ring_phase<2>(k), ws.err);
    }
    __syncwarp();
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
        if (u > 0 && !(ok = ws.wait(L::B_HE, ph ^ 1u))) break;
        if (lane == 0) {
            mbar_expect_tx(ws.bar(L::B_H), 2 * L::HB);
            bulk_load(base + L::OFF_H, p.h + at * 2 * L::HB, 2 * L::HB, ws.bar(L::B_H));
        }
        __syncwarp();
        if (u > 0 && !(ok = ws.wait(L::B_GE, ph ^ 1u))) break;
        if (lane == 0) {
            mbar_expect_tx(ws.bar(L::B_G), 2 * L::HB);
            bulk_load(base + L::OFF_G, p.g + at * 2 * L::HB, 2 * L::HB, ws.bar(L::B_G));
        }
        __syncwarp();
    }
    if (ok) {
        mbar_wait(ws.bar(L::B_BC), 0u, ws.err);
        mbar_wait(ws.bar(L::B_H), (uint32_t)(job.U - 1) & 1u, ws.err);
        mbar_wait(ws.bar(L::B_G), (uint32_t)(job.U - 1) & 1u, ws.err);
    }
    __syncwarp();
}

// dX of each head's columns to memory; then, after a head's last columns, the gradients of its
// steps from the sums: four adjacent tokens a lane.
template <int NB>
__device__ __forceinline__ void grad_sums(const GradParams &p, const Waits &ws, uint8_t *base, const Job &job) {
    using L = LayGrad<NB>;
    const Args &a = p.a;
    const int lane = threadIdx.x & 31;
    const float *sums = reinterpret_cast<const float *>(base + L::OFF_SUM);
    float w[4], ve[4], vg[4], through = 0.f, dd = 0.f;
#pragma unroll 1
    for (int u = 0; u < job.U; ++u) {
        const uint32_t ph = (uint32_t)u & 1u;
        const int h = head_of(p, job, u), pt = u % p.PT, sx = (2 * u + 1) % L::NS;
        const Dec &d = *reinterpret_cast<const Dec *>(base + L::OFF_DEC + (u & 1) * sizeof(Dec));
        if (!ws.wait(L::B_DEC + (u & 1), ring_phase<2>(u)) || !ws.wait(L::B_SUM, ph)) break;
        if (pt == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = ve[i] = vg[i] = 0.f;
            through = dd = 0.f;
        }
        const Decay end = d.s[T - 1];
        Decay s[4];
        float dt[4], sl[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = 4 * lane + i;
            s[i] = d.s[t];
            dt[i] = d.dt[t];
            sl[i] = d.slope[t];
            float x = 0.f, y = 0.f, z = 0.f, g = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                x += sums[k * T + t];
                y += sums[4 * T + k * T + t];
                z += sums[8 * T + k * T + t];
                g += sums[12 * T + k * T + t];
            }
            w[i] += fmaf(d.to[t], z, x);
            ve[i] += y;
            vg[i] = fmaf(factor(end, s[i]), g, vg[i]);
        }
        float th = lane < 16 ? sums[16 * T + lane] : 0.f, dx = lane < 16 ? sums[16 * T + 16 + lane] : 0.f;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) {
            th += __shfl_xor_sync(0xffffffffu, th, o);
            dx += __shfl_xor_sync(0xffffffffu, dx, o);
        }
        through = fmaf(d.end, th, through);
        dd += dx;
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(ws.bar(L::B_SUME));
            mbar_arrive(ws.bar(L::B_DECE + (u & 1)));
        }
        if (pt == p.PT - 1) {
            float suf[4], pre[4], s1 = 0.f, s2 = 0.f;
#pragma unroll
            for (int i = 3; i >= 0; --i) {
                s1 += fmaf(-dt[i], ve[i], w[i]);
                suf[i] = s1;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                pre[i] = s2;
                s2 = fmaf(dt[i], vg[i], s2);
            }
            float xs = s1, xp = s2;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float us = __shfl_down_sync(0xffffffffu, xs, o), up = __shfl_up_sync(0xffffffffu, xp, o);
                if (lane + o < 32) xs += us;
                if (lane >= o) xp += up;
            }
            xs -= s1;
            xp -= s2;
            through = __shfl_sync(0xffffffffu, through, 0);
            const float A = a.A[h];
            float sA = 0.f, sb = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = 4 * lane + i;
                const float da = through + (suf[i] + xs) + (pre[i] + xp), g = fmaf(A, da, ve[i] + vg[i]) * sl[i];
                if (t < job.live) {
                    static_cast<__nv_bfloat16 *>(a.ddt.p)[(size_t)job.b * a.ddt.sb + (size_t)h * a.ddt.sh + (size_t)(job.t0 + t) * a.ddt.st] = __float2bfloat16_rn(g);
                    sA = fmaf(da, dt[i], sA);
                    sb += g;
                }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                sA += __shfl_xor_sync(0xffffffffu, sA, o);
                sb += __shfl_xor_sync(0xffffffffu, sb, o);
            }
            if (lane == 0) {
                float *out = a.sums + ((size_t)job.b * a.nc + job.c) * 3 * a.H + h;
                out[0] = sA;
                out[a.H] = dd;
                out[2 * a.H] = sb;
            }
        }
        if (!ws.wait(L::B_Y + (u & 1), ring_phase<2>(u))) break;
        const uint8_t *x = base + L::OFF_XD + sx * kHalf;
        if (job.live == T) {
            if (lane == 0) {
                tma_store_4d(x, &p.mdx, 64 * pt, job.t0, a.dx.sh ? h : 0, a.dx.sb ? job.b : 0);
                bulk_commit();
                bulk_wait_read();
            }
        } else {  // rows behind the sequence stay as they are
            __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.dx.p) + (size_t)job.b * a.dx.sb + (size_t)h * a.dx.sh + (size_t)job.t0 * a.dx.st;
            for (int i = lane; i < job.live * 8; i += 32) {
                const int r = i >> 3, cc = 64 * pt + 8 * (i & 7);
                if (cc < a.P) *reinterpret_cast<uint4 *>(out + (size_t)r * a.dx.st + cc) = *reinterpret_cast<const uint4 *>(x + tile_off(T, r, 8 * (i & 7)));
            }
        }
        __syncwarp();
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
    if (j.live <= 0) {
        float *out = a.sums + ((size_t)j.b * a.nc + j.c) * 3 * a.H;
        for (int h = j.h0 + threadIdx.x; h < h1; h += kGradThreads) out[h] = out[a.H + h] = out[2 * a.H + h] = 0.f;
        return;
    }
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

template <int NB>
cudaError_t launch(const Params &p, const GradParams &g, cudaStream_t st) {
    using L = LayGrad<NB>;
    static_assert(L::SMEM <= 227 * 1024, "shared memory");
    cudaError_t e = starts<NB>(p, 2, st);
    if (e == cudaSuccess) e = walk<NB, false>(p, st);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(ssm_grad_tc_kernel<NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM);
    if (e != cudaSuccess) return e;
    const Args &a = p.a;
    ssm_grad_tc_kernel<NB><<<(unsigned)((size_t)a.B * a.nc * a.G * g.splits), kGradThreads, L::SMEM, st>>>(g);
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
    Params p;
    GradParams g;
    memset(&p, 0, sizeof p);
    memset(&g, 0, sizeof g);
    p.a = a;
    cudaError_t e = dev_status_ptr(&p.a.err);
    if (e != cudaSuccess) return e;
    p.plan = plan_of(a, kSms);
    p.vx[0] = a.x; p.vx[1] = a.dy;
    p.vb[0] = a.b; p.vb[1] = a.c;
    p.pieces[0] = a.h; p.pieces[1] = a.g;
    p.factor = a.factor;
    p.dec = static_cast<const Dec *>(a.dec);
    p.image[0] = a.image[0]; p.image[1] = a.image[1];
    g.a = p.a;
    g.PT = p.plan.PT;
    g.splits = a.splits;
    g.vx = a.x; g.vdy = a.dy; g.vb = a.b; g.vc = a.c;
    g.dec = p.dec;
    g.h = a.image[0]; g.g = a.image[1];
    if (!encode(&p.mx[0], a.x, a.P, a.n, a.H, a.B, T) || !encode(&p.mx[1], a.dy, a.P, a.n, a.H, a.B, T) ||
        !encode(&p.mb[0], a.b, a.N, a.n, a.G, a.B, T) || !encode(&p.mb[1], a.c, a.N, a.n, a.G, a.B, T) ||
        !encode(&g.mdx, a.dx, a.P, a.n, a.H, a.B, T))
        return cudaErrorNotSupported;
    g.mx = p.mx[0]; g.mdy = p.mx[1]; g.mb = p.mb[0]; g.mc = p.mb[1];
    e = a.N <= 64 ? launch<1>(p, g, st) : launch<2>(p, g, st);
    return e == cudaSuccess ? join(a, HLA_BF16, a.splits > 1, st) : e;
}

}  // namespace ssm
}  // namespace hla
