// hla_window_fwd_tc.cu -- forward of windowed attention for bf16 on the tensor cores.
//
// One CTA takes two tiles of 128 queries that share their keys -- the same rows of two
// heads of one group, or two neighbouring row tiles of a head -- and walks the key tiles
// they can see: per key tile and query tile S = Q K^T into TMEM (128 fp32 columns), the
// softmax of one row per thread (running maximum and sum in fp32), P packed to bf16 over
// S's own columns, O += P V with P read from TMEM.  While the softmax of one query tile
// runs, the tensor cores work on the other.  Warps 0-3 and 4-7: softmax of tile 0 and 1;
// warp 8: MMA; warp 9: TMA into a ring of key and value tiles (10, 11: none).
//
// The running maximum used in the exponent only moves when a row's maximum passes it by
// more than 2^8: P then stays below 2^8, and O in TMEM is rescaled a few times per row
// instead of at every key tile.
#include "hla_window_tc.cuh"

namespace hla {
namespace win {
namespace {

using namespace tcw;

constexpr int kThreads = 384, kWarpMma = 8, kWarpTma = 9;
// Registers per thread of the softmax warpgroups, which hold a row of S, and of the third
// warpgroup: with the 168 that each of the 384 threads is launched with, 2 x 200 + 104 = 3 x 168.
constexpr int kRegsSoftmax = 200, kRegsOther = 104;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f, kSlack = 8.f;

struct Params {
    Args a;
    CUtensorMap mq, mk, mv;
    int pair_heads;  // the two tiles are two heads of a group (else two row tiles of a head)
};

template <int DP>
struct Lay {
    static constexpr int TILE = T * DP * 2;
    static constexpr int NS = DP == 64 ? 8 : 4;  // ring slots
    static constexpr int OFF_Q = 0, OFF_RING = 2 * TILE, OFF_BAR = OFF_RING + NS * TILE;
    static constexpr int B_Q = 0, B_FULL = 1, B_EMPTY = B_FULL + NS, B_S = B_EMPTY + NS, B_P = B_S + 2, B_O = B_P + 4,
                         B_FIN = B_O + 2, NB = B_FIN + 1;
    static constexpr int SMEM = OFF_BAR + NB * 8 + 16;
    static constexpr uint32_t S0 = 0, O0 = 2 * T;  // TMEM columns: S of both tiles, O of both
};

// What the two query tiles of this CTA need.
struct Work {
    int b, hk, h[2], row[2];       // head and first row of each tile
    bool on[2];
    int lo[2], hi[2], sink_tiles;  // key tiles of each: [lo, hi], and those below sink_tiles
    int head, first, total, len, rows;
    HLA_DEVICE Work(const Params &p) {
        const Args &a = p.a;
        const int groups = p.pair_heads ? a.H / 2 : a.H, step = p.pair_heads ? T : 2 * T;
        const int tiles = (a.n + step - 1) / step;
        const int u = blockIdx.x % (a.B * groups);
        const int rt = tiles - 1 - (int)(blockIdx.x / (a.B * groups));  // long rows first
        b = u / groups;
        h[0] = p.pair_heads ? (u % groups) * 2 : u % groups;
        h[1] = p.pair_heads ? h[0] + 1 : h[0];
        hk = h[0] / a.G;
        row[0] = rt * step;
        row[1] = p.pair_heads ? row[0] : row[0] + T;
        len = length_of(a, b);
        rows = min(a.n, len - a.p0);
        sink_tiles = a.sinks > 0 ? (a.sinks - 1) / T + 1 : 0;
        int last = -1;
        first = 0x7fffffff;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            on[t] = row[t] < rows;
            lo[t] = 0;
            hi[t] = -1;
            if (on[t]) {
                const int p_lo = a.p0 + row[t], p_hi = a.p0 + min(row[t] + T, rows) - 1;
                lo[t] = (p_lo >= a.window ? p_lo - a.window + 1 : 0) / T;
                hi[t] = p_hi / T;
                first = min(first, lo[t]);
                last = max(last, hi[t]);
            }
        }
        head = min(sink_tiles, first);
        total = last < 0 ? 0 : head + last - first + 1;
    }
    // Columns of key tile kt that tile t works on: all, or before its window only those of
    // the first tokens, in chunks of 32.
    HLA_DEVICE int columns(const Args &a, int t, int kt) const {
        return kt >= (t ? lo[1] : lo[0]) ? T : min(T, (a.sinks - kt * T + 31) & ~31);
    }
    HLA_DEVICE int key_tile(int i) const { return i < head ? i : first + i - head; }
    HLA_DEVICE bool active(int t, int kt) const {
        return kt <= (t ? hi[1] : hi[0]) && (kt >= (t ? lo[1] : lo[0]) || kt < sink_tiles);
    }
};

// 64 columns (or 32) of fp32 in this warp's lanes
HLA_DEVICE void scale_cols(uint32_t addr, int cols, float f) {
    for (int c = 0; c < cols; c += 16) {
        float v[16];
        tmem_ld16(addr + c, v);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] *= f;
        tmem_st16(addr + c, v);
    }
    tmem_wait_st();
}

template <int DP>
__device__ __forceinline__ void softmax_role(const Params &p, const Work &w, const Waits &ws, uint32_t tb, int t) {
    using L = Lay<DP>;
    const Args &a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row0 = t ? w.row[1] : w.row[0], head = t ? w.h[1] : w.h[0];
    const int r = row0 + (warp & 3) * 32 + lane;  // this thread's query row
    const int pos = a.p0 + r;
    const uint32_t sa = tb + ((uint32_t)(32 * (warp & 3)) << 16) + L::S0 + t * T;
    const uint32_t oa = tb + ((uint32_t)(32 * (warp & 3)) << 16) + L::O0 + t * DP;
    const float c = a.scale * kLog2e;
    const unsigned long long c2 = pair2(c, c);
    const int dvp = (a.dv + 15) & ~15;
    const int p_lo = a.p0 + row0, p_hi = p_lo + T - 1;
    float m = -INFINITY, l = 0.f;  // reference maximum (base 2, scaled), sum
    uint32_t ph = 0;
    bool begun = false, ok = true;
    for (int i = 0; i < w.total; ++i) {
        const int kt = w.key_tile(i);
        if (!w.active(t, kt)) continue;
        if (!ws.wait(L::B_S + t, ph)) { ok = false; break; }
        ph ^= 1u;
        tc_fence_after();
        const int j0 = kt * T;
        const bool masked = !(j0 + T - 1 <= p_lo && (p_hi - j0 < a.window || j0 + T <= a.sinks));
        const int hi = pos - j0, sk = a.sinks - j0, lo = pos >= a.window ? pos - a.window + 1 - j0 : -1;
        const int chunks = w.columns(a, t, kt) >> 5;
        float mx = -INFINITY;
        float s[4][32];
        if (chunks == 4) {
#pragma unroll
            for (int k = 0; k < 4; ++k) tmem_ld32(sa + 32 * k, s[k]);
            tmem_wait_ld();
            if (masked) {
#pragma unroll
                for (int k = 0; k < 4; ++k) mask32(s[k], visible_bits(32 * k, lo, hi + 1, sk), -INFINITY);
            }
            float x[4] = {s[0][0], s[1][0], s[2][0], s[3][0]};
#pragma unroll
            for (int e = 1; e < 31; e += 2)
#pragma unroll
                for (int k = 0; k < 4; ++k) x[k] = max3(x[k], s[k][e], s[k][e + 1]);
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] = fmaxf(x[k], s[k][31]);
            mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
        } else {
#pragma unroll 1
            for (int k = 0; k < chunks; ++k) {
                tmem_ld32(sa + 32 * k, s[0]);
                tmem_wait_ld();
                mask32(s[0], visible_bits(32 * k, lo, hi + 1, sk), -INFINITY);
#pragma unroll
                for (int e = 0; e < 32; e += 2) mx = max3(mx, s[0][e], s[0][e + 1]);
            }
        }
        mx *= c;
        const bool move = mx > m + kSlack || (m == -INFINITY && mx > m);
        if (__any_sync(0xffffffffu, move)) {
            const float mn = move ? mx : m;
            const float f = move ? ex2_approx(m - mn) : 1.f;
            l *= f;
            m = mn;
            if (begun) scale_cols(oa, dvp, f);
        }
        const float base = m == -INFINITY ? 0.f : m;
        const unsigned long long b2 = pair2(-base, -base);
        unsigned long long sum[2] = {0ull, 0ull};
        auto probabilities = [&](const float(&v)[32], uint32_t to) {  // 32 columns of P
            float pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                float x, y;
                unpair2(fma2(pair2(v[2 * e], v[2 * e + 1]), c2, b2), x, y);
                x = ex2_approx(x);
                y = ex2_approx(y);
                sum[e & 1] = add2(sum[e & 1], pair2(x, y));
                pk[e] = __uint_as_float(pack_bf16(x, y));
            }
            tmem_st16(to, pk);
        };
        auto hand_over = [&](int half) {  // half of P is there: its products can begin
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(ws.bar(L::B_P + 2 * t + half));
        };
        if (chunks == 4) {
            probabilities(s[0], sa);
            probabilities(s[1], sa + 16);
            hand_over(0);
            probabilities(s[2], sa + 32);
            probabilities(s[3], sa + 48);
            hand_over(1);
        } else {
#pragma unroll 1
            for (int k = 0; k < chunks; ++k) {
                tmem_ld32(sa + 32 * k, s[0]);
                tmem_wait_ld();
                mask32(s[0], visible_bits(32 * k, lo, hi + 1, sk), -INFINITY);
                probabilities(s[0], sa + 16 * k);
            }
            hand_over(0);
            hand_over(1);
        }
        float l0, l1;
        unpair2(add2(sum[0], sum[1]), l0, l1);
        l += l0 + l1;
        begun = true;
    }
    if (!begun || !ok) return;
    if (!ws.wait(L::B_O + t, 0u)) return;
    tc_fence_after();
    const bool live = r < w.rows;
    const float inv = 1.f / l;
    __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.o.p) + (size_t)w.b * a.o.sb + (size_t)head * a.o.sh + (size_t)r * a.o.st;
    for (int k = 0; k < dvp; k += 16) {
        float v[16];
        tmem_ld16(oa + k, v);
        tmem_wait_ld();
        uint4 u[2];
        uint32_t *q = reinterpret_cast<uint32_t *>(u);
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = pack_bf16(v[2 * e] * inv, v[2 * e + 1] * inv);
        if (live) {
            *reinterpret_cast<uint4 *>(o + k) = u[0];
            if (k + 8 < a.dv) *reinterpret_cast<uint4 *>(o + k + 8) = u[1];
        }
    }
    if (live && a.lse) a.lse[((size_t)w.b * a.H + head) * a.n + r] = (m + log2f(l)) * kLn2;
}

template <int DP>
__device__ __forceinline__ void mma_role(const Params &p, const Work &w, const Waits &ws, uint8_t *base, uint32_t tb) {
    using L = Lay<DP>;
    const Args &a = p.a;
    const int lane = threadIdx.x & 31;
    const uint32_t id_o = make_idesc(T, (a.dv + 15) & ~15, false, true);
    const bool wide = a.d > 64;
    tb = uniform(tb);
    bool pend[2] = {false, false}, begun[2] = {false, false};
    uint32_t php[2] = {0, 0};
    bool ok = ws.wait(L::B_Q, 0u);
    auto slot = [&](int idx) { return base + L::OFF_RING + (idx % L::NS) * L::TILE; };
    auto full = [&](int idx) { return ws.wait(L::B_FULL + idx % L::NS, (uint32_t)(idx / L::NS) & 1u); };
    for (int i = 0; i <= w.total && ok; ++i) {  // the last round only finishes O
        const int kt = i < w.total ? w.key_tile(i) : -1;
        bool k_here = false, v_here = false;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            if (pend[t] && ok) {
                if (!v_here) {
                    ok = full(2 * (i - 1) + 1);
                    v_here = true;
                    // values behind the sequence may be anything, and 0 times that is not 0
                    const int live = w.len - w.key_tile(i - 1) * T;
                    if (ok && live < T) zero_rows<DP>(slot(2 * (i - 1) + 1), live, lane);
                }
                const int chunks = uniform(w.columns(a, t, w.key_tile(i - 1)) / 32);
                const uint64_t dv = make_sdesc(smem_u32(slot(2 * (i - 1) + 1)), T * 128u, 1024u);
                const uint32_t o = tb + L::O0 + t * DP, s = tb + L::S0 + t * T;
#pragma unroll
                for (int g = 0; g < 2; ++g) {  // the halves of P as they come
                    if (ok) ok = ws.wait(L::B_P + 2 * t + g, php[t]);
                    if (!ok) break;
                    tc_fence_after();
                    if (2 * g < chunks) mma_ts32(o, s + 32 * g, dv + 512 * g, id_o, begun[t] || g > 0);
                    if (2 * g + 1 < chunks) mma_ts32(o, s + 32 * g + 16, dv + 512 * g + 256, id_o, true);
                }
                if (!ok) break;
                php[t] ^= 1u;
                begun[t] = true;
                pend[t] = false;
                if (i == w.total || kt > w.hi[t]) umma_commit_warp(ws.bar(L::B_O + t));
            }
            if (i < w.total && ok && w.active(t, kt)) {
                if (!k_here) {
                    ok = full(2 * i);
                    k_here = true;
                }
                if (!ok) break;
                mma_kk<DP>(tb + L::S0 + t * T, base + L::OFF_Q + t * L::TILE, slot(2 * i),
                           make_idesc(T, uniform(w.columns(a, t, kt)), false, false), wide);
                umma_commit_warp(ws.bar(L::B_S + t));
                pend[t] = true;
            }
        }
        if (!ok) break;
        if (i > 0) umma_commit_warp(ws.bar(L::B_EMPTY + (2 * i - 1) % L::NS));
        if (i < w.total) umma_commit_warp(ws.bar(L::B_EMPTY + (2 * i) % L::NS));
    }
    umma_commit_warp(ws.bar(L::B_FIN));  // every MMA issued completes before TMEM is released
    mbar_wait(ws.bar(L::B_FIN), 0u, ws.err);
    __syncwarp();
}

template <int DP>
__device__ __forceinline__ void tma_role(const Params &p, const Work &w, const Waits &ws, uint8_t *base) {
    using L = Lay<DP>;
    const Args &a = p.a;
    const bool one = (threadIdx.x & 31) == 0;
    if (one) {
        mbar_expect_tx(ws.bar(L::B_Q), (w.on[0] + w.on[1]) * L::TILE);
        for (int t = 0; t < 2; ++t)
            if (w.on[t]) load_tile<DP>(base + L::OFF_Q + t * L::TILE, &p.mq, a.q, ws.bar(L::B_Q), w.row[t], w.h[t], w.b);
    }
    int idx = 0;
    for (; idx < 2 * w.total; ++idx) {
        const int s = idx % L::NS, use = idx / L::NS;
        if (use > 0 && !ws.wait(L::B_EMPTY + s, (uint32_t)(use - 1) & 1u)) break;
        if (one) {
            mbar_expect_tx(ws.bar(L::B_FULL + s), L::TILE);
            const bool key = (idx & 1) == 0;
            load_tile<DP>(base + L::OFF_RING + s * L::TILE, key ? &p.mk : &p.mv, key ? a.k : a.v, ws.bar(L::B_FULL + s),
                          w.key_tile(idx >> 1) * T, w.hk, w.b);
        }
        __syncwarp();
    }
    // nothing may land after the CTA has ended (only an aborted CTA still has copies in flight)
    mbar_wait(ws.bar(L::B_Q), 0u, ws.err);
    for (int k = max(0, idx - L::NS); k < idx; ++k)
        mbar_wait(ws.bar(L::B_FULL + k % L::NS), (uint32_t)(k / L::NS) & 1u, ws.err);
    __syncwarp();
}

template <int DP>
__global__ void __launch_bounds__(kThreads, 1) window_fwd_kernel(const __grid_constant__ Params p) {
    using L = Lay<DP>;
    extern __shared__ __align__(1024) uint8_t base[];
    const Work w(p);
    if (w.total == 0) return;  // both tiles lie behind the sequence
    Waits ws{reinterpret_cast<uint64_t *>(base + L::OFF_BAR), nullptr, p.a.err};
    uint32_t *misc = reinterpret_cast<uint32_t *>(base + L::OFF_BAR + L::NB * 8);  // TMEM base, abort
    ws.abort_p = reinterpret_cast<volatile int *>(misc + 1);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        misc[1] = 0u;
        for (int i = 0; i < L::NB; ++i) mbar_init(ws.bar(i), i >= L::B_P && i < L::B_P + 4 ? 4 : 1);
        fence_mbar_init();
        tma_prefetch_desc(&p.mq);
        tma_prefetch_desc(&p.mk);
        tma_prefetch_desc(&p.mv);
    }
    if (warp == kWarpMma) {
        tmem_alloc(misc, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tb = misc[0];
    if (warp >= kWarpMma) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
        if (warp == kWarpTma) tma_role<DP>(p, w, ws, base);
        if (warp == kWarpMma) mma_role<DP>(p, w, ws, base, tb);
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        softmax_role<DP>(p, w, ws, tb, warp >> 2);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kWarpMma) tmem_dealloc(tb, 512);
}

template <int DP>
cudaError_t launch(Params &p, cudaStream_t st) {
    using L = Lay<DP>;
    static_assert(L::SMEM <= 227 * 1024, "shared memory");
    const Args &a = p.a;
    if (!encode(&p.mq, a.q, a.d, a.n, a.H, a.B, T) || !encode(&p.mk, a.k, a.d, a.nk, a.Hkv, a.B, T) ||
        !encode(&p.mv, a.v, a.dv, a.nk, a.Hkv, a.B, T))
        return cudaErrorNotSupported;
    cudaError_t e = cudaFuncSetAttribute(window_fwd_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM);
    if (e != cudaSuccess) return e;
    const size_t items = p.pair_heads ? (size_t)a.B * (a.H / 2) * ((a.n + T - 1) / T)
                                      : (size_t)a.B * a.H * ((a.n + 2 * T - 1) / (2 * T));
    window_fwd_kernel<DP><<<(unsigned)items, kThreads, L::SMEM, st>>>(p);
    return cudaGetLastError();
}

}  // namespace

bool fwd_tc_takes(const Args &a) {
    // a positive scale: the largest product is then the largest score
    return a.scale > 0.f && a.d % 8 == 0 && a.dv % 8 == 0 && tcw::mappable(a.q) && tcw::mappable(a.k) && tcw::mappable(a.v) &&
           (reinterpret_cast<uintptr_t>(a.o.p) & 15u) == 0 && a.o.sb % 8 == 0 && a.o.sh % 8 == 0 && a.o.st % 8 == 0;
}

cudaError_t fwd_tc(const Args &a, cudaStream_t st) {
    Params p;
    memset(&p, 0, sizeof p);
    p.a = a;
    // two heads of one group see the same keys; with an odd group two row tiles of one head
    // share most of theirs
    p.pair_heads = a.G % 2 == 0;
    return a.d <= 64 && a.dv <= 64 ? launch<64>(p, st) : launch<128>(p, st);
}

}  // namespace win
}  // namespace hla
