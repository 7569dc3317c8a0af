// hla_window_fwd_tc.cu -- forward of windowed attention for bf16 on the tensor cores.
//
// Work items: two tiles of 128 queries that share their keys -- the same rows of two heads of
// one group, or two neighbouring row tiles of a head -- walk the key tiles they can see: per
// key tile and query tile S = Q K^T into TMEM (128 fp32 columns), the softmax in fp32 with a
// running maximum and sum, P packed to bf16 over S's own columns, O += P V with P read from
// TMEM.  While the softmax of one query tile runs, the tensor cores work on the other.
// Persistent: one CTA per SM goes through the items, so that an item's output and the next
// one's first loads and products overlap.  Warps 0-15: softmax, four warps per (query tile,
// half of the key columns), one row per thread, the halves' maxima exchanged through shared
// memory (with whole rows per thread the softmax took longer than the products beside it);
// warp 16: MMA; warp 17: TMA into a ring of key and value tiles.
//
// The running maximum used in the exponent only moves when a row's maximum passes it by
// more than 2^8: P then stays below 2^8, and O in TMEM is rescaled a few times per row
// instead of at every key tile.
#include "hla_window_tc.cuh"

namespace hla {
namespace win {
namespace {

using namespace tcw;

// Registers per thread of the softmax warps and of the last warpgroup: 4 x 104 + 64 = 5 x 96,
// the 96 that each of the 640 threads is launched with.
constexpr int kThreads = 640, kWarpMma = 16, kWarpTma = 17, kRegsSoftmax = 104, kRegsOther = 64;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f, kSlack = 8.f;

struct Params {
    Args a;
    CUtensorMap mq, mk, mv;
    int pair_heads;  // the two tiles are two heads of a group (else two row tiles of a head)
    int items;
    int wide_out;    // rows of o start at multiples of 32 bytes
};

template <int DP>
struct Lay {
    static constexpr int TILE = T * DP * 2;
    static constexpr int NS = DP == 64 ? 8 : 4;  // ring slots
    static constexpr int OFF_Q = 0, OFF_RING = 2 * TILE, OFF_ROW = OFF_RING + NS * TILE;
    static constexpr int OFF_BAR = OFF_ROW + 2 * 2 * 2 * T * 4;  // [two uses in turn][tile][half][row]
    // barriers of a query tile: Q landed, Q free, S ready, P ready, O ready, O read
    static constexpr int B_FULL = 0, B_EMPTY = B_FULL + NS, B_Q = B_EMPTY + NS, B_QE = B_Q + 2, B_S = B_QE + 2, B_P = B_S + 2,
                         B_O = B_P + 2, B_OE = B_O + 2, B_FIN = B_OE + 2, NB = B_FIN + 1;
    static constexpr int SMEM = OFF_BAR + NB * 8 + 16;
    static constexpr uint32_t S0 = 0, O0 = 2 * T;  // TMEM columns: S of both tiles, O of both
};

// What the two query tiles of an item need.
struct Work {
    int b, hk, h[2], row[2];       // head and first row of each tile
    bool on[2];
    int lo[2], hi[2], sink_tiles;  // key tiles of each: [lo, hi], and those below sink_tiles
    int head, first, total, len, rows;
    HLA_DEVICE Work(const Params &p, int item) {
        const Args &a = p.a;
        const int groups = p.pair_heads ? a.H / 2 : a.H, step = p.pair_heads ? T : 2 * T;
        const int tiles = (a.n + step - 1) / step;
        const int u = item % (a.B * groups);
        const int rt = tiles - 1 - item / (a.B * groups);  // long rows first
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
    // Chunks of 32 columns of key tile kt that tile t works on: all, or before its window only
    // those with first tokens.
    HLA_DEVICE int chunks(const Args &a, int t, int kt) const {
        return kt >= (t ? lo[1] : lo[0]) ? 4 : min(4, (a.sinks - kt * T + 31) >> 5);
    }
    HLA_DEVICE int key_tile(int i) const { return i < head ? i : first + i - head; }
    HLA_DEVICE bool active(int t, int kt) const {
        return kt <= (t ? hi[1] : hi[0]) && (kt >= (t ? lo[1] : lo[0]) || kt < sink_tiles);
    }
};

// Barrier of the two warpgroups of query tile t.
HLA_DEVICE void pair_sync(int t) {
    if (t == 0)
        asm volatile("bar.sync 1, 256;" ::: "memory");
    else
        asm volatile("bar.sync 2, 256;" ::: "memory");
}

template <int DP>
__device__ __forceinline__ void softmax_role(const Params &p, const Waits &ws, uint8_t *smem, uint32_t tb, int t, int half) {
    using L = Lay<DP>;
    const Args &a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rr = (warp & 3) * 32 + lane;
    const uint32_t quad = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t sa = tb + quad + L::S0 + t * T;         // S of the tile, P over it
    const uint32_t oa = tb + quad + L::O0 + t * DP;
    float *rows_sm = reinterpret_cast<float *>(smem + L::OFF_ROW);
    const float c = a.scale * kLog2e;
    const unsigned long long c2 = pair2(c, c);
    const int dvp = (a.dv + 15) & ~15;
    uint32_t phs = 0, pho = 0, turn = 0;
    bool ok = true;
    // x of this row's other half (every thread of the tile's two warpgroups calls this)
    auto other_half = [&](float x) {
        float *at = rows_sm + ((turn & 1) * 4 + t * 2) * T;
        ++turn;
        at[half * T + rr] = x;
        pair_sync(t);
        return at[(half ^ 1) * T + rr];
    };
    // After an expired wait the loops go on without their work, so that the barriers between
    // the warpgroups stay matched; every further wait returns at once.
    for (int item = blockIdx.x; item < p.items; item += gridDim.x) {
        const Work w(p, item);
        if (!(t ? w.on[1] : w.on[0])) continue;
        const int row0 = t ? w.row[1] : w.row[0], head = t ? w.h[1] : w.h[0];
        const int r = row0 + rr, pos = a.p0 + r, p_lo = a.p0 + row0, p_hi = p_lo + T - 1;
        float m = -INFINITY, l = 0.f;  // reference maximum (base 2, scaled), sum of this half
        bool begun = false;
        for (int i = 0; i < w.total; ++i) {
            const int kt = w.key_tile(i);
            if (!w.active(t, kt)) continue;
            const int j0 = kt * T, col = 64 * half;
            const bool masked = !(j0 + T - 1 <= p_lo && (p_hi - j0 < a.window || j0 + T <= a.sinks));
            const int hi = pos - j0 + 1, sk = a.sinks - j0, lo = pos >= a.window ? pos - a.window + 1 - j0 : -1;
            const int n = min(2, max(0, w.chunks(a, t, kt) - 2 * half));  // chunks of this half
            ok = ok && ws.wait(L::B_S + t, phs);
            phs ^= 1u;
            tc_fence_after();
            float s[2][32];
            float mx = -INFINITY;
            if (ok && n == 2) {
                tmem_ld32(sa + col, s[0]);
                tmem_ld32(sa + col + 32, s[1]);
                tmem_wait_ld();
                if (masked) {
                    mask32(s[0], visible_bits(col, lo, hi, sk), -INFINITY);
                    mask32(s[1], visible_bits(col + 32, lo, hi, sk), -INFINITY);
                }
                float x[4] = {s[0][0], s[0][1], s[1][0], s[1][1]};
#pragma unroll
                for (int e = 2; e < 32; e += 2) {
                    x[(e >> 1) & 1] = max3(x[(e >> 1) & 1], s[0][e], s[0][e + 1]);
                    x[2 + ((e >> 1) & 1)] = max3(x[2 + ((e >> 1) & 1)], s[1][e], s[1][e + 1]);
                }
                mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
            } else if (ok && n == 1) {
                tmem_ld32(sa + col, s[0]);
                tmem_wait_ld();
                mask32(s[0], visible_bits(col, lo, hi, sk), -INFINITY);
#pragma unroll
                for (int e = 0; e < 32; e += 2) mx = max3(mx, s[0][e], s[0][e + 1]);
            }
            mx = fmaxf(mx, other_half(mx)) * c;
            const bool move = mx > m + kSlack || (m == -INFINITY && mx > m);
            if (__any_sync(0xffffffffu, move)) {  // the same rows, and so the same vote, in both halves
                const float mn = move ? mx : m;
                const float f = move ? ex2_approx(m - mn) : 1.f;
                l *= f;
                m = mn;
                if (begun) {  // each half rescales every other 16 columns of O
                    for (int k = 16 * half; k < dvp; k += 32) {
                        float v[16];
                        tmem_ld16(oa + k, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) v[e] *= f;
                        tmem_st16(oa + k, v);
                    }
                }
            }
            begun = true;
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
            // P's half goes over the half of S it was made from (columns 0-31 and 64-95)
            if (n >= 1) probabilities(s[0], sa + col);
            if (n == 2) probabilities(s[1], sa + col + 16);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(ws.bar(L::B_P + t));
            float l0, l1;
            unpair2(add2(sum[0], sum[1]), l0, l1);
            l += l0 + l1;
        }
        l += other_half(l);
        ok = ok && ws.wait(L::B_O + t, pho);
        pho ^= 1u;
        tc_fence_after();
        const bool live = r < w.rows && ok;
        const float inv = 1.f / l;
        __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.o.p) + (size_t)w.b * a.o.sb + (size_t)head * a.o.sh + (size_t)r * a.o.st;
        for (int k = 16 * half; k < dvp; k += 32) {
            float v[16];
            tmem_ld16(oa + k, v);
            tmem_wait_ld();
            uint32_t u[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) u[e] = pack_bf16(v[2 * e] * inv, v[2 * e + 1] * inv);
            if (live && p.wide_out && k + 16 <= a.dv) {  // a whole 32-byte sector
                asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(o + k), "r"(u[0]), "r"(u[1]), "r"(u[2]),
                             "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
                             : "memory");
            } else if (live) {
                *reinterpret_cast<uint4 *>(o + k) = make_uint4(u[0], u[1], u[2], u[3]);
                if (k + 8 < a.dv) *reinterpret_cast<uint4 *>(o + k + 8) = make_uint4(u[4], u[5], u[6], u[7]);
            }
            __syncwarp();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(ws.bar(L::B_OE + t));
        if (live && half == 0 && a.lse) a.lse[((size_t)w.b * a.H + head) * a.n + r] = (m + log2f(l)) * kLn2;
    }
}

template <int DP>
__device__ __forceinline__ void mma_role(const Params &p, const Waits &ws, uint8_t *base, uint32_t tb) {
    using L = Lay<DP>;
    const Args &a = p.a;
    const int lane = threadIdx.x & 31;
    const uint32_t id_o = make_idesc(T, (a.dv + 15) & ~15, false, true);
    const bool wide = a.d > 64;
    tb = uniform(tb);
    uint32_t php[2] = {0, 0}, uses[2] = {0, 0};  // P's phase; items that used the tile
    int ring = 0;                                // ring index of this item's first key tile
    bool ok = true;
    auto slot = [&](int idx) { return base + L::OFF_RING + (idx % L::NS) * L::TILE; };
    auto full = [&](int idx) { return ws.wait(L::B_FULL + idx % L::NS, (uint32_t)(idx / L::NS) & 1u); };
    for (int item = blockIdx.x; item < p.items && ok; item += gridDim.x) {
        const Work w(p, item);
        bool pend[2] = {false, false}, begun[2] = {false, false}, q_here[2] = {false, false};
        for (int i = 0; i <= w.total && ok; ++i) {  // the last round only finishes O
            if (w.total == 0) break;
            const int kt = i < w.total ? w.key_tile(i) : -1;
            bool k_here = false, v_here = false;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if (pend[t] && ok) {
                    const int vi = ring + 2 * i - 1;
                    if (!v_here) {
                        ok = full(vi);
                        v_here = true;
                        // values behind the sequence may be anything, and 0 times that is not 0
                        const int live = w.len - w.key_tile(i - 1) * T;
                        if (ok && live < T) zero_rows<DP>(slot(vi), live, lane);
                    }
                    // O of the tile's last item has been read
                    if (ok && !begun[t] && uses[t] > 0) ok = ws.wait(L::B_OE + t, (uses[t] - 1) & 1u);
                    if (ok) ok = ws.wait(L::B_P + t, php[t]);
                    if (!ok) break;
                    php[t] ^= 1u;
                    tc_fence_after();
                    const int chunks = uniform(w.chunks(a, t, w.key_tile(i - 1)));
                    const uint64_t dv = make_sdesc(smem_u32(slot(vi)), T * 128u, 1024u);
                    const uint32_t o = tb + L::O0 + t * DP, s = tb + L::S0 + t * T;
                    mma_ts32(o, s, dv, id_o, begun[t]);
                    if (chunks > 1) mma_ts32(o, s + 16, dv + 256, id_o, true);
                    if (chunks > 2) mma_ts32(o, s + 64, dv + 512, id_o, true);
                    if (chunks > 3) mma_ts32(o, s + 80, dv + 768, id_o, true);
                    begun[t] = true;
                    pend[t] = false;
                    if (i == w.total || kt > (t ? w.hi[1] : w.hi[0])) {
                        umma_commit_warp(ws.bar(L::B_O + t));
                        ++uses[t];
                    }
                }
                if (i < w.total && ok && w.active(t, kt)) {
                    if (!k_here) {
                        ok = full(ring + 2 * i);
                        k_here = true;
                    }
                    if (ok && !q_here[t]) {
                        ok = ws.wait(L::B_Q + t, uses[t] & 1u);
                        q_here[t] = true;
                    }
                    if (!ok) break;
                    mma_kk<DP>(tb + L::S0 + t * T, base + L::OFF_Q + t * L::TILE, slot(ring + 2 * i),
                               make_idesc(T, 32 * uniform(w.chunks(a, t, kt)), false, false), wide);
                    umma_commit_warp(ws.bar(L::B_S + t));
                    pend[t] = true;
                    if (kt == (t ? w.hi[1] : w.hi[0])) umma_commit_warp(ws.bar(L::B_QE + t));
                }
            }
            if (!ok) break;
            if (i > 0) umma_commit_warp(ws.bar(L::B_EMPTY + (ring + 2 * i - 1) % L::NS));
            if (i < w.total) umma_commit_warp(ws.bar(L::B_EMPTY + (ring + 2 * i) % L::NS));
        }
        ring += 2 * w.total;
    }
    umma_commit_warp(ws.bar(L::B_FIN));  // every MMA issued completes before TMEM is released
    mbar_wait(ws.bar(L::B_FIN), 0u, ws.err);
    __syncwarp();
}

template <int DP>
__device__ __forceinline__ void tma_role(const Params &p, const Waits &ws, uint8_t *base) {
    using L = Lay<DP>;
    const Args &a = p.a;
    const bool one = (threadIdx.x & 31) == 0;
    uint32_t uses[2] = {0, 0};
    int idx = 0;
    bool ok = true;
    for (int item = blockIdx.x; item < p.items && ok; item += gridDim.x) {
        const Work w(p, item);
        for (int i = 0; i < 2 * w.total && ok; ++i, ++idx) {
            const int s = idx % L::NS, use = idx / L::NS;
            if (use > 0 && !(ok = ws.wait(L::B_EMPTY + s, (uint32_t)(use - 1) & 1u))) break;
            if (one) {
                mbar_expect_tx(ws.bar(L::B_FULL + s), L::TILE);
                const bool key = (i & 1) == 0;
                load_tile<DP>(base + L::OFF_RING + s * L::TILE, key ? &p.mk : &p.mv, key ? a.k : a.v, ws.bar(L::B_FULL + s),
                              w.key_tile(i >> 1) * T, w.hk, w.b);
            }
            __syncwarp();
            if (i > 0) continue;
#pragma unroll
            for (int t = 0; t < 2; ++t) {  // behind the first key tile, which needs no wait for the last item's Q
                if (!w.on[t] || !ok) continue;
                if (uses[t] > 0 && !(ok = ws.wait(L::B_QE + t, (uses[t] - 1) & 1u))) break;
                if (one) {
                    mbar_expect_tx(ws.bar(L::B_Q + t), L::TILE);
                    load_tile<DP>(base + L::OFF_Q + t * L::TILE, &p.mq, a.q, ws.bar(L::B_Q + t), w.row[t], w.h[t], w.b);
                }
                ++uses[t];
                __syncwarp();
            }
        }
    }
    // nothing may land after the CTA has ended (only an aborted CTA still has copies in flight)
    for (int t = 0; t < 2; ++t)
        if (uses[t] > 0) mbar_wait(ws.bar(L::B_Q + t), (uses[t] - 1) & 1u, ws.err);
    for (int k = max(0, idx - L::NS); k < idx; ++k)
        mbar_wait(ws.bar(L::B_FULL + k % L::NS), (uint32_t)(k / L::NS) & 1u, ws.err);
    __syncwarp();
}

template <int DP>
__global__ void __launch_bounds__(kThreads, 1) window_fwd_kernel(const __grid_constant__ Params p) {
    using L = Lay<DP>;
    extern __shared__ __align__(1024) uint8_t base[];
    Waits ws{reinterpret_cast<uint64_t *>(base + L::OFF_BAR), nullptr, p.a.err};
    uint32_t *misc = reinterpret_cast<uint32_t *>(base + L::OFF_BAR + L::NB * 8);  // TMEM base, abort
    ws.abort_p = reinterpret_cast<volatile int *>(misc + 1);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        misc[1] = 0u;
        for (int i = 0; i < L::NB; ++i)
            mbar_init(ws.bar(i), (i >= L::B_P && i < L::B_P + 2) || (i >= L::B_OE && i < L::B_OE + 2) ? 8 : 1);
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
        if (warp == kWarpTma) tma_role<DP>(p, ws, base);
        if (warp == kWarpMma) mma_role<DP>(p, ws, base, tb);
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        softmax_role<DP>(p, ws, base, tb, warp >> 3, (warp >> 2) & 1);
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
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(window_fwd_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM);
    if (e != cudaSuccess) return e;
    p.items = p.pair_heads ? a.B * (a.H / 2) * ((a.n + T - 1) / T) : a.B * a.H * ((a.n + 2 * T - 1) / (2 * T));
    window_fwd_kernel<DP><<<p.items < sms ? p.items : sms, kThreads, L::SMEM, st>>>(p);
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
    p.wide_out = reinterpret_cast<uintptr_t>(a.o.p) % 32 == 0 && a.o.sb % 16 == 0 && a.o.sh % 16 == 0 && a.o.st % 16 == 0;
    return a.d <= 64 && a.dv <= 64 ? launch<64>(p, st) : launch<128>(p, st);
}

}  // namespace win
}  // namespace hla
