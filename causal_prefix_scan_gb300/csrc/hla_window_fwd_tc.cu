// hla_window_fwd_tc.cu -- forward of windowed attention for bf16 on the tensor cores.
//
// Work items: two tiles of 128 queries that share their keys -- the same rows of two heads of
// one group, or two neighbouring row tiles of a head -- walk the key tiles they can see: per
// key tile and query tile S = Q K^T into TMEM (128 fp32 columns), the softmax in fp32 with a
// running maximum and sum, P packed to bf16 over S's own columns, O += P V with P read from
// TMEM.  While the softmax of one query tile runs, the tensor cores work on the other.
// Persistent: one CTA per SM goes through the items, so that an item's output and the next
// one's first loads and products overlap (552 -> 523 us on h32 n16384 d128 w2048).  Warps 0-7:
// softmax, four warps per query tile, one row per thread, so that maxima and sums need no
// exchange; warp 8: MMA; warp 9: TMA into a ring of key and value tiles.
//
// The MMA warp takes the two tiles in strict turns, P V of one directly before its next S:
// the tiles stay half a period apart, and the tensor cores have one tile's products while the
// other's softmax runs.  With a warp per tile, or in the order in which P comes, they fall
// into step (576 and 656 us against 444).  A key tile takes both query tiles together some
// 3,500 cycles: their four products are 58 % of that, the waits between softmax and MMA the rest.
//
// Measured: H32 Hkv8 n16384 d128 w2048 450 us, 1,150 TFLOP/s (60 % of cuBLAS' peak rate); B4 H8
// n2048 d64 w256 27 us, where an item is four or five key tiles and the pipeline hardly fills.
//
// The running maximum used in the exponent only moves when a row's maximum passes it by
// more than 2^8: P then stays below 2^8, and O in TMEM is rescaled a few times per row
// instead of at every key tile.  P is rounded to bf16 for the second product, half a step
// (2^-8) of each probability; the sum that divides O is of the unrounded ones.
#include "hla_window_tc.cuh"

namespace hla {
namespace win {
namespace {

using namespace tcw;

// Registers per thread of the softmax warpgroups, which hold a row of S, and of the third
// warpgroup: with the 168 that each of the 384 threads is launched with, 2 x 200 + 104 = 3 x 168.
constexpr int kThreads = 384, kWarpMma = 8, kWarpTma = 9, kRegsSoftmax = 200, kRegsOther = 104;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f, kSlack = 8.f;

struct Params {
    Args a;
    CUtensorMap mq, mk, mv;
    int pair_heads;  // the two tiles are two heads of a group (else two row tiles of a head)
    int items;
};

template <int DP>
struct Lay {
    static constexpr int TILE = T * DP * 2;
    static constexpr int NS = DP == 64 ? 8 : 4;  // ring slots
    static constexpr int OFF_Q = 0, OFF_RING = 2 * TILE, OFF_STAGE = OFF_RING + NS * TILE;  // 4 KB per softmax warp
    static constexpr int OFF_BAR = OFF_STAGE + 8 * 4096;
    // barriers of a query tile: Q landed, Q free, S ready, P ready, O ready, O read
    static constexpr int B_FULL = 0, B_EMPTY = B_FULL + NS, B_Q = B_EMPTY + NS, B_QE = B_Q + 2, B_S = B_QE + 2, B_P = B_S + 2,
                         B_O = B_P + 2, B_OE = B_O + 2, B_FIN = B_OE + 2, B_RAW = B_FIN + 1, NB = B_RAW + 1;
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
        len = (int)uniform(length_of(a, b));
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

template <int DP>
__device__ __forceinline__ void softmax_role(const Params &p, const Waits &ws, uint8_t *smem, uint32_t tb, int t) {
    using L = Lay<DP>;
    const Args &a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rr = (warp & 3) * 32 + lane;
    const uint32_t quad = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t sa = tb + quad + L::S0 + t * T;         // S of the tile, P over it
    const uint32_t oa = tb + quad + L::O0 + t * DP;
    uint8_t *stage = smem + L::OFF_STAGE + warp * 4096;
    const float c = a.scale * kLog2e;
    const int dvp = (a.dv + 15) & ~15;
    uint32_t phs = 0, pho = 0;
    for (int item = blockIdx.x; item < p.items; item += gridDim.x) {
        const Work w(p, item);
        if (!(t ? w.on[1] : w.on[0])) continue;
        const int row0 = t ? w.row[1] : w.row[0], head = t ? w.h[1] : w.h[0];
        const int r = row0 + rr, pos = a.p0 + r, p_lo = a.p0 + row0, p_hi = p_lo + T - 1;
        float m = -INFINITY, l = 0.f;  // reference maximum (base 2, scaled), sum
        bool begun = false;
        for (int i = 0; i < w.total; ++i) {
            const int kt = w.key_tile(i);
            if (!w.active(t, kt)) continue;
            const int j0 = kt * T, chunks = w.chunks(a, t, kt);
            const bool masked = !(j0 + T - 1 <= p_lo && (p_hi - j0 < a.window || j0 + T <= a.sinks));
            const int hi = pos - j0 + 1, sk = a.sinks - j0, lo = pos >= a.window ? pos - a.window + 1 - j0 : -1;
            if (!ws.wait(L::B_S + t, phs)) return;
            phs ^= 1u;
            tc_fence_after();
            float mx = -INFINITY;
            float s[4][32];
            if (chunks == 4) {  // a whole tile is held in registers
#pragma unroll
                for (int k = 0; k < 4; ++k) tmem_ld32(sa + 32 * k, s[k]);
                tmem_wait_ld();
                if (masked) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) mask32(s[k], visible_bits(32 * k, lo, hi, sk), -INFINITY);
                }
                float x[4] = {s[0][0], s[1][0], s[2][0], s[3][0]};
#pragma unroll
                for (int e = 1; e < 31; e += 2)
#pragma unroll
                    for (int k = 0; k < 4; ++k) x[k] = max3(x[k], s[k][e], s[k][e + 1]);
                mx = max3(max3(x[0], s[0][31], x[1]), max3(s[1][31], x[2], s[2][31]), fmaxf(x[3], s[3][31]));
            } else {
#pragma unroll 1
                for (int k = 0; k < chunks; ++k) {
                    tmem_ld32(sa + 32 * k, s[0]);
                    tmem_wait_ld();
                    mask32(s[0], visible_bits(32 * k, lo, hi, sk), -INFINITY);
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
                if (begun) {
                    for (int k = 0; k < dvp; k += 16) {
                        float v[16];
                        tmem_ld16(oa + k, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) v[e] *= f;
                        tmem_st16(oa + k, v);
                    }
                    tmem_wait_st();
                }
            }
            begun = true;
            const float base = m == -INFINITY ? 0.f : m;
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
            // 32 columns of P.  One operation at a time: as pairs (fma.rn.f32x2, add.rn.f32x2) they
            // take as long in the pipe, and moves to form the pairs besides (5.1 cycles per
            // element against 3.4)
            auto probabilities = [&](const float(&v)[32], uint32_t to) {
                float pk[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float x = ex2_approx(fmaf(v[2 * e], c, -base)), y = ex2_approx(fmaf(v[2 * e + 1], c, -base));
                    sum[e & 1] += x;
                    sum[2 + (e & 1)] += y;
                    pk[e] = __uint_as_float(pack_bf16(x, y));
                }
                tmem_st16(to, pk);
            };
            if (chunks == 4) {
                probabilities(s[0], sa);
                probabilities(s[1], sa + 16);
                probabilities(s[2], sa + 32);
                probabilities(s[3], sa + 48);
            } else {
#pragma unroll 1
                for (int k = 0; k < chunks; ++k) {
                    tmem_ld32(sa + 32 * k, s[0]);
                    tmem_wait_ld();
                    mask32(s[0], visible_bits(32 * k, lo, hi, sk), -INFINITY);
                    probabilities(s[0], sa + 16 * k);
                }
            }
            // P is handed over whole: in halves the MMA warp waited for the second half while the
            // other tile's P was ready (484 against 442 us on h32 n16384 d128 w2048)
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(ws.bar(L::B_P + t));
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        }
        if (!ws.wait(L::B_O + t, pho)) return;
        pho ^= 1u;
        tc_fence_after();
        const float inv = 1.f / l;
        __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.o.p) + (size_t)w.b * a.o.sb + (size_t)head * a.o.sh +
                           (size_t)(row0 + (warp & 3) * 32) * a.o.st;
#pragma unroll 1
        for (int c0 = 0; c0 < a.dv; c0 += 64)
            store_rows<64>(stage, oa + c0, inv, o, a.o.st, w.rows - row0 - (warp & 3) * 32, c0, a.dv);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(ws.bar(L::B_OE + t));
        if (r < w.rows && a.lse) a.lse[((size_t)w.b * a.H + head) * a.n + r] = (m + log2f(l)) * kLn2;
    }
}

template <int DP>
__device__ __forceinline__ void mma_role(const Params &p, const Waits &ws, uint8_t *base, uint32_t tb) {
    using L = Lay<DP>;
    const Args &a = p.a;
    const uint32_t id_o = make_idesc(T, (a.dv + 15) & ~15, false, true), id_s = make_idesc(T, T, false, false);
    const bool wide = DP > 64 && a.d > 64;
    constexpr uint32_t STEP = L::TILE >> 4;
    const uint64_t q_desc = kmajor(base + L::OFF_Q), k_desc = kmajor(base + L::OFF_RING), v_desc = mnmajor(base + L::OFF_RING);
    uint32_t php[2] = {0, 0}, uses[2] = {0, 0};  // P's phase; items that used the tile
    Ring<L::NS> ring;                            // the next key tile's slot; its values' is the one behind
    bool ok = true;
    for (int item = blockIdx.x; item < p.items && ok; item += gridDim.x) {
        const Work w(p, item);
        int chunks[2] = {0, 0};  // of the S that the next P comes from; 0: none
        bool begun[2] = {false, false}, q_here[2] = {false, false};
        uint32_t v_slot = 0, v_phase = 0;
        for (int i = 0; i <= w.total && w.total > 0; ++i) {  // the last round only finishes O
            const int kt = i < w.total ? w.key_tile(i) : 0x7fffffff;
            const uint32_t k_slot = ring.slot, k_phase = ring.phase;
            const uint64_t kd = k_desc + k_slot * STEP, vd = v_desc + v_slot * STEP;
            if (i < w.total && !(ok = ws.wait(L::B_FULL + k_slot, k_phase))) break;
            if (i > 0 && !(ok = ws.wait(L::B_FULL + v_slot, v_phase))) break;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const uint32_t s = tb + L::S0 + t * T, o = tb + L::O0 + t * DP;
                const int next = w.active(t, kt) ? w.chunks(a, t, kt) : 0;
                const uint32_t id = next == 4 ? id_s : make_idesc(T, 32 * next, false, false);
                if (next > 0 && !q_here[t]) {
                    if (!(ok = ws.wait(L::B_Q + t, uses[t] & 1u))) break;
                    q_here[t] = true;
                }
                if (chunks[t] > 0) {
                    // before the first product: O of the tile's last item has been read
                    if (!begun[t] && uses[t] > 0 && !(ok = ws.wait(L::B_OE + t, (uses[t] - 1) & 1u))) break;
                    if (!(ok = ws.wait(L::B_P + t, php[t]))) break;
                    tc_fence_after();
                    mma_ts32(o, s, vd, id_o, begun[t]);
                    if (chunks[t] > 1) mma_ts32(o, s + 16, vd + 256, id_o, true);
                    if (chunks[t] > 2) mma_ts32(o, s + 32, vd + 512, id_o, true);
                    if (chunks[t] > 3) mma_ts32(o, s + 48, vd + 768, id_o, true);
                    php[t] ^= 1u;
                    begun[t] = true;
                }
                if (next > 0) {
                    mma_kk<DP>(s, q_desc + t * STEP, kd, id, wide);
                    umma_commit_warp(ws.bar(L::B_S + t));
                    if (kt == w.hi[t]) umma_commit_warp(ws.bar(L::B_QE + t));
                }
                if (chunks[t] > 0 && kt > w.hi[t]) {
                    umma_commit_warp(ws.bar(L::B_O + t));
                    ++uses[t];
                }
                chunks[t] = next;
            }
            if (!ok) break;
            if (i > 0) umma_commit_warp(ws.bar(L::B_EMPTY + v_slot));
            if (i < w.total) {
                umma_commit_warp(ws.bar(L::B_EMPTY + k_slot));
                ring.next();
                v_slot = ring.slot;
                v_phase = ring.phase;
                ring.next();
            }
        }
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
    uint32_t uses[2] = {0, 0}, raw = 0;
    Ring<L::NS> ring;
    int loads = 0;
    bool ok = true;
    for (int item = blockIdx.x; item < p.items && ok; item += gridDim.x) {
        const Work w(p, item);
        for (int i = 0; i < 2 * w.total && ok; ++i) {
            const uint32_t s = ring.slot;
            if (loads >= L::NS && !(ok = ws.wait(L::B_EMPTY + s, ring.phase ^ 1u))) break;
            const bool key = (i & 1) == 0;
            const int kt = w.key_tile(i >> 1), live = w.len - kt * T;
            const bool clean = !key && live < T;  // values behind the sequence: zeros before the MMAs see them
            const int full = clean ? L::B_RAW : L::B_FULL + (int)s;
            if (one) {
                mbar_expect_tx(ws.bar(full), L::TILE);
                load_tile<DP>(base + L::OFF_RING + s * L::TILE, key ? &p.mk : &p.mv, key ? a.k : a.v, ws.bar(full), kt * T, w.hk, w.b);
            }
            __syncwarp();
            if (clean) {
                if (!(ok = ws.wait(L::B_RAW, raw))) break;
                raw ^= 1u;
                zero_rows<DP>(base + L::OFF_RING + s * L::TILE, live, threadIdx.x & 31);
                if (one) mbar_arrive(ws.bar(L::B_FULL + s));
            }
            ring.next();
            ++loads;
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
    for (int k = max(0, loads - L::NS); k < loads; ++k)
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
            mbar_init(ws.bar(i), (i >= L::B_P && i < L::B_P + 2) || (i >= L::B_OE && i < L::B_OE + 2) ? 4 : 1);
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
        if (warp == kWarpMma) mma_role<DP>(p, ws, base, uniform(tb));
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        softmax_role<DP>(p, ws, base, tb, warp >> 2);
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
    // share most of theirs (H32 Hkv8 n16384 w2048 as heads 453 us, as row tiles 475)
    p.pair_heads = a.G % 2 == 0;
    return a.d <= 64 && a.dv <= 64 ? launch<64>(p, st) : launch<128>(p, st);
}

}  // namespace win
}  // namespace hla
