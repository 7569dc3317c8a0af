// hla_window_step.cu -- one token of windowed attention per sequence over its ring cache
// of sinks + window slots, the new key and value written into their slot by the same launch.
//
// Bound by HBM: the visible slots of K and V are read once for all query heads of a
// key/value head.  Few (sequence, head) pairs would leave most SMs idle, so a cluster of
// up to 16 CTAs shares the slots of one pair: each runs a softmax over its own tiles of 64
// slots, and the cluster joins the partial results through distributed shared memory, in
// the order of the ranks (one launch, no workspace, the same bits on every call).
//
// Measured, bf16, 32 query and 8 key/value heads of width 128: 64 sequences with 1,024 + 16 slots
// (ragged) 52 us, 4.5 TB/s; one sequence with 4,096 + 16 slots 14.8 us, 1.1 TB/s, which is the
// latency of a launch in clusters, two dependent loads and the join, not bandwidth.
#include "hla_window.h"

#include <cooperative_groups.h>

namespace cg = cooperative_groups;

namespace hla {
namespace win {
namespace {

constexpr int kThreads = 256, TS = 64, HG = 8;  // slots of a tile, query heads of a CTA
constexpr float kLog2e = 1.4426950408889634f;

template <typename T>
__device__ __forceinline__ float ldf(const void *p, size_t i);
template <>
__device__ __forceinline__ float ldf<float>(const void *p, size_t i) { return static_cast<const float *>(p)[i]; }
template <>
__device__ __forceinline__ float ldf<__nv_bfloat16>(const void *p, size_t i) {
    return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}
template <typename T>
__device__ __forceinline__ void stf(void *p, size_t i, float x);
template <>
__device__ __forceinline__ void stf<float>(void *p, size_t i, float x) { static_cast<float *>(p)[i] = x; }
template <>
__device__ __forceinline__ void stf<__nv_bfloat16>(void *p, size_t i, float x) {
    static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(x);
}

// What the cluster's CTAs show each other.
template <int DP>
struct Partial {
    float m[HG], l[HG];
    float o[HG][DP];
};

// The partial results of the cluster's CTAs, joined: rank r writes the output elements
// r, r + split, ... (in units of the block).  Heads h0 .. h0 + heads - 1.
template <typename T, int DP>
__device__ __forceinline__ void join(const StepArgs &a, Partial<DP> &mine, int b, int h0, int heads) {
    cg::cluster_group cl = cg::this_cluster();
    const int ranks = (int)cl.num_blocks(), rank = (int)cl.block_rank();
    cl.sync();
    for (int e = rank * kThreads + threadIdx.x; e < heads * DP; e += ranks * kThreads) {
        const int h = e / DP, c = e % DP;
        if (c >= a.dv) continue;
        float m = -INFINITY, l = 0.f, o = 0.f;
        for (int r = 0; r < ranks; ++r) m = fmaxf(m, cl.map_shared_rank(&mine, r)->m[h]);
        for (int r = 0; r < ranks; ++r) {
            const Partial<DP> *x = cl.map_shared_rank(&mine, r);
            const float w = exp2f(x->m[h] - m);
            l = fmaf(w, x->l[h], l);
            o = fmaf(w, x->o[h][c], o);
        }
        stf<T>(a.o.p, (size_t)b * a.o.sb + (size_t)(h0 + h) * a.o.sh + c, o / l);
    }
    cl.sync();  // no CTA leaves while another reads its shared memory
}

// This CTA's place and its sequence's token.
struct Place {
    int b, hk, h0, heads;
    long long p;
    int slots, slot;  // visible slots, the new token's slot
    __device__ Place(const StepArgs &a) {
        const int groups = (a.G + HG - 1) / HG;
        const int u = blockIdx.x / a.split, g = u % groups;
        hk = u / groups % a.Hkv;
        b = u / groups / a.Hkv;
        h0 = hk * a.G + g * HG;
        heads = min(HG, a.G - g * HG);
        p = a.pos[b];
        const long long cap = (long long)a.sinks + a.window;
        slots = (int)(p < cap ? p + 1 : cap);
        slot = p < 0 ? 0 : p < a.sinks ? (int)p : a.sinks + (int)((p - a.sinks) % a.window);
    }
};

// ------------------------------------------------------------ CUDA cores
// fp32 caches, and bf16 ones whose rows are not multiples of 16 bytes.  Scores: thread =
// (slot, quarter of the width) for all heads; values: thread = (4 columns, 4 heads,
// slots of one residue), so each K and V element leaves shared memory about once per
// four heads.
template <typename T, int DP>
__global__ void __launch_bounds__(kThreads) step_kernel(const StepArgs a) {
    constexpr int LD = DP + 4, QW = DP / 4, CW = DP / 4, SR = kThreads / (CW * 2);  // SR slot residues
    extern __shared__ __align__(16) float smem[];
    float *K = smem, *V = K + TS * LD, *q = V + TS * LD, *part = q + HG * DP, *P = part + 4 * HG * TS;
    __shared__ Partial<DP> out;
    __shared__ float fac[HG];
    const Place w(a);
    if (w.p < 0) return;  // uniform over the cluster
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = blockIdx.x % a.split, ranks = a.split;
    for (int e = tid; e < HG * DP; e += kThreads) {
        const int h = e / DP, c = e % DP;
        q[e] = h < w.heads && c < a.d
                   ? ldf<T>(a.q.p, (size_t)w.b * a.q.sb + (size_t)(w.h0 + h) * a.q.sh + c) * (a.scale * kLog2e)
                   : 0.f;
    }
    float m = -INFINITY, l = 0.f;  // of head `warp`, the same in all lanes
    float acc[4][4] = {};          // [head][column]
    const int cq = tid % CW, hh = tid / CW % 2, sr = tid / (CW * 2);
    const size_t kc0 = (size_t)w.b * a.kc.sb + (size_t)w.hk * a.kc.sh, vc0 = (size_t)w.b * a.vc.sb + (size_t)w.hk * a.vc.sh;
    const size_t kn = (size_t)w.b * a.k.sb + (size_t)w.hk * a.k.sh, vn = (size_t)w.b * a.v.sb + (size_t)w.hk * a.v.sh;
    const bool writer = w.h0 == w.hk * a.G;  // one CTA of the pair's head groups writes the new row
    for (int t = rank; t * TS < w.slots; t += ranks) {
        const int s0 = t * TS, cnt = min(TS, w.slots - s0);
        __syncthreads();
        for (int e = tid; e < TS * DP; e += kThreads) {
            const int s = e / DP, c = e % DP;
            float kx = 0.f, vx = 0.f;
            if (s < cnt) {
                if (s0 + s == w.slot) {  // the new token: from the arguments, and into the cache
                    if (c < a.d) {
                        kx = ldf<T>(a.k.p, kn + c);
                        if (writer) stf<T>(a.kc.p, kc0 + (size_t)(s0 + s) * a.kc.st + c, kx);
                    }
                    if (c < a.dv) {
                        vx = ldf<T>(a.v.p, vn + c);
                        if (writer) stf<T>(a.vc.p, vc0 + (size_t)(s0 + s) * a.vc.st + c, vx);
                    }
                } else {
                    if (c < a.d) kx = ldf<T>(a.kc.p, kc0 + (size_t)(s0 + s) * a.kc.st + c);
                    if (c < a.dv) vx = ldf<T>(a.vc.p, vc0 + (size_t)(s0 + s) * a.vc.st + c);
                }
            }
            K[s * LD + c] = kx;
            V[s * LD + c] = vx;
        }
        __syncthreads();
        {
            const int s = tid & (TS - 1), part_k = tid / TS;
            float d[HG] = {};
#pragma unroll
            for (int c = 0; c < QW; c += 4) {
                const float4 x = *reinterpret_cast<const float4 *>(K + s * LD + part_k * QW + c);
#pragma unroll
                for (int h = 0; h < HG; ++h) {
                    const float4 y = *reinterpret_cast<const float4 *>(q + h * DP + part_k * QW + c);
                    d[h] += x.x * y.x + x.y * y.y + x.z * y.z + x.w * y.w;
                }
            }
#pragma unroll
            for (int h = 0; h < HG; ++h) part[(part_k * HG + h) * TS + s] = d[h];
        }
        __syncthreads();
        {  // softmax of head `warp` over the tile
            float s[2], mx = m;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int e = lane + 32 * i;
                s[i] = -INFINITY;
                if (e < cnt)
                    s[i] = part[(0 * HG + warp) * TS + e] + part[(1 * HG + warp) * TS + e] + part[(2 * HG + warp) * TS + e] +
                           part[(3 * HG + warp) * TS + e];
                mx = fmaxf(mx, s[i]);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const float base = mx == -INFINITY ? 0.f : mx, f = exp2f(m - base);
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float e = exp2f(s[i] - base);
                P[(lane + 32 * i) * HG + warp] = e;
                sum += e;
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            l = l * f + sum;
            m = mx;
            if (lane == 0) fac[warp] = f;
        }
        __syncthreads();
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            const float f = fac[hh * 4 + h];
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[h][c] *= f;
        }
        for (int s = sr; s < TS; s += SR) {
            const float4 p = *reinterpret_cast<const float4 *>(P + s * HG + hh * 4);
            const float4 v = *reinterpret_cast<const float4 *>(V + s * LD + cq * 4);
            const float ph[4] = {p.x, p.y, p.z, p.w}, vv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int h = 0; h < 4; ++h)
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[h][c] = fmaf(ph[h], vv[c], acc[h][c]);
        }
    }
    // the slot residues of the CTA, added in order
    if (lane == 0) {
        out.m[warp] = m;
        out.l[warp] = l;
    }
    for (int r = 0; r < SR; ++r) {
        __syncthreads();
        if (sr == r) {
#pragma unroll
            for (int h = 0; h < 4; ++h)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float &x = out.o[hh * 4 + h][cq * 4 + c];
                    x = r ? x + acc[h][c] : acc[h][c];
                }
        }
    }
    __syncthreads();
    join<T, DP>(a, out, w.b, w.h0, w.heads);
}

// ------------------------------------------------------------ tensor cores
// bf16 caches with 16-byte rows.  A warp takes 16 slots at a time, keeps its own running
// maximum, sum and O for 8 heads, and needs no shared memory until the end: K and V go from
// global memory straight into the operand registers of mma.m16n8k16, 16 bytes per load.
//   S^T [16 slots x 8 heads] = K Q^T: rows g, g + 8 of K; the 16-byte chunk 4 c + q of a row
//     serves two contraction steps (the order of the contraction index is free, Q's is the same);
//   P^T passes from the accumulator's layout to that of the second operand by an 8 x 8
//     transpose of packed pairs (movmatrix);
//   O^T [16 columns x 8 heads] += V^T P^T: a thread loads four rows' chunk of columns 8 g ..
//     8 g + 7 and packs pairs of rows; row g and g + 8 of product t are columns 8 g + 2 t, + 1.
// (lane = 4 g + q.)  mma.sync suffices: the work per byte is that of 8 heads, and the loads
// bound it (on the CUDA cores, step_kernel, the two sizes above take 852 and 64 us); tcgen05 would want 128 rows of queries and the operands staged in shared memory.
// The next 16 slots' K is loaded while this P is formed, their V while O is added up, so
// a warp has 4 to 8 KB on their way at all times.
constexpr int kWarps = 8, GS = 16;

HLA_DEVICE void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
HLA_DEVICE uint32_t transpose8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
HLA_DEVICE uint4 load16(const __nv_bfloat16 *p) {  // streamed: read once
    uint4 u;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                 : "l"(p));
    return u;
}

template <int DP>
__global__ void __launch_bounds__(kThreads, 2) step_mma_kernel(const StepArgs a) {
    constexpr int KC = DP / 32, VB = DP / 64;  // 16-byte chunks of a K row per thread, 64-column blocks
    __shared__ Partial<DP> part[kWarps];
    __shared__ Partial<DP> out;
    const Place w(a);
    if (w.p < 0) return;  // uniform over the cluster
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
    const int rank = blockIdx.x % a.split, step = a.split * kWarps * GS;
    using bf = __nv_bfloat16;
    const bf *kc = static_cast<const bf *>(a.kc.p) + (size_t)w.b * a.kc.sb + (size_t)w.hk * a.kc.sh;
    const bf *vc = static_cast<const bf *>(a.vc.p) + (size_t)w.b * a.vc.sb + (size_t)w.hk * a.vc.sh;
    const bf *kn = static_cast<const bf *>(a.k.p) + (size_t)w.b * a.k.sb + (size_t)w.hk * a.k.sh;
    const bf *vn = static_cast<const bf *>(a.v.p) + (size_t)w.b * a.v.sb + (size_t)w.hk * a.v.sh;
    if (rank == 0 && w.h0 == w.hk * a.G) {  // the new row goes into the cache; readers take it from k, v
        bf *ko = static_cast<bf *>(a.kc.p) + (kc - static_cast<const bf *>(a.kc.p)) + (size_t)w.slot * a.kc.st;
        bf *vo = static_cast<bf *>(a.vc.p) + (vc - static_cast<const bf *>(a.vc.p)) + (size_t)w.slot * a.vc.st;
        if (tid < a.d) ko[tid] = kn[tid];
        if (tid >= 128 && tid - 128 < a.dv) vo[tid - 128] = vn[tid - 128];
    }
    // Q as the second operand: head g, the chunks of K's rows that this thread loads
    uint32_t qb[KC][4];
    {
        const bf *qr = static_cast<const bf *>(a.q.p) + (size_t)w.b * a.q.sb + (size_t)(w.h0 + g) * a.q.sh;
#pragma unroll
        for (int c = 0; c < KC; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int x = (4 * c + q) * 8 + 2 * e;
                uint32_t lo = 0, hi = 0;
                if (g < w.heads && x < a.d) {
                    lo = __bfloat16_as_ushort(qr[x]);
                    hi = __bfloat16_as_ushort(qr[x + 1]);
                }
                qb[c][e] = lo | (hi << 16);
            }
    }
    const float sc = a.scale * kLog2e;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // heads 2 q, 2 q + 1 (l: this thread's slots)
    float o[VB * 4][4] = {};
    uint4 kr[2][KC], vr[4][VB];
    auto row = [&](const bf *cache, const bf *fresh, long long st, int s) {
        return s == w.slot ? fresh : cache + (size_t)s * st;
    };
    auto load_k = [&](int s0) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int s = s0 + g + 8 * r;
            const bf *p = row(kc, kn, a.kc.st, s);
#pragma unroll
            for (int c = 0; c < KC; ++c)
                kr[r][c] = s < w.slots && (4 * c + q) * 8 < a.d ? load16(p + (4 * c + q) * 8) : make_uint4(0, 0, 0, 0);
        }
    };
    auto load_v = [&](int s0) {  // rows 2 q, 2 q + 1, 2 q + 8, 2 q + 9; zeros where no slot is visible
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int s = s0 + 2 * q + (r & 1) + 8 * (r >> 1);
            const bf *p = row(vc, vn, a.vc.st, s);
#pragma unroll
            for (int c = 0; c < VB; ++c)
                vr[r][c] = s < w.slots && 64 * c + 8 * g < a.dv ? load16(p + 64 * c + 8 * g) : make_uint4(0, 0, 0, 0);
        }
    };
    int s0 = (rank * kWarps + warp) * GS;
    if (s0 < w.slots) {
        load_k(s0);
        load_v(s0);
    }
    for (; s0 < w.slots; s0 += step) {
        float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < KC; ++c) {
            const uint32_t a0[4] = {kr[0][c].x, kr[1][c].x, kr[0][c].y, kr[1][c].y};
            const uint32_t a1[4] = {kr[0][c].z, kr[1][c].z, kr[0][c].w, kr[1][c].w};
            mma16816(s, a0, qb[c][0], qb[c][1]);
            mma16816(s, a1, qb[c][2], qb[c][3]);
        }
        const bool more = s0 + step < w.slots;
        if (more) load_k(s0 + step);
        // s[0], s[1]: slot g, heads 2 q, 2 q + 1; s[2], s[3]: slot g + 8
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = s0 + g + 8 * (i >> 1) < w.slots ? s[i] * sc : -INFINITY;
        // the reference maximum moves only when a score passes it by 2^8: P stays below 2^8
        const bool move = s[0] > m[0] + 8.f || s[2] > m[0] + 8.f || s[1] > m[1] + 8.f || s[3] > m[1] + 8.f;
        if (__any_sync(0xffffffffu, move)) {
            float f[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float x = fmaxf(m[i], fmaxf(s[i], s[i + 2]));
#pragma unroll
                for (int k = 4; k < 32; k <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, k));
                f[i] = x == -INFINITY ? 1.f : ex2_approx(m[i] - x);
                m[i] = x;
                l[i] *= f[i];
            }
#pragma unroll
            for (int t = 0; t < VB * 4; ++t) {
                o[t][0] *= f[0];
                o[t][1] *= f[1];
                o[t][2] *= f[0];
                o[t][3] *= f[1];
            }
        }
        const float b0 = m[0] == -INFINITY ? 0.f : m[0], b1 = m[1] == -INFINITY ? 0.f : m[1];
        s[0] = ex2_approx(s[0] - b0);
        s[1] = ex2_approx(s[1] - b1);
        s[2] = ex2_approx(s[2] - b0);
        s[3] = ex2_approx(s[3] - b1);
        l[0] += s[0] + s[2];
        l[1] += s[1] + s[3];
        const uint32_t p0 = transpose8(pack_bf16(s[0], s[1])), p1 = transpose8(pack_bf16(s[2], s[3]));
#pragma unroll
        for (int c = 0; c < VB; ++c) {
            const uint32_t *r0 = reinterpret_cast<const uint32_t *>(&vr[0][c]), *r1 = reinterpret_cast<const uint32_t *>(&vr[1][c]);
            const uint32_t *r2 = reinterpret_cast<const uint32_t *>(&vr[2][c]), *r3 = reinterpret_cast<const uint32_t *>(&vr[3][c]);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const uint32_t f[4] = {__byte_perm(r0[t], r1[t], 0x5410), __byte_perm(r0[t], r1[t], 0x7632),
                                       __byte_perm(r2[t], r3[t], 0x5410), __byte_perm(r2[t], r3[t], 0x7632)};
                mma16816(o[4 * c + t], f, p0, p1);
            }
        }
        if (more) load_v(s0 + step);
    }
    // the warp's result, then the CTA's: the warps in order
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int k = 4; k < 32; k <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], k);
        if (g == 0) {
            part[warp].m[2 * q + i] = m[i];
            part[warp].l[2 * q + i] = l[i];
        }
#pragma unroll
        for (int t = 0; t < VB * 4; ++t) {
            const int col = 64 * (t >> 2) + 8 * g + 2 * (t & 3);
            part[warp].o[2 * q + i][col] = o[t][i];
            part[warp].o[2 * q + i][col + 1] = o[t][i + 2];
        }
    }
    __syncthreads();
    for (int e = tid; e < HG * DP; e += kThreads) {
        const int h = e / DP, c = e % DP;
        float mx = -INFINITY, lx = 0.f, ox = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) mx = fmaxf(mx, part[k].m[h]);
        const float base = mx == -INFINITY ? 0.f : mx;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            const float f = ex2_approx(part[k].m[h] - base);
            lx = fmaf(f, part[k].l[h], lx);
            ox = fmaf(f, part[k].o[h][c], ox);
        }
        out.o[h][c] = ox;
        if (c == 0) {
            out.m[h] = mx;
            out.l[h] = lx;
        }
    }
    __syncthreads();
    join<bf, DP>(a, out, w.b, w.h0, w.heads);
}

// One cluster of a.split CTAs per (sequence, key/value head, group of HG heads).
template <typename K>
cudaError_t launch_clusters(K fn, const StepArgs &a, size_t bytes, cudaStream_t st) {
    cudaError_t e = cudaSuccess;
    if (bytes > 0) e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess && a.split > 8) e = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((size_t)a.split * a.B * a.Hkv * ((a.G + HG - 1) / HG)), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = a.split;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, a);
}

template <typename T>
cudaError_t by_width(const StepArgs &a, cudaStream_t st) {
    const int w = a.d > a.dv ? a.d : a.dv;
    const auto bytes = [](int dp) { return (size_t)(2 * TS * (dp + 4) + HG * dp + 4 * HG * TS + TS * HG) * 4; };
    if (w <= 32) return launch_clusters(step_kernel<T, 32>, a, bytes(32), st);
    if (w <= 64) return launch_clusters(step_kernel<T, 64>, a, bytes(64), st);
    return launch_clusters(step_kernel<T, 128>, a, bytes(128), st);
}

}  // namespace

cudaError_t step(const StepArgs &in, hla_dtype dt, cudaStream_t st) {
    StepArgs a = in;
    // CTAs for a pair: enough that all pairs together give every SM two, no more than tiles of
    // slots, a power of two up to 16.  64 x 8 pairs: 1 CTA each 52 us, 2 59, 4 80; 8 pairs of
    // 4,112 slots: 16 CTAs each 14.8 us, 8 14.6, 4 19.2.
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const long long pairs = (long long)a.B * a.Hkv * ((a.G + HG - 1) / HG);
    const int unit = a.wide ? kWarps * GS : TS;  // slots a CTA takes at a time
    const long long tiles = ((long long)a.sinks + a.window + unit - 1) / unit;
    a.split = 1;
    while (a.split < 16 && pairs * a.split < 2LL * sms && a.split * 2 <= tiles) a.split *= 2;
    if (a.wide) return a.d <= 64 && a.dv <= 64 ? launch_clusters(step_mma_kernel<64>, a, 0, st) : launch_clusters(step_mma_kernel<128>, a, 0, st);
    return dt == HLA_F32 ? by_width<float>(a, st) : by_width<__nv_bfloat16>(a, st);
}

}  // namespace win
}  // namespace hla
