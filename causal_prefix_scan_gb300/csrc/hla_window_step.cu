// hla_window_step.cu -- one token of windowed attention per sequence over its ring cache
// of sinks + window slots, the new key and value written into their slot by the same launch.
//
// Bound by HBM: the visible slots of K and V are read once for all query heads of a
// key/value head.  Few (sequence, head) pairs would leave most SMs idle, so a cluster of
// up to 16 CTAs shares the slots of one pair: each runs a softmax over its own tiles of 64
// slots, and the cluster joins the partial results through distributed shared memory, in
// the order of the ranks (one launch, no workspace, the same bits on every call).
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
        slots = (int)(p + 1 < cap ? p + 1 : cap);
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

template <typename T, int DP>
cudaError_t launch(const StepArgs &a, cudaStream_t st) {
    constexpr size_t bytes = (size_t)(2 * TS * (DP + 4) + HG * DP + 4 * HG * TS + TS * HG) * 4;
    auto fn = step_kernel<T, DP>;
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
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
    if (w <= 32) return launch<T, 32>(a, st);
    if (w <= 64) return launch<T, 64>(a, st);
    return launch<T, 128>(a, st);
}

}  // namespace

cudaError_t step(const StepArgs &in, hla_dtype dt, cudaStream_t st) {
    StepArgs a = in;
    // CTAs for a pair: enough that all pairs together give every SM some, no more than
    // tiles of slots, a power of two up to 16
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const long long pairs = (long long)a.B * a.Hkv * ((a.G + HG - 1) / HG);
    const long long tiles = ((long long)a.sinks + a.window + TS - 1) / TS;
    a.split = 1;
    while (a.split < 16 && pairs * a.split < 2LL * sms && a.split * 2 <= tiles) a.split *= 2;
    return dt == HLA_F32 ? by_width<float>(a, st) : by_width<__nv_bfloat16>(a, st);
}

}  // namespace win
}  // namespace hla
