// hla_window_simt.cuh -- windowed attention on the CUDA cores in fp32: fp32 inputs, and
// bf16 ones whose rows are not multiples of 16 bytes.  64 x 64 tiles of queries and keys,
// both widths padded with zeros to DP; 256 threads, thread (ty, tx) of 16 x 16 holding
// rows 4 ty .. 4 ty + 3 and columns tx + 16 j of every product, so that a warp reads each
// operand row as float4 without bank conflicts (rows of DP + 4 floats).
// Bound by shared-memory reads: 8 float4 for 64 fmaf.  B4 H8 n2048 d64 w256 268 us forward
// (15 TFLOP/s); B2 H16 n8192 d128 w1024 17.7 ms backward (18 TFLOP/s).
#pragma once
#include "hla_window.h"

namespace hla {
namespace win {
namespace {

constexpr int TQ = 64, TK = 64, kThreads = 256, LP = TK + 4;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

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

// 64 rows r0 .. r0 + 63 (those in [0, rows)) of `width` elements into dst[64][DP + 4], zeros elsewhere.
template <typename T, int DP>
__device__ __forceinline__ void load_tile(float *dst, const View &t, int b, int h, int r0, int rows, int width) {
    const size_t base = (size_t)b * t.sb + (size_t)h * t.sh;
    for (int e = threadIdx.x; e < 64 * DP; e += kThreads) {
        const int r = e / DP, c = e % DP;
        float x = 0.f;
        if (r0 + r >= 0 && r0 + r < rows && c < width) x = ldf<T>(t.p, base + (size_t)(r0 + r) * t.st + c);
        dst[r * (DP + 4) + c] = x;
    }
}

// acc[i][j] += sum_k A[4 ty + i][k] B[tx + 16 j][k] over K columns of two row-major tiles
template <int K>
__device__ __forceinline__ void dot_rows(float (&acc)[4][4], const float *A, const float *Bm, int lda, int ldb, int ty,
                                         int tx) {
#pragma unroll 4
    for (int k = 0; k < K; k += 4) {
        float4 x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4 *>(A + (4 * ty + i) * lda + k);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4 *>(Bm + (tx + 16 * j) * ldb + k);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[i][j] += x[i].x * y[j].x + x[i].y * y[j].y + x[i].z * y[j].z + x[i].w * y[j].w;
    }
}
// acc[i][c] += sum_k P[4 ty + i][k] V[k][column c of this thread], P [64][LP], V [64][DP + 4];
// thread columns: 4 tx .. 4 tx + 3 of each block of 64 (DP = 32: 2 tx, 2 tx + 1)
template <int DP>
struct Cols {
    static constexpr int N = DP / 16;
    static __device__ __forceinline__ int col(int tx, int c) { return DP == 32 ? 2 * tx + c : (c >> 2) * 64 + 4 * tx + (c & 3); }
};
template <int DP>
__device__ __forceinline__ void rows_times(float (&acc)[4][DP / 16], const float *P, const float *V, int ty, int tx) {
#pragma unroll 4
    for (int k = 0; k < 64; ++k) {
        float p[4], v[DP / 16];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = P[(4 * ty + i) * LP + k];
        if constexpr (DP == 32) {
            const float2 x = *reinterpret_cast<const float2 *>(V + k * (DP + 4) + 2 * tx);
            v[0] = x.x;
            v[1] = x.y;
        } else {
#pragma unroll
            for (int c = 0; c < DP / 64; ++c) {
                const float4 x = *reinterpret_cast<const float4 *>(V + k * (DP + 4) + 64 * c + 4 * tx);
                v[4 * c] = x.x; v[4 * c + 1] = x.y; v[4 * c + 2] = x.z; v[4 * c + 3] = x.w;
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < DP / 16; ++c) acc[i][c] = fmaf(p[i], v[c], acc[i][c]);
    }
}
// The same with the transpose of P: acc row 4 ty + i is column 4 ty + i of P.
template <int DP>
__device__ __forceinline__ void cols_times(float (&acc)[4][DP / 16], const float *P, const float *V, int ty, int tx) {
#pragma unroll 4
    for (int k = 0; k < 64; ++k) {
        float v[DP / 16];
        const float4 p4 = *reinterpret_cast<const float4 *>(P + k * LP + 4 * ty);
        const float p[4] = {p4.x, p4.y, p4.z, p4.w};
        if constexpr (DP == 32) {
            const float2 x = *reinterpret_cast<const float2 *>(V + k * (DP + 4) + 2 * tx);
            v[0] = x.x;
            v[1] = x.y;
        } else {
#pragma unroll
            for (int c = 0; c < DP / 64; ++c) {
                const float4 x = *reinterpret_cast<const float4 *>(V + k * (DP + 4) + 64 * c + 4 * tx);
                v[4 * c] = x.x; v[4 * c + 1] = x.y; v[4 * c + 2] = x.z; v[4 * c + 3] = x.w;
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < DP / 16; ++c) acc[i][c] = fmaf(p[i], v[c], acc[i][c]);
    }
}
__device__ __forceinline__ float row_max(float x) {  // over the 16 threads of a row
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// ------------------------------------------------------------ forward
// One CTA per tile of 64 queries of one head; running maximum and sum of the softmax in
// fp32 (base 2, the scale folded into the exponent).
template <typename T, int DP>
__global__ void __launch_bounds__(kThreads) fwd_kernel(const Args a) {
    constexpr int LD = DP + 4;
    extern __shared__ __align__(16) float smem[];
    float *Q = smem, *K = Q + 64 * LD, *V = K + 64 * LD, *P = V + 64 * LD;
    const int tiles = (a.n + TQ - 1) / TQ;
    const int i0 = (int)(blockIdx.x % tiles) * TQ, bh = blockIdx.x / tiles, h = bh % a.H, b = bh / a.H, hk = h / a.G;
    const int len = length_of(a, b), rows = min(a.n, len - a.p0);  // valid query rows
    if (i0 >= rows) return;
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    load_tile<T, DP>(Q, a.q, b, h, i0, rows, a.d);
    const KeyTiles kt(a, a.p0 + i0, a.p0 + min(i0 + TQ, rows) - 1, TK);
    const float sc = a.scale * kLog2e;
    float m[4], l[4], acc[4][DP / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < DP / 16; ++c) acc[i][c] = 0.f;
    }
    for (int it = 0; it < kt.total; ++it) {
        const int j0 = kt[it] * TK;
        __syncthreads();
        load_tile<T, DP>(K, a.k, b, hk, j0, len, a.d);
        load_tile<T, DP>(V, a.v, b, hk, j0, len, a.dv);
        __syncthreads();
        float s[4][4] = {};
        dot_rows<DP>(s, Q, K, LD, LD, ty, tx);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int p = a.p0 + i0 + 4 * ty + i;
            float mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = visible(a, p, j0 + tx + 16 * j) ? s[i][j] * sc : -INFINITY;
                mx = fmaxf(mx, s[i][j]);
            }
            mx = fmaxf(row_max(mx), m[i]);
            const float base = mx == -INFINITY ? 0.f : mx, f = exp2f(m[i] - base);
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float e = exp2f(s[i][j] - base);
                sum += e;
                P[(4 * ty + i) * LP + tx + 16 * j] = e;
            }
            l[i] = l[i] * f + row_sum(sum);
            m[i] = mx;
#pragma unroll
            for (int c = 0; c < DP / 16; ++c) acc[i][c] *= f;
        }
        __syncwarp();  // a row's 16 threads are in one warp, and only they read the row
        rows_times<DP>(acc, P, V, ty, tx);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = i0 + 4 * ty + i;
        if (r >= rows) continue;
        const float inv = 1.f / l[i];
        const size_t o = (size_t)b * a.o.sb + (size_t)h * a.o.sh + (size_t)r * a.o.st;
#pragma unroll
        for (int c = 0; c < DP / 16; ++c) {
            const int col = Cols<DP>::col(tx, c);
            if (col < a.dv) stf<T>(a.o.p, o + col, acc[i][c] * inv);
        }
        if (a.lse && tx == 0) a.lse[(size_t)bh * a.n + r] = (m[i] + log2f(l[i])) * kLn2;
    }
}

// ------------------------------------------------------------ backward
// P and dS of one pair of tiles: P = exp(s - lse), dS = P (do.v - D) scale, zero where
// nothing is visible.
template <int DP>
__device__ __forceinline__ void pair_tile(const Args &a, const float *Q, const float *K, const float *V, const float *dO,
                                          const float *lse, const float *D, float *P, float *dS, int p_lo, int rows,
                                          int j0, int ty, int tx) {
    constexpr int LD = DP + 4;
    float s[4][4] = {}, dp[4][4] = {};
    dot_rows<DP>(s, Q, K, LD, LD, ty, tx);
    dot_rows<DP>(dp, dO, V, LD, LD, ty, tx);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * ty + i;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool see = r < rows && visible(a, p_lo + r, j0 + tx + 16 * j);
            const float p = see ? exp2f(s[i][j] * (a.scale * kLog2e) - lse[r] * kLog2e) : 0.f;
            if (P) P[r * LP + tx + 16 * j] = p;
            dS[r * LP + tx + 16 * j] = see ? p * (dp[i][j] - D[r]) * a.scale : 0.f;
        }
    }
}

// D = rowsum(do o), one warp per row.
template <typename T>
__global__ void __launch_bounds__(kThreads) delta_kernel(const Args a) {
    const size_t row = (size_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (row >= (size_t)a.B * a.H * a.n) return;
    const int i = (int)(row % a.n), h = (int)(row / a.n % a.H), b = (int)(row / a.n / a.H);
    if (a.p0 + i >= length_of(a, b)) return;
    const size_t o = (size_t)b * a.o.sb + (size_t)h * a.o.sh + (size_t)i * a.o.st;
    const size_t g = (size_t)b * a.go.sb + (size_t)h * a.go.sh + (size_t)i * a.go.st;
    float s = 0.f;
    for (int c = threadIdx.x & 31; c < a.dv; c += 32) s = fmaf(ldf<T>(a.o.p, o + c), ldf<T>(a.go.p, g + c), s);
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
    if ((threadIdx.x & 31) == 0) a.delta[row] = s;
}

// dq of one tile of 64 queries.
template <typename T, int DP>
__global__ void __launch_bounds__(kThreads) dq_kernel(const Args a) {
    constexpr int LD = DP + 4;
    extern __shared__ __align__(16) float smem[];
    float *Q = smem, *K = Q + 64 * LD, *V = K + 64 * LD, *dO = V + 64 * LD, *dS = dO + 64 * LD, *lse = dS + 64 * LP,
          *D = lse + 64;
    const int tiles = (a.n + TQ - 1) / TQ;
    const int i0 = (int)(blockIdx.x % tiles) * TQ, bh = blockIdx.x / tiles, h = bh % a.H, b = bh / a.H, hk = h / a.G;
    const int len = length_of(a, b), rows = min(a.n, len - a.p0);
    if (i0 >= rows) return;
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    load_tile<T, DP>(Q, a.q, b, h, i0, rows, a.d);
    load_tile<T, DP>(dO, a.go, b, h, i0, rows, a.dv);
    if (threadIdx.x < 64 && i0 + threadIdx.x < rows) {
        lse[threadIdx.x] = a.lse[(size_t)bh * a.n + i0 + threadIdx.x];
        D[threadIdx.x] = a.delta[(size_t)bh * a.n + i0 + threadIdx.x];
    }
    const KeyTiles kt(a, a.p0 + i0, a.p0 + min(i0 + TQ, rows) - 1, TK);
    float acc[4][DP / 16] = {};
    for (int it = 0; it < kt.total; ++it) {
        const int j0 = kt[it] * TK;
        __syncthreads();
        load_tile<T, DP>(K, a.k, b, hk, j0, len, a.d);
        load_tile<T, DP>(V, a.v, b, hk, j0, len, a.dv);
        __syncthreads();
        pair_tile<DP>(a, Q, K, V, dO, lse, D, nullptr, dS, a.p0 + i0, rows - i0, j0, ty, tx);
        __syncwarp();
        rows_times<DP>(acc, dS, K, ty, tx);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = i0 + 4 * ty + i;
        if (r >= rows) continue;
        const size_t o = (size_t)b * a.dq.sb + (size_t)h * a.dq.sh + (size_t)r * a.dq.st;
#pragma unroll
        for (int c = 0; c < DP / 16; ++c) {
            const int col = Cols<DP>::col(tx, c);
            if (col < a.d) stf<T>(a.dq.p, o + col, acc[i][c]);
        }
    }
}

// dk and dv of one tile of 64 keys, over the query tiles of every head of the group that
// can see it.  Tiles with first tokens are seen by every later query: their far queries
// (beyond the window of the tile's last key) go to blockIdx.y = 1 .. far, an equal share of
// tiles each, and all shares leave as fp32 partial sums that join_kernel adds in order.
template <typename T, int DP>
__global__ void __launch_bounds__(kThreads) dkv_kernel(const Args a) {
    constexpr int LD = DP + 4;
    extern __shared__ __align__(16) float smem[];
    float *Q = smem, *K = Q + 64 * LD, *V = K + 64 * LD, *dO = V + 64 * LD, *P = dO + 64 * LD, *dS = P + 64 * LP,
          *lse = dS + 64 * LP, *D = lse + 64;
    const int tiles = (a.nk + TK - 1) / TK, share = blockIdx.y;
    const int j0 = (int)(blockIdx.x % tiles) * TK, bk = blockIdx.x / tiles, hk = bk % a.Hkv, b = bk / a.Hkv;
    const int len = length_of(a, b), rows = min(a.n, len - a.p0);
    const bool first = j0 < a.far_keys;  // holds first tokens whose sums are split
    if (share > 0 && !first) return;
    if (j0 >= len) return;
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    // query tiles [q_lo, q_hi): the window's, then the far ones
    const int r_lo = max(0, j0 - a.p0), r_win = (int)min((long long)max(rows, 0), (long long)j0 + TK - 1 + a.window - a.p0);
    const int q_mid = max((max(r_win, 0) + TQ - 1) / TQ, r_lo / TQ);
    int q_lo = r_lo / TQ, q_hi = q_mid;
    if (share > 0) {
        const int end = (max(rows, 0) + TQ - 1) / TQ, all = max(end - q_mid, 0), each = (all + a.far - 1) / a.far;
        q_lo = min(q_mid + (share - 1) * each, end);
        q_hi = min(q_lo + each, end);
    }
    load_tile<T, DP>(K, a.k, b, hk, j0, len, a.d);
    load_tile<T, DP>(V, a.v, b, hk, j0, len, a.dv);
    float gk[4][DP / 16] = {}, gv[4][DP / 16] = {};
    for (int g = 0; g < a.G; ++g) {
        const int h = hk * a.G + g;
        const size_t bh = (size_t)b * a.H + h;
        for (int qt = q_lo; qt < q_hi; ++qt) {
            const int i0 = qt * TQ;
            if (i0 >= rows) break;
            __syncthreads();
            load_tile<T, DP>(Q, a.q, b, h, i0, rows, a.d);
            load_tile<T, DP>(dO, a.go, b, h, i0, rows, a.dv);
            if (threadIdx.x < 64 && i0 + threadIdx.x < rows) {
                lse[threadIdx.x] = a.lse[bh * a.n + i0 + threadIdx.x];
                D[threadIdx.x] = a.delta[bh * a.n + i0 + threadIdx.x];
            }
            __syncthreads();
            pair_tile<DP>(a, Q, K, V, dO, lse, D, P, dS, a.p0 + i0, rows - i0, j0, ty, tx);
            __syncthreads();
            cols_times<DP>(gv, P, dO, ty, tx);
            cols_times<DP>(gk, dS, Q, ty, tx);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int j = j0 + 4 * ty + i;
        if (j >= len) continue;
        if (first && a.far > 0) {
            float *w = a.part + (((size_t)share * a.B * a.Hkv + bk) * a.far_keys + j) * (a.d + a.dv);
#pragma unroll
            for (int c = 0; c < DP / 16; ++c) {
                const int col = Cols<DP>::col(tx, c);
                if (col < a.d) w[col] = gk[i][c];
                if (col < a.dv) w[a.d + col] = gv[i][c];
            }
            continue;
        }
        const size_t ok = (size_t)b * a.dk.sb + (size_t)hk * a.dk.sh + (size_t)j * a.dk.st;
        const size_t ov = (size_t)b * a.dv_.sb + (size_t)hk * a.dv_.sh + (size_t)j * a.dv_.st;
#pragma unroll
        for (int c = 0; c < DP / 16; ++c) {
            const int col = Cols<DP>::col(tx, c);
            if (col < a.d) stf<T>(a.dk.p, ok + col, gk[i][c]);
            if (col < a.dv) stf<T>(a.dv_.p, ov + col, gv[i][c]);
        }
    }
}

// dk, dv of the key tiles whose sums were split: the shares added in order.  One thread
// per element, columns fastest.
template <typename T>
__global__ void __launch_bounds__(kThreads) join_kernel(const Args a) {
    const int width = a.d + a.dv;
    const size_t e = (size_t)blockIdx.x * kThreads + threadIdx.x;
    if (e >= (size_t)a.B * a.Hkv * a.far_keys * width) return;
    const int c = (int)(e % width), j = (int)(e / width % a.far_keys), bk = (int)(e / width / a.far_keys);
    const int b = bk / a.Hkv, hk = bk % a.Hkv;
    if (j >= length_of(a, b)) return;
    const size_t step = (size_t)a.B * a.Hkv * a.far_keys * width;
    float s = 0.f;
    for (int i = 0; i <= a.far; ++i) s += a.part[i * step + e];
    if (c < a.d)
        stf<T>(a.dk.p, (size_t)b * a.dk.sb + (size_t)hk * a.dk.sh + (size_t)j * a.dk.st + c, s);
    else
        stf<T>(a.dv_.p, (size_t)b * a.dv_.sb + (size_t)hk * a.dv_.sh + (size_t)j * a.dv_.st + (c - a.d), s);
}

}  // namespace
}  // namespace win
}  // namespace hla
