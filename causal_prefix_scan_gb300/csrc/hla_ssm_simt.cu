// hla_ssm_simt.cu -- selective state space scan on the CUDA cores (formulas in hla_ssm.h): any
// widths up to 128, strides and alignment, fp32 arithmetic on fp32 copies of the tiles in shared
// memory.  Chunks are independent but for their states, so the states come first: what each chunk
// adds, then a scan over the chunks that leaves in place the state before (the gradient behind)
// each chunk.  A call goes through its chunks span by span, so that it holds the states of one span
// (backward the states of all, the gradients of one).  Products run on 4 x 4 register tiles; the fp32 rate and the states' traffic
// (N P 4 bytes per chunk and head, four times) bound it.  Measured, backward b3 n1501 h6 p48 s40 fp32: 145 us,
// 106 of them in grad_kernel, whose 432 CTAs of 8 warps wait for each other's tiles (issue slots 31 %
// busy, two CTAs to an SM by their registers).
#include "hla_smem_tile.cuh"
#include "hla_ssm.h"

namespace hla {
namespace ssm {
namespace {

using tile::kThreads;
using tile::mac;

__host__ __device__ inline int up4(int x) { return (x + 3) & ~3; }

// Every 4x4 tile of an M x N result, one per thread per round; STRIDED as in hla_smem_tile.cuh.
template <bool STRIDED, class Body>
__device__ __forceinline__ void over(int M, int N, Body body) {
    const int tn = N / 4, count = (M / 4) * tn;
    for (int t = threadIdx.x; t < count; t += kThreads) {
        const int m0 = (t / tn) * 4, n0 = STRIDED ? t % tn : (t % tn) * 4, ns = STRIDED ? tn : 1;
        float acc[4][4] = {};
        body(acc, m0, n0, ns);
    }
}

// Rows t0 .. of head (or group) h of a strided tensor into shared rows of ld `ld`, zeros behind
// `live` rows and `w` columns (up to w4).
template <typename T>
__device__ __forceinline__ void load_rows(const View &v, int b, int h, int t0, float *dst, int ld, int rows, int live, int w,
                                          int w4) {
    const T *src = static_cast<const T *>(v.p) + (size_t)b * v.sb + (size_t)h * v.sh + (size_t)t0 * v.st;
    for (int e = threadIdx.x; e < rows * w4; e += kThreads) {
        const int r = e / w4, x = e % w4;
        dst[r * ld + x] = r < live && x < w ? tile::ld_t(src + (size_t)r * v.st, x) : 0.f;
    }
}
// An fp32 [N][P] state into shared rows, zeros behind both widths.
__device__ __forceinline__ void load_state(const float *src, int N, int P, float *dst, int ld, int N4, int P4) {
    for (int e = threadIdx.x; e < N4 * P4; e += kThreads) {
        const int r = e / P4, x = e % P4;
        dst[r * ld + x] = r < N && x < P ? src[(size_t)r * P + x] : 0.f;
    }
}

struct Unit {  // one (sequence, head, chunk of the span)
    int b, h, c, len, t0;
    size_t hat, gat;  // of its state, of the state's gradient
    __device__ Unit(const Args &a, unsigned u, int Q) {
        c = u % a.nc;
        h = u / a.nc % a.H;
        b = u / a.nc / a.H;
        len = clamp_length(a.lengths, b, a.n);
        t0 = a.t0 + c * Q;
        hat = ((size_t)b * a.H + h) * a.hc + a.h0 + c;
        gat = ((size_t)b * a.H + h) * a.nc + c;
    }
};

// What chunk c adds to the state (dir + blockIdx.y 0: B^T diag(dt r) X) or to its gradient (1: C^T diag(e) dY).
template <typename T, int Q>
__global__ void __launch_bounds__(kThreads) ssm_add_kernel(const Args a, int dir) {
    extern __shared__ __align__(16) float sm[];
    __shared__ float dt[Q];
    __shared__ Decay s[Q];
    const Unit u(a, blockIdx.x, Q);
    if (u.t0 >= u.len) return;
    const bool back = dir + blockIdx.y == 1;
    const int N4 = up4(a.N), P4 = up4(a.P), ldn = N4 + 4, ldp = P4 + 4;
    float *B = sm, *X = B + Q * ldn;
    load_rows<T>(back ? a.c : a.b, u.b, u.h / a.R, u.t0, B, ldn, Q, u.len - u.t0, a.N, N4);
    load_rows<T>(back ? a.dy : a.x, u.b, u.h, u.t0, X, ldp, Q, u.len - u.t0, a.P, P4);
    if (threadIdx.x < 32) chunk_decays<T, Q / 32>(a, u.b, u.h, u.t0, u.len, dt, s, nullptr);
    __syncthreads();
    const Decay end = s[Q - 1];
    if (threadIdx.x == 0 && !back) a.factor[u.hat] = factor(end);
    for (int e = threadIdx.x; e < Q * P4; e += kThreads) {
        const int t = e / P4;
        X[t * ldp + e % P4] *= back ? factor(s[t]) : dt[t] * factor(end, s[t]);
    }
    __syncthreads();
    float *out = (back ? a.g + u.gat * a.N * a.P : a.h + u.hat * a.N * a.P);
    over<false>(N4, P4, [&](float (&acc)[4][4], int m0, int n0, int ns) {
        mac<true, false>(acc, B, ldn, X, ldp, m0, n0, ns, Q);
        tile::each(acc, m0, n0, ns, [&](int n, int p, float x) {
            if (n < a.N && p < a.P) out[(size_t)n * a.P + p] = x;
        });
    });
}

// Scan over the chunks: dir + blockIdx.y 0 leaves the state before each chunk, 1 the gradient behind it.
__global__ void __launch_bounds__(256) ssm_scan_kernel(const Args a, int Q, int dir) {
    const int blocks = (a.N * a.P + 255) / 256, e = blockIdx.x % blocks * 256 + threadIdx.x;
    const int u = blockIdx.x / blocks;
    if (e >= a.N * a.P) return;
    const bool back = dir + blockIdx.y == 1;
    const size_t NP = (size_t)a.N * a.P;
    const int left = clamp_length(a.lengths, u / a.H, a.n) - a.t0, used = left <= 0 ? 0 : min((left + Q - 1) / Q, a.nc);
    float *add = (back ? a.g + (size_t)u * a.nc * NP : a.h + ((size_t)u * a.hc + a.h0) * NP) + e;
    const float *f = a.factor + (size_t)u * a.hc + a.h0;
    const float *init = a.from[back];
    float *fin = a.to[back];
    float h = init ? init[u * NP + e] : 0.f;
    constexpr int U = 8;
    for (int i = 0; i < used; i += U) {
        float v[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int c = back ? used - 1 - i - k : i + k;
            if (i + k < used) v[k] = add[c * NP];
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int c = back ? used - 1 - i - k : i + k;
            if (i + k >= used) break;
            add[c * NP] = h;
            h = fmaf(f[c], h, v[k]);
        }
    }
    if (fin) fin[u * NP + e] = h;
}

template <typename T, int Q>
__global__ void __launch_bounds__(kThreads) ssm_out_kernel(const Args a) {
    extern __shared__ __align__(16) float sm[];
    __shared__ float dt[Q];
    __shared__ Decay s[Q];
    const Unit u(a, blockIdx.x, Q);
    if (u.t0 >= u.len) return;
    const int N4 = up4(a.N), P4 = up4(a.P), ldn = N4 + 4, ldp = P4 + 4, ldq = Q + 4, live = u.len - u.t0;
    float *C = sm, *B = C + Q * ldn, *X = B + Q * ldn, *M = X + Q * ldp, *h = M + Q * ldq;
    load_rows<T>(a.c, u.b, u.h / a.R, u.t0, C, ldn, Q, live, a.N, N4);
    load_rows<T>(a.b, u.b, u.h / a.R, u.t0, B, ldn, Q, live, a.N, N4);
    load_rows<T>(a.x, u.b, u.h, u.t0, X, ldp, Q, live, a.P, P4);
    load_state(a.h + u.hat * a.N * a.P, a.N, a.P, h, ldp, N4, P4);
    if (threadIdx.x < 32) chunk_decays<T, Q / 32>(a, u.b, u.h, u.t0, u.len, dt, s, nullptr);
    __syncthreads();
    over<true>(Q, Q, [&](float (&acc)[4][4], int m0, int n0, int ns) {
        mac<false, true>(acc, C, ldn, B, ldn, m0, n0, ns, N4);
        tile::each(acc, m0, n0, ns, [&](int t, int j, float x) { M[t * ldq + j] = j <= t ? x * factor(s[t], s[j]) * dt[j] : 0.f; });
    });
    __syncthreads();
    const float D = a.D ? a.D[u.h] : 0.f;
    T *y = static_cast<T *>(a.y.p) + (size_t)u.b * a.y.sb + (size_t)u.h * a.y.sh + (size_t)u.t0 * a.y.st;
    over<false>(Q, P4, [&](float (&acc)[4][4], int m0, int n0, int ns) {
        mac<false, false>(acc, C, ldn, h, ldp, m0, n0, ns, N4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float e = factor(s[m0 + i]);
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] *= e;
        }
        mac<false, false>(acc, M, ldq, X, ldp, m0, n0, ns, Q);
        tile::each(acc, m0, n0, ns, [&](int t, int p, float x) {
            if (t < live && p < a.P) tile::st_t(y + (size_t)t * a.y.st, p, fmaf(D, X[t * ldp + p], x));
        });
    });
}

// One (sequence, group, chunk, share of the group's heads): the heads one after the other, dB and
// dC added up in this CTA's own part of the workspace, each element by the same thread.
template <typename T, int Q>
__global__ void __launch_bounds__(kThreads) ssm_grad_kernel(const Args a) {
    extern __shared__ __align__(16) float sm[];
    __shared__ float dt[Q], slope[Q], w[Q], ve[Q], vg[Q], diag[Q], red[8];
    __shared__ Decay s[Q];
    const int split = blockIdx.x % a.splits, c = blockIdx.x / a.splits % a.nc, g = blockIdx.x / a.splits / a.nc % a.G,
              b = blockIdx.x / a.splits / a.nc / a.G;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int len = clamp_length(a.lengths, b, a.n), t0 = a.t0 + c * Q, live = len - t0;
    const int h0 = g * a.R + (int)((long long)a.R * split / a.splits), h1 = g * a.R + (int)((long long)a.R * (split + 1) / a.splits);
    float *sums = a.sums + ((size_t)b * a.sumc + a.sum0 + c) * 3 * a.H;
    if (live <= 0) {
        for (int h = h0 + tid; h < h1; h += kThreads) sums[h] = sums[a.H + h] = sums[2 * a.H + h] = 0.f;
        return;
    }
    const int N4 = up4(a.N), P4 = up4(a.P), ldn = N4 + 4, ldp = P4 + 4, ldq = Q + 4, ldr = N4 / 4 + 1;
    float *C = sm, *B = C + Q * ldn, *X = B + Q * ldn, *dY = X + Q * ldp, *CB = dY + Q * ldp, *M = CB + Q * ldq, *S = M + Q * ldq,
          *E = S + Q * ldq, *hg = E + Q * ldq, *rs = hg + N4 * ldp;  // rs [Q][ldr]
    load_rows<T>(a.c, b, g, t0, C, ldn, Q, live, a.N, N4);
    load_rows<T>(a.b, b, g, t0, B, ldn, Q, live, a.N, N4);
    __syncthreads();
    over<true>(Q, Q, [&](float (&acc)[4][4], int m0, int n0, int ns) {
        mac<false, true>(acc, C, ldn, B, ldn, m0, n0, ns, N4);
        tile::each(acc, m0, n0, ns, [&](int t, int j, float x) { CB[t * ldq + j] = x; });
    });
    const size_t half = (size_t)a.B * a.G * a.rows * a.N;
    float *pb = a.dbc + (size_t)split * 2 * half + (((size_t)b * a.G + g) * a.rows + c * Q) * a.N, *pc = pb + half;
    for (int h = h0; h < h1; ++h) {
        __syncthreads();
        load_rows<T>(a.x, b, h, t0, X, ldp, Q, live, a.P, P4);
        load_rows<T>(a.dy, b, h, t0, dY, ldp, Q, live, a.P, P4);
        const size_t hat = (((size_t)b * a.H + h) * a.hc + a.h0 + c) * a.N * a.P, gat = (((size_t)b * a.H + h) * a.nc + c) * a.N * a.P;
        load_state(a.h + hat, a.N, a.P, hg, ldp, N4, P4);
        if (warp == 0) chunk_decays<T, Q / 32>(a, b, h, t0, len, dt, s, slope);
        __syncthreads();
        over<true>(Q, Q, [&](float (&acc)[4][4], int m0, int n0, int ns) {
            mac<false, true>(acc, dY, ldp, X, ldp, m0, n0, ns, P4);
            tile::each(acc, m0, n0, ns, [&](int t, int j, float x) {
                const float L = j <= t ? factor(s[t], s[j]) : 0.f, m = CB[t * ldq + j] * L;
                M[t * ldq + j] = j <= t ? m : 0.f;
                S[t * ldq + j] = j <= t ? x * L : 0.f;
                // E's diagonal is kept apart: it cancels in the gradient of the decays, which differences of
                // E's sums give, and where decays are steep it is most of them
                E[t * ldq + j] = j < t ? m * x : 0.f;
                if (j == t) diag[t] = m * x;
            });
        });
        // dY h^T: its share of dC, and of w
        __syncthreads();
        over<true>(Q, N4, [&](float (&acc)[4][4], int m0, int n0, int ns) {
            mac<false, true>(acc, dY, ldp, hg, ldp, m0, n0, ns, P4);
            float part[4] = {};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float e = factor(s[m0 + i]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    acc[i][j] *= e;
                    part[i] = fmaf(C[(m0 + i) * ldn + n0 + j * ns], acc[i][j], part[i]);
                }
                rs[(m0 + i) * ldr + n0] = part[i];
            }
            mac<false, false>(acc, S, ldq, B, ldn, m0, n0, ns, Q, dt);
            tile::each(acc, m0, n0, ns, [&](int t, int n, float x) {
                if (t < live && n < a.N) pc[(size_t)t * a.N + n] = h == h0 ? x : pc[(size_t)t * a.N + n] + x;
            });
        });
        __syncthreads();
        for (int t = warp; t < Q; t += 8) {  // w, and what stays inside the chunk of v
            float x = 0.f, y = 0.f;
            for (int i = lane; i < N4 / 4; i += 32) x += rs[t * ldr + i];
            for (int j = lane; j < Q; j += 32) {
                x = fmaf(E[t * ldq + j], dt[j], x);
                y += E[j * ldq + t];
            }
            for (int o = 16; o > 0; o >>= 1) {
                x += __shfl_xor_sync(0xffffffffu, x, o);
                y += __shfl_xor_sync(0xffffffffu, y, o);
            }
            if (lane == 0) {
                w[t] = x;
                ve[t] = y;
            }
        }
        // <g, h> while h is here, then g in its place
        float dot = 0.f;
        for (int e = tid; e < a.N * a.P; e += kThreads) dot = fmaf(a.g[gat + e], hg[e / a.P * ldp + e % a.P], dot);
        for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        __syncthreads();
        if (lane == 0) red[warp] = dot;
        load_state(a.g + gat, a.N, a.P, hg, ldp, N4, P4);
        __syncthreads();
        const Decay end = s[Q - 1];
        const float D = a.D ? a.D[h] : 0.f;
        T *dx = static_cast<T *>(a.dx.p) + (size_t)b * a.dx.sb + (size_t)h * a.dx.sh + (size_t)t0 * a.dx.st;
        over<false>(Q, P4, [&](float (&acc)[4][4], int m0, int n0, int ns) {
            mac<false, false>(acc, B, ldn, hg, ldp, m0, n0, ns, N4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float r = factor(end, s[m0 + i]);
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] *= r;
            }
            mac<true, false>(acc, M, ldq, dY, ldp, m0, n0, ns, Q);
            tile::each(acc, m0, n0, ns, [&](int t, int p, float x) {
                if (t < live && p < a.P) tile::st_t(dx + (size_t)t * a.dx.st, p, fmaf(D, dY[t * ldp + p], dt[t] * x));
            });
        });
        over<true>(Q, N4, [&](float (&acc)[4][4], int m0, int n0, int ns) {
            mac<false, true>(acc, X, ldp, hg, ldp, m0, n0, ns, P4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float r = factor(end, s[m0 + i]);
                float part = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    acc[i][j] *= r;
                    part = fmaf(B[(m0 + i) * ldn + n0 + j * ns], acc[i][j], part);
                }
                rs[(m0 + i) * ldr + n0] = part;
            }
            mac<true, false>(acc, S, ldq, C, ldn, m0, n0, ns, Q);
            tile::each(acc, m0, n0, ns, [&](int t, int n, float x) {
                x *= dt[t];
                if (t < live && n < a.N) pb[(size_t)t * a.N + n] = h == h0 ? x : pb[(size_t)t * a.N + n] + x;
            });
        });
        __syncthreads();
        float dd = 0.f;  // dY . X
        for (int e = tid; e < Q * P4; e += kThreads) dd = fmaf(dY[e / P4 * ldp + e % P4], X[e / P4 * ldp + e % P4], dd);
        for (int o = 16; o > 0; o >>= 1) dd += __shfl_xor_sync(0xffffffffu, dd, o);
        for (int t = warp; t < Q; t += 8) {
            float x = 0.f;
            for (int i = lane; i < N4 / 4; i += 32) x += rs[t * ldr + i];
            for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
            if (lane == 0) vg[t] = x;
        }
        float through = 0.f;
        if (warp == 0) {
            for (int i = 0; i < 8; ++i) through += red[i];
            through *= factor(end);
        }
        __syncthreads();
        if (lane == 0) red[warp] = dd;
        __syncthreads();
        if (warp == 0) {
            // suffix sums of w - dt vE (the token among them), prefix sums of dt vg (without it)
            constexpr int PER = Q / 32;
            float suf[PER], pre[PER], a_suf = 0.f, a_pre = 0.f;
#pragma unroll
            for (int i = PER - 1; i >= 0; --i) {
                const int t = lane * PER + i;
                a_suf += fmaf(-dt[t], ve[t], w[t]);
                suf[i] = a_suf;
            }
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int t = lane * PER + i;
                pre[i] = a_pre;
                a_pre = fmaf(dt[t], vg[t], a_pre);
            }
            float xs = a_suf, xp = a_pre;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float us = __shfl_down_sync(0xffffffffu, xs, o), up = __shfl_up_sync(0xffffffffu, xp, o);
                if (lane + o < 32) xs += us;
                if (lane >= o) xp += up;
            }
            xs = __shfl_down_sync(0xffffffffu, xs, 1);  // of the lanes behind, in front
            xp = __shfl_up_sync(0xffffffffu, xp, 1);
            if (lane == 31) xs = 0.f;
            if (lane == 0) xp = 0.f;
            float sA = 0.f, sb = 0.f;
            const float A = a.A[h];
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int t = lane * PER + i;
                const float da = through + (suf[i] + xs) + (pre[i] + xp), d = fmaf(A, da, (ve[t] + diag[t]) + vg[t]) * slope[t];
                if (t < live) {
                    tile::st_t(static_cast<T *>(a.ddt.p) + (size_t)b * a.ddt.sb + (size_t)h * a.ddt.sh + (size_t)(t0 + t) * a.ddt.st, 0, d);
                    sA = fmaf(da, dt[t], sA);
                    sb += d;
                }
            }
            float sd = lane < 8 ? red[lane] : 0.f;
            for (int o = 16; o > 0; o >>= 1) {
                sA += __shfl_xor_sync(0xffffffffu, sA, o);
                sb += __shfl_xor_sync(0xffffffffu, sb, o);
                sd += __shfl_xor_sync(0xffffffffu, sd, o);
            }
            if (lane == 0) {
                sums[h] = sA;
                sums[a.H + h] = sd;
                sums[2 * a.H + h] = sb;
            }
        }
    }
}

// dB, dC of a span: the shares' parts added in order and rounded.  Rows of [B][G][rows] by warps.
template <typename T>
__global__ void __launch_bounds__(256) ssm_join_kernel(const Args a) {
    const size_t rows = (size_t)a.B * a.G * a.rows, half = rows * a.N;
    for (size_t r = (size_t)blockIdx.x * 8 + (threadIdx.x >> 5); r < rows; r += (size_t)gridDim.x * 8) {
        const int t = a.t0 + (int)(r % a.rows), g = (int)(r / a.rows % a.G), b = (int)(r / a.rows / a.G);
        if (t >= clamp_length(a.lengths, b, a.n)) continue;
        const float *p = a.dbc + (blockIdx.y ? half : 0) + r * a.N;
        const View &v = blockIdx.y ? a.dc : a.db;
        T *out = static_cast<T *>(v.p) + (size_t)b * v.sb + (size_t)g * v.sh + (size_t)t * v.st;
        for (int n = threadIdx.x & 31; n < a.N; n += 32) {
            float s = 0.f;
            for (int i = 0; i < a.splits; ++i) s += p[(size_t)i * 2 * half + n];
            tile::st_t(out, n, s);
        }
    }
}
__global__ void __launch_bounds__(256) ssm_sums_kernel(const Args a, int rows) {
    column_sums(a.sums, rows, 3LL * a.H, [=](long long k, float s) {
        float *out = k < a.H ? a.dA : k < 2 * a.H ? a.dD : a.dbias;
        if (out) out[k % a.H] = s;
    });
}

size_t bytes_of(const Args &a, int Q, bool grad) {
    const size_t N4 = up4(a.N), P4 = up4(a.P), n = Q * (N4 + 4), p = Q * (P4 + 4), q = Q * (Q + 4), hg = N4 * (P4 + 4);
    return 4 * (grad ? 2 * n + 2 * p + 4 * q + hg + Q * (N4 / 4 + 1) : 2 * n + p + q + hg);
}

template <typename K>
cudaError_t allow(K fn, size_t bytes) {
    return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

// What the chunks of a span add and the scan over them, `dirs` directions from `dir` on.
template <typename T, int Q>
cudaError_t states(const Args &a, int dir, int dirs, cudaStream_t st) {
    const size_t bytes = 4 * (size_t)Q * (up4(a.N) + 4 + up4(a.P) + 4);
    cudaError_t e = allow(ssm_add_kernel<T, Q>, bytes);
    if (e != cudaSuccess) return e;
    const unsigned units = (unsigned)((size_t)a.B * a.H * a.nc);
    ssm_add_kernel<T, Q><<<dim3(units, dirs), kThreads, bytes, st>>>(a, dir);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    ssm_scan_kernel<<<dim3((unsigned)((size_t)a.B * a.H * ((a.N * a.P + 255) / 256)), dirs), 256, 0, st>>>(a, Q, dir);
    return cudaGetLastError();
}

// Chunks of a span: states of 64 MB, which stay in L2 between the kernels (forward h64 n16384 p64 s128
// fp32 4.4 ms in one span, 4.2 in eight), and 2,048 CTAs at least.
struct Spans {
    int chunks, per, count;
    Spans(const Args &a, int Q) {
        chunks = (int)(((long long)a.n + Q - 1) / Q);
        const long long heads = (long long)a.B * a.H, fit = (64LL << 20) / ((long long)a.N * a.P * 4), units = fit > 2048 ? fit : 2048;
        const long long most = units / heads > 1 ? units / heads : 1;
        count = (int)((chunks + most - 1) / most);
        per = (chunks + count - 1) / count;
        count = (chunks + per - 1) / per;
    }
};
// CTAs that share a group's heads: as many as fill the device about twice; where span comes after span,
// the number whose rounds over the SMs (one CTA each) are shortest, since every span ends in one that is not
// full (backward h64 n16384 p64 s128 fp32, eight spans: 12.6 ms by the first rule, 11.2 by this one, 11.3 in one span).
int splits_of(const Args &a, const Spans &s) {
    constexpr int kSms = 152;
    const long long ctas = (long long)a.B * a.G * s.per, want = (2 * kSms + ctas - 1) / ctas;
    if (s.count == 1) return (int)(want < a.R ? want : a.R);
    long long best = -1;
    int splits = 1;
    for (int k = 1; k <= a.R && k <= 16; ++k) {
        const long long cost = (ctas * k + kSms - 1) / kSms * ((a.R + k - 1) / k + 1);
        if (best < 0 || cost < best) {
            best = cost;
            splits = k;
        }
    }
    return splits;
}
// The span of chunks [c, c + per): the states' arrays hold it alone, or (`all`) every chunk.
Args span_of(Args a, const Spans &s, int c, int per, int Q, bool all) {
    a.nc = per < s.chunks - c ? per : s.chunks - c;
    a.t0 = c * Q;
    a.rows = per * Q < a.n - a.t0 ? per * Q : a.n - a.t0;
    a.hc = all ? s.chunks : a.nc;
    a.h0 = all ? c : 0;
    a.sum0 = c;
    a.sumc = s.chunks;
    a.from[0] = c == 0 ? a.state_in : a.carry;
    a.to[0] = c + a.nc == s.chunks ? a.state_out : a.carry;
    a.from[1] = c + a.nc == s.chunks ? a.d_state_out : a.carry;
    a.to[1] = c == 0 ? a.d_state_in : a.carry;
    return a;
}

template <typename T, int Q>
cudaError_t run_forward(const Args &whole, cudaStream_t st) {
    const Spans s(whole, Q);
    const size_t bytes = bytes_of(whole, Q, false);
    cudaError_t e = allow(ssm_out_kernel<T, Q>, bytes);
    for (int c = 0; c < s.chunks && e == cudaSuccess; c += s.per) {
        const Args a = span_of(whole, s, c, s.per, Q, false);
        if ((e = states<T, Q>(a, 0, 1, st)) != cudaSuccess) break;
        ssm_out_kernel<T, Q><<<(unsigned)((size_t)a.B * a.H * a.nc), kThreads, bytes, st>>>(a);
        e = cudaGetLastError();
    }
    return e;
}
// The states of all chunks, then the spans from the last one on: their gradients and what follows.
template <typename T, int Q>
cudaError_t run_backward(const Args &whole, hla_dtype dt, cudaStream_t st) {
    const Spans s(whole, Q);
    const size_t bytes = bytes_of(whole, Q, true);
    cudaError_t e = allow(ssm_grad_kernel<T, Q>, bytes);
    if (e == cudaSuccess && s.count > 1) e = states<T, Q>(span_of(whole, s, 0, s.chunks, Q, true), 0, 1, st);
    for (int i = s.count - 1; i >= 0 && e == cudaSuccess; --i) {
        const Args a = span_of(whole, s, i * s.per, s.per, Q, true);
        if ((e = s.count > 1 ? states<T, Q>(a, 1, 1, st) : states<T, Q>(a, 0, 2, st)) != cudaSuccess) break;
        ssm_grad_kernel<T, Q><<<(unsigned)((size_t)a.B * a.G * a.nc * a.splits), kThreads, bytes, st>>>(a);
        if ((e = cudaGetLastError()) == cudaSuccess) e = join_parts(a, dt, st);
    }
    return e == cudaSuccess ? join_sums(whole, whole.B * s.chunks, st) : e;
}

}  // namespace

size_t simt_space(Args &a, bool backward, uint8_t *base) {
    const Spans s(a, simt_chunk(a.P, a.N));
    size_t at = 0;
    auto take = [&](size_t floats) {
        float *p = base ? reinterpret_cast<float *>(base + at) : nullptr;
        at += align256(floats * 4);
        return p;
    };
    const size_t heads = (size_t)a.B * a.H, NP = (size_t)a.N * a.P, held = backward ? s.chunks : s.per;
    a.h = take(heads * held * NP);
    a.factor = take(heads * held);
    a.carry = take(s.count > 1 ? heads * NP : 0);
    if (backward) {
        a.splits = splits_of(a, s);
        const size_t rows = (size_t)s.per * simt_chunk(a.P, a.N) < (size_t)a.n ? (size_t)s.per * simt_chunk(a.P, a.N) : (size_t)a.n;
        a.g = take(heads * s.per * NP);
        a.dbc = take((size_t)a.splits * 2 * a.B * a.G * rows * a.N);
        a.sums = take((size_t)a.B * s.chunks * 3 * a.H);
    }
    return at;
}

cudaError_t simt_forward(const Args &a, hla_dtype dt, cudaStream_t st) {
    if (simt_chunk(a.P, a.N) == 64) return dt == HLA_F32 ? run_forward<float, 64>(a, st) : run_forward<__nv_bfloat16, 64>(a, st);
    return dt == HLA_F32 ? run_forward<float, 32>(a, st) : run_forward<__nv_bfloat16, 32>(a, st);
}
cudaError_t simt_backward(const Args &a, hla_dtype dt, cudaStream_t st) {
    if (simt_chunk(a.P, a.N) == 64) return dt == HLA_F32 ? run_backward<float, 64>(a, dt, st) : run_backward<__nv_bfloat16, 64>(a, dt, st);
    return dt == HLA_F32 ? run_backward<float, 32>(a, dt, st) : run_backward<__nv_bfloat16, 32>(a, dt, st);
}

cudaError_t join_parts(const Args &a, hla_dtype dt, cudaStream_t st) {
    const size_t blocks = ((size_t)a.B * a.G * a.rows + 7) / 8;
    const dim3 grid((unsigned)(blocks < 4096 ? blocks : 4096), 2);
    if (dt == HLA_F32)
        ssm_join_kernel<float><<<grid, 256, 0, st>>>(a);
    else
        ssm_join_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(a);
    return cudaGetLastError();
}
cudaError_t join_sums(const Args &a, int rows, cudaStream_t st) {
    ssm_sums_kernel<<<(unsigned)((3LL * a.H + 31) / 32), 256, 0, st>>>(a, rows);
    return cudaGetLastError();
}

}  // namespace ssm
}  // namespace hla
