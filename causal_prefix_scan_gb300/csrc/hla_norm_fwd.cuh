// hla_norm_fwd.cuh -- forward kernels of the grouped norm (see hla_norm.cuh).
#pragma once
#include "hla_norm.cuh"

namespace hla {
namespace norm {
namespace {

template <typename T, int VEC, int E, int TEAM, int GATE>
__global__ void __launch_bounds__(block_of(TEAM), (E == 8 ? kForwardThreads : 1024) / block_of(TEAM)) norm_forward_kernel(const Args a) {
    constexpr int K = E / VEC, PER = block_of(TEAM) / TEAM, ROWS = GATE != GATE_NONE ? 2 : 1;
    __shared__ alignas(16) float2 red[2][block_of(TEAM) / 32];
    __shared__ uint4 slots[ahead_slots<T, VEC, K, block_of(TEAM), ROWS>()];
    const Ahead<T, VEC, K, block_of(TEAM), ROWS> next{slots};
    const int tl = threadIdx.x % TEAM, g = blockIdx.x % a.col_blocks * PER + threadIdx.x / TEAM;
    bool ok[K];
#pragma unroll
    for (int k = 0; k < K; ++k) ok[k] = g < a.groups && (k * TEAM + tl) * VEC < a.m;
    const size_t at = (size_t)g * a.m + (size_t)tl * VEC;
    const float inv = 1.f / (float)a.m;
    int turn = 0;
    Rows r(a, blockIdx.x / a.col_blocks);
    auto ask = [&] {
        if (!next.ON || !r.live()) return;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (ok[k]) {
                next.ask(0, k, row_in<T>(a.x, r.b, r.t) + at + k * TEAM * VEC);
                if (GATE != GATE_NONE) next.ask(1, k, row_in<T>(a.z, r.b, r.t) + at + k * TEAM * VEC);
            }
    };
    ask();
    while (r.live()) {
        const int b = r.b, t = r.t;
        float u[E];
        raw_t<T, VEC> x[K], z[K];
        if (next.ON) next.wait();
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (ok[k]) {
                x[k] = next.ON ? next.take(0, k) : load_raw<T, VEC>(row_in<T>(a.x, b, t) + at + k * TEAM * VEC);
                if (GATE != GATE_NONE) z[k] = next.ON ? next.take(1, k) : load_raw<T, VEC>(row_in<T>(a.z, b, t) + at + k * TEAM * VEC);
            }
        r.next();
        ask();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float f[VEC];
            widen<T, VEC>(x[k], f);
            if (GATE == GATE_BEFORE) {
                float gz[VEC];
                widen<T, VEC>(z[k], gz);
#pragma unroll
                for (int v = 0; v < VEC; ++v) f[v] *= silu(gz[v]);
            }
#pragma unroll
            for (int v = 0; v < VEC; ++v) u[k * VEC + v] = ok[k] ? f[v] : 0.f;
        }
        if (a.center) {
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) s += u[e];
            const float mean = team_sum<TEAM>(s, red[turn]) * inv;
            turn ^= 1;
#pragma unroll
            for (int e = 0; e < E; ++e) u[e] = ok[e / VEC] ? u[e] - mean : 0.f;
        }
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s = fmaf(u[e], u[e], s);
        const float rs = rsqrtf(fmaf(team_sum<TEAM>(s, red[turn]), inv, a.eps));
        turn ^= 1;
        T *y = row_to<T>(a.y, b, t) + at;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (!ok[k]) continue;
            float o[VEC], gz[VEC], w[VEC], bias[VEC];
            scale_of<VEC>(a.weight, at + k * TEAM * VEC, true, 1.f, w);
            scale_of<VEC>(a.bias, at + k * TEAM * VEC, true, 0.f, bias);
            if (GATE == GATE_AFTER) widen<T, VEC>(z[k], gz);
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                o[v] = fmaf(u[k * VEC + v] * rs, w[v], bias[v]);
                if (GATE == GATE_AFTER)
                    o[v] *= silu(gz[v]);
                else if (GATE == GATE_NONE && a.silu)
                    o[v] = silu(o[v]);
            }
            store_raw<T, VEC>(y + k * TEAM * VEC, narrow<T, VEC>(o));
        }
    }
}

// Groups wider than a team holds: one CTA per group and token, three passes.
template <typename T>
__global__ void __launch_bounds__(256) norm_forward_long_kernel(const Args a) {
    __shared__ alignas(16) float2 red[2][8];
    const int g = blockIdx.x % a.col_blocks;
    const size_t at = (size_t)g * a.m;
    const float inv = 1.f / (float)a.m;
    for (Rows r(a, blockIdx.x / a.col_blocks); r.live(); r.next()) {
        const T *x = row_in<T>(a.x, r.b, r.t) + at;
        const T *z = a.gate != GATE_NONE ? row_in<T>(a.z, r.b, r.t) + at : nullptr;
        auto value = [&](int c, float &gate) {
            float v[1];
            widen<T, 1>(load_raw<T, 1>(x + c), v);
            float u = v[0];
            gate = 1.f;
            if (z) {
                widen<T, 1>(load_raw<T, 1>(z + c), v);
                gate = silu(v[0]);
            }
            return a.gate == GATE_BEFORE ? u * gate : u;
        };
        float mean = 0.f, s = 0.f, gate;
        if (a.center) {
            for (int c = threadIdx.x; c < a.m; c += 256) s += value(c, gate);
            mean = team_sum<256>(s, red[0]) * inv;
        }
        s = 0.f;
        for (int c = threadIdx.x; c < a.m; c += 256) {
            const float u = value(c, gate) - mean;
            s = fmaf(u, u, s);
        }
        const float rs = rsqrtf(fmaf(team_sum<256>(s, red[1]), inv, a.eps));
        T *y = row_to<T>(a.y, r.b, r.t) + at;
        for (int c = threadIdx.x; c < a.m; c += 256) {
            const float u = value(c, gate) - mean;
            float o[1] = {fmaf(u * rs, a.weight ? __ldg(a.weight + at + c) : 1.f, a.bias ? __ldg(a.bias + at + c) : 0.f)};
            if (a.gate == GATE_AFTER) o[0] *= gate;
            if (a.gate == GATE_NONE && a.silu) o[0] = silu(o[0]);
            store_raw<T, 1>(y + c, narrow<T, 1>(o));
        }
        __syncthreads();
    }
}

template <typename T, int VEC, int E, int TEAM, int GATE>
struct Forward {
    static void go(const Args &a, cudaStream_t st) {
        norm_forward_kernel<T, VEC, E, TEAM, GATE><<<(unsigned)(a.col_blocks * a.row_blocks), block_of(TEAM), 0, st>>>(a);
    }
};
template <typename T>
void forward(const Args &a, bool wide, cudaStream_t st) {
    const Team t = team_of(a.m);
    if (!t.E)
        norm_forward_long_kernel<T><<<(unsigned)(a.col_blocks * a.row_blocks), 256, 0, st>>>(a);
    else
        wide ? by_team<Forward, T, 16 / sizeof(T)>(a, t, st) : by_team<Forward, T, 1>(a, t, st);
}

}  // namespace
}  // namespace norm
}  // namespace hla
