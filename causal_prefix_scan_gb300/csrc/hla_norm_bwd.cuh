// hla_norm_bwd.cuh -- backward kernels of the grouped norm (see hla_norm.cuh).
#pragma once
#include "hla_norm.cuh"

namespace hla {
namespace norm {
namespace {

// Gradient of v (the scaled and shifted norm) and of the gate behind it.
struct Behind {
    float dv, dgate;
};
HLA_DEVICE Behind behind(int gate_kind, bool act, float dy, float v, float gate) {
    if (gate_kind == GATE_AFTER) {
        const float s = sigmoid(gate);
        return {dy * gate * s, dy * v * silu_slope(gate, s)};
    }
    if (gate_kind == GATE_NONE && act) return {dy * silu_slope(v, sigmoid(v)), 0.f};
    return {dy, 0.f};
}

template <typename T, int VEC, int E, int TEAM, int GATE>
__global__ void __launch_bounds__(block_of(TEAM), (E == 8 ? kBackwardThreads : 512) / block_of(TEAM)) norm_backward_kernel(const Args a) {
    constexpr int K = E / VEC, PER = block_of(TEAM) / TEAM, STEP = TEAM * VEC;
    using Raw = raw_t<T, VEC>;
    __shared__ alignas(16) float2 red[2][block_of(TEAM) / 32];
    constexpr int ROWS = GATE != GATE_NONE ? 3 : 2;
    __shared__ uint4 slots[ahead_slots<T, VEC, K, block_of(TEAM), ROWS>()];
    const Ahead<T, VEC, K, block_of(TEAM), ROWS> next{slots};
    __shared__ alignas(16) float sig[GATE == GATE_BEFORE ? E * block_of(TEAM) : 4];  // the gate's sigmoid, for the end
    const int tl = threadIdx.x % TEAM, g = blockIdx.x % a.col_blocks * PER + threadIdx.x / TEAM;
    bool ok[K];
    float dw[K][VEC], db[K][VEC];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        ok[k] = g < a.groups && (k * TEAM + tl) * VEC < a.m;
        fill_v<VEC>(0.f, dw[k]);
        fill_v<VEC>(0.f, db[k]);
    }
    const size_t at = (size_t)g * a.m + (size_t)tl * VEC;
    const float inv = 1.f / (float)a.m;
    int turn = 0;
    Rows r(a, blockIdx.x / a.col_blocks);
    auto ask = [&] {
        if (!next.ON || !r.live()) return;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (ok[k]) {
                next.ask(0, k, row_in<T>(a.x, r.b, r.t) + at + k * STEP);
                next.ask(1, k, row_in<T>(a.dy, r.b, r.t) + at + k * STEP);
                if (GATE != GATE_NONE) next.ask(2, k, row_in<T>(a.z, r.b, r.t) + at + k * STEP);
            }
    };
    ask();
    while (r.live()) {
        const int b = r.b, t = r.t;
        float u[K][VEC], q[K][VEC];  // the norm's input, then itself; gradients (zeros beside the group)
        Raw x[K], z[K], d[K];
        const T *px = row_in<T>(a.x, b, t) + at, *pd = row_in<T>(a.dy, b, t) + at;
        const T *pz = GATE != GATE_NONE ? row_in<T>(a.z, b, t) + at : nullptr;
        if (next.ON) next.wait();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            x[k] = d[k] = z[k] = Raw{};
            if (ok[k]) {
                x[k] = next.ON ? next.take(0, k) : load_raw<T, VEC>(px + k * STEP);
                d[k] = next.ON ? next.take(1, k) : load_raw<T, VEC>(pd + k * STEP);
                if (GATE != GATE_NONE) z[k] = next.ON ? next.take(2, k) : load_raw<T, VEC>(pz + k * STEP);
            }
        }
        r.next();
        ask();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            widen<T, VEC>(x[k], u[k]);
            if (GATE == GATE_BEFORE) {
                float gz[VEC], s[VEC];
                widen<T, VEC>(z[k], gz);
#pragma unroll
                for (int v = 0; v < VEC; ++v) s[v] = sigmoid(gz[v]);
                lay_aside<VEC, block_of(TEAM)>(sig, k, s);
                mul_v<VEC>(gz, s, gz);
                mul_v<VEC>(u[k], gz, u[k]);
            }
        }
        if (a.center) {
            float s = 0.f;
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int v = 0; v < VEC; ++v) s += u[k][v];
            const float mean = team_sum<TEAM>(s, red[turn]) * inv;
            turn ^= 1;
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int v = 0; v < VEC; ++v) u[k][v] = ok[k] ? u[k][v] - mean : 0.f;
        }
        float sq[VEC], s = 0.f;
        fill_v<VEC>(0.f, sq);
#pragma unroll
        for (int k = 0; k < K; ++k) fma_v<VEC>(u[k], u[k], sq, sq);
#pragma unroll
        for (int v = 0; v < VEC; ++v) s += sq[v];
        const float rs = rsqrtf(fmaf(team_sum<TEAM>(s, red[turn]), inv, a.eps));
        turn ^= 1;
        float fr[VEC], s1[VEC], s0[VEC];
        fill_v<VEC>(rs, fr);
        fill_v<VEC>(0.f, s1);
        fill_v<VEC>(0.f, s0);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float w[VEC];
            scale_of<VEC>(a.weight, at + k * STEP, ok[k], 1.f, w);
            mul_v<VEC>(u[k], fr, u[k]);
            widen<T, VEC>(d[k], q[k]);
            if (GATE == GATE_AFTER || (GATE == GATE_NONE && a.silu)) {
                float c[VEC], gz[VEC], dz[VEC];
                scale_of<VEC>(a.bias, at + k * STEP, ok[k], 0.f, c);
                fma_v<VEC>(u[k], w, c, c);
                if (GATE == GATE_AFTER) widen<T, VEC>(z[k], gz);
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    const Behind o = behind(GATE, true, q[k][v], c[v], GATE == GATE_AFTER ? gz[v] : 0.f);
                    q[k][v] = o.dv;
                    dz[v] = o.dgate;
                }
                if (GATE == GATE_AFTER && ok[k]) store_raw<T, VEC>(row_to<T>(a.dz, b, t) + at + k * STEP, narrow<T, VEC>(dz));
            }
            fma_v<VEC>(q[k], u[k], dw[k], dw[k]);
            add_v<VEC>(db[k], q[k], db[k]);
            mul_v<VEC>(q[k], w, q[k]);
            fma_v<VEC>(q[k], u[k], s1, s1);
            add_v<VEC>(s0, q[k], s0);
        }
        float2 sums = make_float2(0.f, 0.f);
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            sums.x += s1[v];
            sums.y += s0[v];
        }
        sums = team_sum<TEAM>(sums, red[turn]);
        turn ^= 1;
        float c1[VEC], c0[VEC];  // du = rs q - u (rs c1) - rs c0
        fill_v<VEC>(-rs * sums.x * inv, c1);
        fill_v<VEC>(a.center ? -rs * sums.y * inv : 0.f, c0);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (!ok[k]) continue;
            float o[VEC];
            fma_v<VEC>(u[k], c1, c0, o);
            fma_v<VEC>(q[k], fr, o, o);
            if (GATE == GATE_BEFORE) {
                float gz[VEC], f[VEC], s[VEC], sl[VEC];
                widen<T, VEC>(z[k], gz);
                widen<T, VEC>(x[k], f);
                take_back<VEC, block_of(TEAM)>(sig, k, s);
                silu_slope_v<VEC>(gz, s, sl);
                mul_v<VEC>(gz, s, gz);
                mul_v<VEC>(f, sl, f);
                mul_v<VEC>(o, f, f);
                mul_v<VEC>(o, gz, o);
                store_raw<T, VEC>(row_to<T>(a.dz, b, t) + at + k * STEP, narrow<T, VEC>(f));
            }
            store_raw<T, VEC>(row_to<T>(a.dx, b, t) + at + k * STEP, narrow<T, VEC>(o));
        }
    }
    float *part = a.part + (size_t)(blockIdx.x / a.col_blocks) * 2 * a.d + at;
#pragma unroll
    for (int k = 0; k < K; ++k)
        if (ok[k]) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                part[k * STEP + v] = dw[k][v];
                part[a.d + k * STEP + v] = db[k][v];
            }
        }
}

// Groups wider than a team holds: one CTA per group, its rows one after the other in four passes;
// each channel's sums stay with the thread that owns it, in the workspace.
template <typename T>
__global__ void __launch_bounds__(256) norm_backward_long_kernel(const Args a) {
    __shared__ alignas(16) float2 red[3][8];
    const int g = blockIdx.x % a.col_blocks;
    const size_t at = (size_t)g * a.m;
    const float inv = 1.f / (float)a.m;
    float *part = a.part + (size_t)(blockIdx.x / a.col_blocks) * 2 * a.d + at;
    for (int c = threadIdx.x; c < a.m; c += 256) part[c] = part[a.d + c] = 0.f;
    for (Rows r(a, blockIdx.x / a.col_blocks); r.live(); r.next()) {
        const T *x = row_in<T>(a.x, r.b, r.t) + at, *d = row_in<T>(a.dy, r.b, r.t) + at;
        const T *z = a.gate != GATE_NONE ? row_in<T>(a.z, r.b, r.t) + at : nullptr;
        auto read = [](const T *p) {
            float v[1];
            widen<T, 1>(load_raw<T, 1>(p), v);
            return v[0];
        };
        auto value = [&](int c) { return a.gate == GATE_BEFORE ? read(x + c) * silu(read(z + c)) : read(x + c); };
        float mean = 0.f, s = 0.f;
        if (a.center) {
            for (int c = threadIdx.x; c < a.m; c += 256) s += value(c);
            mean = team_sum<256>(s, red[0]) * inv;
        }
        s = 0.f;
        for (int c = threadIdx.x; c < a.m; c += 256) {
            const float u = value(c) - mean;
            s = fmaf(u, u, s);
        }
        const float rs = rsqrtf(fmaf(team_sum<256>(s, red[1]), inv, a.eps));
        float2 sums = make_float2(0.f, 0.f);
        for (int c = threadIdx.x; c < a.m; c += 256) {
            const float u = (value(c) - mean) * rs, w = a.weight ? __ldg(a.weight + at + c) : 1.f;
            const Behind o = behind(a.gate, a.silu, read(d + c), fmaf(u, w, a.bias ? __ldg(a.bias + at + c) : 0.f), z ? read(z + c) : 0.f);
            part[c] = fmaf(o.dv, u, part[c]);
            part[a.d + c] += o.dv;
            sums.x = fmaf(o.dv * w, u, sums.x);
            sums.y = fmaf(o.dv, w, sums.y);
            if (a.gate == GATE_AFTER) {
                const float f[1] = {o.dgate};
                store_raw<T, 1>(row_to<T>(a.dz, r.b, r.t) + at + c, narrow<T, 1>(f));
            }
        }
        sums = team_sum<256>(sums, red[2]);
        const float c1 = sums.x * inv, c0 = a.center ? sums.y * inv : 0.f;
        for (int c = threadIdx.x; c < a.m; c += 256) {
            const float u = (value(c) - mean) * rs, w = a.weight ? __ldg(a.weight + at + c) : 1.f;
            const Behind o = behind(a.gate, a.silu, read(d + c), fmaf(u, w, a.bias ? __ldg(a.bias + at + c) : 0.f), z ? read(z + c) : 0.f);
            float f[1] = {rs * (o.dv * w - fmaf(u, c1, c0))};
            if (a.gate == GATE_BEFORE) {
                const float gz = read(z + c), sg = sigmoid(gz), dz[1] = {f[0] * read(x + c) * silu_slope(gz, sg)};
                f[0] *= gz * sg;
                store_raw<T, 1>(row_to<T>(a.dz, r.b, r.t) + at + c, narrow<T, 1>(dz));
            }
            store_raw<T, 1>(row_to<T>(a.dx, r.b, r.t) + at + c, narrow<T, 1>(f));
        }
        __syncthreads();
    }
}

template <typename T, int VEC, int E, int TEAM, int GATE>
struct Backward {
    static void go(const Args &a, cudaStream_t st) {
        norm_backward_kernel<T, VEC, E, TEAM, GATE><<<(unsigned)(a.col_blocks * a.row_blocks), block_of(TEAM), 0, st>>>(a);
    }
};
template <typename T>
void backward(const Args &a, bool wide, cudaStream_t st) {
    const Team t = team_of(a.m);
    if (!t.E)
        norm_backward_long_kernel<T><<<(unsigned)(a.col_blocks * a.row_blocks), 256, 0, st>>>(a);
    else
        wide ? by_team<Backward, T, 16 / sizeof(T)>(a, t, st) : by_team<Backward, T, 1>(a, t, st);
}

}  // namespace
}  // namespace norm
}  // namespace hla
