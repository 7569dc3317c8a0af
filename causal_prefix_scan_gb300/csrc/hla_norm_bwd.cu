// hla_norm_bwd.cu -- backward of the grouped norm (see hla_norm.cuh).
#include "hla_norm.cuh"

namespace hla {
namespace norm {
namespace {

// Gradient of v (the scaled and shifted norm) and of the gate behind it.
struct Behind {
    float dv, dgate;
};
HLA_DEVICE Behind behind(const Args &a, float dy, float v, float gate) {
    if (a.gate == GATE_AFTER) {
        const float s = sigmoid(gate);
        return {dy * gate * s, dy * v * silu_slope(gate, s)};
    }
    if (a.gate == GATE_NONE && a.silu) return {dy * silu_slope(v, sigmoid(v)), 0.f};
    return {dy, 0.f};
}

template <typename T, int VEC, int E, int TEAM>
__global__ void __launch_bounds__(block_of(TEAM), (E == 8 ? 1024 : 512) / block_of(TEAM)) norm_backward_kernel(const Args a) {
    constexpr int K = E / VEC, PER = block_of(TEAM) / TEAM;
    __shared__ float2 red[2][block_of(TEAM) / 32];
    const int tl = threadIdx.x % TEAM, g = blockIdx.x % a.col_blocks * PER + threadIdx.x / TEAM;
    bool ok[K];
    float dw[E], db[E];
#pragma unroll
    for (int k = 0; k < K; ++k) ok[k] = g < a.groups && (k * TEAM + tl) * VEC < a.m;
#pragma unroll
    for (int e = 0; e < E; ++e) dw[e] = db[e] = 0.f;
    const size_t at = (size_t)g * a.m + (size_t)tl * VEC;
    const float inv = 1.f / (float)a.m;
    int turn = 0;
    for (Rows r(a, blockIdx.x / a.col_blocks); r.live(); r.next()) {
        const int b = r.b, t = r.t;
        float u[E], q[E];  // the norm's input, then itself; gradients
        raw_t<T, VEC> x[K], z[K], d[K];
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (ok[k]) {
                x[k] = load_raw<T, VEC>(row_in<T>(a.x, b, t) + at + k * TEAM * VEC);
                d[k] = load_raw<T, VEC>(row_in<T>(a.dy, b, t) + at + k * TEAM * VEC);
                if (a.gate != GATE_NONE) z[k] = load_raw<T, VEC>(row_in<T>(a.z, b, t) + at + k * TEAM * VEC);
            }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float f[VEC];
            widen<T, VEC>(x[k], f);
            if (a.gate == GATE_BEFORE) {
                float gz[VEC];
                widen<T, VEC>(z[k], gz);
#pragma unroll
                for (int v = 0; v < VEC; ++v) f[v] *= silu(gz[v]);
            }
#pragma unroll
            for (int v = 0; v < VEC; ++v) u[k * VEC + v] = ok[k] ? f[v] : 0.f;
            widen<T, VEC>(d[k], f);
#pragma unroll
            for (int v = 0; v < VEC; ++v) q[k * VEC + v] = f[v];
        }
        if (a.center) {
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) s += u[e];
            const float mean = team_sum<TEAM>(make_float2(s, 0.f), red[turn]).x * inv;
            turn ^= 1;
#pragma unroll
            for (int e = 0; e < E; ++e) u[e] = ok[e / VEC] ? u[e] - mean : 0.f;
        }
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s = fmaf(u[e], u[e], s);
        const float rs = rsqrtf(fmaf(team_sum<TEAM>(make_float2(s, 0.f), red[turn]).x, inv, a.eps));
        turn ^= 1;
        float2 sums = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float gz[VEC], dz[VEC], w[VEC], c[VEC];
            if (a.gate == GATE_AFTER) widen<T, VEC>(z[k], gz);
            scale_of<VEC>(a.weight, at + k * TEAM * VEC, ok[k], 1.f, w);
            scale_of<VEC>(a.bias, at + k * TEAM * VEC, ok[k], 0.f, c);
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const int e = k * VEC + v;
                u[e] *= rs;
                const Behind o = behind(a, q[e], fmaf(u[e], w[v], c[v]), a.gate == GATE_AFTER ? gz[v] : 0.f);
                dz[v] = o.dgate;
                q[e] = ok[k] ? o.dv * w[v] : 0.f;
                if (ok[k]) {
                    dw[e] = fmaf(o.dv, u[e], dw[e]);
                    db[e] += o.dv;
                }
                sums.x = fmaf(q[e], u[e], sums.x);
                sums.y += q[e];
            }
            if (a.gate == GATE_AFTER && ok[k]) store_raw<T, VEC>(row_to<T>(a.dz, b, t) + at + k * TEAM * VEC, narrow<T, VEC>(dz));
        }
        sums = team_sum<TEAM>(sums, red[turn]);
        turn ^= 1;
        const float c1 = sums.x * inv, c0 = a.center ? sums.y * inv : 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (!ok[k]) continue;
            float o[VEC];
#pragma unroll
            for (int v = 0; v < VEC; ++v) o[v] = rs * (q[k * VEC + v] - fmaf(u[k * VEC + v], c1, c0));
            if (a.gate == GATE_BEFORE) {
                float gz[VEC], f[VEC], dz[VEC];
                widen<T, VEC>(z[k], gz);
                widen<T, VEC>(x[k], f);
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    const float sg = sigmoid(gz[v]);
                    dz[v] = o[v] * f[v] * silu_slope(gz[v], sg);
                    o[v] *= gz[v] * sg;
                }
                store_raw<T, VEC>(row_to<T>(a.dz, b, t) + at + k * TEAM * VEC, narrow<T, VEC>(dz));
            }
            store_raw<T, VEC>(row_to<T>(a.dx, b, t) + at + k * TEAM * VEC, narrow<T, VEC>(o));
        }
    }
    float *part = a.part + (size_t)(blockIdx.x / a.col_blocks) * 2 * a.d + at;
#pragma unroll
    for (int k = 0; k < K; ++k)
        if (ok[k]) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                part[k * TEAM * VEC + v] = dw[k * VEC + v];
                part[a.d + k * TEAM * VEC + v] = db[k * VEC + v];
            }
        }
}

// Groups wider than a team holds: one CTA per group, its rows one after the other in four passes;
// each channel's sums stay with the thread that owns it, in the workspace.
template <typename T>
__global__ void __launch_bounds__(256) norm_backward_long_kernel(const Args a) {
    __shared__ float2 red[3][8];
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
            mean = team_sum<256>(make_float2(s, 0.f), red[0]).x * inv;
        }
        s = 0.f;
        for (int c = threadIdx.x; c < a.m; c += 256) {
            const float u = value(c) - mean;
            s = fmaf(u, u, s);
        }
        const float rs = rsqrtf(fmaf(team_sum<256>(make_float2(s, 0.f), red[1]).x, inv, a.eps));
        float2 sums = make_float2(0.f, 0.f);
        for (int c = threadIdx.x; c < a.m; c += 256) {
            const float u = (value(c) - mean) * rs, w = a.weight ? __ldg(a.weight + at + c) : 1.f;
            const Behind o = behind(a, read(d + c), fmaf(u, w, a.bias ? __ldg(a.bias + at + c) : 0.f), z ? read(z + c) : 0.f);
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
            const Behind o = behind(a, read(d + c), fmaf(u, w, a.bias ? __ldg(a.bias + at + c) : 0.f), z ? read(z + c) : 0.f);
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

__global__ void __launch_bounds__(256) norm_sums_kernel(const float *part, int rows, int d, float *dw, float *db) {
    column_sums(part, rows, 2LL * d, [=](long long k, float s) {
        if (k < d) {
            if (dw) dw[k] = s;
        } else if (db) {
            db[k - d] = s;
        }
    });
}

template <typename T, int VEC, int E, int TEAM>
void launch(const Args &a, cudaStream_t st) {
    norm_backward_kernel<T, VEC, E, TEAM><<<(unsigned)(a.col_blocks * a.row_blocks), block_of(TEAM), 0, st>>>(a);
}
template <typename T, int VEC, int E>
void by_team(const Args &a, int team, cudaStream_t st) {
    if (team == 8) return launch<T, VEC, E, 8>(a, st);
    if (team == 32) return launch<T, VEC, E, 32>(a, st);
    if (team == 128) return launch<T, VEC, E, 128>(a, st);
    launch<T, VEC, E, 512>(a, st);
}
template <typename T>
void by_type(const Args &a, bool wide, cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    const Team t = team_of(a.m);
    if (!t.E)
        norm_backward_long_kernel<T><<<(unsigned)(a.col_blocks * a.row_blocks), 256, 0, st>>>(a);
    else if (t.E == 8)
        wide ? by_team<T, V, 8>(a, t.threads, st) : by_team<T, 1, 8>(a, t.threads, st);
    else
        wide ? by_team<T, V, 16>(a, t.threads, st) : by_team<T, 1, 16>(a, t.threads, st);
}

}  // namespace

cudaError_t backward(const Args &a, hla_dtype dt, bool wide, float *dw, float *db, cudaStream_t st) {
    dt == HLA_F32 ? by_type<float>(a, wide, st) : by_type<__nv_bfloat16>(a, wide, st);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || (!dw && !db)) return e;
    norm_sums_kernel<<<(unsigned)((2LL * a.d + 31) / 32), 256, 0, st>>>(a.part, a.row_blocks, a.d, dw, db);
    return cudaGetLastError();
}

}  // namespace norm
}  // namespace hla
