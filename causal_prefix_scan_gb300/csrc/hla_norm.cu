// hla_norm.cu -- forward of the grouped norm (see hla_norm.cuh), and its entry points.
#include <cmath>

#include "hla_norm.cuh"

namespace hla {
namespace norm {
namespace {

constexpr int kThreadsPerSm = 1280;

template <typename T, int VEC, int E, int TEAM>
__global__ void __launch_bounds__(block_of(TEAM), (E == 8 ? kThreadsPerSm : 1024) / block_of(TEAM)) norm_forward_kernel(const Args a) {
    constexpr int K = E / VEC, PER = block_of(TEAM) / TEAM;
    __shared__ float2 red[2][block_of(TEAM) / 32];
    const int tl = threadIdx.x % TEAM, g = blockIdx.x % a.col_blocks * PER + threadIdx.x / TEAM;
    bool ok[K];
#pragma unroll
    for (int k = 0; k < K; ++k) ok[k] = g < a.groups && (k * TEAM + tl) * VEC < a.m;
    const size_t at = (size_t)g * a.m + (size_t)tl * VEC;
    const float inv = 1.f / (float)a.m;
    int turn = 0;
    for (Rows r(a, blockIdx.x / a.col_blocks); r.live(); r.next()) {
        const int b = r.b, t = r.t;
        float u[E];
        raw_t<T, VEC> x[K], z[K];
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (ok[k]) {
                x[k] = load_raw<T, VEC>(row_in<T>(a.x, b, t) + at + k * TEAM * VEC);
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
        T *y = row_to<T>(a.y, b, t) + at;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (!ok[k]) continue;
            float o[VEC], gz[VEC], w[VEC], bias[VEC];
            scale_of<VEC>(a.weight, at + k * TEAM * VEC, true, 1.f, w);
            scale_of<VEC>(a.bias, at + k * TEAM * VEC, true, 0.f, bias);
            if (a.gate == GATE_AFTER) widen<T, VEC>(z[k], gz);
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                o[v] = fmaf(u[k * VEC + v] * rs, w[v], bias[v]);
                if (a.gate == GATE_AFTER)
                    o[v] *= silu(gz[v]);
                else if (a.gate == GATE_NONE && a.silu)
                    o[v] = silu(o[v]);
            }
            store_raw<T, VEC>(y + k * TEAM * VEC, narrow<T, VEC>(o));
        }
    }
}

// Groups wider than a team holds: one CTA per group and token, three passes.
template <typename T>
__global__ void __launch_bounds__(256) norm_forward_long_kernel(const Args a) {
    __shared__ float2 red[2][8];
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
            mean = team_sum<256>(make_float2(s, 0.f), red[0]).x * inv;
        }
        s = 0.f;
        for (int c = threadIdx.x; c < a.m; c += 256) {
            const float u = value(c, gate) - mean;
            s = fmaf(u, u, s);
        }
        const float rs = rsqrtf(fmaf(team_sum<256>(make_float2(s, 0.f), red[1]).x, inv, a.eps));
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

template <typename T, int VEC, int E, int TEAM>
void launch(const Args &a, cudaStream_t st) {
    norm_forward_kernel<T, VEC, E, TEAM><<<(unsigned)(a.col_blocks * a.row_blocks), block_of(TEAM), 0, st>>>(a);
}
template <typename T, int VEC, int E>
void by_team(const Args &a, int team, cudaStream_t st) {
    if (team == 8) return launch<T, VEC, E, 8>(a, st);
    if (team == 32) return launch<T, VEC, E, 32>(a, st);
    if (team == 128) return launch<T, VEC, E, 128>(a, st);
    launch<T, VEC, E, 512>(a, st);
}
template <typename T>
cudaError_t forward(const Args &a, bool wide, cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    const Team t = team_of(a.m);
    if (!t.E)
        norm_forward_long_kernel<T><<<(unsigned)(a.col_blocks * a.row_blocks), 256, 0, st>>>(a);
    else if (t.E == 8)
        wide ? by_team<T, V, 8>(a, t.threads, st) : by_team<T, 1, 8>(a, t.threads, st);
    else
        wide ? by_team<T, V, 16>(a, t.threads, st) : by_team<T, 1, 16>(a, t.threads, st);
    return cudaGetLastError();
}

hla_status check(const hla_norm_params *p) {
    if (!p) return report(HLA_ERR_ARG, "params is NULL");
    if (p->B < 1 || p->d < 1 || p->n < 0) return report(HLA_ERR_ARG, "need B >= 1, d >= 1, n >= 0");
    if (p->groups < 1 || p->d % p->groups) return report(HLA_ERR_ARG, "d must be a multiple of groups >= 1");
    if (p->in_dtype != HLA_F32 && p->in_dtype != HLA_BF16) return report(HLA_ERR_ARG, "unknown in_dtype");
    if (p->activation != HLA_ACT_NONE && p->activation != HLA_ACT_SILU) return report(HLA_ERR_ARG, "unknown activation");
    if (!std::isfinite(p->eps) || p->eps < 0.f) return report(HLA_ERR_ARG, "eps must be finite and not negative");
    if ((reinterpret_cast<uintptr_t>(p->weight) & 3u) || (reinterpret_cast<uintptr_t>(p->bias) & 3u))
        return report(HLA_ERR_ARG, "weight or bias is not aligned to its elements");
    if (p->n > 2147483647 - 1024 || (double)p->B * p->n > 4e18 || p->d > 1 << 30) return report(HLA_ERR_ARG, "problem too large");
    return HLA_OK;
}
hla_status check_gate(const hla_norm_params *p, const hla_tensor *gate) {
    if (!gate && p->gate_first) return report(HLA_ERR_ARG, "gate_first needs a gate");
    if (gate && p->activation != HLA_ACT_SILU) return report(HLA_ERR_ARG, "a gate goes through HLA_ACT_SILU");
    return HLA_OK;
}

Args make(const hla_norm_params *p, bool gated, int threads_per_sm) {
    Args a{};
    a.B = p->B; a.n = p->n; a.d = p->d; a.groups = p->groups;
    a.m = p->d / p->groups;
    a.col_blocks = columns_of(a.groups, a.m);
    a.row_blocks = row_blocks_of((long long)p->B * p->n, a.groups, a.m, threads_per_sm);
    a.gate = !gated ? GATE_NONE : p->gate_first ? GATE_BEFORE : GATE_AFTER;
    a.center = p->center != 0;
    a.silu = p->activation == HLA_ACT_SILU;
    a.eps = p->eps;
    a.weight = p->weight; a.bias = p->bias;
    a.lengths = p->lengths;
    return a;
}
bool wide_rows(const hla_norm_params *p, const Args &a, std::initializer_list<const View *> rows) {
    const size_t el = p->in_dtype == HLA_F32 ? 4 : 2;
    if (a.m * el % 16 || (reinterpret_cast<uintptr_t>(a.weight) & 15u) || (reinterpret_cast<uintptr_t>(a.bias) & 15u)) return false;
    for (const View *v : rows)
        if (v->p && !rows16(*v, el)) return false;
    return true;
}
constexpr int kThreadsPerSmBackward = 1024, kMostRowBlocks = kSms * (kThreadsPerSmBackward / 256);

}  // namespace
}  // namespace norm
}  // namespace hla

using namespace hla;
using namespace hla::norm;

extern "C" {

hla_status hla_norm_forward(const hla_norm_params *p, const hla_tensor *x, const hla_tensor *gate, const hla_tensor *y,
                            void *stream) {
    hla_status s = norm::check(p);
    if (s != HLA_OK || (s = check_gate(p, gate)) != HLA_OK) return s;
    if (p->n == 0) return HLA_OK;
    const hla_dtype dt = p->in_dtype;
    const Dims d{p->B, 1, p->n, p->d};
    if ((s = check_in(x, d, dt, "x must be set")) != HLA_OK ||
        (gate && (s = check_in(gate, d, dt, "gate must be set")) != HLA_OK) ||
        (s = check_out(y, d, dt, "y must be set")) != HLA_OK)
        return s;
    if (y->p == x->p || (gate && y->p == gate->p)) return report(HLA_ERR_ARG, "y may not be an input");
    Args a = make(p, gate != nullptr, kThreadsPerSm);
    a.x = view(x, d); a.y = view(y, d);
    if (gate) a.z = view(gate, d);
    const bool wide = wide_rows(p, a, {&a.x, &a.y, &a.z});
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dt == HLA_F32 ? forward<float>(a, wide, st) : forward<__nv_bfloat16>(a, wide, st);
    return e == cudaSuccess ? HLA_OK : report(HLA_ERR_CUDA, cudaGetErrorString(e));
}

size_t hla_norm_backward_workspace_size(const hla_norm_params *p) {
    if (norm::check(p) != HLA_OK || p->n == 0) return 0;
    const long long rows = (long long)p->B * p->n;  // one size for every number of groups
    return align256((size_t)(rows < kMostRowBlocks ? rows : kMostRowBlocks) * 2 * p->d * 4);
}

hla_status hla_norm_backward(const hla_norm_params *p, const hla_tensor *x, const hla_tensor *gate, const hla_tensor *dy,
                             const hla_tensor *dx, const hla_tensor *d_gate, float *d_weight, float *d_bias,
                             void *workspace, size_t workspace_bytes, void *stream) {
    hla_status s = norm::check(p);
    if (s != HLA_OK || (s = check_gate(p, gate)) != HLA_OK) return s;
    if ((reinterpret_cast<uintptr_t>(d_weight) & 3u) || (reinterpret_cast<uintptr_t>(d_bias) & 3u))
        return report(HLA_ERR_ARG, "d_weight or d_bias is not aligned to its elements");
    if (!gate != !d_gate) return report(HLA_ERR_ARG, "d_gate belongs to a gate, which needs it");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (p->n == 0) {
        cudaError_t e = cudaSuccess;
        if (d_weight) e = cudaMemsetAsync(d_weight, 0, (size_t)p->d * 4, st);
        if (e == cudaSuccess && d_bias) e = cudaMemsetAsync(d_bias, 0, (size_t)p->d * 4, st);
        return e == cudaSuccess ? HLA_OK : report(HLA_ERR_CUDA, cudaGetErrorString(e));
    }
    const hla_dtype dt = p->in_dtype;
    const Dims d{p->B, 1, p->n, p->d};
    if ((s = check_in(x, d, dt, "x must be set")) != HLA_OK || (s = check_in(dy, d, dt, "dy must be set")) != HLA_OK ||
        (gate && (s = check_in(gate, d, dt, "gate must be set")) != HLA_OK) ||
        (s = check_out(dx, d, dt, "dx must be set")) != HLA_OK ||
        (gate && (s = check_out(d_gate, d, dt, "d_gate must be set")) != HLA_OK))
        return s;
    for (const hla_tensor *o : {dx, d_gate})
        for (const hla_tensor *i : {x, dy, gate})
            if (o && i && o->p == i->p) return report(HLA_ERR_ARG, "dx and d_gate may not be inputs");
    if (d_gate && d_gate->p == dx->p) return report(HLA_ERR_ARG, "dx may not be d_gate");
    if (!workspace || workspace_bytes < hla_norm_backward_workspace_size(p))
        return report(HLA_ERR_ARG, "workspace too small (hla_norm_backward_workspace_size)");
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return report(HLA_ERR_ARG, "workspace must be 256-byte aligned");
    Args a = make(p, gate != nullptr, kThreadsPerSmBackward);
    a.x = view(x, d); a.dy = view(dy, d); a.dx = view(dx, d);
    if (gate) a.z = view(gate, d), a.dz = view(d_gate, d);
    a.part = static_cast<float *>(workspace);
    const cudaError_t e = backward(a, dt, wide_rows(p, a, {&a.x, &a.dy, &a.dx, &a.z, &a.dz}), d_weight, d_bias, st);
    return e == cudaSuccess ? HLA_OK : report(HLA_ERR_CUDA, cudaGetErrorString(e));
}

}  // extern "C"
