// hla_ssm.cu -- entry points of the selective state space scan, and its single-token step.
#include "hla_ssm.h"

namespace hla {
namespace ssm {
namespace {

// ------------------------------------------------------------ one token
// h = 2^a h + dt b x^T, y = c h + D x over the fp32 state [N][P] of one (sequence, head): read and
// written once, which bounds it.  LP lanes take VEC adjacent columns each and step down the rows;
// the rows' sums for y meet in shared memory.  kStepAhead rows are in flight, the first of them ahead
// of the decay, which waits for dt and A (b128 h64 p64 s128 67 us, 6.4 TB/s; behind it 73, one row at a
// time 89).  A CTA takes all columns of a head, or a few of them where the heads alone would leave SMs
// idle: columns need no sums between CTAs.
constexpr int kStepThreads = 256, kStepAhead = 4;

template <typename T, int VEC, int LP>
__global__ void __launch_bounds__(kStepThreads, 4) ssm_step_kernel(const Args a, float *state, int parts) {
    constexpr int ROWS = kStepThreads / LP;
    __shared__ float red[kStepThreads / 32][LP * VEC];
    const int part = blockIdx.x % parts, h = blockIdx.x / parts % a.H, b = blockIdx.x / parts / a.H;
    if (a.lengths && a.lengths[b] <= 0) return;
    const int tid = threadIdx.x, lp = tid % LP, p = (part * LP + lp) * VEC;
    const bool ok = p < a.P;
    const T *bt = static_cast<const T *>(a.b.p) + (size_t)b * a.b.sb + (size_t)(h / a.R) * a.b.sh;
    const T *ct = static_cast<const T *>(a.c.p) + (size_t)b * a.c.sb + (size_t)(h / a.R) * a.c.sh;
    const T *xt = static_cast<const T *>(a.x.p) + (size_t)b * a.x.sb + (size_t)h * a.x.sh;
    float *st = state + ((size_t)b * a.H + h) * a.N * a.P + p;
    raw_t<float, VEC> raw[kStepAhead];
    float bn[kStepAhead][1], cn[kStepAhead][1];
    auto fetch = [&](int n0) {
#pragma unroll
        for (int i = 0; i < kStepAhead; ++i) {
            const int n = n0 + i * ROWS;
            if (n < a.N && ok) raw[i] = load_raw<float, VEC>(st + (size_t)n * a.P);
            if (n < a.N) {
                widen<T, 1>(load_raw<T, 1>(bt + n), bn[i]);
                widen<T, 1>(load_raw<T, 1>(ct + n), cn[i]);
            }
        }
    };
    fetch(tid / LP);  // ahead of the decay, which waits for dt and A
    float slope, x[VEC], y[VEC];
    const float dt = step_of<T>(a, b, h, 0, a.softplus && a.dt_bias ? a.dt_bias[h] : 0.f, slope);
    const float decay = ex2_approx(log_decay(dt, a.A[h] * kLog2e));
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        float f[1] = {0.f};
        if (ok) widen<T, 1>(load_raw<T, 1>(xt + p + v), f);
        x[v] = f[0];
        y[v] = 0.f;
    }
    for (int n0 = tid / LP;;) {
#pragma unroll
        for (int i = 0; i < kStepAhead; ++i) {
            const int n = n0 + i * ROWS;
            if (n >= a.N || !ok) break;
            float s[VEC];
            widen<float, VEC>(raw[i], s);
            const float w = dt * bn[i][0];
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                s[v] = fmaf(decay, s[v], w * x[v]);
                y[v] = fmaf(cn[i][0], s[v], y[v]);
            }
            store_raw<float, VEC>(st + (size_t)n * a.P, narrow<float, VEC>(s));
        }
        if ((n0 += ROWS * kStepAhead) >= a.N) break;
        fetch(n0);
    }
#pragma unroll
    for (int o = 16; o >= LP; o >>= 1)
#pragma unroll
        for (int v = 0; v < VEC; ++v) y[v] += __shfl_xor_sync(0xffffffffu, y[v], o);
    if ((tid & 31) < LP) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) red[tid >> 5][lp * VEC + v] = y[v];
    }
    __syncthreads();
    if (tid < LP * VEC && part * LP * VEC + tid < a.P) {
        const int q = part * LP * VEC + tid;
        float s = 0.f, f[1];
#pragma unroll
        for (int w = 0; w < kStepThreads / 32; ++w) s += red[w][tid];
        widen<T, 1>(load_raw<T, 1>(xt + q), f);
        f[0] = fmaf(a.D ? a.D[h] : 0.f, f[0], s);
        store_raw<T, 1>(static_cast<T *>(a.y.p) + (size_t)b * a.y.sb + (size_t)h * a.y.sh + q, narrow<T, 1>(f));
    }
}

template <typename T, int VEC, int LP>
cudaError_t step(const Args &a, float *state, cudaStream_t st) {
    const int parts = (a.P + VEC * LP - 1) / (VEC * LP);
    ssm_step_kernel<T, VEC, LP><<<(unsigned)((size_t)a.B * a.H * parts), kStepThreads, 0, st>>>(a, state, parts);
    return cudaGetLastError();
}
template <typename T>
cudaError_t step_by_layout(const Args &a, float *state, cudaStream_t st) {
    if (a.P % 4 || (reinterpret_cast<uintptr_t>(state) & 15u)) return step<T, 1, 32>(a, state, st);
    if ((size_t)a.B * a.H < 304) return step<T, 4, 4>(a, state, st);
    return a.P <= 64 ? step<T, 4, 16>(a, state, st) : step<T, 4, 32>(a, state, st);
}

// ------------------------------------------------------------ host
hla_status check(const hla_ssm_params *p) {
    if (!p) return report(HLA_ERR_ARG, "params is NULL");
    if (p->B < 1 || p->H < 1 || p->G < 1 || p->H % p->G) return report(HLA_ERR_ARG, "need B >= 1 and H a multiple of G >= 1");
    if (p->n < 0 || p->P < 1 || p->N < 1) return report(HLA_ERR_ARG, "need n >= 0, P, N >= 1");
    if (p->in_dtype != HLA_F32 && p->in_dtype != HLA_BF16) return report(HLA_ERR_ARG, "unknown in_dtype");
    if (p->n > 2147483647 - 1024) return report(HLA_ERR_ARG, "problem too large");
    if ((double)p->B * p->H * (p->n / 32 + 64) > 2147483647.0) return report(HLA_ERR_ARG, "problem too large");
    if (p->P > 128 || p->N > 128) return report(HLA_ERR_UNSUPPORTED, "widths are supported up to 128");
    return HLA_OK;
}
bool aligned(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
// The parameters that a call reads; workspace sizes do without them.
hla_status check_rates(const hla_ssm_params *p) {
    if (!p->A) return report(HLA_ERR_ARG, "A must be set");
    if (!aligned(p->A) || !aligned(p->D) || !aligned(p->dt_bias))
        return report(HLA_ERR_ARG, "A, D or dt_bias is not aligned to its elements");
    if (p->dt_bias && !p->dt_softplus) return report(HLA_ERR_ARG, "dt_bias belongs to dt_softplus");
    return HLA_OK;
}

Args make(const hla_ssm_params *p) {
    Args a{};
    a.B = p->B; a.H = p->H; a.G = p->G; a.R = p->H / p->G;
    a.n = a.rows = p->n; a.P = p->P; a.N = p->N;
    a.softplus = p->dt_softplus != 0;
    a.A = p->A; a.D = p->D; a.dt_bias = p->dt_bias;
    a.lengths = p->lengths;
    return a;
}

struct Sizes {
    Dims x, dt, b;
    explicit Sizes(const hla_ssm_params *p, int n)
        : x{p->B, p->H, n, p->P}, dt{p->B, p->H, n, 1}, b{p->B, p->G, n, p->N} {}
};

hla_status take_workspace(Args &a, bool backward, void *ws, size_t bytes, size_t need) {
    if (!ws || bytes < need) return report(HLA_ERR_ARG, "workspace too small (hla_ssm_workspace_size)");
    if (reinterpret_cast<uintptr_t>(ws) & 255u) return report(HLA_ERR_ARG, "workspace must be 256-byte aligned");
    return HLA_OK;
}

cudaError_t copy_or_clear(float *to, const float *from, size_t bytes, cudaStream_t st) {
    return from ? cudaMemcpyAsync(to, from, bytes, cudaMemcpyDeviceToDevice, st) : cudaMemsetAsync(to, 0, bytes, st);
}
size_t state_bytes(const hla_ssm_params *p) { return (size_t)p->B * p->H * p->N * p->P * 4; }

}  // namespace
}  // namespace ssm
}  // namespace hla

using namespace hla;
using namespace hla::ssm;

extern "C" {

size_t hla_ssm_workspace_size(const hla_ssm_params *p, int backward) {
    if (ssm::check(p) != HLA_OK || p->n == 0) return 0;
    Args a = make(p), t = a;  // for either path: the alignment decides between them
    const size_t s = simt_space(a, backward != 0, nullptr);
    const size_t c = p->in_dtype == HLA_BF16 ? tc_space(t, backward != 0, nullptr) : 0;
    return s > c ? s : c;
}

hla_status hla_ssm_forward(const hla_ssm_params *p, const hla_tensor *x, const hla_tensor *dt, const hla_tensor *b,
                           const hla_tensor *c, const hla_tensor *y, const float *state_in, float *state_out,
                           void *workspace, size_t workspace_bytes, void *stream) {
    hla_status s = ssm::check(p);
    if (s != HLA_OK || (s = check_rates(p)) != HLA_OK) return s;
    if (!ssm::aligned(state_in) || !ssm::aligned(state_out)) return report(HLA_ERR_ARG, "a state is not aligned to its elements");
    if (state_in && state_in == state_out) return report(HLA_ERR_ARG, "state_out may not alias state_in");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (p->n == 0) {
        if (!state_out) return HLA_OK;
        const cudaError_t e = ssm::copy_or_clear(state_out, state_in, ssm::state_bytes(p), st);
        return e == cudaSuccess ? HLA_OK : report(HLA_ERR_CUDA, cudaGetErrorString(e));
    }
    const hla_dtype t = p->in_dtype;
    const Sizes d(p, p->n);
    if ((s = check_in(x, d.x, t, "x must be set")) != HLA_OK || (s = check_in(dt, d.dt, t, "dt must be set")) != HLA_OK ||
        (s = check_in(b, d.b, t, "b must be set")) != HLA_OK || (s = check_in(c, d.b, t, "c must be set")) != HLA_OK ||
        (s = check_out(y, d.x, t, "y must be set")) != HLA_OK)
        return s;
    if (y->p == x->p || y->p == dt->p || y->p == b->p || y->p == c->p) return report(HLA_ERR_ARG, "y may not be an input");
    Args a = make(p);
    if ((s = take_workspace(a, false, workspace, workspace_bytes, hla_ssm_workspace_size(p, 0))) != HLA_OK) return s;
    a.x = view(x, d.x); a.dt = view(dt, d.dt); a.b = view(b, d.b); a.c = view(c, d.b); a.y = view(y, d.x);
    a.state_in = state_in; a.state_out = state_out;
    cudaError_t e = cudaErrorNotSupported;
    if (t == HLA_BF16 && tc_takes(a, false)) {
        tc_space(a, false, static_cast<uint8_t *>(workspace));
        e = tc_forward(a, st);
    }
    if (e == cudaErrorNotSupported) {
        simt_space(a, false, static_cast<uint8_t *>(workspace));
        e = simt_forward(a, t, st);
    }
    return e == cudaSuccess ? HLA_OK : report(HLA_ERR_CUDA, cudaGetErrorString(e));
}

hla_status hla_ssm_backward(const hla_ssm_params *p, const hla_tensor *x, const hla_tensor *dt, const hla_tensor *b,
                            const hla_tensor *c, const hla_tensor *dy, const float *state_in, const float *d_state_out,
                            const hla_ssm_gradients *grads, void *workspace, size_t workspace_bytes, void *stream) {
    hla_status s = ssm::check(p);
    if (s != HLA_OK || (s = check_rates(p)) != HLA_OK) return s;
    if (!grads) return report(HLA_ERR_ARG, "grads must be set");
    const hla_ssm_gradients &g = *grads;
    if (!g.dA) return report(HLA_ERR_ARG, "dA must be set");
    if (g.dD && !p->D) return report(HLA_ERR_ARG, "dD belongs to D");
    if (g.d_dt_bias && !p->dt_bias) return report(HLA_ERR_ARG, "d_dt_bias belongs to dt_bias");
    for (const void *f : {(const void *)state_in, (const void *)d_state_out, (const void *)g.dA, (const void *)g.dD,
                          (const void *)g.d_dt_bias, (const void *)g.d_state_in})
        if (!ssm::aligned(f)) return report(HLA_ERR_ARG, "a state or a sum is not aligned to its elements");
    if (g.d_state_in && (g.d_state_in == d_state_out || g.d_state_in == state_in))
        return report(HLA_ERR_ARG, "d_state_in may not alias another state");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (p->n == 0) {
        cudaError_t e = cudaSuccess;
        for (float *f : {g.dA, g.dD, g.d_dt_bias})
            if (f && e == cudaSuccess) e = cudaMemsetAsync(f, 0, (size_t)p->H * 4, st);
        if (e == cudaSuccess && g.d_state_in) e = ssm::copy_or_clear(g.d_state_in, d_state_out, ssm::state_bytes(p), st);
        return e == cudaSuccess ? HLA_OK : report(HLA_ERR_CUDA, cudaGetErrorString(e));
    }
    const hla_dtype t = p->in_dtype;
    const Sizes d(p, p->n);
    if ((s = check_in(x, d.x, t, "x must be set")) != HLA_OK || (s = check_in(dt, d.dt, t, "dt must be set")) != HLA_OK ||
        (s = check_in(b, d.b, t, "b must be set")) != HLA_OK || (s = check_in(c, d.b, t, "c must be set")) != HLA_OK ||
        (s = check_in(dy, d.x, t, "dy must be set")) != HLA_OK || (s = check_out(&g.dx, d.x, t, "dx must be set")) != HLA_OK ||
        (s = check_out(&g.d_dt, d.dt, t, "d_dt must be set")) != HLA_OK ||
        (s = check_out(&g.db, d.b, t, "db must be set")) != HLA_OK || (s = check_out(&g.dc, d.b, t, "dc must be set")) != HLA_OK)
        return s;
    const hla_tensor *outs[4] = {&g.dx, &g.d_dt, &g.db, &g.dc}, *ins[5] = {x, dt, b, c, dy};
    for (int i = 0; i < 4; ++i) {
        for (const hla_tensor *in : ins)
            if (outs[i]->p == in->p) return report(HLA_ERR_ARG, "a gradient may not be an input");
        for (int j = 0; j < i; ++j)
            if (outs[i]->p == outs[j]->p) return report(HLA_ERR_ARG, "the gradients must differ");
    }
    Args a = make(p);
    if ((s = take_workspace(a, true, workspace, workspace_bytes, hla_ssm_workspace_size(p, 1))) != HLA_OK) return s;
    a.x = view(x, d.x); a.dt = view(dt, d.dt); a.b = view(b, d.b); a.c = view(c, d.b); a.dy = view(dy, d.x);
    a.dx = view(&g.dx, d.x); a.ddt = view(&g.d_dt, d.dt); a.db = view(&g.db, d.b); a.dc = view(&g.dc, d.b);
    a.state_in = state_in; a.d_state_out = d_state_out;
    a.d_state_in = g.d_state_in; a.dA = g.dA; a.dD = g.dD; a.dbias = g.d_dt_bias;
    cudaError_t e = cudaErrorNotSupported;
    if (t == HLA_BF16 && tc_takes(a, true)) {
        tc_space(a, true, static_cast<uint8_t *>(workspace));
        e = tc_backward(a, st);
    }
    if (e == cudaErrorNotSupported) {
        simt_space(a, true, static_cast<uint8_t *>(workspace));
        e = simt_backward(a, t, st);
    }
    return e == cudaSuccess ? HLA_OK : report(HLA_ERR_CUDA, cudaGetErrorString(e));
}

hla_status hla_ssm_step(const hla_ssm_params *p, const hla_tensor *x, const hla_tensor *dt, const hla_tensor *b,
                        const hla_tensor *c, const hla_tensor *y, float *state, void *stream) {
    hla_status s = ssm::check(p);
    if (s != HLA_OK || (s = check_rates(p)) != HLA_OK) return s;
    if (p->n != 1) return report(HLA_ERR_ARG, "a step takes one token: n must be 1");
    if (!state || !ssm::aligned(state)) return report(HLA_ERR_ARG, "state must be set and aligned to its elements");
    const hla_dtype t = p->in_dtype;
    const Sizes d(p, 1);
    if ((s = check_in(x, d.x, t, "x must be set")) != HLA_OK || (s = check_in(dt, d.dt, t, "dt must be set")) != HLA_OK ||
        (s = check_in(b, d.b, t, "b must be set")) != HLA_OK || (s = check_in(c, d.b, t, "c must be set")) != HLA_OK ||
        (s = check_out(y, d.x, t, "y must be set")) != HLA_OK)
        return s;
    for (const hla_tensor *i : {x, dt, b, c})
        if (y->p == i->p || i->p == state) return report(HLA_ERR_ARG, "y and state may not be inputs");
    if (y->p == state) return report(HLA_ERR_ARG, "y may not be the state");
    Args a = make(p);
    a.x = view(x, d.x); a.dt = view(dt, d.dt); a.b = view(b, d.b); a.c = view(c, d.b); a.y = view(y, d.x);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = t == HLA_F32 ? step_by_layout<float>(a, state, st) : step_by_layout<__nv_bfloat16>(a, state, st);
    return e == cudaSuccess ? HLA_OK : report(HLA_ERR_CUDA, cudaGetErrorString(e));
}

}  // extern "C"
