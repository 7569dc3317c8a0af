// hla_norm.cu -- entry points of the grouped norm (see hla_norm.cuh).
#include <cmath>

#include "hla_norm.cuh"

namespace hla {
namespace norm {
namespace {

__global__ void __launch_bounds__(256) norm_sums_kernel(const float *part, int rows, int d, float *dw, float *db) {
    column_sums(part, rows, 2LL * d, [=](long long k, float s) {
        if (k < d) {
            if (dw) dw[k] = s;
        } else if (db) {
            db[k - d] = s;
        }
    });
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
constexpr int kMostRowBlocks = kSms * (kBackwardThreads / 256);

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
    Args a = make(p, gate != nullptr, kForwardThreads);
    a.x = view(x, d); a.y = view(y, d);
    if (gate) a.z = view(gate, d);
    const bool wide = wide_rows(p, a, {&a.x, &a.y, &a.z});
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    dt == HLA_F32 ? forward_f32(a, wide, st) : forward_bf16(a, wide, st);
    const cudaError_t e = cudaGetLastError();
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
    Args a = make(p, gate != nullptr, kBackwardThreads);
    a.x = view(x, d); a.dy = view(dy, d); a.dx = view(dx, d);
    if (gate) a.z = view(gate, d), a.dz = view(d_gate, d);
    a.part = static_cast<float *>(workspace);
    const bool wide = wide_rows(p, a, {&a.x, &a.dy, &a.dx, &a.z, &a.dz});
    dt == HLA_F32 ? backward_f32(a, wide, st) : backward_bf16(a, wide, st);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess && (d_weight || d_bias)) {
        norm_sums_kernel<<<(unsigned)((2LL * a.d + 31) / 32), 256, 0, st>>>(a.part, a.row_blocks, a.d, d_weight, d_bias);
        e = cudaGetLastError();
    }
    return e == cudaSuccess ? HLA_OK : report(HLA_ERR_CUDA, cudaGetErrorString(e));
}

}  // extern "C"
