// hla_window.cu -- C entry points of windowed attention with first tokens that stay
// visible: argument checks, the choice of kernels, the ring cache's fill.
#include <cmath>

#include "hla_window_simt.cuh"

namespace hla {
namespace win {
namespace {

int far_keys(const hla_window_params *p, int tile) {
    const int s = p->sinks < p->nk ? p->sinks : p->nk;
    const long long up = ((long long)s + tile - 1) / tile * tile;
    return (int)(up < p->nk ? up : p->nk);
}

// Far shares of a key tile with first tokens (see dkv_kernel): its queries beyond the
// window are divided so that a share is about as long as a tile's own window (one share for
// all of them: B2 H16 n8192 w1024 backward 857 us against 509, B3 H6 n1501 w301 66 against 45).
// Each share is an fp32 copy of these tiles' dk and dv in the workspace, so there are no more than
// give the far queries kFarCtas CTAs: many tiles fill the device with few shares (B8 H8 n8192 d128
// w512 with 1,024 first tokens: 338 MB and 1,557 us, without the limit 1,009 MB and 1,994 us).
constexpr int kFarMost = 32, kFarCtas = 2048;
int far_shares(const hla_window_params *p, int tile) {
    if (p->sinks == 0 || p->n == 0) return 0;
    const long long far = (long long)p->nk - p->window;  // queries beyond the window of the first keys
    if (far <= 0) return 0;
    const long long win = p->window + tile;
    const long long s = (far + win - 1) / win;
    const long long tiles = (long long)p->B * p->Hkv * ((far_keys(p, tile) + tile - 1LL) / tile);
    const long long fill = kFarCtas / tiles > 1 ? kFarCtas / tiles : 1, most = fill < kFarMost ? fill : kFarMost;
    return (int)(s > most ? most : s);
}

hla_status check(const hla_window_params *p, bool step) {
    if (!p) return report(HLA_ERR_ARG, "params is NULL");
    if (p->B < 1 || p->H < 1 || p->Hkv < 1 || p->H % p->Hkv != 0)
        return report(HLA_ERR_ARG, "need B >= 1 and H a multiple of Hkv >= 1");
    if (p->d < 1 || p->dv < 1) return report(HLA_ERR_ARG, "need d, dv >= 1");
    if (p->in_dtype != HLA_F32 && p->in_dtype != HLA_BF16) return report(HLA_ERR_ARG, "unknown in_dtype");
    if (p->window < 1 || p->sinks < 0) return report(HLA_ERR_ARG, "need window >= 1, sinks >= 0");
    if (!std::isfinite(p->scale)) return report(HLA_ERR_ARG, "scale must be finite");
    if (step) {
        if (p->n != 1) return report(HLA_ERR_ARG, "a step takes one token: n must be 1");
        if ((long long)p->sinks + p->window > 2147483647LL - 4096)  // the kernels' slot counters have 32 bits
            return report(HLA_ERR_ARG, "too many slots");
        if ((double)p->B * p->H > 2147483647.0 / 16) return report(HLA_ERR_ARG, "problem too large");
    } else {
        if (p->n < 0 || p->nk < p->n) return report(HLA_ERR_ARG, "need 0 <= n <= nk");
        if (p->nk > 2147483647 - 1024) return report(HLA_ERR_ARG, "problem too large");
        const double rows = (double)p->B * p->H * ((p->nk + 63) / 64 + 1);
        if (rows > 2147483647.0) return report(HLA_ERR_ARG, "problem too large");
    }
    if (p->d > 128 || p->dv > 128) return report(HLA_ERR_UNSUPPORTED, "widths are supported up to 128");
    return HLA_OK;
}

Args make(const hla_window_params *p) {
    Args a{};
    a.B = p->B; a.H = p->H; a.Hkv = p->Hkv; a.G = p->H / p->Hkv;
    a.n = p->n; a.nk = p->nk; a.p0 = p->nk - p->n;
    a.d = p->d; a.dv = p->dv; a.window = p->window;
    a.sinks = p->sinks < p->nk ? p->sinks : p->nk;  // more than there are tokens means the same
    a.scale = p->scale;
    a.lengths = p->lengths;
    return a;
}

template <typename K>
cudaError_t smem_limit(K fn, size_t bytes) {
    return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <typename T, int DP>
cudaError_t simt_fwd(const Args &a, cudaStream_t st) {
    constexpr size_t bytes = (size_t)(3 * 64 * (DP + 4) + 64 * LP) * 4;
    cudaError_t e = smem_limit(fwd_kernel<T, DP>, bytes);
    if (e != cudaSuccess) return e;
    fwd_kernel<T, DP><<<(unsigned)((size_t)a.B * a.H * ((a.n + TQ - 1) / TQ)), kThreads, bytes, st>>>(a);
    return cudaGetLastError();
}
template <typename T, int DP>
cudaError_t simt_bwd(const Args &a, cudaStream_t st) {
    constexpr size_t dq_bytes = (size_t)(4 * 64 * (DP + 4) + 64 * LP + 128) * 4;
    constexpr size_t dkv_bytes = (size_t)(4 * 64 * (DP + 4) + 2 * 64 * LP + 128) * 4;
    cudaError_t e = smem_limit(dq_kernel<T, DP>, dq_bytes);
    if (e == cudaSuccess) e = smem_limit(dkv_kernel<T, DP>, dkv_bytes);
    if (e != cudaSuccess) return e;
    const size_t rows = (size_t)a.B * a.H * a.n;
    delta_kernel<T><<<(unsigned)((rows + kThreads / 32 - 1) / (kThreads / 32)), kThreads, 0, st>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    dq_kernel<T, DP><<<(unsigned)((size_t)a.B * a.H * ((a.n + TQ - 1) / TQ)), kThreads, dq_bytes, st>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    dkv_kernel<T, DP><<<dim3((unsigned)((size_t)a.B * a.Hkv * ((a.nk + TK - 1) / TK)), a.far + 1), kThreads, dkv_bytes, st>>>(a);
    return cudaGetLastError();
}
// Adds the shares of the key tiles with first tokens.
template <typename T>
cudaError_t join_shares(const Args &a, cudaStream_t st) {
    const size_t el = (size_t)a.B * a.Hkv * a.far_keys * (a.d + a.dv);
    join_kernel<T><<<(unsigned)((el + kThreads - 1) / kThreads), kThreads, 0, st>>>(a);
    return cudaGetLastError();
}
template <typename T>
cudaError_t simt(const Args &a, bool backward, cudaStream_t st) {
    const int w = a.d > a.dv ? a.d : a.dv;
    if (w <= 32) return backward ? simt_bwd<T, 32>(a, st) : simt_fwd<T, 32>(a, st);
    if (w <= 64) return backward ? simt_bwd<T, 64>(a, st) : simt_fwd<T, 64>(a, st);
    return backward ? simt_bwd<T, 128>(a, st) : simt_fwd<T, 128>(a, st);
}

// Copies the tokens that a prompt leaves in the ring, one warp per slot; `blocks` CTAs
// share the slots of one (sequence, key/value head).
template <typename E>
__global__ void __launch_bounds__(128) fill_kernel(const Args a, View kc, View vc, int blocks) {
    const int u = blockIdx.x / blocks, hk = u % a.Hkv, b = u / a.Hkv, len = length_of(a, b);
    const int cap = a.sinks + a.window, used = min(cap, len);
    for (unsigned s = blockIdx.x % blocks * 4 + (threadIdx.x >> 5); s < (unsigned)used; s += blocks * 4) {
        int j = (int)s;  // the last token below len that lies in slot s
        if (j >= a.sinks && len > cap) {
            const int r = j - a.sinks, last = len - 1 - a.sinks;  // (j - sinks) % window == r, j < len
            j = a.sinks + last - (last - r) % a.window;
        }
        const E *k = static_cast<const E *>(a.k.p) + (size_t)b * a.k.sb + (size_t)hk * a.k.sh + (size_t)j * a.k.st;
        const E *v = static_cast<const E *>(a.v.p) + (size_t)b * a.v.sb + (size_t)hk * a.v.sh + (size_t)j * a.v.st;
        E *ko = static_cast<E *>(kc.p) + (size_t)b * kc.sb + (size_t)hk * kc.sh + (size_t)s * kc.st;
        E *vo = static_cast<E *>(vc.p) + (size_t)b * vc.sb + (size_t)hk * vc.sh + (size_t)s * vc.st;
        for (int c = threadIdx.x & 31; c < a.d; c += 32) ko[c] = k[c];
        for (int c = threadIdx.x & 31; c < a.dv; c += 32) vo[c] = v[c];
    }
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
size_t delta_bytes(const hla_window_params *p) { return align256((size_t)p->B * p->H * p->n * 4); }
size_t part_bytes(const hla_window_params *p, int tile) {
    const size_t far = far_shares(p, tile);
    return far ? (far + 1) * p->B * p->Hkv * (size_t)far_keys(p, tile) * (p->d + p->dv) * 4 : 0;
}
size_t backward_bytes(const hla_window_params *p) {  // for either path: the alignment decides between them
    const size_t s = part_bytes(p, TK), t = p->in_dtype == HLA_BF16 ? part_bytes(p, kTcTile) : 0;
    return delta_bytes(p) + (s > t ? s : t);
}
bool wide_rows(const View &v) {
    return (reinterpret_cast<uintptr_t>(v.p) & 15u) == 0 && v.sb % 8 == 0 && v.sh % 8 == 0 && v.st % 8 == 0;
}

}  // namespace
}  // namespace win
}  // namespace hla

using namespace hla;
using namespace hla::win;

extern "C" {

hla_status hla_window_forward(const hla_window_params *p, const hla_tensor *q, const hla_tensor *k, const hla_tensor *v,
                              const hla_tensor *o, float *lse, void *stream) {
    hla_status s = win::check(p, false);
    if (s != HLA_OK) return s;
    if (p->n == 0) return HLA_OK;
    const hla_dtype dt = p->in_dtype;
    const Dims dq{p->B, p->H, p->n, p->d}, dk{p->B, p->Hkv, p->nk, p->d}, dv{p->B, p->Hkv, p->nk, p->dv},
        od{p->B, p->H, p->n, p->dv};
    if ((s = check_in(q, dq, dt, "q must be set")) != HLA_OK || (s = check_in(k, dk, dt, "k must be set")) != HLA_OK ||
        (s = check_in(v, dv, dt, "v must be set")) != HLA_OK || (s = check_out(o, od, dt, "o must be set")) != HLA_OK)
        return s;
    if (o->p == q->p || o->p == k->p || o->p == v->p) return report(HLA_ERR_ARG, "o may not be an input");
    if (reinterpret_cast<uintptr_t>(lse) & 3u) return report(HLA_ERR_ARG, "lse is not aligned to its elements");
    Args a = make(p);
    a.q = view(q, dq); a.k = view(k, dk); a.v = view(v, dv); a.o = view(o, od);
    a.lse = lse;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = dev_status_ptr(&a.err);
    if (e != cudaSuccess) return report(HLA_ERR_CUDA, cudaGetErrorString(e));
    e = dt == HLA_BF16 && fwd_tc_takes(a) ? fwd_tc(a, st) : cudaErrorNotSupported;
    if (e == cudaErrorNotSupported) e = dt == HLA_F32 ? simt<float>(a, false, st) : simt<__nv_bfloat16>(a, false, st);
    return e == cudaSuccess ? HLA_OK : report(HLA_ERR_CUDA, cudaGetErrorString(e));
}

size_t hla_window_backward_workspace_size(const hla_window_params *p) {
    if (win::check(p, false) != HLA_OK || p->n == 0) return 0;
    return backward_bytes(p);
}

hla_status hla_window_backward(const hla_window_params *p, const hla_tensor *q, const hla_tensor *k, const hla_tensor *v,
                               const hla_tensor *o, const float *lse, const hla_tensor *dout, const hla_tensor *dq,
                               const hla_tensor *dk, const hla_tensor *dv, void *workspace, size_t workspace_bytes,
                               void *stream) {
    hla_status s = win::check(p, false);
    if (s != HLA_OK) return s;
    const hla_dtype dt = p->in_dtype;
    const Dims qd{p->B, p->H, p->n, p->d}, kd{p->B, p->Hkv, p->nk, p->d}, vd{p->B, p->Hkv, p->nk, p->dv},
        od{p->B, p->H, p->n, p->dv};
    if (p->n == 0) return p->nk == 0 ? HLA_OK : report(HLA_ERR_ARG, "backward needs n >= 1 when nk >= 1");
    if ((s = check_in(q, qd, dt, "q must be set")) != HLA_OK || (s = check_in(k, kd, dt, "k must be set")) != HLA_OK ||
        (s = check_in(v, vd, dt, "v must be set")) != HLA_OK || (s = check_in(o, od, dt, "o must be set")) != HLA_OK ||
        (s = check_in(dout, od, dt, "dout must be set")) != HLA_OK ||
        (s = check_out(dq, qd, dt, "dq must be set")) != HLA_OK ||
        (s = check_out(dk, kd, dt, "dk must be set")) != HLA_OK ||
        (s = check_out(dv, vd, dt, "dv must be set")) != HLA_OK)
        return s;
    if (!lse || (reinterpret_cast<uintptr_t>(lse) & 3u)) return report(HLA_ERR_ARG, "lse must be set and aligned");
    const hla_tensor *outs[3] = {dq, dk, dv}, *ins[5] = {q, k, v, o, dout};
    for (int i = 0; i < 3; ++i) {
        for (const hla_tensor *t : ins)
            if (outs[i]->p == t->p) return report(HLA_ERR_ARG, "dq, dk and dv may not be inputs");
        for (int j = 0; j < i; ++j)
            if (outs[i]->p == outs[j]->p) return report(HLA_ERR_ARG, "dq, dk and dv must differ");
    }
    const size_t need = backward_bytes(p);
    if (!workspace || workspace_bytes < need)
        return report(HLA_ERR_ARG, "workspace too small (hla_window_backward_workspace_size)");
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return report(HLA_ERR_ARG, "workspace must be 256-byte aligned");
    Args a = make(p);
    a.q = view(q, qd); a.k = view(k, kd); a.v = view(v, vd); a.o = view(o, od); a.go = view(dout, od);
    a.dq = view(dq, qd); a.dk = view(dk, kd); a.dv_ = view(dv, vd);
    a.lse = const_cast<float *>(lse);
    a.delta = static_cast<float *>(workspace);
    a.part = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + delta_bytes(p));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = dev_status_ptr(&a.err);
    if (e != cudaSuccess) return report(HLA_ERR_CUDA, cudaGetErrorString(e));
    e = cudaErrorNotSupported;
    if (dt == HLA_BF16 && bwd_tc_takes(a)) {
        a.far = far_shares(p, kTcTile);
        a.far_keys = a.far ? far_keys(p, kTcTile) : 0;
        e = bwd_tc(a, st);
    }
    if (e == cudaErrorNotSupported) {
        a.far = far_shares(p, TK);
        a.far_keys = a.far ? far_keys(p, TK) : 0;
        e = dt == HLA_F32 ? simt<float>(a, true, st) : simt<__nv_bfloat16>(a, true, st);
    }
    if (e == cudaSuccess && a.far > 0) e = dt == HLA_F32 ? join_shares<float>(a, st) : join_shares<__nv_bfloat16>(a, st);
    return e == cudaSuccess ? HLA_OK : report(HLA_ERR_CUDA, cudaGetErrorString(e));
}

hla_status hla_window_step(const hla_window_params *p, const hla_tensor *q, const hla_tensor *k, const hla_tensor *v,
                           const hla_tensor *kc, const hla_tensor *vc, const long long *pos, const hla_tensor *o,
                           void *stream) {
    hla_status s = win::check(p, true);
    if (s != HLA_OK) return s;
    const hla_dtype dt = p->in_dtype;
    const long long slots = (long long)p->sinks + p->window;
    const Dims qd{p->B, p->H, 1, p->d}, kd{p->B, p->Hkv, 1, p->d}, vd{p->B, p->Hkv, 1, p->dv}, od{p->B, p->H, 1, p->dv},
        kcd{p->B, p->Hkv, slots, p->d}, vcd{p->B, p->Hkv, slots, p->dv};
    if ((s = check_in(q, qd, dt, "q must be set")) != HLA_OK || (s = check_in(k, kd, dt, "k must be set")) != HLA_OK ||
        (s = check_in(v, vd, dt, "v must be set")) != HLA_OK ||
        (s = check_out(kc, kcd, dt, "kc must be set")) != HLA_OK ||
        (s = check_out(vc, vcd, dt, "vc must be set")) != HLA_OK ||
        (s = check_out(o, od, dt, "o must be set")) != HLA_OK)
        return s;
    if (!pos || (reinterpret_cast<uintptr_t>(pos) & 7u)) return report(HLA_ERR_ARG, "pos must be set and aligned");
    const hla_tensor *ins[3] = {q, k, v};
    for (const hla_tensor *t : ins)
        if (o->p == t->p || kc->p == t->p || vc->p == t->p) return report(HLA_ERR_ARG, "o, kc and vc may not be inputs");
    if (kc->p == vc->p || o->p == kc->p || o->p == vc->p) return report(HLA_ERR_ARG, "o, kc and vc must differ");
    StepArgs a{};
    a.B = p->B; a.H = p->H; a.Hkv = p->Hkv; a.G = p->H / p->Hkv;
    a.d = p->d; a.dv = p->dv; a.window = p->window; a.sinks = p->sinks;
    a.scale = p->scale;
    a.pos = pos;
    a.q = view(q, qd); a.k = view(k, kd); a.v = view(v, vd);
    a.kc = view(kc, kcd); a.vc = view(vc, vcd); a.o = view(o, od);
    a.wide = dt == HLA_BF16 && p->d % 8 == 0 && p->dv % 8 == 0 && wide_rows(a.k) && wide_rows(a.v) && wide_rows(a.kc) &&
             wide_rows(a.vc);
    const cudaError_t e = win::step(a, dt, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? HLA_OK : report(HLA_ERR_CUDA, cudaGetErrorString(e));
}

hla_status hla_window_cache_fill(const hla_window_params *p, const hla_tensor *k, const hla_tensor *v,
                                 const hla_tensor *kc, const hla_tensor *vc, void *stream) {
    if (!p) return report(HLA_ERR_ARG, "params is NULL");
    hla_window_params c = *p;
    c.n = 1;
    hla_status s = win::check(&c, true);
    if (s != HLA_OK) return s;
    c.n = 0;
    if ((s = win::check(&c, false)) != HLA_OK) return s;
    const hla_dtype dt = p->in_dtype;
    const long long slots = (long long)p->sinks + p->window;
    if (p->nk == 0) return HLA_OK;
    const Dims kd{p->B, p->Hkv, p->nk, p->d}, vd{p->B, p->Hkv, p->nk, p->dv}, kcd{p->B, p->Hkv, slots, p->d},
        vcd{p->B, p->Hkv, slots, p->dv};
    if ((s = check_in(k, kd, dt, "k must be set")) != HLA_OK || (s = check_in(v, vd, dt, "v must be set")) != HLA_OK ||
        (s = check_out(kc, kcd, dt, "kc must be set")) != HLA_OK ||
        (s = check_out(vc, vcd, dt, "vc must be set")) != HLA_OK)
        return s;
    if (kc->p == vc->p || kc->p == k->p || kc->p == v->p || vc->p == k->p || vc->p == v->p)
        return report(HLA_ERR_ARG, "kc and vc must differ from each other and from k and v");
    Args a = make(&c);
    a.k = view(k, kd); a.v = view(v, vd);
    const View ko = view(kc, kcd), vo = view(vc, vcd);
    const long long used = slots < p->nk ? slots : p->nk;  // later slots stay as they are
    const long long pairs = (long long)p->B * p->Hkv, most = 2147483647LL / pairs, quads = (used + 3) / 4;
    const int blocks = (int)(quads < 4096 ? (quads < most ? quads : most) : (4096 < most ? 4096 : most));
    const unsigned grid = (unsigned)(blocks * pairs);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dt == HLA_F32)
        fill_kernel<float><<<grid, 128, 0, st>>>(a, ko, vo, blocks);
    else
        fill_kernel<__nv_bfloat16><<<grid, 128, 0, st>>>(a, ko, vo, blocks);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? HLA_OK : report(HLA_ERR_CUDA, cudaGetErrorString(e));
}

}  // extern "C"
