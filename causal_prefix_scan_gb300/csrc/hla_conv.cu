// hla_conv.cu -- short causal convolution per channel of [B][n][d], its gradient and its
// single-token step.  With xs = (state of width - 1 inputs, tokens):
//   pre_t = bias + sum_i w_i xs_{t+i},   y_t = act(pre_t),
//   g_t = dy_t act'(pre_t),   dxs_u = sum_i w_i g_{u-i} (+ d_state_out, rows u >= length),
//   dw_i = sum_t g_t xs_{t+i},   dbias = sum_t g_t.
// A few operations on each element, so memory bounds it: each element is read once and each result
// written once.  A warp takes 32 pairs of adjacent channels (single ones where the rows do not allow
// it) down a run of tokens with the last inputs and the filter in registers; runs read width - 1
// rows of their neighbours again (they hit the caches), and the backward computes g of width - 1
// tokens behind its run again.
#include <type_traits>

#include "hla_layer.cuh"

namespace hla {
namespace conv {
namespace {

using namespace layer;

constexpr int kWarps = 8, kThreads = 32 * kWarps, kSms = 152;

struct Args {
    int B, n, d, run, tiles, groups;  // tokens of a warp, tiles of tokens, groups of channels
    bool silu;
    const float *weight, *bias;
    const int *lengths;
    View x, y, dy, dx;
    const void *sin, *dsout;
    void *sout, *dsin;
    float *part;  // [B * tiles][width + 1][d]
};

template <typename T>
HLA_DEVICE const T *row_of(const View &v, int b, long long t, int c) {
    return static_cast<const T *>(v.p) + (size_t)b * v.sb + (size_t)t * v.st + c;
}
template <typename T>
HLA_DEVICE T *row_out(const View &v, int b, long long t, int c) {
    return static_cast<T *>(v.p) + (size_t)b * v.sb + (size_t)t * v.st + c;
}

// xs_u of one sequence (u counts from the state's first row); zeros where there is no state.
template <typename T, int VEC, int W>
HLA_DEVICE raw_t<T, VEC> input_at(const Args &a, int b, int u, int c) {
    if (u >= W - 1) return load_raw<T, VEC>(row_of<T>(a.x, b, u - (W - 1), c));
    if (!a.sin) return raw_t<T, VEC>{};
    return load_raw<T, VEC>(static_cast<const T *>(a.sin) + ((size_t)b * (W - 1) + u) * a.d + c);
}

template <int VEC, int W>
struct Filter {
    float w[W][VEC], bias[VEC];
    HLA_DEVICE Filter(const Args &a, int c) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
#pragma unroll
            for (int i = 0; i < W; ++i) w[i][v] = __ldg(a.weight + (size_t)(c + v) * W + i);
            bias[v] = a.bias ? __ldg(a.bias + c + v) : 0.f;
        }
    }
    // pre of the token whose inputs are xs[0 .. W - 1]
    HLA_DEVICE void apply(const float (*xs)[VEC], float (&pre)[VEC]) const {
        fma_v<VEC>(w[0], xs[0], bias, pre);
#pragma unroll
        for (int i = 1; i < W; ++i) fma_v<VEC>(w[i], xs[i], pre, pre);
    }
};

// Some lanes ask for the rows behind those in flight, one for each 128 bytes of a warp's row: its
// first channel.
template <typename T, int VEC>
constexpr int lines_of() { return VEC * (int)sizeof(T) > 4 ? VEC * (int)sizeof(T) / 4 : 1; }
template <typename T, int VEC>
HLA_DEVICE int line_of(const Args &a, int group, int lane) {
    constexpr int LINES = lines_of<T, VEC>();
    return min(group * 32 * VEC + lane % LINES * (32 * VEC / LINES), a.d - 1);
}

// Runs of tokens in groups of U, the next group's loads ahead of the present one's work and the rows
// behind those on their way to L2 (n32768 d4352 w4 bf16, silu: 100 us, 5.7 TB/s; without the rows
// ahead and with runs of 32 tokens 114; fp32 b2 n8192 d4352 88 us, 6.5 TB/s).
template <typename T, int VEC, int W, bool SILU>
__global__ void __launch_bounds__(kThreads, 4) conv_forward_kernel(const Args a) {
    constexpr int U = 8;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = ((int)(blockIdx.x % a.groups) * 32 + lane) * VEC;
    const int rest = blockIdx.x / a.groups, tile = rest % a.tiles, b = rest / a.tiles;
    if (c >= a.d) return;
    const int len = clamp_length(a.lengths, b, a.n);
    if (a.sout && tile == 0 && warp < W - 1)  // the last W - 1 inputs
        store_raw<T, VEC>(static_cast<T *>(a.sout) + ((size_t)b * (W - 1) + warp) * a.d + c,
                          input_at<T, VEC, W>(a, b, len + warp, c));
    const int t0 = (tile * kWarps + warp) * a.run, count = min(a.run, len - t0);
    if (count <= 0) return;
    const Filter<VEC, W> f(a, c);
    float xs[W - 1 + U][VEC];
#pragma unroll
    for (int i = 0; i < W - 1; ++i) widen<T, VEC>(input_at<T, VEC, W>(a, b, t0 + i, c), xs[i]);
    const T *in = row_of<T>(a.x, b, t0, c);
    T *out = row_out<T>(a.y, b, t0, c);
    constexpr int LINES = lines_of<T, VEC>();
    const int ahead = lane / LINES, line = line_of<T, VEC>(a, blockIdx.x % a.groups, lane);
    raw_t<T, VEC> raw[U];
    auto fetch = [&](int u) {
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (u + i < count) raw[i] = load_raw<T, VEC>(in + (size_t)i * a.x.st);
        in += (size_t)U * a.x.st;
    };
    fetch(0);
#pragma unroll 1
    for (int u = 0; u < count; u += U) {
#pragma unroll
        for (int i = 0; i < U; ++i) widen<T, VEC>(raw[i], xs[W - 1 + i]);
        if (u + U < count) fetch(u + U);
        if (ahead < U && u + 2 * U + ahead < count) prefetch_l2(row_of<T>(a.x, b, t0 + u + 2 * U + ahead, line));
#pragma unroll
        for (int i = 0; i < U; ++i) {
            float y[VEC];
            f.apply(xs + i, y);
            if (SILU) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) y[v] = silu(y[v]);
            }
            if (u + i < count) store_raw<T, VEC>(out + (size_t)i * a.y.st, narrow<T, VEC>(y));
        }
        out += (size_t)U * a.y.st;
#pragma unroll
        for (int i = 0; i < W - 1; ++i)
#pragma unroll
            for (int v = 0; v < VEC; ++v) xs[i][v] = xs[U + i][v];
    }
}

// One warp's run of tokens: their g counts towards the filter's gradient, and g of the
// W - 1 tokens behind them is formed again, so that dxs_u leaves once g_u is known.  Groups of U
// tokens, inputs ahead; the groups inside a run go without the questions that its ends ask.  Issue and
// the latency that 16 warps leave bound it: b2 n8192 d4352 w4 bf16, silu 116 us, 3.7 TB/s (fp32 147 us,
// 5.8 TB/s).  With 24 warps, groups of 4 and no rows ahead it took 139; rows ahead at 24 warps spill, 170.
template <typename T, int VEC, int W, bool SILU>
__global__ void __launch_bounds__(kThreads, 2) conv_backward_kernel(const Args a) {
    constexpr int U = 8;
    __shared__ float red[kWarps][(W + 1) * 32 * VEC];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = blockIdx.x % a.groups, c = (group * 32 + lane) * VEC;
    const int rest = blockIdx.x / a.groups, tile = rest % a.tiles, b = rest / a.tiles;
    const int len = clamp_length(a.lengths, b, a.n);
    const int t0 = (tile * kWarps + warp) * a.run;
    float dw[W + 1][VEC];  // taps, then bias
#pragma unroll
    for (int i = 0; i <= W; ++i) fill_v<VEC>(0.f, dw[i]);
    if (c < a.d && (t0 < len || t0 == 0)) {
        const Filter<VEC, W> f(a, c);
        float xs[W - 1 + U][VEC], g[W - 1 + U][VEC];  // xs_u .. ; g_{u-W+1} ..
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
            fill_v<VEC>(0.f, xs[i]);
            fill_v<VEC>(0.f, g[i]);
            if (t0 + i < len + W - 1) widen<T, VEC>(input_at<T, VEC, W>(a, b, t0 + i, c), xs[i]);
        }
        const int behind = min(t0 + a.run, len), last = behind + W - 1;  // dxs_u for u < last
        const int loads = min(last, len);
        constexpr int LINES = lines_of<T, VEC>();
        const int ahead = lane / LINES, line = line_of<T, VEC>(a, group, lane);
        raw_t<T, VEC> rx[U], rd[U];
        const T *xp = row_of<T>(a.x, b, t0, c), *dp = row_of<T>(a.dy, b, t0, c);
        auto fetch = [&](int t) {
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (t + i < loads) {
                    rx[i] = load_raw<T, VEC>(xp + (size_t)i * a.x.st);
                    rd[i] = load_raw<T, VEC>(dp + (size_t)i * a.dy.st);
                }
            xp += (size_t)U * a.x.st;
            dp += (size_t)U * a.dy.st;
        };
        fetch(t0);
        T *out = static_cast<T *>(a.dx.p) + (ptrdiff_t)b * (ptrdiff_t)a.dx.sb + (ptrdiff_t)(t0 - (W - 1)) * (ptrdiff_t)a.dx.st + c;  // row s of u = t0
        // A group of tokens; `inner`: all of them count, and all their dxs are rows of dx.
        auto tokens = [&](int t, auto inner) {
            constexpr bool INNER = decltype(inner)::value;
#pragma unroll
            for (int i = 0; i < U; ++i) {
                widen<T, VEC>(rx[i], xs[W - 1 + i]);
                widen<T, VEC>(rd[i], g[W - 1 + i]);
            }
            if (t + U < last) fetch(t + U);
            if (ahead < 2 * U) {
                const int row = t + 3 * U + ahead / 2;
                if (row < loads) prefetch_l2(ahead % 2 ? row_of<T>(a.dy, b, row, line) : row_of<T>(a.x, b, row, line));
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                float(&gt)[VEC] = g[W - 1 + i];
                if (SILU) {
                    float pre[VEC], s[VEC], r[VEC];
                    f.apply(xs + i, pre);
#pragma unroll
                    for (int v = 0; v < VEC; ++v) s[v] = sigmoid(pre[v]);
                    silu_slope_v<VEC>(pre, s, r);
                    mul_v<VEC>(gt, r, gt);
                }
                if (!INNER && t + i >= len) fill_v<VEC>(0.f, gt);  // (whatever was in the registers)
                if (INNER || t + i < behind) {
#pragma unroll
                    for (int k = 0; k < W; ++k) fma_v<VEC>(gt, xs[i + k], dw[k], dw[k]);
                    add_v<VEC>(dw[W], gt, dw[W]);
                }
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int u = t + i, s = u - (W - 1);  // dxs_u: row s of dx, or of the state's gradient
                if (!INNER && (u >= last || (s < t0 && t0 > 0))) continue;
                float o[VEC];
                mul_v<VEC>(f.w[0], g[W - 1 + i], o);
#pragma unroll
                for (int k = 1; k < W; ++k) fma_v<VEC>(f.w[k], g[W - 1 + i - k], o, o);
                if (!INNER && u >= len && a.dsout) {
                    float e[VEC];
                    widen<T, VEC>(load_raw<T, VEC>(static_cast<const T *>(a.dsout) + ((size_t)b * (W - 1) + (u - len)) * a.d + c), e);
                    add_v<VEC>(o, e, o);
                }
                if (INNER || s >= 0)
                    store_raw<T, VEC>(out + (ptrdiff_t)i * (ptrdiff_t)a.dx.st, narrow<T, VEC>(o));
                else if (a.dsin)
                    store_raw<T, VEC>(static_cast<T *>(a.dsin) + ((size_t)b * (W - 1) + u) * a.d + c, narrow<T, VEC>(o));
            }
            out += (ptrdiff_t)U * (ptrdiff_t)a.dx.st;
#pragma unroll
            for (int i = 0; i < W - 1; ++i)
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    xs[i][v] = xs[U + i][v];
                    g[i][v] = g[U + i][v];
                }
        };
#pragma unroll 1
        for (int t = t0; t < last; t += U) {
            if (t > t0 && t + U <= behind)
                tokens(t, std::true_type());
            else
                tokens(t, std::false_type());
        }
    }
#pragma unroll
    for (int i = 0; i <= W; ++i)
#pragma unroll
        for (int v = 0; v < VEC; ++v) red[warp][(i * VEC + v) * 32 + lane] = dw[i][v];
    __syncthreads();
    for (int e = threadIdx.x; e < (W + 1) * 32 * VEC; e += kThreads) {
        const int i = e / (32 * VEC), ch = (group * 32 + e % 32) * VEC + e / 32 % VEC;
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s += red[w][e];
        if (ch < a.d) a.part[((size_t)(b * a.tiles + tile) * (W + 1) + i) * a.d + ch] = s;
    }
}

__global__ void __launch_bounds__(256) conv_filter_kernel(const float *part, int rows, int d, int W, float *dw, float *db) {
    column_sums(part, rows, (long long)d * (W + 1), [=](long long k, float s) {
        const int i = (int)(k / d), c = (int)(k % d);
        if (i < W)
            dw[(size_t)c * W + i] = s;
        else if (db)
            db[c] = s;
    });
}

template <typename T, int VEC, int W>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(const Args a) {
    const int cols = (a.d + VEC - 1) / VEC;
    const size_t e = (size_t)blockIdx.x * kThreads + threadIdx.x;
    if (e >= (size_t)cols * a.B) return;
    const int b = (int)(e / cols), c = (int)(e % cols) * VEC;
    if (a.lengths && a.lengths[b] <= 0) return;
    T *state = static_cast<T *>(a.sout) + (size_t)b * (W - 1) * a.d + c;
    raw_t<T, VEC> in[W];
#pragma unroll
    for (int i = 0; i < W - 1; ++i) in[i] = load_raw<T, VEC>(state + (size_t)i * a.d);
    in[W - 1] = load_raw<T, VEC>(row_of<T>(a.x, b, 0, c));
    const Filter<VEC, W> f(a, c);
    float y[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) y[v] = f.bias[v];
#pragma unroll
    for (int i = 0; i < W; ++i) {
        float x[VEC];
        widen<T, VEC>(in[i], x);
#pragma unroll
        for (int v = 0; v < VEC; ++v) y[v] = fmaf(f.w[i][v], x[v], y[v]);
        if (i > 0) store_raw<T, VEC>(state + (size_t)(i - 1) * a.d, in[i]);
    }
    if (a.silu) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) y[v] = silu(y[v]);
    }
    store_raw<T, VEC>(row_out<T>(a.y, b, 0, c), narrow<T, VEC>(y));
}

// ------------------------------------------------------------ host
enum Which { W_FWD, W_BWD, W_STEP };

int tiles_of(int n, int run) { return (int)(((long long)n + kWarps * run - 1) / (kWarps * run)); }
// Tokens of a warp: long runs read less of their neighbours and begin less often, where they leave
// some rounds of CTAs over the SMs (forward n32768 d4352 bf16 111 -> 100 us at 64, but b2 n8192 fp32 88 ->
// 92; backward b2 n8192 125 -> 119 at 128).
int run_of(int B, int n, int d, bool back) {
    const int run = back ? 128 : 64;
    const double ctas = (double)B * tiles_of(n, run) * ((d + 63) / 64);
    return ctas >= kSms * (back ? 2 * 3 : 4 * 6) ? run : run / 2;
}

template <typename T, int VEC, int W>
cudaError_t launch(Which w, Args a, float *dw, float *db, cudaStream_t st) {
    a.groups = (a.d + 32 * VEC - 1) / (32 * VEC);
    // Prompts go two channels at a time: with what four of them hold in registers too few warps fit an
    // SM (forward bf16 n32768 d4352 153 -> 115 us, fp32 b2 n8192 d4352 107 -> 87, its backward 219 -> 182).
    // Steps hold one token and go by 16 bytes.
    constexpr bool STEPS_ALONE = VEC > 2;
    if (w == W_STEP) {
        const size_t work = (size_t)a.B * ((a.d + VEC - 1) / VEC);
        conv_step_kernel<T, VEC, W><<<(unsigned)((work + kThreads - 1) / kThreads), kThreads, 0, st>>>(a);
    } else if constexpr (STEPS_ALONE) {
        return cudaErrorInvalidValue;
    } else if (w == W_FWD) {
        a.run = run_of(a.B, a.n, a.d, false);
        a.tiles = tiles_of(a.n, a.run);
        const unsigned grid = (unsigned)((size_t)a.B * a.tiles * a.groups);
        if (a.silu)
            conv_forward_kernel<T, VEC, W, true><<<grid, kThreads, 0, st>>>(a);
        else
            conv_forward_kernel<T, VEC, W, false><<<grid, kThreads, 0, st>>>(a);
    } else {
        a.run = run_of(a.B, a.n, a.d, true);
        a.tiles = tiles_of(a.n, a.run);
        const unsigned grid = (unsigned)((size_t)a.B * a.tiles * a.groups);
        if (a.silu)
            conv_backward_kernel<T, VEC, W, true><<<grid, kThreads, 0, st>>>(a);
        else
            conv_backward_kernel<T, VEC, W, false><<<grid, kThreads, 0, st>>>(a);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        const long long cols = (long long)a.d * (W + 1);
        conv_filter_kernel<<<(unsigned)((cols + 31) / 32), 256, 0, st>>>(a.part, a.B * a.tiles, a.d, W, dw, db);
    }
    return cudaGetLastError();
}
template <typename T, int VEC>
cudaError_t by_width(int width, Which w, const Args &a, float *dw, float *db, cudaStream_t st) {
    if (width == 2) return launch<T, VEC, 2>(w, a, dw, db, st);
    if (width == 3) return launch<T, VEC, 3>(w, a, dw, db, st);
    return launch<T, VEC, 4>(w, a, dw, db, st);
}

hla_status check(const hla_conv_params *p) {
    if (!p) return report(HLA_ERR_ARG, "params is NULL");
    if (p->B < 1 || p->d < 1 || p->n < 0) return report(HLA_ERR_ARG, "need B >= 1, d >= 1, n >= 0");
    if (p->in_dtype != HLA_F32 && p->in_dtype != HLA_BF16) return report(HLA_ERR_ARG, "unknown in_dtype");
    if (p->activation != HLA_ACT_NONE && p->activation != HLA_ACT_SILU) return report(HLA_ERR_ARG, "unknown activation");
    if (p->width < 1) return report(HLA_ERR_ARG, "need width >= 1");
    if (p->n > 2147483647 - 1024) return report(HLA_ERR_ARG, "problem too large");  // token counters pass n by a tile
    const double rows = (double)p->B * (tiles_of(p->n, 32) + 1);
    if (rows * ((p->d + 31) / 32) > 2147483647.0 || (double)p->d * 5 > 2147483647.0)
        return report(HLA_ERR_ARG, "problem too large");
    if (p->width < 2 || p->width > 4) return report(HLA_ERR_UNSUPPORTED, "widths of 2 to 4 taps are supported");
    return HLA_OK;
}
// The parameters that a call reads; workspace sizes do without them.
hla_status check_filter(const hla_conv_params *p) {
    if (!p->weight) return report(HLA_ERR_ARG, "weight must be set");
    if ((reinterpret_cast<uintptr_t>(p->weight) & 3u) || (reinterpret_cast<uintptr_t>(p->bias) & 3u))
        return report(HLA_ERR_ARG, "weight or bias is not aligned to its elements");
    return HLA_OK;
}

Args make(const hla_conv_params *p) {
    Args a{};
    a.B = p->B; a.n = p->n; a.d = p->d;
    a.silu = p->activation == HLA_ACT_SILU;
    a.weight = p->weight; a.bias = p->bias;
    a.lengths = p->lengths;
    return a;
}

// Channels that `vec` elements at a time divide, every row on their boundary.
bool takes(const hla_conv_params *p, std::initializer_list<const View *> rows, std::initializer_list<const void *> states,
           int vec) {
    const int bytes = vec * (p->in_dtype == HLA_F32 ? 4 : 2);
    if (p->d % vec) return false;
    for (const View *v : rows)
        if (reinterpret_cast<uintptr_t>(v->p) % bytes || v->sb % vec || v->st % vec) return false;
    for (const void *s : states)
        if (reinterpret_cast<uintptr_t>(s) % bytes) return false;
    return true;
}

hla_status run(const hla_conv_params *p, Which w, const Args &a, std::initializer_list<const View *> rows,
               std::initializer_list<const void *> states, float *dw, float *db, cudaStream_t st) {
    const bool step = w == W_STEP;
    auto go = [&](auto by, int vec) { return takes(p, rows, states, vec) ? by(p->width, w, a, dw, db, st) : cudaErrorNotSupported; };
    cudaError_t e = cudaErrorNotSupported;
    if (p->in_dtype == HLA_F32) {
        if (step) e = go(by_width<float, 4>, 4);
        if (e == cudaErrorNotSupported) e = go(by_width<float, 2>, 2);
        if (e == cudaErrorNotSupported) e = go(by_width<float, 1>, 1);
    } else {
        if (step) e = go(by_width<__nv_bfloat16, 8>, 8);
        if (step && e == cudaErrorNotSupported) e = go(by_width<__nv_bfloat16, 4>, 4);
        if (e == cudaErrorNotSupported) e = go(by_width<__nv_bfloat16, 2>, 2);
        if (e == cudaErrorNotSupported) e = go(by_width<__nv_bfloat16, 1>, 1);
    }
    return e == cudaSuccess ? HLA_OK : report(HLA_ERR_CUDA, cudaGetErrorString(e));
}

bool aligned(const void *p, hla_dtype dt) { return reinterpret_cast<uintptr_t>(p) % (dt == HLA_F32 ? 4 : 2) == 0; }

size_t state_bytes(const hla_conv_params *p) { return (size_t)p->B * (p->width - 1) * p->d * (p->in_dtype == HLA_F32 ? 4 : 2); }

cudaError_t copy_or_clear(void *to, const void *from, size_t bytes, cudaStream_t st) {
    return from ? cudaMemcpyAsync(to, from, bytes, cudaMemcpyDeviceToDevice, st) : cudaMemsetAsync(to, 0, bytes, st);
}

}  // namespace
}  // namespace conv
}  // namespace hla

using namespace hla;
using namespace hla::conv;

extern "C" {

hla_status hla_conv_forward(const hla_conv_params *p, const hla_tensor *x, const hla_tensor *y, const void *state_in,
                            void *state_out, void *stream) {
    hla_status s = conv::check(p);
    if (s != HLA_OK || (s = check_filter(p)) != HLA_OK) return s;
    const hla_dtype dt = p->in_dtype;
    if (!aligned(state_in, dt) || !aligned(state_out, dt)) return report(HLA_ERR_ARG, "a state is not aligned to its elements");
    if (state_in && state_in == state_out) return report(HLA_ERR_ARG, "state_out may not alias state_in");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (p->n == 0) {
        if (!state_out) return HLA_OK;
        const cudaError_t e = copy_or_clear(state_out, state_in, state_bytes(p), st);
        return e == cudaSuccess ? HLA_OK : report(HLA_ERR_CUDA, cudaGetErrorString(e));
    }
    const Dims d{p->B, 1, p->n, p->d};
    if ((s = check_in(x, d, dt, "x must be set")) != HLA_OK || (s = check_out(y, d, dt, "y must be set")) != HLA_OK) return s;
    if (y->p == x->p) return report(HLA_ERR_ARG, "y may not be x");
    Args a = make(p);
    a.x = view(x, d); a.y = view(y, d);
    a.sin = state_in; a.sout = state_out;
    return run(p, W_FWD, a, {&a.x, &a.y}, {state_in, state_out}, nullptr, nullptr, st);
}

size_t hla_conv_backward_workspace_size(const hla_conv_params *p) {
    if (conv::check(p) != HLA_OK || p->n == 0) return 0;
    return layer::align256((size_t)p->B * tiles_of(p->n, run_of(p->B, p->n, p->d, true)) * (p->width + 1) * p->d * 4);
}

hla_status hla_conv_backward(const hla_conv_params *p, const hla_tensor *x, const hla_tensor *dy, const hla_tensor *dx,
                             const void *state_in, const void *d_state_out, float *d_weight, float *d_bias,
                             void *d_state_in, void *workspace, size_t workspace_bytes, void *stream) {
    hla_status s = conv::check(p);
    if (s != HLA_OK || (s = check_filter(p)) != HLA_OK) return s;
    const hla_dtype dt = p->in_dtype;
    if (!aligned(state_in, dt) || !aligned(d_state_out, dt) || !aligned(d_state_in, dt))
        return report(HLA_ERR_ARG, "a state is not aligned to its elements");
    if (!d_weight || !aligned(d_weight, HLA_F32) || !aligned(d_bias, HLA_F32))
        return report(HLA_ERR_ARG, "d_weight must be set, it and d_bias aligned to their elements");
    if (d_state_in && (d_state_in == d_state_out || d_state_in == state_in))
        return report(HLA_ERR_ARG, "d_state_in may not alias another state");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (p->n == 0) {
        cudaError_t e = cudaMemsetAsync(d_weight, 0, (size_t)p->d * p->width * 4, st);
        if (e == cudaSuccess && d_bias) e = cudaMemsetAsync(d_bias, 0, (size_t)p->d * 4, st);
        if (e == cudaSuccess && d_state_in) e = copy_or_clear(d_state_in, d_state_out, state_bytes(p), st);
        return e == cudaSuccess ? HLA_OK : report(HLA_ERR_CUDA, cudaGetErrorString(e));
    }
    const Dims d{p->B, 1, p->n, p->d};
    if ((s = check_in(x, d, dt, "x must be set")) != HLA_OK || (s = check_in(dy, d, dt, "dy must be set")) != HLA_OK ||
        (s = check_out(dx, d, dt, "dx must be set")) != HLA_OK)
        return s;
    if (dx->p == x->p || dx->p == dy->p) return report(HLA_ERR_ARG, "dx may not be an input");
    if (!workspace || workspace_bytes < hla_conv_backward_workspace_size(p))
        return report(HLA_ERR_ARG, "workspace too small (hla_conv_backward_workspace_size)");
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return report(HLA_ERR_ARG, "workspace must be 256-byte aligned");
    Args a = make(p);
    a.x = view(x, d); a.dy = view(dy, d); a.dx = view(dx, d);
    a.sin = state_in; a.dsout = d_state_out; a.dsin = d_state_in;
    a.part = static_cast<float *>(workspace);
    return run(p, W_BWD, a, {&a.x, &a.dy, &a.dx}, {state_in, d_state_out, d_state_in}, d_weight, d_bias, st);
}

hla_status hla_conv_step(const hla_conv_params *p, const hla_tensor *x, const hla_tensor *y, void *state, void *stream) {
    hla_status s = conv::check(p);
    if (s != HLA_OK || (s = check_filter(p)) != HLA_OK) return s;
    if (p->n != 1) return report(HLA_ERR_ARG, "a step takes one token: n must be 1");
    const hla_dtype dt = p->in_dtype;
    if (!state || !aligned(state, dt)) return report(HLA_ERR_ARG, "state must be set and aligned to its elements");
    const Dims d{p->B, 1, 1, p->d};
    if ((s = check_in(x, d, dt, "x must be set")) != HLA_OK || (s = check_out(y, d, dt, "y must be set")) != HLA_OK) return s;
    if (y->p == x->p || y->p == state || x->p == state) return report(HLA_ERR_ARG, "x, y and state must differ");
    Args a = make(p);
    a.x = view(x, d); a.y = view(y, d);
    a.sout = state;
    return run(p, W_STEP, a, {&a.x, &a.y}, {state}, nullptr, nullptr, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
