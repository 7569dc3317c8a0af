// hla_gated.cuh -- what the kernels of the gated recurrence share: arguments, access to VEC
// adjacent channels of a token, the gates and their gradients.
#pragma once
#include "hla_internal.h"

namespace hla {
namespace gated {

// Published map or state of one channel of one tile, 16 bytes, read and written whole (see
// the look-back kernels).
struct __align__(16) Record {
    float a, b;
    unsigned long long tag;
};
// Header word 0 counts tickets over all calls, word 1 is the count at which this call
// began: both only grow, so no call number ever returns.
struct Header {
    unsigned long long tickets, base;
};

struct Tensor {
    const void *p;
    long long sb, st;
};

struct Args {
    int B, n, d, tiles, slices;
    const float *rate;
    const int *lengths;
    Tensor x, g, y, dy, o1, o2;   // o1: y or dx, o2: dg
    const float *state_in;        // [B][d]: before the first token (NULL: zeros)
    const float *d_state_out;     // [B][d]: gradient of the state after the last (NULL: zeros)
    float *out_state;             // state after the last token, or d_state_in (NULL: skip)
    Header *hdr;
    Record *rec, *part;           // part: NULL when the rates' gradient is not wanted
    unsigned *err;
};

// ------------------------------------------------------------ element access
// VEC adjacent channels of one token as they lie in memory.
template <typename T, int VEC>
struct Raw;
template <>
struct Raw<float, 1> { using type = float; };
template <>
struct Raw<float, 2> { using type = float2; };
template <>
struct Raw<__nv_bfloat16, 1> { using type = unsigned short; };
template <>
struct Raw<__nv_bfloat16, 2> { using type = unsigned; };
template <typename T, int VEC>
using raw_t = typename Raw<T, VEC>::type;

// (arrays of VEC floats: the members of Vf below)
__device__ __forceinline__ void unpack(float r, float (&v)[1]) { v[0] = r; }
__device__ __forceinline__ void unpack(float2 r, float (&v)[2]) { v[0] = r.x; v[1] = r.y; }
__device__ __forceinline__ void unpack(unsigned short r, float (&v)[1]) { v[0] = __uint_as_float((unsigned)r << 16); }
__device__ __forceinline__ void unpack(unsigned r, float (&v)[2]) {
    v[0] = __uint_as_float(r << 16);
    v[1] = __uint_as_float(r & 0xFFFF0000u);
}
__device__ __forceinline__ void pack(const float (&v)[1], float &r) { r = v[0]; }
__device__ __forceinline__ void pack(const float (&v)[2], float2 &r) { r = make_float2(v[0], v[1]); }
__device__ __forceinline__ void pack(const float (&v)[1], unsigned short &r) {
    r = __bfloat16_as_ushort(__float2bfloat16_rn(v[0]));
}
__device__ __forceinline__ void pack(const float (&v)[2], unsigned &r) { r = pack_bf16(v[0], v[1]); }

template <typename T, int VEC>
__device__ __forceinline__ raw_t<T, VEC> load(const Tensor &t, size_t off) {
    return __ldg(reinterpret_cast<const raw_t<T, VEC> *>(static_cast<const T *>(t.p) + off));
}
// Rows seen by a whole warp: the row's address is the warp's (uniform registers), only the
// channel differs from lane to lane.
template <typename T, int VEC>
struct Slice {
    char *p;
    long long st;
    uint32_t ch;  // bytes
    HLA_DEVICE Slice(const Tensor &t, int b, int c0, long long first, int lane)
        : p(static_cast<char *>(const_cast<void *>(t.p)) + ((long long)b * t.sb + c0 + first * t.st) * (long long)sizeof(T)),
          st(t.st * (long long)sizeof(T)), ch(lane * VEC * (uint32_t)sizeof(T)) {}
    HLA_DEVICE raw_t<T, VEC> load(int i) const { return __ldg(reinterpret_cast<const raw_t<T, VEC> *>(p + i * st + ch)); }
    HLA_DEVICE void store(int i, const float (&v)[VEC]) const {
        raw_t<T, VEC> r;
        pack(v, r);
        *reinterpret_cast<raw_t<T, VEC> *>(p + i * st + ch) = r;
    }
};
template <typename T, int VEC>
__device__ __forceinline__ void store(const Tensor &t, size_t off, const float (&v)[VEC]) {
    raw_t<T, VEC> r;
    pack(v, r);
    *reinterpret_cast<raw_t<T, VEC> *>(const_cast<T *>(static_cast<const T *>(t.p)) + off) = r;
}

// ------------------------------------------------------------ arithmetic on VEC channels
// PAIR: two fp32 numbers go through one instruction (fma.rn.f32x2 and the like, rounded as the
// scalar ones), fewer instructions to issue.  bf16 channels use it (32,768 x 4,096 forward 223
// -> 211 us, 2 x 8,192 x 4,096 backward 238 -> 228 us); fp32 ones, whose inputs take twice the
// registers, do not: pairs want aligned ones (4 x 2,048 x 4,096 forward 90 -> 82 us without).
template <int VEC, bool PAIR>
struct Vf {
    static constexpr int N = VEC;
    float v[VEC];
};
template <typename T, int VEC>
using Num = Vf<VEC, VEC == 2 && sizeof(T) == 2>;
using Pair = Vf<2, true>;

HLA_DEVICE unsigned long long pair(const Pair &x) {
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x.v[0]), "f"(x.v[1]));
    return r;
}
HLA_DEVICE Pair unpair(unsigned long long r) {
    Pair x;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x.v[0]), "=f"(x.v[1]) : "l"(r));
    return x;
}
template <class V, class F>
HLA_DEVICE V each(const V &a, F f) {
    V r;
#pragma unroll
    for (int i = 0; i < V::N; ++i) r.v[i] = f(a.v[i]);
    return r;
}
template <class V>
HLA_DEVICE V splat(float c) {
    return each(V{}, [c](float) { return c; });
}
template <int VEC>
HLA_DEVICE Vf<VEC, false> fma_(const Vf<VEC, false> &a, const Vf<VEC, false> &b, const Vf<VEC, false> &c) {
    Vf<VEC, false> r;
#pragma unroll
    for (int i = 0; i < VEC; ++i) r.v[i] = fmaf(a.v[i], b.v[i], c.v[i]);
    return r;
}
template <int VEC>
HLA_DEVICE Vf<VEC, false> mul_(const Vf<VEC, false> &a, const Vf<VEC, false> &b) {
    Vf<VEC, false> r;
#pragma unroll
    for (int i = 0; i < VEC; ++i) r.v[i] = a.v[i] * b.v[i];
    return r;
}
template <int VEC>
HLA_DEVICE Vf<VEC, false> add_(const Vf<VEC, false> &a, const Vf<VEC, false> &b) {
    Vf<VEC, false> r;
#pragma unroll
    for (int i = 0; i < VEC; ++i) r.v[i] = a.v[i] + b.v[i];
    return r;
}
HLA_DEVICE Pair fma_(const Pair &a, const Pair &b, const Pair &c) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(pair(a)), "l"(pair(b)), "l"(pair(c)));
    return unpair(r);
}
HLA_DEVICE Pair mul_(const Pair &a, const Pair &b) {
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pair(a)), "l"(pair(b)));
    return unpair(r);
}
HLA_DEVICE Pair add_(const Pair &a, const Pair &b) {
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pair(a)), "l"(pair(b)));
    return unpair(r);
}
template <class V>
HLA_DEVICE V sub_(const V &a, const V &b) {  // a - b
    return fma_(b, splat<V>(-1.f), a);
}
HLA_DEVICE float rsqrt_approx(float x) {
    float r;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
HLA_DEVICE float rcp_approx(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// ------------------------------------------------------------ gates
constexpr float kLog2e = 1.4426950408889634f;

// sigma(z) and 1 - sigma(z), both with a relative error of a few units in the last place:
// the smaller is e / (1 + e), e = exp(-|z|) <= 1, and the larger is one minus it, so that a
// gate near one, whose error a long product of gates multiplies, is off by its rounding only.
template <class V>
HLA_DEVICE void sigmoid2(const V &z, V &s, V &c) {
    const V e = each(z, [](float x) { return ex2_approx(fabsf(x) * -kLog2e); });
    const V r = each(add_(e, splat<V>(1.f)), rcp_approx);
    const V lo = mul_(e, r), hi = sub_(splat<V>(1.f), lo);
#pragma unroll
    for (int i = 0; i < V::N; ++i) {
        const bool up = z.v[i] > 0.f;
        s.v[i] = up ? hi.v[i] : lo.v[i];
        c.v[i] = up ? lo.v[i] : hi.v[i];
    }
}
// sigma(z) alone, a few units in the last place off: far below zero the exponential is
// infinite and the quotient zero.
template <class V>
HLA_DEVICE V sigmoid(const V &z) {
    const V e = each(mul_(z, splat<V>(-kLog2e)), ex2_approx);
    return each(add_(e, splat<V>(1.f)), rcp_approx);
}
// a = exp(-u) and w = 1 - a for u >= 0, both to a few units in the last place beside what u is
// off by.  Below 1/16 the difference would cancel: w by Taylor's series to u^5, whose next term is under
// 2^-29 of the sum there, and a = 1 - w, off by its rounding only (a long product of gates near one
// multiplies their errors).  Above, a is the exponential itself: 1 - w would leave a small a with an error of
// 2^-25, of which d_state_in, dg and the rates' gradient, all in proportion to a, are made.
constexpr float kNear = 0.0625f;
template <class V>
HLA_DEVICE void exp_gate(const V &u, V &a, V &w) {
    const V e = each(mul_(u, splat<V>(-kLog2e)), ex2_approx);
    const V far = sub_(splat<V>(1.f), e);
    V p = fma_(u, splat<V>(1.f / 120.f), splat<V>(-1.f / 24.f));
    p = fma_(p, u, splat<V>(1.f / 6.f));
    p = fma_(p, u, splat<V>(-0.5f));
    p = fma_(p, u, splat<V>(1.f));
    p = mul_(p, u);
    const V near = sub_(splat<V>(1.f), p);
#pragma unroll
    for (int i = 0; i < V::N; ++i) {
        const bool small = u.v[i] < kNear;
        w.v[i] = small ? p.v[i] : far.v[i];
        a.v[i] = small ? near.v[i] : e.v[i];
    }
}
// 1 / sqrt(q) for q >= 0, finite at 0
template <class V>
HLA_DEVICE V rsqrt0(const V &q) {
    return each(q, [](float x) { return rsqrt_approx(fmaxf(x, 1.2e-38f)); });
}

// a_t and b_t
template <int GATE, class V>
HLA_DEVICE void gate_fwd(const V &g, const V &r, const V &x, V &a, V &b) {
    if constexpr (GATE == HLA_GATE_GIVEN) {
        a = g;
        b = x;
    } else if constexpr (GATE == HLA_GATE_SIGMOID) {
        V c;
        sigmoid2(g, a, c);
        b = mul_(c, x);
    } else {
        V w;
        exp_gate(mul_(r, sigmoid(g)), a, w);
        const V q = fma_(w, a, w);  // 1 - a^2
        b = mul_(mul_(q, rsqrt0(q)), x);
    }
}
// A token's a, and what the backward pass keeps of its gate: a, or with HLA_GATE_RATE
// whichever of 1 - a (sign bit clear) and a (sign bit set) exp_gate formed first.  The other is one
// minus it, with exp_gate's bits, and the gradients need no second exponential.
template <int GATE, class V>
HLA_DEVICE V gate_keep(const V &g, const V &r, V &a) {
    V b;
    if constexpr (GATE == HLA_GATE_RATE) {
        const V u = mul_(r, sigmoid(g));
        exp_gate(u, a, b);
#pragma unroll
        for (int i = 0; i < V::N; ++i) b.v[i] = u.v[i] < kNear ? b.v[i] : -a.v[i];
        return b;
    } else {
        gate_fwd<GATE>(g, r, splat<V>(0.f), a, b);
        return a;
    }
}
// a and w = 1 - a of what gate_keep returned with HLA_GATE_RATE
template <class V>
HLA_DEVICE void kept_gate(V k, V &a, V &w) {
    V one;
#pragma unroll
    for (int i = 0; i < V::N; ++i) {
        // formed again, not held in registers since gate_keep formed it, as the compiler would
        // (2 x 8,192 x 4,096 backward: 200 bytes of a thread's registers spilled)
        asm("" : "+f"(k.v[i]));
        one.v[i] = __float_as_int(k.v[i]) < 0 ? 0.f : 1.f;  // by the sign bit: a may be zero
    }
    a = sub_(one, k);
    const V o = sub_(splat<V>(1.f), a);
#pragma unroll
    for (int i = 0; i < V::N; ++i) w.v[i] = __float_as_int(k.v[i]) < 0 ? o.v[i] : k.v[i];
}
template <int GATE>
constexpr float kKeptOff = GATE == HLA_GATE_RATE ? 0.f : 1.f;  // a token that is not there: a = 1

// Gradients with respect to x, g and (HLA_GATE_RATE) the rate, from gh = dL/dh_t, x_t,
// y = h_{t-1} and gate_keep's k.  With f = sqrt(1 - a^2), a = exp(-u): df/du = a^2 / f, da/du = -a.
// f = 0 (sigma(g) underflowed) has the limit 0 for every product with du/dg, du/dr.
template <int GATE, class V>
HLA_DEVICE void gate_bwd(const V &g, const V &r, const V &x, const V &y, const V &gh,
                         const V &k, V &dx, V &dg, V &dr, V &a) {
    if constexpr (GATE == HLA_GATE_GIVEN) {
        dx = gh;
        a = k;
        dg = mul_(gh, y);
    } else if constexpr (GATE == HLA_GATE_SIGMOID) {
        V s, c;
        sigmoid2(g, s, c);
        dx = mul_(gh, c);
        a = k;
        dg = mul_(mul_(dx, s), sub_(y, x));
    } else {
        V s, c;
        sigmoid2(g, s, c);
        V w;
        kept_gate(k, a, w);
        const V q = fma_(w, a, w);
        const V rf = rsqrt0(q);
        dx = mul_(gh, mul_(q, rf));
        const V du = mul_(mul_(gh, a), sub_(mul_(mul_(x, a), rf), y));
        dr = mul_(du, s);
        dg = mul_(mul_(dr, r), c);
    }
}

template <int GATE, class V>
HLA_DEVICE V rate_of(const Args &a, int ch) {
    V r = splat<V>(0.f);
    if constexpr (GATE == HLA_GATE_RATE) {
#pragma unroll
        for (int v = 0; v < V::N; ++v)
            if (ch + v < a.d) r.v[v] = a.rate[ch + v];
    }
    return r;
}
HLA_DEVICE int length_of(const Args &a, int b) {
    if (!a.lengths) return a.n;
    const int L = a.lengths[b];
    return L < 0 ? 0 : L > a.n ? a.n : L;
}

// Streaming kernels (hla_gated_stream.cu), for channels in pairs: taken when the sequences'
// channels alone give (nearly) every SM a CTA.  The backward leaves the sequences' sums of the rates'
// gradient in a.part [B][d] and adds them into d_rate (NULL: neither).
bool stream_takes(const Args &a, hla_dtype t, bool backward, int sms);
cudaError_t stream_forward(const Args &a, hla_dtype t, int gate, cudaStream_t st);
cudaError_t stream_backward(const Args &a, hla_dtype t, int gate, float *d_rate, cudaStream_t st);

}  // namespace gated
}  // namespace hla
