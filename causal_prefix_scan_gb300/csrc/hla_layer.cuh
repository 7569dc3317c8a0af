// hla_layer.cuh -- device helpers of the selective state space layer's kernels: typed vector
// access, the activation, lengths, and sums of partial results in a fixed order.
#pragma once
#include "hla_strided.h"

namespace hla {
namespace layer {

// sigma(z) from one exponential and one reciprocal: (16 + 2 |z|) 2^-24 of it off at most, the second part by
// the exponential's argument, which is rounded twice.  The exponential overflows to infinity below -88, where
// sigma is 0 to the last bit that counts.
HLA_DEVICE float sigmoid(float z) { return rcp_approx(1.f + ex2_approx(z * -1.4426950408889634f)); }
HLA_DEVICE float silu(float z) { return z * sigmoid(z); }
HLA_DEVICE float silu_slope(float z, float s) { return s * fmaf(z, 1.f - s, 1.f); }  // s = sigma(z)

HLA_DEVICE int clamp_length(const int *lengths, int b, int n) {
    if (!lengths) return n;
    const int L = lengths[b];
    return L < 0 ? 0 : L > n ? n : L;
}

HLA_DEVICE void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// VEC adjacent elements as raw bits: 2 to 16 bytes.
template <int BYTES>
struct RawOf;
template <>
struct RawOf<2> { using type = unsigned short; };
template <>
struct RawOf<4> { using type = unsigned; };
template <>
struct RawOf<8> { using type = uint2; };
template <>
struct RawOf<16> { using type = uint4; };
template <typename T, int VEC>
using raw_t = typename RawOf<VEC * (int)sizeof(T)>::type;

template <typename T, int VEC>
HLA_DEVICE raw_t<T, VEC> load_raw(const T *p) { return *reinterpret_cast<const raw_t<T, VEC> *>(p); }
template <typename T, int VEC>
HLA_DEVICE void widen(const raw_t<T, VEC> &r, float (&v)[VEC]) {
    if constexpr (sizeof(T) == 4) {
        const float *f = reinterpret_cast<const float *>(&r);
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = f[i];
    } else {
        const unsigned short *f = reinterpret_cast<const unsigned short *>(&r);
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = __uint_as_float((unsigned)f[i] << 16);
    }
}
template <typename T, int VEC>
HLA_DEVICE raw_t<T, VEC> narrow(const float (&v)[VEC]) {
    raw_t<T, VEC> r;
    if constexpr (sizeof(T) == 4) {
        float *f = reinterpret_cast<float *>(&r);
#pragma unroll
        for (int i = 0; i < VEC; ++i) f[i] = v[i];
    } else if constexpr (VEC == 1) {
        r = __bfloat16_as_ushort(__float2bfloat16_rn(v[0]));
    } else {
        unsigned *f = reinterpret_cast<unsigned *>(&r);
#pragma unroll
        for (int i = 0; i < VEC; i += 2) f[i / 2] = pack_bf16(v[i], v[i + 1]);
    }
    return r;
}
template <typename T, int VEC>
HLA_DEVICE void store_raw(T *p, const raw_t<T, VEC> &r) { *reinterpret_cast<raw_t<T, VEC> *>(p) = r; }

// Pairs of fp32: one instruction for two lanes' worth of arithmetic.
HLA_DEVICE float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mul.rn.f32x2 z, x, y;\n mov.b64 {%0, %1}, z;\n}\n"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
HLA_DEVICE float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n add.rn.f32x2 z, x, y;\n mov.b64 {%0, %1}, z;\n}\n"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
HLA_DEVICE float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n .reg .b64 x, y, z, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 w, {%6, %7};\n"
        " fma.rn.f32x2 z, x, y, w;\n mov.b64 {%0, %1}, z;\n}\n"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
HLA_DEVICE float2 both(float x) { return make_float2(x, x); }
// The same on VEC channels: a b + c, a b, a + b, elementwise.
template <int VEC>
HLA_DEVICE void fma_v(const float (&a)[VEC], const float (&b)[VEC], const float (&c)[VEC], float (&r)[VEC]) {
    if constexpr (VEC % 2 == 0) {
#pragma unroll
        for (int i = 0; i < VEC; i += 2) {
            const float2 x = fma2(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]), make_float2(c[i], c[i + 1]));
            r[i] = x.x;
            r[i + 1] = x.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) r[i] = fmaf(a[i], b[i], c[i]);
    }
}
template <int VEC>
HLA_DEVICE void mul_v(const float (&a)[VEC], const float (&b)[VEC], float (&r)[VEC]) {
    if constexpr (VEC % 2 == 0) {
#pragma unroll
        for (int i = 0; i < VEC; i += 2) {
            const float2 x = mul2(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]));
            r[i] = x.x;
            r[i + 1] = x.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) r[i] = a[i] * b[i];
    }
}
template <int VEC>
HLA_DEVICE void add_v(const float (&a)[VEC], const float (&b)[VEC], float (&r)[VEC]) {
    if constexpr (VEC % 2 == 0) {
#pragma unroll
        for (int i = 0; i < VEC; i += 2) {
            const float2 x = add2(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]));
            r[i] = x.x;
            r[i + 1] = x.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) r[i] = a[i] + b[i];
    }
}
template <int VEC>
HLA_DEVICE void fill_v(float x, float (&r)[VEC]) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) r[i] = x;
}
template <int VEC>
HLA_DEVICE void silu_slope_v(const float (&z)[VEC], const float (&s)[VEC], float (&r)[VEC]) {  // s = sigma(z)
    float m[VEC], one[VEC];
    fill_v<VEC>(1.f, one);
    fill_v<VEC>(-1.f, m);
    fma_v<VEC>(s, m, one, r);
    fma_v<VEC>(z, r, one, r);
    mul_v<VEC>(r, s, r);
}

// out[k] = sum over r of part[r][k], k < cols: 8 warps take rows w, w + 8, ..., then the warps are
// added, so the order depends on the sizes alone.
template <class Store>
HLA_DEVICE void column_sums(const float *part, int rows, long long cols, Store store) {
    __shared__ float red[8][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long c = (long long)blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < cols) {
        const float *p = part + c;
        int r = warp;
        for (; r + 24 < rows; r += 32) {
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = __ldg(p + (size_t)(r + 8 * i) * cols);
            s += (v[0] + v[1]) + (v[2] + v[3]);
        }
        for (; r < rows; r += 8) s += __ldg(p + (size_t)r * cols);
    }
    red[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < cols) {
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) t += red[w][lane];
        store(c, t);
    }
}

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace layer
}  // namespace hla
