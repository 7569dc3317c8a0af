// hla_norm.cuh -- norm over groups of adjacent channels of each token, with an activation or an
// activated gate:
//   u = x (or x silu(gate)),  z = (u - mean) r (or u r),  v = z w + bias,  y = v | silu(v) | v silu(gate).
// Backward, with dv the gradient of v, g = dv w, and means over the group:
//   du = r (g - z mean(g z) - mean(g))   (without the last term where the mean is not taken),
//   dw = sum over tokens of dv z,  dbias = sum of dv.
// Memory bounds both: a team of threads holds a group of one token in registers, E channels each,
// so every element is read once and written once; statistics are two-pass over the registers, in
// fp32.  A CTA keeps its channels from token to token (the sums for dw and dbias stay in
// registers); while it reduces, the SM's other CTAs load.  Groups wider than a team holds go through
// a kernel that reads them again for each pass.
// Measured, bf16: forward n16384 d4096 in 64 groups, gate behind, 77 us, 5.2 TB/s; backward b2 n8192
// d4096 in one group, gate in front, no mean, 171 us, 3.9 TB/s: issue slots (59 % busy) and two sums over
// 512 threads a token, one after the other (three with a mean), bound it.  The next token's rows come by way of shared memory and the gate's sigmoid
// waits there for the end: 64 registers a thread hold neither (loaded when due and formed twice: 79 and 191).
#pragma once
#include "hla_layer.cuh"

namespace hla {
namespace norm {

using namespace layer;

enum Gate { GATE_NONE = 0, GATE_AFTER = 1, GATE_BEFORE = 2 };

struct Args {
    int B, n, d, groups, m;  // m = d / groups
    int col_blocks, row_blocks;
    int gate;
    bool center, silu;
    float eps;
    const float *weight, *bias;
    const int *lengths;
    View x, z, y, dy, dx, dz;
    float *part;  // [row_blocks][2][d]
};

// Most channels of a group that a team holds: E = 16 of 512 threads.
constexpr int kHeld = 8192;

// Rows that the CTA's row block takes: every row_blocks-th of all rows that are below their lengths.
// (Counted on by additions: a division for each row is a tenth of a narrow group's work.)
struct Rows {
    const Args &a;
    int b, t;
    HLA_DEVICE Rows(const Args &a_, int first) : a(a_), b(first / a_.n), t(first % a_.n) { settle(); }
    HLA_DEVICE bool live() const { return b < a.B; }
    HLA_DEVICE void next() {
        t += a.row_blocks;
        settle();
    }
    HLA_DEVICE void settle() {
        while (b < a.B) {
            if (t >= a.n) {
                t -= a.n;
                ++b;
            } else if (!a.lengths || t < a.lengths[b]) {
                return;
            } else {
                t += a.row_blocks;
            }
        }
    }
};

template <typename T>
HLA_DEVICE const T *row_in(const View &v, int b, int t) {
    return static_cast<const T *>(v.p) + (size_t)b * v.sb + (size_t)t * v.st;
}
template <typename T>
HLA_DEVICE T *row_to(const View &v, int b, int t) {
    return static_cast<T *>(v.p) + (size_t)b * v.sb + (size_t)t * v.st;
}

// VEC adjacent scales or shifts (16-byte aligned where VEC is a multiple of 4).
template <int VEC>
HLA_DEVICE void scale_of(const float *p, size_t at, bool ok, float none, float (&v)[VEC]) {
    if (!p || !ok) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = none;
    } else if constexpr (VEC % 4 == 0) {
#pragma unroll
        for (int i = 0; i < VEC; i += 4) {
            const float4 f = __ldg(reinterpret_cast<const float4 *>(p + at + i));
            v[i] = f.x; v[i + 1] = f.y; v[i + 2] = f.z; v[i + 3] = f.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = __ldg(p + at + i);
    }
}

// The next token's rows, on their way to shared memory while this one's are worked on: each thread
// copies what it will read itself, so no barrier is needed.  Where a thread's vectors are 16 bytes and
// the block's N rows of K vectors a thread fit.
template <typename T, int VEC, int K, int BLOCK, int N>
struct Ahead {
    static constexpr bool ON = VEC * sizeof(T) == 16 && N * K * BLOCK * 16 <= 24 * 1024;
    uint4 *slot;
    HLA_DEVICE uint4 *at(int row, int k) const { return slot + (row * K + k) * BLOCK + threadIdx.x; }
    HLA_DEVICE void ask(int row, int k, const T *p) const {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(at(row, k))), "l"(p) : "memory");
    }
    HLA_DEVICE void wait() const { asm volatile("cp.async.wait_all;" ::: "memory"); }
    HLA_DEVICE raw_t<T, VEC> take(int row, int k) const {
        if constexpr (ON) return *at(row, k);
        return {};
    }
};
template <typename T, int VEC, int K, int BLOCK, int N>
constexpr int ahead_slots() { return Ahead<T, VEC, K, BLOCK, N>::ON ? N * K * BLOCK : 1; }

// VEC values of a thread that it will need again, in shared memory: [K][VEC / 4][BLOCK] float4, or
// [K][BLOCK] single ones.
template <int VEC, int BLOCK>
HLA_DEVICE void lay_aside(float *keep, int k, const float (&v)[VEC]) {
    if constexpr (VEC % 4 == 0) {
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i)
            reinterpret_cast<float4 *>(keep)[(k * (VEC / 4) + i) * BLOCK + threadIdx.x] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    } else {
        static_assert(VEC == 1, "");
        keep[k * BLOCK + threadIdx.x] = v[0];
    }
}
template <int VEC, int BLOCK>
HLA_DEVICE void take_back(const float *keep, int k, float (&v)[VEC]) {
    if constexpr (VEC % 4 == 0) {
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i) {
            const float4 f = reinterpret_cast<const float4 *>(keep)[(k * (VEC / 4) + i) * BLOCK + threadIdx.x];
            v[4 * i] = f.x; v[4 * i + 1] = f.y; v[4 * i + 2] = f.z; v[4 * i + 3] = f.w;
        }
    } else {
        v[0] = keep[k * BLOCK + threadIdx.x];
    }
}

HLA_DEVICE float plus(float a, float b) { return a + b; }
HLA_DEVICE float2 plus(float2 a, float2 b) { return add2(a, b); }
HLA_DEVICE float across(float v, int o) { return __shfl_xor_sync(0xffffffffu, v, o); }
HLA_DEVICE float2 across(float2 v, int o) { return make_float2(across(v.x, o), across(v.y, o)); }
// Sum of a value, or of two, over a team of TEAM threads; `red` (on a 16-byte boundary) holds one
// float2 for each warp of the block, alternated by the caller so that one barrier per sum is enough.
template <int TEAM, class V>
HLA_DEVICE V team_sum(V v, float2 *red) {
    constexpr int LANES = TEAM < 32 ? TEAM : 32;
#pragma unroll
    for (int o = LANES >> 1; o > 0; o >>= 1) v = plus(v, across(v, o));
    if constexpr (TEAM > 32) {
        constexpr int WARPS = TEAM / 32, WIDE = WARPS * (int)sizeof(V) / 16;
        const int warp = threadIdx.x >> 5;
        V *all = reinterpret_cast<V *>(red);
        if ((threadIdx.x & 31) == 0) all[warp] = v;
        __syncthreads();
        const V *mine = all + warp / WARPS * WARPS;
        alignas(16) V w[WARPS];
        if constexpr (WIDE > 0) {
#pragma unroll
            for (int i = 0; i < WIDE; ++i) reinterpret_cast<float4 *>(w)[i] = reinterpret_cast<const float4 *>(mine)[i];
        } else {
#pragma unroll
            for (int i = 0; i < WARPS; ++i) w[i] = mine[i];
        }
        v = w[0];
#pragma unroll
        for (int i = 1; i < WARPS; ++i) v = plus(v, w[i]);
    }
    return v;
}

// `wide`: rows on 16-byte boundaries and groups of whole 16-byte pieces.
void forward_f32(const Args &a, bool wide, cudaStream_t st);
void forward_bf16(const Args &a, bool wide, cudaStream_t st);
void backward_f32(const Args &a, bool wide, cudaStream_t st);
void backward_bf16(const Args &a, bool wide, cudaStream_t st);

// The team of a group of m <= kHeld channels: eight channels a thread, sixteen for the widest.
struct Team {
    int threads, E;
};
inline Team team_of(int m) {
    for (int t = 8; t <= 512; t *= 2)
        if (m <= 8 * t) return {t, 8};
    if (m <= kHeld) return {512, 16};
    return {256, 0};  // read again for each pass, one CTA per group
}
// Threads per SM that the kernels are built for.
constexpr int kSms = 152, kForwardThreads = 1280, kBackwardThreads = 1024;
constexpr int block_of(int team) { return team > 256 ? team : 256; }
// CTAs side by side over the channels of a token, and over the tokens: about as many as the
// device runs at once (the sums for dw and dbias are kept per CTA).
inline int columns_of(int groups, int m) {
    const Team t = team_of(m);
    if (!t.E) return groups;
    const int per = block_of(t.threads) / t.threads;
    return (groups + per - 1) / per;
}
inline int row_blocks_of(long long rows, int groups, int m, int threads_per_sm) {
    const long long most = (long long)kSms * (threads_per_sm / block_of(team_of(m).threads)) / columns_of(groups, m);
    return (int)(most < 1 ? 1 : most < rows ? most : rows);
}

// Launch<T, VEC, E, TEAM, GATE>::go of a call's sizes.
template <template <typename, int, int, int, int> class Launch, typename T, int VEC, int E, int TEAM>
void by_gate(const Args &a, cudaStream_t st) {
    if (a.gate == GATE_NONE) return Launch<T, VEC, E, TEAM, GATE_NONE>::go(a, st);
    if (a.gate == GATE_AFTER) return Launch<T, VEC, E, TEAM, GATE_AFTER>::go(a, st);
    Launch<T, VEC, E, TEAM, GATE_BEFORE>::go(a, st);
}
template <template <typename, int, int, int, int> class Launch, typename T, int VEC>
void by_team(const Args &a, Team t, cudaStream_t st) {
    if (t.E == 16) return by_gate<Launch, T, VEC, 16, 512>(a, st);
    if (t.threads == 8) return by_gate<Launch, T, VEC, 8, 8>(a, st);
    if (t.threads == 16) return by_gate<Launch, T, VEC, 8, 16>(a, st);
    if (t.threads == 32) return by_gate<Launch, T, VEC, 8, 32>(a, st);
    if (t.threads == 64) return by_gate<Launch, T, VEC, 8, 64>(a, st);
    if (t.threads == 128) return by_gate<Launch, T, VEC, 8, 128>(a, st);
    if (t.threads == 256) return by_gate<Launch, T, VEC, 8, 256>(a, st);
    by_gate<Launch, T, VEC, 8, 512>(a, st);
}

}  // namespace norm
}  // namespace hla
