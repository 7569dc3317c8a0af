// hla_window_tc.cuh -- what the tensor-core kernels of windowed attention share: tensor
// maps over strided [B][H][n][width] bf16 tensors, MMA groups on 128-row tiles, bounded
// barrier waits with an abort flag.
#pragma once
#include <cstring>

#include "hla_tmap.h"
#include "hla_window.h"

namespace hla {
namespace win {
namespace tcw {

constexpr int T = 128;  // rows of a tile (queries or keys)

// Rows that a tensor map can describe: 16-byte aligned, strides in multiples of 16 bytes
// (0 for a broadcast head or sequence), tokens apart.
inline bool mappable(const View &v) {
    return (reinterpret_cast<uintptr_t>(v.p) & 15u) == 0 && v.sb % 8 == 0 && v.sh % 8 == 0 && v.st % 8 == 0 &&
           v.st > 0 && v.sb < (1LL << 38) && v.sh < (1LL << 38) && v.st < (1LL << 38);
}

// Boxes of 64 columns x `rows` rows; rows past n and columns past `width` read as zeros.
// A broadcast dimension (stride 0) is given extent 1; its coordinate is then always 0.
inline bool encode(CUtensorMap *tm, const View &v, int width, int n, int H, int B, int rows) {
    auto enc = tc::get_encoder();
    if (!enc) return false;
    const cuuint64_t st = (cuuint64_t)v.st * 2;
    cuuint64_t dim[4] = {(cuuint64_t)width, (cuuint64_t)n, (cuuint64_t)(v.sh ? H : 1), (cuuint64_t)(v.sb ? B : 1)};
    cuuint64_t str[3] = {st, v.sh ? (cuuint64_t)v.sh * 2 : st, v.sb ? (cuuint64_t)v.sb * 2 : st};
    cuuint32_t box[4] = {64, (cuuint32_t)rows, 1, 1}, es[4] = {1, 1, 1, 1};
    return enc(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, v.p, dim, str, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

HLA_DEVICE void tma_load_4d(void *dst, const void *tmap, uint64_t *bar, int c0, int c1, int c2, int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
        "l"(tmap), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}
// A tile of T rows and DP columns (DP / 64 boxes) at row r0 of (b, h).
template <int DP>
HLA_DEVICE void load_tile(uint8_t *dst, const CUtensorMap *m, const View &v, uint64_t *bar, int r0, int h, int b) {
#pragma unroll
    for (int c = 0; c < DP; c += 64) tma_load_4d(dst + (c >> 6) * T * 128, m, bar, c, r0, v.sh ? h : 0, v.sb ? b : 0);
}

HLA_DEVICE void mbar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Bounded, warp-uniform waits: a poll sleeps in hardware until the phase
// completes or its time is up; the CTA's abort flag or a number of polls (2 s) end the wait,
// and the latter raises the device status word.
struct Waits {
    uint64_t *bars;
    volatile int *abort_p;
    unsigned *err;
    HLA_DEVICE uint64_t *bar(int i) const { return bars + i; }
    HLA_DEVICE bool wait(int b, uint32_t parity) const {
        if (__all_sync(0xffffffffu, mbar_try_wait(bars + b, parity))) return true;
        for (int polls = 0; !*abort_p; ++polls) {
            if (__all_sync(0xffffffffu, mbar_try_wait(bars + b, parity))) return true;
            if (polls == 2000) {
                atomicOr(err, DEV_TIMEOUT);
                *abort_p = 1;
            }
            __syncwarp();
        }
        return false;
    }
};
// Slot and phase of a ring of NS slots, counted up use by use.
template <int NS>
struct Ring {
    uint32_t slot = 0, phase = 0;
    HLA_DEVICE void next() {
        if (++slot == NS) {
            slot = 0;
            phase ^= 1u;
        }
    }
};

// ---- MMA groups, issued by a whole warp in uniform control flow with uniform operands: one
// lane is elected for a group.  The operands then stay in uniform registers (17 cycles per
// instruction against 45 when one thread issues them); a group is one block of instructions.
// D [128 x N] (+)= A B^T over 64 contraction columns: both K-major tiles
HLA_DEVICE void mma_ss64(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n .reg .pred p, e, t;\n .reg .b64 a1, a2, a3, b1, b2, b3;\n"
        " elect.sync _|e, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n setp.eq.b32 t, 0, 0;\n"
        " add.s64 a1, %1, 2;\n add.s64 b1, %2, 2;\n add.s64 a2, %1, 4;\n add.s64 b2, %2, 4;\n"
        " add.s64 a3, %1, 6;\n add.s64 b3, %2, 6;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, t;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, t;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u)
        : "memory");
}
// D [128 x N] (+)= A B over 32 contraction rows of B: A packed bf16 in TMEM (16 columns), B MN-major
HLA_DEVICE void mma_ts32(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n .reg .pred p, e, t;\n .reg .b64 b1;\n .reg .b32 a1;\n elect.sync _|e, 0xffffffff;\n"
        " setp.ne.b32 p, %4, 0;\n setp.eq.b32 t, 0, 0;\n add.s64 b1, %2, 128;\n add.u32 a1, %1, 8;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u)
        : "memory");
}
// A warp-uniform value, known as such to the compiler.
HLA_DEVICE uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }
// Descriptors of a tile: contraction over its columns, or over its rows.
HLA_DEVICE uint64_t kmajor(const uint8_t *tile) { return make_sdesc(smem_u32(tile), 16u, 1024u); }
HLA_DEVICE uint64_t mnmajor(const uint8_t *tile) { return make_sdesc(smem_u32(tile), T * 128u, 1024u); }
// The whole width of two tiles (64 columns per block; zero columns behind the
// tensors' own are multiplied too): `wide` takes both blocks of DP = 128.
template <int DP>
HLA_DEVICE void mma_kk(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool wide) {
    mma_ss64(d, a, b, idesc, false);
    if (DP > 64 && wide) mma_ss64(d, a + T * 8, b + T * 8, idesc, true);
}

// 32 columns of 32-bit words, this warp's lanes.
HLA_DEVICE void tmem_ld32(uint32_t taddr, float (&v)[32]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
                 : "r"(taddr));
}
HLA_DEVICE float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Of 32 columns c0 .. c0 + 31, those in [lo, hi) or in [0, min(sk, hi)) as bits.  Masks go by
// bit tests: comparisons joined by && and || come out as a branch per element.
HLA_DEVICE uint32_t low_bits(int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; }
HLA_DEVICE uint32_t visible_bits(int c0, int lo, int hi, int sk) {
    return low_bits(hi - c0) & (~low_bits(lo - c0) | low_bits(sk - c0));
}
HLA_DEVICE void mask32(float (&v)[32], uint32_t bits, float other) {
#pragma unroll
    for (int e = 0; e < 32; ++e) v[e] = bits & (1u << e) ? v[e] : other;
}

// Zeroes rows [r0, T) of a tile (one warp) and shows the tensor cores the result: rows behind
// a sequence may be anything, and 0 times that is not 0 where they are contracted over.
template <int DP>
HLA_DEVICE void zero_rows(uint8_t *tile, int r0, int lane) {
#pragma unroll
    for (int c = 0; c < DP; c += 64)
        for (int e = (r0 << 3) + lane; e < T * 8; e += 32)
            reinterpret_cast<uint4 *>(tile + (c >> 6) * T * 128)[e] = make_uint4(0, 0, 0, 0);
    fence_async_smem();
    __syncwarp();
}

// CW (32 or 64) accumulator columns of this warp's 32 rows, each lane's row times f, to bf16
// rows `out` (of the warp's first row) at columns col0 .. below `width`, for the first `live`
// rows.  Through shared memory (`stage`, 64 CW bytes), so that a store writes whole pieces of
// rows: a row per thread straight from the registers touches 32 lines per store, and the
// output of a tile of 128 x 128 then took 3 to 4 us.
template <int CW>
HLA_DEVICE void store_rows(uint8_t *stage, uint32_t taddr, float f, __nv_bfloat16 *out, long long st, int live, int col0,
                           int width) {
    constexpr int P = CW / 8;  // 16-byte pieces of a row, swizzled by the row
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int g = 0; g < CW / 32; ++g) {
        float v[32];
        tmem_ld32(taddr + 32 * g, v);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float *x = v + 8 * e;
            *reinterpret_cast<uint4 *>(stage + lane * (P * 16) + (((4 * g + e) ^ ((lane * P / 8) & (P - 1))) << 4)) =
                make_uint4(pack_bf16(x[0] * f, x[1] * f), pack_bf16(x[2] * f, x[3] * f), pack_bf16(x[4] * f, x[5] * f),
                           pack_bf16(x[6] * f, x[7] * f));
        }
    }
    __syncwarp();
    const int col = col0 + 8 * (lane & (P - 1));
#pragma unroll
    for (int e = 0; e < P; ++e) {
        const int row = 32 / P * e + lane / P;
        const uint4 u = *reinterpret_cast<const uint4 *>(stage + row * (P * 16) + (((lane & (P - 1)) ^ ((row * P / 8) & (P - 1))) << 4));
        if (row < live && col < width) *reinterpret_cast<uint4 *>(out + (size_t)row * st + col) = u;
    }
    __syncwarp();
}

}  // namespace tcw
}  // namespace win
}  // namespace hla
