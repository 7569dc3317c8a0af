// hla_ssm.h -- argument bundle and shared pieces of the selective state space scan's kernels.
//
// Per head, with the log decay a_t = dt_t A log2(e) (not below -256) and s its running sum inside
// a chunk of Q tokens (inclusive; e = 2^s from the chunk's start to a token, r = 2^(s_end - s) from
// the token to the chunk's end, L_tj = 2^(s_t - s_j) for j <= t):
//   h' = 2^s_end h + B^T diag(dt r) X                    state after the chunk
//   Y  = ((C B^T) o L diag(dt)) X + diag(e) C h + D X
// and backward, with g the gradient of the state after the chunk and g' that of h:
//   g' = 2^s_end g + C^T diag(e) dY
//   M = (C B^T) o L,  S = (dY X^T) o L,  E = M o (dY X^T)
//   dX = diag(dt) (M^T dY + diag(r) B g) + D dY
//   dB = diag(dt) (S^T C + diag(r) X g^T),   dC = S diag(dt) B + diag(e) dY h^T   (sums over a group's heads)
//   v_j = sum_t E_tj + r_j B_j.(X g^T)_j,  w_t = sum_j E_tj dt_j + e_t C_t.(dY h^T)_t
//   da_t = 2^s_end <g, h> + sum_{i >= t} (w_i - dt_i vE_i) + sum_{j < t} dt_j vg_j
//          (what passes token t from those before it to those behind it; vE, vg the two parts of v)
//   d_dt = A da + v,  dA = sum dt da,  dD = sum dY.X
// Every exponent is a sum of a's between two tokens, so nothing overflows while A <= 0 <= dt.
#pragma once
#include "hla_layer.cuh"

namespace hla {
namespace ssm {

using namespace layer;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLeast = -256.f;  // 2^-256 is 0 next to any other fp32 factor

struct Args {
    int B, H, G, R;  // R = H / G heads to a group
    int n, P, N;
    bool softplus;
    const float *A, *D, *dt_bias;
    const int *lengths;
    View x, dt, b, c, y, dy, dx, ddt, db, dc;
    const float *state_in, *d_state_out;
    float *state_out, *d_state_in, *dA, *dD, *dbias;
    // workspace
    int nc;               // chunks of a sequence (CUDA cores: of the span under way)
    int splits;           // backward: CTAs that share a group's heads
    int t0, rows;         // CUDA cores: first token of the span, its tokens
    int hc, h0;           // CUDA cores: chunks that `h` holds, the span's first among them
    int sum0, sumc;       // CUDA cores: the span's first chunk and all chunks, in `sums`
    const float *from[2]; // CUDA cores: states before the span, gradients behind it
    float *to[2];         // ... states behind it, gradients before it
    float *carry;         // [B][H][N][P]: either, between spans
    float *h, *g;         // [B][H][nc][N][P]: states (`hc` chunks of them) and their gradients
    float *factor;        // [B][H][hc]: 2^s_end
    float *dbc;           // [splits][2][B][G][rows][N]
    void *dec;            // [B][H][nc]: the chunks' weights (tensor cores)
    unsigned char *image[2];  // tensor cores, backward: the chunks' states and their gradients, and fp32 sums of tokens and borders
    float *inter, *aside, *dots, *own, *dd;
    float *sums;          // [rows][3][H]: parts of dA, dD, dt_bias' gradient
    unsigned *err;
};

// dt as the recurrence takes it.
HLA_DEVICE float softplus(float x) {  // log(1 + e^x), both parts a few units in the last place off
    return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x)));
}

// One chunk's steps and running log decays.  The sum is kept in two parts, whole numbers (exact)
// and a remainder of at most one half, and whatever is added to either is settled at once, so that no
// addition rounds by more than 2^-25: a remainder is rounded PER - 1 times by its lane, five times
// across the warp and once when both meet.  2^(s_t - s_j) then comes out within 2^-20.5 for neighbours,
// however far behind a steep decay they are, and for tokens d apart within d 2^-22 more, which is what
// the roundings of A log2(e), of its products with dt and of s_t - s_j amount to.  (With remainders that are
// settled once at the end, a warp's sum of them reaches 60: decays were up to 2^-17.9 off.)
struct Decay {
    float hi, lo;
};
HLA_DEVICE float factor(Decay t, Decay j) { return ex2_approx((t.hi - j.hi) + (t.lo - j.lo)); }
HLA_DEVICE float factor(Decay t) { return ex2_approx(t.hi + t.lo); }

template <typename T>
HLA_DEVICE float raw_step(const Args &a, int b, int h, int t) {
    float raw[1];
    widen<T, 1>(load_raw<T, 1>(static_cast<const T *>(a.dt.p) + (size_t)b * a.dt.sb + (size_t)h * a.dt.sh + (size_t)t * a.dt.st), raw);
    return raw[0];
}
HLA_DEVICE float step_from(const Args &a, float raw, float bias, float &slope) {
    slope = 1.f;
    if (!a.softplus) return raw;
    slope = 1.f / (1.f + expf(-(raw + bias)));
    return softplus(raw + bias);
}
template <typename T>
HLA_DEVICE float step_of(const Args &a, int b, int h, int t, float bias, float &slope) {
    return step_from(a, raw_step<T>(a, b, h, t), bias, slope);
}

// Log decay of one step, A2 = A log2(e).  A step of 0 keeps the state whatever A is (so do the rows
// behind a sequence, which get one); a rate that is not a number stays one, where fmaxf would drop it.
HLA_DEVICE float log_decay(float d, float A2) { return A2 != A2 ? A2 : d == 0.f ? 0.f : fmaxf(d * A2, kLeast); }

// One warp, PER adjacent tokens of a chunk a lane: their steps d to running log decays s.
template <int PER>
HLA_DEVICE void scan_decays(const float (&d)[PER], float A2, Decay (&s)[PER]) {
    const int lane = threadIdx.x & 31;
    auto settle = [](float &h, float &l) {
        const float w = rintf(l);
        h += w;
        l -= w;
    };
    float hi[PER], lo[PER], sh = 0.f, sl = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const float l = log_decay(d[i], A2), w = rintf(l);
        sh += w;
        sl += l - w;
        settle(sh, sl);
        hi[i] = sh;
        lo[i] = sl;
    }
    float ph = sh, pl = sl;  // sums of the lanes up to this one
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float uh = __shfl_up_sync(0xffffffffu, ph, o), ul = __shfl_up_sync(0xffffffffu, pl, o);
        if (lane >= o) {
            ph += uh;
            pl += ul;
            settle(ph, pl);
        }
    }
    ph = __shfl_up_sync(0xffffffffu, ph, 1);  // and of those before it
    pl = __shfl_up_sync(0xffffffffu, pl, 1);
    if (lane == 0) ph = pl = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        s[i] = {hi[i] + ph, lo[i] + pl};
        settle(s[i].hi, s[i].lo);
    }
}

// A chunk of PER * 32 tokens from t0 on (zeros behind `len`), by one warp.
template <typename T, int PER>
HLA_DEVICE void chunk_decays(const Args &a, int b, int h, int t0, int len, float *dt, Decay *s, float *slope) {
    const int lane = threadIdx.x & 31;
    const float bias = a.softplus && a.dt_bias ? a.dt_bias[h] : 0.f;
    float d[PER];
    Decay r[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int t = t0 + lane * PER + i;
        float sp = 0.f;
        d[i] = t < len ? step_of<T>(a, b, h, t, bias, sp) : 0.f;
        if (slope) slope[lane * PER + i] = sp;
    }
    scan_decays(d, a.A[h] * kLog2e, r);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        dt[lane * PER + i] = d[i];
        s[lane * PER + i] = r[i];
    }
}

// CUDA cores (any strides, widths and types): chunks of 64 tokens, 32 where both widths pass 64, taken in
// spans whose states fit a workspace of bounded size.
inline int simt_chunk(int P, int N) { return P > 64 && N > 64 ? 32 : 64; }
size_t simt_space(Args &a, bool backward, uint8_t *base);  // bytes; sets the pointers when `base` is given
cudaError_t simt_forward(const Args &a, hla_dtype dt, cudaStream_t st);
cudaError_t simt_backward(const Args &a, hla_dtype dt, cudaStream_t st);
// What both backward paths end with: dB, dC from their parts; dA, dD and dt_bias' gradient from `rows` sums.
cudaError_t join_parts(const Args &a, hla_dtype dt, cudaStream_t st);
cudaError_t join_sums(const Args &a, int rows, cudaStream_t st);

// Tensor cores: bf16 whose rows start on 16-byte boundaries (tc_takes); the workspace's bytes, its
// pointers set when `base` is given; cudaErrorNotSupported, with nothing launched, when the driver
// cannot describe a tensor to the TMA unit.
bool tc_takes(const Args &a, bool backward);
size_t tc_space(Args &a, bool backward, uint8_t *base);
cudaError_t tc_forward(const Args &a, cudaStream_t st);
cudaError_t tc_backward(const Args &a, cudaStream_t st);
int tc_splits(const Args &a);

}  // namespace ssm
}  // namespace hla
