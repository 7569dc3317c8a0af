// hla_window.h -- argument bundles shared by the windowed-attention kernels.
#pragma once
#include "hla_strided.h"

namespace hla {
namespace win {

struct Args {
    int B, H, Hkv, G;  // G = H / Hkv query heads to a key/value head
    int n, nk, p0;     // query row i stands at position p0 + i, p0 = nk - n
    int d, dv, window, sinks;
    float scale;
    const int *lengths;
    View q, k, v, o, go, dq, dk, dv_;
    float *lse;
    // backward: D = rowsum(do o) [B][H][n]; partial dk, dv of the key tiles that hold
    // first tokens, [far][B][Hkv][keys][d | dv] fp32 (0: those of the window itself)
    float *delta, *part;
    int far, far_keys;
    unsigned *err;
};

// Tokens of sequence b, and the keys a tile of query positions [p_lo, p_hi] can reach.
HLA_DEVICE int length_of(const Args &a, int b) {
    if (!a.lengths) return a.nk;
    const int L = a.lengths[b];
    return L < 0 ? 0 : L > a.nk ? a.nk : L;
}
// p - window >= j without overflow: window may be as large as INT_MAX.
HLA_DEVICE bool visible(const Args &a, int p, int j) { return j <= p && (p - j < a.window || j < a.sinks); }

// The key tiles (of TK keys) of one tile of query positions [p_lo, p_hi], in order:
// those before the window that hold first tokens, then the window's.
struct KeyTiles {
    int head, lo, total;  // tiles 0..head-1, then lo, lo + 1, ...
    HLA_DEVICE KeyTiles(const Args &a, int p_lo, int p_hi, int TK) {
        const int j_lo = p_lo - a.window + 1 > 0 && p_lo >= a.window ? p_lo - a.window + 1 : 0;
        lo = j_lo / TK;
        const int hi = p_hi / TK;  // p_hi < length: the last key is the last query's own
        const int sink_tiles = a.sinks > 0 ? (a.sinks - 1) / TK + 1 : 0;
        head = sink_tiles < lo ? sink_tiles : lo;
        total = head + hi - lo + 1;
    }
    HLA_DEVICE int operator[](int i) const { return i < head ? i : lo + i - head; }
};

struct StepArgs {
    int B, H, Hkv, G, d, dv, window, sinks;
    float scale;
    const long long *pos;
    View q, k, v, kc, vc, o;  // st of q, k, v, o is not used
    bool wide;                // rows of k, v, kc, vc are multiples of 16 bytes
    int split;                // CTAs of one cluster
};
cudaError_t step(const StepArgs &a, hla_dtype dt, cudaStream_t st);

// bf16 tensor-core kernels (rows in multiples of 16 bytes); cudaErrorNotSupported, with
// nothing launched, when the driver cannot describe a tensor to the TMA unit
bool fwd_tc_takes(const Args &a);
cudaError_t fwd_tc(const Args &a, cudaStream_t st);
// (with far shares the caller adds them up afterwards; kTcTile: the keys of one tile)
constexpr int kTcTile = 128;
bool bwd_tc_takes(const Args &a);
cudaError_t bwd_tc(const Args &a, cudaStream_t st);

}  // namespace win
}  // namespace hla
