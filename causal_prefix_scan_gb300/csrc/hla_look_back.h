// hla_look_back.h -- where one channel's look-back starts its fold.  Plain C++ beside the
// kernel that uses it, so that its rules also run on the host under any order of publication.
//
// A look-back reads windows of W records, nearest tile first, and keeps the last N of them:
// record w of window r lies at index slot(r) * W + w.  Rounds 0 .. N - 1 read window r; every later round
// reads the last window again, once all its records are states.
#pragma once

#if defined(__CUDACC__)
#define HLA_LOOK_BACK_FN __host__ __device__ __forceinline__
#else
#define HLA_LOOK_BACK_FN inline
#endif

namespace hla {
namespace gated {

// Kinds of a record; 0 is no record (before the chain's first tile).
enum : unsigned long long { REC_MAP = 1, REC_STATE = 2 };

template <int N, int W>
struct FoldStart {
    int found = -1;  // index of the nearest state, -1: none yet

    static HLA_LOOK_BACK_FN int slot(int r) { return r < N ? r : N - 1; }
    // Whether round r takes a record only once it is a state.
    static HLA_LOOK_BACK_FN bool states_only(int r) { return r >= N; }
    // After round r: kind(w) of its window's records.  A window that is read again holds states
    // where it held maps, also for a channel that needs none: that channel's start moves to the nearest of them.
    template <class Kind>
    HLA_LOOK_BACK_FN void look(int r, Kind kind) {
        if (states_only(r) && found >= slot(r) * W) found = -1;
        if (found >= 0) return;
#if defined(__CUDACC__)
#pragma unroll
#endif
        for (int w = 0; w < W; ++w)
            if (found < 0 && kind(w) == (int)REC_STATE) found = slot(r) * W + w;
    }
    // The state before the tile: from the state found through the maps nearer than it.
    // state(i): the state of record i; step(i, h): h taken through record i's map.
    template <class State, class Step>
    HLA_LOOK_BACK_FN float fold(State state, Step step) const {
        float h = state(found);
        for (int i = found - 1; i >= 0; --i) h = step(i, h);
        return h;
    }
};

}  // namespace gated
}  // namespace hla
