// The look-back of one tile on the host, under orders of publication chosen at random:
// the kernel's rules (hla_look_back.h) with its rounds, its records and its way of ending
// (when every channel has a state), one record per channel of every earlier tile.
//
//   look_back_model(tiles, channels, behind, seed, gate, out)
// Tile `tiles` looks back over tiles 0 .. tiles - 1 of a chain with the map h -> gate h + 1 per
// tile, state 0 before the first.  Between any two records read, further states appear, in
// the chain's order but channel by channel; at first the states of `behind` tiles have yet to.
// out[c]: the state that channel c computes.  Returns the number of rounds.
#include <cstdint>
#include <vector>

#include "hla_look_back.h"

using namespace hla::gated;

namespace {
constexpr int N = 8, W = 8;
struct Rng {
    uint64_t s;
    uint32_t next() {
        s = s * 6364136223846793005ull + 1442695040888963407ull;
        return (uint32_t)(s >> 33);
    }
};
}  // namespace

extern "C" int look_back_model(int tiles, int channels, int behind, uint64_t seed, float gate, float *out) {
    Rng rng{seed * 2 + 1};
    std::vector<float> state(tiles);
    float h = 0.f;
    for (int t = 0; t < tiles; ++t) state[t] = h = gate * h + 1.f;
    std::vector<int> front(channels, tiles - behind);  // states below it are published, maps from it on
    for (int &f : front) f = f < 1 ? 1 : f;            // the first tile publishes nothing but its state
    std::vector<FoldStart<N, W>> start(channels);
    std::vector<std::vector<float>> a(N * W, std::vector<float>(channels)), b = a;
    std::vector<std::vector<int>> kind(W, std::vector<int>(channels));
    for (int r = 0;; ++r) {
        const int slot = FoldStart<N, W>::slot(r);
        for (int w = 0; w < W; ++w) {
            const int prev = tiles - 1 - (slot * W + w);
            for (int c = 0; c < channels; ++c) {
                if (rng.next() % 64 == 0) {
                    int &f = front[rng.next() % channels];
                    f = f + 1 > tiles ? tiles : f + 1;
                }
                kind[w][c] = 0;
                if (prev < 0) continue;
                if (FoldStart<N, W>::states_only(r) && front[c] <= prev) front[c] = prev + 1;  // waited for
                const bool is_state = prev < front[c];
                kind[w][c] = (int)(is_state ? REC_STATE : REC_MAP);
                a[slot * W + w][c] = gate;
                b[slot * W + w][c] = is_state ? state[prev] : 1.f;
            }
        }
        bool all = true;
        for (int c = 0; c < channels; ++c) {
            start[c].look(r, [&](int w) { return kind[w][c]; });
            all = all && start[c].found >= 0;
        }
        if (!all) continue;
        for (int c = 0; c < channels; ++c)
            out[c] = start[c].fold([&](int i) { return b[i][c]; }, [&](int i, float x) { return a[i][c] * x + b[i][c]; });
        return r + 1;
    }
}
