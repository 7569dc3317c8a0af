// hla_gated_stream.cu -- gated recurrence where the channels of all sequences alone fill the
// device: one CTA takes 16 channels of one sequence and walks its tokens from end to end with
// the state on chip, so no CTA waits for another and nothing but the inputs and outputs
// moves.  A tile is NW warps x 4 groups x TS tokens; lane = 8 (group) + pair of channels, so
// a group's row is one 32-byte sector (bf16).  Per tile: gates and maps in registers, a scan of
// the four groups by shuffles, of the warps through shared memory (one barrier), then the
// outputs.  The next tile's inputs are loaded into the registers of the present one as they
// become free, so memory works while the tile is computed.
//
// Measured, bf16 with rates: forward 32,768 x 4,096 211 us (3.8 TB/s), backward 2 x 8,192 x
// 4,096 228 us (3.5 TB/s).  Bound by issue and the latencies under it: two exponentials, a reciprocal
// and a reciprocal root per element beside some thirty other instructions, with 24 (16) warps per SM,
// all that the registers allow (fp32 forward: 88 to 104 bytes spilled); 12 (8) warps of 8 tokens per
// thread were the best of 4 to 16 of 2 to 8.  256 CTAs put two on 104 of the 152 SMs, whose issue
// slots are 63 % (58 %) busy, and one on the others (32, 29 %).
#include <type_traits>

#include "hla_gated.cuh"

namespace hla {
namespace gated {
namespace {

constexpr int VEC = 2, GL = 8, GROUPS = 32 / GL, CW = GL * VEC, TS = 8;
constexpr int kWarpsFwd = 12, kWarpsBwd = 8;  // of a CTA

template <int NW>
struct Shared {
    float4 map[2][NW][GL];  // the warps' maps (A, A', B, B'), two tiles in turn
    float2 carry[2][GL];    // state before the tile
};

template <class V>
HLA_DEVICE V shfl_up(const V &x, int by) {
    return {__shfl_up_sync(0xffffffffu, x.v[0], by), __shfl_up_sync(0xffffffffu, x.v[1], by)};
}

// From the map (A, B) of this thread's tokens to the state before them; the state after the
// tile goes into sh.carry for the next one.  `k` counts tiles.
template <int NW, class V>
HLA_DEVICE V state_before(Shared<NW> &sh, int k, V A, V B) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, grp = lane / GL, c = lane % GL;
#pragma unroll
    for (int by = GL; by < 32; by <<= 1) {
        const V a = shfl_up(A, by), b = shfl_up(B, by);
        if (lane >= by) {
            B = fma_(A, b, B);
            A = mul_(A, a);
        }
    }
    if (grp == GROUPS - 1) sh.map[k & 1][warp][c] = make_float4(A.v[0], A.v[1], B.v[0], B.v[1]);
    V ea = shfl_up(A, GL), eb = shfl_up(B, GL);
    if (grp == 0) {
        ea = splat<V>(1.f);
        eb = splat<V>(0.f);
    }
    __syncthreads();
    const float2 c0 = sh.carry[k & 1][c];
    V h = {c0.x, c0.y};
    for (int w = 0; w < warp; ++w) {
        const float4 m = sh.map[k & 1][w][c];
        h = fma_(V{m.x, m.y}, h, V{m.z, m.w});
    }
    if (warp == NW - 1 && grp == GROUPS - 1) {
        const V after = fma_(A, h, B);
        sh.carry[(k + 1) & 1][c] = make_float2(after.v[0], after.v[1]);
    }
    return fma_(ea, h, eb);
}

// Rows are addressed as base + offset: the base (sequence, slice, tile) is the same for the
// whole CTA, the 32-bit offset of a thread's token in the tile never changes (64-bit addresses
// of every row cost a quarter of the instructions, 26 us of the forward on 32,768 x 4,096).
template <typename T>
struct Rows {
    char *p;
    uint32_t off, step;  // bytes: the thread's first token, one token
    HLA_DEVICE Rows(const Tensor &t, int b, int c0, int first, int t0, int lane_ch)
        : p(static_cast<char *>(const_cast<void *>(t.p)) + ((long long)b * t.sb + c0 + (long long)first * t.st) * (long long)sizeof(T)),
          off(((uint32_t)t0 * (uint32_t)t.st + lane_ch) * (uint32_t)sizeof(T)), step((uint32_t)t.st * (uint32_t)sizeof(T)) {}
    HLA_DEVICE raw_t<T, VEC> load(int i) const { return __ldg(reinterpret_cast<const raw_t<T, VEC> *>(p + (size_t)(off + i * step))); }
    HLA_DEVICE void store(int i, const raw_t<T, VEC> &r) const { *reinterpret_cast<raw_t<T, VEC> *>(p + (size_t)(off + i * step)) = r; }
    HLA_DEVICE void move(int tokens) { p += (long long)tokens * step; }
};

template <class V>
HLA_DEVICE V load_state(const float *p, size_t off, bool ok) {
    V s = splat<V>(0.f);
    if (p && ok) s = {p[off], p[off + 1]};
    return s;
}

// ------------------------------------------------------------ forward
template <typename T, int GATE, int NW>
__global__ void __launch_bounds__(NW * 32, 2) stream_fwd_kernel(const Args a) {
    constexpr int TT = NW * GROUPS * TS;
    __shared__ Shared<NW> sh;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.x / a.slices, ch = (int)(blockIdx.x % a.slices) * CW + lane % GL * VEC;
    const bool mine = ch < a.d;
    const int len = length_of(a, b);
    const size_t so = (size_t)b * a.d + ch;
    if (warp == NW - 1 && lane >= 32 - GL) {
        const Num<T, 2> s = load_state<Num<T, 2>>(a.state_in, so, mine);
        sh.carry[0][lane % GL] = make_float2(s.v[0], s.v[1]);
    }
    const int t0 = (warp * GROUPS + lane / GL) * TS;  // first token of this thread in a tile
    const bool whole = (int)(blockIdx.x % a.slices) * CW + CW <= a.d;
    const int c0 = (int)(blockIdx.x % a.slices) * CW, lc = lane % GL * VEC;
    Rows<T> xs(a.x, b, c0, 0, t0, lc), gs(a.g, b, c0, 0, t0, lc), ys(a.o1, b, c0, 0, t0, lc);
    using R = raw_t<T, VEC>;
    R xr[TS] = {}, gr[TS] = {};
#pragma unroll
    for (int i = 0; i < TS; ++i)
        if (mine && t0 + i < len) {
            gr[i] = gs.load(i);
            xr[i] = xs.load(i);
        }
    const Num<T, 2> r = rate_of<GATE, Num<T, 2>>(a, ch);
    int k = 0;
    // FULL: this tile and the next have all their tokens and the slice all its channels
    auto tile = [&](int base, auto full) {
        constexpr bool FULL = decltype(full)::value;
        xs.move(TT);
        gs.move(TT);
        Num<T, 2> ea[TS], eb[TS], A = splat<Num<T, 2>>(1.f), B = splat<Num<T, 2>>(0.f);
#pragma unroll
        for (int i = 0; i < TS; ++i) {
            Num<T, 2> x, g;
            unpack(xr[i], x.v);
            unpack(gr[i], g.v);
            gate_fwd<GATE>(g, r, x, ea[i], eb[i]);
            if (!FULL && base + t0 + i >= len) {
                ea[i] = splat<Num<T, 2>>(1.f);
                eb[i] = splat<Num<T, 2>>(0.f);
            }
            if (FULL || (mine && base + TT + t0 + i < len)) {
                gr[i] = gs.load(i);
                xr[i] = xs.load(i);
            }
            B = fma_(ea[i], B, eb[i]);
            A = mul_(A, ea[i]);
        }
        Num<T, 2> h = state_before(sh, k++, A, B);
#pragma unroll
        for (int i = 0; i < TS; ++i) {
            h = fma_(ea[i], h, eb[i]);
            if (FULL || (mine && base + t0 + i < len)) {
                R o;
                pack(h.v, o);
                ys.store(i, o);
            }
        }
        ys.move(TT);
    };
    int base = 0;
    if (whole)
        for (; base + 2 * TT <= len; base += TT) tile(base, std::true_type());
    for (; base < len; base += TT) tile(base, std::false_type());
    __syncthreads();
    if (a.out_state && warp == 0 && lane < GL && mine) {
        const float2 s = sh.carry[k & 1][lane];
        a.out_state[so] = s.x;
        a.out_state[so + 1] = s.y;
    }
}

// ------------------------------------------------------------ backward
template <typename T, int GATE, int NW>
__global__ void __launch_bounds__(NW * 32, 2) stream_bwd_kernel(const Args a) {
    constexpr int TT = NW * GROUPS * TS;
    __shared__ Shared<NW> sh;
    __shared__ float2 red[NW][GL];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.x / a.slices, ch = (int)(blockIdx.x % a.slices) * CW + lane % GL * VEC;
    const bool mine = ch < a.d;
    const int len = length_of(a, b);
    const size_t so = (size_t)b * a.d + ch;
    if (warp == NW - 1 && lane >= 32 - GL) {
        const Num<T, 2> s = load_state<Num<T, 2>>(a.d_state_out, so, mine);
        sh.carry[0][lane % GL] = make_float2(s.v[0], s.v[1]);
    }
    // the first group takes a tile's last tokens: groups and warps follow the scan's direction
    const int t0 = (NW * GROUPS - 1 - (warp * GROUPS + lane / GL)) * TS;
    const bool whole = (int)(blockIdx.x % a.slices) * CW + CW <= a.d;
    int base = len > 0 ? (len - 1) / TT * TT : 0;
    const int c0 = (int)(blockIdx.x % a.slices) * CW, lc = lane % GL * VEC;
    Rows<T> xs(a.x, b, c0, base, t0, lc), gs(a.g, b, c0, base, t0, lc), ys(a.y, b, c0, base - 1, t0, lc),  // y: h_{t-1}
        ds(a.dy, b, c0, base, t0, lc), os(a.o1, b, c0, base, t0, lc), qs(a.o2, b, c0, base, t0, lc);
    using R = raw_t<T, VEC>;
    R gr[TS] = {}, dr[TS] = {}, yr[TS] = {}, xr[TS] = {};
    auto fetch = [&](int i, int t) {  // token t = its tile's base + t0 + i
        gr[i] = gs.load(i);
        dr[i] = ds.load(i);
        if (i > 0 || t > 0) yr[i] = ys.load(i);
        if constexpr (GATE != HLA_GATE_GIVEN) xr[i] = xs.load(i);
    };
#pragma unroll
    for (int i = TS - 1; i >= 0; --i)
        if (mine && base + t0 + i < len) fetch(i, base + t0 + i);
    const Num<T, 2> r = rate_of<GATE, Num<T, 2>>(a, ch);
    const Num<T, 2> h0 = load_state<Num<T, 2>>(a.state_in, so, mine && t0 == 0);
    Num<T, 2> sum = splat<Num<T, 2>>(0.f);
    int k = 0;
    // FULL: the tile has all its tokens (every earlier one has) and the slice all its channels
    auto tile = [&](auto full) {
        constexpr bool FULL = decltype(full)::value;
        Num<T, 2> kept[TS], A = splat<Num<T, 2>>(1.f), B = splat<Num<T, 2>>(0.f);
#pragma unroll
        for (int i = TS - 1; i >= 0; --i) {
            Num<T, 2> g, dy;
            unpack(gr[i], g.v);
            unpack(dr[i], dy.v);
            Num<T, 2> at;
            kept[i] = gate_keep<GATE>(g, r, at);
            if (!FULL && (!mine || base + t0 + i >= len)) {
                kept[i] = splat<Num<T, 2>>(kKeptOff<GATE>);
                at = splat<Num<T, 2>>(1.f);
                dy = splat<Num<T, 2>>(0.f);
            }
            B = mul_(at, add_(dy, B));
            A = mul_(A, at);
        }
        Num<T, 2> c = state_before(sh, k++, A, B);
        const bool more = base > 0;  // then the next tile is whole
        gs.move(-TT);
        ds.move(-TT);
        ys.move(-TT);
        if constexpr (GATE != HLA_GATE_GIVEN) xs.move(-TT);
#pragma unroll
        for (int i = TS - 1; i >= 0; --i) {
            Num<T, 2> g, dy, x = splat<Num<T, 2>>(0.f), y, dx, dg, drv, at;
            unpack(gr[i], g.v);
            unpack(dr[i], dy.v);
            unpack(yr[i], y.v);
            if constexpr (GATE != HLA_GATE_GIVEN) unpack(xr[i], x.v);
            if (i == 0 && base + t0 == 0) y = h0;
            if (more && (FULL || mine)) fetch(i, base - TT + t0 + i);
            const Num<T, 2> gh = add_(dy, c);
            gate_bwd<GATE>(g, r, x, y, gh, kept[i], dx, dg, drv, at);
            if (FULL || (mine && base + t0 + i < len)) {
                c = mul_(at, gh);
                if constexpr (GATE == HLA_GATE_RATE) sum = add_(sum, drv);
                R o, q;
                pack(dx.v, o);
                pack(dg.v, q);
                os.store(i, o);
                qs.store(i, q);
            }
        }
        os.move(-TT);
        qs.move(-TT);
    };
    if (len > 0) {
        if (!whole || base + TT > len) {
            tile(std::false_type());
            base -= TT;
        }
        if (whole)
            for (; base >= 0; base -= TT) tile(std::true_type());
        else
            for (; base >= 0; base -= TT) tile(std::false_type());
    }
    __syncthreads();
    if (a.out_state && warp == 0 && lane < GL && mine) {
        const float2 s = sh.carry[k & 1][lane];
        a.out_state[so] = s.x;
        a.out_state[so + 1] = s.y;
    }
    if constexpr (GATE == HLA_GATE_RATE) {
        if (a.part) {  // groups, then warps, in order
#pragma unroll
            for (int by = GL; by < 32; by <<= 1) {
                sum.v[0] += __shfl_xor_sync(0xffffffffu, sum.v[0], by);
                sum.v[1] += __shfl_xor_sync(0xffffffffu, sum.v[1], by);
            }
            if (lane < GL) red[warp][lane] = make_float2(sum.v[0], sum.v[1]);
            __syncthreads();
            if (warp == 0 && lane < GL && mine) {
                float2 s = red[0][lane];
#pragma unroll
                for (int w = 1; w < NW; ++w) {
                    s.x += red[w][lane].x;
                    s.y += red[w][lane].y;
                }
                *reinterpret_cast<float4 *>(a.part + so) = make_float4(s.x, 0.f, 0.f, 0.f);
                *reinterpret_cast<float4 *>(a.part + so + 1) = make_float4(s.y, 0.f, 0.f, 0.f);
            }
        }
    }
}

// d_rate[c] = the sequences' sums in order
__global__ void __launch_bounds__(256) stream_rate_kernel(const Record *part, int B, int d, float *d_rate) {
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= d) return;
    float s = 0.f;
    for (int b = 0; b < B; ++b) s += part[(size_t)b * d + c].a;
    d_rate[c] = s;
}

template <typename T, int GATE>
cudaError_t launch(Args a, bool backward, cudaStream_t st) {
    a.slices = (a.d + CW - 1) / CW;
    const unsigned grid = (unsigned)((size_t)a.B * a.slices);
    if (backward)
        stream_bwd_kernel<T, GATE, kWarpsBwd><<<grid, kWarpsBwd * 32, 0, st>>>(a);
    else
        stream_fwd_kernel<T, GATE, kWarpsFwd><<<grid, kWarpsFwd * 32, 0, st>>>(a);
    return cudaGetLastError();
}
template <typename T>
cudaError_t by_gate(const Args &a, int gate, bool backward, cudaStream_t st) {
    if (gate == HLA_GATE_GIVEN) return launch<T, HLA_GATE_GIVEN>(a, backward, st);
    if (gate == HLA_GATE_SIGMOID) return launch<T, HLA_GATE_SIGMOID>(a, backward, st);
    return launch<T, HLA_GATE_RATE>(a, backward, st);
}

}  // namespace

// Against the look-back kernels (with rates, us): CTAs here, forward and backward of both.
//                               bf16 here   look-back    fp32 here   look-back
//    64  1 x 16,384 x 1,024      66 | 173     47 | 100     77 | 183    52 | 108
//   104  1 x 16,384 x 1,664      72 | 183     73 | 150     82 | 206    77 | 160
//   128  1 x 16,384 x 2,048      71 | 190     87 | 180     82 | 214    91 | 192
//   144  2 x  8,192 x 1,152      41 | 101     51 | 105     46 | 113    54 | 113
//   160  2 x  8,192 x 1,280      56 | 117     55 | 115     70 | 116    59 | 123
//   256  1 x  8,192 x 4,096      58 | 120     82 | 171     72 | 133    88 | 185
//  1024  4 x  2,048 x 4,096      59 | 110     81 | 169     79 | 133    85 | 186
// The forward is ahead from about three quarters of the SMs on (just past all of them, where a few
// get a second CTA, it loses some of it again), the backward from about all of them.
bool stream_takes(const Args &a, hla_dtype t, bool backward, int sms) {
    constexpr int most = (kWarpsFwd > kWarpsBwd ? kWarpsFwd : kWarpsBwd) * GROUPS * TS;  // tokens of a tile
    const long long st_end = (1LL << 32) / (most * (t == HLA_F32 ? 4 : 2));              // a tile's offsets have 32 bits
    for (const Tensor *x : {&a.x, &a.g, &a.y, &a.dy, &a.o1, &a.o2})
        if (x->st >= st_end) return false;
    const long long ctas = (long long)a.B * ((a.d + CW - 1) / CW);
    return 4 * ctas >= (backward ? 4 : 3) * sms;
}
cudaError_t stream_forward(const Args &a, hla_dtype t, int gate, cudaStream_t st) {
    return t == HLA_F32 ? by_gate<float>(a, gate, false, st) : by_gate<__nv_bfloat16>(a, gate, false, st);
}
cudaError_t stream_backward(const Args &a, hla_dtype t, int gate, float *d_rate, cudaStream_t st) {
    const cudaError_t e = t == HLA_F32 ? by_gate<float>(a, gate, true, st) : by_gate<__nv_bfloat16>(a, gate, true, st);
    if (e != cudaSuccess || !d_rate) return e;
    stream_rate_kernel<<<(a.d + 255) / 256, 256, 0, st>>>(a.part, a.B, a.d, d_rate);
    return cudaGetLastError();
}

}  // namespace gated
}  // namespace hla
