// hla_ssm_fwd_tc.cu -- forward of the selective state space scan for bf16 on the tensor cores
// (kernels in hla_ssm_carry.cuh).
#include <cstring>

#include "hla_ssm_carry.cuh"

namespace hla {
namespace ssm {
namespace {

using namespace tcs;

template <int NB>
cudaError_t launch(const Params &p, cudaStream_t st) {
    const cudaError_t e = starts<NB>(p, 1, st);
    return e == cudaSuccess ? walk<NB, true>(p, st) : e;
}

}  // namespace

bool tc_takes(const Args &a, bool backward) {
    const bool in = a.P % 8 == 0 && a.N % 8 == 0 && mappable(a.x) && mappable(a.b) && mappable(a.c);
    if (!backward) return in && mappable(a.y);
    return in && mappable(a.dy) && mappable(a.dx) && rows16(a.db, 2) && rows16(a.dc, 2);
}

size_t tc_space(Args &a, bool backward, uint8_t *base) {
    const Plan plan = plan_of(a, kSms);
    a.nc = (int)(((long long)a.n + T - 1) / T);
    size_t at = 0;
    auto take = [&](size_t floats) {
        float *p = base ? reinterpret_cast<float *>(base + at) : nullptr;
        at += align256(floats * 4);
        return p;
    };
    a.dec = take((size_t)a.B * a.H * a.nc * (sizeof(Dec) / 4));
    const size_t units = plan.pieces > 1 ? (size_t)a.B * a.H * plan.pieces : 0;
    a.h = take(units * a.N * a.P);
    a.factor = take(units);
    if (backward) {
        a.g = take(units * a.N * a.P);
        const size_t image = (size_t)a.B * a.H * plan.PT * a.nc * (a.N <= 64 ? 1 : 2) * (kHalf / 4);  // two parts of 64 rows each
        a.image[0] = reinterpret_cast<unsigned char *>(take(image));
        a.image[1] = reinterpret_cast<unsigned char *>(take(image));
        a.splits = tc_splits(a);
        a.dbc = take(a.splits > 1 ? (size_t)a.splits * 2 * a.B * a.G * a.n * a.N : 0);
        a.sums = take((size_t)a.B * a.nc * 3 * a.H);
    }
    return at;
}

cudaError_t tc_forward(const Args &a, cudaStream_t st) {
    Params p;
    memset(&p, 0, sizeof p);
    p.a = a;
    p.plan = plan_of(a, kSms);
    p.vx[0] = a.x;
    p.vb[0] = a.b;
    p.pieces[0] = a.h;
    p.factor = a.factor;
    p.dec = static_cast<const Dec *>(a.dec);
    const cudaError_t e = dev_status_ptr(&p.a.err);
    if (e != cudaSuccess) return e;
    if (!encode(&p.mx[0], a.x, a.P, a.n, a.H, a.B, T) || !encode(&p.mb[0], a.b, a.N, a.n, a.G, a.B, T) ||
        !encode(&p.mc, a.c, a.N, a.n, a.G, a.B, T) || !encode(&p.my, a.y, a.P, a.n, a.H, a.B, T))
        return cudaErrorNotSupported;
    return a.N <= 64 ? launch<1>(p, st) : launch<2>(p, st);
}

}  // namespace ssm
}  // namespace hla
