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
    using C = LayCarry<NB>;
    static_assert(C::SMEM <= 227 * 1024, "shared memory");
    cudaError_t e = starts<NB>(p, 1, st);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(ssm_carry_kernel<NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    const Args &a = p.a;
    ssm_carry_kernel<NB><<<(unsigned)((size_t)a.B * a.H * p.plan.PT * p.plan.pieces), kCarryThreads, C::SMEM, st>>>(p);
    return cudaGetLastError();
}

}  // namespace

bool tc_takes(const Args &a, bool backward) {
    const bool in = a.P % 8 == 0 && a.N % 8 == 0 && mappable(a.x) && mappable(a.b) && mappable(a.c);
    if (!backward) return in && mappable(a.y);
    return in && mappable(a.dy) && mappable(a.dx) && rows16(a.db, 2) && rows16(a.dc, 2);
}

size_t tc_space(Args &a, bool backward, uint8_t *base) {
    const Plan plan = plan_of(a, backward);
    a.nc = (int)(((long long)a.n + T - 1) / T);
    size_t at = 0;
    auto take = [&](size_t floats) {
        float *p = base ? reinterpret_cast<float *>(base + at) : nullptr;
        at += align256(floats * 4);
        return p;
    };
    a.dec = take((size_t)a.B * a.H * a.nc * (sizeof(Dec) / 4));
    const size_t units = plan.pieces > 1 ? (size_t)a.B * a.H * plan.pieces * plan.cuts : 0;
    a.h = take(units * a.N * a.P);
    a.factor = take(units);
    if (backward) {
        a.g = take(units * a.N * a.P);
        const size_t heads = (size_t)a.B * a.H, image = heads * plan.PT * a.nc * (a.N <= 64 ? 1 : 2) * (kHalf / 8);  // 64 rows of 128 bytes each
        a.image[0] = reinterpret_cast<unsigned char *>(take(image));
        a.image[1] = reinterpret_cast<unsigned char *>(take(image));
        a.inter = take(2 * plan.PT * 4 * heads * a.nc * T);
        a.aside = take(heads * plan.PT * a.nc * 8192);
        a.dots = take(heads * a.nc * plan.PT * 16);
        a.own = take(3 * heads * a.nc * T);
        a.dd = take(heads * a.nc);
        a.splits = tc_splits(a);
        a.dbc = take(a.splits > 1 ? (size_t)a.splits * 2 * a.B * a.G * a.n * a.N : 0);
        a.sums = take((size_t)a.B * plan.pieces * 3 * a.H);
    }
    return at;
}

cudaError_t tc_forward(const Args &a, cudaStream_t st) {
    Params p;
    memset(&p, 0, sizeof p);
    p.a = a;
    p.plan = plan_of(a, false);
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
