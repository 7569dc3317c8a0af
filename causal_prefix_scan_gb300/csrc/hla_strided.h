// hla_strided.h -- the strided [B][H][n][width] tensors of the layers with a constant-size state:
// views for the kernels, checks at the entry points.
#pragma once
#include "hla_internal.h"

namespace hla {

struct View {
    void *p;
    long long sb, sh, st;
};
struct Dims {
    long long B, H, n, w;  // sequences, heads, rows of a head, elements of a row
};
// The stride of a dimension with one element is never used: whatever it is, the kernels are
// chosen by the others.
inline View view(const hla_tensor *t, Dims s) {
    return {t->p, s.B > 1 ? t->sb : 0, s.H > 1 ? t->sh : 0, s.n > 1 ? t->st : (s.w + 7) / 8 * 8};
}

inline hla_status check_in(const hla_tensor *t, Dims s, hla_dtype dt, const char *what) {
    if (!t || !t->p) return report(HLA_ERR_ARG, what);
    if (reinterpret_cast<uintptr_t>(t->p) % (dt == HLA_F32 ? 4 : 2))
        return report(HLA_ERR_ARG, "a tensor is not aligned to its elements");
    if (t->sb < 0 || t->sh < 0 || t->st < 0) return report(HLA_ERR_ARG, "strides must not be negative");
    if ((double)t->sb * (s.B - 1) + (double)t->sh * (s.H - 1) + (double)t->st * (s.n - 1) + s.w > 4e18)
        return report(HLA_ERR_ARG, "a tensor is too large");
    return HLA_OK;
}
// The rows of an output share no memory: taken from the smallest stride up, each stride
// passes what lies inside it.
inline hla_status check_out(const hla_tensor *t, Dims s, hla_dtype dt, const char *what) {
    hla_status r = check_in(t, s, dt, what);
    if (r != HLA_OK) return r;
    long long st[3] = {t->st, t->sh, t->sb}, n[3] = {s.n, s.H, s.B}, inside = s.w;
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (st[j] < st[i]) {
                const long long x = st[i], y = n[i];
                st[i] = st[j]; n[i] = n[j];
                st[j] = x; n[j] = y;
            }
    for (int i = 0; i < 3; ++i) {
        if (n[i] <= 1) continue;
        if (st[i] < inside) return report(HLA_ERR_ARG, "rows of an output overlap");
        inside += st[i] * (n[i] - 1);
    }
    return HLA_OK;
}

// Every row on a 16-byte boundary.
inline bool rows16(const View &v, size_t element) {
    return (reinterpret_cast<uintptr_t>(v.p) & 15u) == 0 && v.sb * element % 16 == 0 && v.sh * element % 16 == 0 &&
           v.st * element % 16 == 0;
}

}  // namespace hla
