// hla_norm_fwd_bf16.cu -- forward of the grouped norm, bf16 tensors.
#include "hla_norm_fwd.cuh"

void hla::norm::forward_bf16(const Args &a, bool wide, cudaStream_t st) { forward<__nv_bfloat16>(a, wide, st); }
