// hla_norm_bwd_bf16.cu -- backward of the grouped norm, bf16 tensors.
#include "hla_norm_bwd.cuh"

void hla::norm::backward_bf16(const Args &a, bool wide, cudaStream_t st) { backward<__nv_bfloat16>(a, wide, st); }
