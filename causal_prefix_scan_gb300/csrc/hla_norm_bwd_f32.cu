// hla_norm_bwd_f32.cu -- backward of the grouped norm, fp32 tensors.
#include "hla_norm_bwd.cuh"

void hla::norm::backward_f32(const Args &a, bool wide, cudaStream_t st) { backward<float>(a, wide, st); }
