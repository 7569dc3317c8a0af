// hla_norm_fwd_f32.cu -- forward of the grouped norm, fp32 tensors.
#include "hla_norm_fwd.cuh"

void hla::norm::forward_f32(const Args &a, bool wide, cudaStream_t st) { forward<float>(a, wide, st); }
