// kd_ops.h -- what the operator sources share on the host side. Internal to libkd.
#pragma once

#include <cuda_runtime.h>

namespace kd {
// The status word of kd_gemm.cu / kd_attention.cu, which is cleared.
int gemm_status(cudaStream_t s, unsigned int* st);
int attention_status(cudaStream_t s, unsigned int* st);
}  // namespace kd
