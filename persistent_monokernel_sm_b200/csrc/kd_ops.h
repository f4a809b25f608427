// kd_ops.h -- what the operator sources share on the host side. Internal to libkd.
#pragma once

#include <cuda_runtime.h>

namespace kd {
int gemm_status(cudaStream_t s, unsigned int* st);  // kd_gemm.cu's status word, cleared
}  // namespace kd
