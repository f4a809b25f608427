// kd_ops.h -- what the operator sources share on the host side. Internal to libkd.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace kd {
// The limit of device-side waits that the calling thread has set, in SM clocks.
long long op_limit();
// The status word of kd_gemm.cu / kd_attention.cu, which is cleared.
int gemm_status(cudaStream_t s, unsigned int* st);
int attention_status(cudaStream_t s, unsigned int* st);
// The most that kd_prompt_attention needs of a workspace: 148 tiles of 128 rows.
constexpr size_t kAttnPartBytes = (size_t)148 * 128 * (128 + 4) * 4 + 256;
}  // namespace kd
