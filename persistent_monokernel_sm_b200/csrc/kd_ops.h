// kd_ops.h -- what the operator sources share on the host side. Internal to libkd.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "kd.h"

namespace kd {
// What a call's device-side waits go by: their limit in SM clocks, and the control words of the
// handle whose kd_sync reports one that runs out (NULL: kd_op_sync does).
struct OpWaits {
    long long limit;
    unsigned long long* ctl;
};
// SM clocks run at less than two a nanosecond.
inline long long op_clocks(long long ns) { return 2 * (ns < (1ll << 61) ? ns : 1ll << 61); }
// The operators as kd_prefill calls them.
int linear_op(const kd_linear_args* args, const OpWaits& waits, cudaStream_t stream);
int gated_op(const kd_gated_args* args, void* h, int64_t ld_h, const OpWaits& waits, cudaStream_t stream);
int attention_op(const kd_attention_args* args, const OpWaits& waits, cudaStream_t stream);
// Of the calling thread's own operator calls.
OpWaits own_waits();
// The status word of kd_gemm.cu / kd_attention.cu, which is cleared.
int gemm_status(cudaStream_t s, unsigned int* st);
int attention_status(cudaStream_t s, unsigned int* st);
// The most that kd_prompt_attention needs of a workspace: 148 tiles of 128 rows.
constexpr size_t kAttnPartBytes = (size_t)148 * 128 * (128 + 4) * 4 + 256;
}  // namespace kd
