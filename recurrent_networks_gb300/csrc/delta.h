// Host side of the gated delta rule's kernels: sizes and launchers.
#pragma once
#include <cuda_runtime.h>

#include "delta.cuh"

namespace rnn {

// Columns of v that one chain of chunks carries: 64 or, where half of the SMs
// would be without a chain then, v has no more, or keys past 128 channels leave
// no shared memory for it, 32. fp32: 32.
inline int delta_bv(bool bf, int B, int N, int Dv, int KP, int sms) {
  if (!bf || KP > 128 || Dv <= 32) return 32;
  return (long long)B * N * ((Dv + 63) / 64) * 2 < sms ? 32 : 64;
}

struct DeltaTcArgs;
cudaError_t delta_fwd_launch(const DeltaArgs& a, cudaStream_t st);  // fp32
cudaError_t delta_bwd_launch(const DeltaArgs& a, cudaStream_t st);
cudaError_t delta_tc_fwd_launch(int BV, const DeltaTcArgs& a, cudaStream_t st);  // bf16
cudaError_t delta_tc_bwd_launch(int BV, const DeltaTcArgs& a, cudaStream_t st);

}  // namespace rnn
