// Host side of the gated delta rule's kernels: sizes and launchers.
#pragma once
#include <cuda_runtime.h>

#include "delta.cuh"

namespace rnn {

// Columns of v that one chain of chunks carries: 64 or, where that would leave
// half of the SMs without a chain (or bf16 keys past 192 channels would not fit
// a chain's shared memory), 32. fp32: 32.
inline int delta_bv(bool bf, int B, int N, int Dv, int DKP, int sms) {
  if (!bf || DKP > 192) return 32;
  return (long long)B * N * ((Dv + 63) / 64) * 2 < sms ? 32 : 64;
}

cudaError_t delta_fwd_launch(bool bf, int BV, const DeltaArgs& a, cudaStream_t st);
cudaError_t delta_bwd_launch(bool bf, int BV, const DeltaArgs& a, cudaStream_t st);

}  // namespace rnn
