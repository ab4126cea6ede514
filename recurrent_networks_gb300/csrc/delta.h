// Host side of the gated delta rule's kernels: sizes and launchers.
#pragma once
#include <cuda_runtime.h>

#include "delta.cuh"

namespace rnn {

// How a bf16 problem's chains of chunks are laid over the GPU: tiles of BV columns
// of v, and segments (delta_tc.cuh). A CTA an SM, so the time is the number of
// rounds that the CTAs take times the chunks of a segment; segments cost the pass
// of maps (the identity's tiles among them, forward) and the join. Microseconds a
// chunk as measured with all SMs taken: forward 4.8 (BV = 64) and 3.4 (32; 5.3 for
// keys past 128 channels), backward 6.2, 4.3 and 6.3; a join 4.2 a segment (11 for
// keys past 128), 15 a further launch.
struct DeltaLay {
  int BV, segs, seglen;
};
inline DeltaLay delta_lay(long long heads, int Dv, int KP, long long nc, int sms, bool keep) {
  DeltaLay best{32, 1, (int)(nc > 0 ? nc : 1)};
  double least = 1e300;
  for (int BV = 64; BV >= 32; BV -= 32) {
    if (BV == 64 && (KP > 128 || Dv <= 32)) continue;
    const double f = BV == 64 ? 4.8 : KP > 128 ? 5.3 : 3.4, w = keep ? (BV == 64 ? 6.2 : KP > 128 ? 6.3 : 4.3) : 0.0;
    const long long nvt = (Dv + BV - 1) / BV, ki = (KP + BV - 1) / BV;
    auto rounds = [&](long long ctas) { return (double)((ctas + sms - 1) / sms); };
    for (int segs = 1; segs <= 64; ++segs) {
      const long long len = ((nc + segs - 1) / segs + 7) / 8 * 8;
      if (segs > 1 && len * (segs - 1) >= nc) continue;  // a segment would be empty
      const double own = rounds(heads * segs * nvt) * (segs > 1 ? len : nc);
      double cost = own * (f + w);
      if (segs > 1)
        cost += rounds(heads * segs * (nvt + ki)) * len * f + own * w + ((KP > 128 ? 11.0 : 4.2) * segs + 30.0) * (keep ? 2 : 1);
      if (cost < least * 0.97) {
        least = cost;
        best = DeltaLay{BV, segs, (int)(segs > 1 ? len : (nc > 0 ? nc : 1))};
      }
    }
  }
  return best;
}

struct DeltaTcArgs;
cudaError_t delta_fwd_launch(const DeltaArgs& a, cudaStream_t st);  // fp32
cudaError_t delta_bwd_launch(const DeltaArgs& a, cudaStream_t st);
cudaError_t delta_tc_fwd_launch(int BV, const DeltaTcArgs& a, cudaStream_t st);  // bf16
cudaError_t delta_tc_bwd_launch(int BV, const DeltaTcArgs& a, cudaStream_t st);
cudaError_t delta_tc_join_back(int BV, const DeltaTcArgs& a, cudaStream_t st);

}  // namespace rnn
