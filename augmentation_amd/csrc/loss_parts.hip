// loss_parts.hip -- the linear cross entropy's large kernels for fp32 operands in
// three bf16 parts.
#include "loss_launch.hpp"

namespace fn {

template <>
void launch_head<Fp32Parts>(int output, bool across_a, HeadLaunch l, hipStream_t st) {
  launch_head_any<Fp32Parts>(output, across_a, l, st);
}

template <>
void launch_head_pair<Fp32Parts>(HeadPairArgs p, int tile, hipStream_t st) {
  launch_head_pair_any<Fp32Parts>(p, tile, st);
}

}  // namespace fn
