// loss_fp32.hip -- the linear cross entropy's large kernels for fp32 operands.
#include "loss_launch.hpp"

namespace fn {

template <>
void launch_head<float>(int output, bool across_a, HeadLaunch l, hipStream_t st) {
  launch_head_any<float>(output, across_a, l, st);
}

template <>
void launch_head_pair<float>(HeadPairArgs p, int tile, hipStream_t st) {
  launch_head_pair_any<float>(p, tile, st);
}

}  // namespace fn
