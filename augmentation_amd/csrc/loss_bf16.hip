// loss_bf16.hip -- the linear cross entropy's large kernels for bf16 operands.
#include "loss_launch.hpp"

namespace fn {

template <>
void launch_head<BF16>(int output, bool across_a, HeadLaunch l, hipStream_t st) {
  launch_head_any<BF16>(output, across_a, l, st);
}

template <>
void launch_head_pair<BF16>(HeadPairArgs p, int tile, hipStream_t st) {
  launch_head_pair_any<BF16>(p, tile, st);
}

}  // namespace fn
