// loss_fp16.hip -- the linear cross entropy's large kernels for fp16 operands.
#include "loss_launch.hpp"

namespace fn {

template <>
void launch_head<_Float16>(int output, bool across_a, HeadLaunch l, hipStream_t st) {
  launch_head_any<_Float16>(output, across_a, l, st);
}

template <>
void launch_head_pair<_Float16>(HeadPairArgs p, int tile, hipStream_t st) {
  launch_head_pair_any<_Float16>(p, tile, st);
}

}  // namespace fn
