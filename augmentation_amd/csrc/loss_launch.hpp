// loss_launch.hpp -- the launches of the linear cross entropy's large kernels.
// They are instantiated in a source file for each type, which compile side by
// side.
#pragma once
#include <hip/hip_runtime.h>

#include "loss_kernels.hpp"

namespace fn {

// Rows and columns of the tiles.
constexpr int kHeadTiles = 5;
constexpr int kHeadTileM[kHeadTiles] = {256, 128, 64, 16, 16};
constexpr int kHeadTileN[kHeadTiles] = {256, 128, 64, 64, 128};
// rows of wavefronts in a tile, each with a row of bias_sums
constexpr int kHeadTileRows[kHeadTiles] = {2, 2, 2, 1, 1};

struct HeadLaunch {
  HeadArgs args;
  int tile;    // which of the sizes
  int splits;  // of the contraction
};

// Whether a 16x64 tile's contraction is divided between groups: where no compute
// unit of 256 has a second tile, and it is long enough (512 elements of bf16 6.1
// us with one group, 6.5 with four; 1024 8.0 / 7.5).
inline bool in_groups(int tile, int64_t tiles, int64_t K) {
  return tile == 3 && tiles <= 256 && K >= 768;
}

template <typename T, int kOutput, bool kAcrossA, bool kAcrossB>
void launch_head_tiles(HeadLaunch& l, hipStream_t st) {
  HeadArgs& p = l.args;
  const int64_t m = kHeadTileM[l.tile], n = kHeadTileN[l.tile];
  p.tiles_m = (uint32_t)((p.M + m - 1) / m);
  p.tiles_n = (uint32_t)((p.N + n - 1) / n);
  const dim3 grid(p.tiles_m * p.tiles_n, (unsigned)l.splits);
  switch (l.tile) {
    case 0:
      head_kernel<T, kOutput, kAcrossA, kAcrossB, 256, 256, 2, 4, 2><<<grid, 512, 0, st>>>(p);
      break;
    case 1:
      head_kernel<T, kOutput, kAcrossA, kAcrossB, 128, 128, 2, 2, 2><<<grid, 256, 0, st>>>(p);
      break;
    case 2:
      head_kernel<T, kOutput, kAcrossA, kAcrossB, 64, 64, 2, 2, 4><<<grid, 256, 0, st>>>(p);
      break;
    // few rows, which only dw's operands do not have; or few tiles
    case 3:
      if constexpr (!kAcrossA) {
        if (in_groups(3, (int64_t)grid.x * grid.y, p.K_split))
          head_kernel<T, kOutput, kAcrossA, kAcrossB, 16, 64, 1, 4, 3, 4><<<grid, 1024, 0, st>>>(p);
        else
          head_kernel<T, kOutput, kAcrossA, kAcrossB, 16, 64, 1, 4, 4><<<grid, 256, 0, st>>>(p);
      }
      break;
    default:
      if constexpr (!kAcrossA)
        head_kernel<T, kOutput, kAcrossA, kAcrossB, 16, 128, 1, 4, 4><<<grid, 256, 0, st>>>(p);
  }
}

// `across_a`: how a lies in the products with g (dw: across, dx: along); b lies
// across in both, and both along in the logits.
template <typename T>
void launch_head(int output, bool across_a, HeadLaunch l, hipStream_t st);

// dx and dw, and dbias, in one launch of tiles of 128x128 or 64x64.
template <typename T>
void launch_head_pair(HeadPairArgs p, int tile, hipStream_t st);

template <typename T>
void launch_head_pair_any(HeadPairArgs& p, int tile, hipStream_t st) {
  const int64_t size = kHeadTileM[tile];
  for (HeadArgs* a : {&p.dx, &p.dw}) {
    a->tiles_m = (uint32_t)((a->M + size - 1) / size);
    a->tiles_n = (uint32_t)((a->N + size - 1) / size);
  }
  p.dx_blocks = p.dx.tiles_m * p.dx.tiles_n;
  p.dw_blocks = p.dw.tiles_m * p.dw.tiles_n;
  const unsigned grid = p.dx_blocks + p.dw_blocks +
                        (p.dbias != nullptr ? (unsigned)((p.dw.M + 63) / 64) : 0u);
  if (tile == 1)
    head_pair_kernel<T, 128, 128, 2, 2, 2><<<grid, 256, 0, st>>>(p);
  else
    head_pair_kernel<T, 64, 64, 2, 2, 4><<<grid, 256, 0, st>>>(p);
}

template <typename T>
void launch_head_any(int output, bool across_a, HeadLaunch& l, hipStream_t st) {
  if (output == kHeadStatistics)
    launch_head_tiles<T, kHeadStatistics, false, false>(l, st);
  else if (output == kHeadGradient)
    launch_head_tiles<T, kHeadGradient, false, false>(l, st);
  else if (output == kHeadRounded && !across_a)
    launch_head_tiles<T, kHeadRounded, false, true>(l, st);
  else if (output == kHeadRounded)
    launch_head_tiles<T, kHeadRounded, true, true>(l, st);
  else if (!across_a)
    launch_head_tiles<T, kHeadSums, false, true>(l, st);
  else
    launch_head_tiles<T, kHeadSums, true, true>(l, st);
}

}  // namespace fn
