// q8_api.hip -- the C ABI of the 8-bit linear layer's operators: argument
// checks, the choice of kernel and the launches.  Declarations, argument
// meaning, layouts and error behaviour are documented in include/fn.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "fn.h"
#include "fn_host.hpp"
#include "fn_rows_host.hpp"
#include "product_kernels.hpp"
#include "row_kernels.hpp"

namespace {

using namespace fnhost;

// ------------------------------------------------------------- row kernels

// Whether many wide fp32 rows are read past the caches: 2^23 elements and more (few
// rows stay in the memory-side cache: gradients of 500x8192 16.8 us past it, 15.7),
// by the threads of a row and how many of them are at work.  In us, past the caches /
// through them:
//   gradients  512x2 (rows to 8,192) 8192x8192 150 / 175, 9000x6720 142 / 159,
//              8192x8185 162 / 173; 256x3 (to 6,144) 12000x5120 140 / 147,
//              11000x6001 160 / 166, but 16384x4100 173 / 165; 256x2 and 512x4 (to
//              4,096 and 16,384) on whole cache lines 16384x4096 with dsum 202 / 214,
//              4096x16384 165 / 183, but 16384x4095 166 / 155, 4096x13440 142 / 138;
//   codes      256x2 to 512x2 on whole lines 16384x4096 56 / 59, 8192x8192 55.6 / 59.2,
//              but 16384x4100 63.5 / 57.5, 4096x14336 55 / 53;
//   norms with a residual  512x4 4096x16384 205 / 247, 4096x15001 196 / 205, but
//              6000x12288 228 / 215; 1024x4 2000x32768 227 / 246.
// All others are faster through the caches, norms by up to a third.
bool many_rows(int64_t rows, int32_t width) { return rows >= ((int64_t)1 << 23) / width; }

// Whether a matrix's rows are whole cache lines (or there is none).
bool on_lines(const void* p, int64_t stride, int64_t e) {
  return p == nullptr || ((uintptr_t)p | (uint64_t)(stride * e)) % 128 == 0;
}

template <int kMode, int kThreads, int kChunks>
bool once_rows(const fn::RowArgs& a) {
  if (!many_rows(a.rows, a.width)) return false;
  if constexpr (kMode == fn::kRowQuantize) return on_lines(a.x, a.x_stride, 4);
  return a.residual != nullptr && a.width >= (kThreads == 1024 ? 0 : 7 * kThreads * kChunks);
}

template <int kThreads, int kChunks>
bool once_backward(const fn::BackwardArgs& a) {
  if (!many_rows(a.rows, a.width)) return false;
  if (kThreads == 512 && kChunks == 2) return true;
  if (kThreads == 256 && kChunks == 3) return a.width >= 5 * 8 * 256 * 3 / 6;
  return a.width >= 7 * kThreads * kChunks && on_lines(a.dout, a.dout_stride, 4) &&
         on_lines(a.h, a.h_stride, 4) && on_lines(a.dsum, a.dsum_stride, 4);
}

template <typename T, int kMode, int kThreads, int kChunks, bool kShort = false>
void launch_rows_k(const fn::RowArgs& a, hipStream_t st) {
  constexpr int kBlock = fn::rows_block<kThreads>(), kRows = kBlock / kThreads;
  const int64_t groups = (a.rows + kRows - 1) / kRows;
  const unsigned grid = (unsigned)std::min<int64_t>(groups, 1 << 20);
  // codes 256x2 to 512x2, norms 512x4 and 1024x4
  constexpr bool kMayBeOnce =
      sizeof(T) == 4 &&
      ((kMode == fn::kRowQuantize && kThreads >= 256 && kThreads * kChunks <= 1024) ||
       (kMode == fn::kRowNorm && kThreads * kChunks >= 2048));
  if constexpr (kMayBeOnce) {
    if (once_rows<kMode, kThreads, kChunks>(a)) {
      fn::rows_kernel<T, kMode, kThreads, kChunks, kShort, true><<<grid, kBlock, 0, st>>>(a);
      return;
    }
  }
  fn::rows_kernel<T, kMode, kThreads, kChunks, kShort><<<grid, kBlock, 0, st>>>(a);
}

template <typename T, int kMode>
void launch_rows(const fn::RowArgs& a, hipStream_t st) {
  const RowShape s = row_shape(a.width, 32768);
  switch (shape_key(s.threads, s.chunks)) {
    case shape_key(1, 0): return launch_rows_k<T, kMode, 1, 1, true>(a, st);
    case shape_key(1, 1): return launch_rows_k<T, kMode, 1, 1>(a, st);
    case shape_key(2, 1): return launch_rows_k<T, kMode, 2, 1>(a, st);
    case shape_key(4, 1): return launch_rows_k<T, kMode, 4, 1>(a, st);
    case shape_key(8, 1): return launch_rows_k<T, kMode, 8, 1>(a, st);
    case shape_key(16, 1): return launch_rows_k<T, kMode, 16, 1>(a, st);
    case shape_key(16, 2): return launch_rows_k<T, kMode, 16, 2>(a, st);
    case shape_key(32, 2): return launch_rows_k<T, kMode, 32, 2>(a, st);
    case shape_key(32, 3): return launch_rows_k<T, kMode, 32, 3>(a, st);
    case shape_key(64, 2): return launch_rows_k<T, kMode, 64, 2>(a, st);
    case shape_key(64, 3): return launch_rows_k<T, kMode, 64, 3>(a, st);
    case shape_key(64, 4): return launch_rows_k<T, kMode, 64, 4>(a, st);
    case shape_key(64, 5): return launch_rows_k<T, kMode, 64, 5>(a, st);
    case shape_key(256, 2): return launch_rows_k<T, kMode, 256, 2>(a, st);
    case shape_key(256, 3): return launch_rows_k<T, kMode, 256, 3>(a, st);
    case shape_key(512, 2): return launch_rows_k<T, kMode, 512, 2>(a, st);
    case shape_key(512, 4):
      // rows of 16 bits have registers for half the threads (12000x12344 to
      // codes: 214 us against 260)
      if constexpr (sizeof(T) == 2)
        return launch_rows_k<T, kMode, 256, 8>(a, st);
      else
        return launch_rows_k<T, kMode, 512, 4>(a, st);
    // 128 registers a thread: fp32 rows to codes spill 8 of them
    case shape_key(1024, 4): return launch_rows_k<T, kMode, 1024, 4>(a, st);
    default:
      fn::rows_wide_kernel<T, kMode>
          <<<(unsigned)std::min<int64_t>(a.rows, 1 << 20), 1024, 0, st>>>(a);
  }
}

template <int kMode>
int launch_rows_type(const fn::RowArgs& a, int32_t dtype, void* stream) {
  hipStream_t st = (hipStream_t)stream;
  if (dtype == FN_OUT_FP32)
    launch_rows<float, kMode>(a, st);
  else if (dtype == FN_OUT_FP16)
    launch_rows<_Float16, kMode>(a, st);
  else
    launch_rows<fn::BF16, kMode>(a, st);
  return launch_status("rows_kernel launch");
}

// Both norms: out_dev (the input's type) or codes_dev and scales_dev.
template <int kMode>
int norm(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
         const void* weight, int64_t rows, int32_t width, float eps, int32_t dtype, void* sum,
         int64_t sum_stride, void* out, int64_t out_stride, float* scales, float* rstd,
         void* stream) {
  constexpr bool kQ8 = kMode == fn::kRowNormQ8;
  FN_TRY(check_size(rows, width));
  FN_TRY(check_type(dtype, "dtype"));
  if (!(eps > 0.0f && eps <= 3.4028234e38f))
    return fail(FN_EINVAL, "eps must be positive and finite");
  if ((residual == nullptr) != (sum == nullptr))
    return fail(FN_EINVAL, "residual_dev and sum_dev come together or not at all");
  const int64_t e = type_bytes(dtype), with_sum = residual != nullptr ? rows : 0;
  // an output of the input's type may replace x or the residual: a thread
  // has read its elements of a row before it writes them
  const Buffer buffers[] = {
      {"x_dev", x, rows, width, x_stride, e, false},
      {"residual_dev", residual, with_sum, width, residual_stride, e, false},
      {"weight_dev", weight, rows ? 1 : 0, width, 0, e, false},
      {"sum_dev", sum, with_sum, width, sum_stride, e, true, 3u},
      {kQ8 ? "codes_dev" : "out_dev", out, rows, width, out_stride, kQ8 ? 1 : e, true,
       kQ8 ? 0u : 3u},
      {"scales_dev", scales, kQ8 && rows ? 1 : 0, rows, 0, 4, true},
      {"rstd_dev", rstd, rstd != nullptr && rows ? 1 : 0, rows, 0, 4, true},
  };
  int dev = -1;
  FN_TRY(check_buffers(buffers, &dev));
  if (rows == 0) return ok();
  fn::RowArgs a{};
  a.x = x;
  a.residual = residual;
  a.weight = weight;
  a.sum = sum;
  a.out = kQ8 ? nullptr : out;
  a.codes = kQ8 ? (int8_t*)out : nullptr;
  a.scales = scales;
  a.rstd = rstd;
  a.rows = rows;
  a.x_stride = x_stride;
  a.residual_stride = residual_stride;
  a.sum_stride = sum_stride;
  a.out_stride = a.codes_stride = out_stride;
  a.width = width;
  a.eps = eps;
  return launch_rows_type<kMode>(a, dtype, stream);
}

// Work-groups of the backward kernels, each with one row of partial sums: two
// for each unit of a 256-unit device for rows of up to 1,024 elements, one for
// wider ones (measured for 256 / 512 / 1,024 partial rows, with their sum, in
// us: 50176x768 - / 59 / 61, 30000x1500 68 / 72 / 77, 8192x4096 50 / 53 / 62,
// 16384x8192 176 / 180 / -, 4099x5003 47 / 48 / 57).  A function of the sizes
// alone, so that results do not depend on the device.
struct BackwardPlan {
  RowShape shape;
  int32_t partials, pitch;
  int64_t rows_per_slice;
  int64_t bytes;
  bool direct;
};

BackwardPlan plan_backward(int64_t rows, int32_t width) {
  BackwardPlan p{};
  p.shape = row_shape(width, 16384);
  p.pitch = (width + 3) / 4 * 4;
  if (p.shape.threads > 0) {
    const int64_t at_once = p.shape.threads <= 64 ? 256 / p.shape.threads : 1;
    const int64_t groups = (rows + at_once - 1) / at_once;
    // one work-group per compute unit, or two where registers hold both and
    // one alone leaves lanes idle (us with 256 / 512 work-groups: 10000x2816 52 /
    // 47, 40000x3328 187 / 175, 10000x3840 57 / 57, 40000x4096 206 / 221) and rows
    // are enough to pay for the longer sum of partial rows (3000x3328 22.7 / 23.2)
    const bool idle = width > 2560 && width <= 3584 && rows >= 6000;
    p.partials = (int32_t)std::min<int64_t>(groups, width <= 1024 || idle ? 512 : 256);
    // so few rows that one work-group's sums are the gradient: it does two
    // groups of rows in less time than the second launch takes
    p.direct = groups == 1 || groups == 2;
    if (p.direct) p.partials = 1;
    p.bytes = p.direct ? 0 : (int64_t)p.partials * p.pitch * 4;
    return p;
  }
  const int64_t slices = std::min<int64_t>(rows, 64);
  p.rows_per_slice = slices ? (rows + slices - 1) / slices : 0;
  p.partials = slices ? (int32_t)((rows + p.rows_per_slice - 1) / p.rows_per_slice) : 0;
  p.bytes = ((int64_t)p.partials * p.pitch * 4 + rows * 4 + 15) / 16 * 16;
  return p;
}

template <typename T, int kThreads, int kChunks, bool kShort = false>
void launch_backward_k(const fn::BackwardArgs& a, hipStream_t st) {
  constexpr int kBlock = fn::rows_block<kThreads>();
  const unsigned grid = (unsigned)a.partials;
  if constexpr (sizeof(T) == 4 && kThreads >= 256) {
    if (once_backward<kThreads, kChunks>(a)) {
      fn::rows_backward_kernel<T, kThreads, kChunks, kShort, true><<<grid, kBlock, 0, st>>>(a);
      return;
    }
  }
  fn::rows_backward_kernel<T, kThreads, kChunks, kShort><<<grid, kBlock, 0, st>>>(a);
}

template <typename T>
void launch_backward(const fn::BackwardArgs& a, const RowShape& s, hipStream_t st) {
  switch (shape_key(s.threads, s.chunks)) {
    case shape_key(1, 0): return launch_backward_k<T, 1, 1, true>(a, st);
    case shape_key(1, 1): return launch_backward_k<T, 1, 1>(a, st);
    case shape_key(2, 1): return launch_backward_k<T, 2, 1>(a, st);
    case shape_key(4, 1): return launch_backward_k<T, 4, 1>(a, st);
    case shape_key(8, 1): return launch_backward_k<T, 8, 1>(a, st);
    case shape_key(16, 1): return launch_backward_k<T, 16, 1>(a, st);
    case shape_key(16, 2): return launch_backward_k<T, 16, 2>(a, st);
    case shape_key(32, 2): return launch_backward_k<T, 32, 2>(a, st);
    case shape_key(32, 3): return launch_backward_k<T, 32, 3>(a, st);
    case shape_key(64, 2): return launch_backward_k<T, 64, 2>(a, st);
    case shape_key(64, 3): return launch_backward_k<T, 64, 3>(a, st);
    case shape_key(64, 4): return launch_backward_k<T, 64, 4>(a, st);
    case shape_key(64, 5): return launch_backward_k<T, 64, 5>(a, st);
    case shape_key(256, 2): return launch_backward_k<T, 256, 2>(a, st);
    case shape_key(256, 3): return launch_backward_k<T, 256, 3>(a, st);
    case shape_key(512, 2): return launch_backward_k<T, 512, 2>(a, st);
    case shape_key(512, 4): return launch_backward_k<T, 512, 4>(a, st);
    default: {
      fn::rows_backward_mean_kernel<T>
          <<<(unsigned)std::min<int64_t>(a.rows, 1 << 20), 1024, 0, st>>>(a);
      const unsigned columns = blocks_for(((int64_t)a.width + 7) / 8, 256);
      fn::rows_backward_columns_kernel<T>
          <<<dim3(columns, (unsigned)a.partials), 256, 0, st>>>(a);
    }
  }
}

// Tiles of kBM tokens x kBN channels: the grid.
template <int kBM, int kBN>
unsigned tile_grid(fn::ProductArgs* p) {
  const int64_t tm = (p->M + kBM - 1) / kBM, tn = (p->N + kBN - 1) / kBN;
  p->tiles_m = (uint32_t)tm;
  p->tiles_n = (uint32_t)tn;
  return (unsigned)(tm * tn);
}

// The time of a product in tiles, in relative units: `first` and `each` for
// every tile on the busiest of `cus` compute units, or `alone` where none has
// a second.
double tile_cost(int64_t M, int64_t N, int bm, int bn, int cus, double alone, double first,
                 double each) {
  const double n = std::ceil((double)((M + bm - 1) / bm) * (double)((N + bn - 1) / bn) / cus);
  return n <= 1.0 ? alone : first + n * each;
}

template <typename T, int kBM, int kBN, int kWM, int kWN, int kStages, bool kLines = true>
void launch_tiles(fn::ProductArgs& p, hipStream_t st) {
  const unsigned grid = tile_grid<kBM, kBN>(&p);
  fn::product_tile_kernel<T, kBM, kBN, kWM, kWN, kStages, kLines>
      <<<grid, 64 * kWM * kWN, 0, st>>>(p);
}

// The cheapest of the four tiles for M tokens, and its cost.
int best_tile(int64_t M, int64_t N, int cus, double* cost) {
  const double c[4] = {tile_cost(M, N, 256, 256, cus, 57, 0, 57),
                       tile_cost(M, N, 128, 128, cus, 22.7, 0, 17.3),
                       tile_cost(M, N, 128, 64, cus, 14.8, 0, 10.3),
                       tile_cost(M, N, 64, 64, cus, 8.9, 3.5, 6.3)};
  const int best = (int)(std::min_element(c, c + 4) - c);
  *cost = c[best];
  return best;
}

template <typename T>
void launch_tiles_of(int tile, fn::ProductArgs& p, hipStream_t st) {
  // Rows off the cache lines, in us as they are / by whole lines: 128x64 tiles,
  // 2048x2048x4112 31 / 25, 1536x1536x1600 12.5 / 11.8; 64x64, 1024x1024x8208
  // 21.4 / 19.7, 1999x1000x1008 8.2 / 7.8.  128x128 would need more
  // stages, and so a compute unit each: with four, 4096x2048x4112 45 / 42, but
  // 4090x2040x1040 18.6 / 19.7.
  const bool lines = ((uintptr_t)p.a | (uintptr_t)p.b | (uint64_t)p.a_stride |
                      (uint64_t)p.b_stride) % fn::kBK == 0;
  switch (tile) {
    case 0: return launch_tiles<T, 256, 256, 2, 4, 2>(p, st);
    case 1: return launch_tiles<T, 128, 128, 2, 2, 2>(p, st);
    case 2:
      return lines ? launch_tiles<T, 128, 64, 2, 2, 3>(p, st)
                   : launch_tiles<T, 128, 64, 2, 2, 3, false>(p, st);
    default:
      return lines ? launch_tiles<T, 64, 64, 2, 2, 4>(p, st)
                   : launch_tiles<T, 64, 64, 2, 2, 4, false>(p, st);
  }
}

// One launch, or two: the tokens that give every compute unit the same number
// of 256x256 tiles, and the rest in whatever tiles suit them, where that costs
// less than a last round of tiles on a few compute units (a launch is 4 us;
// costs are for K = 4096).
template <typename T>
void launch_tiles_best(fn::ProductArgs& p, int cus, hipStream_t st) {
  double cost = 0.0, rest_cost = 0.0;
  int tile = best_tile(p.M, p.N, cus, &cost);
  const int64_t tiles_n = (p.N + 255) / 256, rounds = p.M / 256 * tiles_n / cus;
  const int64_t head = tiles_n <= cus ? rounds * cus / tiles_n * 256 : 0;
  if (head > 0 && head < p.M) {
    const int rest = best_tile(p.M - head, p.N, cus, &rest_cost);
    if (rounds * 57 + rest_cost + 4.0 * 4096 / std::max(p.K, 64) < cost) {
      fn::ProductArgs first = p;
      first.M = head;
      launch_tiles_of<T>(0, first, st);
      p.a += head * p.a_stride;
      p.sa += head;
      p.out = (T*)p.out + head * p.out_stride;
      p.M -= head;
      tile = rest;
    }
  }
  launch_tiles_of<T>(tile, p, st);
}

template <typename T, int kBM, int kBN>
void launch_any(fn::ProductArgs& p, hipStream_t st) {
  const unsigned grid = tile_grid<kBM, kBN>(&p);
  // with fp32 outputs the 256x128 tiles spill 2 of their 256 registers
  fn::product_any_kernel<T, kBM, kBN, 4><<<grid, 512, 0, st>>>(p);
}

// Work-groups of 16 kNT channels x 16 kMT tokens.
template <typename T, int kMT, int kNT, bool kPieces>
void launch_split(const fn::ProductArgs& p, hipStream_t st) {
  const dim3 grid(blocks_for(p.N, 16 * kNT), blocks_for(p.M, 16 * kMT));
  if constexpr (kPieces)
    fn::product_split_kernel<T, kMT, kNT, 2, 8><<<grid, 512, 0, st>>>(p);
  else
    fn::product_split_any_kernel<T, kMT, kNT, 8><<<grid, 512, 0, st>>>(p);
}

// Which kernel.  Times in us, measured on 256 compute units.
//
// Few tokens: K divided between a work-group's wavefronts, for up to 16
// tokens (1x4096x4096 5.1 against 9.7 in 64x64 tiles, 8x8192x8192 13.2
// against 16.2), in groups of 16 channels as long as these give a compute
// unit at most two, else of 64 (16x16384x2048 6.4 against 8.7); and beyond 16
// tokens while 32x32 groups are no more than the compute units (64x4096x4096
// 7.7 against 9.7, 128x2048x8192 9.3 against 15.7; but with twice as many
// 48x8192x4096 12.8 against 9.8, 128x4096x4096 12.9 against 9.8).
//
// Else tiles: large ones move fewer bytes per product, small ones fill the
// device.  The costs are the times of K = 4096 for tiles of 256x256, 128x128,
// 128x64 and 64x64 with one (alone) or more to a compute unit: 8192^3 395 /
// 483 / 611 / 783; 4096^3 57 / 68 / 85 / 102; 4096x2048x4096 45 / 35 / 41 /
// 53; 256x8192x4096 42 / 25 / 14.8 / 16.6; 1024x1024x8192 74 / 42 / 23 / 17.7.
//
// Rows that start anywhere: groups of 32x16 take the place of 32x32
// (128x794x2502 6.1 against 7.7, 32x4096x4095 8.8 against 11.5); tiles of
// 256x128, 128x64 and 64x64: 4000x4000x4001 110 / 160 / 197; 1999x1000x1021
// 18.5 / 11.0 / 11.7; 300x1024x777 16.5 / 8.8 / 7.1.
template <typename T>
void launch_part(fn::ProductArgs p, int cus, hipStream_t st) {
  // whole 16-byte pieces from 16-byte aligned rows, a tile's rows within the
  // 31-bit offsets of its buffer resource
  const bool pieces = ((uintptr_t)p.a | (uintptr_t)p.b | (uint64_t)p.a_stride |
                       (uint64_t)p.b_stride | (uint64_t)p.K) % 16 == 0 &&
                      std::max(p.a_stride, p.b_stride) <= (0x7FFFFFF0 - 131072) / 256;
  const double groups = std::ceil(p.M / 32.0) * std::ceil(p.N / 32.0);
  if (p.M <= 16 && !pieces) {
    launch_split<T, 1, 1, false>(p, st);
  } else if (p.M <= 16 && (p.N + 15) / 16 <= 2 * cus) {
    launch_split<T, 1, 1, true>(p, st);
  } else if (p.M <= 16) {
    launch_split<T, 1, 4, true>(p, st);
  } else if (groups <= cus && pieces) {
    launch_split<T, 2, 2, true>(p, st);
  } else if (groups <= cus) {
    launch_split<T, 2, 1, false>(p, st);
  } else if (pieces) {
    launch_tiles_best<T>(p, cus, st);
  } else {
    const double c[3] = {tile_cost(p.M, p.N, 256, 128, cus, 60, 0, 55),
                         tile_cost(p.M, p.N, 128, 64, cus, 30, 0, 20),
                         tile_cost(p.M, p.N, 64, 64, cus, 20, 0, 12.3)};
    switch (std::min_element(c, c + 3) - c) {
      case 0: launch_any<T, 256, 128>(p, st); break;
      case 1: launch_any<T, 128, 64>(p, st); break;
      default: launch_any<T, 64, 64>(p, st);
    }
  }
}

// The whole product, in parts of fewer than 2^32 threads, which is what HIP
// takes in a launch: at most 2^26 channels (32 threads each in groups of 16
// channels x 16 tokens) and 2^22 tiles of 64x64 (512 threads each).
template <typename T>
int launch_product(const fn::ProductArgs& p, int cus, hipStream_t st) {
  const int64_t channels = std::min<int64_t>(p.N, (int64_t)1 << 26);
  const int64_t tokens = ((int64_t)1 << 22) / ((channels + 63) / 64) / 4 * 256;
  for (int64_t n = 0; n < p.N; n += channels)
    for (int64_t m = 0; m < p.M; m += tokens) {
      fn::ProductArgs part = p;
      part.a += m * p.a_stride;
      part.sa += m;
      part.b += n * p.b_stride;
      part.sb += n;
      if (p.bias != nullptr) part.bias += n;
      part.out = (T*)p.out + m * p.out_stride + n;
      part.M = std::min(tokens, p.M - m);
      part.N = std::min(channels, p.N - n);
      launch_part<T>(part, cus, st);
      FN_TRY(launch_status("product kernel launch"));
    }
  return ok();
}

}  // namespace

FN_EXPORT int fn_rms_norm(const void* x_dev, int64_t x_stride, const void* residual_dev,
                          int64_t residual_stride, const void* weight_dev, int64_t rows,
                          int32_t width, float eps, int32_t dtype, void* sum_dev,
                          int64_t sum_stride, void* out_dev, int64_t out_stride, float* rstd_dev,
                          void* stream) {
  return norm<fn::kRowNorm>(x_dev, x_stride, residual_dev, residual_stride, weight_dev, rows, width,
                            eps, dtype, sum_dev, sum_stride, out_dev, out_stride, nullptr, rstd_dev,
                            stream);
}

FN_EXPORT int fn_rms_norm_q8(const void* x_dev, int64_t x_stride, const void* residual_dev,
                             int64_t residual_stride, const void* weight_dev, int64_t rows,
                             int32_t width, float eps, int32_t dtype, void* sum_dev,
                             int64_t sum_stride, int8_t* codes_dev, int64_t codes_stride,
                             float* scales_dev, float* rstd_dev, void* stream) {
  return norm<fn::kRowNormQ8>(x_dev, x_stride, residual_dev, residual_stride, weight_dev, rows,
                              width, eps, dtype, sum_dev, sum_stride, codes_dev, codes_stride,
                              scales_dev, rstd_dev, stream);
}

FN_EXPORT int fn_quantize_rows(const void* x_dev, int64_t x_stride, int64_t rows, int32_t width,
                               int32_t dtype, int8_t* codes_dev, int64_t codes_stride,
                               float* scales_dev, void* stream) {
  FN_TRY(check_size(rows, width));
  FN_TRY(check_type(dtype, "dtype"));
  const int64_t e = type_bytes(dtype);
  const Buffer buffers[] = {
      {"x_dev", x_dev, rows, width, x_stride, e, false},
      {"codes_dev", codes_dev, rows, width, codes_stride, 1, true},
      {"scales_dev", scales_dev, rows ? 1 : 0, rows, 0, 4, true},
  };
  int dev = -1;
  FN_TRY(check_buffers(buffers, &dev));
  if (rows == 0) return ok();
  fn::RowArgs a{};
  a.x = x_dev;
  a.codes = codes_dev;
  a.scales = scales_dev;
  a.rows = rows;
  a.x_stride = x_stride;
  a.codes_stride = codes_stride;
  a.width = width;
  return launch_rows_type<fn::kRowQuantize>(a, dtype, stream);
}

FN_EXPORT int fn_rms_norm_backward_workspace(int64_t rows, int32_t width, int64_t* bytes) {
  FN_TRY(check_size(rows, width));
  if (bytes == nullptr) return fail(FN_EINVAL, "bytes is NULL");
  *bytes = plan_backward(rows, width).bytes;
  return ok();
}

FN_EXPORT int fn_rms_norm_backward(const void* dout_dev, int64_t dout_stride, const void* h_dev,
                                   int64_t h_stride, const void* weight_dev, const float* rstd_dev,
                                   const void* dsum_dev, int64_t dsum_stride, int64_t rows,
                                   int32_t width, int32_t dtype, void* dx_dev, int64_t dx_stride,
                                   float* dweight_dev, void* workspace_dev,
                                   int64_t workspace_bytes, void* stream) {
  FN_TRY(check_size(rows, width));
  FN_TRY(check_type(dtype, "dtype"));
  const BackwardPlan plan = plan_backward(rows, width);
  if (workspace_bytes < plan.bytes)
    return fail(FN_EINVAL, "workspace of %lld bytes, %lld needed", (long long)workspace_bytes,
                (long long)plan.bytes);
  const int64_t e = type_bytes(dtype);
  const Buffer buffers[] = {
      {"dout_dev", dout_dev, rows, width, dout_stride, e, false},
      {"h_dev", h_dev, rows, width, h_stride, e, false},
      {"dsum_dev", dsum_dev, dsum_dev != nullptr ? rows : 0, width, dsum_stride, e, false},
      {"weight_dev", weight_dev, rows ? 1 : 0, width, 0, e, false},
      {"rstd_dev", rstd_dev, rows ? 1 : 0, rows, 0, 4, false},
      {"dx_dev", dx_dev, rows, width, dx_stride, e, true, 7u},
      {"dweight_dev", dweight_dev, 1, width, 0, 4, true},
      {"workspace_dev", workspace_dev, plan.bytes ? 1 : 0, plan.bytes / 16, 0, 16, true},
  };
  int dev = -1;
  FN_TRY(check_buffers(buffers, &dev));
  fn::BackwardArgs a{};
  a.dout = dout_dev;
  a.h = h_dev;
  a.weight = weight_dev;
  a.rstd = rstd_dev;
  a.dsum = dsum_dev;
  a.dx = dx_dev;
  a.partial = plan.direct ? dweight_dev : (float*)workspace_dev;
  a.row_mean = (float*)workspace_dev + (int64_t)plan.partials * plan.pitch;
  a.rows = rows;
  a.dout_stride = dout_stride;
  a.h_stride = h_stride;
  a.dsum_stride = dsum_stride;
  a.dx_stride = dx_stride;
  a.rows_per_slice = plan.rows_per_slice;
  a.width = width;
  a.partials = plan.partials;
  a.pitch = plan.pitch;
  hipStream_t st = (hipStream_t)stream;
  if (rows > 0) {
    if (dtype == FN_OUT_FP32)
      launch_backward<float>(a, plan.shape, st);
    else if (dtype == FN_OUT_FP16)
      launch_backward<_Float16>(a, plan.shape, st);
    else
      launch_backward<fn::BF16>(a, plan.shape, st);
    FN_TRY(launch_status("rows_backward_kernel launch"));
    if (plan.direct) return ok();
  }
  // no rows: no partial sums, and a gradient of zero.  2^26 columns, 2^30
  // threads, to a launch: HIP takes fewer than 2^32 of them
  for (int32_t c = 0; c < width; c += kColumnsPerLaunch) {
    const int32_t columns = std::min(width - c, kColumnsPerLaunch);
    fn::column_sum_kernel<<<blocks_for(columns, 64), 1024, 0, st>>>(
        rows > 0 ? a.partial + c : nullptr, a.partials, a.pitch, columns, dweight_dev + c);
    FN_TRY(launch_status("column_sum_kernel launch"));
  }
  return ok();
}

FN_EXPORT int fn_matmul_q8(const int8_t* a_dev, int64_t a_stride, const float* a_scales_dev,
                           const int8_t* b_dev, int64_t b_stride, const float* b_scales_dev,
                           const float* bias_dev, int64_t M, int64_t N, int32_t K,
                           int32_t out_dtype, void* out_dev, int64_t out_stride, void* stream) {
  if (M < 0 || N < 0 || K < 0) return fail(FN_EINVAL, "M, N and K must be >= 0");
  if (K > 131071) return fail(FN_EOVERFLOW, "K = %d: sums fit 32 bits up to 131071", K);
  if (M > (int64_t)1 << 40 || N > (int64_t)1 << 40) return fail(FN_EOVERFLOW, "M or N exceeds 2^40");
  FN_TRY(check_type(out_dtype, "out_dtype"));
  const bool none = M == 0 || N == 0;
  const Buffer buffers[] = {
      {"a_dev", a_dev, none ? 0 : M, K, a_stride, 1, false},
      {"b_dev", b_dev, none ? 0 : N, K, b_stride, 1, false},
      {"a_scales_dev", a_scales_dev, none ? 0 : 1, M, 0, 4, false},
      {"b_scales_dev", b_scales_dev, none ? 0 : 1, N, 0, 4, false},
      {"bias_dev", bias_dev, none || bias_dev == nullptr ? 0 : 1, N, 0, 4, false},
      {"out_dev", out_dev, none ? 0 : M, N, out_stride, type_bytes(out_dtype), true},
  };
  int dev = -1;
  FN_TRY(check_buffers(buffers, &dev));
  if (none) return ok();
  fn::ProductArgs p{};
  p.a = a_dev;
  p.b = b_dev;
  p.sa = a_scales_dev;
  p.sb = b_scales_dev;
  p.bias = bias_dev;
  p.out = out_dev;
  p.a_stride = a_stride;
  p.b_stride = b_stride;
  p.out_stride = out_stride;
  p.M = M;
  p.N = N;
  p.K = K;
  hipStream_t st = (hipStream_t)stream;
  int cus = 0;
  FN_TRY(device_cu_count(dev, &cus));
  if (out_dtype == FN_OUT_FP32) return launch_product<float>(p, cus, st);
  if (out_dtype == FN_OUT_FP16) return launch_product<_Float16>(p, cus, st);
  return launch_product<fn::BF16>(p, cus, st);
}
