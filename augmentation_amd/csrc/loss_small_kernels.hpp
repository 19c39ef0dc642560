// loss_small_kernels.hpp -- what the linear cross entropy does around its
// products: joining a row's statistics, the scale of fp16 gradients, the
// rounding of sums and the copies of operands that lie off 16 bytes.
#pragma once
#include <hip/hip_runtime.h>

#include "loss_kernels.hpp"

namespace fn {

struct JoinArgs {
  const f32x2* stats;
  const float* sums;  // or null
  const float* target_z;
  const int64_t* targets;
  float* losses;
  float* lse;
  int64_t rows, classes;
  int64_t tiles;
  float smoothing;
};

// A row's tiles joined: a wavefront per row.
__global__ __launch_bounds__(256) void loss_join_kernel(JoinArgs p) {
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int lane = (int)(threadIdx.x & 63u);
  if (row >= p.rows) return;
  const f32x2* from = p.stats + row * p.tiles;
  const float* sums = p.sums != nullptr ? p.sums + row * p.tiles : nullptr;
  // four tiles at a time, their loads together; a tile without anything has
  // maximum -infinity and sum 0 (or NaN, which stays)
  float top = kMinusInfinity, sum = 0.0f, all = 0.0f;
  for (int64_t i = lane; i < p.tiles; i += 256) {
    f32x2 v[4];
    float s[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool there = i + 64 * j < p.tiles;
      v[j] = there ? from[i + 64 * j] : f32x2{kMinusInfinity, 0.0f};
      s[j] = there && sums != nullptr ? sums[i + 64 * j] : 0.0f;
    }
    const float higher = fmaxf(fmaxf(fmaxf(v[0][0], v[1][0]), fmaxf(v[2][0], v[3][0])), top);
    const float base = higher == kMinusInfinity ? 0.0f : higher;
    sum *= exp_below(top - base);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      sum += v[j][1] * exp_below(v[j][0] - base);
      all += s[j];
    }
    top = higher;
  }
  auto bits = [](float x) { return __builtin_bit_cast(uint32_t, x); };
  const float higher = __builtin_bit_cast(
      float, group_fold<64>(bits(top), [&](uint32_t x, uint32_t y) {
        return bits(fmaxf(__builtin_bit_cast(float, x), __builtin_bit_cast(float, y)));
      }));
  sum = group_sum<64>(sum * exp_below(top - (higher == kMinusInfinity ? 0.0f : higher)));
  top = higher;
  all = group_sum<64>(all);
  if (lane != 0) return;
  const int64_t y = p.targets[row];
  const bool counts = y >= 0 && y < p.classes;
  const LossOf l =
      loss_of(top, sum, all, counts, counts ? p.target_z[row] : 0.0f, p.smoothing);
  p.lse[row] = l.lse;
  p.losses[row] = l.loss;
}

// find_scale's numbers for many rows, which not every work-group shall read.
__global__ __launch_bounds__(1024) void loss_scale_kernel(const float* dlosses, int64_t stride,
                                                          const int64_t* targets, int64_t classes,
                                                          int64_t rows, float to, float* scale) {
  __shared__ uint32_t s_top[16];
  const Scale s = find_scale<1024>(dlosses, stride, targets, classes, rows, to, s_top);
  if (threadIdx.x != 0) return;
  scale[0] = s.up;
  scale[1] = s.down;
}

// out = RN_T(scale[1] * the sum of `splits` products in fp32): a thread takes
// four elements of a row.
template <typename T>
__global__ __launch_bounds__(256) void loss_round_kernel(const float* sums, int64_t pitch,
                                                         int64_t split_stride, int splits,
                                                         uint32_t items, Division vectors,
                                                         int32_t width, const float* scale, T* out,
                                                         int64_t out_stride) {
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  if (i >= items) return;
  const uint32_t m = quotient(i, vectors);
  const int32_t n = 4 * (int32_t)(i - m * vectors.by);
  const float by = scale != nullptr ? scale[1] : 1.0f;
  const float* from = sums + m * pitch + n;
  f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 16
  for (int s = 0; s < splits; ++s) v += *reinterpret_cast<const f32x4*>(from + s * split_stride);
  T* to = out + m * out_stride + n;
#pragma unroll
  for (int c = 0; c < 4; ++c)
    if (n + c < width) {
      if constexpr (sizeof(T) == 4)
        to[c] = v[c] * by;
      else
        reinterpret_cast<uint16_t*>(to)[c] = (uint16_t)two_halves<T>(v[c] * by, 0.0f);
    }
}

// A copy of an operand: rows of any alignment to rows of whole 16-byte pieces, zeros
// at their ends; fp32 in three parts (see Fp32Parts).
struct Copy {
  const void* from;
  int64_t stride;  // in elements
  void* to;
  int64_t part;     // in elements
  uint32_t items;   // pieces of this launch
  Division pieces;  // of a row
  int32_t width;
};

template <typename T>
__device__ __forceinline__ void copy_piece(const Copy& a, uint32_t i) {
  using Element = typename HeadType<T>::Operand;
  using Given = typename HeadType<T>::Output;
  constexpr int kE = 16 / (int)sizeof(Element);
  const uint32_t m = quotient(i, a.pieces);
  const int32_t c = kE * (int32_t)(i - m * a.pieces.by);
  const Given* row = (const Given*)a.from + m * a.stride + c;
  Element* to = (Element*)a.to + (int64_t)i * kE;
  if constexpr (HeadType<T>::kPasses > 1) {
    Vec8<float> v;
    if (c + 8 <= a.width)
      v.load(row);
    else
      v.load_some(row, a.width - c);
    float left[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) left[j] = v.get(j);
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      u32x4 w;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t lo = float_to_bf16(left[2 * j]), hi = float_to_bf16(left[2 * j + 1]);
        w[j] = lo | hi << 16;
        left[2 * j] -= bf16_to_float(lo);
        left[2 * j + 1] -= bf16_to_float(hi);
      }
      *reinterpret_cast<u32x4*>(to + k * a.part) = w;
    }
  } else {
    u32x4 v = {0, 0, 0, 0};
    if (c + kE <= a.width) {
      v = *reinterpret_cast<const u32x4_any*>(row);
    } else {
#pragma unroll
      for (int j = 0; j < kE; ++j)
        if (c + j < a.width) {
          if constexpr (sizeof(Given) == 4)
            v[j] = __builtin_bit_cast(uint32_t, row[j]);
          else
            v[j >> 1] |= (uint32_t)__builtin_bit_cast(uint16_t, row[j]) << (16 * (j & 1));
        }
    }
    *reinterpret_cast<u32x4*>(to) = v;
  }
}

// Both operands' copies in one launch (a's work-groups first): a thread takes a
// piece.
template <typename T>
__global__ __launch_bounds__(256) void loss_copy_kernel(Copy a, Copy b) {
  const uint32_t groups = (a.items + 255u) / 256u;
  if (blockIdx.x < groups) {
    const uint32_t i = blockIdx.x * 256u + threadIdx.x;
    if (i < a.items) copy_piece<T>(a, i);
  } else {
    const uint32_t i = (blockIdx.x - groups) * 256u + threadIdx.x;
    if (i < b.items) copy_piece<T>(b, i);
  }
}

}  // namespace fn
