// layer_kernels.hpp -- dropout, and layer norm of residual + dropout(x) with
// its gradients.
//
// Dropout.  Row r, element j: block j / 8 of the row's stream (the sampler's
// generator with the top bit of the block's number set, which the sampler
// never reaches) holds 128 bits, and element j has its 16 bits number j % 8,
// the low half of a word first.  It is dropped if they are below `share`, and
// else multiplied by 65536 / (65536 - share).  A chunk of eight elements is one
// block, wherever it is computed: the mask is a function of (seed, row, j) alone
// and is never stored.  16 bits an element instead of 32 halve the generator's
// work, which would otherwise be more than the memory's where little is moved
// (50176x768 fp16, out = dropout(x): 28.4 us against 37.6; with a residual 36.8
// / 38.5, 4099x5003 bf16 17.7 / 21.1); a probability is then a multiple of 1/65536.
//
// Layer norm of one row:
//   h = RN_T(residual + dropout(x))
//   mean = sum h / D,  rstd = 1 / sqrt(sum (h - mean)^2 / D + eps)
//   out_j = RN_T((h_j - mean) rstd w_j + b_j)
// The squares are those of the deviations, in a second pass over the row, which
// is in registers: no digits cancel, whatever the mean.
//
// Every element is read once and written once (rows of more than 32,768
// elements, 16,384 of the gradients and of fp32, are read again from the caches or
// memory): the kernels are bound by memory, small calls by their launches.
// Measured on 50176x768 fp16 with a residual and dropout: dropout 37 us, 6.2 TB/s
// of what it must move; layer norm 56 us, 5.5 TB/s; its gradients 77 us, 5.0 TB/s
// (16384x4096 bf16 91 us).  fp32 of 3001x2243 11.7 us; one row of 4096 bf16 8 us.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

#include "fn_device.hpp"
#include "row_kernels.hpp"

namespace fn {

struct Dropout {
  uint64_t seed;
  uint64_t first_row;
  uint32_t share;  // of 65536
  float scale;     // of what is kept
};

// Chunk `chunk` of a row after dropout.
__device__ __forceinline__ void drop_chunk(float (&v)[8], const Dropout& d, uint64_t row,
                                           int32_t chunk) {
  const Block4 b =
      stream_block(d.seed, d.first_row + row, (uint64_t)1 << 63 | (uint64_t)(uint32_t)chunk);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t bits = j & 1 ? b.w[j >> 1] >> 16 : b.w[j >> 1] & 0xFFFFu;
    v[j] = bits < d.share ? 0.0f : v[j] * d.scale;
  }
}

// ------------------------------------------------------------------ dropout

struct DropoutArgs {
  const void* x;
  const void* residual;  // or null
  void* out;
  int64_t x_stride, residual_stride, out_stride;  // in elements
  Dropout drop;
  uint32_t items;   // rows * chunks of this launch
  Division chunks;  // of a row
  int32_t width;
};

// A thread takes one chunk of eight elements.
template <typename T, bool kShort>
__global__ __launch_bounds__(256) void dropout_kernel(DropoutArgs a) {
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  if (i >= a.items) return;
  const uint32_t row = quotient(i, a.chunks);
  const int32_t chunk = (int32_t)(i - row * a.chunks.by);
  const Chunk c = chunk_at(chunk, a.width);
  Vec8<T> x, r;
  load_chunk<kShort>(x, (const T*)a.x + (int64_t)row * a.x_stride, c);
  if (a.residual != nullptr)
    load_chunk<kShort>(r, (const T*)a.residual + (int64_t)row * a.residual_stride, c);
  trim_chunk<kShort>(x, c);
  float t[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) t[j] = x.get(j);
  drop_chunk(t, a.drop, row, chunk);
  if (a.residual != nullptr) {
    trim_chunk<kShort>(r, c);
#pragma unroll
    for (int j = 0; j < 8; ++j) t[j] += r.get(j);
  }
  x.set(t);
  store_chunk(x, (T*)a.out + (int64_t)row * a.out_stride, c);
}

// --------------------------------------------------------------- layer norm

struct LayerArgs {
  const void* x;
  const void* residual;  // or null
  const void* weight;    // or null: ones
  const void* bias;      // or null: zeros
  void* sum;             // null without a residual and dropout
  void* out;
  float* mean;  // or null
  float* rstd;  // or null
  int64_t rows;
  int64_t x_stride, residual_stride, sum_stride, out_stride;  // in elements
  Dropout drop;
  int32_t width;
  float eps;
  bool dropping;
};

// kCount sums over the kThreads threads of a row, as row_reduce: `parity`
// alternates between calls.
template <int kThreads, int kCount>
__device__ __forceinline__ void row_sums(float (&v)[kCount], int parity) {
#pragma unroll
  for (int k = 0; k < kCount; ++k) v[k] = group_sum<kThreads>(v[k]);
  if constexpr (kThreads > 64) {
    constexpr int kWaves = kThreads / 64;
    __shared__ float s_sum[2][kWaves][kCount];
    const int wave = (int)(threadIdx.x >> 6);
    if ((threadIdx.x & 63u) == 0) {
#pragma unroll
      for (int k = 0; k < kCount; ++k) s_sum[parity][wave][k] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kCount; ++k) {
      v[k] = s_sum[parity][0][k];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) v[k] += s_sum[parity][w][k];
    }
  }
}

// The chunk's numbers, as if they changed here: the compiler would compute a
// mask for each element of a row once, before the loop over the rows, keep them
// in scalar registers and spill those.
__device__ __forceinline__ void forget(Chunk& c) {
  asm("" : "+v"(c.at), "+v"(c.skip), "+v"(c.left));
}

// A chunk of the weight (ones without one) or the bias (zeros).
template <bool kShort, typename T>
__device__ __forceinline__ void load_affine(Vec8<T>& v, const void* from, float without,
                                            const Chunk& c) {
  if (from != nullptr) {
    load_chunk<kShort>(v, (const T*)from, c);
  } else {
    const float t[8] = {without, without, without, without, without, without, without, without};
    v.set(t);
  }
}

// Sum of (h - mean)^2 over a chunk's elements in the row.
template <typename T>
__device__ __forceinline__ float deviation_squares(const Vec8<T>& h, const Chunk& c, float mean) {
  float d[8], sum = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) d[j] = h.get(j) - mean;
#pragma unroll
  for (int j = 0; j < 8; ++j) d[j] = j < c.left ? d[j] : 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) sum += d[j] * d[j];
  return sum;
}

template <typename T>
__device__ __forceinline__ void normed_chunk(Vec8<T>& out, const Vec8<T>& h, const Vec8<T>& w,
                                             const Vec8<T>& b, float mean, float rstd) {
  float t[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) t[j] = (h.get(j) - mean) * rstd * w.get(j) + b.get(j);
  out.set(t);
}

// Threads and chunks of a row as in rows_kernel.
template <typename T, bool kDrop, int kThreads, int kChunks, bool kShort = false>
__global__ __launch_bounds__(rows_block<kThreads>()) void layer_norm_kernel(LayerArgs a) {
  constexpr int kRows = rows_block<kThreads>() / kThreads;
  // 128 registers a thread: weight and bias are read again for every row
  constexpr bool kAgain = kThreads == 1024;
  const int lane = (int)threadIdx.x % kThreads;
  const int slot = (int)threadIdx.x / kThreads;
  Chunk c[kChunks];
  Vec8<T> w[kAgain ? 1 : kChunks], b[kAgain ? 1 : kChunks];
#pragma unroll
  for (int k = 0; k < kChunks; ++k) {
    c[k] = chunk_at(k * kThreads + lane, a.width);
    if constexpr (!kAgain) {
      load_affine<kShort>(w[k], a.weight, 1.0f, c[k]);
      load_affine<kShort>(b[k], a.bias, 0.0f, c[k]);
    }
  }
  if constexpr (!kAgain) {
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
      trim_chunk<kShort>(w[k], c[k]);
      trim_chunk<kShort>(b[k], c[k]);
    }
  }
  const bool add = a.residual != nullptr;
  for (int64_t row = (int64_t)blockIdx.x * kRows + slot; row < a.rows;
       row += (int64_t)gridDim.x * kRows) {
#pragma unroll
    for (int k = 0; k < kChunks; ++k) forget(c[k]);
    const T* x = (const T*)a.x + row * a.x_stride;
    Vec8<T> h[kChunks];
#pragma unroll
    for (int k = 0; k < kChunks; ++k) load_chunk<kShort>(h[k], x, c[k]);
    Vec8<T> v[kChunks];
    if (add) {
      const T* r = (const T*)a.residual + row * a.residual_stride;
#pragma unroll
      for (int k = 0; k < kChunks; ++k) load_chunk<kShort>(v[k], r, c[k]);
    }
#pragma unroll
    for (int k = 0; k < kChunks; ++k) trim_chunk<kShort>(h[k], c[k]);
    if (add) {
#pragma unroll
      for (int k = 0; k < kChunks; ++k) trim_chunk<kShort>(v[k], c[k]);
    }
    if (a.sum != nullptr) {
      T* s = (T*)a.sum + row * a.sum_stride;
#pragma unroll
      for (int k = 0; k < kChunks; ++k) {
        float t[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) t[j] = h[k].get(j);
        if constexpr (kDrop) drop_chunk(t, a.drop, (uint64_t)row, k * kThreads + lane);
        if (add) {
#pragma unroll
          for (int j = 0; j < 8; ++j) t[j] += v[k].get(j);
        }
        h[k].set(t);
        store_chunk(h[k], s, c[k]);
      }
    }
    float total[1] = {0.0f};
#pragma unroll
    for (int k = 0; k < kChunks; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) total[0] += h[k].get(j);
    row_sums<kThreads>(total, 0);
    const float mean = total[0] / (float)a.width;
    float squares[1] = {0.0f};
#pragma unroll
    for (int k = 0; k < kChunks; ++k) squares[0] += deviation_squares(h[k], c[k], mean);
    row_sums<kThreads>(squares, 1);
    const float rstd = row_rstd(squares[0], a.width, a.eps);
    if (lane == 0) {
      if (a.mean != nullptr) a.mean[row] = mean;
      if (a.rstd != nullptr) a.rstd[row] = rstd;
    }
    T* o = (T*)a.out + row * a.out_stride;
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
      if constexpr (kAgain) {
        load_affine<kShort>(w[0], a.weight, 1.0f, c[k]);
        load_affine<kShort>(b[0], a.bias, 0.0f, c[k]);
        trim_chunk<kShort>(w[0], c[k]);
        trim_chunk<kShort>(b[0], c[k]);
      }
      Vec8<T> y;
      normed_chunk(y, h[k], w[kAgain ? 0 : k], b[kAgain ? 0 : k], mean, rstd);
      store_chunk(y, o, c[k]);
    }
  }
}

// Rows of any width from 8 on, one work-group of 1,024 threads each, which
// reads a row three times (from the stored sum where there is one).  A thread
// meets the same columns every time, so it may store over what it reads.
template <typename T>
__global__ __launch_bounds__(1024) void layer_norm_wide_kernel(LayerArgs a) {
  constexpr int kThreads = 1024;
  const int lane = (int)threadIdx.x;
  const int32_t chunks = (int32_t)(((int64_t)a.width + 7) / 8);
  const bool add = a.residual != nullptr;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = (const T*)a.x + row * a.x_stride;
    const T* r = add ? (const T*)a.residual + row * a.residual_stride : nullptr;
    T* s = a.sum != nullptr ? (T*)a.sum + row * a.sum_stride : nullptr;
    float total[1] = {0.0f};
    for (int32_t i = lane; i < chunks; i += kThreads) {
      const Chunk c = chunk_at(i, a.width);
      Vec8<T> h, v;
      load_chunk<false>(h, x, c);
      if (add) load_chunk<false>(v, r, c);
      trim_chunk<false>(h, c);
      if (s != nullptr) {
        float t[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) t[j] = h.get(j);
        if (a.dropping) drop_chunk(t, a.drop, (uint64_t)row, i);
        if (add) {
          trim_chunk<false>(v, c);
#pragma unroll
          for (int j = 0; j < 8; ++j) t[j] += v.get(j);
        }
        h.set(t);
        store_chunk(h, s, c);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) total[0] += h.get(j);
    }
    row_sums<kThreads>(total, 0);
    const float mean = total[0] / (float)a.width;
    const T* from = s != nullptr ? s : x;
    float squares[1] = {0.0f};
    for (int32_t i = lane; i < chunks; i += kThreads) {
      const Chunk c = chunk_at(i, a.width);
      Vec8<T> h;
      load_chunk<false>(h, from, c);
      trim_chunk<false>(h, c);
      squares[0] += deviation_squares(h, c, mean);
    }
    row_sums<kThreads>(squares, 1);
    const float rstd = row_rstd(squares[0], a.width, a.eps);
    if (lane == 0) {
      if (a.mean != nullptr) a.mean[row] = mean;
      if (a.rstd != nullptr) a.rstd[row] = rstd;
    }
    for (int32_t i = lane; i < chunks; i += kThreads) {
      const Chunk c = chunk_at(i, a.width);
      Vec8<T> h, w, b;
      load_chunk<false>(h, from, c);
      load_affine<false>(w, a.weight, 1.0f, c);
      load_affine<false>(b, a.bias, 0.0f, c);
      trim_chunk<false>(h, c);
      trim_chunk<false>(w, c);
      trim_chunk<false>(b, c);
      normed_chunk(h, h, w, b, mean, rstd);
      store_chunk(h, (T*)a.out + row * a.out_stride, c);
    }
  }
}

// ----------------------------------------------------------------- backward
//
// With n = (h - mean) rstd and g = dout w:
//   dh = rstd (g - mean(g) - n mean(g n)) [+ dsum],  dx = dropout(dh),
//   dweight = sum over rows of dout n,  dbias = sum over rows of dout.

struct LayerBackwardArgs {
  const void* dout;
  const void* h;
  const void* weight;  // or null: ones
  const float* mean;
  const float* rstd;
  const void* dsum;  // or null
  void* dh;
  void* dx;  // null without dropout
  // sums of dout n and of dout, one row of each per work-group (or slice);
  // null: not wanted
  float* partial_weight;
  float* partial_bias;
  float* row_means;  // rows that do not fit in registers: mean(g), mean(g n)
  int64_t rows;
  int64_t dout_stride, h_stride, dsum_stride, dh_stride, dx_stride;  // in elements
  int64_t rows_per_slice;
  Dropout drop;
  int32_t width;
  int32_t partials;
  int32_t pitch;  // width rounded up to whole vectors of four
};

template <bool kDrop, typename T>
__device__ __forceinline__ void layer_backward_chunk(const LayerBackwardArgs& a, int64_t row,
                                                     int32_t chunk, const Chunk& c,
                                                     const Vec8<T>& d, const Vec8<T>& h,
                                                     const Vec8<T>& w, const Vec8<T>& s, float mean,
                                                     float rstd, float mean_g, float mean_gn) {
  float t[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float n = (h.get(j) - mean) * rstd;
    t[j] = rstd * (d.get(j) * w.get(j) - mean_g - n * mean_gn) + s.get(j);
  }
  Vec8<T> out;
  out.set(t);
  store_chunk(out, (T*)a.dh + row * a.dh_stride, c);
  if constexpr (kDrop) {
    drop_chunk(t, a.drop, (uint64_t)row, chunk);
    out.set(t);
    store_chunk(out, (T*)a.dx + row * a.dx_stride, c);
  }
}

// Layout of threads and rows as in rows_backward_kernel: a work-group takes
// every gridDim.x-th group of rows and keeps its columns' sums in registers
// until the end.
template <typename T, bool kDrop, int kThreads, int kChunks, bool kShort = false>
__global__ __launch_bounds__(rows_block<kThreads>()) void layer_norm_backward_kernel(
    LayerBackwardArgs a) {
  constexpr int kRows = rows_block<kThreads>() / kThreads;
  const int lane = (int)threadIdx.x % kThreads;
  const int slot = (int)threadIdx.x / kThreads;
  Chunk c[kChunks];
  Vec8<T> w[kChunks];
  float sums[2][kChunks][8];
#pragma unroll
  for (int k = 0; k < kChunks; ++k) {
    c[k] = chunk_at(k * kThreads + lane, a.width);
    load_affine<kShort>(w[k], a.weight, 1.0f, c[k]);
#pragma unroll
    for (int j = 0; j < 8; ++j) sums[0][k][j] = sums[1][k][j] = 0.0f;
  }
#pragma unroll
  for (int k = 0; k < kChunks; ++k) trim_chunk<kShort>(w[k], c[k]);
  const bool add = a.dsum != nullptr;
  // the next row is on its way while this one is worked on, where there are
  // registers for both
  constexpr bool kAhead = kChunks <= 3;
  struct Row {
    Vec8<T> d[kChunks], h[kChunks], s[kChunks];
    float mean, rstd;
  };
  auto load = [&](Row& r, int64_t row) {
    const T* pd = (const T*)a.dout + row * a.dout_stride;
    const T* ph = (const T*)a.h + row * a.h_stride;
    r.mean = a.mean[row];
    r.rstd = a.rstd[row];
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
      load_chunk<kShort>(r.d[k], pd, c[k]);
      load_chunk<kShort>(r.h[k], ph, c[k]);
    }
    if (add) {
      const T* ps = (const T*)a.dsum + row * a.dsum_stride;
#pragma unroll
      for (int k = 0; k < kChunks; ++k) load_chunk<kShort>(r.s[k], ps, c[k]);
    } else {
#pragma unroll
      for (int k = 0; k < kChunks; ++k) r.s[k].zero();
    }
  };
  const int64_t step = (int64_t)gridDim.x * kRows;
  int64_t row = (int64_t)blockIdx.x * kRows + slot;
  Row next;
  if (kAhead && row < a.rows) load(next, row);
  for (int parity = 0; row < a.rows; row += step, parity ^= 1) {
#pragma unroll
    for (int k = 0; k < kChunks; ++k) forget(c[k]);
    Row now;
    if constexpr (kAhead) {
      now = next;
      if (row + step < a.rows) load(next, row + step);
    } else {
      load(now, row);
    }
    auto &d = now.d, &h = now.h, &s = now.s;
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
      trim_chunk<kShort>(d[k], c[k]);
      trim_chunk<kShort>(h[k], c[k]);
      if (add) trim_chunk<kShort>(s[k], c[k]);
    }
    float total[2] = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float n = (h[k].get(j) - now.mean) * now.rstd, g = d[k].get(j) * w[k].get(j);
        sums[0][k][j] += d[k].get(j) * n;
        sums[1][k][j] += d[k].get(j);
        total[0] += g;
        total[1] += g * n;
      }
    }
    row_sums<kThreads>(total, parity);
    const float mean_g = total[0] / (float)a.width, mean_gn = total[1] / (float)a.width;
#pragma unroll
    for (int k = 0; k < kChunks; ++k)
      layer_backward_chunk<kDrop>(a, row, k * kThreads + lane, c[k], d[k], h[k], w[k], s[k],
                                  now.mean, now.rstd, mean_g, mean_gn);
  }
  if constexpr (kRows > 1) {
    // the work-group's rows of sums, the upper half onto the lower until one
    // is left
    __shared__ float s_sums[kRows / 2][8 * kChunks][kThreads];
#pragma unroll 1
    for (int half = kRows / 2; half > 0; half /= 2) {
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        if (slot >= half && slot < 2 * half) {
#pragma unroll
          for (int k = 0; k < kChunks; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j) s_sums[slot - half][8 * k + j][lane] = sums[which][k][j];
        }
        __syncthreads();
        if (slot < half) {
#pragma unroll
          for (int k = 0; k < kChunks; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j) sums[which][k][j] += s_sums[slot][8 * k + j][lane];
        }
        __syncthreads();
      }
    }
    if (slot > 0) return;
  }
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float* p = which == 0 ? a.partial_weight : a.partial_bias;
    if (p == nullptr) continue;
    p += (int64_t)blockIdx.x * a.pitch;
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
      Vec8<float> v;
      v.set(sums[which][k]);
      store_chunk(v, p, c[k]);
    }
  }
}

// Rows of any width from 8 on, first step: mean(g) and mean(g n) of each row.
template <typename T>
__global__ __launch_bounds__(1024) void layer_norm_backward_means_kernel(LayerBackwardArgs a) {
  const int32_t chunks = (int32_t)(((int64_t)a.width + 7) / 8);
  int parity = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, parity ^= 1) {
    const T* pd = (const T*)a.dout + row * a.dout_stride;
    const T* ph = (const T*)a.h + row * a.h_stride;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float total[2] = {0.0f, 0.0f};
    for (int32_t i = (int32_t)threadIdx.x; i < chunks; i += 1024) {
      const Chunk c = chunk_at(i, a.width);
      Vec8<T> d, h, w;
      load_chunk<false>(d, pd, c);
      load_chunk<false>(h, ph, c);
      load_affine<false>(w, a.weight, 1.0f, c);
      trim_chunk<false>(d, c);
      trim_chunk<false>(h, c);
      trim_chunk<false>(w, c);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float g = d.get(j) * w.get(j);
        total[0] += g;
        total[1] += g * ((h.get(j) - mean) * rstd);
      }
    }
    row_sums<1024>(total, parity);
    if (threadIdx.x == 0) {
      a.row_means[2 * row] = total[0] / (float)a.width;
      a.row_means[2 * row + 1] = total[1] / (float)a.width;
    }
  }
}

// Second step: a thread takes eight columns of a slice of the rows.
template <typename T, bool kDrop>
__global__ __launch_bounds__(256) void layer_norm_backward_columns_kernel(LayerBackwardArgs a) {
  const int32_t chunks = (int32_t)(((int64_t)a.width + 7) / 8);
  const int32_t i = (int32_t)(blockIdx.x * 256u + threadIdx.x);
  if (i >= chunks) return;
  const Chunk c = chunk_at(i, a.width);
  const int64_t first = (int64_t)blockIdx.y * a.rows_per_slice;
  const int64_t end = min(first + a.rows_per_slice, a.rows);
  Vec8<T> w;
  load_affine<false>(w, a.weight, 1.0f, c);
  trim_chunk<false>(w, c);
  float sums[2][8] = {};
  for (int64_t row = first; row < end; ++row) {
    Vec8<T> d, h, s;
    load_chunk<false>(d, (const T*)a.dout + row * a.dout_stride, c);
    load_chunk<false>(h, (const T*)a.h + row * a.h_stride, c);
    s.zero();
    if (a.dsum != nullptr) load_chunk<false>(s, (const T*)a.dsum + row * a.dsum_stride, c);
    trim_chunk<false>(d, c);
    trim_chunk<false>(h, c);
    trim_chunk<false>(s, c);
    const float mean = a.mean[row], rstd = a.rstd[row];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      sums[0][j] += d.get(j) * ((h.get(j) - mean) * rstd);
      sums[1][j] += d.get(j);
    }
    layer_backward_chunk<kDrop>(a, row, i, c, d, h, w, s, mean, rstd, a.row_means[2 * row],
                                a.row_means[2 * row + 1]);
  }
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float* p = which == 0 ? a.partial_weight : a.partial_bias;
    if (p == nullptr) continue;
    Vec8<float> v;
    v.set(sums[which]);
    store_chunk(v, p + (int64_t)blockIdx.y * a.pitch, c);
  }
}

// dweight (blockIdx.y = 0) and dbias (1) from their partial rows; null: not
// wanted.
static __global__ __launch_bounds__(1024) void two_column_sums_kernel(
    const float* partial_weight, const float* partial_bias, int32_t partials, int32_t pitch,
    int32_t width, float* dweight, float* dbias) {
  float* to = blockIdx.y == 0 ? dweight : dbias;
  if (to != nullptr)
    column_sum(blockIdx.y == 0 ? partial_weight : partial_bias, partials, pitch, width, to);
}

}  // namespace fn
