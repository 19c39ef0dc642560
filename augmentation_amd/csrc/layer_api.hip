// layer_api.hip -- the C ABI of dropout and layer norm: argument checks, the
// choice of kernel and the launches.  Declarations, argument meaning, layouts
// and error behaviour are documented in include/fn.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "fn.h"
#include "fn_host.hpp"
#include "fn_rows_host.hpp"
#include "layer_kernels.hpp"

namespace {

using namespace fnhost;

// What a dropout probability, a seed and a first row stand for.
int dropout_of(float p, uint64_t seed, int64_t first_row, int64_t rows, fn::Dropout* d) {
  if (!in_unit(p)) return fail(FN_EINVAL, "dropout_p must lie in [0, 1]");
  if (first_row < 0) return fail(FN_EINVAL, "first_row must be >= 0");
  if (first_row > INT64_MAX - rows)
    return fail(FN_EOVERFLOW, "first_row + rows exceeds 2^63 - 1");
  d->seed = seed;
  d->first_row = (uint64_t)first_row;
  d->share = (uint32_t)std::nearbyint((double)p * 65536.0);
  d->scale = d->share < 65536 ? (float)(65536.0 / (65536.0 - d->share)) : 0.0f;
  return FN_OK;
}

// --------------------------------------------------------------- layer norm

template <typename T, bool kDrop, int kThreads, int kChunks, bool kShort = false>
void launch_norm_k(const fn::LayerArgs& a, hipStream_t st) {
  constexpr int kBlock = fn::rows_block<kThreads>(), kRows = kBlock / kThreads;
  const int64_t groups = (a.rows + kRows - 1) / kRows;
  fn::layer_norm_kernel<T, kDrop, kThreads, kChunks, kShort>
      <<<(unsigned)std::min<int64_t>(groups, 1 << 20), kBlock, 0, st>>>(a);
}

// The rows' shape, as the other norm's but for two: a second reduction and bias
// and mean beside the weight leave fewer wavefronts room (us with 64 / 128 threads
// a row: 3001x2243 fp32 12.5 / 10.9, 12000x2240 bf16 with a residual 48 / 43,
// 12000x2000 40 / 38; 12000x1500 31.2 / 31.5).  fp32 rows beyond 16,384 elements do
// not fit.
RowShape norm_shape(int32_t width, bool wide_type) {
  if (width > 1536 && width <= 2048) return {2048, 128, 2};
  if (width > 2048 && width <= 2560) return {2560, 128, 3};
  return row_shape(width, wide_type ? 16384 : 32768);
}

template <typename T, bool kDrop>
void launch_norm(const fn::LayerArgs& a, hipStream_t st) {
  const RowShape s = norm_shape(a.width, sizeof(T) == 4);
  switch (shape_key(s.threads, s.chunks)) {
    case shape_key(1, 0): return launch_norm_k<T, kDrop, 1, 1, true>(a, st);
    case shape_key(1, 1): return launch_norm_k<T, kDrop, 1, 1>(a, st);
    case shape_key(2, 1): return launch_norm_k<T, kDrop, 2, 1>(a, st);
    case shape_key(4, 1): return launch_norm_k<T, kDrop, 4, 1>(a, st);
    case shape_key(8, 1): return launch_norm_k<T, kDrop, 8, 1>(a, st);
    case shape_key(16, 1): return launch_norm_k<T, kDrop, 16, 1>(a, st);
    case shape_key(16, 2): return launch_norm_k<T, kDrop, 16, 2>(a, st);
    case shape_key(32, 2): return launch_norm_k<T, kDrop, 32, 2>(a, st);
    case shape_key(32, 3): return launch_norm_k<T, kDrop, 32, 3>(a, st);
    case shape_key(64, 2): return launch_norm_k<T, kDrop, 64, 2>(a, st);
    case shape_key(64, 3): return launch_norm_k<T, kDrop, 64, 3>(a, st);
    case shape_key(128, 2): return launch_norm_k<T, kDrop, 128, 2>(a, st);
    case shape_key(128, 3): return launch_norm_k<T, kDrop, 128, 3>(a, st);
    case shape_key(256, 2): return launch_norm_k<T, kDrop, 256, 2>(a, st);
    case shape_key(256, 3): return launch_norm_k<T, kDrop, 256, 3>(a, st);
    case shape_key(512, 2): return launch_norm_k<T, kDrop, 512, 2>(a, st);
    case shape_key(512, 4):
      // 6000x12344 bf16 with a residual: 141 us against 154; 3000x12344 fp32 126
      // against 119
      if constexpr (sizeof(T) == 2)
        return launch_norm_k<T, kDrop, 1024, 2>(a, st);
      else
        return launch_norm_k<T, kDrop, 512, 4>(a, st);
    case shape_key(1024, 4):
      if constexpr (sizeof(T) == 2) return launch_norm_k<T, kDrop, 1024, 4>(a, st);
    default:
      fn::layer_norm_wide_kernel<T>
          <<<(unsigned)std::min<int64_t>(a.rows, 1 << 20), 1024, 0, st>>>(a);
  }
}

template <bool kDrop>
void launch_norm_type(const fn::LayerArgs& a, int32_t dtype, hipStream_t st) {
  if (dtype == FN_OUT_FP32)
    launch_norm<float, kDrop>(a, st);
  else if (dtype == FN_OUT_FP16)
    launch_norm<_Float16, kDrop>(a, st);
  else
    launch_norm<fn::BF16, kDrop>(a, st);
}

// Work-groups of the backward kernel, each with a row of partial sums of either
// gradient; a function of the sizes alone, so that results do not depend on
// the device.
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
    p.partials = (int32_t)std::min<int64_t>(groups, width <= 1024 ? 512 : 256);
    // So few rows that one work-group's sums are the gradients: a few groups of
    // rows take it less time than the second launch does, which makes 12.4 us of
    // a call.  6 groups: 9.8 us at 512 to 4,096 columns (with one or two chunks
    // a thread), 13.6 at 2,048 (four), 17.2 at 2,560 (five; 3 groups 11.0), 11.9
    // at 8,192; 16,384 columns: 2 rows 9.8 (fp32 14.9), 3 rows 12.3 (19.4).
    const int most = width > 8192 ? 2 : std::min(6, 12 / std::max(1, p.shape.chunks));
    p.direct = groups >= 1 && groups <= most;
    if (p.direct) p.partials = 1;
    p.bytes = p.direct ? 0 : (int64_t)p.partials * p.pitch * 8;
    p.bytes = (p.bytes + 15) / 16 * 16;
    return p;
  }
  const int64_t slices = std::min<int64_t>(rows, 64);
  p.rows_per_slice = slices ? (rows + slices - 1) / slices : 0;
  p.partials = slices ? (int32_t)((rows + p.rows_per_slice - 1) / p.rows_per_slice) : 0;
  p.bytes = ((int64_t)p.partials * p.pitch * 8 + rows * 8 + 15) / 16 * 16;
  return p;
}

template <typename T, bool kDrop, int kThreads, int kChunks, bool kShort = false>
void launch_backward_k(const fn::LayerBackwardArgs& a, hipStream_t st) {
  fn::layer_norm_backward_kernel<T, kDrop, kThreads, kChunks, kShort>
      <<<(unsigned)a.partials, fn::rows_block<kThreads>(), 0, st>>>(a);
}

template <typename T, bool kDrop>
void launch_backward(const fn::LayerBackwardArgs& a, const RowShape& s, hipStream_t st) {
  switch (shape_key(s.threads, s.chunks)) {
    case shape_key(1, 0): return launch_backward_k<T, kDrop, 1, 1, true>(a, st);
    case shape_key(1, 1): return launch_backward_k<T, kDrop, 1, 1>(a, st);
    case shape_key(2, 1): return launch_backward_k<T, kDrop, 2, 1>(a, st);
    case shape_key(4, 1): return launch_backward_k<T, kDrop, 4, 1>(a, st);
    case shape_key(8, 1): return launch_backward_k<T, kDrop, 8, 1>(a, st);
    case shape_key(16, 1): return launch_backward_k<T, kDrop, 16, 1>(a, st);
    case shape_key(16, 2): return launch_backward_k<T, kDrop, 16, 2>(a, st);
    case shape_key(32, 2): return launch_backward_k<T, kDrop, 32, 2>(a, st);
    case shape_key(32, 3): return launch_backward_k<T, kDrop, 32, 3>(a, st);
    case shape_key(64, 2): return launch_backward_k<T, kDrop, 64, 2>(a, st);
    case shape_key(64, 3): return launch_backward_k<T, kDrop, 64, 3>(a, st);
    case shape_key(64, 4): return launch_backward_k<T, kDrop, 64, 4>(a, st);
    case shape_key(64, 5): return launch_backward_k<T, kDrop, 64, 5>(a, st);
    case shape_key(256, 2): return launch_backward_k<T, kDrop, 256, 2>(a, st);
    case shape_key(256, 3): return launch_backward_k<T, kDrop, 256, 3>(a, st);
    case shape_key(512, 2): return launch_backward_k<T, kDrop, 512, 2>(a, st);
    case shape_key(512, 4): return launch_backward_k<T, kDrop, 512, 4>(a, st);
    default: {
      fn::layer_norm_backward_means_kernel<T>
          <<<(unsigned)std::min<int64_t>(a.rows, 1 << 20), 1024, 0, st>>>(a);
      const unsigned columns = blocks_for(((int64_t)a.width + 7) / 8, 256);
      fn::layer_norm_backward_columns_kernel<T, kDrop>
          <<<dim3(columns, (unsigned)a.partials), 256, 0, st>>>(a);
    }
  }
}

template <bool kDrop>
void launch_backward_type(const fn::LayerBackwardArgs& a, const RowShape& s, int32_t dtype,
                          hipStream_t st) {
  if (dtype == FN_OUT_FP32)
    launch_backward<float, kDrop>(a, s, st);
  else if (dtype == FN_OUT_FP16)
    launch_backward<_Float16, kDrop>(a, s, st);
  else
    launch_backward<fn::BF16, kDrop>(a, s, st);
}

template <typename T>
void launch_dropout(const fn::DropoutArgs& a, hipStream_t st) {
  const unsigned grid = blocks_for(a.items, 256);
  if (a.width < 8)
    fn::dropout_kernel<T, true><<<grid, 256, 0, st>>>(a);
  else
    fn::dropout_kernel<T, false><<<grid, 256, 0, st>>>(a);
}

const void* rows_on(const void* p, int64_t rows, int64_t stride, int64_t e) {
  return p == nullptr ? nullptr : (const char*)p + rows * stride * e;
}

}  // namespace

FN_EXPORT int fn_dropout(const void* x_dev, int64_t x_stride, const void* residual_dev,
                         int64_t residual_stride, int64_t rows, int32_t width, float dropout_p,
                         uint64_t seed, int64_t first_row, int32_t dtype, void* out_dev,
                         int64_t out_stride, void* stream) {
  FN_TRY(check_size(rows, width));
  FN_TRY(check_type(dtype, "dtype"));
  fn::DropoutArgs a{};
  FN_TRY(dropout_of(dropout_p, seed, first_row, rows, &a.drop));
  const int64_t e = type_bytes(dtype);
  // out may replace an input: a thread has read its elements before it writes
  // them, and nobody else needs them
  const Buffer buffers[] = {
      {"x_dev", x_dev, rows, width, x_stride, e, false},
      {"residual_dev", residual_dev, residual_dev != nullptr ? rows : 0, width, residual_stride, e,
       false},
      {"out_dev", out_dev, rows, width, out_stride, e, true, 3u},
  };
  int dev = -1;
  FN_TRY(check_buffers(buffers, &dev));
  if (rows == 0) return ok();
  a.x_stride = x_stride;
  a.residual_stride = residual_stride;
  a.out_stride = out_stride;
  a.width = width;
  const int64_t chunks = ((int64_t)width + 7) / 8;
  a.chunks = fn::division_by((uint32_t)chunks);
  // at most 2^31 threads to a launch
  const int64_t most = std::max<int64_t>(((int64_t)1 << 31) / chunks, 1);
  for (int64_t row = 0; row < rows; row += most) {
    const int64_t count = std::min(most, rows - row);
    a.x = rows_on(x_dev, row, x_stride, e);
    a.residual = rows_on(residual_dev, row, residual_stride, e);
    a.out = (void*)rows_on(out_dev, row, out_stride, e);
    a.items = (uint32_t)(count * chunks);
    if (dtype == FN_OUT_FP32)
      launch_dropout<float>(a, (hipStream_t)stream);
    else if (dtype == FN_OUT_FP16)
      launch_dropout<_Float16>(a, (hipStream_t)stream);
    else
      launch_dropout<fn::BF16>(a, (hipStream_t)stream);
    FN_TRY(launch_status("dropout_kernel launch"));
    a.drop.first_row += (uint64_t)count;
  }
  return ok();
}

FN_EXPORT int fn_layer_norm(const void* x_dev, int64_t x_stride, const void* residual_dev,
                            int64_t residual_stride, const void* weight_dev, const void* bias_dev,
                            int64_t rows, int32_t width, float eps, float dropout_p, uint64_t seed,
                            int64_t first_row, int32_t dtype, void* sum_dev, int64_t sum_stride,
                            void* out_dev, int64_t out_stride, float* mean_dev, float* rstd_dev,
                            void* stream) {
  FN_TRY(check_size(rows, width));
  FN_TRY(check_type(dtype, "dtype"));
  if (!(eps > 0.0f && eps <= 3.4028234e38f))
    return fail(FN_EINVAL, "eps must be positive and finite");
  fn::LayerArgs a{};
  FN_TRY(dropout_of(dropout_p, seed, first_row, rows, &a.drop));
  const bool summed = residual_dev != nullptr || dropout_p > 0.0f;
  if (rows > 0 && summed != (sum_dev != nullptr))
    return fail(FN_EINVAL, "sum_dev comes with residual_dev or dropout, and only then");
  const int64_t e = type_bytes(dtype), one = rows ? 1 : 0;
  const Buffer buffers[] = {
      {"x_dev", x_dev, rows, width, x_stride, e, false},
      {"residual_dev", residual_dev, residual_dev != nullptr ? rows : 0, width, residual_stride, e,
       false},
      {"weight_dev", weight_dev, weight_dev != nullptr ? one : 0, width, 0, e, false},
      {"bias_dev", bias_dev, bias_dev != nullptr ? one : 0, width, 0, e, false},
      {"sum_dev", sum_dev, summed ? rows : 0, width, sum_stride, e, true, 3u},
      {"out_dev", out_dev, rows, width, out_stride, e, true, 3u},
      {"mean_dev", mean_dev, mean_dev != nullptr ? one : 0, rows, 0, 4, true},
      {"rstd_dev", rstd_dev, rstd_dev != nullptr ? one : 0, rows, 0, 4, true},
  };
  int dev = -1;
  FN_TRY(check_buffers(buffers, &dev));
  if (rows == 0) return ok();
  a.x = x_dev;
  a.residual = residual_dev;
  a.weight = weight_dev;
  a.bias = bias_dev;
  a.sum = sum_dev;
  a.out = out_dev;
  a.mean = mean_dev;
  a.rstd = rstd_dev;
  a.rows = rows;
  a.x_stride = x_stride;
  a.residual_stride = residual_stride;
  a.sum_stride = sum_stride;
  a.out_stride = out_stride;
  a.width = width;
  a.eps = eps;
  a.dropping = dropout_p > 0.0f;
  hipStream_t st = (hipStream_t)stream;
  if (a.dropping)
    launch_norm_type<true>(a, dtype, st);
  else
    launch_norm_type<false>(a, dtype, st);
  return launch_status("layer_norm_kernel launch");
}

FN_EXPORT int fn_layer_norm_backward_workspace(int64_t rows, int32_t width, int64_t* bytes) {
  FN_TRY(check_size(rows, width));
  if (bytes == nullptr) return fail(FN_EINVAL, "bytes is NULL");
  *bytes = plan_backward(rows, width).bytes;
  return ok();
}

FN_EXPORT int fn_layer_norm_backward(
    const void* dout_dev, int64_t dout_stride, const void* h_dev, int64_t h_stride,
    const void* weight_dev, const float* mean_dev, const float* rstd_dev, const void* dsum_dev,
    int64_t dsum_stride, int64_t rows, int32_t width, float dropout_p, uint64_t seed,
    int64_t first_row, int32_t dtype, void* dh_dev, int64_t dh_stride, void* dx_dev,
    int64_t dx_stride, float* dweight_dev, float* dbias_dev, void* workspace_dev,
    int64_t workspace_bytes, void* stream) {
  FN_TRY(check_size(rows, width));
  FN_TRY(check_type(dtype, "dtype"));
  fn::LayerBackwardArgs a{};
  FN_TRY(dropout_of(dropout_p, seed, first_row, rows, &a.drop));
  if ((dropout_p > 0.0f) != (dx_dev != nullptr) && rows > 0)
    return fail(FN_EINVAL,
                "dx_dev comes with dropout, and only then (else dh is the gradient of x)");
  const BackwardPlan plan = plan_backward(rows, width);
  if (workspace_bytes < plan.bytes)
    return fail(FN_EINVAL, "workspace of %lld bytes, %lld needed", (long long)workspace_bytes,
                (long long)plan.bytes);
  const int64_t e = type_bytes(dtype), one = rows ? 1 : 0;
  const Buffer buffers[] = {
      {"dout_dev", dout_dev, rows, width, dout_stride, e, false},
      {"h_dev", h_dev, rows, width, h_stride, e, false},
      {"dsum_dev", dsum_dev, dsum_dev != nullptr ? rows : 0, width, dsum_stride, e, false},
      {"weight_dev", weight_dev, weight_dev != nullptr ? one : 0, width, 0, e, false},
      {"mean_dev", mean_dev, one, rows, 0, 4, false},
      {"rstd_dev", rstd_dev, one, rows, 0, 4, false},
      {"dh_dev", dh_dev, rows, width, dh_stride, e, true, 7u},
      {"dx_dev", dx_dev, dx_dev != nullptr ? rows : 0, width, dx_stride, e, true, 7u},
      {"dweight_dev", dweight_dev, dweight_dev != nullptr ? 1 : 0, width, 0, 4, true},
      {"dbias_dev", dbias_dev, dbias_dev != nullptr ? 1 : 0, width, 0, 4, true},
      {"workspace_dev", workspace_dev, plan.bytes ? 1 : 0, plan.bytes / 16, 0, 16, true},
  };
  int dev = -1;
  FN_TRY(check_buffers(buffers, &dev));
  const int64_t sums = (int64_t)plan.partials * plan.pitch;
  a.dout = dout_dev;
  a.h = h_dev;
  a.weight = weight_dev;
  a.mean = mean_dev;
  a.rstd = rstd_dev;
  a.dsum = dsum_dev;
  a.dh = dh_dev;
  a.dx = dx_dev;
  float* workspace = (float*)workspace_dev;
  if (dweight_dev != nullptr) a.partial_weight = plan.direct ? dweight_dev : workspace;
  if (dbias_dev != nullptr) a.partial_bias = plan.direct ? dbias_dev : workspace + sums;
  a.row_means = workspace + 2 * sums;
  a.rows = rows;
  a.dout_stride = dout_stride;
  a.h_stride = h_stride;
  a.dsum_stride = dsum_stride;
  a.dh_stride = dh_stride;
  a.dx_stride = dx_stride;
  a.rows_per_slice = plan.rows_per_slice;
  a.width = width;
  a.partials = plan.partials;
  a.pitch = plan.pitch;
  hipStream_t st = (hipStream_t)stream;
  if (rows > 0) {
    if (dropout_p > 0.0f)
      launch_backward_type<true>(a, plan.shape, dtype, st);
    else
      launch_backward_type<false>(a, plan.shape, dtype, st);
    FN_TRY(launch_status("layer_norm_backward_kernel launch"));
    if (plan.direct) return ok();
  }
  if (dweight_dev == nullptr && dbias_dev == nullptr) return ok();
  // no rows: no partial sums, and gradients of zero
  for (int32_t c = 0; c < width; c += kColumnsPerLaunch) {
    const int32_t columns = std::min(width - c, kColumnsPerLaunch);
    fn::two_column_sums_kernel<<<dim3(blocks_for(columns, 64), 2), 1024, 0, st>>>(
        rows > 0 && dweight_dev ? a.partial_weight + c : nullptr,
        rows > 0 && dbias_dev ? a.partial_bias + c : nullptr, rows > 0 ? a.partials : 0, a.pitch,
        columns, dweight_dev ? dweight_dev + c : nullptr, dbias_dev ? dbias_dev + c : nullptr);
    FN_TRY(launch_status("two_column_sums_kernel launch"));
  }
  return ok();
}
