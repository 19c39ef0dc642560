// loss_api.hip -- the C ABI of the linear cross entropy: argument checks, the
// plan of a call (pieces of the classes, tiles, splits, workspace) and the
// launches.  Declarations, argument meaning, layouts and error behaviour are
// documented in include/fn.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "fn.h"
#include "fn_host.hpp"
#include "fn_rows_host.hpp"
#include "loss_launch.hpp"
#include "loss_small_kernels.hpp"

namespace {

using namespace fnhost;

// Results shall not depend on the device, so neither may the choices that
// change an order of summation: they are made for these compute units.
constexpr int64_t kUnits = 256;
// Bytes of the gradient of the logits that a piece of the classes has: enough
// for every product to fill the device, few enough to stay in the memory-side
// cache until both products have read it.
constexpr int64_t kPieceBytes = (int64_t)1 << 27;
constexpr int32_t kMaxFeatures = 1 << 20;
constexpr int64_t kMaxClasses = (int64_t)1 << 28;
// a stage's rows times the stride within the 31-bit offsets of a resource
constexpr int64_t kMaxStrideBytes = ((int64_t)1 << 31) / 256 - 1;

struct Choice {
  int tile = 0, splits = 1;
  int64_t K_split = 0;
};

// The tile and the splits of the contraction for M x N outputs and K elements
// of it, by the time they would take (us; of a tile of 256, 128 or 64 rows, for
// 4,096 bytes of the contraction).
Choice choose(int64_t M, int64_t N, int64_t K, int64_t e, bool splittable) {
  const double each[3] = {e == 2 ? 57.0 : 220.0, e == 2 ? 17.3 : 56.0, e == 2 ? 6.3 : 14.5};
  const int64_t stage = fn::kStageRow / e;
  Choice best;
  double least = 1e300;
  for (int tile = 0; tile < 3; ++tile) {
    const int64_t size = fn::kHeadTileSizes[tile];
    const int64_t tiles = ((M + size - 1) / size) * ((N + size - 1) / size);
    if (tiles >= (int64_t)1 << 22) continue;  // 2^32 threads to a launch
    for (int splits = 1; splits <= 64; splits *= 2) {
      if (splits > 1 && (!splittable || K < 8 * stage * splits || tiles * splits > 4 * kUnits)) break;
      const int64_t K_split = ((K + splits - 1) / splits + stage - 1) / stage * stage;
      const double rounds = std::ceil((double)tiles * splits / kUnits);
      double cost = rounds * (each[tile] * K_split * e / 4096.0 + 1.5);
      // partial products are written and read again, in a launch of their own
      if (splits > 1) cost += 3.0 + (double)M * N * 8.0 * splits / 4e6;
      if (cost < least) {
        least = cost;
        best = {tile, splits, K_split};
      }
    }
  }
  best.K_split = std::max<int64_t>(best.K_split, stage);
  return best;
}

int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// Parts of a workspace, one behind the other.
struct Parts {
  int64_t bytes = 0;
  int64_t take(int64_t n) {
    const int64_t at = bytes;
    bytes += round_up(n, 256);
    return at;
  }
};

struct Plan {
  bool pack_x, pack_w;
  int64_t width_packed;  // elements
  int64_t piece;         // classes
  int64_t pieces;
  Choice logits, dx, dw;
  bool sum_dx, sum_dw;  // in fp32 first
  int64_t pitch;        // of g's rows, elements
  int64_t sum_pitch;    // of fp32 products' rows
  int64_t stat_tiles, bias_rows;
  // places in the workspace
  int64_t scale, x, w, stats, sums, target_z, g, dx_sums, dw_sums, bias_sums;
  int64_t bytes;
};

// `bytes` of a plan without some optional output is at most that of one with
// it.
Plan plan_of(int64_t rows, int64_t classes, int32_t width, int64_t e, bool pack_x, bool pack_w,
             bool backward) {
  Plan p{};
  p.pack_x = pack_x;
  p.pack_w = pack_w;
  p.width_packed = round_up(width, 16 / e);
  const int64_t per_class = std::max<int64_t>(rows, 1) * e;
  // what a piece of the classes has in the workspace: their gradients, or a
  // copy of their weights
  const int64_t piece_bytes =
      backward ? std::max(classes * per_class, pack_w ? classes * p.width_packed * e : 0)
               : (pack_w ? classes * p.width_packed * e : 0);
  p.pieces = std::max<int64_t>((piece_bytes + kPieceBytes - 1) / kPieceBytes, 1);
  p.piece = round_up((classes + p.pieces - 1) / p.pieces, 256);
  p.piece = std::min({classes, p.piece, kMaxStrideBytes / e / 256 * 256});
  p.pieces = (classes + p.piece - 1) / p.piece;
  const int64_t K = pack_x || pack_w ? p.width_packed : width;
  p.logits = choose(rows, p.piece, K, e, false);
  Parts parts;
  p.scale = parts.take(8);
  if (pack_x) p.x = parts.take(rows * p.width_packed * e);
  if (pack_w) p.w = parts.take(p.piece * p.width_packed * e);
  if (!backward) {
    const int64_t size = fn::kHeadTileSizes[p.logits.tile];
    // pieces are whole tiles, but for the last
    p.stat_tiles = (p.pieces - 1) * ((p.piece + size - 1) / size) +
                   (classes - (p.pieces - 1) * p.piece + size - 1) / size;
    p.stats = parts.take(rows * p.stat_tiles * 8);
    p.sums = parts.take(rows * p.stat_tiles * 4);
    p.target_z = parts.take(rows * 4);
  } else {
    const int64_t size = fn::kHeadTileSizes[p.logits.tile];
    p.pitch = round_up(p.piece, 64);
    p.sum_pitch = round_up(width, 4);
    p.dx = choose(rows, width, p.piece, e, true);
    p.dw = choose(p.piece, width, rows, e, true);
    p.sum_dx = p.pieces > 1 || p.dx.splits > 1;
    p.sum_dw = p.dw.splits > 1;
    p.bias_rows = (rows + size - 1) / size * fn::kHeadTileRows;
    p.g = parts.take(rows * p.pitch * e);
    if (p.sum_dx) p.dx_sums = parts.take(p.dx.splits * rows * p.sum_pitch * 4);
    if (p.sum_dw) p.dw_sums = parts.take(p.dw.splits * p.piece * p.sum_pitch * 4);
    p.bias_sums = parts.take(p.bias_rows * p.pitch * 4);
  }
  p.bytes = parts.bytes;
  return p;
}

int check_head(int64_t rows, int64_t classes, int32_t width, int32_t dtype) {
  if (rows < 0) return fail(FN_EINVAL, "rows must be >= 0");
  if (classes < 1) return fail(FN_EINVAL, "classes must be >= 1");
  if (width < 1) return fail(FN_EINVAL, "width must be >= 1 (got %d)", width);
  if (rows > (int64_t)1 << 28) return fail(FN_EOVERFLOW, "rows exceeds 2^28");
  if (classes > kMaxClasses) return fail(FN_EOVERFLOW, "classes exceeds 2^28");
  if (width > kMaxFeatures) return fail(FN_EOVERFLOW, "width %d exceeds 2^20", width);
  // so that every product has fewer than 2^22 tiles, and a launch 2^32 threads
  if (rows > ((int64_t)1 << 36) / classes || rows > ((int64_t)1 << 36) / width ||
      classes > ((int64_t)1 << 36) / width)
    return fail(FN_EOVERFLOW, "rows * classes, rows * width or classes * width exceeds 2^36");
  return check_type(dtype, "dtype");
}

// Rows that the kernels can read where they are.
bool in_place(const void* p, int64_t stride, int32_t width, int64_t e) {
  return ((uintptr_t)p | (uint64_t)(stride * e) | (uint64_t)(width * e)) % 16 == 0 &&
         stride >= width && stride * e <= kMaxStrideBytes;
}

// An operand of the call: where it lies, or its copy.
template <typename T>
fn::Operand operand(const void* from, int64_t stride, int64_t rows, int32_t width, int64_t copied,
                    char* copy, hipStream_t st) {
  constexpr int64_t e = sizeof(T);
  if (copy == nullptr) return {(const char*)from, stride * e, rows, (int64_t)width * e};
  if (rows > 0) {
    const dim3 grid(blocks_for(copied * e / 16, 256), (unsigned)std::min<int64_t>(rows, 65535));
    fn::loss_pack_kernel<T><<<grid, 256, 0, st>>>((const T*)from, stride, rows, width, (T*)copy,
                                                  (int32_t)copied);
  }
  return {copy, copied * e, rows, copied * e};
}

struct Call {
  const void* x;
  int64_t x_stride;
  const void* w;
  int64_t w_stride;
  const float* bias;
  const int64_t* targets;
  int64_t rows, classes;
  int32_t width;
  float smoothing;
  char* workspace;
  hipStream_t st;
};

fn::HeadArgs head_args(const Call& c, const Plan& p, const fn::Operand& x, const fn::Operand& w,
                       int64_t first, int64_t count) {
  fn::HeadArgs a{};
  a.a = x;
  a.b = w;
  a.M = c.rows;
  a.N = count;
  a.K = p.pack_x || p.pack_w ? p.width_packed : c.width;
  a.K_split = p.logits.K_split;
  a.bias = c.bias != nullptr ? c.bias + first : nullptr;
  a.targets = c.targets;
  a.first_class = first;
  a.classes = c.classes;
  a.smoothing = c.smoothing;
  return a;
}

template <typename T>
int forward(const Call& c, const Plan& p, float* losses, float* lse) {
  char* const ws = c.workspace;
  const fn::Operand x = operand<T>(c.x, c.x_stride, c.rows, c.width, p.width_packed,
                                   p.pack_x ? ws + p.x : nullptr, c.st);
  const int64_t size = fn::kHeadTileSizes[p.logits.tile];
  for (int64_t first = 0, tile = 0; first < c.classes; first += p.piece) {
    const int64_t count = std::min(p.piece, c.classes - first);
    const fn::Operand w = operand<T>((const T*)c.w + first * c.w_stride, c.w_stride, count, c.width,
                                     p.width_packed, p.pack_w ? ws + p.w : nullptr, c.st);
    fn::HeadArgs a = head_args(c, p, x, w, first, count);
    a.stats = (fn::f32x2*)(ws + p.stats);
    a.sums = c.smoothing > 0.0f ? (float*)(ws + p.sums) : nullptr;
    a.target_z = (float*)(ws + p.target_z);
    a.stat_tiles = p.stat_tiles;
    a.first_tile = tile;
    fn::launch_head<T>(fn::kHeadStatistics, false, {a, p.logits.tile, 1}, c.st);
    FN_TRY(launch_status("head_kernel launch"));
    tile += (count + size - 1) / size;
  }
  fn::JoinArgs j{};
  j.stats = (const fn::f32x2*)(ws + p.stats);
  j.sums = c.smoothing > 0.0f ? (const float*)(ws + p.sums) : nullptr;
  j.target_z = (const float*)(ws + p.target_z);
  j.targets = c.targets;
  j.losses = losses;
  j.lse = lse;
  j.rows = c.rows;
  j.classes = c.classes;
  j.tiles = p.stat_tiles;
  j.smoothing = c.smoothing;
  // at most 2^24 work-groups of 256 threads to a launch
  for (int64_t row = 0; row < c.rows; row += (int64_t)1 << 25) {
    j.rows = std::min<int64_t>(c.rows - row, (int64_t)1 << 25);
    fn::loss_join_kernel<<<blocks_for(j.rows, 4), 256, 0, c.st>>>(j);
    FN_TRY(launch_status("loss_join_kernel launch"));
    j.stats += j.rows * j.tiles;
    if (j.sums != nullptr) j.sums += j.rows * j.tiles;
    j.target_z += j.rows;
    j.targets += j.rows;
    j.losses += j.rows;
    j.lse += j.rows;
  }
  return ok();
}

struct Gradients {
  const float* dlosses;
  int64_t dloss_stride;
  const float* lse;
  void* dx;
  int64_t dx_stride;
  void* dw;
  int64_t dw_stride;
  float* dbias;
};

template <typename T>
int round_sums(const float* sums, const Plan& p, int64_t split_stride, int splits, int64_t rows,
               int32_t width, const float* scale, T* out, int64_t out_stride, hipStream_t st) {
  if (rows == 0) return FN_OK;
  const dim3 grid(blocks_for(((int64_t)width + 3) / 4, 256),
                  (unsigned)std::min<int64_t>(rows, 65535));
  fn::loss_round_kernel<T><<<grid, 256, 0, st>>>(sums, p.sum_pitch, split_stride, splits, rows,
                                                 width, scale, out, out_stride);
  return launch_status("loss_round_kernel launch");
}

template <typename T>
int backward(const Call& c, const Plan& p, const Gradients& g) {
  constexpr int64_t e = sizeof(T);
  char* const ws = c.workspace;
  const fn::Operand x = operand<T>(c.x, c.x_stride, c.rows, c.width, p.width_packed,
                                   p.pack_x ? ws + p.x : nullptr, c.st);
  const float* scale = nullptr;
  if constexpr (sizeof(T) == 2) {
    fn::loss_scale_kernel<<<1, 1024, 0, c.st>>>(
        g.dlosses, g.dloss_stride, c.rows, std::is_same_v<T, _Float16> ? 16384.0f : 1.0f,
        (float*)(ws + p.scale));
    FN_TRY(launch_status("loss_scale_kernel launch"));
    scale = (const float*)(ws + p.scale);
  }
  for (int64_t first = 0; first < c.classes; first += p.piece) {
    const int64_t count = std::min(p.piece, c.classes - first);
    const fn::Operand w = operand<T>((const T*)c.w + first * c.w_stride, c.w_stride, count, c.width,
                                     p.width_packed, p.pack_w ? ws + p.w : nullptr, c.st);
    if (c.rows > 0) {
      fn::HeadArgs a = head_args(c, p, x, w, first, count);
      a.lse = g.lse;
      a.dlosses = g.dlosses;
      a.dloss_stride = g.dloss_stride;
      a.bias_sums = g.dbias != nullptr ? (float*)(ws + p.bias_sums) : nullptr;
      a.scale = scale;
      a.out = ws + p.g;
      a.out_stride = p.pitch;
      fn::launch_head<T>(fn::kHeadGradient, false, {a, p.logits.tile, 1}, c.st);
      FN_TRY(launch_status("head_kernel launch"));
    }
    if (g.dbias != nullptr) {
      fn::column_sum_kernel<<<blocks_for(count, 64), 1024, 0, c.st>>>(
          (const float*)(ws + p.bias_sums), c.rows > 0 ? (int32_t)p.bias_rows : 0,
          (int32_t)p.pitch, (int32_t)count, g.dbias + first);
      FN_TRY(launch_status("column_sum_kernel launch"));
    }
    const fn::Operand gradient = {ws + p.g, p.pitch * e, c.rows, p.pitch * e};
    if (g.dx != nullptr && c.rows > 0) {
      fn::HeadArgs a{};
      a.a = gradient;
      a.b = w;
      a.M = c.rows;
      a.N = c.width;
      a.K = count;
      a.K_split = p.dx.K_split;
      a.scale = scale;
      a.out = p.sum_dx ? (void*)(ws + p.dx_sums) : g.dx;
      a.out_stride = p.sum_dx ? p.sum_pitch : g.dx_stride;
      a.split_stride = c.rows * p.sum_pitch;
      a.add = first > 0;
      fn::launch_head<T>(p.sum_dx ? fn::kHeadSums : fn::kHeadRounded, false,
                         {a, p.dx.tile, p.dx.splits}, c.st);
      FN_TRY(launch_status("head_kernel launch"));
    }
    if (g.dw != nullptr) {
      fn::HeadArgs a{};
      a.a = gradient;
      a.b = x;
      a.M = count;
      a.N = c.width;
      a.K = c.rows;
      a.K_split = p.dw.K_split;
      a.scale = scale;
      T* const out = (T*)g.dw + first * g.dw_stride;
      a.out = p.sum_dw ? (void*)(ws + p.dw_sums) : out;
      a.out_stride = p.sum_dw ? p.sum_pitch : g.dw_stride;
      a.split_stride = p.piece * p.sum_pitch;
      fn::launch_head<T>(p.sum_dw ? fn::kHeadSums : fn::kHeadRounded, true,
                         {a, p.dw.tile, p.dw.splits}, c.st);
      FN_TRY(launch_status("head_kernel launch"));
      if (p.sum_dw)
        FN_TRY(round_sums<T>((const float*)(ws + p.dw_sums), p, a.split_stride, p.dw.splits, count,
                             c.width, scale, out, g.dw_stride, c.st));
    }
  }
  if (g.dx != nullptr && p.sum_dx)
    FN_TRY(round_sums<T>((const float*)(ws + p.dx_sums), p, c.rows * p.sum_pitch, p.dx.splits,
                         c.rows, c.width, scale, (T*)g.dx, g.dx_stride, c.st));
  return ok();
}

int check_workspace(int64_t given, int64_t needed) {
  if (given < needed)
    return fail(FN_EINVAL, "workspace of %lld bytes, %lld needed", (long long)given,
                (long long)needed);
  return FN_OK;
}

}  // namespace

FN_EXPORT int fn_linear_cross_entropy_workspace(int64_t rows, int64_t classes, int32_t width,
                                                int32_t dtype, int32_t in_place_x,
                                                int32_t in_place_weight, int32_t backward_pass,
                                                int64_t* bytes) {
  FN_TRY(check_head(rows, classes, width, dtype));
  if (bytes == nullptr) return fail(FN_EINVAL, "bytes is NULL");
  *bytes = plan_of(rows, classes, width, type_bytes(dtype), !in_place_x, !in_place_weight,
                   backward_pass != 0)
               .bytes;
  return ok();
}

FN_EXPORT int fn_linear_cross_entropy(const void* x_dev, int64_t x_stride, const void* weight_dev,
                                      int64_t weight_stride, const float* bias_dev,
                                      const int64_t* targets_dev, int64_t rows, int64_t classes,
                                      int32_t width, float smoothing, int32_t dtype,
                                      float* losses_dev, float* lse_dev, void* workspace_dev,
                                      int64_t workspace_bytes, void* stream) {
  FN_TRY(check_head(rows, classes, width, dtype));
  if (!in_unit(smoothing)) return fail(FN_EINVAL, "smoothing must lie in [0, 1]");
  if (rows == 0) return ok();
  const int64_t e = type_bytes(dtype);
  const Plan plan = plan_of(rows, classes, width, e, !in_place(x_dev, x_stride, width, e),
                            !in_place(weight_dev, weight_stride, width, e), false);
  FN_TRY(check_workspace(workspace_bytes, plan.bytes));
  const Buffer buffers[] = {
      {"x_dev", x_dev, rows, width, x_stride, e, false},
      {"weight_dev", weight_dev, classes, width, weight_stride, e, false},
      {"bias_dev", bias_dev, bias_dev != nullptr ? 1 : 0, classes, 0, 4, false},
      {"targets_dev", targets_dev, 1, rows, 0, 8, false},
      {"losses_dev", losses_dev, 1, rows, 0, 4, true},
      {"lse_dev", lse_dev, 1, rows, 0, 4, true},
      {"workspace_dev", workspace_dev, 1, plan.bytes / 16, 0, 16, true},
  };
  int dev = -1;
  FN_TRY(check_buffers(buffers, &dev));
  const Call c = {x_dev, x_stride, weight_dev, weight_stride, bias_dev, targets_dev, rows,
                  classes, width, smoothing, (char*)workspace_dev, (hipStream_t)stream};
  if (dtype == FN_OUT_FP32) return forward<float>(c, plan, losses_dev, lse_dev);
  if (dtype == FN_OUT_FP16) return forward<_Float16>(c, plan, losses_dev, lse_dev);
  return forward<fn::BF16>(c, plan, losses_dev, lse_dev);
}

FN_EXPORT int fn_linear_cross_entropy_backward(
    const float* dlosses_dev, int64_t dlosses_stride, const void* x_dev, int64_t x_stride,
    const void* weight_dev, int64_t weight_stride, const float* bias_dev,
    const int64_t* targets_dev, const float* lse_dev, int64_t rows, int64_t classes, int32_t width,
    float smoothing, int32_t dtype, void* dx_dev, int64_t dx_stride, void* dweight_dev,
    int64_t dweight_stride, float* dbias_dev, void* workspace_dev, int64_t workspace_bytes,
    void* stream) {
  FN_TRY(check_head(rows, classes, width, dtype));
  if (!in_unit(smoothing)) return fail(FN_EINVAL, "smoothing must lie in [0, 1]");
  const int64_t e = type_bytes(dtype), one = rows ? 1 : 0;
  const Plan plan = plan_of(rows, classes, width, e, !in_place(x_dev, x_stride, width, e),
                            !in_place(weight_dev, weight_stride, width, e), true);
  FN_TRY(check_workspace(workspace_bytes, plan.bytes));
  const Buffer buffers[] = {
      {"dlosses_dev", dlosses_dev, rows, 1, dlosses_stride, 4, false},
      {"x_dev", x_dev, rows, width, x_stride, e, false},
      {"weight_dev", weight_dev, classes, width, weight_stride, e, false},
      {"bias_dev", bias_dev, bias_dev != nullptr ? 1 : 0, classes, 0, 4, false},
      {"targets_dev", targets_dev, one, rows, 0, 8, false},
      {"lse_dev", lse_dev, one, rows, 0, 4, false},
      {"dx_dev", dx_dev, dx_dev != nullptr ? rows : 0, width, dx_stride, e, true},
      {"dweight_dev", dweight_dev, dweight_dev != nullptr ? classes : 0, width, dweight_stride, e,
       true},
      {"dbias_dev", dbias_dev, dbias_dev != nullptr ? 1 : 0, classes, 0, 4, true},
      {"workspace_dev", workspace_dev, 1, plan.bytes / 16, 0, 16, true},
  };
  int dev = -1;
  FN_TRY(check_buffers(buffers, &dev));
  const Call c = {x_dev, x_stride, weight_dev, weight_stride, bias_dev, targets_dev, rows,
                  classes, width, smoothing, (char*)workspace_dev, (hipStream_t)stream};
  const Gradients g = {dlosses_dev, dlosses_stride, lse_dev, dx_dev, dx_stride,
                       dweight_dev, dweight_stride, dbias_dev};
  if (dtype == FN_OUT_FP32) return backward<float>(c, plan, g);
  if (dtype == FN_OUT_FP16) return backward<_Float16>(c, plan, g);
  return backward<fn::BF16>(c, plan, g);
}
