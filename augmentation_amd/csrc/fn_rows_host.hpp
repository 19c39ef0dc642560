// fn_rows_host.hpp -- what the entry points that work on rows share on the
// host: the buffers of a call and their checks, and how many threads a row
// gets.
#pragma once
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "fn.h"
#include "fn_host.hpp"

#define FN_TRY(call)        \
  do {                      \
    const int rc_ = (call); \
    if (rc_) return rc_;    \
  } while (0)

namespace fnhost {

constexpr int32_t kMaxWidth = 1 << 30;
constexpr int32_t kColumnsPerLaunch = 1 << 26;  // of the sum of partial rows

inline int type_bytes(int32_t dtype) {
  return dtype == FN_OUT_FP32 ? 4 : dtype == FN_OUT_FP16 || dtype == FN_OUT_BF16 ? 2 : 0;
}

inline int check_type(int32_t dtype, const char* name) {
  if (type_bytes(dtype) == 0) return fail(FN_EINVAL, "unknown %s %d", name, dtype);
  return FN_OK;
}

// A buffer of a call: `rows` rows of `cols` elements, `stride` elements apart.
struct Buffer {
  const char* name;
  const void* p;
  int64_t rows, cols, stride;
  int64_t element;       // bytes
  bool output;
  unsigned replaces = 0;  // outputs: bit i = may lie exactly on buffer i of the call

  int64_t row_bytes() const { return cols * element; }
  int64_t stride_bytes() const { return stride * element; }
  int64_t span() const { return (rows - 1) * stride_bytes() + row_bytes(); }
  bool empty() const { return rows == 0 || cols == 0; }
};

// Strides and spans that fit the index arithmetic; an output's rows may not
// overlap each other, an input's may (stride 0: one row for all).
inline int check_layout(const Buffer& b) {
  if (b.stride < 0) return fail(FN_EINVAL, "%s: its row stride is negative", b.name);
  if (b.output && b.rows > 1 && b.stride < b.cols)
    return fail(FN_EINVAL, "%s: its row stride is shorter than a row", b.name);
  const __int128 span = ((__int128)std::max<int64_t>(b.rows - 1, 0) * b.stride + b.cols) * b.element;
  if (span > (__int128)1 << 62)
    return fail(FN_EOVERFLOW, "%s: its rows span more than 2^62 bytes", b.name);
  return FN_OK;
}

// True if some byte belongs to both.  Buffers of the same stride may lie side
// by side as column ranges of one allocation.
inline bool overlap(const Buffer& x, const Buffer& y) {
  const uintptr_t a0 = (uintptr_t)x.p, a1 = a0 + (uintptr_t)x.span();
  const uintptr_t b0 = (uintptr_t)y.p, b1 = b0 + (uintptr_t)y.span();
  if (a1 <= b0 || b1 <= a0) return false;
  const int64_t s = x.stride_bytes();
  if (s != y.stride_bytes() || s < x.row_bytes() || s < y.row_bytes()) return true;
  // where y's columns begin, counted from x's modulo the common stride
  int64_t d = (int64_t)((b0 >= a0 ? b0 - a0 : a0 - b0) % (uintptr_t)s);
  if (b0 < a0 && d != 0) d = s - d;
  return !(d >= x.row_bytes() && d + y.row_bytes() <= s);
}

inline bool same_place(const Buffer& x, const Buffer& y) {
  return x.p == y.p && x.rows == y.rows && x.row_bytes() == y.row_bytes() &&
         (x.stride_bytes() == y.stride_bytes() || x.rows == 1);
}

// All buffers of a call; optional ones that are absent have rows = 0.
template <int kCount>
int check_buffers(const Buffer (&b)[kCount], int* dev) {
  for (int i = 0; i < kCount; ++i) FN_TRY(check_layout(b[i]));
  for (int i = 0; i < kCount; ++i) {
    if (b[i].empty()) continue;
    if (b[i].p != nullptr && (uintptr_t)b[i].p % (uintptr_t)b[i].element != 0)
      return fail(FN_EINVAL, "%s must be aligned to its element size (%lld bytes)", b[i].name,
                  (long long)b[i].element);
    FN_TRY(check_device_range(b[i].p, (size_t)b[i].span(), b[i].name, dev));
  }
  for (int i = 0; i < kCount; ++i) {
    if (!b[i].output || b[i].empty()) continue;
    for (int j = 0; j < kCount; ++j) {
      if (j == i || b[j].empty() || (b[j].output && j > i)) continue;
      if ((b[i].replaces >> j & 1u) && same_place(b[i], b[j])) continue;
      if (overlap(b[i], b[j])) return fail(FN_EINVAL, "%s and %s overlap", b[i].name, b[j].name);
    }
  }
  return FN_OK;
}

inline int check_size(int64_t rows, int32_t width) {
  if (rows < 0) return fail(FN_EINVAL, "rows must be >= 0");
  if (rows > (int64_t)1 << 40) return fail(FN_EOVERFLOW, "rows exceeds 2^40");
  if (width < 1) return fail(FN_EINVAL, "width must be >= 1 (got %d)", width);
  if (width > kMaxWidth) return fail(FN_EOVERFLOW, "width %d exceeds 2^30", width);
  return FN_OK;
}

// Threads per row and chunks of eight elements per thread, by the row's width:
// the fewest threads that keep a row in registers with all of them at work, a
// wavefront's part for as long as that will do (no barrier).  Measured, norm to
// codes with a residual, us: 1000000x12 with 2 / 4 / 8 threads 26 / 36 / 62;
// 100000x100 with 8 / 16 / 32 24 / 21 / 32; 30000x1500 with 64x3 / 256x1 60 /
// 74; 30000x2040 backward with 64x4 / 128x2 / 256x1 92 / 99 / 101; 13000x2560
// with 64x5 / 256x2 45 / 46, backward 53 / 64, but 300x2560 5.7 / 4.6: the
// choice is by the width alone, so that a row's sums do not depend on how many
// rows there are.  0 threads: rows that do not fit.
struct RowShape {
  int32_t width;  // up to
  int threads, chunks;
};

constexpr RowShape kRowShapes[] = {{7, 1, 0},      {8, 1, 1},      {16, 2, 1},     {32, 4, 1},
                                   {64, 8, 1},     {128, 16, 1},   {256, 16, 2},   {512, 32, 2},
                                   {768, 32, 3},   {1024, 64, 2},  {1536, 64, 3},  {2048, 64, 4},
                                   {2560, 64, 5},  {4096, 256, 2}, {6144, 256, 3}, {8192, 512, 2},
                                   {16384, 512, 4}, {32768, 1024, 4}};

inline RowShape row_shape(int32_t width, int32_t widest) {
  for (const RowShape& s : kRowShapes)
    if (width <= s.width && s.width <= widest) return s;
  return {0, 0, 0};
}

constexpr int shape_key(int threads, int chunks) { return threads * 16 + chunks; }

}  // namespace fnhost
