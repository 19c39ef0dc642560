// loss_api.hip -- the C ABI of the linear cross entropy: argument checks, the
// plan of a call (pieces of the classes, tiles, splits, workspace) and the
// launches.  Declarations, argument meaning, layouts and error behaviour are
// documented in include/fn.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

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
// Weights that do not stay in the memory-side cache until the next call anyway.
constexpr int64_t kCached = (int64_t)1 << 28;
constexpr int64_t kFewRows = 8192;
constexpr int kMostSplits = 64;
constexpr int32_t kMaxFeatures = 1 << 20;
constexpr int64_t kMaxClasses = (int64_t)1 << 28;
// a stage's rows times the stride within the 31-bit offsets of a resource
constexpr int64_t kMaxStrideBytes = ((int64_t)1 << 31) / 256 - 1;

struct Choice {
  int tile = 0, splits = 1;
  int64_t K_split = 0;
  double cost = 0.0;  // us
};

// What the matrix instructions take: bytes of an element, passes over the
// contraction and parts of an operand (Fp32Parts).
struct Elements {
  int64_t size;
  int passes, parts;
};

Elements elements_of(int64_t type_bytes, bool split) {
  return split ? Elements{2, fn::HeadType<fn::Fp32Parts>::kPasses, 3} : Elements{type_bytes, 1, 1};
}

int64_t tiles_of(int tile, int64_t M, int64_t N) {
  const int64_t m = fn::kHeadTileM[tile], n = fn::kHeadTileN[tile];
  return ((M + m - 1) / m) * ((N + n - 1) / n);
}

// The time of a product's tiles in us, from measurements on 256 compute units with
// K of 64 to 8192: a fixed part (first loads, output) and one for every 1,000
// elements of the contraction, where each unit has one tile or where it has more,
// two or more of them at once; of 256x256, 128x128 and 64x64 tiles.  What memory
// gives bounds it from below.
// kStoredLogits: logits whose gradients are stored, in three parts where operands
// have them, which 256x256 tiles cannot do beside their products (1024x65536x384 fp32
// with 256x256 / 128x128 tiles 1421 / 1266 us in all).
enum ProductKind { kLogits = 0, kGradients = 1, kStoredLogits = 2 };

double tiles_time(int tile, ProductKind kind, const Elements& t, int64_t tiles, int64_t M,
                  int64_t N, int64_t K) {
  constexpr double kFixed[2][2][3] = {{{9.0, 4.0, 2.0}, {9.0, 2.6, 1.5}},
                                      {{8.0, 2.7, 1.2}, {8.3, 2.4, 1.3}}};
  constexpr double kFixedParts[2][2][3] = {{{9.0, 6.0, 4.0}, {9.0, 5.0, 2.5}},
                                           {{14.0, 7.0, 3.5}, {14.0, 5.0, 2.7}}};
  constexpr double kEach[3][2][2][3] = {
      {{{16.6, 8.2, 3.4}, {16.2, 5.0, 2.43}}, {{18.0, 10.0, 5.0}, {18.0, 5.5, 3.1}}},
      {{{223.0, 62.0, 18.3}, {223.0, 57.5, 15.9}}, {{230.0, 66.0, 23.5}, {230.0, 59.0, 18.0}}},
      {{{118.0, 60.0, 23.0}, {122.0, 52.0, 15.8}}, {{137.0, 77.0, 41.0}, {137.0, 50.0, 27.0}}}};
  const int type = t.passes > 1 ? 2 : t.size == 4 ? 1 : 0;
  const double memory = (double)(M + N) * K * t.size * t.parts / 5.4e6;
  const double rounds = (double)tiles / kUnits;
  if (tile == 4) {
    const double each = 8e-3 * K * (t.size == 4 ? 2 : 1);
    return std::max(std::ceil(rounds / 2) * (2.0 + each), memory);
  }
  if (tile == 3) {
    constexpr double kNarrow[3][3] = {{4.0, 2.4, 2.3}, {10.5, 6.3, 7.0}, {19.0, 13.5, 14.0}};
    const bool groups = fn::in_groups(tile, tiles, K);
    const double each = kNarrow[type][groups ? 1 : tiles > kUnits ? 2 : 0] * 1e-3 * K;
    return std::max(std::ceil(rounds) * ((groups ? 3.5 : 1.5) + each), memory);
  }
  const int more = tiles > kUnits;
  const bool stored = kind == kStoredLogits;
  if (stored) kind = kLogits;
  double fixed = type == 2 ? kFixedParts[kind][more][tile] : kFixed[kind][more][tile];
  if (stored && type == 2 && tile == 0) fixed += 56.0;
  return std::max(std::ceil(rounds) * (fixed + kEach[type][kind][more][tile] * 1e-3 * K), memory);
}

int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// The tile and the splits of the contraction for M x N outputs and K elements
// of it, by the time they would take.  Up to 16 rows have tiles of 16: the wide
// ones where they give every compute unit one (1x50000x4096 bf16 with 64 / 128
// classes a tile 77 / 71 us, 1x16000x4096 30 / 33); more rows have the narrow ones
// where they are few.  `few_rows`: whether there are kernels for those.
Choice choose(ProductKind kind, int64_t M, int64_t N, int64_t K, const Elements& t, int most_splits,
              bool few_rows = true) {
  const int64_t stage = fn::kStageRow / t.size;
  Choice best;
  best.cost = 1e300;
  const bool few = few_rows && M <= 16;
  const int first = !few ? 0 : N >= 128 * kUnits ? 4 : 3, last = few ? first : few_rows ? 3 : 2;
  for (int tile = first; tile <= last; ++tile) {
    const int64_t tiles = tiles_of(tile, M, N);
    if (tile == 3 && !few && tiles > kUnits) continue;
    if (tiles >= (int64_t)1 << 22) continue;  // 2^32 threads to a launch
    for (int splits = 1; splits <= most_splits; splits *= 2) {
      if (splits > 1 && (K < 8 * stage * splits || tiles * splits > 4 * kUnits)) break;
      const int64_t K_split = std::max(round_up((K + splits - 1) / splits, stage), stage);
      double cost = 3.0 + tiles_time(tile, kind, t, tiles * splits, M, N, K_split);
      // partial products are written and read again, in a launch of their own
      if (splits > 1) cost += 4.0 + 0.1 * splits + (double)M * N * 8.0 * splits / 4e6;
      if (cost < best.cost) best = {tile, splits, K_split, cost};
    }
  }
  return best;
}

// Parts of a workspace, one behind the other.
struct Parts {
  int64_t bytes = 0;
  int64_t take(int64_t n) {
    const int64_t at = bytes;
    bytes += round_up(n, 256);
    return at;
  }
};

// A call goes through its classes in pieces of the same size, but for the last.
struct Plan {
  bool split;  // fp32 as Fp32Parts
  bool pack_x, pack_w;
  int64_t width_packed;  // elements
  int64_t piece;         // classes
  int64_t pieces;
  Choice logits[2], dx[2], dw[2];  // [1]: of a shorter last piece
  int pair_tile;                   // of dx and dw in one launch, or -1
  bool sum_dx;                     // in fp32 first
  int64_t pitch;                   // of g's rows, elements
  int64_t sum_pitch;               // of fp32 products' rows
  int64_t stat_tiles;
  // places in the workspace
  int64_t scale, x, w, stats, sums, target_z, g, dx_sums, dw_sums, bias_sums;
  int64_t bytes;

  int64_t last(int64_t classes) const { return classes - (pieces - 1) * piece; }
  int which(int64_t count) const { return count == piece ? 0 : 1; }
};

// Tiles along the classes of a choice for the logits, and its rows of bias_sums.
int64_t class_tiles(const Choice& c, int64_t classes) {
  return (classes + fn::kHeadTileN[c.tile] - 1) / fn::kHeadTileN[c.tile];
}

int64_t bias_rows_of(const Choice& c, int64_t rows) {
  return (rows + fn::kHeadTileM[c.tile] - 1) / fn::kHeadTileM[c.tile] * fn::kHeadTileRows[c.tile];
}

// Classes of a piece, at most `most` of them: as many as give every compute unit
// the same number of 256x256 tiles (4096x50000x4096 bf16, gradients, with pieces of
// 12544 / 16384: 4.50 / 3.80 ms).
int64_t piece_of(int64_t rows, int64_t most) {
  const int64_t m = (rows + 255) / 256, rounds = m * (most / 256) / kUnits;
  return rounds > 0 ? std::max<int64_t>(rounds * kUnits / m, 1) * 256 : most;
}

// fp32 operands in parts, if six products of bf16 and the copies (ten bytes an
// element) take less time than one of fp32 (1999x21841x1021: 465 us against 730;
// 1024x65536x64 78 / 92).  The parts of the gradients of the logits do not stay in
// the memory-side cache (gradients of 1024x65536x384 1280 / 1226, x1024 2420 / 2977).
bool worth_parts(int64_t rows, int64_t classes, int32_t width, bool backward) {
  double cost[2] = {0.0, 6.0 + (double)(rows + classes) * width * 10.0 / 4e6};
  if (backward) cost[1] += (double)rows * classes * 3.5e-6;
  for (int split = 0; split < 2; ++split) {
    const Elements t = elements_of(4, split);
    cost[split] += choose(backward ? kStoredLogits : kLogits, rows, classes, width, t, 1).cost;
    if (backward)
      cost[split] += choose(kGradients, rows, width, classes, t, kMostSplits).cost +
                     choose(kGradients, classes, width, rows, t, kMostSplits, false).cost;
  }
  return cost[1] < cost[0];
}

Plan plan_of(int64_t rows, int64_t classes, int32_t width, int64_t e, bool pack_x, bool pack_w,
             bool backward) {
  Plan p{};
  p.split = e == 4 && worth_parts(rows, classes, width, backward);
  p.pack_x = pack_x || p.split;
  p.pack_w = pack_w || p.split;
  const Elements t = elements_of(e, p.split);
  const int64_t bytes = t.size * t.parts;  // of an operand's element
  p.width_packed = round_up(width, 16 / t.size);
  const int64_t K = p.pack_x || p.pack_w ? p.width_packed : width;
  // what a class of a piece has in the workspace: its gradients, a copy of its
  // weights
  const int64_t per_class = std::max(backward ? std::max<int64_t>(rows, 1) * bytes : 0,
                                     p.pack_w ? p.width_packed * bytes : 0);
  auto most_in = [&](int64_t room) {
    const int64_t all = round_up(classes, 256);
    return per_class > 0 ? std::min(all, std::max<int64_t>(room / per_class / 256, 1) * 256) : all;
  };
  int64_t most = most_in(kPieceBytes);
  // in parts a class has three times the bytes, but no more products: twice the room
  // for gradients (2048x50000x4096 14.0 -> 12.0 ms, 8192x50000x1024 14.0 -> 13.3), and
  // for losses whose pieces would not give every compute unit a tile (2048x50000x4096
  // 4.64 -> 3.91 ms; others lose up to 4% by it)
  if (p.split && (backward || (rows + 255) / 256 * (most / 256) < kUnits))
    most = most_in(2 * kPieceBytes);
  if (backward) most = std::min(most, kMaxStrideBytes / t.size / 256 * 256);
  p.piece = classes;
  if (most < classes) {
    p.piece = piece_of(rows, most);
  } else if (!backward) {
    // whole rounds of tiles first and the rest in smaller ones, if that is less
    const int64_t piece = piece_of(rows, classes / 256 * 256);
    auto cost = [&](int64_t count) { return choose(kLogits, rows, count, K, t, 1).cost; };
    if (piece > 0 && piece < classes && cost(piece) + cost(classes - piece) < cost(classes))
      p.piece = piece;
  }
  p.pieces = (classes + p.piece - 1) / p.piece;
  const int64_t counts[2] = {p.piece, p.last(classes)};
  Parts parts;
  p.scale = parts.take(8);
  if (p.pack_x) p.x = parts.take(rows * p.width_packed * bytes);
  if (p.pack_w) p.w = parts.take(p.piece * p.width_packed * bytes);
  const ProductKind kind = backward ? kStoredLogits : kLogits;
  for (int k = 0; k < 2; ++k) p.logits[k] = choose(kind, rows, counts[k], K, t, 1);
  if (!backward) {
    p.stat_tiles = (p.pieces - 1) * class_tiles(p.logits[0], p.piece) +
                   class_tiles(p.logits[p.which(counts[1])], counts[1]);
    p.stats = parts.take(rows * p.stat_tiles * 8);
    p.sums = parts.take(rows * p.stat_tiles * 4);
    p.target_z = parts.take(rows * 4);
    p.bytes = parts.bytes;
    return p;
  }
  p.pitch = round_up(p.piece, 64);
  p.sum_pitch = round_up(width, 4);
  p.pair_tile = -1;
  int64_t bias_rows = 0, dw_rows = 0;
  for (int k = 0; k < 2; ++k) {
    // dx's sums of the first piece fill every split's place; the last one may use
    // fewer, but no others (1024x129280x384 fp16: 723 us without any, 505)
    p.dx[k] = choose(kGradients, rows, width, counts[k], t, k == 0 ? kMostSplits : p.dx[0].splits);
    p.dw[k] = choose(kGradients, counts[k], width, rows, t, kMostSplits, false);
    bias_rows = std::max(bias_rows, bias_rows_of(p.logits[k], rows));
    if (p.dw[k].splits > 1) dw_rows = std::max(dw_rows, p.dw[k].splits * counts[k]);
  }
  p.sum_dx = p.pieces > 1 || p.dx[0].splits > 1;
  if (p.pieces == 1 && rows > 0) {
    double least = p.dx[0].cost + p.dw[0].cost;
    for (int tile = 1; tile < 3; ++tile) {
      const int64_t dx = tiles_of(tile, rows, width), dw = tiles_of(tile, classes, width);
      if (dx + dw >= (int64_t)1 << 22) continue;
      // side by side: as if all were of either kind, by their share
      const double cost =
          3.0 + (dx * tiles_time(tile, kGradients, t, dx + dw, rows, width, classes) +
                 dw * tiles_time(tile, kGradients, t, dx + dw, classes, width, rows)) /
                    (dx + dw);
      const double longest =
          3.0 + tiles_time(tile, kGradients, t, 1, 1, 1, std::max(rows, classes));
      if (std::max(cost, longest) < least) {
        least = std::max(cost, longest);
        p.pair_tile = tile;
      }
    }
  }
  p.g = parts.take(rows * p.pitch * bytes);
  if (p.sum_dx) p.dx_sums = parts.take(p.dx[0].splits * rows * p.sum_pitch * 4);
  if (dw_rows > 0) p.dw_sums = parts.take(dw_rows * p.sum_pitch * 4);
  p.bias_sums = parts.take(bias_rows * p.pitch * 4);
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
  return stride >= width && stride <= kMaxStrideBytes / e &&
         ((uintptr_t)p | (uint64_t)(stride * e) | (uint64_t)(width * e)) % 16 == 0;
}

// An operand of the call: where it lies, or the place of its copy, which is still
// to be made.
struct Placed {
  fn::Operand operand;
  fn::Copy copy;
  int64_t rows;  // to copy
};

template <typename T>
Placed place(const void* from, int64_t stride, int64_t rows, int32_t width, int64_t copied,
             char* copy) {
  constexpr int64_t e = sizeof(typename fn::HeadType<T>::Operand);
  if (copy == nullptr) return {{(const char*)from, stride * e, rows, (int64_t)width * e, 0}, {}, 0};
  fn::Copy c{};
  c.from = from;
  c.stride = stride;
  c.to = copy;
  c.part = rows * copied;
  c.pieces = fn::division_by((uint32_t)(copied * e / 16));
  c.width = width;
  return {{copy, copied * e, rows, copied * e, rows * copied * e}, c, rows};
}

// Makes the copies of one or two operands, at most 2^30 pieces of each in a launch.
template <typename T>
int make_copies(Placed a, Placed b, hipStream_t st) {
  while (a.rows > 0 || b.rows > 0) {
    unsigned groups = 0;
    for (Placed* p : {&a, &b}) {
      const int64_t pieces = std::max<int64_t>(p->copy.pieces.by, 1);
      const int64_t count = std::min(p->rows, std::max<int64_t>(((int64_t)1 << 30) / pieces, 1));
      p->copy.items = (uint32_t)(count * pieces);
      if (count == 0) p->copy.items = 0;
      groups += blocks_for(p->copy.items, 256);
    }
    fn::loss_copy_kernel<T><<<groups, 256, 0, st>>>(a.copy, b.copy);
    FN_TRY(launch_status("loss_copy_kernel launch"));
    for (Placed* p : {&a, &b}) {
      const int64_t count = p->copy.items / std::max(p->copy.pieces.by, 1u);
      p->copy.from = (const typename fn::HeadType<T>::Output*)p->copy.from + count * p->copy.stride;
      p->copy.to = (char*)p->copy.to + (int64_t)p->copy.items * 16;
      p->rows -= count;
    }
  }
  return FN_OK;
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
  a.K_split = p.logits[p.which(count)].K_split;
  a.bias = c.bias != nullptr ? c.bias + first : nullptr;
  a.targets = c.targets;
  a.once = w.stride * c.classes > kCached;
  a.first_class = first;
  a.classes = c.classes;
  a.smoothing = c.smoothing;
  return a;
}

template <typename T>
int forward(const Call& c, const Plan& p, float* losses, float* lse) {
  char* const ws = c.workspace;
  using Given = typename fn::HeadType<T>::Output;
  Placed x = place<T>(c.x, c.x_stride, c.rows, c.width, p.width_packed,
                      p.pack_x ? ws + p.x : nullptr);
  for (int64_t first = 0, tile = 0; first < c.classes; first += p.piece) {
    const int64_t count = std::min(p.piece, c.classes - first);
    const Placed w = place<T>((const Given*)c.w + first * c.w_stride, c.w_stride, count, c.width,
                              p.width_packed, p.pack_w ? ws + p.w : nullptr);
    FN_TRY(make_copies<T>(x, w, c.st));
    x.rows = 0;
    fn::HeadArgs a = head_args(c, p, x.operand, w.operand, first, count);
    a.stats = (fn::f32x2*)(ws + p.stats);
    a.sums = c.smoothing > 0.0f ? (float*)(ws + p.sums) : nullptr;
    a.target_z = (float*)(ws + p.target_z);
    a.stat_tiles = p.stat_tiles;
    a.first_tile = tile;
    const bool alone = p.stat_tiles == 1;
    a.losses = alone ? losses : nullptr;
    a.losses_lse = lse;
    const Choice& choice = p.logits[p.which(count)];
    fn::launch_head<T>(fn::kHeadStatistics, false, {a, choice.tile, 1}, c.st);
    FN_TRY(launch_status("head_kernel launch"));
    tile += class_tiles(choice, count);
  }
  if (p.stat_tiles == 1) return ok();
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
  const fn::Division vectors = fn::division_by((uint32_t)((width + 3) / 4));
  // at most 2^31 threads to a launch
  const int64_t most = ((int64_t)1 << 31) / vectors.by;
  for (int64_t row = 0; row < rows; row += most) {
    const uint32_t items = (uint32_t)(std::min(most, rows - row) * vectors.by);
    fn::loss_round_kernel<T><<<blocks_for(items, 256), 256, 0, st>>>(
        sums + row * p.sum_pitch, p.sum_pitch, split_stride, splits, items, vectors, width, scale,
        out + row * out_stride, out_stride);
    FN_TRY(launch_status("loss_round_kernel launch"));
  }
  return FN_OK;
}

template <typename T>
int backward(const Call& c, const Plan& p, const Gradients& g) {
  using Given = typename fn::HeadType<T>::Output;
  constexpr int64_t e = sizeof(typename fn::HeadType<T>::Operand);
  char* const ws = c.workspace;
  Placed x = place<T>(c.x, c.x_stride, c.rows, c.width, p.width_packed,
                      p.pack_x ? ws + p.x : nullptr);
  float* scale = nullptr;
  float scale_to = 0.0f;
  if constexpr (sizeof(Given) == 2) {
    scale = (float*)(ws + p.scale);
    scale_to = std::is_same_v<Given, _Float16> ? 16384.0f : 1.0f;
    // few dlosses: each work-group of the first kernel looks for the largest one,
    // for less than a launch takes
    if (c.rows == 0 || (c.rows > kFewRows && g.dloss_stride != 0)) {
      fn::loss_scale_kernel<<<1, 1024, 0, c.st>>>(g.dlosses, g.dloss_stride, c.targets, c.classes,
                                                  c.rows, scale_to, scale);
      FN_TRY(launch_status("loss_scale_kernel launch"));
      scale_to = 0.0f;
    }
  }
  const bool pair = p.pair_tile > 0 && g.dx != nullptr && g.dw != nullptr;
  for (int64_t first = 0; first < c.classes; first += p.piece) {
    const int64_t count = std::min(p.piece, c.classes - first);
    const int k = p.which(count);
    const int32_t bias_rows = (int32_t)bias_rows_of(p.logits[k], c.rows);
    float* const bias_sums = (float*)(ws + p.bias_sums);
    const Placed w = place<T>((const Given*)c.w + first * c.w_stride, c.w_stride, count, c.width,
                              p.width_packed, p.pack_w ? ws + p.w : nullptr);
    FN_TRY(make_copies<T>(x, w, c.st));
    x.rows = 0;
    if (c.rows > 0) {
      fn::HeadArgs a = head_args(c, p, x.operand, w.operand, first, count);
      a.lse = g.lse;
      a.dlosses = g.dlosses;
      a.dloss_stride = g.dloss_stride;
      a.bias_sums = g.dbias != nullptr ? bias_sums : nullptr;
      a.scale = scale;
      a.scale_to = scale_to;
      a.out = ws + p.g;
      a.out_stride = p.pitch;
      a.out_part = c.rows * p.pitch;
      fn::launch_head<T>(fn::kHeadGradient, false, {a, p.logits[k].tile, 1}, c.st);
      FN_TRY(launch_status("head_kernel launch"));
    }
    const fn::Operand gradient = {ws + p.g, p.pitch * e, c.rows, p.pitch * e,
                                  c.rows * p.pitch * e};
    fn::HeadArgs dx{}, dw{};
    dx.a = dw.a = gradient;
    dx.b = w.operand;
    dx.once = w.operand.stride * c.classes > kCached;
    dw.b = x.operand;
    dx.M = dw.K = c.rows;
    dx.K = dw.M = count;
    dx.N = dw.N = c.width;
    dx.scale = dw.scale = scale;
    dx.out = g.dx;
    dx.out_stride = g.dx_stride;
    Given* const dw_out = (Given*)g.dw + first * g.dw_stride;
    dw.out = dw_out;
    dw.out_stride = g.dw_stride;
    if (pair) {
      fn::HeadPairArgs both{};
      dx.K_split = round_up(count, fn::kStageRow / e);
      dw.K_split = round_up(c.rows, fn::kStageRow / e);
      both.dx = dx;
      both.dw = dw;
      both.bias_sums = bias_sums;
      both.pitch = p.pitch;
      both.bias_rows = bias_rows;
      both.dbias = g.dbias;
      both.dw_first = dw.K > dx.K;
      fn::launch_head_pair<T>(both, p.pair_tile, c.st);
      return launch_status("head_pair_kernel launch");
    }
    if (g.dbias != nullptr) {
      fn::column_sum_kernel<<<blocks_for(count, 64), 1024, 0, c.st>>>(
          bias_sums, c.rows > 0 ? bias_rows : 0, (int32_t)p.pitch, (int32_t)count,
          g.dbias + first);
      FN_TRY(launch_status("column_sum_kernel launch"));
    }
    if (g.dx != nullptr && c.rows > 0) {
      dx.K_split = p.dx[k].K_split;
      if (p.sum_dx) {
        dx.out = ws + p.dx_sums;
        dx.out_stride = p.sum_pitch;
        dx.split_stride = c.rows * p.sum_pitch;
        dx.add = first > 0;
      }
      fn::launch_head<T>(p.sum_dx ? fn::kHeadSums : fn::kHeadRounded, false,
                         {dx, p.dx[k].tile, p.dx[k].splits}, c.st);
      FN_TRY(launch_status("head_kernel launch"));
    }
    if (g.dw != nullptr) {
      const int splits = p.dw[k].splits;
      dw.K_split = p.dw[k].K_split;
      if (splits > 1) {
        dw.out = ws + p.dw_sums;
        dw.out_stride = p.sum_pitch;
        dw.split_stride = count * p.sum_pitch;
      }
      fn::launch_head<T>(splits > 1 ? fn::kHeadSums : fn::kHeadRounded, true,
                         {dw, p.dw[k].tile, splits}, c.st);
      FN_TRY(launch_status("head_kernel launch"));
      if (splits > 1)
        FN_TRY(round_sums<Given>((const float*)(ws + p.dw_sums), p, dw.split_stride, splits, count,
                             c.width, scale, dw_out, g.dw_stride, c.st));
    }
  }
  if (g.dx != nullptr && p.sum_dx)
    FN_TRY(round_sums<Given>((const float*)(ws + p.dx_sums), p, c.rows * p.sum_pitch,
                         p.dx[0].splits, c.rows, c.width, scale, (Given*)g.dx, g.dx_stride, c.st));
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
  // what may turn out to lie in place after all has a plan of its own
  *bytes = 0;
  for (int copied = 0; copied < 4; ++copied) {
    const bool pack_x = copied & 1, pack_w = copied & 2;
    if ((pack_x && in_place_x) || (pack_w && in_place_weight)) continue;
    *bytes = std::max(*bytes, plan_of(rows, classes, width, type_bytes(dtype), pack_x, pack_w,
                                      backward_pass != 0)
                                  .bytes);
  }
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
  if (plan.split) return forward<fn::Fp32Parts>(c, plan, losses_dev, lse_dev);
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
  if (dlosses_stride != 0 && dlosses_stride != 1)
    return fail(FN_EINVAL, "dlosses_stride must be 0 or 1");
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
  if (plan.split) return backward<fn::Fp32Parts>(c, plan, g);
  if (dtype == FN_OUT_FP32) return backward<float>(c, plan, g);
  if (dtype == FN_OUT_FP16) return backward<_Float16>(c, plan, g);
  return backward<fn::BF16>(c, plan, g);
}
