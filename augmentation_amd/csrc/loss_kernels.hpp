// loss_kernels.hpp -- softmax cross entropy of a linear head, whose logits are
// never kept, and its gradients.
//
//   z[t, v] = sum_k x[t, k] w[v, k] + bias[v]                     (fp32)
//   lse[t]  = log sum_v exp z[t, v]
//   loss[t] = lse[t] - (1 - s) z[t, y_t] - s mean_v z[t, v]
//   g[t, v] = dloss[t] (exp(z[t, v] - lse[t]) - (1 - s) [v = y_t] - s / V)
//   dx = g w,  dw = g^T x,  dbias[v] = sum_t g[t, v]
//
// Forward: a product whose epilogue reduces every tile of logits to a maximum
// and a sum of exponentials per row, and a second kernel that joins a row's
// tiles.  Backward: the logits again, in pieces of the classes, turned into g
// where they are (rounded once to the operands' type, as the matrix
// instructions take them), then the two products with it.  What is computed a
// second time is a third of the backward pass; what is not kept is T x V
// logits.
//
// Large calls are bound by the matrix cores, whose clock sinks to 1.7 GHz under
// this load and which are busy 71% of it: 8192x50000x4096 bf16 2.46 ms, 1.36
// PFLOP/s (a library product of that shape alone, its logits written, 2.61 ms);
// gradients of 4096x50000x4096 4.0 ms, 1.26 PFLOP/s.  Few rows are bound by the
// bytes of the weights: 1x50000x4096 bf16 74 us, 5.6 TB/s.  Small calls by their
// launches: gradients of 1024x1000x768 fp16 19.5 us in two.
//
// One kernel serves the three products.  They differ in how their operands lie:
// "along" the contraction (x and w in the logits, g in dx: a row of memory is
// a row of the operand) or "across" it (w in dx, g and x in dw: a row of memory
// is one element of the contraction for all rows of the operand).
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "product_kernels.hpp"
#include "row_kernels.hpp"

namespace fn {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// exp(v) for v <= 0: exp2 of v log2(e), whose rounding error is made good to
// first order (for v near -20 it alone would be 10^-6 of the result).
__device__ __forceinline__ float exp_below(float v) {
  constexpr float kLog2e = 0x1.715476p+0f, kRest = 0x1.4ae0cp-26f, kLn2 = 0x1.62e43p-1f;
  const float t = v * kLog2e;
  const float r = __builtin_fmaf(v, kRest, __builtin_fmaf(v, kLog2e, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  // -infinity gives 0, where r is NaN
  return v < -200.0f ? 0.0f : __builtin_fmaf(e, r * kLn2, e);
}

// The same without the correction, two instructions for six: off by 2^-24 |v| log2(e)
// relative, about as much as a logit of size |v| is by one of its roundings.  For sums,
// those of fp32 too, in which a term is off by 2^-24 log2(e) |v| exp(v) then, no more
// than 0.54 2^-24 of the largest term, and for what is rounded to 16 bits.
__device__ __forceinline__ float exp_roughly(float v) {
  return __builtin_amdgcn_exp2f(v * 0x1.715476p+0f);
}

// A fragment is 16 bytes of a lane: eight 16-bit numbers or four fp32 ones of
// one row, of the contraction's 32 or 16 that a step takes.
template <typename T>
__device__ __forceinline__ f32x4 multiply_add(i32x4 a, i32x4 b, f32x4 c) {
  if constexpr (std::is_same_v<T, BF16>) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  } else if constexpr (std::is_same_v<T, _Float16>) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  } else {
    const f32x4 u = __builtin_bit_cast(f32x4, a), v = __builtin_bit_cast(f32x4, b);
#pragma unroll
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(u[j], v[j], c, 0, 0, 0);
    return c;
  }
}

// fp32 operands as three bf16 numbers each, a = a0 + a1 + a2 with a0 = RN(a), a1 =
// RN(a - a0), a2 = RN(a - a0 - a1): all 24 bits, and the differences are exact.
// A product is then six products of bf16 numbers, exact in fp32 sums:
//   a2 b0 + a0 b2 + a1 b1 + a1 b0 + a0 b1 + a0 b0,
// the smallest first; the three left out come to 2^-24 of a b together, the
// rounding of one product in fp32.  On the matrix cores that is 16 / 6 times the
// rate of the fp32 instruction.  The six follow each other as one long
// contraction.  An infinity in an operand gives NaN in every logit it reaches, and
// so does a number that rounds to one (of 2^128 - 2^119 and more).
struct Fp32Parts {};

template <typename T>
struct HeadType {
  using Operand = T;  // what the matrix instructions take
  using Output = T;
  static constexpr int kPasses = 1;
};

template <>
struct HeadType<Fp32Parts> {
  using Operand = BF16;
  using Output = float;
  static constexpr int kPasses = 6;
};

// The part of each operand in a pass, two bits for each pass.
constexpr uint32_t kPartsOfA = 2 | 0 << 2 | 1 << 4 | 1 << 6 | 0 << 8 | 0 << 10;
constexpr uint32_t kPartsOfB = 0 | 2 << 2 | 1 << 4 | 0 << 6 | 1 << 8 | 0 << 10;

// An operand of a product: `rows` rows of memory of `length` bytes each, `stride`
// bytes apart, all multiples of 16.  Along the contraction a row of memory is a
// row of the operand, across it an element of the contraction.
struct Operand {
  const char* p;
  int64_t stride, rows;
  int64_t length;
  int64_t part;  // Fp32Parts: bytes from one part to the next
};

// Where in the contraction a stage begins: element k of a pass.
struct Walk {
  int64_t k;
  int pass;
};

enum HeadOutput {
  kHeadStatistics = 0,  // of the logits: maximum, sum of exponentials, target
  kHeadGradient = 1,    // the logits' gradient, rounded
  kHeadRounded = 2,     // the product in the operands' type
  kHeadSums = 3,        // the product in fp32, stored or added
};

struct HeadArgs {
  Operand a, b;
  int64_t M, N;     // rows of a and b as operands: rows and columns of the output
  int64_t K;        // elements of the contraction, of which a work-group takes
  int64_t K_split;  // so many (a multiple of a stage's), the blockIdx.y-th
  uint32_t tiles_m, tiles_n;
  // kHeadStatistics and kHeadGradient
  const float* bias;  // of the N classes, or null
  const int64_t* targets;
  int64_t first_class, classes;  // of these N; of the whole head
  float smoothing;
  // kHeadStatistics: [M][stat_tiles] maxima and sums, from tile first_tile on
  f32x2* stats;
  float* sums;     // [M][stat_tiles] sums of logits / classes, or null
  float* target_z; // [M]
  int64_t stat_tiles, first_tile;
  // one tile has all classes: the losses and lse themselves, and no statistics
  float* losses;
  float* losses_lse;
  bool once;  // with few rows: b shall not stay in the caches
  // kHeadGradient
  const float* lse;
  const float* dlosses;
  int64_t dloss_stride;  // 0 or 1
  float* bias_sums;  // [rows of wavefronts][out_stride] sums of g, or null
  // kHeadGradient multiplies by scale[0] and kHeadRounded by scale[1]; null: by
  // 1.  With scale_to > 0 kHeadGradient finds them itself, as loss_scale_kernel
  // does, and leaves them there.
  float* scale;
  float scale_to;
  void* out;
  int64_t out_stride;   // in elements
  int64_t out_part;     // kHeadGradient of Fp32Parts: elements between the parts
  int64_t split_stride; // kHeadSums: elements between the splits' outputs
  bool add;             // kHeadSums: to what is there
};

// load_to_lds for what nobody reads again: past the caches (50000 rows of 8 KiB
// 80 -> 74 us).
__device__ __forceinline__ void load_once_to_lds(i32x4 resource, uint32_t lds, int offset, int k0) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %1, %2, %3 offen nt lds"
      :
      : "s"(lds), "v"(offset), "s"(resource), "s"(k0)
      : "memory");
}

// Bytes of a stage for each row of an operand: eight pieces of 16.  Along the
// contraction it is a line of memory; across it, a stage is as many elements of
// the contraction, each a row of all the tile's rows.
constexpr int kStageRow = 128;

// Brings one operand's share of a stage to LDS, kRows of its rows, and reads
// fragments from there.
//
// Along: LDS holds kRows rows of eight pieces, permuted as staged_piece says.
// Across: kStageRow / sizeof(T) rows, of the contraction, each of kRows
// elements; piece c of row r lies at c ^ swizzle(r).  Sixteen-bit fragments are
// read transposed (two reads of four elements of the contraction each: lanes
// 4 j .. 4 j + 3 of sixteen point to sixteen elements of row j, and lane i
// receives element i of the four rows); fp32 ones are four single reads.
template <typename T, bool kAcross, int kRows, int kWaves, int kTiles, int kPasses, uint32_t kParts,
          bool kMayBeOnce>
struct Stager {
  static constexpr int kE = (int)sizeof(T);
  // Wavefronts that divide the loads; sixteen rows at least for each.  Where that
  // is one, every wavefront loads it all, to the same place.
  static constexpr int kSharers = kRows / 16 < kWaves ? kRows / 16 : kWaves;
  static constexpr int kLoads = kRows / 8 / kSharers;  // of 1,024 bytes, per wavefront and stage
  static constexpr int kStageK = kStageRow / kE;     // elements of the contraction
  static constexpr int kRowBytes = kAcross ? kRows * kE : kStageRow;
  static_assert(kLoads % 2 == 0 && kWaves % kSharers == 0, "sixteen rows to a wavefront");

  int off[kLoads];
  int piece_byte[2];  // along: where in a row this lane's pieces are
  int at[kAcross ? kTiles : 1], at_step[2];
  const char* p;
  int64_t stride, length, part;
  int64_t bytes;  // along: of the tile's rows

  static __device__ __forceinline__ int swizzle(int r) {
    if constexpr (kE == 4) return 4 * ((r >> 2) & 3);
    // the eight rows that 32 lanes read together, over all banks
    if constexpr (kRowBytes >= 256) return 2 * ((r & 3) | ((r >> 3) & 1) << 2);
    return 2 * (((r >> 1) & 1) | ((r >> 3) & 1) << 1);
  }

  static __device__ __forceinline__ i32x4 make_resource(const char* at, int64_t bytes) {
    const uint64_t a = (uint64_t)(uintptr_t)at;
    const int64_t n = bytes < 0 ? 0 : bytes < 0x7FFFFFF0 ? bytes : 0x7FFFFFF0;
    return i32x4{__builtin_amdgcn_readfirstlane((int)(uint32_t)a),
                 __builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32)),
                 __builtin_amdgcn_readfirstlane((int)n), 0x00027000};
  }

  // row0: the tile's first row as an operand; tile0: the wavefront's
  __device__ __forceinline__ void start(const Operand& o, int64_t row0, int wave, int tile0) {
    const int lane = (int)(threadIdx.x & 63u);
    wave %= kSharers;
    stride = o.stride;
    part = o.part;
    if constexpr (kAcross) {
      p = o.p + row0 * kE;
      length = o.length - row0 * kE;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int byte = (wave * kLoads + i) * 1024 + 16 * lane;
        const int r = byte / kRowBytes, c = ((byte % kRowBytes) >> 4) ^ swizzle(r);
        off[i] = 16 * c < length ? r * (int)stride + 16 * c : kOutside;
      }
      const int i = lane & 15, g = lane >> 4;
      if constexpr (kE == 4) {
        const int r = 4 * g;
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
          at[t] = r * kRowBytes + 16 * ((4 * (tile0 + t) + (i >> 2)) ^ swizzle(r)) + 4 * (i & 3);
      } else {
        const int r = 8 * g + (i >> 2);
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
          at[t] = r * kRowBytes + 16 * ((2 * (tile0 + t) + ((i & 3) >> 1)) ^ swizzle(r)) +
                  8 * (i & 1);
      }
    } else {
      p = o.p + row0 * stride;
      length = o.length;
      const int64_t here = min(o.rows - row0, (int64_t)kRows);
      bytes = here > 0 ? (here - 1) * stride + length : 0;
      const int sub = lane / 8;
      piece_byte[0] = 16 * staged_piece(sub, lane % 8);
      piece_byte[1] = 16 * staged_piece(8 + sub, lane % 8);
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int r = (wave * kLoads + i) * 8 + sub;
        off[i] = r < here ? r * (int)stride + piece_byte[i & 1] : kOutside;
      }
      at[0] = (tile0 * 16 + (lane & 15)) * kStageRow;
#pragma unroll
      for (int k = 0; k < 2; ++k) at_step[k] = 16 * staged_piece(lane & 15, 4 * k + (lane >> 4));
    }
  }

  // What the loads of the stage at `w` need; its pass ends before k_end, and
  // elements from there on are zeros.
  struct Stage {
    i32x4 resource;
    int k_byte;
    bool inside[2];
  };

  __device__ __forceinline__ Stage stage(const Walk& w, int64_t k_end) const {
    Stage s;
    const char* from = p;
    if constexpr (kPasses > 1) from += (int64_t)(kParts >> 2 * w.pass & 3u) * part;
    if constexpr (kAcross) {
      // rows beyond the last one lie beyond the resource
      const int64_t left = min(k_end - w.k, (int64_t)kStageK);
      s.resource = make_resource(from + w.k * stride, left > 0 ? (left - 1) * stride + length : 0);
      s.k_byte = 0;
      s.inside[0] = s.inside[1] = true;
    } else {
      s.resource = make_resource(from, bytes);
      s.k_byte = (int)(w.k * kE);
      const int64_t left = (k_end - w.k) * kE;
      s.inside[0] = piece_byte[0] < left;
      s.inside[1] = piece_byte[1] < left;
    }
    return s;
  }

  __device__ __forceinline__ void load(const Stage& s, uint32_t lds, int wave, int i,
                                       bool once) const {
    const uint32_t to = lds + (wave % kSharers * kLoads + i) * 1024;
    const int from = s.inside[i & 1] ? off[i] : kOutside;
    if (kMayBeOnce && once)
      load_once_to_lds(s.resource, to, from, s.k_byte);
    else
      load_to_lds(s.resource, to, from, s.k_byte);
  }

  // Tile t's fragment of step k (of two).
  __device__ __forceinline__ i32x4 fragment(const int8_t* buf, int k, int t) const {
    if constexpr (!kAcross) {
      return *reinterpret_cast<const i32x4*>(buf + at[0] + t * 16 * kStageRow + at_step[k]);
    } else if constexpr (kE == 4) {
      i32x4 v;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[j] = *reinterpret_cast<const int*>(buf + at[t] + (16 * k + j) * kRowBytes);
      return v;
    } else {
      typedef __attribute__((address_space(3))) i16x4 Lds;
      const auto* q =
          (const __attribute__((address_space(3))) int8_t*)buf + at[t] + 32 * k * kRowBytes;
      const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds*)q));
      const u32x2 hi = __builtin_bit_cast(
          u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds*)(q + 4 * kRowBytes)));
      return i32x4{(int)lo[0], (int)lo[1], (int)hi[0], (int)hi[1]};
    }
  }
};

// Values of a wavefront's tiles, in the accumulators' layout, to rows of out:
// through the wavefront's piece of LDS, 64 rows at a time, and out as 16-byte
// stores along rows, as OutputTile does.  value(i, j, c): of row 16 i + lane %
// 16, column 16 j + 4 (lane / 16) + c.
template <typename T, int kTM, int kTN>
struct ValueTile {
  static constexpr int kTokens = kTM < 4 ? 16 * kTM : 64;
  static constexpr int kPitch = 16 * kTN * (int)sizeof(T) + 16;
  static constexpr int kBytes = kTokens * kPitch;

  template <typename F>
  static __device__ __forceinline__ void store(F&& value, int8_t* lds, T* out, int64_t out_stride,
                                               int64_t m0, int64_t n0, int64_t M, int64_t N) {
    constexpr int kE = 16 / (int)sizeof(T);  // outputs per 16-byte store
    constexpr int kLanes = 16 * kTN / kE;    // lanes along a row
    constexpr int kRowsAtOnce = 64 / kLanes < kTokens ? 64 / kLanes : kTokens;
    constexpr int kTiles = kTokens / 16;
    const int lane = (int)(threadIdx.x & 63u);
    const int64_t n = n0 + kE * (lane % kLanes);
    // (a narrow tile's rows need fewer lanes than there are)
    const bool idle = lane / kLanes >= kRowsAtOnce;
    const int left = idle ? 0 : (int)min(max(N - n, (int64_t)0), (int64_t)kE);
#pragma unroll
    for (int i0 = 0; i0 < kTM; i0 += kTiles) {
#pragma unroll
      for (int i = 0; i < kTiles; ++i)
#pragma unroll
        for (int j = 0; j < kTN; ++j) {
          float v[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) v[c] = value(i0 + i, j, c);
          int8_t* at = lds + (16 * i + (lane & 15)) * kPitch +
                       (16 * j + 4 * (lane >> 4)) * (int)sizeof(T);
          if constexpr (sizeof(T) == 4)
            *reinterpret_cast<f32x4*>(at) = f32x4{v[0], v[1], v[2], v[3]};
          else
            *reinterpret_cast<u32x2*>(at) =
                u32x2{two_halves<T>(v[0], v[1]), two_halves<T>(v[2], v[3])};
        }
      // one wavefront's LDS operations take effect in their order
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
#pragma unroll
      for (int i = 0; i < kTokens / kRowsAtOnce; ++i) {
        const int r = i * kRowsAtOnce + lane / kLanes;
        const int64_t m = m0 + 16 * i0 + r;
        const u32x4 v = *reinterpret_cast<const u32x4*>(lds + (idle ? 0 : r) * kPitch +
                                                        16 * (lane % kLanes));
        T* to = out + m * out_stride + n;
        if (m < M && left == kE)
          *reinterpret_cast<u32x4_any*>(to) = v;
        else if (m < M && left > 0)
          OutputTile<T, kTM, kTN>::store_part(v, to, left);
      }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    }
  }
};

// Sum or maximum over the four lanes that hold columns of the same row.
template <typename F>
__device__ __forceinline__ float fold_row(float v, F fold) {
  auto bits = [](float x) { return __builtin_bit_cast(uint32_t, x); };
  auto number = [](uint32_t x) { return __builtin_bit_cast(float, x); };
  const auto r = __builtin_amdgcn_permlane16_swap(bits(v), bits(v), false, false);
  v = fold(number(r[0]), number(r[1]));
  const auto q = __builtin_amdgcn_permlane32_swap(bits(v), bits(v), false, false);
  return fold(number(q[0]), number(q[1]));
}

__device__ __forceinline__ TileAt head_tile_at(uint32_t block, const HeadArgs& p) {
  ProductArgs q{};
  q.tiles_m = p.tiles_m;
  q.tiles_n = p.tiles_n;
  return tile_at(block, q);
}

constexpr float kMinusInfinity = -__builtin_inff();

// A row's lse and loss from the maximum of its logits, the sum of exponentials
// above it, the mean of the logits and the target's.  The loss is made of differences
// from the maximum, not of lse, whose rounding is that of a number of the logits'
// size (logits near 20: steps of 2e-6, where a loss may be 1e-5).
struct LossOf {
  float lse, loss;
};

__device__ __forceinline__ LossOf loss_of(float top, float sum, float mean, bool counts,
                                          float target, float smoothing) {
  LossOf l;
  l.lse = top + logf(sum);
  l.loss = 0.0f;
  if (counts) {
    // (where the target has no part, it may be infinitely low)
    float below = smoothing < 1.0f ? (1.0f - smoothing) * (top - target) : 0.0f;
    if (smoothing > 0.0f) below += smoothing * (top - mean);
    l.loss = below + logf(sum);
  }
  return l;
}

// What brings the largest finite |dloss| of the rows that count to `to`, and back.
// Rounded to 16 bits as they are, the gradients of a mean loss would all be off by
// the rounding of 1 / rows, the same way (4096 rows of bf16: 3.0e-3 of dx against
// 1.7e-3, dx's own rounding); and fp16 holds those of classes of small probability
// only if they are large.  An ignored row's gradients are zeros, and its dloss may
// be anything: it has no say.
struct Scale {
  float up, down;
};

// By all threads of the work-group; s_top: a word for each wavefront.  Of a dloss
// for all rows (stride 0) no target is looked at.
template <int kThreads>
__device__ __forceinline__ Scale find_scale(const float* dlosses, int64_t stride,
                                            const int64_t* targets, int64_t classes, int64_t rows,
                                            float to, uint32_t* s_top) {
  uint32_t top = 0;
  if (stride == 0) rows = min(rows, (int64_t)1);
  // four loads at a time on their way
  for (int64_t i = threadIdx.x; i < rows; i += 4 * kThreads) {
    uint32_t v[4];
    int64_t y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t at = min(i + j * kThreads, rows - 1);
      v[j] = __builtin_bit_cast(uint32_t, dlosses[at * stride]) & 0x7FFFFFFFu;
      y[j] = stride != 0 ? targets[at] : 0;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      top = max(top, v[j] < 0x7F800000u && (uint64_t)y[j] < (uint64_t)classes ? v[j] : 0u);
  }
  top = group_max<64>(top);
  if ((threadIdx.x & 63u) == 0) s_top[threadIdx.x >> 6] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) top = max(top, s_top[w]);
  // numbers so small that the inverse would overflow are scaled by less
  const float largest = fmaxf(__builtin_bit_cast(float, top), 0x1p-100f);
  return {to / largest, largest / to};
}

// A tile of kBM x kBN outputs per work-group of kWM x kWN wavefronts, kStages
// stages of 128 bytes of the contraction on their way, as in
// product_tile_kernel: between the products of a step stand, one at a time, the
// reads of the next step's fragments and the loads of a later stage.
//
// kGroups: sets of wavefronts that divide the contraction, each with stages of its
// own; their sums are joined in LDS.  A small tile's stage is a chain of waits
// (barrier, reads, products) several times as long as its products, and where a
// compute unit has one tile alone, others shall fill them (16x64 tiles of 8192
// elements, one to a unit, with one group / four: bf16 34 / 24 us, fp32 90 / 57).
template <typename T, int kOutput, bool kAcrossA, bool kAcrossB, int kBM, int kBN, int kWM, int kWN,
          int kStages, int kGroups = 1>
struct HeadTile {
  static constexpr int kWaves = kWM * kWN, kTM = kBM / kWM / 16, kTN = kBN / kWN / 16;
  static constexpr int kStageBytes = (kBM + kBN) * kStageRow;
  using Type = HeadType<T>;
  using Element = typename Type::Operand;
  static constexpr int kPasses = Type::kPasses;
  // with few rows of a, b passes by once
  using StagerA = Stager<Element, kAcrossA, kBM, kWaves, kTM, kPasses, kPartsOfA, false>;
  using StagerB = Stager<Element, kAcrossB, kBN, kWaves, kTN, kPasses, kPartsOfB,
                         kBM == 16 && kPasses == 1>;
  // what leaves: products in the operands' type, gradients as the next products
  // take them
  using Out = std::conditional_t<kOutput == kHeadGradient, Element, typename Type::Output>;
  using Tile = ValueTile<Out, kTM, kTN>;
  static constexpr int kLoadsA = StagerA::kLoads, kLoads = kLoadsA + StagerB::kLoads;
  static constexpr int kStageK = StagerA::kStageK, kSteps = 2;
  static constexpr int kOutBytes = kWaves * Tile::kBytes;
  static constexpr int kGroupBytes = kStages * kStageBytes;
  static constexpr int kMainBytes =
      kGroups * kGroupBytes > kOutBytes ? kGroups * kGroupBytes : kOutBytes;
  static constexpr int kThreads = 64 * kWaves * kGroups;
  // what the logits need beside: bias, lse, dlosses, targets, a word for each
  // wavefront
  static constexpr bool kSides = kOutput == kHeadStatistics || kOutput == kHeadGradient;
  static constexpr int kSideM = kBM < 64 ? 64 : kBM;  // loads bring 64 words
  static constexpr int kSideBytes = kSides ? 4 * (kBN + 4 * kSideM + 64) : 0;
  static constexpr int kLds = kMainBytes + kSideBytes;

  // The block-th tile, the split-th part of the contraction.
  static __device__ __forceinline__ void run(const HeadArgs& p, uint32_t block, uint32_t split,
                                             int8_t* s_stages) {
    const int lane = (int)(threadIdx.x & 63u);
    const int wave_of_all = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int wave = wave_of_all % kWaves, group = wave_of_all / kWaves;
    const bool first_group = kGroups == 1 || group == 0;

    const TileAt tile = head_tile_at(block, p);
    const int64_t m0 = (int64_t)tile.m * kBM, n0 = (int64_t)tile.n * kBN;
    // the split's part of the contraction and the group's part of that: the same
    // number of stages for every group, zeros beyond k_end
    int64_t k_begin = (int64_t)split * p.K_split;
    const int64_t k_end = min(k_begin + p.K_split, p.K);
    const int pass_stages =
        k_end > k_begin
            ? (int)((k_end - k_begin + kGroups * kStageK - 1) / (kGroups * kStageK))
            : 0;
    k_begin += (int64_t)group * pass_stages * kStageK;
    const int64_t pass_end = k_begin + (int64_t)pass_stages * kStageK;
    StagerA sa;
    StagerB sb;
    sa.start(p.a, m0, wave, (wave / kWN) * kTM);
    sb.start(p.b, n0, wave, (wave % kWN) * kTN);
    const uint32_t lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)s_stages;
    int8_t* const s_group = s_stages + group * kGroupBytes;
    struct Next {
      typename StagerA::Stage a;
      typename StagerB::Stage b;
    };
    Walk walk = {k_begin, 0};
    // the next stage to load
    auto next_of = [&]() {
      const Next next = {sa.stage(walk, k_end), sb.stage(walk, k_end)};
      walk.k += kStageK;
      if (kPasses > 1 && walk.k >= pass_end) {
        // (beyond the last pass comes the first element again, for nothing)
        walk.k = k_begin;
        ++walk.pass;
      }
      return next;
    };
    auto issue = [&](int stage, int i, const Next& next) {
      const uint32_t to = lds + group * kGroupBytes + stage * kStageBytes;
      if (i < kLoadsA)
        sa.load(next.a, to, wave, i, false);
      else
        sb.load(next.b, to + kBM * kStageRow, wave, i - kLoadsA, p.once);
    };
    i32x4 fa[2][kTM], fb[2][kTN];
    auto fetch = [&](const int8_t* buf, int k, int slot, int i) {
      if (i < kTN)
        fb[slot][i] = sb.fragment(buf + kBM * kStageRow, k, i);
      else
        fa[slot][i - kTN] = sa.fragment(buf, k, i - kTN);
    };
    f32x4 acc[kTM][kTN] = {};

    // They go first and have landed with the first stage: fetched after the last
    // product they would keep the output waiting for memory once more.
    const float* const s_bias = reinterpret_cast<const float*>(s_stages + kMainBytes);
    const float *const s_lse = s_bias + kBN, *const s_dloss = s_lse + kSideM;
    const int64_t* const s_target = reinterpret_cast<const int64_t*>(s_dloss + kSideM);
    if (kSides && first_group) {
      auto words = [&](const void* from, int64_t first, int64_t count, int64_t size, int to) {
        // `count` words of `size` from the first one on, zeros behind them
        const int64_t here = from != nullptr ? max(count - first, (int64_t)0) : 0;
        const i32x4 r = StagerA::make_resource((const char*)from + 4 * first, 4 * min(here, size));
        for (int c = wave; c < ((int)size + 63) / 64; c += kWaves)
          load_words_to_lds(r, lds + kMainBytes + 4 * to + 256 * c, 256 * c + 4 * lane);
      };
      words(p.bias, n0, p.N, kBN, 0);
      if constexpr (kOutput == kHeadGradient) {
        words(p.lse, m0, p.M, kBM, kBN);
        if (p.dloss_stride != 0) words(p.dlosses, m0, p.M, kBM, kBN + kSideM);
      }
      words(p.targets, 2 * m0, 2 * p.M, 2 * kBM, kBN + 2 * kSideM);
    }
#pragma unroll
    for (int s = 0; s < kStages; ++s) {
      const Next next = next_of();
#pragma unroll
      for (int i = 0; i < kLoads; ++i) issue(s, i, next);
    }
    // numbers that the output takes are read here, like the words above
    Scale scale = {1.0f, 1.0f};
    float same_dloss = 0.0f;
    if constexpr (kOutput == kHeadRounded) {
      if (p.scale != nullptr) scale.down = p.scale[1];
    }
    if constexpr (kOutput == kHeadGradient) {
      if (p.dloss_stride == 0) same_dloss = p.dlosses[0];
      if (p.scale_to > 0.0f) {
        scale = find_scale<kThreads>(
            p.dlosses, p.dloss_stride, p.targets, p.classes, p.M, p.scale_to,
            reinterpret_cast<uint32_t*>(s_stages + kMainBytes) + kBN + 4 * kSideM);
        if (block == 0 && threadIdx.x == 0) {
          p.scale[0] = scale.up;
          p.scale[1] = scale.down;
        }
      } else if (p.scale != nullptr) {
        scale = {p.scale[0], p.scale[1]};
      }
    }
    wait_loads<(kStages - 1) * kLoads>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
#pragma unroll
    for (int i = 0; i < kTM + kTN; ++i) fetch(s_group, 0, 0, i);
    int stage = 0;
    for (int left = kPasses * pass_stages; left > 0; --left) {
      const int after = stage + 1 == kStages ? 0 : stage + 1;
      static_for<kSteps>([&](auto step) {
        constexpr int k = decltype(step)::value;
        constexpr bool kLast = k + 1 == kSteps;
        constexpr int kProducts = kTM * kTN, kReads = kTM + kTN, kNewLoads = kLast ? kLoads : 0;
        constexpr int kOthers = kReads + kNewLoads;
        const int8_t* from = s_group + (kLast ? after : stage) * kStageBytes;
        Next next;
        if constexpr (kLast) {
          // this wavefront's loads of the next stage have landed and its reads
          // of this one are done; beyond the barrier, everyone's are: the next
          // stage may be read, and this one's place be filled again
          wait_loads<(kStages - 2) * kLoads>();
          asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
          __builtin_amdgcn_s_barrier();
          asm volatile("" ::: "memory");
          next = next_of();
        }
        __builtin_amdgcn_sched_barrier(0);
        static_for<kProducts>([&](auto product) {
          constexpr int t = decltype(product)::value;
          // the other operations, spread evenly over all products but two, the
          // loads evenly among the reads
          constexpr int kSpan = kProducts > 4 ? kProducts - 2 : kProducts;
          constexpr int kFrom = (t * kOthers + kSpan - 1) / kSpan;
          constexpr int kTo = ((t + 1) * kOthers + kSpan - 1) / kSpan;
          constexpr int kEnd = kTo < kOthers ? kTo : kOthers;
          static_for<(kFrom < kEnd ? kEnd - kFrom : 0)>([&](auto other) {
            constexpr int o = kFrom + decltype(other)::value;
            constexpr int kBefore = o * kNewLoads / kOthers;
            if constexpr ((o + 1) * kNewLoads / kOthers > kBefore)
              issue(stage, kBefore, next);
            else
              fetch(from, kLast ? 0 : k + 1, (k + 1) & 1, o - kBefore);
          });
          __builtin_amdgcn_sched_barrier(0);
          acc[t / kTN][t % kTN] =
              multiply_add<Element>(fb[k & 1][t % kTN], fa[k & 1][t / kTN], acc[t / kTN][t % kTN]);
          __builtin_amdgcn_sched_barrier(0);
        });
      });
      stage = after;
    }
    // loads of stages beyond the end (they bring zeros) end before LDS is used
    // again
    wait_loads<0>();
    __syncthreads();
    if constexpr (kGroups > 1) {
      // in the groups' order
      static_assert((kGroups - 1) * kWaves * kTM * kTN * 1024 <= kMainBytes, "room for the sums");
      f32x4* s_sums = reinterpret_cast<f32x4*>(s_stages) + wave * kTM * kTN * 64 + lane;
      constexpr int kOfGroup = kWaves * kTM * kTN * 64;
      if (!first_group) {
#pragma unroll
        for (int i = 0; i < kTM; ++i)
#pragma unroll
          for (int j = 0; j < kTN; ++j)
            s_sums[(group - 1) * kOfGroup + (i * kTN + j) * 64] = acc[i][j];
      }
      __syncthreads();
      if (first_group) {
#pragma unroll
        for (int g = 1; g < kGroups; ++g)
#pragma unroll
          for (int i = 0; i < kTM; ++i)
#pragma unroll
            for (int j = 0; j < kTN; ++j)
              acc[i][j] += s_sums[(g - 1) * kOfGroup + (i * kTN + j) * 64];
      }
      __syncthreads();
    }

    const int m_wave = (wave / kWN) * kTM * 16, n_wave = (wave % kWN) * kTN * 16;
    const int64_t m_lane = m0 + m_wave + (lane & 15), n_lane = n0 + n_wave + 4 * (lane >> 4);
    int8_t* const own = s_stages + wave * Tile::kBytes;
    // this lane's columns that exist: 16 j + c < columns
    const int columns = (int)min(max(p.N - n_lane, (int64_t)0), (int64_t)kBN);
    // the number of a row's target among them, -1 if it is elsewhere
    auto target_of = [&](int64_t y) {
      const int64_t t = y - p.first_class - n_lane;
      return t >= 0 && t < columns ? (int)t : -1;
    };

    if constexpr (kOutput == kHeadSums) {
      if (!first_group) return;
      float* out = (float*)p.out + (int64_t)split * p.split_stride;
#pragma unroll
      for (int i = 0; i < kTM; ++i)
#pragma unroll
        for (int j = 0; j < kTN; ++j) {
          const int64_t m = m_lane + 16 * i, n = n_lane + 16 * j;
          // rows have room for whole vectors of four
          if (m < p.M && n < p.N) {
            f32x4* to = reinterpret_cast<f32x4*>(out + m * p.out_stride + n);
            *to = p.add ? *to + acc[i][j] : acc[i][j];
          }
        }
    } else if constexpr (kOutput == kHeadRounded) {
      if (!first_group) return;
      Tile::store([&](int i, int j, int c) { return acc[i][j][c] * scale.down; }, own,
                  (Out*)p.out, p.out_stride, m0 + m_wave, n0 + n_wave, p.M, p.N);
    } else {
      // The logits.  What follows is 128 elements a lane in the largest tile, so it
      // counts by the instruction: bias, the edge of the classes and targets are
      // looked at only where there are any (8192x50000x4096 bf16 2.55 -> 2.45 ms);
      // but smoothing's sum of the logits selects by the edge in every tile.
      if (p.bias != nullptr && first_group) {
#pragma unroll
        for (int j = 0; j < kTN; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float bias = s_bias[n_wave + 4 * (lane >> 4) + 16 * j + c];
#pragma unroll
            for (int i = 0; i < kTM; ++i) acc[i][j][c] += bias;
          }
      }
      const bool edge = n0 + kBN > p.N;
      if constexpr (kOutput == kHeadStatistics) {
        // of the work-group's rows in each column of wavefronts
        float* s_top = reinterpret_cast<float*>(s_stages);
        float* s_sum = s_top + kWN * kBM;
        float* s_all = s_sum + kWN * kBM;
        float* s_z = s_all + kWN * kBM;
        const int slot = (wave % kWN) * kBM + m_wave + (lane & 15);
        if (first_group) {
          if (p.smoothing > 0.0f) {
            // the mean's share: a sum would overflow where classes are masked by the
            // lowest number
            const float share = 1.0f / (float)p.classes;
#pragma unroll
            for (int i = 0; i < kTM; ++i) {
              float all = 0.0f;
#pragma unroll
              for (int j = 0; j < kTN; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                  all = __builtin_fmaf(16 * j + c < columns ? acc[i][j][c] : 0.0f, share, all);
              all = fold_row(all, [](float x, float y) { return x + y; });
              if ((lane >> 4) == 0) s_all[slot + 16 * i] = all;
            }
          }
          if (edge) {
#pragma unroll
            for (int j = 0; j < kTN; ++j)
#pragma unroll
              for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int i = 0; i < kTM; ++i)
                  acc[i][j][c] = 16 * j + c < columns ? acc[i][j][c] : kMinusInfinity;
          }
#pragma unroll
          for (int i = 0; i < kTM; ++i) {
            const int64_t m = m_lane + 16 * i;
            float top = kMinusInfinity;
#pragma unroll
            for (int j = 0; j < kTN; ++j)
#pragma unroll
              for (int c = 0; c < 4; ++c) top = fmaxf(top, acc[i][j][c]);
            top = fold_row(top, [](float x, float y) { return fmaxf(x, y); });
            // a row of which nothing is left has no exponentials
            const float base = top == kMinusInfinity ? 0.0f : top;
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < kTN; ++j)
#pragma unroll
              for (int c = 0; c < 4; ++c) sum += exp_roughly(acc[i][j][c] - base);
            sum = fold_row(sum, [](float x, float y) { return x + y; });
            if ((lane >> 4) == 0) {
              s_top[slot + 16 * i] = top;
              s_sum[slot + 16 * i] = sum;
            }
            const int target = m < p.M ? target_of(s_target[m_wave + 16 * i + (lane & 15)]) : -1;
            if (__any(target >= 0)) {
#pragma unroll
              for (int j = 0; j < kTN; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                  if (target == 16 * j + c) {
                    if (p.losses != nullptr)
                      s_z[m_wave + 16 * i + (lane & 15)] = acc[i][j][c];
                    else
                      p.target_z[m] = acc[i][j][c];
                  }
            }
          }
        }
        __syncthreads();
        for (int r = (int)threadIdx.x; r < kBM; r += kThreads) {
          const int64_t m = m0 + r;
          if (m >= p.M) break;
          float top = s_top[r];
#pragma unroll
          for (int w = 1; w < kWN; ++w) top = fmaxf(top, s_top[w * kBM + r]);
          const float base = top == kMinusInfinity ? 0.0f : top;
          float sum = 0.0f, all = 0.0f;
#pragma unroll
          for (int w = 0; w < kWN; ++w) {
            sum += s_sum[w * kBM + r] * exp_below(s_top[w * kBM + r] - base);
            if (p.smoothing > 0.0f) all += s_all[w * kBM + r];
          }
          if (p.losses != nullptr) {
            const int64_t y = s_target[r];
            const bool counts = y >= 0 && y < p.classes;
            const LossOf l =
                loss_of(top, sum, all, counts, counts ? s_z[r] : 0.0f, p.smoothing);
            p.losses_lse[m] = l.lse;
            p.losses[m] = l.loss;
            continue;
          }
          const int64_t at = m * p.stat_tiles + p.first_tile + tile.n;
          p.stats[at] = f32x2{top, sum};
          if (p.sums != nullptr) p.sums[at] = all;
        }
      } else {
        if (!first_group) return;
        const float even = p.smoothing / (float)p.classes;
        // what is rounded to 16 bits needs no exponential of 24
        constexpr bool kRoughly = sizeof(typename Type::Output) == 2;
#pragma unroll
        for (int i = 0; i < kTM; ++i) {
          const int64_t m = m_lane + 16 * i;
          const int at = m_wave + 16 * i + (lane & 15);
          const int64_t y = s_target[at];
          const float lse = s_lse[at];
          const float dloss = (p.dloss_stride != 0 ? s_dloss[at] : same_dloss) * scale.up;
          const bool counts = m < p.M && y >= 0 && y < p.classes;
          const int target = target_of(y);
#pragma unroll
          for (int j = 0; j < kTN; ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const float v = acc[i][j][c] - lse;
              acc[i][j][c] = (kRoughly ? exp_roughly(v) : exp_below(v)) - even;
            }
          if (__any(target >= 0)) {
#pragma unroll
            for (int j = 0; j < kTN; ++j)
#pragma unroll
              for (int c = 0; c < 4; ++c)
                if (target == 16 * j + c) acc[i][j][c] -= 1.0f - p.smoothing;
          }
#pragma unroll
          for (int j = 0; j < kTN; ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[i][j][c] = counts ? acc[i][j][c] * dloss : 0.0f;
        }
        if (edge) {
#pragma unroll
          for (int j = 0; j < kTN; ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int i = 0; i < kTM; ++i)
                acc[i][j][c] = 16 * j + c < columns ? acc[i][j][c] : 0.0f;
        }
        if (p.bias_sums != nullptr) {
          // a wavefront's rows, then the sixteen lanes that hold a column
          float* to = p.bias_sums + ((int64_t)tile.m * kWM + wave / kWN) * p.out_stride;
#pragma unroll
          for (int j = 0; j < kTN; ++j) {
            f32x4 sum = acc[0][j];
#pragma unroll
            for (int i = 1; i < kTM; ++i) sum += acc[i][j];
#pragma unroll
            for (int c = 0; c < 4; ++c) sum[c] = group_sum<16>(sum[c]) * scale.down;
            if ((lane & 15) == 0 && n_lane + 16 * j < p.out_stride)
              *reinterpret_cast<f32x4*>(to + n_lane + 16 * j) = sum;
          }
        }
        // to the end of the row of memory: what lies beyond the classes is zero,
        // and takes part in the next product
        Out* out = (Out*)p.out;
#pragma unroll 1
        for (int part = 0; part < (kPasses > 1 ? 3 : 1); ++part, out += p.out_part) {
          Tile::store([&](int i, int j, int c) { return acc[i][j][c]; }, own, out, p.out_stride,
                      m0 + m_wave, n0 + n_wave, p.M, p.out_stride);
          if constexpr (kPasses > 1) {
            // what the part leaves of each, exactly
#pragma unroll
            for (int i = 0; i < kTM; ++i)
#pragma unroll
              for (int j = 0; j < kTN; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                  acc[i][j][c] -= bf16_to_float(float_to_bf16(acc[i][j][c]));
          }
        }
      }
    }
  }
};

template <typename T, int kOutput, bool kAcrossA, bool kAcrossB, int kBM, int kBN, int kWM, int kWN,
          int kStages, int kGroups = 1>
__global__ __launch_bounds__(64 * kWM * kWN * kGroups, 2) void head_kernel(HeadArgs p) {
  using Head = HeadTile<T, kOutput, kAcrossA, kAcrossB, kBM, kBN, kWM, kWN, kStages, kGroups>;
  __shared__ __align__(1024) int8_t s_stages[Head::kLds];
  Head::run(p, blockIdx.x, blockIdx.y, s_stages);
}

// Both products with g in one launch, for sizes where one alone leaves compute
// units idle, and the sums of dbias: first the tiles of the product with the longer
// contraction, so that none of them starts late, then the other's; the last
// work-groups have 64 classes each.
struct HeadPairArgs {
  HeadArgs dx, dw;
  uint32_t dx_blocks, dw_blocks;
  bool dw_first;
  const float* bias_sums;  // [bias_rows][pitch]
  int64_t pitch;
  int32_t bias_rows;
  float* dbias;
};

template <typename T, int kBM, int kBN, int kWM, int kWN, int kStages, int kGroups = 1>
__global__ __launch_bounds__(64 * kWM * kWN * kGroups, 2) void head_pair_kernel(HeadPairArgs p) {
  using Dx = HeadTile<T, kHeadRounded, false, true, kBM, kBN, kWM, kWN, kStages, kGroups>;
  using Dw = HeadTile<T, kHeadRounded, true, true, kBM, kBN, kWM, kWN, kStages, kGroups>;
  __shared__ __align__(1024) int8_t s_stages[Dx::kLds > Dw::kLds ? Dx::kLds : Dw::kLds];
  const uint32_t tiles = p.dx_blocks + p.dw_blocks, first = p.dw_first ? p.dw_blocks : p.dx_blocks;
  if (blockIdx.x < tiles && (blockIdx.x < first) != p.dw_first) {
    Dx::run(p.dx, blockIdx.x - (p.dw_first ? first : 0u), 0, s_stages);
  } else if (blockIdx.x < tiles) {
    Dw::run(p.dw, blockIdx.x - (p.dw_first ? 0u : first), 0, s_stages);
  } else {
    // 64 classes: a wavefront takes every kWaves-th row of partial sums
    constexpr int kWaves = kWM * kWN * kGroups;
    float* s_sum = reinterpret_cast<float*>(s_stages);
    const int lane = (int)(threadIdx.x & 63u), wave = (int)(threadIdx.x >> 6);
    const int64_t n = (int64_t)(blockIdx.x - tiles) * 64 + lane;
    float sum = 0.0f;
    if (n < p.dw.M)
      for (int32_t r = wave; r < p.bias_rows; r += kWaves) sum += p.bias_sums[r * p.pitch + n];
    s_sum[wave * 64 + lane] = sum;
    __syncthreads();
    if (wave == 0 && n < p.dw.M) {
#pragma unroll
      for (int w = 1; w < kWaves; ++w) sum += s_sum[w * 64 + lane];
      p.dbias[n] = sum;
    }
  }
}

}  // namespace fn
