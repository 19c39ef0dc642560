// row_kernels.hpp -- kernels that work on rows of D elements: RMS norm of
// x + residual with its output in 8 bits or in the input's type, the norm's
// gradients, and the quantisation of rows to 8 bits.
//
// Mathematics of one row:
//   h = RN_T(x + residual)                        (RN_T: round to the type)
//   rstd = 1 / sqrt(mean(h^2) + eps)              (NaN if the mean is not finite)
//   norm:      out_j = RN_T(h_j rstd w_j)
//   8 bits:    t_j = RN32(h_j w_j), A = max |t_j|,
//              code_j = rint(RN32(t_j RN32(127 RN32(1 / A)))), scale = A rstd / 127
// rstd is a common factor of the row, so it cancels in code_j: the codes need
// the maximum alone, which no order of evaluation changes, and h_j w_j is
// exact in fp32 for 16-bit types.  The sum of squares and the maximum are
// taken in the same pass, so one reduction serves both.  One reciprocal for a
// row, instead of a division for each element, costs a code that may fall to
// either side where 127 t_j / A is within 127 * 3 * 2^-24 of half way.
//
// Every element is read once and written once: a row stays in registers
// between the reduction and the output (rows of more than 32,768 elements
// are read twice).  The kernels are bound by memory: 50176x768 fp16 with a
// residual to codes 47.8 us (5.6 TB/s), 16384x8192 bf16 to bf16 176 us (6.1),
// its gradients 175 us (6.1), 8192x4096 bf16 quantised 18.3 us (5.5).
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

namespace fn {

struct BF16 {
  uint16_t bits;
};

enum RowMode { kRowNorm = 0, kRowNormQ8 = 1, kRowQuantize = 2 };

struct RowArgs {
  const void* x;
  const void* residual;  // or null
  const void* weight;    // null when quantising
  void* sum;             // null without a residual
  void* out;             // kRowNorm
  int8_t* codes;         // kRowNormQ8, kRowQuantize
  float* scales;
  float* rstd;  // or null
  int64_t rows;
  int64_t x_stride, residual_stride, sum_stride, out_stride, codes_stride;  // in elements
  int32_t width;
  float eps;
};

// n / by for any 32-bit n, from the upper half of its product with
// floor(2^32 (2^l - by) / by) + 1, l = ceil(log2 by), which is 2^(32 + l) / by
// rounded up without its top bit (Granlund and Montgomery 1994).
struct Division {
  uint32_t by, magic, shift;  // shift = l - 1; by = 1 takes no division
};

inline Division division_by(uint32_t by) {
  if (by <= 1) return {1, 0, 0};
  const int l = 32 - __builtin_clz(by - 1);
  return {by, (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << l) - by)) / by + 1),
          (uint32_t)(l - 1)};
}

__device__ __forceinline__ uint32_t quotient(uint32_t n, const Division& d) {
  const uint32_t t = __umulhi(n, d.magic);
  return d.by == 1 ? n : (((n - t) >> 1) + t) >> d.shift;
}

// ------------------------------------------------------------- vector access
// Eight consecutive elements, at any alignment of the element's size: the
// hardware's global loads and stores take unaligned addresses.  Rows are met
// once, so both are non-temporal (16384x8192 bf16: norm 182 -> 173 us, to
// codes 159 -> 149 us, backward 191 -> 179 us).  Not all loads of fp32: a lane's
// eight numbers are two loads, whose lines the second one finds in the cache only
// if they may stay there (layer norm of 3001x2243 21.3 -> 12.5 us, 12000x1000 with a
// residual 49 -> 36); but many wide rows are faster past the caches (load_once: the
// rows, not the weight, which every work-group reads; see once_rows and
// once_backward).

typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float bf16_to_float(uint32_t bits) {
  return __builtin_bit_cast(float, bits << 16);
}

// float -> bfloat16 bits, to nearest even (the type's own conversion
// instruction); NaN stays NaN
__device__ __forceinline__ uint32_t float_to_bf16(float v) {
  return __builtin_bit_cast(uint16_t, (__bf16)v);
}

template <typename T>
struct Vec8;  // eight elements as they lie in memory

template <>
struct Vec8<float> {
  u32x4 a, b;
  __device__ __forceinline__ void zero() { a = b = u32x4{0, 0, 0, 0}; }
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const u32x4_any*>(p);
    b = *reinterpret_cast<const u32x4_any*>(p + 4);
  }
  __device__ __forceinline__ void load_once(const float* p) {
    a = __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(p));
    b = __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(p + 4));
  }
  __device__ __forceinline__ void load_some(const float* p, int n) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      a[j] = j < n ? __builtin_bit_cast(uint32_t, p[j]) : 0u;
      b[j] = j + 4 < n ? __builtin_bit_cast(uint32_t, p[j + 4]) : 0u;
    }
  }
  // element j becomes element j + n (n = 0..8), zeros from the top
  __device__ __forceinline__ void drop(int n) {
    const u32x4 none = {0, 0, 0, 0};
    if (n & 8) a = b = none;
    if (n & 4) {
      a = b;
      b = none;
    }
    if (n & 2) {
      a = u32x4{a[2], a[3], b[0], b[1]};
      b = u32x4{b[2], b[3], 0, 0};
    }
    if (n & 1) {
      a = u32x4{a[1], a[2], a[3], b[0]};
      b = u32x4{b[1], b[2], b[3], 0};
    }
  }
  __device__ __forceinline__ float get(int j) const {
    return __builtin_bit_cast(float, j < 4 ? a[j & 3] : b[j & 3]);
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      a[j] = __builtin_bit_cast(uint32_t, v[j]);
      b[j] = __builtin_bit_cast(uint32_t, v[j + 4]);
    }
  }
  __device__ __forceinline__ void store(float* p) const {
    __builtin_nontemporal_store(a, reinterpret_cast<u32x4_any*>(p));
    __builtin_nontemporal_store(b, reinterpret_cast<u32x4_any*>(p + 4));
  }
  __device__ __forceinline__ void store_some(float* p, int n) const {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) p[j] = get(j);
  }
};

// the 16-bit types differ in their conversions alone
template <typename T>
struct Half8 {
  u32x4 a;
  __device__ __forceinline__ void zero() { a = u32x4{0, 0, 0, 0}; }
  __device__ __forceinline__ void load(const T* p) {
    a = __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(p));
  }
  __device__ __forceinline__ void load_some(const T* p, int n) {
    const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t lo = 2 * j < n ? q[2 * j] : 0u;
      const uint32_t hi = 2 * j + 1 < n ? q[2 * j + 1] : 0u;
      a[j] = lo | hi << 16;
    }
  }
  __device__ __forceinline__ void drop(int n) {
    if (n & 8) a = u32x4{0, 0, 0, 0};
    if (n & 4) a = u32x4{a[2], a[3], 0, 0};
    if (n & 2) a = u32x4{a[1], a[2], a[3], 0};
    if (n & 1)
      a = u32x4{a[0] >> 16 | a[1] << 16, a[1] >> 16 | a[2] << 16, a[2] >> 16 | a[3] << 16,
                a[3] >> 16};
  }
  __device__ __forceinline__ void drop_last(bool yes) {
    a[3] &= yes ? 0xFFFFu : ~0u;
  }
  __device__ __forceinline__ uint32_t bits(int j) const { return (a[j >> 1] >> (16 * (j & 1))) & 0xFFFFu; }
  __device__ __forceinline__ void store(T* p) const {
    __builtin_nontemporal_store(a, reinterpret_cast<u32x4_any*>(p));
  }
  __device__ __forceinline__ void store_some(T* p, int n) const {
    uint16_t* q = reinterpret_cast<uint16_t*>(p);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) q[j] = (uint16_t)bits(j);
  }
};

template <>
struct Vec8<_Float16> : Half8<_Float16> {
  __device__ __forceinline__ float get(int j) const {
    return (float)__builtin_bit_cast(_Float16, (uint16_t)bits(j));
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t lo = __builtin_bit_cast(uint16_t, (_Float16)v[2 * j]);
      const uint32_t hi = __builtin_bit_cast(uint16_t, (_Float16)v[2 * j + 1]);
      a[j] = lo | hi << 16;
    }
  }
};

template <>
struct Vec8<BF16> : Half8<BF16> {
  __device__ __forceinline__ float get(int j) const {
    return __builtin_bit_cast(float, j & 1 ? a[j >> 1] & 0xFFFF0000u : a[j >> 1] << 16);
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      a[j] = float_to_bf16(v[2 * j]) | float_to_bf16(v[2 * j + 1]) << 16;
  }
};

// Chunk c of a row: elements 8 c .. 8 c + 7, as far as there are any.  A chunk
// that the row's end cuts is read as the last eight elements of the row, and
// the ones before it are dropped afterwards: every lane makes the same load
// with no branch around it, so that a wavefront's loads go out together.  (Where
// an output replaces an input, another thread may already have stored over
// those dropped elements; nothing depends on them.)
//
// With a shift of one, chunks begin an element earlier, and chunk 0 is the
// first seven elements: read as eight, the last of them dropped (skip -1).
struct Chunk {
  int32_t at;    // first element read
  int32_t skip;  // elements to drop: 0 for a whole chunk, 8 for none at all
  int32_t left;  // elements from the chunk's first to the row's end (negative beyond it)
};

__device__ __forceinline__ Chunk chunk_at(int32_t c, int32_t width, int32_t shift = 0) {
  const int32_t first = 8 * c - shift, at = max(min(first, max(width - 8, 0)), 0);
  return {at, min(first - at, 8), first < 0 ? 7 : width - first};
}

// kShort: rows of fewer than eight elements (chunk 0 is all there is); kOnce: fp32
// that shall not stay in the caches
template <bool kShort, bool kOnce = false, typename T>
__device__ __forceinline__ void load_chunk(Vec8<T>& v, const T* row, const Chunk& c) {
  if constexpr (kShort)
    v.load_some(row, c.left);
  else if constexpr (kOnce)
    v.load_once(row + c.at);
  else
    v.load(row + c.at);
}

template <bool kShort, typename T>
__device__ __forceinline__ void trim_chunk(Vec8<T>& v, const Chunk& c) {
  if constexpr (!kShort) {
    if (c.skip != 0) v.drop(c.skip);
  }
}

// Chunk k of a thread in rows that may be shifted and go beyond every thread's
// chunk 0: only that one may begin late, and only the others end early.
template <bool kShort, bool kShift, typename T>
__device__ __forceinline__ void trim_chunk(Vec8<T>& v, const Chunk& c, int k) {
  if constexpr (!kShift)
    trim_chunk<kShort>(v, c);
  else if (k > 0)
    trim_chunk<kShort>(v, c);
  else
    v.drop_last(c.skip < 0);
}

template <typename T>
__device__ __forceinline__ void store_chunk(const Vec8<T>& v, T* row, const Chunk& c) {
  if (c.left >= 8)
    v.store(row + c.at);
  else if (c.left > 0)
    v.store_some(row + c.at + max(c.skip, 0), c.left);
}

// --------------------------------------------------------------- reductions
// Sum (or unsigned maximum) over aligned groups of kLanes lanes of a
// wavefront (1 to 64, a power of two), the same bits in each of them, without
// LDS: exchanges with the neighbour, the neighbouring pair, the mirror image in
// 8 and 16 lanes, the next 16 and the other 32.  The order is fixed, so a result never changes
// from run to run.

template <int kCtrl>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, 0xF, 0xF, true);
}

template <int kLanes, typename F>
__device__ __forceinline__ uint32_t group_fold(uint32_t v, F fold) {
  if constexpr (kLanes >= 2) v = fold(v, dpp<0xB1>(v));    // quad_perm 1 0 3 2
  if constexpr (kLanes >= 4) v = fold(v, dpp<0x4E>(v));    // quad_perm 2 3 0 1
  if constexpr (kLanes >= 8) v = fold(v, dpp<0x141>(v));   // row_half_mirror
  if constexpr (kLanes >= 16) v = fold(v, dpp<0x140>(v));  // row_mirror
  if constexpr (kLanes >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = fold(r[0], r[1]);
  }
  if constexpr (kLanes >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = fold(r[0], r[1]);
  }
  return v;
}

template <int kLanes>
__device__ __forceinline__ float group_sum(float v) {
  return __builtin_bit_cast(
      float, group_fold<kLanes>(__builtin_bit_cast(uint32_t, v), [](uint32_t x, uint32_t y) {
        return __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, x) + __builtin_bit_cast(float, y));
      }));
}

template <int kLanes>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  return group_fold<kLanes>(v, [](uint32_t x, uint32_t y) { return max(x, y); });
}

// Over the kThreads threads of a row: part of a wavefront, or several.
// `parity` alternates between calls, so that one barrier per call is enough: a
// wavefront reaches the next call's writes of the same half only after
// everyone has left this call's reads, one barrier later.
template <int kThreads>
__device__ __forceinline__ void row_reduce(float& sum, uint32_t& top, int parity) {
  sum = group_sum<kThreads>(sum);
  top = group_max<kThreads>(top);
  if constexpr (kThreads > 64) {
    // the row is the work-group's only one (rows_block)
    constexpr int kWaves = kThreads / 64;
    __shared__ float s_sum[2][kWaves];
    __shared__ uint32_t s_top[2][kWaves];
    const int wave = (int)(threadIdx.x >> 6);
    if ((threadIdx.x & 63u) == 0) {
      s_sum[parity][wave] = sum;
      s_top[parity][wave] = top;
    }
    __syncthreads();
    sum = s_sum[parity][0];
    top = s_top[parity][0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) {
      sum += s_sum[parity][w];
      top = max(top, s_top[parity][w]);
    }
  }
}

// ------------------------------------------------------------ quantised rows

// What a row's codes and scale come from.  `top` holds the bits of
// max |t_j|: as unsigned integers, absolute values order like the numbers
// and infinities and NaN above them all, so a NaN is never lost on the way.
struct RowQuant {
  float inverse;   // 127 (1 / A), 0 for an empty row
  float prescale;  // 1, or 2^100 for rows so small that 1 / A is infinite
  float scale;
  bool finite;
};

__device__ __forceinline__ RowQuant row_quant(uint32_t top, float factor) {
  RowQuant q;
  const float A = __builtin_bit_cast(float, top);
  q.finite = top < 0x7F800000u && factor == factor;
  q.prescale = A < 0x1p-100f ? 0x1p100f : 1.0f;
  q.inverse = top == 0u || !q.finite ? 0.0f : 127.0f * (1.0f / (A * q.prescale));
  q.scale = q.finite ? A * factor / 127.0f : __builtin_bit_cast(float, 0x7FC00000u);
  return q;
}

// rint(v) as a byte, |v| <= 127: adding 1.5 * 2^23 rounds to an integer, to
// nearest even, and leaves it in the low bits.
__device__ __forceinline__ uint32_t code_bits(float v) {
  return __builtin_bit_cast(uint32_t, v + 0x1.8p23f);
}

// Eight codes from t_0..t_7.
__device__ __forceinline__ u32x2_any eight_codes(const float (&t)[8], const RowQuant& q) {
  u32x2_any c;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint32_t b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) b[j] = code_bits(t[4 * k + j] * q.prescale * q.inverse);
    const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000C0Cu);
    c[k] = q.finite ? lo | hi : 0u;
  }
  return c;
}

__device__ __forceinline__ void store_codes(u32x2_any v, int8_t* row, const Chunk& c) {
  if (c.left >= 8) {
    __builtin_nontemporal_store(v, reinterpret_cast<u32x2_any*>(row + c.at));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < c.left) row[c.at + max(c.skip, 0) + j] = (int8_t)(v[j >> 2] >> (8 * (j & 3)));
  }
}

__device__ __forceinline__ float row_rstd(float sum_of_squares, int32_t width, float eps) {
  const float ms = sum_of_squares / (float)width;
  // a row that holds an infinity or a NaN, or whose squares overflow, has no
  // norm: its output is NaN throughout rather than a plausible zero
  return ms < __builtin_inff() ? 1.0f / sqrtf(ms + eps) : __builtin_bit_cast(float, 0x7FC00000u);
}

// ------------------------------------------------------------------ forward

// kThreads work on one row, each on up to kChunks chunks (chunk k * kThreads +
// lane): width <= 8 kThreads kChunks.  Rows of up to 64 threads need no
// barrier, and a work-group of 256 takes several; rows of more than 64 threads
// have a work-group each.  kThreads = 1: rows of at most eight elements, of
// any width up to that when kShort.
template <int kThreads>
constexpr int rows_block() {
  return kThreads <= 64 ? 256 : kThreads;
}

template <typename T, int kMode, int kThreads, int kChunks, bool kShort = false, bool kOnce = false>
__global__ __launch_bounds__(rows_block<kThreads>()) void rows_kernel(RowArgs a) {
  constexpr int kRows = rows_block<kThreads>() / kThreads;
  const int lane = (int)threadIdx.x % kThreads;
  const int slot = (int)threadIdx.x / kThreads;
  // Chunks shifted by one element in the odd rows of odd width, as in
  // rows_backward_kernel, where no sum's order depends on it (a row's norm is
  // the same wherever it stands) and a work-group has one row (10000x4095 fp16
  // 25.5 -> 22.7 us; with several 300000x101 28 -> 30).
  constexpr bool kShift = sizeof(T) == 2 && kMode == kRowQuantize && kRows == 1;
  int32_t shift = 0;
  if constexpr (kShift) shift = a.width & (int)a.x_stride & (int)(blockIdx.x & 1u);
  Chunk c[kChunks];
  Vec8<T> w[kChunks];
#pragma unroll
  for (int k = 0; k < kChunks; ++k) {
    c[k] = chunk_at(k * kThreads + lane, a.width, shift);
    if constexpr (kMode != kRowQuantize) load_chunk<kShort>(w[k], (const T*)a.weight, c[k]);
  }
  if constexpr (kMode != kRowQuantize) {
#pragma unroll
    for (int k = 0; k < kChunks; ++k) trim_chunk<kShort>(w[k], c[k]);
  }
  const bool add = kMode != kRowQuantize && a.residual != nullptr;
  int parity = 0;
  for (int64_t row = (int64_t)blockIdx.x * kRows + slot; row < a.rows;
       row += (int64_t)gridDim.x * kRows, parity ^= 1) {
    const T* x = (const T*)a.x + row * a.x_stride;
    Vec8<T> h[kChunks];
#pragma unroll
    for (int k = 0; k < kChunks; ++k) load_chunk<kShort, kOnce>(h[k], x, c[k]);
    if (add) {
      const T* r = (const T*)a.residual + row * a.residual_stride;
      Vec8<T> v[kChunks];
#pragma unroll
      for (int k = 0; k < kChunks; ++k) load_chunk<kShort, kOnce>(v[k], r, c[k]);
#pragma unroll
      for (int k = 0; k < kChunks; ++k) {
        float t[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) t[j] = h[k].get(j) + v[k].get(j);
        h[k].set(t);
      }
    }
#pragma unroll
    for (int k = 0; k < kChunks; ++k) trim_chunk<kShort, kShift>(h[k], c[k], k);
    if (add) {
      T* s = (T*)a.sum + row * a.sum_stride;
#pragma unroll
      for (int k = 0; k < kChunks; ++k) store_chunk(h[k], s, c[k]);
    }
    float sum = 0.0f;
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float v = h[k].get(j);
        if constexpr (kMode != kRowQuantize) sum += v * v;
        if constexpr (kMode != kRowNorm) {
          const float t = kMode == kRowQuantize ? v : v * w[k].get(j);
          top = max(top, __builtin_bit_cast(uint32_t, t) & 0x7FFFFFFFu);
        }
      }
    }
    row_reduce<kThreads>(sum, top, parity);
    float rstd = 1.0f;
    if constexpr (kMode != kRowQuantize) {
      rstd = row_rstd(sum, a.width, a.eps);
      if (lane == 0 && a.rstd != nullptr) a.rstd[row] = rstd;
    }
    if constexpr (kMode == kRowNorm) {
      T* o = (T*)a.out + row * a.out_stride;
#pragma unroll
      for (int k = 0; k < kChunks; ++k) {
        float t[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) t[j] = h[k].get(j) * rstd * w[k].get(j);
        Vec8<T> v;
        v.set(t);
        store_chunk(v, o, c[k]);
      }
    } else {
      const RowQuant q = row_quant(top, rstd);
      int8_t* o = a.codes + row * a.codes_stride;
#pragma unroll
      for (int k = 0; k < kChunks; ++k) {
        float t[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          t[j] = kMode == kRowQuantize ? h[k].get(j) : h[k].get(j) * w[k].get(j);
        store_codes(eight_codes(t, q), o, c[k]);
      }
      if (lane == 0) a.scales[row] = q.scale;
    }
  }
}

// Rows of any width from 8 on, one work-group of 1,024 threads each: the row
// is read a second time (from the stored sum where there is one) instead of
// being kept.  A thread meets the same columns in both passes, so it may store
// over what it reads.
template <typename T, int kMode>
__global__ __launch_bounds__(1024) void rows_wide_kernel(RowArgs a) {
  constexpr int kThreads = 1024;
  const int lane = (int)threadIdx.x;
  const int32_t chunks = (int32_t)(((int64_t)a.width + 7) / 8);
  int parity = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, parity ^= 1) {
    const T* x = (const T*)a.x + row * a.x_stride;
    const bool add = kMode != kRowQuantize && a.residual != nullptr;
    const T* r = add ? (const T*)a.residual + row * a.residual_stride : nullptr;
    T* s = add ? (T*)a.sum + row * a.sum_stride : nullptr;
    float sum = 0.0f;
    uint32_t top = 0;
    for (int32_t i = lane; i < chunks; i += kThreads) {
      const Chunk c = chunk_at(i, a.width);
      Vec8<T> h, v, w;
      load_chunk<false>(h, x, c);
      if (add) {
        load_chunk<false>(v, r, c);
        float t[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) t[j] = h.get(j) + v.get(j);
        h.set(t);
      }
      trim_chunk<false>(h, c);
      if (add) store_chunk(h, s, c);
      if constexpr (kMode == kRowNormQ8) {
        load_chunk<false>(w, (const T*)a.weight, c);
        trim_chunk<false>(w, c);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float u = h.get(j);
        if constexpr (kMode != kRowQuantize) sum += u * u;
        if constexpr (kMode != kRowNorm) {
          const float t = kMode == kRowQuantize ? u : u * w.get(j);
          top = max(top, __builtin_bit_cast(uint32_t, t) & 0x7FFFFFFFu);
        }
      }
    }
    row_reduce<kThreads>(sum, top, parity);
    float rstd = 1.0f;
    if constexpr (kMode != kRowQuantize) {
      rstd = row_rstd(sum, a.width, a.eps);
      if (lane == 0 && a.rstd != nullptr) a.rstd[row] = rstd;
    }
    const RowQuant q = row_quant(top, rstd);
    const T* from = add ? s : x;
    for (int32_t i = lane; i < chunks; i += kThreads) {
      const Chunk c = chunk_at(i, a.width);
      Vec8<T> h, w;
      load_chunk<false>(h, from, c);
      if constexpr (kMode != kRowQuantize) load_chunk<false>(w, (const T*)a.weight, c);
      trim_chunk<false>(h, c);
      if constexpr (kMode != kRowQuantize) trim_chunk<false>(w, c);
      float t[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float v = h.get(j);
        t[j] = kMode == kRowQuantize ? v : kMode == kRowNorm ? v * rstd * w.get(j) : v * w.get(j);
      }
      if constexpr (kMode == kRowNorm) {
        h.set(t);
        store_chunk(h, (T*)a.out + row * a.out_stride, c);
      } else {
        store_codes(eight_codes(t, q), a.codes + row * a.codes_stride, c);
      }
    }
    if (kMode != kRowNorm && lane == 0) a.scales[row] = q.scale;
  }
}

// ----------------------------------------------------------------- backward
//
// With n = h rstd, g = dout w and m = mean(g n):
//   dx = rstd (g - n m) [+ dsum],   dweight = sum over rows of dout n.
// dx is the gradient of x and of the residual alike.

struct BackwardArgs {
  const void* dout;
  const void* h;
  const void* weight;
  const float* rstd;
  const void* dsum;  // or null
  void* dx;
  float* partial;   // [partials][pitch] sums of dout n, one row per work-group (or slice)
  float* row_mean;  // rows that do not fit in registers: m of each row
  int64_t rows;
  int64_t dout_stride, h_stride, dsum_stride, dx_stride;  // in elements
  int64_t rows_per_slice;
  int32_t width;
  int32_t partials;
  int32_t pitch;  // width rounded up to whole vectors of four
};

template <typename T>
__device__ __forceinline__ void backward_chunk(const Vec8<T>& d, const Vec8<T>& h,
                                               const Vec8<T>& w, const Vec8<T>& s, float rstd,
                                               float mean, Vec8<T>& out) {
  float t[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float n = h.get(j) * rstd;
    t[j] = rstd * (d.get(j) * w.get(j) - n * mean) + s.get(j);
  }
  out.set(t);
}

// Layout of threads and rows as in rows_kernel.  A work-group takes every
// gridDim.x-th group of rows and keeps its columns' sums of dout n in
// registers until the end: one row of partial sums per work-group.
template <typename T, int kThreads, int kChunks, bool kShort = false, bool kOnce = false>
__global__ __launch_bounds__(rows_block<kThreads>()) void rows_backward_kernel(BackwardArgs a) {
  constexpr int kRows = rows_block<kThreads>() / kThreads;
  const int lane = (int)threadIdx.x % kThreads;
  const int slot = (int)threadIdx.x / kThreads;
  Chunk c[kChunks];
  Vec8<T> w[kChunks];
  float dw[kChunks][8];
  // Loads that begin within a dword take a quarter more time, as do those of
  // every other row where an odd number of 16-bit elements follow each other.
  // A work-group of the odd rows has its chunks shifted by one element, which
  // changes the order of its rows' means, though not of dweight (row, width and
  // stride decide, not addresses, which would change a row's sums with them;
  // 10000x4095 83 -> 66 us, 4099x5003 47 -> 40, without dsum 68 -> 53 and 39 ->
  // 37; but rows of 4095 at a stride of 4096 54 -> 67, so not these).
  constexpr bool kShift = sizeof(T) == 2 && kRows == 1;
  int32_t shift = 0;
  if constexpr (kShift) shift = a.width & (int)a.dout_stride & (int)(blockIdx.x & 1u);
#pragma unroll
  for (int k = 0; k < kChunks; ++k) {
    c[k] = chunk_at(k * kThreads + lane, a.width, shift);
    load_chunk<kShort>(w[k], (const T*)a.weight, c[k]);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[k][j] = 0.0f;
  }
#pragma unroll
  for (int k = 0; k < kChunks; ++k) trim_chunk<kShort, kShift>(w[k], c[k], k);
  const bool add = a.dsum != nullptr;
  // the next row is on its way while this one is worked on, where there are
  // registers for both
  constexpr bool kAhead = kChunks <= 3;
  struct Row {
    Vec8<T> d[kChunks], h[kChunks], s[kChunks];
    float rstd;
  };
  auto load = [&](Row& r, int64_t row) {
    const T* pd = (const T*)a.dout + row * a.dout_stride;
    const T* ph = (const T*)a.h + row * a.h_stride;
    r.rstd = a.rstd[row];
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
      load_chunk<kShort, kOnce>(r.d[k], pd, c[k]);
      load_chunk<kShort, kOnce>(r.h[k], ph, c[k]);
    }
    if (add) {
      const T* ps = (const T*)a.dsum + row * a.dsum_stride;
#pragma unroll
      for (int k = 0; k < kChunks; ++k) load_chunk<kShort, kOnce>(r.s[k], ps, c[k]);
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
    Row now;
    if constexpr (kAhead) {
      now = next;
      if (row + step < a.rows) load(next, row + step);
    } else {
      load(now, row);
    }
    auto &d = now.d, &h = now.h, &s = now.s;
    const float rstd = now.rstd;
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
      trim_chunk<kShort, kShift>(d[k], c[k], k);
      trim_chunk<kShort, kShift>(h[k], c[k], k);
      if (add) trim_chunk<kShort, kShift>(s[k], c[k], k);
    }
    float sum = 0.0f;
    uint32_t unused = 0;
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float dn = d[k].get(j) * (h[k].get(j) * rstd);
        dw[k][j] += dn;
        sum += dn * w[k].get(j);
      }
    }
    row_reduce<kThreads>(sum, unused, parity);
    const float mean = sum / (float)a.width;
    T* o = (T*)a.dx + row * a.dx_stride;
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
      Vec8<T> v;
      backward_chunk(d[k], h[k], w[k], s[k], rstd, mean, v);
      store_chunk(v, o, c[k]);
    }
  }
  if constexpr (kRows > 1) {
    // the work-group's rows of sums, the upper half onto the lower until one
    // is left
    __shared__ float s_dw[kRows / 2][8 * kChunks][kThreads];
#pragma unroll 1
    for (int half = kRows / 2; half > 0; half /= 2) {
      if (slot >= half && slot < 2 * half) {
#pragma unroll
        for (int k = 0; k < kChunks; ++k)
#pragma unroll
          for (int j = 0; j < 8; ++j) s_dw[slot - half][8 * k + j][lane] = dw[k][j];
      }
      __syncthreads();
      if (slot < half) {
#pragma unroll
        for (int k = 0; k < kChunks; ++k)
#pragma unroll
          for (int j = 0; j < 8; ++j) dw[k][j] += s_dw[slot][8 * k + j][lane];
      }
      __syncthreads();
    }
    if (slot > 0) return;
  }
  float* p = a.partial + (int64_t)blockIdx.x * a.pitch;
#pragma unroll
  for (int k = 0; k < kChunks; ++k) {
    Vec8<float> v;
    v.set(dw[k]);
    store_chunk(v, p, c[k]);
  }
}

// Rows of any width from 8 on, first step: m = mean(g n) of each row.
template <typename T>
__global__ __launch_bounds__(1024) void rows_backward_mean_kernel(BackwardArgs a) {
  const int32_t chunks = (int32_t)(((int64_t)a.width + 7) / 8);
  int parity = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, parity ^= 1) {
    const T* pd = (const T*)a.dout + row * a.dout_stride;
    const T* ph = (const T*)a.h + row * a.h_stride;
    const float rstd = a.rstd[row];
    float sum = 0.0f;
    uint32_t unused = 0;
    for (int32_t i = (int32_t)threadIdx.x; i < chunks; i += 1024) {
      const Chunk c = chunk_at(i, a.width);
      Vec8<T> d, h, w;
      load_chunk<false>(d, pd, c);
      load_chunk<false>(h, ph, c);
      load_chunk<false>(w, (const T*)a.weight, c);
      trim_chunk<false>(d, c);
      trim_chunk<false>(h, c);
      trim_chunk<false>(w, c);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum += d.get(j) * (h.get(j) * rstd) * w.get(j);
    }
    row_reduce<1024>(sum, unused, parity);
    if (threadIdx.x == 0) a.row_mean[row] = sum / (float)a.width;
  }
}

// Second step: a thread takes eight columns of a slice of the rows.
template <typename T>
__global__ __launch_bounds__(256) void rows_backward_columns_kernel(BackwardArgs a) {
  const int32_t chunks = (int32_t)(((int64_t)a.width + 7) / 8);
  const int32_t i = (int32_t)(blockIdx.x * 256u + threadIdx.x);
  if (i >= chunks) return;
  const Chunk c = chunk_at(i, a.width);
  const int64_t first = (int64_t)blockIdx.y * a.rows_per_slice;
  const int64_t end = min(first + a.rows_per_slice, a.rows);
  Vec8<T> w;
  load_chunk<false>(w, (const T*)a.weight, c);
  trim_chunk<false>(w, c);
  float dw[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int64_t row = first; row < end; ++row) {
    Vec8<T> d, h, s, v;
    load_chunk<false>(d, (const T*)a.dout + row * a.dout_stride, c);
    load_chunk<false>(h, (const T*)a.h + row * a.h_stride, c);
    s.zero();
    if (a.dsum != nullptr) load_chunk<false>(s, (const T*)a.dsum + row * a.dsum_stride, c);
    trim_chunk<false>(d, c);
    trim_chunk<false>(h, c);
    trim_chunk<false>(s, c);
    const float rstd = a.rstd[row];
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[j] += d.get(j) * (h.get(j) * rstd);
    backward_chunk(d, h, w, s, rstd, a.row_mean[row], v);
    store_chunk(v, (T*)a.dx + row * a.dx_stride, c);
  }
  Vec8<float> v;
  v.set(dw);
  store_chunk(v, a.partial + (int64_t)blockIdx.y * a.pitch, c);
}

// dweight = the sum of the rows of partial sums: 64 columns per work-group,
// four to a thread, 64 threads to a column, joined in a fixed order.  `width`
// columns from a multiple of four on; a row's last vector of four may be
// partly beyond them, but not beyond the pitch.
__device__ __forceinline__ void column_sum(const float* partial, int32_t partials, int32_t pitch,
                                           int32_t width, float* dweight) {
  __shared__ float s_sum[64][64 + 4];
  const int col = 4 * (int)(threadIdx.x & 15u), part = (int)(threadIdx.x >> 4);
  const int64_t c = (int64_t)blockIdx.x * 64 + col;
  float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (c < width) {
#pragma unroll 8
    for (int32_t p = part; p < partials; p += 64) {
      const f32x4 v = *reinterpret_cast<const f32x4*>(partial + (int64_t)p * pitch + c);
#pragma unroll
      for (int j = 0; j < 4; ++j) sum[j] += v[j];
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) s_sum[part][col + j] = sum[j];
  __syncthreads();
  // sixteen threads to a column, then their neighbours' sums
  const int column = (int)(threadIdx.x >> 4), first = (int)(threadIdx.x & 15u);
  float all = 0.0f;
#pragma unroll
  for (int p = 0; p < 4; ++p) all += s_sum[first + 16 * p][column];
  all = group_sum<16>(all);
  const int64_t out = (int64_t)blockIdx.x * 64 + column;
  if (first == 0 && out < width) dweight[out] = all;
}

[[maybe_unused]] static __global__ __launch_bounds__(1024) void column_sum_kernel(
    const float* partial, int32_t partials, int32_t pitch, int32_t width, float* dweight) {
  column_sum(partial, partials, pitch, width, dweight);
}

}  // namespace fn
