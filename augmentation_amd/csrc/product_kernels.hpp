// product_kernels.hpp -- products of 8-bit integers with a scale per row of
// each operand:
//   out[m, n] = RN_T(sa[m] sb[n] sum_k a[m, k] b[n, k] + bias[n])
// a is M x K (tokens), b is N x K (output channels), both with K contiguous.
//
// The sum is taken in 32-bit integers by the matrix cores and is exact for
// K <= 131,071 (|code| <= 128), so no order of summation changes a result;
// the scales, the bias and the one rounding to T follow in fp32.
//
// The matrix instruction takes b as its row operand and a as its column
// operand: a lane then holds four consecutive output channels of one token
// per register quad, which an LDS round trip turns into whole 16-byte stores
// along a row of the output.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "row_kernels.hpp"

namespace fn {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4_any __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Two numbers rounded to a 16-bit type, in one register.
template <typename T>
__device__ __forceinline__ uint32_t two_halves(float lo, float hi) {
  if constexpr (std::is_same_v<T, BF16>)
    return float_to_bf16(lo) | float_to_bf16(hi) << 16;
  else
    return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)lo) |
           (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)hi) << 16;
}

struct ProductArgs {
  const int8_t* a;
  const int8_t* b;
  const float* sa;
  const float* sb;
  const float* bias;  // or null
  void* out;
  int64_t a_stride, b_stride;  // bytes
  int64_t out_stride;          // elements
  int64_t M, N;
  int32_t K;
  uint32_t tiles_m, tiles_n;
};

// f(0), f(1), ... f(kCount - 1), each with its number as a constant.
template <int kCount, int kFirst = 0, typename F>
__device__ __forceinline__ void static_for(F&& f) {
  if constexpr (kFirst < kCount) {
    f(std::integral_constant<int, kFirst>{});
    static_for<kCount, kFirst + 1>(f);
  }
}

// Waits until at most kLeft of this wavefront's loads are under way.
template <int kLeft>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kLeft) : "memory");
}

// Work-groups are dealt round-robin over the 8 XCDs, each with an L2 of its
// own.  Every XCD takes one run of consecutive tiles, in an order that walks
// kGroup token tiles for each channel tile, so that the tiles in flight on an
// XCD share rows of both operands (8192^3 with 2 / 4 / 8 / 16 / 32: 435 / 421 /
// 422 / 430 / 451 us).
struct TileAt {
  uint32_t m, n;
};

__device__ __forceinline__ TileAt tile_at(uint32_t block, const ProductArgs& p) {
  constexpr uint32_t kXcds = 8, kGroup = 4;
  const uint32_t total = p.tiles_m * p.tiles_n;
  const uint32_t xcd = block % kXcds, each = total / kXcds, more = total % kXcds;
  const uint32_t t = xcd * each + min(xcd, more) + block / kXcds;
  const uint32_t band = t / (kGroup * p.tiles_n), in = t % (kGroup * p.tiles_n);
  const uint32_t height = min(kGroup, p.tiles_m - band * kGroup);
  return {band * kGroup + in % height, in / height};
}

// Sixteen codes k0 .. k0 + 15 of a row, zeros from K on.  Near the end of a
// row the last sixteen are read and shifted down, so that every lane makes one
// load and none reads beyond the row.
__device__ __forceinline__ i32x4 load16(const int8_t* row, int32_t k0, int32_t K) {
  if (K < 16) {
    i32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (k0 + j < K) v[j >> 2] |= (int)((uint32_t)(uint8_t)row[k0 + j] << (8 * (j & 3)));
    return v;
  }
  const int32_t k = min(k0, K - 16);
  const i32x4 v = *reinterpret_cast<const i32x4_any*>(row + k);
  const int32_t bits = 8 * min(k0 - k, 16);
  if (bits == 0) return v;
  uint64_t lo = (uint64_t)(uint32_t)v[1] << 32 | (uint32_t)v[0];
  uint64_t hi = (uint64_t)(uint32_t)v[3] << 32 | (uint32_t)v[2];
  if (bits >= 64) {
    lo = bits == 128 ? 0 : hi >> (bits - 64);
    hi = 0;
  } else {
    lo = lo >> bits | hi << (64 - bits);
    hi >>= bits;
  }
  return i32x4{(int)(uint32_t)lo, (int)(lo >> 32), (int)(uint32_t)hi, (int)(hi >> 32)};
}

// ---------------------------------------------------------------------------
// Tiles through direct global-to-LDS loads, for rows that start at multiples
// of 16 bytes.
//
// A stage is the next kBK codes of K of the tile's tokens and channels in LDS;
// kStages of them are under way at once.  The loads are written out because
// the compiler, which cannot tell a stage that is being read from one that is
// being filled, would wait for all of them before every read; they have no
// destination register, and every wait for them stands in the code below.
// M0 holds the LDS address; nothing else in these kernels uses it.

__device__ __forceinline__ void load_to_lds(i32x4 resource, uint32_t lds, int offset, int k0) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %1, %2, %3 offen lds"
      :
      : "s"(lds), "v"(offset), "s"(resource), "s"(k0)
      : "memory");
}

__device__ __forceinline__ i32x4 tile_resource(const int8_t* p, int64_t stride, int64_t rows,
                                               int32_t K) {
  // bytes from the tile's first row to the end of the last one; loads beyond
  // give zeros
  const int64_t bytes = rows > 0 ? (rows - 1) * stride + K : 0;
  const uint64_t at = (uint64_t)(uintptr_t)p;
  return i32x4{(int)(uint32_t)at, (int)(uint32_t)(at >> 32),
               (int)min(bytes, (int64_t)0x7FFFFFF0), 0x00027000};
}

// Four bytes per lane.
__device__ __forceinline__ void load_words_to_lds(i32x4 resource, uint32_t lds, int offset) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "buffer_load_dword %1, %2, 0 offen lds"
      :
      : "s"(lds), "v"(offset), "s"(resource)
      : "memory");
}

constexpr int kOutside = 0x7FFFFFF8;  // an offset that lies beyond every tile

// Codes of a stage are rows of 128 (eight 16-byte pieces, one cache line, so a
// load of 64 lanes touches eight whole lines; rows of 64 codes took twice the
// time per byte).  Piece c of row r lies at position c ^ (r / 2 mod 8): the
// sixteen rows of which lanes read the same piece at once spread over all
// banks (measured: no conflicts; c ^ (r mod 8) had one conflict per read).
constexpr int kBK = 128;

__device__ __forceinline__ int staged_piece(int row, int piece) {
  return piece ^ ((row >> 1) & 7);
}

// Rows of out from a wavefront's sums.  acc[i][j]: tile of 16 tokens x 16
// channels; lane l holds channels 4 (l / 16) .. + 3 of token l % 16.  Scaled
// and rounded where they are, 64 tokens at a time go through the wavefront's
// own piece of LDS (rows of kPitch bytes; the 16 bytes beyond a row's
// channels keep rows off the same banks) and leave as 16-byte stores along
// rows, non-temporal (50176x1024x768 to fp16: 78 -> 65 us, 8192^3 409 -> 404).
template <typename T, int kTM, int kTN>
struct OutputTile {
  static constexpr int kTokens = kTM < 4 ? 16 * kTM : 64;  // tokens that leave together
  static constexpr int kPitch = 16 * kTN * (int)sizeof(T) + 16;
  static constexpr int kBytes = kTokens * kPitch;
  float sa[kTM];
  f32x4 sb[kTN], bias[kTN];

  // from LDS: the scales of the wavefront's tokens, those of its channels, and
  // its channels' bias
  __device__ __forceinline__ void load_scales(const float* s_sa, const float* s_sb,
                                              const float* s_bias) {
    const int lane = (int)(threadIdx.x & 63u);
#pragma unroll
    for (int i = 0; i < kTM; ++i) sa[i] = s_sa[16 * i + (lane & 15)];
#pragma unroll
    for (int j = 0; j < kTN; ++j) {
      sb[j] = *reinterpret_cast<const f32x4*>(s_sb + 16 * j + 4 * (lane >> 4));
      bias[j] = *reinterpret_cast<const f32x4*>(s_bias + 16 * j + 4 * (lane >> 4));
    }
  }

  __device__ __forceinline__ void store(const ProductArgs& p, const i32x4 (&acc)[kTM][kTN],
                                        int8_t* lds, int64_t m0, int64_t n0) const {
    constexpr int kE = 16 / (int)sizeof(T);    // outputs per 16-byte store
    constexpr int kLanes = 16 * kTN / kE;      // lanes along a row
    constexpr int kRowsAtOnce = 64 / kLanes;
    constexpr int kTiles = kTokens / 16;
    const int lane = (int)(threadIdx.x & 63u);
    const int64_t n = n0 + kE * (lane % kLanes);
    const int left = (int)min(p.N - n, (int64_t)kE);
#pragma unroll
    for (int i0 = 0; i0 < kTM; i0 += kTiles) {
#pragma unroll
      for (int i = 0; i < kTiles; ++i)
#pragma unroll
        for (int j = 0; j < kTN; ++j) {
          float v[4];
#pragma unroll
          for (int c = 0; c < 4; ++c)
            v[c] = (float)acc[i0 + i][j][c] * sa[i0 + i] * sb[j][c] + bias[j][c];
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
        const u32x4 v = *reinterpret_cast<const u32x4*>(lds + r * kPitch + 16 * (lane % kLanes));
        T* to = (T*)p.out + m * p.out_stride + n;
        if (m < p.M && left == kE) {
          __builtin_nontemporal_store(v, reinterpret_cast<u32x4_any*>(to));
        } else if (m < p.M && left > 0) {
          store_part(v, to, left);
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    }
  }

  static __device__ __forceinline__ void store_part(u32x4 v, T* to, int left) {
#pragma unroll
    for (int c = 0; c < 16 / (int)sizeof(T); ++c)
      if (c < left) {
        if constexpr (sizeof(T) == 4)
          reinterpret_cast<uint32_t*>(to)[c] = v[c];
        else
          reinterpret_cast<uint16_t*>(to)[c] = (uint16_t)(v[c >> 1] >> (16 * (c & 1)));
      }
  }
};

// One tile of kBM tokens x kBN channels per work-group of kWM x kWN
// wavefronts, each with kTM x kTN tiles of the 16x16x64 instruction (measured
// against 32x32x32 on 8192^3: 2.54 against 2.42 POP/s; the smaller one moves
// fewer accumulator registers per operation, and the clock that falls under
// load costs such a product more than the count of cycles).
//
// A wavefront's products of one step (64 codes of K) are its time for
// everything else: between them it reads the next step's fragments from LDS
// and, in a stage's last step, issues its share of a later stage's loads.
// 8192^3 takes 395 to 440 us (2.5 to 2.8 POP/s) with the matrix cores 64% busy
// at 1.85 GHz.  The same products alone hold 2.36 GHz and take 290 us, so the
// clock under load is most of the difference; why they are a quarter idle
// even then is not known.  Short sums are bound by what no product covers, the
// first loads and the outputs: 50176x1024x768 50 to 52 us, 28 to 32 at the rate
// of 8192^3.
//
// kLines: every row starts at a cache line.  Else a stage still brings whole
// lines: of row r it has the codes from 128 s - d to 128 s + 127 - d, d the
// distance of the row's start from its line's.  Piece j of the 128 codes from
// 128 s on then stands at its usual place, in stage s if j + d / 16 < 8 and
// otherwise in the next one; rows eight apart have the same d, so a lane has
// one for all its rows.  Read as they are, rows off the lines take two for
// each load (2048x2048x4112 in 128x64 tiles 31 us, so 25, with rows on the lines
// 23), but the next stage has to have landed, too, which 256x256 tiles have no
// room for.
template <typename T, int kBM, int kBN, int kWM, int kWN, int kStages, bool kLines>
__global__ __launch_bounds__(64 * kWM * kWN, 2) void product_tile_kernel(ProductArgs p) {
  constexpr int kWaves = kWM * kWN, kTM = kBM / kWM / 16, kTN = kBN / kWN / 16;
  constexpr int kStageBytes = (kBM + kBN) * kBK;
  constexpr int kLoadsA = kBM / 8 / kWaves, kLoadsB = kBN / 8 / kWaves;  // per wavefront and stage
  constexpr int kLoads = kLoadsA + kLoadsB;
  constexpr int kSteps = kBK / 64;
  static_assert(kBM % 64 == 0 && kBN % 64 == 0, "scales come 64 at a time");
  using Out = OutputTile<T, kTM, kTN>;
  constexpr int kLds =
      kStages * kStageBytes > kWaves * Out::kBytes ? kStages * kStageBytes : kWaves * Out::kBytes;
  __shared__ __align__(1024) int8_t s_stages[kLds];
  __shared__ __align__(1024) float s_scales[kBM + 2 * kBN];
  const int lane = (int)(threadIdx.x & 63u);
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));

  const TileAt tile = tile_at(blockIdx.x, p);
  const int64_t m0 = (int64_t)tile.m * kBM, n0 = (int64_t)tile.n * kBN;
  // the scales and the bias go first, and have landed with the first stage:
  // fetched after the last product they would keep the outputs waiting for
  // memory once more
  {
    const uint32_t to = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)s_scales;
    auto words = [](const float* from, int64_t count) {
      return tile_resource((const int8_t*)from, 0, from != nullptr ? 1 : 0, (int32_t)(4 * count));
    };
    const i32x4 sa = words(p.sa + m0, min(p.M - m0, (int64_t)kBM));
    const i32x4 sb = words(p.sb + n0, min(p.N - n0, (int64_t)kBN));
    const i32x4 bias =
        words(p.bias != nullptr ? p.bias + n0 : nullptr, min(p.N - n0, (int64_t)kBN));
    constexpr int kA = kBM / 64, kB = kBN / 64;
#pragma unroll
    for (int c = 0; c < kA + 2 * kB; ++c)
      if (c % kWaves == wave)
        load_words_to_lds(c < kA ? sa : c < kA + kB ? sb : bias, to + 256 * c,
                          256 * (c < kA ? c : c < kA + kB ? c - kA : c - kA - kB) + 4 * lane);
  }
  const int8_t *a = p.a + m0 * p.a_stride, *b = p.b + n0 * p.b_stride;
  // pieces from the line's start to the first row's and, for each row, more
  const int first_a = kLines ? 0 : (int)((uintptr_t)a >> 4) & 7;
  const int first_b = kLines ? 0 : (int)((uintptr_t)b >> 4) & 7;
  const int more_a = kLines ? 0 : (int)(p.a_stride >> 4), more_b = kLines ? 0 : (int)(p.b_stride >> 4);
  const i32x4 src_a = tile_resource(a - 16 * first_a, p.a_stride, min(p.M - m0, (int64_t)kBM),
                                    p.K + 16 * first_a);
  const i32x4 src_b = tile_resource(b - 16 * first_b, p.b_stride, min(p.N - n0, (int64_t)kBN),
                                    p.K + 16 * first_b);
  // load i of a wavefront brings eight rows; every other one has this lane's
  // piece at the same place
  static_assert(kLoadsA % 2 == 0 && kLoadsB % 2 == 0, "rows per wavefront: a multiple of 16");
  const int sub = lane / 8;
  const int piece[2] = {staged_piece(sub, lane % 8), staged_piece(8 + sub, lane % 8)};
  // this lane's first code in stage 0: before the row, if its piece of the
  // line is
  const int d_a = (first_a + sub * more_a) & 7, d_b = (first_b + sub * more_b) & 7;
  const int code_a[2] = {16 * (((piece[0] + d_a) & 7) - d_a), 16 * (((piece[1] + d_a) & 7) - d_a)};
  const int code_b[2] = {16 * (((piece[0] + d_b) & 7) - d_b), 16 * (((piece[1] + d_b) & 7) - d_b)};
  int off_a[kLoadsA], off_b[kLoadsB];
#pragma unroll
  for (int i = 0; i < kLoadsA; ++i) {
    const int r = (wave * kLoadsA + i) * 8 + sub;
    off_a[i] = m0 + r < p.M ? 16 * first_a + r * (int)p.a_stride + code_a[i & 1] : kOutside;
  }
#pragma unroll
  for (int i = 0; i < kLoadsB; ++i) {
    const int r = (wave * kLoadsB + i) * 8 + sub;
    off_b[i] = n0 + r < p.N ? 16 * first_b + r * (int)p.b_stride + code_b[i & 1] : kOutside;
  }
  const uint32_t lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)s_stages;
  // load i of the stage that begins at code k0; pieces before the row and from
  // K on (K is whole pieces) bring zeros
  struct Inside {
    bool a[2], b[2];
  };
  auto inside_of = [&](int k0) {
    const uint32_t K = (uint32_t)p.K;
    return Inside{{(uint32_t)(k0 + code_a[0]) < K, (uint32_t)(k0 + code_a[1]) < K},
                  {(uint32_t)(k0 + code_b[0]) < K, (uint32_t)(k0 + code_b[1]) < K}};
  };
  auto issue = [&](int stage, int k0, int i, const Inside& inside) {
    const uint32_t to = lds + stage * kStageBytes;
    if (i < kLoadsA)
      load_to_lds(src_a, to + (wave * kLoadsA + i) * 1024, inside.a[i & 1] ? off_a[i] : kOutside,
                  k0);
    else
      load_to_lds(src_b, to + kBM * kBK + (wave * kLoadsB + i - kLoadsA) * 1024,
                  inside.b[i & 1] ? off_b[i - kLoadsA] : kOutside, k0);
  };

  // fragments: lane l holds codes 16 (l / 16) .. + 15 of row l % 16
  const int at_a = ((wave / kWN) * kTM * 16 + (lane & 15)) * kBK;
  const int at_b = kBM * kBK + ((wave % kWN) * kTN * 16 + (lane & 15)) * kBK;
  int at_piece[kSteps];
  bool later_a[kSteps], later_b[kSteps];  // does the piece stand in the next stage
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    const int j = 4 * k + (lane >> 4);
    at_piece[k] = 16 * staged_piece(lane & 15, j);
    later_a[k] = j + ((first_a + (lane & 7) * more_a) & 7) >= 8;
    later_b[k] = j + ((first_b + (lane & 7) * more_b) & 7) >= 8;
  }
  i32x4 fa[2][kTM], fb[2][kTN];
  auto fetch = [&](const int8_t* buf, const int8_t* later, int k, int slot, int i) {
    const int8_t* from_a = !kLines && later_a[k] ? later : buf;
    const int8_t* from_b = !kLines && later_b[k] ? later : buf;
    if (i < kTN)
      fb[slot][i] = *reinterpret_cast<const i32x4*>(from_b + at_b + i * 16 * kBK + at_piece[k]);
    else
      fa[slot][i - kTN] =
          *reinterpret_cast<const i32x4*>(from_a + at_a + (i - kTN) * 16 * kBK + at_piece[k]);
  };
  i32x4 acc[kTM][kTN] = {};

  // the stages that must have landed beyond the one that is worked on
  constexpr int kAhead = kLines ? 0 : 1;
  static_assert(kStages >= 2 + kAhead, "a stage is read while the next one lands");
#pragma unroll
  for (int s = 0; s < kStages; ++s) {
    const Inside inside = inside_of(s * kBK);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) issue(s, s * kBK, i, inside);
  }
  wait_loads<(kStages - 1 - kAhead) * kLoads>();
  __builtin_amdgcn_s_barrier();
#pragma unroll
  for (int i = 0; i < kTM + kTN; ++i) fetch(s_stages, s_stages + kStageBytes, 0, 0, i);
  int stage = 0;
  for (int k0 = 0; k0 < p.K; k0 += kBK) {
    const int next = stage + 1 == kStages ? 0 : stage + 1;
    const int after = next + 1 == kStages ? 0 : next + 1;
    static_for<kSteps>([&](auto step) {
      constexpr int k = decltype(step)::value;
      constexpr bool kLast = k + 1 == kSteps;
      constexpr int kProducts = kTM * kTN, kReads = kTM + kTN, kNewLoads = kLast ? kLoads : 0;
      constexpr int kOthers = kReads + kNewLoads;
      const int8_t* from = s_stages + (kLast ? next : stage) * kStageBytes;
      const int8_t* later = s_stages + (kLast ? after : next) * kStageBytes;
      const int k_new = k0 + kStages * kBK;
      Inside inside = {};
      if constexpr (kLast) {
        // this wavefront's loads of the next stage have landed and its reads
        // of this one are done; beyond the barrier, everyone's are: the next
        // stage may be read, and this one's place be filled again
        wait_loads<(kStages - 2 - kAhead) * kLoads>();
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        inside = inside_of(k_new);
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
            issue(stage, k_new, kBefore, inside);
          else
            fetch(from, later, kLast ? 0 : k + 1, (k + 1) & 1, o - kBefore);
        });
        __builtin_amdgcn_sched_barrier(0);
        acc[t / kTN][t % kTN] = __builtin_amdgcn_mfma_i32_16x16x64_i8(
            fb[k & 1][t % kTN], fa[k & 1][t / kTN], acc[t / kTN][t % kTN], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
      });
    });
    stage = next;
  }
  const int m_wave = (wave / kWN) * kTM * 16, n_wave = (wave % kWN) * kTN * 16;
  Out out;
  out.load_scales(s_scales + m_wave, s_scales + kBM + n_wave, s_scales + kBM + kBN + n_wave);
  // loads of stages beyond K (they bring zeros) end before LDS is used again
  wait_loads<0>();
  __syncthreads();
  out.store(p, acc, s_stages + wave * Out::kBytes, m0 + m_wave, n0 + n_wave);
}

// Tiles through registers: rows may start at any byte and K may be anything,
// which direct loads to LDS cannot serve.  Two stages of 128 codes; the codes
// of two more are on their way to registers meanwhile.  Work-groups of kWM x 2
// wavefronts; the layout of a stage and of the fragments is
// product_tile_kernel's.
template <typename T, int kBM, int kBN, int kWM>
__global__ __launch_bounds__(128 * kWM, 2) void product_any_kernel(ProductArgs p) {
  constexpr int kThreads = 128 * kWM, kTM = kBM / kWM / 16, kTN = kBN / 32;
  constexpr int kRows = kBM + kBN, kStageBytes = kRows * kBK;
  constexpr int kLoads = kRows * 8 / kThreads;  // pieces per thread and stage
  using Out = OutputTile<T, kTM, kTN>;
  constexpr int kOutBytes = 2 * kWM * Out::kBytes;
  __shared__ __align__(1024) int8_t s_stages[2 * kStageBytes > kOutBytes ? 2 * kStageBytes
                                                                         : kOutBytes];
  const int lane = (int)(threadIdx.x & 63u), wave = (int)(threadIdx.x >> 6);
  const TileAt tile = tile_at(blockIdx.x, p);
  const int64_t m0 = (int64_t)tile.m * kBM, n0 = (int64_t)tile.n * kBN;
  __shared__ __align__(16) float s_scales[kBM + 2 * kBN];
  for (int i = (int)threadIdx.x; i < kBM + 2 * kBN; i += kThreads) {
    const int64_t m = m0 + i, n = n0 + (i - kBM) % kBN;
    float v = 0.0f;
    if (i < kBM) {
      if (m < p.M) v = p.sa[m];
    } else if (n < p.N && (i < kBM + kBN || p.bias != nullptr)) {
      v = i < kBM + kBN ? p.sb[n] : p.bias[n];
    }
    s_scales[i] = v;
  }
  // this thread's piece of every kThreads / 8-th row: the tokens' rows first,
  // then the channels'
  const int piece = (int)(threadIdx.x & 7u), row = (int)(threadIdx.x >> 3);
  const int8_t* from[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int r = row + kThreads / 8 * i;
    const int64_t m = m0 + r, n = n0 + r - kBM;
    from[i] = r < kBM ? (m < p.M ? p.a + m * p.a_stride : nullptr)
                      : (n < p.N ? p.b + n * p.b_stride : nullptr);
  }
  // the codes of the next two stages: memory takes longer than one stage's
  // products
  i32x4 held[2][kLoads];
  auto load = [&](i32x4 (&to)[kLoads], int k0) {
    if (k0 >= p.K) return;
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      to[i] = from[i] != nullptr ? load16(from[i], k0 + 16 * piece, p.K) : i32x4{0, 0, 0, 0};
  };
  auto put = [&](const i32x4 (&codes)[kLoads], int stage) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int r = row + kThreads / 8 * i;
      *reinterpret_cast<i32x4*>(s_stages + stage * kStageBytes + r * kBK +
                                16 * staged_piece(r, piece)) = codes[i];
    }
  };
  const int at_a = ((wave >> 1) * kTM * 16 + (lane & 15)) * kBK;
  const int at_b = (kBM + (wave & 1) * kTN * 16 + (lane & 15)) * kBK;
  i32x4 acc[kTM][kTN] = {};
  auto multiply = [&](const int8_t* buf) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int at = 16 * staged_piece(lane & 15, 4 * k + (lane >> 4));
      i32x4 fa[kTM], fb[kTN];
#pragma unroll
      for (int j = 0; j < kTN; ++j)
        fb[j] = *reinterpret_cast<const i32x4*>(buf + at_b + j * 16 * kBK + at);
#pragma unroll
      for (int i = 0; i < kTM; ++i)
        fa[i] = *reinterpret_cast<const i32x4*>(buf + at_a + i * 16 * kBK + at);
#pragma unroll
      for (int i = 0; i < kTM; ++i)
#pragma unroll
        for (int j = 0; j < kTN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[j], fa[i], acc[i][j], 0, 0, 0);
    }
  };
  load(held[0], 0);
  load(held[1], kBK);
  for (int k0 = 0; k0 < p.K; k0 += 2 * kBK) {
    // stage 0 was last read before the barrier of stage 1, and so on
    put(held[0], 0);
    __syncthreads();
    load(held[0], k0 + 2 * kBK);
    multiply(s_stages);
    if (k0 + kBK >= p.K) break;
    put(held[1], 1);
    __syncthreads();
    load(held[1], k0 + 3 * kBK);
    multiply(s_stages + kStageBytes);
  }
  const int m_wave = (wave >> 1) * kTM * 16, n_wave = (wave & 1) * kTN * 16;
  Out out;
  __syncthreads();
  out.load_scales(s_scales + m_wave, s_scales + kBM + n_wave, s_scales + kBM + kBN + n_wave);
  out.store(p, acc, s_stages + wave * Out::kBytes, m0 + m_wave, n0 + n_wave);
}

// The integer sums of kWaves wavefronts that divided K between them, joined in
// LDS, and the outputs from them.
template <typename T, int kMT, int kNT, int kWaves>
__device__ __forceinline__ void join_waves(const ProductArgs& p, const i32x4 (&acc)[kMT][kNT],
                                           int* s_sum, int64_t m0, int64_t n0) {
  constexpr int kOutputs = kMT * kNT * 256;
  const int lane = (int)(threadIdx.x & 63u), wave = (int)(threadIdx.x >> 6);
#pragma unroll
  for (int i = 0; i < kMT; ++i)
#pragma unroll
    for (int j = 0; j < kNT; ++j)
      *reinterpret_cast<i32x4*>(&s_sum[wave * kOutputs + (i * kNT + j) * 256 + 4 * lane]) =
          acc[i][j];
  __syncthreads();
  for (int o = (int)threadIdx.x; o < kOutputs; o += 64 * kWaves) {
    const int channel = o % (16 * kNT), token = o / (16 * kNT);
    const int64_t n = n0 + channel, m = m0 + token;
    if (m >= p.M) break;
    if (n >= p.N) continue;
    const int at = ((token >> 4) * kNT + (channel >> 4)) * 256 +
                   4 * ((channel >> 2 & 3) * 16 + (token & 15)) + (channel & 3);
    int sum = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) sum += s_sum[w * kOutputs + at];
    const float y = (float)sum * p.sa[m] * p.sb[n] + (p.bias != nullptr ? p.bias[n] : 0.0f);
    if constexpr (sizeof(T) == 4)
      ((float*)p.out)[m * p.out_stride + n] = y;
    else
      ((uint16_t*)p.out)[m * p.out_stride + n] = (uint16_t)two_halves<T>(y, 0.0f);
  }
}

// ---------------------------------------------------------------------------
// Few tokens, rows at multiples of 16 bytes: the time is that of reading b,
// and what counts is how much of b is under way.  A work-group takes 16 kNT
// channels (few, so that all compute units have some) and 16 kMT tokens; its
// wavefronts divide K between them, wavefront w taking lines w, w + kWaves,
// ... of 128 codes.  Each has a ring of kStages lines of its own in LDS and
// waits for nobody until the sums are joined.
template <typename T, int kMT, int kNT, int kStages, int kWaves>
__global__ __launch_bounds__(64 * kWaves) void product_split_kernel(ProductArgs p) {
  constexpr int kRows = 16 * (kMT + kNT), kLoads = kRows / 8;
  constexpr int kRing = kStages * kRows * kBK;
  constexpr int kSums = kMT * kNT * 1024;
  __shared__ __align__(1024) int8_t s_ring[kWaves * (kRing > kSums ? kRing : kSums)];
  const int lane = (int)(threadIdx.x & 63u);
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int64_t n0 = (int64_t)blockIdx.x * (16 * kNT), m0 = (int64_t)blockIdx.y * (16 * kMT);
  const i32x4 src_a =
      tile_resource(p.a + m0 * p.a_stride, p.a_stride, min(p.M - m0, (int64_t)(16 * kMT)), p.K);
  const i32x4 src_b =
      tile_resource(p.b + n0 * p.b_stride, p.b_stride, min(p.N - n0, (int64_t)(16 * kNT)), p.K);
  const int sub = lane / 8;
  const int piece[2] = {staged_piece(sub, lane % 8), staged_piece(8 + sub, lane % 8)};
  int off[kLoads];  // the channels' rows first, then the tokens'
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int r = 8 * i + sub, ra = r - 16 * kNT;
    if (i < 2 * kNT)
      off[i] = n0 + r < p.N ? r * (int)p.b_stride + 16 * piece[i & 1] : kOutside;
    else
      off[i] = m0 + ra < p.M ? ra * (int)p.a_stride + 16 * piece[i & 1] : kOutside;
  }
  int8_t* ring = s_ring + wave * kRing;
  const uint32_t lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)ring;
  auto issue = [&](int stage, int k0) {
    const bool inside[2] = {k0 + 16 * piece[0] < p.K, k0 + 16 * piece[1] < p.K};
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      load_to_lds(i < 2 * kNT ? src_b : src_a, lds + stage * kRows * kBK + i * 1024,
                  inside[i & 1] ? off[i] : kOutside, k0);
  };
  const int at[2] = {(lane & 15) * kBK + 16 * staged_piece(lane & 15, lane >> 4),
                     (lane & 15) * kBK + 16 * staged_piece(lane & 15, 4 + (lane >> 4))};
  i32x4 acc[kMT][kNT] = {};
  constexpr int kStride = kWaves * kBK;  // codes from one line of a wavefront to its next
#pragma unroll
  for (int s = 0; s < kStages; ++s) issue(s, wave * kBK + s * kStride);
  int stage = 0;
  for (int k0 = wave * kBK; k0 < p.K; k0 += kStride) {
    wait_loads<(kStages - 1) * kLoads>();
    const int8_t* from = ring + stage * kRows * kBK;
    i32x4 fa[2][kMT], fb[2][kNT];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int j = 0; j < kNT; ++j)
        fb[h][j] = *reinterpret_cast<const i32x4*>(from + 16 * j * kBK + at[h]);
#pragma unroll
      for (int i = 0; i < kMT; ++i)
        fa[h][i] = *reinterpret_cast<const i32x4*>(from + 16 * (kNT + i) * kBK + at[h]);
    }
    // the line is in registers: its place may be filled again
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    issue(stage, k0 + kStages * kStride);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < kMT; ++i)
#pragma unroll
        for (int j = 0; j < kNT; ++j)
          acc[i][j] =
              __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[h][j], fa[h][i], acc[i][j], 0, 0, 0);
    stage = stage + 1 == kStages ? 0 : stage + 1;
  }
  wait_loads<0>();
  __syncthreads();
  join_waves<T, kMT, kNT, kWaves>(p, acc, reinterpret_cast<int*>(s_ring), m0, n0);
}

// Few tokens, rows that start at any byte, any K: product_split_kernel with the
// lines through registers, two of them under way.  Eight lanes read a row's
// 128 codes, which costs unaligned loads little (fragments read straight from
// memory, 64 bytes of a row at a time, took 128x794x2502 16.8 us against 7.7,
// 1x4096x4095 10.2 against 5.6).  A wavefront writes a line to its own piece of
// LDS and reads it back as fragments; its LDS operations take effect in their
// order, and nobody else's matter.
template <typename T, int kMT, int kNT, int kWaves>
__global__ __launch_bounds__(64 * kWaves) void product_split_any_kernel(ProductArgs p) {
  constexpr int kRows = 16 * (kMT + kNT), kLoads = kRows / 8;
  constexpr int kLine = kRows * kBK, kSums = kMT * kNT * 1024;
  __shared__ __align__(1024) int8_t s_lines[kWaves * (kLine > kSums ? kLine : kSums)];
  const int lane = (int)(threadIdx.x & 63u);
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int64_t n0 = (int64_t)blockIdx.x * (16 * kNT), m0 = (int64_t)blockIdx.y * (16 * kMT);
  const int8_t* from[kLoads];  // the channels' rows first, then the tokens'; null: no such row
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int r = 8 * i + lane / 8;
    const int64_t n = n0 + r, m = m0 + r - 16 * kNT;
    from[i] = i < 2 * kNT ? (n < p.N ? p.b + n * p.b_stride : nullptr)
                          : (m < p.M ? p.a + m * p.a_stride : nullptr);
  }
  int8_t* line = s_lines + wave * kLine;
  const int at[2] = {(lane & 15) * kBK + 16 * staged_piece(lane & 15, lane >> 4),
                     (lane & 15) * kBK + 16 * staged_piece(lane & 15, 4 + (lane >> 4))};
  i32x4 acc[kMT][kNT] = {};
  i32x4 held[2][kLoads];
  auto load = [&](i32x4 (&to)[kLoads], int k0) {
    if (k0 >= p.K) return;
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      to[i] = from[i] != nullptr ? load16(from[i], k0 + 16 * (lane % 8), p.K) : i32x4{0, 0, 0, 0};
  };
  auto multiply = [&](const i32x4 (&codes)[kLoads]) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int r = 8 * i + lane / 8;
      *reinterpret_cast<i32x4*>(line + r * kBK + 16 * staged_piece(r, lane % 8)) = codes[i];
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      i32x4 fa[kMT], fb[kNT];
#pragma unroll
      for (int j = 0; j < kNT; ++j)
        fb[j] = *reinterpret_cast<const i32x4*>(line + 16 * j * kBK + at[h]);
#pragma unroll
      for (int i = 0; i < kMT; ++i)
        fa[i] = *reinterpret_cast<const i32x4*>(line + 16 * (kNT + i) * kBK + at[h]);
#pragma unroll
      for (int i = 0; i < kMT; ++i)
#pragma unroll
        for (int j = 0; j < kNT; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[j], fa[i], acc[i][j], 0, 0, 0);
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  };
  constexpr int kStride = kWaves * kBK;
  load(held[0], wave * kBK);
  load(held[1], wave * kBK + kStride);
  for (int k0 = wave * kBK; k0 < p.K; k0 += 2 * kStride) {
    multiply(held[0]);
    load(held[0], k0 + 2 * kStride);
    if (k0 + kStride < p.K) multiply(held[1]);
    load(held[1], k0 + 3 * kStride);
  }
  __syncthreads();
  join_waves<T, kMT, kNT, kWaves>(p, acc, reinterpret_cast<int*>(s_lines), m0, n0);
}

}  // namespace fn
