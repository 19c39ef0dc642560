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

#include "row_kernels.hpp"

namespace fn {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef int i32x4_any __attribute__((ext_vector_type(4), aligned(1)));

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
  uint32_t tiles_n;
};

// Sixteen codes k0 .. k0 + 15 of a row, zeros from K on.
__device__ __forceinline__ i32x4 load16(const int8_t* row, int32_t k0, int32_t K) {
  i32x4 v = {0, 0, 0, 0};
  if (k0 + 16 <= K) {
    v = *reinterpret_cast<const i32x4_any*>(row + k0);
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (k0 + j < K) v[j >> 2] |= (int)((uint32_t)(uint8_t)row[k0 + j] << (8 * (j & 3)));
  }
  return v;
}

// kE consecutive outputs of one row from their integer sums.
template <typename T, int kE>
__device__ __forceinline__ void store_outputs(const int (&acc)[kE], float sa, const float (&sb)[kE],
                                              const float (&bias)[kE], T* p, int n) {
  float v[8];
#pragma unroll
  for (int j = 0; j < kE; ++j) v[j] = (float)acc[j] * sa * sb[j] + bias[j];
  if constexpr (sizeof(T) == 4) {
    if (n >= 4) {
      u32x4_any q;
#pragma unroll
      for (int j = 0; j < 4; ++j) q[j] = __builtin_bit_cast(uint32_t, v[j]);
      *reinterpret_cast<u32x4_any*>(p) = q;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < n) p[j] = v[j];
    }
  } else {
    Vec8<T> q;
    q.set(v);
    if (n >= 8)
      q.store(p);
    else
      q.store_some(p, n);
  }
}

// A wavefront's kTn x 32 channels by 32 tokens of sums go through its own
// piece of LDS and leave as rows of the output.  m0, n0: first token and
// channel.  kPitch: 32-bit words from one token's row in LDS to the next; the
// four words beyond the row keep a quad's 16-byte writes off the same banks.
template <typename T, int kTn>
__device__ __forceinline__ void store_strip(const ProductArgs& p, const i32x16 (&acc)[kTn],
                                            int* lds, int64_t m0, int64_t n0) {
  constexpr int kN = 32 * kTn, kPitch = kN + 4;
  constexpr int kE = 16 / (int)sizeof(T);  // outputs per 16-byte store
  constexpr int kLanes = kN / kE;          // lanes along a row
  constexpr int kRowsAtOnce = 64 / kLanes;
  const int lane = (int)(threadIdx.x & 63u);
#pragma unroll
  for (int t = 0; t < kTn; ++t)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const i32x4 v = {acc[t][4 * q], acc[t][4 * q + 1], acc[t][4 * q + 2], acc[t][4 * q + 3]};
      *reinterpret_cast<i32x4*>(lds + (lane & 31) * kPitch + 32 * t + 8 * q + 4 * (lane >> 5)) = v;
    }
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  const int64_t n = n0 + kE * (lane % kLanes);
  const int left = (int)min(p.N - n, (int64_t)kE);
  if (left > 0) {
    float sb[kE], bias[kE];
#pragma unroll
    for (int j = 0; j < kE; ++j) {
      sb[j] = j < left ? p.sb[n + j] : 0.0f;
      bias[j] = j < left && p.bias != nullptr ? p.bias[n + j] : 0.0f;
    }
#pragma unroll
    for (int r = lane / kLanes; r < 32; r += kRowsAtOnce) {
      const int64_t m = m0 + r;
      if (m >= p.M) break;
      int v[kE];
#pragma unroll
      for (int j = 0; j < kE; j += 4) {
        const i32x4 u = *reinterpret_cast<const i32x4*>(lds + r * kPitch + kE * (lane % kLanes) + j);
        v[j] = u[0];
        v[j + 1] = u[1];
        v[j + 2] = u[2];
        v[j + 3] = u[3];
      }
      store_outputs<T, kE>(v, p.sa[m], sb, bias, (T*)p.out + m * p.out_stride + n, left);
    }
  }
}

// Tiles of 128 tokens x 128 channels through registers: rows may start at any
// byte and K may be anything.  Four wavefronts, each 64 x 64 as 2 x 2 tiles
// of the 32x32x32 instruction; 64 codes of K at a time, the next 64 loaded
// while the matrix cores work on these.
//
// In LDS a row of 64 codes is four 16-byte pieces; piece c of row r lies at
// position c ^ swizzle(r), which spreads the sixteen lanes that read together
// over all banks.
__device__ __forceinline__ int piece_swizzle(int row) {
  return ((row >> 2) & 1) << 1 | (((row >> 1) ^ (row >> 3)) & 1);
}

template <typename T>
__global__ __launch_bounds__(256) void product_any_kernel(ProductArgs p) {
  __shared__ __align__(16) int8_t s_tile[2 * 128 * 64 > 4 * 32 * 68 * 4 ? 2 * 128 * 64
                                                                       : 4 * 32 * 68 * 4];
  int8_t* s_a = s_tile;
  int8_t* s_b = s_tile + 128 * 64;
  const int lane = (int)(threadIdx.x & 63u), wave = (int)(threadIdx.x >> 6);
  const int64_t m0 = (int64_t)(blockIdx.x / p.tiles_n) * 128;
  const int64_t n0 = (int64_t)(blockIdx.x % p.tiles_n) * 128;
  const int row = (int)(threadIdx.x >> 2), piece = (int)(threadIdx.x & 3u);
  i32x4 ra[2], rb[2];
  auto load = [&](int32_t k0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t m = m0 + row + 64 * i, n = n0 + row + 64 * i;
      ra[i] = m < p.M ? load16(p.a + m * p.a_stride, k0 + 16 * piece, p.K) : i32x4{0, 0, 0, 0};
      rb[i] = n < p.N ? load16(p.b + n * p.b_stride, k0 + 16 * piece, p.K) : i32x4{0, 0, 0, 0};
    }
  };
  i32x16 acc[2][2] = {};  // [token tile][channel tile]
  load(0);
  for (int32_t k0 = 0; k0 < p.K; k0 += 64) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = row + 64 * i, at = r * 64 + 16 * (piece ^ piece_swizzle(r));
      *reinterpret_cast<i32x4*>(s_a + at) = ra[i];
      *reinterpret_cast<i32x4*>(s_b + at) = rb[i];
    }
    __syncthreads();
    if (k0 + 64 < p.K) load(k0 + 64);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      i32x4 fa[2], fb[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int r = 32 * t + (lane & 31);
        const int at = 16 * ((2 * k + (lane >> 5)) ^ piece_swizzle(r));
        fa[t] = *reinterpret_cast<const i32x4*>(s_a + (64 * (wave >> 1) + r) * 64 + at);
        fb[t] = *reinterpret_cast<const i32x4*>(s_b + (64 * (wave & 1) + r) * 64 + at);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[j], fa[i], acc[i][j], 0, 0, 0);
    }
  }
  __syncthreads();
  int* strip = reinterpret_cast<int*>(s_tile) + wave * 32 * 68;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    store_strip<T, 2>(p, acc[i], strip, m0 + 64 * (wave >> 1) + 32 * i, n0 + 64 * (wave & 1));
}

}  // namespace fn
