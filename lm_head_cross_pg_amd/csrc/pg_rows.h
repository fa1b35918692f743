// Row-wise kernels' shared pieces: rows of D values spread over lanes in chunks of eight (internal
// header). Chunk c of a row holds values 8 c .. 8 c + 7; a row of `LPR` lanes gives lane l the chunks
// l, l + LPR, ...
#pragma once
#include "pg_common.h"

namespace pg {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));

// Eight values of a row from element 8 c on, zeros past D. A whole chunk is one (bf16) or two (f32)
// 16-byte loads, which need no more than the element's own alignment on this hardware: rows of any
// width are read the same way.
__device__ __forceinline__ void load_chunk(const float* row, int c, int D, float* v) {
  if (8 * c + 8 <= D) {
    const u32x4_a4 a = reinterpret_cast<const u32x4_a4*>(row + 8 * (int64_t)c)[0];
    const u32x4_a4 b = reinterpret_cast<const u32x4_a4*>(row + 8 * (int64_t)c)[1];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = __uint_as_float(a[j]);
      v[4 + j] = __uint_as_float(b[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 8 * c + j < D ? row[8 * (int64_t)c + j] : 0.f;
  }
}
__device__ __forceinline__ void load_chunk(const uint16_t* row, int c, int D, float* v) {
  if (8 * c + 8 <= D) {
    const u32x4_a2 a = *reinterpret_cast<const u32x4_a2*>(row + 8 * (int64_t)c);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(a[j] << 16);
      v[2 * j + 1] = __uint_as_float(a[j] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 8 * c + j < D ? bf16_to_f32(row[8 * (int64_t)c + j]) : 0.f;
  }
}

// The same eight values stored, rounded once to the row's type (to nearest, ties to even).
__device__ __forceinline__ void store_chunk(float* row, int c, int D, const float* v) {
  if (8 * c + 8 <= D) {
    u32x4_a4 a, b;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      a[j] = __float_as_uint(v[j]);
      b[j] = __float_as_uint(v[4 + j]);
    }
    reinterpret_cast<u32x4_a4*>(row + 8 * (int64_t)c)[0] = a;
    reinterpret_cast<u32x4_a4*>(row + 8 * (int64_t)c)[1] = b;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (8 * c + j < D) row[8 * (int64_t)c + j] = v[j];
  }
}
__device__ __forceinline__ void store_chunk(uint16_t* row, int c, int D, const float* v) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  u32x4_a2 o;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f32x2 f;
    f[0] = v[2 * j];
    f[1] = v[2 * j + 1];
    o[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2));
  }
  if (8 * c + 8 <= D) {
    *reinterpret_cast<u32x4_a2*>(row + 8 * (int64_t)c) = o;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (8 * c + j < D) row[8 * (int64_t)c + j] = (uint16_t)(o[j >> 1] >> (16 * (j & 1)));
  }
}

// Sum over a group of LPR lanes, the same value in each (a butterfly: a fixed order).
template <int LPR, typename T>
__device__ __forceinline__ T group_sum(T v) {
#pragma unroll
  for (int off = LPR / 2; off >= 1; off >>= 1) v += __shfl_xor(v, off);
  return v;
}

// Sum over a workgroup of kRowThreads threads, the same value in each: the waves' sums in wave order.
constexpr int kRowThreads = 256;
template <typename T>
__device__ __forceinline__ T workgroup_sum(T v, T* sh) {
  v = group_sum<64>(v);
  __syncthreads();   // the previous sum has been read
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
  __syncthreads();
  T s = sh[0];
#pragma unroll
  for (int w = 1; w < kRowThreads / 64; ++w) s += sh[w];
  return s;
}

// Widest row that a wave holds in registers (64 lanes, four chunks each); wider ones are read once per
// pass by a workgroup each.
constexpr int kRowWaveMax = 64 * 4 * 8;

}  // namespace pg
