// Row-wise kernels' shared pieces: rows of D values spread over lanes in chunks of eight (internal
// header). Chunk c of a row holds values 8 c .. 8 c + 7; a row of `LPR` lanes gives lane l the chunks
// l, l + LPR, ...
#pragma once
#include "pg_common.h"

namespace pg {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));

// A chunk as it lies in memory, so that a load can be held in flight and unpacked when it is used: values
// 8 c .. 8 c + 7, zeros past D. It is one (bf16) or two (f32) 16-byte loads, which need no more than the
// element's own alignment on this hardware: rows of any width are read the same way. A chunk that the row's
// end cuts off is read from D - 8 on and moved into place by `place`, before `unpack` (chunks wholly past the
// end become zeros); nothing waits for a load before that. Rows of less than eight values are for load_chunk below.
constexpr int kRowChunkMin = 8;
__device__ __forceinline__ int chunk_start(int c, int D) { return 8 * c + 8 <= D ? 8 * c : D - 8; }

template <typename T>
struct RawChunk;
template <>
struct RawChunk<uint16_t> {
  u32x4 a;
  __device__ __forceinline__ void load(const uint16_t* row, int c, int D) {
    a = *reinterpret_cast<const u32x4_a2*>(row + chunk_start(c, D));
  }
  __device__ __forceinline__ void place(int c, int D) {
    const int k = 8 * c + 8 - D;   // values past the end
    if (k > 0) {
      uint64_t lo = a[0] | (uint64_t)a[1] << 32, hi = a[2] | (uint64_t)a[3] << 32;
      if (k & 4 || k >= 8) {
        lo = hi;
        hi = 0;
      }
      const int sh = 16 * (k & 3);
      lo = k >= 8 ? 0 : lo >> sh | hi << 1 << (63 - sh);
      hi = k >= 8 ? 0 : hi >> sh;
      a = u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
    }
  }
  __device__ __forceinline__ void unpack(float* v) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(a[j] << 16);
      v[2 * j + 1] = __uint_as_float(a[j] & 0xffff0000u);
    }
  }
};
template <>
struct RawChunk<float> {
  float f[8];
  __device__ __forceinline__ void load(const float* row, int c, int D) {
    const float* p = row + chunk_start(c, D);
    const u32x4_a4 a = reinterpret_cast<const u32x4_a4*>(p)[0], b = reinterpret_cast<const u32x4_a4*>(p)[1];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[j] = __uint_as_float(a[j]);
      f[4 + j] = __uint_as_float(b[j]);
    }
  }
  __device__ __forceinline__ void place(int c, int D) {
    const int k = 8 * c + 8 - D;   // values past the end
    if (k > 0) {
#pragma unroll
      for (int by = 4; by; by >>= 1)
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = k & by ? (j + by < 8 ? f[j + by] : 0.f) : f[j];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = k >= 8 ? 0.f : f[j];
    }
  }
  __device__ __forceinline__ void unpack(float* v) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = f[j];
  }
};

__device__ __forceinline__ float row_value(const float* row, int64_t i) { return row[i]; }
__device__ __forceinline__ float row_value(const uint16_t* row, int64_t i) { return bf16_to_f32(row[i]); }

// A chunk loaded and unpacked at once, of rows of any width.
template <typename T>
__device__ __forceinline__ void load_chunk(const T* row, int c, int D, float* v) {
  if (D >= kRowChunkMin) {
    RawChunk<T> r;
    r.load(row, c, D);
    r.place(c, D);
    r.unpack(v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 8 * c + j < D ? row_value(row, 8 * (int64_t)c + j) : 0.f;
  }
}

// Eight values stored as chunk c, rounded once to the row's type (to nearest, ties to even).
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

// v of the lane that a DPP pattern within 16 lanes names (every lane has a partner in the patterns used
// here), and the sum of v and that.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}
template <int CTRL>
__device__ __forceinline__ float add_dpp(float v) {
  return v + __uint_as_float(dpp<CTRL>(__float_as_uint(v)));
}
template <int CTRL>
__device__ __forceinline__ double add_dpp(double v) {
  return v + __hiloint2double((int)dpp<CTRL>((uint32_t)__double2hiint(v)), (int)dpp<CTRL>((uint32_t)__double2loint(v)));
}
// The same across the neighbouring 16 and 32 lanes: a swap of the halves of two copies leaves the lower
// half's values in one and the upper half's in the other.
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
template <int N>
__device__ __forceinline__ u32x2 swap_lanes(uint32_t v) {
  if constexpr (N == 16) return __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(v, v, false, false));
  else return __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(v, v, false, false));
}
template <int N>
__device__ __forceinline__ float add_swapped(float v) {
  const u32x2 s = swap_lanes<N>(__float_as_uint(v));
  return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}
template <int N>
__device__ __forceinline__ double add_swapped(double v) {
  const u32x2 lo = swap_lanes<N>((uint32_t)__double2loint(v)), hi = swap_lanes<N>((uint32_t)__double2hiint(v));
  return __hiloint2double((int)hi[0], (int)lo[0]) + __hiloint2double((int)hi[1], (int)lo[1]);
}

// Sum over a group of LPR lanes, the same value in each, in a fixed order, without an LDS round trip:
// the neighbour, the other pair of the quad, the mirrored quad and eight, then 16 and 32 lanes.
template <int LPR, typename T>
__device__ __forceinline__ T group_sum(T v) {
  static_assert(LPR >= 16, "runs of 16 lanes");
  v = add_dpp<0xB1>(v);    // quad_perm 1, 0, 3, 2
  v = add_dpp<0x4E>(v);    // quad_perm 2, 3, 0, 1
  v = add_dpp<0x141>(v);   // row_half_mirror
  v = add_dpp<0x140>(v);   // row_mirror
  if constexpr (LPR >= 32) v = add_swapped<16>(v);
  if constexpr (LPR >= 64) v = add_swapped<32>(v);
  return v;
}

// 1 / sqrt(v) in float64: the hardware's approximation (at least 20 bits) and two Newton steps, each of
// which doubles the bits. 0 gives NaN (an infinity times zero in the steps).
__device__ __forceinline__ double rsqrt_f64(double v) {
  double r = __builtin_amdgcn_rsq(v);
#pragma unroll
  for (int i = 0; i < 2; ++i) r = r * __builtin_fma(-0.5 * v * r, r, 1.5);
  return r;
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

// Widest row that a wave holds in registers (64 lanes, two chunks each), and a workgroup (16 waves, a chunk
// per lane); wider ones are read once per pass by a workgroup each.
constexpr int kRowWaveMax = 64 * 2 * 8;
constexpr int kRowGroupWaves = 16;
constexpr int kRowGroupMax = kRowGroupWaves * 64 * 8;

// The waves of a workgroup that holds rows of D values, a chunk per lane.
__host__ __device__ inline int row_group_waves(int32_t D) { return (D + 511) / 512; }

// A barrier for what the waves exchange through LDS alone: loads from memory stay in flight across it (a
// whole __syncthreads waits for them).
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// The first half of a sum over a workgroup of up to kRowGroupWaves waves: each wave's sum to LDS. After the
// barrier, wave_sums gives every lane the whole, in one fixed order. sh is written again two barriers later.
template <typename T>
__device__ __forceinline__ void put_wave_sum(T v, T* sh) {
  v = group_sum<64>(v);
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
}
template <typename T>
__device__ __forceinline__ T wave_sums(const T* sh, int waves) {
  const int l = threadIdx.x & 15;
  return group_sum<16>(l < waves ? sh[l] : (T)0);
}

}  // namespace pg
