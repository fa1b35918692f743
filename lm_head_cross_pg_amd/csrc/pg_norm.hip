// Layer norm of the model's last hidden states (the final norm in front of the tied head: README
// leaderboard and trios issue name the tied head on the model's last states), forward and backward.
//
//   forward    mean = sum_d x / D, var = sum_d (x - mean)^2 / D, r = 1 / sqrt(var + eps)
//              xh = (x - mean) r,  y = xh w + b
//   backward   g = dy w,  dx = r (g - sum_d g / D - xh sum_d (g xh) / D)
//              dw = sum_t dy xh,  db = sum_t dy
//
// Both move each row once and are bound by HBM: a row is held in registers by the lanes that read it, one
// wave's or, past 1024 values, one workgroup's, and the row after it is loaded meanwhile. Measured (a copy
// reaches 5.0 TB/s): forward bf16 to bf16, 65536 x 512 in 24 us and 8192 x 4096 in 28 (5.6 and 4.7 TB/s); to
// 4 bits, 65536 x 512 in 29 us, where the arithmetic and no longer memory is the bound (2.9 TB/s); backward of
// bf16 x, float32 dy and dx, 65536 x 512 in 64 us and 8192 x 4096 in 63 (5.2 TB/s), with the sums' 4 to 5.
// The statistics and the forward's values are formed in float64, which costs no more issue time than
// float32 without packed operations (5.1 against 5.7 cycles per operation and wave) and is hidden
// under the loads: a row with a mean far above its deviation loses nothing, and the float32 value that
// is stored or quantised is the correctly rounded one but for one value in about 10^8, so the 4-bit
// form does not depend on the order of a sum.
// Rows that score_mask leaves out are neither read nor written by the forward; the backward gives them
// zero gradients.
#include "pg_internal.h"
#include "pg_mx4.h"
#include "pg_rows.h"

namespace pg {

struct Mx4Out {};   // output in 4 bits

struct NormParams {
  const void* x;
  const float* weight;   // nullptr: ones
  const float* bias;     // nullptr: zeros
  const uint8_t* mask;
  int64_t T;
  int32_t D;
  double eps, inv_d;       // inv_d = 1 / D
  void* y;               // float or bf16 rows, or the codes
  uint8_t* scales;
};

// Rows that lanes hold in registers; the others (wider than a workgroup's registers, or less than a chunk) are
// read anew for each pass.
static bool row_held(int32_t D) { return D >= kRowChunkMin && D <= kRowGroupMax; }

// The gain and bias of chunk c (ones and zeros where there are none).
__device__ __forceinline__ void norm_params_chunk(const NormParams& p, int c, float* w, float* b) {
  if (p.weight) load_chunk(p.weight, c, p.D, w);
  if (p.bias) load_chunk(p.bias, c, p.D, b);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (!p.weight) w[j] = 1.f;
    if (!p.bias) b[j] = 0.f;
  }
}

// A chunk's values as float32: xh w + b in float64, rounded once.
__device__ __forceinline__ void norm_chunk(const float* x, const float* w, const float* b, double mean, double r,
                                           float* v) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = (float)__builtin_fma(((double)x[j] - mean) * r, (double)w[j], (double)b[j]);
}

template <typename TOut>
__device__ __forceinline__ void norm_store(const NormParams& p, int64_t t, int c, float* v) {
  if constexpr (std::is_same<TOut, Mx4Out>::value) {
    if (8 * c + 8 > p.D) {   // the row's padding is zero whatever its bias
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 8 * c + j < p.D ? v[j] : 0.f;
    }
    mx4_store_chunk(v, c, p.D, static_cast<uint8_t*>(p.y) + t * mx4_code_bytes(p.D),
                    p.scales + t * mx4_scale_bytes(p.D));
  } else {
    store_chunk(static_cast<TOut*>(p.y) + t * p.D, c, p.D, v);
  }
}

// Rows up to kRowWaveMax: LPR lanes hold a row, K chunks each, and a wave 64 / LPR rows.
template <typename TX, typename TOut, int LPR, int K>
__global__ __launch_bounds__(256) void norm_rows_kernel(NormParams p) {
  constexpr int RPW = 64 / LPR;
  const int lane = threadIdx.x & 63, l = lane % LPR;
  const int64_t first = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 6)) * RPW + lane / LPR;
  const int64_t step = (int64_t)gridDim.x * 4 * RPW;
  const bool full = p.D == LPR * K * 8;   // no lane has values past the row's end
  // held as float64 where that leaves enough registers to keep several waves per SIMD
  typename std::conditional<K == 1, double, float>::type w[K][8], b[K][8];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    float wf[8], bf[8];
    norm_params_chunk(p, l + k * LPR, wf, bf);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      w[k][j] = wf[j];
      b[k][j] = bf[j];
    }
  }
  // the row after this one is on its way while this one is worked on
  RawChunk<TX> raw[K];
  auto fetch = [&](int64_t t) {
    const bool scored = t < p.T && !(p.mask && !p.mask[t]);
    if (scored) {
#pragma unroll
      for (int k = 0; k < K; ++k) raw[k].load(static_cast<const TX*>(p.x) + t * p.D, l + k * LPR, p.D);
    }
    return scored;
  };
  bool scored = fetch(first);
  for (int64_t t = first; t < p.T; t += step) {
    float x[K][8];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (!full) raw[k].place(l + k * LPR, p.D);
      raw[k].unpack(x[k]);
    }
    const bool now = scored;
    scored = fetch(t + step);
    if (!now) continue;
    double s = 0.0;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) s += (double)x[k][j];
    const double mean = group_sum<LPR>(s) * p.inv_d;
    double d[K][8];
    s = 0.0;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        d[k][j] = (double)x[k][j] - mean;
      }
    if (!full) {
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) d[k][j] = 8 * (l + k * LPR) + j < p.D ? d[k][j] : 0.0;
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) s = __builtin_fma(d[k][j], d[k][j], s);
    const double r = rsqrt_f64(__builtin_fma(group_sum<LPR>(s), p.inv_d, p.eps));
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = (float)__builtin_fma(d[k][j] * r, (double)w[k][j], (double)b[k][j]);
      norm_store<TOut>(p, t, l + k * LPR, v);
    }
  }
}

// Rows of up to kRowGroupMax: a workgroup holds a row, a chunk per lane (blockDim.x is 64 row_group_waves).
template <typename TX, typename TOut>
__global__ __launch_bounds__(64 * kRowGroupWaves) void norm_group_kernel(NormParams p) {
  __shared__ double sh[2][kRowGroupWaves];
  const int c = threadIdx.x, waves = blockDim.x >> 6;
  const bool full = p.D == 8 * (int)blockDim.x;   // no lane has values past the row's end
  double w[8], b[8];
  {
    float wf[8], bf[8];
    norm_params_chunk(p, c, wf, bf);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      w[j] = wf[j];
      b[j] = bf[j];
    }
  }
  // the row after this one is on its way while this one is worked on
  RawChunk<TX> raw;
  auto fetch = [&](int64_t t) {
    const bool scored = t < p.T && !(p.mask && !p.mask[t]);
    if (scored) raw.load(static_cast<const TX*>(p.x) + t * p.D, c, p.D);
    return scored;
  };
  bool scored = fetch(blockIdx.x);
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
    float x[8];
    if (!full) raw.place(c, p.D);
    raw.unpack(x);
    const bool now = scored;
    scored = fetch(t + gridDim.x);
    if (!now) continue;   // the same in every wave
    double s = 0.0;
#pragma unroll
    for (int j = 0; j < 8; ++j) s += (double)x[j];
    put_wave_sum(s, sh[0]);
    lds_barrier();
    const double mean = wave_sums(sh[0], waves) * p.inv_d;
    double d[8];
    s = 0.0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      d[j] = 8 * c + j < p.D ? (double)x[j] - mean : 0.0;
      s = __builtin_fma(d[j], d[j], s);
    }
    put_wave_sum(s, sh[1]);
    lds_barrier();
    const double r = rsqrt_f64(__builtin_fma(wave_sums(sh[1], waves), p.inv_d, p.eps));
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = (float)__builtin_fma(d[j] * r, w[j], b[j]);
    norm_store<TOut>(p, t, c, v);
  }
}

// Other rows: a workgroup per row, which reads it three times (from L2 after the first).
template <typename TX, typename TOut>
__global__ __launch_bounds__(kRowThreads) void norm_wide_kernel(NormParams p) {
  __shared__ double sh[kRowThreads / 64];
  const int nch = (p.D + 127) / 128 * 16;   // chunks, whole runs of 16 lanes
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
    if (p.mask && !p.mask[t]) continue;
    const TX* row = static_cast<const TX*>(p.x) + t * p.D;
    float x[8];
    double s = 0.0;
    for (int c = threadIdx.x; c < nch; c += kRowThreads) {
      load_chunk(row, c, p.D, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) s += (double)x[j];
    }
    const double mean = workgroup_sum(s, sh) * p.inv_d;
    s = 0.0;
    for (int c = threadIdx.x; c < nch; c += kRowThreads) {
      load_chunk(row, c, p.D, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const double d = 8 * c + j < p.D ? (double)x[j] - mean : 0.0;
        s = __builtin_fma(d, d, s);
      }
    }
    const double r = rsqrt_f64(__builtin_fma(workgroup_sum(s, sh), p.inv_d, p.eps));
    for (int c = threadIdx.x; c < nch; c += kRowThreads) {
      float v[8], w[8], b[8];
      load_chunk(row, c, p.D, x);
      norm_params_chunk(p, c, w, b);
      norm_chunk(x, w, b, mean, r, v);
      norm_store<TOut>(p, t, c, v);
    }
  }
}

// Waves of norm_group_kernel that a CU is given (its registers hold 20 to 28; 16 take 7 % longer at 8192 x 4096,
// 32 9 % longer at 11000 rows of odd length).
constexpr int kGroupResident = 24;
template <typename TX, typename TOut>
static void launch_norm_t(const NormParams& p, const DeviceInfo& dev, hipStream_t st) {
  const int D = p.D;
  if (!row_held(D)) {
    hipLaunchKernelGGL((norm_wide_kernel<TX, TOut>), dim3(stride_blocks(p.T, 1)), dim3(kRowThreads), 0, st, p);
    return;
  }
  if (D > kRowWaveMax) {
    const int waves = row_group_waves(D);
    const int64_t most = (int64_t)kGroupResident / waves * dev.cu_count;
    hipLaunchKernelGGL((norm_group_kernel<TX, TOut>), dim3((unsigned)(p.T < most ? p.T : most)), dim3(64 * waves), 0,
                       st, p);
    return;
  }
#define PG_NORM(LPR, K)                                                                                          \
  hipLaunchKernelGGL((norm_rows_kernel<TX, TOut, LPR, K>), dim3(resident_blocks(dev, p.T, 4 * (64 / LPR))),     \
                     dim3(256), 0, st, p)
  if (D <= 128) PG_NORM(16, 1);
  else if (D <= 256) PG_NORM(32, 1);
  else if (D <= 512) PG_NORM(64, 1);
  else PG_NORM(64, 2);
#undef PG_NORM
}

static NormParams norm_params(const void* x, const float* weight, const float* bias, const uint8_t* mask, int64_t T,
                              int32_t D, float eps, void* y, uint8_t* scales) {
  NormParams p{};
  p.x = x;
  p.weight = weight;
  p.bias = bias;
  p.mask = mask;
  p.T = T;
  p.D = D;
  p.eps = (double)eps;
  p.inv_d = 1.0 / D;
  p.y = y;
  p.scales = scales;
  return p;
}

hipError_t launch_norm(const void* x, int32_t dtype_x, const float* weight, const float* bias, const uint8_t* mask,
                       int64_t T, int32_t D, float eps, void* y, int32_t dtype_y,
                       const DeviceInfo& dev, hipStream_t st) {
  if (T == 0) return hipSuccess;
  const NormParams p = norm_params(x, weight, bias, mask, T, D, eps, y, nullptr);
  if (dtype_x == 0) {
    if (dtype_y == 0) launch_norm_t<uint16_t, uint16_t>(p, dev, st);
    else launch_norm_t<uint16_t, float>(p, dev, st);
  } else {
    if (dtype_y == 0) launch_norm_t<float, uint16_t>(p, dev, st);
    else launch_norm_t<float, float>(p, dev, st);
  }
  return hipGetLastError();
}

hipError_t launch_norm_mx4(const void* x, int32_t dtype_x, const float* weight, const float* bias,
                           const uint8_t* mask, int64_t T, int32_t D, float eps, uint8_t* codes, uint8_t* scales,
                           const DeviceInfo& dev, hipStream_t st) {
  if (T == 0) return hipSuccess;
  const NormParams p = norm_params(x, weight, bias, mask, T, D, eps, codes, scales);
  if (dtype_x == 0) launch_norm_t<uint16_t, Mx4Out>(p, dev, st);
  else launch_norm_t<float, Mx4Out>(p, dev, st);
  return hipGetLastError();
}

// ------------------------------------------------------------------------------------- backward

struct NormBwdParams {
  const void* x;
  const void* dy;
  const float* weight;
  const uint8_t* mask;
  int64_t T;
  int32_t D;
  double eps, inv_d;
  void* dx;       // nullptr: not wanted
  float* part;    // partial sums of dw and db per workgroup [blocks][2][D]; nullptr: not wanted
  double* stats;  // wide rows: mean and r of each row, for the column sums
};

// Rows up to kRowWaveMax. Each lane keeps the sums of dw and db over its rows for its own columns; at
// the end the waves of a workgroup add theirs in wave order through LDS, so that the result does not
// depend on timing.
template <int K>
struct NormBwdShape {
  // threads of a workgroup, at most: as many waves as share one partial sum, within the registers they need
  static constexpr int kThreads = K == 1 ? 1024 : 512;
};

template <typename TX, typename TDY, typename TDX, int LPR, int K>
__global__ __launch_bounds__(NormBwdShape<K>::kThreads) void norm_bwd_rows_kernel(NormBwdParams p) {
  constexpr int RPW = 64 / LPR;
  __shared__ float sums[2][LPR * K * 8];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6, l = lane % LPR;
  const bool full = p.D == LPR * K * 8;   // no lane has values past the row's end
  float w[K][8], dw[K][8], db[K][8];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (p.weight) load_chunk(p.weight, l + k * LPR, p.D, w[k]);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (!p.weight) w[k][j] = 1.f;
      dw[k][j] = db[k][j] = 0.f;
    }
  }
  const float invD = (float)p.inv_d;
  const int64_t first = ((int64_t)blockIdx.x * waves + wave) * RPW + lane / LPR;
  const int64_t step = (int64_t)gridDim.x * waves * RPW;
  // the row after this one is on its way while this one is worked on
  RawChunk<TX> rx[K];
  RawChunk<TDY> rdy[K];
  auto fetch = [&](int64_t t) {
    const bool scored = t < p.T && !(p.mask && !p.mask[t]);
    if (scored) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        rx[k].load(static_cast<const TX*>(p.x) + t * p.D, l + k * LPR, p.D);
        rdy[k].load(static_cast<const TDY*>(p.dy) + t * p.D, l + k * LPR, p.D);
      }
    }
    return scored;
  };
  bool scored = fetch(first);
  for (int64_t t = first; t < p.T; t += step) {
    TDX* dxrow = static_cast<TDX*>(p.dx) + t * p.D;
    float x[K][8], dy[K][8];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (!full) {
        rx[k].place(l + k * LPR, p.D);
        rdy[k].place(l + k * LPR, p.D);
      }
      rx[k].unpack(x[k]);
      rdy[k].unpack(dy[k]);
    }
    const bool now = scored;
    scored = fetch(t + step);
    if (!now) {
      if (p.dx) {
        const float zero[8] = {};
#pragma unroll
        for (int k = 0; k < K; ++k) store_chunk(dxrow, l + k * LPR, p.D, zero);
      }
      continue;
    }
    double s = 0.0;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) s += (double)x[k][j];
    const double mean = group_sum<LPR>(s) * p.inv_d;
    s = 0.0;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        double d = (double)x[k][j] - mean;
        if (8 * (l + k * LPR) + j >= p.D) d = 0.0;
        x[k][j] = (float)d;
        s = __builtin_fma(d, d, s);
      }
    const float r = (float)rsqrt_f64(__builtin_fma(group_sum<LPR>(s), p.inv_d, p.eps));
    float c1 = 0.f, c2 = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float xh = x[k][j] * r, g = dy[k][j] * w[k][j];
        x[k][j] = xh;
        c1 += g;
        c2 = __builtin_fmaf(g, xh, c2);
        dw[k][j] = __builtin_fmaf(dy[k][j], xh, dw[k][j]);
        db[k][j] += dy[k][j];
      }
    c1 = group_sum<LPR>(c1) * invD;
    c2 = group_sum<LPR>(c2) * invD;
    if (p.dx) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = r * (__builtin_fmaf(dy[k][j], w[k][j], -c1) - x[k][j] * c2);
        store_chunk(dxrow, l + k * LPR, p.D, v);
      }
    }
  }
  if (!p.part) return;
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) {   // the rows that the wave's groups hold side by side
#pragma unroll
      for (int off = LPR; off < 64; off <<= 1) {
        dw[k][j] += __shfl_xor(dw[k][j], off);
        db[k][j] += __shfl_xor(db[k][j], off);
      }
    }
  for (int q = 0; q < waves; ++q) {
    if (wave == q && lane < LPR) {
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float* a = &sums[0][(j * K + k) * LPR + l];   // lanes side by side: no two in one bank
          float* b = &sums[1][(j * K + k) * LPR + l];
          *a = q ? *a + dw[k][j] : dw[k][j];
          *b = q ? *b + db[k][j] : db[k][j];
        }
    }
    __syncthreads();
  }
  float* part = p.part + (int64_t)blockIdx.x * 2 * p.D;
  for (int d = threadIdx.x; d < p.D; d += blockDim.x) {
    const int c = d >> 3, at = ((d & 7) * K + c / LPR) * LPR + c % LPR;
    part[d] = sums[0][at];
    part[p.D + d] = sums[1][at];
  }
}

// Rows of up to kRowGroupMax: a workgroup holds a row, a chunk per lane (blockDim.x is 64 row_group_waves),
// and each lane the sums of its own eight columns.
template <typename TX, typename TDY, typename TDX>
__global__ __launch_bounds__(64 * kRowGroupWaves) void norm_bwd_group_kernel(NormBwdParams p) {
  __shared__ double sh[2][kRowGroupWaves];
  __shared__ float shf[2][kRowGroupWaves];
  const int c = threadIdx.x, waves = blockDim.x >> 6;
  const bool full = p.D == 8 * (int)blockDim.x;   // no lane has values past the row's end
  float w[8], dw[8] = {}, db[8] = {};
  if (p.weight) load_chunk(p.weight, c, p.D, w);
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = p.weight ? w[j] : 1.f;
  const float invD = (float)p.inv_d;
  // the row after this one is on its way while this one is worked on
  RawChunk<TX> rx;
  RawChunk<TDY> rdy;
  auto fetch = [&](int64_t t) {
    const bool scored = t < p.T && !(p.mask && !p.mask[t]);
    if (scored) {
      rx.load(static_cast<const TX*>(p.x) + t * p.D, c, p.D);
      rdy.load(static_cast<const TDY*>(p.dy) + t * p.D, c, p.D);
    }
    return scored;
  };
  bool scored = fetch(blockIdx.x);
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
    TDX* dxrow = static_cast<TDX*>(p.dx) + t * p.D;
    float x[8], dy[8];
    if (!full) {
      rx.place(c, p.D);
      rdy.place(c, p.D);
    }
    rx.unpack(x);
    rdy.unpack(dy);
    const bool now = scored;
    scored = fetch(t + gridDim.x);
    if (!now) {   // the same in every wave
      const float zero[8] = {};
      if (p.dx) store_chunk(dxrow, c, p.D, zero);
      continue;
    }
    double s = 0.0;
#pragma unroll
    for (int j = 0; j < 8; ++j) s += (double)x[j];
    put_wave_sum(s, sh[0]);
    lds_barrier();
    const double mean = wave_sums(sh[0], waves) * p.inv_d;
    float c1 = 0.f, c2 = 0.f;
    s = 0.0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const double d = 8 * c + j < p.D ? (double)x[j] - mean : 0.0;
      s = __builtin_fma(d, d, s);
      x[j] = (float)d;
      const float g = dy[j] * w[j];
      c1 += g;
      c2 = __builtin_fmaf(g, x[j], c2);
    }
    put_wave_sum(s, sh[1]);
    put_wave_sum(c1, shf[0]);
    put_wave_sum(c2, shf[1]);
    lds_barrier();
    const float r = (float)rsqrt_f64(__builtin_fma(wave_sums(sh[1], waves), p.inv_d, p.eps));
    c1 = wave_sums(shf[0], waves) * invD;
    c2 = wave_sums(shf[1], waves) * r * invD;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float xh = x[j] * r;
      dw[j] = __builtin_fmaf(dy[j], xh, dw[j]);
      db[j] += dy[j];
      v[j] = r * (__builtin_fmaf(dy[j], w[j], -c1) - xh * c2);
    }
    if (p.dx) store_chunk(dxrow, c, p.D, v);
  }
  if (!p.part) return;
  float* part = p.part + (int64_t)blockIdx.x * 2 * p.D;
  store_chunk(part, c, p.D, dw);
  store_chunk(part + p.D, c, p.D, db);
}

// Other rows: dx by a workgroup per row, the row's statistics kept for the column sums.
template <typename TX, typename TDY, typename TDX>
__global__ __launch_bounds__(kRowThreads) void norm_bwd_wide_kernel(NormBwdParams p) {
  __shared__ double sh[kRowThreads / 64];
  const int nch = (p.D + 7) / 8;
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
    TDX* dxrow = static_cast<TDX*>(p.dx) + t * p.D;
    if (p.mask && !p.mask[t]) {
      const float zero[8] = {};
      if (p.dx)
        for (int c = threadIdx.x; c < nch; c += kRowThreads) store_chunk(dxrow, c, p.D, zero);
      continue;
    }
    const TX* row = static_cast<const TX*>(p.x) + t * p.D;
    const TDY* dyrow = static_cast<const TDY*>(p.dy) + t * p.D;
    float x[8], dy[8], w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = 1.f;
    double s = 0.0;
    for (int c = threadIdx.x; c < nch; c += kRowThreads) {
      load_chunk(row, c, p.D, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) s += (double)x[j];
    }
    const double mean = workgroup_sum(s, sh) * p.inv_d;
    double c1 = 0.0, c2 = 0.0;
    s = 0.0;
    for (int c = threadIdx.x; c < nch; c += kRowThreads) {
      load_chunk(row, c, p.D, x);
      load_chunk(dyrow, c, p.D, dy);
      if (p.weight) load_chunk(p.weight, c, p.D, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const double d = 8 * c + j < p.D ? (double)x[j] - mean : 0.0;
        const double g = (double)dy[j] * (double)w[j];
        s = __builtin_fma(d, d, s);
        c1 += g;
        c2 = __builtin_fma(g, d, c2);
      }
    }
    const double r = rsqrt_f64(__builtin_fma(workgroup_sum(s, sh), p.inv_d, p.eps));
    c1 = workgroup_sum(c1, sh) * p.inv_d;
    c2 = workgroup_sum(c2, sh) * r * p.inv_d;
    if (p.stats && threadIdx.x == 0) {
      p.stats[2 * t] = mean;
      p.stats[2 * t + 1] = r;
    }
    if (!p.dx) continue;
    for (int c = threadIdx.x; c < nch; c += kRowThreads) {
      float v[8];
      load_chunk(row, c, p.D, x);
      load_chunk(dyrow, c, p.D, dy);
      if (p.weight) load_chunk(p.weight, c, p.D, w);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        v[j] = (float)(r * ((double)dy[j] * (double)w[j] - c1 - ((double)x[j] - mean) * r * c2));
      store_chunk(dxrow, c, p.D, v);
    }
  }
}

// Column sums of wide rows: thread = eight columns, workgroup (x, y) = a run of columns of every
// gridDim.y-th row from y on.
template <typename TX, typename TDY>
__global__ __launch_bounds__(kRowThreads) void norm_bwd_columns_kernel(NormBwdParams p) {
  const int c = blockIdx.x * kRowThreads + threadIdx.x;
  if (8 * (int64_t)c >= p.D) return;
  double dw[8] = {}, db[8] = {};
  for (int64_t t = blockIdx.y; t < p.T; t += gridDim.y) {
    if (p.mask && !p.mask[t]) continue;
    float x[8], dy[8];
    load_chunk(static_cast<const TX*>(p.x) + t * p.D, c, p.D, x);
    load_chunk(static_cast<const TDY*>(p.dy) + t * p.D, c, p.D, dy);
    const double mean = p.stats[2 * t], r = p.stats[2 * t + 1];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      dw[j] = __builtin_fma((double)dy[j], ((double)x[j] - mean) * r, dw[j]);
      db[j] += (double)dy[j];
    }
  }
  float* part = p.part + (int64_t)blockIdx.y * 2 * p.D;
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = (float)dw[j];
  store_chunk(part, c, p.D, v);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = (float)db[j];
  store_chunk(part + p.D, c, p.D, v);
}

// dw and db from the partial sums, in block order in float64: wave w of a workgroup takes every 16th
// block from w on for 64 columns, and the waves' sums are added in wave order.
constexpr int kNormSumThreads = 1024;
__global__ __launch_bounds__(kNormSumThreads) void norm_bwd_sum_kernel(const float* part, int blocks, int D, float* dw,
                                                                       float* db) {
  __shared__ double sh[kNormSumThreads / 64][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t i = (int64_t)blockIdx.x * 64 + lane, n = 2 * (int64_t)D;
  constexpr int kWaves = kNormSumThreads / 64, kBatch = 8;   // loads of a batch are in flight together
  double s = 0.0;
  if (i < n) {
    int b = wave;
    for (; b + (kBatch - 1) * kWaves < blocks; b += kBatch * kWaves) {
      float v[kBatch];
#pragma unroll
      for (int q = 0; q < kBatch; ++q) v[q] = part[(int64_t)(b + q * kWaves) * n + i];
#pragma unroll
      for (int q = 0; q < kBatch; ++q) s += (double)v[q];
    }
    for (; b < blocks; b += kWaves) s += (double)part[(int64_t)b * n + i];
  }
  sh[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && i < n) {
    for (int w = 1; w < kNormSumThreads / 64; ++w) s += sh[w][lane];
    if (i < D) {
      if (dw) dw[i] = (float)s;
    } else if (db) {
      db[i - D] = (float)s;
    }
  }
}

// Workgroups of the backward, and partial sums: one per CU, and more where a lane would add over
// kNormLaneRows rows in float32 (the partial sums are added in float64).
constexpr int kNormBwdBlocks = 256;
constexpr int64_t kNormLaneRows = 512;
constexpr int kNormColumnRows = 64;     // rows of T that split the column sums of wide rows, at most

// The backward's launch for rows that waves hold: lanes per row, chunks per lane, waves per workgroup (four
// where that keeps every workgroup at work, up to the most where rows are many), workgroups.
struct NormBwdLaunch {
  int lpr, chunks, waves, blocks;
};
static NormBwdLaunch norm_bwd_launch(int64_t T, int32_t D) {
  NormBwdLaunch L;
  if (D > kRowWaveMax) {   // a workgroup per row, side by side on a CU up to about eight waves (8192 x 4096: one
                           // of eight waves 64 us, two 69, since twice the partial sums are written and read)
    L.lpr = L.chunks = 0;
    L.waves = row_group_waves(D);
    const int64_t side = (T + kNormLaneRows - 1) / kNormLaneRows, least = kNormBwdBlocks * ((7 + L.waves) / L.waves);
    const int64_t most = side > least ? side : least;
    L.blocks = (int)(T < most ? T : most);
    return L;
  }
  L.lpr = D <= 128 ? 16 : D <= 256 ? 32 : 64;
  L.chunks = D <= 512 ? 1 : 2;
  const int most = (L.chunks == 1 ? NormBwdShape<1>::kThreads : NormBwdShape<2>::kThreads) / 64;
  const int64_t rows = (T + 64 / L.lpr - 1) / (64 / L.lpr);   // per wave, side by side
  L.waves = 4;
  while (L.waves < most && rows > (int64_t)L.waves * kNormBwdBlocks) L.waves *= 2;
  const int64_t need = (rows + L.waves - 1) / L.waves;
  const int64_t cap = (need + kNormLaneRows - 1) / kNormLaneRows;
  const int64_t most_blocks = cap > kNormBwdBlocks ? cap : kNormBwdBlocks;
  L.blocks = (int)(need < most_blocks ? need : most_blocks);
  return L;
}

NormBwdWorkspace norm_bwd_workspace(int64_t T, int32_t D) {
  NormBwdWorkspace L;
  const bool wide = !row_held(D);
  L.part = 0;
  L.stats = align256((size_t)(wide ? kNormColumnRows : norm_bwd_launch(T, D).blocks) * 2 * (size_t)D * 4);
  L.total = L.stats + (wide ? align256((size_t)T * 16) : 0);
  return L;
}

template <typename TX, typename TDY, typename TDX>
static void launch_norm_bwd_t(const NormBwdParams& p, int& blocks, hipStream_t st) {
  const int D = p.D;
  if (!row_held(D)) {
    hipLaunchKernelGGL((norm_bwd_wide_kernel<TX, TDY, TDX>), dim3(stride_blocks(p.T, 1)), dim3(kRowThreads), 0, st, p);
    if (p.part) {
      blocks = (int)(p.T < kNormColumnRows ? p.T : kNormColumnRows);
      hipLaunchKernelGGL((norm_bwd_columns_kernel<TX, TDY>), dim3((D + 8 * kRowThreads - 1) / (8 * kRowThreads), blocks),
                         dim3(kRowThreads), 0, st, p);
    }
    return;
  }
  const NormBwdLaunch L = norm_bwd_launch(p.T, D);
  blocks = L.blocks;
#define PG_NORM_BWD(LPR, K) \
  hipLaunchKernelGGL((norm_bwd_rows_kernel<TX, TDY, TDX, LPR, K>), dim3(blocks), dim3(64 * L.waves), 0, st, p)
  if (L.chunks == 0)
    hipLaunchKernelGGL((norm_bwd_group_kernel<TX, TDY, TDX>), dim3(blocks), dim3(64 * L.waves), 0, st, p);
  else if (L.lpr == 16) PG_NORM_BWD(16, 1);
  else if (L.lpr == 32) PG_NORM_BWD(32, 1);
  else if (L.chunks == 1) PG_NORM_BWD(64, 1);
  else PG_NORM_BWD(64, 2);
#undef PG_NORM_BWD
}

hipError_t launch_norm_bwd(const void* x, int32_t dtype_x, const float* weight, const uint8_t* mask, const void* dy,
                           int32_t dtype_dy, int64_t T, int32_t D, float eps, void* dx, int32_t dtype_dx,
                           float* dweight, float* dbias, char* ws, const DeviceInfo& dev, hipStream_t st) {
  const NormBwdWorkspace L = norm_bwd_workspace(T, D);
  NormBwdParams p{};
  p.x = x;
  p.dy = dy;
  p.weight = weight;
  p.mask = mask;
  p.T = T;
  p.D = D;
  p.eps = (double)eps;
  p.inv_d = 1.0 / D;
  p.dx = dx;
  if (dweight || dbias) {
    p.part = reinterpret_cast<float*>(ws + L.part);
    p.stats = reinterpret_cast<double*>(ws + L.stats);
  }
  int blocks = 0;
  if (T > 0) {
    const int code = dtype_x * 4 + dtype_dy * 2 + dtype_dx;
    switch (code) {
      case 0: launch_norm_bwd_t<uint16_t, uint16_t, uint16_t>(p, blocks, st); break;
      case 1: launch_norm_bwd_t<uint16_t, uint16_t, float>(p, blocks, st); break;
      case 2: launch_norm_bwd_t<uint16_t, float, uint16_t>(p, blocks, st); break;
      case 3: launch_norm_bwd_t<uint16_t, float, float>(p, blocks, st); break;
      case 4: launch_norm_bwd_t<float, uint16_t, uint16_t>(p, blocks, st); break;
      case 5: launch_norm_bwd_t<float, uint16_t, float>(p, blocks, st); break;
      case 6: launch_norm_bwd_t<float, float, uint16_t>(p, blocks, st); break;
      default: launch_norm_bwd_t<float, float, float>(p, blocks, st); break;
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!p.part) return hipSuccess;
  // no rows: the sums of nothing
  hipLaunchKernelGGL(norm_bwd_sum_kernel, dim3((unsigned)((2 * (int64_t)D + 63) / 64)), dim3(kNormSumThreads), 0, st,
                     p.part, blocks, D, dweight, dbias);
  return hipGetLastError();
}

}  // namespace pg
