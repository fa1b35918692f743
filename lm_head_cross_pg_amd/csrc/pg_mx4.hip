// Rows of bf16 or float32 values to the microscaled 4-bit format and back (pg_mx4.h): the quantised
// tied embedding and the states that meet it in the 4-bit head, and the fake quantisation of
// quantisation-aware training (trios issue #19, approach table, "Квантование": INT4/INT8; README
// leaderboard, QAT rows). Both are one pass over the data, bound by HBM: a lane holds eight values, four lanes a
// block of 32, so that a block's largest magnitude takes two lane exchanges. 32768 x 1024 float32 values take
// 25 us (6.2 TB/s read and written) to 4 bits and 27 back; 65536 x 512 bf16 ones 16 (5.2) and 15 (5.7 TB/s; 21
// with the levels formed by integer arithmetic instead of the hardware's conversion).
#include "pg_internal.h"
#include "pg_mx4.h"
#include "pg_rows.h"

namespace pg {

// Rows of LPR lanes that walk the row in steps of LPR chunks. Rows that the mask leaves out are neither
// read nor written.
template <typename TIn, int LPR>
__global__ __launch_bounds__(256) void quantize_mx4_kernel(const TIn* x, const uint8_t* mask, int64_t T, int D,
                                                           uint8_t* codes, uint8_t* scales) {
  constexpr int RPW = 64 / LPR;
  const int lane = threadIdx.x & 63, l = lane % LPR;
  const int nch = (D + 127) / 128 * 16;   // chunks, whole runs of 16 lanes
  const int64_t cb = mx4_code_bytes(D), sb = mx4_scale_bytes(D);
  const int64_t first = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 6)) * RPW + lane / LPR;
  for (int64_t t = first; t < T; t += (int64_t)gridDim.x * 4 * RPW) {
    if (mask && !mask[t]) continue;
    for (int c = l; c < nch; c += LPR) {
      float v[8];
      load_chunk(x + t * D, c, D, v);
      mx4_store_chunk(v, c, D, codes + t * cb, scales + t * sb);
    }
  }
}

// Eight values per lane: what the codes stand for, rounded to the output's type (bf16 holds every one of
// them exactly, down to its subnormals; a value past the type's range is infinite).
template <typename TOut, int LPR>
__global__ __launch_bounds__(256) void dequantize_mx4_kernel(const uint8_t* codes, const uint8_t* scales, int64_t T,
                                                             int D, TOut* out) {
  constexpr int RPW = 64 / LPR;
  const int lane = threadIdx.x & 63, l = lane % LPR;
  const int nch = (D + 7) / 8;
  const int64_t cb = mx4_code_bytes(D), sb = mx4_scale_bytes(D);
  const int64_t first = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 6)) * RPW + lane / LPR;
  for (int64_t t = first; t < T; t += (int64_t)gridDim.x * 4 * RPW) {
    for (int c = l; c < nch; c += LPR) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(codes + t * cb + 4 * (int64_t)c);
      const uint32_t byte = scales[t * sb + (c >> 2)];
      float v[8];
      mx4_decode8(w, mx4_scale_value(byte), v);
      if (byte == 255u) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __builtin_nanf("");
      }
      store_chunk(out + t * D, c, D, v);
    }
  }
}

template <typename TIn>
static void launch_quantize_t(const void* x, const uint8_t* mask, int64_t T, int32_t D, uint8_t* codes,
                              uint8_t* scales, const DeviceInfo& dev, hipStream_t st) {
#define PG_QUANT(LPR)                                                                                              \
  hipLaunchKernelGGL((quantize_mx4_kernel<TIn, LPR>), dim3(resident_blocks(dev, T, 4 * (64 / LPR))), dim3(256), 0, st,     \
                     static_cast<const TIn*>(x), mask, T, D, codes, scales)
  if (D <= 128) PG_QUANT(16);
  else if (D <= 256) PG_QUANT(32);
  else PG_QUANT(64);
#undef PG_QUANT
}

hipError_t launch_quantize_mx4(const void* x, int32_t dtype, const uint8_t* mask, int64_t T, int32_t D,
                               uint8_t* codes, uint8_t* scales, const DeviceInfo& dev, hipStream_t st) {
  if (T == 0) return hipSuccess;
  if (dtype == 0) launch_quantize_t<uint16_t>(x, mask, T, D, codes, scales, dev, st);
  else launch_quantize_t<float>(x, mask, T, D, codes, scales, dev, st);
  return hipGetLastError();
}

template <typename TOut>
static void launch_dequantize_t(const uint8_t* codes, const uint8_t* scales, int64_t T, int32_t D, void* out,
                                const DeviceInfo& dev, hipStream_t st) {
#define PG_DEQUANT(LPR)                                                                                            \
  hipLaunchKernelGGL((dequantize_mx4_kernel<TOut, LPR>), dim3(resident_blocks(dev, T, 4 * (64 / LPR))), dim3(256), 0, st,  \
                     codes, scales, T, D, static_cast<TOut*>(out))
  if (D <= 128) PG_DEQUANT(16);
  else if (D <= 256) PG_DEQUANT(32);
  else PG_DEQUANT(64);
#undef PG_DEQUANT
}

hipError_t launch_dequantize_mx4(const uint8_t* codes, const uint8_t* scales, int64_t T, int32_t D, void* out,
                                 int32_t dtype, const DeviceInfo& dev, hipStream_t st) {
  if (T == 0) return hipSuccess;
  if (dtype == 0) launch_dequantize_t<uint16_t>(codes, scales, T, D, out, dev, st);
  else launch_dequantize_t<float>(codes, scales, T, D, out, dev, st);
  return hipGetLastError();
}

}  // namespace pg
