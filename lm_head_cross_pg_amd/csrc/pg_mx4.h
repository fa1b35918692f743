// The microscaled 4-bit format of the quantised head, and its conversions (internal header).
//
// A row of D values is held as blocks of 32 consecutive ones. A block has a scale 2^e, stored as the
// byte e + 127 (0 .. 254; 255 marks a block of NaNs), and each value a 4-bit code: a sign bit and the
// index of one of 0, 0.5, 1, 1.5, 2, 3, 4, 6. Two codes share a byte, the value of even index in the
// low half. A row's codes are padded with zeros to whole 64-value steps of the matrix instruction (32
// bytes) and its scale bytes to 16, so that every row starts on 16 bytes.
#pragma once
#include "pg_common.h"
#include "pg_rows.h"

namespace pg {

constexpr int kMx4Block = 32;   // values that share a scale
constexpr int kMx4Step = 64;    // values of one step of the scaled 32 x 32 x 64 MFMA

__host__ __device__ inline int64_t mx4_code_bytes(int32_t D) { return 32 * (((int64_t)D + 63) / 64); }
__host__ __device__ inline int64_t mx4_scale_bytes(int32_t D) { return 16 * (((int64_t)D + 511) / 512); }

// The scale byte of a block from the largest magnitude's bits (as unsigned numbers, magnitudes
// order like their bits, infinities and NaN above all): the e with max |x| in [3.5, 7) 2^e. Values
// up to 7 2^e round to 6 2^e at most half a step away (the last step is 2), so that no value is
// clipped by more than rounding would move it; the smallest e with that property is also better than
// the one that keeps max |x| in [4, 8) 2^e (relative error of normal values 11.2 % against 11.5 %, of
// Laplace ones 12.4 % against 12.7 %) and than [3, 6) (11.5 %, 13.2 %). Adding 0.25 of the mantissa's
// unit carries mantissas from 1.75 on into the exponent. Byte 252 is the last one: 6 2^125 is the format's
// largest value that float32 and bf16 hold.
__device__ __forceinline__ uint32_t mx4_scale_byte(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return 255u;
  const int b = (int)((amax_bits + 0x00200000u) >> 23) - 2;
  return b < 0 ? 0u : (b > 252 ? 252u : (uint32_t)b);
}

// 2^(byte - 127) as a float: byte 0 is a subnormal, 255 NaN.
__device__ __forceinline__ float mx4_scale_value(uint32_t byte) {
  const uint32_t u = byte == 0u ? 0x00400000u : (byte == 255u ? 0x7fc00000u : byte << 23);
  return __uint_as_float(u);
}

// Eight values as codes (lowest index in the lowest bits): the hardware's conversion divides by the
// scale exactly and rounds to the nearest code, ties to the even one, magnitudes above 6 to 6 (checked
// value by value against the definition over all bf16 bit patterns and scales across the range).
__device__ __forceinline__ uint32_t mx4_encode8(const float* v, float scale) {
  uint32_t o = 0;
  o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, v[0], v[1], scale, 0);
  o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, v[2], v[3], scale, 1);
  o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, v[4], v[5], scale, 2);
  o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, v[6], v[7], scale, 3);
  return o;
}

// What eight codes stand for, exactly (checked for every code at every scale byte but NaN's).
__device__ __forceinline__ void mx4_decode8(uint32_t w, float scale, float* v) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 1);
  const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 3);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    v[j] = a[j];
    v[2 + j] = b[j];
    v[4 + j] = c[j];
    v[6 + j] = d[j];
  }
}

// Lane c of a row's lanes holds chunk c (values 8 c .. 8 c + 7, zeros past D) in v: the four lanes of
// a block agree on its scale, each stores its four bytes of codes, and the first of 16 the four scale
// bytes of its blocks as one word (after the row's last, the zeros up to the padded end). Every lane of
// a run of 16 takes part; chunks past the row's padded end store nothing.
__device__ __forceinline__ void mx4_store_chunk(const float* v, int c, int D, uint8_t* codes, uint8_t* scales) {
  uint32_t a = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t b = __float_as_uint(v[j]) & 0x7fffffffu;
    a = b > a ? b : a;
  }
  uint32_t o = dpp<0xB1>(a);   // quad_perm 1, 0, 3, 2
  a = o > a ? o : a;
  o = dpp<0x4E>(a);            // quad_perm 2, 3, 0, 1
  a = o > a ? o : a;
  const uint32_t s = 8 * c < D ? mx4_scale_byte(a) : 0u;
  const uint32_t code = s == 255u ? 0u : mx4_encode8(v, mx4_scale_value(s));
  // the scales of blocks b, b + 1 in lane 4 b, then of b .. b + 3 (the lanes 4 and 8 further in the run)
  uint32_t w = s | dpp<0x104>(s) << 8;
  w |= dpp<0x108>(w) << 16;
  const int nch = (D + 7) >> 3;
  if (c < 8 * ((D + 63) >> 6)) *reinterpret_cast<uint32_t*>(codes + 4 * (int64_t)c) = code;
  if ((c & 15) == 0 && c < nch) {
    uint32_t* p = reinterpret_cast<uint32_t*>(scales + (c >> 2));
    p[0] = w;
    if (c + 16 >= nch)
      for (int k = 1; ((c >> 4) + k) & 3; ++k) p[k] = 0u;
  }
}

}  // namespace pg
