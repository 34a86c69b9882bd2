// Microscaled (MX) formats: the arithmetic shared by the quantising kernels and
// the epilogues that quantise.
//
// A block is 32 consecutive elements of a row with one shared power of two
// 2^p, held as the byte p + 127 (UE8M0: 0..254; 255 marks a block that held a
// NaN or an infinity).  Elements are E4M3 (MXFP8, largest 448 = 1.75 * 2^8) or
// E2M1 (MXFP4, largest 6 = 1.5 * 2^2).  p is the smallest integer with
// max|v| <= largest * 2^p, so no element saturates: the rule that cuts p to
// floor(log2 max|v|) - 8 (- 2) clips up to 1/8 (1/4) off a block's largest
// element, more than the rounding to the grid costs.  Elements are rounded
// once, to nearest, ties to the even code; v * 2^-p is exact in fp32 wherever
// its code is not 0.
//
// Storage: codes row-major, one byte per E4M3 element, two E2M1 elements per
// byte (the even element in the low nibble); scales as 32-bit words of four
// consecutive blocks (128 elements), [ceil(K/128)][rows] words per matrix, so
// that the words that one K step of a 128-row operand tile needs lie next to
// one another whatever row the tile starts at.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"

namespace rmoe {

constexpr int MX_BLOCK = 32;

template <int FMT>
struct MxFmt;
template <>
struct MxFmt<MOE_MXFP8> {
  static constexpr uint32_t kTopMantissa32 = 0x600000;  // 1.75
  static constexpr int kTopExponent = 8;
  static constexpr int kPerByte = 1;
};
template <>
struct MxFmt<MOE_MXFP4> {
  static constexpr uint32_t kTopMantissa32 = 0x400000;  // 1.5
  static constexpr int kTopExponent = 2;
  static constexpr int kPerByte = 2;
};

// The scale byte of a block from the bits of its largest |v| as fp32.  A
// mantissa above the largest element's carries into the exponent field.
template <int FMT>
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return 255u;
  const int e = (int)((amax_bits + (0x7fffffu - MxFmt<FMT>::kTopMantissa32)) >> 23) -
                MxFmt<FMT>::kTopExponent;
  return (uint32_t)max(e, 0);
}

// 2^-p of a scale byte below 255 (mx_encode gives a NaN block zero codes without it).
__device__ __forceinline__ float mx_inverse_scale(uint32_t byte) {
  return __uint_as_float((254u - min(byte, 254u)) << 23);
}

// The value of a scale byte.
__device__ __forceinline__ float mx_scale_value(uint32_t byte) {
  if (byte == 255u) return __uint_as_float(0x7fffffffu);
  return byte == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(byte << 23);
}

// Four E4M3 codes (lowest element in the lowest byte) of values within +-448.
__device__ __forceinline__ uint32_t mx_pack_e4m3(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// Eight E2M1 codes (lowest element in the lowest nibble) of values within +-6.
__device__ __forceinline__ uint32_t mx_pack_e2m1(const float* v) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// Two E2M1 codes in a byte (lo in the low nibble) of values within +-6.
__device__ __forceinline__ uint8_t mx_pack_e2m1_pair(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0;\n\t.reg .b16 l;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "mov.b16 l, {b0, b0};\n\tcvt.u32.u16 %0, l;\n\t}"
      : "=r"(r)
      : "f"(lo), "f"(hi));
  return static_cast<uint8_t>(r);
}

// Codes of N consecutive elements (N a multiple of 8) of one block whose scale
// byte is given; out holds N / 4 (MXFP8) or N / 8 (MXFP4) words.
template <int FMT, int N>
__device__ __forceinline__ void mx_encode(const float (&v)[N], uint32_t byte, uint32_t* out) {
  if (byte == 255u) {
#pragma unroll
    for (int i = 0; i < N / (4 * MxFmt<FMT>::kPerByte); ++i) out[i] = 0;
    return;
  }
  const float inv = mx_inverse_scale(byte);
  float s[N];
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = v[i] * inv;
  if constexpr (FMT == MOE_MXFP8) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
      out[i] = mx_pack_e4m3(s[4 * i], s[4 * i + 1], s[4 * i + 2], s[4 * i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < N / 8; ++i) out[i] = mx_pack_e2m1(s + 8 * i);
  }
}

// Two elements as floats from two E4M3 codes / one byte of two E2M1 codes.
__device__ __forceinline__ float2 mx_unpack_e4m3(uint32_t two) {
  uint32_t h;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}"
      : "=r"(h)
      : "r"(two));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}

__device__ __forceinline__ float2 mx_unpack_e2m1(uint32_t two) {
  uint32_t h;
  asm("{\n\t.reg .b8 t, u, v, w;\n\tmov.b32 {t, u, v, w}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t;\n\t}"
      : "=r"(h)
      : "r"(two));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}

}  // namespace rmoe
