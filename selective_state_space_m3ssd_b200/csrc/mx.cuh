// Microscaled (MX) formats: blocks of 32 values along a row, each with a power-of-two
// scale 2^E (byte E + 127), and E2M1 (4-bit) or E4M3 (8-bit) codes.
//
// E is the least exponent with amax <= maxval 2^E (maxval = 6 = 1.5 2^2 or
// 448 = 1.75 2^8), so no value saturates; it is read off the bits of amax = m 2^e:
// E = e - 2 (- 8), plus one when m exceeds 1.5 (1.75).  Code = value 2^-E rounded to
// nearest even; the product with a power of two is exact, so a block has one result.  A
// block that holds a NaN or an infinity takes the scale NaN (byte 255) and zero codes.
//
// Storage of a (rows x cols) tensor: rows of Kp codes, Kp = cols rounded up to 128, the
// padding zero (E2M1: two codes a byte, the even index in the low half).  Scales in tiles
// of 128 rows x 4 blocks (512 bytes), the layout the block-scaled products read: byte
// (r % 32) 16 + (r / 32) 4 + k of row r and block k of the tile; tiles in row-block-major
// order; missing rows and blocks have byte 0.
#pragma once

#include <stdint.h>

#include "common.cuh"

namespace m3ssd {
namespace mx {

constexpr int kFp4 = 0, kFp8 = 1;

__host__ __device__ __forceinline__ int64_t pad128(int64_t n) { return (n + 127) & ~int64_t(127); }

// Byte offset of the 32-bit word with the four scales of row r and 128-column group kb.
__device__ __forceinline__ int64_t scale_word(int64_t r, int64_t kb, int64_t nkb) {
  const uint32_t i = (uint32_t)r & 127u;
  return ((r >> 7) * nkb + kb) * 512 + (i & 31u) * 16 + (i >> 5) * 4;
}

// The scale byte for a block whose largest magnitude has these bits: adding what is missing
// from maxval's mantissa to 2 carries into the exponent exactly when m exceeds it.
template <int FMT>
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
  constexpr uint32_t up = FMT == kFp4 ? 0x3fffffu : 0x1fffffu;
  const int e = (int)((amax_bits + up) >> 23) - (FMT == kFp4 ? 2 : 8);  // biased E
  return amax_bits >= 0x7f800000u ? 255u : (uint32_t)max(e, 0);  // 255: NaN or infinity
}
// 2^-E as a float, E = byte - 127, for the bytes scale_byte gives a finite block (at most 253).
__device__ __forceinline__ float inv_scale(uint32_t byte) {
  return __uint_as_float((254u - byte) << 23);
}
// 2^E as a float (byte 0 is the subnormal 2^-127, byte 255 NaN).
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return byte == 0u ? __uint_as_float(0x00400000u)
                    : __uint_as_float(byte == 255u ? 0x7fffffffu : byte << 23);
}

// Eight values to codes, rounded to nearest even: E2M1 packed into 32 bits.
__device__ __forceinline__ uint32_t pack_e2m1(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}\n"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}
// Two values to E4M3 codes, the first in the low byte.
__device__ __forceinline__ uint32_t pack2_e4m3(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ uint32_t pack4_e4m3(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}\n"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
__device__ __forceinline__ float2 half2_bits_to_float2(uint32_t h) {
  float2 f;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\t"
      "cvt.f32.f16 %1, hi;\n\t}\n"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}
// Two E4M3 codes (16 bits) to floats; every E4M3 value is exact in fp16.
__device__ __forceinline__ float2 unpack2_e4m3(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
  return half2_bits_to_float2(h);
}
// Two E2M1 codes (one byte) to floats.
__device__ __forceinline__ float2 unpack2_e2m1(uint32_t codes) {
  uint32_t h;
  asm("{\n\t.reg .b8 b, z0, z1, z2;\n\tmov.b32 {b, z0, z1, z2}, %1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b;\n\t}\n"
      : "=r"(h)
      : "r"(codes));
  return half2_bits_to_float2(h);
}

// The largest magnitude of a, b and c; NaN when one of them is.
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float amax8(const float (&v)[8]) {
  const float m = max3_abs(v[0], v[1], v[2]);
  return max3_abs(max3_abs(m, v[3], v[4]), max3_abs(v[5], v[6], v[7]), 0.f);
}

// A lane's eight of the values of a 128-column group (sixteen lanes; four lanes to a block of
// 32) to codes; returns the group's scale word, in every lane.  Warps call it together.
template <int FMT>
__device__ __forceinline__ uint32_t quant8(const float (&v)[8], uint2& codes) {
  float m = amax8(v);
  m = max3_abs(m, __shfl_xor_sync(0xffffffffu, m, 1), 0.f);
  m = max3_abs(m, __shfl_xor_sync(0xffffffffu, m, 2), 0.f);
  const uint32_t byte = scale_byte<FMT>(__float_as_uint(m));
  const float inv = inv_scale(byte);
  float q[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) q[j] = v[j] * inv;
  if (FMT == kFp4) {
    codes = make_uint2(pack_e2m1(q), 0u);
  } else {
    codes = make_uint2(pack4_e4m3(q[0], q[1], q[2], q[3]), pack4_e4m3(q[4], q[5], q[6], q[7]));
  }
  if (byte == 255u) codes = make_uint2(0u, 0u);
  uint32_t w = byte << (8 * ((threadIdx.x >> 2) & 3));  // the four blocks' bytes
  w |= __shfl_xor_sync(0xffffffffu, w, 4);
  w |= __shfl_xor_sync(0xffffffffu, w, 8);
  return w;
}
// The same with sixteen values a lane: eight lanes to a group, two to a block.
template <int FMT>
__device__ __forceinline__ uint32_t quant16(const float (&v)[16], uint4& codes) {
  float m = max3_abs(v[0], v[1], v[2]);
#pragma unroll
  for (int j = 3; j < 15; j += 2) m = max3_abs(m, v[j], v[j + 1]);
  m = max3_abs(m, v[15], __shfl_xor_sync(0xffffffffu, max3_abs(m, v[15], 0.f), 1));
  const uint32_t byte = scale_byte<FMT>(__float_as_uint(m));
  const float inv = inv_scale(byte);
  float q[2][8];
#pragma unroll
  for (int j = 0; j < 16; ++j) q[j >> 3][j & 7] = v[j] * inv;
  if (FMT == kFp4) {
    codes = make_uint4(pack_e2m1(q[0]), pack_e2m1(q[1]), 0u, 0u);
  } else {
    codes = make_uint4(pack4_e4m3(q[0][0], q[0][1], q[0][2], q[0][3]),
                       pack4_e4m3(q[0][4], q[0][5], q[0][6], q[0][7]),
                       pack4_e4m3(q[1][0], q[1][1], q[1][2], q[1][3]),
                       pack4_e4m3(q[1][4], q[1][5], q[1][6], q[1][7]));
  }
  if (byte == 255u) codes = make_uint4(0u, 0u, 0u, 0u);
  uint32_t w = byte << (8 * ((threadIdx.x >> 1) & 3));
  w |= __shfl_xor_sync(0xffffffffu, w, 2);
  w |= __shfl_xor_sync(0xffffffffu, w, 4);
  return w;
}
// Stores a lane's codes of 128-column group i (counted over the rows' groups).
template <int FMT>
__device__ __forceinline__ void store_codes(uint8_t* codes, int64_t i, uint32_t sub, uint2 c) {
  if (FMT == kFp4)
    *reinterpret_cast<uint32_t*>(codes + i * 64 + sub * 4) = c.x;
  else
    *reinterpret_cast<uint2*>(codes + i * 128 + sub * 8) = c;
}

// Eight elements from global memory as floats in one access (16 bytes of bf16, 32 of fp32,
// aligned to that), or one by one up to `n` valid ones (the rest zero).
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 w = *reinterpret_cast<const uint4*>(p);
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(u[j] << 16);
    v[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]),
                 "=f"(v[6]), "=f"(v[7])
               : "l"(p)
               : "memory");
}
template <typename T>
__device__ __forceinline__ void load8_tail(const T* p, int n, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = j < n ? to_f32(p[j]) : 0.f;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
    u[j] = *reinterpret_cast<uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  asm volatile("st.global.v8.f32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"f"(v[0]), "f"(v[1]),
               "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "l"(p)
               : "memory");
}
// Whether rows of `ld` elements starting at p allow those accesses.
template <typename T>
__host__ __device__ __forceinline__ bool aligned8(const void* p, int64_t ld) {
  return reinterpret_cast<uintptr_t>(p) % (8 * sizeof(T)) == 0 && ld % 8 == 0;
}
template <typename T>
__device__ __forceinline__ void store8_tail(T* p, int n, const float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < n) p[j] = from_f32<T>(v[j]);
}

}  // namespace mx
}  // namespace m3ssd
