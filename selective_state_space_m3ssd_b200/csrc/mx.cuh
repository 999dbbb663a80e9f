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

// The scale byte for a block whose largest magnitude has these bits.
template <int FMT>
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return 255u;  // NaN or infinity
  const int e = (int)(amax_bits >> 23) - (FMT == kFp4 ? 2 : 8);  // biased E
  const uint32_t m = amax_bits & 0x007fffffu;
  return (uint32_t)max(e + (m > (FMT == kFp4 ? 0x400000u : 0x600000u) ? 1 : 0), 0);
}
// 2^-E as a float, E = byte - 127 (byte 255: 0, which makes every finite code 0).
__device__ __forceinline__ float inv_scale(uint32_t byte) {
  // biased exponent of 2^-E: 254 - byte; byte 254 (2^-127) is subnormal
  return byte < 254u ? __uint_as_float((254u - byte) << 23)
                     : __uint_as_float(byte == 254u ? 0x00400000u : 0u);
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

// The largest magnitude's bits of eight values (integer order: NaN > infinity > finite).
__device__ __forceinline__ uint32_t amax_bits8(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
  return m;
}

// Quantises a lane's eight values (columns 8 c .. 8 c + 7 of row r, four lanes to a block
// of 32, sixteen to a scale word; every lane of a 16-lane group is in the same row and
// takes part) and stores the codes; the group's first lane stores the scale word.
template <int FMT>
__device__ __forceinline__ void quant_store8(const float (&v)[8], int64_t r, int64_t c, int64_t Kp,
                                             uint8_t* __restrict__ codes,
                                             uint8_t* __restrict__ scales, bool active,
                                             uint32_t mask) {
  uint32_t m = amax_bits8(v);
  m = max(m, __shfl_xor_sync(mask, m, 1));
  m = max(m, __shfl_xor_sync(mask, m, 2));
  const uint32_t byte = scale_byte<FMT>(m);
  const float inv = inv_scale(byte);
  float q[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) q[j] = byte == 255u ? 0.f : v[j] * inv;
  // the four blocks' bytes into one word
  uint32_t w = byte << (8 * ((threadIdx.x >> 2) & 3));
  w |= __shfl_xor_sync(mask, w, 4);
  w |= __shfl_xor_sync(mask, w, 8);
  if (!active) return;
  if (FMT == kFp4) {
    *reinterpret_cast<uint32_t*>(codes + r * (Kp / 2) + c * 4) = pack_e2m1(q);
  } else {
    *reinterpret_cast<uint2*>(codes + r * Kp + c * 8) = make_uint2(
        pack4_e4m3(q[0], q[1], q[2], q[3]), pack4_e4m3(q[4], q[5], q[6], q[7]));
  }
  if ((threadIdx.x & 15) == 0)
    *reinterpret_cast<uint32_t*>(scales + scale_word(r, c >> 4, Kp >> 7)) = w;
}

// Eight elements from global memory as floats: 16-byte loads, or one by one up to `n`
// valid ones (the rest zero).
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
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
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
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
template <typename T>
__device__ __forceinline__ void store8_tail(T* p, int n, const float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < n) p[j] = from_f32<T>(v[j]);
}

}  // namespace mx
}  // namespace m3ssd
