// Quantisation to the microscaled formats of mx.cuh, and back.
//
// Both are streams: a bf16 element is read once (2 bytes) and leaves as half a byte or a
// byte plus 1/32 byte of scale, so HBM bounds them.  Sixteen lanes take 128 columns of a
// row, eight consecutive values a lane: loads and code stores are contiguous across the
// lanes, a block's largest magnitude is two shuffles, and the four scale bytes of the
// group leave as one 32-bit word, the tile layout's unit.
#include <cuda_runtime.h>

#include "internal.h"
#include "mx.cuh"

namespace m3ssd {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;  // groups a half-warp has in flight

struct MxArgs {
  uint32_t rows, rows_pad, cols, nkb;  // nkb: 128-column groups
  uint32_t total;                      // rows_pad * nkb (quant) or rows * nkb (dequant)
  int64_t ldx;
  void* x;
  uint8_t* codes;
  uint8_t* scales;
};

template <int FMT, typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) mx_quant_kernel(MxArgs a) {
  const uint32_t lane = threadIdx.x & 31, sub = lane & 15;
  const uint32_t nhalf = gridDim.x * (kThreads / 16);
  const uint32_t wbase = (blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * 2;
  const int64_t Kp = (int64_t)a.nkb * 128;
  const T* const x = static_cast<const T*>(a.x);
  for (uint64_t i0 = wbase; i0 < a.total; i0 += (uint64_t)kUnroll * nhalf) {
    float v[kUnroll][8];
    uint32_t row[kUnroll], kb[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint64_t i = i0 + (uint64_t)u * nhalf + (lane >> 4);
      row[u] = i < a.total ? (uint32_t)i / a.nkb : 0xffffffffu;
      kb[u] = (uint32_t)i - row[u] * a.nkb;
      const uint32_t c = kb[u] * 128 + sub * 8;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[u][j] = 0.f;
      if (row[u] < a.rows && c < a.cols) {
        const T* p = x + (int64_t)row[u] * a.ldx + c;
        if (VEC && c + 8 <= a.cols)
          mx::load8(p, v[u]);
        else
          mx::load8_tail(p, (int)(a.cols - c), v[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      mx::quant_store8<FMT>(v[u], row[u], kb[u] * 16 + sub, Kp, a.codes, a.scales,
                            row[u] < a.rows, 0xffffffffu);
      if (row[u] >= a.rows && row[u] < a.rows_pad && sub == 0)  // the last tile's missing rows
        *reinterpret_cast<uint32_t*>(a.scales + mx::scale_word(row[u], kb[u], a.nkb)) = 0;
    }
  }
}

template <int FMT, typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) mx_dequant_kernel(MxArgs a) {
  const uint32_t lane = threadIdx.x & 31, sub = lane & 15;
  const uint32_t nhalf = gridDim.x * (kThreads / 16);
  const int64_t Kp = (int64_t)a.nkb * 128;
  T* const x = static_cast<T*>(a.x);
  const uint32_t hbase = (blockIdx.x * kThreads + threadIdx.x) >> 4;
  for (uint64_t i0 = hbase; i0 < a.total; i0 += (uint64_t)kUnroll * nhalf) {
    uint2 q[kUnroll];
    uint32_t byte[kUnroll], row[kUnroll], kb[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint64_t i = i0 + (uint64_t)u * nhalf;
      row[u] = i < a.total ? (uint32_t)i / a.nkb : 0xffffffffu;
      kb[u] = (uint32_t)i - row[u] * a.nkb;
      if (row[u] < a.rows) {
        const int64_t c = (int64_t)kb[u] * 16 + sub;
        if (FMT == mx::kFp4)
          q[u].x = *reinterpret_cast<const uint32_t*>(a.codes + (int64_t)row[u] * (Kp / 2) + c * 4);
        else
          q[u] = *reinterpret_cast<const uint2*>(a.codes + (int64_t)row[u] * Kp + c * 8);
        byte[u] = a.scales[mx::scale_word(row[u], kb[u], a.nkb) + (sub >> 2)];
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint32_t c = kb[u] * 128 + sub * 8;
      if (row[u] >= a.rows || c >= a.cols) continue;
      const float s = mx::scale_value(byte[u]);
      float v[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = FMT == mx::kFp4 ? mx::unpack2_e2m1((q[u].x >> (8 * j)) & 0xffu)
                                         : mx::unpack2_e4m3((j < 2 ? q[u].x : q[u].y) >> (16 * (j & 1)));
        v[2 * j] = f.x * s;
        v[2 * j + 1] = f.y * s;
      }
      T* p = x + (int64_t)row[u] * a.ldx + c;
      if (VEC && c + 8 <= a.cols)
        mx::store8(p, v);
      else
        mx::store8_tail(p, (int)(a.cols - c), v);
    }
  }
}

template <int FMT, typename T, bool VEC>
cudaError_t launch(const MxArgs& a, bool quant, cudaStream_t s) {
  const uint64_t per = (uint64_t)(kThreads / 16) * kUnroll;  // groups a CTA takes at a time
  const uint64_t want = (a.total + per - 1) / per, most = (uint64_t)current_device_sms() * 16;
  const unsigned grid = (unsigned)(want < most || most == 0 ? want : most);
  if (quant)
    mx_quant_kernel<FMT, T, VEC><<<grid, kThreads, 0, s>>>(a);
  else
    mx_dequant_kernel<FMT, T, VEC><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t dispatch(int fmt, bool bf16, const MxArgs& a, bool quant, cudaStream_t s) {
  // 16-byte accesses need every row to start on a 16-byte boundary
  const int64_t e = bf16 ? 2 : 4;
  const bool vec = (reinterpret_cast<uintptr_t>(a.x) % 16) == 0 && (a.ldx * e) % 16 == 0;
  if (a.total == 0) return cudaSuccess;
  if (fmt == mx::kFp4) {
    if (bf16)
      return vec ? launch<mx::kFp4, __nv_bfloat16, true>(a, quant, s)
                 : launch<mx::kFp4, __nv_bfloat16, false>(a, quant, s);
    return vec ? launch<mx::kFp4, float, true>(a, quant, s)
               : launch<mx::kFp4, float, false>(a, quant, s);
  }
  if (bf16)
    return vec ? launch<mx::kFp8, __nv_bfloat16, true>(a, quant, s)
               : launch<mx::kFp8, __nv_bfloat16, false>(a, quant, s);
  return vec ? launch<mx::kFp8, float, true>(a, quant, s)
             : launch<mx::kFp8, float, false>(a, quant, s);
}

}  // namespace

cudaError_t launch_mx_quant(int fmt, int64_t rows, int64_t cols, bool bf16, const void* x,
                            int64_t ldx, void* codes, void* scales, cudaStream_t s) {
  MxArgs a{};
  a.rows = (uint32_t)rows;
  a.rows_pad = (uint32_t)mx::pad128(rows);
  a.cols = (uint32_t)cols;
  a.nkb = (uint32_t)(mx::pad128(cols) / 128);
  a.total = a.rows_pad * a.nkb;
  a.ldx = ldx;
  a.x = const_cast<void*>(x);
  a.codes = static_cast<uint8_t*>(codes);
  a.scales = static_cast<uint8_t*>(scales);
  return dispatch(fmt, bf16, a, true, s);
}

cudaError_t launch_mx_dequant(int fmt, int64_t rows, int64_t cols, bool bf16, const void* codes,
                              const void* scales, void* x, int64_t ldx, cudaStream_t s) {
  MxArgs a{};
  a.rows = (uint32_t)rows;
  a.cols = (uint32_t)cols;
  a.nkb = (uint32_t)(mx::pad128(cols) / 128);
  a.total = a.rows * a.nkb;
  a.ldx = ldx;
  a.x = x;
  a.codes = static_cast<uint8_t*>(const_cast<void*>(codes));
  a.scales = static_cast<uint8_t*>(const_cast<void*>(scales));
  return dispatch(fmt, bf16, a, false, s);
}

}  // namespace m3ssd
