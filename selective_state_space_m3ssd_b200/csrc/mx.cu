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
  uint32_t rows, cols, nkb;  // nkb: 128-column groups a row
  uint32_t total;            // groups: rows (quant: rounded up to 128) * nkb
  int64_t ldx;
  void* x;
  uint8_t* codes;
  uint8_t* scales;
};

// A half-warp's groups: i, i + step, ...; row and group within the row kept beside i (a
// division a group would cost as much as its conversion).
struct Walk {
  uint32_t i, row, kb, nkb, drow, dkb, step;
  __device__ Walk(uint32_t first, uint32_t step, uint32_t nkb) : i(first), nkb(nkb), step(step) {
    row = i / nkb;
    kb = i - row * nkb;
    drow = step / nkb;
    dkb = step - drow * nkb;
  }
  __device__ void next() {  // i stays below 2^32: at most 2^31 groups and a step below 2^31
    i += step;
    row += drow;
    kb += dkb;
    if (kb >= nkb) {
      kb -= nkb;
      ++row;
    }
  }
};

template <int FMT, typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) mx_quant_kernel(MxArgs a) {
  const uint32_t sub = threadIdx.x & 15, nhalf = gridDim.x * (kThreads / 16);
  Walk w((blockIdx.x * kThreads + threadIdx.x) >> 4, nhalf, a.nkb);
  const T* const x = static_cast<const T*>(a.x) + 8 * sub;
  // the two halves of a warp go round together (quant8's shuffles): i - its half's place
  for (uint32_t base = w.i & ~1u; base < a.total; base += kUnroll * nhalf) {
    float v[kUnroll][8];
    uint32_t at[kUnroll];  // byte offset of the scale word, in words
    bool live[kUnroll];
    const uint32_t i0 = w.i;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint32_t c = w.kb * 128 + sub * 8;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[u][j] = 0.f;
      live[u] = w.row < a.rows;
      if (live[u] && c < a.cols) {
        const T* p = x + ((int64_t)w.row * a.ldx + w.kb * 128);
        if (VEC && c + 8 <= a.cols)
          mx::load8(p, v[u]);
        else
          mx::load8_tail(p, (int)(a.cols - c), v[u]);
      }
      at[u] = (((w.row >> 7) * a.nkb + w.kb) << 7) + ((w.row & 31) << 2) + ((w.row >> 5) & 3);
      w.next();
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint32_t i = i0 + u * nhalf;
      uint2 c;
      const uint32_t word = mx::quant8<FMT>(v[u], c);
      if (live[u]) mx::store_codes<FMT>(a.codes, i, sub, c);
      // rows missing from the last tile have zeros
      if (sub == 0 && i < a.total)
        reinterpret_cast<uint32_t*>(a.scales)[at[u]] = live[u] ? word : 0u;
    }
  }
}

template <int FMT, typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) mx_dequant_kernel(MxArgs a) {
  const uint32_t sub = threadIdx.x & 15, nhalf = gridDim.x * (kThreads / 16);
  Walk w((blockIdx.x * kThreads + threadIdx.x) >> 4, nhalf, a.nkb);
  T* const x = static_cast<T*>(a.x) + 8 * sub;
  while (w.i < a.total) {
    uint2 q[kUnroll];
    uint32_t byte[kUnroll], col[kUnroll];
    T* out[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      col[u] = 0xffffffffu;
      const uint32_t c = w.kb * 128 + sub * 8;
      if (w.i < a.total && c < a.cols) {
        col[u] = c;
        out[u] = x + ((int64_t)w.row * a.ldx + w.kb * 128);
        if (FMT == mx::kFp4)
          q[u].x = *reinterpret_cast<const uint32_t*>(a.codes + (int64_t)w.i * 64 + sub * 4);
        else
          q[u] = *reinterpret_cast<const uint2*>(a.codes + (int64_t)w.i * 128 + sub * 8);
        const uint32_t at =
            (((w.row >> 7) * a.nkb + w.kb) << 7) + ((w.row & 31) << 2) + ((w.row >> 5) & 3);
        byte[u] = a.scales[(int64_t)at * 4 + (sub >> 2)];
      }
      w.next();
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (col[u] == 0xffffffffu) continue;
      const float s = mx::scale_value(byte[u]);
      float v[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = FMT == mx::kFp4 ? mx::unpack2_e2m1((q[u].x >> (8 * j)) & 0xffu)
                                         : mx::unpack2_e4m3((j < 2 ? q[u].x : q[u].y) >> (16 * (j & 1)));
        v[2 * j] = f.x * s;
        v[2 * j + 1] = f.y * s;
      }
      if (VEC && col[u] + 8 <= a.cols)
        mx::store8(out[u], v);
      else
        mx::store8_tail(out[u], (int)(a.cols - col[u]), v);
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
  const bool vec = bf16 ? mx::aligned8<__nv_bfloat16>(a.x, a.ldx) : mx::aligned8<float>(a.x, a.ldx);
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
  a.cols = (uint32_t)cols;
  a.nkb = (uint32_t)(mx::pad128(cols) / 128);
  a.total = (uint32_t)mx::pad128(rows) * a.nkb;
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
