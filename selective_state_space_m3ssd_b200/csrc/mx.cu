// Quantisation to the microscaled formats of mx.cuh, and back.
//
// Both are streams: a bf16 element is read once (2 bytes) and leaves as half a byte or a
// byte plus 1/32 byte of scale, so HBM bounds them as long as the instructions a value
// takes stay few.  Eight lanes take 128 columns of a row, sixteen consecutive values a lane:
// a block's largest magnitude is one shuffle, the four scale bytes of the group leave as one
// 32-bit word, the tile layout's unit, and what a group costs (its place, scale and word)
// is shared by sixteen values.  Rows that do not allow 32-byte accesses pass through shared
// memory, element by element in the lanes' order on the global side.
// 32768 x 2048 bf16 to 4 bits and back on one B200: 60 us for both; HBM takes 3.9 TB/s of
// writes alone (a fill), 6.5 of a copy, so the two cannot take less than 26 and 34.  Eight
// values a lane, with a division a group and 16-byte loads, took 107.
#include <cuda_runtime.h>

#include "internal.h"
#include "mx.cuh"

namespace m3ssd {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kGroup = 8;   // lanes of a 128-column group
constexpr int kUnroll = 2;  // groups a lane has in flight

struct MxArgs {
  uint32_t rows, cols, nkb;  // nkb: 128-column groups a row
  uint32_t total;            // rows * nkb groups
  int64_t ldx;
  void* x;
  uint8_t* codes;
  uint8_t* scales;
};

// A lane's groups: i, i + step, ...; row and group within the row kept beside i (a
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

// Sixteen consecutive elements as loaded in 32-byte accesses (a group in flight holds them so)
// and as floats.
template <typename T>
struct Raw16;
template <>
struct Raw16<__nv_bfloat16> {
  float w[8];  // two bf16 a word
  __device__ void load(const __nv_bfloat16* p) { mx::load8(reinterpret_cast<const float*>(p), w); }
  __device__ void clear() {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = 0.f;
  }
  __device__ void get(float (&v)[16]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t u = __float_as_uint(w[j]);
      v[2 * j] = __uint_as_float(u << 16);
      v[2 * j + 1] = __uint_as_float(u & 0xffff0000u);
    }
  }
};
template <>
struct Raw16<float> {
  float a[8], b[8];
  __device__ void load(const float* p) {
    mx::load8(p, a);
    mx::load8(p + 8, b);
  }
  __device__ void clear() {
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] = b[j] = 0.f;
  }
  __device__ void get(float (&v)[16]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = a[j];
      v[8 + j] = b[j];
    }
  }
};
__device__ __forceinline__ void store16(__nv_bfloat16* p, const float (&v)[16]) {
  float w[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
    w[j] = __uint_as_float(*reinterpret_cast<uint32_t*>(&h));
  }
  mx::store8(reinterpret_cast<float*>(p), w);
}
__device__ __forceinline__ void store16(float* p, const float (&v)[16]) {
  float a[8], b[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    a[j] = v[j];
    b[j] = v[8 + j];
  }
  mx::store8(p, a);
  mx::store8(p + 8, b);
}
// The scale word of a group, counted in words.
__device__ __forceinline__ uint32_t word_index(uint32_t row, uint32_t kb, uint32_t nkb) {
  return (((row >> 7) * nkb + kb) << 7) + ((row & 31) << 2) + ((row >> 5) & 3);
}

// How a row is reached: kFull, 32-byte boundaries and columns a multiple of 128; kVec, columns
// a multiple of 16 (a lane's sixteen values are all there or all padding); kAny.
enum Access { kFull, kVec, kAny };

template <int FMT, typename T, int ACC>
__global__ void __launch_bounds__(kThreads) mx_quant_kernel(MxArgs a) {
  // kAny: a warp's four groups as elements; a lane reads its sixteen at a stride of 17, which
  // spreads over the banks
  __shared__ T stage[ACC == kAny ? kWarps : 1][ACC == kAny ? 32 * 17 : 1];
  const uint32_t lane = threadIdx.x & 31, sub = lane % kGroup, warp = threadIdx.x >> 5;
  const uint32_t step = gridDim.x * (kThreads / kGroup);
  Walk w((blockIdx.x * kThreads + threadIdx.x) / kGroup, step, a.nkb);
  const T* const x = static_cast<const T*>(a.x);
  // a warp goes round together (its shuffles): by its first group
  for (uint32_t base = w.i - lane / kGroup; base < a.total; base += kUnroll * step) {
    Raw16<T> raw[kUnroll];
    float any[ACC == kAny ? kUnroll : 1][16];
    uint32_t at[kUnroll];
    const uint32_t i0 = w.i;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if constexpr (ACC == kAny) {
        // group e / 128 of the warp's four, column e % 128, lane by lane
        T* const buf = stage[warp];
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const uint32_t src = 8 * (j / 4);  // a lane of the group, for its row and place
          const uint32_t row = __shfl_sync(0xffffffffu, w.row, src),
                         kb = __shfl_sync(0xffffffffu, w.kb, src);
          const uint32_t e = 32 * j + lane, col = kb * 128 + (e & 127);
          T val = from_f32<T>(0.f);
          if (row < a.rows && col < a.cols) val = x[(int64_t)row * a.ldx + col];
          buf[(e >> 4) * 17 + (e & 15)] = val;
        }
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 16; ++j) any[u][j] = to_f32(buf[lane * 17 + j]);
      } else {
        const uint32_t c = w.kb * 128 + sub * 16;
        if (w.i < a.total && (ACC == kFull || c < a.cols))
          raw[u].load(x + ((int64_t)w.row * a.ldx + c));
        else if (ACC == kVec)
          raw[u].clear();
      }
      at[u] = word_index(w.row, w.kb, a.nkb);
      w.next();
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint32_t i = i0 + u * step;
      float v[16];
      if constexpr (ACC == kAny) {
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = any[u][j];
      } else {
        raw[u].get(v);
      }
      uint4 c;
      const uint32_t word = mx::quant16<FMT>(v, c);
      if (i < a.total) {
        if (FMT == mx::kFp4)
          *reinterpret_cast<uint2*>(a.codes + (int64_t)i * 64 + sub * 8) = make_uint2(c.x, c.y);
        else
          *reinterpret_cast<uint4*>(a.codes + (int64_t)i * 128 + sub * 16) = c;
        if (sub == 0) reinterpret_cast<uint32_t*>(a.scales)[at[u]] = word;
      }
    }
  }
  // the words of the rows missing from the last tile are zero
  const uint32_t missing = (uint32_t)(mx::pad128(a.rows) - a.rows) * a.nkb;
  for (uint32_t i = blockIdx.x * kThreads + threadIdx.x; i < missing; i += gridDim.x * kThreads)
    reinterpret_cast<uint32_t*>(a.scales)[word_index(a.rows + i / a.nkb, i % a.nkb, a.nkb)] = 0u;
}

template <int FMT, typename T, int ACC>
__global__ void __launch_bounds__(kThreads) mx_dequant_kernel(MxArgs a) {
  __shared__ T stage[ACC == kAny ? kWarps : 1][ACC == kAny ? 32 * 17 : 1];
  const uint32_t lane = threadIdx.x & 31, sub = lane % kGroup, warp = threadIdx.x >> 5;
  const uint32_t step = gridDim.x * (kThreads / kGroup);
  Walk w((blockIdx.x * kThreads + threadIdx.x) / kGroup, step, a.nkb);
  T* const x = static_cast<T*>(a.x);
  for (uint32_t base = w.i - lane / kGroup; base < a.total; base += kUnroll * step) {
    uint4 q[kUnroll];
    uint32_t byte[kUnroll], row[kUnroll], kb[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      row[u] = w.i < a.total ? w.row : 0xffffffffu;
      kb[u] = w.kb;
      q[u] = make_uint4(0u, 0u, 0u, 0u);
      byte[u] = 0;
      if (w.i < a.total) {
        if (FMT == mx::kFp4) {
          const uint2 c =
              *reinterpret_cast<const uint2*>(a.codes + (int64_t)w.i * 64 + sub * 8);
          q[u].x = c.x;
          q[u].y = c.y;
        } else {
          q[u] = *reinterpret_cast<const uint4*>(a.codes + (int64_t)w.i * 128 + sub * 16);
        }
        byte[u] = a.scales[(int64_t)word_index(w.row, w.kb, a.nkb) * 4 + (sub >> 1)];
      }
      w.next();
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const float s = mx::scale_value(byte[u]);
      const uint32_t c4[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
      float v[16];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 f = FMT == mx::kFp4 ? mx::unpack2_e2m1((c4[j >> 2] >> (8 * (j & 3))) & 0xffu)
                                         : mx::unpack2_e4m3(c4[j >> 1] >> (16 * (j & 1)));
        v[2 * j] = f.x * s;
        v[2 * j + 1] = f.y * s;
      }
      if constexpr (ACC == kAny) {
        T* const buf = stage[warp];
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 16; ++j) buf[lane * 17 + j] = from_f32<T>(v[j]);
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const uint32_t src = 8 * (j / 4);
          const uint32_t r = __shfl_sync(0xffffffffu, row[u], src),
                         k = __shfl_sync(0xffffffffu, kb[u], src);
          const uint32_t e = 32 * j + lane, col = k * 128 + (e & 127);
          if (r < a.rows && col < a.cols) x[(int64_t)r * a.ldx + col] = buf[(e >> 4) * 17 + (e & 15)];
        }
      } else {
        const uint32_t c = kb[u] * 128 + sub * 16;
        if (row[u] < a.rows && (ACC == kFull || c < a.cols))
          store16(x + ((int64_t)row[u] * a.ldx + c), v);
      }
    }
  }
}

template <int FMT, typename T, int ACC>
cudaError_t launch(const MxArgs& a, bool quant, cudaStream_t s) {
  const uint64_t per = (uint64_t)(kThreads / kGroup) * kUnroll;  // groups a CTA takes at a time
  const uint64_t want = (a.total + per - 1) / per, most = (uint64_t)current_device_sms() * 16;
  const unsigned grid = (unsigned)(want < most || most == 0 ? want : most);
  if (quant)
    mx_quant_kernel<FMT, T, ACC><<<grid, kThreads, 0, s>>>(a);
  else
    mx_dequant_kernel<FMT, T, ACC><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

template <int FMT, typename T>
cudaError_t by_access(const MxArgs& a, bool quant, cudaStream_t s) {
  const bool vec = reinterpret_cast<uintptr_t>(a.x) % 32 == 0 && a.cols % 16 == 0 &&
                   a.ldx * (int64_t)sizeof(T) % 32 == 0;
  return !vec               ? launch<FMT, T, kAny>(a, quant, s)
         : a.cols % 128 != 0 ? launch<FMT, T, kVec>(a, quant, s)
                             : launch<FMT, T, kFull>(a, quant, s);
}

cudaError_t dispatch(int fmt, bool bf16, const MxArgs& a, bool quant, cudaStream_t s) {
  if (a.rows == 0) return cudaSuccess;
  if (fmt == mx::kFp4)
    return bf16 ? by_access<mx::kFp4, __nv_bfloat16>(a, quant, s)
                : by_access<mx::kFp4, float>(a, quant, s);
  return bf16 ? by_access<mx::kFp8, __nv_bfloat16>(a, quant, s)
              : by_access<mx::kFp8, float>(a, quant, s);
}

}  // namespace

cudaError_t launch_mx_quant(int fmt, int64_t rows, int64_t cols, bool bf16, const void* x,
                            int64_t ldx, void* codes, void* scales, cudaStream_t s) {
  MxArgs a{};
  a.rows = (uint32_t)rows;
  a.cols = (uint32_t)cols;
  a.nkb = (uint32_t)(mx::pad128(cols) / 128);
  a.total = a.rows * a.nkb;
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
