// Quantisation to the microscaled formats of mx.cuh, and back.
//
// Both are streams: a bf16 element is read once (2 bytes) and leaves as half a byte or a
// byte plus 1/32 byte of scale, so HBM bounds them as long as the instructions a value
// takes stay few.  Eight lanes take 128 columns of a row, sixteen consecutive values a lane:
// a block's largest magnitude is one shuffle, the four scale bytes of the group leave as one
// 32-bit word, the tile layout's unit, and what a group costs (its place, scale and word)
// is shared by sixteen values.  Rows that do not allow 32-byte accesses pass through shared
// memory, 32 consecutive elements an access on the global side, 16 bytes a lane on the other.
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
  __device__ float& word(int j) { return w[j]; }
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
  __device__ void put(const float (&v)[16]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
      w[j] = __uint_as_float(*reinterpret_cast<uint32_t*>(&h));
    }
  }
  __device__ void store(__nv_bfloat16* p) const {
    mx::store8(reinterpret_cast<float*>(p), w);
  }
};
template <>
struct Raw16<float> {
  float a[8], b[8];
  __device__ float& word(int j) { return j < 8 ? a[j] : b[j - 8]; }
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
  __device__ void put(const float (&v)[16]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      a[j] = v[j];
      b[j] = v[8 + j];
    }
  }
  __device__ void store(float* p) const {
    mx::store8(p, a);
    mx::store8(p + 8, b);
  }
};
// The scale word of a group, counted in words.
__device__ __forceinline__ uint32_t word_index(uint32_t row, uint32_t kb, uint32_t nkb) {
  return (((row >> 7) * nkb + kb) << 7) + ((row & 31) << 2) + ((row >> 5) & 3);
}

// How a row is reached: kFull, 32-byte boundaries and columns a multiple of 128; kVec, columns
// a multiple of 16 (a lane's sixteen values are all there or all padding); kAny.
enum Access { kFull, kVec, kAny };

// Groups a lane has in flight, and the CTAs an SM is to hold.  Element by element a lane's loads
// are many already and more CTAs serve better: 5300 x 6314 to 4 bits and back 31.9 and 28.0 us
// from fp32 (six CTAs), 26.7 and 20.9 from bf16 (five), against 44.2, 28.5, 31.3 and 21.9 with two
// groups a lane and what registers allow (three or four CTAs); over five tensors in turn, which
// L2 does not hold, 32.8, 28.7, 30.7 and 24.2.
template <int ACC>
constexpr int kUnrollOf = ACC == kAny ? 1 : 2;
template <typename T, int ACC>
constexpr int kCtasOf = ACC != kAny ? 1 : sizeof(T) == 4 ? 6 : 5;

// kAny: a warp's four groups of 128 elements in shared memory.  Element e is lane e / 16's, as
// units of 16 bytes whose order goes round with the lane, so that neither the accesses of 32
// consecutive elements nor the lanes' 16-byte accesses meet in a bank.
template <typename T>
struct Stage {
  static constexpr uint32_t kUnit = 16 / sizeof(T), kUnits = 16 / kUnit;
  T v[512];
  static __device__ __forceinline__ uint32_t turn(uint32_t lane) {
    return kUnits == 4 ? (lane >> 1) & 3 : (lane >> 2) & 1;
  }
  __device__ __forceinline__ T& at(uint32_t e) {
    const uint32_t b = e >> 4;
    return v[b * 16 + ((e / kUnit % kUnits) ^ turn(b)) * kUnit + e % kUnit];
  }
  __device__ __forceinline__ float4& unit(uint32_t lane, uint32_t u) {
    return *reinterpret_cast<float4*>(v + lane * 16 + (u ^ turn(lane)) * kUnit);
  }
};
// Group g's row (null where there is none) and the columns it has from the group's first on;
// row and kb are those of each lane's group.
template <typename T>
__device__ __forceinline__ T* group_row(T* x, int64_t ldx, uint32_t cols, uint32_t rows, int g,
                                        uint32_t row, uint32_t kb, uint32_t& have) {
  const uint32_t r = __shfl_sync(0xffffffffu, row, kGroup * g);
  const uint32_t c = __shfl_sync(0xffffffffu, kb, kGroup * g) * 128;
  have = r < rows ? cols - c : 0;
  return x + ((int64_t)r * ldx + c);
}

template <int FMT, typename T, int ACC>
__global__ void __launch_bounds__(kThreads, kCtasOf<T, ACC>)
    mx_quant_kernel(MxArgs a) {
  constexpr int kUnroll = kUnrollOf<ACC>;
  __shared__ __align__(16) Stage<T> stage[ACC == kAny ? kWarps : 1];
  const uint32_t lane = threadIdx.x & 31, sub = lane % kGroup, warp = threadIdx.x >> 5;
  const uint32_t step = gridDim.x * (kThreads / kGroup);
  Walk w((blockIdx.x * kThreads + threadIdx.x) / kGroup, step, a.nkb);
  const T* const x = static_cast<const T*>(a.x);
  // a warp goes round together (its shuffles): by its first group
  for (uint32_t base = w.i - lane / kGroup; base < a.total; base += kUnroll * step) {
    Raw16<T> raw[kUnroll];
    T any[ACC == kAny ? kUnroll : 1][16];
    uint32_t at[kUnroll];
    const uint32_t i0 = w.i;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if constexpr (ACC == kAny) {  // 32 consecutive elements of a group an access
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          uint32_t have;
          const T* const p = group_row(x, a.ldx, a.cols, a.rows, g, w.row, w.kb, have) + lane;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            any[u][4 * g + j] = lane + 32 * j < have ? p[32 * j] : from_f32<T>(0.f);
        }
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
    if constexpr (ACC == kAny) {
      Stage<T>& st = stage[warp];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 16; ++j) st.at(32 * j + lane) = any[u][j];
        __syncwarp();
#pragma unroll
        for (int n = 0; n < (int)Stage<T>::kUnits; ++n) {
          const float4 f = st.unit(lane, n);
          raw[u].word(4 * n) = f.x;
          raw[u].word(4 * n + 1) = f.y;
          raw[u].word(4 * n + 2) = f.z;
          raw[u].word(4 * n + 3) = f.w;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint32_t i = i0 + u * step;
      float v[16];
      raw[u].get(v);
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
__global__ void __launch_bounds__(kThreads, kCtasOf<T, ACC>)
    mx_dequant_kernel(MxArgs a) {
  constexpr int kUnroll = kUnrollOf<ACC>;
  __shared__ __align__(16) Stage<T> stage[ACC == kAny ? kWarps : 1];
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
        Stage<T>& st = stage[warp];
        Raw16<T> raw;
        raw.put(v);
        __syncwarp();
#pragma unroll
        for (int n = 0; n < (int)Stage<T>::kUnits; ++n)
          st.unit(lane, n) = make_float4(raw.word(4 * n), raw.word(4 * n + 1), raw.word(4 * n + 2),
                                         raw.word(4 * n + 3));
        __syncwarp();
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          uint32_t have;
          T* const p = group_row(x, a.ldx, a.cols, a.rows, g, row[u], kb[u], have) + lane;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (lane + 32 * j < have) p[32 * j] = st.at(32 * (4 * g + j) + lane);
        }
      } else {
        const uint32_t c = kb[u] * 128 + sub * 16;
        if (row[u] < a.rows && (ACC == kFull || c < a.cols)) {
          Raw16<T> raw;
          raw.put(v);
          raw.store(x + ((int64_t)row[u] * a.ldx + c));
        }
      }
    }
  }
}

template <int FMT, typename T, int ACC>
cudaError_t launch(const MxArgs& a, bool quant, cudaStream_t s) {
  const uint64_t per = (uint64_t)(kThreads / kGroup) * kUnrollOf<ACC>;  // groups a CTA takes at a time
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
