// The residual addition with the root-mean-square norm, and its backward.
//
//     r = x + residual (rounded to the residual's type),  rstd = 1 / sqrt(mean r^2 + eps),
//     y = r rstd w,
// y in x's type or quantised to a microscaled format (mx.cuh) as it is produced.  The norm
// is of the stored r, so the backward, which reads r back, differentiates what the forward
// computed.  With g = w dy and rhat = r rstd (means over the row's d values):
//     dr = rstd (g - rhat mean(g rhat)) + dres,   dw = sum over rows of dy rhat.
//
// Streams: every tensor is read once and written once, so HBM bounds them.  A thread keeps eight
// values (times NV) of a row in registers between the row's sum and its outputs, read in one
// access of 16 or 32 bytes (four lanes share a block of 32 of a microscaled output). Rows of a
// width that is no multiple of eight start inside an access: they are taken in the accesses they
// lie in (kShift), a microscaled output's values moved to its blocks by shuffles. 16000 x 1049
// (bf16, fp32 residual) takes 44 us forward, 53 to 8 bits and 40 backward (68 with dres), 94, 71
// and 65 element by element, which tensors that are not aligned themselves still are.  The grid
// is persistent: a CTA walks rows, fetching the next while it finishes one, with its columns of
// w, and in the backward its columns of the dw sum, in registers.  The dw sums leave as one
// partial row a walker, which a second kernel adds in a fixed order.
#include <cuda_runtime.h>

#include "internal.h"
#include "mx.cuh"

namespace m3ssd {
namespace {

constexpr int kMaxThreads = 512;

// Sum over a row's threads (blockDim.x); the result in every thread.  `red` holds one float
// a warp, twice, so that consecutive calls alternate and one barrier a call is enough.
__device__ __forceinline__ float row_sum(float v, float* red, int& flip) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int nw = blockDim.x >> 5;
  if (nw == 1) return v;
  float* buf = red + 16 * flip;
  flip ^= 1;
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.f;
  for (int w = 0; w < nw; ++w) t += buf[w];
  return t;
}

// How a thread's values lie in a row: eight consecutive ones in one access; the same of rows
// that start inside such an access (kShift: columns from 8 i - shift on, shift being the
// row's first element modulo 8; the row's ends one by one); eight consecutive ones one by
// one; or eight that are blockDim.x apart.
enum Access { kVec, kShift, kTail, kStrided };

// Eight values of a row as loaded.
template <typename T>
struct Raw;
template <>
struct Raw<float> {
  float f[8];
};
template <>
struct Raw<__nv_bfloat16> {
  uint4 u;
};
__device__ __forceinline__ void unpack(const Raw<float>& r, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = r.f[j];
}
__device__ __forceinline__ void unpack(const Raw<__nv_bfloat16>& r, float (&v)[8]) {
  const uint32_t u[4] = {r.u.x, r.u.y, r.u.z, r.u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(u[j] << 16);
    v[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
  }
}
__device__ __forceinline__ void pack(const float (&v)[8], Raw<float>& r) {
#pragma unroll
  for (int j = 0; j < 8; ++j) r.f[j] = v[j];
}
__device__ __forceinline__ void pack(const float (&v)[8], Raw<__nv_bfloat16>& r) {
  uint32_t u[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)  // the values are bf16: nothing is rounded
    u[j] = (__float_as_uint(v[2 * j]) >> 16) | (__float_as_uint(v[2 * j + 1]) & 0xffff0000u);
  r.u = make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ void load_vec(const float* p, Raw<float>& r) { mx::load8(p, r.f); }
__device__ __forceinline__ void load_vec(const __nv_bfloat16* p, Raw<__nv_bfloat16>& r) {
  r.u = *reinterpret_cast<const uint4*>(p);
}

// kShift: whether the access of columns c to c + 7 of a row lies in the tensor, which has `left`
// elements from the row's first on (a row of fewer than eight may have the tensor's end
// rows behind it), counted over eight rows at most: none of a row's accesses goes further.
__host__ __device__ __forceinline__ bool in_tensor(int c, int left) { return c + 8 <= left; }
__host__ __device__ __forceinline__ int left_of(int64_t rows, int64_t row, int d) {
  return (int)(rows - row < 8 ? rows - row : 8) * d;
}

// Group k of the thread's values of a row, and back.  With kShift the first and the last access
// of a row bring in its neighbours' ends too (inside() drops them; elements that another
// CTA may be writing, in place, are among them), those that would reach past the tensor's end
// are element by element; else there are zeros outside the row.
template <int ACC, typename T>
__device__ __forceinline__ void load_row(const T* row, int k, int d, int shift, int left,
                                         Raw<T>& r) {
  const int c = 8 * ((int)threadIdx.x + k * (int)blockDim.x) - (ACC == kStrided ? 0 : shift);
  float v[8];
  if constexpr (ACC == kVec || ACC == kShift) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.f;
    pack(v, r);
    if (c < d && (ACC == kVec || in_tensor(c, left))) {
      load_vec(row + c, r);  // with kVec d is a multiple of 8
    } else if (ACC == kShift && c < d) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + j >= 0 && c + j < d) v[j] = to_f32(row[c + j]);
      pack(v, r);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = ACC == kTail ? c + j : (int)threadIdx.x + (8 * k + j) * (int)blockDim.x;
      v[j] = i >= 0 && i < d ? to_f32(row[i]) : 0.f;
    }
    pack(v, r);
  }
}
// Zeros in place of what lies outside the row.
template <int ACC>
__device__ __forceinline__ void inside(float (&v)[8], int k, int d, int shift) {
  const int c = 8 * ((int)threadIdx.x + k * (int)blockDim.x) - shift;
  if (c < 0 || c + 8 > d) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (ACC == kVec ? c >= d : c + j < 0 || c + j >= d) v[j] = 0.f;
  }
}
template <int ACC, typename T>
__device__ __forceinline__ void store_row(T* row, int k, int d, int shift, const float (&v)[8]) {
  const int c = 8 * ((int)threadIdx.x + k * (int)blockDim.x) - (ACC == kStrided ? 0 : shift);
  if (ACC == kVec ? c < d : ACC == kShift && c >= 0 && c + 8 <= d) {
    mx::store8(row + c, v);
  } else if constexpr (ACC != kVec) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = ACC != kStrided ? c + j : (int)threadIdx.x + (8 * k + j) * (int)blockDim.x;
      if (i >= 0 && i < d) row[i] = from_f32<T>(v[j]);
    }
  }
}
// The tensors of a walker's columns (w, dw): aligned to nothing.
template <int ACC>
constexpr int kColumns = ACC == kVec || ACC == kShift ? kTail : ACC;
// kShift: the columns by which the walker's rows start inside an access.  Its rows are a
// multiple of eight apart (grid_of), so all have this one.
template <int ACC>
__device__ __forceinline__ int shift_of(int64_t first_row, int64_t d) {
  return ACC == kShift ? (int)((uint64_t)first_row * (uint64_t)d % 8) : 0;
}
// A microscaled output's blocks start at the row's columns: from values of columns 8 i - shift
// on to those of 8 i on.  A thread's last `shift` values come from the next one: by shuffles, and
// past a warp's end from `edge`, which holds the first values of each warp and group (twice, so
// that one barrier a call is enough).
template <int NV>
struct Edge {
  float v[2][NV * 16][8];
};
template <int NV>
__device__ __forceinline__ void realign(float (&v)[NV][8], int shift, Edge<NV>& edge, int& flip) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const bool shared = nw * NV > 1;
  if (shared) {
    flip ^= 1;
    if (lane == 0) {
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) edge.v[flip][k * nw + warp][j] = v[k][j];
    }
    __syncthreads();
  }
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    float x[16];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[j] = v[k][j];
      x[8 + j] = j < 7 ? __shfl_down_sync(0xffffffffu, v[k][j], 1) : 0.f;
    }
    if (lane == 31) {
      const int next = k * nw + warp + 1;
#pragma unroll
      for (int j = 0; j < 7; ++j) x[8 + j] = next < NV * nw ? edge.v[flip][next][j] : 0.f;
    }
#pragma unroll
    for (int b = 4; b > 0; b >>= 1) {  // by `shift`, a bit at a time
#pragma unroll
      for (int j = 0; j + b < 16; ++j)
        if (shift & b) x[j] = x[j + b];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[k][j] = x[j];
  }
}
// Whether a thread holds the next row's values while it finishes one: up to 16 values a
// tensor; more would spill.
constexpr bool ahead(int nv) { return nv <= 2; }
template <typename T>
__device__ __forceinline__ float round_to(float v) { return to_f32(from_f32<T>(v)); }

// FMT: -1 y in x's type, else the microscaled format.
template <typename T, typename R, bool RES, int FMT, int NV, int ACC>
__global__ void __launch_bounds__(kMaxThreads) add_rmsnorm_kernel(NormArgs a) {
  __shared__ float red[32];
  constexpr bool kRealign = FMT >= 0 && ACC == kShift;
  __shared__ Edge<kRealign ? NV : 1> edge;
  const int d = (int)a.d;
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const int shift = shift_of<ACC>(row, d);
  int flip = 0;
  [[maybe_unused]] int flip_edge = 0;
  float w[NV][8];
  Raw<T> xr[NV];
  Raw<R> rr[RES ? NV : 1];
  auto fetch = [&](int64_t i) {
    const int left = left_of(a.rows, i, d);
#pragma unroll
    for (int k = 0; k < NV; ++k)
      load_row<ACC>(static_cast<const T*>(a.x) + i * d, k, d, shift, left, xr[k]);
    if (RES) {
#pragma unroll
      for (int k = 0; k < NV; ++k)
        load_row<ACC>(static_cast<const R*>(a.res) + i * d, k, d, shift, left, rr[RES ? k : 0]);
    }
  };
  if (ahead(NV) && row < a.rows) fetch(row);
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    Raw<float> t;
    load_row<kColumns<ACC>>(a.w, k, d, shift, d, t);
    unpack(t, w[k]);
  }
  for (; row < a.rows; row += step) {
    float v[NV][8], ss = 0.f;
    if (!ahead(NV)) fetch(row);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      unpack(xr[k], v[k]);
      if (RES) {
        float q[8];
        unpack(rr[RES ? k : 0], q);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[k][j] = round_to<R>(v[k][j] + q[j]);
        store_row<ACC>(static_cast<R*>(a.res_out) + row * d, k, d, shift, v[k]);
      }
      if (ACC == kShift) inside<ACC>(v[k], k, d, shift);
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(v[k][j], v[k][j], ss);
    }
    if (ahead(NV) && row + step < a.rows) fetch(row + step);
    const float rstd = 1.f / sqrtf(row_sum(ss, red, flip) / (float)d + a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[k][j] = v[k][j] * rstd * w[k][j];
      // 0 rstd 0 outside the row is NaN where rstd is not finite
      if (FMT >= 0 && !(rstd < INFINITY)) inside<ACC>(v[k], k, d, shift);
    }
    if constexpr (kRealign) realign<NV>(v, shift, edge, flip_edge);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (FMT < 0) {
        store_row<ACC>(static_cast<T*>(a.y) + row * d, k, d, shift, v[k]);
      } else {
        // columns past d (zero) fill the row's padding; past the padding nothing is stored
        const uint32_t c8 = threadIdx.x + k * blockDim.x, nkb = (uint32_t)(a.Kp >> 7);
        uint2 codes;
        const uint32_t word = mx::quant8<FMT>(v[k], codes);
        if (c8 < 16 * nkb) {
          mx::store_codes<FMT>(a.codes, row * nkb + (c8 >> 4), c8 & 15, codes);
          if ((c8 & 15) == 0)
            *reinterpret_cast<uint32_t*>(a.scales + mx::scale_word(row, c8 >> 4, nkb)) = word;
        }
      }
    }
  }
  if (FMT >= 0) {  // scale bytes of the last tile's missing rows
    const int64_t pad = mx::pad128(a.rows), nkb = a.Kp >> 7, per = blockDim.x * blockDim.y;
    for (int64_t i = blockIdx.x * per + threadIdx.y * blockDim.x + threadIdx.x;
         i < (pad - a.rows) * nkb; i += gridDim.x * per)
      *reinterpret_cast<uint32_t*>(a.scales + mx::scale_word(a.rows + i / nkb, i % nkb, nkb)) = 0;
  }
}

template <typename T, typename R, bool DRES, int NV, int ACC>
__global__ void __launch_bounds__(kMaxThreads) add_rmsnorm_bwd_kernel(NormBwdArgs a) {
  __shared__ float red[32];
  cudaTriggerProgrammaticLaunchCompletion();  // norm_dw_kernel may be launched: it waits itself
  const int d = (int)a.d;
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  const int64_t first = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const int shift = shift_of<ACC>(first, d);
  int flip = 0;
  float w[NV][8], dw[NV][8];
  Raw<T> yr[NV];
  Raw<R> rr[NV];
  Raw<float> ur[DRES ? NV : 1];
  float rs = 0.f;
  auto fetch = [&](int64_t i) {
    const int left = left_of(a.rows, i, d);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      load_row<ACC>(static_cast<const T*>(a.dy) + i * d, k, d, shift, left, yr[k]);
      load_row<ACC>(static_cast<const R*>(a.r) + i * d, k, d, shift, left, rr[k]);
      if (DRES) load_row<ACC>(a.dres + i * d, k, d, shift, left, ur[DRES ? k : 0]);
    }
    rs = a.rstd[i];
  };
  if (ahead(NV) && first < a.rows) fetch(first);
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    Raw<float> t;
    load_row<kColumns<ACC>>(a.w, k, d, shift, d, t);
    unpack(t, w[k]);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[k][j] = 0.f;
  }
  const float inv_d = 1.f / (float)d;
  for (int64_t row = first; row < a.rows; row += step) {
    float g[NV][8], rh[NV][8], o[NV][8];
    if (!ahead(NV)) fetch(row);
    const float rstd = rs;
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      unpack(yr[k], g[k]);
      unpack(rr[k], rh[k]);
      if (ACC == kShift) {
        inside<ACC>(g[k], k, d, shift);
        inside<ACC>(rh[k], k, d, shift);
      }
      if (DRES) unpack(ur[DRES ? k : 0], o[k]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        rh[k][j] *= rstd;
        dw[k][j] = fmaf(g[k][j], rh[k][j], dw[k][j]);
        g[k][j] *= w[k][j];
        s = fmaf(g[k][j], rh[k][j], s);
      }
    }
    if (ahead(NV) && row + step < a.rows) fetch(row + step);
    const float m = row_sum(s, red, flip) * inv_d;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float t = rstd * (g[k][j] - rh[k][j] * m);
        o[k][j] = DRES ? o[k][j] + t : t;
      }
      store_row<ACC>(a.dr + row * d, k, d, shift, o[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < NV; ++k)
    store_row<kColumns<ACC>>(a.part + first * d, k, d, shift, dw[k]);
}

// dw = sum of the partial rows, in a fixed order: a CTA takes eight columns, thread (c, p)
// every 32nd partial row of column c, then the 32 sums.
__global__ void __launch_bounds__(256) norm_dw_kernel(const float* part, int nparts, int64_t d,
                                                      float* dw) {
  __shared__ float red[32][8];
  const int c8 = threadIdx.x & 7, p0 = threadIdx.x >> 3;
  const int64_t c = (int64_t)blockIdx.x * 8 + c8;
  float s = 0.f;
  cudaGridDependencySynchronize();  // launched before the backward's end: its sums are there
  if (c < d) {
#pragma unroll 8
    for (int p = p0; p < nparts; p += 32) s += part[(int64_t)p * d + c];
  }
  red[p0][c8] = s;
  __syncthreads();
  if (threadIdx.x < 8 && c < d) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += red[i][threadIdx.x];
    dw[c] = t;
  }
}

// Threads of a row, rows of a CTA and eight-value groups of a thread for rows of `width`.
struct Shape {
  int threads, rows, nv;
};
Shape shape_of(int64_t width) {
  if (width % 8 != 0) width += 7;  // kShift: a row may lie in one more access
  int64_t t = ((width + 7) / 8 + 31) / 32 * 32;
  if (t > kMaxThreads) t = kMaxThreads;
  const int64_t nv = (width + 8 * t - 1) / (8 * t);
  // a row of one warp needs no barrier: four of them make a CTA
  return {(int)t, t == 32 ? 4 : 1, nv <= 1 ? 1 : nv <= 2 ? 2 : 4};
}

// CTAs: about `threads` threads an SM, `least` rows or more each.  More walkers than keep the
// loads in flight only scatter the reads and writes of HBM: 32768 x 1024 (bf16 with an fp32
// residual) forward 71, 66, 63, 68 and 69 us at 512, 640, 768, 896 and 1024 threads, backward
// 78, 76, 92, 85 and 84; the same order at widths of 256 to 2048.
constexpr int kFwdThreads = 768, kBwdThreads = 640;
// Where d is no multiple of 8 the walkers' rows are a multiple of eight apart (kShift).
unsigned grid_of(int64_t rows, int64_t d, const Shape& h, int threads, int least) {
  const int64_t sms = current_device_sms() > 0 ? current_device_sms() : 148;
  const int cta = h.threads * h.rows, ctas = threads / cta > 1 ? threads / cta : 1;
  const int64_t most = sms * ctas, per = (int64_t)h.rows * least;
  const int64_t want = (rows + per - 1) / per, unit = d % 8 == 0 ? 1 : 8;
  // (more than `most` would wait for an SM: four CTAs too many doubled the time)
  const int64_t up = (want + unit - 1) / unit * unit, down = most < unit ? unit : most / unit * unit;
  return (unsigned)(up < down ? up : down);
}

constexpr int64_t kMaxWidth = (int64_t)kMaxThreads * 8 * 4;

// aligned: the tensors' first elements are.
Access access_of(bool aligned, int64_t d) {
  return !aligned ? kStrided : d % 8 == 0 ? kVec : d + 7 <= kMaxWidth ? kShift : kStrided;
}

template <typename T, typename R, bool RES, int FMT, int NV>
cudaError_t fwd_nv(const NormArgs& a, const Shape& h, Access acc, cudaStream_t s) {
  const dim3 block(h.threads, h.rows);
  // two CTAs where a row takes 512 threads: 69 us against 74 at 8192 x 4096
  const unsigned grid =
      grid_of(a.rows, a.d, h, h.threads == kMaxThreads ? 2 * kMaxThreads : kFwdThreads, 1);
  if (acc == kVec)
    add_rmsnorm_kernel<T, R, RES, FMT, NV, kVec><<<grid, block, 0, s>>>(a);
  else if (acc == kShift)
    add_rmsnorm_kernel<T, R, RES, FMT, NV, kShift><<<grid, block, 0, s>>>(a);
  else  // a microscaled output needs its blocks' values together
    add_rmsnorm_kernel<T, R, RES, FMT, NV, FMT < 0 ? kStrided : kTail><<<grid, block, 0, s>>>(a);
  return cudaGetLastError();
}
template <typename T, typename R, bool RES, int FMT>
cudaError_t fwd_fmt(const NormArgs& a, cudaStream_t s) {
  // a microscaled row is written to its padding's end
  const int64_t held = a.d % 8 == 0 ? a.d : (a.d + 14) / 8 * 8;
  const Shape h = shape_of(FMT < 0 ? a.d : a.Kp > held ? a.Kp : held);
  Access acc = access_of(mx::aligned8<T>(a.x, 8) &&
                             (!RES || (mx::aligned8<R>(a.res, 8) && mx::aligned8<R>(a.res_out, 8))) &&
                             (FMT >= 0 || mx::aligned8<T>(a.y, 8)),
                         a.d);
  // realigning to the blocks pays where a row is long: to 8 bits from bf16 with an fp32
  // residual, 20000 x 513 38.5 us against 42.9 element by element, but from fp32 48.2 against
  // 40.1; at 16000 x 1049 53 against 71 and 47 against 60; at 30000 x 275 40 against 37 and 47
  // against 33
  if (FMT >= 0 && acc == kShift && a.d < 768) acc = kStrided;
  return h.nv == 1   ? fwd_nv<T, R, RES, FMT, 1>(a, h, acc, s)
         : h.nv == 2 ? fwd_nv<T, R, RES, FMT, 2>(a, h, acc, s)
                     : fwd_nv<T, R, RES, FMT, 4>(a, h, acc, s);
}
template <typename T, typename R, bool RES>
cudaError_t fwd_res(const NormArgs& a, cudaStream_t s) {
  return a.fmt < 0           ? fwd_fmt<T, R, RES, -1>(a, s)
         : a.fmt == mx::kFp4 ? fwd_fmt<T, R, RES, mx::kFp4>(a, s)
                             : fwd_fmt<T, R, RES, mx::kFp8>(a, s);
}
template <typename T>
cudaError_t fwd_t(const NormArgs& a, cudaStream_t s) {
  if (!a.res) return fwd_res<T, float, false>(a, s);
  return a.res_bf16 ? fwd_res<T, __nv_bfloat16, true>(a, s) : fwd_res<T, float, true>(a, s);
}

// The backward's CTAs take at least four rows each: every walker costs a partial row.
constexpr int kLeastRows = 4;

template <typename T, typename R, bool DRES, int NV>
cudaError_t bwd_nv(const NormBwdArgs& a, const Shape& h, Access acc, cudaStream_t s) {
  const dim3 block(h.threads, h.rows);
  const unsigned grid = grid_of(a.rows, a.d, h, kBwdThreads, kLeastRows);
  if (acc == kVec)
    add_rmsnorm_bwd_kernel<T, R, DRES, NV, kVec><<<grid, block, 0, s>>>(a);
  else if (acc == kShift)
    add_rmsnorm_bwd_kernel<T, R, DRES, NV, kShift><<<grid, block, 0, s>>>(a);
  else
    add_rmsnorm_bwd_kernel<T, R, DRES, NV, kStrided><<<grid, block, 0, s>>>(a);
  return cudaGetLastError();
}
template <typename T, typename R>
cudaError_t bwd_t(const NormBwdArgs& a, cudaStream_t s) {
  const Shape h = shape_of(a.d);
  const Access acc = access_of(mx::aligned8<T>(a.dy, 8) && mx::aligned8<R>(a.r, 8) &&
                                   mx::aligned8<float>(a.dr, 8) && mx::aligned8<float>(a.dres, 8),
                               a.d);
  if (a.dres)
    return h.nv == 1   ? bwd_nv<T, R, true, 1>(a, h, acc, s)
           : h.nv == 2 ? bwd_nv<T, R, true, 2>(a, h, acc, s)
                       : bwd_nv<T, R, true, 4>(a, h, acc, s);
  return h.nv == 1   ? bwd_nv<T, R, false, 1>(a, h, acc, s)
         : h.nv == 2 ? bwd_nv<T, R, false, 2>(a, h, acc, s)
                     : bwd_nv<T, R, false, 4>(a, h, acc, s);
}

int64_t partial_rows(int64_t rows, int64_t d) {
  const Shape h = shape_of(d);
  return (int64_t)grid_of(rows, d, h, kBwdThreads, kLeastRows) * h.rows;
}

}  // namespace

bool norm_whole_access(int64_t rows, int64_t d, int64_t row, int c) {
  return access_of(true, d) != kStrided && in_tensor(c, left_of(rows, row, (int)d));
}

bool norm_width_ok(int64_t d) { return d <= kMaxWidth; }

cudaError_t launch_add_rmsnorm(const NormArgs& a, cudaStream_t s) {
  if (a.rows == 0) return cudaSuccess;
  return a.bf16 ? fwd_t<__nv_bfloat16>(a, s) : fwd_t<float>(a, s);
}

size_t norm_bwd_workspace_bytes(int64_t rows, int64_t d) {
  return rows == 0 ? 0 : (size_t)partial_rows(rows, d) * (size_t)d * sizeof(float);
}

cudaError_t launch_add_rmsnorm_bwd(const NormBwdArgs& a, cudaStream_t s) {
  if (a.rows == 0) return cudaMemsetAsync(a.dw, 0, (size_t)a.d * sizeof(float), s);
  cudaError_t e = a.bf16 ? (a.res_bf16 ? bwd_t<__nv_bfloat16, __nv_bfloat16>(a, s)
                                       : bwd_t<__nv_bfloat16, float>(a, s))
                         : (a.res_bf16 ? bwd_t<float, __nv_bfloat16>(a, s)
                                       : bwd_t<float, float>(a, s));
  if (e != cudaSuccess) return e;
  // its CTAs may take their places while the backward's last ones run
  cudaLaunchAttribute early[1];
  early[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((a.d + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cfg.attrs = early;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, norm_dw_kernel, (const float*)a.part,
                         (int)partial_rows(a.rows, a.d), (int64_t)a.d, a.dw);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace m3ssd
