// The residual addition with the root-mean-square norm, and its backward.
//
//     r = x + residual (rounded to the residual's type),  rstd = 1 / sqrt(mean r^2 + eps),
//     y = r rstd w,
// y in x's type or quantised to a microscaled format (mx.cuh) as it is produced.  The norm
// is of the stored r, so the backward, which reads r back, differentiates what the forward
// computed.  With g = w dy and rhat = r rstd (means over the row's d values):
//     dr = rstd (g - rhat mean(g rhat)) + dres,   dw = sum over rows of dy rhat.
//
// Streams: every tensor is read once and written once, so HBM bounds them.  A thread keeps
// eight consecutive values (times NV) of a row in registers between the row's sum and its
// outputs; four lanes share a block of 32 of a microscaled output.  The grid is persistent:
// a CTA walks rows, holding its columns of w, and in the backward its columns of the dw sum
// (written once as one partial row a CTA, summed in a fixed order by a second kernel), in
// registers.
#include <cuda_runtime.h>

#include "internal.h"
#include "mx.cuh"

namespace m3ssd {
namespace {

constexpr int kMaxThreads = 512;

// Sum over the CTA; the result in every thread.  `red` holds one float a warp, twice, so
// that consecutive calls alternate and one barrier a call is enough.
__device__ __forceinline__ float cta_sum(float v, float* red, int& flip) {
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

template <typename T, bool VEC>
__device__ __forceinline__ void ld(const T* row, int c, int d, float (&v)[8]) {
  if (VEC && c + 8 <= d) {
    mx::load8(row + c, v);
  } else {
    mx::load8_tail(row + c, d - c, v);
  }
}
template <typename T, bool VEC>
__device__ __forceinline__ void st(T* row, int c, int d, const float (&v)[8]) {
  if (VEC && c + 8 <= d) {
    mx::store8(row + c, v);
  } else {
    mx::store8_tail(row + c, d - c, v);
  }
}
// One eight-value group; loads past the row's end give zeros.
template <typename T>
__device__ __forceinline__ float round_to(float v) { return to_f32(from_f32<T>(v)); }

// FMT: -1 y in x's type, else the microscaled format.
template <typename T, typename R, bool RES, int FMT, int NV, bool VEC>
__global__ void __launch_bounds__(kMaxThreads) add_rmsnorm_kernel(NormArgs a) {
  __shared__ float red[32];
  const int d = (int)a.d, T8 = 8 * blockDim.x, c0 = 8 * threadIdx.x;
  int flip = 0;
  float w[NV][8];
#pragma unroll
  for (int k = 0; k < NV; ++k) mx::load8_tail(a.w + c0 + k * T8, d - c0 - k * T8, w[k]);
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + row * a.d;
    float v[NV][8];
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) ld<T, VEC>(x, c0 + k * T8, d, v[k]);
    if (RES) {
      const R* res = static_cast<const R*>(a.res) + row * a.d;
      R* out = static_cast<R*>(a.res_out) + row * a.d;
      float q[NV][8];
#pragma unroll
      for (int k = 0; k < NV; ++k) ld<R, VEC>(res, c0 + k * T8, d, q[k]);
#pragma unroll
      for (int k = 0; k < NV; ++k) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[k][j] = round_to<R>(v[k][j] + q[k][j]);
        st<R, VEC>(out, c0 + k * T8, d, v[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(v[k][j], v[k][j], ss);
    const float rstd = 1.f / sqrtf(cta_sum(ss, red, flip) / (float)d + a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[k][j] = v[k][j] * rstd * w[k][j];
      if (FMT < 0) {
        st<T, VEC>(static_cast<T*>(a.y) + row * a.d, c0 + k * T8, d, v[k]);
      } else {
        // columns past d (zero) fill the row's padding; past the padding nothing is stored
        mx::quant_store8<FMT>(v[k], row, (c0 + k * T8) / 8, a.Kp, a.codes, a.scales,
                              c0 + k * T8 < a.Kp, 0xffffffffu);
      }
    }
  }
  if (FMT >= 0) {  // scale bytes of the last tile's missing rows
    const int64_t pad = mx::pad128(a.rows), nkb = a.Kp >> 7;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < (pad - a.rows) * nkb;
         i += (int64_t)gridDim.x * blockDim.x)
      *reinterpret_cast<uint32_t*>(a.scales + mx::scale_word(a.rows + i / nkb, i % nkb, nkb)) = 0;
  }
}

template <typename T, typename R, bool DRES, int NV, bool VEC>
__global__ void __launch_bounds__(kMaxThreads) add_rmsnorm_bwd_kernel(NormBwdArgs a) {
  __shared__ float red[32];
  const int d = (int)a.d, T8 = 8 * blockDim.x, c0 = 8 * threadIdx.x;
  int flip = 0;
  float w[NV][8], dw[NV][8];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    mx::load8_tail(a.w + c0 + k * T8, d - c0 - k * T8, w[k]);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[k][j] = 0.f;
  }
  const float inv_d = 1.f / (float)d;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    float g[NV][8], rh[NV][8];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      ld<T, VEC>(static_cast<const T*>(a.dy) + row * a.d, c0 + k * T8, d, g[k]);
      ld<R, VEC>(static_cast<const R*>(a.r) + row * a.d, c0 + k * T8, d, rh[k]);
    }
    const float rstd = a.rstd[row];
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        rh[k][j] *= rstd;
        dw[k][j] = fmaf(g[k][j], rh[k][j], dw[k][j]);
        g[k][j] *= w[k][j];
        s = fmaf(g[k][j], rh[k][j], s);
      }
    const float m = cta_sum(s, red, flip) * inv_d;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float o[8];
      if (DRES) ld<float, VEC>(a.dres + row * a.d, c0 + k * T8, d, o);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float t = rstd * (g[k][j] - rh[k][j] * m);
        o[j] = DRES ? o[j] + t : t;
      }
      st<float, VEC>(a.dr + row * a.d, c0 + k * T8, d, o);
    }
  }
#pragma unroll
  for (int k = 0; k < NV; ++k)
    mx::store8_tail(a.part + (int64_t)blockIdx.x * a.d + c0 + k * T8, d - c0 - k * T8, dw[k]);
}

// dw = sum of the partial rows, in a fixed order: 32 columns a CTA, eight warps taking the
// partial rows in turn, then the eight sums.
__global__ void __launch_bounds__(256) norm_dw_kernel(const float* __restrict__ part, int nparts,
                                                      int64_t d, float* __restrict__ dw) {
  __shared__ float red[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < d)
    for (int p = warp; p < nparts; p += 8) s += part[(int64_t)p * d + c];
  red[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < d) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) t += red[i][lane];
    dw[c] = t;
  }
}

// Threads of a CTA and eight-value groups a thread for rows of `width` values.
struct Shape {
  int threads, nv;
};
Shape shape_of(int64_t width) {
  int64_t t = ((width + 7) / 8 + 31) / 32 * 32;
  if (t > kMaxThreads) t = kMaxThreads;
  const int64_t nv = (width + 8 * t - 1) / (8 * t);
  return {(int)t, nv <= 1 ? 1 : nv <= 2 ? 2 : 4};
}

unsigned grid_of(int64_t rows, int threads) {
  const int64_t sms = current_device_sms() > 0 ? current_device_sms() : 148;
  const int64_t most = sms * (2048 / threads < 16 ? 2048 / threads : 16) / 2;
  return (unsigned)(rows < most ? rows : most);
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <typename T, typename R, bool RES, int FMT, int NV>
cudaError_t fwd_nv(const NormArgs& a, int threads, bool vec, cudaStream_t s) {
  const unsigned grid = grid_of(a.rows, threads);
  if (vec)
    add_rmsnorm_kernel<T, R, RES, FMT, NV, true><<<grid, threads, 0, s>>>(a);
  else
    add_rmsnorm_kernel<T, R, RES, FMT, NV, false><<<grid, threads, 0, s>>>(a);
  return cudaGetLastError();
}
template <typename T, typename R, bool RES, int FMT>
cudaError_t fwd_fmt(const NormArgs& a, cudaStream_t s) {
  const Shape h = shape_of(FMT < 0 ? a.d : a.Kp);
  const bool vec = a.d % 8 == 0 && al16(a.x) && (!RES || (al16(a.res) && al16(a.res_out))) &&
                   (FMT >= 0 || al16(a.y));
  return h.nv == 1   ? fwd_nv<T, R, RES, FMT, 1>(a, h.threads, vec, s)
         : h.nv == 2 ? fwd_nv<T, R, RES, FMT, 2>(a, h.threads, vec, s)
                     : fwd_nv<T, R, RES, FMT, 4>(a, h.threads, vec, s);
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

template <typename T, typename R, bool DRES, int NV>
cudaError_t bwd_nv(const NormBwdArgs& a, int threads, unsigned grid, bool vec, cudaStream_t s) {
  if (vec)
    add_rmsnorm_bwd_kernel<T, R, DRES, NV, true><<<grid, threads, 0, s>>>(a);
  else
    add_rmsnorm_bwd_kernel<T, R, DRES, NV, false><<<grid, threads, 0, s>>>(a);
  return cudaGetLastError();
}
template <typename T, typename R>
cudaError_t bwd_t(const NormBwdArgs& a, cudaStream_t s) {
  const Shape h = shape_of(a.d);
  const unsigned grid = grid_of(a.rows, h.threads);
  const bool vec = a.d % 8 == 0 && al16(a.dy) && al16(a.r) && al16(a.dr) && al16(a.dres);
  if (a.dres)
    return h.nv == 1   ? bwd_nv<T, R, true, 1>(a, h.threads, grid, vec, s)
           : h.nv == 2 ? bwd_nv<T, R, true, 2>(a, h.threads, grid, vec, s)
                       : bwd_nv<T, R, true, 4>(a, h.threads, grid, vec, s);
  return h.nv == 1   ? bwd_nv<T, R, false, 1>(a, h.threads, grid, vec, s)
         : h.nv == 2 ? bwd_nv<T, R, false, 2>(a, h.threads, grid, vec, s)
                     : bwd_nv<T, R, false, 4>(a, h.threads, grid, vec, s);
}

}  // namespace

bool norm_width_ok(int64_t d) { return d <= (int64_t)kMaxThreads * 8 * 4; }

cudaError_t launch_add_rmsnorm(const NormArgs& a, cudaStream_t s) {
  if (a.rows == 0) return cudaSuccess;
  return a.bf16 ? fwd_t<__nv_bfloat16>(a, s) : fwd_t<float>(a, s);
}

size_t norm_bwd_workspace_bytes(int64_t rows, int64_t d) {
  if (rows == 0) return 0;
  return (size_t)grid_of(rows, shape_of(d).threads) * (size_t)d * sizeof(float);
}

cudaError_t launch_add_rmsnorm_bwd(const NormBwdArgs& a, cudaStream_t s) {
  if (a.rows == 0) return cudaMemsetAsync(a.dw, 0, (size_t)a.d * sizeof(float), s);
  cudaError_t e = a.bf16 ? (a.res_bf16 ? bwd_t<__nv_bfloat16, __nv_bfloat16>(a, s)
                                       : bwd_t<__nv_bfloat16, float>(a, s))
                         : (a.res_bf16 ? bwd_t<float, __nv_bfloat16>(a, s)
                                       : bwd_t<float, float>(a, s));
  if (e != cudaSuccess) return e;
  norm_dw_kernel<<<(unsigned)((a.d + 31) / 32), 256, 0, s>>>(
      a.part, (int)grid_of(a.rows, shape_of(a.d).threads), a.d, a.dw);
  return cudaGetLastError();
}

}  // namespace m3ssd
