// The gated linear recurrence over a sequence, its backward, and one step of it (glr.cuh has
// the arithmetic).
#include <cuda_runtime.h>

#include <cstdint>

#include "glr.cuh"
#include "internal.h"

namespace m3ssd {
namespace {

using namespace glr;

constexpr int kThreads = 128;

template <typename T>
__device__ __forceinline__ float2 load2(const T* p, bool in1) {
  return make_float2(to_f32(p[0]), in1 ? to_f32(p[1]) : 0.f);
}
template <typename T>
__device__ __forceinline__ void store2(T* p, float2 v, bool in1) {
  p[0] = from_f32<T>(v.x);
  if (in1) p[1] = from_f32<T>(v.y);
}

// One thread walks two channels of a sequence.
template <typename T>
__global__ void __launch_bounds__(kThreads) glr_fwd_kernel(GlrArgs a) {
  const int64_t pairs = (a.D + 1) / 2, id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (id >= a.b * pairs) return;
  const int64_t b = id / pairs, d = id % pairs * 2;
  const bool in1 = d + 1 < a.D;
  Channel ch;
  channel_of(a.rate, a.bias_r, a.bias_i, a.c, d, d + 1, a.D, ch);
  float2 h = a.h0 ? load2(a.h0 + b * a.D + d, in1) : splat(0.f);
  const int64_t len = a.lengths ? min(max((int64_t)a.lengths[b], (int64_t)0), a.L) : a.L;
  T* y = static_cast<T*>(a.y) + b * a.L * a.D + d;
  for (int64_t t = 0; t < len; ++t) {
    const int64_t row = b * a.L + t;
    float2 al, u;
    const bool cut = a.reset && a.reset[row];
    element(ch, load2(static_cast<const T*>(a.x) + row * a.ldx + d, in1),
            load2(static_cast<const T*>(a.r) + row * a.ldr + d, in1),
            load2(static_cast<const T*>(a.i) + row * a.ldi + d, in1), cut, al, u);
    h = cut ? u : fma2(al, h, u);
    store2(y + t * a.D, h, in1);
  }
  for (int64_t t = len; t < a.L; ++t) store2(y + t * a.D, splat(0.f), in1);
  if (a.hT) store2(a.hT + b * a.D + d, h, in1);
}

// The same walk from the last token; the sums of a sequence go to a row of partial sums.
template <typename T, typename G>
__global__ void __launch_bounds__(kThreads) glr_bwd_kernel(GlrBwdArgs a) {
  const GlrArgs& f = a.f;
  const int64_t pairs = (f.D + 1) / 2, id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (id >= f.b * pairs) return;
  const int64_t b = id / pairs, d = id % pairs * 2;
  const bool in1 = d + 1 < f.D;
  Channel ch;
  channel_of(f.rate, f.bias_r, f.bias_i, f.c, d, d + 1, f.D, ch);
  const int64_t len = f.lengths ? min(max((int64_t)f.lengths[b], (int64_t)0), f.L) : f.L;
  float2 back = a.dhT ? load2(a.dhT + b * f.D + d, in1) : splat(0.f);
  float2 sr = splat(0.f), si = splat(0.f), se = splat(0.f);
  const T* y = static_cast<const T*>(f.y) + b * f.L * f.D + d;
  const T* dy = static_cast<const T*>(a.dy) + b * f.L * f.D + d;
  for (int64_t t = f.L - 1; t >= 0; --t) {
    const int64_t row = b * f.L + t;
    float2 dx = splat(0.f), dr = dx, di = dx, E = dx;
    if (t < len) {
      const bool cut = f.reset && f.reset[row];
      const float2 prev = t > 0     ? load2(y + (t - 1) * f.D, in1)
                          : f.h0 ? load2(f.h0 + b * f.D + d, in1)
                                 : splat(0.f);
      const float2 g = add2(load2(dy + t * f.D, in1), back);
      const float2 al = element_grad(ch, load2(static_cast<const T*>(f.x) + row * f.ldx + d, in1),
                                     load2(static_cast<const T*>(f.r) + row * f.ldr + d, in1),
                                     load2(static_cast<const T*>(f.i) + row * f.ldi + d, in1), cut,
                                     prev, g, dx, dr, di, E);
      back = cut ? splat(0.f) : mul2(al, g);
      sr = add2(sr, dr);
      si = add2(si, di);
      se = add2(se, E);
    }
    store2(static_cast<G*>(a.dx) + row * a.ldg + d, dx, in1);
    store2(static_cast<G*>(a.dr) + row * a.ldg + d, dr, in1);
    store2(static_cast<G*>(a.di) + row * a.ldg + d, di, in1);
  }
  if (a.dh0) store2(a.dh0 + b * f.D + d, back, in1);
  float* part = a.part + 3 * b * f.D + d;
  store2(part, se, in1);
  store2(part + f.D, sr, in1);
  store2(part + 2 * f.D, si, in1);
}

// drate, dbias_r and dbias_i of a channel: its partial sums in a fixed order.
__global__ void __launch_bounds__(kThreads) glr_sum_kernel(const float* part, int64_t parts, int64_t D,
                                                           const float* rate, float* drate,
                                                           float* dbias_r, float* dbias_i) {
  const int64_t d = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (d >= D) return;
  float s[3] = {0.f, 0.f, 0.f};
  for (int64_t p = 0; p < parts; ++p)
#pragma unroll
    for (int j = 0; j < 3; ++j) s[j] += part[(3 * p + j) * D + d];
  drate[d] = s[0] * softplus_slope(rate[d]);
  if (dbias_r) dbias_r[d] = s[1];
  if (dbias_i) dbias_i[d] = s[2];
}

template <typename T>
__global__ void __launch_bounds__(kThreads) glr_step_kernel(GlrStepArgs a) {
  const int64_t pairs = (a.D + 1) / 2, id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (id >= a.b * pairs) return;
  const int64_t b = id / pairs, d = id % pairs * 2;
  const bool in1 = d + 1 < a.D;
  Channel ch;
  channel_of(a.rate, a.bias_r, a.bias_i, a.c, d, d + 1, a.D, ch);
  float2 al, u;
  element(ch, load2(static_cast<const T*>(a.x) + b * a.ldx + d, in1),
          load2(static_cast<const T*>(a.r) + b * a.ldr + d, in1),
          load2(static_cast<const T*>(a.i) + b * a.ldi + d, in1), false, al, u);
  const float2 h = fma2(al, load2(a.h + b * a.D + d, in1), u);
  store2(a.h_out + b * a.D + d, h, in1);
  store2(static_cast<T*>(a.y) + b * a.D + d, h, in1);
}

unsigned grid_for(int64_t n) { return (unsigned)((n + kThreads - 1) / kThreads); }

template <typename T, typename G>
cudaError_t bwd_t(const GlrBwdArgs& a, cudaStream_t s) {
  glr_bwd_kernel<T, G><<<grid_for(a.f.b * ((a.f.D + 1) / 2)), kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_glr_fwd(const GlrArgs& a, cudaStream_t s) {
  const unsigned grid = grid_for(a.b * ((a.D + 1) / 2));
  if (a.bf16)
    glr_fwd_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(a);
  else
    glr_fwd_kernel<float><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

size_t glr_bwd_workspace_bytes(int64_t b, int64_t, int64_t D) {
  return (size_t)b * 3 * (size_t)D * sizeof(float);
}

cudaError_t launch_glr_bwd(const GlrBwdArgs& a, cudaStream_t s) {
  const GlrArgs& f = a.f;
  if (f.b > 0) {
    const cudaError_t e = !f.bf16         ? bwd_t<float, float>(a, s)
                          : a.grad_bf16 ? bwd_t<__nv_bfloat16, __nv_bfloat16>(a, s)
                                        : bwd_t<__nv_bfloat16, float>(a, s);
    if (e != cudaSuccess) return e;
  }
  glr_sum_kernel<<<grid_for(f.D), kThreads, 0, s>>>(a.part, f.b, f.D, f.rate, a.drate, a.dbias_r,
                                                     a.dbias_i);
  return cudaGetLastError();
}

cudaError_t launch_glr_step(const GlrStepArgs& a, cudaStream_t s) {
  if (a.b == 0) return cudaSuccess;
  const unsigned grid = grid_for(a.b * ((a.D + 1) / 2));
  if (a.bf16)
    glr_step_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(a);
  else
    glr_step_kernel<float><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace m3ssd
