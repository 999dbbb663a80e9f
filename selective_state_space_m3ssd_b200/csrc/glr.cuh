// The gated linear recurrence's arithmetic, for two channels at a time (packed fp32).
//
// Per channel, with k = c softplus(rate):
//     rho = sigma(r + bias_r),  iota = sigma(i + bias_i),  a = exp(-k rho),  s = sqrt(1 - a^2),
//     h_t = a_t h_{t-1} + s_t iota_t x_t.
// With e_r = exp(-(r + bias_r)) and e_i alike, one reciprocal serves both gates:
//     R = 1 / ((1 + e_r)(1 + e_i)),  rho = (1 + e_i) R,  iota = (1 + e_r) R,  1 - rho = e_r rho,
// the exponents held below 63 so that the product stays finite (a gate below 2^-63 counts as
// that).  a = 2^t with t = -k log2(e) rho is split into 2^n (1 + q), |f| = |t - n| <= 1/2,
// q = 2^f - 1 by a polynomial, which keeps 1 - a to fp32's relative precision however close a
// is to one: 1 - a = (1 - 2^n) - 2^n q, 1 - a^2 = (1 - a)(1 + a).  So an element takes four
// hardware approximations (two exponentials, a reciprocal, a reciprocal root), each within
// 2^-22 of its value.
#pragma once

#include "common.cuh"

namespace m3ssd {
namespace glr {

constexpr float kLog2e = 1.44269504088896341f;

__device__ __forceinline__ float ex2(float v) {
  float o;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(o) : "f"(v));
  return o;
}
__device__ __forceinline__ float rcp(float v) {
  float o;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(o) : "f"(v));
  return o;
}
__device__ __forceinline__ float rsq(float v) {
  float o;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(o) : "f"(v));
  return o;
}
// Minimum and maximum that keep a NaN.
__device__ __forceinline__ float min_nan(float a, float b) {
  float o;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(o) : "f"(a), "f"(b));
  return o;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float o;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(o) : "f"(a), "f"(b));
  return o;
}
__device__ __forceinline__ float2 splat(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 neg2(float2 a) { return make_float2(-a.x, -a.y); }

// A thread's two channels: t = k2 rho; e_r = 2^(nbr - log2(e) r).
struct Channel {
  float2 k2, nbr, nbi;
};

// softplus(v) and its logarithmic derivative, sigma(v) / softplus(v).
__device__ __forceinline__ float softplus(float v) { return v > 20.f ? v : log1pf(expf(v)); }
__device__ __forceinline__ float softplus_slope(float v) {
  // both are exp(v)(1 - exp(v)/2 + ...) far down; their quotient is 1 there
  if (v < -20.f) return 1.f;
  return 1.f / ((1.f + expf(-v)) * softplus(v));
}

__device__ __forceinline__ void channel_of(const float* rate, const float* bias_r,
                                           const float* bias_i, float c, int64_t d0, int64_t d1,
                                           int64_t width, Channel& ch) {
  float k[2], br[2], bi[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int64_t d = j ? d1 : d0;
    const bool in = d < width;
    // from 2^71 on no gate, 2^-63 or more, leaves any of the state: held there, (log a) times a = 0 is 0
    k[j] = in ? max_nan(-kLog2e * c * softplus(rate[d]), -0x1p71f) : 0.f;
    br[j] = in && bias_r ? -kLog2e * bias_r[d] : 0.f;
    bi[j] = in && bias_i ? -kLog2e * bias_i[d] : 0.f;
  }
  ch.k2 = make_float2(k[0], k[1]);
  ch.nbr = make_float2(br[0], br[1]);
  ch.nbi = make_float2(bi[0], bi[1]);
}

// exp(-(g + bias)), at most 2^63.
__device__ __forceinline__ float2 gate_exp(float2 g, float2 nb) {
  const float2 t = fma2(g, splat(-kLog2e), nb);
  return make_float2(ex2(min_nan(t.x, 63.f)), ex2(min_nan(t.y, 63.f)));
}

// a = 2^t and nz = a^2 - 1 of t <= 0.  (2^f - 1) / f on [-1/2, 1/2] by the polynomial of degree
// five with the least relative error (1.1e-8, found by an exchange algorithm).
__device__ __forceinline__ void decay_of(float2 t, float2& a, float2& nz) {
  // adding 1.5 2^23 rounds to whole numbers, 127 more leaves 2^n's exponent in the low bits
  const float big = 12582912.f + 127.f;
  t = make_float2(max_nan(t.x, -127.f), max_nan(t.y, -127.f));  // 2^-127 is made as zero
  const float2 m = add2(t, splat(big));
  const float2 f = add2(t, fma2(m, splat(-1.f), splat(big)));
  float2 p = fma2(f, splat(1.5403517521e-4f), splat(1.3390735724e-3f));
  p = fma2(f, p, splat(9.6182374772e-3f));
  p = fma2(f, p, splat(5.5503573998e-2f));
  p = fma2(f, p, splat(2.4022649811e-1f));
  p = fma2(f, p, splat(6.9314718793e-1f));
  const float2 q = mul2(f, p);
  const float2 w = make_float2(__int_as_float(__float_as_int(m.x) << 23),
                               __int_as_float(__float_as_int(m.y) << 23));
  a = fma2(w, q, w);
  const float2 nc = fma2(w, q, add2(w, splat(-1.f)));  // a - 1
  nz = fma2(nc, a, nc);
}

__device__ __forceinline__ float root(float v) {
  float o;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(o) : "f"(v));
  return o;
}

// The forward's element: a and u = s iota x.  At a reset a = 0, so s = 1.
__device__ __forceinline__ void element(const Channel& ch, float2 x, float2 r, float2 i, bool reset,
                                        float2& a, float2& u) {
  const float2 dr = add2(gate_exp(r, ch.nbr), splat(1.f));
  const float2 di = add2(gate_exp(i, ch.nbi), splat(1.f));
  const float2 d = mul2(dr, di), R = make_float2(rcp(d.x), rcp(d.y));
  const float2 rho = mul2(di, R), iota = mul2(dr, R);
  float2 nz;
  decay_of(mul2(ch.k2, rho), a, nz);
  float2 s = make_float2(root(-nz.x), root(-nz.y));
  if (reset) {
    a = splat(0.f);
    s = splat(1.f);
  }
  u = mul2(mul2(s, iota), x);
}

// The decay alone, which is all that the walk of g needs, and a^2 - 1.  The gate is held as element()
// and element_grad() hold it: the latter divides its own log a by the root of this a^2 - 1.
__device__ __forceinline__ void decay(const Channel& ch, float2 r, float2& a, float2& nz) {
  const float2 q = add2(gate_exp(r, ch.nbr), splat(1.f));
  decay_of(mul2(ch.k2, make_float2(rcp(q.x), rcp(q.y))), a, nz);
}

// The backward's element, from g = dL/dh_t and h_{t-1} (prev): the gradients of x, i, r and
// E = g dh/d(log a) log a, whose sum gives the rate's.  KNOWN: a and a^2 - 1 are given, else
// they are worked out.  g becomes a g, what goes on to h_{t-1}.
template <bool KNOWN>
__device__ __forceinline__ void element_grad(const Channel& ch, float2 x, float2 r, float2 i, bool reset,
                                             float2 prev, float2 a, float2 nz, float2& g, float2& dx,
                                             float2& dr, float2& di, float2& E) {
  const float2 er = gate_exp(r, ch.nbr), ei = gate_exp(i, ch.nbi);
  const float2 qr = add2(er, splat(1.f)), qi = add2(ei, splat(1.f));
  const float2 d = mul2(qr, qi), R = make_float2(rcp(d.x), rcp(d.y));
  const float2 rho = mul2(qi, R), iota = mul2(qr, R);
  const float2 t = mul2(ch.k2, rho);
  if constexpr (!KNOWN) decay_of(t, a, nz);
  // 1 / s and s; 1e-37 changes no 1 - a^2 above 1e-29, and keeps both finite at zero
  const float2 inv = make_float2(rsq(1e-37f - nz.x), rsq(1e-37f - nz.y));
  float2 s = make_float2(-nz.x * inv.x, -nz.y * inv.y);
  if (reset) s = splat(1.f);
  const float2 v = mul2(iota, x);
  dx = mul2(mul2(g, s), iota);
  di = mul2(mul2(dx, x), mul2(ei, iota));
  if (reset) {
    E = dr = g = splat(0.f);
  } else {
    g = mul2(g, a);
    // a (h_{t-1} - a v / s), times log a: (log a) / s stays finite as s goes to zero
    const float2 la = mul2(t, splat(0.693147180559945309f));
    const float2 w = mul2(mul2(a, v), mul2(la, inv));
    E = mul2(g, fma2(la, prev, neg2(w)));
    dr = mul2(E, mul2(er, rho));
  }
}

}  // namespace glr
}  // namespace m3ssd
