// The decode step on a cache whose state is held in 8 bits, and the state's way into and
// out of that form.
//
// A row (b, h, n) of the state, P values, is held as E4M3 codes with one fp32 scale:
//     s = amax fp32(1 / 448),  code = v (1 / s) rounded to nearest even,  v ~ code s,
// rows with amax < 2^-100 as zeros, a row with a NaN or an infinity with a NaN scale.  A
// decay alone moves only the scale (the row's codes come back the same), so a state that
// receives nothing fades without loss; what a step adds is rounded to 2^-4 relative, with
// a floor of 2^-10 s.  The step is step.cu's on the values the cache stands for:
//     h = alpha code s + beta Bbar_prev x_prev^T + gamma Bbar x_t^T,  y = Cbar^T h + D x_t,
// y from the unrounded h, and h rounded once as it is written.
//
// Bytes set the pace of the fp32 step; at a quarter of them (2 N P + 8 N a (b, h)) the
// instructions a value takes cost as much as HBM does, so the kernel keeps them few:
// conversions two values at a time, multiply-adds two fp32 values at a time (f32x2), two
// 16-byte shared-memory loads for a row's four factors, a sum of y whose exchanges are a
// thirtieth of the work.  At b256 H32 N128 P64 on one B200: 35 us against 24 for the bytes at
// the copy rate (4.5 TB/s, 0.68 of it; the fp32 step takes 87).  The schedulers issue in 56 % of
// the cycles (a two-wide operation takes two of them), 3.6 warps a scheduler: what is left is
// latency, part of it a round's own order (angles and rotations, a barrier, then the rows).
// Without the decoding, the encoding or the maxima it took 1 to 2 us less, without its stores 4,
// with 7 or 9 CTAs an SM 39 and 38 us.
#include <cuda_runtime.h>

#include "internal.h"
#include "mx.cuh"
#include "tc5.cuh"

namespace m3ssd {

__device__ unsigned int g_step_q8_wait_timeouts;

namespace {

constexpr int kN = 128, kP = 64;
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr float kTiny = 7.8886090522101181e-31f;  // 2^-100

__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// max that returns NaN when either input is one
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float rcp_approx(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// A row's scale from its largest magnitude (NaN where that is not finite: amax 0), and its
// reciprocal: the correctly rounded one (EXACT), or the hardware's, within an ulp, which moves
// only values next to a rounding border (rounded correctly the step takes 38.4 us against 35.4
// at b256 H32, 53 against 46 at N64 P64).
template <bool EXACT>
__device__ __forceinline__ void row_scale(float amax, float& s, float& inv) {
  const float t = fmaf(amax, 1.f / 448.f, amax * 0.f);
  s = amax < kTiny ? 0.f : t;
  const float u = fmaxf(t, 1.f / 448.f * kTiny);  // (a NaN row's codes are not read)
  inv = amax < kTiny ? 0.f : EXACT ? 1.f / u : rcp_approx(u);
}

__device__ __forceinline__ void load16(const float* p, float (&v)[16]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float4 f = reinterpret_cast<const float4*>(p)[j];
    v[4 * j] = f.x; v[4 * j + 1] = f.y; v[4 * j + 2] = f.z; v[4 * j + 3] = f.w;
  }
}
__device__ __forceinline__ void load16(const __nv_bfloat16* p, float (&v)[16]) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    float t[8];
    mx::load8(p + 8 * j, t);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[8 * j + i] = t[i];
  }
}

// sin and cos of x, |x| up to about 1e5, to fp32 precision: x - k pi / 2 with pi / 2 split
// into its nearest fp32 value and the remainder (Cody-Waite argument reduction), the Taylor
// series on [-pi/4, pi/4] (the first terms left out are below 2e-9 and 1e-10), and the
// quadrant's exchange and signs.  About half the instructions of sincosf, which also covers
// every larger argument.
__device__ __forceinline__ void sincos_reduced(float x, float* s, float* c) {
  const float k = rintf(x * 0.636619772367581343f);  // 2 / pi
  const int quad = (int)k;
  float r = fmaf(-k, 1.57079637050628662f, x);   // fp32(pi / 2)
  r = fmaf(-k, -4.37113882867379282e-08f, r);    // pi / 2 - fp32(pi / 2)
  const float r2 = r * r;
  float ps = fmaf(r2, 1.f / 362880.f, -1.f / 5040.f);
  ps = fmaf(r2, ps, 1.f / 120.f);
  ps = fmaf(r2, ps, -1.f / 6.f);
  ps = fmaf(r2 * r, ps, r);
  float pc = fmaf(r2, -1.f / 3628800.f, 1.f / 40320.f);
  pc = fmaf(r2, pc, -1.f / 720.f);
  pc = fmaf(r2, pc, 1.f / 24.f);
  pc = fmaf(r2, pc, -0.5f);
  pc = fmaf(r2, pc, 1.f);
  const float a = quad & 1 ? pc : ps, b = quad & 1 ? ps : pc;
  *s = __uint_as_float(__float_as_uint(a) ^ ((uint32_t)(quad & 2) << 30));
  *c = __uint_as_float(__float_as_uint(b) ^ ((uint32_t)((quad + 1) & 2) << 30));
}

// Factors of the state rows, each twice (a pair for the two-wide operations): beta Bbar_prev
// and gamma Bbar, Cbar and alpha s.  Two arrays of 16 bytes a row: the eight rows a warp
// works on are read without bank conflicts.
struct RowCoefs {
  float4 in[kN], out[kN];
  __device__ void set_prev(int n, float bp) { *reinterpret_cast<float2*>(&in[n].x) = make_float2(bp, bp); }
  __device__ void set_new(int n, float bc) { *reinterpret_cast<float2*>(&in[n].z) = make_float2(bc, bc); }
  __device__ void set_c(int n, float cc) { *reinterpret_cast<float2*>(&out[n].x) = make_float2(cc, cc); }
  __device__ void set_decay(int n, float as) { *reinterpret_cast<float2*>(&out[n].z) = make_float2(as, as); }
  __device__ void set_all(int n, float bp, float bc, float cc, float as) {
    in[n] = make_float4(bp, bp, bc, bc);
    out[n] = make_float4(cc, cc, as, as);
  }
};

// N = 128, P = 64: a lane owns 16 columns (lane % 4) of a row, so a row is complete in four
// lanes and a warp's access to eight rows is 512 contiguous bytes.
// Sixteen values of a row: the new ones from the old codes, and their part of amax; adds
// Cbar h to acc.
__device__ __forceinline__ float advance(const uint4& codes, const RowCoefs& f, int n,
                                         const uint64_t (&x2)[8], const uint64_t (&xp2)[8],
                                         uint64_t (&acc)[8], uint64_t (&v)[8]) {
  const ulonglong2 f0 = *reinterpret_cast<const ulonglong2*>(&f.in[n]),
                   f1 = *reinterpret_cast<const ulonglong2*>(&f.out[n]);
  const uint32_t c4[4] = {codes.x, codes.y, codes.z, codes.w};
  float amax = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 c = mx::unpack2_e4m3(c4[j >> 1] >> (16 * (j & 1)));
    v[j] = fma2(f0.y, x2[j], fma2(f0.x, xp2[j], mul2(f1.y, pack2(c.x, c.y))));
    acc[j] = fma2(f1.x, v[j], acc[j]);
    const float2 u = unpack2(v[j]);
    amax = mx::max3_abs(amax, u.x, u.y);
  }
  return amax;
}
__device__ __forceinline__ uint4 to_codes(const uint64_t (&v)[8], float inv) {
  const uint64_t inv2 = pack2(inv, inv);
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 u = unpack2(mul2(v[2 * j], inv2)), w = unpack2(mul2(v[2 * j + 1], inv2));
    o[j] = mx::pack4_e4m3(u.x, u.y, w.x, w.y);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}
// Rows n0 and n1: their new codes and scales.
__device__ __forceinline__ void update_rows(const uint4& h0, const uint4& h1, const RowCoefs& f,
                                            int n0, int n1, const uint64_t (&x2)[8],
                                            const uint64_t (&xp2)[8], uint64_t (&acc)[8],
                                            uint4& o0, uint4& o1, float& s0, float& s1) {
  uint64_t v0[8], v1[8];
  float m0 = advance(h0, f, n0, x2, xp2, acc, v0), m1 = advance(h1, f, n1, x2, xp2, acc, v1);
  m0 = max_nan(m0, __shfl_xor_sync(0xffffffffu, m0, 1));
  m1 = max_nan(m1, __shfl_xor_sync(0xffffffffu, m1, 1));
  m0 = max_nan(m0, __shfl_xor_sync(0xffffffffu, m0, 2));
  m1 = max_nan(m1, __shfl_xor_sync(0xffffffffu, m1, 2));
  float i0, i1;
  row_scale<false>(m0, s0, i0);
  row_scale<false>(m1, s1, i1);
  o0 = to_codes(v0, i0);
  o1 = to_codes(v1, i1);
}

// Sums acc over the lanes with equal lane % 4 (the same 16 columns): each exchange halves
// what a lane keeps, until it has columns col and col + 1 of the warp's sum.
__device__ __forceinline__ float2 sum_columns(const uint64_t (&acc)[8], int lane, int& col) {
  float y[16];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 u = unpack2(acc[j]);
    y[2 * j] = u.x;
    y[2 * j + 1] = u.y;
  }
  col = 16 * (lane & 3);
#pragma unroll
  for (int w = 8, bit = 16; w >= 2; w >>= 1, bit >>= 1) {
    const bool up = lane & bit;
#pragma unroll
    for (int j = 0; j < w; ++j) {
      const float send = up ? y[j] : y[j + w], keep = up ? y[j + w] : y[j];
      y[j] = keep + __shfl_xor_sync(0xffffffffu, send, bit);
    }
    col += up ? w : 0;
  }
  return make_float2(y[0], y[1]);
}

__device__ __forceinline__ void pairs(const float (&v)[16], uint64_t (&p)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) p[j] = pack2(v[2 * j], v[2 * j + 1]);
}

// Few (b, h): a CTA of four warps each, everything loaded at once, the rotations a thread a
// pair and angle.  2.6 us at 72 (b, h) in a graph, where a launch that does nothing takes 2.
template <typename T>
__global__ void __launch_bounds__(128) step_q8_one(StepQ8Args a) {
  constexpr int kRows = 4;  // rows a lane
  __shared__ RowCoefs coef;
  __shared__ float ysum[4][kP];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int64_t bh = blockIdx.x;
  const uint32_t H = (uint32_t)a.H, rep = H / (uint32_t)a.G, b = blockIdx.x / H;
  const uint32_t h = blockIdx.x - b * H, g = h / rep;
  const int q = lane & 3, r0 = warp * 32 + (lane >> 2);

  const uint4* S = reinterpret_cast<const uint4*>(a.ssm + bh * kN * kP);
  uint4 hv[kRows];
#pragma unroll
  for (int k = 0; k < kRows; ++k) hv[k] = S[(r0 + 8 * k) * (kP / 16) + q];
  const T* xt = static_cast<const T*>(a.x_t) + bh * kP;
  float x[16], xp[16];
  load16(xt + 16 * q, x);
  load16(a.x_prev + bh * kP + 16 * q, xp);

  const T* Bt = static_cast<const T*>(a.B_t) + ((int64_t)b * a.G + g) * kN;
  const T* Ct = static_cast<const T*>(a.C_t) + ((int64_t)b * a.G + g) * kN;
  const int i = t & 63;  // rows 2 i and 2 i + 1
  const float ang = a.angle[bh * 64 + i];
  float ph = 0.f, sn, cs;
  if (t < 64) {  // what turns with the new angle
    const float ga = a.gamma_t[bh];
    ph = wrap_angle(ang + (a.theta_t ? a.theta_t[bh * 64 + i] : 0.f));
    sincos_reduced(ph, &sn, &cs);
    const float b0 = to_f32(Bt[2 * i]), b1 = to_f32(Bt[2 * i + 1]);
    const float2 rb = rot2(cs, sn, b0, b1);
    const float2 rc = rot2(cs, sn, to_f32(Ct[2 * i]), to_f32(Ct[2 * i + 1]));
    coef.set_new(2 * i, ga * rb.x);
    coef.set_new(2 * i + 1, ga * rb.y);
    coef.set_c(2 * i, rc.x);
    coef.set_c(2 * i + 1, rc.y);
    if (a.b_prev_out && h % rep == 0)
      *reinterpret_cast<float2*>(a.b_prev_out + ((int64_t)b * a.G + g) * kN + 2 * i) = make_float2(b0, b1);
  } else {  // and with the old
    const float alpha = expf(a.logdecay_t[bh]), be = a.beta_t ? a.beta_t[bh] : 0.f;
    const float2 bp = *reinterpret_cast<const float2*>(a.b_prev + ((int64_t)b * a.G + g) * kN + 2 * i);
    const float2 sc = *reinterpret_cast<const float2*>(a.scale + bh * kN + 2 * i);
    sincos_reduced(ang, &sn, &cs);
    const float2 rp = rot2(cs, sn, bp.x, bp.y);
    coef.set_prev(2 * i, be * rp.x);
    coef.set_prev(2 * i + 1, be * rp.y);
    coef.set_decay(2 * i, alpha * sc.x);
    coef.set_decay(2 * i + 1, alpha * sc.y);
  }
  __syncthreads();

  uint64_t x2[8], xp2[8], acc[8] = {};
  pairs(x, x2);
  pairs(xp, xp2);
  uint4* So = reinterpret_cast<uint4*>(a.ssm_out + bh * kN * kP);
#pragma unroll
  for (int k = 0; k < kRows; k += 2) {
    const int n0 = r0 + 8 * k, n1 = n0 + 8;
    uint4 o0, o1;
    float s0, s1;
    update_rows(hv[k], hv[k + 1], coef, n0, n1, x2, xp2, acc, o0, o1, s0, s1);
    So[n0 * (kP / 16) + q] = o0;
    So[n1 * (kP / 16) + q] = o1;
    if (q == 0) {
      a.scale_out[bh * kN + n0] = s0;
      a.scale_out[bh * kN + n1] = s1;
    }
  }
  int col;
  const float2 y2 = sum_columns(acc, lane, col);
  *reinterpret_cast<float2*>(&ysum[warp][col]) = y2;
  __syncthreads();
  if (t >= 64) return;
  a.angle_out[bh * 64 + t] = ph;  // every old angle and x_prev was read before the barriers
  float y = (ysum[0][t] + ysum[1][t]) + (ysum[2][t] + ysum[3][t]);
  const float xv = to_f32(xt[t]);
  if (a.D) y = fmaf(a.D[h], xv, y);
  static_cast<T*>(a.y_t)[bh * kP + t] = from_f32<T>(y);
  a.x_prev_out[bh * kP + t] = xv;
}

// Many (b, h): CTAs of two warps walk them; bulk copies bring the next one's parts into one
// of two stages while a CTA works on the other, so the state is never waited for with
// registers held, and eight CTAs an SM (128 registers a thread) keep 78 KB in flight.
constexpr int kWalkThreads = 64, kWalkCtas = 8;

template <typename T>
struct alignas(2 * sizeof(T)) Pair {
  T a, b;
};
template <typename T>
struct alignas(128) StepStage {
  uint8_t codes[kN * kP];
  float scale[kN];
  float angle[kN / 2];
  float theta[kN / 2];
  float xp[kP];
  T x[kP];
};

template <typename T>
__global__ void __launch_bounds__(kWalkThreads, kWalkCtas) step_q8_walk(StepQ8Args a) {
  constexpr int kRows = 8;  // rows a lane
  __shared__ StepStage<T> stage[2];
  __shared__ RowCoefs coef;
  __shared__ float ysum[2][kP];
  __shared__ uint64_t full[2];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int q = lane & 3, r0 = warp * 64 + (lane >> 2);
  const int64_t total = a.b * a.H;
  // the (b, h) and group of a round go along without a division by H
  const uint32_t H = (uint32_t)a.H, rep = H / (uint32_t)a.G;
  const uint32_t db = gridDim.x / H, dh = gridDim.x - db * H;
  uint32_t b = blockIdx.x / H, h = blockIdx.x - b * H;
  auto fetch = [&](int64_t bh, int st) {
    StepStage<T>& d = stage[st];
    const uint32_t bytes = sizeof(d.codes) + sizeof(d.scale) + sizeof(d.angle) + sizeof(d.xp) +
                           sizeof(d.x) + (a.theta_t ? sizeof(d.theta) : 0);
    tc5::mbar_arrive_expect_tx(&full[st], bytes);
    tc5::bulk_load(tc5::saddr(d.codes), a.ssm + bh * kN * kP, sizeof(d.codes), &full[st]);
    tc5::bulk_load(tc5::saddr(d.scale), a.scale + bh * kN, sizeof(d.scale), &full[st]);
    tc5::bulk_load(tc5::saddr(d.angle), a.angle + bh * (kN / 2), sizeof(d.angle), &full[st]);
    tc5::bulk_load(tc5::saddr(d.xp), a.x_prev + bh * kP, sizeof(d.xp), &full[st]);
    tc5::bulk_load(tc5::saddr(d.x), static_cast<const T*>(a.x_t) + bh * kP, sizeof(d.x), &full[st]);
    if (a.theta_t)
      tc5::bulk_load(tc5::saddr(d.theta), a.theta_t + bh * (kN / 2), sizeof(d.theta), &full[st]);
  };
  if (t == 0) {
    tc5::mbar_init(&full[0], 1);
    tc5::mbar_init(&full[1], 1);
    tc5::fence_mbar_init();
  }
  __syncthreads();
  // what a round reads outside its stage, loaded a round ahead
  struct Small {
    Pair<T> B, C;
    float2 bp;
    float ld, be, ga, D;
    int64_t at;   // of the pair's B, C and b_prev
    bool first;   // the group's first head
  } cur, nxt;
  auto small = [&](int64_t bh) {
    Small v;
    const uint32_t g = a.G == 1 ? 0u : h / rep;
    v.at = ((int64_t)b * a.G + g) * kN + 2 * t;  // pair t: rows 2 t and 2 t + 1
    v.B = *reinterpret_cast<const Pair<T>*>(static_cast<const T*>(a.B_t) + v.at);
    v.C = *reinterpret_cast<const Pair<T>*>(static_cast<const T*>(a.C_t) + v.at);
    v.bp = *reinterpret_cast<const float2*>(a.b_prev + v.at);
    v.ld = a.logdecay_t[bh];
    v.be = a.beta_t ? a.beta_t[bh] : 0.f;
    v.ga = a.gamma_t[bh];
    v.D = a.D ? a.D[h] : 0.f;
    v.first = h == g * rep;
    b += db;  // to the next round's
    h += dh;
    if (h >= H) {
      h -= H;
      ++b;
    }
    return v;
  };
  int64_t bh = blockIdx.x;
  if (t == 0) fetch(bh, 0);  // the grid is no larger than the walk
  cur = small(bh);
  for (uint32_t it = 0; bh < total; bh += gridDim.x, ++it) {
    const int st = it & 1;
    const int64_t next = bh + gridDim.x;
    // the other stage was last read before the barrier that ended the round before
    if (t == 0 && next < total) fetch(next, st ^ 1);
    if (next < total) nxt = small(next);
    const float b0 = to_f32(cur.B.a), b1 = to_f32(cur.B.b), c0 = to_f32(cur.C.a), c1 = to_f32(cur.C.b);
    const float2 bp = cur.bp;
    const float alpha = expf(cur.ld), be = cur.be, ga = cur.ga;
    const StepStage<T>& d = stage[st];
    // the lanes of give_up do not wait (a test's); a warp is late where one of its lanes is
    const bool late = __any_sync(0xffffffffu, (a.give_up >> lane & 1u) ||
                                 !tc5::mbar_wait(&full[st], (it >> 1) & 1u, kWaitLimitNs));
    float ph;
    {
      float sn, cs;
      const float ang = d.angle[t];
      sincos_reduced(ang, &sn, &cs);
      const float2 rp = rot2(cs, sn, bp.x, bp.y);
      ph = wrap_angle(ang + (a.theta_t ? d.theta[t] : 0.f));
      sincos_reduced(ph, &sn, &cs);
      const float2 rb = rot2(cs, sn, b0, b1), rc = rot2(cs, sn, c0, c1);
      coef.set_all(2 * t, be * rp.x, ga * rb.x, rc.x, alpha * d.scale[2 * t]);
      coef.set_all(2 * t + 1, be * rp.y, ga * rb.y, rc.y, alpha * d.scale[2 * t + 1]);
    }
    if (tc5::bar_or(1, kWalkThreads, late)) {  // the copies in flight land before the CTA ends
      if (t == 0) {
        (void)tc5::mbar_wait(&full[st], (it >> 1) & 1u, kWaitLimitNs);
        if (next < total)
          (void)tc5::mbar_wait(&full[st ^ 1], ((it + 1) >> 1) & 1u, kWaitLimitNs);
        atomicAdd(&g_step_q8_wait_timeouts, 1u);
      }
      return;
    }
    // nothing of this (b, h) is written before no thread was late
    a.angle_out[bh * (kN / 2) + t] = ph;
    if (a.b_prev_out && cur.first)
      *reinterpret_cast<float2*>(a.b_prev_out + cur.at) = make_float2(b0, b1);
    uint64_t x2[8], xp2[8], acc[8] = {};
    {
      float v[16];
      load16(d.x + 16 * q, v);
      pairs(v, x2);
      load16(d.xp + 16 * q, v);
      pairs(v, xp2);
    }
    const float xv = to_f32(d.x[t]);
    const uint4* S = reinterpret_cast<const uint4*>(d.codes);
    uint4* So = reinterpret_cast<uint4*>(a.ssm_out + bh * kN * kP);
    // two rows at a time: their chains of conversions, maxima and exchanges overlap
#pragma unroll
    for (int k = 0; k < kRows; k += 2) {
      const int n0 = r0 + 8 * k, n1 = n0 + 8;
      const uint4 h0 = S[n0 * (kP / 16) + q], h1 = S[n1 * (kP / 16) + q];
      uint4 o0, o1;
      float s0, s1;
      update_rows(h0, h1, coef, n0, n1, x2, xp2, acc, o0, o1, s0, s1);
      So[n0 * (kP / 16) + q] = o0;
      So[n1 * (kP / 16) + q] = o1;
      if (q == 0) {
        a.scale_out[bh * kN + n0] = s0;
        a.scale_out[bh * kN + n1] = s1;
      }
    }
    int col;
    const float2 y2 = sum_columns(acc, lane, col);
    *reinterpret_cast<float2*>(&ysum[warp][col]) = y2;
    __syncthreads();
    float y = ysum[0][t] + ysum[1][t];
    if (a.D) y = fmaf(cur.D, xv, y);
    static_cast<T*>(a.y_t)[bh * kP + t] = from_f32<T>(y);
    a.x_prev_out[bh * kP + t] = xv;
    cur = nxt;
  }
}

// Every other shape: one CTA a (b, h); `lanes` lanes (a power of two) share a row, eight columns
// each.  VEC: rows of a multiple of eight columns, aligned: a lane's codes are one access.
// b256 H32 N64 P64 takes 46 us (13 for the bytes: a CTA's life is mostly its chain of angles,
// rotations, rows and sum, with nothing in flight for the next one), b64 H32 N256 P64 32, b128
// H32 N128 P75 bf16 110 (its codes go byte by byte); with a warp a row, a column of each 32 a
// lane, 3.4, 4.1 and 1.4 times as long.  Measured and not kept: odd rows in the
// accesses they lie in (no faster, and the sums it needs cost the others 10 %), registers for
// 8 or 10 CTAs an SM (spills; 10 to 40 % slower).
constexpr int kGenThreads = 128, kGenWarps = kGenThreads / 32, kGenUnroll = 4;
template <typename T, bool VEC>
__global__ void __launch_bounds__(kGenThreads) step_q8_kernel(StepQ8Args a, int lanes) {
  extern __shared__ float smem[];
  const int N = (int)a.N, P = (int)a.P, NH = N / 2;
  const int64_t bh = blockIdx.x, b = bh / a.H, h = bh % a.H, rep = a.H / a.G, g = h / rep;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int c = 8 * (tid % lanes), r0 = tid / lanes, per = kGenThreads / lanes;
  float* bc = smem;            // N   gamma Bbar
  float* cc = bc + N;          // N   Cbar
  float* bp = cc + N;          // N   beta Bbar_prev
  float* ysum = bp + N;        // kGenWarps * P
  uint2 q[kGenUnroll];
  float sc[kGenUnroll];
  auto fetch = [&](int base) {  // rows base, base + per, ...
#pragma unroll
    for (int u = 0; u < kGenUnroll; ++u) {
      const int n = base + u * per;
      q[u] = make_uint2(0u, 0u);
      sc[u] = 0.f;
      if (n < N) {
        sc[u] = a.scale[bh * N + n];
        const uint8_t* const p = a.ssm + (bh * N + n) * P + c;
        if (VEC) {
          if (c < P) q[u] = *reinterpret_cast<const uint2*>(p);
        } else {
          uint32_t w[2] = {0u, 0u};
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (c + j < P) w[j >> 2] |= (uint32_t)p[j] << (8 * (j & 3));
          q[u] = make_uint2(w[0], w[1]);
        }
      }
    }
  };
  fetch(r0);
  const T* Bt = static_cast<const T*>(a.B_t) + (b * a.G + g) * N;
  const T* Ct = static_cast<const T*>(a.C_t) + (b * a.G + g) * N;
  const float* bprev = a.b_prev + (b * a.G + g) * N;
  const float alpha = expf(a.logdecay_t[bh]);
  const float be = a.beta_t ? a.beta_t[bh] : 0.f, ga = a.gamma_t[bh];
  const T* xt = static_cast<const T*>(a.x_t) + bh * P;
  float x[8], xp[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = xp[j] = 0.f;
  if (VEC) {
    if (c < P) {
      mx::load8(xt + c, x);
      mx::load8(a.x_prev + bh * P + c, xp);
    }
  } else {
    mx::load8_tail(xt + c, P - c, x);
    mx::load8_tail(a.x_prev + bh * P + c, P - c, xp);
  }
  for (int i = tid; i < NH; i += kGenThreads) {
    const float ang = a.angle[bh * NH + i];
    const float ph = wrap_angle(ang + (a.theta_t ? a.theta_t[bh * NH + i] : 0.f));
    float s, c1, s0, c0;
    sincosf(ph, &s, &c1);
    sincosf(ang, &s0, &c0);
    const float b0 = to_f32(Bt[2 * i]), b1 = to_f32(Bt[2 * i + 1]);
    const float2 rb = rot2(c1, s, b0, b1);
    const float2 rc = rot2(c1, s, to_f32(Ct[2 * i]), to_f32(Ct[2 * i + 1]));
    const float2 rp = rot2(c0, s0, bprev[2 * i], bprev[2 * i + 1]);
    bc[2 * i] = ga * rb.x; bc[2 * i + 1] = ga * rb.y;
    cc[2 * i] = rc.x; cc[2 * i + 1] = rc.y;
    bp[2 * i] = be * rp.x; bp[2 * i + 1] = be * rp.y;
    a.angle_out[bh * NH + i] = ph;
    if (a.b_prev_out && h % rep == 0) {
      a.b_prev_out[(b * a.G + g) * N + 2 * i] = b0;
      a.b_prev_out[(b * a.G + g) * N + 2 * i + 1] = b1;
    }
  }
  uint64_t x2[4], xp2[4], acc[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x2[j] = pack2(x[2 * j], x[2 * j + 1]);
    xp2[j] = pack2(xp[2 * j], xp[2 * j + 1]);
    acc[j] = pack2(0.f, 0.f);
  }
  __syncthreads();
  // the CTA's threads go round together (the lanes of a row share shuffles)
  for (int base = 0; base < N; base += kGenUnroll * per) {
    uint2 now[kGenUnroll];
    float ns[kGenUnroll];
#pragma unroll
    for (int u = 0; u < kGenUnroll; ++u) {
      now[u] = q[u];
      ns[u] = sc[u];
    }
    if (base + kGenUnroll * per < N) fetch(base + kGenUnroll * per + r0);
#pragma unroll
    for (int u = 0; u < kGenUnroll; ++u) {
      const int n = base + u * per + r0;
      if (base + u * per >= N) break;
      const bool have = n < N;
      const float as = have ? alpha * ns[u] : 0.f, f0 = have ? bp[n] : 0.f, f1 = have ? bc[n] : 0.f,
                  f2 = have ? cc[n] : 0.f;
      const uint64_t as2 = pack2(as, as), f02 = pack2(f0, f0), f12 = pack2(f1, f1),
                     f22 = pack2(f2, f2);
      float v[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 e = mx::unpack2_e4m3((j < 2 ? now[u].x : now[u].y) >> (16 * (j & 1)));
        const uint64_t w = fma2(f12, x2[j], fma2(f02, xp2[j], mul2(as2, pack2(e.x, e.y))));
        if (have) acc[j] = fma2(f22, w, acc[j]);  // (x may be infinite)
        const float2 f = unpack2(w);
        v[2 * j] = f.x;
        v[2 * j + 1] = f.y;
      }
      if (!VEC) {  // columns past the row's end take no part (a NaN scale or factor)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c + j >= P) v[j] = 0.f;
      } else if (c >= P) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.f;
      }
      float amax = mx::amax8(v);
      for (int o = 1; o < lanes; o <<= 1)
        amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      float s, inv;
      row_scale<false>(amax, s, inv);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= inv;
      if (have) {
        uint8_t* const out = a.ssm_out + (bh * N + n) * P + c;
        if (VEC) {
          if (c < P)
            *reinterpret_cast<uint2*>(out) = make_uint2(mx::pack4_e4m3(v[0], v[1], v[2], v[3]),
                                                        mx::pack4_e4m3(v[4], v[5], v[6], v[7]));
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (c + j < P) out[j] = (uint8_t)mx::pack2_e4m3(v[j], 0.f);
        }
        if (c == 0) a.scale_out[bh * N + n] = s;
      }
    }
  }
  float y[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = unpack2(acc[j]);
    y[2 * j] = f.x;
    y[2 * j + 1] = f.y;
  }
  for (int o = lanes; o < 32; o <<= 1) {  // the warp's rows
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] += __shfl_xor_sync(0xffffffffu, y[j], o);
  }
  if (lane < lanes) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c + j < P) ysum[warp * P + c + j] = y[j];
  }
  __syncthreads();
  for (int p = tid; p < P; p += kGenThreads) {
    const float xv = to_f32(xt[p]);
    float t = a.D ? a.D[h] * xv : 0.f;
    for (int w = 0; w < kGenWarps; ++w) t += ysum[w * P + p];
    static_cast<T*>(a.y_t)[bh * P + p] = from_f32<T>(t);
    a.x_prev_out[bh * P + p] = xv;
  }
}

// b_prev <- B_t where the step writes the cache it read: every head of the group has read
// the old one by now.
template <typename T>
__global__ void bprev_q8_kernel(const T* __restrict__ B_t, float* __restrict__ b_prev, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i < n) b_prev[i] = to_f32(B_t[i]);
}

template <typename T>
cudaError_t launch_step_t(StepQ8Args a, cudaStream_t s) {
  const bool inplace = a.b_prev_out == a.b_prev;
  float* const bprev = a.b_prev_out;
  if (inplace) a.b_prev_out = nullptr;
  const int64_t nbh = a.b * a.H;
  const uintptr_t all = reinterpret_cast<uintptr_t>(a.ssm) | reinterpret_cast<uintptr_t>(a.ssm_out) |
                        reinterpret_cast<uintptr_t>(a.x_t) | reinterpret_cast<uintptr_t>(a.x_prev) |
                        reinterpret_cast<uintptr_t>(a.scale) | reinterpret_cast<uintptr_t>(a.angle) |
                        reinterpret_cast<uintptr_t>(a.theta_t) | reinterpret_cast<uintptr_t>(a.b_prev) |
                        reinterpret_cast<uintptr_t>(a.B_t) | reinterpret_cast<uintptr_t>(a.C_t) |
                        reinterpret_cast<uintptr_t>(bprev);
  if (a.N == kN && a.P == kP && all % 16 == 0) {
    const int64_t sms = current_device_sms() > 0 ? current_device_sms() : 148;
    const int64_t walkers = sms * kWalkCtas;
    // up to two CTAs of four warps an SM run at once; more (b, h) than that are walked
    if (nbh <= 2 * sms) {
      step_q8_one<T><<<(unsigned)nbh, 128, 0, s>>>(a);
    } else {
      a.give_up = take_given_up_lanes();
      step_q8_walk<T><<<(unsigned)(nbh < walkers ? nbh : walkers), kWalkThreads, 0, s>>>(a);
    }
  } else {
    const size_t smem = sizeof(float) * (size_t)(3 * a.N + kGenWarps * a.P);
    int lanes = 1;
    while (8 * lanes < a.P) lanes *= 2;  // P <= 256: at most 32
    if (a.P % 8 == 0 && mx::aligned8<T>(a.x_t, a.P) && mx::aligned8<float>(a.x_prev, a.P) &&
        (reinterpret_cast<uintptr_t>(a.ssm) | reinterpret_cast<uintptr_t>(a.ssm_out)) % 8 == 0)
      step_q8_kernel<T, true><<<(unsigned)nbh, kGenThreads, smem, s>>>(a, lanes);
    else
      step_q8_kernel<T, false><<<(unsigned)nbh, kGenThreads, smem, s>>>(a, lanes);
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !inplace) return e;
  const int64_t nb = a.b * a.G * a.N;
  bprev_q8_kernel<T><<<(unsigned)((nb + 255) / 256), 256, 0, s>>>(static_cast<const T*>(a.B_t),
                                                                  bprev, nb);
  return cudaGetLastError();
}

// ---- the state in and out of the 8-bit form -------------------------------------------
// `lanes` lanes (a power of two) share a row, eight values each.
struct StateArgs {
  int64_t rows;
  int P, lanes;
  float* h;
  uint8_t* codes;
  float* scale;
};

constexpr int kStThreads = 256, kStUnroll = 4;

template <bool VEC>
__global__ void __launch_bounds__(kStThreads) quant_state_kernel(StateArgs a) {
  const int per = kStThreads / a.lanes;  // rows a CTA takes at a time
  const int c = 8 * (threadIdx.x % a.lanes);
  const int64_t stride = (int64_t)gridDim.x * per;
  const int64_t first = (int64_t)blockIdx.x * per;
  for (int64_t base = first; base < a.rows; base += kStUnroll * stride) {
    float v[kStUnroll][8];
#pragma unroll
    for (int u = 0; u < kStUnroll; ++u) {
      const int64_t r = base + u * stride + threadIdx.x / a.lanes;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[u][j] = 0.f;
      if (r < a.rows && c < a.P) {
        if (VEC)
          mx::load8(a.h + r * a.P + c, v[u]);
        else
          mx::load8_tail(a.h + r * a.P + c, a.P - c, v[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < kStUnroll; ++u) {
      const int64_t r = base + u * stride + threadIdx.x / a.lanes;
      float amax = mx::amax8(v[u]);
      for (int o = 1; o < a.lanes; o <<= 1)
        amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      float s, inv;
      row_scale<true>(amax, s, inv);
      if (r >= a.rows || c >= a.P) continue;
      float q[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) q[j] = v[u][j] * inv;
      uint8_t* out = a.codes + r * a.P + c;
      if (VEC) {
        *reinterpret_cast<uint2*>(out) = make_uint2(mx::pack4_e4m3(q[0], q[1], q[2], q[3]),
                                                    mx::pack4_e4m3(q[4], q[5], q[6], q[7]));
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c + j < a.P) out[j] = (uint8_t)mx::pack2_e4m3(q[j], 0.f);
      }
      if (c == 0) a.scale[r] = s;
    }
  }
}

template <bool VEC>
__global__ void __launch_bounds__(kStThreads) dequant_state_kernel(StateArgs a) {
  const int per = kStThreads / a.lanes;
  const int c = 8 * (threadIdx.x % a.lanes);
  if (c >= a.P) return;
  const int64_t stride = (int64_t)gridDim.x * per;
  for (int64_t base = (int64_t)blockIdx.x * per + threadIdx.x / a.lanes; base < a.rows;
       base += kStUnroll * stride) {
    uint2 q[kStUnroll];
    float s[kStUnroll];
#pragma unroll
    for (int u = 0; u < kStUnroll; ++u) {
      const int64_t r = base + u * stride;
      if (r >= a.rows) continue;
      s[u] = a.scale[r];
      const uint8_t* p = a.codes + r * a.P + c;
      if (VEC) {
        q[u] = *reinterpret_cast<const uint2*>(p);
      } else {
        uint32_t w[2] = {0u, 0u};
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c + j < a.P) w[j >> 2] |= (uint32_t)p[j] << (8 * (j & 3));
        q[u] = make_uint2(w[0], w[1]);
      }
    }
#pragma unroll
    for (int u = 0; u < kStUnroll; ++u) {
      const int64_t r = base + u * stride;
      if (r >= a.rows) continue;
      float v[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = mx::unpack2_e4m3((j < 2 ? q[u].x : q[u].y) >> (16 * (j & 1)));
        v[2 * j] = f.x * s[u];
        v[2 * j + 1] = f.y * s[u];
      }
      if (VEC)
        mx::store8(a.h + r * a.P + c, v);
      else
        mx::store8_tail(a.h + r * a.P + c, a.P - c, v);
    }
  }
}

cudaError_t launch_state(bool quant, int64_t rows, int64_t P, float* h, void* codes, float* scale,
                         cudaStream_t s) {
  if (rows == 0) return cudaSuccess;
  StateArgs a{rows, (int)P, 1, h, static_cast<uint8_t*>(codes), scale};
  while (8 * a.lanes < P) a.lanes *= 2;  // P <= 256: at most 32
  const bool vec = mx::aligned8<float>(h, P) && reinterpret_cast<uintptr_t>(codes) % 8 == 0;
  const int64_t per = (int64_t)(kStThreads / a.lanes) * kStUnroll;
  const int64_t want = (rows + per - 1) / per, sms = current_device_sms();
  const unsigned grid = (unsigned)(sms > 0 && want > sms * 8 ? sms * 8 : want);
  if (quant)
    vec ? quant_state_kernel<true><<<grid, kStThreads, 0, s>>>(a)
        : quant_state_kernel<false><<<grid, kStThreads, 0, s>>>(a);
  else
    vec ? dequant_state_kernel<true><<<grid, kStThreads, 0, s>>>(a)
        : dequant_state_kernel<false><<<grid, kStThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_step_q8(const StepQ8Args& a, cudaStream_t s) {
  if (a.b * a.H == 0) return cudaSuccess;
  return a.bf16 ? launch_step_t<__nv_bfloat16>(a, s) : launch_step_t<float>(a, s);
}
cudaError_t read_and_clear_step_q8_wait_timeouts(unsigned int* count) {
  const unsigned int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(count, g_step_q8_wait_timeouts, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_step_q8_wait_timeouts, &zero, sizeof(unsigned int));
}
cudaError_t launch_quant_state(int64_t rows, int64_t P, const float* h, void* codes, float* scale,
                               cudaStream_t s) {
  return launch_state(true, rows, P, const_cast<float*>(h), codes, scale, s);
}
cudaError_t launch_dequant_state(int64_t rows, int64_t P, const void* codes, const float* scale,
                                 float* h, cudaStream_t s) {
  return launch_state(false, rows, P, h, const_cast<void*>(codes), const_cast<float*>(scale), s);
}

}  // namespace m3ssd
