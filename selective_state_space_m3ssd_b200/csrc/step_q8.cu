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
// instructions a value takes come close to the time HBM takes, so the kernel keeps them
// few: conversions two values at a time, multiply-adds two fp32 values at a time (f32x2),
// one 16-byte shared-memory load a row for the row's four factors, and a sum of y whose
// exchanges are a thirtieth of the work.
#include <cuda_runtime.h>

#include "internal.h"
#include "mx.cuh"

namespace m3ssd {
namespace {

constexpr int kN = 128, kP = 64;
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

// A row's scale and its reciprocal from its largest magnitude (NaN where a value is NaN).
// EXACT: the correctly rounded reciprocal; else the hardware's, within an ulp, which moves
// only values next to a rounding border.
template <bool EXACT>
__device__ __forceinline__ void row_scale(float amax, float& s, float& inv) {
  if (!(amax <= 3.402823466e38f)) {
    s = inv = __uint_as_float(0x7fffffffu);
  } else if (amax < kTiny) {
    s = inv = 0.f;
  } else {
    s = amax * (1.f / 448.f);
    inv = EXACT ? 1.f / s : rcp_approx(s);
  }
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

// Factors of one state row.
struct RowCoef {
  float bp, bc, cc, as;  // beta Bbar_prev, gamma Bbar, Cbar, alpha s
};

// N = 128, P = 64: W warps share a (b, h); a lane owns 16 columns (lane % 4) of the rows
// lane / 4 + 8 k, sixteen codes a load, so a warp's load is 512 contiguous bytes and every
// row is complete in four lanes.
template <typename T, int W>
__global__ void __launch_bounds__(128, 4) step_q8_n128p64(StepQ8Args a) {
  constexpr int kGroups = 4 / W;       // (b, h) a CTA
  constexpr int kK = 16 / W;           // rows a lane
  __shared__ RowCoef coef[kGroups][kN];
  __shared__ float ysum[kGroups][W == 1 ? 1 : W][kP];
  const int lane = threadIdx.x & 31, grp = threadIdx.x / (32 * W), t = threadIdx.x % (32 * W);
  const int warp = t >> 5;  // within the group
  const int64_t bh = (int64_t)blockIdx.x * kGroups + grp;
  if (kGroups > 1 && bh >= a.b * a.H) return;
  auto sync = [&]() {
    if (W == 1)
      __syncwarp();
    else if (W == 4)
      __syncthreads();
    else
      asm volatile("bar.sync %0, %1;" ::"r"(grp + 1), "n"(32 * W) : "memory");
  };
  const int64_t b = bh / a.H, h = bh % a.H, rep = a.H / a.G, g = h / rep;
  const int q = lane & 3, r0 = warp * (kN / W) + (lane >> 2);

  const uint4* S = reinterpret_cast<const uint4*>(a.ssm + bh * kN * kP);
  uint4 hv[kK];
#pragma unroll
  for (int k = 0; k < kK; ++k) hv[k] = S[(r0 + 8 * k) * (kP / 16) + q];
  const T* xt = static_cast<const T*>(a.x_t) + bh * kP;
  float x[16], xp[16];
  load16(xt + 16 * q, x);
  load16(a.x_prev + bh * kP + 16 * q, xp);

  const float alpha = expf(a.logdecay_t[bh]);
  const float be = a.beta_t ? a.beta_t[bh] : 0.f, ga = a.gamma_t[bh];
  const T* Bt = static_cast<const T*>(a.B_t) + (b * a.G + g) * kN;
  const T* Ct = static_cast<const T*>(a.C_t) + (b * a.G + g) * kN;
  const float* bprev = a.b_prev + (b * a.G + g) * kN;
  const bool copy_b = a.b_prev_out && h % rep == 0;
  // the factors of the rows 2 i and 2 i + 1 that turn with the new angle, and with the old
  auto turned_new = [&](int i, float ph) {
    float s, c;
    sincosf(ph, &s, &c);
    const float b0 = to_f32(Bt[2 * i]), b1 = to_f32(Bt[2 * i + 1]);
    const float2 rb = rot2(c, s, b0, b1);
    const float2 rc = rot2(c, s, to_f32(Ct[2 * i]), to_f32(Ct[2 * i + 1]));
    coef[grp][2 * i].bc = ga * rb.x;
    coef[grp][2 * i + 1].bc = ga * rb.y;
    coef[grp][2 * i].cc = rc.x;
    coef[grp][2 * i + 1].cc = rc.y;
    if (copy_b)
      *reinterpret_cast<float2*>(a.b_prev_out + (b * a.G + g) * kN + 2 * i) = make_float2(b0, b1);
  };
  auto turned_old = [&](int i, float ang) {
    float s, c;
    sincosf(ang, &s, &c);
    const float2 rp = rot2(c, s, bprev[2 * i], bprev[2 * i + 1]);
    const float2 sc = *reinterpret_cast<const float2*>(a.scale + bh * kN + 2 * i);
    coef[grp][2 * i].bp = be * rp.x;
    coef[grp][2 * i + 1].bp = be * rp.y;
    coef[grp][2 * i].as = alpha * sc.x;
    coef[grp][2 * i + 1].as = alpha * sc.y;
  };
  float ph = 0.f;  // W = 4: phi' of pair t % 64
  if (W <= 2) {
#pragma unroll
    for (int i = t; i < kN / 2; i += 32 * W) {
      const float ang = a.angle[bh * 64 + i];
      const float p = wrap_angle(ang + (a.theta_t ? a.theta_t[bh * 64 + i] : 0.f));
      turned_new(i, p);
      turned_old(i, ang);
      a.angle_out[bh * 64 + i] = p;
    }
  } else {  // a thread a pair and angle
    const int i = t & 63;
    const float ang = a.angle[bh * 64 + i];
    if (t < 64) {
      ph = wrap_angle(ang + (a.theta_t ? a.theta_t[bh * 64 + i] : 0.f));
      turned_new(i, ph);
    } else {
      turned_old(i, ang);
    }
  }
  sync();

  uint64_t x2[8], xp2[8], acc[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    x2[j] = pack2(x[2 * j], x[2 * j + 1]);
    xp2[j] = pack2(xp[2 * j], xp[2 * j + 1]);
    acc[j] = 0;
  }
  uint4* So = reinterpret_cast<uint4*>(a.ssm_out + bh * kN * kP);
#pragma unroll
  for (int k = 0; k < kK; ++k) {
    const int n = r0 + 8 * k;
    const float4 f = *reinterpret_cast<const float4*>(&coef[grp][n]);
    const uint64_t bp = pack2(f.x, f.x), bc = pack2(f.y, f.y), cc = pack2(f.z, f.z),
                   as = pack2(f.w, f.w);
    const uint32_t c4[4] = {hv[k].x, hv[k].y, hv[k].z, hv[k].w};
    uint64_t v[8];
    float amax = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 c = mx::unpack2_e4m3(c4[j >> 1] >> (16 * (j & 1)));
      v[j] = fma2(bc, x2[j], fma2(bp, xp2[j], mul2(as, pack2(c.x, c.y))));
      acc[j] = fma2(cc, v[j], acc[j]);
      const float2 u = unpack2(v[j]);
      amax = mx::max3_abs(amax, u.x, u.y);
    }
    amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    float s, inv;
    row_scale<false>(amax, s, inv);
    const uint64_t inv2 = pack2(inv, inv);
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 u = unpack2(mul2(v[2 * j], inv2)), w = unpack2(mul2(v[2 * j + 1], inv2));
      o[j] = mx::pack4_e4m3(u.x, u.y, w.x, w.y);
    }
    So[n * (kP / 16) + q] = make_uint4(o[0], o[1], o[2], o[3]);
    if (q == 0) a.scale_out[bh * kN + n] = s;
  }
  // y: lanes with equal q hold sums of the same 16 columns; each exchange halves what a
  // lane keeps, until it has two columns of the warp's sum
  float y8[16];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 u = unpack2(acc[j]);
    y8[2 * j] = u.x;
    y8[2 * j + 1] = u.y;
  }
  int col = 16 * q;
#pragma unroll
  for (int w = 8, bit = 16; w >= 2; w >>= 1, bit >>= 1) {
    const bool up = lane & bit;
#pragma unroll
    for (int j = 0; j < w; ++j) {
      const float send = up ? y8[j] : y8[j + w], keep = up ? y8[j + w] : y8[j];
      y8[j] = keep + __shfl_xor_sync(0xffffffffu, send, bit);
    }
    col += up ? w : 0;
  }
  if (W > 1) {
    ysum[grp][warp][col] = y8[0];
    ysum[grp][warp][col + 1] = y8[1];
    sync();
    if (t >= 64) return;
    if (W == 4) a.angle_out[bh * 64 + t] = ph;  // every old angle was read before the barriers
    col = t;
    float y = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) y += ysum[grp][w][col];
    const float xv = to_f32(xt[col]);
    if (a.D) y = fmaf(a.D[h], xv, y);
    static_cast<T*>(a.y_t)[bh * kP + col] = from_f32<T>(y);
    a.x_prev_out[bh * kP + col] = xv;
    return;
  }
  __syncwarp();  // every lane has read x_prev
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const float xv = to_f32(xt[col + j]);
    float y = y8[j];
    if (a.D) y = fmaf(a.D[h], xv, y);
    static_cast<T*>(a.y_t)[bh * kP + col + j] = from_f32<T>(y);
    a.x_prev_out[bh * kP + col + j] = xv;
  }
}

// Every other shape: one CTA a (b, h), a warp a row at a time, up to eight columns a lane.
constexpr int kGenThreads = 256, kGenWarps = kGenThreads / 32;
template <typename T>
__global__ void __launch_bounds__(kGenThreads) step_q8_kernel(StepQ8Args a) {
  extern __shared__ float smem[];
  const int N = (int)a.N, P = (int)a.P, NH = N / 2;
  const int64_t bh = blockIdx.x, b = bh / a.H, h = bh % a.H, rep = a.H / a.G, g = h / rep;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float* bc = smem;            // N   gamma Bbar
  float* cc = bc + N;          // N   Cbar
  float* bp = cc + N;          // N   beta Bbar_prev
  float* ysum = bp + N;        // kGenWarps * P
  const T* Bt = static_cast<const T*>(a.B_t) + (b * a.G + g) * N;
  const T* Ct = static_cast<const T*>(a.C_t) + (b * a.G + g) * N;
  const float* bprev = a.b_prev + (b * a.G + g) * N;
  const float alpha = expf(a.logdecay_t[bh]);
  const float be = a.beta_t ? a.beta_t[bh] : 0.f, ga = a.gamma_t[bh];
  for (int i = tid; i < NH; i += kGenThreads) {
    const float ang = a.angle[bh * NH + i];
    const float ph = wrap_angle(ang + (a.theta_t ? a.theta_t[bh * NH + i] : 0.f));
    float s, c, s0, c0;
    sincosf(ph, &s, &c);
    sincosf(ang, &s0, &c0);
    const float b0 = to_f32(Bt[2 * i]), b1 = to_f32(Bt[2 * i + 1]);
    const float2 rb = rot2(c, s, b0, b1);
    const float2 rc = rot2(c, s, to_f32(Ct[2 * i]), to_f32(Ct[2 * i + 1]));
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
  const T* xt = static_cast<const T*>(a.x_t) + bh * P;
  float x[8], xp[8], acc[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int p = lane + 32 * j;
    x[j] = p < P ? to_f32(xt[p]) : 0.f;
    xp[j] = p < P ? a.x_prev[bh * P + p] : 0.f;
    acc[j] = 0.f;
  }
  __syncthreads();
  for (int n = warp; n < N; n += kGenWarps) {
    const uint8_t* S = a.ssm + (bh * N + n) * P;
    uint8_t* So = a.ssm_out + (bh * N + n) * P;
    const float as = alpha * a.scale[bh * N + n], f0 = bp[n], f1 = bc[n], f2 = cc[n];
    float v[8], amax = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int p = lane + 32 * j;
      v[j] = 0.f;
      if (p < P) {
        v[j] = fmaf(f1, x[j], fmaf(f0, xp[j], as * mx::unpack2_e4m3(S[p]).x));
        acc[j] = fmaf(f2, v[j], acc[j]);
      }
      amax = max_nan(amax, fabsf(v[j]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    float s, inv;
    row_scale<false>(amax, s, inv);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int p = lane + 32 * j;
      if (p < P) So[p] = (uint8_t)mx::pack2_e4m3(v[j] * inv, 0.f);
    }
    __syncwarp();  // every lane has read the row's scale
    if (lane == 0) a.scale_out[bh * N + n] = s;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (lane + 32 * j < P) ysum[warp * P + lane + 32 * j] = acc[j];
  __syncthreads();
  for (int p = tid; p < P; p += kGenThreads) {
    const float xv = to_f32(xt[p]);
    float y = a.D ? a.D[h] * xv : 0.f;
    for (int w = 0; w < kGenWarps; ++w) y += ysum[w * P + p];
    static_cast<T*>(a.y_t)[bh * P + p] = from_f32<T>(y);
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
                        reinterpret_cast<uintptr_t>(a.scale) | reinterpret_cast<uintptr_t>(bprev);
  if (a.N == kN && a.P == kP && all % 16 == 0) {
    const int sms = current_device_sms();
    if (nbh <= 2 * (int64_t)sms)
      step_q8_n128p64<T, 4><<<(unsigned)nbh, 128, 0, s>>>(a);
    else
      step_q8_n128p64<T, 2><<<(unsigned)((nbh + 1) / 2), 128, 0, s>>>(a);
  } else {
    const size_t smem = sizeof(float) * (size_t)(3 * a.N + kGenWarps * a.P);
    step_q8_kernel<T><<<(unsigned)nbh, kGenThreads, smem, s>>>(a);
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
cudaError_t launch_quant_state(int64_t rows, int64_t P, const float* h, void* codes, float* scale,
                               cudaStream_t s) {
  return launch_state(true, rows, P, const_cast<float*>(h), codes, scale, s);
}
cudaError_t launch_dequant_state(int64_t rows, int64_t P, const void* codes, const float* scale,
                                 float* h, cudaStream_t s) {
  return launch_state(false, rows, P, h, const_cast<void*>(codes), const_cast<float*>(scale), s);
}

}  // namespace m3ssd
