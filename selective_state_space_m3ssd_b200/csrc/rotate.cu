// The root-mean-square norm of every head of queries and keys (the scan's C and B) with the
// rotation by position in the same pass, and its backward.
//
//     rstd = 1 / sqrt(mean u^2 + eps),  v = u rstd w,  pair i of the output: R(pos f_i) (pair i of v),
// and back, with dv = R(-pos f_i) d and g = w dv, uh = u rstd (means over the head's N values):
//     du = rstd (g - uh mean(g uh)),   dw = sum over tokens and heads of dv uh.
//
// Streams: every tensor is read once and written once, so HBM bounds them.  A head's N values lie
// eight a lane on the least power of two of lanes that holds them, so that a warp takes 32 / lanes
// heads at once and a mean is a few shuffles.  A warp takes a block of one token's heads, the
// queries', then the keys', so the angles' sines and cosines are worked out once for all of
// them: in turns, pos f / (2 pi), in fp64, of which the whole turns are dropped before
// anything is rounded to fp32, so a far position keeps its angle to 2^-25 of a turn.
#include <cuda_runtime.h>

#include <cstdint>
#include <initializer_list>

#include "common.cuh"
#include "internal.h"
#include "mx.cuh"

namespace m3ssd {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

// How a lane's eight values lie in a head: as one access; as four pairs, the head's lanes apart; or as
// those pairs element by element (rows that are not aligned for either).
enum Access { kWide, kPairs, kSingle };

// A lane's place: lane l of the `lanes` of a head, which is number `sub` of the warp's.
struct Place {
  int lanes, l, sub, per;  // per: heads a warp takes at once
  __device__ __forceinline__ explicit Place(int lanes_) : lanes(lanes_) {
    const int lane = threadIdx.x & 31;
    l = lane & (lanes - 1);
    sub = lane / lanes;
    per = 32 / lanes;
  }
  // First element of the lane's pair p.
  template <int ACC>
  __device__ __forceinline__ int at(int p) const {
    return ACC == kWide ? 8 * l + 2 * p : 2 * (p * lanes + l);
  }
};

template <typename T>
struct Raw;
template <>
struct Raw<float> {
  float f[8];
};
template <>
struct Raw<__nv_bfloat16> {
  uint32_t u[4];
};

template <int ACC>
__device__ __forceinline__ void load(const float* head, const Place& pl, int N, bool on, Raw<float>& r) {
#pragma unroll
  for (int j = 0; j < 8; ++j) r.f[j] = 0.f;
  if constexpr (ACC == kWide) {
    if (on && 8 * pl.l < N) mx::load8(head + 8 * pl.l, r.f);
  } else {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int e = pl.at<ACC>(p);
      if (on && e < N) {
        if constexpr (ACC == kPairs) {
          const float2 v = *reinterpret_cast<const float2*>(head + e);
          r.f[2 * p] = v.x;
          r.f[2 * p + 1] = v.y;
        } else {
          r.f[2 * p] = head[e];
          r.f[2 * p + 1] = head[e + 1];
        }
      }
    }
  }
}
template <int ACC>
__device__ __forceinline__ void load(const __nv_bfloat16* head, const Place& pl, int N, bool on,
                                     Raw<__nv_bfloat16>& r) {
#pragma unroll
  for (int j = 0; j < 4; ++j) r.u[j] = 0;
  if constexpr (ACC == kWide) {
    if (on && 8 * pl.l < N) {
      const uint4 w = *reinterpret_cast<const uint4*>(head + 8 * pl.l);
      r.u[0] = w.x;
      r.u[1] = w.y;
      r.u[2] = w.z;
      r.u[3] = w.w;
    }
  } else {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int e = pl.at<ACC>(p);
      if (on && e < N) {
        if constexpr (ACC == kPairs) {
          r.u[p] = *reinterpret_cast<const uint32_t*>(head + e);
        } else {
          const uint16_t* s = reinterpret_cast<const uint16_t*>(head + e);
          r.u[p] = (uint32_t)s[0] | (uint32_t)s[1] << 16;
        }
      }
    }
  }
}
__device__ __forceinline__ void unpack(const Raw<float>& r, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = r.f[j];
}
__device__ __forceinline__ void unpack(const Raw<__nv_bfloat16>& r, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(r.u[j] << 16);
    v[2 * j + 1] = __uint_as_float(r.u[j] & 0xffff0000u);
  }
}
template <int ACC, typename T>
__device__ __forceinline__ void store(T* head, const Place& pl, int N, const float (&v)[8]) {
  if constexpr (ACC == kWide) {
    if (8 * pl.l < N) mx::store8(head + 8 * pl.l, v);
  } else {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int e = pl.at<ACC>(p);
      if (e < N) {
        if constexpr (ACC == kSingle) {
          head[e] = from_f32<T>(v[2 * p]);
          head[e + 1] = from_f32<T>(v[2 * p + 1]);
        } else if constexpr (sizeof(T) == 2) {
          *reinterpret_cast<__nv_bfloat162*>(head + e) = __floats2bfloat162_rn(v[2 * p], v[2 * p + 1]);
        } else {
          *reinterpret_cast<float2*>(head + e) = make_float2(v[2 * p], v[2 * p + 1]);
        }
      }
    }
  }
}

// Sum over a head's lanes, in each of them.
__device__ __forceinline__ float head_sum(float v, int lanes) {
  for (int o = 1; o < lanes; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A lane's columns of the weights (zeros past the head's end).
template <int ACC>
__device__ __forceinline__ void load_weight(const float* w, const Place& pl, int N, float (&o)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int e = pl.at<ACC>(j / 2) + (j & 1);
    o[j] = e < N ? (w ? w[e] : 1.f) : 0.f;
  }
}
// Turns a position of a lane's pairs, and the cosines and sines of a position.
template <int ACC>
__device__ __forceinline__ void load_freqs(const float* f, const Place& pl, int R, double (&o)[4]) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int i = pl.at<ACC>(p) / 2;
    o[p] = i < R ? (double)f[i] * 0.15915494309189533577 : 0.0;
  }
}
__device__ __forceinline__ void turn(int pos, const double (&f)[4], float (&c)[4], float (&s)[4]) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const double t = (double)pos * f[p];
    sincospif(2.f * (float)(t - rint(t)), &s[p], &c[p]);
  }
}

// Which heads a warp takes: blocks of `block` of a token's heads, queries and keys in a row.
struct Unit {
  int64_t row;
  int lo, hi;
};
__device__ __forceinline__ Unit unit_of(int64_t unit, int blocks, int block, int heads) {
  Unit u;
  u.row = blocks == 1 ? unit : unit / blocks;
  u.lo = blocks == 1 ? 0 : (int)(unit % blocks) * block;
  u.hi = min(u.lo + block, heads);
  return u;
}

// Heads in flight a warp and lane.
template <typename T>
constexpr int kAhead = sizeof(T) == 2 ? 4 : 2;

// The forward of heads lo to hi - 1 of one tensor's row.
template <typename T, int ACC>
__device__ __forceinline__ void forward(const T* in, T* out, int lo, int hi, int N, float inv_n, float eps,
                                        const Place& pl, const float (&w)[8], const float (&c)[4],
                                        const float (&s)[4]) {
  constexpr int A = kAhead<T>;
  for (int h0 = lo; h0 < hi; h0 += A * pl.per) {
    Raw<T> raw[A];
#pragma unroll
    for (int k = 0; k < A; ++k) {
      const int h = h0 + k * pl.per + pl.sub;
      load<ACC>(in + (int64_t)h * N, pl, N, h < hi, raw[k]);
    }
#pragma unroll
    for (int k = 0; k < A; ++k) {
      if (h0 + k * pl.per >= hi) break;
      const int h = h0 + k * pl.per + pl.sub;
      float v[8], ss = 0.f;
      unpack(raw[k], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(v[j], v[j], ss);
      const float rstd = 1.f / sqrtf(fmaf(head_sum(ss, pl.lanes), inv_n, eps));
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const float2 o = rot2(c[p], s[p], v[2 * p] * rstd * w[2 * p], v[2 * p + 1] * rstd * w[2 * p + 1]);
        v[2 * p] = o.x;
        v[2 * p + 1] = o.y;
      }
      if (h < hi) store<ACC>(out + (int64_t)h * N, pl, N, v);
    }
  }
}

template <typename T, int ACC>
__global__ void __launch_bounds__(kThreads, 3) norm_rotate_kernel(RotateArgs a) {
  const Place pl(a.lanes);
  const int N = (int)a.N, Hq = (int)a.Hq, heads = (int)(a.Hq + a.Hk);
  const float inv_n = 1.f / (float)N;
  float wq[8], wk[8];
  double f[4];
  load_weight<ACC>(a.q_w, pl, N, wq);
  load_weight<ACC>(a.k_w, pl, N, wk);
  load_freqs<ACC>(a.freqs, pl, (int)a.R, f);
  for (int64_t i = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); i < a.rows * a.blocks;
       i += (int64_t)gridDim.x * kWarps) {
    const Unit u = unit_of(i, a.blocks, a.block, heads);
    float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
    if (a.R > 0) turn(a.positions[u.row], f, c, s);
    forward<T, ACC>(static_cast<const T*>(a.q) + u.row * a.ldq,
                    static_cast<T*>(a.q_out) + u.row * a.Hq * N, u.lo, min(u.hi, Hq), N, inv_n, a.eps, pl,
                    wq, c, s);
    forward<T, ACC>(static_cast<const T*>(a.k) + u.row * a.ldk,
                    static_cast<T*>(a.k_out) + u.row * a.Hk * N, max(u.lo - Hq, 0), u.hi - Hq, N, inv_n,
                    a.eps, pl, wk, c, s);
  }
}

template <typename T, typename U, typename G, int ACC>
__device__ __forceinline__ void backward(const T* in, const U* up, G* out, int lo, int hi, int N,
                                         float inv_n, float eps, const Place& pl, const float (&w)[8],
                                         const float (&c)[4], const float (&s)[4], float (&dw)[8]) {
  constexpr int A = kAhead<U> / 2;
  for (int h0 = lo; h0 < hi; h0 += A * pl.per) {
    Raw<T> raw[A];
    Raw<U> rup[A];
#pragma unroll
    for (int k = 0; k < A; ++k) {
      const int h = h0 + k * pl.per + pl.sub;
      load<ACC>(in + (int64_t)h * N, pl, N, h < hi, raw[k]);
      load<ACC>(up + (int64_t)h * N, pl, N, h < hi, rup[k]);
    }
#pragma unroll
    for (int k = 0; k < A; ++k) {
      if (h0 + k * pl.per >= hi) break;
      const int h = h0 + k * pl.per + pl.sub;
      float v[8], d[8], ss = 0.f, gs = 0.f;
      unpack(raw[k], v);
      unpack(rup[k], d);
#pragma unroll
      for (int p = 0; p < 4; ++p) {  // dv: turned back
        const float2 o = rot2(c[p], -s[p], d[2 * p], d[2 * p + 1]);
        d[2 * p] = o.x;
        d[2 * p + 1] = o.y;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        ss = fmaf(v[j], v[j], ss);
        gs = fmaf(d[j] * w[j], v[j], gs);
      }
      const float rstd = 1.f / sqrtf(fmaf(head_sum(ss, pl.lanes), inv_n, eps));
      const float m = head_sum(gs, pl.lanes) * rstd * inv_n;  // mean(g uh)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float uh = v[j] * rstd;
        if (h < hi) dw[j] = fmaf(d[j], uh, dw[j]);
        v[j] = rstd * (d[j] * w[j] - uh * m);
      }
      if (h < hi) store<ACC>(out + (int64_t)h * N, pl, N, v);
    }
  }
}

template <typename T, typename U, typename G, int ACC>
__global__ void __launch_bounds__(kThreads, 2) norm_rotate_bwd_kernel(RotateBwdArgs args) {
  __shared__ float red[kWarps][2][256];
  cudaTriggerProgrammaticLaunchCompletion();  // the sums' kernel waits itself
  const RotateArgs& a = args.f;
  const Place pl(a.lanes);
  const int N = (int)a.N, Hq = (int)a.Hq, heads = (int)(a.Hq + a.Hk);
  const float inv_n = 1.f / (float)N;
  float wq[8], wk[8], dwq[8], dwk[8];
  double f[4];
  load_weight<ACC>(a.q_w, pl, N, wq);
  load_weight<ACC>(a.k_w, pl, N, wk);
  load_freqs<ACC>(a.freqs, pl, (int)a.R, f);
#pragma unroll
  for (int j = 0; j < 8; ++j) dwq[j] = dwk[j] = 0.f;
  for (int64_t i = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); i < a.rows * a.blocks;
       i += (int64_t)gridDim.x * kWarps) {
    const Unit u = unit_of(i, a.blocks, a.block, heads);
    float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
    if (a.R > 0) turn(a.positions[u.row], f, c, s);
    backward<T, U, G, ACC>(static_cast<const T*>(a.q) + u.row * a.ldq,
                           static_cast<const U*>(args.dq_out) + u.row * a.Hq * N,
                           static_cast<G*>(args.dq) + u.row * args.ldgq, u.lo, min(u.hi, Hq), N, inv_n,
                           a.eps, pl, wq, c, s, dwq);
    backward<T, U, G, ACC>(static_cast<const T*>(a.k) + u.row * a.ldk,
                           static_cast<const U*>(args.dk_out) + u.row * a.Hk * N,
                           static_cast<G*>(args.dk) + u.row * args.ldgk, max(u.lo - Hq, 0), u.hi - Hq, N,
                           inv_n, a.eps, pl, wk, c, s, dwk);
  }
  // the CTA's sums of each column: over a warp's heads, then over the warps in order
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    for (int o = pl.lanes; o < 32; o <<= 1) {
      dwq[j] += __shfl_xor_sync(0xffffffffu, dwq[j], o);
      dwk[j] += __shfl_xor_sync(0xffffffffu, dwk[j], o);
    }
    const int e = pl.at<ACC>(j / 2) + (j & 1);
    if (pl.sub == 0 && e < N) {
      red[threadIdx.x >> 5][0][e] = dwq[j];
      red[threadIdx.x >> 5][1][e] = dwk[j];
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < 2 * N; e += kThreads) {
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) t += red[w][e >= N][e >= N ? e - N : e];
    args.part[(int64_t)blockIdx.x * 2 * N + e] = t;
  }
}

// dw of the queries, then of the keys: the CTAs' partial sums in a fixed order, 32 of them a column
// at a time.
__global__ void __launch_bounds__(256) norm_rotate_dw_kernel(const float* part, int parts, int N,
                                                             float* dq_w, float* dk_w) {
  __shared__ float red[32][8];
  const int c = threadIdx.x & 7, p0 = threadIdx.x >> 3, e = blockIdx.x * 8 + c;
  cudaGridDependencySynchronize();  // launched before the backward's end: its sums are there
  float s = 0.f;
  if (e < 2 * N) {
#pragma unroll 4
    for (int p = p0; p < parts; p += 32) s += part[(int64_t)p * 2 * N + e];
  }
  red[p0][c] = s;
  __syncthreads();
  if (threadIdx.x < 8 && e < 2 * N) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += red[i][threadIdx.x];
    if (e < N) {
      if (dq_w) dq_w[e] = t;
    } else if (dk_w) {
      dk_w[e - N] = t;
    }
  }
}

int lanes_of(int64_t N) {
  int n = 1;
  while (8 * n < N) n *= 2;
  return n;
}

// Heads of a block and CTAs: a token's heads together where the tokens alone give every SM's warps
// something to do, else in blocks of what a warp has in flight, down to one warp's worth.
void set_blocks(RotateArgs& a, int64_t ctas_an_sm, int ahead) {
  const int64_t sms = current_device_sms() > 0 ? current_device_sms() : 148;
  const int64_t heads = a.Hq + a.Hk, warps = sms * ctas_an_sm * kWarps;
  a.lanes = lanes_of(a.N);
  const int64_t least = 32 / a.lanes * ahead;
  int64_t blocks = a.rows > 0 ? (warps + a.rows - 1) / a.rows : 1, most = (heads + least - 1) / least;
  if (blocks > most) blocks = most;
  if (blocks < 1) blocks = 1;
  a.block = (int)((heads + blocks - 1) / blocks);
  a.blocks = (int)((heads + a.block - 1) / a.block);
}
unsigned grid_of(const RotateArgs& a, int64_t ctas_an_sm) {
  const int64_t sms = current_device_sms() > 0 ? current_device_sms() : 148;
  const int64_t want = (a.rows * a.blocks + kWarps - 1) / kWarps, most = sms * ctas_an_sm;
  return (unsigned)(want < most ? want : most);
}
constexpr int kFwdCtas = 3, kBwdCtas = 2;

struct Strided {
  const void* p;
  int64_t ld;
  int64_t size;  // of an element
};
// The widest access that heads of N at these addresses allow.
Access access_of(int64_t N, std::initializer_list<Strided> ts) {
  bool wide = N % 8 == 0, pairs = true;
  for (const Strided& t : ts) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(t.p);
    wide &= at % (8 * t.size) == 0 && t.ld % 8 == 0;
    pairs &= at % (2 * t.size) == 0 && t.ld % 2 == 0;
  }
  return wide ? kWide : pairs ? kPairs : kSingle;
}

template <typename T>
cudaError_t fwd_t(const RotateArgs& a, cudaStream_t s) {
  const int64_t z = sizeof(T);
  const unsigned grid = grid_of(a, kFwdCtas);
  switch (access_of(a.N, {{a.q, a.ldq, z}, {a.k, a.ldk, z}, {a.q_out, a.N, z}, {a.k_out, a.N, z}})) {
    case kWide: norm_rotate_kernel<T, kWide><<<grid, kThreads, 0, s>>>(a); break;
    case kPairs: norm_rotate_kernel<T, kPairs><<<grid, kThreads, 0, s>>>(a); break;
    default: norm_rotate_kernel<T, kSingle><<<grid, kThreads, 0, s>>>(a);
  }
  return cudaGetLastError();
}
template <typename T, typename U, typename G>
cudaError_t bwd_t(const RotateBwdArgs& a, unsigned grid, cudaStream_t s) {
  const RotateArgs& f = a.f;
  const int64_t z = sizeof(T), zu = sizeof(U), zg = sizeof(G);
  switch (access_of(f.N, {{f.q, f.ldq, z}, {f.k, f.ldk, z}, {a.dq_out, f.N, zu}, {a.dk_out, f.N, zu},
                          {a.dq, a.ldgq, zg}, {a.dk, a.ldgk, zg}})) {
    case kWide: norm_rotate_bwd_kernel<T, U, G, kWide><<<grid, kThreads, 0, s>>>(a); break;
    case kPairs: norm_rotate_bwd_kernel<T, U, G, kPairs><<<grid, kThreads, 0, s>>>(a); break;
    default: norm_rotate_bwd_kernel<T, U, G, kSingle><<<grid, kThreads, 0, s>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rotate(const RotateArgs& args, cudaStream_t s) {
  if (args.rows == 0) return cudaSuccess;
  RotateArgs a = args;
  set_blocks(a, kFwdCtas, a.bf16 ? kAhead<__nv_bfloat16> : kAhead<float>);
  return a.bf16 ? fwd_t<__nv_bfloat16>(a, s) : fwd_t<float>(a, s);
}

namespace {
void set_bwd_blocks(RotateArgs& a) { set_blocks(a, kBwdCtas, 1); }
}  // namespace

size_t norm_rotate_bwd_workspace_bytes(const RotateArgs& args) {
  if (args.rows == 0) return 0;
  RotateArgs a = args;
  set_bwd_blocks(a);
  return (size_t)grid_of(a, kBwdCtas) * 2 * (size_t)a.N * sizeof(float);
}

cudaError_t launch_norm_rotate_bwd(const RotateBwdArgs& args, cudaStream_t s) {
  RotateBwdArgs a = args;
  unsigned grid = 0;
  if (a.f.rows > 0) {
    set_bwd_blocks(a.f);
    grid = grid_of(a.f, kBwdCtas);
    using b16 = __nv_bfloat16;
    const cudaError_t e = !a.f.bf16 ? bwd_t<float, float, float>(a, grid, s)
                          : a.up_bf16 ? (a.grad_bf16 ? bwd_t<b16, b16, b16>(a, grid, s)
                                                     : bwd_t<b16, b16, float>(a, grid, s))
                                      : (a.grad_bf16 ? bwd_t<b16, float, b16>(a, grid, s)
                                                     : bwd_t<b16, float, float>(a, grid, s));
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute early[1];
  early[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((2 * a.f.N + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cfg.attrs = early;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, norm_rotate_dw_kernel, (const float*)a.part, (int)grid,
                                           (int)a.f.N, a.dq_w, a.dk_w);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace m3ssd
