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
// anything is rounded to fp32, so up to 2^25 turns away a position keeps its angle to 2^-25 of a turn
// (further on fp64's own rounding adds up, 2^-51 of the turns at most).  What a warp reads
// comes through a ring of its own in shared memory, copied ahead.  32768 tokens of 40 heads of 128
// in bf16 take 110 us forward (0.93 of HBM's copy rate) and 186 backward (0.83).
#include <cuda_runtime.h>

#include <cstdint>
#include <initializer_list>

#include "common.cuh"
#include "internal.h"
#include "mx.cuh"

namespace m3ssd {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

// How a lane's eight values lie in a head: as one piece of eight (16 bytes, where all tensors are
// bf16), as two of four (so that fp32 lanes read 16 bytes each next to one another) or as four pairs, the
// head's lanes apart; or as those pairs element by element (rows that are not aligned for them).
enum Access { kWide, kQuads, kPairs, kSingle };
template <int ACC>
constexpr int kPiece = ACC == kWide ? 8 : ACC == kQuads ? 4 : 2;

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
    constexpr int P = kPiece<ACC>;
    return P * (2 * p / P * lanes + l) + 2 * p % P;
  }
  // Where its first lies from the first of the warp's heads.
  template <int ACC>
  __device__ __forceinline__ int offset(int N) const {
    return sub * N + at<ACC>(0);
  }
};

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src));
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES));
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 splat(float v) { return make_float2(v, v); }

// A lane's eight values of a head as a slot of the warp's ring holds them: in 16-byte pieces, a
// warp's together.  Each lane copies what it reads itself.  Pointers are to the lane's first
// element; `n` is how many elements there are from it on (its pieces lie `apart` elements apart).
// What is not there is never copied: it stays zero (clear()) in a head's lanes, and is whatever it was in
// lanes without a head, whose values go nowhere.
template <typename T>
struct Slot {
  static constexpr int kBytes = 32 * 8 * (int)sizeof(T);
  // Where pair j is from the lane's place.
  static __device__ __forceinline__ constexpr int pair_at(int j) {
    return sizeof(T) == 2 ? 4 * j : 512 * (j / 2) + 8 * (j % 2);
  }
  template <int ACC>
  static __device__ __forceinline__ void clear(char* slot, int n, int apart) {
    constexpr int P = kPiece<ACC>;
#pragma unroll
    for (int j = 0; j < 8 / P; ++j)
      if (j * apart >= n) {
#pragma unroll
        for (int i = 0; i < P / 2; ++i) {
          T* const at = reinterpret_cast<T*>(slot + pair_at(j * P / 2 + i));
          at[0] = at[1] = from_f32<T>(0.f);
        }
      }
  }
  // `slot` and its address; on: the lane has a head.
  template <int ACC>
  static __device__ __forceinline__ void fetch(char* slot, uint32_t addr, const T* p, int n, int apart,
                                               bool on) {
    constexpr int P = kPiece<ACC>, bytes = P * (int)sizeof(T);
    static_assert(bytes <= 16, "a piece is one copy");
#pragma unroll
    for (int j = 0; j < 8 / P; ++j)
      if (on && j * apart < n) {
        if constexpr (ACC == kSingle) {
          T* const at = reinterpret_cast<T*>(slot + pair_at(j));
          at[0] = p[j * apart];
          at[1] = p[j * apart + 1];
        } else {
          copy_async<bytes>(addr + pair_at(j * P / 2), p + j * apart);
        }
      }
  }
  static __device__ __forceinline__ void read(const char* slot, float2 (&v)[4]) {
    if constexpr (sizeof(T) == 2) {
      const uint4 u = *reinterpret_cast<const uint4*>(slot);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[j] = make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u));
    } else {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float4 f = *reinterpret_cast<const float4*>(slot + 512 * q);
        v[2 * q] = make_float2(f.x, f.y);
        v[2 * q + 1] = make_float2(f.z, f.w);
      }
    }
  }
};

template <int ACC, typename T>
__device__ __forceinline__ void store(T* p, int n, int apart, bool on, const float2 (&v)[4]) {
  constexpr int P = kPiece<ACC>;
#pragma unroll
  for (int j = 0; j < 8 / P; ++j) {
    if (on && j * apart < n) {
      T* const at = p + j * apart;
      if constexpr (ACC == kSingle) {
        at[0] = from_f32<T>(v[j].x);
        at[1] = from_f32<T>(v[j].y);
      } else if constexpr (sizeof(T) == 2) {
        uint32_t u[P / 2];
#pragma unroll
        for (int i = 0; i < P / 2; ++i) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(v[j * P / 2 + i].x, v[j * P / 2 + i].y);
          u[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        if constexpr (P == 8)
          *reinterpret_cast<uint4*>(at) = make_uint4(u[0], u[1], u[2], u[3]);
        else if constexpr (P == 4)
          *reinterpret_cast<uint2*>(at) = make_uint2(u[0], u[1]);
        else
          *reinterpret_cast<uint32_t*>(at) = u[0];
      } else if constexpr (P == 4) {
        *reinterpret_cast<float4*>(at) =
            make_float4(v[2 * j].x, v[2 * j].y, v[2 * j + 1].x, v[2 * j + 1].y);
      } else {
        *reinterpret_cast<float2*>(at) = v[j];
      }
    }
  }
}

// Sum over a head's lanes, in each of them.
__device__ __forceinline__ float head_sum(float v, int lanes) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
    if (o < lanes) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// 1 / sqrt(v), v >= 0: the hardware's approximation and a step of Newton's; infinite at zero.
__device__ __forceinline__ float rsqrt_of(float v) {
  const float y = rsqrtf(v), e = fmaf(-v * y, y, 1.f);
  return e == e ? fmaf(0.5f * y, e, y) : y;  // not at 0 and infinity
}

// A lane's columns of the weights (zeros past the head's end).
template <int ACC>
__device__ __forceinline__ void load_weight(const float* w, const Place& pl, int N, float2 (&o)[4]) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int e = pl.at<ACC>(p);
    o[p] = e >= N ? splat(0.f) : w ? make_float2(w[e], w[e + 1]) : splat(1.f);
  }
}
// Turns a position of a lane's pairs, and the cosines and sines of a position: for the forward's bf16 outputs
// by the hardware's approximations on half a turn either side (2^-21), far below those outputs' steps.  Not in
// the backward, whose dw is fp32 whatever the type of dq (with bf16 dq the approximations took 182.9 instead
// of 185.6 us for 32768 tokens of 40 heads of 128, 37.8 instead of 41.0 for 1 + 1 heads).
template <int ACC>
__device__ __forceinline__ void load_freqs(const float* f, const Place& pl, int R, double (&o)[4]) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int i = pl.at<ACC>(p) / 2;
    o[p] = i < R ? (double)f[i] * 0.15915494309189533577 : 0.0;
  }
}
template <bool APPROX>
__device__ __forceinline__ void turn(int pos, const double (&f)[4], float (&c)[4], float (&s)[4]) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const double t = (double)pos * f[p];
    const float part = (float)(t - rint(t));
    if constexpr (APPROX)
      __sincosf(part * 6.28318530717958648f, &s[p], &c[p]);
    else
      sincospif(2.f * part, &s[p], &c[p]);
  }
}

// A warp's way through its units, a block of a token's slots each (a slot holds `per` heads, the
// queries' slots come first): runs of slots of one token and tensor.
struct Way {
  int unit, total, row;
  int first, left, end;  // the run's first slot in its tensor and the slots left; the unit's end
  bool keys;
  __device__ __forceinline__ explicit Way(const RotateArgs& a) {
    unit = blockIdx.x * kWarps + (threadIdx.x >> 5);
    total = (int)a.rows * a.blocks;  // 31 bits hold the heads of all tokens
    open(a);
  }
  __device__ __forceinline__ void open(const RotateArgs& a) {
    row = a.blocks == 1 ? unit : (int)((uint32_t)unit / (uint32_t)a.blocks);
    first = (unit - row * a.blocks) * a.block;
    end = min(first + a.block, a.slots);
    keys = first >= a.q_slots;
    left = (keys ? end : min(end, a.q_slots)) - first;
    if (keys) first -= a.q_slots;
  }
  __device__ __forceinline__ bool valid() const { return unit < total; }
  __device__ __forceinline__ void next_run(const RotateArgs& a) {
    if (!keys && end > a.q_slots) {
      keys = true;
      first = 0;
      left = end - a.q_slots;
    } else {
      unit += gridDim.x * kWarps;
      open(a);
    }
  }
  // The position of the next row that the warp takes, read while the unit's row is done.  A row of more
  // blocks than there are warps gives a warp several units: those are passed over.
  __device__ __forceinline__ int next_position(const RotateArgs& a) const {
    const int warps = (int)gridDim.x * kWarps, end = (row + 1) * a.blocks;
    int next = unit + warps;
    if (next < end) next += ((end - 1 - next) / warps + 1) * warps;
    if (next >= total || a.R == 0) return 0;
    return a.positions[a.blocks == 1 ? next : (int)((uint32_t)next / (uint32_t)a.blocks)];
  }
  // The slots at the run's end in which the lane has no head (0 or 1).
  __device__ __forceinline__ int missing(const RotateArgs& a, const Place& pl) const {
    const int slots = keys ? a.slots - a.q_slots : a.q_slots, heads = (int)(keys ? a.Hk : a.Hq);
    return first + left == slots && (slots - 1) * pl.per + pl.sub >= heads;
  }
  // The lane's first element of the run in a tensor whose rows are `ld` elements apart.
  template <int ACC, typename P>
  __device__ __forceinline__ P* at(P* q, P* k, int64_t ldq, int64_t ldk, const Place& pl, int N) const {
    return (keys ? k + (int64_t)row * ldk : q + (int64_t)row * ldq) + first * pl.per * N +
           pl.offset<ACC>(N);
  }
};

// Slots in a warp's ring, and CTAs an SM: enough in flight to keep HBM busy, and no more walkers than
// that, as they scatter its reads.  32768 tokens of 40 x 128 bf16 forward: three slots 119 us,
// four 110, six 123 at three CTAs, 138 at four CTAs, 123 at two.
constexpr int kFwdRing = 4, kBwdRing = 4, kFwdCtas = 3, kBwdCtas = 2;

template <typename T, int ACC>
__global__ void __launch_bounds__(kThreads, kFwdCtas) norm_rotate_kernel(RotateArgs a) {
  extern __shared__ __align__(16) char smem[];
  constexpr int kSlot = Slot<T>::kBytes, kRing = kFwdRing * kSlot;
  char* const ring = smem + (threadIdx.x >> 5) * kRing + (threadIdx.x & 31) * 16;
  const uint32_t ring_addr = (uint32_t)__cvta_generic_to_shared(ring);
  const Place pl(a.lanes);
  const int N = (int)a.N, n = N - pl.at<ACC>(0), apart = kPiece<ACC> * pl.lanes, stride = pl.per * N;
  const float inv_n = 1.f / (float)N;
  const T *const q = static_cast<const T*>(a.q), *const k = static_cast<const T*>(a.k);
  float2 wq[4], wk[4];
  float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
  double f[4];
  load_weight<ACC>(a.q_w, pl, N, wq);
  load_weight<ACC>(a.k_w, pl, N, wk);
  load_freqs<ACC>(a.freqs, pl, (int)a.R, f);
  Way in(a), out = in;
  int pos = in.valid() && a.R > 0 ? a.positions[in.row] : 0;
  const T* from = nullptr;
  int missing = 0, in_left = 0;  // 0: nothing more to copy
  auto open = [&] {
    if (in.valid()) {
      from = in.at<ACC>(q, k, a.ldq, a.ldk, pl, N);
      missing = in.missing(a, pl);
      in_left = in.left;
    }
  };
  auto fetch = [&](int slot) {
    if (in_left > 0) {
      Slot<T>::template fetch<ACC>(ring + slot, ring_addr + slot, from, n, apart, in_left > missing);
      from += stride;
      if (--in_left == 0) {
        in.next_run(a);
        open();
      }
    }
    copies_end();
  };
#pragma unroll
  for (int i = 0; i < kFwdRing; ++i) Slot<T>::template clear<ACC>(ring + i * kSlot, n, apart);
  open();
#pragma unroll
  for (int i = 0; i < kFwdRing - 1; ++i) fetch(i * kSlot);
  int slot = 0, before = kRing - kSlot;
  auto run = [&](const float2(&w)[4]) {
    T* to = out.at<ACC>(static_cast<T*>(a.q_out), static_cast<T*>(a.k_out), a.Hq * N, a.Hk * N, pl, N);
    const int none = out.missing(a, pl);
    for (int left = out.left; left > 0; --left) {
      copies_wait<kFwdRing - 2>();
      fetch(before);
      float2 v[4];
      Slot<T>::read(ring + slot, v);
      before = slot;
      slot = slot == kRing - kSlot ? 0 : slot + kSlot;
      float2 ss = mul2(v[0], v[0]);
#pragma unroll
      for (int p = 1; p < 4; ++p) ss = fma2(v[p], v[p], ss);
      const float2 rstd = splat(rsqrt_of(fmaf(head_sum(ss.x + ss.y, pl.lanes), inv_n, a.eps)));
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        v[p] = mul2(mul2(v[p], rstd), w[p]);
        v[p] = rot2(c[p], s[p], v[p].x, v[p].y);
      }
      store<ACC>(to, n, apart, left > none, v);
      to += stride;
    }
  };
  int at = -1;  // the row that c and s are of
  while (out.valid()) {
    if (at != out.row) {
      at = out.row;
      if (a.R > 0) turn<sizeof(T) == 2>(pos, f, c, s);
      pos = out.next_position(a);
    }
    if (out.keys)
      run(wk);
    else
      run(wq);
    out.next_run(a);
  }
}

// The backward of one head.
template <int ACC, typename G>
__device__ __forceinline__ void backward(float2 (&v)[4], float2 (&d)[4], bool on, G* out, int n, int apart,
                                         float inv_n, float eps, int lanes, const float2 (&w)[4],
                                         const float (&c)[4], const float (&s)[4], float2 (&dw)[4]) {
  float2 ss = splat(0.f), gs = ss, g[4];
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    d[p] = rot2(c[p], -s[p], d[p].x, d[p].y);  // dv: turned back
    g[p] = mul2(d[p], w[p]);
    ss = fma2(v[p], v[p], ss);
    gs = fma2(g[p], v[p], gs);
  }
  const float rstd = rsqrt_of(fmaf(head_sum(ss.x + ss.y, lanes), inv_n, eps));
  const float m = head_sum(gs.x + gs.y, lanes) * rstd * inv_n;  // mean(g uh)
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const float2 uh = mul2(v[p], splat(rstd));
    if (on) dw[p] = fma2(d[p], uh, dw[p]);
    v[p] = mul2(fma2(uh, splat(-m), g[p]), splat(rstd));
  }
  store<ACC>(out, n, apart, on, v);
}

template <typename T, typename U, typename G, int ACC>
__global__ void __launch_bounds__(kThreads, kBwdCtas) norm_rotate_bwd_kernel(RotateBwdArgs args) {
  extern __shared__ __align__(16) char smem[];
  constexpr int kSlot = Slot<T>::kBytes + Slot<U>::kBytes, kRing = kBwdRing * kSlot;
  cudaTriggerProgrammaticLaunchCompletion();  // the sums' kernel waits itself
  const RotateArgs& a = args.f;
  char* const ring = smem + (threadIdx.x >> 5) * kRing + (threadIdx.x & 31) * 16;
  const uint32_t ring_addr = (uint32_t)__cvta_generic_to_shared(ring);
  const Place pl(a.lanes);
  const int N = (int)a.N, n = N - pl.at<ACC>(0), apart = kPiece<ACC> * pl.lanes, stride = pl.per * N;
  const float inv_n = 1.f / (float)N;
  const T *const q = static_cast<const T*>(a.q), *const k = static_cast<const T*>(a.k);
  const U *const uq = static_cast<const U*>(args.dq_out), *const uk = static_cast<const U*>(args.dk_out);
  float2 wq[4], wk[4], dwq[4], dwk[4];
  float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
  double f[4];
  load_weight<ACC>(a.q_w, pl, N, wq);
  load_weight<ACC>(a.k_w, pl, N, wk);
  load_freqs<ACC>(a.freqs, pl, (int)a.R, f);
  Way in(a), out = in;
  int pos = in.valid() && a.R > 0 ? a.positions[in.row] : 0;
  const T* from = nullptr;
  const U* ufrom = nullptr;
  int missing = 0, in_left = 0;  // 0: nothing more to copy
  auto open = [&] {
    if (in.valid()) {
      from = in.at<ACC>(q, k, a.ldq, a.ldk, pl, N);
      ufrom = in.at<ACC>(uq, uk, a.Hq * N, a.Hk * N, pl, N);
      missing = in.missing(a, pl);
      in_left = in.left;
    }
  };
  auto fetch = [&](int slot) {
    if (in_left > 0) {
      const bool on = in_left > missing;
      const int up = slot + Slot<T>::kBytes;
      Slot<T>::template fetch<ACC>(ring + slot, ring_addr + slot, from, n, apart, on);
      Slot<U>::template fetch<ACC>(ring + up, ring_addr + up, ufrom, n, apart, on);
      from += stride;
      ufrom += stride;
      if (--in_left == 0) {
        in.next_run(a);
        open();
      }
    }
    copies_end();
  };
#pragma unroll
  for (int i = 0; i < kBwdRing; ++i) {
    Slot<T>::template clear<ACC>(ring + i * kSlot, n, apart);
    Slot<U>::template clear<ACC>(ring + i * kSlot + Slot<T>::kBytes, n, apart);
  }
  open();
#pragma unroll
  for (int i = 0; i < kBwdRing - 1; ++i) fetch(i * kSlot);
#pragma unroll
  for (int p = 0; p < 4; ++p) dwq[p] = dwk[p] = splat(0.f);
  int slot = 0, before = kRing - kSlot;
  auto run = [&](const float2(&w)[4], float2(&dw)[4]) {
    G* to = out.at<ACC>(static_cast<G*>(args.dq), static_cast<G*>(args.dk), args.ldgq, args.ldgk, pl, N);
    const int none = out.missing(a, pl);
    for (int left = out.left; left > 0; --left) {
      copies_wait<kBwdRing - 2>();
      fetch(before);
      float2 v[4], d[4];
      Slot<T>::read(ring + slot, v);
      Slot<U>::read(ring + slot + Slot<T>::kBytes, d);
      before = slot;
      slot = slot == kRing - kSlot ? 0 : slot + kSlot;
      backward<ACC>(v, d, left > none, to, n, apart, inv_n, a.eps, pl.lanes, w, c, s, dw);
      to += stride;
    }
  };
  int at = -1;  // the row that c and s are of
  while (out.valid()) {
    if (at != out.row) {
      at = out.row;
      if (a.R > 0) turn<false>(pos, f, c, s);
      pos = out.next_position(a);
    }
    if (out.keys)
      run(wk, dwk);
    else
      run(wq, dwq);
    out.next_run(a);
  }
  copies_wait<0>();
  __syncthreads();
  float(*red)[2][256] = reinterpret_cast<float(*)[2][256]>(smem);
  // the CTA's sums of each column: over a warp's heads, then over the warps in order
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    for (int o = pl.lanes; o < 32; o <<= 1) {
      dwq[p].x += __shfl_xor_sync(0xffffffffu, dwq[p].x, o);
      dwq[p].y += __shfl_xor_sync(0xffffffffu, dwq[p].y, o);
      dwk[p].x += __shfl_xor_sync(0xffffffffu, dwk[p].x, o);
      dwk[p].y += __shfl_xor_sync(0xffffffffu, dwk[p].y, o);
    }
    const int e = pl.at<ACC>(p);
    if (pl.sub == 0 && e < N) {
      *reinterpret_cast<float2*>(&red[threadIdx.x >> 5][0][e]) = dwq[p];
      *reinterpret_cast<float2*>(&red[threadIdx.x >> 5][1][e]) = dwk[p];
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

// Slots of a token, and the blocks of them that are a warp's unit: all together where the tokens alone
// give every warp eight units or more, so that the last ones leave few idle; else blocks of four
// slots or more that do (a unit costs its angles: all tokens in blocks of four, 141 us instead of
// 110); and smaller ones where there are not even as many units as warps.
void set_blocks(RotateArgs& a, int64_t ctas_an_sm) {
  const int64_t sms = current_device_sms() > 0 ? current_device_sms() : 148;
  const int64_t warps = sms * ctas_an_sm * kWarps;
  a.lanes = lanes_of(a.N);
  const int64_t per = 32 / a.lanes;
  a.q_slots = (int)((a.Hq + per - 1) / per);
  a.slots = a.q_slots + (int)((a.Hk + per - 1) / per);
  int64_t blocks = 1;
  if (a.rows > 0) {
    blocks = (8 * warps + a.rows - 1) / a.rows;
    if (blocks > (a.slots + 3) / 4) blocks = (a.slots + 3) / 4;
    if (a.rows * blocks < warps) blocks = (warps + a.rows - 1) / a.rows;
    if (blocks > a.slots) blocks = a.slots;
  }
  a.block = (int)((a.slots + blocks - 1) / blocks);
  a.blocks = (a.slots + a.block - 1) / a.block;
}
unsigned grid_of(const RotateArgs& a, int64_t ctas_an_sm) {
  const int64_t sms = current_device_sms() > 0 ? current_device_sms() : 148;
  const int64_t want = (a.rows * a.blocks + kWarps - 1) / kWarps, most = sms * ctas_an_sm;
  return (unsigned)(want < most ? want : most);
}

struct Strided {
  const void* p;
  int64_t ld;
  int64_t size;  // of an element
};
// The widest access that heads of N at these addresses allow.
Access access_of(int64_t N, std::initializer_list<Strided> ts) {
  bool ok[3] = {N % 8 == 0, N % 4 == 0, true};
  const int piece[3] = {8, 4, 2};
  for (const Strided& t : ts)
    for (int i = 0; i < 3; ++i)
      ok[i] &= piece[i] * t.size <= 16 && t.ld % piece[i] == 0 &&
               reinterpret_cast<uintptr_t>(t.p) % (piece[i] * t.size) == 0;
  return ok[0] ? kWide : ok[1] ? kQuads : ok[2] ? kPairs : kSingle;
}

template <auto KERNEL, typename A>
cudaError_t launch(const A& a, unsigned grid, int smem, cudaStream_t s) {
  const cudaError_t e = allow_shared<KERNEL>(smem);
  if (e != cudaSuccess) return e;
  KERNEL<<<grid, kThreads, smem, s>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t fwd_t(const RotateArgs& a, cudaStream_t s) {
  constexpr int smem = kWarps * kFwdRing * Slot<T>::kBytes;
  const int64_t z = sizeof(T);
  const unsigned grid = grid_of(a, kFwdCtas);
  switch (access_of(a.N, {{a.q, a.ldq, z}, {a.k, a.ldk, z}, {a.q_out, a.N, z}, {a.k_out, a.N, z}})) {
    case kWide:
      if constexpr (sizeof(T) == 2) return launch<norm_rotate_kernel<T, kWide>>(a, grid, smem, s);
      return cudaErrorInvalidValue;  // not of fp32
    case kQuads: return launch<norm_rotate_kernel<T, kQuads>>(a, grid, smem, s);
    case kPairs: return launch<norm_rotate_kernel<T, kPairs>>(a, grid, smem, s);
    default: return launch<norm_rotate_kernel<T, kSingle>>(a, grid, smem, s);
  }
}
template <typename T, typename U, typename G>
cudaError_t bwd_t(const RotateBwdArgs& a, unsigned grid, cudaStream_t s) {
  constexpr int held = kWarps * kBwdRing * (Slot<T>::kBytes + Slot<U>::kBytes);
  constexpr int sums = kWarps * 2 * 256 * (int)sizeof(float), smem = held > sums ? held : sums;
  const RotateArgs& f = a.f;
  const int64_t z = sizeof(T), zu = sizeof(U), zg = sizeof(G);
  switch (access_of(f.N, {{f.q, f.ldq, z}, {f.k, f.ldk, z}, {a.dq_out, f.N, zu}, {a.dk_out, f.N, zu},
                          {a.dq, a.ldgq, zg}, {a.dk, a.ldgk, zg}})) {
    case kWide:
      if constexpr (sizeof(T) + sizeof(U) + sizeof(G) == 6)
        return launch<norm_rotate_bwd_kernel<T, U, G, kWide>>(a, grid, smem, s);
      return cudaErrorInvalidValue;  // not where one is fp32
    case kQuads: return launch<norm_rotate_bwd_kernel<T, U, G, kQuads>>(a, grid, smem, s);
    case kPairs: return launch<norm_rotate_bwd_kernel<T, U, G, kPairs>>(a, grid, smem, s);
    default: return launch<norm_rotate_bwd_kernel<T, U, G, kSingle>>(a, grid, smem, s);
  }
}

}  // namespace

cudaError_t launch_norm_rotate(const RotateArgs& args, cudaStream_t s) {
  if (args.rows == 0) return cudaSuccess;
  RotateArgs a = args;
  set_blocks(a, kFwdCtas);
  return a.bf16 ? fwd_t<__nv_bfloat16>(a, s) : fwd_t<float>(a, s);
}

namespace {
void set_bwd_blocks(RotateArgs& a) { set_blocks(a, kBwdCtas); }
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
