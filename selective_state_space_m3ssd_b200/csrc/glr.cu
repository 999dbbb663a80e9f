// The gated linear recurrence over a sequence, its backward, and one step of it (glr.cuh has
// the arithmetic).
#include <cuda_runtime.h>

#include <cstdint>
#include <initializer_list>
#include <type_traits>

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

// ---- the scan's pieces -------------------------------------------------------------------
//
// A CTA of eight warps takes 64 channels of a sequence, two a lane, and walks the tokens in
// tiles: a warp composes its kRun tokens into h -> A h + B, the warps' (A, B) meet in shared
// memory, and every warp then finishes its tokens from the state that reaches it.  With few
// (sequence, channels) a cluster's CTAs take consecutive tiles of one and hand each other
// their tiles' (A, B) through shared memory.

#ifndef KW
#define KW 8
#define KR 8
#define KB 2
#endif
constexpr int kWarps = KW, kLanes = 32, kGroup = 64, kMaxCluster = 8;

// Tokens of a warp: 512 bytes of a row's channels either way, so that a stage of three tensors takes
// 3 KB a warp.
template <typename T>
constexpr int kRun = sizeof(T) == 2 ? KR : 4;

// How rows are copied: in 16-byte pieces, 4-byte pieces, or element by element (bf16 rows that
// start in the middle of a word).
enum Copy { kCopy16, kCopy4, kCopyElem };

// A map h -> A h + B of two channels; `cut`: a reset lies in it, so that h does not matter
// (h may be NaN, and 0 h is then not 0).
struct Map {
  float2 A, B;
};
__device__ __forceinline__ float2 apply(const Map& m, float2 h, bool cut) {
  return cut ? m.B : fma2(m.A, h, m.B);
}

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes));
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes));
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// Stores to the same place of another CTA's shared memory.
__device__ __forceinline__ void remote_store(uint32_t local, uint32_t rank, float4 v) {
  uint32_t p;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(p) : "r"(local), "r"(rank));
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(p), "f"(v.x), "f"(v.y),
               "f"(v.z), "f"(v.w)
               : "memory");
}
__device__ __forceinline__ void remote_store(uint32_t local, uint32_t rank, uint32_t v) {
  uint32_t p;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(p) : "r"(local), "r"(rank));
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(p), "r"(v) : "memory");
}

__device__ __forceinline__ float2 pair_of(const float* p) { return *reinterpret_cast<const float2*>(p); }
__device__ __forceinline__ float2 pair_of(const __nv_bfloat16* p) {
  const uint32_t u = *reinterpret_cast<const uint32_t*>(p);
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
// Two channels to global memory: `whole` where pairs are aligned and both exist.
template <typename T>
__device__ __forceinline__ void put_pair(T* p, float2 v, bool whole, bool in0, bool in1) {
  if (whole) {
    if (in0) {
      if constexpr (sizeof(T) == 2)
        *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(v.x, v.y);
      else
        *reinterpret_cast<float2*>(p) = v;
    }
  } else {
    if (in0) p[0] = from_f32<T>(v.x);
    if (in1) p[1] = from_f32<T>(v.y);
  }
}

// A lane's part of its warp's copies of kRun tokens' 64 channels of one tensor.
template <typename T, int MODE>
struct Copier {
  static constexpr int run = kRun<T>;
  static constexpr int per = MODE == kCopy16 ? 16 / (int)sizeof(T) : MODE == kCopy4 ? 4 / (int)sizeof(T) : 1;
  static constexpr int chunks = kGroup / per;                    // of a row
  static constexpr int rows = chunks < kLanes ? kLanes / chunks : 1;  // a warp's at once
  static constexpr int cols = chunks < kLanes ? 1 : chunks / kLanes;  // pieces of a row a lane
  static_assert(run % rows == 0, "a copy of the warp takes whole rows of its run");
  const T* tensor; // where nothing is to be read
  const T* base;   // of the CTA's next tile: its first token, the group's first channel
  int64_t ld, off; // the lane's first piece from there

  __device__ __forceinline__ void init(const void* t, int64_t row, int64_t d0, int64_t ld_, int warp,
                                       int lane) {
    ld = ld_;
    tensor = static_cast<const T*>(t);
    base = tensor + row * ld + d0;
    off = (int64_t)(warp * run + row_of(lane)) * ld + col_of(lane);
  }
  static __device__ __forceinline__ int row_of(int lane) { return rows > 1 ? lane / chunks : 0; }
  static __device__ __forceinline__ int col_of(int lane) { return lane % chunks * per; }
  // All of the warp's tokens and channels.
  __device__ __forceinline__ void copy_all(T* dst, int lane) const {
    const T* p = base + off;
    T* at = dst + row_of(lane) * kGroup + col_of(lane);
#pragma unroll
    for (int j = 0; j < run; j += rows, p += rows * ld, at += rows * kGroup)
#pragma unroll
      for (int c = 0; c < cols; ++c) {
        if constexpr (MODE == kCopy16)
          copy16(smem_addr(at + c * kLanes * per), p + c * kLanes * per, 16);
        else if constexpr (MODE == kCopy4)
          copy4(smem_addr(at + c * kLanes * per), p + c * kLanes * per, 4);
        else
          at[c * kLanes * per] = p[c * kLanes * per];
      }
  }
  // Those of the tokens lo to hi - 1 of the warp and of the first `left` channels; zeros elsewhere.
  __device__ __forceinline__ void copy_some(T* dst, int lo, int hi, int left, int lane) const {
    const T* p = base + off;
#pragma unroll
    for (int j = 0; j < run; j += rows, p += rows * ld) {
      const int r = j + row_of(lane);
#pragma unroll
      for (int c = 0; c < cols; ++c) {
        const int col = col_of(lane) + c * kLanes * per;
        const int n = r >= lo && r < hi ? min(max(left - col, 0), per) * (int)sizeof(T) : 0;
        T* const at = dst + r * kGroup + col;
        const T* const from = n > 0 ? p + c * kLanes * per : tensor;
        if constexpr (MODE == kCopy16)
          copy16(smem_addr(at), from, n);
        else if constexpr (MODE == kCopy4)
          copy4(smem_addr(at), from, n);
        else
          *at = n > 0 ? *from : from_f32<T>(0.f);
      }
    }
  }
};

// The resets among a warp's tokens from t on, a bit each (0 outside [0, len)).
template <int RUN>
__device__ __forceinline__ uint32_t resets_of(const uint8_t* reset, int t, int len, int lane) {
  const bool on = lane < RUN && t + lane < len && reset[t + lane];
  return __ballot_sync(0xffffffffu, on);
}

// What a CTA's warps and a cluster's CTAs hand each other.
struct Chain {  // the state before each warp's tokens
  float2 state[kWarps][kLanes];
};
struct Maps {  // the warps' and the CTAs' maps of two consecutive rounds
  float4 warp[2][kWarps][kLanes];
  float4 cta[2][kMaxCluster][kLanes];
  uint32_t warp_cut[2][kWarps];
  uint32_t cta_cut[2][kMaxCluster];
};
__device__ __forceinline__ float4 pack_map(const Map& m) {
  return make_float4(m.A.x, m.A.y, m.B.x, m.B.y);
}
__device__ __forceinline__ Map unpack_map(float4 v) {
  return {make_float2(v.x, v.y), make_float2(v.z, v.w)};
}

// A CTA on its own: the state goes from warp to warp, in a circle, each waiting at the barrier of
// its link (order + 1) only.  A warp's place is written anew after its state has come round to
// the one before it, so after it was read.  Returns the state before the warp's tokens.
__device__ __forceinline__ float2 pass_on(Chain& ch, const Map& mine, bool cut, int order, bool first,
                                          bool last, int lane) {
  if (!first) asm volatile("bar.sync %0, 64;" ::"r"(order + 1) : "memory");
  const float2 in = ch.state[order][lane];
  const int next = order == kWarps - 1 ? 0 : order + 1;
  ch.state[next][lane] = apply(mine, in, cut);
  if (!last) asm volatile("bar.arrive %0, 64;" ::"r"(next + 1) : "memory");
  return in;
}

// A cluster: the warps' maps make the CTA's, the CTAs' the round's; two barriers a round.  The CTA
// is number `rank_order` of `ranks` along the walk; `carry`, the state before the round, is
// advanced past it.  Returns the state before the warp's tokens.
template <bool RESET>
__device__ __forceinline__ float2 exchange(Maps& ex, int flip, const Map& mine, bool cut, int order,
                                           uint32_t rank_order, uint32_t ranks, float2& carry,
                                           int warp, int lane) {
  ex.warp[flip][order][lane] = pack_map(mine);
  if (RESET && lane == 0) ex.warp_cut[flip][order] = cut;
  __syncthreads();
  Map all = {splat(1.f), splat(0.f)}, before = all;
  bool all_cut = false, before_cut = false;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w == order) {
      before = all;
      before_cut = all_cut;
    }
    const Map m = unpack_map(ex.warp[flip][w][lane]);
    const bool c = RESET && ex.warp_cut[flip][w];
    all.B = apply(m, all.B, c);
    all.A = mul2(m.A, all.A);
    all_cut |= c;
  }
  if (warp < (int)ranks) {  // warp q tells CTA q
    remote_store(smem_addr(&ex.cta[flip][rank_order][lane]), (uint32_t)warp, pack_map(all));
    if (RESET && lane == 0)
      remote_store(smem_addr(&ex.cta_cut[flip][rank_order]), (uint32_t)warp, (uint32_t)all_cut);
  }
  cluster_arrive();
  cluster_wait();
  float2 in = carry;
  for (uint32_t q = 0; q < ranks; ++q) {
    if (q == rank_order) in = carry;
    carry = apply(unpack_map(ex.cta[flip][q][lane]), carry, RESET && ex.cta_cut[flip][q]);
  }
  return apply(before, in, before_cut);
}

#ifndef KS
#define KS 3
#endif
constexpr int kStages = KS;

// Shared memory of `stages` stages of `tensors` runs a warp.
template <typename T>
constexpr int ring_bytes(int tensors, int stages) {
  return stages * kWarps * tensors * kRun<T> * kGroup * (int)sizeof(T);
}

template <typename T, int MODE, bool RESET, bool CLUSTER>
__global__ void __launch_bounds__(kWarps * kLanes, KB) glr_fwd_kernel(GlrArgs a) {
  constexpr int run = kRun<T>, tile = kWarps * run;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ typename std::conditional<CLUSTER, Maps, Chain>::type ex;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CLUSTER ? cluster_rank() : 0, ranks = CLUSTER ? cluster_size() : 1;
  const int64_t groups = (a.D + kGroup - 1) / kGroup, item = blockIdx.x / ranks;
  const int64_t b = item / groups, d0 = item % groups * kGroup, d = d0 + 2 * lane;
  const int left = (int)min(a.D - d0, (int64_t)kGroup), L = (int)a.L;
  const bool in0 = d < a.D, in1 = d + 1 < a.D;
  const int len = a.lengths ? min(max(a.lengths[b], 0), L) : L;
  const int step = (int)ranks * tile;  // tokens of a round
  int t0 = (int)rank * tile;           // the CTA's first one
  const int64_t row = b * a.L + t0;
  Copier<T, MODE> src[3];
  src[0].init(a.x, row, d0, a.ldx, warp, lane);
  src[1].init(a.r, row, d0, a.ldr, warp, lane);
  src[2].init(a.i, row, d0, a.ldi, warp, lane);
  T* y = static_cast<T*>(a.y) + row * a.D + d0;
  const uint32_t D = (uint32_t)a.D, at = warp * run * D + 2 * lane;  // of the warp's first output
  const uint8_t* const reset = RESET ? a.reset + b * a.L : nullptr;
  const bool whole = a.D % 2 == 0 && reinterpret_cast<uintptr_t>(a.y) % (2 * sizeof(T)) == 0;
  Channel ch;
  channel_of(a.rate, a.bias_r, a.bias_i, a.c, d, d + 1, a.D, ch);
  float2 carry = splat(0.f);
  if (a.h0) {
    if (in0) carry.x = a.h0[b * a.D + d];
    if (in1) carry.y = a.h0[b * a.D + d + 1];
  }
  if constexpr (!CLUSTER) {
    if (warp == 0) ex.state[0][lane] = carry;
  }

  T* const ring = reinterpret_cast<T*>(smem) + warp * 3 * run * kGroup;
  auto stage = [&](int k) { return ring + k * (kWarps * 3 * run * kGroup); };
  auto fetch = [&](int k, int t) {  // the tile whose first token is t
    const int hi = len - t - warp * run;
    if (hi >= run && left == kGroup) {
#pragma unroll
      for (int j = 0; j < 3; ++j) src[j].copy_all(stage(k) + j * run * kGroup, lane);
    } else if (hi > 0) {
#pragma unroll
      for (int j = 0; j < 3; ++j) src[j].copy_some(stage(k) + j * run * kGroup, 0, hi, left, lane);
    }
#pragma unroll
    for (int j = 0; j < 3; ++j) src[j].base += step * src[j].ld;
    copies_end();
  };
#pragma unroll
  for (int k = 0; k < kStages - 1; ++k) fetch(k, t0 + k * step);
  int k = 0;
  [[maybe_unused]] int flip = 0;
  for (int done = 0; done < L; done += step, t0 += step) {
    copies_wait<kStages - 2>();
    __syncwarp();
    fetch(k == 0 ? kStages - 1 : k - 1, t0 + (kStages - 1) * step);
    const T* const st = stage(k) + 2 * lane;
    k = k == kStages - 1 ? 0 : k + 1;
    const int t = t0 + warp * run;
    const uint32_t cuts = RESET ? resets_of<run>(reset, t, len, lane) : 0;
    Map m[run];
    if (t + run <= len) {
#pragma unroll
      for (int j = 0; j < run; ++j) {
        const bool cut = RESET && (cuts >> j & 1);
        Map e;
        element(ch, pair_of(st + j * kGroup), pair_of(st + (run + j) * kGroup),
                pair_of(st + (2 * run + j) * kGroup), cut, e.A, e.B);
        m[j].B = j ? apply(e, m[j - 1].B, cut) : e.B;
        m[j].A = !j ? e.A : cut ? splat(0.f) : mul2(e.A, m[j - 1].A);
      }
    } else {  // the last tokens: past them the state stays
#pragma unroll
      for (int j = 0; j < run; ++j) {
        const bool cut = RESET && (cuts >> j & 1);
        Map e = {splat(1.f), splat(0.f)};
        if (t + j < len)
          element(ch, pair_of(st + j * kGroup), pair_of(st + (run + j) * kGroup),
                  pair_of(st + (2 * run + j) * kGroup), cut, e.A, e.B);
        m[j].B = j ? apply(e, m[j - 1].B, cut) : e.B;
        m[j].A = !j ? e.A : cut ? splat(0.f) : mul2(e.A, m[j - 1].A);
      }
    }
    float2 in;
    if constexpr (CLUSTER)
      in = exchange<RESET>(ex, flip, m[run - 1], cuts != 0, warp, rank, ranks, carry, warp, lane);
    else
      in = pass_on(ex, m[run - 1], cuts != 0, warp, done == 0 && warp == 0,
                   done + step >= L && warp == kWarps - 1, lane);
    flip ^= 1;
    if (t + run <= len && whole) {
#pragma unroll
      for (int j = 0; j < run; ++j)
        put_pair(y + (at + j * D), apply(m[j], in, RESET && (cuts & ((2u << j) - 1))), true, in0, in1);
    } else {
#pragma unroll
      for (int j = 0; j < run; ++j) {
        const float2 h = apply(m[j], in, RESET && (cuts & ((2u << j) - 1)));
        if (t + j < L) put_pair(y + (at + j * D), t + j < len ? h : splat(0.f), whole, in0, in1);
      }
    }
    y += step * a.D;
  }
  if constexpr (CLUSTER) {  // no CTA leaves while another may write to its shared memory
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
    carry = ex.state[0][lane];  // after the last warp's last tokens
  }
  if (a.hT && rank == 0 && warp == 0) {
    if (in0) a.hT[b * a.D + d] = carry.x;
    if (in1) a.hT[b * a.D + d + 1] = carry.y;
  }
}

// The walk back: tiles from the last one, a tile's last run first.  With g_t = dy_t + back_t a
// token maps back_t, what comes from later tokens, to back_{t-1} = a_t (back_t + dy_t).  A warp
// first composes its run (the decays alone), and once back has reached it, walks the run again
// with the whole gradient; recomputing the gates costs less than holding them would.
template <typename T, typename G, int MODE, bool RESET, bool CLUSTER>
__global__ void __launch_bounds__(kWarps * kLanes, 2) glr_bwd_kernel(GlrBwdArgs args) {
  constexpr int run = kRun<T>, tile = kWarps * run, kTensors = 5;
  const GlrArgs& a = args.f;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ typename std::conditional<CLUSTER, Maps, Chain>::type ex;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, order = kWarps - 1 - warp;
  const uint32_t rank = CLUSTER ? cluster_rank() : 0, ranks = CLUSTER ? cluster_size() : 1;
  const int64_t groups = (a.D + kGroup - 1) / kGroup, item = blockIdx.x / ranks;
  const int64_t b = item / groups, d0 = item % groups * kGroup, d = d0 + 2 * lane;
  const int left = (int)min(a.D - d0, (int64_t)kGroup), L = (int)a.L;
  const bool in0 = d < a.D, in1 = d + 1 < a.D;
  const int len = a.lengths ? min(max(a.lengths[b], 0), L) : L;
  const int step = (int)ranks * tile, rounds = (L + step - 1) / step;
  int t0 = (rounds - 1) * step + (int)rank * tile;
  const int64_t row = b * a.L + t0;
  Copier<T, MODE> src[kTensors];
  src[0].init(a.x, row, d0, a.ldx, warp, lane);
  src[1].init(a.r, row, d0, a.ldr, warp, lane);
  src[2].init(a.i, row, d0, a.ldi, warp, lane);
  src[3].init(args.dy, row, d0, a.D, warp, lane);
  src[4].init(a.y, row - 1, d0, a.D, warp, lane);  // h_{t-1}
  const uint32_t ldg = (uint32_t)args.ldg, at = warp * run * ldg + 2 * lane;
  G* out[3] = {static_cast<G*>(args.dx) + row * args.ldg + d0,
               static_cast<G*>(args.dr) + row * args.ldg + d0,
               static_cast<G*>(args.di) + row * args.ldg + d0};
  const uint8_t* const reset = RESET ? a.reset + b * a.L : nullptr;
  const bool whole = (a.D | ldg) % 2 == 0 &&
                     (reinterpret_cast<uintptr_t>(args.dx) | reinterpret_cast<uintptr_t>(args.dr) |
                      reinterpret_cast<uintptr_t>(args.di)) % (2 * sizeof(G)) == 0;
  Channel ch;
  channel_of(a.rate, a.bias_r, a.bias_i, a.c, d, d + 1, a.D, ch);
  float2 back = splat(0.f), h0 = splat(0.f);
  if (args.dhT) {
    if (in0) back.x = args.dhT[b * a.D + d];
    if (in1) back.y = args.dhT[b * a.D + d + 1];
  }
  if (a.h0) {
    if (in0) h0.x = a.h0[b * a.D + d];
    if (in1) h0.y = a.h0[b * a.D + d + 1];
  }
  if constexpr (!CLUSTER) {
    if (order == 0) ex.state[0][lane] = back;
  }
  float2 se = splat(0.f), sr = splat(0.f), si = splat(0.f);

  T* const ring = reinterpret_cast<T*>(smem) + warp * kTensors * run * kGroup;
  auto stage = [&](int k) { return ring + k * (kWarps * kTensors * run * kGroup); };
  auto fetch = [&](int k, int t) {
    const int hi = len - t - warp * run;
    if (t >= 0 && hi > 0) {
      const bool all = hi >= run && left == kGroup;
      const int lo = t == 0 && warp == 0 ? 1 : 0;  // no h before the first token
#pragma unroll
      for (int j = 0; j < kTensors; ++j) {
        if (all && (j < 4 || lo == 0))
          src[j].copy_all(stage(k) + j * run * kGroup, lane);
        else
          src[j].copy_some(stage(k) + j * run * kGroup, j < 4 ? 0 : lo, hi, left, lane);
      }
    }
#pragma unroll
    for (int j = 0; j < kTensors; ++j) src[j].base -= step * src[j].ld;
    copies_end();
  };
  fetch(0, t0);
  int k = 0;
  [[maybe_unused]] int flip = 0;
  for (int round = 0; round < rounds; ++round, t0 -= step) {
    copies_wait<0>();
    __syncwarp();
    fetch(k ^ 1, t0 - step);
    const T* const st = stage(k) + 2 * lane;
    k ^= 1;
    const int t = t0 + warp * run;
    const bool full = t + run <= len;
    const uint32_t cuts = RESET ? resets_of<run>(reset, t, len, lane) : 0;
    Map m = {splat(1.f), splat(0.f)};
    auto compose = [&](int j) {
      const bool cut = RESET && (cuts >> j & 1);
      const float2 al = decay(ch, pair_of(st + (run + j) * kGroup), cut);
      const float2 dy = pair_of(st + (3 * run + j) * kGroup);
      m.A = cut ? splat(0.f) : mul2(al, m.A);
      m.B = cut ? splat(0.f) : mul2(al, add2(m.B, dy));
    };
    if (full) {
#pragma unroll
      for (int j = run - 1; j >= 0; --j) compose(j);
    } else {
#pragma unroll
      for (int j = run - 1; j >= 0; --j)
        if (t + j < len) compose(j);
    }
    float2 g;  // what reaches the run from later tokens
    if constexpr (CLUSTER)
      g = exchange<RESET>(ex, flip, m, cuts != 0, order, ranks - 1 - rank, ranks, back, warp, lane);
    else
      g = pass_on(ex, m, cuts != 0, order, round == 0 && order == 0,
                  round == rounds - 1 && order == kWarps - 1, lane);
    flip ^= 1;
    const float2 first = t == 0 ? h0 : splat(0.f);
    auto finish = [&](int j, float2& dx, float2& dr, float2& di) {
      const bool cut = RESET && (cuts >> j & 1);
      g = add2(g, pair_of(st + (3 * run + j) * kGroup));
      float2 prev = pair_of(st + (4 * run + j) * kGroup), E;
      if (j == 0) prev = add2(prev, first);
      const float2 al = element_grad(ch, pair_of(st + j * kGroup), pair_of(st + (run + j) * kGroup),
                                     pair_of(st + (2 * run + j) * kGroup), cut, prev, g, dx, dr, di, E);
      g = cut ? splat(0.f) : mul2(al, g);
      se = add2(se, E);
      sr = add2(sr, dr);
      si = add2(si, di);
    };
    if (full && whole) {
#pragma unroll
      for (int j = run - 1; j >= 0; --j) {
        float2 dx, dr, di;
        finish(j, dx, dr, di);
        put_pair(out[0] + (at + j * ldg), dx, true, in0, in1);
        put_pair(out[1] + (at + j * ldg), dr, true, in0, in1);
        put_pair(out[2] + (at + j * ldg), di, true, in0, in1);
      }
    } else {
#pragma unroll
      for (int j = run - 1; j >= 0; --j) {
        float2 dx = splat(0.f), dr = dx, di = dx;
        if (t + j < len) finish(j, dx, dr, di);
        if (t + j < L) {
          put_pair(out[0] + (at + j * ldg), dx, whole, in0, in1);
          put_pair(out[1] + (at + j * ldg), dr, whole, in0, in1);
          put_pair(out[2] + (at + j * ldg), di, whole, in0, in1);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 3; ++j) out[j] -= step * args.ldg;
  }
  if constexpr (CLUSTER) {
    cluster_arrive();
    cluster_wait();
  }
  // the CTA's sums, the warps' in order: a row of the workspace for each sequence and rank
  copies_wait<0>();
  __syncthreads();
  if constexpr (!CLUSTER) back = ex.state[0][lane];
  float2(*red)[3][kLanes] = reinterpret_cast<float2(*)[3][kLanes]>(smem);
  red[warp][0][lane] = se;
  red[warp][1][lane] = sr;
  red[warp][2][lane] = si;
  __syncthreads();
  if (warp < 3) {
    float2 s = splat(0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s = add2(s, red[w][warp][lane]);
    float* const part = args.part + (3 * (b * ranks + rank) + warp) * a.D + d;
    if (in0) part[0] = s.x;
    if (in1) part[1] = s.y;
  }
  if (args.dh0 && rank == 0 && warp == 0) {
    if (in0) args.dh0[b * a.D + d] = back.x;
    if (in1) args.dh0[b * a.D + d + 1] = back.y;
  }
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

// The widest copies that rows at these addresses and strides allow.
template <typename T>
Copy copy_of(std::initializer_list<const void*> ps, std::initializer_list<int64_t> lds) {
  uint64_t bits = 0;
  for (const void* p : ps) bits |= reinterpret_cast<uintptr_t>(p);
  for (int64_t ld : lds) bits |= (uint64_t)ld * sizeof(T);
  return bits % 16 == 0 ? kCopy16 : bits % 4 == 0 ? kCopy4 : kCopyElem;
}

// CTAs along a sequence: as many (a power of two) as two an SM hold, each with two tiles or more.
int ranks_of(int64_t items, int64_t tiles) {
  const int64_t sms = current_device_sms() > 0 ? current_device_sms() : 148;
  int r = 1;
  while (r < kMaxCluster && items * r * 2 <= sms * 2 && tiles >= 4 * r) r *= 2;
  return r;
}

template <typename K, typename A>
cudaError_t launch(K kernel, const A& args, unsigned grid, int ranks, int smem, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)ranks;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid * (unsigned)ranks);
  cfg.blockDim = dim3(kWarps * kLanes);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = ranks > 1 ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, kernel, args);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T, int MODE, bool RESET>
cudaError_t fwd_m(const GlrArgs& a, cudaStream_t s) {
  const int64_t items = a.b * ((a.D + kGroup - 1) / kGroup);
  const int ranks = ranks_of(items, (a.L + kWarps * kRun<T> - 1) / (kWarps * kRun<T>));
  const unsigned grid = (unsigned)items;
  return ranks > 1 ? launch(glr_fwd_kernel<T, MODE, RESET, true>, a, grid, ranks, ring_bytes<T>(3, kStages), s)
                   : launch(glr_fwd_kernel<T, MODE, RESET, false>, a, grid, 1, ring_bytes<T>(3, kStages), s);
}
template <typename T, int MODE>
cudaError_t fwd_r(const GlrArgs& a, cudaStream_t s) {
  return a.reset ? fwd_m<T, MODE, true>(a, s) : fwd_m<T, MODE, false>(a, s);
}
template <typename T>
cudaError_t fwd_t(const GlrArgs& a, cudaStream_t s) {
  switch (copy_of<T>({a.x, a.r, a.i}, {a.ldx, a.ldr, a.ldi})) {
    case kCopy16: return fwd_r<T, kCopy16>(a, s);
    case kCopy4: return fwd_r<T, kCopy4>(a, s);
    default:
      if constexpr (sizeof(T) == 2) return fwd_r<T, kCopyElem>(a, s);
      return cudaErrorInvalidValue;  // fp32 rows start at whole words
  }
}

int bwd_ranks(int64_t b, int64_t L, int64_t D, bool bf16) {
  const int tile = kWarps * (bf16 ? kRun<__nv_bfloat16> : kRun<float>);
  return ranks_of(b * ((D + kGroup - 1) / kGroup), (L + tile - 1) / tile);
}

template <typename T, typename G, int MODE, bool RESET>
cudaError_t bwd_m(const GlrBwdArgs& a, cudaStream_t s) {
  const GlrArgs& f = a.f;
  const unsigned grid = (unsigned)(f.b * ((f.D + kGroup - 1) / kGroup));
  const int ranks = bwd_ranks(f.b, f.L, f.D, f.bf16), smem = ring_bytes<T>(5, 2);
  return ranks > 1 ? launch(glr_bwd_kernel<T, G, MODE, RESET, true>, a, grid, ranks, smem, s)
                   : launch(glr_bwd_kernel<T, G, MODE, RESET, false>, a, grid, 1, smem, s);
}
template <typename T, typename G, int MODE>
cudaError_t bwd_r(const GlrBwdArgs& a, cudaStream_t s) {
  return a.f.reset ? bwd_m<T, G, MODE, true>(a, s) : bwd_m<T, G, MODE, false>(a, s);
}
template <typename T, typename G>
cudaError_t bwd_t(const GlrBwdArgs& a, cudaStream_t s) {
  const GlrArgs& f = a.f;
  switch (copy_of<T>({f.x, f.r, f.i, f.y, a.dy}, {f.ldx, f.ldr, f.ldi, f.D})) {
    case kCopy16: return bwd_r<T, G, kCopy16>(a, s);
    case kCopy4: return bwd_r<T, G, kCopy4>(a, s);
    default:
      if constexpr (sizeof(T) == 2) return bwd_r<T, G, kCopyElem>(a, s);
      return cudaErrorInvalidValue;  // fp32 rows start at whole words
  }
}

}  // namespace

cudaError_t launch_glr_fwd(const GlrArgs& a, cudaStream_t s) {
  return a.bf16 ? fwd_t<__nv_bfloat16>(a, s) : fwd_t<float>(a, s);
}

size_t glr_bwd_workspace_bytes(int64_t b, int64_t L, int64_t D, bool bf16) {
  return (size_t)b * bwd_ranks(b, L, D, bf16) * 3 * (size_t)D * sizeof(float);
}

cudaError_t launch_glr_bwd(const GlrBwdArgs& a, cudaStream_t s) {
  const GlrArgs& f = a.f;
  if (f.b > 0) {
    const cudaError_t e = !f.bf16         ? bwd_t<float, float>(a, s)
                          : a.grad_bf16 ? bwd_t<__nv_bfloat16, __nv_bfloat16>(a, s)
                                        : bwd_t<__nv_bfloat16, float>(a, s);
    if (e != cudaSuccess) return e;
  }
  glr_sum_kernel<<<grid_for(f.D), kThreads, 0, s>>>(a.part, f.b * bwd_ranks(f.b, f.L, f.D, f.bf16), f.D,
                                                     f.rate, a.drate, a.dbias_r, a.dbias_i);
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
