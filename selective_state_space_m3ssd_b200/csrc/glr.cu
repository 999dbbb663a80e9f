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

// ---- the walks' pieces -------------------------------------------------------------------
//
// A CTA of eight warps takes 64 channels of a sequence, two a lane, and walks the tokens in
// tiles, one run of kRun tokens a warp: a warp composes its run into h -> A h + B, waits for
// the state before it, hands the state after it to the next warp and finishes its tokens.
// So the state's way through a tile is eight short hops, under which the other warps (and
// another CTA) compute.  With too few (sequence, channels) to fill the device a sequence is cut
// into parts instead, one a warp, of as many CTAs as there is room for: a first kernel composes
// every part into its map, and in the walk each warp begins from what the maps before it
// make of h0.  That reads the inputs twice, so it is for launches that would leave SMs idle.
//
// Bytes: the forward reads x, r and i and writes y, the backward reads y and dy too and writes three
// gradients.  Measured at 8 x 4096 tokens, 2048 channels, bf16: forward 106 us (0.77 of HBM's copy
// rate), backward with bf16 gradients 216 (0.76).  Latency bounds both, with eight or 16 warps an SM (256 CTAs
// are two on 108 SMs and one on 40): 66 and 133 warp instructions for a token of two channels a lane, most
// of them the gates', fill 65 % of the issue slots of an SM that has a CTA, 55 % of all; the forward's
// hardware approximations keep their pipe busy for 63 %.  32 x 1024 tokens, 1024 CTAs: 97 and 200 us.

constexpr int kWarps = 8, kLanes = 32, kGroup = 64;

// Tokens of a run: 1 KB of a tensor either way.
template <typename T>
constexpr int kRun = sizeof(T) == 2 ? 8 : 4;

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
  const T* base;   // a row and the group's first channel
  int64_t ld, off; // the lane's first piece from there

  // The warp's run begins `ahead` rows after `row`.
  __device__ __forceinline__ void init(const void* t, int64_t row, int ahead, int64_t d0, int64_t ld_,
                                       int lane) {
    ld = ld_;
    tensor = static_cast<const T*>(t);
    base = tensor + row * ld + d0;
    off = (ahead + row_of(lane)) * ld + col_of(lane);
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

// The resets among a warp's tokens, a bit each (0 outside [0, len)), read a run ahead.
template <int RUN, bool RESET>
struct Resets {
  uint32_t ahead = 0;  // a lane's of the run that is taken next
  __device__ __forceinline__ void read(const uint8_t* reset, int t, int len, int lane) {
    if constexpr (RESET)
      ahead = lane < RUN && (uint32_t)(t + lane) < (uint32_t)len ? reset[t + lane] : 0;
  }
  // Those of the run, and the reading of the one from t on.
  __device__ __forceinline__ uint32_t take(const uint8_t* reset, int t, int len, int lane) {
    if constexpr (!RESET) return 0;
    const uint32_t bits = __ballot_sync(0xffffffffu, ahead != 0);
    read(reset, t, len, lane);
    return bits;
  }
};

// Where a warp walks: `rounds` runs of which the first begins at token t, `step` tokens apart;
// all of a sequence's tiles with its CTA, or (SPLIT) one part of it alone, or with others: `share`
// warps, whole runs each, in order.
template <typename T, bool SPLIT>
struct Way {
  int64_t b, d0;
  int first_row;  // the sequence's token that the CTA's (SPLIT: the warp's) first run counts from
  int ahead;      // the warp's run from there
  int step, rounds, part;

  __device__ __forceinline__ Way(const GlrArgs& a, int warp, int share = 1) {
    const int64_t groups = (a.D + kGroup - 1) / kGroup;
    const uint32_t ctas = SPLIT ? (uint32_t)a.split : 1u;
    const int64_t item = blockIdx.x / ctas;
    b = item / groups;
    d0 = item % groups * kGroup;
    const int L = (int)a.L;
    if constexpr (SPLIT) {
      part = (int)(blockIdx.x % ctas) * kWarps + warp / share;
      const int len = (a.part_len / kRun<T> + share - 1) / share * kRun<T>;
      const int64_t from = min((int64_t)part * a.part_len, (int64_t)L);
      const int64_t end = min(from + a.part_len, (int64_t)L);
      first_row = (int)min(from + warp % share * len, end);
      ahead = 0;
      step = kRun<T>;
      rounds = (min((int)end - first_row, len) + kRun<T> - 1) / kRun<T>;
    } else {
      part = 0;
      first_row = 0;
      ahead = warp * kRun<T>;
      step = kWarps * kRun<T>;
      rounds = (L + step - 1) / step;
    }
  }
};

// The state before each warp's run.
struct Chain {
  float2 state[kWarps][kLanes];
};

// The state goes from warp to warp, in a circle, each waiting at the barrier of its link (order +
// 1) only.  A warp's place is written anew after its state has come round to the one before it,
// so after it was read.  Returns the state before the warp's run.
__device__ __forceinline__ float2 pass_on(Chain& ch, const Map& mine, bool cut, int order, bool first,
                                          bool last, int lane) {
  if (!first) asm volatile("bar.sync %0, 64;" ::"r"(order + 1) : "memory");
  const float2 in = ch.state[order][lane];
  const int next = order == kWarps - 1 ? 0 : order + 1;
  ch.state[next][lane] = apply(mine, in, cut);
  if (!last) asm volatile("bar.arrive %0, 64;" ::"r"(next + 1) : "memory");
  return in;
}

// The workspace of a split: the parts' maps, each CTA's eight as one, which hold a reset, and the
// state that the sequence starts from (a copy: the walk may write the new one in its place).
struct SplitMaps {
  float4* part;
  float4* cta;
  float2* start;
  uint32_t* part_cut;
  uint32_t* cta_cut;
};
__host__ __device__ __forceinline__ SplitMaps split_maps(void* p, int64_t items, int split) {
  const int64_t n = items * split;
  SplitMaps m;
  m.part = static_cast<float4*>(p);
  m.cta = m.part + n * kWarps * kLanes;
  m.start = reinterpret_cast<float2*>(m.cta + n * kLanes);
  m.part_cut = reinterpret_cast<uint32_t*>(m.start + items * kLanes);
  m.cta_cut = m.part_cut + n * kWarps;
  return m;
}
size_t split_bytes(int64_t items, int split) {
  return split ? (size_t)(items * split) * (kWarps + 1) * (kLanes * sizeof(float4) + sizeof(uint32_t)) +
                     (size_t)items * kLanes * sizeof(float2)
               : 0;
}
__device__ __forceinline__ float4 pack_map(const Map& m) {
  return make_float4(m.A.x, m.A.y, m.B.x, m.B.y);
}
__device__ __forceinline__ Map unpack_map(float4 v) {
  return {make_float2(v.x, v.y), make_float2(v.z, v.w)};
}

// What the maps before a warp's part make of the start; BACK: before means later in the sequence.  The
// CTAs' maps are composed by eight warps, an eighth of them each.
struct Fold {
  float4 map[kWarps][kLanes];
  uint32_t cut[kWarps];
};
template <bool RESET, bool BACK>
__device__ __forceinline__ float2 start_of(const GlrArgs& a, Fold& fold, int warp, int lane) {
  const int64_t items = gridDim.x / (uint32_t)a.split, cta0 = blockIdx.x / (uint32_t)a.split * a.split;
  const SplitMaps m = split_maps(a.maps, items, a.split);
  const int mine = (int)(blockIdx.x % (uint32_t)a.split);
  const int n = BACK ? a.split - 1 - mine : mine, eighth = (n + kWarps - 1) / kWarps;
  Map all = {splat(1.f), splat(0.f)};
  bool all_cut = false;
#pragma unroll 2
  for (int i = warp * eighth; i < min(warp * eighth + eighth, n); ++i) {
    const int64_t c = cta0 + (BACK ? a.split - 1 - i : i);
    const Map one = unpack_map(m.cta[c * kLanes + lane]);
    const bool cut = RESET && m.cta_cut[c];
    all.B = apply(one, all.B, cut);
    all.A = mul2(one.A, all.A);
    all_cut |= cut;
  }
  fold.map[warp][lane] = pack_map(all);
  if (RESET && lane == 0) fold.cut[warp] = all_cut;
  __syncthreads();
  float2 h = m.start[blockIdx.x / (uint32_t)a.split * kLanes + lane];
#pragma unroll
  for (int i = 0; i < kWarps; ++i) h = apply(unpack_map(fold.map[i][lane]), h, RESET && fold.cut[i]);
  const int w = BACK ? kWarps - 1 - warp : warp;
#pragma unroll
  for (int i = 0; i < kWarps - 1; ++i) {
    if (i < w) {
      const int64_t p = (cta0 + mine) * kWarps + (BACK ? kWarps - 1 - i : i);
      h = apply(unpack_map(m.part[p * kLanes + lane]), h, RESET && m.part_cut[p]);
    }
  }
  return h;
}

// Shared memory of `stages` stages of `tensors` runs a warp.
template <typename T>
constexpr int ring_bytes(int tensors, int stages) {
  return stages * kWarps * tensors * kRun<T> * kGroup * (int)sizeof(T);
}

constexpr int kStages = 3;

// Channels d and d + 1 of a (b, D) state that may not be there.
__device__ __forceinline__ float2 state_at(const float* state, int64_t b, int64_t d, int64_t D) {
  float2 v = splat(0.f);
  if (state && d < D) v.x = state[b * D + d];
  if (state && d + 1 < D) v.y = state[b * D + d + 1];
  return v;
}

// The map of every part of a split: of the forward (BACK: of the backward, from the end on).  kShare warps
// make one: the backward's maps take half of the gates and fit in 64 registers, so that an SM holds 32
// warps.  Measured, us, the backward with two against one: bf16 1 x 512 x 2048 12.0 / 14.7, 1 x 32768 x 64
// 32.0 / 37.1, 2 x 32768 x 768 with resets 260 / 263; fp32 3 x 1777 x 513 40.8 / 35.0.
template <typename T, bool BACK>
constexpr int kShare = BACK && sizeof(T) == 2 ? 2 : 1;

template <typename T, int MODE, bool RESET, bool BACK>
__global__ void __launch_bounds__(kShare<T, BACK> * kWarps * kLanes, 2)
glr_part_kernel(GlrArgs a, const void* dy, const float* start) {
  constexpr int run = kRun<T>, kTensors = BACK ? 2 : 3, share = kShare<T, BACK>, warps = share * kWarps;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float4 maps[warps][kLanes];
  __shared__ uint32_t cut_of[warps];
  cudaTriggerProgrammaticLaunchCompletion();  // the walk may begin to load; it waits itself
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Way<T, true> way(a, warp, share);
  const int64_t d0 = way.d0, d = d0 + 2 * lane;
  const int left = (int)min(a.D - d0, (int64_t)kGroup), L = (int)a.L;
  const int len = a.lengths ? min(max(a.lengths[way.b], 0), L) : L;
  const int step = BACK ? -way.step : way.step;
  int t = way.first_row + (BACK ? (way.rounds - 1) * way.step : 0);
  const int64_t row = way.b * a.L + t;
  Copier<T, MODE> src[kTensors];
  src[0].init(a.r, row, 0, d0, a.ldr, lane);
  src[1].init(BACK ? dy : a.x, row, 0, d0, BACK ? a.D : a.ldx, lane);
  if constexpr (!BACK) src[kTensors - 1].init(a.i, row, 0, d0, a.ldi, lane);
  const uint8_t* const reset = RESET ? a.reset + way.b * a.L : nullptr;
  T* const ring = reinterpret_cast<T*>(smem) + warp * kTensors * run * kGroup;
  auto stage = [&](int k) { return ring + k * (warps * kTensors * run * kGroup); };
  auto fetch = [&](int k, int t, bool on) {
    const int hi = on ? len - t : 0;
    if (hi >= run && left == kGroup) {
#pragma unroll
      for (int j = 0; j < kTensors; ++j) src[j].copy_all(stage(k) + j * run * kGroup, lane);
    } else if (hi > 0) {
#pragma unroll
      for (int j = 0; j < kTensors; ++j)
        src[j].copy_some(stage(k) + j * run * kGroup, 0, hi, left, lane);
    }
#pragma unroll
    for (int j = 0; j < kTensors; ++j) src[j].base += step * src[j].ld;
    copies_end();
  };
#pragma unroll
  for (int k = 0; k < kStages - 1; ++k) fetch(k, t + k * step, k < way.rounds);
  Channel ch;
  channel_of(a.rate, a.bias_r, a.bias_i, a.c, d, d + 1, a.D, ch);
  Resets<run, RESET> resets;
  resets.read(reset, t, len, lane);
  Map m = {splat(1.f), splat(0.f)};
  bool any = false;
  int k = 0;
  for (int round = 0; round < way.rounds; ++round, t += step) {
    copies_wait<kStages - 2>();
    __syncwarp();
    fetch(k == 0 ? kStages - 1 : k - 1, t + (kStages - 1) * step, round + kStages - 1 < way.rounds);
    const T* const st = stage(k) + 2 * lane;
    k = k == kStages - 1 ? 0 : k + 1;
    const uint32_t cuts = resets.take(reset, t + step, len, lane);
    any |= cuts != 0;
    auto compose = [&](int j, uint32_t cuts) {
      const bool cut = RESET && (cuts >> j & 1);
      const float2 r = pair_of(st + j * kGroup), v = pair_of(st + (run + j) * kGroup);
      if constexpr (BACK) {
        float2 al, nz;
        decay(ch, r, al, nz);
        m.B = cut ? splat(0.f) : mul2(al, add2(m.B, v));
        m.A = cut ? splat(0.f) : mul2(al, m.A);
      } else {
        Map e;
        element(ch, v, r, pair_of(st + ((kTensors - 1) * run + j) * kGroup), cut, e.A, e.B);
        m.B = apply(e, m.B, cut);
        m.A = cut ? splat(0.f) : mul2(e.A, m.A);
      }
    };
    if (t + run <= len && cuts == 0) {  // most runs
#pragma unroll
      for (int j = 0; j < run; ++j) compose(BACK ? run - 1 - j : j, 0);
    } else {
      const int n = min(len - t, run);
#pragma unroll 1
      for (int j = 0; j < n; ++j) compose(BACK ? n - 1 - j : j, cuts);
    }
  }
  maps[warp][lane] = pack_map(m);
  if (lane == 0) cut_of[warp] = any;
  const SplitMaps out = split_maps(a.maps, gridDim.x / (uint32_t)a.split, a.split);
  const int64_t cta = blockIdx.x;
  if (warp == 1 && blockIdx.x % (uint32_t)a.split == 0)
    out.start[blockIdx.x / (uint32_t)a.split * kLanes + lane] = state_at(start, way.b, d, a.D);
  __syncthreads();
  // the maps of n warps from w0 on, as one
  auto composed = [&](int w0, int n, bool& all_cut) {
    Map all = {splat(1.f), splat(0.f)};
    all_cut = false;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const int w = w0 + (BACK ? n - 1 - i : i);
      const Map one = unpack_map(maps[w][lane]);
      const bool c = RESET && cut_of[w];
      all.B = apply(one, all.B, c);
      all.A = mul2(one.A, all.A);
      all_cut |= c;
    }
    return pack_map(all);
  };
  bool cut;
  if (warp < kWarps) {
    out.part[(cta * kWarps + warp) * kLanes + lane] = composed(share * warp, share, cut);
    if (lane == 0) out.part_cut[cta * kWarps + warp] = cut;
  }
  if (warp == warps - 1) {
    out.cta[cta * kLanes + lane] = composed(0, warps, cut);
    if (lane == 0) out.cta_cut[cta] = cut;
  }
}

template <typename T, int MODE, bool RESET, bool SPLIT>
__global__ void __launch_bounds__(kWarps * kLanes, 2) glr_fwd_kernel(GlrArgs a) {
  constexpr int run = kRun<T>;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ typename std::conditional<SPLIT, Fold, Chain>::type chain;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Way<T, SPLIT> way(a, warp);
  const int64_t b = way.b, d0 = way.d0, d = d0 + 2 * lane;
  const int left = (int)min(a.D - d0, (int64_t)kGroup), L = (int)a.L, step = way.step;
  const bool in0 = d < a.D, in1 = d + 1 < a.D;
  const int len = a.lengths ? min(max(a.lengths[b], 0), L) : L;
  const int64_t row = b * a.L + way.first_row;
  Copier<T, MODE> src[3];
  src[0].init(a.x, row, way.ahead, d0, a.ldx, lane);
  src[1].init(a.r, row, way.ahead, d0, a.ldr, lane);
  src[2].init(a.i, row, way.ahead, d0, a.ldi, lane);
  T* y = static_cast<T*>(a.y) + row * a.D + d0;
  const uint32_t D = (uint32_t)a.D, at = way.ahead * D + 2 * lane;  // of the warp's first output
  const uint8_t* const reset = RESET ? a.reset + b * a.L : nullptr;
  const bool whole = a.D % 2 == 0 && reinterpret_cast<uintptr_t>(a.y) % (2 * sizeof(T)) == 0;
  if constexpr (!SPLIT) {
    if (warp == 0) chain.state[0][lane] = state_at(a.h0, b, d, a.D);
  }

  T* const ring = reinterpret_cast<T*>(smem) + warp * 3 * run * kGroup;
  auto stage = [&](int k) { return ring + k * (kWarps * 3 * run * kGroup); };
  auto fetch = [&](int k, int t, bool on) {  // the run whose first token is t
    const int hi = on ? len - t : 0;
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
  int t = way.first_row + way.ahead;
#pragma unroll
  for (int k = 0; k < kStages - 1; ++k) fetch(k, t + k * step, k < way.rounds);
  Channel ch;
  channel_of(a.rate, a.bias_r, a.bias_i, a.c, d, d + 1, a.D, ch);
  Resets<run, RESET> resets;
  resets.read(reset, t, len, lane);
  float2 h = splat(0.f);
  if constexpr (SPLIT) {
    cudaGridDependencySynchronize();  // the parts' maps are there
    h = start_of<RESET, false>(a, chain, warp, lane);
  }
  int k = 0;
  for (int round = 0; round < way.rounds; ++round, t += step) {
    copies_wait<kStages - 2>();
    __syncwarp();
    fetch(k == 0 ? kStages - 1 : k - 1, t + (kStages - 1) * step, round + kStages - 1 < way.rounds);
    const T* const st = stage(k) + 2 * lane;
    k = k == kStages - 1 ? 0 : k + 1;
    const uint32_t cuts = resets.take(reset, t + step, len, lane);
    auto token = [&](int j, bool cut) {
      Map e;
      element(ch, pair_of(st + j * kGroup), pair_of(st + (run + j) * kGroup),
              pair_of(st + (2 * run + j) * kGroup), cut, e.A, e.B);
      return e;
    };
    auto pass = [&](const Map& m) {
      if constexpr (SPLIT) return h;
      else
        return pass_on(chain, m, cuts != 0, warp, round == 0 && warp == 0,
                       round == way.rounds - 1 && warp == kWarps - 1, lane);
    };
    if (t + run <= len && cuts == 0) {  // most runs
      Map m[run];  // SPLIT: B is the state itself
#pragma unroll
      for (int j = 0; j < run; ++j) {
        const Map e = token(j, false);
        if constexpr (SPLIT) {
          h = m[j].B = apply(e, h, false);
        } else {
          m[j].B = j ? apply(e, m[j - 1].B, false) : e.B;
          m[j].A = j ? mul2(e.A, m[j - 1].A) : e.A;
        }
      }
      float2 in;
      if constexpr (!SPLIT) in = pass(m[run - 1]);
      auto state = [&](int j) {
        if constexpr (SPLIT) return m[j].B;
        return apply(m[j], in, false);
      };
      if (whole) {
#pragma unroll
        for (int j = 0; j < run; ++j) put_pair(y + (at + j * D), state(j), true, in0, in1);
      } else {
#pragma unroll
        for (int j = 0; j < run; ++j) put_pair(y + (at + j * D), state(j), false, in0, in1);
      }
    } else if (t >= len) {  // past the sequence's end the state stays
      if constexpr (!SPLIT) pass({splat(1.f), splat(0.f)});
#pragma unroll
      for (int j = 0; j < run; ++j)
        if (t + j < L) put_pair(y + (at + j * D), splat(0.f), whole, in0, in1);
    } else {  // a reset or the end; selects, so that the gates overlap
      Map m[run];
#pragma unroll
      for (int j = 0; j < run; ++j) {
        const bool cut = RESET && (cuts >> j & 1), on = t + j < len;
        Map e = token(j, cut);
        e.A = on ? e.A : splat(1.f);
        e.B = on ? e.B : splat(0.f);
        if constexpr (SPLIT) {
          h = m[j].B = apply(e, h, cut);
        } else {
          m[j].B = j ? apply(e, m[j - 1].B, cut) : e.B;
          m[j].A = !j ? e.A : cut ? splat(0.f) : mul2(e.A, m[j - 1].A);
        }
      }
      float2 in;
      if constexpr (!SPLIT) in = pass(m[run - 1]);
#pragma unroll
      for (int j = 0; j < run; ++j) {
        float2 v = m[j].B;
        if constexpr (!SPLIT) v = apply(m[j], in, RESET && (cuts & ((2u << j) - 1)));
        if (t + j < L) put_pair(y + (at + j * D), t + j < len ? v : splat(0.f), whole, in0, in1);
      }
    }
    y += step * a.D;
  }
  bool mine = SPLIT ? way.rounds > 0 && way.first_row + a.part_len >= L : warp == 0;
  if constexpr (!SPLIT) {
    __syncthreads();
    h = chain.state[0][lane];  // after the last warp's last run
  }
  if (a.hT && mine) {
    if (in0) a.hT[b * a.D + d] = h.x;
    if (in1) a.hT[b * a.D + d + 1] = h.y;
  }
}

// The walk back: tiles from the last one, a tile's last run first.  With g_t = dy_t + back_t a
// token maps back_t, what comes from later tokens, to back_{t-1} = a_t (back_t + dy_t).  A warp
// first composes its run (the decays alone, which it keeps in shared memory), and once back has
// reached it, walks the run again with the whole gradient.
template <typename T, typename G, int MODE, bool RESET, bool SPLIT>
__global__ void __launch_bounds__(kWarps * kLanes, 2) glr_bwd_kernel(GlrBwdArgs args) {
  constexpr int run = kRun<T>, kTensors = 5;
  const GlrArgs& a = args.f;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ typename std::conditional<SPLIT, Fold, Chain>::type chain;
  cudaTriggerProgrammaticLaunchCompletion();  // the sums' kernel waits itself
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, order = kWarps - 1 - warp;
  const Way<T, SPLIT> way(a, warp);
  const int64_t b = way.b, d0 = way.d0, d = d0 + 2 * lane;
  const int left = (int)min(a.D - d0, (int64_t)kGroup), L = (int)a.L, step = way.step;
  const bool in0 = d < a.D, in1 = d + 1 < a.D;
  const int len = a.lengths ? min(max(a.lengths[b], 0), L) : L;
  const int t_base = way.first_row + (way.rounds - 1) * step;
  const int64_t row = b * a.L + t_base;
  Copier<T, MODE> src[kTensors];
  src[0].init(a.x, row, way.ahead, d0, a.ldx, lane);
  src[1].init(a.r, row, way.ahead, d0, a.ldr, lane);
  src[2].init(a.i, row, way.ahead, d0, a.ldi, lane);
  src[3].init(args.dy, row, way.ahead, d0, a.D, lane);
  src[4].init(a.y, row - 1, way.ahead, d0, a.D, lane);  // h_{t-1}
  const uint32_t ldg = (uint32_t)args.ldg, at = way.ahead * ldg + 2 * lane;
  G* out[3] = {static_cast<G*>(args.dx) + row * args.ldg + d0,
               static_cast<G*>(args.dr) + row * args.ldg + d0,
               static_cast<G*>(args.di) + row * args.ldg + d0};
  const uint8_t* const reset = RESET ? a.reset + b * a.L : nullptr;
  const bool whole = (a.D | ldg) % 2 == 0 &&
                     (reinterpret_cast<uintptr_t>(args.dx) | reinterpret_cast<uintptr_t>(args.dr) |
                      reinterpret_cast<uintptr_t>(args.di)) % (2 * sizeof(G)) == 0;
  const float2 h0 = state_at(a.h0, b, d, a.D);
  if constexpr (!SPLIT) {
    if (order == 0) chain.state[0][lane] = state_at(args.dhT, b, d, a.D);
  }
  float2 se = splat(0.f), sr = splat(0.f), si = splat(0.f);

  T* const ring = reinterpret_cast<T*>(smem) + warp * kTensors * run * kGroup;
  float4* const kept = reinterpret_cast<float4*>(smem + ring_bytes<T>(kTensors, 2)) +
                       warp * (run - 1) * kLanes + lane;
  auto stage = [&](int k) { return ring + k * (kWarps * kTensors * run * kGroup); };
  auto fetch = [&](int k, int t, bool on) {
    const int hi = on ? len - t : 0;
    if (hi > 0) {
      const bool all = hi >= run && left == kGroup;
      const int lo = t == 0 ? 1 : 0;  // no h before the first token
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
  int t = t_base + way.ahead, k = 0;
  fetch(0, t, way.rounds > 0);
  Channel ch;
  channel_of(a.rate, a.bias_r, a.bias_i, a.c, d, d + 1, a.D, ch);
  Resets<run, RESET> resets;
  resets.read(reset, t, len, lane);
  float2 g = splat(0.f);  // what comes from later tokens
  if constexpr (SPLIT) {
    cudaGridDependencySynchronize();  // the parts' maps are there
    g = start_of<RESET, true>(a, chain, warp, lane);
  }
  for (int round = 0; round < way.rounds; ++round, t -= step) {
    copies_wait<0>();
    __syncwarp();
    fetch(k ^ 1, t - step, round + 1 < way.rounds);
    const T* const st = stage(k) + 2 * lane;
    k ^= 1;
    const uint32_t cuts = resets.take(reset, t - step, len, lane);
    const float2 first = t == 0 ? h0 : splat(0.f);
    // g after token j is what goes on to j - 1; al and nz only where they are known
    auto finish = [&](auto known, int j, bool cut, float2 al, float2 nz, float2& dx, float2& dr, float2& di) {
      g = add2(g, pair_of(st + (3 * run + j) * kGroup));
      float2 prev = pair_of(st + (4 * run + j) * kGroup), E;
      if (j == 0) prev = add2(prev, first);
      element_grad<decltype(known)::value>(ch, pair_of(st + j * kGroup), pair_of(st + (run + j) * kGroup),
                                           pair_of(st + (2 * run + j) * kGroup), cut, prev, al, nz, g, dx,
                                           dr, di, E);
      return E;
    };
    auto sum = [&](float2 E, float2 dr, float2 di) {
      se = add2(se, E);
      sr = add2(sr, dr);
      si = add2(si, di);
    };
    auto put = [&](int j, float2 dx, float2 dr, float2 di, bool whole) {
      put_pair(out[0] + (at + j * ldg), dx, whole, in0, in1);
      put_pair(out[1] + (at + j * ldg), dr, whole, in0, in1);
      put_pair(out[2] + (at + j * ldg), di, whole, in0, in1);
    };
    auto pass = [&](const Map& m) {
      if constexpr (SPLIT) return g;
      else
        return pass_on(chain, m, cuts != 0, order, round == 0 && order == 0,
                       round == way.rounds - 1 && order == kWarps - 1, lane);
    };
    if (t + run <= len && cuts == 0) {  // most runs
      float2 a0 = splat(0.f), nz0 = a0;
      if constexpr (!SPLIT) {
        Map m = {splat(1.f), splat(0.f)};
#pragma unroll
        for (int j = run - 1; j >= 0; --j) {
          float2 al, nz;
          decay(ch, pair_of(st + (run + j) * kGroup), al, nz);
          if (j == 0) {  // the first token's need no place
            a0 = al;
            nz0 = nz;
          } else {
            kept[(j - 1) * kLanes] = make_float4(al.x, al.y, nz.x, nz.y);
          }
          m.A = mul2(al, m.A);
          m.B = mul2(al, add2(m.B, pair_of(st + (3 * run + j) * kGroup)));
        }
        g = pass(m);
      }
      auto all = [&](bool whole) {
#pragma unroll
        for (int j = run - 1; j >= 0; --j) {
          float2 al = a0, nz = nz0, dx, dr, di;
          if (!SPLIT && j > 0) {
            const float4 v = kept[(j - 1) * kLanes];
            al = make_float2(v.x, v.y);
            nz = make_float2(v.z, v.w);
          }
          const float2 E = finish(std::bool_constant<!SPLIT>{}, j, false, al, nz, dx, dr, di);
          sum(E, dr, di);
          put(j, dx, dr, di, whole);
        }
      };
      if (whole) all(true);
      else all(false);
    } else if (t >= len) {  // past the sequence's end
      if constexpr (!SPLIT) g = pass({splat(1.f), splat(0.f)});
#pragma unroll
      for (int j = 0; j < run; ++j)
        if (t + j < L) put(j, splat(0.f), splat(0.f), splat(0.f), whole);
    } else {  // a reset or the end; selects, so that the gates overlap
      if constexpr (!SPLIT) {
        Map m = {splat(1.f), splat(0.f)};
#pragma unroll
        for (int j = run - 1; j >= 0; --j) {
          const bool cut = RESET && (cuts >> j & 1), on = t + j < len;
          float2 al, nz;
          decay(ch, pair_of(st + (run + j) * kGroup), al, nz);
          const float2 A = mul2(al, m.A), B = mul2(al, add2(m.B, pair_of(st + (3 * run + j) * kGroup)));
          m.A = !on ? m.A : cut ? splat(0.f) : A;
          m.B = !on ? m.B : cut ? splat(0.f) : B;
        }
        g = pass(m);
      }
#pragma unroll
      for (int j = run - 1; j >= 0; --j) {
        const bool on = t + j < len;
        const float2 later = g, none = splat(0.f);
        float2 dx, dr, di;
        const float2 E = finish(std::false_type{}, j, RESET && (cuts >> j & 1), none, none, dx, dr, di);
        g = on ? g : later;
        dx = on ? dx : none;
        dr = on ? dr : none;
        di = on ? di : none;
        sum(on ? E : none, dr, di);
        if (t + j < L) put(j, dx, dr, di, whole);
      }
    }
#pragma unroll
    for (int j = 0; j < 3; ++j) out[j] -= step * args.ldg;
  }
  // the CTA's sums, the warps' in order, are a row of the workspace
  copies_wait<0>();
  __syncthreads();
  if constexpr (!SPLIT) g = chain.state[0][lane];
  float2(*red)[3][kLanes] = reinterpret_cast<float2(*)[3][kLanes]>(smem);
  red[warp][0][lane] = se;
  red[warp][1][lane] = sr;
  red[warp][2][lane] = si;
  __syncthreads();
  if (warp < 3) {
    float2 s = splat(0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s = add2(s, red[w][warp][lane]);
    const int64_t slot = SPLIT ? b * a.split + blockIdx.x % (uint32_t)a.split : b;
    float* const part = args.part + (3 * slot + warp) * a.D + d;
    if (in0) part[0] = s.x;
    if (in1) part[1] = s.y;
  }
  if (args.dh0 && way.part == 0 && warp == 0) {
    if (in0) args.dh0[b * a.D + d] = g.x;
    if (in1) args.dh0[b * a.D + d + 1] = g.y;
  }
}

// drate, dbias_r and dbias_i of a channel: its partial sums in a fixed order.
__global__ void __launch_bounds__(kThreads) glr_sum_kernel(const float* part, int64_t parts, int64_t D,
                                                           const float* rate, float* drate,
                                                           float* dbias_r, float* dbias_i) {
  const int64_t d = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (d >= D) return;
  float s[3] = {0.f, 0.f, 0.f};
  cudaGridDependencySynchronize();  // launched before the backward's end: its sums are there
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

// How many CTAs share a sequence's tokens, a part a warp (0: one walks its tiles): as many as fill two
// places an SM, but one an SM for a lone item.  The split pays for the maps with a second reading and a
// second working out of the gates, so it has to have CTAs enough to gain by; measured split against
// whole, us, bf16, 2048 channels (32 items a sequence, so 9, 4, 3 and 2 CTAs for 1, 2, 3 and 4
// sequences):
//   forward   1 x 256  7.9 / 6.0   1 x 512  8.0 / 9.8   1 x 2048  19 / 32   2 x 2048  31.1 / 31.7
//             3 x 2048  40 / 32    4 x 2048  55 / 32     2 x 32768 391 / 464, in fp32 600 / 533
//   backward  1 x 256 10.3 / 12.5  1 x 512 12.0 / 21.9  1 x 2048  25 / 73   2 x 2048  40 / 73
//             3 x 2048  52 / 74    4 x 2048  70 / 74    4 x 2048 in fp32 115 / 99
// A lone item of 32768 tokens in 148 or 256 CTAs: forward 13.0 / 14.3, backward 37.1 / 44.3 (32 since).
int split_of(bool back, int64_t items, int64_t L, int run) {
  const int64_t sms = current_device_sms() > 0 ? current_device_sms() : 148;
  const int64_t room = items > 1 ? 2 * sms / items : items * sms, most = L / (2 * run * kWarps);
  const int least = back ? 3 : run == kRun<__nv_bfloat16> && L >= 2048 ? 4 : 5;
  if (room < least || (!back && L < 512)) return 0;
  const int64_t n = room < most ? room : most;
  return n >= 2 ? (int)n : 0;
}
// Tokens of a part, whole runs.
int part_len_of(int64_t L, int split, int run) {
  const int64_t parts = (int64_t)split * kWarps, n = (L + parts - 1) / parts;
  return (int)((n + run - 1) / run * run);
}
int run_of(bool bf16) { return bf16 ? kRun<__nv_bfloat16> : kRun<float>; }
int64_t items_of(int64_t b, int64_t D) { return b * ((D + kGroup - 1) / kGroup); }

// `early`: the kernel may begin before the one before it in the stream ends; it waits itself.
template <auto KERNEL, typename... A>
cudaError_t launch(int64_t grid, int threads, int smem, bool early, cudaStream_t s, A... args) {
  cudaError_t e = smem > 0 ? allow_shared<KERNEL>(smem) : cudaSuccess;
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = early ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, KERNEL, args...);
  return e != cudaSuccess ? e : cudaGetLastError();
}
constexpr int kCta = kWarps * kLanes;

template <typename T, int MODE, bool RESET>
cudaError_t fwd_m(const GlrArgs& a, cudaStream_t s) {
  const int64_t items = items_of(a.b, a.D);
  const int smem = ring_bytes<T>(3, kStages);
  if (!a.split) return launch<glr_fwd_kernel<T, MODE, RESET, false>>(items, kCta, smem, false, s, a);
  const cudaError_t e = launch<glr_part_kernel<T, MODE, RESET, false>>(items * a.split, kCta,
                               smem, false, s, a, (const void*)nullptr, a.h0);
  if (e != cudaSuccess) return e;
  return launch<glr_fwd_kernel<T, MODE, RESET, true>>(items * a.split, kCta, smem, true, s, a);
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

template <typename T, typename G, int MODE, bool RESET>
cudaError_t bwd_m(const GlrBwdArgs& a, cudaStream_t s) {
  const GlrArgs& f = a.f;
  const int64_t items = items_of(f.b, f.D);
  const int smem = ring_bytes<T>(5, 2);
  // the decays of all but one token a run fit beside the ring twice an SM
  const int kept = kWarps * (kRun<T> - 1) * kLanes * (int)sizeof(float4);
  if (!f.split)
    return launch<glr_bwd_kernel<T, G, MODE, RESET, false>>(items, kCta, smem + kept, false, s, a);
  const cudaError_t e = launch<glr_part_kernel<T, MODE, RESET, true>>(items * f.split,
                               kShare<T, true> * kCta, kShare<T, true> * ring_bytes<T>(2, kStages), false,
                               s, f, a.dy, a.dhT);
  if (e != cudaSuccess) return e;
  return launch<glr_bwd_kernel<T, G, MODE, RESET, true>>(items * f.split, kCta, smem, true, s, a);
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

void set_split(GlrArgs& a, bool back, void* maps) {
  a.split = split_of(back, items_of(a.b, a.D), a.L, run_of(a.bf16));
  a.part_len = a.split ? part_len_of(a.L, a.split, run_of(a.bf16)) : 0;
  a.maps = maps;
}
// The backward's workspace: the split's maps, then the partial sums.
size_t al256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

size_t glr_fwd_workspace_bytes(int64_t b, int64_t L, int64_t D, bool bf16) {
  const int64_t items = items_of(b, D);
  return split_bytes(items, split_of(false, items, L, run_of(bf16)));
}

cudaError_t launch_glr_fwd(const GlrArgs& args, void* workspace, cudaStream_t s) {
  GlrArgs a = args;
  set_split(a, false, workspace);
  return a.bf16 ? fwd_t<__nv_bfloat16>(a, s) : fwd_t<float>(a, s);
}

size_t glr_bwd_workspace_bytes(int64_t b, int64_t L, int64_t D, bool bf16) {
  const int64_t items = items_of(b, D);
  const int split = split_of(true, items, L, run_of(bf16));
  return al256(split_bytes(items, split)) +
         (size_t)b * (size_t)(split ? split : 1) * 3 * (size_t)D * sizeof(float);
}

cudaError_t launch_glr_bwd(const GlrBwdArgs& args, void* workspace, cudaStream_t s) {
  GlrBwdArgs a = args;
  GlrArgs& f = a.f;
  set_split(f, true, workspace);
  a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                    al256(split_bytes(items_of(f.b, f.D), f.split)));
  if (f.b > 0) {
    const cudaError_t e = !f.bf16         ? bwd_t<float, float>(a, s)
                          : a.grad_bf16 ? bwd_t<__nv_bfloat16, __nv_bfloat16>(a, s)
                                        : bwd_t<__nv_bfloat16, float>(a, s);
    if (e != cudaSuccess) return e;
  }
  return launch<glr_sum_kernel>(grid_for(f.D), kThreads, 0, true, s, (const float*)a.part,
                                (int64_t)(f.b * (f.split ? f.split : 1)), (int64_t)f.D, f.rate,
                                a.drate, a.dbias_r, a.dbias_i);
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
