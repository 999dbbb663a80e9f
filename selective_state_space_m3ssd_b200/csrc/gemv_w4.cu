// The product of a few tokens with 4-bit weights whose groups of columns have a bf16 scale (and a
// zero point), and the weights into that form and back.
//
//     out[m][n] = sum over groups j of scale[j][n] sum over j's k of x[m][k] (code[n][k] - zero[j][n]).
//
// The codes are read once, and HBM bounds the product from about a million weights on; below, it is
// latency.  A warp takes tiles of 16 rows by 128 columns, 1 KB of codes that its lanes read as two
// 16-byte words each, in the order that a lane needs them as an operand of the (legacy) warp-wide
// bf16 product of 16 x 16 weights by 16 x 8 tokens: the k order within a product is free as long as
// both operands share it.  Codes masked out of a word are read as bf16 numbers as they are: bits 0 to 7
// of one are linear, n 2^-133, through its subnormals and first binade, so one multiply-add makes
// (n - zero) 2^-6 of it, exactly, wherever in those bits the code lies, and nothing is rounded
// before the products' fp32 sums; a group's sums are scaled in fp32, and the 2^6 comes last.  tcgen05
// is not for this: its operands would have to go through shared or tensor memory, and the products
// keep the tensor pipe busy for a quarter of the time only.
//
// Measured: 8 tokens x 65536 x 4096 in groups of 64 with zero points (149 MB) 34.6 us, 4.3 TB/s; one token
// 30.3 us without zero points; 16 tokens 58 us (two products a word, fewer warps: the tokens' operands
// come from shared memory for every tile).  1 x 6464 x 1024 3.4 us: a launch, one read of codes after
// another of tokens and scales, a join.
//
// fp32 tokens are three bf16 columns each, their leading 8 bits, the next and the last: exact from 2^-110 on;
// below, the last ones pass bf16's least number, 2^-133, and what is under it is dropped.
// A CTA's warps are WR groups of rows by WK parts of K, joined in shared memory in a fixed
// order; the tokens lie there too, a piece of K at a time.
#include <cuda_runtime.h>

#include <cstdint>
#include <initializer_list>

#include "common.cuh"
#include "internal.h"

namespace m3ssd {
namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32;  // of the kernels that lay weights out
constexpr int kTileRows = 16, kTileCols = 128, kTileBytes = 1024;
constexpr int kRedRow = kTileRows + 1;

// Tiles of codes in a warp's ring, copied ahead.
constexpr int kDeep = 3;

__device__ __forceinline__ void copy_codes(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src));
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 load_shared(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}

__device__ __forceinline__ uint32_t load_shared1(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

// The pairs of codes (i, i + 4), i = 0 to 3, of a word of eight, less the zero point, as bf16 pairs of
// (code - zero) / 64; `offset` is -zero / 64 twice.
__device__ __forceinline__ uint32_t scaled(uint32_t codes, uint32_t by, uint32_t offset) {
  uint32_t o;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(o) : "r"(codes), "r"(by), "r"(offset));
  return o;
}
constexpr float kUnit = 64.f;
__device__ __forceinline__ void decode(uint32_t w, uint32_t offset, uint32_t (&o)[4]) {
  const uint32_t v = w >> 8, low = 0x7f007f00u, high = 0x7d007d00u;  // 2^127, 2^123
  o[0] = scaled(w & 0x000f000fu, low, offset);
  o[1] = scaled(w & 0x00f000f0u, high, offset);
  o[2] = scaled(v & 0x000f000fu, low, offset);
  o[3] = scaled(v & 0x00f000f0u, high, offset);
}

// d += a b, or d = a b where NEW.
template <bool NEW>
__device__ __forceinline__ void product(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  if constexpr (NEW)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Eight consecutive values of a token, from column k of K on (zeros past it), go to shared memory as
// the pairs (i, i + 4).
__device__ __forceinline__ uint32_t low_halves(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x5410); }
__device__ __forceinline__ uint32_t high_halves(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7632); }
__device__ __forceinline__ void stage_eight(const __nv_bfloat16* x, int k, int K, bool wide, char* to, int) {
  uint4 u;
  if (wide && k + 8 <= K) {
    u = *reinterpret_cast<const uint4*>(x + k);
  } else {
    const uint16_t* const p = reinterpret_cast<const uint16_t*>(x);
    uint32_t h[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = k + j < K ? p[k + j] : 0;
    u = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
  }
  *reinterpret_cast<uint4*>(to) = make_uint4(low_halves(u.x, u.z), high_halves(u.x, u.z),
                                             low_halves(u.y, u.w), high_halves(u.y, u.w));
}
// fp32: three columns `stride` bytes apart, each value's leading bf16 part (its high half), that of the rest,
// and the last, which leaves nothing (of a value below 2^-110 less than 2^-133).  What is not finite has no
// further parts.
__device__ __forceinline__ void stage_eight(const float* x, int k, int K, bool wide, char* to, int stride) {
  float v[8];
  if (wide && k + 8 <= K) {
    const float4 a = *reinterpret_cast<const float4*>(x + k), b = *reinterpret_cast<const float4*>(x + k + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = k + j < K ? x[k + j] : 0.f;
  }
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    uint32_t h[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      h[j] = __float_as_uint(v[j]) & 0xffff0000u;
      if ((h[j] & 0x7f800000u) == 0x7f800000u) {
        if (v[j] != v[j]) h[j] = 0x7fc00000u;  // a NaN whose high bits alone might read as infinity
        v[j] = 0.f;
      } else {
        v[j] -= __uint_as_float(h[j]);
      }
    }
    *reinterpret_cast<uint4*>(to + p * stride) = make_uint4(high_halves(h[0], h[4]), high_halves(h[1], h[5]),
                                                            high_halves(h[2], h[6]), high_halves(h[3], h[7]));
  }
}
// A piece of the tokens: for each part of K the columns of `per` (a power of two) tiles from the part's
// tile number `first` on.
template <typename X>
__device__ __forceinline__ void stage_tokens(const GemvW4Args& a, const X* x, int first, int stride,
                                             char* smem) {
  const int in_part = 31 - __clz(a.per * (kTileCols / 8)), in_token = in_part + (31 - __clz(a.wk));
  const int all = (int)a.M << in_token;
#pragma unroll 4
  for (int i = threadIdx.x; i < all; i += blockDim.x) {
    const int m = i >> in_token, q = i & ((1 << in_token) - 1);
    const int k = ((q >> in_part) * a.part + first) * kTileCols + 8 * (q & ((1 << in_part) - 1));
    stage_eight(x + m * a.ldx, k, (int)a.K, a.wide, smem + m * (sizeof(X) == 2 ? 1 : 3) * stride + q * 16,
                stride);
  }
}

// The words of scales and zero points of the same tiles, `G` a tile (a longer group's in each of its
// tiles), for `rows` rows from row0 on: the scale above -zero / 64, both bf16.
template <int G, bool ZEROS>
__device__ __forceinline__ void stage_words(const GemvW4Args& a, int first, int64_t row0, int rows,
                                            uint32_t* to) {
  const int eights = rows / 8, in_part = 31 - __clz(a.per);  // of rows; tiles
  const bool wide = a.wide_scales && row0 + rows <= a.N;
#pragma unroll 2
  for (int i = threadIdx.x; i < a.wk * a.per * G * eights; i += blockDim.x) {
    const int e = __umulhi(i, a.over_eights), r = 8 * (i - e * eights);
    const int place = e / G, tile = (place >> in_part) * a.part + first + (place & (a.per - 1));
    const int j = G > 1 ? tile * G + e % G : a.group_tiles == 1 ? tile : tile / a.group_tiles;
    const int64_t at = j * a.N + row0 + r;
    uint32_t s[4] = {0, 0, 0, 0}, z[2] = {0, 0};
    if (j < a.groups) {
      if (wide) {
        const uint4 v = *reinterpret_cast<const uint4*>(a.scales + at);
        s[0] = v.x, s[1] = v.y, s[2] = v.z, s[3] = v.w;
        if (ZEROS) {
          const uint2 u = *reinterpret_cast<const uint2*>(a.zeros + at);
          z[0] = u.x, z[1] = u.y;
        }
      } else {
#pragma unroll
        for (int h = 0; h < 8; ++h) {
          const bool in = row0 + r + h < a.N;
          s[h / 2] |= in ? (uint32_t)a.scales[at + h] << (16 * (h & 1)) : 0u;
          if (ZEROS) z[h / 4] |= in ? (uint32_t)a.zeros[at + h] << (8 * (h & 3)) : 0u;
        }
      }
    }
    uint32_t w[8];
#pragma unroll
    for (int h = 0; h < 8; ++h) {
      // eight bits are exact in bf16: the high half of the fp32 number
      const uint32_t low =
          ZEROS ? __float_as_uint((float)(z[h / 4] >> (8 * (h & 3)) & 0xffu) * (-1.f / kUnit)) >> 16 : 0u;
      w[h] = __byte_perm(low, s[h / 2], h & 1 ? 0x7610 : 0x5410);
    }
    uint4* const out = reinterpret_cast<uint4*>(to + e * rows + r);
    out[0] = make_uint4(w[0], w[1], w[2], w[3]);
    out[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// Warps that an SM holds, by the registers of the sums: 64 a thread for eight columns, 80 for 16, 128 for
// more (with 8 warps of as many registers as they like 16 fp32 tokens x 16384 x 4096 took 61 us, so 42).
template <int NT>
constexpr int kSmWarps = NT == 1 ? 32 : NT == 2 ? 24 : 16;

// X: the tokens' type; NT: eights of columns (tokens, or thirds of them); W: warps of a CTA; G: groups in a
// tile; ZEROS: zero points given.
template <typename X, int NT, int W, int G, bool ZEROS>
__global__ void __launch_bounds__(W * 32, kSmWarps<NT> / W) gemv_w4_kernel(GemvW4Args a) {
  extern __shared__ __align__(16) char smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int WK = a.wk, WR = W / WK, wk = warp % WK, wr = warp / WK;
  // The CTA's rows of tiles: `mine`, at most WR, from row0 / 16 on.
  const int mine = (int)a.each + (blockIdx.x < a.more);
  const int64_t row0 = (blockIdx.x * a.each + min((int64_t)blockIdx.x, a.more)) * kTileRows;
  const int64_t rb = row0 / kTileRows + wr;
  const bool live = wr < mine;
  const int KB = (int)a.KB, per = a.per, chunk = per * WK;  // tiles: of K, of a warp and of a CTA a piece
  const int cols = a.cols, stride = chunk * kTileCols * 2 + 64;  // bytes of a column in shared memory

  const uint32_t smem_addr = (uint32_t)__cvta_generic_to_shared(smem);
  // The rows' scales and zero points of a piece, after the tokens: a word for each group of a tile (for
  // each tile, where groups are longer) and row of the CTA's.
  const int rows = kTileRows * WR, words_at = cols * stride;

  // The warp's tiles: `tiles` from number wk a.part of K on, `left` of them still to be copied.  A lane
  // copies what it reads: 16 bytes of row g, and of row g + 8.
  char* const ring = smem + words_at + chunk * G * rows * 4 + (warp * kDeep * 2 * 32 + lane) * 16;
  const uint32_t ring_addr = (uint32_t)__cvta_generic_to_shared(ring);
  const int tiles = live ? max(min(KB - wk * a.part, a.part), 0) : 0;
  int left = tiles;
  const uint8_t* codes = a.codes + ((live ? rb : 0) * KB + wk * a.part) * kTileBytes + lane * 16;
  auto copy = [&](int d) {  // d: bytes
    if (left > 0) {
      copy_codes(ring_addr + d, codes);
      copy_codes(ring_addr + d + 512, codes + 512);
    }
    copies_end();
    left -= 1;
    codes += kTileBytes;
  };
#pragma unroll
  for (int d = 0; d < kDeep - 1; ++d) copy(d * kTileBytes);

  float acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;

  // Lanes of columns that are not there read the last one: what they make of it is dropped.
  uint32_t xs[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n)
    xs[n] = smem_addr + min(8 * n + g, cols - 1) * stride + t * 16;
  const uint32_t words = smem_addr + words_at + (wr * kTileRows + g) * 4;
  auto use = [&](int d, int at) {  // the ring's tile at byte d; `at`: the tile's place in the piece
    const uint4 vlo = *reinterpret_cast<const uint4*>(ring + d);
    const uint4 vhi = *reinterpret_cast<const uint4*>(ring + d + 512);
    const uint32_t lo[4] = {vlo.x, vlo.y, vlo.z, vlo.w}, hi[4] = {vhi.x, vhi.y, vhi.z, vhi.w};
    float sum[NT][4];
    uint32_t w0 = 0, w1 = 0, off0 = 0xbe00be00u, off1 = off0;  // -8 / 64
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      constexpr int per_group = 4 / G;
      if (j % per_group == 0) {
        const uint32_t from = words + (at * G + j / per_group) * rows * 4;
        w0 = load_shared1(from);
        w1 = load_shared1(from + 32);
        if (ZEROS) {
          off0 = __byte_perm(w0, w0, 0x1010);
          off1 = __byte_perm(w1, w1, 0x1010);
        }
      }
      uint32_t p[4], q[4];
      decode(lo[j], off0, p);
      decode(hi[j], off1, q);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint4 b = load_shared(xs[n] + at * kTileCols * 2 + j * 64);
        if (j % per_group == 0)
          product<true>(sum[n], p[0], q[0], p[1], q[1], b.x, b.y);
        else
          product<false>(sum[n], p[0], q[0], p[1], q[1], b.x, b.y);
        product<false>(sum[n], p[2], q[2], p[3], q[3], b.z, b.w);
      }
      if (j % per_group == per_group - 1) {
        const float s0 = __uint_as_float(ZEROS ? w0 & 0xffff0000u : w0);
        const float s1 = __uint_as_float(ZEROS ? w1 & 0xffff0000u : w1);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          acc[n][0] = fmaf(s0, sum[n][0], acc[n][0]);
          acc[n][1] = fmaf(s0, sum[n][1], acc[n][1]);
          acc[n][2] = fmaf(s1, sum[n][2], acc[n][2]);
          acc[n][3] = fmaf(s1, sum[n][3], acc[n][3]);
        }
      }
    }
  };
  int d = 0;  // the ring's tile that is used next; the one before it is free
  for (int first = 0; first < a.part; first += per) {
    if (first > 0) __syncthreads();
    stage_tokens(a, static_cast<const X*>(a.x), first, stride, smem);
    stage_words<G, ZEROS>(a, first, row0, rows,
                          reinterpret_cast<uint32_t*>(smem + words_at));
    __syncthreads();
    const int n = min(tiles - first, per);
    for (int at = 0; at < n; ++at) {
      copies_wait<kDeep - 2>();
      copy(d == 0 ? (kDeep - 1) * kTileBytes : d - kTileBytes);
      use(d, wk * per + at);
      d = d == (kDeep - 1) * kTileBytes ? 0 : d + kTileBytes;
    }
  }
  copies_wait<0>();

  // the tile's sums: over the parts of K, and of a token
  __syncthreads();
  float* const red = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int col = 8 * n + 2 * t + (e & 1), r = g + 8 * (e >> 1);
      if (col < cols) red[(warp * cols + col) * kRedRow + r] = acc[n][e];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < mine * (int)a.M * kTileRows; i += W * 32) {
    const int r = i % kTileRows, m = i / kTileRows % (int)a.M, w = i / kTileRows / (int)a.M;
    const int64_t n = row0 + w * kTileRows + r;
    if (n >= a.N) continue;
    float s = 0.f;
    for (int p = 0; p < a.parts; ++p)
      for (int k = 0; k < WK; ++k)
        s += red[((w * WK + k) * cols + m * a.parts + p) * kRedRow + r];
    s *= kUnit;
    if (a.out_bf16)
      static_cast<__nv_bfloat16*>(a.out)[m * a.ldd + n] = __float2bfloat16_rn(s);
    else
      static_cast<float*>(a.out)[m * a.ldd + n] = s;
  }
}

// Where column k of row r lies in the codes: the byte, and whether it is the high half.
__device__ __forceinline__ int64_t code_byte(int64_t r, int64_t k, int64_t KB) {
  const int rr = (int)(r % kTileRows), c = (int)(k % kTileCols);
  return (r / kTileRows * KB + k / kTileCols) * kTileBytes + 512 * (rr / 8) + 64 * (rr % 8) +
         16 * (c / 8 % 4) + 4 * (c / 32) + c % 8 / 2;
}

// A warp quantises a group of a row (rows of the last tile that are not there: codes of zero).  Lane l takes
// pairs of columns, 64 columns a step.
template <typename T>
__global__ void __launch_bounds__(kThreads) w4_quant_kernel(W4Args a, const T* w, int64_t ldw) {
  const int64_t rows = (a.N + kTileRows - 1) / kTileRows * kTileRows, KB = (a.K + kTileCols - 1) / kTileCols;
  const int64_t span = (KB * kTileCols + a.group - 1) / a.group;  // groups, the padding's too
  const int64_t id = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (id >= rows * span) return;
  const int lane = threadIdx.x & 31;
  const int64_t r = id / span, j = id % span, k0 = j * a.group, k1 = min(k0 + a.group, KB * kTileCols);
  const bool there = r < a.N;
  float lo = 0.f, hi = 0.f;
  bool finite = true;
  for (int64_t k = k0 + lane; k < min(k1, a.K); k += 32) {
    const float v = there ? to_f32(w[r * ldw + k]) : 0.f;
    finite &= fabsf(v) < INFINITY;
    lo = fminf(lo, v);
    hi = fmaxf(hi, v);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  finite = __all_sync(0xffffffffu, finite);
  // halves first: the range of the largest values overflows
  const __nv_bfloat16 scale =
      __float2bfloat16_rn(!finite    ? NAN
                          : a.zeros ? 2.f * ((0.5f * hi - 0.5f * lo) / 15.f)
                                    : fmaxf(hi, -lo) / 7.f);
  const float s = to_f32(scale);
  const bool some = s > 0.f;  // not of zeros, not NaN
  const float zero = !a.zeros ? 8.f : some ? fminf(fmaxf(rintf(-lo / s), 0.f), 15.f) : 0.f;
  if (there && j < a.groups && lane == 0) {
    a.scales[j * a.N + r] = __bfloat16_as_ushort(scale);
    if (a.zeros) a.zeros[j * a.N + r] = (uint8_t)zero;
  }
  for (int64_t k = k0 + 2 * lane; k < k1; k += 64) {
    uint32_t c[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float v = there && some && k + e < a.K ? to_f32(w[r * ldw + k + e]) / s : 0.f;
      c[e] = (uint32_t)fminf(fmaxf(rintf(v) + zero, 0.f), 15.f);
    }
    a.codes[code_byte(r, k, KB)] = (uint8_t)(c[0] | c[1] << 4);
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) w4_dequant_kernel(W4Args a, T* w, int64_t ldw) {
  const int64_t pairs = (a.K + 1) / 2, KB = (a.K + kTileCols - 1) / kTileCols;
  for (int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x; id < a.N * pairs;
       id += (int64_t)gridDim.x * kThreads) {
    const int64_t r = id / pairs, k = id % pairs * 2, j = k / a.group;
    const uint32_t c = a.codes[code_byte(r, k, KB)];
    const float s = __uint_as_float((uint32_t)a.scales[j * a.N + r] << 16);
    const float z = a.zeros ? (float)a.zeros[j * a.N + r] : 8.f;
    w[r * ldw + k] = from_f32<T>(((float)(c & 15) - z) * s);
    if (k + 1 < a.K) w[r * ldw + k + 1] = from_f32<T>(((float)(c >> 4) - z) * s);
  }
}

// What the tokens' pieces may take of an SM's shared memory, and the most that an SM's CTAs ask for: the
// tokens' piece, the scales of its tiles and the ring.
constexpr int kStageBytes = 144 * 1024, kMostShared = 200 * 1024;

template <typename X, int NT, int W, int G, bool ZEROS>
cudaError_t run(GemvW4Args a, cudaStream_t s) {
  constexpr int ctas = kSmWarps<NT> / W;
  const int64_t sms = current_device_sms() > 0 ? current_device_sms() : 148, places = sms * ctas;
  // Shared memory for pieces of `per` tiles of each of `wk` parts of K.
  auto tokens = [&](int per, int wk) { return a.cols * (per * wk * kTileCols * 2 + 64); };
  auto held = [&](int per, int wk) {
    return tokens(per, wk) + per * wk * G * (W / wk) * kTileRows * 4 + W * kDeep * kTileBytes;
  };
  // Parts of K: as many as leave no more CTAs than all SMs hold at once (every one stages all tokens).
  a.wk = 1;
  for (int wk = 2; W % wk == 0 && wk <= a.KB && (a.RB * wk + W - 1) / W <= places; wk *= 2)
    if (held(1, wk) <= kMostShared / ctas) a.wk = wk;
  // A part's tiles, and a power of two of them in a piece: all, as far as the piece's tokens fit.
  a.part = (int)((a.KB + a.wk - 1) / a.wk);
  a.per = 1;
  const int64_t wr = W / a.wk;
  a.over_eights = (uint32_t)(((int64_t(1) << 32) + 2 * wr - 1) / (2 * wr));
  while (a.per < 16 && a.per < a.part && tokens(2 * a.per, a.wk) <= kStageBytes / ctas &&
         held(2 * a.per, a.wk) <= kMostShared / ctas)
    a.per *= 2;
  const int sums = W * a.cols * kRedRow * (int)sizeof(float);
  const int smem = held(a.per, a.wk) > sums ? held(a.per, a.wk) : sums;
  if (smem > kMostShared) return cudaErrorInvalidValue;
  const cudaError_t e = allow_shared<gemv_w4_kernel<X, NT, W, G, ZEROS>>(kMostShared);
  if (e != cudaSuccess) return e;
  // As many CTAs for every SM, some of whose warps have no row, rather than SMs that have no CTA: 8 x 65536 x
  // 4096 in 148 CTAs of 27 or 28 warps 34.3 us, in 128 of 32 36.6.
  const int64_t need = (a.RB + wr - 1) / wr, even = (need + sms - 1) / sms * sms;
  const int64_t grid = even < a.RB ? even : a.RB;
  a.each = a.RB / grid;
  a.more = a.RB % grid;
  gemv_w4_kernel<X, NT, W, G, ZEROS><<<(unsigned)grid, W * 32, smem, s>>>(a);
  return cudaGetLastError();
}
template <typename X, int NT, int W>
cudaError_t run_g(const GemvW4Args& a, cudaStream_t s) {
  if (a.zeros)
    return a.group == 32   ? run<X, NT, W, 4, true>(a, s)
           : a.group == 64 ? run<X, NT, W, 2, true>(a, s)
                           : run<X, NT, W, 1, true>(a, s);
  return a.group == 32   ? run<X, NT, W, 4, false>(a, s)
         : a.group == 64 ? run<X, NT, W, 2, false>(a, s)
                         : run<X, NT, W, 1, false>(a, s);
}
// Every CTA stages all the tokens of its part of K.  Few tokens: CTAs of eight warps, which start and join
// sooner; from 12 KB of them on one CTA an SM, which stages them once for all its warps.  Measured, us, eight
// warps against one CTA (tokens x rows x K): 1 x 2048 x 2048 3.0 / 4.1, 1 x 6464 x 1024 3.4 / 4.0, fp32
// 4.0 / 4.6, 3 x 20001 x 1000 7.4 / 8.7; 1 x 8192 x 8192 (16 KB) 12.2 / 11.2, 5 x 6464 x 1024 fp32 6.2 / 5.7,
// 8 x 8192 x 8192 (groups of 32) 31 / 17, 16 x 8192 x 8192 42 / 29, 8 x 65536 x 4096 42 / 37.
template <typename X, int NT>
cudaError_t run_w(const GemvW4Args& a, cudaStream_t s) {
  return a.cols * a.K * 2 >= 12 * 1024 ? run_g<X, NT, kSmWarps<NT>>(a, s) : run_g<X, NT, 8>(a, s);
}

}  // namespace

cudaError_t launch_gemv_w4(const GemvW4Args& args, cudaStream_t s) {
  GemvW4Args a = args;
  a.parts = a.x_bf16 ? 1 : 3;
  a.cols = (int)a.M * a.parts;
  a.RB = (a.N + kTileRows - 1) / kTileRows;
  a.KB = (a.K + kTileCols - 1) / kTileCols;
  a.group_tiles = a.group < kTileCols ? 1 : (int)(a.group / kTileCols);
  a.wide_scales = a.N % 8 == 0 && reinterpret_cast<uintptr_t>(a.scales) % 16 == 0 &&
                  reinterpret_cast<uintptr_t>(a.zeros) % 8 == 0;
  a.wide = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && a.ldx % (a.x_bf16 ? 8 : 4) == 0;
  const int nt = (a.cols + 7) / 8;
  if (a.x_bf16) return nt == 1 ? run_w<__nv_bfloat16, 1>(a, s) : run_w<__nv_bfloat16, 2>(a, s);
  return nt == 1   ? run_w<float, 1>(a, s)
         : nt == 2 ? run_w<float, 2>(a, s)
         : nt <= 4 ? run_w<float, 4>(a, s)
                   : run_w<float, 6>(a, s);
}

cudaError_t launch_w4_quant(const W4Args& a, bool bf16, const void* w, int64_t ldw, cudaStream_t s) {
  const int64_t rows = (a.N + kTileRows - 1) / kTileRows * kTileRows;
  const int64_t cols = (a.K + kTileCols - 1) / kTileCols * kTileCols, span = (cols + a.group - 1) / a.group;
  const unsigned grid = (unsigned)((rows * span + kWarps - 1) / kWarps);
  if (bf16)
    w4_quant_kernel<<<grid, kThreads, 0, s>>>(a, static_cast<const __nv_bfloat16*>(w), ldw);
  else
    w4_quant_kernel<<<grid, kThreads, 0, s>>>(a, static_cast<const float*>(w), ldw);
  return cudaGetLastError();
}

cudaError_t launch_w4_dequant(const W4Args& a, bool bf16, void* w, int64_t ldw, cudaStream_t s) {
  const int64_t n = a.N * ((a.K + 1) / 2), want = (n + kThreads - 1) / kThreads;
  const unsigned grid = (unsigned)(want < 148 * 32 ? want : 148 * 32);
  if (bf16)
    w4_dequant_kernel<<<grid, kThreads, 0, s>>>(a, static_cast<__nv_bfloat16*>(w), ldw);
  else
    w4_dequant_kernel<<<grid, kThreads, 0, s>>>(a, static_cast<float*>(w), ldw);
  return cudaGetLastError();
}

}  // namespace m3ssd
