// Product of microscaled operands on the sm_100a tensor cores:
//     D (M x N, bf16, row-major, row stride ldd) = A (M x K) W^T,
// with A in E2M1 or E4M3 codes and W (N x K) in E2M1 codes, blocks of 32 along K with a
// power-of-two scale each (mx.cuh), and fp32 accumulation in tensor memory.  The tensor
// cores apply the scales: an operand's codes go from global to shared memory by TMA, its
// scales by one bulk copy a 512-byte tile and from there into TMEM (tcgen05.cp), and
// kind::mxf4 (A in 4 bits) or kind::mxf8f6f4 (A in 8 bits; TMA spreads the packed 4-bit
// codes of W over 8-bit containers as it loads them) multiplies value times scale.
//
// A tile is 128 rows of A by BN of W.  One persistent CTA per SM; warp 0 copies, warp 1
// issues the scale copies and the products, four are the epilogue.  The
// accumulators alternate where two fit beside the scales in TMEM; with one, the epilogue's
// first step, the whole row into registers as bf16, is all the products wait for.  Every stage
// of the ring has its own TMEM columns for its scales: they are free when the stage is (the
// products that read them have finished), so a copy never overtakes a product.  A 192-column
// tile may start in the middle of a scale tile: its products read the columns from there on.
// Few tokens, or few tiles with a long K, go to gemm_mx_split.cu.
// Output blocks of 32 x 64 leave by TMA from a swizzled staging buffer (a thread holds a row:
// stores straight from the registers touch 32 lines each), or, where the rows of D are not
// multiples of 16 bytes, row by row from the same buffer.
//
// The two warps stay converged and one elected lane issues: in a branch of one lane the
// compiler cannot keep descriptors and addresses in uniform registers, and the issue of a
// stage was what bounded the products (8192^3 in 4 bits 241 us against 191, 32768 x 6464 x
// 1024 131 against 120).
//
// What bounds it on one B200: writing D where K is short (32768 x 6464 x 1024: 108 us for writes
// at HBM's 3.9 TB/s of them, 120 taken at 1965 MHz; called for seconds, 1000 W hold the SM clock
// near 1510 MHz and it takes 144, so what the SMs do is close behind); with a long K what the
// copies bring in against what the products read: the ring takes in 50 to 55 bytes a cycle and SM,
// 75 to 96 would keep the products at their peak. Measured and not kept: L2 prefetches of the
// stages behind the ring (3 to 8 % slower); pairs of CTAs (256 x 256, W brought in once for both;
// no second accumulator of that width fits beside the scales, one of 192 columns would): with
// pairs 180 and 338 us at 8192^3 against 195 and 353, 36.0 and 55.2 at 32768 x 1024 x 2048 against
// 34.4 and 56.4, 137 and 187 at 32768 x 6464 x 1024 against 119 and 191.
//
// Waits are bounded as in gemm.cu: one that runs out sets a shared flag that ends the
// others, and the launch is counted in a device word the host query reads.
#include <cstddef>
#include <cstring>

#include "gemm_mx.cuh"
#include "internal.h"

namespace m3ssd {

__device__ unsigned int g_gemm_mx_wait_timeouts;

namespace {

using namespace gemm_mx;

constexpr uint32_t kStgBytes = 32 * 128;  // an output block: 32 rows x 64 bf16 columns

// AF: A's format.  A stage is 128 bytes of K a row: 256 values in 4 bits, 128 in 8.
template <int AF, int BN>
struct Cfg {
  static constexpr int ATOMS = AF == mx::kFp4 ? 2 : 1;  // scale tiles along K a stage
  static constexpr int NSB = (BN + 127) / 128;          // scale tiles along the columns
  static constexpr int EPI_WARPS = 4, THREADS = 32 * (2 + EPI_WARPS);
  static constexpr uint32_t A_BYTES = BM * 128, W_BYTES = BN * 128;
  // bytes the copies of a stage count on its barrier: W's 4-bit codes count as they are in
  // global memory, whether or not they are spread
  static constexpr uint32_t W_ROW_TX = AF != mx::kFp4 ? 64 : 128;
  static constexpr uint32_t SA_BYTES = ATOMS * kTile, SW_BYTES = NSB * ATOMS * kTile;
  static constexpr int STAGE = A_BYTES + W_BYTES + SA_BYTES + SW_BYTES;
  static constexpr int ROOM = 226 * 1024 - EPI_WARPS * (int)kStgBytes - 1024;
  static constexpr int STAGES = ROOM / STAGE < 8 ? ROOM / STAGE : 8;
  static constexpr int SF_COLS = ATOMS * 4 * (1 + NSB);  // TMEM columns of a stage's scales
  // two accumulators, where they fit, alternate between the products and the epilogue
  static constexpr int NACC = 2 * BN + STAGES * SF_COLS <= 512 ? 2 : 1;
  static constexpr int COLS = NACC * BN + STAGES * SF_COLS;
  static constexpr uint32_t TMEM_COLS = COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
  static_assert(COLS <= 512, "tensor memory");
  static_assert(EPI_WARPS * (BN / 64) * (int)kStgBytes <= STAGES * (int)(A_BYTES + W_BYTES),
                "the last item's staging");
  // operand formats of the instruction descriptor (kind::mxf4: E2M1 = 1; kind::mxf8f6f4:
  // E4M3 = 0, E2M1 = 5)
  static constexpr uint32_t FA = AF == mx::kFp4 ? 1 : 0, FW = AF == mx::kFp4 ? 1 : 5;
  static constexpr uint32_t IDESC = tc5::idesc_mx(BM, 0, FA, FW);  // the columns are ORed in
};

template <typename C>
struct Smem {
  // every buffer a TMA copy reads or writes starts on a 1024-byte boundary
  uint8_t a[C::STAGES][C::A_BYTES];
  uint8_t w[C::STAGES][C::W_BYTES];
  uint8_t stg[C::EPI_WARPS][kStgBytes];
  uint8_t sa[C::STAGES][C::SA_BYTES];
  uint8_t sw[C::STAGES][C::SW_BYTES];
  uint64_t full[C::STAGES];
  uint64_t empty[C::STAGES];
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint64_t drain;
  uint32_t tmem;
  uint32_t err;
};

struct MMaps {
  CUtensorMap a, w;  // codes, boxes of 128 bytes x 128 and BN rows
  CUtensorMap w64;   // W's in boxes of 64 rows
  CUtensorMap d;     // bf16 (N, M) with row stride ldd, box 64 x 32, 128-byte swizzle (when vec)
};

// What a CTA takes of D: rows of tile row mb, w columns from col0.  Tiles up to `full` whole,
// then the parts of the others.
struct Tiles {
  int nt;           // tiles along N
  int full, items;  // tiles taken whole; those and the parts of the others
  int parts, pw;    // parts of a tile, columns of a part
};
struct Item {
  int mb, col0, w;
};
template <int BN>
__device__ __forceinline__ Item item_of(const Tiles& g, int t) {
  if (t < g.full) return {t / g.nt, t % g.nt * BN, BN};
  const int u = t - g.full, tile = g.full + u / g.parts, c = u % g.parts * g.pw;
  return {tile / g.nt, tile % g.nt * BN + c, min(g.pw, BN - c)};
}

struct MArgs {
  int M, N;  // of D
  int64_t ldd;
  __nv_bfloat16* D;
  const uint8_t *sa, *sw;  // scales
  Tiles tiles;             // the items of the CTAs
  int nkb;                 // 128-column groups of K
  int nb;                  // 128-row blocks of W
  uint32_t give_up;        // lanes of the epilogue that do not wait (tests)
  bool vec;
};

// An epilogue warp's 32 rows of an accumulator, a thread a row, 64 nch columns from TMEM to
// registers as bf16 pairs.
template <int BN>
__device__ __forceinline__ void load_row(uint32_t tbase, int nch, uint32_t (&pk)[BN / 64][32]) {
#pragma unroll
  for (int c = 0; c < BN / 64; ++c) {
    if (c < nch) {
      uint32_t v0[32], v1[32];
      tc5::ld_32x32b_x32(tbase + (uint32_t)(64 * c), v0);
      tc5::ld_32x32b_x32(tbase + (uint32_t)(64 * c + 32), v1);
      tc5::wait_ld();
      tc5::reg_after_ld(v0);
      tc5::reg_after_ld(v1);
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        pk[c][j] = pack2(__uint_as_float(v0[2 * j]), __uint_as_float(v0[2 * j + 1]));
        pk[c][16 + j] = pack2(__uint_as_float(v1[2 * j]), __uint_as_float(v1[2 * j + 1]));
      }
    }
  }
}

// Those rows to D from (row0, col0), block by block of 32 x 64 through swizzled staging: by TMA
// (vec), or row by row.  The warp has one block for staging, so that the ring gets the memory (a
// fourth stage of 128 x 256 is worth 9 %); the last item of a CTA finds the ring idle and
// stages there without waiting (`fresh`: a block for each).
template <int BN>
__device__ __forceinline__ void store_rows(const uint32_t (&pk)[BN / 64][32], int nch, uint8_t* stg,
                                           bool fresh, const CUtensorMap* tm_d, __nv_bfloat16* D,
                                           int64_t ldd, int M, int N, bool vec, int row0,
                                           int col0) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int c = 0; c < BN / 64; ++c) {
    if (c < nch) {
      uint8_t* const blk = fresh ? stg + c * kStgBytes : stg;
      // the block's previous store has read it
      if (vec && !fresh && lane == 0) tc5::bulk_wait_group_read<0>();
      __syncwarp();
      uint4* const dst = reinterpret_cast<uint4*>(blk + lane * 128);
#pragma unroll
      for (int j = 0; j < 8; ++j)  // the 128-byte swizzle: unit j of row r at j ^ (r % 8)
        dst[j ^ (lane & 7)] = make_uint4(pk[c][4 * j], pk[c][4 * j + 1], pk[c][4 * j + 2],
                                         pk[c][4 * j + 3]);
      if (vec) {
        tc5::fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          tc5::tma_store_2d(tm_d, tc5::saddr(blk), col0 + 64 * c, row0);
          tc5::bulk_commit_group();
        }
      } else {  // row by row, consecutive lanes on consecutive columns
        __syncwarp();
        const int c0 = col0 + 64 * c + lane, rows = min(32, M - row0);
        for (int r = 0; r < rows; ++r) {
          const uint8_t* const src = blk + r * 128;
          __nv_bfloat16* const out = D + (int64_t)(row0 + r) * ldd + c0;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int b = 2 * lane + 64 * i;  // byte of the row
            if (c0 + 32 * i < N)
              out[32 * i] = *reinterpret_cast<const __nv_bfloat16*>(
                  src + (((b >> 4) ^ (r & 7)) << 4) + (b & 15));
          }
        }
      }
    }
  }
}

template <int AF, int BN>
__global__ void __launch_bounds__(Cfg<AF, BN>::THREADS, 1)
    gemm_mx_kernel(MArgs g, const __grid_constant__ MMaps tm) {
  using C = Cfg<AF, BN>;
  constexpr int STAGES = C::STAGES, ATOMS = C::ATOMS, NSB = C::NSB;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t raw_addr = tc5::saddr(smem_raw);
  Smem<C>& sm = *reinterpret_cast<Smem<C>*>(smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int nk = (g.nkb + ATOMS - 1) / ATOMS;
  volatile uint32_t* err = &sm.err;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      tc5::mbar_init(&sm.full[s], 1);
      tc5::mbar_init(&sm.empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc5::mbar_init(&sm.tfull[i], 1);
      tc5::mbar_init(&sm.tempty[i], C::EPI_WARPS);
    }
    tc5::mbar_init(&sm.drain, 1);
    tc5::fence_mbar_init();
    sm.err = 0;
  }
  if (warp == 1) tc5::tmem_alloc(&sm.tmem, C::TMEM_COLS);
  tc5::fence_before_sync();
  __syncthreads();
  tc5::fence_after_sync();
  const uint32_t tmem = sm.tmem, sf0 = tmem + C::NACC * BN;

  if (warp == 0) {
    // ---- producer
    const bool leader = tc5::elect();
    int stage = 0;
    uint32_t phase = 0, armed = 0, last_par = 0;
    bool ok = true;
    for (int t = blockIdx.x; ok && t < g.tiles.items; t += gridDim.x) {
      const Item it = item_of<BN>(g.tiles, t);
      const int mb = it.mb, rb0 = it.col0 / 128;  // W's first scale tile
      const int nsb = max(0, min(NSB, g.nb - rb0));
      for (int kb = 0; kb < nk; ++kb) {
        ok = wait_all(&sm.empty[stage], phase ^ 1u, err);
        if (!ok) break;
        if (leader) {
          const int a0 = kb * ATOMS, na = min(ATOMS, g.nkb - a0);
          uint64_t* const full = &sm.full[stage];
          tc5::mbar_arrive_expect_tx(
              full, C::A_BYTES + it.w * C::W_ROW_TX + (uint32_t)((1 + nsb) * na) * kTile);
          tc5::tma_load_2d(tc5::saddr(sm.a[stage]), &tm.a, full, kb * 128, mb * BM);
          if (it.w == BN)
            tc5::tma_load_2d(tc5::saddr(sm.w[stage]), &tm.w, full, kb * 128, it.col0);
          else
            for (int c = 0; c < it.w; c += 64)
              tc5::tma_load_2d(tc5::saddr(sm.w[stage]) + c * 128, &tm.w64, full, kb * 128,
                               it.col0 + c);
          tc5::bulk_load(tc5::saddr(sm.sa[stage]), g.sa + ((int64_t)mb * g.nkb + a0) * kTile,
                         na * kTile, full);
          for (int j = 0; j < nsb; ++j)
            tc5::bulk_load(tc5::saddr(sm.sw[stage]) + j * ATOMS * kTile,
                           g.sw + ((int64_t)(rb0 + j) * g.nkb + a0) * kTile, na * kTile, full);
        }
        __syncwarp();
        armed |= 1u << stage;
        last_par = (last_par & ~(1u << stage)) | (phase << stage);
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    // the copies issued last land before the CTA can exit
    for (int s = 0; s < STAGES; ++s)
      if (armed & (1u << s)) (void)tc5::mbar_wait(&sm.full[s], (last_par >> s) & 1u, kWaitLimitNs);
  } else if (warp == 1) {
    // ---- scale copies and products
    const bool leader = tc5::elect();
    int stage = 0, acc = 0;
    uint32_t phase = 0, aphase = 0;
    bool ok = true;
    for (int t = blockIdx.x; ok && t < g.tiles.items; t += gridDim.x) {
      const Item it = item_of<BN>(g.tiles, t);
      const uint32_t shift = (uint32_t)(it.col0 % 128) / 32;  // inside the first scale tile
      const uint32_t idesc = C::IDESC | (uint32_t)(it.w >> 3) << 17;
      ok = wait_all(&sm.tempty[acc], aphase ^ 1u, err);
      if (!ok) break;
      tc5::fence_after_sync();
      const uint32_t d = tmem + (uint32_t)(acc * BN);
      for (int kb = 0; kb < nk; ++kb) {
        ok = wait_all(&sm.full[stage], phase, err);
        if (!ok) break;
        tc5::fence_after_sync();
        const int na = min(ATOMS, g.nkb - kb * ATOMS);
        // the stage's columns: A's tiles along K, then W's
        const uint32_t sfa = sf0 + (uint32_t)(stage * C::SF_COLS), sfw = sfa + ATOMS * 4;
        const uint64_t dw = tc5::desc_sw128(tc5::saddr(sm.w[stage]), 16, 1024);
        const uint64_t da = tc5::desc_sw128(tc5::saddr(sm.a[stage]), 16, 1024);
        const uint64_t dsa = tc5::desc_scales(tc5::saddr(sm.sa[stage]));
        const uint64_t dsw = tc5::desc_scales(tc5::saddr(sm.sw[stage]));
        if (leader) {
#pragma unroll
          for (int a = 0; a < ATOMS; ++a) {
            if (a < na) {
              tc5::cp_scales(sfa + 4 * a, dsa + a * (kTile / 16));
#pragma unroll
              for (int j = 0; j < NSB; ++j)
                tc5::cp_scales(sfw + 4 * (a * NSB + j), dsw + (j * ATOMS + a) * (kTile / 16));
            }
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {  // +32 bytes a K step inside the swizzle atom
            if (AF == mx::kFp4) {        // 64 values, two of a tile's four blocks
              if (k / 2 < na)
                tc5::mma_mxf4(d, da + (uint64_t)(2 * k), dw + (uint64_t)(2 * k),
                              tc5::idesc_mx_sf(idesc, 2 * (k & 1)), sfa + 4 * (k / 2),
                              sfw + 4 * NSB * (k / 2) + shift, kb > 0 || k > 0);
            } else {  // 32 values, one block
              tc5::mma_mxf8f6f4(d, da + (uint64_t)(2 * k), dw + (uint64_t)(2 * k),
                                tc5::idesc_mx_sf(idesc, k), sfa, sfw + shift, kb > 0 || k > 0);
            }
          }
          tc5::commit(&sm.empty[stage]);
        }
        __syncwarp();
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;
      if (leader) tc5::commit(&sm.tfull[acc]);
      __syncwarp();
      if (++acc == C::NACC) {
        acc = 0;
        aphase ^= 1u;
      }
    }
    // every product issued has finished before TMEM is released
    if (leader) tc5::commit(&sm.drain);
    __syncwarp();
    (void)tc5::mbar_wait(&sm.drain, 0, kWaitLimitNs);
    __syncwarp();
  } else {
    // ---- epilogue: TMEM lane quarter q, one row a thread
    const int q = warp & 3, ew = warp - 2;
    int acc = 0;
    uint32_t aphase = 0;
    for (int t = blockIdx.x; t < g.tiles.items; t += gridDim.x) {
      const Item it = item_of<BN>(g.tiles, t);
      const int row0 = it.mb * BM + 32 * q, col0 = it.col0;
      if (!wait_all(&sm.tfull[acc], aphase, err, g.give_up)) break;
      tc5::fence_after_sync();
      const uint32_t tbase =
          tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(acc * BN);
      // the row into registers as bf16, then TMEM goes back: the stores below drain
      // while the next products run
      const int nch = min(it.w / 64, (g.N - col0 + 63) / 64);
      uint32_t pk[BN / 64][32];
      load_row<BN>(tbase, nch, pk);
      tc5::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc5::mbar_arrive(&sm.tempty[acc]);
      const bool last = t + (int)gridDim.x >= g.tiles.items;
      store_rows<BN>(pk, nch, last ? sm.a[0] + ew * (BN / 64) * kStgBytes : sm.stg[ew], last, &tm.d,
                     g.D, g.ldd, g.M, g.N, g.vec, row0, col0);
      if (++acc == C::NACC) {
        acc = 0;
        aphase ^= 1u;
      }
    }
    if (lane == 0) tc5::bulk_wait_group<0>();  // every store of this warp has landed
    __syncwarp();
  }
  tc5::fence_before_sync();
  __syncthreads();
  tc5::fence_after_sync();
  if (warp == 1) tc5::tmem_dealloc(tmem, C::TMEM_COLS);
  if (threadIdx.x == 0 && sm.err) atomicAdd(&g_gemm_mx_wait_timeouts, 1u);
}

// Where D's rows are multiples of 16 bytes (a TMA store ends a row at one): its map for the
// stores of 32 x 64 blocks.
bool encode_output(CUtensorMap* m, const Operands& o) {
  if (o.N % 8 != 0 || o.ldd % 8 != 0 || (reinterpret_cast<uintptr_t>(o.D) & 15) != 0) return false;
  PFN_cuTensorMapEncodeTiled_v12000 fn = tensor_map_encoder();
  const cuuint64_t dims[2] = {(cuuint64_t)o.N, (cuuint64_t)o.M};
  const cuuint64_t strides[1] = {(cuuint64_t)o.ldd * 2};
  const cuuint32_t box[2] = {64, 32};
  const cuuint32_t estr[2] = {1, 1};
  return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, o.D, dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
                   CUDA_SUCCESS;
}

// How 128 x bn tiles go to the SMs: in whole rounds, and, from three rounds on, the tiles left
// over in the narrowest parts that still make one round (20011 x 1024 x 2048 in 128 x 256
// tiles, four rounds and 36 tiles in four parts each: 25.4 against 27.5 us in 4 bits, 39.7
// against 42.7 with 8-bit A, before the ring's fourth stage; with fewer rounds a smaller tile
// is better: 1000 x 2048 x 4096 8.3 against 10.0).
struct Plan {
  int64_t nt, rounds, left, full, items;
  int pw;  // columns of a part, bn where nothing is split
  Tiles tiles(int bn) const {
    return {(int)nt, (int)full, (int)items, (bn + pw - 1) / pw, pw};
  }
};
Plan plan(int64_t M, int64_t N, int bn, int64_t sms) {
  Plan p;
  p.nt = (N + bn - 1) / bn;
  const int64_t tiles = (M + BM - 1) / BM * p.nt;
  p.rounds = tiles / sms;
  p.left = tiles % sms;
  p.pw = bn;
  for (int pw = 64; p.rounds > 2 && p.left && pw < bn && pw <= 128; pw += 64)
    if (p.left * ((bn + pw - 1) / pw) <= sms) {
      p.pw = pw;
      break;
    }
  p.full = p.pw < bn ? tiles - p.left : tiles;
  p.items = p.full + (tiles - p.full) * ((bn + p.pw - 1) / p.pw);
  return p;
}

template <int AF, int BN>
cudaError_t launch(const Operands& o, int64_t sms, cudaStream_t s) {
  using C = Cfg<AF, BN>;
  const int64_t Kp = mx::pad128(o.K);
  MMaps tm;
  memset(&tm, 0, sizeof(tm));
  const bool ok = encode_codes(&tm.a, o.A, o.M, Kp, AF, false, BM) &&
                  encode_codes(&tm.w, o.W, o.N, Kp, mx::kFp4, AF != mx::kFp4, BN) &&
                  encode_codes(&tm.w64, o.W, o.N, Kp, mx::kFp4, AF != mx::kFp4, 64);
  if (!ok) return cudaErrorInvalidValue;
  MArgs g{};
  g.M = (int)o.M;
  g.N = (int)o.N;
  g.ldd = o.ldd;
  g.D = static_cast<__nv_bfloat16*>(o.D);
  g.sa = static_cast<const uint8_t*>(o.As);
  g.sw = static_cast<const uint8_t*>(o.Ws);
  const Plan p = plan(o.M, o.N, BN, sms);
  if (p.items > INT32_MAX) return cudaErrorInvalidValue;
  g.tiles = p.tiles(BN);
  g.nkb = (int)(Kp / 128);
  g.nb = (int)((o.N + 127) / 128);
  g.vec = encode_output(&tm.d, o);
  g.give_up = take_given_up_lanes();
  const size_t smem = sizeof(Smem<C>) + 1024;
  static_assert(sizeof(Smem<C>) + 1024 <= 232448, "one CTA's shared memory");
  static_assert(offsetof(Smem<C>, w) % 1024 == 0 && offsetof(Smem<C>, stg) % 1024 == 0 &&
                    offsetof(Smem<C>, sa) % 1024 == 0,
                "TMA buffers on 1024-byte boundaries");
  static std::atomic<uint64_t> done;
  const cudaError_t e = once_per_device(done, [&]() {
    return cudaFuncSetAttribute(gemm_mx_kernel<AF, BN>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  });
  if (e != cudaSuccess) return e;
  gemm_mx_kernel<AF, BN>
      <<<(unsigned)(p.items < sms ? p.items : sms), C::THREADS, smem, s>>>(g, tm);
  return cudaGetLastError();
}

// The tile.  A round of 128 x 256, 128 x 192 and 128 x 128 tiles takes about 100, 78 and 59
// parts of the same time, whatever K and A's type (small tiles bring in more bytes for each
// product); of the three the one that needs the least in its rounds and parts.  On one B200, us
// in 4 bits / with 8-bit A:
//   32768 x 6464 x 1024  121 123 133       191 202 225
//   20011 x 1024 x 2048  22.3 25.7 26.3    35.2 40.6 42.9
//   8192 x 8192 x 8192   195 212 231       352 385 440
//   4096 x 6464 x 1024   19.2 18.9 21.0    26.9 28.8 33.3
//   1500 x 6464 x 1024   11.7 10.0 11.0    15.1 14.0 16.4
//   1000 x 2048 x 4096   10.4 9.7 8.3      14.9 13.9 12.6
// (256 x 192 gained 1 to 5 % on a few shapes and lost 15 % on others.)
int tile_of(int64_t M, int64_t N, int64_t sms) {
  auto cost = [&](int bn, int64_t round) {
    const Plan p = plan(M, N, bn, sms);
    return p.rounds * round + (p.left ? round * p.pw / bn : 0);
  };
  const int64_t wide = cost(256, 100), mid = cost(192, 78), small = cost(128, 59);
  return wide <= mid && wide <= small ? 256 : mid <= small ? 192 : 128;
}

template <int AF>
cudaError_t launch_af(const Operands& o, cudaStream_t s) {
  const int64_t sms = current_device_sms() > 0 ? current_device_sms() : 148;
  const int split = split_of(o.M, o.N, o.K, AF, sms);
  if (split > 0) return launch_split(AF, o, split, s);
  const int bn = tile_of(o.M, o.N, sms);
  return bn == 256   ? launch<AF, 256>(o, sms, s)
         : bn == 192 ? launch<AF, 192>(o, sms, s)
                     : launch<AF, 128>(o, sms, s);
}

}  // namespace

cudaError_t launch_gemm_mx(int a_fmt, int64_t M, int64_t N, int64_t K, const void* A,
                           const void* A_scales, const void* W, const void* W_scales, void* D,
                           int64_t ldd, cudaStream_t s) {
  if (M == 0 || N == 0) return cudaSuccess;
  const Operands o{M, N, K, A, A_scales, W, W_scales, D, ldd};
  return a_fmt == mx::kFp4 ? launch_af<mx::kFp4>(o, s) : launch_af<mx::kFp8>(o, s);
}

GemmMxPlan gemm_mx_plan(int a_fmt, int64_t M, int64_t N, int64_t K, int64_t sms) {
  const int split = split_of(M, N, K, a_fmt, sms);
  if (split > 0) return {split, M <= 16 ? 16 : 128, 0};
  const int bn = tile_of(M, N, sms);
  const Plan p = plan(M, N, bn, sms);
  return {0, bn, p.full < p.items ? p.pw : 0};
}

cudaError_t read_and_clear_gemm_mx_wait_timeouts(unsigned int* count) {
  const unsigned int zero = 0;
  unsigned int split = 0;
  cudaError_t e = cudaMemcpyFromSymbol(count, g_gemm_mx_wait_timeouts, sizeof(unsigned int));
  if (e == cudaSuccess)
    e = cudaMemcpyToSymbol(g_gemm_mx_wait_timeouts, &zero, sizeof(unsigned int));
  if (e == cudaSuccess) e = gemm_mx::read_and_clear_split_timeouts(&split);
  if (e == cudaSuccess) *count += split;
  return e;
}

}  // namespace m3ssd
