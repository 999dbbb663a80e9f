// What the microscaled GEMM's kernels share (gemm_mx.cu: a tile a CTA; gemm_mx_pair.cu: a tile
// a pair of CTAs; gemm_mx_split.cu: few tokens or tiles, K split over a cluster).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include <atomic>

#include "mx.cuh"
#include "tc5_mx.cuh"

namespace m3ssd {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

namespace gemm_mx {

constexpr int BM = 128;                      // rows of a product: TMEM's lanes
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr uint32_t kTile = 512;              // bytes of a scale tile (128 rows x 4 blocks)

struct Operands {
  int64_t M, N, K;
  const void *A, *As, *W, *Ws;
  void* D;
  int64_t ldd;
};

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// All lanes of a warp wait; a wait that runs out, for any of them, sets the CTA's error word.
__device__ __forceinline__ bool wait_all(uint64_t* mbar, uint32_t parity, volatile uint32_t* err) {
  if (__all_sync(0xffffffffu, tc5::mbar_wait(mbar, parity, kWaitLimitNs, err))) return true;
  *err = 1;
  return false;
}

// What a CTA (or a pair) takes of D: rows of tile row mb, w columns from col0.  Tiles up to
// `full` whole, then the parts of the others.
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

constexpr uint32_t kStgBytes = 32 * 128;  // an output block: 32 rows x 64 bf16 columns

// Those rows to D from (row0, col0), block by block of 32 x 64 through the warp's NSTG swizzled
// staging blocks: by TMA (vec), or row by row.  nst counts the warp's blocks.
template <int BN, int NSTG>
__device__ __forceinline__ void store_rows(const uint32_t (&pk)[BN / 64][32], int nch, uint8_t* stg,
                                           uint32_t& nst, const CUtensorMap* tm_d,
                                           __nv_bfloat16* D, int64_t ldd, int M, int N, bool vec,
                                           int row0, int col0) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int c = 0; c < BN / 64; ++c) {
    if (c < nch) {
      uint8_t* const blk = stg + nst % NSTG * kStgBytes;
      // the block's previous store has read it
      if (vec && lane == 0) tc5::bulk_wait_group_read<NSTG - 1>();
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
      ++nst;
    }
  }
}

// Codes (rows x Kp) as boxes of 128 bytes of shared memory a row.  spread: packed 4-bit
// codes go to 8-bit containers (16 codes in 8 of 16 bytes).
inline bool encode_codes(CUtensorMap* m, const void* base, int64_t rows, int64_t Kp, int fmt,
                         bool spread, uint32_t box_rows) {
  PFN_cuTensorMapEncodeTiled_v12000 fn = tensor_map_encoder();
  if (!fn) return false;
  const cuuint64_t bytes = (cuuint64_t)(fmt == mx::kFp4 ? Kp / 2 : Kp);
  const cuuint64_t dims[2] = {spread ? (cuuint64_t)Kp : bytes, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {bytes};
  const cuuint32_t box[2] = {128, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, spread ? CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
            const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Where D's rows are multiples of 16 bytes (a TMA store ends a row at one): its map for the
// stores of 32 x 64 blocks.
inline bool encode_output(CUtensorMap* m, const Operands& o) {
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

// How bm x bn tiles go to the SMs (or the pairs): in whole rounds, and, from three rounds on,
// the tiles left over in the narrowest parts, of least_pw or 128 columns, that still make one
// round (20011 x 1024 x 2048 in 128 x 256 tiles, four rounds and 36 tiles in four parts each:
// 25.4 against 27.5 us in 4 bits, 39.7 against 42.7 with 8-bit A; with fewer rounds a smaller
// tile is better: 1000 x 2048 x 4096 8.3 against 10.0).
struct Plan {
  int64_t nt, rounds, left, full, items;
  int pw;  // columns of a part, bn where nothing is split
  Tiles tiles(int bn) const {
    return {(int)nt, (int)full, (int)items, (bn + pw - 1) / pw, pw};
  }
};
inline Plan plan(int64_t M, int64_t N, int64_t bm, int bn, int least_pw, int64_t slots) {
  Plan p;
  p.nt = (N + bn - 1) / bn;
  const int64_t tiles = (M + bm - 1) / bm * p.nt;
  p.rounds = tiles / slots;
  p.left = tiles % slots;
  p.pw = bn;
  for (int pw = least_pw; p.rounds > 2 && p.left && pw < bn && pw <= 128; pw += 64)
    if (p.left * ((bn + pw - 1) / pw) <= slots) {
      p.pw = pw;
      break;
    }
  p.full = p.pw < bn ? tiles - p.left : tiles;
  p.items = p.full + (tiles - p.full) * ((bn + p.pw - 1) / p.pw);
  return p;
}

// Does `allow` (the kernel's shared memory attribute) once on each device; `done` holds a bit a
// device.
template <typename F>
cudaError_t once_per_device(std::atomic<uint64_t>& done, F allow) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = allow();
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Few tokens or few tiles (gemm_mx_split.cu): the number of CTAs a tile's K is split over, 0
// where that kernel is not the one to take.
int split_of(int64_t M, int64_t N, int64_t K, int a_fmt, int64_t sms);
cudaError_t launch_split(int a_fmt, const Operands& o, int split, cudaStream_t s);
cudaError_t read_and_clear_split_timeouts(unsigned int* count);

// Many tiles (gemm_mx_pair.cu): a pair's estimated time in the units of gemm_mx.cu's tiles.
int64_t pair_cost(int64_t M, int64_t N, int64_t K, int a_fmt, int64_t sms);
cudaError_t launch_pair(int a_fmt, const Operands& o, int64_t sms, cudaStream_t s);
cudaError_t read_and_clear_pair_timeouts(unsigned int* count);

}  // namespace gemm_mx
}  // namespace m3ssd
