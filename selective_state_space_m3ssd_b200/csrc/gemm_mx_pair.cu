// The microscaled product (gemm_mx.cu) by pairs of CTAs (tcgen05 cta_group::2), for shapes of
// many tiles and a K long enough: a tile is 256 x 256, each CTA of a cluster of two holding 128
// rows of A, half of W's rows and 128 x 256 outputs.
//
// In each CTA warp 0 copies its own parts; all bytes of a stage, of both CTAs, count on the
// first CTA's barrier.  One elected lane of the first CTA issues the scale copies and products
// of the pair; their completion arrives in both CTAs (stages free, accumulator ready).  Both
// CTAs' epilogue warps return the accumulator to the first CTA's barrier.  Waits are bounded
// as in gemm_mx.cu; the two CTAs leave together, so a barrier or a copy of one never meets the
// other's absence.
//
// Why: a stage of a 128 x 256 tile brings 48 KB into shared memory for 512 cycles of products,
// as much as the copies manage beside the products' own reads; a pair brings W in once for both, 32
// KB a CTA.  Beside the scales TMEM has no room for a second accumulator of 256 columns, so
// every tile pays for the hand-over of the one there is (about 1.3 us; eight epilogue warps
// that release it before they convert made no difference), and a pair starts later than a
// CTA.  What is left is the products: 8192^3 with 8-bit A runs at 3.2 PFLOP/s, 0.96 of twice
// the bf16 rate.  One B200, us with 4-bit / 8-bit A, against gemm_mx.cu's tiles:
//   8192 x 8192 x 8192   183 (192)    344 (372)
//   4096 x 4096 x 4096   33.9 (37.3)  47.8 (52.6)
//   32768 x 1024 x 4096  56.9 (62.6)  100 (114)
//   32768 x 1024 x 2048  38.2 (38.5)  56.7 (62.4)
//   20011 x 1024 x 2048  25.5 (25.5)  38.5 (40.1)
//   18944 x 2048 x 1024  29.6 (28.9)  41.4 (43.2)
//   18944 x 2048 x 512   25.7 (20.0)  29.3 (28.2)
//   9472 x 1024 x 2048   13.9 (13.0)  18.7 (17.5)
#include <cstddef>
#include <cstring>

#include "gemm_mx.cuh"
#include "internal.h"

namespace m3ssd {

__device__ unsigned int g_gemm_mx_pair_wait_timeouts;

namespace {

using namespace gemm_mx;

constexpr int BN = 256;  // columns of a tile
constexpr int kEpiWarps = 4, kThreads = 32 * (2 + kEpiWarps), kStg = 2;

// A stage is 128 bytes of K a row: 256 values of A in 4 bits, 128 in 8.
template <int AF>
struct Cfg {
  static constexpr int ATOMS = AF == mx::kFp4 ? 2 : 1;  // scale tiles along K a stage
  static constexpr int NSB = BN / 128;                  // scale tiles along W's rows (all of them)
  static constexpr uint32_t A_BYTES = BM * 128, W_BYTES = BN / 2 * 128;
  static constexpr uint32_t SA_BYTES = ATOMS * kTile, SW_BYTES = NSB * ATOMS * kTile;
  // bytes a CTA's copies of a stage count: A and the scales, and W's 4-bit codes as in global
  // memory
  static constexpr uint32_t TX = A_BYTES + SA_BYTES + SW_BYTES;
  static constexpr uint32_t W_ROW_TX = AF == mx::kFp4 ? 128 : 64;
  static constexpr int STAGE = A_BYTES + W_BYTES + SA_BYTES + SW_BYTES;
  static constexpr int ROOM = 226 * 1024 - kEpiWarps * kStg * (int)kStgBytes - 1024;
  static constexpr int STAGES = ROOM / STAGE < 8 ? ROOM / STAGE : 8;
  static constexpr int SF_COLS = ATOMS * 4 * (1 + NSB);
  static_assert(BN + STAGES * SF_COLS <= 512, "tensor memory");
  // the CTAs of a pair wait for one another: neither may wait for tensor memory that a CTA of
  // another pair, or of gemm_mx_split.cu, holds on its SM
  static_assert(STAGES * STAGE > 150 * 1024, "alone on an SM");
  static constexpr uint32_t IDESC =  // the columns are ORed in
      tc5::idesc_mx(2 * BM, 0, AF == mx::kFp4 ? 1 : 0, AF == mx::kFp4 ? 1 : 5);
};

template <typename C>
struct Smem {
  uint8_t a[C::STAGES][C::A_BYTES];
  uint8_t w[C::STAGES][C::W_BYTES];
  uint8_t stg[kEpiWarps * kStg][kStgBytes];
  uint8_t sa[C::STAGES][C::SA_BYTES];
  uint8_t sw[C::STAGES][C::SW_BYTES];
  uint64_t full[C::STAGES];   // first CTA: the stage's bytes, of both
  uint64_t empty[C::STAGES];  // the stage's products have finished
  uint64_t tfull;             // accumulator ready
  uint64_t tempty;            // first CTA: accumulator read by both CTAs' epilogue warps
  uint64_t drain;
  uint32_t tmem;
  uint32_t err;
};

struct PMaps {
  CUtensorMap a, w;    // codes, boxes of 128 bytes x 128 rows
  CUtensorMap w64;     // W's codes in boxes of 64 rows, a part's half
  CUtensorMap sa, sw;  // scale tiles as rows of 128 words, boxes of ATOMS tiles
  CUtensorMap d;       // bf16 (N, M), box 64 x 32, 128-byte swizzle (when vec)
};

struct PArgs {
  int M, N;
  int64_t ldd;
  __nv_bfloat16* D;
  Tiles tiles;  // the items of the pairs
  int nkb;      // 128-column groups of K
  bool vec;
};

template <int AF>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    gemm_mx_pair_kernel(PArgs g, const __grid_constant__ PMaps tm) {
  using C = Cfg<AF>;
  constexpr int STAGES = C::STAGES, ATOMS = C::ATOMS, NSB = C::NSB;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t raw_addr = tc5::saddr(smem_raw);
  Smem<C>& sm = *reinterpret_cast<Smem<C>*>(smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = (int)tc5::cluster_rank();
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1;
  const int nk = (g.nkb + ATOMS - 1) / ATOMS;
  volatile uint32_t* err = &sm.err;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      tc5::mbar_init(&sm.full[s], 1);
      tc5::mbar_init(&sm.empty[s], 1);
    }
    tc5::mbar_init(&sm.tfull, 1);
    tc5::mbar_init(&sm.tempty, 2 * kEpiWarps);
    tc5::mbar_init(&sm.drain, 1);
    tc5::fence_mbar_init();
    sm.err = 0;
  }
  if (warp == 1) tc5::tmem_alloc_pair(&sm.tmem, 512);
  tc5::fence_before_sync();
  __syncthreads();
  tc5::cluster_sync();  // the barriers of both CTAs exist
  tc5::fence_after_sync();
  const uint32_t tmem = sm.tmem, sf0 = tmem + BN;

  if (warp == 0) {
    // ---- producer: this CTA's parts
    const bool leader = tc5::elect();
    int stage = 0;
    uint32_t phase = 0, armed = 0, last_par = 0;
    bool ok = true;
    for (int t = first; ok && t < g.tiles.items; t += step) {
      const Item it = item_of<BN>(g.tiles, t);
      const int rb = 2 * it.mb + rank, wb0 = it.col0 / 128, w0 = it.col0 + rank * (it.w / 2);
      for (int kb = 0; kb < nk; ++kb) {
        ok = wait_all(&sm.empty[stage], phase ^ 1u, err);
        if (!ok) break;
        if (leader) {
          if (rank == 0)
            tc5::mbar_arrive_expect_tx(&sm.full[stage], 2 * C::TX + it.w * C::W_ROW_TX);
          const uint32_t full = tc5::cluster_map(tc5::saddr(&sm.full[stage]), 0);
          tc5::tma_load_2d_pair(tc5::saddr(sm.a[stage]), &tm.a, full, kb * 128, rb * BM);
          tc5::tma_load_2d_pair(tc5::saddr(sm.w[stage]), it.w == BN ? &tm.w : &tm.w64, full,
                                kb * 128, w0);
          // past the last tile of scales: zeros
          tc5::tma_load_2d_pair(tc5::saddr(sm.sa[stage]), &tm.sa, full, 0, rb * g.nkb + kb * ATOMS);
#pragma unroll
          for (int j = 0; j < NSB; ++j)
            tc5::tma_load_2d_pair(tc5::saddr(sm.sw[stage]) + j * ATOMS * kTile, &tm.sw, full, 0,
                                  (wb0 + j) * g.nkb + kb * ATOMS);
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
    // the copies issued last (the other CTA's too) land before either CTA leaves
    if (rank == 0)
      for (int s = 0; s < STAGES; ++s)
        if (armed & (1u << s)) (void)tc5::mbar_wait(&sm.full[s], (last_par >> s) & 1u, kWaitLimitNs);
    __syncwarp();
  } else if (warp == 1) {
    // ---- the pair's scale copies and products
    if (rank == 0) {
      const bool leader = tc5::elect();
      int stage = 0;
      uint32_t phase = 0, aphase = 0;
      bool ok = true;
      for (int t = first; ok && t < g.tiles.items; t += step) {
        const uint32_t idesc = C::IDESC | (uint32_t)(item_of<BN>(g.tiles, t).w >> 3) << 17;
        ok = wait_all(&sm.tempty, aphase ^ 1u, err);
        if (!ok) break;
        tc5::fence_after_sync();
        for (int kb = 0; kb < nk; ++kb) {
          ok = wait_all(&sm.full[stage], phase, err);
          if (!ok) break;
          tc5::fence_after_sync();
          const int na = min(ATOMS, g.nkb - kb * ATOMS);
          const uint32_t sfa = sf0 + (uint32_t)(stage * C::SF_COLS), sfw = sfa + ATOMS * 4;
          const uint64_t da = tc5::desc_sw128(tc5::saddr(sm.a[stage]), 16, 1024);
          const uint64_t dw = tc5::desc_sw128(tc5::saddr(sm.w[stage]), 16, 1024);
          const uint64_t dsa = tc5::desc_scales(tc5::saddr(sm.sa[stage]));
          const uint64_t dsw = tc5::desc_scales(tc5::saddr(sm.sw[stage]));
          if (leader) {
#pragma unroll
            for (int a = 0; a < ATOMS; ++a) {
              if (a < na) {
                tc5::cp_scales_pair(sfa + 4 * a, dsa + a * (kTile / 16));
#pragma unroll
                for (int j = 0; j < NSB; ++j)
                  tc5::cp_scales_pair(sfw + 4 * (a * NSB + j),
                                      dsw + (j * ATOMS + a) * (kTile / 16));
              }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {  // +32 bytes a K step inside the swizzle atom
              if (AF == mx::kFp4) {        // 64 values, two of a tile's four blocks
                if (k / 2 < na)
                  tc5::mma_mxf4_pair(tmem, da + (uint64_t)(2 * k), dw + (uint64_t)(2 * k),
                                     tc5::idesc_mx_sf(idesc, 2 * (k & 1)), sfa + 4 * (k / 2),
                                     sfw + 4 * NSB * (k / 2), kb > 0 || k > 0);
              } else {  // 32 values, one block
                tc5::mma_mxf8f6f4_pair(tmem, da + (uint64_t)(2 * k), dw + (uint64_t)(2 * k),
                                       tc5::idesc_mx_sf(idesc, k), sfa, sfw, kb > 0 || k > 0);
              }
            }
            tc5::commit_pair(&sm.empty[stage]);
          }
          __syncwarp();
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        if (leader) tc5::commit_pair(&sm.tfull);
        __syncwarp();
        aphase ^= 1u;
      }
      // every product issued has finished before TMEM is released
      if (leader) tc5::commit_pair(&sm.drain);
      __syncwarp();
      (void)tc5::mbar_wait(&sm.drain, 0, kWaitLimitNs);
      __syncwarp();
    }
  } else {
    // ---- epilogue: TMEM lane quarter q, one row a thread
    const int q = warp & 3, ew = warp - 2;
    uint32_t nst = 0, aphase = 0;
    for (int t = first; t < g.tiles.items; t += step) {
      const Item it = item_of<BN>(g.tiles, t);
      const int row0 = (2 * it.mb + rank) * BM + 32 * q, col0 = it.col0;
      const int nch = min(it.w / 64, (g.N - col0 + 63) / 64);
      if (!tc5::mbar_wait(&sm.tfull, aphase, kWaitLimitNs, err)) {
        *err = 1;
        break;
      }
      tc5::fence_after_sync();
      // the row into registers as bf16, then TMEM goes back: the stores below drain while
      // the next products run
      uint32_t pk[BN / 64][32];
      load_row<BN>(tmem + ((uint32_t)(32 * q) << 16), nch, pk);
      tc5::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc5::mbar_arrive_remote(tc5::cluster_map(tc5::saddr(&sm.tempty), 0));
      store_rows<BN, kStg>(pk, nch, sm.stg[ew * kStg], nst, &tm.d, g.D, g.ldd, g.M, g.N, g.vec,
                           row0, col0);
      aphase ^= 1u;
    }
    if (lane == 0) tc5::bulk_wait_group<0>();  // every store of this warp has landed
    __syncwarp();
  }
  tc5::fence_before_sync();
  __syncthreads();
  tc5::cluster_sync();
  tc5::fence_after_sync();
  if (warp == 1) {
    (void)tc5::mbar_wait(&sm.drain, 0, kWaitLimitNs);  // the second CTA: its arrivals have landed
    __syncwarp();
    tc5::tmem_dealloc_pair(tmem, 512);
  }
  __syncwarp();
  tc5::cluster_sync();
  if (threadIdx.x == 0 && sm.err) atomicAdd(&g_gemm_mx_pair_wait_timeouts, 1u);
}

// Scale tiles as rows of 128 words, boxes of `atoms` rows.
bool encode_scales(CUtensorMap* m, const void* base, int64_t tiles, uint32_t atoms) {
  PFN_cuTensorMapEncodeTiled_v12000 fn = tensor_map_encoder();
  const cuuint64_t dims[2] = {128, (cuuint64_t)tiles};
  const cuuint64_t strides[1] = {kTile};
  const cuuint32_t box[2] = {128, atoms};
  const cuuint32_t estr[2] = {1, 1};
  return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(base), dims, strides, box,
                  estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int AF>
cudaError_t launch(const Operands& o, int64_t pairs, cudaStream_t s) {
  using C = Cfg<AF>;
  const int64_t Kp = mx::pad128(o.K), nkb = Kp / 128;
  constexpr bool spread = AF != mx::kFp4;
  PMaps tm;
  memset(&tm, 0, sizeof(tm));
  if (!encode_codes(&tm.a, o.A, o.M, Kp, AF, false, BM) ||
      !encode_codes(&tm.w, o.W, o.N, Kp, mx::kFp4, spread, BN / 2) ||
      !encode_codes(&tm.w64, o.W, o.N, Kp, mx::kFp4, spread, 64) ||
      !encode_scales(&tm.sa, o.As, (o.M + 127) / 128 * nkb, C::ATOMS) ||
      !encode_scales(&tm.sw, o.Ws, (o.N + 127) / 128 * nkb, C::ATOMS))
    return cudaErrorInvalidValue;
  PArgs g{};
  g.M = (int)o.M;
  g.N = (int)o.N;
  g.ldd = o.ldd;
  g.D = static_cast<__nv_bfloat16*>(o.D);
  g.nkb = (int)nkb;
  g.vec = encode_output(&tm.d, o);
  const Plan p = plan(o.M, o.N, 2 * BM, BN, 128, pairs);
  if (p.items > INT32_MAX) return cudaErrorInvalidValue;
  g.tiles = p.tiles(BN);
  const size_t smem = sizeof(Smem<C>) + 1024;
  static_assert(sizeof(Smem<C>) + 1024 <= 232448, "one CTA's shared memory");
  static_assert(offsetof(Smem<C>, w) % 1024 == 0 && offsetof(Smem<C>, stg) % 1024 == 0 &&
                    offsetof(Smem<C>, sa) % 128 == 0 && offsetof(Smem<C>, sw) % 128 == 0,
                "TMA buffers");
  static std::atomic<uint64_t> done;
  const cudaError_t e = once_per_device(done, [&]() {
    return cudaFuncSetAttribute(gemm_mx_pair_kernel<AF>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  });
  if (e != cudaSuccess) return e;
  gemm_mx_pair_kernel<AF>
      <<<(unsigned)(2 * (p.items < pairs ? p.items : pairs)), kThreads, smem, s>>>(g, tm);
  return cudaGetLastError();
}

}  // namespace

namespace gemm_mx {

// In the units of gemm_mx.cu's costs, fitted to the times above: 120 for a pair's later start;
// a round 290 in 4 bits and 430 with 8-bit A, and 320 over its stages for the hand-over; parts
// of 128 columns two thirds.  Of fewer than three rounds a pair made no shape faster.
int64_t pair_cost(int64_t M, int64_t N, int64_t K, int a_fmt, int64_t sms) {
  const bool a4 = a_fmt == mx::kFp4;
  const int64_t stage = a4 ? 256 : 128, nk = (K + stage - 1) / stage;
  const Plan p = plan(M, N, 2 * BM, BN, 128, sms / 2);
  if (p.rounds < 3) return INT64_MAX;
  const int64_t round = (a4 ? 290 : 430) + 320 / nk;
  return 120 + p.rounds * round + (p.left ? (p.pw < BN ? round * 2 / 3 : round) : 0);
}

cudaError_t launch_pair(int a_fmt, const Operands& o, int64_t sms, cudaStream_t s) {
  return a_fmt == mx::kFp4 ? launch<mx::kFp4>(o, sms / 2, s) : launch<mx::kFp8>(o, sms / 2, s);
}

cudaError_t read_and_clear_pair_timeouts(unsigned int* count) {
  const unsigned int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(count, g_gemm_mx_pair_wait_timeouts, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_gemm_mx_pair_wait_timeouts, &zero, sizeof(unsigned int));
}

}  // namespace gemm_mx
}  // namespace m3ssd
