// The microscaled product (gemm_mx.cu) for few tokens or few tiles: one tile a cluster, K
// split over its CTAs.
//
// A tile is 128 columns of D by BN tokens.  CTA r of the S of a cluster multiplies stages
// [r nk / S, (r + 1) nk / S) of the tile's nk along K into its own tensor memory, leaves the
// partial tile in shared memory as fp32, and after a cluster barrier the CTAs divide the
// tokens among their warps: a warp reads a token's 128 partial sums of every CTA through the
// cluster's shared memory, adds them in the order of the CTAs (the result does not depend on
// their timing), rounds once to bf16 and stores 256 consecutive bytes.  With up to 16 tokens
// (SWAP) W's rows fill the 128 lanes and the tokens are the product's narrow side; beyond
// that the tokens are the lanes.  Two CTAs fit an SM: one loads while the other joins.
//
// Waits are bounded as in gemm_mx.cu.  A CTA whose wait ran out still reaches both cluster
// barriers, so the others of its cluster end too.
#include "gemm_mx.cuh"
#include "internal.h"

namespace m3ssd {

__device__ unsigned int g_gemm_mx_split_wait_timeouts;

namespace {

using namespace gemm_mx;

// AF: A's format.  BN: tokens of a tile.  A stage is 128 bytes of K a row.
template <int AF, int BN, bool SWAP>
struct Cfg {
  static constexpr int ATOMS = AF == mx::kFp4 ? 2 : 1;  // scale tiles along K a stage
  static constexpr int WARPS = 6;                       // copies, products, four of the join
  static constexpr uint32_t R_BYTES = BM * 128, C_BYTES = (SWAP ? BN : 128) * 128;
  // bytes the copies of a stage count on its barrier: W's 4-bit codes as in global memory
  static constexpr uint32_t R_TX = AF != mx::kFp4 && SWAP ? R_BYTES / 2 : R_BYTES;
  static constexpr uint32_t C_TX = AF != mx::kFp4 && !SWAP ? C_BYTES / 2 : C_BYTES;
  static constexpr uint32_t S_BYTES = ATOMS * kTile;
  static constexpr int STAGE = R_BYTES + C_BYTES + 2 * S_BYTES;
  static constexpr int ROOM = 110 * 1024;  // two CTAs on an SM
  static constexpr int STAGES = ROOM / STAGE < 8 ? ROOM / STAGE : 8;
  static constexpr int ACC_COLS = SWAP ? 32 : 128, SF_COLS = ATOMS * 8;
  static constexpr int COLS = ACC_COLS + STAGES * SF_COLS;
  static constexpr uint32_t TMEM_COLS = COLS <= 128 ? 128 : 256;
  // at most two CTAs of this kernel, of any kind, share an SM: CTAs of a cluster wait for one
  // another, so none may wait for tensor memory that another cluster's CTA holds
  static_assert(COLS <= 256, "tensor memory of two CTAs");
  static_assert(STAGES * STAGE > 77 * 1024, "no third CTA on an SM");
  static_assert(BN * 512 <= STAGES * (int)(R_BYTES + C_BYTES), "the partial tile fits the ring");
  static constexpr uint32_t FA = AF == mx::kFp4 ? 1 : 0, FW = AF == mx::kFp4 ? 1 : 5;
  static constexpr uint32_t IDESC =
      SWAP ? tc5::idesc_mx(BM, BN, FW, FA) : tc5::idesc_mx(BM, 128, FA, FW);
};

template <typename C>
struct Smem {
  // rows operand's stages, then the columns operand's; afterwards the partial tile
  uint8_t ring[C::STAGES * (C::R_BYTES + C::C_BYTES)];
  uint8_t sr[C::STAGES][C::S_BYTES];
  uint8_t sc[C::STAGES][C::S_BYTES];
  uint64_t full[C::STAGES];
  uint64_t empty[C::STAGES];
  uint64_t done;
  uint32_t tmem;
  uint32_t err;
};

struct SMaps {
  CUtensorMap r, c;  // codes of the rows and the columns operand
};

struct SArgs {
  int M, N;
  int64_t ldd;
  __nv_bfloat16* D;
  const uint8_t *rs, *cs;  // scales of the rows and the columns operand
  int nt;                  // 128-column tiles of D
  int nkb;                 // 128-column groups of K
  int split;               // CTAs of a cluster
  uint32_t give_up;        // lanes that do not wait for the products (tests)
  bool vec;                // four columns of D are one aligned store
};

// Tokens m0, m0 + step, ... of the tile: the sums of S partial tiles' columns n to n + 3, eight
// loads in flight.
template <int S>
__device__ __forceinline__ void join(const SArgs& g, uint32_t part, __nv_bfloat16* out, int m0,
                                     int step, int tokens, int n) {
  constexpr int TOK = 8 / S;
  uint32_t base[S];
#pragma unroll
  for (int r = 0; r < S; ++r) base[r] = tc5::cluster_map(part, r);
  const int unit = (n >> 2) & 31;
  for (int mb = m0; mb < tokens; mb += TOK * step) {
    float4 v[TOK][S];
#pragma unroll
    for (int t = 0; t < TOK; ++t) {
      const int m = min(mb + t * step, tokens - 1);
#pragma unroll
      for (int r = 0; r < S; ++r)
        v[t][r] = tc5::cluster_ld4(base[r] + m * 512 + ((unit ^ (m & 7)) << 4));
    }
#pragma unroll
    for (int t = 0; t < TOK; ++t) {
      const int m = mb + t * step;
      float4 sum = v[t][0];
#pragma unroll
      for (int r = 1; r < S; ++r) {
        sum.x += v[t][r].x;
        sum.y += v[t][r].y;
        sum.z += v[t][r].z;
        sum.w += v[t][r].w;
      }
      if (m >= tokens) break;
      __nv_bfloat16* const o = out + m * g.ldd + n;
      if (g.vec) {
        if (n < g.N)
          *reinterpret_cast<uint2*>(o) = make_uint2(pack2(sum.x, sum.y), pack2(sum.z, sum.w));
      } else {
        const float f[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n + i < g.N) o[i] = __float2bfloat16_rn(f[i]);
      }
    }
  }
}

template <int AF, int BN, bool SWAP>
__global__ void __launch_bounds__(32 * Cfg<AF, BN, SWAP>::WARPS, 2)
    gemm_mx_split_kernel(SArgs g, const __grid_constant__ SMaps tm) {
  using C = Cfg<AF, BN, SWAP>;
  constexpr int STAGES = C::STAGES, ATOMS = C::ATOMS;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t raw_addr = tc5::saddr(smem_raw);
  Smem<C>& sm = *reinterpret_cast<Smem<C>*>(smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = g.split > 1 ? (int)tc5::cluster_rank() : 0;
  const int tile = blockIdx.x / g.split, nb = tile % g.nt, tok0 = tile / g.nt * BN;
  const int rb = SWAP ? nb : tile / g.nt, cb = SWAP ? 0 : nb;  // 128-row blocks of the operands
  const int nk = (g.nkb + ATOMS - 1) / ATOMS;
  const int k0 = (int)((int64_t)nk * rank / g.split), k1 = (int)((int64_t)nk * (rank + 1) / g.split);
  volatile uint32_t* err = &sm.err;
  uint8_t* const ring_r = sm.ring;
  uint8_t* const ring_c = sm.ring + STAGES * C::R_BYTES;
  const int ahead = min(STAGES, k1 - k0);  // stages loaded before anything else
  auto load = [&](int kb, int stage) {
    const int a0 = kb * ATOMS, na = min(ATOMS, g.nkb - a0);
    uint64_t* const full = &sm.full[stage];
    tc5::mbar_arrive_expect_tx(full, C::R_TX + C::C_TX + (uint32_t)(2 * na) * kTile);
    tc5::tma_load_2d(tc5::saddr(ring_r + stage * C::R_BYTES), &tm.r, full, kb * 128, rb * BM);
    tc5::tma_load_2d(tc5::saddr(ring_c + stage * C::C_BYTES), &tm.c, full, kb * 128, cb * 128);
    tc5::bulk_load(tc5::saddr(sm.sr[stage]), g.rs + ((int64_t)rb * g.nkb + a0) * kTile, na * kTile,
                   full);
    tc5::bulk_load(tc5::saddr(sm.sc[stage]), g.cs + ((int64_t)cb * g.nkb + a0) * kTile, na * kTile,
                   full);
  };
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      tc5::mbar_init(&sm.full[s], 1);
      tc5::mbar_init(&sm.empty[s], 1);
    }
    tc5::mbar_init(&sm.done, 1);
    tc5::fence_mbar_init();
    sm.err = 0;
    for (int s = 0; s < ahead; ++s) load(k0 + s, s);
  }
  if (warp == 1) tc5::tmem_alloc(&sm.tmem, C::TMEM_COLS);
  tc5::fence_before_sync();
  __syncthreads();
  tc5::fence_after_sync();
  const uint32_t tmem = sm.tmem;

  if (warp == 0) {
    // ---- producer
    const bool leader = tc5::elect();
    int stage = 0;
    uint32_t phase = 0, last_par = 0;  // of a stage's next load, of each stage's last
    for (int kb = k0 + ahead; kb < k1; ++kb) {
      if (!wait_all(&sm.empty[stage], phase, err)) break;
      if (leader) load(kb, stage);
      __syncwarp();
      last_par ^= 1u << stage;
      if (++stage == STAGES) {
        stage = 0;
        phase ^= 1u;
      }
    }
    // the copies issued last land before the CTA can exit
    for (int s = 0; s < ahead; ++s)
      (void)tc5::mbar_wait(&sm.full[s], (last_par >> s) & 1u, kWaitLimitNs);
  } else if (warp == 1) {
    // ---- scale copies and products
    const bool leader = tc5::elect();
    int stage = 0;
    uint32_t phase = 0;
    for (int kb = k0; kb < k1; ++kb) {
      if (!wait_all(&sm.full[stage], phase, err)) break;
      tc5::fence_after_sync();
      const int na = min(ATOMS, g.nkb - kb * ATOMS);
      const uint32_t sfr = tmem + (uint32_t)(C::ACC_COLS + stage * C::SF_COLS);
      const uint32_t sfc = sfr + ATOMS * 4;
      const uint64_t dr = tc5::desc_sw128(tc5::saddr(ring_r + stage * C::R_BYTES), 16, 1024);
      const uint64_t dc = tc5::desc_sw128(tc5::saddr(ring_c + stage * C::C_BYTES), 16, 1024);
      const uint64_t dsr = tc5::desc_scales(tc5::saddr(sm.sr[stage]));
      const uint64_t dsc = tc5::desc_scales(tc5::saddr(sm.sc[stage]));
      if (leader) {
#pragma unroll
        for (int a = 0; a < ATOMS; ++a) {
          if (a < na) {
            tc5::cp_scales(sfr + 4 * a, dsr + a * (kTile / 16));
            tc5::cp_scales(sfc + 4 * a, dsc + a * (kTile / 16));
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // +32 bytes a K step inside the swizzle atom
          if (AF == mx::kFp4) {        // 64 values, two of a tile's four blocks
            if (k / 2 < na)
              tc5::mma_mxf4(tmem, dr + (uint64_t)(2 * k), dc + (uint64_t)(2 * k),
                            tc5::idesc_mx_sf(C::IDESC, 2 * (k & 1)), sfr + 4 * (k / 2),
                            sfc + 4 * (k / 2), kb > k0 || k > 0);
          } else {  // 32 values, one block
            tc5::mma_mxf8f6f4(tmem, dr + (uint64_t)(2 * k), dc + (uint64_t)(2 * k),
                              tc5::idesc_mx_sf(C::IDESC, k), sfr, sfc, kb > k0 || k > 0);
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
    // every product issued has finished before the ring is written and TMEM released
    if (leader) tc5::commit(&sm.done);
    __syncwarp();
    (void)tc5::mbar_wait(&sm.done, 0, kWaitLimitNs);
    __syncwarp();
  } else {
    // ---- the partial tile, token by token: 16-byte unit u of a token's 128 sums at u ^ (token % 8)
    const bool ok = wait_all(&sm.done, 0, err, g.give_up);
    tc5::fence_after_sync();
    const int q = warp & 3, row = 32 * q + lane;  // of the tile's lanes
    const uint32_t tbase = tmem + ((uint32_t)(32 * q) << 16);
    if (ok) {
      if constexpr (SWAP) {
        static_assert(!SWAP || BN == 16, "one load of TMEM");
        uint32_t v[16];
        tc5::ld_32x32b_x16(tbase, v);
        tc5::wait_ld();
        tc5::reg_after_ld(v);
#pragma unroll
        for (int m = 0; m < 16; ++m)
          reinterpret_cast<uint32_t*>(sm.ring)[m * 128 + ((row >> 2) ^ (m & 7)) * 4 + (row & 3)] =
              v[m];
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t v[32];
          tc5::ld_32x32b_x32(tbase + (uint32_t)(32 * c), v);
          tc5::wait_ld();
          tc5::reg_after_ld(v);
          uint4* const dst = reinterpret_cast<uint4*>(sm.ring) + row * 32 + 8 * c;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            dst[j ^ (row & 7)] = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        }
      }
    }
  }
  tc5::fence_before_sync();
  __syncthreads();
  tc5::fence_after_sync();
  if (g.split > 1) tc5::cluster_sync();
  if (warp == 1) tc5::tmem_dealloc(tmem, C::TMEM_COLS);

  if (!*err) {
    const int m0 = rank * C::WARPS + warp, step = g.split * C::WARPS;
    const uint32_t part = tc5::saddr(sm.ring);
    __nv_bfloat16* const out = g.D + (int64_t)tok0 * g.ldd;
    const int tokens = min(BN, g.M - tok0), n = nb * 128 + 4 * lane;
    if (g.split == 1)
      join<1>(g, part, out, m0, step, tokens, n);
    else if (g.split == 2)
      join<2>(g, part, out, m0, step, tokens, n);
    else if (g.split == 4)
      join<4>(g, part, out, m0, step, tokens, n);
    else
      join<8>(g, part, out, m0, step, tokens, n);
  }
  __syncwarp();
  if (g.split > 1) tc5::cluster_sync();  // no CTA ends while another reads its partial tile
  if (threadIdx.x == 0 && sm.err) atomicAdd(&g_gemm_mx_split_wait_timeouts, 1u);
}

template <int AF, int BN, bool SWAP>
cudaError_t launch(const Operands& o, int split, cudaStream_t s) {
  using C = Cfg<AF, BN, SWAP>;
  const int64_t Kp = mx::pad128(o.K);
  constexpr bool spread = AF != mx::kFp4;
  SMaps tm;
  const bool ok = SWAP ? encode_codes(&tm.r, o.W, o.N, Kp, mx::kFp4, spread, BM) &&
                             encode_codes(&tm.c, o.A, o.M, Kp, AF, false, BN)
                       : encode_codes(&tm.r, o.A, o.M, Kp, AF, false, BM) &&
                             encode_codes(&tm.c, o.W, o.N, Kp, mx::kFp4, spread, 128);
  if (!ok) return cudaErrorInvalidValue;
  SArgs g{};
  g.M = (int)o.M;
  g.N = (int)o.N;
  g.ldd = o.ldd;
  g.D = static_cast<__nv_bfloat16*>(o.D);
  g.rs = static_cast<const uint8_t*>(SWAP ? o.Ws : o.As);
  g.cs = static_cast<const uint8_t*>(SWAP ? o.As : o.Ws);
  const int64_t nt = (o.N + 127) / 128, tiles = nt * ((o.M + BN - 1) / BN);
  if (tiles * split > INT32_MAX) return cudaErrorInvalidValue;
  g.nt = (int)nt;
  g.nkb = (int)(Kp / 128);
  g.split = split;
  g.give_up = take_given_up_lanes();
  g.vec = o.N % 4 == 0 && o.ldd % 4 == 0 && (reinterpret_cast<uintptr_t>(o.D) & 7) == 0;
  const size_t smem = sizeof(Smem<C>) + 1024;
  static_assert(sizeof(Smem<C>) + 1024 <= 113 * 1024, "two CTAs on an SM");
  static std::atomic<uint64_t> done;
  cudaError_t e = once_per_device(done, [&]() {
    return cudaFuncSetAttribute(gemm_mx_split_kernel<AF, BN, SWAP>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  });
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute cluster[1];
  cluster[0].id = cudaLaunchAttributeClusterDimension;
  cluster[0].val.clusterDim = {(unsigned)split, 1, 1};
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(tiles * split));
  cfg.blockDim = dim3(32 * C::WARPS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = cluster;
  cfg.numAttrs = split > 1 ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, gemm_mx_split_kernel<AF, BN, SWAP>, g, tm);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int AF>
cudaError_t launch_af(const Operands& o, int split, cudaStream_t s) {
  return o.M <= 16 ? launch<AF, 16, true>(o, split, s) : launch<AF, 128, false>(o, split, s);
}

}  // namespace

namespace gemm_mx {

// The split, by estimates in units of 0.1 us: a stage of a CTA 2, 3 where two CTAs share an
// SM; the cluster's barriers and join 16, or 24 against the tile of gemm_mx.cu beyond 16
// tokens, which needs no detour through shared memory; a second CTA an SM 12.  (Clusters of
// eight leave SMs of a GPC over and double up from about two thirds of the SMs on.)  On one
// B200, us with 4-bit / 8-bit A, K over 1, 2, 4 and 8 CTAs:
//   16 x 6464 x 1024     3.8  4.4  5.6        5.0  5.3  5.7  9.0
//   16 x 1024 x 8192     9.5  7.7  6.0  5.2  16.0 10.9  7.7  6.1
//   16 x 8192 x 8192    11.5 11.1 10.6 13.6  17.6 13.1 11.5 15.4
// (weights of more than L2 in turn), and with gemm_mx.cu's tile, over 2, 4 and 8:
//   128 x 6464 x 1024    4.6  6.0  8.9        5.5  6.8  8.9 16.4
//   128 x 1024 x 8192   10.1  9.1  7.8  7.0  16.9 12.8  9.5  8.0
//   128 x 4096 x 4096    7.0  7.5  7.3 11.0  10.4  9.5  8.3 11.1
//   1024 x 1024 x 8192  10.6 10.8 12.0 20.8  17.8 16.5 15.1 23.7
int split_of(int64_t M, int64_t N, int64_t K, int a_fmt, int64_t sms) {
  const int64_t tiles = ((N + 127) / 128) * ((M + 127) / 128);
  const int64_t stage = a_fmt == mx::kFp4 ? 256 : 128, nk = (K + stage - 1) / stage;
  int best = M <= 16 ? 1 : 0;
  int64_t least = 2 * nk;
  for (int s = 2; s <= 8 && s <= nk && tiles * s <= 2 * sms; s *= 2) {
    const bool two = tiles * s > (s == 8 ? sms * 2 / 3 : sms);
    const int64_t cost =
        (nk + s - 1) / s * (two ? 3 : 2) + (M <= 16 ? 16 : 24) + (two ? 12 : 0);
    if (cost < least) {
      best = s;
      least = cost;
    }
  }
  return best;
}

cudaError_t launch_split(int a_fmt, const Operands& o, int split, cudaStream_t s) {
  return a_fmt == mx::kFp4 ? launch_af<mx::kFp4>(o, split, s) : launch_af<mx::kFp8>(o, split, s);
}

cudaError_t read_and_clear_split_timeouts(unsigned int* count) {
  const unsigned int zero = 0;
  cudaError_t e =
      cudaMemcpyFromSymbol(count, g_gemm_mx_split_wait_timeouts, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_gemm_mx_split_wait_timeouts, &zero, sizeof(unsigned int));
}

}  // namespace gemm_mx
}  // namespace m3ssd
