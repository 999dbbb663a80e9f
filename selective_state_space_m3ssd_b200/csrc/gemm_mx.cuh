// What the microscaled GEMM's kernels share (gemm_mx.cu: tiles over all of K;
// gemm_mx_split.cu: few tokens or tiles, K split over a cluster).
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

// All lanes of a warp wait; a wait that runs out, for any of them, sets the CTA's error word, and
// the warp goes on as one (what follows are instructions of whole warps).  The lanes of
// `give_up` do not wait (a test's).
__device__ __forceinline__ bool wait_all(uint64_t* mbar, uint32_t parity, volatile uint32_t* err,
                                         uint32_t give_up = 0) {
  const bool gave_up = give_up >> (threadIdx.x & 31) & 1u;
  if (__all_sync(0xffffffffu, !gave_up && tc5::mbar_wait(mbar, parity, kWaitLimitNs, err)))
    return true;
  *err = 1;
  return false;
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

}  // namespace gemm_mx
}  // namespace m3ssd
