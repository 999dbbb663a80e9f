// Internal launch interface shared by the C-ABI layer and the kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace m3ssd {

// Lets a kernel have `bytes` of dynamic shared memory: asked for once a device, as a call of it costs
// half a microsecond.  The same bytes at every call.
template <auto KERNEL>
cudaError_t allow_shared(int bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// Everything one forward launch needs; validated by the C-ABI layer.
struct FwdArgs {
  int64_t b, L, H, P, N, G;
  int chunk;
  bool bf16;  // X, B, C, Y are bf16 (else fp32)
  const void* X;
  const float* logdecay;
  const float* beta;   // nullable
  const float* gamma;
  const void* B;
  const void* C;
  const float* theta;  // nullable
  const float* D;      // nullable
  const float* h0;     // nullable
  void* Y;
  float* hT;           // nullable
  const float* angle0; // nullable
  const float* xprev0; // nullable
  const float* bprev0; // nullable
  float* angleT;       // nullable
  float* xprevT;       // nullable
  float* bprevT;       // nullable
  // Head-specific additive biases of B and C, (H, N) fp32, nullable: every use
  // of B (including the cache's bprev0) reads B + Bbias[h], likewise C.  Used by
  // the block (its QK-normed B, C per group plus a bias per head); the public
  // scan entry points leave them NULL.
  const float* Bbias;
  const float* Cbias;
  // Elements between consecutive tokens of X (0: H P, a dense (b, L, H, P)
  // tensor).  The block points X into its in_proj rows this way; only the
  // chunked kernel takes a stride (a multiple of 8).
  int64_t x_tok_stride;
  // The block's raw angle projection instead of theta (chunked kernel only):
  // theta(t, h, i) = Delta(t, h) theta16[t * theta16_tok_stride + h N/2 + i]
  // (bf16), with Delta = logdecay / -exp(A_log[h]) recovered from logdecay.
  const void* theta16;
  int64_t theta16_tok_stride;
  const float* A_log;
  // Sequence split of the chunked bf16 forward (0 or 1: one CTA walks each whole
  // sequence).  With nseg > 1, CTA (b h) nseg + k walks chunks [k segc,
  // min((k + 1) segc, chunks)) of sequence (b, h); segment k >= 1 starts from the
  // state hseg + ((b H + h)(nseg - 1) + k - 1) N P (fp32, (n, p)) and the angle
  // aseg + (same index) N / 2 that the segment pass and its combine step wrote,
  // and only the last segment writes hT and the cache outputs.
  int nseg, segc;
  const float* hseg;
  const float* aseg;
};

struct StepArgs {
  int64_t b, H, P, N, G;
  bool bf16;
  const void* x_t;
  const float* logdecay_t;
  const float* beta_t;   // nullable
  const float* gamma_t;
  const void* B_t;
  const void* C_t;
  const float* theta_t;  // nullable
  const float* D;        // nullable
  float* angle;
  float* ssm;
  float* x_prev;
  float* b_prev;
  void* y_t;
  const float* Bbias;  // nullable, as in FwdArgs
  const float* Cbias;  // nullable
};

// Everything one backward launch needs (gradients are fp32; the nullable
// outputs are not written when absent).
struct BwdArgs {
  int64_t b, L, H, P, N, G;
  bool bf16;  // X, B, C, dY are bf16 (else fp32)
  const void* X;
  const float* logdecay;
  const float* beta;    // nullable
  const float* gamma;
  const void* B;
  const void* C;
  const float* theta;   // nullable
  const float* D;       // nullable
  const float* h0;      // nullable
  const float* angle0;  // nullable
  const float* xprev0;  // nullable
  const float* bprev0;  // nullable
  const void* dY;
  const float* dhT;     // nullable
  float *dX, *dlogdecay, *dbeta, *dgamma, *dB, *dC, *dtheta, *dD, *dh0, *dangle0, *dxprev0,
      *dbprev0;
  void* workspace;      // bwd_workspace_bytes(...) bytes, 256-byte aligned
};

// Workspace of the sequential backward: state checkpoints, the states of one
// block per sequence, and per-head shares of the group-summed gradients.
size_t bwd_workspace_bytes(int64_t b, int64_t L, int64_t H, int64_t P, int64_t N);
cudaError_t launch_bwd_seq(const BwdArgs& a, cudaStream_t s);
// The backward with the state's columns split across CTAs (N = 128, P a
// multiple of 16): checkpoints and block states per (b, h, column slice), and
// per-slice partials of the column-summed gradients.
bool bwd_split_supported(int64_t N, int64_t P);
size_t bwd_split_workspace_bytes(int64_t b, int64_t L, int64_t H, int64_t P);
cudaError_t launch_bwd_split(const BwdArgs& a, cudaStream_t s);
// The chunked backward (N = 128, P = 64): one CTA per (b, h) walks chunks of 63
// tokens, forward for the chunk-start states, then in reverse; per-head shares
// of the group-summed gradients in the workspace.
bool bwd_chunk_supported(int64_t N, int64_t P);
// Workspace regions of the chunked backwards (byte offsets): chunk-start
// states (fp32, (p, n) per chunk) and angles, per-head dB and dC shares,
// per-head dbprev0 shares and per-(b, h) dD partials.
struct ChunkWs {
  size_t hs, phs, dBh, dCh, dbph, dDbh, total;
};
ChunkWs chunk_ws_layout(int64_t b, int64_t L, int64_t H);
// A 4-D TMA tensor map (d0 innermost) with a box of d0-extent `box0` by 64
// tokens; d2 (the token axis) is `tok` elements apart (0: dense, d0 d1).
bool encode_map(CUtensorMap* m, CUtensorMapDataType dt, const void* base, uint64_t d0, uint64_t d1,
                uint64_t d2, uint64_t d3, uint64_t esz, uint32_t box0, CUtensorMapSwizzle sw,
                uint64_t tok = 0);

// Sums the per-head shares into dB, dC, dbprev0 and dD, in a fixed order.
cudaError_t launch_bwd_chunk_reduce(const BwdArgs& a, cudaStream_t s);
// The chunked backward on the tensor cores (bf16 X, B, C, dY; N = 128, P = 64;
// 16-byte aligned X, B, C, dY and theta); same workspace as the fp32 one.
bool bwd_tc_supported(const BwdArgs& a);
cudaError_t launch_bwd_tc(const BwdArgs& a, cudaStream_t s);
cudaError_t read_and_clear_bwd_wait_timeouts(unsigned int* count);
size_t bwd_chunk_workspace_bytes(int64_t b, int64_t L, int64_t H);
cudaError_t launch_bwd_chunk(const BwdArgs& a, cudaStream_t s);

// MIMO rank R (1..8): layouts as the SISO ones with a trailing rank axis on X,
// Y, B, C, x_prev, b_prev (and the extra cache inputs / outputs).
bool mimo_shape_ok(int64_t N, int64_t P, int64_t R);
cudaError_t launch_mimo_fwd(const FwdArgs& a, int64_t R, cudaStream_t s);
// Chunked bf16 tensor-core MIMO forward (N = 128, P = 64, R = 2, 4 or 8; 16-byte
// aligned X, B, C, Y, theta, h0, hT): 64 rows of (token, rank) per chunk.
bool fwd_chunk_mimo_supported(const FwdArgs& a, int64_t R);
cudaError_t launch_fwd_chunk_mimo(const FwdArgs& a, int64_t R, cudaStream_t s);
cudaError_t read_and_clear_mimo_wait_timeouts(unsigned int* count);
// The same for fp32 X, B, C, Y with fp16 high / low operand parts.
bool fwd_chunk_mimo32_supported(const FwdArgs& a, int64_t R);
cudaError_t launch_fwd_chunk_mimo32(const FwdArgs& a, int64_t R, cudaStream_t s);
cudaError_t read_and_clear_mimo32_wait_timeouts(unsigned int* count);
cudaError_t launch_mimo_step(const StepArgs& a, int64_t R, cudaStream_t s);

// Sequential fp32 forward: one CTA per (b, h), token by token.
cudaError_t launch_fwd_seq(const FwdArgs& a, cudaStream_t s);
// Chunked bf16 tensor-core forward (N = 128, P = 64).
cudaError_t launch_fwd_chunk(const FwdArgs& a, cudaStream_t s);
bool fwd_chunk_supported(const FwdArgs& a);
// Sequence split of that forward for launches with few (b, h) sequences: the
// number of segments a sequence is cut into (1: no split) and the chunks a
// segment holds, from the shape and the device's SM count; the workspace the
// split needs (0 without a split); and the split launch itself (the segment
// pass, the combine step and the chunked forward over every segment).
struct SplitPlan {
  int nseg, segc;
};
SplitPlan fwd_split_plan(int64_t b, int64_t L, int64_t H, int sms);
size_t fwd_split_workspace_bytes(int64_t b, int64_t H, const SplitPlan& p);
cudaError_t launch_fwd_split(const FwdArgs& a, const SplitPlan& p, void* workspace, cudaStream_t s);
cudaError_t read_and_clear_seg_wait_timeouts(unsigned int* count);
// SM count of the current device (0 when there is none).
int current_device_sms();
// Chunked fp32 forward on the tensor cores with fp16 high / low operand parts
// (fp32 X, B, C, Y; N = 128, P = 64; 16-byte aligned X, B, C, Y, theta, h0, hT).
// Chunked bf16 forward with chunks of 128 or 256 rows (FwdArgs::chunk), 64-row
// sub-tiles; same shapes and alignment as the 64-row kernel.
bool fwd_chunk_wide_supported(const FwdArgs& a);
cudaError_t launch_fwd_chunk_wide(const FwdArgs& a, cudaStream_t s);
cudaError_t read_and_clear_wide_wait_timeouts(unsigned int* count);
bool fwd_chunk32_supported(const FwdArgs& a);
cudaError_t launch_fwd_chunk32(const FwdArgs& a, cudaStream_t s);
cudaError_t read_and_clear_chunk32_wait_timeouts(unsigned int* count);
// Count of bounded device-side waits in the chunked forward that ran out since
// the last call; reading it synchronises the device and clears the count.
cudaError_t read_and_clear_wait_timeouts(unsigned int* count);
// Test settings of the chunked forward (synchronous copies to device symbols):
// the limit of its bounded waits (0 = 2 s), and a one-shot request that the
// next chunk walk drop its first Gram completion signal.
cudaError_t set_wait_limit_ns(unsigned long long ns);
cudaError_t request_dropped_gram_signal();
// The optional non-finite check: scans n elements (bf16 or fp32) at p on the
// stream and sets a device word when one is NaN or infinite; the host query
// reads and clears it (synchronising the device).
cudaError_t launch_nonfinite_check(const void* p, int64_t n, bool bf16, cudaStream_t s);
cudaError_t read_and_clear_nonfinite(unsigned int* flag);
// D (M x N, bf16, row stride ldd) = A (M x K) W^T on the tensor cores, with A
// (M x K) and W (N x K) bf16 row-major, 16-byte aligned, K a multiple of 8.
cudaError_t launch_gemm_bf16(int64_t M, int64_t N, int64_t K, const void* A, const void* W,
                             void* D, int64_t ldd, cudaStream_t s);
cudaError_t read_and_clear_gemm_wait_timeouts(unsigned int* count);
// The residual addition with the RMS norm (csrc/norm.cu): rows of d values; res and res_out
// nullable together; y in x's type (fmt < 0) or quantised (fmt a mx.cuh format, Kp codes a
// row); rstd nullable.
struct NormArgs {
  int64_t rows, d;
  bool bf16, res_bf16;  // types of x and y, and of res and res_out
  float eps;
  const void* x;
  const void* res;
  const float* w;
  void* y;
  void* res_out;
  float* rstd;
  int fmt;
  int64_t Kp;
  uint8_t* codes;
  uint8_t* scales;
};
// Its backward; `part` holds norm_bwd_workspace_bytes(rows, d) bytes (one partial dw row a
// CTA, so the size depends on the current device's SM count).
struct NormBwdArgs {
  int64_t rows, d;
  bool bf16, res_bf16;  // types of dy and of r
  const void* dy;
  const void* r;
  const float* w;
  const float* rstd;
  const float* dres;  // nullable
  float* dr;
  float* dw;
  float* part;
};
bool norm_width_ok(int64_t d);
// Whether the kernels read columns c to c + 7 of `row` in one access (aligned tensors).
bool norm_whole_access(int64_t rows, int64_t d, int64_t row, int c);
cudaError_t launch_add_rmsnorm(const NormArgs& a, cudaStream_t s);
size_t norm_bwd_workspace_bytes(int64_t rows, int64_t d);
cudaError_t launch_add_rmsnorm_bwd(const NormBwdArgs& a, cudaStream_t s);

// Microscaled formats (csrc/mx.cuh, csrc/mx.cu); fmt 0: E2M1, 1: E4M3 codes.
cudaError_t launch_mx_quant(int fmt, int64_t rows, int64_t cols, bool bf16, const void* x,
                            int64_t ldx, void* codes, void* scales, cudaStream_t s);
cudaError_t launch_mx_dequant(int fmt, int64_t rows, int64_t cols, bool bf16, const void* codes,
                              const void* scales, void* x, int64_t ldx, cudaStream_t s);
// D (M x N, bf16, row stride ldd) = A W^T of a microscaled A (a_fmt, M x K) and E2M1 W
// (N x K), fp32 accumulation (csrc/gemm_mx.cu).
cudaError_t launch_gemm_mx(int a_fmt, int64_t M, int64_t N, int64_t K, const void* A,
                           const void* A_scales, const void* W, const void* W_scales, void* D,
                           int64_t ldd, cudaStream_t s);
// How such a product is taken on a device of `sms` SMs: K split over the CTAs of a cluster
// (split > 0), or not; the tile's tokens there, else its columns; the columns of the parts that
// the last tiles go out in (0: whole).
struct GemmMxPlan {
  int split, tile, part;
};
GemmMxPlan gemm_mx_plan(int a_fmt, int64_t M, int64_t N, int64_t K, int64_t sms);
cudaError_t read_and_clear_gemm_mx_wait_timeouts(unsigned int* count);
// The one-shot request of a test, handed to the launch that asks first: the lanes of the warps
// that wait for a launch's results which give up their first waits at once (0: none).
uint32_t take_given_up_lanes();

// Decode step on a cache whose state is held as E4M3 codes with a scale a row
// (csrc/step_q8.cu); every *_out may be the input it replaces.
struct StepQ8Args {
  int64_t b, H, P, N, G;
  bool bf16;
  const void* x_t;
  const float* logdecay_t;
  const float* beta_t;   // nullable
  const float* gamma_t;
  const void* B_t;
  const void* C_t;
  const float* theta_t;  // nullable
  const float* D;        // nullable
  const float* angle;
  const uint8_t* ssm;
  const float* scale;
  const float* x_prev;
  const float* b_prev;
  float* angle_out;
  uint8_t* ssm_out;
  float* scale_out;
  float* x_prev_out;
  float* b_prev_out;
  void* y_t;
  uint32_t give_up;      // lanes that do not wait for their copies (tests; the launch sets it)
};
cudaError_t launch_step_q8(const StepQ8Args& a, cudaStream_t s);
cudaError_t read_and_clear_step_q8_wait_timeouts(unsigned int* count);
// The state (rows of P fp32 values) into that form and back.
cudaError_t launch_quant_state(int64_t rows, int64_t P, const float* h, void* codes, float* scale,
                               cudaStream_t s);
cudaError_t launch_dequant_state(int64_t rows, int64_t P, const void* codes, const float* scale,
                                 float* h, cudaStream_t s);
// The gated linear recurrence (csrc/glr.cu) over b sequences of L tokens and D channels; x, r, i
// with row strides in elements, y, hT and the state dense.
struct GlrArgs {
  int64_t b, L, D;
  int64_t ldx, ldr, ldi;
  bool bf16;  // type of x, r, i, y (and dy)
  float c;
  const void* x;
  const void* r;
  const void* i;
  const float* rate;
  const float* bias_r;      // nullable
  const float* bias_i;      // nullable
  const float* h0;          // nullable
  const uint8_t* reset;     // nullable, (b, L)
  const int32_t* lengths;   // nullable, (b)
  void* y;                  // the backward reads it
  float* hT;                // nullable
  // A sequence cut into parts (the launches set these): CTAs a sequence (0: it is not),
  // tokens of a part, the parts' maps.
  int split, part_len;
  void* maps;
};
// Its backward.
struct GlrBwdArgs {
  GlrArgs f;
  const void* dy;
  const float* dhT;  // nullable
  bool grad_bf16;
  int64_t ldg;
  void* dx;
  void* dr;
  void* di;
  float* drate;
  float* dbias_r;  // nullable
  float* dbias_i;  // nullable
  float* dh0;      // nullable
  float* part;     // partial sums (the launch sets it)
};
// One step of b sequences; h_out may be h.
struct GlrStepArgs {
  int64_t b, D;
  int64_t ldx, ldr, ldi;
  bool bf16;
  float c;
  const void* x;
  const void* r;
  const void* i;
  const float* rate;
  const float* bias_r;
  const float* bias_i;
  const float* h;
  float* h_out;
  void* y;
};
// Bytes of workspace, by the current device's SM count.
size_t glr_fwd_workspace_bytes(int64_t b, int64_t L, int64_t D, bool bf16);
cudaError_t launch_glr_fwd(const GlrArgs& a, void* workspace, cudaStream_t s);
size_t glr_bwd_workspace_bytes(int64_t b, int64_t L, int64_t D, bool bf16);
cudaError_t launch_glr_bwd(const GlrBwdArgs& a, void* workspace, cudaStream_t s);
cudaError_t launch_glr_step(const GlrStepArgs& a, cudaStream_t s);

// The norm of every head of q (rows x Hq x N) and k (rows x Hk x N) with the rotation of the first R
// pairs by position (csrc/rotate.cu); rows of q and k at strides in elements, outputs dense.
struct RotateArgs {
  int64_t rows, Hq, Hk, N, R;
  int64_t ldq, ldk;
  bool bf16;
  float eps;
  const void* q;
  const void* k;               // nullable where Hk is 0
  const float* q_w;            // nullable (ones)
  const float* k_w;            // nullable (ones)
  const int32_t* positions;    // (rows); nullable where R is 0
  const float* freqs;          // (R); nullable where R is 0
  void* q_out;
  void* k_out;
  // Lanes of a head; slots (of 32 / lanes heads) of a token, the queries' first; slots of a warp's
  // unit and units a token (the launch sets these).
  int lanes, q_slots, slots, block, blocks;
};
struct RotateBwdArgs {
  RotateArgs f;
  bool up_bf16, grad_bf16;
  const void* dq_out;
  const void* dk_out;
  int64_t ldgq, ldgk;
  void* dq;
  void* dk;
  float* dq_w;  // nullable
  float* dk_w;  // nullable
  float* part;  // norm_rotate_bwd_workspace_bytes
};
cudaError_t launch_norm_rotate(const RotateArgs& a, cudaStream_t s);
size_t norm_rotate_bwd_workspace_bytes(const RotateArgs& a);
cudaError_t launch_norm_rotate_bwd(const RotateBwdArgs& a, cudaStream_t s);

// 4-bit weights N x K in groups of columns (csrc/gemv_w4.cu): tiled codes, scales (bf16 bits) and zero points
// (groups x N, nullable: 8), into that form and back.
struct W4Args {
  int64_t N, K, group;
  int groups;
  uint8_t* codes;
  uint16_t* scales;
  uint8_t* zeros;
};
cudaError_t launch_w4_quant(const W4Args& a, bool bf16, const void* w, int64_t ldw, cudaStream_t s);
cudaError_t launch_w4_dequant(const W4Args& a, bool bf16, void* w, int64_t ldw, cudaStream_t s);
// out (M x N) = x (M x K) W^T, M up to 16.
struct GemvW4Args {
  int64_t M, N, K, group;
  int groups;
  bool x_bf16, out_bf16;
  const void* x;
  int64_t ldx;
  const uint8_t* codes;
  const uint16_t* scales;
  const uint8_t* zeros;
  void* out;
  int64_t ldd;
  // The launch sets these: bf16 columns a token and in all, tiles along N and K, tiles of a group,
  // parts of K, tiles of a part and of a part in a piece, rows of tiles of a CTA (and of the first `more`
  // one more), 2^32 over the eights of rows of a CTA, whether tokens and scales can be read 16 bytes at a
  // time.
  int parts, cols;
  int64_t RB, KB;
  int group_tiles, wk, part, per;
  int64_t each, more;
  uint32_t over_eights;
  bool wide, wide_scales;
};
cudaError_t launch_gemv_w4(const GemvW4Args& a, cudaStream_t s);

// Decode step (two launches: the state/outputs, then b_prev <- B_t).
cudaError_t launch_step(const StepArgs& a, cudaStream_t s);

}  // namespace m3ssd
