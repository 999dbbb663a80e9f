/*
 * m3ssd.h -- C ABI of libm3ssd, a B200-native (sm_100a) Mamba-3 SISO selective scan.
 *
 * The operation (sources, by page title and section):
 *   "TorchMamba" README, table "Models" (Mamba-3 SISO row) and "Math notes",
 *   paragraph "M3 SISO": the exponential-trapezoidal three-term recurrence
 *
 *       h_t = alpha_t h_{t-1} + beta_t Bbar_{t-1} x_{t-1}^T + gamma_t Bbar_t x_t^T
 *       y_t = Cbar_t^T h_t + D_h x_t
 *
 *   with alpha_t = exp(logdecay_t) and Bbar_t, Cbar_t equal to B_t, C_t rotated
 *   pairwise by the running data-dependent angle phi_t = angle0 + sum_{s<=t} theta_s
 *   (the "RoPE trick" for a complex state).  "VikramLex/mamba3-minimal",
 *   section "Two-SSD Decomposition": the beta term carries the previous step's
 *   B and x.  "TorchMamba" README, "Behavioral notes": lambda = 1 is the exact
 *   two-term path and theta absent is the real-only path; the Mamba-2 SSD scan
 *   is the lambda = 1, theta = 0 special case ("Reductions").
 *
 * Conventions fixed by this library where the pages are silent:
 *   - pair i is components (2i, 2i+1) and is rotated by theta index i;
 *   - R(phi) = [[cos phi, -sin phi], [sin phi, cos phi]] (counter-clockwise),
 *     applied to both B and C;
 *   - the running angle is inclusive: token t is rotated by phi_t, which
 *     already contains theta_t;
 *   - theta is taken as given (already multiplied by the step size);
 *   - head h reads B/C group g = h / (H / G);
 *   - h0 and hT are in the same absolute frame as Bbar (the cache frame);
 *   - angles written by the library (angleT, cache angle) are reduced to
 *     [-pi, pi] (the same rotation; it keeps fp32 angles precise over long runs).
 *
 * Layouts (row-major, contiguous, element strides implied by the shapes):
 *   X, Y        (b, L, H, P)    dtype x_dtype (fp32 or bf16)
 *   logdecay    (b, L, H)       fp32  (alpha = exp(logdecay))
 *   beta, gamma (b, L, H)       fp32
 *   B, C        (b, L, G, N)    dtype x_dtype
 *   theta       (b, L, H, N/2)  fp32
 *   D           (H)             fp32
 *   h0, hT      (b, H, N, P)    fp32
 *   cache:  angle (b, H, N/2), ssm (b, H, N, P), x_prev (b, H, P),
 *           b_prev (b, G, N) -- all fp32; b_prev holds B_{t-1} UNROTATED and
 *           is rotated at use by the stored angle phi_{t-1}.
 * Decode-step tensors drop the L axis.
 *
 * Ownership and execution: every pointer is a DEVICE pointer owned by the
 * caller.  The library allocates no memory, performs no host synchronisation
 * and enqueues all work on the given stream (a cudaStream_t passed as void*;
 * NULL is the legacy default stream).  Results are complete when the stream
 * reaches the enqueued work.  m3ssd_step is safe to capture in a CUDA graph.
 *
 * Errors: arguments are validated on the host before anything is enqueued;
 * a bad argument returns a status and enqueues nothing.  A launch failure
 * returns M3SSD_ERR_CUDA (the CUDA error is cleared).  Nothing aborts or traps.
 */
#ifndef M3SSD_H_
#define M3SSD_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define M3SSD_ABI_VERSION 1

typedef enum {
  M3SSD_OK = 0,
  M3SSD_ERR_INVALID_ARG = 1,  /* NULL required pointer, odd N, H % G != 0, negative size, aliasing */
  M3SSD_ERR_UNSUPPORTED = 2,  /* valid request outside what this build implements (sizes, chunk, flags) */
  M3SSD_ERR_WORKSPACE = 3,    /* workspace smaller than m3ssd_fwd_workspace_size() or misaligned */
  M3SSD_ERR_CUDA = 4,         /* a CUDA launch failed */
  M3SSD_ERR_NONFINITE = 5,    /* m3ssd_nonfinite_outputs: a checked output held NaN or infinity */
  M3SSD_ERR_TIMEOUT = 6       /* reserved: a bounded device-side wait ran out */
} m3ssd_status;

typedef enum { M3SSD_F32 = 0, M3SSD_BF16 = 1 } m3ssd_dtype;

/* flags (m3ssd_dims.flags) */
/* M3SSD_CHECK_FINITE: after its kernels, m3ssd_fwd (and m3ssd_step,
 * m3ssd_step_q8, m3ssd_mimo_fwd, m3ssd_mimo_step) scans the outputs it wrote -- Y and hT, or
 * y_t -- on the same stream for NaN or infinite values (from an input that was,
 * or from an intermediate that overflowed, e.g. a bf16 input beyond fp16's range
 * on the chunked path); m3ssd_nonfinite_outputs reports what the checks found.
 * It reads the outputs once more (about a fifth of the forward's bytes).  The
 * backward does not take the flag (M3SSD_ERR_UNSUPPORTED).  "Crate burn_mamba"
 * carries the same switch (DENY_NAN / DENY_INF). */
#define M3SSD_CHECK_FINITE 1u

typedef struct {
  int64_t batch;    /* b >= 0 */
  int64_t seqlen;   /* L >= 0 (ignored by m3ssd_step) */
  int64_t nheads;   /* H >= 1 */
  int64_t headdim;  /* P >= 1 */
  int64_t dstate;   /* N >= 2, even */
  int64_t ngroups;  /* G >= 1, H % G == 0 */
  int32_t chunk;    /* chunk length of the chunked forward: 0 = library choice (64),
                       64, or 128 / 256 (bf16, N = 128, P = 64 only; m3ssd_fwd) */
  int32_t x_dtype;  /* m3ssd_dtype of X, B, C, Y (and x_t, B_t, C_t, y_t) */
  uint32_t flags;   /* 0 or M3SSD_CHECK_FINITE */
  uint32_t reserved;/* must be 0 */
} m3ssd_dims;

/* Optional cache-shaped inputs and outputs of the forward, so that a forward
 * can start from a decode cache and hand one back (prefill -> decode).
 * Inputs may be NULL (read as zero); outputs may be NULL (not written).
 * angleT/xprevT may alias angle0/xprev0; bprevT must NOT alias bprev0
 * (several heads read a group's b_prev).  Note h0/hT live in m3ssd_fwd's own
 * arguments and may alias each other. */
typedef struct {
  const float* angle0;  /* (b, H, N/2): phi_{-1} */
  const float* xprev0;  /* (b, H, P):   x_{-1}   */
  const float* bprev0;  /* (b, G, N):   B_{-1}, unrotated */
  float* angleT;        /* (b, H, N/2): phi_{L-1} */
  float* xprevT;        /* (b, H, P):   x_{L-1} as fp32 */
  float* bprevT;        /* (b, G, N):   B_{L-1} as fp32, unrotated */
} m3ssd_fwd_extra;

typedef struct {
  float* angle;   /* (b, H, N/2) */
  float* ssm;     /* (b, H, N, P) */
  float* x_prev;  /* (b, H, P) */
  float* b_prev;  /* (b, G, N), unrotated */
} m3ssd_cache;

/* Bytes of device workspace m3ssd_fwd needs for these dims on the current
 * device: non-zero only when the chunked bf16 forward (N = 128, P = 64, chunk 0
 * or 64) splits each sequence into segments (see m3ssd_fwd), which depends on
 * batch, seqlen, nheads and the device's SM count, so query it on the device
 * that runs the call.  0 for invalid dims (m3ssd_fwd then reports the error)
 * and when no device is present. */
size_t m3ssd_fwd_workspace_size(const m3ssd_dims* dims);

/* The segment count and the chunks per segment that m3ssd_fwd would use for
 * batch x nheads sequences of seqlen tokens on a device with `sms` SMs
 * (*nseg = 1: no split).  Host arithmetic only; for tests and tuning.
 * M3SSD_ERR_INVALID_ARG for NULL outputs or negative sizes. */
m3ssd_status m3ssd_test_fwd_split_plan(int64_t batch, int64_t seqlen, int64_t nheads,
                                       int32_t sms, int32_t* nseg, int32_t* segc);

/*
 * Forward scan over a whole sequence ("TorchMamba" README, "Functional cores":
 * trap_rope_loop(X, logdecay, B, C, theta_dt, lam) -> (y, h)).
 *
 *   X, logdecay, gamma, B, C, Y : required when b*L > 0.
 *   beta   : NULL selects the exact two-term path (lambda = 1).
 *   theta  : NULL selects the real-only path (no rotation).
 *   D      : NULL means D = 0.
 *   h0     : NULL means a zero initial state.
 *   hT     : NULL means the final state is not written.
 *   extra  : NULL means no cache inputs/outputs (see m3ssd_fwd_extra).
 *   workspace, workspace_bytes : device scratch of at least
 *            m3ssd_fwd_workspace_size(dims) bytes, 256-byte aligned (may be
 *            NULL when that size is 0).
 *
 * Paths ("TorchMamba" README, "Math notes", M2: chunkwise intra-quadratic with
 * an inter-chunk carry):
 *   x_dtype = BF16, N = 128, P = 64, 16-byte aligned tensors: the chunked
 *     tensor-core forward (fp32 accumulation and state, fp16 operands converted
 *     from the bf16 inputs; X, B, C and their Gram products must stay inside
 *     fp16's range).  dims->chunk = 0 or 64 walks chunks of 64 rows (63 new
 *     tokens); 128 or 256 makes the intra-chunk quadratic form span 128 or 256
 *     rows (one CTA per SM instead of two).  With chunks of 64 rows and too few
     (b, h) sequences to fill the device (b*H at most two thirds of its SM
     count, at least 16 chunks), each sequence is cut into segments of at
     least 8 chunks: a pass builds every segment's state from a zero start
     and the linear recurrence links them (each segment's start state is the
     decayed previous start plus the previous segment's state, rotated to the
     absolute angle), then all segments run at once.  The result equals the
     unsplit walk up to fp32 rounding order; the workspace holds the segment
     states (64 KB per sequence and segment).
 *   x_dtype = F32, N = 128, P = 64, 16-byte aligned tensors: the chunked forward
 *     with every product on fp16 high and low operand parts (about 2^-22 of
 *     each term), chunk 0 or 64.
 *   every other valid request: the sequential fp32 forward (N <= 256,
 *     P <= 256, N*P <= 16384, else M3SSD_ERR_UNSUPPORTED); chunk 0 or 64.
 * A chunk of 128 or 256 outside the bf16 N = 128, P = 64 path returns
 * M3SSD_ERR_UNSUPPORTED.  Y is rounded once to x_dtype (round-to-nearest-even);
 * hT and the extra outputs are fp32.
 */
m3ssd_status m3ssd_fwd(const m3ssd_dims* dims, const void* X, const float* logdecay,
                       const float* beta, const float* gamma, const void* B, const void* C,
                       const float* theta, const float* D, const float* h0, void* Y, float* hT,
                       const m3ssd_fwd_extra* extra, void* workspace, size_t workspace_bytes,
                       void* stream);

/*
 * One decode step on a cache ("TorchMamba" README, "API reference": step(u_t,
 * cache) with Mamba3SisoCache(angle, ssm, x_prev, b_prev)):
 *   phi' = angle + theta_t;  Bbar_prev = R(angle) b_prev;  Bbar = R(phi') B_t;
 *   Cbar = R(phi') C_t;  ssm = alpha ssm + beta Bbar_prev x_prev^T + gamma Bbar x_t^T;
 *   y_t = Cbar^T ssm + D x_t;  then angle = phi', x_prev = x_t, b_prev = B_t.
 * x_t, y_t (b, H, P) and B_t, C_t (b, G, N) have dtype dims->x_dtype;
 * logdecay_t, beta_t, gamma_t (b, H) and theta_t (b, H, N/2) are fp32.
 * beta_t, theta_t, D may be NULL (zero).  dims->seqlen is ignored.
 * Limits: N <= 256, P <= 256, N*P <= 16384.  Capture-safe (no allocation, no sync).
 */
m3ssd_status m3ssd_step(const m3ssd_dims* dims, const void* x_t, const float* logdecay_t,
                        const float* beta_t, const float* gamma_t, const void* B_t,
                        const void* C_t, const float* theta_t, const float* D,
                        const m3ssd_cache* cache, void* y_t, void* stream);

/*
 * MIMO rank R forward ("TorchMamba" README, table "Models", row Mamba-3 MIMO:
 * a rank-R matmul update on a shared (N, P) state; "Functional cores":
 * mimo_loop with X (B,L,H,P,R) -> Y (B,L,H,P,R), h (B,H,N,P)):
 *   h_t = alpha_t h_{t-1} + beta_t sum_r Bbar_{t-1,r} x_{t-1,r}^T + gamma_t sum_r Bbar_{t,r} x_{t,r}^T
 *   y_{t,r} = Cbar_{t,r}^T h_t + D x_{t,r}
 * with every rank column of B and C rotated by the head's angle.  Layouts as
 * m3ssd_fwd with a trailing rank axis: X, Y (b, L, H, P, R); B, C
 * (b, L, G, N, R); extra->xprev0 / xprevT (b, H, P, R) and bprev0 / bprevT
 * (b, G, N, R); the state h0, hT stays (b, H, N, P).  1 <= rank <= 8, N <= 256,
 * P <= 256, N*P <= 16384 (else M3SSD_ERR_UNSUPPORTED).  Sequential fp32 state;
 * Y rounded once to x_dtype.  No workspace, no allocation, no synchronisation.
 */
m3ssd_status m3ssd_mimo_fwd(const m3ssd_dims* dims, int32_t rank, const void* X,
                            const float* logdecay, const float* beta, const float* gamma,
                            const void* B, const void* C, const float* theta, const float* D,
                            const float* h0, void* Y, float* hT, const m3ssd_fwd_extra* extra,
                            void* stream);

/*
 * One MIMO decode step on a cache whose x_prev is (b, H, P, R) and b_prev
 * (b, G, N, R) (angle and ssm as for m3ssd_step); x_t, y_t (b, H, P, R) and
 * B_t, C_t (b, G, N, R) have dtype dims->x_dtype.  Limits as m3ssd_mimo_fwd.
 * Two launches (the step, then b_prev <- B_t).  No allocation, no synchronisation.
 */
m3ssd_status m3ssd_mimo_step(const m3ssd_dims* dims, int32_t rank, const void* x_t,
                             const float* logdecay_t, const float* beta_t, const float* gamma_t,
                             const void* B_t, const void* C_t, const float* theta_t,
                             const float* D, const m3ssd_cache* cache, void* y_t, void* stream);

/* fp32 gradient outputs of m3ssd_bwd, each shaped like the matching input of
 * m3ssd_fwd (dB, dC, dbprev0 per group; dD per head).  dX, dlogdecay, dgamma,
 * dB, dC are required when b*L > 0; the others may be NULL (not written).  An
 * input passed to the forward as NULL is read as zero, and its gradient is the
 * derivative there. */
typedef struct {
  float* dX;         /* (b, L, H, P) */
  float* dlogdecay;  /* (b, L, H) */
  float* dbeta;      /* (b, L, H) */
  float* dgamma;     /* (b, L, H) */
  float* dB;         /* (b, L, G, N) */
  float* dC;         /* (b, L, G, N) */
  float* dtheta;     /* (b, L, H, N/2) */
  float* dD;         /* (H) */
  float* dh0;        /* (b, H, N, P) */
  float* dangle0;    /* (b, H, N/2) */
  float* dxprev0;    /* (b, H, P) */
  float* dbprev0;    /* (b, G, N) */
} m3ssd_bwd_grads;

/* Bytes of device workspace m3ssd_bwd needs for these dims (0 for invalid
 * dims, and for any flags, which the backward refuses); the size depends on
 * the path.  At N = 128, P = 64 it holds every
 * chunk-start state and angle (chunks of 63 tokens) and per-head shares of
 * the group-summed gradients: about 4 (b H ceil(L/63) (N P + N/2) +
 * 2 b L H N) bytes.  Other shapes keep a state checkpoint every 16 or 64
 * tokens, the states of one block per sequence and the same per-head (or
 * per-slice) shares. */
size_t m3ssd_bwd_workspace_size(const m3ssd_dims* dims);

/*
 * Backward of m3ssd_fwd: reverse-mode derivatives of the recurrence of the
 * "TorchMamba" README, "Math notes", M3 SISO.  Training through the scan is on
 * the pages: "mamba-rs" crate page, feature list (CUDA forward and backward
 * kernels); "TorchMamba" README, "Verification" (fp64 gradchecks per core).
 *
 * Takes the forward's inputs (same pointers, dtypes and NULL conventions;
 * extra supplies angle0, xprev0, bprev0 and its outputs are ignored), the
 * upstream gradients dY (b, L, H, P, dtype x_dtype) and dhT (b, H, N, P,
 * fp32, NULL = 0), and writes the fp32 gradients in *grads.  The cache outputs
 * angleT, xprevT and bprevT take no upstream gradient.
 *
 * The backward recomputes the forward.  At N = 128, P = 64 it works chunk by
 * chunk (one CTA per sequence: a forward pass stores the state and angle at
 * every chunk start, then each chunk's adjoint is a set of products, walking
 * the chunks in reverse): with bf16 X, B, C, dY (16-byte aligned, as theta)
 * the products run on the tensor cores with every fp32 operand split into a
 * bf16 high part and residual (about 2^-16 relative error per product term;
 * gradients within about 1e-3 of their RMS at L = 4096), otherwise in fp32.  At N = 128 with
 * another P a multiple of 16 it splits each sequence over P/16 CTAs of 16
 * state columns and sums the per-slice partials of the column-mixing
 * gradients afterwards; other shapes run one CTA per sequence token by
 * token.  Every sum (over slices, the heads of a group, the batch) runs in a
 * fixed order, so results are deterministic.  Limits as the sequential forward:
 * N <= 256, P <= 256, N*P <= 16384 (else M3SSD_ERR_UNSUPPORTED); dims->flags
 * must be 0 (else M3SSD_ERR_UNSUPPORTED).  workspace must hold
 * m3ssd_bwd_workspace_size(dims) bytes, 256-byte aligned (else
 * M3SSD_ERR_WORKSPACE); the size depends on the path.  No allocation, no
 * synchronisation.
 */
m3ssd_status m3ssd_bwd(const m3ssd_dims* dims, const void* X, const float* logdecay,
                       const float* beta, const float* gamma, const void* B, const void* C,
                       const float* theta, const float* D, const float* h0,
                       const m3ssd_fwd_extra* extra, const void* dY, const float* dhT,
                       const m3ssd_bwd_grads* grads, void* workspace, size_t workspace_bytes,
                       void* stream);

/*
 * m3ssd_bwd without a caller workspace, for callers that cannot allocate
 * device memory where they call the backward (code inside a CUDA graph
 * capture, or a runtime whose allocator may not be used from the launching
 * thread).  The scratch is a fixed 64 MiB device array inside the library,
 * reserved when its device code is loaded on a device and kept by every GPU
 * that loads the library until the process exits.  The pages have no
 * counterpart for this entry point; it is a convenience of this library.
 * Arguments and results are those of m3ssd_bwd.  Invalid dims return
 * m3ssd_bwd's status without touching the device; requests whose
 * m3ssd_bwd_workspace_size exceeds 64 MiB return M3SSD_ERR_UNSUPPORTED before
 * any device call.  The first call on a device (with that device current)
 * looks up the array's device address once (cudaGetSymbolAddress); make that
 * first call before any stream capture.  No call allocates.  Every call uses
 * the same array, which keeps the last call's contents, so calls that overlap
 * on the GPU race: issue them on one stream, or synchronise between streams.
 */
m3ssd_status m3ssd_bwd_noalloc(const m3ssd_dims* dims, const void* X, const float* logdecay,
                               const float* beta, const float* gamma, const void* B,
                               const void* C, const float* theta, const float* D,
                               const float* h0, const m3ssd_fwd_extra* extra, const void* dY,
                               const float* dhT, const m3ssd_bwd_grads* grads, void* stream);

/*
 * The Mamba-3 SISO block around the scan ("VikramLex/mamba3-minimal" README,
 * "Architecture", the Mamba3 SSM box; "TorchMamba" README, "API reference",
 * Mamba3SisoBlock with forward / prefill / step and its cache):
 *
 *   zx = u W_in^T                       in_proj, no bias
 *   [z | x | B | C | dt | lam | theta] = zx   (widths H P, H P, G N, G N, H, H, H N/2;
 *                                              heads outermost inside each part)
 *   Delta = softplus(dt + dt_bias), logdecay = -exp(A_log) Delta,
 *   lambda = sigmoid(lam), gamma = lambda Delta, beta = (1 - lambda) Delta exp(logdecay),
 *   theta_dt = Delta theta
 *   B'_h = B_g / sqrt(mean_n B_g^2 + eps) * B_norm_w + B_bias[h]   (QK-norm, then the
 *   C'_h likewise                                                   head-specific BC bias)
 *   y = scan(x, logdecay, beta, gamma, B', C', theta_dt, D)        (the SISO scan above,
 *                                                                    one B/C per head)
 *   out = (y * SiLU(z)) W_out^T          out_proj, no bias
 *
 * The projections are plain GEMMs on this library's tensor-core GEMM
 * (m3ssd_gemm_bf16: bf16 operands, fp32 accumulation, bf16 outputs); the rest
 * runs in this library's kernels too, the head biases inside the scan (added
 * in fp32 before the rotation).  u and out are bf16.  The block cache is an m3ssd_cache with
 * b_prev (b, G, N) holding the QK-normed group vector B_{t-1} (times its norm
 * weight, without the head bias) unrotated; the bias is added at use.
 */
typedef struct {
  int64_t batch;    /* b >= 0 */
  int64_t seqlen;   /* L >= 0 (ignored by m3ssd_block_step) */
  int64_t d_model;  /* >= 1, a multiple of 8 */
  int64_t nheads;   /* H >= 1 */
  int64_t headdim;  /* P >= 1, H * P a multiple of 8 */
  int64_t dstate;   /* N >= 2, even */
  int64_t ngroups;  /* G >= 1, H % G == 0 */
} m3ssd_block_dims;

typedef struct {
  const void* W_in;       /* (2HP + 2GN + 2H + H N/2, d_model) bf16, row-major */
  const void* W_out;      /* (d_model, H P) bf16, row-major */
  const float* dt_bias;   /* (H) */
  const float* A_log;     /* (H) */
  const float* D;         /* (H), may be NULL (zero) */
  const float* B_norm_w;  /* (N) */
  const float* C_norm_w;  /* (N) */
  const float* B_bias;    /* (H, N) */
  const float* C_bias;    /* (H, N) */
  float eps;              /* >= 0 */
} m3ssd_block_weights;

/* Bytes of device workspace m3ssd_block_fwd needs for these dims (with
 * seqlen = 1 it also covers m3ssd_block_step); 0 for invalid dims. */
size_t m3ssd_block_workspace_size(const m3ssd_block_dims* dims);

/*
 * Block forward over a sequence (Mamba3SisoBlock.forward; with cache_out it is
 * prefill).  u, out: (b, L, d_model) bf16.  cache_in (may be NULL: start from
 * zero) is the state the sequence continues from; cache_out (may be NULL) gets
 * the state after the last token and may be the same object as cache_in.
 * workspace: workspace_bytes >= m3ssd_block_workspace_size(dims), 256-byte
 * aligned, not read afterwards.  Errors as m3ssd_fwd.
 */
m3ssd_status m3ssd_block_fwd(const m3ssd_block_dims* dims, const m3ssd_block_weights* w,
                             const void* u, void* out, const m3ssd_cache* cache_in,
                             const m3ssd_cache* cache_out, void* workspace,
                             size_t workspace_bytes, void* stream);

/*
 * The block's projection GEMM ("VikramLex/mamba3-minimal" README,
 * "Architecture": in_proj and out_proj are plain linear maps), exported for
 * callers that compose the block themselves:
 *     D (M x N, row stride ldd elements) = A (M x K) W^T
 * A (M x K) and W (N x K): bf16, row-major (row stride K), 16-byte aligned,
 * K a multiple of 8; D: bf16, ldd >= N, 2-byte aligned (tensor stores when D
 * is 16-byte aligned and N and ldd are multiples of 8).  fp32 accumulation on the
 * tensor cores, each output rounded once to bf16 (nearest even).  M, N, K up
 * to 2^31 - 1 with at most 2^31 - 1 output tiles of 128 x 256; M = 0 or N = 0
 * does nothing.  Other shapes or alignments: M3SSD_ERR_INVALID_ARG (or
 * M3SSD_ERR_CUDA for a tile count past that limit).  No allocation, no
 * synchronisation.
 */
m3ssd_status m3ssd_gemm_bf16(int64_t M, int64_t N, int64_t K, const void* A, const void* W,
                             void* D, int64_t ldd, void* stream);

/*
 * One decode step of the block (Mamba3SisoBlock.step): u_t, out_t (b, d_model)
 * bf16; cache (required) is advanced in place.  workspace as for
 * m3ssd_block_fwd with seqlen = 1.  Capturable in a CUDA graph.
 */
m3ssd_status m3ssd_block_step(const m3ssd_block_dims* dims, const m3ssd_block_weights* w,
                              const void* u_t, void* out_t, const m3ssd_cache* cache,
                              void* workspace, size_t workspace_bytes, void* stream);

/*
 * The residual addition with the root-mean-square norm that stands before the block in a
 * layer ("VikramLex/mamba3-minimal" README, "Architecture": x + mixer(norm(x))), over
 * rows of `width` values:
 *     r = x + residual (rounded once to res_dtype; r = x when residual is NULL),
 *     rstd = 1 / sqrt(mean r^2 + eps),   y = r rstd w
 * computed in fp32, y rounded once to x_dtype or quantised to a microscaled format (below).
 */
typedef struct {
  int64_t rows;      /* >= 0 (tokens) */
  int64_t width;     /* 1 .. 16384 (else M3SSD_ERR_UNSUPPORTED) */
  int32_t x_dtype;   /* m3ssd_dtype of x and y (and of dy) */
  int32_t res_dtype; /* m3ssd_dtype of residual and residual_out (and of r) */
  float eps;         /* >= 0 */
  uint32_t reserved; /* must be 0 */
} m3ssd_norm_dims;

/*
 * Microscaled (MX) tensors: rows of `cols` values in blocks of 32, each block with a
 * power-of-two scale 2^E, the least with amax <= maxval 2^E, and codes value / 2^E rounded
 * to nearest even: E2M1 (4 bits, maxval 6) or E4M3 (8 bits, maxval 448).  E is clamped to
 * [-127, 127] and held as the byte E + 127; a block of zeros takes byte 0; a block with a
 * NaN or an infinity takes byte 255 (NaN) and reads back as NaN.
 *   codes:  rows x Kp codes, Kp = cols rounded up to 128, the padding zero; E2M1 two codes
 *           a byte, the even index in the low half.  m3ssd_mx_codes_size bytes.
 *   scales: tiles of 128 rows x 4 blocks, 512 bytes each, row-block-major: byte
 *           (r % 32) 16 + (r / 32) 4 + k of row r and block k of the tile; bytes of missing
 *           rows 0.  m3ssd_mx_scales_size bytes.
 * Both 128-byte aligned.  At most 2^31 - 1 groups of 128 columns over the rows rounded up
 * to 128 (else M3SSD_ERR_UNSUPPORTED).  The functions that write one write the padding too.
 */
typedef enum { M3SSD_MXFP4 = 0, M3SSD_MXFP8 = 1 } m3ssd_mx_format;
typedef struct {
  int32_t format;    /* m3ssd_mx_format */
  uint32_t reserved; /* must be 0 */
  int64_t rows;      /* >= 0 */
  int64_t cols;      /* >= 1 */
  void* codes;
  void* scales;
} m3ssd_mx;

/* Bytes of the codes and of the scales; 0 for invalid arguments. */
size_t m3ssd_mx_codes_size(int32_t format, int64_t rows, int64_t cols);
size_t m3ssd_mx_scales_size(int64_t rows, int64_t cols);

/* x (rows x cols, row stride ldx >= cols elements, x_dtype) to and from an MX tensor.  Read
 * back, a value is code 2^E, rounded once to x_dtype: exact unless it is subnormal there, or
 * was rounded up from the type's largest values past its range (then infinite). */
m3ssd_status m3ssd_mx_quant(const m3ssd_mx* out, int32_t x_dtype, const void* x, int64_t ldx,
                            void* stream);
m3ssd_status m3ssd_mx_dequant(const m3ssd_mx* in, int32_t x_dtype, void* x, int64_t ldx,
                              void* stream);

/*
 * D (M x N, bf16, row stride ldd >= N) = A W^T of MX operands A (M x K, either format) and
 * W (N x K, M3SSD_MXFP4; else M3SSD_ERR_UNSUPPORTED), beside m3ssd_gemm_bf16 for the block's
 * projections with quantised weights.  Products of the held values, fp32 accumulation on
 * the tensor cores, each output rounded once to bf16.  The order of the sums over K goes by
 * the shapes alone: the same call gives the same bits, one of other M or N may round an
 * output otherwise.  D 2-byte aligned (tensor stores when D is 16-byte aligned and N and ldd
 * are multiples of 8).  No allocation, no synchronisation.
 */
m3ssd_status m3ssd_gemm_mx(const m3ssd_mx* A, const m3ssd_mx* W, void* D, int64_t ldd,
                           void* stream);

/* How m3ssd_gemm_mx takes such a product on a device with `sms` SMs: *split CTAs of a cluster
 * share a tile's K, *tile tokens wide (0: no split; *tile columns of D), and the tiles left
 * over after whole rounds go out in parts of *part columns (0: whole).  Host arithmetic only;
 * for tests and tuning. */
m3ssd_status m3ssd_test_gemm_mx_plan(int32_t a_format, int64_t M, int64_t N, int64_t K,
                                     int32_t sms, int32_t* split, int32_t* tile, int32_t* part);

/*
 * Forward of the residual addition and norm.  residual and residual_out are given together
 * or not at all; residual_out may be residual.  Exactly one of y (rows x width, x_dtype; may
 * be x, not residual_out) and y_mx (an MX tensor of rows x width, the A operand of m3ssd_gemm_mx) is given.
 * rstd (rows), for the backward, may be NULL.  x, y, residual: dense rows.
 */
m3ssd_status m3ssd_add_rmsnorm(const m3ssd_norm_dims* dims, const void* x, const void* residual,
                               const float* w, void* y, const m3ssd_mx* y_mx, void* residual_out,
                               float* rstd, void* stream);

/* Bytes of device workspace m3ssd_add_rmsnorm_bwd needs on the current device (it depends
 * on the SM count); 0 for invalid dims. */
size_t m3ssd_add_rmsnorm_bwd_workspace_size(const m3ssd_norm_dims* dims);

/*
 * Its backward.  dy (rows x width, x_dtype) is the gradient of y, dres (fp32, NULL = 0)
 * that of residual_out; r (res_dtype) is residual_out (or x without a residual, with
 * res_dtype = x_dtype) and rstd the forward's.  Writes fp32 dr (rows x width; may be dres),
 * the gradient of x and of residual alike, and dw (width).  With g = w dy, rhat = r rstd:
 *     dr = rstd (g - rhat mean(g rhat)) + dres,   dw = sum over rows of dy rhat.
 * Sums run in a fixed order, so results are deterministic.  workspace: 256-byte aligned,
 * not read afterwards.
 */
m3ssd_status m3ssd_add_rmsnorm_bwd(const m3ssd_norm_dims* dims, const void* dy, const void* r,
                                   const float* w, const float* rstd, const float* dres, float* dr,
                                   float* dw, void* workspace, size_t workspace_bytes,
                                   void* stream);

/* Whether the norm's kernels read columns `column` to `column` + 7 of `row` in one access, as
 * they may where the columns lie inside an aligned tensor (`column` is negative where a row
 * starts inside the access).  Host arithmetic only; for tests. */
m3ssd_status m3ssd_test_norm_access(const m3ssd_norm_dims* dims, int64_t row, int32_t column,
                                    int32_t* whole);

/*
 * A decode cache whose state is held in 8 bits.  A row (b, h, n) of the state, P values, is
 * E4M3 codes with one fp32 scale: s = amax fp32(1 / 448), code = v (1 / s) rounded to nearest
 * even, v ~ code s.  The reciprocal is correctly rounded in m3ssd_quant_state and within an ulp
 * in m3ssd_step_q8, so that a value at a border between two codes may take either there.  Rows
 * with amax < 2^-100 are held as zeros (s = 0, codes 0 or -0); a row with a NaN or an infinity
 * takes a NaN scale and reads back as NaN.  A held value is within 2^-4 of its magnitude or
 * 2^-10 s, whichever is larger, and 2^-23 of it for the reciprocal.
 */
typedef struct {
  float* angle;      /* (b, H, N/2) */
  void* ssm;         /* (b, H, N, P) E4M3 codes */
  float* ssm_scale;  /* (b, H, N) */
  float* x_prev;     /* (b, H, P) */
  float* b_prev;     /* (b, G, N), unrotated */
} m3ssd_cache_q8;

/* A whole fp32 state (b, H, N, P), as the forward writes hT, to that form and back
 * (prefill -> 8-bit decode).  dims: batch, nheads, headdim, dstate (seqlen and chunk are
 * ignored); limits as m3ssd_step. */
m3ssd_status m3ssd_quant_state(const m3ssd_dims* dims, const float* ssm, void* codes, float* scale,
                               void* stream);
m3ssd_status m3ssd_dequant_state(const m3ssd_dims* dims, const void* codes, const float* scale,
                                 float* ssm, void* stream);

/*
 * m3ssd_step on such a cache: the state is read as code s, y_t comes from the updated fp32
 * state before it is rounded, and the state is rounded once as it is written.  The new
 * cache goes to cache_out, which may be another cache (the old one stays, for a rollback)
 * or NULL or the same (in place); its buffers equal the cache's or do not overlap them.
 * Arguments, limits and flags as m3ssd_step; angles and theta up to about 1e5 in magnitude
 * (the library's own are reduced).  One launch, or two where b_prev is written in place.
 * Capture-safe (no allocation, no sync).
 */
m3ssd_status m3ssd_step_q8(const m3ssd_dims* dims, const void* x_t, const float* logdecay_t,
                           const float* beta_t, const float* gamma_t, const void* B_t,
                           const void* C_t, const float* theta_t, const float* D,
                           const m3ssd_cache_q8* cache, const m3ssd_cache_q8* cache_out, void* y_t,
                           void* stream);

/*
 * The gated linear recurrence, one state a channel ("TorchMamba" README, "Functional cores",
 * has the matrix-state recurrences; a layer that mixes tokens channel by channel runs this one
 * beside them).  Over (b, L, width), per channel, with k = c softplus(rate):
 *     rho = sigma(r + bias_r),  iota = sigma(i + bias_i),  a = exp(-k rho),
 *     h_t = a_t h_{t-1} + sqrt(1 - a_t^2) iota_t x_t,   y_t = h_t,
 * computed in fp32 (1 - a_t^2 to fp32's relative precision however close a_t is to one, down
 * to 1e-37, in the backward to 1e-29 and below that its root within 4e-19; a gate below 2^-63 counts
 * as that, an a_t below 2^-126 as zero), h held in fp32, y rounded once to x_dtype.  A state that is
 * infinite or NaN is one or the other until the next reset.
 */
typedef struct {
  int64_t batch;      /* b >= 0 */
  int64_t seqlen;     /* L >= 0 (ignored by m3ssd_glr_step) */
  int64_t width;      /* channels, >= 1 */
  int64_t ldx;        /* elements from a token's x to the next one's, >= width: x, r and i may */
  int64_t ldr;        /*   be column ranges of one projection's rows; token t of sequence b is */
  int64_t ldi;        /*   row b L + t (row b of the step) */
  int32_t x_dtype;    /* m3ssd_dtype of x, r, i, y and dy */
  float c;            /* > 0, finite */
  uint32_t reserved;  /* must be 0 */
} m3ssd_glr_dims;

/* Bytes of device workspace m3ssd_glr_fwd needs on the current device: non-zero where few
 * sequences are cut into parts, which goes by the sizes and the device's SM count.  0 for
 * invalid dims. */
size_t m3ssd_glr_fwd_workspace_size(const m3ssd_glr_dims* dims);

/*
 * Forward.  rate, bias_r, bias_i (width) and h0, hT (b, width) are fp32; bias_r, bias_i and h0
 * may be NULL (zero), hT may be NULL or h0.  y: dense (b, L, width).
 *   reset (b, L) uint8, may be NULL: where it is not zero a sequence starts anew, a_t = 0
 *     (whatever h_{t-1} was, NaN and infinity included), as between packed documents.
 *   lengths (b) int32, may be NULL (L): the tokens of each sequence, taken between 0 and L.
 *     Later rows of x, r, i and reset are not read, those of y are zero, hT is the state after
 *     the last token (h0 where there is none).
 * width up to 2^25 - 1, L up to 2^30 - 1, b times half the width and every stride up to 2^31 - 1
 * (else M3SSD_ERR_UNSUPPORTED).  y overlaps no input.  workspace: 256-byte aligned, not read
 * afterwards.  No allocation, no synchronisation; capture-safe.
 */
m3ssd_status m3ssd_glr_fwd(const m3ssd_glr_dims* dims, const void* x, const void* r, const void* i,
                           const float* rate, const float* bias_r, const float* bias_i,
                           const float* h0, const uint8_t* reset, const int32_t* lengths, void* y,
                           float* hT, void* workspace, size_t workspace_bytes, void* stream);

/* Gradients: dx, dr, di (b, L, width) in `dtype` (fp32, or bf16 where x_dtype is: each value
 * rounded once), their rows `ld` elements apart, so that they may be column ranges of one
 * projection's gradient; drate, dbias_r, dbias_i (width) and dh0 (b, width) fp32.  dbias_r,
 * dbias_i and dh0 may be NULL. */
typedef struct {
  int64_t ld;         /* width .. 2^25 - 1 */
  int32_t dtype;      /* m3ssd_dtype */
  uint32_t reserved;  /* must be 0 */
  void* dx;
  void* dr;
  void* di;
  float* drate;
  float* dbias_r;
  float* dbias_i;
  float* dh0;
} m3ssd_glr_grads;

/* Bytes of device workspace m3ssd_glr_bwd needs on the current device; 0 for invalid dims. */
size_t m3ssd_glr_bwd_workspace_size(const m3ssd_glr_dims* dims);

/*
 * Backward of m3ssd_glr_fwd: its inputs, its output y, dy (dense, x_dtype) and dhT (b, width,
 * fp32, NULL = 0).  With g_t = dy_t + a_{t+1} g_{t+1} (dhT added at the last token), s =
 * sqrt(1 - a^2):
 *     dx = g s iota,  di = dx x (1 - iota),
 *     E = g a (h_{t-1} - a iota x / s) log a,  dr = E (1 - rho),
 *     drate = sum of E sigma(rate) / softplus(rate),  dbias_r, dbias_i = sums of dr and di,
 *     dh0 = a_0 g_0
 * (E = dr = 0 at a reset).  h_{t-1} is read as the stored y_{t-1}, which saves a second walk
 * forward: in bf16 that is h rounded by up to 2^-8 of its value.  Rows at
 * and past lengths[b] are zero.  Sums run in fp32 in a fixed order: the same call gives
 * the same bits.  dh0 may be dhT; the other outputs overlap no input.  workspace: 256-byte
 * aligned, not read afterwards.
 */
m3ssd_status m3ssd_glr_bwd(const m3ssd_glr_dims* dims, const void* x, const void* r, const void* i,
                           const float* rate, const float* bias_r, const float* bias_i,
                           const float* h0, const uint8_t* reset, const int32_t* lengths,
                           const void* y, const void* dy, const float* dhT,
                           const m3ssd_glr_grads* grads, void* workspace, size_t workspace_bytes,
                           void* stream);

/* One token of each sequence: x_t, r_t, i_t (b, width, rows ldx, ldr, ldi apart), the state h
 * (b, width) fp32 to h_out (NULL: in place; else h or no overlap), y_t dense. */
m3ssd_status m3ssd_glr_step(const m3ssd_glr_dims* dims, const void* x_t, const void* r_t,
                            const void* i_t, const float* rate, const float* bias_r,
                            const float* bias_i, const float* h, float* h_out, void* y_t,
                            void* stream);

/*
 * Queries and keys, the scan's C and B: the root-mean-square norm of every head with the
 * rotation by position in the same pass ("VikramLex/mamba3-minimal" README, "Architecture": B, C:
 * QK-norm, then RoPE).  Of every token (row) and head, over the head's `width` values:
 *     rstd = 1 / sqrt(mean u^2 + eps),   v = u rstd w,
 *     pair i (components 2i, 2i + 1) of the output = R(position freqs[i]) (pair i of v), i < pairs,
 * the other components v, computed in fp32 (the angle's turns in fp64) and rounded once to
 * x_dtype.  With its outputs as C and B, which have the same number of groups (q_heads = k_heads =
 * ngroups), m3ssd_fwd and m3ssd_step run without theta.  Unlike heads are for attention beside the scan.
 */
typedef struct {
  int64_t rows;       /* tokens, >= 0 */
  int64_t q_heads;    /* >= 1 */
  int64_t k_heads;    /* >= 0 (0: queries alone) */
  int64_t width;      /* 2 .. 256, even */
  int64_t pairs;      /* rotated pairs, 0 .. width / 2 */
  int64_t ldq;        /* elements from a token's queries to the next one's, >= q_heads width: */
  int64_t ldk;        /*   q and k may be column ranges of a projection's rows; keys alike */
  int32_t x_dtype;    /* m3ssd_dtype of q, k and the outputs */
  float eps;          /* >= 0 */
  uint32_t reserved;  /* must be 0 */
} m3ssd_rotate_dims;

/*
 * Forward.  q (rows, q_heads, width), k (rows, k_heads, width); q_w, k_w (width) fp32, NULL = 1;
 * positions (rows) int32, any sign; freqs (pairs) fp32, radians a position (both may be NULL where
 * pairs is 0).  q_out, k_out: dense; they may be q and k where those are dense.  width up to 256,
 * heads up to 65535, strides up to 2^31 - 1, the heads of all rows up to 2^31 - 2^16 (else
 * M3SSD_ERR_UNSUPPORTED).  No allocation, no synchronisation.
 */
m3ssd_status m3ssd_norm_rotate(const m3ssd_rotate_dims* dims, const void* q, const void* k,
                               const float* q_w, const float* k_w, const int32_t* positions,
                               const float* freqs, void* q_out, void* k_out, void* stream);

/* Gradients: dq, dk in `dtype` (fp32, or bf16 where x_dtype is), their rows ldq and ldk elements
 * apart; dq_w, dk_w (width) fp32, may be NULL. */
typedef struct {
  int64_t ldq;
  int64_t ldk;
  int32_t dtype;      /* m3ssd_dtype */
  uint32_t reserved;  /* must be 0 */
  void* dq;
  void* dk;
  float* dq_w;
  float* dk_w;
} m3ssd_rotate_grads;

/* Bytes of device workspace m3ssd_norm_rotate_bwd needs on the current device (it depends on the
 * SM count); 0 for invalid dims. */
size_t m3ssd_norm_rotate_bwd_workspace_size(const m3ssd_rotate_dims* dims);

/*
 * Its backward, from the forward's inputs and the gradients dq_out, dk_out of its outputs (dense, in
 * up_dtype: fp32 as m3ssd_bwd writes dC and dB, or bf16 where x_dtype is).  With dv = R(-position
 * freqs[i]) d, g = w dv, uh = u rstd and means over the head:
 *     du = rstd (g - uh mean(g uh)),   dw = sum over tokens and heads of dv uh.
 * Sums run in a fixed order: the same call gives the same bits.  dq and dk overlap no input, but may
 * be dq_out and dk_out where types and strides agree.  workspace: 256-byte aligned, not read
 * afterwards.
 */
m3ssd_status m3ssd_norm_rotate_bwd(const m3ssd_rotate_dims* dims, const void* q, const void* k,
                                   const float* q_w, const float* k_w, const int32_t* positions,
                                   const float* freqs, int32_t up_dtype, const void* dq_out,
                                   const void* dk_out, const m3ssd_rotate_grads* grads,
                                   void* workspace, size_t workspace_bytes, void* stream);

/*
 * Weights in 4 bits with a scale a group of columns, for the projections of a few decoding tokens
 * with activations as they are (beside m3ssd_gemm_mx, whose operands are both in few bits):
 *     W[n][k] = (code[n][k] - zero[k / group][n]) scale[k / group][n],   codes 0 .. 15.
 *   codes:  K padded to a multiple of 128 and N to one of 16, in tiles of 16 rows x 128 columns,
 *           1024 bytes each, row-block-major: byte 512 (r / 8) + 64 (r % 8) + 16 l + 4 j + m of row r
 *           of the tile holds columns 32 j + 8 l + 2 m (low half) and the next one (high half), l, j
 *           and m from 0 to 3.  16-byte aligned, m3ssd_w4_codes_size bytes.
 *   scales: (ceil(cols / group), rows) bf16.
 *   zeros:  (ceil(cols / group), rows) bytes 0 .. 15, or NULL: 8 everywhere.
 */
typedef struct {
  int64_t rows;       /* N >= 0 */
  int64_t cols;       /* K >= 1 */
  int64_t group;      /* columns of a group: 32, 64, or a multiple of 128 */
  uint64_t reserved;  /* must be 0 */
  void* codes;
  void* scales;
  void* zeros;
} m3ssd_w4;

/* Bytes of the codes; 0 for invalid arguments. */
size_t m3ssd_w4_codes_size(int64_t rows, int64_t cols);

/*
 * w (rows x cols, dtype, row stride ldw >= cols) to that form and back.  Without zeros a group's scale
 * is bf16(max |w| / 7) and a code round(w / scale) + 8; with zeros the scale is bf16((hi - lo) / 15) of the
 * group's range, zero included, the zero point round(-lo / scale) and a code round(w / scale) + it,
 * all clamped to 0 .. 15, ties to even.  A group of zeros takes scale 0; one with a NaN or an
 * infinity a NaN scale, and reads back as NaN.  Read back, (code - zero) scale is rounded once to dtype.
 */
m3ssd_status m3ssd_w4_quant(const m3ssd_w4* out, int32_t dtype, const void* w, int64_t ldw, void* stream);
m3ssd_status m3ssd_w4_dequant(const m3ssd_w4* in, int32_t dtype, void* w, int64_t ldw, void* stream);

/*
 * out (tokens x rows, out_dtype, row stride ldd >= rows) = x (tokens x cols, x_dtype, row stride
 * ldx >= cols) W^T for up to 16 tokens (else M3SSD_ERR_UNSUPPORTED: m3ssd_w4_dequant and
 * m3ssd_gemm_bf16 take more).  Products of the held values, exact (of an fp32 token below 2^-110 what is
 * a multiple of 2^-133 counts, the rest is dropped), fp32 sums over a group, each scaled in fp32, and
 * rounded once to out_dtype.  The order of the sums goes by the sizes and the
 * device's SM count: the same call gives the same bits.  No workspace, no allocation, no
 * synchronisation; capture-safe.
 */
m3ssd_status m3ssd_gemv_w4(int64_t tokens, int32_t x_dtype, const void* x, int64_t ldx, const m3ssd_w4* W,
                           int32_t out_dtype, void* out, int64_t ldd, void* stream);

/* Number of bounded device-side waits of the chunked forwards (SISO and
 * MIMO), the tensor-core backward, the GEMMs and the 8-bit step that ran out since
 * the last call (a forward's CTA then stops and leaves its outputs unwritten, a step's those
 * of the (b, h) it had not come to, so that with a cache_out of its own the step can be taken
 * again while a cache written in place is undefined; the backward's and the GEMMs' CTAs skip
 * their remaining waits and leave their outputs undefined); the count is then reset.  This
 * call synchronises the current device and must not be captured in a CUDA graph.  Returns
 * M3SSD_ERR_INVALID_ARG for a NULL pointer and M3SSD_ERR_CUDA if the device cannot be read. */
m3ssd_status m3ssd_device_wait_timeouts(uint32_t* count);

/*
 * Testing hooks for the failure path of the bounded device-side waits (no page
 * counterpart).  They copy to device variables synchronously, so they must not
 * be called while work of this library is in flight or being captured.
 *   m3ssd_test_set_wait_limit: the time limit of the chunked forward's bounded
 *     waits, in nanoseconds (0 restores the default of 2 s).
 *   m3ssd_test_drop_next_gram_signal: the next chunked forward that rotates
 *     (theta or angle0 given) and is not split into segments leaves out the
 *     completion signal of its first Gram product, so its compute warps'
 *     wait for it runs out: that launch counts one timeout in
 *     m3ssd_device_wait_timeouts and leaves its outputs undefined; the GPU
 *     context stays usable and later launches are unaffected.
 */
m3ssd_status m3ssd_test_set_wait_limit(uint64_t nanoseconds);
m3ssd_status m3ssd_test_drop_next_gram_signal(void);
/*   m3ssd_test_give_up_next_waits: in the next launch of m3ssd_gemm_bf16, m3ssd_gemm_mx or
 *     m3ssd_step_q8 (N = 128, P = 64, 16-byte aligned, more than two (b, h) an SM), the lanes
 *     of this mask in every warp that waits for copies or a result give up at once, as waits
 *     that run out do; the rest wait.  That launch is counted in m3ssd_device_wait_timeouts,
 *     its outputs as there; later launches are unaffected.  (Host state only; 0 takes it
 *     back.) */
m3ssd_status m3ssd_test_give_up_next_waits(uint32_t lanes);

/* The result of the M3SSD_CHECK_FINITE checks enqueued since the last call:
 * M3SSD_ERR_NONFINITE if any checked output held a NaN or an infinity, else
 * M3SSD_OK; the record is then cleared.  It synchronises the current device
 * and must not be captured in a CUDA graph; M3SSD_ERR_CUDA if the device
 * cannot be read. */
m3ssd_status m3ssd_nonfinite_outputs(void);

/* Static, human-readable name of a status. */
const char* m3ssd_status_string(m3ssd_status status);

/* M3SSD_ABI_VERSION of the loaded library. */
int m3ssd_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* M3SSD_H_ */
