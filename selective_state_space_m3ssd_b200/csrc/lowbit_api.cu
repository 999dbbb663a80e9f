// C-ABI entry points of the low-bit and normalisation operators: host-side validation and
// dispatch.  As in m3ssd_api.cu, nothing is allocated and nothing synchronises.
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "../../include/m3ssd.h"
#include "internal.h"
#include "mx.cuh"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

m3ssd_status from_cuda(cudaError_t e) {
  if (e == cudaSuccess) return M3SSD_OK;
  (void)cudaGetLastError();
  return M3SSD_ERR_CUDA;
}

bool dtype_ok(int32_t t) { return t == M3SSD_F32 || t == M3SSD_BF16; }
uintptr_t dtype_size(int32_t t) { return t == M3SSD_BF16 ? 2 : 4; }

// Sizes of a microscaled tensor: rows and 128-column groups each, and their product over
// whole tiles of 128 rows, in 31 bits (the kernels count groups in 32).
m3ssd_status check_mx_size(int32_t format, int64_t rows, int64_t cols) {
  if (format != M3SSD_MXFP4 && format != M3SSD_MXFP8) return M3SSD_ERR_INVALID_ARG;
  if (rows < 0 || cols < 1) return M3SSD_ERR_INVALID_ARG;
  if (rows > INT32_MAX - 127 || cols > INT32_MAX - 127) return M3SSD_ERR_UNSUPPORTED;
  if (m3ssd::mx::pad128(rows) * (m3ssd::mx::pad128(cols) / 128) > INT32_MAX)
    return M3SSD_ERR_UNSUPPORTED;
  return M3SSD_OK;
}

m3ssd_status check_mx(const m3ssd_mx* t) {
  if (!t || t->reserved != 0) return M3SSD_ERR_INVALID_ARG;
  const m3ssd_status st = check_mx_size(t->format, t->rows, t->cols);
  if (st != M3SSD_OK) return st;
  if (t->rows > 0 && (!t->codes || !t->scales)) return M3SSD_ERR_INVALID_ARG;
  if (!aligned(t->codes, 128) || !aligned(t->scales, 128)) return M3SSD_ERR_INVALID_ARG;
  return M3SSD_OK;
}

m3ssd_status check_norm(const m3ssd_norm_dims* d) {
  if (!d || d->reserved != 0) return M3SSD_ERR_INVALID_ARG;
  if (d->rows < 0 || d->width < 1 || !dtype_ok(d->x_dtype) || !dtype_ok(d->res_dtype))
    return M3SSD_ERR_INVALID_ARG;
  if (!(d->eps >= 0.f)) return M3SSD_ERR_INVALID_ARG;
  if (d->rows > INT32_MAX || !m3ssd::norm_width_ok(d->width)) return M3SSD_ERR_UNSUPPORTED;
  return M3SSD_OK;
}

// The dims of the decode step and of a held state.
m3ssd_status check_state_dims(const m3ssd_dims* d) {
  if (!d) return M3SSD_ERR_INVALID_ARG;
  if (d->batch < 0 || d->nheads < 1 || d->headdim < 1 || d->ngroups < 1)
    return M3SSD_ERR_INVALID_ARG;
  if (d->dstate < 2 || d->dstate % 2 != 0 || d->nheads % d->ngroups != 0)
    return M3SSD_ERR_INVALID_ARG;
  if (!dtype_ok(d->x_dtype) || d->reserved != 0) return M3SSD_ERR_INVALID_ARG;
  if ((d->flags & ~(uint32_t)M3SSD_CHECK_FINITE) != 0) return M3SSD_ERR_UNSUPPORTED;
  if (d->nheads > INT32_MAX || d->batch > INT32_MAX || d->batch * d->nheads > INT32_MAX)
    return M3SSD_ERR_UNSUPPORTED;
  if (d->dstate > 256 || d->headdim > 256 || d->dstate * d->headdim > 16384)
    return M3SSD_ERR_UNSUPPORTED;
  return M3SSD_OK;
}

bool cache_ok(const m3ssd_cache_q8* c) {
  return c->angle && c->ssm && c->ssm_scale && c->x_prev && c->b_prev;
}
bool cache_aligned(const m3ssd_cache_q8* c) {
  return aligned(c->angle, 4) && aligned(c->ssm_scale, 4) && aligned(c->x_prev, 4) &&
         aligned(c->b_prev, 4);
}

std::atomic<uint32_t> g_given_up_lanes{0};

}  // namespace

uint32_t m3ssd::take_given_up_lanes() {
  return g_given_up_lanes.load(std::memory_order_relaxed) ? g_given_up_lanes.exchange(0) : 0;
}

extern "C" {

m3ssd_status m3ssd_test_give_up_next_waits(uint32_t lanes) {
  g_given_up_lanes.store(lanes);
  return M3SSD_OK;
}

size_t m3ssd_mx_codes_size(int32_t format, int64_t rows, int64_t cols) {
  if (check_mx_size(format, rows, cols) != M3SSD_OK) return 0;
  const size_t n = (size_t)rows * (size_t)m3ssd::mx::pad128(cols);
  return format == M3SSD_MXFP4 ? n / 2 : n;
}

size_t m3ssd_mx_scales_size(int64_t rows, int64_t cols) {
  if (check_mx_size(M3SSD_MXFP4, rows, cols) != M3SSD_OK) return 0;
  return (size_t)m3ssd::mx::pad128(rows) * (size_t)(m3ssd::mx::pad128(cols) / 32);
}

m3ssd_status m3ssd_mx_quant(const m3ssd_mx* out, int32_t x_dtype, const void* x, int64_t ldx,
                            void* stream) {
  const m3ssd_status st = check_mx(out);
  if (st != M3SSD_OK) return st;
  if (!dtype_ok(x_dtype) || ldx < out->cols) return M3SSD_ERR_INVALID_ARG;
  if (out->rows == 0) return M3SSD_OK;
  if (!x || !aligned(x, dtype_size(x_dtype))) return M3SSD_ERR_INVALID_ARG;
  return from_cuda(m3ssd::launch_mx_quant(out->format, out->rows, out->cols,
                                          x_dtype == M3SSD_BF16, x, ldx, out->codes, out->scales,
                                          static_cast<cudaStream_t>(stream)));
}

m3ssd_status m3ssd_mx_dequant(const m3ssd_mx* in, int32_t x_dtype, void* x, int64_t ldx,
                              void* stream) {
  const m3ssd_status st = check_mx(in);
  if (st != M3SSD_OK) return st;
  if (!dtype_ok(x_dtype) || ldx < in->cols) return M3SSD_ERR_INVALID_ARG;
  if (in->rows == 0) return M3SSD_OK;
  if (!x || !aligned(x, dtype_size(x_dtype))) return M3SSD_ERR_INVALID_ARG;
  return from_cuda(m3ssd::launch_mx_dequant(in->format, in->rows, in->cols,
                                            x_dtype == M3SSD_BF16, in->codes, in->scales, x, ldx,
                                            static_cast<cudaStream_t>(stream)));
}

m3ssd_status m3ssd_gemm_mx(const m3ssd_mx* A, const m3ssd_mx* W, void* D, int64_t ldd,
                           void* stream) {
  m3ssd_status st = check_mx(A);
  if (st == M3SSD_OK) st = check_mx(W);
  if (st != M3SSD_OK) return st;
  if (A->cols != W->cols || ldd < W->rows) return M3SSD_ERR_INVALID_ARG;
  if (W->format != M3SSD_MXFP4) return M3SSD_ERR_UNSUPPORTED;
  if (A->rows == 0 || W->rows == 0) return M3SSD_OK;
  if (!D || !aligned(D, 2)) return M3SSD_ERR_INVALID_ARG;
  return from_cuda(m3ssd::launch_gemm_mx(A->format, A->rows, W->rows, A->cols, A->codes, A->scales,
                                         W->codes, W->scales, D, ldd,
                                         static_cast<cudaStream_t>(stream)));
}

m3ssd_status m3ssd_test_gemm_mx_plan(int32_t a_format, int64_t M, int64_t N, int64_t K,
                                     int32_t sms, int32_t* split, int32_t* tile, int32_t* part) {
  m3ssd_status st = check_mx_size(a_format, M, K);
  if (st == M3SSD_OK) st = check_mx_size(M3SSD_MXFP4, N, K);
  if (st != M3SSD_OK) return st;
  if (M < 1 || N < 1 || sms < 1 || !split || !tile || !part) return M3SSD_ERR_INVALID_ARG;
  const m3ssd::GemmMxPlan p = m3ssd::gemm_mx_plan(a_format, M, N, K, sms);
  *split = p.split;
  *tile = p.tile;
  *part = p.part;
  return M3SSD_OK;
}

m3ssd_status m3ssd_add_rmsnorm(const m3ssd_norm_dims* dims, const void* x, const void* residual,
                               const float* w, void* y, const m3ssd_mx* y_mx, void* residual_out,
                               float* rstd, void* stream) {
  m3ssd_status st = check_norm(dims);
  if (st != M3SSD_OK) return st;
  if ((y != nullptr) == (y_mx != nullptr) && (dims->rows > 0 || y)) return M3SSD_ERR_INVALID_ARG;
  if ((residual != nullptr) != (residual_out != nullptr)) return M3SSD_ERR_INVALID_ARG;
  if (y && y == residual_out) return M3SSD_ERR_INVALID_ARG;
  m3ssd::NormArgs a{};
  a.fmt = -1;
  if (y_mx) {
    st = check_mx(y_mx);
    if (st != M3SSD_OK) return st;
    if (y_mx->rows != dims->rows || y_mx->cols != dims->width) return M3SSD_ERR_INVALID_ARG;
    a.fmt = y_mx->format;
    a.Kp = m3ssd::mx::pad128(dims->width);
    a.codes = static_cast<uint8_t*>(y_mx->codes);
    a.scales = static_cast<uint8_t*>(y_mx->scales);
  }
  if (dims->rows == 0) return M3SSD_OK;
  const uintptr_t esz = dtype_size(dims->x_dtype), rsz = dtype_size(dims->res_dtype);
  if (!x || !w || !aligned(x, esz) || !aligned(y, esz) || !aligned(residual, rsz) ||
      !aligned(residual_out, rsz) || !aligned(w, 4) || !aligned(rstd, 4))
    return M3SSD_ERR_INVALID_ARG;
  a.rows = dims->rows; a.d = dims->width; a.eps = dims->eps;
  a.bf16 = dims->x_dtype == M3SSD_BF16;
  a.res_bf16 = dims->res_dtype == M3SSD_BF16;
  a.x = x; a.res = residual; a.w = w; a.y = y; a.res_out = residual_out; a.rstd = rstd;
  return from_cuda(m3ssd::launch_add_rmsnorm(a, static_cast<cudaStream_t>(stream)));
}

size_t m3ssd_add_rmsnorm_bwd_workspace_size(const m3ssd_norm_dims* dims) {
  if (check_norm(dims) != M3SSD_OK) return 0;
  return m3ssd::norm_bwd_workspace_bytes(dims->rows, dims->width);
}

m3ssd_status m3ssd_add_rmsnorm_bwd(const m3ssd_norm_dims* dims, const void* dy, const void* r,
                                   const float* w, const float* rstd, const float* dres, float* dr,
                                   float* dw, void* workspace, size_t workspace_bytes,
                                   void* stream) {
  const m3ssd_status st = check_norm(dims);
  if (st != M3SSD_OK) return st;
  if (!dw || (dims->rows > 0 && (!dy || !r || !w || !rstd || !dr))) return M3SSD_ERR_INVALID_ARG;
  if (!aligned(dy, dtype_size(dims->x_dtype)) || !aligned(r, dtype_size(dims->res_dtype)))
    return M3SSD_ERR_INVALID_ARG;
  const void* f32[] = {w, rstd, dres, dr, dw};
  for (const void* p : f32)
    if (!aligned(p, 4)) return M3SSD_ERR_INVALID_ARG;
  const size_t need = m3ssd::norm_bwd_workspace_bytes(dims->rows, dims->width);
  if (workspace_bytes < need || (need > 0 && (!workspace || !aligned(workspace, 256))))
    return M3SSD_ERR_WORKSPACE;
  m3ssd::NormBwdArgs a{};
  a.rows = dims->rows; a.d = dims->width;
  a.bf16 = dims->x_dtype == M3SSD_BF16;
  a.res_bf16 = dims->res_dtype == M3SSD_BF16;
  a.dy = dy; a.r = r; a.w = w; a.rstd = rstd; a.dres = dres; a.dr = dr; a.dw = dw;
  a.part = static_cast<float*>(workspace);
  return from_cuda(m3ssd::launch_add_rmsnorm_bwd(a, static_cast<cudaStream_t>(stream)));
}

m3ssd_status m3ssd_test_norm_access(const m3ssd_norm_dims* dims, int64_t row, int32_t column,
                                    int32_t* whole) {
  const m3ssd_status st = check_norm(dims);
  if (st != M3SSD_OK) return st;
  if (!whole || row < 0 || row >= dims->rows || column <= -8 || column >= dims->width)
    return M3SSD_ERR_INVALID_ARG;
  *whole = m3ssd::norm_whole_access(dims->rows, dims->width, row, column);
  return M3SSD_OK;
}

m3ssd_status m3ssd_quant_state(const m3ssd_dims* dims, const float* ssm, void* codes, float* scale,
                               void* stream) {
  const m3ssd_status st = check_state_dims(dims);
  if (st != M3SSD_OK) return st;
  if (dims->flags != 0) return M3SSD_ERR_UNSUPPORTED;
  if (dims->batch == 0) return M3SSD_OK;
  if (!ssm || !codes || !scale || !aligned(ssm, 4) || !aligned(scale, 4))
    return M3SSD_ERR_INVALID_ARG;
  return from_cuda(m3ssd::launch_quant_state(dims->batch * dims->nheads * dims->dstate,
                                             dims->headdim, ssm, codes, scale,
                                             static_cast<cudaStream_t>(stream)));
}

m3ssd_status m3ssd_dequant_state(const m3ssd_dims* dims, const void* codes, const float* scale,
                                 float* ssm, void* stream) {
  const m3ssd_status st = check_state_dims(dims);
  if (st != M3SSD_OK) return st;
  if (dims->flags != 0) return M3SSD_ERR_UNSUPPORTED;
  if (dims->batch == 0) return M3SSD_OK;
  if (!ssm || !codes || !scale || !aligned(ssm, 4) || !aligned(scale, 4))
    return M3SSD_ERR_INVALID_ARG;
  return from_cuda(m3ssd::launch_dequant_state(dims->batch * dims->nheads * dims->dstate,
                                               dims->headdim, codes, scale, ssm,
                                               static_cast<cudaStream_t>(stream)));
}

m3ssd_status m3ssd_step_q8(const m3ssd_dims* dims, const void* x_t, const float* logdecay_t,
                           const float* beta_t, const float* gamma_t, const void* B_t,
                           const void* C_t, const float* theta_t, const float* D,
                           const m3ssd_cache_q8* cache, const m3ssd_cache_q8* cache_out, void* y_t,
                           void* stream) {
  m3ssd_status st = check_state_dims(dims);
  if (st != M3SSD_OK) return st;
  if (!cache) return M3SSD_ERR_INVALID_ARG;
  const m3ssd_cache_q8* const out = cache_out ? cache_out : cache;
  const bool bf16 = dims->x_dtype == M3SSD_BF16;
  const uintptr_t esz = dtype_size(dims->x_dtype);
  if (dims->batch > 0) {
    if (!x_t || !logdecay_t || !gamma_t || !B_t || !C_t || !y_t) return M3SSD_ERR_INVALID_ARG;
    if (!cache_ok(cache) || !cache_ok(out)) return M3SSD_ERR_INVALID_ARG;
  }
  if (!aligned(x_t, esz) || !aligned(B_t, esz) || !aligned(C_t, esz) || !aligned(y_t, esz))
    return M3SSD_ERR_INVALID_ARG;
  const void* f32[] = {logdecay_t, beta_t, gamma_t, theta_t, D};
  for (const void* p : f32)
    if (!aligned(p, 4)) return M3SSD_ERR_INVALID_ARG;
  if (!cache_aligned(cache) || !cache_aligned(out)) return M3SSD_ERR_INVALID_ARG;
  if (dims->batch == 0) return M3SSD_OK;

  m3ssd::StepQ8Args a{};
  a.b = dims->batch; a.H = dims->nheads; a.P = dims->headdim; a.N = dims->dstate;
  a.G = dims->ngroups; a.bf16 = bf16;
  a.x_t = x_t; a.logdecay_t = logdecay_t; a.beta_t = beta_t; a.gamma_t = gamma_t;
  a.B_t = B_t; a.C_t = C_t; a.theta_t = theta_t; a.D = D;
  a.angle = cache->angle; a.ssm = static_cast<const uint8_t*>(cache->ssm);
  a.scale = cache->ssm_scale; a.x_prev = cache->x_prev; a.b_prev = cache->b_prev;
  a.angle_out = out->angle; a.ssm_out = static_cast<uint8_t*>(out->ssm);
  a.scale_out = out->ssm_scale; a.x_prev_out = out->x_prev; a.b_prev_out = out->b_prev;
  a.y_t = y_t;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  st = from_cuda(m3ssd::launch_step_q8(a, s));
  if (st == M3SSD_OK && (dims->flags & M3SSD_CHECK_FINITE))
    st = from_cuda(m3ssd::launch_nonfinite_check(
        y_t, dims->batch * dims->nheads * dims->headdim, bf16, s));
  return st;
}

}  // extern "C"
