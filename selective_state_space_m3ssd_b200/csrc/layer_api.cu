// C-ABI entry points of the operators that a layer has around the scan: the gated linear
// recurrence, the norm of heads with their rotation, and 4-bit weights with scales a group.
// Host-side validation and dispatch; nothing is allocated, nothing synchronises.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "../../include/m3ssd.h"
#include "internal.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

m3ssd_status from_cuda(cudaError_t e) {
  if (e == cudaSuccess) return M3SSD_OK;
  (void)cudaGetLastError();
  return M3SSD_ERR_CUDA;
}

bool dtype_ok(int32_t t) { return t == M3SSD_F32 || t == M3SSD_BF16; }
uintptr_t dtype_size(int32_t t) { return t == M3SSD_BF16 ? 2 : 4; }

bool all_aligned4(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!aligned(p, 4)) return false;
  return true;
}

m3ssd_status check_glr(const m3ssd_glr_dims* d, int64_t seqlen) {
  if (!d || d->reserved != 0) return M3SSD_ERR_INVALID_ARG;
  if (d->batch < 0 || seqlen < 0 || d->width < 1) return M3SSD_ERR_INVALID_ARG;
  if (!dtype_ok(d->x_dtype)) return M3SSD_ERR_INVALID_ARG;
  if (d->ldx < d->width || d->ldr < d->width || d->ldi < d->width) return M3SSD_ERR_INVALID_ARG;
  if (!(d->c > 0.f) || !std::isfinite(d->c)) return M3SSD_ERR_INVALID_ARG;
  // tokens, a few rounds past the end too, sequences x channel pairs and the elements of a tile
  // are counted in 31 bits
  const int64_t most = INT32_MAX;
  if (d->width > most / 64 || seqlen > most / 2 || d->batch > most || d->ldx > most || d->ldr > most ||
      d->ldi > most || d->batch * ((d->width + 1) / 2) > most)
    return M3SSD_ERR_UNSUPPORTED;
  return M3SSD_OK;
}

// The inputs that the forward and the backward share.
bool glr_inputs_ok(const m3ssd_glr_dims* d, const void* x, const void* r, const void* i,
                   const float* rate, const float* bias_r, const float* bias_i, const float* h0,
                   const int32_t* lengths) {
  const uintptr_t esz = dtype_size(d->x_dtype);
  if (!rate || (d->batch > 0 && d->seqlen > 0 && (!x || !r || !i))) return false;
  return aligned(x, esz) && aligned(r, esz) && aligned(i, esz) &&
         all_aligned4({rate, bias_r, bias_i, h0, lengths});
}

m3ssd::GlrArgs glr_args(const m3ssd_glr_dims* d, const void* x, const void* r, const void* i,
                        const float* rate, const float* bias_r, const float* bias_i,
                        const float* h0, const uint8_t* reset, const int32_t* lengths) {
  m3ssd::GlrArgs a{};
  a.b = d->batch; a.L = d->seqlen; a.D = d->width;
  a.ldx = d->ldx; a.ldr = d->ldr; a.ldi = d->ldi;
  a.bf16 = d->x_dtype == M3SSD_BF16; a.c = d->c;
  a.x = x; a.r = r; a.i = i; a.rate = rate; a.bias_r = bias_r; a.bias_i = bias_i;
  a.h0 = h0; a.reset = reset; a.lengths = lengths;
  return a;
}

m3ssd_status check_rotate(const m3ssd_rotate_dims* d) {
  if (!d || d->reserved != 0) return M3SSD_ERR_INVALID_ARG;
  if (d->rows < 0 || d->q_heads < 1 || d->k_heads < 0 || d->width < 2 || d->width % 2 != 0 ||
      d->pairs < 0 || d->pairs > d->width / 2)
    return M3SSD_ERR_INVALID_ARG;
  if (!dtype_ok(d->x_dtype) || !(d->eps >= 0.f)) return M3SSD_ERR_INVALID_ARG;
  // blocks of a token's heads are counted in 31 bits, up to a round of all warps past the last
  const int64_t most = INT32_MAX, units = most - 65535;
  if (d->width > 256 || d->q_heads > 65535 || d->k_heads > 65535 || d->rows > most || d->ldq > most ||
      d->ldk > most || d->rows * (d->q_heads + d->k_heads) > units)
    return M3SSD_ERR_UNSUPPORTED;
  if (d->ldq < d->q_heads * d->width || d->ldk < d->k_heads * d->width) return M3SSD_ERR_INVALID_ARG;
  return M3SSD_OK;
}

// The inputs that the forward and the backward share, into `a`; false where one is wrong.
bool rotate_inputs(const m3ssd_rotate_dims* d, const void* q, const void* k, const float* q_w,
                   const float* k_w, const int32_t* positions, const float* freqs,
                   m3ssd::RotateArgs& a) {
  const uintptr_t esz = dtype_size(d->x_dtype);
  if (d->rows > 0 && (!q || (d->k_heads > 0 && !k) || (d->pairs > 0 && !positions))) return false;
  if (d->pairs > 0 && !freqs) return false;
  if (!aligned(q, esz) || !aligned(k, esz) || !all_aligned4({q_w, k_w, positions, freqs})) return false;
  a.rows = d->rows; a.Hq = d->q_heads; a.Hk = d->k_heads; a.N = d->width; a.R = d->pairs;
  a.ldq = d->ldq; a.ldk = d->ldk;
  a.bf16 = d->x_dtype == M3SSD_BF16; a.eps = d->eps;
  a.q = q; a.k = k; a.q_w = q_w; a.k_w = k_w; a.positions = positions; a.freqs = freqs;
  return true;
}

m3ssd_status check_w4_size(int64_t rows, int64_t cols, int64_t group) {
  if (rows < 0 || cols < 1 || group < 32) return M3SSD_ERR_INVALID_ARG;
  if (group != 32 && group != 64 && group % 128 != 0) return M3SSD_ERR_INVALID_ARG;
  const int64_t most = INT32_MAX;  // rows, columns, and tiles of 16 x 128 are counted in 31 bits
  if (rows > most - 15 || cols > most / 8 || group > most) return M3SSD_ERR_UNSUPPORTED;
  if ((rows + 15) / 16 * ((cols + 127) / 128) > most / 8) return M3SSD_ERR_UNSUPPORTED;
  return M3SSD_OK;
}
m3ssd_status check_w4(const m3ssd_w4* w) {
  if (!w || w->reserved != 0) return M3SSD_ERR_INVALID_ARG;
  const m3ssd_status st = check_w4_size(w->rows, w->cols, w->group);
  if (st != M3SSD_OK) return st;
  if (w->rows > 0 && (!w->codes || !w->scales)) return M3SSD_ERR_INVALID_ARG;
  return aligned(w->codes, 16) && aligned(w->scales, 2) ? M3SSD_OK : M3SSD_ERR_INVALID_ARG;
}
m3ssd::W4Args w4_args(const m3ssd_w4* w) {
  m3ssd::W4Args a{};
  a.N = w->rows; a.K = w->cols; a.group = w->group;
  a.groups = (int)((w->cols + w->group - 1) / w->group);
  a.codes = static_cast<uint8_t*>(w->codes);
  a.scales = static_cast<uint16_t*>(w->scales);
  a.zeros = static_cast<uint8_t*>(w->zeros);
  return a;
}

}  // namespace

extern "C" {

size_t m3ssd_glr_fwd_workspace_size(const m3ssd_glr_dims* dims) {
  if (check_glr(dims, dims ? dims->seqlen : 0) != M3SSD_OK) return 0;
  return m3ssd::glr_fwd_workspace_bytes(dims->batch, dims->seqlen, dims->width,
                                        dims->x_dtype == M3SSD_BF16);
}

m3ssd_status m3ssd_glr_fwd(const m3ssd_glr_dims* dims, const void* x, const void* r, const void* i,
                           const float* rate, const float* bias_r, const float* bias_i,
                           const float* h0, const uint8_t* reset, const int32_t* lengths, void* y,
                           float* hT, void* workspace, size_t workspace_bytes, void* stream) {
  const m3ssd_status st = check_glr(dims, dims ? dims->seqlen : 0);
  if (st != M3SSD_OK) return st;
  if (!glr_inputs_ok(dims, x, r, i, rate, bias_r, bias_i, h0, lengths)) return M3SSD_ERR_INVALID_ARG;
  if ((dims->batch > 0 && dims->seqlen > 0 && !y) || !aligned(y, dtype_size(dims->x_dtype)) ||
      !aligned(hT, 4))
    return M3SSD_ERR_INVALID_ARG;
  const size_t need = m3ssd_glr_fwd_workspace_size(dims);
  if (workspace_bytes < need || (need > 0 && (!workspace || !aligned(workspace, 256))))
    return M3SSD_ERR_WORKSPACE;
  if (dims->batch == 0) return M3SSD_OK;
  m3ssd::GlrArgs a = glr_args(dims, x, r, i, rate, bias_r, bias_i, h0, reset, lengths);
  a.y = y;
  a.hT = hT;
  return from_cuda(m3ssd::launch_glr_fwd(a, workspace, static_cast<cudaStream_t>(stream)));
}

size_t m3ssd_glr_bwd_workspace_size(const m3ssd_glr_dims* dims) {
  if (check_glr(dims, dims ? dims->seqlen : 0) != M3SSD_OK) return 0;
  return m3ssd::glr_bwd_workspace_bytes(dims->batch, dims->seqlen, dims->width,
                                        dims->x_dtype == M3SSD_BF16);
}

m3ssd_status m3ssd_glr_bwd(const m3ssd_glr_dims* dims, const void* x, const void* r, const void* i,
                           const float* rate, const float* bias_r, const float* bias_i,
                           const float* h0, const uint8_t* reset, const int32_t* lengths,
                           const void* y, const void* dy, const float* dhT,
                           const m3ssd_glr_grads* grads, void* workspace, size_t workspace_bytes,
                           void* stream) {
  const m3ssd_status st = check_glr(dims, dims ? dims->seqlen : 0);
  if (st != M3SSD_OK) return st;
  if (!grads || grads->reserved != 0 || !dtype_ok(grads->dtype)) return M3SSD_ERR_INVALID_ARG;
  if (grads->dtype == M3SSD_BF16 && dims->x_dtype != M3SSD_BF16) return M3SSD_ERR_UNSUPPORTED;
  if (grads->ld < dims->width) return M3SSD_ERR_INVALID_ARG;
  if (grads->ld > INT32_MAX / 64) return M3SSD_ERR_UNSUPPORTED;  // as the width
  if (!glr_inputs_ok(dims, x, r, i, rate, bias_r, bias_i, h0, lengths)) return M3SSD_ERR_INVALID_ARG;
  const uintptr_t esz = dtype_size(dims->x_dtype), gsz = dtype_size(grads->dtype);
  if (dims->batch > 0 && dims->seqlen > 0 &&
      (!y || !dy || !grads->dx || !grads->dr || !grads->di))
    return M3SSD_ERR_INVALID_ARG;
  if (!grads->drate || !aligned(y, esz) || !aligned(dy, esz) || !aligned(grads->dx, gsz) ||
      !aligned(grads->dr, gsz) || !aligned(grads->di, gsz) ||
      !all_aligned4({dhT, grads->drate, grads->dbias_r, grads->dbias_i, grads->dh0}))
    return M3SSD_ERR_INVALID_ARG;
  const size_t need = m3ssd_glr_bwd_workspace_size(dims);
  if (workspace_bytes < need || (need > 0 && (!workspace || !aligned(workspace, 256))))
    return M3SSD_ERR_WORKSPACE;
  m3ssd::GlrBwdArgs a{};
  a.f = glr_args(dims, x, r, i, rate, bias_r, bias_i, h0, reset, lengths);
  a.f.y = const_cast<void*>(y);
  a.dy = dy; a.dhT = dhT;
  a.grad_bf16 = grads->dtype == M3SSD_BF16;
  a.ldg = grads->ld;
  a.dx = grads->dx; a.dr = grads->dr; a.di = grads->di;
  a.drate = grads->drate; a.dbias_r = grads->dbias_r; a.dbias_i = grads->dbias_i;
  a.dh0 = grads->dh0;
  return from_cuda(m3ssd::launch_glr_bwd(a, workspace, static_cast<cudaStream_t>(stream)));
}

m3ssd_status m3ssd_glr_step(const m3ssd_glr_dims* dims, const void* x_t, const void* r_t,
                            const void* i_t, const float* rate, const float* bias_r,
                            const float* bias_i, const float* h, float* h_out, void* y_t,
                            void* stream) {
  const m3ssd_status st = check_glr(dims, 0);
  if (st != M3SSD_OK) return st;
  const uintptr_t esz = dtype_size(dims->x_dtype);
  float* const out = h_out ? h_out : const_cast<float*>(h);
  if (!rate || (dims->batch > 0 && (!x_t || !r_t || !i_t || !h || !y_t)))
    return M3SSD_ERR_INVALID_ARG;
  if (!aligned(x_t, esz) || !aligned(r_t, esz) || !aligned(i_t, esz) || !aligned(y_t, esz) ||
      !all_aligned4({rate, bias_r, bias_i, h, out}))
    return M3SSD_ERR_INVALID_ARG;
  m3ssd::GlrStepArgs a{};
  a.b = dims->batch; a.D = dims->width;
  a.ldx = dims->ldx; a.ldr = dims->ldr; a.ldi = dims->ldi;
  a.bf16 = dims->x_dtype == M3SSD_BF16; a.c = dims->c;
  a.x = x_t; a.r = r_t; a.i = i_t; a.rate = rate; a.bias_r = bias_r; a.bias_i = bias_i;
  a.h = h; a.h_out = out; a.y = y_t;
  return from_cuda(m3ssd::launch_glr_step(a, static_cast<cudaStream_t>(stream)));
}

m3ssd_status m3ssd_norm_rotate(const m3ssd_rotate_dims* dims, const void* q, const void* k,
                               const float* q_w, const float* k_w, const int32_t* positions,
                               const float* freqs, void* q_out, void* k_out, void* stream) {
  const m3ssd_status st = check_rotate(dims);
  if (st != M3SSD_OK) return st;
  m3ssd::RotateArgs a{};
  if (!rotate_inputs(dims, q, k, q_w, k_w, positions, freqs, a)) return M3SSD_ERR_INVALID_ARG;
  const uintptr_t esz = dtype_size(dims->x_dtype);
  if (!aligned(q_out, esz) || !aligned(k_out, esz)) return M3SSD_ERR_INVALID_ARG;
  if (dims->rows == 0) return M3SSD_OK;
  if (!q_out || (dims->k_heads > 0 && !k_out)) return M3SSD_ERR_INVALID_ARG;
  a.q_out = q_out;
  a.k_out = k_out;
  return from_cuda(m3ssd::launch_norm_rotate(a, static_cast<cudaStream_t>(stream)));
}

size_t m3ssd_norm_rotate_bwd_workspace_size(const m3ssd_rotate_dims* dims) {
  if (check_rotate(dims) != M3SSD_OK) return 0;
  m3ssd::RotateArgs a{};
  a.rows = dims->rows; a.Hq = dims->q_heads; a.Hk = dims->k_heads; a.N = dims->width;
  return m3ssd::norm_rotate_bwd_workspace_bytes(a);
}

m3ssd_status m3ssd_norm_rotate_bwd(const m3ssd_rotate_dims* dims, const void* q, const void* k,
                                   const float* q_w, const float* k_w, const int32_t* positions,
                                   const float* freqs, int32_t up_dtype, const void* dq_out,
                                   const void* dk_out, const m3ssd_rotate_grads* grads,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  const m3ssd_status st = check_rotate(dims);
  if (st != M3SSD_OK) return st;
  if (!grads || grads->reserved != 0 || !dtype_ok(grads->dtype) || !dtype_ok(up_dtype))
    return M3SSD_ERR_INVALID_ARG;
  if (dims->x_dtype == M3SSD_F32 && (grads->dtype != M3SSD_F32 || up_dtype != M3SSD_F32))
    return M3SSD_ERR_UNSUPPORTED;
  if (grads->ldq < dims->q_heads * dims->width || grads->ldk < dims->k_heads * dims->width)
    return M3SSD_ERR_INVALID_ARG;
  m3ssd::RotateBwdArgs a{};
  if (!rotate_inputs(dims, q, k, q_w, k_w, positions, freqs, a.f)) return M3SSD_ERR_INVALID_ARG;
  const uintptr_t usz = dtype_size(up_dtype), gsz = dtype_size(grads->dtype);
  if (!aligned(dq_out, usz) || !aligned(dk_out, usz) || !aligned(grads->dq, gsz) ||
      !aligned(grads->dk, gsz) || !all_aligned4({grads->dq_w, grads->dk_w}))
    return M3SSD_ERR_INVALID_ARG;
  if (dims->rows > 0 && (!dq_out || !grads->dq || (dims->k_heads > 0 && (!dk_out || !grads->dk))))
    return M3SSD_ERR_INVALID_ARG;
  const size_t need = m3ssd_norm_rotate_bwd_workspace_size(dims);
  if (workspace_bytes < need || (need > 0 && (!workspace || !aligned(workspace, 256))))
    return M3SSD_ERR_WORKSPACE;
  a.up_bf16 = up_dtype == M3SSD_BF16;
  a.grad_bf16 = grads->dtype == M3SSD_BF16;
  a.dq_out = dq_out; a.dk_out = dk_out;
  a.ldgq = grads->ldq; a.ldgk = grads->ldk;
  a.dq = grads->dq; a.dk = grads->dk; a.dq_w = grads->dq_w; a.dk_w = grads->dk_w;
  a.part = static_cast<float*>(workspace);
  return from_cuda(m3ssd::launch_norm_rotate_bwd(a, static_cast<cudaStream_t>(stream)));
}

size_t m3ssd_w4_codes_size(int64_t rows, int64_t cols) {
  if (check_w4_size(rows, cols, 32) != M3SSD_OK) return 0;
  return (size_t)((rows + 15) / 16) * (size_t)((cols + 127) / 128) * 1024;
}

m3ssd_status m3ssd_w4_quant(const m3ssd_w4* out, int32_t dtype, const void* w, int64_t ldw, void* stream) {
  const m3ssd_status st = check_w4(out);
  if (st != M3SSD_OK) return st;
  if (!dtype_ok(dtype) || ldw < out->cols) return M3SSD_ERR_INVALID_ARG;
  if (out->rows == 0) return M3SSD_OK;
  if (!w || !aligned(w, dtype_size(dtype))) return M3SSD_ERR_INVALID_ARG;
  return from_cuda(m3ssd::launch_w4_quant(w4_args(out), dtype == M3SSD_BF16, w, ldw,
                                          static_cast<cudaStream_t>(stream)));
}

m3ssd_status m3ssd_w4_dequant(const m3ssd_w4* in, int32_t dtype, void* w, int64_t ldw, void* stream) {
  const m3ssd_status st = check_w4(in);
  if (st != M3SSD_OK) return st;
  if (!dtype_ok(dtype) || ldw < in->cols) return M3SSD_ERR_INVALID_ARG;
  if (in->rows == 0) return M3SSD_OK;
  if (!w || !aligned(w, dtype_size(dtype))) return M3SSD_ERR_INVALID_ARG;
  return from_cuda(m3ssd::launch_w4_dequant(w4_args(in), dtype == M3SSD_BF16, w, ldw,
                                            static_cast<cudaStream_t>(stream)));
}

m3ssd_status m3ssd_gemv_w4(int64_t tokens, int32_t x_dtype, const void* x, int64_t ldx, const m3ssd_w4* W,
                           int32_t out_dtype, void* out, int64_t ldd, void* stream) {
  const m3ssd_status st = check_w4(W);
  if (st != M3SSD_OK) return st;
  if (tokens < 0 || !dtype_ok(x_dtype) || !dtype_ok(out_dtype)) return M3SSD_ERR_INVALID_ARG;
  if (tokens > 16) return M3SSD_ERR_UNSUPPORTED;
  if (ldx < W->cols || ldd < W->rows) return M3SSD_ERR_INVALID_ARG;
  if (tokens == 0 || W->rows == 0) return M3SSD_OK;
  if (!x || !out || !aligned(x, dtype_size(x_dtype)) || !aligned(out, dtype_size(out_dtype)))
    return M3SSD_ERR_INVALID_ARG;
  const m3ssd::W4Args w = w4_args(W);
  m3ssd::GemvW4Args a{};
  a.M = tokens; a.N = w.N; a.K = w.K; a.group = w.group; a.groups = w.groups;
  a.x_bf16 = x_dtype == M3SSD_BF16; a.out_bf16 = out_dtype == M3SSD_BF16;
  a.x = x; a.ldx = ldx; a.codes = w.codes; a.scales = w.scales; a.zeros = w.zeros;
  a.out = out; a.ldd = ldd;
  return from_cuda(m3ssd::launch_gemv_w4(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
