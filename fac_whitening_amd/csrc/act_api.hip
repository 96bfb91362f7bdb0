// C entries of the activation operators: argument checks, then one or two
// kernel launches on the caller's stream.  They keep no state.
#include <cmath>
#include <numeric>

#include "gift_internal.hpp"

namespace {

using gift::kMaxGrid;
constexpr int kMaxCols = 1 << 24;

bool dtype_ok(int32_t t) { return t == GIFT_BF16 || t == GIFT_FP32 || t == GIFT_FP16; }
size_t dtype_size(int32_t t) { return t == GIFT_FP32 ? 4 : 2; }
bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// A matrix of T rows of n elements (a pointer is needed once there are rows).
bool rows_ok(const void* p, int32_t dtype, int64_t ld, int64_t T, int32_t n) {
  return T == 0 || (p && aligned(p, dtype_size(dtype)) && ld >= n);
}

bool sizes_ok(int64_t T, int32_t d) { return T >= 0 && T < ((int64_t)1 << 40) && d >= 1 && d <= kMaxCols; }

// Whether an output [T][n] at q may be written while rows of an input at p are
// still to be read: it is the input itself, element for element, or shares no
// byte with it.  Rows of both repeat every gcd of the strides, so rows side by
// side in one buffer are told apart by their places within it.
bool out_ok(const void* p, int64_t ldp, const void* q, int64_t ldq, int64_t T, int32_t n, int32_t dtype) {
  if (T == 0 || !p) return true;
  const __int128 size = dtype_size(dtype), a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  if (a == b && (ldp == ldq || T == 1)) return true;
  if (a + ((T - 1) * (__int128)ldp + n) * size <= b || b + ((T - 1) * (__int128)ldq + n) * size <= a) return true;
  if (T == 1) return false;
  const __int128 g = std::gcd(ldp, ldq) * size, w = n * size, r = ((b - a) % g + g) % g;
  return r >= w && g - r >= w;
}

bool ckpt_ok(const gift_act_ckpt* c, int64_t T, int32_t d) {
  if (!c || (c->fmt != GIFT_E4M3 && c->fmt != GIFT_E5M2)) return false;
  if (T == 0) return true;
  return c->d_codes && aligned(c->d_codes, 16) && c->d_bscales && aligned(c->d_bscales, 16) && c->ldc % 32 == 0 &&
         c->ldc >= d;
}

gift_status result(hipError_t e) { return e == hipSuccess ? GIFT_OK : gift::hip_failure(e); }

}  // namespace

extern "C" {

size_t gift_act_scale_bytes(int64_t T, int32_t d) {
  if (!sizes_ok(T, d)) return 0;
  return (size_t)(gift::cdiv(T, 8) * gift::cdiv(d, 32) * 8);
}

gift_status gift_act_save(const void* d_x, int32_t dtype, int64_t ldx, int64_t T, int32_t d,
                          const gift_act_ckpt* h_ckpt, gift_stream_t stream) {
  if (!dtype_ok(dtype) || !sizes_ok(T, d) || !rows_ok(d_x, dtype, ldx, T, d) || !ckpt_ok(h_ckpt, T, d))
    return GIFT_ERR_INVALID_ARG;
  if (gift::act_grid(T, d) > kMaxGrid) return GIFT_ERR_UNSUPPORTED;
  return result(gift::launch_act_save(d_x, dtype, ldx, T, d, *h_ckpt, static_cast<hipStream_t>(stream)));
}

gift_status gift_act_restore(const gift_act_ckpt* h_ckpt, int64_t T, int32_t d, void* d_out, int32_t dtype,
                             int64_t ldo, gift_stream_t stream) {
  if (!dtype_ok(dtype) || !sizes_ok(T, d) || !rows_ok(d_out, dtype, ldo, T, d) || !ckpt_ok(h_ckpt, T, d))
    return GIFT_ERR_INVALID_ARG;
  if (gift::act_grid(T, d) > kMaxGrid) return GIFT_ERR_UNSUPPORTED;
  return result(gift::launch_act_restore(*h_ckpt, T, d, d_out, dtype, ldo, static_cast<hipStream_t>(stream)));
}

gift_status gift_norm_forward(int32_t kind, const void* d_x, int32_t dtype, int64_t ldx, int64_t T, int32_t d,
                              const void* d_gamma, const void* d_beta, int32_t wdtype, float eps, void* d_y,
                              int64_t ldy, float* d_mean, float* d_rstd, const gift_act_ckpt* h_ckpt,
                              gift_stream_t stream) {
  if ((kind != GIFT_NORM_LAYER && kind != GIFT_NORM_RMS) || !dtype_ok(dtype) || !sizes_ok(T, d))
    return GIFT_ERR_INVALID_ARG;
  if ((wdtype != dtype && wdtype != GIFT_FP32) || !(eps >= 0.0f) || !std::isfinite(eps)) return GIFT_ERR_INVALID_ARG;
  if (!rows_ok(d_x, dtype, ldx, T, d) || !rows_ok(d_y, dtype, ldy, T, d)) return GIFT_ERR_INVALID_ARG;
  if (!out_ok(d_x, ldx, d_y, ldy, T, d, dtype)) return GIFT_ERR_INVALID_ARG;
  if (!aligned(d_gamma, dtype_size(wdtype)) || !aligned(d_beta, dtype_size(wdtype))) return GIFT_ERR_INVALID_ARG;
  if (!aligned(d_mean, 4) || !aligned(d_rstd, 4)) return GIFT_ERR_INVALID_ARG;
  if (h_ckpt && !ckpt_ok(h_ckpt, T, d)) return GIFT_ERR_INVALID_ARG;
  if (d > gift::kNormMaxCols || gift::norm_forward_grid(T, d) > kMaxGrid) return GIFT_ERR_UNSUPPORTED;
  gift::NormCall c{};
  c.kind = kind;
  c.dtype = dtype;
  c.wdtype = wdtype;
  c.x = d_x;
  c.ldx = ldx;
  c.ckpt = h_ckpt;
  c.T = T;
  c.d = d;
  c.w = d_gamma;
  c.b = d_beta;
  c.eps = eps;
  c.mean = d_mean;
  c.rstd = d_rstd;
  c.y = d_y;
  c.ldy = ldy;
  return result(gift::launch_norm_forward(c, static_cast<hipStream_t>(stream)));
}

size_t gift_norm_workspace_bytes(int64_t T, int32_t d) {
  if (!sizes_ok(T, d) || d > gift::kNormMaxCols) return 0;
  return gift::align256((size_t)gift::norm_partials(T, d) * 2 * (size_t)d * 4);
}

gift_status gift_norm_backward(int32_t kind, const void* d_dy, int32_t dtype, int64_t lddy, const void* d_x,
                               int64_t ldx, const gift_act_ckpt* h_ckpt, int64_t T, int32_t d, const void* d_gamma,
                               int32_t wdtype, const float* d_mean, const float* d_rstd, void* d_dx, int64_t lddx,
                               float* d_dgamma, float* d_dbeta, int32_t accumulate, void* d_work, size_t work_bytes,
                               gift_stream_t stream) {
  if ((kind != GIFT_NORM_LAYER && kind != GIFT_NORM_RMS) || !dtype_ok(dtype) || !sizes_ok(T, d))
    return GIFT_ERR_INVALID_ARG;
  if (wdtype != dtype && wdtype != GIFT_FP32) return GIFT_ERR_INVALID_ARG;
  if (!rows_ok(d_dy, dtype, lddy, T, d) || !rows_ok(d_dx, dtype, lddx, T, d)) return GIFT_ERR_INVALID_ARG;
  if (h_ckpt) {
    if (d_x || !ckpt_ok(h_ckpt, T, d)) return GIFT_ERR_INVALID_ARG;
  } else if (!rows_ok(d_x, dtype, ldx, T, d)) {
    return GIFT_ERR_INVALID_ARG;
  }
  if (!out_ok(d_dy, lddy, d_dx, lddx, T, d, dtype) || !out_ok(d_x, ldx, d_dx, lddx, T, d, dtype))
    return GIFT_ERR_INVALID_ARG;
  if (T > 0 && (!d_rstd || (kind == GIFT_NORM_LAYER && !d_mean))) return GIFT_ERR_INVALID_ARG;
  if (!aligned(d_mean, 4) || !aligned(d_rstd, 4) || !aligned(d_dgamma, 4) || !aligned(d_dbeta, 4) ||
      !aligned(d_gamma, dtype_size(wdtype)))
    return GIFT_ERR_INVALID_ARG;
  if (d > gift::kNormMaxCols) return GIFT_ERR_UNSUPPORTED;
  const bool wanted = d_dgamma || d_dbeta;
  if (wanted) {
    if (!d_work || !aligned(d_work, 16)) return GIFT_ERR_INVALID_ARG;
    if (work_bytes < gift_norm_workspace_bytes(T, d)) return GIFT_ERR_WORKSPACE;
  } else if (T == 0) {
    return GIFT_OK;
  }
  gift::NormCall c{};
  c.kind = kind;
  c.dtype = dtype;
  c.wdtype = wdtype;
  c.x = d_x;
  c.ldx = ldx;
  c.ckpt = h_ckpt;
  c.T = T;
  c.d = d;
  c.w = d_gamma;
  c.mean = const_cast<float*>(d_mean);
  c.rstd = const_cast<float*>(d_rstd);
  c.y = d_dx;
  c.ldy = lddx;
  c.dy = d_dy;
  c.lddy = lddy;
  return result(gift::launch_norm_backward(c, wanted ? static_cast<float*>(d_work) : nullptr, d_dgamma, d_dbeta,
                                           accumulate ? 1 : 0, static_cast<hipStream_t>(stream)));
}

size_t gift_weight_grad_workspace_bytes(int64_t T, int32_t m, int32_t d, int32_t dtype) {
  if (!sizes_ok(T, d) || m < 1 || m > kMaxCols || !dtype_ok(dtype)) return 0;
  return gift::wgrad_workspace(T, m, d, dtype);
}

gift_status gift_weight_grad(const void* d_delta, int32_t dtype, int64_t ldd, int32_t m, const gift_act_ckpt* h_ckpt,
                             int64_t T, int32_t d, float alpha, int32_t accumulate, float* d_W, int64_t ldw,
                             void* d_work, size_t work_bytes, gift_stream_t stream) {
  if (!dtype_ok(dtype) || !sizes_ok(T, d) || m < 1 || m > kMaxCols) return GIFT_ERR_INVALID_ARG;
  if (!rows_ok(d_delta, dtype, ldd, T, m) || !ckpt_ok(h_ckpt, T, d)) return GIFT_ERR_INVALID_ARG;
  if (!d_W || !aligned(d_W, 4) || ldw < d) return GIFT_ERR_INVALID_ARG;
  if (!d_work || !aligned(d_work, 16)) return GIFT_ERR_INVALID_ARG;
  if (gift::wgrad_grid(m, d) > kMaxGrid) return GIFT_ERR_UNSUPPORTED;
  if (work_bytes < gift_weight_grad_workspace_bytes(T, m, d, dtype)) return GIFT_ERR_WORKSPACE;
  gift::WgradCall c{};
  c.delta = d_delta;
  c.dtype = dtype;
  c.ldd = ldd;
  c.m = m;
  c.ckpt = h_ckpt;
  c.T = T;
  c.d = d;
  c.alpha = alpha;
  c.accumulate = accumulate ? 1 : 0;
  c.W = d_W;
  c.ldw = ldw;
  c.work = static_cast<float*>(d_work);
  return result(gift::launch_weight_grad(c, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
