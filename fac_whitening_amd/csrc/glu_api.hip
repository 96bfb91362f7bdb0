// C entries of the gated feed-forward block, of dropout and of the weight
// gradient from a whole activation: argument checks, then the launches on the
// caller's stream.  They keep no state.
#include <cmath>

#include "product.hpp"

namespace {

using gift::kMaxGrid;
constexpr int kMaxCols = 1 << 24;

bool dtype_ok(int32_t t) { return t == GIFT_BF16 || t == GIFT_FP32 || t == GIFT_FP16; }
int64_t dtype_size(int32_t t) { return t == GIFT_FP32 ? 4 : 2; }
bool aligned_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
bool cols_ok(int32_t n) { return n >= 1 && n <= kMaxCols; }
bool rows_count_ok(int64_t T) { return T >= 0 && T < ((int64_t)1 << 40); }

// A matrix in the caller's memory: rows x cols elements of `size` bytes.
struct Matrix {
  const void* p;
  int64_t ld, rows;
  int64_t cols, size;
  bool ok() const { return rows == 0 || (p && aligned_to(p, (size_t)size) && ld >= cols); }
  // what the products need to read it as it is
  bool near() const { return rows <= 1 || ld * size <= gift::kProductRow; }
  bool rows16() const { return near() && aligned_to(p, 16) && (rows <= 1 || ld * size % 16 == 0); }
  __int128 begin() const { return (__int128)reinterpret_cast<uintptr_t>(p); }
  __int128 end() const { return begin() + ((__int128)(rows - 1) * ld + cols) * size; }
};

// Whether no byte belongs to both.  Rows of both repeat every gcd of the
// strides, so rows side by side in one buffer are told apart by their places
// within it.
bool disjoint(const Matrix& a, const Matrix& b) {
  if (a.rows == 0 || b.rows == 0 || !a.p || !b.p) return true;
  if (a.end() <= b.begin() || b.end() <= a.begin()) return true;
  if (a.rows == 1 && b.rows == 1) return false;
  const __int128 ga = a.rows > 1 ? (__int128)a.ld * a.size : 0, gb = b.rows > 1 ? (__int128)b.ld * b.size : 0;
  __int128 g = ga, h = gb;
  while (h) {
    const __int128 r = g % h;
    g = h;
    h = r;
  }
  const __int128 r = ((b.begin() - a.begin()) % g + g) % g;
  return r >= (__int128)a.cols * a.size && g - r >= (__int128)b.cols * b.size;
}
// b is written while elements of a are read one by one: in place, or disjoint.
bool in_place_or_disjoint(const Matrix& a, const Matrix& b) {
  if (a.p == b.p && a.size == b.size && (a.ld == b.ld || a.rows <= 1)) return true;
  return disjoint(a, b);
}

bool drop_ok(const gift_dropout* d) {
  return !d || (d->p >= 0.0 && d->p <= 1.0 && aligned_to(d->d_offset, 8));
}
gift::DropArgs drop_args(const gift_dropout* d) {
  gift::DropArgs a{};
  if (!d) return a;
  a.thr = (uint32_t)std::nearbyint(65536.0 * d->p);
  a.on = a.thr != 0;
  a.scale = a.thr >= 65536 ? 0.f : (float)(65536.0 / (65536 - (int)a.thr));
  a.k0 = (uint32_t)d->seed;
  a.k1 = (uint32_t)(d->seed >> 32);
  a.offset = d->offset;
  a.d_offset = d->d_offset;
  return a;
}
constexpr int64_t kDropRows = (int64_t)1 << 32;

// What a product's launches reach: columns whose rows the kernel's 32-bit offsets span, tiles of the output and their
// stages (12 segments at most) in the counts of wgrad_levels.  (Operands that are laid out anew: see product_reach.)
constexpr int kProductCols = (int)(gift::kProductRow / 2);
bool reach(int64_t M, int64_t N, int64_t K) {
  return gift::product_tiles(M, N) <= kMaxGrid && gift::cdiv(K, 64) * 12 < ((int64_t)1 << 30) &&
         (__int128)gift::product_tiles(M, N) * gift::cdiv(K, 64) * 12 < ((__int128)1 << 38);
}
bool glu_reach(int64_t T, int32_t d, int32_t f) {
  return d <= kProductCols && f <= kProductCols && reach(f, T, d) && reach(d, T, f);
}
bool grad_reach(int64_t T, int32_t m, int32_t d) {
  return d <= kProductCols && m <= kProductCols && reach(d, m, T);
}

bool act_ok(int32_t a) { return a >= GIFT_ACT_SILU && a <= GIFT_ACT_SIGMOID; }
gift_status result(hipError_t e) { return e == hipSuccess ? GIFT_OK : gift::hip_failure(e); }

}  // namespace

extern "C" {

gift_status gift_dropout_apply(const gift_dropout* h_drop, const void* d_x, int32_t dtype, int64_t ldx, int64_t T,
                               int32_t d, const void* d_residual, int64_t ldr, void* d_y, int64_t ldy,
                               gift_stream_t stream) {
  if (!h_drop || !drop_ok(h_drop) || !dtype_ok(dtype) || !rows_count_ok(T) || !cols_ok(d)) return GIFT_ERR_INVALID_ARG;
  const int64_t size = dtype_size(dtype);
  const Matrix x{d_x, ldx, T, d, size}, r{d_residual, ldr, T, d, size}, y{d_y, ldy, T, d, size};
  if (!x.ok() || !y.ok() || (d_residual && !r.ok())) return GIFT_ERR_INVALID_ARG;
  if (!in_place_or_disjoint(x, y) || !in_place_or_disjoint(r, y)) return GIFT_ERR_INVALID_ARG;
  if (T > kDropRows || gift::dropout_grid(T, d) > kMaxGrid) return GIFT_ERR_UNSUPPORTED;
  return result(gift::launch_dropout(drop_args(h_drop), d_x, dtype, ldx, T, d, d_residual, ldr, d_y, ldy,
                                     static_cast<hipStream_t>(stream)));
}

size_t gift_glu_workspace_bytes(int64_t T, int32_t d, int32_t f, int32_t dtype, int32_t aligned) {
  if (!rows_count_ok(T) || !cols_ok(d) || !cols_ok(f) || !dtype_ok(dtype)) return 0;
  if (!glu_reach(T, d, f)) return 0;
  gift::GluCall c{};
  c.dtype = dtype;
  c.T = T;
  c.d = d;
  c.f = f;
  c.aligned = aligned != 0;
  return gift::glu_forward_workspace(c);
}

gift_status gift_glu_forward(int32_t act, const void* d_x, int32_t dtype, int64_t ldx, int64_t T, int32_t d,
                             const void* d_wg, int64_t ldg, const void* d_wu, int64_t ldu, int32_t f,
                             const gift_dropout* h_drop, void* d_h, int64_t ldh, void* d_gate, int64_t ldz, void* d_up,
                             int64_t ldup, const gift_act_ckpt* h_ckpt, void* d_work, size_t work_bytes,
                             gift_stream_t stream) {
  if (!act_ok(act) || !dtype_ok(dtype) || !rows_count_ok(T) || !cols_ok(d) || !cols_ok(f) || !drop_ok(h_drop))
    return GIFT_ERR_INVALID_ARG;
  const int64_t size = dtype_size(dtype);
  const Matrix x{d_x, ldx, T, d, size}, wg{d_wg, ldg, f, d, size}, wu{d_wu, ldu, f, d, size};
  const Matrix h{d_h, ldh, T, f, size}, z{d_gate, ldz, T, f, size}, u{d_up, ldup, T, f, size};
  if (!x.ok() || !wg.ok() || !wu.ok() || !h.ok()) return GIFT_ERR_INVALID_ARG;
  if (!d_gate != !d_up || (d_gate && (!z.ok() || !u.ok()))) return GIFT_ERR_INVALID_ARG;
  if (h_ckpt) {
    if (h_ckpt->fmt != GIFT_E4M3 && h_ckpt->fmt != GIFT_E5M2) return GIFT_ERR_INVALID_ARG;
    if (T > 0 && (!h_ckpt->d_codes || !aligned_to(h_ckpt->d_codes, 16) || !h_ckpt->d_bscales ||
                  !aligned_to(h_ckpt->d_bscales, 16) || h_ckpt->ldc % 32 != 0 || h_ckpt->ldc < f))
      return GIFT_ERR_INVALID_ARG;
  }
  const int64_t nb = gift::cdiv(f, 32);
  const Matrix codes{h_ckpt ? h_ckpt->d_codes : nullptr, h_ckpt ? h_ckpt->ldc : 0, T, 32 * nb, 1};
  const Matrix scales{h_ckpt ? h_ckpt->d_bscales : nullptr, 8 * nb, gift::cdiv(T, 8), 8 * nb, 1};
  const Matrix out[5] = {h, z, u, codes, scales};
  for (int k = 0; k < 5; ++k) {
    for (const Matrix& i : {x, wg, wu})
      if (!disjoint(out[k], i)) return GIFT_ERR_INVALID_ARG;
    for (int l = 0; l < k; ++l)
      if (!disjoint(out[k], out[l])) return GIFT_ERR_INVALID_ARG;
  }
  if (h_drop && T > kDropRows) return GIFT_ERR_UNSUPPORTED;
  if (!glu_reach(T, d, f) || (h_ckpt && gift::act_grid(T, f) > kMaxGrid)) return GIFT_ERR_UNSUPPORTED;
  gift::GluCall c{};
  c.act = act;
  c.dtype = dtype;
  c.x = d_x;
  c.ldx = ldx;
  c.T = T;
  c.d = d;
  c.f = f;
  c.wg = d_wg;
  c.wu = d_wu;
  c.ldg = ldg;
  c.ldu = ldu;
  c.h = d_h;
  c.gate = d_gate;
  c.up = d_up;
  c.ldh = ldh;
  c.ldz = ldz;
  c.ldup = ldup;
  c.aligned = x.rows16() && wg.rows16() && wu.rows16();
  c.work = d_work;
  if (!gift::glu_forward_reach(c)) return GIFT_ERR_UNSUPPORTED;
  const size_t need = gift::glu_forward_workspace(c);
  if (need && (!d_work || !aligned_to(d_work, 16))) return GIFT_ERR_INVALID_ARG;
  if (work_bytes < need) return GIFT_ERR_WORKSPACE;
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = gift::launch_glu_forward(c, drop_args(h_drop), s);
  if (e == hipSuccess && h_ckpt) e = gift::launch_act_save(d_h, dtype, ldh, T, f, *h_ckpt, s);
  return result(e);
}

size_t gift_glu_backward_workspace_bytes(int64_t T, int32_t d, int32_t f, int32_t dtype, int32_t aligned) {
  if (!rows_count_ok(T) || !cols_ok(d) || !cols_ok(f) || !dtype_ok(dtype)) return 0;
  if (!glu_reach(T, d, f)) return 0;
  gift::GluGradCall c{};
  c.dtype = dtype;
  c.T = T;
  c.d = d;
  c.f = f;
  c.aligned = c.near = aligned != 0;
  const size_t apart = gift::glu_backward_workspace(c);
  c.in_place = true;
  const size_t over = gift::glu_backward_workspace(c);
  return apart > over ? apart : over;
}

gift_status gift_glu_backward(int32_t act, const void* d_dh, int32_t dtype, int64_t lddh, int64_t T, int32_t f,
                              const void* d_gate, int64_t ldz, const void* d_up, int64_t ldup,
                              const gift_dropout* h_drop, void* d_dgate, int64_t lddz, void* d_dup, int64_t lddup,
                              const void* d_wg, int64_t ldg, const void* d_wu, int64_t ldu, int32_t d, void* d_dx,
                              int64_t lddx, void* d_work, size_t work_bytes, gift_stream_t stream) {
  if (!act_ok(act) || !dtype_ok(dtype) || !rows_count_ok(T) || !cols_ok(f) || !drop_ok(h_drop))
    return GIFT_ERR_INVALID_ARG;
  const int64_t size = dtype_size(dtype);
  const Matrix dh{d_dh, lddh, T, f, size}, z{d_gate, ldz, T, f, size}, u{d_up, ldup, T, f, size};
  const Matrix dz{d_dgate, lddz, T, f, size}, du{d_dup, lddup, T, f, size};
  if (!dh.ok() || !z.ok() || !u.ok() || !dz.ok() || !du.ok()) return GIFT_ERR_INVALID_ARG;
  for (const Matrix& i : {dh, z, u})
    if (!in_place_or_disjoint(i, dz) || !in_place_or_disjoint(i, du)) return GIFT_ERR_INVALID_ARG;
  if (!disjoint(dz, du)) return GIFT_ERR_INVALID_ARG;
  gift::GluGradCall c{};
  for (const void* i : {d_dh, d_gate, d_up}) c.in_place = c.in_place || i == d_dgate || i == d_dup;
  if (d_dx) {
    if (!cols_ok(d)) return GIFT_ERR_INVALID_ARG;
    const Matrix wg{d_wg, ldg, f, d, size}, wu{d_wu, ldu, f, d, size}, dx{d_dx, lddx, T, d, size};
    if (!wg.ok() || !wu.ok() || !dx.ok()) return GIFT_ERR_INVALID_ARG;
    for (const Matrix& i : {wg, wu})
      if (!disjoint(i, dx) || !disjoint(i, dz) || !disjoint(i, du)) return GIFT_ERR_INVALID_ARG;
    if (!disjoint(dz, dx) || !disjoint(du, dx)) return GIFT_ERR_INVALID_ARG;
    for (const Matrix& i : {dh, z, u}) c.in_place = c.in_place || !disjoint(i, dx);
    if (!glu_reach(T, d, f)) return GIFT_ERR_UNSUPPORTED;
    c.aligned = dz.rows16() && du.rows16() && (T == 1 || lddz == lddup);
    c.near = wg.near() && wu.near() && (f == 1 || ldg == ldu);
  }
  if ((h_drop && T > kDropRows) || gift::glu_gradients_grid(T, f) > kMaxGrid) return GIFT_ERR_UNSUPPORTED;
  c.act = act;
  c.dtype = dtype;
  c.dh = d_dh;
  c.gate = d_gate;
  c.up = d_up;
  c.lddh = lddh;
  c.ldz = ldz;
  c.ldup = ldup;
  c.T = T;
  c.d = d;
  c.f = f;
  c.dgate = d_dgate;
  c.dup = d_dup;
  c.lddz = lddz;
  c.lddup = lddup;
  c.wg = d_wg;
  c.wu = d_wu;
  c.ldg = ldg;
  c.ldu = ldu;
  c.dx = d_dx;
  c.lddx = lddx;
  c.work = d_work;
  if (d_dx) {
    if (!gift::glu_backward_reach(c)) return GIFT_ERR_UNSUPPORTED;
    const size_t need = gift::glu_backward_workspace(c);
    if (need && (!d_work || !aligned_to(d_work, 16))) return GIFT_ERR_INVALID_ARG;
    if (work_bytes < need) return GIFT_ERR_WORKSPACE;
  }
  return result(gift::launch_glu_backward(c, drop_args(h_drop), static_cast<hipStream_t>(stream)));
}

size_t gift_weight_grad_x_workspace_bytes(int64_t T, int32_t m, int32_t d, int32_t dtype, int32_t aligned) {
  if (!rows_count_ok(T) || !cols_ok(d) || !cols_ok(m) || !dtype_ok(dtype)) return 0;
  if (!grad_reach(T, m, d)) return 0;
  gift::WgradXCall c{};
  c.dtype = dtype;
  c.T = T;
  c.m = m;
  c.d = d;
  c.near = aligned != 0;
  return gift::wgrad_x_workspace(c);
}

gift_status gift_weight_grad_x(const void* d_delta, int32_t dtype, int64_t ldd, int32_t m, const void* d_x,
                               int64_t ldx, int64_t T, int32_t d, float alpha, int32_t accumulate, float* d_W,
                               int64_t ldw, void* d_work, size_t work_bytes, gift_stream_t stream) {
  if (!dtype_ok(dtype) || !rows_count_ok(T) || !cols_ok(d) || !cols_ok(m)) return GIFT_ERR_INVALID_ARG;
  const int64_t size = dtype_size(dtype);
  const Matrix delta{d_delta, ldd, T, m, size}, x{d_x, ldx, T, d, size}, W{d_W, ldw, m, d, 4};
  if (!delta.ok() || !x.ok() || !W.ok() || !disjoint(delta, W) || !disjoint(x, W)) return GIFT_ERR_INVALID_ARG;
  if (!grad_reach(T, m, d)) return GIFT_ERR_UNSUPPORTED;
  gift::WgradXCall c{};
  c.delta = d_delta;
  c.dtype = dtype;
  c.ldd = ldd;
  c.m = m;
  c.x = d_x;
  c.ldx = ldx;
  c.T = T;
  c.d = d;
  c.alpha = alpha;
  c.accumulate = accumulate ? 1 : 0;
  c.W = d_W;
  c.ldw = ldw;
  c.near = delta.near() && x.near();
  c.work = d_work;
  if (!gift::wgrad_x_reach(c)) return GIFT_ERR_UNSUPPORTED;
  const size_t need = gift::wgrad_x_workspace(c);
  if (need && (!d_work || !aligned_to(d_work, 16))) return GIFT_ERR_INVALID_ARG;
  if (work_bytes < need) return GIFT_ERR_WORKSPACE;
  return result(gift::launch_wgrad_x(c, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
