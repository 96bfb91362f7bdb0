// Gated feed-forward block, its backward pass, and the weight gradient from
// an activation kept whole: the products that surround the layer whose
// gradient is encoded.
//   forward   z = x Wg^T, u = x Wu^T, h = D(act(z) u)
//   backward  dgate = D(dh) u act'(z), dup = D(dh) act(z), dx = dgate Wg + dup Wu
//   weights   W = alpha delta^T x
// dgate and dup are made here; the products are k_product's, few tokens those
// of k_glu_tokens.hip and k_glu_tokens_backward.hip.
// dgate and dup are rounded to the type before dx is made of them: they are the
// operands of the weight gradients too, and 16-bit ones enter the matrix cores
// as they are.  For bf16 that puts dx off by 0.0024 of its norm, where sums of
// unrounded gradients, rounded once, are off by 0.0017; keeping them in fp32
// would take three planes of each, three times the products.
#include "product.hpp"

namespace gift {

// Eight of a row's rounded values (v: before the rounding, exact for fp32) as
// k_product_pack lays them out, zeros past the row's end.
template <typename T>
__device__ __forceinline__ void lay_out(const Raw8<T>& r, float* v, uint16_t* dst, int64_t t, int j, int nb, int64_t rows, int n) {
  uint16_t* p = dst + (t * nb * 8 + j);
  if constexpr (sizeof(T) == 2) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = 2 * i + 1 < n ? r.w[i] : 2 * i < n ? r.w[i] & 0xFFFFu : 0u;
    store_words<4>(p, w, false);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? v[i] : 0.f;
    split_planes(v, [&](int pl, const uint32_t* w) { store_words<4>(p + pl * rows * nb * 8, w, false); });
  }
}

// dgate and dup: eight columns of a row a thread; pz and pu: also laid out for
// the product that follows.  Bound by memory: 16384 x 6144 bf16 1.0 GB in 170
// us, 5.9 TB/s.
template <typename T, int ACT>
__global__ void __launch_bounds__(256) k_glu_gradients(GluGradCall c, DropArgs drop, int nb, int64_t n,
                                                       uint16_t* pz, uint16_t* pu) {
  const int64_t first = (int64_t)blockIdx.x * 256;
  const int64_t t0 = first / nb;
  if (first + threadIdx.x >= n) return;
  const uint32_t at = (uint32_t)(first - t0 * nb) + threadIdx.x;
  const uint32_t down = at / (uint32_t)nb, b = at - down * (uint32_t)nb;
  const int64_t t = t0 + down;
  const int j = (int)b * 8, m = c.f - j;
  float e[8], z[8], u[8];
  unpack8(load8(static_cast<const T*>(c.dh) + t * c.lddh + j, m), e);
  unpack8(load8(static_cast<const T*>(c.gate) + t * c.ldz + j, m), z);
  unpack8(load8(static_cast<const T*>(c.up) + t * c.ldup + j, m), u);
  if (drop.on) {
    uint32_t w[4];
    drop_bits(drop, drop_offset(drop), (uint32_t)t, b, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = drop_one(drop, w, i, e[i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float g;
    const float a = act_value<ACT>(z[i], &g);
    z[i] = e[i] * u[i] * g;
    u[i] = e[i] * a;
  }
  Raw8<T> o;
  pack8(z, o);
  store8(static_cast<T*>(c.dgate) + t * c.lddz + j, o, m, false);
  if (pz) lay_out(o, z, pz, t, j, nb, c.T, m);
  pack8(u, o);
  store8(static_cast<T*>(c.dup) + t * c.lddup + j, o, m, false);
  if (pz) lay_out(o, u, pu, t, j, nb, c.T, m);
}

// W = 0: the gradient of no tokens.
__global__ void __launch_bounds__(256) k_wgrad_none(float* W, int64_t ldw, int m, int d) {
  for (int i = blockIdx.x; i < m; i += gridDim.x)
    for (int j = threadIdx.x; j < d; j += 256) W[i * ldw + j] = 0.f;
}

int64_t glu_gradients_grid(int64_t T, int f) { return cdiv(T * cdiv(f, 8), 256); }

namespace {

template <typename F>
void with_act(int act, F&& go) {
  switch (act) {
    case GIFT_ACT_SILU: return go(std::integral_constant<int, GIFT_ACT_SILU>{});
    case GIFT_ACT_GELU: return go(std::integral_constant<int, GIFT_ACT_GELU>{});
    case GIFT_ACT_GELU_TANH: return go(std::integral_constant<int, GIFT_ACT_GELU_TANH>{});
    case GIFT_ACT_RELU: return go(std::integral_constant<int, GIFT_ACT_RELU>{});
    default: return go(std::integral_constant<int, GIFT_ACT_SIGMOID>{});
  }
}
template <typename F>
void with_type(int dtype, F&& go) {
  if (dtype == GIFT_BF16) go(Bf16{});
  else if (dtype == GIFT_FP16) go(Fp16{});
  else go(float{});
}

ProductCall glu_product(const GluCall& c) {
  ProductCall p{};
  p.epi = kEpiGlu;
  p.act = c.act;
  p.dtype = c.dtype;
  p.parts = 1;
  p.a[0] = {c.wg, c.ldg, c.f, c.d, c.aligned, false, false};
  p.a[1] = {c.wu, c.ldu, c.f, c.d, c.aligned, false, false};
  p.b[0] = {c.x, c.ldx, c.T, c.d, c.aligned, false, false};
  p.M = c.f;
  p.N = c.T;
  p.K = c.d;
  p.out = c.h;
  p.ldo = c.ldh;
  p.gate = c.gate;
  p.up = c.up;
  p.ldz = c.ldz;
  p.ldup = c.ldup;
  p.work = c.work;
  return p;
}

bool gradients_packed(const GluGradCall& c) { return c.dtype == GIFT_FP32 || c.f % 8 != 0 || !c.aligned; }

ProductCall dx_product(const GluGradCall& c) {
  ProductCall p{};
  p.work = c.work;
  p.epi = kEpiStore;
  p.dtype = c.dtype;
  p.parts = 2;
  p.a[0] = {c.wg, c.ldg, c.f, c.d, false, c.near, false};
  p.a[1] = {c.wu, c.ldu, c.f, c.d, false, c.near, false};
  p.b[0] = {c.dgate, c.lddz, c.T, c.f, c.aligned, false, false};
  p.b[1] = {c.dup, c.lddup, c.T, c.f, c.aligned, false, false};
  if (gradients_packed(c)) {
    // k_glu_gradients lays them out in front of the workspace
    char* w = static_cast<char*>(c.work);
    const size_t bytes = product_packed(c.dtype, c.T, c.f);
    p.b[0] = {w, 0, c.T, c.f, false, false, true};
    p.b[1] = {w + bytes, 0, c.T, c.f, false, false, true};
    p.work = w + 2 * bytes;
  }
  p.M = c.d;
  p.N = c.T;
  p.K = c.f;
  p.out = c.dx;
  p.ldo = c.lddx;
  return p;
}

ProductCall grad_product(const WgradXCall& c) {
  ProductCall p{};
  p.epi = kEpiGrad;
  p.dtype = c.dtype;
  p.parts = 1;
  p.a[0] = {c.x, c.ldx, c.T, c.d, false, c.near, false};
  p.b[0] = {c.delta, c.ldd, c.T, c.m, false, c.near, false};
  p.M = c.d;
  p.N = c.m;
  p.K = c.T;
  p.out = c.W;
  p.ldo = c.ldw;
  p.alpha = c.alpha;
  p.accumulate = c.accumulate;
  p.work = c.work;
  return p;
}

}  // namespace

size_t glu_forward_workspace(const GluCall& c) { return glu_by_tokens(c.dtype, c.T, c.d, c.f) ? 0 : product_workspace(glu_product(c)); }
size_t glu_backward_workspace(const GluGradCall& c) {
  if (c.T == 0) return 0;
  if (glu_backward_by_tokens(c.dtype, c.T, c.in_place)) return glu_tokens_backward_workspace(c.T, c.d, c.f);
  return product_workspace(dx_product(c)) + (gradients_packed(c) ? 2 * product_packed(c.dtype, c.T, c.f) : 0);
}
size_t wgrad_x_workspace(const WgradXCall& c) { return c.T ? product_workspace(grad_product(c)) : 0; }
bool glu_forward_reach(const GluCall& c) { return glu_by_tokens(c.dtype, c.T, c.d, c.f) || product_reach(glu_product(c)); }
bool glu_backward_reach(const GluGradCall& c) { return glu_backward_by_tokens(c.dtype, c.T, c.in_place) || product_reach(dx_product(c)); }
bool wgrad_x_reach(const WgradXCall& c) { return c.T == 0 || product_reach(grad_product(c)); }

hipError_t launch_glu_forward(const GluCall& c, const DropArgs& drop, hipStream_t s) {
  if (c.T == 0) return hipSuccess;
  return glu_by_tokens(c.dtype, c.T, c.d, c.f) ? launch_glu_tokens(c, drop, s) : launch_product(glu_product(c), drop, s);
}

hipError_t launch_glu_backward(const GluGradCall& c, const DropArgs& drop, hipStream_t s) {
  if (c.T == 0) return hipSuccess;
  if (c.dx && glu_backward_by_tokens(c.dtype, c.T, c.in_place)) return launch_glu_tokens_backward(c, drop, s);
  uint16_t* planes[2] = {nullptr, nullptr};
  if (c.dx && gradients_packed(c)) {
    planes[0] = static_cast<uint16_t*>(c.work);
    planes[1] = planes[0] + product_packed(c.dtype, c.T, c.f) / 2;
  }
  with_type(c.dtype, [&](auto t) {
    with_act(c.act, [&](auto a) {
      hipLaunchKernelGGL((k_glu_gradients<decltype(t), decltype(a)::value>), dim3((unsigned)glu_gradients_grid(c.T, c.f)),
                         dim3(256), 0, s, c, drop, (int)cdiv(c.f, 8), c.T * cdiv(c.f, 8), planes[0], planes[1]);
    });
  });
  if (c.dx) return launch_product(dx_product(c), DropArgs{}, s);
  return hipGetLastError();
}

hipError_t launch_wgrad_x(const WgradXCall& c, hipStream_t s) {
  if (c.T == 0) {
    if (c.accumulate) return hipSuccess;
    hipLaunchKernelGGL(k_wgrad_none, dim3((unsigned)(c.m < 4096 ? c.m : 4096)), dim3(256), 0, s, c.W, c.ldw, c.m, c.d);
    return hipGetLastError();
  }
  return launch_product(grad_product(c), DropArgs{}, s);
}

}  // namespace gift
