// Gated feed-forward block, its backward pass, and the weight gradient from
// an activation kept whole: the products that surround the layer whose
// gradient is encoded.
//   forward   z = x Wg^T, u = x Wu^T, h = D(act(z) u)
//   backward  dgate = D(dh) u act'(z), dup = D(dh) act(z), dx = dgate Wg + dup Wu
//   weights   W = alpha delta^T x
//
// First form, on the vector units: 64 x 64 outputs a workgroup, 4 x 4 a
// thread, 32 of the long axis a stage, fp32 products and sums over 256,
// folded into fp64.
#include <type_traits>

#include "glu.hpp"

namespace gift {

__device__ __forceinline__ float value_of(const float* p) { return *p; }
__device__ __forceinline__ float value_of(const Bf16* p) { return __uint_as_float((uint32_t)p->v << 16); }
__device__ __forceinline__ float value_of(const Fp16* p) { return (float)__builtin_bit_cast(_Float16, p->v); }
__device__ __forceinline__ void store_of(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_of(Bf16* p, float v) { p->v = __builtin_bit_cast(uint16_t, (__bf16)v); }
__device__ __forceinline__ void store_of(Fp16* p, float v) { p->v = __builtin_bit_cast(uint16_t, (_Float16)v); }

// Element (i, k) at p + i si + k sk.
struct Operand {
  const void* p;
  int64_t si, sk;
};

// sum_k A(i0 + 4 ty + ., k) B(j0 + 4 tx + ., k) into sum (added).
template <typename T>
__device__ __forceinline__ void tile_product(const Operand& a, const Operand& b, int64_t i0, int64_t mi, int64_t j0, int64_t nj,
                                             int64_t K, float (&A)[32][68], float (&B)[32][68], double (&sum)[4][4]) {
  const int tid = threadIdx.x, ty = tid / 16, tx = tid % 16;
  float acc[4][4] = {};
  for (int64_t k0 = 0; k0 < K; k0 += 32) {
    __syncthreads();
    for (int e = tid; e < 32 * 64; e += 256) {
      // consecutive threads along the axis whose stride is one
      const int ka = a.sk == 1 ? e % 32 : e / 64, ra = a.sk == 1 ? e / 32 : e % 64;
      const int kb = b.sk == 1 ? e % 32 : e / 64, rb = b.sk == 1 ? e / 32 : e % 64;
      A[ka][ra] = k0 + ka < K && i0 + ra < mi ? value_of(static_cast<const T*>(a.p) + (i0 + ra) * a.si + (k0 + ka) * a.sk) : 0.f;
      B[kb][rb] = k0 + kb < K && j0 + rb < nj ? value_of(static_cast<const T*>(b.p) + (j0 + rb) * b.si + (k0 + kb) * b.sk) : 0.f;
    }
    __syncthreads();
#pragma unroll 4
    for (int k = 0; k < 32; ++k) {
      float p[4], q[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        p[x] = A[k][ty * 4 + x];
        q[x] = B[k][tx * 4 + x];
      }
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) acc[x][y] += p[x] * q[y];
    }
    if (((k0 / 32) & 7) == 7 || k0 + 32 >= K) {
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          sum[x][y] += (double)acc[x][y];
          acc[x][y] = 0.f;
        }
    }
  }
}

template <typename T, int ACT>
__global__ void __launch_bounds__(256) k_glu_forward(GluCall c, DropArgs drop) {
  __shared__ float A[32][68], B[32][68];
  const int nbf = (c.f + 63) / 64;
  const int64_t i0 = (int64_t)(blockIdx.x / nbf) * 64, j0 = (int64_t)(blockIdx.x % nbf) * 64;
  double z[4][4] = {}, u[4][4] = {};
  const Operand x{c.x, c.ldx, 1};
  tile_product<T>(x, Operand{c.wg, c.ldg, 1}, i0, c.T, j0, c.f, c.d, A, B, z);
  tile_product<T>(x, Operand{c.wu, c.ldu, 1}, i0, c.T, j0, c.f, c.d, A, B, u);
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  const uint64_t offset = drop.on ? drop_offset(drop) : 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t t = i0 + ty * 4 + k;
    if (t >= c.T) continue;
    uint32_t w[4];
    if (drop.on) drop_bits(drop, offset, (uint32_t)t, (uint32_t)(j0 + tx * 4) / 8, w);
#pragma unroll
    for (int l = 0; l < 4; ++l) {
      const int64_t j = j0 + tx * 4 + l;
      if (j >= c.f) continue;
      const float zz = (float)z[k][l], uu = (float)u[k][l];
      float h = act_value<ACT>(zz) * uu;
      if (drop.on) h = drop_one(drop, w, (int)(j % 8), h);
      store_of(static_cast<T*>(c.h) + t * c.ldh + j, h);
      if (c.gate) {
        store_of(static_cast<T*>(c.gate) + t * c.ldz + j, zz);
        store_of(static_cast<T*>(c.up) + t * c.ldup + j, uu);
      }
    }
  }
}

// dgate and dup: eight columns of a row a thread.
template <typename T, int ACT>
__global__ void __launch_bounds__(256) k_glu_gradients(GluGradCall c, DropArgs drop, int nb, int64_t n) {
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
  pack8(u, o);
  store8(static_cast<T*>(c.dup) + t * c.lddup + j, o, m, false);
}

template <typename T>
__global__ void __launch_bounds__(256) k_glu_dx(GluGradCall c) {
  __shared__ float A[32][68], B[32][68];
  const int nbd = (c.d + 63) / 64;
  const int64_t i0 = (int64_t)(blockIdx.x / nbd) * 64, j0 = (int64_t)(blockIdx.x % nbd) * 64;
  double s[4][4] = {};
  tile_product<T>(Operand{c.dgate, c.lddz, 1}, Operand{c.wg, 1, c.ldg}, i0, c.T, j0, c.d, c.f, A, B, s);
  tile_product<T>(Operand{c.dup, c.lddup, 1}, Operand{c.wu, 1, c.ldu}, i0, c.T, j0, c.d, c.f, A, B, s);
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int l = 0; l < 4; ++l) {
      const int64_t t = i0 + ty * 4 + k, j = j0 + tx * 4 + l;
      if (t < c.T && j < c.d) store_of(static_cast<T*>(c.dx) + t * c.lddx + j, (float)s[k][l]);
    }
}

template <typename T>
__global__ void __launch_bounds__(256) k_wgrad_x(WgradXCall c) {
  __shared__ float A[32][68], B[32][68];
  const int nbd = (c.d + 63) / 64;
  const int64_t i0 = (int64_t)(blockIdx.x / nbd) * 64, j0 = (int64_t)(blockIdx.x % nbd) * 64;
  double s[4][4] = {};
  tile_product<T>(Operand{c.delta, 1, c.ldd}, Operand{c.x, 1, c.ldx}, i0, c.m, j0, c.d, c.T, A, B, s);
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int l = 0; l < 4; ++l) {
      const int64_t i = i0 + ty * 4 + k, j = j0 + tx * 4 + l;
      if (i >= c.m || j >= c.d) continue;
      float* w = c.W + i * c.ldw + j;
      const double v = (double)c.alpha * s[k][l];
      *w = (float)(c.accumulate ? (double)*w + v : v);
    }
}

int64_t glu_grid(int64_t T, int n) { return cdiv(T, 64) * cdiv(n, 64); }
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

}  // namespace

hipError_t launch_glu_forward(const GluCall& c, const DropArgs& drop, hipStream_t s) {
  if (c.T == 0) return hipSuccess;
  with_type(c.dtype, [&](auto t) {
    with_act(c.act, [&](auto a) {
      hipLaunchKernelGGL((k_glu_forward<decltype(t), decltype(a)::value>), dim3((unsigned)glu_grid(c.T, c.f)), dim3(256),
                         0, s, c, drop);
    });
  });
  return hipGetLastError();
}

hipError_t launch_glu_backward(const GluGradCall& c, const DropArgs& drop, hipStream_t s) {
  if (c.T == 0) return hipSuccess;
  with_type(c.dtype, [&](auto t) {
    using E = decltype(t);
    with_act(c.act, [&](auto a) {
      hipLaunchKernelGGL((k_glu_gradients<E, decltype(a)::value>), dim3((unsigned)glu_gradients_grid(c.T, c.f)), dim3(256),
                         0, s, c, drop, (int)cdiv(c.f, 8), c.T * cdiv(c.f, 8));
    });
    if (c.dx) hipLaunchKernelGGL(k_glu_dx<E>, dim3((unsigned)glu_grid(c.T, c.d)), dim3(256), 0, s, c);
  });
  return hipGetLastError();
}

hipError_t launch_wgrad_x(const WgradXCall& c, hipStream_t s) {
  if (c.T == 0 && c.accumulate) return hipSuccess;
  with_type(c.dtype, [&](auto t) {
    hipLaunchKernelGGL(k_wgrad_x<decltype(t)>, dim3((unsigned)glu_grid(c.m, c.d)), dim3(256), 0, s, c);
  });
  return hipGetLastError();
}

}  // namespace gift
