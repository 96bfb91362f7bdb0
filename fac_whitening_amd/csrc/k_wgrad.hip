// Weight gradient from an 8-bit activation checkpoint:
//   W[i][j] (+)= alpha sum_t delta[t][i] a[t][j],
// delta [T][m] the output gradients, a [T][d] the values a checkpoint stands
// for, W fp32 [m][ldw]: the gradient that the codec encodes.
//
// GIFT 阅读笔记, §前置知识 Eq. (4) and §核心想法: W_g = delta^T a of a linear
// layer, averaged over the tokens (alpha = 1 / T).
#include "act8.hpp"

namespace gift {

struct WgradArgs {
  const void* delta;
  int64_t ldd;
  const uint8_t* codes;
  int64_t ldc;
  const uint8_t* bscales;
  int nb, fmt;
  int64_t T;
  int m, d;
  float alpha;
  int accumulate;
  float* W;
  int64_t ldw;
};

__device__ __forceinline__ float elem_f32(const float* p) { return *p; }
__device__ __forceinline__ float elem_f32(const Bf16* p) { return __uint_as_float((uint32_t)p->v << 16); }
__device__ __forceinline__ float elem_f32(const Fp16* p) { return (float)__builtin_bit_cast(_Float16, p->v); }

// 64 x 64 outputs per workgroup, 32 tokens per LDS stage, 4 x 4 outputs per
// thread, fp32 products and sums over 256 tokens, folded into fp64.
template <typename TD>
__global__ void __launch_bounds__(256) k_wgrad_valu(WgradArgs a) {
  __shared__ float A[32][64 + 4], B[32][64 + 4];
  const int tid = threadIdx.x, ty = tid / 16, tx = tid % 16;
  const int nbd = (a.d + 63) / 64;
  const int i0 = (int)(blockIdx.x / nbd) * 64, j0 = (int)(blockIdx.x % nbd) * 64;
  const TD* delta = static_cast<const TD*>(a.delta);
  float acc[4][4] = {};
  double sum[4][4] = {};
  for (int64_t t0 = 0; t0 < a.T; t0 += 32) {
    for (int e = tid; e < 32 * 64; e += 256) {
      const int tt = e / 64, c = e % 64;
      const int64_t t = t0 + tt;
      const int i = i0 + c, j = j0 + c;
      A[tt][c] = t < a.T && i < a.m ? elem_f32(delta + t * a.ldd + i) : 0.f;
      float v = 0.f;
      if (t < a.T && j < a.d) {
        const uint32_t code = a.codes[t * a.ldc + j];
        const uint32_t ex = a.bscales[((t >> 3) * a.nb + j / kActBlock) * kActGroup + (t & 7)];
        const f32x2 f = a.fmt == 0 ? __builtin_amdgcn_cvt_pk_f32_fp8((int)code, false)
                                   : __builtin_amdgcn_cvt_pk_f32_bf8((int)code, false);
        v = f[0] * act_scale(ex);
      }
      B[tt][c] = v;
    }
    __syncthreads();
#pragma unroll 4
    for (int tt = 0; tt < 32; ++tt) {
      float p[4], q[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        p[k] = A[tt][ty * 4 + k];
        q[k] = B[tt][tx * 4 + k];
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int l = 0; l < 4; ++l) acc[k][l] += p[k] * q[l];
    }
    __syncthreads();
    if (((t0 / 32) & 7) == 7 || t0 + 32 >= a.T) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int l = 0; l < 4; ++l) {
          sum[k][l] += (double)acc[k][l];
          acc[k][l] = 0.f;
        }
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int i = i0 + ty * 4 + k;
    if (i >= a.m) continue;
#pragma unroll
    for (int l = 0; l < 4; ++l) {
      const int j = j0 + tx * 4 + l;
      if (j >= a.d) continue;
      float* w = a.W + (int64_t)i * a.ldw + j;
      const double v = (double)a.alpha * sum[k][l];
      *w = (float)(a.accumulate ? (double)*w + v : v);
    }
  }
}

hipError_t launch_weight_grad(const WgradCall& c, hipStream_t s) {
  WgradArgs a{};
  a.delta = c.delta;
  a.ldd = c.ldd;
  a.codes = c.ckpt->d_codes;
  a.ldc = c.ckpt->ldc;
  a.bscales = c.ckpt->d_bscales;
  a.nb = (int)cdiv(c.d, kActBlock);
  a.fmt = c.ckpt->fmt;
  a.T = c.T;
  a.m = c.m;
  a.d = c.d;
  a.alpha = c.alpha;
  a.accumulate = c.accumulate;
  a.W = c.W;
  a.ldw = c.ldw;
  if (c.T == 0 && c.accumulate) return hipSuccess;
  const dim3 grid((unsigned)(cdiv(c.m, 64) * cdiv(c.d, 64)));
  if (c.dtype == GIFT_BF16) hipLaunchKernelGGL(k_wgrad_valu<Bf16>, grid, dim3(256), 0, s, a);
  else if (c.dtype == GIFT_FP16) hipLaunchKernelGGL(k_wgrad_valu<Fp16>, grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL(k_wgrad_valu<float>, grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace gift
