// Shared device code of the gated feed-forward block and of dropout: the
// counter-based generator and the activations.
#pragma once
#include "act8.hpp"

namespace gift {

// Dropout as the kernels take it.  thr = round(65536 p); on == 0: no dropout.
struct DropArgs {
  uint32_t thr;
  float scale;
  uint32_t k0, k1;             // seed
  uint64_t offset;
  const uint64_t* d_offset;
  int on;
};

// Philox4x32-10 (Salmon et al., SC 2011): ten rounds of two 32 x 32 -> 64 bit
// products by fixed odd numbers, mixed with a key that grows by fixed steps.
__device__ __forceinline__ void philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, uint32_t k0, uint32_t k1,
                                       uint32_t* w) {
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  w[0] = c0;
  w[1] = c1;
  w[2] = c2;
  w[3] = c3;
}

__device__ __forceinline__ uint64_t drop_offset(const DropArgs& a) {
  return a.offset + (a.d_offset ? *a.d_offset : 0);
}

// Bits of columns 8 chunk .. 8 chunk + 7 of row t, 16 each, two to a word.
__device__ __forceinline__ void drop_bits(const DropArgs& a, uint64_t offset, uint32_t t, uint32_t chunk, uint32_t* w) {
  philox(chunk, t, (uint32_t)offset, (uint32_t)(offset >> 32), a.k0, a.k1, w);
}
__device__ __forceinline__ float drop_one(const DropArgs& a, const uint32_t* w, int i, float v) {
  const uint32_t r = i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xFFFFu;
  return r >= a.thr ? v * a.scale : 0.f;
}

// act(z) and, where asked for, act'(z), in fp32: every factor relative to its
// own size, also where act tends to zero.  exp2 and the reciprocal are the
// hardware's (1 ulp each); e^-v as 2^(-v log2 e) is off by v 2^-24 of itself.
// The normal distribution's tail is e^(-z^2 / 2) q(t), t = 1 / (1 + |z| / (2
// sqrt 2)): q is a polynomial fitted to it over |z| <= 14.8, below which e^(-z^2 /
// 2) ends.  With its coefficients as fp32 numbers it is off by 8e-8 of the tail at
// most, evaluated in fp32 by 4e-7.
__device__ __forceinline__ float exp_neg(float v) { return __builtin_amdgcn_exp2f(v * -1.4426950408889634f); }
__device__ __forceinline__ float reciprocal(float v) { return __builtin_amdgcn_rcpf(v); }

// s(v) = 1 / (1 + e^-v), and s(-v).  (e^-v is infinite, and s zero, where s is below 2^-128.)
__device__ __forceinline__ float logistic(float v, float* other) {
  const float e = exp_neg(v), s = reciprocal(1.f + e);
  *other = v >= 0.f ? e * s : 1.f - s;
  return s;
}

template <int ACT>
__device__ __forceinline__ float act_value(float z, float* grad = nullptr) {
  if constexpr (ACT == GIFT_ACT_RELU) {
    if (grad) *grad = z > 0.f ? 1.f : z == z ? 0.f : z;
    return z > 0.f ? z : z == z ? 0.f : z;
  } else if constexpr (ACT == GIFT_ACT_SILU || ACT == GIFT_ACT_SIGMOID) {
    float q;
    const float s = logistic(z, &q);
    if constexpr (ACT == GIFT_ACT_SIGMOID) {
      if (grad) *grad = s * q;
      return s;
    } else {
      if (grad) *grad = s * (1.f + z * q);
      return z * s;
    }
  } else if constexpr (ACT == GIFT_ACT_GELU) {
    const float e = exp_neg(0.5f * z * z);
    const float t = reciprocal(1.f + 0.35355339059327373f * __builtin_fabsf(z));
    float q = -0.0279172214f;
    q = q * t + 0.133988569f;
    q = q * t - 0.225301468f;
    q = q * t + 0.116354035f;
    q = q * t + 0.00403949032f;
    q = q * t + 0.0928747958f;
    q = q * t + 0.124178955f;
    q = q * t + 0.140689721f;
    q = q * t + 0.14109541f;
    q = q * t - 2.30335438e-06f;
    const float tail = q * e, n = z >= 0.f ? 1.f - tail : tail;
    if (grad) *grad = n + z * (0.3989422804014327f * e);
    return z * n;
  } else {
    constexpr float k = 1.5957691216057308f;   // 2 sqrt(2 / pi)
    const float w = k * (z + 0.044715f * z * z * z);
    float q;
    const float s = logistic(w, &q);
    // (where z^2 is infinite s q is zero, and 0 times an infinity is no number)
    if (grad) *grad = s + z * (s * q) * (k * (1.f + 0.134145f * __builtin_fminf(z * z, 0x1p100f)));
    return z * s;
  }
}

}  // namespace gift
