// Shared device code of the activation operators: element types, the 8-bit
// checkpoint format, and sums over a group of lanes.
//
// Checkpoint of x [T][d]: one FP8 code per element (E4M3 or E5M2, the OCP
// layouts) and one power-of-two scale per token and 32 columns.  The scale is
// kept as a biased exponent e (the fp32 exponent field): the smallest e >= 32
// with amax <= FMAX 2^(e - 127), so no code saturates.  code = RNE(x 2^(127 -
// e)), value = code 2^(e - 127).  A power of two makes both multiplications
// exact: the only rounding of the round trip is the one to a code.  It is off
// by at most 2^-4 (E4M3: 4 significant bits) or 2^-3 (E5M2: 3) of the value,
// or, for elements so far below their block's largest that they get a
// subnormal code, by half the step of those: 2^-10 2^(e - 127) or 2^-17 2^(e -
// 127).  A value is exact in bf16, but for 2^128, to which elements in the
// last half step of fp32's range round.  The lower limit 32 keeps every value
// at or above 2^-111, a normal bf16 and fp32 number: the conversions and the
// matrix instructions never see a subnormal.  (2^-95 is far below any
// activation; smaller blocks round to the subnormal codes and to zero.)  A
// block that holds an Inf or NaN is stored as e = 255 and codes 0x7F, and its
// values are NaN.
//
// Layout: codes [T][ldc], ldc a multiple of 32 with ldc >= d; the exponents
// are [ceil(T / 8)][nb][8], nb = ceil(d / 32): the eight tokens that one
// matrix operand register holds for one column lie side by side, so the
// weight-gradient product fetches their scales with one 8-byte load.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gift_internal.hpp"

namespace gift {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr int kActBlock = 32;     // columns per scale
constexpr int kActGroup = 8;      // tokens per group of the exponent layout
constexpr uint32_t kActExpMin = 32, kActExpBad = 255;

// FMAX is 1.75 2^8 (E4M3) and 1.75 2^15 (E5M2): amax = 1.f 2^(E - 127) needs
// e = E - 8 (or 15), one more when 1.f exceeds 1.75.
__device__ __forceinline__ uint32_t act_exponent(uint32_t amax_bits, int fmt) {
  if (amax_bits >= 0x7F800000u) return kActExpBad;
  const int e = (int)(amax_bits >> 23) - (fmt == 0 ? 8 : 15) + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return e < (int)kActExpMin ? kActExpMin : (uint32_t)e;
}

// The scale 2^(e - 127) (e in 32..247) and its inverse as floats.
__device__ __forceinline__ float act_scale(uint32_t e) { return __uint_as_float(e << 23); }
__device__ __forceinline__ float act_inverse(uint32_t e) { return __uint_as_float((254u - e) << 23); }

// Codes of eight values under exponent e, four to a word.
__device__ __forceinline__ void act_encode8(const float* v, uint32_t e, int fmt, uint32_t* out) {
  const float r = act_inverse(e);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float a = v[4 * h] * r, b = v[4 * h + 1] * r, c = v[4 * h + 2] * r, d = v[4 * h + 3] * r;
    int w = 0;
    if (fmt == 0) {
      w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, w, false);
      w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
    } else {
      w = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, w, false);
      w = __builtin_amdgcn_cvt_pk_bf8_f32(c, d, w, true);
    }
    out[h] = e == kActExpBad ? 0x7F7F7F7Fu : (uint32_t)w;
  }
}

// Values of eight codes (two words) under exponent e.
__device__ __forceinline__ void act_decode8(const uint32_t* w, uint32_t e, int fmt, float* v) {
  const float s = act_scale(e);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    f32x2 lo, hi;
    if (fmt == 0) {
      lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[h], false);
      hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[h], true);
    } else {
      lo = __builtin_amdgcn_cvt_pk_f32_bf8((int)w[h], false);
      hi = __builtin_amdgcn_cvt_pk_f32_bf8((int)w[h], true);
    }
    v[4 * h] = lo[0] * s;
    v[4 * h + 1] = lo[1] * s;
    v[4 * h + 2] = hi[0] * s;
    v[4 * h + 3] = hi[1] * s;
  }
}

// Element types.  Eight elements are held as 4 (16-bit) or 8 (fp32) words.
struct Bf16 {
  uint16_t v;
};
struct Fp16 {
  uint16_t v;
};

template <typename T>
struct Raw8 {
  uint32_t w[sizeof(T) * 2];
};

__device__ __forceinline__ void unpack8(const Raw8<Bf16>& r, float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(r.w[i] << 16);
    v[2 * i + 1] = __uint_as_float(r.w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void unpack8(const Raw8<Fp16>& r, float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f16x2 h = __builtin_bit_cast(f16x2, r.w[i]);
    v[2 * i] = (float)h[0];
    v[2 * i + 1] = (float)h[1];
  }
}
__device__ __forceinline__ void unpack8(const Raw8<float>& r, float* v) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r.w[i]);
}

// Bits of the largest magnitude of the eight as fp32 (at or above 0x7F800000
// when one is an infinity or NaN).  Magnitudes order like their bits, so a
// 16-bit type compares two at a time.
__device__ __forceinline__ uint32_t amax16(const uint32_t* w) {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  u16x2 m = __builtin_bit_cast(u16x2, w[0] & 0x7FFF7FFFu);
#pragma unroll
  for (int i = 1; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, w[i] & 0x7FFF7FFFu));
  return m[0] > m[1] ? m[0] : m[1];
}
__device__ __forceinline__ uint32_t amax_bits(const Raw8<Bf16>& r) { return amax16(r.w) << 16; }
__device__ __forceinline__ uint32_t amax_bits(const Raw8<Fp16>& r) {
  return __float_as_uint((float)__builtin_bit_cast(_Float16, (uint16_t)amax16(r.w)));
}
__device__ __forceinline__ uint32_t amax_bits(const Raw8<float>& r) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = r.w[i] & 0x7FFFFFFFu;
    m = b > m ? b : m;
  }
  return m;
}

// One rounding to nearest even each (none for fp32).
__device__ __forceinline__ void pack8(const float* v, Raw8<Bf16>& r) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f32x2 f = {v[2 * i], v[2 * i + 1]};
    r.w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2));
  }
}
__device__ __forceinline__ void pack8(const float* v, Raw8<Fp16>& r) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f32x2 f = {v[2 * i], v[2 * i + 1]};
    r.w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, f16x2));
  }
}
__device__ __forceinline__ void pack8(const float* v, Raw8<float>& r) {
#pragma unroll
  for (int i = 0; i < 8; ++i) r.w[i] = __float_as_uint(v[i]);
}

// An output larger than the L2 caches of the eight dies together (4 MB each)
// is gone from them before anyone reads it: written past them it leaves them
// to the inputs (norm forward, 16384 x 1536 bf16: 28.1 -> 20.6 us; save and
// restore, 16384 x 6144 bf16: 120 -> 98 us).  Smaller outputs stay cached
// for the next kernel.
constexpr int64_t kStreamBytes = (int64_t)32 << 20;

// n (<= 8) of the eight elements at p, the others zero.  Whole chunks are
// 16-byte loads at any element alignment (rows of odd length start anywhere;
// the memory pipe takes unaligned vectors); only a row's last, partial chunk
// is fetched element by element.
template <typename T, bool STREAM = false>
__device__ __forceinline__ Raw8<T> load8(const T* p, int n) {
  Raw8<T> r;
  if (n >= 8) {
    if constexpr (STREAM) {   // past the caches
      typedef uint32_t V __attribute__((ext_vector_type(4), aligned(1)));
#pragma unroll
      for (int q = 0; q < (int)sizeof(r.w) / 16; ++q) {
        const V v = __builtin_nontemporal_load(reinterpret_cast<const V*>(p) + q);
#pragma unroll
        for (int i = 0; i < 4; ++i) r.w[4 * q + i] = v[i];
      }
    } else {
      __builtin_memcpy(r.w, p, sizeof(r.w));
    }
  } else {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) * 2); ++i) r.w[i] = 0;
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) {
        if constexpr (sizeof(T) == 2) {
          uint16_t e;
          __builtin_memcpy(&e, p + i, 2);
          r.w[i / 2] |= (uint32_t)e << (16 * (i % 2));
        } else {
          __builtin_memcpy(&r.w[i], p + i, 4);
        }
      }
  }
  return r;
}
// 16 or 8 bytes at an address of any alignment.  stream: a store that does
// not stay in the caches (the empty statements keep the two forms apart:
// merged, the store would lose its hint).
template <int N>
__device__ __forceinline__ void store_words(void* p, const uint32_t* w, bool stream) {
  typedef uint32_t V __attribute__((ext_vector_type(N), aligned(1)));
  V v;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = w[i];
  if (stream) {
    asm volatile("");
    __builtin_nontemporal_store(v, static_cast<V*>(p));
    asm volatile("");
  } else {
    *static_cast<V*>(p) = v;
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const Raw8<T>& r, int n, bool stream) {
  if (n >= 8) {
#pragma unroll
    for (int q = 0; q < (int)sizeof(r.w) / 16; ++q) store_words<4>(p + q * (16 / sizeof(T)), r.w + 4 * q, stream);
  } else {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) {
        if constexpr (sizeof(T) == 2) {
          const uint16_t e = (uint16_t)(r.w[i / 2] >> (16 * (i % 2)));
          __builtin_memcpy(p + i, &e, 2);
        } else {
          __builtin_memcpy(p + i, &r.w[i], 4);
        }
      }
  }
}

// Lane exchanges inside a wave: DPP within 16 lanes (pairs, quads, halves of
// 8 and 16), row swaps across 16 and 32.  Each step combines the two halves
// of a span in both of them, so all lanes end with the same value.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_move(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
constexpr int kDppXor1 = 0xB1, kDppXor2 = 0x4E, kDppHalfMirror = 0x141, kDppMirror = 0x140;

// Maximum over the 4 lanes of one 32-column block.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  uint32_t o = dpp_move<kDppXor1>(v);
  v = o > v ? o : v;
  o = dpp_move<kDppXor2>(v);
  return o > v ? o : v;
}

// Sum over G = 16 or 64 consecutive lanes.
template <int G>
__device__ __forceinline__ float lanes_sum(float v) {
  v += __uint_as_float(dpp_move<kDppXor1>(__float_as_uint(v)));
  v += __uint_as_float(dpp_move<kDppXor2>(__float_as_uint(v)));
  v += __uint_as_float(dpp_move<kDppHalfMirror>(__float_as_uint(v)));
  v += __uint_as_float(dpp_move<kDppMirror>(__float_as_uint(v)));
  if constexpr (G == 64) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(b[0]) + __uint_as_float(b[1]);
  }
  return v;
}

}  // namespace gift
