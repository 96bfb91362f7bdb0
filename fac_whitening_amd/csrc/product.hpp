// Device code of the matrix products of 16-bit operands (k_product.hip):
// how operands reach LDS and the matrix cores.
#pragma once
#include <type_traits>

#include "glu.hpp"
#include "product_plan.hpp"

namespace gift {

typedef __bf16 pbf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 pf16x8 __attribute__((ext_vector_type(8)));
typedef float pf32x16 __attribute__((ext_vector_type(16)));
typedef int pi32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t pu32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t pu32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void p_lds_void;

__device__ __forceinline__ pf32x16 mfma32(const pbf16x8& a, const pbf16x8& b, const pf32x16& c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ pf32x16 mfma32(const pf16x8& a, const pf16x8& b, const pf32x16& c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}
template <typename E>
using Frag8 = std::conditional_t<std::is_same<E, Fp16>::value, pf16x8, pbf16x8>;

// Three bf16 numbers whose sum is v, each the nearest to what the ones before
// it leave: put(plane, four words of eight values).  (The first is at most the
// largest bf16 number, which values beyond it would round past; of an infinity
// or NaN at least one is not finite.  Bits below 2^-133, the smallest bf16
// number, are lost: v below 2^-110 may have some.)
template <typename F>
__device__ __forceinline__ void split_planes(float* v, F&& put) {
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    float r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = p == 0 ? __builtin_amdgcn_fmed3f(v[i], -0x1.FEp127f, 0x1.FEp127f) : v[i];
    Raw8<Bf16> o;
    pack8(r, o);
    unpack8(o, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] -= r[i];
    put(p, o.w);
  }
}

typedef float tf32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ tf32x4 mfma16(const pbf16x8& a, const pbf16x8& b, const tf32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ tf32x4 mfma16(const pf16x8& a, const pf16x8& b, const tf32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// Eight elements as operands: themselves, or an fp32's three planes.
template <typename T>
struct OperandPlanes {
  static constexpr int P = sizeof(T) == 4 ? 3 : 1;
  Frag8<T> v[P];
};
template <typename T>
__device__ __forceinline__ OperandPlanes<T> operand_planes(const Raw8<T>& r) {
  OperandPlanes<T> o;
  if constexpr (sizeof(T) == 2) {
    o.v[0] = __builtin_bit_cast(Frag8<T>, r.w);
  } else {
    float v[8];
    unpack8(r, v);
    split_planes(v, [&](int p, const uint32_t* w) {
      const pu32x4 u = {w[0], w[1], w[2], w[3]};
      o.v[p] = __builtin_bit_cast(pbf16x8, u);
    });
  }
  return o;
}
template <typename T>
__device__ __forceinline__ tf32x4 multiply_planes(const OperandPlanes<T>& a, const OperandPlanes<T>& b, tf32x4 c) {
  if constexpr (sizeof(T) == 2) {
    return mfma16(a.v[0], b.v[0], c);
  } else {
    c = mfma16(a.v[0], b.v[2], c);
    c = mfma16(a.v[1], b.v[1], c);
    c = mfma16(a.v[2], b.v[0], c);
    c = mfma16(a.v[0], b.v[1], c);
    c = mfma16(a.v[1], b.v[0], c);
    return mfma16(a.v[0], b.v[0], c);
  }
}

// The kernels of few tokens: waves of a workgroup.
constexpr int kTokenWaves = 8;

__device__ __forceinline__ void store_value(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_value(Bf16* p, float v) { p->v = __builtin_bit_cast(uint16_t, (__bf16)v); }
__device__ __forceinline__ void store_value(Fp16* p, float v) { p->v = __builtin_bit_cast(uint16_t, (_Float16)v); }

// f(integral_constant<int, B>) ... f(integral_constant<int, E - 1>)
template <int B, int E, typename F>
__device__ __forceinline__ void unrolled(F&& f) {
  if constexpr (B < E) {
    f(std::integral_constant<int, B>{});
    unrolled<B + 1, E>(f);
  }
}

// 16-byte global-to-LDS load of every lane: lane l's 16 bytes from rsrc at
// voff land at LDS byte lds + 16 l (lds wave-uniform, through M0); zeros for
// an offset past the buffer's end.  As inline assembly the compiler does not
// track these LDS writes (it would wait for every load in flight before each
// LDS read); the kernel orders them itself with s_waitcnt vmcnt and barriers.
__device__ __forceinline__ void dma16(pi32x4 rsrc, uint32_t lds, int voff) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %1, %2, 0 offen lds"
      :
      : "s"(lds), "v"(voff), "s"(rsrc)
      : "memory");
}
// Waits until at most N of this wave's vector memory operations are in flight.
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N < 64, "vmcnt has 6 bits");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
// A barrier that waits for nothing else (the kernel's own waits stand before it).
__device__ __forceinline__ void bare_barrier() { asm volatile("s_barrier" ::: "memory"); }

constexpr int kPastEnd = (int)0x80000000u;   // an offset past any buffer

__device__ __forceinline__ pi32x4 buffer_of(uint64_t base, uint32_t bytes) {
  const pi32x4 rs = {__builtin_amdgcn_readfirstlane((int)(uint32_t)base),
                     __builtin_amdgcn_readfirstlane((int)(uint32_t)(base >> 32) & 0xFFFF),
                     __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000};
  return rs;
}

constexpr int kMaxSegs = 12;

// out[j][i] = sum over segments and k of A[i][k] B[j][k].  A direct operand
// has rows of k, a transposing one rows of i (j).
struct ProdArgs {
  uint64_t a[kMaxSegs], a2[kMaxSegs], b[kMaxSegs];   // a2: the second half of A's rows (the up projection)
  int nseg;
  int64_t K;            // of a segment
  int nst;              // stages of 64 of a segment
  int64_t lda, lda2, ldb;
  int64_t acols, bcols; // of a transposing operand's rows: all that may be read
  int M;                // outputs along i
  int64_t N;            // and along j
  int nbm, nbn, unit;   // tiles along i and j; tiles are split at multiples of `unit` stages
  float* part;          // pieces of split tiles
};

struct ProdOut {
  void *out, *gate, *up;
  int64_t ldo, ldz, ldup;
  DropArgs drop;
  float alpha;
  int accumulate;
  int stream;           // outputs larger than the caches are written past them
};

// One operand in the caller's memory, [rows][cols]; rows == 0: none.
struct ProdOperand {
  const void* p;
  int64_t ld, rows, cols;
  bool aligned;         // rows 16-byte aligned and at most kProductRow bytes apart
  bool near;            // rows at most kProductRow bytes apart
  bool packed;          // p is what k_product_pack makes of such an operand
};

// A product of the gated block's (see kEpi*): `parts` pairs of operands, each
// K long, added up (kEpiGlu: both a's with b[0]).
struct ProductCall {
  int epi, act, dtype, parts;
  ProdOperand a[2], b[2];
  int64_t M, N, K;
  void *out, *gate, *up;
  int64_t ldo, ldz, ldup;
  float alpha;
  int accumulate;
  void* work;
};
constexpr int64_t kProductRow = (int64_t)1 << 22;   // bytes: 256 rows' offsets stay below 2^31
int64_t product_tiles(int64_t M, int64_t N);
size_t product_packed(int dtype, int64_t rows, int64_t cols);   // bytes of an operand laid out anew
size_t product_workspace(const ProductCall& c);
bool product_reach(const ProductCall& c);                      // whether one launch lays out what has to be
hipError_t launch_product(const ProductCall& c, const DropArgs& drop, hipStream_t s);

}  // namespace gift
