// Dropout with a mask that is computed where it is needed and never stored:
//   y = D(x) (+ residual),  D(x) = keep ? x / (1 - p) : 0.
// A thread takes eight columns of a row: one Philox call gives their 8 x 16
// bits.  (32 bits an element would take two, about 35 us of multiplications for
// 16384 x 1536; sixteen leave p in steps of 2^-16.)  Bound by memory: 16384 x 1536
// bf16 with a residual 151 MB in 24 us, 6.2 TB/s; 8191 x 1023 fp32, rows anywhere,
// 67 MB in 12 us; one token 2 us of kernel, 7 with its launch and output.
#include "glu.hpp"

namespace gift {

struct DropoutArgs {
  DropArgs drop;
  const void *x, *r;
  void* y;
  int64_t ldx, ldr, ldy, n;   // n: chunks of eight columns, over all rows
  int d, nb;                  // nb: chunks of a row
};

constexpr int kDropChunks = 256;   // chunks of a workgroup

template <typename T>
__global__ void __launch_bounds__(256) k_dropout(DropoutArgs a) {
  const int64_t first = (int64_t)blockIdx.x * kDropChunks;
  const int64_t t0 = first / a.nb;
  const uint32_t at = (uint32_t)(first - t0 * a.nb) + threadIdx.x;
  if (first + threadIdx.x >= a.n) return;
  const uint32_t down = at / (uint32_t)a.nb, c = at - down * (uint32_t)a.nb;
  const int64_t t = t0 + down;
  const int n = a.d - (int)c * 8;
  const Raw8<T> x = load8(static_cast<const T*>(a.x) + t * a.ldx + c * 8, n);
  float v[8], r[8];
  unpack8(x, v);
  uint32_t w[4];
  drop_bits(a.drop, drop_offset(a.drop), (uint32_t)t, c, w);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = drop_one(a.drop, w, i, v[i]);
  if (a.r) {
    unpack8(load8(static_cast<const T*>(a.r) + t * a.ldr + c * 8, n), r);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += r[i];
  }
  Raw8<T> y;
  pack8(v, y);
  store8(static_cast<T*>(a.y) + t * a.ldy + c * 8, y, n, false);
}

int64_t dropout_grid(int64_t T, int d) { return cdiv(T * cdiv(d, 8), kDropChunks); }

hipError_t launch_dropout(const DropArgs& drop, const void* x, int dtype, int64_t ldx, int64_t T, int d, const void* r,
                          int64_t ldr, void* y, int64_t ldy, hipStream_t s) {
  if (T == 0) return hipSuccess;
  DropoutArgs a{};
  a.drop = drop;
  a.x = x;
  a.r = r;
  a.y = y;
  a.ldx = ldx;
  a.ldr = ldr;
  a.ldy = ldy;
  a.d = d;
  a.nb = (int)cdiv(d, 8);
  a.n = T * a.nb;
  const dim3 grid((unsigned)dropout_grid(T, d));
  if (dtype == GIFT_BF16) hipLaunchKernelGGL(k_dropout<Bf16>, grid, dim3(256), 0, s, a);
  else if (dtype == GIFT_FP16) hipLaunchKernelGGL(k_dropout<Fp16>, grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL(k_dropout<float>, grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace gift
