// 8-bit activation checkpoints: save (x -> codes, exponents) and restore.
// The format and its rounding are described in act8.hpp.
//
// GIFT 阅读笔记, Eq. (4): the backward pass needs the layer's input a for
// the weight gradient W_g = delta^T a; the checkpoint keeps it in 33/32 bytes
// an element instead of 2 or 4.
//
// Both kernels only move memory.  A thread owns 8 columns of 8 consecutive
// tokens: eight independent 16-byte loads in flight, the block maximum by two
// lane exchanges among the 4 threads of a 32-column block, and one 8-byte
// store (load) of the 8 tokens' exponents.
#include "act8.hpp"

namespace gift {

namespace {
constexpr int kActThreads = 256;

// Threads across a row: the power of two in 4..256 that covers ldc / 8
// chunks (narrow rows put several token groups into one workgroup).
int row_threads_log(int64_t chunks) {
  int l = 2;
  while (l < 8 && ((int64_t)1 << l) < chunks) ++l;
  return l;
}
}  // namespace

struct ActArgs {
  const void* x;      // save: input; restore: unused
  void* out;          // restore: output
  int64_t ld;         // of x or out
  uint8_t* codes;
  int64_t ldc;
  uint8_t* bscales;
  int64_t T;
  int d, nb, fmt, lxlog;
  int colblocks;      // workgroups across a row
  int stream;         // restore: the output is larger than the caches (act8.hpp)
};

// STREAM: codes larger than the caches (act8.hpp), the input is read past them
// too (16384 x 6144 bf16: 55.7 -> 51 us).
template <typename TX, bool STREAM>
__global__ void __launch_bounds__(kActThreads) k_act_save(ActArgs a) {
  const int lx = 1 << a.lxlog;
  const int cx = threadIdx.x & (lx - 1), ty = threadIdx.x >> a.lxlog;
  const int cb = blockIdx.x % a.colblocks;
  const int64_t g = (int64_t)(blockIdx.x / a.colblocks) * (kActThreads >> a.lxlog) + ty;   // token group
  const int64_t t0 = g * kActGroup;
  const int col = (cb * lx + cx) * 8;
  // the four threads of a block share this condition (32-column granularity)
  if (t0 >= a.T || col >= a.nb * kActBlock) return;
  const TX* x = static_cast<const TX*>(a.x);
  const int n = a.d - col;   // elements of this chunk inside the row (may be <= 0 or > 8)
  Raw8<TX> r[kActGroup];
#pragma unroll
  for (int i = 0; i < kActGroup; ++i) r[i] = load8<TX, STREAM>(x + (t0 + i) * a.ld + col, t0 + i < a.T ? n : 0);
  uint32_t ex[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < kActGroup; ++i) {
    float v[8];
    unpack8(r[i], v);
    const uint32_t e = act_exponent(quad_max(amax_bits(r[i])), a.fmt);
    ex[i / 4] |= e << (8 * (i % 4));
    uint32_t w[2];
    act_encode8(v, e, a.fmt, w);
    if (t0 + i < a.T) store_words<2>(a.codes + (t0 + i) * a.ldc + col, w, STREAM);
  }
  if ((cx & 3) == 0)
    __builtin_memcpy(__builtin_assume_aligned(a.bscales + (g * a.nb + col / kActBlock) * kActGroup, 8), ex, 8);
}

template <typename TX>
__global__ void __launch_bounds__(kActThreads) k_act_restore(ActArgs a) {
  const int lx = 1 << a.lxlog;
  const int cx = threadIdx.x & (lx - 1), ty = threadIdx.x >> a.lxlog;
  const int cb = blockIdx.x % a.colblocks;
  const int64_t g = (int64_t)(blockIdx.x / a.colblocks) * (kActThreads >> a.lxlog) + ty;
  const int64_t t0 = g * kActGroup;
  const int col = (cb * lx + cx) * 8;
  if (t0 >= a.T || col >= a.d) return;
  const int n = a.d - col;
  uint32_t w[kActGroup][2], ex[2];
#pragma unroll
  for (int i = 0; i < kActGroup; ++i) {
    const int64_t t = t0 + i < a.T ? t0 + i : t0;
    __builtin_memcpy(w[i], __builtin_assume_aligned(a.codes + t * a.ldc + col, 8), 8);
  }
  __builtin_memcpy(ex, __builtin_assume_aligned(a.bscales + (g * a.nb + col / kActBlock) * kActGroup, 8), 8);
  TX* out = static_cast<TX*>(a.out);
#pragma unroll
  for (int i = 0; i < kActGroup; ++i) {
    float v[8];
    act_decode8(w[i], (ex[i / 4] >> (8 * (i % 4))) & 0xFFu, a.fmt, v);
    Raw8<TX> r;
    pack8(v, r);
    if (t0 + i < a.T) store8(out + (t0 + i) * a.ld + col, r, n, a.stream != 0);
  }
}

static ActArgs act_args(const gift_act_ckpt& c, int64_t T, int d, int64_t* grid) {
  ActArgs a{};
  a.codes = c.d_codes;
  a.ldc = c.ldc;
  a.bscales = c.d_bscales;
  a.T = T;
  a.d = d;
  a.nb = (int)cdiv(d, kActBlock);
  a.fmt = c.fmt;
  a.lxlog = row_threads_log((int64_t)a.nb * 4);
  a.colblocks = (int)cdiv((int64_t)a.nb * 4, (int64_t)1 << a.lxlog);
  *grid = cdiv(cdiv(T, kActGroup), kActThreads >> a.lxlog) * a.colblocks;
  return a;
}

// Workgroups of a save or restore launch (the host refuses what exceeds a grid).
int64_t act_grid(int64_t T, int d) {
  int64_t grid;
  gift_act_ckpt c{};
  act_args(c, T, d, &grid);
  return grid;
}

hipError_t launch_act_save(const void* x, int dtype, int64_t ld, int64_t T, int d, const gift_act_ckpt& c,
                           hipStream_t s) {
  if (T == 0) return hipSuccess;
  int64_t grid;
  ActArgs a = act_args(c, T, d, &grid);
  a.x = x;
  a.ld = ld;
  const dim3 gd((unsigned)grid), bd(kActThreads);
  auto go = [&](auto tx) {
    using TX = decltype(tx);
    if (T * a.nb * kActBlock > kStreamBytes) hipLaunchKernelGGL((k_act_save<TX, true>), gd, bd, 0, s, a);
    else hipLaunchKernelGGL((k_act_save<TX, false>), gd, bd, 0, s, a);
  };
  if (dtype == GIFT_BF16) go(Bf16{});
  else if (dtype == GIFT_FP16) go(Fp16{});
  else go(float{});
  return hipGetLastError();
}

hipError_t launch_act_restore(const gift_act_ckpt& c, int64_t T, int d, void* out, int dtype, int64_t ld,
                              hipStream_t s) {
  if (T == 0) return hipSuccess;
  int64_t grid;
  ActArgs a = act_args(c, T, d, &grid);
  a.out = out;
  a.ld = ld;
  a.stream = T * d * (dtype == GIFT_FP32 ? 4 : 2) > kStreamBytes;
  const dim3 gd((unsigned)grid), bd(kActThreads);
  if (dtype == GIFT_BF16) hipLaunchKernelGGL(k_act_restore<Bf16>, gd, bd, 0, s, a);
  else if (dtype == GIFT_FP16) hipLaunchKernelGGL(k_act_restore<Fp16>, gd, bd, 0, s, a);
  else hipLaunchKernelGGL(k_act_restore<float>, gd, bd, 0, s, a);
  return hipGetLastError();
}

}  // namespace gift
