// Gated block of few tokens (a decoding step): h = D(act(x Wg^T) (x Wu^T)) for
// few rows of x (glu_by_tokens).  Every weight is read once (33 to 64 fp32 tokens
// run as two sets, 32 tokens and the rest, and read them twice), and the memory
// pipe is what bounds it.
//
// A workgroup of 8 waves makes 16 hidden units of all tokens of a set, or 32
// (glu_token_units).  The waves share
// the long axis in blocks of 64: a lane loads 16 bytes of a weight row (16 rows x 64
// bytes a load; rows may start anywhere) straight into the operand of
// v_mfma_f32_16x16x32, tokens being the other operand, in 16s.  The next block's
// loads are in flight while one is multiplied.  The partial sums of the waves
// meet in LDS and are added in order.  fp32 operands are split into three bf16
// numbers in registers (split_planes); six products are added.
// Measured: 1 token, 1536 x 6144 bf16 9.7 us (weights at a copy's rate 6.1), fp32
// 23 (12.2), 64 tokens fp32 45; 16 tokens, 4096 x 16384 bf16 58 us (43.5; 4.6 TB/s).  A wave has 8 to 16 KB
// of loads in flight; what is left is the loads of x, which every workgroup
// repeats, and the sums' way through LDS.
#include "product.hpp"

namespace gift {

template <typename T, int ACT, int NT, int R>
__global__ void __launch_bounds__(64 * kTokenWaves) k_glu_tokens(GluCall c, DropArgs drop) {
  constexpr int TOK = 16 * NT, PITCH = 16 * R + 4;   // (floats of a token's hidden units)
  __shared__ float part[kTokenWaves][2][TOK][PITCH];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int row = lane & 15, kq = lane >> 4;
  const int f0 = blockIdx.x * 16 * R;
  const T *g[R], *u[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int fr = f0 + 16 * r + row < c.f ? f0 + 16 * r + row : c.f - 1;
    g[r] = static_cast<const T*>(c.wg) + (int64_t)fr * c.ldg;
    u[r] = static_cast<const T*>(c.wu) + (int64_t)fr * c.ldu;
  }
  const T* x[NT];
  const int t0 = blockIdx.y * TOK;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int64_t t = t0 + 16 * n + row < c.T ? t0 + 16 * n + row : c.T - 1;
    x[n] = static_cast<const T*>(c.x) + t * c.ldx;
  }
  tf32x4 z[R][NT], v[R][NT];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) z[r][n][i] = v[r][n][i] = 0.f;
  struct Block {
    Raw8<T> g[2][R], u[2][R], x[2][NT];
  };
  auto load = [&](Block& b, int k0) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int k = k0 + 32 * s + 8 * kq, n = c.d - k;
      if (k0 + 64 <= c.d) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          b.g[s][r] = load8(g[r] + k, 8);
          b.u[s][r] = load8(u[r] + k, 8);
        }
#pragma unroll
        for (int m = 0; m < NT; ++m) b.x[s][m] = load8(x[m] + k, 8);
      } else {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          b.g[s][r] = load8(g[r] + k, n);
          b.u[s][r] = load8(u[r] + k, n);
        }
#pragma unroll
        for (int m = 0; m < NT; ++m) b.x[s][m] = load8(x[m] + k, n);
      }
    }
  };
  auto multiply_block = [&](const Block& b) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      OperandPlanes<T> px[NT];
#pragma unroll
      for (int m = 0; m < NT; ++m) px[m] = operand_planes(b.x[s][m]);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const OperandPlanes<T> pg = operand_planes(b.g[s][r]), pu = operand_planes(b.u[s][r]);
#pragma unroll
        for (int m = 0; m < NT; ++m) {
          z[r][m] = multiply_planes(pg, px[m], z[r][m]);
          v[r][m] = multiply_planes(pu, px[m], v[r][m]);
        }
      }
    }
  };
  constexpr int STEP = 64 * kTokenWaves;
  int k0 = wave * 64;
  if (k0 < c.d) {
    Block b0, b1;
    load(b0, k0);
    while (true) {
      if (k0 + STEP < c.d) load(b1, k0 + STEP);
      multiply_block(b0);
      k0 += STEP;
      if (k0 >= c.d) break;
      if (k0 + STEP < c.d) load(b0, k0 + STEP);
      multiply_block(b1);
      k0 += STEP;
      if (k0 >= c.d) break;
    }
  }
  // register i: hidden unit 4 (lane / 16) + i, token lane % 16
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      *reinterpret_cast<tf32x4*>(&part[wave][0][16 * n + row][16 * r + 4 * kq]) = z[r][n];
      *reinterpret_cast<tf32x4*>(&part[wave][1][16 * n + row][16 * r + 4 * kq]) = v[r][n];
    }
  __syncthreads();
  const int tt = threadIdx.x / (2 * R), h = threadIdx.x % (2 * R) * 8;
  const int64_t t = t0 + tt;
  if (t >= c.T || tt >= TOK || f0 + h >= c.f) return;
  float zz[8] = {}, vv[8] = {};
#pragma unroll
  for (int w = 0; w < kTokenWaves; ++w)
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      const tf32x4 a = *reinterpret_cast<const tf32x4*>(&part[w][0][tt][h + i]);
      const tf32x4 b = *reinterpret_cast<const tf32x4*>(&part[w][1][tt][h + i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        zz[i + j] += a[j];
        vv[i + j] += b[j];
      }
    }
  const int col = f0 + h, n = c.f - col;
  Raw8<T> o;
  if (c.gate) {
    pack8(zz, o);
    store8(static_cast<T*>(c.gate) + t * c.ldz + col, o, n, false);
    pack8(vv, o);
    store8(static_cast<T*>(c.up) + t * c.ldup + col, o, n, false);
  }
  uint32_t w[4];
  if (drop.on) drop_bits(drop, drop_offset(drop), (uint32_t)t, (uint32_t)col / 8, w);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    vv[i] = act_value<ACT>(zz[i]) * vv[i];
    if (drop.on) vv[i] = drop_one(drop, w, i, vv[i]);
  }
  pack8(vv, o);
  store8(static_cast<T*>(c.h) + t * c.ldh + col, o, n, false);
}

namespace {

template <typename T, int ACT, int NT>
void tokens_rows(const GluCall& c, const DropArgs& drop, hipStream_t s) {
  const dim3 block(64 * kTokenWaves);
  if constexpr (sizeof(T) == 2 && NT < 4)
    if (glu_token_units(c.dtype, c.T, c.f) == 2) {
      hipLaunchKernelGGL((k_glu_tokens<T, ACT, NT, 2>), dim3((unsigned)cdiv(c.f, 32)), block, 0, s, c, drop);
      return;
    }
  // (fp32: 32 tokens at a time)
  hipLaunchKernelGGL((k_glu_tokens<T, ACT, NT, 1>), dim3((unsigned)cdiv(c.f, 16), (unsigned)cdiv(c.T, 16 * NT)), block, 0, s, c,
                     drop);
}
template <typename T, int ACT>
void tokens_go(const GluCall& c, const DropArgs& drop, hipStream_t s) {
  if (c.T <= 16) tokens_rows<T, ACT, 1>(c, drop, s);
  else if (c.T <= 32 || sizeof(T) == 4) tokens_rows<T, ACT, 2>(c, drop, s);
  else if constexpr (sizeof(T) == 2) tokens_rows<T, ACT, 4>(c, drop, s);
}
template <typename T>
void tokens_act(const GluCall& c, const DropArgs& drop, hipStream_t s) {
  switch (c.act) {
    case GIFT_ACT_SILU: return tokens_go<T, GIFT_ACT_SILU>(c, drop, s);
    case GIFT_ACT_GELU: return tokens_go<T, GIFT_ACT_GELU>(c, drop, s);
    case GIFT_ACT_GELU_TANH: return tokens_go<T, GIFT_ACT_GELU_TANH>(c, drop, s);
    case GIFT_ACT_RELU: return tokens_go<T, GIFT_ACT_RELU>(c, drop, s);
    default: return tokens_go<T, GIFT_ACT_SIGMOID>(c, drop, s);
  }
}

}  // namespace

hipError_t launch_glu_tokens(const GluCall& c, const DropArgs& drop, hipStream_t s) {
  if (c.dtype == GIFT_BF16) tokens_act<Bf16>(c, drop, s);
  else if (c.dtype == GIFT_FP16) tokens_act<Fp16>(c, drop, s);
  else tokens_act<float>(c, drop, s);
  return hipGetLastError();
}

}  // namespace gift
