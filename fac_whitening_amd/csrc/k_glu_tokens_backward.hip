// Backward pass of the gated block for few tokens:
//   dgate = D(dh) u act'(z), dup = D(dh) act(z),  dx = dgate Wg + dup Wu.
// Every weight is read once, and the memory pipe is what bounds it.
//
// A workgroup of 8 waves makes 128 columns of dx of all tokens over a slab of
// the hidden units, which its waves share in steps of 32.  Of a step a lane loads
// 8 units x 8 columns of each weight (16 bytes of 8 rows, 256 bytes a row over 16
// lanes) and turns them in registers: column c of its 8 is an operand of
// v_mfma_f32_16x16x32 number c, whose 16 rows are columns c, 8 + c, ..., so that no
// LDS is needed.  The other operand is 8 units of a token, which the lane computes
// from dh, z and u, rounded as dgate and dup are (the workgroups of the first
// columns store them): dx is the product of the gradients that the weight
// gradients see, and 16-bit ones enter the matrix cores as they are.  The waves'
// sums meet in LDS, the slabs' in the
// workspace; both are added in order, the latter by a second launch.  fp32
// operands are split into three bf16 numbers in registers.
// Measured: 1 token, 91 x 16173 fp32 12 + 3 us of kernels (as tiles with their join
// 18 + 73); 2 tokens, 73 x 2752 bf16 9 + 3; 16 tokens in all, us and a copy's time of
// the weights: 1536 x 6144 bf16 20 and 6, fp32 33 and 13, 4096 x 16384 bf16 62 and 44,
// fp32 114 and 88 (17 fp32 tokens, as tiles of planes laid out in memory: 88 and 520).
// A step's loads are waited for before its products.
#include "product.hpp"

namespace gift {

struct TokensBack {
  GluGradCall c;
  DropArgs drop;
  float* part;         // [slabs][T][d]
  int slab, slabs;     // hidden units of a slab, a multiple of 256
};

// Column c of a block of 8 rows x 8 columns, as operands.
template <typename T>
__device__ __forceinline__ OperandPlanes<T> turned(const Raw8<T>* r, int c) {
  OperandPlanes<T> o;
  if constexpr (sizeof(T) == 2) {
    pu32x4 v;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      v[k] = __builtin_amdgcn_perm(r[2 * k + 1].w[c / 2], r[2 * k].w[c / 2], c & 1 ? 0x07060302u : 0x05040100u);
    o.v[0] = __builtin_bit_cast(Frag8<T>, v);
  } else {
    Raw8<float> t;
#pragma unroll
    for (int k = 0; k < 8; ++k) t.w[k] = r[k].w[c];
    o = operand_planes(t);
  }
  return o;
}

template <typename T, int ACT, int NT>
__global__ void __launch_bounds__(64 * kTokenWaves) k_glu_tokens_dx(TokensBack a) {
  constexpr int TOK = 16 * NT, W = 128, HALF = kTokenWaves / 2;
  __shared__ float sums[HALF][TOK][W + 4];
  const GluGradCall& c = a.c;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int m = lane & 15, kq = lane >> 4;
  const int i0 = blockIdx.x * W, col = i0 + 8 * m;
  const int cols = c.d - col;                          // of this lane's 8
  const int f0 = blockIdx.y * a.slab, f1 = f0 + a.slab < c.f ? f0 + a.slab : c.f;
  const uint64_t offset = a.drop.on ? drop_offset(a.drop) : 0;
  tf32x4 acc[NT][8];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int k = 0; k < 8; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][k][i] = 0.f;
  struct Step {
    Raw8<T> g[8], u[8], dh[NT], z[NT], v[NT];
  };
  auto load = [&](Step& s, int f) {
    const int k = f + 8 * kq, n = f1 - k;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int64_t row = 16 * t + m < c.T ? 16 * t + m : c.T - 1;
      s.dh[t] = load8(static_cast<const T*>(c.dh) + row * c.lddh + k, n);
      s.z[t] = load8(static_cast<const T*>(c.gate) + row * c.ldz + k, n);
      s.v[t] = load8(static_cast<const T*>(c.up) + row * c.ldup + k, n);
    }
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      // (rows past the slab's end meet zeros of the other operand; they read its last row, which may hold anything finite
      // or not, so they are zero too)
      const int64_t row = r < n ? k + r : f1 - 1;
      s.g[r] = load8(static_cast<const T*>(c.wg) + row * c.ldg + col, r < n ? cols : 0);
      s.u[r] = load8(static_cast<const T*>(c.wu) + row * c.ldu + col, r < n ? cols : 0);
    }
  };
  auto multiply_step = [&](const Step& s, int f) {
    const int k = f + 8 * kq, n = f1 - k;
    OperandPlanes<T> dz[NT], du[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float e[8], z[8], u[8];
      unpack8(s.dh[t], e);
      unpack8(s.z[t], z);
      unpack8(s.v[t], u);
      if (a.drop.on) {
        uint32_t w[4];
        drop_bits(a.drop, offset, (uint32_t)(16 * t + m), (uint32_t)k / 8, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = drop_one(a.drop, w, i, e[i]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float g;
        const float v = act_value<ACT>(z[i], &g);
        z[i] = i < n ? e[i] * u[i] * g : 0.f;
        u[i] = i < n ? e[i] * v : 0.f;
      }
      Raw8<T> pz, pu;
      pack8(z, pz);
      pack8(u, pu);
      if (blockIdx.x == 0 && 16 * t + m < c.T && n > 0) {
        store8(static_cast<T*>(c.dgate) + (int64_t)(16 * t + m) * c.lddz + k, pz, n, false);
        store8(static_cast<T*>(c.dup) + (int64_t)(16 * t + m) * c.lddup + k, pu, n, false);
      }
      dz[t] = operand_planes(pz);
      du[t] = operand_planes(pu);
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const OperandPlanes<T> g = turned<T>(s.g, q), u = turned<T>(s.u, q);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        acc[t][q] = multiply_planes(g, dz[t], acc[t][q]);
        acc[t][q] = multiply_planes(u, du[t], acc[t][q]);
      }
    }
  };
  constexpr int STEP = 32 * kTokenWaves;
  for (int f = f0 + 32 * wave; f < f1; f += STEP) {
    Step s;
    load(s, f);
    multiply_step(s, f);
  }
  // register i of product q: column 8 (4 (lane / 16) + i) + q of the 128, token lane % 16; the upper waves' sums, then
  // all of them added to the lower ones'
#pragma unroll
  for (int half = 1; half >= 0; --half) {
    if (wave / HALF == half) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float* p = &sums[wave % HALF][16 * t + m][8 * (4 * kq + i)];
#pragma unroll
          for (int q = 0; q < 8; q += 4) {
            tf32x4 v = {acc[t][q][i], acc[t][q + 1][i], acc[t][q + 2][i], acc[t][q + 3][i]};
            if (half == 0) {
              const tf32x4 o = *reinterpret_cast<const tf32x4*>(p + q);
#pragma unroll
              for (int j = 0; j < 4; ++j) v[j] += o[j];
            }
            *reinterpret_cast<tf32x4*>(p + q) = v;
          }
        }
    }
    __syncthreads();
  }
  const int width = c.d - i0 < W ? c.d - i0 : W;
  for (int e = threadIdx.x; e < TOK * W; e += 64 * kTokenWaves) {
    const int t = e / W, j = e % W;
    if (t >= c.T || j >= width) continue;
    float v = sums[0][t][j];
#pragma unroll
    for (int h = 1; h < HALF; ++h) v += sums[h][t][j];
    if (a.slabs > 1) a.part[((int64_t)blockIdx.y * c.T + t) * c.d + i0 + j] = v;
    else store_value(static_cast<T*>(c.dx) + t * c.lddx + i0 + j, v);
  }
}

// dx from the slabs' sums.
template <typename T>
__global__ void __launch_bounds__(256) k_glu_tokens_join(const float* part, int slabs, int64_t T_, int d, T* dx, int64_t ld) {
  const int64_t n = T_ * d, e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (e >= n) return;
  float v = 0.f;
  int s = 0;
  for (; s + 8 <= slabs; s += 8) {
    float p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = part[(int64_t)(s + i) * n + e];
#pragma unroll
    for (int i = 0; i < 8; ++i) v += p[i];
  }
  for (; s < slabs; ++s) v += part[(int64_t)s * n + e];
  const int64_t t = e / d;
  store_value(dx + t * ld + (e - t * d), v);
}

namespace {

// Slabs of whole steps of all waves: enough for two workgroups a compute unit,
// as long as a wave has a step of each.
void tokens_slabs(int d, int f, int& slab, int& slabs) {
  constexpr int unit = 32 * kTokenWaves;
  const int64_t groups = cdiv(d, 128), units = cdiv(f, unit);
  const int64_t want = cdiv(512, groups) < units ? cdiv(512, groups) : units;
  slab = (int)cdiv(units, want) * unit;
  slabs = (int)cdiv(f, slab);
}

template <typename T, int ACT>
void tokens_back_go(const TokensBack& a, hipStream_t s) {
  const dim3 grid((unsigned)cdiv(a.c.d, 128), (unsigned)a.slabs), block(64 * kTokenWaves);
  if (a.c.T <= 16) hipLaunchKernelGGL((k_glu_tokens_dx<T, ACT, 1>), grid, block, 0, s, a);
  else if constexpr (sizeof(T) == 2) hipLaunchKernelGGL((k_glu_tokens_dx<T, ACT, 2>), grid, block, 0, s, a);
  if (a.slabs > 1)
    hipLaunchKernelGGL(k_glu_tokens_join<T>, dim3((unsigned)cdiv(a.c.T * a.c.d, 256)), dim3(256), 0, s, a.part, a.slabs, a.c.T,
                       a.c.d, static_cast<T*>(a.c.dx), a.c.lddx);
}
template <typename T>
void tokens_back_act(const TokensBack& a, hipStream_t s) {
  switch (a.c.act) {
    case GIFT_ACT_SILU: return tokens_back_go<T, GIFT_ACT_SILU>(a, s);
    case GIFT_ACT_GELU: return tokens_back_go<T, GIFT_ACT_GELU>(a, s);
    case GIFT_ACT_GELU_TANH: return tokens_back_go<T, GIFT_ACT_GELU_TANH>(a, s);
    case GIFT_ACT_RELU: return tokens_back_go<T, GIFT_ACT_RELU>(a, s);
    default: return tokens_back_go<T, GIFT_ACT_SIGMOID>(a, s);
  }
}

}  // namespace

size_t glu_tokens_backward_workspace(int64_t T, int d, int f) {
  int slab, slabs;
  tokens_slabs(d, f, slab, slabs);
  return slabs > 1 ? align256((size_t)slabs * (size_t)T * (size_t)d * 4) : 0;
}

hipError_t launch_glu_tokens_backward(const GluGradCall& c, const DropArgs& drop, hipStream_t s) {
  TokensBack a{};
  a.c = c;
  a.drop = drop;
  a.part = static_cast<float*>(c.work);
  tokens_slabs(c.d, c.f, a.slab, a.slabs);
  if (c.dtype == GIFT_BF16) tokens_back_act<Bf16>(a, s);
  else if (c.dtype == GIFT_FP16) tokens_back_act<Fp16>(a, s);
  else tokens_back_act<float>(a, s);
  return hipGetLastError();
}

}  // namespace gift
