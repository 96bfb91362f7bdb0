// Weight gradient from an 8-bit activation checkpoint:
//   W[i][j] (+)= alpha sum_t delta[t][i] a[t][j],
// delta [T][m] the output gradients, a [T][d] the values a checkpoint stands
// for, W fp32 [m][ldw]: the gradient that the codec encodes.
//
// GIFT 阅读笔记, §前置知识 Eq. (4) and §核心想法: W_g = delta^T a of a linear
// layer, averaged over the tokens (alpha = 1 / T).
#include <type_traits>

#include "act8.hpp"
#include "wgrad_levels.hpp"

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
  float* part;             // segments of tiles split over workgroups
  int nst;                 // token stages of a tile
  int nbm, nbn;            // output tiles down and across
  int unit;                // stages of a unit: tiles are split at whole units
};

__device__ __forceinline__ float elem_f32(const float* p) { return *p; }
__device__ __forceinline__ float elem_f32(const Bf16* p) { return __uint_as_float((uint32_t)p->v << 16); }
__device__ __forceinline__ float elem_f32(const Fp16* p) { return (float)__builtin_bit_cast(_Float16, p->v); }

// ---------------------------------------------------------------------------
// Matrix-core form.  One workgroup (4 waves, 2 x 2) per output tile of 64 MT x
// 64 NT, KT tokens a stage.
//  * Products are v_mfma_f32_32x32x16_bf16.  A checkpoint value is exact in
//    bf16; delta enters as P bf16 planes whose sum is delta: bf16 itself, fp16
//    (11 bits) as two, fp32 (24 bits) as three, each the leading 8 bits of
//    what the planes before it leave (truncation: no plane overflows, the
//    remainders are exact).  A plane's last bit is 2^-133 at least: an fp32
//    value below 2^-110 loses its bits under that.  Products are exact in
//    fp32, sums are fp32.
//  * The operands want 8 consecutive tokens of a column per lane; memory has
//    tokens in rows.  A thread loads 8 tokens x CA (CB) columns into registers,
//    converts the codes (v_cvt_scalef32_pk_bf16: two columns of one token
//    share their scale), transposes pairs of tokens with v_perm and writes one
//    16-byte operand vector per column and plane: the reads in front of the
//    products are then 16-byte LDS reads at full rate.  Every element is
//    converted once per workgroup.
//  * LDS holds [plane][token group of 8][column] operand vectors; vector c of 8
//    columns sits at c ^ (column / 8 % 8), which keeps the writes (columns CA
//    apart) and the reads (32 adjacent columns) free of bank conflicts.
//  * Two stages of LDS.  While stage s multiplies, stage s + 1 goes from
//    registers to the other buffer and stage s + 2 from memory to registers;
//    one barrier a stage, before the last 16 tokens' products, under which the
//    first operands of the next stage are read.  The pieces of this work are
//    placed between the products at compile time.
//  * Tokens past T read as zero on both sides (buffer bounds; exponents by a
//    mask, they may hold anything).  A column chunk that crosses m is read
//    shifted, ending at m - 1, and its outputs stored accordingly.
// Measured at 1536 x 6144, 16384 tokens, bf16 delta: 283-298 us, 1.06 PFLOP/s (a
// library product of the same shape on bf16 operands already converted: 380
// us as token-major operands, 306 with tokens contiguous).  A stage of 64
// tokens of a 256 x 256 tile takes about 2870 clocks: 2048 of them are the
// products, the rest is their operands' issue (230 vector instructions, 48
// LDS and 17 memory accesses a wave) and the wait at the barrier.  With 256
// compute units of random data the clock falls to 1.96 GHz.
// ---------------------------------------------------------------------------
typedef __bf16 wbf16x8 __attribute__((ext_vector_type(8)));
typedef float wf32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t wu32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t wu32x2 __attribute__((ext_vector_type(2)));

constexpr int kWgradGroups = 256;   // workgroups that share the tiles: the compute units of an MI355X
constexpr int kWOOB = (int)0x80000000u;

template <typename TD>
constexpr int kPlanes = 1;
template <>
constexpr int kPlanes<Fp16> = 2;
template <>
constexpr int kPlanes<float> = 3;

// Tile of index idx: panels of 8 tile rows, walked down first, so that the
// workgroups of one die (consecutive indices) share columns of both operands.
__device__ __forceinline__ void wgrad_tile(int idx, int nbm, int nbn, int& ti, int& tj) {
  const int panel = idx / (8 * nbn);
  const int h = nbm - 8 * panel < 8 ? nbm - 8 * panel : 8;
  const int r = idx - panel * 8 * nbn;
  ti = panel * 8 + r % h;
  tj = r / h;
}

// Work between the products.  A wave issues in order and is alone on its
// SIMD: a product starts late when what is issued in front of it takes longer
// than the product before (32 clocks).  So the work is cut into small items
// and a slot, what follows one product, takes items up to `cap` clocks, the
// least that places all conversions in front of the barrier.  Measured: a
// 16-byte LDS write holds the issue for 20 clocks, other instructions 4.
//   items 0 .. kA - 1: column c of A, kParts steps and P writes
//   .. kCols - 1: scales of 4 + 4 tokens, then for each pair of B columns
//   four steps of two tokens and two writes
//   .. kItems - 1: 8 A and 9 B loads, one every few of all N products (in a
//   burst they fill the memory pipe's queue and stop the wave), each after
//   the steps that empty its registers
// After product n come the items order[begin[n]] .. order[begin[n + 1] - 1].
template <int CA, int CB, int P, int NB, int N, int KS, int READS>
struct WSched {
  static constexpr int kParts = P == 1 ? 1 : 4, kPerA = kParts + P;
  static constexpr int kA = CA * kPerA, kCols = kA + 2 + CB * 3, kItems = kCols + 17;
  int slot[kItems] = {}, begin[N + 1] = {}, order[kItems] = {}, cap = 0;
  static constexpr int cost(int k) {
    if (k < kA) return k % kPerA >= kParts ? 20 : P == 1 ? 16 : P == 2 ? 48 : 76;
    if (k < kA + 2) return 32;
    return (k - kA - 2) % 6 >= 4 ? 20 : 16;
  }
  constexpr bool place(int c) {
    int k = 0, load = 0, a_end = N, b_end = N;
    for (int n = 0; n < N; ++n) {
      int used = n % (N / KS) < READS ? 4 : 0;
      if (load < 17 && n > (load < 8 ? a_end : b_end) && n >= a_end + 1 + load * (N - a_end - 1) / 17) {
        slot[kCols + load++] = n;
        used += 8;
      }
      for (int first = 1; k < kCols && (first || used + cost(k) <= c); first = 0) {
        if (used + cost(k) > c && cost(k) <= c) break;
        used += cost(k);
        if (k == kA - 1) a_end = n;
        if (k == kCols - 1) b_end = n;
        slot[k++] = n;
      }
    }
    while (load < 17) slot[kCols + load++] = N - 1;
    return k == kCols && slot[kCols - 1] < NB - 2;   // (the last writes have time to end)
  }
  constexpr WSched() {
    for (cap = 20; !place(cap); cap += 2) {}
    int at = 0;
    for (int n = 0; n < N; ++n) {
      begin[n] = at;
      for (int k = 0; k < kItems; ++k)
        if (slot[k] == n) order[at++] = k;
    }
    begin[N] = at;
  }
};

// f(integral_constant<int, B>) ... f(integral_constant<int, E - 1>)
template <int B, int E, typename F>
__device__ __forceinline__ void static_for(F&& f) {
  if constexpr (B < E) {
    f(std::integral_constant<int, B>{});
    static_for<B + 1, E>(f);
  }
}

template <typename TD, int FMT, int MT, int NT, int KT>
struct WTile {
  static constexpr int P = kPlanes<TD>;
  static constexpr int SA = 64 * MT, SB = 64 * NT, KG = KT / 8, KS = KT / 16;
  static constexpr int CA = KT * SA / 2048, CB = KT * SB / 2048;   // columns of a thread's block
  static constexpr int NCH = 2048 / KT;                            // blocks across a tile side
  static constexpr int kBytesA = P * KG * SA * 16, kBytesB = KG * SB * 16, kStage = kBytesA + kBytesB;
  static constexpr int kLds = 2 * kStage;
  static constexpr int WA = CA * (int)sizeof(TD) / 4;              // words of a row of a block
  static constexpr int WB = CB / 4;
  static constexpr int PS = P * MT * NT;                           // products of 16 tokens
  static constexpr int NB = (KS - 1) * PS;                         // products in front of the barrier
};

// n words from a buffer at a byte offset (zero past its end).
template <int N>
__device__ __forceinline__ void buffer_words(__amdgpu_buffer_rsrc_t rs, int off, uint32_t* w) {
  if constexpr (N == 4) {
    const auto v = __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = v[i];
  } else if constexpr (N == 2) {
    const auto v = __builtin_amdgcn_raw_buffer_load_b64(rs, off, 0, 0);
    w[0] = v[0];
    w[1] = v[1];
  } else {
    w[0] = __builtin_amdgcn_raw_buffer_load_b32(rs, off, 0, 0);
  }
}

// What x leaves after its leading 8 bits (zero for an infinity; NaN stays NaN).
__device__ __forceinline__ float bf16_rest(float x) {
  const float r = x - __uint_as_float(__float_as_uint(x) & 0xFFFF0000u);
  return __builtin_fabsf(x) == __builtin_inff() ? 0.f : r;
}

// Element c (0 or 1) of a word of two fp16.
__device__ __forceinline__ float half_of(uint32_t w, int c) {
  const f16x2 h = __builtin_bit_cast(f16x2, w);
  return (float)h[c];
}

// Output row of tile row i (both from the tile's first row), -1 if it is not
// this row's to write: the chunk of ca rows that crosses the last row mi - 1
// was read shifted up to end there.
__device__ __forceinline__ int wgrad_row(int i, int ca, int mi) {
  const int cb = i & ~(ca - 1);
  if (cb + ca > mi) i += mi - ca - cb;
  return i >= cb && i < mi ? i : -1;
}

template <typename TD, int FMT, int MT, int NT, int KT>
__device__ __forceinline__ void wgrad_segment(const WgradArgs& a, char* lds, int ti, int tj, int s_a, int s_b,
                                              float* part) {
  using C = WTile<TD, FMT, MT, NT, KT>;
  constexpr int P = C::P;
  // (opaque, here and for the epilogue: what depends on the lane is computed
  // again for each piece instead of being kept in registers over all of them)
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int i0 = ti * C::SA, j0 = tj * C::SB;
  // this thread's block: 8 tokens of group kg, columns ch CA .. and ch CB ..
  const int ch = tid % C::NCH, kg = tid / C::NCH;
  const uint32_t lda = (uint32_t)(a.ldd * (int64_t)sizeof(TD)), ldb = (uint32_t)a.ldc;   // bytes
  int offa, offb, offs;   // of the block's first row
  {
    int ca = i0 + ch * C::CA;
    if (ca > a.m - C::CA) ca = a.m - C::CA;
    const int cb = j0 + ch * C::CB;
    const bool in = cb < a.nb * kActBlock;
    offa = (int)((uint32_t)(kg * 8) * lda) + ca * (int)sizeof(TD);
    offb = in ? (int)((uint32_t)(kg * 8) * ldb) + cb : kWOOB;   // (stays past the end with any row added)
    offs = in ? (kg * a.nb + cb / kActBlock) * kActGroup : kWOOB;
  }
  // LDS byte addresses of column 0 of the block; column c is at ^ (16 c)
  auto vec_addr = [](int kgrp, int col, int side) {
    return (kgrp * side + (col & ~7) + ((col ^ (col >> 3)) & 7)) * 16;
  };
  const int wra = vec_addr(kg, ch * C::CA, C::SA), wrb = vec_addr(kg, ch * C::CB, C::SB) + C::kBytesA;
  // operand reads: [tile parity]
  int rda[2], rdb[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    rda[q] = vec_addr(lane >> 5, wm * 32 * MT + 32 * q + (lane & 31), C::SA);
    rdb[q] = vec_addr(lane >> 5, wn * 32 * NT + 32 * q + (lane & 31), C::SB) + C::kBytesA;
  }

  struct Raw {
    uint32_t a[8][C::WA], b[8][C::WB], e[2];
    int rows;   // tokens of the stage
  };
  // two stages of loads in flight (one where three planes of a 256 x 256 tile leave no registers for it)
  constexpr int SETS = P == 3 && MT * NT > 4 ? 1 : 2;
  Raw raw[SETS];
  uint32_t bv[2][4];   // a pair of converted columns, 8 tokens
  float sc[8];         // scales of the tokens
  struct Rsrc {
    __amdgpu_buffer_rsrc_t a, b, s;
    int rows;   // tokens of the stage
  };
  const uint32_t wa = (uint32_t)a.m * (uint32_t)sizeof(TD), wb = (uint32_t)a.nb * kActBlock;
  // bytes of a whole stage and of the last one, which may hold fewer tokens
  const int tail = (int)(a.T - (int64_t)(a.nst - 1) * KT);
  const uint32_t za = (uint32_t)(KT - 1) * lda + wa, zat = (uint32_t)(tail - 1) * lda + wa;
  const uint32_t zb = (uint32_t)(KT - 1) * ldb + wb, zbt = (uint32_t)(tail - 1) * ldb + wb;
  const uint32_t zs = (uint32_t)C::KG * a.nb * kActGroup, zst = (uint32_t)((tail + 7) / 8) * a.nb * kActGroup;
  // buffers of the next stage to load; past s_b: no bytes, the loads give zeros
  int st_next = s_a;
  const char* pa = static_cast<const char*>(a.delta) + (int64_t)s_a * KT * lda;
  const uint8_t* pb = a.codes + (int64_t)s_a * KT * ldb;
  const uint8_t* ps = a.bscales + (int64_t)s_a * KT * a.nb;
  auto next_stage = [&]() {
    Rsrc R;
    const bool in = st_next < s_b, full = st_next < a.nst - 1;
    R.rows = full ? KT : tail;
    R.a = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(pa), (short)0, in ? (int)(full ? za : zat) : 0, 0x00020000);
    R.b = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(pb), (short)0, in ? (int)(full ? zb : zbt) : 0,
                                            0x00020000);
    R.s = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(ps), (short)0, in ? (int)(full ? zs : zst) : 0,
                                            0x00020000);
    ++st_next;
    pa += (uint64_t)KT * lda;
    pb += (uint64_t)KT * ldb;
    ps += (uint64_t)KT * (uint32_t)a.nb;
    return R;
  };
  // (one addition at each load, opaque: kept as values they would take sixteen registers)
  auto row_off = [](int off, uint32_t r) {
    int o;
    asm volatile("v_add_u32 %0, %1, %2" : "=v"(o) : "s"(r), "v"(off));
    return o;
  };
  auto load_a = [&](Raw& x, const Rsrc& R, int r) { buffer_words<C::WA>(R.a, row_off(offa, r * lda), x.a[r]); };
  auto load_b = [&](Raw& x, const Rsrc& R, int r) {
    if (r < 8) {
      buffer_words<C::WB>(R.b, row_off(offb, r * ldb), x.b[r]);
    } else {
      buffer_words<2>(R.s, offs, x.e);
      x.rows = R.rows;
    }
  };
  auto put = [&](int addr, const uint32_t* w) {
    const wu32x4 v = {w[0], w[1], w[2], w[3]};
    *reinterpret_cast<wu32x4*>(lds + addr) = v;
  };
  // column c of A: token pairs `part` (-1: all) to the planes; then the write of each plane
  uint32_t wv[P][4];
  auto conv_a = [&](Raw& raw, int c, int part) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (part >= 0 && k != part) continue;
      if constexpr (P == 1) {
        wv[0][k] = __builtin_amdgcn_perm(raw.a[2 * k + 1][c / 2], raw.a[2 * k][c / 2], c & 1 ? 0x07060302u : 0x05040100u);
      } else {
        float x, y;
        if constexpr (P == 2) {
          x = half_of(raw.a[2 * k][c / 2], c & 1);
          y = half_of(raw.a[2 * k + 1][c / 2], c & 1);
        } else {
          x = __uint_as_float(raw.a[2 * k][c]);
          y = __uint_as_float(raw.a[2 * k + 1][c]);
        }
#pragma unroll
        for (int p = 0; p < P; ++p) {
          wv[p][k] = __builtin_amdgcn_perm(__float_as_uint(y), __float_as_uint(x), 0x07060302u);
          if (p + 1 < P) {
            x = bf16_rest(x);
            y = bf16_rest(y);
          }
        }
      }
    }
  };
  auto put_a = [&](int c, int p, int base) { put(base + (wra ^ (c << 4)) + p * C::KG * C::SA * 16, wv[p]); };
  // scales of tokens 4 h .. 4 h + 3; exponents of tokens past T may hold anything: zero
  auto scale_b = [&](Raw& raw, int h) {
    uint32_t e = raw.e[h];
    if (raw.rows < KT) {
      const int n = raw.rows - kg * 8 - 4 * h;
      e &= n >= 4 ? ~0u : n <= 0 ? 0u : (1u << (8 * n)) - 1u;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) sc[4 * h + r] = act_scale((e >> (8 * r)) & 0xFFu);
  };
  // columns 2 c, 2 c + 1 of B: token pairs `part`; then the write of each
  auto conv_b = [&](Raw& raw, int c, int part) {
    uint32_t v[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int r = 2 * part + t;
      bf16x2 x;
      if constexpr (FMT == 0) x = c & 1 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(raw.b[r][c / 2], sc[r], true)
                                        : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(raw.b[r][c / 2], sc[r], false);
      else x = c & 1 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(raw.b[r][c / 2], sc[r], true)
                     : __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(raw.b[r][c / 2], sc[r], false);
      v[t] = __builtin_bit_cast(uint32_t, x);
    }
    bv[0][part] = __builtin_amdgcn_perm(v[1], v[0], 0x05040100u);
    bv[1][part] = __builtin_amdgcn_perm(v[1], v[0], 0x07060302u);
  };
  auto put_b = [&](int c, int h, int base) { put(base + (wrb ^ (c << 5) ^ (h << 4)), bv[h]); };

  wf32x16 acc[MT][NT];
#pragma unroll
  for (int x = 0; x < MT; ++x)
#pragma unroll
    for (int y = 0; y < NT; ++y)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[x][y][e] = 0.f;
  struct Frags {
    wbf16x8 a[P][MT], b[NT];
  };
  // operand read k of 16 tokens: B tiles first, then A tiles of each plane
  auto read_frag = [&](Frags& F, int base, int ks, int k) {
    if (k < NT) {
      F.b[k] = *reinterpret_cast<const wbf16x8*>(lds + base + rdb[k & 1] + (k >> 1) * 1024 + ks * 2 * C::SB * 16);
    } else if (k < NT + P * MT) {
      const int p = (k - NT) / MT, t = (k - NT) % MT;
      F.a[p][t] = *reinterpret_cast<const wbf16x8*>(lds + base + rda[t & 1] + (t >> 1) * 1024 +
                                                    (p * C::KG + ks * 2) * C::SA * 16);
    }
  };
  using S = WSched<C::CA, C::CB, P, C::NB, C::KS * C::PS, C::KS, NT + P * MT>;
  constexpr S sched{};
  static_assert(sched.begin[C::KS * C::PS] == S::kItems, "an item has no place");

  __syncthreads();   // the previous segment's waves are done with the LDS
  {
    auto load = [&](Raw& x) {
      const Rsrc R = next_stage();
#pragma unroll
      for (int r = 0; r < 8; ++r) load_a(x, R, r);
#pragma unroll
      for (int r = 0; r < 9; ++r) load_b(x, R, r);
    };
    load(raw[0]);
    if constexpr (SETS == 2) load(raw[1]);
#pragma unroll
    for (int c = 0; c < C::CA; ++c) {
      conv_a(raw[0], c, -1);
#pragma unroll
      for (int p = 0; p < P; ++p) put_a(c, p, 0);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) scale_b(raw[0], h);
#pragma unroll
    for (int c = 0; c < C::CB / 2; ++c) {
#pragma unroll
      for (int q = 0; q < 4; ++q) conv_b(raw[0], c, q);
      put_b(c, 0, 0);
      put_b(c, 1, 0);
    }
    load(raw[0]);
  }
  __syncthreads();
  Frags F[2];
#pragma unroll
  for (int k = 0; k < NT + P * MT; ++k) read_frag(F[0], 0, 0, k);
  // stage in buffer `base` (0 or kStage): its products; the next stage from
  // x to the other buffer; the one after next but one from memory to x
  auto stage = [&](Raw& x, auto BASE) {
    constexpr int base = decltype(BASE)::value, nbase = base ^ C::kStage;
    const Rsrc R = next_stage();
    static_for<0, C::KS>([&](auto KSC) {
      constexpr int ks = decltype(KSC)::value;
      constexpr bool last = ks == C::KS - 1;
      if constexpr (last) {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // this wave's part of the next stage is written
        __syncthreads();
      }
      static_for<0, C::PS>([&](auto QC) {
        constexpr int q = decltype(QC)::value, p = q / (MT * NT), xt = q / NT % MT, y = q % NT, n = ks * C::PS + q;
        acc[xt][y] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(F[ks & 1].a[p][xt], F[ks & 1].b[y], acc[xt][y], 0, 0, 0);
        read_frag(F[(ks + 1) & 1], last ? nbase : base, last ? 0 : ks + 1, q);
        static_for<sched.begin[n], sched.begin[n + 1]>([&](auto KC) {
          constexpr int k = sched.order[decltype(KC)::value];
          if constexpr (k < S::kA) {
            constexpr int c = k / S::kPerA, part = k % S::kPerA;
            if constexpr (part < S::kParts) conv_a(x, c, S::kParts == 1 ? -1 : part);
            else put_a(c, part - S::kParts, nbase);
          } else if constexpr (k < S::kA + 2) {
            scale_b(x, k - S::kA);
          } else if constexpr (k < S::kCols) {
            constexpr int c = (k - S::kA - 2) / 6, part = (k - S::kA - 2) % 6;
            if constexpr (part < 4) conv_b(x, c, part);
            else put_b(c, part - 4, nbase);
          } else if constexpr (k < S::kCols + 8) {
            load_a(x, R, k - S::kCols);
          } else {
            load_b(x, R, k - S::kCols - 8);
          }
        });
        __builtin_amdgcn_sched_barrier(0);
      });
    });
  };
  int st = s_a;
  for (; st + 1 < s_b; st += 2) {
    stage(raw[SETS - 1], std::integral_constant<int, 0>{});
    stage(raw[0], std::integral_constant<int, C::kStage>{});
  }
  if (st < s_b) stage(raw[SETS - 1], std::integral_constant<int, 0>{});

  // Register e of MFMA tile (x, y) is element (8 (e / 4) + 4 (lane / 32) + e %
  // 4, lane % 32) of the 32 x 32 outputs.
  int elane = threadIdx.x & 63;
  asm volatile("" : "+v"(elane));
  // the sums stay in the accumulator registers until their own turn
  auto hold = [](wf32x16& v) {
    if constexpr (MT * NT > 4) asm volatile("" : "+a"(v));
  };
  if (part) {
    // a piece, in the order of the registers: [wave][x][y][e / 4][lane][e % 4]
    float* p = part + (int64_t)wave * MT * NT * 1024 + elane * 4;
#pragma unroll
    for (int x = 0; x < MT; ++x)
#pragma unroll
      for (int y = 0; y < NT; ++y)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          hold(acc[x][y]);
          const float4 v = {acc[x][y][4 * e], acc[x][y][4 * e + 1], acc[x][y][4 * e + 2], acc[x][y][4 * e + 3]};
          *reinterpret_cast<float4*>(p + ((x * NT + y) * 4 + e) * 256) = v;
          __builtin_amdgcn_sched_barrier(0);
        }
    return;
  }
  const int r0 = 32 * wm * MT + 4 * (elane >> 5), c0 = 32 * wn * NT + (elane & 31);
  const int mi = a.m - i0, nj = a.d - j0;
  const float alpha = a.alpha;
  const bool add = a.accumulate != 0;
  float* out = a.W + (int64_t)i0 * a.ldw + j0 + c0;
  if (mi >= C::SA && nj >= C::SB && !add) {   // a whole tile: no checks
    float* row = out + (int64_t)r0 * a.ldw;
#pragma unroll
    for (int x = 0; x < MT; ++x)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
#pragma unroll
        for (int y = 0; y < NT; ++y) {
          hold(acc[x][y]);
          row[32 * y] = alpha * acc[x][y][e];
        }
        row += (e % 4 == 3 ? 5 : 1) * a.ldw;   // rows 0 .. 3 of every eight
        if (e == 15) row = out + (int64_t)(r0 + 32 * (x + 1)) * a.ldw;
        __builtin_amdgcn_sched_barrier(0);
      }
    return;
  }
#pragma unroll
  for (int x = 0; x < MT; ++x)
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int i = wgrad_row(r0 + 32 * x + 8 * (e / 4) + e % 4, C::CA, mi);
      float* row = out + (int64_t)i * a.ldw;
#pragma unroll
      for (int y = 0; y < NT; ++y) {
        hold(acc[x][y]);
        float v = alpha * acc[x][y][e];
        if (i >= 0 && c0 + 32 * y < nj) {
          if (add) v += row[32 * y];
          row[32 * y] = v;
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
}

// One workgroup's pieces (WLevel).  Workgroups of one die have consecutive
// numbers.  A piece that is not a whole tile goes to part at its number, and
// k_wgrad_join adds the pieces of a tile in token order: no atomics, the same
// sums every time.  (128 x 128 tiles: two workgroups fit a compute unit with
// bf16 delta, 64 KB of LDS each; with fp16 and fp32 the planes take 96 and 128
// KB and one fits, whatever the bound below allows in registers.)
template <typename TD, int FMT, int MT, int NT, int KT>
__global__ void __launch_bounds__(256, MT * NT > 4 ? 1 : 2) k_wgrad(WgradArgs a) {
  using C = WTile<TD, FMT, MT, NT, KT>;
  __shared__ __attribute__((aligned(16))) char lds[C::kLds];
  const int G = gridDim.x;
  int g = G % 8 == 0 ? (blockIdx.x & 7) * (G >> 3) + (blockIdx.x >> 3) : blockIdx.x;
  // (divisions run on the vector units: the compiler is told that the results are uniform)
  auto uniform = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
  wgrad_walk(wgrad_levels(a.nbm * a.nbn, (a.nst + a.unit - 1) / a.unit, G), g, uniform,
             [&](int tile, int from, int units, int number) {
               int ti, tj;
               wgrad_tile(tile, a.nbm, a.nbn, ti, tj);
               const int s0 = from * a.unit;
               const int s1 = s0 + units * a.unit < a.nst ? s0 + units * a.unit : a.nst;
               const bool whole = s0 == 0 && s1 == a.nst;
               wgrad_segment<TD, FMT, MT, NT, KT>(a, lds, uniform(ti), uniform(tj), s0, s1,
                                                  whole ? nullptr : a.part + (int64_t)number * C::SA * C::SB);
             });
}

// W of the split tiles from their pieces, added in token order.  Each
// workgroup takes 32 rows of one wave's part of a tile, 32 NT columns, and
// turns them from the order of the registers (see the end of wgrad_segment)
// to rows in LDS: W is written in row segments of 128 NT bytes (in the order
// of the registers, 128 bytes a row at a time: 42 us instead of 28 at 1536 x
// 6144, 101 MB of pieces).
template <int MT, int NT>
__global__ void __launch_bounds__(256) k_wgrad_join(WgradArgs a, int G, int first, int ca) {
  constexpr int SA = 64 * MT, SB = 64 * NT, PER = MT * 4, COLS = 32 * NT;   // PER: workgroups of a tile
  __shared__ float rows[32][COLS + 4];
  const int tile = first + blockIdx.x / PER, q = blockIdx.x % PER;
  const int x = q % MT, wave = q / MT;
  const int lane = threadIdx.x & 63, e = threadIdx.x >> 6;
  const float* base = a.part + (wave * MT + x) * NT * 1024 + threadIdx.x * 4;
  float4 s[NT];
#pragma unroll
  for (int y = 0; y < NT; ++y) s[y] = float4{0.f, 0.f, 0.f, 0.f};
  wgrad_pieces(wgrad_levels(a.nbm * a.nbn, (a.nst + a.unit - 1) / a.unit, G), tile, [&](int number, int stride, int count) {
    constexpr int AT = 16 / NT;   // pieces at once: sixteen loads in flight
    for (int c = 0; c < count; c += AT) {
      float4 v[AT][NT];
#pragma unroll
      for (int k = 0; k < AT; ++k)
#pragma unroll
        for (int y = 0; y < NT; ++y) {
          v[k][y] = float4{0.f, 0.f, 0.f, 0.f};
          if (c + k < count)
            v[k][y] = *reinterpret_cast<const float4*>(base + ((int64_t)number + (int64_t)(c + k) * stride) * SA * SB + y * 1024);
        }
#pragma unroll
      for (int k = 0; k < AT; ++k)
#pragma unroll
        for (int y = 0; y < NT; ++y) {
          s[y].x += v[k][y].x;
          s[y].y += v[k][y].y;
          s[y].z += v[k][y].z;
          s[y].w += v[k][y].w;
        }
    }
  });
#pragma unroll
  for (int y = 0; y < NT; ++y) {
    const float v[4] = {s[y].x, s[y].y, s[y].z, s[y].w};
#pragma unroll
    for (int r = 0; r < 4; ++r) rows[8 * e + 4 * (lane >> 5) + r][32 * y + (lane & 31)] = v[r];
  }
  __syncthreads();
  int ti, tj;
  wgrad_tile(tile, a.nbm, a.nbn, ti, tj);
#pragma unroll
  for (int k = 0; k < NT; ++k) {
    const int f = k * 256 + threadIdx.x, r = f / (COLS / 4), c = f % (COLS / 4) * 4;
    const int i = wgrad_row(32 * ((wave >> 1) * MT + x) + r, ca, a.m - ti * SA);
    const int j = tj * SB + (wave & 1) * COLS + c;
    if (i < 0) continue;
    float* w = a.W + (int64_t)(ti * SA + i) * a.ldw + j;
#pragma unroll
    for (int l = 0; l < 4; ++l)
      if (j + l < a.d) {
        const float o = a.alpha * rows[r][c + l];
        w[l] = a.accumulate ? w[l] + o : o;
      }
  }
}

// Vector-unit form, for what the matrix-core form leaves out (see wgrad_plan):
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


int64_t wgrad_grid(int m, int d) { return cdiv(m, 64) * cdiv(d, 64); }

namespace {

struct WgradPlan {
  int variant;         // 0: vector units, 1: 256 x 256 tiles, 2: 128 x 128
  int kt, side, nbm, nbn, nst, unit, grid;
  int first, split;    // first split tile, split tiles
  size_t bytes;
};

// A plan with tiles of `side`, split at multiples of `units` x 64 tokens (0:
// not split), and what it is expected to take (us): the stages of a
// workgroup, and for split tiles the launch that joins them and their pieces
// written and read.  Per 64 tokens a workgroup takes (measured; bf16, fp16,
// fp32 delta):
//   256 x 256  1.6, 3.8, 5.4      one workgroup a compute unit
//   128 x 128  1.3, 1.3, 1.8      bf16: two workgroups a compute unit, 0.9 where there are no more than units;
//                                 fp16, fp32: one (see k_wgrad)
// and 14 or 2.5 for each whole tile that it writes (128 tokens, 1536 x 6144: 33
// against 22 us with the larger and the smaller tiles).
double wgrad_try(WgradPlan& p, int variant, int units, int64_t T, int m, int d, int dtype) {
  static const double kStage[2][3] = {{1.6, 3.8, 5.4}, {1.3, 1.3, 1.8}};
  const int t = dtype == GIFT_BF16 ? 0 : dtype == GIFT_FP16 ? 1 : 2;
  p.variant = variant;
  p.side = variant == 1 ? 256 : 128;
  p.kt = variant == 1 && dtype != GIFT_BF16 ? 32 : 64;
  p.nbm = (int)cdiv(m, p.side);
  p.nbn = (int)cdiv(d, p.side);
  p.nst = (int)cdiv(T, p.kt);
  p.grid = variant == 2 && dtype == GIFT_BF16 ? 2 * kWgradGroups : kWgradGroups;
  p.unit = units ? units * 64 / p.kt : p.nst;
  const WLevel v = wgrad_levels(p.nbm * p.nbn, (int)cdiv(p.nst, p.unit), p.grid);
  const double stages = (double)v.C * p.unit * p.kt / 64;
  const WSplit w = wgrad_split(v);
  p.first = w.first;
  p.split = w.tiles;
  p.bytes = (size_t)w.pieces * p.side * p.side * 4;
  const bool alone = (int64_t)p.nbm * p.nbn * cdiv(p.nst, p.unit) <= (int64_t)kWgradGroups * v.C;
  const double stage = variant == 2 && t == 0 && alone ? 0.9 : kStage[variant - 1][t];
  const double whole = (double)(v.C * (int64_t)p.unit / p.nst) * (variant == 1 ? 14.0 : 2.5);
  return stages * stage + whole + (p.split ? 5.0 + 2.0 * (double)p.bytes / 4.5e6 : 0.0);
}

WgradPlan wgrad_plan(int64_t T, int m, int d, int dtype, int64_t ldd, int64_t ldc) {
  WgradPlan best{};
  const int size = dtype == GIFT_FP32 ? 4 : 2;
  // The matrix-core form reads chunks of eight columns of delta, its buffer
  // offsets within a stage are 32 bits, and so are its counts of tiles and
  // stages; what is beyond runs on the vector units.
  if (m < 8 || T == 0 || ldd >= ((int64_t)1 << 31) / (64 * size) || ldc >= ((int64_t)1 << 31) / 64) return best;
  // (an output beyond a launch's reach has no plan: its tiles alone can pass 32 bits)
  if (wgrad_grid(m, d) > kMaxGrid) return best;
  if (T >= (int64_t)1 << 34 || cdiv(m, 128) * cdiv(d, 128) * cdiv(T, 64) >= (int64_t)1 << 38) return best;
  double least = 0;
  for (int variant = 1; variant <= 2; ++variant)
    for (int units = 0; units <= 2; ++units) {
      WgradPlan p{};
      const double t = wgrad_try(p, variant, units, T, m, d, dtype);
      if (best.variant == 0 || t < least) {
        best = p;
        least = t;
      }
    }
  return best;
}

template <typename TD, int FMT, int MT, int KT>
void wgrad_go(const WgradArgs& a, const WgradPlan& p, hipStream_t s) {
  hipLaunchKernelGGL((k_wgrad<TD, FMT, MT, MT, KT>), dim3((unsigned)p.grid), dim3(256), 0, s, a);
  if (p.split)
    hipLaunchKernelGGL((k_wgrad_join<MT, MT>), dim3((unsigned)(p.split * MT * 4)), dim3(256), 0, s, a, p.grid,
                       p.first, KT * MT / 32);
}

template <typename TD, int KT>
void wgrad_t(const WgradArgs& a, const WgradPlan& p, hipStream_t s) {
  if (p.variant == 1) {
    if (a.fmt == GIFT_E4M3) wgrad_go<TD, 0, 4, KT>(a, p, s);
    else wgrad_go<TD, 1, 4, KT>(a, p, s);
  } else {
    if (a.fmt == GIFT_E4M3) wgrad_go<TD, 0, 2, 64>(a, p, s);
    else wgrad_go<TD, 1, 2, 64>(a, p, s);
  }
}

}  // namespace

size_t wgrad_workspace(int64_t T, int m, int d, int dtype) {
  return align256(wgrad_plan(T, m, d, dtype, 0, 0).bytes) + 256;
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
  const WgradPlan p = wgrad_plan(c.T, c.m, c.d, c.dtype, c.ldd, c.ckpt->ldc);
  if (p.variant == 0) {
    const dim3 grid((unsigned)wgrad_grid(c.m, c.d));
    if (c.dtype == GIFT_BF16) hipLaunchKernelGGL(k_wgrad_valu<Bf16>, grid, dim3(256), 0, s, a);
    else if (c.dtype == GIFT_FP16) hipLaunchKernelGGL(k_wgrad_valu<Fp16>, grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL(k_wgrad_valu<float>, grid, dim3(256), 0, s, a);
    return hipGetLastError();
  }
  a.part = c.work;
  a.nst = p.nst;
  a.nbm = p.nbm;
  a.nbn = p.nbn;
  a.unit = p.unit;
  if (c.dtype == GIFT_BF16) wgrad_t<Bf16, 64>(a, p, s);
  else if (c.dtype == GIFT_FP16) wgrad_t<Fp16, 32>(a, p, s);
  else wgrad_t<float, 32>(a, p, s);
  return hipGetLastError();
}

}  // namespace gift
