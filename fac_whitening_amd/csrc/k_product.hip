// The matrix products of the gated feed-forward block and of the weight
// gradient from a whole activation:
//   out[j][i] = sum_k A[i][k] B[j][k],  i the contiguous index of the output.
//   kEpiGlu    A = Wg and Wu, B = x: z and u side by side, out = D(act(z) u)
//   kEpiStore  A = Wg^T then Wu^T, B = dgate then dup: dx
//   kEpiGrad   A = x^T, B = delta^T: the weight gradient
// On v_mfma_f32_32x32x16 with fp32 sums.  bf16 and fp16 operands multiply
// exactly.  An fp32 operand is three bf16 planes (split_planes) and the long
// axis six segments, the products of planes (0, 2), (1, 1), (2, 0), (0, 1), (1,
// 0), (0, 0): what is left out is below 2^-24 of |A| |B| (and of operands below
// 2^-110 what lies under 2^-133), and the small products are added before the
// large ones.
//
// One workgroup (4 waves, 2 x 2) makes a tile of 256 x 256, or 128 x 128, in
// stages of 64 of the long axis; of kEpiGlu half of A's rows are the gate's,
// half the up projection's, in turns of 32, so that a lane holds both sums of
// an output.
//  * Direct operands (rows of k) go from memory to LDS without registers, 16
//    bytes a lane.  Transposing ones (rows of i or j: the weights in dx, both
//    sides of the weight gradient) are loaded as blocks of 8 x 8, turned by
//    v_perm and written as 16-byte operand vectors between the products; two
//    stages of them are in flight in registers.  (The LDS's own transposing
//    reads run at 48 bytes a clock; these products need 64.)  The lanes of a
//    load are consecutive in memory: with the lanes along k instead, the address
//    unit took 47 clocks a load in place of 16, and 8192^3 with both sides
//    transposing 1063 us in place of 936.
//  * Two stages in LDS, swizzled (chunk_slot; no bank conflicts).  A stage's
//    products are 64 of 32 clocks a wave; the operands of the next 16 are read
//    under them.  One barrier a stage, in front of the last 16: behind it the
//    stage's buffer is free for the stage after next.  The loads run on
//    through the workgroup's tiles: the next tile's first stages arrive under
//    the epilogue.  Tiles of 128: two workgroups a compute unit, or one with four
//    stages in LDS, whose loads have three stages' time to arrive (256 tokens,
//    1536 x 6144: 23 us in place of 32).
//  * A tile's outputs are turned in 4 KB of LDS a wave and written as rows of 128
//    bytes, one block read back while the next one's activation is computed;
//    outputs larger than the L2 caches past them (16384 x 6144, three outputs:
//    775 -> 727 us; the order of the blocks 727 -> 657).
//  * Tiles are shared among the workgroups in levels (wgrad_levels.hpp), pieces
//    of split tiles joined in the order of the long axis by a second launch.
// Measured (bf16): 8192^3 1.28 PFLOP/s direct, 1.20 transposing (a library
// product 1.37, the clock then bound by power); 16384 tokens, 1536 x 6144:
// forward 568 to 576 us, with dropout 31 more, with both products kept 69 more,
// both 657 to 677 (machines differ), dx 530, weight gradient 291.  Of dx, the
// matrix units are busy 59 % of 1.0 million clocks at 1.92 GHz; waves wait for
// counters and barriers 19 % of the time.  An earlier barrier with all operands of
// a stage read at its start, and reads spread over all products, took the same
// time.
#include "product.hpp"

namespace gift {

// Output tile idx: panels of 8 tiles along i, walked along them first, so
// that the workgroups of one die (consecutive indices) share both operands.
__device__ __forceinline__ void product_tile(int idx, int nbm, int nbn, int& ti, int& tj) {
  const int panel = idx / (8 * nbn);
  const int h = nbm - 8 * panel < 8 ? nbm - 8 * panel : 8;
  const int r = idx - panel * 8 * nbn;
  ti = panel * 8 + r % h;
  tj = r / h;
}

// The kernel's arguments where they lie in memory.  An address that the
// compiler cannot follow keeps it from holding what only a piece's start and
// end need in registers through the products.
typedef const __attribute__((address_space(4))) ProdArgs ConstArgs;
typedef const __attribute__((address_space(4))) ProdOut ConstOut;
struct KernelArgs {
  ProdArgs a;
  ProdOut o;
};
__device__ __forceinline__ const __attribute__((address_space(4))) KernelArgs* kernel_args() {
  auto p = (const __attribute__((address_space(4))) KernelArgs*)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return p;
}

__device__ __forceinline__ DropArgs drop_args_of(ConstOut& o) {
  DropArgs d;
  d.thr = o.drop.thr;
  d.scale = o.drop.scale;
  d.k0 = o.drop.k0;
  d.k1 = o.drop.k1;
  d.offset = o.drop.offset;
  d.d_offset = o.drop.d_offset;
  d.on = o.drop.on;
  return d;
}

// Piece p of workgroup g: tile, stages, number.
struct Piece {
  int tile, s0, s1, number;
};
__device__ __forceinline__ bool product_piece(const ConstArgs* a, int g, int p, Piece& out) {
  const int total = a->nst * a->nseg, unit = a->unit;
  int from, units;
  const WLevel v = wgrad_levels(a->nbm * a->nbn, (total + unit - 1) / unit, gridDim.x);
  if (!wgrad_piece(v, g, p, out.tile, from, units, out.number)) return false;
  out.s0 = from * unit;
  out.s1 = out.s0 + units * unit < total ? out.s0 + units * unit : total;
  return true;
}

__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ uint64_t uni64(uint64_t v) {
  return (uint64_t)(uint32_t)uni((int)(uint32_t)v) | (uint64_t)(uint32_t)uni((int)(uint32_t)(v >> 32)) << 32;
}

// A stage is 64 elements of the long axis, 128 bytes a row.
template <int MT, int NT, int NBUF>
struct PTile {
  static constexpr int SA = 64 * MT, SB = 64 * NT;             // rows of a tile's operands
  static constexpr int kBytesA = SA * 128, kBytesB = SB * 128, kStage = kBytesA + kBytesB;
  static constexpr int kTurn = 4096;                           // a wave's LDS for outputs
  static constexpr int kLds = NBUF * kStage + 4 * kTurn;
  static constexpr int LA = kBytesA / 4096, LB = kBytesB / 4096;   // direct loads of a wave a stage
  static constexpr int PS = MT * NT;                           // products of a step of 16
};

// Slot of 16-byte chunk c of row r of a stage (128 bytes).  A 16-byte LDS
// access of a wave runs in four rounds of 16 lanes, 0-3, 12-15, 20-23, 24-27 the
// first: operand reads (a row a lane) find the 16 rows of a round in 16
// different slots of 256 bytes, and the writes of a transposing side (rows 8
// apart) each slot twice, the least for rows of one parity.
__device__ __forceinline__ int chunk_slot(int r, int c) {
  return c ^ ((r >> 1) & 7) ^ ((r >> 4) & 1) ^ ((r >> 4) & 2);
}

template <typename TO>
struct OutVec {
  static constexpr int N = 16 / (int)sizeof(TO);   // elements of 16 bytes
};

// Four consecutive values, rounded.
template <typename TO>
__device__ __forceinline__ void pack4(const float* v, uint32_t* w) {
  if constexpr (std::is_same<TO, float>::value) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(v[i]);
  } else if constexpr (std::is_same<TO, Bf16>::value) {
    w[0] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{v[0], v[1]}), bf16x2));
    w[1] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{v[2], v[3]}), bf16x2));
  } else {
    w[0] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{v[0], v[1]}), f16x2));
    w[1] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{v[2], v[3]}), f16x2));
  }
}

// 16 bytes of elements to p, n of them valid.
template <typename TO>
__device__ __forceinline__ void store16(TO* p, const uint32_t* w, int n, bool stream) {
  constexpr int N = OutVec<TO>::N;
  if (n >= N) {
    store_words<4>(p, w, stream);
  } else {
#pragma unroll
    for (int i = 0; i < N - 1; ++i)
      if (i < n) {
        if constexpr (sizeof(TO) == 2) {
          const uint16_t e = (uint16_t)(w[i / 2] >> (16 * (i % 2)));
          __builtin_memcpy(p + i, &e, 2);
        } else {
          __builtin_memcpy(p + i, &w[i], 4);
        }
      }
  }
}

// E: operand type, TO: output type, AX, BX: transposing sides, NBUF: stages in LDS, WGS: workgroups a compute unit.
template <typename E, typename TO, int EPI, int ACT, int MT, int NT, bool AX, bool BX, int NBUF, int WGS>
__global__ void __launch_bounds__(256, WGS) k_product(KernelArgs args) {
  const auto* const ka = &args.a;
  using C = PTile<MT, NT, NBUF>;
  using Fr = Frag8<E>;
  constexpr bool GLU = EPI == kEpiGlu;
  constexpr int kLoadsA = AX ? 0 : C::LA, kLoadsB = BX ? 0 : C::LB;
  __shared__ __attribute__((aligned(1024))) char lds[C::kLds];
  const uint32_t lds0 = (uint32_t)(uintptr_t)(p_lds_void*)lds;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = uni(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int G = gridDim.x;
  const int g = G % 8 == 0 ? (blockIdx.x & 7) * (G >> 3) + (blockIdx.x >> 3) : blockIdx.x;
  const int nst = ka->nst, total = nst * ka->nseg;   // stages of a segment, of a tile

  // ---- loads ----
  const uint32_t lda2 = (uint32_t)ka->lda * 2, ldu2 = (uint32_t)ka->lda2 * 2, ldb2 = (uint32_t)ka->ldb * 2;
  // direct: load q of a wave fills rows 32 q + 8 wave .. + 7 of a side: this lane's row and, for even q, its chunk; for
  // odd q it is the chunk ^ 2
  const int drow = 8 * wave + (lane >> 3);
  const int dchunk = chunk_slot(drow, lane & 7);     // (its own inverse)
  // transposing: blocks of 8 (of the long axis, group tk) x 8 (of the outputs, group tc); a thread has one of each
  // transposing side, or, of sides of 128, one: waves 0 and 1 hold A's, 2 and 3 B's
  constexpr bool X = AX || BX;
  constexpr int NS = !X ? 0 : MT == 4 ? AX + BX : 1;
  const int tk = (lane >> 3) & 7, tc = (lane & 7) + 8 * (MT == 4 ? wave : wave & 1);
  auto side_of = [&](int slot) { return MT == 4 ? (AX ? slot : 1) : wave >> 1; };
  const bool idle = MT != 4 && X && !(wave >> 1 ? BX : AX);   // (a wave without a block: its loads are empty)
  int offa, offu = 0, offb;                          // of this lane, from the tile's first row
  if constexpr (!AX) {
    offa = drow * lda2 + dchunk * 16;
    if constexpr (GLU) offu = drow * ldu2 + dchunk * 16;
  }
  if constexpr (!BX) offb = drow * ldb2 + dchunk * 16;

  struct Desc {
    pi32x4 a, u, b;
    int mask[2];       // direct loads, even and odd: past the long axis's end
    pi32x4 x[NS ? NS : 1];
    int offx[NS ? NS : 1];   // transposing: this lane's offset (its columns may be past the end)
  };
  // bytes of a transposing operand's stage, and of a segment's last one
  auto clamp31 = [](int64_t v) { return (uint32_t)(v > 0x7FFFFFFF ? 0x7FFFFFFF : v); };
  const int tail = (int)(ka->K - (int64_t)(nst - 1) * 64);
  int lpiece = 0, left = 0, real = 0, lseg = 0, lk = 0;   // stages left, of them not empty
  uint64_t pa = 0, pu = 0, pb = 0;
  uint32_t za = 0, zu = 0, zb = 0;
  int xoff[NS ? NS : 1];
  uint32_t ldx2[NS ? NS : 1];
  int64_t xbytes[NS ? NS : 1];   // of a row
  if constexpr (X) {
#pragma unroll
    for (int n = 0; n < NS; ++n) {
      ldx2[n] = side_of(n) ? ldb2 : lda2;
      xbytes[n] = 2 * (side_of(n) ? ka->bcols : ka->acols);
    }
  }
  int li = 0, lj = 0;
  auto next_stage = [&]() {
    Desc D;
    bool fresh = lk == 0;
    if (left == 0) {
      Piece w;
      left = 1 << 30;                    // (after the last piece: empty stages)
      real = 0;
      ConstArgs* q = &kernel_args()->a;
      if (product_piece(q, g, lpiece, w)) {
        ++lpiece;
        int ti, tj;
        product_tile(w.tile, q->nbm, q->nbn, ti, tj);
        li = uni(ti);
        lj = uni(tj);
        const int s0 = uni(w.s0);
        real = uni(w.s1) - s0;
        left = X ? (real + 1) & ~1 : real;   // (transposing: stages come in pairs; the last may be empty)
        lseg = uni(s0 / nst);
        lk = s0 - lseg * nst;
        fresh = true;
        if constexpr (X) {
#pragma unroll
          for (int n = 0; n < NS; ++n) {
            const int sd = side_of(n);
            const int64_t c = (sd ? (int64_t)lj * C::SB : (int64_t)li * C::SA) + tc * 8;
            xoff[n] = !idle && c < (sd ? q->N : (int64_t)q->M) ? (int)((uint32_t)(tk * 8) * ldx2[n]) + (int)c * 2 : kPastEnd;
          }
        }
      }
    }
    if (fresh) {
      ConstArgs* q = &kernel_args()->a;
      const int sg = lseg < q->nseg ? lseg : 0;
      const int64_t K8 = (q->K + 7) & ~(int64_t)7;   // (rows are padded with zeros to whole chunks)
      const int i0 = li * (GLU ? C::SA / 2 : C::SA);
      const int64_t j0 = (int64_t)lj * C::SB;
      pa = q->a[sg] + (AX ? (uint64_t)lk * 64 * lda2 : (uint64_t)i0 * lda2 + (uint64_t)lk * 128);
      if constexpr (GLU) pu = q->a2[sg] + (uint64_t)i0 * ldu2 + (uint64_t)lk * 128;
      pb = q->b[sg] + (BX ? (uint64_t)lk * 64 * ldb2 : (uint64_t)j0 * ldb2 + (uint64_t)lk * 128);
      if constexpr (!AX) za = clamp31((int64_t)(q->M - 1 - i0) * lda2 + 2 * K8);
      if constexpr (GLU) zu = clamp31((int64_t)(q->M - 1 - i0) * ldu2 + 2 * K8);
      if constexpr (!BX) zb = clamp31((q->N - 1 - j0) * (int64_t)ldb2 + 2 * K8);
    }
    const bool in = real > 0, last = lk == nst - 1;
    const int rows = last ? tail : 64;
    if constexpr (!AX) D.a = buffer_of(pa, in ? za : 0);
    if constexpr (!BX) D.b = buffer_of(pb, in ? zb : 0);
    if constexpr (GLU) D.u = buffer_of(pu, in ? zu : 0);
    if constexpr (X) {
#pragma unroll
      for (int n = 0; n < NS; ++n) {
        const int sd = side_of(n);
        D.x[n] = buffer_of(sd ? pb : pa, !in ? 0 : clamp31((int64_t)(rows - 1) * ldx2[n] + xbytes[n]));
        D.offx[n] = xoff[n];
      }
    }
    if constexpr (!AX || !BX) {
      D.mask[0] = dchunk * 8 < rows ? 0 : kPastEnd;
      D.mask[1] = (dchunk ^ 2) * 8 < rows ? 0 : kPastEnd;
    }
    pa += AX ? (uint64_t)lda2 * 64 : 128;
    if constexpr (GLU) pu += 128;
    pb += BX ? (uint64_t)ldb2 * 64 : 128;
    --left;
    --real;
    lk = last ? 0 : lk + 1;
    lseg += last;
    return D;
  };
  // (one addition at each load, opaque: kept as values they would take a register each)
  auto row_off = [](int off, uint32_t r) {
    int v;
    asm volatile("v_add_u32 %0, %1, %2" : "=v"(v) : "s"(r), "v"(off));
    return v;
  };
  // direct load q of A (q < kLoadsA) or B into the buffer at byte `base` (row block p of 32: offset + 32 p rows, and for
  // odd p the chunk ^ 2, which is offset ^ 32: the chunks of a row are not reached by carries, rows being 16-byte
  // aligned only, so the difference is added)
  const int odd = (dchunk ^ 2) * 16 - dchunk * 16;
  auto place = [&](int off, int p, uint32_t ld2, const Desc& D) {
    return (p & 1 ? row_off(off + odd, (uint32_t)(p * 32) * ld2) : row_off(off, (uint32_t)(p * 32) * ld2)) | D.mask[p & 1];
  };
  auto direct = [&](const Desc& D, int base, int q) {
    if (q < kLoadsA) {
      const uint32_t to = lds0 + base + (4 * q + wave) * 1024;
      if constexpr (GLU) {
        // row blocks of gate and up in turn: block q is rows 32 (q / 2) of one of them
        const int off = (q & 1 ? offu : offa) + (q & 1 ? odd : 0);
        dma16(q & 1 ? D.u : D.a, to, row_off(off, (uint32_t)((q >> 1) * 32) * (q & 1 ? ldu2 : lda2)) | D.mask[q & 1]);
      } else {
        dma16(D.a, to, place(offa, q, lda2, D));
      }
    } else {
      const int p = q - kLoadsA;
      dma16(D.b, lds0 + base + C::kBytesA + (4 * p + wave) * 1024, place(offb, p, ldb2, D));
    }
  };
  // transposing: element r of the long axis, 8 columns
  struct Raw {
    uint32_t v[NS ? NS : 1][8][4];
  };
  Raw raw[X ? 2 : 1];
  auto load_x = [&](Raw& x, const Desc& D, int n, int r) {
    const uint64_t at = (uint64_t)(uint32_t)D.x[n][0] | (uint64_t)(uint32_t)D.x[n][1] << 32;
    const __amdgpu_buffer_rsrc_t rs =
        __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(at), (short)0, D.x[n][2], 0x00020000);
    const auto v = __builtin_amdgcn_raw_buffer_load_b128(rs, row_off(D.offx[n], (uint32_t)r * ldx2[n]), 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) x.v[n][r][i] = v[i];
  };
  // column c of a block: its 8 elements side by side, to row 8 tc + c, chunk tk
  uint32_t wv[4];
  auto turn = [&](const Raw& x, int n, int c) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      wv[k] = __builtin_amdgcn_perm(x.v[n][2 * k + 1][c / 2], x.v[n][2 * k][c / 2], c & 1 ? 0x07060302u : 0x05040100u);
  };
  // (of row 8 tc + c the swizzle is that of 8 tc ^ c / 2)
  const int wr = 8 * tc * 128 + chunk_slot(8 * tc, tk) * 16;
  auto put = [&](int n, int c, int base) {
    const pu32x4 v = {wv[0], wv[1], wv[2], wv[3]};
    if (!idle)
      *reinterpret_cast<pu32x4*>(lds + base + side_of(n) * C::kBytesA + (wr ^ ((c >> 1) << 4)) + c * 128) = v;
  };

  // ---- products ----
  int rda[4], rdb[4];
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) {
    const int s = chunk_slot(lane & 31, 2 * ks + (lane >> 5)) * 16;
    rda[ks] = (wm * 32 * MT + (lane & 31)) * 128 + s;
    rdb[ks] = C::kBytesA + (wn * 32 * NT + (lane & 31)) * 128 + s;
  }
  struct Frags {
    Fr a[MT], b[NT];
  } F[2];
  auto read = [&](Frags& f, int base, int ks, int k) {
    // (the swizzle of an odd block of 32 rows is that of an even one ^ 2: of step ks ^ 1)
    if (k < NT) f.b[k] = *reinterpret_cast<const Fr*>(lds + base + rdb[ks ^ (k & 1)] + k * 4096);
    else if (k < NT + MT) f.a[k - NT] = *reinterpret_cast<const Fr*>(lds + base + rda[ks ^ (k & 1)] + (k - NT) * 4096);
  };
  pf32x16 acc[MT][NT];

  // ---- prologue ----
  Desc D2;
  if constexpr (!X) {
    static_assert((NBUF - 1) * (kLoadsA + kLoadsB) < 64, "vmcnt");
#pragma unroll
    for (int st = 0; st < NBUF; ++st) {
      D2 = next_stage();
#pragma unroll
      for (int q = 0; q < kLoadsA + kLoadsB; ++q) direct(D2, st * C::kStage, q);
    }
    wait_vm<(NBUF - 1) * (kLoadsA + kLoadsB)>();
    bare_barrier();
  } else {
    static_assert(NBUF == 2, "transposing sides have two buffers");
    auto load_all = [&](Raw& x, const Desc& D) {
#pragma unroll
      for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int r = 0; r < 8; ++r) load_x(x, D, n, r);
    };
    const Desc D0 = next_stage();
#pragma unroll
    for (int q = 0; q < kLoadsA + kLoadsB; ++q) direct(D0, 0, q);
    load_all(raw[0], D0);
    const Desc D1 = next_stage();
#pragma unroll
    for (int q = 0; q < kLoadsA + kLoadsB; ++q) direct(D1, C::kStage, q);
    load_all(raw[1], D1);
#pragma unroll
    for (int n = 0; n < NS; ++n)
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        turn(raw[0], n, c);
        put(n, c, 0);
      }
    D2 = next_stage();
    load_all(raw[0], D2);
    wait_lds();
    wait_vm<0>();
    bare_barrier();
  }
#pragma unroll
  for (int k = 0; k < NT + MT; ++k) read(F[0], 0, 0, k);

  // Stage s in the buffer at `base`, the next one at `nbase`: its products.  Transposing sides turn stage s + 1
  // (registers `x`) into the other buffer and load stage s + 3.  Behind the barrier, which every wave reaches with its
  // last operands read, direct sides load stage s + NBUF into this buffer.
  auto stage = [&](Raw& x, auto BASE, auto NBASE) {
    const int base = BASE, nbase = NBASE;
    constexpr int kBefore = 3 * C::PS;                            // products in front of the barrier
    // items in front of the barrier, 24 a block: turned (a step and a write a column), then loaded
    constexpr int kItems = 24 * NS;
    Desc D3;
    if constexpr (X) D3 = next_stage();
    unrolled<0, 4>([&](auto KSC) {
      constexpr int ks = decltype(KSC)::value;
      if constexpr (ks == 3) {
        wait_lds();
        if constexpr (!X) wait_vm<(NBUF - 2) * (kLoadsA + kLoadsB)>();   // (later stages may be in flight)
        else if constexpr (kLoadsA + kLoadsB > 0) wait_vm<8>();   // (this stage's 8 loads into registers may be in flight)
        bare_barrier();
        if constexpr (!X) D2 = next_stage();
      }
      unrolled<0, C::PS>([&](auto QC) {
        constexpr int q = decltype(QC)::value, xt = q / NT, y = q % NT, n = ks * C::PS + q;
        acc[xt][y] = mfma32(F[ks & 1].a[xt], F[ks & 1].b[y], acc[xt][y]);
        // operands of the next step
        read(F[(ks + 1) & 1], ks == 3 ? nbase : base, (ks + 1) & 3, q);
        if constexpr (ks < 3) {
          unrolled<n * kItems / kBefore, (n + 1) * kItems / kBefore>([&](auto IC) {
            constexpr int i = decltype(IC)::value;
            if constexpr (i % 24 >= 16) load_x(x, D3, i / 24, i % 24 - 16);
            else if constexpr (i % 2 == 0) turn(x, i / 24, i % 24 / 2);
            else put(i / 24, i % 24 / 2, nbase);
          });
        } else {
          constexpr int L = kLoadsA + kLoadsB;
          unrolled<q * L / C::PS, (q + 1) * L / C::PS>([&](auto IC) { direct(D2, base, decltype(IC)::value); });
        }
        __builtin_amdgcn_sched_barrier(0);
      });
    });
    if constexpr (X) D2 = D3;
  };

  int at = 0;   // the buffer of the next stage
  Piece w;
  for (int piece = 0; product_piece(&kernel_args()->a, g, piece, w); ++piece) {
    int ti, tj;
    product_tile(w.tile, kernel_args()->a.nbm, kernel_args()->a.nbn, ti, tj);
    ti = uni(ti);
    tj = uni(tj);
    const int s0 = uni(w.s0), s1 = uni(w.s1);
#pragma unroll
    for (int x = 0; x < MT; ++x)
#pragma unroll
      for (int y = 0; y < NT; ++y)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[x][y][e] = 0.f;
    if constexpr (X) {
      for (int st = s0; st < s1; st += 2) {
        stage(raw[X ? 1 : 0], std::integral_constant<int, 0>{}, std::integral_constant<int, C::kStage>{});
        stage(raw[0], std::integral_constant<int, C::kStage>{}, std::integral_constant<int, 0>{});
      }
    } else {
      for (int st = s0; st < s1; ++st) {
        const int next = at == (NBUF - 1) * C::kStage ? 0 : at + C::kStage;
        stage(raw[0], at, next);
        at = next;
      }
    }
    const auto* const q = kernel_args();
    ConstArgs& a = q->a;
    ConstOut& o = q->o;
    // the sums stay in the accumulator registers until their own turn
    auto hold = [](pf32x16& v) {
      if constexpr (MT * NT > 4) asm volatile("" : "+a"(v));
    };
    // Register e of MFMA tile (x, y) is element (8 (e / 4) + 4 (lane / 32) + e % 4, lane % 32) of its 32 x 32 outputs.
    int el = threadIdx.x & 63;
    asm volatile("" : "+v"(el));   // (what depends on the lane is computed anew for each piece)
    if (s0 > 0 || s1 < total) {
      // a piece, in the order of the registers: [wave][x][y][e / 4][lane][e % 4]
      float* p = a.part + (int64_t)uni(w.number) * (C::SA * C::SB) + wave * MT * NT * 1024 + el * 4;
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
      continue;
    }
    // Each wave turns 32 outputs x 32 (or 64 of 16 bits) into rows in its own 4 KB of LDS.  Its LDS operations run
    // in order, so a block's rows are read back while the next block is computed and written over them.
    constexpr int XO = GLU ? MT / 2 : MT;                            // 32-wide output tiles along i
    constexpr int XB = sizeof(TO) == 2 && XO >= 2 ? 2 : 1;           // of which this many at a time
    constexpr int CH = XB * 32 / OutVec<TO>::N;                      // 16-byte chunks of a row
    constexpr int kRows = CH / 2;
    char* mine = lds + NBUF * C::kStage + wave * C::kTurn;
    const int i0 = ti * (GLU ? C::SA / 2 : C::SA) + wm * 32 * XO;
    const int64_t j0 = (int64_t)tj * C::SB + wn * 32 * NT;
    const bool stream = o.stream != 0;
    DropArgs drop{};
    if constexpr (GLU) drop = drop_args_of(o);
    const uint64_t offset = GLU && drop.on ? drop_offset(drop) : 0;
    // block b of three (z, u and h) or one for each place, places along i first
    auto fill = [&](auto BC, auto WC) {
      constexpr int b = decltype(BC)::value, of = decltype(WC)::value, what = of == 3 ? b % 3 : 2;
      constexpr int xb = b / of % (XO / XB) * XB, y = b / of / (XO / XB);
      char* to = mine;
#pragma unroll
      for (int q = 0; q < XB; ++q) {
        uint32_t bits[4][2];
        if (GLU && what == 2 && drop.on) {
          // the lanes of the lower half draw for columns 0 .. 15 of the 32, those of the upper for 16 .. 31; of each
          // eight columns the lower half then takes the first four
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            uint32_t w[4];
            drop_bits(drop, offset, (uint32_t)(j0 + 32 * y + (el & 31)), (uint32_t)(i0 + 32 * (xb + q)) / 8 + 2 * (el >> 5) + n,
                      w);
            const auto p0 = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
            const auto p1 = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
            bits[n][0] = p0[0];
            bits[n][1] = p1[0];
            bits[n + 2][0] = p0[1];
            bits[n + 2][1] = p1[1];
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float v[4];
          if constexpr (GLU) {
            hold(acc[2 * (xb + q)][y]);
            hold(acc[2 * (xb + q) + 1][y]);
          } else {
            hold(acc[xb + q][y]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if constexpr (GLU) {
              const float z = acc[2 * (xb + q)][y][4 * e + i], u = acc[2 * (xb + q) + 1][y][4 * e + i];
              v[i] = what == 0 ? z : what == 1 ? u : act_value<ACT>(z) * u;
              if (what == 2 && drop.on) v[i] = drop_one(drop, bits[e], i, v[i]);
            } else {
              v[i] = acc[xb + q][y][4 * e + i];
              if constexpr (EPI == kEpiGrad) v[i] *= o.alpha;
            }
          }
          uint32_t w[4];
          pack4<TO>(v, w);
          const int t = el & 31, hi = el >> 5;
          if constexpr (sizeof(TO) == 2) {
            const pu32x2 p = {w[0], w[1]};
            *reinterpret_cast<pu32x2*>(to + t * (CH * 16) + (((4 * q + e) ^ (t & (CH - 1))) * 16 + hi * 8)) = p;
          } else {
            const pu32x4 p = {w[0], w[1], w[2], w[3]};
            *reinterpret_cast<pu32x4*>(to + t * (CH * 16) + ((2 * e + hi) ^ (t & (CH - 1))) * 16) = p;
          }
        }
      }
      __builtin_amdgcn_wave_barrier();
    };
    pu32x4 out[kRows];
    auto fetch = [&]() {
      const char* from = mine;
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const int row = r * (64 / CH) + el / CH;
        out[r] = *reinterpret_cast<const pu32x4*>(from + row * (CH * 16) + ((el % CH) ^ (row & (CH - 1))) * 16);
      }
    };
    auto write = [&](auto BC, auto WC) {
      constexpr int b = decltype(BC)::value, of = decltype(WC)::value, what = of == 3 ? b % 3 : 2;
      constexpr int xb = b / of % (XO / XB) * XB, y = b / of / (XO / XB);
      TO* to = static_cast<TO*>(what == 0 ? o.gate : what == 1 ? o.up : o.out);
      const int64_t ld = what == 0 ? o.ldz : what == 1 ? o.ldup : o.ldo;
      asm volatile("" : "+v"(el));
      const int col = i0 + 32 * xb + (el % CH) * OutVec<TO>::N;
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const int64_t t = j0 + 32 * y + r * (64 / CH) + el / CH;
        if (t < a.N && col < a.M) {
          uint32_t w[4] = {out[r][0], out[r][1], out[r][2], out[r][3]};
          TO* p = to + t * ld + col;
          if (EPI == kEpiGrad && o.accumulate) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (col + i < a.M) w[i] = __float_as_uint(__uint_as_float(w[i]) + reinterpret_cast<const float*>(p)[i]);
          }
          store16<TO>(p, w, a.M - col, stream);
        }
      }
    };
    auto blocks = [&](auto WC) {
      constexpr int n = NT * (XO / XB) * decltype(WC)::value;
      fill(std::integral_constant<int, 0>{}, WC);
      unrolled<0, n>([&](auto BC) {
        constexpr int b = decltype(BC)::value;
        fetch();
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (b + 1 < n) fill(std::integral_constant<int, b + 1>{}, WC);
        __builtin_amdgcn_sched_barrier(0);
        write(BC, WC);
        __builtin_amdgcn_sched_barrier(0);
      });
    };
    if (GLU && o.gate) blocks(std::integral_constant<int, GLU ? 3 : 1>{});
    else blocks(std::integral_constant<int, 1>{});
  }
  wait_vm<0>();   // loads into LDS have to end before the workgroup does
}

// Outputs of the split tiles from their pieces, added in the order of the long
// axis.  A workgroup takes 32 outputs along j of one wave's part of a tile and
// turns them from the order of the registers to rows in LDS.
template <typename TO, int EPI, int ACT, int MT, int NT>
__global__ void __launch_bounds__(256) k_product_join(ProdArgs a, ProdOut o, int G, int first) {
  constexpr bool GLU = EPI == kEpiGlu;
  constexpr int SA = 64 * MT, SB = 64 * NT, PER = NT * 4;           // PER: workgroups of a tile
  constexpr int XO = GLU ? MT / 2 : MT, W = 32 * XO;                // outputs along i
  __shared__ float rows[GLU ? 2 : 1][32][W + 4];
  const int tile = first + blockIdx.x / PER, q = blockIdx.x % PER;
  const int y = q % NT, wave = q / NT;
  const int lane = threadIdx.x & 63, e = threadIdx.x >> 6;
  const float* base = a.part + (wave * MT * NT + y) * 1024 + threadIdx.x * 4;
  float4 s[MT];
#pragma unroll
  for (int x = 0; x < MT; ++x) s[x] = float4{0.f, 0.f, 0.f, 0.f};
  wgrad_pieces(wgrad_levels(a.nbm * a.nbn, (a.nst * a.nseg + a.unit - 1) / a.unit, G), tile,
               [&](int number, int stride, int count) {
    constexpr int AT = 8 / MT;   // pieces at once: eight loads in flight
    for (int c = 0; c < count; c += AT) {
      float4 v[AT][MT];
#pragma unroll
      for (int k = 0; k < AT; ++k)
#pragma unroll
        for (int x = 0; x < MT; ++x) {
          v[k][x] = float4{0.f, 0.f, 0.f, 0.f};
          if (c + k < count)
            v[k][x] = *reinterpret_cast<const float4*>(base + ((int64_t)number + (int64_t)(c + k) * stride) * SA * SB + x * NT * 1024);
        }
#pragma unroll
      for (int k = 0; k < AT; ++k)
#pragma unroll
        for (int x = 0; x < MT; ++x) {
          s[x].x += v[k][x].x;
          s[x].y += v[k][x].y;
          s[x].z += v[k][x].z;
          s[x].w += v[k][x].w;
        }
    }
  });
#pragma unroll
  for (int x = 0; x < MT; ++x)
    *reinterpret_cast<float4*>(&rows[GLU ? x & 1 : 0][lane & 31][32 * (GLU ? x / 2 : x) + 8 * e + 4 * (lane >> 5)]) = s[x];
  __syncthreads();
  int ti, tj;
  product_tile(tile, a.nbm, a.nbn, ti, tj);
  const int i0 = ti * (GLU ? SA / 2 : SA) + (wave >> 1) * W;
  const int64_t j0 = (int64_t)tj * SB + (wave & 1) * 32 * NT + 32 * y;
  const uint64_t offset = GLU && o.drop.on ? drop_offset(o.drop) : 0;
  for (int k = threadIdx.x; k < 32 * W / 8; k += 256) {
    const int r = k / (W / 8), c = k % (W / 8) * 8, n = a.M - (i0 + c);
    const int64_t t = j0 + r;
    if (t >= a.N || n <= 0) continue;
    float v[8], u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = rows[0][r][c + i];
    Raw8<TO> p;
    if constexpr (GLU) {
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] = rows[GLU ? 1 : 0][r][c + i];
      if (o.gate) {
        pack8(v, p);
        store8(static_cast<TO*>(o.gate) + t * o.ldz + i0 + c, p, n, false);
        pack8(u, p);
        store8(static_cast<TO*>(o.up) + t * o.ldup + i0 + c, p, n, false);
      }
      uint32_t w[4];
      if (o.drop.on) drop_bits(o.drop, offset, (uint32_t)t, (uint32_t)(i0 + c) / 8, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = act_value<ACT>(v[i]) * u[i];
        if (o.drop.on) v[i] = drop_one(o.drop, w, i, v[i]);
      }
    }
    TO* out = static_cast<TO*>(o.out) + t * o.ldo + i0 + c;
    if constexpr (EPI == kEpiGrad) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] *= o.alpha;
        if (o.accumulate && i < n) v[i] += reinterpret_cast<const float*>(out)[i];
      }
    }
    pack8(v, p);
    store8(out, p, n, false);
  }
}

// Operands laid out anew: rows 16-byte aligned, padded with zeros to a
// multiple of 8 columns; an fp32 operand as three bf16 planes (split_planes).
struct PackArgs {
  const void* src[4];
  uint16_t* dst[4];
  int64_t ld[4], rows[4], block[5];   // block: first workgroup of each operand
  int cols[4];
};
template <typename T>
__global__ void __launch_bounds__(256) k_product_pack(PackArgs a) {
  int m = 0;
#pragma unroll
  for (int i = 1; i < 4; ++i) m += blockIdx.x >= a.block[i];
  const int cols = a.cols[m], nb = (cols + 7) / 8;
  const int64_t first = ((int64_t)blockIdx.x - a.block[m]) * 256, r0 = first / nb;
  const uint32_t at = (uint32_t)(first - r0 * nb) + threadIdx.x, down = at / (uint32_t)nb;
  const int64_t r = r0 + down, rows = a.rows[m], ldp = (int64_t)nb * 8;
  if (r >= rows) return;
  const int c = (int)(at - down * (uint32_t)nb) * 8;
  const Raw8<T> x = load8(static_cast<const T*>(a.src[m]) + r * a.ld[m] + c, cols - c);
  uint16_t* p = a.dst[m] + r * ldp + c;
  if constexpr (sizeof(T) == 2) {
    store_words<4>(p, x.w, false);
  } else {
    float v[8];
    unpack8(x, v);
    split_planes(v, [&](int pl, const uint32_t* w) { store_words<4>(p + (int64_t)pl * rows * ldp, w, false); });
  }
}

namespace {

template <typename E, typename TO, int EPI, int ACT, bool AX, bool BX>
void product_go(const ProdArgs& a, const ProdOut& o, const ProdPlan& p, hipStream_t s) {
  if (p.side == 256) {
    hipLaunchKernelGGL((k_product<E, TO, EPI, ACT, 4, 4, AX, BX, 2, 1>), dim3((unsigned)p.grid), dim3(256), 0, s,
                       KernelArgs{a, o});
    if (p.split)
      hipLaunchKernelGGL((k_product_join<TO, EPI, ACT, 4, 4>), dim3((unsigned)(p.split * 16)), dim3(256), 0, s, a, o,
                         p.grid, p.first);
  } else {
    if constexpr (!AX && !BX) {
      if (p.deep)
        hipLaunchKernelGGL((k_product<E, TO, EPI, ACT, 2, 2, AX, BX, 4, 1>), dim3((unsigned)p.grid), dim3(256), 0, s,
                           KernelArgs{a, o});
    }
    if (!p.deep)
      hipLaunchKernelGGL((k_product<E, TO, EPI, ACT, 2, 2, AX, BX, 2, 2>), dim3((unsigned)p.grid), dim3(256), 0, s,
                         KernelArgs{a, o});
    if (p.split)
      hipLaunchKernelGGL((k_product_join<TO, EPI, ACT, 2, 2>), dim3((unsigned)(p.split * 8)), dim3(256), 0, s, a, o, p.grid,
                         p.first);
  }
}

template <typename E, typename TO>
void product_types(const ProductCall& c, const ProdArgs& a, const ProdOut& o, const ProdPlan& p, hipStream_t s) {
  if (c.epi == kEpiStore) {
    product_go<E, TO, kEpiStore, 0, true, false>(a, o, p, s);
  } else if (c.epi == kEpiGrad) {
    product_go<E, float, kEpiGrad, 0, true, true>(a, o, p, s);
  } else {
    switch (c.act) {
      case GIFT_ACT_SILU: return product_go<E, TO, kEpiGlu, GIFT_ACT_SILU, false, false>(a, o, p, s);
      case GIFT_ACT_GELU: return product_go<E, TO, kEpiGlu, GIFT_ACT_GELU, false, false>(a, o, p, s);
      case GIFT_ACT_GELU_TANH: return product_go<E, TO, kEpiGlu, GIFT_ACT_GELU_TANH, false, false>(a, o, p, s);
      case GIFT_ACT_RELU: return product_go<E, TO, kEpiGlu, GIFT_ACT_RELU, false, false>(a, o, p, s);
      default: return product_go<E, TO, kEpiGlu, GIFT_ACT_SIGMOID, false, false>(a, o, p, s);
    }
  }
}

int planes_of(int dtype) { return dtype == GIFT_FP32 ? 3 : 1; }
int64_t packed_ld(int64_t cols) { return cdiv(cols, 8) * 8; }
// A direct operand is loaded in whole chunks of 8; a transposing one from any address, in whole words.
bool as_it_is(const ProdOperand& m, int dtype, bool turned) {
  if (dtype == GIFT_FP32 || m.packed) return false;
  return turned ? m.near && m.cols % 2 == 0 : m.aligned && m.cols % 8 == 0;
}
// Whether k_product_pack has to lay an operand out, and can: of the four of a launch each has a quarter of its workgroups.
bool to_pack(const ProdOperand& m, int dtype, bool turned) { return m.rows && !m.packed && !as_it_is(m, dtype, turned); }
bool may_pack(const ProdOperand& m) {
  return m.rows < ((int64_t)1 << 36) && cdiv(m.rows * cdiv(m.cols, 8), 256) <= kMaxGrid / 4;
}

}  // namespace

int64_t product_tiles(int64_t M, int64_t N) { return cdiv(M, 64) * cdiv(N, 128); }

size_t product_packed(int dtype, int64_t rows, int64_t cols) {
  return align256((size_t)planes_of(dtype) * (size_t)rows * (size_t)packed_ld(cols) * 2);
}

bool product_reach(const ProductCall& c) {
  const bool ax = c.epi != kEpiGlu, bx = c.epi == kEpiGrad;
  for (int i = 0; i < 2; ++i) {
    if (to_pack(c.a[i], c.dtype, ax) && !may_pack(c.a[i])) return false;
    if (to_pack(c.b[i], c.dtype, bx) && !may_pack(c.b[i])) return false;
  }
  return true;
}

// Workspace: the operands to pack, one after another, then the pieces.  (A query that knows less of the alignment than
// the call counts nothing for an operand too large to pack: the call reads it as it is, or is refused.)
size_t product_workspace(const ProductCall& c) {
  const bool ax = c.epi != kEpiGlu, bx = c.epi == kEpiGrad;
  size_t b = 0;
  auto add = [&](const ProdOperand& m, bool turned) {
    if (to_pack(m, c.dtype, turned) && may_pack(m)) b += product_packed(c.dtype, m.rows, m.cols);
  };
  for (int i = 0; i < 2; ++i) {
    add(c.a[i], ax);
    add(c.b[i], bx);
  }
  return b + align256(product_plan(c.epi, ax, bx, c.M, c.N, c.K, c.parts * (c.dtype == GIFT_FP32 ? 6 : 1)).bytes);
}

hipError_t launch_product(const ProductCall& c, const DropArgs& drop, hipStream_t s) {
  const bool ax = c.epi != kEpiGlu, bx = c.epi == kEpiGrad;
  ProdArgs a{};
  char* work = static_cast<char*>(c.work);
  // operands as the kernel reads them: first plane, distance of the planes, leading dimension, columns
  struct Laid {
    uint64_t p;
    int64_t plane, ld, cols;
  };
  PackArgs pack{};
  int packs = 0;
  int64_t blocks = 0;
  auto lay = [&](const ProdOperand& m, bool turned) {
    Laid l{};
    if (!m.rows) return l;
    l.cols = packed_ld(m.cols);
    l.ld = l.cols;
    l.plane = m.rows * l.ld * 2;
    l.p = (uint64_t)m.p;
    if (m.packed) return l;
    if (as_it_is(m, c.dtype, turned)) {
      if (m.rows > 1) l.ld = m.ld;
      l.cols = m.cols;
      return l;
    }
    l.p = (uint64_t)work;
    pack.src[packs] = m.p;
    pack.dst[packs] = reinterpret_cast<uint16_t*>(work);
    pack.ld[packs] = m.ld;
    pack.rows[packs] = m.rows;
    pack.cols[packs] = (int)m.cols;
    pack.block[packs++] = blocks;
    blocks += cdiv(m.rows * (l.ld / 8), 256);
    work += product_packed(c.dtype, m.rows, m.cols);
    return l;
  };
  const Laid A[2] = {lay(c.a[0], ax), lay(c.a[1], ax)}, B[2] = {lay(c.b[0], bx), lay(c.b[1], bx)};
  for (int i = packs; i < 5; ++i) pack.block[i] = blocks;
  if (packs) {
    if (c.dtype == GIFT_FP32) hipLaunchKernelGGL(k_product_pack<float>, dim3((unsigned)blocks), dim3(256), 0, s, pack);
    else hipLaunchKernelGGL(k_product_pack<Bf16>, dim3((unsigned)blocks), dim3(256), 0, s, pack);
  }
  // of the nine products of planes the six largest, the smallest of them first
  static const int kPlanes[6][2] = {{0, 2}, {1, 1}, {2, 0}, {0, 1}, {1, 0}, {0, 0}};
  const int n = c.dtype == GIFT_FP32 ? 6 : 1;
  for (int q = 0; q < n; ++q)
    for (int part = 0; part < c.parts; ++part) {
      const int pa = n == 1 ? 0 : kPlanes[q][0], pb = n == 1 ? 0 : kPlanes[q][1];
      const int k = a.nseg++;
      a.a[k] = A[part].p + (uint64_t)(pa * A[part].plane);
      a.b[k] = B[part].p + (uint64_t)(pb * B[part].plane);
      if (c.epi == kEpiGlu) a.a2[k] = A[1].p + (uint64_t)(pa * A[1].plane);
    }
  a.lda = A[0].ld;
  a.lda2 = A[1].ld;
  a.ldb = B[0].ld;
  a.acols = A[0].cols;
  a.bcols = B[0].cols;
  a.K = c.K;
  a.M = (int)c.M;
  a.N = c.N;
  const ProdPlan p = product_plan(c.epi, c.epi != kEpiGlu, c.epi == kEpiGrad, c.M, c.N, c.K, a.nseg);
  a.nst = p.nst;
  a.nbm = p.nbm;
  a.nbn = p.nbn;
  a.unit = p.unit;
  a.part = reinterpret_cast<float*>(work);
  ProdOut o{};
  o.out = c.out;
  o.ldo = c.ldo;
  o.gate = c.gate;
  o.up = c.up;
  o.ldz = c.ldz;
  o.ldup = c.ldup;
  o.drop = drop;
  o.alpha = c.alpha;
  o.accumulate = c.accumulate;
  o.stream = c.N * c.M * (c.dtype == GIFT_FP32 || c.epi == kEpiGrad ? 4 : 2) > kStreamBytes;
  if (c.dtype == GIFT_BF16) product_types<Bf16, Bf16>(c, a, o, p, s);
  else if (c.dtype == GIFT_FP16) product_types<Fp16, Fp16>(c, a, o, p, s);
  else product_types<Bf16, float>(c, a, o, p, s);
  return hipGetLastError();
}

}  // namespace gift
