// Layer norm and RMS norm over rows: forward (optionally keeping its input as
// an 8-bit checkpoint in the same pass) and backward, from the input or from
// its checkpoint, with the reduction of the weight's and bias's gradients.
//
// GIFT 阅读笔记, §实验设置: the layers whose gradients the codec carries are
// the MLP layers of Llama-class models; a norm stands in front of each block
// of them.
//
//   mean = sum_j x_j / d (0 for RMS),  rstd = (sum_j (x_j - mean)^2 / d + eps)^-1/2
//   xh = (x - mean) rstd,              y = xh gamma + beta
//   g = dy gamma,  c1 = sum_j g_j xh_j / d,  c2 = sum_j g_j / d (0 for RMS)
//   dx = rstd (g - c2 - xh c1),  dgamma = sum_t dy xh,  dbeta = sum_t dy
//
// Everything is computed in fp32; y and dx are rounded once to the element
// type.  The variance is the sum of squares about the mean (the row is in
// registers, so the second pass costs no memory traffic and does not cancel).
//
// Both are bound by memory.  A row is held by G lanes, 8 elements (one
// 16-byte load of a 16-bit type) per lane and chunk, CH chunks: G = 16 for
// d <= 128, a wave up to 2048, a workgroup of 256 up to 8192 and of 512 up to
// 16384 columns.  Sums inside 64 lanes are lane exchanges; wider groups add
// their waves' sums through LDS.
#include <type_traits>

#include "act8.hpp"

namespace gift {

struct NormArgs {
  const void* x;
  int64_t ldx;
  uint8_t* codes;       // checkpoint: written by the forward, read by the backward (NULL: none)
  int64_t ldc;
  uint8_t* bscales;
  int nb, fmt;
  const void *w, *b;    // gamma, beta (NULL: ones, zeros)
  int w32;              // gamma, beta in fp32 (otherwise in the element type)
  int layer;            // 1: layer norm, 0: RMS norm
  int64_t T;
  int d;
  float eps, invd;
  float *mean, *rstd;   // forward: written (either may be NULL); backward: read
  void* y;              // forward: y; backward: dx
  int64_t ldy;
  const void* dy;
  int64_t lddy;
  float* part;          // backward: [P][sums][d] partial sums of dgamma, dbeta (NULL: not wanted)
  int sums;             // 2, or 1: dgamma alone
  int P;                // backward: workgroups that take rows
  int steplog;          // backward: a row group is 2^steplog steps
  float *dw, *db;       // backward, columns in the same launch (NULL: not wanted, or by k_norm_reduce)
  int accumulate;
  int stream;           // the output is larger than the caches (act8.hpp)
  int64_t groups;       // backward: row groups
};

namespace {

template <int G>
constexpr int kNormThreads = G > 256 ? G : 256;
// Sums of N values over the G lanes of a row.  Groups wider than a wave pass
// through `red` (two buffers in turn, so one barrier per call is enough).
template <int G, int N>
__device__ __forceinline__ void row_sums(float* v, float (*red)[2][8], int& flip) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = lanes_sum<G == 16 ? 16 : 64>(v[i]);
  if constexpr (G > 64) {
    constexpr int W = G / 64;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) red[flip][i][wave] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = red[flip][i][0];
#pragma unroll
      for (int k = 1; k < W; ++k) s += red[flip][i][k];
      v[i] = s;
    }
    flip ^= 1;
  }
}

// A row's last chunk alone can be partial or empty (norm_variant takes the
// fewest chunks): the others are loaded, counted and stored without checks,
// which is a third of the instructions of these loops.
template <int CH>
__device__ __forceinline__ int chunk_size(int c, int n) {
  return c < CH - 1 ? 8 : n;
}

// Eight weights at column col (n of them inside the row).
template <typename T>
__device__ __forceinline__ void load_weights(const void* p, int w32, int col, int n, float* v) {
  if (w32) unpack8(load8(static_cast<const float*>(p) + col, n), v);
  else unpack8(load8(static_cast<const T*>(p) + col, n), v);
}

// Raw chunk c of the row at t: the elements, or the codes and the exponent
// of the chunk's block.
template <typename T, bool CK>
struct RowChunk {
  Raw8<T> r;
};
template <typename T>
struct RowChunk<T, true> {
  uint32_t w[2];
  uint32_t e;
};

template <typename T>
__device__ __forceinline__ void load_chunk(RowChunk<T, false>& c, const NormArgs& a, int64_t t, int col, int n) {
  c.r = load8(static_cast<const T*>(a.x) + t * a.ldx + col, n);
}
template <typename T>
__device__ __forceinline__ void load_chunk(RowChunk<T, true>& c, const NormArgs& a, int64_t t, int col, int n) {
  c.w[0] = c.w[1] = 0;
  c.e = kActExpMin;
  if (n > 0) {
    __builtin_memcpy(c.w, __builtin_assume_aligned(a.codes + t * a.ldc + col, 8), 8);
    c.e = a.bscales[((t >> 3) * a.nb + col / kActBlock) * kActGroup + (t & 7)];
  }
}
template <typename T>
__device__ __forceinline__ void chunk_values(const RowChunk<T, false>& c, const NormArgs&, float* v) {
  unpack8(c.r, v);
}
template <typename T>
__device__ __forceinline__ void chunk_values(const RowChunk<T, true>& c, const NormArgs& a, float* v) {
  act_decode8(c.w, c.e, a.fmt, v);
}

}  // namespace

// Forward, one row per lane group (two rows at once, for more loads in
// flight, took the registers of a third wave per SIMD: 32.7 against 29.4 us
// with a checkpoint, 20.8 against 19.8 without, at 16384 x 1536 bf16).
// Where a row takes a whole workgroup, consecutive workgroups go to different
// dies (round robin over 8); the row map below gives the 8 rows of one
// exponent group to one die, so their bytes merge in one L2.
template <typename T, int G, int CH>
__global__ void __launch_bounds__(kNormThreads<G>) k_norm_fwd(NormArgs a) {
  __shared__ float red[2][2][8];
  int flip = 0;
  const int lane = threadIdx.x % G;
  int64_t t;
  if constexpr (G > 64) {
    const int64_t b = blockIdx.x;
    t = (b & ~(int64_t)63) + (b & 7) * 8 + ((b >> 3) & 7);
  } else {
    t = (int64_t)blockIdx.x * (kNormThreads<G> / G) + threadIdx.x / G;
  }
  if (t >= a.T) return;   // the lanes of a row together (G <= 64 has no barriers below)
  Raw8<T> raw[CH];
  float v[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int col = (c * G + lane) * 8;
    raw[c] = load8(static_cast<const T*>(a.x) + t * a.ldx + col, chunk_size<CH>(c, a.d - col));
  }
  float s = 0.f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    unpack8(raw[c], v[c]);
#pragma unroll
    for (int j = 0; j < 8; ++j) s += v[c][j];
  }
  float mean = 0.f;
  if (a.layer) {
    row_sums<G, 1>(&s, red, flip);
    mean = s / (float)a.d;   // correctly rounded: a constant row is centred exactly
  }
  float q = 0.f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int n = chunk_size<CH>(c, a.d - (c * G + lane) * 8);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float u = j < n ? v[c][j] - mean : 0.f;
      q += u * u;
    }
  }
  row_sums<G, 1>(&q, red, flip);
  const float rstd = 1.0f / sqrtf(q / (float)a.d + a.eps);
  if (lane == 0) {
    if (a.mean) a.mean[t] = mean;
    if (a.rstd) a.rstd[t] = rstd;
  }
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int col = (c * G + lane) * 8;
    const int n = chunk_size<CH>(c, a.d - col);
    if (a.codes) {
      const uint32_t e = act_exponent(quad_max(amax_bits(raw[c])), a.fmt);
      uint32_t k[2];
      act_encode8(v[c], e, a.fmt, k);
      if (c < CH - 1 || col < a.nb * kActBlock) {
        __builtin_memcpy(__builtin_assume_aligned(a.codes + t * a.ldc + col, 8), k, 8);
        if ((lane & 3) == 0)
          a.bscales[((t >> 3) * a.nb + col / kActBlock) * kActGroup + (t & 7)] = (uint8_t)e;
      }
    }
    float w[8], b[8], y[8];
    if (a.w) load_weights<T>(a.w, a.w32, col, n, w);
    if (a.b) load_weights<T>(a.b, a.w32, col, n, b);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      y[j] = (v[c][j] - mean) * rstd;
      if (a.w) y[j] *= w[j];
      if (a.b) y[j] += b[j];
    }
    Raw8<T> o;
    pack8(y, o);
    store8(static_cast<T*>(a.y) + t * a.ldy + col, o, n, a.stream != 0);
  }
}

// Rows in flight ahead of the present one (see k_norm_bwd).
template <typename T, int G, int CH>
constexpr int kAhead = G == 512 && CH == 4 ? 0 : CH <= 2 || (CH == 3 && sizeof(T) == 2) ? 2 : 1;

// dgamma and dbeta of 32 columns straight from x and dy: 4 lanes across, NT /
// 4 down the rows, whose sums are added through LDS in order.
template <typename T, bool CK, int NT>
__device__ __forceinline__ void norm_columns(const NormArgs& a, int block, float (*part)[kActBlock + 1]) {
  constexpr int ROWS = NT / 4;
  const int lane = threadIdx.x & 3, row = threadIdx.x >> 2;
  const int col = block * kActBlock + lane * 8, n = a.d - col;
  float dg[8], db[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) dg[j] = db[j] = 0.f;
#pragma unroll 4
  for (int64_t t = row; t < a.T; t += ROWS) {
    RowChunk<T, CK> x;
    load_chunk(x, a, t, col, n);
    const Raw8<T> y = load8(static_cast<const T*>(a.dy) + t * a.lddy + col, n);
    const float mean = a.layer ? a.mean[t] : 0.f, rstd = a.rstd[t];
    float xv[8], yv[8];
    chunk_values(x, a, xv);
    unpack8(y, yv);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      dg[j] += yv[j] * ((xv[j] - mean) * rstd);
      db[j] += yv[j];
    }
  }
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float* out = which == 0 ? a.dw : a.db;
    if (!out) continue;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) part[row][lane * 8 + j] = which == 0 ? dg[j] : db[j];
    __syncthreads();
    const int c = block * kActBlock + threadIdx.x;
    if (threadIdx.x < kActBlock && c < a.d) {
      float v = 0.f;
#pragma unroll 8
      for (int r = 0; r < ROWS; ++r) v += part[r][threadIdx.x];
      out[c] = a.accumulate ? out[c] + v : v;
    }
  }
}

// Backward.  Workgroup p takes the row groups p, p + P, ...; each lane keeps
// the dgamma and dbeta sums of its own columns in registers over all of them
// and has the next rows in flight while it works on the present one
// (kAhead): two up to two chunks, or three of a 16-bit type, one with four
// chunks or three of fp32, none above 12288 columns (there the weights come
// from the cache each time too).  Two waves a SIMD are resident: up to two
// chunks (90 to 192 registers) by the number of workgroups launched
// (norm_partials), with three (211 to 232) and, from a 16-bit input, with
// four (at most 255) by the registers.  Four chunks from a checkpoint or from
// fp32 take 257 to 289 up to 8192 columns, and one wave is (8192 x 2048 bf16:
// 34.7 us from a checkpoint, 26.6 from the input, which has more to read).
// The partial sums of the workgroups go to part [P][sums][d] and are added in
// order by k_norm_reduce: no atomics, the same result every time.  Up to
// kDirectRows rows the workgroups past a.P sum the columns instead
// (norm_columns) and there is no part.
template <typename T, bool CK, int G, int CH>
__global__ void __launch_bounds__(kNormThreads<G>) k_norm_bwd(NormArgs a) {
  constexpr int NT = kNormThreads<G>;
  constexpr int S = NT / G;   // rows of a step
  __shared__ float red[2][2][8];
  __shared__ float comb[S > 1 ? S : 1][S > 1 ? G : 1][9];   // padded: 9 words a lane, no bank conflicts
  __shared__ float cols[NT / 4][kActBlock + 1];
  if ((int)blockIdx.x >= a.P) {
    norm_columns<T, CK, NT>(a, (int)blockIdx.x - a.P, cols);
    return;
  }
  int flip = 0;
  const int lane = threadIdx.x % G, sub = S > 1 ? threadIdx.x / G : 0;
  constexpr int AHEAD = kAhead<T, G, CH>, BUF = AHEAD ? AHEAD : 1;
  float wk[AHEAD ? CH : 1][8], dg[CH][8], db[CH][8];
  auto weights = [&](int c, float* v) {
    const int col = (c * G + lane) * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 1.f;
    if (a.w) load_weights<T>(a.w, a.w32, col, chunk_size<CH>(c, a.d - col), v);
  };
#pragma unroll
  for (int c = 0; c < CH; ++c) {
#pragma unroll
    for (int j = 0; j < 8; ++j) dg[c][j] = db[c][j] = 0.f;
    if constexpr (AHEAD > 0) weights(c, wk[c]);
  }
  struct Row {
    RowChunk<T, CK> x[CH];
    Raw8<T> y[CH];
    float mean, rstd;
  };
  Row rows[BUF];
  // step k of this workgroup: row group p + (k / 2^steplog) P, its step k % 2^steplog
  const int64_t mine = a.groups > blockIdx.x ? cdiv(a.groups - blockIdx.x, a.P) : 0;
  const int64_t steps = mine << a.steplog;
  auto row_of = [&](int64_t k) {
    return ((((int64_t)blockIdx.x + (k >> a.steplog) * a.P) << a.steplog) + (k & ((1 << a.steplog) - 1))) * S + sub;
  };
  auto fetch = [&](Row& b, int64_t k) {
    const int64_t t = row_of(k);
    if (k < steps && t < a.T) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int col = (c * G + lane) * 8, n = chunk_size<CH>(c, a.d - col);
        load_chunk(b.x[c], a, t, col, n);
        b.y[c] = load8(static_cast<const T*>(a.dy) + t * a.lddy + col, n);
      }
      b.mean = a.layer ? a.mean[t] : 0.f;
      b.rstd = a.rstd[t];
    }
  };
  auto step = [&](Row& b, int64_t k) {
    const int64_t t = row_of(k);
    if (t >= a.T) return;   // the lanes of a row together (all of the workgroup where row_sums has a barrier)
    if constexpr (AHEAD == 0) fetch(b, k);
    const float mean = b.mean, rstd = b.rstd;
    float xh[CH][8], t8[CH][8];
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int n = chunk_size<CH>(c, a.d - (c * G + lane) * 8);
      float* w = wk[AHEAD ? c : 0];
      if constexpr (AHEAD == 0) weights(c, w);
      chunk_values(b.x[c], a, xh[c]);
      unpack8(b.y[c], t8[c]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // columns past the row add nothing, dy reads zero there
        xh[c][j] = j < n ? (xh[c][j] - mean) * rstd : 0.f;
        s[0] += t8[c][j] * w[j] * xh[c][j];
        dg[c][j] += t8[c][j] * xh[c][j];
      }
      if (a.layer || a.sums == 2) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          s[1] += t8[c][j] * w[j];
          db[c][j] += t8[c][j];
        }
      }
    }
    if constexpr (AHEAD > 0) fetch(b, k + AHEAD);
    row_sums<G, 2>(s, red, flip);
    const float c1 = s[0] * a.invd, c2 = a.layer ? s[1] * a.invd : 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = (c * G + lane) * 8;
      float* w = wk[AHEAD ? c : 0];
      if constexpr (AHEAD == 0) weights(c, w);
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = rstd * (t8[c][j] * w[j] - c2 - xh[c][j] * c1);
      Raw8<T> r;
      pack8(o, r);
      store8(static_cast<T*>(a.y) + t * a.ldy + col, r, chunk_size<CH>(c, a.d - col), a.stream != 0);
    }
  };
#pragma unroll
  for (int q = 0; q < AHEAD; ++q) fetch(rows[q], q);
  for (int64_t k = 0; k < steps; k += BUF) {
    step(rows[0], k);
    if constexpr (BUF == 2)
      if (k + 1 < steps) step(rows[1], k + 1);   // (the same for the whole workgroup)
  }
  if (!a.part) return;
  // this workgroup's sums: the S row slots are added through LDS in order
  float* part = a.part + (int64_t)blockIdx.x * a.sums * a.d;
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      if (which == a.sums) break;
      float* v = which == 0 ? dg[c] : db[c];
      const int col = (c * G + lane) * 8;
      if constexpr (S > 1) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) comb[sub][lane][j] = v[j];
        __syncthreads();
        if (sub != 0) continue;
#pragma unroll
        for (int q = 1; q < S; ++q)
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] += comb[q][lane][j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (col + j < a.d) part[(int64_t)which * a.d + col + j] = v[j];
    }
}

// dgamma, dbeta [d] from part [P][sums][d]: a workgroup adds 32 columns, 32
// threads down the partials of each (eight loads of a thread in flight), then
// the threads' sums in order.  accumulate: added to what the outputs hold.
constexpr int kReduceCols = 32, kReduceRows = 32;
__global__ void __launch_bounds__(kReduceCols* kReduceRows) k_norm_reduce(const float* __restrict__ part, int P, int d,
                                                                         int n, float* __restrict__ dw,
                                                                         float* __restrict__ db, int accumulate) {
  __shared__ float sums[kReduceRows][kReduceCols + 1];
  const int cx = threadIdx.x % kReduceCols, ry = threadIdx.x / kReduceCols;
  const int j = blockIdx.x * kReduceCols + cx;   // column of [sums][d], n in all
  float v = 0.f;
  for (int p = ry; p < P; p += 8 * kReduceRows) {
    float x[8];
#pragma unroll
    for (int q = 0; q < 8; ++q)
      x[q] = j < n && p + q * kReduceRows < P ? part[(int64_t)(p + q * kReduceRows) * n + j] : 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q) v += x[q];
  }
  sums[ry][cx] = v;
  __syncthreads();
  if (ry != 0 || j >= n) return;
#pragma unroll
  for (int q = 1; q < kReduceRows; ++q) v += sums[q][cx];
  float* out = j < d ? (dw ? dw + j : nullptr) : db + (j - d);
  if (out) *out = accumulate ? *out + v : v;
}

namespace {

// Calls f with the lane group and chunk count for d columns.
template <typename F>
void norm_variant(int d, F&& f) {
  using std::integral_constant;
  const integral_constant<int, 64> wave;
  const integral_constant<int, 256> four;
  const integral_constant<int, 512> eight;
  if (d <= 128) f(integral_constant<int, 16>{}, integral_constant<int, 1>{});
  else if (d <= 512) f(wave, integral_constant<int, 1>{});
  else if (d <= 1024) f(wave, integral_constant<int, 2>{});
  else if (d <= 1536) f(wave, integral_constant<int, 3>{});
  else if (d <= 2048) f(wave, integral_constant<int, 4>{});
  else if (d <= 4096) f(four, integral_constant<int, 2>{});
  else if (d <= 6144) f(four, integral_constant<int, 3>{});
  else if (d <= 8192) f(four, integral_constant<int, 4>{});
  else if (d <= 12288) f(eight, integral_constant<int, 3>{});
  else f(eight, integral_constant<int, 4>{});
}

}  // namespace

// Rows of the backward's row groups: one or two groups of 8 rows whose
// exponents share cache lines.
static int norm_group_rows(int d) { return d <= 128 ? 16 : 8; }
// Rows of a step of a workgroup.
static int norm_step_rows(int d) { return d <= 128 ? 16 : d <= 2048 ? 4 : 1; }

// Workgroups of the backward pass: two of 256 threads a compute unit or one of
// 512 (every further one adds 8 d bytes of partial sums to write and read),
// never more than there are row groups.  They are resident together but for
// the four-chunk variants of more than 256 registers (k_norm_bwd), which take
// two rounds.
int norm_partials(int64_t T, int d) {
  const int64_t g = cdiv(T, norm_group_rows(d)), most = d > 8192 ? 256 : 512;
  return (int)(g < most ? (g > 0 ? g : 1) : most);
}

// Up to this many rows the parameter gradients are made in the same launch,
// by workgroups of their own that read x and dy once more (from the cache),
// and the rows are spread over as many workgroups as above up to 2048 columns,
// over half as many beyond (by two launches where dx is written over dy or x).
// The workspace is not used then.  bf16, one launch against two,
// 1024 rows: 6.5 / 9.0 us at 1024 columns, 13.6 / 19.1 at 4096; 2048 rows:
// 9.8 / 10.1 at 1024, 16.1 / 12.0 at 1536 columns.
constexpr int64_t kDirectRows = 1024;

static NormArgs norm_args(const NormCall& c) {
  NormArgs a{};
  a.x = c.x;
  a.ldx = c.ldx;
  if (c.ckpt) {
    a.codes = c.ckpt->d_codes;
    a.ldc = c.ckpt->ldc;
    a.bscales = c.ckpt->d_bscales;
    a.fmt = c.ckpt->fmt;
  }
  a.nb = (int)cdiv(c.d, kActBlock);
  a.w = c.w;
  a.b = c.b;
  a.w32 = c.wdtype == GIFT_FP32;
  a.layer = c.kind == GIFT_NORM_LAYER;
  a.T = c.T;
  a.d = c.d;
  a.eps = c.eps;
  a.invd = (float)(1.0 / c.d);
  a.mean = c.mean;
  a.rstd = c.rstd;
  a.y = c.y;
  a.ldy = c.ldy;
  a.dy = c.dy;
  a.lddy = c.lddy;
  a.stream = c.T * c.d * (c.dtype == GIFT_FP32 ? 4 : 2) > kStreamBytes;
  return a;
}

// Workgroups of the forward: a row each above 2048 columns (whole sets of 64
// for the row map), four or, up to 128 columns, sixteen rows each below.
int64_t norm_forward_grid(int64_t T, int d) { return d > 2048 ? cdiv(T, 64) * 64 : cdiv(T, norm_step_rows(d)); }

template <typename T>
static void norm_fwd_t(const NormArgs& a, hipStream_t s) {
  norm_variant(a.d, [&](auto g, auto ch) {
    constexpr int G = decltype(g)::value, CH = decltype(ch)::value;
    hipLaunchKernelGGL((k_norm_fwd<T, G, CH>), dim3((unsigned)norm_forward_grid(a.T, a.d)),
                       dim3(kNormThreads<G>), 0, s, a);
  });
}

hipError_t launch_norm_forward(const NormCall& c, hipStream_t s) {
  if (c.T == 0) return hipSuccess;
  const NormArgs a = norm_args(c);
  if (c.dtype == GIFT_BF16) norm_fwd_t<Bf16>(a, s);
  else if (c.dtype == GIFT_FP16) norm_fwd_t<Fp16>(a, s);
  else norm_fwd_t<float>(a, s);
  return hipGetLastError();
}

template <typename T, bool CK>
static void norm_bwd_t(const NormArgs& a, int grid, hipStream_t s) {
  norm_variant(a.d, [&](auto g, auto ch) {
    constexpr int G = decltype(g)::value, CH = decltype(ch)::value;
    hipLaunchKernelGGL((k_norm_bwd<T, CK, G, CH>), dim3((unsigned)grid), dim3(kNormThreads<G>), 0, s, a);
  });
}

// Whether dx shares memory with dy or x (it may be either).
static bool norm_in_place(const NormCall& c) {
  const int64_t size = c.dtype == GIFT_FP32 ? 4 : 2;
  auto end = [&](const void* p, int64_t ld) { return (uintptr_t)p + (size_t)(((c.T - 1) * ld + c.d) * size); };
  auto meet = [&](const void* p, int64_t ld) {
    return p && c.T > 0 && (uintptr_t)p < end(c.y, c.ldy) && (uintptr_t)c.y < end(p, ld);
  };
  return meet(c.dy, c.lddy) || meet(c.x, c.ldx);
}

hipError_t launch_norm_backward(const NormCall& c, float* part, float* dw, float* db, int accumulate, hipStream_t s) {
  NormArgs a = norm_args(c);
  const int step = norm_step_rows(c.d);
  a.P = norm_partials(c.T, c.d);
  a.steplog = __builtin_ctz((unsigned)(norm_group_rows(c.d) / step));
  a.sums = db ? 2 : 1;
  const bool direct = c.T <= kDirectRows;
  if (direct) {
    a.steplog = 0;
    const int64_t all = cdiv(c.T, step), most = c.d > 8192 ? 128 : c.d > 2048 ? 256 : 512;
    a.P = (int)(all < most ? all : most);
    a.dw = dw;
    a.db = db;
    a.accumulate = accumulate;
  } else {
    a.part = part;
  }
  a.groups = cdiv(c.T, step << a.steplog);
  auto launch = [&](int grid) {
    if (c.ckpt) {
      if (c.dtype == GIFT_BF16) norm_bwd_t<Bf16, true>(a, grid, s);
      else if (c.dtype == GIFT_FP16) norm_bwd_t<Fp16, true>(a, grid, s);
      else norm_bwd_t<float, true>(a, grid, s);
    } else {
      if (c.dtype == GIFT_BF16) norm_bwd_t<Bf16, false>(a, grid, s);
      else if (c.dtype == GIFT_FP16) norm_bwd_t<Fp16, false>(a, grid, s);
      else norm_bwd_t<float, false>(a, grid, s);
    }
  };
  const int rows = a.P, columns = direct && part ? (int)cdiv(c.d, kActBlock) : 0;
  if (columns && norm_in_place(c)) {
    // all columns are read before any row is written
    a.P = 0;
    launch(columns);
    a.P = rows;
    if (rows) launch(rows);
  } else if (rows + columns) {
    launch(rows + columns);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (a.part)
    hipLaunchKernelGGL(k_norm_reduce, dim3((unsigned)cdiv(a.sums * (int64_t)c.d, kReduceCols)),
                       dim3(kReduceCols * kReduceRows), 0, s, part, a.P, c.d, a.sums * c.d, dw, db, accumulate);
  return hipGetLastError();
}

}  // namespace gift
