// Losses of the NVFP4 lm_head over its whole vocabulary, with their gradients
// (gfx950).
//
//   z[t, n] = gsa gsw sum_d xhat[t, d] what[n, d],   xhat, what = q S
//   lmhead_loss:    lse = log sum_n e^z;  loss = lse - z[t, target]
//   lmhead_distill: q = softmax(z / tau), p = softmax(teacher / tau) over the
//                   teacher's K tokens;  loss = tau^2 sum_j p_j (log p_j - log q_j)
//   both:           dx = weight gsw tau sum_n (q_n - p_n) what[n]
// Cross entropy is the case of one token with p = 1 and tau = 1.
//
// The vocabulary is taken in pieces. A piece's products stay in registers and
// give each row a maximum and a sum for every block of columns
// (softmax_block.hpp); with a gradient they also leave the columns' weights
// e = 2^(y - m), fp16 (of a piece: 512 MB, T x N where that is less), and a second
// product sum_n e[t, n] what[n] is added to what the pieces before gave. The
// weights of a piece are those of the softmax up to a factor per row, which the
// pieces after may change: as a row's maximum rises, its sums so far shrink. So
// the gradient needs two products, not the three of computing the logits again
// once their sum is known.
//
// The K tokens of the loss do not take part in that second product: their
// weights are set to zero there, and q_j - p_j, in fp32, multiplies their rows
// at the end. Where q is near p nothing is lost to fp16.
//
// Their logits are those of the first product, left by the tiles that hold them,
// and everything of them is taken as a difference from the row's m. So q <= 1 and
// loss >= 0 hold at any temperature; what the temperature magnifies is the
// rounding of the logits alone, 2^-24 of |z / tau| and their sums' over D.
#include "../../include/nvfp4_router.h"
#include "experts_tile.hpp"

#include <algorithm>
#include <cmath>

namespace nvr {

constexpr int kHeadTokens = 1024;  // ROUTER_MAX_TEACHER
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// ---------------------------------------------------------------------------
// The tokens of the loss.
// ---------------------------------------------------------------------------
// A row's tokens that the gradient multiplies by themselves: q - p, for each
// place that names a token.
struct TokenList {
  int count;  // -1: the row has no gradient
  int pad;
  int token[kHeadTokens];
  float coef[kHeadTokens];
};

struct HeadArgs {
  const uint8_t* xc;
  const uint8_t* xs;
  const float* gsa;
  const uint8_t* wc;
  const uint8_t* ws;
  const float* gsw;
  int T, D, N, K;
  const int32_t* tokens;  // [T, K]
  const void* teacher;    // NULL (cross entropy: K = 1, p = 1) or [T, K]
  int teacher_bf16;
  float tau;
  const float* weight;  // NULL (1) or [T]
  const float* named;   // [T, K]: y of the tokens
  const float2* stats;  // [T, blocks] (m, s), the first `used` of each row
  int blocks, used;
  float* loss;
  float* lse;
  float* logq;  // [T, K]; NULL for cross entropy
  void* dx;     // bf16 [T, D]
  TokenList* lists;  // with a gradient: [T]
};

__device__ __forceinline__ float teacher_at(const HeadArgs& a, int64_t i) {
  return a.teacher_bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.teacher)[i] << 16)
                        : static_cast<const float*>(a.teacher)[i];
}
// teacher_at over tau, from its row's largest: no quotient overflows.
__device__ __forceinline__ float teacher_below(const HeadArgs& a, int64_t i, float top) {
  return (teacher_at(a, i) - top) / a.tau;
}

// s 2^by for whole by <= 0, exact but where it ends below fp32's numbers. "Nothing
// yet" is s = 0 and not m = -infinity: maxima leave NaN out, so logits of NaN
// alone have (-infinity, NaN), and that NaN has to reach the row's sum. (by is
// NaN where both m are -infinity.)
__device__ __forceinline__ float soft_scaled(float s, float by) {
  return ldexpf(s, (int)fmaxf(by, -1000.0f));
}

__device__ __forceinline__ float2 soft_join(float2 a, float2 b) {
  const float m = fmaxf(a.x, b.x);
  return make_float2(m, soft_scaled(a.y, a.x - m) + soft_scaled(b.y, b.x - m));
}

__device__ __forceinline__ float2 wave_join(float2 v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = soft_join(v, make_float2(__shfl_xor(v.x, o), __shfl_xor(v.y, o)));
  return v;
}

// Teacher's largest entry and sum of exponentials of row t, over entries that
// name a token: (m, sum); sum 0 for a row without any. Every wavefront takes
// the whole row.
__device__ __forceinline__ float2 teacher_row(const HeadArgs& a, int64_t t) {
  const int lane = threadIdx.x & 63;
  float m = -__builtin_inff();
  bool nan = false;  // one of a token that counts; a maximum leaves it out
  for (int j = lane; j < a.K; j += 64) {
    const int n = a.tokens[t * a.K + j];
    if (n >= 0 && n < a.N) {
      const float v = teacher_at(a, t * a.K + j);
      nan = nan || v != v;
      m = fmaxf(m, v);
    }
  }
  m = wave_max(m);
  if (__ballot(nan)) return make_float2(__builtin_nanf(""), __builtin_nanf(""));
  if (!(m > -__builtin_inff())) return make_float2(0.0f, 0.0f);
  float s = 0.0f;
  for (int j = lane; j < a.K; j += 64) {
    const int n = a.tokens[t * a.K + j];
    if (n >= 0 && n < a.N) s += expf(teacher_below(a, t * a.K + j, m));
  }
  return make_float2(m, wave_sum(s));
}

// (m, s) of n blocks, by NT threads of which this is one; 16 loads in flight.
template <int NT>
__device__ __forceinline__ float2 thread_join(const float2* st, int n) {
  constexpr int Q = 16;
  float2 v = make_float2(-__builtin_inff(), 0.0f);
  for (int i0 = threadIdx.x; i0 < n; i0 += Q * NT) {
    float2 u[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) u[q] = i0 + q * NT < n ? st[i0 + q * NT] : make_float2(-__builtin_inff(), 0.0f);
    float m = v.x;
#pragma unroll
    for (int q = 0; q < Q; ++q) m = fmaxf(m, u[q].x);
    float s = soft_scaled(v.y, v.x - m);
#pragma unroll
    for (int q = 0; q < Q; ++q) s += soft_scaled(u[q].y, u[q].x - m);
    v = make_float2(m, s);
  }
  return v;
}

// ---------------------------------------------------------------------------
// Logits of a piece: the experts' tiles, one matrix, with softmax_block.hpp's
// epilogue. D = 7168, N = 129280 (521 MB of weights), the kernel alone:
//   stream  T = 1 84 us, T = 32 with 64 tokens a row 102: HBM, 6.2 and 5.1 TB/s of
//           reads (1 us for the search for the tokens);
//   wide    T = 1024 1.54 ms, T = 4096 6.0 (1.24 and 1.26 PFLOP/s), keeping the
//           weights 1.64 and 6.4: the matrix cores, 64 to 68 % busy at the 1.9
//           GHz that their power leaves. (Cards differ by 6 %.)
// ---------------------------------------------------------------------------
template <Out M, int MR, int KB, int KG, Scales S, int AUX>
__global__ __launch_bounds__(KG * kEsThreads) void head_stream_kernel(ExpertArgs a, int row_tiles) {
  __shared__ StreamLds<MR, KB, KG> lds;
  // The row tiles of one column tile side by side on one XCD: they read the same weights.
  const int n = xcd_order(blockIdx.x, gridDim.x), ct = n / row_tiles, row0 = (n - ct * row_tiles) * MR;
  const ExpertTile tile{{0, row0, min(MR, a.R - row0)}, ct};
  stream_tile<M, MR, KB, KG, S, AUX>(a, tile, lds);
}

template <Out M, Scales S>
__global__ __launch_bounds__(kEtThreads) __attribute__((amdgpu_waves_per_eu(2, 2))) void head_wide_kernel(
    ExpertArgs a, int row_tiles, int tile_rows) {
  __shared__ TileLds lds;
  const int n = xcd_order(blockIdx.x, gridDim.x), ct = n / row_tiles, row0 = (n - ct * row_tiles) * tile_rows;
  const ExpertTile tile{{0, row0, min(tile_rows, a.R - row0)}, ct};
  const int nr = tile.rt.nr;
  if (nr > 96) wide_tile<M, 4, S>(a, tile, lds);
  else if (nr > 64) wide_tile<M, 3, S>(a, tile, lds);
  else if (nr > 32) wide_tile<M, 2, S>(a, tile, lds);
  else wide_tile<M, 1, S>(a, tile, lds);
}

// ---------------------------------------------------------------------------
// The rows' losses.
// ---------------------------------------------------------------------------
// A row's loss by its workgroup, from its logits' sum (m, s).
constexpr int kTokWaves = 4;
struct TokLds {
  float2 part[kTokWaves];
  float terms[kTokWaves], lz[kHeadTokens];
  alignas(16) int tk[kHeadTokens];
};

// (m, s) of a row's blocks, by a workgroup of kTokWaves wavefronts.
__device__ __forceinline__ float2 row_join(const float2* st, int n, TokLds& lds) {
  float2 v = wave_join(thread_join<64 * kTokWaves>(st, n));
  if ((threadIdx.x & 63) == 0) lds.part[threadIdx.x >> 6] = v;
  __syncthreads();
  v = lds.part[0];
#pragma unroll
  for (int w = 1; w < kTokWaves; ++w) v = soft_join(v, lds.part[w]);
  return v;
}

__device__ __forceinline__ void row_loss(const HeadArgs& a, int64_t t, float2 v, TokLds& lds) {
  float (&terms)[kTokWaves] = lds.terms, (&lz)[kHeadTokens] = lds.lz;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const float lsum = logf(v.y);  // log sum, from m on
  float2 tr = make_float2(0.0f, 1.0f);  // log p = 0 for cross entropy
  if (a.teacher) tr = teacher_row(a, t);
  const float logs = a.teacher ? logf(tr.y) : 0.0f;
  float sum = 0.0f;
  for (int j = threadIdx.x; j < a.K; j += 64 * kTokWaves) {
    const int n = a.tokens[t * a.K + j];
    lds.tk[j] = n;
    float logq = 0.0f;
    if (n >= 0 && n < a.N) {
      const float y = a.named[t * a.K + j] - v.x;  // (logq itself is where they stand, if there is one)
      lz[j] = y;
      logq = y * kLn2 - lsum;
      if (logq > 0.0f) logq = 0.0f;  // by the roundings of these two
      if (a.teacher) {
        const float lp = teacher_below(a, t * a.K + j, tr.x) - logs, p = expf(lp);
        if (p != 0.0f) sum += p * (lp - logq);  // p log p is 0 at 0
      } else {
        sum = 0.0f - logq;
      }
    }
    if (a.logq) a.logq[t * a.K + j] = logq;
  }
  sum = wave_sum(sum);
  if (lane == 0) terms[wave] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    float l = terms[0];
#pragma unroll
    for (int w = 1; w < kTokWaves; ++w) l += terms[w];
    a.loss[t] = tr.y == 0.0f ? 0.0f : l * a.tau * a.tau;
    a.lse[t] = v.x * kLn2 + lsum;
  }
  if (!a.lists) return;
  // q - p of each place. A token named more than once has its q at its first
  // place: every place looks at all before it, four at a time. (T = 30, K = 1024,
  // D = 7168: 367 us for the whole call; by one wavefront, a place at a time, 946.)
  const int* tk = lds.tk;
  for (int j = threadIdx.x; j < a.K; j += 64 * kTokWaves) {
    const int n = tk[j];
    int again = 0;
    const int upto = min((j | 63) + 1, a.K);  // of the wavefront
#pragma unroll 4
    for (int i = 0; i < upto; i += 4) {
      const int4 o = *reinterpret_cast<const int4*>(tk + i);
      again |= (int)(o.x == n && i < j) | (int)(o.y == n && i + 1 < j) | (int)(o.z == n && i + 2 < j) | (int)(o.w == n && i + 3 < j);
    }
    if (n >= 0 && n < a.N) {
      const float p = a.teacher ? expf(teacher_below(a, t * a.K + j, tr.x)) / tr.y : 1.0f;
      // 2^y as in the sum, which holds it: the quotient is 1 at most.
      lz[j] = (again ? 0.0f : __builtin_amdgcn_exp2f(lz[j]) / v.y) - p;
    }
  }
  __syncthreads();
  // The first wavefront lists the places that name a token, in order.
  if (wave != 0) return;
  TokenList& list = a.lists[t];
  int out = 0;
  for (int j0 = 0; j0 < a.K; j0 += 64) {
    const int j = j0 + lane;
    const int n = j < a.K ? tk[j] : -1;
    const bool valid = n >= 0 && n < a.N;
    const uint64_t bal = __ballot(valid);
    if (valid) {
      const int at = out + (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(bal >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)bal, 0u));
      list.token[at] = n;
      list.coef[at] = lz[j];
    }
    out += (int)__popcll(bal);
  }
  if (lane == 0) list.count = out == 0 || tr.y == 0.0f ? -1 : out;
}

// Without a gradient: the end of a row, from its blocks' (m, s). Latency at few
// rows (4.9 us at T = 1, N = 129280: 4040 blocks, 32 KB); T = 4096 with 2020
// blocks each: 15 us, 4.5 TB/s.
__global__ __launch_bounds__(64 * kTokWaves) void head_tokens_kernel(HeadArgs a) {
  __shared__ TokLds lds;
  const int64_t t = blockIdx.x;
  row_loss(a, t, row_join(a.stats + t * a.blocks, a.used, lds), lds);
}

// ---------------------------------------------------------------------------
// Gradient, per piece: one scale for a row's weights.
// ---------------------------------------------------------------------------
struct NormArgs {
  const float2* stats;  // [T, blocks]: those of this piece come first in each row
  int blocks, used;
  const float2* before;     // NULL or [T]: (m, s) of the pieces before
  float2* after;            // [T]
  float* shrink;            // [T]: factor of the sums so far
  float* ref;               // [T]: m for the next piece
  _Float16* e;
  int64_t ld_e;
  int T, K, n0, cols;
  const int32_t* tokens;
};

// One workgroup per row. LAST: the sums are complete, and it goes on to the
// row's loss. 5.0 us at T = 203, 6.4 with 37 tokens, 16 at T = 4096: latency.
constexpr int kNormThreads = 64 * kTokWaves;
template <bool LAST>
__global__ __launch_bounds__(kNormThreads) void head_norm_kernel(NormArgs a, HeadArgs ha) {
  __shared__ TokLds lds;
  const int64_t t = blockIdx.x;
  const float2* st = a.stats + t * a.blocks;
  float2 v = row_join(st, a.used, lds);
  const float2 old = a.before ? a.before[t] : make_float2(-__builtin_inff(), 0.0f);
  v = soft_join(v, old);
  if (threadIdx.x == 0) {
    a.after[t] = v;
    a.shrink[t] = a.before ? soft_scaled(1.0f, old.x - v.x) : 0.0f;
    a.ref[t] = v.x;
  }
  // The named tokens' own weights.
  _Float16* e = a.e + t * a.ld_e;
  for (int j = threadIdx.x; j < a.K; j += kNormThreads) {
    const int64_t c = (int64_t)a.tokens[t * a.K + j] - a.n0;
    if (c >= 0 && c < a.cols) e[weight_place(c)] = (_Float16)0.0f;
  }
  if (LAST) row_loss(ha, t, v, lds);
}

// ---------------------------------------------------------------------------
// Gradient, per piece: sum_n e[t, n] what[n, d].
//
// The product runs over the weights' rows, whose codes lie along d. The words
// of two rows (weight_place's neighbours) are put together so that each byte
// holds one column's codes of both: a conversion of a byte then gives what MFMA
// wants, one column's values of two n.
//
// Tiles of up to 128 rows times 512 columns, 8 wavefronts, two per SIMD,
// 32x32x16 MFMAs, 128 weight rows per step.
//  * Weights: loaded in whole lines by the workgroup (8 rows x 8 bytes per
//    thread), bytes transposed in registers, and kept in LDS as [byte
//    column][n], so that a lane reads its two columns' codes of 16 rows at
//    once. Wavefront w takes the columns 16 r + 2 w and 16 r + 2 w + 1 of lane
//    r, all in the scale block r. Scales likewise, as [block][n].
//  * Softmax weights: on their way into LDS they are brought to the row's m
//    from their block's, by a power of two.
//  * K order: in every 64 rows lane (r, h) supplies [16 h + 4 j, +4) and those
//    32 further on to MFMA j.
// All double-buffered in LDS, one barrier per step; a step's loads go out a step
// before they are written there.
// D = 7168, N = 129280: T = 4096 6.4 ms for the two pieces (1.18 PFLOP/s), T =
// 1024 1.65, bound by the matrix cores (68 % busy) and their power as the logits'
// tiles (cards differ by 6 %);
// with few rows by the weights (T = 1 to 8: 117 us for 521 MB, 4.5 TB/s), then
// by splits that leave a workgroup few steps (T = 203, D = 2080, N = 32003: 48
// us for 27 GFLOP, 11 steps and 39 MB of sums).
// Fragments read and converted between the MFMAs rather than ahead of them:
// 14.1 -> 13.7 ms for the whole call at T = 4096; scales kept in fp16: 13.4 ->
// 12.9; sums through LDS: T = 203 131 -> 113 us.
// ---------------------------------------------------------------------------
constexpr int kGwThreads = 512;
constexpr int kGwRows = 128, kGwCols = 512, kGwStep = 128;
constexpr int kGwLd = 144;       // LDS bytes per byte column: 128 rows and 16 of padding
constexpr int kGwScaleLd = 272;  // and per scale block

// Tiles in bands of 8 row tiles, column tile by column tile, so that 32
// neighbours read 8 rows' softmax weights and 4 columns' weights. The first
// `full`, whole rounds of 256 workgroups, take all of a piece's rows; each of
// the others is shared by `splits` workgroups that take a part of the rows
// each, so that the last rounds are full too.
struct GradTiles {
  int row_tiles, col_tiles, full, splits;
  __host__ __device__ int count() const { return row_tiles * col_tiles; }
  __device__ __forceinline__ void place(int t, int& rt, int& ct) const {
    const int band = t / (8 * col_tiles), in = t - band * 8 * col_tiles, bandrows = min(8, row_tiles - 8 * band);
    ct = in / bandrows;
    rt = 8 * band + in - ct * bandrows;
  }
  __device__ __forceinline__ int parts(int rt, int ct) const {  // sums of a tile
    const int band = rt >> 3, bandrows = min(8, row_tiles - 8 * band);
    return 8 * band * col_tiles + ct * bandrows + (rt & 7) < full ? 1 : splits;
  }
};

struct GradArgs {
  const _Float16* e;
  int64_t ld_e;
  const uint8_t* wc;  // of the piece
  const uint8_t* ws;
  int T, D, cols;
  float* part;          // [splits, T, D]
  const float* shrink;  // NULL: the first piece
  const float2* stats;  // [T, blocks] of the piece
  int blocks, block_shift;
  const float* ref;     // [T]: the row's m
  GradTiles tiles;
};

// (And the sums of 64 rows on their way out.)
struct GradLds {
  alignas(16) _Float16 x[2][kGwRows * kGwStep];
  alignas(16) uint8_t codes[2][(kGwCols / 2) * kGwLd];
  alignas(16) uint8_t scales[2][(kGwCols / 16) * kGwScaleLd];  // fp16
};
static_assert(sizeof(GradLds) >= 64 * kGwCols * sizeof(float));

// Halves offset of 16-byte piece c (of 16) of row r of the softmax weights.
__device__ __forceinline__ int grad_x_at(int r, int c) {
  return (((r >> 5) * 16 + c) * 32 + ((r & 31) ^ (4 * (c & 3)))) * 8;
}

// Bytes 0 .. 3 of four words -> four words of one byte place each.
__device__ __forceinline__ void byte_transpose4(const uint32_t (&a)[4], uint32_t (&o)[4]) {
  const uint32_t t0 = __builtin_amdgcn_perm(a[1], a[0], 0x05010400u), t1 = __builtin_amdgcn_perm(a[1], a[0], 0x07030602u);
  const uint32_t t2 = __builtin_amdgcn_perm(a[3], a[2], 0x05010400u), t3 = __builtin_amdgcn_perm(a[3], a[2], 0x07030602u);
  o[0] = __builtin_amdgcn_perm(t2, t0, 0x05040100u);
  o[1] = __builtin_amdgcn_perm(t2, t0, 0x07060302u);
  o[2] = __builtin_amdgcn_perm(t3, t1, 0x05040100u);
  o[3] = __builtin_amdgcn_perm(t3, t1, 0x07060302u);
}

// S4: rows of scales start at multiples of 4 bytes (D a multiple of 64).
template <int RT, bool S4>
__device__ __forceinline__ void grad_tile(const GradArgs& a, int row0, int nr, int ct, int split, int steps,
                                          GradLds& lds) {
  typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
  const int tid = threadIdx.x, lane = tid & 63, r = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t rowc = a.D / 2, rows = a.D / 16;
  const int d0 = ct * kGwCols;
  const int n0 = split * steps * kGwStep, n1 = min(n0 + steps * kGwStep, a.cols);
  const int64_t nrows = max(n1 - n0, 0);
  const int nsteps = (int)((nrows + kGwStep - 1) / kGwStep);
  const __amdgpu_buffer_rsrc_t wcr = make_rsrc(a.wc + n0 * rowc, nrows * rowc);
  const __amdgpu_buffer_rsrc_t wsr = make_rsrc(a.ws + n0 * rows, nrows * rows);
  // Codes: rows 8 o .. 8 o + 7 of a step, bytes 8 c .. 8 c + 7 of the tile's 256.
  const int o = tid >> 5, c = tid & 31;
  const uint32_t oc = d0 + 16 * c < a.D ? (uint32_t)(8 * o * rowc + d0 / 2 + 8 * c) : kMmaOob;
  u32x2_t wv[8];
  // Scales: rows pn and pn + 32, blocks 4 b .. 4 b + 3 of the tile's 32.
  const int p = tid >> 3, b = tid & 7, pn = p + (p & 32);
  const uint32_t os = d0 + 64 * b < a.D ? (uint32_t)(pn * rows + d0 / 16 + 4 * b) : kMmaOob;
  const uint32_t os2 = d0 + 64 * b + 32 < a.D ? os + 2 : kMmaOob;
  uint32_t sv[2][2];
  // Softmax weights: row ar, 16-byte pieces aq, aq + 4, aq + 8, aq + 12.
  const int ar = tid >> 2, aq = tid & 3;
  const bool arow = ar < nr;
  const __amdgpu_buffer_rsrc_t er = make_rsrc(a.e + (int64_t)row0 * a.ld_e, (int64_t)nr * a.ld_e * 2);
  const uint32_t oe = arow ? (uint32_t)(ar * a.ld_e * 2 + 2 * (n0 + 8 * aq)) : kMmaOob;
  const float2* st = a.stats + (int64_t)(row0 + (arow ? ar : 0)) * a.blocks;
  const float ref = a.ref[row0 + (arow ? ar : 0)];
  u32x4_t ev[4];
  float mv[4];
  // A step's loads and stores, half the softmax weights or half the codes at a time. Weights' rows past the split's
  // are zeros; softmax weights past its last step are not wanted, and its last step's are read again.
  const int last = nsteps - 1;
  auto load_x = [&](int s, int u) {
#pragma unroll
    for (int i = 2 * u; i < 2 * u + 2; ++i) {
      mv[i] = st[(n0 + kGwStep * min(s, last) + 32 * i) >> a.block_shift].x;
      ev[i] = __builtin_bit_cast(
          u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(er, oe + 2 * (kGwStep * min(s, last) + 32 * i), 0, 0));
    }
  };
  auto store_x = [&](int buf, int u) {
#pragma unroll
    for (int i = 2 * u; i < 2 * u + 2; ++i) {
      // A power of two, in two factors where one would be below fp16's normal numbers.
      const float by = mv[i] - ref;
      const _Float16 f = (_Float16)__builtin_amdgcn_exp2f(fmaxf(by, -14.0f));
      const _Float16 g = (_Float16)__builtin_amdgcn_exp2f(fminf(by + 14.0f, 0.0f));
      const bool low = __ballot(by < -14.0f) != 0;
      half8_t v = __builtin_bit_cast(half8_t, ev[i]);
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] *= f;
      if (low) {
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] *= g;
      }
      *reinterpret_cast<half8_t*>(&lds.x[buf][grad_x_at(ar, 4 * i + aq)]) = v;
    }
  };
  auto load_w = [&](int s) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      wv[i] = __builtin_bit_cast(
          u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(wcr, oc + (uint32_t)((kGwStep * s + i) * rowc), 0, 0));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t at = (uint32_t)((kGwStep * s + 32 * i) * rows);
      if constexpr (S4) sv[i][0] = __builtin_amdgcn_raw_buffer_load_b32(wsr, os + at, 0, 0);
      else {
        sv[i][0] = __builtin_amdgcn_raw_buffer_load_b16(wsr, os + at, 0, 0);
        sv[i][1] = __builtin_amdgcn_raw_buffer_load_b16(wsr, os2 + at, 0, 0);
      }
    }
  };
  auto store_c = [&](int buf, int w) {
    uint32_t lo[4], hi[4];
    byte_transpose4({wv[0][w], wv[1][w], wv[2][w], wv[3][w]}, lo);
    byte_transpose4({wv[4][w], wv[5][w], wv[6][w], wv[7][w]}, hi);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<u32x2_t*>(&lds.codes[buf][((4 * w + i) * 32 + c) * kGwLd + 8 * o]) = u32x2_t{lo[i], hi[i]};
  };
  auto store_s = [&](int buf) {
    const uint32_t s0 = S4 ? sv[0][0] : sv[0][0] | (sv[0][1] << 16), s1 = S4 ? sv[1][0] : sv[1][0] | (sv[1][1] << 16);
    const uint32_t t0 = __builtin_amdgcn_perm(s1, s0, 0x05010400u), t1 = __builtin_amdgcn_perm(s1, s0, 0x07030602u);
    // Of each block a row's scale next to that of the row 32 further on.
    uint8_t* d = &lds.scales[buf][4 * b * kGwScaleLd + 4 * p];
    *reinterpret_cast<half2_t*>(d) = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(t0, 1.0f, false);
    *reinterpret_cast<half2_t*>(d + kGwScaleLd) = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(t0, 1.0f, true);
    *reinterpret_cast<half2_t*>(d + 2 * kGwScaleLd) = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(t1, 1.0f, false);
    *reinterpret_cast<half2_t*>(d + 3 * kGwScaleLd) = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(t1, 1.0f, true);
  };

  f32x16_t acc[RT][2];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][m][v] = 0.0f;

  // A step is 8 slices of 16 rows. In a slice the MFMAs of the even columns run
  // while the odd columns' weights of the slice are converted, then the other
  // way round for the next slice; softmax weight fragment i is read right
  // after its last MFMA of the slice before, the codes of two slices during the
  // last slice before them. The step's one barrier stands before its last
  // slice: by then every wavefront has read this buffer to the end and written
  // the next one, whose first fragments the last slice reads.
  half8_t A[RT], w[2];
  u32x2_t cx, cy;  // codes of two slices, rows n and n + 32
  u32x4_t sw[2];   // their scales
  uint32_t col[2];
  half2_t sc[4];
  auto afrag = [&](int i, int buf, int sl) {
    return *reinterpret_cast<const half8_t*>(&lds.x[buf][grad_x_at(32 * i + r, 8 * (sl >> 2) + 4 * h + (sl & 3))]);
  };
  auto read_codes = [&](int buf, int pair) {
    const uint8_t* at = &lds.codes[buf][(wave * 32 + r) * kGwLd + 64 * (pair >> 1) + 16 * h + 8 * (pair & 1)];
    cx = *reinterpret_cast<const u32x2_t*>(at);
    cy = *reinterpret_cast<const u32x2_t*>(at + 32);
    const uint8_t* st = &lds.scales[buf][r * kGwScaleLd + 128 * (pair >> 1) + 64 * h + 32 * (pair & 1)];
    sw[0] = *reinterpret_cast<const u32x4_t*>(st);
    sw[1] = *reinterpret_cast<const u32x4_t*>(st + 16);
  };
  auto prepare = [&](auto jc) {  // columns and scales of a slice
    constexpr int j = decltype(jc)::value;
    const uint32_t x = cx[j], y = cy[j];
    col[0] = (x & 0x0F0F0F0Fu) | ((y << 4) & 0xF0F0F0F0u);
    col[1] = ((x >> 4) & 0x0F0F0F0Fu) | (y & 0xF0F0F0F0u);
#pragma unroll
    for (int k = 0; k < 4; ++k) sc[k] = __builtin_bit_cast(half2_t, (uint32_t)sw[j][k]);
  };
  auto convert = [&](auto mc, auto kc) {
    constexpr int m = decltype(mc)::value, k = decltype(kc)::value;
    reinterpret_cast<half2_t*>(&w[m])[k] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(col[m], 1.0f, k) * sc[k];
  };
  if (nsteps > 0) {
    load_x(0, 0);
    load_x(0, 1);
    load_w(0);
    store_x(0, 0);
    store_x(0, 1);
    store_c(0, 0);
    store_c(0, 1);
    store_s(0);
    load_x(1, 0);
    load_x(1, 1);
    load_w(1);
    __syncthreads();
    read_codes(0, 0);
#pragma unroll
    for (int i = 0; i < RT; ++i) A[i] = afrag(i, 0, 0);
    prepare(IntC<0>{});
    static_for<0, 4>([&](auto kc) { convert(IntC<0>{}, kc); });
  }
  for (int s = 0; s < nsteps; ++s) {
    const int buf = s & 1;
    static_for<0, 8>([&](auto slc) {
      constexpr int sl = decltype(slc)::value;
      if constexpr (sl == 7) __syncthreads();
      if constexpr (sl & 1) read_codes(sl == 7 ? buf ^ 1 : buf, ((sl >> 1) + 1) & 3);
      static_for<0, RT>([&](auto ic) {
        constexpr int i = decltype(ic)::value;
        acc[i][0] = mfma32(A[i], w[0], acc[i][0]);
        static_for<i * 4 / RT, (i + 1) * 4 / RT>([&](auto kc) { convert(IntC<1>{}, kc); });
        __builtin_amdgcn_sched_barrier(0);
      });
      prepare(IntC<(sl + 1) & 1>{});
      static_for<0, RT>([&](auto ic) {
        constexpr int i = decltype(ic)::value;
        acc[i][1] = mfma32(A[i], w[1], acc[i][1]);
        A[i] = afrag(i, sl == 7 ? buf ^ 1 : buf, (sl + 1) & 7);
        static_for<i * 4 / RT, (i + 1) * 4 / RT>([&](auto kc) { convert(IntC<0>{}, kc); });
        __builtin_amdgcn_sched_barrier(0);
      });
      // The next step's data into LDS, the one after's from memory.
      if constexpr (sl == 0 || sl == 1) {
        store_x(buf ^ 1, sl);
        load_x(s + 2, sl);
      }
      if constexpr (sl == 2 || sl == 3) store_c(buf ^ 1, sl - 2);
      if constexpr (sl == 4) {
        store_s(buf ^ 1);
        load_w(s + 2);
      }
    });
  }

  // Value v of lane (r, h): row 8 (v / 4) + 4 h + v % 4 of its 32-row tile,
  // columns 16 r + 2 wave and the next. To memory through LDS, 64 rows at a
  // time: stores of 8 bytes 64 apart would be one line each. In LDS every 16
  // columns are turned round by 2 (r / 4), for the banks.
  float* sums = reinterpret_cast<float*>(&lds);
  static_for<0, (RT + 1) / 2>([&](auto pc) {
    constexpr int i0 = 2 * decltype(pc)::value;
    __syncthreads();
    static_for<i0, (i0 + 2 < RT ? i0 + 2 : RT)>([&](auto ic) {
      constexpr int i = decltype(ic)::value;
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int row = 32 * (i - i0) + 8 * (v >> 2) + 4 * h + (v & 3);
        *reinterpret_cast<float2*>(sums + row * kGwCols + 16 * r + ((2 * wave + 2 * (r >> 2)) & 15)) =
            make_float2(acc[i][0][v], acc[i][1][v]);
      }
    });
    __syncthreads();
    const int q = 4 * (tid & (kGwCols / 4 - 1)), g = q >> 4, turn = 2 * (g >> 2);
    const int at0 = 16 * g + (((q & 15) + turn) & 15), at1 = 16 * g + (((q & 15) + 2 + turn) & 15);
    if (d0 + q < a.D) {
#pragma unroll 4
      for (int row = tid / (kGwCols / 4); row < min(64, nr - 32 * i0); row += kGwThreads / (kGwCols / 4)) {
        f32x4_t* out = reinterpret_cast<f32x4_t*>(a.part + ((int64_t)split * a.T + row0 + 32 * i0 + row) * a.D + d0 + q);
        const float2 lo = *reinterpret_cast<const float2*>(sums + row * kGwCols + at0);
        const float2 hi = *reinterpret_cast<const float2*>(sums + row * kGwCols + at1);
        f32x4_t y = {lo.x, lo.y, hi.x, hi.y};
        if (a.shrink) {
          const float f = a.shrink[row0 + 32 * i0 + row];
          const f32x4_t old = *out;
#pragma unroll
          for (int u = 0; u < 4; ++u) y[u] = fmaf(old[u], f, y[u]);
        }
        *out = y;
      }
    }
  });
}

template <bool S4>
__global__ __launch_bounds__(kGwThreads) __attribute__((amdgpu_waves_per_eu(2, 2))) void head_grad_kernel(
    GradArgs a) {
  __shared__ GradLds lds;
  const GradTiles& tl = a.tiles;
  const int rest = tl.count() - tl.full;
  int t = blockIdx.x, split = 0, steps = (a.cols + kGwStep - 1) / kGwStep;
  if (t < tl.full) {
    t = xcd_order(t, tl.full);
  } else {
    const int n = xcd_order(t - tl.full, rest * tl.splits);
    split = n / rest;
    t = tl.full + n - split * rest;
    steps = (steps + tl.splits - 1) / tl.splits;
  }
  int rt, ct;
  tl.place(t, rt, ct);
  const int row0 = rt * kGwRows, nr = min(kGwRows, a.T - row0);
  if (nr > 96) grad_tile<4, S4>(a, row0, nr, ct, split, steps, lds);
  else if (nr > 64) grad_tile<3, S4>(a, row0, nr, ct, split, steps, lds);
  else if (nr > 32) grad_tile<2, S4>(a, row0, nr, ct, split, steps, lds);
  else grad_tile<1, S4>(a, row0, nr, ct, split, steps, lds);
}

// dx: the splits' sums, divided by the softmax's, and the loss's own tokens.
// SHARE: a workgroup's 8 wavefronts share 512 columns, each a part of the
// splits and tokens, joined in a fixed order; otherwise each of four has 512
// of its own. Few workgroups of 512 columns share, up to more of them the more
// tokens there are. us shared and not, one token: 63 workgroups 5.1 and 12.6,
// 448 6.3 and 6.4, 896 9.1 and 8.5, 2842 18.7 and 12.5; 64 tokens: 896 14.9
// and 18.4, 2842 34.6 and 27.4; 1024 tokens: 896 91 and 154, 2842 255 and 228.
// Bound by the sums and the tokens' rows (T = 203, D = 7168, 1024 tokens: 3.7
// TB/s).
struct DxArgs {
  HeadArgs h;
  const float* part;
  GradTiles tiles;
};

template <bool SHARE>
constexpr int dx_waves() {
  return SHARE ? 8 : 4;
}
static bool dx_share(int64_t T, int64_t columns, int64_t K) { return T * columns < (K > kTokWaves ? 2048 : 512); }
template <bool SHARE>
__global__ __launch_bounds__(64 * dx_waves<SHARE>()) void head_dx_kernel(DxArgs a) {
  constexpr int kDxWaves = dx_waves<SHARE>();
  __shared__ float joined[SHARE ? kDxWaves : 1][SHARE ? 64 : 1][9];
  const HeadArgs& h = a.h;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = blockIdx.x;
  const TokenList& list = h.lists[t];
  const int named = list.count;
  const float2 soft = h.stats[t];  // (m, s) of the whole row
  const float f = (h.weight ? h.weight[t] : 1.0f) * load_early(h.gsw) * h.tau, norm = 1.0f / (soft.y * kWeightOne);
  const int d = ((SHARE ? blockIdx.y : blockIdx.y * kDxWaves + wave) * 64 + lane) * 8;
  const int first = SHARE ? wave : 0, step = SHARE ? kDxWaves : 1;
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = 0.0f;
  if (named >= 0 && d < h.D) {
    const int splits = a.tiles.parts((int)(t / kGwRows), d / kGwCols);
    const float* part = a.part + t * h.D + d;
    const int64_t slab = (int64_t)h.T * h.D;
    for (int s0 = first; s0 < splits; s0 += 4 * step) {  // 4 splits' loads in flight
      f32x4_t u[4][2];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x4_t* p = reinterpret_cast<const f32x4_t*>(part + min(s0 + q * step, splits - 1) * slab);
        u[q][0] = p[0];
        u[q][1] = p[1];
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const bool in = s0 + q * step < splits;
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] += in ? u[q][i >> 2][i & 3] : 0.0f;
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] *= norm;
    const uint8_t *wc = h.wc + d / 2, *ws = h.ws + d / 16;
    const int64_t rowc = h.D / 2, rows = h.D / 16;
    for (int j0 = first; j0 < named; j0 += 8 * step) {  // 8 rows' loads in flight
      uint32_t code[8], sb[8];
      float c[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int j = min(j0 + u * step, named - 1);
        const int64_t n = list.token[j];
        c[u] = j0 + u * step < named ? list.coef[j] : 0.0f;
        code[u] = *reinterpret_cast<const uint32_t*>(wc + n * rowc);
        sb[u] = ws[n * rows];
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const half8_t w = fp4x8_to_f16(code[u], e4m3_f16(sb[u]));
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = fmaf(c[u], (float)w[i], y[i]);
      }
    }
  }
  if constexpr (SHARE) {
#pragma unroll
    for (int i = 0; i < 8; ++i) joined[wave][lane][i] = y[i];
    __syncthreads();
    if (wave != 0) return;
#pragma unroll
    for (int w = 1; w < kDxWaves; ++w)
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] += joined[w][lane][i];
  }
  if (d >= h.D) return;
  u32x4_t o = {0u, 0u, 0u, 0u};
  if (named >= 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = bf16_round2(y[2 * i] * f, y[2 * i + 1] * f);
  }
  *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(h.dx) + t * h.D + d) = o;
}

// ---------------------------------------------------------------------------
// Dispatch.
// ---------------------------------------------------------------------------
constexpr int64_t kMaxRange = (int64_t(1) << 31) - 65536;  // bytes a 32-bit buffer offset reaches

// Everything that follows from the sizes. `wide`: the logits' tiles.
struct HeadPlan {
  bool wide;
  int block_shift;   // columns of a statistics block
  int64_t piece;     // columns of a piece, a multiple of 512
  int64_t pieces;
  int64_t blocks;    // statistics blocks per row kept at a time
  GradTiles tiles;   // of the second product
  int64_t ld_e;
  size_t named_at, stats_at, state_at, shrink_at, ref_at, e_at, part_at, lists_at, bytes;
};

static HeadPlan head_plan(int64_t T, int64_t D, int64_t N, bool grad) {
  HeadPlan p{};
  T = std::max(T, int64_t(1));
  // Time over D, in ns, of the stream's 32 x 128 tiles and of the wide kernel, whose 512-column tiles take 64 rows while
  // each compute unit has one at most, else 128 (measured at D = 1056 to 7168, T = 33 to 256, N = 32003 and 129280). The
  // stream: 0.0117 a tile, 0.013 where rows are no multiple of 128 bytes. The wide kernel: a round 13 and 0.046 for 1000
  // weight rows (T = 64, N = 129280: 19), 14 and 0.13 then, as its tiles read lines twice; 4.5 for each 32 rows past 64;
  // 26 for each of several rounds.
  const bool whole = D % 256 == 0;
  const int64_t cols512 = (N + kEtCols - 1) / kEtCols, tiles64 = (T + 63) / 64 * cols512;
  const int64_t tiles128 = (T + 127) / 128 * cols512, tiles32 = (T + 31) / 32 * ((N + 127) / 128);
  double wide_ns = 26.0 * (double)((tiles128 + 255) / 256);
  if (tiles64 <= kOneRound || tiles128 <= kOneRound)
    wide_ns = (whole ? 13.0 + 4.6e-5 * (double)N : 14.0 + 1.3e-4 * (double)N) +
              (tiles64 <= kOneRound ? 0.0 : 4.5 * (double)((std::min(T, int64_t(128)) + 31) / 32 - 2));
  p.wide = T > 32 && wide_ns < std::max(4.8, (whole ? 0.0117 : 0.013) * (double)tiles32);
  p.block_shift = p.wide ? 6 : 5;
  int64_t piece = kMaxRange / (D / 2) / 512 * 512;  // a piece's codes lie within a buffer's range
  // A piece's softmax weights take 512 MB at most, but 4096 columns at least. (T = 2048, D = 7168, N = 129280: 6.44 ms,
  // with 256 MB 6.59, with 1 GB 6.45.)
  if (grad) piece = std::min(piece, std::max((int64_t(1) << 28) / T / 512 * 512, int64_t(4096)));
  // A launch has fewer than 2^32 threads: 512 for a tile of 128 x 512, or of 64 x 512 where those are few.
  piece = std::min(piece, (int64_t(1) << 37) / T / 512 * 512);
  piece = std::max(piece, int64_t(512));
  p.pieces = (N + piece - 1) / piece;
  p.piece = ((N + p.pieces - 1) / p.pieces + 511) / 512 * 512;  // equal pieces
  p.pieces = (N + p.piece - 1) / p.piece;
  const int64_t cols = grad ? p.piece : N;
  p.blocks = (cols + 63) / 64 << (6 - p.block_shift);
  const int64_t rows = std::min(p.piece, N);
  // Whole rounds of 256 workgroups, one on each compute unit, then the tiles left in the splits that end soonest: a
  // split of 1 / s takes 1 / s of a round.
  p.tiles.row_tiles = (int)((T + kGwRows - 1) / kGwRows);
  p.tiles.col_tiles = (int)((D + kGwCols - 1) / kGwCols);
  p.tiles.full = p.tiles.count() / 256 * 256;
  // A tile takes 6 us and for each step 0.25 us and 0.8 for each 32 of its rows, 2.3 at least (the weights'
  // bandwidth); measured 8 to 16 steps, D = 4096: T = 32 2.3 a step, 64 2.35, 96 2.8, 128 3.45. Each split's sums are
  // written and read once more (5 TB/s).
  const int64_t rest = p.tiles.count() - p.tiles.full, most = std::min(int64_t(256), std::max(int64_t(1), rows / 256));
  const double steps = (double)((rows + kGwStep - 1) / kGwStep), sums = (double)T * (double)D * 8e-6 / 5.0;
  const double step_us = std::max(2.3, 0.25 + 0.8 * (double)std::min(int64_t(4), (T + 31) / 32));
  double best = 1e30;
  p.tiles.splits = 1;
  for (int64_t s = 1; grad && rest && s <= most && sums * (double)s < best; ++s) {
    const double us = (6.0 + step_us * std::ceil(steps / (double)s)) * (double)((rest * s + 255) / 256) + sums * (double)s;
    if (us < best) best = us, p.tiles.splits = (int)s;
  }
  p.ld_e = p.piece;
  size_t at = kScratchOffset;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at = (at + bytes + 255) / 256 * 256;
    return here;
  };
  p.named_at = take((size_t)T * sizeof(float));
  p.stats_at = take((size_t)T * p.blocks * sizeof(float2));
  if (grad) {
    p.state_at = take((size_t)T * 2 * sizeof(float2));
    p.shrink_at = take((size_t)T * sizeof(float));
    p.ref_at = take((size_t)T * sizeof(float));
    p.e_at = take((size_t)T * p.ld_e * sizeof(_Float16));
    p.part_at = take((size_t)p.tiles.splits * T * D * sizeof(float));
    p.lists_at = take((size_t)T * sizeof(TokenList));
  }
  p.bytes = at;
  return p;
}

// The weights' loads pass the caches where their lines are read once: D = 7168,
// N = 129280, T = 1 83 us (94 through them), T = 32 97 (111). Not with more
// row tiles (T = 74, D = 5120: 123 us, 118 through the caches), nor for a D
// that is no multiple of 256, whose steps end inside a line (T = 8, D = 5664:
// 74 and 58; T = 1, D = 5280, N = 126034: 101 and 91; T = 74, D = 5184: 165 and
// 133).
template <Out M, int MR, int KB, int KG>
static hipError_t launch_stream(const ExpertArgs& a, Scales sc, int col_tiles, hipStream_t stream) {
  const int row_tiles = (a.R + MR - 1) / MR, grid = row_tiles * col_tiles;
  constexpr int NT = KG * kEsThreads;
  if (sc == Scales::k4) head_stream_kernel<M, MR, KB, KG, Scales::k4, 0><<<grid, NT, 0, stream>>>(a, row_tiles);
  else if (sc == Scales::kSkewed) head_stream_kernel<M, MR, KB, KG, Scales::kSkewed, 0><<<grid, NT, 0, stream>>>(a, row_tiles);
  else if (row_tiles > 1) head_stream_kernel<M, MR, KB, KG, Scales::k16, 0><<<grid, NT, 0, stream>>>(a, row_tiles);
  else head_stream_kernel<M, MR, KB, KG, Scales::k16, kNtAux><<<grid, NT, 0, stream>>>(a, row_tiles);
  return hipGetLastError();
}

// Up to this many 16-row tiles, one to a compute unit, two K groups share each:
// T = 16, D = 7168, N = 32000 27.7 -> 23.0 us; T = 28, D = 5344, N = 3501 24.8 ->
// 19.8; D = 2048 11.9 -> 10.8; level at 1024, 4.8 -> 5.8 at 512.
constexpr int kHeadFewTiles = 256;

template <Out M>
static hipError_t launch_logits(const ExpertArgs& a, bool wide, hipStream_t stream) {
  const Scales sc = scales_of(a);
  if (wide) {
    const int cols = (a.N + kEtCols - 1) / kEtCols;
    // 64 rows while each compute unit then has one tile at most (T = 192, D = 4096, N = 32000: 62 us, with 128 92; more
    // tiles: T = 256, D = 7168, N = 129280 394 us with 128, 484 with 64).
    const int tile_rows = (a.R + 63) / 64 * cols <= kOneRound ? 64 : kEtRows;
    const int row_tiles = (a.R + tile_rows - 1) / tile_rows, grid = row_tiles * cols;
    if (sc == Scales::k16) head_wide_kernel<M, Scales::k16><<<grid, kEtThreads, 0, stream>>>(a, row_tiles, tile_rows);
    else if (sc == Scales::k4) head_wide_kernel<M, Scales::k4><<<grid, kEtThreads, 0, stream>>>(a, row_tiles, tile_rows);
    else head_wide_kernel<M, Scales::kSkewed><<<grid, kEtThreads, 0, stream>>>(a, row_tiles, tile_rows);
    return hipGetLastError();
  }
  const int col_tiles = (a.N + kEsRows * kEsWaves - 1) / (kEsRows * kEsWaves);
  const int tiles16 = (a.R + 15) / 16 * col_tiles;
  if (tiles16 <= kHeadFewTiles && a.D > 1024) return launch_stream<M, 16, 1024, 2>(a, sc, col_tiles, stream);
  if (a.R <= 16) return launch_stream<M, 16, 512, 1>(a, sc, col_tiles, stream);
  return launch_stream<M, 32, 256, 1>(a, sc, col_tiles, stream);
}

static hipError_t launch_head(const HeadArgs& in, bool grad, char* ws, hipStream_t stream) {
  const HeadPlan p = head_plan(in.T, in.D, in.N, grad);
  HeadArgs h = in;
  ExpertArgs a{};
  a.xc = h.xc; a.xs = h.xs; a.gsa = h.gsa; a.gsw = h.gsw;
  a.T = a.R = h.T; a.k = 1; a.G = 1; a.D = h.D;
  float2* stats = reinterpret_cast<float2*>(ws + p.stats_at);
  a.soft.scale = kLog2e / h.tau;
  a.soft.blocks = (int)p.blocks;
  a.soft.tokens = h.tokens;
  a.soft.K = h.K;
  a.soft.named = h.logq ? h.logq : reinterpret_cast<float*>(ws + p.named_at);
  h.named = a.soft.named;
  hipError_t e;
  if (!grad) {
    for (int64_t i = 0; i < p.pieces; ++i) {
      const int64_t n0 = i * p.piece;
      a.wc = h.wc + n0 * (h.D / 2);
      a.ws = h.ws + n0 * (h.D / 16);
      a.N = (int)std::min(p.piece, h.N - n0);
      a.soft.n0 = (int)n0;
      a.soft.stats = stats + (n0 >> p.block_shift);
      a.soft.used = (int)(p.blocks - (n0 >> p.block_shift));
      if ((e = launch_logits<Out::kSums>(a, p.wide, stream)) != hipSuccess) return e;
    }
    h.stats = stats;
    h.blocks = h.used = (int)p.blocks;
    head_tokens_kernel<<<h.T, 64 * kTokWaves, 0, stream>>>(h);
    return hipGetLastError();
  }
  float2* state = reinterpret_cast<float2*>(ws + p.state_at);
  float* shrink = reinterpret_cast<float*>(ws + p.shrink_at);
  float* ref = reinterpret_cast<float*>(ws + p.ref_at);
  float* part = reinterpret_cast<float*>(ws + p.part_at);
  h.lists = reinterpret_cast<TokenList*>(ws + p.lists_at);
  a.soft.stats = stats;
  a.soft.used = (int)p.blocks;
  a.soft.e = reinterpret_cast<_Float16*>(ws + p.e_at);
  a.soft.ld_e = p.ld_e;
  for (int64_t i = 0; i < p.pieces; ++i) {
    const int64_t n0 = i * p.piece;
    a.wc = h.wc + n0 * (h.D / 2);
    a.ws = h.ws + n0 * (h.D / 16);
    a.N = (int)std::min(p.piece, h.N - n0);
    a.soft.n0 = (int)n0;
    a.soft.ref = i ? ref : nullptr;
    if ((e = launch_logits<Out::kWeights>(a, p.wide, stream)) != hipSuccess) return e;
    NormArgs n{};
    n.stats = stats; n.blocks = (int)p.blocks;
    n.used = (a.N + 63) / 64 << (6 - p.block_shift);
    n.before = i ? state + ((i - 1) & 1) * (int64_t)h.T : nullptr;
    n.after = state + (i & 1) * (int64_t)h.T;
    n.shrink = shrink; n.ref = ref; n.e = a.soft.e; n.ld_e = p.ld_e;
    n.T = h.T; n.K = h.K; n.n0 = (int)n0; n.cols = a.N; n.tokens = h.tokens;
    if (i + 1 < p.pieces) head_norm_kernel<false><<<h.T, kNormThreads, 0, stream>>>(n, h);
    else head_norm_kernel<true><<<h.T, kNormThreads, 0, stream>>>(n, h);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    GradArgs g{};
    g.e = a.soft.e; g.ld_e = p.ld_e; g.wc = a.wc; g.ws = a.ws; g.T = h.T; g.D = h.D; g.cols = a.N;
    g.part = part; g.shrink = i ? shrink : nullptr;
    g.stats = stats; g.blocks = (int)p.blocks; g.block_shift = p.block_shift; g.ref = ref; g.tiles = p.tiles;
    const int grid = p.tiles.full + (p.tiles.count() - p.tiles.full) * p.tiles.splits;
    if (h.D % 64 == 0) head_grad_kernel<true><<<grid, kGwThreads, 0, stream>>>(g);
    else head_grad_kernel<false><<<grid, kGwThreads, 0, stream>>>(g);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  h.stats = state + ((p.pieces - 1) & 1) * (int64_t)h.T;
  DxArgs d{h, part, p.tiles};
  const int columns = (h.D + 511) / 512;
  if (dx_share(h.T, columns, h.K))
    head_dx_kernel<true><<<dim3(h.T, columns), 64 * dx_waves<true>(), 0, stream>>>(d);
  else
    head_dx_kernel<false><<<dim3(h.T, (columns + dx_waves<false>() - 1) / dx_waves<false>()), 64 * dx_waves<false>(), 0, stream>>>(d);
  return hipGetLastError();
}

}  // namespace nvr

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int check_head_sizes(int64_t T, int64_t D, int64_t N) {
  if (T < 0 || D < 32 || D % 32 != 0 || N < 1) return ROUTER_EINVAL;
  if (T > ROUTER_MAX_LOSS_ROWS || D > ROUTER_MAX_GATE_D || N > (int64_t(1) << 30)) return ROUTER_EUNSUPPORTED;
  return ROUTER_OK;
}

int head_call(nvr::HeadArgs& h, int64_t T, int64_t D, int64_t N, int64_t K, void* workspace, size_t workspace_bytes,
              void* stream) {
  const int st = check_head_sizes(T, D, N);
  if (st != ROUTER_OK) return st;
  if (K < 1) return ROUTER_EINVAL;
  if (K > ROUTER_MAX_TEACHER) return ROUTER_EUNSUPPORTED;
  if (!h.gsa || !h.gsw || !h.wc || !h.ws) return ROUTER_EINVAL;
  if (T > 0 && (!h.xc || !h.xs || !h.tokens || !h.loss || !h.lse)) return ROUTER_EINVAL;
  if (!aligned(h.xc, 16) || !aligned(h.wc, 16) || !aligned(h.xs, 2) || !aligned(h.ws, 4) || !aligned(h.gsa, 4) ||
      !aligned(h.gsw, 4) || !aligned(h.tokens, 4) || !aligned(h.weight, 4) || !aligned(h.loss, 4) ||
      !aligned(h.lse, 4) || !aligned(h.logq, 4) || !aligned(h.dx, 16) ||
      !aligned(h.teacher, h.teacher_bf16 ? 2 : 4))
    return ROUTER_EINVAL;
  if (T == 0) return ROUTER_OK;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < nvr::head_plan(T, D, N, h.dx != nullptr).bytes)
    return ROUTER_EINVAL;
  h.T = (int)T; h.D = (int)D; h.N = (int)N; h.K = (int)K;
  const hipError_t e = nvr::launch_head(h, h.dx != nullptr, static_cast<char*>(workspace), static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ROUTER_OK : ROUTER_EHIP;
}

}  // namespace

extern "C" {

size_t lmhead_loss_workspace_bytes(int64_t T, int64_t D, int64_t N, int grad) {
  if (check_head_sizes(T, D, N) != ROUTER_OK) return 0;
  // What a call needs falls in places as T grows (other tiles, splits and pieces), so this is the most of all row counts
  // up to T, and with a gradient of the calls without one too: 3 ms at T = 4096.
  size_t bytes = 0;
  for (int64_t t = std::min(T, int64_t(1)); t <= T; ++t) {
    bytes = std::max(bytes, nvr::head_plan(t, D, N, false).bytes);
    if (grad) bytes = std::max(bytes, nvr::head_plan(t, D, N, true).bytes);
  }
  return bytes;
}

int lmhead_loss(const uint8_t* x_codes, const uint8_t* x_scales, const float* gsa, const uint8_t* w_codes,
                const uint8_t* w_scales, const float* gsw, const int32_t* targets, const float* weight, int64_t T,
                int64_t D, int64_t N, float* loss, float* lse, void* dx, void* workspace, size_t workspace_bytes,
                void* stream) {
  nvr::HeadArgs h{};
  h.xc = x_codes; h.xs = x_scales; h.gsa = gsa;
  h.wc = w_codes; h.ws = w_scales; h.gsw = gsw;
  h.tokens = targets; h.weight = weight; h.tau = 1.0f;
  h.loss = loss; h.lse = lse; h.dx = dx;
  return head_call(h, T, D, N, 1, workspace, workspace_bytes, stream);
}

int lmhead_distill(const uint8_t* x_codes, const uint8_t* x_scales, const float* gsa, const uint8_t* w_codes,
                   const uint8_t* w_scales, const float* gsw, const int32_t* tokens, const void* teacher, int dtype,
                   int64_t K, float temperature, const float* weight, int64_t T, int64_t D, int64_t N, float* loss,
                   float* lse, float* logq, void* dx, void* workspace, size_t workspace_bytes, void* stream) {
  if ((dtype != ROUTER_F32 && dtype != ROUTER_BF16) || !(temperature >= 0x1p-20f && temperature <= 0x1p20f))
    return ROUTER_EINVAL;
  if (T > 0 && (!teacher || !logq)) return ROUTER_EINVAL;
  nvr::HeadArgs h{};
  h.xc = x_codes; h.xs = x_scales; h.gsa = gsa;
  h.wc = w_codes; h.ws = w_scales; h.gsw = gsw;
  h.tokens = tokens; h.teacher = teacher; h.teacher_bf16 = dtype == ROUTER_BF16;
  h.weight = weight; h.tau = temperature;
  h.loss = loss; h.lse = lse; h.logq = logq; h.dx = dx;
  return head_call(h, T, D, N, K, workspace, workspace_bytes, stream);
}

}  // extern "C"
