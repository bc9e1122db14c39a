// The routed experts' products (gfx950) over rows sorted by expert:
//
//   grouped_swiglu:  y[p, n] = gsa gsw[e] sum_d (q_x S_x)[t(p), d] (q_w S_w)[e, n, d] + bias[e, n]
//                    h[p, f] = silu(y[p, f]) y[p, F + f]            (bf16)
//   grouped_combine: y[p, n] = gsh gsw[e] sum_f (q_h S_h)[p, f] (q_w S_w)[e, n, f] + bias[e, n]
//                    out[t, n] = residual[t, n] + sum_j w[t, j] y[pos[t, j], n]   (bf16)
//
// with e the expert of row p and t(p) = rows[p] / k its token.
#include "../../include/nvfp4_router.h"
#include "experts_common.hpp"

#include <algorithm>

namespace nvr {

size_t plan_scratch_bytes(int64_t R, int64_t G);  // experts_plan.hip

struct ExpertArgs {
  const uint8_t* xc;       // swiglu: [T, D/2] tokens; combine: [R, D/2] rows
  const uint8_t* xs;
  const float* gsa;
  const uint8_t* wc;       // [G, N, D/2]
  const uint8_t* ws;
  const float* gsw;        // [G]
  const float* bias;       // NULL or [G, N]
  const int32_t* offsets;  // [G + 1]
  const int32_t* rows;     // swiglu: [R]
  void* out;               // swiglu: bf16 [R, N/2]; combine: fp32 [R, N] products
  int T, k, R, G, N, D;
  int col_tiles, nsteps;
  Take take;      // which experts this launch takes
  int tile_cols;  // column tiles of the 128-row tile kernel
};

// Token of row p, or -1.
__device__ __forceinline__ int row_token(const ExpertArgs& a, int p) {
  const int s = a.rows[p];
  const int t = s / a.k;
  return s >= 0 && t < a.T ? t : -1;
}

__device__ __forceinline__ float silu_mul(float g, float u) { return g * sigmoid_fast(g) * u; }

// Work item b -> (row tile, column tile). The products of the experts' rows
// come first, numbered so that consecutive items (the row tiles of one column
// tile of an expert, then its next column tile) run on one XCD and share its
// L2; then, if `others` (grouped_swiglu), one item per row tile of no expert.
// False behind the last item.
struct ExpertTile {
  RowTile rt;
  int ct;
};
__device__ __forceinline__ bool expert_tile(const ExpertArgs& a, const TileScan& scan, bool others, int b,
                                            ExpertTile& t) {
  const int products = scan.experts * a.col_tiles;
  if (b < products) {
    t.rt = scan.at(xcd_order(b, products), a.col_tiles, t.ct);
    return true;
  }
  if (others && b - products < scan.others()) {
    t.ct = 0;
    t.rt = scan.none(b - products);
    return true;
  }
  return false;
}

// Zeros for the rows of no expert: router_quantize runs over all R rows, and
// stale values there would set its global scale. F is a multiple of 16, so
// whole rows are whole 16-byte pieces (a 2-byte store per element and column
// tile took 1.1 ms for the 28672 rows of an eighth of 4096 tokens' experts).
__device__ __forceinline__ void zero_rows(const ExpertArgs& a, const RowTile& t, int nthreads) {
  const int64_t per_row = a.N >> 4;  // F / 8 pieces
  u32x4_t* out = static_cast<u32x4_t*>(a.out) + t.row0 * per_row;
  for (int64_t i = threadIdx.x; i < t.nr * per_row; i += nthreads) out[i] = u32x4_t{0u, 0u, 0u, 0u};
}

// Scale row offsets of a tile of gathered rows (A) and paired weight rows
// (B), from a table in LDS.
struct TableRows {
  const uint32_t* tab;
  int bm;
  __device__ __forceinline__ uint32_t operator()(bool isA, int rr) const { return tab[isA ? rr : bm + rr]; }
};

// LDS of one tile: the A tiles, the scale windows and the row table.
template <bool GLU, int BM, int NTW, int KS, bool STAGED>
struct ExpertLds {
  alignas(16) _Float16 abuf[KS][2][BM * kMmaARow];
  alignas(16) uint8_t swin[STAGED ? mma_win_bytes<BM, NTW>() : 16];
  uint32_t srow[GLU ? BM + 128 * NTW : 1];
};

// One tile of up to BM rows of an expert times 128 NTW weight rows on the
// shared MFMA tile. GLU: the rows are gathered, and each 32-column tile holds
// 16 gate rows and the 16 up rows of the same outputs, so that one lane swap
// brings the two halves of an output together.
template <bool GLU, int BM, int NTW, int KS, bool STAGED>
__device__ __forceinline__ void experts_tile(const ExpertArgs& a, const RowTile& rt, int ct,
                                             ExpertLds<GLU, BM, NTW, KS, STAGED>& lds) {
  static_assert(KS == mma_ksplit<BM, NTW>(), "K groups as the main loop has them");
  constexpr int BN = 128 * NTW;
  static_assert(KS == 1 || BM * BN * sizeof(float) <= sizeof(_Float16) * KS * 2 * BM * kMmaARow,
                "the epilogue's partial sums fit in the A tiles' LDS");
  _Float16* abuf = &lds.abuf[0][0][0];
  uint32_t* srow = lds.srow;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wt = wave & 3, grp = wave >> 2;
  const int row0 = rt.row0, nr = rt.nr;
  const float gsa = load_early(a.gsa), gsw = load_early(a.gsw + rt.g);
  const int64_t rowc = a.D / 2, rows = a.D / 16;
  const int r = lane & 31, h = lane >> 5, F = a.N >> 1;
  const int64_t we = (int64_t)rt.g * a.N;
  MmaPtrs<BM, NTW> P;
  if constexpr (GLU) {
    const int f0 = ct * (BN / 2);
    P.xc = make_rsrc(a.xc, a.T * rowc);
    P.xs = make_rsrc(a.xs, a.T * rows);
    P.wc = make_rsrc(a.wc + we * rowc, a.N * rowc);
    P.ws = make_rsrc(a.ws + we * rows, a.N * rows);
    const int tid = threadIdx.x & (kMmaThreads - 1), q = tid & 3;
    P.ka = 32 * q;
    P.kb = 32 * h;
#pragma unroll
    for (int i = 0; i < mma_row_slots<BM>(); ++i) {
      const int rl = (tid >> 2) + 64 * i;
      const int t = rl < nr ? row_token(a, row0 + min(rl, nr - 1)) : -1;
      P.a[i] = t >= 0 ? (uint32_t)(t * rowc + 16 * q) : kMmaOob;
      P.as[i] = t >= 0 ? (uint32_t)(t * rows + 2 * q) : kMmaOob;
    }
    // Column c of the tile: the 16 gate rows, then the 16 up rows, of 16 outputs.
    auto wrow = [&](int c) {
      const int f = f0 + 16 * (c >> 5) + (c & 15);
      return f < F ? (c & 16 ? F + f : f) : -1;
    };
#pragma unroll
    for (int t = 0; t < NTW; ++t) {
      const int w = wrow((wt + 4 * t) * 32 + r);
      P.b[t] = w >= 0 ? (uint32_t)(w * rowc + 16 * h) : kMmaOob;
      P.bs[t] = w >= 0 ? (uint32_t)(w * rows + 2 * h) : kMmaOob;
    }
    if constexpr (STAGED) {
      for (int i = threadIdx.x; i < BM + BN; i += kMmaThreads * KS) {
        const int v = i < BM ? (i < nr ? row_token(a, row0 + i) : -1) : wrow(i - BM);
        srow[i] = v >= 0 ? (uint32_t)(v * rows) : kMmaOob;
      }
      __syncthreads();
    }
  } else {
    const int col0 = ct * BN;
    P = mma_ptrs<BM, NTW>(a.xc + row0 * rowc, a.xs + row0 * rows, nr, a.wc + (we + col0) * rowc,
                          a.ws + (we + col0) * rows, min(BN, a.N - col0), a.D, wt, lane);
  }
  constexpr int NS = mma_sets<BM, NTW>();
  f32x16_t acc[NS][BM / 32][NTW];
  if constexpr (GLU)
    mma_mainloop<BM, NTW, KS, STAGED>(P, a.D, a.nsteps, abuf, lds.swin, lane, acc, TableRows{srow, BM});
  else
    mma_mainloop<BM, NTW, KS, STAGED>(P, a.D, a.nsteps, abuf, lds.swin, lane, acc);

  // 32x32 accumulator layout: value v of lane (r, h) is row 8(v/4) + 4h +
  // v%4, column r of its tile; wavefront wt holds the column tiles wt + 4t.
  float* part = reinterpret_cast<float*>(abuf);  // [BM][BN], K group 1's sums
  if (KS == 2 && grp == 1) {
#pragma unroll
    for (int rt2 = 0; rt2 < BM / 32; ++rt2)
#pragma unroll
      for (int t = 0; t < NTW; ++t)
#pragma unroll
        for (int v = 0; v < 16; ++v)
          part[(rt2 * 32 + 8 * (v >> 2) + 4 * h + (v & 3)) * BN + (wt + 4 * t) * 32 + r] = acc[0][rt2][t][v];
  }
  if (KS == 2) __syncthreads();
  if (grp != 0) return;
  const float scale = gsa * gsw;
#pragma unroll
  for (int t = 0; t < NTW; ++t) {
    const int c = (wt + 4 * t) * 32 + r;
    if constexpr (GLU) {
      const int f = ct * (BN / 2) + 16 * (wt + 4 * t) + (r & 15);
      const bool ok = f < F;
      float bg = 0.0f, bu = 0.0f;
      if (a.bias) {
        const float* b = a.bias + we + min(f, F - 1);
        bg = b[0];
        bu = b[F];
      }
#pragma unroll
      for (int rt2 = 0; rt2 < BM / 32; ++rt2)
#pragma unroll
        for (int v = 0; v < 8; ++v) {
          float y0 = acc[0][rt2][t][v], y1 = acc[0][rt2][t][v + 8];
          if (KS == 2) {
            const int rr = rt2 * 32 + 8 * (v >> 2) + 4 * h + (v & 3);
            y0 += part[rr * BN + c];
            y1 += part[(rr + 16) * BN + c];
          }
          // Lanes r < 16 hold gates and lanes r >= 16 ups of outputs f; after
          // the swap the former hold both of value v, the latter of v + 8.
          const auto sw = __builtin_amdgcn_permlane16_swap(__float_as_uint(y0), __float_as_uint(y1), false, false);
          const float g = __uint_as_float(sw[0]) * scale + bg, u = __uint_as_float(sw[1]) * scale + bu;
          const int rr = rt2 * 32 + 8 * (v >> 2) + (r & 16) + 4 * h + (v & 3);
          if (rr < nr && ok)
            static_cast<uint16_t*>(a.out)[(int64_t)(row0 + rr) * F + f] = bf16_round(silu_mul(g, u));
        }
    } else {
      const int col = ct * BN + c;
      const bool ok = col < a.N;
      const float b = a.bias ? a.bias[we + min(col, a.N - 1)] : 0.0f;
#pragma unroll
      for (int rt2 = 0; rt2 < BM / 32; ++rt2)
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          const int rr = rt2 * 32 + 8 * (v >> 2) + 4 * h + (v & 3);
          float y = acc[0][rt2][t][v];
          if (KS == 2) y += part[rr * BN + c];
          if (rr < nr && ok) static_cast<float*>(a.out)[(int64_t)(row0 + rr) * a.N + col] = y * scale + b;
        }
    }
  }
}

// Workgroup (row tile of up to BM rows of an expert, column tile). A ragged
// last tile with at most half the rows takes the 64-row tile instead of the
// 128-row one, which costs it little more than half as much.
template <bool GLU, int BM, int NTW, int KS, bool STAGED>
__global__ __launch_bounds__(kMmaThreads * KS) __attribute__((amdgpu_waves_per_eu(KS, KS))) void experts_mfma_kernel(
    ExpertArgs a) {
  constexpr int SH = BM == 32 ? 5 : (BM == 64 ? 6 : 7);
  static_assert(BM == 1 << SH, "rows per tile");
  constexpr bool kHalf = BM == 128 && mma_ksplit<64, NTW>() == KS;
  __shared__ union {
    ExpertLds<GLU, BM, NTW, KS, STAGED> full;
    ExpertLds<GLU, kHalf ? 64 : BM, NTW, KS, STAGED> half;
  } lds;
  const TileScan scan(a.offsets, a.G, a.R, SH, a.take, a.tile_cols);
  ExpertTile tile;
  if (!expert_tile(a, scan, false, blockIdx.x, tile)) return;
  const RowTile& rt = tile.rt;
  const int ct = tile.ct;
  if constexpr (kHalf) {
    if (rt.nr <= 64) {
      experts_tile<GLU, 64, NTW, KS, STAGED>(a, rt, ct, lds.half);
      return;
    }
  }
  experts_tile<GLU, BM, NTW, KS, STAGED>(a, rt, ct, lds.full);
}

// Few rows per expert (up to MR per tile): a stream of the hit experts'
// weights through MFMA. Wavefront = 32 weight rows (GLU: 16 gate rows and the
// 16 up rows of the same outputs) times MR rows on 16x16x32 MFMAs, weights as
// the row operand, so a lane ends up with 4 adjacent outputs of one row (and
// with gate and up of the same output).
//  * Weights: 256 K values (one 128-byte line of codes) per row and step,
//    loaded 8 whole lines per instruction: the address unit takes a pass per
//    line that an instruction touches, and a load in MFMA layout (16 bytes of
//    each of 32 rows) touches four times as many. Two steps are in flight per
//    wavefront; a step's codes pass through 4 KB of LDS private to the
//    wavefront (16-byte pieces XOR-swizzled by row) into MFMA layout: lane
//    (r, q) takes the 32 K values from 32 q of every 128 of row r.
//  * Scales: windows of 512 K (32 bytes per row), likewise.
//  * x: KB K values of the tile's rows, converted to fp16 q S once per
//    workgroup into one of two LDS tiles (one barrier per KB).
//  * Past D the x tile holds zeros, so whatever finite weights a padded step
//    reads there add nothing.
constexpr int kEsWaves = 4;
constexpr int kEsThreads = 64 * kEsWaves;
constexpr int kEsRows = 32;       // weight rows per wavefront
constexpr int kEsSmallGrid = 256 * 6;  // workgroups that share a launch's items: two rounds of three per CU
constexpr int kEsScaleLd = 36;    // LDS bytes per row of a scale window (32 + 4)

template <int MR, int KB>
struct StreamLds {
  alignas(16) _Float16 x[2][MR * KB];
  alignas(16) uint8_t codes[kEsWaves][kEsRows * 128];
  alignas(16) uint8_t scales[kEsWaves][kEsRows * kEsScaleLd];
};

// Halves offset of 16-byte piece c of row r of an x tile.
template <int KB>
__device__ __forceinline__ int stream_x_at(int r, int c) {
  return r * KB + 8 * (c ^ (r & 7));
}

// One tile. ALIGNED: D % 256 == 0, so scale rows can be read 16 bytes at a
// time.
template <bool GLU, int MR, int KB, bool ALIGNED>
__device__ __forceinline__ void stream_tile(const ExpertArgs& a, const ExpertTile& tile, StreamLds<MR, KB>& lds) {
  constexpr int NT = MR / 16, NTHREADS = kEsThreads;
  static_assert(KB == 256 || KB == 512, "whole steps");
  constexpr int XP = MR * (KB / 32) / NTHREADS;  // 32-value pieces of x per thread and block
  static_assert(XP * NTHREADS == MR * (KB / 32), "whole pieces per thread");
  constexpr int SPB = KB / 256;  // steps per x block
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const RowTile& rt = tile.rt;
  const float gsa = load_early(a.gsa), gsw = load_early(a.gsw + rt.g);
  const int nr = rt.nr, F = a.N >> 1;
  const int64_t rowc = a.D / 2, rows = a.D / 16, we = (int64_t)rt.g * a.N;
  // This wavefront's first output (GLU) or weight row, and its two 16-row tiles.
  const int o0 = (tile.ct * kEsWaves + wave) * (GLU ? 16 : 32);
  const bool live0 = o0 < (GLU ? F : a.N), live1 = GLU ? live0 : o0 + 16 < a.N;
  auto wrow = [&](int m) { return GLU ? (m ? F + o0 : o0) : o0 + 16 * m; };

  const __amdgpu_buffer_rsrc_t wcr = make_rsrc(a.wc + we * rowc, a.N * rowc);
  const __amdgpu_buffer_rsrc_t wsr = make_rsrc(a.ws + we * rows, a.N * rows);
  uint32_t wo[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    wo[i] = ((i >> 1) ? live1 : live0) ? (uint32_t)((wrow(i >> 1) + 8 * (i & 1) + (lane >> 3)) * rowc + 16 * (lane & 7))
                                       : kMmaOob;
  u32x4_t wv[2][4];
  auto load_w = [&](int slot, int step) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      wv[slot][i] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(wcr, wo[i] + 128 * step, 0, kNtAux));
  };
  // Scale window: lane = (row lane / 2, 16 bytes) of the 32 rows, or 2 bytes
  // of 4 rows in each of 8 loads.
  constexpr int SL = ALIGNED ? 1 : 8;
  uint32_t so[SL];
  if constexpr (ALIGNED) {
    const int m = lane >> 5;
    so[0] = (m ? live1 : live0) ? (uint32_t)((wrow(m) + ((lane >> 1) & 15)) * rows + 16 * (lane & 1)) : kMmaOob;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int m = i >> 2;
      so[i] = (m ? live1 : live0) ? (uint32_t)((wrow(m) + 4 * (i & 3) + (lane >> 4)) * rows + 2 * (lane & 15)) : kMmaOob;
    }
  }
  u32x4_t sv16;
  uint32_t sv2[SL];
  auto load_s = [&](int win) {
    if constexpr (ALIGNED) sv16 = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(wsr, so[0] + 32 * win, 0, 0));
    else {
#pragma unroll
      for (int i = 0; i < 8; ++i) sv2[i] = __builtin_amdgcn_raw_buffer_load_b16(wsr, so[i] + 32 * win, 0, 0);
    }
  };
  uint8_t* my_codes = lds.codes[wave];
  uint8_t* my_scales = lds.scales[wave];
  auto store_s = [&]() {
    if constexpr (ALIGNED) {
      uint32_t* d = reinterpret_cast<uint32_t*>(my_scales + (lane >> 1) * kEsScaleLd + 16 * (lane & 1));
#pragma unroll
      for (int i = 0; i < 4; ++i) d[i] = sv16[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        *reinterpret_cast<uint16_t*>(my_scales + (4 * i + (lane >> 4)) * kEsScaleLd + 2 * (lane & 15)) = (uint16_t)sv2[i];
    }
  };

  // x pieces of this thread: (row, 32-value piece of the block).
  const uint8_t* xcp[XP];
  const uint8_t* xsp[XP];
  int xk[XP];
#pragma unroll
  for (int i = 0; i < XP; ++i) {
    const int p = threadIdx.x + NTHREADS * i, r = p / (KB / 32);
    xk[i] = 32 * (p % (KB / 32));
    int t = -1;
    if (r < nr) t = GLU ? row_token(a, rt.row0 + r) : rt.row0 + r;
    if (t < 0) xk[i] = a.D;  // no such row: zeros
    xcp[i] = a.xc + (int64_t)max(t, 0) * rowc;
    xsp[i] = a.xs + (int64_t)max(t, 0) * rows;
  }
  u32x4_t xv[XP];
  uint32_t xsv[XP];
  auto load_x = [&](int k0) {
#pragma unroll
    for (int i = 0; i < XP; ++i) {
      // Clamped to the row's first piece past D; those values are zeroed below.
      const int k = k0 + xk[i] < a.D ? k0 + xk[i] : 0;
      xv[i] = *reinterpret_cast<const u32x4_t*>(xcp[i] + k / 2);
      xsv[i] = *reinterpret_cast<const uint16_t*>(xsp[i] + k / 16);
    }
  };
  auto store_x = [&](int k0, int buf) {
#pragma unroll
    for (int i = 0; i < XP; ++i) {
      const int p = threadIdx.x + NTHREADS * i, r = p / (KB / 32), c = p % (KB / 32);
      const half2_t s = e4m3x2_f16(k0 + xk[i] < a.D ? xsv[i] : 0u);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<half8_t*>(&lds.x[buf][stream_x_at<KB>(r, 4 * c + j)]) = fp4x8_scaled(xv[i][j], s, j >> 1);
    }
  };

  const int nsteps = (a.D + 255) / 256;
  load_x(0);
  load_s(0);
  load_w(0, 0);
  load_w(1, 1);
  store_x(0, 0);
  __syncthreads();
  f32x4_t acc[2][NT];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[m][t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  const int r = lane & 15, q = lane >> 4;
  for (int s0 = 0; s0 < nsteps; s0 += 2) {
    // The window's scales; the next one's loads.
    store_s();
    load_s((s0 >> 1) + 1);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int step = s0 + u;
      const int block = step / SPB, in = u % SPB, buf = block & 1;
      // Before the weight loads: loads complete in order, and the wait for x
      // at the end of the block must not wait for weights two steps ahead.
      if (in == 0) load_x((block + 1) * KB);
      // Codes through LDS into MFMA layout.
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 8 * i + (lane >> 3);
        *reinterpret_cast<u32x4_t*>(my_codes + row * 128 + 16 * ((lane & 7) ^ (row & 7))) = wv[u][i];
      }
      load_w(u, step + 2);
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
      if (step < nsteps) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          u32x4_t c[2];
          half2_t s[2];
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            c[m] = *reinterpret_cast<const u32x4_t*>(my_codes + (16 * m + r) * 128 + 16 * ((4 * g + q) ^ (r & 7)));
            s[m] = e4m3x2_f16(lds_u16(my_scales + (16 * m + r) * kEsScaleLd + 16 * u + 8 * g + 2 * q));
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            half8_t w[2];
#pragma unroll
            for (int m = 0; m < 2; ++m) w[m] = fp4x8_scaled(c[m][j], s[m], j >> 1);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              const half8_t xf = *reinterpret_cast<const half8_t*>(
                  &lds.x[buf][stream_x_at<KB>(16 * t + r, 32 * in + 16 * g + 4 * q + j)]);
#pragma unroll
              for (int m = 0; m < 2; ++m) acc[m][t] = mfma16(w[m], xf, acc[m][t]);
            }
          }
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
      if (in == SPB - 1) {
        store_x((block + 1) * KB, buf ^ 1);
        __syncthreads();
      }
    }
  }

  // Lane (r, q), value v of tile m: row r (+ 16 t), weight row 4 q + v of the tile.
  const float scale = gsa * gsw;
  if constexpr (GLU) {
    if (!live0) return;
    const int f = o0 + 4 * q;
    float bg[4] = {0.0f, 0.0f, 0.0f, 0.0f}, bu[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (a.bias) {
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        bg[v] = a.bias[we + f + v];
        bu[v] = a.bias[we + F + f + v];
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float y[4];
#pragma unroll
      for (int v = 0; v < 4; ++v) y[v] = silu_mul(acc[0][t][v] * scale + bg[v], acc[1][t][v] * scale + bu[v]);
      if (16 * t + r < nr) {
        uint2* d = reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + (int64_t)(rt.row0 + 16 * t + r) * F + f);
        *d = make_uint2(bf16_round2(y[0], y[1]), bf16_round2(y[2], y[3]));
      }
    }
  } else {
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      if (!(m ? live1 : live0)) continue;
      const int n = o0 + 16 * m + 4 * q;
      f32x4_t b = {0.0f, 0.0f, 0.0f, 0.0f};
      if (a.bias) {
#pragma unroll
        for (int v = 0; v < 4; ++v) b[v] = a.bias[we + n + v];
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        f32x4_t y;
#pragma unroll
        for (int v = 0; v < 4; ++v) y[v] = acc[m][t][v] * scale + b[v];
        if (16 * t + r < nr)
          *reinterpret_cast<f32x4_t*>(static_cast<float*>(a.out) + (int64_t)(rt.row0 + 16 * t + r) * a.N + n) = y;
      }
    }
  }
}

// SHARED: workgroups take items in turn; else one item each (the loop around
// the tile costs some 50 registers, and with them one of the three workgroups
// per CU that the LDS allows).
template <bool GLU, int MR, int KB, bool ALIGNED, bool SHARED>
__global__ __launch_bounds__(kEsThreads) void experts_stream_kernel(ExpertArgs a) {
  constexpr int SH = MR == 16 ? 4 : 5;
  static_assert(MR == 1 << SH, "rows per tile");
  __shared__ StreamLds<MR, KB> lds;
  const TileScan scan(a.offsets, a.G, a.R, SH, a.take, a.tile_cols);
  ExpertTile tile;
  for (int b = blockIdx.x; expert_tile(a, scan, GLU, b, tile); b += gridDim.x) {
    if (GLU && tile.rt.g == a.G) zero_rows(a, tile.rt, kEsThreads);
    else stream_tile<GLU, MR, KB, ALIGNED>(a, tile, lds);
    if (!SHARED) return;
    __syncthreads();  // the next item writes the LDS tiles
  }
}

// out[t, n] = residual[t, n] + sum_j w[t, j] y[pos[t, j], n], j in order, 8
// columns per thread.
struct CombineArgs {
  const float* y;  // [R, N]
  const int32_t* pos;
  const float* w;
  const uint16_t* residual;  // NULL or bf16 [T, N]
  uint16_t* out;
  int T, k, R, N;
};

__global__ __launch_bounds__(256) void combine_kernel(CombineArgs a) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, nv = a.N / 8;
  if (i >= (int64_t)a.T * nv) return;
  const int64_t t = i / nv;
  const int c = (int)(i - t * nv) * 8;
  typedef float f32x8_t __attribute__((ext_vector_type(8)));
  f32x8_t acc;
  const int64_t o = t * a.N + c;
  if (a.residual) {
    const u32x4_t v = *reinterpret_cast<const u32x4_t*>(a.residual + o);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      acc[2 * q] = bf16_lo(v[q]);
      acc[2 * q + 1] = bf16_hi(v[q]);
    }
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[q] = 0.0f;
  }
  for (int j = 0; j < a.k; ++j) {
    const int p = a.pos[t * a.k + j];
    if (p < 0 || p >= a.R) continue;  // an expert held elsewhere: its weight is not read
    const float w = a.w[t * a.k + j];
    const f32x8_t y = *reinterpret_cast<const f32x8_t*>(a.y + (int64_t)p * a.N + c);
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[q] = fmaf(w, y[q], acc[q]);
  }
  u32x4_t v;
#pragma unroll
  for (int q = 0; q < 4; ++q) v[q] = bf16_round2(acc[2 * q], acc[2 * q + 1]);
  *reinterpret_cast<u32x4_t*>(a.out + o) = v;
}

// ---------------------------------------------------------------------------
// Dispatch. The host knows the rows (R) and experts (G), not the experts'
// sizes.
// ---------------------------------------------------------------------------
template <bool GLU, int BM, int NTW>
static hipError_t launch_mfma(ExpertArgs a, hipStream_t stream) {
  constexpr int KS = mma_ksplit<BM, NTW>(), BN = 128 * NTW, SH = BM == 32 ? 5 : (BM == 64 ? 6 : 7);
  a.col_tiles = (a.N + BN - 1) / BN;
  a.nsteps = mma_padded_steps<BM, NTW>(a.D);
  const int64_t nwg = max_row_tiles(a.R, a.G, SH) * a.col_tiles;
  if (nwg >= (int64_t(1) << 31)) return hipErrorInvalidConfiguration;
  if (a.D % 256 == 0) experts_mfma_kernel<GLU, BM, NTW, KS, true><<<(int)nwg, kMmaThreads * KS, 0, stream>>>(a);
  else experts_mfma_kernel<GLU, BM, NTW, KS, false><<<(int)nwg, kMmaThreads * KS, 0, stream>>>(a);
  return hipGetLastError();
}

template <bool GLU, int MR, int KB, bool SHARED>
static hipError_t launch_stream(ExpertArgs a, hipStream_t stream) {
  a.col_tiles = (a.N + kEsRows * kEsWaves - 1) / (kEsRows * kEsWaves);
  const int64_t items = max_row_tiles(a.R, a.G, MR == 16 ? 4 : 5) * a.col_tiles;
  if (items >= (int64_t(1) << 31)) return hipErrorInvalidConfiguration;
  // A launch of small experts beside the large ones is mostly empty: there
  // each workgroup takes several items (129 thousand workgroups that had
  // nothing to do took 140 us at T = 8192).
  const int nwg = (int)(SHARED ? std::min<int64_t>(items, kEsSmallGrid) : items);
  if (a.D % 256 == 0) experts_stream_kernel<GLU, MR, KB, true, SHARED><<<nwg, kEsThreads, 0, stream>>>(a);
  else experts_stream_kernel<GLU, MR, KB, false, SHARED><<<nwg, kEsThreads, 0, stream>>>(a);
  return hipGetLastError();
}

// By the mean number of rows per expert, were every slot's expert held here:
// up to 8 (T = 64 of 256 experts, k = 8: 433 us with 16-row tiles, 478 with
// 32, 650 with the 128-row ones), up to 32 (T = 1024: 1211 us with 32-row
// tiles, 1484 with 16, 1229 with 128); beyond that two launches share the
// experts by their sizes, which only the device knows (an expert-parallel
// rank's experts have a fraction of the mean, and a layer's popular experts
// several times its others' rows).
template <bool GLU>
static hipError_t launch_products(ExpertArgs a, hipStream_t stream) {
  const int64_t mean = a.R / a.G;
  a.take = Take::kAll;
  if (mean <= 8) return launch_stream<GLU, 16, 512, false>(a, stream);
  if (mean <= 32) return launch_stream<GLU, 32, 256, false>(a, stream);
  constexpr int NTW = 2;
  a.tile_cols = (a.N + 128 * NTW - 1) / (128 * NTW);
  a.take = Take::kSmall;
  const hipError_t e = launch_stream<GLU, 32, 256, true>(a, stream);
  if (e != hipSuccess) return e;
  a.take = Take::kLarge;
  return launch_mfma<GLU, 128, NTW>(a, stream);
}

}  // namespace nvr

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int status_from(hipError_t e) {
  if (e == hipErrorInvalidConfiguration) return ROUTER_EUNSUPPORTED;
  return e == hipSuccess ? ROUTER_OK : ROUTER_EHIP;
}

// Sizes of either product: k K values per row (a multiple of 32), N weight
// rows per expert.
int check_sizes(int64_t T, int64_t k, int64_t G, int64_t N, int64_t K, int64_t operand_rows) {
  if (T < 0 || T >= (int64_t(1) << 31) || k < 1 || G < 1 || N < 1 || K < 16 || K % 16 != 0) return ROUTER_EINVAL;
  if (k > ROUTER_MAX_TOPK || G > ROUTER_MAX_EXPERTS || T * k >= (int64_t(1) << 30) || K % 32 != 0 ||
      K > ROUTER_MAX_GATE_D || N > ROUTER_MAX_GATE_D)
    return ROUTER_EUNSUPPORTED;
  // One buffer descriptor covers the gathered activations, another one
  // expert's weights: 32-bit byte offsets below 2^31.
  if (operand_rows * (K / 2) > (int64_t(1) << 31) - 65536 || N * (K / 2) > (int64_t(1) << 31) - 65536)
    return ROUTER_EUNSUPPORTED;
  return ROUTER_OK;
}

size_t combine_scratch(int64_t T, int64_t k, int64_t N) { return (size_t)(T * k) * (size_t)N * sizeof(float); }

}  // namespace

extern "C" {

size_t grouped_workspace_bytes(int64_t T, int64_t k, int64_t G, int64_t D, int64_t F) {
  if (F < 1 || D < 1 || F > ROUTER_MAX_GATE_D || check_sizes(T, k, G, 1, 32, 0) != ROUTER_OK || D > ROUTER_MAX_GATE_D)
    return 0;
  const size_t p = nvr::plan_scratch_bytes(T * k, G), c = combine_scratch(T, k, D);
  return nvr::kScratchOffset + (p > c ? p : c);
}

int grouped_swiglu(const uint8_t* x_codes, const uint8_t* x_scales, const float* gsa, const uint8_t* w_codes,
                   const uint8_t* w_scales, const float* gsw, const float* bias, const int32_t* offsets,
                   const int32_t* rows, int64_t T, int64_t k, int64_t G, int64_t F, int64_t D, void* out,
                   void* stream) {
  if (F < 16 || F % 16 != 0) return ROUTER_EINVAL;
  const int st = check_sizes(T, k, G, 2 * F, D, T);
  if (st != ROUTER_OK) return st;
  if (!gsa || !w_codes || !w_scales || !gsw || !offsets) return ROUTER_EINVAL;
  if (T > 0 && (!x_codes || !x_scales || !rows || !out)) return ROUTER_EINVAL;
  if (!aligned(x_codes, 16) || !aligned(w_codes, 16) || !aligned(x_scales, 2) || !aligned(w_scales, 2) ||
      !aligned(gsa, 4) || !aligned(gsw, 4) || !aligned(bias, 4) || !aligned(offsets, 4) || !aligned(rows, 4) ||
      !aligned(out, 16))
    return ROUTER_EINVAL;
  if (T == 0) return ROUTER_OK;
  const nvr::ExpertArgs a{x_codes, x_scales, gsa, w_codes, w_scales, gsw, bias, offsets, rows, out,
                          (int)T, (int)k, (int)(T * k), (int)G, (int)(2 * F), (int)D, 0, 0, nvr::Take::kAll, 0};
  return status_from(nvr::launch_products<true>(a, static_cast<hipStream_t>(stream)));
}

int grouped_combine(const uint8_t* h_codes, const uint8_t* h_scales, const float* gsh, const uint8_t* w_codes,
                    const uint8_t* w_scales, const float* gsw, const float* bias, const int32_t* offsets,
                    const int32_t* pos, const float* topk_w, const void* residual, int64_t T, int64_t k, int64_t G,
                    int64_t D, int64_t F, void* out, void* workspace, size_t workspace_bytes, void* stream) {
  if (D < 16 || D % 16 != 0) return ROUTER_EINVAL;
  const int st = check_sizes(T, k, G, D, F, 0);
  if (st != ROUTER_OK) return st;
  if (!gsh || !w_codes || !w_scales || !gsw || !offsets) return ROUTER_EINVAL;
  if (T > 0 && (!h_codes || !h_scales || !pos || !topk_w || !out || !workspace)) return ROUTER_EINVAL;
  if (!aligned(h_codes, 16) || !aligned(w_codes, 16) || !aligned(h_scales, 2) || !aligned(w_scales, 2) ||
      !aligned(gsh, 4) || !aligned(gsw, 4) || !aligned(bias, 4) || !aligned(offsets, 4) || !aligned(pos, 4) ||
      !aligned(topk_w, 4) || !aligned(residual, 16) || !aligned(out, 16) || !aligned(workspace, 256))
    return ROUTER_EINVAL;
  if (T == 0) return ROUTER_OK;
  if (workspace_bytes < nvr::kScratchOffset + combine_scratch(T, k, D)) return ROUTER_EINVAL;
  float* y = reinterpret_cast<float*>(static_cast<char*>(workspace) + nvr::kScratchOffset);
  const nvr::ExpertArgs a{h_codes, h_scales, gsh, w_codes, w_scales, gsw, bias, offsets, nullptr, y,
                          (int)T, (int)k, (int)(T * k), (int)G, (int)D, (int)F, 0, 0, nvr::Take::kAll, 0};
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t cwg = (T * (D / 8) + 255) / 256;
  if (cwg >= (int64_t(1) << 31)) return ROUTER_EUNSUPPORTED;
  const hipError_t e = nvr::launch_products<false>(a, s);
  if (e != hipSuccess) return status_from(e);
  const nvr::CombineArgs c{y, pos, topk_w, static_cast<const uint16_t*>(residual), static_cast<uint16_t*>(out),
                           (int)T, (int)k, (int)(T * k), (int)D};
  nvr::combine_kernel<<<(int)cwg, 256, 0, s>>>(c);
  return status_from(hipGetLastError());
}

}  // extern "C"
