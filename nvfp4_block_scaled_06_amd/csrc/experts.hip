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
};

// Token of row p, or -1.
__device__ __forceinline__ int row_token(const ExpertArgs& a, int p) {
  const int s = a.rows[p];
  const int t = s / a.k;
  return s >= 0 && t < a.T ? t : -1;
}

__device__ __forceinline__ float silu_mul(float g, float u) { return g * sigmoid_fast(g) * u; }

// Zeros for the rows of no expert: router_quantize runs over all R rows, and
// stale values there would set its global scale.
__device__ __forceinline__ void zero_rows(const ExpertArgs& a, const RowTile& t, int col0, int cols, int nthreads) {
  uint16_t* out = static_cast<uint16_t*>(a.out);
  const int F = a.N >> 1, nc = min(cols, F - col0);
  for (int i = threadIdx.x; i < t.nr * nc; i += nthreads)
    out[(int64_t)(t.row0 + i / nc) * F + col0 + i % nc] = 0;
}

// Scale row offsets of a tile of gathered rows (A) and paired weight rows
// (B), from a table in LDS.
struct TableRows {
  const uint32_t* tab;
  int bm;
  __device__ __forceinline__ uint32_t operator()(bool isA, int rr) const { return tab[isA ? rr : bm + rr]; }
};

// One tile of BM rows of an expert times 128 NTW weight rows on the shared
// MFMA tile. GLU: the rows are gathered, and each 32-column tile holds 16
// gate rows and the 16 up rows of the same outputs, so that one lane swap
// brings the two halves of an output together.
template <bool GLU, int BM, int NTW, int KS, bool STAGED>
__global__ __launch_bounds__(kMmaThreads * KS) __attribute__((amdgpu_waves_per_eu(KS, KS))) void experts_mfma_kernel(
    ExpertArgs a) {
  static_assert(KS == mma_ksplit<BM, NTW>(), "K groups as the main loop has them");
  constexpr int BN = 128 * NTW;
  constexpr int SH = BM == 32 ? 5 : (BM == 64 ? 6 : 7);
  static_assert(BM == 1 << SH, "rows per tile");
  static_assert(KS == 1 || BM * BN * sizeof(float) <= sizeof(_Float16) * KS * 2 * BM * kMmaARow,
                "the epilogue's partial sums fit in the A tiles' LDS");
  __shared__ __attribute__((aligned(16))) _Float16 abuf[KS][2][BM * kMmaARow];
  __shared__ __attribute__((aligned(16))) uint8_t swin[STAGED ? mma_win_bytes<BM, NTW>() : 16];
  __shared__ uint32_t srow[GLU ? BM + BN : 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wt = wave & 3, grp = wave >> 2;
  const TileScan scan(a.offsets, a.G, a.R, SH);
  const int total = GLU ? scan.total : scan.experts;
  if ((int)blockIdx.x >= total * a.col_tiles) return;
  // Consecutive tiles (the column tiles of one row tile first) run on one
  // XCD, so a row tile's activations are fetched into one L2.
  const int n = xcd_order(blockIdx.x, total * a.col_tiles);
  const int ct = n % a.col_tiles;
  const RowTile rt = scan.at(n / a.col_tiles);
  const int row0 = rt.row0, nr = rt.nr;
  if (GLU && rt.g == a.G) {
    zero_rows(a, rt, ct * (BN / 2), BN / 2, kMmaThreads * KS);
    return;
  }
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
    mma_mainloop<BM, NTW, KS, STAGED>(P, a.D, a.nsteps, &abuf[0][0][0], swin, lane, acc, TableRows{srow, BM});
  else
    mma_mainloop<BM, NTW, KS, STAGED>(P, a.D, a.nsteps, &abuf[0][0][0], swin, lane, acc);

  // 32x32 accumulator layout: value v of lane (r, h) is row 8(v/4) + 4h +
  // v%4, column r of its tile; wavefront wt holds the column tiles wt + 4t.
  float* part = reinterpret_cast<float*>(&abuf[0][0][0]);  // [BM][BN], K group 1's sums
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

// Few rows per expert: a stream of the hit experts' weights. Workgroup (row
// tile of up to 4 rows of an expert, column tile) = 64 weight rows, four
// wavefronts of 16 rows with the loads of 2 in flight, as in the lm_head
// GEMV. GLU: a wavefront's rows are the gate and up rows of 8 outputs in
// turn.
constexpr int kEvWaves = 4;
constexpr int kEvThreads = 64 * kEvWaves;
constexpr int kEvRowsPerWave = 16;
constexpr int kEvCols = kEvWaves * kEvRowsPerWave;
constexpr int kEvInFlight = 2;
constexpr int kEvMaxRows = 4;
constexpr int kEvMaxXHalves = 32768;  // rows x D of the fp16 x copy in LDS (64 KB)

template <bool GLU, int CPL, int NR>
__global__ __launch_bounds__(kEvThreads) void experts_gemv_kernel(ExpertArgs a) {
  extern __shared__ half8_t xg[];  // [nr][D / 8]
  constexpr int SH = NR == 1 ? 0 : (NR == 2 ? 1 : 2);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const TileScan scan(a.offsets, a.G, a.R, SH);
  const int total = GLU ? scan.total : scan.experts;
  if ((int)blockIdx.x >= total * a.col_tiles) return;
  const int n = xcd_order(blockIdx.x, total * a.col_tiles);
  const int ct = n % a.col_tiles;
  const RowTile rt = scan.at(n / a.col_tiles);
  if (GLU && rt.g == a.G) {
    zero_rows(a, rt, ct * (kEvCols / 2), kEvCols / 2, kEvThreads);
    return;
  }
  const int nr = rt.nr, F = a.N >> 1, nch = a.D >> 5;
  const int64_t rowc = a.D / 2, rows = a.D / 16;
  const float gsa = load_early(a.gsa), gsw = load_early(a.gsw + rt.g);
  for (int i = threadIdx.x; i < nr * nch; i += kEvThreads) {
    const int t = i / nch, c = i - t * nch;
    const int64_t xr = GLU ? row_token(a, rt.row0 + t) : rt.row0 + t;
    u32x4_t v{0u, 0u, 0u, 0u};
    uint32_t sb = 0u;
    if (!GLU || xr >= 0) {
      v = *reinterpret_cast<const u32x4_t*>(a.xc + xr * rowc + 16 * c);
      sb = *reinterpret_cast<const uint16_t*>(a.xs + xr * rows + 2 * c);
    }
    const _Float16 s0 = e4m3_f16(sb & 0xFFu), s1 = e4m3_f16(sb >> 8);
    half8_t* d = xg + (int64_t)t * (nch * 4) + 4 * c;
    d[0] = fp4x8_to_f16(v[0], s0);
    d[1] = fp4x8_to_f16(v[1], s0);
    d[2] = fp4x8_to_f16(v[2], s1);
    d[3] = fp4x8_to_f16(v[3], s1);
  }
  __syncthreads();

  const float scale = gsa * gsw;
  const int64_t we = (int64_t)rt.g * a.N;
  const __amdgpu_buffer_rsrc_t wcr = make_rsrc(a.wc + we * rowc, a.N * rowc);
  const __amdgpu_buffer_rsrc_t wsr = make_rsrc(a.ws + we * rows, a.N * rows);
  // Weight row of this wavefront's u-th row (-1: behind the last one).
  auto wrow = [&](int u) {
    const int i = wave * kEvRowsPerWave + u;
    if constexpr (GLU) {
      const int f = ct * (kEvCols / 2) + (i >> 1);
      return f < F ? (i & 1 ? F + f : f) : -1;
    } else {
      const int c = ct * kEvCols + i;
      return c < a.N ? c : -1;
    }
  };
  uint32_t oc[CPL], os[CPL];
#pragma unroll
  for (int i = 0; i < CPL; ++i) {
    const int c = lane + 64 * i;
    oc[i] = c < nch ? (uint32_t)(16 * c) : kMmaOob;
    os[i] = c < nch ? (uint32_t)(2 * c) : kMmaOob;
  }
  u32x4_t wv[kEvInFlight][CPL];
  uint32_t wsv[kEvInFlight][CPL];
  auto load_row = [&](int slot, int u) {
    // A row behind the last one re-reads row 0 (not used), so every offset
    // stays in range or at kMmaOob plus less than 2^31.
    const int w = max(wrow(u), 0);
    const uint32_t rc = (uint32_t)w * (uint32_t)rowc, rs = (uint32_t)w * (uint32_t)rows;
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      wv[slot][i] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(wcr, oc[i] + rc, 0, kNtAux));
      wsv[slot][i] = __builtin_amdgcn_raw_buffer_load_b16(wsr, os[i] + rs, 0, kNtAux);
    }
  };
#pragma unroll
  for (int u = 0; u < kEvInFlight; ++u) load_row(u, u);
  float gate[NR];
#pragma unroll
  for (int u = 0; u < kEvRowsPerWave; ++u) {
    const int slot = u % kEvInFlight, w = wrow(u);
    float acc[NR];
#pragma unroll
    for (int t = 0; t < NR; ++t) acc[t] = 0.0f;
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      const int c = min(lane + 64 * i, nch - 1);  // chunks past D hold zero weights
      const _Float16 s0 = e4m3_f16(wsv[slot][i] & 0xFFu), s1 = e4m3_f16(wsv[slot][i] >> 8);
      const half8_t w0 = fp4x8_to_f16(wv[slot][i][0], s0), w1 = fp4x8_to_f16(wv[slot][i][1], s0);
      const half8_t w2 = fp4x8_to_f16(wv[slot][i][2], s1), w3 = fp4x8_to_f16(wv[slot][i][3], s1);
#pragma unroll
      for (int t = 0; t < NR; ++t) {
        if (t < nr) {
          const half8_t* xp = xg + (int64_t)t * (nch * 4) + 4 * c;
          acc[t] += dot8(xp[1], w1, dot8(xp[0], w0, 0.0f));
          acc[t] += dot8(xp[3], w3, dot8(xp[2], w2, 0.0f));
        }
      }
    }
    if (u + kEvInFlight < kEvRowsPerWave) load_row(slot, u + kEvInFlight);
    const float b = a.bias && w >= 0 ? a.bias[we + w] : 0.0f;
#pragma unroll
    for (int t = 0; t < NR; ++t) {
      if (t < nr) {
        const float y = wave_sum(acc[t]) * scale + b;
        const int64_t p = rt.row0 + t;
        if constexpr (GLU) {
          if ((u & 1) == 0) gate[t] = y;
          else if (lane == 0 && w >= 0)
            static_cast<uint16_t*>(a.out)[p * F + (w - F)] = bf16_round(silu_mul(gate[t], y));
        } else if (lane == 0 && w >= 0) {
          static_cast<float*>(a.out)[p * a.N + w] = y;
        }
      }
    }
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

template <bool GLU, int CPL, int NR>
static hipError_t launch_gemv_t(ExpertArgs a, hipStream_t stream) {
  a.col_tiles = (a.N + kEvCols - 1) / kEvCols;
  const int64_t nwg = max_row_tiles(a.R, a.G, NR == 1 ? 0 : (NR == 2 ? 1 : 2)) * a.col_tiles;
  if (nwg >= (int64_t(1) << 31)) return hipErrorInvalidConfiguration;
  experts_gemv_kernel<GLU, CPL, NR><<<(int)nwg, kEvThreads, (size_t)NR * a.D * sizeof(_Float16), stream>>>(a);
  return hipGetLastError();
}

template <bool GLU, int CPL>
static hipError_t launch_gemv_n(const ExpertArgs& a, int nr, hipStream_t stream) {
  if (nr == 1) return launch_gemv_t<GLU, CPL, 1>(a, stream);
  if (nr == 2) return launch_gemv_t<GLU, CPL, 2>(a, stream);
  return launch_gemv_t<GLU, CPL, 4>(a, stream);
}

template <bool GLU>
static hipError_t launch_gemv(const ExpertArgs& a, int nr, hipStream_t stream) {
  const int cpl = ((a.D >> 5) + 63) / 64;
  if (cpl <= 1) return launch_gemv_n<GLU, 1>(a, nr, stream);
  if (cpl <= 2) return launch_gemv_n<GLU, 2>(a, nr, stream);
  if (cpl <= 4) return launch_gemv_n<GLU, 4>(a, nr, stream);
  return launch_gemv_n<GLU, 8>(a, nr, stream);
}

// Rows per GEMV tile, or 0 for the MFMA tiles.
static int gemv_rows(int64_t T, int64_t R, int64_t G, int64_t D) {
  if (D > 16384 || R > 4 * G) return 0;
  const int nr = T == 1 ? 1 : (T == 2 ? 2 : 4);
  return nr * D <= kEvMaxXHalves ? nr : (2 * D <= kEvMaxXHalves ? 2 : 1);
}

template <bool GLU>
static hipError_t launch_products(const ExpertArgs& a, hipStream_t stream) {
  const int nr = gemv_rows(a.T, a.R, a.G, a.D);
  if (nr > 0) return launch_gemv<GLU>(a, nr, stream);
  const int64_t mean = a.R / a.G;
  if (mean <= 32) return launch_mfma<GLU, 32, 1>(a, stream);
  if (mean <= 64) return launch_mfma<GLU, 64, 1>(a, stream);
  return launch_mfma<GLU, 128, 2>(a, stream);
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
                          (int)T, (int)k, (int)(T * k), (int)G, (int)(2 * F), (int)D, 0, 0};
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
                          (int)T, (int)k, (int)(T * k), (int)G, (int)D, (int)F, 0, 0};
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
