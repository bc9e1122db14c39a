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
  int col_tiles;
  Take take;      // which experts this launch takes
  int tile_cols;  // column tiles of the 128-row tile kernel
  int max_tiles;  // no plan gives more row tiles
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
// False behind the last item, and for offsets that no plan gives and that ask
// for more tiles than R rows can.
struct ExpertTile {
  RowTile rt;
  int ct;
};
__device__ __forceinline__ bool expert_tile(const ExpertArgs& a, const TileScan& scan, bool others, int b,
                                            ExpertTile& t) {
  if (scan.experts > a.max_tiles) return false;
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

// How weight scales are read: in pieces of 16 bytes (K a multiple of 256), of
// 4 bytes (of 64), or of 4 bytes where the odd rows start 2 bytes past a
// multiple of 4 (other multiples of 32): a window of those takes one piece
// more, from the multiple below, and its scales lie 2 bytes further on in
// LDS. Weights have a multiple of 16 rows, so no piece passes an expert's end.
// (2-byte pieces in twice as many loads, whose registers left the wide tiles
// 96 rows: K = 2016, 112 rows per expert 197 us against 178; K = 6048, 514
// against 486.)
enum class Scales { k16, k4, kSkewed };

// One load of SW bytes of weight scales, and its way into LDS (4-byte aligned
// there).
template <int SW>
struct ScaleLoad {
  static_assert(SW == 16 || SW == 4, "a buffer load's sizes");
  uint32_t v[SW / 4];
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t at) {
    if constexpr (SW == 16) {
      const u32x4_t x = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0));
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = x[i];
    } else v[0] = __builtin_amdgcn_raw_buffer_load_b32(r, at, 0, 0);
  }
  __device__ __forceinline__ void store(uint8_t* d) const {
#pragma unroll
    for (int i = 0; i < SW / 4; ++i) reinterpret_cast<uint32_t*>(d)[i] = v[i];
  }
};

// v in the lanes whose 32 K values lie before the row's end, 0 in those past
// it: each LANES lanes hold the next 32 of a uniform `left` (a multiple of 32)
// K values. The lanes come as a scalar mask: the wide tiles have no register
// for a lane's own bound (spills of 3). Costs up to 0.7 % (T = 1, 64, 1024;
// K = 7104, 7136, 2016, 1984), at T = 1 and K = 7104 1.6 %.
template <int LANES>
__device__ __forceinline__ uint32_t within(uint32_t v, int left) {
  const int n = __builtin_amdgcn_readfirstlane(min(max(left, 0) / 32 * LANES, 64));
  return __builtin_amdgcn_inverse_ballot_w64(n < 64 ? (1ull << n) - 1ull : ~0ull) ? v : 0u;
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
//  * KG = 2: two groups of four wavefronts take the 512-value windows in turn
//    and group 0 adds group 1's sums (fixed order). With few workgroups a
//    wavefront's own chain of steps bounds the time, not the memory.
//  * Past D the x tile holds zeros, and what a padded step reads of the next
//    weight row there takes a scale of zero: codes are finite, but scale bytes
//    0x7F and 0xFF are NaN, and 0 NaN is NaN.
// Bound by HBM: grouped_swiglu at T = 64, D = 7168, F = 2048, k = 8 needs the
// 2.7 GB of the 165 of 256 experts that tokens hit under a mild skew, reads
// 2.9 GB and takes 450 us, 6.5 TB/s; grouped_combine needs 1.36 GB, reads 1.62
// and takes 267 us, 6.1 TB/s. The loads ahead have no bound at K: what they
// read past it (of the rows that follow) is more the shorter K is. At T = 1
// (132 MB, 26 us in the kernel) by the latency of a workgroup's chain of
// steps.
constexpr int kEsWaves = 4;
constexpr int kEsThreads = 64 * kEsWaves;
constexpr int kEsRows = 32;       // weight rows per wavefront
constexpr int kEsSharedGrid = 256 * 6;  // workgroups that share a launch's items
constexpr int kEsManyItems = 12288;
constexpr int kEsFewItems = 256;
constexpr int kEsScaleLd = 36;    // LDS bytes per row of a scale window (32 + 4)

template <int MR, int KB, int KG>
struct StreamLds {
  alignas(16) _Float16 x[2][MR * KB];
  alignas(16) uint8_t codes[KG * kEsWaves][kEsRows * 128];
  alignas(16) uint8_t scales[KG * kEsWaves][kEsRows * kEsScaleLd];
};

// Halves offset of 16-byte piece c of row r of an x tile: the 16 rows of a
// 16-row tile side by side for each piece, so that the rows of one read lie
// in different banks whichever pieces the lanes take; XOR-swizzled so that the
// pieces of one row do too when they are written (row-major tiles swizzled by
// row had half of all LDS cycles in bank conflicts).
template <int MR>
__device__ __forceinline__ int stream_x_at(int r, int c) {
  return ((c * (MR / 16) + (r >> 4)) * 16 + ((r ^ (c >> 2)) & 15)) * 8;
}

// One tile.
template <bool GLU, int MR, int KB, int KG, Scales S>
__device__ __forceinline__ void stream_tile(const ExpertArgs& a, const ExpertTile& tile, StreamLds<MR, KB, KG>& lds) {
  constexpr int NT = MR / 16, NTHREADS = KG * kEsThreads;
  static_assert(KG == 1 ? KB == 256 || KB == 512 : KB == 512 * KG, "whole steps, and a window for each K group");
  constexpr int XP = MR * (KB / 32) / NTHREADS;  // 32-value pieces of x per thread and block
  static_assert(XP * NTHREADS == MR * (KB / 32), "whole pieces per thread");
  constexpr int SPB = KB / 256 / KG;  // steps per x block of a K group
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, grp = KG == 1 ? 0 : wave / kEsWaves;
  const RowTile& rt = tile.rt;
  const float gsa = load_early(a.gsa), gsw = load_early(a.gsw + rt.g);
  const int nr = rt.nr, F = a.N >> 1;
  const int64_t rowc = a.D / 2, rows = a.D / 16, we = (int64_t)rt.g * a.N;
  // This wavefront's first output (GLU) or weight row, and its two 16-row tiles.
  const int o0 = (tile.ct * kEsWaves + wave % kEsWaves) * (GLU ? 16 : 32);
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
  // Scale window: SP pieces of SW bytes per row, 64 / SP rows in each of SL loads; and a load of the rows' last pieces.
  constexpr bool SKEW = S == Scales::kSkewed;
  constexpr int SW = S == Scales::k16 ? 16 : 4, SP = 32 / SW, SL = SP / 2;
  const int srow = lane / SP, sbyte = SW * (lane % SP);
  auto sbase = [&](int m, int row) {
    const uint32_t at = (uint32_t)((wrow(m) + (row & 15)) * rows);
    return (m ? live1 : live0) ? (SKEW ? at & ~3u : at) : kMmaOob;
  };
  uint32_t so[SL], so_last = 0u;
#pragma unroll
  for (int i = 0; i < SL; ++i) {
    const int row = 64 / SP * i + srow;
    so[i] = sbase(SL == 1 ? row >> 4 : i / (SL / 2), row) + sbyte;
  }
  if constexpr (SKEW) so_last = lane < 32 ? sbase(lane >> 4, lane) + 32 : kMmaOob;
  ScaleLoad<SW> sv[SL];
  ScaleLoad<4> sv_last;
  auto load_s = [&](int win) {
#pragma unroll
    for (int i = 0; i < SL; ++i) sv[i].load(wsr, so[i] + 32 * win);
    if constexpr (SKEW) sv_last.load(wsr, so_last + 32 * win);
  };
  uint8_t* my_codes = lds.codes[wave];
  uint8_t* my_scales = lds.scales[wave];
  auto store_s = [&]() {
#pragma unroll
    for (int i = 0; i < SL; ++i) sv[i].store(my_scales + (64 / SP * i + srow) * kEsScaleLd + sbyte);
    if constexpr (SKEW)
      if (lane < 32) sv_last.store(my_scales + lane * kEsScaleLd + 32);
  };

  // The weights' first loads go out before the rows are looked up.
  load_w(0, 2 * grp);
  load_w(1, 2 * grp + 1);
  load_s(grp);
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
        *reinterpret_cast<half8_t*>(&lds.x[buf][stream_x_at<MR>(r, 4 * c + j)]) = fp4x8_scaled(xv[i][j], s, j >> 1);
    }
  };

  const int nsteps = (a.D + 255) / 256;
  load_x(0);
  store_x(0, 0);
  __syncthreads();
  f32x4_t acc[2][NT];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[m][t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  const int r = lane & 15, q = lane >> 4;
  const uint8_t* row_scales = my_scales + r * kEsScaleLd + 2 * q + (SKEW ? 2 * (r & 1) : 0);
  for (int w0 = 0; 2 * w0 < nsteps; w0 += KG) {  // windows, one for each K group
    // The window's scales; the next one's loads.
    store_s();
    load_s(w0 + grp + KG);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int step = 2 * (w0 + grp) + u;
      const int block = KG == 1 ? step / SPB : w0 / KG, in = u % SPB, buf = block & 1;
      // Before the weight loads: loads complete in order, and the wait for x
      // at the end of the block must not wait for weights two steps ahead.
      if (in == 0) load_x((block + 1) * KB);
      // Codes through LDS into MFMA layout.
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 8 * i + (lane >> 3);
        *reinterpret_cast<u32x4_t*>(my_codes + row * 128 + 16 * ((lane & 7) ^ (row & 7))) = wv[u][i];
      }
      load_w(u, step + 2 * KG);
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
            const uint32_t sw = lds_u16(row_scales + 16 * m * kEsScaleLd + 16 * u + 8 * g);
            s[m] = e4m3x2_f16(S == Scales::k16 ? sw : within<16>(sw, a.D - (256 * step + 128 * g)));
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            half8_t w[2];
#pragma unroll
            for (int m = 0; m < 2; ++m) w[m] = fp4x8_scaled(c[m][j], s[m], j >> 1);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              const half8_t xf = *reinterpret_cast<const half8_t*>(
                  &lds.x[buf][stream_x_at<MR>(16 * t + r, 32 * (SPB * grp + in) + 16 * g + 4 * q + j)]);
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

  if constexpr (KG == 2) {
    // The x tiles are done with: group 1's sums go through the first.
    float* part = reinterpret_cast<float*>(&lds.x[0][0]) + (wave % kEsWaves) * (64 * 8 * NT) + lane;
    static_assert(kEsWaves * 64 * 8 * NT * sizeof(float) <= sizeof(lds.x), "partial sums fit");
    if (grp == 1) {
#pragma unroll
      for (int i = 0; i < 8 * NT; ++i) part[64 * i] = acc[i / (4 * NT)][(i >> 2) % NT][i & 3];
    }
    __syncthreads();
    if (grp == 1) return;
#pragma unroll
    for (int i = 0; i < 8 * NT; ++i) acc[i / (4 * NT)][(i >> 2) % NT][i & 3] += part[64 * i];
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
template <bool GLU, int MR, int KB, int KG, Scales S, bool SHARED>
__global__ __launch_bounds__(KG * kEsThreads) void experts_stream_kernel(ExpertArgs a) {
  __shared__ StreamLds<MR, KB, KG> lds;
  const TileScan scan(a.offsets, a.G, a.R, MR, a.take, a.tile_cols);
  ExpertTile tile;
  for (int b = blockIdx.x; expert_tile(a, scan, GLU, b, tile); b += gridDim.x) {
    if (GLU && tile.rt.g == a.G) zero_rows(a, tile.rt, KG * kEsThreads);
    else stream_tile<GLU, MR, KB, KG, S>(a, tile, lds);
    if (!SHARED) return;
    __syncthreads();  // the next item writes the LDS tiles
  }
}

// Many rows per expert: workgroup tile = up to 128 rows of an expert times 512
// weight rows, 8 wavefronts, two per SIMD, so that one's conversions run
// under the other's MFMAs. Wavefront = 64 weight rows (GLU: 32 gate rows and
// the 32 up rows of the same outputs) times every row of the tile on 32x32x16
// MFMAs.
//  * B (weights): as in the stream: 256 K values per row at a time in whole
//    lines, through 8 KB of LDS private to the wavefront into MFMA layout, one
//    conversion for all the tile's rows.
//  * A (rows): 128 K values per step, converted once per workgroup into one
//    of two LDS tiles of fp16 q S values.
//  * K order: in every 64 values lane (r, h) supplies [32h + 8j, +8) to MFMA j,
//    on A and B alike.
//  * Past D, as in the stream: x of zeros, weight scales of zero.
//  * RT: 32-row tiles of the row tile, so a ragged tail costs its own size.
// Bound by the matrix cores and the clock that their power leaves (58 % busy
// at 1.82 GHz): grouped_swiglu at T = 8192, D = 7168, F = 2048, 256 experts
// takes 3.58 ms with its small experts' launch, 1075 TFLOP/s on the rows
// alone; 2.9 ms on x of zeros, and 2.8 without the loop's loads, on stale
// values. Four wavefronts per 128 x 256 tile, one per SIMD: 4.06 ms.
// Full tiles of even experts: 1233 TFLOP/s (256 rows each).
constexpr int kEtWaves = 8;
constexpr int kEtThreads = 64 * kEtWaves;
constexpr int kEtRows = 128;
constexpr int kEtCols = 64 * kEtWaves;
constexpr int kEtScaleLd = 20;  // LDS bytes per weight row of 256 K values' scales (16 + 4)

struct TileLds {
  alignas(16) _Float16 x[2][128 * 128];
  alignas(16) uint8_t codes[kEtWaves][64 * 128];
  alignas(16) uint8_t scales[kEtWaves][64 * kEtScaleLd];
};

// Halves offset of 16-byte piece c (of 16) of row r of an A tile: 32 rows side
// by side for each piece, swizzled for the writes.
__device__ __forceinline__ int tile_x_at(int r, int c) {
  return (((r >> 5) * 16 + c) * 32 + ((r & 31) ^ (c & 12))) * 8;
}

template <bool GLU, int RT, Scales S>
__device__ __forceinline__ void wide_tile(const ExpertArgs& a, const ExpertTile& tile, TileLds& lds) {
  const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const RowTile& rt = tile.rt;
  const float gsa = load_early(a.gsa), gsw = load_early(a.gsw + rt.g);
  const int nr = rt.nr, F = a.N >> 1;
  const int64_t rowc = a.D / 2, rows = a.D / 16, we = (int64_t)rt.g * a.N;
  const int o0 = (tile.ct * kEtWaves + wave) * (GLU ? 32 : 64);  // this wavefront's first output
  // Weight row of its column c (0 .. 63), -1 past the last one (columns come and go 16 at a time).
  auto wrow = [&](int c) {
    const int o = GLU ? o0 + (c & 31) : o0 + c;
    return GLU ? (o < F ? (c & 32 ? F + o : o) : -1) : (o < a.N ? o : -1);
  };
  const __amdgpu_buffer_rsrc_t wcr = make_rsrc(a.wc + we * rowc, a.N * rowc);
  const __amdgpu_buffer_rsrc_t wsr = make_rsrc(a.ws + we * rows, a.N * rows);
  // Load i takes 8 rows: a scalar offset for its first row, a lane's offset within the 8.
  const uint32_t wlane = (uint32_t)((lane >> 3) * rowc + 16 * (lane & 7));
  auto wbase = [&](int c, int64_t ld) { return wrow(c) >= 0 ? (uint32_t)(wrow(c) * ld) : kMmaOob; };
  // Scales of 256 K values: SL pieces of SW bytes per row, SR rows in each of SL loads; and a load of the rows' last
  // pieces.
  constexpr bool SKEW = S == Scales::kSkewed;
  constexpr int SW = S == Scales::k16 ? 16 : 4, SL = 16 / SW, SR = 64 / SL;
  const int srow = lane / SL, sbyte = SW * (lane % SL);
  auto sown = [&](int c) { return wrow(c) >= 0 ? (uint32_t)(wrow(c) * rows) & ~3u : kMmaOob; };
  auto slane = [&](int c) { return SL > 1 ? ((uint32_t)(c / SL * rows) & ~3u) + SW * (c % SL) : sown(c); };
  ScaleLoad<4> sv_last;
  u32x4_t wv[8];
  ScaleLoad<SW> sv[SL];
  auto load_w = [&](int batch) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      wv[i] = __builtin_bit_cast(
          u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(wcr, wlane + (wbase(8 * i, rowc) + 128 * batch), 0, 0));
    int c = lane;
    if constexpr (SKEW) asm volatile("" : "+v"(c));  // offsets computed here each time: no registers hold them
#pragma unroll
    for (int i = 0; i < SL; ++i) sv[i].load(wsr, slane(c) + ((SL > 1 ? wbase(SR * i, rows) : 0u) + 16 * batch));
    if constexpr (SKEW) sv_last.load(wsr, sown(c) + 16 + 16 * batch);
  };
  uint8_t* codes = lds.codes[wave];
  uint8_t* scales = lds.scales[wave];
  auto store_w = [&]() {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = 8 * i + (lane >> 3);
      *reinterpret_cast<u32x4_t*>(codes + row * 128 + 16 * ((lane & 7) ^ ((row >> 1) & 7))) = wv[i];
    }
#pragma unroll
    for (int i = 0; i < SL; ++i) sv[i].store(scales + (SR * i + srow) * kEtScaleLd + sbyte);
    if constexpr (SKEW) sv_last.store(scales + lane * kEtScaleLd + 16);
  };
  load_w(0);

  // A: thread = (row, 32 K values of a step).
  const int ar = threadIdx.x >> 2, aq = threadIdx.x & 3;
  int t = -1;
  if (ar < nr) t = GLU ? row_token(a, rt.row0 + ar) : ar;
  const __amdgpu_buffer_rsrc_t xcr =
      GLU ? make_rsrc(a.xc, a.T * rowc) : make_rsrc(a.xc + rt.row0 * rowc, nr * rowc);
  const __amdgpu_buffer_rsrc_t xsr =
      GLU ? make_rsrc(a.xs, a.T * rows) : make_rsrc(a.xs + rt.row0 * rows, nr * rows);
  const uint32_t xo = t >= 0 ? (uint32_t)(t * rowc + 16 * aq) : kMmaOob;
  const uint32_t xso = t >= 0 ? (uint32_t)(t * rows + 2 * aq) : kMmaOob;
  u32x4_t xv[2];
  uint32_t xsv[2];
  auto load_x = [&](int k, int step) {
    const bool ok = 128 * step + 32 * aq < a.D;  // zeros past D, whatever the weights there
    xv[k] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(xcr, ok ? xo + 64 * step : kMmaOob, 0, 0));
    xsv[k] = __builtin_amdgcn_raw_buffer_load_b16(xsr, ok ? xso + 8 * step : kMmaOob, 0, 0);
  };
  auto store_x = [&](int k, int buf, int j) {  // 8 of the 32 values
    if (RT < 4 && ar >= 32 * RT) return;
    const half2_t s = e4m3x2_f16(xsv[k]);
    *reinterpret_cast<half8_t*>(&lds.x[buf][tile_x_at(ar, 4 * aq + j)]) = fp4x8_scaled(xv[k][j], s, j >> 1);
  };
  // A fragment of row tile i, and a lane's codes and scales of a 64-value group, of slice sl of a batch.
  auto afrag = [&](int i, int sl) {
    return *reinterpret_cast<const half8_t*>(&lds.x[(sl >> 3) & 1][tile_x_at(32 * i + r, 8 * ((sl >> 2) & 1) + 4 * h + (sl & 3))]);
  };
  u32x4_t c[2];
  uint32_t sc[2];
  auto read_codes = [&](int m, int batch, int group) {
    const int row = 32 * m + r;
    c[m] = *reinterpret_cast<const u32x4_t*>(codes + row * 128 + 16 * ((2 * group + h) ^ ((row >> 1) & 7)));
    sc[m] = lds_u16(scales + row * kEtScaleLd + 4 * group + 2 * h + (SKEW ? 2 * (r & 1) : 0));
    if constexpr (S != Scales::k16) sc[m] = within<32>(sc[m], a.D - (256 * batch + 64 * group));
  };
  auto wave_fence = [&]() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  };

  const int nbatch = (a.D + 255) / 256;
  load_x(0, 0);
#pragma unroll
  for (int j = 0; j < 4; ++j) store_x(0, 0, j);
  store_w();
  load_x(0, 1);
  load_x(1, 2);
  // The loop carries xsv as 32-bit values: as zero-extended 16-bit ones the
  // compiler would extend them at the loop's start, ahead of their use, and
  // wait there for every load in flight.
  uint32_t zero = 0u;
  asm volatile("" : "+v"(zero));
  xsv[0] |= zero;
  xsv[1] |= zero;
  __builtin_amdgcn_sched_barrier(0);
  load_w(1);
  __syncthreads();
  f32x16_t acc[RT][2];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][m][v] = 0.0f;

  // One batch is 16 slices of 16 K values: two steps (A tiles) of two groups
  // of four. In a slice the MFMAs of the first 32 columns run while the second
  // 32 columns' weights of the slice are converted, then the other way round
  // for the next slice, so that each has one register set; A fragment i is
  // read right after its last MFMA of the slice before, the codes of a group
  // at the end of the one before. The next batch's codes go to LDS when the
  // last group of this one has been read, and the loads for the batch after
  // follow at once (x before the weights: loads complete in order). No
  // register may spill here: its reload would wait for every load in flight.
  half8_t A[RT], w[2];
  read_codes(0, 0, 0);
  read_codes(1, 0, 0);
  w[0] = fp4x8_scaled(c[0][0], e4m3x2_f16(sc[0]), 0);
  for (int b = 0; b < nbatch; ++b) {
    static_for<0, 16>([&](auto slc) {
      constexpr int sl = decltype(slc)::value, u = sl >> 3, j = sl & 3, group = sl >> 2;
      constexpr bool first = (sl & 7) == 0, last = (sl & 7) == 7;
      if constexpr (first) {
#pragma unroll
        for (int i = 0; i < RT; ++i) A[i] = afrag(i, sl);
      }
      static_for<0, 2>([&](auto mc) {
        constexpr int m = decltype(mc)::value, jn = m == 0 ? j : (j + 1) & 3;
        // Phase m: MFMAs of columns 32 m; w[1 - m] is converted, for this
        // slice (m = 0) or the next (m = 1).
        static_for<0, RT>([&](auto ic) {
          constexpr int i = decltype(ic)::value;
          acc[i][m] = mfma32(A[i], w[m], acc[i][m]);
          if constexpr (m == 1 && !last) A[i] = afrag(i, sl + 1);
          static_for<i * 4 / RT, (i + 1) * 4 / RT>([&](auto kc) {
            constexpr int k = decltype(kc)::value;
            const half2_t s2 = e4m3x2_f16(sc[1 - m]);
            const _Float16 sv = (jn >> 1) ? s2[1] : s2[0];
            reinterpret_cast<half2_t*>(&w[1 - m])[k] =
                __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c[1 - m][jn], 1.0f, k) * half2_t{sv, sv};
          });
          __builtin_amdgcn_sched_barrier(0);
        });
        if constexpr (m == 0 && j == 3 && sl != 15) read_codes(1, b, group + 1);
        if constexpr (m == 0 && sl == 15) read_codes(1, b + 1, 0);
        if constexpr (m == 1 && j == 2 && sl != 14) read_codes(0, b, group + 1);
        if constexpr (m == 1 && sl == 14) read_codes(0, b + 1, 0);
        if constexpr (m == 0 && sl == 13) {
          wave_fence();
          store_w();
          wave_fence();
          load_x(1, 2 * b + 4);
          __builtin_amdgcn_sched_barrier(0);
          load_w(b + 2);
        }
      });
      // The next step's A tile, a quarter in each of four slices; its
      // registers take the step after the next one's.
      if constexpr ((sl & 7) >= 1 && (sl & 7) < 5) store_x(u, u ^ 1, (sl & 7) - 1);
      if constexpr (sl == 5) load_x(0, 2 * b + 3);
      if constexpr (last) __syncthreads();
    });
  }

  // Value v of lane (r, h): row 8 (v / 4) + 4 h + v % 4 of its 32-row tile, column r of its 32 weight rows.
  const float scale = gsa * gsw;
  if constexpr (GLU) {
    const int f = o0 + r;
    if (f >= F) return;
    const float bg = a.bias ? a.bias[we + f] : 0.0f, bu = a.bias ? a.bias[we + F + f] : 0.0f;
    uint16_t* out = static_cast<uint16_t*>(a.out) + (int64_t)rt.row0 * F + f;
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int row = 32 * i + 8 * (v >> 2) + 4 * h + (v & 3);
        if (row < nr)
          out[(int64_t)row * F] = bf16_round(silu_mul(acc[i][0][v] * scale + bg, acc[i][1][v] * scale + bu));
      }
  } else {
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const int n = o0 + 32 * m + r;
      if (n >= a.N) continue;
      const float b = a.bias ? a.bias[we + n] : 0.0f;
      float* out = static_cast<float*>(a.out) + (int64_t)rt.row0 * a.N + n;
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          const int row = 32 * i + 8 * (v >> 2) + 4 * h + (v & 3);
          if (row < nr) __builtin_nontemporal_store(acc[i][m][v] * scale + b, out + (int64_t)row * a.N);
        }
    }
  }
}

template <bool GLU, Scales S>
__global__ __launch_bounds__(kEtThreads) __attribute__((amdgpu_waves_per_eu(2, 2))) void experts_wide_kernel(
    ExpertArgs a) {
  __shared__ TileLds lds;
  const TileScan scan(a.offsets, a.G, a.R, kEtRows, a.take, a.tile_cols);
  ExpertTile tile;
  if (!expert_tile(a, scan, false, blockIdx.x, tile)) return;
  const int nr = tile.rt.nr;
  if (nr > 96) wide_tile<GLU, 4, S>(a, tile, lds);
  else if (nr > 64) wide_tile<GLU, 3, S>(a, tile, lds);
  else if (nr > 32) wide_tile<GLU, 2, S>(a, tile, lds);
  else wide_tile<GLU, 1, S>(a, tile, lds);
}

// out[t, n] = residual[t, n] + sum_j w[t, j] y[pos[t, j], n], j in order, 8
// columns per thread. Bound by HBM: at T = 8192, D = 7168 it reads the 1.88 GB
// of products at 5 TB/s. The products are written past the caches, which they
// would fill with lines that only this kernel reads, and every choice's loads
// are in flight at once: 2.45 ms for the whole call instead of 2.49. (Read
// past the caches too: 2.63 ms. Sums by the last workgroup of a column tile, for one
// launch at few rows, gained nothing: T = 1 23.4 us against 23.8, T = 4 62
// against 59.)
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
#pragma unroll 8
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
// The widest pieces that are aligned and never reach past a row (4-byte ones
// where 16 bytes would do cost 1 - 1.6 % at T = 8192 and 1024).
static Scales scales_of(const ExpertArgs& a) {
  if (a.D % 256 == 0 && reinterpret_cast<uintptr_t>(a.ws) % 16 == 0) return Scales::k16;
  return a.D % 64 == 0 ? Scales::k4 : Scales::kSkewed;
}

template <bool GLU>
static hipError_t launch_wide(ExpertArgs a, hipStream_t stream) {
  a.col_tiles = (a.N + kEtCols - 1) / kEtCols;
  // Tiles of 64 rows only while kOneRound work items take them all.
  a.max_tiles = (int)max_row_tiles(a.R, a.G, kEtRows / 2);
  const int64_t nwg = std::max(max_row_tiles(a.R, a.G, kEtRows) * a.col_tiles,
                               std::min(a.max_tiles * (int64_t)a.col_tiles, (int64_t)kOneRound));
  if (a.max_tiles * (int64_t)a.col_tiles >= (int64_t(1) << 31)) return hipErrorInvalidConfiguration;
  switch (scales_of(a)) {
    case Scales::k16: experts_wide_kernel<GLU, Scales::k16><<<(int)nwg, kEtThreads, 0, stream>>>(a); break;
    case Scales::k4: experts_wide_kernel<GLU, Scales::k4><<<(int)nwg, kEtThreads, 0, stream>>>(a); break;
    case Scales::kSkewed: experts_wide_kernel<GLU, Scales::kSkewed><<<(int)nwg, kEtThreads, 0, stream>>>(a); break;
  }
  return hipGetLastError();
}

template <bool GLU, int MR, int KB, int KG, bool SHARED>
static hipError_t launch_stream_t(const ExpertArgs& a, int nwg, hipStream_t stream) {
  constexpr int NT = KG * kEsThreads;
  switch (scales_of(a)) {
    case Scales::k16: experts_stream_kernel<GLU, MR, KB, KG, Scales::k16, SHARED><<<nwg, NT, 0, stream>>>(a); break;
    case Scales::k4: experts_stream_kernel<GLU, MR, KB, KG, Scales::k4, SHARED><<<nwg, NT, 0, stream>>>(a); break;
    case Scales::kSkewed:
      experts_stream_kernel<GLU, MR, KB, KG, Scales::kSkewed, SHARED><<<nwg, NT, 0, stream>>>(a);
      break;
  }
  return hipGetLastError();
}

template <bool GLU, int MR, int KB>
static hipError_t launch_stream(ExpertArgs a, hipStream_t stream) {
  a.col_tiles = (a.N + kEsRows * kEsWaves - 1) / (kEsRows * kEsWaves);
  a.max_tiles = (int)max_row_tiles(a.R, a.G, MR);
  const int64_t items = (int64_t)a.max_tiles * a.col_tiles;
  if (items >= (int64_t(1) << 31)) return hipErrorInvalidConfiguration;
  if constexpr (MR == 16) {
    // One workgroup per CU at most: two K groups (grouped_swiglu at T = 1:
    // 27.7 us against 31.5; grouped_combine's 448 workgroups of 8 steps:
    // 27.4 against 23.7).
    if (items <= kEsFewItems) return launch_stream_t<GLU, MR, 1024, 2, false>(a, (int)items, stream);
  } else {
    // A launch of small experts beside the large ones is mostly empty, and a
    // workgroup without work takes about a nanosecond (129 thousand of them
    // took 140 us at T = 8192): past kEsManyItems each takes several items.
    if (a.take == Take::kSmall && items > kEsManyItems)
      return launch_stream_t<GLU, MR, KB, 1, true>(a, kEsSharedGrid, stream);
  }
  return launch_stream_t<GLU, MR, KB, 1, false>(a, (int)items, stream);
}

// By the mean number of rows per expert, were every slot's expert held here.
// D = 7168, F = 2048, 256 experts, k = 8, grouped_swiglu:
//   up to 8: 16-row tiles (T = 64: 430 us; 32-row 478, 128-row tiles 650);
//   up to 16: 32-row tiles (T = 512: 860 us; 16-row 968, shared by size 882);
//   beyond: two launches share the experts by their sizes, which only the
//   device knows (T = 1024: 1035 us, 32-row tiles alone 1180; an
//   expert-parallel rank's experts have a fraction of the mean, and a layer's
//   popular experts several times its others' rows).
template <bool GLU>
static hipError_t launch_products(ExpertArgs a, hipStream_t stream) {
  const int64_t mean = a.R / a.G;
  a.take = Take::kAll;
  // Also more rows of few experts, while their 16-row tiles are few enough
  // for two K groups (T = 32, k = 2, two experts, D = 7168, F = 768: 22.0 us,
  // 32-row tiles 31.4; level at K of 512 and less).
  const int64_t stream_cols = (a.N + kEsRows * kEsWaves - 1) / (kEsRows * kEsWaves);
  if (mean <= 8 || max_row_tiles(a.R, a.G, 16) * stream_cols <= kEsFewItems)
    return launch_stream<GLU, 16, 512>(a, stream);
  if (mean <= 16) return launch_stream<GLU, 32, 256>(a, stream);
  a.tile_cols = (a.N + kEtCols - 1) / kEtCols;
  // No split by any sizes: no launch for it.
  if (max_row_tiles(a.R, a.G, 128) * a.tile_cols < kMinTileItems) return launch_stream<GLU, 32, 256>(a, stream);
  a.take = Take::kSmall;
  const hipError_t e = launch_stream<GLU, 32, 256>(a, stream);
  if (e != hipSuccess) return e;
  a.take = Take::kLarge;
  return launch_wide<GLU>(a, stream);
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

int check_swiglu(int64_t T, int64_t k, int64_t G, int64_t F, int64_t D) {
  return F < 16 || F % 16 != 0 ? ROUTER_EINVAL : check_sizes(T, k, G, 2 * F, D, T);
}

int check_combine(int64_t T, int64_t k, int64_t G, int64_t D, int64_t F) {
  return D < 16 || D % 16 != 0 ? ROUTER_EINVAL : check_sizes(T, k, G, D, F, 0);
}

size_t combine_scratch(int64_t T, int64_t k, int64_t N) { return (size_t)(T * k) * (size_t)N * sizeof(float); }

}  // namespace

extern "C" {

size_t grouped_workspace_bytes(int64_t T, int64_t k, int64_t G, int64_t D, int64_t F) {
  if (check_swiglu(T, k, G, F, D) != ROUTER_OK && check_combine(T, k, G, D, F) != ROUTER_OK) return 0;
  const size_t p = nvr::plan_scratch_bytes(T * k, G), c = combine_scratch(T, k, D);
  return nvr::kScratchOffset + (p > c ? p : c);
}

int grouped_swiglu(const uint8_t* x_codes, const uint8_t* x_scales, const float* gsa, const uint8_t* w_codes,
                   const uint8_t* w_scales, const float* gsw, const float* bias, const int32_t* offsets,
                   const int32_t* rows, int64_t T, int64_t k, int64_t G, int64_t F, int64_t D, void* out,
                   void* stream) {
  const int st = check_swiglu(T, k, G, F, D);
  if (st != ROUTER_OK) return st;
  if (!gsa || !w_codes || !w_scales || !gsw || !offsets) return ROUTER_EINVAL;
  if (T > 0 && (!x_codes || !x_scales || !rows || !out)) return ROUTER_EINVAL;
  if (!aligned(x_codes, 16) || !aligned(w_codes, 16) || !aligned(x_scales, 2) || !aligned(w_scales, 4) ||
      !aligned(gsa, 4) || !aligned(gsw, 4) || !aligned(bias, 4) || !aligned(offsets, 4) || !aligned(rows, 4) ||
      !aligned(out, 16))
    return ROUTER_EINVAL;
  if (T == 0) return ROUTER_OK;
  nvr::ExpertArgs a{};
  a.xc = x_codes; a.xs = x_scales; a.gsa = gsa;
  a.wc = w_codes; a.ws = w_scales; a.gsw = gsw;
  a.bias = bias; a.offsets = offsets; a.rows = rows; a.out = out;
  a.T = (int)T; a.k = (int)k; a.R = (int)(T * k); a.G = (int)G; a.N = (int)(2 * F); a.D = (int)D;
  return status_from(nvr::launch_products<true>(a, static_cast<hipStream_t>(stream)));
}

int grouped_combine(const uint8_t* h_codes, const uint8_t* h_scales, const float* gsh, const uint8_t* w_codes,
                    const uint8_t* w_scales, const float* gsw, const float* bias, const int32_t* offsets,
                    const int32_t* pos, const float* topk_w, const void* residual, int64_t T, int64_t k, int64_t G,
                    int64_t D, int64_t F, void* out, void* workspace, size_t workspace_bytes, void* stream) {
  const int st = check_combine(T, k, G, D, F);
  if (st != ROUTER_OK) return st;
  if (!gsh || !w_codes || !w_scales || !gsw || !offsets) return ROUTER_EINVAL;
  if (T > 0 && (!h_codes || !h_scales || !pos || !topk_w || !out || !workspace)) return ROUTER_EINVAL;
  if (!aligned(h_codes, 16) || !aligned(w_codes, 16) || !aligned(h_scales, 2) || !aligned(w_scales, 4) ||
      !aligned(gsh, 4) || !aligned(gsw, 4) || !aligned(bias, 4) || !aligned(offsets, 4) || !aligned(pos, 4) ||
      !aligned(topk_w, 4) || !aligned(residual, 16) || !aligned(out, 16) || !aligned(workspace, 256))
    return ROUTER_EINVAL;
  if (T == 0) return ROUTER_OK;
  if (workspace_bytes < nvr::kScratchOffset + combine_scratch(T, k, D)) return ROUTER_EINVAL;
  float* y = reinterpret_cast<float*>(static_cast<char*>(workspace) + nvr::kScratchOffset);
  const int64_t cwg = (T * (D / 8) + 255) / 256;
  if (cwg >= (int64_t(1) << 31)) return ROUTER_EUNSUPPORTED;
  const nvr::CombineArgs c{y, pos, topk_w, static_cast<const uint16_t*>(residual), static_cast<uint16_t*>(out),
                           (int)T, (int)k, (int)(T * k), (int)D};
  nvr::ExpertArgs a{};
  a.xc = h_codes; a.xs = h_scales; a.gsa = gsh;
  a.wc = w_codes; a.ws = w_scales; a.gsw = gsw;
  a.bias = bias; a.offsets = offsets; a.out = y;
  a.T = (int)T; a.k = (int)k; a.R = (int)(T * k); a.G = (int)G; a.N = (int)D; a.D = (int)F;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const hipError_t e = nvr::launch_products<false>(a, s);
  if (e != hipSuccess) return status_from(e);
  nvr::combine_kernel<<<(int)cwg, 256, 0, s>>>(c);
  return status_from(hipGetLastError());
}

}  // extern "C"
