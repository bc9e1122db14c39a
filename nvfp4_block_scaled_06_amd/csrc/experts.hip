// The routed experts' products (gfx950) over rows sorted by expert:
//
//   grouped_swiglu:  y[p, n] = gsa gsw[e] sum_d (q_x S_x)[t(p), d] (q_w S_w)[e, n, d] + bias[e, n]
//                    h[p, f] = silu(y[p, f]) y[p, F + f]            (bf16)
//   grouped_combine: y[p, n] = gsh gsw[e] sum_f (q_h S_h)[p, f] (q_w S_w)[e, n, f] + bias[e, n]
//                    out[t, n] = residual[t, n] + sum_j w[t, j] y[pos[t, j], n]   (bf16)
//
// with e the expert of row p and t(p) = rows[p] / k its token.
#include "../../include/nvfp4_router.h"
#include "experts_tile.hpp"

#include <algorithm>

namespace nvr {

size_t plan_scratch_bytes(int64_t R, int64_t G);  // experts_plan.hip

// Work item b -> (row tile, column tile). The products of the experts' rows
// come first, numbered so that consecutive items (the row tiles of one column
// tile of an expert, then its next column tile) run on one XCD and share its
// L2; then, if `others` (grouped_swiglu), one item per row tile of no expert.
// False behind the last item, and for offsets that no plan gives and that ask
// for more tiles than R rows can.
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

constexpr int kEsSharedGrid = 256 * 6;  // workgroups that share a launch's items
constexpr int kEsManyItems = 12288;
constexpr int kEsFewItems = 256;

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
    else stream_tile<GLU ? Out::kGlu : Out::kProducts, MR, KB, KG, S>(a, tile, lds);
    if (!SHARED) return;
    __syncthreads();  // the next item writes the LDS tiles
  }
}

template <bool GLU, Scales S>
__global__ __launch_bounds__(kEtThreads) __attribute__((amdgpu_waves_per_eu(2, 2))) void experts_wide_kernel(
    ExpertArgs a) {
  __shared__ TileLds lds;
  const TileScan scan(a.offsets, a.G, a.R, kEtRows, a.take, a.tile_cols);
  ExpertTile tile;
  if (!expert_tile(a, scan, false, blockIdx.x, tile)) return;
  constexpr Out kOut = GLU ? Out::kGlu : Out::kProducts;
  const int nr = tile.rt.nr;
  if (nr > 96) wide_tile<kOut, 4, S>(a, tile, lds);
  else if (nr > 64) wide_tile<kOut, 3, S>(a, tile, lds);
  else if (nr > 32) wide_tile<kOut, 2, S>(a, tile, lds);
  else wide_tile<kOut, 1, S>(a, tile, lds);
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
