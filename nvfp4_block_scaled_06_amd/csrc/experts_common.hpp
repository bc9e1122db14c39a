// Shared by the routed experts' kernels (gfx950): the search that gives a
// workgroup its tile of rows from the experts' device-side offsets.
//
// Rows are sorted by expert: expert g owns rows offsets[g] .. offsets[g + 1] -
// 1, and the rows from offsets[G] to R belong to no expert held here. A tile
// is up to tr consecutive rows of one expert; tiles are numbered expert by
// expert, the rows of no expert last. The host knows neither the sizes nor
// the number of tiles, only that there are at most
//   sum_g ceil(n_g / B) <= R / B + (experts with rows) <= R / B + min(R, G + 1)
// of them.
#pragma once

#include "mma_tile.hpp"

namespace nvr {

constexpr int kMaxGroups = 512;                   // ROUTER_MAX_EXPERTS
constexpr int kGroupsPerLane = kMaxGroups / 64;  // one wavefront scans every expert

// Inclusive prefix sum over the wavefront (row shifts, then row broadcasts).
__device__ __forceinline__ int wave_prefix_sum(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);  // row_shr 1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, kDppRowBcast15, 0xA, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, kDppRowBcast31, 0xC, 0xF, false);
  return v;
}

struct RowTile {
  int g;     // expert; G: rows of no expert
  int row0;  // first row
  int nr;    // rows
};

// Experts by size: those with more rows than kSmallExpert are large (limits
// of 32 and 64 rows: T = 2048 in 1400 and 1500 us) when there are enough of
// them for 128-row tiles, i.e. when `tile_cols` column tiles of their 128-row
// tiles give kMinTileItems work items (for 128 x 512 tiles of full rows the
// stream takes as long at about 90 of them, with 64 rows each at 100);
// otherwise every expert is small.
constexpr int kSmallExpert = 32;
constexpr int kMinTileItems = 128;
// Those tiles have 64 rows instead as long as every compute unit then has one
// of them at most (47 experts of 58 rows, K = 7168, 5 column tiles: swiglu 205
// us with 128 rows, 187 with 64, combine 217 and 200; 130 of 49 rows, K = 4096,
// 2 column tiles: swiglu 138 and 118).
constexpr int kOneRound = 256;
enum class Take { kAll, kSmall, kLarge };

// Every wavefront scans the offsets by itself: lane l holds `per` = G / 64
// (rounded up) adjacent experts. Offsets are clamped to [0, R] and a
// decreasing pair counts as no rows (a precondition violation then stays
// inside the caller's buffers).
struct TileScan {
  int off[kGroupsPerLane + 1];
  int before;   // tiles of the experts of lower lanes
  int experts;  // tiles of every expert taken
  int end;      // first row of no expert
  int G, R, sh, per, above, upto;  // tiles of 1 << sh rows

  __device__ __forceinline__ TileScan(const int32_t* offsets, int G_, int R_, int tr, Take take, int tile_cols)
      : G(G_), R(R_), sh(__builtin_ctz(tr)), per((G_ + 63) >> 6), above(0), upto(0x7FFFFFFF) {
    const int e0 = per * (int)(threadIdx.x & 63);
#pragma unroll
    for (int i = 0; i <= kGroupsPerLane; ++i)
      if (i <= per) off[i] = offsets[min(e0 + i, G)];
    end = min(max(offsets[G], 0), R);
#pragma unroll
    for (int i = 0; i <= kGroupsPerLane; ++i)
      if (i <= per) off[i] = min(max(off[i], 0), R);
    if (take != Take::kAll) {
      int big = 0, half = 0;
#pragma unroll
      for (int i = 0; i < kGroupsPerLane; ++i)
        if (i < per) {
          const int n = off[i + 1] - off[i];
          big += n > kSmallExpert ? (n + 127) >> 7 : 0;
          half += n > kSmallExpert ? (n + 63) >> 6 : 0;
        }
      big = __builtin_amdgcn_readlane(wave_prefix_sum(big), 63);
      if (take == Take::kLarge) {
        // Only counts up to kOneRound matter.
        half = __builtin_amdgcn_readlane(wave_prefix_sum(min(half, kOneRound + 1)), 63);
        if ((int64_t)half * tile_cols <= kOneRound) sh = 6;
      }
      const bool split = (int64_t)big * tile_cols >= kMinTileItems;
      if (take == Take::kSmall) upto = split ? kSmallExpert : upto;
      else above = split ? kSmallExpert : upto;
    }
    int mine = 0;
#pragma unroll
    for (int i = 0; i < kGroupsPerLane; ++i)
      if (i < per) mine += tiles(i);
    // Offsets that no plan gives may name R rows for every other expert: 2^31
    // tiles of R near 2^30. A plan's tiles are at most R / 128 + G where R is large.
    mine = min(mine, 1 << 24);
    const int incl = wave_prefix_sum(mine);
    before = incl - mine;
    experts = __builtin_amdgcn_readlane(incl, 63);
  }
  __device__ __forceinline__ int tiles(int i) const {
    const int n = off[i + 1] - off[i];
    return n > above && n <= upto ? (n + (1 << sh) - 1) >> sh : 0;
  }
  // Tiles of the rows of no expert, and the n-th of them.
  __device__ __forceinline__ int others() const { return (R - end + (1 << sh) - 1) >> sh; }
  __device__ __forceinline__ RowTile none(int n) const {
    const int row0 = end + (n << sh);
    return {G, row0, min(1 << sh, R - row0)};
  }

  // Work item n < experts * cols: an expert's row tiles times `cols` column
  // tiles, the row tiles of one column tile first, so that workgroups that
  // read the same weights run side by side.
  __device__ __forceinline__ RowTile at(int n, int cols, int& ct) const {
    const int q = n / cols;  // a tile of the same expert
    int g = 0, first = 0, rows = 0, base = 0, m = 0, c = before;
#pragma unroll
    for (int i = 0; i < kGroupsPerLane; ++i)
      if (i < per) {
        const int k = tiles(i);
        if (q >= c && q < c + k) {
          g = per * (int)(threadIdx.x & 63) + i;
          first = off[i];
          rows = off[i + 1] - off[i];
          base = c;
          m = k;
        }
        c += k;
      }
    const int lane = (int)__builtin_ctzll(__ballot(m > 0));  // one lane holds the expert
    g = __builtin_amdgcn_readlane(g, lane);
    first = __builtin_amdgcn_readlane(first, lane);
    rows = __builtin_amdgcn_readlane(rows, lane);
    base = __builtin_amdgcn_readlane(base, lane);
    m = __builtin_amdgcn_readlane(m, lane);
    const int i = n - base * cols;  // of m * cols
    ct = i / m;
    const int r0 = (i - ct * m) << sh;
    return {g, first + r0, min(1 << sh, rows - r0)};
  }
};

// Upper bound on the tiles of the experts and of the rows of no expert.
inline int64_t max_row_tiles(int64_t R, int64_t G, int tr) { return R / tr + (R < G + 1 ? R : G + 1); }

// Workgroup b's number among `total` when the 8 XCDs (workgroups go to them
// in turn) each take a contiguous range of numbers.
__device__ __forceinline__ int xcd_order(int b, int total) {
  const int x = b & 7;
  return x * (total >> 3) + min(x, total & 7) + (b >> 3);
}

__device__ __forceinline__ uint16_t bf16_round(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }

__device__ __forceinline__ uint32_t bf16_round2(float lo, float hi) {
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, bf16x2_t{(__bf16)lo, (__bf16)hi});
}

}  // namespace nvr
