// Shared by the routed experts' kernels (gfx950): the search that gives a
// workgroup its tile of rows from the experts' device-side offsets.
//
// Rows are sorted by expert: expert g owns rows offsets[g] .. offsets[g + 1] -
// 1, and the rows from offsets[G] to R belong to no expert held here. A tile
// is up to 2^sh consecutive rows of one expert; tiles are numbered expert by
// expert, the rows of no expert last. The host knows neither the sizes nor
// the number of tiles, only that there are at most
//   sum_g ceil(n_g / B) <= R / B + (experts with rows) <= R / B + min(R, G + 1)
// of them, so it launches that many and the others exit.
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
  int nr;    // rows (0: no such tile)
};

// Every wavefront scans the offsets by itself: lane l holds experts 8l ..
// 8l + 7. Offsets are clamped to [0, R] and a decreasing pair counts as no
// rows (a precondition violation then stays inside the caller's buffers).
struct TileScan {
  int off[kGroupsPerLane + 1];
  int before;  // tiles of the experts of lower lanes
  int experts, total;  // tiles of every expert; and of the rows of no expert too
  int G, R, sh;

  __device__ __forceinline__ TileScan(const int32_t* offsets, int G_, int R_, int sh_) : G(G_), R(R_), sh(sh_) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i <= kGroupsPerLane; ++i)
      off[i] = offsets[min(kGroupsPerLane * lane + i, G)];
#pragma unroll
    for (int i = 0; i <= kGroupsPerLane; ++i) off[i] = min(max(off[i], 0), R);
    int mine = 0;
#pragma unroll
    for (int i = 0; i < kGroupsPerLane; ++i) mine += tiles(i);
    const int upto = wave_prefix_sum(mine);
    before = upto - mine;
    experts = __builtin_amdgcn_readlane(upto, 63);
    total = experts + ((R - end() + (1 << sh) - 1) >> sh);
  }
  __device__ __forceinline__ int tiles(int i) const { return (max(off[i + 1] - off[i], 0) + (1 << sh) - 1) >> sh; }
  // First row of no expert.
  __device__ __forceinline__ int end() const { return __builtin_amdgcn_readlane(off[kGroupsPerLane], 63); }

  __device__ __forceinline__ RowTile at(int n) const {
    RowTile t;
    if (n >= experts) {
      t.g = G;
      t.row0 = end() + ((n - experts) << sh);
      t.nr = min(1 << sh, R - t.row0);
      return t;
    }
    int g = 0, row0 = 0, nr = 0, c = before;
#pragma unroll
    for (int i = 0; i < kGroupsPerLane; ++i) {
      const int m = tiles(i);
      if (n >= c && n < c + m) {
        g = kGroupsPerLane * (int)(threadIdx.x & 63) + i;
        row0 = off[i] + ((n - c) << sh);
        nr = min(1 << sh, off[i + 1] - row0);
      }
      c += m;
    }
    const int lane = (int)__builtin_ctzll(__ballot(nr > 0));  // one lane holds tile n
    t.g = __builtin_amdgcn_readlane(g, lane);
    t.row0 = __builtin_amdgcn_readlane(row0, lane);
    t.nr = __builtin_amdgcn_readlane(nr, lane);
    return t;
  }
};

// Upper bound on TileScan::total.
inline int64_t max_row_tiles(int64_t R, int64_t G, int sh) { return (R >> sh) + (R < G + 1 ? R : G + 1); }

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
