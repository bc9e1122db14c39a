// A tile's part of a softmax over the columns (gfx950): what a wavefront does
// with its block of logits z[row, column] instead of storing them.
//
// In base 2, with y = z log2(e) / temperature, each row of a block gives
// (m, s) with m >= its largest y and s = sum 2^(y - m); joined over the blocks
// of a row they give log sum e^z. kWeights also keeps 2^(y - m) itself, as
// fp16 times 2^15: relative error 2^-11 down to 2^-28 of the row's largest,
// absolute 2^-39 of it below (bf16 would keep 2^-8 of each). m is a whole
// number, the next one up, so that a block's weights and sums are brought to
// another m by powers of two and are rounded this once. `ref` lets m start at
// what earlier columns have reached, so that few blocks have a scale of their
// own.
#pragma once

#include "mma_tile.hpp"

namespace nvr {

struct SoftmaxOut {
  float scale;        // log2(e) / temperature
  const float* ref;   // NULL or [T]: a lower bound of m
  float2* stats;      // [T, blocks] (m, s)
  int blocks;         // stride of stats
  int used;           // blocks that have room for (m, s)
  _Float16* e;        // [T, ld_e]
  int64_t ld_e;       // a multiple of 512
};

constexpr float kWeightOne = 32768.0f;  // a weight of 1 in fp16

// Where the weight of column n stands in its row of e: in every 64 columns n
// and n + 32 are neighbours, as the conversion of the gradient's product takes
// the weights' rows (loss.hip). The blocks of a stream are 32 such places, 16
// columns and the 16 that lie 32 after them.
__device__ __forceinline__ int64_t weight_place(int64_t n) {
  return (n & ~int64_t(63)) | ((n & 31) << 1) | ((n >> 5) & 1);
}

// The larger / the sum of a value and its partner 16 or 32 lanes away.
__device__ __forceinline__ float max_across16(float v) {
  const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
}
__device__ __forceinline__ float sum_across16(float v) {
  const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}
__device__ __forceinline__ float max_across32(float v) {
  const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
}
__device__ __forceinline__ float sum_across32(float v) {
  const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}
template <int CTRL>
__device__ __forceinline__ float dpp_f(float v) {
  return __int_as_float(dpp_i<CTRL>(__float_as_int(v)));
}

// A whole number at least as large as the exact product that y is rounded from
// (by a half step, relative 2^-24), and less than 2 above it; -infinity for none.
__device__ __forceinline__ float whole_above(float y) {
  return y > -__builtin_inff() ? ceilf(fmaf(fabsf(y), 0x1p-22f, y)) : y;
}

// Block of 32 places from the stream's accumulators: lane (r, q), value v of
// tile m: row r (+ 16 t), column col0 + 32 m + 4 q + v, so that a lane's eight
// columns are neighbours in e.
template <bool KEEP, int NT>
__device__ __forceinline__ void softmax_block16(const SoftmaxOut& o, const f32x4_t (&acc)[2][NT], float scale,
                                                int row0, int nr, int col0, int N) {
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int place = (col0 & ~63) + 2 * (col0 & 63);
  const float sc = scale * o.scale;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int row = 16 * t + r;
    float y[8], m = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[i] = col0 + 32 * (i & 1) + 4 * q + (i >> 1) < N ? acc[i & 1][t][i >> 1] * sc : -__builtin_inff();
      m = fmaxf(m, y[i]);
    }
    m = whole_above(max_across32(max_across16(m)));
    // Columns past N have weights of zero and take no part in the sums.
    const bool none = col0 >= N;
    if (KEEP && o.ref && row < nr && !none) m = fmaxf(m, o.ref[row0 + row]);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[i] = none ? 0.0f : __builtin_amdgcn_exp2f(y[i] - m);
      s += y[i];
    }
    s = sum_across32(sum_across16(s));
    if (row >= nr) continue;
    if (q == 0 && (place >> 5) < o.used) o.stats[(int64_t)(row0 + row) * o.blocks + (place >> 5)] = make_float2(m, s);
    if constexpr (KEEP) {
      half8_t h;
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = (_Float16)(y[i] * kWeightOne);
      *reinterpret_cast<half8_t*>(o.e + (int64_t)(row0 + row) * o.ld_e + place + 8 * q) = h;
    }
  }
}

// Block of 64 columns from a wide tile's accumulators: lane (r, h), value v of
// row tile i: row 32 i + 8 (v / 4) + 4 h + v % 4, columns r and 32 + r.
template <bool KEEP, int RT>
__device__ __forceinline__ void softmax_block32(const SoftmaxOut& o, const f32x16_t (&acc)[RT][2], float scale,
                                                int row0, int nr, int col0, int N) {
  const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
  if (col0 >= N) {
    // As there: the gradient's product takes the tile's columns past N too.
    if constexpr (KEEP) {
      for (int row = h; row < nr; row += 2) {
        if (r == 0) o.stats[(int64_t)(row0 + row) * o.blocks + (col0 >> 6)] = make_float2(-__builtin_inff(), 0.0f);
        *reinterpret_cast<uint32_t*>(o.e + (int64_t)(row0 + row) * o.ld_e + col0 + 2 * r) = 0u;
      }
    }
    return;
  }
  const float sc = scale * o.scale;
  const bool in0 = col0 + r < N, in1 = col0 + 32 + r < N;
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const int row = 32 * i + 8 * (v >> 2) + 4 * h + (v & 3);
      const float y0 = in0 ? acc[i][0][v] * sc : -__builtin_inff(), y1 = in1 ? acc[i][1][v] * sc : -__builtin_inff();
      float m = fmaxf(y0, y1);
      m = fmaxf(m, dpp_f<kDppXor1>(m));
      m = fmaxf(m, dpp_f<kDppXor2>(m));
      m = fmaxf(m, dpp_f<kDppHalfMirror>(m));
      m = fmaxf(m, dpp_f<kDppMirror>(m));
      m = whole_above(max_across16(m));
      if (KEEP && o.ref && row < nr) m = fmaxf(m, o.ref[row0 + row]);
      const float e0 = __builtin_amdgcn_exp2f(y0 - m), e1 = __builtin_amdgcn_exp2f(y1 - m);
      float s = e0 + e1;
      s += dpp_f<kDppXor1>(s);
      s += dpp_f<kDppXor2>(s);
      s += dpp_f<kDppHalfMirror>(s);
      s += dpp_f<kDppMirror>(s);
      s = sum_across16(s);
      if (row >= nr) continue;
      if (r == 0) o.stats[(int64_t)(row0 + row) * o.blocks + (col0 >> 6)] = make_float2(m, s);
      if constexpr (KEEP) {
        *reinterpret_cast<half2_t*>(o.e + (int64_t)(row0 + row) * o.ld_e + col0 + 2 * r) =
            half2_t{(_Float16)(e0 * kWeightOne), (_Float16)(e1 * kWeightOne)};
      }
    }
}

}  // namespace nvr
