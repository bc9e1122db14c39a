// A tile's part of a softmax over the columns (gfx950): what a wavefront does
// with its block of logits z[row, column] instead of storing them.
//
// In base 2, with y = z log2(e) / temperature, each row of a block gives
// (m, s) with m >= its largest y and s = sum 2^(y - m); joined over the blocks
// of a row they give log sum e^z. kWeights also keeps 2^(y - m) itself, as
// fp16 times 2^15: relative error 2^-11 down to 2^-28 of the row's largest,
// absolute 2^-39 of it below (bf16 would keep 2^-8 of each). y is rounded
// before m is taken off it, so that no difference is above 0 and equal logits
// give equal weights wherever they stand. m is the next whole number, so that a
// block's weights and sums are brought to another m by powers of two and are
// rounded this once. `ref` lets m start at what earlier columns have reached, so
// that few blocks have a scale of their own.
#pragma once

#include "mma_tile.hpp"

namespace nvr {

struct SoftmaxOut {
  float scale;            // log2(e) / temperature
  const float* ref;       // NULL or [T]: a lower bound of m
  float2* stats;          // [T, blocks] (m, s)
  int blocks;             // stride of stats
  int used;               // blocks that have room for (m, s)
  _Float16* e;            // [T, ld_e]
  int64_t ld_e;           // a multiple of 512
  const int32_t* tokens;  // [T, K]: columns that rows name; any other number is none
  int K;
  int n0;                 // the piece's first column
  float* named;           // [T, K]: their y
};

constexpr float kWeightOne = 32768.0f;  // a weight of 1 in fp16

// Between writes and reads of LDS that is the wavefront's own.
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

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

// Logits of the tokens that a block's rows name, from the block's own sums: the
// rows' losses (loss.hip) then hold them against a sum of which they are a part,
// and no probability comes out above 1, however large the logits are. Every
// wavefront looks through the tokens of its tile's rows for those in its columns
// (STREAM: 16 columns from col0 and the 16 that lie 32 after them, else 64) and
// stores their y; few have any.
//
// Which of 64 x 32 tokens, from p0 on, may be such: bit 31 - u for token p0 + 64 u
// + lane, by its column alone (places past the n-th read as token 0). The tile
// asks for the first of them before its loop, where the loads' latency is not
// felt (after it: T = 4096 0.6 % more).
constexpr int kNamedLoads = 32;
template <bool STREAM, int U>
__device__ __forceinline__ uint32_t named_bits(const int32_t* tokens, int n, uint32_t base, int p0) {
  const __amdgpu_buffer_rsrc_t rsrc = make_rsrc(tokens, (int64_t)n * 4);
  uint32_t c[U], hits = 0u;
  // (The last first where they are many: the compiler would take the loads that two of named_hits' cases begin with out of
  // both, and wait for them before the others.)
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int u = U == kNamedLoads ? U - 1 - i : i;
    c[u] = __builtin_amdgcn_raw_buffer_load_b32(rsrc, 4 * (p0 + (int)(threadIdx.x & 63)) + 256 * u, 0, 0);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) hits = hits + hits + ((c[u] & (STREAM ? ~47u : ~63u)) == base ? 1u : 0u);
  return hits << (32 - U);
}
template <bool STREAM>
__device__ __forceinline__ uint32_t named_hits(const SoftmaxOut& o, int row0, int nr, int col0, int p0) {
  const int n = nr * o.K;
  const int32_t* tokens = o.tokens + (int64_t)row0 * o.K;
  const uint32_t base = (uint32_t)(o.n0 + col0);  // none of the bits that its columns differ in
  uint32_t hits;
  if (n - p0 <= 128) hits = named_bits<STREAM, 2>(tokens, n, base, p0);
  else if (n - p0 <= 1024) hits = named_bits<STREAM, 16>(tokens, n, base, p0);
  else hits = named_bits<STREAM, kNamedLoads>(tokens, n, base, p0);
  asm volatile("" : "+v"(hits));  // here, not where it is used: that would hold the tokens until then
  return hits;
}

// `hits`: named_hits from 0 on. `stage` puts row tile i's y into the wavefront's
// LDS, [32 rows][columns].
template <int RT, bool STREAM, class Stage>
__device__ __forceinline__ void named_logits(const SoftmaxOut& o, int row0, int nr, int col0, int N, uint32_t hits,
                                             const float* lds, Stage stage) {
  const int n = nr * o.K;
  const int32_t* tokens = o.tokens + (int64_t)row0 * o.K;
  float* named = o.named + (int64_t)row0 * o.K;
  int staged = -1;
  for (int p0 = 0;;) {
    while (__ballot(hits != 0u)) {
      const int u = (int)__builtin_clz(hits | 1u), p = p0 + (int)(threadIdx.x & 63) + 64 * u;
      const bool in = hits != 0u && p < n;
      hits &= ~(0x80000000u >> u);
      const uint32_t col = in ? (uint32_t)(tokens[p] - o.n0 - col0) : 0u;
      const int row = in ? p / o.K : 0;
      const uint32_t at = STREAM ? 32 * row + ((col >> 5) << 4) + (col & 15u) : 64 * (row & 31) + col;
      static_for<0, RT>([&](auto ic) {
        constexpr int i = decltype(ic)::value;
        const bool here = in && (row >> 5) == i && col0 + (int)col < N;
        if (!__ballot(here)) return;
        if (staged != i) stage(ic);
        staged = i;
        if (here) named[p] = lds[at];
      });
    }
    p0 += 64 * kNamedLoads;
    if (p0 >= n) return;
    hits = named_hits<STREAM>(o, row0, nr, col0, p0);
  }
}

// Block of 32 places from the stream's accumulators: lane (r, q), value v of
// tile m: row r (+ 16 t), column col0 + 32 m + 4 q + v, so that a lane's eight
// columns are neighbours in e.
// `hits`: named_hits from 0 on; `lds`: 16 NT rows of 32 floats of the wavefront's own.
template <bool KEEP, int NT>
__device__ __forceinline__ void softmax_block16(const SoftmaxOut& o, const f32x4_t (&acc)[2][NT], float scale,
                                                int row0, int nr, int col0, int N, uint32_t hits, float* lds) {
#pragma clang fp contract(off)
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int place = (col0 & ~63) + 2 * (col0 & 63);
  const float sc = scale * o.scale;
  named_logits<1, true>(o, row0, nr, col0, N, hits, lds, [&](auto) {
    wave_lds_fence();
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int m = 0; m < 2; ++m)
        *reinterpret_cast<f32x4_t*>(lds + 32 * (16 * t + r) + 16 * m + 4 * q) = acc[m][t] * sc;
    wave_lds_fence();
  });
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int row = 16 * t + r;
    float y[8], m = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[i] = col0 + 32 * (i & 1) + 4 * q + (i >> 1) < N ? acc[i & 1][t][i >> 1] * sc : -__builtin_inff();
      m = fmaxf(m, y[i]);
    }
    m = ceilf(max_across32(max_across16(m)));
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
// `hits`: named_hits from 0 on; `lds`: 32 rows of 64 floats of the wavefront's own.
template <bool KEEP, int RT>
__device__ __forceinline__ void softmax_block32(const SoftmaxOut& o, const f32x16_t (&acc)[RT][2], float scale,
                                                int row0, int nr, int col0, int N, uint32_t hits, float* lds) {
#pragma clang fp contract(off)
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
  named_logits<RT, false>(o, row0, nr, col0, N, hits, lds, [&](auto ic) {
    constexpr int i = decltype(ic)::value;
    wave_lds_fence();
#pragma unroll
    for (int v = 0; v < 16; ++v)
#pragma unroll
      for (int m = 0; m < 2; ++m) lds[64 * (8 * (v >> 2) + 4 * h + (v & 3)) + 32 * m + r] = acc[i][m][v] * sc;
    wave_lds_fence();
  });
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
      m = ceilf(max_across16(m));
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
