// Routing on given logits and its gradient (gfx950): the rules of choice that
// the gate's fused epilogue does not have.
//
// Per row: s = sigmoid(l) or softmax(l); key = s + bias; of `groups` groups of
// neighbouring experts the `kept` with the largest sums of their one or two
// best keys stay; the k largest keys among them in descending order; w = scale
// s / (1 or the sum of the chosen s).
//
// The order is that of keys computed in 64 bits, so it does not hang on how a
// logistic function rounds; keys that are equal there (saturated scores, say)
// go by their logits, then to the lower expert; groups of equal scores likewise
// where a score is one key, and to the lower group where it is a sum of two. Nearly every row is
// decided in 32 bits: without a bias that order is the logits' own; with
// one, keys computed in 32 bits are off by less than kKeyErr, and where two
// neighbours in the order, or the last group kept and the first one left out,
// are closer than that, the wavefront does its rows again in 64 bits (about
// one row of a thousand at 256 experts and k = 8).
//
// A row is one wavefront's, or 16 lanes' with four rows to a wavefront where
// rows are many. The choice takes no k rounds over all keys: a bound that k
// keys reach (the k-th largest of the lanes' maxima) leaves a few survivors,
// which are put together in LDS and ranked against each other. Rows where too
// many survive (equal logits, for example) take the rounds, as those that 32
// bits cannot decide do.
//
// Measured, k = 8: T = 1, 256 experts with a bias and four of eight groups 4.6
// us (the call 10, which the launch and the binding make); T = 32768, 384
// experts, softmax: 14.6 us, 3.6 TB/s of the 52 MB that it has to read and
// write, part instructions and part memory (as 12.2 for 256 experts); equal
// logits throughout, every row by the rounds: 256 experts 26. Gradient, 256
// experts: T = 8192 6.2 us, T = 32768 11.3, 3.2 TB/s with 34 MB of it stored.
#include "../../include/nvfp4_router.h"
#include <algorithm>

#include "experts_common.hpp"
#include "route16.hpp"

namespace nvr {

constexpr int kSelWaves = 4;
constexpr int kSelThreads = 64 * kSelWaves;
// How far apart two keys computed in 32 bits have to be for their order to
// hold, times the larger one where that is above 1. sigmoid_fast is off by
// s (1 - s) (|l| 2^-24 + 2^-23) for the exponential and s (2^-24 + 2^-23) for
// the sum and the reciprocal, 2.3e-7 at most, and the bias adds 2^-24: 6e-7
// for two keys. A softmax's sum over 512 experts (32 terms in a lane, then 4
// to 6 steps) may be off by 38 2^-24 = 2.3e-6 for all its keys alike, each
// exponential by 0.37 2^-23 + 2^-23 of one, the quotient by 2^-23: 3.1e-6.
constexpr float kKeyErrSigmoid = 1e-6f, kKeyErrSoftmax = 5e-6f;

struct SelectArgs {
  const void* logits;
  int64_t ld;
  const float* bias;
  int bf16, T, E, k;
  int groups, size, kept, top, sh;  // sh: log2 of the lanes per group
  uint32_t inv;                     // 2^20 / size rounded up: e / size = e inv >> 20 for e < 512
  int softmax, renorm, by_logit, vec, many;  // many: 16 lanes to a row
  float scale;
  int lds_row;  // bytes of LDS per row
  int32_t* idx;
  float* w;
};

__device__ __forceinline__ float exp_fast(float x) { return __builtin_amdgcn_exp2f(1.4426950408889634f * x); }

__device__ __forceinline__ float sel_logit(const void* p, int bf16, int64_t i) {
  const float l = bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16)
                       : static_cast<const float*>(p)[i];
  return l == l ? l : -__builtin_inff();  // NaN: masked
}

// The value of a score_key.
__device__ __forceinline__ float key_back(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

// Reductions over a row's lanes, in a fixed order.
template <int LPR>
__device__ __forceinline__ uint32_t row_min(uint32_t v) {
  if constexpr (LPR == 64) return wave_min_u32(v);
  else return ~group_max_u32<16>(~v);
}
template <int LPR, class F>
__device__ __forceinline__ F row_fmax(F v) {
  if constexpr (sizeof(F) == 4) {
    if constexpr (LPR == 64) return wave_max(v);
    v = fmaxf(v, __int_as_float(dpp_i<kDppXor1>(__float_as_int(v))));
    v = fmaxf(v, __int_as_float(dpp_i<kDppXor2>(__float_as_int(v))));
    v = fmaxf(v, __int_as_float(dpp_i<kDppHalfMirror>(__float_as_int(v))));
    return fmaxf(v, __int_as_float(dpp_i<kDppMirror>(__float_as_int(v))));
  } else {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) {
      const F u = __shfl_xor(v, o);
      v = u > v ? u : v;
    }
    return v;
  }
}
template <int LPR, class F>
__device__ __forceinline__ F row_total(F v) {
  if constexpr (sizeof(F) == 4) {
    return LPR == 64 ? wave_sum(v) : row_sum(v);
  } else {
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1) v += __shfl_xor(v, o);
    return v;
  }
}

__device__ __forceinline__ void sel_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Expert of a lane's j-th logit: neighbours 4 by 4 for 16-byte loads, or lane by lane.
template <int LPR, bool VEC>
__device__ __forceinline__ int sel_expert(int li, int j) {
  return VEC ? 4 * LPR * (j >> 2) + 4 * li + (j & 3) : LPR * j + li;
}

// Place of a 32-bit key in LDS: 4 words of padding after every 16, so that the
// lanes of a row, each on a run of its own, read different banks.
template <class F>
__device__ __forceinline__ int sel_place(int e) {
  return sizeof(F) == 4 ? e + ((e >> 4) << 2) : e;
}

// Groups that stay, from the row's keys in LDS: bit g << sh. `unsure`: the
// border is closer than the two scores' errors. A score's goes by the size of
// its keys, not by its own: keys of +b and -b leave a sum near 1 that is off by
// steps of b. (Half of err is more than one key's error, and what is left of
// it more than the sum's rounding; a softmax's error that all its keys share is
// in a sum of two no more than once, as two scores add up to 1 at most.)
// In 64 bits (F = double) equal scores of one key go by that expert's logit,
// which is looked up in the row from logit `base` on; in 32 bits they are
// unsure, or logits themselves.
template <int LPR, class F>
__device__ __forceinline__ uint64_t sel_groups(const SelectArgs& a, const F* vals, int64_t base, float err, bool& unsure) {
  constexpr bool WIDE = sizeof(F) == 8;
  const F ninf = -(F)__builtin_inff();
  const int lane = threadIdx.x & 63, li = lane & (LPR - 1), row = lane & ~(LPR - 1);
  const bool two = a.top == 2 && a.size > 1;
  const int g = li >> a.sh, lpg = 1 << a.sh, run = (a.size + lpg - 1) >> a.sh, sub = li & (lpg - 1);
  F b1 = ninf, b2 = ninf;
  int e1 = 0;                          // WIDE: the expert of b1
  float l1 = -__builtin_inff();  // and its logit
  if (g < a.groups) {
    const int end = min((sub + 1) * run, a.size);
    if (WIDE && !two) {
      for (int i = sub * run; i < end; ++i) {
        const int e = g * a.size + i;
        const F x = vals[sel_place<F>(e)];
        if (x > b1 || (x == b1 && x > ninf && sel_logit(a.logits, a.bf16, base + e) > sel_logit(a.logits, a.bf16, base + e1))) {
          b1 = x;
          e1 = e;
        }
      }
      if (b1 > ninf) l1 = sel_logit(a.logits, a.bf16, base + e1);
    } else {
#pragma unroll 8
      for (int i = sub * run; i < end; ++i) {
        const F x = vals[sel_place<F>(g * a.size + i)];
        const F lo = x < b1 ? x : b1;
        b2 = lo > b2 ? lo : b2;
        b1 = x > b1 ? x : b1;
      }
    }
  }
  for (int o = 1; o < lpg; o <<= 1) {
    const F o1 = __shfl_xor(b1, o), o2 = __shfl_xor(b2, o);
    if (WIDE && !two) {
      const float ol = __shfl_xor(l1, o);
      l1 = o1 > b1 || (o1 == b1 && ol > l1) ? ol : l1;
    }
    const F lo = o1 < b1 ? o1 : b1, hi2 = o2 > b2 ? o2 : b2;
    b2 = lo > hi2 ? lo : hi2;
    b1 = o1 > b1 ? o1 : b1;
  }
  F score = two ? b1 + b2 : b1;
  if (!(score == score) || g >= a.groups) score = ninf;
  int rank = 0;
  for (int j = 0; j < a.groups; ++j) {
    const F s = __shfl(score, row + (j << a.sh));
    bool before = j < g;
    if (WIDE && !two) {
      const float l = __shfl(l1, row + (j << a.sh));
      before = l > l1 || (l == l1 && before);
    }
    rank += s > score || (s == score && before) ? 1 : 0;
  }
  const bool keep = g < a.groups && rank < a.kept;
  if (err > 0.0f) {
    const float m1 = fmaxf(1.0f, fabsf((float)b1)), m2 = fmaxf(1.0f, fabsf((float)b2));
    float slack = err * (two ? 0.5f * (m1 + m2) : m1);
    if (!(slack < __builtin_inff())) slack = 0.0f;  // infinite keys are exact
    const F lowest = -row_fmax<LPR, F>(keep ? (F)slack - score : ninf);
    const F next = row_fmax<LPR, F>(!keep && g < a.groups ? score + (F)slack : ninf);
    if (lowest > ninf && lowest <= next) unsure = true;
    if (b2 > ninf && b1 < -ninf && !(score > ninf && score < -ninf)) unsure = true;  // a sum beyond 32 bits
  }
  return __ballot(keep) >> row;
}

__device__ __forceinline__ bool sel_kept(const SelectArgs& a, uint64_t kept, uint32_t e) {
  const uint32_t g = min((e * a.inv) >> 20, (uint32_t)a.groups - 1u);
  return (kept >> (g << a.sh)) & 1ull;
}

// The choice by k rounds over the row's keys in LDS, which it uses up. Equal keys
// in 64 bits go by the logits of the row, which start at `base`.
template <int LPR, class F>
__device__ __forceinline__ void sel_rounds(const SelectArgs& a, F* vals, int64_t base, int& chosen) {
  const F ninf = -(F)__builtin_inff();
  const int li = threadIdx.x & (LPR - 1);
  chosen = -1;
  for (int r = 0; r < a.k; ++r) {
    F m = ninf;
    uint32_t e = 0xFFFFFFFFu;
#pragma unroll 4
    for (int i = li; i < a.E; i += LPR) {
      const F v = vals[sel_place<F>(i)];
      bool first = v > m;
      if constexpr (sizeof(F) == 8)
        first = first || (v == m && v > ninf && sel_logit(a.logits, a.bf16, base + i) > sel_logit(a.logits, a.bf16, base + e));
      if (first) {
        m = v;
        e = (uint32_t)i;
      }
    }
    const F best = row_fmax<LPR, F>(m);
    bool mine = m == best && best > ninf;
    if constexpr (sizeof(F) == 8) {
      const float l = mine ? sel_logit(a.logits, a.bf16, base + e) : -__builtin_inff();
      const float top = row_fmax<LPR, float>(l);
      mine = mine && l == top;
    }
    const uint32_t at = row_min<LPR>(mine ? e : 0xFFFFFFFFu);
    if (at == e && at != 0xFFFFFFFFu) vals[sel_place<F>((int)at)] = ninf;
    if (li == r) chosen = (int)at;
    sel_fence();
  }
}

// The larger of a value and its partner 32 or 16 lanes away.
__device__ __forceinline__ uint32_t max_turn32(uint32_t v) {
  const auto p = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max((uint32_t)p[0], (uint32_t)p[1]);
}
__device__ __forceinline__ uint32_t max_turn16(uint32_t v) {
  const auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  return max((uint32_t)p[0], (uint32_t)p[1]);
}

// Survivors that a row may have: two for each of 16 lanes, one for each of 64.
template <int LPR>
constexpr int sel_most() {
  return LPR == 16 ? 32 : 64;
}
template <int LPR>
struct SelScratch {
  uint64_t cand[sel_most<LPR>() + 1];  // key << 32 | ~expert; the last one takes what does not survive
  uint32_t key[sel_most<LPR>()];       // in order; if 32 bits do not decide, the logits of cand
  int expert[sel_most<LPR>()];
  double wide[sel_most<LPR>()];  // the survivors' keys in 64 bits, if 32 do not decide
};
enum : int { kSelDecided = 0, kSelOrder = 1, kSelAll = 2 };  // what 64 bits have to look at: nothing, the survivors, all keys

// Expert e's key in 64 bits; `top` and `total` of the row's softmax.
__device__ __forceinline__ double sel_wide(const SelectArgs& a, float logit, int e, double top, double total) {
  const double x = (double)logit, b = a.bias ? (double)a.bias[e] : 0.0;
  double d = exp(a.softmax ? x - top : -x);
  d = (a.softmax ? d / total : 1.0 / (1.0 + d)) + b;
  return x > -(double)__builtin_inff() && d > -(double)__builtin_inff() ? d : -(double)__builtin_inff();
}

// The choice in 32 bits; lane j < k of the row gets the j-th expert, -1 where
// none is left.
template <int LPR, int PER, bool VEC>
__device__ __forceinline__ int sel_survivors(const SelectArgs& a, const float (&v)[PER], char* row_lds, float err,
                                             int& count, int& chosen) {
  constexpr int MOST = sel_most<LPR>(), H = MOST / LPR;
  SelScratch<LPR>& sc = *reinterpret_cast<SelScratch<LPR>*>(row_lds);
  const int li = threadIdx.x & (LPR - 1);
  uint32_t key[PER], lm = 0u;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    key[j] = v[j] > -__builtin_inff() ? score_key(v[j]) : 0u;
    lm = max(lm, key[j]);
  }
  // A bound that at least k keys reach.
  uint32_t tau;
  if constexpr (LPR == 16) {
    const int above = count_above<1>(lm, 0);
    tau = row_min_u32(above < a.k ? lm : 0xFFFFFFFFu);
  } else {
    // Of the largest keys of the lanes l, l + S, l + 2 S, ..., S >= k, the
    // smallest. (Lanes in turn rather than neighbours: groups of experts left
    // out take whole runs of lanes with them.)
    uint32_t m = max_turn32(lm);
    if (a.k <= 16) m = max_turn16(m);
    if (a.k <= 8) m = max(m, dpp_u<0x128>(m));  // row_ror:8
    if (a.k <= 4) m = max(m, dpp_u<0x124>(m));  // row_ror:4
    tau = wave_min_u32(m);
  }
  if (err > 0.0f && tau != 0u) {  // and all that may be the k-th
    const float t = key_back(tau);
    if (t < __builtin_inff()) tau = score_key(t - err * fmaxf(1.0f, fabsf(t)));  // (infinite: of a bias, exact)
  }
  tau = max(tau, 1u);
  int C = 0;
  if constexpr (LPR == 16) {
    int cnt = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) cnt += key[j] >= tau ? 1 : 0;
    int pos = row_scan(cnt) - cnt;
    C = row_sum_i(cnt);
    if (__ballot(C > MOST)) return kSelAll;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const bool in = key[j] >= tau;
      sc.cand[in ? pos : MOST] = ((uint64_t)key[j] << 32) | ~(uint32_t)sel_expert<LPR, VEC>(li, j);
      pos += in ? 1 : 0;
    }
  } else {
    int n[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const uint64_t bal = __ballot(key[j] >= tau);
      n[j] = C + (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(bal >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)bal, 0u));
      C += (int)__popcll(bal);
    }
    if (C > MOST) return kSelAll;
#pragma unroll
    for (int j = 0; j < PER; ++j)
      sc.cand[key[j] >= tau ? n[j] : MOST] =
          ((uint64_t)key[j] << 32) | ~(uint32_t)sel_expert<LPR, VEC>(li, j);
  }
  // Entries past the count rank below all others.
#pragma unroll
  for (int h = 0; h < H; ++h)
    if (li + LPR * h >= C) sc.cand[li + LPR * h] = 0ull;
  sel_fence();
  uint64_t mine[H];
  int rank[H];
#pragma unroll
  for (int h = 0; h < H; ++h) {
    mine[h] = sc.cand[li + LPR * h];
    rank[h] = 0;
  }
#pragma unroll
  for (int u0 = 0; u0 < MOST; u0 += 16) {
    if (u0 && !__ballot(C > u0)) break;
#pragma unroll
    for (int u = u0; u < u0 + 16; ++u) {
      const uint64_t other = sc.cand[u];
#pragma unroll
      for (int h = 0; h < H; ++h) rank[h] += other > mine[h] ? 1 : 0;
    }
  }
#pragma unroll
  for (int h = 0; h < H; ++h) {
    if (li + LPR * h < C) {
      sc.key[rank[h]] = (uint32_t)(mine[h] >> 32);
      sc.expert[rank[h]] = (int)~(uint32_t)mine[h];
    }
  }
  sel_fence();
  chosen = li < a.k && li < C ? sc.expert[li] : -1;
  count = C;
  if (err > 0.0f && li < a.k && li + 1 < C) {
    const float p = key_back(sc.key[li]);
    if (!(p - key_back(sc.key[li + 1]) > err * fmaxf(1.0f, fabsf(p)))) return kSelOrder;  // (two infinite ones too)
  }
  return kSelDecided;
}

// The survivors in the order of their 64-bit keys, equal ones by their logits.
// The bound left out nothing that may be among the k largest.
template <int LPR>
__device__ __forceinline__ void sel_order(const SelectArgs& a, int64_t base, double top, double total, char* row_lds,
                                          int C, int& chosen) {
  constexpr int MOST = sel_most<LPR>(), H = MOST / LPR;
  SelScratch<LPR>& sc = *reinterpret_cast<SelScratch<LPR>*>(row_lds);
  const int li = threadIdx.x & (LPR - 1);
  double mine[H];
  float x[H];
  int e[H], rank[H];
#pragma unroll
  for (int h = 0; h < H; ++h) {
    e[h] = li + LPR * h < C ? (int)~(uint32_t)sc.cand[li + LPR * h] : 0;
    x[h] = sel_logit(a.logits, a.bf16, base + e[h]);
  }
#pragma unroll
  for (int h = 0; h < H; ++h) {
    mine[h] = sel_wide(a, x[h], e[h], top, total);
    rank[h] = 0;
    sc.wide[li + LPR * h] = li + LPR * h < C ? mine[h] : -(double)__builtin_inff();
    sc.key[li + LPR * h] = __float_as_uint(x[h]);
  }
  sel_fence();
  int same[H] = {};  // keys equal to the lane's, its own among them
  for (int u0 = 0; u0 < C; u0 += 8) {
#pragma unroll
    for (int u = u0; u < u0 + 8; ++u) {
      const double other = sc.wide[u];
#pragma unroll
      for (int h = 0; h < H; ++h) {
        rank[h] += other > mine[h] ? 1 : 0;
        same[h] += other == mine[h] ? 1 : 0;
      }
    }
  }
  bool tie = false;
#pragma unroll
  for (int h = 0; h < H; ++h) tie = tie || (li + LPR * h < C && same[h] > 1);
  if (__ballot(tie)) {
    for (int u = 0; u < C; ++u) {
      const double other = sc.wide[u];
      const int at = (int)~(uint32_t)sc.cand[u];
      const float l = __uint_as_float(sc.key[u]);
#pragma unroll
      for (int h = 0; h < H; ++h) rank[h] += other == mine[h] && (l > x[h] || (l == x[h] && at < e[h])) ? 1 : 0;
    }
  }
#pragma unroll
  for (int h = 0; h < H; ++h)
    if (li + LPR * h < C) sc.expert[rank[h]] = e[h];
  sel_fence();
  chosen = li < a.k && li < C ? sc.expert[li] : -1;
}

// The choice of the wavefront's rows, this lane's row starting at logit `base`;
// bias in `bv`.
template <int LPR, int PER, bool VEC>
__device__ __forceinline__ void sel_choose(const SelectArgs& a, const float (&l)[PER], const float (&bv)[PER], float top,
                                           float sum, int64_t base, bool live, char* row_lds, int& chosen) {
  const float ninf = -__builtin_inff();
  const int li = threadIdx.x & (LPR - 1);
  const float err = a.by_logit ? 0.0f : a.softmax ? kKeyErrSoftmax : kKeyErrSigmoid;
  const bool grouped = a.kept < a.groups;
  float v[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) v[j] = l[j];
  if (!a.by_logit) {
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      v[j] = (a.softmax ? exp_fast(l[j] - top) / sum : sigmoid_fast(l[j])) + bv[j];
      if (!(l[j] > ninf) || !(v[j] > ninf)) v[j] = ninf;  // and those past E, whose logits are -inf
    }
  }
  float* vals = reinterpret_cast<float*>(row_lds);
  double* wide = reinterpret_cast<double*>(row_lds);
  double total = 0.0;  // of the row's softmax, in 64 bits
  // All keys in 64 bits into `wide`. The logits pass through the upper half of
  // the same LDS: key i overwrites the logits 2 i - PER LPR and the next, which
  // this or an earlier turn of the loop has read. Four keys of a lane at a time,
  // for their latency.
  auto widen = [&]() {
    constexpr int ALL = PER * LPR;
    sel_fence();
#pragma unroll
    for (int j = 0; j < PER; ++j) vals[ALL + sel_expert<LPR, VEC>(li, j)] = l[j];
    sel_fence();
    if (a.softmax && total == 0.0) {
#pragma unroll 4
      for (int i = li; i < a.E; i += LPR) total += exp((double)vals[ALL + i] - (double)top);
      total = row_total<LPR>(total);
    }
    constexpr int U = PER < 4 ? PER : 4;
    for (int i0 = li; i0 < ALL; i0 += U * LPR) {
      double d[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        d[u] = sel_wide(a, vals[ALL + i0 + u * LPR], min(i0 + u * LPR, a.E - 1), (double)top, total);
      sel_fence();
#pragma unroll
      for (int u = 0; u < U; ++u) wide[i0 + u * LPR] = d[u];
      sel_fence();
    }
  };
  uint64_t kept = ~0ull;
  if (grouped) {
    bool border = false;
#pragma unroll
    for (int j = 0; j < PER; ++j) vals[sel_place<float>(sel_expert<LPR, VEC>(li, j))] = v[j];
    sel_fence();
    kept = sel_groups<LPR, float>(a, vals, base, err, border);
    if (__ballot(border && live)) {
      widen();
      kept = sel_groups<LPR, double>(a, wide, base, 0.0f, border);
    }
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (!sel_kept(a, kept, sel_expert<LPR, VEC>(li, j))) v[j] = ninf;
    sel_fence();
  }
  int C = 0;
  const int state = sel_survivors<LPR, PER, VEC>(a, v, row_lds, err, C, chosen);
  const bool all = __ballot(live && state == kSelAll) != 0;
  if (!all && !__ballot(live && state == kSelOrder)) return;
  if (a.by_logit) {  // exact as it is: too many survivors
    sel_fence();
#pragma unroll
    for (int j = 0; j < PER; ++j) vals[sel_place<float>(sel_expert<LPR, VEC>(li, j))] = v[j];
    sel_fence();
    sel_rounds<LPR, float>(a, vals, base, chosen);
    return;
  }
  if (!all) {
    sel_fence();
    if (a.softmax && total == 0.0) {
#pragma unroll 2
      for (int i = li; i < a.E; i += LPR) total += exp((double)sel_logit(a.logits, a.bf16, base + i) - (double)top);
      total = row_total<LPR>(total);
    }
    sel_order<LPR>(a, base, (double)top, total, row_lds, C, chosen);
    return;
  }
  widen();
  if (grouped) {
    for (int i = li; i < a.E; i += LPR)
      if (!sel_kept(a, kept, (uint32_t)i)) wide[i] = -(double)__builtin_inff();
    sel_fence();
  }
  sel_rounds<LPR, double>(a, wide, base, chosen);
}

// s of a logit, up to a factor common to the row that makes the largest of the
// chosen ones exp(0) or nearly: the quotient s / sum s then holds for any
// finite logits (all of them -1e30, for example). `m` is 0 for s itself.
__device__ __forceinline__ float sel_score(float l, float m, bool softmax) {
  return softmax ? expf(l - m) : expf(fminf(l, 0.0f) - m) / (1.0f + expf(-fabsf(l)));
}

template <int LPR, int PER, bool VEC>
__global__ __launch_bounds__(kSelThreads) void select_kernel(SelectArgs a) {
  extern __shared__ __attribute__((aligned(16))) char sel_lds[];
  constexpr int ROWS = 64 / LPR;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, li = lane & (LPR - 1);
  const int in_wg = wave * ROWS + lane / LPR;
  const int64_t row = (int64_t)blockIdx.x * (kSelWaves * ROWS) + in_wg;
  const bool live = row < a.T;
  if (!__ballot(live)) return;
  const int64_t base = (live ? row : a.T - 1) * a.ld;
  char* row_lds = sel_lds + in_wg * a.lds_row;
  const float ninf = -__builtin_inff();
  float l[PER];
  if constexpr (VEC) {
    typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int q = 0; q < PER / 4; ++q) {
      const int e = sel_expert<LPR, VEC>(li, 4 * q);
      if (e + 4 <= a.E) {
        if (a.bf16) {
          const u32x2_t u = *reinterpret_cast<const u32x2_t*>(static_cast<const uint16_t*>(a.logits) + base + e);
#pragma unroll
          for (int i = 0; i < 4; ++i) l[4 * q + i] = i & 1 ? bf16_hi(u[i >> 1]) : bf16_lo(u[i >> 1]);
        } else {
          const f32x4_t u = *reinterpret_cast<const f32x4_t*>(static_cast<const float*>(a.logits) + base + e);
#pragma unroll
          for (int i = 0; i < 4; ++i) l[4 * q + i] = u[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) l[4 * q + i] = e + i < a.E ? sel_logit(a.logits, a.bf16, base + e + i) : ninf;
      }
    }
#pragma unroll
    for (int j = 0; j < PER; ++j) l[j] = l[j] == l[j] ? l[j] : ninf;
  } else {
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int e = LPR * j + li;
      l[j] = sel_logit(a.logits, a.bf16, base + min(e, a.E - 1));
      if (e >= a.E) l[j] = ninf;
    }
  }
  float bv[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) bv[j] = a.bias ? a.bias[min(sel_expert<LPR, VEC>(li, j), a.E - 1)] : 0.0f;
  float top = 0.0f, sum = 1.0f;  // softmax over the whole row, where that is needed
  if (a.softmax && !(a.by_logit && a.renorm)) {
    top = l[0];
#pragma unroll
    for (int j = 1; j < PER; ++j) top = fmaxf(top, l[j]);
    top = row_fmax<LPR, float>(top);
    sum = 0.0f;
#pragma unroll
    for (int j = 0; j < PER; ++j) sum += exp_fast(l[j] - top);
    sum = row_total<LPR>(sum);
  }
  int chosen;
  sel_choose<LPR, PER, VEC>(a, l, bv, top, sum, base, live, row_lds, chosen);
  const bool mine = chosen >= 0;
  const float cl = mine ? sel_logit(a.logits, a.bf16, base + chosen) : ninf;
  float m = a.softmax ? top : 0.0f;
  if (a.renorm) m = row_fmax<LPR, float>(a.softmax ? cl : fminf(cl, 0.0f));
  const float s = mine ? sel_score(cl, m, a.softmax) : 0.0f;
  float total = sum;  // 1 for plain sigmoid scores
  if (a.renorm) total = row_total<LPR>(s);
  if (live && li < a.k) {
    a.idx[row * a.k + li] = chosen;
    a.w[row * a.k + li] = mine ? a.scale * (s / total) : 0.0f;
  }
}

struct SelectGradArgs {
  const void* logits;
  int64_t ld;
  const int32_t* idx;
  const float* gw;
  int bf16, T, E, k;
  int softmax, renorm;
  float scale;
  int lds_row;
  void* out;
  int64_t ld_out;
};

// The gradient of the logits. Renormalised: with u = s / sum s over the chosen
// and r_j = scale u_j (gw_j - sum_i u_i gw_i), dl = r for softmax and r
// sigmoid(-l) for sigmoid: nothing but the chosen logits is read. Plain
// sigmoid: scale gw s sigmoid(-l). Plain softmax reaches every expert: dl_n =
// scale s_n (gw_n - sum_i s_i gw_i), gw_n = 0 where n was not chosen. A row is
// put together in LDS and stored densely; an expert named twice gets the sum
// in the order of its places.
template <int LPR, int PER>
__global__ __launch_bounds__(kSelThreads) void select_grad_kernel(SelectGradArgs a) {
  extern __shared__ __attribute__((aligned(16))) char sel_lds[];
  constexpr int ROWS = 64 / LPR;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, li = lane & (LPR - 1);
  const int in_wg = wave * ROWS + lane / LPR;
  const int64_t row = (int64_t)blockIdx.x * (kSelWaves * ROWS) + in_wg;
  const bool live = row < a.T;
  const int64_t base = (live ? row : a.T - 1) * a.ld, place = (live ? row : a.T - 1) * a.k;
  float* d = reinterpret_cast<float*>(sel_lds + in_wg * a.lds_row);
  const bool dense = a.softmax && !a.renorm;
  int e = -1;
  float gw = 0.0f, cl = -__builtin_inff();
  if (li < a.k) {
    e = a.idx[place + li];
    gw = a.gw[place + li];
    if (e < 0 || e >= a.E) e = -1;
    if (e >= 0) cl = sel_logit(a.logits, a.bf16, base + e);
  }
  if (e < 0) gw = 0.0f;  // whatever stands there
  float l[PER], top = 0.0f, sum = 1.0f;
  if (dense) {
    top = -__builtin_inff();
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int n = LPR * j + li;
      l[j] = sel_logit(a.logits, a.bf16, base + min(n, a.E - 1));
      if (n >= a.E) l[j] = -__builtin_inff();
      top = fmaxf(top, l[j]);
    }
    top = row_fmax<LPR, float>(top);
    if (!(top > -__builtin_inff())) top = 0.0f;  // nothing but masked logits: zeros
    sum = 0.0f;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      l[j] = exp_fast(l[j] - top);
      sum += l[j];
    }
    sum = row_total<LPR>(sum);
    if (!(sum > 0.0f) && sum == sum) sum = 1.0f;
  }
  float m = a.softmax ? top : 0.0f;
  if (a.renorm) {
    m = row_fmax<LPR, float>(a.softmax ? cl : fminf(cl, 0.0f));
    if (!(m > -__builtin_inff())) m = 0.0f;
  }
  const float s = e >= 0 ? sel_score(cl, m, a.softmax) : 0.0f;
  float total = sum;
  if (a.renorm) total = row_total<LPR>(s);
  const float u = s > 0.0f || s != s ? s / total : 0.0f;
  float dot = 0.0f;
  if (a.softmax || a.renorm) dot = row_total<LPR>(u * gw);
  float mine = a.scale * u * (dense ? gw : a.renorm ? gw - dot : gw);
  if (!a.softmax) mine *= e >= 0 ? sel_score(-cl, 0.0f, false) : 0.0f;

#pragma unroll
  for (int j = 0; j < PER; ++j) d[LPR * j + li] = dense ? -a.scale * dot * (l[j] / sum) : 0.0f;
  sel_fence();
  // Sums of the places that name the same expert; the first of them adds.
  float all = 0.0f;
  bool first = e >= 0;
  for (int j = 0; j < a.k; ++j) {
    const int ej = __shfl(e, (lane & ~(LPR - 1)) + j);
    const float mj = __shfl(mine, (lane & ~(LPR - 1)) + j);
    if (ej == e) {
      all += mj;
      if (j < li) first = false;
    }
  }
  if (first) d[e] += all;
  sel_fence();
  if (!live) return;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int n = LPR * j + li;
    if (n >= a.E) continue;
    if (a.bf16) static_cast<uint16_t*>(a.out)[row * a.ld_out + n] = bf16_round(d[n]);
    else static_cast<float*>(a.out)[row * a.ld_out + n] = d[n];
  }
}

// Rows from which 16 lanes take a row, where its places and groups fit into 16
// lanes (us with 16 and 64 lanes, k = 8, 256 experts): by the logits alone
//   T = 1024 5.2, 4.4; 2048 5.3, 4.7 (384 experts: 5.9, 6.9); 4096 5.4, 6.9;
//   32768 12.2, 21.0;
// with keys, which put more on a lane,
//   T = 1024 8.5, 4.8; 2048 8.4, 5.3; 4096 8.6, 6.1; 6000 11.0, 10.3 (384
//   experts: 11.9, 13.4); 8192 10.0, 9.5 (four of eight groups: 11.3, 16.6);
//   32768 18.7, 27.2;
// the gradient
//   T = 1024 4.7, 3.9; 4096 5.2, 4.9; 8192 5.8, 6.7; 32768 11.3, 17.3.
// Measured at 256 and 384 experts; fewer and more have the same limits.
constexpr int64_t kSelManyLogits = 2048, kSelManyKeys = 6144, kSelManyGrads = 8192;
static bool select_many(int64_t T, int64_t from, int64_t k, int64_t groups) {
  return T >= from && k <= 16 && groups <= 16;
}

template <int LPR, int PER, bool VEC>
static hipError_t launch_select_t(SelectArgs a, hipStream_t stream) {
  constexpr int ROWS = kSelWaves * (64 / LPR);
  a.lds_row = std::max(PER * LPR * (a.by_logit ? 5 : 8), (int)(sizeof(SelScratch<LPR>) + 15) / 16 * 16);
  const int grid = (int)((a.T + (int64_t)ROWS - 1) / ROWS);
  select_kernel<LPR, PER, VEC><<<grid, kSelThreads, (size_t)ROWS * a.lds_row, stream>>>(a);
  return hipGetLastError();
}

// 16-byte loads where they give each of 16 lanes some experts of every group; a
// wavefront's loads of neighbours are whole lines anyway. (With groups of 32 a
// lane's 4 neighbours are of one group in two, and if the other ones are left
// out the bound rests on half the lanes: 8192 x 256, 4 of 8 groups, 18.5 us
// with them, 11.1 without.)
static hipError_t launch_select(SelectArgs a, hipStream_t stream) {
  a.vec = a.vec && a.kept == a.groups;
  if (a.many) {
    if (a.E <= 64) return launch_select_t<16, 4, false>(a, stream);
    if (a.E <= 128) return a.vec ? launch_select_t<16, 8, true>(a, stream) : launch_select_t<16, 8, false>(a, stream);
    if (a.E <= 256) return a.vec ? launch_select_t<16, 16, true>(a, stream) : launch_select_t<16, 16, false>(a, stream);
    if (a.E <= 384) return a.vec ? launch_select_t<16, 24, true>(a, stream) : launch_select_t<16, 24, false>(a, stream);
    return a.vec ? launch_select_t<16, 32, true>(a, stream) : launch_select_t<16, 32, false>(a, stream);
  }
  if (a.E <= 64) return launch_select_t<64, 1, false>(a, stream);
  if (a.E <= 128) return launch_select_t<64, 2, false>(a, stream);
  if (a.E <= 256) return launch_select_t<64, 4, false>(a, stream);
  return launch_select_t<64, 8, false>(a, stream);
}

template <int LPR, int PER>
static hipError_t launch_select_grad_t(SelectGradArgs a, hipStream_t stream) {
  constexpr int ROWS = kSelWaves * (64 / LPR);
  a.lds_row = PER * LPR * 4;
  const int grid = (int)((a.T + (int64_t)ROWS - 1) / ROWS);
  select_grad_kernel<LPR, PER><<<grid, kSelThreads, (size_t)ROWS * a.lds_row, stream>>>(a);
  return hipGetLastError();
}

static hipError_t launch_select_grad(const SelectGradArgs& a, hipStream_t stream) {
  if (select_many(a.T, kSelManyGrads, a.k, 1)) {
    if (a.E <= 64) return launch_select_grad_t<16, 4>(a, stream);
    if (a.E <= 128) return launch_select_grad_t<16, 8>(a, stream);
    if (a.E <= 256) return launch_select_grad_t<16, 16>(a, stream);
    return launch_select_grad_t<16, 32>(a, stream);
  }
  if (a.E <= 128) return launch_select_grad_t<64, 2>(a, stream);
  if (a.E <= 256) return launch_select_grad_t<64, 4>(a, stream);
  return launch_select_grad_t<64, 8>(a, stream);
}

}  // namespace nvr

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int check_select(int dtype, int scoring, int64_t T, int64_t E, int64_t k, int64_t ld) {
  if ((dtype != ROUTER_F32 && dtype != ROUTER_BF16) || (scoring != ROUTER_SIGMOID && scoring != ROUTER_SOFTMAX) ||
      T < 0 || E < 1 || k < 1 || k > E || ld < E)
    return ROUTER_EINVAL;
  if (E > ROUTER_MAX_EXPERTS || k > ROUTER_MAX_TOPK || T > ROUTER_MAX_SELECT_ROWS || ld >= (int64_t(1) << 31))
    return ROUTER_EUNSUPPORTED;
  return ROUTER_OK;
}

}  // namespace

extern "C" {

int router_select(const void* logits, int dtype, int64_t T, int64_t E, int64_t ld, const float* bias, int scoring,
                  int64_t groups, int64_t topk_groups, int64_t group_top, int renormalize, float routed_scale,
                  int64_t k, int32_t* topk_idx, float* topk_w, void* stream) {
  const int st = check_select(dtype, scoring, T, E, k, ld);
  if (groups < 1 || E < 1 || E % groups != 0 || topk_groups < 1 || topk_groups > groups || group_top < 1 ||
      group_top > 2)
    return ROUTER_EINVAL;
  if (st != ROUTER_OK) return st;
  if (k > topk_groups * (E / groups)) return ROUTER_EINVAL;
  if (groups > ROUTER_MAX_GROUPS) return ROUTER_EUNSUPPORTED;
  if (T > 0 && (!logits || !topk_idx || !topk_w)) return ROUTER_EINVAL;
  if (!aligned(logits, dtype == ROUTER_F32 ? 4 : 2) || !aligned(bias, 4) || !aligned(topk_idx, 4) ||
      !aligned(topk_w, 4))
    return ROUTER_EINVAL;
  if (T == 0) return ROUTER_OK;
  if (topk_groups == groups) groups = topk_groups = 1;
  nvr::SelectArgs a{};
  a.logits = logits; a.ld = ld; a.bias = bias; a.bf16 = dtype == ROUTER_BF16;
  a.T = (int)T; a.E = (int)E; a.k = (int)k;
  a.groups = (int)groups; a.size = (int)(E / groups); a.kept = (int)topk_groups; a.top = (int)group_top;
  a.inv = (uint32_t)(((1u << 20) + a.size - 1) / a.size);
  a.softmax = scoring == ROUTER_SOFTMAX; a.renorm = renormalize != 0;
  a.by_logit = !bias && (groups == 1 || group_top == 1);
  a.many = nvr::select_many(T, a.by_logit ? nvr::kSelManyLogits : nvr::kSelManyKeys, k, groups);
  while ((2 << a.sh) * groups <= (a.many ? 16 : 64)) ++a.sh;
  const size_t piece = dtype == ROUTER_F32 ? 16 : 8;  // four logits
  a.vec = aligned(logits, piece) && (size_t)ld * piece / 4 % piece == 0;
  a.scale = routed_scale;
  a.idx = topk_idx; a.w = topk_w;
  const hipError_t e = nvr::launch_select(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ROUTER_OK : ROUTER_EHIP;
}

int router_select_backward(const void* logits, int dtype, int64_t T, int64_t E, int64_t ld, const int32_t* topk_idx,
                           const float* grad_w, int scoring, int renormalize, float routed_scale, int64_t k,
                           void* grad_logits, int64_t ld_grad, void* stream) {
  const int st = check_select(dtype, scoring, T, E, k, ld);
  if (ld_grad < E) return ROUTER_EINVAL;
  if (st != ROUTER_OK) return st;
  if (ld_grad >= (int64_t(1) << 31)) return ROUTER_EUNSUPPORTED;
  if (T > 0 && (!logits || !topk_idx || !grad_w || !grad_logits)) return ROUTER_EINVAL;
  const size_t esize = dtype == ROUTER_F32 ? 4 : 2;
  if (!aligned(logits, esize) || !aligned(topk_idx, 4) || !aligned(grad_w, 4) || !aligned(grad_logits, esize))
    return ROUTER_EINVAL;
  if (T == 0) return ROUTER_OK;
  nvr::SelectGradArgs a{};
  a.logits = logits; a.ld = ld; a.idx = topk_idx; a.gw = grad_w; a.bf16 = dtype == ROUTER_BF16;
  a.T = (int)T; a.E = (int)E; a.k = (int)k;
  a.softmax = scoring == ROUTER_SOFTMAX; a.renorm = renormalize != 0; a.scale = routed_scale;
  a.out = grad_logits; a.ld_out = ld_grad;
  const hipError_t e = nvr::launch_select_grad(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ROUTER_OK : ROUTER_EHIP;
}

}  // extern "C"
