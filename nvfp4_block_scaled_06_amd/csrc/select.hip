// Routing on given logits and its gradient (gfx950): the rules of choice that
// the gate's fused epilogue does not have.
//
// Per row: s = sigmoid(l) or softmax(l); key = s + bias; of `groups` groups of
// neighbouring experts the `kept` with the largest sums of their one or two
// best keys stay; the k largest keys among them in descending order, ties to
// the lower expert; w = scale s / (1 or the sum of the chosen s).
//
// The order is that of keys computed in 64 bits, so it does not hang on how a
// logistic function rounds. Nearly every row is decided in 32 bits: without a
// bias the order of the logits is the order of the keys, and is exact; with
// one, keys computed in 32 bits are off by less than kKeyErr, and where two
// neighbours in the order, or the last group kept and the first one left out,
// are closer than that, the wavefront does its rows again in 64 bits (about
// one row of a thousand at 256 experts and k = 8).
//
// A row is one wavefront's, or 16 lanes' with four rows to a wavefront where
// rows are many: a round of the choice then costs four rows as many
// instructions as it costs one.
#include "../../include/nvfp4_router.h"
#include <type_traits>

#include "experts_common.hpp"

namespace nvr {

constexpr int kSelWaves = 4;
constexpr int kSelThreads = 64 * kSelWaves;
constexpr float kKeyErr = 4e-6f;  // of keys up to 1; fp32 rounding of larger ones (a large bias) scales it

struct SelectArgs {
  const void* logits;
  int64_t ld;
  const float* bias;
  int bf16, T, E, k;
  int groups, size, kept, top, sh;  // sh: log2 of the lanes per group
  uint32_t inv;                     // 2^20 / size rounded up: e / size = e inv >> 20 for e < 512
  int softmax, renorm, by_logit;
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

// Keys: unsigned integers in the order of their values; 0 for experts that cannot be chosen.
__device__ __forceinline__ uint32_t order_key(float v) { return score_key(v); }
__device__ __forceinline__ uint64_t order_key(double v) {
  const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);
  return (u >> 63) ? ~u : (u | (1ull << 63));
}
__device__ __forceinline__ float key_back(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

// Reductions over a row's lanes, in a fixed order.
template <int LPR>
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  if constexpr (LPR == 64) return wave_max_u32(v);
  else return group_max_u32<16>(v);
}
template <int LPR>
__device__ __forceinline__ uint64_t row_max(uint64_t v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) {
    const uint32_t lo = (uint32_t)__shfl_xor((int)(uint32_t)v, o), hi = (uint32_t)__shfl_xor((int)(uint32_t)(v >> 32), o);
    const uint64_t u = ((uint64_t)hi << 32) | lo;
    v = u > v ? u : v;
  }
  return v;
}
template <int LPR>
__device__ __forceinline__ uint32_t row_min(uint32_t v) {
  if constexpr (LPR == 64) return wave_min_u32(v);
  else return ~group_max_u32<16>(~v);
}
template <int LPR, class F>
__device__ __forceinline__ F row_fmax(F v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) {
    const F u = __shfl_xor(v, o);
    v = u > v ? u : v;
  }
  return v;
}
template <int LPR, class F>
__device__ __forceinline__ F row_sum(F v) {
#pragma unroll
  for (int o = 1; o < LPR; o <<= 1) v += __shfl_xor(v, o);
  return v;
}

__device__ __forceinline__ void sel_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The choice with keys of type F; lane j < k of the row gets the j-th expert,
// -1 where none is left. True (for the whole row) where the order is closer
// than the keys' error.
template <int LPR, int PER, class F>
__device__ __forceinline__ bool sel_choose(const SelectArgs& a, const float (&l)[PER], float top, char* row_lds,
                                           int& chosen) {
  typedef typename std::conditional<sizeof(F) == 4, uint32_t, uint64_t>::type key_t;
  constexpr bool kWide = sizeof(F) == 8;
  const F ninf = -(F)__builtin_inff();
  const int lane = threadIdx.x & 63, li = lane & (LPR - 1);
  const bool exact = kWide || a.by_logit;
  bool unsure = false;
  F v[PER];
  if (a.by_logit) {
#pragma unroll
    for (int j = 0; j < PER; ++j) v[j] = (F)l[j];
  } else {
    if (a.softmax) {
      F sum = 0;
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        if constexpr (kWide) v[j] = exp((double)l[j] - (double)top);
        else v[j] = exp_fast(l[j] - top);
        sum += v[j];
      }
      sum = row_sum<LPR>(sum);
#pragma unroll
      for (int j = 0; j < PER; ++j) v[j] /= sum;
    } else {
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        if constexpr (kWide) v[j] = 1.0 / (1.0 + exp(-(double)l[j]));
        else v[j] = sigmoid_fast(l[j]);
      }
    }
    if (a.bias) {
#pragma unroll
      for (int j = 0; j < PER; ++j) v[j] += (F)a.bias[min(LPR * j + li, a.E - 1)];
    }
  }
  key_t key[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const bool alive = LPR * j + li < a.E && l[j] > -__builtin_inff() && v[j] > ninf;
    if (!alive) v[j] = ninf;
    key[j] = alive ? order_key(v[j]) : key_t(0);
  }

  if (a.kept < a.groups) {
    F* vals = reinterpret_cast<F*>(row_lds);
    sel_fence();
#pragma unroll
    for (int j = 0; j < PER; ++j) vals[LPR * j + li] = v[j];
    sel_fence();
    const int g = li >> a.sh, lpg = 1 << a.sh;
    F b1 = ninf, b2 = ninf;
    if (g < a.groups) {
      for (int i = li & (lpg - 1); i < a.size; i += lpg) {
        const F x = vals[g * a.size + i];
        const F lo = x < b1 ? x : b1;
        b2 = lo > b2 ? lo : b2;
        b1 = x > b1 ? x : b1;
      }
    }
    for (int o = 1; o < lpg; o <<= 1) {
      const F o1 = __shfl_xor(b1, o), o2 = __shfl_xor(b2, o);
      const F lo = o1 < b1 ? o1 : b1, hi2 = o2 > b2 ? o2 : b2;
      b2 = lo > hi2 ? lo : hi2;
      b1 = o1 > b1 ? o1 : b1;
    }
    F score = a.top == 2 && a.size > 1 ? b1 + b2 : b1;
    if (!(score == score) || g >= a.groups) score = ninf;
    int rank = 0;
    for (int j = 0; j < a.groups; ++j) {
      const F s = __shfl(score, (lane & ~(LPR - 1)) + (j << a.sh));
      rank += s > score || (s == score && j < g) ? 1 : 0;
    }
    const bool keep = g < a.groups && rank < a.kept;
    const uint64_t kept = __ballot(keep) >> (lane & ~(LPR - 1));
    if (!exact) {
      const F lowest = -row_fmax<LPR, F>(keep ? -score : ninf);
      const F next = row_fmax<LPR, F>(!keep && g < a.groups ? score : ninf);
      if (lowest > ninf && lowest - next <= (F)(2.0f * kKeyErr) * fmaxf(1.0f, fabsf((float)lowest))) unsure = true;
    }
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const uint32_t e = LPR * j + li;
      const uint32_t ge = min((uint32_t)((e * a.inv) >> 20), (uint32_t)a.groups - 1u);
      if (!((kept >> (ge << a.sh)) & 1ull)) key[j] = key_t(0);
    }
  }

  chosen = -1;
  key_t before = 0;
  for (int r = 0; r <= a.k; ++r) {
    key_t m = key[0];
#pragma unroll
    for (int j = 1; j < PER; ++j) m = key[j] > m ? key[j] : m;
    const key_t best = row_max<LPR>(m);
    if constexpr (!kWide) {
      if (!exact && r > 0 && best != 0u) {
        const float p = key_back(before);
        if (p - key_back(best) <= kKeyErr * fmaxf(1.0f, fabsf(p))) unsure = true;
      }
    }
    if (r == a.k) break;
    before = best;
    // The lowest expert with that key.
    uint32_t at = 0xFFFFFFFFu;
#pragma unroll
    for (int j = PER - 1; j >= 0; --j) at = key[j] == best ? (uint32_t)(LPR * j + li) : at;
    at = best ? row_min<LPR>(at) : 0xFFFFFFFFu;
#pragma unroll
    for (int j = 0; j < PER; ++j) key[j] = (uint32_t)(LPR * j + li) == at ? key_t(0) : key[j];
    if (li == r) chosen = (int)at;
  }
  return unsure;
}

// s of a logit, up to a factor common to the row that makes the largest of the
// chosen ones exp(0) or nearly: the quotient s / sum s then holds for any
// finite logits (all of them -1e30, for example). `m` is 0 for s itself.
__device__ __forceinline__ float sel_score(float l, float m, bool softmax) {
  return softmax ? expf(l - m) : expf(fminf(l, 0.0f) - m) / (1.0f + expf(-fabsf(l)));
}

template <int LPR, int PER>
__global__ __launch_bounds__(kSelThreads) void select_kernel(SelectArgs a) {
  extern __shared__ __attribute__((aligned(16))) char sel_lds[];
  constexpr int ROWS = 64 / LPR;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, li = lane & (LPR - 1);
  const int in_wg = wave * ROWS + lane / LPR;
  const int64_t row = (int64_t)blockIdx.x * (kSelWaves * ROWS) + in_wg;
  const bool live = row < a.T;
  const int64_t base = (live ? row : a.T - 1) * a.ld;
  char* row_lds = sel_lds + in_wg * a.lds_row;
  float l[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int e = LPR * j + li;
    l[j] = sel_logit(a.logits, a.bf16, base + min(e, a.E - 1));
    if (e >= a.E) l[j] = -__builtin_inff();
  }
  float top = 0.0f, sum = 1.0f;  // softmax over the whole row, where that is needed
  if (a.softmax && !(a.by_logit && a.renorm)) {
    top = l[0];
#pragma unroll
    for (int j = 1; j < PER; ++j) top = fmaxf(top, l[j]);
    top = row_fmax<LPR, float>(top);
    sum = 0.0f;
#pragma unroll
    for (int j = 0; j < PER; ++j) sum += exp_fast(l[j] - top);
    sum = row_sum<LPR>(sum);
  }
  int chosen;
  const bool unsure = sel_choose<LPR, PER, float>(a, l, top, row_lds, chosen);
  if (__ballot(unsure && live)) sel_choose<LPR, PER, double>(a, l, top, row_lds, chosen);

  // The chosen ones' logits, through LDS.
  float* ll = reinterpret_cast<float*>(row_lds);
  sel_fence();
#pragma unroll
  for (int j = 0; j < PER; ++j) ll[LPR * j + li] = l[j];
  sel_fence();
  const bool mine = chosen >= 0;
  const float cl = mine ? ll[chosen] : -__builtin_inff();
  float m = a.softmax ? top : 0.0f;
  if (a.renorm) m = row_fmax<LPR, float>(a.softmax ? cl : fminf(cl, 0.0f));
  const float s = mine ? sel_score(cl, m, a.softmax) : 0.0f;
  float total = sum;  // 1 for plain sigmoid scores
  if (a.renorm) total = row_sum<LPR>(s);
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
    sum = row_sum<LPR>(sum);
    if (!(sum > 0.0f) && sum == sum) sum = 1.0f;
  }
  float m = a.softmax ? top : 0.0f;
  if (a.renorm) {
    m = row_fmax<LPR, float>(a.softmax ? cl : fminf(cl, 0.0f));
    if (!(m > -__builtin_inff())) m = 0.0f;
  }
  const float s = e >= 0 ? sel_score(cl, m, a.softmax) : 0.0f;
  float total = sum;
  if (a.renorm) total = row_sum<LPR>(s);
  const float u = s > 0.0f || s != s ? s / total : 0.0f;
  float dot = 0.0f;
  if (a.softmax || a.renorm) dot = row_sum<LPR>(u * gw);
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

// 16 lanes to a row from this many rows on, where a row's places and groups
// fit into 16 lanes.
constexpr int64_t kSelManyRows = 1024;

template <int LPR, int PER, class A>
static hipError_t launch_select_t(A& a, hipStream_t stream, bool values64) {
  constexpr int ROWS = kSelWaves * (64 / LPR);
  a.lds_row = PER * LPR * (values64 ? 8 : 4);
  const int grid = (int)((a.T + (int64_t)ROWS - 1) / ROWS);
  if constexpr (std::is_same<A, SelectArgs>::value)
    select_kernel<LPR, PER><<<grid, kSelThreads, (size_t)ROWS * a.lds_row, stream>>>(a);
  else
    select_grad_kernel<LPR, PER><<<grid, kSelThreads, (size_t)ROWS * a.lds_row, stream>>>(a);
  return hipGetLastError();
}

template <class A>
static hipError_t launch_select(A a, int groups, hipStream_t stream) {
  const bool values64 = groups > 1;
  if (a.T >= kSelManyRows && a.k <= 16 && groups <= 16) {
    if (a.E <= 64) return launch_select_t<16, 4>(a, stream, values64);
    if (a.E <= 128) return launch_select_t<16, 8>(a, stream, values64);
    if (a.E <= 256) return launch_select_t<16, 16>(a, stream, values64);
    if (a.E <= 384) return launch_select_t<16, 24>(a, stream, values64);
    return launch_select_t<16, 32>(a, stream, values64);
  }
  if (a.E <= 64) return launch_select_t<64, 1>(a, stream, values64);
  if (a.E <= 128) return launch_select_t<64, 2>(a, stream, values64);
  if (a.E <= 256) return launch_select_t<64, 4>(a, stream, values64);
  if (a.E <= 384) return launch_select_t<64, 6>(a, stream, values64);
  return launch_select_t<64, 8>(a, stream, values64);
}

}  // namespace nvr

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int check_select(int dtype, int scoring, int64_t T, int64_t E, int64_t k, int64_t ld) {
  if ((dtype != ROUTER_F32 && dtype != ROUTER_BF16) || (scoring != ROUTER_SIGMOID && scoring != ROUTER_SOFTMAX) ||
      T < 0 || E < 1 || k < 1 || k > E || ld < E)
    return ROUTER_EINVAL;
  if (E > ROUTER_MAX_EXPERTS || k > ROUTER_MAX_TOPK || T >= (int64_t(1) << 31) || ld >= (int64_t(1) << 31))
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
  const int lanes = T >= nvr::kSelManyRows && k <= 16 && groups <= 16 ? 16 : 64;
  while ((2 << a.sh) * groups <= lanes) ++a.sh;
  a.inv = (uint32_t)(((1u << 20) + a.size - 1) / a.size);
  a.softmax = scoring == ROUTER_SOFTMAX; a.renorm = renormalize != 0;
  a.by_logit = !bias && (groups == 1 || group_top == 1);
  a.scale = routed_scale;
  a.idx = topk_idx; a.w = topk_w;
  const hipError_t e = nvr::launch_select(a, (int)groups, static_cast<hipStream_t>(stream));
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
  const hipError_t e = nvr::launch_select(a, 1, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ROUTER_OK : ROUTER_EHIP;
}

}  // extern "C"
