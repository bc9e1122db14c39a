// Penalties, token biases and a grammar mask on logits, and the greedy token
// (gfx950): what comes after the lm_head of a constrained greedy decoder.
//
// Per row t and token n, in fp32, each operation rounded by itself:
//   x = logits[t, n]
//   seen (n in history[t, :length]):      x = x > 0 ? x / r : x * r
//   made (c > 0 times from prompt on):    x = (x - f * c) - p
//   listed in the row's biases:           x = x + bias
//   mask bit clear:                       x = -inf
// and the largest x of the row (ties to the lower token; -inf and NaN are
// never chosen).
//
// One pass: a workgroup owns kPenChunk tokens of one row. It holds its logits
// in registers while it counts the row's history inside its range in LDS
// (integer atomics, so any order gives the same counts), then applies
// everything and writes once; the history is re-read by every chunk, from L2.
// A biased token listed more than once takes its last entry (an LDS maximum
// over entry numbers). The row's last workgroup to arrive takes the maximum
// over the chunks' candidates.
#include "../../include/nvfp4_router.h"
#include <type_traits>

#include "experts_common.hpp"

namespace nvr {

constexpr int kPenThreads = 512;
constexpr int kPenWaves = kPenThreads / 64;
constexpr int kPenChunk = 4096;

struct PenArgs {
  const void* in;
  void* out;
  int64_t ld;  // elements between rows, of both
  int T, N, chunks, row0;
  const int32_t* history;
  int64_t ld_history;
  int L;
  const int32_t* lengths;
  const int32_t* prompt;
  const float* repetition;
  const float* frequency;
  const float* presence;
  const int32_t* bias_start;
  const int32_t* bias_token;
  const float* bias_value;
  int nbias;
  const uint32_t* mask;
  int64_t ld_mask;
  int32_t* out_idx;
  float* out_logit;
  uint64_t* cand;  // [rows of a launch][chunks]
  uint32_t* counters;
};

__device__ __forceinline__ float pen_read(const float* p) { return *p; }
__device__ __forceinline__ float pen_read(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
__device__ __forceinline__ void pen_write(float* p, float v) { *p = v; }
__device__ __forceinline__ void pen_write(uint16_t* p, float v) { *p = bf16_round(v); }

__device__ __forceinline__ uint64_t pen_max_wave(uint64_t v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const uint32_t lo = (uint32_t)__shfl_xor((int)(uint32_t)v, o);
    const uint32_t hi = (uint32_t)__shfl_xor((int)(uint32_t)(v >> 32), o);
    const uint64_t u = ((uint64_t)hi << 32) | lo;
    v = u > v ? u : v;
  }
  return v;
}

__device__ __forceinline__ void pen_choice(const PenArgs& a, int t, uint64_t best) {
  const uint32_t k = (uint32_t)(best >> 32);
  a.out_idx[t] = best ? (int32_t)(0xFFFFFFFFu - (uint32_t)best) : -1;
  a.out_logit[t] = best ? __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k) : -__builtin_inff();
}

// E: float or uint16_t (bf16). VEC: 16-byte accesses (rows of both tensors
// 16-byte aligned).
template <class E, bool VEC>
__global__ __launch_bounds__(kPenThreads) void penalize_kernel(PenArgs a) {
  __shared__ uint32_t count[kPenChunk];  // bit 0: seen in the prompt; from bit 1: times made
  __shared__ uint32_t entry[kPenChunk];  // bias entry + 1
  __shared__ uint64_t wbest[kPenWaves];
  __shared__ uint32_t s_last;
  constexpr int VE = VEC ? 16 / (int)sizeof(E) : 1;
  constexpr int PER = kPenChunk / kPenThreads / VE;
  const int t = a.row0 + blockIdx.x / a.chunks, chunk = blockIdx.x % a.chunks;
  const int n0 = chunk * kPenChunk, nn = min(kPenChunk, a.N - n0);
  const E* in = static_cast<const E*>(a.in) + t * a.ld + n0;
  E* out = static_cast<E*>(a.out) + t * a.ld + n0;
  typedef E vec_t __attribute__((ext_vector_type(VE)));
  typedef typename std::conditional<VEC, vec_t, E>::type ev_t;
  ev_t v[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int n = (threadIdx.x + i * kPenThreads) * VE;
    if (n + VE <= nn) v[i] = *reinterpret_cast<const ev_t*>(in + n);
    else if constexpr (VEC) {
#pragma unroll
      for (int q = 0; q < VE; ++q) v[i][q] = n + q < nn ? in[n + q] : E(0);
    }
  }
  for (int i = threadIdx.x; i < kPenChunk; i += kPenThreads) {
    count[i] = 0u;
    entry[i] = 0u;
  }
  __syncthreads();
  if (a.history) {
    const int len = min(max(a.lengths ? a.lengths[t] : a.L, 0), a.L);
    const int made = a.prompt ? a.prompt[t] : 0;
    const int32_t* h = a.history + t * a.ld_history;
    for (int i = threadIdx.x; i < len; i += kPenThreads) {
      const uint32_t n = (uint32_t)h[i] - (uint32_t)n0;  // tokens outside this chunk, or the vocabulary, wrap past nn
      if (n < (uint32_t)nn) {
        if (i >= made) atomicAdd(&count[n], 2u);
        else atomicOr(&count[n], 1u);
      }
    }
  }
  if (a.bias_start) {
    const int b0 = max(a.bias_start[t], 0), b1 = min(a.bias_start[t + 1], a.nbias);
    for (int i = b0 + threadIdx.x; i < b1; i += kPenThreads) {
      const uint32_t n = (uint32_t)a.bias_token[i] - (uint32_t)n0;
      if (n < (uint32_t)nn) atomicMax(&entry[n], (uint32_t)(i + 1));
    }
  }
  __syncthreads();
  const float r = a.repetition ? a.repetition[t] : 1.0f;
  const float f = a.frequency ? a.frequency[t] : 0.0f, p = a.presence ? a.presence[t] : 0.0f;
  const uint32_t* mask = a.mask ? a.mask + t * a.ld_mask : nullptr;
  uint64_t best = 0ull;
  auto apply = [&](float x, int n) {
#pragma clang fp contract(off)  // each operation rounds by itself, as the definition says
    const uint32_t c = count[n];
    if (c != 0u) x = x > 0.0f ? x / r : x * r;
    if (c > 1u) {
      const float fc = f * (float)(c >> 1);
      x = (x - fc) - p;
    }
    const uint32_t b = entry[n];
    if (b) x = x + a.bias_value[b - 1];
    const int at = n0 + n;
    if (mask && ((mask[at >> 5] >> (at & 31)) & 1u) == 0u) x = -__builtin_inff();
    if (x > -__builtin_inff()) {
      const uint64_t key = ((uint64_t)score_key(x) << 32) | (0xFFFFFFFFu - (uint32_t)at);
      best = key > best ? key : best;
    }
    return x;
  };
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int n = (threadIdx.x + i * kPenThreads) * VE;
    if (n >= nn) continue;
    if constexpr (VEC) {
      ev_t o;
#pragma unroll
      for (int q = 0; q < VE; ++q) {
        if (n + q >= nn) continue;
        E e = v[i][q];
        pen_write(&e, apply(pen_read(&e), n + q));
        o[q] = e;
      }
      if (n + VE <= nn) *reinterpret_cast<ev_t*>(out + n) = o;
      else {
#pragma unroll
        for (int q = 0; q < VE; ++q)
          if (n + q < nn) out[n + q] = o[q];
      }
    } else {
      E e = v[i];
      pen_write(&e, apply(pen_read(&e), n));
      out[n] = e;
    }
  }
  best = pen_max_wave(best);
  if ((threadIdx.x & 63) == 0) wbest[threadIdx.x >> 6] = best;
  __syncthreads();
  const int row = t - a.row0;
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 1; w < kPenWaves; ++w) best = wbest[w] > best ? wbest[w] : best;
    if (a.chunks == 1) pen_choice(a, t, best);
    else __hip_atomic_store(a.cand + (int64_t)row * a.chunks + chunk, best, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  if (a.chunks == 1) return;
  if (!arrive_last(a.counters + row, a.chunks, &s_last)) return;
  if (threadIdx.x < 64) {
    uint64_t b = 0ull;
    for (int i = threadIdx.x; i < a.chunks; i += 64) {
      const uint64_t u = __hip_atomic_load(a.cand + (int64_t)row * a.chunks + i, __ATOMIC_RELAXED,
                                           __HIP_MEMORY_SCOPE_AGENT);
      b = u > b ? u : b;
    }
    b = pen_max_wave(b);
    if (threadIdx.x == 0) pen_choice(a, t, b);
  }
  release_counter(a.counters + row);
}

}  // namespace nvr

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool pen_shape_ok(int64_t T, int64_t N) {
  return T >= 0 && T < (int64_t(1) << 31) && N >= 1 && N <= (int64_t(1) << 30);
}

int64_t pen_chunks(int64_t N) { return (N + nvr::kPenChunk - 1) / nvr::kPenChunk; }

// Rows of one launch: an arrival counter each, and a grid below 2^31.
int64_t pen_rows(int64_t T) { return T < nvr::kMaxCounters ? T : nvr::kMaxCounters; }

}  // namespace

extern "C" size_t lmhead_penalize_workspace_bytes(int64_t T, int64_t N) {
  if (!pen_shape_ok(T, N)) return 0;
  return nvr::kScratchOffset + (size_t)(pen_rows(T) * pen_chunks(N)) * sizeof(uint64_t);
}

extern "C" int lmhead_penalize(const void* logits, int dtype, int64_t T, int64_t N, int64_t ld,
                               const int32_t* history, int64_t L, int64_t ld_history, const int32_t* lengths,
                               const int32_t* prompt, const float* repetition, const float* frequency,
                               const float* presence, const int32_t* bias_start, const int32_t* bias_token,
                               const float* bias_value, int64_t nbias, const uint32_t* mask, int64_t ld_mask,
                               void* out, int32_t* out_idx, float* out_logit, void* workspace,
                               size_t workspace_bytes, void* stream) {
  if (!pen_shape_ok(T, N) || ld < N || (dtype != ROUTER_F32 && dtype != ROUTER_BF16)) return ROUTER_EINVAL;
  if (T == 0) return ROUTER_OK;
  const size_t esize = dtype == ROUTER_F32 ? 4 : 2;
  if (!logits || !out || !out_idx || !out_logit || !aligned(logits, esize) || !aligned(out, esize) ||
      !aligned(out_idx, 4) || !aligned(out_logit, 4))
    return ROUTER_EINVAL;
  if (history && (L < 0 || L >= (int64_t(1) << 30) || ld_history < L || !aligned(history, 4))) return ROUTER_EINVAL;
  if (!history && (lengths || prompt)) return ROUTER_EINVAL;
  if (!aligned(lengths, 4) || !aligned(prompt, 4) || !aligned(repetition, 4) || !aligned(frequency, 4) ||
      !aligned(presence, 4) || !aligned(bias_start, 4) || !aligned(bias_token, 4) || !aligned(bias_value, 4) ||
      !aligned(mask, 4))
    return ROUTER_EINVAL;
  if (bias_start && (nbias < 0 || nbias >= (int64_t(1) << 31) || (nbias > 0 && (!bias_token || !bias_value))))
    return ROUTER_EINVAL;
  if (mask && ld_mask < (N + 31) / 32) return ROUTER_EINVAL;
  const int64_t chunks = pen_chunks(N);
  if (chunks > 1 && (!workspace || !aligned(workspace, 256) ||
                     workspace_bytes < lmhead_penalize_workspace_bytes(T, N)))
    return ROUTER_EINVAL;
  char* base = static_cast<char*>(workspace);
  const bool vec = aligned(logits, 16) && aligned(out, 16) && (ld * (int64_t)esize) % 16 == 0;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  for (int64_t row0 = 0; row0 < T; row0 += nvr::kMaxCounters) {
    const int64_t rows = pen_rows(T - row0);
    const nvr::PenArgs a{logits, out, ld, (int)T, (int)N, (int)chunks, (int)row0, history, ld_history, (int)L,
                         lengths, prompt, repetition, frequency, presence, bias_start, bias_token, bias_value,
                         (int)nbias, mask, ld_mask, out_idx, out_logit,
                         chunks > 1 ? reinterpret_cast<uint64_t*>(base + nvr::kScratchOffset) : nullptr,
                         reinterpret_cast<uint32_t*>(base)};
    const int grid = (int)(rows * chunks);
    if (dtype == ROUTER_F32) {
      if (vec) nvr::penalize_kernel<float, true><<<grid, nvr::kPenThreads, 0, s>>>(a);
      else nvr::penalize_kernel<float, false><<<grid, nvr::kPenThreads, 0, s>>>(a);
    } else {
      if (vec) nvr::penalize_kernel<uint16_t, true><<<grid, nvr::kPenThreads, 0, s>>>(a);
      else nvr::penalize_kernel<uint16_t, false><<<grid, nvr::kPenThreads, 0, s>>>(a);
    }
    if (hipGetLastError() != hipSuccess) return ROUTER_EHIP;
  }
  return ROUTER_OK;
}
