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
// One pass over the logits, bound by HBM at many rows and by latency at few. A
// workgroup takes chunks of 4096 tokens of one row in turn: it counts the
// row's history that falls into the chunk in LDS (integer atomics, so any
// order gives the same counts), applies everything to the logits it holds in
// registers and writes them once, while the next chunk's logits load. The
// history and the biases are read once per workgroup and stay in registers
// (8 tokens and one bias per thread; longer lists are re-read per chunk). A
// token biased more than once takes its last entry: an LDS maximum over
// (entry, value) pairs. The row's last workgroup to arrive takes the maximum
// over the others' candidates.
//
// T = 256, N = 129280, histories to 4096, 300 biases, masks, fp32: 59 us =
// 4.6 TB/s with nontemporal accesses (65.5 without; the logits fill the
// caches twice over), 123 us with a workgroup per chunk that re-reads the
// history and looks at every token's counts by itself. In bf16 42 us, 3.3
// TB/s: as many instructions for a token as in fp32. T = 1: 7.0 us.
#include "../../include/nvfp4_router.h"
#include <type_traits>

#include "experts_common.hpp"

namespace nvr {

constexpr int kPenThreads = 512;
constexpr int kPenChunk = 4096;
constexpr int kPenHeld = 8;  // history tokens per thread in registers
constexpr uint32_t kPenBias = 0x80000000u, kPenSeen = 0x40000000u;  // flags above a count below 2^30

struct PenArgs {
  const void* in;
  void* out;
  int64_t ld, ld_out;  // elements between rows
  int T, N, chunks, segs, row0;
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
  uint64_t* cand;  // [rows of a launch][segs]
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
  constexpr int NT = kPenThreads, VE = VEC ? 16 / (int)sizeof(E) : 1, PER = kPenChunk / NT / VE;
  __shared__ __attribute__((aligned(16))) uint32_t state[kPenChunk];  // kPenBias | kPenSeen | times made
  __shared__ __attribute__((aligned(16))) unsigned long long entry[kPenChunk];  // bias entry + 1, and its value's bits
  __shared__ uint64_t wbest[NT / 64];
  __shared__ uint32_t s_last;
  const int t = a.row0 + blockIdx.x / a.segs, seg = blockIdx.x % a.segs;
  const int first = (int)((int64_t)a.chunks * seg / a.segs), last = (int)((int64_t)a.chunks * (seg + 1) / a.segs);
  const E* in = static_cast<const E*>(a.in) + t * a.ld;
  E* out = static_cast<E*>(a.out) + t * a.ld_out;
  typedef E vec_t __attribute__((ext_vector_type(VE)));
  typedef typename std::conditional<VEC, vec_t, E>::type ev_t;
  ev_t v[PER];
  auto load = [&](int chunk) {
    const int n0 = chunk * kPenChunk, nn = min(kPenChunk, a.N - n0);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int n = (threadIdx.x + i * NT) * VE;
      if (n + VE <= nn) v[i] = __builtin_nontemporal_load(reinterpret_cast<const ev_t*>(in + n0 + n));
      else if constexpr (VEC) {
#pragma unroll
        for (int q = 0; q < VE; ++q) v[i][q] = n + q < nn ? in[n0 + n + q] : E(0);
      }
    }
  };
  load(first);
  // The row's first kPenHeld * NT history tokens stay in registers.
  const int len = a.history ? min(max(a.lengths ? a.lengths[t] : a.L, 0), a.L) : 0;
  const int made = a.prompt ? a.prompt[t] : 0;
  const int32_t* h = a.history + t * a.ld_history;
  int held[kPenHeld];
#pragma unroll
  for (int j = 0; j < kPenHeld; ++j) {
    const int i = threadIdx.x + j * NT;
    held[j] = i < len ? h[i] : -1;  // -1: in no chunk
  }
  // And the first NT of its nb biases. Both ends are clamped, and indices count
  // from b0 and are unsigned: whatever the starts are, none passes nbias.
  uint32_t b0 = 0u, nb = 0u;
  if (a.bias_start) {
    b0 = (uint32_t)min(max(a.bias_start[t], 0), a.nbias);
    nb = (uint32_t)max(min(a.bias_start[t + 1], a.nbias), (int)b0) - b0;
  }
  int held_token = -1;
  float held_value = 0.0f;
  if (threadIdx.x < nb) {
    held_token = a.bias_token[b0 + threadIdx.x];
    held_value = a.bias_value[b0 + threadIdx.x];
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) reinterpret_cast<u32x4_t*>(state)[threadIdx.x + i * NT] = u32x4_t{0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 4; ++i) reinterpret_cast<u32x4_t*>(entry)[threadIdx.x + i * NT] = u32x4_t{0u, 0u, 0u, 0u};
  const float r = a.repetition ? a.repetition[t] : 1.0f;
  const float f = a.frequency ? a.frequency[t] : 0.0f, p = a.presence ? a.presence[t] : 0.0f;
  const uint32_t* mask = a.mask ? a.mask + t * a.ld_mask : nullptr;
  float best = -__builtin_inff();  // and the first token with it; NaN never compares greater
  int best_at = -1;
  for (int chunk = first; chunk < last; ++chunk) {
    const int n0 = chunk * kPenChunk, nn = min(kPenChunk, a.N - n0);
    __syncthreads();  // the counts are zero again
    auto count = [&](int tok, int i) {
      const uint32_t n = (uint32_t)tok - (uint32_t)n0;  // tokens outside this chunk, or the vocabulary, wrap past nn
      if (n < (uint32_t)nn) {
        if (i >= made) atomicAdd(&state[n], 1u);
        else atomicOr(&state[n], kPenSeen);
      }
    };
#pragma unroll
    for (int j = 0; j < kPenHeld; ++j) count(held[j], threadIdx.x + j * NT);
    for (int i = threadIdx.x + kPenHeld * NT; i < len; i += NT) count(h[i], i);
    auto list = [&](int tok, float value, uint32_t i) {
      const uint32_t n = (uint32_t)tok - (uint32_t)n0;
      if (n < (uint32_t)nn) {
        atomicMax(&entry[n], ((unsigned long long)(i + 1u) << 32) | __float_as_uint(value));
        atomicOr(&state[n], kPenBias);
      }
    };
    list(held_token, held_value, threadIdx.x);
    for (uint32_t i = threadIdx.x + NT; i < nb; i += NT) list(a.bias_token[b0 + i], a.bias_value[b0 + i], i);
    // Everything else that this chunk reads is requested before the next
    // chunk's logits: loads complete in order.
    uint32_t allowed[PER];
    ev_t w[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int n = (threadIdx.x + i * NT) * VE;  // VE tokens of one mask word
      allowed[i] = mask && n < nn ? mask[(n0 + n) >> 5] >> ((n0 + n) & 31) : 0xFFFFFFFFu;
      w[i] = v[i];
    }
    if (chunk + 1 < last) load(chunk + 1);
    __syncthreads();
    auto apply = [&](float x, int n, uint32_t c, uint32_t ok) {
#pragma clang fp contract(off)  // each operation rounds by itself, as the definition says
      if (c != 0u) {
        const uint32_t times = c & (kPenSeen - 1u);
        if (c & ~kPenBias) x = x > 0.0f ? x / r : x * r;
        if (times != 0u) {
          const float fc = f * (float)times;
          x = (x - fc) - p;
        }
        if (c & kPenBias) {
          x = x + __uint_as_float((uint32_t)entry[n]);
          entry[n] = 0ull;
        }
      }
      if (!(ok & 1u)) x = -__builtin_inff();
      if (x > best) {
        best = x;
        best_at = n0 + n;
      }
      return x;
    };
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int n = (threadIdx.x + i * NT) * VE;
      if (n >= nn) continue;
      if constexpr (VEC) {
        uint32_t c[VE];
#pragma unroll
        for (int q = 0; q < VE / 4; ++q) {
          const u32x4_t u = *reinterpret_cast<const u32x4_t*>(&state[n + 4 * q]);
          *reinterpret_cast<u32x4_t*>(&state[n + 4 * q]) = u32x4_t{0u, 0u, 0u, 0u};
#pragma unroll
          for (int j = 0; j < 4; ++j) c[4 * q + j] = u[j];
        }
        ev_t o;
#pragma unroll
        for (int q = 0; q < VE; ++q) {
          E e = w[i][q];
          const float x = n + q < nn ? apply(pen_read(&e), n + q, c[q], allowed[i] >> q) : 0.0f;
          pen_write(&e, x);
          o[q] = e;
        }
        if (n + VE <= nn) __builtin_nontemporal_store(o, reinterpret_cast<ev_t*>(out + n0 + n));
        else {
#pragma unroll
          for (int q = 0; q < VE; ++q)
            if (n + q < nn) out[n0 + n + q] = o[q];
        }
      } else {
        E e = w[i];
        const uint32_t c = state[n];
        state[n] = 0u;
        pen_write(&e, apply(pen_read(&e), n, c, allowed[i]));
        out[n0 + n] = e;
      }
    }
  }
  // A thread's tokens ascend, so its first maximum is its lowest token.
  uint64_t key = best_at >= 0 ? ((uint64_t)score_key(best) << 32) | (0xFFFFFFFFu - (uint32_t)best_at) : 0ull;
  key = pen_max_wave(key);
  if ((threadIdx.x & 63) == 0) wbest[threadIdx.x >> 6] = key;
  __syncthreads();
  const int row = t - a.row0;
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 1; w < NT / 64; ++w) key = wbest[w] > key ? wbest[w] : key;
    if (a.segs == 1) pen_choice(a, t, key);
    else __hip_atomic_store(a.cand + (int64_t)row * a.segs + seg, key, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  if (a.segs == 1) return;
  if (!arrive_last(a.counters + row, a.segs, &s_last)) return;
  if (threadIdx.x < 64) {
    uint64_t b = 0ull;
    for (int i = threadIdx.x; i < a.segs; i += 64) {
      const uint64_t u = __hip_atomic_load(a.cand + (int64_t)row * a.segs + i, __ATOMIC_RELAXED,
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

// Workgroups per row: one per chunk while a launch is no more than the three
// workgroups that each compute unit holds; then each takes several chunks in
// turn, the next one's logits loading meanwhile (T = 256, N = 129280: 65.5 us,
// against 73 with twice as many workgroups and 97 with one per chunk).
int64_t pen_segs(int64_t rows, int64_t chunks) {
  const int64_t per = (rows * chunks + 767) / 768;
  return (chunks + per - 1) / per;
}

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
                               void* out, int64_t ld_out, int32_t* out_idx, float* out_logit, void* workspace,
                               size_t workspace_bytes, void* stream) {
  if (!pen_shape_ok(T, N) || ld < N || ld_out < N || (dtype != ROUTER_F32 && dtype != ROUTER_BF16)) return ROUTER_EINVAL;
  if (T == 0) return ROUTER_OK;
  const size_t esize = dtype == ROUTER_F32 ? 4 : 2;
  if (!logits || !out || !out_idx || !out_logit || !aligned(logits, esize) || !aligned(out, esize) ||
      !aligned(out_idx, 4) || !aligned(out_logit, 4))
    return ROUTER_EINVAL;
  if (out == logits && ld != ld_out && T > 1) return ROUTER_EINVAL;
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
  const bool vec = aligned(logits, 16) && aligned(out, 16) && (ld * (int64_t)esize) % 16 == 0 &&
                   (ld_out * (int64_t)esize) % 16 == 0;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  for (int64_t row0 = 0; row0 < T; row0 += nvr::kMaxCounters) {
    const int64_t rows = pen_rows(T - row0);
    const int64_t segs = pen_segs(rows, chunks);
    const nvr::PenArgs a{logits, out, ld, ld_out, (int)T, (int)N, (int)chunks, (int)segs, (int)row0, history,
                         ld_history, (int)L, lengths, prompt, repetition, frequency, presence, bias_start, bias_token, bias_value,
                         (int)nbias, mask, ld_mask, out_idx, out_logit,
                         chunks > 1 ? reinterpret_cast<uint64_t*>(base + nvr::kScratchOffset) : nullptr,
                         reinterpret_cast<uint32_t*>(base)};
    const int grid = (int)(rows * segs);
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
