// Sorting of routed slots by expert (gfx950): the step between the router's
// top-k and the experts' products.
//
// Slot s = t k + j is token t's j-th choice, e(s) = topk_idx[s] -
// first_expert its expert among the G held here, or none (bin G). A stable
// counting sort gives
//   offsets[g] = number of slots with e < g,
//   rows[p]    = the slot of row p (-1 from offsets[G] on),
//   pos[s]     = the row of slot s (-1 for slots of no expert).
// Stable, so the result is one fixed permutation. Integers only: the
// histograms' LDS atomics may run in any order.
//
// Bound by latency: the chain of load, count, scan and place. T = 1, k = 8,
// 256 experts: 3.2 us in one workgroup of four wavefronts. T = 32768, k = 8,
// 384 experts: 3.2 us for the 64 chunks' histograms and 10.4 us to place the
// slots (3.1 MB in all), each as the profiler takes it by itself; 12.6 us a
// call in a row of calls without the profiler, 28.7 us before the threads
// shared the chunks' histograms.
#include "../../include/nvfp4_router.h"
#include "experts_common.hpp"

namespace nvr {

constexpr int kPlanThreads = 1024;
constexpr int kPlanBins = kMaxGroups + 1;
constexpr int kPlanChunk = 4096;     // slots per workgroup, at least
constexpr int kPlanMaxChunks = 256;  // every workgroup reads every chunk's histogram

struct PlanArgs {
  const int32_t* idx;
  int R, G;
  int64_t first;
  int32_t* offsets;
  int32_t* rows;
  int32_t* pos;
  int32_t* hist;  // [chunks][G + 1] workspace (more than one chunk)
  int chunk;      // slots per workgroup
};

__device__ __forceinline__ int plan_bin(const PlanArgs& a, int s) {
  const int64_t e = (int64_t)a.idx[s] - a.first;
  return e >= 0 && e < a.G ? (int)e : a.G;
}

// One histogram per chunk of slots.
__global__ __launch_bounds__(kPlanThreads) void plan_hist_kernel(PlanArgs a) {
  __shared__ int h[kPlanBins];
  const int s0 = blockIdx.x * a.chunk, s1 = min(s0 + a.chunk, a.R);
  for (int i = threadIdx.x; i <= a.G; i += kPlanThreads) h[i] = 0;
  __syncthreads();
  for (int s = s0 + threadIdx.x; s < s1; s += kPlanThreads) atomicAdd(&h[plan_bin(a, s)], 1);
  __syncthreads();
  for (int i = threadIdx.x; i <= a.G; i += kPlanThreads) a.hist[(int64_t)blockIdx.x * (a.G + 1) + i] = h[i];
}

// Places one chunk's slots. Each of WAVES wavefronts owns a contiguous segment
// of the chunk: it counts its slots per bin, the workgroup turns the counts
// into first rows (bins in order, chunks in order inside a bin, wavefronts in
// order inside a chunk), and the wavefront places 64 slots at a time, a slot's
// rank among the 64 being the number of lower lanes with its bin (one ballot
// per bit of the bin). A thread's first kPlanHeld slots stay in registers
// between the two. With several chunks the threads share the chunks'
// histograms of each bin, all loads of a share in flight at once.
constexpr int kPlanHeld = 4;

template <int WAVES>
__global__ __launch_bounds__(64 * WAVES) void plan_place_kernel(PlanArgs a) {
  constexpr int NT = 64 * WAVES;
  __shared__ int h[WAVES][kPlanBins];
  __shared__ int total[kPlanBins], low[kPlanBins];  // a bin's slots in all chunks, and in lower ones
  __shared__ int wsum[WAVES];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, nb = a.G + 1;
  const int s0 = blockIdx.x * a.chunk, s1 = min(s0 + a.chunk, a.R);
  const int seg = ((s1 - s0 + WAVES - 1) / WAVES + 63) & ~63;
  const int b0 = min(s0 + wave * seg, s1), b1 = min(b0 + seg, s1);
  int held[kPlanHeld];
#pragma unroll
  for (int j = 0; j < kPlanHeld; ++j) held[j] = b0 + 64 * j + lane < b1 ? plan_bin(a, b0 + 64 * j + lane) : -1;
  for (int w = 0; w < WAVES; ++w)
    for (int i = threadIdx.x; i < nb; i += NT) h[w][i] = 0;
  for (int i = threadIdx.x; i < nb; i += NT) total[i] = low[i] = 0;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kPlanHeld; ++j)
    if (held[j] >= 0) atomicAdd(&h[wave][held[j]], 1);
  for (int s = b0 + 64 * kPlanHeld + lane; s < b1; s += 64) atomicAdd(&h[wave][plan_bin(a, s)], 1);
  if (gridDim.x > 1) {
    const int chunks = gridDim.x, shares = max(NT / nb, 1), each = (chunks + shares - 1) / shares;
    for (int i = threadIdx.x; i < shares * nb; i += NT) {
      const int bin = i % nb, c0 = (i / nb) * each, c1 = min(c0 + each, chunks);
      int t = 0, l = 0;
      for (int c = c0; c < c1; c += 16) {
        int v[16];
#pragma unroll
        for (int u = 0; u < 16; ++u) v[u] = a.hist[(int64_t)min(c + u, c1 - 1) * nb + bin];
#pragma unroll
        for (int u = 0; u < 16; ++u) {
          const int n = c + u < c1 ? v[u] : 0;
          t += n;
          l += c + u < (int)blockIdx.x ? n : 0;
        }
      }
      atomicAdd(&total[bin], t);
      atomicAdd(&low[bin], l);
    }
  }
  __syncthreads();

  // Exclusive scan over the bins, kPerThread adjacent ones per thread.
  constexpr int kPerThread = (kPlanBins + NT - 1) / NT;
  const int i0 = threadIdx.x * kPerThread;
  int sum = 0, mine[kPerThread];
#pragma unroll
  for (int j = 0; j < kPerThread; ++j) {
    const int i = i0 + j;
    int n = 0;
    if (i < nb) {
      if (gridDim.x > 1) n = total[i];
      else {
#pragma unroll
        for (int w = 0; w < WAVES; ++w) n += h[w][i];
      }
    }
    mine[j] = n;
    sum += n;
  }
  const int incl = wave_prefix_sum(sum);
  if (lane == 63) wsum[wave] = incl;
  __syncthreads();
  int at = incl - sum;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) at += w < wave ? wsum[w] : 0;
#pragma unroll
  for (int j = 0; j < kPerThread; ++j) {
    const int i = i0 + j;
    if (i < nb) {
      if (blockIdx.x == 0) a.offsets[i] = at;  // offsets[G]: the rows of bins below G
      int p = at + low[i];
#pragma unroll
      for (int w = 0; w < WAVES; ++w) {
        const int n = h[w][i];
        h[w][i] = p;
        p += n;
      }
      at += mine[j];
    }
  }
  __syncthreads();

  const int bits = 32 - __builtin_clz((unsigned)a.G);
  auto place = [&](int s, int e) {  // 64 slots, e < 0: none
    const bool ok = e >= 0;
    uint64_t peers = __ballot(ok);
    for (int b = 0; b < bits; ++b) {
      const uint64_t m = __ballot((e >> b) & 1);
      peers &= ((e >> b) & 1) ? m : ~m;
    }
    if (ok) {
      const int p = h[wave][e] + (int)__popcll(peers & ((1ull << lane) - 1ull));
      a.rows[p] = e < a.G ? s : -1;
      a.pos[s] = e < a.G ? p : -1;
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    // The last peer moves the bin's next row on (LDS accesses of one
    // wavefront are processed in order).
    if (ok && (peers >> lane) == 1ull) h[wave][e] += (int)__popcll(peers);
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  };
#pragma unroll
  for (int j = 0; j < kPlanHeld; ++j)
    if (b0 + 64 * j < b1) place(b0 + 64 * j + lane, held[j]);
  for (int s = b0 + 64 * kPlanHeld; s < b1; s += 64) place(s + lane, s + lane < b1 ? plan_bin(a, s + lane) : -1);
}

static int plan_chunk(int64_t R) {
  const int64_t unit = (int64_t)kPlanChunk * kPlanMaxChunks;
  return kPlanChunk * (int)((R + unit - 1) / unit);
}

size_t plan_scratch_bytes(int64_t R, int64_t G) {
  const int64_t n = R > 0 ? (R + plan_chunk(R) - 1) / plan_chunk(R) : 1;
  return n > 1 ? (size_t)n * (size_t)(G + 1) * sizeof(int32_t) : 0;
}

}  // namespace nvr

namespace {
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
}  // namespace

extern "C" int grouped_plan(const int32_t* topk_idx, int64_t T, int64_t k, int64_t first_expert, int64_t G,
                            int32_t* offsets, int32_t* rows, int32_t* pos, void* workspace, size_t workspace_bytes,
                            void* stream) {
  if (T < 0 || k < 1 || G < 1 || first_expert < 0 || T >= (int64_t(1) << 31)) return ROUTER_EINVAL;
  if (k > ROUTER_MAX_TOPK || G > ROUTER_MAX_EXPERTS || T * k >= (int64_t(1) << 30)) return ROUTER_EUNSUPPORTED;
  const int64_t R = T * k;
  if (!offsets || (R > 0 && (!topk_idx || !rows || !pos))) return ROUTER_EINVAL;
  if (!aligned(topk_idx, 4) || !aligned(offsets, 4) || !aligned(rows, 4) || !aligned(pos, 4)) return ROUTER_EINVAL;
  const size_t need = nvr::plan_scratch_bytes(R, G);
  if (need > 0 && (!workspace || workspace_bytes < nvr::kScratchOffset + need || !aligned(workspace, 256)))
    return ROUTER_EINVAL;
  int32_t* hist = need > 0 ? reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + nvr::kScratchOffset) : nullptr;
  const nvr::PlanArgs a{topk_idx, (int)R, (int)G, first_expert, offsets, rows, pos, hist, nvr::plan_chunk(R)};
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const int chunks = R > 0 ? (int)((R + a.chunk - 1) / a.chunk) : 1;
  if (chunks > 1) {
    nvr::plan_hist_kernel<<<chunks, nvr::kPlanThreads, 0, s>>>(a);
    if (hipGetLastError() != hipSuccess) return ROUTER_EHIP;
  }
  // Few slots: fewer wavefronts, whose counts are quicker to scan.
  if (R <= 256) nvr::plan_place_kernel<4><<<1, 256, 0, s>>>(a);
  else nvr::plan_place_kernel<16><<<chunks, 1024, 0, s>>>(a);
  return hipGetLastError() == hipSuccess ? ROUTER_OK : ROUTER_EHIP;
}
