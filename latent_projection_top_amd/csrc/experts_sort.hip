// Choices sorted by expert: a stable counting sort of up to 2^24 small
// integers, bound by the latency of its few dependent steps.
//
// A block of 16 waves takes choices in rounds, each wave a contiguous run of
// them, 64 at a time. The lanes of a wave that have the same expert find each
// other by ballots over the bits of its number; the place of a choice is then
// the expert's start, what earlier rounds, waves and groups of the wave have of
// it, and its rank among those lanes. That needs each wave's count of each
// expert, which LDS holds in 16 bits. Nothing depends on the order of atomics.
//
// Up to kOne choices are one block's work in one launch. More are dealt to up
// to kBlocks blocks: a first launch counts each block's choices by expert, in
// the second every block adds up what the others have (64 x 896 counts, read
// from L2 by all of them) instead of a launch of its own for that.
#include "block_device.h"
#include "experts_launch.h"

namespace experts {

using block::kWave;

constexpr int kThreads = 1024, kWaves = kThreads / kWave;
constexpr int kOne = 4 * kThreads;
constexpr int kBlocks = 64;

// The expert of choice c counted from `first`, or -1.
__device__ __forceinline__ int local(const SortArgs& p, int c) {
  const int id = p.ids[c];
  const uint32_t e = (uint32_t)id - (uint32_t)p.first;
  return id >= p.first && e < (uint32_t)p.experts ? (int)e : -1;
}

// The choices of block b: whole rounds of kThreads.
__device__ __forceinline__ int64_t chunk_of(const SortArgs& p, int blocks) {
  return ((int64_t)(p.choices + blocks - 1) / blocks + kThreads - 1) / kThreads * kThreads;
}

template <int Most>
__global__ __launch_bounds__(kThreads) void count_kernel(SortArgs p, int* hist) {
  __shared__ int count[Most];
  for (int e = threadIdx.x; e < p.experts; e += kThreads) count[e] = 0;
  __syncthreads();
  const int64_t chunk = chunk_of(p, gridDim.x), c0 = blockIdx.x * chunk;
  const int c1 = (int)min((int64_t)p.choices, c0 + chunk);
  for (int64_t c = c0 + threadIdx.x; c < c1; c += kThreads) {
    const int e = local(p, (int)c);
    if (e >= 0) atomicAdd(&count[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.experts; e += kThreads) hist[(int64_t)blockIdx.x * p.experts + e] = count[e];
}

// Most: the experts there is room for. Per: choices of a lane in a round.
// Alone: one block, one round, no counts from a launch before.
template <int Most, int Per, bool Alone>
__global__ __launch_bounds__(kThreads) void place_kernel(SortArgs p, const int* hist) {
  constexpr int kMine = Most / kThreads;  // experts of a thread: kMine t ..
  __shared__ uint16_t seen[kWaves][Most];  // by wave, then the sum of earlier waves'
  __shared__ int start[Most];
  __shared__ int part[kWaves];
  const int t = threadIdx.x, wave = t / kWave, lane = t & (kWave - 1);
  const int64_t chunk = Alone ? Per * kThreads : chunk_of(p, gridDim.x), c0 = blockIdx.x * chunk;
  const int64_t c1 = min((int64_t)p.choices, c0 + chunk);
  const int bits = 32 - __builtin_clz(p.experts);  // experts itself stands for none
  // waves that have any choice
  const int waves = Alone ? (p.choices + Per * kWave - 1) / (Per * kWave) : kWaves;

  for (int i = t; i < waves * Most / 2; i += kThreads) reinterpret_cast<uint32_t*>(seen)[i] = 0;
  int mine[kMine], before[kMine];
#pragma unroll
  for (int i = 0; i < kMine; ++i) mine[i] = before[i] = 0;
  // starts of the thread's experts from their counts: a prefix sum over the block
  auto scan = [&]() __attribute__((always_inline)) {
    int sum = 0;
#pragma unroll
    for (int i = 0; i < kMine; ++i) sum += mine[i];
    int run = sum;
    for (int d = 1; d < kWave; d *= 2) {
      const int v = __shfl_up(run, d);
      run += lane >= d ? v : 0;
    }
    if (lane == kWave - 1) part[wave] = run;
    __syncthreads();
    int base = run - sum;
    for (int w = 0; w < kWaves; ++w) base += w < wave ? part[w] : 0;
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int e = kMine * t + i;
      if (e < p.experts) {
        if (blockIdx.x == 0) p.offsets[e] = base;
        start[e] = base + before[i];
      }
      base += mine[i];
    }
    if (blockIdx.x == 0 && t == kThreads - 1) p.offsets[p.experts] = base;
  };
  if constexpr (!Alone) {
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int e = min(kMine * t + i, p.experts - 1);
      const bool in = kMine * t + i < p.experts;
      for (int b0 = 0; b0 < (int)gridDim.x; b0 += 32) {
        int n[32];
#pragma unroll
        for (int q = 0; q < 32; ++q) n[q] = hist[(int64_t)min(b0 + q, (int)gridDim.x - 1) * p.experts + e];
#pragma unroll
        for (int q = 0; q < 32; ++q) {
          const int v = in && b0 + q < (int)gridDim.x ? n[q] : 0;
          mine[i] += v;
          before[i] += b0 + q < (int)blockIdx.x ? v : 0;
        }
      }
    }
    scan();
  }
  __syncthreads();
#pragma unroll 1
  for (int64_t r = c0; r < c1; r += Per * kThreads) {
    int e[Per], rank[Per];
#pragma unroll
    for (int i = 0; i < Per; ++i) {
      const int64_t c = r + (wave * Per + i) * kWave + lane;
      e[i] = c < c1 ? local(p, (int)c) : -1;
    }
#pragma unroll
    for (int i = 0; i < Per; ++i) {
      const int key = e[i] < 0 ? p.experts : e[i];
      uint64_t same = ~0ull;
      for (int b = 0; b < bits; ++b) {
        const uint64_t set = __ballot((key >> b) & 1);
        same &= (key >> b) & 1 ? set : ~set;
      }
      const int below = __popcll(same & ((1ull << lane) - 1));
      rank[i] = e[i] >= 0 ? seen[wave][e[i]] + below : 0;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      // the last of them counts for all
      if (e[i] >= 0 && (same >> lane) == 1) seen[wave][e[i]] = (uint16_t)(rank[i] + 1);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
    __syncthreads();
    // each wave's count becomes the sum of the earlier waves'
    int total[kMine];
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int x = kMine * t + i;
      int sum = 0;
      if (x < p.experts)
        for (int w = 0; w < waves; ++w) {
          const int v = seen[w][x];
          seen[w][x] = (uint16_t)sum;
          sum += v;
        }
      total[i] = sum;
    }
    if constexpr (Alone) {
#pragma unroll
      for (int i = 0; i < kMine; ++i) mine[i] = total[i];
      scan();
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < Per; ++i) {
      const int64_t c = r + (wave * Per + i) * kWave + lane;
      if (c >= c1) continue;
      const int at = e[i] >= 0 ? start[e[i]] + seen[wave][e[i]] + rank[i] : -1;
      p.place[c] = at;
      if (at >= 0 && at < p.capacity) p.token[at] = (int)((uint32_t)c / (uint32_t)p.topk);
    }
    if constexpr (!Alone) {
      if (r + Per * kThreads >= c1) break;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int x = kMine * t + i;
        if (x < p.experts) {
          start[x] += total[i];
          for (int w = 0; w < kWaves; ++w) seen[w][x] = 0;
        }
      }
      __syncthreads();
    }
  }
  if constexpr (Alone) {
    if (p.choices == 0) scan();
  }
}

static int blocks_for(int64_t choices) {
  return (int)((choices + kThreads - 1) / kThreads < kBlocks ? (choices + kThreads - 1) / kThreads : kBlocks);
}

size_t sort_workspace_bytes(int64_t choices, int experts) {
  return choices <= kOne ? 0 : (size_t)kBlocks * experts * sizeof(int);
}

template <int Most>
static hipError_t launch_most(const SortArgs& p, hipStream_t stream) {
  int* hist = static_cast<int*>(p.workspace);
  const dim3 one(1), threads(kThreads);
  if (p.choices <= kOne)
    return launch_kernel(p.choices <= kThreads ? place_kernel<Most, 1, true> : place_kernel<Most, 4, true>, one,
                         threads, stream, p, nullptr);
  const dim3 blocks(blocks_for(p.choices));
  const hipError_t e = launch_kernel(count_kernel<Most>, blocks, threads, stream, p, hist);
  if (e != hipSuccess) return e;
  const bool many = p.choices > (int64_t)kBlocks * 2 * kThreads;
  return launch_kernel(many ? place_kernel<Most, 4, false> : place_kernel<Most, 1, false>, blocks, threads, stream, p,
                       hist);
}

hipError_t launch_sort(const SortArgs& p, hipStream_t stream) {
  return p.experts <= 1024 ? launch_most<1024>(p, stream) : launch_most<4096>(p, stream);
}

}  // namespace experts
