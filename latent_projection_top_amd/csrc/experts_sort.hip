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
// Up to kOne choices, a round, are one block's work (16 choices of 896 experts: 3.3
// us; 1024: 4.9). More are dealt to up to kBlocks blocks, each of which has to know
// how many choices of each expert are in the blocks before it and in all (4096
// choices 6.0 us, in one block 8.7). Up to kRead choices every block counts them
// all for itself, in the same launch (32752 choices of 112 of 896 experts: 6.6 us,
// with a launch for the counts 8.1; 65536 of 896: 10.2 and 12.0; 131072: 17.0 and
// 14.8). Of more, a first launch counts each block's, and in the second every block
// adds up what the others have (262144: 17.3 us, with twice the blocks 21.5; 2^20:
// 42 and 33, so it has them there).
#include "block_device.h"
#include "experts_launch.h"

namespace experts {

using block::kWave;

constexpr int kThreads = 1024, kWaves = kThreads / kWave;
constexpr int kOne = kThreads, kRead = 64 * kThreads;
constexpr int kBlocks = 128, kSome = 64, kMany = 512 * kThreads;  // kSome blocks up to kMany choices
enum Counts { kOwn, kAll, kListed, kLonger };  // of its own choices, of all, listed for kSome or kBlocks blocks

// An id counted from `first`, in unsigned arithmetic: below `experts` if it is one
// of them. (Negative ids are all one: -1 - first is never small.)
__device__ __forceinline__ uint32_t local(const SortArgs& p, int id) {
  return (uint32_t)max(id, -1) - (uint32_t)p.first;
}
struct __attribute__((packed, aligned(4))) Four { block::u32x4 v; };  // of ids, at any of them

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
    const uint32_t e = local(p, p.ids[c]);
    if (e < (uint32_t)p.experts) atomicAdd(&count[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.experts; e += kThreads) hist[blockIdx.x * p.experts + e] = count[e];
}

// Most: the experts there is room for. Per: choices of a lane in a round (of many
// rounds four: 262144 choices 17.3 us, with one 20). kOwn: one block, one round.
template <int Most, int Per, Counts From>
__global__ __launch_bounds__(kThreads) void place_kernel(SortArgs p, const int* hist) {
  constexpr int kMine = Most / kThreads;  // experts of a thread: kMine t ..
  __shared__ __attribute__((aligned(16))) uint16_t seen[kWaves][Most];  // by wave, then the sum of earlier waves'
  __shared__ int start[Most];
  __shared__ int part[kWaves];
  constexpr bool Alone = From == kOwn;
  const int t = threadIdx.x, wave = t / kWave, lane = t & (kWave - 1);
  const int64_t chunk = Alone ? Per * kThreads : chunk_of(p, gridDim.x), c0 = blockIdx.x * chunk;
  const int64_t c1 = min((int64_t)p.choices, c0 + chunk);
  const int bits = 32 - __builtin_clz(p.experts);  // experts itself stands for none
  // waves that have any choice
  const int waves = Alone ? (p.choices + Per * kWave - 1) / (Per * kWave) : kWaves;

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
  if constexpr (From == kAll) {
    // `start` counts what is before this block, `after` the rest
    int* after = reinterpret_cast<int*>(seen);
    for (int e = t; e < p.experts; e += kThreads) start[e] = after[e] = 0;
    __syncthreads();
    // (c0 is a multiple of four; a thread has four groups of four at once)
    constexpr int kAtOnce = 4;
    const int groups = p.choices / 4;
    auto count = [&](int* to, int id) __attribute__((always_inline)) {
      const uint32_t e = local(p, id);
      if (e < (uint32_t)p.experts) atomicAdd(to + e, 1);
    };
#pragma unroll 1
    for (int g = t; g < groups; g += kAtOnce * kThreads) {
      block::u32x4 ids[kAtOnce];
#pragma unroll
      for (int q = 0; q < kAtOnce; ++q)
        ids[q] = reinterpret_cast<const Four*>(p.ids + 4 * min(g + q * kThreads, groups - 1))->v;
#pragma unroll
      for (int q = 0; q < kAtOnce; ++q)
        if (g + q * kThreads < groups) {
          int* to = 4 * (g + q * kThreads) < c0 ? start : after;
#pragma unroll
          for (int f = 0; f < 4; ++f) count(to, (int)ids[q][f]);
        }
    }
    if (4 * groups + t < p.choices) count(4 * groups + t < c0 ? start : after, p.ids[4 * groups + t]);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int e = kMine * t + i;
      before[i] = e < p.experts ? start[e] : 0;
      mine[i] = e < p.experts ? before[i] + after[e] : 0;
    }
    scan();
  } else if constexpr (From == kListed || From == kLonger) {
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int e = min(kMine * t + i, p.experts - 1);
#pragma unroll 1
      for (int g = 0; g < (From == kListed ? kSome : (int)gridDim.x); g += kSome) {
        int n[kSome];
#pragma unroll
        for (int b = 0; b < kSome; ++b) n[b] = hist[min(g + b, (int)gridDim.x - 1) * p.experts + e];
        // (which blocks there are, and come before, is the same for all lanes)
#pragma unroll
        for (int b = 0; b < kSome; ++b)
          if (g + b < (int)blockIdx.x)
            before[i] += n[b];
          else if (g + b < (int)gridDim.x)
            mine[i] += n[b];
      }
      mine[i] = kMine * t + i < p.experts ? mine[i] + before[i] : 0;
    }
    scan();
  }
  if constexpr (From == kAll) __syncthreads();  // `after` is read
  for (int i = t; i < waves * Most / 2; i += kThreads) reinterpret_cast<uint32_t*>(seen)[i] = 0;
  __syncthreads();
#pragma unroll 1
  for (int64_t r = c0; r < c1; r += Per * kThreads) {
    int e[Per], rank[Per];
#pragma unroll
    for (int i = 0; i < Per; ++i) {
      const int64_t c = r + (wave * Per + i) * kWave + lane;
      e[i] = c < c1 ? (int)min(local(p, p.ids[c]), (uint32_t)p.experts) : p.experts;
    }
#pragma unroll
    for (int i = 0; i < Per; ++i) {
      uint64_t other = 0;  // lanes whose number has another bit somewhere
      for (int b = 0; b < bits; ++b) {
        const uint64_t set = __ballot((e[i] >> b) & 1);
        const uint32_t mine = (uint32_t)-((e[i] >> b) & 1);
        other |= set ^ (uint64_t)mine << 32 ^ mine;
      }
      const uint64_t same = ~other;
      const int below = __popcll(same & ((1ull << lane) - 1));
      rank[i] = e[i] < p.experts ? seen[wave][e[i]] + below : 0;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      // the last of them counts for all
      if (e[i] < p.experts && (same >> lane) == 1) seen[wave][e[i]] = (uint16_t)(rank[i] + 1);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
    __syncthreads();
    // each wave's count becomes the sum of the earlier waves'
    int total[kMine];
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int x = kMine * t + i;
      int sum = 0, v[kWaves];
      if (x < p.experts) {
#pragma unroll
        for (int w = 0; w < kWaves; ++w) v[w] = w < waves ? seen[w][x] : 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          if (w < waves) seen[w][x] = (uint16_t)sum;
          sum += v[w];
        }
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
      const int at = e[i] < p.experts ? start[e[i]] + seen[wave][e[i]] + rank[i] : -1;
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
  const int64_t most = choices <= kMany ? kSome : kBlocks, rounds = (choices + kThreads - 1) / kThreads;
  return (int)(rounds < most ? rounds : most);
}

size_t sort_workspace_bytes(int64_t choices, int experts) {
  return choices <= kRead ? 0 : (size_t)kBlocks * experts * sizeof(int);
}

template <int Most>
static hipError_t launch_most(const SortArgs& p, hipStream_t stream) {
  int* hist = static_cast<int*>(p.workspace);
  const dim3 blocks(p.choices <= kOne ? 1 : blocks_for(p.choices)), threads(kThreads);
  if (p.choices <= kOne)
    return launch_kernel(place_kernel<Most, 1, kOwn>, blocks, threads, stream, p, nullptr);
  if (p.choices <= kRead) return launch_kernel(place_kernel<Most, 1, kAll>, blocks, threads, stream, p, nullptr);
  const hipError_t e = launch_kernel(count_kernel<Most>, blocks, threads, stream, p, hist);
  if (e != hipSuccess) return e;
  return launch_kernel(blocks.x <= kSome ? place_kernel<Most, 4, kListed> : place_kernel<Most, 4, kLonger>, blocks,
                       threads, stream, p, hist);
}

hipError_t launch_sort(const SortArgs& p, hipStream_t stream) {
  return p.experts <= 1024 ? launch_most<1024>(p, stream) : launch_most<4096>(p, stream);
}

}  // namespace experts
