// Choices sorted by expert: a stable counting sort of at most 2^24 small
// integers.
#include "block_device.h"
#include "experts_launch.h"

namespace experts {

using block::kWave;

constexpr int kThreads = 1024;

// The expert of choice c counted from `first`, or -1.
__device__ __forceinline__ int local(const SortArgs& p, int c) {
  const uint32_t e = (uint32_t)p.ids[c] - (uint32_t)p.first;
  return p.ids[c] >= p.first && e < (uint32_t)p.experts ? (int)e : -1;
}

// One block: counts in LDS, their prefix sums, then one wave takes 64 choices
// after another to their places.
__global__ __launch_bounds__(kThreads) void sort_kernel(SortArgs p) {
  __shared__ int count[EXPERTS_MAX_COUNT];
  __shared__ int part[kThreads];
  const int t = threadIdx.x;
  for (int e = t; e < p.experts; e += kThreads) count[e] = 0;
  __syncthreads();
  for (int c = t; c < p.choices; c += kThreads) {
    const int e = local(p, c);
    if (e >= 0) atomicAdd(&count[e], 1);
  }
  __syncthreads();
  // thread t has experts 4 t .. 4 t + 3
  int mine[EXPERTS_MAX_COUNT / kThreads], sum = 0;
  for (int i = 0; i < EXPERTS_MAX_COUNT / kThreads; ++i) {
    const int e = EXPERTS_MAX_COUNT / kThreads * t + i;
    mine[i] = sum;
    sum += e < p.experts ? count[e] : 0;
  }
  part[t] = sum;
  __syncthreads();
  for (int d = 1; d < kThreads; d *= 2) {
    const int v = t >= d ? part[t - d] : 0;
    __syncthreads();
    part[t] += v;
    __syncthreads();
  }
  for (int i = 0; i < EXPERTS_MAX_COUNT / kThreads; ++i) {
    const int e = EXPERTS_MAX_COUNT / kThreads * t + i;
    if (e < p.experts) p.offsets[e] = count[e] = part[t] - sum + mine[i];
  }
  if (t == kThreads - 1) p.offsets[p.experts] = part[t];
  __syncthreads();
  if (t >= kWave) return;
  for (int c0 = 0; c0 < p.choices; c0 += kWave) {
    const int c = c0 + t;
    const int e = c < p.choices ? local(p, c) : -1;
    // lanes of the same expert
    uint64_t same = __ballot(e >= 0);
    for (int b = 0; b < 12; ++b) {
      const uint64_t set = __ballot((e >> b) & 1);
      same &= (e >> b) & 1 ? set : ~set;
    }
    int at = -1;
    if (e >= 0) at = count[e] + __popcll(same & ((1ull << t) - 1));
    __builtin_amdgcn_wave_barrier();
    if (e >= 0 && (same >> t) == 1) count[e] = at + 1;  // the last of them
    __builtin_amdgcn_wave_barrier();
    if (c < p.choices) p.place[c] = at;
    if (e >= 0 && at < p.capacity) p.token[at] = c / p.topk;
  }
}

size_t sort_workspace_bytes(int64_t, int) { return 256; }

hipError_t launch_sort(const SortArgs& p, hipStream_t stream) {
  return launch_kernel(sort_kernel, dim3(1), dim3(kThreads), stream, p);
}

}  // namespace experts
