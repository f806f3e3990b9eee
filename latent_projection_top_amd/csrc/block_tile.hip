// Matrix products of the layer's operators: the tile kernel, for row counts
// that make the matrix cores, not the weights' bandwidth, the bound.
//
// C[m][n] = sum over r of A(m, r) B(r, n) on v_mfma_f32_16x16x32, one FP32
// accumulator per output from the first r to the last. A 256 x 256 tile has
// eight waves of 128 x 64 outputs in 128 accumulator registers each: two
// waves per SIMD, so that one's LDS reads and barrier run under the other's
// MFMAs, and 12 operand reads for 32 MFMAs, so that LDS, written by the loads
// and read by eight waves, is busy a third of the time. The reduction runs in
// stages of 32 through five LDS buffers (160 KB): one being multiplied, one
// being read into registers, three on their way from memory, which gives a
// load about three stages (2 us) to arrive. One tile per CU at a time.
//   4096 x 4096 x 4096: 103-112 us (1220-1330 TFLOP/s), matrix cores busy
//   0.71-0.77 of the cycles at 1.9-2.1 GHz; 4096 x 3584 x 8192: 172-177 us
//   (1360-1400). The rest is the barrier of every stage and the ends of a
//   tile, which nothing overlaps.
#include "block_device.h"

#include <algorithm>

namespace block {

typedef __attribute__((address_space(3))) void lds_void;

constexpr int kStep = 32;    // reduction per stage: one MFMA deep
constexpr int kStages = 5;   // LDS buffers

template <int BMr, int BNr, int WMr, int WNr>
struct TileShape {
  static constexpr int BM = BMr, BN = BNr, WM = WMr, WN = WNr;
  static constexpr int NW = WM * WN;
  static constexpr int MT = BM / WM / 16, NT = BN / WN / 16;  // 16 x 16 tiles of a wave
  static constexpr int A_BYTES = BM * kStep * 2, B_BYTES = BN * kStep * 2;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int A_PER = BM / 16 / NW, B_PER = BN / 16 / NW;  // 1 KB loads of a wave per stage
  static constexpr int PER = A_PER + B_PER;
  static_assert(A_PER >= 1 && B_PER >= 1 && NT % 2 == 0 && MT % 2 == 0, "");
  static_assert(kStages * STAGE <= 160 * 1024, "LDS");
};

// 16 bytes that lanes outside the reduction's range load.
__device__ __attribute__((aligned(16))) const uint32_t kZeros[4] = {0, 0, 0, 0};

// Global -> LDS, 16 bytes per lane: lane l's bytes land at lds + 16 l. Inline
// assembly, so that the compiler does not wait for every load in flight
// before each LDS read (it cannot tell the stages apart); the kernel's own
// vmcnt waits order them, and the volatile barriers below keep the LDS reads
// on their side.
__device__ __forceinline__ void dma16(const char* base, uint32_t off, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" : : "v"(off), "s"(base), "{m0}"(lds));
}
__device__ __forceinline__ void dma16(const char* addr, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off" : : "v"(addr), "{m0}"(lds));
}

__device__ __forceinline__ u32x4 lds_b128(uint32_t addr) {
  return *(const __attribute__((address_space(3))) u32x4*)(uintptr_t)addr;
}
__device__ __forceinline__ u32x2 lds_tr16(uint32_t addr) {
  return __builtin_bit_cast(
      u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(uintptr_t)addr));
}

// Wait until at most Vm of this wave's loads are in flight and at most Lgkm
// LDS reads are outstanding, then meet the block.
template <int Vm, int Lgkm>
__device__ __forceinline__ void wait_barrier() {
  static_assert(Vm >= 0 && Vm < 64 && Lgkm >= 0 && Lgkm < 16, "counter range");
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(%1)\n\ts_barrier" : : "n"(Vm), "n"(Lgkm) : "memory");
}

// An operand's tile of `Rows` rows (or columns) by 32 of the reduction, and
// how it lies in a stage.
//   RContig (the reduction is contiguous in memory): 64-byte rows; the
//     16-byte piece c of row r sits at position c ^ swizzle(r >> 2). Read with
//     ds_read_b128, which serves the lanes 0-3, 12-15, 20-27 at once, then
//     4-11, 16-19, 28-31, and likewise the upper half: with the swizzle 0, 2,
//     3, 1 each of these sixteen takes another 16-byte column of the 64 banks
//     (with 0, 1, 2, 3 every read met a two-way conflict).
//   otherwise (rows contiguous): blocks of [32 r][32 rows], 64-byte lines,
//     whose two halves are swapped where bit 3 of r is set. The MFMA wants 8
//     consecutive r of one row per lane, which ds_read_tr16_b64 delivers.
__device__ __forceinline__ int swizzle(int r4) { return ((r4 ^ (r4 >> 1)) & 1) << 1 | ((r4 >> 1) & 1); }

template <bool RContig>
struct Operand {
  // this lane's source of load `c` (1 KB): row within the tile and r within
  // the stage of its first element
  static __device__ __forceinline__ int row(int c, int lane) {
    if constexpr (RContig) return 16 * c + (lane >> 2);
    return 32 * (c >> 1) + 8 * ((lane & 3) ^ ((lane >> 5) << 1));
  }
  static __device__ __forceinline__ int red(int c, int lane) {
    if constexpr (RContig) return 8 * ((lane & 3) ^ swizzle(lane >> 4));
    return 16 * (c & 1) + (lane >> 2);
  }
  // addresses of this lane's part of a 16-row fragment: rows 16 t, t even
  // (h = 0) or odd (h = 1), relative to the even tile
  static __device__ __forceinline__ uint32_t base(int lane, int h) {
    const int g = lane >> 4, m = lane & 15;
    if constexpr (RContig) return (uint32_t)((16 * h + m) * 64 + ((g ^ swizzle(m >> 2)) * 16));
    return (uint32_t)((8 * g + (m >> 2)) * 64 + (2 * (h ^ (g & 1)) + ((m & 3) >> 1)) * 16 + (m & 1) * 8);
  }
  static constexpr int kReads = RContig ? 1 : 2;  // LDS reads per fragment
  static __device__ __forceinline__ u32x4 read(uint32_t addr) {
    if constexpr (RContig) return lds_b128(addr);
    const u32x2 lo = lds_tr16(addr), hi = lds_tr16(addr + 4 * 64);
    return u32x4{lo[0], lo[1], hi[0], hi[1]};
  }
  // bytes from one pair of 16-row fragments to the next: the same in both
  static constexpr int kPair = 2048;
};

template <typename T, int Mode, typename S>
__global__ __launch_bounds__(64 * S::NW) __attribute__((amdgpu_waves_per_eu(2, 2)))
void gemm_tile_kernel(GemmArgs p, int mtiles, int ntiles, int splits, float* partial) {
  typedef Operand<Mode != kDw> A;
  typedef Operand<Mode == kDx> B;
  constexpr int kCols = Mode == kGated ? S::BN / 2 : S::BN;  // output columns of a tile
  __shared__ __attribute__((aligned(1024))) char smem[kStages * S::STAGE];

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  const int g = lane >> 4, m = lane & 15;
  const int wm = wave / S::WN, wn = wave % S::WN;

  // Blocks are dealt round-robin over the 8 XCDs: renumber them so that each
  // XCD has a contiguous range of tiles, and walk the range in groups of 8
  // row tiles, column by column, so that one XCD's L2 holds few A and B tiles
  // at a time (1100 rows of gated 3584 x 3600: 83.5 us without, 72.5 with;
  // 333 rows, dx of 3584 x 4224: 28.1 and 23.8). The
  // first total % 8 XCDs have one more.
  const int total = mtiles * ntiles * p.outputs;
  const int split = blockIdx.x / total;
  int lin = blockIdx.x - split * total;
  lin = (lin & 7) * (total >> 3) + min(lin & 7, total & 7) + (lin >> 3);
  const int cols_all = ntiles * p.outputs;
  const int group = lin / (8 * cols_all);
  const int gm = min(mtiles - 8 * group, 8);
  const int loc = lin - group * 8 * cols_all;
  const int64_t row0 = (int64_t)(8 * group + loc % gm) * S::BM;
  const int ct = loc / gm;
  const int which = ct / ntiles;
  const int col0 = (ct - which * ntiles) * kCols;

  const int per_seg = (int)((p.red + kStep - 1) / kStep);
  const int all = per_seg * p.segments;
  const int s0 = (int)((int64_t)all * split / splits);
  const int s1 = (int)((int64_t)all * (split + 1) / splits);
  const int red = (int)p.red;
  const bool ragged = (red & (kStep - 1)) != 0;

  // ---- global -> LDS -------------------------------------------------------
  // Rows past the matrix's end repeat its last one and columns its last eight
  // (their sums are not stored); past the reduction's end lanes load zeros.
  // off: this lane's byte offset of each of the wave's loads from the stage's
  // first byte of its matrix (a wave's loads of B are all of one matrix).
  // Contiguous lengths that are no multiple of 8 are padded to one in memory.
  const int64_t m8 = (p.m + 7) & ~7, n8 = (p.n + 7) & ~7;
  uint32_t off[S::PER];
  int red_of[S::PER];
  auto b_row = [&](int c) {
    const int r = B::row(c, lane);
    // gated: 32-column blocks alternate between the two matrices
    return Mode == kGated ? 32 * (r >> 6) + (r & 31) : r;
  };
#pragma unroll
  for (int i = 0; i < S::PER; ++i) {
    const bool is_a = i < S::A_PER;
    const int c = wave + S::NW * (is_a ? i : i - S::A_PER);
    const int r = is_a ? A::row(c, lane) : b_row(c);
    const int k = is_a ? A::red(c, lane) : B::red(c, lane);
    red_of[i] = k;
    if (is_a)
      off[i] = Mode != kDw ? (uint32_t)((min(row0 + r, p.m - 1) - row0) * p.lda + k) * 2u
                           : (uint32_t)(k * p.lda + min(row0 + r, m8 - 8)) * 2u;
    else
      off[i] = Mode == kDx ? (uint32_t)((min(col0 + r, p.n - 1) - col0) * p.ldb + k) * 2u
                           : (uint32_t)(k * p.ldb + min(col0 + r, (int)n8 - 8)) * 2u;
  }
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_void*)smem;
  // the matrices at stage 0 of each segment, and from one stage to the next
  const int bm = Mode == kGated ? (wave >> 1) & 1 : Mode == kDx ? 0 : which;
  const uintptr_t a_at = Mode != kDw ? row0 * p.lda * 2 : 0, b_at = Mode == kDx ? (int64_t)col0 * p.ldb * 2 : 0;
  const uintptr_t a_seg[2] = {reinterpret_cast<uintptr_t>(p.a[0]) + a_at, reinterpret_cast<uintptr_t>(p.a[1]) + a_at};
  const uintptr_t b_seg[2] = {reinterpret_cast<uintptr_t>(p.b[bm]) + b_at, reinterpret_cast<uintptr_t>(p.b[1]) + b_at};
  const int64_t a_step = kStep * 2 * (Mode != kDw ? 1 : p.lda), b_step = kStep * 2 * (Mode == kDx ? 1 : p.ldb);
  auto base_of = [&](bool is_a, int s) __attribute__((always_inline)) -> uintptr_t {
    const bool second = s >= per_seg;
    const int64_t ks = second ? s - per_seg : s;
    return is_a ? (second ? a_seg[1] : a_seg[0]) + ks * a_step : (second ? b_seg[1] : b_seg[0]) + ks * b_step;
  };
  auto slot = [&](int i) __attribute__((always_inline)) -> uint32_t {  // of load i in a stage
    const bool is_a = i < S::A_PER;
    return (is_a ? 0 : S::A_BYTES) + (wave + S::NW * (is_a ? i : i - S::A_PER)) * 1024;
  };

  // Any stage; the last of a segment may be short.
  auto issue_any = [&](int s, uint32_t buf, int i) __attribute__((always_inline)) {
    const int ks = s >= per_seg ? s - per_seg : s;
    const char* base = reinterpret_cast<const char*>(base_of(i < S::A_PER, s));
    if (ragged && ks == per_seg - 1) {
      const bool in = ks * kStep + red_of[i] < red;
      dma16(in ? base + off[i] : reinterpret_cast<const char*>(kZeros), buf + slot(i));
    } else {
      dma16(base, off[i], buf + slot(i));
    }
  };

  // ---- LDS -> registers ----------------------------------------------------
  uint32_t a_rd[2], b_rd[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    a_rd[h] = A::base(lane, h) + wm * (S::MT / 2) * A::kPair;
    b_rd[h] = B::base(lane, h) + S::A_BYTES + wn * (S::NT / 2) * B::kPair;
  }
  auto read_a = [&](uint32_t buf, int i) { return A::read(buf + a_rd[i & 1] + (i >> 1) * A::kPair); };
  auto read_b = [&](uint32_t buf, int j) { return B::read(buf + b_rd[j & 1] + (j >> 1) * B::kPair); };
  constexpr int kReads = S::MT * A::kReads + S::NT * B::kReads;  // per stage and wave

  f32x4 acc[S::MT][S::NT] = {};
  u32x4 a[S::MT], b0[S::NT], b1[S::NT];

  // Stage s's MFMAs. Meanwhile the operands of stage s + 1 are read (a[i] as
  // soon as its last MFMA is issued, B into the other register set) and this
  // wave's loads of stage s + 4 go out, load(n) the n-th of them, into the
  // buffer of stage s - 1, which the barrier before this step has freed.
  auto step = [&](u32x4(&b)[S::NT], u32x4(&bn)[S::NT], uint32_t next, auto load) __attribute__((always_inline)) {
    constexpr int kEvery = S::MT * S::NT / S::PER;
#pragma unroll
    for (int i = 0; i < S::MT; ++i) {
#pragma unroll
      for (int j = 0; j < S::NT; ++j) {
        const int n = i * S::NT + j;
        if (n % kEvery == kEvery / 2) load(n / kEvery);
        acc[i][j] = T::mfma(b[j], a[i], acc[i][j]);
      }
      if (i < S::NT) bn[i] = read_b(next, i);
      a[i] = read_a(next, i);
    }
  };
  static_assert(S::MT >= S::NT, "every B operand is read");
  // At the end of stage s: stage s + 2 has to be in LDS (at most the loads of
  // the stages after it still in flight), and every read of stage s's buffer
  // has to have returned (at most the reads of stage s + 1 outstanding).
  constexpr int kLgkm = kReads < 15 ? kReads : 15;

  // Each wave turns its sums around in LDS (its own part, so only the first
  // use waits for the block), 16 * kRows rows at a time, so that a lane ends
  // eight columns of a row at once: 16-byte accesses to every matrix, whole
  // lines per row, and the activation's code is there once per turn instead
  // of once per MFMA tile (32 copies cost the 256 x 256 kernel a fifth of
  // its time in instruction fetches).
  constexpr int kPitch = 16 * S::NT + 4;
  constexpr int kRows = S::NW * 64 * kPitch * 4 <= kStages * S::STAGE ? 4 : 2;
  static_assert(S::NW * 16 * kRows * kPitch * 4 <= kStages * S::STAGE && S::MT % kRows == 0, "LDS");
  constexpr int kWide = Mode == kGated ? 8 * S::NT : 16 * S::NT;  // output columns of a wave
  constexpr int kLanes = kWide / 8;                               // lanes of a row
  constexpr int kStepRows = 64 / kLanes;                          // rows of a wave at once
  constexpr int kSteps = 16 * kRows / kStepRows, kGroup = kSteps < 4 ? kSteps : 4;
  float* turn = reinterpret_cast<float*>(smem) + wave * 16 * kRows * kPitch;
  const int64_t wrow = row0 + 16 * S::MT * wm + lane / kLanes;
  const int wcol = 8 * (lane % kLanes), col = col0 + kWide * wn + wcol;
  float bias[8] = {};
  if (Mode == kLinear && p.bias != nullptr && col < p.n)
    load_cols<T, 8>(static_cast<const typename T::raw*>(p.bias) + col, bias, p.n - col);
  // The residual's loads are a group of steps ahead of their use: read where
  // it is used, each of them would cost the wave a trip to HBM (17 us of a
  // 2048 x 3584 -> 7168 product).
  const bool add = Mode == kLinear && p.residual != nullptr;
  u32x4 res[kGroup], ahead[kGroup];
  auto fetch = [&](u32x4(&d)[kGroup], int64_t row) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < kGroup; ++q) {
      d[q] = u32x4{0, 0, 0, 0};
      const int64_t r = row + q * kStepRows;
      const uint16_t* src = static_cast<const uint16_t*>(p.residual) + r * p.ldr + col;
      if (r < p.m && col + 8 <= p.n) {
        d[q] = reinterpret_cast<const Any16*>(src)->v;
      } else if (r < p.m) {
#pragma unroll
        for (int t = 0; t < 7; ++t)
          if (col + t < p.n) d[q][t >> 1] |= (uint32_t)src[t] << (16 * (t & 1));
      }
    }
  };
  const int count = s1 - s0;
  if (count > 0) {
#pragma unroll 1
    for (int s = 0; s < min(count, 4); ++s)
#pragma unroll
      for (int i = 0; i < S::PER; ++i) issue_any(s0 + s, lds0 + s * S::STAGE, i);
    if (count >= 4)
      wait_barrier<2 * S::PER, 0>();
    else
      wait_barrier<0, 0>();
#pragma unroll
    for (int i = 0; i < S::MT; ++i) a[i] = read_a(lds0, i);
#pragma unroll
    for (int j = 0; j < S::NT; ++j) b0[j] = read_b(lds0, j);

    constexpr uint32_t kEnd = kStages * S::STAGE;
    uint32_t next = lds0 + S::STAGE, fill = lds0 + 4 * S::STAGE;  // buffers of stages s + 1 and s + 4
    auto advance = [&]() __attribute__((always_inline)) {
      next = next + S::STAGE == lds0 + kEnd ? lds0 : next + S::STAGE;
      fill = fill + S::STAGE == lds0 + kEnd ? lds0 : fill + S::STAGE;
    };
    // Steady state: the stages to load are whole and follow each other. Two
    // steps a turn, for the two B register sets.
    int s = 0;
    uintptr_t a_next = 0, b_next = 0;
    auto steady = [&](u32x4(&b)[S::NT], u32x4(&bn)[S::NT]) __attribute__((always_inline)) {
      auto load = [&](int n) __attribute__((always_inline)) {
        dma16(reinterpret_cast<const char*>(n < S::A_PER ? a_next : b_next), off[n], fill + slot(n));
      };
      step(b, bn, next, load);
      wait_barrier<2 * S::PER, kLgkm>();
      advance();
      a_next += a_step;
      b_next += b_step;
    };
    // Any step: the ends of the segments.
    auto other = [&](int q, u32x4(&b)[S::NT], u32x4(&bn)[S::NT]) __attribute__((always_inline)) {
      if (q >= count) return;
      const bool issue = q + 4 < count;
      auto load = [&](int n) __attribute__((always_inline)) {
        if (issue) issue_any(s0 + q + 4, fill, n);
      };
      step(b, bn, next, load);
      if (q + 2 < count) {
        if (q + 4 < count)
          wait_barrier<2 * S::PER, kLgkm>();
        else if (q + 3 < count)
          wait_barrier<S::PER, kLgkm>();
        else
          wait_barrier<0, kLgkm>();
      }
      advance();
    };
    auto whole_stages = [&]() __attribute__((always_inline)) {
      const int first = s0 + s + 4;  // the next stage to load
      const int limit = min(s1, (first >= per_seg ? 2 : 1) * per_seg - (ragged ? 1 : 0));
      a_next = base_of(true, first);
      b_next = base_of(false, first);
#pragma unroll 1
      for (int t = first; t + 2 <= limit; t += 2) {
        steady(b0, b1);
        steady(b1, b0);
        s += 2;
      }
    };
    auto other_stages = [&](int end) __attribute__((always_inline)) {
#pragma unroll 1
      for (; s < end; s += 2) {
        other(s, b0, b1);
        other(s + 1, b1, b0);
      }
    };
    whole_stages();
    if constexpr (Mode == kDx) {
      if (s0 < per_seg && s1 > per_seg) {  // over to the second segment
        other_stages(min(count, per_seg - s0 - 4));
        whole_stages();
      }
    }
    // the residual's first loads go out with the last stages still to do (they
    // only make the counted waits stricter)
    if (add && splits == 1) fetch(ahead, wrow);
    other_stages(count);
  } else if (add && splits == 1) {
    fetch(ahead, wrow);
  }

  // lane (g, m) of tile (i, j) holds row 16 i + m, columns 16 j + 4 g .. + 3
  const int64_t pn = (p.n + 3) & ~3;
  if (splits > 1) {
    const int planes = Mode == kGated ? 2 : p.outputs;
#pragma unroll
    for (int i = 0; i < S::MT; ++i) {
      const int64_t row = row0 + 16 * (S::MT * wm + i) + m;
      constexpr int kJ = Mode == kGated ? S::NT / 2 : S::NT;
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        const int col = col0 + 16 * (kJ * wn + j) + 4 * g;
        if (row < p.m && col < p.n) {
          float* d = partial + (((int64_t)split * planes + which) * p.m + row) * pn + col;
          *reinterpret_cast<f32x4*>(d) = acc[i][j];
          if (Mode == kGated) *reinterpret_cast<f32x4*>(d + p.m * pn) = acc[i][S::NT / 2 + j];
        }
      }
    }
    return;
  }
  __syncthreads();
#pragma unroll 1
  for (int c = 0; c < S::MT / kRows; ++c) {
    // (the sums' registers are known by number only: one branch per turn)
#pragma unroll
    for (int cc = 0; cc < S::MT / kRows; ++cc)
      if (c == cc)
#pragma unroll
        for (int i = 0; i < kRows; ++i)
#pragma unroll
          for (int j = 0; j < S::NT; ++j)
            *reinterpret_cast<f32x4*>(turn + (16 * i + m) * kPitch + 16 * j + 4 * g) = acc[kRows * cc + i][j];
    __builtin_amdgcn_wave_barrier();
    with_ending<Mode>(p, [&](auto act, auto save) __attribute__((always_inline)) {
#pragma unroll 1
      for (int k = 0; k < kSteps; k += kGroup) {
        const int64_t row = wrow + 16 * kRows * c + k * kStepRows;
        if (add) {
#pragma unroll
          for (int q = 0; q < kGroup; ++q) res[q] = ahead[q];
          fetch(ahead, row + kGroup * kStepRows);
        }
#pragma unroll
        for (int q = 0; q < kGroup; ++q) {
          const float* t = turn + ((k + q) * kStepRows + lane / kLanes) * kPitch + wcol;
          float v[8], u[8], r[8];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const f32x4 x = *reinterpret_cast<const f32x4*>(t + 4 * h);
            const f32x4 y = *reinterpret_cast<const f32x4*>(t + 4 * h + (Mode == kGated ? 8 * S::NT : 0));
#pragma unroll
            for (int f = 0; f < 4; ++f) {
              v[4 * h + f] = x[f];
              u[4 * h + f] = y[f];
            }
          }
#pragma unroll
          for (int f = 0; f < 8; ++f)
            r[f] = add ? T::load((uint16_t)(res[q][f >> 1] >> (16 * (f & 1)))) : 0.f;
          finish<T, Mode, decltype(act)::value, decltype(save)::value, 8>(p, which, row + q * kStepRows, col, v, u,
                                                                          bias, r);
        }
      }
    });
    __builtin_amdgcn_wave_barrier();
  }
}

template <typename T, int Mode, typename S>
static hipError_t launch_shape(const GemmArgs& p, int splits, float* partial, hipStream_t stream) {
  constexpr int kCols = Mode == kGated ? S::BN / 2 : S::BN;
  const int mt = (int)((p.m + S::BM - 1) / S::BM), nt = (p.n + kCols - 1) / kCols;
  const int64_t blocks = (int64_t)mt * nt * p.outputs * splits;
  const hipError_t e = launch_kernel(gemm_tile_kernel<T, Mode, S>, dim3((unsigned)blocks), dim3(64 * S::NW), stream,
                                     p, mt, nt, splits, partial);
  if (e != hipSuccess || splits == 1) return e;
  return launch_gemm_join(T::code, (enum Mode)Mode, p, splits, partial, stream);
}

typedef TileShape<256, 256, 2, 4> Large;
typedef TileShape<128, 256, 2, 4> Wide;
typedef TileShape<128, 128, 2, 2> Small;

template <typename T, int Mode>
static hipError_t launch_mode(const GemmArgs& p, const TilePlan& t, float* partial, hipStream_t stream) {
  switch (t.shape) {
    case 0: return launch_shape<T, Mode, Large>(p, t.splits, partial, stream);
    case 1: return launch_shape<T, Mode, Wide>(p, t.splits, partial, stream);
    default: return launch_shape<T, Mode, Small>(p, t.splits, partial, stream);
  }
}

template <typename T>
static hipError_t launch_typed(Mode mode, const GemmArgs& p, const TilePlan& t, float* partial,
                               hipStream_t stream) {
  switch (mode) {
    case kLinear: return launch_mode<T, kLinear>(p, t, partial, stream);
    case kGated: return launch_mode<T, kGated>(p, t, partial, stream);
    case kDx: return launch_mode<T, kDx>(p, t, partial, stream);
    default: return launch_mode<T, kDw>(p, t, partial, stream);
  }
}

hipError_t launch_gemm_tile(int dtype, Mode mode, const GemmArgs& p, const TilePlan& t, float* partial,
                            hipStream_t stream) {
  return dtype == BLOCK_BF16 ? launch_typed<BF16>(mode, p, t, partial, stream)
                             : launch_typed<F16>(mode, p, t, partial, stream);
}

int most_tile_splits(int64_t red, int segments) {
  // four stages each at least
  return (int)std::max<int64_t>(1, std::min<int64_t>(16, (red + kStep - 1) / kStep * segments / 4));
}

// Tile shape and K split of a product: the ones whose modelled time is least.
// Stage times in us, measured at K = 3584 with few CUs busy and with all (they
// share HBM and power): 256 x 256 0.55 / 0.81, 128 x 256 0.37 / 0.57, 128 x
// 128 0.25 / 0.31 and 0.64 where two share a CU; each round of blocks starts
// and ends in about 2 us; a split costs 3.5 us and its sums twice at 4.2 TB/s,
// against which forward tiles that end by themselves take 1 us more, the linear
// product's with GELU 4 (its instructions on few CUs); the gated product's GELU
// and the derivatives kept for training are not in the model. Over 106 shapes
// of 40-2048 rows, forward, dx and dw, the choice takes 1.3 % longer than the
// best of all shapes and splits (geometric mean; worst 25 %, 160 rows of gated
// 3584 x 7168: 57 us, 46 in 4 splits of 256 x 256). So large tiles where they
// fill the CUs (4096 x 3584 -> 4096: 99 us against 131 and 152), small ones for
// few rows (128 rows, 3584 -> 4096, 8 splits: 17.8 us; 256 x 256, 12 splits:
// 23.5), splits where even those are too few (2048 rows, 7168 -> 3584: 115 us
// in 2 splits of 256 x 256, 121 in one of 128 x 256).
TilePlan plan_tiles(Mode mode, const GemmArgs& p, size_t partial_bytes) {
  struct Cost { int bm, bn; double few, full; } const shapes[3] = {
      {256, 256, 0.55, 0.81}, {128, 256, 0.37, 0.57}, {128, 128, 0.25, 0.31}};
  const double pair = 0.64;
  const double ending = mode == kDx || mode == kDw                   ? 0.0
                        : mode == kLinear && p.act == BLOCK_ACT_GELU ? 4.0
                                                                     : 1.0;
  const double steps = (double)((p.red + kStep - 1) / kStep) * p.segments;
  const int planes = mode == kGated ? 2 : p.outputs, most = most_tile_splits(p.red, p.segments);
  TilePlan best{2, 1};
  double best_t = 0;
  for (int k = 0; k < 3; ++k) {
    const Cost& c = shapes[k];
    const int bn = mode == kGated ? c.bn / 2 : c.bn;
    const int64_t tiles = (int64_t)((p.m + c.bm - 1) / c.bm) * ((p.n + bn - 1) / bn) * p.outputs;
    for (int s = 1; s <= most; ++s) {
      const double bytes = 4.0 * p.m * ((p.n + 3) & ~3) * planes * s;
      if (s > 1 && bytes > (double)partial_bytes) break;
      const int64_t blocks = tiles * s, slots = k == 2 ? 512 : 256;
      const int64_t rounds = (blocks - 1) / slots, rest = blocks - rounds * slots;
      const double busy = rounds > 0 ? 1.0 : std::min(1.0, (double)rest / 256.0);
      const double last = rest > 256 ? pair : c.few + (c.full - c.few) * busy;
      double t = (double)rounds * (steps / s * (k == 2 ? pair : c.full) + 2.0) + steps / s * last + 2.0;
      t += s > 1 ? 3.5 + 2.0 * bytes / 4.2e6 : ending;
      if (best_t == 0 || t < best_t) {
        best = TilePlan{k, s};
        best_t = t;
      }
    }
  }
  return best;
}

}  // namespace block
