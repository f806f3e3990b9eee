// Matrix products of the layer's operators: the tile kernel, for row counts
// that make the matrix cores, not the weights' bandwidth, the bound.
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
//     16-byte piece c of row r sits at position c ^ ((r >> 2) & 3), so that
//     the 16 rows that the lanes of one group read take 16 different bank
//     groups. Read with ds_read_b128.
//   otherwise (rows contiguous): blocks of [32 r][32 rows], 64-byte lines,
//     whose two halves are swapped where bit 3 of r is set. The MFMA wants 8
//     consecutive r of one row per lane, which ds_read_tr16_b64 delivers.
template <bool RContig>
struct Operand {
  // this lane's source of load `c` (1 KB): row within the tile and r within
  // the stage of its first element
  static __device__ __forceinline__ int row(int c, int lane) {
    if constexpr (RContig) return 16 * c + (lane >> 2);
    return 32 * (c >> 1) + 8 * ((lane & 3) ^ ((lane >> 5) << 1));
  }
  static __device__ __forceinline__ int red(int c, int lane) {
    if constexpr (RContig) return 8 * ((lane & 3) ^ ((lane >> 4) & 3));
    return 16 * (c & 1) + (lane >> 2);
  }
  // addresses of this lane's part of a 16-row fragment: rows 16 t, t even
  // (h = 0) or odd (h = 1), relative to the even tile
  static __device__ __forceinline__ uint32_t base(int lane, int h) {
    const int g = lane >> 4, m = lane & 15;
    if constexpr (RContig) return (uint32_t)((16 * h + m) * 64 + ((g ^ ((m >> 2) & 3)) * 16));
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

// `v` moved down by d elements of 16 bits, zeros from above (d >= 8: all).
__device__ __forceinline__ u32x4 shift_down(u32x4 v, int d) {
  if (d & 4) v = u32x4{v[2], v[3], 0, 0};
  if (d & 2) v = u32x4{v[1], v[2], v[3], 0};
  if (d & 1)
    v = u32x4{v[0] >> 16 | v[1] << 16, v[1] >> 16 | v[2] << 16, v[2] >> 16 | v[3] << 16, v[3] >> 16};
  return d >= 8 ? u32x4{0, 0, 0, 0} : v;
}

// (the address space is said where a pointer is made from an integer: a flat
// load would also wait for LDS)
#define global_mem __attribute__((address_space(1)))
struct __attribute__((packed, aligned(4))) Dwords4 { u32x4 v; };

// Direct: operands go from global memory straight to LDS. Otherwise (rows
// that start at any element, contiguous lengths of any size from 8) they pass
// through registers: a 16-byte load that would run past a row's end starts
// earlier and is shifted into place before it is stored to LDS.
template <typename T, int Mode, typename S, bool Direct>
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
  // at a time.
  const int total = mtiles * ntiles * p.outputs;
  const int split = blockIdx.x / total;
  int lin = blockIdx.x - split * total;
  if ((total & 7) == 0) lin = (lin & 7) * (total >> 3) + (lin >> 3);
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
  // the tile reaches past an operand's rows or columns
  const bool edge = row0 + S::BM > p.m || col0 + kCols > p.n;

  // ---- global -> LDS -------------------------------------------------------
  // Rows past the matrix's end repeat its last one and columns its last eight
  // (their sums are not stored); past the reduction's end lanes load zeros.
  // off: this lane's byte offset of each of the wave's loads from the stage's
  // first byte of its matrix (a wave's loads of B are all of one matrix).
  // (through registers the offset of an r-contiguous piece leaves out r)
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
      off[i] = Mode != kDw ? (uint32_t)((min(row0 + r, p.m - 1) - row0) * p.lda + (Direct ? k : 0)) * 2u
                           : (uint32_t)(k * p.lda + min(row0 + r, p.m - 8)) * 2u;
    else
      off[i] = Mode == kDx ? (uint32_t)((min(col0 + r, p.n - 1) - col0) * p.ldb + (Direct ? k : 0)) * 2u
                           : (uint32_t)(k * p.ldb + min(col0 + r, p.n - 8)) * 2u;
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

  // Direct. Any stage; the last of a segment may be short.
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

  // Through registers. The r of an r-contiguous piece, the r row of the
  // others, and their first column are clamped to the matrix; `shift_down`
  // says by how much on the way to LDS. Rows may start at odd elements: a
  // piece is loaded as the four dwords from its first element's and the dword
  // of its last, and v_alignbit_b32 moves it into place.
  struct Held {
    u32x4 v;
    uint32_t last;
  };
  Held held[4][Direct ? 1 : S::PER];  // stage q in set q % 4
  auto fetch_at = [&](uintptr_t base, uint32_t o) __attribute__((always_inline)) -> Held {
    o += (uint32_t)(base & 2);
    base &= ~(uintptr_t)3;
    Held h;
    h.v = reinterpret_cast<const global_mem Dwords4*>(base + (o & ~3u))->v;
    h.last = *reinterpret_cast<const global_mem uint32_t*>(base + ((o + 14) & ~3u));
    return h;
  };
  constexpr bool kAr = Mode != kDw, kBr = Mode == kDx;  // r-contiguous
  // offset of load i of any stage: what the clamps make of it
  auto off_any = [&](int s, int i) __attribute__((always_inline)) -> uint32_t {
    const int ks = s >= per_seg ? s - per_seg : s;
    const int k = ks * kStep + red_of[i];
    if (i < S::A_PER ? kAr : kBr) return off[i] + (uint32_t)(min(k, red - 8) - ks * kStep) * 2u;
    return off[i] - (uint32_t)max(k - (red - 1), 0) * (uint32_t)(i < S::A_PER ? p.lda : p.ldb) * 2u;
  };
  auto align = [&](Held& h, uint32_t o) __attribute__((always_inline)) {
    const uint32_t by = (o & 2) * 8;
#pragma unroll
    for (int q = 0; q < 3; ++q) h.v[q] = __builtin_amdgcn_alignbit(h.v[q + 1], h.v[q], by);
    h.v[3] = __builtin_amdgcn_alignbit(h.last, h.v[3], by);
  };
  auto trim = [&](int s, Held(&h)[Direct ? 1 : S::PER]) __attribute__((always_inline)) {
    const int ks = s >= per_seg ? s - per_seg : s;
#pragma unroll
    for (int i = 0; i < S::PER; ++i) {
      const bool is_a = i < S::A_PER;
      const int c = wave + S::NW * (is_a ? i : i - S::A_PER);
      const int k = ks * kStep + red_of[i];
      if (is_a ? kAr : kBr) {
        h[i].v = shift_down(h[i].v, min(max(k - (red - 8), 0), 8));
      } else {
        const int over = is_a ? (int)(row0 + A::row(c, lane) - (p.m - 8)) : col0 + b_row(c) - (p.n - 8);
        h[i].v = shift_down(h[i].v, k >= red ? 8 : min(max(over, 0), 8));
      }
    }
  };
  auto put = [&](uint32_t buf, int i, const Held& h) __attribute__((always_inline)) {
    *(__attribute__((address_space(3))) u32x4*)(uintptr_t)(buf + slot(i) + lane * 16) = h.v;
  };
  auto fetch_any = [&](int s, Held(&h)[Direct ? 1 : S::PER]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < S::PER; ++i) {
      uintptr_t base = base_of(i < S::A_PER, s);
      uint32_t o = off_any(s, i);
      // a clamped r can lie before the stage's first: count from the row's
      if (i < S::A_PER ? kAr : kBr) {
        const uint32_t at = (uint32_t)(s >= per_seg ? s - per_seg : s) * (kStep * 2);
        base -= at;
        o += at;
      }
      h[i] = fetch_at(base, o);
    }
  };
  auto arrange_any = [&](int s, Held(&h)[Direct ? 1 : S::PER]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < S::PER; ++i) align(h[i], off_any(s, i) + (uint32_t)(base_of(i < S::A_PER, s) & 2));
    if (edge || (s >= per_seg ? s - per_seg : s) == per_seg - 1) trim(s, h);
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
  // wave's loads of a later stage go out. Direct: stage s + 4's, into the
  // buffer of stage s - 1, which the barrier before this step has freed.
  // Through registers: stage s + 6's, into one of four sets, while the set of
  // stage s + 3 goes to LDS (into the buffer of stage s - 2), so that a load
  // has three steps to arrive. load(n) does the n-th of PER shares of it.
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
  // At the end of stage s: stage s + 2 has to be in LDS (Direct: at most the
  // loads of the stages after it still in flight; through registers: it was
  // stored a step ago), and every read of stage s's buffer has to have
  // returned (at most the reads of stage s + 1 outstanding).
  constexpr int kLgkm = kReads < 15 ? kReads : 15;
  // (through registers the compiler waits for its own loads)
  constexpr int kVm1 = Direct ? S::PER : 63, kVm2 = Direct ? 2 * S::PER : 63, kVm0 = Direct ? 0 : 63;

  const int count = s1 - s0;
  if (count > 0) {
    // the first four stages; through registers: three, and three held
    if constexpr (Direct) {
#pragma unroll 1
      for (int s = 0; s < min(count, 4); ++s)
#pragma unroll
        for (int i = 0; i < S::PER; ++i) issue_any(s0 + s, lds0 + s * S::STAGE, i);
    } else {
      // (stages past the end repeat the last one: no branches here)
#pragma unroll
      for (int s = 0; s < 4; ++s) fetch_any(min(s0 + s, s1 - 1), held[s]);
#pragma unroll
      for (int s = 0; s < 3; ++s) {
        arrange_any(min(s0 + s, s1 - 1), held[s]);
#pragma unroll
        for (int i = 0; i < S::PER; ++i) put(lds0 + s * S::STAGE, i, held[s][i]);
      }
#pragma unroll
      for (int s = 4; s < 6; ++s) fetch_any(min(s0 + s, s1 - 1), held[s & 3]);
    }
    if (count >= 4)
      wait_barrier<kVm2, 0>();
    else
      wait_barrier<kVm0, 0>();
#pragma unroll
    for (int i = 0; i < S::MT; ++i) a[i] = read_a(lds0, i);
#pragma unroll
    for (int j = 0; j < S::NT; ++j) b0[j] = read_b(lds0, j);

    constexpr uint32_t kEnd = kStages * S::STAGE;
    // buffers of stage s + 1, and of stage s + 4 (through registers s + 3)
    uint32_t next = lds0 + S::STAGE, fill = lds0 + (Direct ? 4 : 3) * S::STAGE;
    auto advance = [&]() __attribute__((always_inline)) {
      next = next + S::STAGE == lds0 + kEnd ? lds0 : next + S::STAGE;
      fill = fill + S::STAGE == lds0 + kEnd ? lds0 : fill + S::STAGE;
    };
    // step s with s % kTurns == u: register sets by number
    constexpr int kTurns = Direct ? 2 : 4, kAhead = Direct ? 4 : 6;
    int s = 0;
    // Steady state: the stages to load are whole and follow each other.
    uintptr_t a_next = 0, b_next = 0;
    auto steady = [&](auto u_) __attribute__((always_inline)) {
      constexpr int u = decltype(u_)::value;
      Held(&in)[Direct ? 1 : S::PER] = held[(u + 2) & 3];
      Held(&out)[Direct ? 1 : S::PER] = held[(u + 3) & 3];
      if constexpr (!Direct) {
#pragma unroll
        for (int i = 0; i < S::PER; ++i) {
          const bool is_a = i < S::A_PER;
          const uint32_t o = off[i] + ((is_a ? kAr : kBr) ? 2u * red_of[i] : 0u);
          in[i] = fetch_at(is_a ? a_next : b_next, o);
          align(out[i], o + (uint32_t)((is_a ? a_next : b_next) & 2));
        }
        if (edge) trim(s0 + s + u + 3, out);
      }
      auto load = [&](int n) __attribute__((always_inline)) {
        if constexpr (Direct)
          dma16(reinterpret_cast<const char*>(n < S::A_PER ? a_next : b_next), off[n], fill + slot(n));
        else
          put(fill, n, out[n]);
      };
      step((u & 1) ? b1 : b0, (u & 1) ? b0 : b1, next, load);
      wait_barrier<kVm2, kLgkm>();
      advance();
      a_next += a_step;
      b_next += b_step;
    };
    // Any step: the ends of the segments.
    auto other = [&](auto u_) __attribute__((always_inline)) {
      constexpr int u = decltype(u_)::value;
      const int q = s + u;
      if (q >= count) return;
      const bool issue = q + kAhead < count, write = q + 3 < count;
      Held(&in)[Direct ? 1 : S::PER] = held[(u + 2) & 3];
      Held(&out)[Direct ? 1 : S::PER] = held[(u + 3) & 3];
      if constexpr (!Direct) {
        if (issue) fetch_any(s0 + q + kAhead, in);
        if (write) arrange_any(s0 + q + 3, out);
      }
      auto load = [&](int n) __attribute__((always_inline)) {
        if constexpr (Direct) {
          if (issue) issue_any(s0 + q + kAhead, fill, n);
        } else {
          if (write) put(fill, n, out[n]);
        }
      };
      step((u & 1) ? b1 : b0, (u & 1) ? b0 : b1, next, load);
      if (q + 2 < count) {
        if (q + 4 < count)
          wait_barrier<kVm2, kLgkm>();
        else if (q + 3 < count)
          wait_barrier<kVm1, kLgkm>();
        else
          wait_barrier<kVm0, kLgkm>();
      }
      advance();
    };
    using std::integral_constant;
    auto whole_stages = [&]() __attribute__((always_inline)) {
      const int first = s0 + s + kAhead;  // the next stage to load
      const int limit = min(s1, (first >= per_seg ? 2 : 1) * per_seg - (ragged ? 1 : 0));
      a_next = base_of(true, first);
      b_next = base_of(false, first);
#pragma unroll 1
      for (int t = first; t + kTurns <= limit; t += kTurns) {
        steady(integral_constant<int, 0>{});
        steady(integral_constant<int, 1>{});
        if constexpr (kTurns == 4) {
          steady(integral_constant<int, 2>{});
          steady(integral_constant<int, 3>{});
        }
        s += kTurns;
      }
    };
    auto other_stages = [&](int end) __attribute__((always_inline)) {
#pragma unroll 1
      for (; s < end; s += kTurns) {
        other(integral_constant<int, 0>{});
        other(integral_constant<int, 1>{});
        if constexpr (kTurns == 4) {
          other(integral_constant<int, 2>{});
          other(integral_constant<int, 3>{});
        }
      }
    };
    // (through registers, stage s + 3 on its way to LDS and stage s + 6 to load
    // have to be of one segment)
    if (Direct || Mode != kDx || s0 + 3 >= per_seg || s0 + kAhead < per_seg) whole_stages();
    if constexpr (Mode == kDx) {
      // past the first segment's end: until the next stage to load (through
      // registers: to store) is of the second
      if (s0 < per_seg && s1 > per_seg) {
        other_stages(min(count, per_seg - s0 - (Direct ? kAhead : 3)));
        whole_stages();
      }
    }
    other_stages(count);
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
  float* turn = reinterpret_cast<float*>(smem) + wave * 16 * kRows * kPitch;
  const int64_t wrow = row0 + 16 * S::MT * wm + lane / kLanes;
  const int wcol = 8 * (lane % kLanes);
  __syncthreads();
#pragma unroll
  for (int c = 0; c < S::MT / kRows; ++c) {
#pragma unroll
    for (int i = 0; i < kRows; ++i)
#pragma unroll
      for (int j = 0; j < S::NT; ++j)
        *reinterpret_cast<f32x4*>(turn + (16 * i + m) * kPitch + 16 * j + 4 * g) = acc[kRows * c + i][j];
    __builtin_amdgcn_wave_barrier();
#pragma unroll 2
    for (int r = 0; r < 16 * kRows; r += 64 / kLanes) {
      const float* t = turn + (r + lane / kLanes) * kPitch + wcol;
      float v[8], u[8];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const f32x4 x = *reinterpret_cast<const f32x4*>(t + 4 * q);
        const f32x4 y = *reinterpret_cast<const f32x4*>(t + 4 * q + (Mode == kGated ? 8 * S::NT : 0));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[4 * q + e] = x[e];
          u[4 * q + e] = y[e];
        }
      }
      epilogue<T, Mode, 8>(p, which, wrow + 16 * kRows * c + r, col0 + kWide * wn + wcol, v, u);
    }
    __builtin_amdgcn_wave_barrier();
  }
}

template <typename T, int Mode, typename S, bool Direct>
static hipError_t launch_shape(const GemmArgs& p, int splits, float* partial, hipStream_t stream) {
  constexpr int kCols = Mode == kGated ? S::BN / 2 : S::BN;
  const int mt = (int)((p.m + S::BM - 1) / S::BM), nt = (p.n + kCols - 1) / kCols;
  const int64_t blocks = (int64_t)mt * nt * p.outputs * splits;
  const hipError_t e = launch_kernel(gemm_tile_kernel<T, Mode, S, Direct>, dim3((unsigned)blocks), dim3(64 * S::NW), stream,
                                     p, mt, nt, splits, partial);
  if (e != hipSuccess || splits == 1) return e;
  return launch_gemm_join(T::code, (enum Mode)Mode, p, splits, partial, stream);
}

typedef TileShape<256, 256, 2, 4> Large;
typedef TileShape<128, 256, 2, 4> Wide;
typedef TileShape<128, 128, 2, 2> Small;

template <typename T, int Mode>
static hipError_t launch_mode(const GemmArgs& p, bool aligned, const TilePlan& t, float* partial, hipStream_t stream) {
  switch (t.shape) {
    case 0: return launch_shape<T, Mode, Large, true>(p, t.splits, partial, stream);
    case 1:
      return aligned ? launch_shape<T, Mode, Wide, true>(p, t.splits, partial, stream)
                     : launch_shape<T, Mode, Wide, false>(p, t.splits, partial, stream);
    default:
      return aligned ? launch_shape<T, Mode, Small, true>(p, t.splits, partial, stream)
                     : launch_shape<T, Mode, Small, false>(p, t.splits, partial, stream);
  }
}

template <typename T>
static hipError_t launch_typed(Mode mode, const GemmArgs& p, bool aligned, const TilePlan& t, float* partial,
                               hipStream_t stream) {
  switch (mode) {
    case kLinear: return launch_mode<T, kLinear>(p, aligned, t, partial, stream);
    case kGated: return launch_mode<T, kGated>(p, aligned, t, partial, stream);
    case kDx: return launch_mode<T, kDx>(p, aligned, t, partial, stream);
    default: return launch_mode<T, kDw>(p, aligned, t, partial, stream);
  }
}

hipError_t launch_gemm_tile(int dtype, Mode mode, const GemmArgs& p, bool aligned, const TilePlan& t, float* partial,
                            hipStream_t stream) {
  return dtype == BLOCK_BF16 ? launch_typed<BF16>(mode, p, aligned, t, partial, stream)
                             : launch_typed<F16>(mode, p, aligned, t, partial, stream);
}

// Tile shape and K split of a product: the ones whose modelled time is least.
// Stage times in us, measured at K = 3584 with one block on few CUs and with
// all CUs busy (they share HBM and power): 256 x 256 0.63 / 0.87, 128 x 256
// 0.42 / 0.58, 128 x 128 0.35 / 0.39 and 0.65 where two share a CU; each round
// of blocks starts and ends in about 2 us; a split costs 5 us and its sums
// twice at 4.2 TB/s. So large tiles where they fill the CUs (4096 x 3584 ->
// 4096: 98 us against 129 and 150), small ones for few rows (128 rows, 3584 ->
// 4096, 8 splits: 17.9 us; 256 x 256, 12 splits: 23.7). Through registers
// (unaligned) the large tile's accumulators leave no room for the loads.
TilePlan plan_tiles(Mode mode, const GemmArgs& p, bool aligned, size_t partial_bytes) {
  struct Cost { int bm, bn; double few, full; } const shapes[3] = {
      {256, 256, 0.63, 0.87}, {128, 256, 0.42, 0.58}, {128, 128, 0.35, 0.39}};
  const double pair = 0.65;
  const double steps = (double)((p.red + kStep - 1) / kStep) * p.segments;
  const int planes = mode == kGated ? 2 : p.outputs;
  TilePlan best{2, 1};
  double best_t = 0;
  for (int k = aligned ? 0 : 1; k < 3; ++k) {
    const Cost& c = shapes[k];
    const int bn = mode == kGated ? c.bn / 2 : c.bn;
    const int64_t tiles = (int64_t)((p.m + c.bm - 1) / c.bm) * ((p.n + bn - 1) / bn) * p.outputs;
    for (int s = 1; s <= 16; ++s) {
      const double bytes = 4.0 * p.m * ((p.n + 3) & ~3) * planes * s;
      if (s > 1 && (bytes > (double)partial_bytes || steps / s < 4)) break;
      const int64_t blocks = tiles * s, slots = k == 2 ? 512 : 256;
      const int64_t rounds = (blocks - 1) / slots, rest = blocks - rounds * slots;
      const double busy = rounds > 0 ? 1.0 : std::min(1.0, (double)rest / 256.0);
      const double last = rest > 256 ? pair : c.few + (c.full - c.few) * busy;
      double t = (double)rounds * (steps / s * (k == 2 ? pair : c.full) + 2.0) + steps / s * last + 2.0;
      if (s > 1) t += 5.0 + 2.0 * bytes / 4.2e6;
      if (best_t == 0 || t < best_t) {
        best = TilePlan{k, s};
        best_t = t;
      }
    }
  }
  return best;
}

}  // namespace block
