// 8-bit products of more than 32 rows of an expert, or of many experts with few,
// on v_mfma_i32_16x16x64_i8. How many rows an expert has is known on the device
// only: 256 blocks, one to a CU, go through the lists of items by themselves.
//
// tiles: up to 256 rows by 256 columns of the packed weights (for the gated
// product 128 output columns, gate and up alternating by 16). Eight waves, two
// by four, have half of the rows and a quarter of the columns each. The
// reduction runs in stages of 64, one MFMA deep, through a ring of LDS buffers:
// one is read into registers while the one before is multiplied, the others are
// on their way from memory. Rows lie in LDS as 64-byte lines with a swizzle,
// weights as the packed form has them, so that neither read meets a bank
// conflict. There is a body for 64, 128, 192 and 256 rows (160 rows of 3584 x
// 65536: 60 us, in the next larger one 63; 64 rows 53, in the largest 56). The
// weights of an expert with one row tile pass by the caches (64 rows of 3584 x
// 65536: 45 us, else 53; where row tiles share them it costs 4 %).
//   2048 x 3584 x 7168: 58 us, 1.8 POP/s, 224 tiles of 256 CUs, whose matrix cores
// are busy half of the time: a stage of 256 rows takes 0.67 us, of which the
// MFMAs are 0.43, and 13 us go into start and ending, which nothing overlaps. 8192 x
// 8192 x 8192: 464 us, 2.37 POP/s.
//
// mid items, where there are few tiles, or after them: up to 64 rows by 64
// columns, the reduction dealt to the eight waves, whose operands come straight
// from memory and whose sums meet in LDS: half of the matrix cores' rate at
// best, but an eighth of the steps one after another, which is what the time is
// made of there (256 x 3584 x 7168: 26 us, as 28 tiles 52). The next item's first
// operands are on their way while one ends.
#include "experts_device.h"
#include "lds_device.h"

namespace experts {

using block::dma16;
using block::lds_b128;
using block::wait_barrier;

constexpr int kWaves = 8, kCols = 16 * kTileCols, kLds = 160 * 1024;

// 16-row fragments of a wave, of which there are two above each other.
template <int MT>
struct Shape {
  static constexpr int BM = 32 * MT;
  static constexpr int A_BYTES = BM * kBlockRed, B_BYTES = kCols * kBlockRed, STAGE = A_BYTES + B_BYTES;
  static constexpr int kStages = kLds / STAGE < 8 ? kLds / STAGE : 8;
  static constexpr int A_LOADS = BM / 16, A_PER = (A_LOADS + kWaves - 1) / kWaves;  // of 1 KB; of a wave
  static constexpr int PER = A_PER + kCols / 16 / kWaves;
  static constexpr int kReads = MT + 4;  // LDS reads of a wave and stage
};

// Once: no other row tile reads these weights.
template <typename T, bool Gated, int MT, bool Once>
__device__ __forceinline__ void tile(const ProductArgs& p, char* smem, int expert, int row0, int rows, int tile0) {
  typedef Shape<MT> S;
  typedef typename T::raw raw;
  constexpr int NT = 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int lane = threadIdx.x & (kWave - 1), g = lane >> 4, m = lane & 15;
  const int wm = wave / 4, wn = wave % 4;
  const int tiles = packed_tiles<Gated>(p), count = p.blocks;

  // ---- global -> LDS: rows past the last repeat it, column tiles likewise ----
  const char* src[S::PER];
  uint32_t dst[S::PER];
  constexpr int kStep[2] = {kBlockRed, kBlockBytes};  // from one stage to the next
#pragma unroll
  for (int i = 0; i < S::PER; ++i) {
    if (i < S::A_PER) {
      // fewer loads than waves: some are done twice, so that every wave counts alike
      const int c = (wave + kWaves * i) % S::A_LOADS;
      const int t = token_of(p, row0 + min(16 * c + (lane >> 2), rows - 1));
      src[i] = reinterpret_cast<const char*>(p.q) + (int64_t)t * count * kBlockRed +
               16 * ((lane & 3) ^ block::swizzle(lane >> 4));
      dst[i] = c * 1024;
    } else {
      const int c = wave + kWaves * (i - S::A_PER);
      src[i] = reinterpret_cast<const char*>(packed_tile(p, expert, tiles, min(tile0 + c, tiles - 1))) + 16 * lane;
      dst[i] = S::A_BYTES + c * 1024;
    }
  }
  const uint32_t lds0 = (uint32_t)(uintptr_t)(block::lds_void*)smem;
  auto issue = [&](int i, int s, uint32_t buf) __attribute__((always_inline)) {
    const char* from = src[i] + (int64_t)s * kStep[i < S::A_PER ? 0 : 1];
    if (i >= S::A_PER && Once)
      block::dma16_once(from, buf + dst[i]);
    else
      dma16(from, buf + dst[i]);
  };
  // the row's scale, for the ending
  const int mine = min((int)threadIdx.x, rows - 1);
  const float step = p.step[token_of(p, row0 + mine)];

  // ---- LDS -> registers ----
  const uint32_t a_rd = (uint32_t)(wm * MT * 1024 + m * 64 + (g ^ block::swizzle(m >> 2)) * 16);
  const uint32_t b_rd = (uint32_t)(S::A_BYTES + wn * NT * 1024 + 16 * lane);
  auto read_a = [&](uint32_t buf, int i) { return lds_b128(buf + a_rd + i * 1024); };
  auto read_b = [&](uint32_t buf, int j) { return lds_b128(buf + b_rd + j * 1024); };

  i32x4 acc[MT][NT] = {};
  u32x4 a[MT], b0[NT], b1[NT];
  // Stage s's MFMAs, while stage s + 1 is read (a[i] as soon as its last MFMA is
  // issued, b into the other registers) and the loads of stage s + kStages - 1 go
  // out into the buffer that the last barrier freed.
  auto step_of = [&](u32x4(&b)[NT], u32x4(&bn)[NT], uint32_t next, auto load) __attribute__((always_inline)) {
    constexpr int kEvery = MT * NT / S::PER;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int n = i * NT + j;
        if (n % kEvery == kEvery / 2 && n / kEvery < S::PER) load(n / kEvery);
        acc[i][j] = mfma(b[j], a[i], acc[i][j]);
      }
      if (MT >= NT ? i < NT : true)
#pragma unroll
        for (int j = i; j < NT; j += MT) bn[j] = read_b(next, j);
      a[i] = read_a(next, i);
    }
  };
  constexpr int kLgkm = S::kReads < 15 ? S::kReads : 15;
  constexpr int kAhead = S::kStages - 1;

#pragma unroll 1
  for (int s = 0; s < min(count, kAhead); ++s)
#pragma unroll
    for (int i = 0; i < S::PER; ++i) issue(i, s, lds0 + s * S::STAGE);
  if (count >= kAhead)
    wait_barrier<(kAhead - 2) * S::PER, 0>();
  else
    wait_barrier<0, 0>();
#pragma unroll
  for (int i = 0; i < MT; ++i) a[i] = read_a(lds0, i);
#pragma unroll
  for (int j = 0; j < NT; ++j) b0[j] = read_b(lds0, j);
  constexpr uint32_t kEnd = S::kStages * S::STAGE;
  uint32_t next = lds0 + S::STAGE, fill = lds0 + kAhead * S::STAGE;
  auto advance = [&]() __attribute__((always_inline)) {
    next = next + S::STAGE == lds0 + kEnd ? lds0 : next + S::STAGE;
    fill = fill + S::STAGE == lds0 + kEnd ? lds0 : fill + S::STAGE;
  };
  int s = 0;
  auto steady = [&](u32x4(&b)[NT], u32x4(&bn)[NT], int at) __attribute__((always_inline)) {
    step_of(b, bn, next, [&](int n) __attribute__((always_inline)) { issue(n, at + kAhead, fill); });
    wait_barrier<(kAhead - 2) * S::PER, kLgkm>();
    advance();
  };
#pragma unroll 1
  for (; s + 1 + kAhead < count; s += 2) {
    steady(b0, b1, s);
    steady(b1, b0, s + 1);
  }
  auto other = [&](int at, u32x4(&b)[NT], u32x4(&bn)[NT]) __attribute__((always_inline)) {
    if (at >= count) return;
    const bool more = at + kAhead < count;
    step_of(b, bn, next, [&](int n) __attribute__((always_inline)) {
      if (more) issue(n, at + kAhead, fill);
    });
    // stage at + 2 has to be in LDS
    if (at + 2 < count) {
      const int behind = min(count - 1, at + kAhead) - (at + 2);  // stages that may be in flight
      if (behind >= kAhead - 2)
        wait_barrier<(kAhead - 2) * S::PER, kLgkm>();
      else if (behind >= 1)
        wait_barrier<S::PER, kLgkm>();
      else
        wait_barrier<0, kLgkm>();
    }
    advance();
  };
#pragma unroll 1
  for (; s < count; s += 2) {
    other(s, b0, b1);
    other(s + 1, b1, b0);
  }

  // ---- ending: each wave turns its sums around in LDS, 16 kRows rows at a
  // time, so that a lane ends eight columns of a row at once ----
  constexpr int kPitch = 16 * NT + 4;
  constexpr int kRows = MT % 4 == 0 ? 4 : 2;
  constexpr int kTurn = kWaves * 16 * kRows * kPitch * 4;
  constexpr int kWide = Gated ? 8 * NT : 16 * NT;  // output columns of a wave
  constexpr int kLanes = kWide / 8, kStepRows = kWave / kLanes, kSteps = 16 * kRows / kStepRows;
  static_assert(kTurn + S::BM * 4 <= kLds, "LDS");
  int* turn = reinterpret_cast<int*>(smem) + wave * 16 * kRows * kPitch;
  float* steps = reinterpret_cast<float*>(smem + kTurn);
  const int wcol = 8 * (lane % kLanes), col = (Gated ? tile0 / 2 : tile0) * 16 + kWide * wn + wcol;
  const int from = Gated ? wcol / 16 * 32 + wcol % 16 : wcol;
  const Columns<T, Gated, 8> k(p, expert, col);
  // The residual's loads are a group of steps ahead of their use.
  constexpr int kGroup = kSteps < 4 ? kSteps : 4;
  static_assert(kSteps % kGroup == 0, "");
  const bool add = !Gated && p.residual != nullptr;
  const int wrow = 16 * MT * wm + lane / kLanes;
  u32x4 ahead[kGroup];
  auto fetch = [&](u32x4& d, int l) __attribute__((always_inline)) {
    d = load8(static_cast<const uint16_t*>(p.residual) + (row0 + min(l, rows - 1)) * p.ldr + col, p.n - col);
  };
  if (add)
#pragma unroll
    for (int f = 0; f < kGroup; ++f) fetch(ahead[f], wrow + f * kStepRows);
  __syncthreads();
  if ((int)threadIdx.x < S::BM) steps[threadIdx.x] = step;
  __syncthreads();
#pragma unroll 1
  for (int c = 0; c < MT / kRows; ++c) {
#pragma unroll
    for (int cc = 0; cc < MT / kRows; ++cc)
      if (c == cc)
#pragma unroll
        for (int i = 0; i < kRows; ++i)
#pragma unroll
          for (int j = 0; j < NT; ++j)
            *reinterpret_cast<i32x4*>(turn + (16 * i + m) * kPitch + 16 * j + 4 * g) = acc[kRows * cc + i][j];
    __builtin_amdgcn_wave_barrier();
    with_ending<Gated>(p, [&](auto act) __attribute__((always_inline)) {
#pragma unroll 1
      for (int q = 0; q < kSteps; q += kGroup) {
        const int at = wrow + 16 * kRows * c + q * kStepRows;
#pragma unroll
        for (int f = 0; f < kGroup; ++f) {
          const int local = at + f * kStepRows;
          const int* t = turn + ((q + f) * kStepRows + lane / kLanes) * kPitch + from;
          float v[8], u[8], residual[8];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const i32x4 x = *reinterpret_cast<const i32x4*>(t + 4 * h);
            const i32x4 y = *reinterpret_cast<const i32x4*>(t + 4 * h + (Gated ? 16 : 0));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              v[4 * h + e] = (float)x[e];
              u[4 * h + e] = (float)y[e];
            }
          }
#pragma unroll
          for (int e = 0; e < 8; ++e)
            residual[e] = add ? T::load((uint16_t)(ahead[f][e >> 1] >> (16 * (e & 1)))) : 0.f;
          if (add) fetch(ahead[f], local + kGroup * kStepRows);
          if (local < rows && col < p.n)
            finish<T, Gated, decltype(act)::value, 8>(p, k, row0 + local, col, steps[local], v, u, residual);
        }
      }
    });
    __builtin_amdgcn_wave_barrier();
  }
  __syncthreads();  // before the next tile's loads to LDS
}

// A block's mid items of `end`: next_of(-1) is the first, at(j) the j-th.
template <typename T, bool Gated, typename Next, typename At>
__device__ __forceinline__ void mid_items(const ProductArgs& p, char* smem, int end, Next next_of, At at) {
  typedef typename T::raw raw;
  constexpr int C = kMidCols, RT = kMidRows / 16, kPitch = 16 * C + 4;
  typedef int32_t Slab[kWaves][16][kPitch];
  Slab* slabs = reinterpret_cast<Slab*>(smem);  // one for 16 rows
  static_assert(RT * sizeof(Slab) <= kLds, "LDS");
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int lane = threadIdx.x & (kWave - 1), g = lane >> 4, m = lane & 15;
  const int tiles = packed_tiles<Gated>(p);
  const int count = p.blocks > wave ? (p.blocks - wave + kWaves - 1) / kWaves : 0;
  // a thread ends four columns of one row of every slab that it has a part in
  constexpr int kOut = Gated ? 2 * C : 4 * C;           // groups of 4 output columns
  constexpr int kSlabs = kWave * kWaves / (16 * kOut);  // at once
  constexpr int kTurns = RT / kSlabs;
  const int o = threadIdx.x % kOut, sr = threadIdx.x / kOut % 16, s0 = threadIdx.x / (16 * kOut);
  const int from = 4 * (Gated ? o / 4 * 8 + o % 4 : o);

  struct Step {
    u32x4 w[C], x[RT];
  };
  Item it;
  int tile0;
  const uint8_t* w[C];  // uniform; lanes are 16 bytes apart
  const int8_t* q[RT];
  Step d0, d1;
  auto point = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < C; ++c)
      w[c] = packed_tile(p, it.expert, tiles, min(tile0 + c, tiles - 1)) + (int64_t)wave * kBlockBytes;
#pragma unroll
    for (int r = 0; r < RT; ++r)
      q[r] = p.q + ((int64_t)token_of(p, it.row + min(16 * r + m, it.rows - 1)) * p.blocks + wave) * kBlockRed + 16 * g;
  };
  auto fetch = [&](Step& d, int i, int rows) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < C; ++c)
      d.w[c] = *reinterpret_cast<const u32x4*>(w[c] + (int64_t)i * kWaves * kBlockBytes + (uint32_t)(16 * lane));
#pragma unroll
    for (int r = 0; r < RT; ++r)
      if (16 * r < rows) d.x[r] = *reinterpret_cast<const u32x4*>(q[r] + (int64_t)i * kWaves * kBlockRed);
  };
  auto start = [&]() __attribute__((always_inline)) {
    point();
    if (count > 0) fetch(d0, 0, it.rows);
    if (count > 1) fetch(d1, 1, it.rows);
  };
  int next = next_of(-1);
  if (next < end) {
    it = at(next, tile0);
    start();
  }
#pragma unroll 1
  while (next < end) {
    const Item now = it;
    const int col = (Gated ? tile0 / 2 : tile0) * 16 + 4 * o;
    const Columns<T, Gated, 4> k(p, now.expert, col);
    float step[kTurns], residual[kTurns][4];
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
      const int64_t row = now.row + min(16 * (s0 + kSlabs * i) + sr, now.rows - 1);
      step[i] = p.step[token_of(p, (int)row)];
#pragma unroll
      for (int t = 0; t < 4; ++t) residual[i][t] = 0.f;
      if (!Gated && p.residual != nullptr)
        load_values<T, 4>(static_cast<const uint16_t*>(p.residual) + row * p.ldr + col, residual[i], p.n - col);
    }
    next = next_of(next);
    if (next < end) it = at(next, tile0);  // (early: the list is read from memory)
    i32x4 acc[RT][C] = {};
    auto multiply = [&](const Step& d) __attribute__((always_inline)) {
#pragma unroll
      for (int r = 0; r < RT; ++r)
        if (16 * r < now.rows)
#pragma unroll
          for (int c = 0; c < C; ++c) acc[r][c] = mfma(d.w[c], d.x[r], acc[r][c]);
    };
#pragma unroll 1
    for (int i = 0; i < count; i += 2) {
      multiply(d0);
      __builtin_amdgcn_sched_barrier(0);
      if (i + 2 < count) fetch(d0, i + 2, now.rows);
      if (i + 1 < count) {
        multiply(d1);
        __builtin_amdgcn_sched_barrier(0);
        if (i + 3 < count) fetch(d1, i + 3, now.rows);
      }
    }
    if (next < end) start();
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int c = 0; c < C; ++c) *reinterpret_cast<i32x4*>(&slabs[r][wave][m][16 * c + 4 * g]) = acc[r][c];
    wait_barrier<63, 0>();
    with_ending<Gated>(p, [&](auto act) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < kTurns; ++i) {
        const int r = s0 + kSlabs * i, local = 16 * r + sr;
        if (local >= now.rows || col >= p.n) continue;
        i32x4 v = {}, u = {};
#pragma unroll
        for (int x = 0; x < kWaves; ++x) {
          v += *reinterpret_cast<const i32x4*>(&slabs[r][x][sr][from]);
          if constexpr (Gated) u += *reinterpret_cast<const i32x4*>(&slabs[r][x][sr][from + 16]);
        }
        float sum[4], up[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          sum[t] = (float)v[t];
          up[t] = (float)u[t];
        }
        finish<T, Gated, decltype(act)::value, 4>(p, k, now.row + local, col, step[i], sum, up, residual[i]);
      }
    });
    wait_barrier<63, 0>();  // before the next item's sums
  }
}

template <typename T, bool Gated>
__global__ __launch_bounds__(kWave * kWaves) __attribute__((amdgpu_waves_per_eu(2, 2)))
void tile_kernel(ProductArgs p, Way way) {
  __shared__ __attribute__((aligned(1024))) char smem[kLds];
  const bool listed = p.lists.counts != nullptr;
  const int xcd = blockIdx.x & 7, per = gridDim.x >> 3;
  const int slot = blockIdx.x >> 3;
  const int ntiles = (packed_tiles<Gated>(p) + kTileCols - 1) / kTileCols;
  const int mtiles = listed ? p.lists.counts[2] : way == kFew ? 0 : (p.rows + kTileRows - 1) / kTileRows;
  // (products of items and columns stay below 2^31: 2^24 rows in items of 64 by
  // 2^12 groups of columns at most)
  const int total = mtiles * ntiles;
  // Blocks are dealt round-robin over the 8 XCDs: each XCD has a contiguous
  // range of tiles, which its blocks go through in turn.
  const int begin = (int)((int64_t)total * xcd / 8), end = (int)((int64_t)total * (xcd + 1) / 8);
  for (int at = begin + slot; at < end; at += per) {
    // row tiles of an expert in groups of 8, column by column (8192 x 8192 x 8192:
    // 464 us, without groups 510; 2048 x 3584 x 7168: 58.7 and 60.1)
    const Item it = listed ? p.lists.tiles[at / ntiles] : Item{0, 0, p.rows, 0};
    const int high = (it.rows + kTileRows - 1) / kTileRows;  // its row tiles
    const int local = at - it.first * ntiles;
    const int group = local / (8 * ntiles), in = local - group * 8 * ntiles;
    const int gm = min(high - 8 * group, 8);
    const int height = min(((it.rows + high - 1) / high + 31) / 32 * 32, kTileRows);
    const int mt = 8 * group + in % gm, nt = in / gm;
    const int row0 = it.row + mt * height, rows = min(height, it.rows - mt * height);
    const int tile0 = nt * kTileCols;
    if (high == 1) {
      if (rows <= 64)
        tile<T, Gated, 2, true>(p, smem, it.expert, row0, rows, tile0);
      else if (rows <= 128)
        tile<T, Gated, 4, true>(p, smem, it.expert, row0, rows, tile0);
      else if (rows <= 192)
        tile<T, Gated, 6, true>(p, smem, it.expert, row0, rows, tile0);
      else
        tile<T, Gated, 8, true>(p, smem, it.expert, row0, rows, tile0);
    } else if (rows <= 192) {
      tile<T, Gated, 6, false>(p, smem, it.expert, row0, rows, tile0);
    } else {
      tile<T, Gated, 8, false>(p, smem, it.expert, row0, rows, tile0);
    }
  }
  // Blocks that had a tile less take the four mid items that it is worth first.
  const int groups = (packed_tiles<Gated>(p) + kMidCols - 1) / kMidCols;
  const int mids = listed ? p.lists.counts[1] : way == kFew ? (p.rows + kMidRows - 1) / kMidRows : 0;
  const int all = mids * groups, first = (int)((int64_t)all * xcd / 8);
  const int count = (int)((int64_t)all * (xcd + 1) / 8) - first;
  const int more = (end - begin) % per, less = per - more, extra = more != 0 ? 4 * less : 0;
  auto next_of = [&](int j) __attribute__((always_inline)) {
    if (j < 0) return more != 0 && slot >= more ? slot - more : extra + slot;
    if (j >= extra) return j + per;
    return j + less < extra ? j + less : extra + slot;
  };
  mid_items<T, Gated>(p, smem, count, next_of, [&](int j, int& tile0) __attribute__((always_inline)) {
    // row tiles of the same columns next to each other, where one expert has all
    const int by = listed ? groups : mids, at = (first + j) / by, rest = first + j - at * by;
    tile0 = (listed ? rest : at) * kMidCols;
    return listed ? p.lists.mid[at] : Item{0, rest * kMidRows, min(p.rows - rest * kMidRows, kMidRows), 0};
  });
}

template <typename T, bool Gated>
static hipError_t launch_typed(const ProductArgs& p, Way way, hipStream_t stream) {
  return launch_kernel(tile_kernel<T, Gated>, dim3(256), dim3(kWave * kWaves), stream, p, way);
}

hipError_t launch_tiles(int dtype, const ProductArgs& p, Way way, hipStream_t stream) {
  if (dtype == BLOCK_BF16)
    return p.gated ? launch_typed<BF16, true>(p, way, stream) : launch_typed<BF16, false>(p, way, stream);
  return p.gated ? launch_typed<F16, true>(p, way, stream) : launch_typed<F16, false>(p, way, stream);
}

}  // namespace experts
