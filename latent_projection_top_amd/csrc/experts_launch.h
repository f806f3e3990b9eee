// Host-side launchers of the routed half of a layer (called by the C ABI in
// experts_api.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "experts.h"
#include "route_launch.h"

namespace experts {

using route::launch_kernel;

// At least that many blocks, in two dimensions: one holds fewer than 2^32 threads.
inline dim3 grid_of(int64_t blocks) {
  const int64_t y = (blocks + (1 << 20) - 1) >> 20;
  return dim3((unsigned)((blocks + y - 1) / y), (unsigned)y);
}

// ------------------------------------------------------------------- sort --

struct SortArgs {
  const int32_t* ids;
  int32_t* offsets;
  int32_t* place;
  int32_t* token;
  void* workspace;
  int choices, topk, experts, first, capacity;
};
size_t sort_workspace_bytes(int64_t choices, int experts);
hipError_t launch_sort(const SortArgs& args, hipStream_t stream);

// ------------------------------------------------------- gather / combine --

// Both directions are one of two movements: rows spread to their choices'
// places, or summed from there. `plain` has a row per token, `sorted` one per
// position.
struct RowsArgs {
  const void* plain;      // x, dy
  const void* sorted;     // ys, dxs
  const void* residual;
  const float* weights;   // NULL: 1
  const int32_t* place;
  void* to_plain;         // y, dx
  void* to_sorted;        // xs, dys
  float* dweights;
  int64_t ld_plain, ld_sorted, ld_residual, ld_to_plain, ld_to_sorted;
  int rows, topk, width, capacity;
};
hipError_t launch_spread(int dtype, const RowsArgs& args, hipStream_t stream);   // to_sorted and dweights
hipError_t launch_collect(int dtype, const RowsArgs& args, hipStream_t stream);  // to_plain

// ------------------------------------------------------- 8-bit products --

// A packed matrix is, for each expert, column tiles of 16 by blocks of 64 of
// the reduction, 1 KB each: lane l's 16 bytes at 16 l are the reduction's 16 (l
// / 16) .. + 15 of column l % 16, an operand of v_mfma_i32_16x16x64 as it is.
// Blocks of a column tile follow each other; columns and reduction past the end
// are zeros. The gated product's column tiles alternate, gate and up.
constexpr int kBlockRed = 64, kBlockBytes = 1024;
inline int red_blocks(int k) { return (k + kBlockRed - 1) / kBlockRed; }
inline int column_tiles(int n) { return (n + 15) / 16; }

// How a product's rows are dealt out. How many rows an expert has is known on
// the device only, which makes lists of items:
//   kBrief     all are brief items of up to kStreamRows rows, for a kernel that
//              streams weights
//   kApart     experts of up to kStreamRows rows are brief items; of more, row
//              tiles of up to kTileRows, for another kernel
//   kTogether  short experts are row tiles of up to kMidRows (mid items), which
//              the second kernel takes after its tiles: one launch less
//   kFew       all are mid items
enum Way { kBrief, kApart, kTogether, kFew };
// (of a tile, `rows` is of all of its expert's, which are at `first` and after)
struct Item {
  int32_t expert, row, rows, first;
};
constexpr int kStreamRows = 32, kMidRows = 64, kTileRows = 256;
constexpr int kMidCols = 4, kTileCols = 16;  // packed column tiles of 16 that each takes
struct Lists {
  const int32_t* counts;  // brief, mid, tiles; NULL: one expert has every row
  const Item* brief;
  const Item* mid;
  const Item* tiles;
};
inline int64_t most_live(int64_t rows, int experts) { return rows < experts ? rows : experts; }  // experts with rows
inline int64_t most_brief(int64_t rows, int experts) { return rows / kStreamRows + most_live(rows, experts); }
inline int64_t most_mid(int64_t rows, int experts) { return rows / kMidRows + most_live(rows, experts); }
inline int64_t most_tiles(int64_t rows, int experts) {
  return rows / kTileRows + most_live(rows / (kStreamRows + 1), experts);
}
inline size_t list_bytes(int64_t rows, int experts) {
  return sizeof(Item) *
         (size_t)(1 + most_brief(rows, experts) + most_mid(rows, experts) + most_tiles(rows, experts));
}
inline Lists lists_at(void* area, int64_t rows, int experts) {
  const Item* items = static_cast<const Item*>(area);
  const Item* mid = items + 1 + most_brief(rows, experts);
  return Lists{&items->expert, items + 1, mid, mid + most_mid(rows, experts)};
}

// The way of a product of `rows` rows.
//   kBrief where experts have few rows on average: weights that a few items read
// again come from the caches (gated, in us, this and the next best: 1024 x 16 of
// 896 experts of 512 x 256, 18 rows to each, 75 and 103; 96 x 16 of 64, 24 to
// each, 2048 x 2048, 102 and 115; 30 to each 127 and 113). An expert
// of many rows among them becomes as many items, each of which reads its weights
// (2048 rows of 112 experts of 3584 x 4096, dealt evenly, then with a quarter, half
// and nine tenths of them one expert's: 310, 345, 369 and 417; by the rules below
// 312, 340, 331 and 323).
//   kFew where its modelled time in us is less than the tiles' (256 x 3584 x 7168:
// 27 and 52; 40 x 2048 x 2048: 11 and 17; 333 x 6 of 40 experts of 1019 x 777: 25
// and 33): a mid item's is mostly latency; many wait for each other, 256 at a
// time, or for their operands, 8 KB for each block of the reduction, which the L2s
// deliver at 8 TB/s; tiles come in rounds of 256, and by expert with another
// launch before them. (By expert mid items as many, and tiles as few, as there can
// be.)
//   kApart where the weights are more than the last-level cache holds: streaming
// the short experts' in a kernel of its own is worth a launch (112 experts of 3584
// x 4096, 1.6 GB: 260 us, together 302; 33 of 253 x 320, 3 MB: 26 and 22).
//   What counts is the rows that there is room for, of which the experts may keep
// few (a rank's share; gated, 112 experts of 3584 x 4096 that keep 2048 of 16384 rows:
// 334 us, by the way of 2048 rows 321; 1024 of 8192: 299 and 308).
inline Way way_of(int64_t rows, int experts, int column_tiles, int blocks, bool offsets) {
  if (rows <= kStreamRows || (offsets && rows <= 24 * (int64_t)experts)) return kBrief;
  const int64_t mids = (rows + kMidRows - 1) / kMidRows + (offsets ? most_live(rows, experts) : 0);
  const int64_t tiles = (rows + kTileRows - 1) / kTileRows;
  const int64_t m = mids * ((column_tiles + kMidCols - 1) / kMidCols);
  const int64_t t = tiles * ((column_tiles + kTileCols - 1) / kTileCols);
  const double step = (double)blocks;
  const double busy = (double)m * step * 0.001, rounds = (double)((m + 255) / 256) * (3.0 + 0.1 * step);
  if (3.0 + (busy > rounds ? busy : rounds) <
      (double)((t + 255) / 256) * (12.0 + 0.65 * step) + (offsets ? 8.0 + 0.1 * step : 0.0))
    return kFew;
  const double bytes = (double)experts * column_tiles * blocks * kBlockBytes;
  return offsets && bytes > 256e6 ? kApart : kTogether;
}

// Few rows of a short reduction: the streaming kernel makes the integers by
// itself, in items of up to kFusedItem rows, for every item again, which saves a
// launch (8 x 512 x 7168: 5.0 us and 6.7; 8 x 2048 x 7168: 7.4 and 8.0; gated 32
// x 16 of 64 experts, 2048 x 512: 26.2 and 27.2), but costs more than that in
// longer rows (8 x 3584 x 7168: 10.8 and 10.0; 8 x 7168 x 7168: 18.2 and 14.8) and
// where experts have more rows than an item (30 x 16 of 20, 2048 x 1024: 30 and 22).
constexpr int kFusedItem = 16, kFusedRows = 512, kFusedSteps = 4;
inline bool is_fused(Way way, int64_t rows, int experts, int blocks, bool offsets) {
  if (way != kBrief || blocks > 8 * kFusedSteps) return false;
  return rows <= kFusedItem ||
         (offsets && (rows <= kStreamRows || (rows <= kFusedRows && rows <= kFusedItem * (int64_t)experts)));
}

// What the streaming kernel uses of the workspace: counters of its column
// groups, zero between calls, 64 bytes apart, and split sums, a unit of them
// for each block.
constexpr int kSplitUnits = 256, kUnitInts = kStreamRows * 64;
static_assert(kSplitUnits * 64 <= EXPERTS_WORKSPACE_ZEROED, "what the caller clears");
constexpr size_t kPartialBytes = (size_t)kSplitUnits * kUnitInts * 4;

struct ProductArgs {
  const uint16_t* x;        // rows as they are
  const int8_t* q;          // as integers, stride 64 * blocks, zeros past the end
  const float* step;        // their scales
  const void* packed;
  const float* scale[2];    // [experts][n]; [1] for the gated product
  const void* bias;         // [experts][n]
  const void* residual;
  void* y;
  const int32_t* token;     // NULL: the row itself
  const int32_t* offsets;   // NULL: one expert has every row
  Lists lists;
  uint32_t* counters;
  int32_t* partial;
  int64_t ldx, ldr, ldy;
  int tokens, rows, experts, k, n, blocks, act, gated;
};
// Rows as integers; where there are offsets also the lists of a product of
// `rows` rows (area: list_bytes).
struct QuantiseArgs {
  const uint16_t* x;
  int8_t* q;
  float* step;
  const int32_t* offsets;
  Item* area;
  int64_t ldx;
  int tokens, k, stride, experts, rows;
  bool sorted;  // x has a row for each row of y
  Way way;
  int most_brief, most_mid, most_tiles;
};
hipError_t launch_quantise(int dtype, const QuantiseArgs& args, hipStream_t stream);
// Brief items (without offsets every row, of kStreamRows at most).
hipError_t launch_stream(int dtype, const ProductArgs& args, bool fused, hipStream_t stream);
// Tiles and mid items (without offsets every row, as either).
hipError_t launch_tiles(int dtype, const ProductArgs& args, Way way, hipStream_t stream);

hipError_t launch_pack(const int8_t* const* w, int planes, void* packed, int experts, int k, int n,
                       hipStream_t stream);
hipError_t launch_quantise_weights(int dtype, const void* w, int8_t* w8, float* scale, int experts, int k, int n,
                                   hipStream_t stream);

}  // namespace experts
