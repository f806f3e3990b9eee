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

// The rows of one expert in a product: up to kStreamRows of them (a short item,
// for the kernel that streams weights), or its first-th and later row tiles (an
// entry for each tile; `rows` is of all of them).
struct Item {
  int32_t expert, row, rows, first;
};
constexpr int kStreamRows = 32, kTileRows = 256;
struct Lists {
  const int32_t* counts;  // short items, row tiles; NULL: one expert has every row
  const Item* brief;
  const Item* tiles;
};
inline int64_t most_brief(int64_t rows, int experts) { return rows < experts ? rows : experts; }
inline int64_t most_tiles(int64_t rows, int experts) {
  const int64_t long_ones = rows / (kStreamRows + 1);
  return rows / kTileRows + (long_ones < experts ? long_ones : experts);
}
inline size_t list_bytes(int64_t rows, int experts) {
  return sizeof(Item) * (size_t)(1 + most_brief(rows, experts) + most_tiles(rows, experts));
}
inline Lists lists_at(void* area, int64_t rows, int experts) {
  const Item* items = static_cast<const Item*>(area);
  return Lists{&items->expert, items + 1, items + 1 + most_brief(rows, experts)};
}

// What the streaming kernel uses of the workspace: counters of its column
// groups, zero between calls, 64 bytes apart, and split sums, a unit of them
// for each block.
constexpr int kSplitUnits = 256, kUnitInts = kStreamRows * 64;
static_assert(kSplitUnits * 64 <= EXPERTS_WORKSPACE_ZEROED, "what the caller clears");
constexpr size_t kPartialBytes = (size_t)kSplitUnits * kUnitInts * 4;

struct ProductArgs {
  const int8_t* q;          // rows of x as integers, stride 64 * blocks, zeros past the end
  const float* step;        // their scales
  const void* packed;
  const float* scale[2];    // [experts][n]; [1] for the gated product
  const void* bias;         // [experts][n]
  const void* residual;
  void* y;
  const int32_t* token;     // NULL: the row itself
  Lists lists;
  uint32_t* counters;
  int32_t* partial;
  int64_t ldr, ldy;
  int tokens, rows, n, blocks, act, gated;
};
// Also makes the lists (area: list_bytes) where there are offsets.
hipError_t launch_quantise(int dtype, const void* x, int64_t ldx, int tokens, int k, int8_t* q, float* step,
                           const int32_t* offsets, int experts, int rows, void* area, hipStream_t stream);
// Experts of 1..kStreamRows rows, and those of more.
hipError_t launch_stream(int dtype, const ProductArgs& args, int experts, hipStream_t stream);
hipError_t launch_tiles(int dtype, const ProductArgs& args, int experts, hipStream_t stream);

hipError_t launch_pack(const int8_t* const* w, int planes, void* packed, int experts, int k, int n,
                       hipStream_t stream);
hipError_t launch_quantise_weights(int dtype, const void* w, int8_t* w8, float* scale, int experts, int k, int n,
                                   hipStream_t stream);

}  // namespace experts
