// Host-side launchers of the layer's operators (called by the C ABI in
// block_api.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "block.h"
#include "route_launch.h"

namespace block {

using route::launch_kernel;

// The four products. Every one is C[m][n] = sum over r of A(m, r) * B(r, n),
// with r running over `segments` pairs of operands of length `red` each:
//   kLinear  A = x (r contiguous),  B = W       (n contiguous), 1 segment
//   kGated   the same with two B matrices, whose sums meet in the epilogue
//   kDx      A = dz (r contiguous), B = W^T     (r contiguous), 1 or 2 segments
//   kDw      A = x^T (m contiguous), B = dz     (n contiguous), `outputs`
//            pairs of B and C
enum Mode { kLinear = 0, kGated = 1, kDx = 2, kDw = 3 };

struct GemmArgs {
  const void* a[2];
  const void* b[2];
  void* c[2];
  void* saved[2];        // kGated: d_gate, d_up; kLinear: slope; row stride n
  const void* bias;
  const void* residual;
  int64_t lda, ldb, ldc, ldr;
  int64_t m;
  int n;
  int64_t red;
  int segments;
  int outputs;
  int act;
};

// What a product uses of its operator's workspace: a counter per column tile,
// 64 bytes apart, zero between calls, and an area for split sums.
struct Workspace {
  uint32_t* counters;
  float* partial;
  size_t partial_bytes;
};
constexpr size_t kCounterBytes = (size_t)(BLOCK_MAX_SIZE / 64) * 64;
static_assert(kCounterBytes == BLOCK_WORKSPACE_ZEROED, "what the caller clears");

hipError_t launch_gemm(int dtype, Mode mode, const GemmArgs& args, const Workspace& ws, hipStream_t stream);
// Whether launch_gemm takes the operands as they are (few rows). The other
// products want them copied where needs_copy says so, but for weights at an
// unaligned address whose rows are a multiple of 8 long: contiguous lengths
// are, or are zero-padded to, multiples of 8 in memory.
bool gemm_streams(Mode mode, int64_t m, int64_t n, int64_t red);
// The most that products of up to m rows (dw: of m rows, and a reduction of up
// to `red`) can use for split sums.
size_t gemm_partial_bytes(Mode mode, int64_t m, int n, int64_t red, int segments, int outputs);

// Tile kernel: every operand 16-byte aligned, with row strides that are
// multiples of 8 and contiguous lengths that are, or are zero-padded to,
// multiples of 8. shape 0..2 and K split.
struct TilePlan {
  int shape;
  int splits;
};
TilePlan plan_tiles(Mode mode, const GemmArgs& args, size_t partial_bytes);
int most_tile_splits(int64_t red, int segments);
hipError_t launch_gemm_tile(int dtype, Mode mode, const GemmArgs& args, const TilePlan& plan, float* partial,
                            hipStream_t stream);

// A copy of a matrix of 16-bit values that the tile kernel can read: rows of
// `len` values padded with zeros to a multiple of 8, which is the stride.
struct Copy {
  const void* src;
  void* dst;
  int64_t ld, rows;
  int len;
};
hipError_t launch_copies(const Copy* copies, int count, hipStream_t stream);
inline bool needs_copy(const void* p, int64_t ld, int64_t len) {
  return (reinterpret_cast<uintptr_t>(p) & 15) != 0 || ((ld | len) & 7) != 0;
}

// Adds the splits' sums [splits][planes][m][n rounded up to 4] in split order
// and ends the product (planes: 2 for kGated, else `outputs`).
hipError_t launch_gemm_join(int dtype, Mode mode, const GemmArgs& args, int splits, const float* partial,
                            hipStream_t stream);

// At most kStreamRows rows; not kDw.
constexpr int kStreamRows = 32;
int most_stream_splits(Mode mode, int n, int64_t red, int segments);
hipError_t launch_gemm_stream(int dtype, Mode mode, const GemmArgs& args, const Workspace& ws, hipStream_t stream);

// out[k] [rows][ld] = dy * s[k] for `count` (0..2) matrices of derivatives
// [rows][n]; out[k] may be NULL. With dbias [n] (count 0 or 1), also the column
// sums, through `partial` (column_sum_bytes).
hipError_t launch_scale(int dtype, const void* dy, int64_t dy_stride, const void* const* s, int count,
                        void* const* out, int64_t ld, int64_t rows, int n, void* dbias, float* partial,
                        hipStream_t stream);
size_t column_sum_bytes(int64_t rows, int n);

struct NormArgs {
  const void* x;
  const void* dy;
  const void* weight;
  const void* bias;
  void* y;
  void* dx;
  void* dweight;
  void* dbias;
  float* mean;
  float* rstd;
  float* partial;
  int64_t ldx, lddy, ldy, lddx;
  int64_t rows;
  int width;
  int param_dtype;
  float eps;
};

hipError_t launch_norm(int dtype, const NormArgs& args, hipStream_t stream);
hipError_t launch_norm_backward(int dtype, const NormArgs& args, hipStream_t stream);
size_t norm_backward_bytes(int dtype, int64_t rows, int width);

}  // namespace block
