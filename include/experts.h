/*
 * experts.h - C ABI of the routed half of a layer, on one AMD Instinct MI355X
 * (gfx950): what follows the route (route.h) on its way through the experts.
 * Same library (libroute.so), status codes and conventions as route.h and
 * block.h, whose block_dtype and block_act these operators use.
 *
 * A router gives each of `rows` tokens `topk` choices, ids [rows][topk]. A plan
 * has the experts first .. first + experts - 1 (all of them, or one rank's
 * share); a choice of any other id, negative ones included, is dropped.
 *
 *   sort      the kept choices, numbered r * topk + j, in the order of (expert,
 *             number):
 *               offsets [experts + 1]  offsets[e] of them belong to experts
 *                                      before e, so that those of e are the
 *                                      positions offsets[e] .. offsets[e + 1] - 1
 *               place [rows][topk]     the position of a choice, -1 if dropped
 *               token [capacity]       the row r of a position
 *   gather    xs[place[r, j]] = x[r]
 *   backward  dx[r] = sum_j dxs[place[r, j]]
 *   combine   y[r] = sum_j weights[r, j] * ys[place[r, j]] + residual[r]
 *   backward  dys[place[r, j]] = weights[r, j] * dy[r],
 *             dweights[r, j] = sum_c dy[r, c] * ys[place[r, j], c], 0 if dropped
 *             (the residual's gradient is dy itself)
 *
 * Sums in FP32, in the order of j (dweights: in one fixed order), every output
 * rounded once, nearest-even. A dropped choice is not read: whatever its
 * weight holds, it adds nothing, and a row with none left is 0 (or the
 * residual). Rows of xs, dys and token at positions that no choice has are left
 * as they were. `capacity` is the number of rows that a buffer in sorted order
 * (xs, ys, dxs, dys, token) has: rows * topk hold everything; with fewer, the
 * choices placed at `capacity` or beyond are dropped by every call alike.
 *
 * Products in 8-bit integers, of `rows` sorted rows or of plain ones. A row of
 * x in BF16 or F16 becomes integers with one scale, the weights are integers
 * with a scale for each expert and output channel:
 *   a = max_k |x[t, k]|,  q[k] = rne(127 x[t, k] / a),  s = a / 127
 *   linear8   z = (sum_k q[k] W[e][k, n]) * s * scale[e][n] + bias[e][n],
 *             y = act(z) + residual
 *   gated8    g and u are two such products without bias, h = act(g) * u
 * The integer sums are exact; what follows is FP32, the sum times the channel's
 * scale first, and rounded once. A row of zeros has s = 0. A row that holds an
 * infinity or NaN gives NaN throughout.
 * Row p of y is of the expert whose range of `offsets` holds p, and of row
 * t = token[p] of x (token NULL: t = p). With `offsets` NULL, in a plan of one
 * expert, every row is that expert's. Rows at offsets[experts] and beyond are
 * left as they were. Serving only: there is no backward pass through rounding.
 *
 * Weights W are int8 [experts][K][N] row-major; any values, -128 included. They
 * are laid out once by *_pack (experts_*_packed_bytes) for the matrix cores;
 * the run calls read only the packed form. *_quantize makes W and the scales
 * (max_k |w| / 127) from 16-bit weights by the same rule as for rows; a
 * channel that holds an infinity or NaN gets a scale of NaN.
 *
 * Any size and element-aligned pointer is accepted; row strides are as in
 * block.h. `place`, `token` and `offsets` are read on the device and not
 * trusted: entries out of range are dropped (place), clamped (token) or cut
 * (offsets: the last to 0..rows, the others to 0 and the last), so that no
 * access leaves the buffers. Rows that the ranges of several experts hold get no
 * defined values.
 *
 * Ownership, threading, capture: as in block.h. Run calls only enqueue kernels
 * on `stream` and can be captured into a HIP graph. The first
 * EXPERTS_WORKSPACE_ZEROED bytes of a linear8 or gated8 plan's workspace
 * (256-byte aligned) are zero-filled once before its first use and must not be
 * modified between calls; the rest, and a sort's, may hold anything. Calls that
 * overlap in time use different workspaces. Every call takes 0..(plan rows)
 * rows; with 0 rows sort writes zero offsets and the others do nothing. Results
 * do not depend on timing. An output may share memory with no other argument,
 * except that y may be the residual (same pointer and stride).
 */
#ifndef EXPERTS_H
#define EXPERTS_H

#include "block.h"

#ifdef __cplusplus
extern "C" {
#endif

#define EXPERTS_ABI_VERSION 1u
#define EXPERTS_MAX_COUNT 4096      /* experts of a plan */
#define EXPERTS_MAX_TOPK 64
#define EXPERTS_MAX_CHOICES 16777216 /* 2^24: rows * topk, rows of a product */
#define EXPERTS_MAX_INPUTS 131071   /* K of the 8-bit products: 2^14 K < 2^31 */
#define EXPERTS_WORKSPACE_ZEROED 65536 /* bytes */

/* The *_prepare calls check, in this order and before any HIP call: cfg and
 * out non-NULL, abi_version, dtype, activation (ROUTE_E_ARG); sizes, topk and
 * experts (ROUTE_E_SHAPE); rows, tokens and rows * topk (ROUTE_E_ROWS); then
 * the device must exist and be gfx950 (ROUTE_E_DEVICE). On error *out is NULL.
 *
 * The run calls check: required pointers (ROUTE_E_ARG), rows, tokens and
 * capacity (ROUTE_E_ROWS), strides (ROUTE_E_SHAPE), element alignment of every
 * pointer and 256-byte alignment of workspace and packed weights
 * (ROUTE_E_ALIGN), then the current device (ROUTE_E_DEVICE). An argument error
 * launches nothing. Pointers to row matrices may be NULL where there are 0
 * rows. */

/* ------------------------------------------------------------------ sort -- */

typedef struct {
  uint32_t abi_version; /* EXPERTS_ABI_VERSION */
  int32_t device;       /* HIP device ordinal */
  int32_t rows;         /* the most rows any call on this plan passes */
  int32_t topk;         /* 1..EXPERTS_MAX_TOPK */
  int32_t experts;      /* 1..EXPERTS_MAX_COUNT */
  int32_t first;        /* id of the first of them, >= 0 */
} experts_sort_config;

typedef struct experts_sort_plan experts_sort_plan;

int experts_sort_prepare(const experts_sort_config* cfg, experts_sort_plan** out);
size_t experts_sort_workspace_bytes(const experts_sort_plan* plan); /* at least 256 */
int experts_sort(const experts_sort_plan* plan, const int32_t* ids, int32_t* offsets, int32_t* place,
                 int32_t* token, void* workspace, int32_t capacity, int32_t rows, void* stream);
void experts_sort_destroy(experts_sort_plan* plan);

/* --------------------------------------------------------------- combine -- */

typedef struct {
  uint32_t abi_version;
  int32_t device;
  int32_t rows;
  int32_t topk;
  int32_t width;
  int32_t dtype;        /* block_dtype of x, xs, ys, y and their gradients */
} experts_combine_config;

typedef struct experts_combine_plan experts_combine_plan;

int experts_combine_prepare(const experts_combine_config* cfg, experts_combine_plan** out);
int experts_gather(const experts_combine_plan* plan, const void* x, int64_t x_stride, const int32_t* place,
                   void* xs, int64_t xs_stride, int32_t capacity, int32_t rows, void* stream);
int experts_gather_backward(const experts_combine_plan* plan, const void* dxs, int64_t dxs_stride,
                            const int32_t* place, void* dx, int64_t dx_stride, int32_t capacity,
                            int32_t rows, void* stream);
/* weights [rows][topk] FP32; residual may be NULL. */
int experts_combine(const experts_combine_plan* plan, const void* ys, int64_t ys_stride, const int32_t* place,
                    const float* weights, const void* residual, int64_t residual_stride, void* y,
                    int64_t y_stride, int32_t capacity, int32_t rows, void* stream);
/* dys or dweights may be NULL (not computed), not both; ys is read for
 * dweights only, weights for dys only, and either may be NULL otherwise. */
int experts_combine_backward(const experts_combine_plan* plan, const void* dy, int64_t dy_stride, const void* ys,
                             int64_t ys_stride, const int32_t* place, const float* weights, void* dys,
                             int64_t dys_stride, float* dweights, int32_t capacity, int32_t rows,
                             void* stream);
void experts_combine_destroy(experts_combine_plan* plan);

/* --------------------------------------------------------------- linear8 -- */

typedef struct {
  uint32_t abi_version;
  int32_t device;
  int32_t rows;        /* 1..EXPERTS_MAX_CHOICES: the most rows of y */
  int32_t tokens;      /* 1..EXPERTS_MAX_CHOICES: the most rows of x */
  int32_t inputs;      /* K: 1..EXPERTS_MAX_INPUTS */
  int32_t outputs;     /* N */
  int32_t experts;
  int32_t dtype;       /* BLOCK_BF16 or BLOCK_F16 */
  int32_t activation;  /* block_act */
} experts_linear8_config;

typedef struct experts_linear8_plan experts_linear8_plan;

int experts_linear8_prepare(const experts_linear8_config* cfg, experts_linear8_plan** out);
size_t experts_linear8_workspace_bytes(const experts_linear8_plan* plan);
size_t experts_linear8_packed_bytes(const experts_linear8_plan* plan);
int experts_linear8_quantize(const experts_linear8_plan* plan, const void* w, int8_t* w8, float* scale,
                             void* stream);
int experts_linear8_pack(const experts_linear8_plan* plan, const int8_t* w, void* packed, void* stream);
/* scale [experts][outputs] FP32, bias [experts][outputs] of dtype; bias,
 * residual and token may each be NULL, offsets in a plan of one expert. Without
 * token, tokens has to be rows. */
int experts_linear8(const experts_linear8_plan* plan, const void* x, int64_t x_stride, const void* packed,
                    const float* scale, const int32_t* offsets, const int32_t* token, const void* bias,
                    const void* residual, int64_t residual_stride, void* y, int64_t y_stride, void* workspace,
                    int32_t tokens, int32_t rows, void* stream);
void experts_linear8_destroy(experts_linear8_plan* plan);

/* ---------------------------------------------------------------- gated8 -- */

typedef struct {
  uint32_t abi_version;
  int32_t device;
  int32_t rows;
  int32_t tokens;
  int32_t inputs;
  int32_t inner;       /* N: columns of h */
  int32_t experts;
  int32_t dtype;
  int32_t activation;  /* block_act other than BLOCK_ACT_NONE */
} experts_gated8_config;

typedef struct experts_gated8_plan experts_gated8_plan;

int experts_gated8_prepare(const experts_gated8_config* cfg, experts_gated8_plan** out);
size_t experts_gated8_workspace_bytes(const experts_gated8_plan* plan);
size_t experts_gated8_packed_bytes(const experts_gated8_plan* plan);
int experts_gated8_quantize(const experts_gated8_plan* plan, const void* w, int8_t* w8, float* scale,
                            void* stream);
int experts_gated8_pack(const experts_gated8_plan* plan, const int8_t* w_gate, const int8_t* w_up, void* packed,
                        void* stream);
int experts_gated8(const experts_gated8_plan* plan, const void* x, int64_t x_stride, const void* packed,
                   const float* scale_gate, const float* scale_up, const int32_t* offsets, const int32_t* token,
                   void* h, int64_t h_stride, void* workspace, int32_t tokens, int32_t rows, void* stream);
void experts_gated8_destroy(experts_gated8_plan* plan);

#ifdef __cplusplus
}
#endif

#endif
