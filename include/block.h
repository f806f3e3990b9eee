/*
 * block.h - C ABI of the operators that stand around the route in a layer, on
 * one AMD Instinct MI355X (gfx950): layer norm, the gated feed-forward
 * product, and the linear product with bias, activation and residual, each
 * forward and backward. Same library (libroute.so), status codes and
 * conventions as route.h; route_strerror describes every status.
 *
 * For each row r (sums in FP32, every output rounded once, nearest-even):
 *
 *   norm      mean = sum_i x[r,i] / W,  var = sum_i (x[r,i] - mean)^2 / W,
 *             rstd = 1 / sqrt(var + eps),  xh = (x - mean) * rstd,
 *             y = xh * weight + bias
 *   backward  dx = rstd * (weight*dy - mean_i(weight*dy)
 *                          - xh * mean_i(weight*dy*xh)),
 *             dweight = sum_r dy * xh,  dbias = sum_r dy
 *
 *   gated     g = x Wg,  u = x Wu,  h = act(g) * u
 *             for training also d_gate = u * act'(g) and d_up = act(g): the
 *             derivatives of h, which are all that its backward needs
 *   backward  dg = dh * d_gate,  du = dh * d_up,
 *             dx = dg Wg^T + du Wu^T,  dWg = x^T dg,  dWu = x^T du
 *
 *   linear    z = x W + bias,  y = act(z) + residual
 *             for training with an activation also slope = act'(z)
 *   backward  dz = dy * slope,  dx = dz W^T,  dW = x^T dz,
 *             dbias = sum_r dz  (the residual's gradient is dy itself)
 *
 * Types: `dtype` is that of the activations, their gradients, the matrices
 * and the matrices' gradients: BLOCK_BF16 or BLOCK_F16, for the norm also
 * BLOCK_F32. The norm's weight and bias and their gradients have
 * `param_dtype` (any of the three); mean and rstd are FP32. Products are
 * accumulated in FP32. dg, du and dz are rounded to `dtype` before the
 * backward products, which run on the matrix cores, and the derivatives kept
 * for them are of `dtype` as well: with the result's own rounding, gradients go
 * through three, and have an RMS error of 1.7-1.8 times one rounding's (dbias,
 * summed from the unrounded dz: 1.5 times).
 *
 * Layouts: matrices of weights are [K][N] row-major and contiguous. A matrix
 * of rows (x, y, h, residual and the gradients dy, dh, dx) is row-major with
 * the row stride given in elements beside its pointer (at least its width, at
 * most BLOCK_MAX_STRIDE). d_gate, d_up and slope are contiguous
 * [rows][inner | outputs]. Any size, stride and element-aligned pointer is
 * accepted. Above 32 rows, 16-byte aligned pointers with sizes and strides
 * that are multiples of 8 are fastest: other operands are copied first, into
 * the workspace (which holds room for the rows, and for weights whose rows
 * are no multiple of 8 long), and weights whose rows are a multiple of 8 long
 * at an address that is no multiple of 16 take a kernel of a fifth of the
 * rate (of a ninth at 33 rows).
 *
 * Ownership, threading, capture: as in route.h. The caller owns every buffer,
 * run calls only enqueue kernels on `stream` and can be captured into a HIP
 * graph. The first BLOCK_WORKSPACE_ZEROED bytes of a gated or linear plan's
 * workspace (block_*_workspace_bytes, 256-byte aligned) are zero-filled once
 * before its first use and must not be modified between calls; the rest, and
 * the norm's, may hold anything. Calls that overlap in time use different
 * workspaces. A call passes 0..(plan rows) rows: with 0 rows the forward calls
 * do nothing, the backward calls write zero weight gradients, and row matrices
 * may be NULL. Results do not depend on timing: every sum has a fixed order for
 * a given plan, row count and alignment. An output may share memory with no
 * other argument, except that y of block_linear may be the residual (same
 * pointer and stride).
 */
#ifndef BLOCK_H
#define BLOCK_H

#include "route.h"

#ifdef __cplusplus
extern "C" {
#endif

#define BLOCK_ABI_VERSION 1u
#define BLOCK_MAX_ROWS 1048576   /* 2^20 */
#define BLOCK_MAX_SIZE 131072    /* width, inputs, inner, outputs */
#define BLOCK_MAX_STRIDE 1048576 /* elements */
#define BLOCK_WORKSPACE_ZEROED 131072 /* bytes */

typedef enum { BLOCK_BF16 = 0, BLOCK_F16 = 1, BLOCK_F32 = 2 } block_dtype;
typedef enum {
  BLOCK_ACT_NONE = 0,     /* z (linear only) */
  BLOCK_ACT_RELU = 1,     /* max(z, 0), derivative 0 at 0 */
  BLOCK_ACT_SILU = 2,     /* z / (1 + exp(-z)) */
  BLOCK_ACT_GELU = 3,     /* z (1 + erf(z / sqrt 2)) / 2 */
  BLOCK_ACT_GELU_TANH = 4 /* z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) / 2 */
} block_act;

/* ------------------------------------------------------------------ norm -- */

typedef struct {
  uint32_t abi_version; /* BLOCK_ABI_VERSION */
  int32_t device;       /* HIP device ordinal */
  int32_t rows;         /* the most rows any call on this plan passes */
  int32_t width;
  int32_t dtype;        /* block_dtype */
  int32_t param_dtype;  /* block_dtype of weight, bias and their gradients */
  float eps;            /* finite and > 0 */
} block_norm_config;

typedef struct block_norm_plan block_norm_plan;

/* The *_prepare calls check, in this order and before any HIP call: cfg and
 * out non-NULL, abi_version, dtypes, activation, eps (ROUTE_E_ARG); sizes
 * (ROUTE_E_SHAPE); rows in 1..BLOCK_MAX_ROWS (ROUTE_E_ROWS); then the device
 * must exist and be gfx950 (ROUTE_E_DEVICE). On error *out is NULL.
 *
 * The run calls check: required pointers (ROUTE_E_ARG), rows in 0..plan rows
 * (ROUTE_E_ROWS), strides (ROUTE_E_SHAPE), element alignment of every pointer
 * and 256-byte alignment of the workspace (ROUTE_E_ALIGN), a forward-only
 * plan given to a training call (ROUTE_E_ARG), then the current device
 * (ROUTE_E_DEVICE). An argument error launches nothing. */
int block_norm_prepare(const block_norm_config* cfg, block_norm_plan** out);
size_t block_norm_workspace_bytes(const block_norm_plan* plan); /* for the backward call; at least 256 */
/* weight and bias may each be NULL (1 and 0); mean and rstd (both or neither)
 * are kept for the backward call. */
int block_norm(const block_norm_plan* plan, const void* x, int64_t x_stride, const void* weight,
               const void* bias, void* y, int64_t y_stride, float* mean, float* rstd, int32_t rows,
               void* stream);
/* weight may be NULL (1); dx, dweight and dbias may each be NULL (not
 * computed), but not all three. */
int block_norm_backward(const block_norm_plan* plan, const void* dy, int64_t dy_stride, const void* x,
                        int64_t x_stride, const void* weight, const float* mean, const float* rstd,
                        void* dx, int64_t dx_stride, void* dweight, void* dbias, void* workspace,
                        int32_t rows, void* stream);
void block_norm_destroy(block_norm_plan* plan);

/* ----------------------------------------------------------------- gated -- */

typedef struct {
  uint32_t abi_version;
  int32_t device;
  int32_t rows;
  int32_t inputs;      /* K: columns of x */
  int32_t inner;       /* N: columns of h */
  int32_t dtype;       /* BLOCK_BF16 or BLOCK_F16 */
  int32_t activation;  /* block_act other than BLOCK_ACT_NONE */
  int32_t training;    /* nonzero: the workspace also serves the backward call */
} block_gated_config;

typedef struct block_gated_plan block_gated_plan;

int block_gated_prepare(const block_gated_config* cfg, block_gated_plan** out);
size_t block_gated_workspace_bytes(const block_gated_plan* plan);
/* d_gate and d_up: both or neither. */
int block_gated(const block_gated_plan* plan, const void* x, int64_t x_stride, const void* w_gate,
                const void* w_up, void* h, int64_t h_stride, void* d_gate, void* d_up, void* workspace,
                int32_t rows, void* stream);
/* dx may be NULL; dw_gate and dw_up: both or neither; not all NULL. */
int block_gated_backward(const block_gated_plan* plan, const void* dh, int64_t dh_stride, const void* x,
                         int64_t x_stride, const void* w_gate, const void* w_up, const void* d_gate,
                         const void* d_up, void* dx, int64_t dx_stride, void* dw_gate, void* dw_up,
                         void* workspace, int32_t rows, void* stream);
void block_gated_destroy(block_gated_plan* plan);

/* ---------------------------------------------------------------- linear -- */

typedef struct {
  uint32_t abi_version;
  int32_t device;
  int32_t rows;
  int32_t inputs;
  int32_t outputs;
  int32_t dtype;       /* BLOCK_BF16 or BLOCK_F16 */
  int32_t activation;  /* block_act */
  int32_t training;
} block_linear_config;

typedef struct block_linear_plan block_linear_plan;

int block_linear_prepare(const block_linear_config* cfg, block_linear_plan** out);
size_t block_linear_workspace_bytes(const block_linear_plan* plan);
/* bias [outputs], residual and slope may each be NULL. */
int block_linear(const block_linear_plan* plan, const void* x, int64_t x_stride, const void* w,
                 const void* bias, const void* residual, int64_t residual_stride, void* y,
                 int64_t y_stride, void* slope, void* workspace, int32_t rows, void* stream);
/* slope is required when the plan has an activation and ignored otherwise;
 * dx, dw and dbias may each be NULL, but not all three. */
int block_linear_backward(const block_linear_plan* plan, const void* dy, int64_t dy_stride, const void* x,
                          int64_t x_stride, const void* w, const void* slope, void* dx, int64_t dx_stride,
                          void* dw, void* dbias, void* workspace, int32_t rows, void* stream);
void block_linear_destroy(block_linear_plan* plan);

#ifdef __cplusplus
}
#endif

#endif
