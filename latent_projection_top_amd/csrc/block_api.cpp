// C ABI of the layer's operators (block.h): plan preparation, argument checks
// and launches. Every check runs before any launch; nothing allocates device
// memory or synchronises.
#include "block.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>

#include "block_launch.h"

struct block_norm_plan {
  block_norm_config cfg;
  size_t ws_bytes;
};

// Workspace of the matrix operators: the products' counters, their split sums
// (up to off_dz), then dz (linear) or dg and du (gated) with their rows padded
// to a multiple of 8 elements, the partial column sums of dbias, and padded
// copies of x and (if their rows are no multiple of 8) the weights.
struct block_gated_plan {
  block_gated_config cfg;
  size_t partial_bytes, off_dz, off_du, off_x, off_w, w_bytes, ws_bytes;
};

struct block_linear_plan {
  block_linear_config cfg;
  size_t partial_bytes, off_dz, off_sum, off_x, off_w, w_bytes, ws_bytes;
};

namespace {

using block::GemmArgs;

bool misaligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }
size_t round256(size_t n) { return (n + 255) & ~size_t(255); }
size_t dtype_size(int dtype) { return dtype == BLOCK_F32 ? 4 : 2; }
int64_t padded(int n) { return (n + 7) & ~int64_t(7); }
bool bad_size(int32_t n) { return n < 1 || n > BLOCK_MAX_SIZE; }
bool bad_rows(int32_t n) { return n < 1 || n > BLOCK_MAX_ROWS; }
bool bad_stride(int64_t s, int64_t width) { return s < width || s > BLOCK_MAX_STRIDE; }
int status_of(hipError_t e) { return e == hipSuccess ? ROUTE_OK : ROUTE_E_HIP; }

int find_device(int32_t device) {
  int count = 0;
  if (device < 0 || hipGetDeviceCount(&count) != hipSuccess || device >= count) return ROUTE_E_DEVICE;
  hipDeviceProp_t prop;
  if (hipGetDeviceProperties(&prop, device) != hipSuccess) return ROUTE_E_DEVICE;
  return std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? ROUTE_OK : ROUTE_E_DEVICE;
}

int check_current(int32_t device) {
  int cur = -1;
  return hipGetDevice(&cur) == hipSuccess && cur == device ? ROUTE_OK : ROUTE_E_DEVICE;
}

// The most any of an operator's products can use for split sums: its forward
// product and, for training, dx [rows][k] and dw `outputs` x [k][n].
size_t partial_area(block::Mode mode, int64_t rows, int k, int n, int outputs, bool training) {
  size_t b = block::gemm_partial_bytes(mode, rows, n, k, 1, 1);
  if (training) {
    b = std::max(b, block::gemm_partial_bytes(block::kDx, rows, k, n, outputs, 1));
    b = std::max(b, block::gemm_partial_bytes(block::kDw, k, n, rows, 1, outputs));
  }
  return round256(b);
}

template <typename Plan>
block::Workspace products(const Plan* plan, void* workspace) {
  char* base = static_cast<char*>(workspace);
  return block::Workspace{reinterpret_cast<uint32_t*>(base), reinterpret_cast<float*>(base + block::kCounterBytes),
                          plan->partial_bytes};
}

// The copies a call makes so that the tile kernel can read its operands.
struct Copies {
  block::Copy c[3];
  int n = 0;
  // *p, [rows][len] of stride *ld, is copied to dst if it has to be (and dst
  // is there); *p and *ld then describe the copy.
  void use(const void** p, int64_t* ld, int64_t rows, int len, void* dst) {
    if (dst == nullptr || !block::needs_copy(*p, *ld, len)) return;
    c[n++] = block::Copy{*p, dst, *ld, rows, len};
    *p = dst;
    *ld = padded(len);
  }
  int launch(hipStream_t s) const { return status_of(block::launch_copies(c, n, s)); }
};

template <typename Plan, typename Config>
Plan* new_plan(const Config& cfg) {
  Plan* p = new (std::nothrow) Plan();
  if (p != nullptr) p->cfg = cfg;
  return p;
}

}  // namespace

extern "C" {

// ------------------------------------------------------------------- norm --

int block_norm_prepare(const block_norm_config* cfg, block_norm_plan** out) {
  if (out == nullptr) return ROUTE_E_ARG;
  *out = nullptr;
  if (cfg == nullptr || cfg->abi_version != BLOCK_ABI_VERSION) return ROUTE_E_ARG;
  if (cfg->dtype < BLOCK_BF16 || cfg->dtype > BLOCK_F32 || cfg->param_dtype < BLOCK_BF16 ||
      cfg->param_dtype > BLOCK_F32 || !std::isfinite(cfg->eps) || !(cfg->eps > 0.f))
    return ROUTE_E_ARG;
  if (bad_size(cfg->width)) return ROUTE_E_SHAPE;
  if (bad_rows(cfg->rows)) return ROUTE_E_ROWS;
  if (int st = find_device(cfg->device)) return st;
  block_norm_plan* p = new_plan<block_norm_plan>(*cfg);
  if (p == nullptr) return ROUTE_E_ARG;
  // never 0: the backward call takes no NULL workspace, and an allocation of 0
  // bytes is one
  p->ws_bytes = std::max<size_t>(round256(block::norm_backward_bytes(cfg->dtype, cfg->rows, cfg->width)), 256);
  *out = p;
  return ROUTE_OK;
}

size_t block_norm_workspace_bytes(const block_norm_plan* plan) { return plan ? plan->ws_bytes : 0; }

int block_norm(const block_norm_plan* plan, const void* x, int64_t x_stride, const void* weight,
               const void* bias, void* y, int64_t y_stride, float* mean, float* rstd, int32_t rows,
               void* stream) {
  if (!plan || (mean == nullptr) != (rstd == nullptr)) return ROUTE_E_ARG;
  if (rows != 0 && (!x || !y)) return ROUTE_E_ARG;
  const block_norm_config& c = plan->cfg;
  if (rows < 0 || rows > c.rows) return ROUTE_E_ROWS;
  if (bad_stride(x_stride, c.width) || bad_stride(y_stride, c.width)) return ROUTE_E_SHAPE;
  const size_t e = dtype_size(c.dtype), pe = dtype_size(c.param_dtype);
  if (misaligned(x, e) || misaligned(y, e) || misaligned(weight, pe) || misaligned(bias, pe) ||
      misaligned(mean, 4) || misaligned(rstd, 4))
    return ROUTE_E_ALIGN;
  if (int st = check_current(c.device)) return st;
  if (rows == 0) return ROUTE_OK;
  block::NormArgs a{};
  a.x = x;
  a.ldx = x_stride;
  a.weight = weight;
  a.bias = bias;
  a.y = y;
  a.ldy = y_stride;
  a.mean = mean;
  a.rstd = rstd;
  a.rows = rows;
  a.width = c.width;
  a.param_dtype = c.param_dtype;
  a.eps = c.eps;
  return status_of(block::launch_norm(c.dtype, a, static_cast<hipStream_t>(stream)));
}

int block_norm_backward(const block_norm_plan* plan, const void* dy, int64_t dy_stride, const void* x,
                        int64_t x_stride, const void* weight, const float* mean, const float* rstd,
                        void* dx, int64_t dx_stride, void* dweight, void* dbias, void* workspace,
                        int32_t rows, void* stream) {
  if (!plan || !workspace || (!dx && !dweight && !dbias)) return ROUTE_E_ARG;
  if (rows != 0 && (!dy || !x || !mean || !rstd)) return ROUTE_E_ARG;
  const block_norm_config& c = plan->cfg;
  if (rows < 0 || rows > c.rows) return ROUTE_E_ROWS;
  if (bad_stride(dy_stride, c.width) || bad_stride(x_stride, c.width) ||
      (dx != nullptr && bad_stride(dx_stride, c.width)))
    return ROUTE_E_SHAPE;
  const size_t e = dtype_size(c.dtype), pe = dtype_size(c.param_dtype);
  if (misaligned(dy, e) || misaligned(x, e) || misaligned(dx, e) || misaligned(weight, pe) ||
      misaligned(dweight, pe) || misaligned(dbias, pe) || misaligned(mean, 4) || misaligned(rstd, 4) ||
      misaligned(workspace, 256))
    return ROUTE_E_ALIGN;
  if (int st = check_current(c.device)) return st;
  if (rows == 0 && !dweight && !dbias) return ROUTE_OK;
  block::NormArgs a{};
  a.x = x;
  a.ldx = x_stride;
  a.dy = dy;
  a.lddy = dy_stride;
  a.weight = weight;
  a.dx = dx;
  a.lddx = dx_stride;
  a.dweight = dweight;
  a.dbias = dbias;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.partial = static_cast<float*>(workspace);
  a.rows = rows;
  a.width = c.width;
  a.param_dtype = c.param_dtype;
  return status_of(block::launch_norm_backward(c.dtype, a, static_cast<hipStream_t>(stream)));
}

void block_norm_destroy(block_norm_plan* plan) { delete plan; }

// ------------------------------------------------------------------ gated --

int block_gated_prepare(const block_gated_config* cfg, block_gated_plan** out) {
  if (out == nullptr) return ROUTE_E_ARG;
  *out = nullptr;
  if (cfg == nullptr || cfg->abi_version != BLOCK_ABI_VERSION) return ROUTE_E_ARG;
  if ((cfg->dtype != BLOCK_BF16 && cfg->dtype != BLOCK_F16) || cfg->activation <= BLOCK_ACT_NONE ||
      cfg->activation > BLOCK_ACT_GELU_TANH)
    return ROUTE_E_ARG;
  if (bad_size(cfg->inputs) || bad_size(cfg->inner)) return ROUTE_E_SHAPE;
  if (bad_rows(cfg->rows)) return ROUTE_E_ROWS;
  if (int st = find_device(cfg->device)) return st;
  block_gated_plan* p = new_plan<block_gated_plan>(*cfg);
  if (p == nullptr) return ROUTE_E_ARG;
  p->partial_bytes = partial_area(block::kGated, cfg->rows, cfg->inputs, cfg->inner, 2, cfg->training != 0);
  const size_t dz = cfg->training ? round256((size_t)cfg->rows * padded(cfg->inner) * 2) : 0;
  p->off_dz = block::kCounterBytes + p->partial_bytes;
  p->off_du = p->off_dz + dz;
  p->off_x = p->off_du + dz;
  p->off_w = p->off_x + round256((size_t)cfg->rows * padded(cfg->inputs) * 2);
  p->w_bytes = (cfg->inner & 7) != 0 ? round256((size_t)cfg->inputs * padded(cfg->inner) * 2) : 0;
  p->ws_bytes = p->off_w + 2 * p->w_bytes;
  *out = p;
  return ROUTE_OK;
}

size_t block_gated_workspace_bytes(const block_gated_plan* plan) { return plan ? plan->ws_bytes : 0; }

int block_gated(const block_gated_plan* plan, const void* x, int64_t x_stride, const void* w_gate,
                const void* w_up, void* h, int64_t h_stride, void* d_gate, void* d_up, void* workspace,
                int32_t rows, void* stream) {
  if (!plan || !w_gate || !w_up || !workspace) return ROUTE_E_ARG;
  if (rows != 0 && (!x || !h || (d_gate == nullptr) != (d_up == nullptr))) return ROUTE_E_ARG;
  const block_gated_config& c = plan->cfg;
  if (rows < 0 || rows > c.rows) return ROUTE_E_ROWS;
  if (bad_stride(x_stride, c.inputs) || bad_stride(h_stride, c.inner)) return ROUTE_E_SHAPE;
  if (misaligned(x, 2) || misaligned(w_gate, 2) || misaligned(w_up, 2) || misaligned(h, 2) ||
      misaligned(d_gate, 2) || misaligned(d_up, 2) || misaligned(workspace, 256))
    return ROUTE_E_ALIGN;
  if (int st = check_current(c.device)) return st;
  if (rows == 0) return ROUTE_OK;
  GemmArgs a{};
  a.a[0] = x;
  a.lda = x_stride;
  a.b[0] = w_gate;
  a.b[1] = w_up;
  a.ldb = c.inner;
  a.c[0] = h;
  a.ldc = h_stride;
  a.saved[0] = d_gate;
  a.saved[1] = d_up;
  a.m = rows;
  a.n = c.inner;
  a.red = c.inputs;
  a.segments = a.outputs = 1;
  a.act = c.activation;
  if (!block::gemm_streams(block::kGated, rows, c.inner, c.inputs)) {
    char* ws = static_cast<char*>(workspace);
    Copies copies;
    int64_t ld = a.ldb;
    copies.use(&a.a[0], &a.lda, rows, c.inputs, ws + plan->off_x);
    copies.use(&a.b[0], &ld, c.inputs, c.inner, plan->w_bytes ? ws + plan->off_w : nullptr);
    copies.use(&a.b[1], &a.ldb, c.inputs, c.inner, plan->w_bytes ? ws + plan->off_w + plan->w_bytes : nullptr);
    if (int st = copies.launch(static_cast<hipStream_t>(stream))) return st;
  }
  return status_of(block::launch_gemm(c.dtype, block::kGated, a, products(plan, workspace),
                                      static_cast<hipStream_t>(stream)));
}

int block_gated_backward(const block_gated_plan* plan, const void* dh, int64_t dh_stride, const void* x,
                         int64_t x_stride, const void* w_gate, const void* w_up, const void* d_gate,
                         const void* d_up, void* dx, int64_t dx_stride, void* dw_gate, void* dw_up,
                         void* workspace, int32_t rows, void* stream) {
  if (!plan || !w_gate || !w_up || !workspace || !plan->cfg.training) return ROUTE_E_ARG;
  if ((dw_gate == nullptr) != (dw_up == nullptr)) return ROUTE_E_ARG;
  if (rows != 0 && (!dh || !x || !d_gate || !d_up || (!dx && !dw_gate))) return ROUTE_E_ARG;
  const block_gated_config& c = plan->cfg;
  if (rows < 0 || rows > c.rows) return ROUTE_E_ROWS;
  if (bad_stride(dh_stride, c.inner) || bad_stride(x_stride, c.inputs) ||
      (dx != nullptr && bad_stride(dx_stride, c.inputs)))
    return ROUTE_E_SHAPE;
  if (misaligned(dh, 2) || misaligned(x, 2) || misaligned(w_gate, 2) || misaligned(w_up, 2) ||
      misaligned(d_gate, 2) || misaligned(d_up, 2) || misaligned(dx, 2) || misaligned(dw_gate, 2) ||
      misaligned(dw_up, 2) || misaligned(workspace, 256))
    return ROUTE_E_ALIGN;
  if (int st = check_current(c.device)) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  void* dz[2] = {ws + plan->off_dz, ws + plan->off_du};
  const void* slopes[2] = {d_gate, d_up};
  int st = status_of(block::launch_scale(c.dtype, dh, dh_stride, slopes, 2, dz, padded(c.inner), rows, c.inner,
                                          nullptr, nullptr, s));
  if (st != ROUTE_OK) return st;
  Copies copies;
  int64_t ldg = c.inner, ldu = c.inner;
  if (dx != nullptr && !block::gemm_streams(block::kDx, rows, c.inputs, c.inner)) {
    copies.use(&w_gate, &ldg, c.inputs, c.inner, plan->w_bytes ? ws + plan->off_w : nullptr);
    copies.use(&w_up, &ldu, c.inputs, c.inner, plan->w_bytes ? ws + plan->off_w + plan->w_bytes : nullptr);
  }
  if (dw_gate != nullptr) copies.use(&x, &x_stride, rows, c.inputs, ws + plan->off_x);
  if ((st = copies.launch(s)) != ROUTE_OK) return st;
  if (dx != nullptr && rows != 0) {
    GemmArgs a{};
    a.a[0] = dz[0];
    a.a[1] = dz[1];
    a.lda = padded(c.inner);
    a.b[0] = w_gate;
    a.b[1] = w_up;
    a.ldb = ldu;
    a.c[0] = dx;
    a.ldc = dx_stride;
    a.m = rows;
    a.n = c.inputs;
    a.red = c.inner;
    a.segments = 2;
    a.outputs = 1;
    st = status_of(block::launch_gemm(c.dtype, block::kDx, a, products(plan, workspace), s));
    if (st != ROUTE_OK) return st;
  }
  if (dw_gate == nullptr) return ROUTE_OK;
  GemmArgs a{};
  a.a[0] = x;
  a.lda = x_stride;
  a.b[0] = dz[0];
  a.b[1] = dz[1];
  a.ldb = padded(c.inner);
  a.c[0] = dw_gate;
  a.c[1] = dw_up;
  a.ldc = c.inner;
  a.m = c.inputs;
  a.n = c.inner;
  a.red = rows;
  a.segments = 1;
  a.outputs = 2;
  return status_of(block::launch_gemm(c.dtype, block::kDw, a, products(plan, workspace), s));
}

void block_gated_destroy(block_gated_plan* plan) { delete plan; }

// ----------------------------------------------------------------- linear --

int block_linear_prepare(const block_linear_config* cfg, block_linear_plan** out) {
  if (out == nullptr) return ROUTE_E_ARG;
  *out = nullptr;
  if (cfg == nullptr || cfg->abi_version != BLOCK_ABI_VERSION) return ROUTE_E_ARG;
  if ((cfg->dtype != BLOCK_BF16 && cfg->dtype != BLOCK_F16) || cfg->activation < BLOCK_ACT_NONE ||
      cfg->activation > BLOCK_ACT_GELU_TANH)
    return ROUTE_E_ARG;
  if (bad_size(cfg->inputs) || bad_size(cfg->outputs)) return ROUTE_E_SHAPE;
  if (bad_rows(cfg->rows)) return ROUTE_E_ROWS;
  if (int st = find_device(cfg->device)) return st;
  block_linear_plan* p = new_plan<block_linear_plan>(*cfg);
  if (p == nullptr) return ROUTE_E_ARG;
  p->partial_bytes = partial_area(block::kLinear, cfg->rows, cfg->inputs, cfg->outputs, 1, cfg->training != 0);
  p->off_dz = block::kCounterBytes + p->partial_bytes;
  p->off_sum = p->off_dz + (cfg->training ? round256((size_t)cfg->rows * padded(cfg->outputs) * 2) : 0);
  p->off_x = p->off_sum + (cfg->training ? round256(block::column_sum_bytes(cfg->rows, cfg->outputs)) : 0);
  p->off_w = p->off_x + round256((size_t)cfg->rows * padded(cfg->inputs) * 2);
  p->w_bytes = (cfg->outputs & 7) != 0 ? round256((size_t)cfg->inputs * padded(cfg->outputs) * 2) : 0;
  p->ws_bytes = p->off_w + p->w_bytes;
  *out = p;
  return ROUTE_OK;
}

size_t block_linear_workspace_bytes(const block_linear_plan* plan) { return plan ? plan->ws_bytes : 0; }

int block_linear(const block_linear_plan* plan, const void* x, int64_t x_stride, const void* w,
                 const void* bias, const void* residual, int64_t residual_stride, void* y,
                 int64_t y_stride, void* slope, void* workspace, int32_t rows, void* stream) {
  if (!plan || !w || !workspace) return ROUTE_E_ARG;
  if (rows != 0 && (!x || !y)) return ROUTE_E_ARG;
  const block_linear_config& c = plan->cfg;
  if (rows < 0 || rows > c.rows) return ROUTE_E_ROWS;
  if (bad_stride(x_stride, c.inputs) || bad_stride(y_stride, c.outputs) ||
      (residual != nullptr && bad_stride(residual_stride, c.outputs)))
    return ROUTE_E_SHAPE;
  if (misaligned(x, 2) || misaligned(w, 2) || misaligned(bias, 2) || misaligned(residual, 2) ||
      misaligned(y, 2) || misaligned(slope, 2) || misaligned(workspace, 256))
    return ROUTE_E_ALIGN;
  if (int st = check_current(c.device)) return st;
  if (rows == 0) return ROUTE_OK;
  GemmArgs a{};
  a.a[0] = x;
  a.lda = x_stride;
  a.b[0] = w;
  a.ldb = c.outputs;
  a.c[0] = y;
  a.ldc = y_stride;
  a.saved[0] = slope;
  a.bias = bias;
  a.residual = residual;
  a.ldr = residual_stride;
  a.m = rows;
  a.n = c.outputs;
  a.red = c.inputs;
  a.segments = a.outputs = 1;
  a.act = c.activation;
  if (!block::gemm_streams(block::kLinear, rows, c.outputs, c.inputs)) {
    char* ws = static_cast<char*>(workspace);
    Copies copies;
    copies.use(&a.a[0], &a.lda, rows, c.inputs, ws + plan->off_x);
    copies.use(&a.b[0], &a.ldb, c.inputs, c.outputs, plan->w_bytes ? ws + plan->off_w : nullptr);
    if (int st = copies.launch(static_cast<hipStream_t>(stream))) return st;
  }
  return status_of(block::launch_gemm(c.dtype, block::kLinear, a, products(plan, workspace),
                                      static_cast<hipStream_t>(stream)));
}

int block_linear_backward(const block_linear_plan* plan, const void* dy, int64_t dy_stride, const void* x,
                          int64_t x_stride, const void* w, const void* slope, void* dx, int64_t dx_stride,
                          void* dw, void* dbias, void* workspace, int32_t rows, void* stream) {
  if (!plan || !w || !workspace || !plan->cfg.training) return ROUTE_E_ARG;
  const block_linear_config& c = plan->cfg;
  const bool scaled = c.activation != BLOCK_ACT_NONE;
  if (rows != 0 && (!dy || !x || (scaled && !slope) || (!dx && !dw && !dbias))) return ROUTE_E_ARG;
  if (rows < 0 || rows > c.rows) return ROUTE_E_ROWS;
  if (bad_stride(dy_stride, c.outputs) || bad_stride(x_stride, c.inputs) ||
      (dx != nullptr && bad_stride(dx_stride, c.inputs)))
    return ROUTE_E_SHAPE;
  if (misaligned(dy, 2) || misaligned(x, 2) || misaligned(w, 2) || misaligned(slope, 2) || misaligned(dx, 2) ||
      misaligned(dw, 2) || misaligned(dbias, 2) || misaligned(workspace, 256))
    return ROUTE_E_ALIGN;
  if (int st = check_current(c.device)) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  const void* dz = dy;
  int64_t ldz = dy_stride;
  void* out = scaled && (dx != nullptr || dw != nullptr) ? ws + plan->off_dz : nullptr;
  if (scaled || dbias != nullptr) {
    const int st = status_of(block::launch_scale(c.dtype, dy, dy_stride, &slope, scaled ? 1 : 0, &out,
                                                 padded(c.outputs), rows, c.outputs, dbias,
                                                 reinterpret_cast<float*>(ws + plan->off_sum), s));
    if (st != ROUTE_OK) return st;
  }
  if (scaled) {
    dz = out;
    ldz = padded(c.outputs);
  }
  Copies copies;
  int64_t ldw = c.outputs;
  const bool tiled_dx = dx != nullptr && !block::gemm_streams(block::kDx, rows, c.inputs, c.outputs);
  if (tiled_dx) copies.use(&w, &ldw, c.inputs, c.outputs, plan->w_bytes ? ws + plan->off_w : nullptr);
  if (dw != nullptr) copies.use(&x, &x_stride, rows, c.inputs, ws + plan->off_x);
  if (!scaled && (tiled_dx || dw != nullptr)) copies.use(&dz, &ldz, rows, c.outputs, ws + plan->off_dz);
  if (int st = copies.launch(s)) return st;
  if (dx != nullptr && rows != 0) {
    GemmArgs a{};
    a.a[0] = dz;
    a.lda = ldz;
    a.b[0] = w;
    a.ldb = ldw;
    a.c[0] = dx;
    a.ldc = dx_stride;
    a.m = rows;
    a.n = c.inputs;
    a.red = c.outputs;
    a.segments = a.outputs = 1;
    const int st = status_of(block::launch_gemm(c.dtype, block::kDx, a, products(plan, workspace), s));
    if (st != ROUTE_OK) return st;
  }
  if (dw == nullptr) return ROUTE_OK;
  GemmArgs a{};
  a.a[0] = x;
  a.lda = x_stride;
  a.b[0] = dz;
  a.ldb = ldz;
  a.c[0] = dw;
  a.ldc = c.outputs;
  a.m = c.inputs;
  a.n = c.outputs;
  a.red = rows;
  a.segments = a.outputs = 1;
  return status_of(block::launch_gemm(c.dtype, block::kDw, a, products(plan, workspace), s));
}

void block_linear_destroy(block_linear_plan* plan) { delete plan; }

}  // extern "C"
