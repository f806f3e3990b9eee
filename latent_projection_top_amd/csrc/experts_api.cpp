// C ABI of the routed half of a layer (experts.h): plan preparation, argument
// checks and launches. Every check runs before any launch; nothing allocates
// device memory or synchronises.
#include "experts.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstring>
#include <new>

#include "experts_launch.h"

struct experts_sort_plan {
  experts_sort_config cfg;
  size_t ws_bytes;
};

struct experts_combine_plan {
  experts_combine_config cfg;
};

namespace {

// Workspace of the 8-bit products: the zeroed part (counters), split sums, the
// lists of items, the rows as integers and their scales.
struct Product8 {
  int32_t device, rows, tokens, inputs, outputs, experts, dtype, activation;
  size_t off_lists, off_q, off_step, ws_bytes, packed_bytes;
};

bool misaligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }
size_t round256(size_t n) { return (n + 255) & ~size_t(255); }
size_t dtype_size(int dtype) { return dtype == BLOCK_F32 ? 4 : 2; }
bool bad(int32_t n, int32_t most) { return n < 1 || n > most; }
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

// rows * topk of a plan
bool bad_choices(int32_t rows, int32_t topk) {
  return bad(rows, BLOCK_MAX_ROWS) || (int64_t)rows * topk > EXPERTS_MAX_CHOICES;
}

bool bad_capacity(int32_t n) { return n < 0 || n > EXPERTS_MAX_CHOICES; }

int prepare_product(Product8* p, int planes) {
  if (bad(p->inputs, EXPERTS_MAX_INPUTS) || bad(p->outputs, BLOCK_MAX_SIZE) || bad(p->experts, EXPERTS_MAX_COUNT))
    return ROUTE_E_SHAPE;
  if (bad(p->rows, EXPERTS_MAX_CHOICES) || bad(p->tokens, EXPERTS_MAX_CHOICES)) return ROUTE_E_ROWS;
  if (int st = find_device(p->device)) return st;
  const size_t stride = (size_t)experts::red_blocks(p->inputs) * experts::kBlockRed;
  p->off_lists = EXPERTS_WORKSPACE_ZEROED + experts::kPartialBytes;
  p->off_q = p->off_lists + round256(experts::list_bytes(p->rows, p->experts));
  p->off_step = p->off_q + round256((size_t)p->tokens * stride);
  p->ws_bytes = p->off_step + round256((size_t)p->tokens * sizeof(float));
  p->packed_bytes = (size_t)p->experts * planes * experts::column_tiles(p->outputs) *
                    experts::red_blocks(p->inputs) * experts::kBlockBytes;
  return ROUTE_OK;
}

// The checks and launches that both products share. w[0..1]: their scales.
int run_product(const Product8& c, const void* x, int64_t x_stride, const void* packed, const float* const* scale,
                int planes, const int32_t* offsets, const int32_t* token, const void* bias, const void* residual,
                int64_t residual_stride, void* y, int64_t y_stride, void* workspace, int32_t tokens, int32_t rows,
                void* stream) {
  if (!packed || !scale[0] || !scale[planes - 1] || !workspace || (offsets == nullptr && c.experts != 1))
    return ROUTE_E_ARG;
  if (rows != 0 && tokens != 0 && (!x || !y)) return ROUTE_E_ARG;
  if (rows < 0 || rows > c.rows || tokens < 0 || tokens > c.tokens) return ROUTE_E_ROWS;
  if (token == nullptr ? tokens != rows : (rows != 0 && tokens == 0)) return ROUTE_E_ROWS;
  if (bad_stride(x_stride, c.inputs) || bad_stride(y_stride, c.outputs) ||
      (residual != nullptr && bad_stride(residual_stride, c.outputs)))
    return ROUTE_E_SHAPE;
  if (misaligned(x, 2) || misaligned(y, 2) || misaligned(bias, 2) || misaligned(residual, 2) ||
      misaligned(scale[0], 4) || misaligned(scale[planes - 1], 4) || misaligned(offsets, 4) ||
      misaligned(token, 4) || misaligned(packed, 256) || misaligned(workspace, 256))
    return ROUTE_E_ALIGN;
  if (int st = check_current(c.device)) return st;
  if (rows == 0) return ROUTE_OK;
  hipStream_t s = static_cast<hipStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  experts::ProductArgs a{};
  a.q = reinterpret_cast<int8_t*>(ws + c.off_q);
  a.step = reinterpret_cast<float*>(ws + c.off_step);
  a.packed = packed;
  a.scale[0] = scale[0];
  a.scale[1] = scale[planes - 1];
  a.bias = bias;
  a.residual = residual;
  a.ldr = residual_stride;
  a.y = y;
  a.ldy = y_stride;
  a.token = token;
  if (offsets != nullptr) a.lists = experts::lists_at(ws + c.off_lists, rows, c.experts);
  a.counters = reinterpret_cast<uint32_t*>(ws);
  a.partial = reinterpret_cast<int32_t*>(ws + EXPERTS_WORKSPACE_ZEROED);
  a.tokens = tokens;
  a.rows = rows;
  a.n = c.outputs;
  a.blocks = experts::red_blocks(c.inputs);
  a.act = c.activation;
  a.gated = planes == 2;
  a.x = static_cast<const uint16_t*>(x);
  a.ldx = x_stride;
  a.k = c.inputs;
  a.experts = c.experts;
  a.offsets = offsets;
  const int column_tiles = planes * experts::column_tiles(c.outputs);
  const experts::Way way = experts::way_of(rows, c.experts, column_tiles, a.blocks, offsets != nullptr);
  if (experts::is_fused(way, rows, c.experts, a.blocks, offsets != nullptr))
    return status_of(experts::launch_stream(c.dtype, a, true, s));
  experts::QuantiseArgs z{};
  z.x = a.x;
  z.ldx = x_stride;
  z.q = reinterpret_cast<int8_t*>(ws + c.off_q);
  z.step = reinterpret_cast<float*>(ws + c.off_step);
  z.offsets = offsets;
  z.area = reinterpret_cast<experts::Item*>(ws + c.off_lists);
  z.tokens = tokens;
  z.k = c.inputs;
  z.stride = a.blocks * experts::kBlockRed;
  z.experts = c.experts;
  z.rows = rows;
  z.sorted = offsets != nullptr && token == nullptr;
  z.way = way;
  z.most_brief = (int)experts::most_brief(rows, c.experts);
  z.most_mid = (int)experts::most_mid(rows, c.experts);
  z.most_tiles = (int)experts::most_tiles(rows, c.experts);
  if (int st = status_of(experts::launch_quantise(c.dtype, z, s))) return st;
  if (way == experts::kBrief || way == experts::kApart)
    if (int st = status_of(experts::launch_stream(c.dtype, a, false, s))) return st;
  return way != experts::kBrief ? status_of(experts::launch_tiles(c.dtype, a, way, s)) : ROUTE_OK;
}

int run_quantize(const Product8& c, const void* w, int8_t* w8, float* scale, void* stream) {
  if (!w || !w8 || !scale) return ROUTE_E_ARG;
  if (misaligned(w, 2) || misaligned(scale, 4)) return ROUTE_E_ALIGN;
  if (int st = check_current(c.device)) return st;
  return status_of(experts::launch_quantise_weights(c.dtype, w, w8, scale, c.experts, c.inputs, c.outputs,
                                                    static_cast<hipStream_t>(stream)));
}

int run_pack(const Product8& c, const int8_t* const* w, int planes, void* packed, void* stream) {
  if (!w[0] || !w[planes - 1] || !packed) return ROUTE_E_ARG;
  if (misaligned(packed, 256)) return ROUTE_E_ALIGN;
  if (int st = check_current(c.device)) return st;
  return status_of(experts::launch_pack(w, planes, packed, c.experts, c.inputs, c.outputs,
                                        static_cast<hipStream_t>(stream)));
}

}  // namespace

struct experts_linear8_plan {
  Product8 p;
};

struct experts_gated8_plan {
  Product8 p;
};

extern "C" {

// ------------------------------------------------------------------- sort --

int experts_sort_prepare(const experts_sort_config* cfg, experts_sort_plan** out) {
  if (out == nullptr) return ROUTE_E_ARG;
  *out = nullptr;
  if (cfg == nullptr || cfg->abi_version != EXPERTS_ABI_VERSION || cfg->first < 0) return ROUTE_E_ARG;
  if (bad(cfg->topk, EXPERTS_MAX_TOPK) || bad(cfg->experts, EXPERTS_MAX_COUNT)) return ROUTE_E_SHAPE;
  if (bad_choices(cfg->rows, cfg->topk)) return ROUTE_E_ROWS;
  if (int st = find_device(cfg->device)) return st;
  experts_sort_plan* p = new (std::nothrow) experts_sort_plan();
  if (p == nullptr) return ROUTE_E_ARG;
  p->cfg = *cfg;
  p->ws_bytes = std::max<size_t>(
      round256(experts::sort_workspace_bytes((int64_t)cfg->rows * cfg->topk, cfg->experts)), 256);
  *out = p;
  return ROUTE_OK;
}

size_t experts_sort_workspace_bytes(const experts_sort_plan* plan) { return plan ? plan->ws_bytes : 0; }

int experts_sort(const experts_sort_plan* plan, const int32_t* ids, int32_t* offsets, int32_t* place,
                 int32_t* token, void* workspace, int32_t capacity, int32_t rows, void* stream) {
  if (!plan || !offsets || !workspace) return ROUTE_E_ARG;
  if (rows != 0 && (!ids || !place || (!token && capacity != 0))) return ROUTE_E_ARG;
  const experts_sort_config& c = plan->cfg;
  if (rows < 0 || rows > c.rows || bad_capacity(capacity)) return ROUTE_E_ROWS;
  if (misaligned(ids, 4) || misaligned(offsets, 4) || misaligned(place, 4) || misaligned(token, 4) ||
      misaligned(workspace, 256))
    return ROUTE_E_ALIGN;
  if (int st = check_current(c.device)) return st;
  experts::SortArgs a{};
  a.ids = ids;
  a.offsets = offsets;
  a.place = place;
  a.token = token;
  a.workspace = workspace;
  a.choices = rows * c.topk;
  a.topk = c.topk;
  a.experts = c.experts;
  a.first = c.first;
  a.capacity = capacity;
  return status_of(experts::launch_sort(a, static_cast<hipStream_t>(stream)));
}

void experts_sort_destroy(experts_sort_plan* plan) { delete plan; }

// ---------------------------------------------------------------- combine --

int experts_combine_prepare(const experts_combine_config* cfg, experts_combine_plan** out) {
  if (out == nullptr) return ROUTE_E_ARG;
  *out = nullptr;
  if (cfg == nullptr || cfg->abi_version != EXPERTS_ABI_VERSION || cfg->dtype < BLOCK_BF16 || cfg->dtype > BLOCK_F32)
    return ROUTE_E_ARG;
  if (bad(cfg->topk, EXPERTS_MAX_TOPK) || bad(cfg->width, BLOCK_MAX_SIZE)) return ROUTE_E_SHAPE;
  if (bad_choices(cfg->rows, cfg->topk)) return ROUTE_E_ROWS;
  if (int st = find_device(cfg->device)) return st;
  experts_combine_plan* p = new (std::nothrow) experts_combine_plan();
  if (p == nullptr) return ROUTE_E_ARG;
  p->cfg = *cfg;
  *out = p;
  return ROUTE_OK;
}

int experts_gather(const experts_combine_plan* plan, const void* x, int64_t x_stride, const int32_t* place,
                   void* xs, int64_t xs_stride, int32_t capacity, int32_t rows, void* stream) {
  if (!plan) return ROUTE_E_ARG;
  if (rows != 0 && (!x || !place || (!xs && capacity != 0))) return ROUTE_E_ARG;
  const experts_combine_config& c = plan->cfg;
  if (rows < 0 || rows > c.rows || bad_capacity(capacity)) return ROUTE_E_ROWS;
  if (bad_stride(x_stride, c.width) || bad_stride(xs_stride, c.width)) return ROUTE_E_SHAPE;
  const size_t e = dtype_size(c.dtype);
  if (misaligned(x, e) || misaligned(xs, e) || misaligned(place, 4)) return ROUTE_E_ALIGN;
  if (int st = check_current(c.device)) return st;
  if (rows == 0 || capacity == 0) return ROUTE_OK;
  experts::RowsArgs a{};
  a.plain = x;
  a.ld_plain = x_stride;
  a.place = place;
  a.to_sorted = xs;
  a.ld_to_sorted = xs_stride;
  a.rows = rows;
  a.topk = c.topk;
  a.width = c.width;
  a.capacity = capacity;
  return status_of(experts::launch_spread(c.dtype, a, static_cast<hipStream_t>(stream)));
}

int experts_gather_backward(const experts_combine_plan* plan, const void* dxs, int64_t dxs_stride,
                            const int32_t* place, void* dx, int64_t dx_stride, int32_t capacity, int32_t rows,
                            void* stream) {
  if (!plan) return ROUTE_E_ARG;
  if (rows != 0 && ((!dxs && capacity != 0) || !place || !dx)) return ROUTE_E_ARG;
  const experts_combine_config& c = plan->cfg;
  if (rows < 0 || rows > c.rows || bad_capacity(capacity)) return ROUTE_E_ROWS;
  if (bad_stride(dxs_stride, c.width) || bad_stride(dx_stride, c.width)) return ROUTE_E_SHAPE;
  const size_t e = dtype_size(c.dtype);
  if (misaligned(dxs, e) || misaligned(dx, e) || misaligned(place, 4)) return ROUTE_E_ALIGN;
  if (int st = check_current(c.device)) return st;
  if (rows == 0) return ROUTE_OK;
  experts::RowsArgs a{};
  a.sorted = dxs;
  a.ld_sorted = dxs_stride;
  a.place = place;
  a.to_plain = dx;
  a.ld_to_plain = dx_stride;
  a.rows = rows;
  a.topk = c.topk;
  a.width = c.width;
  a.capacity = capacity;
  return status_of(experts::launch_collect(c.dtype, a, static_cast<hipStream_t>(stream)));
}

int experts_combine(const experts_combine_plan* plan, const void* ys, int64_t ys_stride, const int32_t* place,
                    const float* weights, const void* residual, int64_t residual_stride, void* y,
                    int64_t y_stride, int32_t capacity, int32_t rows, void* stream) {
  if (!plan) return ROUTE_E_ARG;
  if (rows != 0 && ((!ys && capacity != 0) || !place || !weights || !y)) return ROUTE_E_ARG;
  const experts_combine_config& c = plan->cfg;
  if (rows < 0 || rows > c.rows || bad_capacity(capacity)) return ROUTE_E_ROWS;
  if (bad_stride(ys_stride, c.width) || bad_stride(y_stride, c.width) ||
      (residual != nullptr && bad_stride(residual_stride, c.width)))
    return ROUTE_E_SHAPE;
  const size_t e = dtype_size(c.dtype);
  if (misaligned(ys, e) || misaligned(y, e) || misaligned(residual, e) || misaligned(place, 4) ||
      misaligned(weights, 4))
    return ROUTE_E_ALIGN;
  if (int st = check_current(c.device)) return st;
  if (rows == 0) return ROUTE_OK;
  experts::RowsArgs a{};
  a.sorted = ys;
  a.ld_sorted = ys_stride;
  a.place = place;
  a.weights = weights;
  a.residual = residual;
  a.ld_residual = residual_stride;
  a.to_plain = y;
  a.ld_to_plain = y_stride;
  a.rows = rows;
  a.topk = c.topk;
  a.width = c.width;
  a.capacity = capacity;
  return status_of(experts::launch_collect(c.dtype, a, static_cast<hipStream_t>(stream)));
}

int experts_combine_backward(const experts_combine_plan* plan, const void* dy, int64_t dy_stride, const void* ys,
                             int64_t ys_stride, const int32_t* place, const float* weights, void* dys,
                             int64_t dys_stride, float* dweights, int32_t capacity, int32_t rows, void* stream) {
  if (!plan) return ROUTE_E_ARG;
  if (rows != 0 && (!dy || !place || (!dys && !dweights) || (dys && !weights) ||
                    (dweights && !ys && capacity != 0)))
    return ROUTE_E_ARG;
  const experts_combine_config& c = plan->cfg;
  if (rows < 0 || rows > c.rows || bad_capacity(capacity)) return ROUTE_E_ROWS;
  if (bad_stride(dy_stride, c.width) || (dweights != nullptr && bad_stride(ys_stride, c.width)) ||
      (dys != nullptr && bad_stride(dys_stride, c.width)))
    return ROUTE_E_SHAPE;
  const size_t e = dtype_size(c.dtype);
  if (misaligned(dy, e) || misaligned(ys, e) || misaligned(dys, e) || misaligned(place, 4) ||
      misaligned(weights, 4) || misaligned(dweights, 4))
    return ROUTE_E_ALIGN;
  if (int st = check_current(c.device)) return st;
  if (rows == 0) return ROUTE_OK;
  experts::RowsArgs a{};
  a.plain = dy;
  a.ld_plain = dy_stride;
  a.sorted = ys;
  a.ld_sorted = ys_stride;
  a.place = place;
  a.weights = weights;
  a.to_sorted = dys;
  a.ld_to_sorted = dys_stride;
  a.dweights = dweights;
  a.rows = rows;
  a.topk = c.topk;
  a.width = c.width;
  a.capacity = capacity;
  return status_of(experts::launch_spread(c.dtype, a, static_cast<hipStream_t>(stream)));
}

void experts_combine_destroy(experts_combine_plan* plan) { delete plan; }

// ---------------------------------------------------------------- linear8 --

int experts_linear8_prepare(const experts_linear8_config* cfg, experts_linear8_plan** out) {
  if (out == nullptr) return ROUTE_E_ARG;
  *out = nullptr;
  if (cfg == nullptr || cfg->abi_version != EXPERTS_ABI_VERSION ||
      (cfg->dtype != BLOCK_BF16 && cfg->dtype != BLOCK_F16) || cfg->activation < BLOCK_ACT_NONE ||
      cfg->activation > BLOCK_ACT_GELU_TANH)
    return ROUTE_E_ARG;
  experts_linear8_plan plan{};
  plan.p.device = cfg->device;
  plan.p.rows = cfg->rows;
  plan.p.tokens = cfg->tokens;
  plan.p.inputs = cfg->inputs;
  plan.p.outputs = cfg->outputs;
  plan.p.experts = cfg->experts;
  plan.p.dtype = cfg->dtype;
  plan.p.activation = cfg->activation;
  if (int st = prepare_product(&plan.p, 1)) return st;
  *out = new (std::nothrow) experts_linear8_plan(plan);
  return *out != nullptr ? ROUTE_OK : ROUTE_E_ARG;
}

size_t experts_linear8_workspace_bytes(const experts_linear8_plan* plan) { return plan ? plan->p.ws_bytes : 0; }
size_t experts_linear8_packed_bytes(const experts_linear8_plan* plan) { return plan ? plan->p.packed_bytes : 0; }

int experts_linear8_quantize(const experts_linear8_plan* plan, const void* w, int8_t* w8, float* scale,
                             void* stream) {
  return plan ? run_quantize(plan->p, w, w8, scale, stream) : ROUTE_E_ARG;
}

int experts_linear8_pack(const experts_linear8_plan* plan, const int8_t* w, void* packed, void* stream) {
  return plan ? run_pack(plan->p, &w, 1, packed, stream) : ROUTE_E_ARG;
}

int experts_linear8(const experts_linear8_plan* plan, const void* x, int64_t x_stride, const void* packed,
                    const float* scale, const int32_t* offsets, const int32_t* token, const void* bias,
                    const void* residual, int64_t residual_stride, void* y, int64_t y_stride, void* workspace,
                    int32_t tokens, int32_t rows, void* stream) {
  if (!plan) return ROUTE_E_ARG;
  return run_product(plan->p, x, x_stride, packed, &scale, 1, offsets, token, bias, residual, residual_stride, y,
                     y_stride, workspace, tokens, rows, stream);
}

void experts_linear8_destroy(experts_linear8_plan* plan) { delete plan; }

// ----------------------------------------------------------------- gated8 --

int experts_gated8_prepare(const experts_gated8_config* cfg, experts_gated8_plan** out) {
  if (out == nullptr) return ROUTE_E_ARG;
  *out = nullptr;
  if (cfg == nullptr || cfg->abi_version != EXPERTS_ABI_VERSION ||
      (cfg->dtype != BLOCK_BF16 && cfg->dtype != BLOCK_F16) || cfg->activation <= BLOCK_ACT_NONE ||
      cfg->activation > BLOCK_ACT_GELU_TANH)
    return ROUTE_E_ARG;
  experts_gated8_plan plan{};
  plan.p.device = cfg->device;
  plan.p.rows = cfg->rows;
  plan.p.tokens = cfg->tokens;
  plan.p.inputs = cfg->inputs;
  plan.p.outputs = cfg->inner;
  plan.p.experts = cfg->experts;
  plan.p.dtype = cfg->dtype;
  plan.p.activation = cfg->activation;
  if (int st = prepare_product(&plan.p, 2)) return st;
  *out = new (std::nothrow) experts_gated8_plan(plan);
  return *out != nullptr ? ROUTE_OK : ROUTE_E_ARG;
}

size_t experts_gated8_workspace_bytes(const experts_gated8_plan* plan) { return plan ? plan->p.ws_bytes : 0; }
size_t experts_gated8_packed_bytes(const experts_gated8_plan* plan) { return plan ? plan->p.packed_bytes : 0; }

int experts_gated8_quantize(const experts_gated8_plan* plan, const void* w, int8_t* w8, float* scale,
                            void* stream) {
  return plan ? run_quantize(plan->p, w, w8, scale, stream) : ROUTE_E_ARG;
}

int experts_gated8_pack(const experts_gated8_plan* plan, const int8_t* w_gate, const int8_t* w_up, void* packed,
                        void* stream) {
  const int8_t* w[2] = {w_gate, w_up};
  return plan ? run_pack(plan->p, w, 2, packed, stream) : ROUTE_E_ARG;
}

int experts_gated8(const experts_gated8_plan* plan, const void* x, int64_t x_stride, const void* packed,
                   const float* scale_gate, const float* scale_up, const int32_t* offsets, const int32_t* token,
                   void* h, int64_t h_stride, void* workspace, int32_t tokens, int32_t rows, void* stream) {
  const float* scale[2] = {scale_gate, scale_up};
  if (!plan) return ROUTE_E_ARG;
  return run_product(plan->p, x, x_stride, packed, scale, 2, offsets, token, nullptr, nullptr, 0, h, h_stride,
                     workspace, tokens, rows, stream);
}

void experts_gated8_destroy(experts_gated8_plan* plan) { delete plan; }

}  // extern "C"
