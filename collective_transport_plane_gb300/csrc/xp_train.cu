// Host side of include/xp_train.h: argument checks, a group's tables (laid
// out once at create), and the launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>
#include <new>
#include <vector>

#include "xp_checks.h"
#include "xp_train_internal.h"

struct xp_group {
  int device = 0;
  xp_group_config cfg = {};
  int ntensors = 0;
  unsigned nunits = 0;
  bool has_params = false;
  std::vector<unsigned long long> counts;
  char* mem = nullptr;               // one allocation: tensors, units, partial sums, state
  xp::GroupTensor* tensors = nullptr;
  xp::GroupUnit* units = nullptr;
  double* partial = nullptr;
  xp::GroupState* state = nullptr;
};

namespace {

using namespace xp::checks;

bool step_ok(uint64_t step) { return step <= XP_GROUP_MAX_STEP; }

// Elements of a unit.  Small groups are cut finer, so that their elements
// spread over the SMs; a unit is a whole number of turns of its CTA.
constexpr size_t kUnitMin = (size_t)xp::kStepThreads * xp::kVec;   // 2048
constexpr size_t kUnitMax = 4 * kUnitMin;
size_t unit_elements(unsigned long long total) {
  size_t u = kUnitMin;
  while (u < kUnitMax && total / u > 152 * 16) u *= 2;
  return u;
}

xp_status check_tensor(const xp_group_config& c, int i, const xp_tensor& t, bool has_params) {
  if (t.reserved != 0) return fail(XP_ERR_INVALID, "tensor %d: reserved is %d, not 0", i, t.reserved);
  if (t.count > XP_GROUP_MAX_ELEMENTS) return fail(XP_ERR_INVALID, "tensor %d: %zu elements", i, t.count);
  if ((t.param != nullptr) != has_params && t.count) return fail(XP_ERR_INVALID, "tensor %d: param in some tensors only", i);
  if (t.count && !t.grad) return fail(XP_ERR_INVALID, "tensor %d: grad is NULL", i);
  if (!aligned(t.grad, size_of(c.grad_dtype))) return fail(XP_ERR_INVALID, "tensor %d: grad is not aligned to its element", i);
  if (!has_params) return XP_OK;
  const bool s8 = c.state_dtype == XP_U8;
  if (t.count && (!t.m || !t.v)) return fail(XP_ERR_INVALID, "tensor %d: m or v is NULL", i);
  if (t.count && s8 && (!t.m_scale || !t.v_scale)) return fail(XP_ERR_INVALID, "tensor %d: an 8-bit state without scales", i);
  if (!aligned(t.param, size_of(c.param_dtype)) || !aligned(t.copy, 2) || (!s8 && (!aligned(t.m, 4) || !aligned(t.v, 4))))
    return fail(XP_ERR_INVALID, "tensor %d: a pointer is not aligned to its element", i);
  if (!std::isfinite(t.weight_decay)) return fail(XP_ERR_INVALID, "tensor %d: weight_decay is not finite", i);
  return XP_OK;
}

xp_status check_group(const xp_group* g) {
  if (!g) return fail(XP_ERR_INVALID, "group is NULL");
  int d = -1;
  XP_CUDA(cudaGetDevice(&d));
  if (d != g->device) return fail(XP_ERR_INVALID, "current device %d is not the group's device %d", d, g->device);
  return XP_OK;
}

xp_status create(const xp_group_config& cfg, int ntensors, const xp_tensor* tensors, xp_group* g) {
  g->cfg = cfg;
  g->ntensors = ntensors;
  for (int i = 0; i < ntensors; ++i) g->has_params |= tensors[i].param != nullptr;
  unsigned long long total = 0;
  for (int i = 0; i < ntensors; ++i) {
    const xp_status s = check_tensor(cfg, i, tensors[i], g->has_params);
    if (s != XP_OK) return s;
    total += tensors[i].count;
    if (total > XP_GROUP_MAX_ELEMENTS) return fail(XP_ERR_INVALID, "the group's elements are more than 2^40 with tensor %d", i);
  }
  const size_t unit = unit_elements(total);
  std::vector<xp::GroupTensor> table(ntensors);
  std::vector<xp::GroupUnit> units;
  unsigned long long pos = 0;
  for (int i = 0; i < ntensors; ++i) {
    const xp_tensor& t = tensors[i];
    xp::GroupTensor& d = table[i];
    d.param = t.param;
    d.grad = t.grad;
    d.m = t.m;
    d.v = t.v;
    d.m_scale = t.m_scale;
    d.v_scale = t.v_scale;
    d.copy = t.copy;
    d.count = t.count;
    d.pos = pos;
    d.decay = t.weight_decay;
    const size_t sa = cfg.state_dtype == XP_U8 ? 8 : 16;
    d.aligned = aligned(t.param, 16) && aligned(t.copy, 16) && aligned(t.m, sa) && aligned(t.v, sa);
    g->counts.push_back(t.count);
    for (unsigned long long at = 0; at < t.count; at += unit) {
      const unsigned long long n = t.count - at < unit ? t.count - at : unit;
      units.push_back({(unsigned)i, (unsigned)n, at});
    }
    pos += round_up(t.count, XP_STATE8_BLOCK);
  }
  if (units.empty()) units.push_back({0u, 0u, 0ull});   // a step of an empty group still counts
  g->nunits = (unsigned)units.size();

  const size_t at_units = round_up(table.size() * sizeof(xp::GroupTensor), 256);
  const size_t at_partial = at_units + round_up(units.size() * sizeof(xp::GroupUnit), 256);
  const size_t at_state = at_partial + round_up(xp::kNormMaxCtas * sizeof(double), 256);
  XP_CUDA(cudaGetDevice(&g->device));
  XP_CUDA(cudaMalloc(reinterpret_cast<void**>(&g->mem), at_state + 256));
  g->tensors = reinterpret_cast<xp::GroupTensor*>(g->mem);
  g->units = reinterpret_cast<xp::GroupUnit*>(g->mem + at_units);
  g->partial = reinterpret_cast<double*>(g->mem + at_partial);
  g->state = reinterpret_cast<xp::GroupState*>(g->mem + at_state);
  std::vector<char> image(at_state + 256, 0);
  memcpy(image.data(), table.data(), table.size() * sizeof(xp::GroupTensor));
  memcpy(image.data() + at_units, units.data(), units.size() * sizeof(xp::GroupUnit));
  xp::GroupState state = {};
  state.step = cfg.step;
  state.power1 = std::pow(cfg.beta1, (double)(cfg.step + 1));
  state.power2 = std::pow(cfg.beta2, (double)(cfg.step + 1));
  state.inv_bias1 = (float)(1.0 / (1.0 - state.power1));
  state.inv_sqrt_bias2 = (float)(1.0 / std::sqrt(1.0 - state.power2));
  memcpy(image.data() + at_state, &state, sizeof state);
  // on a stream of its own, waited for here: never behind the caller's work
  cudaStream_t st = nullptr;
  XP_CUDA(cudaStreamCreateWithFlags(&st, cudaStreamNonBlocking));
  cudaError_t e = cudaMemcpyAsync(g->mem, image.data(), image.size(), cudaMemcpyHostToDevice, st);
  const cudaError_t e2 = cudaStreamSynchronize(st);
  cudaStreamDestroy(st);
  XP_CUDA(e);
  XP_CUDA(e2);
  return XP_OK;
}

xp_status check_sizes(size_t rows, size_t cols, int dtype, int wdtype) {
  if (!is_float_type(dtype) || !is_float_type(wdtype)) return fail(XP_ERR_INVALID, "dtype %d / %d is neither XP_F32 nor XP_BF16", dtype, wdtype);
  if (cols < 1 || cols > XP_LAYERNORM_MAX_COLS) return fail(XP_ERR_INVALID, "cols %zu not in [1, 131072]", cols);
  if (rows > XP_LAYERNORM_MAX_ROWS) return fail(XP_ERR_INVALID, "rows %zu above 2^28", rows);
  return XP_OK;
}

size_t workspace_bytes_of(const xp::BackwardShape& s, size_t cols) { return (size_t)s.nparts * 2 * cols * sizeof(float); }

}  // namespace

extern "C" {

xp_status xp_group_create(const xp_group_config* cfg, int ntensors, const xp_tensor* tensors, xp_group** out) {
  if (!cfg || !tensors || !out) return fail(XP_ERR_INVALID, "cfg, tensors or out is NULL");
  if (ntensors < 1 || ntensors > (1 << 20)) return fail(XP_ERR_INVALID, "ntensors %d not in [1, 2^20]", ntensors);
  if (!(cfg->beta1 >= 0 && cfg->beta1 < 1) || !(cfg->beta2 >= 0 && cfg->beta2 < 1))
    return fail(XP_ERR_INVALID, "beta1 %g or beta2 %g not in [0, 1)", cfg->beta1, cfg->beta2);
  if (!(cfg->eps > 0) || !((float)cfg->eps > 0.f) || !std::isfinite((float)cfg->eps)) return fail(XP_ERR_INVALID, "eps %g is not a positive fp32 number", cfg->eps);
  if (!is_float_type(cfg->param_dtype) || !is_float_type(cfg->grad_dtype))
    return fail(XP_ERR_INVALID, "param_dtype %d / grad_dtype %d is neither XP_F32 nor XP_BF16", cfg->param_dtype, cfg->grad_dtype);
  if (cfg->state_dtype != XP_F32 && cfg->state_dtype != XP_U8) return fail(XP_ERR_INVALID, "state_dtype %d is neither XP_F32 nor XP_U8", cfg->state_dtype);
  if (!step_ok(cfg->step)) return fail(XP_ERR_INVALID, "step %llu above 2^52", (unsigned long long)cfg->step);
  xp_group* g = nullptr;
  try {
    g = new xp_group();
    const xp_status s = create(*cfg, ntensors, tensors, g);
    if (s != XP_OK) {
      if (g->mem) cudaFree(g->mem);
      delete g;
      return s;
    }
  } catch (const std::exception& e) {
    if (g && g->mem) cudaFree(g->mem);
    delete g;
    return fail(XP_ERR_INTERNAL, "%s", e.what());
  }
  *out = g;
  return XP_OK;
}

xp_status xp_group_destroy(xp_group* g) {
  if (!g) return XP_OK;
  const cudaError_t e = g->mem ? cudaFree(g->mem) : cudaSuccess;   // waits for the device
  delete g;
  XP_CUDA(e);
  return XP_OK;
}

xp_status xp_group_set_grads(xp_group* g, const void* const* grads, xp_stream_t stream) {
  xp_status s = check_group(g);
  if (s != XP_OK) return s;
  if (!grads) return fail(XP_ERR_INVALID, "grads is NULL");
  for (int i = 0; i < g->ntensors; ++i) {
    if (g->counts[i] && !grads[i]) return fail(XP_ERR_INVALID, "tensor %d: grad is NULL", i);
    if (!aligned(grads[i], size_of(g->cfg.grad_dtype))) return fail(XP_ERR_INVALID, "tensor %d: grad is not aligned to its element", i);
  }
  // the pointers travel in the launches' parameters: the host array may go at
  // once, and a captured graph keeps them
  for (int at = 0; at < g->ntensors; at += xp::kSetGradsMax) {
    xp::SetGradsParams p;
    p.tensors = g->tensors;
    p.first = at;
    p.n = g->ntensors - at < xp::kSetGradsMax ? g->ntensors - at : xp::kSetGradsMax;
    for (int i = 0; i < p.n; ++i) p.grad[i] = grads[at + i];
    XP_CUDA(xp::launch_set_grads(p, stream));
  }
  return XP_OK;
}

xp_status xp_group_set_step(xp_group* g, uint64_t step, xp_stream_t stream) {
  xp_status s = check_group(g);
  if (s != XP_OK) return s;
  if (!step_ok(step)) return fail(XP_ERR_INVALID, "step %llu above 2^52", (unsigned long long)step);
  XP_CUDA(xp::launch_set_step(g->state, step, std::pow(g->cfg.beta1, (double)(step + 1)), std::pow(g->cfg.beta2, (double)(step + 1)), stream));
  return XP_OK;
}

xp_status xp_group_get_step(xp_group* g, uint64_t* step, xp_stream_t stream) {
  xp_status s = check_group(g);
  if (s != XP_OK) return s;
  if (!step) return fail(XP_ERR_INVALID, "step is NULL");
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  XP_CUDA(cudaStreamIsCapturing(stream, &capture));
  if (capture != cudaStreamCaptureStatusNone) return fail(XP_ERR_INVALID, "the step count cannot be read within a stream's capture");
  unsigned long long v = 0;
  XP_CUDA(cudaMemcpyAsync(&v, &g->state->step, sizeof v, cudaMemcpyDeviceToHost, stream));
  XP_CUDA(cudaStreamSynchronize(stream));
  *step = v;
  return XP_OK;
}

xp_status xp_grad_norm(xp_group* g, float grad_scale, float max_norm, int accumulate, xp_grad_report* report,
                       xp_stream_t stream) {
  xp_status s = check_group(g);
  if (s != XP_OK) return s;
  if (!report || !aligned(report, 16)) return fail(XP_ERR_INVALID, "report is NULL or not 16-byte aligned");
  if (!std::isfinite(grad_scale) || grad_scale < 0 || std::isnan(max_norm)) return fail(XP_ERR_INVALID, "grad_scale %g or max_norm %g", grad_scale, max_norm);
  xp::NormParams p;
  p.units = g->units;
  p.nunits = g->nunits;
  p.tensors = g->tensors;
  p.state = g->state;
  p.partial = g->partial;
  p.report = report;
  p.grad_scale = grad_scale;
  p.max_norm = max_norm;
  p.accumulate = accumulate;
  XP_CUDA(xp::launch_grad_norm(p, g->cfg.grad_dtype, stream));
  return XP_OK;
}

xp_status xp_adamw_step(xp_group* g, float lr, const float* lr_dev, float grad_scale, const xp_grad_report* report,
                        int flags, xp_stream_t stream) {
  xp_status s = check_group(g);
  if (s != XP_OK) return s;
  if (!g->has_params) return fail(XP_ERR_INVALID, "the group has no weights");
  if (!lr_dev && !std::isfinite(lr)) return fail(XP_ERR_INVALID, "lr is not finite");
  if (!report && !std::isfinite(grad_scale)) return fail(XP_ERR_INVALID, "grad_scale is not finite");
  if (!aligned(lr_dev, 4) || !aligned(report, 16)) return fail(XP_ERR_INVALID, "lr_dev or report is not aligned");
  if (flags & ~XP_ADAMW_SKIP_NONFINITE) return fail(XP_ERR_INVALID, "unknown flags %d", flags);
  if ((flags & XP_ADAMW_SKIP_NONFINITE) && !report) return fail(XP_ERR_INVALID, "XP_ADAMW_SKIP_NONFINITE needs a report");
  xp::StepParams p;
  p.units = g->units;
  p.tensors = g->tensors;
  p.state = g->state;
  p.report = report;
  p.lr_dev = lr_dev;
  p.lr = lr;
  p.grad_scale = grad_scale;
  p.beta1 = (float)g->cfg.beta1;
  p.beta2 = (float)g->cfg.beta2;
  p.one_minus_beta1 = (float)(1.0 - g->cfg.beta1);
  p.one_minus_beta2 = (float)(1.0 - g->cfg.beta2);
  p.eps = (float)g->cfg.eps;
  p.beta1_d = g->cfg.beta1;
  p.beta2_d = g->cfg.beta2;
  p.seed = g->cfg.seed;
  p.skip_nonfinite = flags & XP_ADAMW_SKIP_NONFINITE;
  XP_CUDA(xp::launch_adamw(p, g->nunits, g->cfg.param_dtype, g->cfg.grad_dtype, g->cfg.state_dtype, stream));
  return XP_OK;
}

xp_status xp_state8_decode(const uint8_t* m, const uint8_t* m_scale, const uint8_t* v, const uint8_t* v_scale,
                           size_t count, void* m_out, void* v_out, xp_dtype out_dtype, xp_stream_t stream) {
  if (!is_float_type(out_dtype)) return fail(XP_ERR_INVALID, "out_dtype %d is neither XP_F32 nor XP_BF16", (int)out_dtype);
  if (count > ((size_t)1 << 40)) return fail(XP_ERR_INVALID, "count %zu above 2^40", count);
  if (count == 0) return XP_OK;
  if ((m_out && (!m || !m_scale)) || (v_out && (!v || !v_scale))) return fail(XP_ERR_INVALID, "an output without its codes or scales");
  if (!aligned(m_out, size_of(out_dtype)) || !aligned(v_out, size_of(out_dtype))) return fail(XP_ERR_INVALID, "an output is not aligned to its element");
  if (!m_out && !v_out) return XP_OK;
  xp::DecodeParams p = {{m, v}, {m_scale, v_scale}, {m_out, v_out}, count};
  XP_CUDA(xp::launch_decode(p, out_dtype, stream));
  return XP_OK;
}

xp_status xp_layernorm_forward(const void* x, size_t x_stride, const void* gamma, const void* beta, void* y,
                               size_t y_stride, float* mean, float* rstd, size_t rows, size_t cols, float eps,
                               xp_dtype dtype, xp_dtype wdtype, xp_stream_t stream) {
  xp_status s = check_sizes(rows, cols, dtype, wdtype);
  if (s != XP_OK || rows == 0) return s;
  if ((s = check_rows("x", x, x_stride, rows, cols, dtype)) != XP_OK) return s;
  if ((s = check_rows("y", y, y_stride, rows, cols, dtype)) != XP_OK) return s;
  if (!aligned(gamma, size_of(wdtype)) || !aligned(beta, size_of(wdtype)) || !aligned(mean, 4) || !aligned(rstd, 4))
    return fail(XP_ERR_INVALID, "gamma, beta, mean or rstd is not aligned to its element");
  if (!(eps >= 0) || !std::isfinite(eps)) return fail(XP_ERR_INVALID, "eps %g is negative or not finite", eps);
  const Span sx = span_of(x, x_stride, rows, cols, size_of(dtype)), sy = span_of(y, y_stride, rows, cols, size_of(dtype));
  if (overlap(sx, sy) && !same(sx, sy)) return fail(XP_ERR_INVALID, "x and y overlap");
  xp::NormRowsParams p = {};
  p.x = x;
  p.gamma = gamma;
  p.beta = beta;
  p.out = y;
  p.mean = mean;
  p.rstd = rstd;
  p.x_stride = x_stride;
  p.out_stride = y_stride;
  p.rows = rows;
  p.cols = (unsigned)cols;
  p.eps = eps;
  p.gamma_bf16 = wdtype == XP_BF16;
  XP_CUDA(xp::launch_ln_forward(p, dtype, stream));
  return XP_OK;
}

xp_status xp_layernorm_workspace(size_t rows, size_t cols, size_t* bytes) {
  if (!bytes) return fail(XP_ERR_INVALID, "bytes is NULL");
  if (cols > XP_LAYERNORM_MAX_COLS || rows > XP_LAYERNORM_MAX_ROWS) return fail(XP_ERR_INVALID, "rows %zu or cols %zu too large", rows, cols);
  *bytes = rows && cols ? workspace_bytes_of(xp::ln_backward_shape(rows, cols), cols) : 0;
  return XP_OK;
}

xp_status xp_layernorm_backward(const void* dy, size_t dy_stride, const void* x, size_t x_stride, const void* gamma,
                                const float* mean, const float* rstd, void* dx, size_t dx_stride, float* dgamma,
                                float* dbeta, size_t rows, size_t cols, xp_dtype dtype, xp_dtype wdtype,
                                int accumulate, void* workspace, size_t workspace_bytes, xp_stream_t stream) {
  xp_status s = check_sizes(rows, cols, dtype, wdtype);
  if (s != XP_OK) return s;
  if ((dgamma == nullptr) != (dbeta == nullptr)) return fail(XP_ERR_INVALID, "one of dgamma and dbeta is NULL");
  if (!aligned(dgamma, 4) || !aligned(dbeta, 4)) return fail(XP_ERR_INVALID, "dgamma or dbeta is not aligned to its element");
  if (rows == 0) {
    if (dgamma && !accumulate) {
      XP_CUDA(cudaMemsetAsync(dgamma, 0, cols * sizeof(float), stream));
      XP_CUDA(cudaMemsetAsync(dbeta, 0, cols * sizeof(float), stream));
    }
    return XP_OK;
  }
  if ((s = check_rows("dy", dy, dy_stride, rows, cols, dtype)) != XP_OK) return s;
  if ((s = check_rows("x", x, x_stride, rows, cols, dtype)) != XP_OK) return s;
  if ((s = check_rows("dx", dx, dx_stride, rows, cols, dtype)) != XP_OK) return s;
  if (!mean || !rstd || !aligned(mean, 4) || !aligned(rstd, 4)) return fail(XP_ERR_INVALID, "mean or rstd is NULL or not aligned");
  if (!aligned(gamma, size_of(wdtype))) return fail(XP_ERR_INVALID, "gamma is not aligned to its element");
  const size_t es = size_of(dtype);
  const Span sdy = span_of(dy, dy_stride, rows, cols, es), sx = span_of(x, x_stride, rows, cols, es);
  const Span sdx = span_of(dx, dx_stride, rows, cols, es);
  if (overlap(sdx, sx) || (overlap(sdx, sdy) && !same(sdx, sdy))) return fail(XP_ERR_INVALID, "dx overlaps x or dy");
  const xp::BackwardShape shape = xp::ln_backward_shape(rows, cols);
  if (dgamma) {
    const size_t need = workspace_bytes_of(shape, cols);
    if (!workspace || workspace_bytes < need || !aligned(workspace, 16))
      return fail(XP_ERR_INVALID, "workspace of %zu bytes (NULL, or not 16-byte aligned, or below the %zu needed)", workspace_bytes, need);
  }
  xp::NormRowsParams p = {};
  p.x = x;
  p.dy = dy;
  p.gamma = gamma;
  p.out = dx;
  p.mean = const_cast<float*>(mean);
  p.rstd = const_cast<float*>(rstd);
  p.partial = static_cast<float*>(workspace);
  p.dgamma = dgamma;
  p.dbeta = dbeta;
  p.x_stride = x_stride;
  p.dy_stride = dy_stride;
  p.out_stride = dx_stride;
  p.rows = rows;
  p.cols = (unsigned)cols;
  p.gamma_bf16 = wdtype == XP_BF16;
  p.accumulate = accumulate;
  XP_CUDA(xp::launch_ln_backward(p, shape, dtype, stream));
  return XP_OK;
}

}  // extern "C"
