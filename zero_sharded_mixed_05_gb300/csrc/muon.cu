// muon.cu -- host side of the orthogonalised update (zero_muon.h): checks,
// the workspace and its layout, launches.
#include "muon_kernels.cuh"

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>
#include <vector>

#include "host_util.h"

namespace {

using zo::fail;

zero_status cuda_fail(cudaError_t e, const char* what) {
  return fail(ZERO_ECUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool dtype16(int32_t d) { return d == ZERO_FP16 || d == ZERO_BF16; }

}  // namespace

struct zero_muon_handle {
  zero_muon_config cfg;
  std::vector<zero_muon_shape> shapes;
  std::vector<zm::Entry> entries;
  bool has_device = false;
  int device = -1;
  int sms = 0;
  unsigned char* mem = nullptr;     // the whole workspace
  int64_t bytes = 0;
  zm::Call call = {};               // the fields that no call changes
  int64_t chunks = 0;               // CTAs of the first two stages
  int64_t launches = 0;
};

namespace {

zero_status check(const zero_muon_config* c) {
  if (!dtype16(c->grad_dtype) || !dtype16(c->param_dtype))
    return fail(ZERO_EINVAL, "grad_dtype and param_dtype must be ZERO_FP16 or ZERO_BF16");
  if ((c->nesterov | 1) != 1) return fail(ZERO_EINVAL, "nesterov must be 0 or 1");
  if (c->steps < 1 || c->steps > ZERO_MUON_MAX_STEPS)
    return fail(ZERO_EINVAL, "steps must be in 1..%d", ZERO_MUON_MAX_STEPS);
  if (c->scale_rule < ZERO_MUON_SCALE_ONE || c->scale_rule > ZERO_MUON_SCALE_ASPECT)
    return fail(ZERO_EINVAL, "scale_rule %d is not a zero_muon_scale", c->scale_rule);
  if (!(c->lr >= 0.0)) return fail(ZERO_EINVAL, "lr must be >= 0");
  if (!(c->momentum >= 0.0 && c->momentum < 1.0))
    return fail(ZERO_EINVAL, "momentum must be in [0, 1)");
  if (!(c->weight_decay >= 0.0)) return fail(ZERO_EINVAL, "weight_decay must be >= 0");
  if (!(c->eps >= 0.0)) return fail(ZERO_EINVAL, "eps must be >= 0");
  for (int i = 0; i < c->steps; ++i)
    for (double v : c->coef[i])
      if (!std::isfinite(v)) return fail(ZERO_EINVAL, "coef[%d] is not finite", i);
  return ZERO_OK;
}

// Places of the workspace, 256-byte aligned.
struct Layout {
  int64_t size = 0;
  int64_t take(int64_t bytes) {
    const int64_t at = size;
    size += (bytes + 255) / 256 * 256;
    return at;
  }
};

zero_status launch(zero_muon_t h, const void* fn, int64_t grid, void** params, cudaStream_t s) {
  const cudaError_t e =
      cudaLaunchKernel(fn, dim3((unsigned)grid), dim3(zm::kThreads), params, 0, s);
  if (e != cudaSuccess) return cuda_fail(e, "cudaLaunchKernel");
  ++h->launches;
  return ZERO_OK;
}

template <typename T>
zero_status run(zero_muon_t h, zm::Call& c, cudaStream_t s) {
  if (c.n == 0) return ZERO_OK;
  void* p[] = {&c};
  zero_status st = launch(h, (const void*)zm::muon_stats_kernel<T>, h->chunks, p, s);
  if (st == ZERO_OK) st = launch(h, (const void*)zm::muon_start_kernel<T>, h->chunks, p, s);
  int64_t tiles[3] = {0, 0, 0};
  for (const zm::Entry& e : h->entries) {
    const int64_t k = (e.k + 63) / 64, m = (e.rows + 63) / 64, n = (e.cols + 63) / 64;
    tiles[0] += k * k * e.batch;
    tiles[2] += m * n * e.batch;
  }
  tiles[1] = tiles[0];
  for (int i = 0; i < h->cfg.steps && st == ZERO_OK; ++i)
    for (int which = 0; which < 3 && st == ZERO_OK; ++which) {
      int cur = i % 2, last = i == h->cfg.steps - 1;
      float a = (float)h->cfg.coef[i][0], b = (float)h->cfg.coef[i][1], cc = (float)h->cfg.coef[i][2];
      void* q[] = {&c, &which, &cur, &last, &a, &b, &cc};
      st = launch(h, (const void*)zm::muon_product_kernel, tiles[which], q, s);
    }
  return st;
}

zero_status run_typed(zero_muon_t h, zm::Call& c, cudaStream_t s) {
  if (c.in_type == ZERO_FP16) return run<__half>(h, c, s);
  if (c.in_type == ZERO_BF16) return run<__nv_bfloat16>(h, c, s);
  return run<float>(h, c, s);
}

zero_status check_device(zero_muon_t h) {
  if (!h->has_device) return fail(ZERO_ECUDA, "no CUDA device for this handle");
  int cur = -1;
  const cudaError_t e = cudaGetDevice(&cur);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (cur != h->device)
    return fail(ZERO_ECUDA, "current device %d is not the handle's device %d", cur, h->device);
  return ZERO_OK;
}

// Allocates the workspace and fills in the addresses.
cudaError_t place(zero_muon_t h) {
  Layout lay;
  const int64_t n = (int64_t)h->entries.size();
  int64_t units = 0;
  for (const zm::Entry& e : h->entries) units += e.batch;
  const int64_t ws = lay.take(sizeof(zm::Workspace)), table = lay.take(n * sizeof(zm::Entry));
  const int64_t part = lay.take(h->chunks * sizeof(double)), ticket = lay.take(units * 4),
                inv = lay.take(units * 4);
  const int64_t cleared = lay.size;
  std::vector<int64_t> at;
  for (const zm::Entry& e : h->entries) {
    const int64_t x = e.batch * (int64_t)e.rows * e.ldx * 4, a = e.batch * (int64_t)e.k * e.ldk * 4;
    for (int64_t bytes : {x, x, a, a}) at.push_back(lay.take(bytes));
  }
  h->bytes = lay.size;
  cudaError_t e = cudaMalloc(reinterpret_cast<void**>(&h->mem), (size_t)h->bytes);
  if (e != cudaSuccess) return e;
  for (int64_t i = 0; i < n; ++i) {
    zm::Entry& en = h->entries[i];
    en.x[0] = reinterpret_cast<float*>(h->mem + at[4 * i]);
    en.x[1] = reinterpret_cast<float*>(h->mem + at[4 * i + 1]);
    en.a = reinterpret_cast<float*>(h->mem + at[4 * i + 2]);
    en.b = reinterpret_cast<float*>(h->mem + at[4 * i + 3]);
  }
  e = cudaMemset(h->mem, 0, (size_t)cleared);
  if (e == cudaSuccess && n > 0)
    e = cudaMemcpy(h->mem + table, h->entries.data(), n * sizeof(zm::Entry), cudaMemcpyHostToDevice);
  if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);
  h->call.ws = reinterpret_cast<zm::Workspace*>(h->mem + ws);
  h->call.entries = reinterpret_cast<const zm::Entry*>(h->mem + table);
  h->call.part = reinterpret_cast<double*>(h->mem + part);
  h->call.ticket = reinterpret_cast<unsigned*>(h->mem + ticket);
  h->call.inv = reinterpret_cast<float*>(h->mem + inv);
  return e;
}

}  // namespace

extern "C" {

zero_status zero_muon_config_default(zero_muon_config* cfg) {
  if (!cfg) return fail(ZERO_EINVAL, "cfg is NULL");
  std::memset(cfg, 0, sizeof(*cfg));
  cfg->grad_dtype = cfg->param_dtype = ZERO_FP16;
  cfg->nesterov = 1;
  cfg->steps = 5;
  cfg->scale_rule = ZERO_MUON_SCALE_ONE;
  cfg->lr = 2e-2;
  cfg->momentum = 0.95;
  cfg->eps = 1e-7;
  for (auto& c : cfg->coef) {
    c[0] = 3.4445;
    c[1] = -4.7750;
    c[2] = 2.0315;
  }
  return ZERO_OK;
}

zero_status zero_muon_create(const zero_muon_config* cfg, const zero_muon_shape* shapes, int32_t n,
                             zero_muon_t* out) {
  if (!out) return fail(ZERO_EINVAL, "out is NULL");
  *out = nullptr;
  if (!cfg) return fail(ZERO_EINVAL, "cfg is NULL");
  zero_status st = check(cfg);
  if (st != ZERO_OK) return st;
  if (n < 0 || n > ZERO_MUON_MAX_SHAPES)
    return fail(ZERO_ERANGE, "%d shapes: 0..%d are taken", n, ZERO_MUON_MAX_SHAPES);
  if (n > 0 && !shapes) return fail(ZERO_EINVAL, "shapes is NULL");
  for (int i = 0; i < n; ++i) {
    const zero_muon_shape& s = shapes[i];
    if (s.rows < 1 || s.cols < 1 || s.batch < 1)
      return fail(ZERO_EINVAL, "shape %d: rows, cols and batch must be >= 1", i);
    if (s.rows > 1 << 20 || s.cols > 1 << 20 || s.batch > 1 << 20 ||
        s.rows * s.cols > (int64_t)1 << 34)
      return fail(ZERO_ERANGE, "shape %d: %lld x %lld x %lld is beyond the limits", i,
                  (long long)s.rows, (long long)s.cols, (long long)s.batch);
  }
  zero_muon_handle* h = new (std::nothrow) zero_muon_handle;
  if (!h) return fail(ZERO_ENOMEM, "handle allocation failed");
  h->cfg = *cfg;
  int64_t units = 0;
  try {
    h->shapes.assign(shapes, shapes + n);
    for (int i = 0; i < n; ++i) {
      const zero_muon_shape& s = shapes[i];
      zm::Entry e = {};
      e.rows = (int32_t)s.rows;
      e.cols = (int32_t)s.cols;
      e.batch = (int32_t)s.batch;
      e.tall = s.rows > s.cols;
      e.k = (int32_t)std::min(s.rows, s.cols);
      e.l = (int32_t)std::max(s.rows, s.cols);
      e.ldx = (s.cols + 15) / 16 * 16;
      e.ldk = (e.k + 15) / 16 * 16;
      e.unit0 = (int32_t)units;
      e.vpr = (int32_t)((s.cols + zm::kVec - 1) / zm::kVec);
      e.chunks = (int32_t)(((int64_t)e.rows * e.vpr + zm::kChunk - 1) / zm::kChunk);
      e.chunk0 = (int32_t)h->chunks;
      e.s = (float)(cfg->scale_rule == ZERO_MUON_SCALE_RMS ? 0.2 * std::sqrt((double)e.l)
                    : cfg->scale_rule == ZERO_MUON_SCALE_ASPECT
                        ? std::sqrt(std::max(1.0, (double)s.rows / (double)s.cols))
                        : 1.0);
      units += s.batch;
      h->chunks += (int64_t)e.chunks * s.batch;
      if (units > INT32_MAX / 2 || h->chunks > INT32_MAX / 2) {
        delete h;
        return fail(ZERO_ERANGE, "too many matrices, or too large, for one handle");
      }
      h->entries.push_back(e);
    }
  } catch (const std::bad_alloc&) {
    delete h;
    return fail(ZERO_ENOMEM, "handle allocation failed");
  }
  h->call.n = n;
  h->call.eps = cfg->eps;
  h->call.mu = (float)cfg->momentum;
  h->call.nesterov = cfg->nesterov;
  int count = 0;
  if (cudaGetDeviceCount(&count) != cudaSuccess || count < 1) {
    cudaGetLastError();  // clear the sticky "no device" error
    *out = h;            // host-only handle
    return ZERO_OK;
  }
  cudaError_t e = cudaGetDevice(&h->device);
  if (e == cudaSuccess)
    e = cudaDeviceGetAttribute(&h->sms, cudaDevAttrMultiProcessorCount, h->device);
  try {
    if (e == cudaSuccess) e = place(h);
  } catch (const std::bad_alloc&) {
    e = cudaErrorMemoryAllocation;
  }
  if (e != cudaSuccess) {
    if (h->mem) cudaFree(h->mem);
    delete h;
    cudaGetLastError();
    return e == cudaErrorMemoryAllocation ? fail(ZERO_ENOMEM, "workspace allocation failed")
                                          : cuda_fail(e, "zero_muon_create");
  }
  h->has_device = true;
  *out = h;
  return ZERO_OK;
}

zero_status zero_muon_destroy(zero_muon_t h) {
  if (!h) return ZERO_OK;
  if (h->has_device) {
    int prev = -1;
    cudaGetDevice(&prev);
    cudaSetDevice(h->device);
    cudaDeviceSynchronize();
    cudaFree(h->mem);
    if (prev >= 0) cudaSetDevice(prev);
  }
  delete h;
  return ZERO_OK;
}

zero_status zero_muon_workspace_bytes(zero_muon_t h, int64_t* bytes) {
  if (!h || !bytes) return fail(ZERO_EINVAL, "NULL argument");
  *bytes = h->bytes;
  return ZERO_OK;
}

zero_status zero_muon_set_lr(zero_muon_t h, double lr) {
  if (!h) return fail(ZERO_EINVAL, "handle is NULL");
  if (!(lr >= 0.0)) return fail(ZERO_EINVAL, "lr must be >= 0");
  h->cfg.lr = lr;
  return ZERO_OK;
}

zero_status zero_muon_orthogonalize(zero_muon_t h, const zero_muon_operand* items, int32_t in_dtype,
                                    int32_t out_dtype, void* stream) {
  if (!h) return fail(ZERO_EINVAL, "handle is NULL");
  const int n = (int)h->entries.size();
  if (n > 0 && !items) return fail(ZERO_EINVAL, "items is NULL");
  for (int32_t d : {in_dtype, out_dtype})
    if (!dtype16(d) && d != ZERO_FP32)
      return fail(ZERO_EINVAL, "dtype must be ZERO_FP16, ZERO_BF16 or ZERO_FP32");
  zm::Call c = h->call;
  for (int i = 0; i < n; ++i) {
    const zero_muon_operand& t = items[i];
    const zm::Entry& e = h->entries[i];
    if (!t.in || !t.out) return fail(ZERO_EINVAL, "item %d: in and out must be non-NULL", i);
    if (t.in_row < 0 || t.in_batch < 0 || t.out_row < 0 || t.out_batch < 0)
      return fail(ZERO_EINVAL, "item %d: strides must be >= 0", i);
    if (e.rows > 1 && (t.in_row < e.cols || t.out_row < e.cols))
      return fail(ZERO_EINVAL, "item %d: a row stride is below its %d columns", i, e.cols);
    c.io[i].in = t.in;
    c.io[i].out = t.out;
    c.io[i].in_row = t.in_row;
    c.io[i].in_batch = t.in_batch;
    c.io[i].out_row = t.out_row;
    c.io[i].out_batch = t.out_batch;
  }
  const zero_status st = check_device(h);
  if (st != ZERO_OK) return st;
  c.step = 0;
  c.in_type = in_dtype;
  c.out_type = out_dtype;
  return run_typed(h, c, static_cast<cudaStream_t>(stream));
}

zero_status zero_muon_step(zero_muon_t h, const zero_muon_matrix* items, double grad_scale,
                           const zero_opt_step_info* decision, void* stream) {
  if (!h) return fail(ZERO_EINVAL, "handle is NULL");
  const int n = (int)h->entries.size();
  if (n > 0 && !items) return fail(ZERO_EINVAL, "items is NULL");
  if (!std::isfinite(grad_scale)) return fail(ZERO_EINVAL, "grad_scale is not finite");
  zm::Call c = h->call;
  for (int i = 0; i < n; ++i) {
    const zero_muon_matrix& t = items[i];
    const zm::Entry& e = h->entries[i];
    if (!t.grad || !t.momentum || !t.param16)
      return fail(ZERO_EINVAL, "item %d: grad, momentum and param16 must be non-NULL", i);
    c.io[i].in = t.grad;
    c.io[i].mom = t.momentum;
    c.io[i].master = t.master;
    c.io[i].out = t.param16;
    c.io[i].in_row = c.io[i].out_row = e.cols;
    c.io[i].in_batch = c.io[i].out_batch = (int64_t)e.rows * e.cols;
  }
  const zero_status st = check_device(h);
  if (st != ZERO_OK) return st;
  c.step = 1;
  c.in_type = h->cfg.grad_dtype;
  c.out_type = h->cfg.param_dtype;
  c.grad_scale = (float)grad_scale;
  c.decision = decision;
  c.decay = (float)(1.0 - h->cfg.lr * h->cfg.weight_decay);
  c.lr = (float)h->cfg.lr;
  return run_typed(h, c, static_cast<cudaStream_t>(stream));
}

zero_status zero_muon_last_step(zero_muon_t h, void* stream, zero_muon_info* out) {
  if (!h || !out) return fail(ZERO_EINVAL, "NULL argument");
  const zero_status st = check_device(h);
  if (st != ZERO_OK) return st;
  zm::Workspace w;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaMemcpyAsync(&w, h->call.ws, sizeof(w), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return cuda_fail(e, "zero_muon_last_step");
  out->skipped = w.skipped;
  out->fault = w.fault;
  return ZERO_OK;
}

zero_status zero_muon_launch_count(zero_muon_t h, int64_t* launches) {
  if (!h || !launches) return fail(ZERO_EINVAL, "NULL argument");
  *launches = h->launches;
  return ZERO_OK;
}

}  // extern "C"
