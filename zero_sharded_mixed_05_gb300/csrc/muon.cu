// muon.cu -- host side of the orthogonalised update (zero_muon.h): checks,
// the workspace and its layout, launches.
#include "muon_resident.cuh"

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
  const CUtensorMap* maps = nullptr;
  const int32_t* starts = nullptr;
  float4* parts = nullptr;
  int64_t chunks = 0;               // CTAs of the first two stages
  bool second = false;              // some matrix needs the second
  bool far = false;                 // X, both parts and twice the first, is more than L2 keeps
  int pair = 2;                     // CTAs a tile of the products
  int grid = 0;                     // CTAs of the products
  int smem = 0;
  int32_t count[3] = {0, 0, 0};     // tiles of a product of each kind
  int64_t launches = 0;
  uint32_t inject = 0;              // test hook, one call
  // launches of a handle whose matrices all stay on the chip (muon_resident.cuh)
  struct Launch {
    int32_t first, n, unit0, units, span, cols;
  };
  std::vector<Launch> resident;
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

// `early`: scheduled while the kernel before it still runs; it waits for that
// kernel by itself.
zero_status launch(zero_muon_t h, const void* fn, int64_t grid, void** params, cudaStream_t s,
                   bool early = false) {
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)grid);
  lc.blockDim = dim3(zm::kThreads);
  lc.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = &attr;
  lc.numAttrs = early ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelExC(&lc, fn, params);
  if (e != cudaSuccess) return cuda_fail(e, "cudaLaunchKernelExC");
  ++h->launches;
  return ZERO_OK;
}

const void* products_kernel(int pair) {
  return pair == 2 ? (const void*)zm::muon_products_kernel<2> : (const void*)zm::muon_products_kernel<1>;
}

// One cooperative launch (its CTAs wait for one another), in clusters of the pair.
cudaLaunchConfig_t products_config(zero_muon_t h, cudaLaunchAttribute* attr, cudaStream_t s) {
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)h->grid);
  lc.blockDim = dim3(zm::kProductThreads);
  lc.dynamicSmemBytes = (size_t)h->smem;
  lc.stream = s;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)h->pair;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeCooperative;
  attr[1].val.cooperative = 1;
  lc.attrs = attr;
  lc.numAttrs = 2;
  return lc;
}

// Parts that the depth of X X^T (`stages` of 128) is cut into, so that `tiles`
// tiles of it keep `slots` CTAs or pairs busy.  Each is at least eight stages
// deep and there are three at least, or the adding up costs what it saves
// (whole against cut: 8080x80 x 2 176 and 116 us, 300x5000 152 and 133, 11840x80
// x 24 483 and 368, 700x3000 in three of eight stages 140 and 140; in two
// 1024x4096 x 2 238 and 246, of four stages 400x1800 x 4 130 and 142).
int32_t splits_of(int64_t tiles, int64_t slots, int32_t stages) {
  const int64_t want = std::min<int64_t>({slots / std::max<int64_t>(tiles, 1), stages / 8, 8});
  if (want < 3) return 1;
  const int32_t deep = (int32_t)((stages + want - 1) / want);
  return (stages + deep - 1) / deep;
}

// Estimated cycles of one step's products with tiles of 128 * pair: full waves of
// tiles at what a stage of depth 128 takes (measured: 740 cycles for a single
// CTA's 128 x 128, 1060 for a pair's 256 x 256, whose tensor work alone is 512
// and 1024; a tile's epilogue at 3000 and 5500 where that is more), and a fixed
// part a product (from a tile's needs being met to its count: 5500 and 7500).
// A part of a cut tile writes its sums and the last reads them all: 2500 and
// 5000 a part, by which twenty shapes of 150x4000 to 1536x12000 choose the
// faster, or one within 2 %, with 4000 to 6000 as well; cuts at 2500 in all took
// pairs of 1024x4096 x 2, 1536x4000 and 768x4000 x 3 (257, 307 and 251 us).
// Measured, singles against pairs: 768x768 x 12 174 and
// 186 us, 2048x2048 215 and 241, 1536x1536 x 4 305 and 267, 4096x4096 1164 and
// 922; 1024x4096 x 2 235 and 257, 1536x4000 256 and 307, 768x4000 x 3 232 and 251;
// 1000x8000 x 2 405 and 364, 768x8000 x 4 516 and 426, 1536x12000 590 and 496.
double products_cost(const std::vector<zm::Entry>& entries, int pair, int sms) {
  const int tile = 128 * pair, slots = std::max(1, sms / pair);
  double tiles[2] = {0, 0}, work[3] = {0, 0, 0};
  for (const zm::Entry& e : entries) {
    const double nk = (e.k + tile - 1) / tile;
    const double tri = e.batch * nk * (nk + 1) / 2;
    const double full = (double)e.batch * ((e.rows + tile - 1) / tile) * ((e.cols + tile - 1) / tile);
    tiles[0] += tri;
    tiles[1] += full;
    work[0] += tri * ((e.l + 127) / 128);          // spread over parts below
    work[1] += tri * ((e.k + 127) / 128);
    work[2] += full * ((e.k + 127) / 128);
  }
  double cycles = 0;
  for (int which = 0; which < 3; ++which) {
    const double n = tiles[which == 2];
    if (which == 0) {
      const int32_t deep = (int32_t)(work[0] / n);
      const int32_t parts = splits_of((int64_t)n, slots, deep);
      if (parts > 1) {
        cycles += deep / parts * (pair == 2 ? 1060 : 740) + (pair == 2 ? 7500 : 5500) + parts * (pair == 2 ? 5000 : 2500);
        continue;
      }
    }
    const double tile_cycles = pair == 2 ? std::max(5500.0, 1060 * work[which] / n) : std::max(3000.0, 740 * work[which] / n);
    cycles += std::ceil(n / slots) * tile_cycles + (pair == 2 ? 7500 : 5500);
  }
  return cycles;
}

template <typename T, int N>
const void* resident_kernel(int cols, bool two) {
  return cols == 256 ? (const void*)zm::muon_resident_kernel<T, 256, 1, N>
         : two       ? (const void*)zm::muon_resident_kernel<T, 128, 2, N>
                     : (const void*)zm::muon_resident_kernel<T, 128, 1, N>;
}

int resident_bytes(int cols, int span) {
  return cols == 128 ? zm::resident_bytes<128>(span) : zm::resident_bytes<256>(span);
}

template <typename T, int N>
zero_status run_resident(zero_muon_t h, const zm::Start<N>& start, cudaStream_t s) {
  zm::Resident r = {};
  r.steps = h->cfg.steps;
  for (int i = 0; i < r.steps; ++i)
    for (int j = 0; j < 3; ++j) r.coef[i][j] = (float)h->cfg.coef[i][j];
  r.head = 1;
  r.inject = h->inject != 0;
  h->inject = 0;
  for (const auto& l : h->resident) {
    r.first = l.first;
    r.n = l.n;
    r.unit0 = l.unit0;
    r.span = l.span;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)l.span;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3((unsigned)(l.units * l.span));
    lc.blockDim = dim3(zm::kResidentThreads);
    lc.dynamicSmemBytes = (size_t)resident_bytes(l.cols, l.span);
    lc.stream = s;
    lc.attrs = &attr;
    lc.numAttrs = 1;
    void* p[] = {&r, const_cast<zm::Start<N>*>(&start)};
    const cudaError_t e = cudaLaunchKernelExC(&lc, resident_kernel<T, N>(l.cols, l.units > h->sms), p);
    if (e != cudaSuccess) return cuda_fail(e, "cudaLaunchKernelExC");
    ++h->launches;
    r.head = 0;
  }
  return ZERO_OK;
}

// Every kernel that a call of this handle may launch, readied for its shared memory.
template <typename T, int N>
cudaError_t ready_resident(const zero_muon_handle* h) {
  for (const auto& l : h->resident) {
    const cudaError_t e = cudaFuncSetAttribute(resident_kernel<T, N>(l.cols, l.units > h->sms), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               resident_bytes(l.cols, zm::kResidentSpan));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}
template <int N>
cudaError_t ready_resident(const zero_muon_handle* h) {
  cudaError_t e = ready_resident<__half, N>(h);
  if (e == cudaSuccess) e = ready_resident<__nv_bfloat16, N>(h);
  return e == cudaSuccess ? ready_resident<float, N>(h) : e;
}

// Decides whether the handle's matrices stay on the chip: if each of them can,
// and that takes less time by estimate (with matrices too large among them they
// all go through the workspace, where the small ones cost next to nothing).
// A step of a wave of them takes 5 microseconds with 128 columns a CTA (two on
// an SM), 6.6 with 256 and 10 with more CTAs a matrix, which add up their shares
// of A.  Measured, on the chip against the workspace: 128x128 29 and 64 us,
// 128x1024 x 32 61 and 95, 64x64 x 1000 109 and 204, but 100x1500 x 60 230 and
// 178.  Matrices that need fewer CTAs go in launches of
// their own unless all fit on the device side by side.
void choose_resident(zero_muon_t h) {
  if (h->entries.empty()) return;
  int most = 1;
  int64_t units = 0;
  const auto span_of = [](const zm::Entry& e) {
    int span = 1;
    while (span * 256 < e.l) span *= 2;
    return span;
  };
  for (const zm::Entry& e : h->entries) {
    if (e.k > zm::kResidentSide || e.l > 256 * zm::kResidentSpan) return;
    most = std::max(most, span_of(e));
    units += e.batch;
  }
  const bool together = units * most <= h->sms;
  double here = 0;
  for (const zm::Entry& e : h->entries) {
    const int span = span_of(e);
    const double at_once = e.l <= 128 ? 2 * h->sms : h->sms / span;
    here += (together ? 1.0 / h->entries.size() : std::ceil(e.batch / at_once)) *
            ((span > 1 || (together && most > 1) ? 10.0 : e.l <= 128 ? 5.0 : 6.6) * h->cfg.steps + 6);
  }
  const double there = 25 + products_cost(h->entries, 1, h->sms) * h->cfg.steps / 1900;
  if (here > 1.1 * there) return;
  // entries in order of span, so that a launch's are side by side
  std::stable_sort(h->entries.begin(), h->entries.end(), [&](const zm::Entry& x, const zm::Entry& y) {
    return span_of(x) != span_of(y) ? span_of(x) > span_of(y) : (x.l > 128) > (y.l > 128);
  });
  int32_t unit = 0;
  for (int32_t i = 0; i < (int32_t)h->entries.size(); ++i) {
    zm::Entry& e = h->entries[i];
    e.unit0 = unit;
    unit += e.batch;
    const int span = together ? most : span_of(e);
    const int cols = e.l <= 128 && span == 1 && !(together && h->resident.size()) ? 128 : 256;
    if (h->resident.empty() || (!together && (h->resident.back().span != span || h->resident.back().cols != cols)))
      h->resident.push_back({i, 0, e.unit0, 0, span, cols});
    ++h->resident.back().n;
    h->resident.back().units += e.batch;
  }
}

template <typename T, int N>
zero_status run(zero_muon_t h, const zm::Call& c, const zm::Io* io, cudaStream_t s) {
  zm::Start<N> start;
  start.c = c;
  std::copy(io, io + c.n, start.io);
  if (!h->resident.empty()) return run_resident<T, N>(h, start, s);
  void* p[] = {&start};
  zero_status st = launch(h, (const void*)zm::muon_stats_kernel<T, N>, h->chunks, p, s);
  if (st != ZERO_OK) return st;
  if (h->second) {
    void* q[] = {&start.c};
    st = launch(h, (const void*)zm::muon_start_kernel<T>, h->chunks, q, s, true);
    if (st != ZERO_OK) return st;
  }
  zm::Products pr = {};
  pr.c = c;
  pr.maps = h->maps;
  pr.starts = h->starts;
  pr.parts = h->parts;
  std::copy(h->count, h->count + 3, pr.count);
  pr.tiles = ((int64_t)h->count[0] + h->count[1] + h->count[2]) * h->cfg.steps;
  pr.steps = h->cfg.steps;
  pr.far = h->far;
  pr.inject = h->inject;
  h->inject = 0;
  for (int i = 0; i < pr.steps; ++i)
    for (int j = 0; j < 3; ++j) pr.coef[i][j] = (float)h->cfg.coef[i][j];
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t lc = products_config(h, attr, s);
  void* r[] = {&pr};
  const cudaError_t e = cudaLaunchKernelExC(&lc, products_kernel(h->pair), r);
  if (e != cudaSuccess) return cuda_fail(e, "cudaLaunchKernelExC");
  ++h->launches;
  return ZERO_OK;
}

template <typename T>
zero_status run(zero_muon_t h, const zm::Call& c, const zm::Io* io, cudaStream_t s) {
  if (c.n == 0) return ZERO_OK;
  return c.n <= 8 ? run<T, 8>(h, c, io, s) : run<T, zm::kMaxEntries>(h, c, io, s);
}

zero_status run_typed(zero_muon_t h, const zm::Call& c, const zm::Io* io, cudaStream_t s) {
  if (c.in_type == ZERO_FP16) return run<__half>(h, c, io, s);
  if (c.in_type == ZERO_BF16) return run<__nv_bfloat16>(h, c, io, s);
  return run<float>(h, c, io, s);
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

zero_status read_workspace(zero_muon_t h, void* stream, zm::Workspace* w, const char* what) {
  const zero_status st = check_device(h);
  if (st != ZERO_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaMemcpyAsync(w, h->call.ws, sizeof(*w), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  return e == cudaSuccess ? ZERO_OK : cuda_fail(e, what);
}

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                                CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                CUtensorMapFloatOOBfill);

// Map of a matrix in pieces (muon_kernels.cuh), [batch] of them: a quarter of a
// piece's 128 rows, the quarters, pieces across, rows of pieces, matrices.  A
// box is 128 rows of eight pieces; what lies outside reads as zero.
bool encode(EncodeTiled fn, CUtensorMap* map, __half* p, int64_t rows, int64_t ld, int64_t batch) {
  const cuuint64_t dim[5] = {256, 4, (cuuint64_t)ld / 8, (cuuint64_t)(rows + 127) / 128, (cuuint64_t)batch};
  const cuuint64_t stride[4] = {512, 2048, (cuuint64_t)ld * 256, (cuuint64_t)zm::block_size(rows, ld) * 2};
  const cuuint32_t box[5] = {256, 4, 8, 1, 1}, step[5] = {1, 1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5, p, dim, stride, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Allocates the workspace, fills in the addresses and readies the products.
cudaError_t place(zero_muon_t h) {
  choose_resident(h);
  if (!h->resident.empty()) {
    const int64_t table = 256;
    h->bytes = table + (int64_t)(h->entries.size() * sizeof(zm::Entry));
    cudaError_t e = cudaMalloc(reinterpret_cast<void**>(&h->mem), (size_t)h->bytes);
    if (e == cudaSuccess) e = cudaMemset(h->mem, 0, (size_t)table);
    if (e == cudaSuccess)
      e = cudaMemcpy(h->mem + table, h->entries.data(), h->entries.size() * sizeof(zm::Entry), cudaMemcpyHostToDevice);
    if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);
    h->call.ws = reinterpret_cast<zm::Workspace*>(h->mem);
    h->call.entries = reinterpret_cast<const zm::Entry*>(h->mem + table);
    if (e == cudaSuccess) e = h->entries.size() <= 8 ? ready_resident<8>(h) : ready_resident<zm::kMaxEntries>(h);
    return e;
  }
  Layout lay;
  const int64_t n = (int64_t)h->entries.size();
  h->pair = n > 0 && products_cost(h->entries, 1, h->sms) <= products_cost(h->entries, 2, h->sms) ? 1 : 2;
  int64_t units = 0;
  for (const zm::Entry& e : h->entries) units += e.batch;
  const void* kernel = products_kernel(h->pair);
  h->smem = zm::kProductSmem;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, h->smem);
  // as many pairs as can be on the device at once
  h->grid = h->pair;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t lc = products_config(h, attr, nullptr);
  int clusters = 0;
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&clusters, kernel, &lc);
  if (e != cudaSuccess) return e;
  const int tile = 128 * h->pair;
  clusters = std::max(clusters, 1);
  std::vector<int32_t> starts;
  int32_t cuts = 0, slots = 0, triangles = 0;
  for (const zm::Entry& en : h->entries) {
    const int32_t nk = (en.k + tile - 1) / tile;
    triangles += en.batch * (nk * (nk + 1) / 2);
  }
  for (zm::Entry& en : h->entries) {
    const int32_t nk = (en.k + tile - 1) / tile, ntri = nk * (nk + 1) / 2;
    en.splits = splits_of(triangles, clusters, (en.l + zm::kDepth - 1) / zm::kDepth);
    en.cuts = en.splits > 1 ? ntri * h->pair : 0;
    en.cut0 = cuts;
    en.slot0 = slots;
    cuts += en.batch * en.cuts;
    slots += en.splits > 1 ? en.batch * ntri * en.splits : 0;
    starts.push_back(h->count[0]);
    h->count[0] += en.batch * ntri * en.splits;
  }
  for (const zm::Entry& en : h->entries) {
    const int32_t nk = (en.k + tile - 1) / tile;
    starts.push_back(h->count[1]);
    h->count[1] += en.batch * (nk * (nk + 1) / 2);
  }
  for (const zm::Entry& en : h->entries) {
    starts.push_back(h->count[2]);
    h->count[2] += en.batch * ((en.rows + tile - 1) / tile) * ((en.cols + tile - 1) / tile);
  }
  h->grid = h->pair * std::min(clusters, std::max({1, h->count[0], h->count[1], h->count[2]}));
  const int64_t ws = lay.take(sizeof(zm::Workspace)), table = lay.take(n * sizeof(zm::Entry));
  const int64_t maps = lay.take(4 * n * sizeof(CUtensorMap));
  const int64_t io = lay.take(n * sizeof(zm::Io)), first = lay.take(starts.size() * sizeof(int32_t));
  const int64_t part = lay.take(h->chunks * sizeof(double)), ticket = lay.take(units * 4),
                inv = lay.take(units * 4), done = lay.take(units * 4), cut = lay.take(cuts * 4ll);
  const int64_t parts = lay.take((int64_t)slots * h->pair * 128 * tile * 4);
  std::vector<int64_t> at;
  for (const zm::Entry& e : h->entries) {
    const int64_t x = e.batch * zm::block_size(e.rows, e.ldx) * 2, a = e.batch * zm::block_size(e.k, e.ldk) * 2;
    for (int64_t bytes : {x, x, x, a, a, e.batch * e.ldk * 4}) at.push_back(lay.take(bytes));
  }
  int l2 = 0;
  e = cudaDeviceGetAttribute(&l2, cudaDevAttrL2CacheSize, h->device);
  if (e != cudaSuccess) return e;
  int64_t x_bytes = 0;
  for (const zm::Entry& en : h->entries) x_bytes += en.batch * zm::block_size(en.rows, en.ldx) * 6;
  h->far = x_bytes > l2 / 8 * 7ll;
  h->bytes = lay.size;
  std::vector<CUtensorMap> map(4 * n);
  e = cudaMalloc(reinterpret_cast<void**>(&h->mem), (size_t)h->bytes);
  if (e != cudaSuccess) return e;
  void* sym = nullptr;
  cudaDriverEntryPointQueryResult found;
  e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &sym, 12000, cudaEnableDefault, &found);
  if (e != cudaSuccess) return e;
  if (found != cudaDriverEntryPointSuccess) return cudaErrorSymbolNotFound;
  const EncodeTiled fn = reinterpret_cast<EncodeTiled>(sym);
  for (int64_t i = 0; i < n; ++i) {
    zm::Entry& en = h->entries[i];
    const auto half = [&](int j) { return reinterpret_cast<__half*>(h->mem + at[6 * i + j]); };
    en.x[0] = half(0);
    en.x[1] = half(1);
    en.lo = half(2);
    en.a = half(3);
    en.b = half(4);
    en.diag = reinterpret_cast<float*>(half(5));
    CUtensorMap* m = &map[4 * i];
    const bool ok = encode(fn, m, en.x[0], en.rows, en.ldx, en.batch) &&
                    encode(fn, m + 1, en.x[1], en.rows, en.ldx, en.batch) &&
                    encode(fn, m + 2, en.a, en.k, en.ldk, en.batch) && encode(fn, m + 3, en.b, en.k, en.ldk, en.batch);
    if (!ok) return cudaErrorInvalidValue;
  }
  // counters, and what pads the matrices
  e = cudaMemset(h->mem, 0, (size_t)h->bytes);
  const auto copy = [&](int64_t to, const void* from, size_t bytes) {
    if (e == cudaSuccess && bytes > 0)
      e = cudaMemcpy(h->mem + to, from, bytes, cudaMemcpyHostToDevice);
  };
  copy(table, h->entries.data(), n * sizeof(zm::Entry));
  copy(maps, map.data(), map.size() * sizeof(CUtensorMap));
  copy(first, starts.data(), starts.size() * sizeof(int32_t));
  if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);
  h->call.ws = reinterpret_cast<zm::Workspace*>(h->mem + ws);
  h->call.entries = reinterpret_cast<const zm::Entry*>(h->mem + table);
  h->call.io = reinterpret_cast<zm::Io*>(h->mem + io);
  h->call.part = reinterpret_cast<double*>(h->mem + part);
  h->call.ticket = reinterpret_cast<unsigned*>(h->mem + ticket);
  h->call.inv = reinterpret_cast<float*>(h->mem + inv);
  h->call.done = reinterpret_cast<uint32_t*>(h->mem + done);
  h->call.cut = reinterpret_cast<uint32_t*>(h->mem + cut);
  h->parts = reinterpret_cast<float4*>(h->mem + parts);
  h->maps = reinterpret_cast<const CUtensorMap*>(h->mem + maps);
  h->starts = reinterpret_cast<const int32_t*>(h->mem + first);
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
  int count = 0;
  const bool device = cudaGetDeviceCount(&count) == cudaSuccess && count > 0;
  cudaError_t e = cudaSuccess;
  if (device) {
    e = cudaGetDevice(&h->device);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&h->sms, cudaDevAttrMultiProcessorCount, h->device);
  } else {
    cudaGetLastError();  // clear the sticky "no device" error
  }
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
      e.item = i;
      e.ldx = (s.cols + 31) / 32 * 32;
      e.ldk = (e.k + 31) / 32 * 32;
      e.across = (int32_t)(e.ldx / 32);
      e.s = (float)(cfg->scale_rule == ZERO_MUON_SCALE_RMS ? 0.2 * std::sqrt((double)e.l)
                    : cfg->scale_rule == ZERO_MUON_SCALE_ASPECT
                        ? std::sqrt(std::max(1.0, (double)s.rows / (double)s.cols))
                        : 1.0);
      h->entries.push_back(e);
    }
    // the products' tiles go out from the deepest to the shallowest
    std::stable_sort(h->entries.begin(), h->entries.end(), [](const zm::Entry& x, const zm::Entry& y) {
      return x.k != y.k ? x.k > y.k : x.l > y.l;
    });
    // Blocks a warp of the first two stages: one wave of CTAs, three an SM, up
    // to 8.  (Twelve of 2304x768: 378 us at one block and two waves, 362 at
    // two and one; 14336x4096: 2646 at 16 blocks, 2607 at 8.)
    int64_t blocks = 0;
    for (const zm::Entry& e : h->entries) blocks += (int64_t)e.batch * ((e.rows + 31) / 32) * e.across;
    const int64_t wave = (int64_t)(zm::kThreads / 32) * 3 * std::max(h->sms, 1);
    h->call.blocks = (int32_t)std::max<int64_t>(1, std::min<int64_t>(8, (blocks + wave - 1) / wave));
    const int64_t chunk = h->call.blocks * (zm::kThreads / 32);
    double tiles = 0;
    for (zm::Entry& e : h->entries) {
      e.chunks = (int32_t)(((int64_t)(e.rows + 31) / 32 * e.across + chunk - 1) / chunk);
      e.unit0 = (int32_t)units;
      e.chunk0 = (int32_t)h->chunks;
      units += e.batch;
      h->chunks += (int64_t)e.chunks * e.batch;
      h->second = h->second || e.chunks > 1;
      tiles += (e.rows / 128 + 1.0) * (e.cols / 128 + 1.0) * e.batch;
      if (units > INT32_MAX / 2 || h->chunks > INT32_MAX / 2 || tiles > INT32_MAX / 64) {
        delete h;
        return fail(ZERO_ERANGE, "too many matrices, or too large, for one handle");
      }
    }
  } catch (const std::bad_alloc&) {
    delete h;
    return fail(ZERO_ENOMEM, "handle allocation failed");
  }
  h->call.n = n;
  h->call.eps = cfg->eps;
  h->call.mu = (float)cfg->momentum;
  h->call.nesterov = cfg->nesterov;
  if (!device) {
    *out = h;            // host-only handle
    return ZERO_OK;
  }
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
  zm::Io io[zm::kMaxEntries] = {};
  for (int i = 0; i < n; ++i) {
    const zero_muon_operand& t = items[i];
    const zero_muon_shape& e = h->shapes[i];
    if (!t.in || !t.out) return fail(ZERO_EINVAL, "item %d: in and out must be non-NULL", i);
    if (t.in_row < 0 || t.in_batch < 0 || t.out_row < 0 || t.out_batch < 0)
      return fail(ZERO_EINVAL, "item %d: strides must be >= 0", i);
    if (e.rows > 1 && (t.in_row < e.cols || t.out_row < e.cols))
      return fail(ZERO_EINVAL, "item %d: a row stride is below its %lld columns", i,
                  (long long)e.cols);
    if (e.batch > 1 && t.out_batch < e.cols)
      return fail(ZERO_EINVAL, "item %d: its matrices' results lie on one another", i);
    io[i].in = t.in;
    io[i].out = t.out;
    io[i].in_row = t.in_row;
    io[i].in_batch = t.in_batch;
    io[i].out_row = t.out_row;
    io[i].out_batch = t.out_batch;
  }
  const zero_status st = check_device(h);
  if (st != ZERO_OK) return st;
  c.step = 0;
  c.in_type = in_dtype;
  c.out_type = out_dtype;
  return run_typed(h, c, io, static_cast<cudaStream_t>(stream));
}

zero_status zero_muon_step(zero_muon_t h, const zero_muon_matrix* items, double grad_scale,
                           const zero_opt_step_info* decision, void* stream) {
  if (!h) return fail(ZERO_EINVAL, "handle is NULL");
  const int n = (int)h->entries.size();
  if (n > 0 && !items) return fail(ZERO_EINVAL, "items is NULL");
  if (!std::isfinite(grad_scale)) return fail(ZERO_EINVAL, "grad_scale is not finite");
  zm::Call c = h->call;
  zm::Io io[zm::kMaxEntries] = {};
  for (int i = 0; i < n; ++i) {
    const zero_muon_matrix& t = items[i];
    const zero_muon_shape& e = h->shapes[i];
    if (!t.grad || !t.momentum || !t.param16)
      return fail(ZERO_EINVAL, "item %d: grad, momentum and param16 must be non-NULL", i);
    io[i].in = t.grad;
    io[i].mom = t.momentum;
    io[i].master = t.master;
    io[i].out = t.param16;
    io[i].in_row = io[i].out_row = e.cols;
    io[i].in_batch = io[i].out_batch = e.rows * e.cols;
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
  return run_typed(h, c, io, static_cast<cudaStream_t>(stream));
}

zero_status zero_muon_last_step(zero_muon_t h, void* stream, zero_muon_info* out) {
  if (!h || !out) return fail(ZERO_EINVAL, "NULL argument");
  zm::Workspace w;
  const zero_status st = read_workspace(h, stream, &w, "zero_muon_last_step");
  if (st != ZERO_OK) return st;
  out->skipped = w.skipped;
  out->fault = h->resident.empty() ? w.fault : w.last;
  return ZERO_OK;
}

zero_status zero_muon_fault_count(zero_muon_t h, void* stream, int64_t* faults) {
  if (!h || !faults) return fail(ZERO_EINVAL, "NULL argument");
  zm::Workspace w;
  const zero_status st = read_workspace(h, stream, &w, "zero_muon_fault_count");
  if (st != ZERO_OK) return st;
  *faults = (int64_t)w.faults + (h->resident.empty() ? w.fault : 0);
  return ZERO_OK;
}

zero_status zero_muon_inject_wait_fault(zero_muon_t h) {
  if (!h) return fail(ZERO_EINVAL, "handle is NULL");
  h->inject = 1u << 30;
  return ZERO_OK;
}

zero_status zero_muon_launch_count(zero_muon_t h, int64_t* launches) {
  if (!h || !launches) return fail(ZERO_EINVAL, "NULL argument");
  *launches = h->launches;
  return ZERO_OK;
}

}  // extern "C"
