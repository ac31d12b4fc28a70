// block.cu -- the host side of the join of a block with the residual stream
// (zero_block.h): checks, choice of kernel and launch shape; the sums of the
// gains' gradients over CTAs; and dropout by itself.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <limits>
#include <mutex>
#include <new>

#include "block_host.h"
#include "block_kernels.cuh"
#include "host_util.h"

namespace {

using zo::Drop;
using zo::fail;
using zo::JoinArgs;
using zo::JoinRow;
using zo::Num;

constexpr int kMaxDim = 16384;
// so that a row of each tensor fits shared memory:
constexpr int kMaxDim32 = 8192;          // of binary32 blocks
constexpr int kMaxDimGated = 12288;      // of gated 16-bit blocks on a binary32 stream
constexpr int kMaxSmem = 227 * 1024 - 1024;
constexpr int kMaxPerSm = 4;             // CTAs an SM

struct FoldArgs {
  const float* part;    // as JoinArgs::part
  float* out[2];
  int32_t grid, dim, chunks;
};

// Sums the CTAs' partial gradients in index order: 64 columns a CTA, 32 threads a
// pair of columns, each over every 32nd partial.  Bound by its launch and one or two
// round trips: with the writing of the partials it adds 2.2 us to a small gradient and
// 4.2 to one of 4096 columns.
__global__ void __launch_bounds__(1024) join_fold_kernel(const __grid_constant__ FoldArgs a) {
  __shared__ float s[32][65];
  cudaGridDependencySynchronize();   // launched while the partials are still written
  const int lane = threadIdx.x % 32, part = threadIdx.x / 32, cols = 16 * a.chunks;
  const int col = blockIdx.x * 64 + 2 * lane;
  float2 sum = make_float2(0.0f, 0.0f);
  if (col < cols) {
    const float* at = a.part + col;
    for (int c = part; c < a.grid; c += 320) {
      float2 v[10];                  // ten loads on their way at once
#pragma unroll
      for (int k = 0; k < 10; ++k)
        v[k] = c + 32 * k < a.grid ? *reinterpret_cast<const float2*>(at + (int64_t)(c + 32 * k) * cols)
                                   : make_float2(0.0f, 0.0f);
#pragma unroll
      for (int k = 0; k < 10; ++k) sum = __fadd2_rn(sum, v[k]);
    }
  }
  s[part][2 * lane] = sum.x;
  s[part][2 * lane + 1] = sum.y;
  __syncthreads();
  // a warp a pair of columns: each lane has one thread's sums
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float v = s[lane][2 * part + k];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, o));
    // number col % 4 of the first or the last half of a chunk, of the first gain or the second
    const int at = blockIdx.x * 64 + 2 * part + k, quarter = at / (4 * a.chunks), rest = at - quarter * 4 * a.chunks;
    const int e = rest / 4 * 8 + quarter % 2 * 4 + rest % 4;
    float* out = at < cols ? a.out[quarter / 2] : nullptr;
    if (lane == 0 && out && e < a.dim) out[e] = v;
  }
}

struct DropArgs {
  const char* in;
  char* out;
  int64_t rows, blocks;        // blocks of eight a row
  int64_t cols, in_stride, out_stride;   // strides in bytes
  Drop drop;
};

enum { kFlat, kWide, kTiles };

// kFlat: whole blocks of eight one after another on 16-byte boundaries, of which a
// thread takes kBlocks at a time and has the next ones on their way meanwhile.
// kWide: rows on 16-byte boundaries, a block a thread and step.  kTiles: a warp takes
// 256 numbers of a row, which pass through shared memory so that global memory is
// read and written 32 numbers next to one another (16,000 rows of 4095 in fp16 82 us;
// with the 16-byte granules that they lie in, shifted in registers, 112 and, with four
// tiles on their way, 132: integer work bounds it, and the shifts are more of that).
template <typename T, int kMode>
__global__ void __launch_bounds__(256) drop_kernel(const __grid_constant__ DropArgs a) {
  constexpr int kE = 16 / (int)sizeof(T), kV = 8 / kE;
  const uint32_t step = zo::step_of(a.drop);
  const auto apply = [&](uint4* p, int64_t block) {
    const uint4 m = zo::kept(a.drop, step, block);
    float2 x[4];
#pragma unroll
    for (int v = 0; v < kV; ++v) zo::unpack<T>(p[v], x + v * (kE / 2));
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = __fmul2_rn(x[k], zo::both(a.drop.factor));
    if constexpr (sizeof(T) == 4) zo::mask8(x, m);
#pragma unroll
    for (int v = 0; v < kV; ++v) p[v] = zo::pack<T>(x + v * (kE / 2));
    if constexpr (sizeof(T) == 2) p[0] = make_uint4(p[0].x & m.x, p[0].y & m.y, p[0].z & m.z, p[0].w & m.w);
  };
  if constexpr (kMode == kFlat) {
    constexpr int kBlocks = sizeof(T) == 2 ? 2 : 1;
    const int64_t n = a.blocks, stride = (int64_t)gridDim.x * blockDim.x;
    const uint4* in = reinterpret_cast<const uint4*>(a.in);
    uint4* out = reinterpret_cast<uint4*>(a.out);
    uint4 p[kBlocks][kV], q[kBlocks][kV];
    const auto load = [&](int64_t b0, uint4 (*to)[kV]) {
#pragma unroll
      for (int i = 0; i < kBlocks; ++i)
        if (b0 + i * stride < n)
#pragma unroll
          for (int v = 0; v < kV; ++v) to[i][v] = in[(b0 + i * stride) * kV + v];
    };
    int64_t b0 = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    load(b0, p);
    for (; b0 < n; b0 += kBlocks * stride) {
      load(b0 + kBlocks * stride, q);
#pragma unroll
      for (int i = 0; i < kBlocks; ++i)
        if (b0 + i * stride < n) {
          apply(p[i], b0 + i * stride);
#pragma unroll
          for (int v = 0; v < kV; ++v) out[(b0 + i * stride) * kV + v] = p[i][v];
        }
#pragma unroll
      for (int i = 0; i < kBlocks; ++i)
#pragma unroll
        for (int v = 0; v < kV; ++v) p[i][v] = q[i][v];
    }
  } else if constexpr (kMode == kWide) {
    const int64_t n = a.rows * a.blocks, stride = (int64_t)gridDim.x * blockDim.x;
    for (int64_t b = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; b < n; b += stride) {
      const int64_t row = a.rows == 1 ? 0 : b / a.blocks, c = b - row * a.blocks;
      const T* from = reinterpret_cast<const T*>(a.in + row * a.in_stride) + c * 8;
      T* to = reinterpret_cast<T*>(a.out + row * a.out_stride) + c * 8;
      const int64_t left = a.cols - c * 8;
      if (left >= 8) {
        uint4 p[kV];
#pragma unroll
        for (int v = 0; v < kV; ++v) p[v] = reinterpret_cast<const uint4*>(from)[v];
        apply(p, b);
#pragma unroll
        for (int v = 0; v < kV; ++v) reinterpret_cast<uint4*>(to)[v] = p[v];
      } else {
        const uint4 m = zo::kept(a.drop, step, b);
        for (int k = 0; k < left; ++k)
          to[k] = Num<T>::put(zo::word_of(m, k / 2) >> k % 2 * 16 & 1
                                  ? __fmul_rn(Num<T>::get(from[k]), a.drop.factor) : 0.0f);
      }
    }
  } else {
    __shared__ alignas(16) T s_tile[8][256];
    T* tile = s_tile[threadIdx.x / 32];
    const int l = threadIdx.x % 32;
    const int64_t per = (a.cols + 255) / 256, n = a.rows * per;
    for (int64_t w = (int64_t)blockIdx.x * 8 + threadIdx.x / 32; w < n; w += (int64_t)gridDim.x * 8) {
      const int64_t row = w / per, begin = (w - row * per) * 256;
      const T* from = reinterpret_cast<const T*>(a.in + row * a.in_stride);
      T* to = reinterpret_cast<T*>(a.out + row * a.out_stride);
      T x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int64_t e = begin + k * 32 + l;
        x[k] = e < a.cols ? from[e] : Num<T>::put(0.0f);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) tile[k * 32 + l] = x[k];
      __syncwarp();
      apply(reinterpret_cast<uint4*>(tile + 8 * l), row * a.blocks + begin / 8 + l);
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int64_t e = begin + k * 32 + l;
        if (e < a.cols) to[e] = tile[k * 32 + l];
      }
      __syncwarp();
    }
  }
}

template <typename T>
const void* drop_of_type(int mode) {
  return mode == kFlat   ? (const void*)drop_kernel<T, kFlat>
         : mode == kWide ? (const void*)drop_kernel<T, kWide>
                         : (const void*)drop_kernel<T, kTiles>;
}

zero_status cuda_fail(cudaError_t e, const char* what) {
  cudaGetLastError();
  return fail(ZERO_ECUDA, "%s: %s", what, cudaGetErrorString(e));
}

int elem_size(int32_t dtype) { return dtype == ZERO_FP32 ? 4 : 2; }

bool known(int32_t dtype) { return dtype == ZERO_FP16 || dtype == ZERO_BF16 || dtype == ZERO_FP32; }

bool on16(const void* p, int64_t stride_bytes, int64_t rows) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (rows <= 1 || stride_bytes % 16 == 0);
}

}  // namespace

struct zero_block_handle {
  zero_block_config cfg;
  bool has_device = false;
  int device = -1;
  int sms = 0;
  float* part = nullptr;     // and, behind it, the row of zeros
  float* zeros = nullptr;
  int64_t max_grid = 0;      // CTAs that `part` has room for
  int64_t launches = 0;
  std::mutex mu;
  struct {
    const void* fn;
    int threads, smem, ctas;
  } occ[32] = {};            // launch shapes seen, oldest overwritten
  int seen = 0;

  // CTAs of a kernel that an SM holds at once, at most kMaxPerSm.
  int resident(const void* fn, int threads, int smem) {
    std::lock_guard<std::mutex> lock(mu);
    for (const auto& o : occ)
      if (o.fn == fn && o.threads == threads && o.smem == smem) return o.ctas;
    int n = 0;
    cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, fn, threads, smem) != cudaSuccess) cudaGetLastError();
    n = std::max(1, std::min(n, kMaxPerSm));
    occ[seen++ % 32] = {fn, threads, smem, n};
    return n;
  }
};

namespace {

// A row tensor of the call, or none where `p` is NULL.
JoinRow row_of(const zero_block_rows& r, int es) {
  return {static_cast<char*>(r.data), r.data ? r.stride * es : 0, 0};
}

zero_status run(zero_block_t h, const zero_block_buffers* b, void* stream, bool backward) {
  if (!h) return fail(ZERO_EINVAL, "handle is NULL");
  if (!b) return fail(ZERO_EINVAL, "buffers are NULL");
  const zero_block_config& c = h->cfg;
  if (b->tokens < 0) return fail(ZERO_EINVAL, "tokens must be >= 0");
  const int es = elem_size(c.dtype), ss = elem_size(c.stream_dtype);
  const bool mixed = c.stream_dtype != c.dtype;
  const bool with_y = b->y.data != nullptr, with_gate = with_y && c.gate != ZERO_GATE_NONE;
  JoinArgs a = {};
  if (with_y) a.y = row_of(b->y, es);
  if (with_gate) a.gate = row_of(b->gate, es);
  if (backward) {
    a.x = row_of(b->x_out, ss);
    a.dxo = row_of(b->dx_out, ss);
    if (c.norm_out) a.dh = row_of(b->dh, es);
    a.dx = row_of(b->dx, ss);
    if (with_y) a.dy = row_of(b->dy, es);
    if (with_gate) a.dgate = row_of(b->dgate, es);
  } else {
    a.x = row_of(b->x, ss);
    if (with_y) a.x_out = row_of(b->x_out, ss);
    if (c.norm_out) a.h = row_of(b->h, es);
  }
  // (of zeros a gain would make NaN where it is no number)
  a.y_gain = with_y ? b->y_gain : nullptr;
  a.gain = (backward ? a.dh.data : a.h.data) ? b->gain : nullptr;
  float* const dgain[2] = {backward ? b->dy_gain : nullptr, backward ? b->dgain : nullptr};
  const bool want = dgain[0] || dgain[1], drops = with_y && c.dropout > 0.0;
  const struct {
    JoinRow* r;
    const char* name;
    bool result;
    int size;
  } rows[] = {{&a.x, backward ? "x_out" : "x", false, ss}, {&a.y, "y", false, es},
              {&a.gate, "gate", false, es},                {&a.dxo, "dx_out", false, ss},
              {&a.dh, "dh", false, es},                    {&a.x_out, "x_out", true, ss},
              {&a.h, "h", true, es},                       {&a.dx, "dx", true, ss},
              {&a.dy, "dy", true, es},                     {&a.dgate, "dgate", true, es}};
  if (b->tokens > 0) {
    if (!a.x.data) return fail(ZERO_EINVAL, "%s is NULL", backward ? "x_out" : "x");
    if (with_gate && !a.gate.data) return fail(ZERO_EINVAL, "gate is NULL");
    if (!backward && c.norm_out && !a.h.data) return fail(ZERO_EINVAL, "h is NULL");
    if (!backward && !a.h.data && !a.x_out.data) return fail(ZERO_EINVAL, "no result is wanted");
    if (backward && !a.dxo.data && !a.dh.data) return fail(ZERO_EINVAL, "no gradient is given");
    for (const auto& r : rows) {
      if (!r.r->data) continue;
      if (reinterpret_cast<uintptr_t>(r.r->data) % r.size) return fail(ZERO_EINVAL, "%s is misaligned", r.name);
      if (r.result && b->tokens > 1 && std::abs(r.r->stride) < (int64_t)c.dim * r.size)
        return fail(ZERO_EINVAL, "rows of %s lie on one another", r.name);
    }
    for (const void* p : {(const void*)a.y_gain, (const void*)a.gain, (const void*)dgain[0], (const void*)dgain[1]})
      if (reinterpret_cast<uintptr_t>(p) % 4) return fail(ZERO_EINVAL, "a gain is misaligned");
    if (drops && reinterpret_cast<uintptr_t>(b->rng.step_dev) % 8)
      return fail(ZERO_EINVAL, "step_dev is misaligned");
  }
  if (!h->has_device) return fail(ZERO_ECUDA, "no CUDA device for this handle");
  int cur = -1;
  cudaError_t e = cudaGetDevice(&cur);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (cur != h->device)
    return fail(ZERO_ECUDA, "current device %d is not the handle's device %d", cur, h->device);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (b->tokens == 0) {
    for (float* g : dgain)
      if (g) {
        e = cudaMemsetAsync(g, 0, c.dim * sizeof(float), s);
        if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync");
      }
    return ZERO_OK;
  }

  a.mask = b->mask;
  a.tokens = b->tokens;
  a.drop = zo::drop_of(b->rng, drops ? c.dropout : 0.0);
  a.dim = c.dim;
  a.chunks = (c.dim + 7) / 8;
  a.gate_kind = c.gate;
  // (an eps below binary32's smallest number still makes zero of a row of zeros)
  a.eps = a.eps_y = c.eps > 0.0 ? std::max((float)c.eps, std::numeric_limits<float>::denorm_min()) : 0.0f;
  a.inv_dim = 1.0f / (float)c.dim;
  a.alpha = with_y ? (float)c.alpha : 1.0f;
  a.beta = (float)c.beta;
  // absent inputs are zeros; without dh the stream is not read, and its norm, which
  // then counts for nothing, stays finite
  const JoinRow none = {reinterpret_cast<char*>(h->zeros), 0, 0};
  if (!a.y.data) a.y = none;
  if (backward && !a.dxo.data) a.dxo = none;
  if (backward && !a.dh.data) {
    a.dh = a.x = none;
    a.eps = 1.0f;
  }
  a.part = want ? reinterpret_cast<float4*>(h->part) : nullptr;
  bool wide = c.dim % 8 == 0;
  for (const auto& r : rows) wide = wide && on16(r.r->data, r.r->stride, b->tokens);
  // Chunks a thread.  One where there are few, or few rows (a row is done sooner by
  // more threads); two otherwise forward, which leaves room for three CTAs an SM, and
  // backward unless the gate's registers or a binary32 stream's ring are too many for
  // it; four of long rows.
  const bool one = a.chunks <= 32 || (a.chunks <= 512 && (b->tokens <= 2 * h->sms || !wide));
  int cs = one ? 1 : a.chunks <= 1024 ? 2 : 4;
  if (cs == 2 && backward && a.chunks <= 512 && (with_gate || mixed)) cs = 1;
  a.warps = (a.chunks + 32 * cs - 1) / (32 * cs);
  a.teams = std::max(1, 8 / a.warps);
  a.teams = (int)std::min<int64_t>(a.teams, (b->tokens + h->sms - 1) / h->sms);
  const int threads = a.teams * a.warps * 32;
  // Shifted rows in CTAs of up to 320 threads (4097 to 5120 numbers forward) have a kernel
  // of fewer registers, two CTAs of which fit an SM: 4,000 rows of 4097 in bf16 45 us
  // against 63 with the other's one, of 5119 with a dropout 61 against 82.  From 4609
  // numbers without a dropout the rule below leaves one CTA in any case, and it loses: 70
  // against 66, at 5119 73 against 68.
  const zo::JoinPick pick = {backward, wide, with_y && c.norm_branch, with_gate ? 2 : a.drop.cut > 0 ? 1 : 0, cs,
                             threads > (wide ? 256 : 320)};
  const void* fn = c.dtype == ZERO_FP32   ? zo::join_float(pick)
                   : c.dtype == ZERO_FP16 ? (mixed ? zo::join_half_float(pick) : zo::join_half(pick))
                                          : (mixed ? zo::join_bf16_float(pick) : zo::join_bf16(pick));
  const int vt = es / 2, vs = ss / 2;
  a.vecs = cs * (backward ? 2 * vs + 2 * vt : vs + vt) + (with_gate ? cs * vt : 0);
  const int row = a.vecs * threads / 32 * (wide ? zo::kVecBytesOf<true> : zo::kVecBytesOf<false>);
  // CTAs an SM and rows of their rings.  Memory is quickest with some 16,384 numbers
  // of each tensor on their way to an SM: with fewer it is waited for, with more reads
  // and writes get into one another's way (16,384 rows of 4096 in bf16, two CTAs: two
  // rows each 81 us, three 92; with both norms 84, 91, three CTAs of two rows 92;
  // backward 131 and 143, and without the branch's norm, whose rows are done sooner,
  // one CTA of three rows 125, two of two 142).  A dropout's integer work wants more
  // CTAs (95 us with three, 104 with two).  The constants were found at 4096 and count
  // whole rows: from 4097 numbers on (4609 forward) the room is for three rows, which is
  // one CTA with three.  What that gives of the copy rate, forward and backward, with
  // both norms: 4096 93 and 94 %, 5120 85 and 84, 6144 93 and 94, 7168 96 and 92, 8192 94
  // and 89; without the branch's norm 97 and 99, at 5120 94 and 92, at 7168 87 and 85.
  const int numbers = backward ? (pick.post || pick.has ? 16384 : 12288) : pick.has ? 24576 : 18432;
  int slots = std::max(1, numbers / (a.teams * c.dim));
  int ctas = std::max(1, std::min(h->resident(fn, threads, 2 * row), slots / 2));
  a.ring = ctas == 1 ? 3 : std::max(2, std::min(3, slots / ctas));
  a.ring = std::max(1, std::min(a.ring, kMaxSmem / row));
  size_t smem = (size_t)a.ring * row;
  if (want && a.teams > 1) smem = std::max(smem, (size_t)a.chunks * 16 * sizeof(float));
  ctas = std::min(ctas, h->resident(fn, threads, (int)smem));
  int64_t grid = std::min((b->tokens + a.teams - 1) / a.teams, (int64_t)ctas * h->sms);
  if (want) grid = std::min(grid, h->max_grid);
  for (const auto& r : rows) r.r->step = r.r->stride * grid * a.teams;
  void* params[] = {&a};
  e = cudaLaunchKernel(fn, dim3((unsigned)grid), dim3((unsigned)threads), params, smem, s);
  if (e != cudaSuccess) return cuda_fail(e, "cudaLaunchKernel");
  ++h->launches;
  if (want) {
    FoldArgs f = {h->part, {dgain[0], dgain[1]}, (int)grid, c.dim, a.chunks};
    void* fp[] = {&f};
    cudaLaunchAttribute early;
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3((unsigned)((16 * a.chunks + 63) / 64));
    lc.blockDim = dim3(1024);
    lc.stream = s;
    lc.attrs = &early;
    lc.numAttrs = 1;
    e = cudaLaunchKernelExC(&lc, (const void*)join_fold_kernel, fp);
    if (e != cudaSuccess) return cuda_fail(e, "cudaLaunchKernelExC");
    ++h->launches;
  }
  return ZERO_OK;
}

}  // namespace

extern "C" {

zero_status zero_block_create(const zero_block_config* cfg, zero_block_t* out) {
  if (!out) return fail(ZERO_EINVAL, "out is NULL");
  *out = nullptr;
  if (!cfg) return fail(ZERO_EINVAL, "cfg is NULL");
  if (!known(cfg->dtype)) return fail(ZERO_EINVAL, "dtype must be ZERO_FP16, ZERO_BF16 or ZERO_FP32");
  if (cfg->stream_dtype != cfg->dtype && cfg->stream_dtype != ZERO_FP32)
    return fail(ZERO_EINVAL, "stream_dtype must be dtype or ZERO_FP32");
  const int most = cfg->dtype == ZERO_FP32                                                    ? kMaxDim32
                   : cfg->gate != ZERO_GATE_NONE && cfg->stream_dtype != cfg->dtype ? kMaxDimGated
                                                                                    : kMaxDim;
  if (cfg->dim < 1 || cfg->dim > most) return fail(ZERO_EINVAL, "dim must be in 1..%d", most);
  if ((cfg->norm_branch | 1) != 1 || (cfg->norm_out | 1) != 1)
    return fail(ZERO_EINVAL, "norm_branch and norm_out must be 0 or 1");
  if (cfg->gate < ZERO_GATE_NONE || cfg->gate > ZERO_GATE_SIGMOID)
    return fail(ZERO_EINVAL, "gate must be a ZERO_GATE_*");
  if (!(cfg->eps >= 0.0) || !std::isfinite(cfg->eps)) return fail(ZERO_EINVAL, "eps must be >= 0");
  constexpr double kLargest = std::numeric_limits<float>::max();
  if (!(std::fabs(cfg->alpha) <= kLargest && std::fabs(cfg->beta) <= kLargest))
    return fail(ZERO_EINVAL, "alpha and beta must be finite in binary32");
  if (!(cfg->dropout >= 0.0 && cfg->dropout <= 1.0)) return fail(ZERO_EINVAL, "dropout must be in 0..1");
  zero_block_handle* h = new (std::nothrow) zero_block_handle;
  if (!h) return fail(ZERO_ENOMEM, "handle allocation failed");
  h->cfg = *cfg;
  int count = 0;
  if (cudaGetDeviceCount(&count) != cudaSuccess || count < 1) {
    cudaGetLastError();
    *out = h;
    return ZERO_OK;
  }
  cudaError_t e = cudaGetDevice(&h->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&h->sms, cudaDevAttrMultiProcessorCount, h->device);
  // Partial gradients of every CTA of the largest grid (the backward pass has two rows
  // a CTA or more on their way to an SM, of 16,384 numbers together).
  h->max_grid = (int64_t)h->sms * std::max(1, std::min(kMaxPerSm, 8192 / cfg->dim));
  const size_t numbers = (size_t)h->max_grid * 2 * ((cfg->dim + 7) / 8 * 8), dim = (cfg->dim + 7) / 8 * 8;
  if (e == cudaSuccess)
    e = cudaMalloc(reinterpret_cast<void**>(&h->part), (numbers + dim) * sizeof(float));
  if (e == cudaSuccess) {
    h->zeros = h->part + numbers;
    e = cudaMemset(h->zeros, 0, dim * sizeof(float));
  }
  // (a call's stream need not wait for the default stream)
  if (e == cudaSuccess) e = cudaStreamSynchronize(cudaStreamLegacy);
  if (e != cudaSuccess) {
    cudaFree(h->part);
    cudaGetLastError();
    delete h;
    return e == cudaErrorMemoryAllocation ? fail(ZERO_ENOMEM, "workspace allocation failed")
                                          : cuda_fail(e, "zero_block_create");
  }
  h->has_device = true;
  *out = h;
  return ZERO_OK;
}

zero_status zero_block_destroy(zero_block_t h) {
  if (!h) return ZERO_OK;
  if (h->has_device) {
    int prev = -1;
    cudaGetDevice(&prev);
    cudaSetDevice(h->device);
    cudaDeviceSynchronize();
    cudaFree(h->part);
    if (prev >= 0) cudaSetDevice(prev);
  }
  delete h;
  return ZERO_OK;
}

zero_status zero_block_join(zero_block_t h, const zero_block_buffers* b, void* stream) {
  return run(h, b, stream, false);
}

zero_status zero_block_join_backward(zero_block_t h, const zero_block_buffers* b, void* stream) {
  return run(h, b, stream, true);
}

zero_status zero_block_launch_count(zero_block_t h, int64_t* launches) {
  if (!h || !launches) return fail(ZERO_EINVAL, "NULL argument");
  *launches = h->launches;
  return ZERO_OK;
}

zero_status zero_dropout(const zero_drop_buffers* b, void* stream) {
  if (!b) return fail(ZERO_EINVAL, "buffers are NULL");
  if (b->rows < 0 || b->cols < 0) return fail(ZERO_EINVAL, "rows and cols must be >= 0");
  if (!known(b->dtype)) return fail(ZERO_EINVAL, "dtype must be ZERO_FP16, ZERO_BF16 or ZERO_FP32");
  if (!(b->p >= 0.0 && b->p <= 1.0)) return fail(ZERO_EINVAL, "p must be in 0..1");
  const int es = elem_size(b->dtype);
  const bool any = b->rows > 0 && b->cols > 0;
  if (any) {
    if (!b->in || !b->out) return fail(ZERO_EINVAL, "in or out is NULL");
    if (reinterpret_cast<uintptr_t>(b->in) % es || reinterpret_cast<uintptr_t>(b->out) % es)
      return fail(ZERO_EINVAL, "in or out is misaligned");
    if (b->rows > 1 && std::abs(b->out_stride) < b->cols)
      return fail(ZERO_EINVAL, "rows of the result lie on one another");
    if (reinterpret_cast<uintptr_t>(b->rng.step_dev) % 8) return fail(ZERO_EINVAL, "step_dev is misaligned");
  }
  int device = -1, sms = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device);
  if (e != cudaSuccess) {
    return cuda_fail(e, "no CUDA device");
  }
  if (!any) return ZERO_OK;
  DropArgs a = {};
  a.in = static_cast<const char*>(b->in);
  a.out = static_cast<char*>(b->out);
  a.rows = b->rows;
  a.cols = b->cols;
  a.in_stride = b->in_stride * es;
  a.out_stride = b->out_stride * es;
  a.blocks = (b->cols + 7) / 8;
  a.drop = zo::drop_of(b->rng, b->p);
  // rows that follow one another and are whole blocks: one long row
  if (b->cols % 8 == 0 && b->in_stride == b->cols && b->out_stride == b->cols) {
    a.blocks *= a.rows;
    a.cols *= a.rows;
    a.rows = 1;
  }
  const bool wide = on16(a.in, a.in_stride, a.rows) && on16(a.out, a.out_stride, a.rows);
  const int64_t work = wide ? (a.rows * a.blocks + 255) / 256 : (a.rows * ((a.cols + 255) / 256) + 7) / 8;
  int64_t grid = std::min<int64_t>(work, (int64_t)sms * 16);
  const int mode = !wide ? kTiles : a.rows == 1 && a.cols % 8 == 0 ? kFlat : kWide;
  const void* fn = b->dtype == ZERO_FP16   ? drop_of_type<__half>(mode)
                   : b->dtype == ZERO_BF16 ? drop_of_type<__nv_bfloat16>(mode)
                                           : drop_of_type<float>(mode);
  void* params[] = {&a};
  e = cudaLaunchKernel(fn, dim3((unsigned)grid), dim3(256), params, 0, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "cudaLaunchKernel");
  return ZERO_OK;
}

}  // extern "C"
