// qk.cu -- each head's query and key normalised and rotated in one pass
// (zero_qk.h), forward and backward.
//
// What bounds it: memory.  A row (one token's one head) is read once, its mean
// square reduced in registers by a few lanes, and written once; the backward
// pass reads the row and its output's gradient and writes the row's gradient.
// Nothing else of size is moved: angles and gains are a few hundred bytes a
// token and stay in L1.  Measured, 16,384 tokens of 40 heads of 128 in bf16:
// forward 57 us a call (55 on the device: 5.3 TB/s of DRAM traffic, and 6.3 of
// the bytes that have to move, as L2 keeps some of the result; 60 % of the issue
// slots), backward 100 us (94 and, for the sums of the gains' gradients, 5;
// 5.1 TB/s; 50 % of the issue slots).  One token takes 4 us on the device, less
// than the host's call of 8.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdlib>
#include <limits>
#include <mutex>
#include <new>

#include "host_util.h"
#include "qk_kernels.cuh"
#include "zero_qk.h"

namespace {

using zo::fail;
using zo::kQkThreads;
using zo::QkArgs;
using zo::QkAxesArgs;
using zo::ring_bytes;
using zo::Rows;

constexpr int kMaxDim = 512;
constexpr int kMaxPerSm = 6;      // CTAs an SM: what the workspace has room for
constexpr int kMaxSmem = 200 * 1024;

struct FoldArgs {
  const float* part;
  float* out[2];
  int32_t grid, head_blocks, part_rows, per, dim, q_heads, heads, gain_per_head;
};

// Sums the CTAs' partial gain gradients in index order: 32 columns a CTA, kParts
// threads a column, each over every kParts-th partial: 32 for handles with axes, whose
// sums are done sooner so (3,001 tokens of 16 heads of 64: 15.2 us with eight, 13.6
// with 32); eight with one position, whose gradients have been summed in that order
// before and keep their bits.
template <int kParts>
__global__ void __launch_bounds__(32 * kParts) qk_fold_kernel(const __grid_constant__ FoldArgs a) {
  __shared__ float s[kParts][33];
  cudaGridDependencySynchronize();   // launched while the partials are still written
  const int col = blockIdx.x * 32 + threadIdx.x % 32, part = threadIdx.x / 32;
  const int rows = a.gain_per_head ? a.heads : 2;
  const int row = col / a.dim, d = col % a.dim;
  float sum = 0.0f;
  if (row < rows) {
    const int step = a.gain_per_head ? a.head_blocks : 1;
    const int first = a.gain_per_head ? row / a.per : 0;
    const int local = a.gain_per_head ? row % a.per : row;
    const int64_t one = (int64_t)a.part_rows * a.dim;
    const float* at = a.part + (int64_t)local * a.dim + d;
    int c = first + part * step;
    for (; c + 7 * kParts * step < a.grid; c += 8 * kParts * step) {
      float v[8];                // eight loads on their way at once
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = at[(c + kParts * k * step) * one];
#pragma unroll
      for (int k = 0; k < 8; ++k) sum = __fadd_rn(sum, v[k]);
    }
#pragma unroll 4
    for (; c < a.grid; c += kParts * step) sum = __fadd_rn(sum, at[c * one]);
  }
  s[part][threadIdx.x % 32] = sum;
  __syncthreads();
  if (part == 0 && row < rows) {
#pragma unroll
    for (int k = 1; k < kParts; ++k) sum = __fadd_rn(sum, s[k][threadIdx.x]);
    const int which = a.gain_per_head ? (row >= a.q_heads) : row;
    const int at = a.gain_per_head ? row - (which ? a.q_heads : 0) : 0;
    if (a.out[which]) a.out[which][(int64_t)at * a.dim + d] = sum;
  }
}

bool fits(const void* p, int64_t s0, int64_t s1, int bytes, int esize) {
  return reinterpret_cast<uintptr_t>(p) % bytes == 0 && s0 * esize % bytes == 0 &&
         s1 * esize % bytes == 0;
}

}  // namespace

struct zero_qk_handle {
  zero_qk_config cfg;
  zero_qk_axes axes = {};     // axes 0: one position a token
  bool has_device = false;
  int device = -1;
  int sms = 0;
  float* part = nullptr;
  int64_t launches = 0;
  std::mutex mu;
  struct {
    const void* fn;
    int threads, smem, ctas;
  } occ[32] = {};     // launch shapes seen, oldest overwritten
  int seen = 0;

  // CTAs of a kernel that an SM holds at once, at most kMaxPerSm.
  int resident(const void* fn, int threads, int smem) {
    std::lock_guard<std::mutex> lock(mu);
    for (const auto& o : occ)
      if (o.fn == fn && o.threads == threads && o.smem == smem) return o.ctas;
    int n = 0;
    if (smem > 48 * 1024) cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, fn, threads, smem) != cudaSuccess) n = 1;
    n = std::max(1, std::min(n, kMaxPerSm));
    occ[seen++ % 32] = {fn, threads, smem, n};
    return n;
  }
};

namespace {

zero_status cuda_fail(cudaError_t e, const char* what) {
  return fail(ZERO_ECUDA, "%s: %s", what, cudaGetErrorString(e));
}

int elem_size(int32_t dtype) { return dtype == ZERO_FP32 ? 4 : 2; }

zero_status run(zero_qk_t h, const zero_qk_buffers* b, void* stream, bool backward) {
  if (!h) return fail(ZERO_EINVAL, "handle is NULL");
  if (!b) return fail(ZERO_EINVAL, "buffers are NULL");
  const zero_qk_config& c = h->cfg;
  const zero_qk_axes& ax = h->axes;
  const bool turn_only = ax.axes > 0 && !ax.normalise;
  if (b->tokens < 0 || b->n_pos < 0) return fail(ZERO_EINVAL, "tokens and n_pos must be >= 0");
  const zero_qk_tensor* out[2] = {backward ? &b->dq : &b->q_out, backward ? &b->dk : &b->k_out};
  const zero_qk_tensor* in[2] = {&b->q, &b->k};
  const zero_qk_tensor* go[2] = {&b->q_out, &b->k_out};
  if (turn_only && (b->q_gain || b->k_gain || (backward && (b->dq_gain || b->dk_gain))))
    return fail(ZERO_EINVAL, "without the norm there are no gains");
  if (ax.axes > 0 && b->n_pos > INT32_MAX) return fail(ZERO_EINVAL, "n_pos must be below 2^31 with axes");
  // the gradient of a rotation is the rotation back, which needs no rows
  const bool inverse = turn_only && backward;
  if (inverse) {
    in[0] = go[0];
    in[1] = go[1];
    backward = false;
  }
  if (b->tokens > 0) {
    for (int w = 0; w < (c.k_heads > 0 ? 2 : 1); ++w)
      if (!in[w]->data || !out[w]->data || (backward && !go[w]->data))
        return fail(ZERO_EINVAL, "a %s tensor is NULL", w ? "key" : "query");
    for (int w = 0; w < (c.k_heads > 0 ? 2 : 1); ++w)
      if ((b->tokens > 1 && std::abs(out[w]->token_stride) < c.head_dim) ||
          ((w ? c.k_heads : c.q_heads) > 1 && std::abs(out[w]->head_stride) < c.head_dim))
        return fail(ZERO_EINVAL, "rows of a %s result lie on one another", w ? "key" : "query");
    if (!b->positions) return fail(ZERO_EINVAL, "positions are NULL");
    if (ax.axes > 0 && reinterpret_cast<uintptr_t>(b->positions) % (b->positions64 ? 8 : 4))
      return fail(ZERO_EINVAL, "positions are misaligned");
    if (c.rotary_dim > 0 && b->n_pos > 0 && (!b->cos || !b->sin))
      return fail(ZERO_EINVAL, "cos and sin must be non-NULL");
  }
  if (!h->has_device) return fail(ZERO_ECUDA, "no CUDA device for this handle");
  int cur = -1;
  cudaError_t e = cudaGetDevice(&cur);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (cur != h->device)
    return fail(ZERO_ECUDA, "current device %d is not the handle's device %d", cur, h->device);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  float* dgain[2] = {b->dq_gain, c.k_heads > 0 ? b->dk_gain : nullptr};
  if (b->tokens == 0) {
    for (int w = 0; backward && w < 2; ++w)
      if (dgain[w]) {
        const size_t rows = c.gain_per_head ? (size_t)(w ? c.k_heads : c.q_heads) : 1;
        e = cudaMemsetAsync(dgain[w], 0, rows * c.head_dim * sizeof(float), s);
        if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync");
      }
    return ZERO_OK;
  }

  QkAxesArgs a = {};
  a.axes = ax.axes;
  a.norm = !turn_only;
  a.inverse = inverse;
  for (int j = 0; ax.axes > 0 && j < c.rotary_dim / 2; ++j) a.axis[j / 16] |= (uint32_t)ax.axis[j] << j % 16 * 2;
  a.cos = b->cos;
  a.sin = b->sin;
  a.pos = b->positions;
  a.pos64 = b->positions64;
  a.tokens = b->tokens;
  a.n_pos = b->n_pos;
  a.dim = c.head_dim;
  a.rot = c.rotary_dim;
  a.gain_per_head = c.gain_per_head;
  a.heads = c.q_heads + c.k_heads;
  // (an eps below binary32's smallest number still makes zero of a row of zeros)
  a.eps = c.eps > 0.0 ? std::max((float)c.eps, std::numeric_limits<float>::denorm_min()) : 0.0f;
  a.inv_dim = 1.0f / (float)c.head_dim;
  const int es = elem_size(c.dtype);
  // The widest vector that the head's halves, every address and every stride
  // are multiples of: 16 bytes a load where all are, single numbers at worst.
  int v = es == 2 ? 8 : 4;
  for (; v > 1; v /= 2) {
    bool ok = c.head_dim % (2 * v) == 0 && c.rotary_dim % (2 * v) == 0;
    const int fb = std::min(v, 4) * 4;
    ok = ok && (c.rotary_dim == 0 || (fits(b->cos, 0, 0, fb, 4) && fits(b->sin, 0, 0, fb, 4)));
    ok = ok && fits(b->q_gain, 0, 0, fb, 4) && (c.k_heads == 0 || fits(b->k_gain, 0, 0, fb, 4));
    for (int w = 0; ok && w < (c.k_heads > 0 ? 2 : 1); ++w) {
      ok = fits(in[w]->data, in[w]->token_stride, in[w]->head_stride, v * es, es) &&
           fits(out[w]->data, out[w]->token_stride, out[w]->head_stride, v * es, es);
      if (backward)
        ok = ok && fits(go[w]->data, go[w]->token_stride, go[w]->head_stride, v * es, es);
    }
    if (ok) break;
  }
  a.chunks = c.head_dim / (2 * v);
  const int chunks_lane = v == 8 ? 1 : v == 4 ? 2 : v == 2 ? 4 : 8;
  a.lanes = 1;
  while (a.lanes * chunks_lane < a.chunks) a.lanes *= 2;
  // (4,096 tokens of 32 heads of 80, fp16, only rotated: 15.8 us with 8 lanes a head,
  // 11.5 with five)
  if (turn_only) a.lanes = (a.chunks + chunks_lane - 1) / chunks_lane;
  const int in_warp = 32 / a.lanes;
  for (int w = 0; w < 2; ++w) {
    Rows& r = a.r[w];
    r.heads = w ? c.k_heads : c.q_heads;
    if (r.heads == 0) continue;
    r.in = static_cast<const char*>(in[w]->data);
    r.in_t = in[w]->token_stride;
    r.in_h = in[w]->head_stride;
    r.out = static_cast<char*>(out[w]->data);
    r.out_t = out[w]->token_stride;
    r.out_h = out[w]->head_stride;
    if (backward) {
      r.gout = static_cast<const char*>(go[w]->data);
      r.go_t = go[w]->token_stride;
      r.go_h = go[w]->head_stride;
    }
    r.gain = w ? b->k_gain : b->q_gain;
  }
  const int groups = kQkThreads / 32 * in_warp;
  const int es_vec = v * es;
  const bool want = backward && (dgain[0] || dgain[1]);
  const bool sum = backward && !(want && c.gain_per_head);
  // Heads a group: fewer reads of the angles and fewer bookkeeping
  // instructions a row, as long as both head counts divide and the tokens
  // still fill the device.  The most: what the ring and the registers leave two
  // or three CTAs an SM for (16,384 tokens, 40 heads of 128: forward 58 us with
  // four, 64 with two, 81 with one; backward 100 with two, 122 with one; with sums
  // a head, which keep one head's gain in registers, 8,192 tokens of 40 heads of
  // 128 67 with one, 75 with two, 16,384 of 20 heads of 64 39 and 43).
  int r = 1;
  const int most_r = es_vec < 16 ? 1 : v == 8 ? (!backward ? 4 : sum ? 2 : 1) : (backward ? 1 : 2);
  while (2 * r <= most_r && c.q_heads % (2 * r) == 0 && c.k_heads % (2 * r) == 0 &&
         b->tokens * a.heads >= (int64_t)2 * r * groups * 2 * h->sms)
    r *= 2;
  // the heads' groups spread evenly over as few CTAs as hold a token's
  a.head_blocks = (a.heads / r + groups - 1) / groups;
  a.per = (a.heads / r + a.head_blocks - 1) / a.head_blocks;
  a.reps = groups / a.per;
  a.part_rows = sum ? 2 : a.per * r;
  a.part = want ? h->part : nullptr;
  // no more threads than groups that have a head
  const int threads = (a.per * a.reps + in_warp - 1) / in_warp * 32;
  const auto pick = ax.axes > 0 ? zo::qk_kernel_axes : zo::qk_kernel_one;
  const void* fn = pick(c.dtype, c.interleaved, backward, sum, v, r);
  size_t smem = es_vec == 16 ? (size_t)ring_bytes(threads, chunks_lane, r, backward) : 0;
  if (ax.axes > 0) smem += (size_t)(threads / 32 * in_warp) * zo::kPosSlots * zo::kPosBytes;
  if (want) smem = std::max(smem, (size_t)a.per * a.reps * c.head_dim * sizeof(float));
  const int64_t slots = (b->tokens + a.reps - 1) / a.reps;
  int64_t grid = slots * a.head_blocks;
  const int64_t resident = (int64_t)h->resident(fn, threads, (int)smem) * h->sms;
  const int64_t most = std::max<int64_t>(1, resident / a.head_blocks) * a.head_blocks;
  if (grid > most) grid = most;
  void* params[] = {&a};
  e = cudaLaunchKernel(fn, dim3((unsigned)grid), dim3((unsigned)threads), params, smem, s);
  if (e != cudaSuccess) return cuda_fail(e, "cudaLaunchKernel");
  ++h->launches;
  if (want) {
    FoldArgs f = {};
    f.part = h->part;
    f.out[0] = dgain[0];
    f.out[1] = dgain[1];
    f.grid = (int)grid;
    f.head_blocks = a.head_blocks;
    f.part_rows = a.part_rows;
    f.per = a.per * r;
    f.dim = c.head_dim;
    f.q_heads = c.q_heads;
    f.heads = a.heads;
    f.gain_per_head = c.gain_per_head;
    const int64_t cols = (int64_t)(c.gain_per_head ? a.heads : 2) * c.head_dim;
    void* fp[] = {&f};
    cudaLaunchAttribute early;
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3((unsigned)((cols + 31) / 32));
    lc.blockDim = dim3(ax.axes > 0 ? 1024 : 256);
    lc.stream = s;
    lc.attrs = &early;
    lc.numAttrs = 1;
    e = cudaLaunchKernelExC(&lc, ax.axes > 0 ? (const void*)qk_fold_kernel<32> : (const void*)qk_fold_kernel<8>, fp);
    if (e != cudaSuccess) return cuda_fail(e, "cudaLaunchKernelExC");
    ++h->launches;
  }
  return ZERO_OK;
}

}  // namespace

extern "C" {

zero_status zero_qk_create(const zero_qk_config* cfg, zero_qk_t* out) {
  if (!out) return fail(ZERO_EINVAL, "out is NULL");
  *out = nullptr;
  if (!cfg) return fail(ZERO_EINVAL, "cfg is NULL");
  if (cfg->q_heads < 1 || cfg->k_heads < 0 || (int64_t)cfg->q_heads + cfg->k_heads > 4096)
    return fail(ZERO_EINVAL, "q_heads must be >= 1, k_heads >= 0 and both at most 4096 together");
  if (cfg->head_dim < 2 || cfg->head_dim > kMaxDim || cfg->head_dim % 2)
    return fail(ZERO_EINVAL, "head_dim must be even and in 2..%d", kMaxDim);
  if (cfg->rotary_dim < 0 || cfg->rotary_dim > cfg->head_dim || cfg->rotary_dim % 2)
    return fail(ZERO_EINVAL, "rotary_dim must be even and in 0..head_dim");
  if (cfg->dtype != ZERO_FP16 && cfg->dtype != ZERO_BF16 && cfg->dtype != ZERO_FP32)
    return fail(ZERO_EINVAL, "dtype must be ZERO_FP16, ZERO_BF16 or ZERO_FP32");
  if ((cfg->interleaved | 1) != 1 || (cfg->gain_per_head | 1) != 1)
    return fail(ZERO_EINVAL, "interleaved and gain_per_head must be 0 or 1");
  if (!(cfg->eps >= 0.0)) return fail(ZERO_EINVAL, "eps must be >= 0");
  zero_qk_handle* h = new (std::nothrow) zero_qk_handle;
  if (!h) return fail(ZERO_ENOMEM, "handle allocation failed");
  h->cfg = *cfg;
  int count = 0;
  if (cudaGetDeviceCount(&count) != cudaSuccess || count < 1) {
    cudaGetLastError();
    *out = h;
    return ZERO_OK;
  }
  cudaError_t e = cudaGetDevice(&h->device);
  if (e == cudaSuccess)
    e = cudaDeviceGetAttribute(&h->sms, cudaDevAttrMultiProcessorCount, h->device);
  // Partial gain gradients of every CTA of the largest grid.  A CTA's rows are
  // two, or its heads: at most 256 groups (a group of one lane owns heads of
  // at most 16 numbers), two heads each.
  const int64_t heads = (int64_t)cfg->q_heads + cfg->k_heads;
  const int64_t rows = cfg->gain_per_head ? std::min<int64_t>(2 * kQkThreads, heads) : 2;
  const int64_t blocks = std::max<int64_t>((int64_t)kMaxPerSm * h->sms, heads);
  if (e == cudaSuccess)
    e = cudaMalloc(reinterpret_cast<void**>(&h->part),
                   (size_t)(blocks * rows * cfg->head_dim) * sizeof(float));
  if (e != cudaSuccess) {
    delete h;
    return e == cudaErrorMemoryAllocation ? fail(ZERO_ENOMEM, "workspace allocation failed")
                                          : cuda_fail(e, "zero_qk_create");
  }
  h->has_device = true;
  *out = h;
  return ZERO_OK;
}

zero_status zero_qk_create_axes(const zero_qk_config* cfg, const zero_qk_axes* axes, zero_qk_t* out) {
  if (!out) return fail(ZERO_EINVAL, "out is NULL");
  *out = nullptr;
  if (!axes) return fail(ZERO_EINVAL, "axes is NULL");
  if (axes->axes < 1 || axes->axes > zo::kMaxAxes)
    return fail(ZERO_EINVAL, "axes must be in 1..%d", zo::kMaxAxes);
  if ((axes->normalise | 1) != 1) return fail(ZERO_EINVAL, "normalise must be 0 or 1");
  if (cfg && cfg->rotary_dim <= kMaxDim)
    for (int j = 0; j < cfg->rotary_dim / 2; ++j)
      if (axes->axis[j] >= axes->axes) return fail(ZERO_EINVAL, "axis[%d] is none of the axes", j);
  const zero_status s = zero_qk_create(cfg, out);
  if (s == ZERO_OK) (*out)->axes = *axes;
  return s;
}

zero_status zero_qk_destroy(zero_qk_t h) {
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

zero_status zero_qk_norm_rope(zero_qk_t h, const zero_qk_buffers* b, void* stream) {
  return run(h, b, stream, false);
}

zero_status zero_qk_norm_rope_backward(zero_qk_t h, const zero_qk_buffers* b, void* stream) {
  return run(h, b, stream, true);
}

zero_status zero_qk_launch_count(zero_qk_t h, int64_t* launches) {
  if (!h || !launches) return fail(ZERO_EINVAL, "NULL argument");
  *launches = h->launches;
  return ZERO_OK;
}

}  // extern "C"
