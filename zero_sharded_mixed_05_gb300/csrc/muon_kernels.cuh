// muon_kernels.cuh -- device side of the orthogonalised update (zero_muon.h).
//
// A call is three stages:
//   muon_stats_kernel   reads the input (for the step: gradient and momentum,
//                       and writes the new momentum) and finds |U|_F
//   muon_start_kernel   writes X = U / (|U|_F + eps), held as the sum of two
//                       binary16 numbers, into the workspace
//   muon_products_kernel steps times  A = X X^T,  B = b A + c A A,  X <- a X + B X,
//                       the last with the result's epilogue (muon_products.cuh)
// The workspace holds every matrix in the orientation it came in: for a wide
// matrix the products are X X^T and B X, for a tall one X^T X and X B.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "zero_muon.h"

namespace zm {

constexpr int kThreads = 256;
constexpr int kMaxEntries = ZERO_MUON_MAX_SHAPES;
constexpr int kVec = 8;                        // numbers of a thread's vector in the first two stages

// A and B are held times 4096 and X times 64, so that a product of X by itself
// has A's scale (zero_muon.h).
constexpr float kScale = 4096.0f, kScaleX = 64.0f;
// The second part of X is held times 2^11 more, so that it is a normal number
// wherever the first is.
constexpr float kLoScale = 2048.0f;

struct Entry {
  int32_t rows, cols, batch, k, l, tall;
  int64_t ldx, ldk;          // columns of x and lo, and of a and b, to a multiple of 32
  __half* x[2];              // [batch] blocks of X's first part, read and written in turn
  __half* lo;                // and of its second
  __half* a;                 // [batch] blocks of A and of b A + c A A
  __half* b;
  float* diag;               // [batch][ldk]: A's diagonal
  int32_t unit0;             // first matrix of the entry among all
  int32_t chunk0, chunks;    // first CTA, and CTAs a matrix, of the first two stages
  int32_t across;            // blocks of 32 columns
  int32_t splits, cut0, cuts; // parts of the depth of X X^T; first counter, counters a matrix
  int32_t slot0;             // first part's place among all
  int32_t item;              // the caller's index
  float s;                   // scale_rule's factor
};

// Every matrix of the workspace is in pieces: eight columns of a row are 16
// bytes, the pieces of 128 rows lie side by side, then the next eight columns'
// of the same rows, then the next 128 rows.  One layout serves all: an
// epilogue warp whose threads hold a row each reads and writes whole lines (by
// rows of a row-major array it would touch a line a thread); eight rows of a
// piece are the tensor core's 8 x 16-byte core matrix, for the depth along the
// rows as well as down them; and TMA brings 2 KB a run.  What pads a matrix to
// 128 rows and 32 columns is zero.
__host__ __device__ inline int64_t block_at(int row, int col, int64_t ld) {
  return (row / 128 * (ld / 8) + col / 8) * 1024 + row % 128 * 8;
}
__host__ __device__ inline int64_t block_size(int64_t rows, int64_t ld) { return (rows + 127) / 128 * 128 * ld; }

// What a call was given for one entry.
struct Io {
  const void* in;            // matrix, or gradient
  float* mom;
  float* master;
  void* out;                 // result, or 16-bit parameters
  int64_t in_row, in_batch, out_row, out_batch;
};

struct Workspace {
  int32_t fault;             // a wait has run out in the call that is running, or in the last
  int32_t skipped;
  // On the chip `fault` is a launch's own: zero when it starts, as the last of
  // its CTAs to end takes it from there.
  int32_t last;              // what the last call ended with
  int32_t faults;            // faulted calls; through the workspace, before the last
  unsigned long long ended;  // CTAs of the launch that have ended; times 2^32, without a result
};

struct Call {
  const Entry* entries;
  int32_t n, blocks;         // entries; blocks of 32 x 32 a warp in the first two stages
  int32_t step;              // step: 1 zero_muon_step, 0 zero_muon_orthogonalize
  Workspace* ws;
  double* part;              // sums of squares, one a CTA of the first stage
  unsigned* ticket;          // one a matrix, zero between calls
  float* inv;                // 1 / (|U|_F + eps), one a matrix
  const zero_opt_step_info* decision;
  double eps;
  float grad_scale, mu;
  int32_t nesterov, in_type, out_type;
  float decay, lr;           // 1 - lr * weight_decay; lr
  uint32_t* done;            // finished tiles of each matrix
  uint32_t* cut;             // parts that have arrived, of each tile whose depth is cut
  Io* io;                    // by the caller's index; stage 1 fills it in
};

// Stage 1's arguments: the caller's addresses travel with the launch (a large
// argument costs microseconds, so a handle of few entries has a small one).
template <int N> struct Start {
  Call c;
  Io io[N];
};

template <typename T> __device__ __forceinline__ float num(T x);
template <> __device__ __forceinline__ float num(__half x) { return __half2float(x); }
template <> __device__ __forceinline__ float num(__nv_bfloat16 x) { return __bfloat162float(x); }
template <> __device__ __forceinline__ float num(float x) { return x; }
template <typename T> __device__ __forceinline__ T as(float x);
template <> __device__ __forceinline__ __half as(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 as(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ float as(float x) { return x; }

__device__ __forceinline__ bool skipped(const Call& c) {
  return c.decision && c.decision->skipped;
}

__device__ __forceinline__ float grad_factor(const Call& c) {
  return c.decision ? __fmul_rn(c.grad_scale, c.decision->coef) : c.grad_scale;
}

// What a CTA of the first two stages works on, call.blocks times 8192 numbers:
// stage 1 in the order of the rows (blocks of rows 64 bytes wide read at half
// the rate), stage 2 in blocks of 32 x 32 a warp, four threads a row, so that
// X's pieces are written as whole sectors.  A thread's four vectors are on
// their way at once.
struct Part {
  int entry, b, chunk;       // matrix b of the entry, CTA `chunk` of the matrix
};
__device__ __forceinline__ Part part_of(const Call& c, int cta) {
  __shared__ int found;
  for (int i = threadIdx.x; i < c.n; i += kThreads) {
    const Entry& e = c.entries[i];
    const int at = cta - e.chunk0;
    if (at >= 0 && at < e.chunks * e.batch) found = i;
  }
  __syncthreads();
  const Entry& e = c.entries[found];
  const int at = cta - e.chunk0;
  return {found, at / e.chunks, at % e.chunks};
}

// A thread's four vectors of eight columns: their rows, first columns, and how
// many of the eight are in the matrix (0: the vector is padding).
struct Place {
  int row[4], col[4], n[4];
};
// In a block of 32 x 32 a warp: rows eight apart.  False: past the last block.
__device__ __forceinline__ bool place_block(const Call& c, const Entry& e, int chunk, int i, Place* p) {
  const uint32_t blk = (uint32_t)(chunk * c.blocks + i) * (kThreads / 32) + threadIdx.x / 32;
  const uint32_t down = blk / (uint32_t)e.across, right = blk - down * e.across;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    p->row[q] = (int)down * 32 + 8 * q + threadIdx.x % 32 / 4;
    p->col[q] = (int)right * 32 + threadIdx.x % 4 * kVec;
    p->n[q] = p->row[q] < e.rows ? min(kVec, max(e.cols - p->col[q], 0)) : 0;
  }
  return (int)down * 32 < e.rows;
}
// In the order of the rows, kThreads vectors apart.
__device__ __forceinline__ bool place_flat(const Call& c, const Entry& e, int chunk, int i, Place* p) {
  const uint32_t vpr = (uint32_t)(e.cols + kVec - 1) / kVec;      // vectors a row
  const uint32_t first = (uint32_t)(chunk * c.blocks + i) * (4 * kThreads);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint32_t v = first + q * kThreads + threadIdx.x, row = v / vpr;
    p->row[q] = (int)min(row, (uint32_t)e.rows);
    p->col[q] = (int)(v - row * vpr) * kVec;
    p->n[q] = p->row[q] < e.rows ? min(kVec, e.cols - p->col[q]) : 0;
  }
  return first < vpr * (uint32_t)e.rows;
}

// The numbers there of an array with its rows `ld` apart, p at the matrix's
// first; zero where there are none.  kWhole: every vector is whole and aligned,
// or padding.
template <bool kWhole, typename T>
__device__ __forceinline__ void load_at(const T* p, int64_t ld, const Place& at, float x[4][kVec]) {
  if constexpr (kWhole) {
    constexpr int kWords = kVec * (int)sizeof(T) / 16;
    uint4 raw[4][kWords];
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int w = 0; w < kWords; ++w) {
        raw[q][w] = make_uint4(0, 0, 0, 0);
        if (at.n[q] > 0) raw[q][w] = reinterpret_cast<const uint4*>(p + at.row[q] * ld + at.col[q])[w];
      }
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int j = 0; j < kVec; ++j) x[q][j] = num<T>(reinterpret_cast<const T*>(raw[q])[j]);
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        x[q][j] = 0.0f;
        if (j < at.n[q]) x[q][j] = num<T>(p[at.row[q] * ld + at.col[q] + j]);
      }
  }
}

template <bool kWhole>
__device__ __forceinline__ void store_at(float* p, int64_t ld, const Place& at, const float x[4][kVec]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float* to = p + at.row[q] * ld + at.col[q];
    if constexpr (kWhole) {
      if (at.n[q] == 0) continue;
      reinterpret_cast<float4*>(to)[0] = make_float4(x[q][0], x[q][1], x[q][2], x[q][3]);
      reinterpret_cast<float4*>(to)[1] = make_float4(x[q][4], x[q][5], x[q][6], x[q][7]);
    } else {
#pragma unroll
      for (int j = 0; j < kVec; ++j)
        if (j < at.n[q]) to[j] = x[q][j];
    }
  }
}

__device__ __forceinline__ bool aligned(const void* p, int64_t row, int64_t batch, int esize) {
  const int64_t m = 16 / esize;
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && row % m == 0 && batch % m == 0;
}

// What U of a matrix is made from.
template <typename T>
struct Source {
  const T* in;
  float* mom;                // the step's
  int64_t in_row;
  bool whole;                // all of their vectors are whole and aligned
  float f;
  __device__ __forceinline__ Source(const Call& c, const Entry& e, const Io& io, int b)
      : in(static_cast<const T*>(io.in) + (int64_t)b * io.in_batch),
        mom(c.step ? io.mom + (int64_t)b * e.rows * e.cols : nullptr),
        in_row(io.in_row),
        whole(e.cols % kVec == 0 && aligned(io.in, io.in_row, io.in_batch, sizeof(T)) &&
              (!c.step || aligned(io.mom, e.cols, (int64_t)e.rows * e.cols, 4))),
        f(grad_factor(c)) {}
  // U of a thread's vectors.  kNew: `mom` holds the old momentum and gets the
  // new one; else it holds the new one.
  template <bool kNew, bool kWhole>
  __device__ __forceinline__ void read(const Call& c, const Entry& e, const Place& at, float u[4][kVec]) const {
    load_at<kWhole, T>(in, in_row, at, u);
    if (!c.step) return;
    float m[4][kVec];
    load_at<kWhole, float>(mom, e.cols, at, m);
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        const float g = __fmul_rn(u[q][j], f);
        if (kNew) m[q][j] = __fadd_rn(__fmul_rn(c.mu, m[q][j]), g);
        u[q][j] = c.nesterov ? __fadd_rn(g, __fmul_rn(c.mu, m[q][j])) : m[q][j];
      }
    if (kNew) store_at<kWhole>(mom, e.cols, at, m);
  }
  // Walks a CTA's vectors.
  template <bool kNew, typename Where, typename Work>
  __device__ __forceinline__ void walk(const Call& c, const Entry& e, int chunk, Where where, Work work) const {
    Place at;
    float u[4][kVec];
    if (whole) {
#pragma unroll 1
      for (int i = 0; i < c.blocks && where(c, e, chunk, i, &at); ++i) {
        read<kNew, true>(c, e, at, u);
        work(at, u);
      }
    } else {
#pragma unroll 1
      for (int i = 0; i < c.blocks && where(c, e, chunk, i, &at); ++i) {
        read<kNew, false>(c, e, at, u);
        work(at, u);
      }
    }
  }
};

// x as the sum of two binary16 numbers, the second times kLoScale.
__device__ __forceinline__ void split(float2 x, __half2* hi, __half2* lo) {
  *hi = __float22half2_rn(x);
  const float2 h = __half22float2(*hi);
  *lo = __floats2half2_rn(__fmul_rn(__fadd_rn(x.x, -h.x), kLoScale), __fmul_rn(__fadd_rn(x.y, -h.y), kLoScale));
}

// Writes a thread's vectors of X, padding and all.
__device__ __forceinline__ void put_x(const Entry& e, int b, const Place& p, const float u[4][kVec], float inv) {
  const int64_t at = (int64_t)b * block_size(e.rows, e.ldx) + block_at(p.row[0], p.col[0], e.ldx);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    __align__(16) __half2 hi[kVec / 2], lo[kVec / 2];
#pragma unroll
    for (int j = 0; j < kVec / 2; ++j)
      split(make_float2(__fmul_rn(__fmul_rn(u[q][2 * j], inv), kScaleX), __fmul_rn(__fmul_rn(u[q][2 * j + 1], inv), kScaleX)),
            &hi[j], &lo[j]);
    // 32 rows from a multiple of 32 on are within a piece's 128
    *reinterpret_cast<uint4*>(e.x[0] + at + q * 64) = *reinterpret_cast<const uint4*>(hi);
    *reinterpret_cast<uint4*>(e.lo + at + q * 64) = *reinterpret_cast<const uint4*>(lo);
  }
}

__device__ __forceinline__ float inverse(double squares, double eps) { return (float)(1.0 / (sqrt(squares) + eps)); }

// Counters of a matrix, for the products (a call that ended in a fault leaves
// them anywhere).
__device__ __forceinline__ void clear(const Call& c, const Entry& e, int b) {
  c.done[e.unit0 + b] = 0u;
  for (int i = 0; i < e.cuts; ++i) c.cut[e.cut0 + b * e.cuts + i] = 0u;
}

// Stage 1.  Bound by memory: the step reads 2 + 4 bytes a number and writes 4.
// Squares are added in binary32 within a thread's 32 numbers of a block and its
// blocks (256 numbers at most) and in binary64 beyond; the last CTA of a matrix
// adds the CTAs' sums in index order.  Of a matrix that one CTA holds the
// numbers are still there: it writes X at once.
template <typename T, int N>
__global__ void __launch_bounds__(kThreads, 3) muon_stats_kernel(const __grid_constant__ Start<N> s) {
  const Call& c = s.c;
  __shared__ double red[kThreads / 32];
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    c.ws->faults += c.ws->fault;
    c.ws->fault = 0;
    c.ws->skipped = skipped(c);
  }
  if (skipped(c)) return;
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < c.n; i += kThreads) c.io[i] = s.io[i];
  const Part part = part_of(c, blockIdx.x);
  const Entry& e = c.entries[part.entry];
  const int b = part.b;
  const Source<T> from(c, e, s.io[e.item], b);
  const bool alone = e.chunks == 1;
  float sq = 0.0f;
  from.template walk<true>(c, e, part.chunk, place_flat, [&](const Place&, const float(&u)[4][kVec]) {
    float two[2] = {0.0f, 0.0f};
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int j = 0; j < kVec; ++j) two[j % 2] = __fmaf_rn(u[q][j], u[q][j], two[j % 2]);
    sq = __fadd_rn(sq, __fadd_rn(two[0], two[1]));
  });
  double d = sq;
  for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = d;
  __syncthreads();
  const int unit = e.unit0 + b;
  if (alone) {
    d = 0.0;
    for (int i = 0; i < kThreads / 32; ++i) d += red[i];
    const float inv = inverse(d, c.eps);
    if (threadIdx.x == 0) clear(c, e, b);
    // again from L1 or L2
    from.template walk<false>(c, e, 0, place_block,
                              [&](const Place& at, const float(&u)[4][kVec]) { put_x(e, b, at, u, inv); });
    return;
  }
  // the first warp alone ends the CTA's work: the others make room
  if (threadIdx.x >= 32) return;
  double* sums = c.part + e.chunk0 + (int64_t)b * e.chunks;
  int last = 0;
  if (threadIdx.x == 0) {
    for (int i = 1; i < kThreads / 32; ++i) d += red[i];
    sums[part.chunk] = d;
    __threadfence();
    last = atomicAdd(&c.ticket[unit], 1u) == (unsigned)e.chunks - 1;
    __threadfence();
  }
  if (!__shfl_sync(0xffffffffu, last, 0)) return;
  d = 0.0;
#pragma unroll 8
  for (int i = threadIdx.x; i < e.chunks; i += 32) d += __ldcg(&sums[i]);
  for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
  if (threadIdx.x == 0) {
    c.inv[unit] = inverse(d, c.eps);
    c.ticket[unit] = 0u;
    clear(c, e, b);
  }
}

// Stage 2.  Reads U's sources again and writes X.  From the last CTA's numbers
// to the first's: stage 1 ended with the last, which L2 still holds, and the
// products begin with the first.
template <typename T>
__global__ void __launch_bounds__(kThreads, 3) muon_start_kernel(const __grid_constant__ Call c) {
  cudaGridDependencySynchronize();           // launched while stage 1 still runs
  if (skipped(c)) return;
  const Part part = part_of(c, gridDim.x - 1 - blockIdx.x);
  const Entry& e = c.entries[part.entry];
  if (e.chunks == 1) return;                 // stage 1 wrote it
  const int b = part.b;
  const Source<T> from(c, e, c.io[e.item], b);
  const float inv = c.inv[e.unit0 + b];
  from.template walk<false>(c, e, part.chunk, place_block,
                            [&](const Place& at, const float(&u)[4][kVec]) { put_x(e, b, at, u, inv); });
}

}  // namespace zm
