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
//
// Layout: a row is owned by a group of lanes, each holding two vectors of V
// numbers, chosen so that both members of every rotated pair are in the same
// lane: without interleaving the vectors are V numbers of the first rotated
// half and the V numbers they pair with; interleaved they are 2V numbers in a
// row.  So the rotation needs no exchange between lanes, and a 16-byte load
// per vector covers whole sectors.  A group owns R heads for the whole launch
// and walks the tokens: its R rows of a token share one read of the token's
// angles, and their gains' gradients stay in registers to the end.
//
// 16-byte vectors come by cp.async into a ring of kRing tokens in shared memory
// in which every thread reads only what it copied itself, so that bytes in
// flight cost no registers and no barrier; narrower ones are loaded directly.
// The angles of the next token are fetched while the rows are still on their way.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdlib>
#include <mutex>
#include <new>

#include "host_util.h"
#include "numbers.cuh"
#include "zero_qk.h"

namespace {

using zo::both;
using zo::copy16;
using zo::fail;
using zo::Num;
using zo::Vec;

constexpr int kQkThreads = 256;
constexpr int kMaxDim = 512;
constexpr int kMaxPerSm = 6;      // CTAs an SM: what the workspace has room for
constexpr int kMaxSmem = 200 * 1024;

struct Rows {
  const char* in;      // x
  const char* gout;    // backward: gradient of the result
  char* out;           // forward: result; backward: dx
  int64_t in_t, in_h, go_t, go_h, out_t, out_h;   // strides in elements
  const float* gain;
  int32_t heads;
};

struct QkArgs {
  Rows r[2];           // queries, keys
  const float* cos;
  const float* sin;
  const void* pos;
  int64_t tokens, n_pos;
  float* part;         // backward: [grid][rows a CTA][D] partial gain gradients
  int32_t pos64, dim, rot, chunks, lanes, gain_per_head;
  int32_t heads;       // of both
  int32_t per;         // groups a token in a CTA, each of R heads
  int32_t head_blocks; // CTAs side by side over the heads
  int32_t reps;        // tokens a CTA takes at once
  int32_t part_rows;   // rows of a CTA's partial: 2 (shared gains) or its heads
  float eps, inv_dim;
};

// A chunk: the lane's two vectors one after the other, as V pairs of numbers
// for the two-wide binary32 instructions.
template <typename T, int V>
__device__ __forceinline__ void widen(const Vec<T, V>& u, const Vec<T, V>& v, float2* x) {
  if constexpr (V == 1) {
    x[0] = make_float2(Num<T>::get(u.v[0]), Num<T>::get(v.v[0]));
  } else {
#pragma unroll
    for (int k = 0; k < V / 2; ++k) {
      x[k] = Num<T>::get2(u.v + 2 * k);
      x[V / 2 + k] = Num<T>::get2(v.v + 2 * k);
    }
  }
}

template <typename T, int V>
__device__ __forceinline__ void narrow(const float2* x, Vec<T, V>& u, Vec<T, V>& v) {
  if constexpr (V == 1) {
    u.v[0] = Num<T>::put(x[0].x);
    v.v[0] = Num<T>::put(x[0].y);
  } else {
#pragma unroll
    for (int k = 0; k < V / 2; ++k) {
      Num<T>::put2(u.v + 2 * k, x[k]);
      Num<T>::put2(v.v + 2 * k, x[V / 2 + k]);
    }
  }
}

template <typename T, int V>
__device__ __forceinline__ Vec<T, V> load(const char* p, int e) {
  return *reinterpret_cast<const Vec<T, V>*>(reinterpret_cast<const T*>(p) + e);
}
template <typename T, int V>
__device__ __forceinline__ void store(char* p, int e, const Vec<T, V>& x) {
  *reinterpret_cast<Vec<T, V>*>(reinterpret_cast<T*>(p) + e) = x;
}

// Where the two vectors of chunk c start.
template <int V, bool kInter>
__device__ __forceinline__ void places(const QkArgs& a, int c, int* p0, int* p1) {
  if (kInter || c * 2 * V >= a.rot) {
    *p0 = c * 2 * V;
    *p1 = *p0 + V;
  } else {
    *p0 = c * V;
    *p1 = a.rot / 2 + c * V;
  }
}

__device__ __forceinline__ int64_t position(const QkArgs& a, int64_t t) {
  return a.pos64 ? __ldg(static_cast<const long long*>(a.pos) + t)
                 : (int64_t)__ldg(static_cast<const int*>(a.pos) + t);
}

// The rotation of one chunk, or with -sin its inverse.
template <int V, bool kInter>
__device__ __forceinline__ void turn(float2* x, const float* cs, const float* sn, bool inverse) {
  if constexpr (kInter || V == 1) {
#pragma unroll
    for (int k = 0; k < V; ++k) {          // a pair (u, v) of its own angle
      const float s = inverse ? -sn[k] : sn[k];
      x[k] = __ffma2_rn(x[k], both(cs[k]), __fmul2_rn(make_float2(x[k].y, x[k].x), make_float2(-s, s)));
    }
  } else {
#pragma unroll
    for (int k = 0; k < V / 2; ++k) {      // two u and their two v
      const float2 u = x[k], v = x[V / 2 + k], c = make_float2(cs[2 * k], cs[2 * k + 1]);
      const float2 s = inverse ? make_float2(-sn[2 * k], -sn[2 * k + 1]) : make_float2(sn[2 * k], sn[2 * k + 1]);
      x[k] = __ffma2_rn(u, c, __fmul2_rn(v, make_float2(-s.x, -s.y)));
      x[V / 2 + k] = __ffma2_rn(v, c, __fmul2_rn(u, s));
    }
  }
}

template <int V>
__device__ __forceinline__ void load_f(const float* p, float* x) {
  constexpr int kW = V < 4 ? V : 4;
#pragma unroll
  for (int i = 0; i < V / kW; ++i) {
    const Vec<float, kW> y = reinterpret_cast<const Vec<float, kW>*>(p)[i];
#pragma unroll
    for (int j = 0; j < kW; ++j) x[i * kW + j] = y.v[j];
  }
}

constexpr int kRing = 2;

// Bytes of a CTA's ring: R rows of C chunks of two vectors, for the row and
// (backward) its gradient.
constexpr int ring_bytes(int threads, int c, int r, bool backward) {
  return kRing * threads * r * c * 2 * (backward ? 2 : 1) * 16;
}

// V numbers a vector, C chunks a lane, R heads a group (all queries or all
// keys).  kSum: one sum of gain gradients a group (a shared gain) instead of
// one a head.
template <typename T, int V, int C, int R, bool kInter, bool kBackward, bool kSum>
__global__ void __launch_bounds__(kQkThreads, kBackward ? 2 : 3) qk_kernel(const __grid_constant__ QkArgs a) {
  extern __shared__ __align__(16) unsigned char s_raw[];
  constexpr bool kAsync = sizeof(T) * V == 16;
  constexpr int kEach = kBackward ? 4 : 2;                 // vectors of a chunk
  constexpr int kSums = !kBackward ? 1 : kSum ? 1 : R;
  const int lanes = a.lanes;
  const int group = threadIdx.x / lanes, lane = threadIdx.x % lanes;
  // the group's lanes of its warp: groups of one warp walk on by themselves
  const unsigned mask = (lanes == 32 ? 0xffffffffu : (1u << lanes) - 1u)
                        << (threadIdx.x % 32 / lanes * lanes);
  const int block = blockIdx.x % a.head_blocks;
  const int rep = group / a.per;
  const int head0 = (block * a.per + group % a.per) * R;
  const bool on = rep < a.reps && head0 < a.heads;
  const int64_t slots = (int64_t)(gridDim.x / a.head_blocks) * a.reps;
  const int64_t first = (int64_t)(blockIdx.x / a.head_blocks) * a.reps + rep;
  const Rows& w = a.r[on && head0 >= a.r[0].heads ? 1 : 0];
  const int local = head0 - (head0 >= a.r[0].heads ? a.r[0].heads : 0);
  int p0[C], p1[C];
#pragma unroll
  for (int j = 0; j < C; ++j) places<V, kInter>(a, min(lane + j * lanes, a.chunks - 1), &p0[j], &p1[j]);
  const auto live = [&](int j) { return lane + j * lanes < a.chunks; };

  float2 dgain[kSums][C][V];
  if (kBackward)
#pragma unroll
    for (int r = 0; r < kSums; ++r)
#pragma unroll
      for (int j = 0; j < C; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) dgain[r][j][i] = both(0.0f);
  float2 gain[C][V];
  const auto load_gain = [&](int r) {
#pragma unroll
    for (int j = 0; j < C; ++j)
      if (w.gain && live(j)) {
        const float* gp = w.gain + (a.gain_per_head ? (int64_t)(local + r) * a.dim : 0);
        widen<float, V>(load<float, V>(reinterpret_cast<const char*>(gp), p0[j]),
                        load<float, V>(reinterpret_cast<const char*>(gp), p1[j]), gain[j]);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) gain[j][i] = both(1.0f);
      }
  };

  // the group's rows of its next token, in bytes
  constexpr int kS = (int)sizeof(T);
  const char* in = w.in + (first * w.in_t + (int64_t)local * w.in_h) * kS;
  const char* go = kBackward ? w.gout + (first * w.go_t + (int64_t)local * w.go_h) * kS : nullptr;
  char* out = w.out + (first * w.out_t + (int64_t)local * w.out_h) * kS;
  const int64_t in_t = slots * w.in_t * kS, in_h = w.in_h * kS;
  const int64_t go_t = slots * w.go_t * kS, go_h = w.go_h * kS;
  const int64_t out_t = slots * w.out_t * kS, out_h = w.out_h * kS;
  const int step = blockDim.x * 16;                        // ring: from vector to vector
  unsigned char* const mine = s_raw + threadIdx.x * 16;

  // Starts the copies of a token's rows into slot `at` of the ring.
  const auto fetch = [&](bool there, int at) {
    if constexpr (kAsync) {
      if (there) {
        unsigned char* to = mine + at * (R * C * kEach) * step;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int j = 0; j < C; ++j) {
            if (!live(j)) continue;
            const int n = (r * C + j) * kEach;
            copy16(to + n * step, in + r * in_h + p0[j] * kS);
            copy16(to + (n + 1) * step, in + r * in_h + p1[j] * kS);
            if constexpr (kBackward) {
              copy16(to + (n + 2) * step, go + r * go_h + p0[j] * kS);
              copy16(to + (n + 3) * step, go + r * go_h + p1[j] * kS);
            }
          }
        in += in_t;
        if (kBackward) go += go_t;
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  };
  float cs[C][V], sn[C][V];
  const auto angles = [&](int64_t p) {
    if (p < 0 || p >= a.n_pos) return;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int c = lane + j * lanes;
      if (c < a.chunks && c * 2 * V < a.rot) {
        load_f<V>(a.cos + p * (a.rot / 2) + c * V, cs[j]);
        load_f<V>(a.sin + p * (a.rot / 2) + c * V, sn[j]);
      }
    }
  };

  if (on && first < a.tokens) {
    int64_t p = position(a, first);
    int64_t next = first + slots < a.tokens ? position(a, first + slots) : 0;
#pragma unroll
    for (int k = 0; k < kRing - 1; ++k) fetch(first + k * slots < a.tokens, k);
    angles(p);
    if (R == 1 || !a.gain_per_head) load_gain(0);
    int at = 0;
    for (int64_t t = first; t < a.tokens; t += slots) {
      fetch(t + (kRing - 1) * slots < a.tokens, at == 0 ? kRing - 1 : at - 1);
      if constexpr (kAsync) asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
      // padding, or no angle for this position: a fill of the rows
      const bool skip = p < 0 || (p >= a.n_pos && a.rot > 0);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (skip) {
          const float f = p < 0 ? 0.0f : __int_as_float(0x7fffffff);
          Vec<T, V> z;
#pragma unroll
          for (int i = 0; i < V; ++i) z.v[i] = Num<T>::put(f);
#pragma unroll
          for (int j = 0; j < C; ++j) {
            if (!live(j)) continue;
            store<T, V>(out + r * out_h, p0[j], z);
            store<T, V>(out + r * out_h, p1[j], z);
            if (kBackward && p >= 0)
#pragma unroll
              for (int i = 0; i < V; ++i) dgain[kSum ? 0 : r][j][i] = both(f);
          }
          if (!kBackward && r == R - 1 && t + slots < a.tokens) angles(next);
          continue;
        }
        if (R > 1 && a.gain_per_head) load_gain(r);
        float2 x[C][V], g[C][V];
        float2 sq = both(0.0f), dot = both(0.0f);
#pragma unroll
        for (int j = 0; j < C; ++j) {
          if (!live(j)) continue;
          const bool turned = (lane + j * lanes) * 2 * V < a.rot;
          const unsigned char* from = mine + (at * (R * C * kEach) + (r * C + j) * kEach) * step;
          const auto vec = [&](int k, const char* row, int e) {
            if constexpr (kAsync) return *reinterpret_cast<const Vec<T, V>*>(from + k * step);
            else return load<T, V>(row, e);
          };
          widen<T, V>(vec(0, in + r * in_h, p0[j]), vec(1, in + r * in_h, p1[j]), x[j]);
#pragma unroll
          for (int i = 0; i < V; ++i) sq = __ffma2_rn(x[j][i], x[j][i], sq);
          if constexpr (kBackward) {
            widen<T, V>(vec(2, go + r * go_h, p0[j]), vec(3, go + r * go_h, p1[j]), g[j]);
            if (turned) turn<V, kInter>(g[j], cs[j], sn[j], true);
#pragma unroll
            for (int i = 0; i < V; ++i) dot = __ffma2_rn(__fmul2_rn(g[j][i], gain[j][i]), x[j][i], dot);
          } else {
            // the rotation does not wait for the norm, which scales it as a whole
#pragma unroll
            for (int i = 0; i < V; ++i) x[j][i] = __fmul2_rn(x[j][i], gain[j][i]);
            if (turned) turn<V, kInter>(x[j], cs[j], sn[j], false);
          }
        }
        // forward the next token's angles come as soon as these are done with; the
        // backward pass has no registers to wait for them in
        if (!kBackward && r == R - 1 && t + slots < a.tokens) angles(next);
        float sum = __fadd_rn(sq.x, sq.y), sum_dot = __fadd_rn(dot.x, dot.y);
        for (int o = lanes >> 1; o > 0; o >>= 1) {
          sum = __fadd_rn(sum, __shfl_xor_sync(mask, sum, o));
          if (kBackward) sum_dot = __fadd_rn(sum_dot, __shfl_xor_sync(mask, sum_dot, o));
        }
        const float inv = rsqrtf(__fmaf_rn(sum, a.inv_dim, a.eps));
        const float2 inv2 = both(inv);
        // dx = inv (dn - xhat mean(dn xhat)), dn = dy gain: no power of inv but the
        // first, so that it holds for rows of any size
        const float2 back = both(__fmul_rn(-inv, __fmul_rn(__fmul_rn(inv, sum_dot), a.inv_dim)));
#pragma unroll
        for (int j = 0; j < C; ++j) {
          if (!live(j)) continue;
#pragma unroll
          for (int i = 0; i < V; ++i) {
            if constexpr (kBackward) {
              float2& d = dgain[kSum ? 0 : r][j][i];
              const float2 xhat = __fmul2_rn(x[j][i], inv2);
              d = __ffma2_rn(g[j][i], xhat, d);
              x[j][i] = __ffma2_rn(__fmul2_rn(g[j][i], gain[j][i]), inv2, __fmul2_rn(xhat, back));
            } else {
              x[j][i] = __fmul2_rn(x[j][i], inv2);
            }
          }
          Vec<T, V> u, v;
          narrow<T, V>(x[j], u, v);
          store<T, V>(out + r * out_h, p0[j], u);
          store<T, V>(out + r * out_h, p1[j], v);
        }
      }
      if (!kAsync) {
        in += in_t;
        if (kBackward) go += go_t;
      }
      out += out_t;
      p = next;
      if (kBackward && t + slots < a.tokens) angles(p);
      if (t + 2 * slots < a.tokens) next = position(a, t + 2 * slots);
      at = at == kRing - 1 ? 0 : at + 1;
    }
  }

  if constexpr (kBackward) {
    if (!a.part) return;
    // The CTA's share of the gains' gradients: a group's sums to shared memory
    // (over the ring, which is done with), each column then added over the
    // groups in order.
    if constexpr (kAsync) asm volatile("cp.async.wait_all;" ::: "memory");
    float* s_part = reinterpret_cast<float*>(s_raw);
    float* to = a.part + (int64_t)blockIdx.x * a.part_rows * a.dim;
    // groups of queries among the CTA's
    const int nq = min(max(a.r[0].heads / R - block * a.per, 0), a.per);
#pragma unroll
    for (int r = 0; r < kSums; ++r) {
      __syncthreads();
      if (rep < a.reps)
#pragma unroll
        for (int j = 0; j < C; ++j) {
          if (!live(j)) continue;
          float* s = s_part + group * a.dim;
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const int e = 2 * i;                 // number e of the two vectors
            const float2 d = on ? dgain[r][j][i] : both(0.0f);
            if constexpr (V == 1) {
              s[p0[j]] = d.x;
              s[p1[j]] = d.y;
            } else {
              float* q = s + (e < V ? p0[j] + e : p1[j] + e - V);
              q[0] = d.x;
              q[1] = d.y;
            }
          }
        }
      __syncthreads();
      const int rows = kSum ? 2 : a.per;
      for (int e = threadIdx.x; e < rows * a.dim; e += blockDim.x) {
        const int row = e / a.dim, d = e % a.dim;
        const int lo = !kSum ? row : row ? nq : 0, hi = !kSum ? row + 1 : row ? a.per : nq;
        float s = 0.0f;
        for (int q = 0; q < a.reps; ++q)
          for (int k = lo; k < hi; ++k) s = __fadd_rn(s, s_part[(q * a.per + k) * a.dim + d]);
        to[kSum ? e : (row * R + r) * a.dim + d] = s;
      }
    }
  }
}

struct FoldArgs {
  const float* part;
  float* out[2];
  int32_t grid, head_blocks, part_rows, per, dim, q_heads, heads, gain_per_head;
};

// Sums the CTAs' partial gain gradients in index order: 32 columns a CTA, 8
// threads a column, each over every eighth partial.
__global__ void __launch_bounds__(256) qk_fold_kernel(const __grid_constant__ FoldArgs a) {
  __shared__ float s[8][33];
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
    for (; c + 56 * step < a.grid; c += 64 * step) {
      float v[8];                // eight loads on their way at once
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = at[(c + 8 * k * step) * one];
#pragma unroll
      for (int k = 0; k < 8; ++k) sum = __fadd_rn(sum, v[k]);
    }
#pragma unroll 4
    for (; c < a.grid; c += 8 * step) sum = __fadd_rn(sum, at[c * one]);
  }
  s[part][threadIdx.x % 32] = sum;
  __syncthreads();
  if (part == 0 && row < rows) {
    for (int k = 1; k < 8; ++k) sum = __fadd_rn(sum, s[k][threadIdx.x]);
    const int which = a.gain_per_head ? (row >= a.q_heads) : row;
    const int at = a.gain_per_head ? row - (which ? a.q_heads : 0) : 0;
    if (a.out[which]) a.out[which][(int64_t)at * a.dim + d] = sum;
  }
}

bool fits(const void* p, int64_t s0, int64_t s1, int bytes, int esize) {
  return reinterpret_cast<uintptr_t>(p) % bytes == 0 && s0 * esize % bytes == 0 &&
         s1 * esize % bytes == 0;
}

template <typename T, bool kInter, bool kBackward, bool kSum>
const void* kernel_for(int v, int r) {
  if constexpr (sizeof(T) == 2)
    if (v == 8) {
      if constexpr (!kBackward)
        if (r == 4) return (const void*)qk_kernel<T, 8, 1, 4, kInter, kBackward, kSum>;
      if constexpr (!kBackward || kSum)
        if (r == 2) return (const void*)qk_kernel<T, 8, 1, 2, kInter, kBackward, kSum>;
      return (const void*)qk_kernel<T, 8, 1, 1, kInter, kBackward, kSum>;
    }
  switch (v) {
    case 4:
      if constexpr (sizeof(T) == 4 && !kBackward)
        if (r == 2) return (const void*)qk_kernel<T, 4, 2, 2, kInter, kBackward, kSum>;
      return (const void*)qk_kernel<T, 4, 2, 1, kInter, kBackward, kSum>;
    case 2: return (const void*)qk_kernel<T, 2, 4, 1, kInter, kBackward, kSum>;
    default: return (const void*)qk_kernel<T, 1, 8, 1, kInter, kBackward, kSum>;
  }
}

template <typename T, bool kInter>
const void* kernel_of(bool backward, bool sum, int v, int r) {
  if (!backward) return kernel_for<T, kInter, false, false>(v, r);
  return sum ? kernel_for<T, kInter, true, true>(v, r) : kernel_for<T, kInter, true, false>(v, r);
}

template <typename T>
const void* kernel_of(bool inter, bool backward, bool sum, int v, int r) {
  return inter ? kernel_of<T, true>(backward, sum, v, r) : kernel_of<T, false>(backward, sum, v, r);
}

}  // namespace

struct zero_qk_handle {
  zero_qk_config cfg;
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
  if (b->tokens < 0 || b->n_pos < 0) return fail(ZERO_EINVAL, "tokens and n_pos must be >= 0");
  const zero_qk_tensor* out[2] = {backward ? &b->dq : &b->q_out, backward ? &b->dk : &b->k_out};
  const zero_qk_tensor* in[2] = {&b->q, &b->k};
  const zero_qk_tensor* go[2] = {&b->q_out, &b->k_out};
  if (b->tokens > 0) {
    for (int w = 0; w < (c.k_heads > 0 ? 2 : 1); ++w)
      if (!in[w]->data || !out[w]->data || (backward && !go[w]->data))
        return fail(ZERO_EINVAL, "a %s tensor is NULL", w ? "key" : "query");
    for (int w = 0; w < (c.k_heads > 0 ? 2 : 1); ++w)
      if ((b->tokens > 1 && std::abs(out[w]->token_stride) < c.head_dim) ||
          ((w ? c.k_heads : c.q_heads) > 1 && std::abs(out[w]->head_stride) < c.head_dim))
        return fail(ZERO_EINVAL, "rows of a %s result lie on one another", w ? "key" : "query");
    if (!b->positions) return fail(ZERO_EINVAL, "positions are NULL");
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

  QkArgs a = {};
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
  a.eps = (float)c.eps;
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
  const int groups = kQkThreads / a.lanes;
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
  const int threads = (a.per * a.reps * a.lanes + 31) / 32 * 32;
  const void* fn = c.dtype == ZERO_FP16   ? kernel_of<__half>(c.interleaved, backward, sum, v, r)
                   : c.dtype == ZERO_BF16 ? kernel_of<__nv_bfloat16>(c.interleaved, backward, sum, v, r)
                                          : kernel_of<float>(c.interleaved, backward, sum, v, r);
  size_t smem = es_vec == 16 ? (size_t)ring_bytes(threads, chunks_lane, r, backward) : 0;
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
    lc.blockDim = dim3(256);
    lc.stream = s;
    lc.attrs = &early;
    lc.numAttrs = 1;
    e = cudaLaunchKernelExC(&lc, (const void*)qk_fold_kernel, fp);
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
