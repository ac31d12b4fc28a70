// block_kernels.cuh -- a block's output joined to the residual stream with its
// norms, gate and dropout, forward and backward (zero_block.h).
//
// What bounds it: memory.  Each row is read once and each result written once;
// sums over a row are taken by the threads that hold it.
//
// Layout: a row of D numbers is cut into chunks of eight, and a team of whole
// warps takes a row at a time: thread i of n holds chunks i, i + n, ... (kC at
// most), the same columns of every row that it sees.  So the gains stay in
// registers, the gains' gradients are summed in registers until the end, and a
// chunk is one block of the dropout's generator.  The teams walk the tokens.
//
// Rows come by cp.async into a ring in shared memory in which every thread reads
// only what it copied itself (kWide: all rows on 16-byte boundaries), so bytes
// in flight cost no registers and no barrier.  Other rows are read number by
// number, a warp's 32 next to one another, through the same shared memory, which
// brings each thread its eight, and written the same way.
#pragma once

#include "numbers.cuh"
#include "philox.cuh"

namespace zo {

constexpr int kJoinThreads = 512;   // of a CTA, at most

struct JoinRow {
  char* data;
  int64_t stride;       // in bytes
};

struct JoinArgs {
  // forward: x, y, gate in; x_out, h out.  backward: x (the x' of the forward
  // pass), y, gate, dxo, dh in; dx, dy, dgate out.  NULL where absent.
  JoinRow x, y, gate, x_out, h, dxo, dh, dx, dy, dgate;
  const float* y_gain;
  const float* gain;
  const uint8_t* mask;
  float* part;          // backward: [grid][2][D] partial gradients of y_gain and gain, or NULL
  int64_t tokens;
  Drop drop;
  int32_t dim, chunks;
  int32_t warps, teams; // of a team; of a CTA
  int32_t ring, vecs;   // rows of the ring; 16-byte vectors of a thread in one
  int32_t gate_kind, post, pre;
  float eps, inv_dim, alpha, beta;
};

template <typename E> constexpr int kVecs = (int)sizeof(E) / 2;   // 16-byte vectors of a chunk

// Waits until at most n of the thread's groups of copies are on their way.
__device__ __forceinline__ void copies_left(int n) {
  if (n >= 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
  else if (n == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
  else asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// The place of a thread in its team and in shared memory, and the moves between
// there and the rows.
template <int kC, bool kWide>
struct Lane {
  const JoinArgs& a;
  unsigned char* smem;    // the CTA's ring
  int threads;            // of the CTA
  int team, lane, lanes;  // this thread's team, its place in it, threads of a team

  __device__ __forceinline__ int chunk(int j) const { return lane + j * lanes; }
  __device__ __forceinline__ bool live(int j) const { return chunk(j) < a.chunks; }
  // numbers of the chunk
  __device__ __forceinline__ int count(int j) const { return min(8, a.dim - chunk(j) * 8); }
  // vector n of the thread in the ring's row `at`
  __device__ __forceinline__ unsigned char* vec(int at, int n) const {
    return smem + ((at * a.vecs + n) * threads + threadIdx.x) * 16;
  }

  // A row's chunks into vectors from `first` on.
  template <typename E>
  __device__ __forceinline__ void fetch(const JoinRow& r, int64_t t, int at, int first) const {
    const char* row = r.data + t * r.stride;
#pragma unroll
    for (int j = 0; j < kC; ++j) {
      if constexpr (kWide) {
        if (!live(j)) continue;
        const char* from = row + (int64_t)chunk(j) * (8 * (int)sizeof(E));
        const int bytes = count(j) * (int)sizeof(E);
#pragma unroll
        for (int v = 0; v < kVecs<E>; ++v) {
          unsigned char* to = vec(at, first + j * kVecs<E> + v);
          if (bytes == 8 * (int)sizeof(E)) copy16(to, from + 16 * v);
          else copy16(to, bytes > 16 * v ? from + 16 * v : row, max(0, min(16, bytes - 16 * v)));
        }
      } else {
        const int l = threadIdx.x % 32, begin = (chunk(j) - l) * 8;
        if (begin >= a.dim) continue;
        E x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int e = begin + k * 32 + l;
          x[k] = e < a.dim ? reinterpret_cast<const E*>(row)[e] : Num<E>::put(0.0f);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) *place<E>(at, first + j * kVecs<E>, k * 32 + l) = x[k];
      }
    }
  }
  // Number e of the 256 that the warp holds in a chunk whose vectors start at n.
  template <typename E>
  __device__ __forceinline__ E* place(int at, int n, int e) const {
    const int l = threadIdx.x % 32;
    unsigned char* v = vec(at, n) - l * 16;                 // lane 0's
    if constexpr (sizeof(E) == 2) return reinterpret_cast<E*>(v) + e;
    else return reinterpret_cast<E*>(v + (e % 8 / 4 * threads + e / 8) * 16) + e % 4;
  }

  template <typename E>
  __device__ __forceinline__ void get(int at, int n, float2* x) const {
    constexpr int kE = 16 / (int)sizeof(E);
#pragma unroll
    for (int v = 0; v < kVecs<E>; ++v) {
      const Vec<E, kE> p = *reinterpret_cast<const Vec<E, kE>*>(vec(at, n + v));
#pragma unroll
      for (int k = 0; k < kE / 2; ++k) x[v * (kE / 2) + k] = Num<E>::get2(p.v + 2 * k);
    }
  }

  // A chunk of a result.  Narrow rows pass through the vectors from n on, which
  // are done with.
  template <typename E>
  __device__ __forceinline__ void put(const JoinRow& r, int64_t t, int j, const float2* x, int at,
                                      int n) const {
    constexpr int kE = 16 / (int)sizeof(E);
    E* row = reinterpret_cast<E*>(r.data + t * r.stride);
    Vec<E, kE> p[kVecs<E>];
#pragma unroll
    for (int v = 0; v < kVecs<E>; ++v)
#pragma unroll
      for (int k = 0; k < kE / 2; ++k) Num<E>::put2(p[v].v + 2 * k, x[v * (kE / 2) + k]);
    if constexpr (kWide) {
      if (!live(j)) return;
      E* to = row + chunk(j) * 8;
      const int left = count(j);
      if (left == 8) {
#pragma unroll
        for (int v = 0; v < kVecs<E>; ++v) reinterpret_cast<Vec<E, kE>*>(to)[v] = p[v];
      } else {
#pragma unroll
        for (int k = 0; k < 7; ++k)
          if (k < left) to[k] = p[k / kE].v[k % kE];
      }
    } else {
      const int l = threadIdx.x % 32, begin = (chunk(j) - l) * 8;
      if (begin >= a.dim) return;
#pragma unroll
      for (int v = 0; v < kVecs<E>; ++v) *reinterpret_cast<Vec<E, kE>*>(vec(at, n + v)) = p[v];
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int e = begin + k * 32 + l;
        if (e < a.dim) row[e] = *place<E>(at, n, k * 32 + l);
      }
      __syncwarp();
    }
  }

  // A chunk of a gain (NULL: ones).
  __device__ __forceinline__ void gain(const float* g, int j, float2* x) const {
    const int left = live(j) ? count(j) : 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = both(g ? 0.0f : 1.0f);
    if (!g) return;
    const float* from = g + chunk(j) * 8;
    if (left == 8 && reinterpret_cast<uintptr_t>(from) % 16 == 0) {
      const float4 lo = __ldg(reinterpret_cast<const float4*>(from));
      const float4 hi = __ldg(reinterpret_cast<const float4*>(from) + 1);
      x[0] = make_float2(lo.x, lo.y);
      x[1] = make_float2(lo.z, lo.w);
      x[2] = make_float2(hi.x, hi.y);
      x[3] = make_float2(hi.z, hi.w);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (2 * k < left) x[k].x = __ldg(from + 2 * k);
        if (2 * k + 1 < left) x[k].y = __ldg(from + 2 * k + 1);
      }
    }
  }

  // Sums over the team's threads, in an order fixed by its size; every thread
  // gets them.  `turn` alternates between two pieces of shared memory, so that
  // one barrier a sum is enough: who writes a piece again has passed the
  // barrier of the sum between, which everyone reaches after reading the first.
  template <int kN>
  __device__ __forceinline__ void sum(float (&x)[kN], float4 (*red)[kJoinThreads / 32], int& turn) const {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < kN; ++i) x[i] = __fadd_rn(x[i], __shfl_xor_sync(0xffffffffu, x[i], o));
    if (a.warps == 1) return;
    float4* mine = red[turn] + team * a.warps;
    if (threadIdx.x % 32 == 0) mine[lane / 32] = make_float4(x[0], kN > 1 ? x[kN > 1] : 0.0f, kN > 2 ? x[kN - 1] : 0.0f, 0.0f);
    asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(lanes) : "memory");
    float4 s = mine[0];
    for (int w = 1; w < a.warps; ++w) {
      const float4 y = mine[w];
      s.x = __fadd_rn(s.x, y.x);
      if (kN > 1) s.y = __fadd_rn(s.y, y.y);
      if (kN > 2) s.z = __fadd_rn(s.z, y.z);
    }
    x[0] = s.x;
    if (kN > 1) x[kN > 1] = s.y;
    if (kN > 2) x[kN - 1] = s.z;
    turn ^= 1;
  }
};

// Eight numbers of which the dropped ones become zero.
__device__ __forceinline__ void drop8(float2* x, uint32_t bits) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (!(bits >> 2 * k & 1)) x[k].x = 0.0f;
    if (!(bits >> 2 * k & 2)) x[k].y = 0.0f;
  }
}

// The gate's factor, in place, and the factor's derivative.  The sigmoid by
// e = exp(-|g|), so that neither it nor its derivative e / (1 + e)^2 is a
// difference of nearly equal numbers.
__device__ __forceinline__ float sigmoid(float g, float* slope) {
  const float e = expf(-fabsf(g)), inv = __frcp_rn(__fadd_rn(1.0f, e)), low = __fmul_rn(e, inv);
  *slope = __fmul_rn(low, inv);
  return g >= 0.0f ? inv : low;
}

__device__ __forceinline__ void act8(int kind, float2* g, float2* slope) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (kind == ZERO_GATE_SIGMOID)
      g[k] = make_float2(sigmoid(g[k].x, &slope[k].x), sigmoid(g[k].y, &slope[k].y));
    else
      slope[k] = both(1.0f);
  }
}

__device__ __forceinline__ float add2(float2 x) { return __fadd_rn(x.x, x.y); }

template <typename T, typename S, int kC, bool kWide>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ JoinArgs a) {
  extern __shared__ __align__(16) unsigned char s_ring[];
  __shared__ float4 s_red[2][kJoinThreads / 32];
  const int lanes = a.warps * 32;
  const Lane<kC, kWide> me{a, s_ring, (int)blockDim.x, (int)threadIdx.x / lanes, (int)threadIdx.x % lanes, lanes};
  constexpr int kY = kC * kVecs<S>, kGate = kY + kC * kVecs<T>;   // vectors: x, y, gate
  const bool with_y = a.y.data, with_gate = a.gate.data;
  const int64_t step = (int64_t)gridDim.x * a.teams;
  const int64_t first = (int64_t)blockIdx.x * a.teams + me.team;
  const uint32_t rng_step = a.drop.cut ? step_of(a.drop) : 0;
  const float scale = __fmul_rn(a.beta, a.drop.factor);

  const auto fetch = [&](int64_t t, int at) {
    if (t < a.tokens) {
      me.template fetch<S>(a.x, t, at, 0);
      if (with_y) me.template fetch<T>(a.y, t, at, kY);
      if (with_gate) me.template fetch<T>(a.gate, t, at, kGate);
    }
    if constexpr (kWide) asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // the gains stay in registers where there is room for them
  constexpr bool kKeep = kC <= 2;
  float2 yg_[kKeep ? kC : 1][4], g_[kKeep ? kC : 1][4];
  if constexpr (kKeep)
#pragma unroll
    for (int j = 0; j < kC; ++j) {
      me.gain(a.y_gain, j, yg_[j]);
      me.gain(a.gain, j, g_[j]);
    }

  const int ahead = a.ring - 1;
  for (int k = 0; k < ahead; ++k) fetch(first + k * step, k);
  int at = 0, turn = 0;
  bool there = first < a.tokens && (!a.mask || __ldg(a.mask + first));
  for (int64_t t = first; t < a.tokens; t += step) {
    if (!kWide) __syncwarp();
    fetch(t + ahead * step, at + ahead >= a.ring ? at + ahead - a.ring : at + ahead);
    const bool next = t + step < a.tokens && (!a.mask || __ldg(a.mask + t + step));
    uint32_t bits[kC];
    if (a.drop.cut && there)
#pragma unroll
      for (int j = 0; j < kC; ++j)
        if (me.live(j)) bits[j] = kept(a.drop, rng_step, t * a.chunks + me.chunk(j));
    if constexpr (kWide) copies_left(ahead);
    else __syncwarp();
    float2 v[kC][4];
    if (there) {
      float ry = scale;
      if (with_y && a.post) {
        float2 sq = both(0.0f);
#pragma unroll
        for (int j = 0; j < kC; ++j)
          if (me.live(j)) {
            float2 y[4];
            me.template get<T>(at, kY + j * kVecs<T>, y);
#pragma unroll
            for (int k = 0; k < 4; ++k) sq = __ffma2_rn(y[k], y[k], sq);
          }
        float s[1] = {add2(sq)};
        me.sum(s, s_red, turn);
        ry = __fmul_rn(rsqrtf(__fmaf_rn(s[0], a.inv_dim, a.eps)), scale);
      }
      float2 sq = both(0.0f);
#pragma unroll
      for (int j = 0; j < kC; ++j) {
        if (!me.live(j)) continue;
        me.template get<S>(at, j * kVecs<S>, v[j]);
        if (with_y) {
          float2 b[4], w[4];
          me.template get<T>(at, kY + j * kVecs<T>, b);
          if constexpr (!kKeep) me.gain(a.y_gain, j, w);
#pragma unroll
          for (int k = 0; k < 4; ++k) b[k] = __fmul2_rn(__fmul2_rn(b[k], both(ry)), kKeep ? yg_[j][k] : w[k]);
          if (with_gate) {
            float2 g[4], slope[4];
            me.template get<T>(at, kGate + j * kVecs<T>, g);
            act8(a.gate_kind, g, slope);
#pragma unroll
            for (int k = 0; k < 4; ++k) b[k] = __fmul2_rn(b[k], g[k]);
          }
          if (a.drop.cut) drop8(b, bits[j]);
#pragma unroll
          for (int k = 0; k < 4; ++k) v[j][k] = __ffma2_rn(v[j][k], both(a.alpha), b[k]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) sq = __ffma2_rn(v[j][k], v[j][k], sq);
      }
      // a narrow result goes out through the places of what was read
      if (a.x_out.data) {
#pragma unroll
        for (int j = 0; j < kC; ++j) me.template put<S>(a.x_out, t, j, v[j], at, j * kVecs<S>);
      }
      if (a.pre) {
        float s[1] = {add2(sq)};
        me.sum(s, s_red, turn);
        const float2 r = both(rsqrtf(__fmaf_rn(s[0], a.inv_dim, a.eps)));
#pragma unroll
        for (int j = 0; j < kC; ++j) {
          float2 w[4];
          if constexpr (!kKeep) me.gain(a.gain, j, w);
#pragma unroll
          for (int k = 0; k < 4; ++k) v[j][k] = __fmul2_rn(__fmul2_rn(v[j][k], r), kKeep ? g_[j][k] : w[k]);
          me.template put<T>(a.h, t, j, v[j], at, kY + j * kVecs<T>);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < kC; ++j) {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[j][k] = both(0.0f);
        if (a.x_out.data) me.template put<S>(a.x_out, t, j, v[j], at, j * kVecs<S>);
        if (a.pre) me.template put<T>(a.h, t, j, v[j], at, kY + j * kVecs<T>);
      }
    }
    there = next;
    at = at + 1 == a.ring ? 0 : at + 1;
  }
}

template <typename T, typename S, int kC, bool kWide>
__global__ void __launch_bounds__(kJoinThreads) join_backward_kernel(const __grid_constant__ JoinArgs a) {
  extern __shared__ __align__(16) unsigned char s_ring[];
  __shared__ float4 s_red[2][kJoinThreads / 32];
  const int lanes = a.warps * 32;
  const Lane<kC, kWide> me{a, s_ring, (int)blockDim.x, (int)threadIdx.x / lanes, (int)threadIdx.x % lanes, lanes};
  // vectors: x', dx', dh, y, gate
  constexpr int kDxo = kC * kVecs<S>, kDh = 2 * kDxo, kY = kDh + kC * kVecs<T>, kGate = kY + kC * kVecs<T>;
  const bool with_y = a.y.data, with_gate = a.gate.data;
  const int64_t step = (int64_t)gridDim.x * a.teams;
  const int64_t first = (int64_t)blockIdx.x * a.teams + me.team;
  const uint32_t rng_step = a.drop.cut ? step_of(a.drop) : 0;
  const float scale = __fmul_rn(a.beta, a.drop.factor);

  const auto fetch = [&](int64_t t, int at) {
    if (t < a.tokens) {
      if (a.dh.data) {
        me.template fetch<S>(a.x, t, at, 0);
        me.template fetch<T>(a.dh, t, at, kDh);
      }
      if (a.dxo.data) me.template fetch<S>(a.dxo, t, at, kDxo);
      if (with_y) me.template fetch<T>(a.y, t, at, kY);
      if (with_gate) me.template fetch<T>(a.gate, t, at, kGate);
    }
    if constexpr (kWide) asm volatile("cp.async.commit_group;" ::: "memory");
  };
  constexpr bool kKeep = kC <= 2;
  float2 yg_[kKeep ? kC : 1][4], g_[kKeep ? kC : 1][4];
  if constexpr (kKeep)
#pragma unroll
    for (int j = 0; j < kC; ++j) {
      me.gain(a.y_gain, j, yg_[j]);
      me.gain(a.gain, j, g_[j]);
    }
  float2 dyg[kC][4], dg[kC][4];
#pragma unroll
  for (int j = 0; j < kC; ++j)
#pragma unroll
    for (int k = 0; k < 4; ++k) dyg[j][k] = dg[j][k] = both(0.0f);

  const int ahead = a.ring - 1;
  for (int k = 0; k < ahead; ++k) fetch(first + k * step, k);
  int at = 0, turn = 0;
  bool there = first < a.tokens && (!a.mask || __ldg(a.mask + first));
  for (int64_t t = first; t < a.tokens; t += step) {
    if (!kWide) __syncwarp();
    fetch(t + ahead * step, at + ahead >= a.ring ? at + ahead - a.ring : at + ahead);
    const bool next = t + step < a.tokens && (!a.mask || __ldg(a.mask + t + step));
    uint32_t bits[kC];
    if (a.drop.cut && there && with_y)
#pragma unroll
      for (int j = 0; j < kC; ++j)
        if (me.live(j)) bits[j] = kept(a.drop, rng_step, t * a.chunks + me.chunk(j));
    if constexpr (kWide) copies_left(ahead);
    else __syncwarp();
    float2 G[kC][4];
    if (there) {
      float2 sx = both(0.0f), sd = both(0.0f), sy = both(0.0f);
#pragma unroll
      for (int j = 0; j < kC; ++j) {
        if (!me.live(j)) continue;
        if (a.dh.data) {
          float2 x[4], d[4], w[4];
          me.template get<S>(at, j * kVecs<S>, x);
          me.template get<T>(at, kDh + j * kVecs<T>, d);
          if constexpr (!kKeep) me.gain(a.gain, j, w);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            sx = __ffma2_rn(x[k], x[k], sx);
            sd = __ffma2_rn(__fmul2_rn(d[k], kKeep ? g_[j][k] : w[k]), x[k], sd);
          }
        }
        if (with_y && a.post) {
          float2 y[4];
          me.template get<T>(at, kY + j * kVecs<T>, y);
#pragma unroll
          for (int k = 0; k < 4; ++k) sy = __ffma2_rn(y[k], y[k], sy);
        }
      }
      float s[3] = {add2(sx), add2(sd), add2(sy)};
      me.sum(s, s_red, turn);
      // G = dx' + r (dn - xhat mean(dn xhat)), dn = dh gain: no power of r but the
      // first, so that it holds for rows of any size
      const float r = rsqrtf(__fmaf_rn(s[0], a.inv_dim, a.eps));
      const float back = __fmul_rn(-r, __fmul_rn(__fmul_rn(r, s[1]), a.inv_dim));
      const float ry = a.post ? rsqrtf(__fmaf_rn(s[2], a.inv_dim, a.eps)) : 1.0f;
      float2 dot = both(0.0f);
#pragma unroll
      for (int j = 0; j < kC; ++j) {
        if (me.live(j)) {
#pragma unroll
          for (int k = 0; k < 4; ++k) G[j][k] = both(0.0f);
          if (a.dxo.data) me.template get<S>(at, kDxo + j * kVecs<S>, G[j]);
          if (a.dh.data) {
            float2 x[4], d[4], w[4];
            me.template get<S>(at, j * kVecs<S>, x);
            me.template get<T>(at, kDh + j * kVecs<T>, d);
            if constexpr (!kKeep) me.gain(a.gain, j, w);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 xhat = __fmul2_rn(x[k], both(r));
              dg[j][k] = __ffma2_rn(d[k], xhat, dg[j][k]);
              const float2 dn = __fmul2_rn(d[k], kKeep ? g_[j][k] : w[k]);
              G[j][k] = __fadd2_rn(G[j][k], __ffma2_rn(dn, both(r), __fmul2_rn(xhat, both(back))));
            }
          }
        }
        if (a.dx.data) {
          float2 o[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) o[k] = with_y ? __fmul2_rn(G[j][k], both(a.alpha)) : G[j][k];
          me.template put<S>(a.dx, t, j, o, at, j * kVecs<S>);
        }
        if (!with_y || !me.live(j)) continue;
        // G becomes db, and the dot product of dz y_gain and y is taken
#pragma unroll
        for (int k = 0; k < 4; ++k) G[j][k] = __fmul2_rn(G[j][k], both(scale));
        if (a.drop.cut) drop8(G[j], bits[j]);
        if (a.post) {
          float2 y[4], g[4], w[4], slope[4];
          me.template get<T>(at, kY + j * kVecs<T>, y);
          if (with_gate) {
            me.template get<T>(at, kGate + j * kVecs<T>, g);
            act8(a.gate_kind, g, slope);
            if (a.drop.cut) drop8(g, bits[j]);
          }
          if constexpr (!kKeep) me.gain(a.y_gain, j, w);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 dz = with_gate ? __fmul2_rn(G[j][k], g[k]) : G[j][k];
            dot = __ffma2_rn(__fmul2_rn(dz, kKeep ? yg_[j][k] : w[k]), y[k], dot);
          }
        }
      }
      if (with_y) {
        float backy = 0.0f;
        if (a.post) {
          float s2[1] = {add2(dot)};
          me.sum(s2, s_red, turn);
          backy = __fmul_rn(-ry, __fmul_rn(__fmul_rn(ry, s2[0]), a.inv_dim));
        }
#pragma unroll
        for (int j = 0; j < kC; ++j) {
          float2 slope[4];
          float2 o[4];
          if (me.live(j)) {
            float2 y[4], g[4], w[4];
            me.template get<T>(at, kY + j * kVecs<T>, y);
            if (with_gate) {
              me.template get<T>(at, kGate + j * kVecs<T>, g);
              act8(a.gate_kind, g, slope);
            }
            if constexpr (!kKeep) me.gain(a.y_gain, j, w);
            float2 rest[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              y[k] = __fmul2_rn(y[k], both(ry));
              rest[k] = __fmul2_rn(y[k], both(backy));
            }
            if (a.drop.cut) {            // a dropped number's factors may be anything
              drop8(y, bits[j]);
              if (with_gate) drop8(g, bits[j]);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 yg = kKeep ? yg_[j][k] : w[k];
              const float2 dz = with_gate ? __fmul2_rn(G[j][k], g[k]) : G[j][k];
              if (with_gate) slope[k] = __fmul2_rn(__fmul2_rn(__fmul2_rn(G[j][k], slope[k]), y[k]), yg);
              dyg[j][k] = __ffma2_rn(dz, y[k], dyg[j][k]);
              o[k] = __fmul2_rn(dz, yg);
              if (a.post) o[k] = __ffma2_rn(o[k], both(ry), rest[k]);
            }
            if (a.drop.cut && with_gate) drop8(slope, bits[j]);
          }
          if (a.dy.data) me.template put<T>(a.dy, t, j, o, at, kY + j * kVecs<T>);
          if (a.dgate.data) me.template put<T>(a.dgate, t, j, slope, at, kY + j * kVecs<T>);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < kC; ++j) {
#pragma unroll
        for (int k = 0; k < 4; ++k) G[j][k] = both(0.0f);
        if (a.dx.data) me.template put<S>(a.dx, t, j, G[j], at, j * kVecs<S>);
        if (a.dy.data) me.template put<T>(a.dy, t, j, G[j], at, kY + j * kVecs<T>);
        if (a.dgate.data) me.template put<T>(a.dgate, t, j, G[j], at, kY + j * kVecs<T>);
      }
    }
    there = next;
    at = at + 1 == a.ring ? 0 : at + 1;
  }

  // The CTA's share of the gains' gradients: its teams' one after the other.
  if (!a.part) return;
  float* to = a.part + (int64_t)blockIdx.x * 2 * a.dim;
  float* s_sum = reinterpret_cast<float*>(s_ring);
  if constexpr (kWide) asm volatile("cp.async.wait_all;" ::: "memory");
  for (int team = 0; team < a.teams; ++team) {
    __syncthreads();
    if (me.team != team) continue;
    const bool last = team == a.teams - 1;
#pragma unroll
    for (int j = 0; j < kC; ++j) {
      const int left = me.live(j) ? me.count(j) : 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (k >= left) continue;
        const int e = me.chunk(j) * 8 + k;
        float y = k % 2 ? dyg[j][k / 2].y : dyg[j][k / 2].x, g = k % 2 ? dg[j][k / 2].y : dg[j][k / 2].x;
        if (team > 0) {
          y = __fadd_rn(s_sum[e], y);
          g = __fadd_rn(s_sum[a.dim + e], g);
        }
        float* at_ = last ? to : s_sum;
        at_[e] = y;
        at_[a.dim + e] = g;
      }
    }
  }
}

}  // namespace zo
