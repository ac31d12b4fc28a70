// qk_kernels.cuh -- each head's query and key normalised and rotated in one
// pass (zero_qk.h): the kernel, forward and backward, with one position a token
// or one for each of several axes.
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
#pragma once

#include <cuda_runtime.h>

#include <type_traits>

#include "numbers.cuh"
#include "qk_host.h"
#include "zero_qk.h"

namespace zo {

constexpr int kQkThreads = 256;

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

// The same with a position for each of several axes: pair j turns by the
// position of the axis in bits 2 (j % 16) of word j / 16.
constexpr int kMaxAxes = 4;
struct QkAxesArgs : QkArgs {
  uint32_t axis[16];
  int32_t axes;
  int32_t norm;        // 0: rows are only rotated
  int32_t inverse;     // forward: turned back, which is the rotation's gradient
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

__device__ __forceinline__ int64_t position(const QkArgs& a, int64_t i) {
  return a.pos64 ? __ldg(static_cast<const long long*>(a.pos) + i)
                 : (int64_t)__ldg(static_cast<const int*>(a.pos) + i);
}

// A token's position, or its positions: `first` is negative for padding and n_pos
// or more where an axis has no angle.
struct Position {
  int64_t first;
};
// Several lie in shared memory (kPosSlots tokens' for each group of lanes), where
// they come with the rows, a token ahead of them: in registers, with their checks,
// they left too few for the rows (16,384 tokens over three axes 74 us, 65 so, with two CTAs an SM).
constexpr int kPosSlots = 4, kPosBytes = kMaxAxes * 8;
struct Positions {
  int first;
  const unsigned char* at;
  __device__ __forceinline__ int of(int axis) const { return *reinterpret_cast<const int*>(at + axis * 8); }
};

__device__ __forceinline__ Positions positions(const QkAxesArgs& a, const unsigned char* at) {
  bool low = false, high = false;
  for (int k = 0; k < a.axes; ++k) {
    const int64_t v = a.pos64 ? *reinterpret_cast<const int64_t*>(at + k * 8)
                              : (int64_t)*reinterpret_cast<const int*>(at + k * 8);
    low |= v < 0;
    high |= v >= a.n_pos;
  }
  // n_pos is at most the second
  return {low ? -1 : high ? 0x7fffffff : 0, at};
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
template <typename T, int V, int C, int R, bool kInter, bool kBackward, bool kSum, bool kAxes>
__global__ void __launch_bounds__(kQkThreads, kBackward || kAxes ? 2 : 3)
    qk_kernel(const __grid_constant__ std::conditional_t<kAxes, QkAxesArgs, QkArgs> a) {
  extern __shared__ __align__(16) unsigned char s_raw[];
  constexpr bool kAsync = sizeof(T) * V == 16;
  constexpr int kEach = kBackward ? 4 : 2;                 // vectors of a chunk
  constexpr int kSums = !kBackward ? 1 : kSum ? 1 : R;
  const int lanes = a.lanes;
  // (rows that are only rotated need no power of two lanes: the rest of a warp idles)
  const int in_warp = 32 / lanes;
  const int group = kAxes ? threadIdx.x / 32 * in_warp + threadIdx.x % 32 / lanes : threadIdx.x / lanes;
  const int lane = kAxes ? threadIdx.x % 32 % lanes : threadIdx.x % lanes;
  const bool idle = kAxes && threadIdx.x % 32 >= in_warp * lanes;
  // the group's lanes of its warp: groups of one warp walk on by themselves
  const unsigned mask = (lanes == 32 ? 0xffffffffu : (1u << lanes) - 1u)
                        << (threadIdx.x % 32 / lanes * lanes);
  const int block = blockIdx.x % a.head_blocks;
  const int rep = group / a.per;
  const int head0 = (block * a.per + group % a.per) * R;
  const bool on = rep < a.reps && head0 < a.heads && !idle;
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
  using At = std::conditional_t<kAxes, Positions, Position>;
  // Positions of the group's token number n, or of the token n slots behind its
  // first (one position: loaded a token ahead into `next`, which is not looked at
  // until it is used, so that it is not waited for).
  unsigned char* const pos = s_raw + (kAsync ? kRing * (R * C * kEach) * step : 0) + group * (kPosSlots * kPosBytes);
  const auto fetch_positions = [&](int n, int64_t t) {
    if constexpr (kAxes) {
      if (t >= a.tokens) return;
      for (int k = lane; k < a.axes; k += lanes) {
        const uint32_t to = (uint32_t)__cvta_generic_to_shared(pos + n % kPosSlots * kPosBytes + k * 8);
        if (a.pos64)
          asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to),
                       "l"(static_cast<const int64_t*>(a.pos) + k * a.tokens + t) : "memory");
        else
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to),
                       "l"(static_cast<const int*>(a.pos) + k * a.tokens + t) : "memory");
      }
    }
  };
  int64_t next = 0;
  const auto look = [&](int n) -> At {
    if constexpr (kAxes) return positions(a, pos + n % kPosSlots * kPosBytes);
    else return {next};
  };
  // the axes of a chunk's pairs, two bits each
  uint32_t axis[kAxes ? C : 1];
  if constexpr (kAxes)
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int pair = min(lane + j * lanes, a.chunks - 1) * V;
      axis[j] = a.axis[pair / 16 % 16] >> pair % 16 * 2;
    }
  const auto angles = [&](const At& p) {
    if (p.first < 0 || p.first >= a.n_pos) return;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int c = lane + j * lanes;
      if (c < a.chunks && c * 2 * V < a.rot) {
        if constexpr (kAxes) {
          // four angles of one axis at a time where they have one
          constexpr int kW = V < 4 ? V : 4;
          constexpr uint32_t kOne = kW == 4 ? 0x55 : kW == 2 ? 5 : 1;
#pragma unroll
          for (int i = 0; i < V; i += kW) {
            const uint32_t bits = axis[j] >> 2 * i & (4u << 2 * (kW - 1)) - 1u, ax = bits & 3;
            const int64_t at = (int64_t)p.of(ax) * (a.rot / 2) + c * V + i;
            if (bits == ax * kOne) {
              load_f<kW>(a.cos + at, cs[j] + i);
              load_f<kW>(a.sin + at, sn[j] + i);
            } else {
#pragma unroll
              for (int k = 0; k < kW; ++k) {
                const int64_t e = (int64_t)p.of(bits >> 2 * k & 3) * (a.rot / 2) + c * V + i + k;
                cs[j][i + k] = __ldg(a.cos + e);
                sn[j][i + k] = __ldg(a.sin + e);
              }
            }
          }
        } else {
          load_f<V>(a.cos + p.first * (a.rot / 2) + c * V, cs[j]);
          load_f<V>(a.sin + p.first * (a.rot / 2) + c * V, sn[j]);
        }
      }
    }
  };

  if (on && first < a.tokens) {
    At p;
    if constexpr (kAxes) {
      fetch_positions(0, first);
      fetch_positions(1, first + slots);
      asm volatile("cp.async.commit_group;" ::: "memory");
    } else {
      p.first = position(a, first);
      next = first + slots < a.tokens ? position(a, first + slots) : 0;
    }
#pragma unroll
    for (int k = 0; k < kRing - 1; ++k) fetch(first + k * slots < a.tokens, k);
    if constexpr (kAxes) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kAsync ? kRing - 1 : 0) : "memory");
      __syncwarp(mask);
      p = look(0);
    }
    angles(p);
    if (R == 1 || !a.gain_per_head) load_gain(0);
    int n = 0;                 // the token's number among the group's
    int at = 0;
    for (int64_t t = first; t < a.tokens; t += slots) {
      fetch_positions(n + 2, t + 2 * slots);  // over those of token n - 2, which all lanes have looked at
      fetch(t + (kRing - 1) * slots < a.tokens, at == 0 ? kRing - 1 : at - 1);
      if constexpr (kAxes && !kAsync) asm volatile("cp.async.commit_group;" ::: "memory");
      if constexpr (kAsync || kAxes) asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
      if constexpr (kAxes) __syncwarp(mask);
      // padding, or no angle for this position: a fill of the rows
      const bool skip = p.first < 0 || (p.first >= a.n_pos && a.rot > 0);
      if constexpr (kAxes && !kBackward) {
        // Two rows at a time, so that their sums over the lanes do not wait for one
        // another (16,384 tokens over three axes 66 us a row at a time, 62 so, four
        // at a time, whose registers spill, 81).
        constexpr int kPair = R < 2 ? R : 2;
#pragma unroll
        for (int r0 = 0; r0 < R; r0 += kPair) {
          float2 x[kPair][C][V];
          float sum[kPair];
          if (!skip) {
#pragma unroll
            for (int q = 0; q < kPair; ++q) {
              const int r = r0 + q;
              if (R > 1 && a.gain_per_head) load_gain(r);
              float2 sq = both(0.0f);
#pragma unroll
              for (int j = 0; j < C; ++j) {
                if (!live(j)) continue;
                const unsigned char* from = mine + (at * (R * C * kEach) + (r * C + j) * kEach) * step;
                const auto vec = [&](int k, int e) {
                  if constexpr (kAsync) return *reinterpret_cast<const Vec<T, V>*>(from + k * step);
                  else return load<T, V>(in + r * in_h, e);
                };
                widen<T, V>(vec(0, p0[j]), vec(1, p1[j]), x[q][j]);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                  sq = __ffma2_rn(x[q][j][i], x[q][j][i], sq);
                  x[q][j][i] = __fmul2_rn(x[q][j][i], gain[j][i]);
                }
                if ((lane + j * lanes) * 2 * V < a.rot) turn<V, kInter>(x[q][j], cs[j], sn[j], a.inverse);
              }
              sum[q] = __fadd_rn(sq.x, sq.y);
            }
          }
          if (r0 + kPair >= R && t + slots < a.tokens) angles(look(n + 1));
          if (!skip && a.norm) {
            for (int o = lanes >> 1; o > 0; o >>= 1)
#pragma unroll
              for (int q = 0; q < kPair; ++q) sum[q] = __fadd_rn(sum[q], __shfl_xor_sync(mask, sum[q], o));
#pragma unroll
            for (int q = 0; q < kPair; ++q) {
              const float2 inv = both(rsqrtf(__fmaf_rn(sum[q], a.inv_dim, a.eps)));
#pragma unroll
              for (int j = 0; j < C; ++j)
#pragma unroll
                for (int i = 0; i < V; ++i) x[q][j][i] = __fmul2_rn(x[q][j][i], inv);
            }
          }
#pragma unroll
          for (int q = 0; q < kPair; ++q)
#pragma unroll
            for (int j = 0; j < C; ++j) {
              if (!live(j)) continue;
              if (skip)
#pragma unroll
                for (int i = 0; i < V; ++i) x[q][j][i] = both(p.first < 0 ? 0.0f : __int_as_float(0x7fffffff));
              Vec<T, V> u, v;
              narrow<T, V>(x[q][j], u, v);
              store<T, V>(out + (r0 + q) * out_h, p0[j], u);
              store<T, V>(out + (r0 + q) * out_h, p1[j], v);
            }
        }
      } else {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (skip) {
          const float f = p.first < 0 ? 0.0f : __int_as_float(0x7fffffff);
          Vec<T, V> z;
#pragma unroll
          for (int i = 0; i < V; ++i) z.v[i] = Num<T>::put(f);
#pragma unroll
          for (int j = 0; j < C; ++j) {
            if (!live(j)) continue;
            store<T, V>(out + r * out_h, p0[j], z);
            store<T, V>(out + r * out_h, p1[j], z);
            if (kBackward && p.first >= 0)
#pragma unroll
              for (int i = 0; i < V; ++i) dgain[kSum ? 0 : r][j][i] = both(f);
          }
          if (!kBackward && r == R - 1 && t + slots < a.tokens) angles(look(0));
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
        if (!kBackward && r == R - 1 && t + slots < a.tokens) angles(look(0));
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
      }
      if (!kAsync) {
        in += in_t;
        if (kBackward) go += go_t;
      }
      out += out_t;
      if constexpr (kAxes) {
        if (t + slots < a.tokens) p = look(n + 1);
        ++n;
      } else {
        p.first = next;
      }
      if (kBackward && t + slots < a.tokens) angles(p);
      if (!kAxes && t + 2 * slots < a.tokens) next = position(a, t + 2 * slots);
      at = at == kRing - 1 ? 0 : at + 1;
    }
  }

  if constexpr (kBackward) {
    if (!a.part) return;
    // The CTA's share of the gains' gradients: a group's sums to shared memory
    // (over the ring, which is done with), each column then added over the
    // groups in order.
    if constexpr (kAsync || kAxes) asm volatile("cp.async.wait_all;" ::: "memory");
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
#pragma unroll 8
          for (int k = lo; k < hi; ++k) s = __fadd_rn(s, s_part[(q * a.per + k) * a.dim + d]);
        to[kSum ? e : (row * R + r) * a.dim + d] = s;
      }
    }
  }
}

template <typename T, bool kInter, bool kBackward, bool kSum, bool kAxes>
const void* kernel_for(int v, int r) {
  if constexpr (sizeof(T) == 2)
    if (v == 8) {
      if constexpr (!kBackward)
        if (r == 4) return (const void*)qk_kernel<T, 8, 1, 4, kInter, kBackward, kSum, kAxes>;
      if constexpr (!kBackward || kSum)
        if (r == 2) return (const void*)qk_kernel<T, 8, 1, 2, kInter, kBackward, kSum, kAxes>;
      return (const void*)qk_kernel<T, 8, 1, 1, kInter, kBackward, kSum, kAxes>;
    }
  switch (v) {
    case 4:
      if constexpr (sizeof(T) == 4 && !kBackward)
        if (r == 2) return (const void*)qk_kernel<T, 4, 2, 2, kInter, kBackward, kSum, kAxes>;
      return (const void*)qk_kernel<T, 4, 2, 1, kInter, kBackward, kSum, kAxes>;
    case 2: return (const void*)qk_kernel<T, 2, 4, 1, kInter, kBackward, kSum, kAxes>;
    default: return (const void*)qk_kernel<T, 1, 8, 1, kInter, kBackward, kSum, kAxes>;
  }
}

template <typename T, bool kInter, bool kAxes>
const void* kernel_of(bool backward, bool sum, int v, int r) {
  if (!backward) return kernel_for<T, kInter, false, false, kAxes>(v, r);
  return sum ? kernel_for<T, kInter, true, true, kAxes>(v, r) : kernel_for<T, kInter, true, false, kAxes>(v, r);
}

template <typename T, bool kAxes>
const void* kernel_of(bool inter, bool backward, bool sum, int v, int r) {
  return inter ? kernel_of<T, true, kAxes>(backward, sum, v, r) : kernel_of<T, false, kAxes>(backward, sum, v, r);
}

template <bool kAxes>
const void* kernel_of(int32_t dtype, bool inter, bool backward, bool sum, int v, int r) {
  return dtype == ZERO_FP16   ? kernel_of<__half, kAxes>(inter, backward, sum, v, r)
         : dtype == ZERO_BF16 ? kernel_of<__nv_bfloat16, kAxes>(inter, backward, sum, v, r)
                              : kernel_of<float, kAxes>(inter, backward, sum, v, r);
}

}  // namespace zo
