// block_kernels.cuh -- a block's output joined to the residual stream with its
// norms, gate and dropout, forward and backward (zero_block.h).
//
// What bounds it: memory.  Each row is read once and each result written once;
// sums over a row are taken by the threads that hold it.  Measured on the device,
// 16,384 rows of 4096 in bf16: forward 82 us (97 % of the copy rate), with a norm of
// the branch 85 (93 %: two sums over the team a row, one after the other), backward 120
// and 126 (99 and 94 %, with the sums of the gains' gradients).  A dropout costs some
// 13 integer instructions a number (95 us forward, 152 backward with both norms, at two
// thirds of the issue slots).  A gate's sigmoid and its derivative cost less forward
// (8,192 rows 56 us, 89 %) than backward, where both are made twice (120 us, 66 %).
// Binary32, 8,192 rows: 93 us (86 %) and 139 (86 %).  Long rows have one CTA of sixteen
// warps an SM, and backward their registers spill: 2,048 rows of 16,384 in bf16 67 us
// (60 %) and 137 (43 %).  One row takes 2.8 us, backward 5.9 with its second kernel.
//
// Layout: a row of D numbers is cut into chunks of eight, and a team of whole
// warps takes a row at a time: thread i of n holds chunks i, i + n, ... (kC at
// most), the same columns of every row that it sees.  So the gains stay in
// registers, the gains' gradients are summed in registers until the end, and a
// chunk is one block of the dropout's generator.  The teams walk the tokens.
//
// Rows come by cp.async into a ring in shared memory in which every thread reads
// only what it copied itself, so that bytes in flight cost no registers and no
// barrier (kWide: rows of whole chunks on 16-byte boundaries; those of binary32
// are copied in the warp's order).  Of other rows the 16-byte granules that they
// lie in are copied, and a warp's lanes shift what they hold to where it belongs
// once it is there; results are shifted the other way, so that all but the ends of
// a warp's 256 numbers are written 16 bytes at a time (4,000 rows of 4097 in bf16 with
// both norms: 45 us forward, 96 backward, 43 and 30 % of the copy rate; number by
// number 76 and 171.  They take 56 and 86 thread instructions a number where aligned rows
// take 25 and 40, and have 17 and 9 warps an SM to run them: issue slots are 58 and 44 %
// used and no pipe more than that, so that it is work and latency together).
#pragma once

#include "numbers.cuh"
#include "philox.cuh"

namespace zo {

constexpr int kJoinThreads = 512;   // of a CTA, at most

struct JoinRow {
  char* data;
  int64_t stride;       // in bytes
  int64_t step;         // from a team's row to its next one, in bytes
};

struct JoinArgs {
  // forward: x, y, gate in; x_out, h out.  backward: x (the x' of the forward
  // pass), y, gate, dxo, dh in; dx, dy, dgate out.  An input that is absent is a
  // row of zeros for every token (the gate: NULL); a result that is: NULL.
  JoinRow x, y, gate, x_out, h, dxo, dh, dx, dy, dgate;
  const float* y_gain;
  const float* gain;
  const uint8_t* mask;
  float4* part;         // backward: [grid][2][2][chunks] partial gradients of y_gain and gain, the
                        // first and the last four numbers of every chunk, or NULL
  int64_t tokens;
  Drop drop;
  int32_t dim, chunks;
  int32_t warps, teams; // of a team; of a CTA
  int32_t ring, vecs;   // rows of the ring; 16-byte vectors of a thread in one
  int32_t gate_kind;
  float eps, eps_y, inv_dim, alpha, beta;
};

// A warp's bytes of a vector: 32 lanes' and, of rows that are shifted, one granule
// more (of two vectors' worth for the pair).
template <bool kWide> constexpr int kVecBytesOf = kWide ? 512 : 528;

template <typename E> constexpr int kVecs = (int)sizeof(E) / 2;   // 16-byte vectors of a chunk

// Waits until at most n of the thread's groups of copies are on their way.
__device__ __forceinline__ void copies_left(int n) {
  if (n >= 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
  else if (n == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
  else asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Words a, of which the first is `shift` bytes (a multiple of E's size, below 16)
// before what is wanted, moved down by that.
template <typename E, int kN>
__device__ __forceinline__ void move_down(uint32_t (&a)[kN], uint32_t shift) {
#pragma unroll
  for (int k = 0; k < kN - 2; ++k) a[k] = shift & 8 ? a[k + 2] : a[k];
#pragma unroll
  for (int k = 0; k < kN - 3; ++k) a[k] = shift & 4 ? a[k + 1] : a[k];
  if constexpr (sizeof(E) == 2)
#pragma unroll
    for (int k = 0; k < kN - 4; ++k) a[k] = __funnelshift_r(a[k], a[k + 1], shift % 4 * 8);
}

// The place of a thread in its team and in shared memory, and the moves between
// there and the rows.  A warp's vectors of a row lie one after another, so that
// each is a fixed distance from the row's first.
template <int kC, bool kWide>
struct Lane {
  int dim, chunks, warps;           // as in JoinArgs
  unsigned char* smem;    // the warp's ring
  int team, warp;         // this thread's team, and its warp's place in it
  static constexpr int kVecBytes = kVecBytesOf<kWide>;

  __device__ __forceinline__ int lanes() const { return warps * 32; }
  __device__ __forceinline__ int chunk(int j) const { return (j * warps + warp) * 32 + threadIdx.x % 32; }
  __device__ __forceinline__ bool live(int j) const { return chunk(j) < chunks; }
  // vector n of the thread in the row of the ring that begins at `at`
  __device__ __forceinline__ unsigned char* vec(int at, int n) const {
    return smem + at + n * kVecBytes + threadIdx.x % 32 * 16;
  }
  // Vector u of a warp's chunks of E whose vectors start at n.  Of binary32 a lane's
  // are 2 l and 2 l + 1: every other group of eight swaps neighbours, so that eight
  // lanes that read (or write) their first vectors, or their second, meet in no bank.
  template <typename E>
  __device__ __forceinline__ unsigned char* slot(int at, int n, uint32_t u) const {
    return smem + at + n * kVecBytes + (sizeof(E) == 2 ? u : u ^ (u >> 3 & 1)) * 16;
  }

  // Zeros in the warp's `bytes` of the ring, if some of its lanes have no chunk: what
  // is never copied to counts for nothing, and needs no check where it is read.
  __device__ __forceinline__ void clear(int bytes) const {
    if (((kC - 1) * warps + warp + 1) * 32 <= chunks) return;
    for (int at = threadIdx.x % 32 * 16; at < bytes; at += 512)
      *reinterpret_cast<uint4*>(smem + at) = make_uint4(0, 0, 0, 0);
    __syncwarp();
  }

  // A row's chunks into vectors from `first` on.
  template <typename E>
  __device__ __forceinline__ void fetch(const char* row, int at, int first) const {
    constexpr uint32_t kV = kVecs<E>;
    const uint32_t l = threadIdx.x % 32;
#pragma unroll
    for (int j = 0; j < kC; ++j) {
      if constexpr (kWide && kV == 1) {
        if (live(j)) copy16(vec(at, first + j), row + (uint32_t)chunk(j) * 16);
      } else if constexpr (kWide) {
        const uint32_t begin = (j * warps + warp) * 64;
#pragma unroll
        for (uint32_t u = l; u < 64; u += 32)
          if ((begin + u) * 4 < (uint32_t)dim) copy16(slot<E>(at, first + 2 * j, u), row + (begin + u) * 16);
      } else {
        // the granules that the warp's numbers lie in, as far as the row goes
        const uint32_t shift = reinterpret_cast<uintptr_t>(row) % 16, begin = (j * warps + warp) * (512 * kV);
        const int left = (int)(shift + dim * (uint32_t)sizeof(E) - begin);
        if (left <= (int)shift) continue;
        const char* from = row - shift + begin;
        if (left >= (int)(512 * kV + 16)) {      // not the row's last numbers
#pragma unroll
          for (uint32_t u = l; u < 32 * kV; u += 32) copy16(slot<E>(at, first + j * kV, u), from + 16 * u);
          if (l == 0 && shift) copy16(slot<E>(at, first + j * kV, 32 * kV), from + 512 * kV);
        } else {
#pragma unroll
          for (uint32_t u = l; u <= 32 * kV; u += 32) {
            const int bytes = left - 16 * (int)u;
            copy16(slot<E>(at, first + j * kV, u), bytes > 0 ? from + 16 * u : from, max(0, min(16, bytes)));
          }
        }
      }
    }
  }

  // The 16 bytes `shift` (even, below 16) behind an address on a 16-byte boundary.
  static __device__ __forceinline__ uint4 moved(const unsigned char* from, uint32_t shift) {
    uint32_t a[6];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const uint2 w = *reinterpret_cast<const uint2*>(from + (shift & 8) + 8 * k);
      a[2 * k] = w.x;
      a[2 * k + 1] = w.y;
    }
#pragma unroll
    for (int k = 0; k < 5; ++k) a[k] = shift & 4 ? a[k + 1] : a[k];
#pragma unroll
    for (int k = 0; k < 4; ++k) a[k] = __funnelshift_r(a[k], a[k + 1], shift % 4 * 8);
    return make_uint4(a[0], a[1], a[2], a[3]);
  }

  // Brings what was fetched from an address `shift` above a granule's to its lanes.
  template <typename E>
  __device__ __forceinline__ void settle(int at, int first, uint32_t shift) const {
    constexpr int kV = kVecs<E>;
    if (kWide || shift == 0) return;
    const uint32_t l = threadIdx.x % 32;
#pragma unroll
    for (int j = 0; j < kC; ++j) {
      if ((j * warps + warp) * 256 >= dim) continue;
      if constexpr (kV == 1) {
        unsigned char* const to = slot<E>(at, first + j, l);
        const uint4 w = moved(to, shift);
        __syncwarp();
        *reinterpret_cast<uint4*>(to) = w;
        continue;
      }
      uint32_t a[4 * kV + 4];
#pragma unroll
      for (int v = 0; v <= kV; ++v) {
        const uint4 w = *reinterpret_cast<const uint4*>(slot<E>(at, first + j * kV, l * kV + v));
        a[4 * v] = w.x;
        a[4 * v + 1] = w.y;
        a[4 * v + 2] = w.z;
        a[4 * v + 3] = w.w;
      }
      move_down<E>(a, shift);
      __syncwarp();
#pragma unroll
      for (int v = 0; v < kV; ++v)
        *reinterpret_cast<uint4*>(slot<E>(at, first + j * kV, l * kV + v)) =
            make_uint4(a[4 * v], a[4 * v + 1], a[4 * v + 2], a[4 * v + 3]);
    }
  }

  template <typename E>
  __device__ __forceinline__ void get(int at, int n, float2* x) const {
#pragma unroll
    for (int v = 0; v < kVecs<E>; ++v)
      unpack<E>(*reinterpret_cast<const uint4*>(slot<E>(at, n, threadIdx.x % 32 * kVecs<E> + v)),
                x + v * (8 / (int)sizeof(E)));
  }

  // The same with the dropped numbers zero.
  template <typename E>
  __device__ __forceinline__ void get(int at, int n, float2* x, const uint4& m) const {
    if constexpr (sizeof(E) == 2) {
      uint4 w = *reinterpret_cast<const uint4*>(vec(at, n));
      w = make_uint4(w.x & m.x, w.y & m.y, w.z & m.z, w.w & m.w);
      unpack<E>(w, x);
    } else {
      get<E>(at, n, x);
      mask8(x, m);
    }
  }

  // A chunk of a result.  What a lane does not write as it holds it passes through
  // the vectors from n on, which are done with, to be written in the warp's order.
  template <typename E>
  __device__ __forceinline__ void put(char* row, int j, const float2* x, int at, int n) const {
    constexpr uint32_t kV = kVecs<E>, kS = sizeof(E);
    const uint32_t l = threadIdx.x % 32;
    if constexpr (kWide && kV == 1) {
      if (live(j)) *reinterpret_cast<uint4*>(row + (uint32_t)chunk(j) * 16) = pack<E>(x);
      return;
    }
    const int begin = (j * warps + warp) * 256;
    if (begin >= dim) return;
    if (live(j))                   // what no number comes to stays zero
#pragma unroll
      for (uint32_t v = 0; v < kV; ++v)
        *reinterpret_cast<uint4*>(slot<E>(at, n, l * kV + v)) = pack<E>(x + v * (8 / kS));
    __syncwarp();
    char* to = row + (uint32_t)begin * kS;
    const uint32_t bytes = min(256, dim - begin) * kS;
    const uint32_t shift = kWide ? 0 : reinterpret_cast<uintptr_t>(to) % 16;
    // whole granules [16 u - shift, 16 u - shift + 16) of these bytes
    const int lo = shift ? 1 : 0, hi = (bytes + shift) / 16;
#pragma unroll
    for (uint32_t u = l; u < 32 * kV; u += 32) {
      if ((int)u < lo || (int)u >= hi) continue;
      uint4 w;
      if (kV == 1 && shift) w = moved(slot<E>(at, n, u - 1), 16 - shift);
      else if (kV == 1) w = pack<E>(x);
      else w = *reinterpret_cast<const uint4*>(slot<E>(at, n, u));
      if (!kWide && kV == 2 && shift) {
        const uint4 p = *reinterpret_cast<const uint4*>(slot<E>(at, n, u - 1));
        uint32_t a[8] = {p.x, p.y, p.z, p.w, w.x, w.y, w.z, w.w};
        move_down<E>(a, 16 - shift);
        w = make_uint4(a[0], a[1], a[2], a[3]);
      }
      *reinterpret_cast<uint4*>(to + 16 * u - shift) = w;
    }
    if constexpr (!kWide) {
      // the ends, number by number: those before the first whole granule, and behind the last
      const uint32_t number = l % 8 * kS, head = min(bytes, (16 - shift) % 16);
      const uint32_t rest = max(head, 16u * hi - min(16u * hi, shift));
      const uint32_t e = l < 8 ? number : rest + number;
      if (l < 16 && number < 16 && e < (l < 8 ? head : bytes))
        *reinterpret_cast<E*>(to + e) = *reinterpret_cast<const E*>(slot<E>(at, n, e / 16) + e % 16);
    }
    __syncwarp();
  }

  // A chunk of a gain (NULL: ones).
  __device__ __forceinline__ void gain(const float* g, int j, float2* x) const {
    const int left = min(8, dim - chunk(j) * 8);
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

  // Sums of kN numbers over the team's threads, in an order fixed by its size;
  // every thread gets them.  In a warp the numbers are spread over the lanes as
  // they are added, so that after log2(kP) steps each lane has one of them; the
  // warps' sums meet in shared memory.  `turn` alternates between two pieces of
  // it, so that one barrier a sum is enough: who writes a piece again has passed
  // the barrier of the sum between, which everyone reaches after reading the first.
  template <int kN>
  __device__ __forceinline__ void sum(float* x, float (*red)[kJoinThreads / 32 * 8], int& turn) const {
    constexpr int kP = kN <= 1 ? 1 : kN <= 2 ? 2 : 8, kGroup = 32 / kP;   // lanes of one number
    static_assert(kJoinThreads / 32 <= 16, "16 lanes take the warps' sums");
    const int l = threadIdx.x % 32;
    float v[kP];
#pragma unroll
    for (int i = 0; i < kP; ++i) v[i] = i < kN ? x[i] : 0.0f;
#pragma unroll
    for (int n = kP / 2, o = 16; n > 0; n /= 2, o /= 2) {
      const bool upper = l & o;
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const float send = upper ? v[i] : v[i + n];
        v[i] = __fadd_rn(upper ? v[i + n] : v[i], __shfl_xor_sync(0xffffffffu, send, o));
      }
    }
#pragma unroll
    for (int o = kGroup / 2; o > 0; o /= 2) v[0] = __fadd_rn(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
    if (warps > 1) {
      float* mine = red[turn] + team * warps * kP;
      if (l % kGroup == 0) mine[warp * kP + l / kGroup] = v[0];
      asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(lanes()) : "memory");
      constexpr int kTake = kGroup < 16 ? kGroup : 16;
      float s = 0.0f;
#pragma unroll
      for (int k = 0; k < 16; k += kTake) {
        const int w = k + l % kTake;
        if (w < warps) s = __fadd_rn(s, mine[w * kP + (kP == 1 ? 0 : l / kGroup)]);
      }
#pragma unroll
      for (int o = kTake / 2; o > 0; o /= 2) s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, o));
      v[0] = s;
      turn ^= 1;
    }
#pragma unroll
    for (int i = 0; i < kN; ++i) x[i] = kP == 1 ? v[0] : __shfl_sync(0xffffffffu, v[0], i * kGroup);
  }
};

// The gate's factor, in place, and the factor's derivative.  The sigmoid by
// e = exp(-|g|), so that neither it nor its derivative e / (1 + e)^2 is a
// difference of nearly equal numbers.  W is the widest type that the factor counts
// in: forward the stream's, backward the block's.  Where that has 16 bits e is the quick
// exponential, 2 + 1.2 |g| units in the last place of binary32 off at most, which is
// far below those types' steps wherever e counts beside 1 (and, in y_gain's gradient,
// below the errors of its sum over the tokens, but for gates far below zero).  16-bit
// blocks on a binary32 stream have the exact one and the quick reciprocal, two units off
// at most (8,192 rows of 4096 in bf16 on a binary32 stream, forward: 79 us with both
// quick, 81 so, 93 with the rounded reciprocal).
template <typename T, typename W>
__device__ __forceinline__ float sigmoid(float g, float* slope) {
  const float e = sizeof(W) == 2 ? __expf(-fabsf(g)) : expf(-fabsf(g));
  const float inv = sizeof(T) == 2 ? __fdividef(1.0f, __fadd_rn(1.0f, e)) : __frcp_rn(__fadd_rn(1.0f, e));
  const float low = __fmul_rn(e, inv);
  *slope = __fmul_rn(low, inv);
  return g >= 0.0f ? inv : low;
}

template <typename T, typename W>
__device__ __forceinline__ void act8(int kind, float2* g, float2* slope) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (kind == ZERO_GATE_SIGMOID)
      g[k] = make_float2(sigmoid<T, W>(g[k].x, &slope[k].x), sigmoid<T, W>(g[k].y, &slope[k].y));
    else
      slope[k] = both(1.0f);
  }
}

__device__ __forceinline__ float add2(float2 x) { return __fadd_rn(x.x, x.y); }

// What the branch has, besides a norm (kPost).
enum { kBare = 0, kDrop = 1, kGated = 2 };   // nothing; a dropout; either or both

// kMost: threads of a CTA at most.  Forward three CTAs of 256 threads are to fit an
// SM, or two of more where the rows are shifted.
template <typename T, typename S, int kC, bool kWide, bool kPost, int kHas, int kMost>
__global__ void __launch_bounds__(kMost, kMost == 256 ? 3 : kWide || (kC > 1 && kMost == 512) ? 1 : 2)
    join_kernel(const __grid_constant__ JoinArgs a) {
  extern __shared__ __align__(16) unsigned char s_ring[];
  __shared__ float s_red[2][kJoinThreads / 32 * 8];
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x / 32, 0);     // known to be the warp's
  const int row = a.vecs * kVecBytesOf<kWide>;                             // of the ring, a warp's
  const Lane<kC, kWide> me{a.dim, a.chunks, a.warps, s_ring + warp * a.ring * row, warp / a.warps, warp % a.warps};
  constexpr int kY = kC * kVecs<S>, kGate = kY + kC * kVecs<T>;   // vectors: x, y, gate
  constexpr bool kShared = !kWide || sizeof(S) == 4;   // lanes read what others of their warp copied
  const bool gated = kHas == kGated && a.gate.data, drops = kHas != kBare && a.drop.cut;
  const int64_t step = (int64_t)gridDim.x * a.teams;
  const int64_t first = (int64_t)blockIdx.x * a.teams + me.team;
  const int rows = first < a.tokens ? (int)((a.tokens - first + step - 1) / step) : 0;   // of this team
  const uint32_t rng_step = drops ? step_of(a.drop) : 0;
  const float scale = __fmul_rn(a.beta, a.drop.factor);

  // where the team's next rows are to be read, and its present ones written
  const char* x = a.x.data + first * a.x.stride;
  const char* y = a.y.data + first * a.y.stride;
  const char* gate = gated ? a.gate.data + first * a.gate.stride : nullptr;
  char* x_out = a.x_out.data + first * a.x_out.stride;
  char* h = a.h.data + first * a.h.stride;
  const uint8_t* mask = a.mask + first;
  int64_t block = first * a.chunks;         // of the generator
  const auto fetch = [&](bool on, int at) {
    if (on) {
      me.template fetch<S>(x, at, 0);
      me.template fetch<T>(y, at, kY);
      x += a.x.step;
      y += a.y.step;
      if (gated) {
        me.template fetch<T>(gate, at, kGate);
        gate += a.gate.step;
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // how far the present rows begin above a granule
  uint32_t ux = (uintptr_t)x % 16, uy = (uintptr_t)y % 16, ug = (uintptr_t)gate % 16;
  const auto settle = [&](int at) {
    if constexpr (!kWide) {
      me.template settle<S>(at, 0, ux);
      me.template settle<T>(at, kY, uy);
      if (gated) me.template settle<T>(at, kGate, ug);
      ux = (ux + (uint32_t)a.x.step) % 16;
      uy = (uy + (uint32_t)a.y.step) % 16;
      ug = (ug + (uint32_t)a.gate.step) % 16;
    }
  };
  // the gains stay in registers where there is room for them; columns that no lane
  // has are zeros from here on, which change no sum
  constexpr bool kKeep = kC <= 2;
  float2 yg_[kKeep ? kC : 1][4], g_[kKeep ? kC : 1][4];
  me.clear(a.ring * row);
  const int ahead = a.ring - 1;
  for (int k = 0; k < ahead; ++k) fetch(k < rows, k * row);
  if constexpr (kKeep)
#pragma unroll
    for (int j = 0; j < kC; ++j) {
      me.gain(a.y_gain, j, yg_[j]);
      me.gain(a.gain, j, g_[j]);
    }

  int at = 0, to = ahead * row, turn = 0;     // the rings' rows that are read, and copied to
  bool there = rows > 0 && (!a.mask || __ldg(mask));
  for (int i = 0; i < rows; ++i) {
    if (kShared) __syncwarp();     // all have read what is fetched over
    fetch(i + ahead < rows, to);
    bool next = true;
    if (a.mask && i + 1 < rows) next = __ldg(mask += step);
    uint4 keep[kHas == kBare ? 1 : kC];
    if (drops && there)
#pragma unroll
      for (int j = 0; j < kC; ++j) keep[j] = kept(a.drop, rng_step, block + me.chunk(j));
    copies_left(ahead);
    if (kShared) __syncwarp();
    settle(at);
    float2 v[kC][4];
    if (there) {
      float ry = scale;
      if constexpr (kPost) {
        float2 sq = both(0.0f);
#pragma unroll
        for (int j = 0; j < kC; ++j) {
          float2 b[4];
          me.template get<T>(at, kY + j * kVecs<T>, b);
#pragma unroll
          for (int k = 0; k < 4; ++k) sq = __ffma2_rn(b[k], b[k], sq);
        }
        float s = add2(sq);
        me.template sum<1>(&s, s_red, turn);
        ry = __fmul_rn(rsqrtf(__fmaf_rn(s, a.inv_dim, a.eps_y)), scale);
      }
      float2 sq = both(0.0f);
#pragma unroll
      for (int j = 0; j < kC; ++j) {
        float2 b[4], w[4];
        me.template get<S>(at, j * kVecs<S>, v[j]);
        me.template get<T>(at, kY + j * kVecs<T>, b);
        if constexpr (!kKeep) me.gain(a.y_gain, j, w);
#pragma unroll
        for (int k = 0; k < 4; ++k) b[k] = __fmul2_rn(__fmul2_rn(b[k], both(ry)), kKeep ? yg_[j][k] : w[k]);
        if (gated) {
          float2 g[4], slope[4];
          me.template get<T>(at, kGate + j * kVecs<T>, g);
          act8<T, S>(a.gate_kind, g, slope);
#pragma unroll
          for (int k = 0; k < 4; ++k) b[k] = __fmul2_rn(b[k], g[k]);
        }
        if (drops) mask8(b, keep[kHas == kBare ? 0 : j]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          v[j][k] = __ffma2_rn(v[j][k], both(a.alpha), b[k]);
        }
        // (a factor that is no number makes NaN of a zero that is no number of the row)
        if constexpr (!kWide) {
          const int left = a.dim - me.chunk(j) * 8;
          if (left < 8)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              v[j][k] = make_float2(2 * k < left ? v[j][k].x : 0.0f, 2 * k + 1 < left ? v[j][k].y : 0.0f);
        }
        if (me.live(j))
#pragma unroll
          for (int k = 0; k < 4; ++k) sq = __ffma2_rn(v[j][k], v[j][k], sq);
      }
      // a narrow result goes out through the places of what was read
      if (a.x_out.data) {
#pragma unroll
        for (int j = 0; j < kC; ++j) me.template put<S>(x_out, j, v[j], at, j * kVecs<S>);
      }
      if (a.h.data) {
        float s = add2(sq);
        me.template sum<1>(&s, s_red, turn);
        const float2 r = both(rsqrtf(__fmaf_rn(s, a.inv_dim, a.eps)));
#pragma unroll
        for (int j = 0; j < kC; ++j) {
          float2 w[4];
          if constexpr (!kKeep) me.gain(a.gain, j, w);
#pragma unroll
          for (int k = 0; k < 4; ++k) v[j][k] = __fmul2_rn(__fmul2_rn(v[j][k], r), kKeep ? g_[j][k] : w[k]);
          me.template put<T>(h, j, v[j], at, kY + j * kVecs<T>);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < kC; ++j) {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[j][k] = both(0.0f);
        if (a.x_out.data) me.template put<S>(x_out, j, v[j], at, j * kVecs<S>);
        if (a.h.data) me.template put<T>(h, j, v[j], at, kY + j * kVecs<T>);
      }
    }
    x_out += a.x_out.step;
    h += a.h.step;
    block += step * a.chunks;
    there = next;
    at = at + row == a.ring * row ? 0 : at + row;
    to = to + row == a.ring * row ? 0 : to + row;
  }
}

template <typename T, typename S, int kC, bool kWide, bool kPost, int kHas>
__global__ void __launch_bounds__(kJoinThreads) join_backward_kernel(const __grid_constant__ JoinArgs a) {
  extern __shared__ __align__(16) unsigned char s_ring[];
  __shared__ float s_red[2][kJoinThreads / 32 * 8];
  // the kernel that sums the partial gradients may be set up now; it waits for the end
  if (a.part) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x / 32, 0);     // known to be the warp's
  const int row = a.vecs * kVecBytesOf<kWide>;                             // of the ring, a warp's
  const Lane<kC, kWide> me{a.dim, a.chunks, a.warps, s_ring + warp * a.ring * row, warp / a.warps, warp % a.warps};
  // vectors: x', dx', dh, y, gate
  constexpr int kDxo = kC * kVecs<S>, kDh = 2 * kDxo, kY = kDh + kC * kVecs<T>, kGate = kY + kC * kVecs<T>;
  constexpr bool kShared = !kWide || sizeof(S) == 4;   // lanes read what others of their warp copied
  const bool gated = kHas == kGated && a.gate.data, drops = kHas != kBare && a.drop.cut;
  const int64_t step = (int64_t)gridDim.x * a.teams;
  const int64_t first = (int64_t)blockIdx.x * a.teams + me.team;
  const int rows = first < a.tokens ? (int)((a.tokens - first + step - 1) / step) : 0;
  const uint32_t rng_step = drops ? step_of(a.drop) : 0;
  const float scale = __fmul_rn(a.beta, a.drop.factor);

  const char* x = a.x.data + first * a.x.stride;
  const char* dxo = a.dxo.data + first * a.dxo.stride;
  const char* dh = a.dh.data + first * a.dh.stride;
  const char* y = a.y.data + first * a.y.stride;
  const char* gate = gated ? a.gate.data + first * a.gate.stride : nullptr;
  char* dx = a.dx.data + first * a.dx.stride;
  char* dy = a.dy.data + first * a.dy.stride;
  char* dgate = gated ? a.dgate.data + first * a.dgate.stride : nullptr;
  const uint8_t* mask = a.mask + first;
  int64_t block = first * a.chunks;
  const auto fetch = [&](bool on, int at) {
    if (on) {
      me.template fetch<S>(x, at, 0);
      me.template fetch<S>(dxo, at, kDxo);
      me.template fetch<T>(dh, at, kDh);
      me.template fetch<T>(y, at, kY);
      x += a.x.step;
      dxo += a.dxo.step;
      dh += a.dh.step;
      y += a.y.step;
      if (gated) {
        me.template fetch<T>(gate, at, kGate);
        gate += a.gate.step;
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  uint32_t ux = (uintptr_t)x % 16, uo = (uintptr_t)dxo % 16, uh = (uintptr_t)dh % 16, uy = (uintptr_t)y % 16,
           ug = (uintptr_t)gate % 16;
  const auto settle = [&](int at) {
    if constexpr (!kWide) {
      me.template settle<S>(at, 0, ux);
      me.template settle<S>(at, kDxo, uo);
      me.template settle<T>(at, kDh, uh);
      me.template settle<T>(at, kY, uy);
      if (gated) me.template settle<T>(at, kGate, ug);
      ux = (ux + (uint32_t)a.x.step) % 16;
      uo = (uo + (uint32_t)a.dxo.step) % 16;
      uh = (uh + (uint32_t)a.dh.step) % 16;
      uy = (uy + (uint32_t)a.y.step) % 16;
      ug = (ug + (uint32_t)a.gate.step) % 16;
    }
  };
  constexpr bool kKeep = kC <= 2;
  float2 yg_[kKeep ? kC : 1][4], g_[kKeep ? kC : 1][4];
  me.clear(a.ring * row);
  const int ahead = a.ring - 1;
  for (int k = 0; k < ahead; ++k) fetch(k < rows, k * row);
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

  int at = 0, to = ahead * row, turn = 0;     // the rings' rows that are read, and copied to
  bool there = rows > 0 && (!a.mask || __ldg(mask));
  for (int i = 0; i < rows; ++i) {
    if (kShared) __syncwarp();     // all have read what is fetched over
    fetch(i + ahead < rows, to);
    bool next = true;
    if (a.mask && i + 1 < rows) next = __ldg(mask += step);
    uint4 keep[kHas == kBare ? 1 : kC];
    if (drops && there)
#pragma unroll
      for (int j = 0; j < kC; ++j) keep[j] = kept(a.drop, rng_step, block + me.chunk(j));
    copies_left(ahead);
    if (kShared) __syncwarp();
    settle(at);
    if (there) {
      // With q = act y_gain y where the branch is kept, the branch's own dot product
      // sum G q is linear in G, so that its parts are summed before r is known: one
      // sum over the team a row.
      float2 s2[kPost ? 6 : 2];
#pragma unroll
      for (int k = 0; k < (kPost ? 6 : 2); ++k) s2[k] = both(0.0f);
#pragma unroll
      for (int j = 0; j < kC; ++j) {
        float2 xv[4], d[4], w[4];
        me.template get<S>(at, j * kVecs<S>, xv);
        me.template get<T>(at, kDh + j * kVecs<T>, d);
        if constexpr (!kKeep) me.gain(a.gain, j, w);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          d[k] = __fmul2_rn(d[k], kKeep ? g_[j][k] : w[k]);
          s2[0] = __ffma2_rn(xv[k], xv[k], s2[0]);
          s2[1] = __ffma2_rn(d[k], xv[k], s2[1]);
        }
        if constexpr (kPost) {
          float2 q[4], o[4];
          me.template get<T>(at, kY + j * kVecs<T>, q);
#pragma unroll
          for (int k = 0; k < 4; ++k) s2[2] = __ffma2_rn(q[k], q[k], s2[2]);
          // What is dropped may be anything.  (Of x' and dh not: one of their numbers
          // that is not finite is in every number of G, by the norm's mean; one of y's
          // makes its own place of the norm's gradient NaN.)
          if (drops) {
            me.template get<T>(at, kY + j * kVecs<T>, q, keep[kHas == kBare ? 0 : j]);
            me.template get<S>(at, kDxo + j * kVecs<S>, o, keep[kHas == kBare ? 0 : j]);
          } else {
            me.template get<S>(at, kDxo + j * kVecs<S>, o);
          }
          if constexpr (!kKeep) me.gain(a.y_gain, j, w);
#pragma unroll
          for (int k = 0; k < 4; ++k) q[k] = __fmul2_rn(q[k], kKeep ? yg_[j][k] : w[k]);
          if (gated) {
            float2 g[4], slope[4];
            me.template get<T>(at, kGate + j * kVecs<T>, g);
            act8<T, T>(a.gate_kind, g, slope);
#pragma unroll
            for (int k = 0; k < 4; ++k) q[k] = __fmul2_rn(q[k], g[k]);
            if (drops) mask8(q, keep[kHas == kBare ? 0 : j]);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            s2[3] = __ffma2_rn(o[k], q[k], s2[3]);
            s2[4] = __ffma2_rn(d[k], q[k], s2[4]);
            s2[5] = __ffma2_rn(xv[k], q[k], s2[5]);
          }
        }
      }
      float s[kPost ? 6 : 2];
#pragma unroll
      for (int k = 0; k < (kPost ? 6 : 2); ++k) s[k] = add2(s2[k]);
      me.template sum<kPost ? 6 : 2>(s, s_red, turn);
      // G = dx' + r (dn - xhat mean(dn xhat)), dn = dh gain: no power of r but the
      // first, so that it holds for rows of any size
      const float r = rsqrtf(__fmaf_rn(s[0], a.inv_dim, a.eps));
      const float back = __fmul_rn(-r, __fmul_rn(__fmul_rn(r, s[1]), a.inv_dim));
      float ry = 1.0f, back_y = 0.0f;
      if constexpr (kPost) {
        ry = rsqrtf(__fmaf_rn(s[2], a.inv_dim, a.eps_y));
        const float dot = __fmul_rn(scale, __fmaf_rn(back, __fmul_rn(r, s[5]), __fmaf_rn(r, s[4], s[3])));
        float hat = __fmul_rn(ry, dot);
        // Products of x', dx' and q, which no norm has scaled, may leave binary32's range
        // though each row's squares do not.  Of rows far from order one the sums are taken
        // again, of xhat and yhat (all threads of the team see the same r and ry).  Four
        // chunks in a loop, with the bits made again, which leaves their other registers as
        // they were.
        if (!(fminf(r, ry) > 0x1p-20f && fmaxf(r, ry) < 0x1p20f)) {
          float2 t[3] = {both(0.0f), both(0.0f), both(0.0f)};
          constexpr int kUnroll = kKeep ? kC : 1;
#pragma unroll kUnroll
          for (int j = 0; j < kC; ++j) {
            float2 v[4], q[4], w[4];
            uint4 m = make_uint4(~0u, ~0u, ~0u, ~0u);
            if (drops) m = kKeep ? keep[kHas == kBare ? 0 : j] : kept(a.drop, rng_step, block + me.chunk(j));
            me.template get<T>(at, kY + j * kVecs<T>, q, m);
            if constexpr (!kKeep) me.gain(a.y_gain, j, w);
#pragma unroll
            for (int k = 0; k < 4; ++k) q[k] = __fmul2_rn(__fmul2_rn(q[k], both(ry)), kKeep ? yg_[j][k] : w[k]);
            if (gated) {
              me.template get<T>(at, kGate + j * kVecs<T>, v);
              act8<T, T>(a.gate_kind, v, w);
#pragma unroll
              for (int k = 0; k < 4; ++k) q[k] = __fmul2_rn(q[k], v[k]);
              mask8(q, m);
            }
            me.template get<S>(at, kDxo + j * kVecs<S>, v, m);
#pragma unroll
            for (int k = 0; k < 4; ++k) t[0] = __ffma2_rn(v[k], q[k], t[0]);
            me.template get<T>(at, kDh + j * kVecs<T>, v);
            if constexpr (!kKeep) me.gain(a.gain, j, w);
#pragma unroll
            for (int k = 0; k < 4; ++k) t[1] = __ffma2_rn(__fmul2_rn(v[k], kKeep ? g_[j][k] : w[k]), q[k], t[1]);
            me.template get<S>(at, j * kVecs<S>, v);
#pragma unroll
            for (int k = 0; k < 4; ++k) t[2] = __ffma2_rn(__fmul2_rn(v[k], both(r)), q[k], t[2]);
          }
          float u[3] = {add2(t[0]), add2(t[1]), add2(t[2])};
          me.template sum<3>(u, s_red, turn);
          hat = __fmul_rn(scale, __fmaf_rn(back, u[2], __fmaf_rn(r, u[1], u[0])));
        }
        back_y = __fmul_rn(-ry, __fmul_rn(hat, a.inv_dim));
      }
#pragma unroll
      for (int j = 0; j < kC; ++j) {
        float2 G[4], o[4], slope[4];
        {
          float2 xv[4], d[4], w[4];
          me.template get<S>(at, j * kVecs<S>, xv);
          me.template get<T>(at, kDh + j * kVecs<T>, d);
          me.template get<S>(at, kDxo + j * kVecs<S>, G);
          if constexpr (!kKeep) me.gain(a.gain, j, w);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 xhat = __fmul2_rn(xv[k], both(r));
            dg[j][k] = __ffma2_rn(d[k], xhat, dg[j][k]);
            const float2 dn = __fmul2_rn(d[k], kKeep ? g_[j][k] : w[k]);
            G[k] = __fadd2_rn(G[k], __ffma2_rn(dn, both(r), __fmul2_rn(xhat, both(back))));
            o[k] = __fmul2_rn(G[k], both(a.alpha));
          }
        }
        if (a.dx.data) me.template put<S>(dx, j, o, at, j * kVecs<S>);
        {
          float2 yv[4], g[4], w[4];
          if (!kPost && drops) me.template get<T>(at, kY + j * kVecs<T>, yv, keep[kHas == kBare ? 0 : j]);
          else me.template get<T>(at, kY + j * kVecs<T>, yv);
          if (gated) {
            me.template get<T>(at, kGate + j * kVecs<T>, g);
            act8<T, T>(a.gate_kind, g, slope);
          }
          if constexpr (!kKeep) me.gain(a.y_gain, j, w);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            G[k] = __fmul2_rn(G[k], both(scale));       // db
            if constexpr (kPost) {
              yv[k] = __fmul2_rn(yv[k], both(ry));
              o[k] = __fmul2_rn(yv[k], both(back_y));
            }
          }
          if (drops) {
            const uint4& m = keep[kHas == kBare ? 0 : j];
            mask8(G, m);
            if (gated) {
              mask8(g, m);
              mask8(slope, m);
            }
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 yg = kKeep ? yg_[j][k] : w[k];
            if (gated) {
              slope[k] = __fmul2_rn(__fmul2_rn(__fmul2_rn(G[k], slope[k]), yv[k]), yg);
              G[k] = __fmul2_rn(G[k], g[k]);
            }
            dyg[j][k] = __ffma2_rn(G[k], yv[k], dyg[j][k]);
            G[k] = __fmul2_rn(G[k], yg);
            o[k] = kPost ? __ffma2_rn(G[k], both(ry), o[k]) : G[k];
          }
        }
        if (a.dy.data) me.template put<T>(dy, j, o, at, kY + j * kVecs<T>);
        if (gated && a.dgate.data) me.template put<T>(dgate, j, slope, at, kY + j * kVecs<T>);
      }
    } else {
      const float2 zero[4] = {both(0.0f), both(0.0f), both(0.0f), both(0.0f)};
#pragma unroll
      for (int j = 0; j < kC; ++j) {
        if (a.dx.data) me.template put<S>(dx, j, zero, at, j * kVecs<S>);
        if (a.dy.data) me.template put<T>(dy, j, zero, at, kY + j * kVecs<T>);
        if (gated && a.dgate.data) me.template put<T>(dgate, j, zero, at, kY + j * kVecs<T>);
      }
    }
    dx += a.dx.step;
    dy += a.dy.step;
    if (gated) dgate += a.dgate.step;
    block += step * a.chunks;
    there = next;
    at = at + row == a.ring * row ? 0 : at + row;
    to = to + row == a.ring * row ? 0 : to + row;
  }

  // The CTA's share of the gains' gradients: its teams' one after the other, in
  // shared memory as in `part`, where the lanes of a warp are next to one another.
  if (!a.part) return;
  float4* const part = a.part + (int64_t)blockIdx.x * 4 * a.chunks;
  float4* const s_sum = reinterpret_cast<float4*>(s_ring);
  asm volatile("cp.async.wait_all;" ::: "memory");
  for (int team = 0; team < a.teams; ++team) {
    __syncthreads();
    if (me.team != team) continue;
    float4* const out = team == a.teams - 1 ? part : s_sum;
#pragma unroll
    for (int j = 0; j < kC; ++j) {
      if (!me.live(j)) continue;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2* d = (k < 2 ? dyg[j] : dg[j]) + k % 2 * 2;
        const int at = k * a.chunks + me.chunk(j);
        float4 v = make_float4(d[0].x, d[0].y, d[1].x, d[1].y);
        if (team > 0) {
          const float4 o = s_sum[at];
          v = make_float4(__fadd_rn(o.x, v.x), __fadd_rn(o.y, v.y), __fadd_rn(o.z, v.z), __fadd_rn(o.w, v.w));
        }
        out[at] = v;
      }
    }
  }
}

}  // namespace zo
