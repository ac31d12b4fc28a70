// muon_resident.cuh -- matrices with a side of at most 128 and the other of at
// most 2048, orthogonalised without leaving the chip.
//
// What bounds them is latency: fifteen dependent products of a few hundred
// cycles each, which through global memory take two to five microseconds
// apiece.  Here a cluster of one to eight CTAs holds the matrix from its input
// to its result, each CTA up to kCols columns of X (k rows, k <= 128; a tall
// matrix is held transposed):
//   X       binary32 in registers, a thread a row and kCols / 4 columns;
//           binary16 in shared memory as an operand (H)
//   A, B    in shared memory as an operand, one over the other in a single CTA
// A step is three products of the CTA's own operands, accumulated in TMEM:
//   A = H H^T over the CTA's columns, added up over the cluster by copies
//       between the CTAs (each number once, so that every CTA has the same
//       bits), its diagonal kept in binary32 (muon_products.cuh);
//   B = b A + c A A, in every CTA alike;   X <- a X + B H.
// Measured, a call through the workspace and here: 64x64 49 and 24 us, 32 of
// 128x1024 95 and 61 us.  A step is a chain of three products and their
// epilogues, 4 us, or 6 with 256 columns a CTA, and 10 with a cluster's sums; the
// tensor cores work for 7 % of the cycles.
#pragma once

#include "muon_products.cuh"

namespace zm {

constexpr int kResidentThreads = 512;
constexpr int kResidentSide = 128;       // the shorter side's most
constexpr int kResidentSpan = 8;         // CTAs a cluster at most

struct Resident {
  int32_t first, n, unit0;     // entries of the launch, and their first matrix
  int32_t span;                // CTAs a matrix
  int32_t steps, head;         // head: the call's first launch
  int32_t inject;              // test hook: the products' end is not announced
  float coef[ZERO_MUON_MAX_STEPS][3];
};

template <int kCols>
constexpr int resident_bytes(int span) {
  return 128 * kCols * 2 + 128 * 128 * 2 + 1024 + (span > 1 ? 2 * 128 * 128 * 4 : 0);
}

// Four numbers of a row (fewer at its end, the rest zero) from p, and back.
template <typename T>
__device__ __forceinline__ float4 load4(const T* p, int n, bool vec) {
  if (vec && n >= 4) {
    if constexpr (sizeof(T) == 4) {
      return *reinterpret_cast<const float4*>(p);
    } else {
      const uint2 u = *reinterpret_cast<const uint2*>(p);
      const T* t = reinterpret_cast<const T*>(&u);
      return make_float4(num<T>(t[0]), num<T>(t[1]), num<T>(t[2]), num<T>(t[3]));
    }
  }
  return make_float4(n > 0 ? num<T>(p[0]) : 0.0f, n > 1 ? num<T>(p[1]) : 0.0f, n > 2 ? num<T>(p[2]) : 0.0f,
                     n > 3 ? num<T>(p[3]) : 0.0f);
}
template <typename T>
__device__ __forceinline__ void store4(T* p, int n, bool vec, float4 x) {
  if (vec && n >= 4) {
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float4*>(p) = x;
    } else {
      uint2 u;
      T* t = reinterpret_cast<T*>(&u);
      t[0] = as<T>(x.x); t[1] = as<T>(x.y); t[2] = as<T>(x.z); t[3] = as<T>(x.w);
      *reinterpret_cast<uint2*>(p) = u;
    }
    return;
  }
  if (n > 0) p[0] = as<T>(x.x);
  if (n > 1) p[1] = as<T>(x.y);
  if (n > 2) p[2] = as<T>(x.z);
  if (n > 3) p[3] = as<T>(x.w);
}
__device__ __forceinline__ bool fits4(const void* p, int64_t row, int64_t batch, int esize) {
  return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(row * esize) | (uintptr_t)(batch * esize)) &
          (uintptr_t)(4 * esize - 1)) == 0;
}

// A warp's 32 x 32 binary32 numbers in shared memory, 16-byte pieces of a row
// in an order of the row's own.
__device__ __forceinline__ float4* cell(float* patch, int r, int piece) {
  return reinterpret_cast<float4*>(patch) + r * 8 + (piece ^ (r & 7));
}

// The result of four numbers of a row: O, or the step with it.
__device__ __forceinline__ void finish4(const Call& c, const Entry& e, const Io& io, int b, int row, int col, int n,
                                        bool vout, bool vmaster, float4 o) {
  const int64_t at = (int64_t)b * io.out_batch + (int64_t)row * io.out_row + col;
  if (c.step) {
    float4 w;
    if (io.master) w = load4<float>(io.master + at, n, vmaster);
    else if (c.out_type == ZERO_FP16) w = load4<__half>(static_cast<const __half*>(io.out) + at, n, vout);
    else w = load4<__nv_bfloat16>(static_cast<const __nv_bfloat16*>(io.out) + at, n, vout);
    const float step = -__fmul_rn(c.lr, e.s);
    o.x = __fmaf_rn(step, o.x, __fmul_rn(w.x, c.decay));
    o.y = __fmaf_rn(step, o.y, __fmul_rn(w.y, c.decay));
    o.z = __fmaf_rn(step, o.z, __fmul_rn(w.z, c.decay));
    o.w = __fmaf_rn(step, o.w, __fmul_rn(w.w, c.decay));
    if (io.master) store4<float>(io.master + at, n, vmaster, o);
  }
  if (c.out_type == ZERO_FP16) store4<__half>(static_cast<__half*>(io.out) + at, n, vout, o);
  else if (c.out_type == ZERO_BF16) store4<__nv_bfloat16>(static_cast<__nv_bfloat16*>(io.out) + at, n, vout, o);
  else store4<float>(static_cast<float*>(io.out) + at, n, vout, o);
}

// Takes A's diagonal, if it is there, out of columns `col`.. of row r.
template <int N>
__device__ __forceinline__ void take_diagonal(float* v, int r, int col, float* diag) {
  float d = 0.0f;
#pragma unroll
  for (int q = 0; q < N; ++q) {
    d = q == r - col ? v[q] : d;
    v[q] = q == r - col ? 0.0f : v[q];
  }
  if (r >= col && r < col + N) diag[r] = __fmul_rn(d, 1.0f / kScale);
}

// kPerSm: CTAs an SM, 2 with 128 columns for more matrices than SMs.  One has
// twice the registers: 64x64 24 us against 27, a hundred 100x100 27 against 31,
// but 400 of them 74 against 64.
template <typename T, int kCols, int kPerSm, int N>
__global__ void __launch_bounds__(kResidentThreads, kPerSm)
    muon_resident_kernel(const __grid_constant__ Resident p, const __grid_constant__ Start<N> s) {
  constexpr int kChunks = kCols / 128;            // 32 columns each, of a thread's
  constexpr uint32_t kTmem = kCols == 128 ? 256 : 512;
  extern __shared__ __align__(1024) unsigned char base[];
  const Call& c = s.c;
  if (p.head && blockIdx.x == 0 && threadIdx.x == 0) {
    c.ws->skipped = skipped(c);
    if (skipped(c)) c.ws->last = 0;
  }
  if (skipped(c)) return;
  const int warp = uniform(threadIdx.x / 32), lane = threadIdx.x % 32;
  const int quarter = warp % 4, part = warp / 4;
  const uint32_t rank = p.span > 1 ? cluster_rank() : 0;
  unsigned char* small = base + 128 * kCols * 2 + 128 * 128 * 2;
  float* diag = reinterpret_cast<float*>(small);                        // 128
  double* red = reinterpret_cast<double*>(small + 512);                 // 16 warps' sums, then the CTA's
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(small + 768);
  const uint32_t bar = smem_u32(small + 784);
  const uint32_t shares = bar + 8, totals = bar + 16;                   // barriers of the cluster's sums
  const uint32_t drain = bar + 24, failed = bar + 32;                   // failed: a wait of the cluster's has run out
  float* sums = reinterpret_cast<float*>(small + 1024);                 // A's share, for the cluster; then B
  float* patch = reinterpret_cast<float*>(base) + warp * 1024;          // over both operands, before and after
  const uint32_t x_at = smem_u32(base), a_at = x_at + 128 * kCols * 2;
  int* fault = &c.ws->fault;

  // the matrix of this cluster
  __shared__ int found;
  const int unit = p.unit0 + blockIdx.x / p.span;
  for (int i = threadIdx.x; i < p.n; i += kResidentThreads) {
    const Entry& q = c.entries[p.first + i];
    if (unit >= q.unit0 && unit < q.unit0 + q.batch) found = p.first + i;
  }
  if (threadIdx.x == 0) {
    mbar_init(bar, 1);
    mbar_init(shares, 1);
    mbar_init(totals, 1);
    mbar_init(drain, 1);
    *(volatile int*)(small + 816) = 0;
    mbar_init_fence();
  }
  if (warp == 0) tmem_alloc<1>(smem_u32(tmem_at), kTmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_at, acc_a = tmem + kCols;
  const Entry e = c.entries[found];
  const Io& io = s.io[e.item];
  const int b = unit - e.unit0;
  const int row = quarter * 32 + lane;

  // ---- input: by rows of the caller's arrays, through the patch to a row of X a thread
  float x[kChunks][32];
  {
    const T* in = static_cast<const T*>(io.in) + (int64_t)b * io.in_batch;
    float* mom = c.step ? io.mom + (int64_t)b * e.rows * e.cols : nullptr;
    const bool vin = fits4(io.in, io.in_row, io.in_batch, sizeof(T));
    const bool vmom = c.step && fits4(io.mom, e.cols, (int64_t)e.rows * e.cols, 4);
    const float f = grad_factor(c);
    float sq = 0.0f;
#pragma unroll
    for (int h = 0; h < kChunks; ++h) {
      const int j0 = (int)rank * kCols + (part + 4 * h) * 32, i0 = quarter * 32;
      const int top = e.tall ? j0 : i0, left = e.tall ? i0 : j0;
#pragma unroll 4
      for (int q = 0; q < 8; ++q) {
        const int r = q * 4 + lane / 8, cc = lane % 8 * 4;
        const int n = top + r < e.rows ? e.cols - left - cc : 0;
        const float4 g = load4<T>(in + (int64_t)(top + r) * io.in_row + left + cc, n, vin);
        float u[4] = {g.x, g.y, g.z, g.w};
        if (c.step) {
          float* pm = mom + (int64_t)(top + r) * e.cols + left + cc;
          const float4 m4 = load4<float>(pm, n, vmom);
          float m[4] = {m4.x, m4.y, m4.z, m4.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float gi = __fmul_rn(u[k], f);
            m[k] = __fadd_rn(__fmul_rn(c.mu, m[k]), gi);
            u[k] = c.nesterov ? __fadd_rn(gi, __fmul_rn(c.mu, m[k])) : m[k];
          }
          store4<float>(pm, n, vmom, make_float4(m[0], m[1], m[2], m[3]));
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) sq = __fmaf_rn(u[k], u[k], sq);
        *cell(patch, r, lane % 8) = make_float4(u[0], u[1], u[2], u[3]);
      }
      __syncwarp();
      if (e.tall) {
#pragma unroll
        for (int k = 0; k < 32; ++k)
          x[h][k] = reinterpret_cast<const float*>(cell(patch, k, lane / 4))[lane % 4];
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) reinterpret_cast<float4*>(x[h])[k] = *cell(patch, lane, k);
      }
      __syncwarp();
    }
    double d = sq;
    for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    if (lane == 0) red[warp] = d;
    __syncthreads();
    d = 0.0;
    for (int i = 0; i < kResidentThreads / 32; ++i) d += red[i];
    if (p.span > 1) {
      if (threadIdx.x == 0) red[16] = d;
      cluster_sync();
      d = 0.0;
      for (int r = 0; r < p.span; ++r) {
        double v;
        asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(peer(smem_u32(red + 16), r)) : "memory");
        d += v;
      }
    }
    const float inv = inverse(d, c.eps);
#pragma unroll
    for (int h = 0; h < kChunks; ++h)
#pragma unroll
      for (int k = 0; k < 32; ++k) x[h][k] = __fmul_rn(__fmul_rn(x[h][k], inv), kScaleX);
  }
  // the operand of products: piece of eight columns, 128 rows of 16 bytes
  const auto put = [&](unsigned char* to, int piece, const float* v) {
    *reinterpret_cast<uint4*>(to + piece * 2048 + row * 16) =
        make_uint4(pack(v[0], v[1]), pack(v[2], v[3]), pack(v[4], v[5]), pack(v[6], v[7]));
  };
  const auto put_x = [&] {
#pragma unroll
    for (int h = 0; h < kChunks; ++h)
#pragma unroll
      for (int q = 0; q < 4; ++q) put(base, (part + 4 * h) * 4 + q, x[h] + 8 * q);
  };
  uint32_t phase = 0, sum_phase = 0;
  bool ok = true;                      // no wait of this thread's has run out
  // What threads wrote to shared memory is there for products and copies.
  const auto written = [&] {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    tc_fence_before();
    __syncthreads();
  };
  // Its threads come out of a wait one by one, and what follows is for whole warps.
  const auto wait = [&](uint32_t at, uint32_t parity) {
    ok = ok && mbar_wait(at, parity, fault);
    __syncwarp();
  };
  // Issues products once every thread's operand is written, waits for them.  The
  // issuing thread goes by its own waits: where they were met, what it issued
  // before is over.  After one that ran out it issues nothing more, and no thread
  // waits again once it has given up: the steps that are left pass in no time, on
  // numbers that nobody uses (leaving them by a vote at each barrier cost 64x64
  // a microsecond).
  const auto products = [&](auto issue) {
    written();
    if (warp == 0) {
      tc_fence_after();
      if (elected() && ok) {
        issue();
        if (!p.inject) mma_commit<1>(bar);
      }
      __syncwarp();
    }
    wait(bar, phase);
    phase ^= 1;
    tc_fence_after();
  };

  // A from the CTAs' shares of it (32 columns of a row a thread).  Every CTA adds
  // up some columns, whose shares the others send it in binary32, and sends them
  // the operand and the diagonal that come of it.  Both ways are bulk copies, and
  // what bounds them is the bytes between SMs (loads and stores of each other's
  // memory by the threads, binary32 both ways: 32 of 128x1024 67 us; copies: 63;
  // the operand back: 61).  What a copy overwrites has been read: a CTA sends
  // its next share after its last product, and an operand after it has all shares.
  // What a copy reads stays until it has read it.  The shares: every CTA sends its
  // totals after it has all shares, so when the totals are here nobody reads `own`.
  // The operand and the diagonal: that a CTA has the others' totals says nothing of
  // its own on their way out; those have arrived when the next shares have, and
  // until then neither is written.  So B goes over `own`, not over A.
  const auto add_up = [&](const float* v) {
    float4 *own = reinterpret_cast<float4*>(sums), *theirs = own + 4096;
    const uint32_t pieces = 4096 / p.span, mine = 16 / p.span;   // of four columns, of eight
    unsigned char* const a = base + 128 * kCols * 2;
#pragma unroll
    for (int q = 0; q < 8; ++q)
      own[(part * 8 + q) * 128 + row] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
    written();
    if (warp == 0) {
      if (elected() && ok) {
        mbar_expect(shares, (p.span - 1) * pieces * 16);
        mbar_expect(totals, (p.span - 1) * (mine * 2048 + mine * 32));
        for (int r = 1; r < p.span; ++r) {
          const uint32_t to = (rank + r) % p.span;
          copy_to_peer(peer(smem_u32(theirs + rank * pieces), to), smem_u32(own + to * pieces), pieces * 16,
                       peer(shares, to));
        }
      }
      __syncwarp();
    }
    wait(shares, sum_phase);
    for (int i = threadIdx.x; i < (int)mine * 128; i += kResidentThreads) {
      const int at = i / 128, r = i % 128;       // a row of eight columns
      float t[8];
#pragma unroll
      for (int h = 0; h < 2; ++h)
        reinterpret_cast<float4*>(t)[h] = own[rank * pieces + (2 * at + h) * 128 + r];
#pragma unroll
      for (int k = 1; k < kResidentSpan; ++k)
        if (k < p.span) {
          const float4* from = theirs + (rank + k) % p.span * pieces + 2 * at * 128 + r;
          const float4 y = from[0], z = from[128];
          const float u[8] = {y.x, y.y, y.z, y.w, z.x, z.y, z.z, z.w};
#pragma unroll
          for (int q = 0; q < 8; ++q) t[q] = __fadd_rn(t[q], u[q]);
        }
      const int piece = rank * mine + at;
      take_diagonal<8>(t, r, piece * 8, diag);
      *reinterpret_cast<uint4*>(a + piece * 2048 + r * 16) =
          make_uint4(pack(t[0], t[1]), pack(t[2], t[3]), pack(t[4], t[5]), pack(t[6], t[7]));
    }
    written();
    if (warp == 0) {
      if (elected() && ok) {
        const uint32_t from = smem_u32(a) + rank * mine * 2048, from_d = smem_u32(diag) + rank * mine * 32;
        for (int r = 1; r < p.span; ++r) {
          const uint32_t to = (rank + r) % p.span;
          copy_to_peer(peer(from, to), from, mine * 2048, peer(totals, to));
          copy_to_peer(peer(from_d, to), from_d, mine * 32, peer(totals, to));
        }
      }
      __syncwarp();
    }
    wait(totals, sum_phase);
    sum_phase ^= 1;
  };

  // where B goes: over A, or over this CTA's share of it
  unsigned char* const b_to = kCols == 256 && p.span > 1 ? small + 1024 : base + 128 * kCols * 2;
  const int l0 = (int)rank * kCols;
  const int mine = max(0, min(kCols, e.l - l0));               // the CTA's columns
  const int deep_x = (mine + 15) / 16, deep_k = (e.k + 15) / 16, wide = max(16, deep_x * 16);
  const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
  __syncthreads();                                             // the patches are read
  put_x();
#pragma unroll 1
  for (int step = 0; step < p.steps; ++step) {
    const float ca = p.coef[step][0], cb = p.coef[step][1], cc = p.coef[step][2];
    products([&] {
      const uint32_t idesc = instruction(128, 128, false, false);
      const uint64_t d = operand(x_at, kPieceBytes, 128);
      for (int q = 0; q < max(1, deep_x); ++q)
        mma_f16<1>(acc_a, d + q * (2 * kPieceBytes >> 4), d + q * (2 * kPieceBytes >> 4), idesc, q > 0);
    });
    float v[32];
    tmem_load16(acc_a + lanes + part * 32, v);
    tmem_load16(acc_a + lanes + part * 32 + 16, v + 16);
    tmem_load_wait();
    if (kCols == 256 && p.span > 1) {
      add_up(v);
    } else {
      if (part == quarter) take_diagonal<32>(v, row, part * 32, diag);
#pragma unroll
      for (int q = 0; q < 4; ++q) put(base + 128 * kCols * 2, part * 4 + q, v + 8 * q);
    }
    products([&] {
      const uint32_t idesc = instruction(128, 128, false, false);
      const uint64_t d = operand(a_at, kPieceBytes, 128);
      for (int q = 0; q < deep_k; ++q)
        mma_f16<1>(acc_a, d + q * (2 * kPieceBytes >> 4), d + q * (2 * kPieceBytes >> 4), idesc, q > 0);
    });
    const float di = diag[row], ei = __fmul_rn(di, __fmaf_rn(cc, di, cb));
    tmem_load16(acc_a + lanes + part * 32, v);
    tmem_load16(acc_a + lanes + part * 32 + 16, v + 16);
    tmem_load_wait();
    {
      const float2 scale = both(__fmul_rn(cc, 1.0f / kScale)), ri = both(__fmaf_rn(cc, di, cb)), c2 = both(cc);
      float2* y = reinterpret_cast<float2*>(v);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint4 old = *reinterpret_cast<const uint4*>(base + 128 * kCols * 2 + (part * 4 + q) * 2048 + row * 16);
        const uint32_t o[4] = {old.x, old.y, old.z, old.w};
        const float2* d = reinterpret_cast<const float2*>(diag + part * 32 + q * 8);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          y[4 * q + k] = __ffma2_rn(__ffma2_rn(c2, d[k], ri), unpack(o[k]), __fmul2_rn(scale, y[4 * q + k]));
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) put(b_to, part * 4 + q, v + 8 * q);
    }
    products([&] {
      const uint32_t idesc = instruction(128, wide, false, true);
      const uint64_t da = operand(smem_u32(b_to), kPieceBytes, 128), db = operand(x_at, 128, kPieceBytes);
      for (int q = 0; q < deep_k; ++q)
        mma_f16<1>(tmem, da + q * (2 * kPieceBytes >> 4), db + q * (2 * 128 >> 4), idesc, q > 0);
    });
    const float2 ca2 = both(ca), down = both(1.0f / kScale), e2 = both(ei);
#pragma unroll
    for (int h = 0; h < kChunks; ++h) {
      if ((part + 4 * h) * 32 >= wide) continue;
      tmem_load16(tmem + lanes + (part + 4 * h) * 32, v);
      tmem_load16(tmem + lanes + (part + 4 * h) * 32 + 16, v + 16);
      tmem_load_wait();
      const float2* y = reinterpret_cast<const float2*>(v);
      float2* z = reinterpret_cast<float2*>(x[h]);
#pragma unroll
      for (int q = 0; q < 16; ++q)
        z[q] = __ffma2_rn(y[q], down, __ffma2_rn(ca2, z[q], __fmul2_rn(e2, unpack(pack(z[q].x, z[q].y)))));
    }
    if (step + 1 < p.steps) put_x();
  }

  // ---- the end of all products, in flight or not
  const bool several = kCols == 256 && p.span > 1;
  if (several) {
    if (!ok)             // all of the cluster's CTAs know by the barrier
      for (int r = 0; r < p.span; ++r)
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(peer(failed, r)), "r"(1) : "memory");
    __syncwarp();
    cluster_sync();
  }
  tc_fence_before();
  ok = __syncthreads_and(ok && (!several || *(volatile int*)(small + 816) == 0));
  tc_fence_after();
  if (!ok) {
    // Products in flight still read shared memory and write TMEM: they get a
    // second.  No CTA of a cluster ends before all copies from and to it have.
    // They have where every wait of the cluster's was met; else, as no more are
    // issued once all its CTAs have been here, those in flight get a millisecond.
    if (warp == 0 && elected()) mma_commit<1>(drain);
    __syncwarp();
    for (const uint64_t t0 = now_ns(); !mbar_try(drain, 0) && now_ns() - t0 < 1000000000ull;) {
    }
    if (several)
      for (const uint64_t t0 = now_ns(); now_ns() - t0 < 1000000;) {
      }
    __syncthreads();
  }
  if (warp == 0) tmem_free<1>(tmem, kTmem);
  // This CTA's threads are done with `fault`.  Whether it is the last to be, and
  // whether any had no result, is asked now and looked at once this result is
  // written (asked with fences and a look at `fault`, 64x64 took 24.7 us for 22.7).
  unsigned long long ended = 0;
  if (threadIdx.x == 0) {
    if (!ok) __threadfence();
    ended = atomicAdd(&c.ws->ended, ok ? 1ull : 1ull + (1ull << 32)) + (ok ? 1ull : 1ull + (1ull << 32));
  }
  const auto end = [&] {
    if (threadIdx.x != 0 || (uint32_t)ended != gridDim.x) return;
    const bool failed = ended >> 32;
    if (failed) {
      c.ws->fault = 0;
      if (p.head || !c.ws->last) ++c.ws->faults;     // once a call
    }
    if (failed || p.head) c.ws->last = failed;
    c.ws->ended = 0;
  };
  if (!ok) {
    end();
    return;
  }
  // ---- result: back through the patches, which lie over the operands
  const bool vout = fits4(io.out, io.out_row, io.out_batch, c.out_type == ZERO_FP32 ? 4 : 2);
  const bool vmaster = c.step && io.master && fits4(io.master, e.cols, (int64_t)e.rows * e.cols, 4);
#pragma unroll
  for (int h = 0; h < kChunks; ++h) {
    const int j0 = l0 + (part + 4 * h) * 32, i0 = quarter * 32;
    const int top = e.tall ? j0 : i0, left = e.tall ? i0 : j0;
    if (e.tall) {
#pragma unroll
      for (int k = 0; k < 32; ++k)
        reinterpret_cast<float*>(cell(patch, k, lane / 4))[lane % 4] = __fmul_rn(x[h][k], 1.0f / kScaleX);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        *cell(patch, lane, k) = make_float4(__fmul_rn(x[h][4 * k], 1.0f / kScaleX), __fmul_rn(x[h][4 * k + 1], 1.0f / kScaleX),
                                            __fmul_rn(x[h][4 * k + 2], 1.0f / kScaleX), __fmul_rn(x[h][4 * k + 3], 1.0f / kScaleX));
    }
    __syncwarp();
#pragma unroll 4
    for (int q = 0; q < 8; ++q) {
      const int r = q * 4 + lane / 8, col = lane % 8 * 4;
      if (top + r < e.rows && left + col < e.cols)
        finish4(c, e, io, b, top + r, left + col, e.cols - left - col, vout, vmaster, *cell(patch, r, lane % 8));
    }
    __syncwarp();
  }
  end();
}

}  // namespace zm
