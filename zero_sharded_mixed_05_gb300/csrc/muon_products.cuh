// muon_products.cuh -- all products of an orthogonalisation in one kernel.
//
// For every matrix and step, with H the first part of X (muon_kernels.cuh):
//   which 0   A = H H^T (H^T H for a tall matrix)
//   which 1   B = b A + c A A
//   which 2   X <- a X + B H (a X + H B for a tall matrix); after the last
//             step the result's epilogue
// A and B are symmetric: only their lower triangle of tiles is computed and
// stored, and a tile above the diagonal is read as its mirror image, with the
// tensor core told that the operand's depth runs down the rows.
//
// What bounds it: the tensor cores, for matrices of a few thousand; the
// latency of fifteen dependent products for small ones.  Hence:
// - one persistent CTA pair an SM pair, 256 x 256 tiles (cta_group::2: each CTA
//   stages half of both operands, 64 KB a stage of depth 128, and holds half of
//   the tile's accumulators), or single CTAs with 128 x 128 tiles where 256
//   would mostly be empty;
// - TMA, products and epilogue run in warps of their own, through a ring of
//   stages and two accumulators, so that a tile's epilogue is hidden behind
//   the next tile's products;
// - no launch between dependent products: the tiles of all products of all
//   matrices form one list in which every tile comes after those that it
//   needs, dealt out in turn; a tile waits for its matrix's count of finished
//   tiles.  With several matrices a wait finds another matrix's tiles done.
//
// The diagonals of A and of b A + c A A are near one where everything else is
// small, so most of the rounding error would come from them.  A's is kept in
// binary32 (`diag`, d) and left out of the stored A (A = S + diag d):
//   b A + c A A = c S S + (b + c (d_i + d_j)) S  off the diagonal's share
//                 + diag(e),  e = b d + c d d,
// and e H enters X's update in binary32.
#pragma once

#include <climits>

#include "muon_kernels.cuh"
#include "sm103.cuh"

namespace zm {

using namespace sm103;

constexpr int kStages = 3;
constexpr int kDepth = 128;                        // of a stage
constexpr int kBoxBytes = 128 * 64 * 2;
constexpr int kOperandBytes = 2 * kBoxBytes;       // a CTA's 128 rows (or columns) of it
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kEpiWarps = 8;
constexpr int kProductThreads = 32 * (4 + kEpiWarps);
constexpr int kPatchCols = 16;
constexpr int kPatchBytes = kEpiWarps * 32 * (kPatchCols + 1) * 4;
constexpr int kDiagBytes = 256 * 4;

struct Products {
  Call c;
  const CUtensorMap* maps;   // four an entry: x[0], x[1], a, b
  const int32_t* starts;     // [2][n + 1]: first tile of each entry, triangular and full
  int32_t steps;
  float coef[ZERO_MUON_MAX_STEPS][3];
};

struct Tile {
  int entry, b, step, which, i, j, unit;
  uint32_t need;             // finished CTA tiles of the matrix that it waits for
};

constexpr int smem_bytes(int n) {
  return 1024 + kStages * kStageBytes + kPatchBytes + kDiagBytes + 256 + 2 * (n + 1) * 4;
}

template <int kPair>
__device__ __forceinline__ Tile tile_at(const Products& p, const int32_t* starts, int64_t index) {
  constexpr int kTile = 128 * kPair;
  const int n = p.c.n;
  const int32_t *tri = starts, *full = starts + n + 1;
  const int64_t per = 2ll * tri[n] + full[n];
  Tile t;
  t.step = (int)(index / per);
  int r = (int)(index - t.step * per);
  t.which = r < tri[n] ? 0 : r < 2 * tri[n] ? 1 : 2;
  r -= t.which == 0 ? 0 : t.which == 1 ? tri[n] : 2 * tri[n];
  const int32_t* at = t.which == 2 ? full : tri;
  int lo = 0, hi = n;                      // the last entry that starts at or before r
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (at[mid] <= r) lo = mid; else hi = mid;
  }
  t.entry = lo;
  r -= at[lo];
  const Entry& e = p.c.entries[lo];
  const int nk = (e.k + kTile - 1) / kTile, nr = (e.rows + kTile - 1) / kTile,
            nc = (e.cols + kTile - 1) / kTile;
  const int ntri = nk * (nk + 1) / 2, nfull = nr * nc;
  const int each = t.which == 2 ? nfull : ntri;
  t.b = r / each;
  r -= t.b * each;
  t.unit = e.unit0 + t.b;
  if (t.which == 2) {
    // the short side runs fastest: X streams by once, B stays in L2
    t.i = e.tall ? r / nc : r % nr;
    t.j = e.tall ? r % nc : r / nr;
  } else {
    int i = (int)((sqrtf(8.0f * (float)r + 1.0f) - 1.0f) * 0.5f);
    while ((i + 1) * (i + 2) / 2 <= r) ++i;
    while (i * (i + 1) / 2 > r) --i;
    t.i = i;
    t.j = r - i * (i + 1) / 2;
  }
  t.need = (uint32_t)kPair * ((uint32_t)t.step * (2 * ntri + nfull) +
                              (t.which == 0 ? 0u : t.which == 1 ? (uint32_t)ntri : 2u * ntri));
  return t;
}

// How one side of a product is read: rows `at`.. of a stored matrix with the
// depth along its rows (kAlong), columns with the depth down its rows
// (kAcross), or a symmetric matrix stored by its lower triangle of tiles.
enum Side { kAlong, kAcross, kSymmetric };

__device__ __forceinline__ Side side_of(const Entry& e, int which, int s) {
  if (which == 0) return e.tall ? kAcross : kAlong;
  if (which == 1) return kSymmetric;
  if (e.tall) return s == 0 ? kAlong : kSymmetric;
  return s == 0 ? kSymmetric : kAcross;
}

// The depth from which on the operand's numbers lie down the rows.
template <int kPair>
__device__ __forceinline__ int across_from(Side s, int at) {
  constexpr int kTile = 128 * kPair;
  return s == kAcross ? 0 : s == kAlong ? INT_MAX : (at / kTile + 1) * kTile;
}

// What every lane holds alike, said so to the compiler: the issuing loops run
// on the warp's uniform registers.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

__device__ __forceinline__ uint32_t pack(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack(uint32_t u) {
  return __half22float2(*reinterpret_cast<const __half2*>(&u));
}

// 32 binary16 numbers at a 32-byte address.
__device__ __forceinline__ void load_row(const __half* p, uint32_t* v) {
  load32(p, v);
  load32(p + 16, v + 8);
}
__device__ __forceinline__ void store_row(__half* p, const uint32_t* v) {
  store32(p, v);
  store32(p + 16, v + 8);
}

// The result of 32 numbers of a row a thread, columns col..col+31.
__device__ __forceinline__ void result_row(const Products& p, const Entry& e, const Io& io, int b, int row,
                                           int row0, int col, float* o, float* patch, int lane) {
  const bool half_out = p.c.out_type != ZERO_FP32;
  const int es = half_out ? 2 : 4;
  const int n = min(32, e.cols - col);
  const uintptr_t rows32 = (uintptr_t)(io.out_row * es) | (uintptr_t)(io.out_batch * es);
  bool wide = ((reinterpret_cast<uintptr_t>(io.out) | rows32) & 31) == 0;
  if (p.c.step && io.master)
    wide = wide && ((reinterpret_cast<uintptr_t>(io.master) | ((uintptr_t)e.cols * 4)) & 31) == 0;
  if (wide && n == 32) {
    // whole sectors a thread
    if (row >= e.rows) return;
    const int64_t at = (int64_t)b * io.out_batch + (int64_t)row * io.out_row + col;
    char* out = static_cast<char*>(io.out) + at * es;
    if (p.c.step) {
      const float step = -__fmul_rn(p.c.lr, e.s);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float w[8];
        if (io.master) {
          load32(io.master + at + 8 * q, reinterpret_cast<uint32_t*>(w));
        } else {
          const uint4 u = *reinterpret_cast<const uint4*>(out + 16 * q);
          const uint32_t* h = reinterpret_cast<const uint32_t*>(&u);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 f = p.c.out_type == ZERO_FP16
                                 ? unpack(h[k])
                                 : make_float2(__uint_as_float(h[k] << 16), __uint_as_float(h[k] & 0xffff0000u));
            w[2 * k] = f.x;
            w[2 * k + 1] = f.y;
          }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          w[k] = __fmaf_rn(step, o[8 * q + k], __fmul_rn(w[k], p.c.decay));
          o[8 * q + k] = w[k];
        }
        if (io.master) store32(io.master + at + 8 * q, reinterpret_cast<const uint32_t*>(w));
      }
    }
    if (!half_out) {
#pragma unroll
      for (int q = 0; q < 4; ++q) store32(out + 32 * q, reinterpret_cast<const uint32_t*>(o + 8 * q));
    } else {
      uint32_t h[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        if (p.c.out_type == ZERO_FP16) {
          h[k] = pack(o[2 * k], o[2 * k + 1]);
        } else {
          const __nv_bfloat162 v = __floats2bfloat162_rn(o[2 * k], o[2 * k + 1]);
          h[k] = *reinterpret_cast<const uint32_t*>(&v);
        }
      }
      store32(out, h);
      store32(out + 32, h + 8);
    }
    return;
  }
  // any address: through shared memory, so that a warp writes along rows
#pragma unroll
  for (int c0 = 0; c0 < 32; c0 += kPatchCols) {
#pragma unroll
    for (int k = 0; k < kPatchCols; ++k) patch[lane * (kPatchCols + 1) + k] = o[c0 + k];
    __syncwarp();
    const int cc = c0 + lane % kPatchCols;
    if (cc < n)
      for (int r = lane / kPatchCols; r < 32; r += 32 / kPatchCols)
        if (row0 + r < e.rows)
          finish(p.c, e, io, b, row0 + r, col + cc, patch[r * (kPatchCols + 1) + lane % kPatchCols]);
    __syncwarp();
  }
}

// One tile's epilogue: the warp's 32 rows of the accumulator, half its columns.
// Whatever it reads besides is fetched while the products still run: the
// diagonal's numbers of the tile's columns go to shared memory, and of each
// 32 columns the operands are on their way while those before are worked on.
// False: a wait ran out.
template <int kPair>
__device__ __forceinline__ bool epilogue(const Products& p, const Tile& t, uint32_t acc, uint32_t full_bar,
                                         uint32_t phase, uint32_t empty_bar, int warp, int lane,
                                         uint32_t rank, float* patch, float* cols) {
  constexpr int kTile = 128 * kPair, kCols = kTile / 2;
  const Entry& en = p.c.entries[t.entry];
  const int rows = en.rows, ncols = en.cols, k = en.k, tall = en.tall;
  const int64_t ldx = en.ldx, ldk = en.ldk;
  const int quarter = warp % 4, part = warp / 4;
  const int row0 = t.i * kTile + (int)rank * 128 + quarter * 32, row = row0 + lane;
  const int M = t.which == 2 ? rows : k, N = t.which == 2 ? ncols : k;
  const float ca = p.coef[t.step][0], cb = p.coef[t.step][1], cc = p.coef[t.step][2];
  const bool last = t.step == p.steps - 1;
  const int cur = t.step & 1;
  const int col0 = t.j * kTile;
  const int64_t at_k = ((int64_t)t.b * k + row) * ldk + col0, at_x = ((int64_t)t.b * rows + row) * ldx + col0;
  float* diag = en.diag + (int64_t)t.b * ldk;
  __half* const to = t.which == 0 ? en.a + at_k : t.which == 1 ? en.b + at_k : en.x[cur ^ 1] + at_x;
  const __half* const from = t.which == 1 ? en.a + at_k : en.x[cur] + at_x;
  __half* const lo_at = en.lo + at_x;
  const bool in = row < M;

  int ok = 1;
  float di = 0.0f;
  uint32_t hi[16], lo[16];
  const auto fetch = [&](int c0) {
    if (t.which == 0 || !in || col0 + c0 >= N) return;
    load_row(from + c0, hi);
    if (t.which == 2) load_row(lo_at + c0, lo);
  };
  if (t.which != 0) {
    if (lane == 0) ok = count_wait(p.c.done + t.unit, t.need, &p.c.ws->fault);
    ok = __shfl_sync(0xffffffffu, ok, 0);
    if (in && (t.which == 1 || !tall)) di = __ldcg(diag + row);
    const int c = warp * 32 + lane;
    if (c < kTile && col0 + c < N) {
      const float d = __ldcg(diag + col0 + c);
      // b A + c A A: c d_j; X: e_j of a tall matrix
      cols[c] = t.which == 1 ? __fmul_rn(cc, d) : __fmul_rn(d, __fmaf_rn(cc, d, cb));
    }
    fetch(part * kCols);
  }
  if (lane == 0 && ok) ok = mbar_wait(full_bar, phase, &p.c.ws->fault);
  ok = __shfl_sync(0xffffffffu, ok, 0);
  // all eight warps go on or none: the count of finished tiles is of whole ones
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.ne.b32 p, %1, 0;\n"
      "barrier.red.and.pred q, 1, %2, p;\nselp.b32 %0, 1, 0, q;\n}"
      : "=r"(ok)
      : "r"(ok), "r"(32 * kEpiWarps)
      : "memory");
  if (!ok) return false;
  tc_fence_after();

  const uint32_t lanes = acc + ((uint32_t)(quarter * 32) << 16);
  // the row's share of b A + c A A's factor, or e_i of a wide matrix
  const float ei = t.which == 1 ? __fmaf_rn(cc, di, cb) : __fmul_rn(di, __fmaf_rn(cc, di, cb));
#pragma unroll 1
  for (int c0 = part * kCols; c0 < (part + 1) * kCols; c0 += 32) {
    if (col0 + c0 >= N || row0 >= M) break;
    float v[32];
    tmem_load32(lanes + c0, v);
    tmem_load_wait();
    if (t.which == 0) {
      if (in) {
        const int at = row - (col0 + c0);     // the diagonal's place in this row, if any
#pragma unroll
        for (int q = 0; q < 32; ++q) {
          v[q] = __fmul_rn(v[q], 1.0f / kScale);
          if (q == at) {
            __stcg(diag + row, __fmul_rn(v[q], 1.0f / kScale));
            v[q] = 0.0f;
          }
        }
#pragma unroll
        for (int q = 0; q < 16; ++q) hi[q] = pack(v[2 * q], v[2 * q + 1]);
        // rows are multiples of 32 numbers: nothing of the next row is written
        store_row(to + c0, hi);
      }
    } else if (t.which == 1) {
      if (in) {
        uint32_t h[16];
        const float scale = __fmul_rn(cc, 1.0f / kScale);
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          const float2 f = unpack(hi[q]), d = reinterpret_cast<const float2*>(cols + c0)[q];
          h[q] = pack(__fmaf_rn(__fadd_rn(ei, d.x), f.x, __fmul_rn(scale, v[2 * q])),
                      __fmaf_rn(__fadd_rn(ei, d.y), f.y, __fmul_rn(scale, v[2 * q + 1])));
        }
        if (c0 + 32 < (part + 1) * kCols) fetch(c0 + 32);
        store_row(to + c0, h);
      }
    } else {
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        const float2 h = unpack(hi[q]), l = unpack(lo[q]);
        float2 d = make_float2(ei, ei);
        if (tall) d = reinterpret_cast<const float2*>(cols + c0)[q];
        v[2 * q] = __fmaf_rn(v[2 * q], 1.0f / kScale,
                             __fmaf_rn(ca, __fmaf_rn(l.x, 1.0f / kLoScale, h.x), __fmul_rn(d.x, h.x)));
        v[2 * q + 1] = __fmaf_rn(v[2 * q + 1], 1.0f / kScale,
                                 __fmaf_rn(ca, __fmaf_rn(l.y, 1.0f / kLoScale, h.y), __fmul_rn(d.y, h.y)));
      }
      if (c0 + 32 < (part + 1) * kCols) fetch(c0 + 32);
      if (last) {
#pragma unroll
        for (int q = 0; q < 32; ++q) v[q] = __fmul_rn(v[q], 1.0f / kScale);
        result_row(p, en, p.c.io[en.item], t.b, row, row0, col0 + c0, v, patch, lane);
      } else if (in) {
        uint32_t h[16], l[16];
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          h[q] = pack(v[2 * q], v[2 * q + 1]);
          const float2 f = unpack(h[q]);
          l[q] = pack(__fmul_rn(__fadd_rn(v[2 * q], -f.x), kLoScale),
                      __fmul_rn(__fadd_rn(v[2 * q + 1], -f.y), kLoScale));
        }
        store_row(to + c0, h);
        store_row(lo_at + c0, l);
      }
    }
  }
  // the accumulator may be written again once both CTAs have read it
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive_cluster(kPair == 2 ? peer(empty_bar, 0) : empty_bar);
  // the tile is done when all its warps' writes are made
  fence_proxy_async();
  asm volatile("barrier.sync 1, %0;" ::"r"(32 * kEpiWarps) : "memory");
  if (warp == 0 && lane == 0)
    asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(p.c.done + t.unit) : "memory");
  return true;
}

template <int kPair>
__global__ void __launch_bounds__(kProductThreads, 1)
    muon_products_kernel(const __grid_constant__ Products p) {
  constexpr int kTile = 128 * kPair;
  constexpr uint32_t kTmemCols = 2 * kTile;
  extern __shared__ unsigned char raw[];
  if (skipped(p.c)) return;
  unsigned char* base = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const uint32_t stages = smem_u32(base);
  float* patches = reinterpret_cast<float*>(base + kStages * kStageBytes);
  float* cols = reinterpret_cast<float*>(base + kStages * kStageBytes + kPatchBytes);
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + kStages * kStageBytes + kPatchBytes + kDiagBytes);
  int32_t* starts = reinterpret_cast<int32_t*>(base + kStages * kStageBytes + kPatchBytes + kDiagBytes + 256);
  const uint32_t full = smem_u32(bars), empty = full + 8 * kStages, acc_full = empty + 8 * kStages,
                 acc_empty = acc_full + 16, drain = acc_empty + 16, tmem_at = drain + 8;
  const int warp = uniform(threadIdx.x / 32), lane = threadIdx.x % 32;
  const uint32_t rank = kPair == 2 ? cluster_rank() : 0;
  int* fault = &p.c.ws->fault;

  for (int i = threadIdx.x; i < 2 * (p.c.n + 1); i += kProductThreads) starts[i] = p.starts[i];
  if (warp == 0 && lane == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full + 8 * s, 1);
      mbar_init(empty + 8 * s, 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(acc_full + 8 * s, 1);
      mbar_init(acc_empty + 8 * s, kPair * kEpiWarps);
    }
    mbar_init(drain, 1);
    mbar_init_fence();
  }
  if (warp == 2) tmem_alloc<kPair>(tmem_at, kTmemCols);
  tc_fence_before();
  __syncthreads();
  if (kPair == 2) cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(base + (tmem_at - stages));
  const int64_t total = (2ll * starts[p.c.n] + starts[2 * p.c.n + 1]) * p.steps;
  const int first = blockIdx.x / kPair, stride = gridDim.x / kPair;

  if (warp == 0 || warp == 3) {
    // ---- TMA: warp 0 the first operand, warp 3 the second.  A warp walks
    // together; one lane issues.
    const int side = warp == 3;
    uint32_t s = 0, phase = 1;
    int64_t issued = 0;
    bool ok = true;
    for (int64_t index = first; ok && index < total; index += stride) {
      const Tile t = tile_at<kPair>(p, starts, index);
      const Entry& e = p.c.entries[t.entry];
      const Side how = side_of(e, t.which, side);
      const CUtensorMap* map = p.maps + 4 * t.entry + (how == kSymmetric ? 1 + t.which : t.step & 1);
      const int m0 = (side ? t.j : t.i) * kTile, at = uniform(m0 + (int)rank * 128);
      const int depth = uniform(t.which == 0 ? e.l : e.k), turn = uniform(across_from<kPair>(how, m0));
      const int b = uniform(t.b);
      if (t.need) {
        ok = __all_sync(0xffffffffu, count_wait(p.c.done + t.unit, t.need, fault));
        if (!ok) break;
        fence_proxy_async();
      }
      for (int k0 = 0; k0 < depth; k0 += kDepth) {
        ok = __all_sync(0xffffffffu, mbar_wait(empty + 8 * s, phase, fault));
        if (!ok) break;
        const uint32_t bar = kPair == 2 ? peer(full + 8 * s, 0) : full + 8 * s;
        const uint32_t to = stages + s * kStageBytes + side * kOperandBytes;
        const bool x = k0 >= turn;
        if (elected()) {
          if (rank == 0 && side == 0) mbar_expect(full + 8 * s, kPair * kStageBytes);
          tma_load<kPair>(to, map, bar, x ? at : k0, x ? k0 : at, b);
          tma_load<kPair>(to + kBoxBytes, map, bar, (x ? at : k0) + 64, x ? k0 : at, b);
        }
        __syncwarp();
        ++issued;
        if (++s == kStages) { s = 0; phase ^= 1; }
      }
    }
    // Every stage that was filled is released (or, after a fault, has at
    // least arrived) before the CTA may end.
    if (ok) {
      for (int q = 0; ok && q < kStages && q < issued; ++q) {
        ok = mbar_wait(empty + 8 * s, phase, fault);
        if (++s == kStages) { s = 0; phase ^= 1; }
      }
    }
    if (!ok && rank == 0 && side == 0) {
      const uint64_t t0 = now_ns();
      const int held = (int)(issued < kStages ? issued : kStages);
      for (int q = 0; q < held; ++q) {
        const int64_t at = issued - held + q;
        while (!mbar_try(full + 8 * (uint32_t)(at % kStages), (uint32_t)(at / kStages) & 1) &&
               now_ns() - t0 < 1000000000ull) {
        }
      }
    }
  } else if (warp == 1 && rank == 0) {
    // ---- products.  The warp walks together; one lane issues.
    uint32_t s = 0, phase = 0, acc = 0, acc_phase = 1;
    bool ok = true;
    for (int64_t index = first; ok && index < total; index += stride) {
      const Tile t = tile_at<kPair>(p, starts, index);
      const Entry& e = p.c.entries[t.entry];
      const int ta = uniform(across_from<kPair>(side_of(e, t.which, 0), t.i * kTile));
      const int tb = uniform(across_from<kPair>(side_of(e, t.which, 1), t.j * kTile));
      const int depth = uniform(t.which == 0 ? e.l : e.k);
      ok = __all_sync(0xffffffffu, mbar_wait(acc_empty + 8 * acc, acc_phase, fault));
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = tmem + acc * kTile;
      for (int k0 = 0; k0 < depth; k0 += kDepth) {
        const bool xa = k0 >= ta, xb = k0 >= tb;
        const uint32_t idesc = instruction(kTile, kTile, xa, xb);
        const uint32_t at = stages + s * kStageBytes;
        const uint64_t da = operand(at, kBoxBytes), db = operand(at + kOperandBytes, kBoxBytes);
        ok = __all_sync(0xffffffffu, mbar_wait(full + 8 * s, phase, fault));
        if (!ok) break;
        tc_fence_after();
        if (elected()) {
#pragma unroll
          for (int q = 0; q < kDepth / 16; ++q) {
            // 16 deep: 32 bytes along a row (four to a box), or 16 rows of 128 bytes
            const uint32_t along = (q / 4 * kBoxBytes + q % 4 * 32) >> 4, down = q * 16 * 128 >> 4;
            mma_f16<kPair>(d, da + (xa ? down : along), db + (xb ? down : along), idesc, k0 > 0 || q > 0);
          }
          mma_commit<kPair>(empty + 8 * s);
          if (k0 + kDepth >= depth) mma_commit<kPair>(acc_full + 8 * acc);
        }
        __syncwarp();
        if (++s == kStages) { s = 0; phase ^= 1; }
      }
      if (++acc == 2) { acc = 0; acc_phase ^= 1; }
    }
    if (!ok) {   // products in flight still read shared memory and write TMEM
      if (elected()) mma_commit<kPair>(drain);
      const uint64_t t0 = now_ns();
      while (!mbar_try(drain, 0) && now_ns() - t0 < 1000000000ull) {
      }
    }
  } else if (warp >= 4) {
    // ---- epilogue
    uint32_t acc = 0, phase = 0;
    float* patch = patches + (warp - 4) * 32 * (kPatchCols + 1);
    for (int64_t index = first; index < total; index += stride) {
      const Tile t = tile_at<kPair>(p, starts, index);
      if (!epilogue<kPair>(p, t, tmem + acc * kTile, acc_full + 8 * acc, phase, acc_empty + 8 * acc,
                           warp - 4, lane, rank, patch, cols))
        break;
      if (++acc == 2) { acc = 0; phase ^= 1; }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (kPair == 2) cluster_sync();
  tc_fence_after();
  if (warp == 2) tmem_free<kPair>(tmem, kTmemCols);
}

}  // namespace zm
