// muon_products.cuh -- all products of an orthogonalisation in one kernel.
//
// For every matrix and step, with H the binary16 rounding of X:
//   which 0   A = H H^T (H^T H for a tall matrix)
//   which 1   B = b A + c A A
//   which 2   X <- a X + B H (a X + H B for a tall matrix); after the last
//             step the result's epilogue
// A and B are symmetric: only their lower triangle of tiles is computed and
// stored, and a tile above the diagonal is read as its mirror image, with the
// tensor core told that the operand's depth runs down the rows.
//
// What bounds it: the tensor cores, for matrices of a few thousand (14336x4096:
// 2.39 ms, 83 % of the tensor cores' cycles; 4096x4096, whose 136 tiles of a
// symmetric product make 1.8 waves of 76 pairs: 0.88 ms, 72 %); the latency of
// fifteen dependent products for small ones (1000x777 x 3: 104 us of which the
// tensor cores work 18).  In between, shallow B X, the epilogue: 12 of 2304x768,
// 0.29 ms, 46 %; a tile of depth 768 takes 4.0 us of products and 5.0 of epilogue,
// 1.3 MB between L2 and its SMs, 19 TB/s in all.  Hence:
// - one persistent CTA pair an SM pair, 256 x 256 tiles (cta_group::2: each CTA
//   stages half of both operands, 64 KB a stage of depth 128, and holds half of
//   the tile's accumulators), or single CTAs with 128 x 128 tiles where 256
//   would mostly be empty;
// - TMA, products and epilogue run in warps of their own, through a ring of
//   stages and two accumulators, so that a tile's epilogue is hidden behind
//   the next tile's products; the first TMA warp finds out what the next tile
//   is and waits for what it needs, and tells the others by a ring of tiles;
// - no launch between dependent products: the tiles of all products of all
//   matrices form one list in which every tile comes after those that it
//   needs, dealt out in turn; a tile waits for its matrix's count of finished
//   tiles.  With several matrices a wait finds another matrix's tiles done.
//
// A deep X X^T of few tiles (k x k of a matrix with l far above k) is cut along
// its depth: each part leaves its binary32 sums in the workspace, and the one
// that arrives last adds them up in order and goes on (8080x80 x 2: 176 -> 116 us).
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
constexpr int kBoxBytes = 128 * 64 * 2;            // 128 rows of eight pieces of eight columns
constexpr int kPieceBytes = 128 * 16;              // in shared memory: a piece's 128 rows side by side
constexpr int kOperandBytes = 2 * kBoxBytes;       // a CTA's 128 rows (or columns) of it
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kEpiWarps = 12;
constexpr int kProductThreads = 32 * (4 + kEpiWarps);
constexpr int kPatchBytes = kEpiWarps * 2048;      // a warp's 32 rows of 64 bytes
constexpr int kDiagBytes = 2 * 256 * 4;            // of two tiles
constexpr int kSlots = 16;                         // tiles a CTA has in work: 3 stages, 2 accumulators,
                                                   // 2 being counted; the rest is slack

struct Products {
  Call c;
  const CUtensorMap* maps;   // four an entry: x[0], x[1], a, b
  const int32_t* starts;     // [3][n]: first tile of each entry in a product of each kind
  float4* parts;             // sums of the parts of cut tiles
  int64_t tiles;             // of all products
  int32_t count[3];          // of a product of each kind
  int32_t steps;
  int32_t far;               // X does not stay in L2: its second part is asked for ahead
  uint32_t inject;           // test hook: added to what a tile waits for
  float coef[ZERO_MUON_MAX_STEPS][3];
};

struct Tile {
  Entry e;
  int entry, b, step, which, i, j, unit;
  int from, depth;           // the depth's part: from.. up to depth
  int splits, part, cut, slot;   // parts of the tile, which this is, its counter, its first part's place
  uint32_t need;             // finished CTA tiles of the matrix that it waits for
};

constexpr int kProductSmem = kStages * kStageBytes + kPatchBytes + kDiagBytes + 256 + kSlots * (int)sizeof(Tile);

template <int kPair>
__device__ __forceinline__ void tile_at(const Products& p, int64_t index, int lane, Tile* out) {
  constexpr int kTile = 128 * kPair;
  const int per = p.count[0] + p.count[1] + p.count[2];
  const int step = (int)(index / per);
  int r = (int)(index - (int64_t)step * per);
  const int which = r < p.count[0] ? 0 : r < p.count[0] + p.count[1] ? 1 : 2;
  r -= (which > 0 ? p.count[0] : 0) + (which > 1 ? p.count[1] : 0);
  const int32_t* at = p.starts + which * p.c.n;
  int lo = 0, hi = p.c.n;                  // the last entry that starts at or before r
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (at[mid] <= r) lo = mid; else hi = mid;
  }
  r -= at[lo];
  const Entry& from = p.c.entries[lo];
  static_assert(sizeof(Entry) % 4 == 0 && sizeof(Entry) / 4 <= 64, "copied by one warp");
  for (int w = lane; w < (int)sizeof(Entry) / 4; w += 32)
    reinterpret_cast<uint32_t*>(&out->e)[w] = reinterpret_cast<const uint32_t*>(&from)[w];
  __syncwarp();
  const Entry& e = out->e;
  const int nk = (e.k + kTile - 1) / kTile, nr = (e.rows + kTile - 1) / kTile, nc = (e.cols + kTile - 1) / kTile;
  const int ntri = nk * (nk + 1) / 2, nfull = nr * nc;
  const int splits = which == 0 ? e.splits : 1, part = r % splits;
  r /= splits;
  const int each = which == 2 ? nfull : ntri;
  const int b = r / each;
  r %= each;
  int i, j;
  if (which == 2) {
    // the short side runs fastest: X streams by once, B stays in L2
    i = e.tall ? r / nc : r % nr;
    j = e.tall ? r % nc : r / nr;
  } else {
    i = (int)((sqrtf(8.0f * (float)r + 1.0f) - 1.0f) * 0.5f);
    while ((i + 1) * (i + 2) / 2 <= r) ++i;
    while (i * (i + 1) / 2 > r) --i;
    j = r - i * (i + 1) / 2;
  }
  if (lane == 0) {
    out->entry = lo;
    out->b = b;
    out->step = step;
    out->which = which;
    out->i = i;
    out->j = j;
    out->unit = e.unit0 + b;
    const int depth = which == 0 ? e.l : e.k, stages = ((depth + kDepth - 1) / kDepth + splits - 1) / splits;
    out->from = part * stages * kDepth;
    out->depth = min(depth, (part + 1) * stages * kDepth);
    out->splits = splits;
    out->part = part;
    out->cut = e.cut0 + b * e.cuts + r * kPair;
    out->slot = e.slot0 + (b * ntri + r) * splits;
    const uint32_t need = (uint32_t)kPair * ((uint32_t)step * (2 * ntri + nfull) +
                                   (which == 0 ? 0u : which == 1 ? (uint32_t)ntri : 2u * ntri));
    out->need = need ? need + p.inject : 0u;
  }
  __syncwarp();
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

// The warp's shared memory: 32 rows of 64 bytes, the 16-byte pieces of a row in
// an order of the row's own, so that neither rows nor pieces collide.
__device__ __forceinline__ uint4* piece(float* patch, int row, int at) {
  return reinterpret_cast<uint4*>(patch) + row * 4 + (at ^ (row / 2 & 3));
}

// A warp's 32 x 16 numbers of the result: it reads and writes along rows, at any
// address, a lane one column of every second row.
constexpr int kLaneRows = 16;
template <typename F>
__device__ __forceinline__ void each_row(const Entry& e, int row0, int col0, int lane, F f) {
  const int row = row0 + lane / 16, n = col0 + lane % 16 < e.cols ? e.rows - row : 0;
#pragma unroll
  for (int k = 0; k < kLaneRows; ++k)
    if (2 * k < n) f(k);
}
// The masters there, which the step updates.
__device__ __forceinline__ void fetch_masters(const Call& c, const Entry& e, const Io& io, int b, int row0, int col0,
                                              int lane, float w[kLaneRows]) {
  const int64_t at = ((int64_t)b * e.rows + row0 + lane / 16) * e.cols + col0 + lane % 16, down = 2 * (int64_t)e.cols;
  if (io.master) each_row(e, row0, col0, lane, [&](int k) { w[k] = io.master[at + k * down]; });
  else if (c.out_type == ZERO_FP16)
    each_row(e, row0, col0, lane, [&](int k) { w[k] = num<__half>(static_cast<const __half*>(io.out)[at + k * down]); });
  else
    each_row(e, row0, col0, lane,
             [&](int k) { w[k] = num<__nv_bfloat16>(static_cast<const __nv_bfloat16*>(io.out)[at + k * down]); });
}
// The result from the patch, O itself or the step on the masters `w` with it.
__device__ __forceinline__ void result(const Call& c, const Entry& e, const Io& io, int b, int row0, int col0,
                                       float* patch, int lane, const float w[kLaneRows]) {
  const int64_t ld = c.step ? e.cols : io.out_row;
  const int64_t at = b * (c.step ? (int64_t)e.rows * e.cols : io.out_batch) + (row0 + lane / 16) * ld + col0 + lane % 16;
  const float factor = c.step ? -__fmul_rn(c.lr, e.s) : 1.0f;
  const auto value = [&](int k) {
    const int col = lane % 16;
    const float o = __fmul_rn(reinterpret_cast<const float*>(piece(patch, lane / 16 + 2 * k, col / 4))[col % 4], 1.0f / kScaleX);
    if (!c.step) return o;
    const float x = __fmaf_rn(factor, o, __fmul_rn(w[k], c.decay));
    if (io.master) io.master[at + 2 * k * ld] = x;
    return x;
  };
  if (c.out_type == ZERO_FP16)
    each_row(e, row0, col0, lane, [&](int k) { static_cast<__half*>(io.out)[at + 2 * k * ld] = as<__half>(value(k)); });
  else if (c.out_type == ZERO_BF16)
    each_row(e, row0, col0, lane,
             [&](int k) { static_cast<__nv_bfloat16*>(io.out)[at + 2 * k * ld] = as<__nv_bfloat16>(value(k)); });
  else
    each_row(e, row0, col0, lane, [&](int k) { static_cast<float*>(io.out)[at + 2 * k * ld] = value(k); });
}

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// One tile's epilogue: the warp's 32 rows of the accumulator, every third 16 of
// its columns.  Whatever it reads besides is fetched while the products
// still run: the diagonal's numbers of the tile's columns go to shared memory
// (`cols`), and the numbers of the columns after the next are on their way while
// those before are worked on.  The loops are kept short: a small matrix runs each of them
// once a tile, and straight code of 64 columns waited on instruction fetches
// longer than it ran (64x64 through this kernel: 91 us with it, 53 now).
enum Outcome { kFailed, kDone, kPart };   // a wait ran out; the tile is done; a part of it is
template <int kPair>
__device__ __forceinline__ Outcome epilogue(const Products& p, const Tile& t, bool ready, uint32_t told, uint32_t number,
                                         uint32_t acc, uint32_t full_bar,
                                         uint32_t phase, uint32_t empty_bar, int warp, int lane, uint32_t rank,
                                         float* patch, float* cols, volatile int* arrived) {
  constexpr int kTile = 128 * kPair;
  const Entry& en = t.e;
  const int rows = en.rows, ncols = en.cols, k = en.k, tall = en.tall;
  const int64_t ldx = en.ldx, ldk = en.ldk;
  const int quarter = warp % 4, part = warp / 4;
  const int row0 = t.i * kTile + (int)rank * 128 + quarter * 32, row = row0 + lane;
  const int M = t.which == 2 ? rows : k, N = t.which == 2 ? ncols : k;
  const float ca = p.coef[t.step][0], cb = p.coef[t.step][1], cc = p.coef[t.step][2];
  const bool last = t.step == p.steps - 1;
  // columns of the tile, to whole blocks: padding is written too, as zeros
  const int col0 = t.j * kTile, ncol = row0 < M ? min(kTile, (N + 31) / 32 * 32 - col0) : 0;
  const int64_t ld = t.which == 2 ? ldx : ldk;
  const int64_t at0 = t.b * block_size(M, ld) + block_at(row, col0, ld);
  float* diag = en.diag + t.b * ldk;
  uint4* const to = reinterpret_cast<uint4*>((t.which == 0 ? en.a : t.which == 1 ? en.b : en.x[(t.step & 1) ^ 1]) + at0);
  const uint4* const from = reinterpret_cast<const uint4*>((t.which == 1 ? en.a : en.x[t.step & 1]) + at0);
  uint4* const low = reinterpret_cast<uint4*>(en.lo + at0);

  int ok = ready;
  float di = 0.0f;
  constexpr int kNext = 16 * (kEpiWarps / 4);  // to the warp's next 16 columns
  struct Pieces {
    uint4 hi[2], lo[2];
  } even, odd;
  const auto fetch = [&](Pieces& y, int c) {
    if (c >= ncol) return;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      y.hi[q] = __ldcg(from + c * 16 + q * 128);
      if (t.which == 2) y.lo[q] = __ldcg(low + c * 16 + q * 128);
    }
  };
  const Io io = last && t.which == 2 ? p.c.io[en.item] : Io{};
  float w[kLaneRows];
  if (t.which != 0) {
    ok = __all_sync(0xffffffffu, ok && shared_wait(told, number + 1, &p.c.ws->fault));
    if (ok) {
      fetch(even, part * 16);
      if (t.which == 2 && last) {
        if (p.c.step && part * 16 < ncol) fetch_masters(p.c, en, io, t.b, row0, col0 + part * 16, lane, w);
      } else {
        fetch(odd, part * 16 + kNext);
      }
      const int c = warp * 32 + lane;
      float d = 0.0f;
      // the columns are A's, but those of a wide matrix's X
      if (c < kTile && col0 + c < N && (t.which == 1 || tall)) d = __ldcg(diag + col0 + c);
      if (row < M && (t.which == 1 || !tall)) di = __ldcg(diag + row);
      // b A + c A A: c d_j; X: e_j of a tall matrix
      if (c < kTile) cols[c] = t.which == 1 ? __fmul_rn(cc, d) : __fmul_rn(d, __fmaf_rn(cc, d, cb));
    }
  }
  if (lane == 0 && ok) ok = mbar_wait(full_bar, phase, &p.c.ws->fault);
  ok = __shfl_sync(0xffffffffu, ok, 0);
  // all its warps go on or none: the count of finished tiles is of whole ones
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.ne.b32 p, %1, 0;\n"
      "barrier.red.and.pred q, 1, %2, p;\nselp.b32 %0, 1, 0, q;\n}"
      : "=r"(ok)
      : "r"(ok), "r"(32 * kEpiWarps)
      : "memory");
  if (!ok) return kFailed;
  tc_fence_after();

  const uint32_t lanes = acc + ((uint32_t)(quarter * 32) << 16);
  // the row's share of b A + c A A's factor, or e_i of a wide matrix
  const float ei = t.which == 1 ? __fmaf_rn(cc, di, cb) : __fmul_rn(di, __fmaf_rn(cc, di, cb));
  // the accumulator may be written again once both CTAs have read it
  const auto release = [&] {
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive_cluster(kPair == 2 ? peer(empty_bar, 0) : empty_bar);
  };
  const bool cut = t.splits > 1;             // X X^T alone
  // four columns of the tile's 128 rows of this CTA side by side
  const int slot_size = kTile / 4 * 128;
  float4* sums = p.parts + ((int64_t)t.slot * kPair + rank) * slot_size + quarter * 32 + lane;
  if (cut) {
    float4* own = sums + (int64_t)t.part * kPair * slot_size;
#pragma unroll 1
    for (int c = part * 16; c < ncol; c += kNext) {
      float v[16];
      tmem_load16(lanes + c, v);
      tmem_load_wait();
#pragma unroll
      for (int q = 0; q < 4; ++q) __stcg(own + (c / 4 + q) * 128, reinterpret_cast<const float4*>(v)[q]);
    }
    release();
    asm volatile("barrier.sync 1, %0;" ::"r"(32 * kEpiWarps) : "memory");
    if (warp == 0 && lane == 0) {
      __threadfence();
      uint32_t* counter = p.c.cut + t.cut + rank;
      const bool all = atomicAdd(counter, 1u) == (uint32_t)t.splits - 1;
      if (all) *counter = 0u;
      __threadfence();
      *arrived = all;
    }
    asm volatile("barrier.sync 1, %0;" ::"r"(32 * kEpiWarps) : "memory");
    if (!*arrived) return kPart;
  }
  const auto put = [&](int c, const float2* y) {
#pragma unroll
    for (int q = 0; q < 2; ++q)
      to[c * 16 + q * 128] = make_uint4(pack(y[4 * q].x, y[4 * q].y), pack(y[4 * q + 1].x, y[4 * q + 1].y),
                                        pack(y[4 * q + 2].x, y[4 * q + 2].y), pack(y[4 * q + 3].x, y[4 * q + 3].y));
  };
  // b A + c A A
  const auto second = [&](int c, Pieces& x) {
    float2 y[8];
    tmem_load16(lanes + c, reinterpret_cast<float*>(y));
    tmem_load_wait();
    const float2 scale = both(__fmul_rn(cc, 1.0f / kScale)), e2 = both(ei);
    const uint32_t* s = reinterpret_cast<const uint32_t*>(x.hi);
    const float2* d = reinterpret_cast<const float2*>(cols + c);
#pragma unroll
    for (int q = 0; q < 8; ++q) y[q] = __ffma2_rn(__fadd2_rn(e2, d[q]), unpack(s[q]), __fmul2_rn(scale, y[q]));
    fetch(x, c + 2 * kNext);
    put(c, y);
  };
  // a X + B X
  const auto third = [&](int c, Pieces& x, float2* y, int ahead) {
    tmem_load16(lanes + c, reinterpret_cast<float*>(y));
    tmem_load_wait();
    const uint32_t *h = reinterpret_cast<const uint32_t*>(x.hi), *l = reinterpret_cast<const uint32_t*>(x.lo);
    const float2* d = reinterpret_cast<const float2*>(cols + c);
    const float2 ca2 = both(ca), down = both(1.0f / kScale), e2 = both(ei), low2 = both(1.0f / kLoScale);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const float2 z = unpack(h[q]);
      y[q] = __ffma2_rn(y[q], down,
                        __ffma2_rn(ca2, __ffma2_rn(unpack(l[q]), low2, z), __fmul2_rn(tall ? d[q] : e2, z)));
    }
    fetch(x, c + ahead);
  };
  const auto next_x = [&](int c, Pieces& x) {
    float2 y[8];
    third(c, x, y, 2 * kNext);
    __align__(16) __half2 first[8], rest[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) split(y[q], &first[q], &rest[q]);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      to[c * 16 + q * 128] = reinterpret_cast<const uint4*>(first)[q];
      low[c * 16 + q * 128] = reinterpret_cast<const uint4*>(rest)[q];
    }
  };
  if (t.which == 0) {
#pragma unroll 1
    for (int c = part * 16; c < ncol; c += kNext) {
      float v[16];
      if (cut) {
#pragma unroll
        for (int q = 0; q < 16; ++q) v[q] = 0.0f;
#pragma unroll 4
        for (int s = 0; s < t.splits; ++s)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float4 y = __ldcg(sums + (int64_t)s * kPair * slot_size + (c / 4 + q) * 128);
            v[4 * q] = __fadd_rn(v[4 * q], y.x);
            v[4 * q + 1] = __fadd_rn(v[4 * q + 1], y.y);
            v[4 * q + 2] = __fadd_rn(v[4 * q + 2], y.z);
            v[4 * q + 3] = __fadd_rn(v[4 * q + 3], y.w);
          }
      } else {
        tmem_load16(lanes + c, v);
        tmem_load_wait();
      }
      const int at = row - (col0 + c);         // the diagonal's place, if in these columns
      if (row0 < col0 + c + 16 && row0 + 32 > col0 + c) {
        float d = 0.0f;
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          d = q == at ? v[q] : d;
          v[q] = q == at ? 0.0f : v[q];
        }
        if (at >= 0 && at < 16 && row < M) __stcg(diag + row, __fmul_rn(d, 1.0f / kScale));
      }
      put(c, reinterpret_cast<const float2*>(v));
    }
  } else if (t.which == 1) {
#pragma unroll 1
    for (int c = part * 16; c < ncol; c += 2 * kNext) {
      second(c, even);
      if (c + kNext < ncol) second(c + kNext, odd);
    }
  } else if (!last) {
#pragma unroll 1
    for (int c = part * 16; c < ncol; c += 2 * kNext) {
      next_x(c, even);
      if (c + kNext < ncol) next_x(c + kNext, odd);
    }
  } else {
#pragma unroll 1
    for (int c = part * 16; c < ncol; c += kNext) {
      float2 y[8];
      third(c, even, y, kNext);
#pragma unroll
      for (int q = 0; q < 4; ++q) *piece(patch, lane, q) = reinterpret_cast<const uint4*>(y)[q];
      __syncwarp();
      result(p.c, en, io, t.b, row0, col0 + c, patch, lane, w);
      __syncwarp();
      if (p.c.step && c + kNext < ncol) fetch_masters(p.c, en, io, t.b, row0, col0 + c + kNext, lane, w);
    }
  }
  if (!cut) release();
  return kDone;
}

template <int kPair>
__global__ void __launch_bounds__(kProductThreads, 1)
    muon_products_kernel(const __grid_constant__ Products p) {
  constexpr int kTile = 128 * kPair;
  constexpr uint32_t kTmemCols = 2 * kTile;
  extern __shared__ __align__(1024) unsigned char base[];
  if (skipped(p.c)) return;
  const uint32_t stages = smem_u32(base);
  float* patches = reinterpret_cast<float*>(base + kStages * kStageBytes);
  float* cols = reinterpret_cast<float*>(base + kStages * kStageBytes + kPatchBytes);
  unsigned char* small = base + kStages * kStageBytes + kPatchBytes + kDiagBytes;
  Tile* slots = reinterpret_cast<Tile*>(small + 256);
  const uint32_t full = smem_u32(small), empty = full + 8 * kStages, acc_full = empty + 8 * kStages,
                 acc_empty = acc_full + 16, drain = acc_empty + 16, tmem_at = drain + 8,
                 known = tmem_at + 4,      // tiles that are in the ring
                 told = known + 4,         // and whose needs are met
                 counted = told + 4;       // tiles whose writes the counting warp has seen
  // [0] the epilogue gave up, [1] its tile's parts have all arrived, [2], [3] the tile is only a part
  volatile int* const stop = reinterpret_cast<volatile int*>(small + (counted - full) + 4);
  const int warp = uniform(threadIdx.x / 32), lane = threadIdx.x % 32;
  const uint32_t rank = kPair == 2 ? cluster_rank() : 0;
  int* fault = &p.c.ws->fault;

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
    shared_set(known, 0);
    shared_set(told, 0);
    shared_set(counted, 0);
    *stop = 0;
    mbar_init_fence();
  }
  if (warp == 2) tmem_alloc<kPair>(tmem_at, kTmemCols);
  tc_fence_before();
  __syncthreads();
  if (kPair == 2) cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(small + (tmem_at - full));
  const int first = blockIdx.x / kPair, stride = gridDim.x / kPair;
  const uint32_t mine = first < p.tiles ? (uint32_t)((p.tiles - first + stride - 1) / stride) : 0;   // tiles

  if (warp == 0 || warp == 3) {
    // ---- TMA: warp 0 the first operand, warp 3 the second.  A warp walks
    // together; one lane issues.
    const int side = warp == 3;
    uint32_t s = 0, phase = 1, issued = 0;
    uint32_t fenced = 0;                   // maps of the first eight entries that have been
    bool ok = true;
    for (uint32_t n = 0; ok && n < mine; ++n) {
      Tile& t = slots[n % kSlots];
      if (side == 0) {
        tile_at<kPair>(p, first + (int64_t)n * stride, lane, &t);
        if (lane == 0) shared_set(known, n + 1);
      } else {
        ok = __all_sync(0xffffffffu, shared_wait(known, n + 1, fault));
        if (!ok) break;
      }
      const Side how = side_of(t.e, t.which, side), other = side_of(t.e, t.which, side ^ 1);
      const CUtensorMap* map = p.maps + 4 * t.entry + (how == kSymmetric ? 1 + t.which : t.step & 1);
      const int which_map = (int)(map - p.maps);
      if (which_map >= 32 || !(fenced >> which_map & 1)) {
        tma_map_fence(map);
        if (which_map < 32) fenced |= 1u << which_map;
      }
      const int m0 = (side ? t.j : t.i) * kTile, at = uniform(m0 + (int)rank * 128);
      const int turn = uniform(across_from<kPair>(how, m0));
      const int other_turn = uniform(across_from<kPair>(other, (side ? t.i : t.j) * kTile));
      const int from = uniform(t.from), depth = uniform(t.depth), b = uniform(t.b);
      const uint32_t need = t.need;
      // each waits for the device's count itself: a shared word between them
      // would be one more step before the first load
      if (need) {
        ok = __all_sync(0xffffffffu, count_wait(p.c.done + t.unit, need, fault));
        if (!ok) break;
        fence_proxy_async();
      }
      // The epilogue's second part of X, which no operand brings: this CTA's 128
      // rows of the tile are one run.  For products that are over before it has
      // come.  (36 of 11840x80: 603 us without, 540 with it; 2304x768 x 12 340 and
      // 335, 768x2304 x 24 618 and 616; but 3000x1000 x 12 623 and 632, 4096x2048 x 4
      // 940 and 957, the step on seven matrices 4096 deep 11.40 and 11.54 ms, and
      // 768x768 x 12, whose X stays in L2, 166 and 172.)
      if (p.far && side && t.which == 2 && depth <= 768) {
        const int row = t.i * kTile + (int)rank * 128, col = t.j * kTile;
        if (row < t.e.rows && elected())
          prefetch_l2(t.e.lo + b * block_size(t.e.rows, t.e.ldx) + block_at(row, col, t.e.ldx),
                      min(kTile, (int)t.e.ldx - col) * 256);
        __syncwarp();
      }
      for (int k0 = from; k0 < depth; k0 += kDepth) {
        ok = __all_sync(0xffffffffu, mbar_wait(empty + 8 * s, phase, fault));
        if (!ok) break;
        const uint32_t bar = kPair == 2 ? peer(full + 8 * s, 0) : full + 8 * s;
        const uint32_t to = stages + s * kStageBytes + side * kOperandBytes;
        const bool x = k0 >= turn;
        // a box along the rows that would lie beyond the depth is left out
        const bool both = depth - k0 > 64;
        if (elected()) {
          if (rank == 0 && side == 0)
            mbar_expect(full + 8 * s, kPair * kBoxBytes * (2 + (both || x) + (both || k0 >= other_turn)));
          const int down = (x ? k0 : at) / 128, right = (x ? at : k0) / 8;
          tma_load<kPair>(to, map, bar, right, down, b);
          if (both || x) tma_load<kPair>(to + kBoxBytes, map, bar, right + 8, down, b);
        }
        __syncwarp();
        if (side == 0 && k0 == from && lane == 0) shared_set(told, n + 1);
        ++issued;
        if (++s == kStages) { s = 0; phase ^= 1; }
      }
    }
    // Every stage that was filled is released (or, after a fault, has at
    // least arrived) before the CTA may end.
    if (ok) {
      for (uint32_t q = 0; ok && q < kStages && q < issued; ++q) {
        ok = mbar_wait(empty + 8 * s, phase, fault);
        if (++s == kStages) { s = 0; phase ^= 1; }
      }
    }
    if (!ok && rank == 0 && side == 0) {
      const uint64_t t0 = now_ns();
      const uint32_t held = issued < kStages ? issued : kStages;
      for (uint32_t at = issued - held; at < issued; ++at) {
        while (!mbar_try(full + 8 * (at % kStages), at / kStages & 1) && now_ns() - t0 < 1000000000ull) {
        }
      }
    }
  } else if (warp == 1 && rank == 0) {
    // ---- products.  The warp walks together; one lane issues.
    uint32_t s = 0, phase = 0, acc = 0, acc_phase = 1;
    bool ok = true;
    for (uint32_t n = 0; ok && n < mine; ++n) {
      ok = __all_sync(0xffffffffu, shared_wait(known, n + 1, fault));
      if (!ok) break;
      const Tile& t = slots[n % kSlots];
      const int ta = uniform(across_from<kPair>(side_of(t.e, t.which, 0), t.i * kTile));
      const int tb = uniform(across_from<kPair>(side_of(t.e, t.which, 1), t.j * kTile));
      const int from = uniform(t.from), depth = uniform(t.depth);
      ok = __all_sync(0xffffffffu, mbar_wait(acc_empty + 8 * acc, acc_phase, fault));
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = tmem + acc * kTile;
      for (int k0 = from; k0 < depth; k0 += kDepth) {
        const bool xa = k0 >= ta, xb = k0 >= tb;
        const uint32_t idesc = instruction(kTile, kTile, xa, xb);
        const uint32_t at = stages + s * kStageBytes;
        // core matrices: 128 bytes from eight rows to the next, kPieceBytes from piece to piece
        const auto desc = [](uint32_t addr, bool x) {
          return x ? operand(addr, 128, kPieceBytes) : operand(addr, kPieceBytes, 128);
        };
        const uint64_t da = desc(at, xa), db = desc(at + kOperandBytes, xb);
        ok = __all_sync(0xffffffffu, mbar_wait(full + 8 * s, phase, fault));
        if (!ok) break;
        tc_fence_after();
        if (elected()) {
          const auto four = [&](int q0) {
#pragma unroll
            for (int q = q0; q < q0 + 4; ++q) {
              // 16 deep: two pieces, or sixteen rows
              const uint32_t along = q * 2 * kPieceBytes >> 4, down = q * 2 * 128 >> 4;
              mma_f16<kPair>(d, da + (xa ? down : along), db + (xb ? down : along), idesc, k0 > from || q > 0);
            }
          };
          four(0);
          if (depth - k0 > 64) four(4);
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
    float* patch = patches + (warp - 4) * 512;
    for (uint32_t n = 0; n < mine; ++n) {
      // the tile before the last is counted: its barrier is free again
      bool ok = shared_wait(known, n + 1, fault) && (n < 2 || shared_wait(counted, n - 1, fault));
      ok = __all_sync(0xffffffffu, ok);
      const Outcome is = epilogue<kPair>(p, slots[n % kSlots], ok, told, n, tmem + acc * kTile, acc_full + 8 * acc, phase,
                           acc_empty + 8 * acc, warp - 4, lane, rank, patch, cols + acc * 256, stop + 1);
      ok = is != kFailed;
      if (!ok) *stop = 1;
      if (warp == 4 && lane == 0) stop[2 + acc] = is == kPart;
      // the tile's writes are made: warp 2 counts it
      asm volatile("barrier.arrive %0, %1;" ::"r"(2 + acc), "r"(32 * kEpiWarps + 32) : "memory");
      if (!ok) break;
      if (++acc == 2) { acc = 0; phase ^= 1; }
    }
  } else if (warp == 2) {
    // ---- count of finished tiles: waits for the epilogue's writes to be
    // visible to the device, so that its warps need not
    for (uint32_t n = 0; n < mine; ++n) {
      asm volatile("barrier.sync %0, %1;" ::"r"(2 + n % 2), "r"(32 * kEpiWarps + 32) : "memory");
      if (*stop) break;
      if (lane == 0) {
        const uint32_t unit = (uint32_t)slots[n % kSlots].unit;
        const bool whole = !stop[2 + n % 2];
        shared_set(counted, n + 1);
        if (whole) asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(p.c.done + unit) : "memory");
      }
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (kPair == 2) cluster_sync();
  tc_fence_after();
  if (warp == 2) tmem_free<kPair>(tmem, kTmemCols);
}

}  // namespace zm
