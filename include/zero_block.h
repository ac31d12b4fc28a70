/*
 * zero_block.h -- C ABI of the rows between a block's matrix products: the
 * block's output joined to the residual stream, the norms before and after it,
 * its gate, its scale and its dropout in one pass, and dropout by itself.
 *
 * For every token t, with x its row of the stream and y the block's output, D
 * numbers each:
 *   z  = y * ry * y_gain,  ry = 1 / sqrt(mean(y^2) + eps)   (norm_branch 1)
 *        y * y_gain                                         (norm_branch 0)
 *   b  = drop(beta * z * act(gate))
 *   x' = alpha * x + b
 *   h  = x' * r * gain,    r = 1 / sqrt(mean(x'^2) + eps)   (norm_out 1)
 * act(gate) is 1 (ZERO_GATE_NONE), the gate itself (PLAIN) or
 * 1 / (1 + exp(-gate)) (SIGMOID).  Without y the row is only normalised: x' = x.
 *
 * Backward, from dx' and dh, with xhat = x' * r and yhat = y * ry (or y):
 *   G     = dx' + r * (dh * gain - xhat * mean(dh * gain * xhat))
 *   dx    = alpha * G                     (G without y)
 *   db    = beta * drop(G)
 *   dgate = db * yhat * y_gain * act'(gate)
 *   dz    = db * act(gate)
 *   dy    = ry * (dz * y_gain - yhat * mean(dz * y_gain * yhat))   or dz * y_gain
 *   dy_gain = sum over tokens of dz * yhat,   dgain = sum over tokens of dh * xhat
 *
 * Dropout.  Number d of row t is kept where the 16-bit half d % 8 of the eight
 * (of each of the four words the lower half first) that Philox 4x32 with ten
 * rounds (Salmon, Moraes, Dror, Shaw: "Parallel random numbers: as easy as 1, 2,
 * 3", 2011) makes of
 *   counter  (low and high word of t * ceil(D / 8) + d / 8, call, low word of step)
 *   key      (low and high word of seed)
 * is at least c = floor(65536 p + 0.5); it is then multiplied by
 * 65536 / (65536 - c), and is zero otherwise, whatever it held (p is taken to
 * the nearest 65536th; at 1 everything is zero).  No mask is stored: the backward
 * pass makes the same bits from the same zero_rng, so a program gives each
 * dropout of a step its own `call`, and each step its own `step`.  Every call's rows
 * are counted from 0: the micro-batches of a step, and the shards that ranks have of a
 * batch or of a sequence, drop the same places unless each has a `seed` or `call` of its
 * own, and no call makes the bits that a part of a larger tensor's rows would get.
 *
 * A token whose mask byte is zero is padding: what its inputs hold (NaN and
 * infinity included) is ignored, its results and gradients are zero and it adds
 * nothing to the gains' gradients.
 *
 * Arithmetic is binary32 throughout.  Of every row the squares have to be within
 * its range, numbers from about 1e-18 to 1e18: of x', y, dx', dh * gain, and of the
 * branch behind its norm, z * act(gate), where it has one (products of one with
 * another then are, whatever each one's size).  Results are rounded once, to their
 * tensor's type; h comes from x' before its rounding.  A sigmoid is within 10 2^-24 of
 * itself, but where only 16-bit numbers and the gains' gradients come of it: there up
 * to (10 + 2.4 |gate|) 2^-24.  The gains' gradients are binary32.  Sums, over a row's
 * numbers and over tokens, are taken in an order fixed by the shapes, the device, which
 * tensors are given, and whether all their rows begin on 16-byte boundaries; so equal
 * inputs in an equal layout give equal bits, and in another layout results within the
 * arithmetic's errors of them.
 *
 * Conventions are those of zero_opt.h: a zero_status from every call,
 * arguments checked before any CUDA work, device buffers owned by the caller,
 * asynchronous on `stream`, no allocation after zero_block_create.  Calls on one
 * handle are ordered (its workspace is one), and so are replays of graphs that
 * captured them.  All calls can be captured in a CUDA graph.
 */
#ifndef ZERO_BLOCK_H
#define ZERO_BLOCK_H

#include "zero_opt.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct zero_block_handle* zero_block_t;

#define ZERO_GATE_NONE 0
#define ZERO_GATE_PLAIN 1
#define ZERO_GATE_SIGMOID 2

/* What a dropout's bits are made from. */
typedef struct zero_rng {
  uint64_t seed;
  int64_t step;             /* its low 32 bits count                          */
  const int64_t* step_dev;  /* device; not NULL: read by the kernel in place
                               of `step`, so that a replayed graph's steps differ */
  uint32_t call;
  uint32_t reserved;
} zero_rng;

typedef struct zero_block_config {
  int32_t dim;              /* D: 1..16384; 8192 at most with dtype FP32, 12288 with
                               a gate and a binary32 stream beside 16-bit blocks */
  int32_t dtype;            /* y, gate, h and their gradients: ZERO_FP16/BF16/FP32 */
  int32_t stream_dtype;     /* x, x' and their gradients: `dtype` or ZERO_FP32 */
  int32_t norm_branch;      /* 1: y is normalised                             */
  int32_t norm_out;         /* 1: h is wanted                                 */
  int32_t gate;             /* ZERO_GATE_*                                    */
  int32_t reserved[2];
  double eps;               /* >= 0, added to the mean squares                */
  double alpha, beta;       /* finite in binary32; of the stream and of the branch */
  double dropout;           /* p: 0..1                                        */
} zero_block_config;

/* Rows of D contiguous numbers; the stride is in elements, from one token to
 * the next.  Inputs may be broadcast (stride 0).  A result may be an input of
 * the same call and the same type (same pointer and stride); otherwise results
 * must not overlap inputs or one another. */
typedef struct zero_block_rows {
  void* data;               /* device                                         */
  int64_t stride;
} zero_block_rows;

typedef struct zero_block_buffers {
  int64_t tokens;           /* T >= 0                                         */
  zero_block_rows x;        /* forward: the stream                            */
  zero_block_rows y;        /* the block's output; NULL: none                 */
  zero_block_rows gate;     /* ignored with ZERO_GATE_NONE or without y       */
  zero_block_rows x_out;    /* x'.  forward: result (NULL: not wanted;
                               ignored without y); backward: input (without y: x) */
  zero_block_rows h;        /* forward: result, with norm_out                 */
  zero_block_rows dx_out;   /* backward: gradient of x' (NULL: zero)          */
  zero_block_rows dh;       /* backward: gradient of h (NULL: zero)           */
  zero_block_rows dx, dy, dgate; /* backward: results (NULL: not wanted)      */
  const float* y_gain;      /* device fp32 [D]; NULL: ones.  Ignored without y */
  const float* gain;        /* device fp32 [D]; NULL: ones.  Ignored without h or dh */
  float* dy_gain;           /* backward: device fp32 [D]; NULL: not wanted    */
  float* dgain;             /* backward: device fp32 [D]; NULL: not wanted    */
  const uint8_t* mask;      /* device [T]; NULL: every token counts           */
  zero_rng rng;             /* looked at with dropout > 0 and y               */
} zero_block_buffers;

/* Errors: EINVAL (NULL pointers, a field outside the ranges above); ENOMEM;
 * ECUDA.  *out is NULL on failure.  Without a CUDA device the handle is created
 * and every launching call returns ZERO_ECUDA.  The gradients' workspace is allocated
 * here, for handles that only go forward too: 8 D bytes for each of up to four CTAs
 * an SM, 10 MB at 4096 numbers and 20 MB at most on 152 SMs.  Creating waits for the
 * legacy default stream, so not while a capture is under way. */
zero_status zero_block_create(const zero_block_config* cfg, zero_block_t* out);
zero_status zero_block_destroy(zero_block_t h);

/* Errors of both: EINVAL (NULL handle or buffers, T < 0; with T > 0 a tensor
 * that the call needs is NULL: x, the gate with y, h with norm_out, forward no
 * result wanted, backward x', both dx' and dh (dx' alone without norm_out); a
 * result's stride that lays rows on one another; a pointer that its type's size
 * does not divide), ECUDA (no device, another device current, a launch failure).
 * T = 0 launches nothing, except that the backward call sets the gains' gradients
 * to zero. */
zero_status zero_block_join(zero_block_t h, const zero_block_buffers* b, void* stream);
zero_status zero_block_join_backward(zero_block_t h, const zero_block_buffers* b, void* stream);

/* Kernels launched by this handle since creation. */
zero_status zero_block_launch_count(zero_block_t h, int64_t* launches);

/* Dropout of a [rows, cols] tensor by the rule above (t the row, D = cols);
 * of a gradient the same call with the same rng.  A flat tensor is one row.
 * Without a handle: on the current device, any number of calls at a time. */
typedef struct zero_drop_buffers {
  const void* in;           /* device                                         */
  void* out;                /* device; `in` itself (same stride), or apart from it */
  int64_t rows, cols;       /* >= 0                                           */
  int64_t in_stride, out_stride; /* elements from one row to the next         */
  int32_t dtype;            /* ZERO_FP16/BF16/FP32                            */
  int32_t reserved;
  double p;                 /* 0..1                                           */
  zero_rng rng;
} zero_drop_buffers;

/* Errors: EINVAL (NULL, a field outside the ranges above, a NULL or misaligned
 * pointer, rows of the result on one another), ECUDA. */
zero_status zero_dropout(const zero_drop_buffers* b, void* stream);

#ifdef __cplusplus
}
#endif
#endif
