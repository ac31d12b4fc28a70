/*
 * zero_qk.h -- C ABI of the query/key normalisation with the position rotation.
 *
 * For every token t and head h, with x the head's D numbers:
 *   r = 1 / sqrt(mean(x^2) + eps)
 *   y = x * r * gain                              (gain: D numbers, or D a head)
 *   out = y with its first `rotary_dim` numbers rotated by the token's
 *         position p: the pair (u, v) of angle j becomes
 *         (u cos[p][j] - v sin[p][j], v cos[p][j] + u sin[p][j]).
 * Pairs: number j with number j + rotary_dim/2 (interleaved 0), or numbers 2j
 * and 2j+1 (interleaved 1); j < rotary_dim/2.
 *
 * Backward, with dy the gradient of `out` rotated back:
 *   dgain = sum over tokens (and heads, for a shared gain) of dy * x * r
 *   dx    = r * (dy * gain - x * r * mean(dy * gain * x * r))
 *
 * A handle of zero_qk_create_axes turns each pair by the position that the token
 * has on that pair's axis (time, height, width of a video's patch, ...), and may
 * leave the norm out (y = x), so that rows are only rotated.
 *
 * A token whose position (any of them) is negative is padding: what its inputs hold (NaN
 * and infinity included) is ignored, its outputs and gradients are zero and it adds nothing to the gains' gradients.
 * A position (any) of n_pos or more has no angle: the token's rows come out as NaN.
 *
 * Arithmetic is binary32 throughout (a row's squares have to be within its
 * range: numbers from about 1e-18 to 1e18); results are rounded once, to the
 * data's type.  The gains' gradients are binary32.  Sums, over a row's numbers and over
 * tokens, are taken in an order fixed by the shapes, the device and the widest vector
 * (16 bytes down to one number) that all addresses and strides are multiples of; so
 * equal inputs in an equal layout give equal bits, and in another layout results within
 * the arithmetic's errors of them.
 *
 * Conventions are those of zero_opt.h: a zero_status from every call,
 * arguments checked before any CUDA work, device buffers owned by the caller,
 * asynchronous on `stream`, no allocation after zero_qk_create, calls on one
 * handle ordered.  Both calls can be captured in a CUDA graph.
 */
#ifndef ZERO_QK_H
#define ZERO_QK_H

#include "zero_opt.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct zero_qk_handle* zero_qk_t;

typedef struct zero_qk_config {
  int32_t q_heads;          /* >= 1; q_heads + k_heads <= 4096               */
  int32_t k_heads;          /* >= 0; 0: queries only (k pointers ignored)    */
  int32_t head_dim;         /* D: even, 2..512                               */
  int32_t rotary_dim;       /* even, 0..D; the rest is only normalised       */
  int32_t dtype;            /* q, k and their gradients: ZERO_FP16/BF16/FP32 */
  int32_t interleaved;      /* pairs: 0 (j, j + rotary_dim/2); 1 (2j, 2j+1)  */
  int32_t gain_per_head;    /* 0: one gain of D for all query heads and one
                               for all key heads; 1: D for each head         */
  int32_t reserved;
  double eps;               /* >= 0, added to the mean square                */
} zero_qk_config;

/* One call's tensors.  Strides are in elements; a head's D numbers are
 * contiguous.  Outputs may be the inputs themselves (same pointer and
 * strides); otherwise they must not overlap them. */
typedef struct zero_qk_tensor {
  void* data;               /* device                                        */
  int64_t token_stride;     /* elements from one token to the next           */
  int64_t head_stride;      /* elements from one head to the next            */
} zero_qk_tensor;

typedef struct zero_qk_buffers {
  int64_t tokens;           /* T >= 0                                        */
  int64_t n_pos;            /* rows of the tables (>= 0)                     */
  zero_qk_tensor q, k;      /* inputs: [T][q_heads][D], [T][k_heads][D]      */
  zero_qk_tensor q_out, k_out; /* forward: results.  backward: gradients of
                               the results (inputs)                          */
  zero_qk_tensor dq, dk;    /* backward: gradients of q and k                */
  const float* q_gain;      /* device fp32, [D] or [q_heads][D]; NULL: ones  */
  const float* k_gain;      /* device fp32, [D] or [k_heads][D]; NULL: ones  */
  float* dq_gain;           /* backward: gradients of the gains, as the      */
  float* dk_gain;           /*   gains; NULL: not wanted                     */
  const float* cos;         /* device fp32 [n_pos][rotary_dim/2]             */
  const float* sin;         /* device fp32 [n_pos][rotary_dim/2]             */
  const void* positions;    /* device int32 or int64 [T]; with axes [axes][T] */
  int32_t positions64;      /* 1: int64                                      */
  int32_t reserved;
} zero_qk_buffers;

/* Errors: EINVAL (NULL pointers, a dtype not named above, a count or size
 * outside the ranges above, eps < 0 or NaN); ENOMEM; ECUDA.  *out is NULL on
 * failure.  Without a CUDA device the handle is created and every launching
 * call returns ZERO_ECUDA. */
zero_status zero_qk_create(const zero_qk_config* cfg, zero_qk_t* out);

/* Positions on several axes.  Pair j < rotary_dim/2 turns by
 * cos[p[axis[j]]][j], sin[p[axis[j]]][j], p the token's positions; each axis
 * below n_pos, and n_pos below 2^31.  Without the norm (normalise 0) there are no
 * gains (their pointers, and their gradients', are NULL), eps is not used, and the
 * backward call looks at neither q nor k.
 * Errors: those of zero_qk_create; EINVAL (NULL axes, a field out of range). */
typedef struct zero_qk_axes {
  int32_t axes;             /* 1..4                                          */
  int32_t normalise;        /* 1: as zero_qk_create; 0: rotation alone       */
  uint8_t axis[256];        /* of each pair: 0..axes-1                       */
} zero_qk_axes;
zero_status zero_qk_create_axes(const zero_qk_config* cfg, const zero_qk_axes* axes, zero_qk_t* out);

zero_status zero_qk_destroy(zero_qk_t h);

/* Errors of both: EINVAL (NULL handle or buffers; a NULL tensor with
 * T > 0; tokens or n_pos < 0; NULL tables with rotary_dim and n_pos > 0 or
 * NULL positions, T > 0; a result's token or head stride that lays rows on one
 * another; with axes n_pos of 2^31 or more, gains without the norm, positions off
 * their size's boundary), ECUDA (no device, another device current, a launch
 * failure).  T = 0 launches nothing, except that the backward call sets the
 * gains' gradients to zero. */
zero_status zero_qk_norm_rope(zero_qk_t h, const zero_qk_buffers* b, void* stream);
zero_status zero_qk_norm_rope_backward(zero_qk_t h, const zero_qk_buffers* b, void* stream);

/* Kernels launched by this handle since creation. */
zero_status zero_qk_launch_count(zero_qk_t h, int64_t* launches);

#ifdef __cplusplus
}
#endif
#endif
