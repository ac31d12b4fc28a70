/*
 * zero_muon.h -- C ABI of the orthogonalised matrix update.
 *
 * For a matrix G of rows x cols, k the smaller and l the larger side, its
 * orthogonalised form O is found by `steps` Newton-Schulz steps:
 *   X = G / (|G|_F + eps)
 *   A = X X^T            (X^T X for a tall matrix: always k x k)
 *   X <- a X + (b A + c A A) X      (from the right for a tall matrix)
 * with the coefficients (a, b, c) of each step.  Every singular value of X is
 * taken through p(s) = a s + b s^3 + c s^5 while the singular vectors stay.
 *
 * zero_muon_step is the optimizer step built on it, for a list of matrices:
 *   g = grad * grad_scale * coef           (coef: the decision's, below)
 *   M = momentum * M + g
 *   U = nesterov ? g + momentum * M : M
 *   W = W * (1 - lr * weight_decay) - lr * s * O(U)
 *   param16 = W rounded to nearest even
 * s by scale_rule: ONE 1; RMS 0.2 sqrt(max(rows, cols)), which gives an
 * update the root mean square that AdamW's has; ASPECT sqrt(max(1, rows/cols)).
 *
 * Loss scale, clipping and overflow come from the step of the model's other
 * parameters: zero_opt_decision gives the device address of the decision that
 * zero_opt_step and its kin write, and zero_muon_step reads it there when it
 * runs on the stream.  With a skipped step nothing is read or written here
 * either; otherwise its coef (unscale times clip) multiplies the gradients.
 *
 * Numerics.  Products are of binary16 operands with binary32 sums; A and
 * b A + c A A are held times 4096, X times 64, which keeps them in
 * binary16's normal range for entries from 1.5e-8 (X: 1e-6) to 16 (a
 * coefficient set that takes singular values well beyond one, so that A or
 * b A + c A A pass 16, overflows to infinity and NaN).  X is held as the sum of
 * two binary16 numbers, of which the products take the first and the term a X
 * both, so that the many directions in which a gradient is small or zero are
 * not filled with rounding noise that p would blow up.  How far O may be from
 * the definition in 64 bits (Frobenius, relative): 4.8e-3 with the default
 * coefficients, where roundings average out, and that is with a shorter side
 * of 32 or more (measured: 0.4e-3 to 2.0e-3); 3.2e-2 below (measured: 2.7e-3
 * at most from 16 on, 4.6e-3 from 8, 1.4e-2 at 2 x 2, and 1e-3 to 3.3e-3 in the
 * mean square).  Binary32 results have no more than that; the master moves by
 * lr * s times it.  Norms are summed
 * in binary32 and binary64 (numbers whose squares leave binary32's range,
 * beyond about 1e19 or below 1e-19, are outside what the norm can tell), M
 * and W kept in binary32.  Equal inputs give equal bits.
 *
 * Conventions are those of zero_opt.h: a zero_status from every call,
 * arguments checked before any CUDA work, device buffers owned by the caller,
 * asynchronous on `stream`, the workspace allocated by zero_muon_create and
 * nothing after it, calls on one handle ordered (they share the workspace).
 * The calls can be captured in a CUDA graph.
 */
#ifndef ZERO_MUON_H
#define ZERO_MUON_H

#include "zero_opt.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct zero_muon_handle* zero_muon_t;

typedef enum zero_muon_scale {
  ZERO_MUON_SCALE_ONE = 0,
  ZERO_MUON_SCALE_RMS = 1,
  ZERO_MUON_SCALE_ASPECT = 2
} zero_muon_scale;

#define ZERO_MUON_MAX_STEPS 16
#define ZERO_MUON_MAX_SHAPES 256

typedef struct zero_muon_config {
  int32_t grad_dtype;       /* zero_muon_step: ZERO_FP16 or ZERO_BF16        */
  int32_t param_dtype;      /* zero_muon_step: ZERO_FP16 or ZERO_BF16        */
  int32_t nesterov;         /* 0 or 1                                        */
  int32_t steps;            /* 1..ZERO_MUON_MAX_STEPS                        */
  int32_t scale_rule;       /* zero_muon_scale                               */
  int32_t reserved;
  double lr;                /* >= 0                                          */
  double momentum;          /* in [0, 1)                                     */
  double weight_decay;      /* >= 0, decoupled                               */
  double eps;               /* >= 0, added to the norm; 0 makes a zero matrix
                               NaN                                           */
  double coef[ZERO_MUON_MAX_STEPS][3]; /* (a, b, c) of each step, finite     */
} zero_muon_config;

/* A matrix, or `batch` of one shape that lie one behind the other (the blocks
 * of heads, experts, the same weight of every layer). */
typedef struct zero_muon_shape {
  int64_t rows, cols;       /* 1..2^20 each, rows * cols <= 2^34             */
  int64_t batch;            /* 1..2^20                                       */
} zero_muon_shape;

/* zero_muon_orthogonalize: one per shape.  Strides in elements; the numbers
 * of a row are contiguous, and no two elements of an output may overlap. */
typedef struct zero_muon_operand {
  const void* in;           /* device, in_dtype                              */
  void* out;                /* device, out_dtype; may be `in` (same strides
                               and type)                                     */
  int64_t in_row, in_batch; /* from one row / matrix to the next             */
  int64_t out_row, out_batch;
} zero_muon_operand;

/* zero_muon_step: one per shape, every array contiguous [batch][rows][cols]. */
typedef struct zero_muon_matrix {
  const void* grad;         /* device, grad_dtype                            */
  float* momentum;          /* device fp32, read and written                 */
  float* master;            /* device fp32, read and written; NULL: param16
                               is the master (widened, updated, rounded)     */
  void* param16;            /* device, param_dtype, written                  */
} zero_muon_matrix;

/* What the last call of a handle did (zero_muon_last_step). */
typedef struct zero_muon_info {
  int32_t skipped;          /* 1: the decision said skip, nothing changed    */
  int32_t fault;            /* 1: a bounded wait ran out inside the kernels:
                               outputs (master, param16, O) are not to be
                               used; the momentum has been updated.  The next
                               call starts anew (zero_muon_fault_count)      */
} zero_muon_info;

/* lr 2e-2, momentum 0.95, Nesterov, weight decay 0, eps 1e-7, five steps of
 * (3.4445, -4.7750, 2.0315), scale ONE, fp16.  Errors: EINVAL (NULL). */
zero_status zero_muon_config_default(zero_muon_config* cfg);

/* Make a handle for n shapes (n = 0..ZERO_MUON_MAX_SHAPES) and its workspace:
 * about 6 bytes per element of the matrices, their rows rounded up to 128, and
 * 4 per element of the k x k products (almost nothing where every matrix has a
 * side of at most 128 and the other of at most 2048 and stays on the chip).
 * Errors: EINVAL (NULL pointers, a field outside its range), ERANGE (n or a
 * shape beyond the limits above), ENOMEM, ECUDA.  *out is NULL on failure.
 * Without a CUDA device the handle is created and every launching call
 * returns ZERO_ECUDA. */
zero_status zero_muon_create(const zero_muon_config* cfg, const zero_muon_shape* shapes,
                             int32_t n, zero_muon_t* out);
zero_status zero_muon_destroy(zero_muon_t h);

/* Device bytes of the handle's workspace.  Errors: EINVAL (NULL). */
zero_status zero_muon_workspace_bytes(zero_muon_t h, int64_t* bytes);

/* Learning rate of subsequent steps.  Errors: EINVAL (NULL, lr < 0). */
zero_status zero_muon_set_lr(zero_muon_t h, double lr);

/* O of every matrix.  items: one per shape of the handle.  in_dtype: ZERO_FP16,
 * ZERO_BF16 or ZERO_FP32; out_dtype likewise (binary32 results carry the
 * accuracy stated above).
 * Errors: EINVAL (NULL handle, items or pointer, a bad dtype, a row stride
 * below cols with rows > 1, an out_batch below cols with batch > 1, a negative
 * stride), ECUDA. */
zero_status zero_muon_orthogonalize(zero_muon_t h, const zero_muon_operand* items,
                                    int32_t in_dtype, int32_t out_dtype, void* stream);

/* The optimizer step.  items: one per shape of the handle.  grad_scale: finite,
 * rounded to binary32.  decision: DEVICE record (zero_opt_decision) or NULL:
 * no skip, coef 1.  Errors: EINVAL (NULL handle, items or a NULL array other
 * than master; grad_scale not finite), ECUDA. */
zero_status zero_muon_step(zero_muon_t h, const zero_muon_matrix* items, double grad_scale,
                           const zero_opt_step_info* decision, void* stream);

/* What the last call did.  Synchronizes `stream`.  Errors: EINVAL, ECUDA. */
zero_status zero_muon_last_step(zero_muon_t h, void* stream, zero_muon_info* out);

/* Calls of the handle that have ended in a fault since its creation, the last
 * one included: what a loop that does not ask after every step looks at now and
 * then.  Synchronizes `stream`.  Errors: EINVAL, ECUDA. */
zero_status zero_muon_fault_count(zero_muon_t h, void* stream, int64_t* faults);

/* Failure-detection test hook.  In the next call of this handle something is
 * waited for that never comes: through the workspace, by the tiles of every
 * product but the first, counts that are not reached; on the chip, by every
 * CTA, the end of its first product, which is not announced.  The waits run
 * out after their bound (two seconds), the kernel ends without
 * writing results and zero_muon_last_step reports fault = 1.  Nothing hangs,
 * the context stays usable and the next call is whole again.  Host only.
 * Errors: EINVAL (NULL). */
zero_status zero_muon_inject_wait_fault(zero_muon_t h);

/* Kernels launched by this handle since creation. */
zero_status zero_muon_launch_count(zero_muon_t h, int64_t* launches);

#ifdef __cplusplus
}
#endif
#endif
