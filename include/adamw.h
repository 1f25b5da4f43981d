/* adamw.h -- one AdamW step over many tensors on one GB300 (part of
 * libbirkhoff4.so).
 *
 *   g <- g * grad_scale                         (if grad_scale is given)
 *   m <- beta1 m + (1 - beta1) g
 *   v <- beta2 v + (1 - beta2) g^2
 *   p <- p (1 - lr weight_decay)
 *        - lr / (1 - beta1^step) m / (sqrt(v / (1 - beta2^step)) + eps)
 *
 * Arithmetic is fp32; beta, 1 - beta and the step's other factors are worked
 * out in fp64 and rounded once.  The moments' updates round every product
 * and sum by itself (no fused multiply-add), so they can be reproduced bit for
 * bit.
 *
 * Weights p and gradients g are B4_F32 or B4_BF16.  With `master` given the
 * step is taken on fp32 master weights, and p (bf16) is their rounded copy;
 * without it bf16 weights are widened, updated and rounded to nearest.
 *
 * Moments are fp32 (state_bits 32), or e4m3 numbers with one fp32 scale for
 * ADAMW_BLOCK consecutive elements (state_bits 8): the first moment m, and
 * the root sqrt(v) of the second, which has half of v's range of exponents.
 * A block's scale is the largest finite magnitude in it times the fp32 number
 * 1/448 (448 is e4m3's largest), and a code is the nearest e4m3 number to
 * value * (448 * (1 / largest)), ties to even, every operation rounded.
 * sqrt(v) > 0 never becomes 0: it is at least e4m3's smallest number, so that
 * a denominator does not vanish under a first moment that is kept.  A value
 * that is not finite is stored as e4m3's NaN and leaves the others of its
 * block alone.
 *
 * Layout: every tensor is n contiguous elements.  Any alignment of the
 * element type is taken; tensors on 16-byte boundaries are fastest.
 *
 * Errors (return values, from birkhoff4.h): B4_EINVAL for a NULL pointer with
 * work to do, a negative count, n outside 0..ADAMW_MAX_ELEMENTS, an unknown type, state_bits or hyperparameter
 * outside its range (beta1, beta2 in [0, 1), eps >= 0, lr and weight_decay
 * finite and >= 0, step >= 1), a pointer that is not aligned to its element;
 * B4_ENOTIMPL for master weights beside fp32 weights; B4_ECUDA for a launch
 * error.  Everything is checked before the first launch.  Work is
 * asynchronous on `stream`; the tables of pointers travel in the launches'
 * own arguments, so a captured step replays on the same tensors, and with the
 * same number of the step and learning rate.
 */
#ifndef ADAMW_H
#define ADAMW_H

#include <stddef.h>
#include <stdint.h>

#include "birkhoff4.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ADAMW_BLOCK 128
#define ADAMW_MAX_ELEMENTS (INT64_C(1) << 40) /* of one tensor */

typedef struct {
  void *p;        /* weights [n] */
  const void *g;  /* gradients [n] */
  void *m, *v;    /* moments [n]: fp32, or e4m3 codes of m and of sqrt(v) */
  float *m_scale, *v_scale; /* state_bits 8: [ceil(n / ADAMW_BLOCK)] each */
  float *master;  /* fp32 master weights [n] or NULL: all or none */
  int64_t n;
} adamw_tensor;

typedef struct {
  int32_t p_dtype, g_dtype, state_bits;
  double lr, beta1, beta2, eps, weight_decay;
  int64_t step;            /* number of this step, from 1 */
  const float *grad_scale; /* device scalar or NULL */
} adamw_opts;

int adamw_step(const adamw_tensor *tensors, int32_t count, const adamw_opts *opts,
               birkhoff4_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* ADAMW_H */
