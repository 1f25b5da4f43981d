/* hc_block.h -- the operators around one block of a network with
 * hyper-connections, on one GB300 (part of libbirkhoff4.so).
 *
 * The residual of such a network is S streams of C channels per token,
 * x [T, S, C].  A block reads one row of C channels and writes one:
 *
 *   enter         u = sum_s a_s x_s
 *                 h = w u / sqrt(mean_c u^2 + eps)
 *   leave         z = w y / sqrt(mean_c y^2 + eps)   (norm != 0; else z = w y)
 *                 v = scale act(gate) z
 *                 x'_i = sum_j P_ij x_j + b_i v
 *   leave_enter   leave, then the next block's enter on x' as it is stored:
 *                 u = sum_i a_i x'_i, h = w_next u / sqrt(mean_c u^2 + eps_next)
 *
 * P [T, S, S] is the projected mixing matrix (birkhoff4_forward), a, b [T, S]
 * the read and write coefficients.  With S = 1 and no P, a and b these are
 * the norms before and after a block of an ordinary residual network.
 *
 * Gradients.  With D = dL/dx' and G = w dh:
 *   enter  k = mean(G u) / (mean u^2 + eps), r = 1/sqrt(mean u^2 + eps),
 *          du = r (G - k u), dx_s = a_s du + dres_s, da_s = <du, x_s>,
 *          dw = sum_t r u dh
 *   leave  dx_j = sum_i P_ij D_i, dP_ij = <D_i, x_j>, db_i = <D_i, v>,
 *          dv = sum_i b_i D_i, dz = scale act(gate) dv,
 *          dgate = scale act'(gate) z dv, dy and dw from dz as above
 * Nothing of the forward pass is stored but its inputs (leave_enter: and its
 * output out): a row's statistics are recomputed in the pass that needs them.
 *
 * Types.  x, out, dout, dres and dx have x_dtype; y, gate, h, dh, dy and
 * dgate have y_dtype; both B4_F32 or both B4_BF16, or x B4_F32 with y
 * B4_BF16.  w, w_next (and dw, dw_next) have w_dtype, wn_dtype; P, a, b (and
 * their gradients) have p_dtype, a_dtype, b_dtype: B4_F32 or B4_BF16.  All
 * arithmetic is fp32, each result is rounded once; leave_enter computes h
 * from x' as stored.
 *
 * Layout.  Channels are contiguous.  Inputs have strides, in elements: of
 * tokens (*_ts) and of streams (*_ss); a stride of 0 repeats a row.  P has
 * its S x S matrix contiguous, a and b their S coefficients.  Outputs are
 * contiguous.  Any alignment of the element type is taken; rows on 16-byte
 * boundaries with a row length that is a multiple of 16 bytes are fastest.
 *
 * Optional pointers (NULL): a (all ones), P (identity), b (all ones), gate
 * (act = HCB_ACT_NONE), w and w_next (ones), dres (zero); and any gradient
 * that is not wanted, but dx with dres or with dh.  leave's backward with P ==
 * NULL and without dh has dx == dout: dx is only written if it is given.
 *
 * Errors (return values, from birkhoff4.h): B4_EINVAL for a NULL pointer with
 * work to do, T outside 0..2^31 - 1, S outside 1..8, C outside
 * 1..HCB_MAX_CHANNELS, a negative or non-finite eps, a non-finite scale, a
 * stride outside 0..2^29 - 1, an unknown type or act, a pointer that is not
 * aligned to its element, or a workspace that is too small or not 16-byte
 * aligned; B4_ENOTIMPL for x B4_BF16 with y B4_F32; B4_ECUDA for a launch
 * error.  T == 0 writes zeros to
 * dw and dw_next and does nothing else.  Work is asynchronous on `stream`;
 * the library allocates nothing.  Outputs may not overlap the inputs, but
 * dx may be dres or dout (same strides), and dy may be y.
 */
#ifndef HC_BLOCK_H
#define HC_BLOCK_H

#include <stddef.h>
#include <stdint.h>

#include "birkhoff4.h"

#ifdef __cplusplus
extern "C" {
#endif

#define HCB_MAX_STREAMS 8
#define HCB_MAX_CHANNELS 16384

#define HCB_ACT_NONE 0    /* no gate */
#define HCB_ACT_SIGMOID 1 /* 1 / (1 + e^-gate) */
#define HCB_ACT_SILU 2    /* gate / (1 + e^-gate) */
#define HCB_ACT_LINEAR 3  /* the gate itself */

typedef struct {
  int64_t T;
  int32_t S, C;
  int32_t x_dtype, y_dtype, w_dtype, wn_dtype, p_dtype, a_dtype, b_dtype;
  int32_t act, norm;
  float eps, eps_next, scale;
  /* inputs */
  const void *x, *y, *gate, *P, *a, *b, *w, *w_next;
  const void *dout, *dh, *dres, *out_in; /* out_in: leave_enter's stored x' */
  int64_t x_ts, x_ss, y_ts, gate_ts, P_ts, a_ts, b_ts;
  int64_t dout_ts, dout_ss, dh_ts, dres_ts, dres_ss, out_ts, out_ss;
  /* outputs */
  void *h, *out, *dx, *dy, *dgate, *dP, *da, *db, *dw, *dw_next;
  /* scratch of the backward passes (hcb_workspace_bytes) */
  void *workspace;
  size_t workspace_bytes;
} hcb_args;

/* Bytes of workspace that a backward pass over T tokens of C channels needs:
 * partial weight gradients, `weights` (0, 1 or 2) rows of C per CTA.  0 if
 * nothing is needed or the sizes are invalid. */
size_t hcb_workspace_bytes(int64_t T, int32_t C, int32_t weights);

/* h from x, a, w. */
int hcb_enter(const hcb_args *args, birkhoff4_stream_t stream);
/* dx, da, dw from dh, x, a, w, dres. */
int hcb_enter_backward(const hcb_args *args, birkhoff4_stream_t stream);
/* out from x, y, gate, P, b, w; and, if h is given, h from out, a, w_next. */
int hcb_leave(const hcb_args *args, birkhoff4_stream_t stream);
/* dx, dy, dgate, dP, db, dw from dout, x, y, gate, P, b, w; and, if dh is
 * given, the gradient of leave_enter: da and dw_next too, from out_in, a and
 * w_next, with dout's gradient and the one through h added in fp32. */
int hcb_leave_backward(const hcb_args *args, birkhoff4_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* HC_BLOCK_H */
