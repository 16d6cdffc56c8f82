/*
 * gated_delta.h -- C ABI of the gated delta rule in libsss48.so.
 *
 * What it computes.  A recurrence beside the scans of selective_scan.h and
 * ssd.h whose transition is not diagonal: before a key's value is written,
 * what the state already holds for that key is read and replaced.  For every
 * sequence, head h (group g = h / (nheads / ngroups)), with the state
 * S (headdim x dstate):
 *
 *   a_t = exp(Delta_t A[h]),  Delta_t = softplus(dt[t,h] + dt_bias[h])
 *   b_t = sigmoid(beta[t,h])
 *   u_t = b_t (v_t - a_t S_{t-1} k_t)
 *   S_t = a_t S_{t-1} + u_t k_t^T
 *   y_t = scale * S_t q_t
 *
 * with S before the first step = h0 (or 0).  softplus and sigmoid are
 * optional (dt_softplus, beta_sigmoid: 0 takes the values as they are).
 * Keys are expected to have length about 1 and b_t to lie in [0, 2]: the
 * transition a_t (I - b_t k_t k_t^T) then does not grow the state.  The
 * nheads / ngroups consecutive heads of a group share q and k.
 *
 * How.  Two evaluations of the same map:
 *   recurrent  step by step, the state in registers (fp32 throughout); every
 *              size and type below;
 *   chunked    64 steps at a time on the tensor cores.  With c_t the running
 *              sum of log a inside the chunk, the written rows u solve the
 *              unit lower triangular system
 *                (I + A) U = diag(b) (V - diag(e^c) K H0^T),
 *                A[t,s] = b_t e^(c_t - c_s) (k_t . k_s)   for s < t,
 *              and then Y = diag(e^c) Q H0^T + (Q K^T o e^(c_t - c_s)) U and
 *              S = e^(c_last) H0 + U^T diag(e^(c_last - c)) K.  Operands that
 *              are not bf16 already enter the products as the sum of two
 *              bf16 values, off by 2^-18 of an operand at most, or of three
 *              where that would show: last_state and an fp32 y are off by
 *              about 1e-6 of their size (states that decay slowly, and keys
 *              that lie close together, several times that, in the recurrent
 *              evaluation too).  With a
 *              workspace, long sequences of few heads are cut into segments
 *              that run beside each other: the state passes a segment as
 *              S_end = S_start M + B, with M and B from a first pass.
 *              The running sums c are pairs of fp32 values, so a decay is as
 *              exact behind a step that wipes the state as anywhere else;
 *              log2 a of a step counts as -300 where it is below (a is 0 in
 *              fp32 from -150 on).
 * A NaN in a step's inputs, or an infinity (but in a Delta_t A[h] of minus
 * infinity, which is a decay of 0), spoils that head from the step on
 * (recurrent) or from the first step of its chunk on (chunked), nothing else.
 *
 * Layouts (the last dimension contiguous; batch, step and head strides in
 * elements are given per tensor, so views of a wider projection are read in
 * place):
 *   q, k       (batch, seqlen, ngroups, dstate)   in_dtype
 *   v, y       (batch, seqlen, nheads, headdim)   in_dtype (y: out_dtype)
 *   dt, beta   (batch, seqlen, nheads)            in_dtype
 *   A, dt_bias (nheads)                           fp32 (dt_bias optional)
 *   h0, last_state (sequences, nheads, headdim, dstate) fp32, dense, optional;
 *              they may be the same memory
 * Packed sequences: with cu_seqlens (num_seqs + 1 ascending int32 offsets on
 * the device, within [0, seqlen]; others are clamped to it) batch must be 1
 * and sequence i is the steps cu_seqlens[i] .. cu_seqlens[i+1] - 1, each with
 * its own h0 and last_state; an empty one hands h0 (or 0) to last_state.
 * Rows of y outside every sequence are not written.
 * Limits: dstate <= 256, any headdim.  Pointers are aligned to their element
 * size.  Sizes of 0 are errors.  The chunked evaluation takes bf16 inputs with dstate a multiple of 8
 * up to 128, headdim a multiple of 8, q, k, v 16-byte aligned and their
 * strides multiples of 8; everything else runs the recurrent one, or,
 * with a workspace and dstate <= 128, is copied first.
 *
 * Ownership, streams and errors as in selective_scan.h: device pointers owned
 * by the caller, nothing allocated, work enqueued on `stream` without
 * synchronising; argument errors enqueue nothing.  Outputs must not overlap
 * inputs, except last_state = h0.  The chunked kernel's waits are bounded
 * (spin_timeout_ns, 0 = 2 s; counted in tries of 4 us); one that runs out is
 * recorded in a library status word (one per device) read and cleared by
 * mss_gated_delta_status().  y and last_state are then not to be used.  Copies
 * and products in flight are waited for all the same, for up to 2 s.
 */
#ifndef SSS48_GATED_DELTA_H
#define SSS48_GATED_DELTA_H

#include <stdint.h>

#include "selective_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

/* mss_delta_args.plan: which evaluation runs */
/* AUTO: chosen by type, sizes, alignment and length; of packed sequences by
 * their average length, seqlen / num_seqs, so a pack of a long one and many
 * short ones may be better off with CHUNKED */
#define MSS_DELTA_AUTO 0
#define MSS_DELTA_RECURRENT 1
#define MSS_DELTA_CHUNKED 2   /* MSS_ERR_UNSUPPORTED where it does not apply */

typedef struct mss_delta_args {
  int64_t batch;
  int64_t seqlen;
  int64_t nheads;
  int64_t headdim;
  int64_t ngroups; /* divides nheads */
  int64_t dstate;
  mss_dtype in_dtype;
  mss_dtype out_dtype;
  const void *q;
  const void *k;
  const void *v;
  const void *dt;
  const float *A;
  const void *beta;
  const float *dt_bias; /* NULL: 0 */
  int dt_softplus;
  int beta_sigmoid;
  float scale;
  const float *h0;      /* NULL: the state starts at 0 */
  void *y;
  float *last_state;    /* NULL: not written */
  int64_t stride_q[3];  /* {batch, step, group}, elements, >= 0 */
  int64_t stride_k[3];
  int64_t stride_v[3];  /* {batch, step, head} */
  int64_t stride_dt[3];
  int64_t stride_beta[3];
  int64_t stride_y[3];  /* rows of y must not overlap */
  const int32_t *cu_seqlens; /* NULL: every batch row is one sequence */
  int64_t num_seqs;
  int plan;
  uint64_t spin_timeout_ns;
  void *workspace;      /* optional; 16-byte aligned */
  size_t workspace_bytes;
} mss_delta_args;

/* Forward over whole sequences: y (and last_state). */
mss_status gated_delta_fwd(const mss_delta_args *args, void *stream);

/* Bytes of workspace that the call gains from on the current device (0:
 * nothing).  With one, long sequences of few heads are cut into segments that
 * run beside each other, and bf16 q, k, v of sizes, strides or addresses that
 * the chunked evaluation does not take are copied for it (MSS_DELTA_AUTO).
 * Without one every sequence runs whole, those recurrently.  One that is too
 * small is MSS_ERR_WORKSPACE.  Of the tensors only the strides and whether
 * pointers are 16-byte aligned matter here. */
mss_status mss_gated_delta_workspace_size(const mss_delta_args *args, size_t *bytes);

typedef struct mss_delta_update_args {
  int64_t batch;
  int64_t nheads;
  int64_t headdim;
  int64_t ngroups;
  int64_t dstate;
  mss_dtype in_dtype;
  mss_dtype out_dtype;
  float *state;         /* (batch, nheads, headdim, dstate), in place */
  const void *q;        /* (batch, ngroups, dstate) */
  const void *k;
  const void *v;        /* (batch, nheads, headdim) */
  const void *dt;       /* (batch, nheads) */
  const float *A;
  const void *beta;
  const float *dt_bias; /* NULL: 0 */
  int dt_softplus;
  int beta_sigmoid;
  float scale;
  void *y;              /* (batch, nheads, headdim) */
  int64_t stride_q[2];  /* {batch, group}, elements, >= 0 */
  int64_t stride_k[2];
  int64_t stride_v[2];  /* {batch, head} */
  int64_t stride_dt[2];
  int64_t stride_beta[2];
  int64_t stride_y[2];  /* rows of y must not overlap */
} mss_delta_update_args;

/* One token for every batch row: the state is updated in place. */
mss_status gated_delta_update(const mss_delta_update_args *args, void *stream);

/* Synchronises `stream` and returns the chunked kernel's device status word
 * (MSS_OK or MSS_ERR_TIMEOUT), clearing it; as mss_ssd_status. */
mss_status mss_gated_delta_status(void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SSS48_GATED_DELTA_H */
