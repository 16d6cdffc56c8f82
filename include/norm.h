/*
 * norm.h -- C ABI of the RMS norms before and after a sequence-mixing block
 * (a selective scan, an SSD scan or the gated delta rule) in libsss48.so.
 *
 * Before the block, fused with the residual stream:
 *   r = residual + scale o x          (stored in the residual's type)
 *   y = r / sqrt(mean(r^2) + eps) o weight
 * with a per-channel scale (optional) and the norm taken of the stored r.
 *
 * After the block, fused with its gate, per group of group_size channels:
 *   norm_before_gate 1:  y = (x / sqrt(mean(x^2) + eps) o weight) o silu(z)
 *   norm_before_gate 0:  a = x o silu(z),  y = a / sqrt(mean(a^2) + eps) o weight
 * The weight has width entries, or group_size entries that every group
 * shares (one weight per head channel).
 *
 * Gradients, with n = r rstd (or x rstd, a rstd), dn = dy o weight (times
 * silu(z) for norm_before_gate 1) and the mean over the group:
 *   d(normed) = rstd (dn - n mean(dn o n))
 *   add:   dresidual = d(normed) + dresidual_out, dx = scale o dresidual,
 *          dscale = sum over rows of dresidual o x
 *   gated: dz and dx by the product rule with
 *          silu'(z) = s (1 + z (1 - s)), s = sigmoid(z)
 *   dweight = sum over rows (and groups, if shared) of (d y / d weight) o dy
 * Statistics and sums are fp32; every output is rounded once.  The sums over
 * rows are taken in a fixed order (partial sums in the workspace, no
 * atomics), so a call gives the same bits every time.
 *
 * Layouts: (rows, width) tensors whose rows are contiguous, at any row stride
 * (in elements, >= 0 for inputs, >= width for outputs), so halves of a
 * projection are read in place.  x, z, y, dy, dx, dz have one dtype; the
 * residual, its output and their gradients have res_dtype (fp32, or x's
 * dtype); weight, scale and their gradients are fp32.  group_size and the
 * width of the add form are at most 16384.  Pointers are aligned to their
 * element size; rows of 16-byte vectors run faster.
 * residual_out may be the residual's own memory (same stride), dresidual
 * may be dresidual_out's, dx or dz may be dy's; other outputs must not
 * overlap inputs.  Sizes of 0 are errors.
 *
 * Ownership, streams and errors as in selective_scan.h.
 */
#ifndef SSS48_NORM_H
#define SSS48_NORM_H

#include <stdint.h>

#include "selective_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct mss_gated_norm_args {
  int64_t rows;
  int64_t width;
  int64_t group_size;    /* divides width */
  mss_dtype dtype;
  int norm_before_gate;
  int shared_weight;     /* 1: weight has group_size entries */
  float eps;
  const void *x;
  const void *z;
  const float *weight;
  void *y;               /* forward */
  const void *dy;        /* backward, from here on */
  void *dx;
  void *dz;
  float *dweight;        /* NULL: not computed */
  int64_t stride_x, stride_z, stride_y, stride_dy, stride_dx, stride_dz;
  void *workspace;       /* backward with dweight; 16-byte aligned */
  size_t workspace_bytes;
} mss_gated_norm_args;

mss_status gated_rmsnorm_fwd(const mss_gated_norm_args *args, void *stream);
mss_status gated_rmsnorm_bwd(const mss_gated_norm_args *args, void *stream);
/* Bytes of the backward's workspace on the current device (0 without dweight). */
mss_status mss_gated_rmsnorm_bwd_workspace_size(const mss_gated_norm_args *args, size_t *bytes);

typedef struct mss_add_norm_args {
  int64_t rows;
  int64_t width;
  mss_dtype dtype;       /* x, y, dy, dx */
  mss_dtype res_dtype;   /* residual, residual_out and their gradients */
  float eps;
  const void *x;         /* backward: only read for dscale */
  const void *residual;  /* NULL: 0 */
  const float *scale;    /* NULL: 1 */
  const float *weight;
  void *y;
  void *residual_out;    /* forward: written; backward: read */
  const void *dy;        /* backward, from here on */
  const void *dresidual_out; /* NULL: 0 */
  void *dx;
  void *dresidual;       /* NULL: not written */
  float *dweight;        /* NULL: not computed */
  float *dscale;         /* NULL: not computed */
  int64_t stride_x, stride_residual, stride_y, stride_residual_out, stride_dy,
      stride_dresidual_out, stride_dx, stride_dresidual;
  void *workspace;       /* backward with dweight or dscale; 16-byte aligned */
  size_t workspace_bytes;
} mss_add_norm_args;

mss_status add_rmsnorm_fwd(const mss_add_norm_args *args, void *stream);
mss_status add_rmsnorm_bwd(const mss_add_norm_args *args, void *stream);
mss_status mss_add_rmsnorm_bwd_workspace_size(const mss_add_norm_args *args, size_t *bytes);

#ifdef __cplusplus
}
#endif

#endif /* SSS48_NORM_H */
