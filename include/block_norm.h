/*
 * block_norm.h -- C ABI (in libssd_bwd.so) of the norms before and after a
 * block with what stands next to them in the same pass, and their
 * deterministic backward, on AMD Instinct MI355X (gfx950).
 *
 * add_norm, before a block: the block's input is added to the residual
 * stream, and the sum is normed.  Per row of `width` values, s = alpha *
 * scale:
 *
 *     r = residual + s x            (the new residual; residual zero when NULL)
 *     y = norm(r) w + b
 *
 * gated_norm, after a block (an SSD layer's y, or a recurrence's): the
 * block's output is normed together with its gate z, each of `groups` runs of
 * width / groups channels by itself, and added to the residual where one is
 * given:
 *
 *     n = norm(x act(z)) w + b      (norm_before_gate == 0)
 *     n = (norm(x) w + b) act(z)    (norm_before_gate != 0)
 *     out = residual + s n          (s n when residual is NULL)
 *
 * with act(z) = z sigmoid(z) or sigmoid(z) (1 when z is NULL) and, over the W
 * values of a row or group,
 *
 *     norm(u) = u / sqrt(mean u^2 + eps)               (BLOCK_NORM_RMS)
 *     norm(u) = (u - mean u) / sqrt(var u + eps)       (BLOCK_NORM_LAYER)
 *
 * Everything between the loads and the stores is float32: y is formed from
 * the sum r before r is rounded to the residual's dtype, and the backward
 * forms r again from x and residual.  Squares must stay in float32's range
 * (values up to 1e18 or so).
 *
 * Determinism.  Rows have one writer; the gradients of weight, bias and scale
 * are summed per block in a fixed order into workspace slots, and the slots in
 * slot order in double.  No atomics.
 *
 * Layouts (row-major), D = width:
 *   x, z, y, dy, dx, dz              (batch, seqlen, D)   io dtype
 *   residual, residual_out, out and
 *   their gradients                  (batch, seqlen, D)   residual dtype (out: the io dtype when residual is NULL)
 *   weight, bias, scale and their gradients          (D)  float32
 * x and z may be slices of wider rows (batch and row strides in elements,
 * 0, 0: contiguous); everything else is contiguous.
 *
 * Ownership and calling convention: as for ssd_bwd.  weight, bias and scale
 * need 16-byte addresses like the others.
 */
#ifndef BLOCK_NORM_H
#define BLOCK_NORM_H

#include <stddef.h>
#include <stdint.h>

#include "ssd_bwd.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { BLOCK_NORM_RMS = 0, BLOCK_NORM_LAYER = 1 };
enum { BLOCK_NORM_SILU = 0, BLOCK_NORM_SIGMOID = 1 };

typedef struct {
  int64_t batch;   /* >= 1 */
  int64_t seqlen;  /* >= 1; batch * seqlen < 2^31 */
  int64_t width;   /* D >= 1, <= 2^20, multiple of groups */
  int64_t groups;  /* >= 1 (add_norm: 1); D / groups: multiple of 8 (bf16 io) or 4 (f32 io), <= 16384 */
  int64_t x_batch_stride, x_row_stride; /* elements, multiples of 8 (bf16) or 4 (f32); 0, 0: contiguous */
  int64_t z_batch_stride, z_row_stride;
  int32_t norm;             /* BLOCK_NORM_RMS or BLOCK_NORM_LAYER */
  int32_t gate;             /* BLOCK_NORM_SILU or BLOCK_NORM_SIGMOID (read when z is given) */
  int32_t norm_before_gate; /* 0 or 1 */
  int32_t io_dtype;         /* SSD_IO_BF16 or SSD_IO_F32 */
  int32_t residual_dtype;   /* the io dtype, or SSD_IO_F32 */
  int32_t reserved;         /* must be 0 */
  float eps;                /* >= 0 */
  float alpha;              /* finite */
} block_norm_shape;

/* weight (ones), bias (zeros), scale (ones), residual (zeros) and residual_out (not written) may be NULL.
 * y may be x when x is contiguous, residual_out may be residual. */
int add_norm_fwd(const block_norm_shape* shape, const void* x, const void* residual, const float* weight,
                 const float* bias, const float* scale, void* y, void* residual_out, void* stream);

/* weight, bias, scale, z and residual may be NULL.  With residual NULL, residual_dtype is the io dtype. */
int gated_norm_fwd(const block_norm_shape* shape, const void* x, const void* z, const float* weight,
                   const float* bias, const void* residual, const float* scale, void* out, void* stream);

/* Workspace bytes of add_norm_bwd and of gated_norm_bwd (the blocks' partial sums of the gradients over rows). */
int block_norm_bwd_workspace_size(const block_norm_shape* shape, size_t* bytes);

/*
 * Gradients of l = sum dy * y + sum dresidual_out * residual_out from the
 * inputs of add_norm_fwd.  Either of dy and dresidual_out may be NULL
 * (zeros), not both.  dx, dresidual, dweight, dbias and dscale may be NULL
 * (not computed); with NULL weight or scale the last are the gradients at
 * ones.  dx and dresidual differ in the factor s and the dtype only.
 */
int add_norm_bwd(const block_norm_shape* shape, const void* x, const void* residual, const float* weight,
                 const float* scale, const void* dy, const void* dresidual_out, void* dx, void* dresidual,
                 float* dweight, float* dbias, float* dscale, void* workspace, size_t workspace_bytes,
                 void* stream);

/*
 * Gradients of l = sum dout * out from the inputs of gated_norm_fwd (that of
 * residual is dout).  dout has the residual dtype.  dz goes with z; dx, dz,
 * dweight, dbias and dscale may be NULL (not computed).
 */
int gated_norm_bwd(const block_norm_shape* shape, const void* x, const void* z, const float* weight,
                   const float* bias, const float* scale, const void* dout, void* dx, void* dz, float* dweight,
                   float* dbias, float* dscale, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* BLOCK_NORM_H */
