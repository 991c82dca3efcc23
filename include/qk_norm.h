/*
 * qk_norm.h -- C ABI (in libssd_bwd.so) of the norm of every query and key
 * head with the position rotation in the same pass, and its deterministic
 * backward, on AMD Instinct MI355X (gfx950).
 *
 * The operation, per (batch, position, head) row x in R^N of q and of k:
 *
 *     z = w * x * r,   r = 1 / sqrt(mean x^2 + eps)   (QK_NORM_RMS)
 *                      r = 1 / sqrt(sum  x^2 + eps)   (QK_NORM_L2)
 *     y = z with its first rot_dim values turned by pairs: the pair j
 *         (z_2j, z_2j+1) with `interleaved`, (z_j, z_{j + rot_dim/2}) without,
 *         (a, b) -> (a cos t - b sin t, b cos t + a sin t),
 *         t = positions[b, pos] * inv_freq[j]
 *
 * It prepares q and k (C and B of an SSD layer) for the gated delta rule of
 * gated_delta.h.  Norms, weights and angles are float32 or better (the angle
 * and its reduction to one turn in double, so far positions keep their bits);
 * y is rounded to the io dtype once.
 *
 * Determinism.  Rows have one writer; the weights' gradients are summed per
 * block in a fixed order into workspace slots, and the slots in slot order in
 * double.  No atomics.
 *
 * Layouts (row-major):
 *   q, q_out, dq_out, dq   (batch, seqlen, qheads, dstate)   io dtype
 *   k, k_out, dk_out, dk   (batch, seqlen, kheads, dstate)   io dtype
 *   q_weight, k_weight, dq_weight, dk_weight  (dstate)       float32
 *   positions              (batch, seqlen)                   int32
 *   inv_freq               (rot_dim / 2)                     float32
 * q and k may be slices of wider rows (batch and row strides in elements, 0,
 * 0: contiguous); everything else is contiguous.
 *
 * Ownership and calling convention: as for ssd_bwd.
 */
#ifndef QK_NORM_H
#define QK_NORM_H

#include <stddef.h>
#include <stdint.h>

#include "ssd_bwd.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { QK_NORM_RMS = 0, QK_NORM_L2 = 1 };

typedef struct {
  int64_t batch;   /* >= 1 */
  int64_t seqlen;  /* >= 1; batch * seqlen < 2^31 */
  int64_t qheads;  /* >= 1, <= 65535 */
  int64_t kheads;  /* >= 0, <= 65535 (0: q alone, the k arguments are not read) */
  int64_t dstate;  /* N: multiple of 8 (bf16 io) or 4 (f32 io), <= 256 */
  int64_t q_batch_stride, q_row_stride; /* elements, multiples of 8 (bf16) or 4 (f32); 0, 0: contiguous */
  int64_t k_batch_stride, k_row_stride;
  int32_t rot_dim;     /* even, 0 <= rot_dim <= dstate (0: no rotation) */
  int32_t interleaved; /* 0 or 1 */
  int32_t norm;        /* QK_NORM_RMS or QK_NORM_L2 */
  int32_t io_dtype;    /* SSD_IO_BF16 or SSD_IO_F32 */
  float eps;           /* >= 0 */
  int32_t reserved;    /* must be 0 */
} qk_norm_shape;

/* q_weight and k_weight may be NULL (ones); positions may be NULL (0 .. seqlen - 1 in every batch row);
 * inv_freq may be NULL when rot_dim is 0.  q_out may be q and k_out k when they are contiguous. */
int qk_norm_fwd(const qk_norm_shape* shape, const void* q, const void* k, const float* q_weight,
                const float* k_weight, const int32_t* positions, const float* inv_freq, void* q_out, void* k_out,
                void* stream);

/* Workspace bytes of qk_norm_bwd (the blocks' partial weight gradients). */
int qk_norm_bwd_workspace_size(const qk_norm_shape* shape, size_t* bytes);

/* Gradients of l = sum dq_out * q_out + sum dk_out * k_out from the inputs of qk_norm_fwd.  dq_weight and
 * dk_weight may be NULL (not computed); with NULL weights they are the gradients at weights of one.
 * dq may be dq_out and dk dk_out. */
int qk_norm_bwd(const qk_norm_shape* shape, const void* q, const void* k, const float* q_weight,
                const float* k_weight, const int32_t* positions, const float* inv_freq, const void* dq_out,
                const void* dk_out, void* dq, void* dk, float* dq_weight, float* dk_weight, void* workspace,
                size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* QK_NORM_H */
