/*
 * gated_delta.h -- C ABI (in libssd_bwd.so) of the gated delta rule on AMD
 * Instinct MI355X (gfx950): whole sequences forward and backward, and few
 * tokens at a time on a pool of states.
 *
 * The operation, per sequence and head, on a state S in R^{P x N}:
 *
 *     Sd_t = exp(g_t) S_{t-1}              (decay)
 *     e_t  = v_t - Sd_t k_t                (what the state does not say yet of v_t)
 *     S_t  = Sd_t + beta_t e_t k_t^T       (correction)
 *     o_t  = scale S_t q_t
 *
 * S enters a sequence as its initial state (zeros when there is none).  The
 * state update is the SSD layer's with the input v replaced by the residual
 * e; q, k, v, P and N stand where C, B, x, headdim and dstate stand in
 * ssd_bwd.h, and head h uses group h / (nheads / ngroups) of q and k.
 *
 * Determinism.  Every output element has one writer and every sum one order;
 * no atomics.  The output bytes depend on the inputs, the shape and the
 * library build only.
 *
 * Layouts (row-major):
 *   q, k, dq, dk       (batch, seqlen, ngroups, dstate)   io dtype (ssd_io_dtype)
 *   v, o, dout, dv     (batch, seqlen, nheads, headdim)   io dtype
 *   g, beta, dg, dbeta (batch, seqlen, nheads)            float32
 *   states             (nseqs, nheads, headdim, dstate)   float32
 *   seq_idx            (batch, seqlen)                    int32
 * q, k and v may be slices of wider rows: their batch and row strides are
 * given in elements (0: contiguous), the last two axes are contiguous.
 * Everything else is contiguous.  Sequences are marked by seq_idx and
 * numbered as for ssd_bwd (one per batch row when it is NULL).
 *
 * Values.  g is a log decay: g <= 0, -inf included (the state is dropped);
 * values below -104, where exp is zero in float32, count as -104.  States,
 * gates and every sum are float32; with bf16 io the products take their
 * float32 operands as two bf16 terms (16 bits of mantissa), what is added to a
 * state as three.  dg_t is a sum of terms that all hold exp(g_t): its error is
 * relative to them however strong the decay, and dg is zero where g counts
 * as -104.
 * A NaN or an infinity in a row of q, k, v, g or beta may reach every row of
 * its sequence from the first of its chunk of 64 rows on (in the backward
 * every row), and no other sequence.
 *
 * Ownership and calling convention: as for ssd_bwd (device pointers of the
 * caller, 16-byte aligned; outputs fully overwritten; no allocation; work
 * only enqueued on `stream`; argument errors returned before that as the
 * SSD_* status codes).  Concurrent calls need workspaces of their own.
 */
#ifndef GATED_DELTA_H
#define GATED_DELTA_H

#include <stddef.h>
#include <stdint.h>

#include "ssd_bwd.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
  int64_t batch;    /* >= 1; <= 65535 for delta_step */
  int64_t seqlen;   /* >= 1; batch * seqlen < 2^31 */
  int64_t nheads;   /* >= 1, <= 65535, multiple of ngroups */
  int64_t headdim;  /* P: multiple of 8 (bf16 io) or 4 (f32 io), <= 1024 */
  int64_t ngroups;  /* >= 1 */
  int64_t dstate;   /* N: multiple of 8 (bf16 io) or 4 (f32 io), <= 128 */
  int64_t nseqs;    /* number of sequence starts, 1 .. 65535; == batch without seq_idx */
  int64_t q_batch_stride, q_row_stride; /* elements, multiples of 8 (bf16) or 4 (f32); 0, 0: contiguous; */
  int64_t k_batch_stride, k_row_stride; /* row strides, nheads * headdim and ngroups * dstate <= 2^26 */
  int64_t v_batch_stride, v_row_stride;
  float scale;
  int32_t io_dtype; /* SSD_IO_BF16 or SSD_IO_F32 */
} delta_shape;

/*
 * Workspace bytes of delta_fwd (backward == 0) or delta_bwd (backward != 0):
 * 26 KB for every head and chunk of 64 rows (a sequence has its own chunks),
 * in the backward 38 KB and for every 64 value columns 57 (dstate <= 64) or 89
 * KB: 0.87 and 4.27 GB at 16384 rows of 128 heads of 64 x 128.
 */
int delta_workspace_size(const delta_shape* shape, int backward, size_t* bytes);

/*
 * o, and final_states (nullable): the state after each sequence's last
 * position.  initial_states and seq_idx may be NULL.  nseqs must be the
 * number of sequences that seq_idx marks: sequences past nseqs are not
 * computed (their rows of o are left as they were), and a final state past
 * the last sequence is its initial state.
 */
int delta_fwd(const delta_shape* shape, const void* q, const void* k, const void* v, const float* g,
              const float* beta, const float* initial_states, const int32_t* seq_idx, void* o,
              float* final_states, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Gradients of l = sum dout * o + sum d_final_states * final_states, the
 * forward recomputed from the inputs.  d_final_states (nullable: zeros) and
 * d_initial_states (nullable: not computed) are shaped like the states.
 * Rows of sequences past nseqs are left as they were, as in delta_fwd.
 */
int delta_bwd(const delta_shape* shape, const void* q, const void* k, const void* v, const float* g,
              const float* beta, const float* initial_states, const int32_t* seq_idx, const void* dout,
              const float* d_final_states, void* dq, void* dk, void* dv, float* dg, float* dbeta,
              float* d_initial_states, void* workspace, size_t workspace_bytes, void* stream);

/*
 * The same recurrence for `seqlen` tokens (1 .. 64) of each of `batch`
 * sequences whose states live in a pool (nslots, nheads, headdim, dstate):
 * row b reads and overwrites states[state_indices[b]] (state_indices NULL:
 * states[b], nslots >= batch).  A row whose index is negative or not below
 * nslots is empty: its o is zero and no state changes.  Rows that name the
 * same state take their turns in row order, one after the other's tokens.
 * o may be none of q, k, v and states.  shape->nseqs is not read; no
 * workspace.
 */
int delta_step(const delta_shape* shape, const void* q, const void* k, const void* v, const float* g,
               const float* beta, float* states, int64_t nslots, const int32_t* state_indices, void* o,
               void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GATED_DELTA_H */
