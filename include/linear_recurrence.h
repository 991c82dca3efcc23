/*
 * linear_recurrence.h -- C ABI (in libssd_bwd.so) of the gated linear
 * recurrence on AMD Instinct MI355X (gfx950): whole sequences forward and
 * backward, and few tokens at a time on a pool of states.
 *
 * The operation, per sequence and channel, on a state h of one value:
 *
 *     h_t = a_t h_{t-1} + m_t u_t,   y_t = h_t
 *     u_t = x_t                        (in_gate NULL)
 *         = x_t sigmoid(in_gate_t)
 *
 *     a_t = exp(g_t)                   (LINREC_GATE_LOG: g is a log decay)
 *         = sigmoid(g_t)               (LINREC_GATE_SIGMOID)
 *         = exp(decay_c sigmoid(g_t))  (LINREC_GATE_DECAY: decay <= 0, one a channel)
 *
 *     m_t = 1                          (LINREC_INPUT_ONE)
 *         = 1 - a_t                    (LINREC_INPUT_COMPLEMENT)
 *         = sqrt(1 - a_t^2)            (LINREC_INPUT_UNIT)
 *
 * h enters a sequence as its initial state (zeros when there is none).  It is
 * the SSD layer's state update with one state value a channel and a decay of
 * its own for every channel and token (an SSD head shares one).
 *
 * Determinism.  Every output element has one value and every sum one order;
 * the only atomics hand out work and pass finished values on (blocks wait for
 * blocks that began before them).  The output bytes depend on the inputs, the
 * shape and the library build only.
 *
 * Layouts (row-major), C = channels:
 *   x, y, in_gate, dy, dx, d_in_gate   (batch, seqlen, C)   io dtype (ssd_io_dtype)
 *   g, dg                              (batch, seqlen, C)   io dtype; float32 with LINREC_GATE_LOG
 *   decay, ddecay                      (C)                  float32
 *   states                             (nseqs, C)           float32
 *   chunk_states                       (linrec_chunks, C)   float32
 *   seq_idx                            (batch, seqlen)      int32
 * x, g and in_gate may be slices of wider rows (batch and row strides in
 * elements, 0, 0: contiguous); everything else is contiguous.  Sequences are
 * marked by seq_idx and numbered as for ssd_bwd (one per batch row when it is
 * NULL).
 *
 * Values.  States, gates and every sum are float32; y and the gradients are
 * rounded to their dtype once (the state that goes on is not).  Decays are
 * <= 0 and so are log decays, -inf included (a finite state is dropped).  The
 * gradient of sqrt(1 - a^2) is taken as zero where a is one.  A NaN or an
 * infinity stays in its sequence and channel, and lasts there: products are
 * taken as they stand, a decay of zero times an infinity or a NaN is a NaN, so
 * whatever the sizes, once it is in the state the rest of the sequence (of the
 * gradients: the rows before) is not finite.  Which of the two it is then may
 * depend on how the rows lie in chunks; only a sequence's start drops it.
 *
 * Ownership and calling convention: as for ssd_bwd (device pointers of the
 * caller, 16-byte aligned; outputs fully overwritten; no allocation; work
 * only enqueued on `stream`; argument errors returned before that as the
 * SSD_* status codes).  Concurrent calls need workspaces of their own.
 */
#ifndef LINEAR_RECURRENCE_H
#define LINEAR_RECURRENCE_H

#include <stddef.h>
#include <stdint.h>

#include "ssd_bwd.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { LINREC_GATE_LOG = 0, LINREC_GATE_SIGMOID = 1, LINREC_GATE_DECAY = 2 };
enum { LINREC_INPUT_ONE = 0, LINREC_INPUT_COMPLEMENT = 1, LINREC_INPUT_UNIT = 2 };

typedef struct {
  int64_t batch;    /* >= 1; <= 65535 for linrec_step */
  int64_t seqlen;   /* >= 1; batch * seqlen < 2^31 - 4096 */
  int64_t channels; /* C: multiple of 8 (bf16 io) or 4 (f32 io), <= 2^20 */
  int64_t nseqs;    /* number of sequence starts, 1 .. 2^24; == batch without seq_idx */
  int64_t x_batch_stride, x_row_stride; /* elements, multiples of 8 (bf16) or 4 (f32); 0, 0: contiguous */
  int64_t g_batch_stride, g_row_stride;
  int64_t i_batch_stride, i_row_stride;
  int32_t gate;        /* LINREC_GATE_* */
  int32_t input_scale; /* LINREC_INPUT_* */
  int32_t io_dtype;    /* SSD_IO_BF16 or SSD_IO_F32 */
  int32_t reserved;    /* must be 0 */
} linrec_shape;

/* The rows of chunk_states, which holds the state after every 64 of the batch * seqlen rows, and after the last. */
int linrec_chunks(const linrec_shape* shape, int64_t* chunks);

/* Workspace bytes of linrec_fwd (backward == 0) or linrec_bwd (backward != 0): 12 or 20 for every channel and 64 rows,
 * some KB besides. */
int linrec_workspace_size(const linrec_shape* shape, int backward, size_t* bytes);

/*
 * y, final_states (nullable): the state after each sequence's last position,
 * and chunk_states (nullable): the states between chunks of rows, for linrec_bwd.
 * in_gate, initial_states and seq_idx may be NULL; decay goes with
 * LINREC_GATE_DECAY.  nseqs must be the number of sequences that seq_idx marks
 * whenever states are given or asked for: sequences past nseqs enter with
 * zeros and leave no final state, and a final state past the last sequence is
 * its initial state.
 */
int linrec_fwd(const linrec_shape* shape, const void* x, const void* g, const void* in_gate, const float* decay,
               const float* initial_states, const int32_t* seq_idx, void* y, float* final_states,
               float* chunk_states, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Gradients of l = sum dy * y + sum d_final_states * final_states from the
 * inputs.  chunk_states: as linrec_fwd wrote them for the same inputs, or
 * NULL (they are formed again).  d_final_states (zeros), d_initial_states and
 * ddecay (not computed) may be NULL; d_in_gate goes with in_gate.
 * d_initial_states may not be d_final_states, nor any other gradient an input.
 */
int linrec_bwd(const linrec_shape* shape, const void* x, const void* g, const void* in_gate, const float* decay,
               const float* initial_states, const int32_t* seq_idx, const float* chunk_states, const void* dy,
               const float* d_final_states, void* dx, void* dg, void* d_in_gate, float* ddecay,
               float* d_initial_states, void* workspace, size_t workspace_bytes, void* stream);

/*
 * The same recurrence for `seqlen` tokens (1 .. 64) of each of `batch`
 * sequences whose states live in a pool (nslots, C): row b reads and
 * overwrites states[state_indices[b]] (state_indices NULL: states[b], nslots
 * >= batch).  A row whose index is negative or not below nslots is empty: its
 * y is zero and no state changes.  Rows that name the same state take their
 * turns in row order, one after the other's tokens.  y may be none of the
 * inputs.  shape->nseqs is not read; no workspace.
 */
int linrec_step(const linrec_shape* shape, const void* x, const void* g, const void* in_gate, const float* decay,
                float* states, int64_t nslots, const int32_t* state_indices, void* y, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LINEAR_RECURRENCE_H */
