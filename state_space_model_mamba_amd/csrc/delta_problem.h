// Problem descriptor of the gated delta kernels, and their launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ssd_device.h"

namespace delta {

constexpr int SLICE = 16;   // value columns of a state wave
constexpr int PAD = 32;     // the workspace's value columns are a multiple of this
// the widest row stride of q, k and v, and row of the contiguous tensors, in elements (checked on the host)
constexpr int64_t MAX_ROW_STRIDE = int64_t{1} << 26;

struct Problem {
  // sizes
  int B, L, H, P, G, N, nseqs, hpg;
  int total;      // B * L rows
  int nslots;     // chunk slots: the chunks of sequence s are slots start(s) / 64 + s, ...
  int hb;         // heads of a group that one block of k_delta_prep takes
  int ns, hs;     // parts that k_delta_grad takes a group's heads in, and heads of a part
  int rows;       // P rounded up to a multiple of PAD
  int nsl;        // slices of 16 value columns: rows / SLICE
  float scale;
  int64_t q_sb, q_sl, k_sb, k_sl, v_sb, v_sl;
  // inputs
  const void *q, *k, *v, *dout;
  const float *g, *beta, *h0, *dfinal;
  const int32_t* seq_idx;
  // outputs
  void *o, *dq, *dk, *dv;
  float *final, *dg, *dbeta, *dinit;
  // workspace
  int32_t* starts;   // (nseqs + 1) first rows, then (nseqs) the sequences longest first (seq_idx given)
  float* gates;      // (slots, H, GATES, 64)
  uint4* tf;         // (slots, H, FRAG_PIECES): T' - I, T' = (I + N diag(beta))^-1, rows in pair order
  uint4* pf;         // the same of the causal scores, rows in order (forward)
  uint4* ttf;        // transposed (I + diag(beta) N)^-1 - I, rows in pair order (backward)
  uint4* ptf;        // transposed scores, rows in pair order (backward)
  uint4* e;          // (slots, H, nsl, 4, 64): the residuals, float32, accumulator layout (backward)
  // as the lanes hold them (delta_tiles.h), 2 bf16 terms or float32:
  uint4* s;          // (slots, H, nsl, 2, NQ, 64): entering states (backward)
  uint4* ds;         // (slots, H, nsl, 2, NQ, 64): gradient of the state after the chunk (backward)
  uint4* dvl;        // (slots, H, nsl, 2, 64): second terms of dv, 8 rows of a column a piece (backward, bf16)
  float* be;         // (slots, H, nsl, 64): Du . e over the slice's columns (backward)
  float* parts;      // (slots, G, ns, 2, 64, ND): the parts' dq and dk (ns > 1)
};

// Per slot and head, 64 values each: exp(c_i); beta_i exp(c_last - c_i); beta_i; exp(c_last - c_i); -beta_i exp(c_i);
// and c_i in two floats.  The forward walk reads the first WALK_GATES, the backward's the first RWALK_GATES.
enum { GATE_IN = 0, GATE_BO = 1, GATE_BETA = 2, GATE_OUT = 3, GATE_BI = 4, GATE_C = 5, GATE_CLO = 6, GATES = 7 };
constexpr int WALK_GATES = 3, RWALK_GATES = 5;

int launch_starts(const Problem& p, hipStream_t s);
int launch_prep(const Problem& p, int io, bool backward, hipStream_t s);
int launch_walk(const Problem& p, int io, bool backward, hipStream_t s);
int launch_rwalk(const Problem& p, int io, hipStream_t s);
int launch_grad(const Problem& p, int io, hipStream_t s);
int launch_gates(const Problem& p, hipStream_t s);

#ifdef __HIPCC__
// first row of sequence s (s == nseqs: the end of the last)
__device__ __forceinline__ int seq_start(const Problem& p, int s) { return p.seq_idx ? p.starts[s] : s * p.L; }
__device__ __forceinline__ int slot_base(int start, int s) { return (start >> 6) + s; }

struct Chunk {
  int seq, row, len;   // sequence, first row (flat), rows of the chunk (0: the slot holds none)
};
// Sequence, head and value column block of a walk's block.  Packed sequences go longest first, so that none of them is
// left to run alone at the end.  Within a sequence, consecutive (head, column block)s run on the same XCD, whose L2
// then serves a head's chunk matrices to its column blocks and a group's q and k to its heads.
struct Place {
  int seq, h, ps;
};
__device__ __forceinline__ Place place_of(const Problem& p, int np) {
  const int x = static_cast<int>(ssd::xcd_logical_block(blockIdx.x, gridDim.x)), y = static_cast<int>(blockIdx.y);
  return Place{p.seq_idx ? p.starts[p.nseqs + 1 + y] : y, x / np, x % np};
}

// which chunk a slot holds
__device__ __forceinline__ Chunk chunk_of(const Problem& p, int slot) {
  int lo = 0, hi = p.nseqs;   // the last sequence whose slots begin at or before this one
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (slot_base(seq_start(p, mid), mid) <= slot) lo = mid; else hi = mid;
  }
  const int s0 = seq_start(p, lo), s1 = seq_start(p, lo + 1);
  Chunk c{lo, s0 + 64 * (slot - slot_base(s0, lo)), 0};
  c.len = s1 - c.row < 64 ? s1 - c.row : 64;
  if (c.len < 0) c.len = 0;
  return c;
}
// the batch row's base and the row inside it are taken once: a sequence lies in one batch row
__device__ __forceinline__ int64_t row_offset(int row, int L, int64_t sb, int64_t sl) {
  const int b = row / L;
  return b * sb + static_cast<int64_t>(row - b * L) * sl;
}
#endif

}  // namespace delta
