// C ABI of the gated delta rule over whole sequences (include/gated_delta.h):
// argument checks, the workspace layout and the launches.
#include <limits.h>

#include "delta_problem.h"
#include "delta_tiles.h"
#include "gated_delta.h"

int delta_check(const delta_shape* s) {
  if (!s) return SSD_ERR_INVALID_ARG;
  if (s->io_dtype != SSD_IO_BF16 && s->io_dtype != SSD_IO_F32) return SSD_ERR_UNSUPPORTED_SHAPE;
  const int64_t vec = s->io_dtype == SSD_IO_BF16 ? 8 : 4;
  if (s->batch < 1 || s->seqlen < 1 || s->nheads < 1 || s->ngroups < 1 || s->headdim < 1 || s->dstate < 1 || s->nseqs < 1)
    return SSD_ERR_UNSUPPORTED_SHAPE;
  if (s->batch > INT_MAX || s->seqlen > INT_MAX || s->batch * s->seqlen > INT_MAX - 64) return SSD_ERR_UNSUPPORTED_SHAPE;
  if (s->nheads > 65535 || s->nheads % s->ngroups != 0 || s->nseqs > 65535) return SSD_ERR_UNSUPPORTED_SHAPE;
  if (s->headdim % vec || s->dstate % vec || s->headdim > 1024 || s->dstate > 128) return SSD_ERR_UNSUPPORTED_SHAPE;
  for (const int64_t st : {s->q_batch_stride, s->q_row_stride, s->k_batch_stride, s->k_row_stride, s->v_batch_stride, s->v_row_stride})
    if (st < 0 || st % vec) return SSD_ERR_UNSUPPORTED_SHAPE;
  for (const int64_t st : {s->q_row_stride, s->k_row_stride, s->v_row_stride, s->nheads * s->headdim, s->ngroups * s->dstate})
    if (st > delta::MAX_ROW_STRIDE) return SSD_ERR_UNSUPPORTED_SHAPE;
  return SSD_OK;
}

void delta_strides(const delta_shape& s, int64_t (&st)[6]) {
  const int64_t qk = s.ngroups * s.dstate, v = s.nheads * s.headdim;
  const int64_t in[6] = {s.q_batch_stride, s.q_row_stride, s.k_batch_stride, s.k_row_stride, s.v_batch_stride, s.v_row_stride};
  const int64_t width[3] = {qk, qk, v};
  for (int i = 0; i < 3; ++i) {
    const bool contiguous = in[2 * i] == 0 && in[2 * i + 1] == 0;
    st[2 * i] = contiguous ? s.seqlen * width[i] : in[2 * i];
    st[2 * i + 1] = contiguous ? width[i] : in[2 * i + 1];
  }
}

namespace {

using delta::Problem;

bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

// Places the workspace's arrays from `base` (nullptr: sizes only); returns the bytes.
size_t place(Problem& p, int io, bool backward, char* base) {
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* r = base ? base + at : nullptr;
    at += (bytes + 255) / 256 * 256;
    return r;
  };
  const size_t sh = static_cast<size_t>(p.nslots) * p.H, rows = static_cast<size_t>(p.rows);
  const size_t nd = p.N <= 64 ? 64 : 128, frags = sh * delta::FRAG_PIECES * 16;
  p.starts = reinterpret_cast<int32_t*>(take((2 * static_cast<size_t>(p.nseqs) + 1) * 4));
  p.gates = reinterpret_cast<float*>(take(sh * delta::GATES * delta::CH * 4));
  p.tf = reinterpret_cast<uint4*>(take(frags));
  if (!backward) {
    p.pf = reinterpret_cast<uint4*>(take(frags));
  } else {
    p.ttf = reinterpret_cast<uint4*>(take(frags));
    p.ptf = reinterpret_cast<uint4*>(take(frags));
    p.e = reinterpret_cast<uint4*>(take(sh * rows * delta::CH * 4));
    p.s = reinterpret_cast<uint4*>(take(sh * rows * nd * 4));
    p.ds = reinterpret_cast<uint4*>(take(sh * rows * nd * 4));
    if (io == SSD_IO_BF16) p.dvl = reinterpret_cast<uint4*>(take(sh * rows * delta::CH * 2));
    p.be = reinterpret_cast<float*>(take(sh * p.nsl * delta::CH * 4));
    if (p.ns > 1) p.parts = reinterpret_cast<float*>(take(static_cast<size_t>(p.nslots) * p.G * p.ns * 2 * delta::CH * nd * 4));
  }
  return at;
}

Problem problem(const delta_shape& s) {
  Problem p{};
  p.B = static_cast<int>(s.batch);
  p.L = static_cast<int>(s.seqlen);
  p.H = static_cast<int>(s.nheads);
  p.P = static_cast<int>(s.headdim);
  p.G = static_cast<int>(s.ngroups);
  p.N = static_cast<int>(s.dstate);
  p.nseqs = static_cast<int>(s.nseqs);
  p.hpg = p.H / p.G;
  p.total = p.B * p.L;
  p.nslots = p.total / delta::CH + p.nseqs;
  // Several heads share the group's products while that leaves every CU four blocks: 32 chunks of 128 heads of 8
  // groups take 108 us at one head a block, 65 at four; 256 chunks 678 us at one, 296 at eight.
  p.hb = 1;
  while (p.hb < 8 && p.hb < p.hpg && static_cast<int64_t>(p.nslots) * p.H / (2 * p.hb) >= 1024) p.hb *= 2;
  // and the gradients' groups are cut where there are fewer chunks and groups than CUs: 32 chunks of 64 heads of one
  // group take 526 us in one part, 87 in eight; from 256 blocks on one part is the faster (256 chunks: 581 us, 654 in
  // eight)
  p.ns = 1;
  while (p.ns < p.hpg && static_cast<int64_t>(p.nslots) * p.G * p.ns < 256) p.ns *= 2;
  p.hs = (p.hpg + p.ns - 1) / p.ns;
  p.ns = (p.hpg + p.hs - 1) / p.hs;
  p.rows = (p.P + delta::PAD - 1) / delta::PAD * delta::PAD;
  p.nsl = p.rows / delta::SLICE;
  p.scale = s.scale;
  int64_t st[6];
  delta_strides(s, st);
  p.q_sb = st[0]; p.q_sl = st[1];
  p.k_sb = st[2]; p.k_sl = st[3];
  p.v_sb = st[4]; p.v_sl = st[5];
  return p;
}

}  // namespace

extern "C" {

int delta_workspace_size(const delta_shape* shape, int backward, size_t* bytes) {
  const int rc = delta_check(shape);
  if (rc != SSD_OK) return rc;
  if (!bytes) return SSD_ERR_INVALID_ARG;
  Problem p = problem(*shape);
  *bytes = place(p, shape->io_dtype, backward != 0, nullptr);
  return SSD_OK;
}

int delta_fwd(const delta_shape* shape, const void* q, const void* k, const void* v, const float* g,
              const float* beta, const float* initial_states, const int32_t* seq_idx, void* o,
              float* final_states, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = delta_check(shape);
  if (rc != SSD_OK) return rc;
  if (!q || !k || !v || !g || !beta || !o || !workspace) return SSD_ERR_INVALID_ARG;
  if (!seq_idx && shape->nseqs != shape->batch) return SSD_ERR_INVALID_ARG;
  Problem p = problem(*shape);
  if (workspace_bytes < place(p, shape->io_dtype, false, static_cast<char*>(workspace))) return SSD_ERR_WORKSPACE_TOO_SMALL;
  for (const void* x : {q, k, v, static_cast<const void*>(initial_states), static_cast<const void*>(o),
                        static_cast<const void*>(final_states), static_cast<const void*>(workspace)})
    if (misaligned(x)) return SSD_ERR_MISALIGNED;
  if (o == v || o == q || o == k) return SSD_ERR_INVALID_ARG;
  p.q = q; p.k = k; p.v = v; p.g = g; p.beta = beta;
  p.h0 = initial_states; p.seq_idx = seq_idx; p.o = o; p.final = final_states;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (seq_idx && (rc = delta::launch_starts(p, st)) != SSD_OK) return rc;
  if ((rc = delta::launch_prep(p, shape->io_dtype, false, st)) != SSD_OK) return rc;
  return delta::launch_walk(p, shape->io_dtype, false, st);
}

int delta_bwd(const delta_shape* shape, const void* q, const void* k, const void* v, const float* g,
              const float* beta, const float* initial_states, const int32_t* seq_idx, const void* dout,
              const float* d_final_states, void* dq, void* dk, void* dv, float* dg, float* dbeta,
              float* d_initial_states, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = delta_check(shape);
  if (rc != SSD_OK) return rc;
  if (!q || !k || !v || !g || !beta || !dout || !dq || !dk || !dv || !dg || !dbeta || !workspace) return SSD_ERR_INVALID_ARG;
  if (!seq_idx && shape->nseqs != shape->batch) return SSD_ERR_INVALID_ARG;
  Problem p = problem(*shape);
  if (workspace_bytes < place(p, shape->io_dtype, true, static_cast<char*>(workspace))) return SSD_ERR_WORKSPACE_TOO_SMALL;
  for (const void* x : {q, k, v, dout, static_cast<const void*>(initial_states), static_cast<const void*>(d_final_states),
                        static_cast<const void*>(dq), static_cast<const void*>(dk), static_cast<const void*>(dv),
                        static_cast<const void*>(d_initial_states), static_cast<const void*>(workspace)})
    if (misaligned(x)) return SSD_ERR_MISALIGNED;
  for (const void* x : {static_cast<const void*>(dq), static_cast<const void*>(dk), static_cast<const void*>(dv)})
    for (const void* y : {q, k, v, dout})
      if (x == y) return SSD_ERR_INVALID_ARG;
  p.q = q; p.k = k; p.v = v; p.g = g; p.beta = beta; p.dout = dout;
  p.h0 = initial_states; p.dfinal = d_final_states; p.seq_idx = seq_idx;
  p.dq = dq; p.dk = dk; p.dv = dv; p.dg = dg; p.dbeta = dbeta; p.dinit = d_initial_states;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const int io = shape->io_dtype;
  if (seq_idx && (rc = delta::launch_starts(p, st)) != SSD_OK) return rc;
  if ((rc = delta::launch_prep(p, io, true, st)) != SSD_OK) return rc;
  if ((rc = delta::launch_walk(p, io, true, st)) != SSD_OK) return rc;
  if ((rc = delta::launch_rwalk(p, io, st)) != SSD_OK) return rc;
  if ((rc = delta::launch_grad(p, io, st)) != SSD_OK) return rc;
  return delta::launch_gates(p, st);
}

}  // extern "C"
