// C ABI of the gated linear recurrence over whole sequences
// (include/linear_recurrence.h): argument checks, the workspace layout and the
// launches.
#include <limits.h>

#include "linrec_problem.h"

int linrec_check(const linrec_shape* s) {
  if (!s || s->reserved != 0) return SSD_ERR_INVALID_ARG;
  if (s->io_dtype != SSD_IO_BF16 && s->io_dtype != SSD_IO_F32) return SSD_ERR_UNSUPPORTED_SHAPE;
  const int64_t vec = s->io_dtype == SSD_IO_BF16 ? 8 : 4;
  if (s->batch < 1 || s->seqlen < 1 || s->channels < 1 || s->nseqs < 1) return SSD_ERR_UNSUPPORTED_SHAPE;
  if (s->batch > INT_MAX || s->seqlen > INT_MAX || s->batch * s->seqlen >= INT_MAX - 4095) return SSD_ERR_UNSUPPORTED_SHAPE;
  if (s->channels % vec || s->channels > (1 << 20) || s->nseqs > (1 << 24)) return SSD_ERR_UNSUPPORTED_SHAPE;
  for (const int64_t st : {s->x_batch_stride, s->x_row_stride, s->g_batch_stride, s->g_row_stride, s->i_batch_stride, s->i_row_stride})
    if (st < 0 || st % vec) return SSD_ERR_UNSUPPORTED_SHAPE;
  if (s->gate < LINREC_GATE_LOG || s->gate > LINREC_GATE_DECAY) return SSD_ERR_UNSUPPORTED_SHAPE;
  if (s->input_scale < LINREC_INPUT_ONE || s->input_scale > LINREC_INPUT_UNIT) return SSD_ERR_UNSUPPORTED_SHAPE;
  return SSD_OK;
}

void linrec_strides(const linrec_shape& s, int64_t (&st)[6]) {
  const int64_t in[6] = {s.x_batch_stride, s.x_row_stride, s.g_batch_stride, s.g_row_stride, s.i_batch_stride, s.i_row_stride};
  for (int k = 0; k < 6; k += 2) {
    const bool contiguous = in[k] == 0 && in[k + 1] == 0;
    st[k] = contiguous ? s.seqlen * s.channels : in[k];
    st[k + 1] = contiguous ? s.channels : in[k + 1];
  }
}

namespace {

using linrec::Problem;

bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

// Places the workspace's arrays from `base` (nullptr: sizes only); returns the bytes.
size_t place(Problem& p, bool backward, char* base) {
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* r = base ? base + at : nullptr;
    at += (bytes + 255) / 256 * 256;
    return r;
  };
  const size_t n = static_cast<size_t>(p.spans) * p.C;
  p.starts = reinterpret_cast<int32_t*>(take((static_cast<size_t>(p.nseqs) + 1) * 4));
  p.sync = reinterpret_cast<uint32_t*>(take(static_cast<size_t>(p.cblocks) * (p.spans + linrec::LINE) * 4));
  p.agg = reinterpret_cast<float2*>(take(n * sizeof(float2)));
  p.states = reinterpret_cast<float*>(take(n * 4));
  if (backward) {
    p.carry = reinterpret_cast<float*>(take(n * 4));
    p.slots = reinterpret_cast<float*>(take(n * 4));
  }
  return at;
}

int problem(const linrec_shape* s, Problem& p) {
  const int rc = linrec_check(s);
  if (rc != SSD_OK) return rc;
  p.R = static_cast<int>(s->batch * s->seqlen);
  p.L = static_cast<int>(s->seqlen);
  p.C = static_cast<int>(s->channels);
  p.nseqs = static_cast<int>(s->nseqs);
  p.spans = (p.R + linrec::SPAN - 1) / linrec::SPAN;
  // the backward's, which are the narrower: what is sized by them is enough for the forward's
  const int cb = 64 * (s->io_dtype == SSD_IO_BF16 ? linrec::Bwd::VALS<ssd::bf16_t> : linrec::Bwd::VALS<float>);
  p.cblocks = (p.C + cb - 1) / cb;
  if (static_cast<int64_t>(p.spans) * p.cblocks > INT_MAX / 2) return SSD_ERR_UNSUPPORTED_SHAPE;
  int64_t st[6];
  linrec_strides(*s, st);
  p.x_sb = st[0]; p.x_sl = st[1];
  p.g_sb = st[2]; p.g_sl = st[3];
  p.i_sb = st[4]; p.i_sl = st[5];
  return SSD_OK;
}

// What both directions check and set; the arrays that hold states need the sequences' numbers.
int inputs(const linrec_shape* shape, const void* x, const void* g, const void* in_gate, const float* decay, const float* h0,
           const int32_t* seq_idx, bool backward, bool states, void* workspace, size_t bytes, Problem& p) {
  const int rc = problem(shape, p);
  if (rc != SSD_OK) return rc;
  if (!x || !g || !workspace || (shape->gate == LINREC_GATE_DECAY && !decay)) return SSD_ERR_INVALID_ARG;
  if (!seq_idx && shape->nseqs != shape->batch) return SSD_ERR_INVALID_ARG;
  if (bytes < place(p, backward, static_cast<char*>(workspace))) return SSD_ERR_WORKSPACE_TOO_SMALL;
  for (const void* q : {x, g, in_gate, static_cast<const void*>(decay), static_cast<const void*>(h0), static_cast<const void*>(workspace)})
    if (misaligned(q)) return SSD_ERR_MISALIGNED;
  p.x = x; p.g = g; p.i = in_gate; p.decay = decay; p.h0 = h0; p.seq_idx = seq_idx;
  if (!seq_idx || !states) p.starts = nullptr;
  // Read past the caches what is more than the 256 MB of the last one holds with the forward's result.  The backward moves up
  // to 1.8 times as much, but reads what the forward read: microseconds of both past the caches and by them, 4000 rows of
  // 4096 bf16 channels with all gates (125 MB forward, 218 backward) 109 and 106, 6000 158 and 158, 8192 (256, 448) 210 and
  // 208; without input gate 9000 (210, 351) 188 and 188, 12000 (281, 468) 240 and 238.
  const int64_t io = shape->io_dtype == SSD_IO_BF16 ? 2 : 4, gates = shape->gate == LINREC_GATE_LOG ? 4 : io;
  p.pass = static_cast<int64_t>(p.R) * p.C * (2 * io + gates + (in_gate ? io : 0)) > (int64_t{256} << 20);
  return SSD_OK;
}

}  // namespace

extern "C" {

int linrec_chunks(const linrec_shape* shape, int64_t* chunks) {
  Problem p{};
  const int rc = problem(shape, p);
  if (rc != SSD_OK) return rc;
  if (!chunks) return SSD_ERR_INVALID_ARG;
  *chunks = p.spans;
  return SSD_OK;
}

int linrec_workspace_size(const linrec_shape* shape, int backward, size_t* bytes) {
  Problem p{};
  const int rc = problem(shape, p);
  if (rc != SSD_OK) return rc;
  if (!bytes) return SSD_ERR_INVALID_ARG;
  *bytes = place(p, backward != 0, nullptr);
  return SSD_OK;
}

int linrec_fwd(const linrec_shape* shape, const void* x, const void* g, const void* in_gate, const float* decay,
               const float* initial_states, const int32_t* seq_idx, void* y, float* final_states,
               float* chunk_states, void* workspace, size_t workspace_bytes, void* stream) {
  Problem p{};
  int rc = inputs(shape, x, g, in_gate, decay, initial_states, seq_idx, false, initial_states || final_states, workspace, workspace_bytes, p);
  if (rc != SSD_OK) return rc;
  if (!y) return SSD_ERR_INVALID_ARG;
  for (const void* q : {static_cast<const void*>(y), static_cast<const void*>(final_states), static_cast<const void*>(chunk_states)})
    if (misaligned(q)) return SSD_ERR_MISALIGNED;
  if (y == x || y == g || y == in_gate) return SSD_ERR_INVALID_ARG;
  p.y = y;
  p.final = final_states;
  if (chunk_states) p.states = chunk_states;
  p.keep = chunk_states != nullptr;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if ((rc = linrec::launch_setup(p, linrec::chained_fwd(p), p.starts != nullptr, st)) != SSD_OK) return rc;
  return linrec::launch_fwd(p, *shape, st);
}

int linrec_bwd(const linrec_shape* shape, const void* x, const void* g, const void* in_gate, const float* decay,
               const float* initial_states, const int32_t* seq_idx, const float* chunk_states, const void* dy,
               const float* d_final_states, void* dx, void* dg, void* d_in_gate, float* ddecay,
               float* d_initial_states, void* workspace, size_t workspace_bytes, void* stream) {
  Problem p{};
  int rc = inputs(shape, x, g, in_gate, decay, initial_states, seq_idx, true, initial_states || d_final_states || d_initial_states, workspace,
                  workspace_bytes, p);
  if (rc != SSD_OK) return rc;
  if (!dy || !dx || !dg || (in_gate && !d_in_gate)) return SSD_ERR_INVALID_ARG;
  for (const void* q : {dy, static_cast<const void*>(chunk_states), static_cast<const void*>(d_final_states), static_cast<const void*>(dx),
                        static_cast<const void*>(dg), static_cast<const void*>(d_in_gate), static_cast<const void*>(d_initial_states)})
    if (misaligned(q)) return SSD_ERR_MISALIGNED;
  for (const void* o : {static_cast<const void*>(dx), static_cast<const void*>(dg), static_cast<const void*>(d_in_gate)})
    for (const void* i : {x, g, in_gate, dy})
      if (o && o == i) return SSD_ERR_INVALID_ARG;
  if (d_initial_states && d_initial_states == d_final_states) return SSD_ERR_INVALID_ARG;   // written while others still read
  p.dy = dy; p.dfinal = d_final_states;
  p.dx = dx; p.dg = dg; p.di = d_in_gate; p.ddecay = ddecay; p.dh0 = d_initial_states;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if ((rc = linrec::launch_setup(p, linrec::chained_bwd(p), p.starts != nullptr, st)) != SSD_OK) return rc;
  if (chunk_states) {
    p.states = const_cast<float*>(chunk_states);
  } else {
    p.keep = 1;
    if ((rc = linrec::launch_fwd(p, *shape, st)) != SSD_OK) return rc;
    if (linrec::chained_fwd(p) && (rc = linrec::launch_setup(p, true, false, st)) != SSD_OK) return rc;
  }
  return linrec::launch_bwd(p, *shape, st);
}

}  // extern "C"
