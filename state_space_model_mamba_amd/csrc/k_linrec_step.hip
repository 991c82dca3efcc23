// Gated linear recurrence for few tokens on a pool of states
// (include/linear_recurrence.h, linrec_step).  Channels need each other for
// nothing: a lane holds the states of 8 bytes of channels and takes its row's
// tokens one after the other, the next one's operands in flight.  Bound by
// latency in the calls of decoding: one row of 8192 channels 3.0 us, 64 rows of 4
// tokens of 4096 channels (9.3 MB) 5.0 us.
#include "linrec_problem.h"

namespace linrec {

using ssd::bf16_t;

template <typename T> constexpr int STEP_VALS = 8 / static_cast<int>(sizeof(T));

struct StepArgs {
  const void *x, *g, *i;
  const float* decay;
  float* states;
  const int32_t* index;
  void* y;
  int64_t nslots, x_sb, x_sl, g_sb, g_sl, i_sb, i_sl;
  int B, T, C;
};

template <typename T, int GATE, int SCALE> __global__ __launch_bounds__(64) void k_linrec_step(StepArgs s) {
  constexpr int V = STEP_VALS<T>;
  using G = std::conditional_t<GATE == LINREC_GATE_LOG, float, T>;
  const int l = static_cast<int>(threadIdx.x);
  const int c0 = (static_cast<int>(blockIdx.x) * 64 + l) * V;
  const bool live = c0 < s.C;
  const int c = live ? c0 : s.C - V;
  int b = static_cast<int>(blockIdx.y);
  int64_t slot = b;
  // the next batch row after `from` that names `slot` (s.B: none)
  auto next_of = [&](int from, int64_t which) {
    for (int i0 = (from + 1) & ~63; i0 < s.B; i0 += 64) {
      const int i = i0 + l;
      const uint64_t m = __ballot(i > from && i < s.B && s.index[i < s.B ? i : 0] == which);
      if (m) return i0 + static_cast<int>(__builtin_ctzll(m));
    }
    return s.B;
  };
  if (s.index) {
    slot = s.index[b];
    if (slot < 0 || slot >= s.nslots) {   // an empty row
      float zero[V] = {};
      Raw<T, V> out;
      out.set(zero);
      for (int t = 0; live && t < s.T; ++t) out.store(static_cast<T*>(s.y) + (static_cast<int64_t>(b) * s.T + t) * s.C + c);
      return;
    }
    if (next_of(-1, slot) != b) return;   // an earlier row's block takes this row's tokens too
  }
  Raw<float, V> dk;
  if (GATE == LINREC_GATE_DECAY) dk.load(s.decay + c);
  float* at = s.states + slot * s.C + c;
  Raw<float, V> state;
  state.load(at);
  float h[V];
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = state.get(v);
  do {
    const T* xp = static_cast<const T*>(s.x) + b * s.x_sb + c;
    const G* gp = static_cast<const G*>(s.g) + b * s.g_sb + c;
    const T* ip = static_cast<const T*>(s.i) + b * s.i_sb + c;
    Raw<T, V> x, in;
    Raw<G, V> g;
    auto request = [&](int t) {
      x.load(xp + t * s.x_sl);
      g.load(gp + t * s.g_sl);
      if (s.i) in.load(ip + t * s.i_sl);
    };
    request(0);
    for (int t = 0; t < s.T; ++t) {
      const Raw<T, V> x0 = x, i0 = in;
      const Raw<G, V> g0 = g;
      if (t + 1 < s.T) request(t + 1);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const Factor f = factor_of<T, GATE>(g0.get(v), Decay<T, GATE>(GATE == LINREC_GATE_DECAY ? dk.get(v) : 0.f));
        float u = x0.get(v);
        if (s.i) u *= Fn<T>::sigmoid(i0.get(v));
        h[v] = fmaf(f.a, h[v], scale_of<T, GATE, SCALE>(f) * u);
      }
      Raw<T, V> out;
      out.set(h);
      if (live) out.store(static_cast<T*>(s.y) + (static_cast<int64_t>(b) * s.T + t) * s.C + c);
    }
    b = s.index ? next_of(b, slot) : s.B;
  } while (b < s.B);
  state.set(h);
  if (live) state.store(at);
}

namespace {
template <typename T, int GATE> int by_scale(const StepArgs& s, int scale, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>((s.C + 64 * STEP_VALS<T> - 1) / (64 * STEP_VALS<T>)), static_cast<unsigned>(s.B));
  switch (scale) {
    case LINREC_INPUT_ONE: hipLaunchKernelGGL((k_linrec_step<T, GATE, LINREC_INPUT_ONE>), grid, dim3(64), 0, st, s); break;
    case LINREC_INPUT_COMPLEMENT: hipLaunchKernelGGL((k_linrec_step<T, GATE, LINREC_INPUT_COMPLEMENT>), grid, dim3(64), 0, st, s); break;
    default: hipLaunchKernelGGL((k_linrec_step<T, GATE, LINREC_INPUT_UNIT>), grid, dim3(64), 0, st, s); break;
  }
  return hipGetLastError() == hipSuccess ? SSD_OK : SSD_ERR_HIP;
}
template <typename T> int by_gate(const StepArgs& s, int gate, int scale, hipStream_t st) {
  switch (gate) {
    case LINREC_GATE_LOG: return by_scale<T, LINREC_GATE_LOG>(s, scale, st);
    case LINREC_GATE_SIGMOID: return by_scale<T, LINREC_GATE_SIGMOID>(s, scale, st);
    default: return by_scale<T, LINREC_GATE_DECAY>(s, scale, st);
  }
}
}  // namespace

int launch_step(const StepArgs& s, const linrec_shape& sh, hipStream_t st) {
  return sh.io_dtype == SSD_IO_BF16 ? by_gate<bf16_t>(s, sh.gate, sh.input_scale, st) : by_gate<float>(s, sh.gate, sh.input_scale, st);
}

}  // namespace linrec

int linrec_check(const linrec_shape* s);   // linrec_api.hip
void linrec_strides(const linrec_shape& s, int64_t (&st)[6]);

extern "C" int linrec_step(const linrec_shape* shape, const void* x, const void* g, const void* in_gate, const float* decay,
                           float* states, int64_t nslots, const int32_t* state_indices, void* y, void* stream) {
  if (!shape) return SSD_ERR_INVALID_ARG;
  linrec_shape sh = *shape;
  sh.nseqs = 1;
  const int rc = linrec_check(&sh);
  if (rc != SSD_OK) return rc;
  if (sh.seqlen > 64 || sh.batch > 65535) return SSD_ERR_UNSUPPORTED_SHAPE;
  if (!x || !g || !states || !y || nslots < 1 || (sh.gate == LINREC_GATE_DECAY && !decay)) return SSD_ERR_INVALID_ARG;
  if (!state_indices && nslots < sh.batch) return SSD_ERR_INVALID_ARG;
  for (const void* i : {x, g, in_gate, static_cast<const void*>(decay), static_cast<const void*>(states), static_cast<const void*>(state_indices)})
    if (y == i) return SSD_ERR_INVALID_ARG;   // other blocks may still read them
  for (const void* q : {x, g, in_gate, static_cast<const void*>(decay), static_cast<const void*>(states), static_cast<const void*>(y)})
    if (reinterpret_cast<uintptr_t>(q) & 15u) return SSD_ERR_MISALIGNED;
  int64_t st[6];
  linrec_strides(sh, st);
  const linrec::StepArgs s{x, g, in_gate, decay, states, state_indices, y, nslots, st[0], st[1], st[2], st[3], st[4], st[5],
                           static_cast<int>(sh.batch), static_cast<int>(sh.seqlen), static_cast<int>(sh.channels)};
  return linrec::launch_step(s, sh, static_cast<hipStream_t>(stream));
}
