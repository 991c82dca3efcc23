// Gated linear recurrence over whole sequences, forward (the operation:
// include/linear_recurrence.h).
//
// All batch rows lie behind each other as one run of rows, cut into chunks.  A
// chunk turns the state h that enters it into A h + H, A the product of its
// decays and H what a zero state would have become; a sequence start inside
// makes A zero.  So do a wave's rows within a chunk: their (A, H) meet in LDS,
// the chunks' in memory.
#include "linrec_problem.h"

namespace linrec {

using ssd::bf16_t;

// AGG: only the chunk's (A, H) are formed
template <typename T, int GATE, int SCALE, bool ING, bool AGG> __global__ __launch_bounds__(THR) void k_linrec(Problem p) {
  constexpr int V = VALS<T>, CB = 64 * V;
  using G = std::conditional_t<GATE == LINREC_GATE_LOG, float, T>;
  __shared__ __attribute__((aligned(16))) float fa[WAVES][CB], fh[WAVES][CB];
  const int lane = ssd::lane_id(), wave = ssd::wave_id_s();
  const int chunk = static_cast<int>(blockIdx.x / p.cblocks), cb = static_cast<int>(blockIdx.x % p.cblocks);
  const int c0 = cb * CB + lane * V;
  const bool live = c0 < p.C;
  const int c = live ? c0 : p.C - V;
  const int r0 = chunk * CHUNK + wave * ROWS;
  Raw<T, V> x[ROWS], in[ROWS];
  Raw<G, V> g[ROWS];
#pragma unroll
  for (int j = 0; j < ROWS; ++j) {
    const int r = r0 + j < p.R ? r0 + j : p.R - 1;
    x[j].load(static_cast<const T*>(p.x) + row_offset(r, p, p.x_sb, p.x_sl) + c);
    g[j].load(static_cast<const G*>(p.g) + row_offset(r, p, p.g_sb, p.g_sl) + c);
    if (ING) in[j].load(static_cast<const T*>(p.i) + row_offset(r, p, p.i_sb, p.i_sl) + c);
  }
  Raw<float, V> decay;
  if (GATE == LINREC_GATE_DECAY) decay.load(p.decay + c);
  const uint32_t starts = starts_at(p, r0);
  float a[ROWS][V], b[ROWS][V], A[V], H[V];
#pragma unroll
  for (int v = 0; v < V; ++v) A[v] = 1.f, H[v] = 0.f;
#pragma unroll
  for (int j = 0; j < ROWS; ++j) {
    if (r0 + j < p.R) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const Gate q = gate_of<T, GATE, SCALE>(g[j].get(v), GATE == LINREC_GATE_DECAY ? decay.get(v) : 0.f);
        float u = x[j].get(v);
        if (ING) u *= Fn<T>::sigmoid(in[j].get(v));
        a[j][v] = q.a;
        b[j][v] = q.m * u;
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) a[j][v] = 1.f, b[j][v] = 0.f;
    }
    if ((starts >> j) & 1u) {
      if (p.h0) {
        const int s = sequence_of(p, r0 + j);
        if (s >= 0) {
          Raw<float, V> h0;
          h0.load(p.h0 + static_cast<int64_t>(s) * p.C + c);
#pragma unroll
          for (int v = 0; v < V; ++v) b[j][v] = fmaf(a[j][v], h0.get(v), b[j][v]);
        }
      }
#pragma unroll
      for (int v = 0; v < V; ++v) A[v] = 0.f, H[v] = b[j][v];
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        A[v] *= a[j][v];
        H[v] = fmaf(a[j][v], H[v], b[j][v]);
      }
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    fa[wave][lane * V + v] = A[v];
    fh[wave][lane * V + v] = H[v];
  }
  __syncthreads();
  if constexpr (AGG) {
    if (wave == 0 && live) {
      for (int w = 1; w < WAVES; ++w) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float f = fa[w][lane * V + v];
          A[v] = both(A[v], f);
          H[v] = onto(f, fh[w][lane * V + v], H[v]);
        }
      }
#pragma unroll
      for (int v = 0; v < V; ++v) p.agg[static_cast<int64_t>(chunk) * p.C + c + v] = float2{A[v], H[v]};
    }
  } else {
    float h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = chunk > 0 ? p.states[static_cast<int64_t>(chunk - 1) * p.C + c + v] : 0.f;
    for (int w = 0; w < wave; ++w) {
#pragma unroll
      for (int v = 0; v < V; ++v) h[v] = onto(fa[w][lane * V + v], fh[w][lane * V + v], h[v]);
    }
    const uint32_t lasts = starts >> 1 | (p.R - 1 - r0 < 32 && p.R > r0 ? 1u << (p.R - 1 - r0) : 0u);
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      const int r = r0 + j;
      if (r >= p.R) break;
      const bool start = (starts >> j) & 1u;
#pragma unroll
      for (int v = 0; v < V; ++v) h[v] = start ? b[j][v] : fmaf(a[j][v], h[v], b[j][v]);
      if (live) {
        Raw<T, V> out;
        out.set(h);
        out.store(static_cast<T*>(p.y) + static_cast<int64_t>(r) * p.C + c);
        if (p.final && ((lasts >> j) & 1u)) {
          const int s = sequence_of(p, r);
          if (s >= 0) {
            Raw<float, V> f;
            f.set(h);
            f.store(p.final + static_cast<int64_t>(s) * p.C + c);
          }
        }
      }
    }
    // numbered sequences past the last one
    if (p.final && p.seq_idx && chunk == 0 && wave == 0 && live) {
      for (int s = p.nseqs - 1; s >= 0 && p.starts[s] >= p.R; --s) {
#pragma unroll
        for (int v = 0; v < V; ++v) p.final[static_cast<int64_t>(s) * p.C + c + v] = p.h0 ? p.h0[static_cast<int64_t>(s) * p.C + c + v] : 0.f;
      }
    }
  }
}

// The states between the chunks, a channel a lane.
__global__ __launch_bounds__(64) void k_linrec_chain(Problem p) {
  const int c = static_cast<int>(blockIdx.x) * 64 + static_cast<int>(threadIdx.x);
  if (c >= p.C) return;
  float h = 0.f;
#pragma unroll 8
  for (int k = 0; k < p.chunks; ++k) {
    const float2 f = p.agg[static_cast<int64_t>(k) * p.C + c];
    h = onto(f.x, f.y, h);
    p.states[static_cast<int64_t>(k) * p.C + c] = h;
  }
}

namespace {
template <typename T, int GATE, int SCALE, bool ING> int go(const Problem& p, bool outputs, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(p.chunks * p.cblocks));
  hipLaunchKernelGGL((k_linrec<T, GATE, SCALE, ING, true>), grid, dim3(THR), 0, st, p);
  hipLaunchKernelGGL(k_linrec_chain, dim3(static_cast<unsigned>((p.C + 63) / 64)), dim3(64), 0, st, p);
  if (outputs) hipLaunchKernelGGL((k_linrec<T, GATE, SCALE, ING, false>), grid, dim3(THR), 0, st, p);
  return hipGetLastError() == hipSuccess ? SSD_OK : SSD_ERR_HIP;
}
template <typename T, int GATE, int SCALE> int by_in(const Problem& p, bool o, hipStream_t st) {
  return p.i ? go<T, GATE, SCALE, true>(p, o, st) : go<T, GATE, SCALE, false>(p, o, st);
}
template <typename T, int GATE> int by_scale(const Problem& p, int scale, bool o, hipStream_t st) {
  switch (scale) {
    case LINREC_INPUT_ONE: return by_in<T, GATE, LINREC_INPUT_ONE>(p, o, st);
    case LINREC_INPUT_COMPLEMENT: return by_in<T, GATE, LINREC_INPUT_COMPLEMENT>(p, o, st);
    default: return by_in<T, GATE, LINREC_INPUT_UNIT>(p, o, st);
  }
}
template <typename T> int by_gate(const Problem& p, const linrec_shape& s, bool o, hipStream_t st) {
  switch (s.gate) {
    case LINREC_GATE_LOG: return by_scale<T, LINREC_GATE_LOG>(p, s.input_scale, o, st);
    case LINREC_GATE_SIGMOID: return by_scale<T, LINREC_GATE_SIGMOID>(p, s.input_scale, o, st);
    default: return by_scale<T, LINREC_GATE_DECAY>(p, s.input_scale, o, st);
  }
}
}  // namespace

int launch_fwd(const Problem& p, const linrec_shape& s, bool outputs, hipStream_t st) {
  return s.io_dtype == SSD_IO_BF16 ? by_gate<bf16_t>(p, s, outputs, st) : by_gate<float>(p, s, outputs, st);
}

}  // namespace linrec
