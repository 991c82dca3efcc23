// Gated linear recurrence over whole sequences, backward (the operation:
// include/linear_recurrence.h).  With e_t the gradient of h_t and c_t = a_t e_t
// what row t hands to the row before it (to the initial state where a sequence
// starts),
//
//     e_t = dy_t + c_{t+1}   (+ the final state's gradient at a sequence's last row)
//     du_t = m_t e_t,   dl_t = e_t (a_t h_{t-1} + dm_t u_t)   (l the log decay)
//
// and the gates' gradients follow from dl and du row by row.  The c form the
// same recurrence as the h, read from the end; the h are formed again from the
// states between the chunks, in float32.
#include "linrec_problem.h"

namespace linrec {

using ssd::bf16_t;

template <typename T, int GATE, int SCALE, bool ING> __global__ __launch_bounds__(THR) void k_linrec_bwd(Problem p) {
  constexpr int V = VALS<T>, CB = 64 * V;
  using G = std::conditional_t<GATE == LINREC_GATE_LOG, float, T>;
  __shared__ __attribute__((aligned(16))) float fa[WAVES][CB], fh[WAVES][CB], fc[WAVES][CB], enter[CB];
  __shared__ int cuts;
  const int lane = ssd::lane_id(), wave = ssd::wave_id_s();
  if (threadIdx.x == 0) cuts = 0;
  const uint32_t id = ticket(p);
  const int place = static_cast<int>(id / p.cblocks), cb = static_cast<int>(id % p.cblocks);
  const int chunk = p.chunks - 1 - place;   // from the end
  const int c0 = cb * CB + lane * V;
  const bool live = c0 < p.C;
  const int c = live ? c0 : p.C - V;
  const int r0 = chunk * CHUNK + wave * ROWS;
  Raw<T, V> x[ROWS], in[ROWS], dy[ROWS];
  Raw<G, V> g[ROWS];
#pragma unroll
  for (int j = 0; j < ROWS; ++j) {
    const int r = r0 + j < p.R ? r0 + j : p.R - 1;
    g[j].load(static_cast<const G*>(p.g) + row_offset(r, p, p.g_sb, p.g_sl) + c);
    dy[j].load(static_cast<const T*>(p.dy) + static_cast<int64_t>(r) * p.C + c);
    x[j].load(static_cast<const T*>(p.x) + row_offset(r, p, p.x_sb, p.x_sl) + c);
    if (ING) in[j].load(static_cast<const T*>(p.i) + row_offset(r, p, p.i_sb, p.i_sl) + c);
  }
  Raw<float, V> dk;
  if (GATE == LINREC_GATE_DECAY) dk.load(p.decay + c);
  auto decay = [&](int v) { return GATE == LINREC_GATE_DECAY ? dk.get(v) : 0.f; };
  const uint32_t starts = starts_at(p, r0);
  const uint32_t lasts = starts >> 1 | (p.R - 1 - r0 < 32 && p.R > r0 ? 1u << (p.R - 1 - r0) : 0u);
  float a[ROWS][V], h[ROWS][V];   // h: the state before each row, from a zero one
  float A[V], H[V];
#pragma unroll
  for (int v = 0; v < V; ++v) A[v] = 1.f, H[v] = 0.f;
#pragma unroll
  for (int j = 0; j < ROWS; ++j) {
    if (r0 + j >= p.R) {
#pragma unroll
      for (int v = 0; v < V; ++v) a[j][v] = 1.f, h[j][v] = 0.f;
      continue;
    }
    if ((starts >> j) & 1u) {
      const int s = p.h0 ? sequence_of(p, r0 + j) : -1;
#pragma unroll
      for (int v = 0; v < V; ++v) A[v] = 0.f, H[v] = s >= 0 ? p.h0[static_cast<int64_t>(s) * p.C + c + v] : 0.f;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const Gate q = gate_of<T, GATE, SCALE>(g[j].get(v), decay(v));
      a[j][v] = q.a;
      h[j][v] = H[v];
      float u = x[j].get(v);
      if (ING) u *= Fn<T>::sigmoid(in[j].get(v));
      H[v] = fmaf(q.a, H[v], q.m * u);
      A[v] *= q.a;
    }
  }
  // what the wave hands on, from nothing
  auto final_gradient = [&](int j, float (&e)[V]) {
    if (p.dfinal && ((lasts >> j) & 1u)) {
      const int s = sequence_of(p, r0 + j);
      if (s >= 0) {
#pragma unroll
        for (int v = 0; v < V; ++v) e[v] += p.dfinal[static_cast<int64_t>(s) * p.C + c + v];
      }
    }
  };
  float cr[V];
#pragma unroll
  for (int v = 0; v < V; ++v) cr[v] = 0.f;
#pragma unroll
  for (int j = ROWS - 1; j >= 0; --j) {
    if (r0 + j >= p.R) continue;
    float e[V];
#pragma unroll
    for (int v = 0; v < V; ++v) e[v] = dy[j].get(v) + cr[v];
    final_gradient(j, e);
    const bool start = (starts >> j) & 1u;
#pragma unroll
    for (int v = 0; v < V; ++v) cr[v] = start ? 0.f : a[j][v] * e[v];
  }
  const bool cut = starts & ((1u << ROWS) - 1);   // whatever its decays hold: nothing passes a sequence start, either way
#pragma unroll
  for (int v = 0; v < V; ++v) {
    fa[wave][lane * V + v] = cut ? 0.f : A[v];
    fh[wave][lane * V + v] = H[v];
    fc[wave][lane * V + v] = cr[v];
  }
  if (p.chunks == 1) __syncthreads();   // cuts is cleared
  if (lane == 0 && cut) cuts = 1;
  __syncthreads();
  float hin[V], sum[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    hin[v] = chunk > 0 ? p.states[static_cast<int64_t>(chunk - 1) * p.C + c + v] : 0.f;
    cr[v] = sum[v] = 0.f;
  }
  if (p.chunks > 1) {
    if (wave == 0) {
      float B[V];
#pragma unroll
      for (int v = 0; v < V; ++v) B[v] = 0.f, A[v] = 1.f;
      for (int w = WAVES - 1; w >= 0; --w) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float f = fa[w][lane * V + v];
          B[v] = onto(f, fc[w][lane * V + v], B[v]);
          A[v] = both(A[v], f);
        }
      }
      const int last = p.chunks - 1;
      join<V>(p, p.carry, place, cb, c, live, cuts != 0, A, B, cr, [last](int k) { return last - k; });
#pragma unroll
      for (int v = 0; v < V; ++v) enter[lane * V + v] = cr[v];
    }
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v) cr[v] = enter[lane * V + v];
  }
  for (int w = 0; w < wave; ++w) {
#pragma unroll
    for (int v = 0; v < V; ++v) hin[v] = onto(fa[w][lane * V + v], fh[w][lane * V + v], hin[v]);
  }
  for (int w = WAVES - 1; w > wave; --w) {
#pragma unroll
    for (int v = 0; v < V; ++v) cr[v] = onto(fa[w][lane * V + v], fc[w][lane * V + v], cr[v]);
  }
  // the states before the rows up to the first start get what is left of the entering one
  float left[V];
#pragma unroll
  for (int v = 0; v < V; ++v) left[v] = hin[v];
  bool inside = true;
#pragma unroll
  for (int j = 0; j < ROWS; ++j) {
    if ((starts >> j) & 1u) inside = false;
    if (inside) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        h[j][v] += left[v];
        left[v] *= a[j][v];
      }
    }
  }
#pragma unroll
  for (int j = ROWS - 1; j >= 0; --j) {
    const int r = r0 + j;
    if (r >= p.R) continue;
    float e[V], ox[V], og[V], oi[V];
    const bool start = (starts >> j) & 1u;
#pragma unroll
    for (int v = 0; v < V; ++v) e[v] = dy[j].get(v) + cr[v];
    final_gradient(j, e);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const Gate q = gate_of<T, GATE, SCALE>(g[j].get(v), decay(v));
      const float xv = x[j].get(v);
      float si = 1.f, ri = 0.f;
      if (ING) {
        const float2 sr = Fn<T>::sigmoids(in[j].get(v));
        si = sr.x;
        ri = sr.y;
      }
      const float u = xv * si, du = q.m * e[v];
      const float dl = e[v] * fmaf(q.a, h[j][v], q.dm * u);
      ox[v] = du * si;
      oi[v] = du * u * ri;
      og[v] = dl * q.dg;
      sum[v] += dl * q.sg;
      cr[v] = q.a * e[v];
    }
    if (live) {
      const int64_t at = static_cast<int64_t>(r) * p.C + c;
      Raw<T, V> o;
      o.set(ox);
      o.store(static_cast<T*>(p.dx) + at);
      Raw<G, V> og_;
      og_.set(og);
      og_.store(static_cast<G*>(p.dg) + at);
      if (ING) {
        o.set(oi);
        o.store(static_cast<T*>(p.di) + at);
      }
      if (start && p.dh0) {
        const int s = sequence_of(p, r);
        if (s >= 0) {
#pragma unroll
          for (int v = 0; v < V; ++v) p.dh0[static_cast<int64_t>(s) * p.C + c + v] = cr[v];
        }
      }
    }
    if (start) {
#pragma unroll
      for (int v = 0; v < V; ++v) cr[v] = 0.f;
    }
  }
  if (p.dh0 && p.seq_idx && chunk == 0 && wave == 0 && live) {   // numbered sequences past the last one
    for (int s = p.nseqs - 1; s >= 0 && p.starts[s] >= p.R; --s) {
#pragma unroll
      for (int v = 0; v < V; ++v) p.dh0[static_cast<int64_t>(s) * p.C + c + v] = p.dfinal ? p.dfinal[static_cast<int64_t>(s) * p.C + c + v] : 0.f;
    }
  }
  if constexpr (GATE == LINREC_GATE_DECAY) {
    if (p.ddecay) {
      __syncthreads();
#pragma unroll
      for (int v = 0; v < V; ++v) fc[wave][lane * V + v] = sum[v];
      __syncthreads();
      if (wave == 0 && live) {
        for (int w = 1; w < WAVES; ++w) {
#pragma unroll
          for (int v = 0; v < V; ++v) sum[v] += fc[w][lane * V + v];
        }
#pragma unroll
        for (int v = 0; v < V; ++v) p.slots[static_cast<int64_t>(chunk) * p.C + c + v] = sum[v];
      }
    }
  }
}

// ddecay: a channel per RED_ROWS threads, each adds every RED_ROWS-th chunk's sum in order, then those in order.
constexpr int RED_COLS = 32, RED_ROWS = 32;
__global__ __launch_bounds__(RED_COLS * RED_ROWS) void k_linrec_reduce(Problem p) {
  __shared__ double part[RED_ROWS][RED_COLS + 1];
  const int lc = static_cast<int>(threadIdx.x) % RED_COLS, lr = static_cast<int>(threadIdx.x) / RED_COLS;
  const int c = static_cast<int>(blockIdx.x) * RED_COLS + lc;
  double s = 0.0;
  if (c < p.C) {
#pragma unroll 4
    for (int k = lr; k < p.chunks; k += RED_ROWS) s += static_cast<double>(p.slots[static_cast<int64_t>(k) * p.C + c]);
  }
  part[lr][lc] = s;
  __syncthreads();
  if (lr == 0 && c < p.C) {
#pragma unroll
    for (int i = 1; i < RED_ROWS; ++i) s += part[i][lc];
    p.ddecay[c] = static_cast<float>(s);
  }
}

namespace {
template <typename T, int GATE, int SCALE, bool ING> int go(const Problem& p, hipStream_t st) {
  hipLaunchKernelGGL((k_linrec_bwd<T, GATE, SCALE, ING>), dim3(static_cast<unsigned>(p.chunks * p.cblocks)), dim3(THR), 0, st, p);
  if (GATE == LINREC_GATE_DECAY && p.ddecay)
    hipLaunchKernelGGL(k_linrec_reduce, dim3(static_cast<unsigned>((p.C + RED_COLS - 1) / RED_COLS)), dim3(RED_COLS * RED_ROWS), 0, st, p);
  return hipGetLastError() == hipSuccess ? SSD_OK : SSD_ERR_HIP;
}
template <typename T, int GATE, int SCALE> int by_in(const Problem& p, hipStream_t st) {
  return p.i ? go<T, GATE, SCALE, true>(p, st) : go<T, GATE, SCALE, false>(p, st);
}
template <typename T, int GATE> int by_scale(const Problem& p, int scale, hipStream_t st) {
  switch (scale) {
    case LINREC_INPUT_ONE: return by_in<T, GATE, LINREC_INPUT_ONE>(p, st);
    case LINREC_INPUT_COMPLEMENT: return by_in<T, GATE, LINREC_INPUT_COMPLEMENT>(p, st);
    default: return by_in<T, GATE, LINREC_INPUT_UNIT>(p, st);
  }
}
template <typename T> int by_gate(const Problem& p, const linrec_shape& s, hipStream_t st) {
  switch (s.gate) {
    case LINREC_GATE_LOG: return by_scale<T, LINREC_GATE_LOG>(p, s.input_scale, st);
    case LINREC_GATE_SIGMOID: return by_scale<T, LINREC_GATE_SIGMOID>(p, s.input_scale, st);
    default: return by_scale<T, LINREC_GATE_DECAY>(p, s.input_scale, st);
  }
}
}  // namespace

int launch_bwd(const Problem& p, const linrec_shape& s, hipStream_t st) {
  return s.io_dtype == SSD_IO_BF16 ? by_gate<bf16_t>(p, s, st) : by_gate<float>(p, s, st);
}

}  // namespace linrec
