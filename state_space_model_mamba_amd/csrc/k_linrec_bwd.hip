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
// states between the spans, in float32, so neither they nor y are read.
//
// Bound by HBM and, beside it, by the gates' arithmetic: 476 us at 16384
// rows of 8192 bf16 channels with all gates (1.88 GB, 3.9 TB/s) by itself, 513 to
// 543 in a training pass (least and median of the kernel trace); the vector units
// are busy for 288 of it.  Of 485, before the requests had priority, it took 453
// with the chain cut out, 406 without the gates as well.  Without input gate it
// stands further from the copy's rate: 386 us (1.34 GB, 3.5 TB/s), and 108 to 111 at
// 8192 rows of 4096 (3.1 TB/s); what bounds that was not found out.  8192 rows of 4096
// float32 channels: 215 us with all gates (4.4 TB/s), 144 with log decays (4.7).
// With all seven values of an element kept in registers over the chain, one
// block a CU, it took 900; with the next chunk's operands requested ahead by
// blocks that stay, 735.
#include "linrec_problem.h"

namespace linrec {

using ssd::bf16_t;

// Two blocks a CU need at most 128 registers: the compiler takes up to 126 (decay gates without input gate; 156 us with one
// block a CU, 108 to 111 with two, at 8192 rows of 4096 bf16 channels).
template <typename T, int GATE, int SCALE, bool ING>
__global__ __launch_bounds__(Bwd::THR) void k_linrec_bwd(Problem p) {
  constexpr int ROWS = Bwd::ROWS, WAVES = Bwd::WAVES, THR = Bwd::THR, V = Bwd::VALS<T>, CB = 64 * V;
  constexpr bool DECAY = GATE == LINREC_GATE_DECAY;
  using G = std::conditional_t<GATE == LINREC_GATE_LOG, float, T>;
  __shared__ __attribute__((aligned(16))) float fa[WAVES][CB], fh[WAVES][CB], fc[WAVES][CB], enter[CB];
  __shared__ uint32_t cuts;   // bit w: a sequence starts in the rows of wave w
  const int lane = ssd::lane_id(), wave = ssd::wave_id_s();
  __builtin_amdgcn_s_setprio(2);   // until the requests are out, ahead of the other block's arithmetic (486 -> 479 us)
  if (threadIdx.x == 0) cuts = 0;
  const int cb = channel_block(p), place = ticket(p, cb);
  const int chunk = p.chunks - 1 - place;   // from the end
  // lanes past the last channels take those again: they write the same values to the same places
  const int c = cb * CB + lane * V < p.C ? cb * CB + lane * V : p.C - V;
  const uint32_t ct = lane_offset<T>(c), cg = lane_offset<G>(c);
  const int r0 = __builtin_amdgcn_readfirstlane(chunk * Bwd::CHUNK + wave * ROWS), rows = p.R - r0;   // rows: those there are
  Raw<T, V> x[ROWS], in[ROWS], dy[ROWS];
  Raw<G, V> g[ROWS];
  auto request = [&](auto pass) {
    constexpr bool PASS = decltype(pass)::value;
    Cursor at(p, rows > 0 ? r0 : p.R - 1);
    int64_t yat = static_cast<int64_t>(rows > 0 ? r0 : p.R - 1) * p.C;
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      g[j].template load_at<PASS>(p.g, at.g, cg);
      x[j].template load_at<PASS>(p.x, at.x, ct);
      if (ING) in[j].template load_at<PASS>(p.i, at.i, ct);
      dy[j].template load_at<PASS>(p.dy, yat, ct);
      if (j + 1 < rows) {
        at.next(p);
        yat += p.C;
      }
    }
  };
  if (p.pass) request(std::true_type{});
  else request(std::false_type{});
  __builtin_amdgcn_s_setprio(0);
  Raw<float, V> entering;   // the state that enters the chunk
  if (chunk > 0) entering.load(p.states + static_cast<int64_t>(chunk - 1) * p.C + c);
  else entering.w = 0;
  const uint32_t starts = starts_at<ROWS>(p, r0), ends = p.dfinal ? ends_at<ROWS>(p, r0, starts) : 0;
  const bool cut = starts & ((1u << ROWS) - 1);
  // Of every element its decay, its input factor, and what it adds to the state, later the state before it; and in LDS the
  // sigmoids of its gates: the lane's registers for them as well would leave room for one block a CU.
  constexpr bool KEEP_G = GATE != LINREC_GATE_LOG;
  constexpr int KEPT = (KEEP_G ? V : 0) + (ING ? V : 0);
  __shared__ __attribute__((aligned(16))) float kept[KEPT ? ROWS * THR * KEPT : 1];
  float* mine = kept + static_cast<int>(threadIdx.x) * KEPT;   // row j: THR KEPT j further
  float a[ROWS][V], m[ROWS][V], h[ROWS][V];
  Raw<float, V> dk;
  if (DECAY) dk.load(p.decay + c);
#pragma unroll
  for (int j = 0; j < ROWS; ++j) {
    float k[KEPT + 1];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const Decay<T, GATE> d(DECAY ? dk.get(v) : 0.f);
      float2 s{0.f, 0.f};
      float u = x[j].get(v);
      if (KEEP_G) s.x = Fn<T>::sigmoid(g[j].get(v), k[v]);
      if (GATE == LINREC_GATE_SIGMOID) s.y = Fn<T>::both_of(k[v]).y;
      if (ING) u *= Fn<T>::sigmoid(in[j].get(v), k[(KEEP_G ? V : 0) + v]);
      const Factor f = factor_of<T, GATE>(g[j].get(v), s, d);
      a[j][v] = f.a;
      m[j][v] = scale_of<T, GATE, SCALE>(f);
      h[j][v] = m[j][v] * u;
    }
#pragma unroll
    for (int i = 0; i < KEPT; ++i) mine[THR * KEPT * j + i] = k[i];
  }
  if (rows < ROWS) {   // rows past the last hand on what they get
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      if (j >= rows) {
        dy[j].w = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) a[j][v] = 1.f, h[j][v] = 0.f;
      }
    }
  }
  auto gradient_of = [&](auto all, int j, float (&e)[V]) {   // dy, and the final state's where a sequence ends
#pragma unroll
    for (int v = 0; v < V; ++v) e[v] = dy[j].get(v);
    if (!all.value && ((ends >> j) & 1u)) {
      const int s = sequence_of(p, r0 + j);
      if (s >= 0) {
#pragma unroll
        for (int v = 0; v < V; ++v) e[v] += p.dfinal[static_cast<int64_t>(s) * p.C + c + v];
      }
    }
  };
  // The wave's factor and what a zero state becomes over it, and what it hands back from nothing.  A start drops the
  // state by selection, so that nothing of it (a NaN either) passes, in either direction; A is then not read.
  float A[V], H[V], cr[V];
#pragma unroll
  for (int v = 0; v < V; ++v) A[v] = 1.f, H[v] = cr[v] = 0.f;
  auto initial = [&](int j, float (&h0)[V]) {
    const int s = p.h0 ? sequence_of(p, r0 + j) : -1;
#pragma unroll
    for (int v = 0; v < V; ++v) h0[v] = s >= 0 ? p.h0[static_cast<int64_t>(s) * p.C + c + v] : 0.f;
  };
  auto gather = [&](auto all) {   // all rows are there, and none begins or ends a sequence that matters
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      if (!all.value && ((starts >> j) & 1u)) initial(j, H);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        A[v] *= a[j][v];
        H[v] = fmaf(a[j][v], H[v], h[j][v]);
      }
    }
#pragma unroll
    for (int j = ROWS - 1; j >= 0; --j) {
      const bool start = !all.value && ((starts >> j) & 1u);
      float e[V];
      gradient_of(all, j, e);
#pragma unroll
      for (int v = 0; v < V; ++v) cr[v] = start ? 0.f : a[j][v] * (e[v] + cr[v]);
    }
  };
  const bool some = cut || ends || rows < ROWS;
  if (some) gather(std::false_type{});
  else gather(std::true_type{});
#pragma unroll
  for (int v = 0; v < V; ++v) {
    fa[wave][lane * V + v] = A[v];
    fh[wave][lane * V + v] = H[v];
    fc[wave][lane * V + v] = cr[v];
  }
  if (p.chunks == 1) __syncthreads();   // cuts is cleared
  if (lane == 0 && cut) atomicOr(&cuts, 1u << wave);
  __syncthreads();
  const uint32_t cut_waves = __builtin_amdgcn_readfirstlane(cuts);
#pragma unroll
  for (int v = 0; v < V; ++v) H[v] = entering.get(v), cr[v] = 0.f;
  if (p.chunks > 1) {
    if (wave == 0) {
      float B[V];
#pragma unroll
      for (int v = 0; v < V; ++v) B[v] = 0.f, A[v] = 1.f;
      for (int w = WAVES - 1; w >= 0; --w) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float f = fa[w][lane * V + v];
          B[v] = onto((cut_waves >> w) & 1u, f, fc[w][lane * V + v], B[v]);
          A[v] *= f;
        }
      }
      const int last = p.chunks - 1;
      join<V>(p, p.carry, place, cb, c, cut_waves != 0, A, B, cr, [last](int k) { return last - k; });
#pragma unroll
      for (int v = 0; v < V; ++v) enter[lane * V + v] = cr[v];
    }
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v) cr[v] = enter[lane * V + v];
  }
  for (int w = 0; w < wave; ++w) {
#pragma unroll
    for (int v = 0; v < V; ++v) H[v] = onto((cut_waves >> w) & 1u, fa[w][lane * V + v], fh[w][lane * V + v], H[v]);
  }
  for (int w = WAVES - 1; w > wave; --w) {
#pragma unroll
    for (int v = 0; v < V; ++v) cr[v] = onto((cut_waves >> w) & 1u, fa[w][lane * V + v], fc[w][lane * V + v], cr[v]);
  }
  float sum[V];
#pragma unroll
  for (int v = 0; v < V; ++v) sum[v] = 0.f;
  int64_t out = (static_cast<int64_t>(r0) + ROWS - 1) * p.C;
  auto walk = [&](auto all) {
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {   // h: from what a row adds to the state before it
      if (!all.value && ((starts >> j) & 1u)) initial(j, H);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float add = h[j][v];
        h[j][v] = H[v];
        H[v] = fmaf(a[j][v], H[v], add);
      }
    }
#pragma unroll
    for (int j = ROWS - 1; j >= 0; --j) {
      float e[V], ox[V], og[V], oi[V], k[KEPT + 1];
      gradient_of(all, j, e);
#pragma unroll
      for (int i = 0; i < KEPT; ++i) k[i] = mine[THR * KEPT * j + i];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float ev = e[v] + cr[v], av = a[j][v], mv = m[j][v], du = ev * mv;
        float u = x[j].get(v);
        ox[v] = du;
        if (ING) {
          const float2 s = Fn<T>::both_of(k[(KEEP_G ? V : 0) + v]);
          u *= s.x;
          ox[v] = du * s.x;
          oi[v] = du * u * s.y;
        }
        float dl = av * h[j][v];   // e times the log decay's share: a h, and m's slope times u
        if constexpr (SCALE == LINREC_INPUT_COMPLEMENT) dl = av * (h[j][v] - u);
        if constexpr (SCALE == LINREC_INPUT_UNIT) dl = mv == 0.f ? dl : av * fmaf(-av * Fn<T>::rcp(mv), u, h[j][v]);
        dl *= ev;
        og[v] = dl;
        if constexpr (KEEP_G) {
          const float2 s = Fn<T>::both_of(k[v]);
          og[v] = dl * s.y;
          if (DECAY) {
            const float share = dl * s.x;
            og[v] = dk.get(v) * share * s.y;
            if (all.value || j < rows) sum[v] += share;
          }
        }
        cr[v] = av * ev;
      }
      if (all.value || j < rows) {
        Raw<T, V> o;
        o.set(ox);
        o.store_at(p.dx, out, ct);
        Raw<G, V> q;
        q.set(og);
        q.store_at(p.dg, out, cg);
        if (ING) {
          o.set(oi);
          o.store_at(p.di, out, ct);
        }
      }
      out -= p.C;
      if (!all.value && ((starts >> j) & 1u)) {
        const int s = p.dh0 ? sequence_of(p, r0 + j) : -1;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          if (s >= 0) p.dh0[static_cast<int64_t>(s) * p.C + c + v] = cr[v];
          cr[v] = 0.f;
        }
      }
    }
  };
  if (some) walk(std::false_type{});
  else walk(std::true_type{});
  if (p.dh0 && p.seq_idx && chunk == 0 && wave == 0) {   // numbered sequences past the last one
    for (int s = p.nseqs - 1; s >= 0 && p.starts[s] >= p.R; --s) {
#pragma unroll
      for (int v = 0; v < V; ++v) p.dh0[static_cast<int64_t>(s) * p.C + c + v] = p.dfinal ? p.dfinal[static_cast<int64_t>(s) * p.C + c + v] : 0.f;
    }
  }
  if constexpr (DECAY) {
    if (p.ddecay) {
      __syncthreads();
#pragma unroll
      for (int v = 0; v < V; ++v) fc[wave][lane * V + v] = sum[v];
      __syncthreads();
      if (wave == 0) {
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
    for (int k = lr; k < p.spans; k += RED_ROWS) s += static_cast<double>(p.slots[static_cast<int64_t>(k) * p.C + c]);
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
template <typename T, int GATE, int SCALE, bool ING> int go(Problem p, hipStream_t st) {
  p.cblocks = (p.C + 64 * Bwd::VALS<T> - 1) / (64 * Bwd::VALS<T>);
  p.chunks = p.spans;
  const int rc = in_launches(p, Bwd::THR, [&](dim3 grid) { hipLaunchKernelGGL((k_linrec_bwd<T, GATE, SCALE, ING>), grid, dim3(Bwd::THR), 0, st, p); });
  if (rc != SSD_OK) return rc;
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
