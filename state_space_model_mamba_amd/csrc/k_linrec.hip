// Gated linear recurrence over whole sequences, forward (the operation:
// include/linear_recurrence.h).
//
// All batch rows lie behind each other as one run of rows, cut into chunks.  A
// chunk turns the state h that enters it into A h + H, A the product of its
// decays and H what a zero state would have become, and one with a sequence
// start inside into H.  So do a wave's rows within a chunk: their (A, H) meet in LDS,
// the chunks' in memory (linrec_problem.h).  A lane keeps its rows' a and b
// meanwhile, so every input is read once.
//
// Bound by HBM, and by how well two blocks a CU cover each other's phases.
// 16384 rows of 8192 bf16 channels with all gates (1.07 GB): 240 to 246 us by
// itself (4.4 TB/s), 238 to 260 in a training pass (least and median of the
// kernel trace); 230 with the chain cut out, 220 without the gates' arithmetic
// as well, which takes 137 us of the vector units' time.  8192 rows of 4096
// float32 channels: 117 us (4.6 TB/s); 89 with decay gates without input gate
// (4.5), 79 with log decays (5.1).
#include "linrec_problem.h"

namespace linrec {

using ssd::bf16_t;

// Two blocks a CU, at most 128 registers: asked for where the compiler would take 133 or 134 (log decays with a factor other
// than one and no input gate, bf16: 74 us with one block a CU, 62 with two and a register spilled, at 8192 x 4096).
template <typename L, typename T, int GATE, int SCALE, bool ING>
__global__ __launch_bounds__(L::THR, GATE == LINREC_GATE_LOG && SCALE != LINREC_INPUT_ONE && !ING ? 4 : 1) void k_linrec(Problem p) {
  constexpr int ROWS = L::ROWS, WAVES = L::WAVES, V = L::template VALS<T>, CB = 64 * V;
  using G = std::conditional_t<GATE == LINREC_GATE_LOG, float, T>;
  __shared__ __attribute__((aligned(16))) float fa[WAVES][CB], fh[WAVES][CB], enter[CB];
  __shared__ uint32_t cuts;   // bit w: a sequence starts in the rows of wave w
  const int lane = ssd::lane_id(), wave = ssd::wave_id_s();
  if (threadIdx.x == 0) cuts = 0;
  const int cb = channel_block(p), chunk = ticket(p, cb);
  // lanes past the last channels take those again: they write the same values to the same places
  const int c = cb * CB + lane * V < p.C ? cb * CB + lane * V : p.C - V;
  const uint32_t ct = lane_offset<T>(c), cg = lane_offset<G>(c);
  const int r0 = __builtin_amdgcn_readfirstlane(chunk * L::CHUNK + wave * ROWS), rows = p.R - r0;   // rows: those there are
  Raw<T, V> x[ROWS], in[ROWS];
  Raw<G, V> g[ROWS];
  auto request = [&](auto pass) {
    constexpr bool PASS = decltype(pass)::value;
    Cursor at(p, rows > 0 ? r0 : p.R - 1);
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      x[j].template load_at<PASS>(p.x, at.x, ct);
      g[j].template load_at<PASS>(p.g, at.g, cg);
      if (ING) in[j].template load_at<PASS>(p.i, at.i, ct);
      if (j + 1 < rows) at.next(p);
    }
  };
  if (p.pass) request(std::true_type{});
  else request(std::false_type{});
  Raw<float, V> dk;
  if (GATE == LINREC_GATE_DECAY) dk.load(p.decay + c);
  const uint32_t starts = starts_at<ROWS>(p, r0);
  const bool cut = starts & ((1u << ROWS) - 1);
  float a[ROWS][V], b[ROWS][V];
#pragma unroll
  for (int j = 0; j < ROWS; ++j) {   // rows outside: a row's operands make room for its a and b at once
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const Decay<T, GATE> d(GATE == LINREC_GATE_DECAY ? dk.get(v) : 0.f);
      const Factor f = factor_of<T, GATE>(g[j].get(v), d);
      float u = x[j].get(v);
      if (ING) u *= Fn<T>::sigmoid(in[j].get(v));
      a[j][v] = f.a;
      b[j][v] = scale_of<T, GATE, SCALE>(f) * u;
    }
  }
  if (rows < ROWS) {   // rows past the last leave a state as it is
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      if (j >= rows) {
#pragma unroll
        for (int v = 0; v < V; ++v) a[j][v] = 1.f, b[j][v] = 0.f;
      }
    }
  }
  if (cut && p.h0) {
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      const int s = (starts >> j) & 1u ? sequence_of(p, r0 + j) : -1;
      if (s >= 0) {
        Raw<float, V> h0;
        h0.load(p.h0 + static_cast<int64_t>(s) * p.C + c);
#pragma unroll
        for (int v = 0; v < V; ++v) b[j][v] = fmaf(a[j][v], h0.get(v), b[j][v]);
      }
    }
  }
  float A[V], H[V];
#pragma unroll
  for (int v = 0; v < V; ++v) A[v] = 1.f, H[v] = 0.f;
  // a start drops the state by selection, so that nothing of it (a NaN either) passes; A is then not read
  auto gather = [&](auto with_starts) {
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      const bool start = with_starts.value && ((starts >> j) & 1u);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        A[v] *= a[j][v];
        H[v] = start ? b[j][v] : fmaf(a[j][v], H[v], b[j][v]);
      }
    }
  };
  if (cut) gather(std::true_type{});
  else gather(std::false_type{});
#pragma unroll
  for (int v = 0; v < V; ++v) {
    fa[wave][lane * V + v] = A[v];
    fh[wave][lane * V + v] = H[v];
  }
  if (p.chunks == 1) __syncthreads();   // cuts is cleared
  if (lane == 0 && cut) atomicOr(&cuts, 1u << wave);
  __syncthreads();
  const uint32_t cut_waves = __builtin_amdgcn_readfirstlane(cuts);
  float h[V];
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = 0.f;
  if (p.chunks > 1) {
    if (wave == 0) {
      __builtin_amdgcn_s_setprio(3);   // the other chunks wait for it (250 -> 244 us at 16384 x 8192)
      for (int w = 1; w < WAVES; ++w) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float f = fa[w][lane * V + v];
          A[v] *= f;
          H[v] = onto((cut_waves >> w) & 1u, f, fh[w][lane * V + v], H[v]);
        }
      }
      const int last = p.spans - 1;
      join<V>(p, p.states, chunk, cb, c, cut_waves != 0, A, H, h, [last](int k) {
        const int s = (k + 1) * (L::CHUNK / SPAN) - 1;
        return s < last ? s : last;
      });
#pragma unroll
      for (int v = 0; v < V; ++v) enter[lane * V + v] = h[v];
      __builtin_amdgcn_s_setprio(0);
    }
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = enter[lane * V + v];
  }
  for (int w = 0; w < wave; ++w) {
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = onto((cut_waves >> w) & 1u, fa[w][lane * V + v], fh[w][lane * V + v], h[v]);
  }
  if (p.keep && wave * ROWS % SPAN == 0 && wave > 0 && rows > 0) {   // a span of the chunk ends before the wave's rows
    Raw<float, V> f;
    f.set(h);
    f.store(p.states + (static_cast<int64_t>(chunk) * (L::CHUNK / SPAN) + wave * ROWS / SPAN - 1) * p.C + c);
  }
  if (p.keep && p.chunks == 1 && wave == WAVES - 1) {   // the last, which no chain leaves
    Raw<float, V> f;
    float e[V];
#pragma unroll
    for (int v = 0; v < V; ++v) e[v] = onto(cut, A[v], H[v], h[v]);
    f.set(e);
    f.store(p.states + static_cast<int64_t>(p.spans - 1) * p.C + c);
  }
  if (!p.y) return;
  int64_t y = static_cast<int64_t>(r0) * p.C;
  const uint32_t ends = p.final ? ends_at<ROWS>(p, r0, starts) : 0;
  auto walk = [&](auto all) {   // all rows are there, and none begins or ends a sequence that matters
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      const bool start = !all.value && ((starts >> j) & 1u);
#pragma unroll
      for (int v = 0; v < V; ++v) h[v] = start ? b[j][v] : fmaf(a[j][v], h[v], b[j][v]);
      if (all.value || j < rows) {
        Raw<T, V> out;
        out.set(h);
        out.store_at(p.y, y, ct);
        if (!all.value && ((ends >> j) & 1u)) {
          const int s = sequence_of(p, r0 + j);
          if (s >= 0) {
            Raw<float, V> f;
            f.set(h);
            f.store(p.final + static_cast<int64_t>(s) * p.C + c);
          }
        }
      }
      y += p.C;
    }
  };
  if (cut || ends || rows < ROWS) walk(std::false_type{});
  else walk(std::true_type{});
  // numbered sequences past the last one
  if (p.final && p.seq_idx && chunk == 0 && wave == 0) {
    for (int s = p.nseqs - 1; s >= 0 && p.starts[s] >= p.R; --s) {
#pragma unroll
      for (int v = 0; v < V; ++v) p.final[static_cast<int64_t>(s) * p.C + c + v] = p.h0 ? p.h0[static_cast<int64_t>(s) * p.C + c + v] : 0.f;
    }
  }
}

// The first block numbers the sequences: their first rows in row order, from a stretch of rows at a time, a row a lane
// and all of a stretch's seq_idx in flight; the others (the first too, without sequences) clear the tickets and marks.
constexpr int SET_THR = 1024, SET_ROWS = 16;   // rows of a thread in a stretch
__global__ __launch_bounds__(SET_THR) void k_linrec_setup(Problem p, int number, int64_t n) {
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, wave = tid >> 6;
  if (static_cast<int>(blockIdx.x) >= number) {
    const int64_t from = static_cast<int64_t>(blockIdx.x) - number, step = static_cast<int64_t>(gridDim.x) - number;
    for (int64_t i = from * SET_THR + tid; i < n; i += step * SET_THR) p.sync[i] = 0;
    return;
  }
  constexpr int PARTS = SET_ROWS * SET_THR / 64;   // of 64 rows
  __shared__ int before[PARTS], all;               // starts before a part in its stretch, and in the stretch
  int base = 0;
  for (int64_t first = 0; first < p.R; first += SET_THR * SET_ROWS) {
    uint64_t mask[SET_ROWS];
    int32_t v[SET_ROWS], u[SET_ROWS];
#pragma unroll
    for (int k = 0; k < SET_ROWS; ++k) {
      const int64_t r = first + k * SET_THR + tid, at = r < p.R ? r : p.R - 1;
      v[k] = p.seq_idx[at];
      u[k] = p.seq_idx[at > 0 ? at - 1 : 0];
    }
#pragma unroll
    for (int k = 0; k < SET_ROWS; ++k) {
      const int64_t r = first + k * SET_THR + tid;
      mask[k] = __ballot(r < p.R && (v[k] != u[k] || static_cast<int>(r) % p.L == 0));
      if (lane == 0) before[k * (SET_THR / 64) + wave] = __popcll(mask[k]);
    }
    __syncthreads();
    if (wave == 0) {   // PARTS / 64 parts a lane
      int mine[PARTS / 64], sum = 0;
#pragma unroll
      for (int i = 0; i < PARTS / 64; ++i) {
        mine[i] = sum;
        sum += before[lane * (PARTS / 64) + i];
      }
      int incl = sum;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(incl, d);
        if (lane >= d) incl += o;
      }
#pragma unroll
      for (int i = 0; i < PARTS / 64; ++i) before[lane * (PARTS / 64) + i] = incl - sum + mine[i];
      if (lane == 63) all = incl;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < SET_ROWS; ++k) {
      const int at = base + before[k * (SET_THR / 64) + wave] + __popcll(mask[k] & ((uint64_t{1} << lane) - 1));
      if (((mask[k] >> lane) & 1) && at <= p.nseqs) p.starts[at] = static_cast<int>(first + k * SET_THR + tid);
    }
    base += all;
    __syncthreads();
  }
  for (int64_t s = static_cast<int64_t>(base) + tid; s <= p.nseqs; s += SET_THR) p.starts[s] = p.R;
}

int launch_setup(const Problem& p, bool chain, bool number, hipStream_t st) {
  const int64_t n = !chain ? 0 : static_cast<int64_t>(p.cblocks) * (p.spans + LINE);   // the backward's, which are more
  const int64_t blocks = (n + 4 * SET_THR - 1) / (4 * SET_THR), most = 512;
  const int64_t grid = (blocks < most ? blocks : most) + number;
  if (grid == 0) return SSD_OK;
  hipLaunchKernelGGL(k_linrec_setup, dim3(static_cast<unsigned>(grid)), dim3(SET_THR), 0, st, p, number ? 1 : 0, n);
  return hipGetLastError() == hipSuccess ? SSD_OK : SSD_ERR_HIP;
}

namespace {
template <typename L, typename T, int GATE, int SCALE, bool ING> int run(Problem p, hipStream_t st) {
  p.cblocks = (p.C + 64 * L::template VALS<T> - 1) / (64 * L::template VALS<T>);
  p.chunks = (p.R + L::CHUNK - 1) / L::CHUNK;
  return in_launches(p, L::THR, [&](dim3 grid) { hipLaunchKernelGGL((k_linrec<L, T, GATE, SCALE, ING>), grid, dim3(L::THR), 0, st, p); });
}
template <typename T, int GATE, int SCALE, bool ING> int go(const Problem& p, hipStream_t st) {
  return p.R > Fwd::CHUNK && !chained_fwd(p) ? run<Short, T, GATE, SCALE, ING>(p, st) : run<Fwd, T, GATE, SCALE, ING>(p, st);
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

int launch_fwd(const Problem& p, const linrec_shape& s, hipStream_t st) {
  return s.io_dtype == SSD_IO_BF16 ? by_gate<bf16_t>(p, s, st) : by_gate<float>(p, s, st);
}

}  // namespace linrec
