// Problem descriptor of the gated linear recurrence's kernels, their gates and launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "linear_recurrence.h"
#include "ssd_device.h"
#include "ssd_tiles.h"

namespace linrec {

// The states are kept every SPAN rows, from the forward for the backward.
constexpr int SPAN = 64;

// A chunk, a block's rows: WAVES waves of ROWS rows each, a lane with BYTES of x of every row.  The more rows a chunk has,
// the fewer links the chain; the more values a lane keeps over the chain, the fewer blocks share a CU and its loads.
// Microseconds when they were chosen, at 16384 rows of 8192 bf16 channels with all gates, forward (and of 4096 channels,
// packed): 16 x 8 x 4 bytes 247 (150), 16 x 4 x 4 256 (161), 8 x 8 x 8 267 (168), 16 x 16 x 4 285 (166), 8 x 16 x 4 343
// (192).  Backward: 8 x 8 x 4 485, 16 x 4 x 4 524, 8 x 4 x 4 521, 8 x 4 x 8 575, 4 x 16 x 4 748.  For float32, one channel a
// lane, others were not tried: at 8192 rows of 4096 it stands 1.1 times the copy's time, 1.2 backward.
template <int R, int W, int B> struct Lay {
  static constexpr int ROWS = R, WAVES = W, BYTES = B, CHUNK = R * W, THR = 64 * W;
  template <typename T> static constexpr int VALS = B / static_cast<int>(sizeof(T));
};
using Fwd = Lay<16, 8, 4>;
using Bwd = Lay<8, 8, 4>;
// Rows that fit one chunk of sixteen waves need no chain and no launch before it: 200 rows of 256 channels 12.2 us a call
// and 14.8 in chunks of 128, 256 rows of 8192 channels 13.0 and 14.5.
using Short = Lay<16, 16, 4>;
static_assert(Fwd::CHUNK % SPAN == 0 && SPAN % Fwd::ROWS == 0 && Short::ROWS == Fwd::ROWS && Bwd::CHUNK == SPAN, "states at the ends of spans");
constexpr int LINE = 32;   // words of a cache line

struct Problem {
  int R, L, C, nseqs;      // rows (batch * seqlen), rows of a batch row, channels, sequences
  int spans;               // of SPAN rows
  int chunks, cblocks;     // a kernel's chunks and blocks of 64 VALS channels
  int64_t x_sb, x_sl, g_sb, g_sl, i_sb, i_sl;
  // inputs
  const void *x, *g, *i, *dy;
  const float *decay, *h0, *dfinal;
  const int32_t* seq_idx;
  int pass;                // the forward's operands are more than the last cache holds
  int keep;                // all spans' states are wanted, not only the chain's
  // outputs
  void *y, *dx, *dg, *di;
  float *final, *ddecay, *dh0;
  // workspace
  int32_t* starts;         // (nseqs + 1) first rows (seq_idx and states given)
  uint32_t* sync;          // (cblocks, LINE): tickets; (cblocks, chunks): what of a chunk is there
  float2* agg;             // (spans, C): a chunk's factor and what it adds, at its last span
  float* states;           // (spans, C): the state after each span
  float* carry;            // (spans, C): what a span hands to the rows before it (backward)
  float* slots;            // (spans, C): ddecay of each span (backward)
};

// with `chain` the tickets and marks, with `number` the sequences' first rows, before either of the others
int launch_setup(const Problem& p, bool chain, bool number, hipStream_t st);
inline bool chained_fwd(const Problem& p) { return p.R > Short::CHUNK; }
inline bool chained_bwd(const Problem& p) { return p.R > Bwd::CHUNK; }
// The chunks of one launch: a grid holds less than 2^32 threads (more are cut off without an error).  Those of the next go
// on with the tickets, in the same places of the chain.
inline int64_t chunks_a_launch(int64_t cblocks, int threads) { return ((int64_t{1} << 32) - 1) / threads / cblocks; }
template <typename Launch> int in_launches(const Problem& p, int threads, Launch launch) {
  const int64_t most = chunks_a_launch(p.cblocks, threads);
  for (int64_t left = p.chunks; left > 0; left -= most) {
    launch(dim3(static_cast<unsigned>((left < most ? left : most) * p.cblocks)));
    if (hipGetLastError() != hipSuccess) return SSD_ERR_HIP;
  }
  return SSD_OK;
}
int launch_fwd(const Problem& p, const linrec_shape& s, hipStream_t st);   // (p.y, p.final NULL: the states only)
int launch_bwd(const Problem& p, const linrec_shape& s, hipStream_t st);

#ifdef __HIPCC__
// V values of type S as they lie in memory (4 to 16 bytes).  PASS: not to be kept in the caches (the nontemporal hint).
template <typename S, int V> struct Raw {
  static constexpr int N = V * static_cast<int>(sizeof(S)) / 4;
  typedef uint32_t words __attribute__((ext_vector_type(N)));
  words w;
  __device__ __forceinline__ void load(const S* p) { w = *reinterpret_cast<const words*>(p); }
  // at a lane's byte offset from a row's address, which is the wave's: no 64-bit address per lane
  template <bool PASS> __device__ __forceinline__ void load_at(const void* base, int64_t row, uint32_t off) {
    const words* p = reinterpret_cast<const words*>(reinterpret_cast<const char*>(static_cast<const S*>(base) + row) + off);
    w = PASS ? __builtin_nontemporal_load(p) : *p;
  }
  __device__ __forceinline__ void store_at(void* base, int64_t row, uint32_t off) const {
    *reinterpret_cast<words*>(reinterpret_cast<char*>(static_cast<S*>(base) + row) + off) = w;
  }
  __device__ __forceinline__ float get(int e) const {
    if constexpr (sizeof(S) == 2) return __uint_as_float(e & 1 ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16);
    else return __uint_as_float(w[e]);
  }
  __device__ __forceinline__ void set(const float (&f)[V]) {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = sizeof(S) == 2 ? ssd::pack_bf16x2(f[sizeof(S) == 2 ? 2 * i : i], f[sizeof(S) == 2 ? 2 * i + 1 : i]) : __float_as_uint(f[i]);
  }
  __device__ __forceinline__ void store(S* p) const { *reinterpret_cast<words*>(p) = w; }
};

// A lane's offset in a row of elements of type S: 32 bits of which the compiler knows nothing, or it would widen them
template <typename S> __device__ __forceinline__ uint32_t lane_offset(int c) {
  uint32_t off = static_cast<uint32_t>(c) * static_cast<uint32_t>(sizeof(S));
  asm("" : "+v"(off));
  return off;
}

// With bf16 io the hardware's exponential, reciprocal and root (1 ulp); with float32 io the library's.
template <typename T> struct Fn {
  static constexpr bool FAST = sizeof(T) == 2;
  static constexpr float LOG2E = 1.4426950408889634f;
  static __device__ __forceinline__ float exp(float x) { return FAST ? __builtin_amdgcn_exp2f(x * LOG2E) : expf(x); }
  static __device__ __forceinline__ float rcp(float x) { return FAST ? __builtin_amdgcn_rcpf(x) : 1.f / x; }
  static __device__ __forceinline__ float sqrt(float x) { return FAST ? __builtin_amdgcn_sqrtf(x) : sqrtf(x); }
  static __device__ __forceinline__ float sigmoid(float x) { return rcp(1.f + exp(-x)); }
  // sigmoid(x) and 1 - sigmoid(x), both to their last bits: with e = exp(-x) the latter is e sigmoid(x) where x > 0
  static __device__ __forceinline__ float2 sigmoids(float x) {
    const float e = exp(-x), s = rcp(1.f + e);
    return float2{s, x > 0.f ? e * s : 1.f - s};
  }
  // sigmoid(x), and to keep the smaller of the two (1 - sigmoid(x) with its sign turned), from which both come again
  static __device__ __forceinline__ float sigmoid(float x, float& keep) {
    const float e = exp(-x), s = rcp(1.f + e);
    keep = x > 0.f ? -e * s : s;
    return s;
  }
  static __device__ __forceinline__ float2 both_of(float w) {
    const float o = 1.f - fabsf(w);
    return __float_as_int(w) < 0 ? float2{o, -w} : float2{w, o};
  }
  // 1 - exp(S y), y <= 0, from its direct form: with S y above -1/2 as -S y times the polynomial of degree 5 that is
  // nearest to (exp(t) - 1) / t there (off by 7e-9 of it, found by exchange).  Below it the direct form takes over what exp(y)
  // is off by, times S e / (1 - e) with e = exp(S y), which is most at -1/2: 1.5 for 1 - a, 3.1 for 1 - a^2, halved again by
  // the root that is taken of it.
  template <int S> static __device__ __forceinline__ float one_minus(float y, float direct) {
    constexpr float C[6] = {1.f, 4.999998211860657e-1f, 1.6666224598884583e-1f, 4.1629090905189514e-2f, 8.187386207282543e-3f, 1.1216348502784967e-3f};
    float q = C[5] * (S == 2 ? 64.f : 1.f);   // S^6 and down: powers of two change no bits
    q = fmaf(q, y, C[4] * (S == 2 ? 32.f : 1.f));
    q = fmaf(q, y, C[3] * (S == 2 ? 16.f : 1.f));
    q = fmaf(q, y, C[2] * (S == 2 ? 8.f : 1.f));
    q = fmaf(q, y, C[1] * (S == 2 ? 4.f : 1.f));
    q = fmaf(q, y, C[0] * S);
    return y > -0.5f / S ? -y * q : direct;
  }
};

// A channel's decay as its gates use it
template <typename T, int GATE> struct Decay {
  float k, k2;   // decay, and times log2(e): exp by the hardware's exp2 takes its argument from one product
  __device__ __forceinline__ explicit Decay(float decay) : k(decay), k2(decay * Fn<T>::LOG2E) {}
};

// Decay a, its logarithm la, or with LINREC_GATE_SIGMOID 1 - a
struct Factor {
  float a, la, rest;
};
template <typename T, int GATE> __device__ __forceinline__ Factor factor_of(float g, float2 s, Decay<T, GATE> d) {   // s: g's sigmoids
  using F = Fn<T>;
  Factor f{};
  if constexpr (GATE == LINREC_GATE_LOG) {
    f.la = g;
    f.a = F::exp(g);
  } else if constexpr (GATE == LINREC_GATE_SIGMOID) {
    f.a = s.x;
    f.rest = s.y;
  } else {
    f.la = d.k * s.x;
    f.a = F::FAST ? __builtin_amdgcn_exp2f(d.k2 * s.x) : F::exp(f.la);
  }
  return f;
}
template <typename T, int GATE> __device__ __forceinline__ Factor factor_of(float g, Decay<T, GATE> d) {
  if constexpr (GATE == LINREC_GATE_SIGMOID) return factor_of<T, GATE>(g, Fn<T>::sigmoids(g), d);
  else return factor_of<T, GATE>(g, float2{GATE == LINREC_GATE_DECAY ? Fn<T>::sigmoid(g) : 0.f, 0.f}, d);
}
// the input's factor m
template <typename T, int GATE, int SCALE> __device__ __forceinline__ float scale_of(const Factor& f) {
  using F = Fn<T>;
  if constexpr (SCALE == LINREC_INPUT_ONE) return 1.f;
  else if constexpr (SCALE == LINREC_INPUT_COMPLEMENT) return GATE == LINREC_GATE_SIGMOID ? f.rest : F::template one_minus<1>(f.la, 1.f - f.a);
  else return F::sqrt(GATE == LINREC_GATE_SIGMOID ? fmaf(f.rest, f.a, f.rest) : F::template one_minus<2>(f.la, fmaf(-f.a, f.a, 1.f)));
}
// Rows, a wave's or a chunk's, on a state.  Whether a sequence starts in them is known apart (`cut`), the same in all lanes:
// a product of decays that came to zero is a factor like others, on which a NaN or an infinity stays one, as it does row by row.
__device__ __forceinline__ float onto(bool cut, float factor, float add, float state) { return cut ? add : fmaf(factor, state, add); }

// ---------------------------------------------------------------------------
// The chunks' chain: a single-pass scan with look-back over the chunks before
// (Merrill and Garland, "Single-pass Parallel Prefix Scan with Decoupled
// Look-back", 2016), on states instead of sums, in an order of its own.
// A block takes its chunk by a ticket, so the chunks before it in the chain have
// begun and wait for none after it: every wait ends.  It
// leaves its own (A, H) at once (PART) and the state behind it as soon as the
// state before it is known (WHOLE); the next ones go back to the nearest chunk
// whose state is there and take the parts between up from it, one after the
// other, so that every state is formed in one order, wherever they found it.
//
// What blocks hand each other is written and read past the caches (relaxed
// atomics of the device's scope); a mark is written after its values have
// arrived, and the values are read after the mark was seen.  Nothing else has
// to be seen, so no fence writes an XCD's cache back for it (16384 x 8192
// forward 839 us with one, 238 without).
// ---------------------------------------------------------------------------
enum { NOTHING = 0, PART = 1, WHOLE = 2 };

__device__ __forceinline__ void put(float* p, float v) { __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
__device__ __forceinline__ float take(const float* p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
__device__ __forceinline__ void put(float2* p, float2 v) {
  __hip_atomic_store(reinterpret_cast<uint64_t*>(p), __builtin_bit_cast(uint64_t, v), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float2 take(const float2* p) {
  return __builtin_bit_cast(float2, __hip_atomic_load(reinterpret_cast<const uint64_t*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
}

// A block's channel block (blocks that follow each other take different ones), and its place in that one's chain: the next
// of its ticket counter.  Counters of their own, a cache line apart: one for all blocks served a ticket every 13 ns.
__device__ __forceinline__ int channel_block(const Problem& p) { return static_cast<int>(blockIdx.x % p.cblocks); }
__device__ __forceinline__ int ticket(const Problem& p, int cb) {
  __shared__ uint32_t t;
  if (p.chunks == 1) return 0;
  if (threadIdx.x == 0) t = __hip_atomic_fetch_add(p.sync + static_cast<int64_t>(cb) * LINE, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(t);
}

// One wave, for the lane's V channels from c on: the state before the chunk at `place` of the chain, and A, H onto it left
// for the chunks behind.  row_of(place): where the chunk there has its row in agg and in `after`, the states behind the
// chunks; cut: a sequence starts in it (then H is the state behind it, and A is not read).
template <int V, typename RowOf>
__device__ __forceinline__ void join(const Problem& p, float* after, int place, int cb, int c, bool cut, const float (&A)[V],
                                     const float (&H)[V], float (&before)[V], RowOf row_of) {
  const int lane = static_cast<int>(threadIdx.x) & 63;
  const int64_t mine = static_cast<int64_t>(row_of(place)) * p.C + c;
  uint32_t* marks = p.sync + static_cast<int64_t>(p.cblocks) * LINE + static_cast<int64_t>(cb) * p.chunks;
  auto mark = [&](uint32_t m) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // the values have arrived
    if (lane == 0) __hip_atomic_store(marks + place, m, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  };
  auto leave = [&](const float (&h)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) put(after + mine + v, h[v]);
    mark(WHOLE);
  };
  if (cut) {
    leave(H);
  } else if (place > 0) {
#pragma unroll
    for (int v = 0; v < V; ++v) put(p.agg + mine + v, float2{A[v], H[v]});
    mark(PART);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) before[v] = 0.f;
  if (place > 0) {
    int back = 0;   // places to go back to a known state, less one
    for (;;) {
      const int at = place - 1 - lane;
      uint32_t m = WHOLE;   // before the first chunk: a state of zero
      if (at >= 0) m = __hip_atomic_load(marks + at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      const uint64_t whole = __ballot(m == WHOLE), nothing = __ballot(m == NOTHING);
      if (whole) {
        back = __builtin_ctzll(whole);
        if ((nothing & ((uint64_t{1} << back) - 1)) == 0) break;
      }
      __builtin_amdgcn_s_sleep(1);
    }
    asm volatile("" ::: "memory");
    int from = place - 1 - back;
    if (from >= 0) {
      const int64_t at = static_cast<int64_t>(row_of(from)) * p.C + c;
#pragma unroll
      for (int v = 0; v < V; ++v) before[v] = take(after + at + v);
    }
    constexpr int AHEAD = 4;
    for (int q = from + 1; q < place; q += AHEAD) {
      float2 f[AHEAD][V];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        if (q + i < place && q + i >= 0) {
          const int64_t at = static_cast<int64_t>(row_of(q + i)) * p.C + c;
#pragma unroll
          for (int v = 0; v < V; ++v) f[i][v] = take(p.agg + at + v);
        }
      }
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        if (q + i < place && q + i >= 0) {
#pragma unroll
          for (int v = 0; v < V; ++v) before[v] = fmaf(f[i][v].x, before[v], f[i][v].y);   // no chunk between has a start: those leave a state
        }
      }
    }
  }
  if (!cut) {
    float h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = fmaf(A[v], before[v], H[v]);
    leave(h);
  }
}

// Where a wave's row lies in x, g and in_gate, from row to row
struct Cursor {
  int64_t x, g, i;
  int t;   // row of its batch row
  __device__ __forceinline__ Cursor(const Problem& p, int row) {
    const int b = __builtin_amdgcn_readfirstlane(row / p.L);   // the same in all lanes: addresses stay scalar
    t = row - b * p.L;
    x = b * p.x_sb + t * p.x_sl;
    g = b * p.g_sb + t * p.g_sl;
    i = b * p.i_sb + t * p.i_sl;
  }
  __device__ __forceinline__ void next(const Problem& p) {
    x += p.x_sl;
    g += p.g_sl;
    i += p.i_sl;
    if (++t == p.L) {   // the next batch row's first
      t = 0;
      x += p.x_sb - p.L * p.x_sl;
      g += p.g_sb - p.L * p.g_sl;
      i += p.i_sb - p.L * p.i_sl;
    }
  }
};

// bit j: a sequence starts at row r0 + j (j <= ROWS < 32; the last bit tells whether the wave's last row ends one)
template <int ROWS> __device__ __forceinline__ uint32_t starts_at(const Problem& p, int r0) {
  const int j = static_cast<int>(threadIdx.x) & 63, r = r0 + j;
  bool s = false;
  if (j <= ROWS && r < p.R) s = r % p.L == 0 || (p.seq_idx && p.seq_idx[r] != p.seq_idx[r - 1]);
  return static_cast<uint32_t>(__ballot(s));
}

// bit j: row r0 + j is the last of its sequence
template <int ROWS> __device__ __forceinline__ uint32_t ends_at(const Problem& p, int r0, uint32_t starts) {
  return starts >> 1 | (r0 < p.R && p.R - r0 <= ROWS ? 1u << (p.R - 1 - r0) : 0u);
}

// the sequence of row r, or -1 past the last numbered one
__device__ __forceinline__ int sequence_of(const Problem& p, int r) {
  if (!p.seq_idx) return r / p.L;
  if (p.starts[p.nseqs] <= r) return -1;
  int lo = 0, hi = p.nseqs;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.starts[mid] <= r) lo = mid; else hi = mid;
  }
  return lo;
}
#endif

}  // namespace linrec
