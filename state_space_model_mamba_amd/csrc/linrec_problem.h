// Problem descriptor of the gated linear recurrence's kernels, their gates and launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "linear_recurrence.h"
#include "ssd_device.h"
#include "ssd_tiles.h"

namespace linrec {

// A chunk's rows by a block: WAVES waves of ROWS rows each; a lane holds 8 bytes of x of each row.
constexpr int ROWS = 8, WAVES = 8, CHUNK = ROWS * WAVES, THR = 64 * WAVES;
template <typename T> constexpr int VALS = 8 / static_cast<int>(sizeof(T));

struct Problem {
  int R, L, C, nseqs;      // rows (batch * seqlen), rows of a batch row, channels, sequences
  int chunks, cblocks;     // chunks of CHUNK rows, blocks of 64 VALS channels
  int flat;                // batch rows follow each other at the row strides
  int64_t x_sb, x_sl, g_sb, g_sl, i_sb, i_sl;
  // inputs
  const void *x, *g, *i, *dy;
  const float *decay, *h0, *dfinal;
  const int32_t* seq_idx;
  // outputs
  void *y, *dx, *dg, *di;
  float *final, *ddecay, *dh0;
  // workspace
  int32_t* starts;         // (nseqs + 1) first rows (seq_idx and states given), then nseqs more that only k_delta_starts reads
  uint32_t* sync;          // the next ticket, then (chunks, cblocks): what of a chunk is there
  float2* agg;             // (chunks, C): a chunk's factor and what it adds
  float* states;           // (chunks, C): the state after each chunk
  float* carry;            // (chunks, C): what a chunk hands to the rows before it (backward)
  float* slots;            // (chunks, C): ddecay of each chunk (backward)
};

int launch_clear(const Problem& p, hipStream_t st);   // the tickets, before either of the others
int launch_fwd(const Problem& p, const linrec_shape& s, hipStream_t st);   // (p.y, p.final NULL: the states only)
int launch_bwd(const Problem& p, const linrec_shape& s, hipStream_t st);

#ifdef __HIPCC__
// V values of type S as they lie in memory (4 to 16 bytes)
template <typename S, int V> struct Raw {
  static constexpr int N = V * static_cast<int>(sizeof(S)) / 4;
  typedef uint32_t words __attribute__((ext_vector_type(N)));
  words w;
  __device__ __forceinline__ void load(const S* p) { w = *reinterpret_cast<const words*>(p); }
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

// With bf16 io the hardware's exponential, reciprocal and root (1 ulp); with float32 io the library's.
template <typename T> struct Fn {
  static constexpr bool FAST = sizeof(T) == 2;
  static __device__ __forceinline__ float exp(float x) { return FAST ? __expf(x) : expf(x); }
  static __device__ __forceinline__ float rcp(float x) { return FAST ? __builtin_amdgcn_rcpf(x) : 1.f / x; }
  static __device__ __forceinline__ float sqrt(float x) { return FAST ? __builtin_amdgcn_sqrtf(x) : sqrtf(x); }
  static __device__ __forceinline__ float sigmoid(float x) { return rcp(1.f + exp(-x)); }
  // sigmoid(x) and 1 - sigmoid(x), both to their last bits
  static __device__ __forceinline__ float2 sigmoids(float x) {
    const float e = exp(-fabsf(x)), big = rcp(1.f + e), small = e * big;
    return x < 0.f ? float2{small, big} : float2{big, small};
  }
  // 1 - exp(y) from e = exp(y): for y above -1/2 by the series -y (1 + y/2 (1 + y/3 (...))), whose eighth term is
  // below 2^-22 of the sum there; below it 1 - e loses at most one bit
  static __device__ __forceinline__ float one_minus(float y, float e) {
    float s = 1.f + y * (1.f / 8.f);
    s = fmaf(s, y * (1.f / 7.f), 1.f);
    s = fmaf(s, y * (1.f / 6.f), 1.f);
    s = fmaf(s, y * (1.f / 5.f), 1.f);
    s = fmaf(s, y * (1.f / 4.f), 1.f);
    s = fmaf(s, y * (1.f / 3.f), 1.f);
    s = fmaf(s, y * (1.f / 2.f), 1.f);
    return y > -0.5f ? -y * s : 1.f - e;
  }
};

struct Gate {
  float a, m;       // decay and input factor
  float dm;         // of m by the log decay
  float dg;         // of the log decay by g
  float sg;         // sigmoid(g) (LINREC_GATE_DECAY)
};
template <typename T, int GATE, int SCALE> __device__ __forceinline__ Gate gate_of(float g, float decay) {
  using F = Fn<T>;
  Gate q;
  float la = g, rest = 0.f;   // the log decay, 1 - a
  q.sg = 0.f;
  if constexpr (GATE == LINREC_GATE_SIGMOID) {
    const float2 s = F::sigmoids(g);
    q.a = s.x;
    q.dg = rest = s.y;
  } else {
    q.dg = 1.f;
    if constexpr (GATE == LINREC_GATE_DECAY) {
      const float2 s = F::sigmoids(g);
      q.sg = s.x;
      la = decay * q.sg;
      q.dg = la * s.y;
    }
    q.a = F::exp(la);
  }
  if constexpr (SCALE == LINREC_INPUT_ONE) {
    q.m = 1.f;
    q.dm = 0.f;
  } else if constexpr (SCALE == LINREC_INPUT_COMPLEMENT) {
    q.m = GATE == LINREC_GATE_SIGMOID ? rest : F::one_minus(la, q.a);
    q.dm = -q.a;
  } else {
    q.m = F::sqrt(GATE == LINREC_GATE_SIGMOID ? rest * (1.f + q.a) : F::one_minus(2.f * la, q.a * q.a));
    q.dm = q.m == 0.f ? 0.f : -q.a * q.a * F::rcp(q.m);
  }
  return q;
}

// a chunk or part of it on a state: what decayed to nothing is dropped, so nothing of it (a NaN either) passes on
__device__ __forceinline__ float onto(float factor, float add, float state) { return factor == 0.f ? add : fmaf(factor, state, add); }

// the factor of two parts; one that drops the state drops it whatever the other holds
__device__ __forceinline__ float both(float f, float g) { return f == 0.f || g == 0.f ? 0.f : f * g; }

// ---------------------------------------------------------------------------
// The chunks' chain.  A block takes its chunk by a ticket, so the chunks before
// it in the chain have begun and wait for none after it: every wait ends.  It
// leaves its own (A, H) at once (PART) and the state behind it as soon as the
// state before it is known (WHOLE); the next ones go back to the nearest chunk
// whose state is there and take the parts between up from it, one after the
// other, so that every state is formed in one order, wherever they found it.
//
// What blocks hand each other is written and read past the caches (relaxed
// atomics of the device's scope); a mark is written after its values have
// arrived, and the values are read after the mark was seen.
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

// The place of the block in the chain times cblocks, plus its channel block; the same in all threads.
__device__ __forceinline__ uint32_t ticket(const Problem& p) {
  __shared__ uint32_t t;
  if (p.chunks == 1) return blockIdx.x;
  if (threadIdx.x == 0) t = __hip_atomic_fetch_add(p.sync, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(t);
}

// One wave, for the lane's V channels from c on: the state before the chunk at `place` of the chain, and A, H onto it left
// for the chunks behind.  chunk_at(place): the chunk there; after: the states behind the chunks; cut: a sequence starts in it.
template <int V, typename ChunkAt>
__device__ __forceinline__ void join(const Problem& p, float* after, int place, int cb, int c, bool live, bool cut, const float (&A)[V],
                                     const float (&H)[V], float (&before)[V], ChunkAt chunk_at) {
  const int lane = static_cast<int>(threadIdx.x) & 63;
  const int64_t mine = static_cast<int64_t>(chunk_at(place)) * p.C + c;
  auto mark = [&](uint32_t m) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // the values have arrived
    if (lane == 0) __hip_atomic_store(p.sync + 1 + static_cast<int64_t>(place) * p.cblocks + cb, m, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  };
  auto leave = [&](const float (&h)[V]) {
    if (live) {
#pragma unroll
      for (int v = 0; v < V; ++v) put(after + mine + v, h[v]);
    }
    mark(WHOLE);
  };
  if (cut) {
    leave(H);
  } else if (place > 0) {
    if (live) {
#pragma unroll
      for (int v = 0; v < V; ++v) put(p.agg + mine + v, float2{A[v], H[v]});
    }
    mark(PART);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) before[v] = 0.f;
  if (place > 0) {
    int back = 0;   // places to go back to a known state, less one
    for (;;) {
      const int at = place - 1 - lane;
      uint32_t m = WHOLE;   // before the first chunk: a state of zero
      if (at >= 0) m = __hip_atomic_load(p.sync + 1 + static_cast<int64_t>(at) * p.cblocks + cb, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
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
      const int64_t at = static_cast<int64_t>(chunk_at(from)) * p.C + c;
#pragma unroll
      for (int v = 0; v < V; ++v) before[v] = take(after + at + v);
    }
    constexpr int AHEAD = 4;
    for (int q = from + 1; q < place; q += AHEAD) {
      float2 f[AHEAD][V];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        if (q + i < place && q + i >= 0) {
          const int64_t at = static_cast<int64_t>(chunk_at(q + i)) * p.C + c;
#pragma unroll
          for (int v = 0; v < V; ++v) f[i][v] = take(p.agg + at + v);
        }
      }
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        if (q + i < place && q + i >= 0) {
#pragma unroll
          for (int v = 0; v < V; ++v) before[v] = onto(f[i][v].x, f[i][v].y, before[v]);
        }
      }
    }
  }
  if (!cut) {
    float h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = onto(A[v], H[v], before[v]);
    leave(h);
  }
}

__device__ __forceinline__ int64_t row_offset(int row, const Problem& p, int64_t sb, int64_t sl) {
  if (p.flat) return row * sl;
  const int b = row / p.L;
  return b * sb + (row - b * p.L) * sl;
}

// bit j: a sequence starts at row r0 + j (j <= ROWS)
__device__ __forceinline__ uint32_t starts_at(const Problem& p, int r0) {
  const int j = static_cast<int>(threadIdx.x) & 63, r = r0 + j;
  bool s = false;
  if (j <= ROWS && r < p.R) s = r % p.L == 0 || (p.seq_idx && p.seq_idx[r] != p.seq_idx[r - 1]);
  return static_cast<uint32_t>(__ballot(s));
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
