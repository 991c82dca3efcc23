// Gated delta rule for few tokens on a pool of states (include/gated_delta.h,
// delta_step).
//
// A token costs 7 P N operations on a state of 4 P N bytes that is read and
// written once: bound by HBM (and for one sequence by latency).  A wave holds
// 8 RG rows of one head's state in registers, a row in 8 lanes of 16-byte
// pieces, so a load covers eight 128-byte stretches; rows need each other for
// nothing.  S q is taken with S k from the same decayed state,
//     o = scale (Sd q + beta e (k . q)),
// so the row sums of a token are one round of lane exchanges and not two.
#include <hip/hip_runtime.h>

#include "delta_problem.h"
#include "gated_delta.h"
#include "ssd_device.h"
#include "ssd_tiles.h"

namespace delta {

using ssd::bf16_t;
using ssd::f32x4_t;

struct StepArgs {
  const void *q, *k, *v;
  const float *g, *beta;
  float* states;
  const int32_t* index;
  void* o;
  int64_t nslots, q_sb, q_sl, k_sb, k_sl, v_sb, v_sl;
  int B, T, H, P, G, N, hpg, nblk;
  float scale;
};

// sum over the 8 lanes lane / 8; all receive the same bits
__device__ __forceinline__ float sum8(float v) {
  v += ssd::dpp_move<0xB1>(v);    // quad_perm [1,0,3,2]
  v += ssd::dpp_move<0x4E>(v);    // quad_perm [2,3,0,1]
  v += ssd::dpp_move<0x141>(v);   // row_half_mirror
  return v;
}

constexpr int STEP_WAVES = 4;

// NV: 16-byte pieces of a state row per lane (N <= 32 NV); RG: rows per lane
template <typename T, int NV, int RG> __global__ __launch_bounds__(64 * STEP_WAVES) void k_delta_step(StepArgs a) {
  const int tid = static_cast<int>(threadIdx.x), l = tid & 63, l8 = l & 7;
  const int h = static_cast<int>(blockIdx.x) / a.nblk, pb = static_cast<int>(blockIdx.x) % a.nblk;
  int b = static_cast<int>(blockIdx.y);
  const int grp = h / a.hpg;
  const int row0 = (pb * STEP_WAVES + tid / 64) * 8 * RG + (l >> 3);   // rows row0 + 8 i
  int64_t slot = b;
  int next = a.B;   // the next batch row of this state
  bool skip = false;
  if (a.index) {
    const int mine = a.index[b];
    for (int i0 = 0; i0 < a.B; i0 += 64) {
      const bool same = i0 + l < a.B && a.index[i0 + l] == mine;
      const uint64_t m = __ballot(same);
      const int at = b - i0;   // this row's place in the 64
      if (at > 0 && (m & (at >= 64 ? ~0ull : (1ull << at) - 1))) skip = true;
      const uint64_t later = at < 0 ? m : at >= 63 ? 0 : m >> (at + 1) << (at + 1);
      if (later && next == a.B) next = i0 + __builtin_ctzll(later);
    }
    slot = mine;
    if (mine < 0 || mine >= a.nslots) {   // an empty row
      for (int t = 0; t < a.T; ++t) {
#pragma unroll
        for (int i = 0; i < RG; ++i) {
          const int p = row0 + 8 * i;
          if (l8 == 0 && p < a.P)
            static_cast<T*>(a.o)[((static_cast<int64_t>(b) * a.T + t) * a.H + h) * a.P + p] = ssd::Elem<T>::from_f(0.f);
        }
      }
      return;
    }
    if (skip) return;   // an earlier row's block takes this row's tokens too
  }
  float* sp = a.states + (slot * a.H + h) * static_cast<int64_t>(a.P) * a.N;
  f32x4_t S[RG][NV];
#pragma unroll
  for (int i = 0; i < RG; ++i) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int p = row0 + 8 * i, n = 4 * (l8 + 8 * j);
      S[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      if (p < a.P && n < a.N) S[i][j] = *reinterpret_cast<const f32x4_t*>(sp + static_cast<int64_t>(p) * a.N + n);
    }
  }
  for (;;) {
    const T* qp = static_cast<const T*>(a.q) + b * a.q_sb + static_cast<int64_t>(grp) * a.N;
    const T* kp = static_cast<const T*>(a.k) + b * a.k_sb + static_cast<int64_t>(grp) * a.N;
    const T* vp = static_cast<const T*>(a.v) + b * a.v_sb + static_cast<int64_t>(h) * a.P;
    // a token's operands are requested while the one before is worked on
    struct Token {
      f32x4_t q[NV], k[NV];
      float v[RG], g, beta;
    };
    auto request = [&](int t) {
      Token x;
      const int64_t at = static_cast<int64_t>(b) * a.T + t;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int n = 4 * (l8 + 8 * j);
        x.q[j] = x.k[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        if (n < a.N) {
          x.q[j] = ssd::load4f<T>(qp + t * a.q_sl + n);
          x.k[j] = ssd::load4f<T>(kp + t * a.k_sl + n);
        }
      }
#pragma unroll
      for (int i = 0; i < RG; ++i) x.v[i] = row0 + 8 * i < a.P ? ssd::Elem<T>::to_f(vp[t * a.v_sl + row0 + 8 * i]) : 0.f;
      x.g = a.g[at * a.H + h];
      x.beta = a.beta[at * a.H + h];
      return x;
    };
    Token x = request(0);
    for (int t = 0; t < a.T; ++t) {
      const int64_t at = static_cast<int64_t>(b) * a.T + t;
      const Token y = request(t + 1 < a.T ? t + 1 : t);
      const float dec = expf(x.g);
      float kq = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int r = 0; r < 4; ++r) kq += x.k[j][r] * x.q[j][r];
      }
      kq = sum8(kq);
#pragma unroll
      for (int i = 0; i < RG; ++i) {
        float sk = 0.f, sq = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          S[i][j] *= dec;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            sk += S[i][j][r] * x.k[j][r];
            sq += S[i][j][r] * x.q[j][r];
          }
        }
        sk = sum8(sk);
        sq = sum8(sq);
        const float u = x.beta * (x.v[i] - sk);
#pragma unroll
        for (int j = 0; j < NV; ++j) S[i][j] += u * x.k[j];
        const int p = row0 + 8 * i;
        if (l8 == 0 && p < a.P) static_cast<T*>(a.o)[(at * a.H + h) * a.P + p] = ssd::Elem<T>::from_f(a.scale * (sq + u * kq));
      }
      x = y;
    }
    if (next >= a.B) break;
    b = next;
    next = a.B;
    for (int i0 = (b + 1) & ~63; i0 < a.B && next == a.B; i0 += 64) {
      const uint64_t m = __ballot(i0 + l > b && i0 + l < a.B && a.index[i0 + l < a.B ? i0 + l : 0] == slot);
      if (m) next = i0 + __builtin_ctzll(m);
    }
  }
#pragma unroll
  for (int i = 0; i < RG; ++i) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int p = row0 + 8 * i, n = 4 * (l8 + 8 * j);
      if (p < a.P && n < a.N) *reinterpret_cast<f32x4_t*>(sp + static_cast<int64_t>(p) * a.N + n) = S[i][j];
    }
  }
}

namespace {
template <typename T, int NV, int RG> int go(StepArgs a, hipStream_t s) {
  a.nblk = (a.P + 8 * RG * STEP_WAVES - 1) / (8 * RG * STEP_WAVES);
  hipLaunchKernelGGL((k_delta_step<T, NV, RG>), dim3(a.H * a.nblk, a.B), dim3(64 * STEP_WAVES), 0, s, a);
  return hipGetLastError() == hipSuccess ? SSD_OK : SSD_ERR_HIP;
}
// Two rows a lane where that still gives every CU eight waves, else one.  64 sequences of 128 heads of 64 x 128: 95 us
// at one row, 80.5 at two (480 MB: 6.0 TB/s), 124 at four; one sequence: 5.3 us at one row, 5.9 at two.
template <typename T> int by_size(const StepArgs& a, hipStream_t s) {
  if (static_cast<int64_t>(a.B) * a.H * ((a.P + 15) / 16) >= 8 * 256)
    return a.N <= 32 ? go<T, 1, 2>(a, s) : a.N <= 64 ? go<T, 2, 2>(a, s) : go<T, 4, 2>(a, s);
  return a.N <= 32 ? go<T, 1, 1>(a, s) : a.N <= 64 ? go<T, 2, 1>(a, s) : go<T, 4, 1>(a, s);
}
}  // namespace

int launch_step(const StepArgs& a, int io, hipStream_t s) {
  return io == SSD_IO_BF16 ? by_size<bf16_t>(a, s) : by_size<float>(a, s);
}

}  // namespace delta

int delta_check(const delta_shape* s);   // delta_api.hip
void delta_strides(const delta_shape& s, int64_t (&st)[6]);

extern "C" int delta_step(const delta_shape* shape, const void* q, const void* k, const void* v, const float* g,
                          const float* beta, float* states, int64_t nslots, const int32_t* state_indices, void* o,
                          void* stream) {
  if (!shape) return SSD_ERR_INVALID_ARG;
  delta_shape sh = *shape;
  sh.nseqs = sh.batch;
  const int rc = delta_check(&sh);
  if (rc != SSD_OK) return rc;
  if (sh.seqlen > 64 || sh.batch > 65535) return SSD_ERR_UNSUPPORTED_SHAPE;
  if (!q || !k || !v || !g || !beta || !states || !o || nslots < 1) return SSD_ERR_INVALID_ARG;
  if (!state_indices && nslots < sh.batch) return SSD_ERR_INVALID_ARG;
  if (o == q || o == k || o == v || o == states) return SSD_ERR_INVALID_ARG;   // other blocks may still read them
  for (const void* p : {q, k, v, static_cast<const void*>(states), static_cast<const void*>(o)})
    if (reinterpret_cast<uintptr_t>(p) & 15u) return SSD_ERR_MISALIGNED;
  int64_t st[6];
  delta_strides(sh, st);
  delta::StepArgs a{q, k, v, g, beta, states, state_indices, o, nslots, st[0], st[1], st[2], st[3], st[4], st[5],
                    static_cast<int>(sh.batch), static_cast<int>(sh.seqlen), static_cast<int>(sh.nheads),
                    static_cast<int>(sh.headdim), static_cast<int>(sh.ngroups), static_cast<int>(sh.dstate),
                    static_cast<int>(sh.nheads / sh.ngroups), 0, sh.scale};
  return delta::launch_step(a, sh.io_dtype, static_cast<hipStream_t>(stream));
}
