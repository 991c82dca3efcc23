// Norm of every query and key head with the position rotation in the same
// pass, forward and backward (the operation and its gradients:
// include/qk_norm.h).
//
//     dz = the rotation of dy by -t,   dw = sum dz x r,
//     dx = r w dz - x r^3 (sum w dz x) / m   (m = N for the mean, 1 for the sum)
//
// Bound by HBM: x (and dy) read once, y (or dx) written once.  A row of N
// values lies in LPR lanes of 16 bytes each, so a wave's access is whole rows
// side by side and the row sum is log2 LPR lane exchanges.  The angles of a
// position serve all its heads: a block takes TT positions, fills a table of
// their cosines and sines in LDS (one double product and reduction per angle)
// and then walks their rows.  16384 positions of 16 heads of 128 in bf16, fully
// turned: forward 37 us (3.6 TB/s), backward 46 us (4.4 TB/s) and 4 us for the
// slots' sum.
#include <hip/hip_runtime.h>

#include "qk_norm.h"
#include "ssd_device.h"
#include "ssd_tiles.h"

namespace qkn {

using ssd::bf16_t;

constexpr int THR = 256;
constexpr int MAXN = 256;
constexpr int UNROLL = 2;         // rows of a lane in flight
constexpr int MAX_SLOTS = 1024;   // blocks of the backward, and its workspace slots

struct Args {
  const void *q, *k, *dyq, *dyk;
  const float *wq, *wk, *inv_freq;
  const int32_t* pos;
  void *oq, *ok;      // y, or dx
  float* slots;       // (blocks, 2, N) partial weight gradients
  int64_t q_sb, q_sl, k_sb, k_sl;
  int tokens, L, Gq, Gk, N, half, interleaved, l2, tt;
  int flat;           // batch rows follow each other at the row stride
  uint32_t magic;     // row / (Gq + Gk) = mulhi(row, magic) for the rows of tt > 1 positions of several heads
  float eps;
};

// the partner of a rotated value: in the same lane (interleaved), in the lane `half` values away (half a
// multiple of a lane's values), or anywhere
enum { PAIR_LANE = 0, PAIR_SHUFFLE = 1, PAIR_ANY = 2 };

template <typename T> struct Vec {
  static constexpr int V = ssd::Vec16<T>::N;
  static __device__ __forceinline__ void load(const T* p, float (&f)[V]) {
    const uint4 u = ssd::ld_global16(p);
#pragma unroll
    for (int e = 0; e < V; ++e) f[e] = ssd::vget<T>(u, e);
  }
  static __device__ __forceinline__ void store(T* p, const float (&f)[V]) {
#pragma unroll
    for (int e = 0; e < V; e += 4) ssd::store4f<T>(p + e, ssd::f32x4_t{f[e], f[e + 1], f[e + 2], f[e + 3]});
  }
};

template <int LPR> __device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int d = 1; d < LPR; d <<= 1) v += __shfl_xor(v, d);
  return v;
}

// (first, rotated) of the values f (positions n .. of a row) by the angles of `cs`, the sine times `sign`;
// other(i): the value at position i of the same row
template <int V, int PAIR, int LPR, typename Other>
__device__ __forceinline__ void rotate(float (&f)[V], int n, int half, const float2* cs, float sign, Other other) {
  if constexpr (PAIR == PAIR_LANE) {
#pragma unroll
    for (int e = 0; e < V; e += 2) {
      const int j = (n + e) >> 1;
      if (j < half) {
        const float2 t = cs[j];
        const float a = f[e], b = f[e + 1], s = sign * t.y;
        f[e] = a * t.x - b * s;
        f[e + 1] = b * t.x + a * s;
      }
    }
  } else if constexpr (PAIR == PAIR_SHUFFLE) {
    const bool first = n < half, in = n < 2 * half;
    const int lane = static_cast<int>(threadIdx.x) & 63;
    const int from = in ? (first ? lane + half / V : lane - half / V) : lane;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float o = __shfl(f[e], from);
      if (in) {
        const float2 t = cs[(first ? n : n - half) + e];
        f[e] = f[e] * t.x + (first ? -o : o) * (sign * t.y);
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const int i = n + e;
      if (i < 2 * half) {
        const bool first = i < half;
        const float2 t = cs[first ? i : i - half];
        const float o = other(first ? i + half : i - half);
        f[e] = f[e] * t.x + (first ? -o : o) * (sign * t.y);
      }
    }
  }
}

// BWD: the gradients; else the forward.  Rows of a position: its q heads, then its k heads.
template <typename T, int LPR, int PAIR, bool BWD> __global__ __launch_bounds__(THR) void k_qk_norm(Args a) {
  constexpr int V = Vec<T>::V, ROWS = THR / LPR, UN = PAIR == PAIR_ANY ? 1 : UNROLL;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  float2* table = reinterpret_cast<float2*>(smem);   // [tt][half]: cosines and sines
  const int tid = static_cast<int>(threadIdx.x), rl = tid / LPR, n = (tid % LPR) * V;
  const int heads = a.Gq + a.Gk;
  const bool live = n < a.N;
  float wq[V], wk[V], gq[V], gk[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    wq[e] = a.wq && live ? a.wq[n + e] : 1.f;
    wk[e] = a.wk && live ? a.wk[n + e] : 1.f;
    gq[e] = gk[e] = 0.f;
  }
  const float inv_m = a.l2 ? 1.f : 1.f / static_cast<float>(a.N);
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tt; t0 < a.tokens; t0 += static_cast<int64_t>(gridDim.x) * a.tt) {
    const int nt = static_cast<int>(a.tokens - t0 < a.tt ? a.tokens - t0 : a.tt);
    const int nrows = nt * heads;
    // Every lane runs every turn: lanes past the last row take part in the exchanges with zeros.  The rows of UN turns
    // are requested before the angles are formed.
    for (int r0 = 0; r0 < nrows; r0 += UN * ROWS) {
      struct {
        const T *x, *dy;
        T* out;
        int tl;
        bool ok, isq;
        uint4 xr, yr;
      } rows[UN];
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        const int row = r0 + u * ROWS + rl;
        auto& w = rows[u];
        w.ok = live && row < nrows;
        w.tl = row >= nrows || a.tt == 1 ? 0 : heads == 1 ? row : static_cast<int>(__umulhi(static_cast<uint32_t>(row), a.magic));
        const int hd = row < nrows ? row - w.tl * heads : 0;
        w.isq = hd < a.Gq;
        const int hl = w.isq ? hd : hd - a.Gq, nh = w.isq ? a.Gq : a.Gk;
        const int t = static_cast<int>(t0) + w.tl;
        const int64_t sl = w.isq ? a.q_sl : a.k_sl;
        int64_t at = t * sl;
        if (!a.flat) {
          const int bt = t / a.L;
          at = bt * (w.isq ? a.q_sb : a.k_sb) + (t - bt * a.L) * sl;
        }
        const int64_t packed = (static_cast<int64_t>(t) * nh + hl) * static_cast<int64_t>(a.N);
        w.x = static_cast<const T*>(w.isq ? a.q : a.k) + at + static_cast<int64_t>(hl) * a.N;
        w.out = static_cast<T*>(w.isq ? a.oq : a.ok) + packed + n;
        w.dy = BWD ? static_cast<const T*>(w.isq ? a.dyq : a.dyk) + packed : nullptr;
        w.xr = w.yr = ssd::zero_u4();
        if (w.ok) {
          w.xr = ssd::ld_global16(w.x + n);
          if (BWD) w.yr = ssd::ld_global16(w.dy + n);
        }
      }
      if (r0 == 0 && a.half) {
        __syncthreads();
        for (int i = tid; i < nt * a.half; i += THR) {
          const int t = static_cast<int>(t0) + i / a.half;
          const double at = a.pos ? static_cast<double>(a.pos[t]) : static_cast<double>(t % a.L);
          const double turns = at * static_cast<double>(a.inv_freq[i % a.half]) * 0.15915494309189533577;   // 1 / (2 pi)
          const float part = static_cast<float>(2.0 * (turns - rint(turns)));
          table[i] = float2{cospif(part), sinpif(part)};
        }
        __syncthreads();
      }
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        const auto& row = rows[u];
        const bool ok = row.ok, isq = row.isq;
        const float2* cs = table + row.tl * a.half;
        const float* w = isq ? a.wq : a.wk;
        float f[V], y[V];
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          f[e] = ssd::vget<T>(row.xr, e);
          y[e] = ssd::vget<T>(row.yr, e);
          ss += f[e] * f[e];
        }
        const float r = 1.f / sqrtf(row_sum<LPR>(ss) * inv_m + a.eps);
        if constexpr (!BWD) {
#pragma unroll
          for (int e = 0; e < V; ++e) y[e] = f[e] * r * (isq ? wq[e] : wk[e]);
          rotate<V, PAIR, LPR>(y, n, a.half, cs, 1.f, [&](int i) {
            return ok ? ssd::Elem<T>::to_f(row.x[i]) * r * (w ? w[i] : 1.f) : 0.f; });
          if (ok) Vec<T>::store(row.out, y);
        } else {
          rotate<V, PAIR, LPR>(y, n, a.half, cs, -1.f, [&](int i) { return ok ? ssd::Elem<T>::to_f(row.dy[i]) : 0.f; });
          float dot = 0.f;
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float gw = y[e] * f[e] * r;
            if (ok) {
              if (isq) gq[e] += gw; else gk[e] += gw;
            }
            y[e] *= isq ? wq[e] : wk[e];
            dot += y[e] * f[e];
          }
          const float m = row_sum<LPR>(dot) * inv_m * r * r;
#pragma unroll
          for (int e = 0; e < V; ++e) y[e] = r * (y[e] - f[e] * m);
          if (ok) Vec<T>::store(row.out, y);
        }
      }
    }
  }
  if constexpr (BWD) {
    // the block's sums, over its row places in order
    float* red = reinterpret_cast<float*>(smem);   // [ROWS][2][LPR * V]
    __syncthreads();
#pragma unroll
    for (int e = 0; e < V; ++e) {
      red[(rl * 2 + 0) * LPR * V + n + e] = gq[e];
      red[(rl * 2 + 1) * LPR * V + n + e] = gk[e];
    }
    __syncthreads();
    for (int i = tid; i < 2 * a.N; i += THR) {
      const int which = i / a.N, at = i - which * a.N;
      float s = 0.f;
      for (int rr = 0; rr < ROWS; ++rr) s += red[(rr * 2 + which) * LPR * V + at];
      a.slots[static_cast<int64_t>(blockIdx.x) * 2 * a.N + i] = s;
    }
  }
}

// The slots' sum, a column per 64 threads: each adds every 64th slot in order, then the 64 in order.
constexpr int RED_COLS = 16, RED_ROWS = 64;
__global__ __launch_bounds__(RED_COLS * RED_ROWS) void k_qk_norm_reduce(const float* slots, int nslots, int N, float* dwq, float* dwk) {
  __shared__ double part[RED_ROWS][RED_COLS + 1];
  const int lc = static_cast<int>(threadIdx.x) % RED_COLS, lr = static_cast<int>(threadIdx.x) / RED_COLS;
  const int col = static_cast<int>(blockIdx.x) * RED_COLS + lc;
  double s = 0.0;
  if (col < 2 * N) {
#pragma unroll 8
    for (int i = lr; i < nslots; i += RED_ROWS) s += static_cast<double>(slots[static_cast<int64_t>(i) * 2 * N + col]);
  }
  part[lr][lc] = s;
  __syncthreads();
  if (lr == 0 && col < 2 * N) {
#pragma unroll 16
    for (int i = 1; i < RED_ROWS; ++i) s += part[i][lc];
    if (col < N) {
      if (dwq) dwq[col] = static_cast<float>(s);
    } else if (dwk) {
      dwk[col - N] = static_cast<float>(s);
    }
  }
}

int check(const qk_norm_shape* s) {
  if (!s || s->reserved != 0) return SSD_ERR_INVALID_ARG;
  if (s->io_dtype != SSD_IO_BF16 && s->io_dtype != SSD_IO_F32) return SSD_ERR_UNSUPPORTED_SHAPE;
  const int64_t vec = s->io_dtype == SSD_IO_BF16 ? 8 : 4;
  if (s->batch < 1 || s->seqlen < 1 || s->qheads < 1 || s->kheads < 0 || s->dstate < 1) return SSD_ERR_UNSUPPORTED_SHAPE;
  if (s->batch > INT32_MAX || s->seqlen > INT32_MAX || s->batch * s->seqlen > INT32_MAX) return SSD_ERR_UNSUPPORTED_SHAPE;
  if (s->qheads > 65535 || s->kheads > 65535 || s->dstate > MAXN || s->dstate % vec) return SSD_ERR_UNSUPPORTED_SHAPE;
  for (const int64_t st : {s->q_batch_stride, s->q_row_stride, s->k_batch_stride, s->k_row_stride})
    if (st < 0 || st % vec) return SSD_ERR_UNSUPPORTED_SHAPE;
  if (s->rot_dim < 0 || s->rot_dim % 2 || s->rot_dim > s->dstate) return SSD_ERR_UNSUPPORTED_SHAPE;
  if (s->interleaved != 0 && s->interleaved != 1) return SSD_ERR_UNSUPPORTED_SHAPE;
  if (s->norm != QK_NORM_RMS && s->norm != QK_NORM_L2) return SSD_ERR_UNSUPPORTED_SHAPE;
  if (!(s->eps >= 0.f)) return SSD_ERR_INVALID_ARG;
  return SSD_OK;
}

bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

int lanes_per_row(const qk_norm_shape& s) {
  const int need = static_cast<int>(s.dstate) / (s.io_dtype == SSD_IO_BF16 ? 8 : 4);
  int l = 1;
  while (l < need) l <<= 1;
  return l;
}

// positions per block: enough rows to fill a block's row places, more where there are positions for every
// CU to have several blocks (the table is then shared by more rows in flight)
int positions_per_block(const qk_norm_shape& s) {
  const int64_t tokens = s.batch * s.seqlen, heads = s.qheads + s.kheads, places = THR / lanes_per_row(s);
  int64_t tt = (places + heads - 1) / heads;
  if (tt > tokens) tt = tokens;
  while (heads <= THR && tt < 8 && tokens / (2 * tt) >= 1024) tt *= 2;
  return static_cast<int>(tt < 1 ? 1 : tt);
}

int64_t blocks(const qk_norm_shape& s, bool bwd) {
  const int64_t tt = positions_per_block(s), n = (s.batch * s.seqlen + tt - 1) / tt, most = bwd ? MAX_SLOTS : 65536;
  return n < most ? n : most;
}

template <typename T, int LPR, int PAIR, bool BWD> int go(const Args& a, int64_t grid, hipStream_t st) {
  size_t lds = sizeof(float2) * a.half * static_cast<size_t>(a.tt);
  constexpr size_t red = sizeof(float) * (THR / LPR) * 2 * LPR * Vec<T>::V;   // at most 16 KB
  if (BWD && lds < red) lds = red;
  if (lds > 65536) return SSD_ERR_UNSUPPORTED_SHAPE;   // tt <= 256 places, half <= 128 where a place is 64 lanes
  hipLaunchKernelGGL((k_qk_norm<T, LPR, PAIR, BWD>), dim3(static_cast<unsigned>(grid)), dim3(THR), lds, st, a);
  return hipGetLastError() == hipSuccess ? SSD_OK : SSD_ERR_HIP;
}

template <typename T, int LPR, bool BWD> int by_pair(const qk_norm_shape& s, const Args& a, int64_t grid, hipStream_t st) {
  if (s.interleaved || a.half == 0) return go<T, LPR, PAIR_LANE, BWD>(a, grid, st);
  if (a.half % Vec<T>::V == 0) return go<T, LPR, PAIR_SHUFFLE, BWD>(a, grid, st);
  return go<T, LPR, PAIR_ANY, BWD>(a, grid, st);
}

template <typename T, bool BWD> int by_lanes(const qk_norm_shape& s, const Args& a, int64_t grid, hipStream_t st) {
  switch (lanes_per_row(s)) {
    case 1: return by_pair<T, 1, BWD>(s, a, grid, st);
    case 2: return by_pair<T, 2, BWD>(s, a, grid, st);
    case 4: return by_pair<T, 4, BWD>(s, a, grid, st);
    case 8: return by_pair<T, 8, BWD>(s, a, grid, st);
    case 16: return by_pair<T, 16, BWD>(s, a, grid, st);
    case 32: return by_pair<T, 32, BWD>(s, a, grid, st);
    default: return by_pair<T, 64, BWD>(s, a, grid, st);
  }
}

Args args(const qk_norm_shape& s, const void* q, const void* k, const float* wq, const float* wk, const int32_t* pos, const float* inv_freq) {
  Args a{};
  a.q = q; a.k = k; a.wq = wq; a.wk = wk; a.pos = pos; a.inv_freq = inv_freq;
  const bool qc = s.q_batch_stride == 0 && s.q_row_stride == 0, kc = s.k_batch_stride == 0 && s.k_row_stride == 0;
  a.q_sl = qc ? s.qheads * s.dstate : s.q_row_stride;
  a.q_sb = qc ? s.seqlen * a.q_sl : s.q_batch_stride;
  a.k_sl = kc ? s.kheads * s.dstate : s.k_row_stride;
  a.k_sb = kc ? s.seqlen * a.k_sl : s.k_batch_stride;
  a.tokens = static_cast<int>(s.batch * s.seqlen);
  a.flat = a.q_sb == s.seqlen * a.q_sl && (s.kheads == 0 || a.k_sb == s.seqlen * a.k_sl);
  a.L = static_cast<int>(s.seqlen);
  a.Gq = static_cast<int>(s.qheads);
  a.Gk = static_cast<int>(s.kheads);
  a.N = static_cast<int>(s.dstate);
  a.half = s.rot_dim / 2;
  a.interleaved = s.interleaved;
  a.l2 = s.norm == QK_NORM_L2;
  a.tt = positions_per_block(s);   // tt > 1: fewer than 8 * 256 rows, for which the rounded up reciprocal of 2 .. 256 heads is exact (that of 1 does
  // not fit 32 bits)
  a.magic = a.Gq + a.Gk > 1 ? static_cast<uint32_t>((uint64_t{1} << 32) / static_cast<uint64_t>(a.Gq + a.Gk) + 1) : 0;
  a.eps = s.eps;
  return a;
}

}  // namespace qkn

extern "C" {

int qk_norm_fwd(const qk_norm_shape* shape, const void* q, const void* k, const float* q_weight,
                const float* k_weight, const int32_t* positions, const float* inv_freq, void* q_out, void* k_out,
                void* stream) {
  const int rc = qkn::check(shape);
  if (rc != SSD_OK) return rc;
  if (!q || !q_out || (shape->kheads && (!k || !k_out)) || (shape->rot_dim && !inv_freq)) return SSD_ERR_INVALID_ARG;
  for (const void* p : {q, static_cast<const void*>(q_out), k, static_cast<const void*>(k_out)})
    if (qkn::misaligned(p)) return SSD_ERR_MISALIGNED;
  qkn::Args a = qkn::args(*shape, q, k, q_weight, k_weight, positions, inv_freq);
  a.oq = q_out;
  a.ok = k_out;
  const int64_t grid = qkn::blocks(*shape, false);
  hipStream_t st = static_cast<hipStream_t>(stream);
  return shape->io_dtype == SSD_IO_BF16 ? qkn::by_lanes<ssd::bf16_t, false>(*shape, a, grid, st)
                                        : qkn::by_lanes<float, false>(*shape, a, grid, st);
}

int qk_norm_bwd_workspace_size(const qk_norm_shape* shape, size_t* bytes) {
  const int rc = qkn::check(shape);
  if (rc != SSD_OK) return rc;
  if (!bytes) return SSD_ERR_INVALID_ARG;
  *bytes = static_cast<size_t>(qkn::blocks(*shape, true)) * 2 * static_cast<size_t>(shape->dstate) * sizeof(float);
  return SSD_OK;
}

int qk_norm_bwd(const qk_norm_shape* shape, const void* q, const void* k, const float* q_weight,
                const float* k_weight, const int32_t* positions, const float* inv_freq, const void* dq_out,
                const void* dk_out, void* dq, void* dk, float* dq_weight, float* dk_weight, void* workspace,
                size_t workspace_bytes, void* stream) {
  size_t need = 0;
  const int rc = qk_norm_bwd_workspace_size(shape, &need);
  if (rc != SSD_OK) return rc;
  if (!q || !dq_out || !dq || (shape->kheads && (!k || !dk_out || !dk)) || (shape->rot_dim && !inv_freq) || !workspace)
    return SSD_ERR_INVALID_ARG;
  if (workspace_bytes < need) return SSD_ERR_WORKSPACE_TOO_SMALL;
  for (const void* p : {q, k, dq_out, dk_out, static_cast<const void*>(dq), static_cast<const void*>(dk), static_cast<const void*>(workspace)})
    if (qkn::misaligned(p)) return SSD_ERR_MISALIGNED;
  if (dq == q || (shape->kheads && dk == k)) return SSD_ERR_INVALID_ARG;
  qkn::Args a = qkn::args(*shape, q, k, q_weight, k_weight, positions, inv_freq);
  a.dyq = dq_out; a.dyk = dk_out; a.oq = dq; a.ok = dk;
  a.slots = static_cast<float*>(workspace);
  const int64_t grid = qkn::blocks(*shape, true);
  hipStream_t st = static_cast<hipStream_t>(stream);
  const int r = shape->io_dtype == SSD_IO_BF16 ? qkn::by_lanes<ssd::bf16_t, true>(*shape, a, grid, st)
                                               : qkn::by_lanes<float, true>(*shape, a, grid, st);
  if (r != SSD_OK || (!dq_weight && !dk_weight)) return r;
  hipLaunchKernelGGL(qkn::k_qk_norm_reduce, dim3(static_cast<unsigned>((2 * shape->dstate + qkn::RED_COLS - 1) / qkn::RED_COLS)),
                     dim3(qkn::RED_COLS * qkn::RED_ROWS), 0, st,
                     a.slots, static_cast<int>(grid), a.N, dq_weight, dk_weight);
  return hipGetLastError() == hipSuccess ? SSD_OK : SSD_ERR_HIP;
}

}  // extern "C"
