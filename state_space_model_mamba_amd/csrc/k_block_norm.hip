// Norms before and after a block, forward and backward (the operations:
// include/block_norm.h).  With u the normed values of a row or group of W,
// v = u - mean (u itself without the mean), r = 1 / sqrt(mean v^2 + eps) and d
// the gradient by norm(u):
//
//     du = r (d - v r^2 (sum d v) / W  [- (sum d) / W])
//
// Bound by HBM: every operand read once, every result written once.  A lane
// holds VPL pieces of 16 bytes of x and the same values of the other operands,
// a row lies in LPR lanes of a wave (narrow rows) or in all lanes of a block
// (wide rows).  A block keeps its channels from row to row, so weights stay in
// registers and the gradients over rows are sums in registers; the next row's
// pieces are requested before the present row's sums are exchanged.
//
// 16384 rows of 8192 bf16 in 8 gated groups: forward 144 us (5.6 TB/s), backward
// 268 (5.0 TB/s), each by itself; in turn in a training pass, by the kernel
// trace, 144 to 160 and 240 to 290 us (least and median).  16384 rows of 4096
// bf16 with a float32 residual and a scale a channel: 147 to 151 and 200 to 206
// us there.  1999 rows of 64 float32 heads of 64, gated, with a residual: 25 and
// 29 us.  The slots' sum takes 4 to 5 us.  One row of 4096: 3 us.
//
// Rows past 8192 (1024 threads, 128 registers) keep part of their values in
// scratch memory: nearly every backward, and the forwards but for add_norm of
// bf16 and, without bias and scale, gated_norm of bf16 and add_norm of float32.
// 4096 rows of 16384, gated, without them: bf16 113 and 224 us (3.6 and 3.0
// TB/s), float32 252 and 490 (3.2 and 2.7 TB/s).
#include <hip/hip_runtime.h>

#include "block_norm.h"
#include "ssd_device.h"
#include "ssd_tiles.h"

namespace bnorm {

using ssd::bf16_t;

constexpr int THR = 256;          // threads of a block of narrow rows
constexpr int MAX_WIDTH = 16384;
constexpr int SUMS = 3;           // gradients over rows: weight, bias, scale

struct Args {
  const void *x, *z, *res, *dy, *dr;   // dr: the gradient of residual_out, or of out
  const float *w, *b, *s;
  void *y, *ro, *dx, *dz, *dres;
  float* slots;                        // (blocks, SUMS, D)
  int64_t x_sb, x_sl, z_sb, z_sl;
  int tokens, L, D, W, groups;
  int lpr, gpb, tpb;                   // lanes of a narrow row; groups and tokens a block takes side by side
  int flat;                            // batch rows follow each other at the row stride
  int layer, sigmoid, norm_first;
  int sums;                            // bit i: gradient i over rows is wanted
  float eps, alpha, inv_w;
};

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

// V values of type S, as they lie in memory.  PASS: not to be kept in the caches (the nontemporal hint).
template <typename S, int V> struct Raw {
  static constexpr int N = V * static_cast<int>(sizeof(S)) / 16;
  uint4 u[N];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < N; ++i) u[i] = ssd::zero_u4();
  }
  template <bool PASS = false> __device__ __forceinline__ void load(const S* p) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const u32x4_t* q = reinterpret_cast<const u32x4_t*>(p) + i;
      const u32x4_t t = PASS ? __builtin_nontemporal_load(q) : *q;
      u[i] = uint4{t[0], t[1], t[2], t[3]};
    }
  }
  __device__ __forceinline__ void renew() {   // the same values, of which the compiler knows nothing
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+v"(u[i].x), "+v"(u[i].y), "+v"(u[i].z), "+v"(u[i].w));
  }
  __device__ __forceinline__ float get(int e) const {
    constexpr int PER = 16 / static_cast<int>(sizeof(S));
    return ssd::vget<S>(u[e / PER], e % PER);
  }
};

template <typename S, int V, bool PASS = false> __device__ __forceinline__ void store(S* p, const float (&f)[V]) {
  constexpr int PER = 16 / static_cast<int>(sizeof(S));
#pragma unroll
  for (int e = 0; e < V; e += PER) {
    u32x4_t w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(S) == 2) w[i] = ssd::pack_bf16x2(f[e + 2 * i], f[e + 2 * i + 1]);
      else w[i] = __float_as_uint(f[e + i]);
    }
    u32x4_t* q = reinterpret_cast<u32x4_t*>(p + e);
    if constexpr (PASS) __builtin_nontemporal_store(w, q);
    else *q = w;
  }
}

// sigmoid(z) and 1 - sigmoid(z), both to their last bits; with bf16 io by the hardware's exponential and reciprocal (1 ulp)
template <typename T> __device__ __forceinline__ float2 sigmoids(float z) {
  const float e = ssd::Elem<T>::exp(-fabsf(z)), big = sizeof(T) == 2 ? __builtin_amdgcn_rcpf(1.f + e) : 1.f / (1.f + e), small = e * big;
  return z < 0.f ? float2{small, big} : float2{big, small};
}

// Sums over the lanes of a row, the same bits in every lane.  Wide rows go
// through LDS, one set of places after the other, so that one barrier a sum is
// enough: a set is written again only two sums later.
template <int K, bool WIDE> struct RowSum {
  float (*places)[16][K];
  int lpr, at;
  __device__ __forceinline__ void operator()(float (&v)[K]) {
    if constexpr (!WIDE) {
      for (int d = 1; d < lpr; d <<= 1) {
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += __shfl_xor(v[k], d);
      }
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k) {
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) v[k] += __shfl_xor(v[k], d);
      }
      const int lane = static_cast<int>(threadIdx.x) & 63, wave = static_cast<int>(threadIdx.x) >> 6, waves = static_cast<int>(blockDim.x) >> 6;
      if (lane == 0) {
#pragma unroll
        for (int k = 0; k < K; ++k) places[at][wave][k] = v[k];
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] = places[at][0][k];
      for (int i = 1; i < waves; ++i) {
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += places[at][i][k];
      }
      at ^= 1;
    }
  }
};

// How a row lies in the lanes: in some lanes of a wave, or in all of a block of up to 512 threads (which leaves a lane 256
// registers: the gradients of 16 values fit) with 1, 2 or 4 pieces a lane, or of up to 1024.
enum { NARROW = 0, WIDE1 = 1, WIDE2 = 2, WIDE4 = 3, WIDEST = 4 };
constexpr int max_threads(int lay) { return lay == NARROW ? THR : lay == WIDEST ? 1024 : 512; }
template <typename T> constexpr int pieces_a_lane(int lay) {
  return lay <= WIDE1 ? 1 : lay == WIDE2 || (lay == WIDEST && sizeof(T) == 2) ? 2 : 4;
}

enum { FORWARD = 0, BACKWARD = 1, BACKWARD_PASS = 2 };   // the last: its operands pass the caches by

// PRE: add_norm, else gated_norm.  EXTRA: with a bias, a scale or their gradients.  T: io dtype, R: residual dtype.
template <typename T, typename R, int LAY, bool PRE, int DIR, bool EXTRA>
__global__ __launch_bounds__(max_threads(LAY)) void k_block_norm(Args a) {
  constexpr int V = ssd::Vec16<T>::N, VPL = pieces_a_lane<T>(LAY);
  constexpr bool WIDE = LAY != NARROW, BWD = DIR != FORWARD, PASS = DIR == BACKWARD_PASS;
  // Sixteen values a lane with all their sums leave no registers for the next row's, nor for the gates' values over the
  // exchange of the sums, which are then formed again (4096 rows of 8192 bf16, gated, with a bias and a scale: 119 us, 265
  // with spilled registers; without bias and scale 88 us, 104 formed again).
  constexpr bool AHEAD = !(BWD && (LAY == WIDEST || (EXTRA && VPL * V == 16 && (!PRE || sizeof(T) == 4))));
  constexpr bool AGAIN = !PRE && !AHEAD;
  __shared__ float places1[2][16][1], places3[2][16][3];
  extern __shared__ __attribute__((aligned(16))) char smem[];   // narrow rows, backward: [THR][V] sums
  const int tid = static_cast<int>(threadIdx.x);
  // where the lane stands: its token among the block's, its group, and its first values in the group
  int tl = 0, group = static_cast<int>(blockIdx.x), n0 = tid * V;
  if constexpr (!WIDE) {
    const int place = tid / a.lpr;
    tl = place / a.gpb;
    group = group * a.gpb + place % a.gpb;
    n0 = tid % a.lpr * V;
  }
  const int step = (WIDE ? static_cast<int>(blockDim.x) : a.lpr) * V;   // between a lane's pieces
  bool live[VPL];
  int col[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    live[i] = n0 + i * step < a.W && group < a.groups;
    col[i] = group * a.W + n0 + i * step;
  }
  struct Row {
    Raw<T, V> x[VPL], z[VPL], dy[VPL];
    Raw<R, V> res[VPL], dr[VPL];
  };
  auto request = [&](Row& q, int64_t t) {
    const bool in = t < a.tokens;
    int64_t xo = t * a.x_sl, zo = t * a.z_sl;
    if (!a.flat && in) {
      const int bt = static_cast<int>(t) / a.L, tt = static_cast<int>(t) - bt * a.L;
      xo = bt * a.x_sb + tt * a.x_sl;
      zo = bt * a.z_sb + tt * a.z_sl;
    }
    const int64_t at = t * a.D;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      q.x[i].zero();
      if (!PRE) q.z[i].zero();
      if (PRE || !BWD) q.res[i].zero();
      if (BWD) q.dr[i].zero();
      if (BWD && PRE) q.dy[i].zero();
      if (!in || !live[i]) continue;
      q.x[i].template load<PASS>(static_cast<const T*>(a.x) + xo + col[i]);
      if (!PRE && a.z) q.z[i].template load<PASS>(static_cast<const T*>(a.z) + zo + col[i]);
      if ((PRE || !BWD) && a.res) q.res[i].template load<PASS>(static_cast<const R*>(a.res) + at + col[i]);
      if (BWD && a.dr) q.dr[i].template load<PASS>(static_cast<const R*>(a.dr) + at + col[i]);
      if (BWD && PRE && a.dy) q.dy[i].template load<PASS>(static_cast<const T*>(a.dy) + at + col[i]);
    }
  };
  RowSum<1, WIDE> sum1{places1, a.lpr, 0};
  RowSum<3, WIDE> sum3{places3, a.lpr, 0};
  const int64_t stride = static_cast<int64_t>(gridDim.y) * a.tpb;
  int64_t t = static_cast<int64_t>(blockIdx.y) * a.tpb;
  Row next;
  if (AHEAD) request(next, t + tl);
  float w[VPL][V], s[VPL][V], b[VPL][V], gw[VPL][V], gb[VPL][V], gs[VPL][V];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    Raw<float, V> rw, rs, rb;
    rw.zero();
    rs.zero();
    rb.zero();
    if (a.w && live[i]) rw.load(a.w + col[i]);
    if (EXTRA && a.s && live[i]) rs.load(a.s + col[i]);
    if (EXTRA && a.b && live[i]) rb.load(a.b + col[i]);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      w[i][e] = a.w ? rw.get(e) : 1.f;
      s[i][e] = EXTRA && a.s ? a.alpha * rs.get(e) : a.alpha;
      b[i][e] = rb.get(e);
      gw[i][e] = gb[i][e] = gs[i][e] = 0.f;
    }
  }
  for (; t < a.tokens; t += stride) {
    Row q;
    if (AHEAD) {
      q = next;
      if (t + stride < a.tokens) request(next, t + stride + tl);
    } else {
      request(q, t + tl);
    }
    const bool in = t + tl < a.tokens;
    const int64_t at = (t + tl) * a.D;
    float v[VPL][V];   // the normed values, then without their mean
    constexpr int KI = AGAIN ? 1 : VPL, KE = AGAIN ? 1 : V;
    float acts[KI][KE], slopes[KI][KE];
    auto gate_of = [&](int i, int e, float& act, float& slope) {   // the gate's value, and its slope
      act = 1.f;
      slope = 0.f;
      if (!PRE && a.z) {
        const float z = q.z[i].get(e);
        const float2 sg = sigmoids<T>(z);
        act = a.sigmoid ? sg.x : z * sg.x;
        if (BWD) slope = a.sigmoid ? sg.x * sg.y : sg.x * fmaf(z, sg.y, 1.f);
      }
    };
    auto gate_at = [&](int i, int e, float& act, float& slope) {   // the same, kept or formed again
      if constexpr (AGAIN) {
        gate_of(i, e, act, slope);
      } else {
        act = acts[i][e];
        slope = slopes[i][e];
      }
    };
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float u = q.x[i].get(e);
        if constexpr (PRE) {
          u = live[i] ? fmaf(s[i][e], u, a.res ? q.res[i].get(e) : 0.f) : 0.f;
        } else {
          float act, slope;
          gate_of(i, e, act, slope);
          if constexpr (!AGAIN) acts[i][e] = act, slopes[i][e] = slope;
          if (!a.norm_first) u *= act;
        }
        v[i][e] = u;
      }
      if (PRE && !BWD && a.ro && in && live[i]) store<R, V>(static_cast<R*>(a.ro) + at + col[i], v[i]);
    }
    if (a.layer) {
      float m[1] = {0.f};
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
#pragma unroll
        for (int e = 0; e < V; ++e) m[0] += v[i][e];
      }
      sum1(m);
      m[0] *= a.inv_w;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
#pragma unroll
        for (int e = 0; e < V; ++e) v[i][e] = live[i] ? v[i][e] - m[0] : 0.f;
      }
    }
    if constexpr (!BWD) {
      float ss[1] = {0.f};
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
#pragma unroll
        for (int e = 0; e < V; ++e) ss[0] += v[i][e] * v[i][e];
      }
      sum1(ss);
      const float r = 1.f / sqrtf(ss[0] * a.inv_w + a.eps);
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        float y[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
          y[e] = fmaf(v[i][e] * r, w[i][e], b[i][e]);
          if constexpr (!PRE) {
            if (a.norm_first) {
              float act, slope;
              gate_at(i, e, act, slope);
              y[e] *= act;
            }
            y[e] = a.res ? fmaf(s[i][e], y[e], q.res[i].get(e)) : s[i][e] * y[e];
          }
        }
        if (in && live[i]) {
          if constexpr (PRE) store<T, V>(static_cast<T*>(a.y) + at + col[i], y);
          else store<R, V>(static_cast<R*>(a.y) + at + col[i], y);
        }
      }
    } else {
      // d: the gradient by norm(u), after the weight
      float d[VPL][V], k[3] = {0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          float act = 1.f, slope;
          if (!PRE && a.norm_first) gate_at(i, e, act, slope);
          const float dn = PRE ? (a.dy ? q.dy[i].get(e) : 0.f) : q.dr[i].get(e) * s[i][e] * act;
          d[i][e] = dn * w[i][e];
          if (!live[i]) d[i][e] = 0.f;
          k[0] += v[i][e] * v[i][e];
          k[1] += d[i][e] * v[i][e];
          k[2] += d[i][e];
        }
      }
      sum3(k);
      if constexpr (AGAIN) {   // or the compiler would keep what was formed before
#pragma unroll
        for (int i = 0; i < VPL; ++i) q.z[i].renew();
      }
      const float r = 1.f / sqrtf(k[0] * a.inv_w + a.eps);
      const float dot = k[1] * a.inv_w * r * r, mean = a.layer ? k[2] * a.inv_w : 0.f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        float o1[V], o2[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float hat = v[i][e] * r, du = r * (d[i][e] - mean - v[i][e] * dot);
          if constexpr (PRE) {
            const float dy = a.dy ? q.dy[i].get(e) : 0.f;
            const float dr = du + (a.dr ? q.dr[i].get(e) : 0.f);
            if (in) {   // a row past the last may hold 0 * inf
              gw[i][e] += dy * hat;
              if (EXTRA) gb[i][e] += dy;
              if (EXTRA) gs[i][e] += dr * q.x[i].get(e);
            }
            o1[e] = dr * s[i][e];
            o2[e] = dr;
          } else {
            float act, slope;
            gate_at(i, e, act, slope);
            const float dout = q.dr[i].get(e), after = a.norm_first ? act : 1.f;
            const float dn = dout * s[i][e] * after, n = fmaf(hat, w[i][e], b[i][e]);
            if (in) {
              gw[i][e] += dn * hat;
              if (EXTRA) gb[i][e] += dn;
              if (EXTRA) gs[i][e] += dout * n * after;
            }
            o1[e] = a.norm_first ? du : du * act;
            o2[e] = (a.norm_first ? dout * s[i][e] * n : du * q.x[i].get(e)) * slope;
          }
        }
        if (in && live[i]) {
          if (a.dx) store<T, V, PASS>(static_cast<T*>(a.dx) + at + col[i], o1);
          if constexpr (PRE) {
            if (a.dres) store<R, V, PASS>(static_cast<R*>(a.dres) + at + col[i], o2);
          } else {
            if (a.dz) store<T, V, PASS>(static_cast<T*>(a.dz) + at + col[i], o2);
          }
        }
      }
    }
  }
  if constexpr (BWD) {
    float* slot = a.slots + static_cast<int64_t>(blockIdx.y) * SUMS * a.D;
    for (int k = 0; k < SUMS; ++k) {
      if ((!EXTRA && k) || !((a.sums >> k) & 1)) continue;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        float g[V];
#pragma unroll
        for (int e = 0; e < V; ++e) g[e] = k == 0 ? gw[i][e] : k == 1 ? gb[i][e] : gs[i][e] * a.alpha;
        if constexpr (WIDE) {
          if (live[i]) store<float, V>(slot + static_cast<int64_t>(k) * a.D + col[i], g);
        } else {
          // the block's tokens in order
          float* red = reinterpret_cast<float*>(smem);
          __syncthreads();
          store<float, V>(red + tid * V, g);
          __syncthreads();
          if (tl == 0) {
            const int apart = a.gpb * a.lpr * V;
            for (int j = 1; j < a.tpb; ++j) {
#pragma unroll
              for (int e = 0; e < V; ++e) g[e] += red[tid * V + j * apart + e];
            }
            if (live[i]) store<float, V>(slot + static_cast<int64_t>(k) * a.D + col[i], g);
          }
        }
      }
    }
  }
}

// The slots' sum: a column of a gradient per RED_ROWS threads, each adds every RED_ROWS-th slot in order, then those in order.
constexpr int RED_COLS = 32, RED_ROWS = 32;
__global__ __launch_bounds__(RED_COLS * RED_ROWS) void k_block_norm_reduce(const float* slots, int nslots, int D, float* dw, float* db, float* ds) {
  __shared__ double part[RED_ROWS][RED_COLS + 1];
  float* out = blockIdx.y == 0 ? dw : blockIdx.y == 1 ? db : ds;
  if (!out) return;
  const int lc = static_cast<int>(threadIdx.x) % RED_COLS, lr = static_cast<int>(threadIdx.x) / RED_COLS;
  const int col = static_cast<int>(blockIdx.x) * RED_COLS + lc;
  double s = 0.0;
  if (col < D) {
    const float* p = slots + static_cast<int64_t>(blockIdx.y) * D + col;
#pragma unroll 8
    for (int i = lr; i < nslots; i += RED_ROWS) s += static_cast<double>(p[static_cast<int64_t>(i) * SUMS * D]);
  }
  part[lr][lc] = s;
  __syncthreads();
  if (lr == 0 && col < D) {
#pragma unroll
    for (int i = 1; i < RED_ROWS; ++i) s += part[i][lc];
    out[col] = static_cast<float>(s);
  }
}

int check(const block_norm_shape* s, bool pre) {
  if (!s || s->reserved != 0) return SSD_ERR_INVALID_ARG;
  if (s->io_dtype != SSD_IO_BF16 && s->io_dtype != SSD_IO_F32) return SSD_ERR_UNSUPPORTED_SHAPE;
  if (s->residual_dtype != s->io_dtype && s->residual_dtype != SSD_IO_F32) return SSD_ERR_UNSUPPORTED_SHAPE;
  const int64_t vec = s->io_dtype == SSD_IO_BF16 ? 8 : 4;
  if (s->batch < 1 || s->seqlen < 1 || s->width < 1 || s->groups < 1) return SSD_ERR_UNSUPPORTED_SHAPE;
  if (s->batch > INT32_MAX || s->seqlen > INT32_MAX || s->batch * s->seqlen > INT32_MAX) return SSD_ERR_UNSUPPORTED_SHAPE;
  if (s->width > (1 << 20) || s->width % s->groups || (pre && s->groups != 1)) return SSD_ERR_UNSUPPORTED_SHAPE;
  const int64_t w = s->width / s->groups;
  if (w % vec || w > MAX_WIDTH) return SSD_ERR_UNSUPPORTED_SHAPE;
  for (const int64_t st : {s->x_batch_stride, s->x_row_stride, s->z_batch_stride, s->z_row_stride})
    if (st < 0 || st % vec) return SSD_ERR_UNSUPPORTED_SHAPE;
  if (s->norm != BLOCK_NORM_RMS && s->norm != BLOCK_NORM_LAYER) return SSD_ERR_UNSUPPORTED_SHAPE;
  if (s->gate != BLOCK_NORM_SILU && s->gate != BLOCK_NORM_SIGMOID) return SSD_ERR_UNSUPPORTED_SHAPE;
  if (s->norm_before_gate != 0 && s->norm_before_gate != 1) return SSD_ERR_UNSUPPORTED_SHAPE;
  if (!(s->eps >= 0.f) || !(s->alpha - s->alpha == 0.f)) return SSD_ERR_INVALID_ARG;
  return SSD_OK;
}

bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

// How a row lies in the lanes, and the grid.
struct Plan {
  int lay, threads, lpr, gpb, tpb;
  int64_t gx, gy;                      // blocks of tokens, and of groups (which run side by side)
};

Plan plan(const block_norm_shape& s, bool bwd) {
  Plan p{};
  const int64_t tokens = s.batch * s.seqlen;
  const int pieces = static_cast<int>(s.width / s.groups) / (s.io_dtype == SSD_IO_BF16 ? 8 : 4);
  if (pieces > 64) {
    auto threads = [&](int lay) {
      const int vpl = s.io_dtype == SSD_IO_BF16 ? pieces_a_lane<bf16_t>(lay) : pieces_a_lane<float>(lay);
      return ((pieces + vpl - 1) / vpl + 63) / 64 * 64;
    };
    p.lay = threads(WIDE1) <= 512 ? WIDE1 : threads(WIDE2) <= 512 ? WIDE2 : WIDEST;
    if (p.lay == WIDEST && s.io_dtype == SSD_IO_F32 && threads(WIDE4) <= 512) p.lay = WIDE4;
    p.threads = threads(p.lay);
    p.lpr = 64;
    p.gpb = p.tpb = 1;
    p.gy = s.groups;
  } else {
    p.lay = NARROW;
    p.threads = THR;
    p.lpr = 1;
    while (p.lpr < pieces) p.lpr *= 2;
    const int places = THR / p.lpr;
    p.gpb = 1;
    while (p.gpb < s.groups && p.gpb < places) p.gpb *= 2;
    p.tpb = places / p.gpb;
    p.gy = (s.groups + p.gpb - 1) / p.gpb;
  }
  // Threads in all: the forward eight times what the card holds at once (16384 rows of 8 gated groups of 1024 bf16: 163 us
  // at twice, 150 at four times, 144 at eight; 16384 rows of 4096 with a float32 residual: 150 us, at 16 times 160), the
  // backward half of it, since each block leaves its sums in a slot (278 us there at half, 305 at once and at a quarter)
  const int64_t most = static_cast<int64_t>(256) * (bwd ? 1024 : 16384) / p.threads / p.gy;
  p.gx = (tokens + p.tpb - 1) / p.tpb;
  if (p.gx > most) p.gx = most < 1 ? 1 : most;
  return p;
}

template <typename T, typename R, int LAY, bool PRE, int DIR> int go(const Plan& p, const Args& a, hipStream_t st) {
  const size_t lds = DIR != FORWARD && LAY == NARROW ? sizeof(float) * THR * ssd::Vec16<T>::N : 0;
  const dim3 grid(static_cast<unsigned>(p.gy), static_cast<unsigned>(p.gx)), block(static_cast<unsigned>(p.threads));
  if (a.b || a.s || (a.sums & ~1)) hipLaunchKernelGGL((k_block_norm<T, R, LAY, PRE, DIR, true>), grid, block, lds, st, a);
  else hipLaunchKernelGGL((k_block_norm<T, R, LAY, PRE, DIR, false>), grid, block, lds, st, a);
  return hipGetLastError() == hipSuccess ? SSD_OK : SSD_ERR_HIP;
}

template <typename T, typename R, bool PRE, int DIR> int by_width(const Plan& p, const Args& a, hipStream_t st) {
  switch (p.lay) {
    case NARROW: return go<T, R, NARROW, PRE, DIR>(p, a, st);
    case WIDE1: return go<T, R, WIDE1, PRE, DIR>(p, a, st);
    case WIDE2: return go<T, R, WIDE2, PRE, DIR>(p, a, st);
    case WIDE4:
      if constexpr (sizeof(T) == 4) return go<T, R, WIDE4, PRE, DIR>(p, a, st);
      return SSD_ERR_UNSUPPORTED_SHAPE;   // plan() takes it for float32 only
    default: return go<T, R, WIDEST, PRE, DIR>(p, a, st);
  }
}

template <bool PRE, int DIR> int by_type(const block_norm_shape& s, const Plan& p, const Args& a, hipStream_t st) {
  if (s.io_dtype == SSD_IO_F32) return by_width<float, float, PRE, DIR>(p, a, st);
  if (s.residual_dtype == SSD_IO_F32) return by_width<bf16_t, float, PRE, DIR>(p, a, st);
  return by_width<bf16_t, bf16_t, PRE, DIR>(p, a, st);
}

template <bool PRE, bool BWD> int launch(const block_norm_shape& s, Args& a, hipStream_t st) {
  const Plan p = plan(s, BWD);
  const bool xc = s.x_batch_stride == 0 && s.x_row_stride == 0, zc = s.z_batch_stride == 0 && s.z_row_stride == 0;
  a.x_sl = xc ? s.width : s.x_row_stride;
  a.x_sb = xc ? s.seqlen * s.width : s.x_batch_stride;
  a.z_sl = zc ? s.width : s.z_row_stride;
  a.z_sb = zc ? s.seqlen * s.width : s.z_batch_stride;
  a.flat = a.x_sb == s.seqlen * a.x_sl && (!a.z || a.z_sb == s.seqlen * a.z_sl);
  a.tokens = static_cast<int>(s.batch * s.seqlen);
  a.L = static_cast<int>(s.seqlen);
  a.D = static_cast<int>(s.width);
  a.groups = static_cast<int>(s.groups);
  a.W = a.D / a.groups;
  a.lpr = p.lpr; a.gpb = p.gpb; a.tpb = p.tpb;
  a.layer = s.norm == BLOCK_NORM_LAYER;
  a.sigmoid = s.gate == BLOCK_NORM_SIGMOID;
  a.norm_first = s.norm_before_gate;
  a.eps = s.eps;
  a.alpha = s.alpha;
  a.inv_w = 1.f / static_cast<float>(a.W);
  if constexpr (!BWD) return by_type<PRE, FORWARD>(s, p, a, st);
  // The backward's operands pass the caches by where it moves more than the 256 MB of the last one: what is given, and for
  // add_norm the residual's rows also where there is none, as the forward's r then lies there.  Microseconds past the caches
  // and by them, in brackets with the forward before: gated 16384 x 8192 bf16 271 and 286; 7000 x 4096 (273 MB) 59 and 56 (92,
  // 91), 8500 69 and 74 (109, 108); no z, 9000 x 4096 (210 MB) 52 and 50 (88, 86), float32 3500 x 4096 (164 MB) 49 and 42 (69,
  // 64).  add_norm bf16, float32 residual: 4200 x 4096 (295 MB) 63 and 59 (91, 91), 5500 (386 MB) 79 and 86 (115, 134); no
  // residual, 6300 x 4096 (246 MB with r) 44 and 40 (69, 69), 9000 60 and 56 (91, 101).
  const int64_t io = s.io_dtype == SSD_IO_BF16 ? 2 : 4, res = s.residual_dtype == SSD_IO_BF16 ? 2 : 4;
  int64_t bytes = PRE ? res : 0;   // of a value
  for (const void* t : {a.x, a.z, a.dy, static_cast<const void*>(a.dx), static_cast<const void*>(a.dz)}) bytes += t ? io : 0;
  for (const void* t : {a.dr, static_cast<const void*>(a.dres)}) bytes += t ? res : 0;
  bytes *= static_cast<int64_t>(a.tokens) * a.D;
  return bytes > (int64_t{256} << 20) ? by_type<PRE, BACKWARD_PASS>(s, p, a, st) : by_type<PRE, BACKWARD>(s, p, a, st);
}

// The backward of either: its kernel, then the slots' sums that are wanted
template <bool PRE> int launch_bwd(const block_norm_shape& s, Args& a, float* dw, float* db, float* ds, void* workspace, hipStream_t st) {
  a.slots = static_cast<float*>(workspace);
  a.sums = (dw ? 1 : 0) | (db ? 2 : 0) | (ds ? 4 : 0);
  const int rc = launch<PRE, true>(s, a, st);
  if (rc != SSD_OK || !a.sums) return rc;
  hipLaunchKernelGGL(k_block_norm_reduce, dim3(static_cast<unsigned>((s.width + RED_COLS - 1) / RED_COLS), SUMS), dim3(RED_COLS * RED_ROWS), 0, st,
                     a.slots, static_cast<int>(plan(s, true).gx), a.D, dw, db, ds);
  return hipGetLastError() == hipSuccess ? SSD_OK : SSD_ERR_HIP;
}

}  // namespace bnorm

extern "C" {

int add_norm_fwd(const block_norm_shape* shape, const void* x, const void* residual, const float* weight,
                 const float* bias, const float* scale, void* y, void* residual_out, void* stream) {
  const int rc = bnorm::check(shape, true);
  if (rc != SSD_OK) return rc;
  if (!x || !y || y == residual || y == residual_out || (residual_out && residual_out == x)) return SSD_ERR_INVALID_ARG;
  if (y == x && (shape->x_batch_stride || shape->x_row_stride)) return SSD_ERR_INVALID_ARG;
  for (const void* p : {x, residual, static_cast<const void*>(weight), static_cast<const void*>(bias), static_cast<const void*>(scale),
                        static_cast<const void*>(y), static_cast<const void*>(residual_out)})
    if (bnorm::misaligned(p)) return SSD_ERR_MISALIGNED;
  bnorm::Args a{};
  a.x = x; a.res = residual; a.w = weight; a.b = bias; a.s = scale; a.y = y; a.ro = residual_out;
  return bnorm::launch<true, false>(*shape, a, static_cast<hipStream_t>(stream));
}

int gated_norm_fwd(const block_norm_shape* shape, const void* x, const void* z, const float* weight,
                   const float* bias, const void* residual, const float* scale, void* out, void* stream) {
  const int rc = bnorm::check(shape, false);
  if (rc != SSD_OK) return rc;
  if (!x || !out || (!residual && shape->residual_dtype != shape->io_dtype)) return SSD_ERR_INVALID_ARG;
  if (out == x || out == z) return SSD_ERR_INVALID_ARG;
  for (const void* p : {x, z, residual, static_cast<const void*>(weight), static_cast<const void*>(bias), static_cast<const void*>(scale),
                        static_cast<const void*>(out)})
    if (bnorm::misaligned(p)) return SSD_ERR_MISALIGNED;
  bnorm::Args a{};
  a.x = x; a.z = z; a.res = residual; a.w = weight; a.b = bias; a.s = scale; a.y = out;
  return bnorm::launch<false, false>(*shape, a, static_cast<hipStream_t>(stream));
}

int block_norm_bwd_workspace_size(const block_norm_shape* shape, size_t* bytes) {
  const int rc = bnorm::check(shape, false);
  if (rc != SSD_OK) return rc;
  if (!bytes) return SSD_ERR_INVALID_ARG;
  *bytes = static_cast<size_t>(bnorm::plan(*shape, true).gx) * bnorm::SUMS * static_cast<size_t>(shape->width) * sizeof(float);
  return SSD_OK;
}

int add_norm_bwd(const block_norm_shape* shape, const void* x, const void* residual, const float* weight,
                 const float* scale, const void* dy, const void* dresidual_out, void* dx, void* dresidual,
                 float* dweight, float* dbias, float* dscale, void* workspace, size_t workspace_bytes,
                 void* stream) {
  size_t need = 0;
  int rc = bnorm::check(shape, true);
  if (rc == SSD_OK) rc = block_norm_bwd_workspace_size(shape, &need);
  if (rc != SSD_OK) return rc;
  if (!x || (!dy && !dresidual_out) || !workspace) return SSD_ERR_INVALID_ARG;
  if (workspace_bytes < need) return SSD_ERR_WORKSPACE_TOO_SMALL;
  for (const void* p : {x, residual, dy, dresidual_out, static_cast<const void*>(weight), static_cast<const void*>(scale),
                        static_cast<const void*>(dx), static_cast<const void*>(dresidual), static_cast<const void*>(workspace)})
    if (bnorm::misaligned(p)) return SSD_ERR_MISALIGNED;
  for (const void* o : {static_cast<const void*>(dx), static_cast<const void*>(dresidual)})
    for (const void* i : {x, residual, dy, dresidual_out})
      if (o && o == i) return SSD_ERR_INVALID_ARG;
  if (dx && dx == dresidual) return SSD_ERR_INVALID_ARG;
  bnorm::Args a{};
  a.x = x; a.res = residual; a.w = weight; a.s = scale; a.dy = dy; a.dr = dresidual_out;
  a.dx = dx; a.dres = dresidual;
  return bnorm::launch_bwd<true>(*shape, a, dweight, dbias, dscale, workspace, static_cast<hipStream_t>(stream));
}

int gated_norm_bwd(const block_norm_shape* shape, const void* x, const void* z, const float* weight,
                   const float* bias, const float* scale, const void* dout, void* dx, void* dz, float* dweight,
                   float* dbias, float* dscale, void* workspace, size_t workspace_bytes, void* stream) {
  size_t need = 0;
  const int rc = block_norm_bwd_workspace_size(shape, &need);
  if (rc != SSD_OK) return rc;
  if (!x || !dout || !workspace || (dz && !z)) return SSD_ERR_INVALID_ARG;
  if (workspace_bytes < need) return SSD_ERR_WORKSPACE_TOO_SMALL;
  for (const void* p : {x, z, dout, static_cast<const void*>(weight), static_cast<const void*>(bias), static_cast<const void*>(scale),
                        static_cast<const void*>(dx), static_cast<const void*>(dz), static_cast<const void*>(workspace)})
    if (bnorm::misaligned(p)) return SSD_ERR_MISALIGNED;
  for (const void* o : {static_cast<const void*>(dx), static_cast<const void*>(dz)})
    for (const void* i : {x, z, dout})
      if (o && o == i) return SSD_ERR_INVALID_ARG;
  if (dx && dx == dz) return SSD_ERR_INVALID_ARG;
  bnorm::Args a{};
  a.x = x; a.z = z; a.w = weight; a.b = bias; a.s = scale; a.dr = dout;
  a.dx = dx; a.dz = dz;
  return bnorm::launch_bwd<false>(*shape, a, dweight, dbias, dscale, workspace, static_cast<hipStream_t>(stream));
}

}  // extern "C"
