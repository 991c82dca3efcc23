// Gated delta rule over whole sequences: sequence starts, the chunks' own
// matrices and the walk over a sequence's chunks (the forward, and the
// backward's recomputation of it).
//
// A sequence is cut into chunks of 64 rows.  With c_i the sum of g over the
// chunk's rows up to i and G_ij = exp(c_i - c_j), the chunk's residuals e
// given its entering state S solve a unit lower triangular system:
//
//     e_i + sum_{j<i} G_ij (k_i . k_j) beta_j e_j = r_i,   r_i = v_i - exp(c_i) S k_i
//     e = T' r,   T' = (I + N diag(beta))^-1,   N_ij = G_ij k_i . k_j  (j < i)
//     o_i = scale (exp(c_i) S q_i + sum_{j<=i} G_ij (q_i . k_j) beta_j e_j)
//     S  <- exp(c_last) S + sum_j exp(c_last - c_j) beta_j e_j k_j^T
//
// T' and the scores depend on q, k, g and beta alone, so k_delta_prep forms
// them for all chunks at once; what is sequential, the walk, is three
// products of 64 rows per chunk.  Exponents are differences of sums of g taken
// in double: a strong decay early in a chunk does not cost the later rows'
// differences their last bits.
#include <type_traits>

#include "delta_problem.h"
#include "delta_tiles.h"
#include "ssd_bwd.h"
#include "ssd_problem.h"

namespace delta {

// ---------------------------------------------------------------------------
// k_delta_starts: the first rows of the sequences that seq_idx marks, in row
// order.  One block: every thread takes 16 rows of a stretch of 16384, the
// counts are scanned over the block.
// ---------------------------------------------------------------------------
constexpr int ST_THR = 1024, ST_ROWS = 16;

__global__ __launch_bounds__(ST_THR) void k_delta_starts(Problem p) {
  __shared__ int wsum[ST_THR / 64];
  __shared__ int base;
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, wave = tid >> 6;
  if (tid == 0) base = 0;
  __syncthreads();
  for (int64_t first = 0; first < p.total; first += ST_THR * ST_ROWS) {
    const int64_t r0 = first + tid * ST_ROWS;
    uint32_t mask = 0;
    int prev = (r0 > 0 && r0 < p.total) ? p.seq_idx[r0 - 1] : 0;
#pragma unroll
    for (int i = 0; i < ST_ROWS; ++i) {
      const int64_t r = r0 + i;
      if (r < p.total) {
        const int v = p.seq_idx[r];
        if (r % p.L == 0 || v != prev) mask |= 1u << i;
        prev = v;
      }
    }
    const int mine = __popc(mask);
    int incl = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(incl, d);
      if (lane >= d) incl += o;
    }
    if (lane == 63) wsum[wave] = incl;
    __syncthreads();
    int at = base + incl - mine, all = 0;
    for (int w = 0; w < ST_THR / 64; ++w) {
      if (w < wave) at += wsum[w];
      all += wsum[w];
    }
    for (int i = 0; i < ST_ROWS; ++i) {
      if ((mask >> i) & 1u) {
        if (at <= p.nseqs) p.starts[at] = static_cast<int>(r0 + i);
        ++at;
      }
    }
    __syncthreads();
    if (tid == 0) base += all;
    __syncthreads();
  }
  for (int64_t s = static_cast<int64_t>(base) + tid; s <= p.nseqs; s += ST_THR) p.starts[s] = p.total;
}

// ---------------------------------------------------------------------------
// k_delta_prep: T' (and for the backward the transposed (I + diag(beta) N)^-1
// and the transposed scores) and the scores of one chunk and head, as the
// walks' operand fragments.
//
// The inverse of a unit lower triangular 64 x 64 matrix in float32: the four
// 16 x 16 diagonal blocks by substitution (a lane per column, one wave), then
// 32 x 32 and 64 x 64 by the block formula T21 = -T22 A21 T11 with float32
// MFMA tiles, in place in LDS.
// ---------------------------------------------------------------------------
constexpr int LDM = 68;   // pitch of the float32 64 x 64 matrices

template <typename T, int NT, bool BWD> struct PrepCfg {
  static constexpr int ND = 32 * NT;
  using TileT = Tile<T, CH, ND, 256>;
  static constexpr int NM = BWD ? 2 : 1;
  static constexpr size_t OFF_Q = sizeof(T) * TileT::LDS_ELEMS;
  static constexpr size_t OFF_M = 2 * OFF_Q;
  static constexpr size_t OFF_P = OFF_M + sizeof(float) * NM * CH * LDM;
  static constexpr size_t OFF_C = OFF_P + sizeof(float) * CH * LDM;
  static constexpr size_t OFF_B = OFF_C + sizeof(double) * CH;
  static constexpr size_t LDS = OFF_B + sizeof(float) * CH;
};

// acc += A B of 16 x 16 float32 blocks in LDS
__device__ __forceinline__ f32x4_t block_mma(const float* a, const float* b, f32x4_t acc) {
  const int l = ssd::lane_id();
  return ssd::Mma<float>::mma_rd(*reinterpret_cast<const f32x4_t*>(a + (l & 15) * LDM + 4 * (l >> 4)),
                                 ssd::Mma<float>::rfrag_load_kn(b, LDM), acc);
}
__device__ __forceinline__ void block_store(float* m, f32x4_t v) {
  const int l = ssd::lane_id();
#pragma unroll
  for (int r = 0; r < 4; ++r) m[(4 * (l >> 4) + r) * LDM + (l & 15)] = v[r];
}

template <int NM> __device__ __forceinline__ void invert64(float* m) {
  const int l = ssd::lane_id(), g = l >> 4, c = l & 15, w = ssd::wave_id_s();
  auto blk = [&](int mat, int i, int j) { return m + mat * CH * LDM + 16 * i * LDM + 16 * j; };
  if (w < NM) {
    float* d = blk(w, g, g);
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = i == c ? 1.f : 0.f;
#pragma unroll
    for (int k = 0; k < 15; ++k) {
#pragma unroll
      for (int i = k + 1; i < 16; ++i) x[i] -= d[i * LDM + k] * x[k];
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) d[i * LDM + c] = x[i];
  }
  __syncthreads();
  if (w < 2 * NM) {
    const int mat = w >> 1, q = 2 * (w & 1);
    const f32x4_t y = block_mma(blk(mat, q + 1, q), blk(mat, q, q), zero4());
    const float* t = blk(mat, q + 1, q + 1);
    const f32x4_t x = ssd::Mma<float>::mma_rd(*reinterpret_cast<const f32x4_t*>(t + c * LDM + 4 * g), y, zero4());
    block_store(blk(mat, q + 1, q), -x);
  }
  __syncthreads();
  const int i = 2 + (w >> 1), j = w & 1;
  f32x4_t y[NM];
#pragma unroll
  for (int mat = 0; mat < NM; ++mat) {
    y[mat] = block_mma(blk(mat, i, 1), blk(mat, 1, j), zero4());   // T_01 is zero
    if (j == 0) y[mat] = block_mma(blk(mat, i, 0), blk(mat, 0, 0), y[mat]);
  }
  __syncthreads();
#pragma unroll
  for (int mat = 0; mat < NM; ++mat) block_store(blk(mat, i, j), y[mat]);
  __syncthreads();
#pragma unroll
  for (int mat = 0; mat < NM; ++mat) {
    y[mat] = block_mma(blk(mat, i, 2), blk(mat, 2, j), zero4());
    if (i == 3) y[mat] = block_mma(blk(mat, 3, 3), blk(mat, 3, j), y[mat]);
  }
  __syncthreads();
#pragma unroll
  for (int mat = 0; mat < NM; ++mat) block_store(blk(mat, i, j), -y[mat]);
  __syncthreads();
}

template <typename T, int NT, bool BWD> __global__ __launch_bounds__(256) void k_delta_prep(Problem p) {
  using Cf = PrepCfg<T, NT, BWD>;
  using F = Fr<T>;
  using TileT = typename Cf::TileT;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  T* kt = reinterpret_cast<T*>(smem);
  T* qt = reinterpret_cast<T*>(smem + Cf::OFF_Q);
  float* mm = reinterpret_cast<float*>(smem + Cf::OFF_M);
  float* pm = reinterpret_cast<float*>(smem + Cf::OFF_P);
  double* cs = reinterpret_cast<double*>(smem + Cf::OFF_C);
  float* bs = reinterpret_cast<float*>(smem + Cf::OFF_B);

  const int slot = static_cast<int>(blockIdx.x), h = static_cast<int>(blockIdx.y), grp = h / p.hpg;
  const Chunk ch = chunk_of(p, slot);
  if (ch.len == 0) return;
  const int64_t sh = static_cast<int64_t>(slot) * p.H + h;
  const int tid = static_cast<int>(threadIdx.x), l = tid & 63, g = l >> 4, c = l & 15, w = ssd::wave_id_s();

  TileT tk, tq;
  tk.load(static_cast<const T*>(p.k) + row_offset(ch.row, p.L, p.k_sb, p.k_sl) + static_cast<int64_t>(grp) * p.N, p.k_sl, ch.len, p.N, tid);
  tq.load(static_cast<const T*>(p.q) + row_offset(ch.row, p.L, p.q_sb, p.q_sl) + static_cast<int64_t>(grp) * p.N, p.q_sl, ch.len, p.N, tid);
  if (tid < CH) {
    const int64_t at = static_cast<int64_t>(ch.row + tid) * p.H + h;
    float gv = tid < ch.len ? p.g[at] : 0.f;
    gv = gv < -104.f ? -104.f : gv;
    const float b = tid < ch.len ? p.beta[at] : 0.f;
    double s = gv;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const double o = __shfl_up(s, d);
      if (tid >= d) s += o;
    }
    cs[tid] = s;
    bs[tid] = b;
    const double last = __shfl(s, 63);
    float* gt = p.gates + sh * (GATES * CH) + tid;
    gt[GATE_IN * CH] = expf(static_cast<float>(s));
    gt[GATE_OUT * CH] = expf(static_cast<float>(last - s));
    gt[GATE_BETA * CH] = b;
    const float hi = static_cast<float>(s);
    gt[GATE_C * CH] = hi;
    gt[GATE_CLO * CH] = static_cast<float>(s - hi);
  }
  tk.store(kt, tid);
  tq.store(qt, tid);
  __syncthreads();

  // rows 16 w .. 16 w + 15 of N and of the scores; zero above the diagonal
  for (int ct = 0; ct < 4; ++ct) {
    f32x4_t kk = zero4(), qk = zero4();
    if (ct <= w) {
#pragma unroll
      for (int ks = 0; ks < NT; ++ks) {
        const typename F::X b = F::load(kt + (16 * ct + c) * TileT::LD + 32 * ks + 8 * g);
        kk = mma(F::load(kt + (16 * w + c) * TileT::LD + 32 * ks + 8 * g), b, kk);
        qk = mma(F::load(qt + (16 * w + c) * TileT::LD + 32 * ks + 8 * g), b, qk);
      }
    }
    const int j = 16 * ct + c;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int i = 16 * w + 4 * g + r;
      const float dec = j <= i ? expf(static_cast<float>(cs[i] - cs[j])) : 0.f;
      const float n = j < i ? kk[r] * dec : 0.f;
      mm[i * LDM + j] = n * bs[j];
      if constexpr (BWD) mm[CH * LDM + i * LDM + j] = n * bs[i];
      pm[i * LDM + j] = j <= i ? p.scale * (qk[r] * dec) : 0.f;
    }
  }
  __syncthreads();
  invert64<Cf::NM>(mm);

  auto put = [&](uint4* to, int f, const float (&v)[8]) {
    uint4 u[2];
    F::pieces(F::split(v), u);
    uint4* d = to + sh * FRAG_PIECES + 2 * f * 64 + l;
    d[0] = u[0];
    d[64] = u[1];
  };
  for (int f = w; f < NFRAG; f += 4) {
    // lower: (0,0) (1,0) (2,0) (2,1) (3,0) (3,1); upper: (0,0) (0,1) (1,0) (1,1) (2,1) (3,1)
    const int lt = f < 2 ? f : 2 + ((f - 2) >> 1), lk = f < 2 ? 0 : (f - 2) & 1;
    const int row = perm_row(lt, c);
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = mm[row * LDM + 32 * lk + 8 * g + e] - (row == 32 * lk + 8 * g + e ? 1.f : 0.f);
    put(p.tf, f, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = pm[(16 * lt + c) * LDM + 32 * lk + 8 * g + e];
    put(p.pf, f, v);
    if constexpr (BWD) {
      const int ut = f < 4 ? f >> 1 : f - 2, uk = f < 4 ? f & 1 : 1;
      const int col = perm_row(ut, c);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = mm[CH * LDM + (32 * uk + 8 * g + e) * LDM + col] - (col == 32 * uk + 8 * g + e ? 1.f : 0.f);
      put(p.ttf, f, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = pm[(32 * uk + 8 * g + e) * LDM + col];
      put(p.ptf, f, v);
    }
  }
}

// ---------------------------------------------------------------------------
// k_delta_walk: one sequence's chunks in order, for one head and 16 NSW of its
// value columns.  A column of S needs no other column, so each of the NSW
// state waves keeps 16 columns (N x 16) in registers as accumulator tiles for
// the whole sequence and runs the sequential part alone:
//     k S -> r -> T' r -> S   (three products a chunk, nothing else).
// Beside them, on the other SIMDs, NSW / 2 output waves form the previous
// chunk's o from the entering state and the corrections that two state waves
// each leave in LDS (in the backward dout . o, and the stores of states and
// corrections), and NSW / 2 staging waves bring the coming chunks' rows in:
// their loads are in flight for a whole chunk, which no wave waits for.
//
// Per chunk two barriers: between the first and the second the state waves
// work on chunk i, the output waves on chunk i - 1 and the staging waves on
// k, v of chunk i + 1 and q, scores of chunk i; between the second and the
// next first the output waves take what the state waves left for them.
// ---------------------------------------------------------------------------
template <typename T, int NT, bool BWD, int NSW> struct WalkCfg {
  static constexpr int ND = 32 * NT, PS = SLICE * NSW, NOUT = NSW / 2, HT = 64 * (NSW / 2), THREADS = 128 * NSW;
  using TileN = Tile<T, CH, ND, HT>;
  using TileP = Tile<T, CH, PS, HT>;
  // q and the scores through LDS, or (512-byte rows: no room) straight into the output waves' registers
  static constexpr bool QLDS = sizeof(T) * ND <= 256;
  // terms of the entering states and corrections in o: one where o ends in bf16 (its error then is 2.4e-3, the
  // output's own rounding 1.7e-3 of it), two for the float32 dout . o
  static constexpr int XP = BWD || sizeof(T) == 4 ? 2 : 1;
  static constexpr size_t N_BYTES = sizeof(T) * TileN::LDS_ELEMS, V_BYTES = sizeof(T) * TileP::LDS_ELEMS;
  static constexpr size_t OFF_V = 2 * N_BYTES;
  static constexpr size_t OFF_Q = OFF_V + 2 * V_BYTES;
  static constexpr size_t OFF_P = OFF_Q + (QLDS ? 2 * N_BYTES : 0);
  static constexpr size_t OFF_XS = OFF_P + (QLDS ? 2 * 16 * FRAG_PIECES : 0);
  static constexpr size_t OFF_XU = OFF_XS + 16 * 64 * NSW * NT * XP;
  static constexpr size_t OFF_G = OFF_XU + 16 * 64 * NSW * 4;
  static constexpr size_t LDS = OFF_G + 2 * sizeof(float) * 3 * CH;
};

template <typename T, int NT, bool BWD, int NSW>
__global__ __launch_bounds__(128 * NSW) void k_delta_walk(Problem p) {
  using Cf = WalkCfg<T, NT, BWD, NSW>;
  using F = Fr<T>;
  using TileN = typename Cf::TileN;
  using TileP = typename Cf::TileP;
  constexpr int ND = Cf::ND, LDN = TileN::LD, LDP = TileP::LD, XP = Cf::XP, PS = Cf::PS;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  auto kbuf = [&](int i) { return reinterpret_cast<T*>(smem + (i & 1) * Cf::N_BYTES); };
  auto vbuf = [&](int i) { return reinterpret_cast<T*>(smem + Cf::OFF_V + (i & 1) * Cf::V_BYTES); };
  auto qbuf = [&](int i) { return reinterpret_cast<T*>(smem + Cf::OFF_Q + (i & 1) * Cf::N_BYTES); };
  auto pbuf = [&](int i) { return reinterpret_cast<uint4*>(smem + Cf::OFF_P) + (i & 1) * FRAG_PIECES; };
  auto gbuf = [&](int i) { return reinterpret_cast<float*>(smem + Cf::OFF_G) + (i & 1) * 3 * CH; };
  uint4* xs = reinterpret_cast<uint4*>(smem + Cf::OFF_XS);      // [wave][q][term][lane]
  f32x4_t* xu = reinterpret_cast<f32x4_t*>(smem + Cf::OFF_XU);  // [wave][t][lane]

  const int np = (p.P + PS - 1) / PS;
  const int h = static_cast<int>(blockIdx.x) / np, ps = static_cast<int>(blockIdx.x) % np;
  const int seq = static_cast<int>(blockIdx.y), grp = h / p.hpg;
  const int s0 = seq_start(p, seq), s1 = seq_start(p, seq + 1);
  const int nchunk = (s1 - s0 + CH - 1) / CH, slot0 = slot_base(s0, seq);
  const int tid = static_cast<int>(threadIdx.x), l = tid & 63, g = l >> 4, c = l & 15, w = ssd::wave_id_s();
  auto slot_head = [&](int i) { return static_cast<int64_t>(slot0 + i) * p.H + h; };
  auto length = [&](int i) { return min(CH, s1 - s0 - CH * i); };

  if (w < NSW) {
    // ---- state waves
    const int col = PS * ps + SLICE * w + c;   // this lane's value column
    const int slice = ps * NSW + w;
    const int64_t state_at = ((static_cast<int64_t>(seq) * p.H + h) * p.P + col) * p.N;
    f32x4_t S[2 * NT];
#pragma unroll
    for (int j = 0; j < 2 * NT; ++j) {
      const int n = pair_col(j) + 8 * g;
      S[j] = zero4();
      if (p.h0 && col < p.P && n < p.N) S[j] = *reinterpret_cast<const f32x4_t*>(p.h0 + state_at + n);
    }
    typename F::S sf[NT];
    auto split_state = [&](int q) {
      float v[8];
      pair8(S[2 * q], S[2 * q + 1], v);
      sf[q] = F::split(v);
    };
#pragma unroll
    for (int q = 0; q < NT; ++q) split_state(q);
    FragRegs tf;
    if (nchunk) tf.request(p.tf + slot_head(0) * FRAG_PIECES);
    for (int i = 0; i < nchunk; ++i) {
      const T *kt = kbuf(i), *vt = vbuf(i);
      const float* gs = gbuf(i);
      __syncthreads();
#pragma unroll
      for (int q = 0; q < NT; ++q) {
        uint4 u[2];
        F::pieces(sf[q], u);
#pragma unroll
        for (int t = 0; t < XP; ++t) xs[((w * NT + q) * XP + t) * 64 + l] = u[t];
      }
      // r = v - exp(c) k S, rows in pair order
      f32x4_t x[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) x[t] = zero4();
#pragma unroll
      for (int q = 0; q < NT; ++q) {
#pragma unroll
        for (int t = 0; t < 4; ++t) x[t] = mma(F::load(kt + perm_row(t, c) * LDN + 32 * q + 8 * g), sf[q], x[t]);
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int row = pair_col(t) + 8 * g;
        x[t] = F::load4_tr(vt + SLICE * w, LDP, row) - *reinterpret_cast<const f32x4_t*>(gs + GATE_IN * CH + row) * x[t];
      }
      // e = r + (T' - I) r, u = beta e
      typename F::S f2[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float v[8];
        pair8(x[2 * q], x[2 * q + 1], v);
        f2[q] = F::split(v);
      }
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
#pragma unroll
        for (int t = 2 * ks; t < 4; ++t) x[t] = mma(tf.get<T>(lower_frag(t, ks)), f2[ks], x[t]);
      }
      if (i + 1 < nchunk) tf.request(p.tf + slot_head(i + 1) * FRAG_PIECES);
      typename F::S3 f3[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int row = 32 * q + 8 * g;
        if constexpr (BWD) {
          if (slice < p.nsl) {
            uint4* e = p.e + ((slot_head(i) * p.nsl + slice) * 4 + 2 * q) * 64 + l;
            e[0] = __builtin_bit_cast(uint4, x[2 * q]);
            e[64] = __builtin_bit_cast(uint4, x[2 * q + 1]);
          }
        }
        const f32x4_t u0 = x[2 * q] * *reinterpret_cast<const f32x4_t*>(gs + GATE_BETA * CH + row);
        const f32x4_t u1 = x[2 * q + 1] * *reinterpret_cast<const f32x4_t*>(gs + GATE_BETA * CH + row + 4);
        xu[(w * 4 + 2 * q) * 64 + l] = u0;
        xu[(w * 4 + 2 * q + 1) * 64 + l] = u1;
        float v[8];
        pair8(u0 * *reinterpret_cast<const f32x4_t*>(gs + GATE_OUT * CH + row),
              u1 * *reinterpret_cast<const f32x4_t*>(gs + GATE_OUT * CH + row + 4), v);
        f3[q] = F::split3(v);
      }
      // S <- exp(c_last) S + k^T (exp(c_last - c) u)
      const float last = gs[GATE_IN * CH + CH - 1];
#pragma unroll
      for (int j = 0; j < 2 * NT; ++j) {
        S[j] *= last;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) S[j] = mma(F::template load_tr<8>(kt + pair_col(j), LDN, 32 * ks + 8 * g), f3[ks], S[j]);
        if (j & 1) split_state(j >> 1);
      }
      __syncthreads();
    }
    if constexpr (!BWD) {
      if (p.final && col < p.P) {
#pragma unroll
        for (int j = 0; j < 2 * NT; ++j) {
          const int n = pair_col(j) + 8 * g;
          if (n < p.N) *reinterpret_cast<f32x4_t*>(p.final + state_at + n) = S[j];
        }
      }
    }
    return;
  }
  if (nchunk == 0) return;
  const T* qp = static_cast<const T*>(p.q) + row_offset(s0, p.L, p.q_sb, p.q_sl) + static_cast<int64_t>(grp) * p.N;
  const int64_t hp = static_cast<int64_t>(p.H) * p.P;

  if (w < NSW + Cf::NOUT) {
    // ---- output waves: the columns of state waves 2 ow and 2 ow + 1
    const int ow = w - NSW;
    const int col0 = PS * ps + 2 * SLICE * ow, slice0 = ps * NSW + 2 * ow;
    typename F::X xq[Cf::QLDS ? 1 : 4][NT];
    FragRegs pf;
    typedef typename std::conditional<sizeof(T) == 2, uint2, uint4>::type Raw4;   // four values as they lie
    Raw4 dox[2][4];
    auto request_out = [&](int i) {
      const int len = length(i);
      const int64_t row0 = static_cast<int64_t>(CH) * i;
      if constexpr (!Cf::QLDS) {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
#pragma unroll
          for (int q = 0; q < NT; ++q) {
            const int row = 16 * t + c, n = 32 * q + 8 * g;
            xq[t][q] = F::zero();
            if (row < len && n < p.N) xq[t][q] = F::load_cols(qp + (row0 + row) * p.q_sl + n, p.N - n);
          }
        }
        pf.request(p.pf + slot_head(i) * FRAG_PIECES);
      }
      if constexpr (BWD) {
#pragma unroll
        for (int z = 0; z < 2; ++z) {
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const int row = 16 * t + c, cc = col0 + SLICE * z + 4 * g;
            dox[z][t] = Raw4{};
            if (row < len && cc < p.P)
              dox[z][t] = *reinterpret_cast<const Raw4*>(static_cast<const T*>(p.dout) + (s0 + row0 + row) * hp + static_cast<int64_t>(h) * p.P + cc);
          }
        }
      }
    };
    uint4 us[2][NT][XP];
    f32x4_t uu[2][4];
    float in[4];
    auto take = [&](int i) {
#pragma unroll
      for (int z = 0; z < 2; ++z) {
#pragma unroll
        for (int q = 0; q < NT; ++q) {
#pragma unroll
          for (int t = 0; t < XP; ++t) us[z][q][t] = xs[(((2 * ow + z) * NT + q) * XP + t) * 64 + l];
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) uu[z][t] = xu[((2 * ow + z) * 4 + t) * 64 + l];
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) in[t] = p.scale * gbuf(i)[GATE_IN * CH + 16 * t + c];
    };
    auto out = [&](int i) {
      const int len = length(i);
      const int64_t sh = slot_head(i);
      typename F::S uf[2][2];
#pragma unroll
      for (int z = 0; z < 2; ++z) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float v[8];
          pair8(uu[z][2 * q], uu[z][2 * q + 1], v);
          uf[z][q] = F::split(v);
        }
      }
      if constexpr (BWD) {
        char* base = static_cast<char*>(p.s) + sh * p.rows * ND * 4;
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const int64_t r = col0 + SLICE * z + c;
          if (slice0 + z < p.nsl) {
#pragma unroll
            for (int q = 0; q < NT; ++q) {
#pragma unroll
              for (int t = 0; t < 2; ++t) {
                if constexpr (sizeof(T) == 2)
                  *reinterpret_cast<uint4*>(base + ((static_cast<int64_t>(t) * p.rows + r) * ND + 32 * q + 8 * g) * 2) = us[z][q][t];
                else
                  *reinterpret_cast<uint4*>(base + (r * ND + 32 * q + 8 * g + 4 * t) * 4) = us[z][q][t];
              }
            }
#pragma unroll
            for (int q = 0; q < 2; ++q) F::store(static_cast<T*>(p.u) + (sh * p.rows + r) * CH + 32 * q + 8 * g, F::hi(uf[z][q]));
          }
        }
      }
      const T* qt = qbuf(i);
      const uint4* pt = pbuf(i);
      // o, transposed: rows are value columns 4 g + r, columns are chunk rows 16 t + c
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        f32x4_t acc[2] = {zero4(), zero4()};
#pragma unroll
        for (int q = 0; q < NT; ++q) {
          typename F::X x;
          if constexpr (Cf::QLDS) x = F::load(qt + (16 * t + c) * LDN + 32 * q + 8 * g);
          else x = xq[t][q];
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            if constexpr (XP == 2) acc[z] = mma(F::from_pieces(us[z][q]), x, acc[z]);
            else acc[z] = mma(__builtin_bit_cast(typename F::X, us[z][q][0]), x, acc[z]);
          }
        }
        acc[0] *= in[t];
        acc[1] *= in[t];
#pragma unroll
        for (int ks = 0; ks <= (t >> 1); ++ks) {
          typename F::S sc;
          if constexpr (Cf::QLDS) sc = frag_at<T>(pt, lower_frag(t, ks));
          else sc = pf.get<T>(lower_frag(t, ks));
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            if constexpr (XP == 2) acc[z] = mma(uf[z][ks], sc, acc[z]);
            else acc[z] = mma(F::hi(uf[z][ks]), sc, acc[z]);
          }
        }
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          if constexpr (BWD) {
            const f32x4_t d = acc[z] * ssd::load4f<T>(reinterpret_cast<const T*>(&dox[z][t]));
            const float s = ssd::sum_kgroups((d[0] + d[1]) + (d[2] + d[3]));
            if (g == 0 && slice0 + z < p.nsl) p.oo[(sh * p.nsl + slice0 + z) * CH + 16 * t + c] = s;
          } else {
            const int cc = col0 + SLICE * z + 4 * g;
            if (16 * t + c < len && cc < p.P)
              ssd::store4f<T>(static_cast<T*>(p.o) + (s0 + static_cast<int64_t>(CH) * i + 16 * t + c) * hp + static_cast<int64_t>(h) * p.P + cc, acc[z]);
          }
        }
      }
    };
    request_out(0);
    for (int i = 0; i < nchunk; ++i) {
      if (i > 0) take(i - 1);
      __syncthreads();
      if (i > 0) {
        out(i - 1);
        request_out(i);
      }
      __syncthreads();
    }
    take(nchunk - 1);
    out(nchunk - 1);
    return;
  }

  // ---- staging waves
  const int ht = tid - 64 * (NSW + Cf::NOUT);
  const int pcols = min(PS, p.P - PS * ps);
  const T* kp = static_cast<const T*>(p.k) + row_offset(s0, p.L, p.k_sb, p.k_sl) + static_cast<int64_t>(grp) * p.N;
  const T* vp = static_cast<const T*>(p.v) + row_offset(s0, p.L, p.v_sb, p.v_sl) + static_cast<int64_t>(h) * p.P + PS * ps;
  constexpr int GI = (3 * CH + Cf::HT - 1) / Cf::HT;
  TileN tk, tq;
  TileP tv;
  Pieces<FRAG_PIECES, Cf::HT> tp;
  float tg[GI];
  auto request_state = [&](int i) {
    const int64_t row = static_cast<int64_t>(CH) * i;
    tk.load(kp + row * p.k_sl, p.k_sl, length(i), p.N, ht);
    tv.load(vp + row * p.v_sl, p.v_sl, length(i), pcols, ht);
#pragma unroll
    for (int k = 0; k < GI; ++k) tg[k] = ht + k * Cf::HT < 3 * CH ? p.gates[slot_head(i) * (GATES * CH) + ht + k * Cf::HT] : 0.f;
  };
  auto stage_state = [&](int i) {
    tk.store(kbuf(i), ht);
    tv.store(vbuf(i), ht);
#pragma unroll
    for (int k = 0; k < GI; ++k)
      if (ht + k * Cf::HT < 3 * CH) gbuf(i)[ht + k * Cf::HT] = tg[k];
  };
  auto request_scores = [&](int i) {
    if constexpr (Cf::QLDS) {
      tq.load(qp + static_cast<int64_t>(CH) * i * p.q_sl, p.q_sl, length(i), p.N, ht);
      tp.load(p.pf + slot_head(i) * FRAG_PIECES, ht);
    }
  };
  auto stage_scores = [&](int i) {
    if constexpr (Cf::QLDS) {
      tq.store(qbuf(i), ht);
      tp.store(pbuf(i), ht);
    }
  };
  request_state(0);
  request_scores(0);
  stage_state(0);
  if (nchunk > 1) request_state(1);
  for (int i = 0; i < nchunk; ++i) {
    __syncthreads();
    stage_scores(i);
    if (i + 1 < nchunk) {
      request_scores(i + 1);
      stage_state(i + 1);
      if (i + 2 < nchunk) request_state(i + 2);
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Launchers
// ---------------------------------------------------------------------------
template <typename K> int go(K kernel, dim3 grid, int threads, size_t lds, hipStream_t s, const Problem& p) {
  if (lds > 65536 && ssd::ensure_dynamic_lds(reinterpret_cast<const void*>(kernel), lds) != hipSuccess) return SSD_ERR_HIP;
  hipLaunchKernelGGL(kernel, grid, dim3(threads), lds, s, p);
  return hipGetLastError() == hipSuccess ? SSD_OK : SSD_ERR_HIP;
}

int launch_starts(const Problem& p, hipStream_t s) { return go(k_delta_starts, dim3(1), ST_THR, 0, s, p); }

template <typename T, int NT, bool BWD> int prep(const Problem& p, hipStream_t s) {
  return go(k_delta_prep<T, NT, BWD>, dim3(p.nslots, p.H), 256, PrepCfg<T, NT, BWD>::LDS, s, p);
}
template <typename T, int NT, bool BWD, int NSW> int walk_of(const Problem& p, hipStream_t s) {
  using Cf = WalkCfg<T, NT, BWD, NSW>;
  static_assert(Cf::LDS <= 160 * 1024, "LDS");
  return go(k_delta_walk<T, NT, BWD, NSW>, dim3(p.H * ((p.P + Cf::PS - 1) / Cf::PS), p.nseqs), Cf::THREADS, Cf::LDS, s, p);
}
// A CU holds one block (LDS).  Blocks of 32 value columns while they all fit the 256 CUs at once, of 64 above that
// (twice the columns on each CU for the same staging).
template <typename T, int NT, bool BWD> int walk(const Problem& p, hipStream_t s) {
  if constexpr (sizeof(T) == 2) {
    if (p.P > 32 && static_cast<int64_t>(p.H) * (p.rows / PAD) * p.nseqs > 256) return walk_of<T, NT, BWD, 4>(p, s);
  }
  return walk_of<T, NT, BWD, 2>(p, s);
}

int launch_prep(const Problem& p, int io, bool backward, hipStream_t s) {
  if (io == SSD_IO_BF16)
    return p.N <= 64 ? (backward ? prep<bf16_t, 2, true>(p, s) : prep<bf16_t, 2, false>(p, s))
                     : (backward ? prep<bf16_t, 4, true>(p, s) : prep<bf16_t, 4, false>(p, s));
  return p.N <= 64 ? (backward ? prep<float, 2, true>(p, s) : prep<float, 2, false>(p, s))
                   : (backward ? prep<float, 4, true>(p, s) : prep<float, 4, false>(p, s));
}
int launch_walk(const Problem& p, int io, bool backward, hipStream_t s) {
  if (io == SSD_IO_BF16)
    return p.N <= 64 ? (backward ? walk<bf16_t, 2, true>(p, s) : walk<bf16_t, 2, false>(p, s))
                     : (backward ? walk<bf16_t, 4, true>(p, s) : walk<bf16_t, 4, false>(p, s));
  return p.N <= 64 ? (backward ? walk<float, 2, true>(p, s) : walk<float, 2, false>(p, s))
                   : (backward ? walk<float, 4, true>(p, s) : walk<float, 4, false>(p, s));
}

}  // namespace delta
