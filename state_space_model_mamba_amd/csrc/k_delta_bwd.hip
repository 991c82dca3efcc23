// Backward of the gated delta rule: the walk back over a sequence's chunks
// and the chunks' gradients of q, k, g and beta.
//
// With dS the gradient of the state after a chunk, S the entering state, and
// N, G, e, u = beta e as in k_delta.hip:
//
//     du_j  = scale sum_{i>=j} G_ij (q_i . k_j) dout_i + exp(c_last - c_j) dS^T k_j
//     Du    = (I + diag(beta) N)^-T du                (gradient of u, later rows' e included)
//     dv    = beta Du,   dbeta_i = Du_i . e_i
//     dS_in = exp(c_last) dS + scale sum_i exp(c_i) q_i dout_i^T - sum_i exp(c_i) k_i dv_i^T
//     dq_i  = scale exp(c_i) S dout_i + sum_{j<=i} dP_ij k_j,      dP_ij = scale G_ij dout_i . u_j
//     dk_j  = sum_{i>=j} dP_ij q_i + sum_i (F_ij + F_ji) k_i - exp(c_j) S dv_j + exp(c_last - c_j) dS u_j,
//             F_ij = -G_ij dv_i . u_j  (j < i)
//
// The decay's gradient needs none of the products above once more: scaling
// every row of a chunk's decay history is the same as scaling v and o, so
//     dg_t - dg_{t+1} = dout_t . o_t - dv_t . v_t,
// and at a chunk's first row dg is <S, dS_in>.  dg is that inner product, in
// float32 at every chunk, less the row sums before t: no cancellation reaches
// further than 64 rows.
#include "delta_problem.h"
#include "delta_tiles.h"
#include "ssd_bwd.h"
#include "ssd_problem.h"

namespace delta {

// ---------------------------------------------------------------------------
// k_delta_rwalk: one sequence's chunks from the last to the first, for one
// head and 64 of its value columns, 16 per wave, the wave's columns of dS in
// registers throughout (as the forward walk holds S).
// ---------------------------------------------------------------------------
template <typename T, int NT> struct RwalkCfg {
  static constexpr int ND = 32 * NT;
  using TileN = Tile<T, CH, ND, 256>;
  using TileP = Tile<T, CH, PS, 256>;
  static constexpr size_t OFF_Q = sizeof(T) * TileN::LDS_ELEMS;
  static constexpr size_t OFF_V = 2 * OFF_Q;
  static constexpr size_t OFF_DO = OFF_V + sizeof(T) * TileP::LDS_ELEMS;
  static constexpr size_t OFF_T = OFF_DO + sizeof(T) * TileP::LDS_ELEMS;
  static constexpr size_t OFF_P = OFF_T + 16 * FRAG_PIECES;
  static constexpr size_t OFF_G = OFF_P + 16 * FRAG_PIECES;
  static constexpr size_t OFF_R = OFF_G + sizeof(float) * 3 * CH;
  static constexpr size_t LDS = OFF_R + sizeof(float) * (8 * CH + 4);
};

template <typename T, int NT> __global__ __launch_bounds__(256) void k_delta_rwalk(Problem p) {
  using Cf = RwalkCfg<T, NT>;
  using F = Fr<T>;
  using TileN = typename Cf::TileN;
  using TileP = typename Cf::TileP;
  constexpr int ND = Cf::ND, LDN = TileN::LD, LDP = TileP::LD;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  T* kt = reinterpret_cast<T*>(smem);
  T* qt = reinterpret_cast<T*>(smem + Cf::OFF_Q);
  T* vt = reinterpret_cast<T*>(smem + Cf::OFF_V);
  T* dot = reinterpret_cast<T*>(smem + Cf::OFF_DO);
  uint4* tfr = reinterpret_cast<uint4*>(smem + Cf::OFF_T);
  uint4* pfr = reinterpret_cast<uint4*>(smem + Cf::OFF_P);
  float* gs = reinterpret_cast<float*>(smem + Cf::OFF_G);
  float* red = reinterpret_cast<float*>(smem + Cf::OFF_R);   // [4 waves][64]: dv . v, then Du . e; then <S, dS>

  const int h = static_cast<int>(blockIdx.x) / p.np, ps = static_cast<int>(blockIdx.x) % p.np;
  const int seq = static_cast<int>(blockIdx.y), grp = h / p.hpg;
  const int s0 = seq_start(p, seq), s1 = seq_start(p, seq + 1);
  const int nchunk = (s1 - s0 + CH - 1) / CH, slot0 = slot_base(s0, seq);
  const int tid = static_cast<int>(threadIdx.x), l = tid & 63, g = l >> 4, c = l & 15, w = ssd::wave_id_s();
  const int col = PS * ps + 16 * w + c;
  const int pcols = min(PS, p.P - PS * ps);
  const int64_t state_at = ((static_cast<int64_t>(seq) * p.H + h) * p.P + col) * p.N;

  f32x4_t S[2 * NT];   // dS
#pragma unroll
  for (int j = 0; j < 2 * NT; ++j) {
    const int n = pair_col(j) + 8 * g;
    S[j] = zero4();
    if (p.dfinal && col < p.P && n < p.N) S[j] = *reinterpret_cast<const f32x4_t*>(p.dfinal + state_at + n);
  }

  const T* kp = static_cast<const T*>(p.k);
  const T* qp = static_cast<const T*>(p.q);
  const T* vp = static_cast<const T*>(p.v);
  if (nchunk) {
    kp += row_offset(s0, p.L, p.k_sb, p.k_sl) + static_cast<int64_t>(grp) * p.N;
    qp += row_offset(s0, p.L, p.q_sb, p.q_sl) + static_cast<int64_t>(grp) * p.N;
    vp += row_offset(s0, p.L, p.v_sb, p.v_sl) + static_cast<int64_t>(h) * p.P + PS * ps;
  }
  const int64_t hp = static_cast<int64_t>(p.H) * p.P;
  TileN tk, tq;
  TileP tv, td;
  Pieces<FRAG_PIECES, 256> tt, tp;
  uint4 te[4];
  float tg = 0.f;
  auto request = [&](int i) {
    const int len = min(CH, s1 - s0 - CH * i);
    const int64_t sh = static_cast<int64_t>(slot0 + i) * p.H + h;
    const int64_t row = static_cast<int64_t>(CH) * i;
    tk.load(kp + row * p.k_sl, p.k_sl, len, p.N);
    tq.load(qp + row * p.q_sl, p.q_sl, len, p.N);
    tv.load(vp + row * p.v_sl, p.v_sl, len, pcols);
    td.load(static_cast<const T*>(p.dout) + (s0 + row) * hp + static_cast<int64_t>(h) * p.P + PS * ps, hp, len, pcols);
    tt.load(p.ttf + sh * FRAG_PIECES);
    tp.load(p.ptf + sh * FRAG_PIECES);
#pragma unroll
    for (int t = 0; t < 4; ++t) te[t] = p.e[((((sh * p.np + ps) * 4 + w) * 4) + t) * 64 + l];
    if (tid < 3 * CH) tg = p.gates[sh * (GATES * CH) + tid];
  };
  if (nchunk) request(nchunk - 1);

  for (int i = nchunk - 1; i >= 0; --i) {
    const int len = min(CH, s1 - s0 - CH * i);
    const int64_t sh = static_cast<int64_t>(slot0 + i) * p.H + h;
    const int64_t rows = static_cast<int64_t>(p.np) * PS;
    tk.store(kt);
    tq.store(qt);
    tv.store(vt);
    td.store(dot);
    tt.store(tfr);
    tp.store(pfr);
    f32x4_t e[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) e[t] = __builtin_bit_cast(f32x4_t, te[t]);
    if (tid < 3 * CH) gs[tid] = tg;
    __syncthreads();
    if (i > 0) request(i - 1);

    typename F::S sf[NT];
#pragma unroll
    for (int q = 0; q < NT; ++q) {
      float v[8];
      pair8(S[2 * q], S[2 * q + 1], v);
      sf[q] = F::split(v);
      F::store(static_cast<T*>(p.ds) + (sh * rows + col) * ND + 32 * q + 8 * g, F::hi(sf[q]));
    }
    typename F::X xd[2];   // dout: rows 32 ks + 8 g + e of this lane's column
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) xd[ks] = F::load_tr(dot + 16 * w, LDP, 32 * ks + 8 * g);
    f32x4_t x[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      f32x4_t acc = zero4();
#pragma unroll
      for (int q = 0; q < NT; ++q) acc = mma(F::load(kt + perm_row(t, c) * LDN + 32 * q + 8 * g), sf[q], acc);
      acc *= *reinterpret_cast<const f32x4_t*>(gs + GATE_OUT * CH + pair_col(t) + 8 * g);
#pragma unroll
      for (int ks = (t >> 1); ks < 2; ++ks) acc = mma(load_frag<T>(pfr, upper_frag(t, ks)), xd[ks], acc);
      x[t] = acc;
    }
    typename F::S f2[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      float v[8];
      pair8(x[2 * q], x[2 * q + 1], v);
      f2[q] = F::split(v);
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      f32x4_t acc = zero4();
#pragma unroll
      for (int ks = (t >> 1); ks < 2; ++ks) acc = mma(load_frag<T>(tfr, upper_frag(t, ks)), f2[ks], acc);
      const int row = pair_col(t) + 8 * g;
      x[t] = acc * *reinterpret_cast<const f32x4_t*>(gs + GATE_BETA * CH + row);   // dv
      const f32x4_t v = F::load4_tr(vt + 16 * w, LDP, row);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float dvv = ssd::sum16(x[t][r] * v[r]), due = ssd::sum16(acc[r] * e[t][r]);
        if (c == 0) {
          red[w * CH + row + r] = dvv;
          red[(4 + w) * CH + row + r] = due;
        }
        if (row + r < len && col < p.P)
          static_cast<T*>(p.dv)[(s0 + static_cast<int64_t>(CH) * i + row + r) * hp + static_cast<int64_t>(h) * p.P + col] = ssd::Elem<T>::from_f(x[t][r]);
      }
    }
    // dS <- exp(c_last) dS + q^T (scale exp(c) dout) - k^T (exp(c) dv)
    typename F::S fd[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const f32x4_t i0 = *reinterpret_cast<const f32x4_t*>(gs + GATE_IN * CH + 32 * q + 8 * g);
      const f32x4_t i1 = *reinterpret_cast<const f32x4_t*>(gs + GATE_IN * CH + 32 * q + 8 * g + 4);
      float v[8], d[8];
      pair8(-i0 * x[2 * q], -i1 * x[2 * q + 1], v);
      f2[q] = F::split(v);
      F::floats(xd[q], d);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        d[r] *= p.scale * i0[r];
        d[4 + r] *= p.scale * i1[r];
      }
      fd[q] = F::split(d);
    }
    const float last = gs[GATE_IN * CH + CH - 1];
#pragma unroll
    for (int j = 0; j < 2 * NT; ++j) {
      f32x4_t acc = last * S[j];
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        acc = mma(F::template load_tr<8>(qt + pair_col(j), LDN, 32 * ks + 8 * g), fd[ks], acc);
        acc = mma(F::template load_tr<8>(kt + pair_col(j), LDN, 32 * ks + 8 * g), f2[ks], acc);
      }
      S[j] = acc;
    }
    // <entering state, its gradient>
    float phi = 0.f;
    const char* sb = static_cast<const char*>(p.s) + sh * rows * ND * 4;
#pragma unroll
    for (int q = 0; q < NT; ++q) {
      uint4 u[2];
      if constexpr (sizeof(T) == 2) {
        u[0] = *reinterpret_cast<const uint4*>(sb + (static_cast<int64_t>(col) * ND + 32 * q + 8 * g) * 2);
        u[1] = *reinterpret_cast<const uint4*>(sb + ((rows + col) * ND + 32 * q + 8 * g) * 2);
      } else {
        const uint4* d = reinterpret_cast<const uint4*>(sb + (static_cast<int64_t>(col) * ND + 32 * q + 8 * g) * 4);
        u[0] = d[0];
        u[1] = d[1];
      }
      float v[8];
      F::floats(F::from_pieces(u), v);
#pragma unroll
      for (int r = 0; r < 4; ++r) phi += v[r] * S[2 * q][r] + v[4 + r] * S[2 * q + 1][r];
    }
    phi = ssd::wave_sum(phi);
    if (l == 0) red[8 * CH + w] = phi;
    __syncthreads();
    const int64_t at = (sh * p.np + ps) * CH;
    if (tid < CH) {
      p.dd[at + tid] = p.oo[at + tid] - (((red[tid] + red[CH + tid]) + red[2 * CH + tid]) + red[3 * CH + tid]);
      if (tid == 0) p.phi[sh * p.np + ps] = ((red[8 * CH] + red[8 * CH + 1]) + red[8 * CH + 2]) + red[8 * CH + 3];
    } else if (tid < 2 * CH) {
      const float* r = red + 4 * CH + tid - CH;
      p.be[at + tid - CH] = ((r[0] + r[CH]) + r[2 * CH]) + r[3 * CH];
    }
  }

  if (p.dinit && col < p.P) {
#pragma unroll
    for (int j = 0; j < 2 * NT; ++j) {
      const int n = pair_col(j) + 8 * g;
      if (n < p.N) *reinterpret_cast<f32x4_t*>(p.dinit + state_at + n) = S[j];
    }
  }
}

// ---------------------------------------------------------------------------
// k_delta_grad: dq, dk, dg and dbeta of one chunk and group, its heads one
// after the other (dq and dk are sums over them, taken in registers in head
// order).  Eight waves: 16 rows of the chunk times half of the N columns each.
// All products end in the io type, so every operand is a single term.
// ---------------------------------------------------------------------------
constexpr int GTHR = 512;

template <typename T, int NT> struct GradCfg {
  static constexpr int ND = 32 * NT;
  static constexpr int PSL = sizeof(T) == 2 ? 64 : 32;   // value columns staged at once
  using TileN = Tile<T, CH, ND, GTHR>;
  using TileP = Tile<T, CH, PSL, GTHR>;    // dout, dv
  using TileU = Tile<T, PSL, CH, GTHR>;    // u, a value column per row
  using TileS = Tile<T, PSL, ND, GTHR>;    // S, dS, a value column per row
  using TileM = Tile<T, CH, CH, GTHR>;     // dP, F + F^T (over the tiles above)
  static constexpr size_t OFF_Q = sizeof(T) * TileN::LDS_ELEMS;
  static constexpr size_t OFF_DO = 2 * OFF_Q;
  static constexpr size_t OFF_DV = OFF_DO + sizeof(T) * TileP::LDS_ELEMS;
  static constexpr size_t OFF_U = OFF_DV + sizeof(T) * TileP::LDS_ELEMS;
  static constexpr size_t OFF_S = OFF_U + sizeof(T) * TileU::LDS_ELEMS;
  static constexpr size_t OFF_DS = OFF_S + sizeof(T) * TileS::LDS_ELEMS;
  static constexpr size_t END1 = OFF_DS + sizeof(T) * TileS::LDS_ELEMS;
  static constexpr size_t OFF_F = OFF_DO + sizeof(T) * TileM::LDS_ELEMS;
  static constexpr size_t END2 = OFF_F + sizeof(T) * TileM::LDS_ELEMS;
  static constexpr size_t OFF_G = END1 > END2 ? END1 : END2;
  static constexpr size_t LDS = OFF_G + sizeof(float) * GATES * CH;
};

template <typename T, int NT> __global__ __launch_bounds__(GTHR) void k_delta_grad(Problem p) {
  using Cf = GradCfg<T, NT>;
  using F = Fr<T>;
  constexpr int ND = Cf::ND, LDN = Cf::TileN::LD, LDP = Cf::TileP::LD, LDU = Cf::TileU::LD, LDS_ = Cf::TileS::LD, LDMT = Cf::TileM::LD;
  constexpr int PSL = Cf::PSL;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  T* kt = reinterpret_cast<T*>(smem);
  T* qt = reinterpret_cast<T*>(smem + Cf::OFF_Q);
  T* dot = reinterpret_cast<T*>(smem + Cf::OFF_DO);
  T* dvt = reinterpret_cast<T*>(smem + Cf::OFF_DV);
  T* ut = reinterpret_cast<T*>(smem + Cf::OFF_U);
  T* st = reinterpret_cast<T*>(smem + Cf::OFF_S);
  T* dst = reinterpret_cast<T*>(smem + Cf::OFF_DS);
  T* dpm = reinterpret_cast<T*>(smem + Cf::OFF_DO);
  T* fm = reinterpret_cast<T*>(smem + Cf::OFF_F);
  float* gs = reinterpret_cast<float*>(smem + Cf::OFF_G);

  const int slot = static_cast<int>(blockIdx.x), grp = static_cast<int>(blockIdx.y);
  const Chunk ch = chunk_of(p, slot);
  if (ch.len == 0) return;
  const int tid = static_cast<int>(threadIdx.x), l = tid & 63, g = l >> 4, c = l & 15, w = ssd::wave_id_s();
  const int rt = w & 3, half = w >> 2, row = 16 * rt + c;
  const int64_t hp = static_cast<int64_t>(p.H) * p.P, rows = static_cast<int64_t>(p.np) * PS;
  {
    typename Cf::TileN tk, tq;
    tk.load(static_cast<const T*>(p.k) + row_offset(ch.row, p.L, p.k_sb, p.k_sl) + static_cast<int64_t>(grp) * p.N, p.k_sl, ch.len, p.N);
    tq.load(static_cast<const T*>(p.q) + row_offset(ch.row, p.L, p.q_sb, p.q_sl) + static_cast<int64_t>(grp) * p.N, p.q_sl, ch.len, p.N);
    tk.store(kt);
    tq.store(qt);
  }
  f32x4_t dqa[NT], dka[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) dqa[t] = dka[t] = zero4();

  for (int hh = 0; hh < p.hpg; ++hh) {
    const int h = grp * p.hpg + hh;
    const int64_t sh = static_cast<int64_t>(slot) * p.H + h;
    f32x4_t x1[NT], x2[NT], x3[NT], m1[2], m2[2];
#pragma unroll
    for (int t = 0; t < NT; ++t) x1[t] = x2[t] = x3[t] = zero4();
    m1[0] = m1[1] = m2[0] = m2[1] = zero4();
    for (int p0 = 0; p0 < p.P; p0 += PSL) {
      const int pcols = min(PSL, p.P - p0);
      typename Cf::TileP td, tv;
      typename Cf::TileU tu;
      typename Cf::TileS ts, tds;
      const int64_t at = static_cast<int64_t>(ch.row) * hp + static_cast<int64_t>(h) * p.P + p0;
      td.load(static_cast<const T*>(p.dout) + at, hp, ch.len, pcols);
      tv.load(static_cast<const T*>(p.dv) + at, hp, ch.len, pcols);
      tu.load(static_cast<const T*>(p.u) + (sh * rows + p0) * CH, CH, PSL, CH);
      ts.load(reinterpret_cast<const T*>(static_cast<const char*>(p.s) + sh * rows * ND * 4) + static_cast<int64_t>(p0) * ND, ND, PSL, ND);
      tds.load(static_cast<const T*>(p.ds) + (sh * rows + p0) * ND, ND, PSL, ND);
      const float tg = tid < GATES * CH ? p.gates[sh * (GATES * CH) + tid] : 0.f;
      __syncthreads();   // the previous head's last products are done
      td.store(dot);
      tv.store(dvt);
      tu.store(ut);
      ts.store(st);
      tds.store(dst);
      if (tid < GATES * CH) gs[tid] = tg;
      __syncthreads();
#pragma unroll
      for (int ks = 0; ks < PSL / 32; ++ks) {
        const typename F::X xdo = F::load(dot + row * LDP + 32 * ks + 8 * g), xdv = F::load(dvt + row * LDP + 32 * ks + 8 * g);
        const typename F::X xu = F::load_tr(ut + 16 * rt, LDU, 32 * ks + 8 * g);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const int n0 = 16 * (half * NT + t);
          const typename F::X xs = F::load_tr(st + n0, LDS_, 32 * ks + 8 * g), xds = F::load_tr(dst + n0, LDS_, 32 * ks + 8 * g);
          x1[t] = mma(xs, xdo, x1[t]);
          x2[t] = mma(xs, xdv, x2[t]);
          x3[t] = mma(xds, xu, x3[t]);
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int jt = 2 * half + t;
          if (jt <= rt) {
            const typename F::X xj = F::load_tr(ut + 16 * jt, LDU, 32 * ks + 8 * g);
            m1[t] = mma(xj, xdo, m1[t]);
            m2[t] = mma(xj, xdv, m2[t]);
          }
        }
      }
    }
    const float in = gs[GATE_IN * CH + row], out = gs[GATE_OUT * CH + row];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      dqa[t] += (p.scale * in) * x1[t];
      dka[t] += out * x3[t] - in * x2[t];
    }
    __syncthreads();
    const float ci = gs[GATE_C * CH + row], cl = gs[GATE_CLO * CH + row];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int jt = 2 * half + t;
      f32x4_t dp = zero4();
      if (jt <= rt) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int j = 16 * jt + 4 * g + r;
          const float dec = expf((ci - gs[GATE_C * CH + j]) + (cl - gs[GATE_CLO * CH + j]));
          if (j <= row) dp[r] = p.scale * (dec * m1[t][r]);
          if (j < row) {
            const T f = ssd::Elem<T>::from_f(-dec * m2[t][r]);
            fm[row * LDMT + j] = f;
            fm[j * LDMT + row] = f;
          } else if (j == row) {
            fm[row * LDMT + row] = ssd::Elem<T>::from_f(0.f);
          }
        }
      }
      ssd::store4f<T>(dpm + row * LDMT + 16 * jt + 4 * g, dp);
    }
    __syncthreads();
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const typename F::X xp = F::load(dpm + row * LDMT + 32 * ks + 8 * g), xf = F::load(fm + row * LDMT + 32 * ks + 8 * g);
      const typename F::X xpt = F::load_tr(dpm + 16 * rt, LDMT, 32 * ks + 8 * g);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int n0 = 16 * (half * NT + t);
        const typename F::X xk = F::load_tr(kt + n0, LDN, 32 * ks + 8 * g), xq = F::load_tr(qt + n0, LDN, 32 * ks + 8 * g);
        dqa[t] = mma(xk, xp, dqa[t]);
        dka[t] = mma(xq, xpt, dka[t]);
        dka[t] = mma(xk, xf, dka[t]);
      }
    }
    // the gates' gradients: sums over the blocks of value columns in order, dg by a scan over the rows
    if (w == 0) {
      float d = 0.f, b = 0.f, phi = 0.f;
      for (int s = 0; s < p.np; ++s) {
        d += p.dd[(sh * p.np + s) * CH + l];
        b += p.be[(sh * p.np + s) * CH + l];
        phi += p.phi[sh * p.np + s];
      }
      float run = d;
#pragma unroll
      for (int k = 1; k < 64; k <<= 1) {
        const float o = __shfl_up(run, k);
        if (l >= k) run += o;
      }
      if (l < ch.len) {
        const int64_t at = (static_cast<int64_t>(ch.row) + l) * p.H + h;
        p.dg[at] = phi - (run - d);
        p.dbeta[at] = b;
      }
    }
  }
  if (row < ch.len) {
    const int64_t at = ((static_cast<int64_t>(ch.row) + row) * p.G + grp) * p.N;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int n = 16 * (half * NT + t) + 4 * g;
      if (n < p.N) {
        ssd::store4f<T>(static_cast<T*>(p.dq) + at + n, dqa[t]);
        ssd::store4f<T>(static_cast<T*>(p.dk) + at + n, dka[t]);
      }
    }
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

template <typename T, int NT> int rwalk(const Problem& p, hipStream_t s) {
  static_assert(RwalkCfg<T, NT>::LDS <= 160 * 1024, "LDS");
  return go(k_delta_rwalk<T, NT>, dim3(p.H * p.np, p.nseqs), 256, RwalkCfg<T, NT>::LDS, s, p);
}
template <typename T, int NT> int grad(const Problem& p, hipStream_t s) {
  static_assert(GradCfg<T, NT>::LDS <= 160 * 1024, "LDS");
  return go(k_delta_grad<T, NT>, dim3(p.nslots, p.G), GTHR, GradCfg<T, NT>::LDS, s, p);
}

int launch_rwalk(const Problem& p, int io, hipStream_t s) {
  if (io == SSD_IO_BF16) return p.N <= 64 ? rwalk<bf16_t, 2>(p, s) : rwalk<bf16_t, 4>(p, s);
  return p.N <= 64 ? rwalk<float, 2>(p, s) : rwalk<float, 4>(p, s);
}
int launch_grad(const Problem& p, int io, hipStream_t s) {
  if (io == SSD_IO_BF16) return p.N <= 64 ? grad<bf16_t, 2>(p, s) : grad<bf16_t, 4>(p, s);
  return p.N <= 64 ? grad<float, 2>(p, s) : grad<float, 4>(p, s);
}

}  // namespace delta
