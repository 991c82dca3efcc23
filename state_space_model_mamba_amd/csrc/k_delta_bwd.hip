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
// The decay of row t scales all that passes from before t to t and after:
//     dg_t = sum_{i>=t>j} M_ij + sum_{i>=t} a_i + sum_{j<t} b_j + exp(c_last) <S, dS>,
//     M_ij = dP_ij (q_i . k_j) + F_ij (k_i . k_j)                         (within the chunk)
//     a_i  = exp(c_i) (scale q_i . S dout_i - k_i . S dv_i)               (from the entering state)
//     b_j  = exp(c_last - c_j) k_j . dS u_j                               (to the state after)
// Every term holds exp(g_t), so dg_t keeps its bits however strong the decay.  (dg_t - dg_{t+1} = dout_t . o_t -
// dv_t . v_t is shorter, but a difference of terms that do not get smaller with exp(g_t): at g = -8 dg was 2e-2 off
// with bf16 io, at -30 nothing of it was left.)
#include "delta_problem.h"
#include "delta_tiles.h"
#include "ssd_bwd.h"
#include "ssd_problem.h"

namespace delta {

// ---------------------------------------------------------------------------
// k_delta_rwalk: one sequence's chunks from the last to the first, for one
// head and PS of its value columns, with roles as in the forward walk: a state
// wave keeps 16 columns of dS in registers and runs the sequential part,
//     k dS -> du -> Du -> dS,
// while beside the two of them
//   * one wave forms ahead what does not need dS, for chunk i - 1: the scores'
//     part of du, and q^T dout,
//   * a wave each follows behind with what Du gives, for chunk i + 1: dv, the
//     row sums for dbeta, and the stores,
//   * two waves stage the coming chunks' rows in LDS.
// Bound by memory: a chunk and head reads the residuals (16 KB), matrices (24 KB)
// and dout (8 KB) and writes dS and dv (48 KB, in two terms), 16384 rows of 128
// heads of 64 x 128 in 0.89 ms, 3.6 TB/s; in one kind of wave alone it took 2.7 ms.
// ---------------------------------------------------------------------------
template <typename T, int NT> struct RwalkCfg {
  static constexpr int ND = 32 * NT, NSW = 2, PS = SLICE * NSW, NST = 2, HT = 64 * NST, THREADS = 64 * (2 * NSW + 1 + NST);
  using K = ChunkRows<T, NT, HT>;
  using TileN = typename K::TileT;
  using TileP = Tile<T, CH, PS, HT>;
  static constexpr size_t N_BYTES = sizeof(T) * TileN::LDS_ELEMS, P_BYTES = sizeof(T) * TileP::LDS_ELEMS;
  // k and q twice, staged while the others work; 512-byte rows once, staged between the chunks
  static constexpr int KBUF = sizeof(T) * ND <= 256 ? 2 : 1;
  static constexpr size_t OFF_Q = KBUF * N_BYTES;
  static constexpr size_t OFF_DO = 2 * OFF_Q;
  static constexpr size_t OFF_V = OFF_DO + 2 * P_BYTES;      // dv on its way to its rows
  static constexpr size_t OFF_D0 = OFF_V + P_BYTES;          // scores^T dout
  static constexpr size_t OFF_Q0 = OFF_D0 + 16 * 64 * NSW * 4;
  static constexpr size_t OFF_DU = OFF_Q0 + KBUF * 16 * 64 * NSW * 2 * NT;   // q^T dout, twice as k
  static constexpr size_t OFF_XS = OFF_DU + 16 * 64 * NSW * 4;
  static constexpr size_t OFF_G = OFF_XS + 16 * 64 * NSW * NT * 2;
  static constexpr size_t LDS = OFF_G + 4 * sizeof(float) * RWALK_GATES * CH;   // the gates of four chunks
};

template <typename T, int NT> __global__ __launch_bounds__(64 * 7) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_delta_rwalk(Problem p) {
  using Cf = RwalkCfg<T, NT>;
  using F = Fr<T>;
  using TileN = typename Cf::TileN;
  using TileP = typename Cf::TileP;
  constexpr int LDP = TileP::LD, NSW = Cf::NSW, PS = Cf::PS, KB = Cf::KBUF - 1;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  auto kbuf = [&](int i) { return reinterpret_cast<T*>(smem + (i & KB) * Cf::N_BYTES); };
  auto qbuf = [&](int i) { return reinterpret_cast<T*>(smem + Cf::OFF_Q + (i & KB) * Cf::N_BYTES); };
  auto dobuf = [&](int i) { return reinterpret_cast<T*>(smem + Cf::OFF_DO + (i & 1) * Cf::P_BYTES); };
  auto gbuf = [&](int i) { return reinterpret_cast<float*>(smem + Cf::OFF_G) + (i & 3) * RWALK_GATES * CH; };
  f32x4_t* xd0 = reinterpret_cast<f32x4_t*>(smem + Cf::OFF_D0);   // [wave][t][lane]
  auto xq0 = [&](int i) { return reinterpret_cast<f32x4_t*>(smem + Cf::OFF_Q0) + (i & KB) * 64 * NSW * 2 * NT; };   // [wave][j][lane]
  f32x4_t* xdu = reinterpret_cast<f32x4_t*>(smem + Cf::OFF_DU);   // [wave][t][lane]
  uint4* xs = reinterpret_cast<uint4*>(smem + Cf::OFF_XS);        // [wave][q][term][lane]

  const int np = (p.P + PS - 1) / PS;
  const Place at_block = place_of(p, np);
  const int h = at_block.h, ps = at_block.ps, seq = at_block.seq, grp = h / p.hpg;
  const int s0 = seq_start(p, seq), s1 = seq_start(p, seq + 1);
  const int nchunk = (s1 - s0 + CH - 1) / CH, slot0 = slot_base(s0, seq), last = nchunk - 1;
  const int tid = static_cast<int>(threadIdx.x), l = tid & 63, g = l >> 4, c = l & 15, w = ssd::wave_id_s();
  auto slot_head = [&](int i) { return static_cast<int64_t>(slot0 + i) * p.H + h; };
  auto length = [&](int i) { return min(CH, s1 - s0 - CH * i); };

  if (w < NSW) {
    // ---- state waves
    const int col = PS * ps + SLICE * w + c;
    const int64_t state_at = ((static_cast<int64_t>(seq) * p.H + h) * p.P + col) * p.N;
    f32x4_t S[2 * NT];   // dS
#pragma unroll
    for (int j = 0; j < 2 * NT; ++j) {
      const int n = pair_col(j) + 8 * g;
      S[j] = zero4();
      if (p.dfinal && col < p.P && n < p.N) S[j] = *reinterpret_cast<const f32x4_t*>(p.dfinal + state_at + n);
    }
    if (nchunk) {
      typename F::S sf[NT];
      auto split_state = [&](int q) {
        float v[8];
        pair8(S[2 * q], S[2 * q + 1], v);
        sf[q] = F::split(v);
      };
#pragma unroll
      for (int q = 0; q < NT; ++q) split_state(q);
      FragRegs tf;
      tf.request(p.ttf + slot_head(last) * FRAG_PIECES);
      __syncthreads();
      for (int i = last; i >= 0; --i) {
        const T* kt = kbuf(i);
        const float* gs = gbuf(i);
        auto gate = [&](int which, int row) { return *reinterpret_cast<const f32x4_t*>(gs + which * CH + row); };
        __syncthreads();   // second barrier of the chunk before (the first time: of what came ahead)
        f32x4_t d0[4], q0[2 * NT], out[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          d0[t] = xd0[(w * 4 + t) * 64 + l];
          out[t] = gate(GATE_OUT, pair_col(t) + 8 * g);
        }
        const float dec = gs[GATE_IN * CH + CH - 1];
        if constexpr (KB == 0) {
#pragma unroll
          for (int j = 0; j < 2 * NT; ++j) q0[j] = xq0(i)[(w * 2 * NT + j) * 64 + l];
        }
        typename F::X kf[4][NT];
        if constexpr (KB != 0) {   // k's rows are staged: on their way while the others take what they need
#pragma unroll
          for (int q = 0; q < NT; ++q) {
#pragma unroll
            for (int t = 0; t < 4; ++t) kf[t][q] = Cf::K::rows(kt, t, q);
          }
        }
        __syncthreads();
        if constexpr (KB == 0) {
#pragma unroll
          for (int q = 0; q < NT; ++q) {
#pragma unroll
            for (int t = 0; t < 4; ++t) kf[t][q] = Cf::K::rows(kt, t, q);
          }
        }
#pragma unroll
        for (int q = 0; q < NT; ++q) {
          uint4 u[2];
          F::pieces(sf[q], u);
          xs[((w * NT + q) * 2 + 0) * 64 + l] = u[0];
          xs[((w * NT + q) * 2 + 1) * 64 + l] = u[1];
        }
        f32x4_t x[4];
        typename F::X kc[2 * NT][2];
#pragma unroll
        for (int t = 0; t < 4; ++t) x[t] = zero4();
#pragma unroll
        for (int q = 0; q < NT; ++q) {
#pragma unroll
          for (int term = 0; term < 2; ++term) {
#pragma unroll
            for (int t = 0; t < 4; ++t) x[t] = mma_term(kf[t][q], sf[q], x[t], term);
          }
          // beside it the first part of the next dS, and k's columns for the last product
#pragma unroll
          for (int j = 2 * q; j < 2 * q + 2; ++j) {
            if constexpr (KB != 0) q0[j] = xq0(i)[(w * 2 * NT + j) * 64 + l];
            S[j] = dec * S[j] + q0[j];
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) kc[j][ks] = Cf::K::cols(kt, j, ks);
          }
        }
        f32x4_t bi[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          x[t] = x[t] * out[t] + d0[t];
          bi[t] = gate(GATE_BI, pair_col(t) + 8 * g);
        }
        // Du = du + (T^T - I) du
        typename F::S f2[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float v[8];
          pair8(x[2 * q], x[2 * q + 1], v);
          f2[q] = F::split(v);
        }
#pragma unroll
        for (int ks = 1; ks >= 0; --ks) {
#pragma unroll
          for (int term = 0; term < 3; ++term) {
#pragma unroll
            for (int t = 0; t < 2 * ks + 2; ++t) x[t] = mma_term(tf.get<T>(upper_frag(t, ks)), f2[ks], x[t], term);
          }
        }
        // dS <- exp(c_last) dS + q^T (scale exp(c) dout) - k^T (exp(c) beta Du)
        // (in the forward walk's order)
        const uint4* tnext = p.ttf + slot_head(i > 0 ? i - 1 : i) * FRAG_PIECES + l;
        auto correction = [&](int q) {
          xdu[(w * 4 + 2 * q) * 64 + l] = x[2 * q];
          xdu[(w * 4 + 2 * q + 1) * 64 + l] = x[2 * q + 1];
          float v[8];
          pair8(x[2 * q] * bi[2 * q], x[2 * q + 1] * bi[2 * q + 1], v);
          return F::split3(v);
        };
        const typename F::S3 fa = correction(0);
#pragma unroll
        for (int term = 0; term < 3; ++term) {
#pragma unroll
          for (int j = 0; j < 2 * NT; ++j) S[j] = mma_term(kc[j][0], fa, S[j], term);
          tf.u[2 * term] = tnext[2 * term * 64];
          tf.u[2 * term + 1] = tnext[(2 * term + 1) * 64];
        }
        const typename F::S3 fb = correction(1);
#pragma unroll
        for (int j0 = 0; j0 < 2 * NT; j0 += 4) {
#pragma unroll
          for (int term = 0; term < 3; ++term) {
#pragma unroll
            for (int j = j0; j < j0 + 4; ++j) S[j] = mma_term(kc[j][1], fb, S[j], term);
            if (j0 == 0) {
              tf.u[6 + 2 * term] = tnext[(6 + 2 * term) * 64];
              tf.u[7 + 2 * term] = tnext[(7 + 2 * term) * 64];
            }
          }
          split_state(j0 / 2);
          split_state(j0 / 2 + 1);
        }
      }
      __syncthreads();
    }
    if (p.dinit && col < p.P) {
#pragma unroll
      for (int j = 0; j < 2 * NT; ++j) {
        const int n = pair_col(j) + 8 * g;
        if (n < p.N) *reinterpret_cast<f32x4_t*>(p.dinit + state_at + n) = S[j];
      }
    }
    return;
  }
  if (nchunk == 0) return;
  const int64_t hp = static_cast<int64_t>(p.H) * p.P;

  if (w == NSW) {
    // ---- the wave ahead
    FragRegs pf;
    auto ahead = [&](int i) {
      const T *dot = dobuf(i), *qt = qbuf(i);
      const float* gs = gbuf(i);
      typename F::X xd[NSW][2];   // dout: rows 32 ks + 8 g + e of column c of each slice
      typename F::S3 fd[NSW][2];
#pragma unroll
      for (int z = 0; z < NSW; ++z) {
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) xd[z][ks] = F::load_tr(dot + SLICE * z, LDP, 32 * ks + 8 * g);
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        f32x4_t acc[NSW];
#pragma unroll
        for (int z = 0; z < NSW; ++z) acc[z] = zero4();
#pragma unroll
        for (int ks = (t >> 1); ks < 2; ++ks) {
#pragma unroll
          for (int z = 0; z < NSW; ++z) acc[z] = mma(pf.get<T>(upper_frag(t, ks)), xd[z][ks], acc[z]);
        }
#pragma unroll
        for (int z = 0; z < NSW; ++z) xd0[(z * 4 + t) * 64 + l] = acc[z];
      }
      if (i > 0) pf.request(p.ptf + slot_head(i - 1) * FRAG_PIECES);
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const f32x4_t i0 = p.scale * *reinterpret_cast<const f32x4_t*>(gs + GATE_IN * CH + 32 * ks + 8 * g);
        const f32x4_t i1 = p.scale * *reinterpret_cast<const f32x4_t*>(gs + GATE_IN * CH + 32 * ks + 8 * g + 4);
#pragma unroll
        for (int z = 0; z < NSW; ++z) {
          float d[8];
          F::floats(xd[z][ks], d);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            d[r] *= i0[r];
            d[4 + r] *= i1[r];
          }
          fd[z][ks] = F::split3(d);
        }
      }
#pragma unroll
      for (int j = 0; j < 2 * NT; ++j) {
        f32x4_t acc[NSW];
#pragma unroll
        for (int z = 0; z < NSW; ++z) acc[z] = zero4();
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          const typename F::X xq = Cf::K::cols(qt, j, ks);
#pragma unroll
          for (int z = 0; z < NSW; ++z) acc[z] = mma(xq, fd[z][ks], acc[z]);
        }
#pragma unroll
        for (int z = 0; z < NSW; ++z) xq0(i)[(z * 2 * NT + j) * 64 + l] = acc[z];
      }
    };
    pf.request(p.ptf + slot_head(last) * FRAG_PIECES);
    __syncthreads();
    ahead(last);
    __syncthreads();
    for (int i = last; i >= 0; --i) {
      __syncthreads();
      if (i > 0) ahead(i - 1);
      __syncthreads();
    }
    return;
  }

  if (w < 2 * NSW + 1) {
    // ---- the waves behind, one for each state wave: with the residuals
    const int z = w - NSW - 1, slice = ps * NSW + z;
    T* vt = reinterpret_cast<T*>(smem + Cf::OFF_V) + SLICE * z;   // this wave's columns
    f32x4_t te[4], us[NT][2], du[4];
    auto request = [&](int i) {
      const f32x4_t* e = reinterpret_cast<const f32x4_t*>(p.e) + (slot_head(i) * p.nsl + slice) * 4 * 64 + l;
#pragma unroll
      for (int t = 0; t < 4; ++t) te[t] = e[t * 64];
    };
    auto take = [&]() {
#pragma unroll
      for (int t = 0; t < 4; ++t) du[t] = xdu[(z * 4 + t) * 64 + l];
#pragma unroll
      for (int q = 0; q < NT; ++q) {
#pragma unroll
        for (int t = 0; t < 2; ++t) us[q][t] = reinterpret_cast<const f32x4_t*>(xs)[((z * NT + q) * 2 + t) * 64 + l];
      }
    };
    auto behind = [&](int i) {
      const int len = length(i);
      const float* gs = gbuf(i);
      const int64_t at = (slot_head(i) * p.nsl + slice) * CH;
      f32x4_t be[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        be[t] = du[t] * te[t];
        du[t] *= *reinterpret_cast<const f32x4_t*>(gs + GATE_BETA * CH + pair_col(t) + 8 * g);   // dv
      }
      if (i > 0) request(i - 1);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
#pragma unroll
        for (int r = 0; r < 4; ++r) be[t][r] = ssd::sum16(be[t][r]);
      }
      if (c == 0) {
#pragma unroll
        for (int t = 0; t < 4; ++t) *reinterpret_cast<f32x4_t*>(p.be + at + pair_col(t) + 8 * g) = be[t];
      }
      f32x4_t* ds = reinterpret_cast<f32x4_t*>(p.ds) + (slot_head(i) * p.nsl + slice) * 2 * NT * 64 + l;
#pragma unroll
      for (int q = 0; q < NT; ++q) {
#pragma unroll
        for (int t = 0; t < 2; ++t) ds[(t * NT + q) * 64] = us[q][t];
      }
      if constexpr (sizeof(T) == 2) {   // what dv's own rounding leaves
        uint4* lo = p.dvl + (slot_head(i) * p.nsl + slice) * 2 * 64 + l;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float v[8];
          pair8(du[2 * q], du[2 * q + 1], v);
          lo[q * 64] = __builtin_bit_cast(uint4, F::split(v).lo);
        }
      }
      // dv by rows, through LDS: 16 two-byte stores of four 32-byte stretches each would hold up the
      // memory pipeline
#pragma unroll
      for (int t = 0; t < 4; ++t) {
#pragma unroll
        for (int r = 0; r < 4; ++r) vt[(pair_col(t) + 8 * g + r) * LDP + c] = ssd::Elem<T>::from_f(du[t][r]);
      }
      T* dv = static_cast<T*>(p.dv) + (s0 + static_cast<int64_t>(CH) * i + l) * hp + static_cast<int64_t>(h) * p.P + PS * ps + SLICE * z;
      constexpr int VEC = Vec16<T>::N;
      if (l < len) {
#pragma unroll
        for (int k = 0; k < SLICE; k += VEC)
          if (PS * ps + SLICE * z + k < p.P) *reinterpret_cast<uint4*>(dv + k) = *reinterpret_cast<const uint4*>(vt + l * LDP + k);
      }
    };
    __syncthreads();
    request(last);
    __syncthreads();
    for (int i = last; i >= 0; --i) {
      if (i < last) take();
      __syncthreads();
      if (i < last) behind(i + 1);
      __syncthreads();
    }
    take();
    behind(0);
    return;
  }

  // ---- the staging waves
  const int ht = tid - 64 * (2 * NSW + 1);
  constexpr int GI = (RWALK_GATES * CH + Cf::HT - 1) / Cf::HT;
  const int pcols = min(PS, p.P - PS * ps);
  const T* kp = static_cast<const T*>(p.k) + row_offset(s0, p.L, p.k_sb, p.k_sl) + static_cast<int64_t>(grp) * p.N;
  const T* qp = static_cast<const T*>(p.q) + row_offset(s0, p.L, p.q_sb, p.q_sl) + static_cast<int64_t>(grp) * p.N;
  TileN tk, tq;
  TileP td;
  float tg[GI];
  auto request_k = [&](int i) { tk.load(kp + static_cast<int64_t>(CH) * i * p.k_sl, p.k_sl, length(i), p.N, ht); };
  // for the wave ahead: q, dout and the gates
  auto request_q = [&](int i) {
    const int64_t row = static_cast<int64_t>(CH) * i;
    tq.load(qp + row * p.q_sl, p.q_sl, length(i), p.N, ht);
    td.load(static_cast<const T*>(p.dout) + (s0 + row) * hp + static_cast<int64_t>(h) * p.P + PS * ps, hp, length(i), pcols, ht);
#pragma unroll
    for (int k = 0; k < GI; ++k) tg[k] = ht + k * Cf::HT < RWALK_GATES * CH ? p.gates[slot_head(i) * (GATES * CH) + ht + k * Cf::HT] : 0.f;
  };
  auto stage_q = [&](int i) {
    tq.store(qbuf(i), ht);
    td.store(dobuf(i), ht);
#pragma unroll
    for (int k = 0; k < GI; ++k)
      if (ht + k * Cf::HT < RWALK_GATES * CH) gbuf(i)[ht + k * Cf::HT] = tg[k];
  };
  request_k(last);
  request_q(last);
  tk.store(kbuf(last), ht);
  stage_q(last);
  if (last > 0) request_q(last - 1);
  if (KB && last > 0) request_k(last - 1);
  __syncthreads();
  if (KB && last > 0) {
    stage_q(last - 1);
    if (last > 1) request_q(last - 2);
  }
  __syncthreads();
  for (int i = last; i >= 0; --i) {
    if (!KB) {
      if (i < last) tk.store(kbuf(i), ht);
      if (i > 0) {
        stage_q(i - 1);
        request_k(i - 1);
      }
      if (i > 1) request_q(i - 2);
    }
    __syncthreads();
    if (KB) {
      if (i > 0) tk.store(kbuf(i - 1), ht);
      if (i > 1) {
        stage_q(i - 2);
        request_k(i - 2);
      }
      if (i > 2) request_q(i - 3);
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// k_delta_grad: dq, dk and dg of one chunk and group, its heads one
// after the other (dq and dk are sums over them, taken in registers in head
// order); on small grids parts of the heads, added up by k_delta_parts.  Eight
// waves: 16 rows of the chunk times half of the N columns each.
// For dg a lane holds a row i of M for 8 columns j: the sums over j < t run
// within the row, those over i >= t over the lanes that hold t, and what a row
// has left of its column 32 (CUT_L) enters the rows' sums of the second half.
// With bf16 io every float32 value enters as two terms (S, dS, u, dv, dP, F):
// dq and dk are their exact values rounded once (1.7e-3 off).  With S, dS and
// dv as one term 6% of their values rounded otherwise (1.8e-3), and the kernel
// took 0.79 ms without dg.  Bound by one block a CU (LDS, registers), whose
// products and sums wait for each other at two barriers a head: 1.22 ms at
// 16384 rows of 128 heads of 64 x 128 (104 KB a chunk and head, 2.8 TB/s), 0.96
// without dg.
// ---------------------------------------------------------------------------
constexpr int GTHR = 512;

// four values to LDS: float32 as they are, bf16 as two terms, the second `apart` elements after the first
template <typename T> __device__ __forceinline__ void store_terms(T* at, int apart, f32x4_t v) {
  ssd::store4f<T>(at, v);
  if constexpr (sizeof(T) == 2) {
    f32x4_t r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = v[i] - ssd::Elem<T>::to_f(ssd::Elem<T>::from_f(v[i]));
    ssd::store4f<T>(at + apart, r);
  }
}

// 8 rows of a column as load_tr gives them, from both terms
template <typename T> __device__ __forceinline__ typename Fr<T>::S load_tr_terms(const T* base, int apart, int ld, int row0) {
  const typename Fr<T>::X x = Fr<T>::load_tr(base, ld, row0);
  if constexpr (sizeof(T) == 2) return Fr<T>::terms(x, Fr<T>::load_tr(base + apart, ld, row0));
  else return x;
}

template <typename T, int NT> struct GradCfg {
  static constexpr int ND = 32 * NT;
  static constexpr int PSL = sizeof(T) == 2 ? 64 : 32;   // value columns staged at once
  using TileN = Tile<T, CH, ND, GTHR>;
  using TileP = Tile<T, CH, PSL, GTHR>;    // dout, dv
  static constexpr int LDU = CH + Vec16<T>::N;   // u, a value column per row
  static constexpr size_t U_BYTES = sizeof(T) * PSL * LDU;
  static constexpr int TERMS = sizeof(T) == 2 ? 2 : 1;   // of the float32 values
  using TileL = SliceTile<T, PSL / SLICE, CH / 32, GTHR>;   // dv's second terms, a value column per row
  using TileS = SliceTile<T, PSL / SLICE, NT, GTHR>;   // S, dS, a value column per row
  using TileM = Tile<T, CH, CH, GTHR>;     // dP, F + F^T (over the tiles above)
  static constexpr size_t OFF_Q = sizeof(T) * TileN::LDS_ELEMS;
  static constexpr size_t OFF_DO = 2 * OFF_Q;
  static constexpr size_t OFF_DV = OFF_DO + sizeof(T) * TileP::LDS_ELEMS;
  static constexpr size_t OFF_DVL = OFF_DV + sizeof(T) * TileP::LDS_ELEMS;
  static constexpr size_t OFF_U = OFF_DVL + (TERMS > 1 ? sizeof(T) * TileL::LDS_ELEMS : 0);
  static constexpr size_t OFF_S = OFF_U + TERMS * U_BYTES;
  static constexpr size_t OFF_DS = OFF_S + TERMS * sizeof(T) * TileS::LDS_ELEMS;
  static constexpr size_t END1 = OFF_DS + TERMS * sizeof(T) * TileS::LDS_ELEMS;
  static constexpr size_t OFF_F = OFF_DO + TERMS * sizeof(T) * TileM::LDS_ELEMS;
  static constexpr size_t END2 = OFF_F + TERMS * sizeof(T) * TileM::LDS_ELEMS;
  static constexpr size_t OFF_G = END1 > END2 ? END1 : END2;
  // for dg: a and b from both halves of N, the rows' sums of M left of column 32, M's sums at a column from each row
  // tile, and <S, dS> from every wave
  static constexpr int CUT_A = 0, CUT_B = CUT_A + 2 * CH, CUT_L = CUT_B + 2 * CH, CUT_M = CUT_L + CH, CUT_S = CUT_M + 4 * CH, CUTS = CUT_S + GTHR / 64;
  static constexpr size_t OFF_CUT = OFF_G + sizeof(float) * GATES * CH;
  static constexpr size_t LDS = OFF_CUT + sizeof(float) * CUTS;
};

template <typename T, int NT> __global__ __launch_bounds__(GTHR) void k_delta_grad(Problem p) {
  using Cf = GradCfg<T, NT>;
  using F = Fr<T>;
  constexpr int LDN = Cf::TileN::LD, LDP = Cf::TileP::LD, LDU = Cf::LDU, LDS_ = Cf::TileS::LD, LDMT = Cf::TileM::LD;
  constexpr int PSL = Cf::PSL;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  T* kt = reinterpret_cast<T*>(smem);
  T* qt = reinterpret_cast<T*>(smem + Cf::OFF_Q);
  T* dot = reinterpret_cast<T*>(smem + Cf::OFF_DO);
  T* dvt = reinterpret_cast<T*>(smem + Cf::OFF_DV);
  T* dvl = reinterpret_cast<T*>(smem + Cf::OFF_DVL);
  T* ut = reinterpret_cast<T*>(smem + Cf::OFF_U);
  T* st = reinterpret_cast<T*>(smem + Cf::OFF_S);
  T* dst = reinterpret_cast<T*>(smem + Cf::OFF_DS);
  constexpr int TERMS = Cf::TERMS, UL = Cf::U_BYTES / sizeof(T), SL = Cf::TileS::LDS_ELEMS, ML = Cf::TileM::LDS_ELEMS;   // from first terms to second
  T* dpm = reinterpret_cast<T*>(smem + Cf::OFF_DO);
  T* fm = reinterpret_cast<T*>(smem + Cf::OFF_F);
  float* gs = reinterpret_cast<float*>(smem + Cf::OFF_G);
  float* cut = reinterpret_cast<float*>(smem + Cf::OFF_CUT);

  const int slot = static_cast<int>(blockIdx.x), grp = static_cast<int>(blockIdx.y) / p.ns, part = static_cast<int>(blockIdx.y) % p.ns;
  const int first_head = part * p.hs, end_head = min(p.hpg, first_head + p.hs);   // of the group
  const Chunk ch = chunk_of(p, slot);
  if (ch.len == 0) return;
  const int tid = static_cast<int>(threadIdx.x), l = tid & 63, g = l >> 4, c = l & 15, w = ssd::wave_id_s();
  const int rt = w & 3, half = w >> 2, row = 16 * rt + c;
  const int64_t hp = static_cast<int64_t>(p.H) * p.P;
  {
    typename Cf::TileN tk, tq;
    tk.load(static_cast<const T*>(p.k) + row_offset(ch.row, p.L, p.k_sb, p.k_sl) + static_cast<int64_t>(grp) * p.N, p.k_sl, ch.len, p.N, tid);
    tq.load(static_cast<const T*>(p.q) + row_offset(ch.row, p.L, p.q_sb, p.q_sl) + static_cast<int64_t>(grp) * p.N, p.q_sl, ch.len, p.N, tid);
    tk.store(kt, tid);
    tq.store(qt, tid);
  }
  // A lane's places are taken anew where they are used: the addresses made of them would be kept over the heads, and
  // spill (their reloads then wait for the requests in flight: 2.7 ms instead of 1.2).
  const int tid0 = tid, l0 = l;
  auto anew = [](int v) {
    asm volatile("" : "+v"(v));
    return v;
  };
  f32x4_t dqa[NT], dka[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) dqa[t] = dka[t] = zero4();

  // the states of a head's slice are requested while the one before is worked on
  typename Cf::TileS ts[TERMS], tds[TERMS];
  auto request = [&](int hh, int p0) {
    const int tid = anew(tid0);
    const int64_t first = (static_cast<int64_t>(slot) * p.H + grp * p.hpg + hh) * p.nsl + p0 / SLICE;
    const int nslices = min(PSL / SLICE, p.nsl - p0 / SLICE);
#pragma unroll
    for (int u = 0; u < TERMS; ++u) {
      ts[u].load(p.s + (first * 2 + u) * NT * 64, 2 * NT * 64, nslices, tid);
      tds[u].load(p.ds + (first * 2 + u) * NT * 64, 2 * NT * 64, nslices, tid);
    }
  };
  request(first_head, 0);
  for (int hh = first_head; hh < end_head; ++hh) {
    const int h = grp * p.hpg + hh;
    const int64_t sh = static_cast<int64_t>(slot) * p.H + h;
    f32x4_t x1[NT], x2[NT], x3[NT], m1[2], m2[2];
#pragma unroll
    for (int t = 0; t < NT; ++t) x1[t] = x2[t] = x3[t] = zero4();
    m1[0] = m1[1] = m2[0] = m2[1] = zero4();
    float ssum = 0.f;   // <S, dS>
    for (int p0 = 0; p0 < p.P; p0 += PSL) {
      const int pcols = min(PSL, p.P - p0);
      typename Cf::TileP td, tv;
      // u = beta e from the residuals as the lanes hold them: piece t of lane (g, c) is column c's rows pair_col(t) + 8 g ..
      constexpr int PER = 4 * 64, UIT = PSL / SLICE * PER / GTHR;
      static_assert(PSL / SLICE * PER % GTHR == 0 && GTHR % PER == 0, "residuals");
      f32x4_t tu[UIT];
      const int urow = pair_col(tid % PER / 64) + 8 * g;
      const int64_t at = static_cast<int64_t>(ch.row) * hp + static_cast<int64_t>(h) * p.P + p0;
      td.load(static_cast<const T*>(p.dout) + at, hp, ch.len, pcols, tid);
      tv.load(static_cast<const T*>(p.dv) + at, hp, ch.len, pcols, tid);
      const int64_t first = sh * p.nsl + p0 / SLICE;
      const int nslices = min(PSL / SLICE, p.nsl - p0 / SLICE);
      const f32x4_t be = *reinterpret_cast<const f32x4_t*>(p.gates + sh * (GATES * CH) + GATE_BETA * CH + urow);
#pragma unroll
      for (int k = 0; k < UIT; ++k) {
        tu[k] = zero4();
        if (tid / PER + k * (GTHR / PER) < nslices) tu[k] = reinterpret_cast<const f32x4_t*>(p.e)[first * PER + tid + k * GTHR];
      }
      typename Cf::TileL tl;
      if constexpr (TERMS > 1) tl.load(p.dvl + first * 2 * 64, 2 * 64, nslices, tid);
      const float tg = tid < GATES * CH ? p.gates[sh * (GATES * CH) + tid] : 0.f;
      __syncthreads();   // the previous head's last products are done
      td.store(dot, tid);
      tv.store(dvt, tid);
#pragma unroll
      for (int k = 0; k < UIT; ++k) store_terms<T>(ut + ((tid / PER + k * (GTHR / PER)) * SLICE + c) * LDU + urow, UL, be * tu[k]);
      if constexpr (TERMS > 1) tl.store(dvl, tid);
#pragma unroll
      for (int u = 0; u < TERMS; ++u) {
        ts[u].store(st + u * SL, tid);
        tds[u].store(dst + u * SL, tid);
      }
#pragma unroll
      for (int k = 0; k < Cf::TileS::IT; ++k) {
        if constexpr (TERMS > 1) {
          float x[8], y[8];
          F::floats(F::terms(__builtin_bit_cast(typename F::X, ts[0].buf[k]), __builtin_bit_cast(typename F::X, ts[1].buf[k])), x);
          F::floats(F::terms(__builtin_bit_cast(typename F::X, tds[0].buf[k]), __builtin_bit_cast(typename F::X, tds[1].buf[k])), y);
#pragma unroll
          for (int r = 0; r < 8; ++r) ssum += x[r] * y[r];
        } else {
          const f32x4_t x = ts[0].buf[k] * tds[0].buf[k];
          ssum += (x[0] + x[1]) + (x[2] + x[3]);
        }
      }
      if (tid < GATES * CH) gs[tid] = tg;
      __syncthreads();
      if (p0 + PSL < p.P) request(hh, p0 + PSL);
      else if (hh + 1 < end_head) request(hh + 1, 0);
#pragma unroll 1
      for (int ks = 0; ks < PSL / 32; ++ks) {
        const int k0 = 32 * ks + 8 * g;
        const typename F::X xdo = F::load(dot + row * LDP + k0);
        typename F::S xdv, xu;
        if constexpr (TERMS > 1) xdv = F::terms(F::load(dvt + row * LDP + k0), F::load_tr(dvl + 16 * rt, Cf::TileL::LD, k0));
        else xdv = F::load(dvt + row * LDP + k0);
        xu = load_tr_terms<T>(ut + 16 * rt, UL, LDU, k0);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const int n0 = 16 * (half * NT + t);
          const typename F::S xs = load_tr_terms<T>(st + n0, SL, LDS_, k0), xds = load_tr_terms<T>(dst + n0, SL, LDS_, k0);
          x1[t] = mma(xs, xdo, x1[t]);
          x2[t] = mma(xs, xdv, x2[t]);
          x3[t] = mma(xds, xu, x3[t]);
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int jt = 2 * half + t;
          if (jt <= rt) {
            const typename F::S xj = load_tr_terms<T>(ut + 16 * jt, UL, LDU, k0);
            m1[t] = mma(xj, xdo, m1[t]);
            m2[t] = mma(xj, xdv, m2[t]);
          }
        }
      }
    }
    const int l = anew(l0), g = l >> 4, c = l & 15, row = 16 * rt + c;
    const float in = gs[GATE_IN * CH + row], out = gs[GATE_OUT * CH + row];
    float ca = 0.f, cb = 0.f;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int n = 16 * (half * NT + t) + 4 * g;
      const f32x4_t kv = ssd::load4f<T>(kt + row * LDN + n), qv = ssd::load4f<T>(qt + row * LDN + n);
      x1[t] *= p.scale * in;
      x2[t] *= in;
      x3[t] *= out;
      dqa[t] += x1[t];
      dka[t] += x3[t] - x2[t];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        ca += qv[r] * x1[t][r] - kv[r] * x2[t][r];
        cb += kv[r] * x3[t][r];
      }
    }
    ca = ssd::sum_kgroups(ca);
    cb = ssd::sum_kgroups(cb);
    ssum = ssd::wave_sum(ssum);
    __syncthreads();
    if (g == 0) {
      cut[Cf::CUT_A + half * CH + row] = ca;
      cut[Cf::CUT_B + half * CH + row] = cb;
      if (c == 0) cut[Cf::CUT_S + w] = ssum;
    }
    float left = 0.f;   // the row's sum of M left of the tile
    const float ci = gs[GATE_C * CH + row], cl = gs[GATE_CLO * CH + row];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int jt = 2 * half + t;
      f32x4_t dp = zero4(), m = zero4(), at_col = zero4();
      if (jt <= rt) {
        f32x4_t qk = zero4(), kk = zero4();   // of rows i (columns) and j (rows), as m1 and m2
#pragma unroll
        for (int ks = 0; ks < NT; ++ks) {
          const typename F::X kj = F::load(kt + (16 * jt + c) * LDN + 32 * ks + 8 * g);
          qk = mma(kj, F::load(qt + row * LDN + 32 * ks + 8 * g), qk);
          kk = mma(kj, F::load(kt + row * LDN + 32 * ks + 8 * g), kk);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int j = 16 * jt + 4 * g + r;
          const float dec = expf((ci - gs[GATE_C * CH + j]) + (cl - gs[GATE_CLO * CH + j]));
          if (j <= row) dp[r] = p.scale * (dec * m1[t][r]);
          if (j < row) {
            float f = -dec * m2[t][r];
            m[r] = qk[r] * dp[r] + kk[r] * f;
#pragma unroll
            for (int u = 0; u < TERMS; ++u) {
              const T x = ssd::Elem<T>::from_f(f);
              fm[u * ML + row * LDMT + j] = x;
              fm[u * ML + j * LDMT + row] = x;
              f -= ssd::Elem<T>::to_f(x);
            }
          } else if (j == row) {
#pragma unroll
            for (int u = 0; u < TERMS; ++u) fm[u * ML + row * LDMT + row] = ssd::Elem<T>::from_f(0.f);
          }
        }
      }
      if (jt <= rt) {
        // the sums over the row's columns before j, and of those over the rows from j on
        float by_g[4], before = left;
        ssd::gather_kgroups((m[0] + m[1]) + (m[2] + m[3]), by_g);
#pragma unroll
        for (int q = 0; q < 3; ++q)
          if (q < g) before += by_g[q];
        left += (by_g[0] + by_g[1]) + (by_g[2] + by_g[3]);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          at_col[r] = ssd::sum16(16 * jt + 4 * g + r <= row ? before : 0.f);
          before += m[r];
        }
      }
      if (c == 0) *reinterpret_cast<f32x4_t*>(cut + Cf::CUT_M + rt * CH + 16 * jt + 4 * g) = at_col;
      store_terms<T>(dpm + row * LDMT + 16 * jt + 4 * g, ML, dp);
    }
    if (half == 0 && g == 0) cut[Cf::CUT_L + row] = left;
    __syncthreads();
    if (w == (hh & 7)) {   // dg, row l: suffix sums of a and of what is left of column 32, prefix sums of b
      float a = cut[Cf::CUT_A + l] + cut[Cf::CUT_A + CH + l], b = cut[Cf::CUT_B + l] + cut[Cf::CUT_B + CH + l];
      float lower = l < 32 ? 0.f : cut[Cf::CUT_L + l];
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const float ad = __shfl_down(a, d), ld = __shfl_down(lower, d), bu = __shfl_up(b, d);
        if (l + d < 64) {
          a += ad;
          lower += ld;
        }
        if (l >= d) b += bu;
      }
      b = __shfl_up(b, 1);
      float sum = a + (l > 0 ? b : 0.f) + (l < 32 ? 0.f : lower), ss = 0.f;
#pragma unroll
      for (int q = 0; q < 4; ++q) sum += cut[Cf::CUT_M + q * CH + l];
#pragma unroll
      for (int q = 0; q < GTHR / 64; ++q) ss += cut[Cf::CUT_S + q];
      if (l < ch.len) p.dg[(static_cast<int64_t>(ch.row) + l) * p.H + h] = sum + gs[GATE_IN * CH + CH - 1] * ss;
    }
#pragma unroll 1
    for (int ks = 0; ks < 2; ++ks) {
      typename F::X xp[TERMS], xf[TERMS], xpt[TERMS];
#pragma unroll
      for (int u = 0; u < TERMS; ++u) {
        xp[u] = F::load(dpm + u * ML + row * LDMT + 32 * ks + 8 * g);
        xf[u] = F::load(fm + u * ML + row * LDMT + 32 * ks + 8 * g);
        xpt[u] = F::load_tr(dpm + u * ML + 16 * rt, LDMT, 32 * ks + 8 * g);
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int n0 = 16 * (half * NT + t);
        const typename F::X xk = F::load_tr(kt + n0, LDN, 32 * ks + 8 * g), xq = F::load_tr(qt + n0, LDN, 32 * ks + 8 * g);
#pragma unroll
        for (int u = TERMS - 1; u >= 0; --u) {
          dqa[t] = mma(xk, xp[u], dqa[t]);
          dka[t] = mma(xq, xpt[u], dka[t]);
          dka[t] = mma(xk, xf[u], dka[t]);
        }
      }
    }
  }
  if (p.ns > 1) {   // this part's sums, for k_delta_parts
    float* to = p.parts + ((static_cast<int64_t>(slot) * p.G + grp) * p.ns + part) * 2 * CH * Cf::ND + row * Cf::ND;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int n = 16 * (half * NT + t) + 4 * g;
      *reinterpret_cast<f32x4_t*>(to + n) = dqa[t];
      *reinterpret_cast<f32x4_t*>(to + CH * Cf::ND + n) = dka[t];
    }
    return;
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

// dq and dk from the parts of a group's heads, in order.
constexpr int PARTS_Z = 8;   // blocks of a chunk
template <typename T, int NT> __global__ __launch_bounds__(256) void k_delta_parts(Problem p) {
  constexpr int ND = 32 * NT;
  const int slot = static_cast<int>(blockIdx.x), grp = static_cast<int>(blockIdx.y);
  const Chunk ch = chunk_of(p, slot);
  for (int i = static_cast<int>(blockIdx.z * 256 + threadIdx.x); i < ch.len * (ND / 4); i += 256 * PARTS_Z) {
    const int row = i / (ND / 4), n = 4 * (i % (ND / 4));
    if (n >= p.N) continue;
    const float* from = p.parts + (static_cast<int64_t>(slot) * p.G + grp) * p.ns * 2 * CH * ND + row * ND + n;
    f32x4_t q = zero4(), k = zero4();
#pragma unroll 4
    for (int s = 0; s < p.ns; ++s) {
      q += *reinterpret_cast<const f32x4_t*>(from + s * 2 * CH * ND);
      k += *reinterpret_cast<const f32x4_t*>(from + (2 * s + 1) * CH * ND);
    }
    const int64_t at = ((static_cast<int64_t>(ch.row) + row) * p.G + grp) * p.N + n;
    ssd::store4f<T>(static_cast<T*>(p.dq) + at, q);
    ssd::store4f<T>(static_cast<T*>(p.dk) + at, k);
  }
}

// ---------------------------------------------------------------------------
// k_delta_gates: dbeta of one chunk, a wave per head: the slices' row sums added
// in slice order.
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(256) void k_delta_gates(Problem p) {
  const int slot = static_cast<int>(blockIdx.x), h = static_cast<int>(blockIdx.y) * 4 + ssd::wave_id_s(), l = ssd::lane_id();
  const Chunk ch = chunk_of(p, slot);
  if (ch.len == 0 || h >= p.H) return;
  const int64_t sh = static_cast<int64_t>(slot) * p.H + h;
  float b = 0.f;
#pragma unroll 4
  for (int s = 0; s < p.nsl; ++s) b += p.be[(sh * p.nsl + s) * CH + l];
  if (l < ch.len) p.dbeta[(static_cast<int64_t>(ch.row) + l) * p.H + h] = b;
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
  using Cf = RwalkCfg<T, NT>;
  return go(k_delta_rwalk<T, NT>, dim3(p.H * ((p.P + Cf::PS - 1) / Cf::PS), p.nseqs), Cf::THREADS, Cf::LDS, s, p);
}
template <typename T, int NT> int grad(const Problem& p, hipStream_t s) {
  static_assert(GradCfg<T, NT>::LDS <= 160 * 1024, "LDS");
  const int rc = go(k_delta_grad<T, NT>, dim3(p.nslots, p.G * p.ns), GTHR, GradCfg<T, NT>::LDS, s, p);
  return rc != SSD_OK || p.ns == 1 ? rc : go(k_delta_parts<T, NT>, dim3(p.nslots, p.G, PARTS_Z), 256, 0, s, p);
}

int launch_rwalk(const Problem& p, int io, hipStream_t s) {
  if (io == SSD_IO_BF16) return p.N <= 64 ? rwalk<bf16_t, 2>(p, s) : rwalk<bf16_t, 4>(p, s);
  return p.N <= 64 ? rwalk<float, 2>(p, s) : rwalk<float, 4>(p, s);
}
int launch_grad(const Problem& p, int io, hipStream_t s) {
  if (io == SSD_IO_BF16) return p.N <= 64 ? grad<bf16_t, 2>(p, s) : grad<bf16_t, 4>(p, s);
  return p.N <= 64 ? grad<float, 2>(p, s) : grad<float, 4>(p, s);
}
int launch_gates(const Problem& p, hipStream_t s) { return go(k_delta_gates, dim3(p.nslots, (p.H + 3) / 4), 256, 0, s, p); }

}  // namespace delta
