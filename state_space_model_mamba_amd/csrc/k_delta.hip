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
// order, and the order in which the walks take them.  One block: every thread
// takes 16 rows of a stretch of 16384, the counts are scanned over the block.
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
  // the walks' order: longest first, equal ones by number (more sequences than ST_THR keep their own: with so many
  // blocks no single one is the end)
  __syncthreads();
  int32_t* order = p.starts + p.nseqs + 1;
  if (p.nseqs > ST_THR) {
    for (int s = tid; s < p.nseqs; s += ST_THR) order[s] = s;
    return;
  }
  __shared__ int len[ST_THR];
  if (tid < p.nseqs) len[tid] = p.starts[tid + 1] - p.starts[tid];
  __syncthreads();
  if (tid < p.nseqs) {
    const int mine = len[tid];
    int rank = 0;
    for (int s = 0; s < p.nseqs; ++s) rank += len[s] > mine || (len[s] == mine && s < tid) ? 1 : 0;
    order[rank] = tid;
  }
}

// ---------------------------------------------------------------------------
// k_delta_prep: T' and the scores of one chunk (for the backward T', the
// transposed (I + diag(beta) N)^-1 and the transposed scores), as the walks'
// operand fragments, for up to HB heads of one group.
//
// q k^T and k k^T are the group's: they are taken once, from operands loaded
// straight into registers, and every head scales its copies by its decays.
// With the rows of the first operand in pair order a pair of score tiles is
// the walk's fragment already; only the matrices to invert go through LDS.
//
// The inverse of a unit lower triangular 64 x 64 matrix in float32: the four
// 16 x 16 diagonal blocks by substitution (a lane per column, one wave, while
// others scale the scores), then 32 x 32 and 64 x 64 by the block formula
// T21 = -T22 A21 T11 with float32 MFMA tiles, in place in LDS.
//
// Bound by the instructions of a head (some 1000 a wave, a third of them the
// substitution) and in the backward by its 36 KB of fragments: 256 chunks of
// 128 heads of 64 x 128 take 0.30 ms (24 KB a chunk and head, 2.6 TB/s), in
// the backward 0.41 ms (2.9 TB/s).
// ---------------------------------------------------------------------------
constexpr int LDM = 68;   // pitch of the float32 64 x 64 matrices

template <bool BWD> struct PrepCfg {
  static constexpr int NM = BWD ? 2 : 1;
  static constexpr size_t OFF_C = sizeof(float) * NM * CH * LDM;
  static size_t lds(int heads) { return OFF_C + sizeof(float) * 3 * CH * heads; }
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

// the inverses of the four 16 x 16 diagonal blocks, in place, by one wave: a lane per block and column
__device__ __forceinline__ void invert_diagonal(float* m) {
  const int l = ssd::lane_id(), g = l >> 4, c = l & 15;
  float* d = m + 16 * g * LDM + 16 * g;
  float x[16];
  x[0] = c == 0 ? 1.f : 0.f;
#pragma unroll
  for (int i = 1; i < 16; ++i) {
    f32x4_t row[4];
#pragma unroll
    for (int q = 0; q <= (i - 1) / 4; ++q) row[q] = *reinterpret_cast<const f32x4_t*>(d + i * LDM + 4 * q);
    float s0 = i == c ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
    for (int k = 0; k < i; ++k) {
      if ((i - 1 - k) & 1) s1 -= row[k / 4][k % 4] * x[k]; else s0 -= row[k / 4][k % 4] * x[k];
    }
    x[i] = s0 + s1;
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) d[i * LDM + c] = x[i];
}

// the rest of the inverse: blocks (1, 0) and (3, 2), then the lower left quarter column by column (a wave each,
// the products between in registers)
template <int NM> __device__ __forceinline__ void invert_rest(float* m) {
  const int l = ssd::lane_id(), g = l >> 4, c = l & 15, w = ssd::wave_id_s();
  float* base = m + (w >> 1) * CH * LDM;
  auto blk = [&](int i, int j) { return base + 16 * i * LDM + 16 * j; };
  auto mma_left = [&](const float* t, f32x4_t y, f32x4_t acc) {   // acc + T y, y a tile in registers
    return ssd::Mma<float>::mma_rd(*reinterpret_cast<const f32x4_t*>(t + c * LDM + 4 * g), y, acc);
  };
  if (w < 2 * NM) {
    const int q = 2 * (w & 1);
    const f32x4_t y = block_mma(blk(q + 1, q), blk(q, q), zero4());
    block_store(blk(q + 1, q), -mma_left(blk(q + 1, q + 1), y, zero4()));
  }
  __syncthreads();
  const int j = w & 1;
  f32x4_t y[2];
  if (w < 2 * NM) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      y[i] = block_mma(blk(2 + i, 1), blk(1, j), zero4());   // T_01 is zero
      if (j == 0) y[i] = block_mma(blk(2 + i, 0), blk(0, 0), y[i]);
    }
  }
  __syncthreads();   // column 0 reads blocks (2, 1) and (3, 1), which column 1 overwrites
  if (w < 2 * NM) {
    const f32x4_t t2 = mma_left(blk(2, 2), y[0], zero4());
    const f32x4_t t3 = mma_left(blk(3, 3), y[1], mma_left(blk(3, 2), y[0], zero4()));
    block_store(blk(2, j), -t2);
    block_store(blk(3, j), -t3);
  }
  __syncthreads();
}

template <typename T, int NT, bool BWD> __global__ __launch_bounds__(256, BWD ? 2 : 3) void k_delta_prep(Problem p) {
  using Cf = PrepCfg<BWD>;
  using F = Fr<T>;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  float* mm = reinterpret_cast<float*>(smem);
  float* cb = reinterpret_cast<float*>(smem + Cf::OFF_C);   // per head: the sums of g in two floats, and beta

  const int slot = static_cast<int>(blockIdx.x);
  const int parts = (p.hpg + p.hb - 1) / p.hb, grp = static_cast<int>(blockIdx.y) / parts;
  const int h0 = grp * p.hpg + static_cast<int>(blockIdx.y) % parts * p.hb, h1 = min(h0 + p.hb, (grp + 1) * p.hpg);
  const Chunk ch = chunk_of(p, slot);
  if (ch.len == 0) return;
  const int tid = static_cast<int>(threadIdx.x), l = tid & 63, g = l >> 4, c = l & 15, w = ssd::wave_id_s();

  // the heads' gates, a wave each
  for (int h = h0 + w; h < h1; h += 4) {
    const int64_t at = static_cast<int64_t>(ch.row + l) * p.H + h;
    float gv = l < ch.len ? p.g[at] : 0.f;
    gv = gv < -104.f ? -104.f : gv;
    const float b = l < ch.len ? p.beta[at] : 0.f;
    double s = gv;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const double o = __shfl_up(s, d);
      if (l >= d) s += o;
    }
    const double last = __shfl(s, 63);
    const float hi = static_cast<float>(s), lo = static_cast<float>(s - hi);
    float* cs = cb + (h - h0) * 3 * CH;
    cs[l] = hi;
    cs[CH + l] = lo;
    cs[2 * CH + l] = b;
    float* gt = p.gates + (static_cast<int64_t>(slot) * p.H + h) * (GATES * CH) + l;
    const float in = expf(hi), out = expf(static_cast<float>(last - s));
    gt[GATE_IN * CH] = in;
    gt[GATE_BO * CH] = b * out;
    gt[GATE_BETA * CH] = b;
    gt[GATE_OUT * CH] = out;
    gt[GATE_BI * CH] = -b * in;
    gt[GATE_C * CH] = hi;
    gt[GATE_CLO * CH] = lo;
  }

  const T* kp = static_cast<const T*>(p.k) + row_offset(ch.row, p.L, p.k_sb, p.k_sl) + static_cast<int64_t>(grp) * p.N;
  const T* qp = static_cast<const T*>(p.q) + row_offset(ch.row, p.L, p.q_sb, p.q_sl) + static_cast<int64_t>(grp) * p.N;
  // Rows past the chunk's last stand in as its first: what they give stays in rows past the last (and beta is 0
  // there).  Columns past N have to be zero.
  auto operand = [&](const T* base, int64_t stride, int row, int ks, auto whole) {
    const int n = 32 * ks + 8 * g;
    const T* at = base + (row < ch.len ? row : 0) * stride + n;
    if constexpr (decltype(whole)::value) return F::load(at);
    else return n < p.N ? F::load_cols(at, p.N - n) : F::zero();
  };
  // Row tile w of k k^T (tiles ct <= w, rows 4 g + r and column c), and of the scores the fragments sw, sw + SW, ..
  // (rows i = 16 t + c, values j; transposed: rows j in pair order, values i), sw = w - NM: the first NM waves
  // invert the diagonal blocks meanwhile.
  // lower: (0,0) (1,0) (2,0) (2,1) (3,0) (3,1); upper: (0,0) (0,1) (1,0) (1,1) (2,1) (3,1)
  constexpr int SW = 4 - Cf::NM, SF = NFRAG / SW;
  const int sw = w - Cf::NM;
  auto lower_t = [](int f) { return f < 2 ? f : 2 + ((f - 2) >> 1); };
  auto lower_k = [](int f) { return f < 2 ? 0 : (f - 2) & 1; };
  auto upper_t = [](int f) { return f < 4 ? f >> 1 : f - 2; };
  auto upper_k = [](int f) { return f < 4 ? f & 1 : 1; };
  f32x4_t kk[4], qk[SF][2];
  auto products = [&](auto whole) {
#pragma unroll
    for (int t = 0; t < 4; ++t) kk[t] = zero4();
#pragma unroll
    for (int ks = 0; ks < NT; ++ks) {
      const typename F::X a = operand(kp, p.k_sl, 16 * w + c, ks, whole);
#pragma unroll
      for (int ct = 0; ct < 4; ++ct)
        if (ct <= w) kk[ct] = mma(a, operand(kp, p.k_sl, 16 * ct + c, ks, whole), kk[ct]);
    }
    if (sw < 0) return;
#pragma unroll
    for (int z = 0; z < SF; ++z) {
      const int f = sw + SW * z;
      qk[z][0] = qk[z][1] = zero4();
#pragma unroll
      for (int ks = 0; ks < NT; ++ks) {
        const typename F::X x = BWD ? operand(kp, p.k_sl, perm_row(upper_t(f), c), ks, whole) : operand(qp, p.q_sl, 16 * lower_t(f) + c, ks, whole);
#pragma unroll
        for (int y = 0; y < 2; ++y)
          qk[z][y] = mma(BWD ? operand(qp, p.q_sl, perm_row(2 * upper_k(f) + y, c), ks, whole)
                             : operand(kp, p.k_sl, perm_row(2 * lower_k(f) + y, c), ks, whole), x, qk[z][y]);
      }
    }
  };
  if (p.N == 32 * NT) products(std::true_type{}); else products(std::false_type{});
  __syncthreads();

  for (int h = h0; h < h1; ++h) {
    const int64_t sh = static_cast<int64_t>(slot) * p.H + h;
    const float *chi = cb + (h - h0) * 3 * CH, *clo = chi + CH, *bs = chi + 2 * CH;
    // exp(c_i - c_j) where `low` (j <= i), and 0
    auto decay = [](float hi_i, float lo_i, float hi_j, float lo_j, bool low) {
      const float d = __expf(low ? (hi_i - hi_j) + (lo_i - lo_j) : 0.f);
      return low ? d : 0.f;
    };
    auto load4 = [](const float* x) { return *reinterpret_cast<const f32x4_t*>(x); };
    auto put = [&](uint4* to, int f, const float (&v)[8]) {
      uint4 u[2];
      F::pieces(F::split(v), u);
      uint4* d = to + sh * FRAG_PIECES + 2 * f * 64 + l;
      d[0] = u[0];
      d[64] = u[1];
    };
    // rows 16 w .. 16 w + 15 of N, scaled; zero on and above the diagonal
    {
      const int i0 = 16 * w + 4 * g;
      const f32x4_t hi = load4(chi + i0), lo = load4(clo + i0), bi = load4(bs + i0);
#pragma unroll
      for (int ct = 0; ct < 4; ++ct) {
        const int j = 16 * ct + c;
        const float hj = chi[j], lj = clo[j], bj = bs[j];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float n = ct <= w ? kk[ct][r] * decay(hi[r], lo[r], hj, lj, j < i0 + r) : 0.f;
          mm[(i0 + r) * LDM + j] = n * bj;
          if constexpr (BWD) mm[CH * LDM + (i0 + r) * LDM + j] = n * bi[r];
        }
      }
    }
    __syncthreads();
    if (sw < 0) {
      invert_diagonal(mm + w * CH * LDM);
    } else {
#pragma unroll
      for (int z = 0; z < SF; ++z) {
        const int f = sw + SW * z;
        float v[8];
        if constexpr (!BWD) {
          const int i = 16 * lower_t(f) + c, j0 = 32 * lower_k(f) + 8 * g;
          const float hi = chi[i], li = clo[i];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const f32x4_t hj = load4(chi + j0 + 4 * y), lj = load4(clo + j0 + 4 * y);
#pragma unroll
            for (int r = 0; r < 4; ++r) v[4 * y + r] = p.scale * (qk[z][y][r] * decay(hi, li, hj[r], lj[r], j0 + 4 * y + r <= i));
          }
        } else {
          const int j = perm_row(upper_t(f), c), i0 = 32 * upper_k(f) + 8 * g;
          const float hj = chi[j], lj = clo[j];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const f32x4_t ih = load4(chi + i0 + 4 * y), il = load4(clo + i0 + 4 * y);
#pragma unroll
            for (int r = 0; r < 4; ++r) v[4 * y + r] = p.scale * (qk[z][y][r] * decay(ih[r], il[r], hj, lj, j <= i0 + 4 * y + r));
          }
        }
        put(BWD ? p.ptf : p.pf, f, v);
      }
    }
    __syncthreads();
    invert_rest<Cf::NM>(mm);
    for (int f = w; f < NFRAG; f += 4) {
      const int row = perm_row(lower_t(f), c), k0 = 32 * lower_k(f) + 8 * g;
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = mm[row * LDM + k0 + e] - (row == k0 + e ? 1.f : 0.f);
      put(p.tf, f, v);
      if constexpr (BWD) {
        const int ff = NFRAG - 1 - f;   // a wave with two of the one has one of the other
        const int col = perm_row(upper_t(ff), c), r0 = 32 * upper_k(ff) + 8 * g;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = mm[CH * LDM + (r0 + e) * LDM + col] - (col == r0 + e ? 1.f : 0.f);
        put(p.ttf, ff, v);
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// k_delta_walk: one sequence's chunks in order, for one head and 16 NSW of its
// value columns.  A column of S needs no other column, so each of the NSW
// state waves keeps 16 columns (N x 16) in registers as accumulator tiles for
// the whole sequence and runs the sequential part alone:
//     k S -> r -> T' r -> S   (three products a chunk, nothing else).
// Beside them output waves form the previous chunk's o from the entering
// state and the residuals that the state waves leave in LDS (in the
// backward they store both for the later kernels instead), and two staging
// waves bring the coming chunks' rows in: their loads are in flight for a whole
// chunk, which no wave waits for.
//
// What bounds it is the sequence itself: a chunk takes a state wave some 4400
// cycles (98 MFMAs of 16, 400 vector instructions between them, two LDS round
// trips), 2.0 us; 2048 rows of 128 heads 70 us, 16384 rows 0.55 ms.  One wave
// doing everything took 4.85 us a chunk.  The backward's recomputation writes
// 48 KB a chunk and head beside it in the same time (0.56 ms, 2.9 TB/s).
//
// Between two barriers the state waves work on chunk i, the output waves on
// chunk i - 1 and the staging waves on k, v of chunk i + 1 and q, scores of
// chunk i.  Where LDS holds what the state waves leave only once, a second
// barrier a chunk lets the output waves take it first.
// ---------------------------------------------------------------------------
template <typename T, int NT, bool BWD, int NSW> struct WalkCfg {
  static constexpr int ND = 32 * NT, PS = SLICE * NSW, NOUT = BWD && NSW == 2 ? 2 : NSW / 2, NZ = NSW / NOUT, NST = 2, HT = 64 * NST, THREADS = 64 * (NSW + NOUT + NST);
  using TileN = Tile<T, CH, ND, HT>;
  using TileP = Tile<T, CH, PS, HT>;
  using K = ChunkRows<T, NT, HT>;
  // q and the scores (forward) through LDS, or (512-byte rows: no room) straight into the output waves' registers
  static constexpr bool QLDS = !BWD && sizeof(T) * ND <= 256;
  static constexpr size_t N_BYTES = sizeof(T) * TileN::LDS_ELEMS, V_BYTES = sizeof(T) * TileP::LDS_ELEMS;
  static constexpr size_t K_BYTES = sizeof(T) * K::TileT::LDS_ELEMS;
  static constexpr size_t OFF_V = 2 * K_BYTES;
  static constexpr size_t OFF_Q = OFF_V + 2 * V_BYTES;
  static constexpr size_t OFF_P = OFF_Q + (QLDS ? 2 * N_BYTES : 0);
  static constexpr size_t OFF_XS = OFF_P + (QLDS ? 2 * 16 * FRAG_PIECES : 0);
  // what the state waves leave, twice where there is room: then nobody waits for the output waves to take it
  static constexpr int XBUF = BWD || (QLDS && NSW == 2) ? 2 : 1;
  static constexpr size_t OFF_XE = OFF_XS + XBUF * 16 * 64 * NSW * NT * 2;
  static constexpr size_t OFF_G = OFF_XE + XBUF * 16 * 64 * NSW * 4;
  // gates of the chunks in work: the staged one, the state waves' and (with one barrier) the output waves'
  static constexpr int GBUF = 2 * XBUF;
  static constexpr size_t LDS = OFF_G + GBUF * sizeof(float) * WALK_GATES * CH;
};

template <typename T, int NT, bool BWD, int NSW>
__global__ __launch_bounds__(64 * (NSW + (BWD && NSW == 2 ? 2 : NSW / 2) + 2)) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_delta_walk(Problem p) {
  using Cf = WalkCfg<T, NT, BWD, NSW>;
  using F = Fr<T>;
  using TileN = typename Cf::TileN;
  using TileP = typename Cf::TileP;
  constexpr int LDN = TileN::LD, LDP = TileP::LD, PS = Cf::PS, XB = Cf::XBUF - 1;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  auto kbuf = [&](int i) { return reinterpret_cast<T*>(smem + (i & 1) * Cf::K_BYTES); };
  auto vbuf = [&](int i) { return reinterpret_cast<T*>(smem + Cf::OFF_V + (i & 1) * Cf::V_BYTES); };
  auto qbuf = [&](int i) { return reinterpret_cast<T*>(smem + Cf::OFF_Q + (i & 1) * Cf::N_BYTES); };
  auto pbuf = [&](int i) { return reinterpret_cast<uint4*>(smem + Cf::OFF_P) + (i & 1) * FRAG_PIECES; };
  auto gbuf = [&](int i) { return reinterpret_cast<float*>(smem + Cf::OFF_G) + (i & (Cf::GBUF - 1)) * WALK_GATES * CH; };
  // from the state waves: the entering state's terms [wave][q][term][lane], and the residuals [wave][t][lane]
  auto xs = [&](int i) { return reinterpret_cast<uint4*>(smem + Cf::OFF_XS) + (i & XB) * 64 * NSW * NT * 2; };
  auto xe = [&](int i) { return reinterpret_cast<f32x4_t*>(smem + Cf::OFF_XE) + (i & XB) * 64 * NSW * 4; };

  const int np = (p.P + PS - 1) / PS;
  const Place at_block = place_of(p, np);
  const int h = at_block.h, ps = at_block.ps, seq = at_block.seq, grp = h / p.hpg;
  const int s0 = seq_start(p, seq), s1 = seq_start(p, seq + 1);
  const int nchunk = (s1 - s0 + CH - 1) / CH, slot0 = slot_base(s0, seq);
  const int tid = static_cast<int>(threadIdx.x), l = tid & 63, g = l >> 4, c = l & 15, w = ssd::wave_id_s();
  auto slot_head = [&](int i) { return static_cast<int64_t>(slot0 + i) * p.H + h; };
  auto length = [&](int i) { return min(CH, s1 - s0 - CH * i); };

  if (w < NSW) {
    // ---- state waves
    const int col = PS * ps + SLICE * w + c;   // this lane's value column
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
      auto gate = [&](int which, int row) { return *reinterpret_cast<const f32x4_t*>(gs + which * CH + row); };
      __syncthreads();   // the second barrier of the chunk before (at first: the first chunk is staged)
      typename F::X kf[4][NT];
      typename F::X4 vf[4];
      f32x4_t in[4];
#pragma unroll
      for (int q = 0; q < NT; ++q) {
#pragma unroll
        for (int t = 0; t < 4; ++t) kf[t][q] = Cf::K::rows(kt, t, q);
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        vf[t] = F::load4_raw(vt + SLICE * w, LDP, pair_col(t) + 8 * g);
        in[t] = gate(GATE_IN, pair_col(t) + 8 * g);
      }
      const float last = gs[GATE_IN * CH + CH - 1];
      if constexpr (XB == 0) __syncthreads();   // the output waves have taken what is overwritten now
#pragma unroll
      for (int q = 0; q < NT; ++q) {
        uint4 u[2];
        F::pieces(sf[q], u);
#pragma unroll
        for (int t = 0; t < 2; ++t) xs(i)[((w * NT + q) * 2 + t) * 64 + l] = u[t];
      }
      // r = v - exp(c) k S, rows in pair order; beside it the decay of S, and k's columns for the last product
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
#pragma unroll
        for (int j = 2 * q; j < 2 * q + 2; ++j) {
          S[j] *= last;
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) kc[j][ks] = Cf::K::cols(kt, j, ks);
        }
      }
      f32x4_t bo[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        x[t] = F::floats4(vf[t]) - in[t] * x[t];
        bo[t] = gate(GATE_BO, pair_col(t) + 8 * g);
      }
      // e = r + (T' - I) r
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
        for (int term = 0; term < 3; ++term) {
#pragma unroll
          for (int t = 2 * ks; t < 4; ++t) x[t] = mma_term(tf.get<T>(lower_frag(t, ks)), f2[ks], x[t], term);
        }
      }
      // S <- exp(c_last) S + k^T (beta exp(c_last - c) e), by halves of the chunk's rows: the first half's products run
      // while the second half is split, and of the second half's the last four tiles' while the first four are split
      // for the next chunk.  The next T' is requested piece by piece between them.
      const uint4* tnext = p.tf + slot_head(i + 1 < nchunk ? i + 1 : i) * FRAG_PIECES + l;
      auto correction = [&](int q) {
        xe(i)[(w * 4 + 2 * q) * 64 + l] = x[2 * q];
        xe(i)[(w * 4 + 2 * q + 1) * 64 + l] = x[2 * q + 1];
        float v[8];
        pair8(x[2 * q] * bo[2 * q], x[2 * q + 1] * bo[2 * q + 1], v);
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
    if (nchunk) __syncthreads();
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
    // ---- output waves: the columns of NZ state waves each
    constexpr int NZ = Cf::NZ;
    const int ow = w - NSW;
    const int col0 = PS * ps + NZ * SLICE * ow, slice0 = ps * NSW + NZ * ow;
    if constexpr (BWD) {
      auto keep = [&](int i) {
#pragma unroll
        for (int z = 0; z < NZ; ++z) {
          if (slice0 + z < p.nsl) {
            const int64_t at = slot_head(i) * p.nsl + slice0 + z;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
#pragma unroll
              for (int q = 0; q < NT; ++q) p.s[((at * 2 + t) * NT + q) * 64 + l] = xs(i)[(((NZ * ow + z) * NT + q) * 2 + t) * 64 + l];
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) p.e[(at * 4 + t) * 64 + l] = __builtin_bit_cast(uint4, xe(i)[((NZ * ow + z) * 4 + t) * 64 + l]);
          }
        }
      };
      __syncthreads();
      for (int i = 0; i < nchunk; ++i) {
        if (i > 0) keep(i - 1);   // left twice: the state waves are on the other one
        __syncthreads();
      }
      keep(nchunk - 1);
      return;
    }
    typename F::X xq[Cf::QLDS ? 1 : 4][NT];
    FragRegs pf;
    auto request_out = [&](int i) {
      if constexpr (!Cf::QLDS) {
        const int len = length(i);
        const int64_t row0 = static_cast<int64_t>(CH) * i;
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
    };
    uint4 us[NZ][NT][2];
    f32x4_t ee[NZ][4], be[4];
    float in[4];
    auto take = [&](int i) {
#pragma unroll
      for (int z = 0; z < NZ; ++z) {
#pragma unroll
        for (int q = 0; q < NT; ++q) {
#pragma unroll
          for (int t = 0; t < 2; ++t) us[z][q][t] = xs(i)[(((NZ * ow + z) * NT + q) * 2 + t) * 64 + l];
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) ee[z][t] = xe(i)[((NZ * ow + z) * 4 + t) * 64 + l];
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        in[t] = p.scale * gbuf(i)[GATE_IN * CH + 16 * t + c];
        be[t] = *reinterpret_cast<const f32x4_t*>(gbuf(i) + GATE_BETA * CH + pair_col(t) + 8 * g);
      }
    };
    auto out = [&](int i) {
      const int len = length(i);
      typename F::S uf[NZ][2];
#pragma unroll
      for (int z = 0; z < NZ; ++z) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float v[8];
          pair8(ee[z][2 * q] * be[2 * q], ee[z][2 * q + 1] * be[2 * q + 1], v);
          uf[z][q] = F::split(v);
        }
      }
      const T* qt = qbuf(i);
      const uint4* pt = pbuf(i);
      // o, transposed: rows are value columns 4 g + r, columns are chunk rows 16 t + c
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        f32x4_t acc[NZ];
#pragma unroll
        for (int z = 0; z < NZ; ++z) acc[z] = zero4();
#pragma unroll
        for (int q = 0; q < NT; ++q) {
          typename F::X x;
          if constexpr (Cf::QLDS) x = F::load(qt + (16 * t + c) * LDN + 32 * q + 8 * g);
          else x = xq[t][q];
#pragma unroll
          for (int z = 0; z < NZ; ++z) acc[z] = mma(F::from_pieces(us[z][q]), x, acc[z]);
        }
#pragma unroll
        for (int z = 0; z < NZ; ++z) acc[z] *= in[t];
#pragma unroll
        for (int ks = 0; ks <= (t >> 1); ++ks) {
          typename F::S sc;
          if constexpr (Cf::QLDS) sc = frag_at<T>(pt, lower_frag(t, ks));
          else sc = pf.get<T>(lower_frag(t, ks));
#pragma unroll
          for (int z = 0; z < NZ; ++z) acc[z] = mma(uf[z][ks], sc, acc[z]);
        }
#pragma unroll
        for (int z = 0; z < NZ; ++z) {
          const int cc = col0 + SLICE * z + 4 * g;
          if (16 * t + c < len && cc < p.P)
            ssd::store4f<T>(static_cast<T*>(p.o) + (s0 + static_cast<int64_t>(CH) * i + 16 * t + c) * hp + static_cast<int64_t>(h) * p.P + cc, acc[z]);
        }
      }
    };
    request_out(0);
    __syncthreads();
    for (int i = 0; i < nchunk; ++i) {
      if (i > 0) take(i - 1);
      if constexpr (XB == 0) __syncthreads();
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
  constexpr int GI = (WALK_GATES * CH + Cf::HT - 1) / Cf::HT;
  typename Cf::K::TileT tk;
  TileN tq;
  TileP tv;
  Pieces<FRAG_PIECES, Cf::HT> tp;
  float tg[GI];
  auto request_state = [&](int i) {
    const int64_t row = static_cast<int64_t>(CH) * i;
    tk.load(kp + row * p.k_sl, p.k_sl, length(i), p.N, ht);
    tv.load(vp + row * p.v_sl, p.v_sl, length(i), pcols, ht);
#pragma unroll
    for (int k = 0; k < GI; ++k) tg[k] = ht + k * Cf::HT < WALK_GATES * CH ? p.gates[slot_head(i) * (GATES * CH) + ht + k * Cf::HT] : 0.f;
  };
  auto stage_state = [&](int i) {
    tk.store(kbuf(i), ht);
    tv.store(vbuf(i), ht);
#pragma unroll
    for (int k = 0; k < GI; ++k)
      if (ht + k * Cf::HT < WALK_GATES * CH) gbuf(i)[ht + k * Cf::HT] = tg[k];
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
  __syncthreads();
  for (int i = 0; i < nchunk; ++i) {
    if constexpr (XB == 0) __syncthreads();
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
  return go(k_delta_prep<T, NT, BWD>, dim3(p.nslots, p.G * ((p.hpg + p.hb - 1) / p.hb)), 256, PrepCfg<BWD>::lds(p.hb), s, p);
}
template <typename T, int NT, bool BWD, int NSW> int walk_of(const Problem& p, hipStream_t s) {
  using Cf = WalkCfg<T, NT, BWD, NSW>;
  static_assert(Cf::LDS <= 160 * 1024, "LDS");
  return go(k_delta_walk<T, NT, BWD, NSW>, dim3(p.H * ((p.P + Cf::PS - 1) / Cf::PS), p.nseqs), Cf::THREADS, Cf::LDS, s, p);
}
// A CU holds one block (LDS).  Blocks of 32 value columns while they all fit the 256 CUs at once, of 64 above that
// (twice the columns on each CU for the same staging).  2048 rows of 128 x 64 columns (256 blocks of 32): 72 us with 32,
// 105 with 64 (backward 72, 89); 144 x 64: 127 and 100 (124, 99); twice 128 x 64: 144 and 113 (145, 117).  float32
// takes 32: in the backward 64 have no room in LDS (the forward alone would take 415 instead of 650 us at 144 x 64).
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
