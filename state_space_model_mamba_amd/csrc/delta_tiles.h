// Register tiles, fragments and staging shared by the gated delta kernels.
//
// Every product here is a 16x16 MFMA tile over 32 values of the contraction.
// A lane is (g, c) = (lane / 16, lane % 16).  An operand fragment holds, for
// row (A) or column (B) c, the 8 contraction values 8 g + e; the accumulator
// of a tile holds Out[4 g + r][c].  Two tiles whose A rows are taken in the
// order
//     row(t, m) = 32 (t / 2) + 8 (m / 4) + 4 (t % 2) + m % 4
// therefore hold, together, rows 32 q + 8 g + e of column c in lane (g, c):
// the layout of an operand fragment over those 32 rows, so a pair of
// accumulator tiles becomes the operand of the next product without leaving
// the lane (as B: contraction over its rows; as A: its transpose).
//
// With bf16 io, float32 values that feed a state or a gate's gradient enter
// a product as two bf16 terms, x = hi + lo + O(2^-16 |x|): one MFMA more per
// product with an exact bf16 operand, two more per product of two such values
// (lo * lo is dropped).  What is added to a state enters as three terms
// (2^-24): with two there, states come out 2.6e-6 off, with three 0.8e-6, and
// with single terms throughout 3e-3.  With f32 io every product is
// v_mfma_f32_16x16x4_f32.
#pragma once

#include <type_traits>

#include "delta_problem.h"
#include "ssd_device.h"
#include "ssd_tiles.h"

namespace delta {

using ssd::bf16_t;
using ssd::bf16x8_t;
using ssd::f32x4_t;
using ssd::pack_bf16x2;
using ssd::Vec16;
using ssd::zero4;

constexpr int CH = 64;   // rows of a chunk

typedef float f32x8_t __attribute__((ext_vector_type(8)));

__device__ __forceinline__ int perm_row(int t, int m) { return 32 * (t >> 1) + 8 * (m >> 2) + 4 * (t & 1) + (m & 3); }

// 8 contraction values of one row or column: X as given, S an fp32 value (bf16 io: hi and lo terms)
template <typename T> struct Fr;

template <> struct Fr<bf16_t> {
  typedef bf16x8_t X;
  struct S { bf16x8_t hi, lo; };
  struct S3 { bf16x8_t hi, mid, lo; };
  static __device__ __forceinline__ X zero() { return ssd::Mma<bf16_t>::zero(); }
  static __device__ __forceinline__ X load(const bf16_t* p) { return ssd::Mma<bf16_t>::load_k(p); }
  // of a row with `left` > 0 values from here on (a multiple of 16 bytes)
  static __device__ __forceinline__ X load_cols(const bf16_t* p, int) { return load(p); }
  // Rows row0 .. row0 + 3 of one column of a row-major LDS tile: column CS (c / 4) + c % 4 of base
  // (CS 4: 16 columns side by side; CS 8: the columns of a tile in pair order).
  template <int CS> static __device__ __forceinline__ ssd::s16x4_t tr4(const bf16_t* base, int ld, int row0) {
    const int c = static_cast<int>(threadIdx.x) & 15;
    return ssd::lds_read_tr16(base + (row0 + (c >> 2)) * ld + CS * (c & 3));
  }
  // rows row0 .. row0 + 7 of that column
  template <int CS = 4> static __device__ __forceinline__ X load_tr(const bf16_t* base, int ld, int row0) {
    union { ssd::s16x4_t h[2]; X x; } u;
    u.h[0] = tr4<CS>(base, ld, row0);
    u.h[1] = tr4<CS>(base, ld, row0 + 4);
    return u.x;
  }
  typedef ssd::s16x4_t X4;   // 4 rows of one column as they lie
  static __device__ __forceinline__ X4 load4_raw(const bf16_t* base, int ld, int row0) { return tr4<4>(base, ld, row0); }
  static __device__ __forceinline__ f32x4_t floats4(X4 v) {
    f32x4_t f;
#pragma unroll
    for (int r = 0; r < 4; ++r) f[r] = ssd::bf16_to_f32(static_cast<bf16_t>(v[r]));
    return f;
  }
  static __device__ __forceinline__ X round8(const float (&v)[8]) {
    uint4 u = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
    return __builtin_bit_cast(X, u);
  }
  static __device__ __forceinline__ S split(const float (&v)[8]) {
    S s;
    s.hi = round8(v);
    const uint4 u = __builtin_bit_cast(uint4, s.hi);
    float r[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r[2 * i] = v[2 * i] - __uint_as_float((&u.x)[i] << 16);
      r[2 * i + 1] = v[2 * i + 1] - __uint_as_float((&u.x)[i] & 0xffff0000u);
    }
    s.lo = round8(r);
    return s;
  }
  static __device__ __forceinline__ S3 split3(const float (&v)[8]) {
    S3 s;
    s.hi = round8(v);
    float h[8], r[8];
    floats(s.hi, h);
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = v[e] - h[e];
    const S t = split(r);
    s.mid = t.hi;
    s.lo = t.lo;
    return s;
  }
  static __device__ __forceinline__ void pieces(const S& s, uint4 (&u)[2]) {
    u[0] = __builtin_bit_cast(uint4, s.hi);
    u[1] = __builtin_bit_cast(uint4, s.lo);
  }
  static __device__ __forceinline__ S from_pieces(const uint4 (&u)[2]) {
    return S{__builtin_bit_cast(X, u[0]), __builtin_bit_cast(X, u[1])};
  }
  static __device__ __forceinline__ S terms(X first, X second) { return S{first, second}; }
  static __device__ __forceinline__ void floats(const S& s, float (&v)[8]) {
    const uint4 h = __builtin_bit_cast(uint4, s.hi), l = __builtin_bit_cast(uint4, s.lo);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float((&h.x)[i] << 16) + __uint_as_float((&l.x)[i] << 16);
      v[2 * i + 1] = __uint_as_float((&h.x)[i] & 0xffff0000u) + __uint_as_float((&l.x)[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void floats(X x, float (&v)[8]) {
    const uint4 h = __builtin_bit_cast(uint4, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float((&h.x)[i] << 16);
      v[2 * i + 1] = __uint_as_float((&h.x)[i] & 0xffff0000u);
    }
  }
};

template <> struct Fr<float> {
  typedef f32x8_t X;
  typedef f32x8_t S;
  typedef f32x8_t S3;
  static __device__ __forceinline__ X zero() { return X{0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}; }
  static __device__ __forceinline__ X load(const float* p) {
    union { f32x4_t h[2]; X x; } u;
    u.h[0] = *reinterpret_cast<const f32x4_t*>(p);
    u.h[1] = *reinterpret_cast<const f32x4_t*>(p + 4);
    return u.x;
  }
  static __device__ __forceinline__ X load_cols(const float* p, int left) {
    if (left > 4) return load(p);
    const f32x4_t v = *reinterpret_cast<const f32x4_t*>(p);
    return X{v[0], v[1], v[2], v[3], 0.f, 0.f, 0.f, 0.f};
  }
  template <int CS = 4> static __device__ __forceinline__ X load_tr(const float* base, int ld, int row0) {
    const int c = static_cast<int>(threadIdx.x) & 15;
    const float* p = base + row0 * ld + CS * (c >> 2) + (c & 3);
    X x;
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = p[e * ld];
    return x;
  }
  typedef f32x4_t X4;
  static __device__ __forceinline__ f32x4_t floats4(X4 v) { return v; }
  static __device__ __forceinline__ X4 load4_raw(const float* base, int ld, int row0) {
    const float* p = base + row0 * ld + (static_cast<int>(threadIdx.x) & 15);
    return f32x4_t{p[0], p[ld], p[2 * ld], p[3 * ld]};
  }
  static __device__ __forceinline__ S split(const float (&v)[8]) {
    S s;
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = v[e];
    return s;
  }
  static __device__ __forceinline__ S3 split3(const float (&v)[8]) { return split(v); }
  static __device__ __forceinline__ void pieces(const S& s, uint4 (&u)[2]) {
    u[0] = __builtin_bit_cast(uint4, f32x4_t{s[0], s[1], s[2], s[3]});
    u[1] = __builtin_bit_cast(uint4, f32x4_t{s[4], s[5], s[6], s[7]});
  }
  static __device__ __forceinline__ S from_pieces(const uint4 (&u)[2]) {
    const f32x4_t a = __builtin_bit_cast(f32x4_t, u[0]), b = __builtin_bit_cast(f32x4_t, u[1]);
    return S{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  }
  static __device__ __forceinline__ void floats(const S& s, float (&v)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = s[e];
  }
};

// acc += A B over the fragments' 32 contraction values
__device__ __forceinline__ f32x4_t mma(bf16x8_t a, bf16x8_t b, f32x4_t c) { return ssd::Mma<bf16_t>::mma(a, b, c); }
__device__ __forceinline__ f32x4_t mma(const Fr<bf16_t>::S& a, bf16x8_t b, f32x4_t c) { return mma(a.hi, b, mma(a.lo, b, c)); }
__device__ __forceinline__ f32x4_t mma(bf16x8_t a, const Fr<bf16_t>::S& b, f32x4_t c) { return mma(a, b.hi, mma(a, b.lo, c)); }
__device__ __forceinline__ f32x4_t mma(const Fr<bf16_t>::S& a, const Fr<bf16_t>::S& b, f32x4_t c) {
  return mma(a.hi, b.hi, mma(a.hi, b.lo, mma(a.lo, b.hi, c)));
}
__device__ __forceinline__ f32x4_t mma(bf16x8_t a, const Fr<bf16_t>::S3& b, f32x4_t c) {
  return mma(a, b.hi, mma(a, b.mid, mma(a, b.lo, c)));
}
__device__ __forceinline__ f32x4_t mma(const f32x8_t& a, const f32x8_t& b, f32x4_t c) {
#pragma unroll
  for (int e = 0; e < 8; ++e) c = ssd::Mma<float>::mma(a[e], b[e], c);
  return c;
}

// One term of a split operand's product at a time, smallest first, so that callers can run over independent tiles
// between the terms (a tile's own MFMAs depend on each other).
// exact A times split B: terms lo, hi
__device__ __forceinline__ f32x4_t mma_term(bf16x8_t a, const Fr<bf16_t>::S& b, f32x4_t c, int term) { return mma(a, term ? b.hi : b.lo, c); }
__device__ __forceinline__ f32x4_t mma_term(bf16x8_t a, const Fr<bf16_t>::S3& b, f32x4_t c, int term) {
  return mma(a, term == 0 ? b.lo : term == 1 ? b.mid : b.hi, c);
}
__device__ __forceinline__ f32x4_t mma_term(const Fr<bf16_t>::S& a, const Fr<bf16_t>::S& b, f32x4_t c, int term) {
  return term == 0 ? mma(a.lo, b.hi, c) : term == 1 ? mma(a.hi, b.lo, c) : mma(a.hi, b.hi, c);
}
// float32: the whole product, taken with the first term
__device__ __forceinline__ f32x4_t mma_term(const f32x8_t& a, const f32x8_t& b, f32x4_t c, int term) { return term ? c : mma(a, b, c); }

// What the backward keeps per slice of 16 value columns (states and their gradients) lies in memory as the
// lanes hold it, 16-byte pieces [half][q][lane]: piece (half, q) of lane (g, c) is column c's values 32 q + 8 g .. + 7
// (bf16; half: the term) or 32 q + 8 g + 4 half .. + 3 (float32).  A wave then stores and loads whole kilobytes;
// column by column they took 4 times as long in the memory pipeline.
//
// SLICES slices of such pieces as an LDS tile with a row for every value column and NQ * 32 values in it, by NTHR
// threads; slices >= nslices are zero and not read.
// (Float32: both halves.  bf16: one term, `base` at its first slice's.)
template <typename T, int SLICES, int NQ, int NTHR> struct SliceTile {
  static constexpr int HALVES = sizeof(T) / 2, PER = HALVES * NQ * 64, NV = SLICES * PER, IT = NV / NTHR;
  static constexpr int VEC = Vec16<T>::N, LD = NQ * 32 + VEC, LDS_ELEMS = SLICES * 16 * LD;
  static_assert(NTHR % PER == 0 && NV % NTHR == 0, "slices");
  f32x4_t buf[IT];
  // base: the first slice (uniform); pitch: pieces from one slice to the next.  A thread's pieces share their place in
  // the slice: one 32-bit lane offset, and a uniform base per piece.
  __device__ __forceinline__ void load(const uint4* base, int pitch, int nslices, int tid) {
    const uint32_t off = static_cast<uint32_t>(tid / PER * pitch + tid % PER) * 16u;
    const char* at = reinterpret_cast<const char*>(base);
#pragma unroll
    for (int k = 0; k < IT; ++k) {
      buf[k] = zero4();
      if (tid / PER + k * (NTHR / PER) < nslices) buf[k] = *reinterpret_cast<const f32x4_t*>(at + static_cast<int64_t>(k * (NTHR / PER) * 16) * pitch + off);
    }
  }
  __device__ __forceinline__ void store(T* lds, int tid) const {
#pragma unroll
    for (int k = 0; k < IT; ++k) {
      const int v = tid + k * NTHR, r = v % PER, l = r & 63, q = (r >> 6) % NQ, half = (r >> 6) / NQ;
      *reinterpret_cast<f32x4_t*>(lds + (v / PER * 16 + (l & 15)) * LD + 32 * q + 8 * (l >> 4) + 4 * half) = buf[k];
    }
  }
};

// a pair of accumulator tiles as 8 values in fragment order
__device__ __forceinline__ void pair8(f32x4_t a, f32x4_t b, float (&v)[8]) {
#pragma unroll
  for (int r = 0; r < 4; ++r) { v[r] = a[r]; v[4 + r] = b[r]; }
}

// first column of tile t among columns in pair order, for load_tr<8>
__device__ __forceinline__ constexpr int pair_col(int t) { return 32 * (t >> 1) + 4 * (t & 1); }

// A ROWS x COLS tile of rows `stride` elements apart, held in registers between its loads and its store
// to LDS by NTHR threads (tid: 0 .. NTHR - 1); rows >= nrows and columns >= ncols (a multiple of 16 bytes)
// are zero and not read.  A thread's pieces share their column and lie STEP rows apart, so a whole tile
// takes one vector offset and a uniform base per piece.
//
// SWZ (256-byte rows of bf16): no padding, and row r's 16-byte piece p lies at place p ^ (4 (r % 4) + r / 8 % 4).  The walks
// read such a tile by rows in pair order (16 rows at one piece) and by columns in pair order (4 rows at 4 pieces);
// with any padding one of the two meets itself in the banks 2 to 4 times, so placed neither does.
template <typename T, int ROWS, int COLS, int NTHR, bool SWZ = false> struct Tile {
  static constexpr int VEC = Vec16<T>::N, CV = COLS / VEC, STEP = NTHR / CV, IT = ROWS / STEP;
  static_assert(NTHR % CV == 0 && ROWS % STEP == 0, "tile");
  static_assert(!SWZ || (CV == 16 && STEP % 4 == 0 && (STEP == 4 || STEP == 8)), "swizzled tile");
  static constexpr int LD = SWZ ? COLS : COLS + VEC;   // row pitch in LDS: 16 bytes of padding
  static constexpr int LDS_ELEMS = ROWS * LD;
  f32x4_t buf[IT];
  // A lane's offset in its piece reaches over STEP rows: 32 bits hold it at the widest stride for up to 32 rows of bf16
  // or 16 of float32 (the walks' tiles), not for the 64 that 512 threads take of rows of 128 bytes.
  static constexpr bool WIDE = int64_t{STEP} * MAX_ROW_STRIDE * static_cast<int64_t>(sizeof(T)) > (int64_t{1} << 32);
  typedef typename std::conditional<WIDE, uint64_t, uint32_t>::type Offset;
  // base: uniform; stride <= MAX_ROW_STRIDE
  __device__ __forceinline__ void load(const T* base, int64_t stride, int nrows, int ncols, int tid) {
    const int r = tid / CV, cc = (tid % CV) * VEC;
    const Offset off = (static_cast<Offset>(r) * static_cast<Offset>(stride) + static_cast<Offset>(cc)) * static_cast<Offset>(sizeof(T));
    const char* at = reinterpret_cast<const char*>(base);
    const int64_t step = STEP * stride * static_cast<int64_t>(sizeof(T));
    if (nrows >= ROWS && ncols >= COLS) {
#pragma unroll
      for (int k = 0; k < IT; ++k) buf[k] = *reinterpret_cast<const f32x4_t*>(at + k * step + off);
    } else {
#pragma unroll
      for (int k = 0; k < IT; ++k) {
        buf[k] = zero4();
        if (r + k * STEP < nrows && cc < ncols) buf[k] = *reinterpret_cast<const f32x4_t*>(at + k * step + off);
      }
    }
  }
  __device__ __forceinline__ void store(T* lds, int tid) const {
    if constexpr (SWZ) {
      const int r = tid / CV, p = (tid % CV) ^ (4 * (r & 3));
#pragma unroll
      for (int k = 0; k < IT; ++k)   // rows r + k STEP: r / 8 % 4 is k's share alone
        *reinterpret_cast<f32x4_t*>(lds + (r + k * STEP) * LD + (p ^ (k * STEP / 8 & 3)) * VEC) = buf[k];
    } else {
      T* d = lds + (tid / CV) * LD + (tid % CV) * VEC;
#pragma unroll
      for (int k = 0; k < IT; ++k) *reinterpret_cast<f32x4_t*>(d + k * STEP * LD) = buf[k];
    }
  }
};

// A chunk's rows of k or q as the walks read them: operand fragments of tile t's rows in pair order (columns 32 q ..),
// and of tile j's columns in pair order (rows 32 ks ..)
template <typename T, int NT, int NTHR> struct ChunkRows {
  static constexpr bool SWZ = sizeof(T) == 2 && NT == 4;
  using TileT = Tile<T, CH, 32 * NT, NTHR, SWZ>;
  static __device__ __forceinline__ typename Fr<T>::X rows(const T* m, int t, int q) {
    const int l = static_cast<int>(threadIdx.x) & 63, g = l >> 4, c = l & 15;
    if constexpr (SWZ) return Fr<T>::load(m + perm_row(t, c) * TileT::LD + 8 * (4 * (q ^ (c & 3)) + (g ^ (c >> 2))));
    else return Fr<T>::load(m + perm_row(t, c) * TileT::LD + 32 * q + 8 * g);
  }
  static __device__ __forceinline__ typename Fr<T>::X cols(const T* m, int j, int ks) {
    const int l = static_cast<int>(threadIdx.x) & 63, g = l >> 4, c = l & 15;
    if constexpr (SWZ) {
      const T* at = m + (32 * ks + 8 * g + (c >> 2)) * TileT::LD + 8 * (4 * ((j >> 1) ^ (c >> 2)) + ((c & 3) ^ g)) + 4 * (j & 1);
      union { ssd::s16x4_t h[2]; typename Fr<T>::X x; } u;
      u.h[0] = ssd::lds_read_tr16(at);
      u.h[1] = ssd::lds_read_tr16(at + 4 * TileT::LD);
      return u.x;
    } else {
      return Fr<T>::template load_tr<8>(m + pair_col(j), TileT::LD, 32 * ks + 8 * g);
    }
  }
};

// The six fragments of a lower (tile t, step ks <= t / 2) triangular 64 x 64 operand, and of an upper one
// (ks >= t / 2): place of fragment (t, ks)
__device__ __forceinline__ constexpr int lower_frag(int t, int ks) { return t < 2 ? t : 2 * t - 2 + ks; }
__device__ __forceinline__ constexpr int upper_frag(int t, int ks) { return t < 2 ? 2 * t + ks : 2 + t; }
constexpr int NFRAG = 6;
constexpr int FRAG_PIECES = NFRAG * 2 * 64;   // 16-byte pieces of a split operand: [fragment][piece][lane]

// fragment f of a split operand's pieces in memory
template <typename T> __device__ __forceinline__ typename Fr<T>::S frag_at(const uint4* frags, int f) {
  const int l = static_cast<int>(threadIdx.x) & 63;
  const uint4 v[2] = {frags[2 * f * 64 + l], frags[(2 * f + 1) * 64 + l]};
  return Fr<T>::from_pieces(v);
}

// NV 16-byte pieces copied as they lie by NTHR threads
template <int NV, int NTHR> struct Pieces {
  static constexpr int IT = NV / NTHR;
  static_assert(NV % NTHR == 0, "pieces");
  f32x4_t buf[IT];
  __device__ __forceinline__ void load(const uint4* p, int tid) {
#pragma unroll
    for (int k = 0; k < IT; ++k) buf[k] = reinterpret_cast<const f32x4_t*>(p)[tid + k * NTHR];
  }
  __device__ __forceinline__ void store(uint4* lds, int tid) const {
#pragma unroll
    for (int k = 0; k < IT; ++k) reinterpret_cast<f32x4_t*>(lds)[tid + k * NTHR] = buf[k];
  }
};

// a split operand's fragments in registers, requested from global memory ahead of their use
struct FragRegs {
  uint4 u[2 * NFRAG];
  __device__ __forceinline__ void request(const uint4* frags) {
    const int l = static_cast<int>(threadIdx.x) & 63;
#pragma unroll
    for (int i = 0; i < 2 * NFRAG; ++i) u[i] = frags[i * 64 + l];
  }
  template <typename T> __device__ __forceinline__ typename Fr<T>::S get(int f) const {
    const uint4 v[2] = {u[2 * f], u[2 * f + 1]};
    return Fr<T>::from_pieces(v);
  }
};

}  // namespace delta
