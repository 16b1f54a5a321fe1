// gdn2_linattn_impl.h -- the sweep kernels of the linear attention with a decay for each head.
//
// The recurrence, per (sequence, head), with g = exp(log_decay) and Z an A x E matrix:
//     Z_t = g Z_{t-1} + y_t z_t^T          r_t = Z_t^T x_t
// Over a chunk of C tokens that Z enters (i, j count its tokens, f = `first`):
//     r_i = sum_{j<=i} g^(i-j) (x_i . y_j) z_j + g^(i+f) Z^T x_i
//     Z  <- g^n Z + sum_j g^(n-f-j) y_j z_j^T                          (n valid tokens, n = C but for a last chunk)
// f = 1 is the forward recurrence; f = 0 is the reversed one of the backward, whose state holds g times the
// gradient of the state (so the gradient of the last state enters as it is). Every power of g has an exponent
// >= 0, so nothing overflows for g <= 1 whatever the decay, and no quotient of decays is formed.
//
// Work: one workgroup per (sequence, head, piece, column group of E), which walks its piece chunk by chunk. Per chunk
// x, y, z go to LDS and the C x C scores are formed once; each wave of the state owns 16 of its columns in fp32
// accumulators and forms its columns of r = scores z + decayed x Z and of the state update.
//
// Operands. A 16x16 accumulator tile holds rows 4g+r of column l%16 (g = l/16), and either operand of a product
// takes 8 contraction indices (16 bit; fp32: 4) of row or column l%16 from a lane. State tiles 2u, 2u+1 hold the
// state rows 32u + 8g + r and 32u + 8g + 4 + r (fp32: tile u rows 16u + 4g + r), which is the contraction order
// that x is read in from LDS with one 16-byte access, so the state enters its product from the registers it is
// kept in. The contraction over tokens reads y and z column-wise with the transposing LDS read (16 bit).
//
// What bounds it (B8 H16 T4096 d128 bf16, 256 workgroups, one a CU): 180 us, 3.0 TB/s of the 0.54 GB that it has to read
// and write, once each by the counters (a copy: 5.2 TB/s, 105 us). Nothing is full: of the SIMDs' time vector
// instructions take 44 %, the matrix cores 29 %; LDS is busy for 32 %, a quarter of that in conflicts. The waves wait
// for 39 % of their time (5 % for LDS instructions) and for 20 % to issue. With two bf16 terms for scores and states the
// loads alone took 98 us, the state's waves with their data at hand 126, together 157: with one workgroup a CU, one wave
// of the state a SIMD and a barrier a chunk the two cover each other in part. So the work is split by role: the state's
// waves never wait for memory (two terms: 249 us with one role, 161 with loading waves that also form the scores). 64K
// tokens of one sequence: 490-499 us, 2.2 TB/s of 1.07 GB: y and z are read a second time, for the pieces' states.
// Comparisons of 160 to 167 us below were measured with two terms.
//
// Precision (16-bit inputs): products of two inputs are exact in the matrix cores' fp32 sums. The scores, the decayed
// z and the state as an operand are split into three bf16 terms each, which hold an fp32 value's 24 bits: r and the
// states are fp32 sums of unrounded products, and r is rounded once, at the end.
#pragma once

#include <type_traits>

#include "gdn2_common.h"
#include "gdn2_linattn.h"

namespace gdn2 {

// 2^(l2 n) with the exponent reduced in fp64: one fp32 rounding for any n (n >= 0)
__device__ __forceinline__ float decay_pow(double l2, int n) {
  const double e = l2 * n, r = rint(e);
  return ldexpf(__builtin_amdgcn_exp2f((float)(e - r)), (int)fmax(r, -4096.0));
}

// log2 of the decay; -1e4 stands for anything smaller (its powers are zero in fp32 from the first on), so that
// exponent 0 gives 1 for a decay of zero too. NaN stays.
__device__ __forceinline__ double decay_log2(float l) {
  const double x = l < -1e4f ? -1e4 : (double)l;
  return x * 1.4426950408889634074;
}

// Matrix operand types. unit: the contraction indices of one operand register group.
template <bool F32>
struct LinOp {
  using T = typename std::conditional<F32, float, __bf16>::type;
  using V = typename std::conditional<F32, f32x4, bf16x8>::type;
  static constexpr int KU = F32 ? 16 : 32;
  static constexpr int C = F32 ? 32 : 64;       // tokens a chunk
  static constexpr int ES = F32 ? 4 : 2;        // bytes an element
};

__device__ __forceinline__ void lin_mma(f32x4& acc, const bf16x8& a, const bf16x8& b) { acc = mfma16x16x32(a, b, acc); }
__device__ __forceinline__ void lin_mma(f32x4& acc, const f32x4& a, const f32x4& b) {
#pragma unroll
  for (int i = 0; i < 4; ++i) acc = mfma16x16x4(a[i], b[i], acc);
}

// A tile [rows][W] of the inputs' type in LDS: row after row, the 16-byte blocks of a row permuted so that what the
// lanes served together touch lies in different banks (64 of 4 bytes for reads: 16 blocks wide; 16-byte reads are
// served 16 lanes at a time, 8-byte ones 32, 4-byte ones 64). How a tile is read decides which bits of the row go
// where; rows narrower than 16 blocks share the banks' width, which separates their lowest bits already:
//   kRows: 16 bytes of 16 neighbouring rows (x, the scores);
//   kBoth: that, and, 16 bit, 8 bytes of rows 0-3 and 8-11 of 16, in 4 neighbouring blocks each (the transposing read
//          of y). The latter meets itself once in its banks; exchanging the halves of a block in some rows avoids
//          that, but costs more vector instructions than it saves (forward 160 us either way);
//   kCols: 16 bit: 32 bytes of rows 0-3 and 8-11 (z).
// fp32 reads down the rows 4 bytes wide: 16 columns of rows 4 apart.
enum LinUse { kRows, kBoth, kCols };

template <bool F32, int W, LinUse USE>
struct LinTile {
  using Op = LinOp<F32>;
  using V = typename Op::V;
  static constexpr int kRow = W * Op::ES;       // bytes a row
  static constexpr int NB = kRow / 16;          // blocks a row
  __device__ __forceinline__ static int bit(int r, int from, int to) { return ((r >> from) & 1) << to; }
  __device__ __forceinline__ static int perm(int r) {
    if constexpr (F32) return NB >= 16 ? (r & 15) : NB == 8 ? bit(r, 2, 2) | bit(r, 3, 1) | bit(r, 1, 0) : (r >> 2) & 3;
    else if constexpr (USE == kRows) return NB >= 16 ? (r & 15) : NB == 8 ? (r >> 1) & 7 : (r >> 2) & 3;
    else if constexpr (USE == kBoth)
      return NB >= 16 ? bit(r, 3, 3) | bit(r, 0, 2) | bit(r, 1, 1) | bit(r, 2, 0)
             : NB == 8 ? bit(r, 3, 2) | bit(r, 1, 1) | bit(r, 2, 0) : bit(r, 3, 1) | bit(r, 2, 0);
    else
      return NB >= 16 ? bit(r, 3, 3) | bit(r, 1, 2) | bit(r, 0, 1) : NB == 8 ? bit(r, 3, 2) | bit(r, 1, 1)
             : NB == 4 ? bit(r, 3, 1) : 0;
  }
  // byte offset of block b of row r
  __device__ __forceinline__ static int at(int r, int b) { return r * kRow + ((b ^ perm(r)) << 4); }
  // operand of unit u from row r (contraction along the row), lane group g
  __device__ __forceinline__ static V row(const char* t, int r, int u, int g) {
    return *reinterpret_cast<const V*>(t + at(r, 4 * u + g));
  }
  // Operand whose contraction runs down the rows, 16 bit: 32u + 8g .. + 7, fp32: 16u + 4g .. + 3, of 16 columns.
  // 16 bit: the read takes, for every 16 lanes, 4 rows x 16 columns, lane 4 e + p giving the address of row e,
  // columns 4p..4p+3, and hands lane i column i of the four rows.
  // y: the columns 4p..4p+3 are half h of block b0 + p; z: the 16 columns from block b0 on.
  __device__ __forceinline__ static V col(const char* t, int u, int g, int i, int b0, int h) {
    if constexpr (F32) {
      f32x4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        v[e] = *reinterpret_cast<const float*>(t + at(16 * u + 4 * g + e, b0 + (i >> 2)) + 4 * (i & 3));
      return v;
    } else {
      const int r = 32 * u + 8 * g + (i >> 2), p = i & 3;
      const int b = USE == kBoth ? b0 + p : b0 + (p >> 1), half = 8 * (USE == kBoth ? h : p & 1);
      typedef __attribute__((address_space(3))) bf16x4 lds4;
      const bf16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds4*)(t + at(r, b) + half));
      const bf16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds4*)(t + at(r + 4, b) + half));
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
  }
};

// A chunk's rows of one tensor on their way from HBM to LDS: 16 bytes a thread and pass, NTH threads.
template <bool F32, int W, int WP, LinUse USE, int NTH>
struct LinFetch {
  using Op = LinOp<F32>;
  using Tile = LinTile<F32, WP, USE>;
  static constexpr int NB = W * Op::ES / 16;              // blocks a row in memory
  static constexpr int TOTAL = NB * Op::C;
  static constexpr int NP = (TOTAL + NTH - 1) / NTH;
  static constexpr int RP = NTH / NB;                     // rows a pass
  static_assert(NTH % NB == 0, "a pass takes whole rows");
  using Data = uint4[NP];
  const char* next;      // this thread's address in the chunk that is fetched next, pass 0
  int64_t step;          // bytes from row to row of the walk
  int row, tid;
  // head: this head's first element of token 0; the walk's row 0 is tok0
  __device__ __forceinline__ void begin(const char* head, int64_t row_bytes, int64_t tok0, int dir, int pos0, int t) {
    tid = t;
    row = t / NB;
    step = dir * row_bytes;
    next = head + tok0 * row_bytes + (pos0 + row) * step + (t % NB) * 16;
  }
  // the next chunk's rows, `valid` of them in the sequence; rows past them repeat the last
  __device__ __forceinline__ void load(Data& v, int valid) {
    if (valid >= Op::C) {
#pragma unroll
      for (int p = 0; p < NP; ++p)
        if (TOTAL % NTH == 0 || row + p * RP < Op::C) v[p] = *reinterpret_cast<const uint4*>(next + p * RP * step);
    } else {
#pragma unroll
      for (int p = 0; p < NP; ++p)
        v[p] = *reinterpret_cast<const uint4*>(next + (min(row + p * RP, valid - 1) - row) * step);
    }
    next += Op::C * step;
  }
  // rows past `valid` are zeros
  __device__ __forceinline__ void store(Data& v, char* tile, int valid) {
    if (valid < Op::C) {
#pragma unroll
      for (int p = 0; p < NP; ++p)
        if (row + p * RP >= valid) v[p] = make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int p = 0; p < NP; ++p)
      if (TOTAL % NTH == 0 || row + p * RP < Op::C)
        *reinterpret_cast<uint4*>(tile + Tile::at(row + p * RP, tid % NB)) = v[p];
  }
  // any element of the valid rows is an infinity or NaN (after store)
  __device__ __forceinline__ bool non_finite(const Data& v) const {
    uint32_t odd = 0;
#pragma unroll
    for (int p = 0; p < NP; ++p)
      if (TOTAL % NTH == 0 || row + p * RP < Op::C) {
        const uint32_t w[4] = {v[p].x, v[p].y, v[p].z, v[p].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)  // an exponent of all ones carries into the sign's place
          odd |= F32 ? (w[j] & 0x7f800000u) + 0x00800000u : (w[j] & 0x7f807f80u) + 0x00800080u;
      }
    return (odd & (F32 ? 0x80000000u : 0x80008000u)) != 0;
  }
};

__device__ __forceinline__ bf16x8 pack_hi(const float (&x)[8]) {  // the upper halves: bf16 by truncation
  u32x4 w;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    w[j] = __builtin_amdgcn_perm(__float_as_uint(x[2 * j + 1]), __float_as_uint(x[2 * j]), 0x07060302u);
  return __builtin_bit_cast(bf16x8, w);
}
__device__ __forceinline__ void sub_hi(float (&x)[8]) {           // what truncation left
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] -= __uint_as_float(__float_as_uint(x[j]) & 0xffff0000u);
}
// x in three bf16 terms, the largest first: 8 bits of it each, all of it together. x is used up.
__device__ __forceinline__ void lin_split(float (&x)[8], bf16x8 (&t)[3]) {
  t[0] = pack_hi(x);
  sub_hi(x);
  t[1] = pack_hi(x);
  sub_hi(x);
  t[2] = pack_hi(x);
}

// infinities and NaN replaced by zeros
__device__ __forceinline__ void lin_finite(bf16x8& x) {
  u32x4 w = __builtin_bit_cast(u32x4, x);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if ((w[j] & 0x7f800000u) == 0x7f800000u) w[j] &= 0xffffu;
    if ((w[j] & 0x7f80u) == 0x7f80u) w[j] &= 0xffff0000u;
  }
  x = __builtin_bit_cast(bf16x8, w);
}
__device__ __forceinline__ void lin_finite(f32x4& x) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if ((__float_as_uint(x[j]) & 0x7f800000u) == 0x7f800000u) x[j] = 0.f;
}

constexpr int kLinLoad = 4;  // waves that load and form the scores

template <int A, int NW, bool F32>
struct LinShape {
  using Op = LinOp<F32>;
  static constexpr int AP = A < Op::KU ? Op::KU : A;  // channels of x, y in LDS (16-bit: at least one unit)
  static constexpr int CW = 16 * NW;                  // columns a workgroup
  static constexpr int kXY = Op::C * AP * Op::ES;
  static constexpr int kZ = Op::C * CW * Op::ES;
  static constexpr int kP = Op::C * Op::C * Op::ES;
  static constexpr int kThreads = 64 * (NW + kLinLoad);
  static constexpr int kBuf = kXY + kZ, kBufX = 2 * kXY + kZ;  // y, z; y, z, x
  static constexpr int kScores = F32 ? kP : 2 * kP + kP / 4;
  // three buffers of a chunk's rows, two of its scores, flags; the sums of the pieces: two buffers
  static constexpr int kLds = 3 * kBufX + 2 * kScores + 3 * 4 * kLinLoad;
  static constexpr int kLdsState = 2 * kBuf;
  static_assert(kLds <= 160 * 1024, "a CU's LDS");
};

// What a workgroup has to do. Returns false where there is nothing.
struct LinTask {
  int n, h, seg, nseg, slot;
  int64_t tok0;    // row of the walk's first token
  int len, pos0, pos1;
};

// The scores of a chunk in LDS, 16 bit: a tile for the first terms, one for the second. Tokens of the first half of a
// chunk have no scores with the second half's, so a quarter of each tile is free: the third terms of the first half's
// rows lie in the first tile's, those of the second half's rows with the first half's tokens in the second tile's, the
// rest in a tile of their own (three whole tiles, twice, would not fit beside the rows).
struct LinScores {
  static constexpr int C = LinOp<false>::C, kTile = C * C * 2;
  using T = LinTile<false, C, kRows>;
  using Rest = LinTile<false, C / 2, kRows>;
  // byte offset of term n of block b of row r
  __device__ __forceinline__ static int at(int n, int r, int b) {
    constexpr int H = C / 2, HB = C / 16;  // half a chunk: rows, blocks
    if (n < 2) return n * kTile + T::at(r, b);
    if (r < H) return T::at(r, b + HB);
    return b < HB ? kTile + T::at(r - H, b + HB) : 2 * kTile + Rest::at(r - H, b - HB);
  }
};

__device__ __forceinline__ bool lin_task(const LinArgs& a, int item, bool rev, LinTask& t) {
  // items: head fastest, then sequence (dense), then piece
  t.h = item % a.H;
  int rest = item / a.H;
  int64_t begin;
  if (a.cu) {
    if (rest >= a.max_segs) return false;
    t.slot = rest;
    t.n = a.seg_seq[rest];
    if (t.n < 0) return false;
    t.seg = rest - a.seg_first[t.n];
    t.nseg = a.seg_first[t.n + 1] - a.seg_first[t.n];
    begin = a.cu[t.n];
    t.len = (int)(a.cu[t.n + 1] - begin);
  } else {
    if (rest >= a.max_segs * a.N) return false;
    t.n = rest % a.N;
    t.seg = rest / a.N;
    t.slot = t.seg * a.N + t.n;
    t.nseg = a.max_segs;
    begin = (int64_t)t.n * a.T;
    t.len = a.T;
  }
  t.tok0 = rev ? begin + t.len - 1 : begin;
  t.pos0 = t.seg * a.seg_tok;
  t.pos1 = min(t.len, t.pos0 + a.seg_tok);
  return true;
}

// Block -> (item, sweep, column group): a head's column groups and sweeps take workgroups 8 apart, so that they run on
// one XCD and read what they share through its L2 once.
__device__ __forceinline__ void lin_block(int ncg, int sweeps, int& item, int& sweep, int& cg) {
  const int xcd = blockIdx.x & 7, slot = blockIdx.x >> 3, per = ncg * sweeps;
  item = (slot / per) * 8 + xcd;
  sweep = slot % per / ncg;
  cg = slot % ncg;
}

// State row of accumulator tile m, lane group g, element r.
template <bool F32>
__device__ __forceinline__ int lin_state_row(int m, int g, int r) {
  return F32 ? 16 * m + 4 * g + r : 32 * (m >> 1) + 8 * g + 4 * (m & 1) + r;
}

// The loading waves: the rows of a chunk from memory to LDS, and the scores of a chunk in LDS.
template <int A, int NW, bool F32, bool STATE>
struct LinLoader {
  using Sh = LinShape<A, NW, F32>;
  using Op = LinOp<F32>;
  using V = typename Op::V;
  static constexpr int C = Op::C, UK = Sh::AP / Op::KU, TT = C / 16;
  using TX = LinTile<F32, Sh::AP, kRows>;
  using TY = LinTile<F32, Sh::AP, kBoth>;
  using TP = LinTile<F32, C, kRows>;
  LinFetch<F32, A, Sh::AP, kRows, 64 * kLinLoad> fx;
  LinFetch<F32, A, Sh::AP, kBoth, 64 * kLinLoad> fy;
  LinFetch<F32, Sh::CW, Sh::CW, kCols, 64 * kLinLoad> fz;
  float pd[4], pm[4], g16;

  // a chunk's rows in registers
  struct Rows {
    typename decltype(fx)::Data x, y;
    typename decltype(fz)::Data z;
  };

  __device__ __forceinline__ void load(Rows& r, int valid) {
    if constexpr (!STATE) fx.load(r.x, valid);
    fy.load(r.y, valid);
    fz.load(r.z, valid);
  }
  __device__ __forceinline__ void store(Rows& r, char* buf, int* flags, int w, int valid) {
    fy.store(r.y, buf, valid);
    fz.store(r.z, buf + Sh::kXY, valid);
    if constexpr (!STATE) {
      fx.store(r.x, buf + Sh::kBuf, valid);
      const bool odd = __any(fz.non_finite(r.z));
      if (lane_id() == 0) flags[w] = odd;
    }
  }
  // The n-th score tile of wave w, strip ts against strip jt <= ts, at most three a wave:
  //   w = 0: (3,3) (3,2)   1: (3,1) (3,0) (0,0)   2: (2,2) (2,1) (2,0)   3: (1,1) (1,0)      (chunks of four strips)
  //   w = 0: (1,1)         1: (1,0)               2: (0,0)                                  (two strips)
  static constexpr int strip(int w, int n) {
    return TT == 4 ? (w == 0 ? 3 : w == 1 ? (n < 2 ? 3 : 0) : 4 - w) : (w < 2 ? 1 : 0);
  }
  static constexpr int against(int w, int n) {
    return TT == 4 ? (w == 0 ? 3 - n : w == 1 ? (n < 2 ? 1 - n : 0) : 4 - w - n) : (w == 0 ? 1 : 0);
  }
  static constexpr int tiles(int w) { return TT == 4 ? (w == 1 || w == 2 ? 3 : 2) : (w < 3 ? 1 : 0); }
  __device__ __forceinline__ void scores(const char* buf, char* tp, int w, int g, int i) {
    switch (w) {  // one code a wave: its tiles' places are constants
      case 0: return scores_of<0>(buf, tp, g, i);
      case 1: return scores_of<1>(buf, tp, g, i);
      case 2: return scores_of<2>(buf, tp, g, i);
      default: return scores_of<3>(buf, tp, g, i);
    }
  }
  // scores, transposed: tile (jt, ts) holds tokens j = 16 jt + 4g + r of columns i = 16 ts + l%16
  template <int W>
  __device__ __forceinline__ void scores_of(const char* buf, char* tp, int g, int i) {
    const char* const ty = buf;
    const char* const tx = buf + Sh::kBuf;
    V xv[UK];
#pragma unroll
    for (int n = 0; n < tiles(W); ++n) {
      const int ts = strip(W, n), jt = against(W, n);
      if (n == 0 || ts != strip(W, n - 1)) {
#pragma unroll
        for (int u = 0; u < UK; ++u) xv[u] = TX::row(tx, 16 * ts + i, u, g);
      }
      f32x4 p = zero4(), p2 = zero4();  // two sums side by side: half the wait for one another
#pragma unroll
      for (int u = 0; u < UK; ++u)
        lin_mma((u & 1) ? p2 : p, TY::row(ty, 16 * jt + i, u, g), xv[u]);
      if (ts == jt) {
#pragma unroll
        for (int r = 0; r < 4; ++r) p[r] = i >= 4 * g + r ? (p[r] + p2[r]) * pd[r] : 0.f;
      } else {
        const float far = ts - jt == 1 ? 1.f : ts - jt == 2 ? g16 : g16 * g16;
#pragma unroll
        for (int r = 0; r < 4; ++r) p[r] = (p[r] + p2[r]) * (pm[r] * far);
      }
      if constexpr (F32) {
        *reinterpret_cast<f32x4*>(tp + TP::at(16 * ts + i, 4 * jt + g)) = p;
      } else {
        // in three terms; a unit has 32 tokens: zeros in the tile past the diagonal of an even strip
        const int row = 16 * ts + i, half = 8 * (g & 1);
#pragma unroll
        for (int t2 = 0; t2 < 3; ++t2) {
          uint2 w;
          w.x = __builtin_amdgcn_perm(__float_as_uint(p[1]), __float_as_uint(p[0]), 0x07060302u);
          w.y = __builtin_amdgcn_perm(__float_as_uint(p[3]), __float_as_uint(p[2]), 0x07060302u);
          *reinterpret_cast<uint2*>(tp + LinScores::at(t2, row, 2 * jt + (g >> 1)) + half) = w;
          if (ts == jt && (ts & 1) == 0)
            *reinterpret_cast<uint2*>(tp + LinScores::at(t2, row, 2 * (ts + 1) + (g >> 1)) + half) = make_uint2(0u, 0u);
#pragma unroll
          for (int r = 0; r < 4; ++r) p[r] -= __uint_as_float(__float_as_uint(p[r]) & 0xffff0000u);
        }
      }
    }
  }
};

// STATE: the sum of one piece alone, from a zero state (x, r unused), stored as the entering state of the next
// piece for the join kernel. Otherwise the sweep of one piece.
//
// The first NW waves hold the state, the other kLinLoad work ahead of them: in the step in which the state's waves take
// chunk s, they write chunk s + 2 to LDS, send for chunk s + 3 and form the scores of chunk s + 1 (which do not depend
// on the state), with one barrier a step; in this order the rows are on their way while the scores are formed (161 us
// against 167 for a B8 H16 T4096 d128 forward). (STATE: no scores, chunk s + 1 to LDS, s + 2 sent for.)
template <int A, int NW, bool F32, bool STATE>
__global__ __launch_bounds__((LinShape<A, NW, F32>::kThreads), 2) void gdn2_linattn_kernel(LinArgs a) {
  using Sh = LinShape<A, NW, F32>;
  using Op = LinOp<F32>;
  using V = typename Op::V;
  constexpr int C = Op::C, KU = Op::KU, ES = Op::ES, AP = Sh::AP, CW = Sh::CW;
  constexpr int RT = AP / 16, UK = AP / KU, UC = C / KU, TT = C / 16, EZ = F32 ? 4 : 8;
  constexpr int BUF = STATE ? Sh::kBuf : Sh::kBufX;
  using TX = LinTile<F32, AP, kRows>;
  using TY = LinTile<F32, AP, kBoth>;
  using TZ = LinTile<F32, CW, kCols>;
  using TP = LinTile<F32, C, kRows>;

  extern __shared__ char lds[];  // a buffer: y, z, x
  char* const scores = lds + 3 * BUF;  // two buffers
  int* const flags = reinterpret_cast<int*>(scores + 2 * Sh::kScores);  // [3][kLinLoad]: z has an infinity or NaN

  const int ncg = (a.E + CW - 1) / CW;
  int item, sweep, cg;
  lin_block(ncg, a.sweeps, item, sweep, cg);
  const LinSweep& sw = a.sw[sweep];
  LinTask t;
  if (!lin_task(a, item, sw.rev, t)) return;
  if (STATE && t.seg + 1 >= t.nseg) return;

  const int l = lane_id(), g = l >> 4, i = l & 15;
  const int w = __builtin_amdgcn_readfirstlane(wave_id());
  const int dir = sw.rev ? -1 : 1;
  const int E = a.E;
  const int steps = (t.pos1 - t.pos0 + C - 1) / C;
  const double l2 = decay_log2(a.log_decay[t.h]);

  if constexpr (A < AP) {  // the channels that pad x and y to a unit are zero throughout
    constexpr int tiles = STATE ? 2 : 6;
    for (int id = threadIdx.x; id < tiles * C * 2; id += Sh::kThreads) {
      const int row = (id >> 1) & (C - 1), b = 2 + (id & 1), tile = id / (2 * C);
      const bool x = !STATE && (tile & 1);
      char* const at = STATE ? lds + tile * BUF : lds + (tile >> 1) * BUF + (x ? Sh::kBuf : 0);
      *reinterpret_cast<uint4*>(at + (x ? TX::at(row, b) : TY::at(row, b))) = make_uint4(0, 0, 0, 0);
    }
  }

  if (w >= NW) {
    const int lw = w - NW, tid = threadIdx.x - 64 * NW;
    const int64_t rbx = (int64_t)(a.H / sw.xdiv) * A * ES, rby = (int64_t)(a.H / sw.ydiv) * A * ES;
    const int64_t rbz = (int64_t)(a.H / sw.zdiv) * E * ES;
    LinLoader<A, NW, F32, STATE> ld;
    if constexpr (!STATE)
      ld.fx.begin(static_cast<const char*>(sw.x) + (int64_t)(t.h / sw.xdiv) * A * ES, rbx, t.tok0, dir, t.pos0, tid);
    ld.fy.begin(static_cast<const char*>(sw.y) + (int64_t)(t.h / sw.ydiv) * A * ES, rby, t.tok0, dir, t.pos0, tid);
    ld.fz.begin(static_cast<const char*>(sw.z) + ((int64_t)(t.h / sw.zdiv) * E + cg * CW) * ES, rbz, t.tok0, dir,
                t.pos0, tid);
    auto valid = [&](int s) { return min(C, t.pos1 - (t.pos0 + s * C)); };
    typename decltype(ld)::Rows rows;
    ld.load(rows, valid(0));
    if constexpr (!STATE) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {  // token i of its tile against token 4g + r of the same tile, of the one before
        const int d = i - 4 * g - r;
        ld.pd[r] = d >= 0 ? sw.si * sw.so * decay_pow(l2, d) : 0.f;
        ld.pm[r] = sw.si * sw.so * decay_pow(l2, 16 + d);
      }
      ld.g16 = decay_pow(l2, 16);
    }
    ld.store(rows, lds, flags, lw, valid(0));
    if (steps > 1) ld.load(rows, valid(1));
    if constexpr (STATE) {
      __syncthreads();
      for (int s = 0; s < steps; ++s) {
        if (s + 1 < steps) ld.store(rows, lds + ((s + 1) & 1) * BUF, flags, lw, valid(s + 1));
        if (s + 2 < steps) ld.load(rows, valid(s + 2));
        __syncthreads();
      }
    } else {
      if (steps > 1) ld.store(rows, lds + BUF, flags + kLinLoad, lw, valid(1));
      if (steps > 2) ld.load(rows, valid(2));
      __syncthreads();
      ld.scores(lds, scores, lw, g, i);
      __syncthreads();
      int next = 1, after = 2;  // buffers of chunks s + 1, s + 2
      for (int s = 0; s < steps; ++s) {
        if (s + 2 < steps) ld.store(rows, lds + after * BUF, flags + after * kLinLoad, lw, valid(s + 2));
        if (s + 3 < steps) ld.load(rows, valid(s + 3));
        if (s + 1 < steps) ld.scores(lds + next * BUF, scores + ((s + 1) & 1) * Sh::kScores, lw, g, i);
        next = after;
        after = after == 2 ? 0 : after + 1;
        __syncthreads();
      }
    }
    return;
  }

  const int c0 = 16 * w, e0 = cg * CW + c0;  // this wave's first column in the tile, in the state
  float cz[UC][EZ];                          // powers of the decay in the update, token KU u + EZ g + e
  auto set_cz = [&](int n) {
#pragma unroll
    for (int u = 0; u < UC; ++u)
#pragma unroll
      for (int e = 0; e < EZ; ++e) cz[u][e] = sw.si * decay_pow(l2, max(0, n - sw.first - (KU * u + EZ * g + e)));
  };
  set_cz(C);
  // g^n, and what rounding left of it: a state decays by the same rounded g^C at every chunk, off to the same side
  auto chunk_decay = [&](int n, float& hi, float& rest) {
    const double x = exp2(l2 * n);
    hi = (float)x;
    rest = hi <= 3.4028235e38f ? (float)(x - hi) : 0.f;
  };
  float gC, gRest;
  chunk_decay(C, gC, gRest);
  float ro[TT];
  if constexpr (!STATE) {
#pragma unroll
    for (int k = 0; k < TT; ++k) ro[k] = sw.so * decay_pow(l2, 16 * k + i + sw.first);
  }

  // the entering state
  f32x4 Z[RT];
#pragma unroll
  for (int m = 0; m < RT; ++m) Z[m] = zero4();
  if constexpr (!STATE) {
    const float* src = nullptr;
    int rs = E, cs = 1;
    if (a.pieces) {
      src = sw.seg_state + ((int64_t)t.slot * a.H + t.h) * A * E;
    } else if (sw.Z0) {
      src = sw.Z0 + ((int64_t)t.n * a.H + t.h) * A * E;
      rs = sw.z0_rs;
      cs = sw.z0_cs;
    }
    if (src) {
#pragma unroll
      for (int m = 0; m < RT; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = lin_state_row<F32>(m, g, r);
          if (A >= KU || row < A) Z[m][r] = src[(int64_t)row * rs + (int64_t)(e0 + i) * cs];
        }
    }
  }

  // r: a lane has 4 neighbouring columns of token 16 k + i
  const int64_t rstep = dir * (int64_t)a.H * E;  // elements from row to row of the walk
  int64_t rat = t.tok0 * a.H * E + (t.pos0 + i) * rstep + (int64_t)t.h * E + e0 + 4 * g;

  // operands that are read ahead of their chunk
  V zv[UC];  // this wave's columns of z, contraction over tokens
  V xv[TT];  // rows of x, unit 0
  auto fetch = [&](const char* buf) {
#pragma unroll
    for (int u = 0; u < UC; ++u) zv[u] = TZ::col(buf + Sh::kXY, u, g, i, F32 ? c0 / 4 : c0 / 8, 0);
    if constexpr (!STATE) {
#pragma unroll
      for (int k = 0; k < TT; ++k) xv[k] = TX::row(buf + Sh::kBuf, 16 * k + i, 0, g);
    }
  };
  constexpr int MP = RT >= 4 ? 4 : RT, NS = UC * (RT / MP);  // state tiles a stage of the update; stages, units fastest
  auto y_of = [&](const char* ty, int st, int m) {           // operand of stage st, its tile m
    const int u = st % UC, mt = st / UC * MP + m;
    return F32 ? TY::col(ty, u, g, i, 4 * mt, 0) : TY::col(ty, u, g, i, 4 * (mt >> 1), mt & 1);
  };
  constexpr int TERMS = F32 ? 1 : 3;  // of the state, the scores and c_j z_j as operands
  // unit u of the state as an operand
  V zo[2][TERMS];
  auto state_operand = [&](int u) {
    if constexpr (F32) {
      zo[u & 1][0] = Z[u];
    } else {
      float x[8];
#pragma unroll
      for (int r = 0; r < 4; ++r) x[r] = Z[2 * u][r], x[4 + r] = Z[2 * u + 1][r];
      lin_split(x, zo[u & 1]);
    }
  };
  // c_j z_j of unit u
  V zs[UC][TERMS];
  auto terms = [&](int u) {
    if constexpr (F32) {
#pragma unroll
      for (int e = 0; e < 4; ++e) zs[u][0][e] = cz[u][e] * zv[u][e];
    } else {
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = cz[u][e] * bf16_to_f32(zv[u][e]);
      lin_split(x, zs[u]);
    }
  };
  // The barrier of a step. These waves write nothing to LDS, and what they have read ahead of it stays as it is for
  // two steps, so they need not wait for it. What they read of this step's buffers is in the products that come before
  // (and stay before, at 1 % of the time: the loading waves write those buffers after the barrier).
  auto step_barrier = [] {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  const bool want_last = STATE || (sw.Z1 != nullptr && t.seg + 1 == t.nseg);
  __syncthreads();
  if constexpr (!STATE) __syncthreads();
  int now = 0;  // this chunk's buffer
  fetch(lds);
  if constexpr (!STATE) state_operand(0);
  for (int s = 0; s < steps; ++s) {
    const char* const ty = lds + now * BUF;
    const char* const tz = ty + Sh::kXY;
    const char* const tx = ty + Sh::kBuf;
    const char* const tp = scores + (s & 1) * Sh::kScores;
    const int valid = min(C, t.pos1 - (t.pos0 + s * C));
    const bool last = s + 1 == steps;
    const int before = now;
    now = now == (STATE ? 1 : 2) ? 0 : now + 1;
    const char* const after = lds + now * BUF;
    if (valid < C) {
      set_cz(valid);
      chunk_decay(valid, gC, gRest);
    }
    V y[2][MP];
    // r^T from the state and from the scores: rows are columns of the state, columns are tokens
    f32x4 R[TT], R2[TT];

    if constexpr (!STATE) {
      // scores by unit: row tile k, unit u <= 16 k / KU
      constexpr int NU = F32 ? TT * (TT + 1) / 2 : TT * (TT + 2) / 4, H1 = NU / 2;
      V ps[NU][TERMS];
      auto each_unit = [&](int from, int to, auto f) {
        int n = 0;
#pragma unroll
        for (int k = 0; k < TT; ++k)
#pragma unroll
          for (int u = 0; u <= 16 * k / KU; ++u, ++n)
            if (n >= from && n < to) f(n, k, u);
      };
      auto get_scores = [&](int from, int to) {
        each_unit(from, to, [&](int n, int k, int u) {
          if constexpr (F32) {
            ps[n][0] = TP::row(tp, 16 * k + i, u, g);
          } else {
#pragma unroll
            for (int t2 = 0; t2 < TERMS; ++t2)
              ps[n][t2] = *reinterpret_cast<const V*>(tp + LinScores::at(t2, 16 * k + i, 4 * u + g));
          }
        });
      };
      const int4 odd4 = *reinterpret_cast<const int4*>(flags + before * kLinLoad);
#pragma unroll
      for (int k = 0; k < TT; ++k) R[k] = R2[k] = zero4();
#pragma unroll
      for (int u = 0; u < UK; ++u) {
        V xn[TT];
        if (u + 1 < UK) {
#pragma unroll
          for (int k = 0; k < TT; ++k) xn[k] = TX::row(tx, 16 * k + i, u + 1, g);
        } else {
          get_scores(0, H1);
        }
#pragma unroll
        for (int t2 = TERMS - 1; t2 >= 0; --t2)
#pragma unroll
          for (int k = 0; k < TT; ++k) lin_mma(R[k], zo[u & 1][t2], xv[k]);
        if (u + 1 < UK) {
          state_operand(u + 1);  // beside the products
#pragma unroll
          for (int k = 0; k < TT; ++k) xv[k] = xn[k];
        }
      }

      // a zero score times an infinity or NaN of a later token is NaN: such values of z are taken out of the product,
      // and added to their own and later tokens one by one
      const bool odd = __builtin_amdgcn_readfirstlane(odd4.x | odd4.y | odd4.z | odd4.w) != 0;
      V zp[UC];
#pragma unroll
      for (int u = 0; u < UC; ++u) zp[u] = zv[u];
      if (odd) {
#pragma unroll
        for (int u = 0; u < UC; ++u) lin_finite(zp[u]);
      }
      auto add_scores = [&](int from, int to) {
#pragma unroll
        for (int t2 = TERMS - 1; t2 >= 0; --t2)
          each_unit(from, to, [&](int n, int k, int u) { lin_mma(R2[k], zp[u], ps[n][t2]); });
      };
      get_scores(H1, NU);
      add_scores(0, H1);
      terms(0);
#pragma unroll
      for (int m = 0; m < MP; ++m) y[0][m] = y_of(ty, 0, m);
      add_scores(H1, NU);
      if (odd) {
#pragma unroll
        for (int k = 0; k < TT; ++k)
#pragma unroll 1
          for (int j = 0; j < 16 * (k + 1); ++j) {
            float p;
            if constexpr (F32) {
              p = *reinterpret_cast<const float*>(tp + TP::at(16 * k + i, j >> 2) + 4 * (j & 3));
            } else {
              const auto term = [&](int n) {
                return bf16_to_f32(*reinterpret_cast<const __bf16*>(tp + LinScores::at(n, 16 * k + i, j >> 3) + 2 * (j & 7)));
              };
              p = term(0) + (term(1) + term(2));
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int c = c0 + 4 * g + r;
              const float z = load1<F32>(tz + TZ::at(j, c * ES / 16), c % (16 / ES));
              if (j <= 16 * k + i && !(fabsf(z) <= 3.4028235e38f)) R2[k][r] += p * z;
            }
          }
      }
    } else {
#pragma unroll
      for (int m = 0; m < MP; ++m) y[0][m] = y_of(ty, 0, m);
      terms(0);
    }
    auto store = [&] {
#pragma unroll
      for (int k = 0; k < TT; ++k) {
        if (valid == C || 16 * k + i < valid) {
          const int64_t at = rat + 16 * k * rstep;
          f32x4 x;
#pragma unroll
          for (int r = 0; r < 4; ++r) x[r] = fmaf(R[k][r], ro[k], R2[k][r]);
          if (F32 || sw.r_f32) st4(static_cast<float*>(sw.r) + at, x[0], x[1], x[2], x[3]);
          else st4(static_cast<__bf16*>(sw.r) + at, x[0], x[1], x[2], x[3]);
        }
      }
      rat += C * rstep;
    };

    // Z <- g^n Z + sum_j y_j (c_j z_j)^T, the chunk's sum apart: one rounding a chunk in a state that is carried over
    // thousands (64K tokens of hardly any decay: 3.3e-7 off, 1.2e-6 with every product added to the state itself)
    // T starts from what the rounding of g^n leaves of the state (1 % of the time; 3 % when added at the end)
    f32x4 T[MP];
#pragma unroll
    for (int st = 0; st < NS; ++st) {
      if (st + 1 < NS) {
#pragma unroll
        for (int m = 0; m < MP; ++m) y[(st + 1) & 1][m] = y_of(ty, st + 1, m);
      }
      const int u = st % UC, m0 = st / UC * MP;
      if (u == 0) {
#pragma unroll
        for (int m = 0; m < MP; ++m)
#pragma unroll
          for (int r = 0; r < 4; ++r) T[m][r] = Z[m0 + m][r] * gRest;
      }
#pragma unroll
      for (int t2 = TERMS - 1; t2 >= 0; --t2)
#pragma unroll
        for (int m = 0; m < MP; ++m) lin_mma(T[m], y[st & 1][m], zs[u][t2]);
      if (st + 1 < UC) terms(st + 1);  // beside the products
      if (u == UC - 1) {
#pragma unroll
        for (int m = 0; m < MP; ++m)
#pragma unroll
          for (int r = 0; r < 4; ++r) Z[m0 + m][r] = fmaf(Z[m0 + m][r], gC, T[m][r]);
      }
      if (!STATE && st == 0) store();
    }
    if (!STATE) state_operand(0);
    if constexpr (!STATE) {  // the next chunk is in LDS since the step before
      if (!last) fetch(after);
      step_barrier();
    } else {
      __syncthreads();
      if (!last) fetch(after);
    }
  }

  if (want_last) {
    float* dst = STATE ? sw.seg_state + ((int64_t)(a.cu ? t.slot + 1 : t.slot + a.N) * a.H + t.h) * A * E
                       : sw.Z1 + ((int64_t)t.n * a.H + t.h) * A * E;
#pragma unroll
    for (int m = 0; m < RT; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = lin_state_row<F32>(m, g, r);
        if (A >= KU || row < A) dst[(int64_t)row * E + e0 + i] = Z[m][r];
      }
  }
}

}  // namespace gdn2
