// Tiles of the experts' products (experts.hip): C[m,n] = sum_k A[m,k] B[n,k] over rows sorted by
// expert, on the matrix cores.
//
// Four products share one kernel: the gated half and the projection (A: the rows x, B: the
// expert's weights, both with their k in a row), the rows' gradient (A: d, B: the weights, whose
// rows are now the k) and the weights' gradient (A: d, B: x, both with rows as the k).  An operand
// is staged in LDS as it lies in memory, 128 bytes of k per tile row or one tile row per k, and
// turned where it is read: 16-bit operands whose k runs over rows come back through the
// transposing LDS read.
#pragma once

#include "rows.hpp"

namespace rmoe {

enum { OP_GLU = 0, OP_LINEAR = 1, OP_DX = 2, OP_DW = 3 };

struct ProductArgs {
  const void* a;             // m side: x or d
  const void* b;             // n side: w or x
  const int32_t* offsets;    // [E+1] or null: one expert of all rows
  int64_t lda, ldb, gsb;     // row strides and, for weights, the stride between experts (elements)
  int32_t rows, E;
  int32_t M, N, K;           // OP_DW: M x N weights (K is the expert's rows); else N outputs, K terms
  int32_t act;
  void* out;                 // a, y, dx or dw
  void* aux;                 // gu or z, or null
  const void* residual;      // or null
  const float* bias;         // [E,N] or null
  int64_t ldo, ld_aux, ld_res;
  int32_t out_fmt;           // of out and residual
  bool padded;               // a's rows have zeros up to a multiple of 16 bytes
  uint32_t tiles;            // at most
  int32_t splits;            // of the k, each with a plane of fp32 outputs of its own if there are more than one
  int64_t plane;             // elements
  bool past_caches;          // dw in bf16 whose rows are whole lines
};

// ---------------------------------------------------------------- activations
// z s(q) with s the logistic function: q = z (silu), or twice the cubic of gelu's tanh form,
// since (1 + tanh p) / 2 = s(2 p).  From t = exp(-|q|) neither the value nor the derivative meets
// an infinity or a difference of equal numbers.
struct Act {
  float value, grad;
};
__device__ __forceinline__ Act act_of(float z, int act) {
  if (act == MOE_ACT_NONE) return {z, 1.f};
  constexpr float c = 1.5957691216057308f;  // 2 sqrt(2 / pi)
  const float z2 = z * z;
  const float q = act == MOE_ACT_SILU ? z : c * (z + 0.044715f * z * z2);
  const float dq = act == MOE_ACT_SILU ? 1.f : c * (1.f + 0.134145f * z2);
  const float t = expf(-fabsf(q)), r = 1.f / (1.f + t);
  const float s = q >= 0.f ? r : t * r;
  // where t has run out, q is past 100 and s(q) s(-q) is nothing, whatever dq has become
  return {z * s, t == 0.f ? s : s + z * dq * (t * r * r)};
}

// ---------------------------------------------------------------- eight elements of a row
// The first n of eight elements at p, any alignment, the rest zeros.
__device__ __forceinline__ void read8(const void* base, int64_t at, int fmt, int n, float (&v)[8]) {
  if (fmt == MOE_AFMT_BF16) {
    const uint16_t* p = static_cast<const uint16_t*>(base) + at;
    if (n >= 8) {
      const u32x4 q = load16<false>(reinterpret_cast<const uint8_t*>(p));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(q[i]);
        v[2 * i + 1] = bf16_hi(q[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < n ? bf16_to_f32(p[i]) : 0.f;
    }
  } else {
    const float* p = static_cast<const float*>(base) + at;
    if (n >= 8) {
      const u32x4 a = load16<false>(reinterpret_cast<const uint8_t*>(p));
      const u32x4 b = load16<false>(reinterpret_cast<const uint8_t*>(p + 4));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = __uint_as_float(a[i]);
        v[4 + i] = __uint_as_float(b[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : 0.f;
    }
  }
}
// Rounded to fmt (nearest even) at p.
template <bool NT = false>
__device__ __forceinline__ void write8(void* base, int64_t at, int fmt, int n, const float (&v)[8]) {
  if (fmt == MOE_AFMT_BF16) {
    uint16_t* p = static_cast<uint16_t*>(base) + at;
    u32x4 q;
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    if (n >= 8) {
      store16<NT>(reinterpret_cast<uint8_t*>(p), q);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) p[i] = (uint16_t)(q[i / 2] >> 16 * (i & 1));
    }
  } else {
    float* p = static_cast<float*>(base) + at;
    if (n >= 8) {
      u32x4 a, b;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = __float_as_uint(v[i]);
        b[i] = __float_as_uint(v[4 + i]);
      }
      store16<NT>(reinterpret_cast<uint8_t*>(p), a);
      store16<NT>(reinterpret_cast<uint8_t*>(p + 4), b);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) p[i] = v[i];
    }
  }
}

__device__ __forceinline__ void write1(void* base, int64_t at, int fmt, float v) {
  if (fmt == MOE_AFMT_BF16) static_cast<uint16_t*>(base)[at] = (uint16_t)pack_bf16(v, v);
  else static_cast<float*>(base)[at] = v;
}

// ---------------------------------------------------------------- experts' rows and tiles
// Expert g's rows as the offsets say, brought into [0, rows]: whatever the table holds, nothing
// outside the rows is read or written.
struct Range {
  int first, n;
};
__device__ __forceinline__ Range expert_rows(const int32_t* offsets, int g, int rows) {
  if (!offsets) return {0, rows};
  const int lo = min(max(offsets[g], 0), rows), hi = min(max(offsets[g + 1], 0), rows);
  return {lo, max(hi - lo, 0)};
}

__device__ __forceinline__ Range expert_rows_uniform(const int32_t* offsets, int g, int rows) {
  // by scalar loads: they wait for no vector memory access, of which many may be on their way
  if (!offsets) return {0, rows};
  const auto* o = (const __attribute__((address_space(4))) int32_t*)offsets;
  const int lo = min(max(o[g], 0), rows), hi = min(max(o[g + 1], 0), rows);
  return {lo, max(hi - lo, 0)};
}

// Workgroups go round the eight XCDs; an XCD's i-th takes the i-th entry of its list of tiles.  The
// list is an eighth of all tiles' order, so that tiles that share operands share an L2; -1: none.
__device__ __forceinline__ int64_t tile_of_list(uint32_t total, uint32_t i) {
  const uint32_t per = (total + 7) / 8;
  const uint64_t t = (uint64_t)(blockIdx.x & 7) * per + i;
  return i < per && t < total ? (int64_t)t : -1;
}
// The weights' gradient: an expert's tiles (`each` of them) differ in cost from another's, so every
// expert's are dealt out to all XCDs, in runs of neighbours that share operands.
__host__ __device__ __forceinline__ uint32_t dealt_run(uint32_t each) { return each < 16 ? 1 : each / 8; }
__device__ __forceinline__ int64_t dealt_tile(uint32_t total, uint32_t each, uint32_t i) {
  const uint32_t run = dealt_run(each), x = blockIdx.x & 7;
  const uint64_t t = ((uint64_t)(i / run) * 8 + x) * run + i % run;
  return t < total ? (int64_t)t : -1;
}

__device__ __forceinline__ uint32_t add_sat(uint32_t a, uint32_t b) { return a + b < a ? 0xffffffffu : a + b; }

// Band order: eight row tiles high, then column by column, so about as many row tiles as
// column tiles are in flight on an XCD.
__device__ __forceinline__ void band_order(uint32_t r, int mt, int nt, int& m, int& n) {
  constexpr int kBand = 8;
  const uint32_t band = r / (uint32_t)(kBand * nt), in = r - band * (kBand * nt);
  const int high = min(kBand, mt - (int)band * kBand);
  n = in / high;
  m = band * kBand + in % high;
}

// Where a tile of C lies: M x N outputs of K terms from row row0 (or of them) of expert g's; m0: its
// first row of weights (OP_DW), n0: its first column; split: which part of the k (ProductArgs::splits).
struct Place {
  int g, row0, m0, n0, M, N, K, split;
};

// The row tiles of all experts, counted: each wavefront's lanes count those of E / 64
// experts each, up to and with its own.
template <int OP, int BM>
__device__ __forceinline__ uint32_t count_tiles(const ProductArgs& p) {
  if (OP == OP_DW || !p.offsets) return 0;
  const int lane = threadIdx.x & 63, per = (p.E + 63) / 64, g0 = lane * per;
  uint32_t incl = 0;
  for (int i = 0; i < per; ++i)
    if (g0 + i < p.E) incl += (expert_rows(p.offsets, g0 + i, p.rows).n + BM - 1) / BM;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t v = __shfl_up(incl, o);
    if (lane >= o) incl = add_sat(incl, v);
  }
  return incl;
}

// The i-th tile of this workgroup's XCD; false: it has no more.
template <int OP, int BM, int COLS>
__device__ __forceinline__ bool find_place(const ProductArgs& p, uint32_t counts, uint32_t i, Place& at) {
  const int nt = (p.N + COLS - 1) / COLS;
  int m, n;
  if constexpr (OP == OP_DW) {
    const int mt = (p.M + BM - 1) / BM;
    const int64_t b = dealt_tile((uint32_t)p.E * mt * nt, mt * nt, i);
    if (b < 0) return false;
    at.g = (int)((uint32_t)b / (uint32_t)(mt * nt));
    band_order((uint32_t)b % (uint32_t)(mt * nt), mt, nt, m, n);
    const Range r = expert_rows_uniform(p.offsets, at.g, p.rows);
    at.row0 = r.first;
    at.K = r.n;
    at.m0 = m * BM;
    at.M = min(BM, p.M - at.m0);
  } else {
    at.K = p.K;
    at.m0 = 0;
    if (!p.offsets) {
      const int mt = (p.rows + BM - 1) / BM;
      const int64_t b = tile_of_list((uint32_t)mt * nt, i);
      if (b < 0) return false;
      band_order((uint32_t)b, mt, nt, m, n);
      at.g = 0;
      at.row0 = m * BM;
      at.M = min(BM, p.rows - m * BM);
    } else {
      // (a table that is no offsets may count more tiles than rows allow: no more than those are done)
      const uint64_t all = (uint64_t)(uint32_t)__builtin_amdgcn_readlane(counts, 63) * nt;
      const int64_t b = tile_of_list((uint32_t)min(all, (uint64_t)p.tiles), i);
      if (b < 0) return false;
      const uint64_t past = __ballot((uint64_t)counts * nt > (uint64_t)b);
      const int l = __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)past) - 1);
      uint32_t before = l ? (uint32_t)__builtin_amdgcn_readlane(counts, l - 1) : 0u;
      for (int g = l * ((p.E + 63) / 64);; ++g) {
        const Range r = expert_rows_uniform(p.offsets, g, p.rows);
        const uint32_t mt = (r.n + BM - 1) / BM;
        if ((uint64_t)(before + mt) * nt > (uint64_t)b) {
          band_order((uint32_t)(b - (int64_t)before * nt), mt, nt, m, n);
          at.g = g;
          at.row0 = r.first + m * BM;
          at.M = min(BM, r.n - m * BM);
          break;
        }
        before += mt;
      }
    }
  }
  at.n0 = n * COLS;
  at.N = min(COLS, p.N - at.n0);
  at.g = __builtin_amdgcn_readfirstlane(at.g);
  at.row0 = __builtin_amdgcn_readfirstlane(at.row0);
  at.m0 = __builtin_amdgcn_readfirstlane(at.m0);
  at.n0 = __builtin_amdgcn_readfirstlane(at.n0);
  at.M = __builtin_amdgcn_readfirstlane(at.M);
  at.N = __builtin_amdgcn_readfirstlane(at.N);
  at.K = __builtin_amdgcn_readfirstlane(at.K);
  return true;
}

// ---------------------------------------------------------------- operands
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

// An operand in LDS: R tile rows by 128 bytes of k, in 16-byte pieces.  Sixteen lanes' pieces (or 8 bytes
// of thirty-two) lie in different banks, whatever the k:
//  k in a row (KMAJ = false): the pieces of a tile row one after the other, piece c at c ^ f(row);
//  a tile row per k (KMAJ = true): k's R elements one after the other, piece c at c ^ f(k).
template <typename E, int R, bool KMAJ>
struct Operand {
  static constexpr int kEl = 16 / sizeof(E);       // elements of a piece
  static constexpr int kK = 128 / sizeof(E);       // k of a stage
  static constexpr int kBytes = R * 128;
  static constexpr int kPieces = R * 8;
  static constexpr int kPerRow = KMAJ ? R * (int)sizeof(E) / 16 : 8;
  static_assert(R >= 32 && R % 32 == 0, "f stays inside a row of pieces");

  __device__ static __forceinline__ int swizzle(int i) {  // of tile row or k i
    if constexpr (!KMAJ) return (i >> 1) & 7;
    else if constexpr (sizeof(E) == 4) return 4 * ((i >> 2) & (R >= 64 ? 3 : 1));
    else if constexpr (R >= 128) return 4 * (i & 3) + 2 * ((i >> 3) & 1);
    else if constexpr (R == 64) return 2 * (i & 3);
    else return 2 * ((i >> 3) & 1);
  }
  // Of piece s (16 bytes at 16 s): its tile row and first k, or its k and first tile row.
  __device__ static __forceinline__ void where(int s, int& row, int& k) {
    if constexpr (KMAJ) {
      k = s / kPerRow;
      row = ((s % kPerRow) ^ swizzle(k)) * kEl;
    } else {
      row = s / kPerRow;
      k = ((s % kPerRow) ^ swizzle(row)) * kEl;
    }
  }
  // The matrix instruction's operand of 16 tile rows from r0 (a multiple of 16) at step j of a
  // stage's two: lane l has row r0 + l % 16 and the 16 bytes of k that follow 64 j + 16 (l / 16) bytes.
  // (In fp32 a step is four instructions of four k each, whose order is the same on both sides.)
  __device__ static __forceinline__ u32x4 fragment(const uint8_t* lds, int r0, int j, int lane) {
    const int r = lane & 15, q = lane >> 4;
    if constexpr (!KMAJ) {
      return *reinterpret_cast<const u32x4*>(lds + (r0 + r) * 128 + (((4 * j + q) ^ swizzle(r)) << 4));
    } else if constexpr (sizeof(E) == 2) {
      // 16 lanes read four k of 16 tile rows, 8 bytes each, and get four k of one tile row each
      const int k = 8 * q + (r >> 2), c = r0 / 8 + ((r & 3) >> 1);
      const uint8_t* p = lds + (32 * j + k) * (R * 2) + ((c ^ swizzle(k)) << 4) + ((r & 1) << 3);
      typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p));
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * (R * 2)));
      return __builtin_bit_cast(u32x4, (s16x8)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      u32x4 v;
      const int m = r0 + r;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = *reinterpret_cast<const uint32_t*>(lds + (16 * j + 4 * q + i) * (R * 4) + (((m >> 2) ^ swizzle(4 * q)) << 4) +
                                                  ((m & 3) << 2));
      return v;
    }
  }
};

// 16 x 16 outputs: under this card's power limit the 16 x 16 x 32 instruction sustains 2060 TFLOP/s on
// random operands in registers, the 32 x 32 x 16 one 1820 (2430 and 2460 on zeros).
template <typename E>
__device__ __forceinline__ void multiply(u32x4 a, u32x4 b, f32x4& acc) {
  if constexpr (sizeof(E) == 2) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), acc, 0, 0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[i]), __uint_as_float(b[i]), acc, 0, 0, 0);
  }
}

// The first n of a piece's elements at p, the rest zeros (n <= 0: nothing is read).
template <typename E>
__device__ __forceinline__ u32x4 read_piece(const uint8_t* p, int n) {
  constexpr int el = 16 / sizeof(E);
  if (n >= el) return load16<false>(p);
  u32x4 q = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < el; ++i) {
    if (i >= n) continue;
    if constexpr (sizeof(E) == 2) q[i / 2] |= (uint32_t) reinterpret_cast<const uint16_t*>(p)[i] << 16 * (i & 1);
    else q[i] = reinterpret_cast<const uint32_t*>(p)[i];
  }
  return q;
}

// ---------------------------------------------------------------- the kernel
// A workgroup has a BM x BN tile of C, a wavefront WM x WN of it in fragments of 16 x 16.  The
// matrix instruction's rows are n and its columns m, so that a lane holds four neighbouring
// outputs of one row.
template <typename E, int OP, int BM, int BN, int WM, int WN>
struct ProductTile {
  static constexpr int kWaves = (BM / WM) * (BN / WN), kThreads = 64 * kWaves;
  static constexpr int kMt = WM / 16, kNt = WN / 16;
  static constexpr bool kKmajA = OP == OP_DW, kKmajB = OP == OP_DX || OP == OP_DW;
  static constexpr int kStages = 2 * (BM + BN) * 128;          // two stages in LDS
  static constexpr int kPatch = 16 * WN * 4;                   // sixteen rows of a wavefront in fp32, for the epilogue
  static_assert(kWaves * kPatch <= kStages, "they take the stages' place");
  static_assert(WM % 32 == 0 && WN % 32 == 0, "halves of whole fragments");
  static constexpr int kCols = OP == OP_GLU ? BN / 2 : BN;     // outputs of a tile's row
};

// The source row of row r of the n side's tile where its k lie in a row.
template <int OP, int WN>
__device__ __forceinline__ int64_t n_row(const ProductArgs& p, const Place& at, int r) {
  if constexpr (OP == OP_GLU) {  // a wavefront's columns: WN / 2 of the gate, then the same of up
    const int c = r / WN * (WN / 2) + r % (WN / 2);
    return at.n0 + min(c, at.N - 1) + (r % WN >= WN / 2 ? p.N : 0);
  } else {
    return at.n0 + min(r, at.N - 1);
  }
}

// Epilogue: 16 rows of a wavefront's columns at a time go through LDS (16-byte pieces, piece c of row r at
// c ^ r), so that eight neighbouring outputs of a row meet in one lane and rows are written in whole
// lines.  patch: the wavefront's own.
template <typename E, int OP, int BM, int BN, int WM, int WN>
__device__ __forceinline__ void write_tile(const ProductArgs& p, const Place& at_, uint8_t* patch, int wave, int lane,
                                           const f32x4 (&acc)[WM / 16][WN / 16]) {
  const int wm = wave / (BN / WN) * WM, wn = wave % (BN / WN) * WN;
  constexpr int kSwz = (WN / 4 - 1) & 15;
  constexpr int kOut = OP == OP_GLU ? WN / 2 : WN;        // outputs of a row
  constexpr int kLanes = kOut / 8, kRows = 64 / kLanes;   // lanes of a row, rows at once
  const int cl = 8 * (lane % kLanes);
  const int col = at_.n0 + (OP == OP_GLU ? wn / 2 : wn) + cl, cols = p.N - col;
#pragma unroll
  for (int m = 0; m < WM / 16; ++m) {
    {
      const int r = lane & 15;
#pragma unroll
      for (int n = 0; n < WN / 16; ++n)
        *reinterpret_cast<f32x4*>(patch + r * (WN * 4) + (((4 * n + (lane >> 4)) ^ (r & kSwz)) << 4)) = acc[m][n];
    }
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < (16 + kRows - 1) / kRows; ++i) {
      const int r = i * kRows + lane / kLanes, row = wm + 16 * m + r;
      const auto get = [&](int c, float (&v)[8]) {
        const int q = r & 15;
        const f32x4 x = *reinterpret_cast<const f32x4*>(patch + q * (WN * 4) + (((c / 4) ^ (q & kSwz)) << 4));
        const f32x4 y = *reinterpret_cast<const f32x4*>(patch + q * (WN * 4) + (((c / 4 + 1) ^ (q & kSwz)) << 4));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[e] = x[e];
          v[4 + e] = y[e];
        }
      };
      float v[8];
      get(cl, v);
      float u[8];
      if constexpr (OP == OP_GLU) get(WN / 2 + cl, u);
      if (r >= 16 || row >= at_.M || cols <= 0) continue;
      if constexpr (OP == OP_DW) {
        // past the caches where rows are whole lines: it is read much later, if at all there (1.07 GB of it 333 -> 257 us, 134
        // MB 101 -> 95).  So do wavefronts of 32 columns, each of which has half of a line: 228 MB over 249 experts 97 -> 84,
        // smaller ones level.  Lines that two rows share are put together in the caches: rows of 760 for 109 experts of
        // 512 would take 40 us past them and 22, in fp32 135 and 46.  The empty asm keeps the two kinds of store apart.
        const int64_t at = at_.split * p.plane + ((int64_t)at_.g * p.M + at_.m0 + row) * p.N + col;
        if (p.past_caches) {
          write8<true>(p.out, at, MOE_AFMT_BF16, cols, v);
          asm volatile("");
        } else {
          write8(p.out, at, p.out_fmt, cols, v);
        }
      } else {
        const int64_t at = at_.row0 + row;
        if constexpr (OP == OP_GLU) {
          constexpr int fmt = sizeof(E) == 2 ? MOE_AFMT_BF16 : MOE_AFMT_F32;
          if (p.aux) {
            write8(p.aux, at * p.ld_aux + col, fmt, cols, v);
            write8(p.aux, at * p.ld_aux + p.N + col, fmt, cols, u);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = act_of(v[e], p.act).value * u[e];
          write8(p.out, at * p.ldo + col, fmt, cols, v);
        } else if constexpr (OP == OP_LINEAR) {
          constexpr int fmt = sizeof(E) == 2 ? MOE_AFMT_BF16 : MOE_AFMT_F32;
          float w[8];
          if (p.bias) {
            read8(p.bias, (int64_t)at_.g * p.N + col, MOE_AFMT_F32, cols, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += w[e];
          }
          if (p.aux) write8(p.aux, at * p.ld_aux + col, fmt, cols, v);
          if (p.act != MOE_ACT_NONE) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = act_of(v[e], p.act).value;
          }
          if (p.residual) {
            read8(p.residual, at * p.ld_res + col, p.out_fmt, cols, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += w[e];
          }
          write8(p.out, at * p.ldo + col, p.out_fmt, cols, v);
        } else {
          write8(p.out, at_.split * p.plane + at * p.ldo + col, p.out_fmt, cols, v);
        }
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// Elements `n` and up of a piece, the first one first, zeros behind them (n = all: zeros).
template <typename E>
__device__ __forceinline__ u32x4 elements_from(u32x4 q, int n) {
  uint64_t lo = q[0] | (uint64_t)q[1] << 32, hi = q[2] | (uint64_t)q[3] << 32;
  const int bits = n * 8 * (int)sizeof(E), in = bits & 63;
  const uint64_t up = in ? hi << (64 - in) : 0;
  lo = bits >= 128 ? 0 : bits >= 64 ? hi >> in : lo >> in | up;
  hi = bits >= 64 ? 0 : hi >> in;
  return {(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}

// Operands whose rows start anywhere: pieces go through registers, DEPTH stages ahead.  All but the last
// stage are plain loads.  There a piece at the columns' edge takes the start of the next row with it,
// for outputs that are not written.  In the last stage it is its row's last whole piece, shifted.
// (Rows shorter than a piece: element by element.)
template <typename E, int OP, int BM, int BN, int WM, int WN, int DEPTH>
__device__ __forceinline__ void staged_product(const ProductArgs& p, uint32_t block, int split, uint8_t* lds) {
  using T = ProductTile<E, OP, BM, BN, WM, WN>;
  using OpA = Operand<E, BM, T::kKmajA>;
  using OpB = Operand<E, BN, T::kKmajB>;
  constexpr int kThreads = T::kThreads, kK = OpA::kK, kEl = OpA::kEl, kStage = T::kStages / 2;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / (BN / WN) * WM, wn = wave % (BN / WN) * WN;
  Place at;
  if (!find_place<OP, BM, T::kCols>(p, count_tiles<OP, BM>(p), block >> 3, at)) return;
  at.split = split;
  const int K = at.K, all = (K + kK - 1) / kK, stages = (all + p.splits - 1) / p.splits, first = split * stages;

  // this thread's pieces.  k in a row: the row's start; a row per k: the piece in the first stage's row (or
  // the last column's, past it), and how many of its elements are behind the row
  constexpr int kPa = OpA::kPieces / kThreads, kPb = OpB::kPieces / kThreads;
  const E *pa[kPa], *pb[kPb];
  int ka[kPa], kb[kPb], sa[kPa], sb[kPb];
  const E* a = static_cast<const E*>(p.a) + (int64_t)at.row0 * p.lda;
  const E* b = static_cast<const E*>(p.b) + (OP == OP_DW ? (int64_t)at.row0 * p.ldb : at.g * p.gsb);
  const bool tiny = (T::kKmajA && p.M < kEl) || (T::kKmajB && p.N < kEl) || ((!T::kKmajA || !T::kKmajB) && K < kEl);
  const auto column = [&](int c, int total, int& behind) {
    c = tiny ? c : min(c, total - 1);
    behind = max(c - (total - kEl), 0);
    return c;
  };
#pragma unroll
  for (int i = 0; i < kPa; ++i) {
    int r;
    OpA::where(i * kThreads + tid, r, ka[i]);
    if constexpr (T::kKmajA) pa[i] = a + (int64_t)ka[i] * p.lda + column(at.m0 + r, p.M, sa[i]);
    else pa[i] = a + (int64_t)min(r, at.M - 1) * p.lda;
  }
#pragma unroll
  for (int i = 0; i < kPb; ++i) {
    int r;
    OpB::where(i * kThreads + tid, r, kb[i]);
    if constexpr (T::kKmajB) pb[i] = b + (int64_t)kb[i] * p.ldb + column(at.n0 + r, p.N, sb[i]);
    else pb[i] = b + n_row<OP, WN>(p, at, r) * p.ldb;
  }
  u32x4 qa[DEPTH][kPa], qb[DEPTH][kPb];
  constexpr int kMore = T::kKmajA || T::kKmajB;  // rows that a plain stage needs behind it
  const auto piece = [&](const E* from) { return load16<false>(reinterpret_cast<const uint8_t*>(from)); };
  const auto load = [&](int s, u32x4 (&ga)[kPa], u32x4 (&gb)[kPb]) {
    const int k0 = s * kK;
    if (!tiny && k0 + kK + kMore <= K) {
#pragma unroll
      for (int i = 0; i < kPa; ++i) ga[i] = piece(pa[i] + (T::kKmajA ? k0 * p.lda : k0 + ka[i]));
#pragma unroll
      for (int i = 0; i < kPb; ++i) gb[i] = piece(pb[i] + (T::kKmajB ? k0 * p.ldb : k0 + kb[i]));
    } else if (!tiny) {
      // k past the last: the last row again, or the row's last piece, and then zeros
#pragma unroll
      for (int i = 0; i < kPa; ++i)
        ga[i] = piece(pa[i] + (T::kKmajA ? (min(k0 + ka[i], K - 1) - ka[i]) * p.lda - sa[i] : max(min(k0 + ka[i], K - kEl), 0)));
#pragma unroll
      for (int i = 0; i < kPb; ++i)
        gb[i] = piece(pb[i] + (T::kKmajB ? (min(k0 + kb[i], K - 1) - kb[i]) * p.ldb - sb[i] : max(min(k0 + kb[i], K - kEl), 0)));
#pragma unroll
      for (int i = 0; i < kPa; ++i)
        ga[i] = elements_from<E>(ga[i], T::kKmajA ? (k0 + ka[i] < K ? sa[i] : kEl) : min(max(k0 + ka[i] - (K - kEl), 0), kEl));
#pragma unroll
      for (int i = 0; i < kPb; ++i)
        gb[i] = elements_from<E>(gb[i], T::kKmajB ? (k0 + kb[i] < K ? sb[i] : kEl) : min(max(k0 + kb[i] - (K - kEl), 0), kEl));
    } else {
      const auto some = [&](const E* row, int64_t at_, int n) { return read_piece<E>(reinterpret_cast<const uint8_t*>(row + at_), n); };
#pragma unroll
      for (int i = 0; i < kPa; ++i) {
        int r, k;
        OpA::where(i * kThreads + tid, r, k);
        if constexpr (T::kKmajA) ga[i] = some(pa[i], k0 * p.lda, k0 + k < K ? p.M - at.m0 - r : 0);
        else ga[i] = some(pa[i], k0 + k, K - k0 - k);
      }
#pragma unroll
      for (int i = 0; i < kPb; ++i) {
        int r, k;
        OpB::where(i * kThreads + tid, r, k);
        if constexpr (T::kKmajB) gb[i] = some(pb[i], k0 * p.ldb, k0 + k < K ? p.N - at.n0 - r : 0);
        else gb[i] = some(pb[i], k0 + k, K - k0 - k);
      }
    }
  };
  const auto store = [&](int t, const u32x4 (&ga)[kPa], const u32x4 (&gb)[kPb]) {
    uint8_t* stage = lds + (t & 1) * kStage;
#pragma unroll
    for (int i = 0; i < kPa; ++i) *reinterpret_cast<u32x4*>(stage + 16 * (i * kThreads + tid)) = ga[i];
#pragma unroll
    for (int i = 0; i < kPb; ++i) *reinterpret_cast<u32x4*>(stage + OpA::kBytes + 16 * (i * kThreads + tid)) = gb[i];
  };

  f32x4 acc[T::kMt][T::kNt] = {};
  if (stages) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
      if (d < stages) load(first + d, qa[d], qb[d]);
    store(0, qa[0], qb[0]);
    __syncthreads();
  }
  for (int t0 = 0; t0 < stages; t0 += DEPTH) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      const int t = t0 + d;
      if (t >= stages) break;
      if (t + DEPTH < stages) load(first + t + DEPTH, qa[d], qb[d]);
      const uint8_t* stage = lds + (t & 1) * kStage;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        u32x4 fa[T::kMt], fb[T::kNt];
#pragma unroll
        for (int i = 0; i < T::kMt; ++i) fa[i] = OpA::fragment(stage, wm + 16 * i, j, lane);
#pragma unroll
        for (int i = 0; i < T::kNt; ++i) fb[i] = OpB::fragment(stage + OpA::kBytes, wn + 16 * i, j, lane);
#pragma unroll
        for (int m = 0; m < T::kMt; ++m)
#pragma unroll
          for (int n = 0; n < T::kNt; ++n) multiply<E>(fb[n], fa[m], acc[m][n]);
      }
      if (t + 1 < stages) store(t + 1, qa[(d + 1) % DEPTH], qb[(d + 1) % DEPTH]);
      __syncthreads();
    }
  }
  write_tile<E, OP, BM, BN, WM, WN>(p, at, lds + wave * T::kPatch, wave, lane, acc);
}

template <typename E, int OP, int BM, int BN, int WM, int WN, int DEPTH>
__global__ __launch_bounds__(64 * (BM / WM) * (BN / WN)) void product_kernel(ProductArgs p) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[ProductTile<E, OP, BM, BN, WM, WN>::kStages];
  staged_product<E, OP, BM, BN, WM, WN, DEPTH>(p, blockIdx.x, blockIdx.y, lds);
}

// ---------------------------------------------------------------- operands straight into LDS
// The same for operands whose rows all start on 16 bytes: buffer loads write LDS themselves, 1 KB a
// wavefront and instruction in lane order (the pieces' places are chosen by what each lane reads), so
// a stage costs no registers.  What a piece must not read (rows past the k, columns past the row's end)
// has an offset past the descriptor's size and arrives as zeros.
constexpr uint32_t kPast = 0x80000000u;  // of a descriptor of 2^31 - 1 bytes

__device__ __forceinline__ u32x4 descriptor(const void* p) {
  const uint64_t at = reinterpret_cast<uint64_t>(p);
  return {(uint32_t)at, (uint32_t)(at >> 32) & 0xffffu, 0x7fffffffu, 0x00020000u};
}

// Waits until at most N of this wavefront's loads into LDS are on their way and its reads of LDS are
// done, then for the other wavefronts.  (A barrier of the language waits for every load.)
template <int N>
__device__ __forceinline__ void wait_and_meet() {
  static_assert(N <= 63, "the counter has six bits");
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// 16 bytes at each lane's offset to `lds` and the 1 KB behind it, in lane order.  Not by the builtin: the
// compiler takes every transposing read of LDS to depend on every such load before it and waits for
// them all.  (It has no output register; wait_and_meet does the waiting.  The wait states are those
// between a lane's value moved to a scalar register, or m0's, and a load that reads it.)
__device__ __forceinline__ void load_to_lds(u32x4 from, uint32_t offset, uint8_t* lds) {
  const uint32_t at = (uint32_t)reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)lds);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(at), "v"(offset), "s"(from)
               : "memory", "m0");
}

// Half an operand's tile: the first (or second) half of every wavefront's rows, `W` of them each, one
// wavefront after the other.  Its place in the operand's tile:
template <int W>
__device__ __forceinline__ int tile_row(int r, int half) { return r / (W / 2) * W + half * (W / 2) + r % (W / 2); }

// KS > 1: so many groups of wavefronts share a tile, each with its own part of the k and its own stages;
// their sums meet in LDS, in order.
template <typename E, int OP, int BM, int BN, int WM, int WN, int KS>
__device__ __forceinline__ void direct_product(const ProductArgs& p, uint32_t block, int split, uint8_t* lds_all) {
  using T = ProductTile<E, OP, BM, BN, WM, WN>;
  using OpA = Operand<E, BM / 2, T::kKmajA>;  // of half a tile
  using OpB = Operand<E, BN / 2, T::kKmajB>;
  constexpr int kThreads = T::kThreads, kK = OpA::kK, kMt = T::kMt, kNt = T::kNt, kSteps = 2, kStage = T::kStages / 2;
  constexpr int eb = sizeof(E);
  const int tid = KS == 1 ? threadIdx.x : threadIdx.x % kThreads, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int part = KS == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / kThreads);
  uint8_t* const lds = lds_all + part * T::kStages;

  Place at;
  if (!find_place<OP, BM, T::kCols>(p, count_tiles<OP, BM>(p), block >> 3, at)) return;
  at.split = split;

  // this part's first k and its stages; past the last k, loads bring zeros
  const int all = (at.K + kK - 1) / kK, parts = KS * p.splits, stages = (all + parts - 1) / parts;
  const int first = (split * KS + part) * stages;
  const int left = at.K - first * kK;

  // this thread's pieces of each half: byte offsets at the first k, and their k in a stage
  constexpr int kLa = OpA::kPieces / kThreads, kLb = OpB::kPieces / kThreads;
  static_assert(kLa >= 1 && kLb >= 1, "whole loads");
  uint32_t oa[2][kLa], ob[2][kLb];
  int ka[kLa], kb[kLb];
  const int64_t stepa = (T::kKmajA ? p.lda : 1) * (int64_t)(kK * eb), stepb = (T::kKmajB ? p.ldb : 1) * (int64_t)(kK * eb);
  const uint8_t* a = reinterpret_cast<const uint8_t*>(static_cast<const E*>(p.a) + (int64_t)at.row0 * p.lda + at.m0) + first * stepa;
  const uint8_t* b = static_cast<const uint8_t*>(p.b) + first * stepb;
  if constexpr (OP == OP_DW) b += ((int64_t)at.row0 * p.ldb + at.n0) * eb;
  else if constexpr (OP == OP_DX) b += (at.g * p.gsb + at.n0) * eb;
  else b += (at.g * p.gsb + (int64_t)at.n0 * p.ldb) * eb;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int i = 0; i < kLa; ++i) {
      int r;
      OpA::where(i * kThreads + tid, r, ka[i]);
      r = tile_row<WM>(r, h);
      if constexpr (T::kKmajA) oa[h][i] = r < at.M ? (uint32_t)(ka[i] * p.lda + r) * eb : kPast;
      else oa[h][i] = (uint32_t)(min(r, at.M - 1) * p.lda + ka[i]) * eb;
    }
#pragma unroll
    for (int i = 0; i < kLb; ++i) {
      int r;
      OpB::where(i * kThreads + tid, r, kb[i]);
      r = tile_row<WN>(r, h);
      if constexpr (T::kKmajB) ob[h][i] = r < at.N ? (uint32_t)(kb[i] * p.ldb + r) * eb : kPast;
      else ob[h][i] = (uint32_t)((n_row<OP, WN>(p, at, r) - at.n0) * p.ldb + kb[i]) * eb;
    }
  }

  // A stage in LDS: A's halves, then B's.
  const auto place_a = [&](int s, int h) { return lds + (s & 1) * kStage + h * OpA::kBytes; };
  const auto place_b = [&](int s, int h) { return lds + (s & 1) * kStage + 2 * OpA::kBytes + h * OpB::kBytes; };
  // Half h of stage s on its way (past the k: zeros, from nowhere).
  const auto issue_a = [&](int s, int h) {
    const u32x4 from = descriptor(a + s * stepa);
    uint8_t* to = place_a(s, h) + 1024 * wave;
#pragma unroll
    for (int i = 0; i < kLa; ++i) load_to_lds(from, ka[i] < left - s * kK ? oa[h][i] : kPast, to + 16 * i * kThreads);
  };
  const auto issue_b = [&](int s, int h) {
    const u32x4 from = descriptor(b + s * stepb);
    uint8_t* to = place_b(s, h) + 1024 * wave;
#pragma unroll
    for (int i = 0; i < kLb; ++i) load_to_lds(from, kb[i] < left - s * kK ? ob[h][i] : kPast, to + 16 * i * kThreads);
  };

  // A stage is four phases, the products of A's and B's halves (0,0), (0,1), (1,0), (1,1) over all of its
  // k: a half's operands are in registers for two of them, so its place in LDS is free for the stage
  // after next as soon as every wavefront has read it, long before the stage is over.  Between its matrix
  // instructions a phase reads what the next one lacks and sends for one half:
  //   phase          0            1            2              3
  //   reads          B1           A1           A0 of s + 1    B0 of s + 1
  //   sends for      B0 of s + 2  B1 of s + 2  A1 of s + 2    A0 of s + 3
  // What it reads was sent for seven phases ago: the loads of the six since may be on their way.  The
  // wavefronts meet behind a phase's first instructions, which the matrix cores work on meanwhile.
  f32x4 acc[kMt][kNt] = {};
  constexpr int kMh = kMt / 2, kNh = kNt / 2, kMuls = kMh * kNh * kSteps;
  u32x4 fa[2][kMh][kSteps], fb[2][kNh][kSteps];
  const int wm = wave / (BN / WN) * (WM / 2), wn = wave % (BN / WN) * (WN / 2);  // in a half
  const auto read_a = [&](int s, int h, int i) { fa[h][i % kMh][i / kMh] = OpA::fragment(place_a(s, h), wm + 16 * (i % kMh), i / kMh, lane); };
  const auto read_b = [&](int s, int h, int i) { fb[h][i % kNh][i / kNh] = OpB::fragment(place_b(s, h), wn + 16 * (i % kNh), i / kNh, lane); };
  const auto phase = [&](int s, auto which) {
    constexpr int q = decltype(which)::value, ha = q >> 1, hb = q & 1;
    constexpr int kWait = q == 0 ? 4 * kLa + 2 * kLb : q == 2 ? 2 * kLa + 4 * kLb : 3 * kLa + 3 * kLb;
    constexpr int kFirst = kMuls >= 4 ? 2 : 1, kSlots = kMuls - kFirst, kReads = (q == 1 || q == 2 ? kMh : kNh) * kSteps;
#pragma unroll
    for (int i = 0; i < kMuls; ++i) {
      if (i == kFirst) {
        wait_and_meet<kWait>();
        if constexpr (q == 0) issue_b(s + 2, 0);
        else if constexpr (q == 1) issue_b(s + 2, 1);
        else if constexpr (q == 2) issue_a(s + 2, 1);
        else issue_a(s + 3, 0);
      }
      const int j = i / (kMh * kNh), m = i / kNh % kMh, n = i % kNh;
      multiply<E>(fb[hb][n][j], fa[ha][m][j], acc[ha * kMh + m][hb * kNh + n]);
      const int k = i - kFirst;
      if (k >= 0) {
#pragma unroll
        for (int f = k * kReads / kSlots; f < (k + 1) * kReads / kSlots; ++f) {
          if constexpr (q == 0) read_b(s, 1, f);
          else if constexpr (q == 1) read_a(s, 1, f);
          else if constexpr (q == 2) read_a(s + 1, 0, f);
          else read_b(s + 1, 0, f);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  if (stages) {
    // stages 0 and 1, in the order in which they are read
    issue_a(0, 0);
    issue_b(0, 0);
    issue_b(0, 1);
    issue_a(0, 1);
    issue_a(1, 0);
    issue_b(1, 0);
    issue_b(1, 1);
    issue_a(1, 1);
    wait_and_meet<3 * kLa + 3 * kLb>();
#pragma unroll
    for (int i = 0; i < kMh * kSteps; ++i) read_a(0, 0, i);
#pragma unroll
    for (int i = 0; i < kNh * kSteps; ++i) read_b(0, 0, i);
    wait_and_meet<63>();
    issue_a(2, 0);
    __builtin_amdgcn_sched_barrier(0);
    for (int s = 0; s < stages; ++s) {
      phase(s, std::integral_constant<int, 0>{});
      phase(s, std::integral_constant<int, 1>{});
      phase(s, std::integral_constant<int, 2>{});
      phase(s, std::integral_constant<int, 3>{});
    }
  }
  wait_and_meet<0>();
  if constexpr (KS > 1) {
    static_assert(T::kWaves * kMt * kNt * 1024 <= T::kStages, "a part's sums take its stages' place");
    const auto sum = [&](int from, int m, int n) {
      return reinterpret_cast<f32x4*>(lds_all + from * T::kStages) + ((wave * kMt + m) * kNt + n) * 64 + lane;
    };
    if (part) {
#pragma unroll
      for (int m = 0; m < kMt; ++m)
#pragma unroll
        for (int n = 0; n < kNt; ++n) *sum(part, m, n) = acc[m][n];
    }
    __syncthreads();
    if (part) return;
#pragma unroll
    for (int m = 0; m < kMt; ++m)
#pragma unroll
      for (int n = 0; n < kNt; ++n)
#pragma unroll
        for (int o = 1; o < KS; ++o) acc[m][n] += *sum(o, m, n);
  }
  write_tile<E, OP, BM, BN, WM, WN>(p, at, lds_all + wave * T::kPatch, wave, lane, acc);
}

// (WAVES: of a SIMD unit)
template <typename E, int OP, int BM, int BN, int WM, int WN, int KS, int WAVES>
__global__ __launch_bounds__(KS * 64 * (BM / WM) * (BN / WN), WAVES) void product_direct_kernel(ProductArgs p) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[KS * ProductTile<E, OP, BM, BN, WM, WN>::kStages];
  direct_product<E, OP, BM, BN, WM, WN, KS>(p, blockIdx.x, blockIdx.y, lds);
}

// Both gradients of a projection in one launch, for sizes at which neither fills the CUs for long: the
// first workgroups have dx's tiles (and splits), the others dw's.
template <typename E, int BM, int BN, int WM, int WN, int WAVES, bool STAGED>
__global__ __launch_bounds__(64 * (BM / WM) * (BN / WN), WAVES) void gradients_kernel(ProductArgs dx, uint32_t dx_blocks, ProductArgs dw,
                                                                                      uint32_t dw_blocks) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[ProductTile<E, OP_DX, BM, BN, WM, WN>::kStages];
  static_assert(sizeof(lds) == ProductTile<E, OP_DW, BM, BN, WM, WN>::kStages, "one size for both");
  const uint32_t others = dx_blocks * dx.splits;
  if (blockIdx.x < others) {
    const uint32_t split = blockIdx.x / dx_blocks, block = blockIdx.x - split * dx_blocks;
    if constexpr (STAGED) staged_product<E, OP_DX, BM, BN, WM, WN, 3>(dx, block, split, lds);
    else direct_product<E, OP_DX, BM, BN, WM, WN, 1>(dx, block, split, lds);
  } else {
    const uint32_t i = blockIdx.x - others, split = i / dw_blocks, block = i - split * dw_blocks;
    if constexpr (STAGED) staged_product<E, OP_DW, BM, BN, WM, WN, 3>(dw, block, split, lds);
    else direct_product<E, OP_DW, BM, BN, WM, WN, 1>(dw, block, split, lds);
  }
}

// ---------------------------------------------------------------- few rows
// One token's products, or a few tokens': the weights are read once and everything else is small, so a
// workgroup has sixteen rows of weights (eight outputs' gate and up, or sixteen outputs) and up to
// sixteen rows of x, its eight wavefronts deal out the k in lines of 128 bytes, and operands go from
// memory to registers: no stage to fill, no barrier but the one before the wavefronts' sums are added, in
// order.  Loads of four lines are on their way at once.  (Thirty-two rows of x a workgroup were slower at
// almost every size.)
constexpr int kFewWaves = 8, kFewLines = 4;
template <int OP>
constexpr int kFewCols = OP == OP_GLU ? 8 : 16;

template <typename E, int OP>
__global__ __launch_bounds__(64 * kFewWaves) void few_rows_kernel(ProductArgs p) {
  constexpr int kEl = 16 / sizeof(E), kLine = 128 / sizeof(E), kCols = kFewCols<OP>;
  __shared__ f32x4 sums[kFewWaves][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  Place at;
  if (!find_place<OP, 16, kCols>(p, count_tiles<OP, 16>(p), blockIdx.x >> 3, at)) return;
  const int r = lane & 15, q = lane >> 4, K = p.K;
  const int64_t wrow = at.n0 + min(r % kCols, at.N - 1) + (r < kCols ? 0 : p.N);
  const uint8_t* pw = reinterpret_cast<const uint8_t*>(static_cast<const E*>(p.b) + at.g * p.gsb + wrow * p.ldb);
  const uint8_t* px = reinterpret_cast<const uint8_t*>(static_cast<const E*>(p.a) + (int64_t)(at.row0 + min(r, at.M - 1)) * p.lda);
  f32x4 acc = {};
  const int lines = (K + kLine - 1) / kLine;
  for (int l0 = wave; l0 < lines; l0 += kFewWaves * kFewLines) {
    u32x4 w[kFewLines][2], x[kFewLines][2];
#pragma unroll
    for (int l = 0; l < kFewLines; ++l)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        // a piece past the k is the row's last one instead, and then zeros
        const int64_t k = (int64_t)min((l0 + l * kFewWaves) * kLine + (4 * j + q) * kEl, K - kEl) * sizeof(E);
        w[l][j] = load16<false>(pw + k);
        x[l][j] = load16<false>(px + k);
      }
#pragma unroll
    for (int l = 0; l < kFewLines; ++l)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const bool in = (l0 + l * kFewWaves) * kLine + (4 * j + q) * kEl < K;
        multiply<E>(in ? w[l][j] : u32x4{0, 0, 0, 0}, in ? x[l][j] : u32x4{0, 0, 0, 0}, acc);
      }
  }
  sums[wave][lane] = acc;
  __syncthreads();
  // a lane of the sums has rows of weights 4 (l / 16) + 0..3 of x's row l % 16; here, one output a thread
  const int row = threadIdx.x / kCols, c = threadIdx.x % kCols;
  if (row >= at.M || c >= at.N) return;
  const auto sum = [&](int n) {
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < kFewWaves; ++k) v += sums[k][row + 16 * (n >> 2)][n & 3];
    return v;
  };
  const int64_t i = at.row0 + row;
  const int col = at.n0 + c;
  constexpr int fmt = sizeof(E) == 2 ? MOE_AFMT_BF16 : MOE_AFMT_F32;
  float v = sum(c);
  if constexpr (OP == OP_GLU) {
    const float u = sum(c + kCols);
    if (p.aux) {
      write1(p.aux, i * p.ld_aux + col, fmt, v);
      write1(p.aux, i * p.ld_aux + p.N + col, fmt, u);
    }
    write1(p.out, i * p.ldo + col, fmt, act_of(v, p.act).value * u);
  } else {
    if (p.bias) v += p.bias[(int64_t)at.g * p.N + col];
    if (p.aux) write1(p.aux, i * p.ld_aux + col, fmt, v);
    v = act_of(v, p.act).value;
    if (p.residual) v += p.out_fmt == MOE_AFMT_BF16 ? load_act<MOE_AFMT_BF16>(p.residual, i * p.ld_res + col)
                                                    : load_act<MOE_AFMT_F32>(p.residual, i * p.ld_res + col);
    write1(p.out, i * p.ldo + col, p.out_fmt, v);
  }
}

}  // namespace rmoe
