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
__device__ __forceinline__ void write8(void* base, int64_t at, int fmt, int n, const float (&v)[8]) {
  if (fmt == MOE_AFMT_BF16) {
    uint16_t* p = static_cast<uint16_t*>(base) + at;
    u32x4 q;
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    if (n >= 8) {
      store16<false>(reinterpret_cast<uint8_t*>(p), q);
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
      store16<false>(reinterpret_cast<uint8_t*>(p), a);
      store16<false>(reinterpret_cast<uint8_t*>(p + 4), b);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) p[i] = v[i];
    }
  }
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

// Workgroups go round the eight XCDs; XCD x takes the x-th eighth of the tiles' order, so tiles
// that share operands share an L2.  -1: none.
__device__ __forceinline__ int64_t tile_of_block(uint32_t total) {
  const uint32_t per = (total + 7) / 8, i = blockIdx.x >> 3;
  const uint64_t t = (uint64_t)(blockIdx.x & 7) * per + i;
  return i < per && t < total ? (int64_t)t : -1;
}

__device__ __forceinline__ uint32_t add_sat(uint32_t a, uint32_t b) { return a + b < a ? 0xffffffffu : a + b; }

// A row tile's place: expert, first row, its rows (at most BM), the column tile.
struct TileAt {
  int g, row0, rows, n;
};

// Band order: eight row tiles high, then column by column, so about as many row tiles as
// column tiles are in flight on an XCD.
__device__ __forceinline__ void band_order(uint32_t r, int mt, int nt, int& m, int& n) {
  constexpr int kBand = 8;
  const uint32_t band = r / (uint32_t)(kBand * nt), in = r - band * (kBand * nt);
  const int high = min(kBand, mt - (int)band * kBand);
  n = in / high;
  m = band * kBand + in % high;
}

// The workgroup's row tile among all experts'; every wavefront finds it by itself, its lanes
// counting the tiles of E / 64 experts each.
template <int BM>
__device__ __forceinline__ bool find_tile(const int32_t* offsets, int rows, int E, int nt, TileAt& t) {
  const int lane = threadIdx.x & 63;
  if (!offsets) {
    const int mt = (rows + BM - 1) / BM;
    const int64_t b = tile_of_block((uint32_t)mt * nt);
    if (b < 0) return false;
    int m;
    band_order((uint32_t)b, mt, nt, m, t.n);
    t.g = 0;
    t.row0 = m * BM;
    t.rows = min(BM, rows - m * BM);
    return true;
  }
  const int per = (E + 63) / 64, g0 = lane * per;
  uint32_t mine = 0;
  for (int i = 0; i < per; ++i)
    if (g0 + i < E) mine += (expert_rows(offsets, g0 + i, rows).n + BM - 1) / BM;
  uint32_t incl = mine;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t v = __shfl_up(incl, o);
    if (lane >= o) incl = add_sat(incl, v);
  }
  const uint32_t mts = __builtin_amdgcn_readlane(incl, 63);
  // (tables that are no offsets may count more tiles than rows allow: those past 32 bits have no workgroup)
  const uint64_t all = (uint64_t)mts * nt;
  const int64_t b = tile_of_block(all > 0x7fffffffu ? 0x7fffffffu : (uint32_t)all);
  if (b < 0) return false;
  const uint64_t past = __ballot((uint64_t)incl * nt > (uint64_t)b);
  const int at = __ffsll((unsigned long long)past) - 1;
  uint32_t before = at ? (uint32_t)__builtin_amdgcn_readlane(incl, at - 1) : 0u;
  int g = at * per;
  for (;; ++g) {
    const Range r = expert_rows(offsets, g, rows);
    const uint32_t mt = (r.n + BM - 1) / BM;
    if ((uint64_t)(before + mt) * nt > (uint64_t)b) {
      int m;
      band_order((uint32_t)(b - (int64_t)before * nt), mt, nt, m, t.n);
      t.g = __builtin_amdgcn_readfirstlane(g);
      t.row0 = __builtin_amdgcn_readfirstlane(r.first + m * BM);
      t.rows = __builtin_amdgcn_readfirstlane(min(BM, r.n - m * BM));
      t.n = __builtin_amdgcn_readfirstlane(t.n);
      return true;
    }
    before += mt;
  }
}

// ---------------------------------------------------------------- operands
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

// An operand in LDS: R tile rows by 128 bytes of k, in 16-byte pieces.
//  k in a row (KMAJ = false): piece c of tile row r at (8 r + (c ^ r % 8)): the eight rows that
//    eight lanes read at one c lie in eight different pieces of a 128-byte line of banks;
//  a tile row per k (KMAJ = true): k's R elements in R / n pieces (n elements each), piece c at
//    c ^ f(k): the rows that one transposing read (16-bit) or the two halves of a wavefront
//    (fp32) take together lie 64 or 128 bytes apart.
template <typename E, int R, bool KMAJ>
struct Operand {
  static constexpr int kEl = 16 / sizeof(E);       // elements of a piece
  static constexpr int kK = 128 / sizeof(E);       // k of a stage
  static constexpr int kBytes = R * 128;
  static constexpr int kPieces = R * 8;
  static constexpr int kPerK = R * (int)sizeof(E) / 16;  // pieces of one k (KMAJ)

  __device__ static __forceinline__ int swizzle(int k) {
    return sizeof(E) == 2 ? 4 * (k & 3) : 8 * ((k >> 2) & 1);
  }
  // Of piece s (16 bytes at 16 s): its tile row and first k, or its k and first tile row.
  __device__ static __forceinline__ void where(int s, int& row, int& k) {
    if constexpr (KMAJ) {
      k = s / kPerK;
      row = ((s % kPerK) ^ swizzle(k)) * kEl;
    } else {
      row = s / 8;
      k = ((s % 8) ^ (row % 8)) * kEl;
    }
  }
  // The matrix instruction's operand of 32 tile rows from r0 (a multiple of 32) at step j of a
  // stage's four: lane l has row r0 + l % 32 and the 16 bytes of k that follow (32 j + 16 (l / 32)) bytes.
  // (In fp32 a step is four instructions of two k each, whose order is the same on both sides.)
  __device__ static __forceinline__ u32x4 fragment(const uint8_t* lds, int r0, int j, int lane) {
    const int r = lane & 31, h = lane >> 5;
    if constexpr (!KMAJ) {
      return *reinterpret_cast<const u32x4*>(lds + (r0 + r) * 128 + (((2 * j + h) ^ (r & 7)) << 4));
    } else if constexpr (sizeof(E) == 2) {
      // 16 lanes read four k of 16 tile rows, 8 bytes each, and get four k of one tile row each
      const int i = lane & 15, c = r0 / 8 + 2 * ((lane >> 4) & 1) + ((i & 3) >> 1);
      const uint8_t* p = lds + (16 * j + 8 * h + (i >> 2)) * (R * 2) + ((c ^ (4 * (i >> 2))) << 4) + ((i & 1) << 3);
      typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p));
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * (R * 2)));
      return __builtin_bit_cast(u32x4, (s16x8)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      u32x4 v;
      const int m = r0 + r;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = *reinterpret_cast<const uint32_t*>(lds + (8 * j + 4 * h + i) * (R * 4) + (((m >> 2) ^ (8 * h)) << 4) +
                                                  ((m & 3) << 2));
      return v;
    }
  }
};

template <typename E>
__device__ __forceinline__ void multiply(u32x4 a, u32x4 b, f32x16& acc) {
  if constexpr (sizeof(E) == 2) {
    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), acc, 0, 0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[i]), __uint_as_float(b[i]), acc, 0, 0, 0);
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
// A workgroup has a BM x BN tile of C, a wavefront WM x WN of it in fragments of 32 x 32.  The
// matrix instruction's rows are n and its columns m, so that a lane holds four neighbouring
// outputs of one row.
template <typename E, int OP, int BM, int BN, int WM, int WN>
struct ProductTile {
  static constexpr int kThreads = 64 * (BM / WM) * (BN / WN);
  static constexpr int kMt = WM / 32, kNt = WN / 32;
  using OpA = Operand<E, BM, OP == OP_DW>;
  using OpB = Operand<E, BN, OP == OP_DX || OP == OP_DW>;
  static constexpr int kStage = OpA::kBytes + OpB::kBytes;
  static constexpr int kPatch = 32 * WN * 4;  // a wavefront's fragment row in fp32, for the epilogue
  static constexpr int kLds = 2 * kStage;
  static_assert(kPatch * (kThreads / 64) <= kLds, "the epilogue's patches take the stages' place");
  static constexpr int kCols = OP == OP_GLU ? BN / 2 : BN;  // outputs of a tile's row
};

template <typename E, int OP, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * (BM / WM) * (BN / WN)) void product_kernel(ProductArgs p) {
  using T = ProductTile<E, OP, BM, BN, WM, WN>;
  constexpr int kThreads = T::kThreads, kK = T::OpA::kK, kEl = T::OpA::kEl;
  __shared__ __attribute__((aligned(16))) uint8_t lds[T::kLds];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / (BN / WN) * WM, wn = wave % (BN / WN) * WN;
  const int nt = (p.N + T::kCols - 1) / T::kCols;

  TileAt t;
  int m0 = 0, M, K = p.K;
  if constexpr (OP == OP_DW) {
    const int mt = (p.M + BM - 1) / BM;
    const int64_t b = tile_of_block((uint32_t)p.E * mt * nt);
    if (b < 0) return;
    t.g = (int)(b / (mt * nt));
    int m;
    band_order((uint32_t)(b % (mt * nt)), mt, nt, m, t.n);
    const Range r = expert_rows(p.offsets, t.g, p.rows);
    t.row0 = r.first;
    K = r.n;
    m0 = m * BM;
    M = min(BM, p.M - m0);
  } else {
    if (!find_tile<BM>(p.offsets, p.rows, p.E, nt, t)) return;
    M = t.rows;
  }
  const int n0 = t.n * T::kCols, N = min(T::kCols, p.N - n0);

  // this thread's pieces: an address (k = 0) and, in `left`, how many of its elements there are
  constexpr int kPa = T::OpA::kPieces / kThreads, kPb = T::OpB::kPieces / kThreads;
  const uint8_t *pa[kPa], *pb[kPb];
  int ka[kPa], kb[kPb];  // k of the piece in a stage; where rows are the k, beside it the elements in the row
  int la[kPa], lb[kPb];
  const E* a = static_cast<const E*>(p.a);
  const E* b = static_cast<const E*>(p.b);
#pragma unroll
  for (int i = 0; i < kPa; ++i) {
    int r;
    T::OpA::where(i * kThreads + tid, r, ka[i]);
    if constexpr (OP == OP_DW) {
      la[i] = M - r;
      pa[i] = reinterpret_cast<const uint8_t*>(a + (int64_t)(t.row0 + ka[i]) * p.lda + m0 + r);
    } else {
      la[i] = 0;
      pa[i] = reinterpret_cast<const uint8_t*>(a + (int64_t)(t.row0 + min(r, M - 1)) * p.lda + ka[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < kPb; ++i) {
    int r;
    T::OpB::where(i * kThreads + tid, r, kb[i]);
    if constexpr (OP == OP_DW) {
      lb[i] = N - r;
      pb[i] = reinterpret_cast<const uint8_t*>(b + (int64_t)(t.row0 + kb[i]) * p.ldb + n0 + r);
    } else if constexpr (OP == OP_DX) {
      lb[i] = N - r;
      pb[i] = reinterpret_cast<const uint8_t*>(b + t.g * p.gsb + (int64_t)kb[i] * p.ldb + n0 + r);
    } else {
      lb[i] = 0;
      int64_t row;
      if constexpr (OP == OP_GLU) {  // a wavefront's columns: WN / 2 of the gate, then the same of up
        const int c = r / WN * (WN / 2) + r % (WN / 2);
        row = n0 + min(c, N - 1) + (r % WN >= WN / 2 ? p.N : 0);
      } else {
        row = n0 + min(r, N - 1);
      }
      pb[i] = reinterpret_cast<const uint8_t*>(b + t.g * p.gsb + row * p.ldb + kb[i]);
    }
  }
  u32x4 qa[kPa], qb[kPb];
  const auto load = [&](int k0) {
#pragma unroll
    for (int i = 0; i < kPa; ++i) {
      if constexpr (OP == OP_DW) qa[i] = read_piece<E>(pa[i] + (int64_t)k0 * p.lda * sizeof(E), k0 + ka[i] < K ? la[i] : 0);
      else qa[i] = read_piece<E>(pa[i] + (int64_t)k0 * sizeof(E), K - k0 - ka[i]);
    }
#pragma unroll
    for (int i = 0; i < kPb; ++i) {
      if constexpr (OP == OP_DW || OP == OP_DX)
        qb[i] = read_piece<E>(pb[i] + (int64_t)k0 * p.ldb * sizeof(E), k0 + kb[i] < K ? lb[i] : 0);
      else qb[i] = read_piece<E>(pb[i] + (int64_t)k0 * sizeof(E), K - k0 - kb[i]);
    }
  };
  const auto store = [&](uint8_t* stage) {
#pragma unroll
    for (int i = 0; i < kPa; ++i) *reinterpret_cast<u32x4*>(stage + 16 * (i * kThreads + tid)) = qa[i];
#pragma unroll
    for (int i = 0; i < kPb; ++i) *reinterpret_cast<u32x4*>(stage + T::OpA::kBytes + 16 * (i * kThreads + tid)) = qb[i];
  };

  f32x16 acc[T::kMt][T::kNt] = {};
  const int stages = (K + kK - 1) / kK;
  if (stages) {
    load(0);
    store(lds);
    __syncthreads();
  }
  for (int s = 0; s < stages; ++s) {
    const uint8_t* at = lds + (s & 1) * T::kStage;
    if (s + 1 < stages) load((s + 1) * kK);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u32x4 fa[T::kMt], fb[T::kNt];
#pragma unroll
      for (int i = 0; i < T::kMt; ++i) fa[i] = T::OpA::fragment(at, wm + 32 * i, j, lane);
#pragma unroll
      for (int i = 0; i < T::kNt; ++i) fb[i] = T::OpB::fragment(at + T::OpA::kBytes, wn + 32 * i, j, lane);
#pragma unroll
      for (int m = 0; m < T::kMt; ++m)
#pragma unroll
        for (int n = 0; n < T::kNt; ++n) multiply<E>(fb[n], fa[m], acc[m][n]);
    }
    if (s + 1 < stages) store(lds + ((s + 1) & 1) * T::kStage);
    __syncthreads();
  }

  // Epilogue: 32 rows of the wavefront's columns at a time go through LDS (16-byte pieces, piece c
  // of row r at c ^ r), so that eight neighbouring outputs of a row meet in one lane and rows are
  // written in whole lines.
  uint8_t* patch = lds + wave * T::kPatch;
  constexpr int kSwz = (WN / 4 - 1) & 31;
  constexpr int kOut = OP == OP_GLU ? WN / 2 : WN;        // outputs of a row
  constexpr int kLanes = kOut / 8, kRows = 64 / kLanes;   // lanes of a row, rows at once
  const int cl = 8 * (lane % kLanes);
  const int col = n0 + (OP == OP_GLU ? wn / 2 : wn) + cl, cols = p.N - col;
#pragma unroll
  for (int m = 0; m < T::kMt; ++m) {
    {
      const int r = lane & 31, h = lane >> 5;
#pragma unroll
      for (int n = 0; n < T::kNt; ++n)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x4 v = {acc[m][n][4 * q], acc[m][n][4 * q + 1], acc[m][n][4 * q + 2], acc[m][n][4 * q + 3]};
          *reinterpret_cast<f32x4*>(patch + r * (WN * 4) + (((8 * n + 2 * q + h) ^ (r & kSwz)) << 4)) = v;
        }
    }
    __builtin_amdgcn_wave_barrier();
#pragma unroll 2
    for (int i = 0; i < 32 / kRows; ++i) {
      const int r = i * kRows + lane / kLanes, row = wm + 32 * m + r;
      const auto get = [&](int c, float (&v)[8]) {
        const f32x4 x = *reinterpret_cast<const f32x4*>(patch + r * (WN * 4) + (((c / 4) ^ (r & kSwz)) << 4));
        const f32x4 y = *reinterpret_cast<const f32x4*>(patch + r * (WN * 4) + (((c / 4 + 1) ^ (r & kSwz)) << 4));
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
      if (row >= M || cols <= 0) continue;
      if constexpr (OP == OP_DW) {
        write8(p.out, ((int64_t)t.g * p.M + m0 + row) * p.N + col, p.out_fmt, cols, v);
      } else {
        const int64_t at = t.row0 + row;
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
            read8(p.bias, (int64_t)t.g * p.N + col, MOE_AFMT_F32, cols, w);
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
          write8(p.out, at * p.ldo + col, p.out_fmt, cols, v);
        }
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
}

}  // namespace rmoe
