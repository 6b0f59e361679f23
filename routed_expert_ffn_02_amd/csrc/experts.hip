// The experts' products over rows sorted by expert, and their gradients: the gated half of a
// feed-forward block (both projections, activation and product in one kernel), a projection with
// bias, activation and residual, for experts and shared experts that run outside a context.
//
//   glu      gu = x W^T, a = act(gu_gate) gu_up          dgu = [da u act'(g) | da act(g)], dx = dgu W, dW = dgu^T x
//   linear   z = x W^T + b, y = act(z) + r               dz = dy act'(z), dx = dz W, dW = dz^T x, db = sum dz
//
// The products are tiles on the matrix cores (products.hpp).
#include <cmath>

#include "products.hpp"

namespace rmoe {

constexpr int kProductMaxRows = 1 << 26;
constexpr int kProductMaxSize = 1 << 16;  // of a row of x, of the outputs

// ---------------------------------------------------------------- the gradient before the projection
// d = dgu (glu) or dz (linear), rounded to the operands' type: the products that follow take it as
// an operand, as autograd's do, with zeros up to ld_d behind each row.  Eight elements a lane; rows before
// the first expert's and behind the last one's are left out.
__device__ __forceinline__ void pad_row(void* d, int64_t at, int from, int64_t to, int fmt) {
  for (int e = from; e < to; ++e) write1(d, at + e, fmt, 0.f);
}

// From the first row that any expert has to the last one: offsets[0] and offsets[E] of a table that ascends; the least and
// the greatest entry of another, so that no expert's d is missing.  All of a wavefront's lanes take part.
__device__ __forceinline__ Range rows_in_use(const int32_t* offsets, int E, int rows) {
  if (!offsets) return {0, rows};
  int lo = rows, hi = 0;
  for (int i = threadIdx.x & 63; i <= E; i += 64) {
    const int o = min(max(offsets[i], 0), rows);
    lo = min(lo, o);
    hi = max(hi, o);
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    lo = min(lo, __shfl_xor(lo, o));
    hi = max(hi, __shfl_xor(hi, o));
  }
  return {lo, hi - lo};
}

template <bool GLU>
__global__ __launch_bounds__(256) void pre_gradient_kernel(const void* __restrict__ dy, int dy_fmt, int64_t ld_dy,
                                                           const void* __restrict__ z, int fmt, int64_t ld_z,
                                                           const int32_t* __restrict__ offsets, int rows, int E, int n,
                                                           int act, void* __restrict__ d, int64_t ld_d) {
  const int c = 8 * (blockIdx.y * 64 + (threadIdx.x & 63));
  const Range r = rows_in_use(offsets, E, rows);
  if (c >= n) return;
  const int all = GLU ? 2 * n : n, end = r.first + r.n;
  for (int row = r.first + 4 * blockIdx.x + (threadIdx.x >> 6); row < end; row += 4 * gridDim.x) {
    float g[8], u[8], v[8];
    read8(dy, (int64_t)row * ld_dy + c, dy_fmt, n - c, v);
    if (GLU || act != MOE_ACT_NONE) read8(z, (int64_t)row * ld_z + c, fmt, n - c, g);
    if constexpr (GLU) {
      read8(z, (int64_t)row * ld_z + n + c, fmt, n - c, u);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const Act f = act_of(g[e], act);
        g[e] = v[e] * u[e] * f.grad;
        v[e] *= f.value;
      }
      write8(d, (int64_t)row * ld_d + c, fmt, n - c, g);
      write8(d, (int64_t)row * ld_d + n + c, fmt, n - c, v);
    } else {
      if (act != MOE_ACT_NONE) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= act_of(g[e], act).grad;
      }
      write8(d, (int64_t)row * ld_d + c, fmt, n - c, v);
    }
    if (c + 8 >= n) pad_row(d, row * ld_d, all, ld_d, fmt);
  }
}

// ---------------------------------------------------------------- the bias's gradient
// Column sums of dz in fp32, from dy and z as given (dz is not rounded before), and, where it is asked
// for, dz itself as the products take it (d, as pre_gradient_kernel writes it).  A workgroup has 64
// columns, eight lanes of eight, and 32 rows at once; its rows' sums meet in LDS in a fixed order.
// Splits of a long expert write their own sums, which bias_join adds in order: 32 rows a split and more, up to 64
// splits.  Calls for the bias alone, in bf16, with up to 64 splits and up to 256: 777 rows of 1001 with gelu 8.9 us and 8.9 (19 in
// one split of sixteen wavefronts), 4096 x 4096 13.2 and 19.7, 32768 x 512 14.3 and 20.7, with gelu 40 and 38; in fp32 65536 x 128
// with gelu 52 and 28, 8192 x 2048 19.4 and 26.7.  (Unrolled as the compiler likes, the loop takes the same at all of these.)
constexpr int kBiasRows = 32;  // rows of a split, at least

__global__ __launch_bounds__(256) void bias_gradient_kernel(const void* __restrict__ dy, int dy_fmt, int64_t ld_dy,
                                                            const void* __restrict__ z, int fmt, int64_t ld_z,
                                                            const int32_t* __restrict__ offsets, int rows, int E, int n,
                                                            int act, int splits, float* __restrict__ out,
                                                            void* __restrict__ d, int64_t ld_d) {
  __shared__ float part[4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = 64 * blockIdx.x + 8 * (lane & 7);
  const Range r = expert_rows(offsets, blockIdx.y, rows);
  const int len = (r.n + splits - 1) / splits, from = min(r.n, (int)blockIdx.z * len), to = min(r.n, from + len);
  float sum[8] = {};
  if (c < n) {
#pragma unroll 1
    for (int i = from + 8 * wave + (lane >> 3); i < to; i += 32) {
      float v[8], g[8];
      read8(dy, (int64_t)(r.first + i) * ld_dy + c, dy_fmt, n - c, v);
      if (act != MOE_ACT_NONE) {
        read8(z, (int64_t)(r.first + i) * ld_z + c, fmt, n - c, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= act_of(g[e], act).grad;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] += v[e];
      if (d) {
        const int64_t at = (int64_t)(r.first + i) * ld_d;
        write8(d, at + c, fmt, n - c, v);
        if (c + 8 >= n) pad_row(d, at, n, ld_d, fmt);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
#pragma unroll
    for (int o = 8; o < 64; o <<= 1) sum[e] += __shfl_xor(sum[e], o);
    if (lane < 8) part[wave][8 * lane + e] = sum[e];
  }
  __syncthreads();
  const int col = 64 * blockIdx.x + threadIdx.x;
  if (threadIdx.x >= 64 || col >= n) return;
  out[((int64_t)blockIdx.z * E + blockIdx.y) * n + col] =
      (part[0][threadIdx.x] + part[1][threadIdx.x]) + (part[2][threadIdx.x] + part[3][threadIdx.x]);
}

__global__ __launch_bounds__(256) void bias_join_kernel(const float* __restrict__ part, int64_t total, int splits,
                                                        float* __restrict__ out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= total) return;
  float s = 0.f;
#pragma unroll 8
  for (int k = 0; k < splits; ++k) s += part[k * total + i];
  out[i] = s;
}

// The sums of splits over the k, in order: [splits][rows][n] in fp32, of which rows between the first
// expert's and the last one's are written (offsets NULL: all).
__global__ __launch_bounds__(256) void split_join_kernel(const float* __restrict__ part, int64_t plane, int splits,
                                                         const int32_t* __restrict__ offsets, int E, int rows, int n,
                                                         void* __restrict__ out, int64_t ldo, int fmt) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int row = (int)(i / n), col = (int)(i - (int64_t)row * n);
  if (row >= rows || (offsets && (row < offsets[0] || row >= offsets[E]))) return;
  float s = 0.f;
#pragma unroll 8
  for (int k = 0; k < splits; ++k) s += part[k * plane + i];
  write1(out, row * ldo + col, fmt, s);
}

namespace {

int bias_splits(int64_t rows, int64_t E, int64_t n) {
  return (int)std::clamp<int64_t>(std::min<int64_t>(rows / (E * kBiasRows), (1ll << 20) / (E * ((n + 63) / 64))), 1, 64);
}

// ---------------------------------------------------------------- launches
constexpr int64_t kMaxThreads = (1ll << 32) - 1;  // a launch's are counted in 32 bits

// Row tiles of bm (every expert with a row may end in a part of one) times column tiles of `cols` outputs, and
// the grid over them: whole runs on every XCD.
template <int OP>
int64_t tiles_of(const ProductArgs& p, int bm, int cols) {
  const int64_t nt = (p.N + cols - 1) / cols;
  const int64_t mt = OP == OP_DW ? (int64_t)p.E * ((p.M + bm - 1) / bm)
                                 : ((int64_t)p.rows + (int64_t)std::min(p.E, p.rows) * (bm - 1)) / bm;
  return mt * nt;
}
template <int OP>
int64_t blocks_of(const ProductArgs& p, int bm, int cols) {
  const int64_t tiles = tiles_of<OP>(p, bm, cols);
  const int64_t eight = 8 * (OP == OP_DW ? (int64_t)dealt_run((uint32_t)std::min<int64_t>(tiles / p.E, 1 << 30)) : 1);
  return (tiles + eight - 1) / eight * eight;
}
template <typename T, int OP, int BM>
moe_status run_tiles(void (*kernel)(ProductArgs), ProductArgs p, int threads, hipStream_t s) {
  const int64_t blocks = blocks_of<OP>(p, BM, T::kCols);
  if (blocks * threads * p.splits > kMaxThreads) return MOE_EINVAL;
  p.tiles = (uint32_t)tiles_of<OP>(p, BM, T::kCols);
  return launch(kernel, dim3((unsigned)blocks, p.splits), dim3(threads), s, p);
}

// Whether the operands' rows start on 16 bytes, whole pieces make up every row (a d of the workspace
// has zeros behind its rows), and a tile's offsets stay below the descriptor's size.
template <typename E, int OP>
bool direct_ok(const ProductArgs& p) {
  constexpr int64_t eb = sizeof(E), el = 16 / eb;
  if (!aligned_to(p.a, 16) || !aligned_to(p.b, 16) || p.lda % el || p.ldb % el || p.gsb % el) return false;
  constexpr int64_t most = (1ll << 31) - (1 << 20);
  if (OP == OP_DW) return (p.M % el == 0 || p.padded) && p.N % el == 0 && std::max(p.lda, p.ldb) * 128 < most;
  if ((p.K % el && !p.padded) || (256 * p.lda + p.K) * eb >= most) return false;
  if (OP == OP_DX) return p.N % el == 0 && p.ldb * 128 < most;
  return ((OP == OP_GLU ? (int64_t)p.N : 0) + 256) * p.ldb * eb + p.K * eb < most;
}

constexpr int kCus = 256;  // MI355X

template <typename E, int OP, int BM, int BN, int WM, int WN, int KS, int PER_CU>
moe_status direct(const ProductArgs& p, hipStream_t s) {
  using T = ProductTile<E, OP, BM, BN, WM, WN>;
  return run_tiles<T, OP, BM>(product_direct_kernel<E, OP, BM, BN, WM, WN, KS, KS * T::kWaves * PER_CU / 4>, p, KS * T::kThreads, s);
}
template <typename E, int OP, int BM, int BN, int WM, int WN, int DEPTH>
moe_status staged(const ProductArgs& p, hipStream_t s) {
  using T = ProductTile<E, OP, BM, BN, WM, WN>;
  return run_tiles<T, OP, BM>(product_kernel<E, OP, BM, BN, WM, WN, DEPTH>, p, T::kThreads, s);
}

// A tile's shape, chosen by its estimated time: rounds of workgroups x what a tile costs beside its
// stages, and per stage (128 bytes of k) the longer of what it takes alone on a CU and of what the CU's
// share of all tiles takes.  The figures (us) were fitted to measured times of 45 to 90 shapes a row (1 to 32768
// rows, up to 256 experts, sizes 512 to 8192).  They rank shapes and do not tell times: no term counts bytes, so what
// memory bounds (grouped products, a short k) is estimated at down to 0.4 of its time.  Of 62 products timed in every
// shape, most of them random ones, the choice is 3% above the best on average and 36% at worst (dw of 2384 rows, 448 x 2112).  In
// bf16, 4096^3: 256 x 256 111 us, 128 x 256 130, 128 x 128 135, 64 x 128 173, 64 x 64 220; 1024 x 4096 x 4096: 83, 51, 41, 43, 52;
// one row of 4096 x 4096: 83, 50, 37, 28, 24, and 17 where four groups of wavefronts share the k.  The last two are
// product_kernel's: 2048^3 in bf16 with rows of 2047 takes 44 us forward, 39 and 38 the gradients, where rows on 16 bytes
// take 25, 26 and 26.
struct TileCost {
  int bm, bn, per_cu, parts;
  float fixed, alone, shared;
};
enum { TILE_256, TILE_128_256, TILE_128, TILE_64_128, TILE_64, TILE_64_PARTS, STAGED_128, STAGED_64, TILES };
constexpr TileCost kCosts[2][3][TILES] = {
    {// fp32: forward, rows' gradient, weights' gradient (no kernel: {})
     {{}, {}, {128, 128, 2, 1, 2.47f, 2.33f, 1.96f}, {64, 128, 3, 1, 2.09f, .90f, 1.f}, {64, 64, 5, 1, 3.51f, .62f, .50f}, {64, 64, 1, 4, 4.71f, 1.77f, 1.87f},
      {}, {64, 64, 3, 1, 4.63f, .75f, .59f}},
     {{}, {}, {128, 128, 2, 1, 2.47f, 2.39f, 1.80f}, {64, 128, 3, 1, 2.74f, 1.06f, .90f}, {64, 64, 5, 1, 2.92f, .88f, .45f}, {64, 64, 1, 4, 4.13f, 1.77f, 1.69f},
      {}, {64, 64, 3, 1, 4.50f, .78f, .57f}},
     {{}, {}, {128, 128, 2, 1, 4.41f, 2.39f, 1.48f}, {64, 128, 3, 1, 2.91f, 1.09f, .74f}, {64, 64, 5, 1, 1.95f, .99f, .42f}, {64, 64, 1, 4, 4.77f, 1.77f, 1.58f},
      {}, {64, 64, 3, 1, 5.43f, .78f, .61f}}},
    {{{256, 256, 1, 1, 4.33f, .90f, 1.64f}, {128, 256, 1, 1, 4.11f, .61f, .94f}, {128, 128, 2, 1, 4.19f, .56f, .47f}, {64, 128, 3, 1, 3.18f, .31f, .29f},
      {64, 64, 5, 1, 2.77f, .32f, .20f}, {64, 64, 1, 4, 5.f, .75f, .56f},
      {128, 128, 2, 1, 6.39f, .91f, 1.06f}, {64, 64, 3, 1, 3.91f, .52f, .32f}},
     {{256, 256, 1, 1, 3.75f, 1.44f, 1.35f}, {128, 256, 1, 1, 5.08f, .68f, .79f}, {128, 128, 2, 1, 2.47f, .43f, .44f}, {64, 128, 3, 1, 3.06f, .57f, .28f},
      {64, 64, 5, 1, 3.51f, .26f, .21f}, {64, 64, 1, 4, 5.f, .90f, .92f},
      {128, 128, 2, 1, 6.85f, .46f, .89f}, {64, 64, 3, 1, 4.00f, .61f, .25f}},
     {{256, 256, 1, 1, 3.75f, .94f, 1.54f}, {128, 256, 1, 1, 3.58f, .70f, 1.f}, {128, 128, 2, 1, 3.38f, .67f, .58f}, {64, 128, 3, 1, 3.51f, .45f, .40f},
      {64, 64, 5, 1, 2.98f, .46f, .20f}, {64, 64, 1, 4, 5.f, 1.05f, .81f},
      {128, 128, 2, 1, 7.42f, .86f, .58f}, {64, 64, 3, 1, 4.44f, .63f, .31f}}}};
static_assert(MOE_AFMT_F32 == 0 && MOE_AFMT_BF16 == 1, "kCosts' first index");

// Row tiles of `bm` that rows over E experts come to, about.
float row_tiles(int64_t rows, int E, int bm) {
  const float used = std::min<int64_t>(E, rows);  // experts with a row, at most
  return E == 1 ? std::ceil((float)rows / bm) : std::max((float)rows / bm + .5f * used, used);
}
float tile_time(const TileCost& c, float tiles, float stages) {
  return std::ceil(tiles / (kCus * c.per_cu)) * c.fixed + std::ceil(stages / c.parts) * std::max(c.alone, std::ceil(tiles / kCus) * c.shared);
}
template <typename E, int OP>
const TileCost* costs_of() { return kCosts[sizeof(E) == 2][OP == OP_DW ? 2 : OP == OP_DX]; }
template <typename E, int OP>
float stages_of(const ProductArgs& p) { return std::ceil((OP == OP_DW ? (float)p.rows / p.E : p.K) / (128 / (int)sizeof(E))); }
template <int OP>
float tiles_like(const ProductArgs& p, int bm, int bn) {
  const int cols = OP == OP_GLU ? bn / 2 : bn;
  return (OP == OP_DW ? (float)p.E * ((p.M + bm - 1) / bm) : row_tiles(p.rows, p.E, bm)) * ((p.N + cols - 1) / cols);
}

template <typename E, int OP>
int choose_tile(const ProductArgs& p, std::initializer_list<int> from, float* estimate) {
  const float stages = stages_of<E, OP>(p);
  int best = -1;
  for (const int i : from) {
    const TileCost& c = costs_of<E, OP>()[i];
    const float time = tile_time(c, tiles_like<OP>(p, c.bm, c.bn), stages);
    if (best < 0 || time < *estimate) {
      best = i;
      *estimate = time;
    }
  }
  return best;
}

// A gradient with few tiles and a long k is cut along the k: 64 x 64 tiles times splits fill the CUs once, each
// split writes its own fp32 sums (some 4 MB in all) to the workspace, and a kernel adds them in order.  From the
// sizes alone, as the workspace's size is; 1: not at all.  Whole calls in bf16, uncut and cut: dx of 17 rows of
// 1023 from 4095 45 us and 12, dw of 511 x 511 from 4096 rows 51 and 26; in fp32 107 and 16, 113 and 43.
constexpr float kJoinUs = 4.f;  // the second launch
int splits_for(float tiles, float stages) { return (int)std::clamp(std::min(kCus / tiles, stages / 2), 1.f, 64.f); }

// Whether few_rows_kernel is the faster one: its time is a launch and the CU's share of workgroups, each of
// which reads sixteen rows of weights.  Measured against the tiles (us, bf16): one row of 512 x 2048 4.9 and
// 5.3, sixteen 6.2 and 5.3; one row of 2048 x 1024 4.8 and 9.3, 64 rows 6.5 and 9.9; one row of 4096 x 4096 7.8
// and 14.9, 64 rows 31 and 16.
template <typename E, int OP>
bool few_rows_ok(const ProductArgs& p, float tiles_time) {
  if constexpr (OP != OP_GLU && OP != OP_LINEAR) return false;
  if (p.K % (16 / (int)sizeof(E))) return false;
  const float per_cu = std::ceil(row_tiles(p.rows, p.E, 16) * ((p.N + kFewCols<OP> - 1) / kFewCols<OP>) / kCus);
  return 3.9f + .06f * std::min(p.rows, 16) + per_cu * (.5f + .7e-3f * sizeof(E) * p.K) < tiles_time;
}

template <typename E, int OP>
moe_status few_rows(ProductArgs p, hipStream_t s) {
  if constexpr (OP == OP_GLU || OP == OP_LINEAR) {
    const int64_t tiles = tiles_of<OP>(p, 16, kFewCols<OP>), blocks = (tiles + 7) / 8 * 8;
    if (blocks * 64 * kFewWaves > kMaxThreads) return MOE_EINVAL;
    p.tiles = (uint32_t)tiles;
    return launch(few_rows_kernel<E, OP>, dim3((unsigned)blocks), dim3(64 * kFewWaves), s, p);
  }
  return MOE_EINVAL;
}

// How a product is done: its tile, the splits of a gradient's k, the estimated time.
struct Plan {
  bool straight;  // from memory to LDS
  int tile, splits;
  float time;
};
template <typename E, int OP>
Plan plan_of(const ProductArgs& p) {
  Plan plan{direct_ok<E, OP>(p), 0, 1, 0.f};
  if (!plan.straight) {
    if constexpr (sizeof(E) == 2) plan.tile = choose_tile<E, OP>(p, {STAGED_128, STAGED_64}, &plan.time);
    else plan.tile = choose_tile<E, OP>(p, {STAGED_64}, &plan.time);
  } else if constexpr (sizeof(E) == 2) {
    plan.tile = choose_tile<E, OP>(p, {TILE_256, TILE_128_256, TILE_128, TILE_64_128, TILE_64, TILE_64_PARTS}, &plan.time);
  } else {
    plan.tile = choose_tile<E, OP>(p, {TILE_128, TILE_64_128, TILE_64, TILE_64_PARTS}, &plan.time);
  }
  if constexpr (OP == OP_DX || OP == OP_DW) {
    const int tile = plan.straight ? TILE_64 : STAGED_64;
    const float tiles = tiles_like<OP>(p, 64, 64), stages = stages_of<E, OP>(p);
    const int splits = splits_for(tiles, stages);
    const float time = kJoinUs + tile_time(costs_of<E, OP>()[tile], tiles * splits, std::ceil(stages / splits));
    if (splits > 1 && time < plan.time) plan = {plan.straight, tile, splits, time};
  }
  return plan;
}

// Its arguments with the splits' own outputs, and the kernel that adds those.
template <int OP>
ProductArgs split(ProductArgs p, int splits, float* part) {
  p.splits = splits;
  p.past_caches = OP == OP_DW && splits == 1 && p.out_fmt == MOE_AFMT_BF16 && p.N % 64 == 0 && aligned_to(p.out, 128);
  if (splits == 1) return p;
  p.plane = (OP == OP_DW ? (int64_t)p.E * p.M : p.rows) * p.N;
  p.out = part;
  p.out_fmt = MOE_AFMT_F32;
  p.ldo = p.N;
  return p;
}
template <int OP>
moe_status join(const ProductArgs& p, int splits, const float* part, hipStream_t s) {
  if (splits == 1) return MOE_OK;
  const int rows = OP == OP_DW ? p.E * p.M : p.rows;
  const int64_t plane = (int64_t)rows * p.N;
  return launch(split_join_kernel, dim3((unsigned)((plane + 255) / 256)), dim3(256), s, part, plane, splits,
                OP == OP_DW ? nullptr : p.offsets, p.E, rows, p.N, p.out, OP == OP_DW ? p.N : p.ldo, p.out_fmt);
}

template <typename E, int OP>
moe_status run_plan(const ProductArgs& p, int tile, hipStream_t s) {
  if constexpr (sizeof(E) == 2) {
    if (tile == TILE_256) return direct<E, OP, 256, 256, 128, 64, 1, 1>(p, s);
    if (tile == TILE_128_256) return direct<E, OP, 128, 256, 64, 64, 1, 1>(p, s);
    if (tile == STAGED_128) return staged<E, OP, 128, 128, 64, 64, 2>(p, s);
  }
  if (tile == TILE_128) return direct<E, OP, 128, 128, 64, 64, 1, 2>(p, s);
  if (tile == TILE_64_128) return direct<E, OP, 64, 128, 32, 64, 1, 3>(p, s);
  if (tile == TILE_64) return direct<E, OP, 64, 64, 32, 32, 1, 5>(p, s);
  if (tile == TILE_64_PARTS) return direct<E, OP, 64, 64, 32, 32, 4, 1>(p, s);
  return staged<E, OP, 64, 64, 32, 32, 3>(p, s);
}
template <typename E, int OP>
moe_status product_of(ProductArgs p, hipStream_t s) {
  p.splits = 1;
  const Plan plan = plan_of<E, OP>(p);
  return few_rows_ok<E, OP>(p, plan.time) ? few_rows<E, OP>(p, s) : run_plan<E, OP>(p, plan.tile, s);
}
template <int OP>
moe_status product(int fmt, const ProductArgs& p, hipStream_t s) {
  return fmt == MOE_AFMT_BF16 ? product_of<uint16_t, OP>(p, s) : product_of<float, OP>(p, s);
}

template <typename E, int OP>
moe_status gradient(const ProductArgs& p, const Plan& plan, float* part, hipStream_t s) {
  const moe_status st = run_plan<E, OP>(split<OP>(p, plan.splits, part), plan.tile, s);
  return st == MOE_OK ? join<OP>(p, plan.splits, part, s) : st;
}
template <typename E, int B, int WAVES, bool STAGED>
moe_status pair(ProductArgs dx, ProductArgs dw, hipStream_t s) {
  dx.tiles = (uint32_t)tiles_of<OP_DX>(dx, B, B);
  const int64_t a = blocks_of<OP_DX>(dx, B, B), b = blocks_of<OP_DW>(dw, B, B), blocks = a * dx.splits + b * dw.splits;
  return launch(gradients_kernel<E, B, B, B / 2, B / 2, WAVES, STAGED>, dim3((unsigned)blocks), dim3(256), s, dx, (uint32_t)a, dw, (uint32_t)b);
}
// Both gradients, in one launch where that is estimated to be faster: all workgroups' stages over the CUs' rounds,
// not less than the longest tile alone.  (Of many tiles the launch is no matter, and they stay apart.)
constexpr float kLaunchUs = 2.f, kPairTiles = 1 << 16;
template <typename E>
moe_status both(const ProductArgs& dx, const ProductArgs& dw, float* part, float* part_dw, hipStream_t s) {
  const Plan a = plan_of<E, OP_DX>(dx), b = plan_of<E, OP_DW>(dw);
  if (a.straight == b.straight) {
    float least = a.time + b.time + kLaunchUs;
    int best = -1;
    for (const int i : {TILE_64, TILE_128, STAGED_64}) {
      if ((i == STAGED_64) == a.straight || (i == TILE_128 && (a.splits > 1 || b.splits > 1))) continue;
      const TileCost &ca = costs_of<E, OP_DX>()[i], &cb = costs_of<E, OP_DW>()[i];
      const float ta = a.splits * tiles_like<OP_DX>(dx, ca.bm, ca.bn), tb = b.splits * tiles_like<OP_DW>(dw, cb.bm, cb.bn);
      if (ta + tb > kPairTiles) continue;
      const float sa = std::ceil(stages_of<E, OP_DX>(dx) / a.splits), sb = std::ceil(stages_of<E, OP_DW>(dw) / b.splits);
      const float work = (ta * sa * ca.shared + tb * sb * cb.shared) / (ta + tb) * std::ceil((ta + tb) / kCus);
      const float time = std::max({work, sa * ca.alone, sb * cb.alone}) + std::ceil((ta + tb) / (kCus * ca.per_cu)) * std::max(ca.fixed, cb.fixed) +
                         ((a.splits > 1) + (b.splits > 1)) * kJoinUs;
      if (time < least) {
        least = time;
        best = i;
      }
    }
    if (best >= 0) {
      const ProductArgs p = split<OP_DX>(dx, a.splits, part), q = split<OP_DW>(dw, b.splits, part_dw);
      moe_status st = best == TILE_64    ? pair<E, 64, 4, false>(p, q, s)
                      : best == TILE_128 ? pair<E, 128, 2, false>(p, q, s)
                                         : pair<E, 64, 1, true>(p, q, s);
      if (st == MOE_OK) st = join<OP_DX>(dx, a.splits, part, s);
      return st == MOE_OK ? join<OP_DW>(dw, b.splits, part_dw, s) : st;
    }
  }
  const moe_status st = gradient<E, OP_DX>(dx, a, part, s);
  return st == MOE_OK ? gradient<E, OP_DW>(dw, b, part_dw, s) : st;
}
template <typename E>
moe_status gradients_of(const ProductArgs& dx, const ProductArgs& dw, float* part, float* part_dw, hipStream_t s) {
  if (dx.out && dw.out) return both<E>(dx, dw, part, part_dw, s);
  return dx.out ? gradient<E, OP_DX>(dx, plan_of<E, OP_DX>(dx), part, s) : gradient<E, OP_DW>(dw, plan_of<E, OP_DW>(dw), part_dw, s);
}
// Whether the launch that its plan asks for is one.
template <typename E, int OP>
bool fits(const ProductArgs& p) {
  if (!p.out) return true;
  const Plan plan = plan_of<E, OP>(p);
  const TileCost& c = costs_of<E, OP>()[plan.tile];
  const int threads = (c.bm * c.bn > 128 * 128 ? 512 : 256) * c.parts;
  return blocks_of<OP>(p, c.bm, c.bn) * threads * plan.splits <= kMaxThreads;
}

// ---------------------------------------------------------------- checks
struct Dims {
  int64_t ld_x, ld_dx, ld_w, gs_w, ld_y, ld_dy, ld_r, ld_z;
  int wrows, zcols;  // rows of an expert's weights; columns of gu or z
};

constexpr int64_t kMaxReach = 1ll << 58;  // elements from a matrix's first row to its end: bytes, and sums of them, stay in 64 bits

int64_t stride_of(int64_t ld, int64_t n, int64_t rows) {
  return ld == 0 ? n : (ld >= n && ld <= std::min(kMaxStride, kMaxReach / rows) ? ld : -1);
}

bool dims_ok(const moe_product_config* c, bool glu, bool offsets, Dims& d) {
  if (!c || c->rows < 1 || c->rows > kProductMaxRows || c->n_experts < 1 || c->n_experts > kMaxExperts) return false;
  if (c->K < 1 || c->K > kProductMaxSize || c->N < 1 || c->N > kProductMaxSize) return false;
  if (!offsets && c->n_experts != 1) return false;
  if (!fmt_ok(c->fmt) || !fmt_ok(c->y_fmt) || !fmt_ok(c->dw_fmt)) return false;
  if (c->act < MOE_ACT_NONE || c->act > MOE_ACT_GELU) return false;
  d.wrows = glu ? 2 * c->N : c->N;
  d.zcols = d.wrows;
  d.ld_x = stride_of(c->ld_x, c->K, c->rows);
  d.ld_dx = stride_of(c->ld_dx, c->K, c->rows);
  d.ld_w = stride_of(c->ld_w, c->K, d.wrows);
  if (d.ld_w < 0) return false;
  const int64_t dense = (int64_t)d.wrows * d.ld_w;
  d.gs_w = c->gs_w == 0 ? dense : c->gs_w;
  d.ld_y = stride_of(c->ld_y, c->N, c->rows);
  d.ld_r = stride_of(c->ld_residual, c->N, c->rows);
  d.ld_z = stride_of(c->ld_z, d.zcols, c->rows);
  if (d.ld_x < 0 || d.ld_dx < 0 || d.ld_y < 0 || d.ld_r < 0 || d.ld_z < 0) return false;
  // experts' weights lie apart, and the last one's end is an address of 2^46 elements at most
  return d.gs_w >= (int64_t)(d.wrows - 1) * d.ld_w + c->K && d.gs_w <= kMaxStride;
}

Span matrix(const void* p, int64_t rows, int64_t n, int fmt, int64_t ld) {
  return {p, rows, n * fmt_bytes(fmt), ld * fmt_bytes(fmt)};
}
// The experts' weights: one block where their rows are evenly spaced, else from the first to the last.
Span weights(const void* w, const moe_product_config* c, const Dims& d) {
  if (c->n_experts == 1 || d.gs_w == (int64_t)d.wrows * d.ld_w)
    return matrix(w, (int64_t)c->n_experts * d.wrows, c->K, c->fmt, d.ld_w);
  return flat(w, ((int64_t)(c->n_experts - 1) * d.gs_w + (int64_t)(d.wrows - 1) * d.ld_w + c->K) * fmt_bytes(c->fmt));
}

template <size_t I, size_t O>
bool apart(const Span (&in)[I], const Span (&out)[O]) {
  for (size_t o = 0; o < O; ++o) {
    for (const Span& i : in)
      if (overlap(out[o], i)) return false;
    for (size_t q = 0; q < o; ++q)
      if (overlap(out[o], out[q])) return false;
  }
  return true;
}

template <typename... P>
bool all_aligned(int64_t to, const P*... p) { return (aligned_to(p, to) && ...); }

int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// The workspace: 15 bytes to reach an alignment of 16, d, the bias's partial sums.
struct Workspace {
  int64_t ld_d, d, bias, part, part_dw, bytes;  // elements; offsets and size in bytes
};
// Elements of fp32 sums that splits of the k leave, at most, for these rows or fewer: splits_for's tiles times splits,
// 64 x 64 outputs each, are no more than the CUs.  (What these rows need alone may be less: enough of them are not split.)
template <int OP>
int64_t partials(int fmt, const ProductArgs& p) {
  const float stages = fmt == MOE_AFMT_BF16 ? stages_of<uint16_t, OP>(p) : stages_of<float, OP>(p);
  const int splits = splits_for(1.f, stages);
  const int64_t plane = (OP == OP_DW ? (int64_t)p.E * p.M : p.rows) * p.N;
  return splits > 1 ? std::min<int64_t>(plane * splits, kCus * 64 * 64) : 0;
}
// (k: columns of x; n: of d, 2 N for the gated block; bias_n: of the bias or 0)
Workspace workspace_of(int64_t rows, int E, int64_t k, int64_t n, int64_t bias_n, int fmt) {
  Workspace w;
  ProductArgs dx{}, dw{};
  dx.rows = dw.rows = (int)rows;
  dx.E = dw.E = E;
  dx.K = dw.M = (int)n;
  dx.N = dw.N = (int)k;
  w.ld_d = up(n, 8);
  w.d = 0;
  w.bias = up(rows * w.ld_d * fmt_bytes(fmt), 16);
  const int splits = bias_splits(rows, E, std::max<int64_t>(bias_n, 1));
  w.part = up(w.bias + (bias_n && splits > 1 ? 4 * (int64_t)splits * E * bias_n : 0), 16);
  w.part_dw = up(w.part + 4 * partials<OP_DX>(fmt, dx), 16);
  w.bytes = 15 + w.part_dw + 4 * partials<OP_DW>(fmt, dw);
  return w;
}
// Of a bias's gradient alone, which has no product: its partial sums.
Workspace bias_workspace(int64_t rows, int E, int64_t n) {
  Workspace w{};
  const int splits = bias_splits(rows, E, n);
  w.bytes = 15 + (splits > 1 ? 4 * (int64_t)splits * E * n : 0);
  return w;
}
bool sizes_ok(int32_t rows, int32_t E, int32_t K, int32_t N, int32_t fmt) {
  return rows >= 1 && rows <= kProductMaxRows && E >= 1 && E <= kMaxExperts && K >= 1 && K <= kProductMaxSize && N >= 1 &&
         N <= kProductMaxSize && fmt_ok(fmt);
}
uint8_t* base_of(void* ws) { return reinterpret_cast<uint8_t*>(((uintptr_t)ws + 15) & ~(uintptr_t)15); }

// dx = d W and dW = d^T x, each where it is asked for.
struct Gradients {
  ProductArgs dx, dw;
  float *part, *part_dw;
  int fmt;
  bool fit() const {
    return fmt == MOE_AFMT_BF16 ? fits<uint16_t, OP_DX>(dx) && fits<uint16_t, OP_DW>(dw) : fits<float, OP_DX>(dx) && fits<float, OP_DW>(dw);
  }
  moe_status run(hipStream_t s) const {
    return fmt == MOE_AFMT_BF16 ? gradients_of<uint16_t>(dx, dw, part, part_dw, s) : gradients_of<float>(dx, dw, part, part_dw, s);
  }
};
Gradients gradients(const moe_product_config* c, const Dims& d, const void* dz, int64_t ld_dz, bool padded, const void* x, const void* w,
                    const int32_t* offsets, void* dx, void* dw, uint8_t* ws, const Workspace& k) {
  ProductArgs p{};
  p.a = dz;
  p.lda = ld_dz;
  p.padded = padded;
  p.offsets = offsets;
  p.rows = c->rows;
  p.E = c->n_experts;
  p.N = c->K;
  p.splits = 1;
  ProductArgs q = p;
  p.b = w;
  p.ldb = d.ld_w;
  p.gsb = d.gs_w;
  p.K = d.wrows;
  p.out = dx;
  p.ldo = d.ld_dx;
  p.out_fmt = c->fmt;
  q.b = x;
  q.ldb = d.ld_x;
  q.M = d.wrows;
  q.out = dw;
  q.out_fmt = c->dw_fmt;
  return {p, q, reinterpret_cast<float*>(ws + k.part), reinterpret_cast<float*>(ws + k.part_dw), c->fmt};
}

template <bool GLU>
moe_status pre_gradient(const moe_product_config* c, const Dims& d, const void* dy, int dy_fmt, const void* z,
                        const int32_t* offsets, void* out, int64_t ld_d, hipStream_t s) {
  const int across = (c->N + 511) / 512;
  const dim3 grid((unsigned)std::min((c->rows + 3) / 4, (1 << 22) / across), (unsigned)across);
  return launch(pre_gradient_kernel<GLU>, grid, dim3(256), s, dy, dy_fmt, d.ld_y, z, c->fmt, d.ld_z, offsets, c->rows,
                c->n_experts, c->N, c->act, out, ld_d);
}

}  // namespace
}  // namespace rmoe

using namespace rmoe;

extern "C" MOE_API moe_status moe_glu(const moe_product_config* cfg, const void* x, const void* w, const int32_t* offsets,
                                      void* a, void* gu, moe_stream_t stream) {
  Dims d;
  if (!x || !w || !a || !dims_ok(cfg, true, offsets, d)) return MOE_EINVAL;
  const int64_t eb = fmt_bytes(cfg->fmt), R = cfg->rows;
  if (!all_aligned(eb, x, w, a, gu) || !aligned_to(offsets, 4)) return MOE_EINVAL;
  const Span in[3] = {matrix(x, R, cfg->K, cfg->fmt, d.ld_x), weights(w, cfg, d), flat(offsets, 4 * (cfg->n_experts + 1ll))};
  const Span out[2] = {matrix(a, R, cfg->N, cfg->fmt, d.ld_y), matrix(gu, R, d.zcols, cfg->fmt, d.ld_z)};
  if (!apart(in, out)) return MOE_EINVAL;
  ProductArgs p{};
  p.a = x;
  p.lda = d.ld_x;
  p.b = w;
  p.ldb = d.ld_w;
  p.gsb = d.gs_w;
  p.offsets = offsets;
  p.rows = cfg->rows;
  p.E = cfg->n_experts;
  p.K = cfg->K;
  p.N = cfg->N;
  p.act = cfg->act;
  p.out = a;
  p.ldo = d.ld_y;
  p.out_fmt = cfg->fmt;
  p.aux = gu;
  p.ld_aux = d.ld_z;
  const hipStream_t s = stream_of(stream);
  const StreamDevice on(s);
  return product<OP_GLU>(cfg->fmt, p, s);
}

extern "C" MOE_API int64_t moe_glu_workspace(int32_t rows, int32_t n_experts, int32_t H, int32_t I, int32_t fmt) {
  if (!sizes_ok(rows, n_experts, H, I, fmt)) return -1;
  return workspace_of(rows, n_experts, H, 2ll * I, 0, fmt).bytes;
}

extern "C" MOE_API moe_status moe_glu_backward(const moe_product_config* cfg, const void* da, const void* gu, const void* x,
                                               const void* w, const int32_t* offsets, void* dx, void* dw, void* ws,
                                               size_t ws_bytes, moe_stream_t stream) {
  Dims d;
  if (!da || !gu || (!dx && !dw) || (dx && !w) || (dw && !x) || !ws || !dims_ok(cfg, true, offsets, d)) return MOE_EINVAL;
  const int64_t eb = fmt_bytes(cfg->fmt), R = cfg->rows;
  const Workspace k = workspace_of(R, cfg->n_experts, cfg->K, 2ll * cfg->N, 0, cfg->fmt);
  if (ws_bytes < (size_t)k.bytes) return MOE_EINVAL;
  if (!all_aligned(eb, da, gu, dx ? w : nullptr, dw ? x : nullptr, dx) || !aligned_to(dw, fmt_bytes(cfg->dw_fmt)) ||
      !aligned_to(offsets, 4))
    return MOE_EINVAL;
  const Span none = flat(nullptr, 0);
  const Span in[5] = {matrix(da, R, cfg->N, cfg->fmt, d.ld_y), matrix(gu, R, d.zcols, cfg->fmt, d.ld_z),
                      dw ? matrix(x, R, cfg->K, cfg->fmt, d.ld_x) : none, dx ? weights(w, cfg, d) : none,
                      flat(offsets, 4 * (cfg->n_experts + 1ll))};
  const Span out[3] = {matrix(dx, R, cfg->K, cfg->fmt, d.ld_dx),
                       flat(dw, (int64_t)cfg->n_experts * d.wrows * cfg->K * fmt_bytes(cfg->dw_fmt)), flat(ws, k.bytes)};
  if (!apart(in, out)) return MOE_EINVAL;
  const hipStream_t s = stream_of(stream);
  const StreamDevice on(s);
  uint8_t* const base = base_of(ws);
  void* const dgu = base + k.d;
  const Gradients g = gradients(cfg, d, dgu, k.ld_d, true, x, w, offsets, dx, dw, base, k);
  if (!g.fit()) return MOE_EINVAL;
  const moe_status st = pre_gradient<true>(cfg, d, da, cfg->fmt, gu, offsets, dgu, k.ld_d, s);
  return st == MOE_OK ? g.run(s) : st;
}

extern "C" MOE_API moe_status moe_linear(const moe_product_config* cfg, const void* x, const void* w, const float* bias,
                                         const void* residual, const int32_t* offsets, void* y, void* z,
                                         moe_stream_t stream) {
  Dims d;
  if (!x || !w || !y || !dims_ok(cfg, false, offsets, d)) return MOE_EINVAL;
  const int64_t eb = fmt_bytes(cfg->fmt), yb = fmt_bytes(cfg->y_fmt), R = cfg->rows;
  if (!all_aligned(eb, x, w, z) || !all_aligned(yb, y, residual) || !all_aligned(4, offsets, bias)) return MOE_EINVAL;
  const Span none = flat(nullptr, 0);
  // (y may take the residual's place: each element is read by the lane that writes it)
  const bool in_place = residual == y && d.ld_r == d.ld_y;
  const Span in[5] = {matrix(x, R, cfg->K, cfg->fmt, d.ld_x), weights(w, cfg, d), flat(offsets, 4 * (cfg->n_experts + 1ll)),
                      flat(bias, 4ll * cfg->n_experts * cfg->N),
                      in_place ? none : matrix(residual, R, cfg->N, cfg->y_fmt, d.ld_r)};
  const Span out[2] = {matrix(y, R, cfg->N, cfg->y_fmt, d.ld_y), matrix(z, R, cfg->N, cfg->fmt, d.ld_z)};
  if (!apart(in, out)) return MOE_EINVAL;
  ProductArgs p{};
  p.a = x;
  p.lda = d.ld_x;
  p.b = w;
  p.ldb = d.ld_w;
  p.gsb = d.gs_w;
  p.offsets = offsets;
  p.rows = cfg->rows;
  p.E = cfg->n_experts;
  p.K = cfg->K;
  p.N = cfg->N;
  p.act = cfg->act;
  p.out = y;
  p.ldo = d.ld_y;
  p.out_fmt = cfg->y_fmt;
  p.aux = z;
  p.ld_aux = d.ld_z;
  p.residual = residual;
  p.ld_res = d.ld_r;
  p.bias = bias;
  const hipStream_t s = stream_of(stream);
  const StreamDevice on(s);
  return product<OP_LINEAR>(cfg->fmt, p, s);
}

extern "C" MOE_API int64_t moe_linear_workspace(int32_t rows, int32_t n_experts, int32_t K, int32_t N, int32_t fmt) {
  if (!sizes_ok(rows, n_experts, K, N, fmt)) return -1;
  return workspace_of(rows, n_experts, K, N, N, fmt).bytes;
}

extern "C" MOE_API moe_status moe_linear_backward(const moe_product_config* cfg, const void* dy, const void* z, const void* x,
                                                  const void* w, const int32_t* offsets, void* dx, void* dw, float* dbias,
                                                  void* ws, size_t ws_bytes, moe_stream_t stream) {
  Dims d;
  if (!dy || (!dx && !dw && !dbias) || (dx && !w) || (dw && !x) || !ws || !dims_ok(cfg, false, offsets, d)) return MOE_EINVAL;
  if (cfg->act != MOE_ACT_NONE && !z) return MOE_EINVAL;
  const int64_t eb = fmt_bytes(cfg->fmt), R = cfg->rows;
  const bool products = dx || dw;
  const Workspace k = products ? workspace_of(R, cfg->n_experts, cfg->K, cfg->N, cfg->N, cfg->fmt) : bias_workspace(R, cfg->n_experts, cfg->N);
  if (ws_bytes < (size_t)k.bytes) return MOE_EINVAL;
  const bool zs = cfg->act != MOE_ACT_NONE;
  if (!all_aligned(eb, zs ? z : nullptr, dx ? w : nullptr, dw ? x : nullptr, dx) || !aligned_to(dy, fmt_bytes(cfg->y_fmt)) ||
      !aligned_to(dw, fmt_bytes(cfg->dw_fmt)) || !all_aligned(4, offsets, dbias))
    return MOE_EINVAL;
  const Span none = flat(nullptr, 0);
  const Span in[5] = {matrix(dy, R, cfg->N, cfg->y_fmt, d.ld_y), zs ? matrix(z, R, cfg->N, cfg->fmt, d.ld_z) : none,
                      dw ? matrix(x, R, cfg->K, cfg->fmt, d.ld_x) : none, dx ? weights(w, cfg, d) : none,
                      flat(offsets, 4 * (cfg->n_experts + 1ll))};
  const Span out[4] = {matrix(dx, R, cfg->K, cfg->fmt, d.ld_dx),
                       flat(dw, (int64_t)cfg->n_experts * cfg->N * cfg->K * fmt_bytes(cfg->dw_fmt)),
                       flat(dbias, 4ll * cfg->n_experts * cfg->N), flat(ws, k.bytes)};
  if (!apart(in, out)) return MOE_EINVAL;
  const hipStream_t s = stream_of(stream);
  const StreamDevice on(s);
  uint8_t* const base = base_of(ws);
  moe_status st = MOE_OK;
  // dy itself where nothing changes it and its rows start on 16 bytes, else dz in the operands' type
  const bool as_is = !zs && cfg->y_fmt == cfg->fmt && aligned_to(dy, 16) && (d.ld_y * eb | cfg->N * eb) % 16 == 0;
  void* const dz = products && !as_is ? base + k.d : nullptr;
  const Gradients g = as_is ? gradients(cfg, d, dy, d.ld_y, false, x, w, offsets, dx, dw, base, k)
                            : gradients(cfg, d, dz, k.ld_d, true, x, w, offsets, dx, dw, base, k);
  if (!g.fit()) return MOE_EINVAL;
  if (dbias) {
    const int splits = bias_splits(R, cfg->n_experts, cfg->N);
    float* const part = splits > 1 ? reinterpret_cast<float*>(base + k.bias) : dbias;
    st = launch(bias_gradient_kernel, dim3((cfg->N + 63) / 64, cfg->n_experts, splits), dim3(256), s, dy, cfg->y_fmt, d.ld_y,
                z, cfg->fmt, d.ld_z, offsets, cfg->rows, cfg->n_experts, cfg->N, cfg->act, splits, part, dz, k.ld_d);
    if (st == MOE_OK && splits > 1) {
      const int64_t total = (int64_t)cfg->n_experts * cfg->N;
      st = launch(bias_join_kernel, dim3((unsigned)((total + 255) / 256)), dim3(256), s, part, total, splits, dbias);
    }
  } else if (dz) {
    st = pre_gradient<false>(cfg, d, dy, cfg->y_fmt, z, offsets, dz, k.ld_d, s);
  }
  return st == MOE_OK && products ? g.run(s) : st;
}
