// Tokens sorted by expert, moved, and brought back with their gates; their gradients; the
// gradient of the gates.  The library's own prefill gathers rows inside its GEMMs; these
// are the same steps on their own, for experts that run outside it and for training.
//
// With pairs p = t*k + j (token t, rank j) and expert ids e_p, a pair is kept when
// 0 <= e_p < E.  perm lists the kept pairs stably by (e_p, p), inv is its inverse (-1 for a
// pair left out), and every move reads inv: a token finds its own k rows, so a row of x or
// dy is read once for its k uses, sums over a token run in rank order in registers, and
// nothing is added by atomics (results do not depend on the order of workgroups).
#include <algorithm>

#include "rows.hpp"

namespace rmoe {

constexpr int kMoveMaxH = 1 << 16;       // elements of a row
constexpr int kMoveMaxT = 1 << 22;       // tokens
constexpr int kMoveMaxK = 1024;          // ranks
constexpr int64_t kMoveMaxPairs = 1 << 26;

// ---------------------------------------------------------------------------
// The sort: a counting sort in two launches over at most kSortBlocks chunks of pairs (their
// number, not their size, is bounded, so a chunk's base stays a sum over at most that many
// histogram rows however long the prompt).
constexpr int kSortBlocks = 256;
constexpr int kSortThreads = 256;

struct SortPlan {
  int chunk, blocks;  // pairs per workgroup (a multiple of kSortThreads) and workgroups
};
inline SortPlan sort_plan(int64_t P) {
  const int64_t per = (P + kSortBlocks - 1) / kSortBlocks;
  const int chunk = (int)((per + kSortThreads - 1) / kSortThreads * kSortThreads);
  return {chunk, (int)((P + chunk - 1) / chunk)};
}

__global__ __launch_bounds__(kSortThreads) void dispatch_count(const int32_t* __restrict__ idx, int P, int E, int chunk,
                                                               int32_t* __restrict__ hist) {
  __shared__ int s_n[kMaxExperts];
  for (int e = threadIdx.x; e < E; e += kSortThreads) s_n[e] = 0;
  __syncthreads();
  const int lo = blockIdx.x * chunk, hi = min(lo + chunk, P);
  for (int p = lo + threadIdx.x; p < hi; p += kSortThreads) {
    const int e = idx[p];
    if ((unsigned)e < (unsigned)E) atomicAdd(&s_n[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kSortThreads) hist[(size_t)blockIdx.x * E + e] = s_n[e];
}

// Lanes of the wavefront whose key equals this lane's (key < 2^bits; the inactive pass
// valid = false and get 0).
__device__ __forceinline__ uint64_t wave_peers(int key, bool valid, int bits) {
  uint64_t m = __ballot(valid);
  for (int b = 0; b < bits; ++b) {
    const uint64_t set = __ballot((key >> b) & 1);
    m &= ((key >> b) & 1) ? set : ~set;
  }
  return valid ? m : 0;
}

__global__ __launch_bounds__(kSortThreads) void dispatch_place(const int32_t* __restrict__ idx, int P, int E, int bits,
                                                               int chunk, const int32_t* __restrict__ hist,
                                                               int32_t* __restrict__ perm, int32_t* __restrict__ inv,
                                                               int32_t* __restrict__ offsets) {
  __shared__ int s_base[kMaxExperts];
  __shared__ int s_wave[kSortThreads / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int nblk = gridDim.x, blk = blockIdx.x;
  // an expert's first position in this chunk: kept pairs of lower experts, then its own
  // pairs in earlier chunks
  int carry = 0;
  for (int e0 = 0; e0 < E; e0 += kSortThreads) {
    const int e = e0 + tid;
    int total = 0, before = 0;
    if (e < E) {
#pragma unroll 8
      for (int c = 0; c < nblk; ++c) {
        const int v = hist[(size_t)c * E + e];
        total += v;
        before += c < blk ? v : 0;
      }
    }
    int x = total;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int y = __shfl_up(x, off);
      if (lane >= off) x += y;
    }
    if (lane == 63) s_wave[wave] = x;
    __syncthreads();
    int base = carry;
    for (int w = 0; w < kSortThreads / 64; ++w) {
      if (w < wave) base += s_wave[w];
      carry += s_wave[w];
    }
    base += x - total;
    if (e < E) {
      s_base[e] = base + before;
      if (blk == 0) offsets[e] = base;
    }
    __syncthreads();
  }
  if (blk == 0 && tid == 0) offsets[E] = carry;
  // the chunk's pairs in order, 256 at a time, wavefront after wavefront
  const int lo = blk * chunk, hi = min(lo + chunk, P);
  for (int r0 = lo; r0 < hi; r0 += kSortThreads) {
    const int p = r0 + tid;
    const int e = p < hi ? idx[p] : -1;
    const bool kept = (unsigned)e < (unsigned)E;
    const uint64_t peers = wave_peers(e, kept, bits);
    const int rank = __popcll(peers & ((1ull << lane) - 1));
    for (int w = 0; w < kSortThreads / 64; ++w) {
      if (w == wave) {
        const int pos = kept ? s_base[e] + rank : -1;
        __builtin_amdgcn_wave_barrier();  // every lane has read the base before its first peer moves it
        if (kept && rank == 0) s_base[e] = pos + __popcll(peers);
        if (kept) perm[pos] = p;
        if (p < hi) inv[p] = pos;
      }
      __syncthreads();
    }
  }
}

// ---------------------------------------------------------------------------
// Rows of x to their sorted places: a wavefront takes one token and one segment of its row
// (4 KB), reads it once and writes it k times.
constexpr int kSegLoads = 4;  // 16-byte loads per lane and segment

template <int EB>  // bytes of an element
__global__ __launch_bounds__(256) void dispatch_move(const uint8_t* __restrict__ x, int64_t pitch, int T, int k, int H,
                                                     const int32_t* __restrict__ inv, uint8_t* __restrict__ xs) {
  constexpr int FMT = EB == 2 ? MOE_AFMT_BF16 : MOE_AFMT_F32, N = 16 / EB;
  const int t = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (t >= T) return;
  const int c0 = blockIdx.y * kSegLoads * 64 + lane;  // chunk of the lane's first load
  const uint8_t* row = x + (int64_t)t * pitch;
  Chunk<FMT, N> q[kSegLoads];
#pragma unroll
  for (int u = 0; u < kSegLoads; ++u) {
    const int i = (c0 + 64 * u) * N;
    if (i < H) q[u].load(row + (int64_t)i * EB, H - i);
  }
  const int64_t P = (int64_t)T * k;
  for (int j = 0; j < k; ++j) {
    const int pos = inv[(int64_t)t * k + j];
    if ((unsigned)pos >= (uint64_t)P) continue;
    uint8_t* dst = xs + (int64_t)pos * H * EB;
#pragma unroll
    for (int u = 0; u < kSegLoads; ++u) {
      const int i = (c0 + 64 * u) * N;
      if (i < H) q[u].store(dst + (int64_t)i * EB, H - i);
    }
  }
}

// ---------------------------------------------------------------------------
// y[t] = sum_j w[t,j] rows[inv[t,j]] in rank order (w = nullptr: a plain sum, the gradient
// of the move).  A wavefront takes one token and 64 chunks of its row; kRanks rows are in
// flight per lane.
constexpr int kRanks = 8;

template <int RF, int YF, bool WEIGHTED>
__global__ __launch_bounds__(256) void combine_rows(const uint8_t* __restrict__ rows, const int32_t* __restrict__ inv,
                                                    const float* __restrict__ w, int T, int k, int H,
                                                    uint8_t* __restrict__ y, int64_t pitch) {
  constexpr int N = 8, RB = kElemBytes<RF>, YB = kElemBytes<YF>;
  const int t = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (t >= T) return;
  const int i = (blockIdx.y * 64 + lane) * N;
  if (i >= H) return;
  const int64_t P = (int64_t)T * k, p0 = (int64_t)t * k;
  float acc[N];
#pragma unroll
  for (int n = 0; n < N; ++n) acc[n] = 0.f;
  for (int j0 = 0; j0 < k; j0 += kRanks) {
    Chunk<RF, N> q[kRanks];
    float g[kRanks];
    bool kept[kRanks];
#pragma unroll
    for (int j = 0; j < kRanks; ++j) {
      const int pos = j0 + j < k ? inv[p0 + j0 + j] : -1;
      kept[j] = (unsigned)pos < (uint64_t)P;
      g[j] = 1.f;
      if (kept[j]) {
        if (WEIGHTED) g[j] = w[p0 + j0 + j];
        q[j].load(rows + ((int64_t)pos * H + i) * RB, H - i);
      }
    }
#pragma unroll
    for (int j = 0; j < kRanks; ++j)
      if (kept[j]) {
#pragma unroll
        for (int n = 0; n < N; ++n) acc[n] = WEIGHTED ? fmaf(g[j], q[j].get(n), acc[n]) : acc[n] + q[j].get(n);
      }
  }
  Chunk<YF, N> o;
  o.set(acc);
  o.store(y + (int64_t)t * pitch + (int64_t)i * YB, H - i);
}

// ---------------------------------------------------------------------------
// The weighted return's gradient: dys[inv[t,j]] = w[t,j] dy[t], dw[t,j] = <dy[t], ys[inv[t,j]]>.
// A workgroup takes one token and up to kRanks of its ranks, its wavefronts neighbouring
// pieces of the row; the dot products meet in LDS in wavefront order.
constexpr int kCbWaves = 4;

template <int DF, int RF>
__global__ __launch_bounds__(64 * kCbWaves) void combine_rows_backward(const uint8_t* __restrict__ dy, int64_t pitch,
                                                                       const uint8_t* ys,
                                                                       const int32_t* __restrict__ inv,
                                                                       const float* __restrict__ w, int T, int k, int H,
                                                                       uint8_t* dys, float* __restrict__ dw) {
  constexpr int N = 8, DB = kElemBytes<DF>, RB = kElemBytes<RF>;
  __shared__ float s_dot[kCbWaves][kRanks];
  const int t = blockIdx.x, j0 = blockIdx.y * kRanks, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t P = (int64_t)T * k, p0 = (int64_t)t * k + j0;
  int pos[kRanks];
  float g[kRanks], dot[kRanks];
#pragma unroll
  for (int j = 0; j < kRanks; ++j) {
    pos[j] = j0 + j < k ? inv[p0 + j] : -1;
    if ((unsigned)pos[j] >= (uint64_t)P) pos[j] = -1;
    g[j] = pos[j] >= 0 && dys ? w[p0 + j] : 0.f;
    dot[j] = 0.f;
  }
  for (int i = threadIdx.x * N; i < H; i += 64 * kCbWaves * N) {
    Chunk<DF, N> d;
    Chunk<RF, N> q[kRanks];
    d.load(dy + (int64_t)t * pitch + (int64_t)i * DB, H - i);
    if (dw) {
#pragma unroll
      for (int j = 0; j < kRanks; ++j)
        if (pos[j] >= 0) q[j].load(ys + ((int64_t)pos[j] * H + i) * RB, H - i);
#pragma unroll
      for (int j = 0; j < kRanks; ++j)
        if (pos[j] >= 0) {
#pragma unroll
          for (int n = 0; n < N; ++n) dot[j] = fmaf(d.get(n), q[j].get(n), dot[j]);
        }
    }
    if (dys) {
#pragma unroll
      for (int j = 0; j < kRanks; ++j)
        if (pos[j] >= 0) {
          float v[N];
#pragma unroll
          for (int n = 0; n < N; ++n) v[n] = g[j] * d.get(n);
          q[j].set(v);
          q[j].store(dys + ((int64_t)pos[j] * H + i) * RB, H - i);
        }
    }
  }
  if (!dw) return;
#pragma unroll
  for (int j = 0; j < kRanks; ++j) {
    const float v = wave_sum(dot[j]);
    if (lane == 0) s_dot[wave][j] = v;
  }
  __syncthreads();
  if (threadIdx.x < kRanks && j0 + threadIdx.x < k) {
    float v = 0.f;
#pragma unroll
    for (int x = 0; x < kCbWaves; ++x) v += s_dot[x][threadIdx.x];
    dw[p0 + threadIdx.x] = v;
  }
}

// ---------------------------------------------------------------------------
// The gradient of the gates: one wavefront per token, E / 64 logits per lane.  A token's
// logits are all read before any of its gradients is written (dlogits may be logits).
template <int PL>
__global__ __launch_bounds__(256) void topk_backward_kernel(const float* logits, int T, int E, int k,
                                                            const int32_t* __restrict__ idx,
                                                            const float* __restrict__ dw, int renorm,
                                                            float* dlogits) {
  const int t = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (t >= T) return;
  const float* z = logits + (int64_t)t * E;
  const int32_t* id = idx + (int64_t)t * k;
  const float* dg = dw + (int64_t)t * k;
  // per logit: how often it was chosen and the gates' gradients that fell on it
  float v[PL], n[PL], d[PL];
  float mx = -INFINITY;
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const int e = lane + 64 * i;
    v[i] = e < E ? z[e] : -INFINITY;
    n[i] = 0.f;
    d[i] = 0.f;
  }
  for (int j = 0; j < k; ++j) {
    const int e = id[j];
    if ((unsigned)e >= (unsigned)E) continue;
    const float g = dg[j];
#pragma unroll
    for (int i = 0; i < PL; ++i)
      if (e == lane + 64 * i) {
        n[i] += 1.f;
        d[i] += g;
      }
  }
  // the softmax runs over all experts, or over the chosen ones (each as often as it was)
#pragma unroll
  for (int i = 0; i < PL; ++i) mx = fmaxf(mx, !renorm || n[i] > 0.f ? v[i] : -INFINITY);
  mx = wave_max(mx);
  float sum = 0.f, mean = 0.f;
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const bool in = lane + 64 * i < E && (!renorm || n[i] > 0.f);
    // a masked logit (-inf) has no share, also where every logit is masked
    v[i] = in && v[i] != -INFINITY ? __expf(v[i] - mx) : 0.f;
    sum += renorm ? n[i] * v[i] : v[i];
    mean += d[i] * v[i];
  }
  sum = wave_sum(sum);
  mean = wave_sum(mean);
  const float r = sum == 0.f ? 0.f : 1.f / sum;
  mean *= r;
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const int e = lane + 64 * i;
    if (e < E) dlogits[(int64_t)t * E + e] = v[i] * r * (d[i] - (renorm ? n[i] * mean : mean));
  }
}

namespace {

bool move_shape_ok(int32_t T, int32_t k, int32_t H) {
  return T >= 1 && T <= kMoveMaxT && k >= 1 && k <= kMoveMaxK && (int64_t)T * k <= kMoveMaxPairs && H >= 1 &&
         H <= kMoveMaxH;
}

// A caller's row stride in elements (0: dense rows), or -1.
int64_t row_stride(int64_t ld, int32_t H) { return ld == 0 ? H : (ld >= H && ld <= (1ll << 40) ? ld : -1); }

Span rows_of(const void* p, int64_t rows, int32_t H, int fmt, int64_t ld) {
  return {p, rows, H * fmt_bytes(fmt), ld * fmt_bytes(fmt)};
}

template <bool WEIGHTED>
moe_status run_combine(const void* rows, int fmt, const int32_t* inv, const float* w, int T, int k, int H, void* y,
                       int y_fmt, int64_t ld, hipStream_t s) {
  const dim3 grid((T + 3) / 4, (H + 64 * 8 - 1) / (64 * 8)), block(256);
  const uint8_t* r = static_cast<const uint8_t*>(rows);
  uint8_t* o = static_cast<uint8_t*>(y);
  const int64_t pitch = ld * fmt_bytes(y_fmt);
  constexpr int B = MOE_AFMT_BF16, F = MOE_AFMT_F32;
  if (fmt == B && y_fmt == B) return launch(combine_rows<B, B, WEIGHTED>, grid, block, s, r, inv, w, T, k, H, o, pitch);
  if (fmt == B) return launch(combine_rows<B, F, WEIGHTED>, grid, block, s, r, inv, w, T, k, H, o, pitch);
  if (y_fmt == B) return launch(combine_rows<F, B, WEIGHTED>, grid, block, s, r, inv, w, T, k, H, o, pitch);
  return launch(combine_rows<F, F, WEIGHTED>, grid, block, s, r, inv, w, T, k, H, o, pitch);
}

}  // namespace
}  // namespace rmoe

using namespace rmoe;

extern "C" MOE_API int64_t moe_dispatch_workspace(int32_t T, int32_t k, int32_t n_experts) {
  if (!move_shape_ok(T, k, 1) || n_experts < 1 || n_experts > kMaxExperts) return -1;
  return (int64_t)sort_plan((int64_t)T * k).blocks * n_experts * 4;
}

extern "C" MOE_API moe_status moe_dispatch(const int32_t* topk_idx, int32_t T, int32_t k, int32_t n_experts,
                                           const void* x, int32_t fmt, int32_t H, int64_t ld_x, void* xs,
                                           int32_t* perm, int32_t* inv, int32_t* offsets, void* ws, size_t ws_bytes,
                                           moe_stream_t stream) {
  if (!topk_idx || !perm || !inv || !offsets || (x == nullptr) != (xs == nullptr)) return MOE_EINVAL;
  const int64_t need = moe_dispatch_workspace(T, k, n_experts);
  if (need < 0 || (need > 0 && !ws) || ws_bytes < (size_t)need || !aligned_to(ws, 4)) return MOE_EINVAL;
  const int64_t P = (int64_t)T * k;
  int64_t ld = 0;
  if (x) {
    ld = row_stride(ld_x, H);
    if (!fmt_ok(fmt) || !move_shape_ok(T, k, H) || ld < 0) return MOE_EINVAL;
    if (!aligned_to(x, fmt_bytes(fmt)) || !aligned_to(xs, fmt_bytes(fmt))) return MOE_EINVAL;
  }
  const Span in[2] = {flat(topk_idx, 4 * P), x ? rows_of(x, T, H, fmt, ld) : flat(nullptr, 0)};
  const Span out[5] = {flat(perm, 4 * P), flat(inv, 4 * P), flat(offsets, 4 * ((int64_t)n_experts + 1)),
                       flat(need ? ws : nullptr, need), x ? rows_of(xs, P, H, fmt, H) : flat(nullptr, 0)};
  for (int a = 0; a < 5; ++a) {
    for (const Span& i : in)
      if (overlap(out[a], i)) return MOE_EINVAL;
    for (int b = 0; b < a; ++b)
      if (overlap(out[a], out[b])) return MOE_EINVAL;
  }
  hipStream_t s = static_cast<hipStream_t>(stream);
  const StreamDevice on(s);
  const SortPlan sp = sort_plan(P);
  int bits = 0;
  while ((1 << bits) < n_experts) ++bits;
  int32_t* hist = static_cast<int32_t*>(ws);
  moe_status st = launch(dispatch_count, dim3(sp.blocks), dim3(kSortThreads), s, topk_idx, (int)P, n_experts, sp.chunk, hist);
  if (st == MOE_OK)
    st = launch(dispatch_place, dim3(sp.blocks), dim3(kSortThreads), s, topk_idx, (int)P, n_experts, bits, sp.chunk,
                hist, perm, inv, offsets);
  if (st != MOE_OK || !x) return st;
  const int64_t eb = fmt_bytes(fmt);
  const int seg = kSegLoads * 64 * (int)(16 / eb);
  const dim3 grid((T + 3) / 4, (H + seg - 1) / seg);
  const uint8_t* src = static_cast<const uint8_t*>(x);
  uint8_t* dst = static_cast<uint8_t*>(xs);
  if (eb == 2) return launch(dispatch_move<2>, grid, dim3(256), s, src, ld * eb, T, k, H, inv, dst);
  return launch(dispatch_move<4>, grid, dim3(256), s, src, ld * eb, T, k, H, inv, dst);
}

extern "C" MOE_API moe_status moe_dispatch_backward(const void* dxs, int32_t dxs_fmt, const int32_t* inv, int32_t T,
                                                    int32_t k, int32_t H, void* dx, int32_t dx_fmt, int64_t ld_dx,
                                                    moe_stream_t stream) {
  const int64_t ld = row_stride(ld_dx, H), P = (int64_t)T * k;
  if (!dxs || !inv || !dx || !fmt_ok(dxs_fmt) || !fmt_ok(dx_fmt) || !move_shape_ok(T, k, H) || ld < 0) return MOE_EINVAL;
  if (!aligned_to(dxs, fmt_bytes(dxs_fmt)) || !aligned_to(dx, fmt_bytes(dx_fmt))) return MOE_EINVAL;
  const Span out = rows_of(dx, T, H, dx_fmt, ld);
  if (overlap(out, rows_of(dxs, P, H, dxs_fmt, H)) || overlap(out, flat(inv, 4 * P))) return MOE_EINVAL;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const StreamDevice on(s);
  return run_combine<false>(dxs, dxs_fmt, inv, nullptr, T, k, H, dx, dx_fmt, ld, s);
}

extern "C" MOE_API moe_status moe_combine(const void* ys, int32_t ys_fmt, const int32_t* inv, const float* w, int32_t T,
                                          int32_t k, int32_t H, void* y, int32_t y_fmt, int64_t ld_y,
                                          moe_stream_t stream) {
  const int64_t ld = row_stride(ld_y, H), P = (int64_t)T * k;
  if (!ys || !inv || !w || !y || !fmt_ok(ys_fmt) || !fmt_ok(y_fmt) || !move_shape_ok(T, k, H) || ld < 0)
    return MOE_EINVAL;
  if (!aligned_to(ys, fmt_bytes(ys_fmt)) || !aligned_to(y, fmt_bytes(y_fmt))) return MOE_EINVAL;
  const Span out = rows_of(y, T, H, y_fmt, ld);
  if (overlap(out, rows_of(ys, P, H, ys_fmt, H)) || overlap(out, flat(inv, 4 * P)) || overlap(out, flat(w, 4 * P)))
    return MOE_EINVAL;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const StreamDevice on(s);
  return run_combine<true>(ys, ys_fmt, inv, w, T, k, H, y, y_fmt, ld, s);
}

extern "C" MOE_API moe_status moe_combine_backward(const void* dy, int32_t dy_fmt, int64_t ld_dy, const void* ys,
                                                   int32_t ys_fmt, const int32_t* inv, const float* w, int32_t T,
                                                   int32_t k, int32_t H, void* dys, float* dw, moe_stream_t stream) {
  const int64_t ld = row_stride(ld_dy, H), P = (int64_t)T * k;
  if (!dy || !inv || (!dys && !dw) || (dw && !ys) || (dys && !w)) return MOE_EINVAL;
  if (!fmt_ok(dy_fmt) || !fmt_ok(ys_fmt) || !move_shape_ok(T, k, H) || ld < 0) return MOE_EINVAL;
  if (!aligned_to(dy, fmt_bytes(dy_fmt)) || !aligned_to(ys, fmt_bytes(ys_fmt)) || !aligned_to(dys, fmt_bytes(ys_fmt)))
    return MOE_EINVAL;
  const Span in[4] = {rows_of(dy, T, H, dy_fmt, ld), dys == ys ? flat(nullptr, 0) : rows_of(ys, P, H, ys_fmt, H),
                      flat(inv, 4 * P), flat(w, 4 * P)};
  const Span out[2] = {rows_of(dys, P, H, ys_fmt, H), flat(dw, 4 * P)};
  for (const Span& o : out)
    for (const Span& i : in)
      if (overlap(o, i)) return MOE_EINVAL;
  if (overlap(out[0], out[1])) return MOE_EINVAL;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const StreamDevice on(s);
  const dim3 grid(T, (k + kRanks - 1) / kRanks), block(64 * kCbWaves);
  const uint8_t* d = static_cast<const uint8_t*>(dy);
  const uint8_t* r = static_cast<const uint8_t*>(ys);
  uint8_t* o = static_cast<uint8_t*>(dys);
  const int64_t pitch = ld * fmt_bytes(dy_fmt);
  constexpr int B = MOE_AFMT_BF16, F = MOE_AFMT_F32;
  if (dy_fmt == B && ys_fmt == B)
    return launch(combine_rows_backward<B, B>, grid, block, s, d, pitch, r, inv, w, T, k, H, o, dw);
  if (dy_fmt == B) return launch(combine_rows_backward<B, F>, grid, block, s, d, pitch, r, inv, w, T, k, H, o, dw);
  if (ys_fmt == B) return launch(combine_rows_backward<F, B>, grid, block, s, d, pitch, r, inv, w, T, k, H, o, dw);
  return launch(combine_rows_backward<F, F>, grid, block, s, d, pitch, r, inv, w, T, k, H, o, dw);
}

extern "C" MOE_API moe_status moe_topk_backward(const float* logits, int32_t T, int32_t n_experts,
                                                const int32_t* topk_idx, int32_t k, const float* dw, int32_t renorm,
                                                float* dlogits, moe_stream_t stream) {
  if (!logits || !topk_idx || !dw || !dlogits || !move_shape_ok(T, k, 1)) return MOE_EINVAL;
  if (n_experts < 1 || n_experts > kMaxExperts || (renorm != 0 && renorm != 1)) return MOE_EINVAL;
  const int64_t P = (int64_t)T * k, n = (int64_t)T * n_experts;
  const Span out = flat(dlogits, 4 * n);
  if ((dlogits != logits && overlap(out, flat(logits, 4 * n))) || overlap(out, flat(topk_idx, 4 * P)) ||
      overlap(out, flat(dw, 4 * P)))
    return MOE_EINVAL;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const StreamDevice on(s);
  const dim3 grid((T + 3) / 4), block(256);
  const int E = n_experts;
  if (E <= 256) return launch(topk_backward_kernel<4>, grid, block, s, logits, T, E, k, topk_idx, dw, renorm, dlogits);
  return launch(topk_backward_kernel<16>, grid, block, s, logits, T, E, k, topk_idx, dw, renorm, dlogits);
}
