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
constexpr int kMoveMaxT = 1 << 21;       // tokens
constexpr int kMoveMaxK = 1024;          // ranks
constexpr int64_t kMoveMaxPairs = 1 << 26;

// ---------------------------------------------------------------------------
// The sort: a counting sort, stable by construction (a pair's place is the number of kept
// pairs before it under (expert, pair)).  Three forms by the number of pairs P:
//   P <= kTinyPairs   the kernel that moves the rows counts for itself: every wavefront holds
//                     all keys in registers and a place is one compare and count per 64 pairs
//   P <= kSolePairs   one launch sorts: each workgroup counts all pairs in LDS, those before
//                     its own chunk apart from the others
//   beyond            dispatch_rank leaves each pair's rank within its chunk and one histogram
//                     per chunk, dispatch_scan turns the histograms into first places, and the
//                     move adds the two; the chunks grow with P so that there are at most
//                     kSortChunks of them
// What bounds all three is latency: launches and dependent reads.  E = 256, k = 8, H = 256, kernel
// times and, in brackets, calls in a row:
//    1024 pairs   5.2 us (8.4) in the first form, 4.5 + 3.0 (11.3) in the second
//    8192 pairs   5.2 + 3.7 (10.6) in the second, 3.8 + 3.1 + 4.5 (14.0) in the third
//   16384 pairs   6.2 + 4.9 (11.5) against 3.8 + 3.2 + 5.6 (13.4)
//   32768 pairs   the second's counting alone takes 9.4 us (an LDS atomic of 64 lanes about 32
//                 cycles), the third's two launches 7.4
constexpr int kTinyPairs = 1024;
constexpr int kTinyPieces = 4096;  // and at most this many KB of rows of x: each piece counts again
constexpr int kSolePairs = 1 << 14;
constexpr int kSortChunks = 256;
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;

struct SortPlan {
  int chunk, blocks;  // pairs per workgroup (a multiple of kSortThreads) and workgroups
};
inline SortPlan sort_plan(int64_t P) {
  const int64_t per = (P + kSortChunks - 1) / kSortChunks;
  const int chunk = (int)((per + kSortThreads - 1) / kSortThreads * kSortThreads);
  return {chunk, (int)((P + chunk - 1) / chunk)};
}

template <int CTRL, int ROW_MASK>
__device__ __forceinline__ int dpp_add(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, ROW_MASK, 0xf, false);
}

// Exclusive prefix of one int per thread over a workgroup of W wavefronts; *total receives the
// sum.  s_wave: one int per wavefront.
template <int W>
__device__ __forceinline__ int group_prefix(int v, int* s_wave, int* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int x = v;
  x += dpp_add<0x111, 0xf>(x);  // row_shr:1, 2, 4, 8: prefixes of each 16-lane row
  x += dpp_add<0x112, 0xf>(x);
  x += dpp_add<0x114, 0xf>(x);
  x += dpp_add<0x118, 0xf>(x);
  x += dpp_add<0x142, 0xa>(x);  // row_bcast:15 into rows 1 and 3
  x += dpp_add<0x143, 0xc>(x);  // row_bcast:31 into rows 2 and 3
  if (lane == 63) s_wave[wave] = x;
  __syncthreads();
  int base = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    const int n = s_wave[w];
    base += w < wave ? n : 0;
    sum += n;
  }
  *total = sum;
  return base + x - v;
}

// Lanes of the wavefront whose key (< kMaxExperts) equals this lane's; a lane with valid = false
// gets 0.
__device__ __forceinline__ uint64_t wave_peers(int key, bool valid) {
  static_assert(kMaxExperts <= 1 << 10, "ten bits");
  uint64_t m = __ballot(valid);
#pragma unroll
  for (int b = 0; b < 10; ++b) {
    const uint64_t set = __ballot((key >> b) & 1);
    m &= ((key >> b) & 1) ? set : ~set;
  }
  return valid ? m : 0;
}

// One round of a chunk: kSortThreads pairs in order, e the thread's expert.  Returns the pair's
// rank among the round's pairs of its expert (lanes of its wavefront before it, then earlier
// wavefronts), and leaves the wavefronts' counts in s_cnt (zeroed here).
__device__ __forceinline__ int round_rank(int e, bool kept, int E, uint16_t (*s_cnt)[kMaxExperts]) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (tid < E) {
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) s_cnt[w][tid] = 0;
  }
  __syncthreads();
  const uint64_t peers = wave_peers(e, kept);
  int rank = __popcll(peers & ((1ull << lane) - 1));
  if (kept && rank == 0) s_cnt[wave][e] = (uint16_t)__popcll(peers);
  __syncthreads();
  if (kept) {
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) rank += w < wave ? s_cnt[w][e] : 0;
  }
  return rank;
}
__device__ __forceinline__ int round_total(int e, const uint16_t (*s_cnt)[kMaxExperts]) {
  int n = 0;
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) n += s_cnt[w][e];
  return n;
}

// The whole sort, one workgroup per chunk of kSortThreads pairs; LOADS: four-pair loads per
// thread that cover all pairs.
template <int LOADS>
__global__ __launch_bounds__(kSortThreads) void dispatch_place(const int32_t* __restrict__ idx, int P, int E,
                                                               int32_t* __restrict__ perm, int32_t* __restrict__ inv,
                                                               int32_t* __restrict__ offsets) {
  __shared__ int s_before[kMaxExperts], s_rest[kMaxExperts];
  __shared__ uint16_t s_cnt[kSortWaves][kMaxExperts];
  __shared__ int s_wave[kSortWaves];
  const int tid = threadIdx.x, lo = blockIdx.x * kSortThreads, p = lo + tid;
  const int mine = p < P ? idx[p] : -1;
  if (tid < E) s_before[tid] = s_rest[tid] = 0;
  __syncthreads();
  // four pairs to a load (chunks are multiples of four, so four neighbours lie on one side
  // of lo), all of them in flight
  u32x4 e[LOADS];
#pragma unroll
  for (int u = 0; u < LOADS; ++u) {
    const int p0 = 4 * (u * kSortThreads + tid);
    e[u] = ~(u32x4)0;
    if (p0 + 4 <= P) {
      e[u] = load16<false>(reinterpret_cast<const uint8_t*>(idx + p0));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (p0 + i < P) e[u][i] = idx[p0 + i];
    }
  }
#pragma unroll
  for (int u = 0; u < LOADS; ++u) {
    int* side = 4 * (u * kSortThreads + tid) < lo ? s_before : s_rest;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (e[u][i] < (unsigned)E) atomicAdd(&side[e[u][i]], 1);
  }
  const bool kept = (unsigned)mine < (unsigned)E;
  const int rank = round_rank(mine, kept, E, s_cnt);  // its barriers end the counting
  // an expert's first place in this chunk: kept pairs of lower experts, then its own pairs
  // in earlier chunks
  const int before = tid < E ? s_before[tid] : 0;
  int kept_all;
  const int base = group_prefix<kSortWaves>(before + (tid < E ? s_rest[tid] : 0), s_wave, &kept_all);
  if (blockIdx.x == 0) {
    if (tid < E) offsets[tid] = base;
    if (tid == 0) offsets[E] = kept_all;
  }
  if (tid < E) s_before[tid] = base + before;
  __syncthreads();
  int pos = kept ? s_before[mine] + rank : -1;
  if (pos >= P) pos = -1;  // only if the ids changed under the kernel
  if (pos >= 0) perm[pos] = p;
  if (p < P) inv[p] = pos;
}

__global__ __launch_bounds__(kSortThreads) void dispatch_rank(const int32_t* __restrict__ idx, int P, int E,
                                                              int chunk, int32_t* __restrict__ hist,
                                                              int32_t* __restrict__ ranks) {
  __shared__ int s_run[kMaxExperts];
  __shared__ uint16_t s_cnt[kSortWaves][kMaxExperts];
  const int tid = threadIdx.x, lo = blockIdx.x * chunk, hi = min(lo + chunk, P);
  if (tid < E) s_run[tid] = 0;
  for (int r0 = lo; r0 < hi; r0 += kSortThreads) {
    const int p = r0 + tid, e = p < hi ? idx[p] : -1;
    const bool kept = (unsigned)e < (unsigned)E;
    const int rank = round_rank(e, kept, E, s_cnt);
    if (kept) ranks[p] = s_run[e] + rank;
    __syncthreads();
    if (tid < E) s_run[tid] += round_total(tid, s_cnt);
  }
  if (tid < E) hist[(size_t)blockIdx.x * E + tid] = s_run[tid];
}

// hist[c][e] (pairs of expert e in chunk c) to the first place of those pairs, and the offsets.
// One workgroup; where there are fewer experts than threads, up to kScanParts share a column.
constexpr int kScanParts = 16;
__global__ __launch_bounds__(kSortThreads) void dispatch_scan(int32_t* __restrict__ hist, int E, int chunks,
                                                              int32_t* __restrict__ offsets) {
  __shared__ int s_part[kSortThreads], s_base[kMaxExperts], s_wave[kSortWaves];
  const int tid = threadIdx.x, parts = min(kSortThreads / E, kScanParts), e = tid % E, part = tid / E;
  const int per = (chunks + parts - 1) / parts, c0 = part * per, c1 = part < parts ? min(c0 + per, chunks) : 0;
  // a column's piece stays in registers up to this length; beyond it (65 chunks and more of 256
  // experts, 17 of more than 512) the rest is read twice, entry by entry the second time
  constexpr int kHold = 16;
  int v[kHold], sum = 0;
#pragma unroll
  for (int i = 0; i < kHold; ++i) v[i] = hist[(size_t)min(c0 + i, chunks - 1) * E + e];  // all in flight
#pragma unroll
  for (int i = 0; i < kHold; ++i) {
    v[i] = c0 + i < c1 ? v[i] : 0;
    sum += v[i];
  }
#pragma unroll 8
  for (int c = c0 + kHold; c < c1; ++c) sum += hist[(size_t)c * E + e];
  s_part[tid] = sum;
  __syncthreads();
  int total = 0;
  if (tid < E)
    for (int q = 0; q < parts; ++q) total += s_part[q * E + tid];
  int kept_all;
  const int base = group_prefix<kSortWaves>(total, s_wave, &kept_all);
  if (tid < E) {
    offsets[tid] = base;
    s_base[tid] = base;
  }
  if (tid == 0) offsets[E] = kept_all;
  __syncthreads();
  if (part >= parts) return;
  int at = s_base[e];
  for (int q = 0; q < part; ++q) at += s_part[q * E + e];
#pragma unroll
  for (int i = 0; i < kHold; ++i)
    if (c0 + i < c1) {
      hist[(size_t)(c0 + i) * E + e] = at;
      at += v[i];
    }
  for (int c = c0 + kHold; c < c1; ++c) {
    const int n = hist[(size_t)c * E + e];
    hist[(size_t)c * E + e] = at;
    at += n;
  }
}

// Between a wavefront's writes to LDS and its other lanes' reads: LDS serves one wavefront in
// order, so only the compiler has to keep the order.
__device__ __forceinline__ void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// The token of a wavefront, four to a workgroup, as a uniform value: its table entries and row
// addresses are then scalar, and a pair left out is a uniform branch.
__device__ __forceinline__ int wave_token() {
  return blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
}

// ---------------------------------------------------------------------------
// Rows of x to their sorted places.  A workgroup takes one token and 4 KB of its row, 16 bytes
// a thread, reads them once and writes them k times.  Bound by memory: 151 MB at 4096 tokens,
// k = 8, H = 2048 in bf16 take 27.2 us (5.5 TB/s; a fill of as many bytes writes 6.6).
// FIND: the pairs' places come from their ranks and the chunks' first places (lane j finds rank
// j's), and the tables are written beside the rows (by the workgroup of blockIdx.y = 0);
// otherwise from inv.  NT: stores that do not stay in the caches, see stream_rows.
struct MoveArgs {
  const uint8_t* x;         // nullptr: the tables alone
  int64_t pitch;
  int T, k, E, H;
  uint8_t* xs;
  int32_t* inv;             // [T,k] read, or written (FIND)
  const int32_t* idx;       // FIND: [T,k] expert ids,
  int chunk;                // pairs of a chunk,
  const int32_t* first;     // [chunks,E] first places,
  const int32_t* ranks;     // [T,k] ranks within the chunk
  int32_t* perm;            // and the other table
};

template <int EB, bool FIND, bool NT>
__global__ __launch_bounds__(256) void dispatch_move(MoveArgs a) {
  constexpr int FMT = EB == 2 ? MOE_AFMT_BF16 : MOE_AFMT_F32, N = 16 / EB;
  const int t = blockIdx.x, lane = threadIdx.x & 63;
  const Piece<N> at(blockIdx.y * blockDim.x + threadIdx.x, a.H);
  Chunk<FMT, N> q;
  if (a.x && at.on) q.load(a.x + (int64_t)t * a.pitch, at);
  for (int j0 = 0; j0 < a.k; j0 += 64) {
    const int p = t * a.k + j0 + lane, n = min(64, a.k - j0);
    int mine = -1;
    if (lane < n) {
      if constexpr (FIND) {
        const int e = a.idx[p];
        if ((unsigned)e < (unsigned)a.E) mine = a.first[(size_t)(p / a.chunk) * a.E + e] + a.ranks[p];
        if ((unsigned)mine >= (unsigned)(a.T * a.k)) mine = -1;  // none, or the ids changed under the call
        if (blockIdx.y == 0 && threadIdx.x < 64) {
          a.inv[p] = mine;
          if (mine >= 0) a.perm[mine] = p;
        }
      } else {
        mine = a.inv[p];
        if ((unsigned)mine >= (unsigned)(a.T * a.k)) mine = -1;
      }
    }
    if (!a.x) continue;
    for (int j = 0; j < n; ++j) {
      const int pos = __builtin_amdgcn_readlane(mine, j);
      if (pos >= 0 && at.on) q.template store<NT>(a.xs + (int64_t)pos * a.H * EB, at);
    }
  }
}

// The sort and the move of at most kTinyPairs pairs in one launch.  A pair's key is
// (expert, pair) in one word; its place is the number of smaller keys.  A wavefront takes one
// token and 1 KB of its row, so that a few tokens' rows spread over the chip (3.1 us at 4 tokens,
// k = 8, H = 2048); the last workgroup (of blockIdx.y = 0) writes the offsets.
template <int EB, int R>  // R: 64-pair registers of keys
__global__ __launch_bounds__(256) void dispatch_tiny(const int32_t* __restrict__ idx, int T, int k, int E,
                                                     const uint8_t* __restrict__ x, int64_t pitch, int H,
                                                     uint8_t* __restrict__ xs, int32_t* __restrict__ perm,
                                                     int32_t* __restrict__ inv, int32_t* __restrict__ offsets) {
  const int P = T * k, lane = threadIdx.x & 63;
  if (blockIdx.x == gridDim.x - 1) {
    __shared__ int s_n[kMaxExperts], s_wave[4];
    if (blockIdx.y != 0) return;
    int ids[kTinyPairs / 256];
#pragma unroll
    for (int i = 0; i < kTinyPairs / 256; ++i) {
      const int p = 256 * i + threadIdx.x, e = idx[min(p, P - 1)];  // no branch: the loads overlap
      ids[i] = p < P ? e : -1;
    }
    for (int e = threadIdx.x; e < kMaxExperts; e += 256) s_n[e] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kTinyPairs / 256; ++i)
      if ((unsigned)ids[i] < (unsigned)E) atomicAdd(&s_n[ids[i]], 1);
    __syncthreads();
    // four neighbouring experts per thread
    int n[4], total;
#pragma unroll
    for (int i = 0; i < 4; ++i) n[i] = s_n[4 * threadIdx.x + i];
    int at = group_prefix<4>(n[0] + n[1] + n[2] + n[3], s_wave, &total);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = 4 * threadIdx.x + i;
      if (e < E) offsets[e] = at;
      at += n[i];
    }
    if (threadIdx.x == 0) offsets[E] = total;
    return;
  }
  const int t = wave_token();
  if (t >= T) return;
  constexpr int FMT = EB == 2 ? MOE_AFMT_BF16 : MOE_AFMT_F32, N = 16 / EB;
  const Piece<N> at(blockIdx.y * 64 + lane, H);
  Chunk<FMT, N> q;
  if (x && at.on) q.load(x + (int64_t)t * pitch, at);
  uint32_t key[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int p = 64 * i + lane;
    key[i] = idx[min(p, P - 1)];
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int p = 64 * i + lane;
    key[i] = p < P && key[i] < (unsigned)E ? key[i] << 10 | p : 0xffffffffu;
  }
  constexpr int kAtOnce = 8;  // ranks counted together: the counts of one hide the others' waits
  for (int j0 = 0; j0 < k; j0 += 64) {
    const int n = min(64, k - j0), p0 = t * k + j0;
    const int id = lane < n ? idx[p0 + lane] : -1;
    const uint32_t mine = (unsigned)id < (unsigned)E ? (uint32_t)id << 10 | (p0 + lane) : 0xffffffffu;
    int place = -1;  // of rank j0 + lane
    for (int j1 = 0; j1 < n; j1 += kAtOnce) {
      uint32_t own[kAtOnce];
      int pos[kAtOnce];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        own[j] = __builtin_amdgcn_readlane(mine, j1 + j);  // lanes behind the ranks hold no key
        pos[j] = 0;
      }
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) pos[j] += __popcll(__ballot(key[i] < own[j]));
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        if (own[j] == 0xffffffffu) continue;
        pos[j] = min(pos[j], P - 1);  // P only if the ids changed under the kernel
        if (lane == j1 + j) place = pos[j];
        if (x && at.on) q.store(xs + (int64_t)pos[j] * H * EB, at);
      }
    }
    if (blockIdx.y == 0 && lane < n) {
      inv[p0 + lane] = place;
      if (place >= 0) perm[place] = p0 + lane;
    }
  }
}

// ---------------------------------------------------------------------------
// y[t] = sum_j w[t,j] rows[inv[t,j]] in rank order (w = nullptr: a plain sum, the gradient
// of the move).  A workgroup takes one token and 2048 elements of its row, so that the
// scattered rows are read in pieces of 4 KB and more (a wavefront per token and 512 elements:
// 46 us where this takes 28.5, 168 MB at 4096 tokens, k = 8, H = 2048, bf16 to fp32: 5.9 TB/s);
// kRanks rows are in flight per lane, more ranks go round again.  Outputs go out by
// non-temporal stores: 33.8 us against 38.2 there with ordinary loads, and a kernel that reads y
// next takes no longer (1024 tokens: 12.5 us for both against 15.3).
constexpr int kRanks = 8;

// A token's ranks j0 .. j0 + kRanks - 1: places (-1: left out) and gates, in scalar registers.  The
// lanes read them at once and every lane is asked for its own: one load each, where reading
// them rank by rank is a chain of scalar loads and branches.
template <bool WEIGHTED>
struct TokenRanks {
  int pos[kRanks];
  float w[kRanks];
  __device__ __forceinline__ TokenRanks(const int32_t* inv, const float* gates, int j0, int k, int T) {
    const int lane = threadIdx.x & 63, j = min(j0 + (lane & (kRanks - 1)), k - 1);
    int p = inv[j];
    const float g = WEIGHTED ? gates[j] : 1.f;
    if (j0 + (lane & (kRanks - 1)) >= k || (unsigned)p >= (unsigned)(T * k)) p = -1;
#pragma unroll
    for (int i = 0; i < kRanks; ++i) {
      pos[i] = __builtin_amdgcn_readlane(p, i);
      w[i] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(g), i));
    }
  }
  __device__ __forceinline__ bool kept(int j) const { return pos[j] >= 0; }
};

template <int RF, int YF, bool WEIGHTED, bool NT>
__global__ __launch_bounds__(256) void combine_rows(const uint8_t* __restrict__ rows, const int32_t* __restrict__ inv,
                                                    const float* __restrict__ w, int T, int k, int H,
                                                    uint8_t* __restrict__ y, int64_t pitch) {
  constexpr int N = 8, RB = kElemBytes<RF>;
  const int t = blockIdx.x;
  const Piece<N> at(blockIdx.y * blockDim.x + threadIdx.x, H);
  const int64_t p0 = (int64_t)t * k;
  float acc[N];
#pragma unroll
  for (int n = 0; n < N; ++n) acc[n] = 0.f;
  for (int j0 = 0; j0 < k; j0 += kRanks) {
    const TokenRanks<WEIGHTED> ranks(inv + p0, WEIGHTED ? w + p0 : nullptr, j0, k, T);
    Chunk<RF, N> q[kRanks];
#pragma unroll
    for (int j = 0; j < kRanks; ++j)
      if (at.on && ranks.kept(j)) q[j].template load<NT>(rows + (int64_t)ranks.pos[j] * H * RB, at);
#pragma unroll
    for (int j = 0; j < kRanks; ++j)
      if (ranks.kept(j)) {
#pragma unroll
        for (int n = 0; n < N; ++n) acc[n] = WEIGHTED ? fmaf(ranks.w[j], q[j].get(n), acc[n]) : acc[n] + q[j].get(n);
      }
  }
  if (!at.on) return;
  Chunk<YF, N> o;
  o.set(acc);
  o.template store_wave<true>(y + (int64_t)t * pitch, at, H);
}

// ---------------------------------------------------------------------------
// The weighted return's gradient: dys[inv[t,j]] = w[t,j] dy[t], dw[t,j] = <dy[t], ys[inv[t,j]]>.
// A workgroup takes one token and up to kRanks of its ranks, its wavefronts neighbouring
// pieces of the row; the dot products meet in LDS in wavefront order.  Bound by memory: 297 MB at
// 4096 tokens, k = 8, H = 2048 (dy fp32, rows bf16) take 56.4 us (5.3 TB/s); with one wavefront
// 70.0, with two 74.4.
constexpr int kCbWaves = 4;

template <int DF, int RF, bool NT>
__global__ __launch_bounds__(64 * kCbWaves) void combine_rows_backward(const uint8_t* __restrict__ dy, int64_t pitch,
                                                                       const uint8_t* ys,
                                                                       const int32_t* __restrict__ inv,
                                                                       const float* __restrict__ w, int T, int k, int H,
                                                                       uint8_t* dys, float* __restrict__ dw) {
  constexpr int N = 8, RB = kElemBytes<RF>;
  __shared__ float s_dot[kCbWaves][kRanks];
  const int t = blockIdx.x, j0 = blockIdx.y * kRanks, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t p0 = (int64_t)t * k;
  // the gates only for dys; read as inv otherwise, and not used
  const TokenRanks<true> ranks(inv + p0, dys ? w + p0 : reinterpret_cast<const float*>(inv + p0), j0, k, T);
  float dot[kRanks];
#pragma unroll
  for (int j = 0; j < kRanks; ++j) dot[j] = 0.f;
  for (int c = threadIdx.x; c * N < H; c += blockDim.x) {
    const Piece<N> at(c, H);
    Chunk<DF, N> d;
    Chunk<RF, N> q[kRanks];
    d.load(dy + (int64_t)t * pitch, at);
    if (dw) {
#pragma unroll
      for (int j = 0; j < kRanks; ++j)
        if (ranks.kept(j)) q[j].template load<NT>(ys + (int64_t)ranks.pos[j] * H * RB, at);
      if (at.skip) {
        d.drop(at.skip);
#pragma unroll
        for (int j = 0; j < kRanks; ++j) q[j].drop(at.skip);
      }
#pragma unroll
      for (int j = 0; j < kRanks; ++j)
        if (ranks.kept(j)) {
#pragma unroll
          for (int n = 0; n < N; ++n) dot[j] = fmaf(d.get(n), q[j].get(n), dot[j]);
        }
    }
    if (dys) {
#pragma unroll
      for (int j = 0; j < kRanks; ++j)
        if (ranks.kept(j)) {
          float v[N];
#pragma unroll
          for (int n = 0; n < N; ++n) v[n] = ranks.w[j] * d.get(n);
          q[j].set(v);
          q[j].template store_wave<true>(dys + (int64_t)ranks.pos[j] * H * RB, at, H);
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
    for (int x = 0; x < (int)blockDim.x / 64; ++x) v += s_dot[x][threadIdx.x];
    dw[p0 + j0 + threadIdx.x] = v;
  }
}

// ---------------------------------------------------------------------------
// The gradient of the gates: one wavefront per token, four neighbouring logits per lane and
// load.  The gates' gradients are first gathered by expert in the wavefront's table in LDS (their
// sum and number per expert): a lane per rank, at once where a token's experts differ;
// otherwise the first lane of an expert adds up its ranks in order.  A token's logits are
// all read before any of its gradients is written (dlogits may be logits).  Bound by one round trip
// to memory and three wavefront sums: 4.0 us at 4096 tokens of 256 logits, k = 8 (4.6 when every
// token's ranks were compared one by one), 4.8 at 997 of 1000 with k = 16 (5.4; 10.5 when
// every lane compared its logits with every rank).
template <int C>  // loads of 256 logits
__global__ __launch_bounds__(256) void topk_backward_kernel(const float* logits, int T, int E, int k,
                                                            const int32_t* __restrict__ idx,
                                                            const float* __restrict__ dw, int renorm,
                                                            float* dlogits) {
  __shared__ __attribute__((aligned(16))) float2 s_tab[4][256 * C];
  const int t = wave_token(), lane = threadIdx.x & 63;
  if (t >= T) return;
  float2* tab = s_tab[threadIdx.x >> 6];
  const uint8_t* z = reinterpret_cast<const uint8_t*>(logits + (int64_t)t * E);
  Chunk<MOE_AFMT_F32, 4> q[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const Piece<4> at(64 * c + lane, E);
    if (at.on) q[c].load(z, at);
    // by lane, a stride of 64 entries: neighbours in neighbouring banks
#pragma unroll
    for (int n = 0; n < 4; ++n) tab[256 * c + 64 * n + lane] = make_float2(0.f, 0.f);
  }
  wave_lds_order();
  for (int j0 = 0; j0 < k; j0 += 64) {
    const int j = j0 + lane, nj = min(64, k - j0);
    const int e = j < k ? idx[(int64_t)t * k + j] : -1;
    const float g = j < k ? dw[(int64_t)t * k + j] : 0.f;
    const bool kept = (unsigned)e < (unsigned)E;
    // a token's experts usually differ (as moe_topk leaves them): then no lane finds another's
    // number in its expert's entry, and its own gradient is the sum
    const float2 was = kept ? tab[e] : make_float2(0.f, 0.f);
    wave_lds_order();
    if (kept) tab[e].x = __int_as_float(lane);
    wave_lds_order();
    const bool shared = kept && __float_as_int(tab[e].x) != lane;
    float sum = g, cnt = 1.f;
    bool first = kept;
    if (__ballot(shared)) {
      sum = cnt = 0.f;
      for (int i = 0; i < nj; ++i) {
        const int ei = __builtin_amdgcn_readlane(e, i);
        const float gi = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(g), i));
        const bool same = ei == e;
        sum += same ? gi : 0.f;
        cnt += same ? 1.f : 0.f;
        first = first && !(same && i < lane);
      }
    }
    wave_lds_order();
    if (first) tab[e] = make_float2(was.x + sum, was.y + cnt);
    wave_lds_order();
  }
  float v[C][4], n[C][4], d[C][4];
  float mx = -INFINITY;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const Piece<4> at(64 * c + lane, E);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool own = at.on && i >= at.skip && i < at.n;
      const float2 a = tab[at.i + i];  // in the table also where it is not the lane's own
      d[c][i] = own ? a.x : 0.f;
      n[c][i] = own ? a.y : 0.f;
      // the softmax runs over all experts, or over the chosen ones (each as often as it was)
      v[c][i] = own && (!renorm || a.y > 0.f) ? q[c].get(i) : -INFINITY;
      mx = fmaxf(mx, v[c][i]);
    }
  }
  mx = wave_max(mx);
  float sum = 0.f, mean = 0.f;
  uint32_t live = 0;  // a bit for each of the lane's logits that is in the softmax
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // a masked logit (-inf) has no share, also where every logit is masked, and no part in
      // the mean, whatever the gate's gradient there (0 * inf would be NaN)
      const bool in = v[c][i] != -INFINITY;
      live |= in ? 1u << (4 * c + i) : 0u;
      v[c][i] = in ? __expf(v[c][i] - mx) : 0.f;
      sum += renorm ? n[c][i] * v[c][i] : v[c][i];
      mean += in ? d[c][i] * v[c][i] : 0.f;
    }
  sum = wave_sum(sum);
  mean = wave_sum(mean);
  const float r = sum == 0.f ? 0.f : 1.f / sum;
  mean *= r;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    float o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // 0 where there is no share (masked, or not chosen with renorm), also under a NaN mean
      o[i] = live >> (4 * c + i) & 1 ? v[c][i] * r * (d[c][i] - (renorm ? n[c][i] * mean : mean)) : 0.f;
    }
    Chunk<MOE_AFMT_F32, 4> out;
    out.set(o);
    out.store_own(reinterpret_cast<uint8_t*>(dlogits + (int64_t)t * E), Piece<4>(64 * c + lane, E));
  }
}

namespace {

bool move_shape_ok(int32_t T, int32_t k, int32_t H) {
  return T >= 1 && T <= kMoveMaxT && k >= 1 && k <= kMoveMaxK && (int64_t)T * k <= kMoveMaxPairs && H >= 1 &&
         H <= kMoveMaxH;
}

// int32 and fp32 tables: aligned to their elements (a null one is).
template <typename... P>
bool tables_aligned(const P*... p) { return (aligned_to(p, 4) && ...); }

// A caller's row stride in elements (0: dense rows), or -1.
int64_t row_stride(int64_t ld, int32_t H) { return ld == 0 ? H : (ld >= H && ld <= kMaxStride ? ld : -1); }

Span rows_of(const void* p, int64_t rows, int32_t H, int fmt, int64_t ld) {
  return {p, rows, H * fmt_bytes(fmt), ld * fmt_bytes(fmt)};
}

// The workgroup of a row of H in chunks of n elements: up to four wavefronts, none without a
// chunk (4096 tokens, k = 8, rows of 256: combine 5.8 us against 8.0 with four, its gradient 8.6
// against 14.1, the move 6.5 against 8.6).
dim3 row_block(int H, int n) { return dim3(64 * std::clamp((H + 64 * n - 1) / (64 * n), 1, 4)); }

// One instantiation of `f` by two formats and a truth value.
template <typename F>
moe_status by_formats(int a, int b, bool nt, F f) {
  constexpr auto B = std::integral_constant<int, MOE_AFMT_BF16>{};
  constexpr auto S = std::integral_constant<int, MOE_AFMT_F32>{};
  const auto with = [&](auto x, auto y) { return nt ? f(x, y, std::true_type{}) : f(x, y, std::false_type{}); };
  if (a == MOE_AFMT_BF16) return b == MOE_AFMT_BF16 ? with(B, B) : with(B, S);
  return b == MOE_AFMT_BF16 ? with(S, B) : with(S, S);
}

template <bool WEIGHTED>
moe_status run_combine(const void* rows, int fmt, const int32_t* inv, const float* w, int T, int k, int H, void* y,
                       int y_fmt, int64_t ld, hipStream_t s) {
  const bool nt = stream_rows((int64_t)T * k * H * fmt_bytes(fmt));
  return by_formats(fmt, y_fmt, nt, [&](auto rf, auto yf, auto n) {
    return launch(combine_rows<rf(), yf(), WEIGHTED, n()>, dim3(T, (H + 256 * 8 - 1) / (256 * 8)), row_block(H, 8), s,
                  static_cast<const uint8_t*>(rows), inv, w, T, k, H, static_cast<uint8_t*>(y), ld * fmt_bytes(y_fmt));
  });
}

}  // namespace
}  // namespace rmoe

using namespace rmoe;

extern "C" MOE_API int64_t moe_dispatch_workspace(int32_t T, int32_t k, int32_t n_experts) {
  if (!move_shape_ok(T, k, 1) || n_experts < 1 || n_experts > kMaxExperts) return -1;
  const int64_t P = (int64_t)T * k;
  return P <= kSolePairs ? 0 : 4 * ((int64_t)sort_plan(P).blocks * n_experts + P);
}

extern "C" MOE_API moe_status moe_dispatch(const int32_t* topk_idx, int32_t T, int32_t k, int32_t n_experts,
                                           const void* x, int32_t fmt, int32_t H, int64_t ld_x, void* xs,
                                           int32_t* perm, int32_t* inv, int32_t* offsets, void* ws, size_t ws_bytes,
                                           moe_stream_t stream) {
  if (!topk_idx || !perm || !inv || !offsets || (x == nullptr) != (xs == nullptr)) return MOE_EINVAL;
  const int64_t need = moe_dispatch_workspace(T, k, n_experts);
  if (need < 0 || (need > 0 && !ws) || ws_bytes < (size_t)need || !aligned_to(ws, 4)) return MOE_EINVAL;
  if (!tables_aligned(topk_idx, perm, inv, offsets)) return MOE_EINVAL;
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
  const hipStream_t s = stream_of(stream);
  const StreamDevice on(s);
  const uint8_t* src = static_cast<const uint8_t*>(x);
  uint8_t* dst = static_cast<uint8_t*>(xs);
  const int width = x ? H : 1;  // H says nothing of a sort alone
  const int64_t eb = x ? fmt_bytes(fmt) : 4, pitch = ld * eb, row_bytes = x ? H * eb : 1;
  if (P <= kTinyPairs && T * ((row_bytes + 1023) / 1024) <= kTinyPieces) {
    const dim3 grid((T + 3) / 4 + 1, (unsigned)((row_bytes + 1023) / 1024)), block(256);
    const auto go = [&](auto kernel) {
      return launch(kernel, grid, block, s, topk_idx, T, k, n_experts, src, pitch, width, dst, perm, inv, offsets);
    };
    if (P <= 64) return eb == 2 ? go(dispatch_tiny<2, 1>) : go(dispatch_tiny<4, 1>);
    if (P <= 256) return eb == 2 ? go(dispatch_tiny<2, 4>) : go(dispatch_tiny<4, 4>);
    return eb == 2 ? go(dispatch_tiny<2, kTinyPairs / 64>) : go(dispatch_tiny<4, kTinyPairs / 64>);
  }
  const dim3 threads(kSortThreads);
  MoveArgs m{src, pitch, T, k, n_experts, width, dst, inv};
  const auto move = [&](auto find) {
    constexpr bool F = find();
    const bool nt = stream_rows(P * row_bytes);
    const auto kernel = eb == 2 ? (nt ? dispatch_move<2, F, true> : dispatch_move<2, F, false>)
                                : (nt ? dispatch_move<4, F, true> : dispatch_move<4, F, false>);
    return launch(kernel, dim3(T, (unsigned)((row_bytes + 4095) / 4096)), row_block(width, (int)(16 / eb)), s, m);
  };
  if (P <= kSolePairs) {
    const dim3 chunks((unsigned)((P + kSortThreads - 1) / kSortThreads));
    static_assert(kSolePairs <= 4 * 4 * kSortThreads, "LOADS");
    const moe_status st = launch(P <= 2 * 4 * kSortThreads ? dispatch_place<2> : dispatch_place<4>, chunks, threads, s,
                                 topk_idx, (int)P, n_experts, perm, inv, offsets);
    return st != MOE_OK || !x ? st : move(std::false_type{});
  }
  const SortPlan sp = sort_plan(P);
  int32_t* hist = static_cast<int32_t*>(ws);
  int32_t* ranks = hist + (int64_t)sp.blocks * n_experts;
  moe_status st = launch(dispatch_rank, dim3(sp.blocks), threads, s, topk_idx, (int)P, n_experts, sp.chunk, hist, ranks);
  if (st == MOE_OK) st = launch(dispatch_scan, dim3(1), threads, s, hist, n_experts, sp.blocks, offsets);
  if (st != MOE_OK) return st;
  m.idx = topk_idx;
  m.chunk = sp.chunk;
  m.first = hist;
  m.ranks = ranks;
  m.perm = perm;
  return move(std::true_type{});
}

extern "C" MOE_API moe_status moe_dispatch_backward(const void* dxs, int32_t dxs_fmt, const int32_t* inv, int32_t T,
                                                    int32_t k, int32_t H, void* dx, int32_t dx_fmt, int64_t ld_dx,
                                                    moe_stream_t stream) {
  const int64_t ld = row_stride(ld_dx, H), P = (int64_t)T * k;
  if (!dxs || !inv || !dx || !fmt_ok(dxs_fmt) || !fmt_ok(dx_fmt) || !move_shape_ok(T, k, H) || ld < 0) return MOE_EINVAL;
  if (!aligned_to(dxs, fmt_bytes(dxs_fmt)) || !aligned_to(dx, fmt_bytes(dx_fmt)) || !tables_aligned(inv)) return MOE_EINVAL;
  const Span out = rows_of(dx, T, H, dx_fmt, ld);
  if (overlap(out, rows_of(dxs, P, H, dxs_fmt, H)) || overlap(out, flat(inv, 4 * P))) return MOE_EINVAL;
  const hipStream_t s = stream_of(stream);
  const StreamDevice on(s);
  return run_combine<false>(dxs, dxs_fmt, inv, nullptr, T, k, H, dx, dx_fmt, ld, s);
}

extern "C" MOE_API moe_status moe_combine(const void* ys, int32_t ys_fmt, const int32_t* inv, const float* w, int32_t T,
                                          int32_t k, int32_t H, void* y, int32_t y_fmt, int64_t ld_y,
                                          moe_stream_t stream) {
  const int64_t ld = row_stride(ld_y, H), P = (int64_t)T * k;
  if (!ys || !inv || !w || !y || !fmt_ok(ys_fmt) || !fmt_ok(y_fmt) || !move_shape_ok(T, k, H) || ld < 0)
    return MOE_EINVAL;
  if (!aligned_to(ys, fmt_bytes(ys_fmt)) || !aligned_to(y, fmt_bytes(y_fmt)) || !tables_aligned(inv, w)) return MOE_EINVAL;
  const Span out = rows_of(y, T, H, y_fmt, ld);
  if (overlap(out, rows_of(ys, P, H, ys_fmt, H)) || overlap(out, flat(inv, 4 * P)) || overlap(out, flat(w, 4 * P)))
    return MOE_EINVAL;
  const hipStream_t s = stream_of(stream);
  const StreamDevice on(s);
  return run_combine<true>(ys, ys_fmt, inv, w, T, k, H, y, y_fmt, ld, s);
}

extern "C" MOE_API moe_status moe_combine_backward(const void* dy, int32_t dy_fmt, int64_t ld_dy, const void* ys,
                                                   int32_t ys_fmt, const int32_t* inv, const float* w, int32_t T,
                                                   int32_t k, int32_t H, void* dys, float* dw, moe_stream_t stream) {
  const int64_t ld = row_stride(ld_dy, H), P = (int64_t)T * k;
  if (!dy || !inv || (!dys && !dw) || (dw && !ys) || (dys && !w)) return MOE_EINVAL;
  if (!fmt_ok(dy_fmt) || !fmt_ok(ys_fmt) || !move_shape_ok(T, k, H) || ld < 0) return MOE_EINVAL;
  if (!aligned_to(dy, fmt_bytes(dy_fmt)) || !aligned_to(ys, fmt_bytes(ys_fmt)) || !aligned_to(dys, fmt_bytes(ys_fmt)) ||
      !tables_aligned(inv, w, dw))
    return MOE_EINVAL;
  const Span in[4] = {rows_of(dy, T, H, dy_fmt, ld), dys == ys ? flat(nullptr, 0) : rows_of(ys, P, H, ys_fmt, H),
                      flat(inv, 4 * P), flat(w, 4 * P)};
  const Span out[2] = {rows_of(dys, P, H, ys_fmt, H), flat(dw, 4 * P)};
  for (const Span& o : out)
    for (const Span& i : in)
      if (overlap(o, i)) return MOE_EINVAL;
  if (overlap(out[0], out[1])) return MOE_EINVAL;
  const hipStream_t s = stream_of(stream);
  const StreamDevice on(s);
  const bool nt = stream_rows(P * H * fmt_bytes(ys_fmt));
  return by_formats(dy_fmt, ys_fmt, nt, [&](auto df, auto rf, auto n) {
    return launch(combine_rows_backward<df(), rf(), n()>, dim3(T, (k + kRanks - 1) / kRanks), row_block(H, 8), s,
                  static_cast<const uint8_t*>(dy), ld * fmt_bytes(dy_fmt), static_cast<const uint8_t*>(ys), inv, w, T, k, H,
                  static_cast<uint8_t*>(dys), dw);
  });
}

extern "C" MOE_API moe_status moe_topk_backward(const float* logits, int32_t T, int32_t n_experts,
                                                const int32_t* topk_idx, int32_t k, const float* dw, int32_t renorm,
                                                float* dlogits, moe_stream_t stream) {
  if (!logits || !topk_idx || !dw || !dlogits || !move_shape_ok(T, k, 1)) return MOE_EINVAL;
  if (n_experts < 1 || n_experts > kMaxExperts || (renorm != 0 && renorm != 1)) return MOE_EINVAL;
  if (!tables_aligned(logits, topk_idx, dw, dlogits)) return MOE_EINVAL;
  const int64_t P = (int64_t)T * k, n = (int64_t)T * n_experts;
  const Span out = flat(dlogits, 4 * n);
  if ((dlogits != logits && overlap(out, flat(logits, 4 * n))) || overlap(out, flat(topk_idx, 4 * P)) ||
      overlap(out, flat(dw, 4 * P)))
    return MOE_EINVAL;
  const hipStream_t s = stream_of(stream);
  const StreamDevice on(s);
  const dim3 grid((T + 3) / 4), block(256);
  const int E = n_experts;
  const auto kernel = E <= 256 ? topk_backward_kernel<1> : E <= 512 ? topk_backward_kernel<2>
                      : E <= 768 ? topk_backward_kernel<3> : topk_backward_kernel<4>;
  return launch(kernel, grid, block, s, logits, T, E, k, topk_idx, dw, renorm, dlogits);
}
