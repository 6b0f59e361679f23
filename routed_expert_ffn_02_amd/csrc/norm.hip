// The norms before and after a block, fused with the block's gate and residual scale:
//   u  = w_post * y / rms(y)      (w_post = nullptr: u = y)
//   h' = h + alpha * g * u        (g: none, one per token, or one per channel)
//   x  = w_pre * h' / rms(h')     rms(v) = sqrt(mean(v^2) + eps)
// and its gradient.  Memory-bound: a row is read once, kept in registers across its
// reductions, and written once (117 MB at 4096 rows of 2048, h and y fp32, x bf16: 18.1 us, 6.5
// TB/s; one row: 2.4 us, a launch and one round trip).  Statistics and all arithmetic are fp32;
// x is formed from h' before h' is rounded to its own type, so each output is rounded once.
#include <algorithm>

#include "rows.hpp"

namespace rmoe {

constexpr int kNormN = 8;          // elements of a lane's chunk
constexpr int kNormMaxWaves = 16;  // of a workgroup
// A row is one chunk per thread of one workgroup.  (With two, the gradient's rows and sums did
// not fit the 128 registers of a 1024-thread workgroup: 165 us at 1000 rows of 16384, bf16,
// against 27.3 at 8192.)
constexpr int kNormMaxH = 64 * kNormMaxWaves * kNormN;
constexpr int kNormMaxT = 1 << 21;  // a launch of T workgroups of 1024 threads stays below 2^32

struct NormArgs {
  int T, H, gate_kind;
  int64_t h_pitch, y_pitch, x_pitch;  // bytes between rows
  float alpha, eps, per_h;            // per_h = 1 / H
  const uint8_t *h, *y;
  const float *w_post, *gate, *w_pre;
  uint8_t *h_out, *x_out;             // forward
  const uint8_t *dh_in, *dx;          // backward
  uint8_t *dh, *dy;
  float* dgate_token;                 // [T]
  float* part;                        // partial sums of the weights' gradients [kinds][G][H]
  int part_pre, part_post;            // index of each kind in part, or -1
};

// The sum over the workgroup's wavefronts (at most W) of NV values per thread, in wavefront
// order.  Its one barrier stands between the wavefronts' writes and the reads of all of them, none
// behind the reads: before the next sum of the same object, the caller passes another barrier
// (that of a second object's sum, or its own), or a fast wavefront overwrites what a slow one has
// yet to read.
template <int NV, int W>
struct BlockSum {
  float v[NV][W];
  __device__ __forceinline__ void init() {
    for (int i = threadIdx.x; i < NV * W; i += blockDim.x) (&v[0][0])[i] = 0.f;
    __syncthreads();
  }
  __device__ __forceinline__ void sum(float (&s)[NV]) {
    const int wave = threadIdx.x >> 6;
#pragma unroll
    for (int i = 0; i < NV; ++i) s[i] = wave_sum(s[i]);
    if (blockDim.x == 64) return;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i][wave] = s[i];
    }
    __syncthreads();
    // all entries are read at once; those without a wavefront add nothing
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float all[W];
#pragma unroll
      for (int w = 0; w < W; ++w) all[w] = v[i][w];
      s[i] = all[0];
#pragma unroll
      for (int w = 1; w < W; ++w) s[i] += all[w];
    }
  }
};

// 1 / sqrt of a normal number (v_rsq_f32: within one unit in the last place).
__device__ __forceinline__ float inv_sqrt(float v) { return __builtin_amdgcn_rsqf(v); }

// fp32 weights of a chunk, 1 where there are none.
__device__ __forceinline__ void load_w(const float* w, const Piece<kNormN>& at, float (&v)[kNormN]) {
  Chunk<MOE_AFMT_F32, kNormN> q;
  if (w && at.on) q.load(reinterpret_cast<const uint8_t*>(w), at);
#pragma unroll
  for (int n = 0; n < kNormN; ++n) v[n] = w && at.on ? q.get(n) : 1.f;
}

// One workgroup per row.  Stores are non-temporal: at 4096 rows of 2048 (h, y fp32, x bf16) 20.4
// us against 25.9, and a kernel that reads x next takes as long as after ordinary stores, at 1 row
// and at 4096.  h_out may be h: a thread writes the elements that it alone sums, and what
// other threads read of them is dropped.
template <int HF, int YF, int XF, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void block_norm_kernel(NormArgs a) {
  constexpr int N = kNormN;
  __shared__ __attribute__((aligned(16))) BlockSum<1, WAVES> s_y, s_h;
  const int64_t t = blockIdx.x;
  const Piece<N> at(threadIdx.x, a.H);
  Chunk<HF, N> qh;
  Chunk<YF, N> qy;
  float wq[N], g[N], wp[N];
  if (a.y) qy.load_own(a.y + t * a.y_pitch, at);
  qh.load_own(a.h + t * a.h_pitch, at);
  load_w(a.w_post, at, wq);
  load_w(a.gate_kind == MOE_GATE_CHANNEL ? a.gate : nullptr, at, g);
  load_w(a.w_pre, at, wp);
  s_y.init();  // the loads are on their way
  s_h.init();
  float h[N];
#pragma unroll
  for (int n = 0; n < N; ++n) h[n] = qh.get(n);
  if (a.y) {
    float scale = a.alpha;
    if (a.gate_kind == MOE_GATE_TOKEN) scale *= a.gate[t];
    if (a.w_post) {
      float s[1] = {0.f};
#pragma unroll
      for (int n = 0; n < N; ++n) s[0] = fmaf(qy.get(n), qy.get(n), s[0]);
      s_y.sum(s);
      scale *= inv_sqrt(s[0] * a.per_h + a.eps);
    }
#pragma unroll
    for (int n = 0; n < N; ++n) h[n] = fmaf(scale * qy.get(n), wq[n] * g[n], h[n]);
    Chunk<HF, N> o;
    o.set(h);
    o.template store_wave<true>(a.h_out + t * a.h_pitch, at, a.H);
  }
  if (!a.x_out) return;
  float s[1] = {0.f};
#pragma unroll
  for (int n = 0; n < N; ++n) s[0] = fmaf(h[n], h[n], s[0]);
  s_h.sum(s);
  const float r = inv_sqrt(s[0] * a.per_h + a.eps);
#pragma unroll
  for (int n = 0; n < N; ++n) wp[n] = h[n] * r * wp[n];
  Chunk<XF, N> o;
  o.set(wp);
  o.template store_wave<true>(a.x_out + t * a.x_pitch, at, a.H);
}

// A chunk of one token's rows in the gradient, as stored.
template <int HF, int YF, int XF>
struct NormRows {
  Chunk<HF, kNormN> h, d;
  Chunk<YF, kNormN> y;
  Chunk<XF, kNormN> x;
  // Zeros for a gradient that does not come in.
  __device__ __forceinline__ void load(const NormArgs& a, int64_t t, const Piece<kNormN>& at) {
    h.zero();
    x.zero();
    d.zero();
    y.zero();
    if (a.dx) {
      h.load_own(a.h + t * a.h_pitch, at);
      x.load_own(a.dx + t * a.x_pitch, at);
    }
    if (a.dh_in) d.load_own(a.dh_in + t * a.h_pitch, at);
    if (a.y) y.load_own(a.y + t * a.y_pitch, at);
  }
  // All four come in and a row has 8 elements or more: loads without a branch, so that the
  // wait for one row does not become a wait for all that is under way.  keep_own follows.
  __device__ __forceinline__ void load_all(const NormArgs& a, int64_t t, const Piece<kNormN>& at) {
    const int64_t i = at.i;  // 0 in a lane behind the row
    h.load_at(a.h + t * a.h_pitch + i * kElemBytes<HF>);
    x.load_at(a.dx + t * a.x_pitch + i * kElemBytes<XF>);
    d.load_at(a.dh_in + t * a.h_pitch + i * kElemBytes<HF>);
    y.load_at(a.y + t * a.y_pitch + i * kElemBytes<YF>);
  }
  __device__ __forceinline__ void keep_own(const Piece<kNormN>& at) {
    const int skip = at.on ? at.skip : kNormN;
    h.keep_from(skip);
    x.keep_from(skip);
    d.keep_from(skip);
    y.keep_from(skip);
  }
};

// The gradient.  With r = 1 / rms(h'), d = w_pre dx, ry = 1 / rms(y), D = sum(dh' g_c w_post y):
//   dh = dh' + r (d - h' r^2 mean(d h'))          (dh' from the stream behind the block)
//   du = alpha g dh,  dy = ry (w_post du - y ry^2 mean(w_post du y))
//   dw_pre = sum_t dx h' r,  dw_post = sum_t du y ry,  dgate = alpha sum dh u
// A workgroup walks rows b, b + G, ...; its threads keep the weights' gradients of their
// own channels in registers over those rows and write one partial row at the end, which
// norm_reduce adds in workgroup order: no atomics, the same bits every time.  A channel gate g_c
// and w_post share one sum, S = sum_t alpha dh y ry: dw_post = g_c S, dgate = w_post S.
// REGULAR: every row comes in (load_all).  With up to eight wavefronts, whose threads have 256
// registers, the next row is then loaded before the current one's sums (AHEAD): 18.9 us at 2048
// rows of 4096 in bf16 with a channel gate, against 27.2 without.  A token gate is read behind both sums,
// a wait per row that AHEAD does not hide: 21.0 us there.  Otherwise (an input left out) loads are
// conditional: 17.6 us without y at that size, for 67 MB against 101.
template <int HF, int YF, int XF, int WAVES, bool REGULAR>
__global__ __launch_bounds__(64 * WAVES) void block_norm_backward_kernel(NormArgs a) {
  constexpr int N = kNormN;
  constexpr bool AHEAD = REGULAR && WAVES <= 8;
  __shared__ __attribute__((aligned(16))) BlockSum<3, WAVES> s_a;
  __shared__ __attribute__((aligned(16))) BlockSum<1, WAVES> s_b;
  const Piece<N> at(threadIdx.x, a.H);
  NormRows<HF, YF, XF> next;
  if (AHEAD) next.load_all(a, blockIdx.x, at);
  // wg = w_post g_c: du w_post = alpha g_t dh (g_c w_post), only the product is needed
  float wp[N], wg[N], gc[N], acc_pre[N], acc_post[N];
  load_w(a.w_pre, at, wp);
  load_w(a.w_post, at, wg);
  load_w(a.gate_kind == MOE_GATE_CHANNEL ? a.gate : nullptr, at, gc);
#pragma unroll
  for (int n = 0; n < N; ++n) {
    wg[n] *= gc[n];
    acc_pre[n] = acc_post[n] = 0.f;
  }
  s_a.init();
  s_b.init();
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    NormRows<HF, YF, XF> q;
    if constexpr (AHEAD) {
      q = next;
      next.load_all(a, min(t + gridDim.x, (int64_t)a.T - 1), at);
      q.keep_own(at);
    } else if constexpr (REGULAR) {
      q.load_all(a, t, at);
      q.keep_own(at);
    } else {
      q.load(a, t, at);
    }
    float s[3] = {0.f, 0.f, 0.f};  // sums of h'^2, d h', y^2
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const float hv = q.h.get(n), yv = q.y.get(n);
      s[0] = fmaf(hv, hv, s[0]);
      s[1] = fmaf(wp[n] * q.x.get(n), hv, s[1]);
      s[2] = fmaf(yv, yv, s[2]);
    }
    s_a.sum(s);
    const float r = inv_sqrt(s[0] * a.per_h + a.eps), hm = r * r * (s[1] * a.per_h);
    const float ry = a.w_post ? inv_sqrt(s[2] * a.per_h + a.eps) : 1.f;
    float dh[N], dot[1] = {0.f};
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const float hv = q.h.get(n), xv = q.x.get(n);
      dh[n] = fmaf(r, wp[n] * xv - hv * hm, q.d.get(n));
      acc_pre[n] = fmaf(xv, hv * r, acc_pre[n]);
      dot[0] = fmaf(dh[n] * wg[n], q.y.get(n), dot[0]);
    }
    if (a.dh) {
      Chunk<HF, N> o;
      o.set(dh);
      o.template store_wave<true>(a.dh + t * a.h_pitch, at, a.H);
    }
    if (!a.y) {
      __syncthreads();  // behind the reads of s_a, where the second sum's barrier does not come
      continue;
    }
    s_b.sum(dot);
    const float ag = a.gate_kind == MOE_GATE_TOKEN ? a.alpha * a.gate[t] : a.alpha;
    const float ym = a.w_post ? ag * ry * ry * (dot[0] * a.per_h) : 0.f;
    if (a.dgate_token && threadIdx.x == 0) a.dgate_token[t] = a.alpha * ry * dot[0];
    float v[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const float yv = q.y.get(n), du = ag * dh[n];
      v[n] = ry * (wg[n] * du - yv * ym);
      acc_post[n] = fmaf(du, yv * ry, acc_post[n]);
    }
    if (a.dy) {
      Chunk<YF, N> o;
      o.set(v);
      o.template store_wave<true>(a.dy + t * a.y_pitch, at, a.H);
    }
  }
  const auto put = [&](int kind, const float(&v)[N]) {
    if (kind < 0) return;
    Chunk<MOE_AFMT_F32, N> o;
    o.set(v);
    o.store_wave(reinterpret_cast<uint8_t*>(a.part + ((int64_t)kind * gridDim.x + blockIdx.x) * a.H), at, a.H);
  };
  put(a.part_pre, acc_pre);
  put(a.part_post, acc_post);
}

// The sum over the workgroups' partial rows, 32 channels per workgroup of this kernel: 32
// groups of 32 lanes take rows g, g + 32, ... and are added in order.  Each kind goes to up to
// two outputs, each with a factor per channel or none.  4.0 us for 8.4 MB of partial rows (256
// of 4096, two kinds): a launch and one read.
struct NormOut {
  float* p[2][2];
  const float* by[2][2];
};
__global__ __launch_bounds__(1024) void norm_reduce(const float* __restrict__ part, int G, int H, NormOut out) {
  __shared__ float s_v[32][33];
  const int lane = threadIdx.x & 31, group = threadIdx.x >> 5, i = blockIdx.x * 32 + lane, kind = blockIdx.y;
  const float* p = part + (int64_t)kind * G * H;
  float v = 0.f;
  for (int g0 = group; g0 < G; g0 += 256) {
    float r[8];  // eight rows in flight, without a branch
#pragma unroll
    for (int u = 0; u < 8; ++u) r[u] = p[(int64_t)min(g0 + 32 * u, G - 1) * H + min(i, H - 1)];
#pragma unroll
    for (int u = 0; u < 8; ++u) v += g0 + 32 * u < G ? r[u] : 0.f;
  }
  s_v[group][lane] = v;
  __syncthreads();
  if (group != 0 || i >= H) return;
  v = 0.f;
#pragma unroll
  for (int g = 0; g < 32; ++g) v += s_v[g][lane];
  for (int o = 0; o < 2; ++o)
    if (out.p[kind][o]) out.p[kind][o][i] = out.by[kind][o] ? v * out.by[kind][o][i] : v;
}

namespace {

// Wavefronts of a row of H.
int norm_waves(int H) { return (H + 64 * kNormN - 1) / (64 * kNormN); }

// Workgroups of the gradient kernel when weights' gradients are wanted: eight wavefronts per
// CU (of 256), in workgroups of 1 to 8, or one workgroup of up to 16.  Each leaves a partial row
// per kind, so their number is kept low: at 2048 rows of 4096, 512 workgroups took 22.1 + 4.7 us
// where 256 took 19.9 + 3.9 (18.9 + 4.0 since).
int norm_groups(int T, int H) { return std::min(T, 256 * std::clamp(8 / norm_waves(H), 1, 4)); }

template <bool BACK, int HF, int YF, int XF>
moe_status launch_norm_f(const NormArgs& a, int groups, hipStream_t s) {
  const int waves = norm_waves(a.H);
  const dim3 grid(groups), block(64 * waves);
  if constexpr (BACK) {
    const bool regular = a.H >= kNormN && a.dx && a.dh_in && a.y;
    const auto kernel = !regular    ? block_norm_backward_kernel<HF, YF, XF, kNormMaxWaves, false>
                        : waves > 8 ? block_norm_backward_kernel<HF, YF, XF, kNormMaxWaves, true>
                                    : block_norm_backward_kernel<HF, YF, XF, 8, true>;
    return launch(kernel, grid, block, s, a);
  } else {
    const auto kernel = waves > 4 ? block_norm_kernel<HF, YF, XF, kNormMaxWaves> : block_norm_kernel<HF, YF, XF, 4>;
    return launch(kernel, grid, block, s, a);
  }
}

template <bool BACK>
moe_status launch_norm(const moe_norm_config& c, const NormArgs& a, int groups, hipStream_t s) {
  constexpr int B = MOE_AFMT_BF16, F = MOE_AFMT_F32;
  const int kind = (c.h_fmt == B ? 4 : 0) + (c.y_fmt == B ? 2 : 0) + (c.x_fmt == B ? 1 : 0);
  switch (kind) {
    case 0: return launch_norm_f<BACK, F, F, F>(a, groups, s);
    case 1: return launch_norm_f<BACK, F, F, B>(a, groups, s);
    case 2: return launch_norm_f<BACK, F, B, F>(a, groups, s);
    case 3: return launch_norm_f<BACK, F, B, B>(a, groups, s);
    case 4: return launch_norm_f<BACK, B, F, F>(a, groups, s);
    case 5: return launch_norm_f<BACK, B, F, B>(a, groups, s);
    case 6: return launch_norm_f<BACK, B, B, F>(a, groups, s);
    default: return launch_norm_f<BACK, B, B, B>(a, groups, s);
  }
}

// Checks of the configuration shared by both directions; fills the strides.
bool norm_config_ok(const moe_norm_config* c, NormArgs* a) {
  if (!c || c->T < 1 || c->T > kNormMaxT || c->H < 1 || c->H > kNormMaxH) return false;
  if (!fmt_ok(c->h_fmt) || !fmt_ok(c->y_fmt) || !fmt_ok(c->x_fmt)) return false;
  if (c->gate_kind < MOE_GATE_NONE || c->gate_kind > MOE_GATE_CHANNEL) return false;
  if (!(c->eps >= 0x1p-126f) || !(c->eps <= 1.f) || !(c->alpha - c->alpha == 0.f)) return false;
  const int64_t ld[3] = {c->ld_h ? c->ld_h : c->H, c->ld_y ? c->ld_y : c->H, c->ld_x ? c->ld_x : c->H};
  for (int64_t v : ld)
    if (v < c->H || v > kMaxStride) return false;
  a->T = c->T;
  a->H = c->H;
  a->gate_kind = c->gate_kind;
  a->alpha = c->alpha;
  a->eps = c->eps;
  a->per_h = 1.f / (float)c->H;
  a->h_pitch = ld[0] * fmt_bytes(c->h_fmt);
  a->y_pitch = ld[1] * fmt_bytes(c->y_fmt);
  a->x_pitch = ld[2] * fmt_bytes(c->x_fmt);
  return true;
}

struct NormSpans {
  const moe_norm_config& c;
  const NormArgs& a;
  Span h(const void* p) const { return {p, c.T, c.H * fmt_bytes(c.h_fmt), a.h_pitch}; }
  Span y(const void* p) const { return {p, c.T, c.H * fmt_bytes(c.y_fmt), a.y_pitch}; }
  Span x(const void* p) const { return {p, c.T, c.H * fmt_bytes(c.x_fmt), a.x_pitch}; }
  Span w(const void* p) const { return flat(p, 4ll * c.H); }
  Span gate(const void* p) const {
    return flat(p, c.gate_kind == MOE_GATE_NONE ? 0 : 4ll * (c.gate_kind == MOE_GATE_TOKEN ? c.T : c.H));
  }
};

// Whether an output shares bytes with an input or another output.  same[o]: the input that
// output o may be one and the same block with, or -1.
bool any_overlap(const Span* in, int n_in, const Span* out, int n_out, const int* same) {
  for (int o = 0; o < n_out; ++o) {
    for (int i = 0; i < n_in; ++i)
      if (!(same[o] == i && out[o].p == in[i].p) && overlap(out[o], in[i])) return true;
    for (int q = 0; q < o; ++q)
      if (overlap(out[o], out[q])) return true;
  }
  return false;
}

}  // namespace
}  // namespace rmoe

using namespace rmoe;

moe_status rmoe::block_norm(const moe_norm_config* cfg, const void* h, const void* y, const float* w_post,
                            const float* gate, const float* w_pre, void* h_out, void* x_out, hipStream_t s,
                            bool check_only) {
  NormArgs a{};
  if (!norm_config_ok(cfg, &a) || !h) return MOE_EINVAL;
  if (y ? !h_out : (h_out || w_post || !x_out)) return MOE_EINVAL;
  if ((gate != nullptr) != (cfg->gate_kind != MOE_GATE_NONE) || (gate && !y)) return MOE_EINVAL;
  if ((w_pre != nullptr) != (x_out != nullptr)) return MOE_EINVAL;
  const int64_t hb = fmt_bytes(cfg->h_fmt), yb = fmt_bytes(cfg->y_fmt), xb = fmt_bytes(cfg->x_fmt);
  if (!aligned_to(h, hb) || !aligned_to(y, yb) || !aligned_to(h_out, hb) || !aligned_to(x_out, xb) ||
      !aligned_to(w_post, 4) || !aligned_to(gate, 4) || !aligned_to(w_pre, 4))
    return MOE_EINVAL;
  const NormSpans sp{*cfg, a};
  const Span in[5] = {sp.h(h), sp.y(y), sp.w(w_post), sp.gate(gate), sp.w(w_pre)};
  const Span out[2] = {sp.h(h_out), sp.x(x_out)};
  const int same[2] = {0, -1};  // h_out may be h
  if (any_overlap(in, 5, out, 2, same)) return MOE_EINVAL;
  if (check_only) return MOE_OK;
  a.h = static_cast<const uint8_t*>(h);
  a.y = static_cast<const uint8_t*>(y);
  a.w_post = w_post;
  a.gate = gate;
  a.w_pre = w_pre;
  a.h_out = static_cast<uint8_t*>(h_out);
  a.x_out = static_cast<uint8_t*>(x_out);
  s = stream_of(s);
  const StreamDevice on(s);
  return launch_norm<false>(*cfg, a, cfg->T, s);
}

moe_status rmoe::block_step_check(const moe_norm_config* cfg, const void* x, int afmt, const void* h, const float* y,
                                  const float* w_post, const float* gate, const float* w_pre, const void* x_next,
                                  const Region* other, int n) {
  NormArgs a{};
  if (!y || block_norm(cfg, h, y, w_post, gate, w_pre, const_cast<void*>(h), const_cast<void*>(x_next), nullptr, true) != MOE_OK ||
      !norm_config_ok(cfg, &a))
    return MOE_EINVAL;
  const NormSpans sp{*cfg, a};
  const Span step_x = {x, cfg->T, cfg->H * fmt_bytes(afmt), cfg->H * fmt_bytes(afmt)}, step_y = sp.y(y);
  if (overlap(step_y, sp.w(w_post)) || overlap(step_y, sp.gate(gate)) || overlap(step_y, sp.w(w_pre))) return MOE_EINVAL;
  const Span out[2] = {sp.h(h), sp.x(x_next)};
  const int fmt[2] = {cfg->h_fmt, cfg->x_fmt};
  for (int o = 0; o < 2; ++o) {
    const bool is_x = out[o].p == x && fmt[o] == afmt && (cfg->T == 1 || out[o].pitch == step_x.pitch);
    if (!is_x && overlap(out[o], step_x)) return MOE_EINVAL;
    for (int i = 0; i < n; ++i)
      if (overlap(out[o], flat(other[i].p, other[i].bytes))) return MOE_EINVAL;
  }
  return MOE_OK;
}

extern "C" MOE_API moe_status moe_block_norm(const moe_norm_config* cfg, const void* h, const void* y,
                                             const float* w_post, const float* gate, const float* w_pre, void* h_out,
                                             void* x_out, moe_stream_t stream) {
  return block_norm(cfg, h, y, w_post, gate, w_pre, h_out, x_out, static_cast<hipStream_t>(stream), false);
}

extern "C" MOE_API int64_t moe_block_norm_workspace(int32_t T, int32_t H) {
  if (T < 1 || T > kNormMaxT || H < 1 || H > kNormMaxH) return -1;
  return 2ll * norm_groups(T, H) * H * 4;
}

extern "C" MOE_API moe_status moe_block_norm_backward(const moe_norm_config* cfg, const void* h_out, const void* y,
                                                      const float* w_post, const float* gate, const float* w_pre,
                                                      const void* dh_out, const void* dx, void* dh, void* dy,
                                                      float* dw_post, float* dgate, float* dw_pre, void* ws,
                                                      size_t ws_bytes, moe_stream_t stream) {
  NormArgs a{};
  if (!norm_config_ok(cfg, &a)) return MOE_EINVAL;
  if (!dh_out && !dx) return MOE_EINVAL;                                // no gradient comes in
  if (!dh && !dy && !dw_post && !dgate && !dw_pre) return MOE_EINVAL;   // none is asked for
  if (dx ? (!h_out || !w_pre) : (w_pre || dw_pre)) return MOE_EINVAL;
  if (!y && (dy || w_post || gate || dgate)) return MOE_EINVAL;
  if (dw_post && !w_post) return MOE_EINVAL;
  if ((gate != nullptr) != (cfg->gate_kind != MOE_GATE_NONE) || (dgate && !gate)) return MOE_EINVAL;
  const bool partial = dw_pre || dw_post || (dgate && cfg->gate_kind == MOE_GATE_CHANNEL);
  const int64_t need = partial ? moe_block_norm_workspace(cfg->T, cfg->H) : 0;
  if (need && (!ws || ws_bytes < (size_t)need || !aligned_to(ws, 4))) return MOE_EINVAL;
  const int64_t hb = fmt_bytes(cfg->h_fmt), yb = fmt_bytes(cfg->y_fmt), xb = fmt_bytes(cfg->x_fmt);
  if (!aligned_to(h_out, hb) || !aligned_to(y, yb) || !aligned_to(dh_out, hb) || !aligned_to(dx, xb) ||
      !aligned_to(dh, hb) || !aligned_to(dy, yb) || !aligned_to(w_post, 4) || !aligned_to(gate, 4) ||
      !aligned_to(w_pre, 4) || !aligned_to(dw_post, 4) || !aligned_to(dgate, 4) || !aligned_to(dw_pre, 4))
    return MOE_EINVAL;
  const NormSpans sp{*cfg, a};
  const Span in[7] = {sp.h(h_out), sp.y(y), sp.w(w_post), sp.gate(gate), sp.w(w_pre), sp.h(dh_out), sp.x(dx)};
  const Span out[6] = {sp.h(dh), sp.y(dy), sp.w(dw_post), sp.gate(dgate), sp.w(dw_pre), flat(need ? ws : nullptr, need)};
  const int same[6] = {5, 1, -1, -1, -1, -1};  // dh may be dh_out, dy may be y
  if (any_overlap(in, 7, out, 6, same)) return MOE_EINVAL;
  a.h = static_cast<const uint8_t*>(h_out);
  a.y = static_cast<const uint8_t*>(y);
  a.w_post = w_post;
  a.gate = gate;
  a.w_pre = w_pre;
  a.dh_in = static_cast<const uint8_t*>(dh_out);
  a.dx = static_cast<const uint8_t*>(dx);
  a.dh = static_cast<uint8_t*>(dh);
  a.dy = static_cast<uint8_t*>(dy);
  a.dgate_token = cfg->gate_kind == MOE_GATE_TOKEN ? dgate : nullptr;
  a.part = static_cast<float*>(ws);
  // the kinds of partial sums and where each goes: dx h' r to dw_pre, alpha dh y ry to dw_post
  // (by the channel gate) and the channel gate's gradient (by w_post)
  NormOut out_w{};
  int kinds = 0;
  a.part_pre = a.part_post = -1;
  if (dw_pre) {
    out_w.p[kinds][0] = dw_pre;
    a.part_pre = kinds++;
  }
  float* const dgate_c = cfg->gate_kind == MOE_GATE_CHANNEL ? dgate : nullptr;
  if (dw_post || dgate_c) {
    out_w.p[kinds][0] = dw_post;
    out_w.by[kinds][0] = cfg->gate_kind == MOE_GATE_CHANNEL ? gate : nullptr;
    out_w.p[kinds][1] = dgate_c;
    out_w.by[kinds][1] = w_post;
    a.part_post = kinds++;
  }
  const hipStream_t s = stream_of(stream);
  const StreamDevice on(s);
  const int G = partial ? norm_groups(cfg->T, cfg->H) : cfg->T;
  const moe_status st = launch_norm<true>(*cfg, a, G, s);
  if (st != MOE_OK || !partial) return st;
  return launch(norm_reduce, dim3((cfg->H + 31) / 32, kinds), dim3(1024), s, static_cast<const float*>(ws), G,
                (int)cfg->H, out_w);
}
