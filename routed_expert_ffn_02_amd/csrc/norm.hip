// The norms before and after a block, fused with the block's gate and residual scale:
//   u  = w_post * y / rms(y)      (w_post = nullptr: u = y)
//   h' = h + alpha * g * u        (g: none, one per token, or one per channel)
//   x  = w_pre * h' / rms(h')     rms(v) = sqrt(mean(v^2) + eps)
// and its gradient.  Memory-bound: a row is read once, kept in registers across its
// reductions, and written once.  Statistics and all arithmetic are fp32; x is formed from
// h' before h' is rounded to its own type, so each output is rounded once.
#include <algorithm>

#include "rows.hpp"

namespace rmoe {

constexpr int kNormMaxH = kDecodeMaxTH;  // a row fits one workgroup's registers
constexpr int kNormMaxT = 1 << 22;
constexpr int kNormN = 8;                // elements of a lane's chunk
constexpr int kNormMaxWaves = 16;

struct NormArgs {
  int T, H, gate_kind;
  int64_t h_pitch, y_pitch, x_pitch;  // bytes between rows
  float alpha, eps;
  const uint8_t *h, *y;
  const float *w_post, *gate, *w_pre;
  uint8_t *h_out, *x_out;             // forward
  const uint8_t *dh_in, *dx;          // backward
  uint8_t *dh, *dy;
  float* dgate_token;                 // [T]
  float* part;                        // partial sums of the weights' gradients [kinds][G][H]
  int part_pre, part_post, part_gate; // index of each kind in part, or -1
};

// The sum over the workgroup's wavefronts of NV values per thread, in wavefront order.
template <int NV>
__device__ __forceinline__ void block_sum(float (&v)[NV], float (*s_red)[NV]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, nw = blockDim.x >> 6;
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = wave_sum(v[i]);
  if (nw == 1) return;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) s_red[wave][i] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    v[i] = 0.f;
    for (int w = 0; w < nw; ++w) v[i] += s_red[w][i];
  }
}

// fp32 weights of a chunk, 1 where there are none.
__device__ __forceinline__ void load_w(const float* w, const Piece<kNormN>& at, float (&v)[kNormN]) {
  Chunk<MOE_AFMT_F32, kNormN> q;
  if (w && at.on) q.load(reinterpret_cast<const uint8_t*>(w), at);
#pragma unroll
  for (int n = 0; n < kNormN; ++n) v[n] = w && at.on ? q.get(n) : 1.f;
}

// One workgroup per row, C chunks of 8 elements per thread.  h_out may be h: a thread writes
// only elements that it alone has read for sums and sums, and no other thread's reads of
// them count.
template <int HF, int YF, int XF, int C>
__global__ __launch_bounds__(64 * kNormMaxWaves) void block_norm_kernel(NormArgs a) {
  constexpr int N = kNormN;
  __shared__ float s_y[kNormMaxWaves][1], s_h[kNormMaxWaves][1];
  const int64_t t = blockIdx.x;
  const int H = a.H;
  Chunk<HF, N> qh[C];
  Chunk<YF, N> qy[C];
  float wq[C][N], g[C][N], wp[C][N];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const Piece<N> at(threadIdx.x + c * blockDim.x, H);
    if (a.y) qy[c].load_own(a.y + t * a.y_pitch, at);
    qh[c].load_own(a.h + t * a.h_pitch, at);
    load_w(a.w_post, at, wq[c]);
    load_w(a.gate_kind == MOE_GATE_CHANNEL ? a.gate : nullptr, at, g[c]);
    load_w(a.w_pre, at, wp[c]);
  }
  float h[C][N];
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int n = 0; n < N; ++n) h[c][n] = qh[c].get(n);
  if (a.y) {
    float scale = a.alpha;
    if (a.gate_kind == MOE_GATE_TOKEN) scale *= a.gate[t];
    if (a.w_post) {
      float s[1] = {0.f};
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int n = 0; n < N; ++n) s[0] = fmaf(qy[c].get(n), qy[c].get(n), s[0]);
      block_sum(s, s_y);
      scale *= 1.f / sqrtf(s[0] / H + a.eps);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const Piece<N> at(threadIdx.x + c * blockDim.x, H);
#pragma unroll
      for (int n = 0; n < N; ++n) h[c][n] = fmaf(scale * qy[c].get(n), wq[c][n] * g[c][n], h[c][n]);
      Chunk<HF, N> o;
      o.set(h[c]);
      o.template store_own<true>(a.h_out + t * a.h_pitch, at);
    }
  }
  if (!a.x_out) return;
  float s[1] = {0.f};
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int n = 0; n < N; ++n) s[0] = fmaf(h[c][n], h[c][n], s[0]);
  block_sum(s, s_h);
  const float r = 1.f / sqrtf(s[0] / H + a.eps);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const Piece<N> at(threadIdx.x + c * blockDim.x, H);
#pragma unroll
    for (int n = 0; n < N; ++n) wp[c][n] = h[c][n] * r * wp[c][n];
    Chunk<XF, N> o;
    o.set(wp[c]);
    o.template store_own<true>(a.x_out + t * a.x_pitch, at);
  }
}

// The rows of one token in the gradient, as stored; zeros for a gradient that does not come in.
template <int HF, int YF, int XF, int C>
struct NormRows {
  Chunk<HF, kNormN> h[C], d[C];
  Chunk<YF, kNormN> y[C];
  Chunk<XF, kNormN> x[C];
  __device__ __forceinline__ void load(const NormArgs& a, int64_t t) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const Piece<kNormN> at(threadIdx.x + c * blockDim.x, a.H);
      h[c].zero();
      x[c].zero();
      d[c].zero();
      y[c].zero();
      if (a.dx) {
        h[c].load_own(a.h + t * a.h_pitch, at);
        x[c].load_own(a.dx + t * a.x_pitch, at);
      }
      if (a.dh_in) d[c].load_own(a.dh_in + t * a.h_pitch, at);
      if (a.y) y[c].load_own(a.y + t * a.y_pitch, at);
    }
  }
};

// The gradient.  With r = 1 / rms(h'), d = w_pre dx, ry = 1 / rms(y), D = sum(dh' g_c w_post y):
//   dh = dh' + r (d - h' r^2 mean(d h'))          (dh' from the stream behind the block)
//   du = alpha g dh,  dy = ry (w_post du - y ry^2 mean(w_post du y))
//   dw_pre = sum_t dx h' r,  dw_post = sum_t du y ry,  dgate = alpha sum dh u
// A workgroup walks rows b, b + G, ...; its threads keep the weights' gradients of their
// own channels in registers over those rows and write one partial row at the end, which
// norm_reduce adds in workgroup order: no atomics, the same bits every time.  AHEAD: the
// next row is loaded before the current one's sums.
template <int HF, int YF, int XF, int C, int WAVES, bool AHEAD>
__global__ __launch_bounds__(64 * WAVES) void block_norm_backward_kernel(NormArgs a) {
  constexpr int N = kNormN;
  __shared__ float s_a[WAVES][3], s_b[WAVES][1];
  const int H = a.H;
  float wp[C][N], wq[C][N], gc[C][N], acc_pre[C][N], acc_post[C][N], acc_gate[C][N];
  NormRows<HF, YF, XF, C> next;
  if (AHEAD) next.load(a, blockIdx.x);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const Piece<N> at(threadIdx.x + c * blockDim.x, H);
    load_w(a.w_pre, at, wp[c]);
    load_w(a.w_post, at, wq[c]);
    load_w(a.gate_kind == MOE_GATE_CHANNEL ? a.gate : nullptr, at, gc[c]);
#pragma unroll
    for (int n = 0; n < N; ++n) acc_pre[c][n] = acc_post[c][n] = acc_gate[c][n] = 0.f;
  }
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    NormRows<HF, YF, XF, C> q;
    if (AHEAD) {
      q = next;
      if (t + gridDim.x < a.T) next.load(a, t + gridDim.x);
    } else {
      q.load(a, t);
    }
    float s[3] = {0.f, 0.f, 0.f};  // sums of h'^2, d h', y^2
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const float hv = q.h[c].get(n), yv = q.y[c].get(n);
        s[0] = fmaf(hv, hv, s[0]);
        s[1] = fmaf(wp[c][n] * q.x[c].get(n), hv, s[1]);
        s[2] = fmaf(yv, yv, s[2]);
      }
    block_sum(s, s_a);
    const float r = 1.f / sqrtf(s[0] / H + a.eps), hm = r * r * (s[1] / H);
    const float ry = a.w_post ? 1.f / sqrtf(s[2] / H + a.eps) : 1.f;
    float dh[C][N], dot[1] = {0.f};
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const float hv = q.h[c].get(n), xv = q.x[c].get(n);
        dh[c][n] = fmaf(r, wp[c][n] * xv - hv * hm, q.d[c].get(n));
        acc_pre[c][n] = fmaf(xv, hv * r, acc_pre[c][n]);
        dot[0] = fmaf(dh[c][n] * gc[c][n] * wq[c][n], q.y[c].get(n), dot[0]);
      }
      if (a.dh) {
        Chunk<HF, N> o;
        o.set(dh[c]);
        o.template store_own<true>(a.dh + t * a.h_pitch, Piece<N>(threadIdx.x + c * blockDim.x, H));
      }
    }
    if (!a.y) continue;
    block_sum(dot, s_b);
    const float gt = a.gate_kind == MOE_GATE_TOKEN ? a.gate[t] : 1.f, ag = a.alpha * gt;
    const float ym = a.w_post ? ag * ry * ry * (dot[0] / H) : 0.f;
    if (a.dgate_token && threadIdx.x == 0) a.dgate_token[t] = a.alpha * ry * dot[0];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float v[N];
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const float yv = q.y[c].get(n), du = ag * gc[c][n] * dh[c][n], yr = yv * ry;
        v[n] = ry * (wq[c][n] * du - yv * ym);
        acc_post[c][n] = fmaf(du, yr, acc_post[c][n]);
        acc_gate[c][n] = fmaf(a.alpha * dh[c][n], wq[c][n] * yr, acc_gate[c][n]);
      }
      if (a.dy) {
        Chunk<YF, N> o;
        o.set(v);
        o.template store_own<true>(a.dy + t * a.y_pitch, Piece<N>(threadIdx.x + c * blockDim.x, H));
      }
    }
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const Piece<N> at(threadIdx.x + c * blockDim.x, H);
    const auto put = [&](int kind, const float(&v)[N]) {
      if (kind < 0) return;
      Chunk<MOE_AFMT_F32, N> o;
      o.set(v);
      o.store_own(reinterpret_cast<uint8_t*>(a.part + ((int64_t)kind * gridDim.x + blockIdx.x) * H), at);
    };
    put(a.part_pre, acc_pre[c]);
    put(a.part_post, acc_post[c]);
    put(a.part_gate, acc_gate[c]);
  }
}

// out[kind][i] = sum over g of part[kind][g][i]: 64 channels per workgroup, its wavefronts
// take rows w, w + 16, ... and are added in order.
struct NormOut {
  float* p[3];
};
__global__ __launch_bounds__(1024) void norm_reduce(const float* __restrict__ part, int G, int H, NormOut out) {
  __shared__ float s_v[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = blockIdx.x * 64 + lane;
  const float* p = part + (int64_t)blockIdx.y * G * H;
  float v = 0.f;
  if (i < H) {
#pragma unroll 16
    for (int g = wave; g < G; g += 16) v += p[(int64_t)g * H + i];
  }
  s_v[wave][lane] = v;
  __syncthreads();
  if (wave != 0 || i >= H) return;
  v = 0.f;
  for (int w = 0; w < 16; ++w) v += s_v[w][lane];
  out.p[blockIdx.y][i] = v;
}

namespace {

int norm_waves(int H) { return std::min(kNormMaxWaves, (H + 64 * kNormN - 1) / (64 * kNormN)); }

// Workgroups of the gradient kernel when weights' gradients are wanted: one per CU, so that
// the partial rows stay small beside the rows themselves.
constexpr int kNormGroups = 256;
int norm_groups(int T) { return std::min(T, kNormGroups); }

template <bool BACK, int HF, int YF, int XF>
moe_status launch_norm_f(const NormArgs& a, int groups, hipStream_t s) {
  const int waves = norm_waves(a.H);
  const dim3 grid(groups), block(64 * waves);
  const bool two = a.H > 64 * kNormMaxWaves * kNormN;
  if constexpr (BACK) {
    if (two) return launch(block_norm_backward_kernel<HF, YF, XF, 2, kNormMaxWaves, false>, grid, block, s, a);
    if (waves > 8) return launch(block_norm_backward_kernel<HF, YF, XF, 1, kNormMaxWaves, false>, grid, block, s, a);
    return launch(block_norm_backward_kernel<HF, YF, XF, 1, 8, true>, grid, block, s, a);
  } else {
    if (two) return launch(block_norm_kernel<HF, YF, XF, 2>, grid, block, s, a);
    return launch(block_norm_kernel<HF, YF, XF, 1>, grid, block, s, a);
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
  if (!(c->eps > 0.f) || !(c->eps <= 1.f) || !(c->alpha - c->alpha == 0.f)) return false;
  const int64_t ld[3] = {c->ld_h ? c->ld_h : c->H, c->ld_y ? c->ld_y : c->H, c->ld_x ? c->ld_x : c->H};
  for (int64_t v : ld)
    if (v < c->H || v > (1ll << 40)) return false;
  a->T = c->T;
  a->H = c->H;
  a->gate_kind = c->gate_kind;
  a->alpha = c->alpha;
  a->eps = c->eps;
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
  const StreamDevice on(s);
  return launch_norm<false>(*cfg, a, cfg->T, s);
}

extern "C" MOE_API moe_status moe_block_norm(const moe_norm_config* cfg, const void* h, const void* y,
                                             const float* w_post, const float* gate, const float* w_pre, void* h_out,
                                             void* x_out, moe_stream_t stream) {
  return block_norm(cfg, h, y, w_post, gate, w_pre, h_out, x_out, static_cast<hipStream_t>(stream), false);
}

extern "C" MOE_API int64_t moe_block_norm_workspace(int32_t T, int32_t H) {
  if (T < 1 || T > kNormMaxT || H < 1 || H > kNormMaxH) return -1;
  return 3ll * norm_groups(T) * H * 4;
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
  NormOut out_w{};
  int kinds = 0;
  const auto want = [&](float* p) {
    if (!p) return -1;
    out_w.p[kinds] = p;
    return kinds++;
  };
  a.part_pre = want(dw_pre);
  a.part_post = want(dw_post);
  a.part_gate = want(cfg->gate_kind == MOE_GATE_CHANNEL ? dgate : nullptr);
  hipStream_t s = static_cast<hipStream_t>(stream);
  const StreamDevice on(s);
  const int G = partial ? norm_groups(cfg->T) : cfg->T;
  const moe_status st = launch_norm<true>(*cfg, a, G, s);
  if (st != MOE_OK || !partial) return st;
  return launch(norm_reduce, dim3((cfg->H + 63) / 64, kinds), dim3(1024), s, static_cast<const float*>(ws), G,
                (int)cfg->H, out_w);
}
