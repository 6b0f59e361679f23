// Rows of activations in chunks of N elements per lane, for the operators around the
// experts (tokens.hip, norm.hip): loads and stores at any element alignment, fp32 values
// in registers, and the host helpers their entry points share.
#pragma once

#include <tuple>

#include "common.hpp"

namespace rmoe {

// 16 or 8 bytes at an address that is only element-aligned.  Code objects for the HSA
// runtime run with unaligned access on, so each is one global load or store whatever the
// address: a row of odd length needs no path of its own, only its last chunk does.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));

// NT: the non-temporal form.  A template parameter, since the two forms of one access under a
// runtime condition are merged into the ordinary one.
template <bool NT>
__device__ __forceinline__ u32x4 load16(const uint8_t* p) {
  if constexpr (NT) return __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(p));
  else return *reinterpret_cast<const u32x4_any*>(p);
}
template <bool NT>
__device__ __forceinline__ u32x2 load8(const uint8_t* p) {
  if constexpr (NT) return __builtin_nontemporal_load(reinterpret_cast<const u32x2_any*>(p));
  else return *reinterpret_cast<const u32x2_any*>(p);
}
template <bool NT>
__device__ __forceinline__ void store16(uint8_t* p, u32x4 v) {
  if constexpr (NT) __builtin_nontemporal_store(v, reinterpret_cast<u32x4_any*>(p));
  else *reinterpret_cast<u32x4_any*>(p) = v;
}
template <bool NT>
__device__ __forceinline__ void store8(uint8_t* p, u32x2 v) {
  if constexpr (NT) __builtin_nontemporal_store(v, reinterpret_cast<u32x2_any*>(p));
  else *reinterpret_cast<u32x2_any*>(p) = v;
}

template <int FMT>
constexpr int kElemBytes = FMT == MOE_AFMT_BF16 ? 2 : 4;

// Two fp32 values rounded to bf16 (nearest even, NaN kept), the first in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, bf16x2));
}

// A lane's N elements of a row of H.  Chunk c starts at element c * N; the last one of a row whose
// length N does not divide moves back to end with the row, so that it too is one vector
// access, and shares its first `skip` elements with the chunk before.  Moves compute and
// store the shared ones twice, the same values; sums and writes in place leave them out.
// Rows shorter than N (n = H < N) are read and written element by element.
template <int N>
struct Piece {
  int i, skip, n;  // first element, elements another chunk has, elements of the access
  bool on;         // the chunk lies in the row
  __device__ __forceinline__ Piece(int c, int H) {
    on = c * N < H;
    n = min(N, H);
    i = on ? min(c * N, H - n) : 0;
    skip = on ? c * N - i : 0;
  }
};

// N elements of a row, as stored (N = 8, or 4 for fp32 alone).
template <int FMT, int N>
struct Chunk {
  static constexpr int kWords = N * kElemBytes<FMT> / 4;
  static_assert(kWords == 2 || kWords % 4 == 0, "whole 8- or 16-byte accesses");
  uint32_t q[kWords];

  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) q[i] = 0;
  }

  // N elements at p.
  __device__ __forceinline__ void load_at(const uint8_t* p) {
    static_assert(kWords % 4 == 0, "16-byte accesses");
#pragma unroll
    for (int i = 0; i < kWords; i += 4) {
      const u32x4 v = load16<false>(p + 4 * i);
      q[i] = v[0];
      q[i + 1] = v[1];
      q[i + 2] = v[2];
      q[i + 3] = v[3];
    }
  }
  // Zeros for the first `skip` elements, without a branch.
  __device__ __forceinline__ void keep_from(int skip) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (FMT == MOE_AFMT_BF16) q[i] &= (2 * i >= skip ? 0xffffu : 0u) | (2 * i + 1 >= skip ? 0xffff0000u : 0u);
      else q[i] = i >= skip ? q[i] : 0;
    }
  }

  // The piece at its place in `row` (which must be on).  NT: a non-temporal load.
  template <bool NT = false>
  __device__ __forceinline__ void load(const uint8_t* row, const Piece<N>& s) {
    const uint8_t* p = row + (int64_t)s.i * kElemBytes<FMT>;
    if (s.n == N) {
      if constexpr (kWords == 2) {
        const u32x2 v = load8<NT>(p);
        q[0] = v[0];
        q[1] = v[1];
      } else {
#pragma unroll
        for (int i = 0; i < kWords; i += 4) {
          const u32x4 v = load16<NT>(p + 4 * i);
          q[i] = v[0];
          q[i + 1] = v[1];
          q[i + 2] = v[2];
          q[i + 3] = v[3];
        }
      }
    } else {
      zero();
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (i >= s.n) continue;
        if constexpr (FMT == MOE_AFMT_BF16) q[i / 2] |= (uint32_t) reinterpret_cast<const uint16_t*>(p)[i] << 16 * (i & 1);
        else q[i] = reinterpret_cast<const uint32_t*>(p)[i];
      }
    }
  }

  // The same for sums: zeros outside the row and for the shared elements.
  template <bool NT = false>
  __device__ __forceinline__ void load_own(const uint8_t* row, const Piece<N>& s) {
    if (!s.on) {
      zero();
      return;
    }
    load<NT>(row, s);
    if (s.skip) drop(s.skip);
  }
  __device__ __forceinline__ void drop(int skip) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < skip) {
        if constexpr (FMT == MOE_AFMT_BF16) q[i / 2] &= (i & 1) ? 0xffffu : 0xffff0000u;
        else q[i] = 0;
      }
  }

  template <bool NT = false>
  __device__ __forceinline__ void store(uint8_t* row, const Piece<N>& s) const {
    uint8_t* p = row + (int64_t)s.i * kElemBytes<FMT>;
    if (s.n == N) {
      if constexpr (kWords == 2) {
        store8<NT>(p, (u32x2){q[0], q[1]});
      } else {
#pragma unroll
        for (int i = 0; i < kWords; i += 4) store16<NT>(p + 4 * i, (u32x4){q[i], q[i + 1], q[i + 2], q[i + 3]});
      }
    } else {
      elements(p, 0, s.n);
    }
  }

  // The same by a wavefront whose lanes hold neighbouring chunks of a row of H.  Eight fp32
  // values are two stores per lane, 16 bytes out of every 32 each, which go out of the caches
  // as partial lines (13% more bytes written by the move's gradient at 1531 rows of 4096): lanes
  // l and l + 32 exchange a half first, and each store covers 1 KB without a gap.
  template <bool NT = false>
  __device__ __forceinline__ void store_wave(uint8_t* row, const Piece<N>& s, int H) {
    if constexpr (FMT == MOE_AFMT_F32 && N == 8) {
      const int i0 = __builtin_amdgcn_readfirstlane(s.i), lane = threadIdx.x & 63;
      if (i0 + 64 * N <= H) {  // every lane has a whole chunk of its own
        u32x4 a, b;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const auto v = __builtin_amdgcn_permlane32_swap(q[i], q[4 + i], false, false);
          a[i] = v[0];
          b[i] = v[1];
        }
        uint8_t* p = row + 4ll * (i0 + 8 * (lane & 31) + 4 * (lane >> 5));
        store16<NT>(p, a);
        store16<NT>(p + 1024, b);
        return;
      }
    }
    store_own<NT>(row, s);
  }

  // The same without the shared elements.
  template <bool NT = false>
  __device__ __forceinline__ void store_own(uint8_t* row, const Piece<N>& s) const {
    if (!s.on) return;
    if (s.skip) elements(row + (int64_t)s.i * kElemBytes<FMT>, s.skip, N);
    else store<NT>(row, s);
  }
  __device__ __forceinline__ void elements(uint8_t* p, int from, int to) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i < from || i >= to) continue;
      if constexpr (FMT == MOE_AFMT_BF16) reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)(q[i / 2] >> 16 * (i & 1));
      else reinterpret_cast<uint32_t*>(p)[i] = q[i];
    }
  }

  __device__ __forceinline__ float get(int i) const {
    if constexpr (FMT == MOE_AFMT_BF16) return (i & 1) ? bf16_hi(q[i / 2]) : bf16_lo(q[i / 2]);
    else return __uint_as_float(q[i]);
  }

  __device__ __forceinline__ void set(const float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (FMT == MOE_AFMT_BF16) q[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
      else q[i] = __float_as_uint(v[i]);
    }
  }
};

// ---------------------------------------------------------------- host side
// Whether sorted rows of this many bytes pass by the caches (non-temporal loads where they
// are read, stores where they are written): half of the 256 MB last-level cache and more.  What
// it costs and gains, in us with ordinary / non-temporal accesses, k = 8 rows of 2048 in bf16:
//                                     48 MB         64 MB         96 MB         128 MB        192 MB
//   rows from memory: dispatch        16.1 / 16.2   19.8 / 20.2   30.6 / 28.1   39.7 / 34.8   53.1 / 47.9
//     combine                         10.9 / 11.7   14.2 / 15.3   24.4 / 22.1   32.0 / 29.4   46.6 / 43.1
//     its gradient                    19.1 / 21.8   33.1 / 31.4   48.0 / 44.8   63.7 / 58.4   93.7 / 84.9
//   rows written, then combine        26.2 / 26.2   34.6 / 33.8   53.5 / 51.3   69.8 / 65.6   103 / 101
//   dispatch, then its rows read      31.1 / 33.4   39.8 / 42.1   58.0 / 65.6   78.8 / 84.6   118 / 121
//   combine, then its gradient        30.3 / 33.7   41.6 / 48.0   57.7 / 70.7   77.9 / 90.8   116 / 136
// (4 rows of 1000 in bf16 and 6 of 4096 in fp32 cross over at the same sizes but for combine, which is
// even there from 96 MB on.)  Rows from memory gain from about 80 MB on; rows that the next
// kernel takes from the cache lose up to 256 MB, most around 128.  The call does not know which it is:
// the rule stands between the two.
inline bool stream_rows(int64_t bytes) { return bytes >= (128ll << 20); }

constexpr int64_t kMaxStride = 1ll << 36;  // elements between rows: byte offsets of 2^21 rows stay in 64 bits
inline bool fmt_ok(int fmt) { return fmt == MOE_AFMT_F32 || fmt == MOE_AFMT_BF16; }
inline int64_t fmt_bytes(int fmt) { return fmt == MOE_AFMT_BF16 ? 2 : 4; }
inline bool aligned_to(const void* p, int64_t a) { return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(a - 1)) == 0; }

// A block of memory: `rows` rows of `width` bytes, `pitch` bytes apart.
struct Span {
  const void* p;
  int64_t rows, width, pitch;
};
inline Span flat(const void* p, int64_t bytes) { return {p, 1, bytes, bytes}; }

// Whether two blocks share a byte (a null one shares none).  Blocks of one pitch that lie
// side by side in the same rows do not; of two pitches in one range, they count as sharing.
inline bool overlap(const Span& a, const Span& b) {
  if (!a.p || !b.p || !a.rows || !b.rows) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  const uintptr_t a1 = a0 + (uintptr_t)((a.rows - 1) * a.pitch + a.width);
  const uintptr_t b1 = b0 + (uintptr_t)((b.rows - 1) * b.pitch + b.width);
  if (a1 <= b0 || b1 <= a0) return false;
  if (a.pitch != b.pitch) return true;
  const int64_t d = a0 <= b0 ? (int64_t)((b0 - a0) % (uintptr_t)a.pitch)
                             : (a.pitch - (int64_t)((a0 - b0) % (uintptr_t)a.pitch)) % a.pitch;
  return d < a.width || a.pitch - d < b.width;
}

// A caller's stream as it is handed on.  The handles that HIP reserves are no stream objects: the
// legacy default stream's is the null stream's other name, and asking either it or the thread's own
// for its device is left out: they belong to the current one, and hipStreamGetDevice of such a handle
// has ended the process with a segmentation fault.
inline hipStream_t stream_of(moe_stream_t stream) {
  return stream == hipStreamLegacy ? nullptr : static_cast<hipStream_t>(stream);
}

// The device of `stream` made current for a launch and the caller's restored after it: a
// stream of another device than the current one gets its kernels on its own device.
class StreamDevice {
 public:
  explicit StreamDevice(hipStream_t s) {
    hipDevice_t dev = -1;
    if (s == nullptr || s == hipStreamPerThread || hipStreamGetDevice(s, &dev) != hipSuccess) return;
    if (hipGetDevice(&before_) != hipSuccess || before_ == dev) {
      before_ = -1;
      return;
    }
    (void)hipSetDevice(dev);
  }
  ~StreamDevice() {
    if (before_ >= 0) (void)hipSetDevice(before_);
  }
  StreamDevice(const StreamDevice&) = delete;
  StreamDevice& operator=(const StreamDevice&) = delete;

 private:
  int before_ = -1;
};

// Launch with the launch's own status, so that an error another call left is not taken for
// this one's.
template <typename... KArgs, typename... Args>
inline moe_status launch(void (*kernel)(KArgs...), dim3 grid, dim3 block, hipStream_t s, Args... args) {
  std::tuple<KArgs...> vals(args...);
  void* ptrs[sizeof...(KArgs)];
  std::apply([&](auto&... v) { int i = 0; ((ptrs[i++] = (void*)&v), ...); }, vals);
  if (hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, block, ptrs, 0, s) == hipSuccess) return MOE_OK;
  (void)hipGetLastError();
  return MOE_EHIP;
}

}  // namespace rmoe
