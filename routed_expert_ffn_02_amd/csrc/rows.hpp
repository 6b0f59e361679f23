// Rows of activations in chunks of N elements per lane, for the operators around the
// experts (tokens.hip, norm.hip): loads and stores at any element alignment, fp32 values
// in registers, and the host helpers their entry points share.
#pragma once

#include <tuple>

#include "common.hpp"

namespace rmoe {

// 16, 8 and 4 bytes at an address that is only element-aligned.  Code objects for the HSA
// runtime run with unaligned access on, so each is one global load or store whatever the
// address: a row of odd length needs no path of its own, only its last chunk does.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));

template <int FMT>
constexpr int kElemBytes = FMT == MOE_AFMT_BF16 ? 2 : 4;

// Two fp32 values rounded to bf16 (nearest even, NaN kept), the first in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, bf16x2));
}

// N elements of a row, as stored (N = 8, or 4 for fp32 alone).
template <int FMT, int N>
struct Chunk {
  static constexpr int kWords = N * kElemBytes<FMT> / 4;
  uint32_t q[kWords];

  // The first n elements at p; all of them when n >= N, zeros behind them.
  __device__ __forceinline__ void load(const uint8_t* p, int n) {
    if (n >= N) {
      if constexpr (kWords == 2) {
        const u32x2 v = *reinterpret_cast<const u32x2_any*>(p);
        q[0] = v[0];
        q[1] = v[1];
      } else {
#pragma unroll
        for (int i = 0; i < kWords; i += 4) {
          const u32x4 v = *reinterpret_cast<const u32x4_any*>(p + 4 * i);
          q[i] = v[0];
          q[i + 1] = v[1];
          q[i + 2] = v[2];
          q[i + 3] = v[3];
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        q[i] = 0;
        if constexpr (FMT == MOE_AFMT_BF16) {
          if (2 * i < n) q[i] = reinterpret_cast<const uint16_t*>(p)[2 * i];
          if (2 * i + 1 < n) q[i] |= (uint32_t) reinterpret_cast<const uint16_t*>(p)[2 * i + 1] << 16;
        } else {
          if (i < n) q[i] = reinterpret_cast<const uint32_t*>(p)[i];
        }
      }
    }
  }

  __device__ __forceinline__ void store(uint8_t* p, int n) const {
    if (n >= N) {
      if constexpr (kWords == 2) {
        *reinterpret_cast<u32x2_any*>(p) = (u32x2){q[0], q[1]};
      } else {
#pragma unroll
        for (int i = 0; i < kWords; i += 4)
          *reinterpret_cast<u32x4_any*>(p + 4 * i) = (u32x4){q[i], q[i + 1], q[i + 2], q[i + 3]};
      }
    } else {
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        if constexpr (FMT == MOE_AFMT_BF16) {
          if (2 * i < n) reinterpret_cast<uint16_t*>(p)[2 * i] = (uint16_t)q[i];
          if (2 * i + 1 < n) reinterpret_cast<uint16_t*>(p)[2 * i + 1] = (uint16_t)(q[i] >> 16);
        } else {
          if (i < n) reinterpret_cast<uint32_t*>(p)[i] = q[i];
        }
      }
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

// The device of `stream` made current for a launch and the caller's restored after it: a
// stream of another device than the current one gets its kernels on its own device.
class StreamDevice {
 public:
  explicit StreamDevice(hipStream_t s) {
    hipDevice_t dev = -1;
    if (s == nullptr || hipStreamGetDevice(s, &dev) != hipSuccess) return;
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
