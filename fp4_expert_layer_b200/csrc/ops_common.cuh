// ops_common.cuh -- what the stand-alone operators (moe_ops.h) share: argument
// checks, launch helpers, and 16-bit / 32-bit element access.
#pragma once

#include <algorithm>
#include <atomic>
#include <string>

#include "device_utils.cuh"
#include "launch.cuh"
#include "moe_internal.h"
#include "moe_ops.h"

namespace moe {

const char *set_error_text(const std::string &s);   // defined in api.cu

inline moe_status_t ops_fail(moe_status_t st, const char *fn, const std::string &what) {
  set_error_text(std::string(fn) + ": " + what);
  return st;
}
inline moe_status_t ops_invalid(const char *fn, const std::string &what) {
  return ops_fail(MOE_ERR_INVALID_ARG, fn, what);
}
// The status of the launches just made.  A launch error is not sticky.
inline moe_status_t ops_launched(const char *fn, cudaError_t e) {
  if (e == cudaSuccess) e = cudaGetLastError();
  else cudaGetLastError();
  return e == cudaSuccess ? MOE_OK : ops_fail(MOE_ERR_CUDA, fn, cudaGetErrorString(e));
}

inline int dtype_bytes(int32_t dt) {
  return dt == MOE_DT_F32 ? 4 : dt == MOE_DT_U8 ? 1 : 2;
}
inline bool is_float_dtype(int32_t dt) { return dt == MOE_DT_F32 || dt == MOE_DT_BF16 || dt == MOE_DT_F16; }
inline bool aligned_to(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// The largest power of two up to 32 that divides a row's address at every row.
inline int row_alignment(const void *p, int64_t ld_bytes) {
  const uintptr_t v = reinterpret_cast<uintptr_t>(p) | (uintptr_t)ld_bytes | 32u;
  return (int)(v & (~v + 1));
}

// The current device's SM count, looked up once per device.
inline int sm_count() {
  static std::atomic<int> known[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
  if ((n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) n = 148;
  known[dev].store(n, std::memory_order_relaxed);
  return n;
}

// Shared memory above 48 KB has to be asked for, once per kernel and device
// (`asked`: a bit for each device, kept beside the kernel's launch).
template <typename... Args>
inline cudaError_t ask_shared(void (*fn)(Args...), size_t bytes, std::atomic<uint64_t> &asked) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = (uint64_t)1 << (dev & 63);
  if (dev < 64 && (asked.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess && dev < 64) asked.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// A launch that may start while its predecessor on the stream drains; the
// kernel runs wait_prior_grid() before it touches memory.
template <typename... Args>
inline cudaError_t launch_op(void (*fn)(Args...), dim3 grid, int block, size_t smem, cudaStream_t s,
                             const Args &...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, args...);
}

// Division of numbers below 2^31 by one that is known at launch (Granlund and
// Montgomery 1994): a multiplication
// by m = ceil(2^(31 + l) / d), l = ceil(log2 d), is exact there (the hardware's own
// 32-bit division takes three turns of the slow conversion pipe).
struct FastDiv {
  uint32_t d, m, s;
  FastDiv() = default;
  explicit FastDiv(uint32_t d_) : d(d_), m(0), s(0) {
    uint32_t l = 0;
    while (((uint64_t)1 << l) < d) ++l;
    if (l) {
      m = (uint32_t)((((uint64_t)1 << (31 + l)) + d - 1) / d);
      s = l - 1;
    }
  }
  __device__ __forceinline__ uint32_t div(uint32_t i) const { return d == 1 ? i : __umulhi(i, m) >> s; }
};

// ------------------------------------------------------------------ elements
struct F32 {
  using raw = float;
  static __device__ __forceinline__ float to(raw v) { return v; }
  static __device__ __forceinline__ raw from(float v) { return v; }
};
struct BF16 {
  using raw = uint16_t;
  static __device__ __forceinline__ float to(raw v) { return bf16_bits_to_float(v); }
  static __device__ __forceinline__ raw from(float v) { return bf16_bits(v); }
};
struct F16 {
  using raw = uint16_t;
  static __device__ __forceinline__ float to(raw v) { return __half2float(__ushort_as_half(v)); }
  static __device__ __forceinline__ raw from(float v) { return f16_bits(v); }
};

// 32 bytes of one lane at once (sm_100): a whole sector, where two 16-byte accesses
// at a 32-byte stride would touch every sector twice, half of it each time.
__device__ __forceinline__ void ld32(const void *p, uint32_t *w) {
  asm volatile("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p));
}
__device__ __forceinline__ void st32(void *p, const uint32_t *w) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// N consecutive elements of a lane.  ALIGN is what every pack's address is a
// multiple of: 32 or 16 bytes, or the element (0: one access an element).
template <typename T, int N, int ALIGN>
struct Pack {
  alignas(16) typename T::raw v[N];
  static constexpr int kBytes = N * (int)sizeof(typename T::raw);
  __device__ __forceinline__ void load(const typename T::raw *p) {
    uint32_t *w = reinterpret_cast<uint32_t *>(v);
    if constexpr (ALIGN == 32 && kBytes % 32 == 0) {
#pragma unroll
      for (int i = 0; i < kBytes / 32; ++i) ld32(reinterpret_cast<const char *>(p) + 32 * i, w + 8 * i);
    } else if constexpr (ALIGN >= 16) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i)
        reinterpret_cast<uint4 *>(v)[i] = __ldg(reinterpret_cast<const uint4 *>(p) + i);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = __ldg(p + i);
    }
  }
  __device__ __forceinline__ void store(typename T::raw *p) const {
    const uint32_t *w = reinterpret_cast<const uint32_t *>(v);
    if constexpr (ALIGN == 32 && kBytes % 32 == 0) {
#pragma unroll
      for (int i = 0; i < kBytes / 32; ++i) st32(reinterpret_cast<char *>(p) + 32 * i, w + 8 * i);
    } else if constexpr (ALIGN >= 16) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i) reinterpret_cast<uint4 *>(p)[i] = reinterpret_cast<const uint4 *>(v)[i];
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) p[i] = v[i];
    }
  }
  __device__ __forceinline__ float get(int i) const { return T::to(v[i]); }
  __device__ __forceinline__ void set(int i, float f) { v[i] = T::from(f); }
};

}  // namespace moe
