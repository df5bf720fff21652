// ops_common.cuh -- what the stand-alone operators (moe_ops.h) share: argument
// checks, launch helpers, and 16-bit / 32-bit element access.
#pragma once

#include <algorithm>
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

// The largest power of two up to 16 that divides a row's address at every row.
inline int row_alignment(const void *p, int64_t ld_bytes) {
  const uintptr_t v = reinterpret_cast<uintptr_t>(p) | (uintptr_t)ld_bytes | 16u;
  return (int)(v & (~v + 1));
}

// The current device and its SM count, looked up once per device.
inline int sm_count() {
  static int n[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
  if (!n[dev]) {
    int v = 0;
    n[dev] = cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && v > 0 ? v : 148;
  }
  return n[dev];
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

// N consecutive elements: one access when VEC (p is then aligned to the whole),
// else N accesses, of which those at and behind `n` are left out.
template <typename T, int N, bool VEC>
struct Pack {
  alignas(16) typename T::raw v[N];
  __device__ __forceinline__ void load(const typename T::raw *p, int n) {
    if constexpr (VEC) {
      static_assert(sizeof(v) % 16 == 0, "whole 16-byte words");
      uint4 *w = reinterpret_cast<uint4 *>(v);
#pragma unroll
      for (int i = 0; i < (int)(sizeof(v) / 16); ++i) w[i] = __ldg(reinterpret_cast<const uint4 *>(p) + i);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = i < n ? __ldg(p + i) : typename T::raw(0);
    }
  }
  __device__ __forceinline__ void store(typename T::raw *p, int n) const {
    if constexpr (VEC) {
      const uint4 *w = reinterpret_cast<const uint4 *>(v);
#pragma unroll
      for (int i = 0; i < (int)(sizeof(v) / 16); ++i) reinterpret_cast<uint4 *>(p)[i] = w[i];
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i < n) p[i] = v[i];
    }
  }
  __device__ __forceinline__ float get(int i) const { return T::to(v[i]); }
  __device__ __forceinline__ void set(int i, float f) { v[i] = T::from(f); }
};

}  // namespace moe
