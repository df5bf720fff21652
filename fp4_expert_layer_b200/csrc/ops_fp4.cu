// ops_fp4.cu -- rows to FP4 codes and block scales, and back to values.
//
//   MXFP4, block of 32:  X = clamp(floor(log2 amax) - 2, -126, 127),  c = RNE(v / 2^X)
//   NVFP4, block of 16:  G = 2^ceil(log2(amax_group / 2688)),  s = RNE_E4M3(amax / (6 G)),
//                        c = RNE(v / (s G))
//
// Every rounding is that of the real quotient, with no double rounding:
//  * 2^X is a power of two: v * 2^-X is exact.
//  * The borders between codes, and between scales, have few digits: times d = s G
//    (4 digits) or 6 G they are fp32 numbers, and a correctly rounded fp32 quotient
//    lies on a border only where the real one does.  v / d is formed as q = v r,
//    q' = q + (v - q d) r with r = 1 / d rounded: the residual of an fma is exact,
//    and the corrected quotient is the correctly rounded one (Markstein 1990),
//    for three multiply-adds an element instead of a division.
//
// Bound by memory: x is read once and 0.53 or 0.56 bytes an element are written.
// A thread takes 16 consecutive elements (one NVFP4 block, half an MXFP4 block).
#include "ops_common.cuh"

namespace moe {
namespace {

__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 b;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\t"
      "cvt.u32.u8 %0, b;\n\t}"
      : "=r"(r)
      : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_code(float v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(v));
  return r & 0xFFu;
}
__device__ __forceinline__ float e4m3_value(uint32_t code) {
  const uint32_t h2 = e4m3x2_to_f16x2((uint16_t)code);
  return __half2float(__ushort_as_half((unsigned short)(h2 & 0xFFFFu)));
}

constexpr uint32_t kInfBits = 0x7F800000u;

// Bits of the largest |v| (non-negative floats order like their bits; NaN and
// infinity are at or above kInfBits).
template <typename P>
__device__ __forceinline__ uint32_t amax_bits16(const P &v) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(v.get(i)) & 0x7FFFFFFFu);
  return m;
}

// Bits of G for a group whose largest finite |v| has these bits: 2688 = 1.3125 *
// 2^11, so the exponent is that of amax - 11, and one more above that fraction.
__device__ __forceinline__ uint32_t global_bits(uint32_t amax) {
  if (amax == 0) return 0;
  const int ex = (int)(amax >> 23) + ((amax & 0x7FFFFFu) > 0x280000u ? 1 : 0) - 11;
  return (uint32_t)max(ex, 127 - 100) << 23;
}

template <typename P>
__device__ __forceinline__ uint2 codes_times(const P &v, float inv) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    w[i] = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[i] |= e2m1x2(v.get(8 * i + 2 * j) * inv, v.get(8 * i + 2 * j + 1) * inv) << (8 * j);
  }
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ float quotient(float v, float d, float r) {
  const float q = v * r;
  return fmaf(fmaf(-q, d, v), r, q);
}

// Scale code and codes of one NVFP4 block.
template <typename P>
__device__ __forceinline__ uint32_t nv_block(const P &v, uint32_t amax, float G, uint2 *codes) {
  *codes = make_uint2(0u, 0u);
  if (amax >= kInfBits) return 0x7Fu;
  const uint32_t sc = e4m3_code(__fdiv_rn(__uint_as_float(amax), 6.0f * G));
  if (sc == 0) return 0;
  const float d = e4m3_value(sc) * G;
  const float r = __frcp_rn(d);
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    w[i] = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[i] |= e2m1x2(quotient(v.get(8 * i + 2 * j), d, r), quotient(v.get(8 * i + 2 * j + 1), d, r)) << (8 * j);
  }
  *codes = make_uint2(w[0], w[1]);
  return sc;
}

struct FpArgs {
  const void *x;
  uint8_t *codes;
  uint8_t *scales;
  float *G;
  int64_t ldx;               // elements
  uint32_t rows, cols16;     // cols16 = K / 16
  uint32_t rows_per_scale;
  uint32_t total;            // rows * cols16, at most 2^31
};

// ------------------------------------------------------------------- quantise
// One thread per 16 elements, flat over the rows.  MXFP4 halves meet by shuffle
// (K is a multiple of 32, so a block's halves are neighbouring lanes).  NVFP4
// finds its group's G in memory.
template <typename T, bool VEC, bool MX>
__global__ void __launch_bounds__(256) quantize_flat_kernel(const FpArgs a) {
  wait_prior_grid();
  const uint32_t i = blockIdx.x * 256 + threadIdx.x;
  const bool in = i < a.total;
  const uint32_t row = in ? i / a.cols16 : 0, c = in ? i - row * a.cols16 : 0;
  Pack<T, 16, VEC> v;
  v.load(static_cast<const typename T::raw *>(a.x) + row * a.ldx + 16 * c, in ? 16 : 0);
  uint32_t am = amax_bits16(v);
  if constexpr (MX) {
    am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
    uint32_t code = 1;
    uint2 w = make_uint2(0u, 0u);
    if (am >= kInfBits) {
      code = 255;
    } else {
      code = (uint32_t)max(1, (int)(am >> 23) - 2);
      w = codes_times(v, __uint_as_float((254u - code) << 23));
    }
    if (!in) return;
    reinterpret_cast<uint2 *>(a.codes)[i] = w;
    if ((i & 1) == 0) a.scales[i >> 1] = (uint8_t)code;
  } else {
    if (!in) return;
    const uint32_t g = row / a.rows_per_scale;
    float G = __ldcg(a.G + g);
    if (G == 0.0f) {                                   // nothing but zeros (and non-finite blocks) in the group
      G = 1.0f;
      if (c == 0 && row == g * a.rows_per_scale) a.G[g] = 1.0f;
    }
    uint2 w;
    const uint32_t sc = nv_block(v, am, G, &w);
    reinterpret_cast<uint2 *>(a.codes)[i] = w;
    a.scales[i] = (uint8_t)sc;
  }
}

// NVFP4 with a scale per row: the row's threads keep it in registers, agree on G
// and quantise: one pass.  `tpr` threads (whole warps) to a row.
template <typename T, bool VEC>
__global__ void __launch_bounds__(1024) quantize_rows_kernel(const FpArgs a, int tpr) {
  __shared__ uint32_t wmax[32];
  wait_prior_grid();
  const int rows_here = blockDim.x / tpr, lr = threadIdx.x / tpr, tc = threadIdx.x - lr * tpr;
  const uint64_t row = (uint64_t)blockIdx.x * rows_here + lr;
  const bool in = row < a.rows;
  const auto *x = static_cast<const typename T::raw *>(a.x) + (in ? row : 0) * a.ldx;
  Pack<T, 16, VEC> v;
  uint32_t am = 0, finite = 0;
  for (uint32_t c = tc; c < a.cols16; c += tpr) {      // one turn up to 16 * 1024 columns
    v.load(x + 16 * (uint64_t)c, in ? 16 : 0);
    am = amax_bits16(v);
    if (am < kInfBits) finite = max(finite, am);
  }
  finite = __reduce_max_sync(0xffffffffu, finite);
  if (tpr > 32) {
    if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = finite;
    __syncthreads();
    const int w0 = lr * tpr / 32;
    for (int w = 0; w < tpr / 32; ++w) finite = max(finite, wmax[w0 + w]);
  }
  if (!in) return;
  const float G = finite ? __uint_as_float(global_bits(finite)) : 1.0f;
  if (tc == 0) a.G[row] = G;
  const bool one = a.cols16 <= (uint32_t)tpr;
  for (uint32_t c = tc; c < a.cols16; c += tpr) {
    if (!one) {
      v.load(x + 16 * (uint64_t)c, 16);
      am = amax_bits16(v);
    }
    uint2 w;
    const uint32_t sc = nv_block(v, am, G, &w);
    const uint32_t i = (uint32_t)row * a.cols16 + c;
    reinterpret_cast<uint2 *>(a.codes)[i] = w;
    a.scales[i] = (uint8_t)sc;
  }
}

// NVFP4 with a scale per group of rows, first pass: G of every group.  G grows
// with amax, so each CTA puts its own maximum's G into the group's word (zero
// before) by an integer maximum, whose order does not matter.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) group_scale_kernel(const FpArgs a, uint32_t per_group, uint32_t blocks) {
  __shared__ uint32_t wmax[8];
  wait_prior_grid();
  const uint32_t g = blockIdx.x / blocks, b = blockIdx.x - g * blocks;
  const uint32_t row0 = g * a.rows_per_scale;
  uint32_t finite = 0;
  for (uint32_t i = b * 256 + threadIdx.x; i < per_group; i += blocks * 256) {
    const uint32_t r = i / a.cols16, c = i - r * a.cols16;
    Pack<T, 16, VEC> v;
    v.load(static_cast<const typename T::raw *>(a.x) + (int64_t)(row0 + r) * a.ldx + 16 * c, 16);
    const uint32_t am = amax_bits16(v);
    if (am < kInfBits) finite = max(finite, am);
  }
  finite = __reduce_max_sync(0xffffffffu, finite);
  if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = finite;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 8; ++w) finite = max(finite, wmax[w]);
    if (finite) atomicMax(reinterpret_cast<uint32_t *>(a.G) + g, global_bits(finite));
  }
}

// ----------------------------------------------------------------- dequantise
template <typename T, bool VEC, bool MX>
__global__ void __launch_bounds__(256) dequantize_kernel(const FpArgs a) {
  wait_prior_grid();
  const uint32_t i = blockIdx.x * 256 + threadIdx.x;
  if (i >= a.total) return;
  const uint32_t row = i / a.cols16, c = i - row * a.cols16;
  const uint2 w = __ldg(reinterpret_cast<const uint2 *>(a.codes) + i);
  float d;
  if constexpr (MX) {
    const uint32_t code = __ldg(a.scales + (i >> 1));
    d = code == 255 ? __uint_as_float(0x7FC00000u)
                    : code == 0 ? __uint_as_float(1u << 22) : __uint_as_float(code << 23);   // 0 is 2^-127
  } else {
    d = e4m3_value(__ldg(a.scales + i)) * __ldg(a.G + row / a.rows_per_scale);
  }
  Pack<T, 16, VEC> out;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t f[4];
    e2m1x8_to_f16x2(h ? w.y : w.x, f);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 p = __half22float2(*reinterpret_cast<__half2 *>(&f[j]));
      out.set(8 * h + 2 * j, p.x * d);
      out.set(8 * h + 2 * j + 1, p.y * d);
    }
  }
  out.store(static_cast<typename T::raw *>(const_cast<void *>(a.x)) + row * a.ldx + 16 * c, 16);
}

moe_status_t check_fp4(const char *fn, int32_t dtype, int64_t rows, int64_t K, int64_t ld, int32_t fmt,
                       int64_t rows_per_scale, const void *dense, const void *codes, const void *scales,
                       const void *G) {
  if (!is_float_dtype(dtype)) return ops_invalid(fn, "dtype must be F32, BF16 or F16");
  if (fmt != MOE_FMT_MXFP4 && fmt != MOE_FMT_NVFP4) return ops_invalid(fn, "fmt must be MOE_FMT_MXFP4 or MOE_FMT_NVFP4");
  if (rows < 0 || K < 32 || K % 32 || K > (int64_t)1 << 30) return ops_invalid(fn, "need rows >= 0 and K a multiple of 32");
  if (rows > ((int64_t)1 << 31) - 1 || (rows && K / 16 > ((int64_t)1 << 31) / rows))
    return ops_invalid(fn, "rows must be below 2^31 and rows * K at most 2^35");
  if (ld < K) return ops_invalid(fn, "the row stride must be at least K");
  if (rows_per_scale < 1 || rows % rows_per_scale) return ops_invalid(fn, "rows must be a multiple of rows_per_scale");
  if (rows == 0) return MOE_OK;
  if (!dense || !codes || !scales) return ops_invalid(fn, "rows, codes and scales must be device pointers");
  if (fmt == MOE_FMT_NVFP4 && !G) return ops_invalid(fn, "NVFP4 needs global_scale");
  if (!aligned_to(codes, 16)) return ops_invalid(fn, "codes must be 16-byte aligned");
  if (!aligned_to(dense, dtype_bytes(dtype)) || !aligned_to(G, 4))
    return ops_invalid(fn, "rows and global_scale must be aligned to their type");
  return MOE_OK;
}

FpArgs fp_args(const void *x, int64_t rows, int64_t K, int64_t ld, int64_t rows_per_scale, const uint8_t *codes,
               const uint8_t *scales, const float *G) {
  FpArgs a{};
  a.x = x;
  a.codes = const_cast<uint8_t *>(codes);
  a.scales = const_cast<uint8_t *>(scales);
  a.G = const_cast<float *>(G);
  a.ldx = ld;
  a.rows = (uint32_t)rows;
  a.cols16 = (uint32_t)(K / 16);
  a.rows_per_scale = (uint32_t)rows_per_scale;
  a.total = a.rows * a.cols16;
  return a;
}

dim3 flat_grid(const FpArgs &a) { return dim3(a.total / 256 + (a.total % 256 != 0)); }

template <typename T, bool VEC>
cudaError_t quantize(const FpArgs &a, int32_t fmt, cudaStream_t s) {
  if (fmt == MOE_FMT_MXFP4) return launch_op(quantize_flat_kernel<T, VEC, true>, flat_grid(a), 256, 0, s, a);
  if (a.rows_per_scale == 1) {
    const int tpr = (int)std::min<uint32_t>(1024, (a.cols16 + 31) / 32 * 32);
    const int rows_here = std::max(1, 256 / tpr);
    return launch_op(quantize_rows_kernel<T, VEC>, dim3((a.rows + rows_here - 1) / rows_here), tpr * rows_here, 0, s, a,
                     tpr);
  }
  const uint32_t groups = a.rows / a.rows_per_scale, per_group = a.rows_per_scale * a.cols16;
  const uint32_t want = std::max<uint32_t>(1, (uint32_t)(8 * sm_count()) / groups);
  const uint32_t blocks = std::min<uint32_t>(want, (per_group + 1023) / 1024);
  cudaError_t e = cudaMemsetAsync(a.G, 0, (size_t)groups * sizeof(float), s);
  if (e == cudaSuccess) e = launch_op(group_scale_kernel<T, VEC>, dim3(groups * blocks), 256, 0, s, a, per_group, blocks);
  if (e == cudaSuccess) e = launch_op(quantize_flat_kernel<T, VEC, false>, flat_grid(a), 256, 0, s, a);
  return e;
}

template <typename T, bool VEC>
cudaError_t dequantize(const FpArgs &a, int32_t fmt, cudaStream_t s) {
  return launch_op(fmt == MOE_FMT_MXFP4 ? dequantize_kernel<T, VEC, true> : dequantize_kernel<T, VEC, false>,
                   flat_grid(a), 256, 0, s, a);
}

}  // namespace
}  // namespace moe

using namespace moe;

#define MOE_BY_TYPE(f)                                                                       \
  (dtype == MOE_DT_F32    ? (vec ? f<F32, true>(a, fmt, s) : f<F32, false>(a, fmt, s))       \
   : dtype == MOE_DT_BF16 ? (vec ? f<BF16, true>(a, fmt, s) : f<BF16, false>(a, fmt, s))     \
                          : (vec ? f<F16, true>(a, fmt, s) : f<F16, false>(a, fmt, s)))

extern "C" {

moe_status_t moe_fp4_quantize(const void *x, int32_t dtype, int64_t rows, int64_t K, int64_t ldx, int32_t fmt,
                              int64_t rows_per_scale, uint8_t *codes, uint8_t *scales, float *global_scale,
                              void *stream) {
  static const char fn[] = "moe_fp4_quantize";
  const moe_status_t st = check_fp4(fn, dtype, rows, K, ldx, fmt, rows_per_scale, x, codes, scales, global_scale);
  if (st != MOE_OK || rows == 0) return st;
  const FpArgs a = fp_args(x, rows, K, ldx, rows_per_scale, codes, scales, global_scale);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool vec = row_alignment(x, ldx * dtype_bytes(dtype)) == 16;
  return ops_launched(fn, MOE_BY_TYPE(quantize));
}

moe_status_t moe_fp4_dequantize(const uint8_t *codes, const uint8_t *scales, const float *global_scale, int32_t fmt,
                                int64_t rows, int64_t K, int64_t rows_per_scale, void *out, int32_t dtype,
                                int64_t ldo, void *stream) {
  static const char fn[] = "moe_fp4_dequantize";
  const moe_status_t st = check_fp4(fn, dtype, rows, K, ldo, fmt, rows_per_scale, out, codes, scales, global_scale);
  if (st != MOE_OK || rows == 0) return st;
  const FpArgs a = fp_args(out, rows, K, ldo, rows_per_scale, codes, scales, global_scale);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool vec = row_alignment(out, ldo * dtype_bytes(dtype)) == 16;
  return ops_launched(fn, MOE_BY_TYPE(dequantize));
}

}  // extern "C"
