// ops_fp4.cu -- rows to FP4 codes and block scales, and back to values.
//
//   MXFP4, block of 32:  X = clamp(floor(log2 amax) - 2, -126, 127),  c = RNE(v / 2^X)
//   NVFP4, block of 16:  G = 2^ceil(log2(amax_group / 2688)),  s = RNE_E4M3(amax / (6 G)),
//                        c = RNE(v / (s G))
//
// Every rounding to codes and scales is that of the real quotient, with no double
// rounding (the way back has its own section below):
//  * 2^X is a power of two: v * 2^-X is exact.
//  * The borders between codes, and between scales, have few digits: times d = s G
//    (4 digits) or 6 G they are fp32 numbers, so a quotient that is not on a border
//    is at least 0.53 ulp away from it, and the nearest fp32 number to it lies on
//    the right side.  v / d is formed as q = v r, q' = q + (v - q d) r with r within
//    an ulp or two of 1 / d: the residual of an fma is exact, q' is off by 2^-20 ulp
//    before its rounding (Markstein 1990), so it is that nearest number, and a
//    border exactly where the quotient is one: three multiply-adds an element, two
//    elements an instruction, instead of a division.
//  * 16-bit elements have 11 digits at most: a quotient that is not on a border b is
//    b 2^-11 >= 2^-13 away from it.  There v r + 192 - 192, which rounds to a
//    multiple of 2^-16 (|v / d| <= 9), does in two operations.
//
// Bound by memory: x is read once and 0.53 or 0.56 bytes an element are written.
// A thread takes pieces of 16 consecutive elements (one NVFP4 block, half an MXFP4
// block), 32 bytes of 16-bit elements in one access.  8192 x 4096 bf16: MXFP4 13.8
// us quantised, 13.6 read back (94% and 95% of the copy rate); NVFP4 by rows 15.7
// and 14.6 (83%, 90%): there the arithmetic, some 150 instructions a piece, shows.
// An NVFP4 scale over many rows needs a pass over x before the codes: 64 matrices of
// 1024 x 2048 97.6 us (53% of the copy rate for x once and the codes), of 93 for the two
// reads and the codes (a cluster a matrix, to read it again from L2, takes 97 to 147).
#include <type_traits>

#include "ops_common.cuh"

namespace moe {
namespace {

// Eight values to codes (round to nearest even, saturating), the first in bits 0..3.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_code(float v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(v));
  return r & 0xFFu;
}
// The value of a finite, non-negative code: its fields in place of a float's,
// whose exponents lie 120 higher (exact for the subnormal codes too).
__device__ __forceinline__ float e4m3_value(uint32_t code) { return __uint_as_float(code << 20) * 0x1p120f; }
// The value of any code.
__device__ __forceinline__ float e4m3_any(uint32_t code) {
  const float v = e4m3_value(code & 127u);
  return (code & 127u) == 127u ? __uint_as_float(0x7FC00000u) : code & 128u ? -v : v;
}

// The value of an E2M1 code: its fields in place of a float's, as above.
__device__ __forceinline__ float e2m1_value(uint32_t code) {
  return __uint_as_float((code & 7u) << 22 | (code & 8u) << 28) * 0x1p126f;
}

constexpr uint32_t kInfBits = 0x7F800000u;

// Bits of the largest |v| (non-negative floats order like their bits; NaN and
// infinity are at or above kInfBits).
template <typename T, int ALIGN>
__device__ __forceinline__ uint32_t amax_bits16(const Pack<T, 16, ALIGN> &v) {
  if constexpr (sizeof(typename T::raw) == 4) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(v.get(i)) & 0x7FFFFFFFu);
    return m;
  } else {
    // 16-bit magnitudes order like their bits too: two at a time
    const uint32_t *w = reinterpret_cast<const uint32_t *>(v.v);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
    const uint32_t top = max(m & 0xFFFFu, m >> 16);
    return __float_as_uint(T::to((uint16_t)top)) & 0x7FFFFFFFu;
  }
}

// Bits of G for a group whose largest finite |v| has these bits: 2688 = 1.3125 *
// 2^11, so the exponent is that of amax - 11, and one more above that fraction.
__device__ __forceinline__ uint32_t global_bits(uint32_t amax) {
  if (amax == 0) return 0;
  const int ex = (int)(amax >> 23) + ((amax & 0x7FFFFFu) > 0x280000u ? 1 : 0) - 11;
  return (uint32_t)max(ex, 127 - 100) << 23;
}

__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float rcp_approx(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// Codes of 16 elements times `inv`, or, with DIV, divided by d (inv near 1 / d).
template <bool DIV, typename P>
__device__ __forceinline__ uint2 codes16(const P &v, float inv, float d) {
  const uint64_t r = pack2(inv, inv), minus_d = pack2(-d, -d);
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float f[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint64_t x = pack2(v.get(8 * i + 2 * j), v.get(8 * i + 2 * j + 1));
      uint64_t q;
      if constexpr (!DIV) {
        q = mul2(x, r);
      } else if constexpr (sizeof(v.v[0]) == 2) {
        q = add2(fma2(x, r, pack2(192.0f, 192.0f)), pack2(-192.0f, -192.0f));
      } else {
        q = mul2(x, r);
        q = fma2(fma2(q, minus_d, x), r, q);
      }
      asm("mov.b64 {%0, %1}, %2;" : "=f"(f[2 * j]), "=f"(f[2 * j + 1]) : "l"(q));
    }
    w[i] = e2m1x8(f);
  }
  return make_uint2(w[0], w[1]);
}

// Scale code and codes of one NVFP4 block.
template <typename P>
__device__ __forceinline__ uint32_t nv_block(const P &v, uint32_t amax, float G, uint2 *codes) {
  *codes = make_uint2(0u, 0u);
  if (amax >= kInfBits) return 0x7Fu;
  // amax / 6 correctly rounded (6's reciprocal is), then / G, a power of two
  const float invG = __uint_as_float((254u << 23) - __float_as_uint(G));
  const float top = __uint_as_float(amax), r6 = 1.0f / 6.0f, q6 = top * r6;
  const uint32_t sc = e4m3_code(fmaf(fmaf(-6.0f, q6, top), r6, q6) * invG);
  if (sc == 0) return 0;
  const float s = e4m3_value(sc);
  *codes = codes16<true>(v, rcp_approx(s) * invG, s * G);
  return sc;
}

struct FpArgs {
  const void *x;
  uint8_t *codes;
  uint8_t *scales;
  float *G;
  int64_t ldx;               // elements
  uint32_t rows, cols16;     // cols16 = K / 16
  FastDiv by_cols, by_group; // / cols16, / rows_per_scale
  uint32_t rows_per_scale;
  uint32_t total;            // rows * cols16, at most 2^31
};

// ------------------------------------------------------------------- quantise
// A thread takes U pieces of 16 elements, flat over the rows, loads in flight
// together.  MXFP4 halves meet by shuffle (K is a multiple of 32, so a block's
// halves are neighbouring lanes); one piece a thread keeps HBM busy (65536 x 2048
// bf16: 49.1 us, the copy rate).  NVFP4 finds its group's G in memory and takes two
// (with the pass for G 98.3 us; with one 101.7, with four 100.4).
template <typename T, int ALIGN, bool MX, int U>
__global__ void __launch_bounds__(256) quantize_flat_kernel(const FpArgs a) {
  wait_prior_grid();
  const uint32_t i0 = blockIdx.x * (256 * U) + threadIdx.x;
  Pack<T, 16, ALIGN> v[U];
  uint32_t row[U];
  float G[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t i = i0 + 256 * u;
    if (i < a.total) {
      row[u] = a.by_cols.div(i);
      v[u].load(static_cast<const typename T::raw *>(a.x) + row[u] * a.ldx + 16 * (i - row[u] * a.cols16));
      if constexpr (!MX) G[u] = a.G[a.by_group.div(row[u])];   // from L1: one word for many threads
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t i = i0 + 256 * u;
    const bool in = i < a.total;
    uint32_t am = in ? amax_bits16(v[u]) : 0;
    if constexpr (MX) am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
    if (!in) break;
    uint2 w = make_uint2(0u, 0u);
    if constexpr (MX) {
      uint32_t code = 255;
      if (am < kInfBits) {
        code = (uint32_t)max(1, (int)(am >> 23) - 2);
        w = codes16<false>(v[u], __uint_as_float((254u - code) << 23), 0.0f);
      }
      if ((i & 1) == 0) a.scales[i >> 1] = (uint8_t)code;
    } else {
      if (G[u] == 0.0f) {                              // nothing but zeros (and non-finite blocks) in the group
        G[u] = 1.0f;
        const uint32_t g = a.by_group.div(row[u]);
        if (i == g * a.rows_per_scale * a.cols16) a.G[g] = 1.0f;
      }
      a.scales[i] = (uint8_t)nv_block(v[u], am, G[u], &w);
    }
    reinterpret_cast<uint2 *>(a.codes)[i] = w;
  }
}

// NVFP4 with a scale per row: the row's threads keep it in registers (NCH pieces
// of 16 each), agree on G and quantise: one pass.  `tpr` threads (whole warps) to
// a row; a row beyond what they hold (16384 elements and more) is read again for the codes.
template <typename T, int ALIGN, int NCH>
__global__ void __launch_bounds__(NCH == 1 ? 1024 : 512) quantize_rows_kernel(const FpArgs a, int tpr) {
  __shared__ uint32_t wmax[32];
  wait_prior_grid();
  const int rows_here = blockDim.x / tpr, lr = threadIdx.x / tpr, tc = threadIdx.x - lr * tpr;
  const uint64_t row = (uint64_t)blockIdx.x * rows_here + lr;
  const bool in = row < a.rows;
  const auto *x = static_cast<const typename T::raw *>(a.x) + (in ? row : 0) * a.ldx;
  Pack<T, 16, ALIGN> v[NCH];
  uint32_t am[NCH], finite = 0;
  for (uint32_t c0 = tc; c0 < a.cols16; c0 += NCH * tpr) {
#pragma unroll
    for (int i = 0; i < NCH; ++i)
      if (in && c0 + i * tpr < a.cols16) v[i].load(x + 16 * (uint64_t)(c0 + i * tpr));
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      am[i] = in && c0 + i * tpr < a.cols16 ? amax_bits16(v[i]) : 0;
      if (am[i] < kInfBits) finite = max(finite, am[i]);
    }
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
  const bool one = a.cols16 <= (uint32_t)(NCH * tpr);
  for (uint32_t c0 = tc; c0 < a.cols16; c0 += NCH * tpr) {
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const uint32_t c = c0 + i * tpr;
      if (c >= a.cols16) break;
      if (!one) {
        v[i].load(x + 16 * (uint64_t)c);
        am[i] = amax_bits16(v[i]);
      }
      uint2 w;
      const uint32_t sc = nv_block(v[i], am[i], G, &w);
      const uint32_t at = (uint32_t)row * a.cols16 + c;
      reinterpret_cast<uint2 *>(a.codes)[at] = w;
      a.scales[at] = (uint8_t)sc;
    }
  }
}

// NVFP4 with a scale per group of rows, first pass: G of every group.  G grows
// with amax, so each CTA puts its own maximum's G into the group's word (zero
// before) by an integer maximum, whose order does not matter.
template <typename T, int ALIGN>
__global__ void __launch_bounds__(256) group_scale_kernel(const FpArgs a, uint32_t per_group, uint32_t blocks) {
  __shared__ uint32_t wmax[8];
  wait_prior_grid();
  const uint32_t g = blockIdx.x / blocks, b = blockIdx.x - g * blocks;
  const uint32_t row0 = g * a.rows_per_scale;
  uint32_t finite = 0;
  constexpr int U = sizeof(typename T::raw) == 4 ? 2 : 4;   // loads in flight together
  const uint32_t step = blocks * 256;
  for (uint32_t i = b * 256 + threadIdx.x; i < per_group; i += U * step) {
    Pack<T, 16, ALIGN> v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t j = i + u * step;
      if (j < per_group) {
        const uint32_t r = a.by_cols.div(j);
        v[u].load(static_cast<const typename T::raw *>(a.x) + (int64_t)(row0 + r) * a.ldx + 16 * (j - r * a.cols16));
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t am = i + u * step < per_group ? amax_bits16(v[u]) : 0;
      if (am < kInfBits) finite = max(finite, am);
    }
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
//   value = (code scale) G, rounded once to the type.
//
// code times scale has 6 digits and is exact; times G it is rounded to fp32, and for
// 16-bit results once more.  The second rounding errs only where the first one ended on
// a border between two 16-bit numbers: seldom, and never where G is a power of two.  A
// piece that has such a border in it (Borders) is done again with fp32 products rounded
// to odd (towards zero, the last digit set where something was cut off), which stay on
// their side of every border (Boldo and Melquiond 2008).  8192 x 4096 to bf16, with all
// in L2: 12.9 us, with any G 12.8, with every product rounded to odd 17.8; to f16 13.5, and
// 26 where all values are below 2^-9 and G has more than 18 digits (small() below).
template <typename T>
struct Borders {
  uint32_t least = 0xFFFFFFFFu;                            // two at a time: 0 where one was met
  __device__ __forceinline__ void look(float a, float b) {
    // low digits of an fp32 number on a border of the 16-bit type's normal numbers: 1 and zeros
    constexpr uint32_t digits = std::is_same<T, BF16>::value ? 0xFFFFFFFFu : 0x1FFF1FFFu;
    constexpr uint32_t border = std::is_same<T, BF16>::value ? 0x80008000u : 0x10001000u;
    const uint32_t low = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x5410);
    least = __vminu2(least, (low & digits) ^ border);
  }
  // f16: the borders of its subnormal numbers are odd multiples of 2^-25, whatever their
  // digits.  Asked of pieces whose smallest values are that small (all of a piece's are
  // below 2^-9 then), unless G has so few digits (18) that the fp32 products are exact.
  static __device__ __forceinline__ bool small(float d, float G) {
    const float unit = fabsf(d * G);
    return std::is_same<T, F16>::value && unit > 0.0f && unit < 0x1p-13f && (__float_as_uint(G) & 63u);
  }
  static __device__ __forceinline__ bool small_border(float v) { return (v + 0.375f) - 0.375f == v && v != 0.0f; }
  __device__ __forceinline__ bool met() const { return (least & 0xFFFFu) == 0 || least >> 16 == 0; }
};
__device__ __forceinline__ float mul_to_odd(float a, float b) {
  const float lo = __fmul_rd(fabsf(a), fabsf(b)), hi = __fmul_ru(fabsf(a), fabsf(b));
  const uint32_t sign = (__float_as_uint(a) ^ __float_as_uint(b)) & 0x80000000u;
  return __uint_as_float(__float_as_uint(lo) | (lo != hi ? 1u : 0u) | sign);
}

template <typename T, int ALIGN, bool MX, int U>
__global__ void __launch_bounds__(256) dequantize_kernel(const FpArgs a) {
  wait_prior_grid();
  // U pieces a thread, their loads in flight together
  const uint32_t i0 = blockIdx.x * (256 * U) + threadIdx.x;
  uint2 code[U];
  uint32_t scale[U], row[U];
  float G[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t i = i0 + 256 * u;
    if (i >= a.total) break;
    row[u] = a.by_cols.div(i);
    code[u] = __ldg(reinterpret_cast<const uint2 *>(a.codes) + i);
    scale[u] = __ldg(a.scales + (MX ? i >> 1 : i));
    G[u] = MX ? 1.0f : __ldg(a.G + a.by_group.div(row[u]));
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t i = i0 + 256 * u;
    if (i >= a.total) break;
    float d;
    if constexpr (MX) {
      d = scale[u] == 255 ? __uint_as_float(0x7FC00000u)
                          : scale[u] == 0 ? __uint_as_float(1u << 22) : __uint_as_float(scale[u] << 23);   // 0 is 2^-127
    } else {
      d = e4m3_any(scale[u]);
    }
    Pack<T, 16, ALIGN> out;
    constexpr bool kTwice = !MX && sizeof(typename T::raw) == 2;
    Borders<T> borders;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t f[4];
      e2m1x8_to_f16x2(h ? code[u].y : code[u].x, f);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 p = __half22float2(*reinterpret_cast<__half2 *>(&f[j]));
        float v0 = p.x * d, v1 = p.y * d;
        if constexpr (!MX) {
          v0 *= G[u];
          v1 *= G[u];
        }
        if constexpr (kTwice) borders.look(v0, v1);
        out.set(8 * h + 2 * j, v0);
        out.set(8 * h + 2 * j + 1, v1);
      }
    }
    auto *dst = static_cast<typename T::raw *>(const_cast<void *>(a.x)) + row[u] * a.ldx + 16 * (i - row[u] * a.cols16);
    bool again = kTwice && borders.met();
    if (kTwice && Borders<T>::small(d, G[u])) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const uint32_t c = (e < 8 ? code[u].x : code[u].y) >> (4 * (e & 7)) & 15u;
        again = again || Borders<T>::small_border(e2m1_value(c) * d * G[u]);
      }
    }
    if (again) {
#pragma unroll 1
      for (int e = 0; e < 16; ++e) {
        const uint32_t c = (e < 8 ? code[u].x : code[u].y) >> (4 * (e & 7)) & 15u;
        dst[e] = T::from(mul_to_odd(e2m1_value(c) * d, G[u]));
      }
    } else {
      out.store(dst);
    }
  }
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
  a.by_cols = FastDiv(a.cols16);
  a.by_group = FastDiv(a.rows_per_scale);
  a.total = a.rows * a.cols16;
  return a;
}

// CTAs of 256 threads with `u` pieces to a thread.
dim3 flat_grid(const FpArgs &a, uint32_t u) { return dim3(a.total / (256 * u) + (a.total % (256 * u) != 0)); }

template <typename T, int ALIGN>
cudaError_t quantize(FpArgs a, int32_t fmt, cudaStream_t s) {
  if (fmt == MOE_FMT_MXFP4) return launch_op(quantize_flat_kernel<T, ALIGN, true, 1>, flat_grid(a, 1), 256, 0, s, a);
  // A group whose rows follow one another without a gap is one long row: one launch,
  // a CTA a group.  Up to 4096 pieces it is the faster way (1 group of 4096 5.6 us,
  // by two passes 6.3; 1024 groups 38 and 53), up to 8192 with a group for every SM
  // (1 group 9.5 and 6.3; 256 groups 24 and 29).
  const uint64_t long_row = (uint64_t)a.rows_per_scale * a.cols16;
  if (a.rows_per_scale > 1 && a.ldx == (int64_t)a.cols16 * 16 &&
      (long_row <= 4096 || (long_row <= 8192 && a.rows / a.rows_per_scale >= (uint32_t)sm_count()))) {
    a.rows /= a.rows_per_scale;
    a.cols16 *= a.rows_per_scale;
    a.ldx *= a.rows_per_scale;
    a.rows_per_scale = 1;
  }
  if (a.rows_per_scale == 1) {
    // few rows: a thread takes one piece, so that a row is spread wide; rows that
    // fill the GPU: as many as leave every lane of a row's warp one (four, of fp32
    // two, at most), whose loads are in flight together
    constexpr uint32_t kMost = sizeof(typename T::raw) == 4 ? 2 : 4;
    const uint32_t nch = a.total < (uint32_t)(sm_count() * 2048) || a.cols16 <= 32 ? 1
                         : a.cols16 <= 64                                         ? 2
                                                                                  : kMost;
    const int tpr = (int)std::min<uint32_t>(nch > 1 ? 512 : 1024, ((a.cols16 + nch - 1) / nch + 31) / 32 * 32);
    const int rows_here = std::max(1, 256 / tpr);
    return launch_op(nch == 1   ? quantize_rows_kernel<T, ALIGN, 1>
                     : nch == 2 ? quantize_rows_kernel<T, ALIGN, 2>
                                : quantize_rows_kernel<T, ALIGN, kMost>,
                     dim3((a.rows + rows_here - 1) / rows_here), tpr * rows_here, 0, s, a, tpr);
  }
  const uint32_t groups = a.rows / a.rows_per_scale, per_group = a.rows_per_scale * a.cols16;
  const uint32_t want = std::max<uint32_t>(1, (uint32_t)(8 * sm_count()) / groups);
  const uint32_t blocks = std::min<uint32_t>(want, (per_group + 1023) / 1024);   // four turns of a CTA at least
  cudaError_t e = cudaMemsetAsync(a.G, 0, (size_t)groups * sizeof(float), s);
  if (e == cudaSuccess) e = launch_op(group_scale_kernel<T, ALIGN>, dim3(groups * blocks), 256, 0, s, a, per_group, blocks);
  if (e == cudaSuccess) e = launch_op(quantize_flat_kernel<T, ALIGN, false, 2>, flat_grid(a, 2), 256, 0, s, a);
  return e;
}

template <typename T, int ALIGN>
cudaError_t dequantize(const FpArgs &a, int32_t fmt, cudaStream_t s) {
  // one piece a thread until that fills the GPU, then four (MXFP4 to bf16, 8 x 2048:
  // 1.2 us, with four 1.7; 8192 x 4096: 13.6, with one 14.6)
  const bool mx = fmt == MOE_FMT_MXFP4;
  if (a.total < (uint32_t)(sm_count() * 2048))
    return launch_op(mx ? dequantize_kernel<T, ALIGN, true, 1> : dequantize_kernel<T, ALIGN, false, 1>, flat_grid(a, 1),
                     256, 0, s, a);
  return launch_op(mx ? dequantize_kernel<T, ALIGN, true, 4> : dequantize_kernel<T, ALIGN, false, 4>, flat_grid(a, 4),
                   256, 0, s, a);
}

}  // namespace
}  // namespace moe

using namespace moe;

#define MOE_BY_ALIGN(f, T) (al == 32 ? f<T, 32>(a, fmt, s) : al == 16 ? f<T, 16>(a, fmt, s) : f<T, 0>(a, fmt, s))
#define MOE_BY_TYPE(f)                                    \
  (dtype == MOE_DT_F32    ? MOE_BY_ALIGN(f, F32)          \
   : dtype == MOE_DT_BF16 ? MOE_BY_ALIGN(f, BF16)         \
                          : MOE_BY_ALIGN(f, F16))

extern "C" {

moe_status_t moe_fp4_quantize(const void *x, int32_t dtype, int64_t rows, int64_t K, int64_t ldx, int32_t fmt,
                              int64_t rows_per_scale, uint8_t *codes, uint8_t *scales, float *global_scale,
                              void *stream) {
  static const char fn[] = "moe_fp4_quantize";
  const moe_status_t st = check_fp4(fn, dtype, rows, K, ldx, fmt, rows_per_scale, x, codes, scales, global_scale);
  if (st != MOE_OK || rows == 0) return st;
  const FpArgs a = fp_args(x, rows, K, ldx, rows_per_scale, codes, scales, global_scale);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int al = row_alignment(x, ldx * dtype_bytes(dtype));
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
  const int al = row_alignment(out, ldo * dtype_bytes(dtype));
  return ops_launched(fn, MOE_BY_TYPE(dequantize));
}

}  // extern "C"
