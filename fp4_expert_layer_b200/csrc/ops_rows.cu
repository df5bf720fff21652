// ops_rows.cu -- rows sent to their experts and brought back, with gradients.
//
//   dispatch            xs[inv[t,j]] = x[t]
//   dispatch backward   dx[t] = sum_j dxs[inv[t,j]]
//   combine             y[t] = sum_j g[t,j] ys[inv[t,j]]
//   combine backward    dys[inv[t,j]] = g[t,j] dy[t],  dg[t,j] = <dy[t], ys[inv[t,j]]>
//
// All four are bound by memory: one multiply-add an element at most.  They run
// by token, not by sorted row, so that a token's row is read once for its k
// pairs (dispatch and both gradients) and a sum over pairs stays in fp32
// registers in ascending j: no atomics, one rounding, the same bits each time.
//
// Measured, bf16, 8192 tokens x 8 pairs, H 2048 (share of the copy rate): dispatch
// 48.7 us (94%), its backward 48.7 (95%), combine 48.9 (94%), its backward 97.8
// (89%); 33 tokens 2.2 to 3.0 us.  More rows in flight a warp (8, or wider columns)
// cost registers and with them warps: 59 to 74 us for combine.
#include <type_traits>

#include "ops_common.cuh"

namespace moe {
namespace {

// A warp's 256 columns of one row, eight to a lane, moved N at a time: 8 where rows
// start on 16 bytes, 2 where rows start and end on pairs, else 1 (lane l then has
// columns N l ..., N (l + 32) ..., so that narrow accesses still coalesce).
constexpr int kCols = 256;

// STREAM: the rows are read once and the results written once, and take no place in
// the caches that others would use.
template <typename T, int N, bool STREAM = false>
struct Lane8 {
  using raw = typename T::raw;
  using pair = std::conditional_t<sizeof(raw) == 2, uint32_t, uint2>;
  alignas(16) raw v[8];
  __device__ __forceinline__ void load(const raw *row, int c0, int H, int lane) {
    if constexpr (N == 8) {
      const int c = c0 + 8 * lane;
      if (c + 8 <= H) {
        uint4 *w = reinterpret_cast<uint4 *>(v);
        const uint4 *p = reinterpret_cast<const uint4 *>(row + c);
#pragma unroll
        for (int i = 0; i < (int)(sizeof(v) / 16); ++i) w[i] = STREAM ? __ldcs(p + i) : __ldg(p + i);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = c + i < H ? __ldg(row + c + i) : raw(0);
      }
    } else if constexpr (N == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = c0 + 64 * i + 2 * lane;
        reinterpret_cast<pair *>(v)[i] = c < H ? __ldg(reinterpret_cast<const pair *>(row + c)) : pair{};
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = c0 + 32 * i + lane;
        v[i] = c < H ? __ldg(row + c) : raw(0);
      }
    }
  }
  __device__ __forceinline__ void store(raw *row, int c0, int H, int lane) const {
    if constexpr (N == 8) {
      const int c = c0 + 8 * lane;
      if (c + 8 <= H) {
        const uint4 *w = reinterpret_cast<const uint4 *>(v);
        uint4 *p = reinterpret_cast<uint4 *>(row + c);
#pragma unroll
        for (int i = 0; i < (int)(sizeof(v) / 16); ++i) {
          if constexpr (STREAM) __stcs(p + i, w[i]);
          else p[i] = w[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (c + i < H) row[c + i] = v[i];
      }
    } else if constexpr (N == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = c0 + 64 * i + 2 * lane;
        if (c < H) *reinterpret_cast<pair *>(row + c) = reinterpret_cast<const pair *>(v)[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = c0 + 32 * i + lane;
        if (c < H) row[c] = v[i];
      }
    }
  }
  __device__ __forceinline__ float get(int i) const { return T::to(v[i]); }
  __device__ __forceinline__ void set(int i, float f) { v[i] = T::from(f); }
};

// ------------------------------------------------------------------ dispatch
struct DispatchArgs {
  const uint8_t *x;
  uint8_t *xs;
  const int *inv;
  int64_t ldx, ldxs;      // bytes
  int T, k, rows, units;  // units of V bytes in a row
  int chunks;             // per row
};

constexpr int kCopyUnits = 4;   // units a lane holds

// A warp copies 32 * kCopyUnits units of one token's row: loaded once, stored to
// each of its pairs.
template <typename V>
__global__ void __launch_bounds__(128) dispatch_kernel(const DispatchArgs a) {
  const int lane = threadIdx.x & 31;
  wait_prior_grid();
  const long long items = (long long)a.T * a.chunks;
  for (long long it = (long long)blockIdx.x * 4 + (threadIdx.x >> 5); it < items; it += (long long)gridDim.x * 4) {
    const long long t = it / a.chunks;
    const int u0 = (int)(it - t * a.chunks) * 32 * kCopyUnits + lane;
    const int pos = lane < a.k ? __ldg(a.inv + t * a.k + lane) : -1;
    const V *src = reinterpret_cast<const V *>(a.x + t * a.ldx);
    V v[kCopyUnits];
#pragma unroll
    for (int i = 0; i < kCopyUnits; ++i)
      if (u0 + 32 * i < a.units) v[i] = __ldg(src + u0 + 32 * i);
    for (int j = 0; j < a.k; ++j) {
      const int r = __shfl_sync(0xffffffffu, pos, j);
      if (r < 0 || r >= a.rows) continue;
      V *dst = reinterpret_cast<V *>(a.xs + (int64_t)r * a.ldxs);
#pragma unroll
      for (int i = 0; i < kCopyUnits; ++i)
        if (u0 + 32 * i < a.units) dst[u0 + 32 * i] = v[i];
    }
  }
}

template <typename V>
cudaError_t launch_dispatch(DispatchArgs a, int64_t row_bytes, cudaStream_t s) {
  a.units = (int)(row_bytes / (int64_t)sizeof(V));
  a.chunks = (a.units + 32 * kCopyUnits - 1) / (32 * kCopyUnits);
  const long long blocks = ((long long)a.T * a.chunks + 3) / 4;
  return launch_op(dispatch_kernel<V>, dim3((unsigned)std::min<long long>(blocks, 1 << 20)), 128, 0, s, a);
}

// ------------------------------------------------------------------- combine
struct CombineOpArgs {
  const void *ys;
  void *y;
  const int *inv;
  const float *gates;     // NULL: ones
  int64_t ldys, ldy;      // elements
  int T, k, rows, H, chunks;
};

// A warp sums 256 columns of one token over its pairs.  The rows of four pairs
// are loaded before the first is used.  (As streams 48.9 us of 8192 x 8, H 2048, bf16,
// else 51.8; the backward pass loses by it, 105 and 98.)
template <typename TI, typename TO, int N>
__global__ void __launch_bounds__(128) combine_op_kernel(const CombineOpArgs a) {
  const int lane = threadIdx.x & 31;
  wait_prior_grid();
  const auto *ys = static_cast<const typename TI::raw *>(a.ys);
  auto *y = static_cast<typename TO::raw *>(a.y);
  const long long items = (long long)a.T * a.chunks;
  for (long long it = (long long)blockIdx.x * 4 + (threadIdx.x >> 5); it < items; it += (long long)gridDim.x * 4) {
    const long long t = it / a.chunks;
    const int c0 = (int)(it - t * a.chunks) * kCols;
    const int pos = lane < a.k ? __ldg(a.inv + t * a.k + lane) : -1;
    const float gate = lane < a.k && a.gates ? __ldg(a.gates + t * a.k + lane) : 1.0f;
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
    for (int j0 = 0; j0 < a.k; j0 += 4) {
      Lane8<TI, N, true> v[4];
      int r[4];
      float g[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        r[u] = __shfl_sync(0xffffffffu, pos, (j0 + u) & 31);
        g[u] = __shfl_sync(0xffffffffu, gate, (j0 + u) & 31);
        if (j0 + u >= a.k || r[u] >= a.rows) r[u] = -1;
        if (r[u] >= 0) v[u].load(ys + (int64_t)r[u] * a.ldys, c0, a.H, lane);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (r[u] < 0) continue;
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = fmaf(g[u], v[u].get(i), acc[i]);
      }
    }
    Lane8<TO, N, true> out;
#pragma unroll
    for (int i = 0; i < 8; ++i) out.set(i, acc[i]);
    out.store(y + t * a.ldy, c0, a.H, lane);
  }
}

template <typename TI, typename TO>
cudaError_t launch_combine_op(CombineOpArgs a, int n, cudaStream_t s) {
  a.chunks = (a.H + kCols - 1) / kCols;
  const long long blocks = std::min<long long>(((long long)a.T * a.chunks + 3) / 4, 1 << 20);
  auto fn = n == 8 ? combine_op_kernel<TI, TO, 8> : n == 2 ? combine_op_kernel<TI, TO, 2> : combine_op_kernel<TI, TO, 1>;
  return launch_op(fn, dim3((unsigned)blocks), 128, 0, s, a);
}

// ---------------------------------------------------------- combine backward
struct CombineBwdArgs {
  const void *dy, *ys;
  void *dys;              // may be NULL
  float *dgates;          // may be NULL
  const int *inv;
  const float *gates;     // NULL: ones
  int64_t lddy, ldys, lddys;
  int T, k, rows, H, chunks, pairs;
};

// A CTA takes one token and `pairs` of its pairs; its warps take the 256-column
// chunks in turn.  A warp keeps its chunk of dy in registers over the token's pairs: the pair's row of ys
// gives a partial of its gate's gradient, gate * dy goes out as its row of dys.
template <typename TD, typename TS, int N>
__global__ void __launch_bounds__(256) combine_bwd_kernel(const CombineBwdArgs a) {
  __shared__ float part[8][kMaxTopK];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, W = blockDim.x >> 5;
  wait_prior_grid();
  const auto *dy = static_cast<const typename TD::raw *>(a.dy);
  const auto *ys = static_cast<const typename TS::raw *>(a.ys);
  auto *dys = static_cast<typename TS::raw *>(a.dys);
  const int jb = blockIdx.y * a.pairs, je = min(a.k, jb + a.pairs);
  for (long long t = blockIdx.x; t < a.T; t += gridDim.x) {
    const int pos = lane < a.k ? __ldg(a.inv + t * a.k + lane) : -1;
    const float gate = lane < a.k && a.gates ? __ldg(a.gates + t * a.k + lane) : 1.0f;
    float mine = 0.0f;                                  // lane j: this warp's part of pair j's dot product
    for (int c = warp; c < a.chunks; c += W) {
      const int c0 = c * kCols;
      Lane8<TD, N> d;
      d.load(dy + t * a.lddy, c0, a.H, lane);
      for (int j0 = jb; j0 < je; j0 += 4) {
        Lane8<TS, N> v[4];
        int r[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          r[u] = __shfl_sync(0xffffffffu, pos, (j0 + u) & 31);
          if (j0 + u >= je || r[u] >= a.rows) r[u] = -1;
          if (r[u] >= 0 && a.dgates) v[u].load(ys + (int64_t)r[u] * a.ldys, c0, a.H, lane);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float g = __shfl_sync(0xffffffffu, gate, (j0 + u) & 31);
          if (r[u] < 0) continue;
          if (a.dgates) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) s = fmaf(d.get(i), v[u].get(i), s);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            if (lane == j0 + u) mine += s;
          }
          if (dys) {
            Lane8<TS, N> out;
#pragma unroll
            for (int i = 0; i < 8; ++i) out.set(i, g * d.get(i));
            out.store(dys + (int64_t)r[u] * a.lddys, c0, a.H, lane);
          }
        }
      }
    }
    if (!a.dgates) continue;
    part[warp][lane] = mine;
    __syncthreads();
    const int j = jb + threadIdx.x;
    if (j < je) {
      float s = 0.0f;
      for (int w = 0; w < W; ++w) s += part[w][j];
      a.dgates[t * a.k + j] = s;
    }
    __syncthreads();
  }
}

template <typename TD, typename TS>
cudaError_t launch_combine_bwd(CombineBwdArgs a, int n, cudaStream_t s) {
  a.chunks = (a.H + kCols - 1) / kCols;
  // eight warps to a token while tokens are few; once they fill the GPU four leave
  // fewer waits at the barrier (8192 tokens x 8, H 2048, bf16: 104 us with 8, 98
  // with 4, 99 with 2; 33 tokens: 4.2, 6.5, 11.5)
  const int W = std::min(a.T >= 8 * sm_count() ? 4 : 8, a.chunks);
  // fewer tokens than SMs: four pairs to a CTA (33 tokens x 8, H 2048, bf16: 3.0 us,
  // with all pairs to a CTA 4.2)
  a.pairs = a.T < sm_count() ? 4 : a.k;
  const dim3 grid((unsigned)std::min(a.T, 1 << 20), (unsigned)((a.k + a.pairs - 1) / a.pairs));
  auto fn = n == 8 ? combine_bwd_kernel<TD, TS, 8> : n == 2 ? combine_bwd_kernel<TD, TS, 2> : combine_bwd_kernel<TD, TS, 1>;
  return launch_op(fn, grid, 32 * W, 0, s, a);
}

// ------------------------------------------------------------ argument checks
moe_status_t check_shape(const char *fn, int32_t T, int32_t k, int32_t H, int32_t rows) {
  if (T < 0 || k < 1 || k > kMaxTopK || H < 1 || H > 1 << 28 || rows < 0)
    return ops_invalid(fn, "need T >= 0, 1 <= k <= 32, 1 <= H <= 2^28 and rows >= 0");
  if ((int64_t)T * k >= (int64_t)1 << 31) return ops_invalid(fn, "T * k must be below 2^31");
  return MOE_OK;
}

// How many elements an access may take where rows of H start at p and every ld.
int at_a_time(const void *p, int64_t ld, int32_t dt, int32_t H) {
  if (!p) return 8;
  const int es = dtype_bytes(dt), al = row_alignment(p, ld * es);
  return al >= 16 ? 8 : al >= 2 * es && H % 2 == 0 ? 2 : 1;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_dispatch(const void *x, int32_t dtype, int32_t T, int32_t k, int32_t H, int64_t ldx,
                          const int32_t *inv, int32_t rows, void *xs, int64_t ldxs, void *stream) {
  static const char fn[] = "moe_dispatch";
  moe_status_t st = check_shape(fn, T, k, H, rows);
  if (st != MOE_OK) return st;
  if (dtype < MOE_DT_F32 || dtype > MOE_DT_U8) return ops_invalid(fn, "dtype must be F32, BF16, F16 or U8");
  if (ldx < H || ldxs < H) return ops_invalid(fn, "ldx and ldxs must be at least H");
  if (T == 0 || rows == 0) return MOE_OK;
  if (!x || !inv || !xs) return ops_invalid(fn, "x, inv and xs must be device pointers");
  const int es = dtype_bytes(dtype);
  if (!aligned_to(x, es) || !aligned_to(xs, es)) return ops_invalid(fn, "x and xs must be aligned to their type");
  DispatchArgs a{};
  a.x = static_cast<const uint8_t *>(x);
  a.xs = static_cast<uint8_t *>(xs);
  a.inv = inv;
  a.ldx = ldx * es; a.ldxs = ldxs * es;
  a.T = T; a.k = k; a.rows = rows;
  const int64_t row_bytes = (int64_t)H * es;
  // the widest unit that every row starts and ends on
  const int v = std::min({16, row_alignment(x, a.ldx), row_alignment(xs, a.ldxs), row_alignment(nullptr, row_bytes)});
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = v == 16  ? launch_dispatch<uint4>(a, row_bytes, s)
                  : v == 8 ? launch_dispatch<uint2>(a, row_bytes, s)
                  : v == 4 ? launch_dispatch<uint32_t>(a, row_bytes, s)
                  : v == 2 ? launch_dispatch<uint16_t>(a, row_bytes, s)
                           : launch_dispatch<uint8_t>(a, row_bytes, s);
  return ops_launched(fn, e);
}

static moe_status_t combine_rows(const char *fn, const void *ys, int32_t ti, int32_t rows, int32_t T, int32_t k,
                                 int32_t H, int64_t ldys, const int32_t *inv, const float *gates, void *y, int32_t to,
                                 int64_t ldy, void *stream) {
  moe_status_t st = check_shape(fn, T, k, H, rows);
  if (st != MOE_OK) return st;
  if (!is_float_dtype(ti) || !is_float_dtype(to)) return ops_invalid(fn, "dtypes must be F32, BF16 or F16");
  if (ldys < H || ldy < H) return ops_invalid(fn, "row strides must be at least H");
  if (T == 0) return MOE_OK;
  if ((!ys && rows > 0) || !inv || !y) return ops_invalid(fn, "rows, inv and the output must be device pointers");
  if (!aligned_to(ys, dtype_bytes(ti)) || !aligned_to(y, dtype_bytes(to)))
    return ops_invalid(fn, "rows and the output must be aligned to their type");
  CombineOpArgs a{ys, y, inv, gates, ldys, ldy, T, k, rows, H, 0};
  const int n = std::min(at_a_time(ys, ldys, ti, H), at_a_time(y, ldy, to, H));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
#define MOE_CASE(I, TI) \
  (to == MOE_DT_F32 ? launch_combine_op<TI, F32>(a, n, s) : to == MOE_DT_BF16 ? launch_combine_op<TI, BF16>(a, n, s) \
                                                                                 : launch_combine_op<TI, F16>(a, n, s))
  e = ti == MOE_DT_F32 ? MOE_CASE(0, F32) : ti == MOE_DT_BF16 ? MOE_CASE(1, BF16) : MOE_CASE(2, F16);
#undef MOE_CASE
  return ops_launched(fn, e);
}

moe_status_t moe_dispatch_backward(const void *dxs, int32_t dtype, int32_t rows, int32_t T, int32_t k, int32_t H,
                                   int64_t lddxs, const int32_t *inv, void *dx, int64_t lddx, void *stream) {
  return combine_rows("moe_dispatch_backward", dxs, dtype, rows, T, k, H, lddxs, inv, nullptr, dx, dtype, lddx, stream);
}

moe_status_t moe_combine(const void *ys, int32_t ys_dtype, int32_t rows, int32_t T, int32_t k, int32_t H,
                         int64_t ldys, const int32_t *inv, const float *gates, void *y, int32_t y_dtype, int64_t ldy,
                         void *stream) {
  return combine_rows("moe_combine", ys, ys_dtype, rows, T, k, H, ldys, inv, gates, y, y_dtype, ldy, stream);
}

moe_status_t moe_combine_backward(const void *dy, int32_t dy_dtype, int64_t lddy, const void *ys, int32_t ys_dtype,
                                  int64_t ldys, int32_t rows, int32_t T, int32_t k, int32_t H, const int32_t *inv,
                                  const float *gates, void *dys, int64_t lddys, float *dgates, void *stream) {
  static const char fn[] = "moe_combine_backward";
  moe_status_t st = check_shape(fn, T, k, H, rows);
  if (st != MOE_OK) return st;
  if (!is_float_dtype(dy_dtype) || !is_float_dtype(ys_dtype)) return ops_invalid(fn, "dtypes must be F32, BF16 or F16");
  if (T == 0) return MOE_OK;
  if (!dys && !dgates) return ops_invalid(fn, "dys and dgates are both NULL");
  if (lddy < H || (dgates && ldys < H) || (dys && lddys < H)) return ops_invalid(fn, "row strides must be at least H");
  if (!dy || !inv || (dgates && !ys && rows > 0)) return ops_invalid(fn, "dy, inv and ys must be device pointers");
  if (!aligned_to(dy, dtype_bytes(dy_dtype)) || !aligned_to(ys, dtype_bytes(ys_dtype)) ||
      !aligned_to(dys, dtype_bytes(ys_dtype)))
    return ops_invalid(fn, "dy, ys and dys must be aligned to their type");
  CombineBwdArgs a{dy, ys, dys, dgates, inv, gates, lddy, ldys, lddys, T, k, rows, H, 0, 0};
  const int n = std::min({at_a_time(dy, lddy, dy_dtype, H), dgates ? at_a_time(ys, ldys, ys_dtype, H) : 8,
                          at_a_time(dys, lddys, ys_dtype, H)});
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
#define MOE_CASE(TD)                                                                                       \
  (ys_dtype == MOE_DT_F32 ? launch_combine_bwd<TD, F32>(a, n, s)                                         \
                          : ys_dtype == MOE_DT_BF16 ? launch_combine_bwd<TD, BF16>(a, n, s)              \
                                                    : launch_combine_bwd<TD, F16>(a, n, s))
  e = dy_dtype == MOE_DT_F32 ? MOE_CASE(F32) : dy_dtype == MOE_DT_BF16 ? MOE_CASE(BF16) : MOE_CASE(F16);
#undef MOE_CASE
  return ops_launched(fn, e);
}

}  // extern "C"
