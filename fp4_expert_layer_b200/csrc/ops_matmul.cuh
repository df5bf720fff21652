// ops_matmul.cuh -- what the two kernels of the grouped FP4 product share: the
// arguments, the list of work items, the scales' way into registers, the store.
#pragma once

#include <cooperative_groups.h>

#include "ops_common.cuh"
#include "tcgen05.cuh"
#include "tma.cuh"

namespace moe {

constexpr int kMmMaxGroups = 1024;
constexpr int kMmMaxRows = 1 << 27;   // the tile counts of 1024 groups then add up below 2^31

struct MatmulArgs {
  CUtensorMap xmap, wmap;
  const uint8_t *xs, *ws;        // block scales
  const float *xG, *wG;          // NVFP4 only
  const int *offsets;            // NULL: one group of all rows
  void *y;
  int64_t ldy;
  int *err;
  int rows, groups, N, K;
  int nsf;                       // scales in a row
  int sf_mode;                   // 0: a stage's scales in one load, 1: words of four, 2: bytes
  int sf_wide;                   // 1: scale rows start on 16 bytes and are whole stages
  int dtype;
  int y_vec;                     // rows of y start on 16 bytes
};

// ------------------------------------------------------------------ work items
// Tables of the groups in shared memory: rows [begin, end) and the tiles before.
struct MmGroups {
  int begin[kMmMaxGroups], end[kMmMaxGroups];
  int tiles[kMmMaxGroups + 1];
  int wsum[32];
};

// Every CTA makes the tables for itself: thread t takes `per` consecutive groups.
// Called by all threads; offsets are cut to [0, rows].
template <int NT>
__device__ __forceinline__ void mm_scan_groups(const MatmulArgs &a, MmGroups &t) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = blockDim.x;
  const int per = (a.groups + n - 1) / n;
  const int g0 = min(a.groups, tid * per), g1 = min(a.groups, g0 + per);
  int sum = 0;
  for (int g = g0; g < g1; ++g) {
    const int b = a.offsets ? min(max(__ldg(a.offsets + g), 0), a.rows) : 0;
    const int e = a.offsets ? min(max(__ldg(a.offsets + g + 1), 0), a.rows) : a.rows;
    t.begin[g] = b;
    t.end[g] = max(b, e);
    t.tiles[g] = sum;
    sum += (max(b, e) - b + NT - 1) / NT;
  }
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) t.wsum[warp] = inc;
  __syncthreads();
  int earlier = inc - sum, all = 0;
  for (int w = 0; w < n / 32; ++w) {
    if (w < warp) earlier += t.wsum[w];
    all += t.wsum[w];
  }
  for (int g = g0; g < g1; ++g) t.tiles[g] += earlier;
  if (tid == 0) t.tiles[a.groups] = all;
}

// A warp's walk over the items first, first + step, ...: item = tile * nrb + row
// block, the tiles in group order.  Whole warps walk (the groups are searched 32
// at a time); values are warp-uniform.
template <int NT>
struct MmWalk {
  int g, row0, nrows, rb;        // of the item: group, first row, rows, block of weight rows
  int tile, dtile, drb, nrb, ntiles;
  __device__ __forceinline__ MmWalk(const MatmulArgs &a, const MmGroups &t, int nrb_, long long first, long long step)
      : g(0), nrb(nrb_), ntiles(t.tiles[a.groups]) {
    tile = (int)(first / nrb);
    rb = (int)(first - (long long)tile * nrb);
    dtile = (int)(step / nrb);
    drb = (int)(step - (long long)dtile * nrb);
    find(a, t);
  }
  __device__ __forceinline__ bool more() const { return tile < ntiles; }
  __device__ __forceinline__ void next(const MatmulArgs &a, const MmGroups &t) {
    tile += dtile;
    rb += drb;
    if (rb >= nrb) {
      rb -= nrb;
      ++tile;
    }
    find(a, t);
  }
  __device__ __forceinline__ void find(const MatmulArgs &a, const MmGroups &t) {
    if (!more()) return;
    const int lane = threadIdx.x & 31;
    while (true) {               // the last group that starts at or before the tile
      const int c = g + 1 + lane;
      const unsigned passed = __ballot_sync(0xffffffffu, c < a.groups && t.tiles[c] <= tile);
      g += __popc(passed);
      if (passed != 0xffffffffu) break;
    }
    row0 = t.begin[g] + (tile - t.tiles[g]) * NT;
    nrows = min(NT, t.end[g] - row0);
  }
};

// ---------------------------------------------------------------------- scales
// The scales of one row for one stage (K elements 256 * it ..): WORDS words.
// Columns past the row's end read as 1.0 (their codes are zero).
template <int WORDS>
__device__ __forceinline__ void load_sf(const uint8_t *row, int it, int nsf, int mode, uint32_t fill, uint32_t *w) {
  const int c0 = it * WORDS * 4;
  if (mode == 0) {
    if constexpr (WORDS == 4) {
      const uint4 v = __ldg(reinterpret_cast<const uint4 *>(row + c0));
      w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else {
      const uint2 v = __ldg(reinterpret_cast<const uint2 *>(row + c0));
      w[0] = v.x; w[1] = v.y;
    }
  } else if (mode == 1) {
#pragma unroll
    for (int i = 0; i < WORDS; ++i)
      w[i] = c0 + 4 * i < nsf ? __ldg(reinterpret_cast<const uint32_t *>(row + c0 + 4 * i)) : fill;
  } else {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) {
      w[i] = 0;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int c = c0 + 4 * i + b;
        w[i] |= (c < nsf ? (uint32_t)__ldg(row + c) : (fill & 0xFFu)) << (8 * b);
      }
    }
  }
}
template <int WF>
constexpr uint32_t kSfOne = WF == WF_MX ? 0x7F7F7F7Fu : 0x38383838u;

__device__ __forceinline__ void store_out(void *y, int dtype, int64_t at, float v) {
  if (dtype == MOE_DT_F32) static_cast<float *>(y)[at] = v;
  else if (dtype == MOE_DT_BF16) static_cast<uint16_t *>(y)[at] = bf16_bits(v);
  else static_cast<uint16_t *>(y)[at] = f16_bits(v);
}

// The pair kernel (ops_matmul_pair.cu): items of 256 rows x 256 weight rows.
cudaError_t launch_matmul_pair(int wf, const MatmulArgs &a, int pairs, cudaStream_t s);
constexpr int kPairRows = 256;        // rows of a token tile
constexpr int kPairBox = 64;          // rows of its TMA boxes

}  // namespace moe
