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
  int *err;                      // the device's error word (an ErrWord), which the waits poll
  int *err_host;                 // its mirror in mapped host memory
  int rows, groups, N, K;
  int nsf;                       // scales in a row
  int sf_mode;                   // 0: a stage's scales in one load, 1: words of four, 2: bytes
  int sf_wide;                   // 1: scale rows start on 16 bytes and are whole stages
  int dtype;
  int y_vec;                     // rows of y start on 16 bytes
};

// The error word knows its mirror; every CTA says so before it waits for anything.
__device__ __forceinline__ void mm_set_mirror(const MatmulArgs &a) {
  reinterpret_cast<ErrWord *>(a.err)->host = a.err_host;
}

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
  if (!a.offsets) {                                        // one group of all rows: no scan
    if (tid == 0) {
      t.begin[0] = 0;
      t.end[0] = a.rows;
      t.tiles[0] = 0;
      t.tiles[1] = (a.rows + NT - 1) / NT;
    }
    return;
  }
  const int per = (a.groups + n - 1) / n;
  const int g0 = min(a.groups, tid * per), g1 = min(a.groups, g0 + per);
  int sum = 0;
  for (int g = g0; g < g1; ++g) {
    const int b = min(max(__ldg(a.offsets + g), 0), a.rows);
    const int e = min(max(__ldg(a.offsets + g + 1), 0), a.rows);
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
  int through = lane < n / 32 ? t.wsum[lane] : 0;          // every warp scans the warps' sums for itself
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, through, o);
    if (lane >= o) through += v;
  }
  const int prior = __shfl_sync(0xffffffffu, through, (warp + 31) & 31);
  const int earlier = (warp ? prior : 0) + inc - sum;
  for (int g = g0; g < g1; ++g) t.tiles[g] += earlier;
  if (tid == n - 1) t.tiles[a.groups] = earlier + sum;
}

// A warp's walk over the items first, first + step, ...: item = tile * nrb + row
// block, the tiles in group order.  Whole warps walk (the groups are searched 32
// at a time); values are warp-uniform.
template <int NT>
struct MmWalk {
  int g, row0, nrows, rb;        // of the item: group, first row, rows, block of weight rows
  int tile, dtile, drb, nrb, ntiles;
  // step 0: the first item alone
  __device__ __forceinline__ MmWalk(const MatmulArgs &a, const MmGroups &t, int nrb_, unsigned first, unsigned step)
      : g(0), nrb(nrb_), ntiles(t.tiles[a.groups]) {
    tile = (int)(first / (unsigned)nrb);
    rb = (int)(first - (unsigned)(tile * nrb));
    dtile = step ? (int)(step / (unsigned)nrb) : ntiles;
    drb = step ? (int)(step - (unsigned)(dtile * nrb)) : 0;
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

// Scales come 32 bytes of a row at a time, a whole sector of memory: AHEAD stages.
template <int WF>
constexpr int kSfWords = WF == WF_MX ? 2 : 4;              // words of scales a row has in a stage
template <int WF>
constexpr int kSfAhead = 8 / kSfWords<WF>;

// 32 bytes of four rows' scales from stage it0 on (as far as stage k1).
template <int WF>
__device__ __forceinline__ void fetch_sf(const MatmulArgs &a, const uint8_t *const (&row)[4], int rows, int it0, int k1,
                                         uint32_t (&w)[4][8]) {
  constexpr int WORDS = kSfWords<WF>, AHEAD = kSfAhead<WF>;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (j >= rows) break;
    if (a.sf_wide && it0 + AHEAD <= k1) {
      const uint4 *p = reinterpret_cast<const uint4 *>(row[j] + it0 * 4 * WORDS);
      const uint4 lo = __ldg(p), hi = __ldg(p + 1);
      w[j][0] = lo.x; w[j][1] = lo.y; w[j][2] = lo.z; w[j][3] = lo.w;
      w[j][4] = hi.x; w[j][5] = hi.y; w[j][6] = hi.z; w[j][7] = hi.w;
      continue;
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (it0 + i < k1) load_sf<WORDS>(row[j], it0 + i, a.nsf, a.sf_mode, kSfOne<WF>, &w[j][i * WORDS]);
  }
}

// A scale warp's work: of the sequence (item, steps of AHEAD stages in [k0, k1)) it
// takes every `stride`-th step from `phase` on, loads the next of them while it
// stores the last.  rows_of(walk) sets the row pointers of an item; put(walk) gives
// the function that stores stage i of a step of that item into ring place s.
// A step's stages are stored one by one, or (BATCH) all before the one fence that
// shows them to the tensor core, which costs some 500 clocks: with a ring of two
// steps and more the copies lose nothing by it.
template <int WF, int S, bool BATCH, typename Walk, typename RowsOf, typename Fetch, typename Wait, typename Put,
          typename Arrive>
__device__ __forceinline__ void feed_scales(const MatmulArgs &a, const MmGroups &t, Walk m, int k0, int k1, int phase,
                                            int stride, RowsOf rows_of, Fetch fetch, Wait wait_empty, Put put,
                                            Arrive arrive) {
  constexpr int AHEAD = kSfAhead<WF>;
  int it0 = k0, seq = 0;                                   // seq: stages before this step, over all items
  bool more = m.more() && k1 > k0;
  auto advance = [&]() {
    seq += min(AHEAD, k1 - it0);
    it0 += AHEAD;
    if (it0 < k1) return;
    it0 = k0;
    m.next(a, t);
    more = m.more();
    if (more) rows_of(m);
  };
  if (more) rows_of(m);
  for (int i = 0; i < phase && more; ++i) advance();
  uint32_t cur[4][8];
  if (more) fetch(it0, cur);
  while (more) {
    uint32_t hold[4][8];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) hold[j][i] = cur[j][i];
    const int stages = min(AHEAD, k1 - it0), first = seq;
    const auto ticket = put(m);                            // what put has to know of the step's item
    for (int i = 0; i < stride && more; ++i) advance();
    if (more) fetch(it0, cur);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      if (i >= stages) break;
      const int s = (first + i) % S, round = (first + i) / S;
      if (round > 0 && !wait_empty(s, (round - 1) & 1)) return;
      ticket(s, hold, i);
      if (BATCH) continue;
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      arrive(s);
    }
    if (!BATCH) continue;
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    for (int i = 0; i < stages; ++i) arrive((first + i) % S);
  }
}

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
