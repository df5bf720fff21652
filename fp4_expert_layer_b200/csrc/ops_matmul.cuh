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
constexpr int kMmMaxSide = 1 << 30;   // N and K: rounded up to tiles and stages they stay below 2^31

struct MatmulArgs {
  CUtensorMap xmap, wmap;
  const uint8_t *xs, *ws;        // block scales
  const float *xG, *wG;          // NVFP4 only
  const int *offsets;            // NULL: one group of all rows
  void *y;
  int64_t ldy;
  int *err;                      // the device's error word, in mapped host memory: written by waits that gave up
  int rows, groups, N, K;
  int tile_log;                  // a token tile has 2^tile_log rows
  int nsf;                       // scales in a row
  int sf_wide;                   // 1: scale rows start on 16 bytes
  int dtype;
  int y_vec;                     // rows of y start on 16 bytes
  int rank_log;                  // 2^rank_log CTAs of a cluster share an item's K
};

// Bounded wait for phase `parity` of a barrier.  A wait that reaches its limit says so
// in its CTA's flag, so that the CTA's other waits end too, and in the device's error
// word, which the next call of the host reads.  Nothing that outlives the CTA is
// polled: a launch that fails cannot end a wait of another launch, of its own next
// replay, or of a CTA that works.
//
// The limit is kWaitLimitNs, and 4 us more for each stage that is waited for: a wait for
// an accumulator lasts as long as its item's K range, and 2^30 elements are 4 M stages of
// some 0.4 us (100 groups of two rows each, N 1: 1.7 s).
__device__ __forceinline__ bool mm_wait(uint32_t bar, uint32_t parity, int *gave_up, int *err, int code, int stages = 0,
                                        unsigned long long limit = kWaitLimitNs) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = global_ns();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 255u) == 0) {
      if (*(volatile int *)gave_up != 0) return false;
      if (global_ns() - t0 > limit + 4000ull * (unsigned)stages) {
        *(volatile int *)gave_up = 1;
        *(volatile int *)err = code;
        __threadfence_system();
        return false;
      }
    }
  }
}
// The same by every lane of a warp, true only when it succeeded for all of them.
__device__ __forceinline__ bool mm_wait_warp(uint32_t bar, uint32_t parity, int *gave_up, int *err, int code,
                                             int stages = 0, unsigned long long limit = kWaitLimitNs) {
  return __all_sync(0xffffffffu, mm_wait(bar, parity, gave_up, err, code, stages, limit));
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
__device__ __forceinline__ void mm_scan_groups(const MatmulArgs &a, MmGroups &t) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = blockDim.x;
  if (!a.offsets) {                                        // one group of all rows: no scan
    if (tid == 0) {
      t.begin[0] = 0;
      t.end[0] = a.rows;
      t.tiles[0] = 0;
      t.tiles[1] = (a.rows + (1 << a.tile_log) - 1) >> a.tile_log;
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
    sum += (max(b, e) - b + (1 << a.tile_log) - 1) >> a.tile_log;
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
    row0 = t.begin[g] + ((tile - t.tiles[g]) << a.tile_log);
    nrows = min(1 << a.tile_log, t.end[g] - row0);
  }
};

// ---------------------------------------------------------------------- scales
// Rows of scales lie where nsf bytes a row put them: at any byte.  A lane reads 32
// bytes of a row at a time, a whole sector of memory.

// The aligned 16-byte pieces that hold the n bytes (up to 32) from p on.
__device__ __forceinline__ void load_pieces(const uint8_t *p, int n, uint4 (&v)[3]) {
  const int off = (int)(reinterpret_cast<uintptr_t>(p) & 15u);
  const uint4 *q = reinterpret_cast<const uint4 *>(p - off);
#pragma unroll
  for (int j = 0; j < 3; ++j) v[j] = 16 * j < off + n ? __ldg(q + j) : make_uint4(0u, 0u, 0u, 0u);
}
// Those bytes out of them, then `fill`, as eight words.
__device__ __forceinline__ void shift_pieces(const uint8_t *p, int n, const uint4 (&v)[3], uint32_t fill,
                                             uint32_t (&out)[8]) {
  const int off = (int)(reinterpret_cast<uintptr_t>(p) & 15u);
  uint32_t w[12];
#pragma unroll
  for (int j = 0; j < 3; ++j) { w[4 * j] = v[j].x; w[4 * j + 1] = v[j].y; w[4 * j + 2] = v[j].z; w[4 * j + 3] = v[j].w; }
#pragma unroll
  for (int i = 0; i < 11; ++i) w[i] = off & 4 ? w[i + 1] : w[i];
#pragma unroll
  for (int i = 0; i < 9; ++i) w[i] = off & 8 ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < 8; ++i) out[i] = __funnelshift_r(w[i], w[i + 1], 8 * (off & 3));
  if (n == 32) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int have = min(max(n - 4 * i, 0), 4);
    const uint32_t mask = have == 4 ? 0xFFFFFFFFu : (1u << (8 * have)) - 1u;
    out[i] = (out[i] & mask) | (fill & ~mask);
  }
}

// A scale of 1.0 four times: what the columns past a row's end have (their codes are zero).
template <int WF>
constexpr uint32_t kSfOne = WF == WF_MX ? 0x7F7F7F7Fu : 0x38383838u;

template <int WF>
constexpr int kSfWords = WF == WF_MX ? 2 : 4;              // words of scales a row has in a stage
template <int WF>
constexpr int kSfAhead = 8 / kSfWords<WF>;                 // stages that 32 bytes of scales are

// 32 bytes of `rows` (up to four) rows' scales from stage it0 on, as far as stage k1.
// WIDE: scale rows start on 16 bytes.
template <int WF, bool WIDE>
__device__ __forceinline__ void fetch_sf(const MatmulArgs &a, const uint8_t *const (&row)[4], int rows, int it0, int k1,
                                         const uint8_t *lo, const uint8_t *hi, uint32_t (&w)[4][8]) {
  const int c0 = it0 * 4 * kSfWords<WF>, n = min(32, min(k1 * 4 * kSfWords<WF>, a.nsf) - c0);
  if constexpr (WIDE) {                                    // n is a multiple of 8; rows go on in 16s
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j >= rows) break;
      const uint4 *p = reinterpret_cast<const uint4 *>(row[j] + c0);
      const uint4 one = make_uint4(kSfOne<WF>, kSfOne<WF>, kSfOne<WF>, kSfOne<WF>);
      const uint4 x = __ldg(p), y = n > 16 ? __ldg(p + 1) : one;
      w[j][0] = x.x; w[j][1] = x.y; w[j][2] = x.z; w[j][3] = x.w;
      w[j][4] = y.x; w[j][5] = y.y; w[j][6] = y.z; w[j][7] = y.w;
    }
    return;
  }
  // do the pieces reach past the scales' ends?
  bool past = false;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (j >= rows) break;
    const uint8_t *p = row[j] + c0;
    const int off = (int)(reinterpret_cast<uintptr_t>(p) & 15u);
    past = past || p - off < lo || p - off + (off + n + 15) / 16 * 16 > hi;
  }
  if (!__any_sync(0xffffffffu, past)) {
#pragma unroll
    for (int j = 0; j < 4; j += 2) {                       // two rows' loads in flight together
      if (j >= rows) break;
      uint4 v0[3], v1[3];
      load_pieces(row[j] + c0, n, v0);
      if (j + 1 < rows) load_pieces(row[j + 1] + c0, n, v1);
      shift_pieces(row[j] + c0, n, v0, kSfOne<WF>, w[j]);
      if (j + 1 < rows) shift_pieces(row[j + 1] + c0, n, v1, kSfOne<WF>, w[j + 1]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {                          // byte by byte: the first and last rows alone
      if (j >= rows) break;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        w[j][i] = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b)
          w[j][i] |= (4 * i + b < n ? (uint32_t)__ldg(row[j] + c0 + 4 * i + b) : kSfOne<WF> & 0xFFu) << (8 * b);
      }
    }
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

// The two global scales of a result as one factor, xG wG: rounded once, which is
// harmless while it is a normal number.  Where it is not (2^-75 and 2^-80; 2^70 and
// 2^80 with a sum of 0) the result may still be one, and scaled() takes the scales
// one by one in 64 bits, where nothing between 2^-320 and 2^320 is lost.
__device__ __forceinline__ bool whole_factor(float f) {
  const uint32_t e = __float_as_uint(f) & 0x7F800000u;
  return e != 0u && e != 0x7F800000u;
}
__device__ __forceinline__ float scaled(float sum, float xG, float wG) {
  return (float)((double)sum * ((double)xG * (double)wG));
}

__device__ __forceinline__ void store_out(void *y, int dtype, int64_t at, float v) {
  if (dtype == MOE_DT_F32) static_cast<float *>(y)[at] = v;
  else if (dtype == MOE_DT_BF16) static_cast<uint16_t *>(y)[at] = bf16_bits(v);
  else static_cast<uint16_t *>(y)[at] = f16_bits(v);
}

// n columns of an accumulator from `acc` on, token rows row0 ..., to column `col` of y,
// where a factor is not whole: one by one, since it is seldom and the way that all
// others take is short of registers (as a branch inside it the pair kernel took 73 us
// instead of 66, 16384 rows over 128 groups).
__device__ __forceinline__ void store_far(const MatmulArgs &a, uint32_t acc, int row0, int n, int col, float wG) {
#pragma unroll 1
  for (int j = 0; j < n; ++j) {
    const uint32_t d = tmem_ld1(acc + (uint32_t)j);
    tmem_ld_wait();
    if (col < a.N)
      store_out(a.y, a.dtype, (int64_t)(row0 + j) * a.ldy + col, scaled(__uint_as_float(d), __ldg(a.xG + row0 + j), wG));
    __syncwarp();
  }
}

// The pair kernel (ops_matmul_pair.cu): items of 64, 128 or 256 rows x 256 weight rows.
cudaError_t launch_matmul_pair(int wf, const MatmulArgs &a, int pairs, cudaStream_t s);
constexpr int kPairRows = 256;        // rows of a token tile at most
constexpr int kPairBox = 64;          // rows of its TMA boxes

}  // namespace moe
