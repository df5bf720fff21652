// ops_sort.cu -- pairs (token, choice) sorted by expert: a stable counting sort.
//
//   counts[e] = #{p : ids[p] = e},  offsets = exclusive scan of counts,
//   inv[p] = offsets[ids[p]] + #{q < p : ids[q] = ids[p]},  perm[inv[p]] = p.
//
// Every warp owns a contiguous range of pairs.  It counts its range into a
// histogram of its own (a row of shared memory; the lanes of one step that hold
// the same expert find one another with ballots), which gives each pair its place
// among its expert's pairs of the range; the histograms are scanned over the warps
// of a CTA, over the CTAs, and over the experts; then the pairs are put in place.
// No atomic decides an order: it is that of the pairs.
//
// Few pairs: one launch of one thread-block cluster, the CTAs' counts meeting in
// distributed shared memory.  Many: eight SMs are too few for the counting (some
// 70 clocks a warp's step an SM, and scattered stores), so chunks of pairs go to
// all SMs in three launches: count, scan over the chunks, place.  The chunks'
// counts wait in inv, each in its own chunk's part, which that chunk's CTA reads
// before it writes there, so there is no workspace either.
//
// Bound by latency: 12 bytes a pair are nothing next to the launches.  264 pairs 2.8
// us, 12K 7.0, 82K of 512 experts 8.1 (one cluster: 19), 524K 14 (81).
#include <cooperative_groups.h>

#include "ops_common.cuh"

namespace cg = cooperative_groups;

namespace moe {
namespace {

constexpr int kSortMaxCluster = 8;      // the portable cluster size
// Pairs from which the three launches are faster: 7.2 us against 8.1 at 16384 pairs
// of 512 experts, 8.8 against 6.9 at 12282 of 256.
constexpr int kSortChunked = 16384;

struct SortArgs {
  const int *ids;
  int n, E;
  int *counts, *offsets, *perm, *inv;
  int chunk, chunks;                    // pairs of a chunk; the last one has the remainder too
};

// shared memory: hist[W][E], total[E] (this CTA's counts), base[E], wsum[32]
inline size_t sort_smem(int E, int W) { return ((size_t)(W + 2) * E + 32) * sizeof(int); }

// The lanes that hold the same expert: one ballot for each bit of it.  match_any
// takes a turn for each value a warp holds, some 60 clocks a step.
__device__ __forceinline__ unsigned same_expert(int e, int bits) {
  unsigned other = 0;
#pragma unroll
  for (int b = 0; b < 11; ++b)
    if (b < bits) other |= __ballot_sync(0xffffffffu, e & (1 << b)) ^ (unsigned)((e << (31 - b)) >> 31);
  return ~other;
}
__device__ __forceinline__ int warp_scan(int v, int lane) {   // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  return v;
}

// The CTA's warps count the pairs [lo, hi): afterwards hist[w][e] is the number of
// expert e's pairs in the ranges of the warps before w, total[e] the CTA's, and
// inv[p] the place of p in its warp's range.  W warps, `steps` of 32 pairs to each.
__device__ __forceinline__ void count_pairs(const SortArgs &a, int lo, int hi, int steps, int *hist, int *total) {
  const int E = a.E, W = blockDim.x >> 5, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const unsigned below = (1u << lane) - 1u;
  const int bits = 32 - __clz(E);                      // dropped pairs count as expert E
  int *mine = hist + warp * E;
  const int p0 = (int)min((long long)hi, lo + (long long)warp * steps * 32);
  const int p1 = (int)min((long long)hi, p0 + (long long)steps * 32);
  int next = p0 + lane < p1 ? __ldg(a.ids + p0 + lane) : -1;
#pragma unroll 1
  for (int p = p0; p < p1; p += 32) {
    const int e = next < 0 || next >= E ? E : next;
    next = p + 32 + lane < p1 ? __ldg(a.ids + p + 32 + lane) : -1;
    const unsigned same = same_expert(e, bits);
    const int ahead = __popc(same & below);
    const int place = e < E ? mine[e] + ahead : 0;
    __syncwarp();
    if (e < E && ahead == 0) mine[e] += __popc(same);
    __syncwarp();
    if (p + lane < p1) a.inv[p + lane] = place;
  }
  __syncthreads();
  for (int e = tid; e < E; e += blockDim.x) {          // over the warps, eight loads at a time
    int run = 0;
    for (int w = 0; w < W; w += 8) {
      int c[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) c[u] = w + u < W ? hist[(w + u) * E + e] : 0;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if (w + u < W) hist[(w + u) * E + e] = run;
        run += c[u];
      }
    }
    total[e] = run;
  }
}

// Exclusive scan over the experts of all[e] (every thread's `per` of them summed in
// `sum`): the sum before this thread's first one, and everything.
__device__ __forceinline__ int before_mine(int sum, int *wsum, int *everything) {
  const int W = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int inc = warp_scan(sum, lane);
  if (lane == 31) wsum[warp] = inc;
  __syncthreads();
  const int through = warp_scan(lane < W ? wsum[lane] : 0, lane);   // every warp scans the sums for itself
  *everything = __shfl_sync(0xffffffffu, through, 31);
  const int prior = __shfl_sync(0xffffffffu, through, (warp + 31) & 31);
  return (warp ? prior : 0) + inc - sum;
}

// The warp's pairs to their places: base[e] + hist[w][e] + place.
__device__ __forceinline__ void put_pairs(const SortArgs &a, int lo, int hi, int steps, const int *hist,
                                          const int *base) {
  const int E = a.E, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int *mine = hist + warp * E;
  const int p0 = (int)min((long long)hi, lo + (long long)warp * steps * 32);
  const int p1 = (int)min((long long)hi, p0 + (long long)steps * 32);
#pragma unroll 4
  for (int p = p0 + lane; p < p1; p += 32) {
    const int e = __ldg(a.ids + p);
    const bool kept = e >= 0 && e < E;
    const int at = kept ? base[e] + mine[e] + a.inv[p] : -1;
    a.inv[p] = at;
    if (kept) a.perm[at] = p;
  }
}

// ----------------------------------------------------------- one cluster
__global__ void __launch_bounds__(512) sort_pairs_kernel(const SortArgs a) {
  extern __shared__ int sm[];
  const int E = a.E, W = blockDim.x >> 5, tid = threadIdx.x, NT = blockDim.x;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  int *hist = sm, *total = sm + (size_t)W * E, *base = total + E, *wsum = base + E;

  for (int i = tid; i < W * E; i += NT) hist[i] = 0;
  wait_prior_grid();
  __syncthreads();
  const int steps = ((a.n + 31) / 32 + C * W - 1) / (C * W);
  const int lo = (int)min((long long)a.n, (long long)rank * W * steps * 32);
  const int hi = (int)min((long long)a.n, lo + (long long)W * steps * 32);
  count_pairs(a, lo, hi, steps, hist, total);
  if (C > 1) cluster.sync(); else __syncthreads();

  const int per = (E + NT - 1) / NT, e0 = min(E, tid * per), e1 = min(E, e0 + per);
  int sum = 0;
  for (int e = e0; e < e1; ++e) {
    int c[kSortMaxCluster];
#pragma unroll
    for (int q = 0; q < kSortMaxCluster; ++q)
      c[q] = q >= C ? 0 : C > 1 ? *cluster.map_shared_rank(total + e, q) : total[e];
    int before = 0, all = 0;
#pragma unroll
    for (int q = 0; q < kSortMaxCluster; ++q) {
      before += q < rank ? c[q] : 0;
      all += c[q];
    }
    base[e] = before + sum;
    if (rank == 0) a.counts[e] = all;
    sum += all;
  }
  int everything;
  const int earlier = before_mine(sum, wsum, &everything);
  for (int e = e0; e < e1; ++e) {
    base[e] += earlier;
    if (rank == 0) a.offsets[e] = base[e];             // rank 0 has nothing before it
  }
  if (rank == 0 && tid == 0) a.offsets[E] = everything;
  __syncthreads();
  put_pairs(a, lo, hi, steps, hist, base);
  for (long long p = everything + (long long)rank * NT + tid; p < a.n; p += (long long)C * NT) a.perm[p] = -1;
  if (C > 1) cluster.sync();                           // no CTA leaves while another reads its counts
}

// ----------------------------------------------------------- three launches
constexpr int kChunkThreads = 512;

__device__ __forceinline__ int chunk_begin(const SortArgs &a, int c) { return c * a.chunk; }
__device__ __forceinline__ int chunk_end(const SortArgs &a, int c) { return c + 1 == a.chunks ? a.n : (c + 1) * a.chunk; }

// Each chunk's counts, into the first E entries of its part of inv.
__global__ void __launch_bounds__(kChunkThreads) sort_count_kernel(const SortArgs a) {
  __shared__ int hist[kMaxExperts];
  const int lo = chunk_begin(a, blockIdx.x), hi = chunk_end(a, blockIdx.x);
  for (int e = threadIdx.x; e < a.E; e += kChunkThreads) hist[e] = 0;
  wait_prior_grid();
  __syncthreads();
#pragma unroll 4
  for (int p = lo + threadIdx.x; p < hi; p += kChunkThreads) {
    const int e = __ldg(a.ids + p);
    if (e >= 0 && e < a.E) atomicAdd(&hist[e], 1);     // counts do not depend on the order
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += kChunkThreads) a.inv[lo + e] = hist[e];
}

// Those counts to the numbers before each chunk: a CTA takes 32 experts (a lane
// each), its 32 warps a share of the chunks.
__global__ void __launch_bounds__(1024) sort_scan_kernel(const SortArgs a) {
  __shared__ int sums[32][33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e = blockIdx.x * 32 + lane;
  const int per = (a.chunks + 31) / 32, c0 = min(a.chunks, warp * per), c1 = min(a.chunks, c0 + per);
  wait_prior_grid();
  int sum = 0;
  if (e < a.E) {
#pragma unroll 4
    for (int c = c0; c < c1; ++c) sum += a.inv[chunk_begin(a, c) + e];
  }
  sums[lane][warp] = sum;
  __syncthreads();
  const int inc = warp_scan(sums[warp][lane], lane);   // expert `warp` of the CTA, over the warps' shares
  const int mine = sums[warp][lane];
  if (lane == 31 && (int)blockIdx.x * 32 + warp < a.E) a.counts[blockIdx.x * 32 + warp] = inc;
  __syncthreads();
  sums[warp][lane] = inc - mine;
  __syncthreads();
  if (e >= a.E) return;
  int run = sums[lane][warp];
  for (int c = c0; c < c1; ++c) {
    int *p = a.inv + chunk_begin(a, c) + e;
    const int n = *p;
    *p = run;
    run += n;
  }
}

__global__ void __launch_bounds__(kChunkThreads) sort_place_kernel(const SortArgs a) {
  extern __shared__ int sm[];
  const int E = a.E, W = kChunkThreads / 32, tid = threadIdx.x, NT = kChunkThreads;
  int *hist = sm, *total = sm + (size_t)W * E, *base = total + E, *wsum = base + E;
  const int lo = chunk_begin(a, blockIdx.x), hi = chunk_end(a, blockIdx.x);
  for (int i = tid; i < W * E; i += NT) hist[i] = 0;
  wait_prior_grid();
  // the numbers before this chunk leave inv before places go there
  const int per = (E + NT - 1) / NT, e0 = min(E, tid * per), e1 = min(E, e0 + per);
  int sum = 0;
  for (int e = e0; e < e1; ++e) {
    base[e] = a.inv[lo + e] + sum;
    sum += a.counts[e];
  }
  int everything;
  const int earlier = before_mine(sum, wsum, &everything);
  sum = 0;
  for (int e = e0; e < e1; ++e) {
    base[e] += earlier;
    if (blockIdx.x == 0) a.offsets[e] = earlier + sum;
    if (blockIdx.x == 0) sum += a.counts[e];
  }
  if (blockIdx.x == 0 && tid == 0) a.offsets[E] = everything;
  __syncthreads();
  const int steps = ((hi - lo + 31) / 32 + W - 1) / W;
  count_pairs(a, lo, hi, steps, hist, total);
  __syncthreads();
  put_pairs(a, lo, hi, steps, hist, base);
  for (long long p = everything + (long long)blockIdx.x * NT + tid; p < a.n; p += (long long)gridDim.x * NT)
    a.perm[p] = -1;
}

cudaError_t sort_by_cluster(const SortArgs &a, cudaStream_t s) {
  // a step costs some 150 instructions, so steps are spread over SMs first: one CTA
  // up to 512 pairs (2.8 us; eight CTAs 3.6), eight CTAs of up to 16 warps above
  // (4096 pairs of 128 experts: 4.3 us; one CTA of 32 warps 8.4, eight of 32 5.8)
  const int steps = std::max(1, (a.n + 31) / 32);
  const int C = steps <= 16 ? 1 : kSortMaxCluster;
  int W = 4;
  while (W < 16 && W * C < steps) W *= 2;
  static_assert((16 + 2) * kMaxExperts * 4 + 128 <= 227 * 1024, "histograms fit a CTA");
  static std::atomic<uint64_t> asked{0};
  cudaError_t e = ask_shared(sort_pairs_kernel, sort_smem(kMaxExperts, 16), asked);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)C);
  cfg.blockDim = dim3((unsigned)(32 * W));
  cfg.dynamicSmemBytes = sort_smem(a.E, W);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, sort_pairs_kernel, a);
}

cudaError_t sort_by_chunks(SortArgs a, cudaStream_t s) {
  // a chunk has room for E counts; two chunks an SM at most
  const int least = std::max(1024, (a.E + 31) / 32 * 32), most = 2 * sm_count();
  a.chunk = std::max(least, ((a.n + most - 1) / most + 31) / 32 * 32);
  a.chunks = std::max(1, a.n / a.chunk);
  const size_t smem = sort_smem(a.E, kChunkThreads / 32);
  static std::atomic<uint64_t> asked{0};
  cudaError_t e = ask_shared(sort_place_kernel, sort_smem(kMaxExperts, kChunkThreads / 32), asked);
  if (e == cudaSuccess) e = launch_op(sort_count_kernel, dim3(a.chunks), kChunkThreads, 0, s, a);
  if (e == cudaSuccess) e = launch_op(sort_scan_kernel, dim3((a.E + 31) / 32), 1024, 0, s, a);
  if (e == cudaSuccess) e = launch_op(sort_place_kernel, dim3(a.chunks), kChunkThreads, smem, s, a);
  return e;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_sort_tokens(const int32_t *ids, int32_t T, int32_t k, int32_t E, int32_t *counts,
                                        int32_t *offsets, int32_t *perm, int32_t *inv, void *stream) {
  static const char fn[] = "moe_sort_tokens";
  if (T < 0 || k < 1 || k > kMaxTopK || E < 1 || E > kMaxExperts || (int64_t)T * k > (int64_t)1 << 30)
    return ops_invalid(fn, "need T >= 0, 1 <= k <= 32, 1 <= E <= 1024 and T * k <= 2^30");
  if (!counts || !offsets) return ops_invalid(fn, "counts and offsets must be device pointers");
  if (T > 0 && (!ids || !perm || !inv)) return ops_invalid(fn, "ids, perm and inv must be device pointers");
  SortArgs a{ids, T * k, E, counts, offsets, perm, inv, 0, 0};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return ops_launched(fn, a.n >= kSortChunked ? sort_by_chunks(a, s) : sort_by_cluster(a, s));
}
