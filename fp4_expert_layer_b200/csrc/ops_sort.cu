// ops_sort.cu -- pairs (token, choice) sorted by expert: a stable counting sort.
//
//   counts[e] = #{p : ids[p] = e},  offsets = exclusive scan of counts,
//   inv[p] = offsets[ids[p]] + #{q < p : ids[q] = ids[p]},  perm[inv[p]] = p.
//
// One launch of one thread-block cluster, whatever the size.  Every warp of the
// cluster owns a contiguous range of pairs.  It counts its range into a
// histogram of its own (a row of shared memory; the lanes of one step that hold
// the same expert find one another with match_any), the histograms are scanned
// over the warps of a CTA, then over the cluster's CTAs through distributed
// shared memory, then over the experts, and the warp places its range in order.
// No workspace, no atomics, no other launch: the order is that of the pairs.
//
// Bound by latency: 12 bytes a pair is nothing next to the launch.  A cluster of
// up to 8 CTAs (256 warps) keeps a warp's range short: 82K pairs are 10 steps.
#include <cooperative_groups.h>

#include "ops_common.cuh"

namespace cg = cooperative_groups;

namespace moe {
namespace {

constexpr int kSortMaxCluster = 8;      // the portable cluster size

struct SortArgs {
  const int *ids;
  int n, E;
  int *counts, *offsets, *perm, *inv;
};

// shared memory: hist[W][E], total[E] (this CTA's counts), base[E], wsum[32]
inline size_t sort_smem(int E, int W) { return ((size_t)(W + 2) * E + 32) * sizeof(int); }

__global__ void __launch_bounds__(1024, 1) sort_pairs_kernel(const SortArgs a) {
  extern __shared__ int sm[];
  const int E = a.E, W = blockDim.x >> 5, tid = threadIdx.x, NT = blockDim.x;
  const int warp = tid >> 5, lane = tid & 31;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  int *hist = sm, *total = sm + (size_t)W * E, *base = total + E, *wsum = base + E;

  for (int i = tid; i < W * E; i += NT) hist[i] = 0;
  wait_prior_grid();
  __syncthreads();

  // this warp's pairs: a multiple of 32 of them, so that ranges start aligned
  const int warps = C * W;
  const int steps = ((a.n + 31) / 32 + warps - 1) / warps;
  const long long lo = (long long)(rank * W + warp) * steps * 32;
  const int p0 = (int)min((long long)a.n, lo), p1 = (int)min((long long)a.n, lo + (long long)steps * 32);
  int *mine = hist + warp * E;
  const unsigned below = (1u << lane) - 1u;

  for (int p = p0 + lane; p - lane < p1; p += 32) {
    const int e = p < p1 ? __ldg(a.ids + p) : -1;
    const bool kept = e >= 0 && e < E;
    const unsigned same = __match_any_sync(0xffffffffu, e);
    if (kept && (same & below) == 0) mine[e] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  for (int e = tid; e < E; e += NT) {                  // over the CTA's warps
    int run = 0;
    for (int w = 0; w < W; ++w) {
      const int c = hist[w * E + e];
      hist[w * E + e] = run;
      run += c;
    }
    total[e] = run;
  }
  if (C > 1) cluster.sync(); else __syncthreads();

  // over the cluster, then over the experts: thread t takes `per` experts
  const int per = (E + NT - 1) / NT, e0 = min(E, tid * per), e1 = min(E, e0 + per);
  int sum = 0;
  for (int e = e0; e < e1; ++e) {
    int before = 0, all = 0;
    for (int q = 0; q < C; ++q) {
      const int c = C > 1 ? *cluster.map_shared_rank(total + e, q) : total[e];
      if (q < rank) before += c;
      all += c;
    }
    base[e] = before + sum;                            // + the sum of earlier threads' experts, below
    if (rank == 0) a.counts[e] = all;
    sum += all;
  }
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) wsum[warp] = inc;
  __syncthreads();
  int earlier = inc - sum, everything = 0;
  for (int w = 0; w < W; ++w) {
    if (w < warp) earlier += wsum[w];
    everything += wsum[w];
  }
  for (int e = e0; e < e1; ++e) {
    base[e] += earlier;
    if (rank == 0) a.offsets[e] = base[e];             // rank 0 has nothing before it
  }
  if (rank == 0 && tid == 0) a.offsets[E] = everything;
  __syncthreads();

  for (int p = p0 + lane; p - lane < p1; p += 32) {
    const int e = p < p1 ? __ldg(a.ids + p) : -1;
    const bool kept = e >= 0 && e < E;
    const unsigned same = __match_any_sync(0xffffffffu, e);
    const int ahead = __popc(same & below);
    const int at = kept ? base[e] + mine[e] + ahead : -1;
    __syncwarp();
    if (kept && ahead == 0) mine[e] += __popc(same);
    __syncwarp();
    if (p < p1) a.inv[p] = at;
    if (kept) a.perm[at] = p;
  }
  for (long long p = everything + (long long)rank * NT + tid; p < a.n; p += (long long)C * NT) a.perm[p] = -1;
  if (C > 1) cluster.sync();                           // no CTA leaves while another reads its counts
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
  SortArgs a{ids, T * k, E, counts, offsets, perm, inv};
  // as few warps as give each one step, up to 32 to a CTA (16 where the
  // histograms of 32 would not fit beside the rest), then more CTAs
  const int steps = std::max(1, (a.n + 31) / 32);
  const int most = 32;
  int W = 4, C = 1;
  while (W < most && W < steps) W *= 2;
  while (C < kSortMaxCluster && C * W * 4 < steps) C *= 2;
  const size_t smem = sort_smem(E, W);
  static_assert((32 + 2) * kMaxExperts * 4 + 128 <= 227 * 1024, "histograms fit a CTA");
  cudaError_t e = cudaFuncSetAttribute(sort_pairs_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)sort_smem(kMaxExperts, 32));
  if (e == cudaSuccess) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)C);
    cfg.blockDim = dim3((unsigned)(32 * W));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)C;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, sort_pairs_kernel, a);
  }
  return ops_launched(fn, e);
}
