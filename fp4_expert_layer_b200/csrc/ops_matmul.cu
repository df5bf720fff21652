// ops_matmul.cu -- grouped product of FP4 operands on tcgen05 block-scaled MMA:
// the entry point, and the kernel for few rows (ops_matmul_pair.cu has many).
//
//   y[r, n] = xG[r] wG[g] sum_k x[r, k] w[g, n, k],  r in [offsets[g], offsets[g+1])
//
// Few rows are bound by the weights: each is read once, 0.53 or 0.56 bytes.  A work
// item is one token tile (up to NT rows of one group) and one block of 128 weight
// rows; weights are the A operand (M = 128), tokens the B operand (N = NT), so that
// a small batch costs no more tensor work than its tile.  Codes arrive by TMA (256 K
// elements, 128 bytes a row, a stage; 128-byte swizzle; a box may start at any row,
// so ragged segments need no padding: what a box brings of the next segment's rows
// ends in columns that are not stored).  Block scales stay in the rows' own order in
// memory; a warp reads a sector of each of 128 rows' scales at a time and turns them
// over into the 512-byte blocks (32 rows x 4 row groups x 4 scales) that tcgen05.cp
// moves to TMEM.
//
// Persistent, one CTA per SM; the item list is the scan of the groups' tile counts,
// which every CTA makes for itself, so there is no workspace and no counter.  With
// few items (SPLIT) a cluster of CTAs shares an item's K range and adds the parts in
// rank order through distributed shared memory.
//
// Measured, from a graph: 256 rows over 64 groups, N = K = 2048, NVFP4: 29.0 us, 5.2 TB/s (some 3
// us of it are the way to the first stage); 1 row, N = K = 4096, MXFP4: 5.6 us, of
// which the weights need 1.4 and the way through launch, first stage and the
// cluster's meeting the rest.
//
// Warp roles: 0 copies codes, 1 allocates TMEM and issues the MMAs, 2..5 read the
// accumulators back and store, 6..9 bring the scales.  All mbarrier waits are bounded.
#include <cooperative_groups.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "ops_matmul.cuh"

namespace cg = cooperative_groups;

namespace moe {
namespace {

constexpr int kMmThreads = 320;

template <int WF, int NT, bool SPLIT>
struct MmGeom {
  static constexpr int NBLK = (WF == WF_MX) ? 2 : 4;       // 4-scale blocks of 256 K
  static constexpr int SF_BYTES = NBLK * 512;
  static constexpr int A_BYTES = 128 * 128;
  static constexpr int B_BYTES = NT * 128;
  static constexpr int SF_OFF = A_BYTES + B_BYTES;
  static constexpr int STAGE = (SF_OFF + 2 * SF_BYTES + 1023) / 1024 * 1024;
  static constexpr int RECV = SPLIT ? 128 * NT * 4 : 0;    // the cluster's parts, beside the stages
  static constexpr int FIT = (205 * 1024 - RECV) / STAGE;
  static constexpr int NBUF = 2;
  static constexpr int SF_COLS = 2 * NBLK * 4;             // TMEM columns a stage's scales take
  static constexpr int SF_TMEM = NBUF * NT;
  static constexpr int SF_FIT = (512 - SF_TMEM) / SF_COLS;
  static constexpr int STAGES = FIT < 8 ? (FIT < SF_FIT ? FIT : SF_FIT) : (8 < SF_FIT ? 8 : SF_FIT);
  static constexpr size_t SMEM = (size_t)STAGES * STAGE + RECV + 1024;
  static_assert(STAGES >= 3, "a pipeline");
  static_assert(SF_TMEM + STAGES * SF_COLS <= 512, "TMEM budget");
  static_assert(SMEM + 17 * 1024 <= 227 * 1024, "shared-memory budget");
};

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }

template <int WF, int NT, bool SPLIT>
__global__ void __launch_bounds__(kMmThreads, 1) fp4_matmul_kernel(const __grid_constant__ MatmulArgs a) {
  using Geo = MmGeom<WF, NT, SPLIT>;
  constexpr int S = Geo::STAGES, NBUF = Geo::NBUF, WORDS = kSfWords<WF>;
  extern __shared__ __align__(1024) uint8_t mm_raw[];
  __shared__ __align__(8) uint64_t full_bar[S];
  __shared__ __align__(8) uint64_t empty_bar[S];
  __shared__ __align__(8) uint64_t accf_bar[NBUF];
  __shared__ __align__(8) uint64_t acce_bar[NBUF];
  __shared__ __align__(8) uint64_t quiesce_bar;
  __shared__ uint32_t tmem_base_s;
  __shared__ int gave_up;                                  // a wait of this CTA has
  __shared__ float xG_s[SPLIT ? NT : 1];
  __shared__ MmGroups groups;

  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(mm_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid < S) {
    mbar_init(smem_u32(&full_bar[tid]), 3);                // the codes' copies and two scale warps
    mbar_init(smem_u32(&empty_bar[tid]), 1);
    mbar_fence_init();
  }
  if (tid == 32 * 2) {
    gave_up = 0;
    tmap_prefetch(&a.wmap);
    tmap_prefetch(&a.xmap);
    for (int b = 0; b < NBUF; ++b) {
      mbar_init(smem_u32(&accf_bar[b]), 1);
      mbar_init(smem_u32(&acce_bar[b]), 4);
    }
    mbar_init(smem_u32(&quiesce_bar), 1);
    mbar_fence_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_base_s), 512);
    tmem_relinquish();
  }
  const int nrb = (a.N + 127) / 128, nk_all = (a.K + 255) / 256;

  // SPLIT: cluster c takes item c and rank r of it the K range [k0, k1)
  const int rlog = SPLIT ? a.rank_log : 0, ranks = 1 << rlog, rank = SPLIT ? (int)cg::this_cluster().block_rank() : 0;
  // ranges of whole steps of the scales, so that a step starts on a sector
  constexpr int AHEAD = kSfAhead<WF>;
  const int steps = (nk_all + AHEAD - 1) / AHEAD;
  const int k0 = min(nk_all, (steps * rank >> rlog) * AHEAD), k1 = min(nk_all, (steps * (rank + 1) >> rlog) * AHEAD);
  const unsigned first = blockIdx.x >> rlog, step = SPLIT ? 0u : gridDim.x;
  wait_prior_grid();
  // Few rows: the next kernel is small too and may be placed now (products one after
  // another 6.0 -> 5.75 us).  Not after the streamed kernel: a wide kernel placed
  // early crowds the SMs that are free first (32 x 8 tokens, two products and what
  // lies between them: 73 -> 75 us).
  if (SPLIT) trigger_dependents();
  mm_scan_groups(a, groups);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_s;
  if constexpr (SPLIT) cluster_arrive();                   // this CTA's shared memory may be written from now on
  using Walk = MmWalk;

  if (warp == 0) {
    // ---------------- codes
    int s = 0, issued = 0;
    uint32_t ph = 0;
    bool failed = false;
    for (Walk m(a, groups, nrb, first, step); m.more() && !failed; m.next(a, groups)) {
      for (int it = k0; it < k1; ++it) {
        if (issued >= S && !mm_wait_warp(smem_u32(&empty_bar[s]), ph ^ 1u, &gave_up, a.err, 61)) { failed = true; break; }
        const uint32_t bar = smem_u32(&full_bar[s]);
        const uint32_t st = smem_u32(smem + (size_t)s * Geo::STAGE);
        if (elect_one()) {
          mbar_arrive_expect_tx(bar, (uint32_t)(Geo::A_BYTES + Geo::B_BYTES));
          tma_load_3d(st, &a.wmap, bar, it * 128, m.rb * 128, m.g);
          tma_load_2d(st + Geo::A_BYTES, &a.xmap, bar, it * 128, m.row0);
        }
        __syncwarp();
        ++issued;
        if (++s == S) { s = 0; ph ^= 1u; }
      }
    }
    // every copy has landed before the CTA leaves (a stage whose scales never
    // came keeps its phase: the wait then ends by its limit)
    if (lane == 0) {
      int s2 = 0;
      uint32_t ph2 = 0;
      for (int i = 0; i < issued; ++i) {
        if (i >= issued - S) mbar_drain(smem_u32(&full_bar[s2]), ph2);
        if (++s2 == S) { s2 = 0; ph2 ^= 1u; }
      }
    }
  } else if (warp == 1) {
    // ---------------- MMA issue: the whole warp runs the loop, one lane issues
    int s = 0, n = 0;
    uint32_t ph = 0;
    bool failed = false;
    for (Walk m(a, groups, nrb, first, step); m.more() && !failed; m.next(a, groups)) {
      const int buf = n % NBUF;
      if (n >= NBUF && !mm_wait_warp(smem_u32(&acce_bar[buf]), ((n / NBUF) - 1) & 1, &gave_up, a.err, 62)) break;
      tc_fence_after();
      const uint32_t acc = tmem + (uint32_t)(buf * NT);
      for (int it = k0; it < k1; ++it) {
        if (!mm_wait_warp(smem_u32(&full_bar[s]), ph, &gave_up, a.err, 63)) { failed = true; break; }
        tc_fence_after();
        const uint32_t st = smem_u32(smem + (size_t)s * Geo::STAGE);
        const uint32_t sf_t = tmem + (uint32_t)(Geo::SF_TMEM + s * Geo::SF_COLS);
        if (elect_one()) {
#pragma unroll
          for (int b = 0; b < 2 * Geo::NBLK; ++b) tc_cp_sf_block(sf_t + 4 * b, st + Geo::SF_OFF + 512 * b);
#pragma unroll
          for (int k = 0; k < 4; ++k) {                    // K = 64 an MMA
            const int blk = (WF == WF_MX) ? (k >> 1) : k;
            const uint32_t byte = (WF == WF_MX) ? (uint32_t)(2 * (k & 1)) : 0u;
            const uint64_t adesc = umma_desc(st + k * 32, 16, 1024, 2);
            const uint64_t bdesc = umma_desc(st + Geo::A_BYTES + k * 32, 16, 1024, 2);
            const uint32_t sfa = (sf_t + (uint32_t)(blk * 4)) | (byte << 30);
            const uint32_t sfb = (sf_t + (uint32_t)((Geo::NBLK + blk) * 4)) | (byte << 30);
            const uint32_t idesc = idesc_fp4_block(128, NT, WF == WF_MX, byte, byte);
            const uint32_t accum = (it > k0 || k > 0) ? 1u : 0u;
            if constexpr (WF == WF_MX) umma_mxf4(acc, adesc, bdesc, idesc, sfa, sfb, accum);
            else umma_nvf4(acc, adesc, bdesc, idesc, sfa, sfb, accum);
          }
          tc_commit(smem_u32(&empty_bar[s]));
        }
        __syncwarp();
        if (++s == S) { s = 0; ph ^= 1u; }
      }
      if (failed) break;
      if (elect_one()) tc_commit(smem_u32(&accf_bar[buf]));
      __syncwarp();
      ++n;
    }
    // every MMA has completed before TMEM is freed (and, when split, before the
    // cluster meets), also when a wait gave up
    __syncwarp();
    if (elect_one()) tc_commit(smem_u32(&quiesce_bar));
    __syncwarp();
    mbar_drain(smem_u32(&quiesce_bar), 0);
  } else if (warp < 6) {
    // ---------------- accumulators to y: warp w has TMEM lanes 32 * (w % 4) ..
    if constexpr (!SPLIT) {
      const int quad = warp & 3;
      int n = 0;
      for (Walk m(a, groups, nrb, first, step); m.more(); m.next(a, groups)) {
        const int buf = n % NBUF;
        float f = 1.0f;                                    // lane r: the factor of the item's row r
        bool far = false;
        const float wG = (WF == WF_NV) ? __ldg(a.wG + m.g) : 1.0f;
        if constexpr (WF == WF_NV) {
          static_assert(NT <= 32, "a row a lane");
          if (lane < m.nrows) f = wG * __ldg(a.xG + m.row0 + lane);
          far = !__all_sync(0xffffffffu, whole_factor(f));
        }
        if (!mm_wait_warp(smem_u32(&accf_bar[buf]), (n / NBUF) & 1, &gave_up, a.err, 64, k1 - k0)) break;
        tc_fence_after();
        const uint32_t acc = tmem + (uint32_t)(buf * NT) + ((uint32_t)(32 * quad) << 16);
        const int col = m.rb * 128 + 32 * quad + lane;
        if (far) store_far(a, acc, m.row0, m.nrows, col, wG);
#pragma unroll 1
        for (int c0 = far ? m.nrows : 0; c0 < m.nrows; c0 += 16) {
          uint32_t d[16];
          tmem_ld16(acc + (uint32_t)c0, d);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float sc = (WF == WF_NV) ? __shfl_sync(0xffffffffu, f, c0 + j) : 1.0f;
            if (c0 + j < m.nrows && col < a.N)
              store_out(a.y, a.dtype, (int64_t)(m.row0 + c0 + j) * a.ldy + col, __uint_as_float(d[j]) * sc);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&acce_bar[buf]));
        ++n;
      }
    }
  } else {
    // ---------------- scales: warps 6 and 8 the weights', 7 and 9 the tokens', on
    // alternate steps
    const bool tokens = (warp & 1) != 0;
    constexpr int RG = (NT + 31) / 32 < 4 ? (NT + 31) / 32 : 4;        // 32-row groups of a token tile
    const uint8_t *rowp[4];
    const uint8_t *lo = tokens ? a.xs : a.ws, *hi = lo + (tokens ? (size_t)a.rows : (size_t)a.groups * a.N) * a.nsf;
    const uint32_t off = Geo::SF_OFF + (tokens ? Geo::SF_BYTES : 0) + 16 * lane;
    feed_scales<WF, S, true>(
        a, groups, Walk(a, groups, nrb, first, step), k0, k1, (warp - 6) >> 1, 2,
        [&](const Walk &m) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            rowp[j] = tokens ? a.xs + (size_t)min(m.row0 + 32 * j + lane, a.rows - 1) * a.nsf
                             : a.ws + ((size_t)m.g * a.N + min(m.rb * 128 + 32 * j + lane, a.N - 1)) * a.nsf;
        },
        [&](int it0, uint32_t(&w)[4][8]) {
          if (a.sf_wide) fetch_sf<WF, true>(a, rowp, tokens ? RG : 4, it0, k1, lo, hi, w);
          else fetch_sf<WF, false>(a, rowp, tokens ? RG : 4, it0, k1, lo, hi, w);
        },
        [&](int s, uint32_t parity) { return mm_wait_warp(smem_u32(&empty_bar[s]), parity, &gave_up, a.err, 65); },
        [&](const Walk &) {
          return [&](int s, const uint32_t(&w)[4][8], int i) {
            const uint32_t dst = smem_u32(smem + (size_t)s * Geo::STAGE) + off;
#pragma unroll
            for (int b = 0; b < WORDS; ++b)                // rows past the tile's: any number, their columns go nowhere
              sts128(dst + 512 * b, make_uint4(w[0][i * WORDS + b], w[1][i * WORDS + b], w[2][i * WORDS + b],
                                               w[3][i * WORDS + b]));
          };
        },
        [&](int s) {
          if (lane == 0) mbar_arrive(smem_u32(&full_bar[s]));
        });
  }

  if constexpr (SPLIT) {
    // parts meet: rank q finishes weight rows [128 q / ranks, 128 (q + 1) / ranks)
    cg::cluster_group cluster = cg::this_cluster();
    float *recv = reinterpret_cast<float *>(smem + (size_t)S * Geo::STAGE);   // [source][rows of a rank][NT]
    const Walk m(a, groups, nrb, first, step);
    const bool any = m.more();                             // the same for the whole cluster
    bool ok = k1 > k0;                                     // a rank without stages adds nothing
    const float wG = (WF == WF_NV && any) ? __ldg(a.wG + m.g) : 1.0f;       // on their way while the products end
    if (WF == WF_NV && any && tid < m.nrows) xG_s[tid] = __ldg(a.xG + m.row0 + tid);
    if (any && warp >= 2 && warp < 6) ok = mm_wait_warp(smem_u32(&accf_bar[0]), 0, &gave_up, a.err, 66, k1 - k0) && ok;
    __syncwarp();
    cluster_wait();                                        // every rank has begun (long ago)
    const int plog = 7 - rlog, per = 1 << plog;
    if (any && warp >= 2 && warp < 6) {
      tc_fence_after();
      const int quad = warp & 3, row = 32 * quad + lane;
      float *dst = cluster.map_shared_rank(recv, row >> plog) + ((size_t)rank * per + (row & (per - 1))) * NT;
#pragma unroll 1
      for (int c0 = 0; c0 < NT; c0 += 16) {
        uint32_t v[16];
        tmem_ld16(tmem + (uint32_t)c0 + ((uint32_t)(32 * quad) << 16), v);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; j += 4)
          *reinterpret_cast<float4 *>(dst + c0 + j) =
              ok ? make_float4(__uint_as_float(v[j]), __uint_as_float(v[j + 1]), __uint_as_float(v[j + 2]),
                               __uint_as_float(v[j + 3]))
                 : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
    cluster.sync();                                        // every part is where it is added
    if (any) {
      for (int i = tid; i < per * m.nrows; i += kMmThreads) {
        const int c = i >> plog, r = i & (per - 1);            // neighbouring threads: neighbouring columns of y
        float v = 0.0f;
        for (int q = 0; q < ranks; ++q) v += recv[((size_t)q * per + r) * NT + c];
        const int col = m.rb * 128 + rank * per + r;
        if (WF == WF_NV) {
          const float f = wG * xG_s[c];
          v = whole_factor(f) ? v * f : scaled(v, xG_s[c], wG);
        }
        if (col < a.N) store_out(a.y, a.dtype, (int64_t)(m.row0 + c) * a.ldy + col, v);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ host side
PFN_cuTensorMapEncodeTiled_v12000 map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}

// Error word of each device's products, in mapped host memory: a wait that gives up
// writes its code there, and the next call takes it.  Made by a device's first product,
// also inside a stream capture, in which the allocation takes no part.
struct MatmulErrors {
  std::mutex mu;
  int *word[64] = {};
};
MatmulErrors &matmul_errors() {
  static MatmulErrors all;
  return all;
}

moe_status_t matmul_error_word(const char *fn, int **out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev < 0 || dev >= 64) return ops_fail(MOE_ERR_CUDA, fn, "no current device");
  MatmulErrors &all = matmul_errors();
  std::lock_guard<std::mutex> lock(all.mu);
  if (!all.word[dev]) {
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    cudaThreadExchangeStreamCaptureMode(&mode);
    void *h = nullptr;
    e = cudaHostAlloc(&h, sizeof(int), cudaHostAllocMapped | cudaHostAllocPortable);
    cudaThreadExchangeStreamCaptureMode(&mode);
    if (e != cudaSuccess) {
      cudaGetLastError();
      return ops_fail(MOE_ERR_CUDA, fn, std::string("no error word: ") + cudaGetErrorString(e));
    }
    *static_cast<int *>(h) = 0;
    all.word[dev] = static_cast<int *>(h);
  }
  *out = all.word[dev];
  return MOE_OK;
}

// Takes the failure that the current device's word holds, if any: read and cleared in
// one step, so that one recorded meanwhile stays for the next call.
moe_status_t matmul_take_error(const char *fn) {
  int dev = 0, *word = nullptr;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return MOE_OK;
  }
  {
    MatmulErrors &all = matmul_errors();
    std::lock_guard<std::mutex> lock(all.mu);
    word = all.word[dev];
  }
  if (!word || !*(volatile int *)word) return MOE_OK;
  const int code = __atomic_exchange_n(word, 0, __ATOMIC_SEQ_CST);
  if (!code) return MOE_OK;                                // another thread's call took it
  return ops_fail(MOE_ERR_CUDA, fn, "a device-side wait of an earlier call gave up (code " + std::to_string(code) + ")");
}

// A wait that nothing ends, as the kernels wait, for a millisecond and what `stages` add.
__global__ void __launch_bounds__(32) give_up_kernel(int *err, int stages) {
  __shared__ __align__(8) uint64_t bar;
  __shared__ int gave_up;
  if (threadIdx.x == 0) {
    gave_up = 0;
    mbar_init(smem_u32(&bar), 1);
    mbar_fence_init();
  }
  __syncwarp();
  mm_wait_warp(smem_u32(&bar), 0, &gave_up, err, 60, stages, 1000000ull);
}

template <int WF, int NT, bool SPLIT>
cudaLaunchConfig_t matmul_config(int items, int rank_log, cudaLaunchAttribute (&attr)[2], cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)items << rank_log);
  cfg.blockDim = dim3(kMmThreads);
  cfg.dynamicSmemBytes = MmGeom<WF, NT, SPLIT>::SMEM;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1u << rank_log;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = SPLIT ? attr : attr + 1;
  cfg.numAttrs = SPLIT ? 2 : 1;
  return cfg;
}

// Clusters of 2^rank_log CTAs of the split kernel that run at once: fewer than the
// SMs have room for, since a cluster stays within a GPC.  Asked once a device.
template <int WF>
int resident_clusters(int rank_log) {
  using Geo = MmGeom<WF, 16, true>;
  auto fn = fp4_matmul_kernel<WF, 16, true>;
  static std::atomic<int> known[64][4];
  static std::atomic<uint64_t> asked{0};
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  if ((n = known[dev][rank_log].load(std::memory_order_relaxed))) return n - 1;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = matmul_config<WF, 16, true>(1, rank_log, attr, nullptr);
  cfg.numAttrs = 1;                                        // the cluster alone
  if (ask_shared(fn, Geo::SMEM, asked) != cudaSuccess || cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  known[dev][rank_log].store(n + 1, std::memory_order_relaxed);
  return n;
}

template <int WF, int NT, bool SPLIT>
cudaError_t launch_matmul(const MatmulArgs &a, int items, cudaStream_t s) {
  using Geo = MmGeom<WF, NT, SPLIT>;
  auto fn = fp4_matmul_kernel<WF, NT, SPLIT>;
  static std::atomic<uint64_t> asked{0};
  const cudaError_t e = ask_shared(fn, Geo::SMEM, asked);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = matmul_config<WF, NT, SPLIT>(items, a.rank_log, attr, s);
  return cudaLaunchKernelEx(&cfg, fn, a);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_fp4_matmul(const uint8_t *x_codes, const uint8_t *x_scales, const float *x_global,
                                       int32_t rows, const uint8_t *w_codes, const uint8_t *w_scales,
                                       const float *w_global, int32_t n_groups, int32_t N, int32_t K, int32_t fmt,
                                       const int32_t *offsets, void *y, int32_t dtype, int64_t ldy, void *stream) {
  static const char fn[] = "moe_fp4_matmul";
  if (fmt != MOE_FMT_MXFP4 && fmt != MOE_FMT_NVFP4) return ops_invalid(fn, "fmt must be MOE_FMT_MXFP4 or MOE_FMT_NVFP4");
  if (!is_float_dtype(dtype)) return ops_invalid(fn, "dtype must be F32, BF16 or F16");
  if (rows < 0 || rows > kMmMaxRows || N < 1 || N > kMmMaxSide || K < 32 || K % 32 || K > kMmMaxSide)
    return ops_invalid(fn, "need 0 <= rows <= 2^27, 1 <= N <= 2^30 and K a multiple of 32, at most 2^30");
  if (n_groups < 1 || n_groups > kMmMaxGroups || (int64_t)n_groups * N >= (int64_t)1 << 31)
    return ops_invalid(fn, "need 1 <= n_groups <= 1024 and n_groups * N below 2^31");
  if (!offsets && n_groups != 1) return ops_invalid(fn, "more than one group needs offsets");
  if (ldy < N) return ops_invalid(fn, "ldy must be at least N");
  if (const moe_status_t st = matmul_take_error(fn); st != MOE_OK) return st;
  if (rows == 0) return MOE_OK;
  if (!x_codes || !x_scales || !w_codes || !w_scales || !y) return ops_invalid(fn, "operands and y must be device pointers");
  if (fmt == MOE_FMT_NVFP4 && (!x_global || !w_global)) return ops_invalid(fn, "NVFP4 needs both global scales");
  if (!aligned_to(x_codes, 16) || !aligned_to(w_codes, 16)) return ops_invalid(fn, "codes must be 16-byte aligned");
  if (!aligned_to(y, dtype_bytes(dtype)) || !aligned_to(offsets, 4) || !aligned_to(x_global, 4) ||
      !aligned_to(w_global, 4))
    return ops_invalid(fn, "y, offsets and global scales must be aligned to their type");

  MatmulArgs a{};
  auto enc = map_encoder();
  if (!enc) return ops_fail(MOE_ERR_CUDA, fn, "cuTensorMapEncodeTiled is unavailable");
  // Which kernel, by the rows a group has on average and the blocks of 128 weight
  // rows that can be in use (graph-timed us, NVFP4, N = K = 2048 unless said):
  //  * up to 32 rows and blocks for every SM: weights are streamed, one CTA a block
  //    with token tiles of 32 (64 groups: 29.9 at 8 rows a group and 31.2 at 20;
  //    pairs 35.3 and 36.0; 38.0 and 37.7 at 40);
  //  * items of 16 rows x 128 weight rows so few that clusters of 2, 4 or 8 SMs can
  //    share each one's K, and the largest cluster with which all run at once (dense,
  //    16 rows: 4 ways 5.7, 2 ways 6.7, unsplit 8.3, pairs 7.3; 8 ways, of which one
  //    cluster waits for the others: 10.1; 64 rows, N 512, K 4096: 6.4, pairs 10.1).
  //    Not for little K where it is cut in two or four and the tiles are full (K 512,
  //    16 rows, N 8192: 5.8, pairs 5.4), nor unsplit but for single rows (K 512,
  //    N 8192: 4.7, pairs 5.1; with 8 rows 5.5 and 5.2);
  //  * else pairs (dense, 64 rows, N 4096: 7.9, one CTA a block 10.2; 128 rows a
  //    group, 64 groups: 46; 92).
  const int sms = sm_count();
  const int64_t mean = (rows + n_groups - 1) / n_groups, blocks = std::min<int64_t>(n_groups, rows) * ((N + 127) / 128);
  // tiles there can be at most (without offsets: there are)
  auto tiles = [&](int64_t nt) {
    return offsets ? std::min<int64_t>(rows, rows / nt + n_groups) : (rows + nt - 1) / nt;
  };
  const bool mx = fmt == MOE_FMT_MXFP4;
  const int nk = (K + 255) / 256;
  const bool streamed = mean <= 32 && blocks >= sms;
  bool split = false;
  if (const int64_t items = tiles(16) * ((N + 127) / 128); !streamed && items <= sms) {
    // one row of one or two stages: the meeting costs what the cut saves (4.2; 4.4)
    const int most = nk > 2 || mean > 1 ? 3 : 0;
    while (a.rank_log < most && items << (a.rank_log + 1) <= sms &&
           items <= (mx ? resident_clusters<WF_MX>(a.rank_log + 1) : resident_clusters<WF_NV>(a.rank_log + 1)))
      ++a.rank_log;
    split = a.rank_log ? mean <= 8 || nk << a.rank_log >= 8 : mean == 1;
    if (!split) a.rank_log = 0;
  }
  // pairs: the smallest tile whose items still run at once, for its shorter
  // epilogue; else the largest, which moves the least
  const int64_t wide_blocks = (N + 255) / 256;
  int nt = streamed ? 32 : split ? 16 : 64;
  if (!streamed && !split)
    while (nt < kPairRows && tiles(nt) * wide_blocks > sms / 2) nt *= 2;
  if (nt >= 64 && tiles(nt) * wide_blocks > sms / 2) nt = kPairRows;
  const cuuint64_t kb = (cuuint64_t)(K / 2);
  const cuuint32_t ones[3] = {1, 1, 1};
  {
    const cuuint64_t dims[2] = {kb, (cuuint64_t)rows}, strides[1] = {kb};
    const cuuint32_t box[2] = {128, (cuuint32_t)(nt >= 64 ? kPairBox : nt)};
    if (enc(&a.xmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(x_codes), dims, strides, box, ones,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return ops_fail(MOE_ERR_CUDA, fn, "cuTensorMapEncodeTiled failed for x");
  }
  {
    const cuuint64_t dims[3] = {kb, (cuuint64_t)N, (cuuint64_t)n_groups}, strides[2] = {kb, kb * (cuuint64_t)N};
    const cuuint32_t box[3] = {128, 128, 1};
    if (enc(&a.wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t *>(w_codes), dims, strides, box, ones,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return ops_fail(MOE_ERR_CUDA, fn, "cuTensorMapEncodeTiled failed for w");
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (const moe_status_t st = matmul_error_word(fn, &a.err); st != MOE_OK) return st;
  a.xs = x_scales; a.ws = w_scales;
  a.xG = x_global; a.wG = w_global;
  a.offsets = offsets;
  a.y = y; a.ldy = ldy;
  a.rows = rows; a.groups = n_groups; a.N = N; a.K = K;
  while ((1 << a.tile_log) < nt) ++a.tile_log;
  a.nsf = K / (fmt == MOE_FMT_MXFP4 ? 32 : 16);
  a.dtype = dtype;
  a.sf_wide = a.nsf % 16 == 0 && aligned_to(x_scales, 16) && aligned_to(w_scales, 16);
  a.y_vec = row_alignment(y, ldy * dtype_bytes(dtype)) >= 16;
  cudaError_t e;
  if (streamed) {
    const int grid = (int)std::min<int64_t>(tiles(32) * ((N + 127) / 128), sms);
    e = mx ? launch_matmul<WF_MX, 32, false>(a, grid, s) : launch_matmul<WF_NV, 32, false>(a, grid, s);
  } else if (split) {
    const int items = (int)(tiles(16) * ((N + 127) / 128));  // one a cluster
    e = mx ? launch_matmul<WF_MX, 16, true>(a, items, s) : launch_matmul<WF_NV, 16, true>(a, items, s);
  } else {
    const int pairs = (int)std::min<int64_t>(tiles(nt) * wide_blocks, sms / 2);
    e = launch_matmul_pair(mx ? WF_MX : WF_NV, a, pairs, s);
  }
  return ops_launched(fn, e);
}

extern "C" moe_status_t moe_debug_give_up(int32_t stages, void *stream) {
  static const char fn[] = "moe_debug_give_up";
  if (stages < 0 || stages > 250000) return ops_invalid(fn, "stages must be 0 to 250000 (a second)");
  int *err = nullptr;
  if (const moe_status_t st = matmul_error_word(fn, &err); st != MOE_OK) return st;
  give_up_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(err, stages);
  return ops_launched(fn, cudaSuccess);
}
