// ops_matmul_pair.cu -- the grouped FP4 product for many rows: CTA pairs.
//
//   y[r, n] = xG[r] wG[g] sum_k x[r, k] w[g, n, k]
//
// Two CTAs of a cluster share one MMA of 256 weight rows x up to 256 token rows
// (cta_group::2): each holds 128 weight rows and half the tokens' rows, so that a
// stage of 256 K elements brings 32 KB of codes to an SM for 128 x 256 x 256
// multiply-adds.  One CTA's 128 x 128 tile brings the same for half of them, and is
// then bound by this fill, L2 to shared memory (some 50 bytes a clock an SM), at half
// of what the tensor pipe does.
//
// Measured, 20 launches from a graph: 8192 x 4096 x 4096, MXFP4, fp32 result 61.2 to 63 us
// (4.4 PFLOP/s; the MMAs alone, with no operand copied, 51.7); 16384 rows over 128 groups,
// N 1536, K 2048, NVFP4, bf16 66.2 us (4.5 TB/s, of 45 us for its bytes).  Called in a row
// for a second the power cap takes the clock to 1.7 GHz and the times to 74 and 75.  One
// CTA a 128 x 128 tile took 120 and 151.
//
// The MMA is as wide as the item has rows (rounded up to 32), and boxes of 64 rows
// that it does not need are not copied, so a ragged segment costs what it holds.
//
// TMEM: items put their accumulators in turn at the lower and the upper end of the
// columns that two stages' scales leave (416 or 464), where wide ones overlap in
// the middle.  An epilogue reads the middle first and hands it on, then stores
// while the next item multiplies.  tcgen05.cp and MMAs of one thread run in order,
// so scales need no more than two places.
//
// Warps of each CTA: 0 copies codes; 1 allocates TMEM and, in the even CTA, issues
// for both; 2..9 read accumulators back (two a lane quadrant, on alternate 32-token
// chunks); 10 brings the scales of the weights, 11 and 12 those of the tokens' two
// halves: 32 bytes of a row at a time (a whole sector: two stages' NVFP4 scales,
// four stages' MXFP4 ones), one such step ahead, turned over into the blocks that
// tcgen05.cp copies.
#include "ops_matmul.cuh"

namespace cg = cooperative_groups;

namespace moe {
namespace {

constexpr int kPairThreads = 13 * 32;
constexpr int kPairEpi = 8;                                // epilogue warps of a CTA

template <int WF>
struct PairGeom {
  static constexpr int NBLK = (WF == WF_MX) ? 2 : 4;       // 4-scale blocks of 256 K
  static constexpr int A_BYTES = 128 * 128;
  static constexpr int BOX_BYTES = kPairBox * 128;
  static constexpr int SFA_OFF = 2 * A_BYTES;              // codes: 128 weight rows, then 128 token rows
  static constexpr int SFB_OFF = SFA_OFF + NBLK * 512;
  static constexpr int STAGE = SFB_OFF + NBLK * 1024;      // 35 KB (MXFP4), 38 KB (NVFP4)
  static constexpr int STAGES = 5;
  static constexpr int SF_COLS = 12 * NBLK;                // TMEM columns of a stage's scales
  static constexpr int SF_TMEM = 512 - 2 * SF_COLS;
  static constexpr int TURN = 32 * 80;                     // an epilogue warp's turning space
  static constexpr size_t SMEM = (size_t)STAGES * STAGE + kPairEpi * TURN + 1024;
  static_assert(STAGE % 1024 == 0, "stages keep the 1024-byte swizzle alignment");
  static_assert(SMEM + 13 * 1024 <= 227 * 1024, "shared-memory budget");
};

template <int WF, bool WIDE>
__global__ void __launch_bounds__(kPairThreads, 1) fp4_matmul_pair_kernel(const __grid_constant__ MatmulArgs a) {
  using Geo = PairGeom<WF>;
  constexpr int S = Geo::STAGES, WORDS = kSfWords<WF>, NBLK = Geo::NBLK;
  extern __shared__ __align__(1024) uint8_t pm_raw[];
  __shared__ __align__(8) uint64_t full_bar[S];            // the even CTA's: both CTAs' copies and scales
  __shared__ __align__(8) uint64_t empty_bar[S];           // each CTA's: the MMAs of the stage are done
  __shared__ __align__(8) uint64_t accf_bar[2];            // each CTA's: an accumulator is complete
  __shared__ __align__(8) uint64_t free_bar;               // the even CTA's: the shared columns are read
  __shared__ __align__(8) uint64_t quiesce_bar;
  __shared__ uint32_t tmem_base_s;
  __shared__ int gave_up;                                  // a wait of this CTA has
  __shared__ MmGroups groups;

  cg::cluster_group cluster = cg::this_cluster();
  const uint32_t rank = cluster.block_rank();
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(pm_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid < S) {
    mbar_init(smem_u32(&full_bar[tid]), 1 + 2 * 3);        // the copies' bytes, three scale warps of each CTA
    mbar_init(smem_u32(&empty_bar[tid]), 1);
    mbar_fence_init();
  }
  if (tid == 32 * 2) {
    gave_up = 0;
    tmap_prefetch(&a.wmap);
    tmap_prefetch(&a.xmap);
    mbar_init(smem_u32(&accf_bar[0]), 1);
    mbar_init(smem_u32(&accf_bar[1]), 1);
    mbar_init(smem_u32(&free_bar), 2 * kPairEpi);
    mbar_init(smem_u32(&quiesce_bar), 1);
    mbar_fence_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(&tmem_base_s), 512);
    tmem_relinquish_pair();
  }
  wait_prior_grid();
  mm_scan_groups(a, groups);
  tc_fence_before();
  __syncthreads();
  cluster.sync();                                          // both CTAs' barriers and TMEM are ready
  tc_fence_after();
  const uint32_t tmem = tmem_base_s;
  const int nrb = (a.N + 255) / 256;
  const int nk = (a.K + 255) / 256;
  const unsigned first = blockIdx.x >> 1, step = gridDim.x >> 1;
  using Walk = MmWalk;

  if (warp == 0) {
    // ---------------- codes of this CTA's rows; their bytes count on the even CTA's barrier
    int s = 0, issued = 0;
    uint32_t ph = 0;
    bool failed = false;
    for (Walk m(a, groups, nrb, first, step); m.more() && !failed; m.next(a, groups)) {
      const int half = (m.nrows + 31) / 32 * 16;           // token rows of each CTA
      const int boxes = (half + kPairBox - 1) / kPairBox;
      const int wrow = m.rb * 256 + (int)rank * 128, xrow = m.row0 + (int)rank * half;
      for (int it = 0; it < nk; ++it) {
        if (issued >= S && !mm_wait_warp(smem_u32(&empty_bar[s]), ph ^ 1u, &gave_up, a.err, 71)) { failed = true; break; }
        const uint32_t bar = cluster_addr(smem_u32(&full_bar[s]), 0);
        const uint32_t st = smem_u32(smem + (size_t)s * Geo::STAGE);
        if (elect_one()) {
          if (rank == 0)
            mbar_arrive_expect_tx(smem_u32(&full_bar[s]), (uint32_t)(2 * (Geo::A_BYTES + boxes * Geo::BOX_BYTES)));
          tma_load_3d_pair(st, &a.wmap, bar, it * 128, wrow, m.g);
          for (int b = 0; b < boxes; ++b)
            tma_load_2d_pair(st + Geo::A_BYTES + b * Geo::BOX_BYTES, &a.xmap, bar, it * 128, xrow + b * kPairBox);
        }
        __syncwarp();
        ++issued;
        if (++s == S) { s = 0; ph ^= 1u; }
      }
    }
    // every copy of the pair has landed before it leaves (the other CTA waits at
    // the cluster's last barrier)
    if (rank == 0 && lane == 0) {
      int s2 = 0;
      uint32_t ph2 = 0;
      for (int i = 0; i < issued; ++i) {
        if (i >= issued - S) mbar_drain(smem_u32(&full_bar[s2]), ph2);
        if (++s2 == S) { s2 = 0; ph2 ^= 1u; }
      }
    }
  } else if (warp == 1) {
    // ---------------- MMAs of the pair, issued by the even CTA
    if (rank == 0) {
      int s = 0, n = 0, turn = 0;
      uint32_t ph = 0;
      bool failed = false;
      Walk m(a, groups, nrb, first, step);
      while (m.more() && !failed) {
        const int cols = __shfl_sync(0xffffffffu, (m.nrows + 31) / 32 * 32, 0);
        const uint32_t acc = tmem + ((n & 1) ? (uint32_t)(Geo::SF_TMEM - cols) : 0u);
        m.next(a, groups);                                 // ahead of the waits
        const uint32_t id0 = idesc_fp4_block(256, cols, WF == WF_MX, 0, 0);
        const uint32_t id2 = idesc_fp4_block(256, cols, WF == WF_MX, 2, 2);
        if (n > 0 && !mm_wait_warp(smem_u32(&free_bar), (n - 1) & 1, &gave_up, a.err, 72)) break;
        tc_fence_after();
        for (int it = 0; it < nk; ++it) {
          if (!mm_wait_warp(smem_u32(&full_bar[s]), ph, &gave_up, a.err, 73)) { failed = true; break; }
          tc_fence_after();
          const uint32_t st = smem_u32(smem + (size_t)s * Geo::STAGE);
          const uint32_t sf = tmem + (uint32_t)(Geo::SF_TMEM + turn * Geo::SF_COLS);
          if (elect_one()) {
#pragma unroll
            for (int b = 0; b < NBLK; ++b) {
              tc_cp_sf_block_pair(sf + 4 * b, st + Geo::SFA_OFF + 512 * b);
              tc_cp_sf_block_pair(sf + 4 * NBLK + 8 * b, st + Geo::SFB_OFF + 1024 * b);
              if (cols > 128) tc_cp_sf_block_pair(sf + 4 * NBLK + 8 * b + 4, st + Geo::SFB_OFF + 1024 * b + 512);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {                  // K = 64 an MMA
              const int blk = (WF == WF_MX) ? (k >> 1) : k;
              const uint32_t byte = (WF == WF_MX) ? (uint32_t)(2 * (k & 1)) : 0u;
              const uint64_t adesc = umma_desc(st + k * 32, 16, 1024, 2);
              const uint64_t bdesc = umma_desc(st + Geo::A_BYTES + k * 32, 16, 1024, 2);
              const uint32_t sfa = (sf + (uint32_t)(4 * blk)) | (byte << 30);
              const uint32_t sfb = (sf + (uint32_t)(4 * NBLK + 8 * blk)) | (byte << 30);
              const uint32_t accum = (it > 0 || k > 0) ? 1u : 0u;
              if constexpr (WF == WF_MX) umma_mxf4_pair(acc, adesc, bdesc, byte ? id2 : id0, sfa, sfb, accum);
              else umma_nvf4_pair(acc, adesc, bdesc, id0, sfa, sfb, accum);
            }
            tc_commit_pair(smem_u32(&empty_bar[s]), 3);
          }
          __syncwarp();
          turn ^= 1;
          if (++s == S) { s = 0; ph ^= 1u; }
        }
        if (failed) break;
        if (elect_one()) tc_commit_pair(smem_u32(&accf_bar[n & 1]), 3);
        __syncwarp();
        ++n;
      }
      __syncwarp();
      if (elect_one()) tc_commit_pair(smem_u32(&quiesce_bar), 1);   // all done, also after a wait gave up
      __syncwarp();
      mbar_drain(smem_u32(&quiesce_bar), 0);
    }
  } else if (warp < 2 + kPairEpi) {
    // ---------------- accumulators to y: TMEM lanes 32 * (w % 4) .. are weight rows,
    // columns are token rows
    const int quad = warp & 3, odd = (warp - 2) >> 2;
    uint8_t *turn = smem + (size_t)S * Geo::STAGE + (warp - 2) * Geo::TURN;
    const uint32_t free_even = cluster_addr(smem_u32(&free_bar), 0);
    const int es = a.dtype == MOE_DT_F32 ? 4 : 2;
    int n = 0;
    for (Walk m(a, groups, nrb, first, step); m.more(); m.next(a, groups), ++n) {
      const int buf = n & 1;
      const int chunks = (m.nrows + 31) / 32;
      const int col0 = m.rb * 256 + (int)rank * 128 + 32 * quad, col = col0 + lane;
      const bool rows16 = es == 2 && a.y_vec && col0 + 32 <= a.N;
      // the chunk of a turn: the first accumulator shares its last columns with the
      // second, which shares its first ones, so those chunks go first
      auto chunk = [&](int i) { return buf ? i : chunks - 1 - i; };
      float xG[4];                                         // this warp's chunks' row scales times the matrix's
      bool far = false;
      if constexpr (WF == WF_NV) {
        const float wG = __ldg(a.wG + m.g);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 32 * chunk(2 * i + odd) + lane;
          xG[i] = 2 * i + odd < chunks && r < m.nrows ? wG * __ldg(a.xG + m.row0 + r) : 1.0f;
        }
        far = !__all_sync(0xffffffffu, whole_factor(xG[0]) && whole_factor(xG[1]) && whole_factor(xG[2]) && whole_factor(xG[3]));
      }
      if (!mm_wait_warp(smem_u32(&accf_bar[buf]), (n >> 1) & 1, &gave_up, a.err, 74, nk)) break;
      tc_fence_after();
      const uint32_t acc = tmem + (buf ? (uint32_t)(Geo::SF_TMEM - 32 * chunks) : 0u) + ((uint32_t)(32 * quad) << 16);
      if constexpr (WF == WF_NV) {
        if (far) {
          const float wG = __ldg(a.wG + m.g);
          for (int t = odd; t < chunks; t += 2) {
            const int c = chunk(t);
            store_far(a, acc + (uint32_t)(32 * c), m.row0 + 32 * c, min(32, m.nrows - 32 * c), col, wG);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(free_even);
          continue;
        }
      }

      auto store = [&](const uint32_t (&d)[32], int c, float g) {
        const int have = min(32, m.nrows - 32 * c);
        float v[32];
#pragma unroll
        for (int j = 0; j < 32; ++j)
          v[j] = (WF == WF_NV) ? __uint_as_float(d[j]) * __shfl_sync(0xffffffffu, g, j) : __uint_as_float(d[j]);
        const int64_t at = (int64_t)(m.row0 + 32 * c) * a.ldy;
        if (rows16) {
          // 16-bit rows: turned over in shared memory to 64 bytes of a token's row
          uint16_t *mine = reinterpret_cast<uint16_t *>(turn) + lane;
          if (a.dtype == MOE_DT_BF16) {
#pragma unroll
            for (int j = 0; j < 32; ++j) mine[40 * j] = bf16_bits(v[j]);
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) mine[40 * j] = f16_bits(v[j]);
          }
          __syncwarp();
          uint16_t *y = static_cast<uint16_t *>(a.y) + at + col0 + 8 * (lane & 3);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int r = 8 * q + (lane >> 2);
            const uint4 w = *reinterpret_cast<const uint4 *>(turn + 80 * r + 16 * (lane & 3));
            if (r < have) *reinterpret_cast<uint4 *>(y + (int64_t)r * a.ldy) = w;
          }
          __syncwarp();
        } else if (col < a.N) {
          if (a.dtype == MOE_DT_F32) {
            float *y = static_cast<float *>(a.y) + at + col;
#pragma unroll
            for (int j = 0; j < 32; ++j, y += a.ldy)
              if (j < have) *y = v[j];
          } else {
            uint16_t *y = static_cast<uint16_t *>(a.y) + at + col;
#pragma unroll
            for (int j = 0; j < 32; ++j, y += a.ldy)
              if (j < have) *y = a.dtype == MOE_DT_BF16 ? bf16_bits(v[j]) : f16_bits(v[j]);
          }
        }
      };
      // a warp has at most two chunks with shared columns: once its first two turns
      // are in registers the next item may have them
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        const int t0 = 2 * i + odd, t1 = t0 + 2;
        uint32_t d0[32], d1[32];
        if (t0 < chunks) tmem_ld32(acc + (uint32_t)(32 * chunk(t0)), d0);
        if (t1 < chunks) tmem_ld32(acc + (uint32_t)(32 * chunk(t1)), d1);
        tmem_ld_wait();
        if (i == 0) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(free_even);
        }
        if (t0 < chunks) store(d0, chunk(t0), xG[i]);
        if (t1 < chunks) store(d1, chunk(t1), xG[i + 1]);
      }
    }
  } else {
    // ---------------- scales: `which` 0 the weights', 1 and 2 the tokens' halves
    const int which = warp - (2 + kPairEpi);
    const uint32_t off = (which == 0 ? Geo::SFA_OFF : Geo::SFB_OFF + 512 * (which - 1)) + 16 * lane;
    const int pitch = which == 0 ? 512 : 1024;             // between a stage's blocks
    const uint8_t *rowp[4];
    const uint8_t *lo = which ? a.xs : a.ws, *hi = lo + (which ? (size_t)a.rows : (size_t)a.groups * a.N) * a.nsf;
    bool wanted = false;                                   // the second half of a narrow tile is not read
    feed_scales<WF, S, false>(
        a, groups, Walk(a, groups, nrb, first, step), 0, nk, 0, 1,
        [&](const Walk &m) {
          wanted = which < 2 || m.nrows > 128;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            rowp[j] = which == 0
                          ? a.ws + ((size_t)m.g * a.N + min(m.rb * 256 + (int)rank * 128 + 32 * j + lane, a.N - 1)) * a.nsf
                          : a.xs + (size_t)min(m.row0 + 128 * (which - 1) + 32 * j + lane, a.rows - 1) * a.nsf;
        },
        [&](int it0, uint32_t(&w)[4][8]) { fetch_sf<WF, WIDE>(a, rowp, wanted ? 4 : 0, it0, nk, lo, hi, w); },
        [&](int s, uint32_t parity) { return mm_wait_warp(smem_u32(&empty_bar[s]), parity, &gave_up, a.err, 75); },
        [&](const Walk &) {
          return [&, store = wanted](int s, const uint32_t(&w)[4][8], int i) {
            if (!store) return;
            const uint32_t dst = smem_u32(smem + (size_t)s * Geo::STAGE) + off;
#pragma unroll
            for (int b = 0; b < WORDS; ++b)
              sts128(dst + pitch * b, make_uint4(w[0][i * WORDS + b], w[1][i * WORDS + b], w[2][i * WORDS + b],
                                                 w[3][i * WORDS + b]));
          };
        },
        [&](int s) {
          if (lane == 0) mbar_arrive_cluster(cluster_addr(smem_u32(&full_bar[s]), 0));
        });
  }

  __syncwarp();
  tc_fence_before();
  cluster.sync();                                          // no CTA leaves, or frees TMEM, while the other works
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

template <int WF, bool WIDE>
cudaError_t launch_pair(const MatmulArgs &a, int pairs, cudaStream_t s) {
  using Geo = PairGeom<WF>;
  auto fn = fp4_matmul_pair_kernel<WF, WIDE>;
  static std::atomic<uint64_t> asked{0};
  const cudaError_t e = ask_shared(fn, Geo::SMEM, asked);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * pairs));
  cfg.blockDim = dim3(kPairThreads);
  cfg.dynamicSmemBytes = Geo::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, fn, a);
}

}  // namespace

cudaError_t launch_matmul_pair(int wf, const MatmulArgs &a, int pairs, cudaStream_t s) {
  // scale rows at any byte take registers that cost the others a tenth (grouped
  // prefill 71 us; 66 with the kernel that has them on 16 bytes)
  if (wf == WF_MX) return a.sf_wide ? launch_pair<WF_MX, true>(a, pairs, s) : launch_pair<WF_MX, false>(a, pairs, s);
  return a.sf_wide ? launch_pair<WF_NV, true>(a, pairs, s) : launch_pair<WF_NV, false>(a, pairs, s);
}

}  // namespace moe
