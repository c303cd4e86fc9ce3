// Product of two block-scaled FP4 operands on pairs of SMs (tcgen05
// cta_group::2): the form for groups of many rows.  The formula, the operands'
// layouts and the treatment of groups are those of fp4_gemm.cuh.
//
// What bounds it.  At the FP4 rate of the tensor core the operands' way from L2
// into shared memory is the narrow place: an SM takes in about 60 bytes a cycle,
// and a unit of 128 weight rows x 192 activation rows on one SM needs 46 KB for
// 384 cycles of products (measured at N = K = 4096, 4096 rows: 42 us with the
// products, 33 us with the copies alone).  Two SMs that share a unit of 256
// weight rows x 256 activation rows each hold their own 128 weight rows and half
// of the activation rows: 38 KB for 512 cycles.  The copies of scales into tensor
// memory run on the same pipe as the products, 18 cycles each, twelve a stage of
// NVFP4 and six of MXFP4.
//
// Each CTA copies its weight rows, its half of the activation rows, its weights'
// scales and the scales of all activation rows into its own shared memory; every
// copy signals the leader's barrier.  The leader's warp 1 issues the pair's
// products and scale copies, and commits to the barriers of both.  The epilogue
// warps take a unit's accumulator (128 lanes x 256 columns a CTA) whole into
// registers, hand it back, and only then scale, round and store, under the next
// unit's products.  Roles of the warps as in fp4_gemm.cuh (2 and 3 also look up the
// rows' scales and places ahead of the epilogue).
//
// Measured (three sets of operands in turn): N = K = 4096, 4096 rows 28.7 us (4.8 PFLOP/s; the
// tensor pipe busy 48 % of it), 8192 x 8192 x 4096 87.4 us (6.3 PFLOP/s); 64 groups of 256 rows,
// N = 2816, K = 2048 55.0 us (318 MB moved, 5.8 TB/s).

#include "fp4_mma.cuh"

namespace b4 {

cudaError_t ensure_smem_limit(const void* func, size_t bytes);

namespace fp4 {

// NR: activation rows of a unit, 256 or 128.
template <int FMT, int NR>
struct PairCfg {
  static constexpr int kSfTiles = sf_tiles(FMT);
  static constexpr int kSfBytes = kSfTiles * kSfTile;               // scales of 128 rows of a stage
  static constexpr int kBlocks = NR / 128;                          // scale tiles of the activation rows
  static constexpr int kBox = NR / 4;                               // activation rows of a box: two a CTA
  static constexpr int kAStage = NR / 2 * 128;
  static constexpr int kStage = kWStage + kAStage + (1 + kBlocks) * kSfBytes;
  static constexpr int kStages = NR == 256 ? 5 : 7;
  static constexpr int kAccs = NR == 256 ? 1 : 2;
  static constexpr int kSfCols = 4 * kSfTiles * (1 + kBlocks);      // tensor-memory columns of a stage's scales
  static constexpr size_t a = (size_t)kStages * kWStage;
  static constexpr size_t sf = a + (size_t)kStages * kAStage;
  static constexpr size_t epi = sf + (size_t)kStages * (1 + kBlocks) * kSfBytes;
  static constexpr size_t rows = epi + kEpiBytes;
  static constexpr size_t bars = rows + sizeof(RowTable<NR>);
  static constexpr int kNumBars = 2 * kStages + 4 + 1 + 4;
  static constexpr size_t misc = bars + 8 * kNumBars;
  static constexpr size_t total(bool ragged) { return misc + 16 + (ragged ? sizeof(Groups) : 0); }
  static_assert(kAccs * NR + kStages * kSfCols <= 512, "a stage's scale columns are free once its shared memory is");
};

// LONG: the issuing loop is unrolled over the ring.
template <int FMT, int OUT, bool RAGGED, int NR, bool LONG>
__global__ void __launch_bounds__(kThreads, 1) fp4_pair_kernel(const __grid_constant__ Fp4GemmParams p) {
  using C = PairCfg<FMT, NR>;
  constexpr int NS = C::kStages;
  constexpr int kUnroll = LONG ? NS : 1;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw;  // aligned as declared: the swizzled stages need 1024 bytes
  Groups& groups = *reinterpret_cast<Groups*>(smem + C::misc + 16);  // ragged only
  uint8_t* s_a = smem + C::a;
  uint8_t* s_sf = smem + C::sf;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::bars);  // the leader's: copies of both CTAs
  uint64_t* empty = full + NS;                                   // each CTA's own
  uint64_t* full_acc = empty + NS;                               // each CTA's own
  uint64_t* empty_acc = full_acc + 2;                            // the leader's: epilogue warps of both
  uint64_t* drain = empty_acc + 2;
  uint64_t* full_rows = drain + 1;                               // each CTA's own, two deep
  uint64_t* empty_rows = full_rows + 2;
  RowTable<NR>& tab = *reinterpret_cast<RowTable<NR>*>(smem + C::rows);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + C::misc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + C::misc + 4);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const Abort ab{p.status, s_abort};

  if (threadIdx.x == 0) {
    *s_abort = 0;
    for (int i = 0; i < NS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(drain, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&full_acc[i], 1);
      mbar_init(&empty_acc[i], 2 * kEpiWarps);
      mbar_init(&full_rows[i], 2);
      mbar_init(&empty_rows[i], kEpiWarps);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(s_tmem, 512);
    tmem_relinquish_pair();
  }
  if (!p.a_is_new) pdl_wait();  // standalone: every input may come from the kernel before
  const int wpairs = cdiv(p.n, 256);
  if (RAGGED) build_groups<NR>(p, groups);
  tc_fence_before();
  cluster_sync();  // both CTAs' barriers exist before either signals
  tc_fence_after();
  if (threadIdx.x == 0) pdl_launch_dependents();
  const uint32_t tmem = *s_tmem;
  int n_units = (RAGGED ? groups.tiles[p.groups] : p.groups * cdiv(p.m, NR)) * wpairs;
  if (!RAGGED && NR == 256) n_units += max(n_units - p.halves_from, 0);
  const int k64 = cdiv(p.k, 64);                       // matrix instructions along K
  const int stages = cdiv(k64, 4);
  const int k_tiles = cdiv(p.k, 4 * fp4_group(FMT));   // scale tiles along K
  const int wtiles = cdiv(p.n, 128);
  const int u0 = blockIdx.x >> 1, du = gridDim.x >> 1;

  if (warp == 0) {
    // ----------------------------------------------------------- copies
    if (p.a_is_new) pdl_wait();
    uint32_t ss = 0;
    bool ok = true;
    const uint32_t full0 = warp_uniform(map_rank(full, 0));
    for (int u = u0; u < n_units && ok; u += du) {
      const Unit U = get_unit<NR, RAGGED>(p, groups, wpairs, u);
      const int rows = (int)warp_uniform(U.rows), first = (int)warp_uniform(U.first);
      const int group = (int)warp_uniform(U.group), atile = (int)warp_uniform(U.atile);
      const int wtile = 2 * (int)warp_uniform(U.wtile) + (int)rank;
      const int half = round_up(rows, 32) / 2;  // activation rows a CTA holds
      const bool two = rows > 128;
      const bool boxes2 = half > C::kBox;
      const int wrow = group * p.n + wtile * 128;
      const int arow = first + (int)rank * half;
      const int wsf = (group * wtiles + wtile) * k_tiles, asf = atile * k_tiles;
      const uint32_t bytes = 2 * (kWStage + (boxes2 ? 2 : 1) * C::kBox * 128 + (two ? 3 : 2) * C::kSfBytes);
      for (int s = 0; s < stages; ++s, ++ss) {
        const uint32_t slot = ss % NS;
        ok = __all_sync(0xffffffffu, wait(&empty[slot], ((ss / NS) & 1) ^ 1, ab, 111));
        if (!ok) break;
        const int kt0 = s * C::kSfTiles;
        uint8_t* sf = s_sf + slot * (1 + C::kBlocks) * C::kSfBytes;
        uint8_t* sa = s_a + slot * C::kAStage;
        const uint32_t bar = full0 + 8 * slot;
        if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(&full[slot], bytes);
          tma_load_2d_pair(smem + slot * kWStage, &p.tmap_w, s * 128, wrow, bar);
          tma_load_2d_pair(sa, &p.tmap_a, s * 128, arow, bar);
          if (boxes2) tma_load_2d_pair(sa + C::kBox * 128, &p.tmap_a, s * 128, arow + C::kBox, bar);
          // (a box past the row tile's last scale tile brings the next tile's, which no product reads)
          tma_load_2d_pair(sf, &p.tmap_ws, 0, wsf + kt0, bar);
          tma_load_2d_pair(sf + C::kSfBytes, &p.tmap_as, 0, asf + kt0, bar);
          if (C::kBlocks > 1 && two) tma_load_2d_pair(sf + 2 * C::kSfBytes, &p.tmap_as, 0, asf + k_tiles + kt0, bar);
        }
        __syncwarp();
      }
    }
    if (ab.raised() && lane == 0) {
      // copies already issued land before the CTA's shared memory goes away:
      // their barrier may be the other CTA's, so give them a fixed time
      const unsigned long long t0 = globaltimer();
      while (globaltimer() - t0 < 2000000ull) {
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------- matrix instructions
    if (rank == 0) {
      // Where a pair takes many units the loop over a stage's slot is unrolled over the
      // ring, so that slots and scale columns are constants: with them in registers a
      // stage takes longer to issue than its products take to run (8192 x 8192 x 4096 87.5
      // us, rolled 88.2; 4096^3 28.7 and 29.0).  In one round or two the smaller code, fetched cold, gains more
      // (N = K = 4096, 1024 rows 11.3 us, unrolled 11.7; N = 2048, K = 1408, 1024 rows 6.5, 6.8).
      const uint32_t w_desc = desc_lo(smem_u32(smem)), a_desc = desc_lo(smem_u32(s_a)), s_desc = desc_lo(smem_u32(s_sf));
      uint32_t phase = 0, acc_i = 0, d = 0, abuf = 0;
      int u = u0, s = 0;
      uint32_t idesc = 0;
      bool two = false;
      bool ok = u < n_units;
      bool seen = false;  // the stage's copies were seen complete during the stage before
      while (ok) {
#pragma unroll kUnroll
        for (int slot = 0; slot < NS; ++slot) {
          if (s == 0) {
            const int rows = (int)warp_uniform(get_unit<NR, RAGGED>(p, groups, wpairs, u).rows);
            two = C::kBlocks > 1 && rows > 128;
            idesc = idesc_fp4(FMT, 256, (uint32_t)round_up(rows, 32));
            abuf = acc_i % C::kAccs;
            ok = __all_sync(0xffffffffu, wait(&empty_acc[abuf], ((acc_i / C::kAccs) & 1) ^ 1, ab, 112));
            if (!ok) break;
            if constexpr (C::kAccs > 1) d = abuf * NR;
            ++acc_i;
          }
          if (!seen) {
            ok = __all_sync(0xffffffffu, wait(&full[slot], phase, ab, 114));
            if (!ok) break;
          }
          tc_fence_after();
          // the next stage's barrier, looked at while this stage's instructions issue
          const bool look = mbar_test(&full[(slot + 1) % NS], slot + 1 == NS ? phase ^ 1 : phase);
          const int kn = min(4, k64 - 4 * s);
          const bool last = s + 1 == stages;
          if (elect_one()) {
            constexpr uint32_t kStep = kSfTile / 16;
            const uint32_t sfw = C::kAccs * NR + slot * C::kSfCols, sfa = sfw + 4 * C::kSfTiles;
            const uint32_t sd = s_desc + slot * ((1 + C::kBlocks) * C::kSfBytes / 16);
            const uint32_t wd = w_desc + slot * (kWStage / 16), ad = a_desc + slot * (C::kAStage / 16);
            // (past the last scale tile of K the copies bring what no product reads)
#pragma unroll
            for (int i = 0; i < C::kSfTiles; ++i) {
              copy_scales<2>(sfw + 4 * i, sd + i * kStep);
              copy_scales<2>(sfa + 4 * C::kBlocks * i, sd + C::kSfBytes / 16 + i * kStep);
            }
            if (two) {
#pragma unroll
              for (int i = 0; i < C::kSfTiles; ++i) copy_scales<2>(sfa + 4 * C::kBlocks * i + 4, sd + 2 * C::kSfBytes / 16 + i * kStep);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (i < kn) {
                const int t = FMT == 0 ? i : i >> 1;  // MXFP4: a scale tile serves two instructions
                const uint32_t sf = FMT == 0 ? 0 : 2 * (i & 1);
                mma_fp4<FMT, 2>(d, wd + 2 * i, ad + 2 * i, idesc | sf << 4 | sf << 29, sfw + 4 * t, sfa + 4 * C::kBlocks * t,
                                i > 0 || s > 0);
              }
            mma_commit_pair(&empty[slot]);
            if (last) mma_commit_pair(&full_acc[abuf]);
          }
          seen = __all_sync(0xffffffffu, look);
          ++s;
          if (last) {
            s = 0;
            u += du;
            ok = u < n_units;
            if (!ok) break;
          }
        }
        phase ^= 1;
      }
      // drain: every instruction issued has completed
      if (elect_one()) mma_commit_pair(drain);
      const unsigned long long t0 = globaltimer();
      while (!mbar_try_wait(drain, 0) && globaltimer() - t0 < kWaitLimitNs) {
      }
      __syncwarp();
    }
  } else if (warp < 4) {
    // ------- the epilogue's row tables; rows past the last group are zero
    if (p.a_is_new) pdl_wait();
    fill_rows<NR, RAGGED>(p, groups, tab, full_rows, empty_rows, wpairs, u0, du, n_units, ab);
    if (RAGGED && !p.out_rows) clear_tail(p, groups.first[p.groups], threadIdx.x - 64);
  } else {
    // --------------------------------------------------------- epilogue
    if (p.a_is_new) pdl_wait();
    constexpr int kChunks = NR / 64;  // 32-row chunks a warp takes
    const int q4 = warp & 3;
    const int turn = (warp - 4) >> 2;
    uint8_t* stage = smem + C::epi + (warp - 4) * 32 * kEpiRow;
    const uint32_t done = map_rank(empty_acc, 0);
    const uint32_t taddr = tmem + ((uint32_t)(32 * q4) << 16) + 32 * turn;
    uint32_t i = 0;
    for (int u = u0; u < n_units; u += du, ++i) {
      const uint32_t b = i & 1;
      bool ok = wait(&full_rows[b], (i >> 1) & 1, ab, 107);
      if (!__all_sync(0xffffffffu, ok)) break;
      const int rows = tab.rows[b];
      const uint32_t abuf = i % C::kAccs;
      ok = wait(&full_acc[abuf], (i / C::kAccs) & 1, ab, 115);
      if (!__all_sync(0xffffffffu, ok)) break;
      const int n0 = (2 * tab.wtile[b] + (int)rank) * 128 + 32 * q4;
      tc_fence_after();
      uint32_t lo[kChunks][16], hi[kChunks][16];
#pragma unroll
      for (int c = 0; c < kChunks; ++c)
        if (64 * c + 32 * turn < rows) {
          tmem_ld16x256b_x4(taddr + abuf * NR + 64 * c, lo[c]);
          tmem_ld16x256b_x4(taddr + abuf * NR + (16u << 16) + 64 * c, hi[c]);
        }
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(done + 8 * abuf);
#pragma unroll
      for (int c = 0; c < kChunks; ++c)
        if (64 * c + 32 * turn < rows && n0 < p.n) {
          const int r = 64 * c + 32 * turn;
          store_chunk<OUT>(p, lo[c], hi[c], RowInfo{tab.g[b] + r, tab.to[b] + r}, n0, stage, lane);
        }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty_rows[b]);
    }
  }

  tc_fence_before();
  cluster_sync();  // neither CTA leaves while the pair's copies, products or signals may touch it
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

template <int FMT, int OUT, bool RAGGED, int NR, bool LONG>
cudaError_t launch_pair(const Fp4GemmParams& p, int pairs, bool pdl, cudaStream_t stream) {
  auto kern = fp4_pair_kernel<FMT, OUT, RAGGED, NR, LONG>;
  const size_t smem = PairCfg<FMT, NR>::total(RAGGED);
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * pairs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace fp4

// nr: activation rows of a unit, 128 or 256; the activation map's box holds a quarter of
// them.  rounds: units a pair takes at most.
cudaError_t launch_fp4_gemm_pair(const Fp4GemmParams& p, int fmt, int nr, int pairs, int rounds, bool pdl,
                                 cudaStream_t stream) {
  return fp4::with_forms(p, fmt, [&](auto f, auto out, auto ragged) {
    constexpr int F = f.value, O = out.value;
    constexpr bool G = ragged.value;
    const bool many = G || rounds > 2;
    if (nr == 128)
      return many ? fp4::launch_pair<F, O, G, 128, true>(p, pairs, pdl, stream)
                  : fp4::launch_pair<F, O, G, 128, G>(p, pairs, pdl, stream);
    return many ? fp4::launch_pair<F, O, G, 256, true>(p, pairs, pdl, stream)
                : fp4::launch_pair<F, O, G, 256, G>(p, pairs, pdl, stream);
  });
}

}  // namespace b4
