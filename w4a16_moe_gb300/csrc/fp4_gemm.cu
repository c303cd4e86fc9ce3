// Product of two block-scaled FP4 operands on tcgen05 (sm_103a), dense and
// grouped by expert with ragged sizes:
//
//   out[t][n] = gs_a[t] gs_w[e] sum_k (c s)_a[t][k] (c s)_w[e][n][k]
//
// for the rows t of group e.  The tensor core multiplies the E2M1 codes, applies
// both operands' block scales and accumulates in fp32 (tcgen05.mma with
// .block_scale: NVFP4 as kind::mxf4nvf4 with an E4M3 scale per 16 along K, MXFP4
// as kind::mxf4 with an E8M0 scale per 32); the epilogue applies the two global
// scales and rounds once.
//
// Weights are on M (128 rows a unit), activation rows on N (up to NT a unit,
// the instruction's N the unit's rows rounded up to 16): a group of few rows
// then costs few tensor-core cycles, and its weight tile streams through once.
// Operands come by TMA as 128-byte rows (256 K) with the 128-byte swizzle, the
// scales as whole 512-byte tiles by bulk copies next to them and from shared
// into tensor memory by tcgen05.cp, which the instructions that read them
// follow in order.  Roles of the twelve warps: 0 copies, 1 matrix instructions,
// 2 and 3 the epilogue's tables of row scales and places, and zeros in rows of a
// ragged output past the last group, 4 to 11 epilogue.
// Two accumulators, so a unit's epilogue runs under the next unit's products.
// Every wait is bounded (ptx.cuh).

#include "fp4_mma.cuh"

namespace b4 {

cudaError_t ensure_smem_limit(const void* func, size_t bytes);

namespace fp4 {

// FMT 0 NVFP4, 1 MXFP4; NT: activation rows of a unit.
template <int FMT, int NT>
struct Cfg {
  static constexpr int kSfTiles = sf_tiles(FMT);
  static constexpr int kSfRows = kSfTiles * kSfTile;            // scales of 128 rows of a stage
  static constexpr int kABlocks = NT > 64 ? 2 : 1;              // 128-row scale tiles a unit's rows touch
  static constexpr int kAStage = NT * 128;
  static constexpr int kStage = kWStage + kAStage + 2048 * (1 + kABlocks);
  static constexpr int kStages = (214 * 1024 - kEpiBytes - (int)sizeof(RowTable<NT>)) / kStage;
  static constexpr int kSfCols = 4 * kSfTiles * (1 + kABlocks);  // tensor-memory columns of a stage's scales
  // scale buffers in tensor memory: one per stage where they fit, then a stage's
  // scales are free to overwrite once its shared memory is
  static constexpr int kSfFit = (512 - 2 * NT) / kSfCols;
  static constexpr int kSfRing = kSfFit < kStages ? kSfFit : kStages;
  static constexpr uint32_t kTmemCols = 512;
  static constexpr size_t a = (size_t)kStages * kWStage;
  static constexpr size_t sf = a + (size_t)kStages * kAStage;
  static constexpr size_t epi = sf + (size_t)kStages * 2048 * (1 + kABlocks);
  static constexpr size_t rows = epi + kEpiBytes;
  static constexpr size_t bars = rows + sizeof(RowTable<NT>);
  static constexpr int kNumBars = 2 * kStages + 4 + 1 + 4;
  static constexpr size_t misc = bars + 8 * kNumBars;
  static constexpr size_t total = misc + 16 + 1024;             // + alignment slack
  static_assert(kSfRing >= 2, "tensor memory budget");
  static_assert(kAStage % 1024 == 0, "swizzle atoms stay 1024-byte aligned");
};

template <int FMT, int NT, int OUT, bool RAGGED>
__global__ void __launch_bounds__(kThreads, 1) fp4_gemm_kernel(const __grid_constant__ Fp4GemmParams p) {
  using C = Cfg<FMT, NT>;
  constexpr int NS = C::kStages;
  constexpr int kBox = fp4_box_rows(NT);
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ Groups groups;
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* s_a = smem + C::a;
  uint8_t* s_sf = smem + C::sf;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::bars);
  uint64_t* empty = full + NS;
  uint64_t* full_acc = empty + NS;
  uint64_t* empty_acc = full_acc + 2;
  uint64_t* drain = empty_acc + 2;
  uint64_t* full_rows = drain + 1;
  uint64_t* empty_rows = full_rows + 2;
  RowTable<NT>& tab = *reinterpret_cast<RowTable<NT>*>(smem + C::rows);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + C::misc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + C::misc + 4);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const Abort ab{p.status, s_abort};

  if (threadIdx.x == 0) {
    *s_abort = 0;
    for (int i = 0; i < NS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&full_acc[i], 1);
      mbar_init(&empty_acc[i], kEpiWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&full_rows[i], 2);
      mbar_init(&empty_rows[i], kEpiWarps);
    }
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(s_tmem, C::kTmemCols);
    tmem_relinquish();
  }
  if (!p.a_is_new) pdl_wait();  // standalone: every input may come from the kernel before

  const int wtiles = cdiv(p.n, 128);
  if (RAGGED) build_groups<NT>(p, groups);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0) pdl_launch_dependents();
  const uint32_t tmem = *s_tmem;
  const int n_units = (RAGGED ? groups.tiles[p.groups] : p.groups * cdiv(p.m, NT)) * wtiles;
  const int k64 = cdiv(p.k, 64);                       // matrix instructions along K
  const int stages = cdiv(k64, 4);
  const int k_tiles = cdiv(p.k, 4 * fp4_group(FMT));   // scale tiles along K

  if (warp == 0) {
    // ----------------------------------------------------------- copies
    // (the whole warp loops and one elected lane issues, as for the products)
    if (p.a_is_new) pdl_wait();
    const uint32_t tile_pitch = (uint32_t)k_tiles * kSfTile;
    uint32_t ss = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < n_units && ok; u += gridDim.x) {
      const Unit U = get_unit<NT, RAGGED>(p, groups, wtiles, u);
      const int rows = (int)warp_uniform(U.rows), shift = (int)warp_uniform(U.shift);
      const int first = (int)warp_uniform(U.first), atile = (int)warp_uniform(U.atile);
      const int group = (int)warp_uniform(U.group), wtile = (int)warp_uniform(U.wtile);
      const int boxes = (rows + kBox - 1) / kBox;
      const bool two = C::kABlocks == 2 && shift * 32 + rows > 128;
      const uint8_t* wsf = p.w_scales + ((size_t)group * wtiles + wtile) * tile_pitch;
      const uint8_t* asf = p.a_scales + (size_t)atile * tile_pitch;
      const int wrow = group * p.n + wtile * 128;
      const uint32_t code_bytes = kWStage + boxes * kBox * 128;
      for (int s = 0; s < stages; ++s, ++ss) {
        const uint32_t slot = ss % NS;
        ok = __all_sync(0xffffffffu, wait(&empty[slot], ((ss / NS) & 1) ^ 1, ab, 101));
        if (!ok) break;
        const int kt0 = s * C::kSfTiles;
        const uint32_t sfb = (uint32_t)min(C::kSfTiles, k_tiles - kt0) * kSfTile;
        uint8_t* sf = s_sf + slot * 2048 * (1 + C::kABlocks);
        uint8_t* sa = s_a + slot * C::kAStage;
        if (elect_one()) {
          mbar_arrive_expect_tx(&full[slot], code_bytes + (two ? 3 : 2) * sfb);
          tma_load_2d(smem + slot * kWStage, &p.tmap_w, s * 128, wrow, &full[slot]);
          bulk_g2s(sf, wsf + kt0 * kSfTile, sfb, &full[slot]);
          tma_load_2d(sa, &p.tmap_a, s * 128, first, &full[slot]);
#pragma unroll
          for (int b = 1; b < NT / kBox; ++b)
            if (b < boxes) tma_load_2d(sa + b * kBox * 128, &p.tmap_a, s * 128, first + b * kBox, &full[slot]);
          bulk_g2s(sf + 2048, asf + kt0 * kSfTile, sfb, &full[slot]);
          if (two) bulk_g2s(sf + 4096, asf + tile_pitch + kt0 * kSfTile, sfb, &full[slot]);
        }
        __syncwarp();
      }
    }
    if (ab.raised() && lane == 0) {
      // let copies already issued land before the CTA's shared memory goes away
      const uint32_t n = ss < (uint32_t)NS ? ss : (uint32_t)NS;
      for (uint32_t i = ss - n; i < ss; ++i) {
        const unsigned long long t0 = globaltimer();
        while (!mbar_try_wait(&full[i % NS], (i / NS) & 1) && globaltimer() - t0 < kWaitLimitNs) {
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------- matrix instructions
    // The whole warp runs the loop and one elected lane issues: every operand
    // is then warp-uniform to the compiler, which keeps descriptors in uniform
    // registers.  (Issued from a one-lane branch the same instructions took
    // 100 - 120 cycles each, five times what the tensor core needs.)
    uint32_t ss = 0, acc_i = 0;
    constexpr uint32_t tm = 0;  // all of tensor memory: it starts at column 0
    const uint32_t w_desc = desc_lo(smem_u32(smem)), a_desc = desc_lo(smem_u32(s_a)), s_desc = desc_lo(smem_u32(s_sf));
    for (int u = blockIdx.x; u < n_units; u += gridDim.x) {
      const Unit U = get_unit<NT, RAGGED>(p, groups, wtiles, u);
      const int rows = (int)warp_uniform(U.rows), shift = (int)warp_uniform(U.shift);
      const bool two = C::kABlocks == 2 && shift * 32 + rows > 128;
      const uint32_t idesc = idesc_fp4(FMT, 128, (uint32_t)round_up(rows, 16));
      const uint32_t abuf = acc_i & 1;
      if (!__all_sync(0xffffffffu, wait(&empty_acc[abuf], ((acc_i >> 1) & 1) ^ 1, ab, 102))) break;
      tc_fence_after();
      const uint32_t d = tm + abuf * NT;
      bool ok = true;
      for (int s = 0; s < stages; ++s, ++ss) {
        const uint32_t slot = ss % NS;
        // with fewer scale buffers than stages, the products that last read this one come first
        if (C::kSfRing < NS && ss >= C::kSfRing)
          ok = wait(&empty[(ss - C::kSfRing) % NS], ((ss - C::kSfRing) / NS) & 1, ab, 103);
        ok = ok && wait(&full[slot], (ss / NS) & 1, ab, 104);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t sfw = tm + 2 * NT + (ss % C::kSfRing) * C::kSfCols;
        const uint32_t sfa = sfw + 4 * C::kSfTiles;
        const uint32_t sd = s_desc + slot * (2048 * (1 + C::kABlocks) / 16);
        const uint32_t wd = w_desc + slot * (kWStage / 16), ad = a_desc + slot * (C::kAStage / 16);
        const int kts = min(C::kSfTiles, k_tiles - s * C::kSfTiles);
        const int kn = min(4, k64 - 4 * s);
        if (elect_one()) {
#pragma unroll
          for (int i = 0; i < C::kSfTiles; ++i)
            if (i < kts) {
              copy_scales<1>(sfw + 4 * i, sd + i * (kSfTile / 16));
              copy_scales<1>(sfa + 4 * i * C::kABlocks, sd + 128 + i * (kSfTile / 16));
              if (two) copy_scales<1>(sfa + 4 * (i * C::kABlocks + 1), sd + 256 + i * (kSfTile / 16));
            }
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i < kn) {
              const int t = FMT == 0 ? i : i >> 1;  // MXFP4: a scale tile serves two instructions
              const uint32_t sf = FMT == 0 ? 0 : 2 * (i & 1);
              mma_fp4<FMT, 1>(d, wd + 2 * i, ad + 2 * i, idesc | sf << 4 | sf << 29, sfw + 4 * t,
                           sfa + 4 * t * C::kABlocks + shift, s > 0 || i > 0);
            }
          mma_commit(&empty[slot]);
          if (s + 1 == stages) mma_commit(&full_acc[abuf]);
        }
        __syncwarp();
      }
      if (!ok) break;
      ++acc_i;
    }
    // drain: every instruction issued has completed
    if (elect_one()) mma_commit(drain);
    const unsigned long long t0 = globaltimer();
    while (!mbar_try_wait(drain, 0) && globaltimer() - t0 < kWaitLimitNs) {
    }
    __syncwarp();
  } else if (warp < 4) {
    // ------- the epilogue's row tables; rows past the last group are zero
    if (p.a_is_new) pdl_wait();
    fill_rows<NT, RAGGED>(p, groups, tab, full_rows, empty_rows, wtiles, blockIdx.x, gridDim.x, n_units, ab);
    if (RAGGED && !p.out_rows) clear_tail(p, groups.first[p.groups], threadIdx.x - 64);
  } else {
    // --------------------------------------------------------- epilogue
    if (p.a_is_new) pdl_wait();
    static_assert(NT == 64, "a chunk for each warp");
    const int q4 = warp & 3;
    const int turn = (warp - 4) >> 2;
    uint8_t* stage = smem + C::epi + (warp - 4) * 32 * kEpiRow;
    uint32_t i = 0;
    for (int u = blockIdx.x; u < n_units; u += gridDim.x, ++i) {
      const uint32_t b = i & 1;
      bool ok = wait(&full_rows[b], (i >> 1) & 1, ab, 107);
      ok = ok && wait(&full_acc[b], (i >> 1) & 1, ab, 105);
      if (!__all_sync(0xffffffffu, ok)) break;
      const int rows = tab.rows[b];
      const int n0 = tab.wtile[b] * 128 + 32 * q4;
      tc_fence_after();
      const uint32_t taddr = tmem + ((uint32_t)(32 * q4) << 16) + b * NT + 32 * turn;
      if (32 * turn < rows) {
        uint32_t lo[16], hi[16];
        tmem_ld16x256b_x4(taddr, lo);
        tmem_ld16x256b_x4(taddr + (16u << 16), hi);
        const int r = 32 * turn + lane;
        const RowInfo info{tab.g[b][r], tab.to[b][r]};
        tmem_ld_wait();
        if (n0 < p.n) store_chunk<OUT>(p, lo, hi, info, n0, stage, lane);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&empty_acc[b]);
        mbar_arrive(&empty_rows[b]);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, C::kTmemCols);
}

template <int FMT, int OUT, bool RAGGED, int NT = 64>
cudaError_t launch(const Fp4GemmParams& p, int grid, bool pdl, cudaStream_t stream) {
  auto kern = fp4_gemm_kernel<FMT, NT, OUT, RAGGED>;
  const size_t smem = Cfg<FMT, NT>::total;
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace fp4

cudaError_t launch_fp4_gemm(const Fp4GemmParams& p, int fmt, int grid, bool pdl, cudaStream_t stream) {
  return fp4::with_forms(p, fmt, [&](auto f, auto out, auto ragged) {
    return fp4::launch<f.value, out.value, ragged.value>(p, grid, pdl, stream);
  });
}

}  // namespace b4
