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
// This is the form for groups of few rows, bound by the stream of weights
// (fp4_gemm_pair.cu is the one for many rows).  Weights are on M (128 rows a
// unit), activation rows on N (up to 64 a unit, the instruction's N the unit's
// rows rounded up to 16), so a group of few rows costs few tensor-core cycles and
// its weight tile streams through once.  Operands come by TMA as 128-byte rows
// (256 K) with the 128-byte swizzle, the scales as whole 512-byte tiles by bulk
// copies next to them and from shared into tensor memory by tcgen05.cp, which the
// instructions that read them follow in order.  Roles of the twelve warps:
// 0 copies, 1 matrix instructions, 2 and 3 the epilogue's tables of row scales and
// places, and zeros in rows of a ragged output past the last group, 4 to 11
// epilogue.  Two accumulators, so a unit's epilogue runs under the next unit's
// products.  As the second kernel of a call, it fills its ring with weights while
// the quantiser still runs.
//
// SPLIT: where the units are fewer than the SMs, a cluster of 2 to 8 CTAs shares
// a unit along K.  The partial accumulators go to the first CTA's shared memory
// as asynchronous stores that count on its barrier, and it adds them in rank
// order, so the result does not depend on timing.
//
// Every wait is bounded (ptx.cuh).

#include "fp4_mma.cuh"

namespace b4 {

cudaError_t ensure_smem_limit(const void* func, size_t bytes);

namespace fp4 {

constexpr int kRows = 64;                       // activation rows of a unit
constexpr int kBox = 32;                        // rows of an activation box
constexpr int kPart16 = 4 * 32 * 16 * 4;        // bytes of 16 rows' partial sums: 4 warps x 32 lanes x 16 values

template <int FMT, bool SPLIT>
struct Cfg {
  static constexpr int kSfTiles = sf_tiles(FMT);
  static constexpr int kSfBytes = kSfTiles * kSfTile;           // scales of 128 rows of a stage
  static constexpr int kAStage = kRows * 128;
  static constexpr int kStage = kWStage + kAStage + 2 * kSfBytes;
  static constexpr int kPart = SPLIT ? kSplitPartBytes : 0;
  static constexpr int kFit = (216 * 1024 - kEpiBytes - (int)sizeof(RowTable<kRows>) - kPart) / kStage;
  static constexpr int kStages = kFit < 7 ? kFit : 7;
  static constexpr int kSfCols = 8 * kSfTiles;                  // tensor-memory columns of a stage's scales
  static constexpr size_t a = (size_t)kStages * kWStage;
  static constexpr size_t sf = a + (size_t)kStages * kAStage;
  static constexpr size_t part = sf + (size_t)kStages * 2 * kSfBytes;
  static constexpr size_t epi = part + kPart;
  static constexpr size_t rows = epi + kEpiBytes;
  static constexpr size_t bars = rows + sizeof(RowTable<kRows>);
  static constexpr int kNumBars = 2 * kStages + 4 + 1 + 4 + 1;
  static constexpr size_t misc = bars + 8 * kNumBars;
  static constexpr size_t total(bool ragged) { return misc + 16 + (ragged ? sizeof(Groups) : 0); }
  static_assert(2 * kRows + kStages * kSfCols <= 512, "a stage's scale columns are free once its shared memory is");
  static_assert(kStages >= 3, "shared memory budget");
};

template <int FMT, int OUT, bool RAGGED, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1) fp4_gemm_kernel(const __grid_constant__ Fp4GemmParams p) {
  using C = Cfg<FMT, SPLIT>;
  constexpr int NS = C::kStages;
  constexpr int kUnroll = SPLIT ? NS : 1;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw;  // aligned as declared: the swizzled stages need 1024 bytes
  Groups& groups = *reinterpret_cast<Groups*>(smem + C::misc + 16);  // ragged only
  uint8_t* s_a = smem + C::a;
  uint8_t* s_sf = smem + C::sf;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::bars);
  uint64_t* empty = full + NS;
  uint64_t* full_acc = empty + NS;
  uint64_t* empty_acc = full_acc + 2;
  uint64_t* drain = empty_acc + 2;
  uint64_t* full_rows = drain + 1;
  uint64_t* empty_rows = full_rows + 2;
  uint64_t* part_bar = empty_rows + 2;  // SPLIT: the other CTAs' partial sums have arrived
  RowTable<kRows>& tab = *reinterpret_cast<RowTable<kRows>*>(smem + C::rows);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + C::misc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + C::misc + 4);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int splits = SPLIT ? (int)cluster_size() : 1;
  const int rank = SPLIT ? (int)cluster_rank() : 0;
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
      mbar_init(&full_rows[i], 2);
      mbar_init(&empty_rows[i], kEpiWarps);
    }
    mbar_init(drain, 1);
    mbar_init(part_bar, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(s_tmem, 512);
    tmem_relinquish();
  }
  if (!p.a_is_new) pdl_wait();  // standalone: every input may come from the kernel before

  const int wtiles = cdiv(p.n, 128);
  if (RAGGED) build_groups<kRows>(p, groups);
  tc_fence_before();
  if constexpr (SPLIT) cluster_sync();  // every CTA's barriers exist before another signals them
  else __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0) pdl_launch_dependents();
  const uint32_t tmem = *s_tmem;
  const int n_units = (RAGGED ? groups.tiles[p.groups] : p.groups * cdiv(p.m, kRows)) * wtiles;
  const int k64 = cdiv(p.k, 64);                       // matrix instructions along K
  const int k_tiles = cdiv(p.k, 4 * fp4_group(FMT));   // scale tiles along K
  const int all_stages = cdiv(k64, 4);
  // this CTA's stages, and its units: a cluster takes one
  const int s_beg = SPLIT ? rank * all_stages / splits : 0;
  const int s_end = SPLIT ? (rank + 1) * all_stages / splits : all_stages;
  const int u0 = SPLIT ? (int)blockIdx.x / splits : (int)blockIdx.x;
  const int du = SPLIT ? n_units : (int)gridDim.x;

  if (warp == 0) {
    // ----------------------------------------------------------- copies
    // (the whole warp loops and one elected lane issues, so that operands stay
    // in uniform registers; unrolled over the ring, so that addresses are constant)
    const uint32_t tile_pitch = (uint32_t)k_tiles * kSfTile;
    uint32_t phase = 1;
    int u = u0, s = s_beg;
    bool ok = u < n_units;
    // while the kernel before still writes the activations: weights first, for as
    // much of the ring as the first unit fills
    int early = 0;
    if (p.a_is_new) {
      early = ok ? min(NS, s_end - s_beg) : 0;
      if (early == 0) pdl_wait();
    }
    int boxes = 0, first = 0, wrow = 0;
    const uint8_t *wsf = nullptr, *asf = nullptr;
    auto load_unit = [&]() {
      const Unit U = get_unit<kRows, RAGGED>(p, groups, wtiles, u);
      boxes = ((int)warp_uniform(U.rows) + kBox - 1) / kBox;
      first = (int)warp_uniform(U.first);
      const int group = (int)warp_uniform(U.group), wtile = (int)warp_uniform(U.wtile);
      wsf = p.w_scales + ((size_t)group * wtiles + wtile) * tile_pitch;
      asf = p.a_scales + (size_t)warp_uniform(U.atile) * tile_pitch;
      wrow = group * p.n + wtile * 128;
    };
    auto sf_bytes = [&](int st) { return (uint32_t)min(C::kSfTiles, k_tiles - st * C::kSfTiles) * kSfTile; };
    auto copy_w = [&](int slot, int st) {
      mbar_arrive_expect_tx(&full[slot], kWStage + boxes * kBox * 128 + 2 * sf_bytes(st));
      tma_load_2d(smem + slot * kWStage, &p.tmap_w, st * 128, wrow, &full[slot]);
      bulk_g2s(s_sf + slot * 2 * C::kSfBytes, wsf + st * C::kSfBytes, sf_bytes(st), &full[slot]);
    };
    auto copy_a = [&](int slot, int st) {
      tma_load_2d(s_a + slot * C::kAStage, &p.tmap_a, st * 128, first, &full[slot]);
      if (boxes > 1) tma_load_2d(s_a + slot * C::kAStage + kBox * 128, &p.tmap_a, st * 128, first + kBox, &full[slot]);
      bulk_g2s(s_sf + slot * 2 * C::kSfBytes + C::kSfBytes, asf + st * C::kSfBytes, sf_bytes(st), &full[slot]);
    };
    if (early > 0) {
      load_unit();
      if (elect_one())
        for (int i = 0; i < early; ++i) copy_w(i, s_beg + i);
      pdl_wait();
    }
    uint32_t issued = 0;
    while (ok) {
#pragma unroll kUnroll
      for (int slot = 0; slot < NS; ++slot) {
        if (s == s_beg) load_unit();
        ok = __all_sync(0xffffffffu, wait(&empty[slot], phase, ab, 101));
        if (!ok) break;
        if (elect_one()) {
          if (early <= 0) copy_w(slot, s);
          copy_a(slot, s);
        }
        __syncwarp();
        --early;
        ++issued;
        if (++s == s_end) {
          s = s_beg;
          u += du;
          ok = u < n_units;
          if (!ok) break;
        }
      }
      phase ^= 1;
    }
    if (ab.raised() && lane == 0) {
      // let copies already issued land before the CTA's shared memory goes away
      const uint32_t n = issued < (uint32_t)NS ? issued : (uint32_t)NS;
      for (uint32_t i = issued - n; i < issued; ++i) {
        const unsigned long long t0 = globaltimer();
        while (!mbar_try_wait(&full[i % NS], (i / NS) & 1) && globaltimer() - t0 < kWaitLimitNs) {
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------- matrix instructions
    const uint32_t w_desc = desc_lo(smem_u32(smem)), a_desc = desc_lo(smem_u32(s_a)), s_desc = desc_lo(smem_u32(s_sf));
    uint32_t phase = 0, acc_i = 0;
    int u = u0, s = s_beg;
    uint32_t idesc = 0, d = 0, shift = 0;
    bool ok = u < n_units;
    bool seen = false;  // the stage's copies were seen complete during the stage before
    while (ok) {
#pragma unroll kUnroll
      for (int slot = 0; slot < NS; ++slot) {
        if (s == s_beg) {
          const Unit U = get_unit<kRows, RAGGED>(p, groups, wtiles, u);
          idesc = idesc_fp4(FMT, 128, (uint32_t)round_up((int)warp_uniform(U.rows), 16));
          shift = warp_uniform(U.shift);
          d = (acc_i & 1) * kRows;
          ok = __all_sync(0xffffffffu, wait(&empty_acc[acc_i & 1], ((acc_i >> 1) & 1) ^ 1, ab, 102));
          if (!ok) break;
        }
        if (!seen) {
          ok = __all_sync(0xffffffffu, wait(&full[slot], phase, ab, 104));
          if (!ok) break;
        }
        tc_fence_after();
        // the next stage's barrier, looked at while this stage's instructions issue
        const bool look = mbar_test(&full[(slot + 1) % NS], slot + 1 == NS ? phase ^ 1 : phase);
        const int kts = min(C::kSfTiles, k_tiles - s * C::kSfTiles);
        const int kn = min(4, k64 - 4 * s);
        const bool last = s + 1 == s_end;
        if (elect_one()) {
          constexpr uint32_t kStep = kSfTile / 16;
          const uint32_t sfw = 2 * kRows + slot * C::kSfCols, sfa = sfw + 4 * C::kSfTiles;
          const uint32_t sd = s_desc + slot * (2 * C::kSfBytes / 16);
          const uint32_t wd = w_desc + slot * (kWStage / 16), ad = a_desc + slot * (C::kAStage / 16);
#pragma unroll
          for (int i = 0; i < C::kSfTiles; ++i)
            if (i < kts) {
              copy_scales<1>(sfw + 4 * i, sd + i * kStep);
              copy_scales<1>(sfa + 4 * i, sd + C::kSfBytes / 16 + i * kStep);
            }
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i < kn) {
              const int t = FMT == 0 ? i : i >> 1;  // MXFP4: a scale tile serves two instructions
              const uint32_t sf = FMT == 0 ? 0 : 2 * (i & 1);
              mma_fp4<FMT, 1>(d, wd + 2 * i, ad + 2 * i, idesc | sf << 4 | sf << 29, sfw + 4 * t, sfa + 4 * t + shift,
                              i > 0 || s > s_beg);
            }
          mma_commit(&empty[slot]);
          if (last) mma_commit(&full_acc[acc_i & 1]);
        }
        seen = __all_sync(0xffffffffu, look);
        ++s;
        if (last) {
          s = s_beg;
          ++acc_i;
          u += du;
          ok = u < n_units;
          if (!ok) break;
        }
      }
      phase ^= 1;
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
    if (rank == 0)
      fill_rows<kRows, RAGGED>(p, groups, tab, full_rows, empty_rows, wtiles, u0, du, n_units, ab);
    if (RAGGED && !p.out_rows) clear_tail(p, groups.first[p.groups], threadIdx.x - 64);
  } else {
    // --------------------------------------------------------- epilogue
    if (p.a_is_new) pdl_wait();
    const int q4 = warp & 3;
    const int turn = (warp - 4) >> 2;
    uint8_t* stage = smem + C::epi + (warp - 4) * 32 * kEpiRow;
    if constexpr (SPLIT) {
      if (u0 < n_units) {
        const int rows = get_unit<kRows, RAGGED>(p, groups, wtiles, u0).rows;
        const int parts = cdiv(rows, 16);
        const bool mine = 2 * turn < parts;
        // a CTA's partial sums: [16 rows][quarter][4 x 4 values][lane]
        float4* part = reinterpret_cast<float4*>(smem + C::part) + (2 * turn * 4 + q4) * 128 + lane;
        const size_t pitch = (size_t)parts * (kPart16 / 16);
        if (rank == 0 && warp == 4 && lane == 0)
          mbar_arrive_expect_tx(part_bar, (uint32_t)(splits - 1) * parts * kPart16);
        bool ok = wait(&full_acc[0], 0, ab, 105);
        if (__all_sync(0xffffffffu, ok) && mine) {
          tc_fence_after();
          uint32_t lo[16], hi[16];
          const uint32_t taddr = tmem + ((uint32_t)(32 * q4) << 16) + 32 * turn;
          tmem_ld16x256b_x4(taddr, lo);
          tmem_ld16x256b_x4(taddr + (16u << 16), hi);
          tmem_ld_wait();
          if (rank > 0) {
            const uint32_t dst = map_rank(part + (rank - 1) * pitch, 0);
            const uint32_t bar = map_rank(part_bar, 0);
#pragma unroll
            for (int h = 0; h < 2; ++h)
              if (2 * turn + h < parts) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  const uint32_t* l = &lo[8 * h + 4 * i];
                  const uint32_t* g = &hi[8 * h + 4 * i];
                  store_async4(dst + 8192 * h + 1024 * i, l[0], l[1], l[2], l[3], bar);
                  store_async4(dst + 8192 * h + 1024 * i + 512, g[0], g[1], g[2], g[3], bar);
                }
              }
          } else {
            ok = wait(&full_rows[0], 0, ab, 107) && wait_cluster(part_bar, 0, ab, 108);
            if (__all_sync(0xffffffffu, ok)) {
              for (int r = 0; r + 1 < splits; ++r) {
                const float4* from = part + r * pitch;
#pragma unroll
                for (int h = 0; h < 2; ++h)
                  if (2 * turn + h < parts) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                      add4(&lo[8 * h + 4 * i], from[512 * h + 64 * i]);
                      add4(&hi[8 * h + 4 * i], from[512 * h + 64 * i + 32]);
                    }
                  }
              }
              const int n0 = tab.wtile[0] * 128 + 32 * q4;
              const int at = 32 * turn + lane;
              const RowInfo info{tab.g[0][at], tab.to[0][at]};
              if (n0 < p.n) store_chunk<OUT>(p, lo, hi, info, n0, stage, lane);
            }
          }
        }
      }
    } else {
      uint32_t i = 0;
      for (int u = u0; u < n_units; u += du, ++i) {
        const uint32_t b = i & 1;
        bool ok = wait(&full_rows[b], (i >> 1) & 1, ab, 107);
        ok = ok && wait(&full_acc[b], (i >> 1) & 1, ab, 105);
        if (!__all_sync(0xffffffffu, ok)) break;
        const int rows = tab.rows[b];
        const int n0 = tab.wtile[b] * 128 + 32 * q4;
        tc_fence_after();
        const uint32_t taddr = tmem + ((uint32_t)(32 * q4) << 16) + b * kRows + 32 * turn;
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
  }

  tc_fence_before();
  if constexpr (SPLIT) cluster_sync();  // the first CTA's shared memory outlives the others' stores
  else __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

template <int FMT, int OUT, bool RAGGED, bool SPLIT>
cudaError_t launch(const Fp4GemmParams& p, int grid, int splits, bool pdl, cudaStream_t stream) {
  auto kern = fp4_gemm_kernel<FMT, OUT, RAGGED, SPLIT>;
  const size_t smem = Cfg<FMT, SPLIT>::total(RAGGED);
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid * splits);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (SPLIT) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = splits;
    attr[n].val.clusterDim.y = 1;
    attr[n++].val.clusterDim.z = 1;
  }
  if (pdl) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace fp4

// grid: CTAs (splits == 1) or clusters, one for each unit the call can have.
cudaError_t launch_fp4_gemm(const Fp4GemmParams& p, int fmt, int grid, int splits, bool pdl, cudaStream_t stream) {
  return fp4::with_forms(p, fmt, [&](auto f, auto out, auto ragged) {
    return splits > 1 ? fp4::launch<f.value, out.value, ragged.value, true>(p, grid, splits, pdl, stream)
                      : fp4::launch<f.value, out.value, ragged.value, false>(p, grid, 1, pdl, stream);
  });
}

}  // namespace b4
