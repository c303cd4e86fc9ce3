// Product of two FP8 operands with scales per block of 128 along K on pairs of SMs
// (tcgen05 cta_group::2): the form for many rows.  The formula is that of fp8_gemm.cu.
//
// A pair takes units of 256 activation rows x 256 weight rows: each CTA holds its own 128
// activation rows and half of the weight rows (32 KB a stage of 128 K, for 512 cycles of
// products), and accumulates its 128 rows x 256 outputs in its own tensor memory.  A stage is
// one block of K.  It has two accumulators of 128 columns, one for each block of 128 weight
// rows, twice: while the tensor core fills one of each pair, four warps read the other,
// 32 lanes x 128 columns each, and add it to fp32 registers times the row's scale and the
// weights'.
// The 128 registers a thread holds its sums in come from the other warps (setmaxnreg).

#include "fp8_mma.cuh"

namespace b4 {

cudaError_t ensure_smem_limit(const void* func, size_t bytes);

namespace fp8 {

constexpr int kPairRows = 256;
constexpr int kPairSlots = 6;
constexpr int kPairBox = 64;                    // activation rows of a box
constexpr int kPairAStage = 128 * 128;
constexpr size_t kPairOffA = (size_t)kPairSlots * kWStage;
constexpr size_t kPairOffBars = kPairOffA + (size_t)kPairSlots * kPairAStage;
constexpr int kAhead = 4;                       // units looked up ahead of the promoting warps
constexpr int kPairBars = 2 * kPairSlots + 8 + 1 + 2 * kAhead;
constexpr size_t kPairOffUnits = kPairOffBars + 8 * (kPairBars + 1);
constexpr int kScaleDepth = 4;                  // stages of scales
constexpr size_t kPairOffScales = kPairOffUnits + 16 * kAhead;
constexpr size_t kPairOffMisc = kPairOffScales + kScaleDepth * 2 * 128 * sizeof(float);
constexpr size_t pair_smem(bool ragged) { return kPairOffMisc + 16 + (ragged ? sizeof(Groups) : 0); }

// Registers of a thread after the split: 128 x 136 + 256 x 184 = 384 x 168, what the block is launched with.
constexpr int kRegsLaunch = 168, kRegsIssue = 136, kRegsPromote = 184;
static_assert(128 * kRegsIssue + 256 * kRegsPromote <= kThreads * kRegsLaunch, "the split fits the launch's registers");

// A wait that is a link of the chain between products and promotion: looked at without
// pause first (a suspended thread wakes late).
__device__ __forceinline__ bool wait_spin(uint64_t* bar, uint32_t parity, const Abort& ab, uint32_t where) {
#pragma unroll 1
  for (int i = 0; i < 256; ++i)
    if (__all_sync(0xffffffffu, mbar_test(bar, parity))) return true;
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, ab, where));
}

template <int OUT, bool RAGGED>
__global__ void __launch_bounds__(kThreads, 1) fp8_pair_kernel(const __grid_constant__ Fp8GemmParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Groups& groups = *reinterpret_cast<Groups*>(smem + kPairOffMisc + 16);  // ragged only
  uint8_t* s_a = smem + kPairOffA;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kPairOffBars);  // the leader's: copies of both CTAs
  uint64_t* empty = full + kPairSlots;                                // each CTA's own
  uint64_t* full_acc = empty + kPairSlots;                            // each CTA's own
  uint64_t* empty_acc = full_acc + 4;                                 // the leader's: promoting warps of both
  uint64_t* drain = empty_acc + 4;
  uint64_t* full_unit = drain + 1;                                    // each CTA's own
  uint64_t* empty_unit = full_unit + kAhead;
  int4* s_unit = reinterpret_cast<int4*>(smem + kPairOffUnits);       // group, weight unit, first row, rows
  float* s_scale = reinterpret_cast<float*>(smem + kPairOffScales);   // [stage][block of weights][row]
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + kPairOffMisc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + kPairOffMisc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const Fp4GemmParams& g = p.g;
  const Abort ab{g.status, s_abort};

  if (threadIdx.x == 0) {
    *s_abort = 0;
    for (int i = 0; i < kPairSlots; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(drain, 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&full_acc[i], 3);              // the products and two warps' scales
      mbar_init(&empty_acc[i], kEpiWarps);  // four warps of each CTA
    }
    for (int i = 0; i < kAhead; ++i) {
      mbar_init(&full_unit[i], 1);
      mbar_init(&empty_unit[i], kEpiWarps);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(s_tmem, 512);
    tmem_relinquish_pair();
  }
  if (!g.a_is_new) pdl_wait();  // alone in its call: every input may come from the kernel before
  const int wpairs = cdiv(g.n, 256);
  const int wtiles = cdiv(g.n, 128);
  if (RAGGED) build_groups<kPairRows>(g, groups);
  tc_fence_before();
  cluster_sync();  // both CTAs' barriers exist before either signals
  tc_fence_after();
  if (threadIdx.x == 0) pdl_launch_dependents();
  const uint32_t tmem = *s_tmem;
  const int n_units = (RAGGED ? groups.tiles[g.groups] : g.groups * cdiv(g.m, kPairRows)) * wpairs;
  const int u0 = blockIdx.x >> 1, du = gridDim.x >> 1;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    if (warp == 0) {
      // --------------------------------------------------------- copies
      if (g.a_is_new) pdl_wait();
      uint32_t i = 0;
      bool ok = true;
      const uint32_t full0 = warp_uniform(map_rank(full, 0));
      for (int u = u0; u < n_units && ok; u += du) {
        const Unit U = get_unit<kPairRows, RAGGED>(g, groups, wpairs, u);
        const int rows = (int)warp_uniform(U.rows);
        const int first = (int)warp_uniform(U.first) + 128 * (int)rank;
        const int wrow = (int)warp_uniform(U.group) * g.n + (int)warp_uniform(U.wtile) * 256 + (int)rank * 64;
        const int boxes = cdiv(min(max(rows - 128 * (int)rank, 0), 128), kPairBox);
        const int all_boxes = cdiv(min(rows, 128), kPairBox) + cdiv(max(rows - 128, 0), kPairBox);
        const uint32_t bytes = 2 * kWStage + all_boxes * kPairBox * 128;
        for (int s = 0; s < p.kb; ++s, ++i) {
          const uint32_t slot = i % kPairSlots;
          ok = __all_sync(0xffffffffu, mbar_wait(&empty[slot], ((i / kPairSlots) & 1) ^ 1, ab, 131));
          if (!ok) break;
          const uint32_t bar = full0 + 8 * slot;
          if (elect_one()) {
            if (rank == 0) mbar_arrive_expect_tx(&full[slot], bytes);
            // of each block of 128 weight rows, which is N of one accumulator, a CTA holds half
            tma_load_2d_pair(smem + slot * kWStage, &p.tmap_w, s * 128, wrow, bar);
            tma_load_2d_pair(smem + slot * kWStage + kWStage / 2, &p.tmap_w, s * 128, wrow + 128, bar);
            if (boxes > 0) tma_load_2d_pair(s_a + slot * kPairAStage, &p.tmap_a, s * 128, first, bar);
            if (boxes > 1)
              tma_load_2d_pair(s_a + slot * kPairAStage + kPairBox * 128, &p.tmap_a, s * 128, first + kPairBox, bar);
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
      // -------------------------------------------- matrix instructions
      if (rank == 0) {
        const uint32_t w_desc = desc_lo(smem_u32(smem)), a_desc = desc_lo(smem_u32(s_a));
        constexpr uint32_t idesc = idesc_fp8(256, 128);
        // Every unit has kb stages, so units do not show here.  The loop is unrolled over the ring, so
        // that slots and accumulators are constants, and each barrier is looked at while the
        // instructions before those that wait for it issue: otherwise a stage takes longer to
        // issue (1300 cycles) than its products to run.
        int left = u0 < n_units ? ((n_units - 1 - u0) / du + 1) * p.kb : 0;
        uint32_t phase = 0, acc_phase = 1;
        bool ok = left > 0, full_seen = false, acc_seen = false;
        while (ok) {
#pragma unroll
          for (int slot = 0; slot < kPairSlots; ++slot) {
            constexpr int kHalf = kWStage / 32;
            const uint32_t wd = w_desc + slot * (kWStage / 16), ad = a_desc + slot * (kPairAStage / 16);
            const int acc = 2 * (slot & 1), next = (slot + 1) % kPairSlots;
            if (!full_seen) ok = wait_spin(&full[slot], phase, ab, 133);
            if (!acc_seen) ok = ok && wait_spin(&empty_acc[acc], acc_phase, ab, 132);
            if (!ok) break;
            tc_fence_after();
            const bool look1 = mbar_test(&empty_acc[acc + 1], acc_phase);
            if (elect_one()) {
#pragma unroll
              for (int j = 0; j < 4; ++j) mma_fp8<2>(acc * 128, ad + 2 * j, wd + 2 * j, idesc, j > 0);
              mma_commit_pair(&full_acc[acc]);
            }
            if (!__all_sync(0xffffffffu, look1)) {
              ok = wait_spin(&empty_acc[acc + 1], acc_phase, ab, 132);
              if (!ok) break;
            }
            tc_fence_after();
            if (slot & 1) acc_phase ^= 1;
            const bool look_full = mbar_test(&full[next], next == 0 ? phase ^ 1 : phase);
            const bool look_acc = mbar_test(&empty_acc[2 * (next & 1)], acc_phase);
            if (elect_one()) {
#pragma unroll
              for (int j = 0; j < 4; ++j) mma_fp8<2>((acc + 1) * 128, ad + 2 * j, wd + kHalf + 2 * j, idesc, j > 0);
              mma_commit_pair(&full_acc[acc + 1]);
              mma_commit_pair(&empty[slot]);
            }
            full_seen = __all_sync(0xffffffffu, look_full);
            acc_seen = __all_sync(0xffffffffu, look_acc);
            if (--left == 0) {
              ok = false;
              break;
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
    } else {
      // --- units and scales for the promoting warps, ahead of them (their registers are all taken, and
      // what they look up themselves holds up their sums); rows past the last group are zero
      if (g.a_is_new) pdl_wait();
      const int j = threadIdx.x - 64;
      uint32_t i = 0, n = 0;
      bool ok = true;
      for (int u = u0; u < n_units && ok; u += du, ++n) {
        const Unit U = get_unit<kPairRows, RAGGED>(g, groups, wpairs, u);
        const uint32_t b = n % kAhead;
        if (warp == 2) {
          ok = __all_sync(0xffffffffu, mbar_wait(&empty_unit[b], ((n / kAhead) & 1) ^ 1, ab, 135));
          if (!ok) break;
          if (lane == 0) {
            s_unit[b] = make_int4(U.group, U.wtile, U.first, U.rows);
            mbar_arrive(&full_unit[b]);
          }
          __syncwarp();
        }
        const int r0 = 128 * (int)rank + j, r1 = r0 + 64;
        const float* sa0 = p.a_scales + (int64_t)(U.first + min(r0, U.rows - 1)) * p.kb;
        const float* sa1 = p.a_scales + (int64_t)(U.first + min(r1, U.rows - 1)) * p.kb;
        const float* sw0 = p.w_scales + ((int64_t)U.group * wtiles + 2 * U.wtile) * p.kb;
        const float* sw1 = 2 * U.wtile + 1 < wtiles ? sw0 + p.kb : sw0;
        float4 now0 = load_scales(p, sa0, 0, true), now1 = load_scales(p, sa1, 0, true);
        float4 next0 = now0, next1 = now1;
        float w0 = 0.f, w1 = 0.f;
        for (int s = 0; s < p.kb; ++s, ++i) {
          if ((s & 31) == 0 && s + lane < p.kb) w0 = __ldg(sw0 + s + lane), w1 = __ldg(sw1 + s + lane);
          if ((s & 3) == 0) {
            if (s > 0) now0 = next0, now1 = next1;
            next0 = load_scales(p, sa0, s + 4, true), next1 = load_scales(p, sa1, s + 4, true);
          }
          const float a0 = (s & 3) == 0 ? now0.x : (s & 3) == 1 ? now0.y : (s & 3) == 2 ? now0.z : now0.w;
          const float a1 = (s & 3) == 0 ? now1.x : (s & 3) == 1 ? now1.y : (s & 3) == 2 ? now1.z : now1.w;
          const float v0 = __shfl_sync(0xffffffffu, w0, s & 31), v1 = __shfl_sync(0xffffffffu, w1, s & 31);
          // The stage before the last on these barriers is complete: so its products were issued,
          // after the promoters had let go of the stage two further back, whose scales lie where
          // this stage's go.
          if (i >= 2) {
            ok = __all_sync(0xffffffffu, mbar_wait(&full_acc[2 * (i & 1)], ((i >> 1) & 1) ^ 1, ab, 137) &&
                                             mbar_wait(&full_acc[2 * (i & 1) + 1], ((i >> 1) & 1) ^ 1, ab, 137));
            if (!ok) break;
          }
          float* to = s_scale + (i % kScaleDepth) * 256 + j;
          to[0] = a0 * v0;
          to[64] = a1 * v0;
          to[128] = a0 * v1;
          to[192] = a1 * v1;
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&full_acc[2 * (i & 1)]);
            mbar_arrive(&full_acc[2 * (i & 1) + 1]);
          }
        }
      }
      if (RAGGED && !g.out_rows) clear_tail(g, groups.first[g.groups], threadIdx.x - 64);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsPromote));
    // ------------------------------------------- promotion and epilogue
    if (g.a_is_new) pdl_wait();  // (the output's last readers)
    const int q4 = warp & 3, half = (warp - 4) >> 2;
    const int r = 128 * (int)rank + 32 * q4 + lane;
    const uint32_t taddr = tmem + ((uint32_t)(32 * q4) << 16) + 128 * half;
    uint64_t* mine_acc = full_acc + half;  // this warp's two accumulators: 2 apart
    const uint32_t done = map_rank(empty_acc + half, 0);
    const float* scales = s_scale + 128 * half + 32 * q4 + lane;
    uint32_t i = 0, n = 0;
    bool ok = true;
    for (int u = u0; u < n_units && ok; u += du, ++n) {
      ok = __all_sync(0xffffffffu, mbar_wait(&full_unit[n % kAhead], (n / kAhead) & 1, ab, 136));
      if (!ok) break;
      const int4 U = s_unit[n % kAhead];  // group, weight unit, first row, rows
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty_unit[n % kAhead]);
      const int col = U.y * 256 + 128 * half;
      if (r - lane >= U.w || col >= g.n) {  // nothing of this warp's
        for (int s = 0; s < p.kb && ok; ++s, ++i) {
          ok = __all_sync(0xffffffffu, mbar_wait(&mine_acc[2 * (i & 1)], (i >> 1) & 1, ab, 134));
          if (ok && lane == 0) mbar_arrive_cluster(done + 16 * (i & 1));
        }
        continue;
      }
      const bool live = r < U.w;
      float2 acc[64];
#pragma unroll
      for (int c = 0; c < 64; ++c) acc[c] = make_float2(0.f, 0.f);
      bool seen = false;  // the block's accumulator was seen complete during the block before
      // (one way out of the loop: with a second the compiler copies the sums every time round; once a
      // wait has run out, the others return at once and nothing is stored)
      for (int s = 0; s < p.kb; ++s, ++i) {
        if (!seen) ok = wait_spin(&mine_acc[2 * (i & 1)], (i >> 1) & 1, ab, 134) && ok;
        tc_fence_after();
        const uint32_t at = taddr + 256 * (i & 1);
        const float scale = scales[(i % kScaleDepth) * 256];
        bool look = false;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t t[32];
          tmem_ld32(at + 32 * c, t);
          tmem_ld_wait();
          if (c == 3) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(done + 16 * (i & 1));
            look = mbar_test(&mine_acc[2 * (~i & 1)], ((i + 1) >> 1) & 1);
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) fma2(acc[16 * c + e], t[2 * e], t[2 * e + 1], scale);
        }
        seen = __all_sync(0xffffffffu, look);
      }
      if (!ok || !live) continue;
      int to = U.z + r;
      if (g.out_rows) to = __ldg(g.out_rows + to);
      if (to >= 0 && to < g.out_rows_end) store_row<OUT>(g, (int64_t)to * g.out_stride, col, acc);
    }
  }

  tc_fence_before();
  cluster_sync();  // neither CTA leaves while the pair's copies, products or signals may touch it
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

template <int OUT, bool RAGGED>
cudaError_t launch_pair(const Fp8GemmParams& p, int pairs, cudaStream_t stream) {
  auto kern = fp8_pair_kernel<OUT, RAGGED>;
  const size_t smem = pair_smem(RAGGED);
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
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace fp8

cudaError_t launch_fp8_gemm_pair(const Fp8GemmParams& p, int pairs, cudaStream_t stream) {
  return fp8::with_out(p, [&](auto out, auto ragged) { return fp8::launch_pair<out.value, ragged.value>(p, pairs, stream); });
}

}  // namespace b4
