// Product of two FP8 operands with scales per block of 128 along K on pairs of SMs: the
// form for many rows.  The formula is that of fp8_gemm.cuh.
//
// A pair takes units of 256 activation rows x 256 weight rows, each CTA 128 of the activation
// rows and all of the weight rows, which it loads for itself: 48 KB a stage of 128 K, for 512
// cycles of products (copies alone take 756 cycles a stage on all SMs, less than the chain
// below).  The rows that are left of a group, 128 or fewer, make wide units: both CTAs take
// them, each with 256 weight rows of its own.  The two share no memory; they are a cluster so
// that they run side by side and meet each other's weights in L2 (layer of E64 H2048 I1408, 2048
// tokens 190.6 us, 193 as CTAs by themselves; dense products the same).
//
// H: the product is the first of a layer (b4_fused_moe_fp8).  A unit's sums become h, 128
// columns of a gated activation (its weight rows are 128 gate rows and the 128 up rows that go
// with them, 64 of each in an accumulator, so that a lane holds both of a column) or 256 of
// ReLU^2, and h leaves quantised, codes and scales as b4_fp8_quantize writes them: it never
// goes to memory in 32 bits.
//
// A stage is one block of K.  It has two accumulators of 128 columns, one for each block of 128
// weight rows, twice: while the tensor core fills one of each pair, four warps read the other,
// 32 lanes x 128 columns each, and add it to fp32 registers times the row's scale and the
// weights'.  Tensor memory, 512 columns, is renewed by a chain of steps: 256 cycles of
// products, 270 until a waiting warp has seen them done, 500 of promotion (of which 350 are
// the loads and multiply-adds of two warps a scheduler), 200 until the next products issue.
// That chain, 760 to 830 cycles a stage, bounds the kernel, not the 512 cycles of products.
// Scales come through shared memory from warps of their own, and two warps share the
// products' issue: what these looked up or issued for themselves held up the chain.
//
// What else counts.  4096 rows of N = K = 4096: outputs stored by the warps from registers
// 70.6 us, through shared memory 67.4, as TMA boxes 65.8; the copying warp's loop with
// decisions in it 72.3, without 65.8.  64 groups of 192 rows, N = 2816, K = 2048: scales of a
// unit looked up at its start 112, under the last stages of the one before 106; three stages
// in the ring 104.4, four where no boxes are staged 103.3; weights asked into L2 ahead of their
// copies 103, not 99.5.
//
// Measured: N = K = 4096, 4096 rows 63 us (2.2 PFLOP/s), 8192 x 8192 x 4096 215 us (2.6
// PFLOP/s); 64 groups of 192 rows, N = 2816, K = 2048 99.5 us.

#include "fp8_mma.cuh"
#include "fp8_quant.cuh"

namespace b4 {

cudaError_t ensure_smem_limit(const void* func, size_t bytes);

namespace fp8 {

constexpr int kPairRows = 256;
constexpr int kPairBox = 64;                    // activation rows of a box
constexpr int kPairAStage = 128 * 128;
constexpr int kPairWStage = 2 * kWStage;        // both blocks of weight rows
constexpr int kOutTile = 2 * 32 * 128;          // staged outputs of a warp: 32 rows of two times 64, 128-byte swizzle
constexpr int kAhead = 4;                       // units looked up ahead of the promoting warps
constexpr int kScaleQuad = 130 * 4;             // scales of four stages: 128 rows, two blocks of weights; two of these

// BOXES: outputs leave as boxes from 64 KB of staging, which costs the ring a fourth stage.
template <bool BOXES>
struct PairCfg {
  static constexpr int kSlots = BOXES ? 3 : 4;
  static constexpr int kBars = 2 * kSlots + 8 + 1 + 2 * kAhead + 4 + 4;
  static constexpr size_t a = (size_t)kSlots * kPairWStage;
  static constexpr size_t stage = a + (size_t)kSlots * kPairAStage;
  static constexpr size_t bars = stage + kEpiWarps * (BOXES ? kOutTile : kStagePiece);
  static constexpr size_t units = (bars + 8 * kBars + 15) / 16 * 16;
  static constexpr size_t scales = units + 16 * kAhead;
  static constexpr size_t misc = scales + 2 * kScaleQuad * sizeof(float);
  static constexpr size_t total(bool ragged) {
    return misc + 16 + (ragged ? 2 * sizeof(int) * (kMaxGroups + 1) + sizeof(int) * kThreads / 32 : 0);
  }
};

enum PairH : int { kPlain = 0, kGated = 1, kRelu2 = 2 };

// Tables of the groups in shared memory: first row, and units before the group.
struct PairGroups {
  int first[kMaxGroups + 1];
  int units[kMaxGroups + 1];
  int warp[kThreads / 32];
};
// Units of a group of `rows` rows, where all its weights are wp blocks of 256: tall ones, then wide.
__device__ __forceinline__ int units_of(int rows, int wp) {
  const int rest = rows % kPairRows;
  return (rows / kPairRows + (rest > 128)) * wp + (rest > 0 && rest <= 128 ? (wp + 1) / 2 : 0);
}

// A block scan of the groups' units, four groups a thread; ends with the tables written but
// not yet synchronised.
__device__ __forceinline__ void build_pair_groups(const Fp4GemmParams& p, PairGroups& g, int wp) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int cnt[4], sum = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = 4 * threadIdx.x + i;
    cnt[i] = 0;
    if (e <= p.groups) {
      const int lo = min(max(__ldg(p.offsets + e), 0), p.m);
      g.first[e] = lo;
      if (e < p.groups) cnt[i] = units_of(max(min(__ldg(p.offsets + e + 1), p.m) - lo, 0), wp);
    }
    sum += cnt[i];
  }
  int scan = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += v;
  }
  if (lane == 31) g.warp[warp] = scan;
  __syncthreads();
  int before = scan - sum;
  for (int w = 0; w < warp; ++w) before += g.warp[w];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = 4 * threadIdx.x + i;
    if (e <= p.groups) g.units[e] = before;
    before += cnt[i];
  }
}

// A CTA's part of unit u: its group, block of 256 weight rows, first row and rows (128 at most).  Weight
// blocks are outermost within a group, so that neighbouring units read the same weights.
// Ragged units are taken from each third of them in turn: those of large groups are bound by the
// chain of promotion, those of small groups by the stream of weights, and the two mix better than they
// follow one another.
struct PairUnit {
  int group, wt, first, rows;
  bool wide;
};
template <bool RAGGED>
__device__ __noinline__ static int4 find_pair_unit(int groups, int m, const PairGroups* g, int wp, int u, int rank) {
  int e = 0, first, rows;
  if constexpr (RAGGED) {
    const int run = g->units[groups] / kMix;
    if (u < run * kMix) u = u % kMix * run + u / kMix;
    int hi = groups - 1;  // last group whose units start at or before this one
    while (e < hi) {
      const int mid = (e + hi + 1) >> 1;
      if (g->units[mid] <= u) e = mid;
      else hi = mid - 1;
    }
    u -= g->units[e];
    first = g->first[e];
    rows = g->first[e + 1] - first;
  } else {
    const int per = units_of(m, wp);
    e = groups == 1 ? 0 : u / per;
    u -= e * per;
    first = e * m;
    rows = m;
  }
  const int rest = rows % kPairRows, tall = rows / kPairRows + (rest > 128);
  int wt, mine, wide = 0;
  if (u < tall * wp) {
    wt = tall == 1 ? u : u / tall;
    const int t = u - wt * tall;
    first += t * kPairRows + 128 * rank;
    mine = min(max(rows - t * kPairRows - 128 * rank, 0), 128);
  } else {
    wide = 1;
    wt = 2 * (u - tall * wp) + rank;
    first += tall * kPairRows;
    mine = wt < wp ? rest : 0;
  }
  return make_int4(e, wt, first, mine | wide << 16);
}
template <bool RAGGED>
__device__ __forceinline__ PairUnit pair_unit(const Fp4GemmParams& p, const PairGroups& g, int wp, int u, int rank) {
  const int4 v = find_pair_unit<RAGGED>(p.groups, p.m, &g, wp, u, rank);
  return PairUnit{v.x, v.y, v.z, v.w & 0xffff, v.w >> 16 != 0};
}

// Two columns of h, as the quantiser's prologue forms them (fp4_quant.cuh).
__device__ __forceinline__ float2 gated2(float2 a, float2 b, const GluParams& p) {
  using namespace fp4q;
  const float scale = -1.44269504f * p.alpha;
  const float gx = min_nan(a.x, p.limit), gy = min_nan(a.y, p.limit);
  const float ux = max_nan(min_nan(b.x, p.limit), -p.limit), uy = max_nan(min_nan(b.y, p.limit), -p.limit);
  return make_float2(gx * rcp_approx(exp2_approx(gx * scale) + 1.f) * (ux + p.beta),
                     gy * rcp_approx(exp2_approx(gy * scale) + 1.f) * (uy + p.beta));
}

// Sixteen values in registers as a chunk of the quantiser.
struct Sixteen {
  const float2* v;
  __device__ __forceinline__ float2 pair(int j) const { return v[j]; }
};

// OUT: 0 bf16, 1 f16, 2 f32 outputs; H: kPlain, or h as the next product's operand.
template <int OUT, bool RAGGED, int H, bool BOXES>
__global__ void __launch_bounds__(kThreads, 1) fp8_pair_kernel(const __grid_constant__ Fp8GemmParams p) {
  using C = PairCfg<BOXES>;
  constexpr int kPairSlots = C::kSlots;
  extern __shared__ __align__(1024) uint8_t smem[];
  PairGroups& groups = *reinterpret_cast<PairGroups*>(smem + C::misc + 16);  // ragged only
  uint8_t* s_a = smem + C::a;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::bars);
  uint64_t* empty = full + kPairSlots;                                // the products are through with the slot
  uint64_t* full_acc = empty + kPairSlots;
  uint64_t* empty_acc = full_acc + 4;
  uint64_t* drain = empty_acc + 4;
  uint64_t* full_unit = drain + 1;
  uint64_t* empty_unit = full_unit + kAhead;
  uint64_t* full_scale = empty_unit + kAhead;
  uint64_t* empty_scale = full_scale + 2;
  uint64_t* both_halves = empty_scale + 2;                            // gated: a quarter's two warps have their maxima
  int4* s_unit = reinterpret_cast<int4*>(smem + C::units);       // group, weight unit, first row, rows
  float* s_scale = reinterpret_cast<float*>(smem + C::scales);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + C::misc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + C::misc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = blockIdx.x & 1;
  const Fp4GemmParams& g = p.g;
  const Abort ab{g.status, s_abort};

  if (threadIdx.x == 0) {
    *s_abort = 0;
    for (int i = 0; i < kPairSlots; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(drain, 2);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&both_halves[i], 2);
      mbar_init(&full_acc[i], 1);
      mbar_init(&empty_acc[i], kEpiWarps / 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&full_scale[i], 1);
      mbar_init(&empty_scale[i], kEpiWarps);
    }
    for (int i = 0; i < kAhead; ++i) {
      mbar_init(&full_unit[i], 1);
      mbar_init(&empty_unit[i], kEpiWarps);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(s_tmem, 512);
    tmem_relinquish();
  }
  if (!g.a_is_new) pdl_wait();  // alone in its call: every input may come from the kernel before
  const int wp = cdiv(g.n, 256);  // blocks of 256 weight rows
  const int wtiles = cdiv(g.n, 128);
  if (RAGGED) build_pair_groups(g, groups, wp);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0) pdl_launch_dependents();
  const uint32_t tmem = *s_tmem;
  const int n_units = RAGGED ? groups.units[g.groups] : g.groups * units_of(g.m, wp);
  const int u0 = blockIdx.x >> 1, du = gridDim.x >> 1;

  if (warp < 4) {
    if (warp == 0) {
      // --------------------------------------------------------- copies
      // (None are asked into L2 ahead: what the SMs have in flight is enough for DRAM, and more is fetched twice.
      // 128 groups of 128 rows, N = 4096, K = 1536 173 us with ten stages ahead, 172 with one, 165 so; the layer of
      // E128 H4096 I1536, 2048 tokens 585, 543, 536.)
      uint32_t i = 0;
      bool ok = true;
      // A unit's boxes of weights in a stage: both blocks of 128 rows; gated, a block is 64 gate rows and their up rows.
      constexpr int kBox = H == kGated ? 64 : 128;
      if (g.a_is_new) pdl_wait();
      for (int u = u0; u < n_units && ok; u += du) {
        const PairUnit U = pair_unit<RAGGED>(g, groups, wp, u, rank);
        const bool none = U.wide && U.wt >= wp;
        const int row = (int)warp_uniform(U.group * g.n + U.wt * 2 * kBox);
        const int first = (int)warp_uniform(U.first), rows = (int)warp_uniform(U.rows);
        const uint32_t bytes = (none ? 0 : kPairWStage) + cdiv(rows, kPairBox) * kPairBox * 128;
        for (int s = 0; s < p.kb; ++s, ++i) {
          const uint32_t slot = i % kPairSlots;
          ok = __all_sync(0xffffffffu, wait(&empty[slot], ((i / kPairSlots) & 1) ^ 1, ab, 131));
          if (!ok) break;
          if (elect_one()) {
            mbar_arrive_expect_tx(&full[slot], bytes);
            uint8_t *sw = smem + slot * kPairWStage, *sa = s_a + slot * kPairAStage;
            if (!none) {
              tma_load_2d(sw, &p.tmap_w, s * 128, row, &full[slot]);
              tma_load_2d(sw + kWStage, &p.tmap_w, s * 128, row + kBox, &full[slot]);
              if (H == kGated) {
                tma_load_2d(sw + kWStage / 2, &p.tmap_w, s * 128, row + g.n / 2, &full[slot]);
                tma_load_2d(sw + kWStage * 3 / 2, &p.tmap_w, s * 128, row + g.n / 2 + kBox, &full[slot]);
              }
            }
            if (rows > 0) tma_load_2d(sa, &p.tmap_a, s * 128, first, &full[slot]);
            if (rows > kPairBox) tma_load_2d(sa + kPairBox * 128, &p.tmap_a, s * 128, first + kPairBox, &full[slot]);
          }
          __syncwarp();
        }
      }
      if (ab.raised() && lane == 0) {
        // copies already issued land before the shared memory goes away: give them a fixed time
        const unsigned long long t0 = globaltimer();
        while (globaltimer() - t0 < 2000000ull) {
        }
      }
      __syncwarp();
    } else if (warp & 1) {
      // -------------------------------------------- matrix instructions
      // Warp 1 issues the even stages, warp 3 the odd ones: between waits, votes and the fetching of
      // its code a warp takes some 800 cycles to issue a stage's eight, longer than they take to
      // run.  Every unit has kb stages, so units do not show here.
      const int w = warp >> 1;
      const uint32_t w_desc = desc_lo(smem_u32(smem)), a_desc = desc_lo(smem_u32(s_a));
      const uint32_t d = tmem + 256 * w;
      constexpr uint32_t idesc = idesc_fp8(128, 128);
      const int total = u0 < n_units ? ((n_units - 1 - u0) / du + 1) * p.kb : 0;
      uint32_t slot = w, phase = 0, acc_phase = 1;
      for (int i = w; i < total; i += 2) {
        // (the accumulator first: it is free once the stage before the last is promoted, and with it the
        // stage before has run, so that the slot's barrier is not two phases behind, where it would
        // look complete)
        if (!__all_sync(0xffffffffu, wait(&empty_acc[2 * w], acc_phase, ab, 132))) break;
        if (!__all_sync(0xffffffffu, wait(&full[slot], phase, ab, 133))) break;
        tc_fence_after();
        const bool look = mbar_test(&empty_acc[2 * w + 1], acc_phase);
        const uint32_t wd = w_desc + slot * (kPairWStage / 16), ad = a_desc + slot * (kPairAStage / 16);
        if (elect_one()) {
#pragma unroll
          for (int j = 0; j < 4; ++j) mma_fp8(d, ad + 2 * j, wd + 2 * j, idesc, j > 0);
          mma_commit(&full_acc[2 * w]);
        }
        if (!__all_sync(0xffffffffu, look) && !__all_sync(0xffffffffu, wait(&empty_acc[2 * w + 1], acc_phase, ab, 132))) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int j = 0; j < 4; ++j) mma_fp8(d + 128, ad + 2 * j, wd + kWStage / 16 + 2 * j, idesc, j > 0);
          mma_commit(&full_acc[2 * w + 1]);
          mma_commit(&empty[slot]);
        }
        __syncwarp();
        slot += 2;
        if (slot >= kPairSlots) slot -= kPairSlots, phase ^= 1;
        acc_phase ^= 1;
      }
      // drain: every instruction issued has completed
      if (elect_one()) mma_commit(drain);
      const unsigned long long t0 = globaltimer();
      while (!mbar_try_wait(drain, 0) && globaltimer() - t0 < kWaitLimitNs) {
      }
      __syncwarp();
    } else {
      // --- units and scales for the promoting warps, ahead of them (their registers are all taken, and
      // what they look up themselves holds up their sums); rows past the last group are zero
      if (g.a_is_new) pdl_wait();
      // Four stages of a unit at a time, looked up eight stages ahead of their turn, into the next
      // unit too: a load from L2 takes a microsecond and more under the operands' traffic.
      const float *sa[4], *sw;  // of rows lane, lane + 32, ..; lanes 0 and 1: of the accumulators' weight rows
      int lu = u0, ls = 0;      // looked up next
      uint32_t n = 0;
      bool ok = true;
      auto enter = [&]() {  // unit lu: told to the promoters, its scales found
        const PairUnit U = pair_unit<RAGGED>(g, groups, wp, lu, rank);
        const uint32_t b = n % kAhead;
        ok = ok && __all_sync(0xffffffffu, wait(&empty_unit[b], ((n / kAhead) & 1) ^ 1, ab, 135));
        if (ok && lane == 0) {
          s_unit[b] = make_int4(U.group, U.wt, U.first, U.rows);
          mbar_arrive(&full_unit[b]);
        }
        __syncwarp();
        ++n;
#pragma unroll
        for (int j = 0; j < 4; ++j)  // (a CTA without rows in the unit: any)
          sa[j] = p.a_scales + (int64_t)(U.rows > 0 ? U.first + min(32 * j + lane, U.rows - 1) : 0) * p.kb;
        // gated: the gate rows' and the up rows'
        const int t = H == kGated ? U.wt + (lane & 1) * (wtiles / 2) : 2 * U.wt + (lane & 1);
        sw = p.w_scales + ((int64_t)U.group * wtiles + min(t, wtiles - 1)) * p.kb;
      };
      float4 next[2][4], w[2];
      auto look_up = [&](int d) {
        if (lu >= n_units) return;
        if (ls == 0) enter();
        w[d] = load_scales(sw, ls, p.kb, p.w_vec);
#pragma unroll
        for (int j = 0; j < 4; ++j) next[d][j] = load_scales(sa[j], ls, p.kb, p.a_vec);
        ls += 4;
        if (ls >= p.kb) ls = 0, lu += du;
      };
      look_up(0);
      look_up(1);
      const int quads = u0 < n_units ? ((n_units - 1 - u0) / du + 1) * cdiv(p.kb, 4) : 0;
      for (int i = 0; i < quads && ok; i += 2) {
#pragma unroll
        for (int d = 0; d < 2; ++d)
          if (i + d < quads && ok) {
            ok = __all_sync(0xffffffffu, wait(&empty_scale[d], ((i >> 1) & 1) ^ 1, ab, 137));
            if (ok) {
              float4* to = reinterpret_cast<float4*>(s_scale + d * kScaleQuad) + lane;
#pragma unroll
              for (int j = 0; j < 4; ++j) to[32 * j] = next[d][j];
              if (lane < 2) to[128] = w[d];
              __syncwarp();
              if (lane == 0) mbar_arrive(&full_scale[d]);
              look_up(d);
            }
          }
      }
      if (H == kPlain && RAGGED && !g.out_rows) clear_tail<32>(g, groups.first[g.groups], lane);
    }
  } else {
    // ------------------------------------------- promotion and epilogue
    if (g.a_is_new) pdl_wait();  // (the output's last readers)
    const int q4 = warp & 3, half = (warp - 4) >> 2;
    const int r = 32 * q4 + lane;
    const uint32_t taddr = tmem + ((uint32_t)(32 * q4) << 16) + 128 * half;
    uint64_t* mine_acc = full_acc + half;  // this warp's two accumulators: 2 apart
    uint64_t* done = empty_acc + half;
    uint8_t* stage = smem + C::stage + (warp - 4) * (BOXES ? kOutTile : kStagePiece);
    const float4* scales = reinterpret_cast<const float4*>(s_scale);
    uint32_t i = 0, n = 0, quad = 0, done_units = 0;
    bool ok = true;
    for (int u = u0; u < n_units && ok; u += du, ++n) {
      ok = __all_sync(0xffffffffu,  wait(&full_unit[n % kAhead], (n / kAhead) & 1, ab, 136));
      if (!ok) break;
      const int4 U = s_unit[n % kAhead];  // group, block of weights, first row, rows
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty_unit[n % kAhead]);
      const int col = U.y * 256 + 128 * half;  // (of the sums)
      if (32 * q4 >= U.w || (H != kGated && col >= g.n)) {  // nothing of this warp's
        for (int s = 0; s < p.kb && ok; ++s, ++i) {
          if ((s & 3) == 0) {
            ok = __all_sync(0xffffffffu,  wait(&full_scale[quad & 1], (quad >> 1) & 1, ab, 138));
            if (ok && lane == 0) mbar_arrive(&empty_scale[quad & 1]);
            ++quad;
          }
          ok = ok && __all_sync(0xffffffffu,  wait(&mine_acc[2 * (i & 1)], (i >> 1) & 1, ab, 134));
          if (ok && lane == 0) mbar_arrive(&done[2 * (i & 1)]);
        }
        continue;
      }
      const int entry = output_entry(g, U.z + r, r < U.w);
      float2 acc[64];
#pragma unroll
      for (int c = 0; c < 64; ++c) acc[c] = make_float2(0.f, 0.f);
      bool seen = false;  // the block's accumulator was seen complete during the block before
      // (one way out of the loop: with a second the compiler copies the sums every time round; once a
      // wait has run out, the others return at once and nothing is stored)
      float4 four = make_float4(0.f, 0.f, 0.f, 0.f), up = four;
      for (int s = 0; s < p.kb; ++s, ++i) {
        if ((s & 3) == 0) {
          ok = __all_sync(0xffffffffu, wait(&full_scale[quad & 1], (quad >> 1) & 1, ab, 138)) && ok;
          four = scales[(quad & 1) * (kScaleQuad / 4) + r];
          const float4 w = scales[(quad & 1) * (kScaleQuad / 4) + 128 + (H == kGated ? 0 : half)];
          if constexpr (H == kGated) {
            const float4 v = scales[(quad & 1) * (kScaleQuad / 4) + 129];
            up = make_float4(four.x * v.x, four.y * v.y, four.z * v.z, four.w * v.w);
          }
          four = make_float4(four.x * w.x, four.y * w.y, four.z * w.z, four.w * w.w);
          __syncwarp();
          if (lane == 0) mbar_arrive(&empty_scale[quad & 1]);
          ++quad;
        }
        const float scale = four.x, scale_up = H == kGated ? up.x : scale;
        four = make_float4(four.y, four.z, four.w, 0.f);
        if constexpr (H == kGated) up = make_float4(up.y, up.z, up.w, 0.f);
        if (!seen) ok = __all_sync(0xffffffffu, wait(&mine_acc[2 * (i & 1)], (i >> 1) & 1, ab, 134)) && ok;
        tc_fence_after();
        const uint32_t at = taddr + 256 * (i & 1);
        bool look = false;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint32_t t[16];
          tmem_ld16(at + 16 * c, t);
          tmem_ld_wait();
          if (c == 7) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&done[2 * (i & 1)]);
            look = mbar_test(&mine_acc[2 * (~i & 1)], ((i + 1) >> 1) & 1);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) fma2(acc[8 * c + e], t[2 * e], t[2 * e + 1], c < 4 ? scale : scale_up);
        }
        seen = __all_sync(0xffffffffu, look);
      }
      if (!ok) break;
      const int to = output_row(g, entry);
      if constexpr (H != kPlain) {
        // h in place of the sums, its block's scale (gated: with the warp of the other 64 columns), codes
        constexpr int kCols = H == kGated ? 32 : 64;  // pairs of columns of this warp
        uint32_t a = 0;
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          if constexpr (H == kGated) {
            acc[c] = gated2(acc[c], acc[32 + c], p.q.q.glu);
          } else {
            const float x = fp4q::max_nan(acc[c].x, 0.f), y = fp4q::max_nan(acc[c].y, 0.f);
            acc[c] = make_float2(x * x, y * y);
          }
          a = max(a, max(__float_as_uint(acc[c].x) & 0x7fffffffu, __float_as_uint(acc[c].y) & 0x7fffffffu));
        }
        if constexpr (H == kGated) {
          uint32_t* most = reinterpret_cast<uint32_t*>(smem + C::stage) + (done_units & 1) * 256;
          most[half * 128 + r] = a;
          __syncwarp();
          if (lane == 0) mbar_arrive(&both_halves[q4]);
          ok = __all_sync(0xffffffffu, wait(&both_halves[q4], done_units & 1, ab, 139));
          if (!ok) break;
          a = max(a, most[(half ^ 1) * 128 + r]);
          ++done_units;
        }
        const float s = fp8q::block_scale<false>(a);
        if (to >= 0) {
          const int width = H == kGated ? g.n / 2 : g.n;
          const int at = H == kGated ? 128 * U.y + 64 * half : col;
          uint4* codes = reinterpret_cast<uint4*>(p.q.q.codes + (int64_t)to * width + at);
#pragma unroll
          for (int c = 0; c < kCols / 8; ++c) codes[c] = fp8q::encode8<false>(Sixteen{acc + 8 * c}, s);
          if (H != kGated || half == 0) p.q.scales[(int64_t)to * (width / 128) + at / 128] = s;
        }
      } else if constexpr (BOXES) {
        // Through shared memory.  Full tiles leave from there as boxes of 32 rows x 64, under the next
        // unit: stores of all SMs at once take 4000 cycles to drain, and what the warp does next
        // queues behind them.  Others (the end of a group) as 256 bytes of two rows a store.
        const bool boxes = __all_sync(0xffffffffu, to >= 0) || (!RAGGED && g.groups == 1);
        if (lane == 0) bulk_wait_read();
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 16; ++c)
          *reinterpret_cast<uint4*>(stage + (c >> 3) * (kOutTile / 2) + lane * 128 + (((c ^ lane) & 7) << 4)) =
              make_uint4(pack16<OUT & 1>(acc[4 * c]), pack16<OUT & 1>(acc[4 * c + 1]), pack16<OUT & 1>(acc[4 * c + 2]),
                         pack16<OUT & 1>(acc[4 * c + 3]));
        if (boxes) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&p.tmap_out, col, U.z + 32 * q4, stage);
            if (col + 64 < g.n) tma_store_2d(&p.tmap_out, col + 64, U.z + 32 * q4, stage + kOutTile / 2);
            bulk_commit();
          }
        } else {
          __syncwarp();
          const int half8 = (lane >> 3) & 1;
          uint16_t* out = reinterpret_cast<uint16_t*>(g.out) + col + 8 * (lane & 15);
          const bool inside = col + 8 * (lane & 15) < g.n;
          uint4 piece[16];
          int o[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const int row = 2 * c + (lane >> 4);
            piece[c] = *reinterpret_cast<const uint4*>(stage + half8 * (kOutTile / 2) + row * 128 + (((row ^ lane) & 7) << 4));
            o[c] = __shfl_sync(0xffffffffu, to, row);
          }
#pragma unroll
          for (int c = 0; c < 16; ++c)
            if (o[c] >= 0 && inside) *reinterpret_cast<uint4*>(out + (int64_t)o[c] * g.out_stride) = piece[c];
          __syncwarp();
        }
      } else {
        store_rows<OUT>(g, to, col, acc, stage, lane);
      }
    }
  }

  if (BOXES && warp >= 4 && lane == 0) bulk_wait();  // the boxes have left
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

template <int OUT, bool RAGGED, int H, bool BOXES>
cudaError_t launch_pair(const Fp8GemmParams& p, int pairs, cudaStream_t stream) {
  auto kern = fp8_pair_kernel<OUT, RAGGED, H, BOXES>;
  const size_t smem = PairCfg<BOXES>::total(RAGGED);
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * pairs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace fp8

cudaError_t launch_fp8_gemm_pair(const Fp8GemmParams& p, int pairs, cudaStream_t stream) {
  return fp8::with_out(p, [&](auto out, auto ragged) {
    constexpr int O = out.value;
    constexpr bool G = ragged.value;
    return p.out_boxes ? fp8::launch_pair<O & 1, G, fp8::kPlain, true>(p, pairs, stream)
                       : fp8::launch_pair<O, G, fp8::kPlain, false>(p, pairs, stream);
  });
}

// The first product of a layer: p.q takes h (codes, scales, glu).
cudaError_t launch_fp8_gemm_h(const Fp8GemmParams& p, bool gated, int pairs, cudaStream_t stream) {
  return gated ? fp8::launch_pair<0, true, fp8::kGated, false>(p, pairs, stream)
               : fp8::launch_pair<0, true, fp8::kRelu2, false>(p, pairs, stream);
}

}  // namespace b4
