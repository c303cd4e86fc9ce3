// Product of two FP8 operands with an fp32 scale per block of 128 along K, on tcgen05
// (sm_103a), dense and grouped by expert with ragged sizes:
//
//   out[t][n] = sum_b sa[t][b] sw[e][n / 128][b] sum_{k in block b} a[t][k] w[e][n][k]
//
// for the rows t of group e.  The block-scaled instructions take powers of two only, so a
// block of 128 along K is an accumulation of its own in tensor memory (four K = 32
// instructions of kind::f8f6f4), which the promoting warps add to fp32 registers times the
// two scales, while the tensor core fills the next of four accumulators.
//
// This is the form for groups of few rows, bound by the stream of weights
// (fp8_gemm_pair.cu is the one for many rows).  Activation rows are on M (128 lanes of tensor
// memory; up to ROWS of them live, the others multiply whatever lies behind them in shared
// memory and are not read), 128 weight rows on N: a lane's scale is one register for all of
// its columns, and the 128 weight rows share theirs.  Roles of the twelve warps: 0 copies,
// 1 (and 3) matrix instructions, 2 (or 3 too) scales (both factors' product, ahead of the promoting
// warps, which a load would hold up) and zeros in rows of a ragged output past the last group, 4 to
// 11 promotion and output, 32 lanes x 64 columns each.  As the second kernel of a call, it
// fills its ring with weights while the quantiser still runs.
//
// DIRECT: few rows altogether (a decode step).  The kernel quantises its unit's rows for
// itself while the first weights are on their way, so a call is one launch.
//
// SPLIT: where the units are fewer than the SMs, a cluster of 2 to 8 CTAs shares a unit along
// K.  The partial sums go to the first CTA's shared memory as asynchronous stores that count
// on its barrier, and it adds them in rank order, so the result does not depend on timing.
//
// Measured: 64 groups of 6 rows, N = 2816, K = 2048 61.9 us (372 MB, 6.0 TB/s), of 96 rows 70 us (5.9 TB/s); one row, N = K = 4096
// 7.6 us, direct 7.7; eight groups of one row, N = 1536, K = 4096 (50 MB) direct 13.5 us: 96 CTAs of a unit each,
// whose 32 stages follow one another.
//
// Every wait is bounded (ptx.cuh).
#pragma once

#include "fp8_mma.cuh"
#include "fp8_quant.cuh"

namespace b4 {

cudaError_t ensure_smem_limit(const void* func, size_t bytes);

namespace fp8 {

constexpr int kAccs = 4;                     // accumulators of 128 columns
constexpr int kScaleRing = 2 * kAccs;        // stages of scales
constexpr int kABox = 32;                    // activation rows of a box

template <int ROWS, bool SPLIT, bool DIRECT>
struct Cfg {
  static constexpr int kAStage = ROWS * 128;
  static constexpr int kPart = SPLIT ? kFp8PartBytes : 0;
  // DIRECT: the activations of all the CTA's stages stay, the ring holds weights
  static constexpr int kOwnStages = SPLIT ? kFp8DirectSplitStages : kFp8DirectStages;
  static constexpr int kOwn = DIRECT ? kOwnStages * kFp8DirectTile * 128 : 0;
  static constexpr int kStage = kWStage + (DIRECT ? 0 : kAStage);
  static constexpr int kScaleRows = DIRECT ? kFp8DirectTile : ROWS;
  static constexpr int kScales = (DIRECT ? kOwnStages : kScaleRing) * kScaleRows * 4;
  static constexpr int kFit = (200 * 1024 - kPart - kOwn - kScales) / kStage;
  static constexpr int kSlots = kFit < 12 ? kFit : 12;
  // activations first: the instructions read 128 rows of 128 bytes from each tile's start
  static constexpr size_t w = DIRECT ? kOwn : (size_t)kSlots * kAStage;
  static constexpr size_t part = w + (size_t)kSlots * kWStage;
  static constexpr size_t scales = part + kPart;
  static constexpr size_t stage = scales + kScales;
  static constexpr size_t bars = stage + kEpiWarps * kStagePiece;
  static constexpr int kNumBars = 2 * kSlots + 2 * kAccs + 3;
  static constexpr size_t misc = bars + 8 * (kNumBars + 1);
  static constexpr size_t total(bool ragged) { return misc + 16 + (ragged ? sizeof(Groups) : 0); }
  static constexpr int kPromoters = ROWS / 16;  // warps that have rows: two a quarter
  static constexpr int kIssuers = ROWS == 32 ? 2 : 1, kScalers = 3 - kIssuers;  // of warps 1 to 3
  static_assert(kSlots >= kAccs && kWStage * kSlots >= 128 * 128, "shared memory budget");
};

// DIRECT: rows first .. first + rows of the operand, quantised by 256 threads: codes of the
// stages s_beg .. s_end to s_a as K-major rows of 128 bytes with the 128-byte swizzle, scales
// times the weights' to s_scale.  Eight neighbouring threads take a block of a row.
template <typename T, bool ACT, bool POW2>
__device__ __forceinline__ void quantize_unit(const Fp8GemmParams& p, const Unit& U, const float* sw, int s_beg, int s_end,
                                              uint8_t* s_a, float* s_scale) {
  const Fp4QuantParams& q = p.q.q;
  const int e = threadIdx.x - 128;
  const int blocks = U.rows * (s_end - s_beg);
  for (int b0 = 0; b0 < blocks; b0 += 32) {
    const int b = b0 + (e >> 3);
    const bool live = b < blocks;
    const int st = live ? b / U.rows : 0, r = live ? b - st * U.rows : 0;
    const int s = s_beg + st, chunk = 8 * s + (e & 7);
    int64_t src = U.first + r;
    if (live && q.rows) {
      const int i = __ldg(q.rows + src);
      src = i < 0 ? -1 : i / q.row_div;
      if (q.x_rows > 0 && src >= q.x_rows) src = -1;
    }
    const float ws = live ? __ldg(sw + s) : 0.f;
    fp4q::Chunk<T, ACT> h;
    if (live && src >= 0 && 16 * chunk < q.k) h.get(q, reinterpret_cast<const T*>(q.x) + src * q.x_stride, chunk);
    else h.zero();
    uint32_t a = h.amax();
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
    const float scale = fp8q::block_scale<POW2>(a);
    uint4 w = fp8q::encode8<POW2>(h, scale);
    if (16 * chunk >= q.k) w = make_uint4(0, 0, 0, 0);  // (past K, under a scale of NaN too)
    if (live) {
      *reinterpret_cast<uint4*>(s_a + st * (kFp8DirectTile * 128) + (r >> 3) * 1024 + (r & 7) * 128 +
                                (((e & 7) ^ (r & 7)) << 4)) = w;
      if ((e & 7) == 0) s_scale[st * kFp8DirectTile + r] = scale * ws;
    }
  }
}

template <typename T>
__device__ __forceinline__ void quantize_unit_t(const Fp8GemmParams& p, const Unit& U, const float* sw, int s_beg, int s_end,
                                                uint8_t* s_a, float* s_scale) {
  if (p.q.q.act < 0) {
    if (p.q.pow2) quantize_unit<T, false, true>(p, U, sw, s_beg, s_end, s_a, s_scale);
    else quantize_unit<T, false, false>(p, U, sw, s_beg, s_end, s_a, s_scale);
  } else {
    if (p.q.pow2) quantize_unit<T, true, true>(p, U, sw, s_beg, s_end, s_a, s_scale);
    else quantize_unit<T, true, false>(p, U, sw, s_beg, s_end, s_a, s_scale);
  }
}

template <int OUT, bool RAGGED, int ROWS, bool SPLIT, bool DIRECT>
__global__ void __launch_bounds__(kThreads, 1) fp8_gemm_kernel(const __grid_constant__ Fp8GemmParams p) {
  using C = Cfg<ROWS, SPLIT, DIRECT>;
  constexpr int NS = C::kSlots;
  extern __shared__ __align__(1024) uint8_t smem[];
  Groups& groups = *reinterpret_cast<Groups*>(smem + C::misc + 16);  // ragged only
  uint8_t* s_a = smem;
  uint8_t* s_w = smem + C::w;
  float* s_scale = reinterpret_cast<float*>(smem + C::scales);  // [stage][row]
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::bars);
  uint64_t* empty = full + NS;
  uint64_t* full_acc = empty + NS;       // the products and (not DIRECT) the stage's scales
  uint64_t* empty_acc = full_acc + kAccs;
  uint64_t* drain = empty_acc + kAccs;
  uint64_t* part_bar = drain + 1;        // SPLIT: the other CTAs' partial sums have arrived
  uint64_t* own_bar = part_bar + 1;      // DIRECT: the activations are in shared memory
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + C::misc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + C::misc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Fp4GemmParams& g = p.g;
  const int splits = SPLIT ? (int)cluster_size() : 1;
  const int rank = SPLIT ? (int)cluster_rank() : 0;
  const Abort ab{g.status, s_abort};

  if (threadIdx.x == 0) {
    *s_abort = 0;
    for (int i = 0; i < NS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < kAccs; ++i) {
      mbar_init(&full_acc[i], DIRECT ? 1 : 2);
      mbar_init(&empty_acc[i], C::kPromoters);
    }
    mbar_init(drain, C::kIssuers);
    mbar_init(part_bar, 1);
    mbar_init(own_bar, kEpiWarps);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(s_tmem, 512);
    tmem_relinquish();
  }
  if (!g.a_is_new) pdl_wait();  // alone in its call: every input may come from the kernel before
  if (DIRECT && g.clear_status && blockIdx.x == 0 && threadIdx.x < 2) g.status[threadIdx.x] = 0;
  const int wtiles = cdiv(g.n, 128);
  if (RAGGED) build_groups<ROWS>(g, groups);
  tc_fence_before();
  if constexpr (SPLIT) cluster_sync();  // every CTA's barriers exist before another signals them
  else __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0) pdl_launch_dependents();
  const uint32_t tmem = *s_tmem;
  const int n_units = (RAGGED ? groups.tiles[g.groups] : g.groups * cdiv(g.m, ROWS)) * wtiles;
  // this CTA's stages, and its units: a cluster takes one
  const int s_beg = SPLIT ? rank * p.kb / splits : 0;
  const int s_end = SPLIT ? (rank + 1) * p.kb / splits : p.kb;
  const int u0 = SPLIT ? (int)blockIdx.x / splits : (int)blockIdx.x;
  const int du = SPLIT || DIRECT ? n_units : (int)gridDim.x;

  if (warp == 0) {
    // ----------------------------------------------------------- copies
    uint32_t i = 0;
    bool ok = u0 < n_units;
    // while the kernel before still writes the activations: weights first, for as much
    // of the ring as the first unit fills
    int early = 0;
    if (g.a_is_new) {
      early = ok ? min(NS, s_end - s_beg) : 0;
      if (early == 0) pdl_wait();
    }
    auto weights = [&](uint32_t slot, int s, int wrow, int boxes) {
      mbar_arrive_expect_tx(&full[slot], kWStage + (DIRECT ? 0 : boxes * kABox * 128));
      tma_load_2d(s_w + slot * kWStage, &p.tmap_w, s * 128, wrow, &full[slot]);
    };
    for (int u = u0; u < n_units && ok; u += du) {
      const Unit U = get_unit<ROWS, RAGGED>(g, groups, wtiles, u);
      const int wrow = (int)warp_uniform(U.group) * g.n + (int)warp_uniform(U.wtile) * 128;
      const int first = (int)warp_uniform(U.first), boxes = cdiv((int)warp_uniform(U.rows), kABox);
      if (early > 0) {
        if (elect_one())
          for (int j = 0; j < early; ++j) weights(j, s_beg + j, wrow, boxes);
        __syncwarp();
        pdl_wait();
      }
      for (int s = s_beg; s < s_end; ++s, ++i) {
        const uint32_t slot = i % NS;
        ok = __all_sync(0xffffffffu, wait(&empty[slot], ((i / NS) & 1) ^ 1, ab, 121));
        if (!ok) break;
        if (elect_one()) {
          if (early <= 0) weights(slot, s, wrow, boxes);
          if constexpr (!DIRECT)
            for (int b = 0; b < boxes; ++b)
              tma_load_2d(s_a + slot * C::kAStage + b * kABox * 128, &p.tmap_a, s * 128, first + b * kABox, &full[slot]);
        }
        __syncwarp();
        --early;
      }
    }
    if (ab.raised() && lane == 0) {
      // copies already issued land before the shared memory goes away: give them a fixed time
      const unsigned long long t0 = globaltimer();
      while (globaltimer() - t0 < 2000000ull) {
      }
    }
    __syncwarp();
  } else if (warp == 1 || (warp == 3 && C::kIssuers == 2)) {
    // ---------------------------------------------- matrix instructions
    // Units of 32 rows: warp 1 issues the even stages, warp 3 the odd ones, since one warp takes some
    // 600 cycles for a stage, more than DRAM takes to bring it.  (With 128 rows scales take that
    // long too, and need the warp more: 64 groups of 96 rows 70 us, 92 the other way.)
    const int w = C::kIssuers == 2 ? warp >> 1 : 0;
    const uint32_t w_desc = desc_lo(smem_u32(s_w)), a_desc = desc_lo(smem_u32(s_a));
    constexpr uint32_t idesc = idesc_fp8(128, 128);
    const int stages = s_end - s_beg;
    const int total = u0 < n_units ? (SPLIT || DIRECT ? 1 : (n_units - 1 - u0) / du + 1) * stages : 0;
    bool ok = true;
    if (DIRECT && total > 0) ok = __all_sync(0xffffffffu, wait(own_bar, 0, ab, 129));
    for (int i = w; i < total && ok; i += C::kIssuers) {
      const uint32_t slot = i % NS, acc = i % kAccs;
      // (the accumulator first: with it the stages kAccs back have run, so that the slot's barrier is not
      // two phases behind, where it would look complete)
      ok = __all_sync(0xffffffffu, wait(&empty_acc[acc], ((i / kAccs) & 1) ^ 1, ab, 122));
      ok = ok && __all_sync(0xffffffffu, wait(&full[slot], (i / NS) & 1, ab, 123));
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
        const uint32_t wd = w_desc + slot * (kWStage / 16);
        const uint32_t ad = a_desc + (DIRECT ? i * (kFp8DirectTile * 128 / 16) : slot * (C::kAStage / 16));
#pragma unroll
        for (int j = 0; j < 4; ++j) mma_fp8(tmem + acc * 128, ad + 2 * j, wd + 2 * j, idesc, j > 0);
        mma_commit(&full_acc[acc]);
        mma_commit(&empty[slot]);
      }
      __syncwarp();
    }
    // drain: every instruction issued has completed
    if (elect_one()) mma_commit(drain);
    const unsigned long long t0 = globaltimer();
    while (!mbar_try_wait(drain, 0) && globaltimer() - t0 < kWaitLimitNs) {
    }
    __syncwarp();
  } else if (warp < 4) {
    // ---- scales, stages by turns; rows of a ragged output past the last group are zero
    if (g.a_is_new) pdl_wait();
    if constexpr (!DIRECT) {
      // Looked up kDeep stages of this warp ahead of their turn, into the next unit too: a load from L2
      // takes a microsecond and more under the weights' traffic (64 groups of 6 rows, N = 2048, K = 1408
      // 34.0 us with each unit for itself, 32.8).  No deeper: in a layer, whose kernels follow one another, a
      // launch fetches its code anew (8 deep, twice unrolled: 64 tokens, 6 of 64 experts 118 us, 111 so).
      constexpr int kTurn = C::kScalers, kPer = ROWS / 32;
      constexpr int kDeep = 4;
      const int stages = s_end - s_beg;
      const int total = u0 < n_units ? (SPLIT ? 1 : (n_units - 1 - u0) / du + 1) * stages : 0;
      const int i0 = kTurn == 2 ? warp & 1 : 0;
      const float *sw = p.w_scales, *sa[kPer];  // of unit lu, its rows lane, lane + 32, ..
      bool live[kPer];
      int lu = u0 - du, ls = s_beg + i0 + stages;  // looked up next (the first: stage i0 of the first unit)
      float f[kDeep], v[kDeep][kPer];
      auto look_up = [&](int d) {
        while (ls >= s_end) {
          ls -= stages;
          lu += du;
          if (ls >= s_end) continue;
          if (lu >= n_units) return;
          const Unit U = get_unit<ROWS, RAGGED>(g, groups, wtiles, lu);
          sw = p.w_scales + ((int64_t)U.group * wtiles + U.wtile) * p.kb;
#pragma unroll
          for (int j = 0; j < kPer; ++j) {
            live[j] = 32 * j + lane < U.rows;
            sa[j] = p.a_scales + (int64_t)(U.first + (live[j] ? 32 * j + lane : 0)) * p.kb;
          }
        }
        if (lu >= n_units) return;
        f[d] = __ldg(sw + ls);
#pragma unroll
        for (int j = 0; j < kPer; ++j) v[d][j] = live[j] ? sa[j][ls] : 0.f;
        ls += kTurn;
      };
      bool ok = true;
      // (the first turn only looks up: one copy of the code, which a launch has to fetch)
      for (int base = i0 - kTurn * kDeep; base < total && ok; base += kTurn * kDeep) {
#pragma unroll
        for (int d = 0; d < kDeep; ++d) {
          const int i = base + kTurn * d;
          if (i >= total || !ok) continue;
          if (i >= 0) {
            // the products before the last on this accumulator are complete: so they were issued, after the
            // promoters had let go of the stage before that, whose scales lie where this stage's go
            if (i >= kAccs) ok = __all_sync(0xffffffffu, wait(&full_acc[i % kAccs], ((i / kAccs) & 1) ^ 1, ab, 127));
            if (!ok) continue;
#pragma unroll
            for (int j = 0; j < kPer; ++j) s_scale[(i % kScaleRing) * ROWS + 32 * j + lane] = f[d] * v[d][j];
            __syncwarp();
            if (lane == 0) mbar_arrive(&full_acc[i % kAccs]);
          }
          look_up(d);
        }
      }
    }
    if (RAGGED && !g.out_rows) clear_tail<32 * C::kScalers>(g, groups.first[g.groups], threadIdx.x - 64);
  } else {
    // ------------------------------------------- promotion and output
    if (g.a_is_new) pdl_wait();
    if constexpr (DIRECT) {
      if (u0 < n_units) {
        const Unit U = get_unit<ROWS, RAGGED>(g, groups, wtiles, u0);
        const float* sw = p.w_scales + ((int64_t)U.group * wtiles + U.wtile) * p.kb;
        if (p.x_dtype == 0) quantize_unit_t<__nv_bfloat16>(p, U, sw, s_beg, s_end, s_a, s_scale);
        else if (p.x_dtype == 1) quantize_unit_t<__half>(p, U, sw, s_beg, s_end, s_a, s_scale);
        else quantize_unit_t<float>(p, U, sw, s_beg, s_end, s_a, s_scale);
        fence_proxy_async_smem();  // generic stores -> the tensor core's async-proxy reads
        __syncwarp();
        if (lane == 0) mbar_arrive(own_bar);
        named_bar_sync(1, 256);    // the scales are complete
      }
    }
    const int q4 = warp & 3, half = (warp - 4) >> 2;
    const int r = 32 * q4 + lane;
    const uint32_t taddr = tmem + ((uint32_t)(32 * q4) << 16) + 64 * half;
    uint8_t* stage = smem + C::stage + (warp - 4) * kStagePiece;
    uint32_t i = 0;
    bool ok = true;
    for (int u = u0; u < n_units && ok && 32 * q4 < ROWS; u += du) {
      const Unit U = get_unit<ROWS, RAGGED>(g, groups, wtiles, u);
      if (32 * q4 >= U.rows) {  // no row of this warp's
        for (int s = s_beg; s < s_end && ok; ++s, ++i) {
          ok = __all_sync(0xffffffffu, wait(&full_acc[i % kAccs], (i / kAccs) & 1, ab, 124));
          if (ok && lane == 0) mbar_arrive(&empty_acc[i % kAccs]);
        }
        continue;
      }
      const int entry = output_entry(g, U.first + r, r < U.rows);
      float2 acc[32];
#pragma unroll
      for (int c = 0; c < 32; ++c) acc[c] = make_float2(0.f, 0.f);
      bool seen = false;
      for (int s = s_beg; s < s_end; ++s, ++i) {  // (one way out: see fp8_gemm_pair.cu)
        const uint32_t b = i % kAccs;
        if (!seen) ok = __all_sync(0xffffffffu, wait(&full_acc[b], (i / kAccs) & 1, ab, 124)) && ok;
        tc_fence_after();
        const float scale = DIRECT ? s_scale[(s - s_beg) * kFp8DirectTile + (lane & (kFp8DirectTile - 1))]
                                   : s_scale[(i % kScaleRing) * ROWS + r];
        uint32_t t[2][32];
        tmem_ld32(taddr + 128 * b, t[0]);
        tmem_ld32(taddr + 128 * b + 32, t[1]);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty_acc[b]);
        const bool look = mbar_test(&full_acc[(i + 1) % kAccs], ((i + 1) / kAccs) & 1);
#pragma unroll
        for (int c = 0; c < 32; ++c) fma2(acc[c], t[c >> 4][2 * (c & 15)], t[c >> 4][2 * (c & 15) + 1], scale);
        seen = __all_sync(0xffffffffu, look);
      }
      if (!ok) break;
      if constexpr (SPLIT) {
        // a CTA's partial sums: [half][4 columns][row]
        float4* part = reinterpret_cast<float4*>(smem + C::part) + half * 16 * U.rows + lane;
        const size_t pitch = (size_t)U.rows * 32;
        if (rank > 0) {
          const uint32_t dst = map_rank(part + (rank - 1) * pitch, 0);
          const uint32_t bar = map_rank(part_bar, 0);
          if (lane < U.rows) {
#pragma unroll
            for (int c = 0; c < 16; ++c)
              store_async4(dst + c * U.rows * 16, __float_as_uint(acc[2 * c].x), __float_as_uint(acc[2 * c].y),
                           __float_as_uint(acc[2 * c + 1].x), __float_as_uint(acc[2 * c + 1].y), bar);
          }
          continue;
        }
        if (warp == 4 && lane == 0) mbar_arrive_expect_tx(part_bar, (uint32_t)(splits - 1) * U.rows * 512);
        ok = __all_sync(0xffffffffu, wait_cluster(part_bar, 0, ab, 128));
        if (!ok) break;
        if (lane < U.rows)
          for (int k = 0; k + 1 < splits; ++k) {
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              const float4 v = part[k * pitch + c * U.rows];
              acc[2 * c].x += v.x, acc[2 * c].y += v.y, acc[2 * c + 1].x += v.z, acc[2 * c + 1].y += v.w;
            }
          }
      }
      store_rows<OUT>(g, output_row(g, entry), U.wtile * 128 + 64 * half, acc, stage, lane);
    }
  }

  tc_fence_before();
  if constexpr (SPLIT) cluster_sync();  // the first CTA's shared memory outlives the others' stores
  else __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

template <int OUT, bool RAGGED, int ROWS, bool SPLIT, bool DIRECT>
cudaError_t launch(const Fp8GemmParams& p, int grid, int splits, cudaStream_t stream) {
  auto kern = fp8_gemm_kernel<OUT, RAGGED, ROWS, SPLIT, DIRECT>;
  const size_t smem = Cfg<ROWS, SPLIT, DIRECT>::total(RAGGED);
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid * splits);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = splits;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = SPLIT ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace fp8
}  // namespace b4
