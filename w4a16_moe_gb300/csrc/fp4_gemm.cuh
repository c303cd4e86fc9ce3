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
// DIRECT: few rows altogether (a decode step).  The kernel quantises its unit's rows
// for itself while the first weights are on their way: the epilogue warps take the
// rows' maxima over all of K and write the codes and scales of the CTA's stages into
// shared memory as the products read them, so a call is one launch.
//
// SPLIT: where the units are fewer than the SMs, a cluster of 2 to 8 CTAs shares
// a unit along K.  The partial accumulators go to the first CTA's shared memory
// as asynchronous stores that count on its barrier, and it adds them in rank
// order, so the result does not depend on timing.
//
// Measured: 64 groups of 16 rows, N = 2816, K = 2048 38.7 us (207 MB of weights and scales,
// 5.4 TB/s), of 64 rows 41.6 us; one row, N = K = 4096 6.0 us (quantised before), 6.6 us direct;
// eight groups of one row, N = 1536, K = 4096 (28 MB) 10.1 us direct.
//
// Every wait is bounded (ptx.cuh).

#pragma once

#include "fp4_mma.cuh"
#include "fp4_quant.cuh"

namespace b4 {

cudaError_t ensure_smem_limit(const void* func, size_t bytes);

namespace fp4 {

constexpr int kRows = 64;                       // activation rows of a unit
constexpr int kBox = 32;                        // rows of an activation box
constexpr int kPart16 = 4 * 32 * 16 * 4;        // bytes of 16 rows' partial sums: 4 warps x 32 lanes x 16 values

template <int FMT, bool SPLIT, bool DIRECT>
struct Cfg {
  static constexpr int kSfTiles = sf_tiles(FMT);
  static constexpr int kSfBytes = kSfTiles * kSfTile;           // scales of 128 rows of a stage
  static constexpr int kAStage = kRows * 128;
  // DIRECT: the activations of all the CTA's stages stay, the ring holds weights
  static constexpr int kOwn = DIRECT ? fp4_direct_stages(SPLIT) * (kDirectTile * 128 + kSfBytes) : 0;
  static constexpr int kStage = kWStage + kSfBytes + (DIRECT ? 0 : kAStage + kSfBytes);
  static constexpr int kPart = !SPLIT ? 0 : DIRECT ? kSplitPartBytes * 7 / 12 : kSplitPartBytes;  // one part of 16 rows
  static constexpr int kFit = (216 * 1024 - kEpiBytes - (int)sizeof(RowTable<kRows>) - kPart - kOwn) / kStage;
  static constexpr int kStages = kFit < 7 ? kFit : 7;
  static constexpr int kSfCols = 8 * kSfTiles;                  // tensor-memory columns of a stage's scales
  static constexpr int kSfStage = (DIRECT ? 1 : 2) * kSfBytes;   // scales of a ring stage
  static constexpr size_t a = (size_t)kStages * kWStage;         // activations: the ring's, or DIRECT all
  static constexpr size_t sf = a + (DIRECT ? fp4_direct_stages(SPLIT) * kDirectTile * 128 : (size_t)kStages * kAStage);
  static constexpr size_t sfa = sf + (size_t)kStages * kSfStage;  // DIRECT: the activations' scales
  static constexpr size_t part = sfa + (DIRECT ? fp4_direct_stages(SPLIT) * kSfBytes : 0);
  static constexpr size_t epi = part + kPart;
  static constexpr size_t rows = epi + kEpiBytes;
  static constexpr size_t bars = rows + sizeof(RowTable<kRows>);
  static constexpr int kNumBars = 2 * kStages + 4 + 1 + 4 + 1 + 1;
  static constexpr size_t misc = bars + 8 * kNumBars;
  static constexpr size_t total(bool ragged) { return misc + 48 + (ragged ? sizeof(Groups) : 0); }
  static_assert(2 * kRows + kStages * kSfCols <= 512, "a stage's scale columns are free once its shared memory is");
  static_assert(kStages >= 3, "shared memory budget");
};

// DIRECT: rows first .. first + rows of the operand (group `group`), quantised by 256
// threads: codes of stages s_beg .. s_end to s_a as K-major rows of 128 bytes with the
// 128-byte swizzle, scales to s_sf as tiles, scales of the rows and their places to
// the epilogue's table.  One to eight warps a row, by how many rows there are.
template <typename T, bool ACT, int FMT>
__device__ __forceinline__ void quantize_unit(const Fp4GemmParams& p, const Unit& U, int s_beg, int s_end,
                                              uint8_t* s_a, uint8_t* s_sf, RowTable<kRows>& tab, uint32_t* s_max) {
  using namespace fp4q;
  const Fp4QuantParams& q = p.q;
  constexpr int kSfBytes = sf_tiles(FMT) * kSfTile;
  const int e = threadIdx.x - 128, warp = e >> 5, lane = e & 31;
  const int wpr_log2 = U.rows == 1 ? 3 : U.rows == 2 ? 2 : U.rows <= 4 ? 1 : 0;
  const int tpr = 32 << wpr_log2;
  const int t = e & (tpr - 1);
  const int chunks = q.k / 16;
  const float gw = p.w_gs ? __ldg(p.w_gs + U.group) : 1.f;
  if (e >= U.rows && e < kRows) {  // the table's other rows go nowhere
    tab.g[0][e] = 0.f;
    tab.to[0][e] = -1;
  }
  const int r = warp >> wpr_log2;
  const bool live = r < U.rows;
  const int at = U.first + r;
  int64_t src = at;
  if (live && q.rows) {
    const int i = __ldg(q.rows + at);
    src = i < 0 ? -1 : i / q.row_div;
    if (q.x_rows > 0 && src >= q.x_rows) src = -1;
  }
  const T* x = reinterpret_cast<const T*>(q.x) + (src < 0 ? 0 : src * q.x_stride);
  const int filled = live && src >= 0 ? chunks : 0;
  float gs = 1.f;
  if (FMT == 0 && q.gs_mode == kGsRow) {
    uint32_t a = 0;
    for (int c = t; c < filled; c += tpr) {
      Chunk<T, ACT> h;
      h.get(q, x, c);
      a = max(a, h.amax());
    }
    for (int o = 16; o > 0; o >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
    if (wpr_log2 > 0) {
      if (lane == 0) s_max[warp] = a;
      named_bar_sync(1, 256);
      const int w0 = warp >> wpr_log2 << wpr_log2;
      for (int w = 0; w < 1 << wpr_log2; ++w) a = max(a, s_max[w0 + w]);
    }
    gs = row_gs(a);
  } else if (FMT == 0) {
    gs = __ldg(q.gs + U.group);
  }
  if (live && t == 0) {
    int to = at;
    if (p.out_rows) {
      to = __ldg(p.out_rows + at);
      if (to >= p.out_rows_end) to = -1;
    }
    tab.g[0][r] = gw * gs;
    tab.to[0][r] = to;
  }
  const RowScale rs(gs);
  uint8_t* row_a = s_a + (r >> 3) * 1024 + (r & 7) * 128;
  for (int c0 = 16 * s_beg; c0 < 16 * s_end; c0 += tpr) {  // whole stages: past K zeros
    const int c = c0 + t;
    Chunk<T, ACT> h;
    if (c < filled) h.get(q, x, c);
    else h.zero();
    uint32_t a = h.amax();
    if (FMT != 0) a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
    Quantized o = quantize_block<FMT>(h, a, rs);
    if (c >= chunks) o.w = make_uint2(0, 0), o.code = 0;
    const int st = (c >> 4) - s_beg, in = c & 15;
    if (live && c < 16 * s_end) {
      *reinterpret_cast<uint2*>(row_a + st * (kDirectTile * 128) + (((in >> 1) ^ (r & 7)) << 4) + (in & 1) * 8) = o.w;
      if (FMT == 0) s_sf[st * kSfBytes + (in >> 2) * kSfTile + r * 16 + (in & 3)] = (uint8_t)o.code;
      else if (!(in & 1)) s_sf[st * kSfBytes + (in >> 3) * kSfTile + r * 16 + ((in >> 1) & 3)] = (uint8_t)o.code;
    }
  }
}

template <int FMT, int OUT, bool RAGGED, bool SPLIT, bool DIRECT>
__global__ void __launch_bounds__(kThreads, 1) fp4_gemm_kernel(const __grid_constant__ Fp4GemmParams p) {
  using C = Cfg<FMT, SPLIT, DIRECT>;
  constexpr int NS = C::kStages;
  constexpr int kUnroll = SPLIT && !DIRECT ? NS : 1;  // (a direct call runs its code once, cold)
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw;  // aligned as declared: the swizzled stages need 1024 bytes
  Groups& groups = *reinterpret_cast<Groups*>(smem + C::misc + 48);  // ragged only
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
  uint64_t* own_bar = part_bar + 1;     // DIRECT: the activations are in shared memory
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
    mbar_init(own_bar, kEpiWarps);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(s_tmem, 512);
    tmem_relinquish();
  }
  if (!p.a_is_new) pdl_wait();  // alone in its call: every input may come from the kernel before
  if (DIRECT && p.clear_status && blockIdx.x == 0 && threadIdx.x < 2) p.status[threadIdx.x] = 0;

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
  const int du = SPLIT || DIRECT ? n_units : (int)gridDim.x;

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
      mbar_arrive_expect_tx(&full[slot], kWStage + (DIRECT ? sf_bytes(st) : boxes * kBox * 128 + 2 * sf_bytes(st)));
      tma_load_2d(smem + slot * kWStage, &p.tmap_w, st * 128, wrow, &full[slot]);
      bulk_g2s(s_sf + slot * C::kSfStage, wsf + st * C::kSfBytes, sf_bytes(st), &full[slot]);
    };
    auto copy_a = [&](int slot, int st) {
      if constexpr (DIRECT) return;
      tma_load_2d(s_a + slot * C::kAStage, &p.tmap_a, st * 128, first, &full[slot]);
      if (boxes > 1) tma_load_2d(s_a + slot * C::kAStage + kBox * 128, &p.tmap_a, st * 128, first + kBox, &full[slot]);
      bulk_g2s(s_sf + slot * C::kSfStage + C::kSfBytes, asf + st * C::kSfBytes, sf_bytes(st), &full[slot]);
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
    if (DIRECT && ok) ok = __all_sync(0xffffffffu, wait(own_bar, 0, ab, 109));
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
          const uint32_t sd = s_desc + slot * (C::kSfStage / 16), wd = w_desc + slot * (kWStage / 16);
          const uint32_t ad = a_desc + (DIRECT ? (s - s_beg) * (kDirectTile * 128 / 16) : slot * (C::kAStage / 16));
          const uint32_t sda = DIRECT ? desc_lo(smem_u32(smem + C::sfa)) + (s - s_beg) * (C::kSfBytes / 16) : sd + C::kSfBytes / 16;
#pragma unroll
          for (int i = 0; i < C::kSfTiles; ++i)
            if (i < kts) {
              copy_scales<1>(sfw + 4 * i, sd + i * kStep);
              copy_scales<1>(sfa + 4 * i, sda + i * kStep);
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
    if (!DIRECT && rank == 0)
      fill_rows<kRows, RAGGED>(p, groups, tab, full_rows, empty_rows, wtiles, u0, du, n_units, ab);
    if (RAGGED && !p.out_rows) clear_tail(p, groups.first[p.groups], threadIdx.x - 64);
  } else {
    // --------------------------------------------------------- epilogue
    if (p.a_is_new) pdl_wait();
    if constexpr (DIRECT) {
      if (u0 < n_units) {
        const Unit U = get_unit<kRows, RAGGED>(p, groups, wtiles, u0);
        uint32_t* s_max = s_tmem + 2;
        uint8_t* sfa = smem + C::sfa;
        if (p.q.act < 0) {
          if (p.x_dtype == 0) quantize_unit<__nv_bfloat16, false, FMT>(p, U, s_beg, s_end, s_a, sfa, tab, s_max);
          else if (p.x_dtype == 1) quantize_unit<__half, false, FMT>(p, U, s_beg, s_end, s_a, sfa, tab, s_max);
          else quantize_unit<float, false, FMT>(p, U, s_beg, s_end, s_a, sfa, tab, s_max);
        } else {
          if (p.x_dtype == 0) quantize_unit<__nv_bfloat16, true, FMT>(p, U, s_beg, s_end, s_a, sfa, tab, s_max);
          else if (p.x_dtype == 1) quantize_unit<__half, true, FMT>(p, U, s_beg, s_end, s_a, sfa, tab, s_max);
          else quantize_unit<float, true, FMT>(p, U, s_beg, s_end, s_a, sfa, tab, s_max);
        }
        if (threadIdx.x == 128) {
          tab.rows[0] = U.rows;
          tab.wtile[0] = U.wtile;
        }
        fence_proxy_async_smem();  // generic stores -> the tensor core's async-proxy reads
        __syncwarp();
        if (lane == 0) mbar_arrive(own_bar);
        named_bar_sync(1, 256);    // the row table is complete
      }
    }
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
            ok = (DIRECT || wait(&full_rows[0], 0, ab, 107)) && wait_cluster(part_bar, 0, ab, 108);
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
              const RowInfo info{tab.g[0] + 32 * turn, tab.to[0] + 32 * turn};
              if (n0 < p.n) store_chunk<OUT>(p, lo, hi, info, n0, stage, lane);
            }
          }
        }
      }
    } else {
      uint32_t i = 0;
      for (int u = u0; u < n_units; u += du, ++i) {
        const uint32_t b = i & 1;
        bool ok = DIRECT || wait(&full_rows[b], (i >> 1) & 1, ab, 107);
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
          const RowInfo info{tab.g[b] + 32 * turn, tab.to[b] + 32 * turn};
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

template <int FMT, int OUT, bool RAGGED, bool SPLIT, bool DIRECT>
cudaError_t launch(const Fp4GemmParams& p, int grid, int splits, bool pdl, cudaStream_t stream) {
  auto kern = fp4_gemm_kernel<FMT, OUT, RAGGED, SPLIT, DIRECT>;
  const size_t smem = Cfg<FMT, SPLIT, DIRECT>::total(RAGGED);
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
}  // namespace b4
