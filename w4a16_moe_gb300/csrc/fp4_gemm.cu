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
// 2 and 3 rows of a ragged output past the last group (zeros), 4 to 11 epilogue.
// Two accumulators, so a unit's epilogue runs under the next unit's products.
// Every wait is bounded (ptx.cuh).

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fp4.cuh"
#include "ptx.cuh"
#include "tma.cuh"

namespace b4 {

cudaError_t ensure_smem_limit(const void* func, size_t bytes);

namespace fp4 {

constexpr int kThreads = 384;
constexpr int kEpiWarps = 8;                 // two per quarter of the lanes, alternating 32-column chunks
constexpr int kEpiRow = 80;                  // staged 64-byte row, padded so that eight rows hit eight bank groups
constexpr int kWStage = 128 * 128;           // weight codes of a stage
constexpr int kMaxGroups = 1024;

// FMT 0 NVFP4, 1 MXFP4; NT: activation rows of a unit.
template <int FMT, int NT>
struct Cfg {
  static constexpr int kSfTiles = FMT == 0 ? 4 : 2;             // scale tiles of a stage (per 128 rows)
  static constexpr int kSfRows = kSfTiles * kSfTile;            // scales of 128 rows of a stage
  static constexpr int kABlocks = NT > 64 ? 2 : 1;              // 128-row scale tiles a unit's rows touch
  static constexpr int kAStage = NT * 128;
  static constexpr int kStage = kWStage + kAStage + 2048 * (1 + kABlocks);
  static constexpr int kEpi = kEpiWarps * 32 * kEpiRow;
  static constexpr int kStages = (216 * 1024 - kEpi) / kStage;
  static constexpr int kSfCols = 4 * kSfTiles * (1 + kABlocks);  // tensor-memory columns of a stage's scales
  // scale buffers in tensor memory: one per stage where they fit, then a stage's
  // scales are free to overwrite once its shared memory is
  static constexpr int kSfFit = (512 - 2 * NT) / kSfCols;
  static constexpr int kSfRing = kSfFit < kStages ? kSfFit : kStages;
  static constexpr uint32_t kTmemCols = 512;
  static constexpr size_t a = (size_t)kStages * kWStage;
  static constexpr size_t sf = a + (size_t)kStages * kAStage;
  static constexpr size_t epi = sf + (size_t)kStages * 2048 * (1 + kABlocks);
  static constexpr size_t bars = epi + kEpi;
  static constexpr int kNumBars = 2 * kStages + 4 + 1;
  static constexpr size_t misc = bars + 8 * kNumBars;
  static constexpr size_t total = misc + 16 + 1024;             // + alignment slack
  static_assert(kSfRing >= 2, "tensor memory budget");
  static_assert(kAStage % 1024 == 0, "swizzle atoms stay 1024-byte aligned");
};

// Instruction descriptor of the block-scaled kinds: E2M1 operands, both
// K-major, M = 128, scales E4M3 (0) or E8M0 (1); `sf` is the byte of a scale
// word that the instruction starts at.
__device__ __forceinline__ uint32_t idesc_fp4(int fmt, uint32_t n, uint32_t sf) {
  return (sf << 4)               // B scale byte
         | (1u << 7)             // A: E2M1
         | (1u << 10)            // B: E2M1
         | ((n >> 3) << 17)      // N >> 3
         | ((uint32_t)fmt << 23) // scale type
         | ((128u >> 4) << 24)   // M >> 4
         | (sf << 29);           // A scale byte
}

template <int FMT>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                        uint32_t accumulate) {
  if constexpr (FMT == 0)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// One 512-byte scale tile (32 rows of 16 bytes) into four columns of tensor
// memory, the same in all four lane quarters.
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

struct Unit {
  int group, wtile, first, rows;  // first: packed row; rows: live rows
  int atile;                      // scale tile of row `first`
  int shift;                      // 32-row groups of that tile before `first`
};

// Shared tables of the groups: first packed row, and activation tiles before the group.
struct Groups {
  const int* first;  // [groups + 1], ragged only
  const int* tiles;  // [groups + 1]
};

template <int NT>
__device__ __forceinline__ Unit get_unit(const Fp4GemmParams& p, const Groups& g, int wtiles, int u) {
  int lo = 0;
  int t;
  Unit U;
  if (p.offsets) {
    int hi = p.groups - 1;  // last group whose tiles start at or before the unit's
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((long long)g.tiles[mid] * wtiles <= u) lo = mid;
      else hi = mid - 1;
    }
    const int nt = g.tiles[lo + 1] - g.tiles[lo];
    const int v = u - g.tiles[lo] * wtiles;
    U.wtile = v / nt;
    t = v - U.wtile * nt;
    U.first = g.first[lo] + t * NT;
    U.rows = min(NT, g.first[lo + 1] - U.first);
    U.atile = g.first[lo] / 128 + lo + t * NT / 128;
  } else {
    const int nt = cdiv(p.m, NT);
    lo = u / (nt * wtiles);
    const int v = u - lo * nt * wtiles;
    U.wtile = v / nt;
    t = v - U.wtile * nt;
    U.first = lo * p.m + t * NT;
    U.rows = min(NT, p.m - t * NT);
    U.atile = lo * cdiv(p.m, 128) + t * NT / 128;
  }
  U.group = lo;
  U.shift = (t * NT & 127) >> 5;
  return U;
}

__device__ __forceinline__ void store_out(const Fp4GemmParams& p, int64_t at, float v) {
  if (p.out_dtype == 0) reinterpret_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(v);
  else if (p.out_dtype == 1) reinterpret_cast<__half*>(p.out)[at] = __float2half_rn(v);
  else reinterpret_cast<float*>(p.out)[at] = v;
}

__device__ __forceinline__ uint32_t pack16(int dtype, float lo, float hi) {
  if (dtype == 0) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

template <int FMT, int NT>
__global__ void __launch_bounds__(kThreads, 1) fp4_gemm_kernel(const __grid_constant__ Fp4GemmParams p) {
  using C = Cfg<FMT, NT>;
  constexpr int NS = C::kStages;
  constexpr int kBox = fp4_box_rows(NT);
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ int s_first[kMaxGroups + 1], s_tiles[kMaxGroups + 1], s_warp[kThreads / 32];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* s_a = smem + C::a;
  uint8_t* s_sf = smem + C::sf;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::bars);
  uint64_t* empty = full + NS;
  uint64_t* full_acc = empty + NS;
  uint64_t* empty_acc = full_acc + 2;
  uint64_t* drain = empty_acc + 2;
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
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(s_tmem, C::kTmemCols);
    tmem_relinquish();
  }
  if (!p.a_is_new) pdl_wait();  // standalone: every input may come from the kernel before

  // group tables: a block scan of the groups' tile counts, four groups a thread
  const int wtiles = cdiv(p.n, 128);
  if (p.offsets) {
    int cnt[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = 4 * threadIdx.x + i;
      cnt[i] = 0;
      if (e <= p.groups) {
        const int lo = min(max(__ldg(p.offsets + e), 0), p.m);
        s_first[e] = lo;
        if (e < p.groups) cnt[i] = cdiv(max(min(__ldg(p.offsets + e + 1), p.m) - lo, 0), NT);
      }
      sum += cnt[i];
    }
    if (threadIdx.x == 0 && p.groups == kMaxGroups)
      s_first[kMaxGroups] = min(max(__ldg(p.offsets + kMaxGroups), 0), p.m);
    int scan = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan += v;
    }
    if (lane == 31) s_warp[warp] = scan;
    __syncthreads();
    int before = scan - sum;
    for (int w = 0; w < warp; ++w) before += s_warp[w];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = 4 * threadIdx.x + i;
      if (e <= p.groups) s_tiles[e] = before;
      before += cnt[i];
      if (e + 1 == kMaxGroups) s_tiles[kMaxGroups] = before;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0) pdl_launch_dependents();
  const uint32_t tmem = *s_tmem;
  const Groups groups{s_first, s_tiles};
  const int n_units = (p.offsets ? s_tiles[p.groups] : p.groups * cdiv(p.m, NT)) * wtiles;
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
      const Unit U = get_unit<NT>(p, groups, wtiles, u);
      const int rows = __shfl_sync(0xffffffffu, U.rows, 0), shift = __shfl_sync(0xffffffffu, U.shift, 0);
      const int first = __shfl_sync(0xffffffffu, U.first, 0), atile = __shfl_sync(0xffffffffu, U.atile, 0);
      const int group = __shfl_sync(0xffffffffu, U.group, 0), wtile = __shfl_sync(0xffffffffu, U.wtile, 0);
      const int boxes = (rows + kBox - 1) / kBox;
      const bool two = C::kABlocks == 2 && shift * 32 + rows > 128;
      const uint8_t* wsf = p.w_scales + ((size_t)group * wtiles + wtile) * tile_pitch;
      const uint8_t* asf = p.a_scales + (size_t)atile * tile_pitch;
      const int wrow = group * p.n + wtile * 128;
      const uint32_t code_bytes = kWStage + boxes * kBox * 128;
      for (int s = 0; s < stages; ++s, ++ss) {
        const uint32_t slot = ss % NS;
        ok = __all_sync(0xffffffffu, mbar_wait(&empty[slot], ((ss / NS) & 1) ^ 1, ab, 101));
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
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t w_desc = smem_desc_sw128(__shfl_sync(0xffffffffu, smem_u32(smem), 0));
    const uint64_t a_desc = smem_desc_sw128(__shfl_sync(0xffffffffu, smem_u32(s_a), 0));
    const uint64_t s_desc = smem_desc_noswizzle(__shfl_sync(0xffffffffu, smem_u32(s_sf), 0), 16, 128);
    for (int u = blockIdx.x; u < n_units; u += gridDim.x) {
      const Unit U = get_unit<NT>(p, groups, wtiles, u);
      const int rows = __shfl_sync(0xffffffffu, U.rows, 0), shift = __shfl_sync(0xffffffffu, U.shift, 0);
      const bool two = C::kABlocks == 2 && shift * 32 + rows > 128;
      const uint32_t idesc = idesc_fp4(FMT, (uint32_t)round_up(rows, 16), 0);
      const uint32_t abuf = acc_i & 1;
      if (!__all_sync(0xffffffffu, mbar_wait(&empty_acc[abuf], ((acc_i >> 1) & 1) ^ 1, ab, 102))) break;
      tc_fence_after();
      const uint32_t d = tm + abuf * NT;
      bool ok = true;
      for (int s = 0; s < stages; ++s, ++ss) {
        const uint32_t slot = ss % NS;
        // with fewer scale buffers than stages, the products that last read this one come first
        if (C::kSfRing < NS && ss >= C::kSfRing)
          ok = mbar_wait(&empty[(ss - C::kSfRing) % NS], ((ss - C::kSfRing) / NS) & 1, ab, 103);
        ok = ok && mbar_wait(&full[slot], (ss / NS) & 1, ab, 104);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t sfw = tm + 2 * NT + (ss % C::kSfRing) * C::kSfCols;
        const uint32_t sfa = sfw + 4 * C::kSfTiles;
        const uint64_t sd = s_desc + slot * (2048 * (1 + C::kABlocks) / 16);
        const uint64_t wd = w_desc + slot * (kWStage / 16), ad = a_desc + slot * (C::kAStage / 16);
        const int kts = min(C::kSfTiles, k_tiles - s * C::kSfTiles);
        const int kn = min(4, k64 - 4 * s);
        if (elect_one()) {
#pragma unroll
          for (int i = 0; i < C::kSfTiles; ++i)
            if (i < kts) {
              copy_scales(sfw + 4 * i, sd + i * (kSfTile / 16));
              copy_scales(sfa + 4 * i * C::kABlocks, sd + 128 + i * (kSfTile / 16));
              if (two) copy_scales(sfa + 4 * (i * C::kABlocks + 1), sd + 256 + i * (kSfTile / 16));
            }
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i < kn) {
              const int t = FMT == 0 ? i : i >> 1;  // MXFP4: a scale tile serves two instructions
              const uint32_t sf = FMT == 0 ? 0 : 2 * (i & 1);
              mma_fp4<FMT>(d, wd + 2 * i, ad + 2 * i, idesc | sf << 4 | sf << 29, sfw + 4 * t,
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
    // ------------------- rows of a ragged output past the last group: zero
    if (p.offsets && !p.out_rows) {
      if (p.a_is_new) pdl_wait();
      const int width = p.out_dtype == 2 ? 4 : 2;
      const int live = s_first[p.groups];
      for (int r = live + blockIdx.x; r < p.m; r += gridDim.x)
        for (int c = threadIdx.x - 64; c < p.n; c += 64) {
          if (width == 4) reinterpret_cast<uint32_t*>(p.out)[(int64_t)r * p.out_stride + c] = 0;
          else reinterpret_cast<uint16_t*>(p.out)[(int64_t)r * p.out_stride + c] = 0;
        }
    }
  } else {
    // --------------------------------------------------------- epilogue
    if (p.a_is_new) pdl_wait();
    // Chunks of 32 rows of the unit: fragments of 8 x 8 (weight row x activation
    // row) leave tensor memory, take their scales, and go through a transposing
    // store to shared memory, so that the chunk leaves as 16-byte pieces of
    // output rows (64 bytes a row and warp).  Outputs that are not 16-bit or not
    // 16-byte aligned go straight from the fragments.
    const int q4 = warp & 3;
    const int turn = (warp - 4) >> 2;
    uint8_t* stage = smem + C::epi + (warp - 4) * 32 * kEpiRow;
    const uint32_t st_addr = smem_u32(stage) + (lane & 7) * kEpiRow + (lane >> 3) * 16;
    const bool staged = p.vec && p.out_dtype != 2;
    uint32_t acc_i = 0;
    for (int u = blockIdx.x; u < n_units; u += gridDim.x) {
      const Unit U = get_unit<NT>(p, groups, wtiles, u);
      const uint32_t abuf = acc_i & 1;
      const int n0 = U.wtile * 128 + 32 * q4;
      const float gw = (p.w_gs ? __ldg(p.w_gs + U.group) : 1.f) *
                       (p.a_gs && !p.a_gs_per_row ? __ldg(p.a_gs + U.group) : 1.f);
      const bool ok = mbar_wait(&full_acc[abuf], (acc_i >> 1) & 1, ab, 105);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      const uint32_t taddr = tmem + ((uint32_t)(32 * q4) << 16) + abuf * NT;
      for (int c0 = 32 * turn; c0 < U.rows; c0 += 64) {
        uint32_t lo[16], hi[16];
        tmem_ld16x256b_x4(taddr + c0, lo);
        tmem_ld16x256b_x4(taddr + (16u << 16) + c0, hi);
        // scale and output row of the chunk's rows, one lane each
        const int r = U.first + c0 + lane;
        float ga = gw;
        int to = -1;
        if (c0 + lane < U.rows) {
          if (p.a_gs && p.a_gs_per_row) ga *= __ldg(p.a_gs + r);
          to = r;
          if (p.out_rows) {
            to = __ldg(p.out_rows + r);
            if (to >= p.m) to = -1;
          }
        }
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = 8 * i + 2 * (lane & 3);
          const float g0 = __shfl_sync(0xffffffffu, ga, t), g1 = __shfl_sync(0xffffffffu, ga, t + 1);
          float v[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            v[j] = __uint_as_float(lo[4 * i + j]) * (j & 1 ? g1 : g0);
            v[4 + j] = __uint_as_float(hi[4 * i + j]) * (j & 1 ? g1 : g0);
          }
          if (staged) {
            stmatrix_x4_trans(st_addr + 8 * i * kEpiRow, pack16(p.out_dtype, v[0], v[1]), pack16(p.out_dtype, v[2], v[3]),
                              pack16(p.out_dtype, v[4], v[5]), pack16(p.out_dtype, v[6], v[7]));
          } else {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int o = __shfl_sync(0xffffffffu, to, t + j);
#pragma unroll
              for (int h = 0; h < 4; ++h) {
                const int n = n0 + 8 * h + (lane >> 2);
                if (o >= 0 && n < p.n) store_out(p, (int64_t)o * p.out_stride + n, v[2 * h + j]);
              }
            }
          }
        }
        if (staged) {
          __syncwarp();
          const int n = n0 + 8 * (lane & 3);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = 8 * i + (lane >> 2);
            const int o = __shfl_sync(0xffffffffu, to, row);
            const uint4 w = *reinterpret_cast<const uint4*>(stage + row * kEpiRow + 16 * (lane & 3));
            if (o >= 0 && n < p.n)
              *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p.out) + (int64_t)o * p.out_stride + n) = w;
          }
          __syncwarp();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty_acc[abuf]);
      ++acc_i;
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, C::kTmemCols);
}

template <int FMT, int NT>
cudaError_t launch(const Fp4GemmParams& p, int grid, bool pdl, cudaStream_t stream) {
  auto kern = fp4_gemm_kernel<FMT, NT>;
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

cudaError_t launch_fp4_gemm(const Fp4GemmParams& p, int fmt, int nt, int grid, bool pdl, cudaStream_t stream) {
  if (nt == 64) return fmt == 0 ? fp4::launch<0, 64>(p, grid, pdl, stream) : fp4::launch<1, 64>(p, grid, pdl, stream);
  return fmt == 0 ? fp4::launch<0, 192>(p, grid, pdl, stream) : fp4::launch<1, 192>(p, grid, pdl, stream);
}

}  // namespace b4
