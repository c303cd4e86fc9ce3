// Product of two FP8 operands with an fp32 scale per block of 128 along K, on tcgen05
// (sm_103a), dense and grouped by expert with ragged sizes:
//
//   out[t][n] = sum_b sa[t][b] sw[e][n / 128][b] sum_{k in block b} a[t][k] w[e][n][k]
//
// for the rows t of group e.  The block-scaled instructions take powers of two only, so a
// block of 128 along K is an accumulation of its own in tensor memory (four K = 32
// instructions of kind::f8f6f4), which the epilogue warps add to fp32 registers times the
// two scales, while the tensor core fills the next of four accumulators.
//
// Activation rows are on M (128 lanes of tensor memory): a lane's scale is one register for
// all of its columns, and the 128 weight rows on N share theirs.

#include "fp4_mma.cuh"
#include "fp8.cuh"

namespace b4 {

cudaError_t ensure_smem_limit(const void* func, size_t bytes);

namespace fp8 {

using namespace fp4;

constexpr int kRows8 = 128;                  // activation rows of a unit
constexpr int kAStage8 = kRows8 * 128;
constexpr int kSlots = 6;
constexpr int kAccs = 4;                     // accumulators of 128 columns
constexpr size_t kOffA = (size_t)kSlots * kWStage;
constexpr size_t kOffBars = kOffA + (size_t)kSlots * kAStage8;
constexpr int kNumBars8 = 2 * kSlots + 2 * kAccs + 1;
constexpr size_t kOffMisc = kOffBars + 8 * kNumBars8 + 8;
constexpr size_t smem_total(bool ragged) { return kOffMisc + 16 + (ragged ? sizeof(Groups) : 0); }

// Instruction descriptor of kind::f8f6f4: E4M3 operands, both K-major, fp32 accumulator.
__device__ __forceinline__ constexpr uint32_t idesc_fp8(uint32_t m, uint32_t n) {
  return (1u << 4) | ((n >> 3) << 17) | ((m >> 4) << 24);
}
__device__ __forceinline__ void mma_fp8(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, "
      "%5};\n\ttcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHiSw128)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void fma2(float2& acc, uint32_t a, uint32_t b, float s) {
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %4};\n\tmov.b64 z, {%0, %1};\n\t"
      "fma.rn.f32x2 z, x, y, z;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "+f"(acc.x), "+f"(acc.y)
      : "r"(a), "r"(b), "f"(s));
}

// A lane's scales of activation row `row`, four blocks at a time.
__device__ __forceinline__ float4 load_scales(const Fp8GemmParams& p, const float* row, int b, bool live) {
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (live && b < p.kb) {
    if (p.a_vec) return *reinterpret_cast<const float4*>(row + b);
    v.x = row[b];
    if (b + 1 < p.kb) v.y = row[b + 1];
    if (b + 2 < p.kb) v.z = row[b + 2];
    if (b + 3 < p.kb) v.w = row[b + 3];
  }
  return v;
}

// Columns [n, n + 2 C) of a row from registers.
template <int OUT, int C>
__device__ __forceinline__ void store_row(const Fp4GemmParams& g, int64_t at, int n, const float2 (&v)[C]) {
  if (OUT < 2 && g.vec && n + 2 * C <= g.n) {
    uint16_t* out = reinterpret_cast<uint16_t*>(g.out) + at + n;
#pragma unroll
    for (int i = 0; i < C / 4; ++i)
      reinterpret_cast<uint4*>(out)[i] = make_uint4(pack16<OUT & 1>(v[4 * i]), pack16<OUT & 1>(v[4 * i + 1]),
                                                    pack16<OUT & 1>(v[4 * i + 2]), pack16<OUT & 1>(v[4 * i + 3]));
  } else if (OUT == 2 && g.vec && n + 2 * C <= g.n) {
    float* out = reinterpret_cast<float*>(g.out) + at + n;
#pragma unroll
    for (int i = 0; i < C / 2; ++i)
      reinterpret_cast<float4*>(out)[i] = make_float4(v[2 * i].x, v[2 * i].y, v[2 * i + 1].x, v[2 * i + 1].y);
  } else {
#pragma unroll
    for (int i = 0; i < C; ++i) {
      if (n + 2 * i < g.n) store_out(g, at + n + 2 * i, v[i].x);
      if (n + 2 * i + 1 < g.n) store_out(g, at + n + 2 * i + 1, v[i].y);
    }
  }
}

template <int OUT, bool RAGGED>
__global__ void __launch_bounds__(kThreads, 1) fp8_gemm_kernel(const __grid_constant__ Fp8GemmParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Groups& groups = *reinterpret_cast<Groups*>(smem + kOffMisc + 16);  // ragged only
  uint8_t* s_a = smem + kOffA;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kOffBars);
  uint64_t* empty = full + kSlots;
  uint64_t* full_acc = empty + kSlots;
  uint64_t* empty_acc = full_acc + kAccs;
  uint64_t* drain = empty_acc + kAccs;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + kOffMisc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + kOffMisc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Fp4GemmParams& g = p.g;
  const Abort ab{g.status, s_abort};

  if (threadIdx.x == 0) {
    *s_abort = 0;
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < kAccs; ++i) {
      mbar_init(&full_acc[i], 1);
      mbar_init(&empty_acc[i], kEpiWarps);
    }
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(s_tmem, 512);
    tmem_relinquish();
  }
  pdl_wait();
  const int wtiles = cdiv(g.n, 128);
  if (RAGGED) build_groups<kRows8>(g, groups);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0) pdl_launch_dependents();
  const uint32_t tmem = *s_tmem;
  const int n_units = (RAGGED ? groups.tiles[g.groups] : g.groups * cdiv(g.m, kRows8)) * wtiles;

  if (warp == 0) {
    // ----------------------------------------------------------- copies
    uint32_t i = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < n_units && ok; u += gridDim.x) {
      const Unit U = get_unit<kRows8, RAGGED>(g, groups, wtiles, u);
      const int wrow = (int)warp_uniform(U.group) * g.n + (int)warp_uniform(U.wtile) * 128;
      const int first = (int)warp_uniform(U.first);
      for (int s = 0; s < p.kb; ++s, ++i) {
        const uint32_t slot = i % kSlots;
        ok = __all_sync(0xffffffffu, wait(&empty[slot], ((i / kSlots) & 1) ^ 1, ab, 121));
        if (!ok) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(&full[slot], kWStage + kAStage8);
          tma_load_2d(smem + slot * kWStage, &p.tmap_w, s * 128, wrow, &full[slot]);
          tma_load_2d(s_a + slot * kAStage8, &p.tmap_a, s * 128, first, &full[slot]);
        }
        __syncwarp();
      }
    }
    if (ab.raised() && lane == 0) {
      // let copies already issued land before the CTA's shared memory goes away
      const uint32_t n = i < (uint32_t)kSlots ? i : (uint32_t)kSlots;
      for (uint32_t j = i - n; j < i; ++j) {
        const unsigned long long t0 = globaltimer();
        while (!mbar_try_wait(&full[j % kSlots], (j / kSlots) & 1) && globaltimer() - t0 < kWaitLimitNs) {
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------- matrix instructions
    const uint32_t w_desc = desc_lo(smem_u32(smem)), a_desc = desc_lo(smem_u32(s_a));
    uint32_t i = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < n_units && ok; u += gridDim.x) {
      for (int s = 0; s < p.kb; ++s, ++i) {
        const uint32_t slot = i % kSlots, acc = i % kAccs;
        ok = __all_sync(0xffffffffu, wait(&empty_acc[acc], ((i / kAccs) & 1) ^ 1, ab, 122) &&
                                         wait(&full[slot], (i / kSlots) & 1, ab, 123));
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t wd = w_desc + slot * (kWStage / 16), ad = a_desc + slot * (kAStage8 / 16);
#pragma unroll
          for (int j = 0; j < 4; ++j) mma_fp8(tmem + acc * 128, ad + 2 * j, wd + 2 * j, idesc_fp8(128, 128), j > 0);
          mma_commit(&empty[slot]);
          mma_commit(&full_acc[acc]);
        }
        __syncwarp();
      }
    }
    // drain: every instruction issued has completed
    if (elect_one()) mma_commit(drain);
    const unsigned long long t0 = globaltimer();
    while (!mbar_try_wait(drain, 0) && globaltimer() - t0 < kWaitLimitNs) {
    }
    __syncwarp();
  } else if (warp < 4) {
    if (RAGGED && !g.out_rows) clear_tail(g, groups.first[g.groups], threadIdx.x - 64);
  } else {
    // ------------------------------------------- promotion and epilogue
    const int q4 = warp & 3, half = (warp - 4) >> 2;
    const int r = 32 * q4 + lane;
    const uint32_t taddr = tmem + ((uint32_t)(32 * q4) << 16) + 64 * half;
    uint32_t i = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < n_units && ok; u += gridDim.x) {
      const Unit U = get_unit<kRows8, RAGGED>(g, groups, wtiles, u);
      const bool mine = 32 * q4 < U.rows, live = r < U.rows;
      const float* sa = p.a_scales + (int64_t)(U.first + (live ? r : 0)) * p.kb;
      const float* sw = p.w_scales + ((int64_t)U.group * wtiles + U.wtile) * p.kb;
      float2 acc[32];
#pragma unroll
      for (int c = 0; c < 32; ++c) acc[c] = make_float2(0.f, 0.f);
      float4 now = load_scales(p, sa, 0, live), next = now;
      float ws = 0.f;
      for (int s = 0; s < p.kb; ++s, ++i) {
        if ((s & 31) == 0) ws = s + lane < p.kb ? __ldg(sw + s + lane) : 0.f;
        if ((s & 3) == 0) {
          if (s > 0) now = next;
          next = load_scales(p, sa, s + 4, live);
        }
        const float scale = ((s & 3) == 0 ? now.x : (s & 3) == 1 ? now.y : (s & 3) == 2 ? now.z : now.w) *
                            __shfl_sync(0xffffffffu, ws, s & 31);
        const uint32_t b = i % kAccs;
        ok = __all_sync(0xffffffffu, wait(&full_acc[b], (i / kAccs) & 1, ab, 124));
        if (!ok) break;
        tc_fence_after();
        uint32_t t[2][32];
        if (mine) {
          tmem_ld32(taddr + 128 * b, t[0]);
          tmem_ld32(taddr + 128 * b + 32, t[1]);
          tmem_ld_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty_acc[b]);
        if (mine) {
#pragma unroll
          for (int c = 0; c < 16; ++c) fma2(acc[c], t[0][2 * c], t[0][2 * c + 1], scale);
#pragma unroll
          for (int c = 0; c < 16; ++c) fma2(acc[16 + c], t[1][2 * c], t[1][2 * c + 1], scale);
        }
      }
      if (!ok || !live) continue;
      int to = U.first + r;
      if (g.out_rows) to = __ldg(g.out_rows + to);
      if (to >= 0 && to < g.out_rows_end) store_row<OUT>(g, (int64_t)to * g.out_stride, U.wtile * 128 + 64 * half, acc);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

template <int OUT, bool RAGGED>
cudaError_t launch(const Fp8GemmParams& p, int grid, cudaStream_t stream) {
  auto kern = fp8_gemm_kernel<OUT, RAGGED>;
  const size_t smem = smem_total(RAGGED);
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
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace fp8

cudaError_t launch_fp8_gemm(const Fp8GemmParams& p, int grid, cudaStream_t stream) {
  auto by_groups = [&](auto out) {
    constexpr int O = decltype(out)::value;
    return p.g.offsets ? fp8::launch<O, true>(p, grid, stream) : fp8::launch<O, false>(p, grid, stream);
  };
  return p.g.out_dtype == 0   ? by_groups(std::integral_constant<int, 0>{})
         : p.g.out_dtype == 1 ? by_groups(std::integral_constant<int, 1>{})
                              : by_groups(std::integral_constant<int, 2>{});
}

}  // namespace b4
