// Device code shared by the FP4 x FP4 product kernels: block-scaled matrix
// instructions, scale copies, the tables of ragged groups, units of work and
// the epilogue.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "fp4.cuh"
#include "fp4_ptx.cuh"

namespace b4 {
namespace fp4 {

constexpr int kThreads = 384;
constexpr int kEpiWarps = 8;                 // two per quarter of the lanes, alternating 32-column chunks
constexpr int kEpiRow = 80;                  // staged 64-byte row, padded so that eight rows hit eight bank groups
constexpr int kEpiBytes = kEpiWarps * 32 * kEpiRow;
constexpr int kWStage = 128 * 128;           // weight codes of a stage: 128 rows x 256 K
constexpr int kMaxGroups = 1024;

__host__ __device__ constexpr int sf_tiles(int fmt) { return fmt == 0 ? 4 : 2; }  // scale tiles of a stage (per 128 rows)

// Instruction descriptor of the block-scaled kinds: E2M1 operands, both
// K-major, scales E4M3 (0) or E8M0 (1); bits 4 and 29 take the byte of a scale
// word that the instruction starts at.
__device__ __forceinline__ uint32_t idesc_fp4(int fmt, uint32_t m, uint32_t n) {
  return (1u << 7)               // A: E2M1
         | (1u << 10)            // B: E2M1
         | ((n >> 3) << 17)      // N >> 3
         | ((uint32_t)fmt << 23) // scale type
         | ((m >> 4) << 24);     // M >> 4
}

// Shared-memory descriptors as the low word (address >> 4 and the leading
// offset) and a constant high word: offsets are then 32-bit additions.
constexpr uint32_t kDescHiSw128 = (1024 >> 4) | (1u << 14) | (2u << 29);  // 8-row atoms of 1024 bytes, 128-byte swizzle
constexpr uint32_t kDescHiTile = (128 >> 4) | (1u << 14);                 // 8-row core matrices of 128 bytes
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr) { return (saddr >> 4) | (1u << 16); }

// D (+)= A B^T with block scales from tensor memory; CG CTAs of a pair.
template <int FMT, int CG>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                        uint32_t accumulate) {
#define FP4_MMA(kind)                                                                                              \
  asm volatile(                                                                                                    \
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %6, 0;\n\tmov.b64 x, {%1, %7};\n\tmov.b64 y, {%2, " \
      "%7};\n\t" kind " [%0], x, y, %3, [%4], [%5], p;\n\t}" ::"r"(d),                                             \
      "r"(a), "r"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate), "n"(kDescHiSw128)                           \
      : "memory")
  if constexpr (FMT == 0 && CG == 1) FP4_MMA("tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X");
  if constexpr (FMT == 1 && CG == 1) FP4_MMA("tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X");
  if constexpr (FMT == 0 && CG == 2) FP4_MMA("tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X");
  if constexpr (FMT == 1 && CG == 2) FP4_MMA("tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X");
#undef FP4_MMA
}

// One 512-byte scale tile (32 rows of 16 bytes) into four columns of tensor
// memory, the same in all four lane quarters (of both CTAs of a pair, each from
// its own shared memory).
template <int CG>
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t lo) {
  if constexpr (CG == 1)
    asm volatile("{\n\t.reg .b64 x;\n\tmov.b64 x, {%1, %2};\n\ttcgen05.cp.cta_group::1.32x128b.warpx4 [%0], x;\n\t}" ::"r"(taddr),
                 "r"(lo), "n"(kDescHiTile)
                 : "memory");
  else
    asm volatile("{\n\t.reg .b64 x;\n\tmov.b64 x, {%1, %2};\n\ttcgen05.cp.cta_group::2.32x128b.warpx4 [%0], x;\n\t}" ::"r"(taddr),
                 "r"(lo), "n"(kDescHiTile)
                 : "memory");
}

// mbar_wait with the waiting itself out of line: the kernels' loops stay small
// (see store_chunk on the instruction cache).
__device__ __noinline__ static bool wait_long(uint64_t* bar, uint32_t parity, uint32_t* status, volatile int* flag,
                                              uint32_t where) {
  return mbar_wait(bar, parity, Abort{status, flag}, where);
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, const Abort& ab, uint32_t where) {
  return mbar_test(bar, parity) || wait_long(bar, parity, ab.status, ab.flag, where);
}

// As wait, for a barrier that other CTAs' asynchronous stores complete.
__device__ __forceinline__ bool wait_cluster(uint64_t* bar, uint32_t parity, const Abort& ab, uint32_t where) {
  const bool ok = wait(bar, parity, ab, where);
  asm volatile("fence.acq_rel.cluster;" ::: "memory");
  return ok;
}
__device__ __forceinline__ void add4(uint32_t* v, const float4& x) {
  v[0] = __float_as_uint(__uint_as_float(v[0]) + x.x);
  v[1] = __float_as_uint(__uint_as_float(v[1]) + x.y);
  v[2] = __float_as_uint(__uint_as_float(v[2]) + x.z);
  v[3] = __float_as_uint(__uint_as_float(v[3]) + x.w);
}

// ------------------------------------------------------------------ units
struct Unit {
  int group, wtile, first, rows;  // first: packed row; rows: live rows
  int atile;                      // scale tile of row `first`
  int shift;                      // 32-row groups of that tile before `first`
};

// Tables of ragged groups in shared memory: first packed row, and activation
// tiles of NT rows before the group.
struct Groups {
  int first[kMaxGroups + 1];
  int tiles[kMaxGroups + 1];
  int warp[kThreads / 32];
};

// A block scan of the groups' tile counts, four groups a thread; ends with the
// tables written but not yet synchronised.
template <int NT>
__device__ __forceinline__ void build_groups(const Fp4GemmParams& p, Groups& g) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int cnt[4], sum = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = 4 * threadIdx.x + i;
    cnt[i] = 0;
    if (e <= p.groups) {
      const int lo = min(max(__ldg(p.offsets + e), 0), p.m);
      g.first[e] = lo;
      if (e < p.groups) cnt[i] = cdiv(max(min(__ldg(p.offsets + e + 1), p.m) - lo, 0), NT);
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
    if (e <= p.groups) g.tiles[e] = before;
    before += cnt[i];
  }
}

// Unit u: weight rows outermost within a group, so that neighbouring units
// read the same weights.  wtiles: weight units of a group.  The search is out of
// line, one copy for all of a kernel's loops (unrolled over their rings): returns
// group, weight unit << 1 | half, first packed row, and rows | token tile << 9.
// Dense units of 256 rows from halves_from on are two units of 128 each.
// Ragged units of 256 rows are taken from each third of them in turn: units of large groups
// are bound by the way into shared memory, those of small groups by the stream of weights from
// DRAM, and the two mix better than they follow one another (8 groups of 1100 rows and 56 of
// 60, N = 2816, K = 2048: 57.4 us where the large ones are neighbours, in order 60.8; in a random
// order 58.0 and 57.7).
constexpr int kMix = 3;
template <int NT, bool RAGGED>
__device__ __noinline__ static int4 find_unit(int groups, int m, const Groups* g, int wtiles, int u, int halves_from) {
  int lo, t, nt, first, rows, half = -1;
  if (!RAGGED && NT == 256 && u >= halves_from) {
    half = (u - halves_from) & 1;
    u = halves_from + ((u - halves_from) >> 1);
  }
  if constexpr (RAGGED) {
    if (NT == 256) {
      const int run = (g->tiles[groups] * wtiles) / kMix;
      if (u < run * kMix) u = u % kMix * run + u / kMix;
    }
    lo = 0;
    int hi = groups - 1;  // last group whose tiles start at or before the unit's
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((long long)g->tiles[mid] * wtiles <= u) lo = mid;
      else hi = mid - 1;
    }
    nt = g->tiles[lo + 1] - g->tiles[lo];
    u -= g->tiles[lo] * wtiles;
  } else {
    nt = cdiv(m, NT);
    lo = groups == 1 ? 0 : u / (nt * wtiles);
    u -= lo * nt * wtiles;
  }
  const int wtile = nt == 1 ? u : u / nt;
  t = u - wtile * nt;
  if constexpr (RAGGED) {
    first = g->first[lo] + t * NT;
    rows = min(NT, g->first[lo + 1] - first);
  } else {
    first = lo * m + t * NT;
    rows = min(NT, m - t * NT);
    if (half >= 0) {
      first += 128 * half;
      rows = min(128, rows - 128 * half);
    }
  }
  return make_int4(lo, 2 * wtile + max(half, 0), first, rows | t << 9);
}
template <int NT, bool RAGGED>
__device__ __forceinline__ Unit get_unit(const Fp4GemmParams& p, const Groups& g, int wtiles, int u) {
  const int4 v = find_unit<NT, RAGGED>(p.groups, p.m, &g, wtiles, u, p.halves_from);
  const int t = v.w >> 9;
  Unit U;
  U.group = v.x;
  U.wtile = v.y >> 1;
  U.first = v.z;
  U.rows = v.w & 511;
  U.atile = (RAGGED ? (v.z - t * NT) / 128 + v.x : v.x * cdiv(p.m, 128)) + t * NT / 128 + (v.y & 1);
  U.shift = (t * NT & 127) >> 5;
  return U;
}

// Rows of a ragged output past the last group are zero: THREADS threads.
template <int THREADS = 64>
__device__ __forceinline__ void clear_tail(const Fp4GemmParams& p, int live, int thread) {
  const int width = p.out_dtype == 2 ? 4 : 2;
  for (int r = live + blockIdx.x; r < p.m; r += gridDim.x) {
    uint8_t* row = reinterpret_cast<uint8_t*>(p.out) + (int64_t)r * p.out_stride * width;
    if (p.vec) {
      for (int c = thread; c < p.n * width / 16; c += THREADS) reinterpret_cast<uint4*>(row)[c] = make_uint4(0, 0, 0, 0);
    } else {
      for (int c = thread; c < p.n; c += THREADS) {
        if (width == 4) reinterpret_cast<uint32_t*>(row)[c] = 0;
        else reinterpret_cast<uint16_t*>(row)[c] = 0;
      }
    }
  }
}

// --------------------------------------------------------------- epilogue
__device__ __forceinline__ void store_out(const Fp4GemmParams& p, int64_t at, float v) {
  if (p.out_dtype == 0) reinterpret_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(v);
  else if (p.out_dtype == 1) reinterpret_cast<__half*>(p.out)[at] = __float2half_rn(v);
  else reinterpret_cast<float*>(p.out)[at] = v;
}

// Two accumulators times their rows' scales, in one instruction.
__device__ __forceinline__ float2 times2(uint32_t a, uint32_t b, float2 g) {
  float2 r;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(a), "r"(b), "f"(g.x), "f"(g.y));
  return r;
}

template <int DT>
__device__ __forceinline__ uint32_t pack16(float2 v2) {
  const float lo = v2.x, hi = v2.y;
  if constexpr (DT == 0) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}

// What the epilogue needs to know of a unit, two units deep in shared memory:
// warps 2 and 3 look it up ahead, since under the operands' traffic a load from
// L2 takes some 3000 cycles, as long as half a unit's stores.
template <int NT>
struct RowTable {
  float g[2][NT];   // scale of each activation row, the weights' included
  int to[2][NT];    // its output row, or -1
  int rows[2], wtile[2];
};
struct RowInfo {  // of 32 rows of the table
  const float* g;
  const int* to;
};

template <int NT, bool RAGGED>
__device__ __forceinline__ void fill_rows(const Fp4GemmParams& p, const Groups& groups, RowTable<NT>& tab, uint64_t* full,
                                          uint64_t* empty, int wunits, int u0, int du, int n_units, const Abort& ab) {
  const int thread = threadIdx.x - 64, lane = threadIdx.x & 31;
  uint32_t i = 0;
  for (int u = u0; u < n_units; u += du, ++i) {
    const uint32_t b = i & 1;
    if (!__all_sync(0xffffffffu, wait(&empty[b], ((i >> 1) & 1) ^ 1, ab, 106))) break;
    const Unit U = get_unit<NT, RAGGED>(p, groups, wunits, u);
    const float gw = (p.w_gs ? __ldg(p.w_gs + U.group) : 1.f) *
                     (p.a_gs && !p.a_gs_per_row ? __ldg(p.a_gs + U.group) : 1.f);
    for (int r = thread; r < NT; r += 64) {
      float g = gw;
      int to = -1;
      if (r < U.rows) {
        const int at = U.first + r;
        if (p.a_gs && p.a_gs_per_row) g *= __ldg(p.a_gs + at);
        to = at;
        if (p.out_rows) {
          to = __ldg(p.out_rows + at);
          if (to >= p.out_rows_end) to = -1;
        }
      }
      tab.g[b][r] = g;
      tab.to[b][r] = to;
    }
    if (thread == 0) {
      tab.rows[b] = U.rows;
      tab.wtile[b] = U.wtile;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&full[b]);
  }
}

// A chunk of 32 activation rows x 32 weight rows (from n0) out of fragments of
// 8 x 8 (weight row x activation row; lo: weight rows 0 .. 15, hi: 16 .. 31):
// scaled, rounded, and through a transposing store to the warp's staging area,
// so that it leaves as 16-byte pieces of output rows (64 bytes a row and warp).
template <int DT>
__device__ __forceinline__ void store_staged(const Fp4GemmParams& p, const uint32_t (&lo)[16], const uint32_t (&hi)[16],
                                             const RowInfo& info, int n0, uint8_t* stage, int lane) {
  uint32_t h[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = 8 * i + 2 * (lane & 3);
    const float2 g = *reinterpret_cast<const float2*>(info.g + t);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      h[i][j] = pack16<DT>(times2(lo[4 * i + 2 * j], lo[4 * i + 2 * j + 1], g));
      h[i][2 + j] = pack16<DT>(times2(hi[4 * i + 2 * j], hi[4 * i + 2 * j + 1], g));
    }
  }
  const uint32_t st_addr = smem_u32(stage) + (lane & 7) * kEpiRow + (lane >> 3) * 16;
#pragma unroll
  for (int i = 0; i < 4; ++i) stmatrix_x4_trans(st_addr + 8 * i * kEpiRow, h[i][0], h[i][1], h[i][2], h[i][3]);
  __syncwarp();
  const int n = n0 + 8 * (lane & 3);
  uint16_t* out = reinterpret_cast<uint16_t*>(p.out) + n;
  const uint8_t* src = stage + (lane >> 2) * kEpiRow + 16 * (lane & 3);
  uint4 w[4];
  int o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = *reinterpret_cast<const uint4*>(src + 8 * i * kEpiRow);
    o[i] = info.to[8 * i + (lane >> 2)];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (o[i] >= 0 && n < p.n) *reinterpret_cast<uint4*>(out + (int64_t)o[i] * p.out_stride) = w[i];
  __syncwarp();
}

// The same chunk straight from the fragments, for outputs that are not 16-bit
// or not 16-byte aligned.
__device__ __forceinline__ void store_direct(const Fp4GemmParams& p, const uint32_t (&lo)[16], const uint32_t (&hi)[16],
                                          const RowInfo& info, int n0, int lane) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int t = 8 * i + 2 * (lane & 3) + j;
      const float g = info.g[t];
      const int o = info.to[t];
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const int n = n0 + 8 * h + (lane >> 2);
        const uint32_t v = h < 2 ? lo[4 * i + 2 * h + j] : hi[4 * i + 2 * (h - 2) + j];
        if (o >= 0 && n < p.n) store_out(p, (int64_t)o * p.out_stride + n, __uint_as_float(v) * g);
      }
    }
}

// OUT: 0 bf16, 1 f16, both in 16-byte pieces; 2: any type, straight.  (A kernel
// holds one form: with all three in it, the epilogue's code alone slowed the
// issuing warps through the instruction cache, 29 -> 33 us at 4096^3.)
template <int OUT>
__device__ __forceinline__ void store_chunk(const Fp4GemmParams& p, const uint32_t (&lo)[16], const uint32_t (&hi)[16],
                                            const RowInfo& info, int n0, uint8_t* stage, int lane) {
  if constexpr (OUT == 2) store_direct(p, lo, hi, info, n0, lane);
  else store_staged<OUT>(p, lo, hi, info, n0, stage, lane);
}

// Calls f with a kernel's forms as compile-time values: format, output, ragged.
template <typename F>
cudaError_t with_forms(const Fp4GemmParams& p, int fmt, F f) {
  auto by_out = [&](auto fm) {
    auto by_groups = [&](auto out) {
      return p.offsets ? f(fm, out, std::true_type{}) : f(fm, out, std::false_type{});
    };
    const int form = p.vec ? p.out_dtype : 2;
    return form == 0   ? by_groups(std::integral_constant<int, 0>{})
           : form == 1 ? by_groups(std::integral_constant<int, 1>{})
                       : by_groups(std::integral_constant<int, 2>{});
  };
  return fmt == 0 ? by_out(std::integral_constant<int, 0>{}) : by_out(std::integral_constant<int, 1>{});
}

}  // namespace fp4
}  // namespace b4
