// Block-scaled FP4 quantisation of activation and weight rows (NVFP4: E2M1
// codes, an E4M3 scale per 16 elements, fp32 global scales; MXFP4: an E8M0
// scale per 32), with the product's prologue folded in: rows gathered through
// an index, a SwiGLU / clamped swiglu / ReLU^2 of the row, the row's own global
// scale.
//
//   NVFP4  s = e4m3(amax_block / (6 gs)),  d = s gs,  c = e2m1(h / d), 0 where d = 0
//   MXFP4  s = 2^j, j the least with amax_block <= 6 2^j,  c = e2m1(h / s)
//   gs     per row: 2^j, j >= -126 the least with amax_row <= 6 448 2^j: a power
//          of two costs E4M3 scales no precision and makes d exact, so ties are
//          the true ties; per matrix: amax / (6 448).
//
// A thread holds chunks of 16 consecutive elements: an NVFP4 block, half an
// MXFP4 block (the pair joins by one shuffle).  Threads of a row stand side by
// side, so a chunk is one 32-byte load of a contiguous stretch (two of fp32) and
// its codes one 8-byte store; a thread loads all of its chunks (cached_chunks)
// before it uses any, and keeps them between the row's maximum and its codes
// (longer rows are read again, from L1).  Every step is fp32 in the order of
// the formula, rounded to nearest, but for the quotients amax / (6 gs) and h / d: h / d is
// h y + h z in one fused multiply-add, y an approximate reciprocal of d and z what it
// lacks (z = (1 - y d) y, the residual exact): the quotient to 46 bits before its one
// rounding, so every tie of the codes is met where d is exact, in two operations an
// element, two elements an instruction, where a division costs a dozen.
//
// Bound by DRAM where rows are many, but for the gated prologue: 16384 rows of 4096
// bf16, per matrix (given) 29.1 us, 5.9 TB/s, by row 31.7 us, as MXFP4 26.9 us, 6.3 TB/s;
// by the ramp of one wave below (4096 rows 10.8 us, 512 rows 2.9 us, one row 2.2 us).
// Behind SwiGLU by the issue of instructions: 12288 rows of 1408 23.8 us, 3.3 TB/s, at 37
// instructions an element, 0.71 a cycle and scheduler (DRAM 34 % busy, the pipe of the two
// transcendental operations 19 to 26 %), 6.7 warps a scheduler of which 1.75 are ready: a
// block has one row, and nothing of the next is in flight while it waits for its loads.

#include <algorithm>

#include "fp4_quant.cuh"

namespace b4 {

using namespace fp4q;

namespace {

constexpr int kQThreads = 128;  // small blocks: their load and compute phases interleave on an SM

// Group of row r of a ragged operand: the warp counts the offsets at or below
// r, 32 at a time (two rounds for up to 1024 groups).  All lanes of the warp
// ask for the same row.
__device__ __forceinline__ int find_group(const int32_t* offsets, int groups, int r, int lane) {
  const int step = (groups + 31) / 32;
  const int i = min((lane + 1) * step, groups);
  const int coarse = __popc(__ballot_sync(0xffffffffu, __ldg(offsets + i) <= r && (lane + 1) * step < groups));
  const int j = coarse * step + lane + 1;
  const int fine = __popc(__ballot_sync(0xffffffffu, lane < step - 1 && j < groups && __ldg(offsets + min(j, groups)) <= r));
  return min(coarse * step + fine, groups - 1);
}

// What codes of step d stand for, in x's type (NaN under a NaN scale).
template <typename T>
__device__ __forceinline__ void store_values(T* dst, int level, const uint2& w, float d, bool is_nan) {
  T e[16];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t byte = ((j < 4 ? w.x : w.y) >> (8 * (j & 3))) & 0xffu;
    const float2 v = __half22float2(__half2(__nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)byte, __NV_E2M1)));
    from_f32(&e[2 * j], is_nan ? __uint_as_float(0x7fffffffu) : __fmul_rn(v.x, d));
    from_f32(&e[2 * j + 1], is_nan ? __uint_as_float(0x7fffffffu) : __fmul_rn(v.y, d));
  }
  uint32_t o[16 * sizeof(T) / 4];
  memcpy(o, e, sizeof(o));
  store_words(dst, level, o);
}

// Chunks a thread keeps, and resident blocks asked of the compiler: 4096 rows of 4096
// bf16 10.8 us (11.1 with seven blocks, 13.4 with two chunks and ten); 16384 such rows of
// fp32 56.6 us (58.4 with eight blocks, 68 with five); 2048 SwiGLU rows of 1408 5.0 us (5.3
// with two chunks and seven blocks, 5.5 with ten blocks).
template <typename T, bool ACT>
__host__ __device__ constexpr int cached_chunks() {
  return ACT ? 1 : sizeof(T) == 2 ? 4 : 2;
}
template <typename T, bool ACT>
__host__ __device__ constexpr int resident_blocks() {
  return sizeof(T) == 2 || ACT ? 8 : 7;
}

}  // namespace

// shape: threads per row, as their logarithm, or behind an activation their number: a power
// of two up to 32, or the whole block.  Rows beyond the operand (pad_rows) only clear
// their scales.
template <typename T, int FMT, bool ACT, bool ROW, bool VALUES>
__global__ void __launch_bounds__(kQThreads, resident_blocks<T, ACT>()) fp4_quantize_kernel(const __grid_constant__ Fp4QuantParams p,
                                                                 int shape) {
  constexpr int kCached = cached_chunks<T, ACT>();
  constexpr int kPerTile = FMT == 0 ? 4 : 8;  // chunks of a scale tile
  __shared__ uint32_t s_max[kQThreads / 32];
  const int tpr = ACT ? shape : 1 << shape;
  const int t = ACT && tpr > 32 ? threadIdx.x : threadIdx.x & (tpr - 1);
  const int lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  if (p.status && blockIdx.x == 0 && threadIdx.x < 2) p.status[threadIdx.x] = 0;

  // this thread's row: packed index (codes, gs, values), scale tile and row in it
  const uint32_t block = p.gs_mode == kGsTensor ? gridDim.x - 1 - blockIdx.x : blockIdx.x;
  const int64_t vrow = ACT ? tpr > 32 ? block : ((int64_t)block * blockDim.x + threadIdx.x) >> (31 - __clz(tpr))
                           : (int64_t)block * (blockDim.x >> shape) + (threadIdx.x >> shape);
  const int tiles_per = cdiv(p.m, 128);
  bool live = false, pad = false;
  int64_t row = 0, tile = 0;
  int lr = 0, group = 0;
  if (p.offsets) {  // ragged: tpr >= 32, so a warp holds one row
    const int total = min(max(__ldg(p.offsets + p.groups), 0), p.m);
    group = find_group(p.offsets, p.groups, (int)min(vrow, (int64_t)p.m), lane);
    const int first = __ldg(p.offsets + group);
    row = vrow;
    lr = (int)(vrow - first);
    tile = (int64_t)(first / 128) + group + lr / 128;
    live = vrow < total && first >= 0 && lr >= 0 && tile < (int64_t)p.m / 128 + p.groups;
  } else {
    const int per = p.pad_rows ? tiles_per * 128 : p.m;
    if (p.groups == 1) {
      lr = (int)vrow;
      group = vrow < per ? 0 : 1;
    } else {
      group = (int)(vrow / per);
      lr = (int)(vrow - (int64_t)group * per);
    }
    live = group < p.groups && lr < p.m;
    pad = group < p.groups && lr >= p.m;
    row = (int64_t)group * p.m + lr;
    tile = (int64_t)group * tiles_per + lr / 128;
  }
  int64_t src = row;
  bool zero = false;
  if (p.rows && live) {
    const int r = __ldg(p.rows + row);
    src = r < 0 ? -1 : r / p.row_div;
    zero = src < 0 || (p.x_rows > 0 && src >= p.x_rows);
  }
  const T* x = reinterpret_cast<const T*>(p.x) + (zero ? 0 : src * p.x_stride);
  const int chunks = live ? p.k / 16 : 0;
  const int filled = zero ? 0 : chunks;  // chunks with anything to read
  const int n_it = cdiv(p.k_tiles * kPerTile, tpr);

  Chunk<T, ACT> h[kCached];
#pragma unroll
  for (int it = 0; it < kCached; ++it) {
    const int c = it * tpr + t;
    if (c < filled) h[it].get(p, x, c);
    else h[it].zero();
  }
  uint32_t amax[kCached];
#pragma unroll
  for (int it = 0; it < kCached; ++it) amax[it] = h[it].amax();
  float gs = 1.f;
  if constexpr (ROW) {
    uint32_t a = amax[0];
#pragma unroll
    for (int it = 1; it < kCached; ++it) a = max(a, amax[it]);
    for (int it = kCached; it < n_it; ++it) {
      const int c = it * tpr + t;
      if (c < filled) {
        Chunk<T, ACT> v;
        v.get(p, x, c);
        a = max(a, v.amax());
      }
    }
    for (int o = min(tpr, 32) / 2; o > 0; o >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
    if (tpr > 32) {
      if (lane == 0) s_max[threadIdx.x >> 5] = a;
      __syncthreads();
      const int w0 = ACT ? 0 : (threadIdx.x >> shape) << (shape - 5);
      for (int w = 0; w < (tpr >> 5); ++w) a = max(a, s_max[w0 + w]);
    }
    gs = row_gs(a);
    if (live && t == 0) p.gs[row] = gs;
  } else if (FMT == 0 && live) {
    gs = __ldg(p.gs + group);
  }
  const RowScale rs(gs);

  // this thread's first chunk in each output, and the way to its next one; the
  // scale of block b is at [row][b] or, tiled, in byte b % 4 of the row's word of
  // tile b / 4 (an MXFP4 block's even chunk stores it)
  uint8_t* codes = p.codes + row * p.ld + 8 * t;
  T* values = VALUES ? reinterpret_cast<T*>(p.values) + row * p.k + 16 * t : nullptr;
  const int blk = FMT == 0 ? t : t >> 1, blk_step = FMT == 0 ? tpr : tpr >> 1;
  uint8_t* scales;
  int scale_step, scale_chunks;  // chunks that have a scale to store
  if (p.rowmajor_scales) {
    scales = p.scales + row * (p.k / (FMT == 0 ? 16 : 32)) + blk;
    scale_step = blk_step;
    scale_chunks = chunks;
  } else {
    scales = p.scales + (tile * p.k_tiles + (blk >> 2)) * kSfTile + (lr & 31) * 16 + ((lr >> 5) & 3) * 4 + (blk & 3);
    scale_step = (blk_step >> 2) * kSfTile;
    scale_chunks = live || pad ? p.k_tiles * kPerTile : 0;
  }
  if (FMT != 0 && (t & 1)) scale_chunks = 0;

  auto emit = [&](int it, const Chunk<T, ACT>& v, uint32_t a) {
    const int c = it * tpr + t;
    if (FMT != 0) a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
    Quantized q = quantize_block<FMT>(v, a, rs);
    if (c < chunks) {
      *reinterpret_cast<uint2*>(codes + (int64_t)it * (8 * tpr)) = q.w;
      if constexpr (VALUES)
        store_values(values + (int64_t)it * (16 * tpr), p.values_vec, q.w, q.d, q.code == (FMT == 0 ? 0x7fu : 255u));
    } else {
      q.code = 0;
    }
    if (c < scale_chunks) scales[(int64_t)it * scale_step] = (uint8_t)q.code;
  };
#pragma unroll
  for (int it = 0; it < kCached; ++it)
    if (it < n_it) emit(it, h[it], amax[it]);
  for (int it = kCached; it < n_it; ++it) {
    const int c = it * tpr + t;
    Chunk<T, ACT> v;
    if (c < filled) v.get(p, x, c);
    else v.zero();
    emit(it, v, v.amax());
  }
}

// ------------------------------------------- one global scale per matrix
// Largest magnitude of each matrix of a stack, as fp32 bits (order of the
// atomics does not matter to a maximum), then amax / (6 448) in place.  Blocks
// take the matrices in order and the quantiser takes them from the end, so that what
// the cache still holds is read from there: 16 fp32 matrices of 2816 x 2048 with their
// values 180 us for 182 (both passes move 6.4 TB/s).
constexpr int kAmaxChunks = 8;  // of a thread
template <typename T, bool ACT>
__global__ void __launch_bounds__(kQThreads) fp4_amax_kernel(const __grid_constant__ Fp4QuantParams p) {
  __shared__ uint32_t s_max[kQThreads / 32];
  const int group = blockIdx.y;
  const uint32_t per_row = p.k / 16;
  const int64_t n = (int64_t)p.m * per_row;
  const T* x = reinterpret_cast<const T*>(p.x) + (int64_t)group * p.m * p.x_stride;
  uint32_t a = 0;
  for (int64_t b = (int64_t)blockIdx.x * (kQThreads * kAmaxChunks); b < n; b += (int64_t)gridDim.x * (kQThreads * kAmaxChunks)) {
    // the block's first chunk by a division, the others from there
    const int64_t r0 = b / per_row;
    const uint32_t c0 = (uint32_t)(b - r0 * per_row);
#pragma unroll
    for (int it = 0; it < kAmaxChunks; ++it) {
      const uint32_t j = c0 + it * kQThreads + threadIdx.x;
      const uint32_t r = j / per_row;
      if (b + it * kQThreads + threadIdx.x < n) {
        Chunk<T, ACT> h;
        h.get(p, x + (r0 + r) * p.x_stride, (int)(j - r * per_row));
        a = max(a, h.amax());
      }
    }
  }
  for (int o = 16; o > 0; o >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = a;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kQThreads / 32; ++w) a = max(a, s_max[w]);
    atomicMax(reinterpret_cast<uint32_t*>(p.gs) + group, a);
  }
}

__global__ void fp4_gs_kernel(float* gs, int groups) {
  pdl_wait();
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= groups) return;
  const float a = gs[i];
  gs[i] = a == 0.f ? 1.f : __fdiv_rn(a, 2688.f);
}

// -------------------------------------------- row-major scales -> tiles
__global__ void __launch_bounds__(256) fp4_tile_scales_kernel(const uint8_t* src, uint8_t* dst, int groups, int m,
                                                              int blocks, int k_tiles) {
  const int64_t tiles = cdiv(m, 128);
  const int64_t n = groups * tiles * k_tiles * 128;  // one word of four scales each
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int word = (int)(i & 127);
    const int64_t tk = i >> 7;
    const int kt = (int)(tk % k_tiles);
    const int64_t gt = tk / k_tiles;
    const int64_t g = gt / tiles;
    const int lr = (int)(gt - g * tiles) * 128 + (word & 3) * 32 + (word >> 2);
    uint32_t w = 0;
    if (lr < m)
      for (int j = 0; j < 4; ++j)
        if (kt * 4 + j < blocks) w |= (uint32_t)__ldg(src + (g * m + lr) * blocks + kt * 4 + j) << (8 * j);
    reinterpret_cast<uint32_t*>(dst)[i] = w;
  }
}

// ------------------------------------------------------ weighted combine
// out[t] = bf16(sum_j w[t, j] y[t top_k + j]) over the valid routes, j
// ascending in fp32: no atomics, so the same call gives the same bits.
__global__ void __launch_bounds__(256) fp4_combine_kernel(const __grid_constant__ Fp4CombineParams p) {
  __shared__ float s_w[32];
  __shared__ uint32_t s_valid;
  const int t = blockIdx.x;
  if (threadIdx.x < 32) {
    const int j = threadIdx.x;
    int l = -1;
    float w = 0.f;
    if (j < p.top_k) {
      const int id = __ldg(p.topk_ids + (int64_t)t * p.top_k + j);
      if (id >= 0 && id < p.num_global_experts) l = p.expert_map ? __ldg(p.expert_map + id) : id;
      w = __ldg(p.topk_weights + (int64_t)t * p.top_k + j);
    }
    s_w[j] = w;
    const uint32_t v = __ballot_sync(0xffffffffu, l >= 0 && l < p.num_local_experts);
    if (j == 0) s_valid = v;
  }
  pdl_wait();
  __syncthreads();
  const uint32_t valid = s_valid;
  for (int c = threadIdx.x + blockIdx.y * 256; c < p.hidden / 8; c += 256 * gridDim.y) {
    float acc[8] = {};
    for (uint32_t left = valid; left; left &= left - 1) {
      const int j = __ffs(left) - 1;
      const uint4 v = *reinterpret_cast<const uint4*>(p.y + ((int64_t)t * p.top_k + j) * p.hidden + 8 * (int64_t)c);
      const float w = s_w[j];
      const uint32_t r[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[2 * i] += w * __uint_as_float(r[i] << 16);
        acc[2 * i + 1] += w * __uint_as_float(r[i] & 0xffff0000u);
      }
    }
    __align__(16) __nv_bfloat16 o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = __float2bfloat16_rn(acc[i]);
    *reinterpret_cast<uint4*>(p.out + (int64_t)t * p.hidden + 8 * (int64_t)c) = *reinterpret_cast<const uint4*>(o);
  }
}

// ----------------------------------------------------- host-side launchers
namespace {

template <typename K, typename... A>
cudaError_t launch_pdl(K kern, dim3 grid, dim3 block, size_t smem, bool pdl, cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <typename T, int FMT, bool ACT>
cudaError_t quantize_t(const Fp4QuantParams& p, int num_sms, bool pdl, cudaStream_t stream) {
  // Threads per row: as many as it takes for a thread to hold its share, and
  // while all rows together are a few chunks for every SM's threads, down to one
  // chunk each; at least a warp for ragged rows (the whole warp finds their group)
  // and eight for a scale word.  Shares of four from 512 chunks an SM on (2048 bf16 rows of
  // 2048 3.5 us, single chunks 5.4; 768 of 4096 3.3, 4.0; 384 of 4096 3.0, 2.8).
  const int slots = p.k_tiles * (FMT == 0 ? 4 : 8);
  const int64_t rows = p.offsets ? p.m : (int64_t)p.groups * (p.pad_rows ? cdiv(p.m, 128) * 128 : p.m);
  const int64_t live = p.offsets ? p.m : (int64_t)p.groups * p.m;
  const int share = live * slots <= (int64_t)num_sms * 512 ? 1 : cached_chunks<T, ACT>();
  int lg = p.offsets ? 5 : 3;
  while ((1 << lg) < kQThreads && (1 << lg) * share < slots) ++lg;
  // a block of its own for a row of two warps: 16384 rows of 4096 31.7 us, two in a block 32.8
  // (rows of one warp the other way round: 12288 of 2048 11.7 us, in blocks of two 12.0)
  int shape = lg, rows_per = 1, threads = share > 1 && lg == 6 ? 64 : kQThreads;
  if (ACT) {
    // and for every row of several warps behind an activation, of no more warps than it
    // fills: 12288 SwiGLU rows of 1408 23.7 us, on 128 threads each 27.1
    shape = lg > 5 && slots < kQThreads ? round_up(slots, 32) : 1 << lg;
    threads = lg > 5 ? shape : kQThreads;
    rows_per = threads / shape;
  } else {
    rows_per = threads >> lg;
  }
  const int64_t grid = (rows + rows_per - 1) / rows_per;
  if (p.gs_mode == kGsTensor) {
    cudaError_t e = cudaMemsetAsync(p.gs, 0, sizeof(float) * p.groups, stream);
    if (e != cudaSuccess) return e;
    const int64_t work = ((int64_t)p.m * (p.k / 16) + kAmaxChunks * kQThreads - 1) / (kAmaxChunks * kQThreads);
    e = launch_pdl(fp4_amax_kernel<T, ACT>, dim3((unsigned)std::min<int64_t>(work, 1 << 30), p.groups), dim3(kQThreads), 0, false, stream, p);
    if (e != cudaSuccess) return e;
    e = launch_pdl(fp4_gs_kernel, dim3(cdiv(p.groups, 256)), dim3(256), 0, true, stream, p.gs, p.groups);
    if (e != cudaSuccess) return e;
    pdl = true;
  }
  auto go = [&](auto kern) { return launch_pdl(kern, dim3((unsigned)grid), dim3(threads), 0, pdl, stream, p, shape); };
  if constexpr (FMT == 0)
    if (p.gs_mode == kGsRow)
      return p.values ? go(fp4_quantize_kernel<T, FMT, ACT, true, true>) : go(fp4_quantize_kernel<T, FMT, ACT, true, false>);
  return p.values ? go(fp4_quantize_kernel<T, FMT, ACT, false, true>) : go(fp4_quantize_kernel<T, FMT, ACT, false, false>);
}

template <typename T>
cudaError_t quantize_fmt(const Fp4QuantParams& p, int num_sms, bool pdl, cudaStream_t stream) {
  if (p.act < 0)
    return p.fmt == 0 ? quantize_t<T, 0, false>(p, num_sms, pdl, stream) : quantize_t<T, 1, false>(p, num_sms, pdl, stream);
  return p.fmt == 0 ? quantize_t<T, 0, true>(p, num_sms, pdl, stream) : quantize_t<T, 1, true>(p, num_sms, pdl, stream);
}

}  // namespace

cudaError_t launch_fp4_quantize(const Fp4QuantParams& p, int dtype, int num_sms, bool pdl, cudaStream_t stream) {
  if (dtype == 0) return quantize_fmt<__nv_bfloat16>(p, num_sms, pdl, stream);
  if (dtype == 1) return quantize_fmt<__half>(p, num_sms, pdl, stream);
  return quantize_fmt<float>(p, num_sms, pdl, stream);
}

cudaError_t launch_fp4_tile_scales(const uint8_t* src, uint8_t* dst, int groups, int m, int blocks, int k_tiles,
                                   int num_sms, cudaStream_t stream) {
  const int64_t n = (int64_t)groups * cdiv(m, 128) * k_tiles * 128;
  int64_t grid = (n + 255) / 256;
  if (grid > 16 * num_sms) grid = 16 * num_sms;
  return launch_pdl(fp4_tile_scales_kernel, dim3((unsigned)grid), dim3(256), 0, false, stream, src, dst, groups, m,
                    blocks, k_tiles);
}

cudaError_t launch_fp4_combine(const Fp4CombineParams& p, cudaStream_t stream) {
  const int gy = cdiv(p.hidden / 8, 256);
  return launch_pdl(fp4_combine_kernel, dim3(p.m, gy), dim3(256), 0, true, stream, p);
}

}  // namespace b4
