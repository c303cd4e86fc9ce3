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
// A thread holds 16 consecutive elements: one NVFP4 block, half an MXFP4 block
// (the pair joins by one shuffle).  Threads of a row stand side by side, so
// loads are 32-byte pieces of a contiguous stretch and code stores 8-byte
// pieces; with a per-row global scale the row stays in registers between its
// maximum and its codes (up to two chunks a thread; longer rows are read again,
// from L1).  Every step is IEEE fp32 in the order of the formula; h / d is the
// quotient corrected once by its fused-multiply-add residual (Markstein's
// scheme: the reciprocal correctly rounded, then r = h - q d exactly, q + r / d),
// which costs three operations an element where a division costs a dozen.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "fp4.cuh"
#include "ptx.cuh"

namespace b4 {

namespace {

constexpr int kQThreads = 256;
constexpr int kCached = 2;  // chunks a thread keeps between the row's maximum and its codes

__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ void from_f32(__nv_bfloat16* d, float v) { *d = __float2bfloat16_rn(v); }
__device__ __forceinline__ void from_f32(__half* d, float v) { *d = __float2half_rn(v); }
__device__ __forceinline__ void from_f32(float* d, float v) { *d = v; }

// 16 consecutive elements as fp32.
template <typename T>
__device__ __forceinline__ void load16(const T* src, bool vec, float (&h)[16]) {
  T raw[16];
  if (vec) {
#pragma unroll
    for (int i = 0; i < (int)(16 * sizeof(T) / 16); ++i)
      reinterpret_cast<uint4*>(raw)[i] = __ldg(reinterpret_cast<const uint4*>(src) + i);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) raw[i] = src[i];
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) h[i] = to_f32(raw[i]);
}

// Chunk c of the row after the prologue.
template <typename T, bool GATED>
__device__ __forceinline__ void load_chunk(const Fp4QuantParams& p, const T* row, int c, float (&h)[16]) {
  load16(row + 16 * c, p.vec, h);
  if constexpr (GATED) {
    float u[16];
    load16(row + p.k + 16 * c, p.vec, u);
#pragma unroll
    for (int i = 0; i < 16; ++i) h[i] = gated_act(h[i], u[i], p.glu);
  } else if (p.act == 1) {
#pragma unroll
    for (int i = 0; i < 16; ++i) h[i] = h[i] < 0.f ? 0.f : h[i] * h[i];  // NaN stays NaN
  }
}

// Bits of the largest magnitude; a NaN's bits exceed every number's, so it stays.
__device__ __forceinline__ uint32_t amax_bits(const float (&h)[16]) {
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) a = max(a, __float_as_uint(h[i]) & 0x7fffffffu);
  return a;
}

constexpr uint32_t kInfBits = 0x7f800000u;

// The row's global scale from the bits of its largest magnitude; NaN for a row
// with an infinity or a NaN in it, whose products are NaN.
__device__ __forceinline__ float row_gs(uint32_t a) {
  if (a == 0) return 1.f;
  if (a >= kInfBits) return __uint_as_float(0x7fffffffu);
  const int j = (int)(a >> 23) - 127 - 11 + ((a & 0x7fffffu) > 0x280000u);  // 6 448 = 1.3125 2^11
  return __uint_as_float((uint32_t)(max(j, -126) + 127) << 23);
}

struct BlockScale {
  uint32_t code;  // the scale's byte
  float d, inv;   // step of the codes and its reciprocal
  int kind;       // 0: all codes zero, 1: corrected reciprocal, 2: true division
};

__device__ __forceinline__ BlockScale block_scale(int fmt, uint32_t a, float gs) {
  BlockScale b;
  const float amax = __uint_as_float(a);
  if (fmt != 0) {
    const int e = a > kInfBits ? 255
                  : a == kInfBits ? 254
                                  : max((int)(a >> 23) - 2 + ((a & 0x7fffffu) > 0x400000u), 0);
    b.code = (uint32_t)e;
    b.d = e == 0 ? __uint_as_float(0x00400000u) : __uint_as_float((uint32_t)e << 23);  // 2^(e - 127)
    b.inv = e >= 254 ? __uint_as_float(0x00400000u) : __uint_as_float((uint32_t)(254 - e) << 23);
    b.kind = e == 255 ? 0 : 1;
    return b;
  }
  const float ratio = __fdiv_rn(amax, __fmul_rn(6.f, gs));
  b.code = ratio != ratio ? 0x7fu : (uint32_t)__nv_cvt_float_to_fp8(ratio, __NV_SATFINITE, __NV_E4M3);
  const float s = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)b.code, __NV_E4M3)));
  b.d = __fmul_rn(s, gs);
  if (!(b.d > 0.f) || a > kInfBits) {
    b.kind = 0;
    b.inv = 0.f;
  } else {
    b.inv = __frcp_rn(b.d);
    // the residual is exact while no product leaves the normal range
    b.kind = b.d >= 0x1p-100f && b.d <= 0x1p100f && amax * b.inv < 0x1p20f ? 1 : 2;
  }
  return b;
}

// E2M1 codes of 16 elements, element 2j in the low nibble of byte j.
__device__ __forceinline__ uint2 encode(int fmt, const float (&h)[16], const BlockScale& b) {
  if (b.kind == 0) return make_uint2(0, 0);
  uint32_t w[2];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t v = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float q[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float x = h[8 * half + 2 * j + i];
        if (b.kind == 2) {
          q[i] = __fdiv_rn(x, b.d);
        } else {
          q[i] = x * b.inv;  // MXFP4: exact, a power of two
          if (fmt == 0) q[i] = __fmaf_rn(__fmaf_rn(-q[i], b.d, x), b.inv, q[i]);
        }
      }
      v |= (uint32_t)__nv_cvt_float2_to_fp4x2(make_float2(q[0], q[1]), __NV_E2M1, cudaRoundNearest) << (8 * j);
    }
    w[half] = v;
  }
  return make_uint2(w[0], w[1]);
}

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

template <typename T>
__device__ __forceinline__ void store_values(T* dst, const uint2& w, float d, uint32_t code_nan) {
  T raw[16];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t byte = ((j < 4 ? w.x : w.y) >> (8 * (j & 3))) & 0xffu;
    const float2 v = __half22float2(__half2(__nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)byte, __NV_E2M1)));
    from_f32(&raw[2 * j], code_nan ? __uint_as_float(0x7fffffffu) : __fmul_rn(v.x, d));
    from_f32(&raw[2 * j + 1], code_nan ? __uint_as_float(0x7fffffffu) : __fmul_rn(v.y, d));
  }
#pragma unroll
  for (int i = 0; i < (int)(16 * sizeof(T) / 16); ++i)
    reinterpret_cast<uint4*>(dst)[i] = reinterpret_cast<const uint4*>(raw)[i];
}

}  // namespace

// tpr_log2: threads per row.  Rows beyond the operand (pad_rows) only clear
// their scales.
template <typename T, bool GATED, bool ROW>
__global__ void __launch_bounds__(kQThreads) fp4_quantize_kernel(const __grid_constant__ Fp4QuantParams p,
                                                                 int tpr_log2) {
  __shared__ uint32_t s_max[kQThreads / 32];
  const int tpr = 1 << tpr_log2;
  const int t = threadIdx.x & (tpr - 1);
  const int lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  if (p.status && blockIdx.x == 0 && threadIdx.x < 2) p.status[threadIdx.x] = 0;

  // this thread's row: packed index (codes, gs, values), scale tile and row in it
  const int64_t vrow = (int64_t)blockIdx.x * (kQThreads >> tpr_log2) + (threadIdx.x >> tpr_log2);
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
    const int64_t per = p.pad_rows ? (int64_t)tiles_per * 128 : p.m;
    group = (int)(vrow / per);
    lr = (int)(vrow - group * per);
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
  const int per_tile = p.fmt == 0 ? 4 : 8;  // chunks of a scale tile
  const int n_it = cdiv(p.k_tiles * per_tile, tpr);

  float h[ROW ? kCached : 1][16];
  float gs = 1.f;
  if constexpr (ROW) {
    uint32_t a = 0;
#pragma unroll
    for (int it = 0; it < kCached; ++it) {
      const int c = it * tpr + t;
      if (c < chunks && !zero) load_chunk<T, GATED>(p, x, c, h[it]);
      else {
#pragma unroll
        for (int i = 0; i < 16; ++i) h[it][i] = 0.f;
      }
      a = max(a, amax_bits(h[it]));
    }
    for (int it = kCached; it < n_it; ++it) {
      const int c = it * tpr + t;
      if (c < chunks && !zero) {
        float v[16];
        load_chunk<T, GATED>(p, x, c, v);
        a = max(a, amax_bits(v));
      }
    }
    for (int o = min(tpr, 32) / 2; o > 0; o >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
    if (tpr > 32) {
      if (lane == 0) s_max[threadIdx.x >> 5] = a;
      __syncthreads();
      const int w0 = (threadIdx.x >> tpr_log2) << (tpr_log2 - 5);
      for (int w = 0; w < (tpr >> 5); ++w) a = max(a, s_max[w0 + w]);
    }
    gs = row_gs(a);
    if (live && t == 0) p.gs[row] = gs;
  } else if (p.gs_mode != kGsNone && live) {
    gs = __ldg(p.gs + group);
  }

  auto emit = [&](int c, const float(&v)[16]) {
    uint32_t a = amax_bits(v);
    if (p.fmt != 0) a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
    const bool in = c < chunks;
    BlockScale b = block_scale(p.fmt, a, gs);
    if (!in) b.code = 0;
    if (in) {
      const uint2 w = encode(p.fmt, v, b);
      *reinterpret_cast<uint2*>(p.codes + row * p.ld + 8 * (int64_t)c) = w;
      if (p.values)
        store_values(reinterpret_cast<T*>(p.values) + row * p.k + 16 * (int64_t)c, w, b.d,
                     p.fmt == 0 ? b.code == 0x7fu : b.code == 255u);
    }
    if (p.rowmajor_scales) {
      if (in && (p.fmt == 0 || !(c & 1))) {
        const int nb = p.k / fp4_group(p.fmt);
        p.scales[row * nb + (p.fmt == 0 ? c : c >> 1)] = (uint8_t)b.code;
      }
    } else {
      // the four scales of a tile row gather into one word
      const int pos = p.fmt == 0 ? c & 3 : (c >> 1) & 3;
      uint32_t w = b.code << (8 * pos);
      if (p.fmt == 0) w |= __shfl_xor_sync(0xffffffffu, w, 1);
      w |= __shfl_xor_sync(0xffffffffu, w, 2);
      if (p.fmt != 0) w |= __shfl_xor_sync(0xffffffffu, w, 4);
      const int kt = c / per_tile;
      if ((c & (per_tile - 1)) == 0 && kt < p.k_tiles && (live || pad))
        *reinterpret_cast<uint32_t*>(p.scales + (tile * p.k_tiles + kt) * kSfTile + (lr & 31) * 16 +
                                     ((lr >> 5) & 3) * 4) = w;
    }
  };
  if constexpr (ROW) {
#pragma unroll
    for (int it = 0; it < kCached; ++it)
      if (it < n_it) emit(it * tpr + t, h[it]);
  }
  for (int it = ROW ? kCached : 0; it < n_it; ++it) {
    const int c = it * tpr + t;
    float v[16];
    if (c < chunks && !zero) load_chunk<T, GATED>(p, x, c, v);
    else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = 0.f;
    }
    emit(c, v);
  }
}

// ------------------------------------------- one global scale per matrix
// Largest magnitude of each matrix of a stack, as fp32 bits (order of the
// atomics does not matter to a maximum), then amax / (6 448) in place.
template <typename T, bool GATED>
__global__ void __launch_bounds__(kQThreads) fp4_amax_kernel(const __grid_constant__ Fp4QuantParams p) {
  __shared__ uint32_t s_max[kQThreads / 32];
  const int group = blockIdx.y;
  const int per_row = p.k / 16;
  const int64_t n = (int64_t)p.m * per_row;
  uint32_t a = 0;
  for (int64_t i = (int64_t)blockIdx.x * kQThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kQThreads) {
    const int64_t r = i / per_row;
    float h[16];
    load_chunk<T, GATED>(p, reinterpret_cast<const T*>(p.x) + ((int64_t)group * p.m + r) * p.x_stride,
                         (int)(i - r * per_row), h);
    a = max(a, amax_bits(h));
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

template <typename T, bool GATED>
cudaError_t quantize_t(const Fp4QuantParams& p, int num_sms, bool pdl, cudaStream_t stream) {
  // threads per row: two chunks each, at least a warp for ragged rows (their
  // group is found by the whole warp) and eight for a scale word
  const int slots = p.k_tiles * (p.fmt == 0 ? 4 : 8);
  int lg = p.offsets ? 5 : 3;
  while ((1 << lg) < kQThreads && (1 << lg) * 2 < slots) ++lg;
  const int64_t rows = p.offsets ? p.m : (int64_t)p.groups * (p.pad_rows ? cdiv(p.m, 128) * 128 : p.m);
  const int64_t grid = (rows + (kQThreads >> lg) - 1) / (kQThreads >> lg);
  if (p.gs_mode == kGsTensor) {
    cudaError_t e = cudaMemsetAsync(p.gs, 0, sizeof(float) * p.groups, stream);
    if (e != cudaSuccess) return e;
    const int64_t work = ((int64_t)p.m * (p.k / 16) + 4 * kQThreads - 1) / (4 * kQThreads);
    int gx = (8 * num_sms + p.groups - 1) / p.groups;
    if (gx > work) gx = (int)work;
    if (gx < 1) gx = 1;
    e = launch_pdl(fp4_amax_kernel<T, GATED>, dim3(gx, p.groups), dim3(kQThreads), 0, false, stream, p);
    if (e != cudaSuccess) return e;
    e = launch_pdl(fp4_gs_kernel, dim3(cdiv(p.groups, 256)), dim3(256), 0, false, stream, p.gs, p.groups);
    if (e != cudaSuccess) return e;
  }
  if (p.gs_mode == kGsRow)
    return launch_pdl(fp4_quantize_kernel<T, GATED, true>, dim3((unsigned)grid), dim3(kQThreads), 0, pdl, stream, p, lg);
  return launch_pdl(fp4_quantize_kernel<T, GATED, false>, dim3((unsigned)grid), dim3(kQThreads), 0, pdl, stream, p, lg);
}

}  // namespace

cudaError_t launch_fp4_quantize(const Fp4QuantParams& p, int dtype, int num_sms, bool pdl, cudaStream_t stream) {
  const bool gated = p.act == 0;
  if (dtype == 0)
    return gated ? quantize_t<__nv_bfloat16, true>(p, num_sms, pdl, stream)
                 : quantize_t<__nv_bfloat16, false>(p, num_sms, pdl, stream);
  if (dtype == 1)
    return gated ? quantize_t<__half, true>(p, num_sms, pdl, stream) : quantize_t<__half, false>(p, num_sms, pdl, stream);
  return gated ? quantize_t<float, true>(p, num_sms, pdl, stream) : quantize_t<float, false>(p, num_sms, pdl, stream);
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
