// FP8 block quantisation: rows of x (gathered through an index, behind SwiGLU / clamped
// swiglu / ReLU^2) into E4M3 codes with an fp32 scale per block of 128 along K, or weight
// matrices with one per 128 x 128.
//
//   s = amax / 448, or 2^j, j the least with amax <= 448 2^j;  at least 2^-126; 1 where amax is 0
//   c = e4m3(h / s), nearest even of the quotient in fp32; a block with an infinity or a
//       NaN has the scale NaN
//
// A thread takes pieces of 16 consecutive elements, one, two or four of a block of 128: a
// 32-byte load (two of fp32) and a 16-byte store of codes each; the block's threads are
// neighbours and join their maxima by shuffles.  The quotient is h y + h z in one fused
// multiply-add, y an approximate reciprocal of s and z what it lacks: to 46 bits before its
// rounding, two operations an element.
//
// Bound by DRAM where x comes from there; gathered rows, which L2 holds, by the issue of
// instructions.  A 128 x 128 block is read once and stays in the registers of 512 threads
// between its maximum and its codes (with 256 threads 145 us for the second line below).
//
// Measured: 8192 rows of 4096 bf16 16.8 us (6.0 TB/s), with values too 26.0 (6.5 TB/s); 12288 gathered rows
// of 2048 10.4; 16 fp32 matrices of 2816 x 2048, values too, 128 us (6.5 TB/s).

#include <type_traits>

#include "fp8_quant.cuh"

namespace b4 {

using namespace fp8q;

namespace {

constexpr int kThreads8 = 128;
constexpr int kBlockThreads = 512;  // of a 128 x 128 block: two chunks a thread
constexpr int kBlockChunks = 1024 / kBlockThreads, kBlockStep = kBlockThreads / 8, kBlockResident = 2;

// What the codes stand for, in x's type.
template <typename T>
__device__ __forceinline__ void store_values8(T* dst, int level, const uint4& w, float s) {
  const uint32_t word[4] = {w.x, w.y, w.z, w.w};
  T e[16];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const __nv_fp8x2_storage_t pair = (__nv_fp8x2_storage_t)(word[j >> 1] >> (16 * (j & 1)));
    const float2 v = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(pair, __NV_E4M3)));
    from_f32(&e[2 * j], __fmul_rn(v.x, s));
    from_f32(&e[2 * j + 1], __fmul_rn(v.y, s));
  }
  uint32_t o[16 * sizeof(T) / 4];
  memcpy(o, e, sizeof(o));
  store_words(dst, level, o);
}

}  // namespace

// A scale per row and 128 columns: 8 / N threads take a block, N chunks each, and share its scale.
template <typename T, bool ACT, bool POW2, int N>
__global__ void __launch_bounds__(kThreads8) fp8_quantize_kernel(const __grid_constant__ Fp8QuantParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const Fp4QuantParams& q = p.q;
  if (q.status && blockIdx.x == 0 && threadIdx.x < 2) q.status[threadIdx.x] = 0;
  constexpr int kLanes = 8 / N;                // of a block
  const uint32_t slots = kLanes * p.kb;        // threads of a row
  int64_t rows = (int64_t)q.groups * q.m;
  if (q.offsets) rows = min(max(__ldg(q.offsets + q.groups), 0), q.m);
  const uint64_t base = (uint64_t)blockIdx.x * kThreads8;
  int64_t row = base >> 32 ? (int64_t)(base / slots) : (int64_t)((uint32_t)base / slots);
  uint32_t j = (uint32_t)(base - row * slots) + threadIdx.x;
  while (j >= slots) j -= slots, ++row;  // (seldom more than twice: cheaper than a division)
  const uint32_t block = j / kLanes;
  const int chunk = (int)(8 * block + j % kLanes);  // and every kLanes-th of the block's from there
  const bool live = row < rows;
  int64_t src = row;
  if (q.rows && live) {
    const int r = __ldg(q.rows + row);
    src = r < 0 ? -1 : r / q.row_div;
    if (q.x_rows > 0 && src >= q.x_rows) src = -1;
  }
  Chunk<T, ACT> h[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (live && src >= 0 && 16 * (chunk + kLanes * i) < q.k)
      h[i].get(q, reinterpret_cast<const T*>(q.x) + src * q.x_stride, chunk + kLanes * i);
    else h[i].zero();
  }
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) a = max(a, h[i].amax());
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
  const float s = block_scale<POW2>(a);
  if (!live) return;
  if (j % kLanes == 0) p.scales[row * p.kb + block] = s;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = chunk + kLanes * i;
    if (16 * c < q.k) {
      const uint4 w = encode8<POW2>(h[i], s);
      *reinterpret_cast<uint4*>(q.codes + row * q.ld + 16 * c) = w;
      if (q.values) store_values8(reinterpret_cast<T*>(q.values) + row * q.k + 16 * c, q.values_vec, w, s);
    }
  }
}

// A scale per 128 x 128: a block of threads takes one.
template <typename T, bool ACT, bool POW2>
__global__ void __launch_bounds__(kBlockThreads, kBlockResident) fp8_quantize_block_kernel(const __grid_constant__ Fp8QuantParams p) {
  __shared__ uint32_t s_max[kBlockThreads / 32];
  pdl_wait();
  pdl_launch_dependents();
  const Fp4QuantParams& q = p.q;
  const int row_blocks = cdiv(q.m, kFp8Block);
  const int64_t gb = blockIdx.x / (uint32_t)p.kb;  // group and row block
  const int kb = blockIdx.x % (uint32_t)p.kb;
  const int64_t group = gb / row_blocks;
  const int r0 = (int)(gb - group * row_blocks) * kFp8Block + (threadIdx.x >> 3);
  const int chunk = 8 * kb + (threadIdx.x & 7);
  const bool in = 16 * chunk < q.k;
  Chunk<T, ACT> h[kBlockChunks];
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < kBlockChunks; ++i) {
    const int r = r0 + kBlockStep * i;
    if (in && r < q.m) h[i].get(q, reinterpret_cast<const T*>(q.x) + (group * q.m + r) * q.x_stride, chunk);
    else h[i].zero();
  }
#pragma unroll
  for (int i = 0; i < kBlockChunks; ++i) a = max(a, h[i].amax());
  a = __reduce_max_sync(0xffffffffu, a);
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = a;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kBlockThreads / 32; ++w) a = max(a, s_max[w]);
  const float s = block_scale<POW2>(a);
  if (threadIdx.x == 0) p.scales[blockIdx.x] = s;
#pragma unroll
  for (int i = 0; i < kBlockChunks; ++i) {
    const int r = r0 + kBlockStep * i;
    if (in && r < q.m) {
      const int64_t row = group * q.m + r;
      const uint4 w = encode8<POW2>(h[i], s);
      *reinterpret_cast<uint4*>(q.codes + row * q.ld + 16 * chunk) = w;
      if (q.values) store_values8(reinterpret_cast<T*>(q.values) + row * q.k + 16 * chunk, q.values_vec, w, s);
    }
  }
}

namespace {

template <typename K>
cudaError_t launch8(K kern, int64_t grid, int threads, cudaStream_t stream, const Fp8QuantParams& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <typename T, bool ACT, bool POW2>
cudaError_t quantize8(const Fp8QuantParams& p, int block_rows, int sms, cudaStream_t stream) {
  const Fp4QuantParams& q = p.q;
  if (block_rows > 1)
    return launch8(fp8_quantize_block_kernel<T, ACT, POW2>, (int64_t)q.groups * cdiv(q.m, kFp8Block) * p.kb, kBlockThreads,
                   stream, p);
  const int64_t chunks = (q.offsets ? q.m : (int64_t)q.groups * q.m) * p.kb * 8;
  auto run = [&](auto n) {
    constexpr int N = n.value;
    return launch8(fp8_quantize_kernel<T, ACT, POW2, N>, (chunks / N + kThreads8 - 1) / kThreads8, kThreads8, stream, p);
  };
  // Chunks of a thread: more share a block's scale and a row's index among more elements, but leave
  // fewer threads to hide latencies.  In us with 1 / 2 / 4: 16-bit x, 512 rows of 4096 - / 2.5 / 2.8, 2036
  // gathered rows of 2880 - / 4.0 / 5.0, 12288 of 2048 14.6 / 11.4 / 10.4, 8192 rows of 4096 19.4 / 17.1 / 16.8; fp32
  // - / 27.2 / 33.7; behind SwiGLU, 12288 rows of 1408 fp32 24.1 / 25.1 / 29.6.
  if constexpr (!ACT) {
    if (sizeof(T) == 2 && chunks > (int64_t)sms * 2560) return run(std::integral_constant<int, sizeof(T) == 2 ? 4 : 2>{});
    if (chunks > (int64_t)sms * 512) return run(std::integral_constant<int, 2>{});
  }
  return run(std::integral_constant<int, 1>{});
}

template <typename T>
cudaError_t quantize8_t(const Fp8QuantParams& p, int block_rows, int sms, cudaStream_t stream) {
  if (p.q.act < 0)
    return p.pow2 ? quantize8<T, false, true>(p, block_rows, sms, stream) : quantize8<T, false, false>(p, block_rows, sms, stream);
  return p.pow2 ? quantize8<T, true, true>(p, block_rows, sms, stream) : quantize8<T, true, false>(p, block_rows, sms, stream);
}

}  // namespace

cudaError_t launch_fp8_quantize(const Fp8QuantParams& p, int dtype, int block_rows, int num_sms, cudaStream_t stream) {
  if (dtype == 0) return quantize8_t<__nv_bfloat16>(p, block_rows, num_sms, stream);
  if (dtype == 1) return quantize8_t<__half>(p, block_rows, num_sms, stream);
  return quantize8_t<float>(p, block_rows, num_sms, stream);
}

}  // namespace b4
