// Routing to experts (b4_route_topk in b4moe.h): from the router's logits to the ids and
// weights that b4_fused_moe, b4_fused_moe_a4, b4_fused_moe_fp8 and b4_route_pack read.
//
//   s = softmax(z) or sigmoid(z) over a token's experts,  c = s + bias  (no bias: the order of z)
//   groups: the E experts in equal neighbouring groups; a group counts with its largest c
//           or the sum of its two largest, and the best top_groups of them stay
//   ids:    the top_k largest c that are left, descending, ties to the lowest index
//   weight: s of the chosen, over their sum where renormalised, times a constant
//
// A warp takes a token: lane l holds up to V neighbouring experts in registers, a power of
// two of lanes to a group, so that lanes in order are experts in order and a tie's lowest
// index is the lowest lane.  A choice is one redux over order-preserving integer keys and
// one ballot.
//
// The order is that of the real numbers c, not of their roundings: scores differ by less
// than fp32 resolves about once in a thousand tokens, and another order there would send
// a token to another expert.  Without a bias the logits' own order decides (scores are
// monotone).  With one, neighbours in the order (and the last group taken and the first
// left) closer than fp32's error have their row done again in 64 bits, unless their
// logits and biases are equal, which is a true tie.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "b4moe.h"
#include "ptx.cuh"

namespace b4 {
void set_last_error(const char* fmt, ...);
b4_status require_device(int* sms);

namespace {

struct RouteParams {
  const void* logits;
  int64_t stride;
  const float* bias;          // or null
  const int32_t* num_tokens;  // or null
  int m, experts, top_k;
  int groups, top_groups, group_top;
  int per, lanes_log2, each;  // experts of a group, lanes of a group, experts of a lane
  int vec;                    // a lane's logits are one aligned piece
  int softmax, renorm;
  float scale;
  int32_t* ids;
  float* weights;
};

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kNone = INT32_MIN + 0x7fffff;  // the key of -inf

__device__ __forceinline__ int key_of(float c) {
  const int b = __float_as_int(c + 0.f);  // (-0 and 0 are one value)
  return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float value_of(int key) { return __int_as_float(key ^ ((key >> 31) & 0x7fffffff)); }
__device__ __forceinline__ int warp_max(int v) { return __reduce_max_sync(kAll, v); }
__device__ __forceinline__ float warp_max(float v) { return value_of(warp_max(key_of(v))); }
template <typename R>
__device__ __forceinline__ R warp_sum(R v) {
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float exp_(float x) { return expf(x); }
__device__ __forceinline__ double exp_(double x) { return exp(x); }

// e^(z - top) for z <= top, 1 where they are equal (infinities too)
template <typename R>
__device__ __forceinline__ R exp_below(R z, R top) {
  return z == top ? R(1) : exp_(z - top);
}
template <typename R>
__device__ __forceinline__ R sigmoid(R z) {
  const R e = exp_(-fabs(z));
  return (z >= R(0) ? R(1) : e) / (R(1) + e);
}

// A logit as it counts: a NaN does not.
template <typename T>
__device__ __forceinline__ float logit(const T* row, int e) {
  const float z = to_f32(row[e]);
  return z == z ? z : -INFINITY;
}

template <int V, typename T>
__device__ __forceinline__ void load_logits(const RouteParams& p, const T* row, int first, int count, float (&z)[V]) {
  constexpr int kBytes = V * (int)sizeof(T);
  if (kBytes >= 4 && p.vec) {
    T raw[V];
    if (count > 0) {
      if constexpr (kBytes >= 16) {
#pragma unroll
        for (int i = 0; i < kBytes / 16; ++i)
          reinterpret_cast<uint4*>(raw)[i] = __ldg(reinterpret_cast<const uint4*>(row + first) + i);
      } else if constexpr (kBytes >= 4) {
#pragma unroll
        for (int i = 0; i < kBytes / 4; ++i)
          reinterpret_cast<uint32_t*>(raw)[i] = __ldg(reinterpret_cast<const uint32_t*>(row + first) + i);
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float v = to_f32(raw[i]);
      z[i] = count > 0 && v == v ? v : -INFINITY;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) z[i] = i < count ? logit(row, first + i) : -INFINITY;
  }
}

// Largest two of a lane's group, in every lane of it.
template <typename R>
__device__ __forceinline__ void merge_top2(R& a, R& b, int lanes_log2) {
  for (int o = 0; o < lanes_log2; ++o) {
    const R x = __shfl_xor_sync(kAll, a, 1 << o), y = __shfl_xor_sync(kAll, b, 1 << o);
    const R second = fmax(b, y);
    b = fmax(fmin(a, x), second);
    a = fmax(a, x);
  }
}
template <typename R>
__device__ __forceinline__ R group_value(R a, R b, int group_top) {
  return group_top == 2 && b > -INFINITY ? a + b : a;
}
// Place of this lane's group in the order of the groups.
template <typename R>
__device__ __forceinline__ int group_rank(const RouteParams& p, R value, int group) {
  int rank = 0;
  for (int g = 0; g < p.groups; ++g) {
    const R v = __shfl_sync(kAll, value, g << p.lanes_log2);
    rank += v > value || (v == value && g < group);
  }
  return rank;
}

// The row's choice in 64 bits: expert j of the order in lane j, -1 past the last.
template <int V, typename T>
__device__ __noinline__ int choose64(const RouteParams& p, const T* row, int lane) {
  const int group = lane >> p.lanes_log2, at = (lane & ((1 << p.lanes_log2) - 1)) * p.each;
  const int count = group < p.groups ? max(min(p.each, p.per - at), 0) : 0, first = group * p.per + at;
  double c[V];
  double top = -INFINITY;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    c[i] = i < count ? (double)logit(row, first + i) : -INFINITY;
    top = fmax(top, c[i]);
  }
  double sum = 1.0;
  if (p.softmax) {
    for (int o = 16; o > 0; o >>= 1) top = fmax(top, __shfl_xor_sync(kAll, top, o));
    sum = 0.0;
#pragma unroll 1
    for (int i = 0; i < V; ++i)
      if (c[i] > -INFINITY) sum += exp_below(c[i], top);
    sum = warp_sum(sum);
  }
  double a = -INFINITY, b = -INFINITY;  // the lane's largest two
#pragma unroll 1
  for (int i = 0; i < V; ++i) {
    if (c[i] > -INFINITY) {
      const double z = c[i];
      const double s = p.softmax ? exp_below(z, top) / sum : sigmoid(z);
      const float bias = p.bias ? __ldg(p.bias + first + i) : 0.f;
      const double v = bias > -INFINITY ? s + (double)bias : -INFINITY;
      c[i] = p.bias ? v : z;
      b = fmax(b, fmin(a, v));
      a = fmax(a, v);
    }
  }
  bool keep = true;
  if (p.groups > 1) {
    merge_top2(a, b, p.lanes_log2);
    const double value = group < p.groups ? group_value(a, b, p.group_top) : -INFINITY;
    const int rank = group_rank(p, value, group);  // (every lane shuffles, those without a group too)
    keep = group < p.groups && rank < p.top_groups;
  }
  int chosen = -1;
  for (int j = 0; j < p.top_k; ++j) {
    double best = -INFINITY;
    int pos = 0;
    if (keep)
      for (int i = 0; i < V; ++i)
        if (c[i] > best) best = c[i], pos = i;
    double all = best;
    for (int o = 16; o > 0; o >>= 1) all = fmax(all, __shfl_xor_sync(kAll, all, o));
    if (!(all > -INFINITY)) break;
    const int owner = __ffs(__ballot_sync(kAll, best == all)) - 1;
    const int e = __shfl_sync(kAll, first + pos, owner);
    if (lane == j) chosen = e;
    if (lane == owner) c[pos] = -INFINITY;
  }
  return chosen;
}

// Whether two values of the order may stand the other way round: the sum of what their
// fp32 forms can be off by.  A score is at most 1 and off by 2^-21 (its exponential one ulp of
// an argument off by 2^-24 |z - top|, the sum of exponentials and the quotient another
// three); the sum with the bias adds 2^-24 of itself.
__device__ __forceinline__ bool close_(float a, float b, float terms) {
  return a - b <= terms * (0x1p-20f + 0x1p-23f * fabsf(a));
}

template <int V, typename T>
__global__ void __launch_bounds__(128) route_topk_kernel(const __grid_constant__ RouteParams p) {
  const int lane = threadIdx.x & 31;
  const int token = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  pdl_wait();
  pdl_launch_dependents();
  if (token >= p.m) return;
  int32_t* ids = p.ids + (int64_t)token * p.top_k;
  float* weights = p.weights + (int64_t)token * p.top_k;
  if (p.num_tokens && token >= __ldg(p.num_tokens)) {
    if (lane < p.top_k) ids[lane] = -1, weights[lane] = 0.f;
    return;
  }
  const T* row = reinterpret_cast<const T*>(p.logits) + (int64_t)token * p.stride;
  const int group = lane >> p.lanes_log2, at = (lane & ((1 << p.lanes_log2) - 1)) * p.each;
  const int count = group < p.groups ? max(min(p.each, p.per - at), 0) : 0, first = group * p.per + at;

  float z[V];
  load_logits<V>(p, row, first, count, z);
  // softmax over all experts, where more than its order is needed
  const bool scores = p.bias || (p.groups > 1 && p.group_top == 2);
  float top = 0.f, inv = 1.f;
  if (p.softmax && (scores || !p.renorm)) {
    float t = z[0];
#pragma unroll
    for (int i = 1; i < V; ++i) t = fmaxf(t, z[i]);
    top = warp_max(t);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) sum += z[i] > -INFINITY ? exp_below(z[i], top) : 0.f;
    inv = 1.f / warp_sum(sum);
  }
  int key[V];
  float a = -INFINITY, b = -INFINITY;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float c = z[i];
    if (scores && c > -INFINITY) {
      c = p.softmax ? exp_below(c, top) * inv : sigmoid(c);
      if (p.bias) {
        const float bias = __ldg(p.bias + first + i);
        c = bias > -INFINITY ? c + bias : -INFINITY;
      }
    }
    key[i] = key_of(p.bias ? c : z[i]);
    b = fmaxf(b, fminf(a, c));
    a = fmaxf(a, c);
  }
  bool again = false;  // fp32 does not decide
  if (p.groups > 1) {
    merge_top2(a, b, p.lanes_log2);
    const float value = group < p.groups ? group_value(a, b, p.group_top) : -INFINITY;
    const int rank = group_rank(p, value, group);
    if (scores && p.top_groups < p.groups) {
      const uint32_t in = __ballot_sync(kAll, rank == p.top_groups - 1 && group < p.groups);
      const uint32_t out = __ballot_sync(kAll, rank == p.top_groups && group < p.groups);
      const float last = __shfl_sync(kAll, value, __ffs(in) - 1), next = __shfl_sync(kAll, value, __ffs(out) - 1);
      again = next > -INFINITY && close_(last, next, 4.f);
    }
    if (rank >= p.top_groups || group >= p.groups) {
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = kNone;
    }
  }
  int chosen = -1, its_key = kNone;
  const int rounds = p.bias ? p.top_k + 1 : p.top_k;  // with a bias the first left is looked at too
  for (int j = 0; j < rounds; ++j) {
    int best = key[0];
#pragma unroll
    for (int i = 1; i < V; ++i) best = max(best, key[i]);
    const int all = warp_max(best);
    if (all <= kNone) break;
    const int owner = __ffs(__ballot_sync(kAll, best == all)) - 1;
    int pos = 0;
#pragma unroll
    for (int i = V - 1; i >= 0; --i) pos = key[i] == all ? i : pos;
    const int e = __shfl_sync(kAll, first + pos, owner);
    if (lane == owner) {
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = i == pos ? kNone : key[i];
    }
    if (lane == j) chosen = e, its_key = all;
    if (p.bias && j > 0 && !again) {
      // neighbours j - 1 and j of the order
      const int before = __shfl_sync(kAll, its_key, j - 1), e0 = __shfl_sync(kAll, chosen, j - 1);
      if (close_(value_of(before), value_of(all), 2.f))
        again = !(logit(row, e0) == logit(row, e) && __ldg(p.bias + e0) == __ldg(p.bias + e));
    }
  }
  if (again) chosen = choose64<V>(p, row, lane);

  const bool have = lane < p.top_k && chosen >= 0;
  const float zc = have ? logit(row, chosen) : -INFINITY;
  float w = 0.f;
  if (p.renorm) {
    const float most = warp_max(zc);
    // of sigmoids, times e^-most below zero: their ratio where they themselves underflow
    if (have) w = p.softmax ? exp_below(zc, most) : exp_below(fminf(zc, 0.f), fminf(most, 0.f)) / (1.f + expf(-fabsf(zc)));
    const float sum = warp_sum(w);
    w = have ? w / sum : 0.f;
  } else if (have) {
    w = p.softmax ? exp_below(zc, top) * inv : sigmoid(zc);
  }
  if (lane < p.top_k) {
    ids[lane] = chosen;
    weights[lane] = have ? w * p.scale : 0.f;
  }
}

#define ROUTE_FAIL(st, ...)      \
  do {                           \
    set_last_error(__VA_ARGS__); \
    return st;                   \
  } while (0)
#define ROUTE_INVALID(...) ROUTE_FAIL(B4_ERR_INVALID_ARGUMENT, __VA_ARGS__)

template <int V, typename T>
cudaError_t launch_route(const RouteParams& p, int sms, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  const int warps = p.m <= 4 * sms ? 1 : 4;
  cfg.gridDim = dim3((p.m + warps - 1) / warps);
  cfg.blockDim = dim3(32 * warps);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, route_topk_kernel<V, T>, p);
}

template <typename T>
cudaError_t launch_each(RouteParams& p, int sms, cudaStream_t stream) {
  int v = 1;
  while (v < p.each) v *= 2;
  const int bytes = v * (int)sizeof(T), align = bytes < 16 ? bytes : 16;
  p.vec = p.each == v && p.per % v == 0 && reinterpret_cast<uintptr_t>(p.logits) % align == 0 &&
          p.stride * (int)sizeof(T) % align == 0;
  switch (v) {
    case 1: return launch_route<1, T>(p, sms, stream);
    case 2: return launch_route<2, T>(p, sms, stream);
    case 4: return launch_route<4, T>(p, sms, stream);
    case 8: return launch_route<8, T>(p, sms, stream);
    case 16: return launch_route<16, T>(p, sms, stream);
    default: return launch_route<32, T>(p, sms, stream);
  }
}

}  // namespace
}  // namespace b4

using namespace b4;

extern "C" b4_status b4_route_topk(const b4_route_config* cfg, const void* logits, const float* bias,
                                   const int32_t* num_tokens, int32_t* topk_ids, float* topk_weights,
                                   b4_stream_t stream) {
  if (!cfg) ROUTE_INVALID("cfg is NULL");
  if (cfg->m < 0 || cfg->m > (1 << 25)) ROUTE_INVALID("m = %d not in [0, 2^25]", cfg->m);
  if (cfg->num_experts < 1 || cfg->num_experts > 1024) ROUTE_INVALID("num_experts = %d not in [1, 1024]", cfg->num_experts);
  if (cfg->top_k < 1 || cfg->top_k > 32 || cfg->top_k > cfg->num_experts)
    ROUTE_INVALID("top_k = %d not in [1, min(32, num_experts = %d)]", cfg->top_k, cfg->num_experts);
  if (cfg->num_groups < 1 || cfg->num_groups > 32 || cfg->num_experts % cfg->num_groups)
    ROUTE_INVALID("num_groups = %d must be in [1, 32] and divide num_experts = %d", cfg->num_groups, cfg->num_experts);
  if (cfg->top_groups < 1 || cfg->top_groups > cfg->num_groups)
    ROUTE_INVALID("top_groups = %d not in [1, num_groups = %d]", cfg->top_groups, cfg->num_groups);
  if (cfg->top_groups * (cfg->num_experts / cfg->num_groups) < cfg->top_k)
    ROUTE_INVALID("top_groups = %d groups of %d experts hold fewer than top_k = %d", cfg->top_groups,
                  cfg->num_experts / cfg->num_groups, cfg->top_k);
  if (cfg->group_top < 1 || cfg->group_top > 2) ROUTE_INVALID("group_top = %d is neither 1 nor 2", cfg->group_top);
  if (cfg->score != B4_SCORE_SOFTMAX && cfg->score != B4_SCORE_SIGMOID) ROUTE_INVALID("score = %d unknown", cfg->score);
  if (cfg->logits_dtype < B4_DTYPE_BF16 || cfg->logits_dtype > B4_DTYPE_F32)
    ROUTE_INVALID("logits_dtype = %d unknown", cfg->logits_dtype);
  if (!std::isfinite(cfg->scale)) ROUTE_INVALID("scale = %g must be finite", (double)cfg->scale);
  if (cfg->logits_stride != 0 && cfg->logits_stride < cfg->num_experts)
    ROUTE_INVALID("logits_stride = %lld below num_experts = %d", (long long)cfg->logits_stride, cfg->num_experts);
  if (cfg->m == 0) return B4_OK;
  if (!logits || !topk_ids || !topk_weights) ROUTE_INVALID("null pointer argument");
  const size_t width = cfg->logits_dtype == B4_DTYPE_F32 ? 4 : 2;
  auto off = [](const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; };
  if (off(logits, width) || off(bias, 4) || off(num_tokens, 4) || off(topk_ids, 4) || off(topk_weights, 4))
    ROUTE_INVALID("misaligned logits, bias, num_tokens, topk_ids or topk_weights");
  int sms = 0;
  const b4_status st = require_device(&sms);
  if (st != B4_OK) return st;
  RouteParams p{};
  p.logits = logits;
  p.stride = cfg->logits_stride ? cfg->logits_stride : cfg->num_experts;
  p.bias = bias;
  p.num_tokens = num_tokens;
  p.m = cfg->m;
  p.experts = cfg->num_experts;
  p.top_k = cfg->top_k;
  p.groups = cfg->num_groups;
  p.top_groups = cfg->top_groups;
  p.group_top = cfg->group_top;
  p.per = cfg->num_experts / cfg->num_groups;
  p.lanes_log2 = 5;
  while ((cfg->num_groups << p.lanes_log2) > 32) --p.lanes_log2;
  p.each = (p.per + (1 << p.lanes_log2) - 1) >> p.lanes_log2;
  p.softmax = cfg->score == B4_SCORE_SOFTMAX;
  p.renorm = cfg->renormalize != 0;
  p.scale = cfg->scale;
  p.ids = topk_ids;
  p.weights = topk_weights;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = cfg->logits_dtype == B4_DTYPE_BF16  ? launch_each<__nv_bfloat16>(p, sms, s)
                        : cfg->logits_dtype == B4_DTYPE_F16 ? launch_each<__half>(p, sms, s)
                                                            : launch_each<float>(p, sms, s);
  if (e != cudaSuccess) ROUTE_FAIL(B4_ERR_CUDA, "route top-k: %s (%s)", cudaGetErrorName(e), cudaGetErrorString(e));
  return B4_OK;
}
