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
// index is the lowest lane.  V is 64 at most: 1020 experts in 17 groups are 60 a lane (with one
// group, or a power of two of them, 1024 are 32; 16384 tokens of 960 experts in 20 groups, 48 a lane,
// 1.13 ms).  A lane sorts its experts once; a choice is then one redux over
// the lanes' first keys (integers of the floats' order) and one ballot.
//
// The order is that of the real numbers c, not of their roundings: scores differ by less
// than fp32 resolves about once in a thousand tokens, and another order there would send
// a token to another expert.  Without a bias the logits' own order decides (scores are
// monotone).  With one, where neighbours in the order are closer than fp32's error, the
// chosen and the next are compared again in 64 bits, a lane each; where groups taken and
// groups left may stand the other way round, these are, from the experts that may be their
// largest (softmax, whose scores need the row's sum: the whole row); where a third expert comes
// close, the row is done again in 64 bits.
//
// Bound by latency for few tokens (one launch: 2.3 us for 1 token of 128 experts) and by the
// issue of instructions for many: 16384 tokens of 256 experts in 8 groups, sigmoid with a bias,
// bf16 22 us (8.4 MB of logits, read once).  A row done again as a whole holds its warp for 5 us,
// which the last ones show: with close groups done so too it was 27.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <climits>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "b4moe.h"
#include "fp4_quant.cuh"

namespace b4 {
void set_last_error(const char* fmt, ...);
b4_status require_device(int* sms);

namespace {

using fp4q::exp2_approx;
using fp4q::rcp_approx;

struct RouteParams {
  const void* logits;
  int64_t stride;
  const float* bias;          // or null
  const int32_t* num_tokens;  // or null
  int m, experts, top_k;
  int groups, top_groups, group_top;
  int per, lanes_log2, each;  // experts of a group, lanes of a group, experts of a lane
  int vec, bias_vec;          // a lane's logits, its biases are one aligned piece
  int softmax, renorm;
  float scale;
  int32_t* ids;
  float* weights;
};

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kNone = INT32_MIN + 0x7fffff;  // the key of -inf
constexpr int kMaxEach = 64;  // experts of a lane
constexpr int kMaxVec = 32;   // a lane with more of them never holds a whole power of two
// A bit for each of a lane's V experts.
template <int V>
using Mask = std::conditional_t<(V > 32), unsigned long long, uint32_t>;
__device__ __forceinline__ int first_bit(uint32_t m) { return __ffs(m) - 1; }
__device__ __forceinline__ int first_bit(unsigned long long m) { return __ffsll(m) - 1; }

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

// For the order alone: the machine's exponential and reciprocal (2^-22 each), far cheaper.
__device__ __forceinline__ float exp_order(float x) { return exp2_approx(1.44269504f * x); }
__device__ __forceinline__ float sigmoid_order(float z) { return rcp_approx(1.f + exp_order(-z)); }

// A logit as it counts: a NaN does not.
template <typename T>
__device__ __forceinline__ float logit(const T* row, int e) {
  const float z = to_f32(row[e]);
  return z == z ? z : -INFINITY;
}

template <int V, typename T>
__device__ __forceinline__ void load_logits(const RouteParams& p, const T* row, int first, int count, int vec, float (&z)[V]) {
  constexpr int kBytes = V * (int)sizeof(T);
  if (kBytes >= 4 && V <= kMaxVec && vec) {
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

// 64-bit values as integers of the same order.
__device__ __forceinline__ long long key64(double c) {
  const long long b = __double_as_longlong(c + 0.0);
  return b ^ ((b >> 63) & 0x7fffffffffffffffll);
}
constexpr long long kNone64 = LLONG_MIN + 0xfffffffffffffll;  // the key of -inf
__device__ __forceinline__ long long warp_max(long long v) {
  for (int o = 16; o > 0; o >>= 1) {
    const long long x = __shfl_xor_sync(kAll, v, o);
    v = x > v ? x : v;
  }
  return v;
}

// The row's choice in 64 bits: expert j of the order in lane j, -1 past the last.
template <int V, typename T>
__device__ __noinline__ int choose64(const RouteParams& p, const T* row, int lane) {
  const int group = lane >> p.lanes_log2, at = (lane & ((1 << p.lanes_log2) - 1)) * p.each;
  const int count = group < p.groups ? max(min(p.each, p.per - at), 0) : 0, first = group * p.per + at;
  double top = -INFINITY, sum = 1.0;
  if (p.softmax) {
    float t = -INFINITY;
    for (int i = 0; i < count; ++i) t = fmaxf(t, logit(row, first + i));
    top = warp_max(t);
    sum = 0.0;
#pragma unroll 1
    for (int i = 0; i < count; ++i) {
      const double z = logit(row, first + i);
      if (z > -INFINITY) sum += exp_below(z, top);
    }
    sum = warp_sum(sum);
  }
  long long key[V];
  double a = -INFINITY, b = -INFINITY;  // the lane's largest two
#pragma unroll 1
  for (int i = 0; i < V; ++i) {
    const double z = i < count ? (double)logit(row, first + i) : -INFINITY;
    const float bias = p.bias && i < count ? __ldg(p.bias + first + i) : 0.f;
    double v = -INFINITY;
    if (z > -INFINITY && bias > -INFINITY) v = (p.softmax ? exp_below(z, top) / sum : sigmoid(z)) + (double)bias;
    key[i] = key64(p.bias ? v : z);
    b = fmax(b, fmin(a, v));
    a = fmax(a, v);
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
    long long best = kNone64;
    int pos = 0;
    for (int i = 0; i < V; ++i)
      if (keep && key[i] > best) best = key[i], pos = i;
    const long long all = warp_max(best);
    if (all <= kNone64) break;
    const int owner = __ffs(__ballot_sync(kAll, best == all)) - 1;
    const int e = __shfl_sync(kAll, first + pos, owner);
    if (lane == j) chosen = e;
    if (lane == owner) key[pos] = kNone64;
  }
  return chosen;
}

// Whether two values of the order may stand the other way round: twice what their fp32 forms
// can be off by, the biases' part, and the scores' part once.  A score is at most `most` (1, or the largest of a
// softmax) and off by 6 2^-24 of that for itself (its exponential 2^-22, an argument off by 2^-23 |z|,
// which a score of at most e^-|z| makes small, and a product); what a softmax's scores share, the sum of
// exponentials with 11 roundings at most (by halves in a lane, then five shuffles; one by one 31 small ones
// beside a large one could all be rounded up) and the quotient, moves two of them apart by 15 2^-24 of
// their difference.  So 27 2^-24 in all, taken as 32; the sum with the bias adds 2^-24 of itself.
__device__ __forceinline__ bool close_(float a, float b, float terms, float most) {
  return a - b <= terms * (0x1p-20f * most + 0x1p-23f * fabsf(a));
}

// Where a group's real value lies, from its fp32 one and its largest two: twice what the biases' part can be off by.  Each of
// the two is off by 6 2^-24 of `most` and by 2^-24 of itself, and what a softmax's scores share moves two
// groups apart by 30 2^-24 (see close_): 27 2^-24 a group, taken as 32, once.  The sum adds 2^-24 of
// itself, which is far less than of the two where they cancel.  (a is the larger; sums past fp32's range are not
// infinite.)
struct Range {
  float low, high;
};
__device__ __forceinline__ Range group_range(float value, float a, float b, int group_top, float most) {
  const float off = 0x1p-19f * most + 0x1p-22f * fabsf(a) + (group_top == 2 && b > -INFINITY ? 0x1p-22f * fabsf(b) : 0.f);
  if (fabsf(value) < INFINITY) return Range{value - off, value + off};
  return Range{value > 0.f && a < INFINITY ? FLT_MAX : value, value < 0.f && a > -INFINITY ? -FLT_MAX : value};
}

// Of sigmoid scores in 64 bits, the largest two among a lane's experts in `mask`.
template <typename T, typename M>
__device__ __noinline__ double2 top2_64(const RouteParams& p, const T* row, int first, M mask) {
  double a = -INFINITY, b = -INFINITY;
  while (__any_sync(kAll, mask != 0)) {
    if (mask) {
      const int e = first + first_bit(mask);
      mask &= mask - 1;
      const double v = sigmoid((double)logit(row, e)) + (p.bias ? (double)__ldg(p.bias + e) : 0.0);
      b = fmax(b, fmin(a, v));
      a = fmax(a, v);
    }
  }
  return make_double2(a, b);
}

// A lane's experts, sorted: keys descending, equal ones by index.  (An odd-even merge network.)
template <int V>
__device__ __forceinline__ void sort_keys(int (&key)[V], int (&pos)[V]) {
#pragma unroll
  for (int p = 1; p < V; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < V; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < V && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
            const int a = i + j, b = i + j + k;
            const bool swap = key[b] > key[a] || (key[b] == key[a] && pos[b] < pos[a]);
            const int ka = key[a], pa = pos[a];
            key[a] = swap ? key[b] : ka, pos[a] = swap ? pos[b] : pa;
            key[b] = swap ? ka : key[b], pos[b] = swap ? pa : pos[b];
          }
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
  load_logits<V>(p, row, first, count, p.vec, z);
  // softmax over all experts, where more than its order is needed
  const bool scores = p.bias || (p.groups > 1 && p.group_top == 2);
  float top = 0.f, inv = 1.f;  // (1 / the sum: the largest of the softmax)
  if (p.softmax && (scores || !p.renorm)) {
    float t = z[0];
#pragma unroll
    for (int i = 1; i < V; ++i) t = fmaxf(t, z[i]);
    top = warp_max(t);
    float e[V];
#pragma unroll
    for (int i = 0; i < V; ++i) e[i] = z[i] > -INFINITY ? exp_below(z[i], top) : 0.f;
#pragma unroll
    for (int o = V / 2; o > 0; o /= 2)  // (by halves: see close_)
#pragma unroll
      for (int i = 0; i < o; ++i) e[i] += e[i + o];
    inv = 1.f / warp_sum(e[0]);
  }
  int key[V], pos[V];
  float a = -INFINITY, b = -INFINITY;
  if (scores) {
    float bias[V];
    if (p.bias) load_logits<V>(p, p.bias, first, count, p.bias_vec, bias);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float c = z[i];
      if (c > -INFINITY) c = p.softmax ? (c == top ? 1.f : exp_order(c - top)) * inv : sigmoid_order(c);
      if (p.bias) c = c > -INFINITY && bias[i] > -INFINITY ? c + bias[i] : -INFINITY;
      key[i] = key_of(p.bias ? c : z[i]);
      b = fmaxf(b, fminf(a, c));
      a = fmaxf(a, c);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      key[i] = key_of(z[i]);
      a = fmaxf(a, z[i]);
    }
  }
  bool again = false;  // fp32 does not decide
  if (p.groups > 1) {
    merge_top2(a, b, p.lanes_log2);
    const float value = group < p.groups ? group_value(a, b, p.group_top) : -INFINITY;
    int rank = group_rank(p, value, group);
    if (scores && p.top_groups < p.groups) {
      const bool kept = group < p.groups && rank < p.top_groups, left = group < p.groups && rank >= p.top_groups;
      const Range r = group_range(value, a, b, p.group_top, inv);
      const float least_kept = -warp_max(kept ? -r.low : -INFINITY), most_left = warp_max(left ? r.high : -INFINITY);
      const bool open = most_left > -INFINITY && most_left >= least_kept;
      again = open && p.softmax;
      if (open && !p.softmax) {
        // The groups about the line in 64 bits, from the experts that may be their largest (softmax needs
        // the row's sum for it: the whole row).  The others stay on the side where they are.
        const bool near = kept ? r.low <= most_left : left && r.high >= least_kept;
        const float least = p.group_top == 2 && b > -INFINITY ? b : a;
        Mask<V> mask = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float k = value_of(key[i]), c = p.bias ? k : sigmoid_order(k);
          if (near && i < count && k > -INFINITY && (c >= least || close_(least, c, 2.f, inv))) mask |= Mask<V>(1) << i;
        }
        double2 t = top2_64(p, row, first, mask);
        merge_top2(t.x, t.y, p.lanes_log2);
        const double exact = group_value(t.x, t.y, p.group_top);
        const uint32_t nears = __ballot_sync(kAll, near), keeps = __ballot_sync(kAll, kept);
        int before = 0;
        for (int g = 0; g < p.groups; ++g) {
          const int from = g << p.lanes_log2;
          const double v = __shfl_sync(kAll, exact, from);
          before += nears >> from & 1 ? v > exact || (v == exact && g < group) : (int)(keeps >> from & 1);
        }
        if (near) rank = before;
      }
    }
    if (rank >= p.top_groups || group >= p.groups) {
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = kNone;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) pos[i] = i;
  sort_keys<V>(key, pos);
  int chosen = -1, its_key = kNone, next_key = kNone;
  auto take = [&](int j) {  // the best that is left, into lane j
    const int all = warp_max(key[0]);
    const int owner = __ffs(__ballot_sync(kAll, key[0] == all)) - 1;
    const int e = __shfl_sync(kAll, first + pos[0], owner);
    if (lane == j && all > kNone) chosen = e, its_key = all;
    const bool mine = lane == owner;
#pragma unroll
    for (int i = 0; i + 1 < V; ++i) key[i] = mine ? key[i + 1] : key[i], pos[i] = mine ? pos[i + 1] : pos[i];
    if (mine) key[V - 1] = kNone;
  };
  for (int j = 0; j < p.top_k; ++j) take(j);
  if (p.bias && !again) {
    // neighbours of the order, the last chosen and the first left among them
    next_key = warp_max(key[0]);
    const int below = __shfl_down_sync(kAll, its_key, 1);
    const int after = lane == p.top_k - 1 ? next_key : below;
    bool tie = lane < p.top_k && after > kNone && close_(value_of(its_key), value_of(after), 2.f, inv);
    if (__any_sync(kAll, tie)) {
      const int owner = __ffs(__ballot_sync(kAll, key[0] == next_key)) - 1;
      const int extra = next_key > kNone ? __shfl_sync(kAll, first + pos[0], owner) : -1;
      // equal logits and biases are a true tie, which stands as it is
      const int mine = lane < p.top_k ? chosen : extra;
      const float zm = mine >= 0 ? logit(row, mine) : 0.f, bm = mine >= 0 ? __ldg(p.bias + mine) : 0.f;
      const float zn = __shfl_down_sync(kAll, zm, 1), bn = __shfl_down_sync(kAll, bm, 1);
      const float ze = extra >= 0 ? logit(row, extra) : 0.f, be = extra >= 0 ? __ldg(p.bias + extra) : 0.f;
      const bool last_lane = lane == p.top_k - 1;
      const bool same = zm == (last_lane ? ze : zn) && bm == (last_lane ? be : bn);
      const bool at_end = last_lane && tie && same;
      tie = tie && !same;
      if (__any_sync(kAll, at_end)) {
        // behind a true tie of the last chosen with the first left another may stand who is close, and not equal
        const float zl = __shfl_sync(kAll, zm, p.top_k - 1), bl = __shfl_sync(kAll, bm, p.top_k - 1);
        const float cl = value_of(__shfl_sync(kAll, its_key, p.top_k - 1));
        bool other = false;
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (key[i] > kNone && close_(cl, value_of(key[i]), 2.f, inv))
            other = other || logit(row, first + pos[i]) != zl || __ldg(p.bias + first + pos[i]) != bl;
        const bool any_other = __any_sync(kAll, other);  // (every lane votes)
        tie = tie || (any_other && last_lane);
      }
    }
    if (__any_sync(kAll, tie)) {
      // one more, and who stands behind it; then, unless that one may belong among them too, only
      // these in 64 bits (softmax needs the row's sum for it: the whole row)
      const int owner = __ffs(__ballot_sync(kAll, key[0] == next_key)) - 1;
      const int extra = next_key > kNone ? __shfl_sync(kAll, first + pos[0], owner) : -1;
      if (p.top_k < 32) take(p.top_k);
      const int third = warp_max(key[0]), last = __shfl_sync(kAll, its_key, p.top_k - 1);
      if (p.softmax || p.top_k == 32 || (third > kNone && close_(value_of(last), value_of(third), 2.f, inv))) {
        again = true;
      } else {
        const int n = p.top_k + (extra >= 0 ? 1 : 0);
        double c = 0.0;
        if (lane < n && chosen >= 0) c = sigmoid((double)logit(row, chosen)) + (double)__ldg(p.bias + chosen);
        const long long k64 = lane < n && chosen >= 0 ? key64(c) : kNone64;
        int rank = 0;
        for (int j = 0; j < n; ++j) {
          const long long o = __shfl_sync(kAll, k64, j);
          const int oe = __shfl_sync(kAll, chosen, j);
          rank += o > k64 || (o == k64 && oe < chosen);
        }
        int sorted = -1;
        for (int j = 0; j < n; ++j) {
          const int to = __shfl_sync(kAll, rank, j), e = __shfl_sync(kAll, chosen, j);
          if (lane == to) sorted = e;
        }
        chosen = lane < p.top_k ? sorted : -1;
      }
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
  p.bias_vec = p.each == v && p.per % v == 0 && reinterpret_cast<uintptr_t>(p.bias) % (v < 4 ? 4 * v : 16) == 0;
  switch (v) {
    case 1: return launch_route<1, T>(p, sms, stream);
    case 2: return launch_route<2, T>(p, sms, stream);
    case 4: return launch_route<4, T>(p, sms, stream);
    case 8: return launch_route<8, T>(p, sms, stream);
    case 16: return launch_route<16, T>(p, sms, stream);
    case 32: return launch_route<32, T>(p, sms, stream);
    case kMaxEach: return launch_route<kMaxEach, T>(p, sms, stream);
    default: return cudaErrorInvalidValue;  // (1024 experts in 32 groups at most leave no such lane)
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
