// Device code of the FP8 quantisation, shared by the quantiser and by the product kernel that
// quantises a few rows for itself: scales of blocks, codes.
#pragma once

#include "fp4_quant.cuh"
#include "fp8.cuh"

namespace b4 {
namespace fp8q {

using namespace fp4q;

// The scale of a block from the bits of its largest magnitude.
template <bool POW2>
__device__ __forceinline__ float block_scale(uint32_t a) {
  if (a == 0) return 1.f;
  if (a >= kInfBits) return __uint_as_float(0x7fffffffu);
  if (POW2) {
    const int e = (int)(a >> 23) - 8 + ((a & 0x7fffffu) > 0x600000u);  // 448 = 1.75 2^8
    return __uint_as_float((uint32_t)max(e, 1) << 23);
  }
  return fmaxf(__fdiv_rn(__uint_as_float(a), 448.f), 0x1p-126f);
}

// Sixteen codes of a chunk under the scale s.
template <bool POW2, typename C>
__device__ __forceinline__ uint4 encode8(const C& h, float s) {
  float2 q[8];
  if (POW2 && s == s) {
    const float inv = __uint_as_float((254u << 23) - __float_as_uint(s));
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 x = h.pair(j);
      q[j] = make_float2(x.x * inv, x.y * inv);
    }
  } else if (s >= 0x1p-80f && s <= 0x1p80f) {
    const Recip r = recip(s);
    const uint64_t y = pack2(r.y, r.y), z = pack2(r.z, r.z);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 x = h.pair(j);
      const uint64_t xx = pack2(x.x, x.y);
      q[j] = unpack2(fma2(xx, y, mul2(xx, z)));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 x = h.pair(j);
      q[j] = s == s ? make_float2(true_quotient(x.x, s), true_quotient(x.y, s)) : make_float2(s, s);
    }
  }
  uint32_t w[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = __nv_cvt_float2_to_fp8x2(q[j], __NV_SATFINITE, __NV_E4M3);
  return make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
}

}  // namespace fp8q
}  // namespace b4
