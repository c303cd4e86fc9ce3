// Device code of the FP4 quantisation, shared by the quantiser and by the product
// kernel that quantises a few rows for itself: chunks of 16 elements in registers,
// block scales, codes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include <cstring>

#include "fp4.cuh"
#include "ptx.cuh"

namespace b4 {
namespace fp4q {

__device__ __forceinline__ void from_f32(__nv_bfloat16* d, float v) { *d = __float2bfloat16_rn(v); }
__device__ __forceinline__ void from_f32(__half* d, float v) { *d = __float2half_rn(v); }
__device__ __forceinline__ void from_f32(float* d, float v) { *d = v; }

__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// N words (8 or 16) from or to consecutive global memory.  level 2: 32-byte
// aligned, 1: 16-byte.
template <int N>
__device__ __forceinline__ void load_words(const void* src, int level, uint32_t (&w)[N]) {
  if (level == 2) {
#pragma unroll
    for (int i = 0; i < N; i += 8)
      asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3]), "=r"(w[i + 4]), "=r"(w[i + 5]),
                     "=r"(w[i + 6]), "=r"(w[i + 7])
                   : "l"(reinterpret_cast<const uint32_t*>(src) + i));
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(src) + i / 4);
      w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
    }
  }
}
template <int N>
__device__ __forceinline__ void store_words(void* dst, int level, const uint32_t (&w)[N]) {
  if (level == 2) {
#pragma unroll
    for (int i = 0; i < N; i += 8)
      asm volatile("st.global.v8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(w[i]), "r"(w[i + 1]), "r"(w[i + 2]),
                   "r"(w[i + 3]), "r"(w[i + 4]), "r"(w[i + 5]), "r"(w[i + 6]), "r"(w[i + 7]),
                   "l"(reinterpret_cast<uint32_t*>(dst) + i)
                   : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      reinterpret_cast<uint4*>(dst)[i / 4] = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
  }
}

// 16 elements of a row as they are in memory.
template <typename T>
struct Raw {
  static constexpr int kWords = 16 * (int)sizeof(T) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* src, int level) {
    if (level) {
      load_words(src, level, w);
    } else {
      T e[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) e[i] = src[i];
      memcpy(w, e, sizeof(w));
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }
  __device__ __forceinline__ float2 pair(int i) const;  // elements 2i, 2i + 1
  // Bits of the largest magnitude as fp32; a NaN's bits exceed every number's, so it stays.
  __device__ __forceinline__ uint32_t amax() const;
};
template <>
__device__ __forceinline__ float2 Raw<__nv_bfloat16>::pair(int i) const {
  return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 Raw<__half>::pair(int i) const {
  return __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
}
template <>
__device__ __forceinline__ float2 Raw<float>::pair(int i) const {
  return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
}
__device__ __forceinline__ uint32_t amax16x2(const uint32_t (&w)[8]) {
  uint32_t m = w[0] & 0x7fff7fffu;
#pragma unroll
  for (int i = 1; i < 8; ++i) asm("max.u16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i] & 0x7fff7fffu));
  return max(m >> 16, m & 0xffffu);
}
template <>
__device__ __forceinline__ uint32_t Raw<__nv_bfloat16>::amax() const {
  return amax16x2(w) << 16;
}
template <>
__device__ __forceinline__ uint32_t Raw<__half>::amax() const {
  return __float_as_uint(__half2float(__ushort_as_half((unsigned short)amax16x2(w))));
}
template <>
__device__ __forceinline__ uint32_t Raw<float>::amax() const {
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) a = max(a, w[i] & 0x7fffffffu);
  return a;
}

// Chunk c of a row: as it is, or through the activation in fp32.
template <typename T, bool ACT>
struct Chunk : Raw<T> {
  __device__ __forceinline__ void get(const Fp4QuantParams& p, const T* row, int c) { this->load(row + 16 * c, p.vec); }
};
template <typename T>
struct Chunk<T, true> : Raw<float> {
  __device__ __forceinline__ void get(const Fp4QuantParams& p, const T* row, int c) {
    Raw<T> g, u;
    g.load(row + 16 * c, p.vec);
    if (p.act == 0) {
      u.load(row + p.k + 16 * c, p.vec);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 a = g.pair(i), b = u.pair(i);
        this->w[2 * i] = __float_as_uint(gated_act(a.x, b.x, p.glu));
        this->w[2 * i + 1] = __float_as_uint(gated_act(a.y, b.y, p.glu));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {  // NaN stays NaN
        const float2 a = g.pair(i);
        this->w[2 * i] = __float_as_uint(a.x < 0.f ? 0.f : a.x * a.x);
        this->w[2 * i + 1] = __float_as_uint(a.y < 0.f ? 0.f : a.y * a.y);
      }
    }
  }
};

constexpr uint32_t kInfBits = 0x7f800000u;

// The row's global scale from the bits of its largest magnitude; NaN for a row
// with an infinity or a NaN in it, whose products are NaN.
__device__ __forceinline__ float row_gs(uint32_t a) {
  if (a == 0) return 1.f;
  if (a >= kInfBits) return __uint_as_float(0x7fffffffu);
  const int j = (int)(a >> 23) - 127 - 11 + ((a & 0x7fffffu) > 0x280000u);  // 6 448 = 1.3125 2^11
  return __uint_as_float((uint32_t)(max(j, -126) + 127) << 23);
}

// A reciprocal to 46 bits: y the rounded one, z what it lacks.
struct Recip {
  float y, z;
};
__device__ __forceinline__ Recip recip(float d) {
  const float y = __frcp_rn(d);
  return Recip{y, __fmaf_rn(-y, d, 1.f) * y};
}
__device__ __forceinline__ float quotient(float a, const Recip& r) { return __fmaf_rn(a, r.y, a * r.z); }

// 6 gs and its reciprocal, for the block scales of a row.
struct RowScale {
  float gs, six;
  Recip inv;
  bool safe;  // the reciprocal's terms stay normal
  __device__ __forceinline__ explicit RowScale(float g) : gs(g) {
    six = __fmul_rn(6.f, g);
    safe = six >= 0x1p-80f && six <= 0x1p80f;
    inv = recip(safe ? six : 1.f);
  }
};

struct BlockScale {
  uint32_t code;  // the scale's byte
  float d;        // step of the codes
  Recip inv;      // its reciprocal
  int kind;       // 0: all codes zero, 1: by the reciprocal, 2: true division
};

// True divisions, for scales outside the range where the reciprocal's terms are normal
// (kept out of line: no ordinary block comes here).
static __device__ __noinline__ float true_quotient(float a, float b) { return __fdiv_rn(a, b); }

template <int FMT>
__device__ __forceinline__ BlockScale block_scale(uint32_t a, const RowScale& r) {
  BlockScale b;
  const float amax = __uint_as_float(a);
  if constexpr (FMT != 0) {
    const int e = a > kInfBits ? 255
                  : a == kInfBits ? 254
                                  : max((int)(a >> 23) - 2 + ((a & 0x7fffffu) > 0x400000u), 0);
    b.code = (uint32_t)e;
    b.d = e == 0 ? __uint_as_float(0x00400000u) : __uint_as_float((uint32_t)e << 23);  // 2^(e - 127)
    b.inv = Recip{e >= 254 ? __uint_as_float(0x00400000u) : __uint_as_float((uint32_t)(254 - e) << 23), 0.f};
    b.kind = e == 255 ? 0 : 1;
    return b;
  }
  float ratio = quotient(amax, r.inv);
  if (!(r.safe && ratio < 0x1p20f)) ratio = true_quotient(amax, r.six);
  b.code = ratio != ratio ? 0x7fu : (uint32_t)__nv_cvt_float_to_fp8(ratio, __NV_SATFINITE, __NV_E4M3);
  const float s = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)b.code, __NV_E4M3)));
  b.d = __fmul_rn(s, r.gs);
  const bool safe = b.d >= 0x1p-80f && b.d <= 0x1p80f;
  b.inv = recip(safe ? b.d : 1.f);
  b.kind = safe && amax * b.inv.y < 0x1p20f ? 1 : b.d > 0.f && a <= kInfBits ? 2 : 0;
  return b;
}

// E4M3 scales by code with their reciprocals (0 for the zero scale, whose codes
// are then zeros): under a power-of-two global scale a block's step and its
// reciprocal are these times 2^j and 2^-j, exactly.
__device__ __forceinline__ float4 e4m3_and_reciprocal(uint32_t code) {
  const float s = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)code, __NV_E4M3)));
  if (!(s > 0.f)) return make_float4(s, 0.f, 0.f, 0.f);
  const Recip r = recip(s);
  return make_float4(s, r.y, r.z, 0.f);
}

// Eight fp32 values as E2M1 codes, the first in the low nibble of byte 0.
__device__ __forceinline__ uint32_t e2m1x8(float2 a, float2 b, float2 c, float2 d) {
  uint32_t r;
  asm("{\n\t.reg .b8 p, q, r, s;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 p, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 q, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 r, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 s, %8, %7;\n\t"
      "mov.b32 %0, {p, q, r, s};\n\t}"
      : "=r"(r)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y), "f"(d.x), "f"(d.y));
  return r;
}

// E2M1 codes of a chunk, element 2j in the low nibble of byte j, by the step's
// reciprocal (MXFP4: a power of two, its products exact).
template <int FMT, typename C>
__device__ __forceinline__ uint2 encode(const C& h, const Recip& r) {
  const uint64_t y = pack2(r.y, r.y), z = pack2(r.z, r.z);
  float2 q[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 x = h.pair(j);
    const uint64_t xx = pack2(x.x, x.y);
    q[j] = unpack2(FMT == 0 ? fma2(xx, y, mul2(xx, z)) : mul2(xx, y));
  }
  return make_uint2(e2m1x8(q[0], q[1], q[2], q[3]), e2m1x8(q[4], q[5], q[6], q[7]));
}
template <typename C>
__device__ __forceinline__ uint2 encode_by_division(const C& h, float d) {
  float2 q[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 x = h.pair(j);
    q[j] = make_float2(true_quotient(x.x, d), true_quotient(x.y, d));
  }
  return make_uint2(e2m1x8(q[0], q[1], q[2], q[3]), e2m1x8(q[4], q[5], q[6], q[7]));
}

}  // namespace fp4q
}  // namespace b4
