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

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// Of these a NaN operand gives NaN.
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max3_abs_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
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
// (the maximum of magnitudes with the operands' signs multiplied: the sign is dropped at the end)
template <>
__device__ __forceinline__ uint32_t Raw<__nv_bfloat16>::amax() const {
  uint32_t m = w[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) asm("max.NaN.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i]));
  return max(m << 16 & 0x7fff0000u, m & 0x7fff0000u);
}
template <>
__device__ __forceinline__ uint32_t Raw<__half>::amax() const {
  uint32_t m = w[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) asm("max.NaN.xorsign.abs.f16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i]));
  m = max(m >> 16 & 0x7fffu, m & 0x7fffu);
  return __float_as_uint(__half2float(__ushort_as_half((unsigned short)m)));
}
template <>
__device__ __forceinline__ uint32_t Raw<float>::amax() const {
  float a = __uint_as_float(w[0] & 0x7fffffffu);
#pragma unroll
  for (int i = 1; i < 15; i += 2) a = max3_abs_nan(a, __uint_as_float(w[i]), __uint_as_float(w[i + 1]));
  return __float_as_uint(max3_abs_nan(a, __uint_as_float(w[15]), 0.f));
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
      // g sigmoid(alpha g) (u + beta) of the clamped g and u, two columns an instruction; the
      // exponential and the reciprocal are the machine's approximations (2^-22 each), on an
      // argument rounded to fp32 (another |alpha g| 2^-23 of the exponential: 2^-20 at g = -10,
      // alpha = 1), and the sigmoid is 0 where 1 + e^(-alpha g) passes 2^126.  The codes keep
      // two bits, so an error of 2^-19 moves one only next to a tie.
      u.load(row + p.k + 16 * c, p.vec);
      const float limit = p.glu.limit, scale = -1.44269504f * p.glu.alpha;
      const uint64_t scale2 = pack2(scale, scale), beta2 = pack2(p.glu.beta, p.glu.beta), one2 = pack2(1.f, 1.f);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 a = g.pair(i), b = u.pair(i);
        const uint64_t gc = pack2(min_nan(a.x, limit), min_nan(a.y, limit));
        const uint64_t uc = pack2(max_nan(min_nan(b.x, limit), -limit), max_nan(min_nan(b.y, limit), -limit));
        const float2 t = unpack2(mul2(gc, scale2));
        const float2 d = unpack2(add2(pack2(exp2_approx(t.x), exp2_approx(t.y)), one2));
        const float2 h = unpack2(mul2(mul2(gc, pack2(rcp_approx(d.x), rcp_approx(d.y))), add2(uc, beta2)));
        this->w[2 * i] = __float_as_uint(h.x);
        this->w[2 * i + 1] = __float_as_uint(h.y);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 a = g.pair(i);
        const float x = max_nan(a.x, 0.f), y = max_nan(a.y, 0.f);
        this->w[2 * i] = __float_as_uint(x * x);
        this->w[2 * i + 1] = __float_as_uint(y * y);
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

// A reciprocal of a number from 2^-92 to 2^92, to 46 bits: y the machine's approximation
// (2^-23), z what it lacks, from the exact residual.
struct Recip {
  float y, z;
};
__device__ __forceinline__ Recip recip(float d) {
  const float y = rcp_approx(d);
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

// The number an E4M3 code without its sign stands for (not NaN): its bits are the top of an
// fp32's, but for the exponent's bias.
__device__ __forceinline__ float e4m3_value(uint32_t code) { return __uint_as_float(code << 20) * 0x1p120f; }

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
// True divisions, for steps outside the range where the reciprocal's terms are normal
// (kept out of line: no ordinary block comes here).
static __device__ __noinline__ float true_quotient(float a, float b) { return __fdiv_rn(a, b); }
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

// A quantised chunk: its codes, the byte of its scale, the step of its codes.
struct Quantized {
  uint2 w;
  uint32_t code;
  float d;
};

// Chunk h with the bits a of its block's largest magnitude, in a row of scales r.
template <int FMT, typename C>
__device__ __forceinline__ Quantized quantize_block(const C& h, uint32_t a, const RowScale& r) {
  Quantized q;
  if constexpr (FMT != 0) {
    const int e = a > kInfBits ? 255
                  : a == kInfBits ? 254
                                  : max((int)(a >> 23) - 2 + ((a & 0x7fffffu) > 0x400000u), 0);
    q.code = (uint32_t)e;
    q.d = e == 0 ? __uint_as_float(0x00400000u) : __uint_as_float((uint32_t)e << 23);  // 2^(e - 127)
    const float inv = e >= 254 ? __uint_as_float(0x00400000u) : __uint_as_float((uint32_t)(254 - e) << 23);
    q.w = encode<FMT>(h, Recip{inv, 0.f});
    if (e == 255) q.w = make_uint2(0, 0);
    return q;
  }
  const float amax = __uint_as_float(a);
  float ratio = quotient(amax, r.inv);
  if (r.safe && ratio < 0x1p20f) {  // every block, unless a scale was given that is far off
    q.code = (uint32_t)__nv_cvt_float_to_fp8(ratio, __NV_SATFINITE, __NV_E4M3);
    q.d = e4m3_value(q.code) * r.gs;
    q.w = encode<FMT>(h, recip(q.d));
    if (q.code == 0) q.w = make_uint2(0, 0);
  } else {
    // (under a global scale of zero, or one so small that 6 gs is, a zero block is zero, not 0 / 0)
    ratio = r.six == 0.f && a == 0 ? 0.f : true_quotient(amax, r.six);
    q.code = ratio != ratio ? 0x7fu : (uint32_t)__nv_cvt_float_to_fp8(ratio, __NV_SATFINITE, __NV_E4M3);
    q.d = q.code == 0x7fu ? __uint_as_float(0x7fffffffu) : __fmul_rn(e4m3_value(q.code), r.gs);
    q.w = q.d > 0.f && a <= kInfBits ? encode_by_division(h, q.d) : make_uint2(0, 0);
  }
  return q;
}

}  // namespace fp4q
}  // namespace b4
