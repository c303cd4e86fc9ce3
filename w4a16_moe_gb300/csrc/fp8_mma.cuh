// Device code shared by the FP8 product kernels: matrix instructions, promotion of a
// block's sums, rows of the output.
#pragma once

#include "fp4_mma.cuh"
#include "fp8.cuh"

namespace b4 {
namespace fp8 {

using namespace fp4;

// Instruction descriptor of kind::f8f6f4: E4M3 operands, both K-major, fp32 accumulator.
__device__ __forceinline__ constexpr uint32_t idesc_fp8(uint32_t m, uint32_t n) {
  return (1u << 4) | ((n >> 3) << 17) | ((m >> 4) << 24);
}
// D (+)= A B^T, both operands in shared memory with the 128-byte swizzle; CG CTAs of a pair.
template <int CG>
__device__ __forceinline__ void mma_fp8(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
#define FP8_MMA(group)                                                                                               \
  asm volatile(                                                                                                      \
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, " \
      "%5};\n\ttcgen05.mma.cta_group::" group ".kind::f8f6f4 [%0], x, y, %3, p;\n\t}" ::"r"(d),                     \
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHiSw128)                                                 \
      : "memory")
  if constexpr (CG == 1) FP8_MMA("1");
  else FP8_MMA("2");
#undef FP8_MMA
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
// Two sums plus two of a block's times the scale.  (float2 and the intrinsic: sums held as 64-bit
// asm operands are copied once a step.)
__device__ __forceinline__ void fma2(float2& acc, uint32_t a, uint32_t b, float s) {
  acc = __ffma2_rn(make_float2(__uint_as_float(a), __uint_as_float(b)), make_float2(s, s), acc);
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

// Calls f with the output's type and whether the rows are grouped as compile-time values.
template <typename F>
cudaError_t with_out(const Fp8GemmParams& p, F f) {
  auto by_groups = [&](auto out) { return p.g.offsets ? f(out, std::true_type{}) : f(out, std::false_type{}); };
  return p.g.out_dtype == 0   ? by_groups(std::integral_constant<int, 0>{})
         : p.g.out_dtype == 1 ? by_groups(std::integral_constant<int, 1>{})
                              : by_groups(std::integral_constant<int, 2>{});
}

}  // namespace fp8
}  // namespace b4
