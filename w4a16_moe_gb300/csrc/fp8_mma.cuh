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
// D (+)= A B^T, both operands in shared memory with the 128-byte swizzle.
__device__ __forceinline__ void mma_fp8(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, "
      "%5};\n\ttcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHiSw128)
      : "memory");
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

// Four neighbouring scales of a row of kb, from block b on (0 past the last).
__device__ __forceinline__ float4 load_scales(const float* row, int b, int kb, bool vec) {
  if (vec && b < kb) return __ldg(reinterpret_cast<const float4*>(row + b));
  return make_float4(b < kb ? __ldg(row + b) : 0.f, b + 1 < kb ? __ldg(row + b + 1) : 0.f,
                     b + 2 < kb ? __ldg(row + b + 2) : 0.f, b + 3 < kb ? __ldg(row + b + 3) : 0.f);
}

constexpr int kStagePiece = 32 * 64;  // bytes a warp stages at a time: 64 of each of 32 rows

// Columns [n, n + 2 C) of 32 rows, a lane's in v, to rows `to` of the output (-1: none).  In
// 16-byte pieces they go through the warp's staging area, 64 bytes of a row at a time
// (pieces swizzled by the row), so that four neighbouring lanes write 64 bytes of one row: a
// lane writing its own row touches 32 lines an instruction (4096 cycles for a unit of
// 256 x 256, during which the tensor core runs out of accumulators).
template <int OUT, int C>
__device__ __forceinline__ void store_rows(const Fp4GemmParams& g, int to, int n, const float2 (&v)[C], uint8_t* stage,
                                           int lane) {
  if (g.vec) {
    constexpr int kCols = OUT == 2 ? 16 : 32;  // of a piece
    uint8_t* mine = stage + lane * 64;
    const int key = (lane >> 1) & 3;
    const uint8_t* from = stage + (lane >> 2) * 64;
#pragma unroll
    for (int c = 0; c < 2 * C / kCols; ++c) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint4 w;
        if constexpr (OUT == 2) {
          const float2 x = v[8 * c + 2 * i], y = v[8 * c + 2 * i + 1];
          w = make_uint4(__float_as_uint(x.x), __float_as_uint(x.y), __float_as_uint(y.x), __float_as_uint(y.y));
        } else {
          const float2* x = v + 16 * c + 4 * i;
          w = make_uint4(pack16<OUT>(x[0]), pack16<OUT>(x[1]), pack16<OUT>(x[2]), pack16<OUT>(x[3]));
        }
        *reinterpret_cast<uint4*>(mine + ((i ^ key) << 4)) = w;
      }
      __syncwarp();
      const int col = n + kCols * c + (kCols / 4) * (lane & 3);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 8 * i + (lane >> 2);
        const int o = __shfl_sync(0xffffffffu, to, row);
        const uint4 w = *reinterpret_cast<const uint4*>(from + 512 * i + (((lane & 3) ^ ((row >> 1) & 3)) << 4));
        if (o >= 0 && col < g.n)
          *reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(g.out) + ((int64_t)o * g.out_stride + col) * (OUT == 2 ? 4 : 2)) = w;
      }
      __syncwarp();
    }
  } else if (to >= 0) {
    const int64_t at = (int64_t)to * g.out_stride;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      if (n + 2 * i < g.n) store_out(g, at + n + 2 * i, v[i].x);
      if (n + 2 * i + 1 < g.n) store_out(g, at + n + 2 * i + 1, v[i].y);
    }
  }
}

// The entry of operand row `at` in out_rows, read before its sums are made and looked at after (a load
// takes a microsecond and more under the operands' traffic), and its output row, -1 where it is dropped.
__device__ __forceinline__ int output_entry(const Fp4GemmParams& g, int at, bool live) {
  return !live ? -1 : g.out_rows ? __ldg(g.out_rows + at) : at;
}
__device__ __forceinline__ int output_row(const Fp4GemmParams& g, int entry) {
  return entry < g.out_rows_end ? entry : -1;
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
