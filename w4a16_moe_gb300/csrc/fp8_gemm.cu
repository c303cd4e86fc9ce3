// The product kernel of fp8_gemm.cuh on rows quantised before.

#include "fp8_gemm.cuh"

namespace b4 {

// rows: activation rows of a unit, 32 or 128.  grid: CTAs (splits == 1) or clusters, one for each
// unit the call can have (32 rows only).
cudaError_t launch_fp8_gemm(const Fp8GemmParams& p, int rows, int grid, int splits, cudaStream_t stream) {
  return fp8::with_out(p, [&](auto out, auto ragged) {
    constexpr int O = out.value;
    constexpr bool G = ragged.value;
    if (splits > 1) return fp8::launch<O, G, 32, true, false>(p, grid, splits, stream);
    return rows == 32 ? fp8::launch<O, G, 32, false, false>(p, grid, 1, stream)
                      : fp8::launch<O, G, 128, false, false>(p, grid, 1, stream);
  });
}

}  // namespace b4
