// The product kernel of fp4_gemm.cuh on operands quantised before.

#include "fp4_gemm.cuh"

namespace b4 {

// grid: CTAs (splits == 1) or clusters, one for each unit the call can have.
cudaError_t launch_fp4_gemm(const Fp4GemmParams& p, int fmt, int grid, int splits, bool pdl, cudaStream_t stream) {
  return fp4::with_forms(p, fmt, [&](auto f, auto out, auto ragged) {
    return splits > 1 ? fp4::launch<f.value, out.value, ragged.value, true, false>(p, grid, splits, pdl, stream)
                      : fp4::launch<f.value, out.value, ragged.value, false, false>(p, grid, 1, pdl, stream);
  });
}

}  // namespace b4
