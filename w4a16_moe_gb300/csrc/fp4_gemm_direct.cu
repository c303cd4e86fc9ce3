// The product kernel of fp4_gemm.cuh on rows that it quantises for itself.

#include "fp4_gemm.cuh"

namespace b4 {

// grid: CTAs (splits == 1) or clusters, one for each unit the call can have.
cudaError_t launch_fp4_gemm_direct(const Fp4GemmParams& p, int fmt, int grid, int splits, bool pdl, cudaStream_t stream) {
  return fp4::with_forms(p, fmt, [&](auto f, auto out, auto ragged) {
    return splits > 1 ? fp4::launch<f.value, out.value, ragged.value, true, true>(p, grid, splits, pdl, stream)
                      : fp4::launch<f.value, out.value, ragged.value, false, true>(p, grid, 1, pdl, stream);
  });
}

}  // namespace b4
