// The product kernel of fp8_gemm.cuh on rows that it quantises for itself.

#include "fp8_gemm.cuh"

namespace b4 {

// grid: CTAs (splits == 1) or clusters, one for each unit the call can have.
cudaError_t launch_fp8_gemm_direct(const Fp8GemmParams& p, int grid, int splits, cudaStream_t stream) {
  return fp8::with_out(p, [&](auto out, auto ragged) {
    return splits > 1 ? fp8::launch<out.value, ragged.value, 32, true, true>(p, grid, splits, stream)
                      : fp8::launch<out.value, ragged.value, 32, false, true>(p, grid, 1, stream);
  });
}

}  // namespace b4
