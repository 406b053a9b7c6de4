// Instantiations of the tcgen05 GEMM with the log-probability epilogues: the row sums
// with the ranking, and the gradient G from per-token upstream gradients.
//
// Bound by the tensor cores: 8192 tokens, D = 4096, V = 128256 with 5 alternatives 4.65 ms for the
// call (1850 TFLOP/s); 4096 tokens, D = 2048, V = 32000 forward and backward 1.28 ms (four products,
// 1673 TFLOP/s).
#include "flce_gemm.cuh"
#include "flce_internal.h"

namespace flce {

cudaError_t launch_gemm_logp(const CUtensorMap& a, const CUtensorMap& b, const GemmParams& p,
                             int grid, cudaStream_t stream) {
  GemmArgs g{};  // no output map: this epilogue writes no tiles
  g.a = a;
  g.b = b;
  g.p = p;
  return p.top_k > 0 ? launch_gemm<EPI_LOGP_TOP, 2, 0, 0>(g, g, grid, stream)
                     : launch_gemm<EPI_LOGP, 2, 0, 0>(g, g, grid, stream);
}

cudaError_t launch_gemm_logp_grad(int cta_group, const CUtensorMap& a, const CUtensorMap& b,
                                  const CUtensorMap& c, const GemmParams& p, int grid,
                                  cudaStream_t stream, int fp8) {
  if (cta_group != 2 || fp8) return cudaErrorInvalidValue;  // only the bf16 pair kernel is built
  GemmArgs g{};
  g.a = a;
  g.b = b;
  g.c = c;
  g.p = p;
  return launch_gemm<EPI_LOGP_GRAD, 2, 0, 0>(g, g, grid, stream);
}

}  // namespace flce
