// Grouped GEMM instantiations: bf16, fused gate+up SwiGLU that keeps both projections in 8 bits.
#include "grouped_gemm.hpp"

namespace moe {

hipError_t launch_gemm_bf16_gateup_save(int BM, const GemmArgs& a, hipStream_t stream) {
  return gemm::dispatch_bm<TBF16, true, false, true>(BM, a, stream);
}

}  // namespace moe
