// Grouped GEMM instantiations: fp32, fused gate+up SwiGLU that keeps both projections in 8 bits.
#include "grouped_gemm.hpp"

namespace moe {

hipError_t launch_gemm_f32_gateup_save(int BM, const GemmArgs& a, hipStream_t stream) {
  return gemm::dispatch_bm<TF32, true, false, true>(BM, a, stream);
}

}  // namespace moe
