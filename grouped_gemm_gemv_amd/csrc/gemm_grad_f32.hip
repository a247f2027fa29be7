// Backward grouped GEMM instantiations: fp32, and the tile choice of both types.
#include "gemm_grad.hpp"

namespace moe {
namespace {
using namespace grad;
// fp32 MFMAs run at a sixteenth of the bf16 rate, so small tiles keep up (a ring
// of 8 stages gained nothing at the tiny layer, 64 tokens of 128 columns)
using D64 = Tile<TF32, 64, 64, 2, 2, kPanelK, kRows, 4, 4, false>;
using W64 = Tile<TF32, 64, 64, 2, 2, kSteps, kPanelR, 4, 4, false>;
}  // namespace

hipError_t launch_dgrad_f32(bool dh, int BM, const DgradArgs& a, long long max_tiles, hipStream_t stream) {
  if (BM != D64::BM) return hipErrorInvalidValue;
  return dh ? launch_dgrad_cfg<TF32, D64, true>(a, max_tiles, stream)
            : launch_dgrad_cfg<TF32, D64, false>(a, max_tiles, stream);
}

hipError_t launch_wgrad_f32(const WgradArgs& a, hipStream_t stream) {
  return launch_wgrad_cfg<TF32, W64>(a, stream);
}

hipError_t launch_gather_backward_f32(const GatherArgs& a, long long max_steps, hipStream_t stream) {
  return launch_gather_cfg<TF32, W64>(a, max_steps, stream);
}

hipError_t launch_route_wgrad_f32(const RouteWgradArgs& a, int ranges, hipStream_t stream) {
  hipLaunchKernelGGL((route_wgrad_kernel<TF32, D64>),
                     dim3((a.d + D64::BN - 1) / D64::BN, (a.E + D64::BM - 1) / D64::BM, ranges), dim3(D64::NTH), 0,
                     stream, a);
  return hipGetLastError();
}

// Rows of a data gradient's tile.  bf16: 64 rows (three workgroups for each
// compute unit) where an expert's rows fit one such tile; past 48 rows on
// average many do not, and their weights would be read twice.  Both data
// gradients, 64- against 256-row tiles, us: the Mixtral shape with 32 rows for each
// expert 202 + 307 against 193 + 387, with 64 rows 269 + 497 against 205 + 402; 64
// experts of d = 2048, F = 1408 with 48 rows 96 + 162 against 121 + 138, of
// d = 3584, F = 2560 with 64 rows 331 + 589 against 291 + 446.
int dgrad_tile_rows(int dtype, int mean) { return dtype == 1 && mean > 48 ? 256 : 64; }

// one partial sum per wavefront column
int dgrad_dot_cols(int dtype, int mean) { return dgrad_tile_rows(dtype, mean) == 256 ? 64 : 32; }

hipError_t launch_dgrad(int dtype, bool dh, int mean, const DgradArgs& a, long long max_tiles, hipStream_t stream) {
  const int BM = dgrad_tile_rows(dtype, mean);
  return dtype == 1 ? launch_dgrad_bf16(dh, BM, mean, a, max_tiles, stream)
                    : launch_dgrad_f32(dh, BM, a, max_tiles, stream);
}

hipError_t launch_gather_backward(int dtype, const GatherArgs& a, long long max_steps, hipStream_t stream) {
  return dtype == 1 ? launch_gather_backward_bf16(a, max_steps, stream)
                    : launch_gather_backward_f32(a, max_steps, stream);
}

hipError_t launch_wgrad(int dtype, const WgradArgs& a, hipStream_t stream) {
  return dtype == 1 ? launch_wgrad_bf16(a, stream) : launch_wgrad_f32(a, stream);
}

}  // namespace moe
