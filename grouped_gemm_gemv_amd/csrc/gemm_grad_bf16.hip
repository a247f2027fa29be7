// Backward grouped GEMM instantiations: bf16.
#include "gemm_grad.hpp"

namespace moe {
namespace {
using namespace grad;
// data gradients, by rows and columns of a tile
using D256 = Tile<TBF16, 256, 256, 2, 4, kPanelK, kRows, 4, 1, true>;
using D192 = Tile<TBF16, 192, 256, 2, 4, kPanelK, kRows, 5, 1, true>;
using D256N = Tile<TBF16, 256, 128, 4, 2, kPanelK, kRows, 5, 1, true>;
using D128 = Tile<TBF16, 128, 128, 2, 2, kPanelK, kRows, 4, 2, false>;
using D64 = Tile<TBF16, 64, 128, 1, 4, kPanelK, kRows, 4, 2, false>;
// weight gradients, whatever the rows: with 16 rows per expert, when the stores of
// the gradients are all there is, 128 x 128 tiles (two workgroups for each compute
// unit) took 904 us at the Mixtral shape and 956 against 747 us with 64 rows
using W256 = Tile<TBF16, 256, 256, 2, 4, kSteps, kPanelR, 4, 1, true>;
// router weight gradient: experts by columns
using R64 = Tile<TBF16, 64, 128, 1, 4, kPanelK, kRows, 4, 3, false>;

template <bool DH>
hipError_t dgrad_tiles(DgradTile t, const DgradArgs& a, long long max_tiles, hipStream_t stream) {
  if (t.rows == D64::BM) return launch_dgrad_cfg<TBF16, D64, DH>(a, max_tiles, stream);
  if (t.rows == D128::BM) return launch_dgrad_cfg<TBF16, D128, DH>(a, max_tiles, stream);
  if (t.rows == D192::BM) return launch_dgrad_cfg<TBF16, D192, DH>(a, max_tiles, stream);
  if (t.rows != D256::BM) return hipErrorInvalidValue;
  return t.cols == D256N::BN ? launch_dgrad_cfg<TBF16, D256N, DH>(a, max_tiles, stream)
                             : launch_dgrad_cfg<TBF16, D256, DH>(a, max_tiles, stream);
}
}  // namespace

hipError_t launch_dgrad_bf16(bool dh, DgradTile tile, const DgradArgs& a, long long max_tiles, hipStream_t stream) {
  return dh ? dgrad_tiles<true>(tile, a, max_tiles, stream) : dgrad_tiles<false>(tile, a, max_tiles, stream);
}

hipError_t launch_wgrad_bf16(const WgradArgs& a, hipStream_t stream) {
  return launch_wgrad_cfg<TBF16, W256>(a, stream);
}

hipError_t launch_gather_backward_bf16(const GatherArgs& a, long long max_steps, hipStream_t stream) {
  return launch_gather_cfg<TBF16, W256>(a, max_steps, stream);
}

hipError_t launch_route_wgrad_bf16(const RouteWgradArgs& a, int ranges, hipStream_t stream) {
  hipLaunchKernelGGL((route_wgrad_kernel<TBF16, R64>),
                     dim3((a.d + R64::BN - 1) / R64::BN, (a.E + R64::BM - 1) / R64::BM, ranges), dim3(R64::NTH), 0,
                     stream, a);
  return hipGetLastError();
}

}  // namespace moe
