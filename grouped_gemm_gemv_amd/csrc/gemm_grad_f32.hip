// Backward grouped GEMM instantiations: fp32, and the tile choice of both types.
#include "gemm_grad.hpp"

namespace moe {
namespace {
using namespace grad;
// fp32 MFMAs run at a sixteenth of the bf16 rate, so small tiles keep up (a ring
// of 8 stages gained nothing at the tiny layer, 64 tokens of 128 columns)
using D64 = Tile<TF32, 64, 64, 2, 2, kPanelK, kRows, 4, 4, false>;
using D32 = Tile<TF32, 32, 64, 1, 4, kPanelK, kRows, 4, 4, false>;
using W64 = Tile<TF32, 64, 64, 2, 2, kSteps, kPanelR, 4, 4, false>;
}  // namespace

hipError_t launch_dgrad_f32(bool dh, DgradTile tile, const DgradArgs& a, long long max_tiles, hipStream_t stream) {
  if (tile.rows == D32::BM && !dh) return launch_dgrad_cfg<TF32, D32, false>(a, max_tiles, stream);
  if (tile.rows != D64::BM) return hipErrorInvalidValue;
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

// The tile of a data gradient.  fp32: 64 x 64, but the second one (dh false) of up
// to 32 rows on average 32 x 64 with the four wavefronts side by side, each with
// half the MFMAs in a step: 246 against 334 us for 39 experts of d = 448, F = 6528
// with 7 rows, 13.7 against 14.6 for 8 of d = 128, F = 256 with 16, 76.3 against 76.5
// for 8 of d = 1024, F = 2048 with 25.  bf16, us of kernel time on each side:
//  * 64 x 128 (two workgroups for each compute unit: a third has no room in LDS, and
//    a grid of three ran its last third alone: 64 experts of d = 3584, F = 2560 with 48
//    rows 274 + 506 against 277 + 451; with room made for it 277 + 450) up to 48 rows
//    on average; past them many experts have more than one such tile
//    and their weights would be read twice.  First + second data gradient, 64-row
//    tiles against what the rules below choose.  8 experts of d = 1024, F = 2048 with
//    25 rows 12 + 30 against 18 + 38; 39 of d = 448, F = 6528 with 7 rows 54 + 116
//    against 85 + 124; 64 of d = 2048, F = 1408 with 3, 12, 24, 48 rows 72 + 133,
//    76 + 141, 80 + 145, 89 + 168 against 98 + 123, 101 + 129, 104 + 132, 112 + 140; 64 of
//    d = 3584, F = 2560 with 2, 16, 48 rows 207 + 377, 236 + 418, 278 + 452 against
//    233 + 382, 251 + 408, 274 + 439, with 64 rows 327 + 543 against 287 + 444; the
//    Mixtral shape with 1, 4, 16, 48, 64 rows 137 + 243, 186 + 292, 196 + 301,
//    225 + 312, 278 + 498 against 162 + 254, 176 + 286, 181 + 291, 196 + 308, 202 + 350:
//    ahead for small layers, many experts and a few tokens, up to 8 % behind between
//    4 and 48 rows of large experts;
//  * 256 x 128 where these make one round of the compute units at most (an
//    expert takes its mean row count and half a tile more).  256 x 256 against
//    256 x 128: second data gradient at the Mixtral shape 448 against 409 with 512
//    rows, 537 against 466 with 1024, but 600 against 823 with 2048; 16 experts of
//    d = 3584, F = 2560 with 1024 rows (more than one round) 93 against 126 and 109
//    against 162.  Up to 96 rows on average 128 x 128 instead, whose 4 wavefronts
//    need no turns.  Second data gradient, 128 x 128 against 256 x 128: the Mixtral
//    shape with 52, 64, 80, 96, 112 rows for each expert 307, 331, 355, 367, 364 against
//    398, 412, 397, 393, 423; 16 experts of d = 2048, F = 4096 with 64, 80, 96, 112 rows
//    106, 109, 116, 126 against 138, 138, 141, 134; 4 of d = 4096, F = 8192 with 64 to 112
//    rows 183 to 193 against 208 to 222.  With 128 rows, when half of the experts take
//    two such tiles, 642 against 457 and 194 against 157: 96 leaves an expert a
//    third above the mean in one tile;
//  * else 192 or 256 rows by 256, whichever takes fewer rounds times rows; 192
//    only from an eighth less on, as the lower tile does less with each byte it
//    loads.  256 against 192 rows, second data gradient at the Mixtral shape with 8192
//    rows (3 rounds either way) 1787 against 1611, with 4096 1133 against 1019;
//    first with 8192 rows (8 rounds against 11) 931 against 1018.
DgradTile dgrad_tile(int dtype, bool dh, int mean, int E, int N) {
  if (dtype != 1) return DgradTile{!dh && mean <= 32 ? 32 : 64, 64};
  if (mean <= 48) return DgradTile{64, 128};
  auto tiles = [&](int rows) { return (long long)E * std::max(mean + rows / 2, rows) / rows; };
  if (tiles(256) * ((N + 127) / 128) <= kComputeUnits) return DgradTile{mean <= 96 ? 128 : 256, 128};
  auto cost = [&](int rows) {
    return (tiles(rows) * ((N + 255) / 256) + kComputeUnits - 1) / kComputeUnits * rows;
  };
  return DgradTile{9 * cost(192) < 8 * cost(256) ? 192 : 256, 256};
}

// one partial sum per wavefront column
int dgrad_dot_cols(int dtype, int mean) { return dtype == 1 && mean > 48 ? 64 : 32; }

hipError_t launch_dgrad(int dtype, bool dh, DgradTile tile, const DgradArgs& a, long long max_tiles,
                        hipStream_t stream) {
  return dtype == 1 ? launch_dgrad_bf16(dh, tile, a, max_tiles, stream)
                    : launch_dgrad_f32(dh, tile, a, max_tiles, stream);
}

hipError_t launch_gather_backward(int dtype, const GatherArgs& a, long long max_steps, hipStream_t stream) {
  return dtype == 1 ? launch_gather_backward_bf16(a, max_steps, stream)
                    : launch_gather_backward_f32(a, max_steps, stream);
}

hipError_t launch_wgrad(int dtype, const WgradArgs& a, hipStream_t stream) {
  return dtype == 1 ? launch_wgrad_bf16(a, stream) : launch_wgrad_f32(a, stream);
}

}  // namespace moe
