// Kernel launchers of libmoe (internal; called by api.cpp after validation).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

// Entries handled by one block of the counting and scatter kernels.
constexpr int kCountChunk = 2048;
// Tokens per block of the router kernel.
constexpr int kRouteSmallBatch = 2048;  // below: 4 tokens per router workgroup, else 16

hipError_t launch_route(int dtype, const void* x, const void* w_router, const float* bias, int T, int d,
                        int E, int k, int32_t* topk_ids, float* topk_w, hipStream_t stream);

hipError_t launch_count(const int32_t* ids, int Tk, int E, int nblk, int32_t* block_counts,
                        uint32_t* block_err, int32_t* token_of, int64_t fill_rows, hipStream_t stream);

struct ScanArgs {
  int32_t* block_counts;  // [nblk][E] in: per-block counts; out: per-block base ranks
  const uint32_t* block_err;
  int nblk, E, C, BM, max_tiles;
  int32_t* counts;
  int32_t* offsets;
  int32_t* spill_counts;
  int32_t* spill_offsets;
  int32_t* tile_off;  // [2][E+1]
  int32_t* tile_map;  // [2][max_tiles][4]
  int32_t* n_tiles;   // [2]
  uint32_t* err_flags;
};
hipError_t launch_scan(const ScanArgs& a, hipStream_t stream);

// Entries up to which one 1024-thread block does the whole dispatch.
constexpr int kSmallDispatch = 16384;
// Limits of the one-wavefront dispatch (a decode step): entries, experts, rows.
constexpr int kTinyDispatchEntries = 64;
constexpr int kTinyDispatchExperts = 64;
constexpr int kTinyDispatchRows = 4096;
__host__ __device__ inline bool tiny_dispatch(int Tk, int E, int64_t rows) {
  return Tk <= kTinyDispatchEntries && E <= kTinyDispatchExperts && rows <= kTinyDispatchRows;
}

struct SmallDispatchArgs {
  const int32_t* ids;
  int Tk, k, E, C, BM, max_tiles;
  int64_t rows;  // R: every row's token_of is reset to -1 first
  int32_t* counts;
  int32_t* offsets;
  int32_t* spill_counts;
  int32_t* spill_offsets;
  int32_t* row_of;
  int32_t* token_of;
  int32_t* tile_off;
  int32_t* tile_map;
  int32_t* n_tiles;
  uint32_t* err_flags;
};
hipError_t launch_dispatch_small(const SmallDispatchArgs& a, hipStream_t stream);

// Tokens up to which a batch with router weights (E <= 64) is routed and
// dispatched by one workgroup in one launch (a.ids must be topk_ids).
constexpr int kRouteDispatchTokens = 16;
hipError_t launch_route_dispatch(int dtype, const void* x, const void* w_router, const float* bias, int T, int d,
                                 int E, int k, int32_t* topk_ids, float* topk_w, const SmallDispatchArgs& a,
                                 hipStream_t stream);

hipError_t launch_scatter(const int32_t* ids, int Tk, int k, int E, int C, int nblk,
                          const int32_t* block_base, const int32_t* offsets, const int32_t* spill_offsets,
                          int32_t* row_of, int32_t* token_of, hipStream_t stream);

hipError_t launch_gather(const void* x, const int32_t* row_of, int Tk, int k, int64_t row_bytes,
                         void* x_perm, hipStream_t stream);

// One 16-byte piece per thread: groups of 16 rows of `row_bytes` bytes into
// 1024-byte blocks (see MOE_LAYOUT_BLOCKED16).
hipError_t launch_pack_blocked16(const void* src, void* dst, int64_t groups, int64_t row_bytes, hipStream_t stream);

hipError_t launch_combine(int dtype, const void* y, const float* topk_w, const int32_t* row_of, int T,
                          int k, int d, void* out, hipStream_t stream);

struct GemmArgs {
  const void* act;           // [R][K] activation rows, or (act_rows set) the source rows they come from
  const int32_t* act_rows;   // null, or [R]: row r of the activations is row act_rows[r] of `act`
  int act_nrows;             // rows of `act` when act_rows is set
  const void* w0;            // [E][N][K]
  const void* w1;            // [E][N][K] (gate+up: the up projection), else null
  const float* s0;           // fp8 weights: [E][N] per-channel scales of w0, else null
  const float* s1;           // fp8 weights: [E][N] per-channel scales of w1, else null
  void* out;                 // [R][N]
  const int32_t* tile_off;   // [E+1] of this pass
  const int32_t* tile_map;   // [max_tiles][4] of this pass
  const int32_t* n_tiles;    // [1] of this pass
  // Both passes of the capacity mode in one launch: the overflow pass's tile
  // offsets, map and count (else null).  Each expert's overflow tiles follow
  // its first-pass tiles, so both read its weights while they are in L2.
  const int32_t* tile_off2;
  const int32_t* tile_map2;
  const int32_t* n_tiles2;
  int E, K, N;
  int max_tiles;             // tiles of the map(s) the grid must cover
  int skew_map;              // 1: uneven tile counts per expert deal chunks of units to the XCDs in turn
  int blocked16;             // 1: weights in 16-row blocked order (moe_weight_layout_t)
  int wide;                  // 1: bf16 gate+up on the 160-row map may take the two-width kernel (one pass)
  float* kpart;              // non-null: bf16 down on the 160-row map splits K in two; fp32 partial sums,
                             // plane ks of [2][R][N] (kplane floats per plane)
  size_t kplane;
  // Down GEMM of a decode batch (16-row tiles, one pass) with the combine
  // folded in: non-null comb_out makes each workgroup compute its column
  // slice of y for every tile of the map, store it, and then weight it into
  // out[t] = sum_j comb_w[t k + j] y[comb_row_of[t k + j]] for that slice.
  void* comb_out;
  const float* comb_w;
  const int32_t* comb_row_of;
  int comb_T, comb_k;
  // Gate+up that also keeps both projections in 8 bits (moe_saved8_t): codes
  // [R][N] and exponents [R][N / 16], else null.
  int8_t* save_gate;
  int8_t* save_up;
  uint8_t* save_gate_exp;
  uint8_t* save_up_exp;
};

// y[r] = rounded(part[0][r] + part[1][r]) for every row r with token_of[r] >= 0:
// the sum of the two K ranges of the split down GEMM, added in that order.
// combine straight from the split down GEMM's fp32 planes part[2][R][d]
// (plane = R*d floats): y rows formed as launch_k_split_finish forms them are
// stored and weighted into out as launch_combine weights them.
hipError_t launch_combine_split(int dtype, const float* part, size_t plane, const float* topk_w,
                                const int32_t* row_of, int T, int k, int d, void* y, void* out, hipStream_t stream);
hipError_t launch_k_split_finish(int dtype, const float* part, size_t plane, const int32_t* token_of, int64_t rows,
                                 int N, void* y, hipStream_t stream);

// Bytes of the device scratch array of moe_forward_noalloc (MOE_NOALLOC_SCRATCH_BYTES).
constexpr size_t kNoallocScratchBytes = size_t(128) << 20;

// Device address of that array on the current device, taken once per device
// (hipGetSymbolAddress) and kept; never the array's host-side name.
hipError_t noalloc_scratch(void** out);

hipError_t launch_gemm_bf16_gateup(int BM, const GemmArgs& a, hipStream_t stream);
hipError_t launch_gemm_bf16_gateup_save(int BM, const GemmArgs& a, hipStream_t stream);
hipError_t launch_gemm_f32_gateup_save(int BM, const GemmArgs& a, hipStream_t stream);
hipError_t launch_gemm_bf16_down(int BM, const GemmArgs& a, hipStream_t stream);
hipError_t launch_gemm_f32_gateup(int BM, const GemmArgs& a, hipStream_t stream);
hipError_t launch_gemm_f32_down(int BM, const GemmArgs& a, hipStream_t stream);
hipError_t launch_gemm_fp8w_gateup(int BM, const GemmArgs& a, hipStream_t stream);
hipError_t launch_gemm_fp8w_down(int BM, const GemmArgs& a, hipStream_t stream);

inline hipError_t launch_grouped_gemm(int dtype, bool gated, int BM, const GemmArgs& a, hipStream_t stream) {
  if (gated && a.save_gate != nullptr)
    return dtype == 1 ? launch_gemm_bf16_gateup_save(BM, a, stream) : launch_gemm_f32_gateup_save(BM, a, stream);
  if (a.s0 != nullptr) return gated ? launch_gemm_fp8w_gateup(BM, a, stream) : launch_gemm_fp8w_down(BM, a, stream);
  if (dtype == 1) return gated ? launch_gemm_bf16_gateup(BM, a, stream) : launch_gemm_bf16_down(BM, a, stream);
  return gated ? launch_gemm_f32_gateup(BM, a, stream) : launch_gemm_f32_down(BM, a, stream);
}

// ---- backward pass ----

// dy[row_of[f]] = w_f dout[f / k] and dw_f = <dout[f / k], y[row_of[f]]>.
hipError_t launch_combine_backward(int dtype, const void* dout, const void* y, const float* topk_w,
                                   const int32_t* row_of, int T, int k, int d, void* dy, float* dw,
                                   hipStream_t stream);

// The end of the router's gradients: the weight gradient's partial sums over
// `ranges` token ranges [ranges][E][d], and the bias gradient's over the K steps
// [steps][E].  Nothing with part and dbias null.
struct RouteFinish {
  const float* part;
  const float* sums;
  void* dw_router;
  float* dbias;
  int ranges, steps;
  int sum_blocks, blocks;  // workgroups (set by the launcher)
};

// dx[t] = sum_j dx_perm[row_of[t k + j]], plus, with dz set, sum_j dz[t k + j]
// w_router[ids[t k + j]] (dx_perm may then be null); and fin's work.  f32: dx_perm
// is fp32 whatever the type.
hipError_t launch_token_backward(int dtype, const void* dx_perm, bool f32, const int32_t* row_of, const float* dz,
                                 const int32_t* ids, const void* w_router, int T, int k, int d, int E, void* dx,
                                 RouteFinish fin, hipStream_t stream);

// dz_f = w_f (dw_f - sum_i w_i dw_i), and its dense form by K step for the
// router's weight gradient (hi, and with bf16 lo: [ceil(T / KS)][E][KS]) with
// its sums over each step's tokens ([ceil(T / KS)][E]) and which of these have an
// expert at all ([ceil(T / KS)], a bit each).
hipError_t launch_route_dz(int dtype, const int32_t* ids, const float* w, const float* dw, int T, int k, int E,
                           float* dz, void* dense_hi, void* dense_lo, float* sums, unsigned* taken,
                           hipStream_t stream);

struct RouteWgradArgs {
  const void* dz_hi;  // [steps of all tokens][E][64 bytes]
  const void* dz_lo;  // the same, or null (fp32)
  const void* x;      // [T][d]
  const unsigned* taken;  // [steps of all tokens]: which of a step's tokens have an expert, a bit each
  float* part;        // [ranges][E][d]
  int T, E, d;
  int steps;          // K steps of one range of tokens
};
// Columns of x that one workgroup of it takes, by moe_dtype_t (64 experts each).
constexpr int kRouteGradCols[2] = {64, 128};
hipError_t launch_route_wgrad_bf16(const RouteWgradArgs& a, int ranges, hipStream_t stream);
hipError_t launch_route_wgrad_f32(const RouteWgradArgs& a, int ranges, hipStream_t stream);

// Values of the 8-bit projections of every live row (bf16 holds each exactly).
hipError_t launch_saved8_unpack(const int8_t* g8, const int8_t* u8, const uint8_t* gx, const uint8_t* ux,
                                const int32_t* token_of, int64_t rows, int F, void* gate, void* up,
                                hipStream_t stream);

// Where each expert's rows lie (C = 0: one run from offsets[e]).
struct GradRows {
  const int32_t* counts;
  const int32_t* offsets;
  const int32_t* spill_offsets;
  int E, C;
};

struct DgradArgs {
  GradRows rows;
  // activations in panels ([columns of 64 bytes][R][64 bytes]; `panel` bytes each)
  const void* a0;  // K columns
  const void* a1;  // second activation operand, or null
  size_t panel;
  const void* b0;  // [E][K][N]
  const void* b1;
  int K, N, blocked16;
  void* out;   // [R][N]
  int out_f32;  // whether out is fp32 whatever the type
  // with the SwiGLU's gradient (out unused): a0 = dout, K = d, N = F
  const float* wrow;
  const int8_t* g8;
  const int8_t* u8;
  const uint8_t* gx;
  const uint8_t* ux;
  void* dg;    // panels
  void* du;
  void* hw;    // w_r h, or null
  float* dot;  // [R][dot_ld] partial sums of <D, h>
  int dot_ld;
  // without it: dw[f] = the sum of dot's row row_of[f] (0 where that is -1)
  const int32_t* row_of;
  int entries;
  float* dw;
};

// Division of n < 2^31 by d: m = (2^32 - 1) / d puts n m / 2^32 between n / d - 1/2
// and n / d, so its whole part is the quotient or one less.
struct Divisor {
  unsigned d, m;
};
inline Divisor divisor(unsigned d) { return Divisor{d, 0xffffffffu / d}; }

// One weight gradient, by expert P^T Q: [E][M][N], or with swap [E][N][M].
struct WgradProduct {
  const void* P;  // [steps][M][64 bytes]
  const void* Q;  // panels of N columns
  void* out;
  int swap;
  // set by the launcher: the product's first unit inside an expert, its tiles down
  // out's rows, the units of a band of kBand of them, those of the last band
  int first, RT;
  Divisor band, last;
};

constexpr int kBand = 2;
struct WgradArgs {
  GradRows rows;
  int n;          // products
  WgradProduct prod[3];
  int M, N;
  size_t panel;   // bytes of a panel
  Divisor per_e;  // units of an expert (set by the launcher, as the next)
  int units;
  int blocked16;
};

// x and dout in expert order, dout in panels ([row bytes / 64][R][64 bytes]) and
// both, unless null, in K steps of the weight gradients ([steps][d][64 bytes], an
// expert's rows from a step of its own on, either run of them), and the
// routing weight of each row.  Rows without a token are left as they are.
struct GatherArgs {
  GradRows rows;
  const void* x;  // [T][d]
  const void* dout;
  const float* topk_w;
  const int32_t* token_of;
  const int32_t* row_of;
  int k, d;
  size_t panel;
  char* x_steps;
  char* dout_steps;
  char* dout_panels;
  float* wrow;
};
hipError_t launch_gather_backward(int dtype, const GatherArgs& a, long long max_steps, hipStream_t stream);
hipError_t launch_gather_backward_bf16(const GatherArgs& a, long long max_steps, hipStream_t stream);
hipError_t launch_gather_backward_f32(const GatherArgs& a, long long max_steps, hipStream_t stream);

// Columns of one partial sum of <D, h>, by the mean row count of an expert, and
// the tile of the first (dh) or second data gradient with N columns.
int dgrad_dot_cols(int dtype, int mean);
struct DgradTile {
  int rows, cols;
};
DgradTile dgrad_tile(int dtype, bool dh, int mean, int E, int N);
// max_tiles: row tiles of tile.rows at most, over all experts
hipError_t launch_dgrad(int dtype, bool dh, DgradTile tile, const DgradArgs& a, long long max_tiles,
                        hipStream_t stream);
hipError_t launch_wgrad(int dtype, const WgradArgs& a, hipStream_t stream);
hipError_t launch_dgrad_bf16(bool dh, DgradTile tile, const DgradArgs& a, long long max_tiles, hipStream_t stream);
hipError_t launch_dgrad_f32(bool dh, DgradTile tile, const DgradArgs& a, long long max_tiles, hipStream_t stream);
hipError_t launch_wgrad_bf16(const WgradArgs& a, hipStream_t stream);
hipError_t launch_wgrad_f32(const WgradArgs& a, hipStream_t stream);

}  // namespace moe
