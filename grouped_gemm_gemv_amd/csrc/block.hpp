// Launchers of the operators around the layer (block_rows.hip) and of the
// layer for a few tokens (decode.hip); internal, called by api.cpp after
// validation.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

// Widest row of the norms: the row stays in a workgroup's registers.
constexpr int kNormMaxWidth = 16384;

// out = res + scale sigmoid(gate) drop(v), v = y r(y) post_w or y, and
// n = out r(out) next_w.  y null: out is res itself (a norm alone).
struct ResidualArgs {
  const void* res;
  const void* y;
  const void* post_w;
  const void* gate;         // [T] or [T][d], or null
  const uint64_t* rng;      // {seed, step}, or null
  const void* next_w;
  void* out;
  void* n;
  int T, d;
  int gate_full;            // gate is [T][d]
  float eps, scale;
  unsigned threshold;       // dropout: kept from this 16-bit half on (0: every one)
  float keep_scale;         // 65536 / (65536 - threshold)
};
hipError_t launch_residual(int dtype, const ResidualArgs& a, hipStream_t stream);

// The gradients of it.  x is what the forward pass left in out.
struct ResidualBackwardArgs {
  const void* x;
  const void* y;            // null: a norm alone
  const void* post_w;
  const void* gate;
  const uint64_t* rng;
  const void* next_w;       // null: no norm behind the sum
  const void* dout;         // null: zero
  const void* dn;           // null where next_w is
  void* dres;
  void* dy;
  void* dgate;              // null: not computed, as the next two
  void* dpost_w;
  void* dnext_w;
  float* part;              // [2][groups][d]: column sums of dpost_w and dnext_w
  int T, d;
  int gate_full;
  float eps, scale;
  unsigned threshold;
  float keep_scale;
};
// Workgroups of the gradient, which is also the rows of its partial sums.
int residual_backward_groups(int T, int d);
hipError_t launch_residual_backward(int dtype, const ResidualBackwardArgs& a, hipStream_t stream);

hipError_t launch_dropout(int dtype, const void* x, int64_t n, unsigned threshold, float keep_scale,
                          const uint64_t* rng, void* out, hipStream_t stream);

// ---- the layer for a few tokens ----

// Most tokens of it: the columns of one matrix instruction.
constexpr int kDecodeTokens = 16;

// What the first kernel leaves for the second besides h: the active experts in
// ascending order and each token's weight of each (0: not chosen).
struct DecodeTable {
  int n_active;
  int pad[63];
  int claimed;  // turns of the first kernel's deal that are taken
  int pad2[63];
  int expert[256];
  float weight[256][kDecodeTokens];
  int arrived[4480];  // per column tile of the second kernel: workgroups that are done (zeroed by the first)
};
// Columns of d that a workgroup of the second kernel takes.  Up to four tokens 16, the
// most workgroups; past them 64 where tiles and parts still fill the compute units,
// because every tile of columns reads all of h, from L2.  With 16 and with 64, Mixtral shape:
// one token 117 and 120 us, 5 tokens 272 and 275, 8 379 and 378, 16 465 and 450, with E4M3
// weights 1 token 69.6 and 70.4, 4 153 and 150, 8 216 and 207, 16 300 and 269; 64 experts of 2048,
// 4 tokens 70.0 and 71.2, 8 112 and 115, 16 155.6 and 155.0; of 1024, 8 tokens 62.5 and 65.4, 16
// 100 and 102 (16 columns would do there); of 512, 16 tokens 59.5 and 65.7.
constexpr int kDownWaves = 8, kDownMaxParts = 16;
inline int decode_down_cols(int T, int d) { return T <= 4 || d < 256 / kDownMaxParts * 64 ? 16 : 64; }
// How many workgroups share a tile's K: enough tiles and parts to fill the compute
// units, with eight 64-byte chunks, its loads in flight, for each wavefront at least.
inline int decode_parts(int64_t chunks, int d, int T) {
  const int64_t fill = 256 / (d / decode_down_cols(T, d)), most = chunks / (8 * kDownWaves);
  const int64_t p = fill < most ? fill : most;
  return (int)(p < 1 ? 1 : p > kDownMaxParts ? kDownMaxParts : p);
}

// The router as a kernel of its own from this many bytes of its weights on (a quarter of it
// for bf16 batches whose second terms have no room in LDS and are made beside the
// products), and the 64-byte blocks of K of one workgroup of it.  Measured, apart against
// in the first kernel: 64 experts of 2048 and one token 35.5 vs 37.6 us, of 3584 and 16
// tokens 467 vs 479.  And from this many bytes of the experts that may be active on, for the
// deal of units that it makes possible (see the first kernel's main loop): 8 tokens of the
// Mixtral shape 375 vs 385 us, with E4M3 weights 206 vs 209, one token 118.1 vs 117.6.
constexpr int kRouteApart = 128 * 1024, kRouteBlocks = 32;
constexpr size_t kDealApart = size_t(256) << 20;

struct DecodeArgs {
  const void* x;            // [T][d]
  const void* norm_w;       // [d] or null
  const void* w_router;     // [E][d], or null: ids and w are read
  const float* bias;
  int32_t* ids;             // [T][k]: read, or written where not null
  float* w;
  const void* w_gate;       // [E][F][d]
  const void* w_up;
  const void* w_down;       // [E][d][F]
  const float* s_gate;      // E4M3 weights: scales, else null
  const float* s_up;
  const float* s_down;
  const void* res;          // [T][d] or null
  void* out;                // [T][d]
  DecodeTable* table;
  void* h;                  // [active][F / KC][T, with h_low 2 T][KC], KC elements in 64 bytes
  int T, d, E, k, F;
  int blocked16;
  int h_low;                // h is kept in two terms
  int x_low;                // x norm_w is in LDS in two terms (set by the launcher)
  float* logits;            // [ranges][e16][16]: decode_route_kernel's sums, or null: routed in the first kernel
  int ranges, e16;
  float* part;              // [d / 64][parts][64 columns x 16 tokens], where parts > 1
  int parts;
  float eps, scale;
};
inline bool decode_h_low(int dtype) { return dtype == 1; }
// LDS that the first kernel needs at run time, and what a compute unit has beside its own arrays.
constexpr size_t kDecodeLds = 154 * 1024;  // (so d is at most 70656: 4416 tiles)
size_t decode_lds_bytes(int elt_bytes, int T, int d, int E);
// Whether LDS has room for the second terms of x norm_w too.
bool decode_x_low(int elt_bytes, int T, int d, int E);
hipError_t launch_decode(int dtype, const DecodeArgs& a, hipStream_t stream);  // (h_low set)

}  // namespace moe
