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
  int expert[256];
  float weight[256][kDecodeTokens];
};

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
  void* h;                  // [active][F / KC][T][KC], KC elements in 64 bytes
  int T, d, E, k, F;
  int blocked16;
  float eps, scale;
};
// LDS that the first kernel needs at run time, and what a compute unit has beside its own arrays.
constexpr size_t kDecodeLds = 158 * 1024;
size_t decode_lds_bytes(int elt_bytes, int T, int d, int E);
hipError_t launch_decode(int dtype, const DecodeArgs& a, hipStream_t stream);

}  // namespace moe
