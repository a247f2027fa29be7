// The layer for a few tokens (T <= 16): norm, router, experts, combine and
// residual in two kernels, or three where the router's weights are many.
//
// With at most 16 tokens every product of the layer has at most 16 columns, the
// width of one 16x16 matrix instruction, so the weights are the instruction's rows
// and all of the batch's tokens its columns: an expert is multiplied with every
// token, chosen or not, and the combine picks.  That needs no permutation and
// no dispatch arrays, the matrix cores have the room (16 rows x 64 bytes of weights
// per instruction: at the rate of HBM one in 90 cycles of a compute unit), and the
// work is a single stream over the active experts' weights, which is what bounds
// it.  Mixtral shape, one token, blocked bf16: 77 us and 37 us of the two kernels for
// 470 and 235 MB, 6.1 and 6.3 TB/s; 8 tokens with E4M3 weights: 133 and 70 us for 0.85 and
// 0.42 GB, 6.4 and 6.1 TB/s (a streaming read alone reaches 7.0); 64 experts of 2048 with
// row-major weights, 4 tokens: 47 and 23 us, of which 6 pass before the first weights.
//
//   decode_up_kernel    every workgroup norms the tokens into LDS, routes them
//                       (all of them, each workgroup for itself: E d weights
//                       from L2; many of them get a launch of their own,
//                       decode_route_kernel), and works units
//                       of 8 columns of F of an active expert: an MFMA tile of
//                       8 gate rows above 8 up rows, K split over the
//                       wavefronts, h = silu(g) u
//   decode_down_kernel  a workgroup for 16 or 64 columns of d and a part of the
//                       sum over the active experts' F columns, split over the
//                       wavefronts; where an expert ends, its sum is weighted
//                       into the total, token by token; the parts are added
//                       up, in order, by the workgroup that is done last
//
// Norm: 1 / rms is a factor of each fp32 sum.  p = x norm_w is exact in two bf16 terms where
// both are bf16, and h is kept in two, so that only the output is rounded: the error
// against 64 bits at the Mixtral shape is 0.0017, and 0.0029 with first terms alone.  The
// second terms of up to 8 tokens are in the instruction's idle columns and cost nothing;
// those of more are instructions of their own (16 tokens: 447 us, 435 without them).
// Where LDS has no room for p twice (16 tokens of more than about 2200), it has x, and each
// wavefront makes both terms beside its loads of weights: some 50 vector instructions for each
// 16 bytes of a lane, so a unit is 16 columns of F there and they serve two tiles (447 us; 486
// for one; with E4M3 weights 268 and 360, and 244 without second terms).
#include <algorithm>
#include <type_traits>

#include "block.hpp"
#include "device_common.hpp"
#include "vec.hpp"

namespace moe {
namespace {

// Weights: read once, by one workgroup, past the caches (PAST) where a load takes whole lines: 8
// tokens of the Mixtral shape take 391 us so and 423 with the default policy, row-major 400
// and 425.  A load of half a line of each of 16 rows leaves the other half to the next
// one, which finds it where the line was kept: 64 experts and 16 tokens 184 us, 197 past the
// caches, and 161 in whole lines.
template <bool PAST>
__device__ __forceinline__ uint4 load_weights(const char* p) {
  if constexpr (PAST)
    return __builtin_bit_cast(uint4, __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p)));
  else
    return load16(p);
}

// Eight OCP E4M3 codes to the bf16 values they are exactly.
__device__ __forceinline__ uint4 widen8(unsigned lo, unsigned hi) {
  return uint4{__builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false)),
               __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true)),
               __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false)),
               __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true))};
}

constexpr int kWaves = 8;        // wavefronts of the first kernel
constexpr int kDepth = 8;        // weight loads of a wavefront in flight
constexpr int kUnitCols = 8;     // columns of F of a unit
constexpr int kMaxGrid = 256;    // workgroups of the first kernel: one for each compute unit
constexpr int kMaxPieces = 160;  // rows of x in pieces of 64 x 16 bytes: T d element size / 1024 + T
constexpr size_t kRedBytes = 2 * kWaves * 1024;

// Storage of the weights: bytes from one row, and from one 64-byte piece of a row, to
// the next.
template <bool B16, bool LINES>
struct Rows {
  size_t row_bytes;
  __device__ __forceinline__ size_t at(int row) const {
    return B16 ? (size_t)(row >> 4) * 16 * row_bytes + (size_t)(row & 15) * 64 : (size_t)row * row_bytes;
  }
  static constexpr int step = B16 ? 1024 : LINES ? 128 : 64;
};

// Row-major weights are loaded in whole lines (LINES), 128 bytes of 8 rows at a time:
// lane l has piece l >> 3 of row l & 7 and, from a second load, of row 8 + (l & 7).  A
// change between the halves of each sixteen lanes makes two operands of that: lane l has
// row l & 15, and of its 8 pieces 2 (l >> 4) in the first and the next one in the
// second.  (E4M3 rows of an odd number of 64 bytes have no last line: they are loaded by 16
// rows of half a line.)
__device__ __forceinline__ void change_halves(uint4& v0, uint4& v1) {
  const auto from = [](unsigned keep, unsigned other, auto banks) {  // lane l takes lane l ^ 8's in these banks of 4
    return (unsigned)__builtin_amdgcn_update_dpp((int)keep, (int)other, 0x128, 0xf, decltype(banks)::value, false);
  };
  constexpr std::integral_constant<int, 0xC> upper{};
  constexpr std::integral_constant<int, 0x3> lower{};
  const uint4 a{from(v0.x, v1.x, upper), from(v0.y, v1.y, upper), from(v0.z, v1.z, upper), from(v0.w, v1.w, upper)};
  v1 = uint4{from(v1.x, v0.x, lower), from(v1.y, v0.y, lower), from(v1.z, v0.z, lower), from(v1.w, v0.w, lower)};
  v0 = a;
}

// Where a lane's part of x norm_w and h starts in a step's blocks [columns][64 bytes]: it is as
// long as its weights', which in lines are two pieces of 16 bytes and in E4M3 half as long as
// their operands.
template <bool Q, bool LINES>
__device__ __forceinline__ size_t act_offset(int piece, int col, int cols) {
  constexpr int parts = Q && LINES ? 1 : Q || LINES ? 2 : 4;  // of a block
  return ((size_t)(piece / parts) * cols + col) * 64 + piece % parts * (64 / parts);
}

// Operand h of a step's: NB chunks of it.
template <int NB, int N>
__device__ __forceinline__ const uint4 (&pick(const uint4 (&v)[N], int h))[NB] {
  return reinterpret_cast<const uint4(&)[NB]>(v[h * NB]);
}

template <class Tr, bool Q>
__device__ __forceinline__ f32x4_t mma_chunk(const uint4& w, const uint4 (&b)[Q ? 2 : 1], f32x4_t acc) {
  if constexpr (Q) {
    acc = mma16<Tr>(widen8(w.x, w.y), b[0], acc);
    return mma16<Tr>(widen8(w.z, w.w), b[1], acc);
  } else {
    return mma16<Tr>(w, b[0], acc);
  }
}

// What rounding left of fp32 values: the second terms.
template <class Tr>
__device__ __forceinline__ uint4 low_terms(float* v, const uint4& rounded) {
  float r[Tr::EPC];
  widen<Tr>(rounded, r);
#pragma unroll
  for (int j = 0; j < Tr::EPC; ++j) v[j] -= r[j];
  return round_to<Tr>(v);
}

// Logits apart, where the router's weights are too many for every workgroup to read
// (launch_decode): 16 experts and kRouteBlocks 64-byte blocks of K for a workgroup,
// four loads of a wavefront side by side; sums [range][experts][16 tokens], before 1 / rms
// and the bias.  4.7 us for 8 experts of 4096, one round of loads and its latency.
template <class Tr>
__global__ __launch_bounds__(64 * kWaves) void decode_route_kernel(DecodeArgs a) {
  using Elt = typename Tr::T;
  constexpr int EB = sizeof(Elt), U = kRouteBlocks / kWaves;
  __shared__ float part[kWaves][256];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, tok = lane & 15, piece = lane >> 4;
  const size_t xrow = (size_t)a.d * EB;
  const int blocks = a.d * EB / 64, b0 = (int)blockIdx.x * kRouteBlocks + wave * U, e0 = (int)blockIdx.y * 16;
  const bool normed = a.norm_w != nullptr;
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) a.table->claimed = 0;
  uint4 xv[U], gv[U], wv[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const size_t o = (size_t)min(b0 + u, blocks - 1) * 64 + piece * 16;
    wv[u] = load16(static_cast<const char*>(a.w_router) + (size_t)min(e0 + tok, a.E - 1) * xrow + o);
    xv[u] = load16(static_cast<const char*>(a.x) + (size_t)min(tok, a.T - 1) * xrow + o);
    if (normed) gv[u] = load16(static_cast<const char*>(a.norm_w) + o);
  }
  f32x4_t acc{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (b0 + u >= blocks) continue;
    if (normed) {
      float x[Tr::EPC], g[Tr::EPC];
      widen<Tr>(xv[u], x);
      widen<Tr>(gv[u], g);
#pragma unroll
      for (int j = 0; j < Tr::EPC; ++j) g[j] *= x[j];
      const uint4 hi = round_to<Tr>(g);
      acc = mma16<Tr>(wv[u], hi, acc);
      if constexpr (EB == 2) acc = mma16<Tr>(wv[u], low_terms<Tr>(g, hi), acc);
    } else {
      acc = mma16<Tr>(wv[u], xv[u], acc);
    }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) part[wave][(piece * 4 + r) * 16 + tok] = acc[r];
  __syncthreads();
  if (threadIdx.x >= 256) return;
  float s = part[0][threadIdx.x];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) s += part[w][threadIdx.x];
  a.logits[((size_t)blockIdx.x * a.e16 + e0) * kDecodeTokens + threadIdx.x] = s;
}

// Both terms of x norm_w.
template <class Tr>
__device__ __forceinline__ void two_terms(const uint4& x, const uint4& norm_w, uint4& hi, uint4& lo) {
  float v[Tr::EPC], g[Tr::EPC];
  widen<Tr>(x, v);
  widen<Tr>(norm_w, g);
#pragma unroll
  for (int j = 0; j < Tr::EPC; ++j) v[j] *= g[j];
  hi = round_to<Tr>(v);
  lo = low_terms<Tr>(v, hi);
}

// A logit and its expert's bias: one of -inf masks the expert, whatever its router row holds
// (a NaN, or +inf, and -inf would be a NaN).
__device__ __forceinline__ float biased(float s, const float* bias, int e) {
  const float b = bias != nullptr ? bias[e] : 0.f;
  return b == -INFINITY ? b : s + b;
}

// Q: E4M3 weights.  B16: the blocked order.  NE: 16-expert tiles of the router at a time; NQ: experts of a lane in
// the choice.  RAW: x is in LDS as it is, both terms of p are made for each chunk of weights, and a unit is two
// tiles, 16 gate rows and 16 up rows.
template <class Tr, bool Q, bool B16, bool LINES, int NE, int NQ, bool RAW>
__global__ __launch_bounds__(64 * kWaves) void decode_up_kernel(DecodeArgs a) {
  using Elt = typename Tr::T;
  constexpr int EB = sizeof(Elt), WB = Q ? 1 : EB, KB = 64 / EB, NB = Q ? 2 : 1;
  // (with E4M3 a load is two chunks of work: 16 of them in flight take 268 us at 16 tokens of
  // the Mixtral shape and 8 take 277; bf16 449 and 450)
  constexpr int CH = LINES ? 2 : 1;  // 64-byte chunks of K of a step
  constexpr int TU = RAW ? 2 : 1, kCols = kUnitCols * TU, D = (RAW && !Q ? kDepth / 2 : kDepth) / CH;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  __shared__ float part_sq[kMaxPieces];
  __shared__ int list[256], wave_count[4];
  __shared__ uint8_t chosen[256];
  __shared__ int claims[8];
  __shared__ __attribute__((aligned(16))) float scales[Q ? 4 : 1][kWaves * 16 * TU];
  const int T = a.T, E = a.E, d = a.d, F = a.F;
  const size_t plane = (size_t)T * d * EB;
  char* xs = lds;                                                       // [1, with x_low 2][d / KB][T][64 bytes]
  f32x4_t* red = reinterpret_cast<f32x4_t*>(lds + (a.x_low ? 2 : 1) * plane);  // [2][kWaves][64]
  float* logit = reinterpret_cast<float*>(reinterpret_cast<char*>(red) + kRedBytes);  // [T][E]
  float* wt = logit + T * E;                                            // [E][T]

  const int lane = threadIdx.x & 63, tok = lane & 15, piece = lane >> 4, tc = min(tok, T - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool normed = a.norm_w != nullptr, route = a.w_router != nullptr;
  const size_t xrow = (size_t)d * EB;
  const int blocks = d / KB;
  // the second terms of p: in the columns that T leaves, or instructions of their own
  const bool spare = a.x_low && T <= 8, second = a.x_low && T > 8;

  for (int i = threadIdx.x; i < T * E; i += 64 * kWaves) wt[i] = 0.f;
  if (threadIdx.x < 256) chosen[threadIdx.x] = 0;

  constexpr int U = NE == 1 ? 4 : 2;
  const bool inside = route && a.logits == nullptr;
  const int b0 = blocks * wave / kWaves, b1 = blocks * (wave + 1) / kWaves;
  uint4 wv[U][NE];
  const auto load_router = [&](int e0, int u, int b) {
#pragma unroll
    for (int i = 0; i < NE; ++i)
      wv[u][i] = load16(static_cast<const char*>(a.w_router) + (size_t)min(e0 + i * 16 + tok, E - 1) * xrow +
                        (size_t)min(b, blocks - 1) * 64 + piece * 16);
  };

  // x norm_w into LDS, and the sums of squares: a wavefront takes 1 KB of a token's row at a
  // time, four of them side by side
  const int chunk16 = d / Tr::EPC, per_row = (chunk16 + 63) / 64, pieces = T * per_row;
  for (int i0 = wave; i0 < pieces; i0 += kWaves * 4) {
    uint4 xv[4], gv[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = min(i0 + u * kWaves, pieces - 1), t = i / per_row, c = min((i - t * per_row) * 64 + lane, chunk16 - 1);
      xv[u] = load16(static_cast<const char*>(a.x) + t * xrow + (size_t)c * 16);
      if (normed) gv[u] = load16(static_cast<const char*>(a.norm_w) + (size_t)c * 16);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + u * kWaves, t = i / per_row, c = (i - t * per_row) * 64 + lane;
      if (i >= pieces) break;
      const bool in = c < chunk16;
      uint4 hi = xv[u], lo = make_uint4(0, 0, 0, 0);
      if (normed) {
        float x[Tr::EPC], g[Tr::EPC], sq = 0.f;
        widen<Tr>(xv[u], x);
        widen<Tr>(gv[u], g);
#pragma unroll
        for (int j = 0; j < Tr::EPC; ++j) {
          sq = fmaf(x[j], x[j], sq);
          g[j] *= x[j];
        }
        sq = wave_fold(in ? sq : 0.f, [](float p, float q) { return p + q; });
        if (lane == 0) part_sq[i] = sq;
        if constexpr (!RAW) {
          hi = round_to<Tr>(g);
          if constexpr (EB == 2) lo = low_terms<Tr>(g, hi);
        }
      }
      if (in) {
        char* to = xs + ((size_t)(c >> 2) * T + t) * 64 + (c & 3) * 16;
        *reinterpret_cast<uint4*>(to) = hi;
        if (a.x_low) *reinterpret_cast<uint4*>(to + plane) = lo;
      }
    }
  }
  // (behind x's loads, which answer in order)
  if (inside) {
#pragma unroll
    for (int u = 0; u < U; ++u) load_router(0, u, b0 + u);
  }
  __syncthreads();
  float inv = 1.f;
  if (normed) {
    float s = 0.f;
    for (int i = 0; i < per_row; ++i) s += part_sq[tc * per_row + i];
    inv = rsqrtf(s / (float)d + a.eps);  // of token `tok`, in every lane
  }

  // The router: each wavefront a run of K, all experts and tokens
  for (int e0 = 0; inside && e0 < E; e0 += 16 * NE) {
    f32x4_t acc[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) acc[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    if (e0 != 0) {
#pragma unroll
      for (int u = 0; u < U; ++u) load_router(e0, u, b0 + u);
    }
    for (int base = b0; base < b1; base += U) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int b = base + u;
        if (b >= b1) continue;
        const char* from = xs + ((size_t)b * T + tc) * 64 + piece * 16;
        uint4 hi = *reinterpret_cast<const uint4*>(from), lo = make_uint4(0, 0, 0, 0);
        if constexpr (RAW)
          two_terms<Tr>(hi, load16(static_cast<const char*>(a.norm_w) + (size_t)b * 64 + piece * 16), hi, lo);
        else if (EB == 2 && normed)
          lo = *reinterpret_cast<const uint4*>(from + plane);
#pragma unroll
        for (int i = 0; i < NE; ++i) {
          acc[i] = mma16<Tr>(wv[u][i], hi, acc[i]);
          if (EB == 2 && normed) acc[i] = mma16<Tr>(wv[u][i], lo, acc[i]);
        }
        if (b + U < b1) load_router(e0, u, b + U);
      }
    }
    // sums of the wavefronts, two tiles at a time: wavefront w has tile w / 4, and 64
    // of its 256 logits
#pragma unroll
    for (int i0 = 0; i0 < NE; i0 += 2) {
#pragma unroll
      for (int i = i0; i < i0 + 2 && i < NE; ++i) red[((i - i0) * kWaves + wave) * 64 + lane] = acc[i];
      __syncthreads();
      const int i = i0 + (wave >> 2), quarter = wave & 3;
      if (i < NE) {
        // value r = wave & 3 of every lane of that tile: expert 4 piece + r, token tok
        float s = red[(wave >> 2) * kWaves * 64 + lane][quarter];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) s += red[((wave >> 2) * kWaves + w) * 64 + lane][quarter];
        const int e = e0 + i * 16 + piece * 4 + quarter;
        if (e < E && tok < T) logit[tok * E + e] = biased(s * inv, a.bias, e);
      }
      __syncthreads();
    }
  }

  if (route && !inside) {  // decode_route_kernel's sums over ranges of K, in order
    for (int i = threadIdx.x; i < E * kDecodeTokens; i += 64 * kWaves) {  // (expert i / 16, token i % 16 = tok)
      float s = 0.f;
#pragma unroll 4
      for (int r = 0; r < a.ranges; ++r) s += a.logits[(size_t)r * a.e16 * kDecodeTokens + i];
      if (tok < T) logit[tok * E + i / kDecodeTokens] = biased(s * inv, a.bias, i / kDecodeTokens);
    }
    __syncthreads();
  }

  const bool first = blockIdx.x == 0;
  if (route) {
    // Top-k: k times the largest logit, at the lowest index that has it.  What is taken
    // becomes a NaN, which no maximum sees; so a NaN logit is not seen either, and ranks below
    // every other, those of -inf among them: where no key is the maximum only such are left.
    for (int t = wave; t < T; t += kWaves) {
      float v[NQ], key[NQ];
      int slot[NQ];
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        const int e = lane + 64 * q;
        v[q] = e < E ? logit[t * E + e] : 0.f;
        key[q] = e < E ? v[q] : NAN;
        slot[q] = -1;
      }
      float top = 0.f;
      for (int j = 0; j < a.k; ++j) {
        float m = key[0];
#pragma unroll
        for (int q = 1; q < NQ; ++q) m = fmaxf(m, key[q]);
        m = wave_fold(m, [](float x, float y) { return fmaxf(x, y); });
        if (j == 0) top = m;
        bool found = false;
        const auto take = [&](int q, bool candidate) {  // the first lane that has one
          const uint64_t at = __ballot(candidate);
          if (!found && at != 0) {
            found = true;
            if (lane == __ffsll((unsigned long long)at) - 1) {
              slot[q] = j;
              key[q] = NAN;
            }
          }
        };
#pragma unroll
        for (int q = 0; q < NQ; ++q) take(q, key[q] == m);
        if (found) continue;
#pragma unroll
        for (int q = 0; q < NQ; ++q) take(q, slot[q] < 0 && lane + 64 * q < E);
      }
      float ex[NQ], sum = 0.f;
      bool nan = false;
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        ex[q] = slot[q] >= 0 && v[q] != -INFINITY ? expf(v[q] - top) : 0.f;
        sum += ex[q];
        nan |= v[q] != v[q];
      }
      sum = wave_fold(sum, [](float x, float y) { return x + y; });
      // no expert with a number above -inf: none at all where every one is masked, but what has
      // a NaN (that of x, for one) is not to be taken for that
      const float none = __ballot(nan) != 0 ? NAN : 0.f;
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        if (slot[q] < 0) continue;
        const int e = lane + 64 * q;
        const float w = sum == 0.f ? none : ex[q] / sum;
        wt[e * T + t] = w;
        if (w != 0.f) chosen[e] = 1;
        if (first && a.ids != nullptr) a.ids[t * a.k + slot[q]] = e;
        if (first && a.w != nullptr) a.w[t * a.k + slot[q]] = w;
      }
    }
  } else if ((int)threadIdx.x < T) {
    // the caller's routing: slots in order, so that an expert chosen twice has one weight
    for (int j = 0; j < a.k; ++j) {
      const int e = a.ids[threadIdx.x * a.k + j];
      if (e < 0 || e >= E) continue;
      const float w = wt[e * T + threadIdx.x] + a.w[threadIdx.x * a.k + j];
      wt[e * T + threadIdx.x] = w;
      if (w != 0.f) chosen[e] = 1;
    }
  }
  __syncthreads();

  // the experts with a weight for any token, ascending
  const bool active = threadIdx.x < 256 && chosen[threadIdx.x & 255] != 0;
  const uint64_t ballot = __ballot(active);
  if (wave < 4 && lane == 0) wave_count[wave] = __popcll(ballot);
  __syncthreads();
  int n_active = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) n_active += wave_count[w];
  if (active) {
    int at = __popcll(ballot & lanemask_lt(lane));
    for (int w = 0; w < wave; ++w) at += wave_count[w];
    list[at] = threadIdx.x;
  }
  __syncthreads();
  n_active = __builtin_amdgcn_readfirstlane(n_active);
  if (first) {
    if (threadIdx.x == 0) a.table->n_active = n_active;
    for (int i = threadIdx.x; i < d / 16; i += 64 * kWaves) a.table->arrived[i] = 0;
    for (int i = threadIdx.x; i < n_active; i += 64 * kWaves) a.table->expert[i] = list[i];
    for (int i = threadIdx.x; i < n_active * T; i += 64 * kWaves) a.table->weight[i / T][i % T] = wt[list[i / T] * T + i % T];
  }

  // ---- gate and up: units of 8 columns (RAW: 16), dealt to groups of wavefronts in turn.  A group
  // splits K; it is the whole workgroup unless that left a wavefront fewer than 2 kDepth
  // chunks of a unit: with one round of loads between two barriers, 8 tokens with E4M3
  // weights take 237 us and not 213 at the Mixtral shape.  A round then ends one unit at
  // the most, and the code behind a unit's end stands once (inlined at each load the
  // kernel was 60 KB, whose fetches took longer than the first loads of data)
  const int per = F / kCols, total = n_active * per, chunks = d * WB / 64 / CH;
  const int split = chunks * CH >= 16 * kDepth ? 8 : chunks * CH >= 8 * kDepth ? 4 : chunks * CH >= 4 * kDepth ? 2 : 1;
  const int groups = kWaves / split, group = wave / split, part = wave % split;
  const int c0 = chunks * part / split, mine = chunks * (part + 1) / split - c0;
  const int round = max(mine, D);  // (a narrow unit is padded to a round)
  // The deal: turn i of a workgroup is a unit for each of its groups, from slot base_of(i).
  // The first turns are dealt evenly, the last sixth to whoever is there first, from a
  // counter that decode_route_kernel has cleared: odd dies take 5 to 10 % longer for the
  // same share.  A claim is made four turns ahead and posted in LDS three ahead.
  const int stride = (int)gridDim.x * groups, u0 = (int)blockIdx.x * groups;
  const int even = total / stride, fixed = a.logits != nullptr && even >= 8 ? max(4, even * 5 / 6) : 0x7fffffff;
  const auto base_of = [&](int i) { return i < fixed ? u0 + i * stride : fixed * stride + claims[i & 7] * groups; };
  const auto there = [&](int slot) { return slot < total; };
  if (!there(u0)) return;
  // Two units share each 1 KB of a blocked matrix's 16 rows: they go to workgroups 8
  // apart, which are on one die
  const auto unit = [&](int slot) {
    return TU == 1 && groups == 1 && (slot | 15) < total ? (slot & ~15) | ((slot & 7) << 1) | ((slot >> 3) & 1) : slot;
  };
  const Rows<B16, LINES> rows{(size_t)d * WB};
  constexpr int step = Rows<B16, LINES>::step;
  const int my_piece = LINES ? lane >> 3 : piece;
  const char* base = static_cast<const char*>(LINES || TU == 2 || tok < 8 ? a.w_gate : a.w_up) + my_piece * 16 + (size_t)c0 * step;
  const int64_t to_up = reinterpret_cast<intptr_t>(a.w_up) - reinterpret_cast<intptr_t>(a.w_gate);
  // to the second load of a tile in lines: its rows 8 .. 15
  const int64_t to_half = TU == 2 ? (int64_t)(8 * rows.row_bytes) : to_up;
  const auto unit_at = [&](int slot) {
    const int u = unit(slot), e = list[u / per];
    return base + (size_t)e * F * rows.row_bytes + rows.at((u % per) * kCols + (TU == 2 && !LINES ? tok : tok & 7));
  };
  // E4M3: the scales of a turn's units, 8 of gate's and 8 of up's each, one for a thread; in
  // LDS a turn before they are used, so that finishing a unit waits for no load
  const auto scale_of = [&](int i) {
    const int slot = base_of(i) + (int)threadIdx.x / (2 * kCols), u = unit(slot);
    if ((int)threadIdx.x >= groups * 2 * kCols || !there(slot)) return 0.f;
    return ((threadIdx.x & kCols) ? a.s_up : a.s_gate)[(size_t)list[u / per] * F + (u % per) * kCols + (threadIdx.x & (kCols - 1))];
  };
  float scale_next = 0.f;
  int claim_next = 0;
  if constexpr (Q) {
    if (threadIdx.x < kWaves * 2 * kCols) {
      scales[0][threadIdx.x] = scale_of(0);
      scale_next = scale_of(1);
    }
    __syncthreads();
  }
  // turn i's sums, which the wavefronts have left in LDS, to h: by one wavefront of each
  // group, each turn another
  const auto finish = [&](int i) {
    if (Q && threadIdx.x < kWaves * 2 * kCols) scales[(i + 1) & 3][threadIdx.x] = scale_next;
    if (i + 3 >= fixed && threadIdx.x == 0) claims[(i + 3) & 7] = claim_next;
    lds_barrier();
    if (i + 4 >= fixed && threadIdx.x == 0)
      claim_next = __hip_atomic_fetch_add(&a.table->claimed, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (Q && threadIdx.x < kWaves * 2 * kCols) scale_next = scale_of(i + 2);
    const int slot = base_of(i) + group;
    const bool mine = part == i % split && there(slot);
    f32x4_t s[TU];
    if (mine) {
#pragma unroll
      for (int q = 0; q < TU; ++q) {
        const f32x4_t* from = red + ((TU == 2 ? q : i & 1) * kWaves + group * split) * 64 + lane;
        s[q] = from[0];
        for (int w = 1; w < split; ++w) s[q] += from[w * 64];
      }
    }
    if constexpr (TU == 2) lds_barrier();  // (one place for the sums: the next turn's come behind this)
    if (!mine) return;
    const int u = unit(slot), n = u / per, f0 = (u % per) * kCols;
#pragma unroll
    for (int q = 0; q < TU; ++q) {
#pragma unroll
      for (int r = 0; r < 4; ++r) s[q][r] = (spare ? s[q][r] + __shfl_down(s[q][r], 8) : s[q][r]) * inv;
      if constexpr (Q) {
        const float4 sc = *reinterpret_cast<const float4*>(&scales[i & 3][(group * TU + q) * 16 + piece * 4]);
        s[q][0] *= sc.x, s[q][1] *= sc.y, s[q][2] *= sc.z, s[q][3] *= sc.w;
      }
    }
    // one tile: rows 0..7 (pieces 0, 1) are the gate's columns, rows 8..15 the same of up
    float hv[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float up = TU == 2 ? s[TU - 1][r] : __shfl_down(s[0][r], 32);
      hv[r] = s[0][r] / (1.f + __expf(-s[0][r])) * up;
    }
    if ((TU == 2 || piece < 2) && tok < T) {
      const int f = f0 + piece * 4;
      char* to = static_cast<char*>(a.h) + (((size_t)n * (F / KB) + f / KB) * (a.h_low ? 2 * T : T) + tok) * 64 + (f % KB) * EB;
      store4<Tr>(to, hv[0], hv[1], hv[2], hv[3]);
      if (EB == 2 && a.h_low) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float hi = bf16_to_f32(f32_to_bf16(hv[r]));
          hv[r] = fabsf(hi) < INFINITY ? hv[r] - hi : 0.f;
        }
        store4<Tr>(to + (size_t)T * 64, hv[0], hv[1], hv[2], hv[3]);
      }
    }
  };
  int turn = 0;  // turns finished
  if (there(u0 + group)) {
    // kDepth loads in flight, across units: the cursor is at chunk lc of turn li, and
    // behind the last unit repeats its last chunk
    int li = 0, lc = 0, slot = base_of(1) + group;
    const char *lp = unit_at(u0 + group), *next = unit_at(there(slot) ? slot : u0 + group);
    const char* const g0 = static_cast<const char*>(a.norm_w) + (size_t)c0 * CH * NB * 64 + piece * (Q && LINES ? 64 : Q || LINES ? 32 : 16);
    const char* gp = g0;
    bool more = there(slot), moved = false;
    uint4 ring[D][TU][CH], gains[RAW ? D : 1][CH][NB];
    const auto load = [&](int j) {
#pragma unroll
      for (int h = 0; h < CH; ++h) {
        ring[j][0][h] = load_weights<B16 || LINES>(lp + h * to_half);
        if constexpr (TU == 2) ring[j][TU - 1][h] = load_weights<B16 || LINES>(lp + to_up + h * to_half);
        if constexpr (RAW) {
#pragma unroll
          for (int q = 0; q < NB; ++q) gains[j][h][q] = load16(gp + (h * NB + q) * 16);
        }
      }
      if (++lc < mine) {
        lp += step;
        gp += CH * NB * 64;
      }
      if (lc == round && more) {
        ++li;
        lc = 0;
        lp = next;
        gp = g0;
        moved = true;
      }
    };
    const int col = spare ? min(tok & 7, T - 1) : tc;
    const char* xlane = xs + (spare && tok >= 8 ? plane : 0) + (size_t)c0 * CH * NB * T * 64 +
                        act_offset<Q, LINES>(piece, col, T);
    int uc = 0;
    bool alive = true, ended = false;
    f32x4_t acc[TU];
#pragma unroll
    for (int q = 0; q < TU; ++q) acc[q] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    const auto work = [&](int j) {
      if (!alive) return;
      if (uc < mine) {
        if constexpr (LINES) {
#pragma unroll
          for (int q = 0; q < TU; ++q) change_halves(ring[j][q][0], ring[j][q][CH - 1]);
        }
        const char* const from = xlane + (size_t)uc * CH * NB * T * 64;
#pragma unroll
        for (int h = 0; h < CH; ++h) {
          uint4 b[NB];
#pragma unroll
          for (int q = 0; q < NB; ++q) b[q] = *reinterpret_cast<const uint4*>(from + (h * NB + q) * 16);
          if constexpr (RAW) {
            uint4 lo[NB];
#pragma unroll
            for (int q = 0; q < NB; ++q) two_terms<Tr>(b[q], gains[j][h][q], b[q], lo[q]);
#pragma unroll
            for (int q = 0; q < TU; ++q) acc[q] = mma_chunk<Tr, Q>(ring[j][q][h], lo, acc[q]);
          }
#pragma unroll
          for (int q = 0; q < TU; ++q) acc[q] = mma_chunk<Tr, Q>(ring[j][q][h], b, acc[q]);
          if (EB == 2 && !RAW && second) {
#pragma unroll
            for (int q = 0; q < NB; ++q) b[q] = *reinterpret_cast<const uint4*>(from + plane + (h * NB + q) * 16);
            acc[0] = mma_chunk<Tr, Q>(ring[j][0][h], b, acc[0]);
          }
        }
      }
      if (++uc == round) {
#pragma unroll
        for (int q = 0; q < TU; ++q) {
          red[((TU == 2 ? q : turn & 1) * kWaves + wave) * 64 + lane] = acc[q];
          acc[q] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        }
        uc = 0;
        ended = true;
        alive = li > turn;  // the cursor is kDepth loads ahead, in the next unit if there is one
      }
    };
#pragma unroll
    for (int j = 0; j < D; ++j) load(j);
    while (alive) {
      if (moved) {
        slot = base_of(li + 1) + group;
        more = there(slot);
        if (more) next = unit_at(slot);
        moved = false;
      }
#pragma unroll
      for (int j = 0; j < D; ++j) {
        work(j);
        load(j);
      }
      if (ended) {
        finish(turn++);
        ended = false;
      }
    }
  }
  for (; there(base_of(turn)); ++turn) finish(turn);  // (others' barriers)
}

// One part of the K range of 16 NR columns of d: out's columns where the tile has one part,
// else partial sums, which the workgroup that is done last adds up in the parts'
// order.  The columns share each load of h, which every tile reads whole.  TWO: h's second
// terms are loads and instructions of their own.
template <class Tr, bool Q, bool B16, bool LINES, int NR, bool TWO>
__global__ __launch_bounds__(64 * kDownWaves) void decode_down_kernel(DecodeArgs a) {
  using Elt = typename Tr::T;
  constexpr int EB = sizeof(Elt), WB = Q ? 1 : EB, NB = Q ? 2 : 1, kCols = NR * 16;
  constexpr int CH = LINES ? 2 : 1, D = (NR == 1 ? 8 : 4) / CH;  // chunks of K of a step, steps in flight
  __shared__ f32x4_t red[kDownWaves][NR][64];
  __shared__ float wts[256][kDecodeTokens];
  __shared__ float scale[Q ? 256 : 1][kCols];
  __shared__ int list[256];
  __shared__ int last;
  const int T = a.T, d = a.d, F = a.F;
  const int lane = threadIdx.x & 63, tok = lane & 15, piece = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tile = (int)blockIdx.x, part = (int)blockIdx.y, o0 = tile * kCols;
  // the table, as much of it as there may be, without waiting for its length
  const int most = min(a.E, T * a.k);
  for (int i = threadIdx.x; i < most * kDecodeTokens; i += 64 * kDownWaves) {
    const int n = i / kDecodeTokens, t = i % kDecodeTokens;
    wts[n][t] = a.table->weight[n][t];
    if (t == 0) list[n] = a.table->expert[n];
  }
  const int n_active = __builtin_amdgcn_readfirstlane(a.table->n_active);
  const int per = F * WB / 64 / CH, total = n_active * per;  // steps of an expert, of all
  const int p0 = (int)((long long)total * part / a.parts), p1 = (int)((long long)total * (part + 1) / a.parts);
  const int i0 = p0 + (int)((long long)(p1 - p0) * wave / kDownWaves);
  const int i1 = p0 + (int)((long long)(p1 - p0) * (wave + 1) / kDownWaves);
  __syncthreads();
  if constexpr (Q) {
    const int n0 = p0 / per, n1 = (p1 + per - 1) / per;
    for (int i = n0 * kCols + threadIdx.x; i < n1 * kCols; i += 64 * kDownWaves)
      scale[i / kCols][i % kCols] = a.s_down[(size_t)list[i / kCols] * d + o0 + i % kCols];
    __syncthreads();
  }

  f32x4_t sum[NR];
#pragma unroll
  for (int q = 0; q < NR; ++q) sum[q] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  if (i0 < i1) {
    const Rows<B16, LINES> rows{(size_t)F * WB};
    constexpr int step = Rows<B16, LINES>::step;
    const char* base = static_cast<const char*>(a.w_down) + (LINES ? rows.at(o0 + (lane & 7)) + (lane >> 3) * 16 : rows.at(o0 + tok) + piece * 16);
    const size_t tile_bytes = 16 * rows.row_bytes, expert_bytes = (size_t)d * rows.row_bytes;
    const int cols = a.h_low ? 2 * T : T, bstep = cols * 64 * NB * CH;
    const bool spare = !TWO && a.h_low;
    const int wcol = spare ? tok & 7 : tok;
    // h's column for this lane: its token's, or, where that did not choose the expert,
    // the first's that did, so that no line is read for it
    const auto column = [&](int n) {
      const bool has = wcol < T && wts[n][wcol] != 0.f;
      const int any = max(__ffsll((unsigned long long)__ballot(has)) - 1, 0) & (spare ? 7 : 15);
      const int col = (has ? wcol : any) + (spare && tok >= 8 ? T : 0);
      return static_cast<const char*>(a.h) +
             act_offset<Q, LINES>(piece, col, cols);
    };
    int ln = i0 / per, lc = i0 % per, li = i0;
    const char* lp = base + list[ln] * expert_bytes + (size_t)lc * step;
    const char* bp = column(ln) + (size_t)i0 * bstep;
    uint4 ring[D][NR][CH], act[D][CH * NB], low[D][CH * NB];
    const auto load = [&](int j) {
#pragma unroll
      for (int q = 0; q < NR; ++q)
#pragma unroll
        for (int h = 0; h < CH; ++h) ring[j][q][h] = load_weights<B16 || LINES>(lp + q * tile_bytes + h * 8 * rows.row_bytes);
#pragma unroll
      for (int q = 0; q < CH * NB; ++q) {
        act[j][q] = load16(bp + q * 16);
        if constexpr (TWO) low[j][q] = load16(bp + (size_t)T * 64 + q * 16);
      }
      if (++li >= i1) return;  // behind the last chunk: it again
      bp += bstep;
      if (++lc < per) {
        lp += step;
      } else {
        lc = 0;
        lp = base + list[++ln] * expert_bytes;
        bp = column(ln) + (size_t)li * bstep;
      }
    };
    int n = i0 / per, c = i0 % per, since = 0;
    f32x4_t acc[NR];
#pragma unroll
    for (int q = 0; q < NR; ++q) acc[q] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    // a token that did not choose the expert takes nothing of its sum, whatever that holds
    const auto fold = [&]() {
      const float w = wts[n][wcol];
#pragma unroll
      for (int q = 0; q < NR; ++q) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float v = acc[q][r];
          if constexpr (Q) v *= scale[n][q * 16 + piece * 4 + r];
          sum[q][r] = w != 0.f ? fmaf(w, v, sum[q][r]) : sum[q][r];
        }
        acc[q] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      }
      since = 0;
    };
    const auto work = [&](int j) {
#pragma unroll
      for (int q = 0; q < NR; ++q) {
        if constexpr (LINES) change_halves(ring[j][q][0], ring[j][q][CH - 1]);
#pragma unroll
        for (int h = 0; h < CH; ++h) {
          acc[q] = mma_chunk<Tr, Q>(ring[j][q][h], pick<NB>(act[j], h), acc[q]);
          if constexpr (TWO) acc[q] = mma_chunk<Tr, Q>(ring[j][q][h], pick<NB>(low[j], h), acc[q]);
        }
      }
      ++since;
      if (++c == per) {
        fold();
        ++n;
        c = 0;
      }
    };
#pragma unroll
    for (int j = 0; j < D; ++j) load(j);
    int left = i1 - i0;
    for (; left >= D; left -= D) {
#pragma unroll
      for (int j = 0; j < D; ++j) {
        work(j);
        load(j);
      }
    }
#pragma unroll
    for (int j = 0; j < D; ++j)
      if (j < left) work(j);
    if (since != 0) fold();
  }
#pragma unroll
  for (int q = 0; q < NR; ++q) red[wave][q][lane] = sum[q];
  __syncthreads();
  // thread (q, lane) has columns 16 q + 4 piece .. + 3 of token tok; with low terms
  // their products are eight lanes on
  const int q = wave & (NR - 1);
  const bool mine = wave < NR && tok < T;
  f32x4_t v{0.f, 0.f, 0.f, 0.f};
  if (mine) {
    v = red[0][q][lane];
#pragma unroll
    for (int w = 1; w < kDownWaves; ++w) v += red[w][q][lane];
    if (!TWO && a.h_low) {
#pragma unroll
      for (int w = 0; w < kDownWaves; ++w) v += red[w][q][lane + 8];
    }
  }
  if (a.parts > 1) {
    // Stored and loaded past the caches that other dies do not share (agent scope): every
    // wavefront's stores are done before the barrier, the count comes behind it, and
    // nobody waits for anybody.  A fence of that scope would write back and drop all of L2.
    float* all = a.part + ((size_t)tile * a.parts * (NR * 64) + q * 64 + lane) * 4;
    if (mine) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        __hip_atomic_store(all + (size_t)part * (NR * 256) + r, v[r], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    if (threadIdx.x == 0)
      last = __hip_atomic_fetch_add(&a.table->arrived[tile], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == a.parts - 1;
    __syncthreads();
    if (!last) return;
    if (mine) {
      v = f32x4_t{0.f, 0.f, 0.f, 0.f};
      for (int p = 0; p < a.parts; ++p)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          v[r] += __hip_atomic_load(all + (size_t)p * (NR * 256) + r, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
  }
  if (!mine) return;
  const size_t at = ((size_t)tok * d + o0 + q * 16 + piece * 4) * EB;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    v[r] *= a.scale;
    if (a.res != nullptr) {
      const char* p = static_cast<const char*>(a.res) + at + r * EB;
      v[r] += EB == 2 ? bf16_to_f32(*reinterpret_cast<const uint16_t*>(p)) : *reinterpret_cast<const float*>(p);
    }
  }
  store4<Tr>(static_cast<char*>(a.out) + at, v[0], v[1], v[2], v[3]);
}

template <class Tr, bool Q, bool B16>
hipError_t decode_t(DecodeArgs a, hipStream_t stream) {
  constexpr int EB = sizeof(typename Tr::T);
  size_t lds = decode_lds_bytes(EB, a.T, a.d, a.E);
  a.x_low = a.norm_w != nullptr && decode_x_low(EB, a.T, a.d, a.E);
  if (a.x_low) lds += (size_t)a.T * a.d * EB;
  if (a.logits != nullptr) {
    hipLaunchKernelGGL(decode_route_kernel<Tr>, dim3(a.ranges, a.e16 / 16), dim3(64 * kWaves), 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const bool raw = EB == 2 && a.norm_w != nullptr && !a.x_low;
  const int64_t units = (int64_t)std::min(a.E, a.T * a.k) * (a.F / (raw ? 2 * kUnitCols : kUnitCols));
  const dim3 grid((unsigned)std::min<int64_t>(units, kMaxGrid));
  const auto up = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(64 * kWaves), lds, stream, a); };
  const auto up_of = [&](auto lines) {
    constexpr bool L = decltype(lines)::value;
    if constexpr (EB == 2) {
      if (raw && a.E <= 64)  // (rows so wide route up to 7 experts in this kernel and more of them apart)
        return up(decode_up_kernel<Tr, Q, B16, L, 1, 1, true>);
      if (raw) return up(decode_up_kernel<Tr, Q, B16, L, 1, 4, true>);
    }
    if (a.E <= 16) return up(decode_up_kernel<Tr, Q, B16, L, 1, 1, false>);
    if (a.E <= 64) return up(decode_up_kernel<Tr, Q, B16, L, 4, 1, false>);
    up(decode_up_kernel<Tr, Q, B16, L, 4, 4, false>);
  };
  const dim3 tiles(a.d / decode_down_cols(a.T, a.d), a.parts);
  const auto down = [&](auto kernel) { hipLaunchKernelGGL(kernel, tiles, dim3(64 * kDownWaves), 0, stream, a); };
  const auto down_of = [&](auto lines) {
    constexpr bool L = decltype(lines)::value;
    const bool narrow = decode_down_cols(a.T, a.d) == 16;
    if constexpr (EB == 2) {
      if (a.T > 8 && narrow) return down(decode_down_kernel<Tr, Q, B16, L, 1, true>);
      if (a.T > 8) return down(decode_down_kernel<Tr, Q, B16, L, 4, true>);
    }
    if (narrow) return down(decode_down_kernel<Tr, Q, B16, L, 1, false>);
    down(decode_down_kernel<Tr, Q, B16, L, 4, false>);
  };
  // row-major rows in whole lines: all but E4M3 rows of an odd number of 64 bytes
  const auto by_width = [&](int row, auto&& of) {
    if constexpr (B16)
      of(std::false_type{});
    else if constexpr (!Q)
      of(std::true_type{});
    else if (row % 128 == 0)
      of(std::true_type{});
    else
      of(std::false_type{});
  };
  by_width(a.d, up_of);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  by_width(a.F, down_of);
  return hipGetLastError();
}

}  // namespace

// x [T][d], the wavefronts' sums, logits and weights [T][E] each.
size_t decode_lds_bytes(int elt_bytes, int T, int d, int E) {
  return (size_t)T * d * elt_bytes + kRedBytes + (size_t)8 * T * E;
}

bool decode_x_low(int elt_bytes, int T, int d, int E) {
  return elt_bytes == 2 && decode_lds_bytes(elt_bytes, T, d, E) + (size_t)T * d * elt_bytes <= kDecodeLds;
}

hipError_t launch_decode(int dtype, const DecodeArgs& a, hipStream_t stream) {
  if (a.s_gate != nullptr) return a.blocked16 ? decode_t<TBF16, true, true>(a, stream) : decode_t<TBF16, true, false>(a, stream);
  if (dtype == 1) return a.blocked16 ? decode_t<TBF16, false, true>(a, stream) : decode_t<TBF16, false, false>(a, stream);
  return a.blocked16 ? decode_t<TF32, false, true>(a, stream) : decode_t<TF32, false, false>(a, stream);
}

}  // namespace moe
