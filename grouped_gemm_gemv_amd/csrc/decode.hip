// The layer for a few tokens (T <= 16): norm, router, experts, combine and
// residual in two kernels.
//
// With at most 16 tokens every product of the layer has at most 16 columns, the
// width of one 16x16 matrix instruction, so the weights are the instruction's rows
// and all of the batch's tokens its columns: an expert is multiplied with every
// token, chosen or not, and the combine picks.  That needs no permutation and
// no dispatch arrays, the matrix cores have the room (16 rows x 64 bytes of weights
// per instruction: at the rate of HBM one in 90 cycles of a compute unit), and the
// work is a single stream over the active experts' weights, which is what bounds
// it.
//
//   decode_up_kernel    every workgroup norms the tokens into LDS, routes them
//                       (all of them, each workgroup for itself: E d weights
//                       from L2 against a launch of its own), and works units
//                       of 8 columns of F of an active expert: an MFMA tile of
//                       8 gate rows above 8 up rows, K split over the
//                       wavefronts, h = silu(g) u
//   decode_down_kernel  a workgroup for each 16 columns of d: one sum over
//                       the active experts' F columns, split over the
//                       wavefronts; where an expert ends, its sum is weighted
//                       into the total, token by token
//
// Norm: with p = x norm_w (exact in two bf16 terms where both are bf16), the router
// takes both terms and the experts the first, p rounded to bf16; 1 / rms is a
// factor of each fp32 sum.  So logits have fp32's accuracy.  h is rounded to the
// shape's type; nothing else is before the output.
#include <algorithm>

#include "block.hpp"
#include "device_common.hpp"

namespace moe {
namespace {

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

// Weights: read once, by one workgroup.
__device__ __forceinline__ uint4 load_stream(const char* p) {
  return __builtin_bit_cast(uint4, __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p)));
}
__device__ __forceinline__ uint4 load16(const char* p) { return *reinterpret_cast<const uint4*>(p); }

// Eight OCP E4M3 codes to the bf16 values they are exactly.
__device__ __forceinline__ uint4 widen8(unsigned lo, unsigned hi) {
  return uint4{__builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false)),
               __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true)),
               __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false)),
               __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true))};
}

// Barrier over LDS alone: loads from memory stay in flight across it.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
}

constexpr int kWaves = 8;        // wavefronts of either kernel
constexpr int kDepth = 8;        // weight loads of a wavefront in flight
constexpr int kUnitCols = 8;     // columns of F of a unit
constexpr int kMaxGrid = 256;    // workgroups of the first kernel: one for each compute unit
constexpr size_t kRedBytes = 2 * kWaves * 1024;

// Storage of the weights: bytes from one row, and from one 64-byte piece of a row, to
// the next.
struct Rows {
  size_t row_bytes;
  int blocked;
  __device__ __forceinline__ size_t at(int row) const {
    return blocked ? (size_t)(row >> 4) * 16 * row_bytes + (size_t)(row & 15) * 64 : (size_t)row * row_bytes;
  }
  __device__ __forceinline__ int step() const { return blocked ? 1024 : 64; }
};

template <class Tr, bool Q>
__device__ __forceinline__ f32x4_t mma_chunk(const uint4& w, const uint4 (&b)[Q ? 2 : 1], f32x4_t acc) {
  if constexpr (Q) {
    acc = mma16<Tr>(widen8(w.x, w.y), b[0], acc);
    return mma16<Tr>(widen8(w.z, w.w), b[1], acc);
  } else {
    return mma16<Tr>(w, b[0], acc);
  }
}

// Q: E4M3 weights.  NE: 16-expert tiles of the router at a time.
template <class Tr, bool Q, int NE>
__global__ __launch_bounds__(64 * kWaves) void decode_up_kernel(DecodeArgs a) {
  using Elt = typename Tr::T;
  constexpr int EB = sizeof(Elt), WB = Q ? 1 : EB, KB = 64 / EB, NB = Q ? 2 : 1;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  __shared__ float part_sq[kWaves][kDecodeTokens];
  __shared__ int list[256], wave_count[4];
  const int T = a.T, E = a.E, d = a.d, F = a.F;
  char* xs = lds;                                                       // [d / KB][T][64 bytes]
  f32x4_t* red = reinterpret_cast<f32x4_t*>(lds + (size_t)T * d * EB);  // [2][kWaves][64]
  float* logit = reinterpret_cast<float*>(reinterpret_cast<char*>(red) + kRedBytes);  // [T][E]
  float* wt = logit + T * E;                                            // [E][T]

  const int lane = threadIdx.x & 63, tok = lane & 15, piece = lane >> 4, tc = min(tok, T - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool normed = a.norm_w != nullptr, route = a.w_router != nullptr;
  const size_t xrow = (size_t)d * EB;
  const int blocks = d / KB;

  for (int i = threadIdx.x; i < T * E; i += 64 * kWaves) wt[i] = 0.f;

  // x norm_w into LDS, the tokens' squares, and the router's products
  float sq = 0.f, inv = 1.f;
  for (int e0 = 0; e0 == 0 || (route && e0 < E); e0 += 16 * NE) {
    constexpr int U = NE == 1 ? 8 : 4;
    f32x4_t acc[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) acc[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int base = wave; base < blocks; base += kWaves * U) {
      uint4 xv[U], gv[U], wv[U][NE];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const size_t o = (size_t)min(base + u * kWaves, blocks - 1) * 64 + piece * 16;
        xv[u] = load16(static_cast<const char*>(a.x) + tc * xrow + o);
        if (normed) gv[u] = load16(static_cast<const char*>(a.norm_w) + o);
        if (route) {
#pragma unroll
          for (int i = 0; i < NE; ++i)
            wv[u][i] = load16(static_cast<const char*>(a.w_router) + (size_t)min(e0 + i * 16 + tok, E - 1) * xrow + o);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int b = base + u * kWaves;
        if (b >= blocks) continue;
        uint4 hi = xv[u], lo = make_uint4(0, 0, 0, 0);
        if (normed) {
          float x[Tr::EPC], g[Tr::EPC];
          widen<Tr>(xv[u], x);
          widen<Tr>(gv[u], g);
          if (e0 == 0) {
#pragma unroll
            for (int j = 0; j < Tr::EPC; ++j) sq = fmaf(x[j], x[j], sq);
          }
#pragma unroll
          for (int j = 0; j < Tr::EPC; ++j) g[j] *= x[j];
          hi = narrow<Tr>(g);
          if constexpr (EB == 2) {
            widen<Tr>(hi, x);
#pragma unroll
            for (int j = 0; j < Tr::EPC; ++j) g[j] -= x[j];
            lo = narrow<Tr>(g);
          }
        }
        if (e0 == 0 && tok < T) *reinterpret_cast<uint4*>(xs + ((size_t)b * T + tok) * 64 + piece * 16) = hi;
        if (route) {
#pragma unroll
          for (int i = 0; i < NE; ++i) {
            acc[i] = mma16<Tr>(wv[u][i], hi, acc[i]);
            if (EB == 2 && normed) acc[i] = mma16<Tr>(wv[u][i], lo, acc[i]);
          }
        }
      }
    }
    if (e0 == 0 && normed) {
      sq += __shfl_xor(sq, 16);
      sq += __shfl_xor(sq, 32);
      if (lane < kDecodeTokens) part_sq[wave][lane] = sq;
    }
    __syncthreads();
    if (e0 == 0 && normed) {
      float s = part_sq[0][tok];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) s += part_sq[w][tok];
      inv = rsqrtf(s / (float)d + a.eps);  // of token `tok`, in every lane
    }
    if (!route) break;
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
        if (e < E && tok < T) logit[tok * E + e] = s * inv + (a.bias != nullptr ? a.bias[e] : 0.f);
      }
      __syncthreads();
    }
  }

  const bool first = blockIdx.x == 0;
  if (route) {
    // Top-k by rank: an expert's slot is the number of experts ahead of it (a larger
    // logit, or an equal one at a lower index).  A NaN ranks lowest.
    for (int t = wave; t < T; t += kWaves) {
      const float* z = logit + t * E;
      float v[4], key[4];
      int rank[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int e = lane + 64 * q;
        v[q] = e < E ? z[e] : 0.f;
        key[q] = fmaxf(v[q], -INFINITY);
        rank[q] = e < E ? 0 : 256;
      }
      for (int f = 0; f < E; ++f) {
        const float zf = fmaxf(z[f], -INFINITY);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (64 * q < E) rank[q] += (zf > key[q] || (zf == key[q] && f < lane + 64 * q)) ? 1 : 0;
      }
      float top = -INFINITY;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (rank[q] < a.k) top = fmaxf(top, key[q]);
#pragma unroll
      for (int o = 32; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
      float ex[4], sum = 0.f;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        ex[q] = rank[q] < a.k && v[q] != -INFINITY ? expf(v[q] - top) : 0.f;
        sum += ex[q];
      }
      sum = wave_sum(sum);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (rank[q] >= a.k) continue;
        const int e = lane + 64 * q;
        const float w = sum == 0.f ? 0.f : ex[q] / sum;  // (every expert masked by a bias of -inf)
        wt[e * T + t] = w;
        if (first && a.ids != nullptr) a.ids[t * a.k + rank[q]] = e;
        if (first && a.w != nullptr) a.w[t * a.k + rank[q]] = w;
      }
    }
  } else if ((int)threadIdx.x < T) {
    // the caller's routing: slots in order, so that an expert chosen twice has one weight
    for (int j = 0; j < a.k; ++j) {
      const int e = a.ids[threadIdx.x * a.k + j];
      if (e >= 0 && e < E) wt[e * T + threadIdx.x] += a.w[threadIdx.x * a.k + j];
    }
  }
  __syncthreads();

  // the experts with a weight for any token, ascending
  bool active = false;
  if ((int)threadIdx.x < E)
    for (int t = 0; t < T; ++t) active = active || wt[threadIdx.x * T + t] != 0.f;
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
    for (int i = threadIdx.x; i < n_active; i += 64 * kWaves) a.table->expert[i] = list[i];
    for (int i = threadIdx.x; i < n_active * T; i += 64 * kWaves) a.table->weight[i / T][i % T] = wt[list[i / T] * T + i % T];
  }

  // ---- gate and up: units of 8 columns, dealt to the workgroups in turn
  const int per = F / kUnitCols, total = n_active * per;
  const int chunks = d * WB / 64;
  const int c0 = chunks * wave / kWaves, mine = chunks * (wave + 1) / kWaves - c0;
  const int grid = (int)gridDim.x;
  const int units = (int)blockIdx.x < total ? (total - (int)blockIdx.x + grid - 1) / grid : 0;
  if (units == 0) return;
  const Rows rows{(size_t)d * WB, a.blocked16};
  const int step = rows.step();
  const char* base = static_cast<const char*>(tok < 8 ? a.w_gate : a.w_up) + piece * 16 + (size_t)c0 * step;
  const auto unit_at = [&](int i) {
    const int u = (int)blockIdx.x + i * grid, e = list[u / per];
    return base + (size_t)e * F * rows.row_bytes + rows.at((u % per) * kUnitCols + (tok & 7));
  };
  // a unit's sums of all wavefronts to h, by one wavefront, each unit another's turn
  const auto finish = [&](int i, f32x4_t acc) {
    red[((i & 1) * kWaves + wave) * 64 + lane] = acc;
    lds_barrier();
    if (wave != i % kWaves) return;
    f32x4_t s = red[(i & 1) * kWaves * 64 + lane];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) s += red[((i & 1) * kWaves + w) * 64 + lane];
    const int u = (int)blockIdx.x + i * grid, n = u / per, f0 = (u % per) * kUnitCols;
#pragma unroll
    for (int r = 0; r < 4; ++r) s[r] *= inv;
    if constexpr (Q) {
      const float4 sc = *reinterpret_cast<const float4*>((piece < 2 ? a.s_gate : a.s_up) + (size_t)list[n] * F + f0 + (piece & 1) * 4);
      s[0] *= sc.x, s[1] *= sc.y, s[2] *= sc.z, s[3] *= sc.w;
    }
    // rows 0..7 (pieces 0, 1) are the gate's columns, rows 8..15 the same columns of up
    float hv[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float up = __shfl_down(s[r], 32);
      hv[r] = s[r] / (1.f + __expf(-s[r])) * up;
    }
    if (piece < 2 && tok < T) {
      const int f = f0 + piece * 4;
      store4<Tr>(static_cast<char*>(a.h) + (((size_t)n * (F / KB) + f / KB) * T + tok) * 64 + (f % KB) * EB, hv[0], hv[1],
                 hv[2], hv[3]);
    }
  };
  if (mine == 0) {  // (fewer chunks than wavefronts)
    for (int i = 0; i < units; ++i) finish(i, f32x4_t{0.f, 0.f, 0.f, 0.f});
    return;
  }
  // kDepth loads in flight, across units; behind the last unit the cursor repeats its
  // last chunk
  int li = 0, lc = 0;
  const char* lp = unit_at(0);
  const auto load = [&]() {
    const uint4 v = load_stream(lp);
    if (++lc < mine) {
      lp += step;
    } else if (li + 1 < units) {
      lp = unit_at(++li);
      lc = 0;
    } else {
      --lc;
    }
    return v;
  };
  const char* xlane = xs + (Q ? ((size_t)(piece >> 1) * T + tc) * 64 + (piece & 1) * 32 : (size_t)tc * 64 + piece * 16) +
                      (size_t)c0 * NB * T * 64;
  int ui = 0, uc = 0;
  f32x4_t acc{0.f, 0.f, 0.f, 0.f};
  const auto work = [&](const uint4& w) {
    uint4 b[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j) b[j] = *reinterpret_cast<const uint4*>(xlane + (size_t)uc * NB * T * 64 + j * 16);
    acc = mma_chunk<Tr, Q>(w, b, acc);
    if (++uc == mine) {
      finish(ui, acc);
      ++ui;
      uc = 0;
      acc = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
  };
  uint4 ring[kDepth];
#pragma unroll
  for (int j = 0; j < kDepth; ++j) ring[j] = load();
  int left = units * mine;
  for (; left >= kDepth; left -= kDepth) {
#pragma unroll
    for (int j = 0; j < kDepth; ++j) {
      work(ring[j]);
      ring[j] = load();
    }
  }
#pragma unroll
  for (int j = 0; j < kDepth; ++j)
    if (j < left) work(ring[j]);
}

template <class Tr, bool Q>
__global__ __launch_bounds__(64 * kWaves) void decode_down_kernel(DecodeArgs a) {
  using Elt = typename Tr::T;
  constexpr int EB = sizeof(Elt), WB = Q ? 1 : EB, NB = Q ? 2 : 1;
  __shared__ f32x4_t red[kWaves][64];
  __shared__ float wts[256][kDecodeTokens];
  __shared__ float scale[Q ? 256 : 1][16];
  __shared__ int list[256];
  const int T = a.T, d = a.d, F = a.F;
  const int lane = threadIdx.x & 63, tok = lane & 15, piece = lane >> 4, tc = min(tok, T - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int o0 = (int)blockIdx.x * 16;
  const int n_active = __builtin_amdgcn_readfirstlane(a.table->n_active);
  for (int i = threadIdx.x; i < n_active; i += 64 * kWaves) list[i] = a.table->expert[i];
  for (int i = threadIdx.x; i < n_active * kDecodeTokens; i += 64 * kWaves) {
    const int n = i / kDecodeTokens, t = i % kDecodeTokens;
    wts[n][t] = t < T ? a.table->weight[n][t] : 0.f;
    if constexpr (Q) scale[n][t] = a.s_down[(size_t)a.table->expert[n] * d + o0 + t];
  }
  __syncthreads();

  const int per = F * WB / 64, total = n_active * per;  // chunks of an expert, of all
  const int i0 = (int)((long long)total * wave / kWaves), i1 = (int)((long long)total * (wave + 1) / kWaves);
  f32x4_t sum{0.f, 0.f, 0.f, 0.f};
  if (i0 < i1) {
    const Rows rows{(size_t)F * WB, a.blocked16};
    const int step = rows.step();
    const char* base = static_cast<const char*>(a.w_down) + rows.at(o0 + tok) + piece * 16;
    const size_t expert_bytes = (size_t)d * rows.row_bytes;
    const int bstep = T * 64 * NB;
    int ln = i0 / per, lc = i0 % per, li = i0;
    const char* lp = base + list[ln] * expert_bytes + (size_t)lc * step;
    const char* bp = static_cast<const char*>(a.h) + (size_t)i0 * bstep +
                     (Q ? ((size_t)(piece >> 1) * T + tc) * 64 + (piece & 1) * 32 : (size_t)tc * 64 + piece * 16);
    uint4 ring[kDepth], act[kDepth][NB];
    const auto load = [&](int j) {
      ring[j] = load_stream(lp);
#pragma unroll
      for (int q = 0; q < NB; ++q) act[j][q] = load16(bp + q * 16);
      if (++li >= i1) return;  // behind the last chunk: it again
      bp += bstep;
      if (++lc < per) {
        lp += step;
      } else {
        lc = 0;
        lp = base + list[++ln] * expert_bytes;
      }
    };
    int n = i0 / per, c = i0 % per;
    f32x4_t acc{0.f, 0.f, 0.f, 0.f};
    // a token that did not choose the expert takes nothing of its sum, whatever that holds
    const auto fold = [&]() {
      const float w = wts[n][tok];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float v = acc[r];
        if constexpr (Q) v *= scale[n][piece * 4 + r];
        sum[r] = w != 0.f ? fmaf(w, v, sum[r]) : sum[r];
      }
      acc = f32x4_t{0.f, 0.f, 0.f, 0.f};
    };
    const auto work = [&](int j) {
      acc = mma_chunk<Tr, Q>(ring[j], act[j], acc);
      if (++c == per) {
        fold();
        ++n;
        c = 0;
      }
    };
#pragma unroll
    for (int j = 0; j < kDepth; ++j) load(j);
    int left = i1 - i0;
    for (; left >= kDepth; left -= kDepth) {
#pragma unroll
      for (int j = 0; j < kDepth; ++j) {
        work(j);
        load(j);
      }
    }
#pragma unroll
    for (int j = 0; j < kDepth; ++j)
      if (j < left) work(j);
    if (c != 0) fold();
  }
  red[wave][lane] = sum;
  __syncthreads();
  if (wave != 0 || tok >= T) return;
#pragma unroll
  for (int w = 1; w < kWaves; ++w) sum += red[w][lane];
  const size_t at = ((size_t)tok * d + o0 + piece * 4) * EB;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    sum[r] *= a.scale;
    if (a.res != nullptr) {
      const char* p = static_cast<const char*>(a.res) + at + r * EB;
      sum[r] += EB == 2 ? bf16_to_f32(*reinterpret_cast<const uint16_t*>(p)) : *reinterpret_cast<const float*>(p);
    }
  }
  store4<Tr>(static_cast<char*>(a.out) + at, sum[0], sum[1], sum[2], sum[3]);
}

template <class Tr, bool Q>
hipError_t decode_t(const DecodeArgs& a, hipStream_t stream) {
  const size_t lds = decode_lds_bytes(sizeof(typename Tr::T), a.T, a.d, a.E);
  const int64_t units = (int64_t)std::min(a.E, a.T * a.k) * (a.F / kUnitCols);
  const dim3 grid((unsigned)std::min<int64_t>(units, kMaxGrid));
  if (a.E <= 16)
    hipLaunchKernelGGL((decode_up_kernel<Tr, Q, 1>), grid, dim3(64 * kWaves), lds, stream, a);
  else
    hipLaunchKernelGGL((decode_up_kernel<Tr, Q, 4>), grid, dim3(64 * kWaves), lds, stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((decode_down_kernel<Tr, Q>), dim3(a.d / 16), dim3(64 * kWaves), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

// x [T][d], the wavefronts' sums, logits and weights [T][E] each.
size_t decode_lds_bytes(int elt_bytes, int T, int d, int E) {
  return (size_t)T * d * elt_bytes + kRedBytes + (size_t)8 * T * E;
}

hipError_t launch_decode(int dtype, const DecodeArgs& a, hipStream_t stream) {
  if (a.s_gate != nullptr) return decode_t<TBF16, true>(a, stream);
  return dtype == 1 ? decode_t<TBF16, false>(a, stream) : decode_t<TF32, false>(a, stream);
}

}  // namespace moe
