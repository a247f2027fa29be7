// The operators around the layer: the norm before a block, the norm, gate,
// dropout and residual scale behind it, and their gradients.  All of them move
// whole rows once and are bound by that; a row stays in the registers of the
// threads that work on it, and every sum is fp32 in a fixed order.
#include <algorithm>

#include "block.hpp"
#include "device_common.hpp"
#include "philox.hpp"
#include "rounding.hpp"

namespace moe {
namespace {

// 1 / sqrt(mean square + eps)
__device__ __forceinline__ float inv_rms(float sum_sq, int d, float eps) { return rsqrtf(sum_sq / (float)d + eps); }

// sigmoid and its slope from e = exp(-|g|), which neither overflows nor cancels
__device__ __forceinline__ float sigmoid(float g, float* slope = nullptr) {
  const float e = expf(-fabsf(g)), inv = 1.f / (1.f + e);
  if (slope != nullptr) *slope = e * inv * inv;
  return g >= 0.f ? inv : e * inv;
}

// Sums of N values over the NT threads of a row, in every one of them: lanes,
// then wavefronts in order.  part: [N][wavefronts of the workgroup], a place that
// no thread still reads.
template <int NT, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float* part) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if constexpr (NT > 64) {
    constexpr int W = NT / 64;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) part[i * W + wave] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = part[i * W];
#pragma unroll
      for (int w = 1; w < W; ++w) v[i] += part[i * W + w];
    }
  }
}

// Which of the EPC elements of 16-byte chunk c of row t are kept, a bit each: the
// generator's block is the eight elements from (t d + c EPC) / 8 8 on.
template <class Tr>
__device__ __forceinline__ unsigned kept(size_t t, int d, int c, uint64_t seed, uint64_t step, unsigned threshold) {
  const uint64_t at = (uint64_t)t * d + (uint64_t)c * Tr::EPC;
  const Philox r = philox(at >> 3, step, seed);
  unsigned bits = 0;
#pragma unroll
  for (int i = 0; i < Tr::EPC; ++i) {
    const unsigned h = Tr::EPC == 8 ? r.half(i) : (at & 4) ? r.half(4 + (i & 3)) : r.half(i);
    bits |= (h >= threshold ? 1u : 0u) << i;
  }
  return bits;
}

template <class Tr>
__device__ __forceinline__ uint4 chunk(const void* row, int c) {
  return static_cast<const uint4*>(row)[c];
}

// NT threads of a row, V 16-byte chunks each; 256 / NT rows (one past 256) for a
// workgroup.
template <class Tr, int NT, int V>
__global__ __launch_bounds__(NT > 256 ? NT : 256) void residual_kernel(ResidualArgs a) {
  using Elt = typename Tr::T;
  constexpr int EPC = Tr::EPC, G = NT < 256 ? 256 / NT : 1;
  __shared__ float part[2][2][NT / 64];
  const int tid = threadIdx.x % NT, chunks = a.d / EPC;
  const uint64_t seed = a.rng != nullptr ? a.rng[0] : 0, step = a.rng != nullptr ? a.rng[1] : 0;
  // (groups of one wavefront meet no barrier; larger ones are the whole workgroup.  A row's
  // sums go where the row before had none: a row may have one barrier only)
  int place = 0;
  for (size_t t = (size_t)blockIdx.x * G + threadIdx.x / NT; t < (size_t)a.T; t += (size_t)gridDim.x * G, place ^= 1) {
    const size_t row = t * a.d * sizeof(Elt);
    const auto at = [&](const void* p) { return static_cast<const char*>(p) + row; };
    uint4 rc[V], yc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * NT;
      const bool in = c < chunks;
      yc[i] = a.y != nullptr && in ? chunk<Tr>(at(a.y), c) : make_uint4(0, 0, 0, 0);
      rc[i] = in ? chunk<Tr>(at(a.res), c) : make_uint4(0, 0, 0, 0);
    }
    float o[V][EPC];
#pragma unroll
    for (int i = 0; i < V; ++i) widen<Tr>(rc[i], o[i]);
    if (a.y != nullptr) {
      float r = 1.f;
      if (a.post_w != nullptr) {
        float s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float y[EPC];
          widen<Tr>(yc[i], y);
#pragma unroll
          for (int j = 0; j < EPC; ++j) s[0] = fmaf(y[j], y[j], s[0]);
        }
        row_sum<NT>(s, part[place][0]);
        r = inv_rms(s[0], a.d, a.eps);
      }
      float mul = a.scale * a.keep_scale;
      if (a.gate != nullptr && !a.gate_full) {
        float g[EPC];
        widen<Tr>(make_uint4(sizeof(Elt) == 2 ? static_cast<const uint16_t*>(a.gate)[t] : static_cast<const uint32_t*>(a.gate)[t], 0, 0, 0), g);
        mul *= sigmoid(g[0]);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = tid + i * NT;
        if (c >= chunks) continue;
        float v[EPC];
        widen<Tr>(yc[i], v);
        if (a.post_w != nullptr) {
          float w[EPC];
          widen<Tr>(chunk<Tr>(a.post_w, c), w);
#pragma unroll
          for (int j = 0; j < EPC; ++j) v[j] *= r * w[j];
        }
        if (a.gate_full) {
          float g[EPC];
          widen<Tr>(chunk<Tr>(at(a.gate), c), g);
#pragma unroll
          for (int j = 0; j < EPC; ++j) v[j] *= sigmoid(g[j]);
        }
        // a dropped element adds nothing, whatever it holds
        const unsigned keep = a.threshold != 0 ? kept<Tr>(t, a.d, c, seed, step, a.threshold) : ~0u;
#pragma unroll
        for (int j = 0; j < EPC; ++j)
          if ((keep >> j) & 1u) o[i][j] = fmaf(mul, v[j], o[i][j]);
        static_cast<uint4*>(static_cast<void*>(static_cast<char*>(a.out) + row))[c] = round_to<Tr>(o[i]);
      }
    }
    if (a.next_w == nullptr) continue;
    // n comes from the fp32 sums, so that it is rounded once
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < EPC; ++j) s[0] = fmaf(o[i][j], o[i][j], s[0]);
    row_sum<NT>(s, part[place][1]);
    const float r = inv_rms(s[0], a.d, a.eps);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * NT;
      if (c >= chunks) continue;
      float w[EPC];
      widen<Tr>(chunk<Tr>(a.next_w, c), w);
#pragma unroll
      for (int j = 0; j < EPC; ++j) w[j] *= o[i][j] * r;
      static_cast<uint4*>(static_cast<void*>(static_cast<char*>(a.n) + row))[c] = round_to<Tr>(w);
    }
  }
}

// Gradient of residual_kernel's sum, one row at a time.  With r1 = r(x), r2 = r(y),
// z = dn next_w, D the gradient of the sum, m = keep scale / (1 - p), q = m D,
// v = y r2 post_w (or y) and c = sigmoid q post_w:
//   D = dout + r1 (z - x r1^2 mean(z x))          dres = D
//   dy = r2 (c - y r2^2 mean(c y))  (or sigmoid q)
//   dgate = sigmoid' q v  (its sum over the row for a gate per token)
//   dpost_w = sum_t sigmoid q y r2                dnext_w = sum_t dn x r1
// The sums over tokens: each thread keeps its columns' over the rows that its
// workgroup works, rows in ascending order.
template <class Tr, int NT, int V>
__global__ __launch_bounds__(NT > 256 ? NT : 256) void residual_backward_kernel(ResidualBackwardArgs a) {
  using Elt = typename Tr::T;
  constexpr int EPC = Tr::EPC, G = NT < 256 ? 256 / NT : 1;
  extern __shared__ float sums[];  // [G > 1 ? G : 0][d]
  __shared__ float part1[2][3 * (NT / 64)], part2[NT / 64];
  const int tid = threadIdx.x % NT, group = threadIdx.x / NT, chunks = a.d / EPC;
  float gp[V][EPC], gn[V][EPC];  // columns' sums of dpost_w and dnext_w
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < EPC; ++j) gp[i][j] = gn[i][j] = 0.f;
  const uint64_t seed = a.rng != nullptr ? a.rng[0] : 0, step = a.rng != nullptr ? a.rng[1] : 0;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  // (groups of one wavefront meet no barrier in the loop; larger ones are the whole workgroup;
  // a row's first sums go to the place that the row before did not use, since a norm alone
  // has no second barrier behind their reading)
  int place = 0;
  for (size_t t = (size_t)blockIdx.x * G + group; t < (size_t)a.T; t += (size_t)gridDim.x * G, place ^= 1) {
    const size_t row = t * a.d * sizeof(Elt);
    const auto at = [&](const void* p) { return static_cast<const char*>(p) + row; };
    uint4 xc[V], yc[V], dnc[V], doc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * NT;
      const bool in = c < chunks;
      xc[i] = a.next_w != nullptr && in ? chunk<Tr>(at(a.x), c) : zero;
      dnc[i] = a.next_w != nullptr && in ? chunk<Tr>(at(a.dn), c) : zero;
      yc[i] = a.y != nullptr && in ? chunk<Tr>(at(a.y), c) : zero;
      doc[i] = a.dout != nullptr && in ? chunk<Tr>(at(a.dout), c) : zero;
    }
    // squares of x, z x, squares of y
    float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * NT;
      float y[EPC];
      widen<Tr>(yc[i], y);
#pragma unroll
      for (int j = 0; j < EPC; ++j) s[2] = fmaf(y[j], y[j], s[2]);
      if (a.next_w != nullptr && c < chunks) {
        float x[EPC], dn[EPC], w[EPC];
        widen<Tr>(xc[i], x);
        widen<Tr>(dnc[i], dn);
        widen<Tr>(chunk<Tr>(a.next_w, c), w);
#pragma unroll
        for (int j = 0; j < EPC; ++j) {
          s[0] = fmaf(x[j], x[j], s[0]);
          s[1] = fmaf(dn[j] * w[j], x[j], s[1]);
        }
      }
    }
    row_sum<NT>(s, part1[place]);
    const float r1 = inv_rms(s[0], a.d, a.eps), k1 = r1 * r1 * (s[1] / (float)a.d);
    const float r2 = a.post_w != nullptr ? inv_rms(s[2], a.d, a.eps) : 1.f;
    float D[V][EPC];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * NT;
      widen<Tr>(doc[i], D[i]);
      if (c >= chunks) continue;
      if (a.next_w != nullptr) {
        float x[EPC], dn[EPC], w[EPC];
        widen<Tr>(xc[i], x);
        widen<Tr>(dnc[i], dn);
        widen<Tr>(chunk<Tr>(a.next_w, c), w);
#pragma unroll
        for (int j = 0; j < EPC; ++j) {
          gn[i][j] = fmaf(dn[j] * r1, x[j], gn[i][j]);
          D[i][j] = fmaf(r1, fmaf(dn[j], w[j], -x[j] * k1), D[i][j]);
        }
      }
      static_cast<uint4*>(static_cast<void*>(static_cast<char*>(a.dres) + row))[c] = round_to<Tr>(D[i]);
    }
    if (a.y == nullptr) continue;
    const float m = a.scale * a.keep_scale;
    float gate = 1.f, slope = 0.f;
    if (a.gate != nullptr && !a.gate_full) {
      float g[EPC];
      widen<Tr>(make_uint4(sizeof(Elt) == 2 ? static_cast<const uint16_t*>(a.gate)[t] : static_cast<const uint32_t*>(a.gate)[t], 0, 0, 0), g);
      gate = sigmoid(g[0], &slope);
    }
    // D becomes c (or sigmoid q without a norm); its product with y, and with a gate
    // for each token the same before the sigmoid, are one sum: sigmoid is a factor of it
    float cy[1] = {0.f};
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * NT;
      if (c >= chunks) continue;
      float y[EPC], w[EPC];
      widen<Tr>(yc[i], y);
#pragma unroll
      for (int j = 0; j < EPC; ++j) w[j] = 1.f;
      if (a.post_w != nullptr) widen<Tr>(chunk<Tr>(a.post_w, c), w);
      const unsigned keep = a.threshold != 0 ? kept<Tr>(t, a.d, c, seed, step, a.threshold) : ~0u;
#pragma unroll
      for (int j = 0; j < EPC; ++j) {  // what is dropped takes no part, whatever it holds
        D[i][j] = (keep >> j) & 1u ? m * D[i][j] : 0.f;
        y[j] = (keep >> j) & 1u ? y[j] : 0.f;
      }
      if (a.gate_full) {
        float g[EPC], dg[EPC];
        widen<Tr>(chunk<Tr>(at(a.gate), c), g);
#pragma unroll
        for (int j = 0; j < EPC; ++j) {
          float sl;
          const float sg = sigmoid(g[j], &sl);
          dg[j] = sl * D[i][j] * (y[j] * r2 * w[j]);
          D[i][j] *= sg;
        }
        if (a.dgate != nullptr)
          static_cast<uint4*>(static_cast<void*>(static_cast<char*>(a.dgate) + row))[c] = round_to<Tr>(dg);
      }
#pragma unroll
      for (int j = 0; j < EPC; ++j) {
        gp[i][j] = fmaf(gate * D[i][j] * r2, y[j], gp[i][j]);
        D[i][j] *= w[j];
        cy[0] = fmaf(D[i][j], y[j], cy[0]);
      }
    }
    row_sum<NT>(cy, part2);
    if (a.gate != nullptr && !a.gate_full && a.dgate != nullptr && tid == 0) {
      const float g = slope * r2 * cy[0];
      if constexpr (sizeof(Elt) == 2)
        static_cast<uint16_t*>(a.dgate)[t] = (uint16_t)f32_to_bf16(g);
      else
        static_cast<float*>(a.dgate)[t] = g;
    }
    const float k2 = r2 * r2 * (cy[0] / (float)a.d), mul = gate * r2;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * NT;
      if (c >= chunks) continue;
      if (a.post_w != nullptr) {
        float y[EPC];
        widen<Tr>(yc[i], y);
#pragma unroll
        for (int j = 0; j < EPC; ++j) D[i][j] -= y[j] * k2;
      }
#pragma unroll
      for (int j = 0; j < EPC; ++j) D[i][j] *= mul;
      static_cast<uint4*>(static_cast<void*>(static_cast<char*>(a.dy) + row))[c] = round_to<Tr>(D[i]);
    }
  }
  // this workgroup's sums: groups in order
  const auto flush = [&](float (&g)[V][EPC], float* dst) {
    if constexpr (G > 1) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = tid + i * NT;
        if (c >= chunks) continue;
#pragma unroll
        for (int j = 0; j < EPC; ++j) sums[(size_t)group * a.d + c * EPC + j] = g[i][j];
      }
      __syncthreads();
      for (int c = threadIdx.x; c < a.d; c += 256) {
        float v = sums[c];
#pragma unroll
        for (int w = 1; w < G; ++w) v += sums[(size_t)w * a.d + c];
        dst[c] = v;
      }
      __syncthreads();
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = tid + i * NT;
        if (c >= chunks) continue;
#pragma unroll
        for (int j = 0; j < EPC; j += 4)
          *reinterpret_cast<float4*>(dst + c * EPC + j) = make_float4(g[i][j], g[i][j + 1], g[i][j + 2], g[i][j + 3]);
      }
    }
  };
  if (a.dpost_w != nullptr) flush(gp, a.part + (size_t)blockIdx.x * a.d);
  if (a.dnext_w != nullptr) flush(gn, a.part + ((size_t)gridDim.x + blockIdx.x) * a.d);
}

// A weight's gradient from the workgroups' sums [groups][d]: 16 threads take 4
// columns each, 64 ranges of groups side by side, eight loads of a thread in
// flight; ranges joined in order.
__device__ __forceinline__ void add4(float4& s, const float4& v) {
  s.x += v.x;
  s.y += v.y;
  s.z += v.z;
  s.w += v.w;
}
template <class Tr>
__global__ __launch_bounds__(1024) void column_sum_kernel(const float* __restrict__ part, int groups, int d,
                                                          char* __restrict__ dpost, char* __restrict__ dnext) {
  using Elt = typename Tr::T;
  char* dst = blockIdx.y == 0 ? dpost : dnext;
  if (dst == nullptr) return;
  __shared__ float4 sums[64][16], joined[8][16];
  const int q = threadIdx.x & 15, range = threadIdx.x >> 4;
  const int c = ((int)blockIdx.x * 16 + q) * 4;
  const float* src = part + (size_t)blockIdx.y * groups * d + c;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int g0 = range; g0 < groups; g0 += 64 * 8) {
    float4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = g0 + i * 64 < groups ? *reinterpret_cast<const float4*>(src + (size_t)(g0 + i * 64) * d)
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 8; ++i) add4(s, v[i]);
  }
  sums[range][q] = s;
  __syncthreads();
  if (range < 8) {
    s = sums[range * 8][q];
#pragma unroll
    for (int i = 1; i < 8; ++i) add4(s, sums[range * 8 + i][q]);
    joined[range][q] = s;
  }
  __syncthreads();
  if (range != 0) return;
  s = joined[0][q];
#pragma unroll
  for (int i = 1; i < 8; ++i) add4(s, joined[i][q]);
  store4<Tr>(dst + (size_t)c * sizeof(Elt), s.x, s.y, s.z, s.w);
}

// out = keep x / (1 - p): eight elements for each call of the generator, kDropBlocks
// such blocks of a thread, loaded first.  out may be x.
constexpr int kDropBlocks = 2;
template <class Tr>
__global__ __launch_bounds__(256) void dropout_kernel(const char* x, int64_t n, unsigned threshold, float keep_scale,
                                                      const uint64_t* rng, char* out) {
  using Elt = typename Tr::T;
  constexpr int P = 8 / Tr::EPC;  // 16-byte chunks of a block
  const uint64_t seed = rng[0], step = rng[1];
  const int64_t full = n / 8, stride = (int64_t)gridDim.x * (256 * kDropBlocks);
  for (int64_t b0 = (int64_t)blockIdx.x * (256 * kDropBlocks) + threadIdx.x; b0 < full; b0 += stride) {
    uint4 c[kDropBlocks][P];
#pragma unroll
    for (int i = 0; i < kDropBlocks; ++i)
#pragma unroll
      for (int p = 0; p < P; ++p)
        c[i][p] = reinterpret_cast<const uint4*>(x)[min(b0 + i * 256, full - 1) * P + p];
#pragma unroll
    for (int i = 0; i < kDropBlocks; ++i) {
      const int64_t b = b0 + i * 256;
      const Philox r = philox((uint64_t)b, step, seed);
#pragma unroll
      for (int p = 0; p < P; ++p) {
        float v[Tr::EPC];
        widen<Tr>(c[i][p], v);
#pragma unroll
        for (int j = 0; j < Tr::EPC; ++j) v[j] = r.half(p * Tr::EPC + j) >= threshold ? v[j] * keep_scale : 0.f;
        if (b < full) reinterpret_cast<uint4*>(out)[b * P + p] = round_to<Tr>(v);
      }
    }
  }
  // the last, shorter block
  if (blockIdx.x == 0 && threadIdx.x == 0 && (n & 7) != 0) {
    const Philox r = philox((uint64_t)full, step, seed);
#pragma unroll
    for (int j = 0; j < 7; ++j) {
      if (j >= (int)(n & 7)) break;
      const bool keep = r.half(j) >= threshold;
      const int64_t i = full * 8 + j;
      if constexpr (sizeof(Elt) == 2) {
        const float v = bf16_to_f32(reinterpret_cast<const uint16_t*>(x)[i]);
        reinterpret_cast<uint16_t*>(out)[i] = (uint16_t)(keep ? f32_to_bf16(v * keep_scale) : 0u);
      } else {
        reinterpret_cast<float*>(out)[i] = keep ? reinterpret_cast<const float*>(x)[i] * keep_scale : 0.f;
      }
    }
  }
}

constexpr int kBackwardGroups = 512;

// Threads of a row and elements of each: the first whose product holds the row.
#define MOE_ROW_SHAPES(M) M(64, 8) M(64, 16) M(256, 8) M(256, 16) M(512, 16) M(512, 32)

template <class Tr>
hipError_t residual_t(const ResidualArgs& a, hipStream_t stream) {
#define MOE_TRY(NT, N)                                                                                      \
  if (a.d <= NT * N) {                                                                                      \
    constexpr int G = NT < 256 ? 256 / NT : 1;                                                              \
    hipLaunchKernelGGL((residual_kernel<Tr, NT, N / Tr::EPC>), dim3(std::min((a.T - 1) / G + 1, 1 << 20)),  \
                       dim3(NT > 256 ? NT : 256), 0, stream, a);                                            \
    return hipGetLastError();                                                                               \
  }
  MOE_ROW_SHAPES(MOE_TRY)
#undef MOE_TRY
  return hipErrorInvalidValue;
}

template <class Tr>
hipError_t residual_backward_t(const ResidualBackwardArgs& a, hipStream_t stream) {
  const int groups = residual_backward_groups(a.T, a.d);
  hipError_t e = hipErrorInvalidValue;
  bool launched = false;
#define MOE_TRY(NT, N)                                                                                      \
  if (!launched && a.d <= NT * N) {                                                                         \
    launched = true;                                                                                        \
    hipLaunchKernelGGL((residual_backward_kernel<Tr, NT, N / Tr::EPC>), dim3(groups),                       \
                       dim3(NT > 256 ? NT : 256), NT < 256 ? (size_t)(256 / NT) * a.d * 4 : 0, stream, a);  \
    e = hipGetLastError();                                                                                  \
  }
  MOE_ROW_SHAPES(MOE_TRY)
#undef MOE_TRY
  if (e != hipSuccess || (a.dpost_w == nullptr && a.dnext_w == nullptr)) return e;
  hipLaunchKernelGGL(column_sum_kernel<Tr>, dim3(a.d / 64, 2), dim3(1024), 0, stream, a.part, groups, a.d,
                     static_cast<char*>(a.dpost_w), static_cast<char*>(a.dnext_w));
  return hipGetLastError();
}

}  // namespace

int residual_backward_groups(int T, int d) {
  const int per = d <= 1024 ? 4 : 1;  // rows side by side in a workgroup
  return std::min((T - 1) / per + 1, kBackwardGroups);
}

hipError_t launch_residual(int dtype, const ResidualArgs& a, hipStream_t stream) {
  return dtype == 1 ? residual_t<TBF16>(a, stream) : residual_t<TF32>(a, stream);
}

hipError_t launch_residual_backward(int dtype, const ResidualBackwardArgs& a, hipStream_t stream) {
  return dtype == 1 ? residual_backward_t<TBF16>(a, stream) : residual_backward_t<TF32>(a, stream);
}

hipError_t launch_dropout(int dtype, const void* x, int64_t n, unsigned threshold, float keep_scale,
                          const uint64_t* rng, void* out, hipStream_t stream) {
  const int64_t per = 256 * kDropBlocks, blocks = (n + 7) / 8;
  const dim3 grid((unsigned)std::min<int64_t>((blocks + per - 1) / per, 1 << 20));
  if (dtype == 1)
    hipLaunchKernelGGL(dropout_kernel<TBF16>, grid, dim3(256), 0, stream, static_cast<const char*>(x), n, threshold,
                       keep_scale, rng, static_cast<char*>(out));
  else
    hipLaunchKernelGGL(dropout_kernel<TF32>, grid, dim3(256), 0, stream, static_cast<const char*>(x), n, threshold,
                       keep_scale, rng, static_cast<char*>(out));
  return hipGetLastError();
}

}  // namespace moe
