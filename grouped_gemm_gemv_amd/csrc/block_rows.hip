// The operators around the layer: the norm before a block, the norm, gate,
// dropout and residual scale behind it, and their gradients.  All of them move
// whole rows once and are bound by that; a row stays in the registers of the
// threads that work on it, and every sum is fp32 in a fixed order.  (Gradients of wide rows
// need more registers than 1024 threads have: past 8192 elements of bf16 64 of them spill, in
// fp32 12 past 4096 and 90 past 8192.)
#include <algorithm>

#include "block.hpp"
#include "device_common.hpp"
#include "philox.hpp"
#include "vec.hpp"

namespace moe {
namespace {

// 1 / sqrt(mean square + eps); inv_d = 1 / d, as a division is ten instructions and a row has
// four of them
__device__ __forceinline__ float inv_rms(float sum_sq, float inv_d, float eps) { return rsqrtf(fmaf(sum_sq, inv_d, eps)); }

// sigmoid and its slope from e = exp(-|g|), which neither overflows nor cancels
__device__ __forceinline__ float sigmoid(float g, float* slope = nullptr) {
  const float e = expf(-fabsf(g)), inv = __builtin_amdgcn_rcpf(1.f + e);
  if (slope != nullptr) *slope = e * inv * inv;
  return g >= 0.f ? inv : e * inv;
}

// Sums of N values over the NT threads of a row, in every one of them: lanes,
// then wavefronts in order.  part: [N][wavefronts of the workgroup], a place that
// no thread still reads.
template <int NT, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float* part) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_fold(v[i], [](float x, float y) { return x + y; });
  if constexpr (NT > 64) {
    constexpr int W = NT / 64;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) part[i * W + wave] = v[i];
    }
    lds_barrier();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = part[i * W];
#pragma unroll
      for (int w = 1; w < W; ++w) v[i] += part[i * W + w];
    }
  }
}

// Which of the EPC elements of 16-byte chunk c of row t are kept: the generator's block
// is the eight elements that hold them.
template <class Tr>
struct Kept {
  Philox r;
  unsigned threshold;
  __device__ __forceinline__ Kept(size_t t, int d, int c, uint64_t seed, uint64_t step, unsigned threshold)
      : threshold(threshold) {
    const uint64_t at = (uint64_t)t * d + (uint64_t)c * Tr::EPC;
    r = philox(at >> 3, step, seed);
    if (Tr::EPC == 4 && (at & 4)) r.w[0] = r.w[2], r.w[1] = r.w[3];
  }
  __device__ __forceinline__ bool operator()(int j) const { return r.half(j) >= threshold; }
};

// Chunk c of a row, zeros past its last one.
__device__ __forceinline__ uint4 chunk(const void* row, int c, int chunks) {
  uint4 v = make_uint4(0, 0, 0, 0);
  if (c < chunks) v = load16(static_cast<const char*>(row) + (unsigned)c * 16u);
  return v;
}
__device__ __forceinline__ void put(void* row, int c, int chunks, const uint4& v) {
  if (c < chunks) *reinterpret_cast<u32x4*>(static_cast<char*>(row) + (unsigned)c * 16u) = __builtin_bit_cast(u32x4, v);
}

// Threads of a workgroup for rows of NT threads: short rows share one.
constexpr int block_of(int NT) { return NT == 64 ? 256 : NT; }

// A bf16 or fp32 value in a chunk of its own.
template <class Tr>
__device__ __forceinline__ float element(const void* p, size_t i) {
  if constexpr (Tr::EPC == 8)
    return bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
  else
    return static_cast<const float*>(p)[i];
}

// The sum, and a norm behind it, one row at a time: NT threads of a row, V 16-byte chunks
// each.  Bound by memory: 4096 x 4096 bf16 with both norms, a gate a token and dropout takes
// 25 to 26 us for 134 MB, 5.1 to 5.5 TB/s with its ramp; a norm alone 11.4 in a loop of calls, 5.9 TB/s.
template <class Tr, int NT, int V>
__global__ __launch_bounds__(block_of(NT)) void residual_kernel(ResidualArgs a) {
  constexpr int EPC = Tr::EPC, G = block_of(NT) / NT;
  __shared__ float part[2][2][NT / 64];
  const int tid = threadIdx.x % NT, chunks = a.d / EPC;
  const uint64_t seed = a.rng != nullptr ? a.rng[0] : 0, step = a.rng != nullptr ? a.rng[1] : 0;
  const size_t width = (size_t)a.d * sizeof(typename Tr::T);
  const float inv_d = 1.f / (float)a.d;
  // The weights stay in registers, and where these allow a row is loaded while the one
  // before it is worked
  constexpr bool kAhead = V * EPC <= 8;
  uint4 rc[V], yc[V], pwc[V], nwc[V];
  const auto load_row = [&](size_t t) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * NT;
      yc[i] = a.y != nullptr ? chunk(static_cast<const char*>(a.y) + t * width, c, chunks) : make_uint4(0, 0, 0, 0);
      rc[i] = chunk(static_cast<const char*>(a.res) + t * width, c, chunks);
    }
  };
#pragma unroll
  for (int i = 0; i < V; ++i) {
    pwc[i] = a.post_w != nullptr ? chunk(a.post_w, tid + i * NT, chunks) : make_uint4(0, 0, 0, 0);
    nwc[i] = a.next_w != nullptr ? chunk(a.next_w, tid + i * NT, chunks) : make_uint4(0, 0, 0, 0);
  }
  const size_t first = (size_t)blockIdx.x * G + __builtin_amdgcn_readfirstlane(threadIdx.x / NT);
  const size_t ahead = (size_t)gridDim.x * G;
  if (kAhead && first < (size_t)a.T) load_row(first);
  // (groups of one wavefront meet no barrier; larger ones are the whole workgroup.  A row's
  // sums go where the row before had none: a row may have one barrier only)
  int place = 0;
  for (size_t t = first; t < (size_t)a.T; t += ahead, place ^= 1) {
    const auto at = [&](const void* p) { return static_cast<const char*>(p) + t * width; };
    const auto to = [&](void* p) { return static_cast<char*>(p) + t * width; };
    if (!kAhead) load_row(t);
    float o[V][EPC];
#pragma unroll
    for (int i = 0; i < V; ++i) widen<Tr>(rc[i], o[i]);
    if (a.y != nullptr) {
      float mul = a.scale * a.keep_scale;
      if (a.gate != nullptr && !a.gate_full) mul *= sigmoid(element<Tr>(a.gate, t));
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
        mul *= inv_rms(s[0], inv_d, a.eps);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = tid + i * NT;
        float v[EPC];
        widen<Tr>(yc[i], v);
        if (a.post_w != nullptr) {
          float w[EPC];
          widen<Tr>(pwc[i], w);
#pragma unroll
          for (int j = 0; j < EPC; ++j) v[j] *= w[j];
        }
        if (a.gate_full) {
          float g[EPC];
          widen<Tr>(chunk(at(a.gate), c, chunks), g);
#pragma unroll
          for (int j = 0; j < EPC; ++j) v[j] *= sigmoid(g[j]);
        }
        if (a.threshold != 0) {  // a dropped element adds nothing, whatever it holds
          const Kept<Tr> keep(t, a.d, c, seed, step, a.threshold);
#pragma unroll
          for (int j = 0; j < EPC; ++j) v[j] = keep(j) ? v[j] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < EPC; ++j) o[i][j] = fmaf(mul, v[j], o[i][j]);
        put(to(a.out), c, chunks, round_to<Tr>(o[i]));
      }
    }
    if (kAhead && t + ahead < (size_t)a.T) load_row(t + ahead);  // (this row's are used up)
    if (a.next_w == nullptr) continue;
    // n comes from the fp32 sums, so that it is rounded once
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < EPC; ++j) s[0] = fmaf(o[i][j], o[i][j], s[0]);
    row_sum<NT>(s, part[place][1]);
    const float r = inv_rms(s[0], inv_d, a.eps);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * NT;
      float w[EPC];
      widen<Tr>(nwc[i], w);
#pragma unroll
      for (int j = 0; j < EPC; ++j) w[j] *= o[i][j] * r;
      put(to(a.n), c, chunks, round_to<Tr>(w));
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
// workgroup works, rows in ascending order.  4096 x 4096 bf16 with both norms, a gate a token
// and dropout: 201 MB and 17 of partial sums in 47 to 51 us, 4.5 TB/s; the generator is 2.5 us of
// that and the sums over a row most of the rest of what memory does not take.  With what spills it
// is slower by far (both kernels, 201 to 203 MB: 2048 x 8192 45 us, 2048 x 8256 173, 1024 x 16384 120).
template <class Tr, int NT, int V>
__global__ __launch_bounds__(block_of(NT)) void residual_backward_kernel(ResidualBackwardArgs a) {
  using Elt = typename Tr::T;
  constexpr int EPC = Tr::EPC, B = block_of(NT), G = B / NT;
  extern __shared__ float sums[];  // [G > 1 ? G : 0][d]
  __shared__ float part1[2][3 * (NT / 64)], part2[2][NT / 64];
  const int tid = threadIdx.x % NT, group = __builtin_amdgcn_readfirstlane(threadIdx.x / NT), chunks = a.d / EPC;
  float gp[V][EPC], gn[V][EPC];  // columns' sums of dpost_w and dnext_w
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < EPC; ++j) gp[i][j] = gn[i][j] = 0.f;
  const uint64_t seed = a.rng != nullptr ? a.rng[0] : 0, step = a.rng != nullptr ? a.rng[1] : 0;
  const size_t width = (size_t)a.d * sizeof(Elt);
  const float inv_d = 1.f / (float)a.d;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  // Rows' loads run a row ahead where their registers allow: they are issued between the two
  // sums of the row before, when its own are used up, and no barrier waits for them
  // (4096 x 4096 with everything: 52 us, 59 without)
  constexpr bool kAhead = V * EPC <= 8;
  uint4 xc[V], yc[V], dnc[V], doc[V], pwc[V], nwc[V];
  const auto load_y = [&](size_t t, uint4 (&y)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      y[i] = a.y != nullptr ? chunk(static_cast<const char*>(a.y) + t * width, tid + i * NT, chunks) : zero;
  };
  const auto load_row = [&](size_t t, uint4 (&x)[V], uint4 (&dn)[V], uint4 (&dout)[V]) {
    const auto at = [&](const void* p) { return static_cast<const char*>(p) + t * width; };
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * NT;
      x[i] = a.next_w != nullptr ? chunk(at(a.x), c, chunks) : zero;
      dn[i] = a.next_w != nullptr ? chunk(at(a.dn), c, chunks) : zero;
      dout[i] = a.dout != nullptr ? chunk(at(a.dout), c, chunks) : zero;
    }
  };
#pragma unroll
  for (int i = 0; i < V; ++i) {
    pwc[i] = a.post_w != nullptr ? chunk(a.post_w, tid + i * NT, chunks) : zero;
    nwc[i] = a.next_w != nullptr ? chunk(a.next_w, tid + i * NT, chunks) : zero;
  }
  const size_t first = (size_t)blockIdx.x * G + group, ahead = (size_t)gridDim.x * G;
  if (kAhead && first < (size_t)a.T) {
    load_row(first, xc, dnc, doc);
    load_y(first, yc);
  }
  // (groups of one wavefront meet no barrier in the loop; larger ones are the whole workgroup.
  // A row may have one barrier only: the first sums' for a norm alone, the second's for a gate a
  // token without norms.  So both go to the place that the row before did not use: a wavefront
  // writes there again only two rows on, behind a barrier that all have reached after reading)
  int place = 0;
  for (size_t t = first; t < (size_t)a.T; t += ahead, place ^= 1) {
    const auto at = [&](const void* p) { return static_cast<const char*>(p) + t * width; };
    const auto to = [&](void* p) { return static_cast<char*>(p) + t * width; };
    if (!kAhead) {
      load_row(t, xc, dnc, doc);
      load_y(t, yc);
    }
    // squares of x, z x, squares of y
    float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (a.post_w != nullptr) {
        float y[EPC];
        widen<Tr>(yc[i], y);
#pragma unroll
        for (int j = 0; j < EPC; ++j) s[2] = fmaf(y[j], y[j], s[2]);
      }
      if (a.next_w != nullptr) {
        float x[EPC], dn[EPC], w[EPC];
        widen<Tr>(xc[i], x);
        widen<Tr>(dnc[i], dn);
        widen<Tr>(nwc[i], w);
#pragma unroll
        for (int j = 0; j < EPC; ++j) {
          s[0] = fmaf(x[j], x[j], s[0]);
          s[1] = fmaf(dn[j] * x[j], w[j], s[1]);
        }
      }
    }
    if (a.next_w != nullptr || a.post_w != nullptr) row_sum<NT>(s, part1[place]);
    // (the mean first: r1^3 alone leaves fp32 for rows below 1e-12 or above 1e12)
    const float r1 = inv_rms(s[0], inv_d, a.eps), k1 = -(s[1] * inv_d * r1) * r1 * r1;
    const float r2 = a.post_w != nullptr ? inv_rms(s[2], inv_d, a.eps) : 1.f;
    float D[V][EPC];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * NT;
      widen<Tr>(doc[i], D[i]);
      if (a.next_w != nullptr) {
        float x[EPC], dn[EPC], w[EPC];
        widen<Tr>(xc[i], x);
        widen<Tr>(dnc[i], dn);
        widen<Tr>(nwc[i], w);
#pragma unroll
        for (int j = 0; j < EPC; ++j) {
          dn[j] *= r1;
          gn[i][j] = fmaf(dn[j], x[j], gn[i][j]);
          D[i][j] += fmaf(dn[j], w[j], x[j] * k1);
        }
      }
      put(to(a.dres), c, chunks, round_to<Tr>(D[i]));
    }
    // the next row's loads: of what is used up, and of y beside this row's
    uint4 yn[V];
    if (kAhead && t + ahead < (size_t)a.T) {
      load_row(t + ahead, xc, dnc, doc);
      load_y(t + ahead, yn);
    }
    if (a.y == nullptr) continue;
    float gate = 1.f, slope = 0.f;
    if (a.gate != nullptr && !a.gate_full) gate = sigmoid(element<Tr>(a.gate, t), &slope);
    // D becomes q (times the sigmoid of a full gate); its product with y and post_w, q v r2
    // and c y up to factors of the row, is one sum
    const float m = a.scale * a.keep_scale, mg = m * gate * r2;
    float cy[1] = {0.f};
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * NT;
      float y[EPC], w[EPC];
      widen<Tr>(yc[i], y);
#pragma unroll
      for (int j = 0; j < EPC; ++j) w[j] = 1.f;
      if (a.post_w != nullptr) widen<Tr>(pwc[i], w);
      if (a.threshold != 0) {  // what is dropped takes no part, whatever it holds
        const Kept<Tr> keep(t, a.d, c, seed, step, a.threshold);
#pragma unroll
        for (int j = 0; j < EPC; ++j) {
          D[i][j] = keep(j) ? D[i][j] : 0.f;
          y[j] = keep(j) ? y[j] : 0.f;
        }
      }
      if (a.gate_full) {
        float g[EPC], dg[EPC];
        widen<Tr>(chunk(at(a.gate), c, chunks), g);
#pragma unroll
        for (int j = 0; j < EPC; ++j) {
          float sl;
          const float sg = sigmoid(g[j], &sl);
          dg[j] = sl * (m * D[i][j]) * (y[j] * r2 * w[j]);
          D[i][j] *= sg;
        }
        if (a.dgate != nullptr) put(to(a.dgate), c, chunks, round_to<Tr>(dg));
      }
#pragma unroll
      for (int j = 0; j < EPC; ++j) {
        const float p = D[i][j] * y[j];
        gp[i][j] = fmaf(mg, p, gp[i][j]);
        cy[0] = fmaf(p, w[j], cy[0]);
        D[i][j] *= w[j];
      }
    }
    if (a.post_w != nullptr || (a.gate != nullptr && !a.gate_full)) row_sum<NT>(cy, part2[place]);
    if (a.gate != nullptr && !a.gate_full && a.dgate != nullptr && tid == 0) {
      const float g = slope * r2 * m * cy[0];
      if constexpr (sizeof(Elt) == 2)
        static_cast<uint16_t*>(a.dgate)[t] = (uint16_t)f32_to_bf16(g);
      else
        static_cast<float*>(a.dgate)[t] = g;
    }
    const float k2 = -(cy[0] * inv_d * r2) * r2;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * NT;
      if (a.post_w != nullptr) {
        float y[EPC];
        widen<Tr>(yc[i], y);
#pragma unroll
        for (int j = 0; j < EPC; ++j) D[i][j] = fmaf(y[j], k2, D[i][j]);
      }
#pragma unroll
      for (int j = 0; j < EPC; ++j) D[i][j] *= mg;
      put(to(a.dy), c, chunks, round_to<Tr>(D[i]));
    }
    if (kAhead) {
#pragma unroll
      for (int i = 0; i < V; ++i) yc[i] = yn[i];
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
      for (int c = threadIdx.x; c < a.d; c += B) {
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
// flight; ranges joined in order.  17 MB of sums in 5 us: one round of loads, and its latency.
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
// such blocks of a thread, loaded first.  out may be x.  Bound by memory: 8192 x 14336 bf16 in
// 81 us, 5.8 TB/s.
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

// Threads of a launch of the forward kernel at most: sixteen wavefronts for each compute
// unit (4096 rows of 4096 with everything 27.5 us, with 32 wavefronts 30.6, with as many as
// rows need 29.6).
constexpr int kForwardThreads = 256 * 1024;

// Threads of a row and elements of each: the first whose product holds the row.
#define MOE_ROW_SHAPES(M) M(64, 8) M(128, 8) M(256, 8) M(512, 8) M(1024, 8) M(1024, 16)

template <class Tr>
hipError_t residual_t(const ResidualArgs& a, hipStream_t stream) {
#define MOE_TRY(NT, N)                                                                                          \
  if (a.d <= NT * N) {                                                                                          \
    constexpr int B = block_of(NT);                                                                             \
    hipLaunchKernelGGL((residual_kernel<Tr, NT, N / Tr::EPC>), dim3(std::min((a.T - 1) / (B / NT) + 1, kForwardThreads / B)), \
                       dim3(B), 0, stream, a);                                                                  \
    return hipGetLastError();                                                                                   \
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
#define MOE_TRY(NT, N)                                                                                          \
  if (!launched && a.d <= NT * N) {                                                                             \
    constexpr int B = block_of(NT);                                                                             \
    launched = true;                                                                                            \
    hipLaunchKernelGGL((residual_backward_kernel<Tr, NT, N / Tr::EPC>), dim3(groups), dim3(B),                  \
                       B > NT ? (size_t)(B / NT) * a.d * 4 : 0, stream, a);                                     \
    e = hipGetLastError();                                                                                      \
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
  const int per = d <= 512 ? 4 : 1;  // rows side by side in a workgroup
  int threads = 64;                  // of a workgroup, as MOE_ROW_SHAPES has them
  while (threads < 1024 && d > threads * 8) threads *= 2;
  threads = block_of(threads);
  // sixteen wavefronts for each compute unit, all that their registers allow (fp32 rows of 2112
  // to 4096 take 149 of them, so that eight are resident and the workgroups come in two rounds):
  // half or twice as many take 58 and 64 us for 16384 rows of 1024 bf16 against 54, and 62 and 65
  // against 53 for 4096 of 4096
  return std::min((T - 1) / per + 1, 256 * 1024 / threads);
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
