// Row kernels of the backward pass: the gradients of the weighted combine and
// of the sorted dispatch, the router's gradient apart from its matrix product,
// and the values of the 8-bit projections.  All of them move whole rows once and
// are bound by that; every sum is fp32 in a fixed order.
#include <algorithm>

#include "device_common.hpp"
#include "launch.hpp"

namespace moe {
namespace {

constexpr int kSlots = 4;  // slots of a token worked at a time

// Gradient of out_t = sum_j w_j y_j for slots 4 blockIdx.y .. + 3 of token
// blockIdx.x: dy_j = w_j dout_t (one rounding) and dw_j = <dout_t, y_j>.  dout_t
// is read once for the four slots, and not at all if none of them has a row.  dw:
// thread partials over its chunks, then lanes, then wavefronts in order.  Bound by
// memory: 4096 tokens of 2048 bf16 with 6 experts each take 37 us (5.9 TB/s).
template <class Tr>
__global__ __launch_bounds__(256) void combine_backward_kernel(const char* __restrict__ dout,
                                                               const char* __restrict__ y,
                                                               const float* __restrict__ topk_w,
                                                               const int32_t* __restrict__ row_of, int k, int d,
                                                               char* __restrict__ dy, float* __restrict__ dw) {
  using Elt = typename Tr::T;
  constexpr int EPC = Tr::EPC;
  __shared__ float part[4][kSlots];
  const size_t row_bytes = (size_t)d * sizeof(Elt);
  const int nchunk = d / EPC;
  const size_t t = blockIdx.x;
  const int j0 = blockIdx.y * kSlots;
  size_t at[kSlots];
  float w[kSlots], acc[kSlots];
  bool ok[kSlots], any = false;
#pragma unroll
  for (int u = 0; u < kSlots; ++u) {
    const int row = j0 + u < k ? row_of[t * k + j0 + u] : -1;
    ok[u] = row >= 0;
    w[u] = ok[u] ? topk_w[t * k + j0 + u] : 0.f;
    at[u] = ok[u] ? (size_t)row * row_bytes : 0;
    acc[u] = 0.f;
    any = any || ok[u];
  }
  const char* dt = dout + t * row_bytes;
  for (int c = threadIdx.x; any && c < nchunk; c += blockDim.x) {
    const size_t o = (size_t)c * 16;
    float g[EPC];
    const uint4 gc = *reinterpret_cast<const uint4*>(dt + o);
    uint4 yc[kSlots];
#pragma unroll
    for (int u = 0; u < kSlots; ++u)
      yc[u] = ok[u] ? *reinterpret_cast<const uint4*>(y + at[u] + o) : make_uint4(0, 0, 0, 0);
    widen<Tr>(gc, g);
#pragma unroll
    for (int u = 0; u < kSlots; ++u) {
      if (!ok[u]) continue;
      float v[EPC];
      widen<Tr>(yc[u], v);
#pragma unroll
      for (int i = 0; i < EPC; ++i) acc[u] = fmaf(g[i], v[i], acc[u]);
#pragma unroll
      for (int i = 0; i < EPC; ++i) v[i] = w[u] * g[i];
      *reinterpret_cast<uint4*>(dy + at[u] + o) = narrow<Tr>(v);
    }
  }
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
#pragma unroll
  for (int u = 0; u < kSlots; ++u) {
    acc[u] = wave_sum(acc[u]);
    if (lane == 0) part[wave][u] = acc[u];
  }
  __syncthreads();
  if (threadIdx.x < kSlots && j0 + (int)threadIdx.x < k) {
    float s = part[0][threadIdx.x];
    for (int i = 1; i < waves; ++i) s += part[i][threadIdx.x];
    dw[t * k + j0 + threadIdx.x] = s;
  }
}

// dw_router = the token ranges' partial sums in order, one rounding
// (workgroups 0 .. sum_blocks - 1); dbias_e = expert e's sums over the K steps (the
// E workgroups behind them: threads, lanes, then wavefronts in order).
template <class Tr>
__device__ __forceinline__ void route_finish(const RouteFinish& p, int E, int d) {
  using Elt = typename Tr::T;
  if ((int)blockIdx.x < p.sum_blocks) {
    const int64_t Ed = (int64_t)E * d, i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= Ed) return;
    float4 s = *reinterpret_cast<const float4*>(p.part + i);
    for (int r = 1; r < p.ranges; ++r) {
      const float4 v = *reinterpret_cast<const float4*>(p.part + r * Ed + i);
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
    store4<Tr>(static_cast<char*>(p.dw_router) + i * sizeof(Elt), s.x, s.y, s.z, s.w);
    return;
  }
  __shared__ float wave_part[4];
  const int e = blockIdx.x - p.sum_blocks;
  float s = 0.f;
  for (int i = threadIdx.x; i < p.steps; i += 256) s += p.sums[(size_t)i * E + e];
  s = wave_sum(s);
  if ((threadIdx.x & 63) == 0) wave_part[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) p.dbias[e] = (wave_part[0] + wave_part[1]) + (wave_part[2] + wave_part[3]);
}

// dx_t = sum_j dx_perm[row_j] + sum_j dz_j w_router[id_j]: fp32, the rows in
// slot order and then the router's part, one rounding.  Either sum may be
// absent (row_of or dz null).  dx_perm has In's type: fp32 inside moe_backward, whose
// dx is then rounded once.  The router's rows stay in L2.  `lanes` threads
// (64 or 256) work on a token.  The first fin.blocks workgroups finish the
// router's other gradients instead (nothing here needs them, and they would be
// a launch of their own).  Bound by memory: the sum of 8 rows of 3584 bf16 for
// 4096 tokens takes 39 us (6.8 TB/s); the router's part for 4096 tokens of 2048
// with 64 experts, 6 chosen, 14 us with the finish (6 us as its own launch).
template <class Tr, class In>
__global__ __launch_bounds__(256) void token_backward_kernel(const char* __restrict__ dx_perm,
                                                             const int32_t* __restrict__ row_of,
                                                             const float* __restrict__ dz,
                                                             const int32_t* __restrict__ ids,
                                                             const char* __restrict__ w_router, int T, int k, int d,
                                                             int E, int lanes, char* __restrict__ dx,
                                                             RouteFinish fin) {
  using Elt = typename Tr::T;
  if ((int)blockIdx.x < fin.blocks) {
    route_finish<Tr>(fin, E, d);
    return;
  }
  constexpr int EPC = Tr::EPC, PER = EPC / In::EPC;  // 16-byte loads of dx_perm for 16 bytes of dx
  const size_t row_bytes = (size_t)d * sizeof(Elt);
  const int nchunk = d / EPC;
  const int per = 256 / lanes;
  const size_t t = (size_t)((int)blockIdx.x - fin.blocks) * per + threadIdx.x / lanes;
  if (t >= (size_t)T) return;
  for (int c = threadIdx.x & (lanes - 1); c < nchunk; c += lanes) {
    const size_t o = (size_t)c * 16;
    float acc[EPC];
#pragma unroll
    for (int i = 0; i < EPC; ++i) acc[i] = 0.f;
    if (row_of != nullptr) {
      for (int j0 = 0; j0 < k; j0 += kSlots) {
        uint4 ch[kSlots][PER];
        bool ok[kSlots];
#pragma unroll
        for (int u = 0; u < kSlots; ++u) {
          const int row = j0 + u < k ? row_of[t * k + j0 + u] : -1;
          ok[u] = row >= 0;
#pragma unroll
          for (int i = 0; i < PER; ++i)
            ch[u][i] = ok[u] ? *reinterpret_cast<const uint4*>(dx_perm + (size_t)row * row_bytes * PER + o * PER + i * 16)
                             : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < kSlots; ++u) {
          if (!ok[u]) continue;
          float v[EPC];
#pragma unroll
          for (int i = 0; i < PER; ++i) widen<In>(ch[u][i], v + i * In::EPC);
#pragma unroll
          for (int i = 0; i < EPC; ++i) acc[i] += v[i];
        }
      }
    }
    if (dz != nullptr) {
      for (int j0 = 0; j0 < k; j0 += kSlots) {
        uint4 ch[kSlots];
        float z[kSlots];
        bool ok[kSlots];
#pragma unroll
        for (int u = 0; u < kSlots; ++u) {
          const int id = j0 + u < k ? ids[t * k + j0 + u] : -1;
          ok[u] = id >= 0 && id < E;
          z[u] = ok[u] ? dz[t * k + j0 + u] : 0.f;
          ch[u] = ok[u] ? *reinterpret_cast<const uint4*>(w_router + (size_t)id * row_bytes + o)
                        : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < kSlots; ++u) {
          if (!ok[u]) continue;
          float v[EPC];
          widen<Tr>(ch[u], v);
#pragma unroll
          for (int i = 0; i < EPC; ++i) acc[i] = fmaf(z[u], v[i], acc[i]);
        }
      }
    }
    *reinterpret_cast<uint4*>(dx + t * row_bytes + o) = narrow<Tr>(acc);
  }
}

// The softmax's gradient over the chosen logits, dz_j = w_j (dw_j - sum_i w_i
// dw_i), and its dense form for the router's weight gradient: workgroup b
// holds the KS tokens of one K step, one thread each, and writes [E][KS]
// (bf16: the rounded value, and the rounded rest) and each expert's sum over
// the step, the first half of dbias.  Slots without an expert are left out of
// the sum: their weight and its gradient may hold anything, and zero times a NaN
// would reach the token's other slots.  Bound by latency: 7 us for 4096 tokens and
// 64 experts.
template <class Tr>
__global__ __launch_bounds__(256) void route_dz_kernel(const int32_t* __restrict__ ids, const float* __restrict__ w,
                                                       const float* __restrict__ dw, int T, int k, int E,
                                                       float* __restrict__ dz, typename Tr::T* __restrict__ hi,
                                                       typename Tr::T* __restrict__ lo, float* __restrict__ sums,
                                                       unsigned* __restrict__ taken) {
  constexpr int KS = 64 / sizeof(typename Tr::T);
  extern __shared__ float dense[];  // [E][KS]
  for (int i = threadIdx.x; i < E * KS; i += 256) dense[i] = 0.f;
  __syncthreads();
  const int64_t t = (int64_t)blockIdx.x * KS + threadIdx.x;
  bool any = false;
  if (threadIdx.x < KS && t < T) {
    const float* wt = w + t * k;
    const float* dt = dw + t * k;
    const int* it = ids + t * k;
    const auto live = [&](int j) { return it[j] >= 0 && it[j] < E; };
    float s = 0.f;
    for (int j = 0; j < k; ++j)
      if (live(j)) s = fmaf(wt[j], dt[j], s);
    for (int j = 0; j < k; ++j) {
      const float z = live(j) ? wt[j] * (dt[j] - s) : 0.f;
      dz[t * k + j] = z;
      if (live(j)) dense[it[j] * KS + threadIdx.x] += z, any = true;
    }
  }
  const uint64_t bits = __ballot(any);
  if (threadIdx.x == 0) taken[blockIdx.x] = (unsigned)bits;
  __syncthreads();
  const size_t base = (size_t)blockIdx.x * E * KS;
  for (int i = threadIdx.x; i < E * KS; i += 256) {
    const float v = dense[i];
    if constexpr (sizeof(typename Tr::T) == 2) {
      const uint32_t h = f32_to_bf16(v);
      hi[base + i] = (uint16_t)h;
      lo[base + i] = (uint16_t)f32_to_bf16(v - bf16_to_f32(h));
    } else {
      hi[base + i] = v;
    }
  }
  for (int e = threadIdx.x; e < E; e += 256) {
    float v = 0.f;
    for (int i = 0; i < KS; ++i) v += dense[e * KS + (i + e) % KS];  // (e + i: rows of equal length share banks)
    sums[(size_t)blockIdx.x * E + e] = v;
  }
}

// Values of one projection's codes (blockIdx.y: gate, up): a thread turns one
// block of 16 into bf16, which holds every such value exactly.  Bound by memory:
// 18 us for 1024 rows of 14336 (5 TB/s).
__global__ __launch_bounds__(256) void saved8_unpack_kernel(const int8_t* __restrict__ g8,
                                                            const int8_t* __restrict__ u8,
                                                            const uint8_t* __restrict__ gx,
                                                            const uint8_t* __restrict__ ux,
                                                            const int32_t* __restrict__ token_of, int64_t blocks,
                                                            int per_row, uint16_t* __restrict__ gate,
                                                            uint16_t* __restrict__ up) {
  const int8_t* codes = blockIdx.y ? u8 : g8;
  const uint8_t* exps = blockIdx.y ? ux : gx;
  uint16_t* out = blockIdx.y ? up : gate;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < blocks; i += (int64_t)gridDim.x * 256) {
    if (token_of[i / per_row] < 0) continue;
    const uint4 c = *reinterpret_cast<const uint4*>(codes + i * 16);
    const float s = exp_scale(exps[i]);
    const unsigned w[4] = {c.x, c.y, c.z, c.w};
    float v[16];
#pragma unroll
    for (int q = 0; q < 16; ++q) v[q] = code_of(w[q >> 2], q & 3) * s;
    *reinterpret_cast<uint4*>(out + i * 16) = narrow<TBF16>(v);
    *reinterpret_cast<uint4*>(out + i * 16 + 8) = narrow<TBF16>(v + 8);
  }
}

int row_threads(int dtype, int d) { return d / (dtype == 1 ? 8 : 4) <= 64 ? 64 : 256; }

}  // namespace

hipError_t launch_combine_backward(int dtype, const void* dout, const void* y, const float* topk_w,
                                   const int32_t* row_of, int T, int k, int d, void* dy, float* dw,
                                   hipStream_t stream) {
  const dim3 grid(T, (k + kSlots - 1) / kSlots), block(row_threads(dtype, d));
  if (dtype == 1)
    hipLaunchKernelGGL(combine_backward_kernel<TBF16>, grid, block, 0, stream, static_cast<const char*>(dout),
                       static_cast<const char*>(y), topk_w, row_of, k, d, static_cast<char*>(dy), dw);
  else
    hipLaunchKernelGGL(combine_backward_kernel<TF32>, grid, block, 0, stream, static_cast<const char*>(dout),
                       static_cast<const char*>(y), topk_w, row_of, k, d, static_cast<char*>(dy), dw);
  return hipGetLastError();
}

hipError_t launch_token_backward(int dtype, const void* dx_perm, bool f32, const int32_t* row_of, const float* dz,
                                 const int32_t* ids, const void* w_router, int T, int k, int d, int E, void* dx,
                                 RouteFinish fin, hipStream_t stream) {
  const int lanes = row_threads(dtype, d), per = 256 / lanes;
  fin.sum_blocks = fin.part != nullptr ? (int)(((int64_t)E * d / 4 + 255) / 256) : 0;
  fin.blocks = fin.sum_blocks + (fin.dbias != nullptr ? E : 0);
  const dim3 grid((unsigned)fin.blocks + ((unsigned)T + per - 1) / per), block(256);
  auto launch = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, block, 0, stream, static_cast<const char*>(dx_perm), row_of, dz, ids,
                       static_cast<const char*>(w_router), T, k, d, E, lanes, static_cast<char*>(dx), fin);
  };
  if (dtype != 1)
    launch(token_backward_kernel<TF32, TF32>);
  else if (f32)
    launch(token_backward_kernel<TBF16, TF32>);
  else
    launch(token_backward_kernel<TBF16, TBF16>);
  return hipGetLastError();
}

hipError_t launch_route_dz(int dtype, const int32_t* ids, const float* w, const float* dw, int T, int k, int E,
                           float* dz, void* dense_hi, void* dense_lo, float* sums, unsigned* taken,
                           hipStream_t stream) {
  const int KS = dtype == 1 ? 32 : 16;
  const dim3 grid((unsigned)(((int64_t)T + KS - 1) / KS)), block(256);
  const size_t lds = (size_t)E * KS * sizeof(float);
  if (dtype == 1)
    hipLaunchKernelGGL(route_dz_kernel<TBF16>, grid, block, lds, stream, ids, w, dw, T, k, E, dz,
                       static_cast<uint16_t*>(dense_hi), static_cast<uint16_t*>(dense_lo), sums, taken);
  else
    hipLaunchKernelGGL(route_dz_kernel<TF32>, grid, block, lds, stream, ids, w, dw, T, k, E, dz,
                       static_cast<float*>(dense_hi), static_cast<float*>(nullptr), sums, taken);
  return hipGetLastError();
}

hipError_t launch_saved8_unpack(const int8_t* g8, const int8_t* u8, const uint8_t* gx, const uint8_t* ux,
                                const int32_t* token_of, int64_t rows, int F, void* gate, void* up,
                                hipStream_t stream) {
  const int64_t blocks = rows * (F / 16);
  hipLaunchKernelGGL(saved8_unpack_kernel, dim3((unsigned)std::min<int64_t>((blocks + 255) / 256, 1 << 20), 2), dim3(256), 0, stream, g8, u8,
                     gx, ux, token_of, blocks, F / 16, static_cast<uint16_t*>(gate), static_cast<uint16_t*>(up));
  return hipGetLastError();
}

}  // namespace moe
