// Grouped GEMMs of the experts' backward pass on the gfx950 matrix cores
// (implementation; instantiated per element type in gemm_grad_<type>.hip).
//
// For the rows r of expert e (t = token of row r, w_r its routing weight; g, u
// the saved projections, s = 1 / (1 + exp(-g)), h = g s u):
//   D = dout_t W_down               (gradient of h before the routing weight)
//   dw_r = <D, h>                   (= <dout_t, y_r>: no y is kept)
//   du = w_r D g s,  dg = w_r D u s (1 + g (1 - s))
//   dx_perm_r = dg W_gate + du W_up
//   dW_down = sum_r dout_t^T (w_r h),  dW_gate = sum_r dg^T x_t,  dW_up = sum_r du^T x_t
//
// The data gradients contract over the rows of a weight matrix, the weight
// gradients over the rows of the activations, so at least one operand of
// every product has its K index on the strided axis of memory.  Such an
// operand is staged in LDS as it lies in memory ([K][columns]) and turned on
// the way to the registers: bf16 by the transposing LDS read (in each group
// of 16 lanes, lane i receives column i of a 4 x 16 block), fp32 by reading
// one element per K row.
//
// out[m][n] = sum_k Mop[m][k] Nop[k][n]; a workgroup owns a BM x BN tile,
// WM x WN wavefronts of TM x TN each.  The N operand always has K on the
// strided axis; the M operand has it contiguous (activation rows of the data
// gradients) or strided (MKS: the weight gradients).  N is the MFMA "A"
// operand, so a lane ends with 4 consecutive n of one m, as the outputs lie
// in memory.
//
// A K step is 64 bytes of a K-contiguous row (32 bf16 or 16 fp32), so each
// operand takes 64 bytes of LDS per tile row or column whatever its
// orientation.  The steps go through a ring of S LDS stages written by
// LDS-direct buffer loads S - 1 steps ahead.  Reads past a descriptor's bound
// return zero, which pads rows past an expert's last one, columns past the
// matrix and steps past the last.
#pragma once

#include <type_traits>

#include "device_common.hpp"
#include "launch.hpp"

namespace moe {
namespace grad {

template <int N, int I = 0, class F>
__device__ __forceinline__ void static_for(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    static_for<N, I + 1>(f);
  }
}

typedef short s16x4_t __attribute__((ext_vector_type(4)));

// Transposing LDS read of 4 x 16 bf16 per 16 lanes: the lanes' addresses name
// four rows of 16 elements (8 bytes each), lane i receives element i of the rows.
__device__ __forceinline__ uint2 read_tr16(const char* p) {
#ifdef __HIP_DEVICE_COMPILE__  // the host pass does not know the builtin
  return __builtin_bit_cast(
      uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4_t*)(p)));
#else
  return uint2{(unsigned)*p, 0};
#endif
}

constexpr int kOutside = 0x7ff00000;  // a lane offset past every descriptor's bound

template <int n>
__device__ __forceinline__ void wait_vm() {
  static_assert(n >= 0 && n < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((n & 15) | ((n >> 4) << 14) | (7 << 4) | (15 << 8));
}
__device__ __forceinline__ void wait_lds() { __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4) | (0 << 8)); }

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const char* base, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), (short)0, bytes, 0x00020000);
}

// Where the operands of one K step lie: base addresses and descriptor bounds.
struct Step {
  const char* m;
  const char* n;
  int mbytes, nbytes;
};

template <class Tr, int BM_, int BN_, int WM_, int WN_, bool MKS, int S_, bool PP>
struct Tile {
  using Elt = typename Tr::T;
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, S = S_;
  static constexpr int EB = sizeof(Elt);
  static constexpr int KS = 64 / EB;  // K elements per step
  static constexpr int NW = WM * WN, NTH = 64 * NW;
  static constexpr int TM = BM / WM, TN = BN / WN, MI = TM / 16, NI = TN / 16;
  static constexpr int MBYTES = 64 * BM, STAGE = 64 * (BM + BN);
  // 1 KB LDS-direct loads per stage and operand, and per wavefront (the last
  // ones repeat an operand's final load, so every wavefront issues NL)
  static constexpr int QM = BM / 16, QN = BN / 16;
  static constexpr int LM = (QM + NW - 1) / NW, LN = (QN + NW - 1) / NW, NL = LM + LN;
  static_assert(TM % 16 == 0 && TN % 16 == 0, "wavefront tile");
  static_assert(BN * EB % 256 == 0 && (!MKS || BM * EB % 256 == 0), "K-strided operands are swizzled within 256 bytes");
  static_assert(S == 4 && (S - 2) * NL < 64, "ring");

  // LDS swizzle.  A K-contiguous row is 64 bytes: chunk c (16 bytes) of row r
  // sits at c ^ (r / 4 & 3), so the 16 rows of one operand read spread over all
  // banks.  A K-strided row k holds BM or BN columns (a multiple of 256 bytes):
  // its chunks are moved in pairs (bf16: a transposing read takes 32 bytes of
  // 4 rows per 16 lanes; the 8 rows of 32 lanes get 8 different pairs) or in
  // fours (fp32: 64 bytes of one row per 16 lanes).
  __device__ __forceinline__ static int swz_c(int r) { return (r >> 2) & 3; }
  __device__ __forceinline__ static int swz_k(int k) {
    return EB == 2 ? (((k & 3) | ((k >> 1) & 4)) << 1) : ((k >> 2) & 3) << 2;
  }

  // Byte offset inside the operand's step and LDS offset of this lane's slot
  // in load q of a K-strided operand of `width` columns starting at column
  // col0 of rows of `cols` elements (ld bytes each).  blocked16: the rows are in
  // groups of 16, each stored as 1024-byte blocks of 64 bytes from every row.
  template <int WIDTH>
  __device__ __forceinline__ static int strided_offset(int q, int lane, int col0, int cols, int ld, int blocked16) {
    constexpr int CPR = WIDTH * EB / 16;  // chunks per K row
    const int pos = q * 64 + lane;
    const int k = pos / CPR;
    const int c = (pos - k * CPR) ^ swz_k(k);
    const int col = col0 + c * (16 / EB);
    if (col >= cols) return kOutside;
    const int byte = col * EB;
    return blocked16 ? (k >> 4) * 16 * ld + (byte >> 6) * 1024 + (k & 15) * 64 + (byte & 63) : k * ld + byte;
  }

  // Offset of load q of a K-contiguous operand: 16 rows of 64 bytes.
  __device__ __forceinline__ static int rows_offset(int q, int lane, int ld) {
    const int r = q * 16 + (lane >> 2);
    return r * ld + (((lane & 3) ^ swz_c(r)) << 4);
  }

  struct Ctx {
    int moff[LM], noff[LN];  // lane offsets of the loads
  };

  __device__ __forceinline__ static int mq(int wave, int i) { return min(wave + i * NW, QM - 1); }
  __device__ __forceinline__ static int nq(int wave, int i) { return min(wave + i * NW, QN - 1); }

  __device__ __forceinline__ static void load(const Ctx& c, const Step& s, char* st, int wave) {
#ifdef __HIP_DEVICE_COMPILE__  // the host pass cannot pass descriptors by value
    const __amdgpu_buffer_rsrc_t m = rsrc(s.m, s.mbytes), n = rsrc(s.n, s.nbytes);
#pragma unroll
    for (int i = 0; i < LM; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          m, (__attribute__((address_space(3))) void*)(st + mq(wave, i) * 1024), 16, c.moff[i], 0, 0, 0);
#pragma unroll
    for (int i = 0; i < LN; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          n, (__attribute__((address_space(3))) void*)(st + MBYTES + nq(wave, i) * 1024), 16, c.noff[i], 0, 0, 0);
#endif
  }

  // Operand of the 16 columns (or rows) starting at sub * 16 of the
  // wavefront's part.  Lane group g = lane / 16 holds K elements 8g..8g+7 (bf16)
  // or 4g..4g+3 (fp32), whatever the orientation.  `lane0`: lane part of the LDS
  // address, from frag_lane.
  template <bool STRIDED, int WIDTH>
  __device__ __forceinline__ static int frag_lane(int lane, int first) {
    const int g = lane >> 4, i = lane & 15;
    if constexpr (!STRIDED) {
      const int r = first + i;
      return r * 64 + ((g ^ swz_c(r)) << 4);
    } else if constexpr (EB == 2) {
      const int k = 8 * g + (i >> 2);
      const int byte = first * 2 + (i & 3) * 8;
      return k * WIDTH * 2 + ((((byte >> 4) ^ swz_k(k)) << 4) | (byte & 15));
    } else {
      const int k = 4 * g;
      const int byte = (first + i) * 4;
      return k * WIDTH * 4 + ((((byte >> 4) ^ swz_k(k)) << 4) | (byte & 15));
    }
  }
  template <bool STRIDED, int WIDTH>
  __device__ __forceinline__ static uint4 frag(const char* st, int lane0, int sub) {
    if constexpr (!STRIDED) {
      return *reinterpret_cast<const uint4*>(st + lane0 + sub * 1024);
    } else if constexpr (EB == 2) {
      // 16 columns are 32 bytes, one pair of chunks: column blocks differ by an
      // exclusive or in the address (the swizzle stays within 256 bytes)
      const char* p = st + (lane0 ^ ((sub & 7) << 5)) + (sub >> 3) * 256;
      const uint2 a = read_tr16(p), b = read_tr16(p + 4 * WIDTH * 2);
      return uint4{a.x, a.y, b.x, b.y};
    } else {
      const char* p = st + (lane0 ^ ((sub & 3) << 6)) + (sub >> 2) * 256;
      const unsigned* q = reinterpret_cast<const unsigned*>(p);
      return uint4{q[0], q[WIDTH], q[2 * WIDTH], q[3 * WIDTH]};
    }
  }

  // Step j (u = j mod S): this wavefront's loads of the step have landed (those
  // of the S - 2 after it may be in flight); after the barrier everyone's have,
  // and everyone is done with the stage of step j - 1, which takes step
  // j + S - 1.
  template <int u, class Src>
  __device__ __forceinline__ static void step(const Ctx& c, char* const (&st)[S], int j, Src& src, int wave, int ml,
                                              int nl, f32x4_t (&acc)[MI][NI]) {
    wait_vm<(S - 2) * NL>();
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
    load(c, src(j + S - 1), st[(u + S - 1) % S], wave);
    __builtin_amdgcn_sched_barrier(0);
    uint4 nf[NI], mf[MI];
#pragma unroll
    for (int ni = 0; ni < NI; ++ni) nf[ni] = frag<true, BN>(st[u], nl, ni);
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) mf[mi] = frag<MKS, BM>(st[u], ml, mi);
#pragma unroll
    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
      for (int ni = 0; ni < NI; ++ni) acc[mi][ni] = mma16<Tr>(nf[ni], mf[mi], acc[mi][ni]);
    __builtin_amdgcn_sched_barrier(0);
  }

  // acc[mi][ni] over `steps` K steps; src(j) gives step j (empty descriptors
  // past the last).
  template <class Src>
  __device__ __forceinline__ static void run(const Ctx& c, char* const (&st)[S], int steps, Src& src,
                                             f32x4_t (&acc)[MI][NI]) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int ml = frag_lane<MKS, BM>(lane, (wave / WN) * TM);
    const int nl = MBYTES + frag_lane<true, BN>(lane, (wave % WN) * TN);
#pragma unroll
    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
      for (int ni = 0; ni < NI; ++ni) acc[mi][ni] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int u = 0; u < S - 1; ++u) load(c, src(u), st[u], wave);
    int j = 0;
    for (; j + S <= steps; j += S)
      static_for<S>([&](auto uc) { step<decltype(uc)::value>(c, st, j + decltype(uc)::value, src, wave, ml, nl, acc); });
    static_for<S - 1>([&](auto uc) {
      if (j + decltype(uc)::value < steps)
        step<decltype(uc)::value>(c, st, j + decltype(uc)::value, src, wave, ml, nl, acc);
    });
    // the loads of steps past the last still write LDS
    wait_vm<0>();
    __syncthreads();
  }
};

// ---- data gradients ---------------------------------------------------------

// Rows of expert i: n0 from row r0 on and, behind the capacity, n1 from r1 on.
struct ExpertRows {
  int r0, n0, r1, n1;
};
__device__ __forceinline__ ExpertRows expert_rows(const GradRows& p, int i) {
  const int n = p.counts[i];
  if (p.C == 0) return ExpertRows{p.offsets[i], n, 0, 0};
  const int n0 = min(n, p.C);
  return ExpertRows{i * p.C, n0, p.E * p.C + p.spill_offsets[i], n - n0};
}

// Which expert holds tile L of all experts' row tiles of BM rows: (expert,
// index of the tile inside it), or expert -1 past the last.  Every lane of the
// wavefront takes part; the result is uniform.
template <int BM>
__device__ __forceinline__ int2 find_tile(const GradRows& p, int units_per_tile, int L) {
  const int lane = threadIdx.x & 63;
  int e = 0, before = 0, carry = 0;
  for (int b = 0; b < p.E; b += 64) {
    const int i = b + lane;
    int t = 0;
    if (i < p.E) {
      const ExpertRows r = expert_rows(p, i);
      t = (r.n0 + BM - 1) / BM + (r.n1 + BM - 1) / BM;
    }
    int inc = t;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(inc, o);
      if (lane >= o) inc += v;
    }
    const bool done = i < p.E && (long long)(carry + inc) * units_per_tile <= (long long)L;
    e += __popcll(__ballot(done));
    int bt = done ? t : 0;
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) bt += __shfl_xor(bt, o);
    before += bt;
    carry += __shfl(inc, 63);
  }
  e = __builtin_amdgcn_readfirstlane(e);
  before = __builtin_amdgcn_readfirstlane(before);
  return int2{e < p.E ? e : -1, before};
}

template <int BM>
__device__ __forceinline__ int count_tiles(const GradRows& p) {
  const int lane = threadIdx.x & 63;
  int total = 0;
  for (int b = 0; b < p.E; b += 64) {
    const int i = b + lane;
    int t = 0;
    if (i < p.E) {
      const ExpertRows r = expert_rows(p, i);
      t = (r.n0 + BM - 1) / BM + (r.n1 + BM - 1) / BM;
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) t += __shfl_xor(t, o);
    total += t;
  }
  return __builtin_amdgcn_readfirstlane(total);
}

// out tile = act rows x weights (DH: with the SwiGLU's gradient in the epilogue).
template <class Tr, class T, bool DH>
__global__ __launch_bounds__(T::NTH) void dgrad_kernel(DgradArgs p) {
  constexpr int EB = T::EB;
  __shared__ __attribute__((aligned(16))) char s0[T::STAGE];
  __shared__ __attribute__((aligned(16))) char s1[T::STAGE];
  __shared__ __attribute__((aligned(16))) char s2[T::STAGE];
  __shared__ __attribute__((aligned(16))) char s3[T::STAGE];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int NT = (p.N + T::BN - 1) / T::BN;
  // each XCD (workgroup id modulo 8) walks a contiguous range of the units:
  // expert, then column tile, then row tile, so the row tiles that read the
  // same weights follow each other in one L2
  const int total = count_tiles<T::BM>(p.rows) * NT;
  const int J = (total + 7) >> 3;
  const int jj = blockIdx.x >> 3;
  const int L = (blockIdx.x & 7) * J + jj;
  if (jj >= J || L >= total) return;
  const int2 at = find_tile<T::BM>(p.rows, NT, L);
  if (at.x < 0) return;
  const int e = at.x;
  const ExpertRows er = expert_rows(p.rows, e);
  const int t0 = (er.n0 + T::BM - 1) / T::BM, t1 = (er.n1 + T::BM - 1) / T::BM;
  const int local = L - at.y * NT;
  const int nt = local / (t0 + t1);
  const int ti = local - nt * (t0 + t1);
  const int first = ti < t0 ? ti * T::BM : (ti - t0) * T::BM;
  const int row0 = (ti < t0 ? er.r0 : er.r1) + first;
  const int rows = min(T::BM, (ti < t0 ? er.n0 : er.n1) - first);
  const int nbase = nt * T::BN;

  const int ldm = p.K * EB, ldn = p.N * EB;
  typename T::Ctx c;
#pragma unroll
  for (int i = 0; i < T::LM; ++i) c.moff[i] = T::rows_offset(T::mq(wave, i), lane, ldm);
#pragma unroll
  for (int i = 0; i < T::LN; ++i)
    c.noff[i] = T::template strided_offset<T::BN>(T::nq(wave, i), lane, nbase, p.N, ldn, p.blocked16);
  const int per = p.K / T::KS, steps = per * (p.a1 != nullptr ? 2 : 1);
  const char* a0 = static_cast<const char*>(p.a0) + (size_t)row0 * ldm;
  const char* a1 = p.a1 != nullptr ? static_cast<const char*>(p.a1) + (size_t)row0 * ldm : nullptr;
  const size_t mat = (size_t)e * p.K * ldn;
  const char* b0 = static_cast<const char*>(p.b0) + mat;
  const char* b1 = p.a1 != nullptr ? static_cast<const char*>(p.b1) + mat : nullptr;
  auto src = [&](int j) {
    Step s;
    const bool second = j >= per;
    const int q = second ? j - per : j;
    const bool in = j < steps;
    s.m = (second && in ? a1 : a0) + (in ? (size_t)q * 64 : 0);
    s.n = (second && in ? b1 : b0) + (in ? (size_t)q * T::KS * ldn : 0);
    s.mbytes = in ? rows * ldm - q * 64 : 0;
    s.nbytes = in ? T::KS * ldn : 0;
    return s;
  };
  f32x4_t acc[T::MI][T::NI];
  char* const stages[T::S] = {s0, s1, s2, s3};
  T::run(c, stages, steps, src, acc);

  const int wm = wave / T::WN, wn = wave % T::WN, g4 = (lane >> 4) * 4, i16 = lane & 15;
#pragma unroll
  for (int mi = 0; mi < T::MI; ++mi) {
    const int m = wm * T::TM + mi * 16 + i16;
    const bool live = m < rows;
    const size_t row = (size_t)row0 + (live ? m : 0);
    if constexpr (!DH) {
      if (live) {
#pragma unroll
        for (int ni = 0; ni < T::NI; ++ni) {
          const int n = nbase + wn * T::TN + ni * 16 + g4;
          if (n < p.N)
            store4<Tr>(static_cast<char*>(p.out) + (row * p.N + n) * EB, acc[mi][ni][0], acc[mi][ni][1],
                       acc[mi][ni][2], acc[mi][ni][3]);
        }
      }
    } else {
      const float wr = p.wrow[row];
      float dot = 0.f;
#pragma unroll
      for (int ni = 0; ni < T::NI; ++ni) {
        const int n = nbase + wn * T::TN + ni * 16 + g4;
        if (live && n < p.N) {
          const size_t o = row * p.N + n;
          const unsigned gc = *reinterpret_cast<const unsigned*>(p.g8 + o);
          const unsigned uc = *reinterpret_cast<const unsigned*>(p.u8 + o);
          const float gs = exp_scale(p.gx[o >> 4]), us = exp_scale(p.ux[o >> 4]);
          float dg[4], du[4], hw[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float D = acc[mi][ni][r];
            const float g = code_of(gc, r) * gs, u = code_of(uc, r) * us;
            const float sg = 1.0f / (1.0f + __expf(-g));
            const float a = g * sg, h = a * u;
            dot = fmaf(D, h, dot);
            const float dh = wr * D;
            du[r] = dh * a;
            dg[r] = dh * (u * sg * fmaf(g, 1.0f - sg, 1.0f));
            hw[r] = wr * h;
          }
          store4<Tr>(static_cast<char*>(p.dg) + o * EB, dg[0], dg[1], dg[2], dg[3]);
          store4<Tr>(static_cast<char*>(p.du) + o * EB, du[0], du[1], du[2], du[3]);
          if (p.hw != nullptr) store4<Tr>(static_cast<char*>(p.hw) + o * EB, hw[0], hw[1], hw[2], hw[3]);
        }
      }
      // the wavefront's columns of <D, h>: the four lanes of a row, then one
      // partial sum per wavefront column, added in order by a later step
      dot += __shfl_xor(dot, 16);
      dot += __shfl_xor(dot, 32);
      if (live && lane < 16) p.dot[row * (size_t)p.dot_ld + nt * T::WN + wn] = dot;
    }
  }
}

// ---- weight gradients ---------------------------------------------------------

// out[e][m][n] = sum over the rows r of expert e of P[r][m] Q[r][n]: up to three
// such products in one launch.  An expert without rows gets zeros.
template <class Tr, class T>
__global__ __launch_bounds__(T::NTH) void wgrad_kernel(WgradArgs p) {
  constexpr int EB = T::EB;
  __shared__ __attribute__((aligned(16))) char s0[T::STAGE];
  __shared__ __attribute__((aligned(16))) char s1[T::STAGE];
  __shared__ __attribute__((aligned(16))) char s2[T::STAGE];
  __shared__ __attribute__((aligned(16))) char s3[T::STAGE];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int J = (p.units + 7) >> 3;
  const int jj = blockIdx.x >> 3;
  int L = (blockIdx.x & 7) * J + jj;
  if (jj >= J || L >= p.units) return;
  const int per_e = p.units / p.rows.E;
  const int e = L / per_e;
  L -= e * per_e;
  int w = 0;
  if (p.n > 1 && L >= p.first[1]) w = 1;
  if (p.n > 2 && L >= p.first[2]) w = 2;
  L -= p.first[w];
  const int M = p.M[w], N = p.N[w];
  const int MT = (M + T::BM - 1) / T::BM, NT = (N + T::BN - 1) / T::BN;
  // groups of 8 row tiles by all column tiles, so the tiles at work at a time
  // form a near-square patch of the output that shares both operands in L2
  const int gsz = 8 * NT;
  const int grp = L / gsz, in = L - grp * gsz;
  const int gm = min(8, MT - grp * 8);
  const int nt = in / gm, mt = grp * 8 + in - nt * gm;
  const int mbase = mt * T::BM, nbase = nt * T::BN;
  const ExpertRows er = expert_rows(p.rows, e);

  const int ldm = M * EB, ldn = N * EB;
  typename T::Ctx c;
#pragma unroll
  for (int i = 0; i < T::LM; ++i)
    c.moff[i] = T::template strided_offset<T::BM>(T::mq(wave, i), lane, mbase, M, ldm, 0);
#pragma unroll
  for (int i = 0; i < T::LN; ++i)
    c.noff[i] = T::template strided_offset<T::BN>(T::nq(wave, i), lane, nbase, N, ldn, 0);
  const int steps0 = (er.n0 + T::KS - 1) / T::KS, steps = steps0 + (er.n1 + T::KS - 1) / T::KS;
  const char* P = static_cast<const char*>(p.P[w]);
  const char* Q = static_cast<const char*>(p.Q[w]);
  auto src = [&](int j) {
    Step s;
    const bool second = j >= steps0;
    const int q = (second ? j - steps0 : j) * T::KS;
    const int left = j < steps ? min(T::KS, (second ? er.n1 : er.n0) - q) : 0;
    const size_t row = left > 0 ? (size_t)((second ? er.r1 : er.r0) + q) : 0;
    s.m = P + row * ldm;
    s.n = Q + row * ldn;
    s.mbytes = left * ldm;
    s.nbytes = left * ldn;
    return s;
  };
  f32x4_t acc[T::MI][T::NI];
  char* const stages[T::S] = {s0, s1, s2, s3};
  T::run(c, stages, steps, src, acc);

  const int wm = wave / T::WN, wn = wave % T::WN, g4 = (lane >> 4) * 4, i16 = lane & 15;
  char* out = static_cast<char*>(p.out[w]) + (size_t)e * M * N * EB;
#pragma unroll
  for (int mi = 0; mi < T::MI; ++mi) {
    const int m = mbase + wm * T::TM + mi * 16 + i16;
    if (m < M) {
#pragma unroll
      for (int ni = 0; ni < T::NI; ++ni) {
        const int n = nbase + wn * T::TN + ni * 16 + g4;
        if (n < N) {
          const size_t o = p.blocked16 ? (size_t)(m >> 4) * 16 * N + (size_t)(n / T::KS) * (16 * T::KS) +
                                             (m & 15) * T::KS + n % T::KS
                                       : (size_t)m * N + n;
          store4<Tr>(out + o * EB, acc[mi][ni][0], acc[mi][ni][1], acc[mi][ni][2], acc[mi][ni][3]);
        }
      }
    }
  }
}

// ---- router weight gradient ---------------------------------------------------

// part[z][e][i] = sum over tokens t of range z of dz[e][t] x[t][i] (fp32 partial
// sums).  dz is dense with zeros where expert e did not take token t, laid out
// by K step: [step][E][64 bytes].  bf16 carries it as two terms (high and low
// part), which keeps 16 bits of its significand.
template <class Tr, class T>
__global__ __launch_bounds__(T::NTH) void route_wgrad_kernel(RouteWgradArgs p) {
  constexpr int EB = T::EB;
  __shared__ __attribute__((aligned(16))) char s0[T::STAGE];
  __shared__ __attribute__((aligned(16))) char s1[T::STAGE];
  __shared__ __attribute__((aligned(16))) char s2[T::STAGE];
  __shared__ __attribute__((aligned(16))) char s3[T::STAGE];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nbase = blockIdx.x * T::BN, mbase = blockIdx.y * T::BM, z = blockIdx.z;
  const int rows = min(T::BM, p.E - mbase);
  const int ldn = p.d * EB;
  typename T::Ctx c;
#pragma unroll
  for (int i = 0; i < T::LM; ++i) c.moff[i] = T::rows_offset(T::mq(wave, i), lane, 64);
#pragma unroll
  for (int i = 0; i < T::LN; ++i)
    c.noff[i] = T::template strided_offset<T::BN>(T::nq(wave, i), lane, nbase, p.d, ldn, 0);
  const int all = (p.T + T::KS - 1) / T::KS;
  const int j0 = min(all, z * p.steps), per = min(all - j0, p.steps);
  const int steps = per * (p.dz_lo != nullptr ? 2 : 1);
  const char* hi = static_cast<const char*>(p.dz_hi) + (size_t)mbase * 64;
  const char* lo = p.dz_lo != nullptr ? static_cast<const char*>(p.dz_lo) + (size_t)mbase * 64 : nullptr;
  const char* x = static_cast<const char*>(p.x);
  auto src = [&](int j) {
    Step s;
    const bool in = j < steps;
    const bool second = in && j >= per;
    const int q = in ? j0 + (second ? j - per : j) : 0;
    s.m = (second ? lo : hi) + (size_t)q * p.E * 64;
    s.n = x + (size_t)q * T::KS * ldn;
    s.mbytes = in ? rows * 64 : 0;
    s.nbytes = in ? min(T::KS, p.T - q * T::KS) * ldn : 0;
    return s;
  };
  f32x4_t acc[T::MI][T::NI];
  char* const stages[T::S] = {s0, s1, s2, s3};
  T::run(c, stages, steps, src, acc);
  const int wm = wave / T::WN, wn = wave % T::WN, g4 = (lane >> 4) * 4, i16 = lane & 15;
#pragma unroll
  for (int mi = 0; mi < T::MI; ++mi) {
    const int m = wm * T::TM + mi * 16 + i16;
    if (m < rows) {
#pragma unroll
      for (int ni = 0; ni < T::NI; ++ni) {
        const int n = nbase + wn * T::TN + ni * 16 + g4;
        if (n < p.d)
          store4<TF32>(p.part + ((size_t)z * p.E + mbase + m) * p.d + n, acc[mi][ni][0], acc[mi][ni][1],
                       acc[mi][ni][2], acc[mi][ni][3]);
      }
    }
  }
}

// ---- launches -----------------------------------------------------------------

inline unsigned whole_rounds(long long units) { return (unsigned)((units + 7) / 8 * 8); }

template <class Tr, class T, bool DH>
hipError_t launch_dgrad_cfg(const DgradArgs& a, long long max_tiles, hipStream_t stream) {
  const long long units = max_tiles * ((a.N + T::BN - 1) / T::BN);
  if (units == 0) return hipSuccess;
  hipLaunchKernelGGL((dgrad_kernel<Tr, T, DH>), dim3(whole_rounds(units)), dim3(T::NTH), 0, stream, a);
  return hipGetLastError();
}

template <class Tr, class T>
hipError_t launch_wgrad_cfg(WgradArgs a, hipStream_t stream) {
  long long per_e = 0;
  for (int w = 0; w < a.n; ++w) {
    a.first[w] = (int)per_e;
    per_e += (long long)((a.M[w] + T::BM - 1) / T::BM) * ((a.N[w] + T::BN - 1) / T::BN);
  }
  if (per_e == 0) return hipSuccess;
  if (per_e * a.rows.E > 0x7ffffff0LL) return hipErrorInvalidValue;
  a.units = (int)(per_e * a.rows.E);
  hipLaunchKernelGGL((wgrad_kernel<Tr, T>), dim3(whole_rounds(a.units)), dim3(T::NTH), 0, stream, a);
  return hipGetLastError();
}

}  // namespace grad
}  // namespace moe
