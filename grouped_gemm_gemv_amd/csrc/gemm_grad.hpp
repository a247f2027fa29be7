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
//
// The workgroups are persistent: each takes every so-many-th unit (tile) of
// its XCD's range, and the ring runs on across units, so the first steps of
// the next tile are on their way while the last ones of this one are
// multiplied and its results are stored.
#pragma once

#include <type_traits>

#include "device_common.hpp"
#include "launch.hpp"

namespace moe {
namespace grad {

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

// Waits: until at most n of this wavefront's vector-memory operations are
// outstanding; until its LDS reads have returned.
template <int n>
__device__ __forceinline__ void wait_vm() {
  static_assert(n >= 0 && n < 64, "vmcnt range");
#ifdef __HIP_DEVICE_COMPILE__
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(n) : "memory");
#endif
}
__device__ __forceinline__ void wait_lds() {
#ifdef __HIP_DEVICE_COMPILE__
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#endif
}

// Lane offset of an LDS-direct load (16 bytes per lane to 16 consecutive bytes
// per lane from lds_base on) from a buffer of `bytes` bytes at `base`; past the
// bound it writes zeros.  In assembler because the compiler, which sees only
// that such a load writes some LDS, would wait for all of them before every
// LDS read of a ring whose stage is not a constant; the kernel waits for its
// own loads instead (wait_vm).  It has no output registers.  The compiler looks
// after no wait states inside an asm block: s_nop 4 covers m0 (1) and a scalar
// operand that a vector instruction has just written (5 with the s_mov).
typedef unsigned u32x4_t __attribute__((ext_vector_type(4)));
__device__ __forceinline__ u32x4_t descriptor(const char* base, int bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  return u32x4_t{(unsigned)__builtin_amdgcn_readfirstlane((int)a),
                 (unsigned)__builtin_amdgcn_readfirstlane((int)(a >> 32)) & 0xffffu,
                 (unsigned)__builtin_amdgcn_readfirstlane(bytes), 0x00020000u};
}
__device__ __forceinline__ void load_lds(const u32x4_t& desc, int lane_offset, unsigned lds_base) {
#ifdef __HIP_DEVICE_COMPILE__
  lds_base = (unsigned)__builtin_amdgcn_readfirstlane((int)lds_base);
  asm volatile(
      "s_mov_b32 m0, %2\n\t"
      "s_nop 4\n\t"
      "buffer_load_dwordx4 %0, %1, 0 offen lds"
      :
      : "v"(lane_offset), "s"(desc), "s"(lds_base)
      : "memory");  // m0 is reserved: nothing else in these kernels uses it
#endif
}

// Two fp32 values to two bf16 in one word (round to nearest even).
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ unsigned pack2(float a, float b) {
  return __builtin_bit_cast(unsigned, bf16x2_t{(__bf16)a, (__bf16)b});
}
// Lanes 16..31 and 48..63 of a trade places with lanes 0..15 and 32..47 of b.
__device__ __forceinline__ void swap16(unsigned& a, unsigned& b) {
#ifdef __HIP_DEVICE_COMPILE__
  const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  a = r[0];
  b = r[1];
#endif
}

// Stores one row's NI blocks of 16 columns, of which lane group g = lane / 16
// holds columns 4g .. 4g + 3 (v[ni][0..3]).  at(n) gives the address of column n
// of the run; the NI * 16 columns are within a row of a matrix whose storage
// order keeps 8 (bf16) columns together.  bf16: two blocks at a time, lanes 16
// apart trade halves so that each lane stores 16 bytes (half the store
// instructions of 8 bytes a lane, in 64-byte pieces).
template <class Tr, int NI, class At>
__device__ __forceinline__ void store_blocks(const float (&v)[NI][4], bool live, int lane, At&& at) {
  const int g = lane >> 4;
  if constexpr (sizeof(typename Tr::T) == 2) {
    static_assert(NI % 2 == 0, "blocks pair up");
#pragma unroll
    for (int ni = 0; ni < NI; ni += 2) {
      unsigned a0 = pack2(v[ni][0], v[ni][1]), a1 = pack2(v[ni][2], v[ni][3]);
      unsigned b0 = pack2(v[ni + 1][0], v[ni + 1][1]), b1 = pack2(v[ni + 1][2], v[ni + 1][3]);
      swap16(a0, b0);
      swap16(a1, b1);
      // lane groups 0, 2: columns 0-7, 8-15 of block ni; groups 1, 3: of block ni + 1
      if (live) *reinterpret_cast<uint4*>(at((ni + (g & 1)) * 16 + (g >> 1) * 8)) = make_uint4(a0, a1, b0, b1);
    }
  } else {
#pragma unroll
    for (int ni = 0; ni < NI; ++ni)
      if (live)
        *reinterpret_cast<float4*>(at(ni * 16 + g * 4)) = make_float4(v[ni][0], v[ni][1], v[ni][2], v[ni][3]);
  }
}

// Where the operands of one K step lie: base addresses and descriptor bounds.
struct Step {
  const char* m;
  const char* n;
  int mbytes, nbytes;
};

template <class Tr, int BM_, int BN_, int WM_, int WN_, bool MKS, int S_, int OCC_, bool PP>
struct Tile {
  using Elt = typename Tr::T;
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, S = S_, OCC = OCC_;
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
  static_assert(S >= 3 && (S - 2) * NL < 64, "ring");

  // LDS swizzle.  A K-contiguous row is 64 bytes: chunk c (16 bytes) of row r
  // sits at c ^ (r / 2 & 3), so the 8 rows that eight lanes of an operand read
  // take spread over all banks (r / 4 & 3 took 40 % more LDS cycles).  A K-strided row k holds BM or BN columns (a multiple of 256 bytes):
  // its chunks are moved in pairs (bf16: a transposing read takes 32 bytes of
  // 4 rows per 16 lanes; the 8 rows of 32 lanes get 8 different pairs) or in
  // fours (fp32: 64 bytes of one row per 16 lanes).
  __device__ __forceinline__ static int swz_c(int r) { return (r >> 1) & 3; }
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

  __device__ __forceinline__ static int mq(int wave, int i) { return min(wave + i * NW, QM - 1); }
  __device__ __forceinline__ static int nq(int wave, int i) { return min(wave + i * NW, QN - 1); }

  // The loads of one step into the stage at LDS address `st`: lane offsets moff, noff.
  __device__ __forceinline__ static void load(const int (&moff)[LM], const int (&noff)[LN], const Step& s, unsigned st,
                                              int wave) {
    const u32x4_t m = descriptor(s.m, s.mbytes), n = descriptor(s.n, s.nbytes);
#pragma unroll
    for (int i = 0; i < LM; ++i) load_lds(m, moff[i], st + mq(wave, i) * 1024);
#pragma unroll
    for (int i = 0; i < LN; ++i) load_lds(n, noff[i], st + MBYTES + nq(wave, i) * 1024);
  }

  // Operand of the 16 columns (or rows) number sub of the wavefront's part:
  // columns in one run, rows dealt to the WM wavefront rows in turn, so that a
  // tile that is not full loads them evenly.  Lane group g = lane / 16 holds K elements 8g..8g+7 (bf16)
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
      return *reinterpret_cast<const uint4*>(st + lane0 + sub * WM * 1024);
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

  static __device__ __forceinline__ int m_first(int wave) { return MKS ? (wave / WN) * TM : (wave / WN) * 16; }
  // Row (or column) of the tile that accumulator block mi of this lane holds.
  static __device__ __forceinline__ int m_of(int wave, int mi, int lane) {
    return MKS ? (wave / WN) * TM + mi * 16 + (lane & 15) : (mi * WM + wave / WN) * 16 + (lane & 15);
  }
  static __device__ __forceinline__ int n_of(int wave, int ni, int lane) {
    return (wave % WN) * TN + ni * 16 + (lane >> 4) * 4;
  }

  // (job.store returns whether this wavefront issued every one of its stores.)
  // Works the units first, first + stride, ... < end of `job`.  `ring`: S stages
  // of LDS, at LDS address `ring_at`.
  template <class Job>
  struct Runner {
    using Info = typename Job::Info;
    Job& job;
    const char* const ring;
    const unsigned ring_at;
    const int stride, end, lane, wave, ml, nl;
    int L, lj, lpad;  // unit and step that the next loads are for, and the unit's padded steps
    int ls, cs;       // stages of the next load and of the next step
    Info lt, ct;      // the unit being loaded, the unit being multiplied
    Step ld;          // the next loads
    int stores;       // steps left for which this wavefront's ST stores of the unit before may be in flight
    int moff[LM], noff[LN];
    uint4 nf[NI], mf[MI];
    f32x4_t acc[MI][NI];

    __device__ __forceinline__ Runner(Job& job_, const char* ring_, unsigned ring_at_, int first, int stride_, int end_,
                                      int lane_, int wave_)
        : job(job_), ring(ring_), ring_at(ring_at_), stride(stride_), end(end_), lane(lane_), wave(wave_),
          ml(frag_lane<MKS, BM>(lane_, m_first(wave_))),
          nl(MBYTES + frag_lane<true, BN>(lane_, (wave_ % WN) * TN)), L(first), lj(0), lpad(0), ls(0), cs(0), stores(0) {}

    // A unit takes at least S steps (empty ones behind its own), so the loads,
    // S - 1 steps ahead, are never more than one unit ahead.
    __device__ __forceinline__ static int padded(const Info& t) { return t.steps > S ? t.steps : S; }
    __device__ __forceinline__ void open() {
      const bool in = L < end;  // else past the last unit: empty loads from here on
      if (in) {
        lt = job.decode(L);
        job.offsets(lt, wave, lane, moff, noff);
      }
      // (selects, not an else branch: stores of two branches merged into one
      // through a pointer would keep the state in scratch memory)
      lt.steps = in ? lt.steps : 0;
      lpad = in ? padded(lt) : 0x7fffffff;
      lj = 0;
      ld = job.first(lt);
    }
    // issue the next loads; move on to the ones after them
    __device__ __forceinline__ void feed() { load(moff, noff, ld, ring_at + ls * STAGE, wave); }
    __device__ __forceinline__ void advance() {
      ls = ls == S - 1 ? 0 : ls + 1;
      if (++lj == lpad) {
        L += stride;
        open();
      } else {
        job.next(lt, lj, ld);
      }
    }
    __device__ __forceinline__ static void barrier() {
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
      __builtin_amdgcn_sched_barrier(0);
    }
    template <int MB>
    __device__ __forceinline__ void read_frags() {
      const char* st = ring + cs * STAGE;
#pragma unroll
      for (int ni = 0; ni < NI; ++ni) nf[ni] = frag<true, BN>(st, nl, ni);
#pragma unroll
      for (int mi = 0; mi < MB; ++mi) mf[mi] = frag<MKS, BM>(st, ml, mi);
      cs = cs == S - 1 ? 0 : cs + 1;
    }
    template <int MB>
    __device__ __forceinline__ void multiply() {
#pragma unroll
      for (int mi = 0; mi < MB; ++mi)
#pragma unroll
        for (int ni = 0; ni < NI; ++ni) acc[mi][ni] = mma16<Tr>(nf[ni], mf[mi], acc[mi][ni]);
    }

    // One step.  This wavefront's loads of the step have landed (those of the
    // S - 2 after it may be in flight); after the barrier everyone's have, and
    // everyone is done with the stage of the step before, which takes the step
    // S - 1 ahead.
    template <int MB>
    __device__ __forceinline__ void step() {
      wait_step();
      barrier();
      feed();
      read_frags<MB>();
      advance();
      multiply<MB>();
    }

    // Ping-pong step (PP): the two wavefronts of each SIMD (w and w + NW / 2) take
    // turns, one multiplies while the other moves data, with a barrier between
    // the phases; the second half runs one phase behind.  The data phase of a
    // step issues the loads S - 1 steps ahead (into the stage of the step before,
    // which both halves have read: the second one in the phase just ended),
    // reads this step's operands, and waits until its own loads of the next step
    // have landed (both halves wait so before the first one reads that stage).
    // Where the next loads lie is worked out between the multiplications: with
    // it in the data phase, that phase was the longer one and set the pace.
    template <int MB>
    __device__ __forceinline__ void step_pp() {
      read_frags<MB>();
      feed();
      wait_step();
      wait_lds();
      barrier();
      advance();
      multiply<MB>();
      barrier();
    }
    // Waits until this wavefront's loads of one step have landed, with those of the
    // S - 2 steps issued after them in flight.  vmcnt counts loads and stores in
    // the order of their issue, so in the first S - 2 steps of a unit the ST
    // stores of the unit before it, if all of them were issued, lie behind the
    // awaited loads and are allowed for.
    static constexpr int ST = MI * NI * EB / 4;
    __device__ __forceinline__ void wait_step() {
      if (stores > 0) {
        --stores;
        wait_vm<(S - 2) * NL + ST>();
      } else {
        wait_vm<(S - 2) * NL>();
      }
    }

    // The steps of a unit, for its first MB blocks of 16 rows per wavefront.
    template <int MB>
    __device__ __forceinline__ void steps(int n) {
#pragma unroll 1
      for (int j = 0; j < n; ++j) {
        if constexpr (PP)
          step_pp<MB>();
        else
          step<MB>();
      }
    }

    __device__ __forceinline__ void run() {
      if (L >= end) return;
      open();
      ct = lt;
#pragma unroll 1
      for (int u = 0; u < S - 1; ++u) {  // within the first unit's padded steps
        feed();
        advance();
      }
      const bool second = wave >= NW / 2;
      if constexpr (PP) {
        static_assert(NW % 2 == 0, "wavefronts pair up");
        wait_vm<(S - 2) * NL>();
        barrier();
        if (second) barrier();
      }
#pragma unroll 1
      for (;;) {
#pragma unroll
        for (int mi = 0; mi < MI; ++mi)
#pragma unroll
          for (int ni = 0; ni < NI; ++ni) acc[mi][ni] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        // a tile of at most half the rows multiplies half the blocks
        if (!MKS && MI % 2 == 0 && ct.rows <= BM / 2)
          steps<(MI + 1) / 2>(padded(ct));
        else
          steps<MI>(padded(ct));
        stores = job.store(ct, wave, lane, acc) ? S - 2 : 0;
        if (L >= end) break;
        ct = lt;  // the next unit
      }
      if (PP && !second) barrier();
      wait_vm<0>();  // the empty loads past the last unit still write LDS
    }
  };
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

// The experts' rows and their row tiles' running count, in LDS: what a
// persistent workgroup looks up for each unit, without global loads whose
// wait would drain the ring.
struct ExpertTable {
  ExpertRows rows[256];
  int tiles[257];  // tiles of BM rows in front of expert i
};

__device__ __forceinline__ int tiles_of(int n, int BM) { return (n + BM - 1) / BM; }

// Filled by a whole workgroup of NTH >= 256 threads.
template <int BM>
__device__ __forceinline__ void fill_table(const GradRows& p, ExpertTable& t) {
  __shared__ int wave_sum[4];
  const int i = threadIdx.x, lane = i & 63;
  int n = 0;
  if (i < p.E) {
    const ExpertRows r = expert_rows(p, i);
    t.rows[i] = r;
    n = tiles_of(r.n0, BM) + tiles_of(r.n1, BM);
  }
  int inc = n;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(inc, o);
    if (lane >= o) inc += v;
  }
  if (i < 256 && lane == 63) wave_sum[i >> 6] = inc;
  __syncthreads();
  if (i < 256) {
    for (int w = 0; w < (i >> 6); ++w) inc += wave_sum[w];
    t.tiles[i + 1] = inc;  // experts past the last hold no tiles
    if (i == 0) t.tiles[0] = 0;
  }
  __syncthreads();
}

// Units of the persistent workgroup b of a grid that is a multiple of 8: XCD
// b mod 8 (workgroup ids go round the XCDs) owns a contiguous range of units,
// its workgroups take them in turn, so units at work at a time are neighbours.
struct Units {
  int first, stride, end;
};
__device__ __forceinline__ Units my_units(int total) {
  const int J = (total + 7) >> 3, x = blockIdx.x & 7;
  return Units{x * J + ((int)blockIdx.x >> 3), (int)gridDim.x >> 3, min(total, (x + 1) * J)};
}

// out tile = act rows x weights (DH: with the SwiGLU's gradient in the epilogue).
template <class Tr, class T, bool DH>
struct DgradJob {
  static constexpr int EB = T::EB;
  struct Info {
    int steps, row0, rows, nbase, e;
    const char *a0, *a1, *b0, *b1;  // operands of the tile's rows and expert
  };
  const DgradArgs& p;
  const ExpertTable& tab;
  const int NT, per;

  __device__ __forceinline__ DgradJob(const DgradArgs& p_, const ExpertTable& t)
      : p(p_), tab(t), NT((p_.N + T::BN - 1) / T::BN), per(p_.K / T::KS) {}
  __device__ __forceinline__ int units() const {
    return __builtin_amdgcn_readfirstlane(tab.tiles[256]) * NT;
  }

  // units: expert, then column tile, then row tile, so the row tiles that read
  // the same weights follow each other in one L2
  __device__ __forceinline__ Info decode(int L) const {
    const int lane = threadIdx.x & 63;
    int e = 0;
    for (int b = 0; b < p.rows.E; b += 64)
      e += __popcll(__ballot(b + lane < p.rows.E && tab.tiles[b + lane + 1] * NT <= L));
    e = __builtin_amdgcn_readfirstlane(e);
    const int before = __builtin_amdgcn_readfirstlane(tab.tiles[e]);
    const int r0 = __builtin_amdgcn_readfirstlane(tab.rows[e].r0), n0 = __builtin_amdgcn_readfirstlane(tab.rows[e].n0);
    const int r1 = __builtin_amdgcn_readfirstlane(tab.rows[e].r1), n1 = __builtin_amdgcn_readfirstlane(tab.rows[e].n1);
    const int t0 = tiles_of(n0, T::BM), t1 = tiles_of(n1, T::BM);
    const int local = L - before * NT;
    const int nt = local / (t0 + t1);
    const int ti = local - nt * (t0 + t1);
    const int n = ti < t0 ? n0 : n1, first = (ti < t0 ? ti : ti - t0) * T::BM;
    Info i;
    i.e = e;
    i.row0 = (ti < t0 ? r0 : r1) + first;
    i.rows = min(T::BM, n - first);
    i.nbase = nt * T::BN;
    i.steps = per * (p.a1 != nullptr ? 2 : 1);
    const size_t act = (size_t)i.row0 * p.K * EB, mat = (size_t)e * p.K * p.N * EB;
    i.a0 = static_cast<const char*>(p.a0) + act;
    i.b0 = static_cast<const char*>(p.b0) + mat;
    i.a1 = DH ? i.a0 : static_cast<const char*>(p.a1) + act;
    i.b1 = DH ? i.b0 : static_cast<const char*>(p.b1) + mat;
    return i;
  }
  __device__ __forceinline__ void offsets(const Info& t, int wave, int lane, int (&moff)[T::LM],
                                          int (&noff)[T::LN]) const {
#pragma unroll
    for (int i = 0; i < T::LM; ++i) moff[i] = T::rows_offset(T::mq(wave, i), lane, p.K * EB);
#pragma unroll
    for (int i = 0; i < T::LN; ++i)
      noff[i] = T::template strided_offset<T::BN>(T::nq(wave, i), lane, t.nbase, p.N, p.N * EB, p.blocked16);
  }
  __device__ __forceinline__ Step first(const Info& t) const {
    return t.steps > 0 ? Step{t.a0, t.b0, t.rows * p.K * EB, T::KS * p.N * EB} : Step{t.a0, t.b0, 0, 0};
  }
  // Step j: 64 bytes on in the activation rows, KS rows on in the weights.
  __device__ __forceinline__ void next(const Info& t, int j, Step& s) const {
    const int nrows = T::KS * p.N * EB;
    s.m += 64;
    s.n += nrows;
    s.mbytes = max(s.mbytes - 64, 0);
    if (!DH && j == per) {
      s.m = t.a1;
      s.n = t.b1;
      s.mbytes = t.rows * p.K * EB;
    }
    if (j >= t.steps) s.mbytes = s.nbytes = 0;
  }
  // The saved projections of one row's NI blocks of 16 columns.
  struct Saved {
    unsigned g[T::NI], u[T::NI], gx, ux;  // four codes each; the blocks' exponents, one byte each
    float w;
  };
  __device__ __forceinline__ void read_saved(const Info& t, int mi, int n0, int wave, int lane, Saved& s) const {
    const int m = T::m_of(wave, mi, lane);
    const size_t row = (size_t)t.row0 + (m < t.rows ? m : 0);
    const size_t o = row * p.N + n0;
#pragma unroll
    for (int ni = 0; ni < T::NI; ++ni) {
      s.g[ni] = *reinterpret_cast<const unsigned*>(p.g8 + o + ni * 16 + (lane >> 4) * 4);
      s.u[ni] = *reinterpret_cast<const unsigned*>(p.u8 + o + ni * 16 + (lane >> 4) * 4);
    }
    using Exps = std::conditional_t<T::NI == 4, uint32_t, uint16_t>;
    static_assert(T::NI == 4 || T::NI == 2, "exponents of a wavefront's columns in one load");
    s.gx = *reinterpret_cast<const Exps*>(p.gx + (o >> 4));
    s.ux = *reinterpret_cast<const Exps*>(p.ux + (o >> 4));
    s.w = p.wrow[row];
  }
  __device__ __forceinline__ bool store(const Info& t, int wave, int lane, f32x4_t (&acc)[T::MI][T::NI]) const {
    // a wavefront's columns are all inside the matrix or all behind it (both
    // are multiples of 64, or of 32 with tiles of 128 columns)
    const int n0 = t.nbase + (wave % T::WN) * T::TN;
    if constexpr (!DH) {
      if (n0 >= p.N) return false;
#pragma unroll
      for (int mi = 0; mi < T::MI; ++mi) {
        const int m = T::m_of(wave, mi, lane);
        char* row = static_cast<char*>(p.out) + (((size_t)t.row0 + m) * p.N + n0) * EB;
        float v[T::NI][4];
#pragma unroll
        for (int ni = 0; ni < T::NI; ++ni)
#pragma unroll
          for (int r = 0; r < 4; ++r) v[ni][r] = acc[mi][ni][r];
        store_blocks<Tr, T::NI>(v, m < t.rows, lane, [&](int n) { return row + n * EB; });
      }
      return t.rows == T::BM;
    } else {
      const bool in = n0 < p.N;
      // the next block's codes are on their way while this one's are worked
      Saved s[2];
      if (in) read_saved(t, 0, n0, wave, lane, s[0]);
#pragma unroll
      for (int mi = 0; mi < T::MI; ++mi) {
        const int m = T::m_of(wave, mi, lane);
        const bool live = m < t.rows;
        const size_t row = (size_t)t.row0 + (live ? m : 0);
        float dot = 0.f;
        if (in) {
          if (mi + 1 < T::MI) read_saved(t, mi + 1, n0, wave, lane, s[(mi + 1) & 1]);
          const Saved& q = s[mi & 1];
          float dg[T::NI][4], du[T::NI][4], hw[T::NI][4];
#pragma unroll
          for (int ni = 0; ni < T::NI; ++ni) {
            const float gs = exp_scale((q.gx >> (8 * ni)) & 255u), us = exp_scale((q.ux >> (8 * ni)) & 255u);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float D = acc[mi][ni][r];
              const float g = code_of(q.g[ni], r) * gs, u = code_of(q.u[ni], r) * us;
              const float sg = __builtin_amdgcn_rcpf(1.0f + __expf(-g));
              const float a = g * sg, h = a * u;
              dot = fmaf(D, h, dot);
              const float dh = q.w * D;
              du[ni][r] = dh * a;
              dg[ni][r] = dh * (u * sg * fmaf(g, 1.0f - sg, 1.0f));
              hw[ni][r] = q.w * h;
            }
          }
          const size_t o = (row * p.N + n0) * EB;
          store_blocks<Tr, T::NI>(dg, live, lane, [&](int n) { return static_cast<char*>(p.dg) + o + n * EB; });
          store_blocks<Tr, T::NI>(du, live, lane, [&](int n) { return static_cast<char*>(p.du) + o + n * EB; });
          if (p.hw != nullptr)
            store_blocks<Tr, T::NI>(hw, live, lane, [&](int n) { return static_cast<char*>(p.hw) + o + n * EB; });
        }
        // the wavefront's columns of <D, h>: the four lanes of a row, then one
        // partial sum per wavefront column, added in order by a later step
        dot += __shfl_xor(dot, 16);
        dot += __shfl_xor(dot, 32);
        if (live && lane < 16)
          p.dot[row * (size_t)p.dot_ld + (t.nbase / T::BN) * T::WN + wave % T::WN] = dot;
        __builtin_amdgcn_sched_barrier(0);  // one block's values at a time, or the registers overflow
      }
      return false;
    }
  }
};

#define MOE_GRAD_RING                                                                                  \
  __shared__ __attribute__((aligned(1024))) char ring[T::S * T::STAGE];                               \
  const unsigned ring_at = (unsigned)(uintptr_t)(__attribute__((address_space(3))) char*)(ring);      \
  const int lane = threadIdx.x & 63;                                                                   \
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)

template <class Tr, class T, bool DH>
__global__ __launch_bounds__(T::NTH) void dgrad_kernel(DgradArgs p) {
  MOE_GRAD_RING;
  __shared__ ExpertTable tab;
  fill_table<T::BM>(p.rows, tab);
  DgradJob<Tr, T, DH> job(p, tab);
  const Units u = my_units(job.units());
  typename T::template Runner<DgradJob<Tr, T, DH>>(job, ring, ring_at, u.first, u.stride, u.end, lane, wave).run();
}

// ---- weight gradients ---------------------------------------------------------

// out[e][m][n] = sum over the rows r of expert e of P[r][m] Q[r][n]: up to three
// such products in one launch.  An expert without rows gets zeros.
template <class Tr, class T>
struct WgradJob {
  static constexpr int EB = T::EB;
  struct Info {
    int steps, rows, steps0, e, w, mbase, nbase, ldm, ldn;
    int n0, n1;
    const char *p0, *q0, *p1, *q1;  // the operands' first rows of either run
  };
  const WgradArgs& p;
  const ExpertTable& tab;
  __device__ __forceinline__ WgradJob(const WgradArgs& p_, const ExpertTable& t) : p(p_), tab(t) {}

  __device__ __forceinline__ Info decode(int L) const {
    const int per_e = p.units / p.rows.E;
    Info i;
    i.e = L / per_e;
    L -= i.e * per_e;
    i.w = (p.n > 1 && L >= p.first[1] ? 1 : 0) + (p.n > 2 && L >= p.first[2] ? 1 : 0);
    L -= p.first[i.w];
    const int MT = (p.M[i.w] + T::BM - 1) / T::BM, NT = (p.N[i.w] + T::BN - 1) / T::BN;
    // groups of 8 row tiles by all column tiles, so the tiles at work at a time
    // form a near-square patch of the output that shares both operands in L2
    const int gsz = 8 * NT;
    const int grp = L / gsz, in = L - grp * gsz;
    const int gm = min(8, MT - grp * 8);
    const int nt = in / gm;
    i.mbase = (grp * 8 + in - nt * gm) * T::BM;
    i.nbase = nt * T::BN;
    i.rows = T::BM;
    const int r0 = __builtin_amdgcn_readfirstlane(tab.rows[i.e].r0);
    i.n0 = __builtin_amdgcn_readfirstlane(tab.rows[i.e].n0);
    const int r1 = __builtin_amdgcn_readfirstlane(tab.rows[i.e].r1);
    i.n1 = __builtin_amdgcn_readfirstlane(tab.rows[i.e].n1);
    i.ldm = p.M[i.w] * EB;
    i.ldn = p.N[i.w] * EB;
    i.p0 = static_cast<const char*>(p.P[i.w]) + (size_t)r0 * i.ldm;
    i.q0 = static_cast<const char*>(p.Q[i.w]) + (size_t)r0 * i.ldn;
    i.p1 = static_cast<const char*>(p.P[i.w]) + (size_t)r1 * i.ldm;
    i.q1 = static_cast<const char*>(p.Q[i.w]) + (size_t)r1 * i.ldn;
    i.steps0 = (i.n0 + T::KS - 1) / T::KS;
    i.steps = i.steps0 + (i.n1 + T::KS - 1) / T::KS;
    return i;
  }
  __device__ __forceinline__ void offsets(const Info& t, int wave, int lane, int (&moff)[T::LM],
                                          int (&noff)[T::LN]) const {
    const int M = p.M[t.w], N = p.N[t.w];
#pragma unroll
    for (int i = 0; i < T::LM; ++i)
      moff[i] = T::template strided_offset<T::BM>(T::mq(wave, i), lane, t.mbase, M, t.ldm, 0);
#pragma unroll
    for (int i = 0; i < T::LN; ++i)
      noff[i] = T::template strided_offset<T::BN>(T::nq(wave, i), lane, t.nbase, N, t.ldn, 0);
  }
  __device__ __forceinline__ Step first(const Info& t) const {
    Step s{t.n0 > 0 ? t.p0 : t.p1, t.n0 > 0 ? t.q0 : t.q1, 0, 0};
    const int left = t.steps > 0 ? min(T::KS, t.n0 > 0 ? t.n0 : t.n1) : 0;
    s.mbytes = left * t.ldm;
    s.nbytes = left * t.ldn;
    return s;
  }
  // Step j: KS rows on; the rows behind the capacity follow those in front of it.
  __device__ __forceinline__ void next(const Info& t, int j, Step& s) const {
    s.m += (size_t)(T::KS * t.ldm);
    s.n += (size_t)(T::KS * t.ldn);
    const bool second = j >= t.steps0;
    if (j == t.steps0) {
      s.m = t.p1;
      s.n = t.q1;
    }
    const int left = max(0, min(T::KS, second ? t.n1 - (j - t.steps0) * T::KS : t.n0 - j * T::KS));
    const int rows = j < t.steps ? left : 0;
    s.mbytes = rows * t.ldm;
    s.nbytes = rows * t.ldn;
  }
  __device__ __forceinline__ bool store(const Info& t, int wave, int lane, f32x4_t (&acc)[T::MI][T::NI]) const {
    const int M = p.M[t.w], N = p.N[t.w];
    const int n0 = t.nbase + (wave % T::WN) * T::TN;  // as in DgradJob: all in or all out
    if (n0 >= N) return false;
    char* out = static_cast<char*>(p.out[t.w]) + (size_t)t.e * M * N * EB;
    const int m0 = T::m_of(wave, 0, 0);
#pragma unroll
    for (int mi = 0; mi < T::MI; ++mi) {
      const int m = t.mbase + T::m_of(wave, mi, lane);
      float v[T::NI][4];
#pragma unroll
      for (int ni = 0; ni < T::NI; ++ni)
#pragma unroll
        for (int r = 0; r < 4; ++r) v[ni][r] = acc[mi][ni][r];
      // the weight's storage order: rows, or 64-byte pieces of 16 rows in turn
      char* row = out + (p.blocked16 ? ((size_t)(m >> 4) * 16 * N + (m & 15) * T::KS) * EB : (size_t)m * N * EB);
      store_blocks<Tr, T::NI>(v, m < M, lane, [&](int n) {
        const int c = n0 + n;
        return row + (p.blocked16 ? (size_t)(c / T::KS) * (16 * T::KS) + c % T::KS : (size_t)c) * EB;
      });
    }
    return t.mbase + m0 + T::TM <= M;
  }
};

template <class Tr, class T>
__global__ __launch_bounds__(T::NTH) void wgrad_kernel(WgradArgs p) {
  MOE_GRAD_RING;
  __shared__ ExpertTable tab;
  fill_table<T::BM>(p.rows, tab);
  WgradJob<Tr, T> job(p, tab);
  const Units u = my_units(p.units);
  typename T::template Runner<WgradJob<Tr, T>>(job, ring, ring_at, u.first, u.stride, u.end, lane, wave).run();
}

// ---- router weight gradient ---------------------------------------------------

// part[z][e][i] = sum over tokens t of range z of dz[e][t] x[t][i] (fp32 partial
// sums).  dz is dense with zeros where expert e did not take token t, laid out
// by K step: [step][E][64 bytes].  bf16 carries it as two terms (high and low
// part), which keeps 16 bits of its significand.  One tile per workgroup.
template <class Tr, class T>
struct RouteJob {
  static constexpr int EB = T::EB;
  struct Info {
    int steps, rows;
  };
  const RouteWgradArgs& p;
  const int nbase, mbase, rows, j0, per;
  __device__ __forceinline__ explicit RouteJob(const RouteWgradArgs& p_)
      : p(p_), nbase(blockIdx.x * T::BN), mbase(blockIdx.y * T::BM), rows(min(T::BM, p_.E - mbase)),
        j0(min((p_.T + T::KS - 1) / T::KS, (int)blockIdx.z * p_.steps)),
        per(min((p_.T + T::KS - 1) / T::KS - j0, p_.steps)) {}
  __device__ __forceinline__ Info decode(int) const { return Info{per * (p.dz_lo != nullptr ? 2 : 1), rows}; }
  __device__ __forceinline__ void offsets(const Info&, int wave, int lane, int (&moff)[T::LM],
                                          int (&noff)[T::LN]) const {
#pragma unroll
    for (int i = 0; i < T::LM; ++i) moff[i] = T::rows_offset(T::mq(wave, i), lane, 64);
#pragma unroll
    for (int i = 0; i < T::LN; ++i)
      noff[i] = T::template strided_offset<T::BN>(T::nq(wave, i), lane, nbase, p.d, p.d * EB, 0);
  }
  __device__ __forceinline__ Step first(const Info& t) const {
    Step s{};
    next(t, 0, s);
    return s;
  }
  __device__ __forceinline__ void next(const Info& t, int j, Step& s) const {
    const int ldn = p.d * EB;
    const bool in = j < t.steps, second = in && j >= per;
    const int q = in ? j0 + (second ? j - per : j) : 0;
    s.m = static_cast<const char*>(second ? p.dz_lo : p.dz_hi) + ((size_t)q * p.E + mbase) * 64;
    s.n = static_cast<const char*>(p.x) + (size_t)q * T::KS * ldn;
    s.mbytes = in ? rows * 64 : 0;
    s.nbytes = in ? min(T::KS, p.T - q * T::KS) * ldn : 0;
  }
  __device__ __forceinline__ bool store(const Info&, int wave, int lane, f32x4_t (&acc)[T::MI][T::NI]) const {
#pragma unroll
    for (int mi = 0; mi < T::MI; ++mi) {
      const int m = T::m_of(wave, mi, lane);
      if (m < rows) {
#pragma unroll
        for (int ni = 0; ni < T::NI; ++ni) {
          const int n = nbase + T::n_of(wave, ni, lane);
          if (n < p.d)
            store4<TF32>(p.part + ((size_t)blockIdx.z * p.E + mbase + m) * p.d + n, acc[mi][ni][0], acc[mi][ni][1],
                         acc[mi][ni][2], acc[mi][ni][3]);
        }
      }
    }
    return false;
  }
};

template <class Tr, class T>
__global__ __launch_bounds__(T::NTH) void route_wgrad_kernel(RouteWgradArgs p) {
  MOE_GRAD_RING;
  RouteJob<Tr, T> job(p);
  typename T::template Runner<RouteJob<Tr, T>>(job, ring, ring_at, 0, 1, 1, lane, wave).run();
}

// ---- launches -----------------------------------------------------------------

constexpr int kComputeUnits = 256;

// Persistent workgroups: T::OCC for each compute unit (what LDS and registers
// admit), in whole rounds of the XCDs, no more than there are units.
template <class T>
inline unsigned grid_of(long long units) {
  const long long most = (long long)kComputeUnits * T::OCC;
  return (unsigned)((units < most ? (units + 7) / 8 * 8 : most));
}

template <class Tr, class T, bool DH>
hipError_t launch_dgrad_cfg(const DgradArgs& a, long long max_tiles, hipStream_t stream) {
  const long long units = max_tiles * ((a.N + T::BN - 1) / T::BN);
  if (units == 0) return hipSuccess;
  if (units > 0x7fffff00LL) return hipErrorInvalidValue;
  hipLaunchKernelGGL((dgrad_kernel<Tr, T, DH>), dim3(grid_of<T>(units)), dim3(T::NTH), 0, stream, a);
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
  if (per_e * a.rows.E > 0x7fffff00LL) return hipErrorInvalidValue;
  a.units = (int)(per_e * a.rows.E);
  hipLaunchKernelGGL((wgrad_kernel<Tr, T>), dim3(grid_of<T>(a.units)), dim3(T::NTH), 0, stream, a);
  return hipGetLastError();
}

}  // namespace grad
}  // namespace moe
