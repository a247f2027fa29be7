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
// operand is staged in LDS as it lies in memory and turned on the way to the
// registers: bf16 by the transposing LDS read (in each group of 16 lanes, lane
// i receives column i of a 4 x 16 block), fp32 by reading one element per K row.
//
// out[m][n] = sum_k Mop[m][k] Nop[k][n]; a workgroup owns a BM x BN tile,
// WM x WN wavefronts of TM x TN each.  N is the MFMA "A" operand, so a lane ends
// with 4 consecutive n of one m, as the outputs lie in memory.
//
// Activations between the products (dout in expert order, dg, du, w_r h) are
// kept in panels: [columns of 64 bytes][R rows][64 bytes].  A K step of the data
// gradients (64 bytes of every row of a tile) and 16 K rows of 64 bytes of the
// weight gradients are then both one run of memory, whatever the width of a
// row: with rows of 28 KB, a multiple of 4 KB apart, the second data gradient
// took 2049 instead of 1722 us (8192 rows, d = 4096, F = 14336).  The weight
// gradients' other operand, x and dout, is turned once by the gather in front
// (gather_backward_kernel) and read at the full rate of LDS, twice that of the
// transposing read (2769 instead of 2923 us).  Weights are read as the caller
// keeps them.
//
// A K step is 64 bytes of a K-contiguous row (32 bf16 or 16 fp32), so each
// operand takes 64 bytes of LDS per tile row or column whatever its
// orientation.  The steps go through a ring of S LDS stages written by
// LDS-direct buffer loads S - 1 steps ahead.  Reads past a descriptor's bound
// return zero, which pads rows past an expert's last one, columns past the
// matrix and steps past the last.
//
// The workgroups are persistent: each takes every so-many-th unit (tile) of
// its XCD's range or of the whole, and the ring runs on across units, so the first steps of
// the next tile are on their way while the last ones of this one are
// multiplied and its results are stored.
//
// What bounds them, at d = 4096, F = 14336 with 8 experts (bf16):
//  * many rows: the matrix cores.  8192 rows take 927 us (first data gradient,
//    1.04 PF/s), 1584 (second, 1.21) and 2879 (weight gradients, 1.00), where a
//    library product of 8192 cubed reaches 1.28, or 1.12 with a transposed
//    operand; the clock falls to 2.0 GHz.  What is left: the codes and the
//    epilogue of the first, the stores between the tiles of the last;
//  * few rows: memory.  32 rows take 186 and 291 us (0.94 and 1.88 GB of
//    weights, 5.1 and 6.5 TB/s) and 606 (2.8 GB of weight gradients, 4.7 TB/s
//    where a fill reaches 6.9: a tile's rows are 512-byte pieces).
#pragma once

#include <algorithm>
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

// Lanes 32..63 of a trade places with lanes 0..31 of b.
__device__ __forceinline__ void swap32(unsigned& a, unsigned& b) {
#ifdef __HIP_DEVICE_COMPILE__
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r[0];
  b = r[1];
#endif
}
// In each row of 16 lanes, lanes 8..15 of a trade places with lanes 0..7 of b.
__device__ __forceinline__ void swap8(unsigned& a, unsigned& b) {
#ifdef __HIP_DEVICE_COMPILE__
  constexpr int kRor8 = 0x128;  // rotate within a row of 16 lanes by 8
  const unsigned x = a;
  a = (unsigned)__builtin_amdgcn_update_dpp((int)a, (int)b, kRor8, 0xf, 0xc, false);
  b = (unsigned)__builtin_amdgcn_update_dpp((int)b, (int)x, kRor8, 0xf, 0x3, false);
#endif
}
// Word w of lane group g (of 16 lanes) becomes word g of lane group w.
__device__ __forceinline__ void transpose4(unsigned (&w)[4]) {
  swap32(w[0], w[2]);
  swap32(w[1], w[3]);
  swap16(w[0], w[1]);
  swap16(w[2], w[3]);
}

// Stores and loads of a buffer of `bytes` bytes at `base`, which the compiler
// counts itself: past the bound, stores are dropped and loads return zero.  The
// 16-byte stores are the GEMMs' results, streamed past the caches (nt): kept
// there, the gradients of the weights were still being written back while the
// next kernel read (the first data gradient of the next call took 243 instead of
// 181 us with 16 rows at the Mixtral shape, the weight gradients the same time).
constexpr int kNonTemporal = 2;
__device__ __forceinline__ void buf_store16(const char* base, int bytes, int offset, const uint4& v) {
#ifdef __HIP_DEVICE_COMPILE__  // the host pass knows no descriptors
  const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), (short)0, bytes, 0x00020000);
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, v), r, offset, 0, kNonTemporal);
#endif
}
__device__ __forceinline__ void buf_store4(const char* base, int bytes, int offset, unsigned v) {
#ifdef __HIP_DEVICE_COMPILE__
  const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), (short)0, bytes, 0x00020000);
  __builtin_amdgcn_raw_buffer_store_b32(v, r, offset, 0, 0);
#endif
}
__device__ __forceinline__ uint4 buf_load16(const char* base, int bytes, int offset) {
#ifdef __HIP_DEVICE_COMPILE__
  const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), (short)0, bytes, 0x00020000);
  return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r, offset, 0, 0));
#else
  return uint4{};
#endif
}
__device__ __forceinline__ unsigned buf_load4(const char* base, int bytes, int offset) {
#ifdef __HIP_DEVICE_COMPILE__
  const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), (short)0, bytes, 0x00020000);
  return __builtin_amdgcn_raw_buffer_load_b32(r, offset, 0, 0);
#else
  return 0;
#endif
}

// Where a lane's 16 bytes of a wavefront's tile of an output matrix lie: the
// rows of the matrix (ld bytes), 64-byte pieces of 16 rows in turn (the blocked
// weight order), or panels.  A piece is 64 bytes of columns of 16 rows: two
// blocks of 16 columns (bf16) or one (fp32).  Rows past the bound are dropped.
template <class Tr>
struct OutTile {
  static constexpr int EB = sizeof(typename Tr::T);
  const char* base;  // of the tile's first row
  size_t piece;      // bytes to the next 64 bytes of columns
  int bytes, ld, lane0;
  int half;          // rows of a matrix: bytes to the second half of a pair's rows, else 0
  // a lane's bytes in the 64: bf16, after the trade below, 16 of block g mod 2
  __device__ __forceinline__ static int lane_byte(int g) { return EB == 2 ? (g & 1) * 32 + (g >> 1) * 16 : g * 16; }
  // a row-major or blocked matrix: m0, col0 the wavefront's first row and column,
  // `pairs` whether its pieces pair up
  __device__ __forceinline__ static OutTile matrix(const char* base, int rows, int ld, int m0, int col0, int lane,
                                                   int blocked16, bool pairs) {
    const int g = lane >> 4, i = lane & 15;
    const int r = blocked16 ? i * 64 : pairs ? (i & 7) * ld + (i >> 3) * 64 : i * ld;
    return OutTile{base + (size_t)(blocked16 ? col0 * EB * 16 : col0 * EB), (size_t)(blocked16 ? 1024 : 64),
                   rows > 0 ? rows * ld - (blocked16 ? 0 : col0 * EB) : 0, ld, m0 * ld + r + lane_byte(g),
                   !blocked16 && pairs ? 8 * ld : 0};
  }
  // panels: base of the tile's first row in the panel of the wavefront's first columns
  __device__ __forceinline__ static OutTile panels(const char* base, size_t panel, int rows, int m0, int lane) {
    return OutTile{base, panel, rows * 64, 64, (m0 + (lane & 15)) * 64 + lane_byte(lane >> 4), 0};
  }
  // Rows m .. m + 15 (m a multiple of 16, from m0 on), NI blocks of 16 columns of
  // which lane group g = lane / 16 holds columns 4g .. 4g + 3.  bf16: lanes 16
  // apart trade halves, so that each stores 16 bytes.  In blocks and panels a
  // piece is one run of 1 KB.  In rows it is half a cache line of each of 16 rows;
  // two pieces trade rows, so that a store takes whole lines of 8 rows (weight
  // gradients of 1024 rows at d = 4096, F = 14336: 939 against 969 us).
  template <int NI>
  __device__ __forceinline__ void put(int m, const float (&v)[NI][4]) const {
    constexpr int PC = NI * EB / 4;
    unsigned w[PC][4];
    if constexpr (EB == 2) {
      static_assert(NI % 2 == 0, "blocks pair up");
#pragma unroll
      for (int q = 0; q < PC; ++q) {
        const float(&a)[4] = v[2 * q];
        const float(&b)[4] = v[2 * q + 1];
        w[q][0] = pack2(a[0], a[1]), w[q][1] = pack2(a[2], a[3]);
        w[q][2] = pack2(b[0], b[1]), w[q][3] = pack2(b[2], b[3]);
        // lane groups 0, 2: columns 0-7, 8-15 of block 2q; groups 1, 3: of block 2q + 1
        swap16(w[q][0], w[q][2]);
        swap16(w[q][1], w[q][3]);
      }
    } else {
#pragma unroll
      for (int q = 0; q < PC; ++q)
#pragma unroll
        for (int r = 0; r < 4; ++r) w[q][r] = __float_as_uint(v[q][r]);
    }
    const int at = lane0 + m * ld;
    if (PC % 2 == 0 && half != 0) {
#pragma unroll
      for (int q = 0; q + 1 < PC; q += 2) {
#pragma unroll
        for (int r = 0; r < 4; ++r) swap8(w[q][r], w[q + 1][r]);
        buf_store16(base + q * piece, bytes - q * 64, at, make_uint4(w[q][0], w[q][1], w[q][2], w[q][3]));
        buf_store16(base + q * piece, bytes - q * 64, at + half,
                make_uint4(w[q + 1][0], w[q + 1][1], w[q + 1][2], w[q + 1][3]));
      }
    } else {
#pragma unroll
      for (int q = 0; q < PC; ++q)
        buf_store16(base + q * piece, bytes, at, make_uint4(w[q][0], w[q][1], w[q][2], w[q][3]));
    }
  }
};

// Where the operands of one K step lie: base addresses and descriptor bounds.
struct Step {
  const char* m;
  const char* n;
  int mbytes, nbytes;
};

// How an operand lies in memory and LDS.
enum Operand {
  kPanelK,  // panels, K along the columns: a step is one panel
  kSteps,   // [step][columns of the tile's matrix][64 bytes of K]: turned by the gather
  kPanelR,  // panels, K along the rows: a step is KS rows of every panel of the tile
  kRows     // a matrix (or blocked weights), K along its rows: a step is KS rows
};

template <class Tr, int BM_, int BN_, int WM_, int WN_, Operand MOP_, Operand NOP_, int S_, int OCC_, bool PP>
struct Tile {
  using Elt = typename Tr::T;
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, S = S_, OCC = OCC_;
  static constexpr Operand MOP = MOP_, NOP = NOP_;
  static constexpr int EB = sizeof(Elt);
  static constexpr int KS = 64 / EB;  // K elements per step
  static constexpr int NW = WM * WN, NTH = 64 * NW;
  static constexpr int TM = BM / WM, TN = BN / WN, MI = TM / 16, NI = TN / 16;
  static constexpr int MBYTES = 64 * BM, STAGE = 64 * (BM + BN);
  // 1 KB LDS-direct loads per stage and operand, and per wavefront (the last
  // ones repeat an operand's final load, so every wavefront issues NL)
  static constexpr bool DEALT = MOP == kPanelK;
  static constexpr int M_STEP = DEALT ? 16 * WM : 16;  // rows between a wavefront's blocks
  static constexpr int QM = BM / 16, QN = BN / 16;
  static constexpr int LM = (QM + NW - 1) / NW, LN = (QN + NW - 1) / NW, NL = LM + LN;
  static constexpr int PL = EB == 2 ? 2 : 1;  // loads per panel of KS rows (kPanelR)
  static_assert(MOP != kRows && NOP != kPanelK, "the M operand comes in panels, the N operand has K along the rows");
  static_assert(TM % 16 == 0 && TN % 16 == 0, "wavefront tile");
  static_assert(MOP != kPanelR, "K along the rows is the N operand's");
  static_assert(NOP != kRows || BN * EB % 256 == 0, "rows are swizzled within 256 bytes");
  static_assert(NOP != kPanelR || (QN % NW == 0 && NW % 2 == 0 && TN * EB % 64 == 0), "panels of the N operand");
  static_assert(S >= 3 && (S - 2) * NL + MI * NI * EB / 4 < 64, "ring");

  // LDS layouts, each free of bank conflicts:
  //  kPanelK, kSteps: rows of 64 bytes; chunk c (16 bytes) of row r sits at c ^ (r / 2 & 3),
  //    so the 8 rows that eight lanes of a 16-byte read take cover 128 bytes of
  //    banks twice over (with r / 4 & 3 the reads took 40 % more cycles);
  //  kPanelR: the tile's panels in turn, KS rows of 64 bytes each.  bf16: a
  //    transposing read takes 32 bytes of 4 rows per 16 lanes, 8 rows per 32
  //    lanes; the halves of rows with bit 3 set trade places.  fp32: 16 lanes
  //    read 64 bytes of one row, lane groups rows 4 apart; rows are stored in the
  //    order 0 4 8 12 1 5 ..;
  //  kRows: KS rows of BN columns (a multiple of 256 bytes); pairs of chunks (bf16)
  //    or fours (fp32) move within 256 bytes so that the 8 rows (lane groups) of
  //    32 lanes get different ones.
  __device__ __forceinline__ static int swz_c(int r) { return (r >> 1) & 3; }
  __device__ __forceinline__ static int swz_k(int k) {
    return EB == 2 ? (((k & 3) | ((k >> 1) & 4)) << 1) : ((k >> 2) & 3) << 2;
  }

  __device__ __forceinline__ static int mq(int wave, int i) { return min(wave + i * NW, QM - 1); }
  __device__ __forceinline__ static int nq(int wave, int i) { return min(wave + i * NW, QN - 1); }

  // Offset in memory of this lane's 16 bytes of a load whose LDS slot is lane * 16:
  // 16 rows of 64 bytes from one run.
  template <Operand OP>
  __device__ __forceinline__ static int panel_offset(int q, int lane) {
    const int s = lane >> 2, c = lane & 3;
    if constexpr (OP == kPanelK || OP == kSteps) {
      const int r = q * 16 + s;
      return r * 64 + ((c ^ swz_c(r)) << 4);
    } else if constexpr (EB == 2) {
      return s * 64 + ((c ^ ((s >> 2) & 2)) << 4);
    } else {
      return ((s >> 2) | (s & 3) << 2) * 64 + (c << 4);
    }
  }
  // kRows: K row of this lane's slot in load q.
  __device__ __forceinline__ static int k_row(int q, int lane) { return (q * 64 + lane) / (BN * EB / 16); }
  // kRows: byte offset inside the step of this lane's slot in load q, for a tile
  // from column col0 on of rows of `cols` elements (ld bytes each).  blocked16: the
  // rows are in groups of 16, each stored as 1024-byte blocks of 64 bytes from
  // every row.
  __device__ __forceinline__ static int rows_offset(int q, int lane, int col0, int cols, int ld, int blocked16) {
    constexpr int CPR = BN * EB / 16;  // chunks per K row
    const int pos = q * 64 + lane;
    const int k = pos / CPR;
    const int c = (pos - k * CPR) ^ swz_k(k);
    const int col = col0 + c * (16 / EB);
    if (col >= cols) return kOutside;
    const int byte = col * EB;
    return blocked16 ? (k >> 4) * 16 * ld + (byte >> 6) * 1024 + (k & 15) * 64 + (byte & 63) : k * ld + byte;
  }

  // Operand of the 16 columns (or rows) number sub of the wavefront's part: in one
  // run, but rows of kPanelK dealt to the WM wavefront rows in turn, so that a
  // tile that is not full loads them evenly.  Lane group g = lane / 16
  // holds K elements 8g..8g+7 (bf16) or 4g..4g+3 (fp32), whatever the layout.
  // lane0: lane part of the LDS address, from frag_lane.
  template <Operand OP>
  __device__ __forceinline__ static int frag_lane(int lane, int first) {
    const int g = lane >> 4, i = lane & 15;
    if constexpr (OP == kPanelK || OP == kSteps) {
      const int r = first + i;
      return r * 64 + ((g ^ swz_c(r)) << 4);
    } else if constexpr (OP == kPanelR) {
      const int panel = first * EB / 64 * (KS * 64);
      return panel + (EB == 2 ? (8 * g + (i >> 2)) * 64 + ((i & 3) * 8 ^ (g & 1) * 32) : g * 64 + i * 4);
    } else if constexpr (EB == 2) {
      const int k = 8 * g + (i >> 2);
      const int byte = first * 2 + (i & 3) * 8;
      return k * BN * 2 + ((((byte >> 4) ^ swz_k(k)) << 4) | (byte & 15));
    } else {
      const int k = 4 * g;
      const int byte = (first + i) * 4;
      return k * BN * 4 + ((((byte >> 4) ^ swz_k(k)) << 4) | (byte & 15));
    }
  }
  template <Operand OP>
  __device__ __forceinline__ static uint4 frag(const char* st, int lane0, int sub) {
    if constexpr (OP == kPanelK || OP == kSteps) {
      return *reinterpret_cast<const uint4*>(st + lane0 + sub * M_STEP * 64);
    } else if constexpr (EB == 2) {
      // kRows: 16 columns are 32 bytes, and column blocks differ by an exclusive
      // or in the address (the swizzle stays within 256 bytes)
      const char* p = OP == kPanelR ? st + (lane0 ^ ((sub & 1) << 5)) + (sub >> 1) * 2048
                                    : st + (lane0 ^ ((sub & 7) << 5)) + (sub >> 3) * 256;
      const uint2 a = read_tr16(p), b = read_tr16(p + 4 * (OP == kPanelR ? 64 : BN * 2));
      return uint4{a.x, a.y, b.x, b.y};
    } else {
      const char* p = OP == kPanelR ? st + lane0 + sub * 1024 : st + (lane0 ^ ((sub & 3) << 6)) + (sub >> 2) * 256;
      constexpr int NEXT = OP == kPanelR ? 64 : BN;  // elements to the lane group's next K row
      const unsigned* q = reinterpret_cast<const unsigned*>(p);
      return uint4{q[0], q[NEXT], q[2 * NEXT], q[3 * NEXT]};
    }
  }

  static __device__ __forceinline__ int m_first(int wave) { return DEALT ? (wave / WN) * 16 : (wave / WN) * TM; }
  // Row (or column) of the tile that accumulator block mi of this lane holds.
  static __device__ __forceinline__ int m_of(int wave, int mi, int lane) {
    return m_first(wave) + mi * M_STEP + (lane & 15);
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
    unsigned mask;    // MASKED: which of their K rows are read, a bit each; the others are zeros
    int stores;       // steps left for which this wavefront's ST stores of the unit before may be in flight
    int moff[LM], noff[LN];
    uint4 nf[NI], mf[MI];
    f32x4_t acc[MI][NI];

    __device__ __forceinline__ Runner(Job& job_, const char* ring_, unsigned ring_at_, int first, int stride_, int end_,
                                      int lane_, int wave_)
        : job(job_), ring(ring_), ring_at(ring_at_), stride(stride_), end(end_), lane(lane_), wave(wave_),
          ml(frag_lane<MOP>(lane_, m_first(wave_))), nl(MBYTES + frag_lane<NOP>(lane_, (wave_ % WN) * TN)), L(first), lj(0), lpad(0), ls(0), cs(0), stores(0) {}

    // A unit takes at least S steps (empty ones behind its own), so the loads,
    // S - 1 steps ahead, are never more than one unit ahead.
    __device__ __forceinline__ static int padded(const Info& t) { return t.steps > S ? t.steps : S; }
    __device__ __forceinline__ void open() {
      const bool in = L < end;  // else past the last unit: empty loads from here on
      if (in) {
        lt = job.decode(L);
        if constexpr (NOP == kRows) {
#pragma unroll
          for (int i = 0; i < LN; ++i) noff[i] = job.rows_offset(lt, nq(wave, i), lane);
        }
      }
      if constexpr (Job::MASKED) mask = job.mask(0);
      // (selects, not an else branch: stores of two branches merged into one
      // through a pointer would keep the state in scratch memory)
      lt.steps = in ? lt.steps : 0;
      lpad = in ? padded(lt) : 0x7fffffff;
      lj = 0;
      ld = job.first(lt);
    }
    // Where the loads after the next ones lie: worked out without a branch
    // (`turn`, behind it, opens the next unit), so that it fits between MFMAs.
    __device__ __forceinline__ void advance() {
      ls = ls == S - 1 ? 0 : ls + 1;
      ++lj;
      job.next(lt, lj, ld);
      if constexpr (Job::MASKED) mask = job.mask(lj);
    }
    __device__ __forceinline__ void turn() {
      if (lj == lpad) {
        L += stride;
        open();
      }
    }
    // Load i of this wavefront of an operand in panels with K along the rows: 16
    // of the step's rows of one panel, nothing behind the last row or panel.
    __device__ __forceinline__ u32x4_t panel_desc(const char* base, int bytes, int i, int panels) const {
      const int q = wave + i * NW, panel = q / PL, half = q % PL * 1024;
      const int n = panel < panels ? min(max(bytes - half, 0), 1024) : 0;
      return descriptor(base + panel * lt.panel + half, n);
    }
    // Issues the next loads and, from i = 0 on, an equal share of the work `between`
    // after each of them.
    template <class Between>
    __device__ __forceinline__ void feed(Between&& between) {
      const u32x4_t m = descriptor(ld.m, ld.mbytes), n = descriptor(ld.n, ld.nbytes);
      const unsigned at = ring_at + ls * STAGE;
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const int in = i < LM ? 0 : i - LM;
        if (i < LM)
          load_lds(m, moff[i < LM ? i : 0], at + mq(wave, i) * 1024);
        else
          load_lds(NOP == kPanelR ? panel_desc(ld.n, ld.nbytes, in, lt.npanels) : n,
                   !Job::MASKED || (mask >> k_row(nq(wave, in), lane) & 1) != 0 ? noff[in] : kOutside,
                   at + MBYTES + nq(wave, in) * 1024);
        between(i);
      }
    }
    __device__ __forceinline__ static void barrier() {
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
      __builtin_amdgcn_sched_barrier(0);
    }
    // The next loads and this step's operands.  The loads go through the vector
    // memory path (64 bytes a cycle and compute unit), the operands through LDS:
    // issued in turn, they overlap.
    template <int MB>
    __device__ __forceinline__ void move() {
      const char* st = ring + cs * STAGE;
      constexpr int FR = NI + MB, PER = (FR + NL - 1) / NL;  // operands behind each load
      feed([&](int i) {
#pragma unroll
        for (int f = i * PER; f < (i + 1) * PER && f < FR; ++f) {
          if (f < NI)
            nf[f < NI ? f : 0] = frag<NOP>(st, nl, f);
          else
            mf[f < NI ? 0 : f - NI] = frag<MOP>(st, ml, f - NI);
        }
      });
      cs = cs == S - 1 ? 0 : cs + 1;
    }
    // SWAP: the other operand is the MFMA's first, and a lane ends with 4
    // consecutive m of one n.
    template <int MB, bool SWAP>
    __device__ __forceinline__ void multiply() {
#pragma unroll
      for (int mi = 0; mi < MB; ++mi)
#pragma unroll
        for (int ni = 0; ni < NI; ++ni)
          acc[mi][ni] = SWAP ? mma16<Tr>(mf[mi], nf[ni], acc[mi][ni]) : mma16<Tr>(nf[ni], mf[mi], acc[mi][ni]);
    }

    // One step.  This wavefront's loads of the step have landed (those of the
    // S - 2 after it may be in flight); after the barrier everyone's have, and
    // everyone is done with the stage of the step before, which takes the step
    // S - 1 ahead.
    template <int MB, bool SWAP>
    __device__ __forceinline__ void step() {
      wait_step();
      barrier();
      move<MB>();
      advance();
      multiply<MB, SWAP>();
      turn();
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
    template <int MB, bool SWAP>
    __device__ __forceinline__ void step_pp() {
      move<MB>();
      wait_step();
      wait_lds();
      barrier();
      advance();
      multiply<MB, SWAP>();
#pragma unroll
      for (int i = 0; i < MB * NI; ++i) {  // one MFMA, then up to two scalar instructions in its shadow
        __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x4, 2, 0);
      }
      turn();
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

    // The steps of a unit, for its first MB blocks of 16 rows per wavefront, and
    // the empty ones behind them, which keep the ring going and nothing else.
    template <int MB, bool SWAP>
    __device__ __forceinline__ void steps(int n) {
#pragma unroll 1
      for (int j = 0; j < n; ++j) {
        if constexpr (PP)
          step_pp<MB, SWAP>();
        else
          step<MB, SWAP>();
      }
    }
    __device__ __forceinline__ void empty_steps(int n) {
#pragma unroll 1
      for (int j = 0; j < n; ++j) {
        if constexpr (!PP) {
          wait_step();
          barrier();
        }
        feed([](int) {});
        if constexpr (PP) {
          wait_step();
          barrier();
        }
        cs = cs == S - 1 ? 0 : cs + 1;
        advance();
        turn();
        if constexpr (PP) barrier();
      }
    }

    __device__ __forceinline__ bool done() const { return L >= end; }

    __device__ __forceinline__ void run() {
      if (L >= end) return;
#pragma unroll
      for (int i = 0; i < LM; ++i) moff[i] = panel_offset<MOP>(mq(wave, i), lane);
#pragma unroll
      for (int i = 0; i < LN; ++i) noff[i] = NOP == kPanelR ? panel_offset<NOP>(0, lane) : 0;
      open();
      ct = lt;
#pragma unroll 1
      for (int u = 0; u < S - 1; ++u) {  // within the first unit's padded steps
        feed([](int) {});
        advance();
        turn();
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
        if constexpr (MOP == kSteps) {
          if (ct.swap)
            steps<MI, true>(ct.steps);
          else
            steps<MI, false>(ct.steps);
        } else {
          // a tile of at most half the rows multiplies half the blocks
          if (MI % 2 == 0 && ct.rows <= BM / 2)
            steps<(MI + 1) / 2, false>(ct.steps);
          else
            steps<MI, false>(ct.steps);
        }
        empty_steps(padded(ct) - ct.steps);
        // both halves store at the same time: in turn, each would wait for the
        // other's stores.  (Kept in registers and stored a few at a time in the
        // next unit's steps, weight gradients took no less: 3128 against 3071 us
        // with 8192 rows at d = 4096, F = 14336, 1094 against 1072 with 1024.)
        if (PP && !second) barrier();
        stores = job.store(ct, wave, lane, acc) ? S - 2 : 0;
        if (done()) break;
        if (PP && second) barrier();
        ct = lt;  // the next unit: the loads are S - 1 steps ahead, less than a unit
      }
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
  Divisor own[256];  // tiles of BM rows of expert i
  int tiles[257];    // those in front of it
};

__device__ __forceinline__ int quotient(int n, Divisor by) {
  const unsigned q = __umulhi((unsigned)n, by.m);
  return (int)(q + ((unsigned)n - q * by.d >= by.d ? 1u : 0u));
}

__device__ __forceinline__ int tiles_of(int n, int BM) { return (n + BM - 1) / BM; }

// Filled by a whole workgroup of NTH >= 256 threads.
template <int BM>
__device__ __forceinline__ void fill_table(const GradRows& p, ExpertTable& t) {
  __shared__ int part[4];
  const int i = threadIdx.x, lane = i & 63;
  int n = 0;
  if (i < p.E) {
    const ExpertRows r = expert_rows(p, i);
    t.rows[i] = r;
    n = tiles_of(r.n0, BM) + tiles_of(r.n1, BM);
    t.own[i] = Divisor{(unsigned)n, 0xffffffffu / (unsigned)max(n, 1)};
  }
  int inc = n;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(inc, o);
    if (lane >= o) inc += v;
  }
  if (i < 256 && lane == 63) part[i >> 6] = inc;
  __syncthreads();
  if (i < 256) {
    for (int w = 0; w < (i >> 6); ++w) inc += part[w];
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

// The weight gradients' units, whose cost is their expert's rows: dealt to the XCDs in
// runs of one unit for each of their workgroups, so that every XCD takes part in
// every expert and units at work at a time in one L2 are still neighbours.  With a
// contiguous eighth for each XCD, as above (with 8 experts just one of them), the hot
// expert's XCD set the pace.  Contiguous against dealt, us of the launch:
//  * Zipf 1.2 routing, the Mixtral shape with 1024 rows 1207 against 802, with 8192 6300
//    against 2881; 64 experts of d = 3584, F = 2560 with 32768 rows 3928 against 2310 (Zipf 2.0:
//    4085 against 2403); fp32, 8 experts of d = 1024, F = 4096 with 2048 rows 1347 against 584;
//  * uniform routing, the Mixtral shape with 128, 512, 1024, 4096, 8192 rows 617, 767, 887,
//    1700, 2785 against 614, 726, 875, 1666, 2795; 64 experts of d = 3584, F = 2560 with 4096 and
//    32768 rows 903 and 2151 against 880 and 2218; fp32 as above 573 against 575.
__device__ __forceinline__ Units dealt_units(int total) {
  const int per = (int)gridDim.x >> 3;
  return Units{((int)blockIdx.x & 7) * per + ((int)blockIdx.x >> 3), (int)gridDim.x, total};
}

// out tile = act rows x weights (DH: with the SwiGLU's gradient in the epilogue).
// A unit's steps go over K, a1 x b1 behind a0 x b0 into the same accumulators.
// Out: type of the results (a choice at run time cost the main loop 8 %, in
// registers).
template <class Tr, class T, bool DH, class Out>
struct DgradJob {
  static constexpr int EB = T::EB;
  static constexpr bool MASKED = false;
  struct Info {
    int steps, row0, rows, nbase, e;
    const char *a0, *a1, *b0, *b1;  // operands of the tile's rows and expert
    size_t panel;                   // bytes of a panel of activations
    int npanels;
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
    const Divisor own{(unsigned)__builtin_amdgcn_readfirstlane((int)tab.own[e].d),
                      (unsigned)__builtin_amdgcn_readfirstlane((int)tab.own[e].m)};
    const int t0 = tiles_of(n0, T::BM);
    const int local = L - before * NT;
    const int nt = quotient(local, own);
    const int ti = local - nt * (int)own.d;
    const int n = ti < t0 ? n0 : n1, first = (ti < t0 ? ti : ti - t0) * T::BM;
    Info i;
    i.e = e;
    i.row0 = (ti < t0 ? r0 : r1) + first;
    i.rows = min(T::BM, n - first);
    i.nbase = nt * T::BN;
    i.steps = per * (p.a1 != nullptr ? 2 : 1);
    const size_t act = (size_t)i.row0 * 64, mat = (size_t)e * p.K * p.N * EB;
    i.panel = p.panel;
    i.a0 = static_cast<const char*>(p.a0) + act;
    i.b0 = static_cast<const char*>(p.b0) + mat;
    i.a1 = DH ? i.a0 : static_cast<const char*>(p.a1) + act;
    i.b1 = DH ? i.b0 : static_cast<const char*>(p.b1) + mat;
    return i;
  }
  __device__ __forceinline__ int rows_offset(const Info& t, int q, int lane) const {
    return T::rows_offset(q, lane, t.nbase, p.N, p.N * EB, p.blocked16);
  }
  __device__ __forceinline__ Step first(const Info& t) const {
    return t.steps > 0 ? Step{t.a0, t.b0, t.rows * 64, T::KS * p.N * EB} : Step{t.a0, t.b0, 0, 0};
  }
  // Step j: a panel on in the activations, KS rows on in the weights.
  __device__ __forceinline__ void next(const Info& t, int j, Step& s) const {
    const int nrows = T::KS * p.N * EB;
    const bool turn = !DH && j == per, in = j < t.steps;
    s.m = turn ? t.a1 : s.m + t.panel;
    s.n = turn ? t.b1 : s.n + nrows;
    s.mbytes = in ? t.rows * 64 : 0;
    s.nbytes = in ? nrows : 0;
  }
  // The saved projections of one row's NI blocks of 16 columns.
  struct Saved {
    unsigned g[4], u[4], gx, ux;  // NI words of four codes each; the blocks' exponents, one byte each
    float w;
  };
  // With four blocks a lane reads the 16 codes of block g = lane / 16 of its row;
  // `turn` then deals out the words, so that it holds its four columns of every
  // block (a word at a time, the reads of the scattered rows took 0.8 ms of the
  // 1.7 of 8192 rows at d = 4096, F = 14336).  Rows past the tile's last read zeros.
  __device__ __forceinline__ void read_saved(const Info& t, int m, int n0, int lane, Saved& s) const {
    const size_t o = (size_t)t.row0 * p.N;
    const char *g8 = reinterpret_cast<const char*>(p.g8) + o, *u8 = reinterpret_cast<const char*>(p.u8) + o;
    const char *gx = reinterpret_cast<const char*>(p.gx) + (o >> 4), *ux = reinterpret_cast<const char*>(p.ux) + (o >> 4);
    const int row = m * p.N + n0, bytes = t.rows * p.N, g = lane >> 4;
    if constexpr (T::NI == 4) {
      const uint4 a = buf_load16(g8, bytes, row + g * 16), b = buf_load16(u8, bytes, row + g * 16);
      s.g[0] = a.x, s.g[1] = a.y, s.g[2] = a.z, s.g[3] = a.w;
      s.u[0] = b.x, s.u[1] = b.y, s.u[2] = b.z, s.u[3] = b.w;
    } else {
#pragma unroll
      for (int ni = 0; ni < T::NI; ++ni) {
        s.g[ni] = buf_load4(g8, bytes, row + ni * 16 + g * 4);
        s.u[ni] = buf_load4(u8, bytes, row + ni * 16 + g * 4);
      }
    }
    // exponents of four blocks, of which two are this wavefront's with NI = 2
    static_assert(T::NI == 4 || T::NI == 2, "exponents of a wavefront's columns in one load");
    const int xb = T::NI == 2 ? (n0 >> 4) & 2 : 0;
    s.gx = buf_load4(gx, bytes >> 4, (row >> 4) - xb);
    s.ux = buf_load4(ux, bytes >> 4, (row >> 4) - xb);
    s.w = __uint_as_float(buf_load4(reinterpret_cast<const char*>(p.wrow + t.row0), t.rows * 4, m * 4));
  }
  __device__ __forceinline__ void turn(Saved& s, int n0) const {
    if constexpr (T::NI == 4) {
      transpose4(s.g);
      transpose4(s.u);
    } else {
      const int xb = (n0 >> 4) & 2;
      s.gx >>= 8 * xb;
      s.ux >>= 8 * xb;
    }
  }
  __device__ __forceinline__ bool store(const Info& t, int wave, int lane, f32x4_t (&acc)[T::MI][T::NI]) const {
    // a wavefront's columns are all inside the matrix or all behind it (both
    // are multiples of 64, or of 32 with tiles of 128 columns)
    const int n0 = t.nbase + (wave % T::WN) * T::TN;
    if (n0 >= p.N) return false;
    const int m0 = T::m_first(wave);
    if constexpr (!DH) {
      constexpr int OB = sizeof(typename Out::T);
      const int ld = p.N * OB;
      const OutTile<Out> out =
          OutTile<Out>::matrix(static_cast<const char*>(p.out) + (size_t)t.row0 * ld, t.rows, ld, m0, n0, lane, 0,
                               T::TN * OB >= 128);
#pragma unroll
      for (int mi = 0; mi < T::MI; ++mi) {
        float v[T::NI][4];
#pragma unroll
        for (int ni = 0; ni < T::NI; ++ni)
#pragma unroll
          for (int r = 0; r < 4; ++r) v[ni][r] = acc[mi][ni][r];
        out.template put<T::NI>(mi * T::M_STEP, v);
      }
      return true;
    } else {
      const size_t o = (size_t)(n0 / T::KS) * p.panel + (size_t)t.row0 * 64;
      const OutTile<Tr> odg = OutTile<Tr>::panels(static_cast<const char*>(p.dg) + o, p.panel, t.rows, m0, lane);
      const OutTile<Tr> odu = OutTile<Tr>::panels(static_cast<const char*>(p.du) + o, p.panel, t.rows, m0, lane);
      const OutTile<Tr> ohw = OutTile<Tr>::panels(static_cast<const char*>(p.hw) + o, p.panel,
                                                  p.hw != nullptr ? t.rows : 0, m0, lane);
      // The codes of the next AHEAD blocks are on their way while one's are
      // worked.  No branch from here on: the compiler's waits count the loads and
      // stores in flight, and where a branch left it in doubt it waited for the
      // stores of the block before (1.7 ms instead of 0.9 in all).
      constexpr int AHEAD = T::MI < 3 ? T::MI - 1 : 2;
      Saved s[AHEAD + 1];
#pragma unroll
      for (int mi = 0; mi < AHEAD; ++mi) read_saved(t, T::m_of(wave, mi, lane), n0, lane, s[mi]);
      char* dots = reinterpret_cast<char*>(p.dot + (size_t)t.row0 * p.dot_ld);
      const int dots_bytes = t.rows * p.dot_ld * 4;
#pragma unroll
      for (int mi = 0; mi < T::MI; ++mi) {
        const int m = T::m_of(wave, mi, lane);
        if (mi + AHEAD < T::MI)
          read_saved(t, T::m_of(wave, mi + AHEAD, lane), n0, lane, s[(mi + AHEAD) % (AHEAD + 1)]);
        Saved& q = s[mi % (AHEAD + 1)];
        turn(q, n0);
        float dg[T::NI][4], du[T::NI][4], hw[T::NI][4], dot = 0.f;
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
        odg.template put<T::NI>(mi * T::M_STEP, dg);
        odu.template put<T::NI>(mi * T::M_STEP, du);
        ohw.template put<T::NI>(mi * T::M_STEP, hw);
        // the wavefront's columns of <D, h>: the four lanes of a row, then one
        // partial sum per wavefront column, added in order by a later step
        dot += __shfl_xor(dot, 16);
        dot += __shfl_xor(dot, 32);
        buf_store4(dots, dots_bytes, lane < 16 ? (m * p.dot_ld + n0 / T::TN) * 4 : kOutside, __float_as_uint(dot));
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

template <class Tr, class T, bool DH, class Out>
__global__ __launch_bounds__(T::NTH) void dgrad_kernel(DgradArgs p) {
  MOE_GRAD_RING;
  __shared__ ExpertTable tab;
  if constexpr (!DH) {
    // the routing weights' gradients, from the launch before: each wavefront sums
    // some entries' rows of `dot`, lane i the columns i, i + 64, .. in order
    for (int f = blockIdx.x * T::NW + wave; f < p.entries; f += gridDim.x * T::NW) {
      const int row = p.row_of[f];
      float s = 0.f;
      if (row >= 0)
        for (int i = lane; i < p.dot_ld; i += 64) s += p.dot[(size_t)row * p.dot_ld + i];
      s = wave_sum(s);
      if (lane == 0) p.dw[f] = s;
    }
  }
  fill_table<T::BM>(p.rows, tab);
  DgradJob<Tr, T, DH, Out> job(p, tab);
  const Units u = my_units(job.units());
  typename T::template Runner<DgradJob<Tr, T, DH, Out>>(job, ring, ring_at, u.first, u.stride, u.end, lane, wave).run();
}

// ---- weight gradients ---------------------------------------------------------

// Rows of x and dout in expert order for the GEMMs, and the routing weight of
// each row.  A workgroup takes one K step of the weight gradients (KS rows of
// one run of an expert) and a share of the columns.  The steps of x and dout are
// turned, [step][d][64 bytes], with zeros behind a run's last row: through LDS
// in the layout and with the reads of an operand in panels, so that what a
// lane reads there are the 16 bytes it writes.  dout goes to panels as well, for
// the first data gradient.  x_steps and dout_steps may be null: not wanted.
// Bound by memory: 54 us for 8192 rows of 4096 bf16 (336 MB read and written,
// 6.2 TB/s); by latency for the smallest, 4 us.
template <class Tr, class T>
__global__ __launch_bounds__(256) void gather_backward_kernel(GatherArgs p) {
  constexpr int KS = T::KS, EB = T::EB, LD = KS / 16;  // 16-byte loads of 256 columns' bytes per thread and tensor
  __shared__ __attribute__((aligned(1024))) char st[2][4 * KS * 64];
  __shared__ ExpertTable tab;
  fill_table<KS>(p.rows, tab);
  const int step = blockIdx.x;
  if (step >= tab.tiles[256]) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int e = 0;
  for (int b = 0; b < p.rows.E; b += 64)
    e += __popcll(__ballot(b + lane < p.rows.E && tab.tiles[b + lane + 1] <= step));
  const ExpertRows x = tab.rows[e];
  const int j = step - tab.tiles[e], t0 = tiles_of(x.n0, KS);
  const int first = (j < t0 ? j : j - t0) * KS, row0 = (j < t0 ? x.r0 : x.r1) + first;
  const int n = min(KS, (j < t0 ? x.n0 : x.n1) - first);
  if (blockIdx.y == 0 && (int)threadIdx.x < n) {
    const int r = row0 + threadIdx.x, t = p.token_of[r];
    for (int i = 0; i < p.k; ++i)
      if (t >= 0 && p.row_of[(size_t)t * p.k + i] == r) p.wrow[r] = p.topk_w[(size_t)t * p.k + i];
  }
  const int row_bytes = p.d * EB, panels = row_bytes / 64;
  const int c0 = (int)((int64_t)((panels + 3) / 4) * blockIdx.y / gridDim.y) * 4;
  const int c1 = min(panels, (int)((int64_t)((panels + 3) / 4) * (blockIdx.y + 1) / gridDim.y) * 4);
  const int c = threadIdx.x & 15;  // 16 lanes read 256 bytes of a row
  int tok[LD];
#pragma unroll
  for (int u = 0; u < LD; ++u) {
    const int r = u * 16 + (threadIdx.x >> 4);
    tok[u] = r < n ? p.token_of[row0 + r] : -1;
  }
  const int fl = T::template frag_lane<kPanelR>(lane, 0);
  for (int q = c0; q < c1; q += 4) {
    const int at = q + (c >> 2);  // this thread's panel
#pragma unroll
    for (int u = 0; u < LD; ++u) {
      const int r = u * 16 + (threadIdx.x >> 4);
      uint4 a = make_uint4(0, 0, 0, 0), b = a;
      if (tok[u] >= 0 && at < c1) {
        const size_t o = (size_t)tok[u] * row_bytes + (size_t)q * 64 + c * 16;
        if (p.x_steps != nullptr) a = *reinterpret_cast<const uint4*>(static_cast<const char*>(p.x) + o);
        b = *reinterpret_cast<const uint4*>(static_cast<const char*>(p.dout) + o);
        *reinterpret_cast<uint4*>(p.dout_panels + at * p.panel + (size_t)(row0 + r) * 64 + (c & 3) * 16) = b;
      }
      const int slot = EB == 2 ? r * 64 + (((c & 3) ^ ((r >> 2) & 2)) << 4)
                               : ((r >> 2) | (r & 3) << 2) * 64 + ((c & 3) << 4);
      *reinterpret_cast<uint4*>(st[0] + (c >> 2) * KS * 64 + slot) = a;
      *reinterpret_cast<uint4*>(st[1] + (c >> 2) * KS * 64 + slot) = b;
    }
    __syncthreads();
    if (q + wave < c1) {  // a wavefront turns one panel
#pragma unroll
      for (int s = 0; s < 2 / (EB / 2); ++s) {
        const int i = lane & 15, g = lane >> 4;
        const size_t o = ((size_t)step * p.d + (q + wave) * KS + s * 16 + i) * 64 + g * 16;
        if (p.x_steps != nullptr)
          *reinterpret_cast<uint4*>(p.x_steps + o) = T::template frag<kPanelR>(st[0] + wave * KS * 64, fl, s);
        if (p.dout_steps != nullptr)
          *reinterpret_cast<uint4*>(p.dout_steps + o) = T::template frag<kPanelR>(st[1] + wave * KS * 64, fl, s);
      }
    }
    __syncthreads();
  }
}

// Sums over the rows r of expert e, up to three in one launch: out[m][n] =
// sum P[r][m] Q[r][n] with m over d and n over F, or (swap) out[n][m] the same
// value.  P in steps, Q in panels.  An expert without rows gets zeros.
template <class Tr, class T>
struct WgradJob {
  static constexpr int EB = T::EB;
  static constexpr bool MASKED = false;
  struct Info {
    int steps, rows, steps0, e, w, mbase, nbase, swap;
    int n0, n1;
    size_t panel;
    int npanels;               // panels of Q from the tile's first on
    const char *p0, *q0, *q1;  // the first step of P, the first rows of Q's either run
  };
  const WgradArgs& p;
  const ExpertTable& tab;  // of KS rows: tiles[e] is expert e's first step
  __device__ __forceinline__ WgradJob(const WgradArgs& p_, const ExpertTable& t) : p(p_), tab(t) {}

  __device__ __forceinline__ Info decode(int L) const {
    Info i;
    i.e = quotient(L, p.per_e);
    L -= i.e * (int)p.per_e.d;
    i.w = (p.n > 1 && L >= p.prod[1].first ? 1 : 0) + (p.n > 2 && L >= p.prod[2].first ? 1 : 0);
    const WgradProduct& w = p.prod[i.w];
    L -= w.first;
    // bands of kBand tiles of out's rows by all tiles of its columns: the tiles that
    // an XCD works at a time share both operands in L2 and store long runs of
    // each row (bands of 1, 2, 4, 8 tiles, the Mixtral shape: 599, 595, 609, 615 us
    // with 16 rows in all, 2894, 2884, 2886, 2920 with 8192; 64 experts of d = 3584,
    // F = 2560 with 32768 rows 2300, 2297, 2288, 2301)
    const int band = quotient(L, w.band), in = L - band * (int)w.band.d;
    const bool whole = (band + 1) * kBand <= w.RT;
    const int ct = whole ? in / kBand : quotient(in, w.last);
    const int rt = band * kBand + in - ct * (whole ? kBand : (int)w.last.d);
    i.swap = w.swap;
    i.mbase = (w.swap ? ct : rt) * T::BM;
    i.nbase = (w.swap ? rt : ct) * T::BN;
    i.rows = min(T::BM, p.M - i.mbase);
    const int r0 = __builtin_amdgcn_readfirstlane(tab.rows[i.e].r0);
    i.n0 = __builtin_amdgcn_readfirstlane(tab.rows[i.e].n0);
    const int r1 = __builtin_amdgcn_readfirstlane(tab.rows[i.e].r1);
    i.n1 = __builtin_amdgcn_readfirstlane(tab.rows[i.e].n1);
    const int step = __builtin_amdgcn_readfirstlane(tab.tiles[i.e]);
    i.panel = p.panel;
    i.npanels = (p.N - i.nbase) / T::KS;  // (N is a multiple of 64)
    i.p0 = static_cast<const char*>(w.P) + ((size_t)step * p.M + i.mbase) * 64;
    const char* Q = static_cast<const char*>(w.Q) + (size_t)(i.nbase / T::KS) * p.panel;
    i.q0 = Q + (size_t)r0 * 64;
    i.q1 = Q + (size_t)r1 * 64;
    i.steps0 = (i.n0 + T::KS - 1) / T::KS;
    i.steps = i.steps0 + (i.n1 + T::KS - 1) / T::KS;
    return i;
  }
  __device__ __forceinline__ Step first(const Info& t) const {
    const bool in = t.steps > 0;
    return Step{t.p0, t.n0 > 0 ? t.q0 : t.q1, in ? t.rows * 64 : 0,
                in ? min(T::KS, t.n0 > 0 ? t.n0 : t.n1) * 64 : 0};
  }
  // Step j: KS rows on; the rows behind the capacity follow those in front of it.
  __device__ __forceinline__ void next(const Info& t, int j, Step& s) const {
    const bool second = j >= t.steps0, in = j < t.steps;
    s.m += (size_t)p.M * 64;
    s.n = j == t.steps0 ? t.q1 : s.n + T::KS * 64;
    const int left = max(0, min(T::KS, second ? t.n1 - (j - t.steps0) * T::KS : t.n0 - j * T::KS));
    s.mbytes = in ? t.rows * 64 : 0;
    s.nbytes = in ? left * 64 : 0;
  }
  __device__ __forceinline__ bool store(const Info& t, int wave, int lane, f32x4_t (&acc)[T::MI][T::NI]) const {
    const int M = p.M, N = p.N, m0 = T::m_first(wave), n0 = (wave % T::WN) * T::TN;
    const char* base = static_cast<const char*>(p.prod[t.w].out) + (size_t)t.e * M * N * EB;
    // M and N are multiples of 64, so whole groups of 16 rows are in or out, and so
    // are the columns of a wavefront (64 or 32) or of a part of it (64)
    if (!t.swap) {
      if (t.nbase + n0 >= N) return false;
      const int ld = N * EB;
      const OutTile<Tr> out = OutTile<Tr>::matrix(base + (size_t)t.mbase * ld, t.rows, ld, m0, t.nbase + n0, lane,
                                                  p.blocked16, T::TN * EB >= 128);
#pragma unroll
      for (int mi = 0; mi < T::MI; ++mi) {
        float v[T::NI][4];
#pragma unroll
        for (int ni = 0; ni < T::NI; ++ni)
#pragma unroll
          for (int r = 0; r < 4; ++r) v[ni][r] = acc[mi][ni][r];
        out.template put<T::NI>(mi * 16, v);
      }
      return true;
    }
    constexpr int PART = T::MI < 4 ? T::MI : 4, PARTS = T::MI / PART;  // blocks of 16 columns in a part
    const int ld = M * EB, rows = min(T::BN, N - t.nbase);
    OutTile<Tr> out[PARTS];
#pragma unroll
    for (int h = 0; h < PARTS; ++h) {
      const int col = t.mbase + m0 + h * PART * 16;
      out[h] = OutTile<Tr>::matrix(base + (size_t)t.nbase * ld, col < M ? rows : 0, ld, n0, col, lane, p.blocked16,
                                   PART * 16 * EB >= 128);
    }
#pragma unroll
    for (int ni = 0; ni < T::NI; ++ni)
#pragma unroll
      for (int h = 0; h < PARTS; ++h) {
        float v[PART][4];
#pragma unroll
        for (int mi = 0; mi < PART; ++mi)
#pragma unroll
          for (int r = 0; r < 4; ++r) v[mi][r] = acc[h * PART + mi][ni][r];
        out[h].template put<PART>(ni * 16, v);
      }
    return true;
  }
};

template <class Tr, class T>
__global__ __launch_bounds__(T::NTH) void wgrad_kernel(WgradArgs p) {
  MOE_GRAD_RING;
  __shared__ ExpertTable tab;
  fill_table<T::KS>(p.rows, tab);
  WgradJob<Tr, T> job(p, tab);
  const Units u = dealt_units(p.units);
  typename T::template Runner<WgradJob<Tr, T>>(job, ring, ring_at, u.first, u.stride, u.end, lane, wave).run();
}

// ---- router weight gradient ---------------------------------------------------

// part[z][e][i] = sum over tokens t of range z of dz[e][t] x[t][i] (fp32 partial
// sums).  dz is dense with zeros where expert e did not take token t, laid out
// by K step: [step][E][64 bytes].  bf16 carries it as two terms (high and low
// part), which keeps 16 bits of its significand.  A NaN or an infinity in x of a
// token with experts reaches all of them, the zeros being multiplied too.  One
// tile per workgroup, over enough token ranges for two on each compute unit: 14 us
// for 4096 tokens of 2048 bf16 and 64 experts, most of it the latency of a
// range's 8 to 16 steps.
template <class Tr, class T>
struct RouteJob {
  static constexpr int EB = T::EB;
  static constexpr bool MASKED = true;
  struct Info {
    int steps, rows;
    size_t panel;
    int npanels;
  };
  const RouteWgradArgs& p;
  const int nbase, mbase, rows, j0, per;
  __device__ __forceinline__ explicit RouteJob(const RouteWgradArgs& p_)
      : p(p_), nbase(blockIdx.x * T::BN), mbase(blockIdx.y * T::BM), rows(min(T::BM, p_.E - mbase)),
        j0(min((p_.T + T::KS - 1) / T::KS, (int)blockIdx.z * p_.steps)),
        per(min((p_.T + T::KS - 1) / T::KS - j0, p_.steps)) {}
  __device__ __forceinline__ Info decode(int) const { return Info{per * (p.dz_lo != nullptr ? 2 : 1), rows, 0, 0}; }
  __device__ __forceinline__ int rows_offset(const Info&, int q, int lane) const {
    return T::rows_offset(q, lane, nbase, p.d, p.d * EB, 0);
  }
  // Tokens of step j that any expert took.  The rows of x of the others, which
  // may hold anything, are not read: zero times a NaN there would reach every
  // expert.  (A scalar load: the wait for a vector load would drain the ring.)
  __device__ __forceinline__ unsigned mask(int j) const {
#ifdef __HIP_DEVICE_COMPILE__
    const bool second = j >= per;
    const int q = j < per * (p.dz_lo != nullptr ? 2 : 1) ? j0 + (second ? j - per : j) : 0;
    return ((const __attribute__((address_space(4))) unsigned*)(uintptr_t)p.taken)[q];
#else
    return 0;
#endif
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
  static_assert(T::OCC * (T::S * T::STAGE + sizeof(ExpertTable) + 4 * sizeof(int)) <= 160 * 1024,
                "ring and table of the workgroups that share a compute unit");
  const long long most = (long long)kComputeUnits * T::OCC;
  return (unsigned)((units < most ? (units + 7) / 8 * 8 : most));
}

template <class Tr, class T, bool DH>
hipError_t launch_dgrad_cfg(const DgradArgs& a, long long max_tiles, hipStream_t stream) {
  const long long units = max_tiles * ((a.N + T::BN - 1) / T::BN);
  if (units == 0) return hipSuccess;
  if (units > 0x7fffff00LL) return hipErrorInvalidValue;
  if constexpr (!DH && sizeof(typename Tr::T) == 2) {
    if (a.out_f32 != 0) {
      hipLaunchKernelGGL((dgrad_kernel<Tr, T, DH, TF32>), dim3(grid_of<T>(units)), dim3(T::NTH), 0, stream, a);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((dgrad_kernel<Tr, T, DH, Tr>), dim3(grid_of<T>(units)), dim3(T::NTH), 0, stream, a);
  return hipGetLastError();
}

template <class Tr, class T>
hipError_t launch_wgrad_cfg(WgradArgs a, hipStream_t stream) {
  const long long MT = (a.M + T::BM - 1) / T::BM, NT = (a.N + T::BN - 1) / T::BN;
  // (a unit number plus the grid still fits 32 bits)
  if (kBand * MT * NT > 0x7fff0000LL || a.n * MT * NT * a.rows.E > 0x7fff0000LL) return hipErrorInvalidValue;
  for (int w = 0; w < a.n; ++w) {
    WgradProduct& p = a.prod[w];
    p.first = (int)(w * MT * NT);
    p.RT = (int)(p.swap ? NT : MT);
    p.band = divisor((unsigned)(kBand * (p.swap ? MT : NT)));
    p.last = divisor(p.RT % kBand != 0 ? p.RT % kBand : kBand);
  }
  a.units = (int)(a.n * MT * NT * a.rows.E);
  a.per_e = divisor((unsigned)(a.n * MT * NT));
  if (a.units == 0) return hipSuccess;
  hipLaunchKernelGGL((wgrad_kernel<Tr, T>), dim3(grid_of<T>(a.units)), dim3(T::NTH), 0, stream, a);
  return hipGetLastError();
}

template <class Tr, class T>
hipError_t launch_gather_cfg(const GatherArgs& a, long long max_steps, hipStream_t stream) {
  // about four workgroups for each compute unit, as far as the columns go
  const long long quads = ((long long)a.d * T::EB + 255) / 256;
  const long long shares = std::max(1LL, std::min(quads, 4LL * kComputeUnits / std::max(1LL, max_steps)));
  if (max_steps > 0x7fffffLL) return hipErrorInvalidValue;
  hipLaunchKernelGGL((gather_backward_kernel<Tr, T>), dim3((unsigned)max_steps, (unsigned)shares), dim3(256), 0,
                     stream, a);
  return hipGetLastError();
}

}  // namespace grad
}  // namespace moe
