// Device helpers of the operators around the layer and of the layer for a few tokens: 16-byte
// loads, rounding, folds over a wavefront.
#pragma once

#include <type_traits>

#include "device_common.hpp"

namespace moe {

typedef float f32x8_t __attribute__((ext_vector_type(8)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

// 16 bytes in one load.  (As a struct of four words, loads behind a condition came apart
// into four.)
__device__ __forceinline__ uint4 load16(const void* p) {
  return __builtin_bit_cast(uint4, *static_cast<const u32x4*>(p));
}

// EPC fp32 values to one 16-byte chunk: bf16 by the conversion instruction (to
// nearest, ties to even; a NaN stays one), four for eight values where the same in
// integer steps takes some forty.  Dropout of 8192 x 14336 bf16 takes 81 us with it and
// 98 without.
template <class Tr>
__device__ __forceinline__ uint4 round_to(const float* v) {
  if constexpr (Tr::EPC == 8) {
    const f32x8_t f{v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]};
    return __builtin_bit_cast(uint4, __builtin_convertvector(f, bf16x8_t));
  } else {
    return narrow<Tr>(v);
  }
}

// Sum and maximum over a wavefront without LDS: sixteen lanes by exchanges inside the
// registers, then the four sixteens in order.
template <class F>
__device__ __forceinline__ float wave_fold(float v, F&& op) {
  const auto dpp = [&](auto ctrl) {
    return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), decltype(ctrl)::value, 0xf, 0xf, true));
  };
  v = op(v, dpp(std::integral_constant<int, 0xB1>{}));   // quad_perm 1 0 3 2
  v = op(v, dpp(std::integral_constant<int, 0x4E>{}));   // quad_perm 2 3 0 1
  v = op(v, dpp(std::integral_constant<int, 0x141>{}));  // row_half_mirror
  v = op(v, dpp(std::integral_constant<int, 0x140>{}));  // row_mirror
  const auto lane = [&](int l) { return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), l)); };
  return op(op(lane(0), lane(16)), op(lane(32), lane(48)));
}

// Barrier over LDS alone: loads from memory stay in flight across it, and
// nothing waits for stores to be done.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
}

}  // namespace moe
