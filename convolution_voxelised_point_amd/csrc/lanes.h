// Device helpers of the kernels beside attention.
//
// Reductions over 2, 4, ... 64 adjacent, aligned lanes, the result in all of them.  Up to 16 lanes the exchange is part of the instruction that uses it (DPP); a
// mirror serves as well as an exclusive or, since both sides are uniform by then.
#pragma once

#include "common.h"

namespace ts {

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t x) {
  return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), CTRL, 0xF, 0xF, true));
}

// F(own, other) over `lanes` lanes (the same number in the whole wave).
template <typename F>
__device__ __forceinline__ uint32_t reduce_lanes_u32(uint32_t x, int lanes, F&& f) {
  if (lanes > 1) x = f(x, dpp_u32<0xB1>(x));   // 1 0 3 2
  if (lanes > 2) x = f(x, dpp_u32<0x4E>(x));   // 2 3 0 1
  if (lanes > 4) x = f(x, dpp_u32<0x141>(x));  // 8 lanes mirrored
  if (lanes > 8) x = f(x, dpp_u32<0x140>(x));  // 16 lanes mirrored
  if (lanes > 16) x = f(x, static_cast<uint32_t>(__shfl_xor(static_cast<int>(x), 16)));
  if (lanes > 32) x = f(x, static_cast<uint32_t>(__shfl_xor(static_cast<int>(x), 32)));
  return x;
}
__device__ __forceinline__ float sum_lanes(float x, int lanes) {
  return __builtin_bit_cast(float, reduce_lanes_u32(__builtin_bit_cast(uint32_t, x), lanes, [](uint32_t a, uint32_t b) {
                              return __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b));
                            }));
}
__device__ __forceinline__ uint32_t max_lanes(uint32_t x, int lanes) {
  return reduce_lanes_u32(x, lanes, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
__device__ __forceinline__ uint32_t min_lanes(uint32_t x, int lanes) {
  return reduce_lanes_u32(x, lanes, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}

// exp(d) for d <= 0, off by about 3 * 2^-24 of itself: exp2 of the product with log2(e) in two
// parts (one alone is off by |d| 2^-24), at half of expf's instructions.  NaN stays (in the maximum too).
__device__ __forceinline__ float exp_below(float d) {
  d = __builtin_elementwise_maximum(d, -1e4f);
  const float hi = d * 1.44269504f, lo = fmaf(d, 1.92596299e-8f, fmaf(d, 1.44269504f, -hi));
  const float e = __builtin_amdgcn_exp2f(hi);
  return fmaf(e, lo * 0.693147181f, e);
}

// A store that L2 need not keep, for kernels that stream (passes over changing inputs: the
// rotation of 304,878 x 8 heads forward and back 184 -> 174 us, the combining sum of 304,878 x 128
// 119 -> 109; a kernel that reads the results right afterwards was as fast as after plain stores,
// at 25, 78 and 156 MB).
template <typename V>
__device__ __forceinline__ void store_once(void* p, const V& v) {
  typedef unsigned u4 __attribute__((ext_vector_type(4)));
  typedef unsigned u2 __attribute__((ext_vector_type(2)));
  typedef u4 loose4 __attribute__((aligned(2)));
  typedef u2 loose2 __attribute__((aligned(2)));
  if constexpr (sizeof(V) == 32) {
    struct Two {
      u4 a, b;
    };
    const Two t = __builtin_bit_cast(Two, v);
    __builtin_nontemporal_store(t.a, reinterpret_cast<loose4*>(p));
    __builtin_nontemporal_store(t.b, reinterpret_cast<loose4*>(p) + 1);
  } else if constexpr (sizeof(V) == 16) {
    __builtin_nontemporal_store(__builtin_bit_cast(u4, v), reinterpret_cast<loose4*>(p));
  } else if constexpr (sizeof(V) == 8) {
    __builtin_nontemporal_store(__builtin_bit_cast(u2, v), reinterpret_cast<loose2*>(p));
  } else {
    *reinterpret_cast<V*>(p) = v;
  }
}

}  // namespace ts
