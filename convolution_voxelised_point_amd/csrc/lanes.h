// Reductions over 2, 4, ... 64 adjacent, aligned lanes, the result in all of them (device
// helpers).  Up to 16 lanes the exchange is part of the instruction that uses it (DPP); a
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
// parts (one alone is off by |d| 2^-24), at half of expf's instructions.  NaN stays.
__device__ __forceinline__ float exp_below(float d) {
  d = d < -1e4f ? -1e4f : d;
  const float hi = d * 1.44269504f, lo = fmaf(d, 1.92596299e-8f, fmaf(d, 1.44269504f, -hi));
  const float e = __builtin_amdgcn_exp2f(hi);
  return fmaf(e, lo * 0.693147181f, e);
}

}  // namespace ts
