// Activations in 8 bits (device helpers).  Blocks of 32 consecutive channels
// of a row share a quantum 2^(e - 127) with e = max(floor(log2 max|x|) + 127 -
// 6, 1), kept as the byte e; a value is the integer clamp(rint(x / quantum),
// -127, 127), half to even.  A power-of-two quantum makes both directions
// exact but for that one rounding: x / quantum is a change of exponent, and
// an integer of 7 bits times the quantum is an fp32 and a bf16 number, and an fp16
// number too where x was one.  (Of other values fp16's range may lack some: above
// 65504 they are read as infinity, and bits below 2^-24 are rounded off.)
// A block that holds an infinity or a NaN keeps byte 255 and stands for NaN.
//
// Threads work on 8 consecutive channels; the 4 threads of a block are 4
// adjacent, aligned lanes.
#pragma once

#include "common.h"

namespace ts {

constexpr int kActBlock = TS_ACT8_BLOCK;
constexpr int kActNaN = 255;

typedef _Float16 h16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 b16x8 __attribute__((ext_vector_type(8)));
typedef float fx4 __attribute__((ext_vector_type(4)));
typedef unsigned ux2 __attribute__((ext_vector_type(2)));

// Channels c0..c0+7 of a row of c channels as floats, zeros past c.  vec: rows
// and base allow 16-byte accesses (c a multiple of 8).  Otherwise a whole unit is
// still one access, of the alignment of an element (the hardware takes it), and
// only a row's last, partial unit goes element by element.
template <typename T>
struct __attribute__((aligned(16))) Unit {
  T e[8];
};
template <typename T>
struct __attribute__((packed, aligned(sizeof(T)))) LooseUnit {
  T e[8];
};
template <typename T>
__device__ __forceinline__ void load_unit(const T* row, int c0, int c, bool vec, float (&f)[8]) {
  if (c0 + 8 <= c) {
    Unit<T> v;
    if (vec) {
      v = *reinterpret_cast<const Unit<T>*>(row + c0);
    } else {
      const LooseUnit<T> w = *reinterpret_cast<const LooseUnit<T>*>(row + c0);
#pragma unroll
      for (int e = 0; e < 8; ++e) v.e[e] = w.e[e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = static_cast<float>(v.e[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = c0 + e < c ? static_cast<float>(row[c0 + e]) : 0.f;
  }
}

template <typename T>
__device__ __forceinline__ void store_unit(T* row, int c0, int c, bool vec, const float (&f)[8]) {
  if (c0 + 8 <= c) {
    if (vec) {
      Unit<T> v;
#pragma unroll
      for (int e = 0; e < 8; ++e) v.e[e] = static_cast<T>(f[e]);
      *reinterpret_cast<Unit<T>*>(row + c0) = v;
    } else {
      LooseUnit<T> v;
#pragma unroll
      for (int e = 0; e < 8; ++e) v.e[e] = static_cast<T>(f[e]);
      *reinterpret_cast<LooseUnit<T>*>(row + c0) = v;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c0 + e < c) row[c0 + e] = static_cast<T>(f[e]);
  }
}

// Largest unsigned value over 4 adjacent lanes.
__device__ __forceinline__ uint32_t quad_max(uint32_t x) {
  uint32_t y = static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), 0xB1, 0xF, 0xF, true));  // 1 0 3 2
  x = x > y ? x : y;
  y = static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), 0x4E, 0xF, 0xF, true));  // 2 3 0 1
  return x > y ? x : y;
}

// Codes of 8 channels and the block's byte; all 4 lanes of a block call it.
__device__ __forceinline__ ux2 act8_encode(const float (&f)[8], uint32_t* byte) {
  uint32_t top = 0;  // magnitudes compare as integers: NaN above infinity above every number
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t b = __builtin_bit_cast(uint32_t, f[e]) & 0x7fffffffu;
    top = top > b ? top : b;
  }
  const uint32_t ex = quad_max(top) >> 23;
  const uint32_t q = ex > 7 ? ex - 6 : 1;
  *byte = ex == 255 ? kActNaN : q;
  const float inv = __builtin_bit_cast(float, (254 - q) << 23);
  uint32_t c[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float x = __builtin_amdgcn_fmed3f(f[e] * inv, -127.f, 127.f);
    // adding 1.5 * 2^23 rounds to an integer, half to even, and leaves it in the low byte
    c[e] = __builtin_bit_cast(uint32_t, x + 12582912.f) & 0xffu;
  }
  ux2 out{c[0] | (c[1] << 8) | (c[2] << 16) | (c[3] << 24), c[4] | (c[5] << 8) | (c[6] << 16) | (c[7] << 24)};
  if (ex == 255) out = ux2{0u, 0u};
  return out;
}

// The quantum a byte stands for (NaN for 255).
__device__ __forceinline__ float act8_quantum(uint32_t byte) {
  return __builtin_bit_cast(float, byte == kActNaN ? 0x7fc00000u : byte << 23);
}

__device__ __forceinline__ void act8_decode(ux2 codes, float quantum, float (&f)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t w = e < 4 ? codes[0] : codes[1];
    f[e] = static_cast<float>(static_cast<int32_t>(w << (24 - 8 * (e & 3))) >> 24) * quantum;
  }
}

// A checkpoint of n rows of c channels: codes [n][c], a byte per block [n][ceil(c / 32)].
struct Act8 {
  int8_t* codes;
  uint8_t* scales;
  bool vec;  // codes in 8-byte accesses
};

__device__ __forceinline__ void act8_store(const Act8& a, int64_t row, int c0, int c, ux2 codes, uint32_t byte) {
  if (c0 >= c) return;
  int8_t* p = a.codes + row * c + c0;
  if (a.vec) {
    *reinterpret_cast<ux2*>(p) = codes;
  } else if (c0 + 8 <= c) {
    *reinterpret_cast<LooseUnit<int8_t>*>(p) = __builtin_bit_cast(LooseUnit<int8_t>, codes);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c0 + e < c) p[e] = static_cast<int8_t>((e < 4 ? codes[0] : codes[1]) >> (8 * (e & 3)));
  }
  if ((c0 & (kActBlock - 1)) == 0) a.scales[row * ((c + kActBlock - 1) / kActBlock) + c0 / kActBlock] = static_cast<uint8_t>(byte);
}

__device__ __forceinline__ void act8_load(const Act8& a, int64_t row, int c0, int c, float (&f)[8]) {
  if (c0 >= c) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = 0.f;
    return;
  }
  const int8_t* p = a.codes + row * c + c0;
  ux2 codes{0u, 0u};
  if (a.vec) {
    codes = *reinterpret_cast<const ux2*>(p);
  } else if (c0 + 8 <= c) {
    codes = __builtin_bit_cast(ux2, *reinterpret_cast<const LooseUnit<int8_t>*>(p));
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c0 + e < c) codes[e >> 2] |= static_cast<uint32_t>(static_cast<uint8_t>(p[e])) << (8 * (e & 3));
  }
  act8_decode(codes, act8_quantum(a.scales[row * ((c + kActBlock - 1) / kActBlock) + c0 / kActBlock]), f);
}

}  // namespace ts
