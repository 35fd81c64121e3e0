// Arguments of the query and key rotation kernels (rope.hip).
#pragma once

#include <stdint.h>

#include "launch.h"

namespace ts {

constexpr int kRopeMaxWidth = 128;

// Queries or keys; heads 0: absent.
struct RopeSide {
  int heads;
  unsigned by_heads;  // filled in by the launcher: 2^32 / heads, rounded up
  int64_t x_stride, y_stride, dy_stride, dx_stride;
  const void* x;
  const float* w;  // null: no norm
  void* y;
  const void* dy;
  void* dx;
  float* dw;
};

struct RopeK {
  RopeSide side[2];
  const int32_t* coords;
  const float* freqs;
  float* part;  // dw shares [2][blocks][d]
  int64_t n;
  float eps, inv_d;
  int d, ndim, pairs, upto[2];  // pairs of all axes; of the first and of the first two
  int rest;                     // pairs of channels that are not turned; odd: and one channel more
  bool odd;
  int blocks;                   // of the backward pass
  // filled in by the launcher
  int slots, turned_slots, log_lanes, table_pairs, rows;
  unsigned by_pairs;
  bool mixed;
  int64_t tiles;
};

// Blocks of the backward pass at most, of 2048 channels or more: each leaves one share of dw.
inline int rope_blocks(int64_t n, int heads, int d) {
  if (heads > 0 && n >= 1 << 21) return 1024;  // (the product below stays within 64 bits)
  const int64_t b = ceil_div<int64_t>(n * heads * d, 2048);
  return static_cast<int>(b < 1024 ? b : 1024);
}

hipError_t launch_rope_fwd(RopeK& k, ts_dtype dt, bool interleaved, hipStream_t s);
hipError_t launch_rope_bwd(RopeK& k, ts_dtype dt, bool interleaved, hipStream_t s);

}  // namespace ts
