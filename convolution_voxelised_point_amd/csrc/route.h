// Arguments of the router's kernels (route.hip).
#pragma once

#include <stdint.h>

#include "launch.h"

namespace ts {

constexpr int kRouteMaxTop = 16, kRouteMaxExperts = 512;
constexpr int kRouteSmall = 2048;  // pairs that one block takes on alone

struct RouteK {
  const void* logits;
  int64_t n;
  int e, top;
  bool over_all;
  int32_t* experts;
  float* gates;
  int64_t* starts;
  int32_t *rows, *place;
  int32_t* counts;  // [e + 1][blocks], and their sums [e + 1]
  const float* dgates;
  void* dlogits;
  // filled in by the launcher
  int log_lanes, bits, blocks;
};

inline bool route_small(int64_t n, int top) { return n * top <= kRouteSmall; }

// Blocks of 1024 threads: two for each CU, and at most 2^18 counts.
inline int route_blocks(int64_t n, int e) {
  int lanes = 1;
  while (8 * lanes < e) lanes *= 2;
  const int64_t rows = 1024 / lanes, b = (n + rows - 1) / rows, most = (1 << 18) / (e + 1);
  const int64_t cap = most < 512 ? most : 512;
  return static_cast<int>(b < cap ? b : cap);
}

hipError_t launch_route(RouteK& k, ts_dtype dt, bool back, hipStream_t s);

}  // namespace ts
