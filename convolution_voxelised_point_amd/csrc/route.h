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

// Threads of a row: 8 experts each.
inline int route_log_lanes(int e) {
  int l = 0;
  while ((8 << l) < e) ++l;
  return l;
}

// Whether one block of 1024 threads does a call alone: in at most two passes over its rows.  (Top 2, us
// alone / in three launches: 8 experts, 1024 rows 6.9 / 10.4; 64 experts, 256 rows 8.5 / 11.5, 512 rows 12.4 / 11.6;
// top 8 of 256, 39 rows 16.4 / 17.4, 128 rows 28.0 / 17.4.)
inline bool route_small(int64_t n, int e, int top) { return n * top <= kRouteSmall && n << route_log_lanes(e) <= 2048; }

// Blocks of 1024 threads: two for each CU, and at most 2^18 counts.
constexpr int kRouteMaxBlocks = 512;
inline int route_blocks(int64_t n, int e) {
  const int64_t rows = 1024 >> route_log_lanes(e), b = (n + rows - 1) / rows, most = (1 << 18) / (e + 1);
  const int64_t cap = most < kRouteMaxBlocks ? most : kRouteMaxBlocks;
  return static_cast<int>(b < cap ? b : cap);
}

hipError_t launch_route(RouteK& k, ts_dtype dt, bool back, hipStream_t s);

}  // namespace ts
