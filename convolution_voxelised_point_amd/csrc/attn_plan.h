// How the attention kernels cut up their work: plain host code.
#pragma once

#include <stdint.h>

namespace ts {

constexpr int kAttnMaxSplits = 512;

// How a walk is cut up: columns per block, column blocks per wave, key-value heads
// per block, parts of the other side, and whether the waves of a block share one
// column block.
struct AttnPlan {
  int bm, nc, heads, splits;
  bool share_keys;
};

inline int64_t parts(int64_t n, int64_t of) { return (n + of - 1) / of; }

inline int padded_width(int d) { return d <= 32 ? 32 : d <= 64 ? 64 : 128; }

// How the walk over `other` rows for `own` rows (both counted over all sets,
// the heads that share a key head included) is cut up:
//   - up to 16 rows a set: the waves of a block share the keys (attn_fwd.hip);
//   - long sets, with enough blocks for every CU: two column blocks a wave (2 x 8192
//     rows, dk and dv: 1030 us, with one 1325);
//   - short walks: a block takes several heads one after the other (2400 windows: forward
//     161 us, with one head a block 191; dq 226 / 252; dk and dv 266 / 304).
inline AttnPlan plan_walk(int64_t own, int64_t other, int64_t n_sets, int hk, int dp, bool may_share, int max_nc) {
  AttnPlan p{64, 1, 1, 1, false};
  const int64_t sets = n_sets > 0 ? n_sets : 1;
  const int64_t own_per = parts(own, sets), other_per = other / sets;
  if (may_share && own_per <= 16) {
    p.share_keys = true;
    p.bm = 16;
  } else if (max_nc >= 2 && own_per >= 512 && parts(own, 128) * hk >= 256) {
    p.nc = 2;
    p.bm = 128;
  } else if (dp <= 64 && other_per <= 512) {
    // as many heads as leave 1024 blocks
    const int64_t tiles = parts(own, 64) > n_sets ? parts(own, 64) : n_sets;
    while (p.heads < 4 && p.heads * 2 <= hk && tiles * (hk / (p.heads * 2)) >= 1024) p.heads *= 2;
  }
  const int64_t tiles = parts(own, p.bm);
  const int64_t blocks = (tiles > n_sets ? tiles : n_sets < own ? n_sets : own) * parts(hk, p.heads);
  // Walks are split until 512 blocks run (at least 256 rows each: a short walk is
  // mostly its beginning).  One query over 102,835 keys: 18 us and 5 for the join, unsplit
  // 741; 13 sets of 37 queries over 1000 keys: 16 and 4, unsplit 35.  Where that leaves
  // fewer than two rounds of blocks, long ones are split further (at least 1024 rows
  // each), so that the last round is a small part of the whole (2 x 8192 rows: forward
  // 705 -> 662 us, dq 1091 -> 1013, dk and dv 1218 -> 1030).
  int64_t s = blocks > 0 ? 512 / blocks : 1;
  if (s > other_per / 256) s = other_per / 256;
  int64_t fine = blocks > 0 && blocks < 1024 ? 2048 / blocks : 1;
  if (fine > other_per / 1024) fine = other_per / 1024;
  if (s < fine) s = fine;
  if (s > kAttnMaxSplits) s = kAttnMaxSplits;
  p.splits = s < 2 ? 1 : static_cast<int>(s);
  return p;
}

// Query rows walk over keys (forward, dq); keys walk over query rows (dk and dv).
inline AttnPlan plan_fwd(int64_t nq, int64_t nk, int64_t n_sets, int hq, int hk, int d) {
  const int dp = padded_width(d);
  return plan_walk(nq * (hq / hk), nk, n_sets, hk, dp, true, dp <= 64 ? 2 : 1);
}
inline AttnPlan plan_dkv(int64_t nq, int64_t nk, int64_t n_sets, int hq, int hk, int d) {
  const int dp = padded_width(d);
  return plan_walk(nk, nq * (hq / hk), n_sets, hk, dp, false, dp <= 64 ? 2 : 1);
}

}  // namespace ts
