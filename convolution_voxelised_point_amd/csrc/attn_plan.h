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

// So few query rows (times heads) that a result's error is that of a few roundings:
// probabilities and score gradients then go into their products as two 16-bit parts.
// (With one part, errors are 1.4 times the last rounding's when many roundings average,
// but of 185 calls of at most 64 rows every seventh had a result with more than 1.5
// times, up to 4.9.)  Such calls are bound by latency: 13 x 12 queries over 1000 keys, 6 / 3 heads of 40, forward and
// backward 53 -> 57 us.
inline bool few_rows(int64_t rows) { return rows <= 2048; }

// dq: whether what delta was short of is taken off at the end (attn_bwd.hip).
inline bool mends_dq(int d, int64_t rows) { return d <= 64 || few_rows(rows); }

enum class Walk { kForward, kDq, kDkv };

// How the walk over `other` rows for `own` rows (both counted over all sets,
// the heads that share a key head included) is cut up:
//   - up to 16 rows a set, of at most 64 channels: the waves of a block may share the keys
//     (attn_fwd.hip).  Forward where there are so few sets and heads that every block is
//     waited for: 4 in all, 8 at 32 channels (us, shared / not: one query of 2 key heads
//     over 10,000 keys of 64 channels 9.1 / 10.9, of 8 over 100,000 of 32 38 / 44, of 64
//     53 / 47; 16 sets of 20,000 keys of 32 33 / 30; 2000 sets of 12 rows of 64 107 / 32).
//     dq from 128 keys a set on (500 sets of 60 keys of 64 channels 31 / 25, of 150 38 / 40,
//     of 500 57 / 81; of 32 channels 19 / 15, 23 / 22, 42 / 44).  At 128 channels it lost
//     everywhere (one query over 100,000 keys 29 / 21 forward, 30 / 26 dq) and is not built;
//   - long sets, with enough blocks for every CU: two column blocks a wave (2 x 8192
//     rows of 64 channels, dk and dv: 1030 us, with one 1325; of 32 850 / 916, forward 559 /
//     638);
//   - short walks: a block takes several heads one after the other (2400 windows: forward
//     161 us, with one head a block 191; dq 226 / 252; dk and dv 266 / 304).
inline AttnPlan plan_walk(int64_t own, int64_t other, int64_t n_sets, int hk, int dp, Walk walk) {
  AttnPlan p{64, 1, 1, 1, false};
  const int64_t sets = n_sets > 0 ? n_sets : 1;
  const int64_t own_per = parts(own, sets), other_per = other / sets;
  const bool few = walk == Walk::kForward ? n_sets * hk <= (dp == 32 ? 8 : 4) : walk == Walk::kDq && other_per >= 128;
  if (own_per <= 16 && few && dp <= 64) {
    p.share_keys = true;
    p.bm = 16;
  } else if (dp <= 64 && !(walk == Walk::kDkv && few_rows(other * hk)) && own_per >= 512 && parts(own, 128) * hk >= 256) {
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
  return plan_walk(nq * (hq / hk), nk, n_sets, hk, padded_width(d), Walk::kForward);
}
inline AttnPlan plan_dq(int64_t nq, int64_t nk, int64_t n_sets, int hq, int hk, int d) {
  return plan_walk(nq * (hq / hk), nk, n_sets, hk, padded_width(d), Walk::kDq);
}
inline AttnPlan plan_dkv(int64_t nq, int64_t nk, int64_t n_sets, int hq, int hk, int d) {
  return plan_walk(nk, nq * (hq / hk), n_sets, hk, padded_width(d), Walk::kDkv);
}

}  // namespace ts
