// Which kernel does a call of the products grouped by expert, and how it cuts the work up: plain
// host code.
#pragma once

#include <stdint.h>

namespace ts {

enum GroupOp { kGroupFwd = 0, kGroupDgrad = 1, kGroupWgrad = 2 };

constexpr int kGroupStep = 64;  // of the reduction, in group.hip

inline int64_t group_parts(int64_t n, int64_t of) { return (n + of - 1) / of; }

// Runs at most: every expert may end in a short one, and so do the rows that none owns.
inline int64_t group_runs(int64_t n_rows, int e, int len) { return n_rows / len + e + 2; }
// Partial sums of the weight gradient at most: every expert may end in a short one.
inline int64_t group_chunks(int64_t n_rows, int e, int chunk) { return n_rows / chunk + e; }

// Whether the kernel for few rows does a call (columns: of W, or of its transpose).  Its blocks split the
// reduction, which is what counts where tiles of 128 columns leave CUs idle; where they do not, the other
// kernel's copies into LDS have more under way.
// (Rows an expert, us here / there, weights not in the caches: 8 experts of 2048 x 2048, 8: 22 / 37, 48: 24 / 38;
// 32 of 1024 x 1024, 4: 17 / 23, 24: 22 / 23, 48: 27 / 24; 64 of them, 1: 20 / 24, 4: 30 / 27, 32: 43 / 30; 64 of 1023 x 1025,
// whose rows go through registers there, 8: 41 / 59, 48: 76 / 69, the gradient 2: 60 / 40.)
inline bool group_few(GroupOp op, int64_t n_rows, int e, int cin, int columns) {
  const int64_t tiles = (n_rows < e ? n_rows : e) * group_parts(columns, 128);
  const bool loose = op == kGroupFwd && (cin % 8 != 0 || columns % 8 != 0);
  return n_rows / e <= (tiles <= 128 ? 48 : tiles < 384 ? 16 : loose ? 8 : 1);
}

// Whether the weight gradient's tiles are 256 x 256 (a block a CU) rather than 128 x 128 (two).  Large
// ones read less, but where there is about one for each CU a long expert's keep the others waiting, and a
// short run is all prologue and epilogue.  (Rows an expert, us large / small: 16 experts of 512 x 512,
// 256: 37 / 31, 1024: 46 / 50, 8000: 120 / 191; 8 of 1024 x 1024, 512: 66 / 50, 2048: 108 / 103, 8000: 271 / 315;
// 16 of 1024 x 2048, 512: 95 / 83, 2000: 226 / 242; 64 of 1024 x 1376, 96: 108 / 124, 768: 263 / 335.)
inline bool large_wgrad(int64_t n_rows, int e, int cin, int cout) {
  if (cin < 256 || cout < 256) return false;
  const int64_t tiles = group_parts(cin, 256) * group_parts(cout, 256), whole = e * tiles;
  const int64_t rows_a_cu = n_rows / 256 * tiles;
  return whole >= 1024 || rows_a_cu >= (whole < 128 ? 200 : 1536);
}

// Rows of a run of the weight gradient.  Where every expert's rows can be one run without leaving
// blocks idle, a run is what one block has to do on average; otherwise as many runs as there are
// blocks (an expert may end in a short one).
inline int group_chunk(int64_t n_rows, int e, int cin, int cout) {
  const bool large = large_wgrad(n_rows, e, cin, cout);
  const int edge = large ? 256 : 128, slots = large ? 256 : 512;
  const int64_t tiles = group_parts(cin, edge) * group_parts(cout, edge), whole = e * tiles;
  const int64_t share = whole < slots / 2 ? slots - whole : slots;
  const int64_t c = n_rows / share * tiles + group_parts(n_rows % share * tiles, share);
  const int64_t most = int64_t{1} << 28;  // (row numbers of a run lie within 32 bits)
  return static_cast<int>(group_parts(c < 256 ? 256 : c > most ? most : c, kGroupStep) * kGroupStep);
}

// The kernel of a call.
struct GroupForm {
  bool few;    // that of group_few.hip
  int rows;    // of a tile; few: of a run
  int cols;    // of a tile
  bool whole;  // rows move in whole, aligned 16-byte accesses
};

// aligned: every matrix begins at 16 bytes; looked_up: rows of x that are read by number, 0: none.
inline GroupForm group_form(GroupOp op, bool glu, bool aligned, int64_t n_rows, int e, int cin, int cout, int64_t looked_up) {
  const int N = op == kGroupDgrad ? cin : op == kGroupFwd && glu ? 2 * cout : cout;  // columns
  const bool whole = aligned && cin % 8 == 0 && cout % 8 == 0;
  // Rows of a run: 32 where most experts have more than 16.  (8 experts of 2048 x 2048, us with 16 / 32:
  // 24 rows each 22.5 / 23.1, 48 rows 32.1 / 23.9; the gradient 25.5 / 27.8 and 42.2 / 28.0.)
  if (op != kGroupWgrad && group_few(op, n_rows, e, cin, N)) return {true, n_rows / e <= 24 ? 16 : 32, 128, whole};
  // (rows looked up have 32-bit offsets)
  if (!whole || looked_up * cin >= (int64_t{1} << 31) - 8) return {false, 128, 128, false};
  if (op == kGroupWgrad) return large_wgrad(n_rows, e, cin, cout) ? GroupForm{false, 256, 256, true} : GroupForm{false, 128, 128, true};
  // (Forward, rows an expert, us large / 128 x 128: 64 experts of 1024 x 1376, 384: 117 / 97, 768: 196 / 192; 16 of 512 x
  // 512, 256: 16.2 / 11.1, 1024: 19.5 / 21.9; 8 of 1024 x 2048, 256: 25.5 / 22.0, 512: 28.5 / 33.8, 6000: 195 / 223.)
  // With glu the input gradient's epilogue, which reads and writes 2 N columns, is most of its work where the
  // reduction (cout) is short: two blocks a CU take turns at it.  (bf16, us 128 x 128 / 192 or 256 rows, at a reduction
  // of 64, 128, 256 | beyond the rule 264, 512, 1024:
  //   8 experts of 76,000 rows, N 256: 313 / 328, 336 / 349, 378 / 378 | 435 / 428, 464 / 449, 646 / 599
  //                             N 512: 651 / 614, 675 / 651, 745 / 702 | 876 / 791, 898 / 815
  //   16 of 2000,               N 256: 28.6 / 26.5, 30.2 / 28.1, 34.0 / 30.2 | 36.6 / 32.6, 46.3 / 42.0, 62.3 / 52.7
  //                             N 512: 53.6 / 57.3, 54.9 / 60.3, 59.0 / 63.4 | 63.7 / 68.3, 70.4 / 72.8, 94.6 / 90.8
  //   24 of 600,                N 256: 18.9 / 25.1, 20.0 / 27.0, 23.2 / 28.6 | 24.3 / 30.5, 24.4 / 32.6, 30.2 / 40.7
  // So it costs up to 8% where large tiles would fill the CUs, and where they do not, beyond it, the small ones were
  // faster too.  The forward product with glu, whose epilogue only writes, has no such rule: 8 of 76,000, 2 x 256
  // columns, 64, 128, 256: 295 / 255, 382 / 332, 466 / 376; 16 of 2000: 27.2 / 28.9, 28.6 / 31.8, 33.7 / 35.7.)
  if (N < 256 || n_rows / e < 512 || (op == kGroupDgrad && glu && cout <= 256)) return {false, 128, 128, true};
  // 192 rows a tile where that fills the rounds of the 256 CUs better by a sixteenth or more (half a tile
  // an expert is lost; the gradient of 32,768 rows 1024 -> 4096: 290 us, 256 rows 312; 24 experts of 600 rows,
  // 1120 -> 1888: 78 and 95; where both fill them, 609,756 rows 128 -> 2 x 256: 356 and 347)
  const int64_t across = group_parts(N, 256);
  const int64_t cost192 = group_parts((n_rows / 192 + e / 2) * across, 256) * 192;
  const int64_t cost256 = group_parts((n_rows / 256 + e / 2) * across, 256) * 256;
  return {false, 16 * cost192 < 15 * cost256 ? 192 : 256, 256, true};
}

}  // namespace ts
