// Shared parts of the attention kernels (attn_fwd.hip, attn_bwd.hip).
//
// Rows of packed sets attend to the keys of their own set.  Every kernel owns
// a few columns (16 per MFMA column block) of one set and one key-value head
// and streams the other side of that set through LDS in tiles of rows:
//   forward and dq: columns = query rows, tile rows = keys;
//   dk and dv:      columns = keys,       tile rows = query rows.
// The query rows of a set and key-value head are its queries times the heads
// that share the key-value head: packed row r is query r / grp, head
// kvh * grp + r % grp.  So a single query of grp heads fills grp columns of one
// block, which reads the keys once, and the gradients of a shared head sum
// over its query heads inside the kernel.
//
// Products use v_mfma_f32_16x16x32 with the tile as the A operand (lane (g, c):
// row c, contracted elements 8g..8g+7) and the columns as B, held in registers
// for the whole walk.  The result has lane (g, c) holding rows 4g..4g+3 of
// column c: two such results over 32 tile rows, rounded to 16 bits, are the B
// operand of the second product as they stand, provided its A operand (the
// transposed tile) takes the contracted rows in the same order: 4g..4g+3 of
// the first 16 rows, then of the second.  The transposing LDS reads name
// exactly those rows, so probabilities never leave the registers.
//
// A tile row is DP elements (the head width padded with zeros to 32, 64 or
// 128) in 16-byte chunks, XOR-swizzled by the row so that the 16 rows of a
// straight read fall on 16 different 16-byte bank groups, and a transposing
// read (8 bytes a lane) on each group twice.
#pragma once

#include "common.h"
#include "launch.h"

namespace ts {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <typename T>
struct AMfma;
template <>
struct AMfma<_Float16> {
  typedef f16x8 frag;
  static __device__ __forceinline__ f32x4 run(frag a, frag b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
};
template <>
struct AMfma<__bf16> {
  typedef bf16x8 frag;
  static __device__ __forceinline__ f32x4 run(frag a, frag b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};

// Byte offset of 16-byte chunk ch of tile row r.
template <int DP>
__device__ __forceinline__ int tile_at(int r, int ch) {
  constexpr int CH = DP / 8, SH = DP == 128 ? 0 : DP == 64 ? 1 : 2;
  return r * (DP * 2) + ((ch ^ ((r >> SH) & (CH - 1))) * 16);
}

// Transposing LDS reads (gfx950): in each 16-lane group, lane q + 4m names 4
// consecutive 16-bit values and lane 4q + r receives value r of the runs named
// by lanes q, q+4, q+8, q+12.  Kept out of the kernel templates: clang emits
// no host launch stub for a kernel template whose body names the builtin.
typedef __attribute__((__vector_size__(4 * sizeof(__fp16)))) __fp16 h4tr;
typedef __attribute__((address_space(3))) h4tr lds_h4tr;
static __device__ __forceinline__ u32x4 lds_tr_pair(const char* p0, const char* p1) {
  const h4tr lo = __builtin_amdgcn_ds_read_tr16_b64_v4f16((lds_h4tr*)p0);
  const h4tr hi = __builtin_amdgcn_ds_read_tr16_b64_v4f16((lds_h4tr*)p1);
  const u32x2 l = __builtin_bit_cast(u32x2, lo), h = __builtin_bit_cast(u32x2, hi);
  return u32x4{l[0], l[1], h[0], h[1]};
}

// A operand: rows r0..r0+15 of the tile, elements 32 kb + 8g..+7.
template <typename T, int DP>
__device__ __forceinline__ typename AMfma<T>::frag tile_frag(const char* tile, int r0, int kb, int lane) {
  return __builtin_bit_cast(typename AMfma<T>::frag,
                            *reinterpret_cast<const u32x4*>(tile + tile_at<DP>(r0 + (lane & 15), kb * 4 + (lane >> 4))));
}
// A operand of the second product: row d = 16 i + lane % 16 of the transposed
// tile, contracted over tile rows r0 + 4g..+3 and r0 + 16 + 4g..+3.
template <typename T, int DP>
__device__ __forceinline__ typename AMfma<T>::frag tile_frag_t(const char* tile, int r0, int i, int lane) {
  const int q = lane & 3, m = (lane >> 2) & 3, g = lane >> 4;
  const int r = r0 + 4 * g + m, ch = 2 * i + (q >> 1), half = (q & 1) * 8;
  return __builtin_bit_cast(typename AMfma<T>::frag, lds_tr_pair(tile + tile_at<DP>(r, ch) + half,
                                                                 tile + tile_at<DP>(r + 16, ch) + half));
}

// Elements d0..d0+7 of a row of d elements (zeros past d).  vec: the row is
// 16-byte aligned and d is a multiple of 8.
template <typename T>
__device__ __forceinline__ u32x4 load8(const T* row, int d0, int d, bool vec) {
  u32x4 v{0u, 0u, 0u, 0u};
  if (vec) {
    if (d0 < d) v = *reinterpret_cast<const u32x4*>(row + d0);
  } else {
    typename AMfma<T>::frag f;
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = d0 + e < d ? row[d0 + e] : static_cast<T>(0.f);
    v = __builtin_bit_cast(u32x4, f);
  }
  return v;
}

// 4 consecutive results of a row, d0 a multiple of 4.  vec: 8-byte aligned rows.
template <typename T>
__device__ __forceinline__ void store4(T* row, int d0, int d, bool vec, f32x4 x) {
  typedef T t4 __attribute__((ext_vector_type(4)));
  if (vec) {
    if (d0 < d) *reinterpret_cast<t4*>(row + d0) = __builtin_convertvector(x, t4);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (d0 + e < d) row[d0 + e] = static_cast<T>(x[e]);
  }
}

// x of the lane 32 away and 16 away combined with this lane's: the two halves
// of a swap of x with itself hold both lanes' values on either lane.  (The
// elements are copied out first: clang takes element 0 twice when a vector
// element goes straight into the bit cast.)
template <bool WIDE>
__device__ __forceinline__ void both_lanes(float x, float* p, float* q) {
  const unsigned u = __builtin_bit_cast(unsigned, x);
  unsigned r0, r1;
  if constexpr (WIDE) {
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    r0 = r[0];
    r1 = r[1];
  } else {
    const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    r0 = r[0];
    r1 = r[1];
  }
  *p = __builtin_bit_cast(float, r0);
  *q = __builtin_bit_cast(float, r1);
}

// Maximum / sum over the four lanes (one per group g) that share a column.
__device__ __forceinline__ float col_max(float x) {
  float a, b;
  both_lanes<true>(x, &a, &b);
  x = fmaxf(a, b);
  both_lanes<false>(x, &a, &b);
  return fmaxf(a, b);
}
__device__ __forceinline__ float col_sum(float x) {
  float a, b;
  both_lanes<true>(x, &a, &b);
  x = a + b;
  both_lanes<false>(x, &a, &b);
  return a + b;
}

struct AttnArgs {
  const void *q, *k, *v, *o, *dout;
  void *out, *dq, *dk, *dv;
  float *lse, *delta;    // [nq][hq]
  float *part, *part_ml; // partial results of split walks
  const int64_t *qs, *ks;
  const float* slopes;
  const int32_t *qc, *kc;
  uint32_t* flags;
  int64_t nq, nk, n_sets, q_stride, k_stride, v_stride, o_stride, tiles;
  int hq, hk, grp, d, ndim, splits;
  // score s = scale q.k in units of log 2: without a cap z = c1 s'; with one
  // z = c2 tanh(..) written with exp2(c1 s')
  float c1, c2, scale;
  bool vec_in, vec_out;
};

// Rows of set i, counted with an empty-keyed set before the first and after
// the last one, so that every row belongs to a set: boundaries 0..n_sets + 2.
// Values a caller got wrong are held inside [0, n].
__device__ __forceinline__ int64_t set_bound(const int64_t* starts, int64_t n_sets, int64_t n, int64_t i) {
  if (i <= 0) return 0;
  if (i >= n_sets + 2) return n;
  const int64_t v = starts[i - 1];
  return v < 0 ? 0 : v > n ? n : v;
}

// Tile slots: set i owns slots bound(i) * mul / BM + i up to that of set
// i + 1, at least as many as its bound(i+1) - bound(i) rows times mul need, so
// no table of tiles has to be built.  Number of slots for n rows:
inline int64_t attn_tiles(int64_t n, int64_t mul, int64_t bm, int64_t n_sets) { return n * mul / bm + n_sets + 2; }

struct SetTile {
  int64_t own0, row0, rows;  // first row of the set; first packed row of the tile; packed rows of the set
  int64_t st0, st_len;       // the other side's rows of the set
};

// The set and tile of slot t (the same on every lane), by a search that reads
// 64 boundaries at a time; false for a slot without rows.
template <int BM>
__device__ __forceinline__ bool find_tile(const int64_t* own, int64_t n_own, int mul, const int64_t* st, int64_t n_st,
                                          int64_t n_sets, int64_t t, SetTile* r) {
  int64_t lo = 0, hi = n_sets + 2;  // slot(lo) <= t < slot(hi)
  const int lane = threadIdx.x & 63;
  while (hi - lo > 1) {
    const int64_t step = (hi - lo + 63) / 64;
    const int64_t i = lo + lane * step;
    const bool in = i < hi && set_bound(own, n_sets, n_own, i) * mul / BM + i <= t;
    const int c = __popcll(__ballot(in));
    const int64_t at = lo + (c > 0 ? c - 1 : 0) * step;
    lo = at;
    if (at + step < hi) hi = at + step;
  }
  const int64_t b0 = set_bound(own, n_sets, n_own, lo), b1 = set_bound(own, n_sets, n_own, lo + 1);
  r->own0 = b0;
  r->rows = (b1 - b0) * mul;
  r->row0 = (t - (b0 * mul / BM + lo)) * BM;
  r->st0 = 0;
  r->st_len = 0;
  if (lo >= 1 && lo <= n_sets) {
    const int64_t s0 = set_bound(st, n_sets, n_st, lo), s1 = set_bound(st, n_sets, n_st, lo + 1);
    r->st0 = s0;
    r->st_len = s1 > s0 ? s1 - s0 : 0;
  }
  return r->row0 >= 0 && r->row0 < r->rows;
}

// Starts that decrease or leave [0, n] raise TS_FLAG_RANGE: slot t of the first
// head looks at boundary t (there are more slots than boundaries).
__device__ __forceinline__ void check_starts(const int64_t* starts, int64_t n, int64_t n_sets, int64_t t,
                                             uint32_t* flags) {
  if (t > n_sets) return;
  const int64_t v = starts[t];
  if (v < 0 || v > n || (t < n_sets && starts[t + 1] < v)) atomicOr(flags, TS_FLAG_RANGE);
}

// Consecutive blocks go to the 8 XCDs in turn; numbering them so that each XCD
// gets a contiguous range lets the tiles of a set share that XCD's L2.
__device__ __forceinline__ uint32_t xcd_block() {
  const uint32_t n = gridDim.x, b = blockIdx.x, x = b & 7, per = n >> 3, rest = n & 7;
  return x * per + (x < rest ? x : rest) + (b >> 3);
}

struct Where {
  int64_t tile;
  int split, kvh;
};
__device__ __forceinline__ Where where(const AttnArgs& a) {
  const uint32_t id = xcd_block(), tiles = static_cast<uint32_t>(a.tiles);
  const uint32_t rest = id / tiles;
  Where w;
  w.tile = id - rest * tiles;
  w.split = static_cast<int>(rest % static_cast<uint32_t>(a.splits));
  w.kvh = static_cast<int>(rest / static_cast<uint32_t>(a.splits));
  return w;
}

// The part of [0, len) that split s of `splits` walks, in whole tiles of bn.
__device__ __forceinline__ void split_range(int64_t len, int bn, int splits, int s, int64_t* b, int64_t* e) {
  const int64_t per = (ceil_div<int64_t>(ceil_div<int64_t>(len, bn), splits)) * bn;
  const int64_t lo = per * s, hi = lo + per;
  *b = lo < len ? lo : len;
  *e = hi < len ? hi : len;
}

__device__ __forceinline__ f32x4 load_coord(const int32_t* c, int64_t row, int ndim, float w) {
  const int32_t* p = c + row * (ndim + 1) + 1;
  return f32x4{static_cast<float>(p[0]), static_cast<float>(p[1]), ndim == 3 ? static_cast<float>(p[2]) : 0.f, w};
}

__device__ __forceinline__ float distance(const f32x4& a, const f32x4& b) {
  const float x = a[0] - b[0], y = a[1] - b[1], z = a[2] - b[2];
  return __builtin_amdgcn_sqrtf(fmaf(x, x, fmaf(y, y, z * z)));
}

}  // namespace ts
