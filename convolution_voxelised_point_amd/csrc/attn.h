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

// 4 consecutive results of a row, d0 a multiple of 4.
template <typename T>
__device__ __forceinline__ void store4(T* row, int d0, int d, f32x4 x) {
  typedef T t4 __attribute__((ext_vector_type(4)));
  if (d0 < d) *reinterpret_cast<t4*>(row + d0) = __builtin_convertvector(x, t4);
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

// (heads: query head = kvh * grp + its place among those that share kvh)
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
  int hq, hk, grp, d, ndim, splits, heads;  // heads: key-value heads a block takes, one after the other
  // scores in units of log 2 from s = q.k: c1 s, or with a cap
  // c2 tanh(scale s / cap) = c2 - 2 c2 / (exp2(c1 s) + 1); c1 is made of |scale|,
  // and negate says that q enters with its sign turned
  float c1, c2, scale;
  bool negate;
  bool two;    // 16-bit operands made of probabilities and score gradients go in as two parts
  bool mend;   // dq: what delta was short of is taken off at the end (attn_bwd.hip)
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

// A value that is the same on every lane, in scalar registers.
__device__ __forceinline__ int64_t lane_value(int64_t x, int lane) {
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<uint32_t>(x), lane);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<uint32_t>(static_cast<uint64_t>(x) >> 32), lane);
  return static_cast<int64_t>(static_cast<uint64_t>(hi) << 32 | lo);
}

struct SetTile {
  int64_t own0, row0, rows;  // first row of the set; first packed row of the tile; packed rows of the set
  int64_t st0, st_len;       // the other side's rows of the set
};

// The set and tile of slot t (the same on every lane); false for a slot without
// rows.  Each step reads 64 boundaries at once: first the 64 about where sets of
// equal length would put the slot, which holds it when lengths vary at random,
// then evenly spaced ones over what is left of either side.  The ends of the set
// are among the boundaries read last.
template <int BM>
__device__ __forceinline__ bool find_tile(const int64_t* own, int64_t n_own, int mul, const int64_t* st, int64_t n_st,
                                          int64_t n_sets, int64_t t, int64_t slots, SetTile* r) {
  if (t >= slots) return false;
  const int lane = threadIdx.x & 63;
  int64_t lo = 0, hi = n_sets + 2;  // slot(lo) <= t < slot(hi)
  int64_t at = static_cast<int64_t>(static_cast<float>(t) / static_cast<float>(slots) * static_cast<float>(hi)) - 31;
  at = at < 0 ? 0 : at > hi - 63 ? (hi > 63 ? hi - 63 : 0) : at;
  int64_t step = 1, b0, b1;
  // each step leaves at most a 63rd: 7 do for any count; starts that decrease may never converge
  for (int tries = 0;; ++tries) {
    if (tries == 12) return false;
    const int64_t i = at + lane * step;
    const int64_t v = set_bound(own, n_sets, n_own, i < hi ? i : hi);
    const int c = __popcll(__ballot(i < hi && v * mul / BM + i <= t));  // boundaries at or before the slot
    if (c == 0) {  // before the window
      hi = at;
    } else if (c == 64) {  // after it, or after its last sample
      lo = at + 63 * step;
    } else {
      lo = at + (c - 1) * step;
      if (lo + step < hi) hi = lo + step;
    }
    if (hi - lo == 1 && step == 1 && c > 0 && c < 64) {
      b0 = lane_value(v, c - 1);
      b1 = lane_value(v, c);
      break;
    }
    at = lo;
    step = (hi - lo + 62) / 63;  // 63 steps reach hi
  }
  r->own0 = b0;
  r->rows = (b1 - b0) * mul;
  r->row0 = (t - (b0 * mul / BM + lo)) * BM;
  r->st0 = 0;
  r->st_len = 0;
  if (lo >= 1 && lo <= n_sets) {
    const int64_t s0 = st == own && n_st == n_own ? b0 : set_bound(st, n_sets, n_st, lo);
    const int64_t s1 = st == own && n_st == n_own ? b1 : set_bound(st, n_sets, n_st, lo + 1);
    r->st0 = lane_value(s0, 0);
    r->st_len = s1 > s0 ? lane_value(s1 - s0, 0) : 0;
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

// Grid: x = tile slots, y = groups of `heads` key-value heads, z = splits.  Consecutive
// blocks go to the 8 XCDs in turn.  With many slots, each XCD gets runs of four
// consecutive tiles, so that the tiles of a set share that XCD's L2 while long and
// short sets still spread over all of them (one contiguous range per XCD left the
// XCD with the longest set running alone); x is then a multiple of 32.  With few
// slots x is odd, so that the heads and splits of one tile lie on different XCDs.
constexpr uint32_t kXcds = 8, kXcdRun = 4, kXcdMany = 256;
inline unsigned attn_grid_x(int64_t tiles) {
  if (tiles < kXcdMany) return static_cast<unsigned>(tiles) | 1u;
  return static_cast<unsigned>((tiles + kXcds * kXcdRun - 1) / (kXcds * kXcdRun) * (kXcds * kXcdRun));
}
__device__ __forceinline__ int64_t block_tile() {
  const uint32_t b = blockIdx.x;
  if (gridDim.x < kXcdMany) return b;
  const uint32_t i = b / kXcds;
  return (i / kXcdRun * kXcds + b % kXcds) * kXcdRun + i % kXcdRun;
}

// The part of [0, len) that split s of `splits` walks, in whole tiles of bn.
__device__ __forceinline__ void split_range(int64_t len, int bn, int splits, int s, int64_t* b, int64_t* e) {
  const int64_t per = (ceil_div<int64_t>(ceil_div<int64_t>(len, bn), splits)) * bn;
  const int64_t lo = per * s, hi = lo + per;
  *b = lo < len ? lo : len;
  *e = hi < len ? hi : len;
}

// The value, unknown to the compiler as equal to x: what is computed from it here is
// not computed before the walk and kept in registers through it.
__device__ __forceinline__ uint32_t late(uint32_t x) {
  asm volatile("" : "+v"(x));
  return x;
}

// Distances.  Coordinates are taken relative to one row of the block, in integers
// (so they are exact wherever the set lies, and as floats too while they are below
// 2^24), with the squared norm beside them: {x, y, z, x^2 + y^2 + z^2}.  While every norm is at most 2048, |a - b|^2 = |a|^2 + |b|^2 - 2 a.b
// is a sum of integers below 2^24, exact in fp32 in any order, and one
// v_mfma_f32_16x16x4_f32 gives a 16 x 16 tile of squares: A = the tile row's four
// values, B = (-2x, -2y, -2z, 1) of the column, C = the column's norm.  Beyond
// that the differences are formed one by one (the walk's slow form).
constexpr float kNearNorm = 4194304.f;  // 2048^2

// Coordinates as read (with ndim 2, z is y): turned into floats where they are used,
// so that the read is not waited for where it is issued.
struct Place {
  int32_t x, y, z;
};
__device__ __forceinline__ Place load_place(const int32_t* c, int64_t row, int ndim) {
  const int32_t* p = c + row * (ndim + 1) + 1;
  return Place{p[0], p[1], p[ndim - 1]};
}
// Of a row that is the same on every lane, in scalar registers.
__device__ __forceinline__ Place uniform_origin(const Place& p) {
  const auto u = [](int x) { return __builtin_amdgcn_readfirstlane(x); };
  return Place{u(p.x), u(p.y), u(p.z)};
}
__device__ __forceinline__ f32x4 relative(const Place& p, const Place& o, int ndim) {
  const auto sub = [](int32_t a, int32_t b) {
    return static_cast<float>(static_cast<int32_t>(static_cast<uint32_t>(a) - static_cast<uint32_t>(b)));
  };
  const float x = sub(p.x, o.x), y = sub(p.y, o.y), z = ndim == 3 ? sub(p.z, o.z) : 0.f;
  return f32x4{x, y, z, fmaf(x, x, fmaf(y, y, z * z))};
}
// The column's B value of lane (g, c) for the product above.
__device__ __forceinline__ float col_term(const f32x4& c, int g) {
  return g == 0 ? -2.f * c[0] : g == 1 ? -2.f * c[1] : g == 2 ? -2.f * c[2] : 1.f;
}

template <bool V>
struct Flag {
  static constexpr bool v = V;
};

// An offset past every tile, for which buffer loads give zeros.  A tile has at most 128
// rows of at most 2^23 elements (2^24 bytes) between them, so it ends at or before this,
// and a row's offset (below 127 2^24 + 2^24) added to it stays within 32 bits.
constexpr uint32_t kOutside = 0x80000000u;

// A wave-uniform address, stated as such (a buffer descriptor is built from it).
template <typename T>
__device__ __forceinline__ T* uniform_ptr(T* p) {
  const uint64_t x = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(x));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(x >> 32));
  return reinterpret_cast<T*>((static_cast<uint64_t>(hi) << 32) | lo);
}

// 16 bytes at `off` of the `bytes` bytes at `base`; zeros past them.
static __device__ __forceinline__ u32x4 load16_in(const void* base, uint32_t bytes, uint32_t off) {
  const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
      uniform_ptr(const_cast<void*>(base)), 0, static_cast<int>(__builtin_amdgcn_readfirstlane(bytes)), 0x00020000);
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, static_cast<int>(off), 0, 0));
}

// A tile of BN rows of two matrices on its way from memory to LDS.  A thread
// moves one 16-byte chunk of every (256 / CH)-th row.  Rows past the end and chunks
// past the head width come as zeros from the bounds check of the buffer loads (0 *
// NaN of another set's row would be NaN), without a mask.
template <typename T, int DP, int BN>
struct TileLoad {
  static constexpr int CH = DP / 8, CT = BN * CH / 256, STEP = 256 / CH;
  u32x4 a[CT], b[CT];

  static __device__ __forceinline__ int row(int i) { return i * STEP + threadIdx.x / CH; }
  static __device__ __forceinline__ int chunk() { return threadIdx.x % CH; }
  // fa, fb: byte offsets of the rows from the bases; na, nb: bytes up to the end of the last row.
  template <typename FA, typename FB>
  __device__ __forceinline__ void fetch(const T* pa, uint32_t na, FA&& fa, const T* pb, uint32_t nb, FB&& fb, int d) {
    const uint32_t c0 = chunk() * 8 < d ? chunk() * 16u : kOutside;
#pragma unroll
    for (int i = 0; i < CT; ++i) {
      a[i] = load16_in(pa, na, fa(i) + c0);
      b[i] = load16_in(pb, nb, fb(i) + c0);
    }
  }
  __device__ __forceinline__ void put(char* x, char* y) const {
#pragma unroll
    for (int i = 0; i < CT; ++i) {
      const int at = tile_at<DP>(row(i), chunk());
      *reinterpret_cast<u32x4*>(x + at) = a[i];
      *reinterpret_cast<u32x4*>(y + at) = b[i];
    }
  }
};

// Coordinates of a tile's rows on their way: thread r < BN brings row r's.
template <int BN>
struct TileCoords {
  Place c;
  __device__ __forceinline__ void fetch(const int32_t* coords, int64_t first, int rows, int ndim) {
    const int r = threadIdx.x;
    if (r < BN && r < rows) c = load_place(coords, first + r, ndim);
  }
  // The flag of a wave's rows: whether one is too far out for the product form.
  __device__ __forceinline__ void put(f32x4* tc, uint32_t* far_rows, const Place& org, int ndim) const {
    if (threadIdx.x >= BN) return;
    const f32x4 x = relative(c, org, ndim);
    tc[threadIdx.x] = x;
    const bool any = __any(x[3] > kNearNorm);
    if (threadIdx.x % 64 == 0) far_rows[threadIdx.x / 64] = any;
  }
};
template <int BN>
__device__ __forceinline__ bool tile_far(const uint32_t* far_rows) {
  uint32_t f = far_rows[0];
  if constexpr (BN > 64) f |= far_rows[1];
  return __builtin_amdgcn_readfirstlane(f) != 0;
}

// Where a block takes several heads one after the other over at most this many
// tiles, the tiles' coordinates stay in LDS for all of them (2400 windows forward: 183 ->
// 174 us; in the backward kernels it gained nothing).
constexpr int kCoordTiles = 4;

// The key side of a walk over n_keys keys from row `first`: tiles of keys and values of one key-value head, and the
// keys' coordinates.
template <typename T, int DP, int BN, bool BIAS>
struct KeyTiles {
  TileLoad<T, DP, BN> ld;
  TileCoords<BN> lc;
  const T *kp, *vp;
  int64_t first;
  int n_keys;

  __device__ __forceinline__ KeyTiles(const AttnArgs& a, int64_t first_key, int keys)
      : kp(static_cast<const T*>(a.k) + first_key * a.k_stride),
        vp(static_cast<const T*>(a.v) + first_key * a.v_stride),
        first(first_key),
        n_keys(keys) {
    lc.c = Place{0, 0, 0};
  }
  __device__ __forceinline__ void fetch(const AttnArgs& a, int h, int k0, bool coords) {
    const uint32_t ks = static_cast<uint32_t>(a.k_stride) * 2u, vs = static_cast<uint32_t>(a.v_stride) * 2u;
    const uint32_t last = (n_keys - k0 < BN ? n_keys - k0 : BN) - 1, w = a.d * 2u;
    ld.fetch(kp + k0 * a.k_stride + h * a.d, last * ks + w, [&](int i) { return ld.row(i) * ks; },
             vp + k0 * a.v_stride + h * a.d, last * vs + w, [&](int i) { return ld.row(i) * vs; }, a.d);
    if (BIAS && coords) lc.fetch(a.kc, first + k0, n_keys - k0, a.ndim);
  }
  __device__ __forceinline__ void put(char* tk, char* tv, bool coords, f32x4* tc, uint32_t* far_rows, const Place& org,
                                      int ndim) {
    ld.put(tk, tv);
    if (BIAS && coords) lc.put(tc, far_rows, org, ndim);
  }
};

// B operands of one head's columns: NC blocks of 16 rows whose byte offsets from a
// uniform base are given (kOutside: none).
template <typename T, int DP, int NC>
struct ColLoad {
  u32x4 x[NC][DP / 32];
  __device__ __forceinline__ void fetch(const T* base, uint32_t bytes, const uint32_t (&off)[NC], int d) {
    const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int j = 0; j < NC; ++j)
#pragma unroll
      for (int kb = 0; kb < DP / 32; ++kb) {
        const int c = kb * 32 + g * 8;
        x[j][kb] = load16_in(base, bytes, c < d ? off[j] + c * 2u : kOutside);
      }
  }
  __device__ __forceinline__ typename AMfma<T>::frag frag(int j, int kb) const {
    return __builtin_bit_cast(typename AMfma<T>::frag, x[j][kb]);
  }
  __device__ __forceinline__ typename AMfma<T>::frag frag_signed(int j, int kb, bool negate) const {
    return __builtin_bit_cast(typename AMfma<T>::frag, negate ? x[j][kb] ^ 0x80008000u : x[j][kb]);
  }
};

// Distances of the 16 tile rows from r0 to the columns, rows 4g..4g+3 in the lane's
// four values; qb: col_term of the column, norm: its squared norm.  The far form
// reads the column's coordinates again (row first + row of c): it is rare, and they
// would cost registers everywhere else.
__device__ __forceinline__ f32x4 distances(const f32x4* tc, int r0, float norm, float qb, bool far, int lane,
                                           const int32_t* c, int64_t first, uint32_t row, int ndim, const Place& org) {
  f32x4 d;
  if (far) {
    const f32x4 p = relative(load_place(c, first + late(row), ndim), org, ndim);
    const float x = p[0], y = p[1], z = p[2];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float* t = reinterpret_cast<const float*>(tc + r0 + 4 * (lane >> 4) + e);
      const float u = x - t[0], v = y - t[1], w = z - t[2];
      d[e] = fmaf(u, u, fmaf(v, v, w * w));
      __builtin_amdgcn_sched_barrier(0);  // one row at a time, for the registers' sake
    }
  } else {
    d = __builtin_amdgcn_mfma_f32_16x16x4f32(tc[r0 + (lane & 15)][lane >> 4], qb, f32x4{norm, norm, norm, norm}, 0, 0, 0);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) d[e] = __builtin_amdgcn_sqrtf(d[e]);
  return d;
}

// The query rows that are a wave's columns: NC blocks of 16 packed rows, BM columns
// apart per block of waves.  Offsets are from the tile's first query.
template <int NC, bool SHARE>
struct QueryCols {
  int64_t query0;                // uniform: query of the tile's first row
  uint32_t dq[NC], place[NC];    // query from there, place among the heads that share a key head
  bool live[NC], busy;
  uint32_t last;                 // query of the tile's last row, from query0
  __device__ __forceinline__ QueryCols(const AttnArgs& a, const SetTile& st, int bm) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t grp = a.grp, r0 = static_cast<uint32_t>(st.row0), rows = static_cast<uint32_t>(st.rows);
    const uint32_t q0 = grp == 1 ? r0 : r0 / grp;
    query0 = st.own0 + q0;
    const uint32_t lr = (r0 + bm < rows ? r0 + bm : rows) - 1;
    last = (grp == 1 ? lr : lr / grp) - q0;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const uint32_t r = r0 + (SHARE ? 0 : j * 4 + wave) * 16 + (lane & 15);
      live[j] = r < rows;
      const uint32_t x = live[j] ? r : r0, q = grp == 1 ? x : x / grp;
      dq[j] = q - q0;
      place[j] = x - q * grp;
    }
    // column blocks of a wave come 64 rows apart: it computes while its first is inside the set
    busy = r0 + (SHARE ? 0 : wave * 16) < rows;
  }
  // byte offset of column j's row of a matrix with this row stride, from row query0 of key-value head h
  __device__ __forceinline__ uint32_t offset(int j, int64_t stride, int d) const {
    return live[j] ? (late(dq[j]) * static_cast<uint32_t>(stride) + late(place[j]) * d) * 2u : kOutside;
  }
  __device__ __forceinline__ uint32_t bytes(int64_t stride, int width) const {
    return (last * static_cast<uint32_t>(stride) + width) * 2u;
  }
};

}  // namespace ts
