// Products grouped by expert (device helpers and arguments; group.hip, group_few.hip).
#pragma once

#include "common.h"
#include "launch.h"

namespace ts {

enum GroupOp { kGroupFwd = 0, kGroupDgrad = 1, kGroupWgrad = 2 };

struct GroupK {
  const void* x;      // fwd, wgrad: [n_src][cin], read by `rows`
  const void* dy;     // dgrad, wgrad: [n_rows][cout]
  const void* w;      // [e][cin][ldw]
  const void* h;      // dgrad with glu: [n_rows][2 cin]
  void* y;            // fwd: [n_rows][cout]; dgrad: dx [n_rows][cin], with glu dh [n_rows][2 cin]
  void* h_out;        // fwd with glu, optional: [n_rows][2 cout]
  float* dw;          // wgrad: [e][cin][cout]
  float* part;        // wgrad: [chunks][cin][cout]
  const int64_t* starts;
  const int32_t* rows;
  uint32_t* flags;
  int64_t n_rows, n_src;
  int e, cin, cout, ldw;  // ldw: cout, or with glu 2 cout
  int chunk;              // wgrad: grouped rows of a partial sum
  unsigned n_tiles;       // blocks along the columns
};

// Blocks over `runs` runs times n_tiles columns: neighbouring ones to one XCD (blocks go to
// the 8 of them in turn).
struct GroupBlock {
  int64_t at;     // -1: none
  int64_t spare;  // or this one of the blocks behind them, from 0 on
};
__device__ __forceinline__ GroupBlock group_block(int64_t runs, unsigned n_tiles) {
  const int64_t total = runs * n_tiles, per = (total + 7) / 8, in = blockIdx.x >> 3;
  GroupBlock b{-1, -1};
  if (in < per) {
    const int64_t at = (blockIdx.x & 7) * per + in;
    if (at < total) b.at = at;
  } else {
    b.spare = static_cast<int64_t>(blockIdx.x) - per * 8;
  }
  return b;
}
// Blocks to launch for at most `runs` runs (those of rows that no expert owns among them).
inline int64_t group_grid(int64_t runs, unsigned n_tiles) { return (runs * n_tiles + 7) / 8 * 8 + 8; }
// Runs at most: every expert may end in a short one, and so do the rows that none owns.
inline int64_t group_runs(int64_t n_rows, int e, int len) { return n_rows / len + e + 2; }

typedef unsigned gu32x4 __attribute__((ext_vector_type(4)));
typedef float gf32x4 __attribute__((ext_vector_type(4)));

template <typename T>
struct GMfma;
template <>
struct GMfma<_Float16> {
  typedef _Float16 frag __attribute__((ext_vector_type(8)));
  static __device__ __forceinline__ gf32x4 run(gu32x4 a, gu32x4 b, gf32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(frag, a), __builtin_bit_cast(frag, b), c, 0, 0, 0);
  }
};
template <>
struct GMfma<__bf16> {
  typedef __bf16 frag __attribute__((ext_vector_type(8)));
  static __device__ __forceinline__ gf32x4 run(gu32x4 a, gu32x4 b, gf32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(frag, a), __builtin_bit_cast(frag, b), c, 0, 0, 0);
  }
};

// Run of at most `len` grouped rows; every expert's rows are cut into runs from its first
// row on, and the runs are counted expert by expert.
struct GroupTile {
  int e;              // -1: past the last run
  int64_t row0;       // first grouped row
  int rows;           // of this run
  int64_t first;      // the expert's first run
  int count;          // and how many it has
};

__device__ __forceinline__ int64_t lane_i64(int64_t x, int lane) {
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<uint32_t>(x), lane);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<uint32_t>(static_cast<uint64_t>(x) >> 32), lane);
  return static_cast<int64_t>((static_cast<uint64_t>(hi) << 32) | lo);
}

// Grouped rows [*a, *b) of expert e (empty for e >= k.e); starts that decrease or leave [0,
// n_rows] are clamped, so no row outside is touched, and raise the flag.
__device__ __forceinline__ void expert_rows(const GroupK& k, int e, int64_t* a, int64_t* b) {
  *a = *b = 0;
  if (e >= k.e) return;
  const int64_t s = k.starts[e], t = k.starts[e + 1];
  *a = s < 0 ? 0 : s > k.n_rows ? k.n_rows : s;
  *b = t < *a ? *a : t > k.n_rows ? k.n_rows : t;
  if ((s != *a || t != *b) && k.flags) atomicOr(k.flags, TS_FLAG_RANGE);
}

__device__ __forceinline__ int runs_of(int64_t a, int64_t b, int len) { return static_cast<int>((b - a + len - 1) / len); }

// Runs of all experts.  This and find_tile are called by whole waves; their results are the
// same in every lane.  (64-bit: starts that make the experts overlap may add up to many.)
__device__ __forceinline__ int64_t total_runs(const GroupK& k, int len) {
  const int lane = threadIdx.x & 63;
  int64_t n = 0;
  for (int e0 = 0; e0 < k.e; e0 += 64) {
    int64_t a, b;
    expert_rows(k, e0 + lane, &a, &b);
    n += runs_of(a, b, len);
  }
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) n += __shfl_xor(n, m);
  return lane_i64(n, 0);
}

__device__ __forceinline__ GroupTile find_tile(const GroupK& k, int64_t index, int len) {
  const int lane = threadIdx.x & 63;
  GroupTile t{};
  t.e = -1;
  int64_t before = 0;
  for (int e0 = 0; e0 < k.e; e0 += 64) {
    int64_t a, b;
    expert_rows(k, e0 + lane, &a, &b);
    const int n = runs_of(a, b, len);
    int64_t inc = n;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      const int64_t up = __shfl_up(inc, m);
      if (lane >= m) inc += up;
    }
    const uint64_t hit = __ballot(index < before + inc);
    if (hit) {
      const int l = __ffsll(static_cast<unsigned long long>(hit)) - 1;
      t.e = e0 + l;
      t.count = __builtin_amdgcn_readlane(n, l);
      t.first = before + lane_i64(inc, l) - t.count;
      const int64_t r0 = lane_i64(a, l), r1 = lane_i64(b, l);
      t.row0 = r0 + (index - t.first) * len;
      t.rows = r1 - t.row0 < len ? static_cast<int>(r1 - t.row0) : len;
      return t;
    }
    before += lane_i64(inc, 63);
  }
  return t;
}

// Grouped rows that no expert owns get zeros: run `index` of `len` of them, `cols` wide from
// column c0, in a matrix of `width` columns.
template <typename T>
__device__ __forceinline__ void zero_unowned(const GroupK& k, int64_t index, int len, T* y, int width, int c0, int cols) {
  int64_t a, b, last, none;
  expert_rows(k, 0, &a, &none);
  expert_rows(k, k.e - 1, &none, &last);
  b = k.n_rows - last;
  const int64_t r0 = index * len;
  if (r0 >= a + b) return;
  const int n = static_cast<int>(a + b - r0 < len ? a + b - r0 : len);
  const int w = width - c0 < cols ? width - c0 : cols;
  for (int i = threadIdx.x; i < n * w; i += blockDim.x) {
    const int r = i / w;
    const int64_t at = r0 + r < a ? r0 + r : last + (r0 + r - a);
    y[at * width + c0 + (i - r * w)] = static_cast<T>(0.f);
  }
}

// silu(a) b and its derivatives
__device__ __forceinline__ float sigmoid(float a) { return 1.f / (1.f + expf(-a)); }

// group.hip, group_few.hip
bool group_few(GroupOp op, int64_t n_rows, int e);
hipError_t launch_group(GroupK& k, GroupOp op, ts_dtype dt, bool glu, hipStream_t s);
hipError_t launch_group_few(GroupK& k, GroupOp op, ts_dtype dt, bool glu, hipStream_t s);
int group_chunk(int64_t n_rows, int cin, int cout);
// Partial sums of the weight gradient at most: every expert may end in a short one.
inline int64_t group_chunks(int64_t n_rows, int e, int chunk) { return n_rows / chunk + e; }

}  // namespace ts
