// Products grouped by expert (device helpers and arguments; group.hip, group_few.hip).
#pragma once

#include "common.h"
#include "group_plan.h"
#include "launch.h"

namespace ts {

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
  int64_t run;        // its number, expert by expert
  int count;          // runs of the expert
};

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

// (At most 2^24, more than 2^31 rows make in runs of 128; only starts that make the experts
// overlap could add up to more than 2^31 of them otherwise.)
__device__ __forceinline__ int runs_of(int64_t a, int64_t b, int len) {
  const int64_t n = (b - a + len - 1) / len;
  return n < (1 << 24) ? static_cast<int>(n) : 1 << 24;
}

// Finds runs.  Used by all waves of a block, with the same result in every lane; of up to 64
// experts each one's rows are kept in LDS.  SORTED: these in the order of their lengths, the longest
// first, so that what is taken last is short (a run's number `first` stays that of the experts' own
// order).
struct GroupLane {
  int a, b, n, inc;  // an expert's rows, its runs, and runs up to and with it
  int e, first;      // SORTED: which expert, and its first run
};
template <bool SORTED>
struct GroupFinder {
  GroupLane* kept;
  int len;
  int64_t total;  // all runs

  static __device__ __forceinline__ int scan(int x) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      const int up = __shfl_up(x, m);
      if (static_cast<int>(threadIdx.x & 63) >= m) x += up;
    }
    return x;
  }
  __device__ __forceinline__ GroupLane batch(const GroupK& k, int e0) const {
    int64_t r0, r1;
    expert_rows(k, e0 + (threadIdx.x & 63), &r0, &r1);
    GroupLane l;
    l.a = static_cast<int>(r0);
    l.b = static_cast<int>(r1);
    l.n = runs_of(r0, r1, len);
    l.inc = scan(l.n);
    l.e = e0 + (threadIdx.x & 63);
    l.first = l.inc - l.n;
    return l;
  }
  // lds: 64 entries.
  __device__ __forceinline__ GroupFinder(const GroupK& k, int run_rows, GroupLane* lds) : kept(lds), len(run_rows), total(0) {
    const int lane = threadIdx.x & 63;
    for (int e0 = 0; e0 < k.e; e0 += 64) {
      GroupLane l = batch(k, e0);
      total += __builtin_amdgcn_readlane(l.inc, 63);
      if (k.e > 64) continue;
      int at = lane;
      if (SORTED) {
        at = 0;
        l.inc = l.n;
        for (int o = 0; o < 64; ++o) {
          const int rows = __builtin_amdgcn_readlane(l.b - l.a, o), n = __builtin_amdgcn_readlane(l.n, o);
          const bool ahead = rows > l.b - l.a || (rows == l.b - l.a && o < lane);
          at += ahead;
          l.inc += ahead ? n : 0;
        }
      }
      kept[at] = l;  // (every wave writes the same, once, and reads what it wrote itself)
    }
  }
  __device__ __forceinline__ GroupTile find(const GroupK& k, int64_t index) const {
    GroupTile t{};
    t.e = -1;
    int64_t before = 0;
    for (int e0 = 0; e0 < k.e; e0 += 64) {
      const GroupLane own = k.e > 64 ? batch(k, e0) : kept[threadIdx.x & 63];
      const uint64_t hit = __ballot(index - before < own.inc);
      if (hit) {
        const int l = __ffsll(static_cast<unsigned long long>(hit)) - 1;
        t.e = __builtin_amdgcn_readlane(own.e, l);
        t.count = __builtin_amdgcn_readlane(own.n, l);
        const int64_t nth = index - (before + __builtin_amdgcn_readlane(own.inc, l) - t.count);
        t.run = (SORTED && k.e <= 64 ? __builtin_amdgcn_readlane(own.first, l) : index - nth) + nth;
        const int64_t r0 = __builtin_amdgcn_readlane(own.a, l), r1 = __builtin_amdgcn_readlane(own.b, l);
        t.row0 = r0 + nth * len;
        t.rows = r1 - t.row0 < len ? static_cast<int>(r1 - t.row0) : len;
        return t;
      }
      before += __builtin_amdgcn_readlane(own.inc, 63);
    }
    return t;
  }
};

// Grouped rows that no expert owns.
struct GroupRest {
  int64_t before, last, n;  // rows before the first expert's; the first behind the last one's; all of them
};
__device__ __forceinline__ GroupRest rows_unowned(const GroupK& k) {
  GroupRest r;
  int64_t none;
  expert_rows(k, 0, &r.before, &none);
  expert_rows(k, k.e - 1, &none, &r.last);
  r.n = r.before + k.n_rows - r.last;
  return r;
}
// They get zeros: those from r0 on, `len` at most, `cols` columns from c0 on in a matrix of
// `width` columns.
template <typename T>
__device__ __forceinline__ void zero_unowned(const GroupRest& rest, int64_t r0, int len, T* y, int width, int c0, int cols) {
  const int n = static_cast<int>(rest.n - r0 < len ? rest.n - r0 : len);
  const int w = width - c0 < cols ? width - c0 : cols;
  for (int i = threadIdx.x; i < n * w; i += blockDim.x) {
    const int r = i / w;
    const int64_t at = r0 + r < rest.before ? r0 + r : rest.last + (r0 + r - rest.before);
    y[at * width + c0 + (i - r * w)] = static_cast<T>(0.f);
  }
}
// Of the results of op: columns n0.. (`cols` of them) of y, and of what goes with it.
template <typename T, GroupOp OP, bool GLU>
__device__ __forceinline__ void zero_results(const GroupK& k, const GroupRest& rest, int64_t r0, int len, int N, int n0, int cols) {
  T* y = static_cast<T*>(k.y);
  if (N - n0 < cols) cols = N - n0;
  zero_unowned(rest, r0, len, y, OP == kGroupDgrad && GLU ? 2 * N : N, n0, cols);
  if (GLU) {
    T* h = OP == kGroupDgrad ? y : static_cast<T*>(k.h_out);
    if (h && OP == kGroupFwd) zero_unowned(rest, r0, len, h, 2 * N, n0, cols);
    if (h) zero_unowned(rest, r0, len, h, 2 * N, N + n0, cols);
  }
}

// 1 / (1 + exp(-a)), off by about 4 * 2^-24 of itself: the exponential through exp2 of the product
// with log2(e) in two parts (one part alone is off by |a| 2^-24; the instruction itself by one
// unit), at a third of the instructions of expf and a division.  (Beyond 10^4 either way the
// result is 0 or 1; infinities stay out of the second part.)
__device__ __forceinline__ float sigmoid(float a) {
  const float q = __builtin_amdgcn_fmed3f(-a, -1e4f, 1e4f);
  const float hi = q * 1.44269504f, lo = fmaf(q, 1.92596299e-8f, fmaf(q, 1.44269504f, -hi));
  const float e = __builtin_amdgcn_exp2f(hi);
  return __builtin_amdgcn_rcpf(fmaf(e, fmaf(lo, 0.693147181f, 1.f), 1.f));
}

// How a call is done.
inline GroupForm form_of(const GroupK& k, GroupOp op, bool glu) {
  uintptr_t bits = 0;
  for (const void* p : {k.x, k.dy, k.w, k.h, static_cast<const void*>(k.y), static_cast<const void*>(k.h_out),
                        static_cast<const void*>(k.dw), static_cast<const void*>(k.part)})
    bits |= reinterpret_cast<uintptr_t>(p);
  return group_form(op, glu, (bits & 15) == 0, k.n_rows, k.e, k.cin, k.cout,
                    k.rows && op != kGroupDgrad ? k.n_src : 0);
}

// group.hip, group_few.hip
hipError_t launch_group(GroupK& k, GroupOp op, ts_dtype dt, bool glu, hipStream_t s);
hipError_t launch_group_few(GroupK& k, GroupOp op, ts_dtype dt, bool glu, hipStream_t s);

}  // namespace ts
