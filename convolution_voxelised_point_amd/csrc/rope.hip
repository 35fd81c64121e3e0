// Norm of each query and key head and its rotation by the voxel's position, in one
// pass over the rows (ts_rope_fwd), and its backward pass (ts_rope_bwd).
//
//   xn = x rstd,  rstd = 1 / sqrt(mean(x^2) + eps);  (a, b) = (xn w) at a pair's channels
//   y = (a cos t - b sin t, a sin t + b cos t),      t = coordinate * freq of the pair
//   g = dy turned back by t;  dw = sum g xn;  dx = rstd (g w - xn mean(g w xn))
//
// Memory bound: every element is read and written once.  A thread owns V pairs of one
// head (two accesses of V elements), the next power of two of a head's threads lie side
// by side in a wave and sum with shuffles.  Where V does not divide a head's pairs the
// last thread starts earlier and shares some with the one before: both write the same
// values, and its sums leave them out.  A block takes some rows: it computes their sines and
// cosines once, into LDS, for all query and key heads.
//
// Angles.  The product of coordinate and frequency is formed and reduced to an eighth of a
// turn either way in fp64 (a position of 32,768 times 1 rad needs 15 bits more than fp32
// has) and rounded to fp32 once; sine and cosine there are Taylor polynomials in fp32, off by at
// most 1.2 and 1.4 times 2^-24.
//
// 304,878 voxels of 4 + 4 heads of 32, bf16: forward 58 us (317 MB, 5.5 TB/s), backward 96 (473 MB,
// 4.9 TB/s: fewer waves, for the sums of dw) and 5 for dw.  102,835 of 6 + 3 heads of 40, fp32: 53
// and 93.  Results are stored past the L2, which nothing reads them from (both passes 184 -> 174 us).
#include "common.h"
#include "lanes.h"
#include "launch.h"
#include "rope.h"

namespace ts {
namespace {

constexpr int kRopeThreads = 256;

template <typename T, int V>
struct __attribute__((packed, aligned(sizeof(T)))) Vals {
  T e[V];
};

// cos and sin of c * f
__device__ __forceinline__ float2 turn_of(int32_t c, float f) {
  const double turns = static_cast<double>(c) * static_cast<double>(f) * 0.15915494309189533577;
  const double part = __builtin_amdgcn_fract(turns), n = rint(4.0 * part);  // which quarter, 0 to 4
  const float x = static_cast<float>(fma(4.0, part, -n) * 1.57079632679489662);
  const float z = x * x;
  float s = fmaf(z, 2.7557319e-6f, -1.9841270e-4f);
  s = fmaf(z, s, 8.3333333e-3f);
  s = fmaf(z, s, -1.6666667e-1f);
  s = fmaf(z * x, s, x);
  float k = fmaf(z, -2.7557319e-7f, 2.4801587e-5f);
  k = fmaf(z, k, -1.3888889e-3f);
  k = fmaf(z, k, 4.1666667e-2f);
  k = fmaf(z, k, -0.5f);
  k = fmaf(z, k, 1.f);
  const unsigned m = static_cast<unsigned>(static_cast<int>(n));
  const unsigned cs = __builtin_bit_cast(unsigned, (m & 1) ? s : k), sn = __builtin_bit_cast(unsigned, (m & 1) ? k : s);
  return float2{__builtin_bit_cast(float, cs ^ ((m + 1) << 30 & 0x80000000u)), __builtin_bit_cast(float, sn ^ (m << 30 & 0x80000000u))};
}

// What a thread works on within a head.
struct Slot {
  int a, b;   // first channels of its two accesses
  int pair;   // its first pair in the table of angles, -1: not turned
  int skip;   // pairs that the thread before it has too
  bool live;
};

template <int V, bool IL>
__device__ __forceinline__ Slot slot_of(const RopeK& k, int s) {
  Slot o;
  o.live = s < k.slots;
  const bool rest = !IL && s >= k.turned_slots;
  const int t = rest ? s - k.turned_slots : s;
  const int pairs = IL ? k.d / 2 : rest ? k.rest : k.pairs;
  const int at = t * V, p0 = at + V <= pairs ? at : pairs - V;
  o.skip = at - p0;
  // (a head of one channel has no pair: its only thread takes it as the odd one)
  if (!o.live || pairs < V) {
    o.a = o.b = 0;
    o.pair = -1;
    o.skip = V;
    return o;
  }
  if (IL) {
    o.a = 2 * p0;
    o.b = 2 * p0 + V;
    o.pair = p0 < k.pairs ? p0 : -1;
  } else if (rest) {
    o.a = 2 * k.pairs + p0;
    o.b = o.a + k.rest;
    o.pair = -1;
  } else {
    o.a = p0;
    o.b = p0 + k.pairs;
    o.pair = p0;
  }
  return o;
}

// The elements of the two accesses as pairs (and back: the map is its own inverse only
// for halves, so both directions are written out).
template <typename F, int V, bool IL>
__device__ __forceinline__ void to_pairs(const F (&x)[2 * V], float (&a)[V], float (&b)[V]) {
#pragma unroll
  for (int e = 0; e < V; ++e) {
    a[e] = static_cast<float>(x[IL ? 2 * e : e]);
    b[e] = static_cast<float>(x[IL ? 2 * e + 1 : V + e]);
  }
}

template <typename T, int V>
__device__ __forceinline__ void load2(const T* p, const Slot& s, T (&x)[2 * V]) {
  const auto lo = *reinterpret_cast<const Vals<T, V>*>(p + s.a);
  const auto hi = *reinterpret_cast<const Vals<T, V>*>(p + s.b);
#pragma unroll
  for (int e = 0; e < V; ++e) x[e] = lo.e[e], x[V + e] = hi.e[e];
}

template <typename T, int V, bool IL>
__device__ __forceinline__ void store2(T* p, const Slot& s, const float (&a)[V], const float (&b)[V]) {
  Vals<T, V> v[2];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const int i = IL ? 2 * e : e, j = IL ? 2 * e + 1 : V + e;
    v[i / V].e[i % V] = static_cast<T>(a[e]);
    v[j / V].e[j % V] = static_cast<T>(b[e]);
  }
  store_once(p + s.a, v[0]);
  store_once(p + s.b, v[1]);
}

template <int V, bool IL>
__device__ __forceinline__ void load_w(const float* w, const Slot& s, float (&wa)[V], float (&wb)[V]) {
  float t[2 * V];
  load2<float, V>(w, s, t);
  to_pairs<float, V, IL>(t, wa, wb);
}

// The table of angles of rows row0.. (`rows` of them): [row][table_pairs] (cos, sin).
__device__ __forceinline__ void fill_angles(const RopeK& k, int64_t row0, int rows, float2* tab) {
  for (int i = threadIdx.x; i < rows * k.table_pairs; i += kRopeThreads) {
    const int row = k.table_pairs == 1 ? i : static_cast<int>(__umulhi(i, k.by_pairs)), p = i - row * k.table_pairs;
    float2 t{1.f, 0.f};
    if (p < k.pairs) {
      const int axis = p < k.upto[0] ? 0 : p < k.upto[1] ? 1 : 2;
      t = turn_of(k.coords[(row0 + row) * (k.ndim + 1) + 1 + axis], k.freqs[p]);
    }
    tab[i] = t;
  }
}

// The V pairs whose angles are cs, turned by them, or (BACK) the other way; only the first `n`, if SOME: adjacent
// pairs behind the turned ones may share their access, and stay as they are (products with a cosine of 1 and
// a sine of 0 do not leave them so beside a neighbour's infinity).
template <int V, bool BACK, bool SOME>
__device__ __forceinline__ void turn(const float2* cs, int n, float (&a)[V], float (&b)[V]) {
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const float2 t = cs[e];
    const float p = a[e], q = b[e];
    const float ta = fmaf(p, t.x, BACK ? q * t.y : -q * t.y), tb = BACK ? fmaf(q, t.x, -p * t.y) : fmaf(p, t.y, q * t.x);
    a[e] = !SOME || e < n ? ta : p;
    b[e] = !SOME || e < n ? tb : q;
  }
}
template <int V, bool IL, bool BACK>
__device__ __forceinline__ void turn(const RopeK& k, const Slot& s, const float2* row, float (&a)[V], float (&b)[V]) {
  if (s.pair < 0) return;
  if (IL && k.mixed) turn<V, BACK, true>(row + s.pair, k.pairs - s.pair, a, b);
  else
    turn<V, BACK, false>(row + s.pair, V, a, b);
}

// This thread's items of a block's rows: a slot of a head each.
struct Item {
  int row, head;
  bool on;
};
__device__ __forceinline__ Item item_of(const RopeK& k, const RopeSide& side, int i, int rows) {
  const int rh = i >> k.log_lanes;
  Item it;
  it.row = side.heads == 1 ? rh : static_cast<int>(__umulhi(rh, side.by_heads));
  it.head = rh - it.row * side.heads;
  it.on = it.row < rows;
  return it;
}

template <typename T, int V, bool IL, int U>
__device__ __forceinline__ void rope_fwd_side(const RopeK& k, const RopeSide& side, const Slot& s, int64_t row0, int rows,
                                              const float2* tab) {
  const int lanes = 1 << k.log_lanes, count = (rows * side.heads) << k.log_lanes;
  const bool first = (threadIdx.x & (lanes - 1)) == 0;
  const T* x = static_cast<const T*>(side.x) + row0 * side.x_stride;
  T* y = static_cast<T*>(side.y) + row0 * side.y_stride;
  float wa[V], wb[V], w_odd = 1.f;
  if (side.w) {
    load_w<V, IL>(side.w, s, wa, wb);
    if (k.odd) w_odd = side.w[k.d - 1];
  }
  for (int i0 = threadIdx.x; i0 < count; i0 += U * kRopeThreads) {
    T v[U][2 * V];
    T odd[U];
    Item it[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      it[u] = item_of(k, side, i0 + u * kRopeThreads, rows);
      it[u].on = it[u].on && s.live;
      const T* p = x + (it[u].on ? it[u].row * side.x_stride + it[u].head * k.d : 0);
      load2<T, V>(p, s, v[u]);
      odd[u] = k.odd ? p[k.d - 1] : static_cast<T>(0.f);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float a[V], b[V];
      to_pairs<T, V, IL>(v[u], a, b);
      float last = static_cast<float>(odd[u]);
      if (side.w) {
        float sum = k.odd && first ? last * last : 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) sum += e >= s.skip ? fmaf(a[e], a[e], b[e] * b[e]) : 0.f;
        const float rstd = 1.f / sqrtf(fmaf(sum_lanes(sum, lanes), k.inv_d, k.eps));
#pragma unroll
        for (int e = 0; e < V; ++e) a[e] *= rstd * wa[e], b[e] *= rstd * wb[e];
        last *= rstd * w_odd;
      }
      turn<V, IL, false>(k, s, tab + (it[u].on ? it[u].row * k.table_pairs : 0), a, b);
      if (it[u].on) {
        T* p = y + (it[u].row * side.y_stride + it[u].head * k.d);
        store2<T, V, IL>(p, s, a, b);
        if (k.odd && first) p[k.d - 1] = static_cast<T>(last);
      }
    }
  }
}

template <typename T, int V, bool IL, int U>
__global__ __launch_bounds__(kRopeThreads) void k_rope_fwd(const RopeK k) {
  extern __shared__ float2 tab[];
  const Slot s = slot_of<V, IL>(k, threadIdx.x & ((1 << k.log_lanes) - 1));
  for (int64_t tile = blockIdx.x; tile < k.tiles; tile += gridDim.x) {
    const int64_t row0 = tile * k.rows;
    const int rows = static_cast<int>(k.n - row0 < k.rows ? k.n - row0 : k.rows);
    if (k.table_pairs) {
      if (tile != blockIdx.x) __syncthreads();  // the table of the tile before has been read
      fill_angles(k, row0, rows, tab);
      __syncthreads();
    }
    rope_fwd_side<T, V, IL, U>(k, k.side[0], s, row0, rows, tab);
    rope_fwd_side<T, V, IL, U>(k, k.side[1], s, row0, rows, tab);
  }
}

// Gradients of a block's rows, and what they add to dw.
template <typename T, int V, bool IL, int U>
__device__ __forceinline__ void rope_bwd_side(const RopeK& k, const RopeSide& side, const Slot& s, int64_t row0, int rows,
                                              const float2* tab, float (&da)[V], float (&db)[V], float& d_odd) {
  const int lanes = 1 << k.log_lanes, count = (rows * side.heads) << k.log_lanes;
  const bool first = (threadIdx.x & (lanes - 1)) == 0;
  const T* x = static_cast<const T*>(side.x) + row0 * side.x_stride;
  const T* dy = static_cast<const T*>(side.dy) + row0 * side.dy_stride;
  T* dx = static_cast<T*>(side.dx) + row0 * side.dx_stride;
  float wa[V], wb[V], w_odd = 1.f;
  if (side.w) {
    load_w<V, IL>(side.w, s, wa, wb);
    if (k.odd) w_odd = side.w[k.d - 1];
  }
  for (int i0 = threadIdx.x; i0 < count; i0 += U * kRopeThreads) {
    T v[U][2 * V], gv[U][2 * V];
    T odd[U], godd[U];
    Item it[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      it[u] = item_of(k, side, i0 + u * kRopeThreads, rows);
      it[u].on = it[u].on && s.live;
      const int col = it[u].head * k.d;
      const T* p = dy + (it[u].on ? it[u].row * side.dy_stride + col : 0);
      load2<T, V>(p, s, gv[u]);
      godd[u] = k.odd ? p[k.d - 1] : static_cast<T>(0.f);
      if (side.w) {
        p = x + (it[u].on ? it[u].row * side.x_stride + col : 0);
        load2<T, V>(p, s, v[u]);
        odd[u] = k.odd ? p[k.d - 1] : static_cast<T>(0.f);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float a[V], b[V];
      to_pairs<T, V, IL>(gv[u], a, b);
      float last = static_cast<float>(godd[u]);
      turn<V, IL, true>(k, s, tab + (it[u].on ? it[u].row * k.table_pairs : 0), a, b);
      if (side.w) {
        float xa[V], xb[V];
        to_pairs<T, V, IL>(v[u], xa, xb);
        const float xo = static_cast<float>(odd[u]);
        float sum = k.odd && first ? xo * xo : 0.f, dot = k.odd && first ? xo * last * w_odd : 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const bool mine = e >= s.skip;
          sum += mine ? fmaf(xa[e], xa[e], xb[e] * xb[e]) : 0.f;
          dot += mine ? fmaf(xa[e], a[e] * wa[e], xb[e] * b[e] * wb[e]) : 0.f;
        }
        sum = sum_lanes(sum, lanes);
        dot = sum_lanes(dot, lanes);
        const float rstd = 1.f / sqrtf(fmaf(sum, k.inv_d, k.eps));
        const float c = dot * rstd * k.inv_d;  // mean(g w xn)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const bool mine = it[u].on && e >= s.skip;
          const float na = xa[e] * rstd, nb = xb[e] * rstd;
          da[e] = mine ? fmaf(a[e], na, da[e]) : da[e];
          db[e] = mine ? fmaf(b[e], nb, db[e]) : db[e];
          a[e] = fmaf(-na, c, a[e] * wa[e]) * rstd;
          b[e] = fmaf(-nb, c, b[e] * wb[e]) * rstd;
        }
        if (k.odd) {
          const float no = xo * rstd;
          d_odd = it[u].on && first ? fmaf(last, no, d_odd) : d_odd;
          last = fmaf(-no, c, last * w_odd) * rstd;
        }
      }
      if (it[u].on) {
        T* p = dx + (it[u].row * side.dx_stride + it[u].head * k.d);
        store2<T, V, IL>(p, s, a, b);
        if (k.odd && first) p[k.d - 1] = static_cast<T>(last);
      }
    }
  }
}

// Each block walks over tiles and adds up its share of dw; dw is summed from those
// shares in a fixed order afterwards.
// (304,878 x 8 heads of 32, bf16, a pass forward and back: three waves per SIMD with two items a
// thread 177 us, with one 178, four waves 186 with spills; fp32, 102,835 x 9 of 40: four waves 186,
// three 197.)
constexpr int rope_bwd_waves(int v) { return v == 8 ? 3 : 4; }
template <typename T, int V, bool IL, int U>
__global__ __launch_bounds__(kRopeThreads, rope_bwd_waves(V)) void k_rope_bwd(const RopeK k) {
  extern __shared__ float2 tab[];
  __shared__ float red[kRopeThreads / 64][kRopeMaxWidth + 1];
  const int tid = threadIdx.x, lanes = 1 << k.log_lanes;
  const Slot s = slot_of<V, IL>(k, tid & (lanes - 1));
  float da[2][V], db[2][V], d_odd[2] = {0.f, 0.f};
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int e = 0; e < V; ++e) da[h][e] = db[h][e] = 0.f;

  for (int64_t tile = blockIdx.x; tile < k.tiles; tile += gridDim.x) {
    const int64_t row0 = tile * k.rows;
    const int rows = static_cast<int>(k.n - row0 < k.rows ? k.n - row0 : k.rows);
    if (k.table_pairs) {
      if (tile != blockIdx.x) __syncthreads();  // the table of the tile before has been read
      fill_angles(k, row0, rows, tab);
      __syncthreads();
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) rope_bwd_side<T, V, IL, U>(k, k.side[h], s, row0, rows, tab, da[h], db[h], d_odd[h]);
  }

#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (!k.side[h].dw) continue;
    // the threads of one slot, within the wave, then over the waves
    for (int m = lanes; m < 64; m <<= 1) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        da[h][e] += __shfl_xor(da[h][e], m);
        db[h][e] += __shfl_xor(db[h][e], m);
      }
      d_odd[h] += __shfl_xor(d_odd[h], m);
    }
    __syncthreads();
    if ((tid & 63) < lanes && s.live) {
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (e >= s.skip) {
          red[tid >> 6][IL ? s.a + 2 * e : s.a + e] = da[h][e];
          red[tid >> 6][IL ? s.a + 2 * e + 1 : s.b + e] = db[h][e];
        }
      if (k.odd && (tid & (lanes - 1)) == 0) red[tid >> 6][k.d - 1] = d_odd[h];
    }
    __syncthreads();
    float* part = k.part + (static_cast<int64_t>(h) * k.blocks + blockIdx.x) * k.d;
    for (int i = tid; i < k.d; i += kRopeThreads) {
      float sum = 0.f;
#pragma unroll
      for (int wv = 0; wv < kRopeThreads / 64; ++wv) sum += red[wv][i];
      part[i] = sum;
    }
  }
}

// dw of a side (blockIdx.y) = sum of its blocks' shares; 16 channels a block, 64 threads each.
__global__ __launch_bounds__(1024) void k_rope_dw(const RopeK k) {
  __shared__ float red[64][17];
  const RopeSide side = k.side[blockIdx.y];
  if (!side.dw) return;
  const int rows = k.blocks;
  const float* part = k.part + static_cast<int64_t>(blockIdx.y) * k.blocks * k.d;
  const int x = threadIdx.x & 15, share = threadIdx.x >> 4, ch = blockIdx.x * 16 + x;
  float s = 0.f;
  if (ch < k.d)
#pragma unroll 4
    for (int r = share; r < rows; r += 64) s += part[static_cast<int64_t>(r) * k.d + ch];
  red[share][x] = s;
  __syncthreads();
  if (share != 0 || ch >= k.d) return;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < 64; ++i) s += red[i][x];
  side.dw[ch] = s;
}

// Pairs per thread: as many as both the turned and the remaining part of a head hold, up to
// 16 bytes an access (one where a head is a single channel and has no pair).
template <typename T, bool IL>
int pairs_per_thread(const RopeK& k) {
  const int turned = IL ? k.d / 2 : k.pairs, rest = IL ? 0 : k.rest;
  for (int v = 16 / sizeof(T); v > 1 && turned + rest > 0; v /= 2)
    if ((turned == 0 || turned >= v) && (rest == 0 || rest >= v)) return v;
  return 1;
}

template <typename T, int V, bool IL>
void run(RopeK& k, bool back, hipStream_t s) {
  k.turned_slots = IL ? 0 : ceil_div(k.pairs, V);
  k.slots = IL ? ceil_div(k.d / 2, V) : k.turned_slots + ceil_div(k.rest, V);
  if (k.slots < 1) k.slots = 1;
  k.log_lanes = 0;
  while ((1 << k.log_lanes) < k.slots) ++k.log_lanes;
  // (mixed: an access of adjacent pairs holds turned ones and others; it then reads the table past them)
  k.mixed = IL && k.pairs > 0 && k.pairs < k.d / 2 && (k.pairs % V != 0 || k.pairs > k.d / 2 - V);
  k.table_pairs = k.mixed ? k.d / 2 : k.pairs;
  if (k.table_pairs > 1) k.by_pairs = static_cast<unsigned>((uint64_t{1} << 32) / k.table_pairs + 1);
  for (RopeSide& side : k.side)
    if (side.heads > 1) side.by_heads = static_cast<unsigned>((uint64_t{1} << 32) / side.heads + 1);
  // Rows of a tile: 1024 items, in a table of at most 32 KB; fewer where that leaves CUs without a
  // tile, though on the way back no fewer than give each block one (440 rows of 4 heads of 40, both
  // ways: 46 us, with tiles of one row 118).
  const int heads = k.side[0].heads + k.side[1].heads;
  int64_t rows = 4 * kRopeThreads / (heads << k.log_lanes);
  const int64_t few = back ? std::max<int64_t>(k.n / 512, ceil_div<int64_t>(k.n, k.blocks)) : k.n / 512;
  if (rows > few) rows = few;
  if (k.table_pairs && rows > 4096 / k.table_pairs) rows = 4096 / k.table_pairs;
  k.rows = static_cast<int>(rows < 1 ? 1 : rows);
  k.tiles = ceil_div<int64_t>(k.n, k.rows);
  const size_t lds = static_cast<size_t>(k.rows) * k.table_pairs * sizeof(float2);
  if (back) {
    const int resident = 256 * rope_bwd_waves(V);
    k.blocks = k.blocks < resident ? k.blocks : resident;
    k_rope_bwd<T, V, IL, V == 8 ? 2 : 1><<<k.blocks, kRopeThreads, lds, s>>>(k);
  } else  // (at most 2^23 blocks: a launch may have 2^32 threads)
    k_rope_fwd<T, V, IL, 2><<<static_cast<unsigned>(k.tiles < (1 << 23) ? k.tiles : 1 << 23), kRopeThreads, lds, s>>>(k);
}

template <typename T, bool IL>
void run(RopeK& k, bool back, hipStream_t s) {
  switch (pairs_per_thread<T, IL>(k)) {
    case 8:
      if constexpr (sizeof(T) == 2) return run<T, 8, IL>(k, back, s);
      break;
    case 4: return run<T, 4, IL>(k, back, s);
    case 2: return run<T, 2, IL>(k, back, s);
    default: return run<T, 1, IL>(k, back, s);
  }
}

void run(RopeK& k, ts_dtype dt, bool il, bool back, hipStream_t s) {
  switch (dt) {
    case TS_F32: return il ? run<float, true>(k, back, s) : run<float, false>(k, back, s);
    case TS_F16: return il ? run<_Float16, true>(k, back, s) : run<_Float16, false>(k, back, s);
    default: return il ? run<__bf16, true>(k, back, s) : run<__bf16, false>(k, back, s);
  }
}

}  // namespace

hipError_t launch_rope_fwd(RopeK& k, ts_dtype dt, bool interleaved, hipStream_t s) {
  if (k.n == 0 || k.side[0].heads + k.side[1].heads == 0) return hipSuccess;
  run(k, dt, interleaved, false, s);
  return hipGetLastError();
}

hipError_t launch_rope_bwd(RopeK& k, ts_dtype dt, bool interleaved, hipStream_t s) {
  if (k.n > 0) run(k, dt, interleaved, true, s);
  if (k.side[0].dw || k.side[1].dw) k_rope_dw<<<dim3(ceil_div(k.d, 16), 2), 1024, 0, s>>>(k);
  return hipGetLastError();
}

}  // namespace ts
