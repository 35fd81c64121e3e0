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
// values, and its sums leave them out.  The rows' sines and cosines are computed once per
// block into LDS and serve all heads of the row.
//
// Angles.  The product of coordinate and frequency is formed and reduced to an eighth of a
// turn either way in fp64 (a position of 32,768 times 1 rad needs 15 bits more than fp32
// has), sine and cosine there are Taylor polynomials in fp32, off by about 2^-24.
#include "common.h"
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
  const double q = static_cast<double>(c) * static_cast<double>(f) * 0.63661977236758134308;  // in quarter turns
  const double n = rint(q);
  const float x = static_cast<float>((q - n) * 1.57079632679489661923);
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
  // which quarter: n mod 4, also where n passes 32 bits
  const int m = static_cast<int>(n - 4.0 * floor(n * 0.25));
  const float cs = (m & 1) ? s : k, sn = (m & 1) ? k : s;
  return float2{m == 1 || m == 2 ? -cs : cs, m >= 2 ? -sn : sn};
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
    o.pair = p0;
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
  *reinterpret_cast<Vals<T, V>*>(p + s.a) = v[0];
  *reinterpret_cast<Vals<T, V>*>(p + s.b) = v[1];
}

template <int V, bool IL>
__device__ __forceinline__ void load_w(const float* w, const Slot& s, float (&wa)[V], float (&wb)[V]) {
  float t[2 * V];
  load2<float, V>(w, s, t);
  to_pairs<float, V, IL>(t, wa, wb);
}

__device__ __forceinline__ float sum_lanes(float x, int lanes) {
  for (int m = 1; m < lanes; m <<= 1) x += __shfl_xor(x, m);
  return x;
}

// Rows of a tile of `per` heads that starts at head number h0 (over all rows).
struct Rows {
  int64_t first;
  int at;  // heads of the first row that lie before the tile
  int n;
};
__device__ __forceinline__ Rows rows_of(int64_t h0, int per, int heads) {
  Rows r;
  r.first = h0 / heads;
  r.at = static_cast<int>(h0 - r.first * heads);
  r.n = (r.at + per - 1) / heads + 1;
  return r;
}

// The block's table of angles: [row][table_pairs] (cos, sin).
__device__ __forceinline__ void fill_angles(const RopeK& k, const Rows& r, float2* tab) {
  const int total = r.n * k.table_pairs;
  for (int i = threadIdx.x; i < total; i += kRopeThreads) {
    const int row = static_cast<int>(static_cast<unsigned>(i) / static_cast<unsigned>(k.table_pairs));
    const int p = i - row * k.table_pairs;
    float2 t{1.f, 0.f};
    if (r.first + row < k.n && p < k.pairs) {
      const int axis = p < k.upto[0] ? 0 : p < k.upto[1] ? 1 : 2;
      t = turn_of(k.coords[(r.first + row) * (k.ndim + 1) + 1 + axis], k.freqs[p]);
    }
    tab[i] = t;
  }
}

template <typename T, int V, bool IL, int U>
__global__ __launch_bounds__(kRopeThreads) void k_rope_fwd(const RopeK k) {
  extern __shared__ float2 smem[];
  const bool is_k = blockIdx.x >= static_cast<unsigned>(k.blocks_q);
  const RopeSide side = is_k ? k.side[1] : k.side[0];
  const int block = is_k ? blockIdx.x - k.blocks_q : blockIdx.x, blocks = is_k ? k.blocks_k : k.blocks_q;
  const int tid = threadIdx.x, per = kRopeThreads * U >> k.log_lanes;
  const int lanes = 1 << k.log_lanes;
  const Slot s = slot_of<V, IL>(k, tid & (lanes - 1));
  const bool first = (tid & (lanes - 1)) == 0;
  float2* tab = smem;
  const T* x = static_cast<const T*>(side.x);
  T* y = static_cast<T*>(side.y);
  float wa[V], wb[V], w_odd = 1.f;

  // one tile a block, but for the largest calls
  for (int64_t tile = block; tile < side.tiles; tile += blocks) {
    const Rows rows = rows_of(tile * per, per, side.heads);
    // reads in flight while the angles are computed
    T v[U][2 * V];
    T odd[U];
    int64_t at[U];
    int lrow[U];
    bool on[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = rows.at + ((u * kRopeThreads + tid) >> k.log_lanes);
      lrow[u] = static_cast<int>(static_cast<unsigned>(h) / static_cast<unsigned>(side.heads));
      const int head = h - lrow[u] * side.heads;
      const int64_t row = rows.first + lrow[u];
      on[u] = s.live && row < k.n;
      const int64_t from = on[u] ? row * side.x_stride + head * k.d : 0;
      at[u] = row * side.y_stride + head * k.d;
      load2<T, V>(x + from, s, v[u]);
      odd[u] = k.odd ? x[from + k.d - 1] : static_cast<T>(0.f);
    }
    if (tile == block && side.w) {
      load_w<V, IL>(side.w, s, wa, wb);
      if (k.odd) w_odd = side.w[k.d - 1];
    }
    if (k.table_pairs) {
      if (tile != block) __syncthreads();  // the table of the tile before has been read
      fill_angles(k, rows, tab);
      __syncthreads();
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
      if (s.pair >= 0 && k.table_pairs) {
        const float2* t = tab + lrow[u] * k.table_pairs + s.pair;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float2 cs = t[e];
          const float p = a[e], q = b[e];
          a[e] = fmaf(p, cs.x, -q * cs.y);
          b[e] = fmaf(p, cs.y, q * cs.x);
        }
      }
      if (on[u]) {
        store2<T, V, IL>(y + at[u], s, a, b);
        if (k.odd && first) y[at[u] + k.d - 1] = static_cast<T>(last);
      }
    }
  }
}

// Each block walks over tiles and adds up its share of dw; dw is summed from those
// shares in a fixed order afterwards.
template <typename T, int V, bool IL, int U>
__global__ __launch_bounds__(kRopeThreads) void k_rope_bwd(const RopeK k) {
  extern __shared__ float2 smem[];
  __shared__ float red[kRopeThreads / 64][kRopeMaxWidth + 1];
  const bool is_k = blockIdx.x >= static_cast<unsigned>(k.blocks_q);
  const RopeSide side = is_k ? k.side[1] : k.side[0];
  const int block = is_k ? blockIdx.x - k.blocks_q : blockIdx.x, blocks = is_k ? k.blocks_k : k.blocks_q;
  const int tid = threadIdx.x, per = kRopeThreads * U >> k.log_lanes;
  const int lanes = 1 << k.log_lanes;
  const Slot s = slot_of<V, IL>(k, tid & (lanes - 1));
  const bool first = (tid & (lanes - 1)) == 0;
  float2* tab = smem;
  const T* x = static_cast<const T*>(side.x);
  const T* dy = static_cast<const T*>(side.dy);
  T* dx = static_cast<T*>(side.dx);
  float wa[V], wb[V], w_odd = 1.f;
  if (side.w) {
    load_w<V, IL>(side.w, s, wa, wb);
    if (k.odd) w_odd = side.w[k.d - 1];
  }
  float da[V], db[V], d_odd = 0.f;
#pragma unroll
  for (int e = 0; e < V; ++e) da[e] = db[e] = 0.f;

  for (int64_t tile = block; tile < side.tiles; tile += blocks) {
    const Rows rows = rows_of(tile * per, per, side.heads);
    T v[U][2 * V], gv[U][2 * V];
    T odd[U], godd[U];
    int64_t at[U];
    int lrow[U];
    bool on[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = rows.at + ((u * kRopeThreads + tid) >> k.log_lanes);
      lrow[u] = static_cast<int>(static_cast<unsigned>(h) / static_cast<unsigned>(side.heads));
      const int head = h - lrow[u] * side.heads;
      const int64_t row = rows.first + lrow[u];
      on[u] = s.live && row < k.n;
      const int64_t from = on[u] ? row * side.x_stride + head * k.d : 0;
      const int64_t gfrom = on[u] ? row * side.dy_stride + head * k.d : 0;
      at[u] = row * side.dx_stride + head * k.d;
      if (side.w) {
        load2<T, V>(x + from, s, v[u]);
        odd[u] = k.odd ? x[from + k.d - 1] : static_cast<T>(0.f);
      }
      load2<T, V>(dy + gfrom, s, gv[u]);
      godd[u] = k.odd ? dy[gfrom + k.d - 1] : static_cast<T>(0.f);
    }
    __syncthreads();  // the table of the tile before has been read
    if (k.table_pairs) fill_angles(k, rows, tab);
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float a[V], b[V];
      to_pairs<T, V, IL>(gv[u], a, b);
      float last = static_cast<float>(godd[u]);
      if (s.pair >= 0 && k.table_pairs) {
        const float2* t = tab + lrow[u] * k.table_pairs + s.pair;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float2 cs = t[e];
          const float p = a[e], q = b[e];
          a[e] = fmaf(p, cs.x, q * cs.y);
          b[e] = fmaf(q, cs.x, -p * cs.y);
        }
      }
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
          const bool mine = on[u] && e >= s.skip;
          const float na = xa[e] * rstd, nb = xb[e] * rstd;
          da[e] = mine ? fmaf(a[e], na, da[e]) : da[e];
          db[e] = mine ? fmaf(b[e], nb, db[e]) : db[e];
          a[e] = fmaf(-na, c, a[e] * wa[e]) * rstd;
          b[e] = fmaf(-nb, c, b[e] * wb[e]) * rstd;
        }
        if (k.odd) {
          const float no = xo * rstd;
          d_odd = on[u] && first ? fmaf(last, no, d_odd) : d_odd;
          last = fmaf(-no, c, last * w_odd) * rstd;
        }
      }
      if (on[u]) {
        store2<T, V, IL>(dx + at[u], s, a, b);
        if (k.odd && first) dx[at[u] + k.d - 1] = static_cast<T>(last);
      }
    }
  }
  if (!side.w) return;

  // the threads of one slot, within the wave, then over the waves
  for (int m = lanes; m < 64; m <<= 1) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      da[e] += __shfl_xor(da[e], m);
      db[e] += __shfl_xor(db[e], m);
    }
    d_odd += __shfl_xor(d_odd, m);
  }
  if ((tid & 63) < lanes && s.live) {
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (e >= s.skip) {
        red[tid >> 6][IL ? s.a + 2 * e : s.a + e] = da[e];
        red[tid >> 6][IL ? s.a + 2 * e + 1 : s.b + e] = db[e];
      }
    if (k.odd && first) red[tid >> 6][k.d - 1] = d_odd;
  }
  __syncthreads();
  float* part = k.part + (static_cast<int64_t>(is_k ? k.blocks_q : 0) + block) * k.d;
  for (int i = tid; i < k.d; i += kRopeThreads) {
    float sum = 0.f;
#pragma unroll
    for (int wv = 0; wv < kRopeThreads / 64; ++wv) sum += red[wv][i];
    part[i] = sum;
  }
}

// dw of a side (blockIdx.y) = sum of its blocks' shares; 16 channels a block, 64 threads each.
__global__ __launch_bounds__(1024) void k_rope_dw(const RopeK k) {
  __shared__ float red[64][17];
  const RopeSide side = k.side[blockIdx.y];
  if (!side.dw) return;
  const int rows = blockIdx.y ? k.blocks_k : k.blocks_q;
  const float* part = k.part + (blockIdx.y ? static_cast<int64_t>(k.blocks_q) * k.d : 0);
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

// Pairs per thread: as many as both the turned and the remaining part of a head hold.
// 16-byte accesses for 16-bit types at 8; below, the same sectors in more instructions.
int pairs_per_thread(const RopeK& k, bool il) {
  const int turned = il ? k.d / 2 : k.pairs, rest = il ? 0 : k.rest;
  for (int v = 8; v > 1; v /= 2)
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
  k.table_pairs = k.pairs == 0 ? 0 : IL ? k.d / 2 : k.pairs;
  // heads of both sides: small calls spread over the card with one item a thread; the table
  // of a side with few heads has many rows and stays within 32 KB
  const int64_t items = k.n * (k.side[0].heads + k.side[1].heads) << k.log_lanes;
  int u = back ? 2 : items <= int64_t{4} * 256 * kRopeThreads ? 1 : 4;
  size_t lds = 0;
  for (;; u /= 2) {
    const int per = kRopeThreads * u >> k.log_lanes;
    int rows = 0;
    for (RopeSide& side : k.side) {
      if (side.heads == 0) continue;
      const int r = (side.heads - 1 + per - 1) / side.heads + 1;
      rows = rows > r ? rows : r;
      side.tiles = ceil_div<int64_t>(k.n * side.heads, per);
    }
    lds = static_cast<size_t>(rows) * k.table_pairs * sizeof(float2);
    if (u == 1 || lds <= 32 * 1024) break;
  }
  if (!back) {
    // at most 2^22 blocks of a side: a launch may have 2^32 threads
    k.blocks_q = static_cast<int>(k.side[0].tiles < (1 << 22) ? k.side[0].tiles : 1 << 22);
    k.blocks_k = static_cast<int>(k.side[1].tiles < (1 << 22) ? k.side[1].tiles : 1 << 22);
  }
  const unsigned grid = static_cast<unsigned>(k.blocks_q + k.blocks_k);
  if (back) {
    if (u == 1)
      k_rope_bwd<T, V, IL, 1><<<grid, kRopeThreads, lds, s>>>(k);
    else
      k_rope_bwd<T, V, IL, 2><<<grid, kRopeThreads, lds, s>>>(k);
  } else if (u == 1) {
    k_rope_fwd<T, V, IL, 1><<<grid, kRopeThreads, lds, s>>>(k);
  } else if (u == 2) {
    k_rope_fwd<T, V, IL, 2><<<grid, kRopeThreads, lds, s>>>(k);
  } else {
    k_rope_fwd<T, V, IL, 4><<<grid, kRopeThreads, lds, s>>>(k);
  }
}

template <typename T, bool IL>
void run(RopeK& k, bool back, hipStream_t s) {
  switch (pairs_per_thread(k, IL)) {
    case 8: return run<T, 8, IL>(k, back, s);
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
  else
    k.blocks_q = k.blocks_k = 0;
  if (k.side[0].dw || k.side[1].dw) k_rope_dw<<<dim3(ceil_div(k.d, 16), 2), 1024, 0, s>>>(k);
  return hipGetLastError();
}

}  // namespace ts
