// Router of rows to experts (ts_route_fwd) and its backward pass.
//
// A row's `top` largest logits are picked one after the other: the threads of a row hold
// 8 experts each and agree on the largest.  Values are compared as integers that order like
// the floats (-0 made 0, NaN above infinity); 16-bit ones share a word with their expert's number,
// so that one maximum finds both and the lowest expert wins among equals.  Gates are a softmax
// in fp32.
//
// The chosen pairs (row, j) are then put in order of their expert, by a counting sort
// without atomics on memory: blocks own runs of rows and count their pairs per expert, a
// block per expert adds up these counts, and every block gives its pairs their places, wave
// after wave, by counting the lanes before that chose the same expert.  Pairs without an
// expert form one more bucket behind the last.  Small calls do all of it in one block.
//
// 304,878 rows of 64 bf16 logits, top 2 over all experts: 29 us for the picks, 4.7 and 8 for the places, 21 for the
// gradient (4.2 TB/s).  Reading the logits is 8 us of the 29; the rest is vector instructions, which take 85% of the
// issue cycles: about 370 for the 8 logits of a thread, 50 of them for each pick, 75 for the exponentials
// over all experts, most of the others to make the keys.  39 rows of 8: 5 us, a chain of loads and passes.
#include "act8.h"
#include "lanes.h"
#include "launch.h"
#include "route.h"

namespace ts {
namespace {

constexpr int kRouteThreads = 1024;
constexpr int kRouteWaves = kRouteThreads / 64;

// A logit as an integer that orders like it; what orders at or below that of -infinity is
// never picked.
template <typename T>
struct Order;
template <>
struct Order<float> {
  static constexpr uint32_t kLow = 0x007fffffu;
  static __device__ __forceinline__ uint32_t of(float z) {
    const uint32_t b = __builtin_bit_cast(uint32_t, z + 0.f);
    return z != z ? ~0u : b & 0x80000000u ? ~b : b | 0x80000000u;
  }
  static __device__ __forceinline__ float value(uint32_t o) {
    return __builtin_bit_cast(float, o == ~0u ? 0x7fc00000u : o & 0x80000000u ? o & 0x7fffffffu : ~o);
  }
};
template <typename T, uint32_t LOW, uint32_t INF>
struct Order16 {
  static constexpr uint32_t kLow = LOW;
  static __device__ __forceinline__ uint32_t of(T z) {
    uint32_t b = __builtin_bit_cast(uint16_t, z);
    b = b == 0x8000u ? 0u : b;
    return (b & 0x7fffu) > INF ? 0xffffu : b & 0x8000u ? ~b & 0xffffu : b | 0x8000u;
  }
  static __device__ __forceinline__ float value(uint32_t o) {
    const uint32_t b = o & 0x8000u ? o & 0x7fffu : ~o & 0xffffu;  // (0xffff stays a NaN)
    return static_cast<float>(__builtin_bit_cast(T, static_cast<uint16_t>(b)));
  }
};
template <>
struct Order<_Float16> : Order16<_Float16, 0x03ffu, 0x7c00u> {};
template <>
struct Order<__bf16> : Order16<__bf16, 0x007fu, 0x7f80u> {};

// Logits c0..c0+7 of a row of c, anything past it.  VEC: whole, aligned units only.  Otherwise the
// last unit is the row's last 8 logits moved down (a branch of its own would break up the whole
// ones' accesses as well).
template <typename T>
struct __attribute__((packed, aligned(sizeof(T)))) LooseLogits {
  T e[8];
};
template <typename T, bool VEC>
__device__ __forceinline__ void load_logits(const T* row, int c0, int c, T (&v)[8]) {
  if (VEC) {
    const Unit<T> u = *reinterpret_cast<const Unit<T>*>(row + c0);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = u.e[e];
  } else if (c < 8) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < c ? row[e] : static_cast<T>(0.f);
  } else {
    const int by = c0 + 8 <= c ? 0 : c0 + 8 - c;
    const LooseLogits<T> u = *reinterpret_cast<const LooseLogits<T>*>(row + c0 - by);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = u.e[e];
#pragma unroll
    for (int m = 4; m > 0; m >>= 1)
#pragma unroll
      for (int e = 0; e + m < 8; ++e) v[e] = by & m ? v[e + m] : v[e];
  }
}

// The largest of the row's keys (0: no expert) and its expert, in all of the row's threads;
// taken out of the keys.
template <typename T>
__device__ __forceinline__ uint32_t take_largest(uint32_t (&key)[8], int first, int lanes, int* expert) {
  uint32_t o = key[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) o = key[i] > o ? key[i] : o;
  o = max_lanes(o, lanes);
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) key[i] = key[i] == o ? 0u : key[i];
    *expert = 0xffff - static_cast<int>(o & 0xffffu);
    return o >> 16;
  } else {
    uint32_t at = ~0u;
#pragma unroll
    for (int i = 7; i >= 0; --i) at = key[i] == o ? static_cast<uint32_t>(first + i) : at;
    at = min_lanes(at, lanes);
    *expert = static_cast<int>(at);
#pragma unroll
    for (int i = 0; i < 8; ++i) key[i] = at == static_cast<uint32_t>(first + i) ? 0u : key[i];
    return o;
  }
}

// Experts and gates of rows [r0, r1): G threads a row (8 experts each).  on_pick(row, j,
// expert) is called once per pair, by one thread.  Every thread of the block calls this;
// zs and es hold a pass's picks, `top` for each of its rows.
template <typename T, bool VEC, typename F>
__device__ __forceinline__ void pick(const RouteK& k, int64_t r0, int64_t r1, float* zs, int16_t* es, F&& on_pick) {
  const int g = 1 << k.log_lanes, lane = threadIdx.x & (g - 1), slot = threadIdx.x >> k.log_lanes;
  const int per = kRouteThreads >> k.log_lanes;
  T z[8], ahead[8];  // logits of this pass and of the next
  auto load = [&](int64_t row, T (&v)[8]) {
    if (row < r1 && lane * 8 < k.e) load_logits<T, VEC>(static_cast<const T*>(k.logits) + row * k.e, lane * 8, k.e, v);
  };
  load(r0 + slot, ahead);
  for (int64_t base = r0; base < r1; base += per) {
    const int64_t row = base + slot;
    const bool on = row < r1;
    uint32_t key[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = ahead[i];
    load(row + per, ahead);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = lane * 8 + i;
      const uint32_t o = Order<T>::of(z[i]);
      key[i] = !on || e >= k.e ? 0u : sizeof(T) == 2 ? o << 16 | (0xffffu - e) : o;
    }
    float best = 0.f, sum = 0.f;
    for (int j = 0; j < k.top; ++j) {
      int at;
      const uint32_t o = take_largest<T>(key, lane * 8, g, &at);
      const bool some = o > Order<T>::kLow;
      const float v = Order<T>::value(o);
      if (j == 0) best = v;
      if (some && !k.over_all) sum += exp_below(v - best);
      if (on && lane == 0) {
        zs[slot * k.top + j] = v;
        es[slot * k.top + j] = static_cast<int16_t>(some ? at : -1);
      }
    }
    if (k.over_all) {
      // (the terms that the backward pass forms again.  With the exponent in one part, off by |d| 1.2 2^-24 at the
      // distance d, 511 experts at 3 to 7 below the largest left its gate off by 8.0 2^-24 at most, instead of
      // 5.9; k_route 28 us instead of 29)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        sum += on && lane * 8 + i < k.e ? exp_below(static_cast<float>(z[i]) - best) : 0.f;
      sum = sum_lanes(sum, g);
    }
    // a row's threads lie in one wave: what its first one wrote is there
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    if (on)
      for (int j = lane; j < k.top; j += g) {
        const int e = es[slot * k.top + j];
        k.experts[row * k.top + j] = e;
        k.gates[row * k.top + j] = e < 0 ? 0.f : exp_below(zs[slot * k.top + j] - best) / sum;
        on_pick(row, j, e);
      }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

// Lanes of the wave that hold the same bucket, out of `live` ones.
__device__ __forceinline__ uint64_t same_bucket(int bucket, int bits, uint64_t live) {
  uint64_t m = live;
  for (int b = 0; b < bits; ++b) {
    const bool set = (bucket >> b) & 1;
    const uint64_t v = __ballot(set);
    m &= set ? v : ~v;
  }
  return m;
}
__device__ __forceinline__ int lanes_before(uint64_t m) {
  return static_cast<int>(__builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(m >> 32), __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(m), 0u)));
}

// Places of the pairs [p0, p1) of this wave, in order; next[bucket] is where the bucket's
// next pair goes (LDS, this wave's own).
template <typename E>
__device__ __forceinline__ void give_places(const RouteK& k, int64_t p0, int64_t p1, const E& expert_of, int32_t* next) {
  const int lane = threadIdx.x & 63;
  for (int64_t b = p0; b < p1; b += 64) {
    const int64_t p = b + lane;
    const bool on = p < p1;
    const int e = on ? expert_of(p) : 0;
    const int bucket = e < 0 ? k.e : e;
    const uint64_t m = same_bucket(bucket, k.bits, __ballot(on));
    const int before = lanes_before(m);
    if (on) {
      const int64_t at = next[bucket] + before;
      k.rows[at] = e < 0 ? -1 : static_cast<int32_t>(p / k.top);
      k.place[p] = e < 0 ? -1 : static_cast<int32_t>(at);
    }
    __builtin_amdgcn_wave_barrier();
    if (on && before == 0) next[bucket] += __popcll(m);
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }
}

struct Span {
  int64_t a, b;
};
// Run `i` of `n` things in `parts` parts of equal size (the last ones may be empty).
__device__ __forceinline__ Span span_of(int64_t n, int parts, int i) {
  const int64_t per = (n + parts - 1) / parts;
  const int64_t a = per * i < n ? per * i : n, b = a + per < n ? a + per : n;
  return {a, b};
}

// One block's rows; counts[bucket][block].
template <typename T, bool VEC>
__global__ __launch_bounds__(kRouteThreads) void k_route(const RouteK k) {
  extern __shared__ float zs[];  // [rows of a pass][top], then the experts
  int16_t* es = reinterpret_cast<int16_t*>(zs + (kRouteThreads >> k.log_lanes) * k.top);
  __shared__ int32_t count[kRouteMaxExperts + 1];
  for (int i = threadIdx.x; i <= k.e; i += kRouteThreads) count[i] = 0;
  __syncthreads();
  const Span r = span_of(k.n, k.blocks, blockIdx.x);
  pick<T, VEC>(k, r.a, r.b, zs, es, [&](int64_t, int, int e) { atomicAdd(&count[e < 0 ? k.e : e], 1); });
  __syncthreads();
  for (int i = threadIdx.x; i <= k.e; i += kRouteThreads) k.counts[static_cast<int64_t>(i) * k.blocks + blockIdx.x] = count[i];
}

__device__ __forceinline__ int32_t scan_inclusive(int32_t x) {
  const int lane = threadIdx.x & 63;
  for (int m = 1; m < 64; m <<= 1) {
    const int32_t y = __shfl_up(x, m);
    if (lane >= m) x += y;
  }
  return x;
}

// counts[bucket][block] -> the pairs of the bucket in the blocks before; their number behind them.
__global__ __launch_bounds__(256) void k_route_scan(const RouteK k) {
  static_assert(kRouteMaxBlocks <= 2 * 256, "two counts a thread");
  __shared__ int32_t wave_sum[4];
  int32_t* row = k.counts + static_cast<int64_t>(blockIdx.x) * k.blocks;
  const int wave = threadIdx.x >> 6, at = static_cast<int>(threadIdx.x) * 2;
  const int32_t a = at < k.blocks ? row[at] : 0, b = at + 1 < k.blocks ? row[at + 1] : 0;
  const int32_t inc = scan_inclusive(a + b);
  if ((threadIdx.x & 63) == 63) wave_sum[wave] = inc;
  __syncthreads();
  int32_t sum = inc - a - b, all = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    sum += w < wave ? wave_sum[w] : 0;
    all += wave_sum[w];
  }
  if (at < k.blocks) row[at] = sum;
  if (at + 1 < k.blocks) row[at + 1] = sum + a;
  if (threadIdx.x == 0) k.counts[static_cast<int64_t>(k.e + 1) * k.blocks + blockIdx.x] = all;
}

// Places of one block's pairs.
__global__ __launch_bounds__(kRouteThreads) void k_route_place(const RouteK k) {
  extern __shared__ int32_t next[];  // [waves][e + 1]
  __shared__ int32_t base[kRouteMaxExperts + 1];
  const int wave = threadIdx.x >> 6, buckets = k.e + 1;
  const Span r = span_of(k.n, k.blocks, blockIdx.x);
  const Span mine = span_of((r.b - r.a) * k.top, kRouteWaves, wave);
  const int64_t p0 = r.a * k.top + mine.a, p1 = r.a * k.top + mine.b;
  for (int i = threadIdx.x; i < kRouteWaves * buckets; i += kRouteThreads) next[i] = 0;
  __syncthreads();
  for (int64_t p = p0 + (threadIdx.x & 63); p < p1; p += 64) {
    const int e = k.experts[p];
    atomicAdd(&next[wave * buckets + (e < 0 ? k.e : e)], 1);
  }
  if (wave == 0) {  // first places of the buckets
    int32_t carry = 0;
    for (int b0 = 0; b0 < buckets; b0 += 64) {
      const int b = b0 + static_cast<int>(threadIdx.x);
      const int32_t c = b < buckets ? k.counts[static_cast<int64_t>(buckets) * k.blocks + b] : 0;
      const int32_t inc = scan_inclusive(c);
      if (b < buckets) {
        base[b] = carry + inc - c;
        if (blockIdx.x == 0) k.starts[b] = carry + inc - c;
      }
      carry += __shfl(inc, 63);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < buckets; i += kRouteThreads) {
    int32_t at = base[i] + k.counts[static_cast<int64_t>(i) * k.blocks + blockIdx.x];
    for (int w = 0; w < kRouteWaves; ++w) {
      const int32_t c = next[w * buckets + i];
      next[w * buckets + i] = at;
      at += c;
    }
  }
  __syncthreads();
  give_places(k, p0, p1, [&](int64_t p) { return k.experts[p]; }, next + wave * buckets);
}

// All of it in one block, for calls of at most kRouteSmall pairs.
template <typename T, bool VEC>
__global__ __launch_bounds__(kRouteThreads) void k_route_small(const RouteK k) {
  __shared__ float zs[kRouteSmall];
  __shared__ int16_t es[kRouteSmall];
  __shared__ int16_t expert[kRouteSmall];
  __shared__ int32_t base[kRouteMaxExperts + 2];
  extern __shared__ int32_t next[];  // [waves][e + 1]
  const int wave = threadIdx.x >> 6, buckets = k.e + 1;
  for (int i = threadIdx.x; i < kRouteWaves * buckets; i += kRouteThreads) next[i] = 0;
  __syncthreads();
  const int pairs = static_cast<int>(k.n) * k.top;
  const int per = ceil_div(pairs, kRouteWaves);
  pick<T, VEC>(k, 0, k.n, zs, es, [&](int64_t row, int j, int e) {
    const int p = static_cast<int>(row) * k.top + j;
    expert[p] = static_cast<int16_t>(e);
    atomicAdd(&next[p / per * buckets + (e < 0 ? k.e : e)], 1);
  });
  __syncthreads();
  if (wave == 0) {  // first places of the buckets
    int32_t carry = 0;
    for (int b0 = 0; b0 < buckets; b0 += 64) {
      const int b = b0 + static_cast<int>(threadIdx.x);
      int32_t c = 0;
      if (b < buckets)
        for (int w = 0; w < kRouteWaves; ++w) c += next[w * buckets + b];
      const int32_t inc = scan_inclusive(c);
      if (b < buckets) {
        base[b] = carry + inc - c;
        k.starts[b] = carry + inc - c;
      }
      carry += __shfl(inc, 63);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < buckets; i += kRouteThreads) {
    int32_t at = base[i];
    for (int w = 0; w < kRouteWaves; ++w) {
      const int32_t c = next[w * buckets + i];
      next[w * buckets + i] = at;
      at += c;
    }
  }
  __syncthreads();
  const Span mine = span_of(pairs, kRouteWaves, wave);
  give_places(k, mine.a, mine.b, [&](int64_t p) { return static_cast<int>(expert[p]); }, next + wave * buckets);
}

// dlogits: with normalised gates g_j (dg_j - sum g dg) at the chosen experts, else
// [chosen] g_j dg_j - p sum g dg at all of them, p = softmax(logits) = g_0 exp(logits - the largest).
template <typename T, bool VEC>
__global__ __launch_bounds__(256) void k_route_bwd(const RouteK k) {
  const int g = 1 << k.log_lanes, lane = threadIdx.x & (g - 1);
  const int64_t step = static_cast<int64_t>(gridDim.x) * (256 >> k.log_lanes);
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * (256 >> k.log_lanes) + (threadIdx.x >> k.log_lanes); row < k.n; row += step) {
    const T* logits = static_cast<const T*>(k.logits) + row * k.e;
    T z[8];
    float d[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) d[i] = 0.f;
    if (k.over_all && lane * 8 < k.e) load_logits<T, VEC>(logits, lane * 8, k.e, z);
    float inner = 0.f;
    bool some = false;
    for (int j = 0; j < k.top; ++j) {
      const int64_t p = row * k.top + j;
      if (k.experts[p] < 0) continue;
      some = true;
      inner = fmaf(k.gates[p], k.dgates[p], inner);
    }
    if (some) {  // the same in all of the row's threads
      for (int j = 0; j < k.top; ++j) {
        const int64_t p = row * k.top + j;
        const int e = k.experts[p];
        const float x = k.gates[p] * (k.over_all ? k.dgates[p] : k.dgates[p] - inner);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (e == lane * 8 + i) d[i] += x;
      }
      if (k.over_all) {
        // the first expert has the largest logit, and its gate is 1 over the softmax's sum
        const int64_t p = row * k.top;
        const int top1 = k.experts[p];
        const float best = static_cast<float>(logits[top1 < 0 ? 0 : top1 < k.e ? top1 : k.e - 1]), c = inner * k.gates[p];
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = fmaf(-exp_below(static_cast<float>(z[i]) - best), c, d[i]);
      }
    }
    if (lane * 8 < k.e) store_unit(static_cast<T*>(k.dlogits) + row * k.e, lane * 8, k.e, VEC, d);
  }
}

template <typename T, bool VEC>
void run(const RouteK& k, bool back, hipStream_t s) {
  if (back) {
    const int64_t b = ceil_div<int64_t>(k.n, 256 >> k.log_lanes), most = int64_t{1} << 23;
    k_route_bwd<T, VEC><<<static_cast<unsigned>(b < most ? b : most), 256, 0, s>>>(k);
    return;
  }
  const size_t lds = static_cast<size_t>(kRouteWaves) * (k.e + 1) * sizeof(int32_t);
  if (route_small(k.n, k.e, k.top)) {
    k_route_small<T, VEC><<<1, kRouteThreads, lds, s>>>(k);
    return;
  }
  const size_t picks = static_cast<size_t>(kRouteThreads >> k.log_lanes) * k.top * 6;  // at most 48 KB
  k_route<T, VEC><<<k.blocks, kRouteThreads, picks, s>>>(k);
  k_route_scan<<<k.e + 1, 256, 0, s>>>(k);
  k_route_place<<<k.blocks, kRouteThreads, lds, s>>>(k);
}

}  // namespace

hipError_t launch_route(RouteK& k, ts_dtype dt, bool back, hipStream_t s) {
  if (k.n == 0) return back ? hipSuccess : fill_i64(k.starts, k.e + 1, 0, s);
  k.log_lanes = route_log_lanes(k.e);
  k.bits = 1;
  while ((1 << k.bits) < k.e + 1) ++k.bits;
  const bool vec = k.e % 8 == 0 && ((reinterpret_cast<uintptr_t>(k.logits) | reinterpret_cast<uintptr_t>(k.dlogits)) & 15) == 0;
  k.blocks = route_blocks(k.n, k.e);
  switch (dt) {
    case TS_F32: vec ? run<float, true>(k, back, s) : run<float, false>(k, back, s); break;
    case TS_F16: vec ? run<_Float16, true>(k, back, s) : run<_Float16, false>(k, back, s); break;
    default: vec ? run<__bf16, true>(k, back, s) : run<__bf16, false>(k, back, s); break;
  }
  return hipGetLastError();
}

}  // namespace ts
