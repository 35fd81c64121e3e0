// Sum of what a row's experts returned (ts_combine_fwd) and its backward pass.
//
//   out[t] = sum_j gates[t][j] y[place[t][j]]
//   dy[place[t][j]] = gates[t][j] dout[t],   dgates[t][j] = <dout[t], y[place[t][j]]>
//
// Memory bound: every grouped row is read (and written) once; a thread owns 8 channels
// of a row, so a row is one or a few wide accesses wherever it lies.  Gathering by
// `place` keeps the order of the sum fixed, and needs no atomics.  Sums are fp32.  Results are
// stored past the L2, which nothing reads them from (both passes 119 -> 109 us).
//
// 304,878 rows of 2 experts of 8, 128 channels, bf16: 36 us (239 MB, 6.6 TB/s: part of what the
// products wrote is still in the last-level cache), backward 57 (400 MB, 7.0 TB/s likewise).
#include "act8.h"
#include "lanes.h"
#include "launch.h"

namespace ts {
namespace {

struct CombineK {
  const void* y;
  const int32_t* place;
  const float* gates;
  const void* dout;
  void *out, *dy;
  float* dgates;
  uint32_t* flags;
  int64_t n, n_rows;
  int top, c, units;
  bool vec, vec_d;  // 16-byte accesses allowed: y, out and dy; dout
};

// Grouped row of (t, j), -1 where there is none.
__device__ __forceinline__ int64_t row_at(const CombineK& k, int64_t t, int j) {
  const int32_t p = k.place[t * k.top + j];
  if (p >= k.n_rows || p < -1) {
    if (k.flags) atomicOr(k.flags, TS_FLAG_RANGE);
    return -1;
  }
  return p;
}

// 8 channels of a result.
template <typename T>
__device__ __forceinline__ void put_unit(T* row, int c0, int c, bool vec, const float (&f)[8]) {
  if (!vec) return store_unit(row, c0, c, vec, f);
  Unit<T> v;
#pragma unroll
  for (int e = 0; e < 8; ++e) v.e[e] = static_cast<T>(f[e]);
  store_once(row + c0, v);
}

// AHEAD grouped rows of a row are read at once: as many as there mostly are, up to 4.
template <typename T, int AHEAD>
__global__ __launch_bounds__(256) void k_combine_fwd(const CombineK k) {
  const int64_t items = k.n * k.units;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < items; i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t t = items <= UINT32_MAX ? static_cast<uint32_t>(i) / static_cast<uint32_t>(k.units) : i / k.units;
    const int c0 = static_cast<int>(i - t * k.units) * 8;
    float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < k.top; j0 += AHEAD) {
      float f[AHEAD][8], g[AHEAD];
      int64_t p[AHEAD];
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        p[j] = j0 + j < k.top ? row_at(k, t, j0 + j) : -1;
        g[j] = p[j] < 0 ? 0.f : k.gates ? k.gates[t * k.top + j0 + j] : 1.f;
      }
#pragma unroll
      for (int j = 0; j < AHEAD; ++j)
        if (p[j] >= 0) load_unit(static_cast<const T*>(k.y) + p[j] * k.c, c0, k.c, k.vec, f[j]);
#pragma unroll
      for (int j = 0; j < AHEAD; ++j)
        if (p[j] >= 0) {
#pragma unroll
          for (int e = 0; e < 8; ++e) sum[e] = fmaf(g[j], f[j][e], sum[e]);
        }
    }
    put_unit(static_cast<T*>(k.out) + t * k.c, c0, k.c, k.vec, sum);
  }
}

// LPR threads own a row; ONE: they hold all of it, and dout is read once.
template <typename T, int LPR, bool ONE>
__global__ __launch_bounds__(256) void k_combine_bwd(const CombineK k) {
  const int lane = threadIdx.x % LPR;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (256 / LPR);
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * (256 / LPR) + threadIdx.x / LPR; t < k.n; t += step) {
    const T* dout = static_cast<const T*>(k.dout) + t * k.c;
    float d[8];
    if (ONE && lane < k.units) load_unit(dout, lane * 8, k.c, k.vec_d, d);
    for (int j = 0; j < k.top; ++j) {
      const int64_t p = row_at(k, t, j);
      float dot = 0.f;
      if (p >= 0) {
        const float g = k.gates[t * k.top + j];
        const T* y = static_cast<const T*>(k.y) + p * k.c;
        T* dy = static_cast<T*>(k.dy) + p * k.c;
        for (int u = lane; u < k.units; u += LPR) {
          float f[8], r[8];
          load_unit(y, u * 8, k.c, k.vec, f);
          if (!ONE) load_unit(dout, u * 8, k.c, k.vec_d, d);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            // (channels past the row's end are zeros of both)
            dot = fmaf(d[e], f[e], dot);
            r[e] = g * d[e];
          }
          put_unit(dy, u * 8, k.c, k.vec, r);
          if (ONE) break;
        }
      }
      dot = sum_lanes(dot, LPR);
      if (lane == 0) k.dgates[t * k.top + j] = dot;
    }
  }
}

// At most 2^23 blocks (a launch may have 2^32 threads); the kernels step over the rest.
unsigned blocks_for(int64_t n) {
  const int64_t most = int64_t{1} << 23;
  return static_cast<unsigned>(n < most ? n : most);
}

template <typename T, int LPR>
void run_bwd(const CombineK& k, hipStream_t s) {
  const unsigned grid = blocks_for(ceil_div<int64_t>(k.n, 256 / LPR));
  if constexpr (LPR == 64) {
    if (k.units > LPR) {
      k_combine_bwd<T, LPR, false><<<grid, 256, 0, s>>>(k);
      return;
    }
  }
  k_combine_bwd<T, LPR, true><<<grid, 256, 0, s>>>(k);
}

template <typename T>
void run(const CombineK& k, bool back, hipStream_t s) {
  if (!back) {
    const unsigned grid = blocks_for(ceil_div<int64_t>(k.n * k.units, 256));
    if (k.top <= 2)
      k_combine_fwd<T, 2><<<grid, 256, 0, s>>>(k);
    else
      k_combine_fwd<T, 4><<<grid, 256, 0, s>>>(k);
    return;
  }
  if (k.units <= 1) return run_bwd<T, 1>(k, s);
  if (k.units <= 4) return run_bwd<T, 4>(k, s);
  if (k.units <= 16) return run_bwd<T, 16>(k, s);
  run_bwd<T, 64>(k, s);
}

void run(const CombineK& k, ts_dtype dt, bool back, hipStream_t s) {
  switch (dt) {
    case TS_F32: return run<float>(k, back, s);
    case TS_F16: return run<_Float16>(k, back, s);
    default: return run<__bf16>(k, back, s);
  }
}

bool at16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

hipError_t launch_combine_fwd(const void* y, int64_t n_rows, const int32_t* place, const float* gates, int64_t n, int top,
                              int c, ts_dtype dt, void* out, uint32_t* flags, hipStream_t s) {
  if (n == 0) return hipSuccess;
  CombineK k{};
  k.y = y;
  k.place = place;
  k.gates = gates;
  k.out = out;
  k.flags = flags;
  k.n = n;
  k.n_rows = n_rows;
  k.top = top;
  k.c = c;
  k.units = ceil_div(c, 8);
  k.vec = c % 8 == 0 && at16(y) && at16(out);
  run(k, dt, false, s);
  return hipGetLastError();
}

hipError_t launch_combine_bwd(const void* dout, const void* y, int64_t n_rows, const int32_t* place, const float* gates,
                              int64_t n, int top, int c, ts_dtype dt, void* dy, float* dgates, uint32_t* flags,
                              hipStream_t s) {
  if (n == 0) return hipSuccess;
  CombineK k{};
  k.y = y;
  k.place = place;
  k.gates = gates;
  k.dout = dout;
  k.dy = dy;
  k.dgates = dgates;
  k.flags = flags;
  k.n = n;
  k.n_rows = n_rows;
  k.top = top;
  k.c = c;
  k.units = ceil_div(c, 8);
  k.vec = c % 8 == 0 && at16(y) && at16(dy);
  k.vec_d = c % 8 == 0 && at16(dout);
  run(k, dt, true, s);
  return hipGetLastError();
}

}  // namespace ts
