// Root-mean-square norm with the residual's addition, forward and backward:
//   h = x + residual (rounded to the feature type: what follows reads that)
//   rstd = 1 / sqrt(mean(h^2) + eps),  y = h rstd w
//   xn = h rstd, g = dy w:  dx = rstd (g - xn mean(g xn)) + dh,  dw = sum over rows of dy xn
// Memory bound: every operand is read once and every result written once.
// Sums are fp32 in a fixed order, without atomics.
//
// Up to 2048 channels, LPR lanes hold a row (64 / LPR rows per wave), each 8
// channels in VPL places, so the row never leaves the registers; dw is summed
// per lane over the block's rows, then over blocks by a second kernel.  Wider
// rows take a block each and are read twice.
//
// Measured: 304,878 x 128 bf16 with residual and an 8-bit h, forward 60 us (354 MB, 5.9
// TB/s), backward from the 8 bits 61 + 5 us (273 MB, 4.5 TB/s); 102,835 x 77 fp32,
// forward 28 us (127 MB, 4.5 TB/s), backward 26 + 4 us (127 MB, 4.9 TB/s).  A copy
// of 2 GiB runs at 5.0 TB/s, one that fits the last-level cache at 6.3 to 7.1.
#include "act8.h"
#include "launch.h"

namespace ts {

namespace {

struct NormK {
  const void *x, *res, *dy, *h, *dh;
  const float *w, *rstd_in;
  void *h_out, *y, *dx;
  float *rstd, *dw;
  Act8 y8, h8;
  int64_t n;
  int c;
  float eps, inv_c;
  bool vec, wvec;
};

template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int d = LPR / 2; d > 0; d >>= 1) x += __shfl_xor(x, d);
  return x;
}

template <typename T, int LPR, int VPL>
__global__ __launch_bounds__(256) void k_norm_fwd(const NormK a) {
  constexpr int ROWS = 256 / LPR;
  const int lane = threadIdx.x % LPR;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * ROWS; r0 < a.n; r0 += static_cast<int64_t>(gridDim.x) * ROWS) {
    const int64_t r = r0 + threadIdx.x / LPR;
    const bool ok = r < a.n;
    const int64_t row = ok ? r : 0;
    const T* x = static_cast<const T*>(a.x) + row * a.c;
    float f[VPL][8], sq = 0.f;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int c0 = (v * LPR + lane) * 8;
      load_unit(x, c0, a.c, a.vec, f[v]);
      if (a.res) {
        float g[8];
        load_unit(static_cast<const T*>(a.res) + row * a.c, c0, a.c, a.vec, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[v][e] = static_cast<float>(static_cast<T>(f[v][e] + g[e]));
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sq = fmaf(f[v][e], f[v][e], sq);
    }
    sq = row_sum<LPR>(sq);
    const float rstd = 1.f / sqrtf(fmaf(sq, a.inv_c, a.eps));
    if (ok && lane == 0 && a.rstd) a.rstd[row] = rstd;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int c0 = (v * LPR + lane) * 8;
      if (ok && a.h_out) store_unit(static_cast<T*>(a.h_out) + row * a.c, c0, a.c, a.vec, f[v]);
      if (a.h8.codes) {
        uint32_t byte;
        const ux2 codes = act8_encode(f[v], &byte);
        if (ok) act8_store(a.h8, row, c0, a.c, codes, byte);
      }
      float w[8], y[8];
      load_unit(a.w, c0, a.c, a.wvec, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = f[v][e] * rstd * w[e];
      if (ok && a.y) store_unit(static_cast<T*>(a.y) + row * a.c, c0, a.c, a.vec, y);
      if (a.y8.codes) {
        uint32_t byte;
        const ux2 codes = act8_encode(y, &byte);
        if (ok) act8_store(a.y8, row, c0, a.c, codes, byte);
      }
    }
  }
}

template <typename T, int LPR, int VPL>
__global__ __launch_bounds__(256) void k_norm_bwd(const NormK a) {
  constexpr int ROWS = 256 / LPR;
  __shared__ float part[ROWS > 1 ? ROWS : 1][LPR * 8 + 4];
  const int lane = threadIdx.x % LPR, sub = threadIdx.x / LPR;
  float w[VPL][8], dw[VPL][8];
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    load_unit(a.w, (v * LPR + lane) * 8, a.c, a.wvec, w[v]);
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[v][e] = 0.f;
  }
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * ROWS; r0 < a.n; r0 += static_cast<int64_t>(gridDim.x) * ROWS) {
    const int64_t r = r0 + sub;
    const bool ok = r < a.n;
    const int64_t row = ok ? r : 0;
    const float rstd = ok ? a.rstd_in[row] : 0.f;
    float xn[VPL][8], g[VPL][8], dot = 0.f;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int c0 = ok ? (v * LPR + lane) * 8 : a.c;
      if (a.h8.codes)
        act8_load(a.h8, row, c0, a.c, xn[v]);
      else
        load_unit(static_cast<const T*>(a.h) + row * a.c, c0, a.c, a.vec, xn[v]);
      load_unit(static_cast<const T*>(a.dy) + row * a.c, c0, a.c, a.vec, g[v]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        xn[v][e] *= rstd;
        dw[v][e] = fmaf(g[v][e], xn[v][e], dw[v][e]);
        g[v][e] *= w[v][e];
        dot = fmaf(g[v][e], xn[v][e], dot);
      }
    }
    dot = row_sum<LPR>(dot) * a.inv_c;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int c0 = ok ? (v * LPR + lane) * 8 : a.c;
      float dx[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) dx[e] = rstd * fmaf(-xn[v][e], dot, g[v][e]);
      if (a.dh) {
        float d[8];
        load_unit(static_cast<const T*>(a.dh) + row * a.c, c0, a.c, a.vec, d);
#pragma unroll
        for (int e = 0; e < 8; ++e) dx[e] += d[e];
      }
      store_unit(static_cast<T*>(a.dx) + row * a.c, c0, a.c, a.vec, dx);
    }
  }
  // the block's dw: over the rows that share a lane's channels, in order
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) part[sub][lane * 8 + e] = dw[v][e];
    __syncthreads();
    for (int i = threadIdx.x; i < LPR * 8; i += 256) {
      float s = 0.f;
#pragma unroll
      for (int x = 0; x < ROWS; ++x) s += part[x][i];
      const int c = v * LPR * 8 + i;
      if (c < a.c) a.dw[static_cast<int64_t>(blockIdx.x) * a.c + c] = s;
    }
  }
}

// Sum over the block of one value per thread.
__device__ __forceinline__ float block_sum(float x, float* red) {
  x = row_sum<64>(x);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
  __syncthreads();
  return (red[0] + red[1]) + (red[2] + red[3]);
}

// Rows of more than 2048 channels: a block per row.
template <typename T>
__global__ __launch_bounds__(256) void k_norm_fwd_wide(const NormK a) {
  __shared__ float red[4];
  const int units = ceil_div(a.c, kActBlock) * 4;  // whole blocks: the lanes of a block stay together
  auto load_h = [&](int64_t row, int c0, float(&f)[8]) {
    load_unit(static_cast<const T*>(a.x) + row * a.c, c0, a.c, a.vec, f);
    if (a.res) {
      float g[8];
      load_unit(static_cast<const T*>(a.res) + row * a.c, c0, a.c, a.vec, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = static_cast<float>(static_cast<T>(f[e] + g[e]));
    }
  };
  for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x) {
    float sq = 0.f;
    for (int u = threadIdx.x; u < units; u += 256) {
      float f[8];
      load_h(row, u * 8, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) sq = fmaf(f[e], f[e], sq);
    }
    const float rstd = 1.f / sqrtf(fmaf(block_sum(sq, red), a.inv_c, a.eps));
    if (threadIdx.x == 0 && a.rstd) a.rstd[row] = rstd;
    for (int u = threadIdx.x; u < units; u += 256) {
      float f[8], w[8], y[8];
      uint32_t byte;
      load_h(row, u * 8, f);
      load_unit(a.w, u * 8, a.c, a.wvec, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = f[e] * rstd * w[e];
      if (a.h8.codes) {
        const ux2 codes = act8_encode(f, &byte);
        act8_store(a.h8, row, u * 8, a.c, codes, byte);
      }
      if (a.y8.codes) {
        const ux2 codes = act8_encode(y, &byte);
        act8_store(a.y8, row, u * 8, a.c, codes, byte);
      }
      // last, since h or y may lie where x or the residual does
      if (a.h_out) store_unit(static_cast<T*>(a.h_out) + row * a.c, u * 8, a.c, a.vec, f);
      if (a.y) store_unit(static_cast<T*>(a.y) + row * a.c, u * 8, a.c, a.vec, y);
    }
  }
}

template <typename T>
__device__ __forceinline__ void load_xn(const NormK& a, int64_t row, int c0, float rstd, float (&xn)[8]) {
  if (a.h8.codes)
    act8_load(a.h8, row, c0, a.c, xn);
  else
    load_unit(static_cast<const T*>(a.h) + row * a.c, c0, a.c, a.vec, xn);
#pragma unroll
  for (int e = 0; e < 8; ++e) xn[e] *= rstd;
}

template <typename T>
__global__ __launch_bounds__(256) void k_norm_bwd_wide(const NormK a) {
  __shared__ float red[4];
  const int units = ceil_div(a.c, 8);
  for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x) {
    const float rstd = a.rstd_in[row];
    float dot = 0.f;
    for (int u = threadIdx.x; u < units; u += 256) {
      float xn[8], g[8], w[8];
      load_xn<T>(a, row, u * 8, rstd, xn);
      load_unit(static_cast<const T*>(a.dy) + row * a.c, u * 8, a.c, a.vec, g);
      load_unit(a.w, u * 8, a.c, a.wvec, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) dot = fmaf(g[e] * w[e], xn[e], dot);
    }
    dot = block_sum(dot, red) * a.inv_c;
    for (int u = threadIdx.x; u < units; u += 256) {
      float xn[8], g[8], w[8], dx[8];
      load_xn<T>(a, row, u * 8, rstd, xn);
      load_unit(static_cast<const T*>(a.dy) + row * a.c, u * 8, a.c, a.vec, g);
      load_unit(a.w, u * 8, a.c, a.wvec, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) dx[e] = rstd * fmaf(-xn[e], dot, g[e] * w[e]);
      if (a.dh) {
        float d[8];
        load_unit(static_cast<const T*>(a.dh) + row * a.c, u * 8, a.c, a.vec, d);
#pragma unroll
        for (int e = 0; e < 8; ++e) dx[e] += d[e];
      }
      store_unit(static_cast<T*>(a.dx) + row * a.c, u * 8, a.c, a.vec, dx);
    }
  }
}

// dw partials of wide rows: thread = 8 channels, block row = a share of the rows.
template <typename T>
__global__ __launch_bounds__(256) void k_norm_dw_wide(const NormK a) {
  const int c0 = (blockIdx.x * 256 + threadIdx.x) * 8;
  if (c0 >= a.c) return;
  float dw[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int64_t row = blockIdx.y; row < a.n; row += gridDim.y) {
    float xn[8], g[8];
    load_xn<T>(a, row, c0, a.rstd_in[row], xn);
    load_unit(static_cast<const T*>(a.dy) + row * a.c, c0, a.c, a.vec, g);
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[e] = fmaf(g[e], xn[e], dw[e]);
  }
  store_unit(a.dw + static_cast<int64_t>(blockIdx.y) * a.c, c0, a.c, false, dw);
}

// dw = sum of the partials, 16 channels per block and 64 shares of the rows.
__global__ __launch_bounds__(1024) void k_norm_dw(const float* __restrict__ part, int rows, int c,
                                                  float* __restrict__ dw) {
  __shared__ float red[64][17];
  const int x = threadIdx.x & 15, sh = threadIdx.x >> 4, ch = blockIdx.x * 16 + x;
  float s = 0.f;
  if (ch < c)
#pragma unroll 8
    for (int r = sh; r < rows; r += 64) s += part[static_cast<int64_t>(r) * c + ch];
  red[sh][x] = s;
  __syncthreads();
  if (sh != 0 || ch >= c) return;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < 64; ++i) s += red[i][x];
  dw[ch] = s;
}

constexpr int kNormRegChannels = 2048;  // widest row held in registers
constexpr int kNormBlocks = 1024;       // blocks of the backward pass (dw partials)

int lanes_per_row(int c) {
  const int u = ceil_div(c, 8);
  return u <= 4 ? 4 : u <= 8 ? 8 : u <= 16 ? 16 : u <= 32 ? 32 : 64;
}
int bwd_blocks(int64_t n, int c) {
  const int64_t rows = c > kNormRegChannels ? 1 : 256 / lanes_per_row(c);
  const int64_t b = ceil_div<int64_t>(n, rows);
  const int64_t most = c > kNormRegChannels ? 64 : kNormBlocks;
  return static_cast<int>(b < most ? b : most);
}

// At most 2^23 blocks (a launch may have 2^32 threads); the kernels step over the rest.
unsigned grid_rows(int64_t blocks) {
  const int64_t most = int64_t{1} << 23;
  return static_cast<unsigned>(blocks < most ? blocks : most);
}

template <typename T, int LPR, int VPL>
void run(const NormK& a, bool back, hipStream_t s) {
  if (back)
    k_norm_bwd<T, LPR, VPL><<<bwd_blocks(a.n, a.c), 256, 0, s>>>(a);
  else
    k_norm_fwd<T, LPR, VPL><<<grid_rows(ceil_div<int64_t>(a.n, 256 / LPR)), 256, 0, s>>>(a);
}

template <typename T>
void run(const NormK& a, bool back, hipStream_t s) {
  if (a.c > kNormRegChannels) {
    const unsigned n = grid_rows(a.n);
    if (back) {
      k_norm_dw_wide<T><<<dim3(ceil_div(a.c, 2048), bwd_blocks(a.n, a.c)), 256, 0, s>>>(a);  // first: dx may be dy
      k_norm_bwd_wide<T><<<n, 256, 0, s>>>(a);
    } else {
      k_norm_fwd_wide<T><<<n, 256, 0, s>>>(a);
    }
    return;
  }
  switch (lanes_per_row(a.c)) {
    case 4: return run<T, 4, 1>(a, back, s);
    case 8: return run<T, 8, 1>(a, back, s);
    case 16: return run<T, 16, 1>(a, back, s);
    case 32: return run<T, 32, 1>(a, back, s);
  }
  if (a.c <= 512) return run<T, 64, 1>(a, back, s);
  if (a.c <= 1024) return run<T, 64, 2>(a, back, s);
  run<T, 64, 4>(a, back, s);
}

void run(const NormK& a, ts_dtype dt, bool back, hipStream_t s) {
  switch (dt) {
    case TS_F32: return run<float>(a, back, s);
    case TS_F16: return run<_Float16>(a, back, s);
    default: return run<__bf16>(a, back, s);
  }
}

bool at16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

size_t norm_workspace_bytes(int64_t n, int c) { return static_cast<size_t>(bwd_blocks(n, c)) * c * 4; }

hipError_t launch_norm_fwd(const void* x, const void* res, const float* w, int64_t n, int c, float eps, ts_dtype dt,
                           void* h, void* y, float* rstd, const Act8& y8, const Act8& h8, hipStream_t s) {
  if (n == 0) return hipSuccess;
  NormK a{};
  a.x = x;
  a.res = res;
  a.w = w;
  a.n = n;
  a.c = c;
  a.eps = eps;
  a.inv_c = 1.f / static_cast<float>(c);
  a.h_out = h;
  a.y = y;
  a.rstd = rstd;
  a.y8 = y8;
  a.h8 = h8;
  a.vec = c % 8 == 0 && at16(x) && at16(res) && at16(h) && at16(y);
  a.wvec = c % 8 == 0 && at16(w);
  run(a, dt, false, s);
  return hipGetLastError();
}

hipError_t launch_norm_bwd(const void* dy, const void* h, const Act8& h8, const float* w, const float* rstd,
                           const void* dh, int64_t n, int c, ts_dtype dt, void* dx, float* dw, void* ws,
                           hipStream_t s) {
  if (n == 0) return fill_f32(dw, c, 0.f, s);
  NormK a{};
  a.dy = dy;
  a.h = h;
  a.h8 = h8;
  a.w = w;
  a.rstd_in = rstd;
  a.dh = dh;
  a.n = n;
  a.c = c;
  a.inv_c = 1.f / static_cast<float>(c);
  a.dx = dx;
  a.dw = static_cast<float*>(ws);
  a.vec = c % 8 == 0 && at16(dy) && at16(h) && at16(dh) && at16(dx);
  a.wvec = c % 8 == 0 && at16(w);
  run(a, dt, true, s);
  k_norm_dw<<<ceil_div(c, 16), 1024, 0, s>>>(static_cast<const float*>(ws), bwd_blocks(n, c), c, dw);
  return hipGetLastError();
}

}  // namespace ts
