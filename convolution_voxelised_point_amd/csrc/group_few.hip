// Products grouped by expert for few rows an expert: serving single tokens and small batches
// (forward), and the input gradient of the same sizes (group_few says which).
//
// The weights are all there is to read, so they go straight from memory to the registers of
// the matrix instructions, each once per 16 MT rows.  A wave multiplies up to 16 MT rows
// with 128 columns over its share of the reduction; the 8 waves of a block take turns along
// it and add up in LDS.
//   forward: a lane reads 8 columns of 8 consecutive rows of W, and 32 byte permutes turn that
//     into fragments of 8 rows of one column; column j of every lane's 8 makes matrix
//     instruction j.
//   input gradient: rows of W run along the reduction and are fragments as they lie.
//
// One row to 2 of 8 experts, 256 -> 2 x 512, fp16: 5 us, the latency of one load and one sum.  8
// experts of 2048 x 2048, 24 rows each: 22.5 us (67 MB, 3 TB/s).
#include "group.h"

namespace ts {
namespace {

constexpr int kWaves = 8, kCols = 128, kPitch = kCols + 4;

template <typename T>
struct __attribute__((packed, aligned(2))) Few8 {
  T e[8];
};
// Values c0..c0+7 of a row of `width`, zeros past it.
template <typename T, bool VEC>
__device__ __forceinline__ gu32x4 load8(const T* row, int c0, int width) {
  if (c0 + 8 <= width) {
    if (VEC) return *reinterpret_cast<const gu32x4*>(row + c0);
    return __builtin_bit_cast(gu32x4, *reinterpret_cast<const Few8<T>*>(row + c0));
  }
  if (VEC || c0 >= width) return gu32x4{0u, 0u, 0u, 0u};
  T v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = c0 + i < width ? row[c0 + i] : static_cast<T>(0.f);
  return __builtin_bit_cast(gu32x4, v);
}

template <typename T, GroupOp OP, bool GLU, int MT, bool VEC>
__global__ __launch_bounds__(kWaves * 64) void k_group_few(const GroupK k) {
  __shared__ float red[kWaves][16][kPitch];
  constexpr int BM = 16 * MT;
  constexpr bool PAIR = GLU && OP == kGroupFwd;  // 64 columns of a, 64 of b
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, c16 = lane & 15;
  __shared__ GroupLane lanes[64];
  const GroupFinder<false> finder(k, BM, lanes);
  const GroupBlock block = group_block(finder.total, k.n_tiles);
  const int N = OP == kGroupDgrad ? k.cin : k.cout, K = OP == kGroupDgrad ? k.cout : k.cin;
  constexpr int kOut = PAIR ? kCols / 2 : kCols;
  T* y = static_cast<T*>(k.y);
  if (block.at < 0) {
    if (block.spare < 0) return;
    const int64_t run = block.spare / k.n_tiles;
    const GroupRest rest = rows_unowned(k);
    if (run * BM < rest.n) zero_results<T, OP, GLU>(k, rest, run * BM, BM, N, static_cast<int>(block.spare - run * k.n_tiles) * kOut, kOut);
    return;
  }
  const int64_t run = block.at / k.n_tiles;
  const int n0 = static_cast<int>(block.at - run * k.n_tiles) * kOut;
  const GroupTile t = finder.find(k, run);
  if (t.e < 0) return;
  const T* wt = static_cast<const T*>(k.w) + static_cast<int64_t>(t.e) * k.cin * k.ldw;

  // this lane's rows of x (or dy)
  const T* px[MT];
  bool ok[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int r = i * 16 + c16;
    const int64_t row = t.row0 + (r < t.rows ? r : 0);
    int64_t src = row;
    if (OP == kGroupFwd && k.rows) {
      src = k.rows[row];
      if (src < 0 || src >= k.n_src) {
        if (k.flags) atomicOr(k.flags, TS_FLAG_RANGE);
        src = -1;
      }
    }
    ok[i] = src >= 0;
    px[i] = static_cast<const T*>(OP == kGroupFwd ? k.x : k.dy) + (src < 0 ? 0 : src) * K;
  }
  // forward: this lane's 8 columns; of b behind those of a
  int col = 0, width = 0;
  if (OP == kGroupFwd) {
    const int c = n0 + (PAIR ? c16 & 7 : c16) * 8;
    col = PAIR && c16 >= 8 ? c + k.cout : c;
    width = c >= k.cout ? 0 : PAIR && c16 >= 8 ? k.ldw : k.cout;
  }

  gf32x4 acc[MT][8];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = gf32x4{0.f, 0.f, 0.f, 0.f};

  auto load_w = [&](int s, gu32x4 (&w)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (OP == kGroupFwd) {
        const int r = s * 32 + 8 * g + i;
        w[i] = r < K ? load8<T, VEC>(wt + static_cast<int64_t>(r) * k.ldw, col, width) : gu32x4{0u, 0u, 0u, 0u};
      } else {
        const int n = n0 + i * 16 + c16;
        w[i] = n < N ? load8<T, VEC>(wt + static_cast<int64_t>(n) * k.ldw, s * 32 + 8 * g, K) : gu32x4{0u, 0u, 0u, 0u};
      }
    }
  };
  auto load_x = [&](int s, gu32x4 (&x)[MT]) {
#pragma unroll
    for (int i = 0; i < MT; ++i) x[i] = ok[i] ? load8<T, VEC>(px[i], s * 32 + 8 * g, K) : gu32x4{0u, 0u, 0u, 0u};
  };
  const int steps = ceil_div(K, 32);
  gu32x4 w[8], x[MT];
  if (wave < steps) {
    load_w(wave, w);
    load_x(wave, x);
  }
  for (int s = wave; s < steps; s += kWaves) {
    gu32x4 w1[8], x1[MT];
    const bool more = s + kWaves < steps;
    if (more) {
      load_w(s + kWaves, w1);
      load_x(s + kWaves, x1);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      gu32x4 f = w[j];
      if (OP == kGroupFwd) {
        constexpr unsigned lo = 0x05040100u, hi = 0x07060302u;
#pragma unroll
        for (int d = 0; d < 4; ++d) f[d] = __builtin_amdgcn_perm(w[2 * d + 1][j >> 1], w[2 * d][j >> 1], j & 1 ? hi : lo);
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) acc[i][j] = GMfma<T>::run(f, x[i], acc[i][j]);
    }
    if (more) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = w1[i];
#pragma unroll
      for (int i = 0; i < MT; ++i) x[i] = x1[i];
    }
  }

#pragma unroll
  for (int i = 0; i < MT; ++i) {
    // lane (g, c16), element r: row c16; column 8 (4g + r) + j, or 16 j + 4g + r
    if (i > 0) __syncthreads();
    float* mine = red[wave][c16];
    if (OP == kGroupFwd) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        *reinterpret_cast<gf32x4*>(mine + 8 * (4 * g + r)) = gf32x4{acc[i][0][r], acc[i][1][r], acc[i][2][r], acc[i][3][r]};
        *reinterpret_cast<gf32x4*>(mine + 8 * (4 * g + r) + 4) = gf32x4{acc[i][4][r], acc[i][5][r], acc[i][6][r], acc[i][7][r]};
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) *reinterpret_cast<gf32x4*>(mine + 16 * j + 4 * g) = acc[i][j];
    }
    __syncthreads();
    const int part = kOut / 4, r = tid / part, n = tid % part * 4;  // 4 columns a thread
    const int64_t row = t.row0 + i * 16 + r;
    if (r >= 16 || i * 16 + r >= t.rows || n0 + n >= N) continue;
    gf32x4 a{0.f, 0.f, 0.f, 0.f}, b = a;
#pragma unroll
    for (int v = 0; v < kWaves; ++v) {
      a += *reinterpret_cast<const gf32x4*>(&red[v][r][n]);
      if (PAIR) b += *reinterpret_cast<const gf32x4*>(&red[v][r][kCols / 2 + n]);
    }
    typedef T t4 __attribute__((ext_vector_type(4)));
    auto store = [&](T* p, gf32x4 v) {
      if (VEC) {
        *reinterpret_cast<t4*>(p + n0 + n) = __builtin_convertvector(v, t4);
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (n0 + n + q < N) p[n0 + n + q] = static_cast<T>(v[q]);
      }
    };
    if (PAIR) {
      gf32x4 v;
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = a[q] * sigmoid(a[q]) * b[q];
      store(y + row * N, v);
      if (k.h_out) {
        T* h = static_cast<T*>(k.h_out) + row * 2 * N;
        store(h, a);
        store(h + N, b);
      }
    } else if (GLU) {
      const T* h = static_cast<const T*>(k.h) + row * 2 * N + n0 + n;
      gf32x4 da, db;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const bool in = VEC || n0 + n + q < N;
        const float p = in ? static_cast<float>(h[q]) : 0.f, o = in ? static_cast<float>(h[N + q]) : 0.f, s = sigmoid(p);
        da[q] = a[q] * o * s * fmaf(p, 1.f - s, 1.f);
        db[q] = a[q] * p * s;
      }
      store(y + row * 2 * N, da);
      store(y + row * 2 * N + N, db);
    } else {
      store(y + row * N, a);
    }
  }
}

template <typename T, GroupOp OP, bool GLU, int MT>
void run(GroupK& k, bool whole, hipStream_t s) {
  const int N = OP == kGroupDgrad ? k.cin : k.cout;
  k.n_tiles = ceil_div(N, GLU && OP == kGroupFwd ? kCols / 2 : kCols);
  const unsigned grid = static_cast<unsigned>(group_grid(group_runs(k.n_rows, k.e, 16 * MT), k.n_tiles));
  if (whole)
    k_group_few<T, OP, GLU, MT, true><<<grid, kWaves * 64, 0, s>>>(k);
  else
    k_group_few<T, OP, GLU, MT, false><<<grid, kWaves * 64, 0, s>>>(k);
}

template <typename T, GroupOp OP, bool GLU>
void run(GroupK& k, hipStream_t s) {
  const GroupForm f = form_of(k, OP, GLU);
  if (f.rows == 16) run<T, OP, GLU, 1>(k, f.whole, s);
  else
    run<T, OP, GLU, 2>(k, f.whole, s);
}

template <typename T>
void run(GroupK& k, GroupOp op, bool glu, hipStream_t s) {
  if (op == kGroupFwd) return glu ? run<T, kGroupFwd, true>(k, s) : run<T, kGroupFwd, false>(k, s);
  glu ? run<T, kGroupDgrad, true>(k, s) : run<T, kGroupDgrad, false>(k, s);
}

}  // namespace

hipError_t launch_group_few(GroupK& k, GroupOp op, ts_dtype dt, bool glu, hipStream_t s) {
  if (dt == TS_F16) run<_Float16>(k, op, glu, s);
  else
    run<__bf16>(k, op, glu, s);
  return hipGetLastError();
}

}  // namespace ts
