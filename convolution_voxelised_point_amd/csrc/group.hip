// Products grouped by expert on the matrix cores, for many rows an expert (few rows:
// group_few.hip).
//
//   forward          y[p]  = x[rows[p]] W[e]        reduced over cin
//   input gradient   dx[p] = dy[p] W[e]^T           reduced over cout
//   weight gradient  dW[e] = sum over its p of x[rows[p]]^T dy[p]
//
// One kernel for the three: a tile of BM x BN results is reduced over steps of 32.  Both
// operands' steps are copied straight into LDS (16 bytes a lane, no registers), four
// steps in a ring, three of them in flight while one is multiplied, so a step takes one
// barrier.  An operand whose rows run along the reduction (x and dy of the first two, W of
// the second) is read from LDS as it lies; one whose rows run across it is read with the
// transposing LDS reads.  Chunks of 16 bytes are stored xor-ed with their row so that
// neither read meets a bank twice.  Gathered rows cost nothing: every lane names its
// own source anyway.  Sources past the matrix (the last step's, rows that are not there)
// are 16 bytes of zeros.
//
// Tiles are found from the starts on the device, expert by expert, so lengths of any mix
// share one launch and nothing is read back.  Blocks of one XCD take neighbouring tiles, in
// groups of a few row tiles, whose operands stay in that XCD's L2.
//
// With glu W has the columns of a and of b; a block's tile takes 16 of each in turn, so
// silu(a) b is formed in the lane that holds both.  The input gradient with glu goes on
// through silu(a) b in its epilogue.
#include "group.h"

namespace ts {
namespace {

constexpr int kStep = 32, kRing = 4;

__device__ const gu32x4 kZeros = {0u, 0u, 0u, 0u};

// 16 bytes per lane from memory into LDS: lane l writes dst + 16 l (dst is the same in the wave).
// Not a template: clang emits no host launch stub for a kernel template whose body names
// this builtin directly (nor for the transposing reads).
typedef __attribute__((address_space(3))) gu32x4 lds_gu32x4;
__device__ __forceinline__ void to_lds(const void* src, char* dst) {
  __builtin_amdgcn_global_load_lds(static_cast<const gu32x4*>(src), (lds_gu32x4*)dst, 16, 0, 0);
}
// In each 16-lane group lane q + 4m names 4 consecutive values and lane 4q + r receives value r
// of the runs named by lanes q, q+4, q+8, q+12.
typedef __attribute__((__vector_size__(4 * sizeof(__fp16)))) __fp16 gh4;
typedef __attribute__((address_space(3))) gh4 lds_gh4;
__device__ __forceinline__ gu32x4 read_tr(const char* lo, const char* hi) {
  typedef unsigned u2 __attribute__((ext_vector_type(2)));
  const u2 l = __builtin_bit_cast(u2, __builtin_amdgcn_ds_read_tr16_b64_v4f16((lds_gh4*)lo));
  const u2 h = __builtin_bit_cast(u2, __builtin_amdgcn_ds_read_tr16_b64_v4f16((lds_gh4*)hi));
  return gu32x4{l[0], l[1], h[0], h[1]};
}

// At most N vector-memory operations of this wave still out (they end in the order of issue),
// and none of its LDS reads.
template <int N>
__device__ __forceinline__ void wait_copies() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | 0x70 | ((N >> 4) << 14));
}
__device__ __forceinline__ void barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Where chunk ch (8 values) of row r lies within its row.
// Rows along the reduction: 4 chunks, 16 rows a read: rows 2i and 2i + 1 fill 128 bytes.
__device__ __forceinline__ int along_at(int r, int ch) { return ch ^ ((r >> 1) & 3); }
// Rows across it: a read takes 32 bytes of rows 8g + m and 8g + 4 + m.
__device__ __forceinline__ int across_at(int r, int ch) { return ch ^ (((r & 3) << 1) | (((r >> 3) & 1) << 3)); }

// (only starts that make the experts overlap have more runs than there are partial sums)
__device__ __forceinline__ int64_t group_chunks_on_device(const GroupK& k) { return k.n_rows / k.chunk + k.e; }

// A loose 16 bytes: columns c0.. of a row of `width` values, zeros past it.
template <typename T>
struct __attribute__((packed, aligned(2))) Loose8 {
  T e[8];
};
template <typename T>
__device__ __forceinline__ gu32x4 load_loose(const T* row, int c0, int width) {
  if (c0 + 8 <= width) return __builtin_bit_cast(gu32x4, *reinterpret_cast<const Loose8<T>*>(row + c0));
  T v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = c0 + i < width ? row[c0 + i] : static_cast<T>(0.f);
  return __builtin_bit_cast(gu32x4, v);
}

template <typename T, int R, int NT, int ACROSS>
struct Operand {
  static constexpr int kChunks = R * kStep / 8;
  static constexpr int kCopies = kChunks / NT;
  static constexpr int kPerRow = ACROSS ? R / 8 : 4;
  static constexpr int kBytes = R * kStep * 2;
  static_assert(kChunks % NT == 0, "whole copies");
};

// BM x BN results a block, WM x WN waves.  VEC: rows in whole, aligned 16-byte chunks;
// otherwise chunks go through registers.
template <typename T, GroupOp OP, bool GLU, int BM, int BN, int WM, int WN, bool VEC>
__global__ __launch_bounds__(WM* WN * 64) void k_group(const GroupK k) {
  constexpr int NT = WM * WN * 64;
  constexpr int MI = BM / WM / 16, NI = BN / WN / 16;
  constexpr bool A_ACROSS = OP == kGroupWgrad, B_ACROSS = OP != kGroupDgrad;
  typedef Operand<T, BM, NT, A_ACROSS> OA;
  typedef Operand<T, BN, NT, B_ACROSS> OB;
  constexpr int CA = OA::kCopies, CB = OB::kCopies;
  __shared__ __attribute__((aligned(16))) char lds_a[kRing * OA::kBytes];
  __shared__ __attribute__((aligned(16))) char lds_b[kRing * OB::kBytes];

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int len = OP == kGroupWgrad ? k.chunk : BM;
  const int along = OP == kGroupWgrad ? ceil_div(k.cin, BM) : 1;  // weight gradient: tiles along cin of each run
  const int64_t runs = total_runs(k, len);
  const GroupBlock block = group_block(runs, k.n_tiles * along);
  const int N = OP == kGroupDgrad ? k.cin : k.cout;  // columns of the result
  constexpr int kCols = GLU && OP == kGroupFwd ? BN / 2 : BN;
  if (block.at < 0) {
    if (OP == kGroupWgrad || block.spare < 0) return;
    const int64_t run = block.spare / k.n_tiles;
    const int n0 = static_cast<int>(block.spare - run * k.n_tiles) * kCols, cols = N - n0 < kCols ? N - n0 : kCols;
    T* y = static_cast<T*>(k.y);
    zero_unowned(k, run, BM, y, OP == kGroupDgrad && GLU ? 2 * N : N, n0, cols);
    if (GLU) {
      T* h = OP == kGroupDgrad ? y : static_cast<T*>(k.h_out);
      if (h && OP == kGroupFwd) zero_unowned(k, run, BM, h, 2 * N, n0, cols);
      if (h) zero_unowned(k, run, BM, h, 2 * N, N + n0, cols);
    }
    return;
  }
  // row tiles in fours (weight gradient: a run's tiles one after the other)
  constexpr int64_t kHigh = OP == kGroupWgrad ? 1 : 4;
  const int64_t band = block.at / (kHigh * k.n_tiles), in = block.at - band * kHigh * k.n_tiles;
  const int64_t rows = runs * along - band * kHigh, high = rows < kHigh ? rows : kHigh;
  const int nt = static_cast<int>(in / high), n0 = nt * kCols;
  const int64_t mt = band * kHigh + (in - nt * high), run = mt / along;
  const int m0 = static_cast<int>(mt - run * along) * BM;
  const GroupTile t = find_tile(k, run, len);
  if (t.e < 0 || (OP == kGroupWgrad && run >= group_chunks_on_device(k))) return;
  const int K = OP == kGroupFwd ? k.cin : OP == kGroupDgrad ? k.cout : t.rows;
  const int steps = ceil_div(K, kStep);
  const T* zeros = reinterpret_cast<const T*>(&kZeros);
  const T* wt = static_cast<const T*>(k.w) + static_cast<int64_t>(t.e) * k.cin * k.ldw;

  // Source of this lane's copies: of the first step, and how far the next one's lies.  at: what
  // is compared with K (a row, or a first column).
  const T* pa[CA];
  const T* pb[CB];
  int at_a[CA], at_b[CB], col_a[CA], col_b[CB];
#pragma unroll
  for (int i = 0; i < CA; ++i) {
    const int id = i * NT + tid, r = id / OA::kPerRow, pos = id % OA::kPerRow;
    if (A_ACROSS) {
      const int c = m0 + across_at(r, pos) * 8;
      at_a[i] = r;
      col_a[i] = c < k.cin ? c : -1;
      pa[i] = nullptr;  // found row by row
    } else {
      const int ch = along_at(r, pos);
      const int64_t row = t.row0 + (r < t.rows ? r : 0);  // rows past the tile: any, their results go nowhere
      int64_t src = row;
      if (OP == kGroupFwd && k.rows) {
        src = k.rows[row];
        if (src < 0 || src >= k.n_src) {
          if (k.flags) atomicOr(k.flags, TS_FLAG_RANGE);
          src = -1;
        }
      }
      at_a[i] = ch * 8;
      col_a[i] = src < 0 ? -1 : 0;
      pa[i] = static_cast<const T*>(OP == kGroupFwd ? k.x : k.dy) + (src < 0 ? 0 : src) * K + ch * 8;
    }
  }
#pragma unroll
  for (int i = 0; i < CB; ++i) {
    const int id = i * NT + tid, r = id / OB::kPerRow, pos = id % OB::kPerRow;
    if (B_ACROSS) {
      const int ch = across_at(r, pos);
      int c, width;
      if (GLU) {  // 16 columns of a, 16 of b
        c = n0 + (ch >> 2) * 16 + (ch & 1) * 8;
        width = k.cout;
        col_b[i] = c < width ? c + ((ch >> 1) & 1) * k.cout : -1;
      } else {
        c = n0 + ch * 8;
        col_b[i] = c < k.cout ? c : -1;
      }
      at_b[i] = r;
      pb[i] = OP == kGroupWgrad ? static_cast<const T*>(k.dy) + (t.row0 + r) * k.cout : wt + static_cast<int64_t>(r) * k.ldw;
    } else {
      const int ch = along_at(r, pos), n = n0 + r;
      at_b[i] = ch * 8;
      col_b[i] = n < N ? 0 : -1;
      pb[i] = wt + static_cast<int64_t>(n < N ? n : 0) * k.ldw + ch * 8;
    }
  }

  // one lane's 16 bytes of step s: their address, or the zeros'
  auto src_a = [&](int i, int s) -> const T* {
    const int at = at_a[i] + s * kStep;
    if (A_ACROSS) {
      if (at >= K || col_a[i] < 0) return zeros;
      const int64_t p = t.row0 + at;
      int64_t row = p;
      if (k.rows) {
        row = k.rows[p];
        if (row < 0 || row >= k.n_src) {
          if (k.flags) atomicOr(k.flags, TS_FLAG_RANGE);
          return zeros;
        }
      }
      return static_cast<const T*>(k.x) + row * k.cin + col_a[i];
    }
    return at < K && col_a[i] >= 0 ? pa[i] + s * kStep : zeros;
  };
  auto src_b = [&](int i, int s) -> const T* {
    const int at = at_b[i] + s * kStep;
    if (at >= K || col_b[i] < 0) return zeros;
    return B_ACROSS ? pb[i] + static_cast<int64_t>(s) * kStep * (OP == kGroupWgrad ? k.cout : k.ldw) + col_b[i] : pb[i] + s * kStep;
  };
  gu32x4 ra[VEC ? 1 : CA], rb[VEC ? 1 : CB];
  auto copy = [&](int s, int slot) {
#pragma unroll
    for (int i = 0; i < CA; ++i) {
      const T* p = src_a(i, s);
      if constexpr (VEC) {
        to_lds(p, lds_a + slot * OA::kBytes + (i * NT + wave * 64) * 16);
      } else {
        const int left = p == zeros ? 8 : A_ACROSS ? k.cin - col_a[i] : K - at_a[i] - s * kStep;
        ra[i] = load_loose(p, 0, left);
      }
    }
#pragma unroll
    for (int i = 0; i < CB; ++i) {
      const T* p = src_b(i, s);
      if constexpr (VEC) {
        to_lds(p, lds_b + slot * OB::kBytes + (i * NT + wave * 64) * 16);
      } else {
        const int c = GLU && col_b[i] >= k.cout ? col_b[i] - k.cout : col_b[i];
        const int left = p == zeros ? 8 : B_ACROSS ? k.cout - c : K - at_b[i] - s * kStep;
        rb[i] = load_loose(p, 0, left);
      }
    }
  };
  auto put = [&](int slot) {
    if constexpr (!VEC) {
#pragma unroll
      for (int i = 0; i < CA; ++i) *reinterpret_cast<gu32x4*>(lds_a + slot * OA::kBytes + (i * NT + tid) * 16) = ra[i];
#pragma unroll
      for (int i = 0; i < CB; ++i) *reinterpret_cast<gu32x4*>(lds_b + slot * OB::kBytes + (i * NT + tid) * 16) = rb[i];
    }
  };

  const int wm = wave / WN, wn = wave % WN;
  const int g = lane >> 4, c16 = lane & 15;
  // LDS addresses of this lane's fragments, without the ring's offset
  auto frag_at = [&](bool across, int r0, int width) {
    if (across) {
      const int q = lane & 3, m = (lane >> 2) & 3, row = 8 * g + m;
      return row * width * 2 + across_at(row, r0 / 8 + (q >> 1)) * 16 + (q & 1) * 8;
    }
    return (r0 + c16) * kStep * 2 + along_at(c16, g) * 16;
  };
  int fa[MI], fb[NI];
#pragma unroll
  for (int i = 0; i < MI; ++i) fa[i] = frag_at(A_ACROSS, wm * MI * 16 + i * 16, BM);
#pragma unroll
  for (int i = 0; i < NI; ++i) fb[i] = frag_at(B_ACROSS, wn * NI * 16 + i * 16, BN);
  auto read_a = [&](int i, int slot) {
    const char* p = lds_a + slot * OA::kBytes + fa[i];
    if constexpr (A_ACROSS) return read_tr(p, p + 4 * BM * 2);
    else return *reinterpret_cast<const gu32x4*>(p);
  };
  auto read_b = [&](int i, int slot) {
    const char* p = lds_b + slot * OB::kBytes + fb[i];
    if constexpr (B_ACROSS) return read_tr(p, p + 4 * BN * 2);
    else return *reinterpret_cast<const gu32x4*>(p);
  };

  gf32x4 acc[MI][NI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j) acc[i][j] = gf32x4{0.f, 0.f, 0.f, 0.f};

  auto multiply = [&](int slot) {
    gu32x4 b[NI];
#pragma unroll
    for (int j = 0; j < NI; ++j) b[j] = read_b(j, slot);
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const gu32x4 a = read_a(i, slot);
#pragma unroll
      for (int j = 0; j < NI; ++j) acc[i][j] = GMfma<T>::run(b[j], a, acc[i][j]);
    }
  };

  if constexpr (VEC) {
#pragma unroll
    for (int s = 0; s < kRing - 1; ++s)
      if (s < steps) copy(s, s);
    for (int s0 = 0; s0 < steps; s0 += kRing) {
#pragma unroll
      for (int slot = 0; slot < kRing; ++slot) {
        const int s = s0 + slot;
        if (s >= steps) break;
        // step s has landed: of the copies after it those of the next two may be out
        if (s + 2 < steps) wait_copies<2 * (CA + CB)>();
        else if (s + 1 < steps) wait_copies<CA + CB>();
        else wait_copies<0>();
        barrier();  // and everyone is done with the step before, whose place is free
        if (s + kRing - 1 < steps) copy(s + kRing - 1, (slot + kRing - 1) % kRing);
        multiply(slot);
      }
    }
  } else {
    copy(0, 0);
    for (int s = 0; s < steps; ++s) {
      const int slot = s & (kRing - 1);
      put(slot);  // its last readers were done before the barrier three steps ago
      if (s + 1 < steps) copy(s + 1, 0);
      __syncthreads();
      multiply(slot);
    }
  }

  // Lane (g, c16) holds columns 4g..4g+3 of row c16 of each 16 x 16 tile.
  if constexpr (OP == kGroupWgrad) {
    float* out = t.count == 1 ? k.dw + static_cast<int64_t>(t.e) * k.cin * k.cout : k.part + static_cast<int64_t>(run) * k.cin * k.cout;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int m = m0 + wm * MI * 16 + i * 16 + c16;
      if (m >= k.cin) continue;
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        const int n = n0 + wn * NI * 16 + j * 16 + 4 * g;
        float* p = out + static_cast<int64_t>(m) * k.cout + n;
        if (VEC) {
          if (n < k.cout) *reinterpret_cast<gf32x4*>(p) = acc[i][j];
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (n + r < k.cout) p[r] = acc[i][j][r];
        }
      }
    }
    return;
  } else {
    typedef T t4 __attribute__((ext_vector_type(4)));
    auto store = [&](T* row, int n, int width, gf32x4 v) {
      if (VEC) {
        if (n < width) *reinterpret_cast<t4*>(row + n) = __builtin_convertvector(v, t4);
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (n + r < width) row[n + r] = static_cast<T>(v[r]);
      }
    };
    T* y = static_cast<T*>(k.y);
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int r = wm * MI * 16 + i * 16 + c16;
      if (r >= t.rows) continue;
      const int64_t row = t.row0 + r;
      if constexpr (GLU && OP == kGroupFwd) {
#pragma unroll
        for (int j = 0; j < NI; j += 2) {
          const int n = n0 + wn * NI * 8 + j * 8 + 4 * g;
          const gf32x4 a = acc[i][j], b = acc[i][j + 1];
          gf32x4 v;
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = a[e] * sigmoid(a[e]) * b[e];
          store(y + row * N, n, N, v);
          if (k.h_out) {
            T* h = static_cast<T*>(k.h_out) + row * 2 * N;
            store(h, n, N, a);
            store(h + N, n, N, b);
          }
        }
      } else if constexpr (GLU) {
#pragma unroll
        for (int j = 0; j < NI; ++j) {
          const int n = n0 + wn * NI * 16 + j * 16 + 4 * g;
          if (n >= N) continue;
          const T* h = static_cast<const T*>(k.h) + row * 2 * N + n;
          gf32x4 a{}, b{}, da, db;
          if (VEC) {
            a = __builtin_convertvector(*reinterpret_cast<const t4*>(h), gf32x4);
            b = __builtin_convertvector(*reinterpret_cast<const t4*>(h + N), gf32x4);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (n + e < N) a[e] = static_cast<float>(h[e]), b[e] = static_cast<float>(h[N + e]);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float s = sigmoid(a[e]), d = acc[i][j][e];
            da[e] = d * b[e] * s * fmaf(a[e], 1.f - s, 1.f);
            db[e] = d * a[e] * s;
          }
          T* out = y + row * 2 * N;
          store(out, n, N, da);
          store(out + N, n, N, db);
        }
      } else {
#pragma unroll
        for (int j = 0; j < NI; ++j) store(y + row * N, n0 + wn * NI * 16 + j * 16 + 4 * g, N, acc[i][j]);
      }
    }
  }
}

// dw of the experts whose rows were cut into several runs (or are none): their partial
// sums, in order.
__global__ __launch_bounds__(256) void k_group_sum(const GroupK k) {
  const int e = blockIdx.y, lane = threadIdx.x & 63;
  int64_t first = 0;
  int count = 0;
  for (int e0 = 0; e0 <= e; e0 += 64) {
    int64_t a, b;
    expert_rows(k, e0 + lane, &a, &b);
    int64_t n = runs_of(a, b, k.chunk);
    if (e0 + 64 > e) count = __builtin_amdgcn_readlane(static_cast<int>(n), e - e0);
    if (e0 + lane >= e) n = 0;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) n += __shfl_xor(n, m);
    first += n;
  }
  const int64_t left = group_chunks_on_device(k) - first;
  if (count > left) count = left < 0 ? 0 : static_cast<int>(left);
  if (count == 1) return;
  const int64_t size = static_cast<int64_t>(k.cin) * k.cout;
  float* dw = k.dw + e * size;
  const float* part = k.part + first * size;
  const int64_t step = static_cast<int64_t>(gridDim.x) * 256;
  if (size % 4 == 0) {
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < size / 4; i += step) {
      gf32x4 s{0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
      for (int c = 0; c < count; ++c) s += *reinterpret_cast<const gf32x4*>(part + c * size + 4 * i);
      *reinterpret_cast<gf32x4*>(dw + 4 * i) = s;
    }
  } else {
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < size; i += step) {
      float s = 0.f;
#pragma unroll 8
      for (int c = 0; c < count; ++c) s += part[c * size + i];
      dw[i] = s;
    }
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <typename T, GroupOp OP, bool GLU, int BM, int BN, int WM, int WN, bool VEC>
void run(GroupK& k, hipStream_t s) {
  const int N = OP == kGroupDgrad ? k.cin : k.cout;
  k.n_tiles = ceil_div(N, GLU && OP == kGroupFwd ? BN / 2 : BN);
  const int64_t grid = OP == kGroupWgrad ? group_grid(group_chunks(k.n_rows, k.e, k.chunk), k.n_tiles * ceil_div(k.cin, BM))
                                         : group_grid(group_runs(k.n_rows, k.e, BM), k.n_tiles);
  k_group<T, OP, GLU, BM, BN, WM, WN, VEC><<<static_cast<unsigned>(grid), WM * WN * 64, 0, s>>>(k);
}

template <typename T, GroupOp OP, bool GLU>
void run(GroupK& k, hipStream_t s) {
  const bool vec = k.cin % 8 == 0 && k.cout % 8 == 0 && aligned16(k.x) && aligned16(k.dy) && aligned16(k.w) && aligned16(k.h) &&
                   aligned16(k.y) && aligned16(k.h_out) && aligned16(k.dw) && aligned16(k.part);
  if (!vec) return run<T, OP, GLU, 128, 128, 2, 2, false>(k, s);
  const int N = OP == kGroupDgrad ? k.cin : k.ldw;
  const bool large = N >= 256 && (OP == kGroupWgrad ? k.cin >= 256 : k.n_rows / k.e >= 512);
  if (large) return run<T, OP, GLU, 256, 256, 2, 4, true>(k, s);
  run<T, OP, GLU, 128, 128, 2, 2, true>(k, s);
}

template <typename T>
void run(GroupK& k, GroupOp op, bool glu, hipStream_t s) {
  if (op == kGroupFwd) return glu ? run<T, kGroupFwd, true>(k, s) : run<T, kGroupFwd, false>(k, s);
  if (op == kGroupDgrad) return glu ? run<T, kGroupDgrad, true>(k, s) : run<T, kGroupDgrad, false>(k, s);
  run<T, kGroupWgrad, false>(k, s);
  const int64_t size = static_cast<int64_t>(k.cin) * k.cout;
  const int64_t blocks = ceil_div<int64_t>(size, 1024);
  k_group_sum<<<dim3(static_cast<unsigned>(blocks < 4096 ? blocks : 4096), k.e), 256, 0, s>>>(k);
}

}  // namespace

// Rows of a partial sum: about 512 blocks of 128 x 128 in all, 256 to 4096 rows each.
int group_chunk(int64_t n_rows, int cin, int cout) {
  const int64_t tiles = static_cast<int64_t>(ceil_div(cin, 128)) * ceil_div(cout, 128);
  const int64_t want = ceil_div<int64_t>(512, tiles), rows = ceil_div<int64_t>(n_rows, want);
  const int64_t c = rows < 256 ? 256 : rows > 4096 ? 4096 : rows;
  return static_cast<int>((c + kStep - 1) / kStep * kStep);
}

hipError_t launch_group(GroupK& k, GroupOp op, ts_dtype dt, bool glu, hipStream_t s) {
  if (dt == TS_F16) run<_Float16>(k, op, glu, s);
  else
    run<__bf16>(k, op, glu, s);
  return hipGetLastError();
}

}  // namespace ts
