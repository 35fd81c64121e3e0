// Products grouped by expert on the matrix cores, for many rows an expert (few rows:
// group_few.hip).
//
//   forward          y[p]  = x[rows[p]] W[e]        reduced over cin
//   input gradient   dx[p] = dy[p] W[e]^T           reduced over cout
//   weight gradient  dW[e] = sum over its p of x[rows[p]]^T dy[p]
//
// One kernel for the three: a tile of BM x BN results is reduced over steps of 64.  Both
// operands' steps are copied straight into LDS (16 bytes a lane, no registers; 128 bytes of a
// row at once, whole lines), into two places in turn.  A step is done in parts, 32 of a wave's
// rows over 32 of the reduction each: while one is multiplied the fragments of the next are
// read, the first ones of the next step among them, so matrix instructions wait neither for
// LDS nor behind the step's one barrier.  Behind it the step's place is free and the copies of
// the step after the next start.  Blocks stay for several tiles, and the next one's first copies
// are under way while a tile's results are written.  An operand whose rows run along the
// reduction (x and dy of the first two, W of the second) is read from LDS as it lies; one whose
// rows run across it is read with the transposing LDS reads.  Chunks of 16 bytes are stored
// xor-ed with their row so that neither read meets a bank twice.  Gathered rows cost nothing:
// every lane names its own source anyway.  Sources past the matrix (the last step's, rows that
// are not there) lie behind their buffer's end and read as zeros.
//
// Tiles are found from the starts on the device, expert by expert, so lengths of any mix
// share one launch and nothing is read back.  Blocks of one XCD take neighbouring tiles, in
// groups of a few row tiles, whose operands stay in that XCD's L2.
//
// With glu W has the columns of a and of b; a block's tile takes 16 of each in turn, so
// silu(a) b is formed in the lane that holds both.  The input gradient with glu goes on
// through silu(a) b in its epilogue.
//
// 32,768 rows to 16 experts of 1024 x 4096, bf16: forward 292 us (0.94 PFLOP/s), input gradient 298,
// weight gradient 336 and 9 for its partial sums; the matrix units are busy for 49, 51 and 38% of
// the cycles, the rest is a tile's prologue and epilogue, LDS latency and experts that end in a
// part of a tile.  609,756 rows to 8 experts of 128 -> 2 x 256 with silu(a) b and h: 346 us, its
// gradient 351: two steps a tile, so writing 0.94 GB (0.67 GB, and 0.4 read) is most of the work.
// 4,999 x 3 rows of 77 -> 133: 11, 11 and 20 us, latency.  256 rows to 64 experts of 1024 x 1024:
// 21 us, 134 MB of weights, about half of them from the last-level cache.
#include "group.h"

namespace ts {
namespace {

constexpr int kStep = kGroupStep;
constexpr int kRowHalf = 1024;  // row numbers of the weight gradient in half of their place in LDS

// 16 bytes per lane from a buffer into LDS: lane l writes dst + 16 l (dst is the same in the
// wave), zeros where its offset lies behind the buffer's end.  Not a template: clang emits no host
// launch stub for a kernel template whose body names this builtin directly (nor for the
// transposing reads).  (Buffer instructions: after the global ones every wait for LDS reads
// is one for all of them.)
constexpr uint32_t kNowhere = ~0u;
typedef __attribute__((address_space(3))) gu32x4 lds_gu32x4;
typedef __attribute__((address_space(3))) uint32_t lds_u32;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* base, int64_t bytes) {
  const uint64_t v = reinterpret_cast<uint64_t>(base);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v)), hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>((static_cast<uint64_t>(hi) << 32) | lo), 0,
                                           __builtin_amdgcn_readfirstlane(static_cast<int>(bytes)), 0x00020000);
}
__device__ __forceinline__ void to_lds(__amdgpu_buffer_rsrc_t buf, uint32_t off, char* dst) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(buf, (lds_gu32x4*)dst, 16, static_cast<int>(off), 0, 0, 0);
}
// 4 bytes per lane: lane l writes dst[l].
__device__ __forceinline__ void to_lds4(__amdgpu_buffer_rsrc_t buf, uint32_t off, int32_t* dst) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(buf, (lds_u32*)dst, 4, static_cast<int>(off), 0, 0, 0);
}
__device__ __forceinline__ uint32_t further(uint32_t off, uint32_t by) { return __builtin_elementwise_add_sat(off, by); }  // nowhere stays nowhere
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
__device__ __forceinline__ void wait_lds() { __builtin_amdgcn_s_waitcnt(0xC07F); }
__device__ __forceinline__ void barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Where chunk ch (8 values) of row r lies within its row.
// Rows along the reduction: 8 chunks, one of each of 16 rows a read.
__device__ __forceinline__ int along_at(int r, int ch) { return ch ^ (r & 7); }
// Rows across it: a read takes 32 bytes of rows 8g + m and 8g + 4 + m.
__device__ __forceinline__ int across_at(int r, int ch) { return ch ^ (((r & 3) << 1) | (((r >> 3) & 1) << 3)); }

// The value as if it were new: what is computed from it is not kept in registers over the steps.
template <typename V>
__device__ __forceinline__ V fresh(V v) {
  asm volatile("" : "+v"(v));
  return v;
}
// Lane group g of 4 holds elements 4g..4g+3 of two blocks of 16 columns, p and q: afterwards
// it holds 8 consecutive ones, group 0 and 1 of p's, 2 and 3 of q's.
__device__ __forceinline__ void join8(unsigned& p, unsigned& q) {
  const auto a = __builtin_amdgcn_permlane32_swap(p, q, false, false);
  const auto b = __builtin_amdgcn_permlane16_swap(a[0], a[1], false, false);
  p = b[0];
  q = b[1];
}
// Partial sums of the weight gradient that there is room for.
__device__ __forceinline__ int64_t group_chunks_on_device(const GroupK& k) { return k.n_rows / k.chunk + k.e; }

// A loose 16 bytes: columns c0.. of a row of `width` values, zeros past it.
template <typename T>
struct __attribute__((packed, aligned(2))) Loose8 {
  T e[8];
};
// (Of a row's last, partial chunk the row's last 8 values are read instead and moved down by
// `over`; where that is done later the load need not have ended before.)
__device__ __forceinline__ int over(int c0, int width) { return width < 8 || c0 + 8 <= width ? 0 : c0 + 8 - width; }
__device__ __forceinline__ gu32x4 moved_down(gu32x4 v, int by) {
  if (by & 4) v = gu32x4{v[2], v[3], 0u, 0u};
  if (by & 2) v = gu32x4{v[1], v[2], v[3], 0u};
  if (by & 1) v = gu32x4{(v[0] >> 16) | (v[1] << 16), (v[1] >> 16) | (v[2] << 16), (v[2] >> 16) | (v[3] << 16), v[3] >> 16};
  return v;
}
template <typename T>
__device__ __forceinline__ gu32x4 load_unmoved(const T* row, int c0, int width) {
  if (width < 8) {
    T v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c0 + i < width ? row[c0 + i] : static_cast<T>(0.f);
    return __builtin_bit_cast(gu32x4, v);
  }
  return __builtin_bit_cast(gu32x4, *reinterpret_cast<const Loose8<T>*>(row + (c0 - over(c0, width))));
}
template <typename T>
__device__ __forceinline__ gu32x4 load_loose(const T* row, int c0, int width) {
  return moved_down(load_unmoved(row, c0, width), over(c0, width));
}
struct __attribute__((packed, aligned(4))) Loose4 {
  float e[4];
};
template <typename T>
__device__ __forceinline__ void store_loose(T* row, int c0, int width, gu32x4 v) {
  if (c0 + 8 <= width) {
    *reinterpret_cast<Loose8<T>*>(row + c0) = __builtin_bit_cast(Loose8<T>, v);
  } else {
    const Loose8<T> w = __builtin_bit_cast(Loose8<T>, v);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c0 + i < width) row[c0 + i] = w.e[i];
  }
}

template <typename T, int R, int NT, int ACROSS>
struct Operand {
  static constexpr int kChunks = R * kStep / 8;
  static constexpr int kCopies = kChunks / NT;
  static constexpr int kPerRow = ACROSS ? R / 8 : kStep / 8;
  static constexpr int kBytes = R * kStep * 2;
  static_assert(kChunks % NT == 0, "whole copies");
};

// A tile and where this lane's copies of its first step come from.
template <int CA>
struct TileSource {
  GroupTile t;
  int m0, n0, steps, K;
  // VEC: offsets within the buffers.  Otherwise: rows of x or dy (-1: none); columns of W or dy
  uint32_t va[CA], vb;
};

// BM x BN results a tile, WM x WN waves.  VEC: rows in whole, aligned 16-byte chunks;
// otherwise chunks go through registers.
template <typename T, GroupOp OP, bool GLU, int BM, int BN, int WM, int WN, bool VEC>
__global__ __launch_bounds__(WM* WN * 64, BM * BN / (WM * WN) > 8192 ? 1 : 2) void k_group(const GroupK k) {
  constexpr int NT = WM * WN * 64;
  constexpr int MI = BM / WM / 16, NI = BN / WN / 16;
  constexpr bool A_ACROSS = OP == kGroupWgrad, B_ACROSS = OP != kGroupDgrad;
  typedef Operand<T, BM, NT, A_ACROSS> OA;
  typedef Operand<T, BN, NT, B_ACROSS> OB;
  constexpr int CA = OA::kCopies, CB = OB::kCopies;
  constexpr int kCols = GLU && OP == kGroupFwd ? BN / 2 : BN;
  constexpr bool EARLY = MI < 8;  // whether registers are left to look up the next tile's rows meanwhile
  __shared__ __attribute__((aligned(16))) char lds_a[2 * OA::kBytes];
  __shared__ __attribute__((aligned(16))) char lds_b[2 * OB::kBytes];
  __shared__ int32_t lds_rows[A_ACROSS ? 2 * kRowHalf : 1];

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int along = OP == kGroupWgrad ? ceil_div(k.cin, BM) : 1;  // weight gradient: tiles along cin of each run
  const int N = OP == kGroupDgrad ? k.cin : k.cout;               // columns of the result
  __shared__ GroupLane lds_lanes[64];
  const GroupFinder<OP == kGroupWgrad> finder(k, OP == kGroupWgrad ? k.chunk : BM, lds_lanes);
  // (only starts that make the experts overlap have more runs than were planned for; 32 bits hold
  // all the tiles there are)
  const int64_t planned = OP == kGroupWgrad ? group_chunks_on_device(k) : k.n_rows / BM + k.e;
  const int runs = static_cast<int>(finder.total < planned ? finder.total : planned);
  // The i-th tile of this block.  Blocks go to the 8 XCDs in turn: those of one XCD take neighbouring
  // tiles.  Weight gradient: the runs have lengths of their own, the longest ones first, so blocks
  // take them to and fro; of a run each XCD gets some columns.
  const int n_tiles = k.n_tiles, total = runs * along * n_tiles, per_xcd = (total + 7) / 8;
  auto tile_of = [&](int i) {
    const int grid = gridDim.x, block = blockIdx.x;
    if (OP == kGroupWgrad) {
      const int tile = i * grid + (i & 1 ? grid - 1 - block : block);
      return tile < total ? tile : -1;
    }
    const int in = (block >> 3) + i * (grid >> 3), tile = (block & 7) * per_xcd + in;
    return in < per_xcd && tile < total ? tile : -1;
  };
  // This lane's copies: the row of the operand's tile, and the chunk of it.  Of the next copy the
  // row is NT / kPerRow further, and the chunk the same.
  constexpr int NEXT_A = NT / OA::kPerRow, NEXT_B = NT / OB::kPerRow;
  static_assert(NEXT_A % (A_ACROSS ? 16 : 8) == 0 && NEXT_B % (B_ACROSS ? 16 : 8) == 0, "such rows store their chunks in the same places");
  typedef TileSource<A_ACROSS ? 1 : CA> Source;
  // (computed where they are used: the accumulators leave few registers to keep them in)
  auto row_a = [&]() { return fresh(tid) / OA::kPerRow; };
  auto row_b = [&]() { return fresh(tid) / OB::kPerRow; };
  auto chunk_a = [&]() {
    const int t = fresh(tid), r = t / OA::kPerRow;
    return A_ACROSS ? across_at(r, t % OA::kPerRow) : along_at(r, t % 8);
  };
  auto chunk_b = [&]() {
    const int t = fresh(tid), r = t / OB::kPerRow;
    return B_ACROSS ? across_at(r, t % OB::kPerRow) : along_at(r, t % 8);
  };
  // its first column in the tile; with glu 16 columns of a, then 16 of b
  auto col_b = [&]() {
    const int ch = chunk_b();
    return GLU && B_ACROSS ? (ch >> 2) * 16 + (ch & 1) * 8 : ch * 8;
  };

  // Where a tile lies; the rows that its copies read are asked for early.
  auto locate = [&](Source& x, int tile) {
    // row tiles in fours (weight gradient: a run's tiles one after the other)
    constexpr int kHigh = OP == kGroupWgrad ? 1 : 4;
    const int band = tile / (kHigh * n_tiles), in = tile - band * kHigh * n_tiles;
    const int rows = runs * along - band * kHigh, high = rows < kHigh ? rows : kHigh;
    const int nt = in / high, mt = band * kHigh + (in - nt * high);
    x.n0 = nt * kCols;
    const int run = mt / along;
    x.m0 = (mt - run * along) * BM;
    x.t = finder.find(k, run);
    x.K = OP == kGroupFwd ? k.cin : OP == kGroupDgrad ? k.cout : x.t.rows;
    x.steps = ceil_div(x.K, kStep);
    if constexpr (!A_ACROSS) {
#pragma unroll
      for (int i = 0; i < CA; ++i) {
        const int r = row_a() + i * NEXT_A;
        int32_t src = r < x.t.rows ? r : -1;  // from the tile's first row on
        if (OP == kGroupFwd && k.rows && r < x.t.rows) src = k.rows[x.t.row0 + r];
        x.va[i] = static_cast<uint32_t>(src);
      }
    }
  };
  auto set_up = [&](Source& x) {
    if constexpr (!A_ACROSS) {
#pragma unroll
      for (int i = 0; i < CA; ++i) {
        int32_t src = static_cast<int32_t>(x.va[i]);
        if (OP == kGroupFwd && k.rows && (src < 0 || src >= k.n_src)) {
          if (row_a() + i * NEXT_A < x.t.rows && k.flags) atomicOr(k.flags, TS_FLAG_RANGE);
          src = -1;
        }
        x.va[i] = !VEC || src < 0 ? static_cast<uint32_t>(src)
                                  : static_cast<uint32_t>(src) * static_cast<uint32_t>(x.K * 2) + static_cast<uint32_t>(chunk_a() * 16);
      }
    }
    if constexpr (OP == kGroupDgrad) {
      x.vb = static_cast<uint32_t>(row_b() * k.ldw * 2 + chunk_b() * 16);
    } else {
      const int c = x.n0 + col_b(), at = c + (GLU ? ((chunk_b() >> 1) & 1) * k.cout : 0);
      x.vb = c >= k.cout ? kNowhere : static_cast<uint32_t>(VEC ? (row_b() * k.ldw + at) * 2 : at);
    }
  };

  // Weight gradient: which rows of x are read.  Their numbers go through LDS, kRowHalf of them at
  // once; a lane reads those of its next copies with the fragments.
  int32_t row_ids[A_ACROSS ? CA : 1];
  auto fetch_rows = [&](const Source& x, int s) {
    if constexpr (A_ACROSS) {
      if (!k.rows) return;
#pragma unroll
      for (int i = 0; i < CA; ++i) row_ids[i] = lds_rows[(row_a() + i * NEXT_A + s * kStep) & (2 * kRowHalf - 1)];
    }
  };
  // those from `from` on (a multiple of kRowHalf) on their way into LDS
  auto copy_rows = [&](const Source& x, int from) {
    if constexpr (A_ACROSS) {
      if (!k.rows) return;
#pragma unroll
      for (int i = 0; i < kRowHalf / NT; ++i) {
        const int at = from + i * NT + wave * 64;
        if (at < x.K) to_lds4(buffer_of(k.rows + x.t.row0, static_cast<int64_t>(x.K) * 4), (at + lane) * 4, &lds_rows[at & (2 * kRowHalf - 1)]);
      }
    }
  };
  // Copies of step s.  `in` is the same for all of a lane's copies where rows run along.
  gu32x4 ra[VEC ? 1 : CA], rb[VEC ? 1 : CB];
  auto copy_a = [&](const Source& x, int s, int slot) {
    const int from = s * kStep, left = x.K - from;
    const T* base = static_cast<const T*>(OP == kGroupDgrad ? k.dy : k.x);
    if constexpr (A_ACROSS) {
      const int64_t first = k.rows ? 0 : x.t.row0 + from;
      const __amdgpu_buffer_rsrc_t buf =
          buffer_of(base + first * k.cin, (k.rows ? k.n_src : static_cast<int64_t>(left < kStep ? left : kStep)) * k.cin * 2);
#pragma unroll
      for (int i = 0; i < CA; ++i) {
        const int r = row_a() + i * NEXT_A, c = x.m0 + chunk_a() * 8;
        const int32_t row = k.rows ? row_ids[i] : r;
        bool in = r < left && c < k.cin;
        if (in && k.rows && (row < 0 || row >= k.n_src)) {
          if (k.flags) atomicOr(k.flags, TS_FLAG_RANGE);
          in = false;
        }
        if constexpr (VEC)
          to_lds(buf, in ? (static_cast<uint32_t>(row) * static_cast<uint32_t>(k.cin) + c) * 2 : kNowhere,
                 lds_a + slot * OA::kBytes + (i * NT + wave * 64) * 16);
        else
          ra[i] = in ? load_unmoved(base + (first + row) * k.cin, c, k.cin) : gu32x4{0u, 0u, 0u, 0u};
      }
    } else {
      const bool gather = OP == kGroupFwd && k.rows;
      const int64_t first = gather ? 0 : x.t.row0;
      const __amdgpu_buffer_rsrc_t buf = buffer_of(base + first * x.K, (gather ? k.n_src : static_cast<int64_t>(x.t.rows)) * x.K * 2);
      const int c = chunk_a() * 8;
#pragma unroll
      for (int i = 0; i < CA; ++i) {
        if constexpr (VEC) {
          to_lds(buf, c < left ? further(x.va[i], from * 2) : kNowhere, lds_a + slot * OA::kBytes + (i * NT + wave * 64) * 16);
        } else {
          const int32_t row = static_cast<int32_t>(x.va[i]);
          ra[i] = c < left && row >= 0 ? load_unmoved(base + (first + row) * x.K, from + c, x.K) : gu32x4{0u, 0u, 0u, 0u};
        }
      }
    }
  };
  auto end_b = [&](uint32_t column) { return GLU && column < static_cast<uint32_t>(k.cout) ? k.cout : k.ldw; };
  auto copy_b = [&](const Source& x, int s, int slot) {
    const int from = s * kStep, left = x.K - from;
    const T* base = OP == kGroupWgrad ? static_cast<const T*>(k.dy) : static_cast<const T*>(k.w) + static_cast<int64_t>(x.t.e) * k.cin * k.ldw;
    const int64_t first = OP == kGroupDgrad ? x.n0 : OP == kGroupWgrad ? x.t.row0 + from : from;  // row of the buffer's start
    const int rows = OP == kGroupDgrad ? (N - x.n0 < BN ? N - x.n0 : BN) : left < kStep ? left : kStep;
    const __amdgpu_buffer_rsrc_t buf = buffer_of(base + first * k.ldw, static_cast<int64_t>(rows) * k.ldw * 2);
#pragma unroll
    for (int i = 0; i < CB; ++i) {
      char* dst = lds_b + slot * OB::kBytes + (i * NT + wave * 64) * 16;
      const int r = row_b() + i * NEXT_B;
      if constexpr (OP == kGroupDgrad) {
        const int c = chunk_b() * 8;
        if constexpr (VEC)
          to_lds(buf, c < left ? x.vb + static_cast<uint32_t>(i * NEXT_B * k.ldw + from) * 2 : kNowhere, dst);
        else
          rb[i] = c < left && r < rows ? load_unmoved(base + (first + r) * k.ldw, from + c, x.K) : gu32x4{0u, 0u, 0u, 0u};
      } else {
        const uint32_t v = x.vb;
        if constexpr (VEC)
          to_lds(buf, further(v, static_cast<uint32_t>(i * NEXT_B * k.ldw * 2)), dst);
        else
          rb[i] = r < rows && v != kNowhere ? load_unmoved(base + (first + r) * k.ldw, static_cast<int>(v), end_b(v)) : gu32x4{0u, 0u, 0u, 0u};
      }
    }
  };
  // Step s of chunks in registers into LDS.  Few waves hold a row's last chunk.
  auto put = [&](const Source& x, int s, int slot) {
    if constexpr (!VEC) {
#pragma unroll
      for (int i = 0; i < CA; ++i) {
        const int by = A_ACROSS ? over(x.m0 + chunk_a() * 8, k.cin) : over(s * kStep + chunk_a() * 8, x.K);
        if (__builtin_amdgcn_ballot_w64(by != 0)) ra[i] = moved_down(ra[i], by);
        *reinterpret_cast<gu32x4*>(lds_a + slot * OA::kBytes + (i * NT + tid) * 16) = ra[i];
      }
#pragma unroll
      for (int i = 0; i < CB; ++i) {
        int by;
        if constexpr (OP == kGroupDgrad) by = over(s * kStep + chunk_b() * 8, x.K);
        else
          by = x.vb == kNowhere ? 0 : over(static_cast<int>(x.vb), end_b(x.vb));
        if (__builtin_amdgcn_ballot_w64(by != 0)) rb[i] = moved_down(rb[i], by);
        *reinterpret_cast<gu32x4*>(lds_b + slot * OB::kBytes + (i * NT + tid) * 16) = rb[i];
      }
    }
  };
  // The first steps of a tile; nobody reads the ring any more.
  auto start = [&](const Source& x) {
    if constexpr (A_ACROSS) {
      if (k.rows) {
        copy_rows(x, 0);
        if (x.K > kRowHalf) copy_rows(x, kRowHalf);
        wait_copies<0>();
        barrier();
      }
      fetch_rows(x, 0);
    }
    copy_a(x, 0, 0);
    copy_b(x, 0, 0);
    fetch_rows(x, 1);
    if (VEC && x.steps > 1) {
      copy_a(x, 1, 1);
      copy_b(x, 1, 1);
      fetch_rows(x, 2);
    }
  };
  // Rows from half of lds_rows further on: that half is free.
  auto more_rows = [&](const Source& x, int s) {
    if constexpr (A_ACROSS) {
      const int from = s * kStep + kRowHalf;
      if (s > 0 && (s * kStep) % kRowHalf == 0 && from < x.K) copy_rows(x, from);
    }
  };

  const int wm = wave / WN, wn = wave % WN;
  const int g = lane >> 4, c16 = lane & 15;
  // LDS address of this lane's first fragment, without its place's offset.  Fragment i is 16 rows
  // or columns further, and half kk of a step 32 along the reduction: one of the two changes
  // only bits of the chunk's number.
  auto frag_at = [&](bool across, int r0, int width) {
    if (across) {
      const int q = lane & 3, m = (lane >> 2) & 3, row = 8 * g + m;
      return row * width * 2 + across_at(row, r0 / 8 + (q >> 1)) * 16 + (q & 1) * 8;
    }
    return (r0 + c16) * kStep * 2 + along_at(c16, g) * 16;
  };
  const int fa = frag_at(A_ACROSS, wm * MI * 16, BM), fb = frag_at(B_ACROSS, wn * NI * 16, BN);
  auto read_a = [&](int i, int kk, int slot) {
    const char* p = lds_a + slot * OA::kBytes;
    if constexpr (A_ACROSS) {
      p += (i ? fresh(fa) ^ (i * 32) : fa) + kk * 64 * BM;
      return read_tr(p, p + 4 * BM * 2);
    } else return *reinterpret_cast<const gu32x4*>(p + (fa ^ (kk * 64)) + i * 16 * kStep * 2);
  };
  auto read_b = [&](int i, int kk, int slot) {
    const char* p = lds_b + slot * OB::kBytes;
    if constexpr (B_ACROSS) {
      p += (i ? fresh(fb) ^ (i * 32) : fb) + kk * 64 * BN;
      return read_tr(p, p + 4 * BN * 2);
    } else return *reinterpret_cast<const gu32x4*>(p + (fb ^ (kk * 64)) + i * 16 * kStep * 2);
  };

  int tile = tile_of(0), done = 0;
  Source x;
  if (tile >= 0) {
    locate(x, tile);
    set_up(x);
    start(x);
  }
  while (tile >= 0) {
    Source next;
    tile = tile_of(++done);
    if constexpr (EARLY) {
      if (tile >= 0) locate(next, tile);
    }
    gf32x4 acc[MI][NI];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j) acc[i][j] = gf32x4{0.f, 0.f, 0.f, 0.f};
    if constexpr (VEC) {
      constexpr int PI = 2, ROWS = MI / PI, PARTS = 2 * ROWS;  // blocks of rows in a part; parts over 32, and of a step
      gu32x4 a[2][PI], b[2][NI];
      // the first step has landed (the second one may be out, or stores of the tile before instead)
      if (x.steps > 1) wait_copies<CA + CB>();
      else wait_copies<0>();
      barrier();
#pragma unroll
      for (int j = 0; j < NI; ++j) b[0][j] = read_b(j, 0, 0);
#pragma unroll
      for (int i = 0; i < PI; ++i) a[0][i] = read_a(i, 0, 0);
      for (int s0 = 0; s0 < x.steps; s0 += 2) {
#pragma unroll
        for (int slot = 0; slot < 2; ++slot) {
          const int s = s0 + slot;
          if (s >= x.steps) break;
#pragma unroll
          for (int part = 0; part < PARTS; ++part) {
            if (part + 1 < PARTS) {
              const int kk = (part + 1) / ROWS, row = (part + 1) % ROWS * PI;
              wait_lds();  // this part's fragments, before the next one's are asked for
              if (row == 0) {
#pragma unroll
                for (int j = 0; j < NI; ++j) b[kk][j] = read_b(j, kk, slot);
              }
#pragma unroll
              for (int i = 0; i < PI; ++i) a[(part + 1) & 1][i] = read_a(row + i, kk, slot);
            } else {
              wait_copies<0>();  // step s is in registers, and this wave's copies of step s + 1 have landed
              barrier();
              if (s + 1 < x.steps) {
#pragma unroll
                for (int j = 0; j < NI; ++j) b[0][j] = read_b(j, 0, slot ^ 1);
#pragma unroll
                for (int i = 0; i < PI; ++i) a[0][i] = read_a(i, 0, slot ^ 1);
              }
            }
            __builtin_amdgcn_sched_barrier(0);
            // the copies of the next step but one begin where everyone has read this one
            if (part == PARTS - 1 && s + 2 < x.steps) {
              more_rows(x, s);
              copy_a(x, s + 2, slot);
            }
            if (part == 0 && s > 0 && s + 1 < x.steps) copy_b(x, s + 1, slot ^ 1);
            if (part == 1) fetch_rows(x, s + 2);
#pragma unroll
            for (int i = 0; i < PI; ++i)
#pragma unroll
              for (int j = 0; j < NI; ++j) {
                gf32x4& c = acc[part % ROWS * PI + i][j];
                c = GMfma<T>::run(b[part / ROWS][j], a[part & 1][i], c);
              }
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      }
    } else {
      for (int s = 0; s < x.steps; ++s) {
        const int slot = s & 1;
        put(x, s, slot);  // its last readers were done before the last barrier
        more_rows(x, s);
        if (s + 1 < x.steps) {
          copy_a(x, s + 1, 0);
          copy_b(x, s + 1, 0);
        }
        wait_lds();  // (the copies stay under way; row numbers come 14 steps before they are read)
        barrier();
        fetch_rows(x, s + 2);
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
          gu32x4 b[NI];
#pragma unroll
          for (int j = 0; j < NI; ++j) b[j] = read_b(j, kk, slot);
#pragma unroll
          for (int i = 0; i < MI; ++i) {
            const gu32x4 a = read_a(i, kk, slot);
#pragma unroll
            for (int j = 0; j < NI; ++j) acc[i][j] = GMfma<T>::run(b[j], a, acc[i][j]);
          }
        }
      }
      wait_copies<0>();
      barrier();
    }

    // Lane (g, c16) holds columns 4g..4g+3 of row c16 of each 16 x 16 block.
    const int g = fresh(tid) >> 4 & 3, c16 = fresh(tid) & 15;
    const GroupTile t = x.t;
    const int m0 = x.m0, n0 = x.n0;
    if (tile >= 0) {
      if constexpr (EARLY) x = next;
      else
        locate(x, tile);
      set_up(x);
      start(x);
    }

    if constexpr (OP == kGroupWgrad) {
      // (of experts that overlap the longest runs, taken first, may be numbered past the planned ones)
      const bool room = t.count == 1 || t.run < planned;
      float* out = t.count == 1 ? k.dw + static_cast<int64_t>(t.e) * k.cin * k.cout : k.part + t.run * k.cin * k.cout;
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const int m = m0 + wm * MI * 16 + i * 16 + c16;
        if (m >= k.cin || !room) continue;
#pragma unroll
        for (int j = 0; j < NI; ++j) {
          const int n = n0 + wn * NI * 16 + j * 16 + 4 * g;
          float* p = out + static_cast<int64_t>(m) * k.cout + n;
          if (VEC) {
            if (n < k.cout) *reinterpret_cast<gf32x4*>(p) = acc[i][j];
          } else if (n + 4 <= k.cout) {
            *reinterpret_cast<Loose4*>(p) = __builtin_bit_cast(Loose4, acc[i][j]);
          } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (n + r < k.cout) p[r] = acc[i][j][r];
          }
        }
      }
    } else {
      typedef T t4 __attribute__((ext_vector_type(4)));
      typedef T t8 __attribute__((ext_vector_type(8)));
      typedef unsigned u2 __attribute__((ext_vector_type(2)));
      T* y = static_cast<T*>(k.y);
      // Blocks j0 and j1 of a row, whose first columns are c and c + 16: 64 bytes of 4 lanes at
      // once (a lane's own 8 bytes would make twice the requests).  Results stay in L2.  (Stored past it, us
      // plain / past, 609,756 rows 128 -> 2 x 256 with h: the same call over and over 363 / 276, but 345 / 392 after any
      // other one, the product that reads y 128 / 111, the gradient with glu 327 / 353 as part of a step; a layer's
      // products and sum forward 527 / 553, and back 1223 / 1277.)
      auto store = [&](T* row, int c, gf32x4 p, gf32x4 q) {
        const u2 a = __builtin_bit_cast(u2, __builtin_convertvector(p, t4)), b = __builtin_bit_cast(u2, __builtin_convertvector(q, t4));
        unsigned a0 = a[0], a1 = a[1], b0 = b[0], b1 = b[1];
        join8(a0, b0);
        join8(a1, b1);
        const gu32x4 v{a0, a1, b0, b1};
        const int n = c + 8 * g;
        if (!row || n >= N) return;
        if (VEC) *reinterpret_cast<gu32x4*>(row + n) = v;
        else store_loose(row, n, N, v);
      };
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const int r = wm * MI * 16 + i * 16 + c16;
        const bool in = r < t.rows;  // (all lanes take part in the exchange)
        const int64_t row = t.row0 + r;
        if constexpr (GLU && OP == kGroupFwd) {
          T* yr = in ? y + row * N : nullptr;
          T* h = in && k.h_out ? static_cast<T*>(k.h_out) + row * 2 * N : nullptr;
          gf32x4 v[NI / 2];
#pragma unroll
          for (int j = 0; j < NI / 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) v[j][e] = acc[i][2 * j][e] * sigmoid(acc[i][2 * j][e]) * acc[i][2 * j + 1][e];
#pragma unroll
          for (int j = 0; j < NI / 2; j += 2) {
            const int c = n0 + wn * NI * 8 + j * 16;
            store(yr, c, v[j], v[j + 1]);
            if (k.h_out) {
              store(h, c, acc[i][2 * j], acc[i][2 * j + 2]);
              store(h ? h + N : h, c, acc[i][2 * j + 1], acc[i][2 * j + 3]);
            }
          }
        } else if constexpr (GLU) {
          const T* h = in ? static_cast<const T*>(k.h) + row * 2 * N : nullptr;
          T* out = in ? y + row * 2 * N : nullptr;
#pragma unroll
          for (int j = 0; j < NI; j += 2) {
            const int c = n0 + wn * NI * 16 + j * 16;
            const int n = c + 8 * g;
            t8 a{}, b{};
            if (in && n < N) {
              if constexpr (VEC) {
                a = *reinterpret_cast<const t8*>(h + n);
                b = *reinterpret_cast<const t8*>(h + N + n);
              } else {
                a = __builtin_bit_cast(t8, load_loose(h, n, N));
                b = __builtin_bit_cast(t8, load_loose(h + N, n, N));
              }
            }
            float d[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              unsigned p = __builtin_bit_cast(unsigned, static_cast<float>(acc[i][j][e])), q = __builtin_bit_cast(unsigned, static_cast<float>(acc[i][j + 1][e]));
              join8(p, q);
              d[e] = __builtin_bit_cast(float, p);
              d[4 + e] = __builtin_bit_cast(float, q);
            }
            t8 da, db;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float av = static_cast<float>(a[e]), bv = static_cast<float>(b[e]), s = sigmoid(av);
              da[e] = static_cast<T>(d[e] * bv * s * fmaf(av, 1.f - s, 1.f));
              db[e] = static_cast<T>(d[e] * av * s);
            }
            if (in && n < N) {
              if constexpr (VEC) {
                *reinterpret_cast<t8*>(out + n) = da;
                *reinterpret_cast<t8*>(out + N + n) = db;
              } else {
                store_loose(out, n, N, __builtin_bit_cast(gu32x4, da));
                store_loose(out + N, n, N, __builtin_bit_cast(gu32x4, db));
              }
            }
          }
        } else {
          T* yr = in ? y + row * N : nullptr;
#pragma unroll
          for (int j = 0; j < NI; j += 2) store(yr, n0 + wn * NI * 16 + j * 16, acc[i][j], acc[i][j + 1]);
        }
      }
    }
  }

  if constexpr (OP != kGroupWgrad) {
    const GroupRest rest = rows_unowned(k);
    for (int64_t i = blockIdx.x;; i += gridDim.x) {
      const int64_t r = i / k.n_tiles;
      if (r * BM >= rest.n) break;
      zero_results<T, OP, GLU>(k, rest, r * BM, BM, N, static_cast<int>(i - r * k.n_tiles) * kCols, kCols);
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
  for (int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4; i < size; i += 4 * step) {
    if (i + 4 <= size) {
      gf32x4 s{0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
      for (int c = 0; c < count; ++c) s += __builtin_bit_cast(gf32x4, *reinterpret_cast<const Loose4*>(part + c * size + i));
      *reinterpret_cast<Loose4*>(dw + i) = __builtin_bit_cast(Loose4, s);
    } else {
      for (int64_t j = i; j < size; ++j) {
        float s = 0.f;
#pragma unroll 8
        for (int c = 0; c < count; ++c) s += part[c * size + j];
        dw[j] = s;
      }
    }
  }
}

template <typename T, GroupOp OP, bool GLU, int BM, int BN, int WM, int WN, bool VEC>
void run(GroupK& k, hipStream_t s) {
  const int N = OP == kGroupDgrad ? k.cin : k.cout;
  k.n_tiles = ceil_div(N, GLU && OP == kGroupFwd ? BN / 2 : BN);
  // as many blocks as are resident: one of 128 KB, or two of 64 KB, of LDS on each of 256 CUs
  const int64_t runs = OP == kGroupWgrad ? group_chunks(k.n_rows, k.e, k.chunk) * ceil_div(k.cin, BM) : group_runs(k.n_rows, k.e, BM);
  const int64_t tiles = (runs * k.n_tiles + 7) / 8 * 8, most = BM == 128 ? 512 : 256;
  k_group<T, OP, GLU, BM, BN, WM, WN, VEC><<<static_cast<unsigned>(tiles < most ? tiles : most), WM * WN * 64, 0, s>>>(k);
}

template <typename T, GroupOp OP, bool GLU>
void run(GroupK& k, hipStream_t s) {
  const GroupForm f = form_of(k, OP, GLU);
  if (!f.whole) return run<T, OP, GLU, 128, 128, 2, 2, false>(k, s);
  if (f.rows == 128) return run<T, OP, GLU, 128, 128, 2, 2, true>(k, s);
  if constexpr (OP != kGroupWgrad) {
    if (f.rows == 192) return run<T, OP, GLU, 192, 256, 2, 4, true>(k, s);
  }
  run<T, OP, GLU, 256, 256, 2, 4, true>(k, s);
}

template <typename T>
void run(GroupK& k, GroupOp op, bool glu, hipStream_t s) {
  if (op == kGroupFwd) return glu ? run<T, kGroupFwd, true>(k, s) : run<T, kGroupFwd, false>(k, s);
  if (op == kGroupDgrad) return glu ? run<T, kGroupDgrad, true>(k, s) : run<T, kGroupDgrad, false>(k, s);
  run<T, kGroupWgrad, false>(k, s);
  const int64_t size = static_cast<int64_t>(k.cin) * k.cout;
  // (most experts have nothing to add up: a few thousand blocks in all)
  const int64_t blocks = ceil_div<int64_t>(size, 1024), most = k.e < 2048 ? 4096 / k.e : 2;
  k_group_sum<<<dim3(static_cast<unsigned>(blocks < most ? blocks : most), k.e), 256, 0, s>>>(k);
}

}  // namespace

hipError_t launch_group(GroupK& k, GroupOp op, ts_dtype dt, bool glu, hipStream_t s) {
  if (dt == TS_F16) run<_Float16>(k, op, glu, s);
  else
    run<__bf16>(k, op, glu, s);
  return hipGetLastError();
}

}  // namespace ts
