// Weight gradient: dW[o] = sum over the pairs (i, j) of offset o of
// x[i]^T dy[j]  -- one (Cin x M_o) . (M_o x Cout) product per offset, needed
// for the mixed-precision training the TorchSparse++ abstract reports.
//
// The pairs of each offset are cut into chunks of kChunk pairs.  A block
// reduces one chunk for one (Cin, Cout) tile into a private fp32 partial;
// k_wgrad_reduce then sums the partials of each offset in chunk order, so
// the result does not depend on scheduling (no atomics).
//
// fp16/bf16 with channel counts that are multiples of 16 use MFMA.  A block
// owns a TW x TW tile of dW[o] (2 x 2 waves) and walks its chunk in steps of
// 64 pairs.  Per step, each staging thread gathers 8 rows x 8 channels
// (16-byte loads of x[pair_in] or dy[pair_out]), transposes the 8 x 8 block
// in registers and writes 8 channel rows of 8 consecutive pairs to LDS, so
// every MFMA fragment (8 consecutive pairs of one channel) is one 16-byte
// LDS read.  Pair indices are loaded three steps ahead and rows two steps
// ahead (register rings), the LDS slab is double-buffered, one barrier per
// step.
//
// x may also come in 8 bits (act8.h): the staging threads of x then read 8 codes
// and their block's byte per row and turn them into 16-bit values (act8.h) on the way to
// LDS; nothing else differs.  That form takes channel counts in
// multiples of 8 and halves the bytes gathered from x.
#include "act8.h"
#include "common.h"
#include "launch.h"

namespace ts {

namespace {

constexpr int kChunk = 2048;   // pairs per partial
// With x in 8 bits the chunk is what cuts the map's pairs into about as many
// chunks as the GPU runs blocks at once, found on the device (only it knows the
// pairs): a whole round of blocks, instead of one and a part, and a workspace that
// does not grow with the rows.
// 305k rows, 128 -> 128: 68 us and 11 for the sum; for 256 103 + 10, for 1024 78 + 17.
constexpr int kBlocks8 = 512;  // 256 CUs with 2 blocks of k_wgrad_mfma each
// 161k pixels, 8 -> 8: 15.2 us and 3.9 for the sum; for 2048 16.6 + 4.2, for 4096 17.6 + 4.3.
constexpr int kBlocks8Small = 1024;
constexpr int kWStep = 64;     // pairs per step
constexpr int kWStride = kWStep;  // halves per LDS channel row (128 bytes)

// LDS address (in halves) of the 16-byte chunk pc (8 pairs) of channel row
// ch.  The chunk index is XOR-swizzled with bits of ch so that the 16 lanes
// of a fragment read (16 consecutive channels, one chunk) hit 16 different
// 16-byte bank groups, and the transposed stores (16 channels 8 apart) at
// most two lanes per group.
__device__ __forceinline__ int slab_at(int ch, int pc) { return ch * kWStride + ((pc ^ ((ch >> 1) ^ (ch >> 3))) & 7) * 8; }

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

template <typename T>
struct WMfma;
template <>
struct WMfma<_Float16> {
  typedef f16x8 frag;
  static __device__ __forceinline__ f32x4 run(frag a, frag b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
};
template <>
struct WMfma<__bf16> {
  typedef bf16x8 frag;
  static __device__ __forceinline__ f32x4 run(frag a, frag b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};

// chunk_base[o] = number of chunks of offsets < o; chunk_base[kvol] = total.
__global__ void k_wgrad_chunks(const int64_t* __restrict__ pair_start, int kvol, int32_t* __restrict__ chunk_base) {
  if (threadIdx.x != 0) return;
  int32_t acc = 0;
  for (int o = 0; o < kvol; ++o) {
    chunk_base[o] = acc;
    const int64_t cnt = pair_start[o + 1] - pair_start[o];
    acc += static_cast<int32_t>((cnt + kChunk - 1) / kChunk);
  }
  chunk_base[kvol] = acc;
}

// Which offset / pair range block `c` covers; false for blocks past the end.
__device__ __forceinline__ bool chunk_range(const int32_t* chunk_base, const int64_t* pair_start, int kvol, int c,
                                            int* o_out, int64_t* p0, int64_t* p1) {
  if (c >= chunk_base[kvol]) return false;
  int o = 0;
  while (o + 1 < kvol && chunk_base[o + 1] <= c) ++o;
  const int64_t begin = pair_start[o] + static_cast<int64_t>(c - chunk_base[o]) * kChunk;
  const int64_t end = pair_start[o + 1];
  *o_out = o;
  *p0 = begin;
  *p1 = begin + kChunk < end ? begin + kChunk : end;
  return true;
}

// A lane's value as a wave-uniform one (a vector register per use otherwise).
__device__ __forceinline__ int32_t lane_value(int32_t v, int lane) { return __builtin_amdgcn_readlane(v, lane); }
__device__ __forceinline__ int64_t lane_value(int64_t v, int lane) {
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int32_t>(v), lane);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int32_t>(v >> 32), lane);
  return static_cast<int64_t>((static_cast<uint64_t>(hi) << 32) | lo);
}

// The chunks of x in 8 bits: at most target + kvol, of a multiple of 64 pairs.  Every
// wave works them out from the pair starts, lane o those of offset o (kvol <= 64):
// one read of at most 65 words instead of a launch before the product.
struct WaveChunks {
  int64_t chunk, start, end;  // pairs per chunk; this lane's offset: its pairs,
  int32_t first, count;       // first chunk and chunks
  __device__ __forceinline__ WaveChunks(const int64_t* pair_start, int kvol, int target) {
    const int o = threadIdx.x & 63;
    start = pair_start[o < kvol ? o : kvol];
    end = pair_start[o < kvol ? o + 1 : kvol];
    const int64_t total = lane_value(end, kvol - 1) - lane_value(start, 0);
    const int64_t per = (total + target - 1) / target;
    chunk = per < 256 ? 256 : (per + 63) / 64 * 64;
    count = static_cast<int32_t>((end - start + chunk - 1) / chunk);
    int32_t sum = count;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int32_t v = __shfl_up(sum, d);
      if (o >= d) sum += v;
    }
    first = sum - count;
  }
  // Chunk c's offset and pairs; false past the last chunk.
  __device__ __forceinline__ bool range(int c, int* o, int64_t* p0, int64_t* p1) const {
    const uint64_t in = __ballot(c >= first && c < first + count);
    if (in == 0) return false;
    *o = __ffsll(static_cast<unsigned long long>(in)) - 1;
    *p0 = lane_value(start, *o) + (c - lane_value(first, *o)) * chunk;
    const int64_t e = lane_value(end, *o);
    *p1 = *p0 + chunk < e ? *p0 + chunk : e;
    return true;
  }
};

template <int I>
struct WIc {
  static constexpr int v = I;
};

template <typename T, int TW, bool ACT8>
__global__ __launch_bounds__(256, 2) void k_wgrad_mfma(const int32_t* __restrict__ chunk_base, int target,
                                                    const int64_t* __restrict__ pair_start, int kvol,
                                                    const int32_t* __restrict__ pair_in,
                                                    const int32_t* __restrict__ pair_out, const T* __restrict__ x,
                                                    const Act8 x8, int cin, const T* __restrict__ dy, int cout,
                                                    float* __restrict__ partial, int64_t n_x, int64_t n_dy) {
  typedef typename WMfma<T>::frag Frag;
  constexpr int HT = TW / 2;   // channels per wave in each dim
  constexpr int NT = HT / 16;  // 16 x 16 MFMA tiles per wave in each dim
  constexpr int CG = TW / 8;   // 8-channel groups per operand
  __shared__ __attribute__((aligned(16))) T slab[2][2][TW * kWStride];  // [buffer][x | dy][channel][pair]
  const int c = blockIdx.x;
  int o;
  int64_t p0, p1;
  if constexpr (ACT8) {
    if (!WaveChunks(pair_start, kvol, target).range(c, &o, &p0, &p1)) return;
  } else {
    if (!chunk_range(chunk_base, pair_start, kvol, c, &o, &p0, &p1)) return;
  }
  const int ci0 = blockIdx.y * TW, co0 = blockIdx.z * TW;
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int wm = wave >> 1, wn = wave & 1;
  // staging role: operand, 8-pair group, 8-channel group
  const int op = threadIdx.x >> 7;
  const int tt = threadIdx.x & 127;
  const bool stager = tt < 8 * CG;
  const int pg = tt / CG, cg = tt % CG;
  const T* src = op ? dy : x;
  const int C = op ? cout : cin;
  const int ch = (op ? co0 : ci0) + cg * 8;
  const bool cok = stager && ch < C;
  const int32_t* rows = op ? pair_out : pair_in;
  const int nsteps = static_cast<int>((p1 - p0 + kWStep - 1) / kWStep);
  const bool from8 = ACT8 && __builtin_amdgcn_readfirstlane(op) == 0;  // this wave stages x (op is the same in a wave)
  const int blocks8 = ceil_div(cin, kActBlock);

  f32x4 acc[NT][NT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // Pair r of this thread's group at step st exists when it lies inside the
  // chunk (validity never depends on a loaded value, so no load is ever
  // placed under a branch).
  auto valid = [&](int st, int r) -> bool {
    return cok && p0 + static_cast<int64_t>(st) * kWStep + pg * 8 + r < p1;
  };
  // row indices of step st (clamped address; meaningful where valid)
  auto load_idx = [&](int st, int32_t (&id)[8]) __attribute__((always_inline)) {
    const int64_t q = p0 + static_cast<int64_t>(st) * kWStep + pg * 8;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const int64_t p = q + r;
      id[r] = rows[p < p1 ? p : p1 - 1];
    }
  };
  // rows of step st; absent pairs read row 0 and are zeroed when staged
  auto row_of = [&](int st, const int32_t (&id)[8], int r) __attribute__((always_inline)) -> int64_t {
    return valid(st, r) ? dbg_req(id[r], op ? n_dy : n_x, op ? TS_DEBUG_DST_ROW : TS_DEBUG_SRC_ROW) : 0;
  };
  auto load_rows = [&](int st, const int32_t (&id)[8], u32x4 (&v)[8]) __attribute__((always_inline)) {
    if (ACT8 && from8) {
      const int c0 = cok ? ch : 0;
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const int64_t row = row_of(st, id, r);
        const ux2 codes = *reinterpret_cast<const ux2*>(x8.codes + row * cin + c0);
        v[r] = u32x4{codes[0], codes[1], x8.scales[row * blocks8 + c0 / kActBlock], 0u};
      }
    } else {
#pragma unroll
      for (int r = 0; r < 8; ++r)
        v[r] = *reinterpret_cast<const u32x4*>(src + row_of(st, id, r) * C + (cok ? ch : 0));
    }
  };
  // 8 x 8 transpose of 16-bit values: out row e = channel ch+e over the 8 pairs
  auto stage = [&](int st, u32x4 (&in)[8], T* buf) __attribute__((always_inline)) {
    if (!stager) return;
#pragma unroll
    for (int r = 0; r < 8; ++r) in[r] = valid(st, r) ? in[r] : u32x4{0u, 0u, 0u, 0u};  // in place
    if (ACT8 && from8) {
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        float f[8];
        act8_decode(ux2{in[r][0], in[r][1]}, act8_quantum(in[r][2]), f);
        Frag t;
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = static_cast<T>(f[e]);
        in[r] = __builtin_bit_cast(u32x4, t);
      }
    }
    T* base = buf + (op ? TW * kWStride : 0);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      u32x4 outv;
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const uint32_t a = in[2 * m][e >> 1], b = in[2 * m + 1][e >> 1];
        outv[m] = (e & 1) ? ((a >> 16) | (b & 0xffff0000u)) : ((a & 0xffffu) | (b << 16));
      }
      *reinterpret_cast<u32x4*>(base + slab_at(cg * 8 + e, pg)) = outv;
    }
  };
  auto mma = [&](const T* buf) __attribute__((always_inline)) {
    const T* xa = buf;
    const T* yb = buf + TW * kWStride;
#pragma unroll
    for (int kb = 0; kb < kWStep / 32; ++kb) {
      Frag af[NT], bf[NT];
#pragma unroll
      for (int i = 0; i < NT; ++i)
        af[i] = __builtin_bit_cast(
            Frag, *reinterpret_cast<const u32x4*>(xa + slab_at(wm * HT + i * 16 + (lane & 15), kb * 4 + (lane >> 4))));
#pragma unroll
      for (int j = 0; j < NT; ++j)
        bf[j] = __builtin_bit_cast(
            Frag, *reinterpret_cast<const u32x4*>(yb + slab_at(wn * HT + j * 16 + (lane & 15), kb * 4 + (lane >> 4))));
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = WMfma<T>::run(af[i], bf[j], acc[i][j]);
    }
  };

  // prologue: indices of steps 0..2, rows of steps 0..1, slab of step 0.
  // Index sets alternate: the set of step s+3 is loaded at step s into the
  // one whose rows (step s+1) were issued at step s-1.
  int32_t id[2][8];
  u32x4 rv[2][8];
  load_idx(0, id[0]);
  load_idx(1, id[1]);
  load_rows(0, id[0], rv[0]);
  load_rows(1, id[1], rv[1]);
  load_idx(2, id[0]);
  stage(0, rv[0], &slab[0][0][0]);
  __syncthreads();
  int s = 0;
  // step s: indices of s+3, rows of s+2, multiplies of s, staging of s+1
  auto step = [&](auto ic) __attribute__((always_inline)) -> bool {
    constexpr int i = decltype(ic)::v;
    load_idx(s + 3, id[(i + 3) & 1]);
    load_rows(s + 2, id[(i + 2) & 1], rv[i & 1]);
    mma(&slab[i & 1][0][0]);
    if (++s >= nsteps) return false;
    stage(s, rv[(i + 1) & 1], &slab[(i + 1) & 1][0][0]);
    __syncthreads();
    return true;
  };
  while (step(WIc<0>{}) && step(WIc<1>{}) && step(WIc<2>{}) && step(WIc<3>{})) {
  }

  // D[m][n]: lane holds n = lane%16, m = 4*(lane/16) + e
  float* part = partial + static_cast<int64_t>(c) * cin * cout;
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int co = co0 + wn * HT + j * 16 + (lane & 15);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int ci = ci0 + wm * HT + i * 16 + (lane >> 4) * 4 + e;
        if (ci < cin && co < cout) part[static_cast<int64_t>(ci) * cout + co] = acc[i][j][e];
      }
    }
}

// FMA fallback: thread = one (ci, co) element of a 256-element tile.  305k rows from 8
// bits, 27 -> 65 channels 0.89 ms, 129 -> 33 2.98 ms (the matrix cores take 128 -> 128 in
// 0.08): bound by the loads of each pair's two values.
template <typename T, bool ACT8>
__global__ __launch_bounds__(256) void k_wgrad_fma(const int32_t* __restrict__ chunk_base, int target,
                                                   const int64_t* __restrict__ pair_start, int kvol,
                                                   const int32_t* __restrict__ pair_in,
                                                   const int32_t* __restrict__ pair_out, const T* __restrict__ x,
                                                   const Act8 x8, int cin, const T* __restrict__ dy, int cout,
                                                   float* __restrict__ partial, int64_t n_x, int64_t n_dy) {
  const int c = blockIdx.x;
  int o;
  int64_t p0, p1;
  if constexpr (ACT8) {
    if (!WaveChunks(pair_start, kvol, target).range(c, &o, &p0, &p1)) return;
  } else {
    if (!chunk_range(chunk_base, pair_start, kvol, c, &o, &p0, &p1)) return;
  }
  const int64_t e = static_cast<int64_t>(blockIdx.y) * 256 + threadIdx.x;
  if (e >= static_cast<int64_t>(cin) * cout) return;
  const int ci = static_cast<int>(e / cout), co = static_cast<int>(e % cout);
  float acc = 0.f;
  for (int64_t p = p0; p < p1; ++p) {
    const int64_t i = dbg_req(pair_in[p], n_x, TS_DEBUG_SRC_ROW);
    float xv;
    if constexpr (ACT8)
      // as a T: what the other forms multiply, and what unpacking gives
      xv = static_cast<float>(static_cast<T>(static_cast<float>(x8.codes[i * cin + ci]) *
                                             act8_quantum(x8.scales[i * ceil_div(cin, kActBlock) + ci / kActBlock])));
    else
      xv = static_cast<float>(x[i * cin + ci]);
    acc = fmaf(xv,
               static_cast<float>(dy[static_cast<int64_t>(dbg_req(pair_out[p], n_dy, TS_DEBUG_DST_ROW)) * cout + co]),
               acc);
  }
  partial[static_cast<int64_t>(c) * cin * cout + e] = acc;
}

// x in 8 bits with at most 16 channels on either side: dW[o] is one 16 x 16 MFMA
// tile, and a row is one or two 16-byte pieces, so the fragments (8 pairs of one
// channel per lane) are gathered straight from memory, without LDS.  A wave takes
// 32 pairs at a time, the four waves of a block in turn; indices are read two
// steps ahead and rows one.  Any channel count and alignment.
template <typename T>
__global__ __launch_bounds__(256) void k_wgrad_small(int target, const int64_t* __restrict__ pair_start, int kvol,
                                                     const int32_t* __restrict__ pair_in,
                                                     const int32_t* __restrict__ pair_out, const Act8 x8, int cin,
                                                     const T* __restrict__ dy, int cout, float* __restrict__ partial,
                                                     int64_t n_x, int64_t n_dy) {
  typedef typename WMfma<T>::frag Frag;
  __shared__ f32x4 sums[4][64];
  const int c = blockIdx.x;
  int o;
  int64_t p0, p1;
  if (!WaveChunks(pair_start, kvol, target).range(c, &o, &p0, &p1)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, ch = lane & 15, g = lane >> 4;
  const int ci = ch < cin ? ch : 0, co = ch < cout ? ch : 0;
  struct Rows {
    int8_t code[8];
    uint8_t byte[8];
    T y[8];
  };
  auto load_idx = [&](int64_t p, int32_t (&a)[8], int32_t (&b)[8]) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t q = p + g * 8 + j < p1 ? p + g * 8 + j : p1 - 1;
      a[j] = pair_in[q];
      b[j] = pair_out[q];
    }
  };
  auto load_rows = [&](const int32_t (&a)[8], const int32_t (&b)[8], Rows& r) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t i = dbg_req(a[j], n_x, TS_DEBUG_SRC_ROW), q = dbg_req(b[j], n_dy, TS_DEBUG_DST_ROW);
      r.code[j] = x8.codes[i * cin + ci];
      r.byte[j] = x8.scales[i];
      r.y[j] = dy[q * cout + co];
    }
  };
  f32x4 acc{0.f, 0.f, 0.f, 0.f};
  int32_t ia[8], ib[8];
  Rows cur;
  int64_t p = p0 + wave * 32;
  if (p < p1) {
    load_idx(p, ia, ib);
    load_rows(ia, ib, cur);
    load_idx(p + 128, ia, ib);
    for (; p < p1; p += 128) {
      Rows next;
      load_rows(ia, ib, next);
      load_idx(p + 256, ia, ib);
      Frag af, bf;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool ok = p + g * 8 + j < p1;
        af[j] = static_cast<T>(ok && ch < cin ? static_cast<float>(cur.code[j]) * act8_quantum(cur.byte[j]) : 0.f);
        bf[j] = ok && ch < cout ? cur.y[j] : static_cast<T>(0.f);
      }
      acc = WMfma<T>::run(af, bf, acc);
      cur = next;
    }
  }
  sums[wave][lane] = acc;
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float v = (sums[0][lane][e] + sums[1][lane][e]) + (sums[2][lane][e] + sums[3][lane][e]);
    const int row = g * 4 + e;  // D: lane holds column lane % 16, rows 4g..4g+3
    if (row < cin && ch < cout) partial[(static_cast<int64_t>(c) * cin + row) * cout + ch] = v;
  }
}

// dw[o][e] = sum of the partials of offset o in chunk order.
__global__ __launch_bounds__(256) void k_wgrad_reduce(const int32_t* __restrict__ chunk_base, int kvol,
                                                      const float* __restrict__ partial, int64_t elems,
                                                      float* __restrict__ dw) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= elems * kvol) return;
  const int o = static_cast<int>(i / elems);
  const int64_t e = i % elems;
  const int c0 = chunk_base[o], c1 = chunk_base[o + 1];
  float s = 0.f;
  int c = c0;
  for (; c + 8 <= c1; c += 8) {  // loads issued together, summed in chunk order
    float v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = partial[static_cast<int64_t>(c + u) * elems + e];
#pragma unroll
    for (int u = 0; u < 8; ++u) s += v[u];
  }
  for (; c < c1; ++c) s += partial[static_cast<int64_t>(c) * elems + e];
  dw[i] = s;
}

// The same over the chunks of x in 8 bits: block row o, 256 / SH elements a block,
// SH shares of the chunks (c, c + SH, ...) joined in LDS in order.
template <int SH>
__global__ __launch_bounds__(256) void k_wgrad_reduce_act8(const int64_t* __restrict__ pair_start, int kvol, int target,
                                                           const float* __restrict__ partial, int64_t elems,
                                                           float* __restrict__ dw) {
  constexpr int EL = 256 / SH;
  __shared__ float sums[SH][EL];
  const WaveChunks w(pair_start, kvol, target);
  const int o = blockIdx.y, c0 = lane_value(w.first, o), c1 = c0 + lane_value(w.count, o);
  const int x = threadIdx.x % EL, sh = threadIdx.x / EL;
  const int64_t e = static_cast<int64_t>(blockIdx.x) * EL + x;
  float s = 0.f;
  if (e < elems)
#pragma unroll 4
    for (int c = c0 + sh; c < c1; c += SH) s += partial[static_cast<int64_t>(c) * elems + e];
  sums[sh][x] = s;
  __syncthreads();
  if (sh != 0 || e >= elems) return;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < SH; ++i) s += sums[i][x];
  dw[o * elems + e] = s;
}

int64_t max_chunks(const ts_kmap* map) { return map->pair_cap / kChunk + map->kvol + 1; }

dim3 grid_chunks(unsigned nch, int cin, int cout, int tw) {
  return dim3(nch, static_cast<unsigned>(ceil_div(cin, tw)), static_cast<unsigned>(ceil_div(cout, tw)));
}

template <int TW, bool ACT8>
void launch_wgrad_mfma(dim3 grid, ts_dtype dt, const ts_kmap* map, const void* x, const Act8& x8, int cin, const void* dy,
                       int cout, const int32_t* chunk_base, int target, float* partial, hipStream_t s) {
  if (dt == TS_F16)
    k_wgrad_mfma<_Float16, TW, ACT8><<<grid, 256, 0, s>>>(chunk_base, target, map->pair_start, map->kvol, map->pair_in,
                                                          map->pair_out, static_cast<const _Float16*>(x), x8, cin,
                                                          static_cast<const _Float16*>(dy), cout, partial, map->n_in,
                                                          map->n_out_cap);
  else
    k_wgrad_mfma<__bf16, TW, ACT8><<<grid, 256, 0, s>>>(chunk_base, target, map->pair_start, map->kvol, map->pair_in,
                                                        map->pair_out, static_cast<const __bf16*>(x), x8, cin,
                                                        static_cast<const __bf16*>(dy), cout, partial, map->n_in,
                                                        map->n_out_cap);
}

template <typename T, bool ACT8>
void launch_wgrad_fma(dim3 grid, const ts_kmap* map, const void* x, const Act8& x8, int cin, const void* dy, int cout,
                      const int32_t* chunk_base, int target, float* partial, hipStream_t s) {
  k_wgrad_fma<T, ACT8><<<grid, 256, 0, s>>>(chunk_base, target, map->pair_start, map->kvol, map->pair_in, map->pair_out,
                                            static_cast<const T*>(x), x8, cin, static_cast<const T*>(dy), cout, partial,
                                            map->n_in, map->n_out_cap);
}

}  // namespace

size_t wgrad_workspace_bytes(const ts_kmap* map, int cin, int cout) {
  return align_up(static_cast<size_t>(map->kvol + 1) * 4, 256) +
         static_cast<size_t>(max_chunks(map)) * cin * cout * 4;
}

hipError_t launch_wgrad(const ts_kmap* map, const void* x, int cin, const void* dy, int cout, ts_dtype dt, float* dw,
                        void* ws, hipStream_t s) {
  int32_t* chunk_base = static_cast<int32_t*>(ws);
  float* partial = reinterpret_cast<float*>(static_cast<char*>(ws) + align_up(static_cast<size_t>(map->kvol + 1) * 4, 256));
  const int64_t elems = static_cast<int64_t>(cin) * cout;
  k_wgrad_chunks<<<1, 64, 0, s>>>(map->pair_start, map->kvol, chunk_base);
  const unsigned nch = static_cast<unsigned>(max_chunks(map));
  // The MFMA kernel stages rows with 16-byte loads: rows of 16-channel
  // multiples are 16-byte aligned when the matrices are; otherwise the FMA
  // kernel, which reads element by element, takes the layer.
  const bool aligned = (reinterpret_cast<uintptr_t>(x) & 15) == 0 && (reinterpret_cast<uintptr_t>(dy) & 15) == 0;
  const bool mfma = dt != TS_F32 && cin % 16 == 0 && cout % 16 == 0 && aligned;
  const Act8 none{nullptr, nullptr, false};
  if (mfma) {
    if (cin >= 128 && cout >= 128)
      launch_wgrad_mfma<128, false>(grid_chunks(nch, cin, cout, 128), dt, map, x, none, cin, dy, cout, chunk_base, 0, partial, s);
    else
      launch_wgrad_mfma<64, false>(grid_chunks(nch, cin, cout, 64), dt, map, x, none, cin, dy, cout, chunk_base, 0, partial, s);
  } else {
    dim3 grid(nch, static_cast<unsigned>(ceil_div<int64_t>(elems, 256)));
    switch (dt) {
      case TS_F32: launch_wgrad_fma<float, false>(grid, map, x, none, cin, dy, cout, chunk_base, 0, partial, s); break;
      case TS_F16: launch_wgrad_fma<_Float16, false>(grid, map, x, none, cin, dy, cout, chunk_base, 0, partial, s); break;
      default: launch_wgrad_fma<__bf16, false>(grid, map, x, none, cin, dy, cout, chunk_base, 0, partial, s); break;
    }
  }
  const int64_t total = elems * map->kvol;
  k_wgrad_reduce<<<static_cast<unsigned>(ceil_div<int64_t>(total, 256)), 256, 0, s>>>(chunk_base, map->kvol, partial,
                                                                                     elems, dw);
  return hipGetLastError();
}

namespace {
// (161k pixels, 8 -> 8: 16.6 us against 40 for the tiles of the matrix cores, which
// would be 1/64 full)
bool wgrad_is_small(int cin, int cout) { return cin <= 16 && cout <= 16; }
// Chunks aimed at: blocks that run at once, over the dW tiles of each chunk.
int wgrad_act8_target(int cin, int cout) {
  if (wgrad_is_small(cin, cout)) return kBlocks8Small;
  const int tw = cin >= 128 && cout >= 128 ? 128 : 64;
  const int t = kBlocks8 / (ceil_div(cin, tw) * ceil_div(cout, tw));
  return t < 32 ? 32 : t;
}
}  // namespace

size_t wgrad_act8_workspace_bytes(const ts_kmap* map, int cin, int cout) {
  return static_cast<size_t>(wgrad_act8_target(cin, cout) + map->kvol) * cin * cout * 4;
}

hipError_t launch_wgrad_act8(const ts_kmap* map, const Act8& x, int cin, const void* dy, int cout, ts_dtype dt, float* dw,
                             void* ws, hipStream_t s) {
  float* partial = static_cast<float*>(ws);
  const int64_t elems = static_cast<int64_t>(cin) * cout;
  // the offsets' last chunks are not whole: kvol fewer are aimed at, so that about `target` come out
  const int most = wgrad_act8_target(cin, cout), target = most > 2 * map->kvol ? most - map->kvol : most;
  const unsigned nch = static_cast<unsigned>(target + map->kvol);
  const bool mfma = x.vec && cout % 8 == 0 && (reinterpret_cast<uintptr_t>(dy) & 15) == 0;
  if (wgrad_is_small(cin, cout)) {
    if (dt == TS_F16)
      k_wgrad_small<_Float16><<<nch, 256, 0, s>>>(target, map->pair_start, map->kvol, map->pair_in, map->pair_out, x, cin,
                                                  static_cast<const _Float16*>(dy), cout, partial, map->n_in, map->n_out_cap);
    else
      k_wgrad_small<__bf16><<<nch, 256, 0, s>>>(target, map->pair_start, map->kvol, map->pair_in, map->pair_out, x, cin,
                                                static_cast<const __bf16*>(dy), cout, partial, map->n_in, map->n_out_cap);
  } else if (mfma) {
    if (cin >= 128 && cout >= 128)
      launch_wgrad_mfma<128, true>(grid_chunks(nch, cin, cout, 128), dt, map, nullptr, x, cin, dy, cout, nullptr, target, partial, s);
    else
      launch_wgrad_mfma<64, true>(grid_chunks(nch, cin, cout, 64), dt, map, nullptr, x, cin, dy, cout, nullptr, target, partial, s);
  } else {
    const dim3 grid(nch, static_cast<unsigned>(ceil_div<int64_t>(elems, 256)));
    if (dt == TS_F16)
      launch_wgrad_fma<_Float16, true>(grid, map, nullptr, x, cin, dy, cout, nullptr, target, partial, s);
    else
      launch_wgrad_fma<__bf16, true>(grid, map, nullptr, x, cin, dy, cout, nullptr, target, partial, s);
  }
  // shares per element: about 8 partials each
  const int per_offset = target / map->kvol;
  const auto blocks = [&](int shares) { return dim3(static_cast<unsigned>(ceil_div<int64_t>(elems, 256 / shares)), map->kvol); };
  if (per_offset > 64)
    k_wgrad_reduce_act8<32><<<blocks(32), 256, 0, s>>>(map->pair_start, map->kvol, target, partial, elems, dw);
  else
    k_wgrad_reduce_act8<4><<<blocks(4), 256, 0, s>>>(map->pair_start, map->kvol, target, partial, elems, dw);
  return hipGetLastError();
}

}  // namespace ts

TS_DEBUG_TU(wgrad)
