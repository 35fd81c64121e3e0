// Attention within packed sets, forward: one walk over the keys with a running
// maximum and sum (see attn.h for the operand layout).
//
// Vector instructions bound it: 64 scores of 64 channels take 16 cycles of a SIMD in
// matrix instructions and, with a cap, 36 in vector ones (4 each, 8 for exp2, rcp and
// sqrt), one after the other; together they fill 80 % of the kernel at 4 x 4096 capped
// rows, 71 % at 2 x 8192 biased ones and 63 to 68 % in windows of 32 channels, where
// waves wait for LDS and memory in between.  So each score gets as few as possible:
//   - scores are kept in units of log 2 and relative to the column's reference
//     m, which is folded into the multiply-add that scales them;
//   - m follows the maximum only when a score passes it by more than a slack:
//     larger probabilities cost nothing in the 16-bit operand (rounding is
//     relative) nor in the fp32 sums, and most tiles need neither a maximum
//     across lanes nor a change of the accumulators;
//   - squared distances come from a matrix product (attn.h).
// A tile that moves a reference, and the first and a partial one, take the slow
// form: scores first, then their maximum, then p = exp2(z - m).  (It is also the
// accurate form where z and m are large: folding -m in rounds to m's precision.)  With
// the slow form alone 4 x 4096 capped rows take 354 us instead of 282, 2 x 8192 capped
// and biased ones 785 instead of 662.
// Probabilities are rounded to 16 bits for their product with the values (out is 1.05 to
// 1.41 times as far from 64 bits as its last rounding alone); calls of few rows (TWO,
// attn_plan.h) take what the rounding left as a second operand (1.0; one query over
// 102,835 keys 18.1 -> 18.7 us).
// Rows without a finite score give zeros and lse = -inf.
//
// Measured, whole calls in long runs: 4 sets of 4096, 8 heads of 64, capped, fp16 235 us
// (585 TFLOP/s); 1024 windows of about 100, 4 heads of 32, biased, bf16 55 us (1.8 TB/s);
// one query over 102,835 keys 22.7 us (2.4 TB/s); 1200 windows of about 127, 4 heads of
// 128, biased, bf16 235 us (2.4 TB/s); 2 sets of 4096, 8 heads of 128, capped 255 us (472
// TFLOP/s).  Times of one form against another, here and beside the rules, are kernel
// times by the profiler, twelve calls after a pause, which are up to 15 % longer (the
// first of these 286).
#include "attn.h"

namespace ts {

namespace {

// Where a reference is put, `lift` below the maximum that moves it, and how far a score
// may pass it, `top`: probabilities up to 2^top.  In fp16 the whole range is used, since
// what is 2^-24 or less is lost from the product while the sum counts it: a row's largest
// probability lies between 2^7 and 2^15, so one has to be 2^32 times smaller to be lost,
// and the maximum may still rise by 2^8 before the reference moves.  (From 1 to 2^12,
// 500 keys 2^-26 below the largest were a row's error.)  bf16 has fp32's range.
template <typename T>
struct Reach {
  static constexpr float lift = 0.f, top = 12.f;
};
template <>
struct Reach<_Float16> {
  static constexpr float lift = 7.f, top = 15.f;
};
// References up to this fold into the scores: that rounds them to 2^-24 of it.
constexpr float kFold = 256.f;

// A wave owns NC column blocks of 16 query rows.  NC 2 (long sets): a key tile read
// from LDS feeds both (2 x 8192 rows: 662 us, with NC 1 785).  KS (few query rows): all
// four waves own the same 16 columns and share out the keys of each tile, 32 each;
// their results are joined in LDS (one query over 102,835 keys: 18.0 us against 19.9 with
// one wave at work; attn_plan.h says where).
//
// A block takes a.heads key-value heads of its rows one after the other, as one walk
// over (head, tile): for short sets, finding the set and the first reads would
// cost more than a head's work, and the next head's rows are read while this one's
// last tile is computed.
template <typename T, int DP, int NC, bool CAP, bool BIAS, bool KS, bool TWO>
__global__ __launch_bounds__(256, attn_waves_fwd(DP, NC, CAP, BIAS, TWO)) void k_attn_fwd(const AttnArgs a) {
  typedef typename AMfma<T>::frag Frag;
  constexpr int KB = DP / 32, DI = DP / 16;
  constexpr int BN = KS ? 128 : 64;  // keys per tile
  constexpr int NT = KS ? 2 : 4;     // 16-key steps of a wave per tile
  constexpr int BM = KS ? 16 : 64 * NC;
  constexpr int TB = BN * DP * 2;
  constexpr bool MULTI = NC == 1 && !KS && DP <= 64;  // a.heads may be more than 1
  static_assert(!KS || (NC == 1 && DP <= 64 && TWO), "one column block of at most 64 channels, few rows when the waves share the keys");
  __shared__ __attribute__((aligned(16))) char tk[2][TB], tv[2][TB];
  constexpr int TCS = MULTI ? kCoordTiles : 2;
  __shared__ f32x4 tc[TCS][BIAS ? BN : 1];
  __shared__ uint32_t far_rows[TCS][2];

  const int64_t slot = block_tile();
  const int split = blockIdx.z;
  if (a.flags && blockIdx.y == 0 && split == 0 && threadIdx.x == 0) {
    check_starts(a.qs, a.nq, a.n_sets, slot, a.flags);
    if (a.ks != a.qs) check_starts(a.ks, a.nk, a.n_sets, slot, a.flags);
  }
  SetTile st;
  if (!find_tile<BM>(a.qs, a.nq, a.grp, a.ks, a.nk, a.n_sets, slot, a.tiles, &st)) return;
  int64_t kbeg, kend;
  split_range(st.st_len, BN, a.splits, split, &kbeg, &kend);

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4;
  const int kt0 = KS ? wave * 32 : 0;
  const int n_keys = static_cast<int>(kend - kbeg);
  const int h0 = blockIdx.y * a.heads;
  int h = h0;
  int cb = 0;  // where the tile's coordinates are
  const int h_end = !MULTI ? h + 1 : h + a.heads < a.hk ? h + a.heads : a.hk;

  const QueryCols<NC, KS> col(a, st, BM);
  const int width = a.grp * a.d;  // a key-value head's part of a query row
  const T* qp = static_cast<const T*>(a.q) + col.query0 * a.q_stride;
  const uint32_t qbytes = col.bytes(a.q_stride, width);
  Place org{0, 0, 0};
  Place oraw, qraw[NC];
  if constexpr (BIAS) {
    oraw = load_place(a.qc, st.own0, a.ndim);
#pragma unroll
    for (int j = 0; j < NC; ++j) qraw[j] = load_place(a.qc, col.query0 + col.dq[j], a.ndim);
  }
  ColLoad<T, DP, NC> qld;
  float next_slope[NC];
  auto fetch_cols = [&](int hn) {
    uint32_t qoff[NC];
#pragma unroll
    for (int j = 0; j < NC; ++j) qoff[j] = col.offset(j, a.q_stride, a.d);
    qld.fetch(qp + static_cast<int64_t>(hn) * width, qbytes, qoff, a.d);
    if constexpr (BIAS)
#pragma unroll
      for (int j = 0; j < NC; ++j) next_slope[j] = a.slopes[hn * a.grp + col.place[j]];
  };
  fetch_cols(h);
  KeyTiles<T, DP, BN, BIAS> keys(a, st.st0 + kbeg, n_keys);
  const bool stay = MULTI && n_keys <= TCS * BN;  // tile i's coordinates are in tc[i] from the first head on
  if (n_keys > 0) keys.fetch(a, h, 0, true);

  float slope[NC], qb[NC], qn[NC];  // (the last two: for the distances)
  bool far_cols = false;
  if constexpr (BIAS) {
    org = uniform_origin(oraw);
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const f32x4 c = relative(qraw[j], org, a.ndim);
      qb[j] = col_term(c, g);
      qn[j] = c[3];
      far_cols |= __any(c[3] > kNearNorm) != 0;
    }
  }

  const f32x4 zero{0.f, 0.f, 0.f, 0.f};
  Frag qf[NC][KB];
  f32x4 o[NC][DI];
  float l[NC], m[NC];  // m -inf: no finite score yet
  bool fold;           // every column has a reference that folds
  auto begin = [&]() {  // of head h, whose columns have been read
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      m[j] = -INFINITY;
      l[j] = 0.f;
#pragma unroll
      for (int i = 0; i < DI; ++i) o[j][i] = zero;
      // a negative scale is moved into q, so that c1 >= 0
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) qf[j][kb] = qld.frag_signed(j, kb, a.negate);
      if constexpr (BIAS) slope[j] = next_slope[j] * kLog2e;
    }
    fold = false;
  };

  // s = k . q of 16 keys
  auto product = [&](int b, int n, f32x4(&s)[NC]) {
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      const Frag f = tile_frag<T, DP>(tk[b], kt0 + n * 16, kb, lane);
#pragma unroll
      for (int j = 0; j < NC; ++j) s[j] = AMfma<T>::run(f, qf[j][kb], kb == 0 ? zero : s[j]);
    }
  };
  auto dist_of = [&](int b, int n, int j, bool far) {
    return distances(tc[cb], kt0 + n * 16, qn[j], qb[j], far, lane, a.qc, col.query0, col.dq[j], a.ndim, org);
  };
  // the score relative to `base`
  auto score = [&](int j, float s, float dist, float base) {
    if constexpr (BIAS) base = fmaf(-slope[j], dist, base);
    if constexpr (CAP)  // c2 tanh(x) = c2 - 2 c2 / (exp(2x) + 1)
      return fmaf(-2.f * a.c2, __builtin_amdgcn_rcpf(__builtin_amdgcn_exp2f(s * a.c1) + 1.f), base);
    else
      return fmaf(s, a.c1, base);
  };
  // o += V^T p for 32 keys
  auto gather = [&](int b, int u, const Frag(&p)[NC]) {
#pragma unroll
    for (int i = 0; i < DI; ++i) {
      const Frag f = tile_frag_t<T, DP>(tv[b], kt0 + u * 32, i, lane);
#pragma unroll
      for (int j = 0; j < NC; ++j) o[j][i] = AMfma<T>::run(f, p[j], o[j][i]);
    }
  };

  // the same of what rounding the probabilities s to p left
  auto gather_rest = [&](int b, int u, const f32x4(&s)[NC][NT], Frag(&p)[NC]) {
#pragma unroll
    for (int j = 0; j < NC; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        p[j][e] = static_cast<T>(s[j][2 * u + (e >> 2)][e & 3] - static_cast<float>(p[j][e]));
    gather(b, u, p);
  };

  // A whole tile against references that hold; false (and nothing changed) if one does not.
  auto fast = [&](int b) {
    f32x4 s[NC][NT];
    float base[NC], top[NC];
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      base[j] = CAP ? a.c2 - m[j] : -m[j];
      top[j] = -INFINITY;
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      f32x4 x[NC];
      product(b, n, x);
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        f32x4 dist = zero;
        if constexpr (BIAS) dist = dist_of(b, n, j, false);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[j][n][e] = score(j, x[j][e], dist[e], base[j]);
          top[j] = fmaxf(top[j], s[j][n][e]);
        }
      }
    }
    bool up = false;
#pragma unroll
    for (int j = 0; j < NC; ++j) up |= top[j] > Reach<T>::top;
    if (__any(up)) return false;
#pragma unroll
    for (int u = 0; u < NT / 2; ++u) {
      Frag p[NC];
#pragma unroll
      for (int j = 0; j < NC; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x = __builtin_amdgcn_exp2f(s[j][2 * u + (e >> 2)][e & 3]);
          l[j] += x;  // unrounded: the backward pass needs lse to fp32
          p[j][e] = static_cast<T>(x);
          if constexpr (TWO) s[j][2 * u + (e >> 2)][e & 3] = x;
        }
      gather(b, u, p);
      if constexpr (TWO) gather_rest(b, u, s, p);
    }
    return true;
  };

  auto slow = [&](int b, int left, bool far) {
    f32x4 s[NC][NT];
    float top[NC];
#pragma unroll
    for (int j = 0; j < NC; ++j) top[j] = -INFINITY;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (n * 16 >= left) {
#pragma unroll
        for (int j = 0; j < NC; ++j) s[j][n] = f32x4{-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        continue;
      }
      f32x4 x[NC];
      product(b, n, x);
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        f32x4 dist = zero;
        if constexpr (BIAS) dist = dist_of(b, n, j, far);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[j][n][e] = score(j, x[j][e], dist[e], CAP ? a.c2 : 0.f);
      }
    }
    if (left < NT * 16) {
      const int own = left - 4 * g;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int j = 0; j < NC; ++j) s[j][n][e] = n * 16 + e < own ? s[j][n][e] : -INFINITY;
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < NC; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) top[j] = fmaxf(top[j], s[j][n][e]);
    fold = true;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const float t = col_max(top[j]);
      const float mn = t > m[j] + Reach<T>::top ? t - Reach<T>::lift : m[j];  // t > -inf when there is no reference
      const float f = m[j] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m[j] - mn);
      m[j] = mn;
      l[j] *= f;
#pragma unroll
      for (int i = 0; i < DI; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][i][e] *= f;
      fold &= fabsf(mn) <= kFold;
    }
    fold = __all(fold);
#pragma unroll
    for (int u = 0; u < NT / 2; ++u) {
      if (u * 32 >= left) continue;
      Frag p[NC];
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const float ms = m[j] == -INFINITY ? 0.f : m[j];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x = __builtin_amdgcn_exp2f(s[j][2 * u + (e >> 2)][e & 3] - ms);
          l[j] += x;
          p[j][e] = static_cast<T>(x);
          if constexpr (TWO) s[j][2 * u + (e >> 2)][e & 3] = x;
        }
      }
      gather(b, u, p);
      if constexpr (TWO) gather_rest(b, u, s, p);
    }
  };

  // Results of head h.
  auto finish = [&]() {
#pragma unroll
    for (int j = 0; j < NC; ++j) l[j] = col_sum(l[j]);
    if constexpr (KS) {  // join the four waves: their shares of the sum relative to the largest maximum
      float* jm = reinterpret_cast<float*>(tk);  // [4][16] maxima, then sums
      float* jo = reinterpret_cast<float*>(tv);  // [4][16][DP]
      __syncthreads();
      if (g == 0) {
        jm[wave * 16 + lane] = m[0];
        jm[64 + wave * 16 + lane] = l[0];
      }
#pragma unroll
      for (int i = 0; i < DI; ++i)
        *reinterpret_cast<f32x4*>(jo + (wave * 16 + (lane & 15)) * DP + i * 16 + g * 4) = o[0][i];
      __syncthreads();
      float mw[4], mt = -INFINITY, lt = 0.f;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        mw[x] = jm[x * 16 + (lane & 15)];
        mt = fmaxf(mt, mw[x]);
      }
#pragma unroll
      for (int i = 0; i < DI; ++i) o[0][i] = zero;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float f = mw[x] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(mw[x] - mt);
        lt = fmaf(f, jm[64 + x * 16 + (lane & 15)], lt);
#pragma unroll
        for (int i = 0; i < DI; ++i) {
          const f32x4 y = *reinterpret_cast<const f32x4*>(jo + (x * 16 + (lane & 15)) * DP + i * 16 + g * 4);
#pragma unroll
          for (int e = 0; e < 4; ++e) o[0][i][e] = fmaf(f, y[e], o[0][i][e]);
        }
      }
      m[0] = mt;
      l[0] = lt;
      __syncthreads();  // the next head's tiles go where the shares were
      if (wave != 0) return;
    }
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      if (!col.live[j]) continue;
      const int d4 = static_cast<int>(late(g)) * 4;
      const int64_t query = col.query0 + late(col.dq[j]);
      const int head = h * a.grp + static_cast<int>(late(col.place[j]));
      const int64_t at = (static_cast<int64_t>(split) * a.nq + query) * a.hq + head;
      if (a.splits > 1) {
        if (g == 0) {
          a.part_ml[at * 2] = m[j];
          a.part_ml[at * 2 + 1] = l[j];
        }
#pragma unroll
        for (int i = 0; i < DI; ++i) *reinterpret_cast<f32x4*>(a.part + at * DP + i * 16 + d4) = o[j][i];
        continue;
      }
      const float inv = l[j] == 0.f ? 0.f : 1.f / l[j];
      T* op = static_cast<T*>(a.out) + query * a.o_stride + static_cast<int64_t>(head) * a.d;
#pragma unroll
      for (int i = 0; i < DI; ++i) {
        f32x4 y = o[j][i];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] *= inv;
        store4(op, i * 16 + d4, a.d, y);
      }
      if (g == 0) a.lse[at] = l[j] == 0.f ? -INFINITY : (m[j] + __builtin_amdgcn_logf(l[j])) * kLn2;
    }
  };

  if (n_keys <= 0) {
    for (; h < h_end; ++h) {
      begin();
      finish();
    }
    return;
  }
  keys.put(tk[0], tv[0], true, tc[0], far_rows[0], org, a.ndim);
  begin();
  for (int k0 = 0, b = 0;; b ^= 1) {
    const bool wrap = k0 + BN >= n_keys;
    const int hn = wrap ? h + 1 : h, kn = wrap ? 0 : k0 + BN;  // the next tile
    const bool more = hn < h_end;
    if (more) {
      if (MULTI && wrap) fetch_cols(hn);
      keys.fetch(a, hn, kn, !stay || hn == h0);
    }
    __syncthreads();
    if (col.busy) {
      const int left = n_keys - k0 - kt0;  // keys of this wave's part
      const bool far = BIAS && (far_cols || tile_far<BN>(far_rows[cb]));
      bool done = false;
      if (fold && !far && k0 + BN <= n_keys) done = fast(b);
      if (!done) slow(b, left, far);
    }
    if (wrap) finish();
    if (!more) break;
    h = hn;
    k0 = kn;
    if (MULTI && wrap) begin();
    cb = stay ? k0 / BN : b ^ 1;
    keys.put(tk[b ^ 1], tv[b ^ 1], !stay || h == h0, tc[cb], far_rows[cb], org, a.ndim);
  }
}

// Joins the splits of one row: weights exp2(m_s - max m) over all splits, then
// the weighted sums, a quarter of the splits per wave.
template <typename T, int DP>
__global__ __launch_bounds__(256) void k_attn_join(const AttnArgs a) {
  constexpr int MAXS = kAttnMaxSplits;
  __shared__ float wt[MAXS];
  __shared__ float red[8];
  __shared__ f32x4 acc[16][DP / 4];
  const int64_t row = blockIdx.x, rows = a.nq * a.hq;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  float mx = -INFINITY;
  for (int s = tid; s < a.splits; s += 256) {
    wt[s] = a.part_ml[(s * rows + row) * 2];
    mx = fmaxf(mx, wt[s]);
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor(mx, d));
  if (lane == 0) red[wave] = mx;
  __syncthreads();
  mx = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  float l = 0.f;
  for (int s = tid; s < a.splits; s += 256) {
    const float f = wt[s] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(wt[s] - mx);
    l += f * a.part_ml[(s * rows + row) * 2 + 1];
    wt[s] = f;
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) l += __shfl_xor(l, d);
  if (lane == 0) red[4 + wave] = l;
  __syncthreads();
  l = red[4] + red[5] + red[6] + red[7];
  // thread = (share of the splits, 4 elements)
  constexpr int Q = DP / 4, SH = 256 / Q < 16 ? 256 / Q : 16;
  const int d4 = tid % Q, sh = tid / Q;
  f32x4 y{0.f, 0.f, 0.f, 0.f};
  if (sh < SH) {
#pragma unroll 4
    for (int s = sh; s < a.splits; s += SH) {
      const float f = wt[s];
      const f32x4 v = *reinterpret_cast<const f32x4*>(a.part + (s * rows + row) * DP + d4 * 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = fmaf(f, v[e], y[e]);
    }
    acc[sh][d4] = y;
  }
  __syncthreads();
  if (sh != 0) return;
  for (int x = 1; x < SH; ++x)
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] += acc[x][d4][e];
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] *= inv;
  const int64_t query = row / a.hq;
  store4(static_cast<T*>(a.out) + query * a.o_stride + (row - query * a.hq) * a.d, d4 * 4, a.d, y);
  if (tid == 0) a.lse[row] = l == 0.f ? -INFINITY : (mx + __builtin_amdgcn_logf(l)) * kLn2;
}

// The same for few splits of many rows: a thread per row and 4 elements.
template <typename T, int DP>
__global__ __launch_bounds__(256) void k_attn_join_few(const AttnArgs a) {
  constexpr int Q = DP / 4;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, row = i / Q, rows = a.nq * a.hq;
  const int d0 = static_cast<int>(i % Q) * 4;
  if (row >= rows) return;
  float m[kAttnFewSplits], l[kAttnFewSplits], mx = -INFINITY;
#pragma unroll
  for (int s = 0; s < kAttnFewSplits; ++s) {
    m[s] = s < a.splits ? a.part_ml[(s * rows + row) * 2] : -INFINITY;
    l[s] = s < a.splits ? a.part_ml[(s * rows + row) * 2 + 1] : 0.f;
    mx = fmaxf(mx, m[s]);
  }
  f32x4 y{0.f, 0.f, 0.f, 0.f};
  float lt = 0.f;
#pragma unroll
  for (int s = 0; s < kAttnFewSplits; ++s) {
    if (s >= a.splits) continue;
    const float f = m[s] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m[s] - mx);
    lt = fmaf(f, l[s], lt);
    const f32x4 v = *reinterpret_cast<const f32x4*>(a.part + (s * rows + row) * DP + d0);
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = fmaf(f, v[e], y[e]);
  }
  const float inv = lt == 0.f ? 0.f : 1.f / lt;
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] *= inv;
  const int64_t query = row / a.hq;
  store4(static_cast<T*>(a.out) + query * a.o_stride + (row - query * a.hq) * a.d, d0, a.d, y);
  if (d0 == 0) a.lse[row] = lt == 0.f ? -INFINITY : (mx + __builtin_amdgcn_logf(lt)) * kLn2;
}

template <typename T, int DP, int NC, bool KS, bool TWO>
void run_fwd(const AttnArgs& a, bool cap, hipStream_t s) {
  const dim3 grid(attn_grid_x(a.tiles), ceil_div(a.hk, a.heads), a.splits);
  const bool bias = a.slopes != nullptr;
  if (cap && bias)
    k_attn_fwd<T, DP, NC, true, true, KS, TWO><<<grid, 256, 0, s>>>(a);
  else if (cap)
    k_attn_fwd<T, DP, NC, true, false, KS, TWO><<<grid, 256, 0, s>>>(a);
  else if (bias)
    k_attn_fwd<T, DP, NC, false, true, KS, TWO><<<grid, 256, 0, s>>>(a);
  else
    k_attn_fwd<T, DP, NC, false, false, KS, TWO><<<grid, 256, 0, s>>>(a);
}

template <typename T, int DP>
void run_fwd(AttnArgs& a, const AttnPlan& p, bool cap, hipStream_t s) {
  a.tiles = attn_tiles(a.nq, a.grp, p.bm, a.n_sets);
  a.splits = p.splits;
  a.heads = p.heads;
  if (DP <= 64 && p.share_keys)
    run_fwd<T, DP, 1, DP <= 64, true>(a, cap, s);  // (few rows always)
  else if (DP <= 64 && p.nc == 2)
    run_fwd<T, DP, DP <= 64 ? 2 : 1, false, false>(a, cap, s);
  else if (a.two)
    run_fwd<T, DP, 1, false, true>(a, cap, s);
  else
    run_fwd<T, DP, 1, false, false>(a, cap, s);
  const int64_t rows = a.nq * a.hq;
  if (a.splits > kAttnFewSplits)
    k_attn_join<T, DP><<<static_cast<unsigned>(rows), 256, 0, s>>>(a);
  else if (a.splits > 1)
    k_attn_join_few<T, DP><<<static_cast<unsigned>(ceil_div<int64_t>(rows * (DP / 4), 256)), 256, 0, s>>>(a);
}

template <typename T>
void run_fwd(AttnArgs& a, const AttnPlan& p, bool cap, hipStream_t s) {
  if (a.d <= 32)
    run_fwd<T, 32>(a, p, cap, s);
  else if (a.d <= 64)
    run_fwd<T, 64>(a, p, cap, s);
  else
    run_fwd<T, 128>(a, p, cap, s);
}

}  // namespace

// Rows of `heads` heads of d elements, `stride` apart, to or from rows of heads of d8
// elements, dense; the elements between d and d8 become zeros.
__global__ __launch_bounds__(256) void k_attn_repack(const uint16_t* __restrict__ src, int64_t src_stride, int src_d,
                                                     uint16_t* __restrict__ dst, int64_t dst_stride, int dst_d,
                                                     int64_t n, int heads) {
  const int64_t per = static_cast<int64_t>(heads) * dst_d, total = n * per;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total; i += int64_t{256} * gridDim.x) {
    const int64_t r = i / per;
    const int c = static_cast<int>(i - r * per), h = c / dst_d, e = c - h * dst_d;
    dst[r * dst_stride + c] = e < src_d ? src[r * src_stride + h * src_d + e] : uint16_t{0};
  }
}

hipError_t launch_attn_repack(const void* src, int64_t src_stride, int src_d, void* dst, int64_t dst_stride, int dst_d,
                              int64_t n, int heads, hipStream_t s) {
  const int64_t total = n * heads * dst_d, blocks = ceil_div<int64_t>(total, 256), most = 1 << 16;
  if (total == 0) return hipSuccess;
  k_attn_repack<<<static_cast<unsigned>(blocks < most ? blocks : most), 256, 0, s>>>(
      static_cast<const uint16_t*>(src), src_stride, src_d, static_cast<uint16_t*>(dst), dst_stride, dst_d, n, heads);
  return hipGetLastError();
}

hipError_t launch_attn_fwd(AttnArgs& a, const AttnPlan& p, ts_dtype dt, bool cap, hipStream_t s) {
  if (dt == TS_F16)
    run_fwd<_Float16>(a, p, cap, s);
  else
    run_fwd<__bf16>(a, p, cap, s);
  return hipGetLastError();
}

}  // namespace ts
