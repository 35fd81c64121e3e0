// Attention within packed sets, backward.  With p = exp2(z - lse) recomputed,
// dp = dout . v and delta = sum over the head width of dout * out:
//   dv = sum over rows of p dout
//   ds = p (dp - delta) (1 - tanh^2 where the scores are capped)
//   dq = scale * sum over keys of ds k,    dk = scale * sum over rows of ds q
// Two kernels, each walking the side its results sum over (attn.h): k_attn_dq
// owns query rows and streams keys, k_attn_dkv owns keys and streams the query
// rows of every head that shares them.  Scores are computed in both, so there
// are no atomics and the gradients are the same bits on every run.
//
// 1 - tanh^2 = 4 r (1 - r) with r = 1 / (exp(2x) + 1); the 4 is taken into the
// exponent of p (so dv is scaled back by 1/4 when it is written; in fp16, see kValueScale).
//
// Roundings to 16 bits.  p for dv and ds for dk once per term: both are 1.4 times as far
// from 64 bits as their last rounding alone.  dq would be 1.2 to 1.7 times as far off with
// ds in two parts (ds, and what its rounding left) and up to 5 times where few keys
// matter, because delta is formed from an out that is rounded already.  The sum of
// p (dp - delta) over a row is 0 in exact arithmetic: what it comes to, rho, is what delta
// was short of.  dk uses delta + rho.  For dq the sum of w k (ds = w (dp - delta)) is
// formed beside that of ds k, and rho times it taken off at the end (MEND; by k_attn_sum
// where the walk is split); where a row has at most 32 keys rho is known before ds is
// needed and taken off there.  Two parts and MEND: 1.0 (2400 windows of 32 channels,
// biased, 280 us, without MEND 237; of 16 channels 235 / 194; 1200 of 64 202 / 207).
//   - Two column blocks of 64 channels have registers for one part and MEND only: 1.45
//     (2 x 8192 rows 920 us, two parts without MEND 1016).
//   - Heads wider than 64 have them for two parts only: 1.05 to 1.35.
//   - Calls of few rows (attn_plan.h) have all of it, dk and dv of two parts too: 1.0.
//
// A key dropped by a score of -inf has an infinite element, and 0 times that is NaN in
// the product that forms dq; so is, in dk's, the query of a row whose scores are all
// -inf.  Looking for them in every tile would cost several per cent of both kernels, so
// the results are looked at instead: a column that has NaN in it is formed once more by
// its wave, pair by pair from memory (RowAgain), leaving out what an infinite element
// would add, and rows without a finite score.  That hides no NaN there should be: an
// infinite element makes its score infinite or NaN, so its score gradient 0 or NaN, and
// where one is NaN (or overflows fp16) the column is left as it is.
//
// As in the forward pass, a wave owns NC column blocks of 16 and a block takes
// a.heads key-value heads one after the other; delta enters as the accumulator
// that dp starts from.
//
// Bound by vector instructions, as the forward pass, and with two to four waves per
// SIMD by the latency of LDS reads and matrix results.  Measured (by the profiler, as
// every time beside a kernel here: twelve calls after a pause; long runs are 10 to 15 %
// faster): 2 x 8192 rows, 8 query and 4 key heads of 64, cap and bias: dq 930 us, dk and
// dv 1020 (NC 1: 1274 and 1325); 2400 windows of about 127 rows, 4 heads of 32, biased:
// dq 280, dk and dv 270.
#include "attn.h"

namespace ts {

namespace {

// p of one score and w, with ds = w dp.  s = q.k; dist the distance; base = -lse
// (plus c2 for a capped score) in units of log 2.
template <bool CAP, bool BIAS>
__device__ __forceinline__ void grad_score(const AttnArgs& a, float s, float base, float slope, float dist, float* p,
                                           float* w) {
  if constexpr (BIAS) base = fmaf(-slope, dist, base);
  if constexpr (CAP) {
    const float r = __builtin_amdgcn_rcpf(__builtin_amdgcn_exp2f(s * a.c1) + 1.f);
    *p = __builtin_amdgcn_exp2f(fmaf(-2.f * a.c2, r, base));
    *w = *p * fmaf(-r, r, r);
  } else {
    *p = *w = __builtin_amdgcn_exp2f(fmaf(s, a.c1, base));
  }
}

// What p is multiplied by on its way into dv's product (and dv divided by): fp16 has
// nothing below 2^-24, and over 100,000 keys p is about 2^-17, so it goes in times 2^15,
// the most that p = 1 leaves room for; no scale of dout could do that.  bf16 has fp32's
// range.  (A multiplication per score: 2 x 8192 fp16 rows, 8 / 4 heads of 64, dk and dv
// 1042 -> 1080 us, windows nothing; scaled and rounded by one mixed-precision
// instruction each 1085 to 1110.)
template <typename T>
constexpr float kValueScale = 1.f;
template <>
constexpr float kValueScale<_Float16> = 32768.f;

// What the exponent starts from: -lse in units of log 2, with c2 for a capped
// score and 2 more where p is to hold the factor 4; rows without a finite score
// get -inf, so their probabilities are 0.
template <bool CAP>
__device__ __forceinline__ float exp_base(const AttnArgs& a, float lse) {
  return lse == -INFINITY ? -INFINITY : fmaf(-lse, kLog2e, CAP ? a.c2 + 2.f : 0.f);
}

// The arguments of this kernel (its only parameter), read from where the launch put them:
// kept from the start of the kernel for RowAgain they would displace others.
__device__ __forceinline__ AttnArgs read_args() {
  typedef const __attribute__((address_space(4))) uint64_t* Words;
  uint64_t at = (uint64_t)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(at));
  const Words p = (Words)at;
  struct {
    uint64_t w[sizeof(AttnArgs) / 8];
  } copy;
  static_assert(sizeof(copy) == sizeof(AttnArgs), "whole words");
#pragma unroll
  for (unsigned i = 0; i < sizeof(AttnArgs) / 8; ++i) copy.w[i] = p[i];
  return __builtin_bit_cast(AttnArgs, copy);
}

// One query row or key formed again by a wave, 64 rows of the other side at a time:
// first a lane per row for the score gradients, then a lane per channel for the sums.
// Slow (2 x 8192 rows, 8 / 4 heads of 64, biased: 1.9 ms for the pass, 60 where a set of
// them has an infinite key), but it takes next to no registers of the walk's.
template <typename T, int DP, bool CAP, bool BIAS>
struct RowAgain {
  static constexpr int W = DP > 64 ? 2 : 1;  // channels of a lane: lane + 64 w
  const AttnArgs a = read_args();
  const int lane = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
  bool lost = false;  // a score gradient that no 16-bit number holds

  static __device__ __forceinline__ float dot8(const T* x, const T* y, float sum) {
    typedef T t8 __attribute__((ext_vector_type(8)));
    const t8 u = *reinterpret_cast<const t8*>(x), v = *reinterpret_cast<const t8*>(y);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = fmaf(static_cast<float>(u[e]), static_cast<float>(v[e]), sum);
    return sum;
  }
  __device__ __forceinline__ const T* row(const void* m, int64_t r, int64_t stride, int head) const {
    return static_cast<const T*>(m) + r * stride + static_cast<int64_t>(head) * a.d;
  }
  // the score gradient of a query row and a key; p as grad_score gives it
  __device__ __forceinline__ float pair(int64_t query, int head, int64_t key, int h, float lse, float delta, float* p) {
    const T *q = row(a.q, query, a.q_stride, head), *k = row(a.k, key, a.k_stride, h);
    const T *g = row(a.dout, query, a.o_stride, head), *v = row(a.v, key, a.v_stride, h);
    float s = 0.f, dp = -delta, dist = 0.f, slope = 0.f, w;
#pragma unroll 1
    for (int c = 0; c < a.d; c += 8) {
      s = dot8(q + c, k + c, s);
      dp = dot8(g + c, v + c, dp);
    }
    if constexpr (BIAS) {
      const f32x4 x = relative(load_place(a.qc, query, a.ndim), load_place(a.kc, key, a.ndim), a.ndim);
      dist = __builtin_amdgcn_sqrtf(x[3]);
      slope = a.slopes[head] * kLog2e;
    }
    grad_score<CAP, BIAS>(a, a.negate ? -s : s, exp_base<CAP>(a, lse), slope, dist, p, &w);
    const float ds = w * dp;
    lost |= !(fabsf(static_cast<float>(static_cast<T>(ds))) < INFINITY);
    return ds;
  }
  // sum += f times this lane's channels of a row; any: infinities and NaN too
  __device__ __forceinline__ void add(const T* x, float f, float (&sum)[W], bool any) const {
#pragma unroll
    for (int w = 0; w < W; ++w)
      if (lane + 64 * w < a.d) {
        const float v = static_cast<float>(x[lane + 64 * w]);
        sum[w] = fmaf(f, any || fabsf(v) < INFINITY ? v : 0.f, sum[w]);
      }
  }
  // f times the sums to a row of results, or to a split's part
  __device__ __forceinline__ void put(const float (&sum)[W], float f, T* out, float* part) const {
#pragma unroll
    for (int w = 0; w < W; ++w)
      if (lane + 64 * w < a.d) {
        if (a.splits > 1)
          part[lane + 64 * w] = sum[w] * f;
        else
          out[lane + 64 * w] = static_cast<T>(sum[w] * f);
      }
  }
  static __device__ __forceinline__ float of_lane(float x, int i) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), i));
  }
  // dq of packed row r of the set whose queries begin at q0 over n keys from `first`
  __device__ __forceinline__ void query(int64_t q0, uint32_t r, int h, int64_t first, int n, int split) {
    const int64_t q = q0 + r / static_cast<uint32_t>(a.grp);
    const int head = h * a.grp + static_cast<int>(r % static_cast<uint32_t>(a.grp));
    const float lse = a.lse[q * a.hq + head];
    const T *g = row(a.dout, q, a.o_stride, head), *o = row(a.o, q, a.o_stride, head);
    float delta = 0.f, sum[W] = {};
    if (a.splits == 1)
      delta = a.delta[q * a.hq + head];  // this wave's, corrected
    else
#pragma unroll 1
      for (int c = 0; c < a.d; c += 8) delta = dot8(g + c, o + c, delta);
#pragma unroll 1
    for (int k0 = 0; k0 < n; k0 += 64) {
      float p, ds = 0.f;
      if (k0 + lane < n) ds = pair(q, head, first + k0 + lane, h, lse, delta, &p);
      if (__any(lost)) return;
      const T* k = row(a.k, first + k0, a.k_stride, h);
      const int rows = n - k0 < 64 ? n - k0 : 64;
#pragma unroll 1
      for (int i = 0; i < rows; i += 4)
#pragma unroll
        for (int e = 0; e < 4; ++e)  // (past the last row ds is 0)
          add(k + (i + e < rows ? i + e : rows - 1) * a.k_stride, of_lane(ds, i + e), sum, false);
    }
    float* part = a.part + ((static_cast<int64_t>(split) * a.nq + q) * a.hq + head) * DP;
    put(sum, a.scale, const_cast<T*>(row(a.dq, q, a.q_stride, head)), part);
    if (a.mend && a.splits > 1)  // nothing to take off
#pragma unroll
      for (int w = 0; w < W; ++w)
        if (lane + 64 * w < a.d) part[a.splits * a.nq * a.hq * DP + lane + 64 * w] = 0.f;
  }
  // dk and dv of a key over n packed rows from `beg` of the set whose queries begin at q0
  __device__ __forceinline__ void key(int64_t k, int h, int64_t q0, uint32_t beg, int n, int split) {
    const uint32_t grp = a.grp;
    float dk[W] = {}, dv[W] = {};
#pragma unroll 1
    for (int r0 = 0; r0 < n; r0 += 64) {
      const uint32_t r = beg + r0 + lane;
      const int64_t q = q0 + r / grp;
      const int head = h * a.grp + static_cast<int>(r % grp);
      const float lse = r0 + lane < n ? a.lse[q * a.hq + head] : -INFINITY;
      float p = 0.f, ds = 0.f;
      if (lse != -INFINITY) ds = pair(q, head, k, h, lse, a.delta[q * a.hq + head], &p);
      if (__any(lost)) return;
#pragma unroll 1
      for (uint64_t seen = __ballot(lse != -INFINITY); seen != 0; seen &= seen - 1) {
        const int i = __ffsll(static_cast<unsigned long long>(seen)) - 1;
        const uint32_t ri = beg + r0 + i, qi = ri / grp;
        const int hi = h * a.grp + static_cast<int>(ri - qi * grp);
        add(row(a.q, q0 + qi, a.q_stride, hi), of_lane(ds, i), dk, false);
        add(row(a.dout, q0 + qi, a.o_stride, hi), of_lane(p, i), dv, true);
      }
    }
    const int64_t rows = a.nk * a.hk;
    float* part = a.part + (static_cast<int64_t>(split) * rows + k * a.hk + h) * DP;
    put(dk, a.scale, const_cast<T*>(row(a.dk, k, a.k_stride, h)), part);
    put(dv, CAP ? 0.25f : 1.f, const_cast<T*>(row(a.dv, k, a.v_stride, h)), part + a.splits * rows * DP);
  }
};

// The columns (of the 16 lanes share) in which some lane has a value that is not a number.
__device__ __forceinline__ uint64_t nan_columns(float sum, bool live) {
  uint64_t m = __ballot(live && sum != sum);
  m |= m >> 32;
  return (m | m >> 16) & 0xffffu;
}

template <typename T, int DP, int NC, bool CAP, bool BIAS, bool KS, bool MEND>
__global__ __launch_bounds__(256, attn_waves_dq(DP, NC, CAP, BIAS, KS, MEND)) void k_attn_dq(const AttnArgs a) {
  typedef typename AMfma<T>::frag Frag;
  constexpr int KB = DP / 32, DI = DP / 16;
  constexpr int BN = KS ? 128 : 64, NT = KS ? 2 : 4, BM = KS ? 16 : 64 * NC;
  constexpr int TB = BN * DP * 2;
  constexpr bool MULTI = NC == 1 && !KS && DP <= 64;
  constexpr bool REST = !(NC == 2 && DP == 64);  // ds in two parts
  static_assert(!KS || (NC == 1 && DP <= 64), "one column block of at most 64 channels when the waves share the keys");
  __shared__ __attribute__((aligned(16))) char tk[2][TB], tv[2][TB];
  __shared__ f32x4 tc[2][BIAS ? BN : 1];
  __shared__ uint32_t far_rows[2][2];

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
  // NC 2: not held as uniform, or both forms of a step are scheduled as one and their
  // registers do not fit (2 x 8192 rows, dk and dv: 1225 against 1020 us; dq, where the gain
  // was first seen, 1010 / 945 before it had MEND)
  const int n_keys = static_cast<int>(NC == 2 ? late(kend - kbeg) : kend - kbeg);
  const int h0 = blockIdx.y * a.heads;
  int h = h0;
  const int h_end = !MULTI ? h + 1 : h + a.heads < a.hk ? h + a.heads : a.hk;
  uint64_t again = 0;  // columns to form again: 16 bits for each head (at most 4) or column block

  const QueryCols<NC, KS> col(a, st, BM);
  uint32_t qoff[NC], ooff[NC];
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    qoff[j] = col.offset(j, a.q_stride, a.d);
    ooff[j] = col.offset(j, a.o_stride, a.d);
  }
  const int width = a.grp * a.d;  // a key-value head's part of a query row
  Place org{0, 0, 0};
  Place oraw, qraw[NC];
  if constexpr (BIAS) {
    oraw = load_place(a.qc, st.own0, a.ndim);
#pragma unroll
    for (int j = 0; j < NC; ++j) qraw[j] = load_place(a.qc, col.query0 + col.dq[j], a.ndim);
  }
  ColLoad<T, DP, NC> qld, gld, old;
  float next_slope[NC], next_lse[NC];
  auto fetch_cols = [&](int hn) {
    const int64_t q0 = col.query0 * a.q_stride + static_cast<int64_t>(hn) * width;
    const int64_t o0 = col.query0 * a.o_stride + static_cast<int64_t>(hn) * width;
    qld.fetch(static_cast<const T*>(a.q) + q0, col.bytes(a.q_stride, width), qoff, a.d);
    gld.fetch(static_cast<const T*>(a.dout) + o0, col.bytes(a.o_stride, width), ooff, a.d);
    old.fetch(static_cast<const T*>(a.o) + o0, col.bytes(a.o_stride, width), ooff, a.d);
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int head = hn * a.grp + static_cast<int>(col.place[j]);
      next_lse[j] = col.live[j] ? a.lse[(col.query0 + col.dq[j]) * a.hq + head] : -INFINITY;
      if constexpr (BIAS) next_slope[j] = a.slopes[head];
    }
  };
  fetch_cols(h);
  KeyTiles<T, DP, BN, BIAS> keys(a, st.st0 + kbeg, n_keys);
  if (n_keys > 0) keys.fetch(a, h, 0, true);

  float slope[NC], qb[NC], qn[NC];
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
  Frag qf[NC][KB], gf[NC][KB];
  f32x4 dq[NC][DI], pk[NC][MEND ? DI : 1];  // pk: sum of w k, ds = w dp
  float base[NC], delta[NC], rho[NC];
  const float rho_scale = CAP ? 0.25f : 1.f;
  const bool whole = a.splits == 1 && kend - kbeg <= 32;  // one step sees the whole row
  auto begin = [&]() {
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      float dl = 0.f;
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        qf[j][kb] = qld.frag_signed(j, kb, a.negate);
        gf[j][kb] = gld.frag(j, kb);
        const Frag of = old.frag(j, kb);
#pragma unroll
        for (int e = 0; e < 8; ++e) dl = fmaf(static_cast<float>(gf[j][kb][e]), static_cast<float>(of[e]), dl);
      }
      delta[j] = col_sum(dl);
      base[j] = exp_base<CAP>(a, next_lse[j]);
      if constexpr (BIAS) slope[j] = next_slope[j] * kLog2e;
      rho[j] = 0.f;
#pragma unroll
      for (int i = 0; i < DI; ++i) {
        dq[j][i] = zero;
        if constexpr (MEND) pk[j][i] = zero;
      }
    }
  };

  // 32 keys; part: keys may end inside them, distances may be long
  auto step = [&](auto part, int b, int u, int left, bool far) {
    constexpr bool PART = decltype(part)::v;
    f32x4 s[NC][2], dp[NC][2];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        const Frag fk = tile_frag<T, DP>(tk[b], kt0 + u * 32 + n * 16, kb, lane);
        const Frag fv = tile_frag<T, DP>(tv[b], kt0 + u * 32 + n * 16, kb, lane);
#pragma unroll
        for (int j = 0; j < NC; ++j) {
          s[j][n] = AMfma<T>::run(fk, qf[j][kb], kb == 0 ? zero : s[j][n]);
          dp[j][n] = AMfma<T>::run(fv, gf[j][kb], kb == 0 ? f32x4{-delta[j], -delta[j], -delta[j], -delta[j]} : dp[j][n]);
        }
      }
    Frag df[NC], dr[REST ? NC : 1], wf[MEND ? NC : 1];
    auto split = [&](int j, int e, float ds) {
      df[j][e] = static_cast<T>(ds);
      if constexpr (REST) dr[j][e] = static_cast<T>(ds - static_cast<float>(df[j][e]));
    };
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        f32x4 dist = zero;
        if constexpr (BIAS)
          dist = distances(tc[b], kt0 + u * 32 + n * 16, qn[j], qb[j], PART && far, lane, a.qc, col.query0,
                           col.dq[j], a.ndim, org);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float p, w;
          grad_score<CAP, BIAS>(a, s[j][n][e], base[j], BIAS ? slope[j] : 0.f, dist[e], &p, &w);
          if constexpr (PART)
            if (u * 32 + n * 16 + 4 * g + e >= left) p = w = 0.f;
          rho[j] = fmaf(p, dp[j][n][e], rho[j]);
          if constexpr (MEND) wf[j][n * 4 + e] = static_cast<T>(w);
          if constexpr (PART)
            s[j][n][e] = w;
          else
            split(j, n * 4 + e, w * dp[j][n][e]);
        }
      }
    if constexpr (PART) {
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const float more = whole ? col_sum(rho[j]) * rho_scale : 0.f;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) split(j, n * 4 + e, s[j][n][e] * (dp[j][n][e] - more));
      }
    }
#pragma unroll
    for (int i = 0; i < DI; ++i) {
      const Frag f = tile_frag_t<T, DP>(tk[b], kt0 + u * 32, i, lane);
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        dq[j][i] = AMfma<T>::run(f, df[j], dq[j][i]);
        if constexpr (REST) dq[j][i] = AMfma<T>::run(f, dr[j], dq[j][i]);
        if constexpr (MEND) pk[j][i] = AMfma<T>::run(f, wf[j], pk[j][i]);
      }
    }
  };

  // dq with what delta was short of taken off: known here if the walk is not split
  auto mend = [&](int j, float short_of) {
    if constexpr (MEND)
      if (a.splits == 1 && !whole)
#pragma unroll
        for (int i = 0; i < DI; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) dq[j][i][e] = fmaf(-short_of, pk[j][i][e], dq[j][i][e]);
  };

  auto finish = [&]() {
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      rho[j] = col_sum(rho[j]) * rho_scale;
      if constexpr (!KS) mend(j, rho[j]);
    }
    if constexpr (KS) {
      float* jo = reinterpret_cast<float*>(tv);  // [4][16][DP]
      float* jr = reinterpret_cast<float*>(tk);  // [4][16]
      __syncthreads();
      if (g == 0) jr[wave * 16 + lane] = rho[0];
      if constexpr (MEND) {
        __syncthreads();
        float all = 0.f;
#pragma unroll
        for (int x = 0; x < 4; ++x) all += jr[x * 16 + (lane & 15)];
        mend(0, all);
      }
#pragma unroll
      for (int i = 0; i < DI; ++i)
        *reinterpret_cast<f32x4*>(jo + (wave * 16 + (lane & 15)) * DP + i * 16 + g * 4) = dq[0][i];
      __syncthreads();
      if constexpr (MEND)
        if (a.splits > 1) {  // the same of pk, and so to both parts
          float* jp = reinterpret_cast<float*>(tk) + 64;
#pragma unroll
          for (int i = 0; i < DI; ++i)
            *reinterpret_cast<f32x4*>(jp + (wave * 16 + (lane & 15)) * DP + i * 16 + g * 4) = pk[0][i];
          __syncthreads();
#pragma unroll
          for (int i = 0; i < DI; ++i) {
            pk[0][i] = zero;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const f32x4 y = *reinterpret_cast<const f32x4*>(jp + (x * 16 + (lane & 15)) * DP + i * 16 + g * 4);
#pragma unroll
              for (int e = 0; e < 4; ++e) pk[0][i][e] += y[e];
            }
          }
        }
      if (wave != 0) return;
#pragma unroll
      for (int x = 1; x < 4; ++x) rho[0] += jr[x * 16 + (lane & 15)];
#pragma unroll
      for (int x = 1; x < 4; ++x)
#pragma unroll
        for (int i = 0; i < DI; ++i) {
          const f32x4 y = *reinterpret_cast<const f32x4*>(jo + (x * 16 + (lane & 15)) * DP + i * 16 + g * 4);
#pragma unroll
          for (int e = 0; e < 4; ++e) dq[0][i][e] += y[e];
        }
    }
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < DI; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sum += dq[j][i][e];
          if constexpr (MEND) sum += pk[j][i][e];
        }
      again |= nan_columns(sum, col.live[j] && base[j] != -INFINITY) << (16 * (MULTI ? h - h0 : j));
    }
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      if (!col.live[j]) continue;
      const int64_t query = col.query0 + late(col.dq[j]);
      const int head = h * a.grp + static_cast<int>(late(col.place[j]));
      const bool none = base[j] == -INFINITY;  // no finite score
      if (none) rho[j] = delta[j] = 0.f;  // (its dout may be anything)
      if (g == 0) {
        // rho: what delta was short of
        if (split == 0) a.delta[query * a.hq + head] = a.splits == 1 ? delta[j] + rho[j] : delta[j];
        if (a.splits > 1) a.part_ml[(static_cast<int64_t>(split) * a.nq + query) * a.hq + head] = rho[j];
      }
      T* dst = static_cast<T*>(a.dq) + query * a.q_stride + static_cast<int64_t>(head) * a.d;
      float* part = a.part + ((static_cast<int64_t>(split) * a.nq + query) * a.hq + head) * DP;
#pragma unroll
      for (int i = 0; i < DI; ++i) {
        f32x4 y = dq[j][i];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = none ? 0.f : y[e] * a.scale;
        if constexpr (MEND)
          if (a.splits > 1) {
            f32x4 x = pk[j][i];
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = none ? 0.f : x[e] * a.scale;
            *reinterpret_cast<f32x4*>(part + a.splits * a.nq * a.hq * DP + i * 16 + g * 4) = x;
          }
        if (a.splits > 1)
          *reinterpret_cast<f32x4*>(part + i * 16 + g * 4) = y;
        else
          store4(dst, i * 16 + g * 4, a.d, y);
      }
    }
  };

  if (n_keys <= 0) {
    for (;;) {
      begin();
      finish();
      if (!MULTI || ++h >= h_end) return;
      fetch_cols(h);
    }
  }
  keys.put(tk[0], tv[0], true, tc[0], far_rows[0], org, a.ndim);
  begin();
  for (int k0 = 0, b = 0;; b ^= 1) {
    const bool wrap = k0 + BN >= n_keys;
    const int hn = wrap ? h + 1 : h, kn = wrap ? 0 : k0 + BN;
    const bool more = hn < h_end;
    if (more) {
      if (MULTI && wrap) fetch_cols(hn);
      keys.fetch(a, hn, kn, true);
    }
    __syncthreads();
    if (col.busy) {
      const int left = n_keys - k0 - kt0;
      const bool far = BIAS && (far_cols || tile_far<BN>(far_rows[b]));
#pragma unroll
      for (int u = 0; u < NT / 2; ++u) {
        if (u * 32 >= left) continue;
        if (u * 32 + 32 <= left && !far && !whole)
          step(Flag<false>{}, b, u, left, false);
        else
          step(Flag<true>{}, b, u, left, far);
      }
    }
    if (wrap) finish();
    if (!more) break;
    h = hn;
    k0 = kn;
    if (MULTI && wrap) begin();
    keys.put(tk[b ^ 1], tv[b ^ 1], true, tc[b ^ 1], far_rows[b ^ 1], org, a.ndim);
  }
  if (again == 0) return;
  __threadfence();  // the columns as first written
  for (; again != 0; again &= again - 1) {
    const int bit = __ffsll(static_cast<unsigned long long>(again)) - 1, c = bit & 15, u = bit >> 4;
    const uint32_t r = static_cast<uint32_t>(st.row0) + (KS ? 0 : (MULTI ? 0 : u * 4) + wave) * 16 + c;
    RowAgain<T, DP, CAP, BIAS>().query(st.own0, r, MULTI ? h0 + u : h0, keys.first, n_keys, split);
  }
}

template <typename T, int DP, int NC, bool CAP, bool BIAS>
__global__ __launch_bounds__(256, attn_waves_dkv(DP, NC, BIAS)) void k_attn_dkv(const AttnArgs a) {
  typedef typename AMfma<T>::frag Frag;
  constexpr int KB = DP / 32, DI = DP / 16;
  constexpr int BN = DP == 128 ? 32 : 64;  // 32 rows where the accumulators leave room for no more
  constexpr int BM = 64 * NC;
  constexpr int TB = BN * DP * 2;
  constexpr bool MULTI = NC == 1 && DP <= 64;
  __shared__ __attribute__((aligned(16))) char tq[2][TB], tg[2][TB];
  __shared__ f32x4 tc[2][BIAS ? BN : 1];                                  // coordinates of the row
  __shared__ __attribute__((aligned(16))) float tsl[2][BIAS ? BN : 4];    // its slope,
  __shared__ __attribute__((aligned(16))) float tl[2][BN], td[2][BN];     // exponent base and -delta
  __shared__ uint32_t far_rows[2][2];

  const int64_t slot = block_tile();
  const int split = blockIdx.z;
  SetTile st;
  if (!find_tile<BM>(a.ks, a.nk, 1, a.qs, a.nq, a.n_sets, slot, a.tiles, &st)) return;
  int64_t rbeg, rend;
  split_range(st.st_len * a.grp, BN, a.splits, split, &rbeg, &rend);

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), g = lane >> 4;
  const int n_rows = static_cast<int>(NC == 2 ? late(rend - rbeg) : rend - rbeg);  // see k_attn_dq
  const int h0 = blockIdx.y * a.heads;
  int h = h0;
  const int h_end = !MULTI ? h + 1 : h + a.heads < a.hk ? h + a.heads : a.hk;
  uint64_t again = 0;  // see k_attn_dq
  const int width = a.grp * a.d;

  // columns: keys
  const int64_t key0 = st.own0 + st.row0;
  const uint32_t cols = st.rows - st.row0 < BM ? static_cast<uint32_t>(st.rows - st.row0) : BM;
  bool live[NC];
  uint32_t ck[NC], koff[NC], voff[NC];
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const uint32_t c = (j * 4 + wave) * 16 + (lane & 15);
    live[j] = c < cols;
    ck[j] = live[j] ? c : 0;
    koff[j] = live[j] ? c * static_cast<uint32_t>(a.k_stride) * 2u : kOutside;
    voff[j] = live[j] ? c * static_cast<uint32_t>(a.v_stride) * 2u : kOutside;
  }
  const bool busy = static_cast<uint32_t>(wave * 16) < cols;
  Place org{0, 0, 0};
  Place oraw, kraw[NC];
  if constexpr (BIAS) {
    oraw = load_place(a.kc, st.own0, a.ndim);
#pragma unroll
    for (int j = 0; j < NC; ++j) kraw[j] = load_place(a.kc, key0 + ck[j], a.ndim);
  }
  ColLoad<T, DP, NC> kld, vld;
  auto fetch_cols = [&](int hn) {
    kld.fetch(static_cast<const T*>(a.k) + key0 * a.k_stride + static_cast<int64_t>(hn) * a.d,
              ((cols - 1) * static_cast<uint32_t>(a.k_stride) + a.d) * 2u, koff, a.d);
    vld.fetch(static_cast<const T*>(a.v) + key0 * a.v_stride + static_cast<int64_t>(hn) * a.d,
              ((cols - 1) * static_cast<uint32_t>(a.v_stride) + a.d) * 2u, voff, a.d);
  };
  fetch_cols(h);

  // packed row r of this walk: its query, relative to the set, and its place among the heads that share a key head
  auto at_row = [&](uint32_t r, uint32_t* query, uint32_t* place) {
    const uint32_t x = static_cast<uint32_t>(rbeg) + r;
    *query = a.grp == 1 ? x : x / static_cast<uint32_t>(a.grp);
    *place = x - *query * a.grp;
  };
  TileLoad<T, DP, BN> ld;
  TileCoords<BN> lc;
  lc.c = Place{0, 0, 0};
  float rl = 0.f, rd = 0.f, rs = 0.f;
  // Tile rows of this thread: 2^16 times the query from the tile's first one, and
  // place.  The same in every tile where the heads that share a key head divide BN,
  // else formed anew.
  uint32_t trow[ld.CT];
  auto place_rows = [&](int r0, uint32_t q0) {
#pragma unroll
    for (int i = 0; i < ld.CT; ++i) {
      uint32_t q, p;
      at_row(r0 + ld.row(i), &q, &p);
      trow[i] = (q - q0) << 16 | p;
    }
  };
  const bool even = BN % a.grp == 0;
  {
    uint32_t q0, p0;
    at_row(0, &q0, &p0);
    place_rows(0, q0);
  }
  auto off = [&](int i, int64_t stride) {
    // NC 2: taken apart where it is used, two registers fewer through the walk
    const uint32_t r = NC == 2 ? late(trow[i]) : trow[i];
    return ((r >> 16) * static_cast<uint32_t>(stride) + (r & 0xffffu) * a.d) * 2u;
  };
  auto off_q = [&](int i) { return off(i, a.q_stride); };
  auto off_g = [&](int i) { return off(i, a.o_stride); };
  auto fetch = [&](int hn, int r0) {
    uint32_t q0, p0, q1, p1;
    at_row(r0, &q0, &p0);
    if (!even) place_rows(r0, q0);
    const int64_t query0 = st.st0 + q0;
    at_row(n_rows - r0 < BN ? n_rows - 1 : r0 + BN - 1, &q1, &p1);  // the last row: offsets rise with the row
    const uint32_t end = (p1 + 1) * a.d;
    ld.fetch(static_cast<const T*>(a.q) + query0 * a.q_stride + static_cast<int64_t>(hn) * width,
             ((q1 - q0) * static_cast<uint32_t>(a.q_stride) + end) * 2u, off_q,
             static_cast<const T*>(a.dout) + query0 * a.o_stride + static_cast<int64_t>(hn) * width,
             ((q1 - q0) * static_cast<uint32_t>(a.o_stride) + end) * 2u, off_g, a.d);
    if (tid < BN && r0 + tid < n_rows) {
      uint32_t q, p;
      at_row(r0 + tid, &q, &p);
      const int64_t query = st.st0 + q;
      const int head = hn * a.grp + static_cast<int>(p);
      rl = a.lse[query * a.hq + head];
      rd = a.delta[query * a.hq + head];
      if constexpr (BIAS) {
        lc.c = load_place(a.qc, query, a.ndim);
        rs = a.slopes[head];
      }
    }
  };
  auto put = [&](int b) {
    ld.put(tq[b], tg[b]);
    if (tid < BN) {
      tl[b][tid] = exp_base<CAP>(a, rl);
      td[b][tid] = -rd;
      if constexpr (BIAS) tsl[b][tid] = rs * kLog2e;
    }
    if constexpr (BIAS) lc.put(tc[b], far_rows[b], org, a.ndim);
  };
  if (n_rows > 0) fetch(h, 0);

  float kb_[NC], kn[NC];
  bool far_cols = false;
  if constexpr (BIAS) {
    org = uniform_origin(oraw);
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const f32x4 c = relative(kraw[j], org, a.ndim);
      kb_[j] = col_term(c, g);
      kn[j] = c[3];
      far_cols |= __any(c[3] > kNearNorm) != 0;
    }
  }

  const f32x4 zero{0.f, 0.f, 0.f, 0.f};
  Frag kf[NC][KB], vf[NC][KB];
  f32x4 dk[NC][DI], dv[NC][DI];
  auto begin = [&]() {
#pragma unroll
    for (int j = 0; j < NC; ++j) {
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        kf[j][kb] = kld.frag_signed(j, kb, a.negate);
        vf[j][kb] = vld.frag(j, kb);
      }
#pragma unroll
      for (int i = 0; i < DI; ++i) dk[j][i] = dv[j][i] = zero;
    }
  };

  // 32 rows; part: rows may end inside them, distances may be long
  auto step = [&](auto part, int b, int u, int left, bool far) {
    constexpr bool PART = decltype(part)::v;
    f32x4 s[NC][2], dp[NC][2];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const f32x4 nd = *reinterpret_cast<const f32x4*>(&td[b][u * 32 + n * 16 + 4 * g]);
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        const Frag fq = tile_frag<T, DP>(tq[b], u * 32 + n * 16, kb, lane);
        const Frag fg = tile_frag<T, DP>(tg[b], u * 32 + n * 16, kb, lane);
#pragma unroll
        for (int j = 0; j < NC; ++j) {
          s[j][n] = AMfma<T>::run(fq, kf[j][kb], kb == 0 ? zero : s[j][n]);
          dp[j][n] = AMfma<T>::run(fg, vf[j][kb], kb == 0 ? nd : dp[j][n]);
        }
      }
    }
    constexpr float PS = kValueScale<T> == 1.f ? 1.f : kValueScale<T> * (CAP ? 0.25f : 1.f);
    Frag pf[NC], df[NC];
    auto gather = [&]() {
#pragma unroll
      for (int i = 0; i < DI; ++i) {
        const Frag fg = tile_frag_t<T, DP>(tg[b], u * 32, i, lane);
        const Frag fq = tile_frag_t<T, DP>(tq[b], u * 32, i, lane);
#pragma unroll
        for (int j = 0; j < NC; ++j) {
          dv[j][i] = AMfma<T>::run(fg, pf[j], dv[j][i]);
          dk[j][i] = AMfma<T>::run(fq, df[j], dk[j][i]);
        }
      }
    };
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int r = u * 32 + n * 16 + 4 * g;
      const f32x4 base = *reinterpret_cast<const f32x4*>(&tl[b][r]);
      f32x4 slope = zero;
      if constexpr (BIAS) slope = *reinterpret_cast<const f32x4*>(&tsl[b][r]);
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        f32x4 dist = zero;
        if constexpr (BIAS)
          dist = distances(tc[b], u * 32 + n * 16, kn[j], kb_[j], PART && far, lane, a.kc, key0, ck[j], a.ndim, org);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float p, w;
          grad_score<CAP, BIAS>(a, s[j][n][e], base[e], slope[e], dist[e], &p, &w);
          float ds = w * dp[j][n][e];
          if constexpr (PART)
            if (r + e >= left) p = ds = 0.f;  // a zero row times an infinite key is NaN
          if constexpr (PS != 1.f) p *= PS;
          pf[j][n * 4 + e] = static_cast<T>(p);
          df[j][n * 4 + e] = static_cast<T>(ds);
          if constexpr (PART && NC == 1) {
            s[j][n][e] = p;
            dp[j][n][e] = ds;
          }
        }
      }
    }
    gather();
    if constexpr (PART && NC == 1)
      if (a.two) {  // and what the roundings left
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            pf[0][n * 4 + e] = static_cast<T>(s[0][n][e] - static_cast<float>(pf[0][n * 4 + e]));
            df[0][n * 4 + e] = static_cast<T>(dp[0][n][e] - static_cast<float>(df[0][n * 4 + e]));
          }
        gather();
      }
  };

  const float vs = kValueScale<T> == 1.f ? (CAP ? 0.25f : 1.f) : 1.f / kValueScale<T>;
  auto finish = [&]() {
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < DI; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) sum += dk[j][i][e] + dv[j][i][e];
      again |= nan_columns(sum, live[j]) << (16 * (MULTI ? h - h0 : j));
    }
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      if (!live[j]) continue;
      const int64_t key = key0 + late(ck[j]), rows = a.nk * a.hk;
      T* kd = static_cast<T*>(a.dk) + key * a.k_stride + static_cast<int64_t>(h) * a.d;
      T* vd = static_cast<T*>(a.dv) + key * a.v_stride + static_cast<int64_t>(h) * a.d;
      float* part = a.part + (static_cast<int64_t>(split) * rows + key * a.hk + h) * DP;
#pragma unroll
      for (int i = 0; i < DI; ++i) {
        f32x4 y = dk[j][i], x = dv[j][i];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          y[e] *= a.scale;
          x[e] *= vs;
        }
        if (a.splits > 1) {
          *reinterpret_cast<f32x4*>(part + i * 16 + g * 4) = y;
          *reinterpret_cast<f32x4*>(part + a.splits * rows * DP + i * 16 + g * 4) = x;
        } else {
          store4(kd, i * 16 + g * 4, a.d, y);
          store4(vd, i * 16 + g * 4, a.d, x);
        }
      }
    }
  };

  if (n_rows <= 0) {
    begin();
    for (; h < h_end; ++h) finish();
    return;
  }
  put(0);
  begin();
  for (int r0 = 0, b = 0;; b ^= 1) {
    const bool wrap = r0 + BN >= n_rows;
    const int hn = wrap ? h + 1 : h, rn = wrap ? 0 : r0 + BN;
    const bool more = hn < h_end;
    if (more) {
      if (MULTI && wrap) fetch_cols(hn);
      fetch(hn, rn);
    }
    __syncthreads();
    if (busy) {
      const int left = n_rows - r0;
      const bool far = BIAS && (far_cols || tile_far<BN>(far_rows[b]));
#pragma unroll
      for (int u = 0; u < BN / 32; ++u) {
        if (u * 32 >= left) continue;
        if (u * 32 + 32 <= left && !far && !(NC == 1 && a.two))
          step(Flag<false>{}, b, u, left, false);
        else
          step(Flag<true>{}, b, u, left, far);
      }
    }
    if (wrap) finish();
    if (!more) break;
    h = hn;
    r0 = rn;
    if (MULTI && wrap) begin();
    put(b ^ 1);
  }
  if (again == 0) return;
  __threadfence();
  for (; again != 0; again &= again - 1) {
    const int bit = __ffsll(static_cast<unsigned long long>(again)) - 1, c = bit & 15, u = bit >> 4;
    RowAgain<T, DP, CAP, BIAS>().key(key0 + ((MULTI ? 0 : u * 4) + wave) * 16 + c, MULTI ? h0 + u : h0, st.st0,
                                     static_cast<uint32_t>(rbeg), n_rows, split);
  }
}

// out row r (row / heads, head row % heads) = sum over the splits, in order; the same
// of what the splits found delta short of
template <typename T, int DP>
__global__ __launch_bounds__(256) void k_attn_sum(const float* __restrict__ part, int64_t rows, int splits, int heads,
                                                  int d, T* out, int64_t stride, const float* __restrict__ short_of,
                                                  float* delta, const float* __restrict__ pk) {
  constexpr int Q = DP / 4;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, row = i / Q;
  const int d0 = static_cast<int>(i % Q) * 4;
  if (row >= rows) return;
  f32x4 y{0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < splits; ++s) {
    const f32x4 v = *reinterpret_cast<const f32x4*>(part + (s * rows + row) * DP + d0);
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] += v[e];
  }
  if (pk) {  // dq: delta was short of this sum
    f32x4 x{0.f, 0.f, 0.f, 0.f};
    float rho = 0.f;
    for (int s = 0; s < splits; ++s) {
      const f32x4 v = *reinterpret_cast<const f32x4*>(pk + (s * rows + row) * DP + d0);
      rho += short_of[s * rows + row];
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] += v[e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = fmaf(-rho, x[e], y[e]);
  }
  const int64_t n = row / heads;
  store4(out + n * stride + (row - n * heads) * d, d0, d, y);
  if (delta && d0 == 0) {
    float x = delta[row];
    for (int s = 0; s < splits; ++s) x += short_of[s * rows + row];
    delta[row] = x;
  }
}

// The same for many splits, a block per row: the splits in shares, joined in order.
template <typename T, int DP>
__global__ __launch_bounds__(256) void k_attn_sum_many(const float* __restrict__ part, int64_t rows, int splits,
                                                       int heads, int d, T* out, int64_t stride,
                                                       const float* __restrict__ short_of, float* delta,
                                                       const float* __restrict__ pk) {
  constexpr int Q = DP / 4, SH = 256 / Q;
  __shared__ f32x4 acc[2][SH][Q];
  __shared__ float red[4];
  const int64_t row = blockIdx.x;
  const int d4 = threadIdx.x % Q, sh = threadIdx.x / Q;
  f32x4 y{0.f, 0.f, 0.f, 0.f}, x = y;
  float rho = 0.f;
#pragma unroll 4
  for (int s = sh; s < splits; s += SH) {
    const int64_t at = (s * rows + row) * DP + d4 * 4;
    y += *reinterpret_cast<const f32x4*>(part + at);
    if (pk) x += *reinterpret_cast<const f32x4*>(pk + at);
  }
  if (delta)
    for (int s = threadIdx.x; s < splits; s += 256) rho += short_of[s * rows + row];
#pragma unroll
  for (int i = 32; i > 0; i >>= 1) rho += __shfl_xor(rho, i);
  if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = rho;
  acc[0][sh][d4] = y;
  acc[1][sh][d4] = x;
  __syncthreads();
  if (sh != 0) return;
  rho = (red[0] + red[1]) + (red[2] + red[3]);
#pragma unroll
  for (int i = 1; i < SH; ++i) {
    y += acc[0][i][d4];
    x += acc[1][i][d4];
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = fmaf(-rho, x[e], y[e]);
  const int64_t n = row / heads;
  store4(out + n * stride + (row - n * heads) * d, d4 * 4, d, y);
  if (delta && d4 == 0) delta[row] += rho;
}

template <typename T, int DP>
void run_sum(const float* part, int64_t rows, int splits, int heads, const AttnArgs& a, void* out, int64_t stride,
             float* delta, const float* pk, hipStream_t s) {
  if (splits > kAttnFewSplits)  // (few rows then)
    k_attn_sum_many<T, DP><<<static_cast<unsigned>(rows), 256, 0, s>>>(part, rows, splits, heads, a.d, static_cast<T*>(out),
                                                                       stride, a.part_ml, delta, pk);
  else
    k_attn_sum<T, DP><<<static_cast<unsigned>(ceil_div<int64_t>(rows * (DP / 4), 256)), 256, 0, s>>>(
      part, rows, splits, heads, a.d, static_cast<T*>(out), stride, a.part_ml, delta, pk);
}

template <typename T, int DP, int NC, bool CAP, bool BIAS, bool KS, bool MEND>
void run_dq(const AttnArgs& a, hipStream_t s) {
  k_attn_dq<T, DP, NC, CAP, BIAS, KS, MEND>
      <<<dim3(attn_grid_x(a.tiles), ceil_div(a.hk, a.heads), a.splits), 256, 0, s>>>(a);
}
template <typename T, int DP, int NC, bool CAP, bool BIAS>
void run_dkv(const AttnArgs& a, hipStream_t s) {
  k_attn_dkv<T, DP, NC, CAP, BIAS><<<dim3(attn_grid_x(a.tiles), ceil_div(a.hk, a.heads), a.splits), 256, 0, s>>>(a);
}

template <typename T, int DP, bool CAP, bool BIAS>
void run_bwd(AttnArgs& a, const AttnPlan& pq, const AttnPlan& pk, hipStream_t s) {
  if (a.nq > 0 || a.flags) {  // k_attn_dq checks the starts
    a.tiles = attn_tiles(a.nq, a.grp, pq.bm, a.n_sets);
    a.splits = pq.splits;
    a.heads = pq.heads;
    if constexpr (DP == 128) {
      if (a.mend)
        run_dq<T, DP, 1, CAP, BIAS, false, true>(a, s);
      else
        run_dq<T, DP, 1, CAP, BIAS, false, false>(a, s);
    } else if (pq.share_keys) {
      run_dq<T, DP, 1, CAP, BIAS, true, true>(a, s);
    } else if (pq.nc == 2) {
      run_dq<T, DP, 2, CAP, BIAS, false, true>(a, s);
    } else {
      run_dq<T, DP, 1, CAP, BIAS, false, true>(a, s);
    }
    if (a.splits > 1)
      run_sum<T, DP>(a.part, a.nq * a.hq, a.splits, a.hq, a, a.dq, a.q_stride, a.delta,
                     a.mend ? a.part + a.splits * a.nq * a.hq * DP : nullptr, s);
  }
  if (a.nk == 0) return;
  a.tiles = attn_tiles(a.nk, 1, pk.bm, a.n_sets);
  a.splits = pk.splits;
  a.heads = pk.heads;
  if (DP <= 64 && pk.nc == 2)
    run_dkv<T, DP, DP <= 64 ? 2 : 1, CAP, BIAS>(a, s);
  else
    run_dkv<T, DP, 1, CAP, BIAS>(a, s);
  if (a.splits > 1) {
    const int64_t rows = a.nk * a.hk;
    run_sum<T, DP>(a.part, rows, a.splits, a.hk, a, a.dk, a.k_stride, nullptr, nullptr, s);
    run_sum<T, DP>(a.part + a.splits * rows * DP, rows, a.splits, a.hk, a, a.dv, a.v_stride, nullptr, nullptr, s);
  }
}

template <typename T, int DP>
void run_bwd(AttnArgs& a, const AttnPlan& pq, const AttnPlan& pk, bool cap, hipStream_t s) {
  const bool bias = a.slopes != nullptr;
  if (cap && bias)
    run_bwd<T, DP, true, true>(a, pq, pk, s);
  else if (cap)
    run_bwd<T, DP, true, false>(a, pq, pk, s);
  else if (bias)
    run_bwd<T, DP, false, true>(a, pq, pk, s);
  else
    run_bwd<T, DP, false, false>(a, pq, pk, s);
}

template <typename T>
void run_bwd(AttnArgs& a, const AttnPlan& pq, const AttnPlan& pk, bool cap, hipStream_t s) {
  if (a.d <= 32)
    run_bwd<T, 32>(a, pq, pk, cap, s);
  else if (a.d <= 64)
    run_bwd<T, 64>(a, pq, pk, cap, s);
  else
    run_bwd<T, 128>(a, pq, pk, cap, s);
}

}  // namespace

hipError_t launch_attn_bwd(AttnArgs& a, const AttnPlan& pq, const AttnPlan& pk, ts_dtype dt, bool cap, hipStream_t s) {
  if (dt == TS_F16)
    run_bwd<_Float16>(a, pq, pk, cap, s);
  else
    run_bwd<__bf16>(a, pq, pk, cap, s);
  return hipGetLastError();
}

}  // namespace ts
