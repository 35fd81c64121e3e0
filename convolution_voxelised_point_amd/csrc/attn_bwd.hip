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
// exponent of p (so dv is scaled back by 1/4 when it is written).
#include "attn.h"

namespace ts {

namespace {

// p and ds of one score: s = q.k, the column's or row's terms as described
template <bool CAP, bool BIAS>
__device__ __forceinline__ void grad_score(const AttnArgs& a, float s, float dp, float lse2, float delta, float slope,
                                           const f32x4& ca, const f32x4& cb, float* p, float* ds) {
  float z, r = 0.f;
  if constexpr (CAP) {
    r = __builtin_amdgcn_rcpf(__builtin_amdgcn_exp2f(s * a.c1) + 1.f);
    z = fmaf(-2.f * a.c2, r, a.c2 - lse2);
  } else {
    z = fmaf(s, a.c1, -lse2);
  }
  if constexpr (BIAS) z = fmaf(-slope, distance(ca, cb), z);
  *p = __builtin_amdgcn_exp2f(z);
  *ds = *p * (dp - delta);
  if constexpr (CAP) *ds *= fmaf(-r, r, r);
}

// lse in units of log 2, less 2 where p is to hold the factor 4; rows without
// a finite score get +inf, so their probabilities are 0.
template <bool CAP>
__device__ __forceinline__ float lse_term(float lse) {
  return lse == -INFINITY ? INFINITY : fmaf(lse, kLog2e, CAP ? -2.f : 0.f);
}

template <typename T, int DP, int NC, bool CAP, bool BIAS, bool KS>
__global__ __launch_bounds__(256, KS && DP == 128 ? 1 : 2) void k_attn_dq(const AttnArgs a) {
  typedef typename AMfma<T>::frag Frag;
  constexpr int KB = DP / 32, DI = DP / 16, CH = DP / 8;
  constexpr int BN = KS ? 128 : 64, NT = KS ? 2 : 4, BM = KS ? 16 * NC : 64 * NC;
  constexpr int CT = BN * CH / 256;
  static_assert(!KS || NC == 1, "one column block when the waves share the keys");
  __shared__ __attribute__((aligned(16))) char tk[2][BN * DP * 2], tv[2][BN * DP * 2];
  __shared__ f32x4 tc[2][BIAS ? BN : 1];

  const Where w = where(a);
  if (a.flags && w.kvh == 0 && w.split == 0 && threadIdx.x == 0) {
    check_starts(a.qs, a.nq, a.n_sets, w.tile, a.flags);
    if (a.ks != a.qs) check_starts(a.ks, a.nk, a.n_sets, w.tile, a.flags);
  }
  SetTile st;
  if (!find_tile<BM>(a.qs, a.nq, a.grp, a.ks, a.nk, a.n_sets, w.tile, &st)) return;
  int64_t kbeg, kend;
  split_range(st.st_len, BN, a.splits, w.split, &kbeg, &kend);

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, g = lane >> 4;
  const int kt0 = KS ? wave * 32 : 0;
  const T* kp = static_cast<const T*>(a.k) + (st.st0 + kbeg) * a.k_stride + static_cast<int64_t>(w.kvh) * a.d;
  const T* vp = static_cast<const T*>(a.v) + (st.st0 + kbeg) * a.v_stride + static_cast<int64_t>(w.kvh) * a.d;
  const int n_keys = static_cast<int>(kend - kbeg);

  int64_t row[NC];
  bool live[NC];
  Frag qf[NC][KB], gf[NC][KB];
  f32x4 qc[NC];
  float lse2[NC], delta[NC];
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const int64_t r = st.row0 + ((KS ? 0 : wave * NC) + j) * 16 + (lane & 15);
    live[j] = r < st.rows;
    const uint32_t rr = live[j] ? static_cast<uint32_t>(r) : 0;
    const uint32_t qi = a.grp == 1 ? rr : rr / static_cast<uint32_t>(a.grp);
    const int64_t query = st.own0 + qi;
    const int head = w.kvh * a.grp + static_cast<int>(rr - qi * a.grp);
    row[j] = query * a.hq + head;
    const T* qp = static_cast<const T*>(a.q) + query * a.q_stride + static_cast<int64_t>(head) * a.d;
    const int64_t oo = query * a.o_stride + static_cast<int64_t>(head) * a.d;
    const T *gp = static_cast<const T*>(a.dout) + oo, *op = static_cast<const T*>(a.o) + oo;
    float dl = 0.f;
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      const u32x4 none{0u, 0u, 0u, 0u};
      const int d0 = kb * 32 + g * 8;
      qf[j][kb] = __builtin_bit_cast(Frag, live[j] ? load8(qp, d0, a.d, a.vec_in) : none);
      gf[j][kb] = __builtin_bit_cast(Frag, live[j] ? load8(gp, d0, a.d, a.vec_in) : none);
      const Frag of = __builtin_bit_cast(Frag, live[j] ? load8(op, d0, a.d, a.vec_in) : none);
#pragma unroll
      for (int e = 0; e < 8; ++e) dl = fmaf(static_cast<float>(gf[j][kb][e]), static_cast<float>(of[e]), dl);
    }
    delta[j] = col_sum(dl);
    lse2[j] = lse_term<CAP>(live[j] ? a.lse[row[j]] : -INFINITY);
    if (live[j] && g == 0 && w.split == 0 && (!KS || wave == 0)) a.delta[row[j]] = delta[j];
    if constexpr (BIAS) qc[j] = load_coord(a.qc, query, a.ndim, a.slopes[head] * kLog2e);
  }

  u32x4 rk[CT], rv[CT];
  f32x4 rc{0.f, 0.f, 0.f, 0.f};
  auto fetch = [&](int k0) {
#pragma unroll
    for (int i = 0; i < CT; ++i) {
      const int c = i * 256 + tid, r = k0 + c / CH, d0 = (c % CH) * 8;
      const bool ok = r < n_keys;
      rk[i] = ok ? load8(kp + static_cast<int64_t>(r) * a.k_stride, d0, a.d, a.vec_in) : u32x4{0u, 0u, 0u, 0u};
      rv[i] = ok ? load8(vp + static_cast<int64_t>(r) * a.v_stride, d0, a.d, a.vec_in) : u32x4{0u, 0u, 0u, 0u};
    }
    if constexpr (BIAS)
      if (tid < BN && k0 + tid < n_keys) rc = load_coord(a.kc, st.st0 + kbeg + k0 + tid, a.ndim, 0.f);
  };
  auto put = [&](int b) {
#pragma unroll
    for (int i = 0; i < CT; ++i) {
      const int c = i * 256 + tid, at = tile_at<DP>(c / CH, c % CH);
      *reinterpret_cast<u32x4*>(tk[b] + at) = rk[i];
      *reinterpret_cast<u32x4*>(tv[b] + at) = rv[i];
    }
    if constexpr (BIAS)
      if (tid < BN) tc[b][tid] = rc;
  };

  f32x4 dq[NC][DI];
#pragma unroll
  for (int j = 0; j < NC; ++j)
#pragma unroll
    for (int i = 0; i < DI; ++i) dq[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};

  if (n_keys > 0) {
    fetch(0);
    put(0);
  }
  for (int k0 = 0, b = 0; k0 < n_keys; k0 += BN, b ^= 1) {
    const bool more = k0 + BN < n_keys;
    if (more) fetch(k0 + BN);
    __syncthreads();
#pragma unroll
    for (int u = 0; u < NT / 2; ++u) {
      f32x4 s[NC][2], dp[NC][2];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
          const Frag fk = tile_frag<T, DP>(tk[b], kt0 + u * 32 + n * 16, kb, lane);
          const Frag fv = tile_frag<T, DP>(tv[b], kt0 + u * 32 + n * 16, kb, lane);
#pragma unroll
          for (int j = 0; j < NC; ++j) {
            s[j][n] = AMfma<T>::run(fk, qf[j][kb], kb == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : s[j][n]);
            dp[j][n] = AMfma<T>::run(fv, gf[j][kb], kb == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : dp[j][n]);
          }
        }
      Frag df[NC];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int kr = kt0 + u * 32 + n * 16 + 4 * g + e;
          f32x4 kc{0.f, 0.f, 0.f, 0.f};
          if constexpr (BIAS) kc = tc[b][kr];
#pragma unroll
          for (int j = 0; j < NC; ++j) {
            float p, ds;
            grad_score<CAP, BIAS>(a, s[j][n][e], dp[j][n][e], lse2[j], delta[j], BIAS ? qc[j][3] : 0.f, qc[j], kc, &p, &ds);
            if (!more) ds = k0 + kr < n_keys ? ds : 0.f;
            df[j][n * 4 + e] = static_cast<T>(ds);
          }
        }
#pragma unroll
      for (int i = 0; i < DI; ++i) {
        const Frag f = tile_frag_t<T, DP>(tk[b], kt0 + u * 32, i, lane);
#pragma unroll
        for (int j = 0; j < NC; ++j) dq[j][i] = AMfma<T>::run(f, df[j], dq[j][i]);
      }
    }
    if (more) put(b ^ 1);
  }

  if constexpr (KS) {
    float* jo = reinterpret_cast<float*>(tv);  // [4][16][DP]
    __syncthreads();
#pragma unroll
    for (int i = 0; i < DI; ++i)
      *reinterpret_cast<f32x4*>(jo + (wave * 16 + (lane & 15)) * DP + i * 16 + g * 4) = dq[0][i];
    __syncthreads();
    if (wave != 0) return;
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
    if (!live[j]) continue;
    const int64_t query = row[j] / a.hq;
    T* dst = static_cast<T*>(a.dq) + query * a.q_stride + (row[j] - query * a.hq) * a.d;
    float* part = a.part + (static_cast<int64_t>(w.split) * a.nq * a.hq + row[j]) * DP;
#pragma unroll
    for (int i = 0; i < DI; ++i) {
      f32x4 y = dq[j][i];
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] *= a.scale;
      if (a.splits > 1)
        *reinterpret_cast<f32x4*>(part + i * 16 + g * 4) = y;
      else
        store4(dst, i * 16 + g * 4, a.d, a.vec_out, y);
    }
  }
}

template <typename T, int DP, int NC, bool CAP, bool BIAS>
__global__ __launch_bounds__(256, 2) void k_attn_dkv(const AttnArgs a) {
  typedef typename AMfma<T>::frag Frag;
  constexpr int KB = DP / 32, DI = DP / 16, CH = DP / 8;
  constexpr int BN = 64, BM = 64 * NC;
  constexpr int CT = BN * CH / 256;
  __shared__ __attribute__((aligned(16))) char tq[2][BN * DP * 2], tg[2][BN * DP * 2];
  __shared__ f32x4 tc[2][BIAS ? BN : 1];  // coordinates and slope of the row
  __shared__ float tl[2][BN], td[2][BN];  // its lse term and delta

  const Where w = where(a);
  SetTile st;
  if (!find_tile<BM>(a.ks, a.nk, 1, a.qs, a.nq, a.n_sets, w.tile, &st)) return;
  int64_t rbeg, rend;
  split_range(st.st_len * a.grp, BN, a.splits, w.split, &rbeg, &rend);

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, g = lane >> 4;
  const uint32_t n_rows = static_cast<uint32_t>(rend - rbeg);

  int64_t key[NC];
  bool live[NC];
  Frag kf[NC][KB], vf[NC][KB];
  f32x4 kc[NC];
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const int64_t r = st.row0 + (wave * NC + j) * 16 + (lane & 15);
    live[j] = r < st.rows;
    key[j] = st.own0 + (live[j] ? r : 0);
    const T* kp = static_cast<const T*>(a.k) + key[j] * a.k_stride + static_cast<int64_t>(w.kvh) * a.d;
    const T* vp = static_cast<const T*>(a.v) + key[j] * a.v_stride + static_cast<int64_t>(w.kvh) * a.d;
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      kf[j][kb] = __builtin_bit_cast(Frag, live[j] ? load8(kp, kb * 32 + g * 8, a.d, a.vec_in) : u32x4{0u, 0u, 0u, 0u});
      vf[j][kb] = __builtin_bit_cast(Frag, live[j] ? load8(vp, kb * 32 + g * 8, a.d, a.vec_in) : u32x4{0u, 0u, 0u, 0u});
    }
    if constexpr (BIAS) kc[j] = load_coord(a.kc, key[j], a.ndim, 0.f);
  }

  u32x4 rq[CT], rg[CT];
  f32x4 rc{0.f, 0.f, 0.f, 0.f};
  float rl = 0.f, rd = 0.f;
  // packed row r of this walk: its query and head
  auto at_row = [&](uint32_t r, int64_t* query, int* head) {
    const uint32_t x = static_cast<uint32_t>(rbeg) + r;
    const uint32_t qi = a.grp == 1 ? x : x / static_cast<uint32_t>(a.grp);
    *query = st.st0 + qi;
    *head = w.kvh * a.grp + static_cast<int>(x - qi * a.grp);
  };
  auto fetch = [&](uint32_t r0) {
#pragma unroll
    for (int i = 0; i < CT; ++i) {
      const uint32_t c = i * 256 + tid, r = r0 + c / CH;
      const int d0 = (c % CH) * 8;
      rq[i] = rg[i] = u32x4{0u, 0u, 0u, 0u};
      if (r < n_rows) {
        int64_t query;
        int head;
        at_row(r, &query, &head);
        rq[i] = load8(static_cast<const T*>(a.q) + query * a.q_stride + static_cast<int64_t>(head) * a.d, d0, a.d, a.vec_in);
        rg[i] = load8(static_cast<const T*>(a.dout) + query * a.o_stride + static_cast<int64_t>(head) * a.d, d0, a.d,
                      a.vec_in);
      }
    }
    if (tid < BN) {
      if (r0 + tid < n_rows) {
        int64_t query;
        int head;
        at_row(r0 + tid, &query, &head);
        rl = lse_term<CAP>(a.lse[query * a.hq + head]);
        rd = a.delta[query * a.hq + head];
        if constexpr (BIAS) rc = load_coord(a.qc, query, a.ndim, a.slopes[head] * kLog2e);
      }
    }
  };
  auto put = [&](int b) {
#pragma unroll
    for (int i = 0; i < CT; ++i) {
      const int c = i * 256 + tid, at = tile_at<DP>(c / CH, c % CH);
      *reinterpret_cast<u32x4*>(tq[b] + at) = rq[i];
      *reinterpret_cast<u32x4*>(tg[b] + at) = rg[i];
    }
    if (tid < BN) {
      tl[b][tid] = rl;
      td[b][tid] = rd;
      if constexpr (BIAS) tc[b][tid] = rc;
    }
  };

  f32x4 dk[NC][DI], dv[NC][DI];
#pragma unroll
  for (int j = 0; j < NC; ++j)
#pragma unroll
    for (int i = 0; i < DI; ++i) dk[j][i] = dv[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};

  if (n_rows > 0) {
    fetch(0);
    put(0);
  }
  for (uint32_t r0 = 0, b = 0; r0 < n_rows; r0 += BN, b ^= 1) {
    const bool more = r0 + BN < n_rows;
    if (more) fetch(r0 + BN);
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      f32x4 s[NC][2], dp[NC][2];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
          const Frag fq = tile_frag<T, DP>(tq[b], u * 32 + n * 16, kb, lane);
          const Frag fg = tile_frag<T, DP>(tg[b], u * 32 + n * 16, kb, lane);
#pragma unroll
          for (int j = 0; j < NC; ++j) {
            s[j][n] = AMfma<T>::run(fq, kf[j][kb], kb == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : s[j][n]);
            dp[j][n] = AMfma<T>::run(fg, vf[j][kb], kb == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : dp[j][n]);
          }
        }
      Frag pf[NC], df[NC];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int r = u * 32 + n * 16 + 4 * g;
        const f32x4 lse2 = *reinterpret_cast<const f32x4*>(&tl[b][r]);
        const f32x4 delta = *reinterpret_cast<const f32x4*>(&td[b][r]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          f32x4 qc{0.f, 0.f, 0.f, 0.f};
          if constexpr (BIAS) qc = tc[b][r + e];
#pragma unroll
          for (int j = 0; j < NC; ++j) {
            float p, ds;
            grad_score<CAP, BIAS>(a, s[j][n][e], dp[j][n][e], lse2[e], delta[e], qc[3], kc[j], qc, &p, &ds);
            if (!more && r0 + r + e >= n_rows) p = ds = 0.f;  // a zero row times an infinite key is NaN
            pf[j][n * 4 + e] = static_cast<T>(p);
            df[j][n * 4 + e] = static_cast<T>(ds);
          }
        }
      }
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
    }
    if (more) put(b ^ 1);
  }

  const float vs = CAP ? 0.25f : 1.f;
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    if (!live[j]) continue;
    T* kd = static_cast<T*>(a.dk) + key[j] * a.k_stride + static_cast<int64_t>(w.kvh) * a.d;
    T* vd = static_cast<T*>(a.dv) + key[j] * a.v_stride + static_cast<int64_t>(w.kvh) * a.d;
    const int64_t rows = a.nk * a.hk;
    float* part = a.part + (static_cast<int64_t>(w.split) * rows + key[j] * a.hk + w.kvh) * DP;
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
        store4(kd, i * 16 + g * 4, a.d, a.vec_out, y);
        store4(vd, i * 16 + g * 4, a.d, a.vec_out, x);
      }
    }
  }
}

// out row r (row / heads, head row % heads) = sum over the splits, in order
template <typename T, int DP>
__global__ __launch_bounds__(256) void k_attn_sum(const float* __restrict__ part, int64_t rows, int splits, int heads,
                                                  int d, T* out, int64_t stride, bool vec) {
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
  const int64_t n = row / heads;
  store4(out + n * stride + (row - n * heads) * d, d0, d, vec, y);
}

template <typename T, int DP>
void run_sum(const float* part, int64_t rows, int splits, int heads, const AttnArgs& a, void* out, int64_t stride,
             hipStream_t s) {
  k_attn_sum<T, DP><<<static_cast<unsigned>(ceil_div<int64_t>(rows * (DP / 4), 256)), 256, 0, s>>>(
      part, rows, splits, heads, a.d, static_cast<T*>(out), stride, a.vec_out);
}

// Two column blocks per wave only where their accumulators fit the registers.
template <typename T, int DP, bool CAP, bool BIAS>
void run_dq(const AttnArgs& a, const AttnPlan& p, unsigned grid, hipStream_t s) {
  if constexpr (DP <= 64) {
    if (p.nc == 2) {
      k_attn_dq<T, DP, 2, CAP, BIAS, false><<<grid, 256, 0, s>>>(a);
      return;
    }
  }
  k_attn_dq<T, DP, 1, CAP, BIAS, false><<<grid, 256, 0, s>>>(a);
}

template <typename T, int DP, bool CAP, bool BIAS>
void run_bwd(AttnArgs& a, const AttnPlan& pq, const AttnPlan& pk, hipStream_t s) {
  a.tiles = attn_tiles(a.nq, a.grp, pq.bm, a.n_sets);
  a.splits = pq.splits;
  unsigned grid = static_cast<unsigned>(a.tiles * a.hk * a.splits);
  if (a.nq > 0) {
    if (pq.share_keys)
      k_attn_dq<T, DP, 1, CAP, BIAS, true><<<grid, 256, 0, s>>>(a);
    else
      run_dq<T, DP, CAP, BIAS>(a, pq, grid, s);
    if (a.splits > 1) run_sum<T, DP>(a.part, a.nq * a.hq, a.splits, a.hq, a, a.dq, a.q_stride, s);
  }
  if (a.nk == 0) return;
  a.tiles = attn_tiles(a.nk, 1, pk.bm, a.n_sets);
  a.splits = pk.splits;
  grid = static_cast<unsigned>(a.tiles * a.hk * a.splits);
  if constexpr (DP <= 32) {
    if (pk.nc == 2) {
      k_attn_dkv<T, DP, 2, CAP, BIAS><<<grid, 256, 0, s>>>(a);
    } else {
      k_attn_dkv<T, DP, 1, CAP, BIAS><<<grid, 256, 0, s>>>(a);
    }
  } else {
    k_attn_dkv<T, DP, 1, CAP, BIAS><<<grid, 256, 0, s>>>(a);
  }
  if (a.splits > 1) {
    const int64_t rows = a.nk * a.hk;
    run_sum<T, DP>(a.part, rows, a.splits, a.hk, a, a.dk, a.k_stride, s);
    run_sum<T, DP>(a.part + a.splits * rows * DP, rows, a.splits, a.hk, a, a.dv, a.v_stride, s);
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
