// Attention within packed sets, forward: one walk over the keys with a running
// maximum and sum (see attn.h for the operand layout).
//
// Scores are kept in units of log 2, so probabilities are exp2(z - m).  The
// maximum m that the accumulators refer to is raised only when a score passes
// it by more than 8: probabilities stay below 2^8, which loses nothing in the
// 16-bit operand (rounding is relative) nor in the fp32 sums, and most tiles
// leave the accumulators as they are.  Rows without a finite score give zeros
// and lse = -inf.
#include "attn.h"

namespace ts {

namespace {

constexpr float kSlack = 8.f;

// KS (few query rows): all four waves of a block own the same 16 columns and
// share out the keys of each tile, 32 rows each; their results are joined in
// LDS.  Otherwise each wave owns NC column blocks of its own.
template <typename T, int DP, int NC, bool CAP, bool BIAS, bool KS>
__global__ __launch_bounds__(256, KS && DP == 128 ? 1 : 2) void k_attn_fwd(const AttnArgs a) {
  typedef typename AMfma<T>::frag Frag;
  constexpr int KB = DP / 32, DI = DP / 16, CH = DP / 8;
  constexpr int BN = KS ? 128 : 64;  // keys per tile
  constexpr int NT = KS ? 2 : 4;     // 16-key steps of a wave per tile
  constexpr int BM = KS ? 16 * NC : 64 * NC;
  constexpr int CT = BN * CH / 256;  // chunks a thread stages per matrix
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

  // columns
  int64_t row[NC];  // query * hq + head
  bool live[NC];
  Frag qf[NC][KB];
  f32x4 qc[NC];  // coordinates and the slope in units of log 2
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
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
      qf[j][kb] = __builtin_bit_cast(Frag, live[j] ? load8(qp, kb * 32 + g * 8, a.d, a.vec_in) : u32x4{0u, 0u, 0u, 0u});
    if constexpr (BIAS) qc[j] = load_coord(a.qc, query, a.ndim, a.slopes[head] * kLog2e);
  }

  u32x4 rk[CT], rv[CT];
  f32x4 rc{0.f, 0.f, 0.f, 0.f};
  auto fetch = [&](int k0) {
#pragma unroll
    for (int i = 0; i < CT; ++i) {
      const int c = i * 256 + tid, r = k0 + c / CH, d0 = (c % CH) * 8;
      const bool ok = r < n_keys;  // rows past the end become zeros: 0 * NaN of another set's row would be NaN
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

  f32x4 o[NC][DI];
  float m[NC], l[NC];
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    m[j] = -INFINITY;
    l[j] = 0.f;
#pragma unroll
    for (int i = 0; i < DI; ++i) o[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  if (n_keys > 0) {
    fetch(0);
    put(0);
  }
  for (int k0 = 0, b = 0; k0 < n_keys; k0 += BN, b ^= 1) {
    const bool more = k0 + BN < n_keys;
    if (more) fetch(k0 + BN);
    __syncthreads();
    f32x4 s[NC][NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        const Frag f = tile_frag<T, DP>(tk[b], kt0 + n * 16, kb, lane);
#pragma unroll
        for (int j = 0; j < NC; ++j)
          s[j][n] = AMfma<T>::run(f, qf[j][kb], kb == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : s[j][n]);
      }
    }
    float top[NC];
#pragma unroll
    for (int j = 0; j < NC; ++j) top[j] = -INFINITY;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int kr = kt0 + n * 16 + 4 * g + e;
        f32x4 kc;
        if constexpr (BIAS) kc = tc[b][kr];
#pragma unroll
        for (int j = 0; j < NC; ++j) {
          float z = s[j][n][e];
          if constexpr (CAP) {
            // c2 tanh(x) = c2 - 2 c2 / (exp(2x) + 1)
            const float r = __builtin_amdgcn_rcpf(__builtin_amdgcn_exp2f(z * a.c1) + 1.f);
            z = fmaf(-2.f * a.c2, r, a.c2);
          } else {
            z *= a.c1;
          }
          if constexpr (BIAS) z = fmaf(-qc[j][3], distance(qc[j], kc), z);
          if (!more) z = k0 + kr < n_keys ? z : -INFINITY;
          s[j][n][e] = z;
          top[j] = fmaxf(top[j], z);
        }
      }
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      top[j] = col_max(top[j]);
      const bool raise = top[j] > m[j] + kSlack;
      if (__any(raise)) {
        const float mn = raise ? top[j] : m[j];
        const float f = raise ? __builtin_amdgcn_exp2f(m[j] - mn) : 1.f;
        m[j] = mn;
        l[j] *= f;
#pragma unroll
        for (int i = 0; i < DI; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[j][i][e] *= f;
      }
    }
    Frag p[NC][NT / 2];
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const float ms = m[j] == -INFINITY ? 0.f : m[j];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = __builtin_amdgcn_exp2f(s[j][n][e] - ms);
          l[j] += x;
          p[j][n / 2][(n & 1) * 4 + e] = static_cast<T>(x);
        }
    }
#pragma unroll
    for (int u = 0; u < NT / 2; ++u)
#pragma unroll
      for (int i = 0; i < DI; ++i) {
        const Frag f = tile_frag_t<T, DP>(tv[b], kt0 + u * 32, i, lane);
#pragma unroll
        for (int j = 0; j < NC; ++j) o[j][i] = AMfma<T>::run(f, p[j][u], o[j][i]);
      }
    if (more) put(b ^ 1);
  }

#pragma unroll
  for (int j = 0; j < NC; ++j) l[j] = col_sum(l[j]);

  if constexpr (KS) {  // join the four waves: their shares of the sum relative to the largest maximum
    float* jm = reinterpret_cast<float*>(tk);          // [4][16] maxima, then sums
    float* jo = reinterpret_cast<float*>(tv);          // [4][16][DP]
    __syncthreads();
    if (g == 0) {
      jm[wave * 16 + lane] = m[0];
      jm[64 + wave * 16 + lane] = l[0];
    }
#pragma unroll
    for (int i = 0; i < DI; ++i)
      *reinterpret_cast<f32x4*>(jo + (wave * 16 + (lane & 15)) * DP + i * 16 + g * 4) = o[0][i];
    __syncthreads();
    if (wave != 0) return;
    float mw[4], mt = -INFINITY, lt = 0.f;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      mw[x] = jm[x * 16 + (lane & 15)];
      mt = fmaxf(mt, mw[x]);
    }
#pragma unroll
    for (int i = 0; i < DI; ++i) o[0][i] = f32x4{0.f, 0.f, 0.f, 0.f};
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
  }

#pragma unroll
  for (int j = 0; j < NC; ++j) {
    if (!live[j]) continue;
    if (a.splits > 1) {
      const int64_t at = static_cast<int64_t>(w.split) * a.nq * a.hq + row[j];
      if (g == 0) {
        a.part_ml[at * 2] = m[j];
        a.part_ml[at * 2 + 1] = l[j];
      }
      if (n_keys > 0)
#pragma unroll
        for (int i = 0; i < DI; ++i) *reinterpret_cast<f32x4*>(a.part + at * DP + i * 16 + g * 4) = o[j][i];
      continue;
    }
    const float inv = l[j] == 0.f ? 0.f : 1.f / l[j];
    const int64_t query = row[j] / a.hq;
    T* op = static_cast<T*>(a.out) + query * a.o_stride + (row[j] - query * a.hq) * a.d;
#pragma unroll
    for (int i = 0; i < DI; ++i) {
      f32x4 y = o[j][i];
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] *= inv;
      store4(op, i * 16 + g * 4, a.d, a.vec_out, y);
    }
    if (g == 0) a.lse[row[j]] = l[j] == 0.f ? -INFINITY : (m[j] + __builtin_amdgcn_logf(l[j])) * kLn2;
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
    for (int s = sh; s < a.splits; s += SH) {
      const float f = wt[s];
      if (f == 0.f) continue;  // a split without keys wrote no sums
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
  store4(static_cast<T*>(a.out) + query * a.o_stride + (row - query * a.hq) * a.d, d4 * 4, a.d, a.vec_out, y);
  if (tid == 0) a.lse[row] = l == 0.f ? -INFINITY : (mx + __builtin_amdgcn_logf(l)) * kLn2;
}

template <typename T, int DP, int NC, bool KS>
void run_fwd(const AttnArgs& a, bool cap, unsigned grid, hipStream_t s) {
  const bool bias = a.slopes != nullptr;
  if (cap && bias)
    k_attn_fwd<T, DP, NC, true, true, KS><<<grid, 256, 0, s>>>(a);
  else if (cap)
    k_attn_fwd<T, DP, NC, true, false, KS><<<grid, 256, 0, s>>>(a);
  else if (bias)
    k_attn_fwd<T, DP, NC, false, true, KS><<<grid, 256, 0, s>>>(a);
  else
    k_attn_fwd<T, DP, NC, false, false, KS><<<grid, 256, 0, s>>>(a);
}

template <typename T, int DP>
void run_fwd(AttnArgs& a, const AttnPlan& p, bool cap, hipStream_t s) {
  a.tiles = attn_tiles(a.nq, a.grp, p.bm, a.n_sets);
  a.splits = p.splits;
  const unsigned grid = static_cast<unsigned>(a.tiles * a.hk * a.splits);
  bool done = false;
  if constexpr (DP <= 64) {  // two column blocks per wave only where their accumulators fit the registers
    if (p.nc == 2) {
      run_fwd<T, DP, 2, false>(a, cap, grid, s);
      done = true;
    }
  }
  if (!done && p.share_keys)
    run_fwd<T, DP, 1, true>(a, cap, grid, s);
  else if (!done)
    run_fwd<T, DP, 1, false>(a, cap, grid, s);
  if (a.splits > 1) k_attn_join<T, DP><<<static_cast<unsigned>(a.nq * a.hq), 256, 0, s>>>(a);
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

hipError_t launch_attn_fwd(AttnArgs& a, const AttnPlan& p, ts_dtype dt, bool cap, hipStream_t s) {
  if (dt == TS_F16)
    run_fwd<_Float16>(a, p, cap, s);
  else
    run_fwd<__bf16>(a, p, cap, s);
  return hipGetLastError();
}

}  // namespace ts
