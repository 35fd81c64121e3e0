// C entry points of the voxel-transformer operators: host-side validation,
// workspace layout and the choice of how a walk is cut up.
#include <cmath>

#include "act8.h"
#include "attn.h"

using namespace ts;

namespace {

#define TS_TRY(expr)                        \
  do {                                      \
    if ((expr) != hipSuccess) return TS_ERR_HIP; \
  } while (0)

constexpr int64_t kMaxRows = (int64_t{1} << 31) - 1;
constexpr float kMaxCap = 1024.f;
constexpr int64_t kMaxStride = int64_t{1} << 23;

bool at16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool at8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7) == 0; }

float cap_factor(const ts_attn* at) { return 2.f * kLog2e * fabsf(at->scale) / at->cap; }

ts_status check_attn(const ts_attn* at) {
  if (!at) return TS_ERR_INVALID_ARG;
  if (at->dtype != TS_F32 && at->dtype != TS_F16 && at->dtype != TS_BF16) return TS_ERR_INVALID_ARG;
  if (at->hq < 1 || at->hk < 1 || at->d < 1 || at->hq % at->hk != 0) return TS_ERR_INVALID_ARG;
  if (at->nq < 0 || at->nk < 0 || at->n_sets < 0) return TS_ERR_INVALID_ARG;
  if (!std::isfinite(at->scale) || !std::isfinite(at->cap) || at->cap < 0.f) return TS_ERR_INVALID_ARG;
  if (at->cap > 0.f && !std::isfinite(cap_factor(at))) return TS_ERR_INVALID_ARG;
  // c2 - 2 c2 / (exp + 1) keeps a score to about 2 c2 / 2^24: 2e-4 at the largest cap
  if (at->dtype == TS_F32 || at->d > 128 || at->cap > kMaxCap) return TS_ERR_UNSUPPORTED;
  if (at->hq > 65535 || at->nq > kMaxRows / at->hq || at->nk > kMaxRows / at->hk || at->n_sets > kMaxRows)
    return TS_ERR_UNSUPPORTED;
  const int64_t qw = static_cast<int64_t>(at->hq) * at->d, kw = static_cast<int64_t>(at->hk) * at->d;
  // a tile's row offsets are 32-bit
  if (at->q_stride > kMaxStride || at->k_stride > kMaxStride || at->v_stride > kMaxStride || at->o_stride > kMaxStride)
    return TS_ERR_UNSUPPORTED;
  if (at->q_stride < qw || at->o_stride < qw || at->k_stride < kw || at->v_stride < kw) return TS_ERR_INVALID_ARG;
  if (!at->q_starts || (!at->k_starts && at->nk != at->nq)) return TS_ERR_INVALID_ARG;
  if (at->slopes) {
    if (at->ndim != 2 && at->ndim != 3) return TS_ERR_INVALID_ARG;
    if (at->nq > 0 && !at->q_coords) return TS_ERR_INVALID_ARG;
    if (at->nk > 0 && !at->k_coords && (!at->q_coords || at->nk != at->nq)) return TS_ERR_INVALID_ARG;
  }
  return TS_OK;
}

AttnPlan plan_fwd(const ts_attn* at) { return ts::plan_fwd(at->nq, at->nk, at->n_sets, at->hq, at->hk, at->d); }
AttnPlan plan_dq(const ts_attn* at) { return ts::plan_dq(at->nq, at->nk, at->n_sets, at->hq, at->hk, at->d); }
AttnPlan plan_dkv(const ts_attn* at) { return ts::plan_dkv(at->nq, at->nk, at->n_sets, at->hq, at->hk, at->d); }

size_t part_floats(const ts_attn* at, const AttnPlan& p, int64_t rows, int extra) {
  return p.splits > 1 ? static_cast<size_t>(p.splits) * rows * (padded_width(at->d) + extra) : 0;
}

// The kernels read rows in 16-byte pieces.  Where the head width or a stride does
// not allow that, the operands are copied to dense rows of heads of a multiple of
// 8 elements in the workspace, and the results copied back.
bool repacks(const ts_attn* at) {
  return ((at->d | at->q_stride | at->k_stride | at->v_stride | at->o_stride) & 7) != 0;
}
int width8(const ts_attn* at) { return (at->d + 7) / 8 * 8; }
size_t q_copy_bytes(const ts_attn* at) {
  return align_up(static_cast<size_t>(at->nq) * at->hq * width8(at) * 2, 256);
}
size_t k_copy_bytes(const ts_attn* at) {
  return align_up(static_cast<size_t>(at->nk) * at->hk * width8(at) * 2, 256);
}

// q, out; k, v
size_t fwd_bytes(const ts_attn* at) {
  return (repacks(at) ? 2 * q_copy_bytes(at) + 2 * k_copy_bytes(at) : 0) +
         part_floats(at, plan_fwd(at), at->nq * at->hq, 2) * 4;
}

// floats beside a row's part of dq where it is mended
int mend_width(const ts_attn* at) { return mends_dq(at->d, at->nq * at->hq) ? padded_width(at->d) : 0; }

// q, out, dout, dq; k, v, dk, dv
size_t delta_bytes(const ts_attn* at) { return align_up(static_cast<size_t>(at->nq) * at->hq * 4, 256); }
size_t bwd_bytes(const ts_attn* at) {
  const size_t q = part_floats(at, plan_dq(at), at->nq * at->hq, 1 + mend_width(at));
  const size_t k = 2 * part_floats(at, plan_dkv(at), at->nk * at->hk, 0);
  return (repacks(at) ? 4 * q_copy_bytes(at) + 4 * k_copy_bytes(at) : 0) + delta_bytes(at) + (q > k ? q : k) * 4;
}

// fewer than 2^24 blocks of 256 threads along x: a launch dimension may have 2^32 threads
bool grid_ok(const ts_attn* at, const AttnPlan& p, int64_t n, int64_t mul) {
  return attn_tiles(n, mul, p.bm, at->n_sets) < (int64_t{1} << 24) - 64;
}

struct Carver {
  char* base;
  size_t off = 0;
  void* take(size_t bytes) {
    void* p = base + off;
    off += bytes;
    return p;
  }
};
// *p (n rows of `heads` heads) copied into the workspace; *p and *new_stride then name the copy.
hipError_t copy_in(const ts_attn* at, int heads, int64_t n, int64_t stride, const void** p, int64_t* new_stride,
                   Carver& c, hipStream_t s) {
  const int d8 = width8(at);
  *new_stride = static_cast<int64_t>(heads) * d8;
  void* dst = c.take(align_up(static_cast<size_t>(n) * *new_stride * 2, 256));
  const void* src = *p;
  *p = dst;
  return launch_attn_repack(src, stride, at->d, dst, *new_stride, d8, n, heads, s);
}
hipError_t copy_out(const ts_attn* at, const void* src, int heads, int64_t n, void* dst, int64_t stride, hipStream_t s) {
  const int d8 = width8(at);
  return launch_attn_repack(src, static_cast<int64_t>(heads) * d8, d8, dst, stride, at->d, n, heads, s);
}

AttnArgs attn_args(const ts_attn* at, const void* q, const void* k, const void* v, uint32_t* flags) {
  AttnArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.qs = at->q_starts;
  a.ks = at->k_starts ? at->k_starts : at->q_starts;
  a.slopes = at->slopes;
  a.qc = at->q_coords;
  a.kc = at->k_coords ? at->k_coords : at->q_coords;
  a.flags = flags;
  a.nq = at->nq;
  a.nk = at->nk;
  a.n_sets = at->n_sets;
  a.q_stride = at->q_stride;
  a.k_stride = at->k_stride;
  a.v_stride = at->v_stride;
  a.o_stride = at->o_stride;
  a.hq = at->hq;
  a.hk = at->hk;
  a.grp = at->hq / at->hk;
  a.d = at->d;
  a.ndim = at->ndim;
  a.scale = at->scale;
  a.negate = at->scale < 0.f;
  a.two = few_rows(at->nq * at->hq);
  a.mend = mends_dq(at->d, at->nq * at->hq);
  if (at->cap > 0.f) {
    a.c1 = cap_factor(at);
    a.c2 = at->cap * kLog2e;
  } else {
    a.c1 = fabsf(at->scale) * kLog2e;
  }
  return a;
}

bool dtype_ok(int d) { return d == TS_F32 || d == TS_F16 || d == TS_BF16; }

bool rows_ok(int64_t n, int c, ts_dtype dtype) {
  return n >= 0 && n <= kMaxRows && c >= 1 && c <= (1 << 16) && dtype_ok(dtype);
}
bool act_ok(const ts_act8* a) { return a && a->codes && a->scales; }
Act8 act_view(const ts_act8* a, int c) {
  return a ? Act8{a->codes, a->scales, c % 8 == 0 && at8(a->codes)} : Act8{nullptr, nullptr, false};
}

}  // namespace

extern "C" {

size_t ts_attn_workspace_bytes(const ts_attn* at, int backward) {
  if (check_attn(at) != TS_OK) return 0;
  return backward ? bwd_bytes(at) : fwd_bytes(at);
}

ts_status ts_attn_fwd(const ts_attn* at, const void* q, const void* k, const void* v, void* out, float* lse, void* ws,
                      size_t ws_bytes, uint32_t* err_flags, hipStream_t stream) {
  const ts_status st = check_attn(at);
  if (st != TS_OK) return st;
  if ((at->nq > 0 && (!q || !out || !lse)) || (at->nk > 0 && (!k || !v))) return TS_ERR_INVALID_ARG;
  const size_t need = fwd_bytes(at);
  if (need > 0 && (!ws || ws_bytes < need || !at16(ws))) return TS_ERR_INVALID_ARG;
  const AttnPlan p = plan_fwd(at);
  const int grp = at->hq / at->hk;
  if (!grid_ok(at, p, at->nq, grp)) return TS_ERR_UNSUPPORTED;
  if (at->nq == 0 && !err_flags) return TS_OK;  // (without rows the blocks look at the starts and end)
  AttnArgs a = attn_args(at, q, k, v, err_flags);
  a.out = out;
  a.lse = lse;
  Carver c{static_cast<char*>(ws)};
  if (repacks(at)) {
    TS_TRY(copy_in(at, at->hq, at->nq, at->q_stride, &a.q, &a.q_stride, c, stream));
    TS_TRY(copy_in(at, at->hk, at->nk, at->k_stride, &a.k, &a.k_stride, c, stream));
    TS_TRY(copy_in(at, at->hk, at->nk, at->v_stride, &a.v, &a.v_stride, c, stream));
    a.out = c.take(q_copy_bytes(at));
    a.o_stride = static_cast<int64_t>(at->hq) * width8(at);
    a.d = width8(at);
  } else if (!at16(q) || !at16(k) || !at16(v) || !at8(out)) {
    return TS_ERR_INVALID_ARG;
  }
  a.part = static_cast<float*>(c.take(0));
  a.part_ml = a.part + static_cast<size_t>(p.splits) * at->nq * at->hq * padded_width(at->d);
  TS_TRY(launch_attn_fwd(a, p, at->dtype, at->cap > 0.f, stream));
  if (repacks(at)) TS_TRY(copy_out(at, a.out, at->hq, at->nq, out, at->o_stride, stream));
  return TS_OK;
}

ts_status ts_attn_bwd(const ts_attn* at, const void* q, const void* k, const void* v, const void* out,
                      const float* lse, const void* dout, void* dq, void* dk, void* dv, void* ws, size_t ws_bytes,
                      uint32_t* err_flags, hipStream_t stream) {
  const ts_status st = check_attn(at);
  if (st != TS_OK) return st;
  if ((at->nq > 0 && (!q || !out || !lse || !dout || !dq)) || (at->nk > 0 && (!k || !v || !dk || !dv)))
    return TS_ERR_INVALID_ARG;
  const size_t need = bwd_bytes(at);
  if (need > 0 && (!ws || ws_bytes < need || !at16(ws))) return TS_ERR_INVALID_ARG;
  const AttnPlan pq = plan_dq(at), pk = plan_dkv(at);
  if (!grid_ok(at, pq, at->nq, at->hq / at->hk) || !grid_ok(at, pk, at->nk, 1)) return TS_ERR_UNSUPPORTED;
  AttnArgs a = attn_args(at, q, k, v, err_flags);
  a.o = out;
  a.dout = dout;
  a.lse = const_cast<float*>(lse);
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  Carver c{static_cast<char*>(ws)};
  if (repacks(at)) {
    TS_TRY(copy_in(at, at->hq, at->nq, at->q_stride, &a.q, &a.q_stride, c, stream));
    TS_TRY(copy_in(at, at->hq, at->nq, at->o_stride, &a.o, &a.o_stride, c, stream));
    TS_TRY(copy_in(at, at->hq, at->nq, at->o_stride, &a.dout, &a.o_stride, c, stream));
    TS_TRY(copy_in(at, at->hk, at->nk, at->k_stride, &a.k, &a.k_stride, c, stream));
    TS_TRY(copy_in(at, at->hk, at->nk, at->v_stride, &a.v, &a.v_stride, c, stream));
    a.dq = c.take(q_copy_bytes(at));
    a.dk = c.take(k_copy_bytes(at));
    a.dv = c.take(k_copy_bytes(at));
    a.d = width8(at);
  } else if (!at16(q) || !at16(k) || !at16(v) || !at16(out) || !at16(dout) || !at8(dq) || !at8(dk) || !at8(dv)) {
    return TS_ERR_INVALID_ARG;
  }
  a.delta = static_cast<float*>(c.take(delta_bytes(at)));
  a.part = static_cast<float*>(c.take(0));
  a.part_ml = a.part + static_cast<size_t>(pq.splits) * at->nq * at->hq * (padded_width(at->d) + mend_width(at));
  TS_TRY(launch_attn_bwd(a, pq, pk, at->dtype, at->cap > 0.f, stream));
  if (repacks(at)) {
    TS_TRY(copy_out(at, a.dq, at->hq, at->nq, dq, at->q_stride, stream));
    TS_TRY(copy_out(at, a.dk, at->hk, at->nk, dk, at->k_stride, stream));
    TS_TRY(copy_out(at, a.dv, at->hk, at->nk, dv, at->v_stride, stream));
  }
  return TS_OK;
}

ts_status ts_act_pack(const void* x, int64_t n, int c, ts_dtype dtype, const ts_act8* a, hipStream_t stream) {
  if (!rows_ok(n, c, dtype)) return TS_ERR_INVALID_ARG;
  if (n > 0 && (!x || !act_ok(a))) return TS_ERR_INVALID_ARG;
  return launch_act_pack(x, n, c, dtype, act_view(a, c), stream) == hipSuccess ? TS_OK : TS_ERR_HIP;
}

ts_status ts_act_unpack(const ts_act8* a, int64_t n, int c, void* x, ts_dtype dtype, hipStream_t stream) {
  if (!rows_ok(n, c, dtype)) return TS_ERR_INVALID_ARG;
  if (n > 0 && (!x || !act_ok(a))) return TS_ERR_INVALID_ARG;
  return launch_act_unpack(act_view(a, c), n, c, x, dtype, stream) == hipSuccess ? TS_OK : TS_ERR_HIP;
}

size_t ts_conv_wgrad_act8_workspace_bytes(const ts_kmap* map, int cin, int cout) {
  if (!map || cin < 1 || cout < 1) return 0;
  return wgrad_act8_workspace_bytes(map, cin, cout);
}

ts_status ts_conv_bwd_wgrad_act8(const ts_kmap* map, const ts_act8* x, int cin, const void* dy, int cout,
                                 ts_dtype dtype, float* dw, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (!map || map->kvol < 1 || map->kvol > TS_MAX_KVOL || !map->fwd.row_mask) return TS_ERR_INVALID_ARG;
  if (cin < 1 || cout < 1 || cin > (1 << 16) || cout > (1 << 16) || !dtype_ok(dtype)) return TS_ERR_INVALID_ARG;
  if (dtype == TS_F32) return TS_ERR_UNSUPPORTED;
  if (!(map->flags & TS_KMAP_PAIRS) || !dw || (map->n_in > 0 && !act_ok(x)) || (map->n_out_cap > 0 && !dy))
    return TS_ERR_INVALID_ARG;
  if (!ws || ws_bytes < wgrad_act8_workspace_bytes(map, cin, cout)) return TS_ERR_INVALID_ARG;
  TS_TRY(launch_wgrad_act8(map, act_view(x, cin), cin, dy, cout, dtype, dw, ws, stream));
  return TS_OK;
}

ts_status ts_norm_fwd(const void* x, const void* residual, const float* w, int64_t n, int c, float eps,
                      ts_dtype dtype, void* h, void* y, float* rstd, const ts_act8* y8, const ts_act8* h8,
                      hipStream_t stream) {
  if (!rows_ok(n, c, dtype)) return TS_ERR_INVALID_ARG;
  if (!std::isfinite(eps) || eps < 0.f || (n > 0 && (!x || !w))) return TS_ERR_INVALID_ARG;
  if (!h && !y && !y8 && !h8) return TS_ERR_INVALID_ARG;
  if (n > 0 && ((y8 && !act_ok(y8)) || (h8 && !act_ok(h8)))) return TS_ERR_INVALID_ARG;
  return launch_norm_fwd(x, residual, w, n, c, eps, dtype, h, y, rstd, act_view(y8, c), act_view(h8, c), stream) ==
                 hipSuccess
             ? TS_OK
             : TS_ERR_HIP;
}

size_t ts_norm_workspace_bytes(int64_t n, int c) {
  return rows_ok(n, c, TS_F32) ? norm_workspace_bytes(n, c) : 0;
}

ts_status ts_norm_bwd(const void* dy, const void* h, const ts_act8* h8, const float* w, const float* rstd,
                      const void* dh, int64_t n, int c, ts_dtype dtype, void* dx, float* dw, void* ws,
                      size_t ws_bytes, hipStream_t stream) {
  if (!rows_ok(n, c, dtype)) return TS_ERR_INVALID_ARG;
  if (!dw || (n > 0 && (!dy || !w || !rstd || !dx || (h != nullptr) == (h8 != nullptr) || (h8 && !act_ok(h8)))))
    return TS_ERR_INVALID_ARG;
  if (n > 0 && (!ws || ws_bytes < norm_workspace_bytes(n, c))) return TS_ERR_INVALID_ARG;
  return launch_norm_bwd(dy, h, act_view(h8, c), w, rstd, dh, n, c, dtype, dx, dw, ws, stream) == hipSuccess
             ? TS_OK
             : TS_ERR_HIP;
}

}  // extern "C"
