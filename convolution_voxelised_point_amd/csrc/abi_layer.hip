// C entry points of the rest of a voxel-transformer layer (query and key rotation,
// routing to experts, their products and the sum of what they returned): host-side
// validation and workspace layout.
#include <cmath>

#include "common.h"
#include "group.h"
#include "rope.h"
#include "route.h"

using namespace ts;

namespace {

constexpr int64_t kMaxRows = (int64_t{1} << 31) - 1;
constexpr int64_t kMaxChannels = 1 << 16;

bool dtype_ok(int d) { return d == TS_F32 || d == TS_F16 || d == TS_BF16; }
ts_status status(hipError_t e) { return e == hipSuccess ? TS_OK : TS_ERR_HIP; }

// ---------------------------------------------------------------- rotation
int64_t pairs_of(const ts_rope* r) {
  int64_t p = 0;
  for (int a = 0; a < r->ndim; ++a) p += r->pairs[a];
  return p;
}

ts_status check_rope(const ts_rope* r) {
  if (!r || !dtype_ok(r->dtype) || r->d < 1 || r->n < 0 || (r->ndim != 2 && r->ndim != 3)) return TS_ERR_INVALID_ARG;
  if (!std::isfinite(r->eps) || r->eps < 0.f) return TS_ERR_INVALID_ARG;
  for (int a = 0; a < r->ndim; ++a)
    if (r->pairs[a] < 0 || r->pairs[a] > r->d) return TS_ERR_INVALID_ARG;
  const int64_t p = pairs_of(r);
  if (2 * p > r->d || (p > 0 && r->n > 0 && (!r->coords || !r->freqs))) return TS_ERR_INVALID_ARG;
  if (r->d > kRopeMaxWidth) return TS_ERR_UNSUPPORTED;
  return TS_OK;
}

int heads_of(const ts_rope_heads* h) { return h ? h->heads : 0; }

ts_status check_heads(const ts_rope* r, const ts_rope_heads* h, bool back) {
  if (!h || h->heads == 0) return TS_OK;
  if (h->heads < 0) return TS_ERR_INVALID_ARG;
  if (h->heads > 65535 || r->n > kMaxRows / h->heads) return TS_ERR_UNSUPPORTED;
  const int64_t row = static_cast<int64_t>(h->heads) * r->d;
  if (r->n == 0) return back && h->w && !h->dw ? TS_ERR_INVALID_ARG : TS_OK;
  if (!back) return !h->x || !h->y || h->x_stride < row || h->y_stride < row ? TS_ERR_INVALID_ARG : TS_OK;
  if (!h->dy || !h->dx || h->dy_stride < row || h->dx_stride < row) return TS_ERR_INVALID_ARG;
  if (h->w && (!h->x || h->x_stride < row || !h->dw)) return TS_ERR_INVALID_ARG;
  return TS_OK;
}

RopeSide side_of(const ts_rope_heads* h) {
  RopeSide s{};
  if (!h) return s;
  s.heads = h->heads;
  s.x_stride = h->x_stride;
  s.y_stride = h->y_stride;
  s.dy_stride = h->dy_stride;
  s.dx_stride = h->dx_stride;
  s.x = h->x;
  s.w = h->w;
  s.y = h->y;
  s.dy = h->dy;
  s.dx = h->dx;
  s.dw = h->w ? h->dw : nullptr;
  return s;
}

RopeK rope_args(const ts_rope* r, const ts_rope_heads* q, const ts_rope_heads* k) {
  RopeK a{};
  a.side[0] = side_of(q);
  a.side[1] = side_of(k);
  a.coords = r->coords;
  a.freqs = r->freqs;
  a.n = r->n;
  a.eps = r->eps;
  a.inv_d = 1.f / static_cast<float>(r->d);
  a.d = r->d;
  a.ndim = r->ndim;
  a.pairs = static_cast<int>(pairs_of(r));
  a.upto[0] = r->pairs[0];
  a.upto[1] = r->pairs[0] + r->pairs[1];
  a.rest = (r->d - 2 * a.pairs) / 2;
  a.odd = r->d & 1;
  return a;
}

size_t rope_bytes(const ts_rope* r, int hq, int hk) {
  return 2 * static_cast<size_t>(rope_blocks(r->n, hq + hk, r->d)) * r->d * sizeof(float);
}

// ---------------------------------------------------------------- routing
ts_status check_route(int64_t n, int e, ts_dtype dt, int top) {
  if (n < 0 || e < 1 || top < 1 || top > e || !dtype_ok(dt)) return TS_ERR_INVALID_ARG;
  if (e > kRouteMaxExperts || top > kRouteMaxTop || n > kMaxRows / top) return TS_ERR_UNSUPPORTED;
  return TS_OK;
}

ts_status check_combine(int64_t n, int64_t n_rows, int top, int c, ts_dtype dt) {
  if (n < 0 || n_rows < 0 || n > kMaxRows || n_rows > kMaxRows || top < 1 || c < 1 || c > kMaxChannels || !dtype_ok(dt))
    return TS_ERR_INVALID_ARG;
  return TS_OK;
}

// ---------------------------------------------------------------- products grouped by expert
constexpr int kMaxGroups = 4096;

ts_status check_groups(const ts_groups* g, int cin, int cout, ts_dtype dt) {
  if (!g || g->n_groups < 1 || g->n_rows < 0 || g->n_rows > kMaxRows || !g->starts || !dtype_ok(dt)) return TS_ERR_INVALID_ARG;
  if (cin < 1 || cout < 1 || cin > kMaxChannels || cout > kMaxChannels) return TS_ERR_INVALID_ARG;
  if (g->rows && (g->n_src < 0 || g->n_src > kMaxRows)) return TS_ERR_INVALID_ARG;
  if (dt == TS_F32 || g->n_groups > kMaxGroups) return TS_ERR_UNSUPPORTED;
  return TS_OK;
}

// Tiles are fewer than 2^22.  The kernel for few rows has a block of 512 threads for each, and a launch may
// have 2^32 threads; the other one's few blocks number them in 32 bits, in bands of four rows of tiles.
bool grid_ok(const ts_groups* g, GroupOp op, int cin, int columns) {
  int64_t blocks;
  if (op == kGroupWgrad) {
    const int64_t tiles = static_cast<int64_t>(ceil_div(cin, 128)) * ceil_div(columns, 128);
    blocks = group_grid(group_chunks(g->n_rows, g->n_groups, group_chunk(g->n_rows, g->n_groups, cin, columns)), 1) * tiles;
  } else {
    const int64_t runs = group_runs(g->n_rows, g->n_groups, group_few(op, g->n_rows, g->n_groups, cin, columns) ? 16 : 128);
    blocks = group_grid(runs, static_cast<unsigned>(ceil_div(columns, 128)));
  }
  return blocks < (int64_t{1} << 22);
}

GroupK group_args(const ts_groups* g, int cin, int cout, uint32_t* flags) {
  GroupK k{};
  k.starts = g->starts;
  k.rows = g->rows;
  k.flags = flags;
  k.n_rows = g->n_rows;
  k.n_src = g->rows ? g->n_src : g->n_rows;
  k.e = g->n_groups;
  k.cin = cin;
  k.cout = k.ldw = cout;
  return k;
}

size_t wgrad_bytes(const ts_groups* g, int cin, int cout) {
  return static_cast<size_t>(group_chunks(g->n_rows, g->n_groups, group_chunk(g->n_rows, g->n_groups, cin, cout))) * cin * cout * sizeof(float);
}

}  // namespace

extern "C" {

size_t ts_rope_workspace_bytes(const ts_rope* r, int hq, int hk) {
  if (check_rope(r) != TS_OK || hq < 0 || hk < 0) return 0;
  return rope_bytes(r, hq, hk);
}

ts_status ts_rope_fwd(const ts_rope* r, const ts_rope_heads* q, const ts_rope_heads* k, hipStream_t stream) {
  ts_status st = check_rope(r);
  if (st == TS_OK) st = check_heads(r, q, false);
  if (st == TS_OK) st = check_heads(r, k, false);
  if (st != TS_OK) return st;
  RopeK a = rope_args(r, q, k);
  return status(launch_rope_fwd(a, r->dtype, r->interleaved != 0, stream));
}

ts_status ts_rope_bwd(const ts_rope* r, const ts_rope_heads* q, const ts_rope_heads* k, void* ws, size_t ws_bytes,
                      hipStream_t stream) {
  ts_status st = check_rope(r);
  if (st == TS_OK) st = check_heads(r, q, true);
  if (st == TS_OK) st = check_heads(r, k, true);
  if (st != TS_OK) return st;
  const int hq = heads_of(q), hk = heads_of(k);
  const size_t need = rope_bytes(r, hq, hk);
  if (need > 0 && (!ws || ws_bytes < need)) return TS_ERR_INVALID_ARG;
  if (hq + hk == 0) return TS_OK;
  RopeK a = rope_args(r, q, k);
  a.part = static_cast<float*>(ws);
  a.blocks = rope_blocks(r->n, hq + hk, r->d);
  return status(launch_rope_bwd(a, r->dtype, r->interleaved != 0, stream));
}

size_t ts_route_workspace_bytes(int64_t n, int n_experts, int top) {
  if (check_route(n, n_experts, TS_F32, top) != TS_OK || n == 0 || route_small(n, n_experts, top)) return 0;
  return static_cast<size_t>(n_experts + 1) * (route_blocks(n, n_experts) + 1) * sizeof(int32_t);
}

ts_status ts_route_fwd(const void* logits, int64_t n, int n_experts, ts_dtype dtype, int top, int over_all,
                       int32_t* experts, float* gates, int64_t* starts, int32_t* rows, int32_t* place, void* ws,
                       size_t ws_bytes, hipStream_t stream) {
  const ts_status st = check_route(n, n_experts, dtype, top);
  if (st != TS_OK) return st;
  if (!starts || (n > 0 && (!logits || !experts || !gates || !rows || !place))) return TS_ERR_INVALID_ARG;
  const size_t need = ts_route_workspace_bytes(n, n_experts, top);
  if (need > 0 && (!ws || ws_bytes < need)) return TS_ERR_INVALID_ARG;
  RouteK k{};
  k.logits = logits;
  k.n = n;
  k.e = n_experts;
  k.top = top;
  k.over_all = over_all != 0;
  k.experts = experts;
  k.gates = gates;
  k.starts = starts;
  k.rows = rows;
  k.place = place;
  k.counts = static_cast<int32_t*>(ws);
  return status(launch_route(k, dtype, false, stream));
}

ts_status ts_route_bwd(const float* dgates, const void* logits, const int32_t* experts, const float* gates, int64_t n,
                       int n_experts, ts_dtype dtype, int top, int over_all, void* dlogits, hipStream_t stream) {
  const ts_status st = check_route(n, n_experts, dtype, top);
  if (st != TS_OK) return st;
  if (n > 0 && (!dgates || (over_all && !logits) || !experts || !gates || !dlogits)) return TS_ERR_INVALID_ARG;
  RouteK k{};
  k.logits = logits;
  k.n = n;
  k.e = n_experts;
  k.top = top;
  k.over_all = over_all != 0;
  k.experts = const_cast<int32_t*>(experts);
  k.gates = const_cast<float*>(gates);
  k.dgates = dgates;
  k.dlogits = dlogits;
  return status(launch_route(k, dtype, true, stream));
}

ts_status ts_combine_fwd(const void* y, int64_t n_rows, const int32_t* place, const float* gates, int64_t n, int top, int c,
                         ts_dtype dtype, void* out, uint32_t* err_flags, hipStream_t stream) {
  const ts_status st = check_combine(n, n_rows, top, c, dtype);
  if (st != TS_OK) return st;
  if (n > 0 && (!place || !out || (n_rows > 0 && !y))) return TS_ERR_INVALID_ARG;
  return status(launch_combine_fwd(y, n_rows, place, gates, n, top, c, dtype, out, err_flags, stream));
}

ts_status ts_combine_bwd(const void* dout, const void* y, int64_t n_rows, const int32_t* place, const float* gates,
                         int64_t n, int top, int c, ts_dtype dtype, void* dy, float* dgates, uint32_t* err_flags,
                         hipStream_t stream) {
  const ts_status st = check_combine(n, n_rows, top, c, dtype);
  if (st != TS_OK) return st;
  if (n > 0 && (!place || !dout || !gates || !dgates || (n_rows > 0 && (!y || !dy)))) return TS_ERR_INVALID_ARG;
  return status(launch_combine_bwd(dout, y, n_rows, place, gates, n, top, c, dtype, dy, dgates, err_flags, stream));
}

ts_status ts_group_fwd(const ts_groups* g, const void* x, int cin, const void* w, int cout, ts_dtype dtype, int glu, void* y,
                       void* h, uint32_t* err_flags, hipStream_t stream) {
  const ts_status st = check_groups(g, cin, cout, dtype);
  if (st != TS_OK) return st;
  if (!w || (h && !glu) || (g->n_rows > 0 && (!y || (!x && (!g->rows || g->n_src > 0))))) return TS_ERR_INVALID_ARG;
  if (!grid_ok(g, kGroupFwd, cin, glu ? 2 * cout : cout)) return TS_ERR_UNSUPPORTED;
  if (g->n_rows == 0) return TS_OK;
  GroupK k = group_args(g, cin, cout, err_flags);
  k.x = x;
  k.w = w;
  k.y = y;
  k.h_out = h;
  if (glu) k.ldw = 2 * cout;
  return status(group_few(kGroupFwd, k.n_rows, k.e, cin, k.ldw) ? launch_group_few(k, kGroupFwd, dtype, glu != 0, stream)
                                                    : launch_group(k, kGroupFwd, dtype, glu != 0, stream));
}

ts_status ts_group_bwd_dgrad(const ts_groups* g, const void* dy, int cout, const void* w, int cin, ts_dtype dtype,
                             const void* h, void* dx, uint32_t* err_flags, hipStream_t stream) {
  const ts_status st = check_groups(g, cin, cout, dtype);
  if (st != TS_OK) return st;
  if (!w || (g->n_rows > 0 && (!dy || !dx))) return TS_ERR_INVALID_ARG;
  if (!grid_ok(g, kGroupDgrad, cin, cin)) return TS_ERR_UNSUPPORTED;
  if (g->n_rows == 0) return TS_OK;
  GroupK k = group_args(g, cin, cout, err_flags);
  k.dy = dy;
  k.w = w;
  k.h = h;
  k.y = dx;
  return status(group_few(kGroupDgrad, k.n_rows, k.e, cin, cin) ? launch_group_few(k, kGroupDgrad, dtype, h != nullptr, stream)
                                                      : launch_group(k, kGroupDgrad, dtype, h != nullptr, stream));
}

size_t ts_group_wgrad_workspace_bytes(const ts_groups* g, int cin, int cout) {
  return check_groups(g, cin, cout, TS_F16) == TS_OK ? wgrad_bytes(g, cin, cout) : 0;
}

ts_status ts_group_bwd_wgrad(const ts_groups* g, const void* x, int cin, const void* dy, int cout, ts_dtype dtype, float* dw,
                             void* ws, size_t ws_bytes, uint32_t* err_flags, hipStream_t stream) {
  const ts_status st = check_groups(g, cin, cout, dtype);
  if (st != TS_OK) return st;
  if (!dw || (g->n_rows > 0 && (!dy || (!x && (!g->rows || g->n_src > 0))))) return TS_ERR_INVALID_ARG;
  if (!grid_ok(g, kGroupWgrad, cin, cout)) return TS_ERR_UNSUPPORTED;
  if (!ws || ws_bytes < wgrad_bytes(g, cin, cout)) return TS_ERR_INVALID_ARG;
  GroupK k = group_args(g, cin, cout, err_flags);
  k.x = x;
  k.dy = dy;
  k.dw = dw;
  k.part = static_cast<float*>(ws);
  k.chunk = group_chunk(g->n_rows, g->n_groups, cin, cout);
  return status(launch_group(k, kGroupWgrad, dtype, false, stream));
}

}  // extern "C"
