// C ABI of the verify step's operators around the products (cache append, with
// and without rotation, attention, with and without a common prefix, draft
// acceptance, routing, adapters): argument validation and launch (contracts in include/qgemv.h).

#include <stdint.h>

#include <algorithm>

#include "qgemv_kv.h"

using qgemv::AppendArgs;
using qgemv::AttendArgs;
using qgemv::KvView;
using qgemv::VerifyArgs;

namespace {

// Of 256 threads, in a grid: its threads are counted in 32 bits.
constexpr int kMaxWorkgroups = (1 << 24) - 1;
// Values of a row's keys that the append takes: it counts them in 32 bits.
constexpr int64_t kMaxRow = 1 << 30;

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int elem_bytes(int dtype) { return dtype == QGEMV_F32 ? 4 : dtype == QGEMV_E4M3 ? 1 : 2; }

int view_of(const qgemv_kv_cache *c, KvView *v) {
  if (!c) return QGEMV_EINVAL;
  if (c->dim != 64 && c->dim != 128 && c->dim != 256) return QGEMV_EINVAL;
  if (c->dtype != QGEMV_BF16 && c->dtype != QGEMV_F16 && c->dtype != QGEMV_E4M3) return QGEMV_EINVAL;
  if (c->heads < 1 || c->pages < 1 || c->page < 1 || c->width < 1 || c->batch < 1) return QGEMV_EINVAL;
  if ((int64_t)c->page * c->width > QGEMV_MAX_CONTEXT) return QGEMV_EINVAL;
  if (c->stride_page < 1 || c->stride_slot < 1 || c->stride_head < 1) return QGEMV_EINVAL;
  if (!c->k || !c->v || !c->table) return QGEMV_EINVAL;
  const bool f8 = c->dtype == QGEMV_E4M3;
  if (f8 != (c->k_scale != nullptr) || f8 != (c->v_scale != nullptr)) return QGEMV_EINVAL;
  if (c->stride_page % 16 || c->stride_slot % 16 || c->stride_head % 16) return QGEMV_EALIGN;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->table, 4) || !aligned(c->k_scale, 4) ||
      !aligned(c->v_scale, 4))
    return QGEMV_EALIGN;
  v->k = static_cast<uint8_t *>(c->k);
  v->v = static_cast<uint8_t *>(c->v);
  v->table = c->table;
  v->k_scale = c->k_scale;
  v->v_scale = c->v_scale;
  v->stride_page = c->stride_page;
  v->stride_slot = c->stride_slot;
  v->stride_head = c->stride_head;
  v->pages = c->pages;
  v->page = c->page;
  v->width = c->width;
  v->H = c->heads;
  v->D = c->dim;
  v->dtype = c->dtype;
  qgemv::page_magic(c->page, &v->magic, &v->shift);
  return QGEMV_OK;
}

int rows_status(const int32_t *start, const int32_t *len, int T) {
  if (T < 0 || !start || !len) return QGEMV_EINVAL;
  return aligned(start, 4) && aligned(len, 4) ? QGEMV_OK : QGEMV_EALIGN;
}

// A [T][heads][dim] operand: strides in elements, at least one row's and one
// head's extent apart.
int operand_status(const void *p, int64_t row, int64_t head, int dim, int dtype) {
  if (!p || head < dim || row < dim) return QGEMV_EINVAL;
  const int64_t b = elem_bytes(dtype);
  return aligned(p, 16) && row * b % 16 == 0 && head * b % 16 == 0 ? QGEMV_OK : QGEMV_EALIGN;
}

int attend_shape(const qgemv_kv_cache *c, int M, int q_heads, int T) {
  if (M < 1 || M > QGEMV_MAX_M || T < 0 || q_heads < 1 || q_heads % c->heads) return QGEMV_EINVAL;
  return q_heads / c->heads <= QGEMV_MAX_GROUP ? QGEMV_OK : QGEMV_EUNSUPPORTED;
}

// Whether two operands lie in common memory, by where they begin and end.
bool overlap(const void *p, int64_t p_bytes, const void *q, int64_t q_bytes) {
  const uint8_t *a = static_cast<const uint8_t *>(p), *b = static_cast<const uint8_t *>(q);
  return a < b + q_bytes && b < a + p_bytes;
}
int64_t extent(int64_t T, int64_t row, int64_t heads, int64_t head, int64_t dim, int64_t bytes) {
  return T < 1 ? 0 : ((T - 1) * row + (heads - 1) * head + dim) * bytes;
}

// Whether two operands of rows `row` bytes apart, of which they take so many bytes
// each, are different columns of one buffer: no row of one meets any of the other.
bool columns_apart(const void *p, int64_t p_bytes, const void *q, int64_t q_bytes, int64_t row) {
  const int64_t d = (int64_t)(reinterpret_cast<uintptr_t>(q) - reinterpret_cast<uintptr_t>(p)) % row;
  const int64_t from = d < 0 ? d + row : d;  // where q's columns begin in p's row
  return from >= p_bytes && row - from >= q_bytes;
}

// Whether no two values of an operand lie in one place: rows apart, or heads.
bool distinct(int64_t T, int64_t row, int64_t heads, int64_t head, int64_t dim) {
  return T <= 1 || heads <= 1 || row >= (heads - 1) * head + dim || head >= (T - 1) * row + dim;
}

// What attention calls have in common, but for the workspace.
int attend_args(const qgemv_kv_cache *cache, const void *q, int64_t q_row, int64_t q_head, void *out, int64_t out_row,
                int64_t out_head, int q_dtype, float *lse, const int32_t *start, const int32_t *len, int T, int M,
                int q_heads, int window, int sinks, float scale, const void *workspace, AttendArgs *a) {
  int s = view_of(cache, &a->c);
  if (s != QGEMV_OK) return s;
  if ((s = attend_shape(cache, M, q_heads, T)) != QGEMV_OK) return s;
  if (q_dtype != QGEMV_BF16 && q_dtype != QGEMV_F16) return QGEMV_EINVAL;
  if (a->c.dtype != QGEMV_E4M3 && a->c.dtype != q_dtype) return QGEMV_EINVAL;
  if (window < 0 || sinks < 0) return QGEMV_EINVAL;
  if ((s = rows_status(start, len, T)) != QGEMV_OK) return s;
  if ((s = operand_status(q, q_row, q_head, a->c.D, q_dtype)) != QGEMV_OK) return s;
  if ((s = operand_status(out, out_row, out_head, a->c.D, q_dtype)) != QGEMV_OK) return s;
  if (!workspace) return QGEMV_EINVAL;
  if (!aligned(lse, 4) || !aligned(workspace, 16)) return QGEMV_EALIGN;
  a->q = static_cast<const uint8_t *>(q);
  a->out = static_cast<uint8_t *>(out);
  a->lse = lse;
  a->start = start;
  a->len = len;
  a->q_row = q_row * 2;
  a->q_head = q_head * 2;
  a->out_row = out_row * 2;
  a->out_head = out_head * 2;
  a->B = cache->batch;
  a->T = T;
  a->M = M;
  a->G = q_heads / cache->heads;
  // no position reaches QGEMV_MAX_CONTEXT, so a wider window sees the same
  a->window = window < QGEMV_MAX_CONTEXT ? window : QGEMV_MAX_CONTEXT;
  a->sinks = sinks;
  a->q_dtype = q_dtype;
  a->scale = scale;
  a->common = nullptr;
  return QGEMV_OK;
}

// Fewer rows can need more (other tiles a wave, items shared where M rows are
// walked whole): what the call of any M up to this one needs.
int64_t attend_most(AttendArgs *a, int M, bool after_prefix) {
  a->window = a->sinks = 0;  // the most that any window needs
  int64_t most = 0;
  for (a->M = 1; a->M <= M; ++a->M) {
    const int64_t need = qgemv::plan_attend(a, nullptr, after_prefix);
    if (need < 0) return need;
    most = std::max(most, need);
  }
  return most;
}

}  // namespace

extern "C" {

int qgemv_kv_append(const qgemv_kv_cache *cache, const void *new_k, int64_t k_row, int64_t k_head,
                    const void *new_v, int64_t v_row, int64_t v_head, int src_dtype,
                    const int32_t *start, const int32_t *len, int T, void *stream) {
  AppendArgs a;
  int s = view_of(cache, &a.c);
  if (s != QGEMV_OK) return s;
  if (src_dtype != QGEMV_F32 && src_dtype != QGEMV_BF16 && src_dtype != QGEMV_F16) return QGEMV_EINVAL;
  if ((s = rows_status(start, len, T)) != QGEMV_OK) return s;
  if ((s = operand_status(new_k, k_row, k_head, a.c.D, src_dtype)) != QGEMV_OK) return s;
  if ((s = operand_status(new_v, v_row, v_head, a.c.D, src_dtype)) != QGEMV_OK) return s;
  if (T == 0) return QGEMV_OK;
  if (T > kMaxWorkgroups || (int64_t)a.c.H * a.c.D > kMaxRow) return QGEMV_EUNSUPPORTED;
  const int64_t b = elem_bytes(src_dtype);
  a.nk = static_cast<const uint8_t *>(new_k);
  a.nv = static_cast<const uint8_t *>(new_v);
  a.k_row = k_row * b;
  a.k_head = k_head * b;
  a.v_row = v_row * b;
  a.v_head = v_head * b;
  a.start = start;
  a.len = len;
  a.B = cache->batch;
  a.T = T;
  a.src = src_dtype;
  return qgemv::launch_append(a, reinterpret_cast<hipStream_t>(stream));
}

int64_t qgemv_kv_attend_workspace(const qgemv_kv_cache *cache, int M, int q_heads, int T) {
  KvView v;
  int s = view_of(cache, &v);
  if (s != QGEMV_OK) return s;
  if ((s = attend_shape(cache, M, q_heads, T)) != QGEMV_OK) return s;
  AttendArgs a;
  a.c = v;
  a.B = cache->batch;
  a.T = T;
  a.G = q_heads / cache->heads;
  return attend_most(&a, M, false);
}

int qgemv_kv_attend(const qgemv_kv_cache *cache, const void *q, int64_t q_row, int64_t q_head,
                    void *out, int64_t out_row, int64_t out_head, int q_dtype, float *lse,
                    const int32_t *start, const int32_t *len, int T, int M, int q_heads, int window,
                    int sinks, float scale, void *workspace, int64_t workspace_bytes, void *stream) {
  AttendArgs a;
  const int s = attend_args(cache, q, q_row, q_head, out, out_row, out_head, q_dtype, lse, start, len, T, M, q_heads,
                            window, sinks, scale, workspace, &a);
  if (s != QGEMV_OK) return s;
  const int64_t need = qgemv::plan_attend(&a, workspace);
  if (need < 0) return (int)need;
  if (need > workspace_bytes) return QGEMV_EINVAL;
  if (T == 0) return QGEMV_OK;
  return qgemv::launch_attend(a, reinterpret_cast<hipStream_t>(stream));
}

int64_t qgemv_kv_attend_shared_workspace(const qgemv_kv_cache *cache, int M, int q_heads, int T) {
  AttendArgs a;
  int s = view_of(cache, &a.c);
  if (s != QGEMV_OK) return s;
  if ((s = attend_shape(cache, M, q_heads, T)) != QGEMV_OK) return s;
  a.B = cache->batch;
  a.T = T;
  a.G = q_heads / cache->heads;
  const int64_t prefix = qgemv::plan_prefix(&a, nullptr);
  const int64_t own = attend_most(&a, M, true);
  return prefix < 0 ? prefix : own < 0 ? own : prefix + own;
}

int qgemv_kv_attend_shared(const qgemv_kv_cache *cache, const void *q, int64_t q_row, int64_t q_head,
                           void *out, int64_t out_row, int64_t out_head, int q_dtype, float *lse,
                           const int32_t *start, const int32_t *len, const int32_t *shared, int T, int M,
                           int q_heads, int window, int sinks, float scale, void *workspace,
                           int64_t workspace_bytes, void *stream) {
  AttendArgs a;
  const int s = attend_args(cache, q, q_row, q_head, out, out_row, out_head, q_dtype, lse, start, len, T, M, q_heads,
                            window, sinks, scale, workspace, &a);
  if (s != QGEMV_OK) return s;
  if (!shared) return QGEMV_EINVAL;
  if (!aligned(shared, 4)) return QGEMV_EALIGN;
  a.common = shared;
  const int64_t prefix = qgemv::plan_prefix(&a, workspace);
  if (prefix < 0) return (int)prefix;
  const int64_t own = qgemv::plan_attend(&a, static_cast<uint8_t *>(workspace) + prefix, true);
  if (own < 0) return (int)own;
  if (prefix + own > workspace_bytes) return QGEMV_EINVAL;
  if (T == 0) return QGEMV_OK;
  return qgemv::launch_attend_shared(a, reinterpret_cast<hipStream_t>(stream));
}

int qgemv_kv_append_rotated(const qgemv_kv_cache *cache, const void *q, int64_t q_row, int64_t q_head, int q_heads,
                            void *out, int64_t out_row, int64_t out_head, int out_dtype, const void *new_k,
                            int64_t k_row, int64_t k_head, const void *new_v, int64_t v_row, int64_t v_head,
                            int src_dtype, const int32_t *start, const int32_t *len, int T, const float *freq,
                            int pairs, const int32_t *position, int64_t position_axis, int axes,
                            const int32_t *axis, int interleaved, void *stream) {
  qgemv::RotateArgs r;
  AppendArgs &a = r.rows;
  int s = view_of(cache, &a.c);
  if (s != QGEMV_OK) return s;
  if (src_dtype != QGEMV_F32 && src_dtype != QGEMV_BF16 && src_dtype != QGEMV_F16) return QGEMV_EINVAL;
  if (out_dtype != QGEMV_BF16 && out_dtype != QGEMV_F16) return QGEMV_EINVAL;
  if (q_heads < 1) return QGEMV_EINVAL;
  if (pairs < 8 || pairs % 8 || pairs > a.c.D / 2 || !freq) return QGEMV_EINVAL;
  if (position ? axes < 1 || (axes > 1 && position_axis < T) : axis != nullptr) return QGEMV_EINVAL;
  if (interleaved != 0 && interleaved != 1) return QGEMV_EINVAL;
  if ((s = rows_status(start, len, T)) != QGEMV_OK) return s;
  if ((s = operand_status(q, q_row, q_head, a.c.D, src_dtype)) != QGEMV_OK) return s;
  if ((s = operand_status(out, out_row, out_head, a.c.D, out_dtype)) != QGEMV_OK) return s;
  if ((s = operand_status(new_k, k_row, k_head, a.c.D, src_dtype)) != QGEMV_OK) return s;
  if ((s = operand_status(new_v, v_row, v_head, a.c.D, src_dtype)) != QGEMV_OK) return s;
  if (!aligned(freq, 4) || !aligned(position, 4) || !aligned(axis, 4)) return QGEMV_EALIGN;
  if (T == 0) return QGEMV_OK;
  if (T > kMaxWorkgroups || (q_heads + 2 * (int64_t)a.c.H) * a.c.D > kMaxRow) return QGEMV_EUNSUPPORTED;
  const int64_t b = elem_bytes(src_dtype);
  if (!distinct(T, out_row, q_heads, out_head, a.c.D)) return QGEMV_EINVAL;
  // in place, value for value, or apart
  const bool in_place = out == q && out_dtype == src_dtype && out_row == q_row && out_head == q_head;
  auto meets_out = [&](const void *p, int64_t row, int64_t heads, int64_t head) {
    if (!overlap(p, extent(T, row, heads, head, a.c.D, b), out, extent(T, out_row, q_heads, out_head, a.c.D, 2)))
      return false;
    // columns of rows, or of heads where those of all rows are equally far apart (a
    // head's query, key and value side by side)
    if (row * b == out_row * 2 && columns_apart(p, extent(1, row, heads, head, a.c.D, b), out,
                                                extent(1, out_row, q_heads, out_head, a.c.D, 2), row * b))
      return false;
    const int64_t step = std::min(row, head), out_step = std::min(out_row, out_head);
    return !(step * b == out_step * 2 && row % step == 0 && head % step == 0 && out_row % out_step == 0 &&
             out_head % out_step == 0 && columns_apart(p, a.c.D * b, out, (int64_t)a.c.D * 2, step * b));
  };
  if ((!in_place && meets_out(q, q_row, q_heads, q_head)) || meets_out(new_k, k_row, a.c.H, k_head) ||
      meets_out(new_v, v_row, a.c.H, v_head))
    return QGEMV_EINVAL;
  a.nk = static_cast<const uint8_t *>(new_k);
  a.nv = static_cast<const uint8_t *>(new_v);
  a.k_row = k_row * b;
  a.k_head = k_head * b;
  a.v_row = v_row * b;
  a.v_head = v_head * b;
  a.start = start;
  a.len = len;
  a.B = cache->batch;
  a.T = T;
  a.src = src_dtype;
  r.q = static_cast<const uint8_t *>(q);
  r.out = static_cast<uint8_t *>(out);
  r.q_row = q_row * b;
  r.q_head = q_head * b;
  r.out_row = out_row * 2;
  r.out_head = out_head * 2;
  r.freq = freq;
  r.position = position;
  r.axis = axis;
  r.position_axis = position_axis;
  r.q_heads = q_heads;
  r.out_dtype = out_dtype;
  r.pairs = pairs;
  r.axes = axes;
  r.interleaved = interleaved != 0;
  return qgemv::launch_rotate(r, reinterpret_cast<hipStream_t>(stream));
}

int qgemv_route(const void *logits, int64_t row, int dtype, const float *bias, int32_t *experts, float *weights,
                int T, int E, int k, int score, int groups, int keep, int best, int renormalise, float scale,
                void *stream) {
  if (dtype != QGEMV_F32 && dtype != QGEMV_BF16 && dtype != QGEMV_F16) return QGEMV_EINVAL;
  if (score != QGEMV_SOFTMAX && score != QGEMV_SIGMOID) return QGEMV_EINVAL;
  if (T < 0 || E < 1 || row < E || groups < 1 || E % groups || keep < 1 || keep > groups) return QGEMV_EINVAL;
  if (best < 1 || best > 2 || (renormalise != 0 && renormalise != 1)) return QGEMV_EINVAL;
  if (k < 1 || k > E / groups * keep) return QGEMV_EINVAL;
  if (E > QGEMV_MAX_ROUTED || k > QGEMV_MAX_CHOSEN || groups > QGEMV_MAX_GROUPS) return QGEMV_EUNSUPPORTED;
  if (!logits || !experts || !weights) return QGEMV_EINVAL;
  if (!aligned(logits, (uintptr_t)elem_bytes(dtype)) || !aligned(bias, 4) || !aligned(experts, 4) || !aligned(weights, 4))
    return QGEMV_EALIGN;
  if (T == 0) return QGEMV_OK;
  if (T > kMaxWorkgroups) return QGEMV_EUNSUPPORTED;
  qgemv::RouteArgs a;
  a.logits = static_cast<const uint8_t *>(logits);
  a.row = row;
  a.bias = bias;
  a.experts = experts;
  a.weights = weights;
  a.T = T;
  a.E = E;
  a.k = k;
  a.dtype = dtype;
  a.groups = groups;
  a.keep = keep;
  a.best = groups > 1 ? best : 1;  // of one group nothing depends on it
  a.over_size = (1u << 20) / (uint32_t)(E / groups) + 1;
  a.softmax = score == QGEMV_SOFTMAX;
  a.renormalise = renormalise != 0;
  a.scale = scale;
  return qgemv::launch_route(a, reinterpret_cast<hipStream_t>(stream));
}

int64_t qgemv_adapt_workspace(int T, int r) {
  if (T < 0 || r < 8 || r % 8) return QGEMV_EINVAL;
  if (r > QGEMV_MAX_RANK) return QGEMV_EUNSUPPORTED;
  return std::max<int64_t>(16, (int64_t)4 * qgemv::kAdaptSplits * std::min(T, qgemv::kAdaptRows) * r);
}

int qgemv_adapt(const float *y, int64_t y_row, float *out, int64_t out_row, const void *x, int64_t x_row,
                const void *a, const void *b, int dtype, const int32_t *adapter, const float *scales, int T, int n,
                int r, int K, int N, void *workspace, int64_t workspace_bytes, void *stream) {
  if (dtype != QGEMV_BF16 && dtype != QGEMV_F16) return QGEMV_EINVAL;
  if (T < 0 || n < 1 || r < 8 || r % 8 || K < 8 || K % 8 || N < 1) return QGEMV_EINVAL;
  if (r > QGEMV_MAX_RANK || K > QGEMV_MAX_K || N > QGEMV_MAX_N) return QGEMV_EUNSUPPORTED;
  if (!y || !out || !x || !a || !b || !adapter || !workspace) return QGEMV_EINVAL;
  if (y_row < N || out_row < N || x_row < K) return QGEMV_EINVAL;
  if (!aligned(y, 4) || !aligned(out, 4) || !aligned(x, 16) || x_row % 8 || !aligned(a, 16) || !aligned(b, 16) ||
      !aligned(adapter, 4) || !aligned(scales, 4) || !aligned(workspace, 16))
    return QGEMV_EALIGN;
  if (out == y ? out_row != y_row
               : overlap(y, extent(T, y_row, 1, 0, N, 4), out, extent(T, out_row, 1, 0, N, 4)) &&
                     !(y_row == out_row && columns_apart(y, 4 * (int64_t)N, out, 4 * (int64_t)N, 4 * y_row)))
    return QGEMV_EINVAL;
  if (workspace_bytes < qgemv_adapt_workspace(T, r)) return QGEMV_EINVAL;
  if (T > kMaxWorkgroups) return QGEMV_EUNSUPPORTED;
  // The kernels look for the rows of an adapter among kAdaptRows at a time.
  for (int t = 0; t < T; t += qgemv::kAdaptRows) {
    qgemv::AdaptArgs p;
    p.y = y + t * y_row;
    p.out = out + t * out_row;
    p.x = static_cast<const uint8_t *>(x) + 2 * t * x_row;
    p.a = static_cast<const uint8_t *>(a);
    p.b = static_cast<const uint8_t *>(b);
    p.adapter = adapter + t;
    p.scales = scales;
    p.part = static_cast<float *>(workspace);
    p.y_row = y_row;
    p.out_row = out_row;
    p.x_row = x_row;
    p.T = std::min(T - t, qgemv::kAdaptRows);
    p.n = n;
    p.r = r;
    p.K = K;
    p.N = N;
    p.dtype = dtype;
    qgemv::plan_adapt(&p);
    const int s = qgemv::launch_adapt(p, reinterpret_cast<hipStream_t>(stream));
    if (s != QGEMV_OK) return s;
  }
  return QGEMV_OK;
}

int64_t qgemv_verify_drafts_workspace(int B, int V) {
  if (B < 1 || V < 1 || V > QGEMV_MAX_VOCABULARY) return QGEMV_EINVAL;
  if (B > kMaxWorkgroups) return QGEMV_EUNSUPPORTED;
  VerifyArgs a;
  a.B = B;
  a.V = V;
  return qgemv::plan_verify(&a, nullptr);
}

int qgemv_verify_drafts(const void *p, int64_t p_row, const void *q, int64_t q_row, int dtype,
                        const int32_t *tokens, const float *u, const int32_t *start, int32_t *out,
                        int32_t *count, int B, int T, int M, int V, void *workspace,
                        int64_t workspace_bytes, void *stream) {
  if (dtype != QGEMV_F32 && dtype != QGEMV_BF16 && dtype != QGEMV_F16) return QGEMV_EINVAL;
  if (B < 1 || V < 1 || V > QGEMV_MAX_VOCABULARY || T < 0 || M < 1 || M > QGEMV_MAX_M) return QGEMV_EINVAL;
  if (B > kMaxWorkgroups) return QGEMV_EUNSUPPORTED;
  if (!p || !tokens || !u || !start || !out || !count || !workspace) return QGEMV_EINVAL;
  if (p_row < V || (q && q_row < V)) return QGEMV_EINVAL;
  const uintptr_t b = (uintptr_t)elem_bytes(dtype);
  if (!aligned(p, b) || !aligned(q, b) || !aligned(tokens, 4) || !aligned(u, 4) || !aligned(start, 4) ||
      !aligned(out, 4) || !aligned(count, 4) || !aligned(workspace, 16))
    return QGEMV_EALIGN;
  VerifyArgs a;
  a.p = static_cast<const uint8_t *>(p);
  a.q = static_cast<const uint8_t *>(q);
  a.p_row = p_row;
  a.q_row = q_row;
  a.tokens = tokens;
  a.u = u;
  a.start = start;
  a.out = out;
  a.count = count;
  a.B = B;
  a.T = T;
  a.M = M;
  a.V = V;
  a.dtype = dtype;
  if (qgemv::plan_verify(&a, workspace) > workspace_bytes) return QGEMV_EINVAL;
  return qgemv::launch_verify(a, reinterpret_cast<hipStream_t>(stream));
}

}  // extern "C"
