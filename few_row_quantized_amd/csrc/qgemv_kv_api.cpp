// C ABI of the verify step's cache append, attention and draft acceptance:
// argument validation and launch (contracts in include/qgemv.h).

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
  a.window = a.sinks = 0;  // the most that any window needs
  // Fewer rows can need more (other tiles a wave, items shared where M rows are
  // walked whole): what the call of any M up to this one needs.
  int64_t most = 0;
  for (a.M = 1; a.M <= M; ++a.M) {
    const int64_t need = qgemv::plan_attend(&a, nullptr);
    if (need < 0) return need;
    most = std::max(most, need);
  }
  return most;
}

int qgemv_kv_attend(const qgemv_kv_cache *cache, const void *q, int64_t q_row, int64_t q_head,
                    void *out, int64_t out_row, int64_t out_head, int q_dtype, float *lse,
                    const int32_t *start, const int32_t *len, int T, int M, int q_heads, int window,
                    int sinks, float scale, void *workspace, int64_t workspace_bytes, void *stream) {
  AttendArgs a;
  int s = view_of(cache, &a.c);
  if (s != QGEMV_OK) return s;
  if ((s = attend_shape(cache, M, q_heads, T)) != QGEMV_OK) return s;
  if (q_dtype != QGEMV_BF16 && q_dtype != QGEMV_F16) return QGEMV_EINVAL;
  if (a.c.dtype != QGEMV_E4M3 && a.c.dtype != q_dtype) return QGEMV_EINVAL;
  if (window < 0 || sinks < 0) return QGEMV_EINVAL;
  if ((s = rows_status(start, len, T)) != QGEMV_OK) return s;
  if ((s = operand_status(q, q_row, q_head, a.c.D, q_dtype)) != QGEMV_OK) return s;
  if ((s = operand_status(out, out_row, out_head, a.c.D, q_dtype)) != QGEMV_OK) return s;
  if (!workspace) return QGEMV_EINVAL;
  if (!aligned(lse, 4) || !aligned(workspace, 16)) return QGEMV_EALIGN;
  a.q = static_cast<const uint8_t *>(q);
  a.out = static_cast<uint8_t *>(out);
  a.lse = lse;
  a.start = start;
  a.len = len;
  a.q_row = q_row * 2;
  a.q_head = q_head * 2;
  a.out_row = out_row * 2;
  a.out_head = out_head * 2;
  a.B = cache->batch;
  a.T = T;
  a.M = M;
  a.G = q_heads / cache->heads;
  // no position reaches QGEMV_MAX_CONTEXT, so a wider window sees the same
  a.window = window < QGEMV_MAX_CONTEXT ? window : QGEMV_MAX_CONTEXT;
  a.sinks = sinks;
  a.q_dtype = q_dtype;
  a.scale = scale;
  const int64_t need = qgemv::plan_attend(&a, workspace);
  if (need < 0) return (int)need;
  if (need > workspace_bytes) return QGEMV_EINVAL;
  if (T == 0) return QGEMV_OK;
  return qgemv::launch_attend(a, reinterpret_cast<hipStream_t>(stream));
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
