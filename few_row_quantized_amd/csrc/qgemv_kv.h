// Shared by the kernels of the verify step's cache operators: the arguments,
// the page lookup and the per-sequence geometry.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qgemv_internal.h"

namespace qgemv {

// A paged cache as the kernels see it.  Strides are in bytes and shared by
// keys and values; slot s of page p of head h starts at
// p * stride_page + s * stride_slot + h * stride_head.
struct KvView {
  uint8_t *k, *v;
  const int32_t *table;  // [B][width] page ids
  const float *k_scale, *v_scale;  // [H], or null
  int64_t stride_page, stride_slot, stride_head;
  int pages, page, width, H, D, dtype;
  uint32_t magic;  // token / page = (2 token * magic) >> (32 + shift) for token < 2^30
  int shift;
};

// ceil(2^(31 + L) / d) with L = ceil(log2 d): the quotient by an invariant
// divisor as one multiplication and a shift by 31 + L, exact for every
// dividend below 2^31.
inline void page_magic(int d, uint32_t *magic, int *shift) {
  int L = 0;
  while ((1ll << L) < d) ++L;
  *magic = (uint32_t)(((1ull << (31 + L)) + (uint64_t)d - 1) / (uint64_t)d);
  *shift = L;
}

__device__ __forceinline__ int page_of(const KvView &c, int token) {
  return (int)(__umulhi(c.magic, 2u * (uint32_t)token) >> c.shift);
}

struct AppendArgs {
  KvView c;
  const uint8_t *nk, *nv;
  int64_t k_row, k_head, v_row, v_head;  // bytes
  const int32_t *start, *len;
  int B, T, src;
};

struct AttendArgs {
  KvView c;
  const uint8_t *q;
  uint8_t *out;
  float *lse;  // [T][Hq], or null
  const int32_t *start, *len;
  int32_t *plan;  // [0]: granules of all; [1 + b]: granules before sequence b
  float *ml;      // [2 * workgroups][rows of an item][2]: maximum and sum of a part
  float *part;    // [2 * workgroups][rows of an item][D]: its sums
  int64_t q_row, q_head, out_row, out_head;  // bytes
  int B, T, M, G, window, sinks, q_dtype;
  float scale;
  bool shared;     // the four waves split the rows and share the tokens' loads
  int rt;          // 16-row tiles of a wave
  int group_magic; // row / G = row * group_magic >> 16 for row < 1024, G <= 64
  int workgroups;  // of the main kernel
  int ranks;       // of them, one for each workgroup of a CU
  int rank_size;   // workgroups of a rank, and the division by them
  uint32_t rank_magic;
  int rank_shift;
  int span;        // tiles of a wave in a granule
  int row_splits;  // workgroups of the join for one item
  int seq_items;   // items of a sequence of M rows
  bool joins;      // whether an item can lie in more than one workgroup
};

struct VerifyArgs {
  const uint8_t *p, *q;  // q null: drafts without probabilities
  int64_t p_row, q_row;  // elements
  const int32_t *tokens;
  const float *u;
  const int32_t *start;
  int32_t *out, *count;
  double *sums;       // [B][pieces][2]: of what is left, of p
  int32_t *arrived;   // one for each sequence, where slices > 1
  int B, T, M, V, dtype;
  int per, pieces;    // tokens of a piece, pieces of a row
  int each, slices;   // pieces of a wave, workgroups of a sequence
};

int launch_append(const AppendArgs &a, hipStream_t stream);
// Fills in the launch (shared .. joins) and the workspace's layout from
// `work`, and returns its size in bytes.
int64_t plan_attend(AttendArgs *a, void *work);
int launch_attend(const AttendArgs &a, hipStream_t stream);
int64_t plan_verify(VerifyArgs *a, void *work);  // slices and workspace alike
int launch_verify(const VerifyArgs &a, hipStream_t stream);

}  // namespace qgemv
