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
  // attention over a common prefix (qgemv_prefix_impl.h)
  const int32_t *common;  // its tokens, or null
  int32_t *pre_plan;      // granules of an item, granules of a workgroup
  float *pre_ml;          // [items][pre_most][pre_rows][2]
  float *pre_part;        // [items][pre_most][pre_rows][D]
  int pre_rows;           // rows of an item
  int pre_tiles;          // items of a head: groups of so many rows of all
  int pre_workgroups, pre_most;
  int grid;               // of the launch that has both
};

struct RotateArgs {
  AppendArgs rows;
  const uint8_t *q;
  uint8_t *out;
  int64_t q_row, q_head, out_row, out_head;  // bytes
  const float *freq;        // [pairs]
  const int32_t *position;  // [axes][T], or null: the row's place in the cache
  const int32_t *axis;      // [pairs], or null: the first
  int64_t position_axis;    // elements between axes
  int q_heads, out_dtype, pairs, axes;
  bool interleaved;
};

struct RouteArgs {
  const uint8_t *logits;
  int64_t row;        // elements
  const float *bias;  // [E], or null
  int32_t *experts;   // [T][k]
  float *weights;     // [T][k]
  int T, E, k, dtype, groups, keep, best;
  uint32_t over_size;  // floor(2^20 / (E / groups)) + 1: e * over_size >> 20 is e's group
  bool softmax, renormalise;
  float scale;
};

struct AdaptArgs {
  const float *y;
  float *out;
  const uint8_t *x, *a, *b;
  const int32_t *adapter;
  const float *scales;  // [n], or null
  float *part;          // [splits][T][r]: sums of the first product
  int64_t y_row, out_row, x_row;  // elements
  int T, n, r, K, N, dtype;
  int tiles;   // of rows: the most there can be
  int splits;  // of K
  int rt;      // 16-row tiles of a tile of rows
  int rk;      // 16-rank tiles of a wave of the first product
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
int64_t plan_attend(AttendArgs *a, void *work, bool after_prefix = false);
int launch_attend(const AttendArgs &a, hipStream_t stream);
// The same for the part of the common tokens, which with plan_attend(.., true)
// makes a call of launch_attend_shared; the size grows with T.
int64_t plan_prefix(AttendArgs *a, void *work);
int launch_attend_shared(const AttendArgs &a, hipStream_t stream);
int launch_rotate(const RotateArgs &a, hipStream_t stream);
int launch_route(const RouteArgs &a, hipStream_t stream);
// Fills in the launch (tiles, splits, rt) for up to kAdaptRows rows, and returns
// the workspace's size in bytes.
constexpr int kAdaptRows = 512, kAdaptSplits = 8;
int64_t plan_adapt(AdaptArgs *a);
int launch_adapt(const AdaptArgs &a, hipStream_t stream);
int64_t plan_verify(VerifyArgs *a, void *work);  // slices and workspace alike
int launch_verify(const VerifyArgs &a, hipStream_t stream);

}  // namespace qgemv
