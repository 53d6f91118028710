// Attention: the launch of a call (kernels in qgemv_attend_impl.h).

#include <algorithm>

#include "qgemv_prefix_impl.h"

namespace qgemv {

int launch_attend_bf16(const AttendArgs &a, hipStream_t stream);
int launch_attend_f16(const AttendArgs &a, hipStream_t stream);
int launch_attend_bf16_e4m3(const AttendArgs &a, hipStream_t stream);
int launch_attend_f16_e4m3(const AttendArgs &a, hipStream_t stream);

int launch_shared_bf16(const AttendArgs &a, hipStream_t stream);
int launch_shared_f16(const AttendArgs &a, hipStream_t stream);
int launch_shared_bf16_e4m3(const AttendArgs &a, hipStream_t stream);
int launch_shared_f16_e4m3(const AttendArgs &a, hipStream_t stream);

int64_t plan_attend(AttendArgs *a, void *work, bool after_prefix) {
  const int D = a->c.D, R = a->M * a->G;
  const bool f8 = a->c.dtype == QGEMV_E4M3;
  // The longest item that the table and the window allow, in tiles: lengths are
  // on the device, so a table wider than its sequences costs calls on short ones
  // the shared form (one of 200 tokens: 6.9 us, with a table for 32768 9.6; 16 of
  // 300..1000, 30 rows: 19.0 and 22.3).
  int64_t tiles = ((int64_t)a->c.page * a->c.width + 31) / 32;
  if (a->window)
    tiles = std::min(tiles, ((int64_t)a->window + a->M + 30) / 32 + 1 + ((int64_t)a->sinks + 31) / 32);
  // Up to 64 rows of an item (32 at D = 256, whose output takes twice the
  // registers) are one wave's, and the four waves of a workgroup share the
  // tokens.  More are split over the four waves, which share the loads; so are
  // 49 to 64 at D = 128 and 16 bits where no wave has more than one tile, since
  // such a wave has the CU's registers for itself (64 rows, 4 heads, up to 85 and
  // up to 128 tokens: 8 sequences 13.0 -> 7.0 and 13.1 -> 8.2 us, 95 of them 26.5
  // -> 10.9 and 27.3 -> 12.3; of 110..160 tokens, where the rule ends, 16.7 and
  // 12.3 for 8, but 16.9 and 21.0 for 32, and 32.0 and 13.3 for 95).
  // (After a common prefix and at D = 128: 48, what two workgroups a CU hold.)
  const int rt_max = D == 256 ? 2 : after_prefix && D == 128 ? 3 : 4;
  a->shared = R > rt_max * 16 || (R > 48 && D == 128 && !f8 && tiles <= 4);
  a->group_magic = (65536 + a->G - 1) / a->G;
  const int waves = a->shared ? 4 : 1, tw = 4 / waves;
  const int groups = (R + waves * rt_max * 16 - 1) / (waves * rt_max * 16);
  a->rt = (R + groups * waves * 16 - 1) / (groups * waves * 16);
  const int item_rows = waves * a->rt * 16;
  const int64_t granules = (tiles + tw - 1) / tw;
  const int64_t items = (int64_t)a->B * a->c.H * groups;
  const int occupancy = after_prefix && D < 256 ? 2 : attend_occupancy(f8, D, a->rt, a->shared);
  const int64_t most = (int64_t)occupancy * device_cu_count();
  // Whether items are shared by workgroups, or walked by one each: without parts
  // and a second kernel, and given out as workgroups end.  They are not where
  // they are short, up to 4 granules (16 sequences of 100..200 tokens, 6 rows, 8
  // heads: 11.4 -> 8.1 us), or up to 32 tiles with items for a quarter of the
  // workgroups that run at once (of 300..1000 tokens, 30 rows: 16 sequences 22.2
  // -> 20.2, 64 of them 49.7 -> 39.5; 8, below the quarter: 18.5 and 18.8), or up
  // to 64 with items for half of them and parts of more than 16 rows (of
  // 500..2000: 48 rows, 32 sequences 54.5 -> 42.8; 30 rows, 16 sequences, below
  // the half: 30.5 and 32.0; 6 rows, 128 sequences: 122 and 128).
  const int64_t walked = granules * tw;
  // After a common prefix all items have something to be joined with.
  a->joins = after_prefix || (granules > 4 && !(walked <= 32 && items * 4 >= most) &&
             !(walked <= 64 && !a->shared && a->rt > 1 && items * 2 >= most));
  a->span = a->joins ? 1 : (int)granules;
  // counted in 32 bits on the device, and threads of a grid on the host
  if (items * granules >= (1 << 30) || items >= (1 << 24)) return QGEMV_EUNSUPPORTED;
  a->seq_items = a->c.H * groups;
  a->workgroups = (int)(a->joins ? std::min(most, items * granules) : items);
  // ranks: workgroups of a CU, where all of them run
  a->ranks = a->joins && a->workgroups == most && !(after_prefix && D < 256) ? occupancy : 1;
  a->rank_size = a->workgroups / a->ranks;
  page_magic(a->rank_size, &a->rank_magic, &a->rank_shift);
  a->row_splits = (int)std::max<int64_t>(1, std::min<int64_t>(std::min(item_rows, R), 1024 / items));
  // workspace: the plan, maxima and sums, parts
  const auto up = [](int64_t n) { return (n + 255) & ~(int64_t)255; };
  const int64_t plan_bytes = a->joins ? up(4 * ((int64_t)a->B + 2)) : 256, parts = a->joins ? (2 * most + (after_prefix ? items : 0)) * item_rows : 0;
  uint8_t *p = static_cast<uint8_t *>(work);
  a->plan = reinterpret_cast<int32_t *>(p);
  a->ml = reinterpret_cast<float *>(p + plan_bytes);
  a->part = reinterpret_cast<float *>(p + plan_bytes + up(8 * parts));
  if (after_prefix) a->grid = (int)std::min(most, (int64_t)a->pre_workgroups + a->workgroups);
  return plan_bytes + up(8 * parts) + 4 * parts * D;
}

int64_t plan_prefix(AttendArgs *a, void *work) {
  const int D = a->c.D, tokens = kPrefixTokens;
  const int64_t rows = (int64_t)a->T * a->G;
  a->pre_rows = kPrefixRows;
  const int64_t tiles = (rows + a->pre_rows - 1) / a->pre_rows;
  const int64_t items = tiles * a->c.H;
  // what the table can have in common: all of it but each sequence's last page
  const int64_t granules = std::max<int64_t>(1, ((int64_t)a->c.page * (a->c.width - 1) + tokens - 1) / tokens);
  // counted in 32 bits on the device
  if (rows >= (1 << 30) || items * granules >= (1 << 30)) return QGEMV_EUNSUPPORTED;
  const int64_t slots = (int64_t)prefix_occupancy(D) * device_cu_count();
  int64_t workgroups = std::max<int64_t>(1, std::min(slots, items * granules));
  if (workgroups > 8) workgroups &= ~(int64_t)7;  // as many on each XCD
  a->pre_tiles = (int)tiles;
  a->pre_workgroups = (int)workgroups;
  a->pre_most = items ? (int)(workgroups / items) + 2 : 0;
  const auto up = [](int64_t n) { return (n + 255) & ~(int64_t)255; };
  // items * pre_most is at most workgroups + 2 items: so much in units that grow
  // with T, whatever rows the call takes together
  const int64_t parts = (2 * (int64_t)device_cu_count() + 2 * items) * a->pre_rows;
  uint8_t *p = static_cast<uint8_t *>(work);
  a->pre_plan = reinterpret_cast<int32_t *>(p);
  a->pre_ml = reinterpret_cast<float *>(p + 256);
  a->pre_part = reinterpret_cast<float *>(p + 256 + up(8 * parts));
  return 256 + up(8 * parts) + 4 * parts * D;
}

int launch_attend_shared(const AttendArgs &a, hipStream_t stream) {
  const bool f8 = a.c.dtype == QGEMV_E4M3;
  if (a.q_dtype == QGEMV_BF16) return f8 ? launch_shared_bf16_e4m3(a, stream) : launch_shared_bf16(a, stream);
  return f8 ? launch_shared_f16_e4m3(a, stream) : launch_shared_f16(a, stream);
}

int launch_attend(const AttendArgs &a, hipStream_t stream) {
  const bool f8 = a.c.dtype == QGEMV_E4M3;
  if (a.q_dtype == QGEMV_BF16) return f8 ? launch_attend_bf16_e4m3(a, stream) : launch_attend_bf16(a, stream);
  return f8 ? launch_attend_f16_e4m3(a, stream) : launch_attend_f16(a, stream);
}

}  // namespace qgemv
