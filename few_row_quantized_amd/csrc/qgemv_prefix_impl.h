// Attention of all sequences' rows over the tokens that they have in common.
//
// A batch whose sequences begin with the same pages reads them once: the rows
// of all sequences, R = T G of them for a key-value head, are one product against
// the common tokens,
//
//   m = max_j s_j,  l = sum_j 2^(s_j - m),  o = sum_j 2^(s_j - m) v_j,
//   s_j = scale * k_scale[h] * log2(e) * (q . k_j),
//
// which is joined with what each sequence's own tokens give (qgemv_attend_impl.h,
// PRE).  4 R D flops for 4 D bytes of a token's keys and values, R in the hundreds
// or thousands: the matrix units bound it, not the memory.
//
// A workgroup has 128 rows of a head, 32 a wave, and goes over granules of 64
// tokens.  Scores are taken as S^T = K Q^T, which leaves a query row in a lane, so
// that its maximum, its sum and its weights need no exchange but one with the lane
// 32 away, and the weights are in registers as the second product, O^T = V^T P^T,
// wants them; the queries stay in registers too.  Keys and values go through the
// LDS, once for four waves.
//
// 64 sequences of up to 8 rows, 8 heads of 6 query heads over 16384 common tokens
// of D = 128 and 500..2000 of their own, bf16: 304 us, where 190 GFLOP at the rate
// of a product of 16384^3 would take 137.  What bounds it is waiting between two
// products, for the LDS and for exponentials, with two waves of a SIMD: 256
// registers of each hold 64 sums, 32 scores and 32 queries.  Without the
// exponentials, the reads of the LDS or the loads, each by itself, it would take
// less than a tenth off.
#pragma once

#include <type_traits>

#include "qgemv_attend_impl.h"

namespace qgemv {

template <int N>
using Const = std::integral_constant<int, N>;

typedef float f32x16_t __attribute__((ext_vector_type(16)));

template <bool BF>
__device__ __forceinline__ f32x16_t mfma_32x32x16(u32x4_t a, u32x4_t b, f32x16_t c) {
  if constexpr (BF)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b),
                                                   c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c,
                                                  0, 0, 0);
}

// Maximum / sum over the two lanes of a query row (lanes c and c + 32).
__device__ __forceinline__ float pair_max(float x) {
  const auto a = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x),
                                                  false, false);
  return fmaxf(__builtin_bit_cast(float, (uint32_t)a[0]), __builtin_bit_cast(float, (uint32_t)a[1]));
}
__device__ __forceinline__ float pair_sum(float x) {
  const auto a = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x),
                                                  false, false);
  return __builtin_bit_cast(float, (uint32_t)a[0]) + __builtin_bit_cast(float, (uint32_t)a[1]);
}

// The smallest of a wave's values, in all lanes.
__device__ __forceinline__ int wave_least(int x) {
  x = min(x, __builtin_amdgcn_update_dpp(x, x, 0x111, 0xF, 0xF, false));
  x = min(x, __builtin_amdgcn_update_dpp(x, x, 0x112, 0xF, 0xF, false));
  x = min(x, __builtin_amdgcn_update_dpp(x, x, 0x114, 0xF, 0xF, false));
  x = min(x, __builtin_amdgcn_update_dpp(x, x, 0x118, 0xF, 0xF, false));
  x = min(x, __builtin_amdgcn_update_dpp(x, x, 0x142, 0xA, 0xF, false));
  x = min(x, __builtin_amdgcn_update_dpp(x, x, 0x143, 0xC, 0xF, false));
  return __builtin_amdgcn_readlane(x, 63);
}

constexpr int kPrefixRows = 128;   // of an item: 32 a wave
constexpr int kPrefixTokens = 64;  // of a granule
constexpr int prefix_occupancy(int D) { return D == 256 ? 1 : 2; }  // workgroups of a CU

// LDS of a workgroup: positions of the rows and the reductions, then keys of two
// tiles and values of two.  Rows are padded, so that lanes of consecutive tokens
// that read one chunk of 16 bytes each (keys), or 64 bytes of 4 tokens (values),
// find them in different banks, at distances that a load's offset can hold.
constexpr int kPrefixHead = 1024 + 4096;  // the latter: each wave's places of two tiles' tokens
constexpr int key_row(int D) { return 2 * D + 16; }
constexpr int value_row(int D) { return 2 * D + 64; }
constexpr size_t prefix_lds(int D) { return kPrefixHead + (size_t)2 * kPrefixTokens * (key_row(D) + value_row(D)); }

// 16-bit caches at D = 128 are loaded straight to the LDS, 4 tokens and 1 KiB an
// instruction, so rows lie together in fours with 16 bytes after them, and a row's
// quarters of 64 bytes are exchanged by the token's place in its four: lanes read
// different banks as above.  (The case above, through registers 314, so 306 us; a head of D = 128 over
// 64 sequences of 1 row 46.6 and 43.1.)  E4M3 passes registers, where it is widened.
// So do rows of D = 64 and D = 256: what they would gain was not measured, and their
// fours do not fill an instruction's 1 KiB, so that the layout would be another.
constexpr int kFour = 4 * 256 + 16;

// Operands of four matrix instructions, 8 tokens of one d a lane, out of rows of
// values in the LDS: each of the reads turns 4 tokens by 16 d.  All are on their way
// together, and waited for here: as builtins they were each waited for on their
// own, and for loads from the memory to the LDS as well.
template <int OFFSET, int EIGHT>
__device__ __forceinline__ void read_turned(uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, u32x4_t *to) {
  uint64_t x0, y0, x1, y1, x2, y2, x3, y3;
  asm volatile(
      "ds_read_b64_tr_b16 %0, %8 offset:%12\n\t"
      "ds_read_b64_tr_b16 %1, %8 offset:%13\n\t"
      "ds_read_b64_tr_b16 %2, %9 offset:%12\n\t"
      "ds_read_b64_tr_b16 %3, %9 offset:%13\n\t"
      "ds_read_b64_tr_b16 %4, %10 offset:%12\n\t"
      "ds_read_b64_tr_b16 %5, %10 offset:%13\n\t"
      "ds_read_b64_tr_b16 %6, %11 offset:%12\n\t"
      "ds_read_b64_tr_b16 %7, %11 offset:%13\n\t"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(x0), "=&v"(y0), "=&v"(x1), "=&v"(y1), "=&v"(x2), "=&v"(y2), "=&v"(x3), "=&v"(y3)
      : "v"(a0), "v"(a1), "v"(a2), "v"(a3), "i"(OFFSET), "i"(OFFSET + EIGHT)
      : "memory");
  to[0] = u32x4_t{(uint32_t)x0, (uint32_t)(x0 >> 32), (uint32_t)y0, (uint32_t)(y0 >> 32)};
  to[1] = u32x4_t{(uint32_t)x1, (uint32_t)(x1 >> 32), (uint32_t)y1, (uint32_t)(y1 >> 32)};
  to[2] = u32x4_t{(uint32_t)x2, (uint32_t)(x2 >> 32), (uint32_t)y2, (uint32_t)(y2 >> 32)};
  to[3] = u32x4_t{(uint32_t)x3, (uint32_t)(x3 >> 32), (uint32_t)y3, (uint32_t)(y3 >> 32)};
}

// The first token that a row's window can reach: of the sequence with the lowest
// position.  (The workgroup's threads together; 4 words of LDS.)
template <class Args>
__device__ __forceinline__ int lowest_token(Args &a, int before, int *lds) {
  if (!a.window) return 0;
  int least = 0x7FFFFFFF;
  for (int b = threadIdx.x; b < a.B; b += 256) {
    const int s0 = min(max(a.start[b], 0), a.T), s1 = min(max(a.start[b + 1], s0), a.T);
    const int len = min(max(a.len[b], 0), QGEMV_MAX_CONTEXT);
    if (s1 > s0) least = min(least, len - (s1 - s0));
  }
  lds[threadIdx.x >> 6] = wave_least(least);
  __syncthreads();
  least = min(min(lds[0], lds[1]), min(lds[2], lds[3]));
  return __builtin_amdgcn_readfirstlane(min(max(least - a.window + 1, 0), before));
}

// What workgroups spend, in common granules (us of the cases that change most):
// a granule of own tokens, in halves (1, 2, 3: 64 sequences of 4 rows over 6000
// tokens of E4M3 and 0..2500 of their own 137, 104, 106; 16 of 16 rows, D = 64,
// window 4096, 65, 62, 67);
constexpr int kOwnCost = 2;
// an item's start and end, in halves (0, 2, 4, 8: 64 of 8 rows over 4000 and
// 25..100 of their own 211, 124, 99, 95; 24 of 4 over 6001 of E4M3 and 0..2500
// 69, 69, 68, 75);
constexpr int kItemCost = 4;
// a second item in a range (with ranges always within an item, with ranges always
// equal, with this: 32 of 4 rows, window 1024, 44, 51, 44; 64 of 8 over 16000 and
// 25..100 237, 243, 237; for none but equal costs, 0: 244);
constexpr int kRangeCost = 2;
// and the walk of a workgroup from which both are long (32 and 72 as 48 within 1 %
// but for 64 of 8 over 4000 and 500..2000: 141, 136, 137).
constexpr int kLongWalk = 48;

// What the sequences' own tokens cost, in halves of a common granule.
template <class Args>
__device__ __forceinline__ int64_t own_cost(Args &a, int before, int *lds) {
  uint32_t sum = 0;  // below 2^32 with 2^30 granules and 2^24 items
  for (int b = threadIdx.x; b < a.B; b += 256) {
    const SeqWork w = seq_work<true>(a, b, before);
    sum += (uint32_t)w.items * ((uint32_t)w.granules * kOwnCost + kItemCost);
  }
  sum += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)sum, 0x111, 0xF, 0xF, false);
  sum += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)sum, 0x112, 0xF, 0xF, false);
  sum += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)sum, 0x114, 0xF, 0xF, false);
  sum += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)sum, 0x118, 0xF, 0xF, false);
  sum += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)sum, 0x142, 0xA, 0xF, false);
  sum += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)sum, 0x143, 0xC, 0xF, false);
  lds[threadIdx.x >> 6] = (int)__builtin_amdgcn_readlane(sum, 63);
  __syncthreads();
  return (uint32_t)__builtin_amdgcn_readfirstlane(lds[0] + lds[1] + lds[2] + lds[3]);
}

template <bool BF, bool F8, int D>
__device__ __forceinline__ void prefix_body(KernArgs *ap, uint8_t *const lds, const int index, const int workgroups) {
  constexpr int TOK = kPrefixTokens, C = D / 8, DB = D / 32, QS = D / 16;
  constexpr int L = TOK * C / 256;  // chunks of a thread, of keys and of values
  constexpr bool DIRECT = D == 128 && !F8;
  constexpr int KR = key_row(D), VR = value_row(D);
  constexpr int KT = DIRECT ? TOK / 4 * kFour : TOK * KR, VT = DIRECT ? TOK / 4 * kFour : TOK * VR;  // bytes of a tile
  // Exponentials placed between matrix instructions by hand, part by part: left to
  // itself the compiler takes registers past the limit at D = 128 (queries spilled,
  // each reload a wait for all loads in flight); at D = 64, where there are enough,
  // its own order is better (a window of 4096, 16 rows: 60 us, 65 by hand).
  constexpr bool ORDER = D == 128;
  constexpr int CB = F8 ? 1 : 2;
  int *const row_pos = reinterpret_cast<int *>(lds);        // [128] rows of T
  int *const bounds = reinterpret_cast<int *>(lds + 512);   // of each wave: smallest end, largest begin; then strays
  int64_t *const ring = reinterpret_cast<int64_t *>(lds + 1024) + (threadIdx.x >> 6) * 128;
  uint8_t *const keys = lds + kPrefixHead, *const values = keys + 2 * KT;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 31, half = lane >> 5;
  const int common = common_pages<true>(*ap), before = common * ap->c.page;
  const int G = ap->G, T = ap->T, R = T * G, B = ap->B;
  const int window = ap->window ? ap->window : 1 << 30, sinks = ap->sinks;

  const int low = lowest_token(*ap, before, bounds);
  const int all = (before + TOK - 1) / TOK, low_tile = low / TOK;
  const int sink_tiles = ap->window ? min((int)(((int64_t)sinks + TOK - 1) / TOK), low_tile) : 0;
  const int n = sink_tiles + all - low_tile;
  const int items = ap->pre_tiles * ap->c.H;
  // Equal ranges of all items' granules; or as many workgroups for each item, so
  // that none walks parts of two, where that makes ranges longer by less than a
  // second start and end cost.
  const int parts = (int)((uint32_t)workgroups / (uint32_t)items);
  int per = max((items * n + workgroups - 1) / workgroups, 1), padded = n;
  if (parts && n && (n + parts - 1) / parts <= per + kRangeCost) {
    per = (n + parts - 1) / parts;
    padded = (n + per - 1) / per * per;
  }
  const int total = items * padded;
  if (index == 0 && tid == 0) {
    ap->pre_plan[0] = padded;
    ap->pre_plan[1] = per;
  }
  if (index >= workgroups) return;
  // Workgroups of an XCD, which share its L2, walk neighbouring ranges.
  int wg = index;
  if (workgroups % 8 == 0) wg = (wg & 7) * (workgroups >> 3) + (wg >> 3);
  int cur = wg * per;
  const int end = min(cur + per, total);

  while (cur < end) {
    const int item = (int)((uint32_t)cur / (uint32_t)padded), first = cur - item * padded;
    const int count = min(n - first, end - cur);
    cur += min(padded - first, end - cur);
    const int h = (int)((uint32_t)item / (uint32_t)ap->pre_tiles), tile0 = item - h * ap->pre_tiles;
    const int r0 = tile0 * kPrefixRows, row = r0 + wave * 32 + c;

    const uint8_t *const kbase = ap->c.k + h * ap->c.stride_head;
    const uint8_t *const vbase = ap->c.v + h * ap->c.stride_head;
    const int32_t *const table = ap->c.table;
    const int64_t stride_page = ap->c.stride_page, stride_slot = ap->c.stride_slot;
    const int page = ap->c.page, pages = ap->c.pages, shift = ap->c.shift;
    const uint32_t magic = ap->c.magic;
    const float signed_sc = ap->scale * (ap->c.k_scale ? constant(ap->c.k_scale)[h] : 1.0f) * kLog2e;

    // ---- the first tiles' page ids and the queries, on their way while the
    // rows' positions are found.  The queries take the scale's sign (and are 0
    // where it is 0, with a NaN where one is not finite), so that the largest
    // product has the largest score.
    auto tile_base = [&](int tile) { return (tile < sink_tiles ? tile : tile - sink_tiles + low_tile) * TOK; };
    // the page id of a lane's token
    auto load_id = [&](int tile) -> int {
      const int token = min(tile_base(tile) + lane, max(before - 1, 0));
      return table[__umulhi(magic, 2 * token) >> shift];
    };
    int t = first;
    const int t_end = first + count;
    int id = load_id(t), id_next = load_id(t + 1);
    u32x4_t qf[QS];
    {
      const int at = min(row, R - 1), t = at / G, hq = h * G + at - t * G;
      const uint8_t *q = ap->q + (int64_t)t * ap->q_row + hq * ap->q_head;
#pragma unroll
      for (int s = 0; s < QS; ++s) qf[s] = *reinterpret_cast<const u32x4_t *>(q + (s * 16 + half * 8) * 2);
    }

    // ---- positions of the item's rows
    const int t0 = r0 / G, t1 = min((r0 + kPrefixRows - 1) / G + 1, T);
    __syncthreads();
    if (tid < 128) row_pos[tid] = 0x7FFFFFFF;  // a row of no sequence: sees what it likes, and is not read
    if (tid == 0) bounds[8] = 0;
    __syncthreads();
    for (int b = tid; b < B; b += 256) {
      const int s0 = min(max(ap->start[b], 0), T), s1 = min(max(ap->start[b + 1], s0), T);
      const int len = min(max(ap->len[b], 0), QGEMV_MAX_CONTEXT);
      for (int t = max(s0, t0); t < min(s1, t1); ++t) row_pos[t - t0] = len - (s1 - t);
    }
    __syncthreads();
    int hi = before, lo = 0;  // the row sees tokens below hi, of them those from lo on or below the sinks
    if (row < R) {
      const int pos = row_pos[row / G - t0];
      if (pos != 0x7FFFFFFF) {
        hi = min(before, pos + 1);
        lo = max(pos - window + 1, 0);
      }
    }
    bounds[wave] = wave_least(hi);
    bounds[4 + wave] = -wave_least(-lo);
    __syncthreads();
    const int least_hi = __builtin_amdgcn_readfirstlane(min(min(bounds[0], bounds[1]), min(bounds[2], bounds[3])));
    const int most_lo = __builtin_amdgcn_readfirstlane(max(max(bounds[4], bounds[5]), max(bounds[6], bounds[7])));
    const float sc = signed_sc == 0.0f ? 1.0f : __builtin_fabsf(signed_sc);
    {
      const uint32_t flip = signed_sc < 0.0f ? 0x80008000u : 0u, keep = signed_sc == 0.0f ? 0u : ~0u;
      uint32_t odd = 0;
#pragma unroll
      for (int s = 0; s < QS; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          odd |= nonfinite_signs<BF, false>(qf[s][i]);
          qf[s][i] = (qf[s][i] ^ flip) & keep;
        }
      qf[0][0] |= (odd & kSigns<false>) != 0 ? ~keep : 0u;
    }

    auto is_edge = [&](int tb, uint64_t present) {
      return (present != ~0ull) | (tb + TOK > least_hi) | ((tb < most_lo) & (tb + TOK > sinks));
    };
    // a lane's place of a tile's token into the ring, 0 where it is not there
    auto put = [&](int tile, int id) -> uint64_t {
      const int token = tile_base(tile) + lane;
      const bool ok = ((uint32_t)id < (uint32_t)pages) & (tile < first + count) & (token < before);
      const int in_page = token - (int)(__umulhi(magic, 2 * token) >> shift) * page;
      ring[(tile & 1) * 64 + lane] = ok ? id * stride_page + in_page * stride_slot : 0;
      // a wave's LDS accesses stay in order; this keeps the compiler from moving them
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      return __ballot(ok);
    };
    // A thread's share of a tile's keys, and of another's values, on their way: its
    // chunk of 8 values of every (256 / C)th token.
    u32x4_t kt[L], vt[L];
    // (What follows from the thread alone is computed anew for each tile, not kept
    // in registers.)
    auto anew = [](int x) {
      asm volatile("" : "+v"(x));
      return x;
    };
    typedef int64_t Places[L];
    auto look_up = [&](int tile, Places &to) {
      const int64_t *const from = ring + (tile & 1) * 64 + anew(tid) / C;
#pragma unroll
      for (int i = 0; i < L; ++i) to[i] = from[i * (256 / C)];
    };
    auto load_rows = [&](const uint8_t *from, const Places &at, u32x4_t (&to)[L]) {
      const int within = anew(tid) % C * (8 * CB);
#pragma unroll
      for (int i = 0; i < L; ++i) {
        const uint8_t *const p = from + at[i] + within;
        if constexpr (F8) {
          const u32x2_t x = *reinterpret_cast<const u32x2_t *>(p);
          to[i][0] = x[0];
          to[i][1] = x[1];
        } else {
          to[i] = *reinterpret_cast<const u32x4_t *>(p);
        }
      }
    };
    // the same straight to a tile's place in the LDS
    auto fetch_rows = [&](const uint8_t *from, const Places &at, uint8_t *to) {
      const int me = anew(lane), within = ((me & 15) ^ (me >> 4) * 4) * 16;
#pragma unroll
      for (int i = 0; i < L; ++i)
        __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)(from + at[i] + within),
                                         (__attribute__((address_space(3))) void *)(to + (i * 4 + wave) * kFour), 16, 0, 0);
    };
    // and the values of one that some row does not see some tokens of (as below)
    auto clean_values = [&](int tile, uint64_t present) {
      const int me = anew(tid);
      u32x4_t *const at = reinterpret_cast<u32x4_t *>(values + (tile & 1) * VT + wave * kFour + (me & 63) * 16);
      uint32_t odd = 0;
#pragma unroll
      for (int i = 0; i < L; ++i) {
        const uint32_t ok = 0u - (uint32_t)(present >> (i * 16 + me / 16) & 1);
        u32x4_t v = at[i * (4 * kFour / 16)];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          v[x] &= ok;
          odd |= nonfinite_signs<BF, false>(v[x]);
          v[x] &= ~nonfinite<BF, false>(v[x]);
        }
        at[i * (4 * kFour / 16)] = v;
      }
      if ((odd & kSigns<false>) != 0) bounds[8] = 1;
      __syncthreads();
    };
    auto widen = [](u32x4_t x) -> u32x4_t {
      if constexpr (!F8) return x;
      return u32x4_t{e4m3_pair<BF, false>(x[0]), e4m3_pair<BF, true>(x[0]), e4m3_pair<BF, false>(x[1]),
                     e4m3_pair<BF, true>(x[1])};
    };
    auto store_keys = [&](int tile, const u32x4_t (&from)[L]) {
      const int me = anew(tid);
      uint8_t *const to = keys + (tile & 1) * KT + me / C * KR + me % C * 16;
#pragma unroll
      for (int i = 0; i < L; ++i) *reinterpret_cast<u32x4_t *>(to + i * (256 / C) * KR) = widen(from[i]);
    };
    // Where some row does not see some of a tile's tokens: without the values that
    // are not there, and without NaNs and infinities (0 times one is not 0), which
    // are given to the rows that see them after the tiles.
    auto store_values = [&](int tile, bool edge, uint64_t present) {
      const int me = anew(tid);
      uint8_t *const to = values + (tile & 1) * VT + me / C * VR + me % C * 16;
      if (edge) {
        uint32_t odd = 0;
#pragma unroll
        for (int i = 0; i < L; ++i) {
          const uint32_t ok = 0u - (uint32_t)(present >> (i * (256 / C) + me / C) & 1);
          u32x4_t v = widen(vt[i]);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            v[x] &= ok;
            odd |= nonfinite_signs<BF, false>(v[x]);
            v[x] &= ~nonfinite<BF, false>(v[x]);
          }
          *reinterpret_cast<u32x4_t *>(to + i * (256 / C) * VR) = v;
        }
        if ((odd & kSigns<false>) != 0) bounds[8] = 1;
      } else {
#pragma unroll
        for (int i = 0; i < L; ++i) *reinterpret_cast<u32x4_t *>(to + i * (256 / C) * VR) = widen(vt[i]);
      }
    };

    f32x16_t acc[DB];
    float m = kNegInf, l = 0.0f;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[d][i] = 0.0f;
    // Scores of half a tile: lane (c, half) has row c, tokens 32 b + 8 (i / 4) +
    // 4 half + i % 4.
    f32x16_t s[2];
    u32x4_t p[2][2];  // their weights, as operands of the second product
    auto products = [&](int tile, int b) {
      const int me = anew(lane);
      const uint8_t *const from = keys + (tile & 1) * KT + (me >> 5) * 16 +
                                  (DIRECT ? (me & 31) / 4 * kFour + (me & 3) * 256 : (me & 31) * KR);
      const f32x16_t none = {};
#pragma unroll
      for (int st = 0; st < QS; ++st) {
        const int to = DIRECT ? b * (8 * kFour) + ((st / 2 ^ (me & 3)) * 64) + st % 2 * 32 : b * (32 * KR) + st * 32;
        s[b] = mfma_32x32x16<BF>(*reinterpret_cast<const u32x4_t *>(from + to), qf[st], st ? s[b] : none);
      }
    };
    // Weights leave fp32 for the matrix product: half a step of q's type each, as
    // in the attention over a sequence's own tokens, whose parts these are joined
    // with.  Their sum takes them in fp32 before.  That is what the output's error is
    // beside its own rounding (in norm, against 64 bits: bf16 0.0023, 0.0017 of them
    // the output's rounding alone; fp16 0.00028 and 0.00021).  A second part of the
    // weights would take that away, for half as many matrix instructions again and
    // registers that are not there.
    auto weigh = [&](int b) {
      const float mm = m == kNegInf ? 0.0f : m;
      float sum = 0.0f;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float w0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[b][u * 8 + x * 2], sc, -mm));
          const float w1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[b][u * 8 + x * 2 + 1], sc, -mm));
          sum += w0;
          sum += w1;
          p[b][u][x] = pair_of<BF>(w0, w1);
        }
      l += sum;
    };
    // Half a tile's values by their weights; a lane's operand is 8 tokens of one d,
    // turned by the LDS.
    auto add = [&](int tile, auto which) {
      constexpr int b = decltype(which)::value;
      const int me = anew(lane);
      const int place = (me & 15) / 4;  // of the token in its four
      const uint8_t *const from = values + (tile & 1) * VT + (me >> 4 & 1) * 32 + (me & 3) * 8 +
                                  (DIRECT ? (me >> 5) * kFour + place * 256 : (4 * (me >> 5) + place) * VR);
      const uint32_t at = (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t *)from;
      constexpr int FIRST = DIRECT ? b * 8 * kFour : b * 32 * VR;
      constexpr int NEXT = DIRECT ? 4 * kFour : 16 * VR, EIGHT = NEXT / 2;  // 16 tokens, 8 tokens
      auto d_at = [&](int d) { return at + (DIRECT ? (d ^ place) * 64 : d * 64); };
      if constexpr (DB == 2) {
        u32x4_t v[4];
        read_turned<FIRST, EIGHT>(d_at(0), d_at(1), d_at(0) + NEXT, d_at(1) + NEXT, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i & 1] = mfma_32x32x16<BF>(v[i], p[b][i >> 1], acc[i & 1]);
      } else {
        auto step = [&](auto part) {
          constexpr int u = decltype(part)::value;
#pragma unroll
          for (int d0 = 0; d0 < DB; d0 += 4) {
            u32x4_t v[4];
            read_turned<FIRST + u * NEXT, EIGHT>(d_at(d0), d_at(d0 + 1), d_at(d0 + 2), d_at(d0 + 3), v);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[d0 + i] = mfma_32x32x16<BF>(v[i], p[b][u], acc[d0 + i]);
          }
        };
        step(Const<0>{});
        step(Const<1>{});
      }
    };
    // Scores of a tile that have no part, and the reference of the weights.
    auto look = [&](int tile, uint64_t present) {
      const int tb = tile_base(tile);
      if (is_edge(tb, present)) {
        const int from = 4 * anew(half);  // the lane's first token
        const uint64_t mine = present >> from;
        const int j0 = tb + from;
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int o = b * 32 + 8 * (i / 4) + i % 4;
            const bool sees = ((mine >> o & 1) != 0) & (o < hi - j0) & ((o >= lo - j0) | (o < sinks - j0));
            s[b][i] = sees ? s[b][i] : kNegInf;
          }
      }
      float top = s[0][0];
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, s[b][i]);
      top = pair_max(top) * sc;
      // (a difference, which is exact: m + 8 would round where scores pass 2^25)
      if (__any(top - m > 8.0f + kHeadroom<BF>)) {
        // The reference is a whole number, and what is scaled by powers of two
        // keeps its bits: also the weights that are yet to be added up (in fp16 those
        // above 2^-14; smaller ones are rounded again, to steps of 2^-24 where the
        // largest weight is 2^7 or more).
        const float mn = fmaxf(m, __builtin_floorf(top) - kHeadroom<BF>);
        const float f = __builtin_amdgcn_ldexpf(1.0f, max((int)(m - mn), -300));
        m = mn;
        l *= f;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[d][i] *= f;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint32_t w = p[1][u][x];
            p[1][u][x] = pair_of<BF>(value_of<BF, false>(w, 0) * f, value_of<BF, false>(w, 1) * f);
          }
      }
    };

    // ---- While a tile's scores are weighed, the tile after it is multiplied with
    // the queries and the one before it added up, half a tile of each at a time:
    // matrix and vector instructions of different halves fill one another's time
    // without more registers.  At the top of step t LDS holds the keys of t + 1 and
    // the values of t - 1 and t; registers bring the keys of t + 2 and the values
    // of t + 1.  One barrier a tile: after it, the keys of t and the values of
    // t - 1 have been read by all, and what was stored in the step before is there.
    uint64_t there0, there1, there2, there3;  // of t, t + 1, ..
    if constexpr (DIRECT) {
      Places at;
      there0 = put(t, id);
      look_up(t, at);
      fetch_rows(kbase, at, keys + (t & 1) * KT);
      fetch_rows(vbase, at, values + (t & 1) * VT);
      there1 = put(t + 1, id_next);
      look_up(t + 1, at);
      fetch_rows(kbase, at, keys + (~t & 1) * KT);
      id = load_id(t + 2);
      id_next = load_id(t + 3);
#pragma unroll
      for (int i = 0; i < L; ++i)
        *reinterpret_cast<u32x4_t *>(values + (~t & 1) * VT + (i * 4 + wave) * kFour + lane * 16) = u32x4_t{0, 0, 0, 0};
#pragma unroll
      for (int u = 0; u < 2; ++u) p[1][u] = u32x4_t{0, 0, 0, 0};
      there2 = put(t + 2, id);
      id = id_next;
      there3 = 0;
      __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
      __syncthreads();
      products(t, 0);
      products(t, 1);
      look(t, there0);
    } else {
      u32x4_t second[L];
      Places at;
      there0 = put(t, id);
      look_up(t, at);
      load_rows(kbase, at, kt);
      load_rows(vbase, at, vt);
      there1 = put(t + 1, id_next);
      look_up(t + 1, at);
      load_rows(kbase, at, second);
      id = load_id(t + 2);
      id_next = load_id(t + 3);
      // (before the first tile there are no values: weights of 0, which need
      // finite numbers to stand there)
      uint8_t *const none = values + (~t & 1) * (TOK * VR) + tid / C * VR + tid % C * 16;
#pragma unroll
      for (int i = 0; i < L; ++i) *reinterpret_cast<u32x4_t *>(none + i * (256 / C) * VR) = u32x4_t{0, 0, 0, 0};
#pragma unroll
      for (int u = 0; u < 2; ++u) p[1][u] = u32x4_t{0, 0, 0, 0};
      store_keys(t, kt);
      store_values(t, is_edge(tile_base(t), there0), there0);
      store_keys(t + 1, second);
      load_rows(vbase, at, vt);
      there2 = put(t + 2, id);
      look_up(t + 2, at);
      load_rows(kbase, at, kt);
      there3 = put(t + 3, id_next);
      id = load_id(t + 4);
      __syncthreads();
      products(t, 0);
      products(t, 1);
      look(t, there0);
    }
    do {
      weigh(0);
      add(t - 1, Const<1>{});
      if constexpr (ORDER) {
        __builtin_amdgcn_iglp_opt(2);
#pragma unroll
        for (int d = 0; d < DB; ++d) asm volatile("" : "+v"(acc[d]));
#pragma unroll
        for (int u = 0; u < 2; ++u) asm volatile("" : "+v"(p[0][u]));
        __builtin_amdgcn_sched_barrier(0);
      }
      Places at2, at3;
      look_up(t + 2, at2);
      look_up(t + (DIRECT ? 1 : 3), at3);
      if constexpr (DIRECT) {
        __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): the keys of t + 1 and the values of t are there
        __syncthreads();
        fetch_rows(kbase, at2, keys + (t & 1) * KT);
        fetch_rows(vbase, at3, values + (~t & 1) * VT);
        if (is_edge(tile_base(t), there0)) clean_values(t, there0);
      } else {
        __syncthreads();
        // (past the last tile: keys and values of the first slot, which nothing reads)
        store_keys(t + 2, kt);
        store_values(t + 1, is_edge(tile_base(t + 1), there1), there1);
        load_rows(kbase, at3, kt);
        load_rows(vbase, at2, vt);
      }
      if constexpr (ORDER) __builtin_amdgcn_sched_barrier(0);
      products(t + 1, 0);
      weigh(1);
      if constexpr (ORDER) {
        __builtin_amdgcn_iglp_opt(2);
        asm volatile("" : "+v"(s[0]));
      }
      // (computed here, beside the products, not where it is used next)
#pragma unroll
      for (int u = 0; u < 2; ++u) asm volatile("" : "+v"(p[1][u]));
      if constexpr (ORDER) __builtin_amdgcn_sched_barrier(0);
      products(t + 1, 1);
      add(t, Const<0>{});
      ++t;
      look(t, there1);  // (past the last tile nothing is there)
      there0 = there1;
      there1 = there2;
      if constexpr (DIRECT) {
        there2 = put(t + 2, id);
        id = load_id(t + 3);
      } else {
        there2 = there3;
        there3 = put(t + 3, id);
        id = load_id(t + 4);
      }
    } while (t < t_end);
    if constexpr (DIRECT) __builtin_amdgcn_s_waitcnt(0x0F70);  // nothing on its way to the LDS any more
    add(t - 1, Const<1>{});

    if (bounds[8]) {
      // The NaNs and infinities of the tiles above, to the rows that see their
      // tokens.
#pragma unroll 1
      for (int t2 = first; t2 < t_end; ++t2) {
        const uint64_t present = put(t2, load_id(t2));
        const int tb = tile_base(t2);
        if (!is_edge(tb, present)) continue;
#pragma unroll 1
        for (int o = 0; o < TOK; ++o) {
          if (!(present >> o & 1)) continue;
          const int j = tb + o;
          uint32_t sees = (j < hi) & ((j >= lo) | (j < sinks)) ? ~0u : 0u;
          asm volatile("" : "+v"(sees));  // a mask in a register, no branch for each value
          const uint8_t *const p = vbase + ring[(t2 & 1) * 64 + o] + 4 * half * CB;
#pragma unroll
          for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
              uint32_t v[CB];
              load_words<false, CB>(p + (d * 32 + 2 * i) * CB, v);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                constexpr int PER = 4 / CB;
                const uint32_t is = 0u - (nonfinite<BF, F8>(v[k / PER]) >> (k % PER * 8 * CB) & 1u);
                const uint32_t x = __builtin_bit_cast(uint32_t, value_of<BF, F8>(v[k / PER], k % PER));
                acc[d][i + k] += __builtin_bit_cast(float, x & is & sees);
              }
            }
        }
      }
    }

    // ---- write: lane (c, half) has row c and d = 32 b + 8 (i / 4) + 4 half + i % 4
    l = pair_sum(l);
    if (row < R) {
      const int part = (int)((uint32_t)(item * padded + first) / (uint32_t)per) - (int)((uint32_t)(item * padded) / (uint32_t)per);
      const int64_t to = ((int64_t)item * ap->pre_most + part) * kPrefixRows + wave * 32 + c;
      float *const o = ap->pre_part + to * D;
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int i = 0; i < 16; i += 4)
          *reinterpret_cast<f32x4_t *>(o + d * 32 + 2 * i + 4 * half) =
              f32x4_t{acc[d][i], acc[d][i + 1], acc[d][i + 2], acc[d][i + 3]};
      if (half == 0) {
        ap->pre_ml[to * 2] = m;
        ap->pre_ml[to * 2 + 1] = l;
      }
    }
  }
}

// The common tokens and the sequences' own in one launch.  Where both are short,
// each workgroup has one of the two, so that what their walks begin and end with
// is at the same time: as many for each as its cost is of all.  Where they are
// long, a workgroup takes its range of one, then its range of the other: the first
// half of them the own tokens first, the second half the common ones, so that of
// the two workgroups of a CU one is bound by the memory while the other is by the
// matrix units, and none ends early.  (Separate, in turn, us: 24 sequences of 4
// rows over 6001 tokens of E4M3 and 0..2500 of their own 69 and 84; 32 of 4 over
// 1000 and 500..2000 48 and 59; 64 of 8 over 16000 and 25..100 580 and 239; over
// 16000 and 500..2000 312 and 290.  The border takes 64 of 8 over 4000 and 25..100
// for short, where it loses: 98 and 91.)
template <bool BF, bool F8, int D, int RT, bool SH>
__global__ __launch_bounds__(256, 2) void shared_kernel(AttendArgs) {
  extern __shared__ __align__(16) uint8_t lds[];
  KernArgs *ap = kern_args();
  const int block = blockIdx.x, grid = gridDim.x;
  // (in small calls there are workgroups for the most that either can be cut in)
  int common = ap->pre_workgroups, own = ap->workgroups;
  if (common + own > grid) {
    int *const words = reinterpret_cast<int *>(lds);
    const int before = common_pages<true>(*ap) * ap->c.page;
    const int low = lowest_token(*ap, before, words);
    const int granules = (before - low + kPrefixTokens - 1) / kPrefixTokens;
    const int64_t first = (int64_t)granules * ap->pre_tiles * ap->c.H;
    const int64_t second = own_cost(*ap, before, words + 4) / 2;
    if (first + second < (int64_t)kLongWalk * grid && grid >= 16) {
      const int share = (int)((uint32_t)(first * grid) / (uint32_t)(first + second + 1)) & ~7;
      common = min(common, min(max(share, 8), grid - 8));
      own = min(own, grid - common);
    }
    __syncthreads();
  }
  const bool one = common + own <= grid;
  const bool prefix_first = one ? block >= own : 2 * block >= grid;
#pragma unroll 1
  for (int turn = 0; turn < (one ? 1 : 2); ++turn) {
    if ((turn == 0) == prefix_first)
      prefix_body<BF, F8, D>(reload(ap), lds, one ? block - own : grid - 1 - block, common);
    else
      attend_body<BF, F8, D, RT, SH, true>(reload(ap), lds, block, own);
    __syncthreads();
  }
}

// At D = 256 either needs the registers of a CU's one workgroup for itself.
template <bool BF, bool F8, int D>
__global__ __launch_bounds__(256, 1) void prefix_kernel(AttendArgs) {
  extern __shared__ __align__(16) uint8_t lds[];
  prefix_body<BF, F8, D>(kern_args(), lds, blockIdx.x, gridDim.x);
}

template <bool BF, bool F8, int D, int RT, bool SH>
int launch_shared_rt(const AttendArgs &a, hipStream_t stream) {
  constexpr size_t own = attend_lds(F8, D, RT, SH), common = prefix_lds(D);
  if constexpr (D == 256) {
    const auto first = prefix_kernel<BF, F8, D>;
    if (!allow_max_dynamic_lds(reinterpret_cast<const void *>(first))) return QGEMV_EHIP;
    hipLaunchKernelGGL(first, dim3(a.pre_workgroups), dim3(256), common, stream, a);
    if (hipGetLastError() != hipSuccess) return QGEMV_EHIP;
    const auto second = attend_kernel<BF, F8, D, RT, SH, attend_occupancy(F8, D, RT, SH), true>;
    if (own > 64 * 1024 && !allow_max_dynamic_lds(reinterpret_cast<const void *>(second))) return QGEMV_EHIP;
    hipLaunchKernelGGL(second, dim3(a.workgroups), dim3(256), own, stream, a);
  } else {
    constexpr size_t bytes = own > common ? own : common;
    const auto kern = shared_kernel<BF, F8, D, RT, SH>;
    if (bytes > 64 * 1024 && !allow_max_dynamic_lds(reinterpret_cast<const void *>(kern))) return QGEMV_EHIP;
    hipLaunchKernelGGL(kern, dim3(a.grid), dim3(256), bytes, stream, a);
  }
  if (hipGetLastError() != hipSuccess) return QGEMV_EHIP;
  return launch_join<BF, D, true>(a, stream);
}

template <bool BF, bool F8, int D, bool SH>
int launch_shared_d(const AttendArgs &a, hipStream_t stream) {
  if constexpr (D < 256)
    if (a.rt == 3) return launch_shared_rt<BF, F8, D, 3, SH>(a, stream);
  if constexpr (D == 64)
    if (a.rt == 4) return launch_shared_rt<BF, F8, D, 4, SH>(a, stream);
  if constexpr (one_tile(F8, D, SH, true))
    if (a.rt == 1) return launch_shared_rt<BF, F8, D, 1, SH>(a, stream);
  return launch_shared_rt<BF, F8, D, 2, SH>(a, stream);
}

template <bool BF, bool F8>
int launch_shared_t(const AttendArgs &a, hipStream_t stream) {
  switch (a.c.D) {
    case 64: return a.shared ? launch_shared_d<BF, F8, 64, true>(a, stream) : launch_shared_d<BF, F8, 64, false>(a, stream);
    case 128: return a.shared ? launch_shared_d<BF, F8, 128, true>(a, stream) : launch_shared_d<BF, F8, 128, false>(a, stream);
  }
  return a.shared ? launch_shared_d<BF, F8, 256, true>(a, stream) : launch_shared_d<BF, F8, 256, false>(a, stream);
}

}  // namespace qgemv
