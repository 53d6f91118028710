// Attention of the new rows of each sequence over its paged cache.
//
//   s_j = scale * k_scale[h] * (q . k_j) over the tokens j that the row sees:
//         j <= pos, and with a window W also j > pos - W or j < sinks
//   lse = log sum_j exp(s_j),  out = v_scale[h] * sum_j exp(s_j - lse) v_j
//
// A key-value head's G query heads and its sequence's rows share its keys, so
// they are one product: R = rows * G query rows against n tokens, 4 R D flops
// for 4 D bytes of cache (16 bits).  Up to R of some hundred it is bound by
// reading the cache, which every design choice serves.
//
// * A wave takes tiles of 32 tokens, up to 64 query rows (RT tiles of 16) and
//   all of D.  S^T = K Q^T: the A operand's lane (c, g) holds 8 consecutive d
//   of token c.  Loads in that shape take 64 bytes of 16 keys at a time, half
//   a line each, so keys are loaded in whole rows instead and pass through a
//   stage in LDS of the wave's own, of which it reads the operands (loads
//   alone, 3.2 GB of pages: 5.75 TB/s by half lines, 6.6 by whole rows past
//   the caches).
//   O^T += V^T P^T: P^T's operand lane holds 8 tokens of one query row, and
//   the order of the tokens within the product is free, so the 4 + 4 scores
//   that the first product leaves in a lane are that operand as they stand.
//   V^T's lane holds 8 tokens of one d: each lane loads 8 consecutive d of
//   those 8 tokens (whole rows of the cache per load instruction) and turns
//   the block with byte permutes, 2 dwords an instruction.  No wave waits for
//   another before an item's end.
// * More rows than that (SH) are split over the four waves of a workgroup,
//   which share every tile: each loads 8 of its tokens, and one barrier a tile
//   lies between the two halves of a stage.  16 sequences of 4000..9000 tokens
//   and 192 rows take 157 us; when each wave read all tokens for its rows, 265.
// * Running maximum and sum per row, in base 2.  The reference that weights are
//   taken against moves only when a score passes the maximum it was set by by
//   more than 8: most tiles then leave the output's registers alone.  For bf16
//   it is that maximum (the largest weight is 1 to 2^8), for fp16 7 below it
//   (2^7 to 2^15): fp16 ends at 2^16 above and at 2^-24 below, and with the largest
//   weight near 1 a long tail of weights below 2^-25 was lost to the output
//   while the sum counted it (65536 tokens 18 nats below one, 96 rows: all).
// * Keys of the next tile are loaded as soon as this tile's product has read
//   the stage, values as soon as theirs has read them: while a wave computes,
//   a whole tile is on its way.
// * The work of a call is cut in ranges of granules (one tile for each wave
//   that shares the tokens), whatever the lengths are: a workgroup walks its
//   range over (sequence, head) items, joins its waves at the end of each item
//   and writes the result, or its part of an item that other workgroups share,
//   which a second kernel joins in a fixed order.  Short items have a workgroup
//   each.
//
// On an MI355X: 64 sequences of 8k..16k tokens, 8 heads of 128, 48 rows: 3.25 GB
// in 572 us (5.7 TB/s; a pure read of as much: 468 us).  64 sequences of
// 300..8000, 6 rows: 1.1 GB in 183 us.  One sequence of 200: 7 us, latency.
#pragma once

#include "qgemv_device.h"
#include "qgemv_kv.h"

namespace qgemv {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kNegInf = -__builtin_inff();

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));

template <bool BF>
__device__ __forceinline__ f32x4_t mfma_16x16x32(u32x4_t a, u32x4_t b, f32x4_t c) {
  if constexpr (BF)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                   __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a),
                                                  __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
}

// How far below the largest score the reference of the weights lies, in base 2.
template <bool BF>
constexpr float kHeadroom = BF ? 0.0f : 7.0f;

// log sum exp of weights summed against reference m, from base 2.
template <bool BF>
__device__ __forceinline__ float log_of(float m, float l) {
  // (both terms near the score itself, so that their rounding is no more than its)
  constexpr float down = BF ? 1.0f : 0.0078125f;  // 2^-headroom
  return ((m + kHeadroom<BF>) + __builtin_log2f(l * down)) * kLn2;
}

// Two E4M3 bytes (bytes 2 HI, 2 HI + 1) as a pair of the product's type, exact.
template <bool BF, bool HI>
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t w) {
  if constexpr (BF)
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI));
  else
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HI));
}

// Two floats as a pair of the product's type, rounded to nearest even.
template <bool BF>
__device__ __forceinline__ uint32_t pair_of(float lo, float hi) {
  if constexpr (BF) {
    const bf16x2_t v = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(uint32_t, v);
  } else {
    return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)lo) |
           (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)hi) << 16;
  }
}

// Maximum / sum over the four lanes of a query row (lanes c, c+16, c+32, c+48).
__device__ __forceinline__ float row_max(float x) {
  auto a = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x),
                                            false, false);
  x = fmaxf(__builtin_bit_cast(float, (uint32_t)a[0]), __builtin_bit_cast(float, (uint32_t)a[1]));
  auto b = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x),
                                            false, false);
  return fmaxf(__builtin_bit_cast(float, (uint32_t)b[0]), __builtin_bit_cast(float, (uint32_t)b[1]));
}
__device__ __forceinline__ float row_sum(float x) {
  auto a = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x),
                                            false, false);
  x = __builtin_bit_cast(float, (uint32_t)a[0]) + __builtin_bit_cast(float, (uint32_t)a[1]);
  auto b = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x),
                                            false, false);
  return __builtin_bit_cast(float, (uint32_t)b[0]) + __builtin_bit_cast(float, (uint32_t)b[1]);
}

// 2^(x - m) for a maximum m of x, 0 where both are -inf.
__device__ __forceinline__ float weight_of(float x, float m) {
  return __builtin_amdgcn_exp2f(x - (m == kNegInf ? 0.0f : m));
}

// What one sequence asks for.
struct SeqWork {
  int row0, rows;   // its rows in q
  int pos0;         // position of its first row
  int end;          // tokens [0, end) can be seen
  int low_tile;     // first tile of the window (0 without one)
  int sink_tiles;   // tiles of the sinks before it
  int tiles;        // of both
  int granules;     // of one item
  int groups;       // of rows, an item each
  int items;        // (head, group of rows)
};

// A kernel's arguments where the launch put them.  Read through a pointer that
// is made opaque between the parts of the kernel, so that what only one part
// needs is loaded there and not kept in scalar registers across the tile loop.
typedef const __attribute__((address_space(4))) AttendArgs KernArgs;
__device__ __forceinline__ KernArgs *kern_args() {
  return (KernArgs *)__builtin_amdgcn_kernarg_segment_ptr();
}
__device__ __forceinline__ KernArgs *reload(KernArgs *p) {
  asm volatile("" : "+s"(p));
  return p;
}

// What no kernel writes: at a uniform index it takes scalar loads, which do not
// wait for the vector loads in flight.
template <class T>
__device__ __forceinline__ const __attribute__((address_space(4))) T *constant(const T *p) {
  return (const __attribute__((address_space(4))) T *)(uintptr_t)p;
}

// PRE: tokens that all sequences have in the same pages are another kernel's
// (qgemv_prefix_impl.h).  Here a sequence begins after them: positions, the
// table and the sinks are counted from there, and a row before it sees nothing.
template <bool PRE, class Args>
__device__ __forceinline__ int common_pages(Args &a) {
  if constexpr (!PRE) return 0;
  // never the table's last page, so that each sequence has an id to look up
  return min((int)(__umulhi(a.c.magic, 2u * (uint32_t)min(max(constant(a.common)[0], 0), QGEMV_MAX_CONTEXT - 1)) >>
                   a.c.shift),
             a.c.width - 1);
}

template <bool PRE, class Args>
__device__ __forceinline__ SeqWork seq_work(Args &a, int b, int before) {
  SeqWork w;
  const auto start = constant(a.start), lens = constant(a.len);
  const int s0 = min(max(start[b], 0), a.T), s1 = min(max(start[b + 1], s0), a.T);
  // the rows' positions follow the length itself, what they can see the table:
  // past its end there are rows, but no tokens
  const int all_tokens = min(max(lens[b], 0), QGEMV_MAX_CONTEXT);
  const int len = PRE ? max(all_tokens - before, 0) : all_tokens;
  w.row0 = s0;
  w.rows = min(s1 - s0, a.M);
  w.pos0 = len - (s1 - s0);
  w.end = min(a.c.width * a.c.page - (PRE ? before : 0), max(w.pos0 + w.rows, 0));
  const int low = a.window ? min(max(0, w.pos0 - a.window + 1), w.end) : 0;
  const int all = (w.end + 31) >> 5;
  w.low_tile = low >> 5;
  const int sinks = PRE ? max(a.sinks - before, 0) : a.sinks;
  w.sink_tiles = a.window ? min(min((sinks >> 5) + ((sinks & 31) != 0), w.low_tile), all) : 0;
  w.tiles = w.sink_tiles + max(all - w.low_tile, 0);
  // an item without tokens still writes its rows; one that no workgroups share
  // is one granule
  w.granules = !a.joins ? 1 : max(a.shared ? w.tiles : (w.tiles + 3) >> 2, 1);
  const int item_rows = (a.shared ? 64 : 16) * a.rt, R = w.rows * a.G;
  w.groups = R <= item_rows ? 1 : (R + item_rows - 1) / item_rows;
  w.items = w.rows > 0 ? a.c.H * w.groups : 0;
  return w;
}

// Values of one tile as they lie in memory: 8 tokens of the lane's group, E
// consecutive d of each half of D (one half below D = 256).
template <bool F8, int D>
struct Tile {
  static constexpr int ROW = D * (F8 ? 1 : 2);     // bytes of a key or value
  static constexpr int KL = ROW / 32;              // loads of a wave for the tile's keys
  static constexpr int KC = ROW / 16;              // 16-byte chunks of a key
  static constexpr bool NT = ROW >= 128;           // whole lines are read at once
  // a wave's 8 tokens of a shared tile: bytes of a load, loads of a row, of a wave
  static constexpr int SB = ROW >= 128 ? 16 : 8, SC = ROW / SB, SL = SC / 8;
  static constexpr int VH = D == 256 ? 2 : 1;
  static constexpr int E = D / 16 / VH;
  static constexpr int VW = E * (F8 ? 1 : 2) / 4;  // dwords of one token's values in a half
};

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

// A load of the cache, past the caches where it reads whole lines (NT).
template <bool NT, class T>
__device__ __forceinline__ T load_cache(const uint8_t *p) {
  if constexpr (NT) return __builtin_nontemporal_load(reinterpret_cast<const T *>(p));
  return *reinterpret_cast<const T *>(p);
}

template <bool NT, int VW>
__device__ __forceinline__ void load_words(const uint8_t *p, uint32_t (&w)[VW]) {
  if constexpr (VW == 4) {
    const u32x4_t v = load_cache<NT, u32x4_t>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = v[i];
  } else if constexpr (VW == 2) {
    const u32x2_t v = load_cache<NT, u32x2_t>(p);
    w[0] = v[0];
    w[1] = v[1];
  } else {
    w[0] = load_cache<NT, uint32_t>(p);
  }
}

// V^T operands of d = E-chunk element e (and e + 1 for 16 bits; e .. e + 3 for
// 8): slots (2 i, 2 i + 1) of the lane's 8 tokens in dword i.
template <bool BF, bool F8, int VW>
__device__ __forceinline__ void turn(const uint32_t (&v)[8][VW], int word, u32x4_t *o) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = v[2 * i][word], b = v[2 * i + 1][word];
    if constexpr (F8) {
      const uint32_t lo = perm_b32(b, a, 0x05010400u), hi = perm_b32(b, a, 0x07030602u);
      o[0][i] = e4m3_pair<BF, false>(lo);
      o[1][i] = e4m3_pair<BF, true>(lo);
      o[2][i] = e4m3_pair<BF, false>(hi);
      o[3][i] = e4m3_pair<BF, true>(hi);
    } else {
      o[0][i] = perm_b32(b, a, 0x05040100u);
      o[1][i] = perm_b32(b, a, 0x07060302u);
    }
  }
}

// The sign bits of a dword's NaNs and infinities set, of its other values not:
// an exponent of all ones (for E4M3 also all mantissa bits) carries into them.
template <bool BF, bool F8>
__device__ __forceinline__ uint32_t nonfinite_signs(uint32_t w) {
  if constexpr (F8) return (w & 0x7F7F7F7Fu) + 0x01010101u;
  return BF ? (w & 0x7F807F80u) + 0x00800080u : (w & 0x7C007C00u) + 0x04000400u;
}
template <bool F8>
constexpr uint32_t kSigns = F8 ? 0x80808080u : 0x80008000u;

// The bits of a dword of cached values that belong to NaNs and infinities.
template <bool BF, bool F8>
__device__ __forceinline__ uint32_t nonfinite(uint32_t w) {
  const uint32_t t = nonfinite_signs<BF, F8>(w) & kSigns<F8>;
  return t | (t - (t >> (F8 ? 7 : 15)));
}

// Element i of a dword of cached values.
template <bool BF, bool F8>
__device__ __forceinline__ float value_of(uint32_t w, int i) {
  if constexpr (F8) return e4m3_to_float(w >> (8 * i));
  const uint32_t h = i ? w >> 16 : w & 0xFFFFu;
  return BF ? bf16_bits_to_float(h) : half_bits_to_float(h);
}

// Workgroups of 256 threads that a CU holds, by registers and LDS: the output
// takes D / 4 registers a tile of rows, keys and values of a wave D / 2 (16 bits).
// With 64 rows at D = 128 they fit two workgroups only from an 8-bit cache (32
// sequences of 4000..12000 tokens: 225 -> 155 us; 16 bits would spill: 236 -> 328).
constexpr int attend_occupancy(bool f8, int D, int rt, bool sh) {
  return D * rt <= 128 ? 3 : D * rt <= 384 || (D == 128 && f8 && !sh) ? 2 : 1;
}

// Queries stay in registers (D / 8 a tile of rows) while they take less than
// 32, or 64 where keys and values do not wait in registers.
constexpr bool queries_in_lds(int D, int rt, bool sh) { return D * rt >= (sh ? 512 : 256); }

// Whether one tile of rows a wave can be the plan's choice: not where rows are split
// over the waves (sh) from 65 on, since those are two tiles a wave at least.
constexpr bool one_tile(bool f8, int D, bool sh, bool after_prefix) {
  return !sh || D == 256 || (D == 128 && (after_prefix || !f8));
}

constexpr size_t kLdsHead = 2048 + 64;  // token offsets and the scan
constexpr size_t attend_lds(bool f8, int D, int rt, bool sh) {
  const size_t q = queries_in_lds(D, rt, sh) ? (size_t)(sh ? 4 : 1) * rt * D * 32 : 0;
  const size_t stage = (size_t)4 * 32 * D * (f8 ? 1 : 2);  // each wave's keys, or keys and values twice
  const size_t give = sh ? 0 : (size_t)2 * rt * (512 + D * 64);
  return kLdsHead + (q + stage > give ? q + stage : give);
}

// Where the stage of a wave's keys holds chunk `chunk` of token `token`: lanes
// of 16 tokens that read one chunk each find it in different banks.
template <int ROW>
__device__ __forceinline__ int stage_at(int token, int chunk) {
  constexpr int PER = ROW >= 256 ? 1 : 256 / ROW;  // keys side by side in the 64 banks
  constexpr int MASK = (ROW >= 256 ? 256 : ROW) / 16 - 1;
  return token * (ROW / 16) + (chunk ^ (token / PER & MASK));
}

// How the granules of a call lie on its workgroups: equal ranges within a rank.
// The workgroups of a CU do not run alike: in equal ranges, of two the one that
// came first was done in 395 us where the other took 500, of three in 95, 140
// and 163 us (the older waves' loads go first).  So the ranks take unequal
// shares: 64 sequences of 8k..16k tokens, 8 rows 597 -> 584 us, 300..8000
// tokens, one row 194 -> 190; the optima are flat (within 2% from 158 to 188 of
// 256).  Short ranges are equal: there the loads of all start at once, and a
// granule more costs more than a share gains (one sequence of 32768, 4 granules
// each: 36 us, 39 with shares).
constexpr int kShareOfTwo = 176, kShareOfTwoShared = 158;  // 256ths, of the first rank
constexpr int kShareOfThree = 108, kShareOfRest = 138;     // of the first, and of the second in what is left
constexpr int kRankTiles = 24;                             // tiles of a range from which on

struct Split {
  int ranks, n;          // ranks of n workgroups each
  int per0, per1, per2;  // granules of a workgroup
};

template <bool PRE, class Args>
__device__ __forceinline__ Split split_of(Args &a, int total, int workgroups) {
  if constexpr (PRE) return Split{1, workgroups, max((total + workgroups - 1) / workgroups, 1), 0, 0};
  const int ranks = a.ranks, n = a.rank_size;
  auto per = [&](int left, int share) {  // share 256ths of what is left, over n workgroups
    const int part = (left >> 8) * share + ((left & 255) * share >> 8);
    return max((int)(__umulhi(a.rank_magic, 2u * (uint32_t)(part + n - 1)) >> a.rank_shift), 1);
  };
  const bool equal = total * (a.shared ? 1 : 4) < kRankTiles * ranks * n;
  const int two = equal ? 128 : a.shared ? kShareOfTwoShared : kShareOfTwo;
  Split s{ranks, n, 0, 0, 0};
  s.per0 = per(total, ranks == 3 ? (equal ? 86 : kShareOfThree) : ranks == 2 ? two : 256);
  total = max(total - n * s.per0, 0);
  s.per1 = per(total, ranks == 3 ? (equal ? 128 : kShareOfRest) : 256);
  s.per2 = per(max(total - n * s.per1, 0), 256);
  return s;
}

// Granules [start, end) of a workgroup.
__device__ __forceinline__ void split_range(const Split &s, int wg, int *start, int *end) {
  const int p0 = s.per0, p1 = s.per1, p2 = s.per2;  // (selected as members they go through memory)
  const bool r1 = wg >= s.n, r2 = wg >= 2 * s.n;
  const int before = r2 ? p0 + p1 : r1 ? p0 : 0, per = r2 ? p2 : r1 ? p1 : p0;
  *start = before * s.n + (wg - (r2 ? 2 * s.n : r1 ? s.n : 0)) * per;
  *end = *start + per;
}

// The workgroup of a granule.
__device__ __forceinline__ int split_owner(const Split &s, int granule) {
  const int p0 = s.per0, p1 = s.per1, p2 = s.per2;
  const int first = s.n * p0, second = first + s.n * p1;
  const bool r1 = s.ranks > 1 && granule >= first, r2 = s.ranks > 2 && granule >= second;
  const int at = granule - (r2 ? second : r1 ? first : 0), per = r2 ? p2 : r1 ? p1 : p0;
  return (r2 ? 2 * s.n : r1 ? s.n : 0) + (int)((uint32_t)at / (uint32_t)per);
}

// The range of this workgroup: granules [cur, range1) of all items in order,
// the first of them in sequence b, before which lie `base`.  False if there is
// none.  Workgroup 0 writes the plan for the join.
template <bool PRE, class Args>
__device__ __forceinline__ bool attend_range(Args &a, int before, int wg, int workgroups, int *scan, int *b, int *base, int *cur, int *range1) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int B = a.B;
  int total = 0;
  int at = 0, end = 0;
  auto place = [&]() { split_range(split_of<PRE>(a, total, workgroups), wg, &at, &end); };
  auto granules_of = [&](int s) {
    const SeqWork w = seq_work<PRE>(a, s, before);
    return w.items * w.granules;
  };
  auto inclusive = [&](int in) {  // sums over the lanes up to each, by DPP: shifts within 16, then broadcasts
    in += __builtin_amdgcn_update_dpp(0, in, 0x111, 0xF, 0xF, false);
    in += __builtin_amdgcn_update_dpp(0, in, 0x112, 0xF, 0xF, false);
    in += __builtin_amdgcn_update_dpp(0, in, 0x114, 0xF, 0xF, false);
    in += __builtin_amdgcn_update_dpp(0, in, 0x118, 0xF, 0xF, false);
    in += __builtin_amdgcn_update_dpp(0, in, 0x142, 0xA, 0xF, false);  // lane 15 to lanes 16..31, 47 to 48..63
    in += __builtin_amdgcn_update_dpp(0, in, 0x143, 0xC, 0xF, false);  // lane 31 to lanes 32..63
    return in;
  };
  if (B == 1) {
    total = granules_of(0);
    place();
    if (wg == 0 && threadIdx.x == 0) a.plan[2] = total;
    *b = 0;
    *base = 0;
  } else if (B <= 64) {  // every wave by itself
    const int n = lane < B ? granules_of(lane) : 0, in = inclusive(n);
    total = __builtin_amdgcn_readlane(in, 63);
    place();
    if (wg == 0 && wave == 0 && lane < B) a.plan[2 + lane] = in;
    const uint64_t mine = __ballot(n && at >= in - n && at < in);
    const int at_lane = mine ? (int)__ffsll((long long)mine) - 1 : 0;
    *b = __builtin_amdgcn_readfirstlane(at_lane);
    *base = __builtin_amdgcn_readfirstlane(__builtin_amdgcn_readlane(in - n, at_lane));
  } else {
    // Steps of 256 sequences, one a thread.  The total is needed before a range
    // can be placed: with more sequences the steps are taken twice.
    for (int round = B <= 256; round < 2; ++round) {
      int carry = 0;
      for (int s0 = 0; s0 < B; s0 += 256) {
        const int s = s0 + (int)threadIdx.x;
        const int n = s < B ? granules_of(s) : 0;
        int in = inclusive(n);
        if (lane == 63) scan[wave] = in;
        __syncthreads();
        const int n0 = scan[0], n1 = scan[1], n2 = scan[2], n3 = scan[3];
        in += carry + (wave > 0 ? n0 : 0) + (wave > 1 ? n1 : 0) + (wave > 2 ? n2 : 0);
        carry += n0 + n1 + n2 + n3;
        if (B <= 256) total = carry;
        if (round) {
          place();
          if (n && at >= in - n && at < in) {
            scan[4] = s;
            scan[5] = in - n;
          }
          if (wg == 0 && s < B) a.plan[2 + s] = in;
        }
        __syncthreads();
      }
      total = carry;
    }
    *b = __builtin_amdgcn_readfirstlane(scan[4]);
    *base = __builtin_amdgcn_readfirstlane(scan[5]);
  }
  if (PRE && wg == 0 && threadIdx.x == 0) a.pre_plan[2] = workgroups;
  if (wg == 0 && threadIdx.x == 0) {
    a.plan[0] = total;
    a.plan[1] = 0;
  }
  if (__builtin_amdgcn_readfirstlane((int)(at >= total))) return false;
  *cur = __builtin_amdgcn_readfirstlane(at);
  *range1 = __builtin_amdgcn_readfirstlane(min(end, total));
  return true;
}

template <bool BF, bool F8, int D, int RT, bool SH, bool PRE>
__device__ __forceinline__ void attend_body(KernArgs *ap, uint8_t *const lds, const int wg, const int workgroups) {
  using T = Tile<F8, D>;
  constexpr int KL = T::KL, KC = T::KC, VH = T::VH, E = T::E, VW = T::VW, NE = VH * E;
  constexpr int CB = F8 ? 1 : 2;
  constexpr int QS = D / 32;  // steps of the first product
  constexpr bool QLDS = queries_in_lds(D, RT, SH);
  constexpr int CHUNKS = SH ? 4 : 1, TW = 4 / CHUNKS;  // waves that split the rows, and the tokens
  // LDS: [4 waves][2][32] token offsets, the scan, then the queries and the waves'
  // keys and, after the tokens, in the same place what waves hand over
  int64_t *const ring = reinterpret_cast<int64_t *>(lds);
  int *const scan = reinterpret_cast<int *>(lds + 2048);
  u32x4_t *const queries = reinterpret_cast<u32x4_t *>(lds + kLdsHead);
  float *const give_ml = reinterpret_cast<float *>(lds + kLdsHead);
  f32x4_t *const give = reinterpret_cast<f32x4_t *>(lds + kLdsHead + 2 * RT * 64 * 2 * 4);

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int chunk = SH ? wave : 0, tw = SH ? 0 : wave;

  // Items that no two workgroups share have a workgroup each; the others are
  // walked in equal ranges.
  const int common = common_pages<PRE>(*ap), before = PRE ? common * ap->c.page : 0;
  const bool joins = PRE || ap->joins;
  int b, base = 0, cur = 0, range1 = 1;
  if (joins) {
    if (!attend_range<PRE>(*ap, before, wg, workgroups, scan, &b, &base, &cur, &range1)) return;
  } else {
    b = wg / ap->seq_items;
  }

  int64_t *const my_ring = ring + wave * 64;
  int half = 0;  // of the shared stage: what the waves may still read, and what they write
  u32x4_t *const stage = queries + (QLDS ? CHUNKS * RT * QS * 64 : 0) + (SH ? 0 : wave * (32 * KC));

  while (cur < range1) {
    ap = reload(ap);
    const SeqWork w = seq_work<PRE>(*ap, b, before);
    const int seq_granules = w.items * w.granules, groups = w.groups;
    int item, first = 0;
    if (joins) {
      if (cur >= base + seq_granules) {  // past this sequence (or it has no rows)
        base += seq_granules;
        ++b;
        continue;
      }
      item = (int)((uint32_t)(cur - base) / (uint32_t)w.granules);
      first = (cur - base) - item * w.granules;
    } else {
      item = wg - b * ap->seq_items;
      if (item >= w.items) return;
    }
    const int n_granules = min(w.granules - first, range1 - cur);
    const int h = groups == 1 ? item : (int)((uint32_t)item / (uint32_t)groups), group = item - h * groups;
    cur += n_granules;

    const int R = w.rows * ap->G;
    const int row_first = (group * CHUNKS + chunk) * RT * 16;

    ap = reload(ap);
    const uint8_t *const kbase = ap->c.k + h * ap->c.stride_head;
    const uint8_t *const vbase = ap->c.v + h * ap->c.stride_head;
    const int32_t *const table = ap->c.table + (int64_t)b * ap->c.width + (PRE ? common : 0);
    const int64_t stride_page = ap->c.stride_page, stride_slot = ap->c.stride_slot;
    const int page = ap->c.page, pages = ap->c.pages, shift = ap->c.shift;
    const uint32_t magic = ap->c.magic;
    const int window = ap->window ? ap->window : 1 << 30;  // none: as wide as any position
    const int sinks = PRE ? max(ap->sinks - before, 0) : ap->sinks;
    const float sc = ap->scale * (ap->c.k_scale ? constant(ap->c.k_scale)[h] : 1.0f) * kLog2e;
    const int t_end = min((first + n_granules) * TW * ap->span, w.tiles);
    int t = first * TW * ap->span + tw;

    auto tile_base = [&](int tile) { return (tile < w.sink_tiles ? tile : tile - w.sink_tiles + w.low_tile) * 32; };
    // No load of the loop lies in a branch: with one that may not have been
    // issued the compiler cannot count what is in flight and waits for all.
    // Past the last tile, ids are those of the last token, and keys and values
    // the first slot's, a row that stays in the caches.
    auto load_id = [&](int tile) -> int {
      const int token = min(tile_base(tile) + (lane & 31), max(w.end - 1, 0));
      return table[__umulhi(magic, 2 * token) >> shift];
    };
    // offsets of a tile's tokens into the ring; bit i: token i is there
    auto put = [&](int tile, int id, int slot) -> uint32_t {
      const int token = tile_base(tile) + (lane & 31);
      const bool ok = ((uint32_t)id < (uint32_t)pages) & (tile < t_end) & (token < w.end);
      const int in_page = token - (int)(__umulhi(magic, 2 * token) >> shift) * page;
      const int64_t at = ok ? id * stride_page + in_page * stride_slot : 0;
      if (lane < 32) my_ring[slot * 32 + lane] = at;
      // a wave's LDS accesses stay in order; this keeps the compiler from moving them
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      return (uint32_t)__ballot(ok);
    };
    // whether some row does not see some token of a tile
    auto is_edge = [&](int tb, uint32_t present) {
      return (present != 0xFFFFFFFFu) | (tb + 31 > w.pos0) |
             ((tb <= w.pos0 + w.rows - 1 - window) & (tb + 31 >= sinks));
    };
    // this wave's share of a tile's keys and values: all of them, or 8 tokens
    u32x4_t kt[SH ? T::SL : KL];
    u32x4_t vs[SH ? T::SL : 1];
    uint32_t vt[VH][8][VW];
    auto load_share = [&](const uint8_t *from, int slot, u32x4_t *to) {
#pragma unroll
      for (int s = 0; s < T::SL; ++s) {
        const int at = s * 64 + lane;
        const uint8_t *p = from + my_ring[slot * 32 + wave * 8 + at / T::SC] + at % T::SC * T::SB;
        if constexpr (T::SB == 16) {
          to[s] = load_cache<T::NT, u32x4_t>(p);
        } else {
          const u32x2_t x = load_cache<T::NT, u32x2_t>(p);
          to[s][0] = x[0];
          to[s][1] = x[1];
        }
      }
    };
    auto load_k = [&](int slot) {
      if constexpr (SH) return load_share(kbase, slot, kt);
#pragma unroll
      for (int s = 0; s < KL; ++s) {
        const int token = (s * 64 + lane) / KC, chunk = lane % KC;
        kt[s] = load_cache<T::NT, u32x4_t>(kbase + my_ring[slot * 32 + token] + chunk * 16);
      }
    };
    auto load_v = [&](int slot) {
      if constexpr (SH) return load_share(vbase, slot, vs);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint8_t *p = vbase + my_ring[slot * 32 + (j >> 2) * 16 + g * 4 + (j & 3)] + c * (E * CB);
#pragma unroll
        for (int x = 0; x < VH; ++x) load_words<T::NT, VW>(p + x * (128 * CB), vt[x][j]);
      }
    };

    int slot = 0;
    uint32_t there = 0, there_next = 0;
    bool strays = false;  // values that were taken out
    // ---- page ids, then the query rows, then the first keys and values: all on
    // their way together.  A lane has one row of each 16-row tile; rows past R
    // repeat the last one and see nothing.
    const int id0 = load_id(t);
    int id = load_id(t + TW);
    int pos[RT];
    constexpr int NQ = QLDS ? CHUNKS * RT * QS / 4 : RT * QS;
    u32x4_t qf[NQ];
    {
      const int G = ap->G, div = ap->group_magic;
      auto query = [&](int row, int s) -> u32x4_t {
        const int at = min(row, R - 1), i = at * div >> 16, hq = h * G + at - i * G;
        // the d of a lane's 8 slots follow the key loads
        const int d = F8 ? (s >> 1) * 64 + g * 16 + (s & 1) * 8 : s * 32 + g * 8;
        return *reinterpret_cast<const u32x4_t *>(ap->q + (int64_t)(w.row0 + i) * ap->q_row + hq * ap->q_head + d * 2);
      };
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const int row = row_first + r * 16 + c;
        pos[r] = row < R ? w.pos0 + (row * div >> 16) : -1;
      }
#pragma unroll
      for (int u = 0; u < NQ; ++u) {
        if constexpr (QLDS)  // [wave's rows][tile][step][lane], every wave a quarter of the steps
          qf[u] = query(group * CHUNKS * RT * 16 + (u * 4 + wave) / QS * 16 + c, (u * 4 + wave) % QS);
        else
          qf[u] = query(row_first + u / QS * 16 + c, u % QS);
      }
    }
    there = put(t, id0, 0);
    __builtin_amdgcn_sched_barrier(0);
    load_k(0);
    load_v(0);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (QLDS) {
      __syncthreads();  // the last item's queries, or hand-over, have been read
#pragma unroll
      for (int u = 0; u < NQ; ++u) queries[(u * 4 + wave) * 64 + lane] = qf[u];
      __syncthreads();
    } else {
      // they have arrived: no wait for them, and what came later, in the loop
#pragma unroll
      for (int u = 0; u < NQ; ++u) asm volatile("" : "+v"(qf[u]));
    }
    const u32x4_t *const ql = queries + chunk * RT * QS * 64 + lane;

    f32x4_t acc[RT][NE];
    float m[RT], l[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      m[r] = kNegInf;
      l[r] = 0.0f;
#pragma unroll
      for (int e = 0; e < NE; ++e) acc[r][e] = f32x4_t{0, 0, 0, 0};
    }

    for (; t < t_end; t += TW) {
      there_next = put(t + TW, id, slot ^ 1);
      id = load_id(t + 2 * TW);

      // ---- keys to the stage
      int at = lane;
      asm volatile("" : "+v"(at));  // places computed anew for each tile, not kept in registers
      u32x4_t *const keys = stage + (SH ? half * (64 * KC) : 0);
      const uint8_t *const values = reinterpret_cast<const uint8_t *>(keys + 32 * KC);
      if constexpr (SH) {
#pragma unroll
        for (int s = 0; s < T::SL; ++s) {
          const int token = wave * 8 + (s * 64 + at) / T::SC, part = (s * 64 + at) % T::SC;
          if constexpr (T::SB == 16) {
            keys[stage_at<T::ROW>(token, part)] = kt[s];
            keys[32 * KC + token * KC + part] = vs[s];
          } else {
            u32x2_t *const k2 = reinterpret_cast<u32x2_t *>(keys), x = {kt[s][0], kt[s][1]}, y = {vs[s][0], vs[s][1]};
            k2[stage_at<T::ROW>(token, part >> 1) * 2 + (part & 1)] = x;
            k2[64 * KC + token * KC * 2 + part] = y;
          }
        }
        __builtin_amdgcn_sched_barrier(0);
        load_k(slot ^ 1);
        load_v(slot ^ 1);
        __builtin_amdgcn_sched_barrier(0);
        __syncthreads();
        half ^= 1;
      } else {
#pragma unroll
        for (int s = 0; s < KL; ++s) keys[stage_at<T::ROW>((s * 64 + at) / KC, at % KC)] = kt[s];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      }

      // ---- scores of 32 tokens: lane (c, g) has row c, tokens tt * 16 + 4 g + i
      f32x4_t s[RT][2];
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) s[r][tt] = f32x4_t{0, 0, 0, 0};
#pragma unroll
      for (int st = 0; st < QS; ++st) {
        u32x4_t ka[2];
        const int chunk = (F8 ? st >> 1 : st) * 4 + (at >> 4);
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) {
          const u32x4_t x = keys[stage_at<T::ROW>(tt * 16 + (at & 15), chunk)];
          if constexpr (F8) {
            const uint32_t x0 = x[2 * (st & 1)], x1 = x[2 * (st & 1) + 1];
            ka[tt] = u32x4_t{e4m3_pair<BF, false>(x0), e4m3_pair<BF, true>(x0), e4m3_pair<BF, false>(x1),
                             e4m3_pair<BF, true>(x1)};
          } else {
            ka[tt] = x;
          }
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          u32x4_t qa;
          if constexpr (QLDS)
            qa = ql[(r * QS + st) * 64];
          else
            qa = qf[r * QS + st];
#pragma unroll
          for (int tt = 0; tt < 2; ++tt) s[r][tt] = mfma_16x16x32<BF>(ka[tt], qa, s[r][tt]);
        }
      }
      if constexpr (!SH) {
        __builtin_amdgcn_sched_barrier(0);
        load_k(slot ^ 1);
        __builtin_amdgcn_sched_barrier(0);
      }

      const int tb = tile_base(t);
      const bool edge = is_edge(tb, there);
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int tt = 0; tt < 2; ++tt)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[r][tt][i] *= sc;
      if (edge) {
        const uint32_t mine = there >> (g * 4);
        const int j0 = tb + g * 4;
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int tt = 0; tt < 2; ++tt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int o = tt * 16 + i;
              const bool sees = ((mine >> o & 1) != 0) & (o <= pos[r] - j0) &
                                ((o > pos[r] - window - j0) | (o < sinks - j0));
              s[r][tt][i] = sees ? s[r][tt][i] : kNegInf;
            }
      }

      // ---- weights, in place of the scores, and their pairs
      u32x4_t pf[RT];
      bool moves = false;
      float top[RT];
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        float x = fmaxf(fmaxf(fmaxf(s[r][0][0], s[r][0][1]), fmaxf(s[r][0][2], s[r][0][3])),
                        fmaxf(fmaxf(s[r][1][0], s[r][1][1]), fmaxf(s[r][1][2], s[r][1][3])));
        top[r] = row_max(x);
        // (a difference, which is exact: m + 8 would round where scores pass 2^25)
        moves |= top[r] - m[r] > 8.0f + kHeadroom<BF>;
      }
      if (__any(moves)) {
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          const float mn = fmaxf(m[r], top[r] - kHeadroom<BF>);
          const float f = weight_of(m[r], mn);
          m[r] = mn;
          l[r] *= f;
#pragma unroll
          for (int e = 0; e < NE; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[r][e][i] *= f;
        }
      }
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const float mm = m[r] == kNegInf ? 0.0f : m[r];
        float sum = 0.0f;
#pragma unroll
        for (int tt = 0; tt < 2; ++tt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s[r][tt][i] = __builtin_amdgcn_exp2f(s[r][tt][i] - mm);
            sum += s[r][tt][i];
          }
        l[r] += sum;
        // weights leave fp32 here, for the matrix product: half a step of q's
        // type each, as much as the output's own rounding; in fp16 half of 2^-24
        // absolute below 2^-14, the largest weight being at least 2^7
        pf[r] = u32x4_t{pair_of<BF>(s[r][0][0], s[r][0][1]), pair_of<BF>(s[r][0][2], s[r][0][3]),
                        pair_of<BF>(s[r][1][0], s[r][1][1]), pair_of<BF>(s[r][1][2], s[r][1][3])};
      }

      // ---- values
      if constexpr (SH) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint8_t *p = values + ((j >> 2) * 16 + (at >> 4) * 4 + (j & 3)) * T::ROW + (at & 15) * (E * CB);
#pragma unroll
          for (int x = 0; x < VH; ++x) load_words<false, VW>(p + x * (128 * CB), vt[x][j]);
        }
      }
      if (edge) {
        // a token that is not there, or that only some rows see, may hold
        // anything, and 0 times a NaN or an infinity is not 0: these are taken
        // out here and given to the rows that see them after the tiles
        uint32_t odd = 0;
        const uint32_t mine = there >> (g * 4);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t ok = 0u - (mine >> ((j >> 2) * 16 + (j & 3)) & 1u);
#pragma unroll
          for (int x = 0; x < VH; ++x)
#pragma unroll
            for (int y = 0; y < VW; ++y) {
              vt[x][j][y] &= ok;
              odd |= nonfinite_signs<BF, F8>(vt[x][j][y]);
            }
        }
        if (__any((odd & kSigns<F8>) != 0)) {
          strays = true;
#pragma unroll
          for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int x = 0; x < VH; ++x)
#pragma unroll
              for (int y = 0; y < VW; ++y) {
                asm volatile("" : "+v"(vt[x][j][y]));  // nothing kept from the test for this rare part
                vt[x][j][y] &= ~nonfinite<BF, F8>(vt[x][j][y]);
              }
        }
      }
      constexpr int PW = F8 ? 4 : 2;  // operands of one dword column
#pragma unroll
      for (int x = 0; x < VH; ++x)
#pragma unroll
        for (int y = 0; y < VW; ++y) {
          u32x4_t o[PW];
          turn<BF, F8, VW>(vt[x], y, o);
#pragma unroll
          for (int z = 0; z < PW; ++z)
#pragma unroll
            for (int r = 0; r < RT; ++r)
              acc[r][x * E + y * PW + z] = mfma_16x16x32<BF>(o[z], pf[r], acc[r][x * E + y * PW + z]);
        }
      if constexpr (!SH) {
        __builtin_amdgcn_sched_barrier(0);
        load_v(slot ^ 1);
        __builtin_amdgcn_sched_barrier(0);
      }
      slot ^= 1;
      there = there_next;
    }

    if (strays) {
      // The NaNs and infinities of the tiles above, to the rows that see their
      // tokens: lane (c, g) holds row c and, of each half of D, the 4 E
      // consecutive d from 4 E g on.
#pragma unroll 1
      for (int t2 = first * TW * ap->span + tw; t2 < t_end; t2 += TW) {
        const uint32_t present = put(t2, load_id(t2), 0);
        const int tb = tile_base(t2);
        if (!is_edge(tb, present)) continue;
#pragma unroll 1
        for (int o = 0; o < 32; ++o) {
          if (!(present >> o & 1)) continue;
          const uint8_t *p = vbase + my_ring[o] + g * 4 * E * CB;
          uint32_t sees[RT];
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            const int j = tb + o;
            sees[r] = (j <= pos[r]) & ((j > pos[r] - window) | (j < sinks)) ? ~0u : 0u;
            asm volatile("" : "+v"(sees[r]));  // a mask in a register, no select for each value
          }
#pragma unroll
          for (int x = 0; x < VH; ++x)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t v[VW];
              load_words<false, VW>(p + (x * 128 + k * E) * CB, v);
#pragma unroll
              for (int e = 0; e < E; ++e) {
                constexpr int PER = 4 / CB;
                const uint32_t word = v[e / PER];
                const bool is = nonfinite<BF, F8>(word) >> (e % PER * 8 * CB) & 1;
                const uint32_t val = is ? __builtin_bit_cast(uint32_t, value_of<BF, F8>(word, e % PER)) : 0u;
#pragma unroll
                for (int r = 0; r < RT; ++r)
                  acc[r][x * E + e][k] += __builtin_bit_cast(float, val & sees[r]);
              }
            }
        }
      }
    }

    // ---- the waves that shared the tokens: the upper half gives, the lower takes
    ap = reload(ap);
    if constexpr (!SH) __syncthreads();  // the queries and keys have been read
#pragma unroll
    for (int r = 0; r < RT; ++r) l[r] = row_sum(l[r]);
    for (int over = TW >> 1; over; over >>= 1) {
      const int seat = tw - over;  // of 2 at most
      if (tw >= over && tw < 2 * over) {
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          give_ml[((seat * RT + r) * 2 + 0) * 64 + lane] = m[r];
          give_ml[((seat * RT + r) * 2 + 1) * 64 + lane] = l[r];
#pragma unroll
          for (int e = 0; e < NE; ++e) give[((seat * RT + r) * NE + e) * 64 + lane] = acc[r][e];
        }
      }
      __syncthreads();
      if (tw < over) {
        const int from = tw;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          const float m2 = give_ml[((from * RT + r) * 2 + 0) * 64 + lane];
          const float l2 = give_ml[((from * RT + r) * 2 + 1) * 64 + lane];
          const float mn = fmaxf(m[r], m2);
          const float f1 = weight_of(m[r], mn), f2 = weight_of(m2, mn);
          m[r] = mn;
          // (which product is rounded is written out: the compiler's choice changes
          // with the code around it)
          l[r] = __builtin_fmaf(l[r], f1, l2 * f2);
#pragma unroll
          for (int e = 0; e < NE; ++e) {
            const f32x4_t y = give[((from * RT + r) * NE + e) * 64 + lane];
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[r][e][i] = __builtin_fmaf(y[i], f2, acc[r][e][i] * f1);
          }
        }
      }
      __syncthreads();
    }

    // ---- write: lane (c, g) has row c and, in each half of D, the 4 E
    // consecutive d from 4 E g on
    if (tw == 0) {
      const int G = ap->G;
      const float vs = ap->c.v_scale ? constant(ap->c.v_scale)[h] : 1.0f;
      // a part that does not begin its item is its workgroup's first, one that
      // begins it and does not end it is its last
      int64_t part = 2 * (int64_t)wg + (first == 0 ? 1 : 0);
      const bool whole = n_granules == w.granules;
      // (what others walked has to be joined to it, so it is a part in any case)
      if (PRE && whole)
        part = 2 * (int64_t)ap->workgroups + (int64_t)b * ap->seq_items + h * (ap->seq_items / ap->c.H) + group;
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const int row = row_first + r * 16 + c;
        if (row >= R) continue;
        if (!PRE && whole) {
          const int i = row / G, hq = h * G + row - i * G;
          const float f = l[r] == 0.0f ? 0.0f : vs / l[r];
          uint8_t *o = ap->out + (int64_t)(w.row0 + i) * ap->out_row + hq * ap->out_head;
#pragma unroll
          for (int x = 0; x < VH; ++x)
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int e = 0; e < E; e += 4) {
                uint2 y;
                y.x = pair_of<BF>(acc[r][x * E + e][k] * f, acc[r][x * E + e + 1][k] * f);
                y.y = pair_of<BF>(acc[r][x * E + e + 2][k] * f, acc[r][x * E + e + 3][k] * f);
                *reinterpret_cast<uint2 *>(o + (x * 128 + (g * 4 + k) * E + e) * 2) = y;
              }
          if (ap->lse && g == 0)
            ap->lse[(int64_t)(w.row0 + i) * (ap->c.H * G) + hq] =
                l[r] == 0.0f ? kNegInf : log_of<BF>(m[r], l[r]);
        } else {
          const int64_t at = (part * CHUNKS + chunk) * RT * 16 + r * 16 + c;
          float *o = ap->part + at * D;
#pragma unroll
          for (int x = 0; x < VH; ++x)
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int e = 0; e < E; e += 4)
                *reinterpret_cast<f32x4_t *>(o + x * 128 + (g * 4 + k) * E + e) =
                    f32x4_t{acc[r][x * E + e][k], acc[r][x * E + e + 1][k], acc[r][x * E + e + 2][k],
                            acc[r][x * E + e + 3][k]};
          if (g == 0) {
            ap->ml[at * 2] = m[r];
            ap->ml[at * 2 + 1] = l[r];
          }
        }
      }
    }
  }
}

template <bool BF, bool F8, int D, int RT, bool SH, int OCC, bool PRE = false>
__global__ __launch_bounds__(256, OCC) void attend_kernel(AttendArgs) {
  extern __shared__ __align__(16) uint8_t lds[];
  attend_body<BF, F8, D, RT, SH, PRE>(kern_args(), lds, blockIdx.x, gridDim.x);
}

// The parts of the common tokens (qgemv_prefix_impl.h): an item is 128 rows of a
// head of all the call's, and has n granules; workgroups take per of them each.
// Where there are workgroups for several parts of each item, n is filled up to
// whole parts.
struct PrefixPlan {
  int n, per;
  int most;  // parts that an item can have
};

template <class Args>
__device__ __forceinline__ PrefixPlan prefix_plan(Args &a) {
  PrefixPlan p;
  p.n = a.pre_plan[0];
  p.per = a.pre_plan[1];
  p.most = p.n ? min((p.n + p.per - 2) / p.per + 1, a.pre_most) : 0;
  return p;
}

// Where a row's first part is, and how many it has; the next are a.pre_rows
// further on.
template <class Args>
__device__ __forceinline__ int64_t prefix_parts(Args &a, const PrefixPlan &p, int h, int row, int *count) {
  const int tile = (int)((uint32_t)row / (uint32_t)a.pre_rows), item = h * a.pre_tiles + tile;
  const uint32_t g0 = (uint32_t)item * (uint32_t)p.n;
  *count = p.n ? (int)((g0 + p.n - 1) / (uint32_t)p.per - g0 / (uint32_t)p.per) + 1 : 0;
  return (int64_t)item * a.pre_most * a.pre_rows + row - tile * a.pre_rows;
}

// Joins the parts of the items that several workgroups shared.  A team of D / 4
// threads takes a row and all or every 8th of its parts, in order, with a
// running maximum; teams of one row are joined in order through LDS.
//
// PRE: all items, with the parts of the tokens before them.
template <bool BF, int D, bool PRE = false>
__global__ __launch_bounds__(256) void join_kernel(AttendArgs a) {
  constexpr int TEAM = D / 4, TEAMS = 256 / TEAM;
  const int item_rows = (a.shared ? 4 : 1) * a.rt * 16;
  const int groups_max = (a.M * a.G + item_rows - 1) / item_rows;
  const int b = blockIdx.x / (a.c.H * groups_max), hg = blockIdx.x - b * (a.c.H * groups_max);
  const SeqWork w = seq_work<PRE>(a, b, common_pages<PRE>(a) * a.c.page);
  const int groups = w.items ? w.groups : 0, h = hg / groups_max, group = hg - h * groups_max;
  if (group >= groups) return;
  const Split split = split_of<PRE>(a, a.plan[0], PRE ? a.pre_plan[2] : 0);
  const PrefixPlan pre = PRE ? prefix_plan(a) : PrefixPlan{};
  const int first_row = w.row0 * a.G + group * item_rows;  // of all rows of the call
  const int g0 = a.plan[1 + b] + (h * groups + group) * w.granules, g1 = g0 + w.granules;
  const int w0 = split_owner(split, g0), w1 = split_owner(split, g1 - 1);
  if (!PRE && w0 == w1) return;  // written by its workgroup
  const int rows = min(w.rows * a.G - group * item_rows, item_rows);
  const int own = w1 - w0 + 1, parts = own + pre.most;
  const int per_row = parts >= 2 * TEAMS ? TEAMS : 1;  // teams of a row
  const int team = threadIdx.x / TEAM, d = (threadIdx.x % TEAM) * 4;
  const int sub = team % per_row, at_once = TEAMS / per_row;
  __shared__ f32x4_t sums[256];
  __shared__ float stats[TEAMS][2];
  const float vs = a.c.v_scale ? constant(a.c.v_scale)[h] : 1.0f;
  for (int r0 = blockIdx.y * at_once; r0 < rows; r0 += gridDim.y * at_once) {
    const int row = r0 + team / per_row;
    float m = kNegInf, l = 0.0f;
    f32x4_t acc = {0, 0, 0, 0};
    if (row < rows) {
      int has = parts, prefix = 0;
      int64_t prefix_at = 0;
      if constexpr (PRE) {
        prefix_at = prefix_parts(a, pre, h, first_row + row, &prefix);
        has = own + prefix;
      }
#pragma unroll 4
      for (int i = sub; i < has; i += per_row) {
        int64_t at = (2 * (int64_t)(w0 + i) + (i == 0 ? 1 : 0)) * item_rows + row;
        const float *ml = a.ml, *part = a.part;
        if constexpr (PRE) {
          // (selected, not branched to: the loads of several parts are on their way)
          const bool common = i >= own;
          if (own == 1) at = (2 * (int64_t)a.workgroups + blockIdx.x) * item_rows + row;
          at = common ? prefix_at + (int64_t)(i - own) * a.pre_rows : at;
          ml = common ? a.pre_ml : ml;
          part = common ? a.pre_part : part;
        }
        const float m2 = ml[at * 2], l2 = ml[at * 2 + 1];
        const f32x4_t y = *reinterpret_cast<const f32x4_t *>(part + at * D + d);
        const float mn = fmaxf(m, m2), f1 = weight_of(m, mn), f2 = weight_of(m2, mn);
        m = mn;
        l = l * f1 + l2 * f2;
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[k] = acc[k] * f1 + y[k] * f2;
      }
    }
    if (per_row > 1) {  // one row in flight
      if (d == 0) {
        stats[team][0] = m;
        stats[team][1] = l;
      }
      sums[threadIdx.x] = acc;
      __syncthreads();
      if (team == 0) {
        for (int i = 1; i < per_row; ++i) {
          const float m2 = stats[i][0], l2 = stats[i][1];
          const f32x4_t y = sums[i * TEAM + threadIdx.x];
          const float mn = fmaxf(m, m2), f1 = weight_of(m, mn), f2 = weight_of(m2, mn);
          m = mn;
          l = l * f1 + l2 * f2;
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[k] = acc[k] * f1 + y[k] * f2;
        }
      }
      __syncthreads();
    }
    if (row < rows && sub == 0) {
      const int r = group * item_rows + row, i = r / a.G, hq = h * a.G + r - i * a.G;
      const float f = l == 0.0f ? 0.0f : vs / l;
      uint2 y;
      y.x = pair_of<BF>(acc[0] * f, acc[1] * f);
      y.y = pair_of<BF>(acc[2] * f, acc[3] * f);
      *reinterpret_cast<uint2 *>(a.out + (int64_t)(w.row0 + i) * a.out_row + hq * a.out_head + d * 2) = y;
      if (a.lse && d == 0)
        a.lse[(int64_t)(w.row0 + i) * (a.c.H * a.G) + hq] =
            l == 0.0f ? kNegInf : log_of<BF>(m, l);
    }
  }
}

template <bool BF, int D, bool PRE>
int launch_join(const AttendArgs &a, hipStream_t stream) {
  hipLaunchKernelGGL((join_kernel<BF, D, PRE>), dim3(a.B * a.seq_items, a.row_splits), dim3(256), 0, stream, a);
  return hipGetLastError() == hipSuccess ? QGEMV_OK : QGEMV_EHIP;
}

template <bool BF, bool F8, int D, int RT, bool SH>
int launch_attend_rt(const AttendArgs &a, hipStream_t stream) {
  constexpr int OCC = attend_occupancy(F8, D, RT, SH);
  constexpr size_t bytes = attend_lds(F8, D, RT, SH);
  const auto kern = attend_kernel<BF, F8, D, RT, SH, OCC>;
  if (bytes > 64 * 1024 && !allow_max_dynamic_lds(reinterpret_cast<const void *>(kern))) return QGEMV_EHIP;
  hipLaunchKernelGGL(kern, dim3(a.workgroups), dim3(256), bytes, stream, a);
  if (hipGetLastError() != hipSuccess) return QGEMV_EHIP;
  return a.joins ? launch_join<BF, D, false>(a, stream) : QGEMV_OK;
}

template <bool BF, bool F8, int D, bool SH>
int launch_attend_d(const AttendArgs &a, hipStream_t stream) {
  if constexpr (D < 256) {
    if (a.rt == 3) return launch_attend_rt<BF, F8, D, 3, SH>(a, stream);
    if (a.rt == 4) return launch_attend_rt<BF, F8, D, 4, SH>(a, stream);
  }
  if constexpr (one_tile(F8, D, SH, false))
    if (a.rt == 1) return launch_attend_rt<BF, F8, D, 1, SH>(a, stream);
  return launch_attend_rt<BF, F8, D, 2, SH>(a, stream);
}

template <bool BF, bool F8>
int launch_attend_t(const AttendArgs &a, hipStream_t stream) {
  switch (a.c.D) {
    case 64: return a.shared ? launch_attend_d<BF, F8, 64, true>(a, stream) : launch_attend_d<BF, F8, 64, false>(a, stream);
    case 128: return a.shared ? launch_attend_d<BF, F8, 128, true>(a, stream) : launch_attend_d<BF, F8, 128, false>(a, stream);
  }
  return a.shared ? launch_attend_d<BF, F8, 256, true>(a, stream) : launch_attend_d<BF, F8, 256, false>(a, stream);
}

}  // namespace qgemv
