// Low-rank adapters of many requests beside a shared projection.
//
//   out[t] = y[t] + scale[a] * B[a] (A[a] x[t]),  a = adapter[t]
//
// A [n][r][K] and B [n][N][r] are small beside the projection's own weights, and
// each that is used is read once for every tile of the rows that have it, and anew
// for every 512 rows of a call: rows of one adapter, wherever they are among the
// T, make tiles of 16, 32 or 64 and go through the matrix units together (of 16
// where larger ones would leave CUs without work: plan_adapt).  Two launches: the
// first product with K cut over workgroups, whose partial sums the second adds
// up in order.  Each workgroup finds the rows of its tile by itself among the
// adapters of all rows (512 at most in a call of the kernels).
//
// The sums of the first product enter the second in parts of the weights' type,
// three in bf16 and two in fp16, which have all their 24 bits (fp16: 22 of the
// row's largest, for which the row is scaled by a power of two first).
//
// Bound by memory where there is work, by latency where there is little.  On an
// MI355X: 5 rows of one request, rank 16, 5120 to 6144: 4.2 + 4.4 us; 438 rows of
// 64 requests, 31 adapters of rank 64, 5120 to 17408: 14 + 32 us for 25 MB (A 20,
// x 5) and 130 MB (B 69, y and out 30.5 each); by the counters 31 and 151 past L2.

#include <algorithm>
#include <type_traits>

#include "qgemv_attend_impl.h"

namespace qgemv {

namespace {

// Rows of tile `tile`, of up to 16 RT rows of one adapter: their number, and
// the rows themselves in rows[].  Adapters in the order of their first rows;
// rows without one come last where `rest` asks for them (adapter -1).
template <int NC>
__device__ __forceinline__ int find_rows(const int32_t *adapter, int T, int n, bool rest, int tile, int size,
                                         int lane, int *rows, int *which) {
  int mine[NC];
  uint64_t left[NC], none[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int t = i * 64 + lane;
    mine[i] = t < T ? adapter[t] : -1;
    const bool has = (uint32_t)mine[i] < (uint32_t)n;
    left[i] = __ballot(t < T && has);
    none[i] = __ballot(t < T && !has);
  }
  bool last = false;
  while (true) {
    int a = -1;
    uint64_t mask[NC];
    int count = 0;
    bool found = false;
#pragma unroll
    for (int i = 0; i < NC; ++i)
      if (!found && left[i]) {
        a = __builtin_amdgcn_readlane(mine[i], (int)__ffsll((long long)left[i]) - 1);
        found = true;
      }
    if (!found) {
      if (last || !rest) return 0;
      last = true;
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      mask[i] = found ? __ballot(mine[i] == a) & left[i] : none[i];
      left[i] &= ~mask[i];
      count += __popcll(mask[i]);
    }
    const int tiles = (count + size - 1) / size;
    if (tile < tiles) {
      *which = a;
      int rank = -tile * size;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int at = rank + (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(mask[i] >> 32),
                                                             __builtin_amdgcn_mbcnt_lo((uint32_t)mask[i], 0));
        if ((mask[i] >> lane & 1) && at >= 0 && at < size) rows[at] = i * 64 + lane;
        rank += __popcll(mask[i]);
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      return min(count - tile * size, size);
    }
    tile -= tiles;
  }
}

// The same for up to 64 rows, a lane's row beside all: the rows that share its
// adapter are those whose adapters agree in every bit, the first of them counts
// their tiles.  (64 adapters of a row each: 13 us, 24 with a step for each
// adapter before the tile's.)
template <int S>
__device__ __forceinline__ int find_rows_wave(const int32_t *adapter, int T, int n, bool rest, int tile, int lane,
                                              int *rows, int *which) {
  const int mine = lane < T ? adapter[lane] : -1;
  const bool has = (uint32_t)mine < (uint32_t)n;
  const uint64_t none = __ballot(lane < T && !has);
  uint64_t same = __ballot(has);
  for (int bits = n - 1, bit = 0; bits >> bit; ++bit) {
    const bool is = mine >> bit & 1;
    const uint64_t with = __ballot(is);
    same &= is ? with : ~with;
  }
  const bool leads = has && (int)__ffsll((long long)same) - 1 == lane;
  const int tiles = leads ? (__popcll(same) + S - 1) / S : 0;
  int in = tiles;  // sums over the lanes up to each
  in += __builtin_amdgcn_update_dpp(0, in, 0x111, 0xF, 0xF, false);
  in += __builtin_amdgcn_update_dpp(0, in, 0x112, 0xF, 0xF, false);
  in += __builtin_amdgcn_update_dpp(0, in, 0x114, 0xF, 0xF, false);
  in += __builtin_amdgcn_update_dpp(0, in, 0x118, 0xF, 0xF, false);
  in += __builtin_amdgcn_update_dpp(0, in, 0x142, 0xA, 0xF, false);
  in += __builtin_amdgcn_update_dpp(0, in, 0x143, 0xC, 0xF, false);
  const uint64_t hit = __ballot(leads && tile >= in - tiles && tile < in);
  uint64_t mask = none;
  int first = (tile - __builtin_amdgcn_readlane(in, 63)) * S;
  *which = -1;
  if (hit) {
    const int from = (int)__ffsll((long long)hit) - 1;
    *which = __builtin_amdgcn_readlane(mine, from);
    mask = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(same >> 32), from) << 32 |
           (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)same, from);
    first = (tile - __builtin_amdgcn_readlane(in - tiles, from)) * S;
  } else if (!rest) {
    return 0;
  }
  const int count = __popcll(mask) - first;
  if (count <= 0) return 0;
  const int at = (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0)) - first;
  if ((mask >> lane & 1) && at >= 0 && at < S) rows[at] = lane;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  return min(count, S);
}

// The same by the whole workgroup for more rows, of at most kMapped adapters: a
// bit for each row and adapter in LDS, whose counts give the tiles (adapters in
// their own order).  64 adapters among 512 rows: one pass of some steps where the
// ballots above take one for each adapter before the tile's.
constexpr int kMapped = 256;
constexpr int kMapRow = kAdaptRows / 32 + 1;  // words of an adapter, one to spare: threads of neighbours in different banks

__device__ int find_rows_mapped(const int32_t *adapter, int T, int n, bool rest, int tile, int size,
                                uint32_t (*map)[kMapRow], int *words, int *rows, int *which) {
  constexpr int W = kAdaptRows / 32;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int total = n + 1;  // the last: rows without an adapter
  int mine[kAdaptRows / 256];
#pragma unroll
  for (int i = 0; i < kAdaptRows / 256; ++i) {
    const int t = i * 256 + tid;
    mine[i] = t < T ? adapter[t] : -1;
    mine[i] = (uint32_t)mine[i] < (uint32_t)n ? mine[i] : t < T && rest ? n : -1;
  }
  for (int i = tid; i < total * kMapRow; i += 256) (&map[0][0])[i] = 0;
  if (tid == 0) words[4] = -1;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kAdaptRows / 256; ++i) {
    const int t = i * 256 + tid;
    if (mine[i] >= 0) atomicOr(&map[mine[i]][t >> 5], 1u << (t & 31));
  }
  __syncthreads();
  // thread a has adapter a, and thread 0 the last besides
  int count = 0, last = 0;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    if (tid < n) count += __popc(map[tid][i]);
    last += __popc(map[n][i]);
  }
  const int tiles = (count + size - 1) / size;
  int in = tiles;  // sums over the lanes up to each
  in += __builtin_amdgcn_update_dpp(0, in, 0x111, 0xF, 0xF, false);
  in += __builtin_amdgcn_update_dpp(0, in, 0x112, 0xF, 0xF, false);
  in += __builtin_amdgcn_update_dpp(0, in, 0x114, 0xF, 0xF, false);
  in += __builtin_amdgcn_update_dpp(0, in, 0x118, 0xF, 0xF, false);
  in += __builtin_amdgcn_update_dpp(0, in, 0x142, 0xA, 0xF, false);
  in += __builtin_amdgcn_update_dpp(0, in, 0x143, 0xC, 0xF, false);
  if (lane == 63) words[wave] = in;
  __syncthreads();
  const int w0 = words[0], w1 = words[1], w2 = words[2], w3 = words[3], all = w0 + w1 + w2 + w3;
  const int before = in - tiles + (wave > 0 ? w0 : 0) + (wave > 1 ? w1 : 0) + (wave > 2 ? w2 : 0);
  if (tile >= before && tile < before + tiles) {
    words[4] = tid;
    words[5] = tile - before;
    words[6] = count;
  }
  if (tid == 0 && tile >= all && tile < all + (last + size - 1) / size) {
    words[4] = n;
    words[5] = tile - all;
    words[6] = last;
  }
  __syncthreads();
  const int a = words[4], first = words[5] * size, rows_of = words[6];
  if (a < 0) return 0;
#pragma unroll
  for (int i = 0; i < kAdaptRows / 256; ++i) {
    if (mine[i] != a) continue;
    const int t = i * 256 + tid;
    int rank = -first;
#pragma unroll
    for (int k = 0; k < W; ++k) {
      const uint32_t below = k < (t >> 5) ? ~0u : k == (t >> 5) ? (1u << (t & 31)) - 1 : 0u;
      rank += __popc(map[a][k] & below);
    }
    if (rank >= 0 && rank < size) rows[rank] = t;
  }
  __syncthreads();
  *which = a == n ? -1 : a;
  return min(rows_of - first, size);
}

// Either, with the rows where each wave finds them; `scratch` is free afterwards.
constexpr size_t kMapBytes = ((kMapped + 1) * kMapRow * 4 + 32 + 15) / 16 * 16;

template <int NC, int S>
__device__ __forceinline__ int find(const AdaptArgs &a, bool rest, int lane, int wave, uint8_t *scratch, int *rows,
                                    int *which) {
  if constexpr (NC > 1) {
    if (a.n <= kMapped)
      return find_rows_mapped(a.adapter, a.T, a.n, rest, blockIdx.x, S,
                              reinterpret_cast<uint32_t(*)[kMapRow]>(scratch + 32),
                              reinterpret_cast<int *>(scratch), rows, which);
  }
  if constexpr (NC == 1)
    return find_rows_wave<S>(a.adapter, a.T, a.n, rest, blockIdx.x, lane, rows + wave * S, which);
  else
    return find_rows<NC>(a.adapter, a.T, a.n, rest, blockIdx.x, S, lane, rows + wave * S, which);
}

// First product: part[split][t][i] = sum over the split's k of A[i][k] x[t][k].
// A wave takes RK tiles of 16 ranks; the waves of a workgroup cut its K once more
// and add up through LDS, where the bitmaps have been (64 rows by 64 ranks: 50 KB of
// it, 67 with both side by side, past the 64 that a kernel has without asking).
template <bool BF, int NC, int RT, int RK>
__global__ __launch_bounds__(256) void adapt_down_kernel(AdaptArgs a) {
  __shared__ int all_rows[4 * 16 * RT];
  constexpr size_t kSums = (size_t)3 * RT * RK * 64 * sizeof(f32x4_t);
  __shared__ __align__(16) uint8_t scratch[NC > 1 && kMapBytes > kSums ? kMapBytes : kSums];
  static_assert(sizeof(all_rows) + sizeof(scratch) <= 64 * 1024, "LDS that a kernel has without asking");
  // (the search for the rows ends with a barrier)
  f32x4_t(*const sums)[RT * RK][64] = reinterpret_cast<f32x4_t(*)[RT * RK][64]>(scratch);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  int which = -1;
  const int count = __builtin_amdgcn_readfirstlane(find<NC, 16 * RT>(a, false, lane, wave, scratch, all_rows, &which));
  if (count == 0) return;
  const int *const rows = NC > 1 && a.n <= kMapped ? all_rows : all_rows + wave * (16 * RT);
  which = __builtin_amdgcn_readfirstlane(which);
  const int steps = (a.K + 31) / 32, waves = a.splits * 4;
  const int per = (steps + waves - 1) / waves;
  const int s0 = (blockIdx.y * 4 + wave) * per, s1 = min(s0 + per, steps);
  const int r0 = blockIdx.z * (16 * RK);
  const uint8_t *xr[RT], *ar[RK];
#pragma unroll
  for (int i = 0; i < RT; ++i) xr[i] = a.x + (int64_t)rows[min(i * 16 + c, count - 1)] * a.x_row * 2;
#pragma unroll
  for (int i = 0; i < RK; ++i) ar[i] = a.a + ((int64_t)which * a.r + min(r0 + i * 16 + c, a.r - 1)) * a.K * 2;
  f32x4_t acc[RT][RK];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < RK; ++j) acc[i][j] = f32x4_t{0, 0, 0, 0};
  // steps whose loads are on their way together
  constexpr int U = RT + RK <= 2 ? 8 : RT + RK <= 5 ? 4 : 2;
  for (int s = s0; s < s1; s += U) {
    u32x4_t w[U][RK], x[U][RT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = (s + u) * 32 + g * 8;
      const bool in = (s + u < s1) & (k < a.K);
      const int64_t at = in ? 2 * (int64_t)k : 0;
      const uint32_t keep = in ? ~0u : 0u;
#pragma unroll
      for (int j = 0; j < RK; ++j) w[u][j] = *reinterpret_cast<const u32x4_t *>(ar[j] + at) & keep;
#pragma unroll
      for (int i = 0; i < RT; ++i) x[u][i] = *reinterpret_cast<const u32x4_t *>(xr[i] + at) & keep;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < RK; ++j)
          acc[i][j] = mfma_16x16x32<BF>(w[u][j], x[u][i], acc[i][j]);  // lane (c, g): row c, ranks 4 g ..
  }
  if (wave > 0)
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < RK; ++j) sums[wave - 1][i * RK + j][lane] = acc[i][j];
  __syncthreads();
  if (wave > 0) return;
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < RK; ++j) {
#pragma unroll
      for (int w = 0; w < 3; ++w)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[i][j][k] += sums[w][i * RK + j][lane][k];
      const int r = r0 + j * 16 + g * 4;
      if (i * 16 + c < count && r < a.r)
        *reinterpret_cast<f32x4_t *>(a.part + ((int64_t)blockIdx.y * a.T + rows[i * 16 + c]) * a.r + r) = acc[i][j];
    }
}

// The most rank tiles of a wave of the first product: up to 64 rows make at most
// six tiles of 32 rows and three of 64, with which more would leave CUs without a
// workgroup (plan_adapt's rule on 256 CUs comes to this by itself).
constexpr int adapt_ranks(bool many_rows, int rt) { return many_rows ? 4 : 4 / rt; }

typedef float f32x4_free_t __attribute__((ext_vector_type(4), aligned(4)));

// Second product and the sum.  STEPS of 32 ranks; a wave takes NB tiles of 16
// columns at a time, whose loads, and those of y, are on their way together.
template <bool BF, int NC, int RT, int STEPS>
__global__ __launch_bounds__(256) void adapt_up_kernel(AdaptArgs a) {
  constexpr int S = 16 * RT, NB = STEPS > 2 ? 2 : 4;
  constexpr int W = STEPS * 32 + 8;  // values of a row in LDS: 16 bytes past whole banks
  constexpr int PARTS = BF ? 3 : 2;
  extern __shared__ __align__(16) uint8_t lds[];  // rows of each wave's tile, what a row's sums are scaled by, the sums
  int *const all_rows = reinterpret_cast<int *>(lds);
  float *const back = reinterpret_cast<float *>(lds + 16 * S);
  uint16_t *const sums = reinterpret_cast<uint16_t *>(lds + 20 * S);  // [PARTS][S][W]
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  int which = -1;
  const int count = __builtin_amdgcn_readfirstlane(find<NC, S>(a, a.out != a.y, lane, wave, lds + 20 * S, all_rows, &which));
  if (count == 0) return;
  const int *const rows = NC > 1 && a.n <= kMapped ? all_rows : all_rows + wave * S;
  which = __builtin_amdgcn_readfirstlane(which);
  // lane (c, g) has row c of each 16, columns n0 + 16 j + 4 g ..: of y, and of B
  // the rows n0 + 16 j + c
  const uint8_t *const b = a.b + (int64_t)max(which, 0) * a.N * a.r * 2;
  const int blocks = (a.N + NB * 16 - 1) / (NB * 16);
  f32x4_free_t y[RT][NB];
  u32x4_t w[NB][STEPS];
  auto load = [&](int n) {
    const int n0 = n * (NB * 16);
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const float *const p = a.y + rows[min(i * 16 + c, count - 1)] * a.y_row;
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const int col = n0 + j * 16 + g * 4;
        if (col + 4 <= a.N) {
          y[i][j] = *reinterpret_cast<const f32x4_free_t *>(p + col);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) y[i][j][k] = p[min(col + k, a.N - 1)];
        }
      }
    }
    if (which < 0) return;
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        const int k = s * 32 + g * 8;
        w[j][s] = *reinterpret_cast<const u32x4_t *>(
            b + ((int64_t)min(n0 + j * 16 + c, a.N - 1) * a.r + (k < a.r ? k : 0)) * 2);
      }
  };
  // the first columns, on their way while the sums are put together
  int n = blockIdx.y * 4 + wave;
  load(min(n, blocks - 1));
  if (which >= 0) {
    const float scale = a.scales ? a.scales[which] : 1.0f;
    // 16 lanes a row, which cut its ranks
    for (int i = threadIdx.x >> 4; i < S; i += 16) {
      const float *const p = a.part + (int64_t)rows[min(i, count - 1)] * a.r;
      constexpr int Q = (STEPS + 1) / 2;  // fours of a lane
      f32x4_t v[Q];
      float most = 0.0f;
#pragma unroll
      for (int x = 0; x < Q; ++x) {
        const int k = (x * 16 + c) * 4;
        // the most parts that there can be, on their way together
        f32x4_t part[kAdaptSplits];
#pragma unroll
        for (int s = 0; s < kAdaptSplits; ++s)
          part[s] = *reinterpret_cast<const f32x4_t *>(p + (int64_t)min(s, a.splits - 1) * a.T * a.r + (k < a.r ? k : 0));
        v[x] = f32x4_t{0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < kAdaptSplits; ++s)
#pragma unroll
          for (int j = 0; j < 4; ++j) v[x][j] += s < a.splits && k < a.r ? part[s][j] : 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) most = fmaxf(most, __builtin_fabsf(v[x][j]));
      }
      int up = 0;
      if constexpr (!BF) {  // scaled to 2^13 .. 2^14
        auto ror = [](float x, auto by) {
          return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), decltype(by)::value, 0xF, 0xF, true));
        };
        most = fmaxf(most, ror(most, std::integral_constant<int, 0x128>{}));
        most = fmaxf(most, ror(most, std::integral_constant<int, 0x124>{}));
        most = fmaxf(most, ror(most, std::integral_constant<int, 0x122>{}));
        most = fmaxf(most, ror(most, std::integral_constant<int, 0x121>{}));
        up = most > 0.0f && __builtin_isfinite(most) ? min(14 - __builtin_amdgcn_frexp_expf(most), 120) : 0;
      }
#pragma unroll
      for (int x = 0; x < Q; ++x) {
        const int k = (x * 16 + c) * 4;
        if constexpr (!BF)
#pragma unroll
          for (int j = 0; j < 4; ++j) v[x][j] = __builtin_amdgcn_ldexpf(v[x][j], up);
#pragma unroll
        for (int q = 0; q < PARTS; ++q) {
          float top[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            top[j] = BF ? (float)(__bf16)v[x][j] : (float)(_Float16)v[x][j];
            v[x][j] = __builtin_isfinite(top[j]) ? v[x][j] - top[j] : 0.0f;
          }
          if (k < STEPS * 32)
            *reinterpret_cast<uint2 *>(sums + (q * S + i) * W + k) = make_uint2(pair_of<BF>(top[0], top[1]), pair_of<BF>(top[2], top[3]));
        }
      }
      if (c == 0) back[i] = BF ? scale : __builtin_amdgcn_ldexpf(scale, -up);
    }
    __syncthreads();
  }
  while (n < blocks) {
    const int n0 = n * (NB * 16);
    if (which >= 0) {
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        const uint32_t keep = s * 32 + g * 8 < a.r ? ~0u : 0u;
#pragma unroll
        for (int j = 0; j < NB; ++j) w[j][s] &= keep;
      }
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        f32x4_t acc[NB];
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[j] = f32x4_t{0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
#pragma unroll
          for (int q = 0; q < PARTS; ++q) {
            const u32x4_t v = *reinterpret_cast<const u32x4_t *>(sums + (q * S + i * 16 + c) * W + s * 32 + g * 8);
#pragma unroll
            for (int j = 0; j < NB; ++j) acc[j] = mfma_16x16x32<BF>(w[j][s], v, acc[j]);
          }
        const float f = back[i * 16 + c];
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k) y[i][j][k] += f * acc[j][k];
      }
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      if (i * 16 + c >= count) continue;
      float *const p = a.out + rows[i * 16 + c] * a.out_row;
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const int col = n0 + j * 16 + g * 4;
        if (col + 4 <= a.N) {
          *reinterpret_cast<f32x4_free_t *>(p + col) = y[i][j];
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (col + k < a.N) p[col + k] = y[i][j][k];
        }
      }
    }
    n += gridDim.y * 4;
    if (n < blocks) load(n);
  }
}

template <bool BF, int NC, int RT, int STEPS>
int launch_adapt_up(const AdaptArgs &a, hipStream_t stream) {
  constexpr size_t bytes = (size_t)16 * RT * 20 + std::max((size_t)16 * RT * 2 * (BF ? 3 : 2) * (STEPS * 32 + 8), NC > 1 ? kMapBytes : 0);
  constexpr int columns = STEPS > 2 ? 128 : 256;  // of a workgroup
  const auto kern = adapt_up_kernel<BF, NC, RT, STEPS>;
  if (bytes > 64 * 1024 && !allow_max_dynamic_lds(reinterpret_cast<const void *>(kern))) return QGEMV_EHIP;
  const int blocks = (a.N + columns - 1) / columns, want = std::max(1, 4 * device_cu_count() / a.tiles);
  hipLaunchKernelGGL(kern, dim3(a.tiles, std::min(blocks, want)), dim3(256), bytes, stream, a);
  return hipGetLastError() == hipSuccess ? QGEMV_OK : QGEMV_EHIP;
}

template <bool BF, int NC, int RT>
int launch_adapt_rt(const AdaptArgs &a, hipStream_t stream) {
  const dim3 grid(a.tiles, a.splits, (a.r + 16 * a.rk - 1) / (16 * a.rk)), block(256);
  constexpr int most = adapt_ranks(NC > 1, RT);
  if (a.rk == 1) {
    hipLaunchKernelGGL((adapt_down_kernel<BF, NC, RT, 1>), grid, block, 0, stream, a);
  } else if (a.rk == 2) {
    if constexpr (most >= 2) hipLaunchKernelGGL((adapt_down_kernel<BF, NC, RT, 2>), grid, block, 0, stream, a);
  } else {
    if constexpr (most >= 4) hipLaunchKernelGGL((adapt_down_kernel<BF, NC, RT, 4>), grid, block, 0, stream, a);
  }
  if (hipGetLastError() != hipSuccess) return QGEMV_EHIP;
  return a.r <= 32 ? launch_adapt_up<BF, NC, RT, 1>(a, stream)
         : a.r <= 64 ? launch_adapt_up<BF, NC, RT, 2>(a, stream)
         : a.r <= 128 ? launch_adapt_up<BF, NC, RT, 4>(a, stream)
                      : launch_adapt_up<BF, NC, RT, 8>(a, stream);
}

template <bool BF, int NC>
int launch_adapt_nc(const AdaptArgs &a, hipStream_t stream) {
  return a.rt == 1 ? launch_adapt_rt<BF, NC, 1>(a, stream)
         : a.rt == 2 ? launch_adapt_rt<BF, NC, 2>(a, stream)
                     : launch_adapt_rt<BF, NC, 4>(a, stream);
}

template <bool BF>
int launch_adapt_t(const AdaptArgs &a, hipStream_t stream) {
  if (a.T <= 64) return launch_adapt_nc<BF, 1>(a, stream);
  return launch_adapt_nc<BF, kAdaptRows / 64>(a, stream);
}

}  // namespace

// Workgroups of the first product for each CU, counted as if every tile were there
// (2, 4 and 8: parts that the second product has to read as well; the 438 rows above
// 41.3 us with 1, 44.5 with 8).
constexpr int kAdaptFill = 1;

int64_t plan_adapt(AdaptArgs *a) {
  const int each = (a->T - 1) / a->n + 1;  // rows of an adapter, where all have as many
  a->rt = each <= 16 ? 1 : each <= 32 ? 2 : 4;
  // the most tiles: every adapter, and the rows without one, end in a part of one
  const auto tiles = [&] { return std::min(a->T, a->T / (16 * a->rt) + std::min(a->n, a->T - 1) + 1); };
  const int columns = a->r <= 64 ? 256 : 128;  // of a workgroup of the second product
  // Larger tiles read an adapter less often, smaller ones make more workgroups of
  // the second product, which are wanted up to the four that a CU has (us, as the
  // rows of an adapter say and so: 64 rows of one adapter of rank 16, 5120 to 6144,
  // 16.8 and 8.9; of rank 128 to 17408 20.1 and 14.6; 512 rows of 8 of rank 64 to
  // 6144 29 and 25, of one to 17408 35 and 31).
  while (a->rt > 1 && tiles() * ((a->N + columns - 1) / columns) < 4 * device_cu_count()) a->rt /= 2;
  a->tiles = tiles();
  a->rk = a->r <= 16 ? 1 : a->r <= 32 ? 2 : 4;
  // Fewer ranks a wave read x more often, and leave no CU without a workgroup of the
  // first product (5 rows of rank 128, 17408 to 5120: 17.2 us with 4 tiles of ranks,
  // 12.3 so; for two a CU 512 rows of 16 adapters of rank 64 lose, 35 and 41).
  a->rk = std::min(a->rk, adapt_ranks(a->T > 64, a->rt));
  while (a->rk > 1 && a->tiles * ((a->r + 16 * a->rk - 1) / (16 * a->rk)) * kAdaptSplits < device_cu_count()) a->rk /= 2;
  const int ranks = (a->r + 16 * a->rk - 1) / (16 * a->rk), steps = (a->K + 31) / 32;
  a->splits = std::max(1, std::min({kAdaptSplits, steps / 8, kAdaptFill * device_cu_count() / (a->tiles * ranks)}));
  // the most splits: so the size grows with T and r alone
  return (int64_t)4 * kAdaptSplits * a->T * a->r;
}

int launch_adapt(const AdaptArgs &a, hipStream_t stream) {
  return a.dtype == QGEMV_BF16 ? launch_adapt_t<true>(a, stream) : launch_adapt_t<false>(a, stream);
}

}  // namespace qgemv
