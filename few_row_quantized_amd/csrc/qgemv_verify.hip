// Acceptance of drafted tokens and the draw of the next one.
//
// Row t of a sequence holds the target's probabilities p[t] after the token
// fed there; the draft checked against it is the token of row t + 1.  A draft
// d is accepted while u[t] * q[t][d] < p[t][d] (u uniform, q the draft model's
// probability, 1 without one).  At the first refusal, row r, the token is
// drawn from w = max(p[r] - q[r], 0) (without q: p[r] but for the refused
// token; p[r] itself where nothing is left); with no refusal from w = p of
// the last row.  The draw is the first token whose running sum passes
// u[last row] * sum(w).
//
// Products and sums are taken in 64 bits: u * q of two fp32 values is exact
// there, and a sum of 10^5 probabilities leaves a token's share of the number
// line where it is.
//
// One launch.  A row is cut into at most 256 pieces, whole loads of a wave, as
// its length alone says; each wave checks the drafts itself (they decide which
// row is summed; at most 15 pairs of loads, one a lane), sums its pieces and
// leaves the sums in the workspace.  The workgroup that arrives last at the
// sequence's counter scans the sums in order, finds the piece where the running
// sum passes the number, scans that piece again and writes the answer; it also
// sets the counter back to 0.  Neither which workgroup is last nor how many
// share a sequence changes a result.
//
// On an MI355X: one sequence of 32000 tokens 7 us, the latency of some eight
// loads that wait for one another; 64 of 151936 fp32 tokens with the drafts'
// probabilities 18 us (78 MB, 4.3 TB/s); 200 of 128257 bf16 tokens without
// them 20 us (51 MB), where nearly each load of a wave ends a piece of 512 in two
// wave sums and two stores past the caches.

#include "qgemv_kv.h"
#include "qgemv_device.h"

namespace qgemv {

namespace {

constexpr int kMaxPieces = 256;       // of a row: the last workgroup has one thread for each
constexpr int kMaxWorkgroups = 2048;  // all of them at once on the card, 8 on a CU
// Counters lie in lines of their own: atomics on one line are taken one after
// the other, some 10 ns each (32 sequences of 128257 bf16 tokens took 28 us).
constexpr int kCounterInts = 64;

template <int DT>
__device__ __forceinline__ float prob(const uint8_t *row, int i) {
  if constexpr (DT == QGEMV_F32) {
    return reinterpret_cast<const float *>(row)[i];
  } else {
    const uint32_t b = reinterpret_cast<const uint16_t *>(row)[i];
    return DT == QGEMV_BF16 ? bf16_bits_to_float(b) : half_bits_to_float(b);
  }
}

// 16 bytes of a row.  Rows start at any element (an odd vocabulary), so the
// load is only element-aligned; the hardware takes that.
template <int DT>
__device__ __forceinline__ u32x4_t load16(const uint8_t *row, int i) {
  u32x4_t w;
  __builtin_memcpy(&w, row + (int64_t)i * (DT == QGEMV_F32 ? 4 : 2), 16);
  return w;
}

// Element k of them.
template <int DT>
__device__ __forceinline__ float elem(u32x4_t w, int k) {
  if constexpr (DT == QGEMV_F32) {
    const uint32_t b = w[k];  // (a bit cast of the element itself takes the vector's first)
    return __builtin_bit_cast(float, b);
  }
  const uint32_t b = k & 1 ? w[k >> 1] >> 16 : w[k >> 1] & 0xFFFFu;
  return DT == QGEMV_BF16 ? bf16_bits_to_float(b) : half_bits_to_float(b);
}

// x of the lane that a DPP control names.
template <int CTRL>
__device__ __forceinline__ double dpp_lane(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)b, CTRL, 0xF, 0xF, true);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(b >> 32), CTRL, 0xF, 0xF, true);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ double pair_sum(uint32_t lo0, uint32_t lo1, uint32_t hi0, uint32_t hi1) {
  return __builtin_bit_cast(double, (uint64_t)hi0 << 32 | lo0) + __builtin_bit_cast(double, (uint64_t)hi1 << 32 | lo1);
}

// The sum over the wave, in every lane, without the LDS permutes: a wave sums
// a pair of numbers for each piece, and 24 permutes a piece bound the kernel
// (200 rows of 128257 bf16 tokens: 25 us, 21 without them).
__device__ __forceinline__ double wave_sum(double x) {
  x += dpp_lane<0xB1>(x);   // the other of two
  x += dpp_lane<0x4E>(x);   // the other pair of four
  x += dpp_lane<0x141>(x);  // the other four of eight
  x += dpp_lane<0x140>(x);  // the other eight of sixteen
  uint64_t b = __builtin_bit_cast(uint64_t, x);
  const auto l16 = __builtin_amdgcn_permlane16_swap((uint32_t)b, (uint32_t)b, false, false);
  const auto h16 = __builtin_amdgcn_permlane16_swap((uint32_t)(b >> 32), (uint32_t)(b >> 32), false, false);
  x = pair_sum(l16[0], l16[1], h16[0], h16[1]);
  b = __builtin_bit_cast(uint64_t, x);
  const auto l32 = __builtin_amdgcn_permlane32_swap((uint32_t)b, (uint32_t)b, false, false);
  const auto h32 = __builtin_amdgcn_permlane32_swap((uint32_t)(b >> 32), (uint32_t)(b >> 32), false, false);
  return pair_sum(l32[0], l32[1], h32[0], h32[1]);
}

// Inclusive sums of x over the workgroup's threads; `part`: LDS of 4.
__device__ __forceinline__ double block_scan(double x, double *part, double *total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) {
    const double y = __shfl_up(x, s);
    if (lane >= s) x += y;
  }
  if (lane == 63) part[wave] = x;
  __syncthreads();
  double before = 0.0;
  for (int w = 0; w < wave; ++w) before += part[w];
  *total = part[0] + part[1] + part[2] + part[3];
  __syncthreads();
  return x + before;
}

// The lowest thread whose flag is set, 256 if none is; `part`: LDS of 4.
__device__ __forceinline__ int block_first(bool flag, int *part) {
  const uint64_t v = __ballot(flag);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v ? (int)__ffsll((long long)v) - 1 : 64;
  __syncthreads();
  int r = 256;
  for (int w = 3; w >= 0; --w)
    if (part[w] < 64) r = w * 64 + part[w];
  __syncthreads();
  return r;
}

// The highest thread whose flag is set, 0 if none is.
__device__ __forceinline__ int block_last(bool flag, int *part) {
  const uint64_t v = __ballot(flag);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v ? 63 - (int)__clzll((long long)v) : -1;
  __syncthreads();
  int r = 0;
  for (int w = 0; w < 4; ++w)
    if (part[w] >= 0) r = w * 64 + part[w];
  __syncthreads();
  return r;
}

// max(p - q, 0) that a NaN passes
__device__ __forceinline__ double rest_of(float p, float q) {
  const double d = (double)p - (double)q;
  return d < 0.0 ? 0.0 : d;
}

// A wave's pieces [first, last) of a row: sums of what is left of p, and of p
// itself, into the workspace.  Loads of U steps (64 lanes of 16 bytes) are in
// flight before the first of them is summed.
template <int DT, bool HAS_Q>
__device__ __forceinline__ void sum_pieces(const uint8_t *p, const uint8_t *q, int drop, int first, int last,
                                           int per, int V, double *sums) {
  constexpr int N = DT == QGEMV_F32 ? 4 : 8, U = HAS_Q ? 2 : 4, STEP = 64 * N;
  const int lane = threadIdx.x & 63, v_end = min(last * per, V);
  if (V < N) {  // no whole load: the first wave's first lane takes all
    if (first > 0 || lane > 0) return;
    double left = 0.0, all = 0.0;
    for (int v = 0; v < V; ++v) {
      const float z = prob<DT>(p, v);
      all += z;
      left += HAS_Q ? rest_of(z, prob<DT>(q, v)) : v == drop ? 0.0 : (double)z;
    }
    __hip_atomic_store(sums, left, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __hip_atomic_store(sums + 1, all, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return;
  }
  double left = 0.0, all = 0.0;
  int piece = first, edge = min((first + 1) * per, V);  // where the piece ends
  for (int v0 = first * per; v0 < v_end; v0 += U * STEP) {
    u32x4_t x[U], y[U];
#pragma unroll
    for (int s = 0; s < U; ++s) {
      const int i = v0 + s * STEP + lane * N;
      // a lane without a whole load takes the row's first (no load lies in a
      // branch, so that the compiler can count what is in flight)
      const int j = i + N <= v_end ? i : 0;
      x[s] = load16<DT>(p, j);
      if (HAS_Q) y[s] = load16<DT>(q, j);
    }
#pragma unroll
    for (int s = 0; s < U; ++s) {
      const int at = v0 + s * STEP, i = at + lane * N;
      double sum = 0.0, rest = 0.0;
      if (i + N <= v_end) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
          const float z = elem<DT>(x[s], k);
          sum += z;
          if (HAS_Q) rest += rest_of(z, elem<DT>(y[s], k));
        }
      } else {
        for (int v = i; v < v_end; ++v) {  // at most one lane holds the row's ragged end
          const float z = prob<DT>(p, v);
          sum += z;
          if (HAS_Q) rest += rest_of(z, prob<DT>(q, v));
        }
      }
      if (!HAS_Q) {
        rest = sum;
        if (drop >= i && drop < min(i + N, v_end)) {  // without its weight, never by a difference
          rest = 0.0;
          for (int v = i; v < min(i + N, v_end); ++v) rest += v == drop ? 0.0 : (double)prob<DT>(p, v);
        }
      }
      all += sum;
      left += rest;
      if (piece < last && at + STEP >= edge) {
        // stored past this XCD's caches, as agent-scope atomics are
        left = wave_sum(left);
        all = wave_sum(all);
        if (lane == 0) {
          __hip_atomic_store(sums + piece * 2, left, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          __hip_atomic_store(sums + piece * 2 + 1, all, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        left = all = 0.0;
        ++piece;
        edge = min(edge + per, V);
      }
    }
  }
}

template <int DT>
__global__ __launch_bounds__(256, 8) void verify_kernel(VerifyArgs a) {
  constexpr int SB = DT == QGEMV_F32 ? 4 : 2;
  const int b = blockIdx.x / a.slices, slice = blockIdx.x - b * a.slices;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int s0 = min(max(a.start[b], 0), a.T);
  const int rows = min(min(max(a.start[b + 1], s0), a.T) - s0, a.M);
  if (rows <= 0) {
    if (threadIdx.x == 0 && slice == 0) a.count[b] = 0;
    return;
  }
  int draft = -1;
  bool ok = false;
  if (lane < rows - 1) {
    const int t = s0 + lane;
    draft = a.tokens[t + 1];
    if (draft >= 0 && draft < a.V) {
      const double pd = prob<DT>(a.p + t * a.p_row * SB, draft);
      const double qd = a.q ? (double)prob<DT>(a.q + t * a.q_row * SB, draft) : 1.0;
      ok = (double)a.u[t] * qd < pd;
    }
  }
  const int n = min((int)__ffsll(~__ballot(ok)) - 1, rows - 1);  // drafts accepted before the first refusal
  const bool refused = n < rows - 1;
  const int drop = refused && !a.q ? __shfl(draft, n) : -1;
  const uint8_t *p = a.p + (s0 + n) * a.p_row * SB;
  const uint8_t *q = refused && a.q ? a.q + (s0 + n) * a.q_row * SB : nullptr;

  // ---- this wave's pieces
  double *const sums = a.sums + (int64_t)b * a.pieces * 2;
  const int first = (slice * 4 + wave) * a.each, last = min(first + a.each, a.pieces);
  if (q)
    sum_pieces<DT, true>(p, q, drop, first, last, a.per, a.V, sums);
  else
    sum_pieces<DT, false>(p, q, drop, first, last, a.per, a.V, sums);

  // ---- the last workgroup of the sequence goes on
  __shared__ double part[4];
  __shared__ int ints[4];
  if (a.slices > 1) {
    // Every wave waits until its sums have arrived, then the count goes up.  A
    // release on the counter would also write back this XCD's whole L2, one
    // workgroup after the other (64 sequences of 151936 tokens: 55 us, not 23).
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (threadIdx.x == 0) {
      const int before = __hip_atomic_fetch_add(a.arrived + b * kCounterInts, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      ints[0] = before == a.slices - 1;
      if (before == a.slices - 1)
        __hip_atomic_store(a.arrived + b * kCounterInts, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
  }
  __syncthreads();
  if (a.slices > 1) {
    const bool last = ints[0] != 0;
    __syncthreads();
    if (!last) return;
  }

  const bool has = (int)threadIdx.x < a.pieces;
  const double my_left =
      has ? __hip_atomic_load(sums + threadIdx.x * 2, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0.0;
  const double my_all =
      has ? __hip_atomic_load(sums + threadIdx.x * 2 + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0.0;
  double total, run = block_scan(my_left, part, &total);
  bool use_all = false;
  if (!(total > 0.0)) {
    use_all = true;
    run = block_scan(my_all, part, &total);
  }
  const double share = (double)a.u[s0 + rows - 1] * total;
  int token = a.V - 1;  // where no running sum passes the share
  if (!(share == share)) {
    token = 0;
  } else if (share < total) {
    // A running sum of the scan is rounded by the way its terms are grouped, so
    // that it may pass the share first at a place that adds nothing: pieces,
    // threads and tokens without a weight are never taken.
    const double my_sum = use_all ? my_all : my_left;
    int at = block_first(my_sum > 0.0 && run > share, ints);
    if (at == 256) at = block_last(my_sum > 0.0, ints);
    __shared__ double before_at;
    if ((int)threadIdx.x == at) before_at = run - my_sum;
    // the piece again, consecutive tokens a thread, four loads at a time
    const int a0 = at * a.per, a1 = min(a0 + a.per, a.V), each = (a.per + 255) / 256;
    const int t0 = min(a0 + (int)threadIdx.x * each, a1), t1 = min(t0 + each, a1);
    float x[4], y[4];
    auto load4 = [&](int v) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = min(v + k, a.V - 1);
        x[k] = prob<DT>(p, i);
        y[k] = q ? prob<DT>(q, i) : 0.0f;
      }
    };
    auto weight = [&](int v, int k) -> double {
      return use_all ? (double)x[k] : q ? rest_of(x[k], y[k]) : v + k == drop ? 0.0 : (double)x[k];
    };
    double mine = 0.0;
    int weighted = -1;  // the last token here that has a weight
    for (int v = t0; v < t1; v += 4) {
      load4(v);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (v + k >= t1) continue;
        const double w = weight(v, k);
        mine += w;
        if (w > 0.0) weighted = v + k;
      }
    }
    double ignored;
    double upto = block_scan(mine, part, &ignored);
    upto += before_at;  // after the scan's barriers
    const int who = block_first(weighted >= 0 && upto > share, ints);
    __shared__ int drawn;
    if (threadIdx.x == 0) drawn = -1;
    __syncthreads();
    if (who == 256) {
      // the piece's sum was rounded another way and nothing in it passes: the
      // last of its tokens that has a weight
      if (weighted >= 0) atomicMax(&drawn, weighted);
    } else if ((int)threadIdx.x == who) {
      // (rounded another way: the last with a weight)
      double c = upto - mine;
      int found = weighted;
      for (int v = t0, done = 0; v < t1 && !done; v += 4) {
        if (t1 - t0 > 4) load4(v);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (done || v + k >= t1) continue;
          const double w = weight(v, k);
          c += w;
          if (w > 0.0 && c > share) {
            found = v + k;
            done = 1;
          }
        }
      }
      drawn = found;
    }
    __syncthreads();
    if (drawn >= 0) token = drawn;
  }
  if (wave == 0) {
    for (int k = lane; k < rows; k += 64) a.out[s0 + k] = k < n ? draft : k == n ? token : -1;
    if (lane == 0) a.count[b] = n + 1;
  }
}

}  // namespace

int64_t plan_verify(VerifyArgs *a, void *work) {
  // The counters have a place of their own whatever B and V are, so that calls
  // of several sizes can share a workspace: sequences of more than one
  // workgroup are at most half of kMaxWorkgroups.
  constexpr int64_t counters = kMaxWorkgroups / 2 * kCounterInts * 4;
  // Pieces are whole steps of a wave (16 bytes a lane, of the smallest type).
  const int step = 512;
  a->per = ((a->V + kMaxPieces - 1) / kMaxPieces + step - 1) / step * step;
  a->pieces = (a->V + a->per - 1) / a->per;
  int most = kMaxWorkgroups / a->B;
  if (most < 1) most = 1;
  a->each = (a->pieces + 4 * most - 1) / (4 * most);
  a->slices = (a->pieces + 4 * a->each - 1) / (4 * a->each);
  a->arrived = static_cast<int32_t *>(work);
  a->sums = reinterpret_cast<double *>(static_cast<uint8_t *>(work) + counters);
  return counters + (int64_t)a->B * a->pieces * 16;
}

int launch_verify(const VerifyArgs &a, hipStream_t stream) {
  const dim3 grid((unsigned)a.B * (unsigned)a.slices), block(256);
  switch (a.dtype) {
    case QGEMV_F32: hipLaunchKernelGGL(verify_kernel<QGEMV_F32>, grid, block, 0, stream, a); break;
    case QGEMV_BF16: hipLaunchKernelGGL(verify_kernel<QGEMV_BF16>, grid, block, 0, stream, a); break;
    case QGEMV_F16: hipLaunchKernelGGL(verify_kernel<QGEMV_F16>, grid, block, 0, stream, a); break;
    default: return QGEMV_EINVAL;
  }
  return hipGetLastError() == hipSuccess ? QGEMV_OK : QGEMV_EHIP;
}

}  // namespace qgemv
