// Routing of rows to experts.
//
//   score_e = exp(x_e) / sum exp(x)  or  1 / (1 + exp(-x_e)),
//   choice_e = score_e + bias_e,
//
// the experts of the `keep` groups whose `best` largest choices have the
// greatest sum, of these the k of greatest choice, weights their scores, over
// their sum where asked.  Equal choices go to the lower expert.
//
// A wave takes a row; a lane has V consecutive experts, so that the lowest lane
// that holds the maximum has the lowest expert of it.  Choices are fp64: which
// expert is the k-th is decided between neighbours some 10^-3 apart on average,
// and in fp32 one in some thousand rows would be decided by rounding.  Without
// a bias (and without sums over a group) the scores' order is the logits', and
// nothing rounds at all.
//
// Bound by latency and, for thousands of rows, by what a step of the choice
// costs: a lane sorts its choices once, as 64-bit keys in order, and a step
// compares the lanes' first ones, by their upper halves in six instructions and by
// their lower halves only where two lanes share the upper.
//
// On an MI355X, 8 experts of each row: 5 rows of 128 5.0 us, as long as the call
// takes; 4096 rows of 256 6.0 us by their logits, 7.6 by a sigmoid with a bias, 9.6
// with that in 4 of 8 groups (2 MB, 0.3 us of memory): 800 vector instructions a
// wave, four waves a SIMD.  A row's 64 lanes have 4 experts each there; half as many
// lanes with 8 each would halve the steps, not the exponentials and the sorting.

#include "qgemv_device.h"
#include "qgemv_kv.h"

namespace qgemv {

namespace {

constexpr double kNone = -__builtin_inf();

__device__ __forceinline__ double read_lane(double x, int lane) {
  const uint64_t v = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)v, lane);
  const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)(v >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Sum / maximum over the wave, by DPP: shifts within 16 lanes, then broadcasts;
// the last lane has it.  Lanes that nothing is shifted into keep their own.
template <int CTRL, int ROWS>
__device__ __forceinline__ double shifted(double x, double otherwise) {
  const uint64_t v = __builtin_bit_cast(uint64_t, x), o = __builtin_bit_cast(uint64_t, otherwise);
  const uint32_t lo = __builtin_amdgcn_update_dpp((uint32_t)o, (uint32_t)v, CTRL, ROWS, 0xF, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp((uint32_t)(o >> 32), (uint32_t)(v >> 32), CTRL, ROWS, 0xF, false);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
template <class F>
__device__ __forceinline__ double wave_join(double x, double neutral, F f) {
  x = f(x, shifted<0x111, 0xF>(x, neutral));
  x = f(x, shifted<0x112, 0xF>(x, neutral));
  x = f(x, shifted<0x114, 0xF>(x, neutral));
  x = f(x, shifted<0x118, 0xF>(x, neutral));
  x = f(x, shifted<0x142, 0xA>(x, neutral));
  x = f(x, shifted<0x143, 0xC>(x, neutral));
  return read_lane(x, 63);
}
__device__ __forceinline__ double wave_sum(double x) {
  return wave_join(x, 0.0, [](double a, double b) { return a + b; });
}
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
  x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x111, 0xF, 0xF, false));
  x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x112, 0xF, 0xF, false));
  x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x114, 0xF, 0xF, false));
  x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x118, 0xF, 0xF, false));
  x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x142, 0xA, 0xF, false));
  x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x143, 0xC, 0xF, false));
  return __builtin_amdgcn_readlane(x, 63);
}
__device__ __forceinline__ float wave_max(float x) {  // in the order of unsigned numbers
  const uint32_t v = __builtin_bit_cast(uint32_t, x);
  const uint32_t m = wave_max(v >> 31 ? ~v : v | 0x80000000u);
  return __builtin_bit_cast(float, m >> 31 ? m & 0x7FFFFFFFu : ~m);
}

// A choice as a number in the same order; 0 for one that is not there.
__device__ __forceinline__ uint64_t key_of(double x) {
  const uint64_t v = __builtin_bit_cast(uint64_t, x + 0.0);  // (-0 is 0)
  return !(x > kNone) ? 0 : v >> 63 ? ~v : v | 1ull << 63;
}
// Its last 4 bits make room for the expert's place within its lane, the first
// largest: choices count as equal within 2^-48 of their value.
constexpr uint64_t kPlace = 15;
__device__ __forceinline__ uint64_t placed(uint64_t key, int j) { return key ? (key & ~kPlace) | (kPlace - j) : 0; }

// The largest first: Batcher's odd-even merge sort of V keys (V a power of two).
template <int V>
__device__ __forceinline__ void sort_keys(uint64_t (&key)[V]) {
#pragma unroll
  for (int p = 1; p < V; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < V; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < V && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
            const uint64_t a = key[i + j], b = key[i + j + k];
            key[i + j] = a > b ? a : b;
            key[i + j + k] = a > b ? b : a;
          }
}

// The value of the lane `distance` away, where lanes that lie closer together hold
// the same already: 1, 2, 4 and 8 by DPP.
__device__ __forceinline__ double across(double x, int distance) {
  switch (distance) {
    case 1: return shifted<0xB1, 0xF>(x, x);   // quad_perm 1 0 3 2
    case 2: return shifted<0x4E, 0xF>(x, x);   // quad_perm 2 3 0 1
    case 4: return shifted<0x141, 0xF>(x, x);  // row_half_mirror
    case 8: return shifted<0x140, 0xF>(x, x);  // row_mirror
  }
  return __shfl_xor(x, distance);
}

template <int DT>
__device__ __forceinline__ float logit(const uint8_t *p, int64_t i) {
  if constexpr (DT == QGEMV_F32) return reinterpret_cast<const float *>(p)[i];
  const uint32_t h = reinterpret_cast<const uint16_t *>(p)[i];
  return DT == QGEMV_BF16 ? bf16_bits_to_float(h) : half_bits_to_float(h);
}

// V experts of a lane, a row of a wave.
template <int DT, int V>
__global__ __launch_bounds__(256) void route_kernel(RouteArgs a) {
  extern __shared__ __align__(16) double choices[];  // with groups: [waves][64 V]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int t = blockIdx.x * (blockDim.x >> 6) + wave;
  if (t >= a.T) return;  // (no barrier below)
  const int E = a.E, e0 = lane * V;
  const uint8_t *const row = a.logits + (int64_t)t * a.row * (DT == QGEMV_F32 ? 4 : 2);

  float x[V];
  float top = -__builtin_inff();
#pragma unroll
  for (int j = 0; j < V; ++j) {
    x[j] = e0 + j < E ? logit<DT>(row, e0 + j) : -__builtin_inff();
    top = fmaxf(top, x[j]);  // (a NaN is passed over)
  }
  // Scores, a softmax's times their sum, where the choice or the weights need all
  // of them.
  const bool by_logit = !a.bias && a.best == 1;
  const double m = a.softmax ? (double)wave_max(top) : 0.0;
  double choice[V], total = 1.0;
  if (!by_logit || (a.softmax && !a.renormalise)) {
    // (one block of exponentials, so that they share their constants' registers)
    const double sign = a.softmax ? 1.0 : -1.0;
#pragma unroll
    for (int j = 0; j < V; ++j) choice[j] = exp(sign * (double)x[j] - m);
    if (a.softmax) {
      double sum = 0.0;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        choice[j] = x[j] > -__builtin_inff() ? choice[j] : 0.0;
        sum += choice[j];
      }
      total = wave_sum(sum);
      const double over = 1.0 / total;
#pragma unroll
      for (int j = 0; j < V; ++j) choice[j] *= over;
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) choice[j] = 1.0 / (1.0 + choice[j]);
    }
  }
  // the choices' keys, of the experts that are there: neither -inf nor NaN
  uint64_t key[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const double c = by_logit ? (double)x[j] : choice[j] + (a.bias && e0 + j < E ? (double)a.bias[e0 + j] : 0.0);
    choice[j] = x[j] > -__builtin_inff() && c > kNone ? c : kNone;
    key[j] = key_of(choice[j]);
  }

  if (a.groups > 1) {
    const int size = E / a.groups, lanes = size / V;
    // lane `at` of a group g has its value
    double first = kNone, second = kNone;
    auto take = [&](double c) {
      second = fmax(second, fmin(first, c));
      first = fmax(first, c);
    };
    int at = 1;
    if (lanes * V == size && (lanes & (lanes - 1)) == 0) {  // whole lanes, a power of two of them
      at = lanes;
#pragma unroll
      for (int j = 0; j < V; ++j) take(choice[j]);
      for (int over = 1; over < lanes; over <<= 1) {
        const double f = across(first, over), s = across(second, over);
        take(f);
        take(s);
      }
    } else {  // lane g reads group g
      double *const all = choices + wave * (64 * V);
#pragma unroll
      for (int j = 0; j < V; ++j) all[e0 + j] = choice[j];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      if (lane < a.groups)
        for (int i = 0; i < size; ++i) take(all[lane * size + i]);
    }
    const double value = a.best == 2 && second > kNone ? first + second : first;
    const uint64_t mine = key_of(value);
    // lane g: how many groups come before it
    const uint64_t its = __shfl(mine, min(lane * at, 63)), of_lane = lane < a.groups ? its : 0;
    int before = 0;
#pragma unroll 4
    for (int g = 0; g < (a.groups + 3) / 4 * 4; ++g) {  // (lanes past the groups have 0, which is before none)
      const uint64_t other = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((uint32_t)(of_lane >> 32), g) << 32 |
                             (uint32_t)__builtin_amdgcn_readlane((uint32_t)of_lane, g);
      before += other > of_lane || (other == of_lane && g < lane);
    }
    const uint64_t kept = __ballot(lane < a.groups && before < a.keep && of_lane);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int g = min((int)((uint32_t)(e0 + j) * a.over_size >> 20), 63);
      if (!(kept >> g & 1)) key[j] = 0;
    }
  }

  // ---- the k of greatest choice, one after another; lane i keeps the i-th
#pragma unroll
  for (int j = 0; j < V; ++j) key[j] = placed(key[j], j);
  sort_keys(key);
  int expert = -1;
  for (int i = 0; i < a.k; ++i) {
    const uint32_t hi = (uint32_t)(key[0] >> 32), lo = (uint32_t)key[0];
    const uint32_t most = wave_max(hi);
    if (most == 0) break;  // none is left
    uint64_t with = __ballot(hi == most);
    if (with & (with - 1)) {
      const uint32_t below = wave_max(hi == most ? lo >> 4 : 0u);
      with = __ballot(hi == most && lo >> 4 == below);
    }
    const int from = (int)__ffsll((long long)with) - 1;
    const int place = (int)kPlace - (int)(__builtin_amdgcn_readlane(lo, from) & (uint32_t)kPlace);
    expert = lane == i ? from * V + place : expert;
    // that lane's next one comes first (a choice by bits: one instruction a word)
    const uint64_t stay = lane != from ? ~0ull : 0ull;
#pragma unroll
    for (int j = 0; j < V; ++j) key[j] = (key[j] & stay) | ((j + 1 < V ? key[j + 1] : 0) & ~stay);
  }
  double weight = 0.0;
  if (lane < a.k && expert >= 0) {
    const double v = (double)logit<DT>(row, expert);
    weight = a.softmax ? exp(v - m) : 1.0 / (1.0 + exp(-v));
  }
  if (a.renormalise) total = wave_sum(weight);
  if (lane < a.k) {
    a.experts[(int64_t)t * a.k + lane] = expert;
    a.weights[(int64_t)t * a.k + lane] =
        expert < 0 || total == 0.0 ? 0.0f : (float)(weight / total * (double)a.scale);
  }
}

template <int DT, int V>
int launch_route_v(const RouteArgs &a, hipStream_t stream) {
  const int waves = a.T <= 256 ? 1 : 4;  // a CU for each row while there are as many
  const size_t bytes = a.groups > 1 ? (size_t)waves * 64 * V * 8 : 0;
  hipLaunchKernelGGL((route_kernel<DT, V>), dim3((a.T + waves - 1) / waves), dim3(64 * waves), bytes, stream, a);
  return hipGetLastError() == hipSuccess ? QGEMV_OK : QGEMV_EHIP;
}

template <int DT>
int launch_route_t(const RouteArgs &a, hipStream_t stream) {
  if (a.E <= 64) return launch_route_v<DT, 1>(a, stream);
  if (a.E <= 128) return launch_route_v<DT, 2>(a, stream);
  if (a.E <= 256) return launch_route_v<DT, 4>(a, stream);
  if (a.E <= 512) return launch_route_v<DT, 8>(a, stream);
  return launch_route_v<DT, 16>(a, stream);  // up to QGEMV_MAX_ROUTED
}

}  // namespace

int launch_route(const RouteArgs &a, hipStream_t stream) {
  switch (a.dtype) {
    case QGEMV_F32: return launch_route_t<QGEMV_F32>(a, stream);
    case QGEMV_BF16: return launch_route_t<QGEMV_BF16>(a, stream);
    case QGEMV_F16: return launch_route_t<QGEMV_F16>(a, stream);
  }
  return QGEMV_EINVAL;
}

}  // namespace qgemv
