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
__device__ __forceinline__ double wave_max(double x) {
  return wave_join(x, kNone, [](double a, double b) { return a > b ? a : b; });
}
__device__ __forceinline__ double wave_sum(double x) {
  return wave_join(x, 0.0, [](double a, double b) { return a + b; });
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
  // which experts are there: neither -inf nor NaN
  double score[V], choice[V];
  if (a.softmax) {
    const double m = wave_max((double)top);
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      score[j] = x[j] > -__builtin_inff() ? exp((double)x[j] - m) : 0.0;
      sum += score[j];
    }
    sum = wave_sum(sum);
#pragma unroll
    for (int j = 0; j < V; ++j) score[j] = score[j] / sum;
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) score[j] = 1.0 / (1.0 + exp(-(double)x[j]));
  }
  const bool by_logit = !a.bias && a.best == 1;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const bool there = x[j] > -__builtin_inff();
    const double c = by_logit ? (double)x[j] : score[j] + (a.bias && e0 + j < E ? (double)a.bias[e0 + j] : 0.0);
    choice[j] = there && c > kNone ? c : kNone;
  }

  if (a.groups > 1) {
    double *const all = choices + wave * (64 * V);
#pragma unroll
    for (int j = 0; j < V; ++j) all[e0 + j] = choice[j];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const int size = E / a.groups;
    // lane g has group g
    double first = kNone, second = kNone;
    if (lane < a.groups) {
      for (int i = 0; i < size; ++i) {
        const double c = all[lane * size + i];
        second = c > first ? first : c > second ? c : second;
        first = c > first ? c : first;
      }
    }
    const double value = a.best == 2 && second > kNone ? first + second : first;
    int before = 0;  // groups that come first
    for (int g = 0; g < a.groups; ++g) {
      const double other = read_lane(value, g);
      before += other > value || (other == value && g < lane);
    }
    const uint64_t kept = __ballot(lane < a.groups && before < a.keep && value > kNone);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int g = min((int)((uint32_t)(e0 + j) / (uint32_t)size), 63);
      if (!(kept >> g & 1)) choice[j] = kNone;
    }
  }

  // ---- the k of greatest choice, one after another; lane i keeps the i-th
  int expert = -1;
  double weight = 0.0;
  for (int i = 0; i < a.k; ++i) {
    double best = choice[0], its = score[0];
    int at = 0;
#pragma unroll
    for (int j = 1; j < V; ++j) {
      const bool more = choice[j] > best;
      best = more ? choice[j] : best;
      its = more ? score[j] : its;
      at = more ? j : at;
    }
    const double most = wave_max(best);
    if (!(most > kNone)) break;  // none is left
    const int from = (int)__ffsll((long long)__ballot(best == most)) - 1;
    const int e = __builtin_amdgcn_readlane(e0 + at, from);
    const double w = read_lane(its, from);
    if (lane == i) {
      expert = e;
      weight = w;
    }
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (e0 + j == e) choice[j] = kNone;
  }
  if (a.renormalise) {
    const double sum = wave_sum(weight);
    weight = sum > 0.0 ? weight / sum : sum == 0.0 ? 0.0 : weight / sum;
  }
  if (lane < a.k) {
    a.experts[(int64_t)t * a.k + lane] = expert;
    a.weights[(int64_t)t * a.k + lane] = (float)(weight * (double)a.scale);
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
