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

#include "qgemv_kv.h"
#include "qgemv_device.h"

namespace qgemv {

namespace {

template <int DT>
__device__ __forceinline__ float prob(const uint8_t *row, int i) {
  if constexpr (DT == QGEMV_F32) {
    return reinterpret_cast<const float *>(row)[i];
  } else {
    const uint32_t b = reinterpret_cast<const uint16_t *>(row)[i];
    return DT == QGEMV_BF16 ? bf16_bits_to_float(b) : half_bits_to_float(b);
  }
}

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
  for (int s = 32; s; s >>= 1) x += __shfl_xor(x, s);
  return x;
}

// max(p - q, 0) that a NaN passes
__device__ __forceinline__ double rest_of(float p, float q) {
  const double d = (double)p - (double)q;
  return d < 0.0 ? 0.0 : d;
}

template <int DT>
__global__ __launch_bounds__(256) void verify_kernel(VerifyArgs a) {
  const int b = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int s0 = min(max(a.start[b], 0), a.T);
  const int rows = min(min(max(a.start[b + 1], s0), a.T) - s0, a.M);
  if (rows <= 0) {
    if (threadIdx.x == 0) a.count[b] = 0;
    return;
  }
  constexpr int SB = DT == QGEMV_F32 ? 4 : 2;
  // every wave checks all drafts, one a lane
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
  __shared__ double part[4][2];
  // each wave sums a quarter: what is left of p, and p itself
  const int per = (a.V + 3) / 4, v0 = wave * per, v1 = min(v0 + per, a.V);
  double left = 0.0, all = 0.0;
  for (int i = v0 + lane; i < v1; i += 64) {
    const float x = prob<DT>(p, i);
    all += x;
    left += q ? rest_of(x, prob<DT>(q, i)) : i == drop ? 0.0 : (double)x;
  }
  left = wave_sum(left);
  all = wave_sum(all);
  if (lane == 0) {
    part[wave][0] = left;
    part[wave][1] = all;
  }
  __syncthreads();
  if (wave != 0) return;
  const double total_left = part[0][0] + part[1][0] + part[2][0] + part[3][0];
  const bool use_all = !(total_left > 0.0);
  const int which = use_all ? 1 : 0;
  const double total = use_all ? part[0][1] + part[1][1] + part[2][1] + part[3][1] : total_left;
  const double share = (double)a.u[s0 + rows - 1] * total;
  int token = a.V - 1;
  if (!(share == share)) {
    token = 0;
  } else if (share < total) {
    double before = 0.0;
    int w = 0;
    while (w < 3 && !(before + part[w][which] > share)) before += part[w++][which];
    int last = -1;  // the last token of the quarter that has a weight
    bool found = false;
    for (int i0 = w * per; i0 < min((w + 1) * per, a.V) && !found; i0 += 64) {
      const int i = i0 + lane;
      double x = 0.0;
      if (i < min((w + 1) * per, a.V)) {
        const float pi = prob<DT>(p, i);
        x = use_all ? (double)pi : q ? rest_of(pi, prob<DT>(q, i)) : i == drop ? 0.0 : (double)pi;
      }
      const bool has = x > 0.0;
#pragma unroll
      for (int s = 1; s < 64; s <<= 1) {
        const double y = __shfl_up(x, s);
        if (lane >= s) x += y;
      }
      const uint64_t over = __ballot(before + x > share);
      const uint64_t weighted = __ballot(has);
      if (over) {
        token = i0 + (int)__ffsll((long long)over) - 1;
        found = true;
      } else if (weighted) {
        last = i0 + 63 - __clzll((long long)weighted);
      }
      before += __shfl(x, 63);
    }
    if (!found && last >= 0) token = last;
  }
  for (int i = lane; i < rows; i += 64) a.out[s0 + i] = i < n ? draft : i == n ? token : -1;
  if (lane == 0) a.count[b] = n + 1;
}

}  // namespace

int launch_verify(const VerifyArgs &a, hipStream_t stream) {
  const dim3 grid(a.B), block(256);
  switch (a.dtype) {
    case QGEMV_F32: hipLaunchKernelGGL(verify_kernel<QGEMV_F32>, grid, block, 0, stream, a); break;
    case QGEMV_BF16: hipLaunchKernelGGL(verify_kernel<QGEMV_BF16>, grid, block, 0, stream, a); break;
    case QGEMV_F16: hipLaunchKernelGGL(verify_kernel<QGEMV_F16>, grid, block, 0, stream, a); break;
    default: return QGEMV_EINVAL;
  }
  return hipGetLastError() == hipSuccess ? QGEMV_OK : QGEMV_EHIP;
}

}  // namespace qgemv
