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
// One launch.  A sequence's row is cut into pieces, one a wave, 4 waves a
// workgroup: each wave checks the drafts itself (they decide which row is
// summed; at most 15 pairs of loads, one a lane), sums its piece and leaves
// the sum in the workspace.  The workgroup that arrives last at the sequence's
// counter scans the sums in order, finds the piece where the running sum
// passes the number, scans that piece again and writes the answer; it also
// sets the counter back to 0.  Which workgroup is last changes nothing in the
// result.

#include "qgemv_kv.h"
#include "qgemv_device.h"

namespace qgemv {

namespace {

constexpr int kMaxPieces = 256;  // of a row: the last workgroup has one thread for each

template <int DT>
__device__ __forceinline__ float prob(const uint8_t *row, int i) {
  if constexpr (DT == QGEMV_F32) {
    return reinterpret_cast<const float *>(row)[i];
  } else {
    const uint32_t b = reinterpret_cast<const uint16_t *>(row)[i];
    return DT == QGEMV_BF16 ? bf16_bits_to_float(b) : half_bits_to_float(b);
  }
}

// 16 bytes of a row as floats.  Rows start at any element (an odd vocabulary),
// so the load is only element-aligned; the hardware takes that.
template <int DT>
struct Piece16 {
  static constexpr int N = DT == QGEMV_F32 ? 4 : 8;
  static __device__ __forceinline__ void load(const uint8_t *row, int i, float (&x)[N]) {
    u32x4_t w;
    __builtin_memcpy(&w, row + (int64_t)i * (16 / N), 16);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      if constexpr (DT == QGEMV_F32) {
        const uint32_t b = w[k];  // (a bit cast of the element itself takes the vector's first)
        x[k] = __builtin_bit_cast(float, b);
      } else {
        const uint32_t b = k & 1 ? w[k >> 1] >> 16 : w[k >> 1] & 0xFFFFu;
        x[k] = DT == QGEMV_BF16 ? bf16_bits_to_float(b) : half_bits_to_float(b);
      }
    }
  }
};

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
  for (int s = 32; s; s >>= 1) x += __shfl_xor(x, s);
  return x;
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

// max(p - q, 0) that a NaN passes
__device__ __forceinline__ double rest_of(float p, float q) {
  const double d = (double)p - (double)q;
  return d < 0.0 ? 0.0 : d;
}

template <int DT>
__global__ __launch_bounds__(256) void verify_kernel(VerifyArgs a) {
  constexpr int SB = DT == QGEMV_F32 ? 4 : 2, N = Piece16<DT>::N;
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

  // ---- this wave's piece: what is left of p, and p itself
  const int pieces = 4 * a.slices, per = (a.V + pieces - 1) / pieces;
  const int piece = slice * 4 + wave;
  const int v0 = min(piece * per, a.V), v1 = min(v0 + per, a.V);
  double left = 0.0, all = 0.0;
  int i = v0 + lane * N;
#pragma unroll 4
  for (; i + N <= v1; i += 64 * N) {
    float x[N], y[N];
    Piece16<DT>::load(p, i, x);
    if (q) Piece16<DT>::load(q, i, y);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      all += x[k];
      left += q ? rest_of(x[k], y[k]) : i + k == drop ? 0.0 : (double)x[k];
    }
  }
  for (; i < v1; ++i) {  // at most one lane holds the piece's ragged end
    const float x = prob<DT>(p, i);
    all += x;
    left += q ? rest_of(x, prob<DT>(q, i)) : i == drop ? 0.0 : (double)x;
  }
  left = wave_sum(left);
  all = wave_sum(all);

  // ---- leave the sums; the last workgroup of the sequence goes on.  The sums
  // are stored past the caches of this XCD, and the counter's release and
  // acquire order them for the workgroup that reads them.
  double *const sums = a.sums + (int64_t)b * pieces * 2;
  if (lane == 0) {
    __hip_atomic_store(sums + piece * 2, left, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __hip_atomic_store(sums + piece * 2 + 1, all, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __shared__ double part[4];
  __shared__ int ints[4];
  if (a.slices > 1) {
    __syncthreads();
    if (threadIdx.x == 0) {
      const int before = __hip_atomic_fetch_add(a.arrived + b, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
      ints[0] = before == a.slices - 1;
      if (before == a.slices - 1)
        __hip_atomic_store(a.arrived + b, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
  }
  __syncthreads();
  if (a.slices > 1) {
    const bool last = ints[0] != 0;
    __syncthreads();
    if (!last) return;
  }

  const bool has = (int)threadIdx.x < pieces;
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
    const int at = min(block_first(has && run > share, ints), pieces - 1);
    __shared__ double before_at;
    if ((int)threadIdx.x == at) before_at = run - (use_all ? my_all : my_left);
    // the piece again, consecutive tokens a thread
    const int a0 = min(at * per, a.V), a1 = min(a0 + per, a.V), each = (per + 255) / 256;
    const int t0 = min(a0 + (int)threadIdx.x * each, a1), t1 = min(t0 + each, a1);
    auto weight = [&](int v) -> double {
      const float x = prob<DT>(p, v);
      return use_all ? (double)x : q ? rest_of(x, prob<DT>(q, v)) : v == drop ? 0.0 : (double)x;
    };
    double mine = 0.0;
    int weighted = -1;  // the last token here that has a weight
    for (int v = t0; v < t1; ++v) {
      const double w = weight(v);
      mine += w;
      if (w > 0.0) weighted = v;
    }
    double ignored;
    double upto = block_scan(mine, part, &ignored);
    upto += before_at;  // after the scan's barriers
    const int who = block_first(upto > share, ints);
    __shared__ int drawn;
    if (threadIdx.x == 0) drawn = -1;
    __syncthreads();
    if (who == 256) {
      // the piece's sum was rounded another way and nothing in it passes: the
      // last of its tokens that has a weight
      if (weighted >= 0) atomicMax(&drawn, weighted);
    } else if ((int)threadIdx.x == who) {
      double c = upto - mine;
      int v = t0;
      for (; v < t1 - 1; ++v) {
        c += weight(v);
        if (c > share) break;
      }
      // (rounded another way: the last with a weight)
      drawn = v == t1 - 1 && weighted >= 0 ? weighted : v;
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
  // Pieces of at least 512 tokens (two 16-byte loads of fp32 a lane), about
  // 1024 workgroups in all.
  int slices = (int)(((int64_t)a->V + 2047) / 2048);
  const int most = 1024 / a->B;
  if (slices > most) slices = most;
  if (slices > kMaxPieces / 4) slices = kMaxPieces / 4;
  if (slices < 1) slices = 1;
  a->slices = slices;
  const int64_t sums = (int64_t)a->B * slices * 4 * 2 * 8;
  a->sums = static_cast<double *>(work);
  a->arrived = reinterpret_cast<int32_t *>(static_cast<uint8_t *>(work) + sums);
  return sums + 4 * (int64_t)a->B;
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
