// Attention of the new rows of each sequence over its paged cache.
//
//   s_j = scale * k_scale[h] * (q . k_j) over the tokens j that the row sees:
//         j <= pos, and with a window W also j > pos - W or j < sinks
//   lse = log sum_j exp(s_j),  out = v_scale[h] * sum_j exp(s_j - lse) v_j
//
// A row that sees nothing gives 0 and -inf.  One workgroup takes one row and
// query head; its waves take every fourth token, the lanes split D, and the
// running maximum, sum and output of each wave are joined at the end.

#include "qgemv_kv.h"
#include "qgemv_device.h"

namespace qgemv {

namespace {

// Values DT at p, as floats.
template <int DT, int N>
__device__ __forceinline__ void load_values(const uint8_t *p, float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (DT == QGEMV_E4M3) {
      x[i] = __builtin_amdgcn_cvt_f32_fp8((int)p[i], 0);
    } else {
      const uint32_t b = reinterpret_cast<const uint16_t *>(p)[i];
      x[i] = DT == QGEMV_BF16 ? bf16_bits_to_float(b) : half_bits_to_float(b);
    }
  }
}

template <int QT, int CT, int D>
__global__ __launch_bounds__(256) void attend_kernel(AttendArgs a) {
  constexpr int N = D / 64;
  constexpr int CB = CT == QGEMV_E4M3 ? 1 : 2;
  const int t = blockIdx.x, hq = blockIdx.y, h = hq / a.G;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int seq = 0;
  for (int base = 0; base < a.B; base += 256) {
    const int b = base + (int)threadIdx.x;
    seq += __syncthreads_count(b < a.B && a.start[b + 1] <= t);
  }
  if (seq >= a.B || t < a.start[0] || t - a.start[seq] >= a.M) return;
  const int cap = a.c.width * a.c.page;
  const int len = min(max(a.len[seq], 0), cap);
  const int pos = len - (a.start[seq + 1] - t);
  float q[N], k[N], o[N] = {};
  load_values<QT>(a.q + t * a.q_row + hq * a.q_head + lane * N * 2, q);
  const float sc = a.scale * (a.c.k_scale ? a.c.k_scale[h] : 1.0f) * 1.44269504088896340736f;
  float m = -__builtin_inff(), l = 0.0f;
  for (int j = wave; j <= pos; j += 4) {
    if (a.window && !(j > pos - a.window || j < a.sinks)) continue;
    const int idx = page_of(a.c, j);
    const int id = a.c.table[(int64_t)seq * a.c.width + idx];
    if (id < 0 || id >= a.c.pages) continue;  // a page that is not there holds nothing to see
    const int64_t at = id * a.c.stride_page + (j - idx * a.c.page) * a.c.stride_slot + h * a.c.stride_head + lane * N * CB;
    load_values<CT>(a.c.k + at, k);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) s += q[i] * k[i];
#pragma unroll
    for (int x = 32; x; x >>= 1) s += __shfl_xor(s, x);
    s *= sc;
    const float mn = fmaxf(m, s), ms = mn == -__builtin_inff() ? 0.0f : mn;
    const float f = __builtin_amdgcn_exp2f(m - ms), e = __builtin_amdgcn_exp2f(s - ms);
    m = mn;
    l = l * f + e;
    load_values<CT>(a.c.v + at, k);
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = o[i] * f + e * k[i];
  }
  __shared__ float ml[4][2], sums[4][D];
  ml[wave][0] = m;
  ml[wave][1] = l;
#pragma unroll
  for (int i = 0; i < N; ++i) sums[wave][lane * N + i] = o[i];
  __syncthreads();
  float top = fmaxf(fmaxf(ml[0][0], ml[1][0]), fmaxf(ml[2][0], ml[3][0]));
  if (top == -__builtin_inff()) top = 0.0f;
  float f[4], total = 0.0f;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    f[w] = __builtin_amdgcn_exp2f(ml[w][0] - top);
    total += f[w] * ml[w][1];
  }
  const float vs = a.c.v_scale ? a.c.v_scale[h] : 1.0f;
  for (int d = threadIdx.x; d < D; d += 256) {
    const float x = f[0] * sums[0][d] + f[1] * sums[1][d] + f[2] * sums[2][d] + f[3] * sums[3][d];
    const float y = total == 0.0f ? 0.0f : x / total * vs;
    uint16_t *dst = reinterpret_cast<uint16_t *>(a.out + t * a.out_row + hq * a.out_head) + d;
    *dst = QT == QGEMV_BF16 ? __builtin_bit_cast(uint16_t, (__bf16)y) : __builtin_bit_cast(uint16_t, (_Float16)y);
  }
  if (a.lse && threadIdx.x == 0)
    a.lse[(int64_t)t * (a.c.H * a.G) + hq] = (top + __builtin_log2f(total)) * 0.69314718055994530942f;
}

template <int QT, int CT>
int launch_attend_t(const AttendArgs &a, hipStream_t stream) {
  const dim3 grid(a.T, a.c.H * a.G), block(256);
  switch (a.c.D) {
    case 64: hipLaunchKernelGGL((attend_kernel<QT, CT, 64>), grid, block, 0, stream, a); break;
    case 128: hipLaunchKernelGGL((attend_kernel<QT, CT, 128>), grid, block, 0, stream, a); break;
    case 256: hipLaunchKernelGGL((attend_kernel<QT, CT, 256>), grid, block, 0, stream, a); break;
    default: return QGEMV_EUNSUPPORTED;
  }
  return hipGetLastError() == hipSuccess ? QGEMV_OK : QGEMV_EHIP;
}

}  // namespace

int launch_attend(const AttendArgs &a, hipStream_t stream) {
  if (a.q_dtype == QGEMV_BF16)
    return a.c.dtype == QGEMV_E4M3 ? launch_attend_t<QGEMV_BF16, QGEMV_E4M3>(a, stream)
                                   : launch_attend_t<QGEMV_BF16, QGEMV_BF16>(a, stream);
  return a.c.dtype == QGEMV_E4M3 ? launch_attend_t<QGEMV_F16, QGEMV_E4M3>(a, stream)
                                 : launch_attend_t<QGEMV_F16, QGEMV_F16>(a, stream);
}

}  // namespace qgemv
