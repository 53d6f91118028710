// Appending the new rows' keys and values to a paged cache.
//
//   K[slot(b, pos)][h] = cast(new_k[t][h]),  pos = len[b] - (start[b+1] - t)
//
// and V alike; an 8-bit cache stores clamp(new / scale[h], -448, 448) rounded
// once to E4M3.  One workgroup takes one row t for both K and V: 2 H D values,
// eight to a thread and step.  The first step's values are loaded before the
// slot is known, so that reading them and finding it overlap.  The row's
// sequence is found by counting the starts that are not after t, one start a
// thread, so that finding it costs one load's latency whatever B is (a binary
// search: log2 B dependent loads).
//
// On an MI355X: 5 rows of one request 2.8 us, as long as the shortest kernel
// takes; 3476 rows of 256 sequences from fp32 into E4M3, 35.6 MB, 10 us (a pure
// read of 34 MB: 9 us).

#include "qgemv_kv.h"
#include "qgemv_device.h"

namespace qgemv {

namespace {

typedef float f32x8_t __attribute__((ext_vector_type(8)));

template <int SRC>
__device__ __forceinline__ f32x8_t load8(const uint8_t *p) {
  f32x8_t r;
  if constexpr (SRC == QGEMV_F32) {
    const f32x4_t a = *reinterpret_cast<const f32x4_t *>(p);
    const f32x4_t b = *reinterpret_cast<const f32x4_t *>(p + 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r[i] = a[i];
      r[4 + i] = b[i];
    }
  } else {
    const u32x4_t a = *reinterpret_cast<const u32x4_t *>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (SRC == QGEMV_BF16) {
        r[2 * i] = __builtin_bit_cast(float, a[i] << 16);
        r[2 * i + 1] = __builtin_bit_cast(float, a[i] & 0xFFFF0000u);
      } else {
        r[2 * i] = half_bits_to_float(a[i] & 0xFFFFu);
        r[2 * i + 1] = half_bits_to_float(a[i] >> 16);
      }
    }
  }
  return r;
}

// Eight values in the cache's type: one rounding, to nearest even.  E4M3 has no
// infinity: values are limited to +-448 first (two compares, which a NaN passes
// unchanged).
template <int DST>
struct Packed {
  static constexpr int N = DST == QGEMV_E4M3 ? 2 : 4;
  uint32_t w[N];
};

template <int DST>
__device__ __forceinline__ Packed<DST> pack8(f32x8_t x, float scale) {
  Packed<DST> o;
  if constexpr (DST == QGEMV_E4M3) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v = x[i] / scale;
      v = v > 448.0f ? 448.0f : v;
      x[i] = v < -448.0f ? -448.0f : v;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      int d = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * i], x[4 * i + 1], 0, false);
      o.w[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x[4 * i + 2], x[4 * i + 3], d, true);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DST == QGEMV_BF16) {
        o.w[i] = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x[2 * i]) |
                 (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x[2 * i + 1]) << 16;
      } else {
        o.w[i] = (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)x[2 * i]) |
                 (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)x[2 * i + 1]) << 16;
      }
    }
  }
  return o;
}

template <int DST>
__device__ __forceinline__ void store8(uint8_t *p, const Packed<DST> &o) {
  if constexpr (DST == QGEMV_E4M3) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(o.w[0], o.w[1]);
  } else {
    u32x4_t v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = o.w[i];
    *reinterpret_cast<u32x4_t *>(p) = v;
  }
}

template <int SRC, int DST>
__global__ __launch_bounds__(256) void append_kernel(AppendArgs a) {
  constexpr int SB = SRC == QGEMV_F32 ? 4 : 2, DB = DST == QGEMV_E4M3 ? 1 : 2;
  const int t = blockIdx.x;
  const int shift = __builtin_ctz(a.c.D) - 3, n = a.c.H << shift;  // eights of a head, of a row's keys
  int i = threadIdx.x, h = 0, d = 0;
  bool is_v = false;
  float scale = 1.0f;
  auto load = [&]() {
    is_v = i >= n;
    const int e = is_v ? i - n : i;
    h = e >> shift;
    d = (e - (h << shift)) * 8;
    if (DST == QGEMV_E4M3) scale = (is_v ? a.c.v_scale : a.c.k_scale)[h];
    return load8<SRC>((is_v ? a.nv + t * a.v_row + h * a.v_head : a.nk + t * a.k_row + h * a.k_head) + d * SB);
  };
  f32x8_t x = {};
  if (i < 2 * n) x = load();

  int seq = 0;
  for (int base = 0; base < a.B; base += 256) {
    const int b = base + (int)threadIdx.x;
    seq += __syncthreads_count(b < a.B && a.start[b + 1] <= t);
  }
  if (seq >= a.B || t < a.start[seq]) return;  // no sequence's row
  // (starts are limited to T, as the attention limits them)
  const int64_t pos = (int64_t)min(a.len[seq], QGEMV_MAX_CONTEXT) - (min(a.start[seq + 1], a.T) - t);
  if (pos < 0 || pos >= (int64_t)a.c.width * a.c.page) return;
  const int idx = page_of(a.c, (int)pos);
  const int id = a.c.table[(int64_t)seq * a.c.width + idx];
  // the first values in the cache's type while the page id is on its way
  Packed<DST> o = {};
  if (i < 2 * n) o = pack8<DST>(x, scale);
#pragma unroll
  for (int k = 0; k < Packed<DST>::N; ++k) asm volatile("" : "+v"(o.w[k]));
  if (id < 0 || id >= a.c.pages) return;
  const int64_t slot = id * a.c.stride_page + ((int)pos - idx * a.c.page) * a.c.stride_slot;
  while (i < 2 * n) {
    store8<DST>((is_v ? a.c.v : a.c.k) + slot + h * a.c.stride_head + d * DB, o);
    i += 256;
    if (i < 2 * n) o = pack8<DST>(load(), scale);
  }
}

template <int SRC>
int launch_append_src(const AppendArgs &a, hipStream_t stream) {
  const dim3 grid(a.T), block(256);
  switch (a.c.dtype) {
    case QGEMV_BF16: hipLaunchKernelGGL((append_kernel<SRC, QGEMV_BF16>), grid, block, 0, stream, a); break;
    case QGEMV_F16: hipLaunchKernelGGL((append_kernel<SRC, QGEMV_F16>), grid, block, 0, stream, a); break;
    case QGEMV_E4M3: hipLaunchKernelGGL((append_kernel<SRC, QGEMV_E4M3>), grid, block, 0, stream, a); break;
    default: return QGEMV_EINVAL;
  }
  return hipGetLastError() == hipSuccess ? QGEMV_OK : QGEMV_EHIP;
}

// ---- with the rotation of positions on the way
//
//   angle(i) = position[axis(i)] * freq[i],  i < pairs
//   (a, b) -> (a cos - b sin, a sin + b cos) of the pair i of a head's values:
//   2 i and 2 i + 1 (interleaved), or i and pairs + i; the values after the
//   pairs stay.  Queries and keys are turned, values are not.
//
// One workgroup takes a row: its angles once, for all heads, then 16 values of
// a head to a thread and step, two pieces of eight that hold whole pairs.
//
// On an MI355X: 5 rows of one request, 48 query and 8 key-value heads of 128, 4.3
// us (the append alone 2.8); 3476 rows of
// 256 sequences from fp32 into bf16 queries and an E4M3 cache, positions of three
// axes, 164 MB, 30 us (5.3 TB/s, past what a large copy reaches).

// cos and sin of position * freq, in quarter turns: positions reach billions of
// them.  The product of 31 and 24 bits and that with 2 / pi, itself in two parts
// (its first 53 bits and the next), are each a fp64 number and what it rounds
// off, so that below 2^40 what is left over whole ones is off by its own fp64 step
// alone.  (With the numbers alone, angles near 2^40 were off by 2^-13.)  It is at
// most an eighth of a turn and 2^-12, where the series of sin and cos end at their
// 9th and 10th power (next terms below 2^-29 and 2^-30).
__device__ __forceinline__ float2 turn_of(int position, float freq) {
  constexpr double kQuarters = 0.63661977236758134308, kQuartersRest = -3.935735335036497e-17;  // 2 / pi
  double whole, left;
  {
#pragma clang fp contract(off)  // (what a product rounds off is added below)
    const double p = position, f = freq, angle = p * f, angle_rest = __builtin_fma(p, f, -angle);
    const double quarters = angle * kQuarters, quarters_rest = __builtin_fma(angle, kQuarters, -quarters);
    whole = __builtin_rint(quarters);
    left = (quarters - whole) + (quarters_rest + __builtin_fma(angle_rest, kQuarters, angle * kQuartersRest));
  }
  const float x = (float)(left * 1.57079632679489661923);
  const float y = x * x;
  const float s = x + x * y * (-1.0f / 6 + y * (1.0f / 120 + y * (-1.0f / 5040 + y * (1.0f / 362880))));
  const float c = 1.0f + y * (-0.5f + y * (1.0f / 24 + y * (-1.0f / 720 + y * (1.0f / 40320 + y * (-1.0f / 3628800)))));
  const int q = (int)(long long)whole & 3;
  const float u = q & 1 ? s : c, v = q & 1 ? c : s;
  return make_float2(q == 1 || q == 2 ? -u : u, q >= 2 ? -v : v);
}

template <int DST>
__device__ __forceinline__ void put8(uint8_t *p, f32x8_t x, float scale) {
  store8<DST>(p, pack8<DST>(x, scale));
}

template <int SRC, int DST, int OUT>
__global__ __launch_bounds__(256) void rotate_kernel(RotateArgs a) {
  constexpr int SB = SRC == QGEMV_F32 ? 4 : 2, DB = DST == QGEMV_E4M3 ? 1 : 2;
  __shared__ float2 turns[128];
  const int t = blockIdx.x, tid = threadIdx.x, T = a.rows.T, B = a.rows.B, pairs = a.pairs;
  const KvView &c = a.rows.c;
  const int shift = __builtin_ctz(c.D) - 4, per_head = 1 << shift;  // 16 values each
  const int n = (a.q_heads + 2 * c.H) << shift;
  // this thread's frequency and its given position, while the sequence is searched
  float freq = 0.0f;
  int position = 0;
  if (tid < pairs) {
    freq = a.freq[tid];
    if (a.position) {
      const int axis = a.axis ? min(max(a.axis[tid], 0), a.axes - 1) : 0;
      position = a.position[axis * a.position_axis + t];
    }
  }
  // the values of a step: two pieces of eight
  f32x8_t x, y;
  int h = 0, d0 = 0, d1 = 0;
  bool turned = false;
  auto load = [&](int i) {
    const int u = i & (per_head - 1);
    h = i >> shift;
    turned = false;
    if (h < a.q_heads + c.H && !a.interleaved) {
      turned = u * 8 < pairs;
      const int rest = u * 8 - pairs;
      d0 = turned ? u * 8 : 2 * pairs + rest;
      d1 = turned ? pairs + u * 8 : 2 * pairs + rest + (c.D / 2 - pairs);
    } else {
      d0 = u * 8;
      d1 = c.D / 2 + u * 8;
    }
    const int hk = h - a.q_heads, hv = hk - c.H;
    const uint8_t *p = hk < 0 ? a.q + t * a.q_row + h * a.q_head
                       : hv < 0 ? a.rows.nk + t * a.rows.k_row + hk * a.rows.k_head
                                : a.rows.nv + t * a.rows.v_row + hv * a.rows.v_head;
    x = load8<SRC>(p + d0 * SB);
    y = load8<SRC>(p + d1 * SB);
  };
  if (tid < n) load(tid);

  int seq = 0;
  for (int base = 0; base < B; base += 256) {
    const int b = base + tid;
    seq += __syncthreads_count(b < B && a.rows.start[b + 1] <= t);
  }
  if (seq >= B || t < a.rows.start[seq]) return;  // no sequence's row
  const int64_t pos = (int64_t)min(a.rows.len[seq], QGEMV_MAX_CONTEXT) - (min(a.rows.start[seq + 1], T) - t);
  if (tid < pairs) turns[tid] = turn_of(a.position ? position : (int)pos, freq);
  // the row's slot, below 0 where it has none
  int64_t slot = -1;
  if (pos >= 0 && pos < (int64_t)c.width * c.page) {
    const int idx = page_of(c, (int)pos);
    const int id = c.table[(int64_t)seq * c.width + idx];
    if (id >= 0 && id < c.pages) slot = id * c.stride_page + ((int)pos - idx * c.page) * c.stride_slot;
  }
  __syncthreads();

  for (int i = tid; i < n; i += 256) {
    if (i != tid) load(i);
    const int hk = h - a.q_heads, hv = hk - c.H;
    if (turned) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 w = turns[d0 + e];
        const float u = x[e], v = y[e];
        x[e] = u * w.x - v * w.y;
        y[e] = u * w.y + v * w.x;
      }
    } else if (hv < 0 && a.interleaved) {
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        if (d0 < 2 * pairs) {
          const float2 w = turns[(d0 + e) / 2];
          const float u = x[e], v = x[e + 1];
          x[e] = u * w.x - v * w.y;
          x[e + 1] = u * w.y + v * w.x;
        }
        if (d1 < 2 * pairs) {
          const float2 w = turns[(d1 + e) / 2];
          const float u = y[e], v = y[e + 1];
          y[e] = u * w.x - v * w.y;
          y[e + 1] = u * w.y + v * w.x;
        }
      }
    }
    if (hk < 0) {
      uint8_t *const o = a.out + t * a.out_row + h * a.out_head;
      put8<OUT>(o + d0 * 2, x, 1.0f);
      put8<OUT>(o + d1 * 2, y, 1.0f);
    } else if (slot >= 0) {
      uint8_t *const o = hv < 0 ? c.k + slot + hk * c.stride_head : c.v + slot + hv * c.stride_head;
      const float scale = DST != QGEMV_E4M3 ? 1.0f : hv < 0 ? c.k_scale[hk] : c.v_scale[hv];
      put8<DST>(o + d0 * DB, x, scale);
      put8<DST>(o + d1 * DB, y, scale);
    }
  }
}

template <int SRC, int DST>
int launch_rotate_dst(const RotateArgs &a, hipStream_t stream) {
  const dim3 grid(a.rows.T), block(256);
  if (a.out_dtype == QGEMV_BF16)
    hipLaunchKernelGGL((rotate_kernel<SRC, DST, QGEMV_BF16>), grid, block, 0, stream, a);
  else
    hipLaunchKernelGGL((rotate_kernel<SRC, DST, QGEMV_F16>), grid, block, 0, stream, a);
  return hipGetLastError() == hipSuccess ? QGEMV_OK : QGEMV_EHIP;
}

template <int SRC>
int launch_rotate_src(const RotateArgs &a, hipStream_t stream) {
  switch (a.rows.c.dtype) {
    case QGEMV_BF16: return launch_rotate_dst<SRC, QGEMV_BF16>(a, stream);
    case QGEMV_F16: return launch_rotate_dst<SRC, QGEMV_F16>(a, stream);
    case QGEMV_E4M3: return launch_rotate_dst<SRC, QGEMV_E4M3>(a, stream);
  }
  return QGEMV_EINVAL;
}

}  // namespace

int launch_rotate(const RotateArgs &a, hipStream_t stream) {
  switch (a.rows.src) {
    case QGEMV_F32: return launch_rotate_src<QGEMV_F32>(a, stream);
    case QGEMV_BF16: return launch_rotate_src<QGEMV_BF16>(a, stream);
    case QGEMV_F16: return launch_rotate_src<QGEMV_F16>(a, stream);
  }
  return QGEMV_EINVAL;
}

int launch_append(const AppendArgs &a, hipStream_t stream) {
  switch (a.src) {
    case QGEMV_F32: return launch_append_src<QGEMV_F32>(a, stream);
    case QGEMV_BF16: return launch_append_src<QGEMV_BF16>(a, stream);
    case QGEMV_F16: return launch_append_src<QGEMV_F16>(a, stream);
  }
  return QGEMV_EINVAL;
}

}  // namespace qgemv
