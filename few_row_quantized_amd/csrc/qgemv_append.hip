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

}  // namespace

int launch_append(const AppendArgs &a, hipStream_t stream) {
  switch (a.src) {
    case QGEMV_F32: return launch_append_src<QGEMV_F32>(a, stream);
    case QGEMV_BF16: return launch_append_src<QGEMV_BF16>(a, stream);
    case QGEMV_F16: return launch_append_src<QGEMV_F16>(a, stream);
  }
  return QGEMV_EINVAL;
}

}  // namespace qgemv
