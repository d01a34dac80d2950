// Rows of elements in registers, for the kernels that keep a row across its
// reductions (norm.cu, post_norm.cu): vectors of eight, their loads and stores at
// any alignment, the row sums and the reciprocal root of a mean square.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "mok_internal.h"
#include "ptx.cuh"

namespace mok {

namespace {

// Eight elements of a row held by one thread.  The rows' vectors v = 0 ..
// ceil(d/8)-1 go round the threads of the row.  VEC: vector v is elements
// 8v .. 8v+7 (one or two 16-byte accesses; 16-byte aligned rows, d a multiple
// of 8).  Otherwise a warp's 32 vectors are 256 elements, of which lane l holds
// pairs 64 j + 2l, + 1 (j = 0..3): a warp's accesses are then whole words that
// follow one another, whatever the row's alignment.  bf16 rows that start in
// the middle of a word are read and written in words too, each lane passing
// one of its two elements to its neighbour (4099 x 2881 bf16 element by element:
// 2.8 times the aligned form's time forward, 5 times backward).
template <bool VEC>
__device__ __forceinline__ int elem_of(int v, int j) {
  return VEC ? 8 * v + j : 256 * (v >> 5) + 64 * (j >> 1) + 2 * (v & 31) + (j & 1);
}

__device__ __forceinline__ uint32_t load_u16(const __nv_bfloat16* p) {
  return *reinterpret_cast<const unsigned short*>(p);
}
__device__ __forceinline__ void store_u16(__nv_bfloat16* p, uint32_t v) {
  *reinterpret_cast<unsigned short*>(p) = static_cast<unsigned short>(v);
}
__device__ __forceinline__ bool mid_word(const __nv_bfloat16* p) {
  return (reinterpret_cast<uintptr_t>(p) & 2) != 0;
}

// The pairs of vector v of a bf16 row (w[j]: elements i, i + 1 with i = 2 lane +
// 64 j + the warp's first).  In a row that starts mid-word, a word holds the
// second element of one pair and the first of the next: each lane gets the other
// half of its word from its neighbour (lane 0 and lane 31 from the pairs before
// and after), and only the warp's two ends are halfwords.  The halves are joined
// by a funnel shift whose amount is 0 for aligned rows.  Whole warps call these.
__device__ __forceinline__ void store_pairs(__nv_bfloat16* p, int v, int d,
                                            const uint32_t (&w)[4]) {
  const int lane = threadIdx.x & 31, i0 = 256 * (v >> 5) + 2 * lane;
  const bool mid = mid_word(p);
  const int back = mid ? 1 : 0;
  uint32_t u[4];  // the word before and at pair j
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t give = lane == 31 && j > 0 ? w[j - 1] : w[j];
    u[j] = __funnelshift_l(__shfl_sync(0xffffffffu, give, (lane + 31) & 31), w[j], 16 * back);
  }
  if (i0 - 2 * lane + 256 <= d) {  // all of the warp's pairs lie in the row
    if (mid && lane == 0) store_u16(p + i0, w[0]);
    else *reinterpret_cast<uint32_t*>(p + i0 - back) = u[0];
#pragma unroll
    for (int j = 1; j < 4; ++j) *reinterpret_cast<uint32_t*>(p + i0 + 64 * j - back) = u[j];
    if (mid && lane == 31) store_u16(p + i0 + 193, w[3] >> 16);
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int i = i0 + 64 * j;
    if (!mid) {
      if (i + 1 < d) *reinterpret_cast<uint32_t*>(p + i) = w[j];
      else if (i < d) store_u16(p + i, w[j]);
    } else {
      if (lane == 0 && j == 0) {
        if (i < d) store_u16(p + i, w[j]);
      } else if (i < d) {
        *reinterpret_cast<uint32_t*>(p + i - 1) = u[j];
      } else if (i == d) {
        store_u16(p + i - 1, u[j]);
      }
    }
  }
}

// A vector as it lies in memory (bf16 stays packed), so that all of a row's
// loads can be in flight before the first is used.  Plain loads: the outputs
// may be the same memory as inputs.  Without VEC whole warps call load and store.
template <bool F32, bool VEC>
struct Raw8 {
  float f[8];
  __device__ __forceinline__ void load(const void* row, int v, int d) {
    if (VEC) {
      const float4* p = reinterpret_cast<const float4*>(row) + 2 * v;
      const float4 a = p[0], b = p[1];
      f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
      f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
      const float* p = static_cast<const float*>(row);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int i = elem_of<false>(v, j);
        f[j] = i < d ? p[i] : 0.f;
      }
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = 0.f;
  }
  __device__ __forceinline__ void get(float (&o)[8]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = f[j];
  }
};
template <>
struct Raw8<false, true> {
  uint4 u;
  __device__ __forceinline__ void load(const void* row, int v, int) {
    u = reinterpret_cast<const uint4*>(row)[v];
  }
  __device__ __forceinline__ void zero() { u = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(float (&o)[8]) const {
    o[0] = bf16lo(u.x); o[1] = bf16hi(u.x); o[2] = bf16lo(u.y); o[3] = bf16hi(u.y);
    o[4] = bf16lo(u.z); o[5] = bf16hi(u.z); o[6] = bf16lo(u.w); o[7] = bf16hi(u.w);
  }
};
// The words of store_pairs' layout as they lie in memory, and the warp's last
// element; the lanes exchange halves in get, so that no load waits for a shuffle.
template <>
struct Raw8<false, false> {
  uint32_t a[4], end;
  int shift;  // 16: the row starts mid-word
  __device__ __forceinline__ void load(const void* row, int v, int d) {
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(row);
    const int lane = threadIdx.x & 31, first = 256 * (v >> 5), i0 = first + 2 * lane;
    const bool mid = mid_word(p);
    const int back = mid ? 1 : 0;
    shift = 16 * back;
    end = 0u;
    if (first + 256 <= d) {  // all of the warp's pairs lie in the row
      a[0] = mid && i0 == 0 ? load_u16(p) << 16 : *reinterpret_cast<const uint32_t*>(p + i0 - back);
#pragma unroll
      for (int j = 1; j < 4; ++j)
        a[j] = *reinterpret_cast<const uint32_t*>(p + i0 + 64 * j - back);
      if (mid && lane == 31) end = load_u16(p + i0 + 193);
      return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = i0 + 64 * j;
      a[j] = 0u;
      if (!mid) {
        if (i + 1 < d) a[j] = *reinterpret_cast<const uint32_t*>(p + i);
        else if (i < d) a[j] = load_u16(p + i);
      } else {
        if (i < d) a[j] = i > 0 ? *reinterpret_cast<const uint32_t*>(p + i - 1) : load_u16(p) << 16;
        else if (i == d) a[j] = load_u16(p + i - 1);
      }
    }
  }
  __device__ __forceinline__ void zero() {
    a[0] = a[1] = a[2] = a[3] = end = 0u;
    shift = 0;
  }
  __device__ __forceinline__ void get(float (&o)[8]) const {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t give = lane == 0 && j < 3 ? a[j < 3 ? j + 1 : 3] : a[j];
      uint32_t n = __shfl_sync(0xffffffffu, give, (lane + 1) & 31);
      if (j == 3 && lane == 31) n = end;
      const uint32_t w = __funnelshift_r(a[j], n, shift);
      o[2 * j] = bf16lo(w);
      o[2 * j + 1] = bf16hi(w);
    }
  }
};

template <bool F32, bool VEC>
__device__ __forceinline__ void load8(const void* row, int v, int d, float (&o)[8]) {
  Raw8<F32, VEC> r;
  r.load(row, v, d);
  r.get(o);
}

template <bool F32, bool VEC>
__device__ __forceinline__ void store8(void* row, int v, int d, const float (&o)[8]) {
  if (F32) {
    if (VEC) {
      float4* p = reinterpret_cast<float4*>(row) + 2 * v;
      p[0] = make_float4(o[0], o[1], o[2], o[3]);
      p[1] = make_float4(o[4], o[5], o[6], o[7]);
    } else {
      float* p = static_cast<float*>(row);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int i = elem_of<false>(v, j);
        if (i < d) p[i] = o[j];
      }
    }
  } else {
    const uint4 u = make_uint4(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]),
                               pack_bf16x2(o[4], o[5]), pack_bf16x2(o[6], o[7]));
    if (VEC) {
      reinterpret_cast<uint4*>(row)[v] = u;
    } else {
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
      store_pairs(static_cast<__nv_bfloat16*>(row), v, d, w);
    }
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// 1 / sqrt(sum / d + eps), to within an ulp: the hardware's approximation and one
// Newton step with the residual 1 - v r^2 in twice the precision.  An error of
// rstd shifts a whole row, and with it which E4M3 code its values round to.
__device__ __forceinline__ float row_rstd(float sum, float d, float eps) {
  const float v = __fdiv_rn(sum, d) + eps;
  const float r = rsqrtf(v);
  const float h = v * r, l = fmaf(v, r, -h);
  const float e = fmaf(-h, r, 1.0f) - l * r;
  // (v = 0 or infinite: r is infinite or 0 and e not a number)
  return fabsf(e) < 1.0f ? fmaf(0.5f * r, e, r) : r;
}

// Row `r` of an array with row stride ld, F32 or bf16 elements.
template <bool F32>
__device__ __forceinline__ const void* row_at(const void* base, long long r, long long ld) {
  return static_cast<const char*>(base) + r * ld * (F32 ? 4 : 2);
}
template <bool F32>
__device__ __forceinline__ void* row_at(void* base, long long r, long long ld) {
  return static_cast<char*>(base) + r * ld * (F32 ? 4 : 2);
}

// Threads of a row (a multiple of 32) and vectors per thread (1, 2 or 4; at
// most 1024 threads of one vector, 512 of more).  Few rows: one vector per
// thread where that fits, so that a row's loads are all in flight at once.
// Many rows: up to max_nv, so that several rows share an SM.
inline void norm_shape(long long rows, int nvec, int max_nv, int* tpr, int* nv) {
  int n = rows >= 4LL * kGb300Sms ? max_nv : 1;
  if (nvec > 1024) n = 4;
  while (n > 1 && nvec <= 32 * (n / 2)) n /= 2;
  const int th = (nvec + n - 1) / n;
  *tpr = (th + 31) / 32 * 32;
  *nv = n;
}

inline bool vec_rows(const void* p, long long ld, int esz) {
  return p == nullptr || ((reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld * esz % 16 == 0);
}

}  // namespace

}  // namespace mok
