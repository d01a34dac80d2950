// Dropout with the residual's addition, from a counter-based generator:
//
//   y = r + (u >= p 2^32 ? x / (1 - p) : 0)
//
// u of element n = row d + column is word n mod 4 of Philox4x32-10 at the counter
// (n / 4, step, site) under the key seed, so that no mask is stored: the backward,
// the same map of dy without a residual, draws it again.
//
// Bound by HBM bytes: 20 wide multiplications per four elements stay below the
// time of their 16 to 48 bytes.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "mok_internal.h"
#include "philox.cuh"
#include "ptx.cuh"

namespace mok {

struct DropArgs {
  const void *x, *r;
  const int64_t* rng;  // seed, step
  void* y;
  long long rows, ld_x, ld_r, ld_y;
  long long cols;    // elements of a row as it is walked (FLAT: all of them, one row)
  long long groups;  // groups of a row: 8 elements (VEC), or the row's blocks of four
  uint32_t threshold, site;
  float scale;
  int all;  // every element is dropped
};

namespace {

__device__ __forceinline__ uint4 words(const DropArgs& a, uint2 key, uint32_t step,
                                       uint64_t block) {
  return philox4x32_10(make_uint4(static_cast<uint32_t>(block), static_cast<uint32_t>(block >> 32),
                                  step, a.site),
                       key);
}

template <bool F32>
__device__ __forceinline__ void get8(const void* base, long long i, float (&o)[8]) {
  if (F32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
    const float4 a = p[0], b = p[1];
    o[0] = a.x; o[1] = a.y; o[2] = a.z; o[3] = a.w;
    o[4] = b.x; o[5] = b.y; o[6] = b.z; o[7] = b.w;
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + i);
    o[0] = bf16lo(u.x); o[1] = bf16hi(u.x); o[2] = bf16lo(u.y); o[3] = bf16hi(u.y);
    o[4] = bf16lo(u.z); o[5] = bf16hi(u.z); o[6] = bf16lo(u.w); o[7] = bf16hi(u.w);
  }
}
template <bool F32>
__device__ __forceinline__ void put8(void* base, long long i, const float (&o)[8]) {
  if (F32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + i);
    p[0] = make_float4(o[0], o[1], o[2], o[3]);
    p[1] = make_float4(o[4], o[5], o[6], o[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + i) =
        make_uint4(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]),
                   pack_bf16x2(o[6], o[7]));
  }
}
template <bool F32>
__device__ __forceinline__ float get1(const void* base, long long i) {
  return F32 ? static_cast<const float*>(base)[i]
             : __bfloat162float(static_cast<const __nv_bfloat16*>(base)[i]);
}
template <bool F32>
__device__ __forceinline__ void put1(void* base, long long i, float v) {
  if (F32) static_cast<float*>(base)[i] = v;
  else static_cast<__nv_bfloat16*>(base)[i] = __float2bfloat16_rn(v);
}

}  // namespace

// VEC: rows of whole, aligned groups of eight elements (contiguous tensors: one row
// of them all, its last elements apart).  Otherwise a group is a block of the
// generator, of whose four elements those of the row are taken one by one.
template <bool XF32, bool YF32, bool VEC>
__global__ void __launch_bounds__(256) dropout_kernel(DropArgs a) {
  grid_dep_launch();
  grid_dep_wait();
  const uint64_t seed = static_cast<uint64_t>(a.rng[0]);
  const uint2 key = make_uint2(static_cast<uint32_t>(seed), static_cast<uint32_t>(seed >> 32));
  const uint32_t step = static_cast<uint32_t>(a.rng[1]);
  auto drop = [&](float x, uint32_t u, float r) {
    return u >= a.threshold && !a.all ? fmaf(x, a.scale, r) : r;
  };
  // (one division; then row and group advance together)
  const long long first = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  const long long stride = static_cast<long long>(gridDim.x) * blockDim.x;
  long long row = first / a.groups, g = first - row * a.groups;
  const long long row_step = stride / a.groups, g_step = stride - row_step * a.groups;
  while (row < a.rows) {
    if (VEC) {
      const uint64_t n = static_cast<uint64_t>(row) * a.cols + 8 * g;
      const long long ix = row * a.ld_x + 8 * g, ir = row * a.ld_r + 8 * g,
                      iy = row * a.ld_y + 8 * g;
      if (8 * g + 8 <= a.cols) {
        float x[8], r[8];
        get8<XF32>(a.x, ix, x);
        if (a.r) {
          get8<YF32>(a.r, ir, r);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) r[j] = 0.f;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 u = words(a, key, step, n / 4 + h);
          x[4 * h] = drop(x[4 * h], u.x, r[4 * h]);
          x[4 * h + 1] = drop(x[4 * h + 1], u.y, r[4 * h + 1]);
          x[4 * h + 2] = drop(x[4 * h + 2], u.z, r[4 * h + 2]);
          x[4 * h + 3] = drop(x[4 * h + 3], u.w, r[4 * h + 3]);
        }
        put8<YF32>(a.y, iy, x);
      } else {  // the last elements of a contiguous tensor
        const int left = static_cast<int>(a.cols - 8 * g);
        for (int j = 0; j < left; ++j) {
          const uint4 u = words(a, key, step, (n + j) / 4);
          const uint32_t w = (j & 3) == 0 ? u.x : (j & 3) == 1 ? u.y : (j & 3) == 2 ? u.z : u.w;
          put1<YF32>(a.y, iy + j,
                     drop(get1<XF32>(a.x, ix + j), w, a.r ? get1<YF32>(a.r, ir + j) : 0.f));
        }
      }
    } else {
      const uint64_t n0 = static_cast<uint64_t>(row) * a.cols;  // the row's first element
      const uint64_t block = n0 / 4 + g;
      const uint4 u = words(a, key, step, block);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const long long c = static_cast<long long>(block * 4 + j - n0);
        if (c < 0 || c >= a.cols) continue;
        put1<YF32>(a.y, row * a.ld_y + c,
                   drop(get1<XF32>(a.x, row * a.ld_x + c), w[j],
                        a.r ? get1<YF32>(a.r, row * a.ld_r + c) : 0.f));
      }
    }
    row += row_step;
    g += g_step;
    if (g >= a.groups) {
      g -= a.groups;
      ++row;
    }
  }
}

cudaError_t launch_dropout(const mok_dropout_desc& D, const void* x, const void* res,
                           const int64_t* rng, void* y, cudaStream_t st) {
  if (D.rows == 0) return cudaSuccess;
  const bool xf = D.x_elem == MOK_ELEM_F32, yf = D.y_elem == MOK_ELEM_F32;
  const int xe = xf ? 4 : 2, ye = yf ? 4 : 2;
  DropArgs a;
  a.x = x; a.r = res; a.rng = rng; a.y = y;
  a.rows = D.rows;
  a.cols = D.d;
  a.ld_x = D.ld_x; a.ld_r = D.ld_res; a.ld_y = D.ld_y;
  const uint64_t t = dropout_threshold(D.p);
  a.all = t > 0xFFFFFFFFull;
  a.threshold = static_cast<uint32_t>(a.all ? 0 : t);
  a.scale = a.all ? 0.f : static_cast<float>(1.0 / (1.0 - D.p));
  a.site = D.site;
  if (a.rows == 1 || (a.ld_x == a.cols && a.ld_y == a.cols && (!res || a.ld_r == a.cols))) {
    a.cols *= a.rows;
    a.rows = 1;
  }
  auto aligned = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
  bool vec = aligned(x) && aligned(res) && aligned(y);
  if (a.rows > 1)
    vec = vec && a.cols % 8 == 0 && a.ld_x * xe % 16 == 0 && a.ld_y * ye % 16 == 0 &&
          (!res || a.ld_r * ye % 16 == 0);
  a.groups = vec ? (a.cols + 7) / 8 : (a.cols + 3) / 4 + (a.rows > 1 ? 1 : 0);
  const long long blocks = (a.rows * a.groups + 255) / 256;
  const unsigned grid = static_cast<unsigned>(blocks < kGb300Sms * 8 ? blocks : kGb300Sms * 8);
  ProfScope prof("dropout", st);
  auto run = [&](auto X, auto Y) {
    constexpr bool f = decltype(X)::value, g = decltype(Y)::value;
    return launch_dependent(vec ? dropout_kernel<f, g, true> : dropout_kernel<f, g, false>,
                            dim3(grid), dim3(256), 0, st, a);
  };
  cudaError_t e;
  if (xf) e = yf ? run(std::true_type(), std::true_type()) : run(std::true_type(), std::false_type());
  else e = yf ? run(std::false_type(), std::true_type()) : run(std::false_type(), std::false_type());
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace mok
