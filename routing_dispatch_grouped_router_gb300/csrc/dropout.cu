// Dropout with the residual's addition, from a counter-based generator:
//
//   y = r + (u >= p 2^32 ? x / (1 - p) : 0)
//
// u of element n = row d + column is word n mod 4 of Philox4x32-10 at the counter
// (n / 4, step, site) under the key seed, so that no mask is stored: the backward,
// the same map of dy without a residual, draws it again.
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
  long long groups;  // groups of a row: 8 elements, or the row's blocks of four (kAny)
  uint32_t threshold, site;
  float scale;
  int all;  // every element is dropped
};

namespace {

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

// How the elements are walked: kFlat, contiguous tensors as one row of groups of
// eight (its last elements apart); kRows, rows of whole groups at their strides; kAny,
// rows of any length and alignment, a block of the generator at a time, of whose four
// elements those of the row are taken one by one.
enum class Walk { kFlat, kRows, kAny };
constexpr int kBlocks = 5;  // of an SM

// A group of eight per thread and step, its two blocks of the generator round by round
// together.  SMALL: fewer than 2^34 elements, so that the counter's second word is 0:
// the first two rounds' products of what is alike for all blocks then leave the loop,
// 18 of 20 stay.
//
// Bound by HBM bytes where there are 8 or more of them per element (8192 x 7168, fp32
// and a bf16 residual in: 69 us, floor 70), else by the products: a wide multiplication
// holds its pipe for several cycles (bf16 alone 58 us, floor 35).  Blocks of 256
// threads, five on an SM (two groups per thread 72 and 70 us; eight blocks of 32
// registers 109 and 74).
template <bool XF32, bool YF32, Walk W, bool SMALL>
__global__ void __launch_bounds__(256, kBlocks) dropout_kernel(DropArgs a) {
  using Index = std::conditional_t<SMALL, uint32_t, uint64_t>;
  grid_dep_launch();
  grid_dep_wait();
  const uint64_t seed = static_cast<uint64_t>(a.rng[0]);
  const uint2 key = make_uint2(static_cast<uint32_t>(seed), static_cast<uint32_t>(seed >> 32));
  const uint32_t step = static_cast<uint32_t>(a.rng[1]);
  auto counter = [&](uint64_t block) {
    return make_uint4(static_cast<uint32_t>(block),
                      SMALL ? 0u : static_cast<uint32_t>(block >> 32), step, a.site);
  };
  // (where all are dropped, x is not read but 0)
  auto drop = [&](float x, uint32_t u, float r) {
    return u >= a.threshold ? fmaf(x, a.scale, r) : r;
  };
  const Index stride = gridDim.x * static_cast<Index>(blockDim.x);
  const Index total = static_cast<Index>(a.rows * a.groups);
  const Index groups = static_cast<Index>(a.groups);
  for (Index i = blockIdx.x * static_cast<Index>(blockDim.x) + threadIdx.x; i < total;
       i += stride) {
    if (W == Walk::kAny) {
      const Index row = i / groups, g = i - row * groups;
      const uint64_t n0 = static_cast<uint64_t>(row) * a.cols;  // the row's first element
      const uint64_t block = n0 / 4 + g;
      uint4 u[1] = {counter(block)};
      philox4x32_10(u, key);
      const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const long long c = static_cast<long long>(block * 4 + j - n0);
        if (c < 0 || c >= a.cols) continue;
        put1<YF32>(a.y, row * a.ld_y + c,
                   drop(a.all ? 0.f : get1<XF32>(a.x, row * a.ld_x + c), w[j],
                        a.r ? get1<YF32>(a.r, row * a.ld_r + c) : 0.f));
      }
      continue;
    }
    uint64_t n;  // the group's first element
    long long ix, ir, iy;
    if (W == Walk::kFlat) {
      n = 8 * static_cast<uint64_t>(i);
      if (static_cast<long long>(n) + 8 > a.cols) break;
      ix = ir = iy = static_cast<long long>(n);
    } else {
      const Index row = i / groups;
      const long long c = 8 * static_cast<long long>(i - row * groups);
      n = static_cast<uint64_t>(row) * a.cols + c;
      ix = row * a.ld_x + c;
      ir = row * a.ld_r + c;
      iy = row * a.ld_y + c;
    }
    float x[8], r[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = r[e] = 0.f;
    if (!a.all) get8<XF32>(a.x, ix, x);
    if (a.r) get8<YF32>(a.r, ir, r);
    uint4 u[2] = {counter(n / 4), counter(n / 4 + 1)};
    philox4x32_10(u, key);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      x[4 * h] = drop(x[4 * h], u[h].x, r[4 * h]);
      x[4 * h + 1] = drop(x[4 * h + 1], u[h].y, r[4 * h + 1]);
      x[4 * h + 2] = drop(x[4 * h + 2], u[h].z, r[4 * h + 2]);
      x[4 * h + 3] = drop(x[4 * h + 3], u[h].w, r[4 * h + 3]);
    }
    put8<YF32>(a.y, iy, x);
  }
  if (W == Walk::kFlat && blockIdx.x == 0 && threadIdx.x < a.cols % 8) {  // the last elements
    const long long n = a.cols / 8 * 8 + threadIdx.x;
    uint4 u[1] = {counter(static_cast<uint64_t>(n) / 4)};
    philox4x32_10(u, key);
    const int j = threadIdx.x & 3;
    const uint32_t w = j == 0 ? u[0].x : j == 1 ? u[0].y : j == 2 ? u[0].z : u[0].w;
    put1<YF32>(a.y, n, drop(a.all ? 0.f : get1<XF32>(a.x, n), w,
                            a.r ? get1<YF32>(a.r, n) : 0.f));
  }
}

namespace {

template <bool XF32, bool YF32, Walk W>
cudaError_t launch(const DropArgs& a, bool small, cudaStream_t st) {
  const long long blocks = (a.rows * a.groups + 255) / 256, most = kGb300Sms * kBlocks;
  return launch_dependent(
      small ? dropout_kernel<XF32, YF32, W, true> : dropout_kernel<XF32, YF32, W, false>,
      dim3(static_cast<unsigned>(blocks < most ? blocks : most)), dim3(256), 0, st, a);
}

}  // namespace

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
  const Walk walk = !vec ? Walk::kAny : a.rows > 1 ? Walk::kRows : Walk::kFlat;
  a.groups = walk == Walk::kRows   ? a.cols / 8
             : walk == Walk::kFlat ? (a.cols + 7) / 8
                                   : (a.cols + 3) / 4 + (a.rows > 1 ? 1 : 0);
  const bool small = D.rows * D.d < (1LL << 34) && a.rows * a.groups < (1LL << 31);
  ProfScope prof("dropout", st);
  auto run = [&](auto X, auto Y) {
    constexpr bool f = decltype(X)::value, g = decltype(Y)::value;
    return walk == Walk::kFlat   ? launch<f, g, Walk::kFlat>(a, small, st)
           : walk == Walk::kRows ? launch<f, g, Walk::kRows>(a, small, st)
                                 : launch<f, g, Walk::kAny>(a, small, st);
  };
  cudaError_t e;
  if (xf) e = yf ? run(std::true_type(), std::true_type()) : run(std::true_type(), std::false_type());
  else e = yf ? run(std::false_type(), std::true_type()) : run(std::false_type(), std::false_type());
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace mok
