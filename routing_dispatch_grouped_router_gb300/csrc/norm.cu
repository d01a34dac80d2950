// Residual addition with RMS norm, forward (bf16 and MXFP8 out) and backward.
//
//   s = x + r (rounded once to the stream's type),  y = w s rstd,
//   rstd = 1 / sqrt(mean(s^2) + eps)
//   backward: n = s rstd, g = dy w:  dx = rstd (g - n mean(g n)) + ds,
//   dw = sum over rows of dy n
//
// Bound by HBM bytes: a row is read once, kept in registers across the row
// reductions and written once.  (8192 x 7168 to MXFP8, fp32 into a bf16 stream:
// 106 us, 6.1 TB/s; backward of 16384 x 4096 fp32: 161.5 us, 6.7 TB/s; a copy runs
// at 6.8.  4099 x 2880 bf16 backward: 22.7 us, floor 13.9, a third of it the ramp
// of a few rows per block and the column sums' kernel.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "mok_internal.h"
#include "mx.cuh"
#include "ptx.cuh"
#include "rows.cuh"

namespace mok {

namespace {

// An unevaluated sum hi + lo of two fp32 values, lo far below hi.
struct Pair {
  float hi, lo;
};
// (the _rn forms: these must not be contracted into fused products)
__device__ __forceinline__ Pair two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Pair pair_add(Pair a, Pair b) {
  Pair s = two_sum(a.hi, b.hi);
  s.lo += a.lo + b.lo;
  return s;  // (an infinite sum has a low part that is no number: row_rstd drops it)
}
// The sum of a thread's squares as a pair.  The sum starts at a power of two that
// no square exceeds, so that hi - s is exact at every step and the second fused
// product gives what the step rounded away, the square's own low bits with it; it
// is taken off in the end, exactly.  (A general error-free addition takes twice the
// instructions: 8192 x 7168 109.9 us so.)  plain: their sum in fp32, for squares
// near or past the end of its range.
template <int N>
__device__ __forceinline__ Pair sum_squares(const float (&v)[N][8], float plain) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(v[i][j]));
  top = __fmul_rn(top, top);
  if (!(top < 0x1p120f)) return {plain, 0.f};
  const float c = __uint_as_float((__float_as_uint(top) & 0x7f800000u) + 0x00800000u);
  Pair s = {c, 0.f};
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float hi = __fmaf_rn(v[i][j], v[i][j], s.hi);
      s.lo = __fadd_rn(s.lo, __fmaf_rn(v[i][j], v[i][j], __fsub_rn(s.hi, hi)));
      s.hi = hi;
    }
  s.hi = __fsub_rn(s.hi, c);
  return s;  // (a NaN is not in `top`, but in both sums)
}
__device__ __forceinline__ Pair warp_sum(Pair v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    v = pair_add(v, {__shfl_xor_sync(0xffffffffu, v.hi, o), __shfl_xor_sync(0xffffffffu, v.lo, o)});
  return v;
}

// row_rstd as a pair, from the sum of squares as one.
__device__ __forceinline__ Pair row_rstd(Pair sum, float d, float eps) {
  const float q = __fdiv_rn(sum.hi, d);
  Pair v = two_sum(q, eps);
  v.lo += (fmaf(-q, d, sum.hi) + sum.lo) / d;
  // the low parts of many terms may add up: hi once more the nearest value, so
  // that the Newton step starts from rsqrtf's error alone (no number: see above)
  if (fabsf(v.lo) < INFINITY) v = two_sum(v.hi, v.lo);
  const float r = rsqrtf(v.hi);
  const float h = v.hi * r, l = fmaf(v.hi, r, -h) + v.lo * r;
  const float e = fmaf(-h, r, 1.0f) - l * r;
  if (!(fabsf(e) < 1.0f)) return {r, 0.f};  // the mean square is 0, infinite or NaN
  return {r, 0.5f * r * e};
}

// s rstd w, rounded to odd: cut off, with the last bit set where anything was
// cut.  A further rounding to fewer bits then gives what rounding the exact
// value would.
__device__ __forceinline__ float norm_to_odd(float s, Pair rstd, float w) {
  const float q = __fmul_rn(s, rstd.hi);
  const float ql = fmaf(s, rstd.lo, fmaf(s, rstd.hi, -q));
  const float m = __fmul_rn(q, w);
  const float ml = fmaf(ql, w, fmaf(q, w, -m));
  const float n = __fadd_rz(m, ml);
  const float rest = __fsub_rn(ml, __fsub_rn(n, m));
  // (not where n is infinite: the rest is no number then)
  return fabsf(rest) > 0.f ? __uint_as_float(__float_as_uint(n) | 1u) : n;
}

}  // namespace

struct NormFwd {
  const void *x, *r, *w;
  void *s, *y, *values;
  uint8_t *codes, *scales;
  long long rows, ld_x, ld_r, ld_s, ld_y;
  int d, nvec, w_f32;
  float eps;
};

// MXFP8 of the vector's elements: the block's 32 columns are 4 threads'
// vectors (VEC) or a pair of each of 16 lanes.
template <bool VEC>
__device__ __forceinline__ void mx_store(const NormFwd& a, long long r, int v, bool in,
                                         const float (&n)[8]) {
  if (VEC) {
    float amax = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(n[j]));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    if (!in) return;
    const int shared = mx_shared_exp(amax);
    const float down = exp2i(-shared), up = exp2i(shared);
    uint32_t w[2];
    float q[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint16_t p01 = cvt_e4m3x2(n[4 * h + 1] * down, n[4 * h] * down);
      const uint16_t p23 = cvt_e4m3x2(n[4 * h + 3] * down, n[4 * h + 2] * down);
      w[h] = static_cast<uint32_t>(p01) | (static_cast<uint32_t>(p23) << 16);
      e4m3x2_to_f32(p01, &q[4 * h + 1], &q[4 * h]);
      e4m3x2_to_f32(p23, &q[4 * h + 3], &q[4 * h + 2]);
    }
    if (a.codes) {
      *reinterpret_cast<uint2*>(a.codes + r * a.d + 8 * v) = make_uint2(w[0], w[1]);
      if ((v & 3) == 0)
        a.scales[r * (a.d >> 5) + (v >> 2)] = static_cast<uint8_t>(shared + 127);
    }
    if (a.values) {
#pragma unroll
      for (int j = 0; j < 8; ++j) q[j] *= up;
      store8<false, true>(static_cast<__nv_bfloat16*>(a.values) + r * a.d, v, a.d, q);
    }
  } else {
    // a block is a pair of each of 16 lanes
    uint32_t vals[4];
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      float amax = fmaxf(fabsf(n[j]), fabsf(n[j + 1]));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const int i = elem_of<false>(v, j);  // (d is a multiple of 32: i and i + 1 alike)
      const int shared = mx_shared_exp(amax);
      const float down = exp2i(-shared), up = exp2i(shared);
      const uint16_t p = cvt_e4m3x2(n[j + 1] * down, n[j] * down);
      if (a.codes && in && i < a.d) {
        a.codes[r * a.d + i] = static_cast<uint8_t>(p & 0xFFu);
        a.codes[r * a.d + i + 1] = static_cast<uint8_t>(p >> 8);
        if ((i & 31) == 0)
          a.scales[r * (a.d >> 5) + (i >> 5)] = static_cast<uint8_t>(shared + 127);
      }
      float hi, lo;
      e4m3x2_to_f32(p, &hi, &lo);
      vals[j >> 1] = pack_bf16x2(lo * up, hi * up);
    }
    if (a.values && in)  // (in: alike for the warp)
      store_pairs(static_cast<__nv_bfloat16*>(a.values) + r * a.d, v, a.d, vals);
  }
}

// One row per threadIdx.y; blockDim.x threads of whole warps hold it, NV
// vectors each.  MX: mean square and norm are formed in pairs of fp32 and the norm
// rounded to odd: codes and values are the roundings of the norm to within 2^-42 of
// it, the exact one's unless it lies that near a boundary.  A plain fp32 norm lands
// on the wrong side of an E4M3 boundary about once in a million values, an eighth of
// the value each time (8192 x 7168: 96.5 us from plain fp32, 105.9 us so).
template <bool XF32, bool SF32, bool VEC, int NV, bool MX>
__global__ void __launch_bounds__(NV == 1 ? 1024 : 512) add_rmsnorm_kernel(NormFwd a) {
  __shared__ float red[3][32];
  grid_dep_launch();
  grid_dep_wait();
  const int t = threadIdx.x, tpr = blockDim.x;
  const long long r = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
  const bool row_in = r < a.rows;
  Raw8<XF32, VEC> x[NV];
  Raw8<SF32, VEC> res[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int vi = t + i * tpr;
    x[i].zero();
    res[i].zero();
    if (row_in && vi < a.nvec) {
      x[i].load(row_at<XF32>(a.x, r, a.ld_x), vi, a.d);
      if (a.r) res[i].load(row_at<SF32>(a.r, r, a.ld_r), vi, a.d);
    }
  }
  float v[NV][8];
  float sq[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int vi = t + i * tpr;
    x[i].get(v[i]);
    if (a.r) {
      float b[8];
      res[i].get(b);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[i][j] += b[j];
        if (!SF32) v[i][j] = bf16_round(v[i][j]);
      }
    }
    if (a.s && row_in && vi < a.nvec)
      store8<SF32, VEC>(row_at<SF32>(a.s, r, a.ld_s), vi, a.d, v[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) sq[j] = fmaf(v[i][j], v[i][j], sq[j]);
  }
  const float df = static_cast<float>(a.d);
  float sum = ((sq[0] + sq[1]) + (sq[2] + sq[3])) + ((sq[4] + sq[5]) + (sq[6] + sq[7]));
  Pair sum2 = {0.f, 0.f};
  if (MX) sum2 = warp_sum(sum_squares<NV>(v, sum));
  sum = warp_sum(sum);
  if (tpr > 32) {  // one row per block
    if ((t & 31) == 0) {
      red[0][t >> 5] = sum;
      if (MX) {
        red[1][t >> 5] = sum2.hi;
        red[2][t >> 5] = sum2.lo;
      }
    }
    __syncthreads();
    const bool in = (t & 31) < (tpr >> 5);
    sum = warp_sum(in ? red[0][t & 31] : 0.f);
    if (MX) sum2 = warp_sum(Pair{in ? red[1][t & 31] : 0.f, in ? red[2][t & 31] : 0.f});
  }
  const float rstd = row_rstd(sum, df, a.eps);
  Pair rstd2 = {0.f, 0.f};
  if (MX) rstd2 = row_rstd(sum2, df, a.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int vi = t + i * tpr;
    const bool in = row_in && vi < a.nvec;
    if (!MX && !in) continue;
    float w[8];
    if (in) {
      if (a.w_f32) load8<true, VEC>(a.w, vi, a.d, w);
      else load8<false, VEC>(a.w, vi, a.d, w);
    }
    if (in && a.y) {
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = v[i][j] * rstd * w[j];
      store8<false, VEC>(row_at<false>(a.y, r, a.ld_y), vi, a.d, y);
    }
    if (MX) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = in ? norm_to_odd(v[i][j], rstd2, w[j]) : 0.f;
    }
    if (MX) mx_store<VEC>(a, r, vi, in, v[i]);
  }
}

namespace {

template <bool XF32, bool SF32, bool VEC, bool MX>
cudaError_t fwd_launch(const NormFwd& a, cudaStream_t st) {
  int tpr, nv;
  norm_shape(a.rows, a.nvec, 4, &tpr, &nv);
  const int rpb = tpr == 32 ? 4 : 1;
  const dim3 block(tpr, rpb);
  const unsigned grid = static_cast<unsigned>((a.rows + rpb - 1) / rpb);
  ProfScope prof("add_rmsnorm", st);
  auto kern = nv == 1 ? add_rmsnorm_kernel<XF32, SF32, VEC, 1, MX>
                      : (nv == 2 ? add_rmsnorm_kernel<XF32, SF32, VEC, 2, MX>
                                 : add_rmsnorm_kernel<XF32, SF32, VEC, 4, MX>);
  const cudaError_t e = launch_dependent(kern, dim3(grid), block, 0, st, a);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <bool XF32, bool SF32>
cudaError_t fwd_pick(const NormFwd& a, bool vec, bool mx, cudaStream_t st) {
  if (vec) return mx ? fwd_launch<XF32, SF32, true, true>(a, st)
                     : fwd_launch<XF32, SF32, true, false>(a, st);
  return mx ? fwd_launch<XF32, SF32, false, true>(a, st)
            : fwd_launch<XF32, SF32, false, false>(a, st);
}

}  // namespace

cudaError_t launch_add_rmsnorm(const mok_rmsnorm_desc& D, const void* x, const void* res,
                               const void* w, void* s, void* y, void* values, uint8_t* codes,
                               uint8_t* scales, cudaStream_t st) {
  if (D.rows == 0) return cudaSuccess;
  const bool xf = D.x_elem == MOK_ELEM_F32, sf = D.s_elem == MOK_ELEM_F32;
  NormFwd a;
  a.x = x; a.r = res; a.w = w; a.s = s; a.y = y; a.values = values;
  a.codes = codes; a.scales = scales;
  a.rows = D.rows;
  a.ld_x = D.ld_x; a.ld_r = D.ld_res; a.ld_s = D.ld_s; a.ld_y = D.ld_y;
  a.d = static_cast<int>(D.d);
  a.nvec = (a.d + 7) / 8;
  a.w_f32 = D.weight_elem == MOK_ELEM_F32;
  a.eps = D.eps;
  const int xe = xf ? 4 : 2, se = sf ? 4 : 2;
  const bool vec = a.d % 8 == 0 && vec_rows(x, a.ld_x, xe) && vec_rows(res, a.ld_r, se) &&
                   vec_rows(s, a.ld_s, se) && vec_rows(y, a.ld_y, 2) && vec_rows(w, 0, 4) &&
                   vec_rows(values, a.d, 2) && (reinterpret_cast<uintptr_t>(codes) & 7) == 0;
  if (!vec) a.nvec = (a.d + 255) / 256 * 32;  // whole groups of 256 elements
  const bool mx = values || codes;
  if (xf) return sf ? fwd_pick<true, true>(a, vec, mx, st) : fwd_pick<true, false>(a, vec, mx, st);
  return sf ? fwd_pick<false, true>(a, vec, mx, st) : fwd_pick<false, false>(a, vec, mx, st);
}

// ----------------------------------------------------------------- backward --

constexpr int kBulkMaxDepth = 4;
struct NormBwd {
  int* status;
  const void *dy, *s, *w, *ds;
  void* dx;
  float* part;  // [gridDim.x, d] partial weight gradients (NULL: not computed)
  long long rows, ld_dy, ld_s, ld_ds, ld_dx;
  int d, nvec, w_f32;
  int ld8;  // SHIFT: elements from one row to the next, mod 8
  float inv_d, eps;
};

// The three inputs of a thread's vectors of one row.
template <bool DYF32, bool SF32, bool VEC, int NV>
struct BwdRow {
  Raw8<SF32, VEC> s[NV], ds[NV];
  Raw8<DYF32, VEC> dy[NV];
  __device__ __forceinline__ void load(const NormBwd& a, long long r, int t, int tpr) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int vi = t + i * tpr;
      s[i].zero();
      dy[i].zero();
      ds[i].zero();
      if (r < a.rows && vi < a.nvec) {
        s[i].load(row_at<SF32>(a.s, r, a.ld_s), vi, a.d);
        dy[i].load(row_at<DYF32>(a.dy, r, a.ld_dy), vi, a.d);
        if (a.ds) ds[i].load(row_at<SF32>(a.ds, r, a.ld_ds), vi, a.d);
      }
    }
  }
};

// blockDim.x threads of whole warps hold a row, blockDim.y rows are in a block
// at a time (more than one only for rows of one warp).  Row group b takes rows
// b, b + groups, ..; its threads keep the weight gradient of their columns in
// registers over those rows.
template <bool DYF32, bool SF32, bool VEC, int NV>
__global__ void __launch_bounds__(512) add_rmsnorm_bwd_kernel(NormBwd a) {
  __shared__ float red[2][2][16];  // [row parity][sum][warp]
  __shared__ float s_dw[NV <= 2 ? 8 : 1][NV * 256];
  grid_dep_launch();
  grid_dep_wait();
  const int t = threadIdx.x, tpr = blockDim.x, nw = tpr >> 5;
  float dw[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.f;
  const long long step = static_cast<long long>(gridDim.x) * blockDim.y;
  long long r = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
  for (int par = 0; r < a.rows; r += step, par ^= 1) {
    BwdRow<DYF32, SF32, VEC, NV> row;
    row.load(a, r, t, tpr);
    float ss = 0.f, gs = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int vi = t + i * tpr;
      if (vi < a.nvec) {
        float w[8], s[8], dy[8];
        if (a.w_f32) load8<true, VEC>(a.w, vi, a.d, w);
        else load8<false, VEC>(a.w, vi, a.d, w);
        row.s[i].get(s);
        row.dy[i].get(dy);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          ss = fmaf(s[j], s[j], ss);
          gs = fmaf(dy[j] * w[j], s[j], gs);
        }
      }
    }
    ss = warp_sum(ss);
    gs = warp_sum(gs);
    if (nw > 1) {
      if ((t & 31) == 0) {
        red[par][0][t >> 5] = ss;
        red[par][1][t >> 5] = gs;
      }
      __syncthreads();  // (the other parity's buffer may still be read)
      const bool in = (t & 31) < nw;
      ss = warp_sum(in ? red[par][0][t & 31] : 0.f);
      gs = warp_sum(in ? red[par][1][t & 31] : 0.f);
    }
    const float rstd = row_rstd(ss, static_cast<float>(a.d), a.eps);
    const float c = gs * rstd * rstd * a.inv_d;  // rstd mean(g n) = c; n c = s rstd c
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int vi = t + i * tpr;
      if (vi >= a.nvec) continue;
      float w[8], s[8], dy[8], o[8];
      if (a.w_f32) load8<true, VEC>(a.w, vi, a.d, w);
      else load8<false, VEC>(a.w, vi, a.d, w);
      row.s[i].get(s);
      row.dy[i].get(dy);
      row.ds[i].get(o);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        o[j] = rstd * (dy[j] * w[j] - s[j] * c) + o[j];
        dw[i][j] = fmaf(dy[j], s[j] * rstd, dw[i][j]);
      }
      store8<SF32, VEC>(row_at<SF32>(a.dx, r, a.ld_dx), vi, a.d, o);
    }
  }
  if (!a.part) return;
  float* p = a.part + static_cast<long long>(blockIdx.x) * a.d;
  if (blockDim.y > 1) {  // rows of one warp: the block's rows in order
    if (NV <= 2) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) s_dw[threadIdx.y][(t + 32 * i) * 8 + j] = dw[i][j];
      __syncthreads();
      for (int i = threadIdx.y * 32 + t; i < NV * 256; i += 256) {  // vector i / 8
        float v = 0.f;
#pragma unroll
        for (int y = 0; y < 8; ++y) v += s_dw[y][i];
        const int e = elem_of<VEC>(i >> 3, i & 7);
        if ((i >> 3) < a.nvec && e < a.d) p[e] = v;
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int vi = t + i * tpr;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = elem_of<VEC>(vi, j);
      if (vi < a.nvec && e < a.d) p[e] = dw[i][j];
    }
  }
}

// The same for aligned rows of at least kBulkMinD elements: rows come into a
// ring of `depth` rows in shared memory by bulk copies (s, dy, ds each one
// copy), issued a row or more ahead, so that the reductions and barriers of one
// row do not interrupt the stream of loads.  A slot is filled again after the
// next row's barrier, which every thread reaches only when done with it.
//
// SHIFT: rows of any length in aligned tensors.  Row r begins r ld8 elements (mod
// 8) past a multiple of eight, in all of them alike; a block's rows are a multiple
// of eight apart, so all of its rows begin at the same h.  A thread's eight columns
// are 8 v - h .. + 7: aligned words everywhere, and fixed columns for its weights
// and their gradients.  The copies take whole 16-byte words (a few elements of the
// rows next to it with them), except past the end of the last row.
// (13142 x 2373 bf16: 55 us, 148 by word loads; floor 37.  8192 x 4095 fp32: 88 and
// 111; floor 79.)
constexpr int kBulkMinD = 1024;
constexpr int kShiftMinD = 512;
template <bool F32>
__device__ __forceinline__ void bulk_row(uint8_t* dst, const void* base, long long r, long long ld,
                                         int h, uint32_t bytes, uint32_t whole, uint64_t* bar) {
  constexpr int es = F32 ? 4 : 2;
  const char* src = static_cast<const char*>(row_at<F32>(base, r, ld)) - h * es;
  bulk_load(dst, src, whole, bar);
  for (uint32_t i = whole; i < bytes; i += es) {  // (the last row's last elements)
    if (F32) *reinterpret_cast<float*>(dst + i) = *reinterpret_cast<const float*>(src + i);
    else *reinterpret_cast<uint16_t*>(dst + i) = *reinterpret_cast<const uint16_t*>(src + i);
  }
}

// (launch bounds: the registers that 768 threads on an SM leave, see bwd_shape)
template <bool DYF32, bool SF32, int NV, bool SHIFT>
__global__ void __launch_bounds__(NV == 2 ? 768 : 512)
    add_rmsnorm_bwd_bulk_kernel(NormBwd a, int depth) {
  extern __shared__ __align__(128) uint8_t s_rows[];
  __shared__ __align__(8) uint64_t full[kBulkMaxDepth];
  __shared__ float red[2][2][16];
  __shared__ int s_abort;
  grid_dep_launch();
  const int t = threadIdx.x, tpr = blockDim.x, nw = tpr >> 5;
  const int h = SHIFT ? (blockIdx.x * a.ld8) & 7 : 0;
  const int nvec = SHIFT ? (a.d + h + 7) >> 3 : a.nvec;
  const uint32_t s_bytes = nvec * (SF32 ? 32 : 16), y_bytes = nvec * (DYF32 ? 32 : 16);
  const uint32_t row_bytes = s_bytes + y_bytes + (a.ds ? s_bytes : 0);
  if (t == 0) {
    for (int i = 0; i < depth; ++i) mbar_init(&full[i], 1);
    s_abort = 0;
    fence_barrier_init();
  }
  __syncthreads();
  grid_dep_wait();
  volatile int* vabort = &s_abort;
  auto fill = [&](int slot, long long r) {  // thread 0
    uint8_t* p = s_rows + slot * row_bytes;
    if (SHIFT && r == a.rows - 1) {
      const uint32_t se = (a.d + h) * (SF32 ? 4 : 2), ye = (a.d + h) * (DYF32 ? 4 : 2);
      const uint32_t sw = se & ~15u, yw = ye & ~15u;
      bulk_row<SF32>(p, a.s, r, a.ld_s, h, se, sw, &full[slot]);
      bulk_row<DYF32>(p + s_bytes, a.dy, r, a.ld_dy, h, ye, yw, &full[slot]);
      if (a.ds) bulk_row<SF32>(p + s_bytes + y_bytes, a.ds, r, a.ld_ds, h, se, sw, &full[slot]);
      mbar_arrive_expect_tx(&full[slot], sw + yw + (a.ds ? sw : 0));
      return;
    }
    mbar_arrive_expect_tx(&full[slot], row_bytes);
    bulk_row<SF32>(p, a.s, r, a.ld_s, h, s_bytes, s_bytes, &full[slot]);
    bulk_row<DYF32>(p + s_bytes, a.dy, r, a.ld_dy, h, y_bytes, y_bytes, &full[slot]);
    if (a.ds)
      bulk_row<SF32>(p + s_bytes + y_bytes, a.ds, r, a.ld_ds, h, s_bytes, s_bytes, &full[slot]);
  };
  // SHIFT: which elements of this thread's vectors are the rows' own
  uint32_t own[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    own[i] = 0xffu;
    if (!SHIFT) continue;
    const int e = 8 * (t + i * tpr) - h;  // element 0's column
    if (e < 0) own[i] &= 0xffu << -e;
    if (e + 8 > a.d) own[i] &= e < a.d ? 0xffu >> (e + 8 - a.d) : 0u;
  }
  auto mask = [&](uint32_t m, float (&v)[8]) {
    if (SHIFT && m != 0xffu) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = (m >> j & 1u) ? v[j] : 0.f;
    }
  };
  const long long step = gridDim.x;
  int filled = 0;  // thread 0: rows requested
  if (t == 0) {
    for (long long r = blockIdx.x; filled < depth && r < a.rows; r += step) fill(filled++, r);
  }
  float dw[NV][8], w[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int vi = t + i * tpr;
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = w[i][j] = 0.f;
    if (vi < nvec) {
      if (SHIFT) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int e = 8 * vi - h + j;
          if (own[i] >> j & 1u)
            w[i][j] = a.w_f32 ? static_cast<const float*>(a.w)[e]
                              : __bfloat162float(static_cast<const __nv_bfloat16*>(a.w)[e]);
        }
      } else if (a.w_f32) {
        load8<true, true>(a.w, vi, a.d, w[i]);
      } else {
        load8<false, true>(a.w, vi, a.d, w[i]);
      }
    }
  }
  int it = 0;
  for (long long r = blockIdx.x; r < a.rows; r += step, ++it) {
    const int slot = it % depth;
    const uint8_t* p = s_rows + slot * row_bytes;
    if (!mbar_wait(&full[slot], static_cast<uint32_t>((it / depth) & 1), vabort)) {
      *vabort = 1;
      set_status(a.status, MOK_ERR_DEVICE_TIMEOUT);
    }
    float ss = 0.f, gs = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int vi = t + i * tpr;
      if (vi < nvec) {
        float s[8], dy[8];
        load8<SF32, true>(p, vi, a.d, s);
        load8<DYF32, true>(p + s_bytes, vi, a.d, dy);
        mask(own[i], s);
        mask(own[i], dy);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          ss = fmaf(s[j], s[j], ss);
          gs = fmaf(dy[j] * w[i][j], s[j], gs);
        }
      }
    }
    ss = warp_sum(ss);
    gs = warp_sum(gs);
    const int par = it & 1;
    if ((t & 31) == 0) {
      red[par][0][t >> 5] = ss;
      red[par][1][t >> 5] = gs;
    }
    __syncthreads();  // (the other parity's buffer may still be read)
    if (*vabort) break;  // (set before the barrier: every thread sees it)
    if (t == 0 && it > 0) {  // the row before is done with its slot
      const long long next = r + (depth - 1) * step;
      if (next < a.rows) fill((it - 1) % depth, next);
    }
    const bool in = (t & 31) < nw;
    ss = warp_sum(in ? red[par][0][t & 31] : 0.f);
    gs = warp_sum(in ? red[par][1][t & 31] : 0.f);
    const float rstd = row_rstd(ss, static_cast<float>(a.d), a.eps);
    const float c = gs * rstd * rstd * a.inv_d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int vi = t + i * tpr;
      if (vi >= nvec) continue;
      float s[8], dy[8], o[8];
      load8<SF32, true>(p, vi, a.d, s);
      load8<DYF32, true>(p + s_bytes, vi, a.d, dy);
      if (a.ds) {
        load8<SF32, true>(p + s_bytes + y_bytes, vi, a.d, o);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = 0.f;
      }
      mask(own[i], s);
      mask(own[i], dy);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        o[j] = rstd * (dy[j] * w[i][j] - s[j] * c) + o[j];
        dw[i][j] = fmaf(dy[j], s[j] * rstd, dw[i][j]);
      }
      char* out = static_cast<char*>(row_at<SF32>(a.dx, r, a.ld_dx)) - h * (SF32 ? 4 : 2);
      if (SHIFT && own[i] != 0xffu) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (!(own[i] >> j & 1u)) continue;
          if (SF32) reinterpret_cast<float*>(out)[8 * vi + j] = o[j];
          else reinterpret_cast<__nv_bfloat16*>(out)[8 * vi + j] = __float2bfloat16_rn(o[j]);
        }
      } else {
        store8<SF32, true>(out, vi, a.d, o);
      }
    }
  }
  if (*vabort) {
    spin_ns(1000000ull);  // copies in flight land before the block leaves
    return;
  }
  if (!a.part) return;
  float* out = a.part + static_cast<long long>(blockIdx.x) * a.d;
  if (SHIFT) {  // through the ring's memory, for whole sectors
    float* s_dw = reinterpret_cast<float*>(s_rows);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int vi = t + i * tpr;
      if (vi >= nvec) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (own[i] >> j & 1u) s_dw[8 * vi - h + j] = dw[i][j];
    }
    __syncthreads();
    for (int e = t; e < a.d; e += blockDim.x) out[e] = s_dw[e];
    return;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int vi = t + i * tpr;
    if (vi < nvec) store8<true, true>(out, vi, a.d, dw[i]);
  }
}

// out[c] (+)= sum over g < n of part[g, c]: 16 columns per block (so that more
// SMs take part), 64 threads of each take every 64th partial, their loads in
// flight together, then their sums in a fixed tree.
__global__ void __launch_bounds__(1024) column_sum_kernel(const float* part, long long n, int d,
                                                          float* out, int accumulate) {
  __shared__ float s[64][17];
  grid_dep_launch();
  grid_dep_wait();
  const int c = blockIdx.x * 16 + threadIdx.x;
  float acc = 0.f;
  if (c < d) {
#pragma unroll 10
    for (long long g = threadIdx.y; g < n; g += 64) acc += part[g * d + c];
  }
  s[threadIdx.y][threadIdx.x] = acc;
  __syncthreads();
  const int t = threadIdx.y * 16 + threadIdx.x, col = t >> 5, lane = t & 31;
  if (col >= 16) return;
  const float v = warp_sum(s[lane][col] + s[lane + 32][col]);
  const int o = blockIdx.x * 16 + col;
  if (lane == 0 && o < d) out[o] = accumulate ? out[o] + v : v;
}

cudaError_t launch_column_sum(const float* part, int64_t n, int64_t d, float* out,
                              bool accumulate, cudaStream_t st) {
  ProfScope prof("column_sum", st);
  const cudaError_t e =
      launch_dependent(column_sum_kernel, dim3(static_cast<unsigned>((d + 15) / 16)),
                       dim3(16, 64), 0, st, part, n, d, out, accumulate ? 1 : 0);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

namespace {

// Threads of a row, rows of a block and blocks of the backward, by the
// descriptor alone: the sums do not depend on the device.
struct BwdShape {
  int tpr, nv, rpb, depth;
  int64_t blocks;
};
constexpr int kBulkSmem = 216 * 1024;  // of an SM's shared memory, for all its blocks
// How a row's elements are taken: words at any alignment by register loads,
// aligned vectors, or aligned vectors of rows at a common shift.
enum class Rows { kAny, kVec, kShift };
int64_t bwd_row_bytes(int64_t d, int64_t per_elem, Rows how) {
  return how == Rows::kShift ? (d + 14) / 8 * 8 * per_elem : d * per_elem;
}
BwdShape bwd_shape(int64_t rows, int64_t d, Rows how, int64_t row_bytes) {
  const bool bulk = how == Rows::kShift || (how == Rows::kVec && d >= kBulkMinD);
  const int nvec = static_cast<int>(how == Rows::kVec     ? d / 8
                                    : how == Rows::kShift ? (d + 14) / 8
                                                          : (d + 255) / 256 * 32);
  BwdShape b;
  b.nv = nvec <= 32 ? 1 : (nvec <= 1024 ? 2 : 4);
  b.tpr = ((nvec + b.nv - 1) / b.nv + 31) / 32 * 32;
  b.rpb = b.tpr == 32 ? 8 : 1;
  if (how == Rows::kShift) b.rpb = 1;
  b.depth = 0;
  int per_sm = (b.rpb > 1 ? 1536 : 768) / (b.tpr * b.rpb);
  if (bulk) {
    // a row's chain of barrier and reductions takes a block long enough for an
    // SM's share of the memory to move some 70 KB: enough blocks to cover it
    // (4099 x 2880 bf16: 29.7 us with two, 24.5 with three, 23.8 with four or
    // more), and no more, since each leaves a partial weight gradient
    const int64_t cover = 72 * 1024 / (row_bytes + row_bytes / 3) + 1;
    if (per_sm > cover) per_sm = static_cast<int>(cover < 2 ? 2 : cover);
    // a ring of at least three rows per block where that leaves two blocks
    while (per_sm > 2 && per_sm * 3 * row_bytes > kBulkSmem) --per_sm;
    while (per_sm > 1 && per_sm * 2 * row_bytes > kBulkSmem) --per_sm;
  }
  per_sm = per_sm < 1 ? 1 : (per_sm > 16 ? 16 : per_sm);
  if (bulk) {
    b.depth = static_cast<int>(kBulkSmem / per_sm / row_bytes);
    if (b.depth > kBulkMaxDepth) b.depth = kBulkMaxDepth;
  }
  const int64_t need = (rows + b.rpb - 1) / b.rpb;
  b.blocks = need < kGb300Sms * per_sm ? need : kGb300Sms * per_sm;  // (kShift: a multiple of eight)
  return b;
}

template <bool DYF32, bool SF32, int NV, bool SHIFT>
cudaError_t bulk_launch(const NormBwd& a, const BwdShape& b, int64_t row_bytes, cudaStream_t st) {
  auto kern = add_rmsnorm_bwd_bulk_kernel<DYF32, SF32, NV, SHIFT>;
  const int smem = static_cast<int>(b.depth * row_bytes);
  // (the limit is the kernel's, not the call's: the most that any call takes, so
  // that no host thread lowers it between another's setting and launch)
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kBulkSmem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, dim3(static_cast<unsigned>(b.blocks)), dim3(b.tpr), smem, st, a,
                          b.depth);
}

template <bool DYF32, bool SF32, Rows HOW>
cudaError_t bwd_launch(const NormBwd& a, int64_t row_bytes, cudaStream_t st) {
  const BwdShape b = bwd_shape(a.rows, a.d, HOW, row_bytes);
  ProfScope prof("add_rmsnorm_bwd", st);
  count_launch();
  constexpr bool kShift = HOW == Rows::kShift;
  if constexpr (HOW != Rows::kAny) {
    // (with at least two rows in the ring: the next one's copy is under way)
    if (b.depth >= 2)
      return b.nv == 2 ? bulk_launch<DYF32, SF32, 2, kShift>(a, b, row_bytes, st)
                       : bulk_launch<DYF32, SF32, 4, kShift>(a, b, row_bytes, st);
  }
  if constexpr (kShift) {
    return cudaErrorInvalidValue;  // (not chosen: see shift_rows)
  } else {
    constexpr bool kVec = HOW == Rows::kVec;
    auto kern = b.nv == 1 ? add_rmsnorm_bwd_kernel<DYF32, SF32, kVec, 1>
                          : (b.nv == 2 ? add_rmsnorm_bwd_kernel<DYF32, SF32, kVec, 2>
                                       : add_rmsnorm_bwd_kernel<DYF32, SF32, kVec, 4>);
    return launch_dependent(kern, dim3(static_cast<unsigned>(b.blocks)), dim3(b.tpr, b.rpb), 0, st,
                            a);
  }
}

// Whether rows of this length are taken at a common shift where the tensors'
// alignment allows it: more of them than blocks, so that the ring has a row ahead
// (499 x 1109: 10.2 us so, 8.8 by word loads; 3988 x 660: 16 and 19).
bool shift_rows(int64_t rows, int64_t d, int64_t row_bytes) {
  if (d < kShiftMinD || (d + 14) / 8 > 4 * 512) return false;
  const BwdShape b = bwd_shape(rows, d, Rows::kShift, row_bytes);
  return b.depth >= 2 && rows > b.blocks;
}

}  // namespace

int64_t norm_bwd_blocks(const mok_rmsnorm_desc& D) {
  // the most that any alignment of the pointers leads to
  const int64_t se = D.s_elem == MOK_ELEM_F32 ? 4 : 2, ye = D.x_elem == MOK_ELEM_F32 ? 4 : 2;
  int64_t most = bwd_shape(D.rows, D.d, Rows::kAny, 0).blocks;
  for (int skip = 0; skip < 2; ++skip) {
    const int64_t per_elem = se * (1 + skip) + ye;
    int64_t b = 0, n = bwd_row_bytes(D.d, per_elem, Rows::kShift);
    if (shift_rows(D.rows, D.d, n)) b = bwd_shape(D.rows, D.d, Rows::kShift, n).blocks;
    if (b > most) most = b;
    if (D.d % 8 != 0) continue;
    b = bwd_shape(D.rows, D.d, Rows::kVec, D.d * per_elem).blocks;
    if (b > most) most = b;
  }
  return most;
}

cudaError_t launch_add_rmsnorm_bwd(const mok_rmsnorm_desc& D, const void* dy, const void* s,
                                   const void* w, const void* ds, void* dx, float* dweight,
                                   float* part, int* status, cudaStream_t st) {
  const bool yf = D.x_elem == MOK_ELEM_F32, sf = D.s_elem == MOK_ELEM_F32;
  cudaError_t e = cudaSuccess;
  int64_t grid = 0;
  if (D.rows > 0) {
    NormBwd a;
    a.status = status;
    a.dy = dy; a.s = s; a.w = w; a.ds = ds; a.dx = dx;
    a.part = dweight ? part : nullptr;
    a.rows = D.rows;
    a.ld_dy = D.ld_x; a.ld_s = D.ld_s; a.ld_ds = D.ld_res; a.ld_dx = D.ld_y;
    a.d = static_cast<int>(D.d);
    a.nvec = (a.d + 7) / 8;
    a.w_f32 = D.weight_elem == MOK_ELEM_F32;
    a.inv_d = 1.0f / static_cast<float>(a.d);
    a.eps = D.eps;
    const int ye = yf ? 4 : 2, se = sf ? 4 : 2;
    const bool vec = a.d % 8 == 0 && vec_rows(dy, a.ld_dy, ye) && vec_rows(s, a.ld_s, se) &&
                     vec_rows(ds, a.ld_ds, se) && vec_rows(dx, a.ld_dx, se) && vec_rows(w, 0, 4);
    // every tensor's rows begin alike: aligned bases, lengths that agree mod 8
    // (fp32 alone: mod 4)
    const int64_t step = !yf ? a.ld_dy : a.ld_s;
    auto alike = [&](const void* p, int64_t ld, bool f) {
      return !p || ((reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld - step) % (f ? 4 : 8) == 0);
    };
    const int64_t per_elem = se * (ds ? 2 : 1) + ye;
    Rows how = vec ? Rows::kVec : Rows::kAny;
    if (!vec && alike(dy, a.ld_dy, yf) && alike(s, a.ld_s, sf) && alike(ds, a.ld_ds, sf) &&
        alike(dx, a.ld_dx, sf) &&
        shift_rows(D.rows, D.d, bwd_row_bytes(D.d, per_elem, Rows::kShift)))
      how = Rows::kShift;
    if (how == Rows::kAny) a.nvec = (a.d + 255) / 256 * 32;
    a.ld8 = static_cast<int>(step & 7);
    const int64_t row_bytes = bwd_row_bytes(D.d, per_elem, how);
    grid = bwd_shape(D.rows, D.d, how, row_bytes).blocks;
    auto run = [&](auto Y, auto S) {
      constexpr bool y = decltype(Y)::value, f = decltype(S)::value;
      if (how == Rows::kVec) return bwd_launch<y, f, Rows::kVec>(a, row_bytes, st);
      if (how == Rows::kShift) return bwd_launch<y, f, Rows::kShift>(a, row_bytes, st);
      return bwd_launch<y, f, Rows::kAny>(a, row_bytes, st);
    };
    if (yf) e = sf ? run(std::true_type(), std::true_type()) : run(std::true_type(), std::false_type());
    else e = sf ? run(std::false_type(), std::true_type()) : run(std::false_type(), std::false_type());
  }
  if (e != cudaSuccess || !dweight) return e;
  return launch_column_sum(part, grid, D.d, dweight, D.accumulate != 0, st);
}

}  // namespace mok
