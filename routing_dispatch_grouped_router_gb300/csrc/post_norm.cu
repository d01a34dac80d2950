// The norms after and before a block with its gate and the residual's scale:
//
//   n = x rstd(x),  s = alpha r + gate w1 n (rounded once to the stream's type),
//   y = w2 s rstd(s),        rstd(v) = 1 / sqrt(mean(v^2) + eps)
//   backward, from dy and ds:
//     m = s rstd(s), g = dy w2:      t = rstd(s) (g - m mean(g m)) + ds
//     dr = alpha t,  q = t gate w1:  dx = rstd(x) (q - n mean(q n))
//     dw2 = sum over rows of dy m,  dw1 = of t gate n,  dgate = of t w1 n (along
//     the rows for a gate per channel, along the columns for one per token)
//
// Bound by HBM bytes: a row is read once, kept in registers across both norms'
// reductions and written once.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "mok_internal.h"
#include "ptx.cuh"
#include "rows.cuh"

namespace mok {

namespace {

__device__ __forceinline__ float elem_at(const void* p, long long i, int f32) {
  return f32 ? static_cast<const float*>(p)[i]
             : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

template <bool VEC>
__device__ __forceinline__ void load_weight(const void* w, int f32, int v, int d, float (&o)[8]) {
  if (f32) load8<true, VEC>(w, v, d, o);
  else load8<false, VEC>(w, v, d, o);
}

// The sum over a row of `nw` warps of the values whose warp sums are in red.
template <int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*red)[32], int t, int nw) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
  if (nw == 1) return;
  if ((t & 31) == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) red[i][t >> 5] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum((t & 31) < nw ? red[i][t & 31] : 0.f);
}

}  // namespace

struct PostPreFwd {
  const void *x, *r, *w1, *w2, *gate;
  void *s, *y;
  long long rows, ld_x, ld_r, ld_s, ld_y;
  int d, nvec, w_f32, gate_f32, gate_kind;
  float alpha, eps;
};

// One row per threadIdx.y; blockDim.x threads of whole warps hold it, NV vectors
// each.
template <bool XF32, bool SF32, bool VEC, int NV>
__global__ void __launch_bounds__(NV == 1 ? 1024 : 512) post_pre_kernel(PostPreFwd a) {
  __shared__ float red[2][32];
  grid_dep_launch();
  grid_dep_wait();
  const int t = threadIdx.x, tpr = blockDim.x, nw = tpr >> 5;
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
      res[i].load(row_at<SF32>(a.r, r, a.ld_r), vi, a.d);
    }
  }
  const float df = static_cast<float>(a.d);
  float v[NV][8];
  float sum[1] = {0.f};
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    x[i].get(v[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[0] = fmaf(v[i][j], v[i][j], sum[0]);
  }
  row_sums(sum, &red[0], t, nw);
  float scale = row_rstd(sum[0], df, a.eps);
  if (a.gate_kind == MOK_GATE_TOKEN && row_in) scale *= elem_at(a.gate, r, a.gate_f32);
  sum[0] = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int vi = t + i * tpr;
    const bool in = row_in && vi < a.nvec;
    float w[8], b[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = 0.f;
    if (in) {
      load_weight<VEC>(a.w1, a.w_f32, vi, a.d, w);
      if (a.gate_kind == MOK_GATE_CHANNEL) {
        float g[8];
        load_weight<VEC>(a.gate, a.gate_f32, vi, a.d, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] *= g[j];
      }
    }
    res[i].get(b);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[i][j] = fmaf(a.alpha, b[j], v[i][j] * scale * w[j]);
      if (!SF32) v[i][j] = bf16_round(v[i][j]);
    }
    if (!in) {  // (past the row's end: not 0 for an infinite scale)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
      continue;
    }
    store8<SF32, VEC>(row_at<SF32>(a.s, r, a.ld_s), vi, a.d, v[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (!VEC && elem_of<VEC>(vi, j) >= a.d) v[i][j] = 0.f;
      sum[0] = fmaf(v[i][j], v[i][j], sum[0]);
    }
  }
  row_sums(sum, &red[1], t, nw);
  const float rstd = row_rstd(sum[0], df, a.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int vi = t + i * tpr;
    if (!row_in || vi >= a.nvec) continue;
    float w[8];
    load_weight<VEC>(a.w2, a.w_f32, vi, a.d, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] *= v[i][j] * rstd;
    store8<false, VEC>(row_at<false>(a.y, r, a.ld_y), vi, a.d, w);
  }
}

namespace {

template <bool XF32, bool SF32, bool VEC>
cudaError_t fwd_launch(const PostPreFwd& a, cudaStream_t st) {
  int tpr, nv;
  norm_shape(a.rows, a.nvec, 4, &tpr, &nv);
  const int rpb = tpr == 32 ? 4 : 1;
  const unsigned grid = static_cast<unsigned>((a.rows + rpb - 1) / rpb);
  ProfScope prof("post_pre_rmsnorm", st);
  auto kern = nv == 1 ? post_pre_kernel<XF32, SF32, VEC, 1>
                      : (nv == 2 ? post_pre_kernel<XF32, SF32, VEC, 2>
                                 : post_pre_kernel<XF32, SF32, VEC, 4>);
  const cudaError_t e = launch_dependent(kern, dim3(grid), dim3(tpr, rpb), 0, st, a);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

int esize(bool f32) { return f32 ? 4 : 2; }

}  // namespace

cudaError_t launch_post_pre(const mok_post_pre_desc& D, const void* x, const void* res,
                            const void* w1, const void* w2, const void* gate, void* s, void* y,
                            cudaStream_t st) {
  if (D.rows == 0) return cudaSuccess;
  const bool xf = D.x_elem == MOK_ELEM_F32, sf = D.s_elem == MOK_ELEM_F32;
  PostPreFwd a;
  a.x = x; a.r = res; a.w1 = w1; a.w2 = w2; a.gate = gate; a.s = s; a.y = y;
  a.rows = D.rows;
  a.ld_x = D.ld_x; a.ld_r = D.ld_res; a.ld_s = D.ld_s; a.ld_y = D.ld_y;
  a.d = static_cast<int>(D.d);
  a.nvec = (a.d + 7) / 8;
  a.w_f32 = D.weight_elem == MOK_ELEM_F32;
  a.gate_f32 = D.gate_elem == MOK_ELEM_F32;
  a.gate_kind = D.gate;
  a.alpha = D.residual_scale;
  a.eps = D.eps;
  const bool vec = a.d % 8 == 0 && vec_rows(x, a.ld_x, esize(xf)) &&
                   vec_rows(res, a.ld_r, esize(sf)) && vec_rows(s, a.ld_s, esize(sf)) &&
                   vec_rows(y, a.ld_y, 2) && vec_rows(w1, 0, 4) && vec_rows(w2, 0, 4) &&
                   (D.gate != MOK_GATE_CHANNEL || vec_rows(gate, 0, 4));
  if (!vec) a.nvec = (a.d + 255) / 256 * 32;  // whole groups of 256 elements
  auto run = [&](auto X, auto S) {
    constexpr bool f = decltype(X)::value, g = decltype(S)::value;
    return vec ? fwd_launch<f, g, true>(a, st) : fwd_launch<f, g, false>(a, st);
  };
  if (xf) return sf ? run(std::true_type(), std::true_type()) : run(std::true_type(), std::false_type());
  return sf ? run(std::false_type(), std::true_type()) : run(std::false_type(), std::false_type());
}

// ----------------------------------------------------------------- backward --

struct PostPreBwd {
  int* status;
  const void *dy, *x, *s, *ds, *w1, *w2, *gate;
  void *dx, *dr;
  float* dgate;  // per token: [rows] (NULL: not computed)
  float* part;   // [2][gridDim.x, d]: partial sums of t gate n (without a channel's
                 // gate), then of dy m (NULL: neither)
  long long rows, ld_dy, ld_x, ld_s, ld_ds, ld_dx, ld_dr;
  int d, nvec, w_f32, gate_f32, gate_kind, dx_f32, accumulate;
  float alpha, inv_d, eps;
};

// w1 of a thread's vector, with a channel's gate in it.
template <bool VEC>
__device__ __forceinline__ void gated_weight(const PostPreBwd& a, int v, float (&w)[8]) {
  load_weight<VEC>(a.w1, a.w_f32, v, a.d, w);
  if (a.gate_kind == MOK_GATE_CHANNEL) {
    float g[8];
    load_weight<VEC>(a.gate, a.gate_f32, v, a.d, g);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] *= g[j];
  }
}

// blockDim.x threads of whole warps hold a row, blockDim.y rows are in a block at a
// time (more than one only for rows of one warp).  Row group b takes rows b, b +
// groups, ..; its threads keep the weight gradients of their columns in registers
// over those rows.
template <bool DYF32, bool XF32, bool SF32, bool VEC, int NV>
__global__ void __launch_bounds__(512) post_pre_bwd_kernel(PostPreBwd a) {
  __shared__ float red[2][4][32];  // [row parity][sum][warp]
  __shared__ float s_dw[NV == 1 ? 8 : 1][256];
  grid_dep_launch();
  grid_dep_wait();
  const int t = threadIdx.x, tpr = blockDim.x, nw = tpr >> 5;
  const float df = static_cast<float>(a.d);
  float dw1[NV][8], dw2[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw1[i][j] = dw2[i][j] = 0.f;
  const long long step = static_cast<long long>(gridDim.x) * blockDim.y;
  long long r = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
  for (int par = 0; r < a.rows; r += step, par ^= 1) {
    Raw8<XF32, VEC> rx[NV];
    Raw8<SF32, VEC> rs[NV], rd[NV];
    Raw8<DYF32, VEC> ry[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int vi = t + i * tpr;
      rx[i].zero();
      rs[i].zero();
      rd[i].zero();
      ry[i].zero();
      if (vi < a.nvec) {
        rs[i].load(row_at<SF32>(a.s, r, a.ld_s), vi, a.d);
        ry[i].load(row_at<DYF32>(a.dy, r, a.ld_dy), vi, a.d);
        rx[i].load(row_at<XF32>(a.x, r, a.ld_x), vi, a.d);
        if (a.ds) rd[i].load(row_at<SF32>(a.ds, r, a.ld_ds), vi, a.d);
      }
    }
    const float gt =
        a.gate_kind == MOK_GATE_TOKEN ? elem_at(a.gate, r, a.gate_f32) : 1.0f;
    float sum[3] = {0.f, 0.f, 0.f};  // of s^2, dy w2 s, x^2
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int vi = t + i * tpr;
      if (vi >= a.nvec) continue;
      float w[8], s[8], dy[8], x[8];
      load_weight<VEC>(a.w2, a.w_f32, vi, a.d, w);
      rs[i].get(s);
      ry[i].get(dy);
      rx[i].get(x);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        sum[0] = fmaf(s[j], s[j], sum[0]);
        sum[1] = fmaf(dy[j] * w[j], s[j], sum[1]);
        sum[2] = fmaf(x[j], x[j], sum[2]);
      }
    }
    row_sums(sum, &red[par][0], t, nw);
    const float rstd2 = row_rstd(sum[0], df, a.eps), rstd1 = row_rstd(sum[2], df, a.eps);
    const float c = sum[1] * rstd2 * rstd2 * a.inv_d;
    float tt[NV][8];
    float dot[1] = {0.f};  // of t w1 n
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int vi = t + i * tpr;
      if (vi >= a.nvec) continue;
      float w[8], w1[8], s[8], dy[8], x[8], o[8];
      load_weight<VEC>(a.w2, a.w_f32, vi, a.d, w);
      gated_weight<VEC>(a, vi, w1);
      rs[i].get(s);
      ry[i].get(dy);
      rx[i].get(x);
      rd[i].get(tt[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        tt[i][j] = rstd2 * (dy[j] * w[j] - s[j] * c) + tt[i][j];
        if (!VEC && elem_of<VEC>(vi, j) >= a.d) tt[i][j] = 0.f;
        dw2[i][j] = fmaf(dy[j], s[j] * rstd2, dw2[i][j]);
        dw1[i][j] = fmaf(tt[i][j] * gt, x[j] * rstd1, dw1[i][j]);
        dot[0] = fmaf(tt[i][j] * w1[j], x[j] * rstd1, dot[0]);
        o[j] = a.alpha * tt[i][j];
      }
      store8<SF32, VEC>(row_at<SF32>(a.dr, r, a.ld_dr), vi, a.d, o);
    }
    row_sums(dot, &red[par][3], t, nw);
    if (a.dgate && t == 0) a.dgate[r] = a.accumulate ? a.dgate[r] + dot[0] : dot[0];
    const float k = gt * dot[0] * rstd1 * rstd1 * a.inv_d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int vi = t + i * tpr;
      if (vi >= a.nvec) continue;
      float w1[8], x[8], o[8];
      gated_weight<VEC>(a, vi, w1);
      rx[i].get(x);
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = rstd1 * (tt[i][j] * gt * w1[j]) - x[j] * k;
      if (a.dx_f32) store8<true, VEC>(row_at<true>(a.dx, r, a.ld_dx), vi, a.d, o);
      else store8<false, VEC>(row_at<false>(a.dx, r, a.ld_dx), vi, a.d, o);
    }
  }
  if (!a.part) return;
  float* p = a.part + static_cast<long long>(blockIdx.x) * a.d;
  const long long second = static_cast<long long>(gridDim.x) * a.d;
  if (NV == 1 && blockDim.y > 1) {  // rows of one warp: the block's rows in order
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) s_dw[threadIdx.y][t * 8 + j] = h ? dw2[0][j] : dw1[0][j];
      __syncthreads();
      const int i = threadIdx.y * 32 + t;  // element i & 7 of vector i / 8
      float v = 0.f;
#pragma unroll
      for (int y = 0; y < 8; ++y) v += s_dw[y][i];
      const int e = elem_of<VEC>(i >> 3, i & 7);
      if ((i >> 3) < a.nvec && e < a.d) p[h * second + e] = v;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int vi = t + i * tpr;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = elem_of<VEC>(vi, j);
      if (vi < a.nvec && e < a.d) {
        p[e] = dw1[i][j];
        p[second + e] = dw2[i][j];
      }
    }
  }
}

// The partial sums over the blocks in a fixed tree, 16 columns per block (as
// column_sum_kernel): dw1 (blockIdx.y = 0) with a channel's gate and its gradient,
// dw2 (1).
__global__ void __launch_bounds__(1024)
    post_pre_sums_kernel(PostPreBwd a, long long n, float* dw1, float* dw2, float* dgate) {
  __shared__ float s[64][17];
  grid_dep_launch();
  grid_dep_wait();
  const int c = blockIdx.x * 16 + threadIdx.x;
  const float* part = a.part + static_cast<long long>(blockIdx.y) * n * a.d;
  float acc = 0.f;
  if (c < a.d) {
#pragma unroll 10
    for (long long g = threadIdx.y; g < n; g += 64) acc += part[g * a.d + c];
  }
  s[threadIdx.y][threadIdx.x] = acc;
  __syncthreads();
  const int t = threadIdx.y * 16 + threadIdx.x, col = t >> 5, lane = t & 31;
  if (col >= 16) return;
  const float v = warp_sum(s[lane][col] + s[lane + 32][col]);
  const int o = blockIdx.x * 16 + col;
  if (lane != 0 || o >= a.d) return;
  auto put = [&](float* p, float x) {
    if (p) p[o] = a.accumulate ? p[o] + x : x;
  };
  if (blockIdx.y) {
    put(dw2, v);
  } else if (a.gate_kind == MOK_GATE_CHANNEL) {
    put(dw1, v * elem_at(a.gate, o, a.gate_f32));
    put(dgate, v * elem_at(a.w1, o, a.w_f32));
  } else {
    put(dw1, v);
  }
}

namespace {

// Threads of a row, rows of a block and blocks of the backward, by the descriptor
// alone: the sums do not depend on the device.
struct BwdShape {
  int tpr, nv, rpb;
  int64_t blocks;
};
BwdShape bwd_shape(int64_t rows, int64_t d, bool vec) {
  const int nvec = static_cast<int>(vec ? d / 8 : (d + 255) / 256 * 32);
  BwdShape b;
  b.nv = nvec <= 32 ? 1 : (nvec <= 1024 ? 2 : 4);
  b.tpr = ((nvec + b.nv - 1) / b.nv + 31) / 32 * 32;
  b.rpb = b.tpr == 32 && b.nv == 1 ? 8 : 1;
  int per_sm = 512 / (b.tpr * b.rpb);
  per_sm = per_sm < 1 ? 1 : (per_sm > 16 ? 16 : per_sm);
  const int64_t need = (rows + b.rpb - 1) / b.rpb;
  b.blocks = need < kGb300Sms * per_sm ? need : kGb300Sms * per_sm;
  return b;
}

template <bool DYF32, bool XF32, bool SF32, bool VEC>
cudaError_t bwd_launch(const PostPreBwd& a, cudaStream_t st) {
  const BwdShape b = bwd_shape(a.rows, a.d, VEC);
  ProfScope prof("post_pre_rmsnorm_bwd", st);
  count_launch();
  auto kern = b.nv == 1 ? post_pre_bwd_kernel<DYF32, XF32, SF32, VEC, 1>
                        : (b.nv == 2 ? post_pre_bwd_kernel<DYF32, XF32, SF32, VEC, 2>
                                     : post_pre_bwd_kernel<DYF32, XF32, SF32, VEC, 4>);
  return launch_dependent(kern, dim3(static_cast<unsigned>(b.blocks)), dim3(b.tpr, b.rpb), 0, st,
                          a);
}

}  // namespace

int64_t post_pre_bwd_blocks(const mok_post_pre_desc& D) {
  // the most that any alignment of the pointers leads to
  int64_t most = bwd_shape(D.rows, D.d, false).blocks;
  if (D.d % 8 == 0) {
    const int64_t b = bwd_shape(D.rows, D.d, true).blocks;
    if (b > most) most = b;
  }
  return most;
}

cudaError_t launch_post_pre_bwd(const mok_post_pre_desc& D, const void* dy, const void* x,
                                const void* s, const void* w1, const void* w2, const void* gate,
                                const void* ds, void* dx, void* dr, float* dw1, float* dw2,
                                float* dgate, float* part, int* status, cudaStream_t st) {
  const bool yf = D.y_elem == MOK_ELEM_F32, xf = D.x_elem == MOK_ELEM_F32,
             sf = D.s_elem == MOK_ELEM_F32;
  PostPreBwd a;
  a.status = status;
  a.dy = dy; a.x = x; a.s = s; a.ds = ds; a.w1 = w1; a.w2 = w2; a.gate = gate;
  a.dx = dx; a.dr = dr;
  a.dgate = D.gate == MOK_GATE_TOKEN ? dgate : nullptr;
  const bool sums = dw1 || dw2 || (dgate && D.gate == MOK_GATE_CHANNEL);
  a.part = sums ? part : nullptr;
  a.rows = D.rows;
  a.ld_dy = D.ld_y; a.ld_x = D.ld_x; a.ld_s = D.ld_s; a.ld_ds = D.ld_res; a.ld_dx = D.ld_dx;
  a.ld_dr = D.ld_dr;
  a.d = static_cast<int>(D.d);
  a.nvec = (a.d + 7) / 8;
  a.w_f32 = D.weight_elem == MOK_ELEM_F32;
  a.gate_f32 = D.gate_elem == MOK_ELEM_F32;
  a.gate_kind = D.gate;
  a.dx_f32 = D.dx_elem == MOK_ELEM_F32;
  a.accumulate = D.accumulate;
  a.alpha = D.residual_scale;
  a.inv_d = 1.0f / static_cast<float>(a.d);
  a.eps = D.eps;
  cudaError_t e = cudaSuccess;
  int64_t grid = 0;
  if (D.rows > 0) {
    const bool vec = a.d % 8 == 0 && vec_rows(dy, a.ld_dy, esize(yf)) &&
                     vec_rows(x, a.ld_x, esize(xf)) && vec_rows(s, a.ld_s, esize(sf)) &&
                     vec_rows(ds, a.ld_ds, esize(sf)) && vec_rows(dr, a.ld_dr, esize(sf)) &&
                     vec_rows(dx, a.ld_dx, esize(a.dx_f32)) && vec_rows(w1, 0, 4) &&
                     vec_rows(w2, 0, 4) && (D.gate != MOK_GATE_CHANNEL || vec_rows(gate, 0, 4));
    if (!vec) a.nvec = (a.d + 255) / 256 * 32;
    grid = bwd_shape(D.rows, D.d, vec).blocks;
    auto run = [&](auto Y, auto X, auto S) {
      constexpr bool y = decltype(Y)::value, f = decltype(X)::value, g = decltype(S)::value;
      return vec ? bwd_launch<y, f, g, true>(a, st) : bwd_launch<y, f, g, false>(a, st);
    };
    auto run2 = [&](auto Y, auto X) {
      return sf ? run(Y, X, std::true_type()) : run(Y, X, std::false_type());
    };
    auto run3 = [&](auto Y) { return xf ? run2(Y, std::true_type()) : run2(Y, std::false_type()); };
    e = yf ? run3(std::true_type()) : run3(std::false_type());
  }
  if (e != cudaSuccess || !sums) return e;
  ProfScope prof("post_pre_rmsnorm_sums", st);
  e = launch_dependent(post_pre_sums_kernel, dim3(static_cast<unsigned>((a.d + 15) / 16), 2),
                       dim3(16, 64), 0, st, a, grid, dw1, dw2,
                       D.gate == MOK_GATE_CHANNEL ? dgate : nullptr);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace mok
