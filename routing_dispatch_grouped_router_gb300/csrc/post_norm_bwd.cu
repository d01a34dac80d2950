// Backward of the norms after and before a block (post_norm.cu has the formulas).
#include "post_norm.cuh"

namespace mok {

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

// One reduction a row, in all of these kernels: with u = w1 (a channel's gate in it) x,
//   sum of t w1 x = rstd(s) sum of dy w2 u  -  rstd(s) c sum of s u  +  sum of ds u,
// c = rstd(s)^2 sum of dy w2 s / d, so that all six sums come from one pass.

// blockDim.x threads of whole warps hold a row, blockDim.y rows are in a block at a
// time (more than one only for rows of one warp).  Row group b takes rows b, b +
// groups, ..; its threads keep the weight gradients of their columns in registers
// over those rows and read the row's elements a second time, from L1 or L2, after its
// sums.
template <bool DYF32, bool XF32, bool SF32, bool VEC, int NV>
__global__ void __launch_bounds__(512) post_pre_bwd_kernel(PostPreBwd a) {
  __shared__ float red[2][8][16];  // [row parity][sum][warp]
  __shared__ float s_dw[NV == 1 ? 8 : 1][256];
  grid_dep_launch();
  grid_dep_wait();
  const int t = threadIdx.x, tpr = blockDim.x, nw = tpr >> 5, lane = t & 31;
  const float df = static_cast<float>(a.d);
  float dw1[NV][8], dw2[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw1[i][j] = dw2[i][j] = 0.f;
  const long long step = static_cast<long long>(gridDim.x) * blockDim.y;
  long long r = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
  for (int par = 0; r < a.rows; r += step, par ^= 1) {
    const void *sr = row_at<SF32>(a.s, r, a.ld_s), *yr = row_at<DYF32>(a.dy, r, a.ld_dy),
               *xr = row_at<XF32>(a.x, r, a.ld_x), *dr = row_at<SF32>(a.ds, r, a.ld_ds);
    const float gt =
        a.gate_kind == MOK_GATE_TOKEN ? elem_at(a.gate, r, a.gate_f32) : 1.0f;
    float q[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int vi = t + i * tpr;
      if (vi >= a.nvec) continue;
      Raw8<SF32, VEC> rs, rd;
      Raw8<DYF32, VEC> ry;
      Raw8<XF32, VEC> rx;
      rs.load(sr, vi, a.d);
      ry.load(yr, vi, a.d);
      rx.load(xr, vi, a.d);
      rd.zero();
      if (a.ds) rd.load(dr, vi, a.d);
      float w1[8], w2[8], s[8], dy[8], x[8], ds[8];
      gated_weight<VEC>(a, vi, w1);
      load_weight<VEC>(a.w2, a.w_f32, vi, a.d, w2);
      rs.get(s);
      ry.get(dy);
      rx.get(x);
      rd.get(ds);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float g = dy[j] * w2[j], u = x[j] * w1[j];
        q[0] = fmaf(s[j], s[j], q[0]);
        q[1] = fmaf(x[j], x[j], q[1]);
        q[2] = fmaf(g, s[j], q[2]);
        q[3] = fmaf(g, u, q[3]);
        q[4] = fmaf(s[j], u, q[4]);
        q[5] = fmaf(ds[j], u, q[5]);
      }
    }
    const float w = warp_sums(q, lane);
    float sum[8];
    if (nw == 1) {
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] = __shfl_sync(0xffffffffu, w, 4 * i);
    } else {
      if ((lane & 3) == 0) red[par][lane >> 2][t >> 5] = w;
      __syncthreads();  // (the other parity's buffer may still be read)
      block_sums<8>(red[par], nw, lane, sum);
    }
    const float rstd2 = row_rstd(sum[0], df, a.eps), rstd1 = row_rstd(sum[1], df, a.eps);
    const float c = sum[2] * rstd2 * rstd2 * a.inv_d * rstd2;
    const float dot = (sum[3] * rstd2 - sum[4] * c + sum[5]) * rstd1;
    if (a.dgate && t == 0) a.dgate[r] = a.accumulate ? a.dgate[r] + dot : dot;
    const float k = gt * dot * rstd1 * rstd1 * a.inv_d, nr = rstd1 * gt;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int vi = t + i * tpr;
      if (vi >= a.nvec) continue;
      Raw8<SF32, VEC> rs, rd;
      Raw8<DYF32, VEC> ry;
      Raw8<XF32, VEC> rx;
      rs.load(sr, vi, a.d);
      ry.load(yr, vi, a.d);
      rx.load(xr, vi, a.d);
      rd.zero();
      if (a.ds) rd.load(dr, vi, a.d);
      float w1[8], w2[8], s[8], dy[8], x[8], tt[8];
      gated_weight<VEC>(a, vi, w1);
      load_weight<VEC>(a.w2, a.w_f32, vi, a.d, w2);
      rs.get(s);
      ry.get(dy);
      rx.get(x);
      rd.get(tt);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        tt[j] = fmaf(dy[j] * w2[j], rstd2, fmaf(-s[j], c, tt[j]));
        dw2[i][j] = fmaf(dy[j], s[j] * rstd2, dw2[i][j]);
        dw1[i][j] = fmaf(tt[j], x[j] * nr, dw1[i][j]);
        x[j] = fmaf(tt[j] * w1[j], nr, -x[j] * k);
        tt[j] *= a.alpha;
      }
      store8<SF32, VEC>(row_at<SF32>(a.dr, r, a.ld_dr), vi, a.d, tt);
      if (a.dx_f32) store8<true, VEC>(row_at<true>(a.dx, r, a.ld_dx), vi, a.d, x);
      else store8<false, VEC>(row_at<false>(a.dx, r, a.ld_dx), vi, a.d, x);
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

// Bytes of an element's inputs.
int64_t bwd_elem_bytes(const mok_post_pre_desc& D, bool ds) {
  return esize(D.y_elem == MOK_ELEM_F32) + esize(D.x_elem == MOK_ELEM_F32) +
         esize(D.s_elem == MOK_ELEM_F32) * (ds ? 2 : 1);
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
  // the most that any alignment of the pointers, and any ds, leads to
  int64_t most = bwd_shape(D.rows, D.d, false).blocks;
  auto at_least = [&](int64_t b) {
    if (b > most) most = b;
  };
  if (D.d % 8 == 0) at_least(bwd_shape(D.rows, D.d, true).blocks);
  for (int skip = 0; skip < 2; ++skip)
    for (int shift = 0; shift < 2; ++shift)
      if (shift || D.d % 8 == 0)
        at_least(ring_shape(D.rows, D.d, shift != 0, bwd_elem_bytes(D, skip != 0),
                            shift ? kBwdShiftThreads : kBwdRingThreads)
                     .blocks);
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
    const int64_t step = a.ld_s;
    const bool shift = !vec && alike(dy, a.ld_dy, yf, step) && alike(x, a.ld_x, xf, step) &&
                       alike(s, a.ld_s, sf, step) && alike(ds, a.ld_ds, sf, step) &&
                       alike(dr, a.ld_dr, sf, step) && alike(dx, a.ld_dx, a.dx_f32, step);
    RingShape b = {};
    if (vec || shift)
      b = ring_shape(D.rows, D.d, shift, bwd_elem_bytes(D, ds != nullptr),
                     shift ? kBwdShiftThreads : kBwdRingThreads);
    if (!vec) a.nvec = (a.d + 255) / 256 * 32;
    grid = b.blocks > 0 ? b.blocks : bwd_shape(D.rows, D.d, vec).blocks;
    if (b.blocks > 0) {
      Ring<4> g = {{s, dy, x, ds}, {a.ld_s, a.ld_dy, a.ld_x, a.ld_ds}, {sf, yf, xf, sf},
                   {0, 0, 0, 0}, 0, 0, static_cast<int>(step & 7)};
      ProfScope prof("post_pre_rmsnorm_bwd", st);
      count_launch();
      e = launch_post_pre_bwd_ring(a, g, b, yf, xf, sf, shift, st);
    } else {
      e = with_types(
          [&](auto Y, auto X, auto S, auto V) {
            return bwd_launch<decltype(Y)::value, decltype(X)::value, decltype(S)::value,
                              decltype(V)::value>(a, st);
          },
          yf, xf, sf, vec);
    }
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
