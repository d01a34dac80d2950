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
// Bound by HBM bytes: a row is read once, kept on the chip across both norms'
// reductions and written once.  Forward, 8192 x 7168, fp32 into a bf16 stream: 100 us
// (5.9 TB/s, floor 88); backward, 16384 x 4096, fp32 x and stream: 240 us (6.1 TB/s,
// floor 221).  Short bf16 rows in the backward wait on latency instead: 4099 x 2880 44
// us (3.2 TB/s, floor 21), with three warps a scheduler, of which one issues in 47% of
// the cycles (its instructions alone are 16 us), and the sums' kernel after it (10 us
// by itself, in part under the first one's end).
#include "post_norm.cuh"

namespace mok {

struct PostPreFwd {
  int* status;
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

// The same through a ring of rows (x, residual), two vectors per thread.
template <bool XF32, bool SF32, bool SHIFT>
__global__ void __launch_bounds__(kRingThreads) post_pre_ring_kernel(PostPreFwd a, Ring<2> g) {
  extern __shared__ __align__(128) uint8_t s_rows[];
  __shared__ __align__(8) uint64_t full[kRingMaxDepth];
  __shared__ float red[2][2][16];  // [row parity][sum][warp]
  __shared__ int s_abort;
  grid_dep_launch();
  const int t = threadIdx.x, tpr = blockDim.x, nw = tpr >> 5, lane = t & 31;
  const int h = SHIFT ? (blockIdx.x * g.ld8) & 7 : 0;
  uint32_t own[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) own[i] = ring_own(t + i * tpr, h, a.d);
  if (t == 0) {
    for (uint32_t i = 0; i < g.depth; ++i) mbar_init(&full[i], 1);
    s_abort = 0;
    fence_barrier_init();
  }
  __syncthreads();
  grid_dep_wait();
  volatile int* vabort = &s_abort;
  const long long step = gridDim.x;
  auto fill = [&](uint32_t slot, long long r) {
    ring_fill<2, SHIFT>(g, s_rows + slot * g.row_bytes, &full[slot], r, a.rows, a.d, h);
  };
  if (t == 0)
    for (uint32_t i = 0; i < g.depth && blockIdx.x + i * step < a.rows; ++i)
      fill(i, blockIdx.x + i * step);
  F2 w1[2][4], w2[2][4];
  // (by elements: vectors, 16 loads instead of 48 a thread, made 8192 x 7168 111 us)
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    ring_weight<false>(a.w1, a.w_f32, t + i * tpr, h, own[i], w1[i]);
    ring_weight<false>(a.w2, a.w_f32, t + i * tpr, h, own[i], w2[i]);
    if (a.gate_kind == MOK_GATE_CHANNEL) {
      F2 z[4];
      ring_weight<false>(a.gate, a.gate_f32, t + i * tpr, h, own[i], z);
#pragma unroll
      for (int j = 0; j < 4; ++j) w1[i][j] = mul2(w1[i][j], z[j]);
    }
  }
  const float df = static_cast<float>(a.d);
  const F2 alpha = f2(a.alpha);
  uint32_t slot = 0, phase = 0;
  // the sum of row r's x^2, from the slot that comes next
  auto square = [&](uint32_t sl, uint32_t ph) {
    if (!mbar_wait(&full[sl], ph, vabort)) {
      *vabort = 1;
      set_status(a.status, MOK_ERR_DEVICE_TIMEOUT);
    }
    F2 sq[2] = {0ull, 0ull};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (!own[i]) continue;
      F2 x[4];
      ring_get<XF32, SHIFT>(g, s_rows + sl * g.row_bytes, 0, t + i * tpr, own[i], x);
#pragma unroll
      for (int j = 0; j < 4; ++j) sq[i] = fma2(x[j], x[j], sq[i]);
    }
    return (lo_of(sq[0]) + hi_of(sq[0])) + (lo_of(sq[1]) + hi_of(sq[1]));
  };
  // both sums of the block: of s^2 of this row, of x^2 of the next
  auto sums = [&](float s, float x, int par, float (&out)[2]) {
    float v[2] = {s, x};
    const float w = warp_sums(v, lane);
    if ((lane & 15) == 0) red[par][lane >> 4][t >> 5] = w;
    __syncthreads();
    block_sums<2>(red[par], nw, lane, out);
  };
  float sum[2];
  sums(0.f, square(0, 0), 1, sum);
  int par = 0;
  for (long long r = blockIdx.x; r < a.rows && !*vabort; r += step, par ^= 1) {
    const uint8_t* p = s_rows + slot * g.row_bytes;
    float scale = row_rstd(sum[1], df, a.eps);
    if (a.gate_kind == MOK_GATE_TOKEN) scale *= elem_at(a.gate, r, a.gate_f32);
    F2 v[2][4];
    F2 sq[2] = {0ull, 0ull};
    uint8_t* sr = out_row(a.s, r, a.ld_s, h, SF32);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (!own[i]) continue;
      F2 b[4];
      ring_get<XF32, SHIFT>(g, p, 0, t + i * tpr, own[i], v[i]);
      ring_get<SF32, SHIFT>(g, p, 1, t + i * tpr, own[i], b);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[i][j] = fma2(mul2(v[i][j], f2(scale)), w1[i][j], mul2(alpha, b[j]));
      if (!SF32) {  // as it is stored
        const uint4 u = pack_bf16(v[i]);
        v[i][0] = f2(bf16lo(u.x), bf16hi(u.x));
        v[i][1] = f2(bf16lo(u.y), bf16hi(u.y));
        v[i][2] = f2(bf16lo(u.z), bf16hi(u.z));
        v[i][3] = f2(bf16lo(u.w), bf16hi(u.w));
      }
      ring_put<SHIFT>(sr, SF32, t + i * tpr, own[i], v[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (SHIFT) v[i][j] = keep(v[i][j], own[i] >> (2 * j));  // (not 0 for an infinite scale)
        sq[i] = fma2(v[i][j], v[i][j], sq[i]);
      }
    }
    const uint32_t next_slot = slot + 1 == g.depth ? 0 : slot + 1;
    const uint32_t next_phase = slot + 1 == g.depth ? phase ^ 1u : phase;
    const float x2 = r + step < a.rows ? square(next_slot, next_phase) : 0.f;
    sums((lo_of(sq[0]) + hi_of(sq[0])) + (lo_of(sq[1]) + hi_of(sq[1])), x2, par, sum);
    if (t == 0 && !*vabort) {  // everyone is done with the row's slot
      const long long next = r + g.depth * step;
      if (next < a.rows) fill(slot, next);
    }
    const F2 rstd = f2(row_rstd(sum[0], df, a.eps));
    uint8_t* yr = out_row(a.y, r, a.ld_y, h, 0);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (!own[i]) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i][j] = mul2(w2[i][j], mul2(v[i][j], rstd));
      ring_put<SHIFT>(yr, 0, t + i * tpr, own[i], v[i]);
    }
    slot = next_slot;
    phase = next_phase;
  }
  if (*vabort) spin_ns(1000000ull);  // copies in flight land before the block leaves
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

}  // namespace

cudaError_t launch_post_pre(const mok_post_pre_desc& D, const void* x, const void* res,
                            const void* w1, const void* w2, const void* gate, void* s, void* y,
                            int* status, cudaStream_t st) {
  if (D.rows == 0) return cudaSuccess;
  const bool xf = D.x_elem == MOK_ELEM_F32, sf = D.s_elem == MOK_ELEM_F32;
  PostPreFwd a;
  a.status = status;
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
  const bool shift = !vec && alike(x, a.ld_x, xf, a.ld_y) && alike(res, a.ld_r, sf, a.ld_y) &&
                     alike(s, a.ld_s, sf, a.ld_y) && alike(y, a.ld_y, false, a.ld_y);
  if (vec || shift) {
    const RingShape b = ring_shape(D.rows, D.d, shift, esize(xf) + esize(sf),
                                   shift ? kFwdShiftThreads : kFwdRingThreads);
    if (b.blocks > 0) {
      Ring<2> g = {{x, res}, {a.ld_x, a.ld_r}, {xf, sf}, {0, 0}, 0, 0,
                   static_cast<int>(a.ld_y & 7)};
      ProfScope prof("post_pre_rmsnorm", st);
      count_launch();
      auto run = [&](auto X, auto S) {
        constexpr bool f = decltype(X)::value, q = decltype(S)::value;
        return shift ? ring_launch(post_pre_ring_kernel<f, q, true>, a, g, b, st)
                     : ring_launch(post_pre_ring_kernel<f, q, false>, a, g, b, st);
      };
      return with_types(run, xf, sf);
    }
  }
  if (!vec) a.nvec = (a.d + 255) / 256 * 32;  // whole groups of 256 elements
  auto run = [&](auto X, auto S) {
    constexpr bool f = decltype(X)::value, g = decltype(S)::value;
    return vec ? fwd_launch<f, g, true>(a, st) : fwd_launch<f, g, false>(a, st);
  };
  return with_types(run, xf, sf);
}

}  // namespace mok
