// Backward of the norms after and before a block through a ring of rows in shared
// memory (post_norm.cu has the formulas).
#include "post_norm.cuh"

namespace mok {

// A ring of rows (s, dy, x, ds), two vectors per thread, one reduction a row
// (post_norm_bwd.cu has the sums).
template <bool DYF32, bool XF32, bool SF32, bool SHIFT, int THREADS>
__global__ void __launch_bounds__(THREADS)
    post_pre_bwd_ring_kernel(PostPreBwd a, Ring<4> g) {
  extern __shared__ __align__(128) uint8_t s_rows[];
  __shared__ __align__(8) uint64_t full[kRingMaxDepth];
  __shared__ float red[2][8][16];  // [row parity][sum][warp]
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
    ring_fill<4, SHIFT>(g, s_rows + slot * g.row_bytes, &full[slot], r, a.rows, a.d, h);
  };
  if (t == 0)
    for (uint32_t i = 0; i < g.depth && blockIdx.x + i * step < a.rows; ++i)
      fill(i, blockIdx.x + i * step);
  F2 w1[2][4], w2[2][4], dw1[2][4], dw2[2][4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    ring_weight<!SHIFT>(a.w1, a.w_f32, t + i * tpr, h, own[i], w1[i]);
    ring_weight<!SHIFT>(a.w2, a.w_f32, t + i * tpr, h, own[i], w2[i]);
    if (a.gate_kind == MOK_GATE_CHANNEL) {
      F2 z[4];
      ring_weight<!SHIFT>(a.gate, a.gate_f32, t + i * tpr, h, own[i], z);
#pragma unroll
      for (int j = 0; j < 4; ++j) w1[i][j] = mul2(w1[i][j], z[j]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) dw1[i][j] = dw2[i][j] = 0ull;
  }
  const float df = static_cast<float>(a.d);
  uint32_t slot = 0, phase = 0;
  // the warps' sums of the row in a slot: of s^2, x^2, dy w2 s, dy w2 u, s u, ds u
  auto first_pass = [&](uint32_t sl, uint32_t ph, int par) {
    if (!mbar_wait(&full[sl], ph, vabort)) {
      *vabort = 1;
      set_status(a.status, MOK_ERR_DEVICE_TIMEOUT);
    }
    const uint8_t* p = s_rows + sl * g.row_bytes;
    F2 q[6] = {0ull, 0ull, 0ull, 0ull, 0ull, 0ull};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (!own[i]) continue;
      F2 s[4], dy[4], x[4];
      ring_get<SF32, SHIFT>(g, p, 0, t + i * tpr, own[i], s);
      ring_get<DYF32, SHIFT>(g, p, 1, t + i * tpr, own[i], dy);
      ring_get<XF32, SHIFT>(g, p, 2, t + i * tpr, own[i], x);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const F2 gw = mul2(dy[j], w2[i][j]);
        q[0] = fma2(s[j], s[j], q[0]);
        q[1] = fma2(x[j], x[j], q[1]);
        q[2] = fma2(gw, s[j], q[2]);
        x[j] = mul2(x[j], w1[i][j]);
        q[3] = fma2(gw, x[j], q[3]);
        q[4] = fma2(s[j], x[j], q[4]);
      }
      if (a.ds) {
        ring_get<SF32, SHIFT>(g, p, 3, t + i * tpr, own[i], dy);
#pragma unroll
        for (int j = 0; j < 4; ++j) q[5] = fma2(dy[j], x[j], q[5]);
      }
    }
    float v[8];
#pragma unroll
    for (int i = 0; i < 6; ++i) v[i] = lo_of(q[i]) + hi_of(q[i]);
    v[6] = v[7] = 0.f;
    const float w = warp_sums(v, lane);
    if ((lane & 3) == 0) red[par][lane >> 2][t >> 5] = w;
  };
  first_pass(0, 0, 0);
  // (with a third slot the next row's first pass comes before this one's second)
  const bool early = g.depth > 2;
  int par = 0;
  for (long long r = blockIdx.x; r < a.rows; r += step, par ^= 1) {
    __syncthreads();
    if (*vabort) break;  // (set before the barrier: every thread sees it)
    const uint32_t next_slot = slot + 1 == g.depth ? 0 : slot + 1;
    const uint32_t next_phase = slot + 1 == g.depth ? phase ^ 1u : phase;
    if (t == 0 && r >= step) {  // everyone is done with the row before's slot
      const long long next = r + (g.depth - 1) * step;
      if (next < a.rows) fill(slot == 0 ? g.depth - 1 : slot - 1, next);
    }
    const float gt = a.gate_kind == MOK_GATE_TOKEN ? elem_at(a.gate, r, a.gate_f32) : 1.0f;
    float sum[8];
    block_sums<8>(red[par], nw, lane, sum);
    const bool more = r + step < a.rows;
    if (early && more) first_pass(next_slot, next_phase, par ^ 1);
    const float rstd2 = row_rstd(sum[0], df, a.eps), rstd1 = row_rstd(sum[1], df, a.eps);
    const float c = sum[2] * rstd2 * rstd2 * a.inv_d * rstd2;
    const float dot = (sum[3] * rstd2 - sum[4] * c + sum[5]) * rstd1;
    if (a.dgate && t == 0) a.dgate[r] = a.accumulate ? a.dgate[r] + dot : dot;
    const F2 k = f2(-gt * dot * rstd1 * rstd1 * a.inv_d);
    const F2 nc = f2(-c), r2 = f2(rstd2), nr = f2(rstd1 * gt);
    const uint8_t* p = s_rows + slot * g.row_bytes;
    uint8_t* dr = out_row(a.dr, r, a.ld_dr, h, SF32);
    uint8_t* dx = out_row(a.dx, r, a.ld_dx, h, a.dx_f32);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (!own[i]) continue;
      F2 s[4], dy[4], x[4], tt[4];
      ring_get<SF32, SHIFT>(g, p, 0, t + i * tpr, own[i], s);
      ring_get<DYF32, SHIFT>(g, p, 1, t + i * tpr, own[i], dy);
      ring_get<XF32, SHIFT>(g, p, 2, t + i * tpr, own[i], x);
      if (a.ds) {
        ring_get<SF32, SHIFT>(g, p, 3, t + i * tpr, own[i], tt);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) tt[j] = 0ull;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        tt[j] = fma2(mul2(dy[j], w2[i][j]), r2, fma2(s[j], nc, tt[j]));
        dw2[i][j] = fma2(dy[j], mul2(s[j], r2), dw2[i][j]);
        dw1[i][j] = fma2(tt[j], mul2(x[j], nr), dw1[i][j]);
        x[j] = fma2(mul2(tt[j], w1[i][j]), nr, mul2(x[j], k));
        tt[j] = mul2(tt[j], f2(a.alpha));
      }
      ring_put<SHIFT>(dr, SF32, t + i * tpr, own[i], tt);
      ring_put<SHIFT>(dx, a.dx_f32, t + i * tpr, own[i], x);
    }
    if (!early && more) first_pass(next_slot, next_phase, par ^ 1);
    slot = next_slot;
    phase = next_phase;
  }
  if (*vabort) {
    spin_ns(1000000ull);  // copies in flight land before the block leaves
    return;
  }
  if (!a.part) return;
  float* out = a.part + static_cast<long long>(blockIdx.x) * a.d;
  const long long second = static_cast<long long>(gridDim.x) * a.d;
  // through the ring's memory, for whole sectors
  float* s_dw = reinterpret_cast<float*>(s_rows);
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const F2 v = q ? dw2[i][j >> 1] : dw1[i][j >> 1];
        if (own[i] >> j & 1u) s_dw[8 * (t + i * tpr) - h + j] = j & 1 ? hi_of(v) : lo_of(v);
      }
    __syncthreads();
    for (int e = t; e < a.d; e += blockDim.x) out[q * second + e] = s_dw[e];
  }
}

cudaError_t launch_post_pre_bwd_ring(const PostPreBwd& a, Ring<4>& g, const RingShape& b, bool yf,
                                     bool xf, bool sf, bool shift, cudaStream_t st) {
  return with_types(
      [&](auto Y, auto X, auto S) {
        constexpr bool y = decltype(Y)::value, f = decltype(X)::value, q = decltype(S)::value;
        if (!shift)
          return ring_launch(post_pre_bwd_ring_kernel<y, f, q, false, kRingThreads>, a, g, b,
                             st);
        if (b.tpr <= kBwdShiftThreads)
          return ring_launch(post_pre_bwd_ring_kernel<y, f, q, true, kBwdShiftThreads>, a, g,
                             b, st);
        return ring_launch(post_pre_bwd_ring_kernel<y, f, q, true, kRingThreads>, a, g, b, st);
      },
      yf, xf, sf);
}

}  // namespace mok
