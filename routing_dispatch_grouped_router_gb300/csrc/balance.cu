// The router's auxiliary losses (load balance and z) with the per-expert
// counts, and their gradient.
//
//   P_t = softmax(l_t), prob = mean over valid tokens of P_t, f = counts/(N k)
//   loss0 = a E sum f prob,  loss1 = b mean lse^2
//   dl_te = P_te (u0 a E (f_e - sum_j f_j P_tj) + u1 2 b lse_t) / N
//
// Bound by the bytes of the logits, and for small routers by the latency of
// its launches.  L lanes hold a token's E logits (NJ chunks of 4 each), so
// softmax and dot products are shuffles inside the warp; the sums over tokens
// stay in registers, then shared memory, then per-block partials that the last
// block to arrive adds in block order: no floating-point atomics.
#include <cuda_runtime.h>
#include <math.h>

#include <type_traits>

#include "mok_internal.h"
#include "ptx.cuh"

namespace mok {

namespace {

constexpr int kBalThreads = 256;

struct BalArgs {
  const float* logits;
  const int32_t* idx;
  const uint8_t* mask;
  float *loss, *prob, *lse;
  int32_t *counts, *n_valid;
  int* status;       // sticky device status (may be null)
  int* arrivals;     // blocks done (zero before the launch)
  float* part_prob;  // [gridDim.x, E]
  int32_t* part_cnt; // [gridDim.x, E]
  float* part_z;     // [gridDim.x]
  int32_t* part_n;   // [gridDim.x]
  long long T, ld;
  int E, k;
  float balance_coef, z_coef;
};

// Reduction over the L lanes of a token's group.
template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int L>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Logits 4 (g + L j) .. + 3 of a row for lane g, -inf past E; NaN and +inf are
// taken as -inf (*bad).
template <int L, int NJ>
__device__ __forceinline__ void load_logits(const float* row, int g, int E, bool in, bool vec,
                                            float (&l)[4 * NJ], bool* bad) {
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int e = 4 * (g + L * j);
    float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    if (in && vec && e < E) {
      v = *reinterpret_cast<const float4*>(row + e);
    } else if (in) {
      if (e < E) v.x = row[e];
      if (e + 1 < E) v.y = row[e + 1];
      if (e + 2 < E) v.z = row[e + 2];
      if (e + 3 < E) v.w = row[e + 3];
    }
    const float q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool ok = q[i] < INFINITY;
      if (!ok) *bad = true;
      l[4 * j + i] = ok ? q[i] : -INFINITY;
    }
  }
}

template <int L, int NJ>
__global__ void __launch_bounds__(kBalThreads) balance_fwd_kernel(BalArgs a, int vec) {
  constexpr int kGroups = kBalThreads / L;  // tokens in flight per block
  constexpr int kEP = 4 * L * NJ;           // E padded to the group's lanes
  __shared__ float s_prob[kGroups * kEP];
  __shared__ int32_t s_cnt[kMaxExperts];
  __shared__ float s_z[kGroups];
  __shared__ int32_t s_n[kGroups];
  __shared__ int s_last;
  const int t = threadIdx.x, g = t & (L - 1), grp = t / L;
  for (int e = t; e < a.E; e += kBalThreads) s_cnt[e] = 0;
  __syncthreads();
  float acc[4 * NJ];
#pragma unroll
  for (int i = 0; i < 4 * NJ; ++i) acc[i] = 0.f;
  float z = 0.f;
  int n = 0;
  bool bad = false, bad_idx = false;
  const long long step = static_cast<long long>(gridDim.x) * kGroups;
  // every group of a warp makes the same number of rounds (shuffles)
  for (long long base = static_cast<long long>(blockIdx.x) * kGroups; base < a.T; base += step) {
    const long long tok = base + grp;
    const bool in = tok < a.T;
    const bool valid = in && (!a.mask || a.mask[tok] != 0);
    float l[4 * NJ];
    bool bad_tok = false;
    load_logits<L, NJ>(a.logits + tok * a.ld, g, a.E, in, vec != 0, l, &bad_tok);
    bad = bad || (bad_tok && valid);
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < 4 * NJ; ++i) top = fmaxf(top, l[i]);
    top = group_max<L>(top);
    float sum = 0.f;
    const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (int i = 0; i < 4 * NJ; ++i) {
      l[i] = expf(l[i] - ref);
      sum += l[i];
    }
    sum = group_sum<L>(sum);
    const float lse = sum > 0.f ? ref + logf(sum) : -INFINITY;
    if (in && g == 0) a.lse[tok] = lse;
    if (valid) {
      if (sum > 0.f) {
        const float inv = 1.0f / sum;
#pragma unroll
        for (int i = 0; i < 4 * NJ; ++i) acc[i] = fmaf(l[i], inv, acc[i]);
        if (g == 0) z = fmaf(lse, lse, z);
      }
      if (g == 0) ++n;
      for (int s = g; s < a.k; s += L) {
        const int e = a.idx[tok * a.k + s];
        if (e >= 0 && e < a.E) atomicAdd(&s_cnt[e], 1);
        else bad_idx = true;
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) s_prob[grp * kEP + 4 * (g + L * j) + i] = acc[4 * j + i];
  if (g == 0) {
    s_z[grp] = z;
    s_n[grp] = n;
  }
  if (bad) set_status(a.status, MOK_ERR_DEVICE_NONFINITE);
  if (bad_idx) set_status(a.status, MOK_ERR_DEVICE_INDEX);
  __syncthreads();
  for (int e = t; e < a.E; e += kBalThreads) {
    float p = 0.f;
    for (int q = 0; q < kGroups; ++q) p += s_prob[q * kEP + e];
    a.part_prob[static_cast<long long>(blockIdx.x) * a.E + e] = p;
    a.part_cnt[static_cast<long long>(blockIdx.x) * a.E + e] = s_cnt[e];
  }
  if (t == 0) {
    float zz = 0.f;
    int nn = 0;
    for (int q = 0; q < kGroups; ++q) {
      zz += s_z[q];
      nn += s_n[q];
    }
    a.part_z[blockIdx.x] = zz;
    a.part_n[blockIdx.x] = nn;
  }
  // the last block to arrive adds the partials in block order
  __threadfence();
  __syncthreads();
  if (t == 0) s_last = gridDim.x == 1 || atomicAdd(a.arrivals, 1) == static_cast<int>(gridDim.x) - 1;
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  const int G = gridDim.x;
  __shared__ float s_red[kBalThreads];
  __shared__ int s_nall;
  if (t == 0) {
    float zz = 0.f;
    int nn = 0;
    for (int b = 0; b < G; ++b) {
      zz += __ldcg(a.part_z + b);
      nn += __ldcg(a.part_n + b);
    }
    s_nall = nn;
    a.n_valid[0] = nn;
    // (without a z loss its sum may be beyond fp32: 0 inf would be NaN)
    a.loss[1] = nn > 0 && a.z_coef != 0.f ? a.z_coef * zz / static_cast<float>(nn) : 0.f;
  }
  __syncthreads();
  const float inv_n = s_nall > 0 ? 1.0f / static_cast<float>(s_nall) : 0.f;
  float dot = 0.f;
  for (int e = t; e < a.E; e += kBalThreads) {
    float p = 0.f;
    int c = 0;
#pragma unroll 8
    for (int b = 0; b < G; ++b) {
      p += __ldcg(a.part_prob + static_cast<long long>(b) * a.E + e);
      c += __ldcg(a.part_cnt + static_cast<long long>(b) * a.E + e);
    }
    p *= inv_n;
    a.prob[e] = p;
    a.counts[e] = c;
    dot = fmaf(static_cast<float>(c), p, dot);
  }
  s_red[t] = dot;
  __syncthreads();
  for (int o = kBalThreads / 2; o > 0; o >>= 1) {
    if (t < o) s_red[t] += s_red[t + o];
    __syncthreads();
  }
  if (t == 0)
    a.loss[0] = a.balance_coef * static_cast<float>(a.E) / static_cast<float>(a.k) * s_red[0] * inv_n;
}

struct BalBwd {
  const float *dloss, *logits, *lse;
  const int32_t *counts, *n_valid;
  const uint8_t* mask;
  float* dlogits;
  long long T, ld;
  int E, k;
  float balance_coef, z_coef;
};

template <int L, int NJ>
__global__ void __launch_bounds__(kBalThreads) balance_bwd_kernel(BalBwd a, int vec) {
  constexpr int kGroups = kBalThreads / L;
  const int t = threadIdx.x, g = t & (L - 1), grp = t / L;
  const int nv = *a.n_valid;
  const float inv_n = nv > 0 ? 1.0f / static_cast<float>(nv) : 0.f;
  // balance: A (f_e - 1/E), with f_e - 1/E = (c_e E - N k) / (N k E) exact in
  // the integer numerator; subtracting the constant 1/E changes nothing (sum
  // of P = 1) and keeps the difference f_e - sum f P from cancelling
  const float A = a.dloss[0] * a.balance_coef * inv_n * inv_n / static_cast<float>(a.k);
  const float Z = a.dloss[1] * 2.0f * a.z_coef * inv_n;
  float f[4 * NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = 4 * (g + L * j) + i;
      f[4 * j + i] = e < a.E ? static_cast<float>(static_cast<long long>(a.counts[e]) * a.E -
                                                  static_cast<long long>(nv) * a.k) * A
                             : 0.f;
    }
  const long long step = static_cast<long long>(gridDim.x) * kGroups;
  for (long long base = static_cast<long long>(blockIdx.x) * kGroups; base < a.T; base += step) {
    const long long tok = base + grp;
    const bool in = tok < a.T;
    const bool valid = in && (!a.mask || a.mask[tok] != 0);
    float l[4 * NJ];
    bool bad = false;
    load_logits<L, NJ>(a.logits + tok * a.ld, g, a.E, in, vec != 0, l, &bad);
    const float lse = in ? a.lse[tok] : 0.f;
    const bool some = valid && lse > -INFINITY;
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < 4 * NJ; ++i) {
      l[i] = some ? expf(l[i] - lse) : 0.f;
      dot = fmaf(f[i], l[i], dot);
    }
    dot = group_sum<L>(dot);
    const float c = some ? Z * lse - dot : 0.f;
    float* row = a.dlogits + tok * a.ld;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int e = 4 * (g + L * j);
      float4 o;
      o.x = l[4 * j] * (f[4 * j] + c);
      o.y = l[4 * j + 1] * (f[4 * j + 1] + c);
      o.z = l[4 * j + 2] * (f[4 * j + 2] + c);
      o.w = l[4 * j + 3] * (f[4 * j + 3] + c);
      if (in && vec && e < a.E) {
        *reinterpret_cast<float4*>(row + e) = o;
      } else if (in) {
        if (e < a.E) row[e] = o.x;
        if (e + 1 < a.E) row[e + 1] = o.y;
        if (e + 2 < a.E) row[e + 2] = o.z;
        if (e + 3 < a.E) row[e + 3] = o.w;
      }
    }
  }
}

// Lanes and chunks of a token by E: the fewest lanes that hold E in one chunk
// each, all 32 with up to four chunks beyond.
template <typename F>
void by_width(int E, const F& f) {
  if (E <= 16) f(std::integral_constant<int, 4>(), std::integral_constant<int, 1>());
  else if (E <= 32) f(std::integral_constant<int, 8>(), std::integral_constant<int, 1>());
  else if (E <= 64) f(std::integral_constant<int, 16>(), std::integral_constant<int, 1>());
  else if (E <= 128) f(std::integral_constant<int, 32>(), std::integral_constant<int, 1>());
  else if (E <= 256) f(std::integral_constant<int, 32>(), std::integral_constant<int, 2>());
  else if (E <= 384) f(std::integral_constant<int, 32>(), std::integral_constant<int, 3>());
  else f(std::integral_constant<int, 32>(), std::integral_constant<int, 4>());
}

int lanes_of(int E) { return E <= 16 ? 4 : E <= 32 ? 8 : E <= 64 ? 16 : 32; }

bool vec4(const void* p, long long ld, int E) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % 4 == 0 && E % 4 == 0;
}

}  // namespace

int64_t balance_blocks(const mok_balance_desc& D) {
  const int64_t groups = kBalThreads / lanes_of(D.E);
  const int64_t b = (D.T + groups - 1) / groups;
  return b < 1 ? 1 : (b < 152 ? b : 152);  // whatever the device: the sums do not depend on it
}

void balance_layout(const mok_balance_desc& D, BalanceWs* W) {
  const size_t G = static_cast<size_t>(balance_blocks(D));
  auto al = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  W->arrivals = 0;
  W->part_prob = 256;
  W->part_cnt = W->part_prob + al(G * D.E * 4);
  W->part_z = W->part_cnt + al(G * D.E * 4);
  W->part_n = W->part_z + al(G * 4);
  W->total = W->part_n + al(G * 4);
}

cudaError_t launch_balance_fwd(const mok_balance_desc& D, const float* logits,
                               const int32_t* idx, const uint8_t* mask, float* loss,
                               int32_t* counts, float* prob, float* lse, int32_t* n_valid,
                               void* ws, int* status, cudaStream_t st) {
  BalanceWs W;
  balance_layout(D, &W);
  char* b = static_cast<char*>(ws);
  BalArgs a;
  a.logits = logits; a.idx = idx; a.mask = mask;
  a.loss = loss; a.prob = prob; a.lse = lse; a.counts = counts; a.n_valid = n_valid;
  a.status = status;
  a.arrivals = reinterpret_cast<int*>(b + W.arrivals);
  a.part_prob = reinterpret_cast<float*>(b + W.part_prob);
  a.part_cnt = reinterpret_cast<int32_t*>(b + W.part_cnt);
  a.part_z = reinterpret_cast<float*>(b + W.part_z);
  a.part_n = reinterpret_cast<int32_t*>(b + W.part_n);
  a.T = D.T; a.ld = D.ld_logits; a.E = D.E; a.k = D.k;
  a.balance_coef = D.balance_coef; a.z_coef = D.z_coef;
  const unsigned grid = static_cast<unsigned>(balance_blocks(D));
  if (grid > 1) {
    cudaError_t e = cudaMemsetAsync(a.arrivals, 0, 4, st);
    if (e != cudaSuccess) return e;
  }
  const int vec = vec4(logits, a.ld, a.E);
  ProfScope prof("router_balance", st);
  by_width(D.E, [&](auto L, auto NJ) {
    balance_fwd_kernel<decltype(L)::value, decltype(NJ)::value><<<grid, kBalThreads, 0, st>>>(a, vec);
  });
  count_launch();
  return cudaGetLastError();
}

cudaError_t launch_balance_bwd(const mok_balance_desc& D, const float* dloss,
                               const float* logits, const float* lse, const int32_t* counts,
                               const int32_t* n_valid, const uint8_t* mask, float* dlogits,
                               cudaStream_t st) {
  if (D.T == 0) return cudaSuccess;
  BalBwd a;
  a.dloss = dloss; a.logits = logits; a.lse = lse; a.counts = counts; a.n_valid = n_valid;
  a.mask = mask; a.dlogits = dlogits;
  a.T = D.T; a.ld = D.ld_logits; a.E = D.E; a.k = D.k;
  a.balance_coef = D.balance_coef; a.z_coef = D.z_coef;
  const int64_t groups = kBalThreads / lanes_of(D.E);
  const int64_t need = (D.T + groups - 1) / groups;
  const int64_t cap = 8LL * num_sms_current_device();
  const unsigned grid = static_cast<unsigned>(need < cap ? need : cap);
  const int vec = vec4(logits, a.ld, a.E) && vec4(dlogits, a.ld, a.E);
  ProfScope prof("router_balance_bwd", st);
  by_width(D.E, [&](auto L, auto NJ) {
    balance_bwd_kernel<decltype(L)::value, decltype(NJ)::value><<<grid, kBalThreads, 0, st>>>(a, vec);
  });
  count_launch();
  return cudaGetLastError();
}

}  // namespace mok
