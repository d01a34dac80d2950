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
// stay in registers, then shared memory, then per-block partials that a second
// kernel (launched while the first drains) adds in block order: no
// floating-point atomics.  (256 tokens of 8 experts: 4.7 us, one launch; 16384 of
// 128: 11.5 us, of which the sum 4, floor 1.3; the backward of 8192 of 384: 8.5 us,
// 3.0 TB/s of logits and gradients, which L2 mostly holds; floor 3.7.)
#include <cuda_runtime.h>
#include <math.h>

#include <type_traits>

#include "mok_internal.h"
#include "ptx.cuh"

namespace mok {

namespace {

// Threads of the forward's blocks: 1024 so that the tokens of a large batch are
// in flight at once; 256 where one block does it all (shorter barriers).
constexpr int kManyThreads = 1024;
constexpr int kFewThreads = 256;
constexpr int kBwdThreads = 256;
// Blocks of the forward.
constexpr int kFwdBlocks = kGb300Sms;

struct BalArgs {
  const float* logits;
  const int32_t* idx;
  const uint8_t* mask;
  float *loss, *prob, *lse;
  int32_t *counts, *n_valid;
  int* status;       // sticky device status (may be null)
  float* part_prob;  // [gridDim.x, E rounded up to 4]
  int32_t* part_cnt; // [gridDim.x, E rounded up to 4]
  float* part_z;     // [gridDim.x]
  int32_t* part_n;   // [gridDim.x]
  int blocks;        // of the first kernel
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

// Logits 4 (g + L j) .. + 3 of a row for lane g, -inf past E.
template <int L, int NJ>
__device__ __forceinline__ void load_logits(const float* row, int g, int E, bool in, bool vec,
                                            float (&l)[4 * NJ]) {
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
    l[4 * j] = v.x; l[4 * j + 1] = v.y; l[4 * j + 2] = v.z; l[4 * j + 3] = v.w;
  }
}

// NaN and +inf become -inf; returns whether there were any.
template <int N>
__device__ __forceinline__ bool clean(float (&l)[N]) {
  bool bad = false;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const bool ok = l[i] < INFINITY;
    bad = bad || !ok;
    l[i] = ok ? l[i] : -INFINITY;
  }
  return bad;
}

// Sums over the threads of a block: thread t holds float4 / int4 column
// t % cols (a power of two, at most 128) of slice t / cols, and z, n of its own.
// On return threads t < cols hold column t's sums, and threads t < 128 z's and
// n's.  A fixed tree: lanes, then warps in order.
template <int TH>
__device__ __forceinline__ void block_columns(int cols, float4& p, int4& c, float& z, int& n,
                                              float4* s_f4, int4* s_i4, float* s_z, int* s_n) {
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  constexpr int W = TH / 32;
  __syncthreads();  // the shared buffers are free
  for (int o = 16; o >= cols; o >>= 1) {
    p.x += __shfl_xor_sync(0xffffffffu, p.x, o);
    p.y += __shfl_xor_sync(0xffffffffu, p.y, o);
    p.z += __shfl_xor_sync(0xffffffffu, p.z, o);
    p.w += __shfl_xor_sync(0xffffffffu, p.w, o);
    c.x += __shfl_xor_sync(0xffffffffu, c.x, o);
    c.y += __shfl_xor_sync(0xffffffffu, c.y, o);
    c.z += __shfl_xor_sync(0xffffffffu, c.z, o);
    c.w += __shfl_xor_sync(0xffffffffu, c.w, o);
  }
  z = group_sum<32>(z);
  n = __reduce_add_sync(0xffffffffu, n);
  s_f4[t] = p;
  s_i4[t] = c;
  if (lane == 0) {
    s_z[warp] = z;
    s_n[warp] = n;
  }
  __syncthreads();
  if (t < cols) {  // warps (cols <= 32) or slices of several warps
    const int step = cols < 32 ? 32 : cols;
    p = make_float4(0.f, 0.f, 0.f, 0.f);
    c = make_int4(0, 0, 0, 0);
#pragma unroll 4
    for (int i = t; i < TH; i += step) {
      const float4 f = s_f4[i];
      const int4 k = s_i4[i];
      p.x += f.x; p.y += f.y; p.z += f.z; p.w += f.w;
      c.x += k.x; c.y += k.y; c.z += k.z; c.w += k.w;
    }
  }
  if (t < 128) {  // the threads that columns go to
    z = group_sum<32>(lane < W ? s_z[lane] : 0.f);
    n = __reduce_add_sync(0xffffffffu, lane < W ? s_n[lane] : 0);
  }
}

template <int TH>
struct BalShared {
  float4 f4[TH];
  int4 i4[TH];
  float z[TH / 32];
  int n[TH / 32];
};

// Float4 columns of E, padded to a power of two.
__device__ __forceinline__ int pow2_cols(int e4) {
  int cols = 1;
  while (cols < e4) cols *= 2;
  return cols;
}

// The outputs from the column sums p, c of threads t < E/4 and z, n.
__device__ __forceinline__ void balance_out(const BalArgs& a, float4 p, int4 c, float z, int n,
                                            float* s_z) {
  const int t = threadIdx.x, e4 = (a.E + 3) / 4;
  const float inv_n = n > 0 ? 1.0f / static_cast<float>(n) : 0.f;
  float dot = 0.f;
  if (t < e4) {
    const float pv[4] = {p.x * inv_n, p.y * inv_n, p.z * inv_n, p.w * inv_n};
    const int cv[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (4 * t + i < a.E) {
        a.prob[4 * t + i] = pv[i];
        a.counts[4 * t + i] = cv[i];
        dot = fmaf(static_cast<float>(cv[i]), pv[i], dot);
      }
    }
  }
  __syncthreads();  // s_z has been read
  if (t < 128) {  // E/4 <= 128: four warps hold every product
    dot = group_sum<32>(dot);
    if ((t & 31) == 0) s_z[t >> 5] = dot;
  }
  __syncthreads();
  if (t == 0) {
    a.n_valid[0] = n;
    a.loss[0] = a.balance_coef * static_cast<float>(a.E) / static_cast<float>(a.k) *
                ((s_z[0] + s_z[1]) + (s_z[2] + s_z[3])) * inv_n;
    // (without a z loss its sum may be beyond fp32: 0 inf would be NaN)
    a.loss[1] = n > 0 && a.z_coef != 0.f ? a.z_coef * z * inv_n : 0.f;
  }
}

// The second kernel: one block adds the first one's partials in block order by
// slices of its threads.
__global__ void __launch_bounds__(kManyThreads) balance_sum_kernel(BalArgs a) {
  __shared__ BalShared<kManyThreads> s;
  grid_dep_launch();
  grid_dep_wait();
  const int t = threadIdx.x, e4 = (a.E + 3) / 4, cols = pow2_cols(e4);
  const int col = t & (cols - 1), slices = kManyThreads / cols, G = a.blocks;
  float z = t < G ? a.part_z[t] : 0.f;  // (fewer blocks than threads)
  int n = t < G ? a.part_n[t] : 0;
  float4 p = make_float4(0.f, 0.f, 0.f, 0.f);
  int4 c = make_int4(0, 0, 0, 0);
  if (col < e4) {
    const float4* pp = reinterpret_cast<const float4*>(a.part_prob) + col;
    const int4* pc = reinterpret_cast<const int4*>(a.part_cnt) + col;
#pragma unroll 10
    for (int b = t / cols; b < G; b += slices) {
      const float4 q = pp[static_cast<long long>(b) * e4];
      const int4 k = pc[static_cast<long long>(b) * e4];
      p.x += q.x; p.y += q.y; p.z += q.z; p.w += q.w;
      c.x += k.x; c.y += k.y; c.z += k.z; c.w += k.w;
    }
  }
  block_columns<kManyThreads>(cols, p, c, z, n, s.f4, s.i4, s.z, s.n);
  balance_out(a, p, c, z, n, s.z);
}

template <int TH, int L, int NJ>
__global__ void __launch_bounds__(TH) balance_fwd_kernel(BalArgs a, int vec) {
  constexpr int kGroups = TH / L;           // tokens of a block at a time
  constexpr int kE4 = L * NJ;               // float4 columns of the group's lanes
  // tokens whose loads a group has in flight (registers: 64 a thread)
  constexpr int U = NJ == 1 ? 4 : (NJ == 2 ? 2 : 1);
  extern __shared__ __align__(16) float4 s_prob[];  // [kGroups][kE4]
  __shared__ BalShared<TH> s;
  __shared__ __align__(16) int32_t s_cnt[kMaxExperts];
  grid_dep_launch();
  const int t = threadIdx.x, g = t & (L - 1), grp = t / L;
  for (int e = t; e < kMaxExperts; e += TH) s_cnt[e] = 0;
  __syncthreads();
  grid_dep_wait();
  float acc[4 * NJ];
#pragma unroll
  for (int i = 0; i < 4 * NJ; ++i) acc[i] = 0.f;
  float z = 0.f;
  int n = 0;
  bool bad = false, bad_idx = false;
  const long long step = static_cast<long long>(gridDim.x) * kGroups;
  // every group of a warp makes the same number of rounds (shuffles)
  for (long long base = static_cast<long long>(blockIdx.x) * kGroups; base < a.T;
       base += U * step) {
    float l[U][4 * NJ];
    int id[U][2];
    bool in[U], valid[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {  // all loads first
      const long long tok = base + u * step + grp;
      in[u] = tok < a.T;
      load_logits<L, NJ>(a.logits + tok * a.ld, g, a.E, in[u], vec != 0, l[u]);
      valid[u] = in[u] && (!a.mask || a.mask[tok] != 0);
#pragma unroll
      for (int i = 0; i < 2; ++i)  // (k <= 8 slots over at least 4 lanes)
        id[u][i] = in[u] && g + i * L < a.k ? a.idx[tok * a.k + g + i * L] : -1;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      bad = (clean(l[u]) && valid[u]) || bad;
      float top = -INFINITY;
#pragma unroll
      for (int i = 0; i < 4 * NJ; ++i) top = fmaxf(top, l[u][i]);
      top = group_max<L>(top);
      float sum = 0.f;
      const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
      for (int i = 0; i < 4 * NJ; ++i) {
        l[u][i] = expf(l[u][i] - ref);
        sum += l[u][i];
      }
      sum = group_sum<L>(sum);
      const float lse = sum > 0.f ? ref + logf(sum) : -INFINITY;
      if (in[u] && g == 0) a.lse[base + u * step + grp] = lse;
      if (valid[u]) {
        if (sum > 0.f) {
          const float inv = 1.0f / sum;
#pragma unroll
          for (int i = 0; i < 4 * NJ; ++i) acc[i] = fmaf(l[u][i], inv, acc[i]);
          if (g == 0) z = fmaf(lse, lse, z);
        }
        if (g == 0) ++n;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (g + i * L >= a.k) break;
          const int e = id[u][i];
          if (e >= 0 && e < a.E) atomicAdd(&s_cnt[e], 1);
          else bad_idx = true;
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NJ; ++j)
    s_prob[grp * kE4 + g + L * j] =
        make_float4(acc[4 * j], acc[4 * j + 1], acc[4 * j + 2], acc[4 * j + 3]);
  if (bad) set_status(a.status, MOK_ERR_DEVICE_NONFINITE);
  if (bad_idx) set_status(a.status, MOK_ERR_DEVICE_INDEX);
  __syncthreads();
  // the groups' sums: slices of the threads over the float4 columns
  const int e4 = (a.E + 3) / 4, cols = pow2_cols(e4);
  const int col = t & (cols - 1), sl = t / cols, slices = TH / cols;
  float4 p = make_float4(0.f, 0.f, 0.f, 0.f);
  int4 c = make_int4(0, 0, 0, 0);
  if (col < e4) {
    for (int q = sl; q < kGroups; q += slices) {
      const float4 f = s_prob[q * kE4 + col];
      p.x += f.x; p.y += f.y; p.z += f.z; p.w += f.w;
    }
    if (sl == 0) c = *reinterpret_cast<const int4*>(s_cnt + 4 * col);
  }
  block_columns<TH>(cols, p, c, z, n, s.f4, s.i4, s.z, s.n);
  if (gridDim.x == 1) {
    balance_out(a, p, c, z, n, s.z);
    return;
  }
  const long long b = blockIdx.x;  // this block's partials
  if (t < e4) {
    reinterpret_cast<float4*>(a.part_prob)[b * e4 + t] = p;
    reinterpret_cast<int4*>(a.part_cnt)[b * e4 + t] = c;
  }
  if (t == 0) {
    a.part_z[b] = z;
    a.part_n[b] = n;
  }
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

// Tokens whose loads a group of the backward has in flight at once: 64 registers
// a thread, so that four blocks share an SM.
constexpr int bwd_unroll(int nj) { return nj <= 3 ? 2 : 1; }

template <int L, int NJ>
__global__ void __launch_bounds__(kBwdThreads, 4) balance_bwd_kernel(BalBwd a, int vec) {
  constexpr int kUnroll = bwd_unroll(NJ);
  constexpr int kGroups = kBwdThreads / L;
  const int t = threadIdx.x, g = t & (L - 1), grp = t / L;
  const long long step = static_cast<long long>(gridDim.x) * kGroups;
  grid_dep_launch();
  grid_dep_wait();
  float f[4 * NJ];
  float Z = 0.f;
  for (long long base = static_cast<long long>(blockIdx.x) * kGroups; base < a.T;
       base += kUnroll * step) {
    float l[kUnroll][4 * NJ], lse[kUnroll];
    bool in[kUnroll], some[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {  // all loads first
      const long long tok = base + u * step + grp;
      in[u] = tok < a.T;
      load_logits<L, NJ>(a.logits + tok * a.ld, g, a.E, in[u], vec != 0, l[u]);
      lse[u] = in[u] ? a.lse[tok] : -INFINITY;
      some[u] = in[u] && (!a.mask || a.mask[tok] != 0);
    }
    if (base == static_cast<long long>(blockIdx.x) * kGroups) {
      // (after the first tokens' loads have gone out)
      // balance: A (f_e - 1/E), with f_e - 1/E = (c_e E - N k) / (N k E) exact
      // in the integer numerator; subtracting the constant 1/E changes nothing
      // (sum of P = 1) and keeps the difference f_e - sum f P from cancelling
      const int nv = *a.n_valid;
      const float inv_n = nv > 0 ? 1.0f / static_cast<float>(nv) : 0.f;
      const float A = a.dloss[0] * a.balance_coef * inv_n * inv_n / static_cast<float>(a.k);
      Z = a.dloss[1] * 2.0f * a.z_coef * inv_n;
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = 4 * (g + L * j) + i;
          f[4 * j + i] = e < a.E ? static_cast<float>(static_cast<long long>(a.counts[e]) * a.E -
                                                      static_cast<long long>(nv) * a.k) * A
                                 : 0.f;
        }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      clean(l[u]);
      // P = exp(l - lse) / its sum over the row: lse's rounding (1e-3 at 1e4; from
      // 1e8 on all of log E) shifts every term of a row alike, and without the
      // division the row would not sum to 1
      some[u] = some[u] && lse[u] > -INFINITY;
      float sum = 0.f, dot = 0.f;
#pragma unroll
      for (int i = 0; i < 4 * NJ; ++i) {
        l[u][i] = some[u] ? expf(l[u][i] - lse[u]) : 0.f;
        sum += l[u][i];
        dot = fmaf(f[i], l[u][i], dot);
      }
      sum = group_sum<L>(sum);  // (about 1: the quick division's 2 ulp, and no spills)
      const float inv = sum > 0.f ? __fdividef(1.0f, sum) : 0.f;
#pragma unroll
      for (int i = 0; i < 4 * NJ; ++i) l[u][i] *= inv;
      dot = group_sum<L>(dot) * inv;
      const float c = some[u] ? Z * lse[u] - dot : 0.f;
      float* row = a.dlogits + (base + u * step + grp) * a.ld;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int e = 4 * (g + L * j);
        float4 o;
        o.x = l[u][4 * j] * (f[4 * j] + c);
        o.y = l[u][4 * j + 1] * (f[4 * j + 1] + c);
        o.z = l[u][4 * j + 2] * (f[4 * j + 2] + c);
        o.w = l[u][4 * j + 3] * (f[4 * j + 3] + c);
        if (in[u] && vec && e < a.E) {
          *reinterpret_cast<float4*>(row + e) = o;
        } else if (in[u]) {
          if (e < a.E) row[e] = o.x;
          if (e + 1 < a.E) row[e + 1] = o.y;
          if (e + 2 < a.E) row[e + 2] = o.z;
          if (e + 3 < a.E) row[e + 3] = o.w;
        }
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
  // one block while its groups take their tokens in one round of loads: faster
  // than several blocks and their sum (128 tokens of 128 experts: 7.5 and 8.8 us;
  // 256: 11.7 and 8.8; 64 of 384: 9.4 and 7.9)
  const int64_t groups = kManyThreads / lanes_of(D.E);
  if (D.T <= (D.E <= 128 ? 4 : 1) * groups) return 1;
  const int64_t b = (D.T + groups - 1) / groups;
  return b < kFwdBlocks ? b : kFwdBlocks;
}

void balance_layout(const mok_balance_desc& D, BalanceWs* W) {
  // (one block leaves no partials)
  const size_t G = balance_blocks(D) > 1 ? static_cast<size_t>(balance_blocks(D)) : 0;
  auto al = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  const size_t e_pad = (static_cast<size_t>(D.E) + 3) / 4 * 4;
  W->part_prob = 0;
  W->part_cnt = W->part_prob + al(G * e_pad * 4);
  W->part_z = W->part_cnt + al(G * e_pad * 4);
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
  a.part_prob = reinterpret_cast<float*>(b + W.part_prob);
  a.part_cnt = reinterpret_cast<int32_t*>(b + W.part_cnt);
  a.part_z = reinterpret_cast<float*>(b + W.part_z);
  a.part_n = reinterpret_cast<int32_t*>(b + W.part_n);
  a.T = D.T; a.ld = D.ld_logits; a.E = D.E; a.k = D.k;
  a.balance_coef = D.balance_coef; a.z_coef = D.z_coef;
  const unsigned grid = static_cast<unsigned>(balance_blocks(D));
  a.blocks = static_cast<int>(grid);
  const int vec = vec4(logits, a.ld, a.E);
  cudaError_t e = cudaSuccess;
  {
    ProfScope prof("router_balance", st);
    by_width(D.E, [&](auto L, auto NJ) {
      constexpr int l = decltype(L)::value, nj = decltype(NJ)::value;
      const bool few = grid == 1 && D.T <= 8 * (kFewThreads / l);
      auto kern = few ? balance_fwd_kernel<kFewThreads, l, nj> : balance_fwd_kernel<kManyThreads, l, nj>;
      const int th = few ? kFewThreads : kManyThreads;
      const int smem = th * nj * 16;
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e == cudaSuccess) e = launch_dependent(kern, dim3(grid), dim3(th), smem, st, a, vec);
    });
    count_launch();
  }
  if (e != cudaSuccess) return e;
  if (grid > 1) {
    ProfScope prof("router_balance_sum", st);
    e = launch_dependent(balance_sum_kernel, dim3(1), dim3(kManyThreads), 0, st, a);
    count_launch();
  }
  return e != cudaSuccess ? e : cudaGetLastError();
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
  const int64_t round = bwd_unroll((D.E + 127) / 128) * (kBwdThreads / lanes_of(D.E));
  const int64_t need = (D.T + round - 1) / round;
  const int64_t cap = 4LL * num_sms_current_device();
  const unsigned grid = static_cast<unsigned>(need < cap ? need : cap);
  const int vec = vec4(logits, a.ld, a.E) && vec4(dlogits, a.ld, a.E);
  ProfScope prof("router_balance_bwd", st);
  cudaError_t e = cudaSuccess;
  by_width(D.E, [&](auto L, auto NJ) {
    e = launch_dependent(balance_bwd_kernel<decltype(L)::value, decltype(NJ)::value>, dim3(grid),
                         dim3(kBwdThreads), 0, st, a, vec);
  });
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace mok
