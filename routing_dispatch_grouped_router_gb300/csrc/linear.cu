// Dense product with bias, activation and residual in its epilogue:
//   z = x w^T + bias,  y = act(z) + residual
// on tcgen05, for few tokens and for shapes the persistent engine does not
// take.
//
// The tokens are the narrow operand here: a tile is 128 rows of w (the MMA's
// M) by BN tokens (its N), so one token costs 16 MMA columns and the ring in
// shared memory is spent on the weights, whose bytes bound the call.  When the
// tiles do not fill the GPU, a cluster of up to 8 CTAs splits K: each leaves
// its fp32 partial in its own shared memory and takes a share of the tokens,
// which it sums over the cluster in rank order, so the result does not depend
// on timing.  (128 tokens, 2048 x 7168: 14.7 us; 7168 x 2048: 15.1.)
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "act.cuh"
#include "mok_internal.h"
#include "ptx.cuh"

namespace mok {

namespace {

// (These kernels may start before the one in front of them on the stream has
// ended, so they read with plain loads, after grid_dep_wait: the non-coherent
// path is for memory that nothing writes while a kernel lives.)
constexpr int kFewTokens = 8;
constexpr int kMaxSplits = 8;  // CTAs of a portable cluster
constexpr int kLinThreads = 192;  // TMA warp, MMA warp, four epilogue warps

template <int BN>
struct LinCfg {
  static constexpr int A_BYTES = 128 * 64 * 2;
  static constexpr int B_BYTES = BN * 64 * 2;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  // two CTAs per SM, so that a cluster's CTAs find room (with one CTA of 220 KB
  // per SM, 16 clusters of 8 did not all fit at once: 22 us instead of 13.5)
  static constexpr int ROOM = 108 * 1024;
  static constexpr int STAGES = ROOM / STAGE_BYTES;
  static constexpr int BAR_OFF = STAGES * STAGE_BYTES;
  static constexpr int SMEM_BYTES = 1024 + BAR_OFF + 256;
  static constexpr int ACC_COLS = BN;  // two accumulators
  static constexpr int TMEM_COLS = 2 * BN;
  static_assert(BN * 128 * 4 <= BAR_OFF, "the partial sums fit the operand ring");
  static_assert(SMEM_BYTES <= 232448 / 2 && STAGES >= 3 && (2 * STAGES + 4) * 8 + 8 <= 256, "smem");
};

struct LinArgs {
  const float* bias;
  const void* res;
  void *y, *z;
  int M, N, nkb, act;
  int chunk_kb;  // K blocks of one accumulation on the tensor cores
  int vec;       // rows of y, z, res and the bias take four elements at a time
  int* status;
};

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));
  return v;
}

template <bool F32>
__device__ __forceinline__ void load4(const void* p, long long o, float (&v)[4]) {
  if (F32) {
    const float4 t = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + o);
    v[0] = t.x; v[1] = t.y; v[2] = t.z; v[3] = t.w;
  } else {
    const uint2 t = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p) + o);
    v[0] = bf16lo(t.x); v[1] = bf16hi(t.x); v[2] = bf16lo(t.y); v[3] = bf16hi(t.y);
  }
}

template <bool F32>
__device__ __forceinline__ void store4(void* p, long long o, const float (&v)[4]) {
  if (F32)
    *reinterpret_cast<float4*>(static_cast<float*>(p) + o) = make_float4(v[0], v[1], v[2], v[3]);
  else
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p) + o) =
        make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}

template <bool F32>
__device__ __forceinline__ float load1(const void* p, long long o) {
  return F32 ? static_cast<const float*>(p)[o]
             : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[o]);
}
template <bool F32>
__device__ __forceinline__ void store1(void* p, long long o, float v) {
  if (F32) static_cast<float*>(p)[o] = v;
  else static_cast<__nv_bfloat16*>(p)[o] = __float2bfloat16_rn(v);
}

// The bias of features n .. n+3, and the residual of token m there (zeros where
// there is none).
__device__ __forceinline__ void bias4(const LinArgs& a, int n, float (&t)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) t[j] = 0.f;
  if (!a.bias || n >= a.N) return;
  if (a.vec) {
    load4<true>(a.bias, n, t);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (n + j < a.N) t[j] = a.bias[n + j];
  }
}
template <bool F32>
__device__ __forceinline__ void res4(const LinArgs& a, long long m, int n, float (&t)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) t[j] = 0.f;
  if (!a.res || n >= a.N) return;
  const long long o = m * a.N + n;
  if (a.vec) {
    load4<F32>(a.res, o, t);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (n + j < a.N) t[j] = load1<F32>(a.res, o + j);
  }
}

// Features n .. n+3 of token m from their sums, with their bias and residual
// (loaded beforehand: the stores here would hold the loads of the next back).
template <bool F32>
__device__ __forceinline__ void finish4(const LinArgs& a, long long m, int n, float (&v)[4],
                                        const float (&bias)[4], const float (&res)[4]) {
  if (n >= a.N) return;
  const long long o = m * a.N + n;
  float y[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[j] += bias[j];
    y[j] = act_value(v[j], a.act) + res[j];
  }
  if (a.vec) {
    if (a.z) store4<F32>(a.z, o, v);
    store4<F32>(a.y, o, y);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (n + j >= a.N) break;
      if (a.z) store1<F32>(a.z, o + j, v[j]);
      store1<F32>(a.y, o + j, y[j]);
    }
  }
}

// One output element (token m, feature n) from its sum.
template <bool F32>
__device__ __forceinline__ void finish1(const LinArgs& a, long long m, int n, float v) {
  const long long o = m * a.N + n;
  if (a.bias) v += a.bias[n];
  if (a.z) store1<F32>(a.z, o, v);
  v = act_value(v, a.act);
  if (a.res) v += load1<F32>(a.res, o);
  store1<F32>(a.y, o, v);
}

// Up to MT tokens, on the CUDA cores: bound by the bytes of w, which each
// thread streams with 16-byte loads, sixteen of them in flight; no ring, tensor
// memory or cluster to set up (one token, N = 2048, K = 7168: 13.5 us on the
// tensor cores, 5.9 here).  A warp takes R rows of w and goes round the
// 256-value chunks of K, a lane eight values of each; `wk` of the block's eight
// warps share K (a power of two), the others take further rows.  The sums are
// the lanes' (shuffles), then the wk warps' in order.
constexpr int kFewThreads = 256;
template <int MT, int R, int wk, bool F32>
__global__ void __launch_bounds__(kFewThreads)
    linear_few_kernel(const __nv_bfloat16* x, long long ld_x, const __nv_bfloat16* w, int K,
                      LinArgs a) {
  constexpr int U = 16 / R;  // chunks in flight
  __shared__ float s_sum[8][R * MT];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int kw = warp & (wk - 1), rw = warp / wk;  // share of K, row group
  const int n0 = (blockIdx.x * (8 / wk) + rw) * R;
  grid_dep_launch();
  grid_dep_wait();
  float acc[R][MT];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[r][m] = 0.f;
  constexpr int step = wk * 256;
  for (int c0 = kw * 256 + lane * 8; c0 < K; c0 += step * U) {
    uint4 wv[U][R];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = c0 + u * step;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        wv[u][r] = make_uint4(0u, 0u, 0u, 0u);
        if (k < K && n0 + r < a.N)
          wv[u][r] = *reinterpret_cast<const uint4*>(w + static_cast<long long>(n0 + r) * K + k);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = c0 + u * step;
      if (k >= K) break;
      float xf[MT][8];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        uint4 t = make_uint4(0u, 0u, 0u, 0u);
        if (m < a.M) t = *reinterpret_cast<const uint4*>(x + m * ld_x + k);
        xf[m][0] = bf16lo(t.x); xf[m][1] = bf16hi(t.x); xf[m][2] = bf16lo(t.y);
        xf[m][3] = bf16hi(t.y); xf[m][4] = bf16lo(t.z); xf[m][5] = bf16hi(t.z);
        xf[m][6] = bf16lo(t.w); xf[m][7] = bf16hi(t.w);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const uint4 t = wv[u][r];
        const float wf[8] = {bf16lo(t.x), bf16hi(t.x), bf16lo(t.y), bf16hi(t.y),
                             bf16lo(t.z), bf16hi(t.z), bf16lo(t.w), bf16hi(t.w)};
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[r][m] = fmaf(wf[j], xf[m][j], acc[r][m]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      float v = acc[r][m];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane == 0) s_sum[warp][m * R + r] = v;
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 8 / wk * R * MT; i += kFewThreads) {
    const int g = i / (R * MT), o = i % (R * MT);  // row group, element
    const int m = o / R, n = (blockIdx.x * (8 / wk) + g) * R + o % R;
    float v = 0.f;
#pragma unroll
    for (int q = 0; q < wk; ++q) v += s_sum[g * wk + q][o];
    if (m < a.M && n < a.N) finish1<F32>(a, m, n, v);
  }
}

// grid (feature tiles x K splits, a tile's splits being its cluster; token tiles)
template <int BN, bool F32, int KS>
__global__ void __launch_bounds__(kLinThreads)
    linear_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                  const LinArgs args) {
  using C = LinCfg<BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
  uint64_t* empty = full + C::STAGES;
  uint64_t* tfull = empty + C::STAGES;  // accumulators written (two)
  uint64_t* tempty = tfull + 2;         // accumulators read by the four epilogue warps
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tempty + 2);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int ks = KS;  // the cluster
  const int split = blockIdx.x % ks;
  const int n0 = blockIdx.x / ks * 128, m0 = blockIdx.y * BN;
  const int kb0 = static_cast<int>(static_cast<long long>(args.nkb) * split / ks);
  const int kb1 = static_cast<int>(static_cast<long long>(args.nkb) * (split + 1) / ks);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 4);
    }
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  grid_dep_wait();
  grid_dep_launch();
  const uint32_t tmem = *tmem_slot;
  volatile int* vabort = abort_flag;
  bool ok = true;

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int issued = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(&empty[stage], phase ^ 1u, vabort)) {
          ok = false;
          break;
        }
        uint8_t* sW = smem + stage * C::STAGE_BYTES;
        mbar_arrive_expect_tx(&full[stage], C::STAGE_BYTES);
        tma_load_2d(sW, &tmW, &full[stage], kb * 64, n0);
        tma_load_2d(sW + C::A_BYTES, &tmX, &full[stage], kb * 64, m0);
        ++issued;
        if (++stage == C::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) {
        *vabort = 1;
        set_status(args.status, MOK_ERR_DEVICE_TIMEOUT);
        // copies already issued land before the CTA can exit: the last fill
        // of each stage
        const int zero = 0;
        for (int s = 0; s < C::STAGES && s < issued; ++s) {
          const int fills = (issued - 1 - s) / C::STAGES;
          mbar_wait(&full[s], static_cast<uint32_t>(fills & 1), &zero);
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_bf16_f32(128, BN, false, false);
      int stage = 0;
      uint32_t phase = 0;
      int it = 0;
      for (int c0 = kb0; c0 < kb1 && ok; c0 += args.chunk_kb, ++it) {
        const int acc = it & 1;
        const uint32_t par = static_cast<uint32_t>((it >> 1) & 1);
        if (!mbar_wait(&tempty[acc], par ^ 1u, vabort)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const int c1 = c0 + args.chunk_kb < kb1 ? c0 + args.chunk_kb : kb1;
        for (int kb = c0; kb < c1; ++kb) {
          if (!mbar_wait(&full[stage], phase, vabort)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t a_base = smem_addr(smem + stage * C::STAGE_BYTES);
          const uint32_t b_base = a_base + C::A_BYTES;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma_bf16(tmem + acc * C::ACC_COLS, smem_desc_sw128(a_base + j * 32, 16, 1024),
                     smem_desc_sw128(b_base + j * 32, 16, 1024), idesc,
                     (kb > c0 || j > 0) ? 1u : 0u);
          mma_commit(&empty[stage]);
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        mma_commit(&tfull[acc]);
      }
      if (!ok) {
        // the MMAs issued are done before TMEM is freed: the last commit above
        *vabort = 1;
        set_status(args.status, MOK_ERR_DEVICE_TIMEOUT);
        const int zero = 0;
        if (it > 0) mbar_wait(&tfull[(it - 1) & 1], static_cast<uint32_t>(((it - 1) >> 1) & 1), &zero);
      }
    }
  } else {
    // ---- the chunks' sums: lane f of the tile's 128 features, BN tokens ----
    const int q = warp & 3;  // TMEM lane quarter this warp may read
    const int f = q * 32 + lane;
    float sum[BN];
#pragma unroll
    for (int j = 0; j < BN; ++j) sum[j] = 0.f;
    int it = 0;
    for (int c0 = kb0; c0 < kb1; c0 += args.chunk_kb, ++it) {
      const int acc = it & 1;
      ok = __all_sync(0xffffffffu,
                      mbar_wait(&tfull[acc], static_cast<uint32_t>((it >> 1) & 1), vabort));
      if (!ok) {
        *vabort = 1;
        set_status(args.status, MOK_ERR_DEVICE_TIMEOUT);
        break;
      }
      tc_fence_after_sync();
#pragma unroll
      for (int c = 0; c < BN; c += 16) {
        if (m0 + c < args.M) {
          uint32_t r[16];
          tmem_ld16(tmem + (static_cast<uint32_t>(q * 32) << 16) + acc * C::ACC_COLS + c, r);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) sum[c + j] += __uint_as_float(r[j]);
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[acc]);
    }
    // every MMA has read its operands (the last chunk is complete), so the
    // sums take the ring's place: [BN tokens][128 features]
    float* part = reinterpret_cast<float*>(smem);
    if (ok) {
#pragma unroll
      for (int j = 0; j < BN; ++j)
        if (m0 + j < args.M) part[j * 128 + f] = sum[j];
    }
  }
  __syncwarp();
  if (ks > 1) cluster_sync(); else __syncthreads();
  // this CTA's share of the tokens, four features per thread, the cluster's
  // sums in rank order; the remote loads of several elements go out together
  // (their latency is most of a small call's epilogue)
  if (!*vabort) {
    const uint32_t part = smem_addr(smem) + lane * 16u;
    const int n = n0 + 4 * lane;
    float bias[4];
    bias4(args, n, bias);
    const int tokens = args.M - m0 < BN ? args.M - m0 : BN;
    constexpr int B = KS >= 8 ? 2 : (KS == 4 ? 4 : 8);  // a warp's tokens at a time
    constexpr int kStep = ks * (kLinThreads / 32);
    for (int t0 = split + ks * warp; t0 < tokens; t0 += B * kStep) {
      float4 p[B][KS];
      float res[B][4];
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const int m = t0 + b * kStep;
        if (m >= tokens || n >= args.N) break;
        res4<F32>(args, m0 + m, n, res[b]);
#pragma unroll
        for (int r = 0; r < KS; ++r)
          p[b][r] = KS == 1 ? *reinterpret_cast<const float4*>(smem + (m * 128 + 4 * lane) * 4)
                            : ld_cluster_f4(mapa_shared(part + static_cast<uint32_t>(m) * 512u, r));
      }
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const int m = t0 + b * kStep;
        if (m >= tokens || n >= args.N) break;
        float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int r = 0; r < KS; ++r) {
          v[0] += p[b][r].x; v[1] += p[b][r].y; v[2] += p[b][r].z; v[3] += p[b][r].w;
        }
        finish4<F32>(args, m0 + m, n, v, bias, res[b]);
      }
    }
  }
  __syncwarp();
  tc_fence_before_sync();
  // no CTA leaves while another reads its sums
  if (ks > 1) cluster_sync(); else __syncthreads();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

template <int BN, bool F32>
cudaError_t run_linear(const mok_linear_desc& D, const void* x, const void* w, const LinArgs& a,
                       cudaStream_t st) {
  using C = LinCfg<BN>;
  CUtensorMap tw, tx;
  const auto bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const auto sw = CU_TENSOR_MAP_SWIZZLE_128B;
  if (!make_tensor_map_2d(&tw, bf, 2, w, D.K, D.N, D.K, 64, 128, sw) ||
      !make_tensor_map_2d(&tx, bf, 2, x, D.K, D.M, D.ld_x, 64, BN, sw))
    return cudaErrorInvalidValue;
  const int64_t nt = (D.N + 127) / 128, mt = (D.M + BN - 1) / BN;
  // K splits: a power of two, as many as the CTAs that fit at once leave room
  // for, at least four 64-value blocks each
  constexpr int64_t slots = 2 * kGb300Sms;
  int ks = 1;
  while (ks < kMaxSplits && nt * mt * ks * 2 <= slots && a.nkb >= ks * 8) ks *= 2;
  auto kern = ks == 1   ? linear_kernel<BN, F32, 1>
              : ks == 2 ? linear_kernel<BN, F32, 2>
              : ks == 4 ? linear_kernel<BN, F32, 4>
                        : linear_kernel<BN, F32, 8>;
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(ks);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(ks * nt), static_cast<unsigned>(mt));
  cfg.blockDim = dim3(kLinThreads, 1, 1);
  cfg.dynamicSmemBytes = C::SMEM_BYTES;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  ProfScope prof("linear", st);
  e = cudaLaunchKernelEx(&cfg, kern, tw, tx, a);
  count_launch();
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

// Split products: y = act(sum of the parts + bias) + residual, part s from float4
// s * stride of `part` (row stride N rounded up to 4), added in order.
template <bool F32>
__global__ void __launch_bounds__(256) linear_finish_kernel(LinArgs a, const float* part,
                                                            int splits, long long stride) {
  grid_dep_launch();
  grid_dep_wait();
  const int n4 = (a.N + 3) / 4;
  const long long items = static_cast<long long>(a.M) * n4;
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < items; i += gridDim.x * 256LL) {
    const float4* p = reinterpret_cast<const float4*>(part) + i;
    const long long m = i / n4;
    const int n = static_cast<int>(i - m * n4) * 4;
    float v[4] = {0.f, 0.f, 0.f, 0.f}, bias[4], res[4];
    bias4(a, n, bias);
    res4<F32>(a, m, n, res);
#pragma unroll 4
    for (int s = 0; s < splits; ++s) {
      const float4 t = p[s * stride];
      v[0] += t.x; v[1] += t.y; v[2] += t.z; v[3] += t.w;
    }
    finish4<F32>(a, m, n, v, bias, res);
  }
}

// (rows: of a part)
cudaError_t launch_finish(const LinArgs& a, const float* part, int splits, int64_t rows, bool f32,
                          cudaStream_t st) {
  const long long n4 = (a.N + 3) / 4, items = a.M * n4, stride = rows * n4;
  long long blocks = (items + 255) / 256;
  const long long cap = 8LL * num_sms_current_device();
  if (blocks > cap) blocks = cap;
  ProfScope prof("linear_finish", st);
  const cudaError_t e =
      launch_dependent(f32 ? linear_finish_kernel<true> : linear_finish_kernel<false>,
                       dim3(static_cast<unsigned>(blocks)), dim3(256), 0, st, a, part, splits,
                       stride);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

// Shapes for the persistent engine: more than one 128-row tile of tokens.
bool engine_takes(const mok_linear_desc& D) { return D.M > 128; }

// Splits of a reduction of nkb 64-value blocks, A in `parts`, over the CTAs (or
// CTA pairs) that `tiles` of `slots` leave: those of the least time by what was
// measured, 260 ns a block on the tensor cores, 1.5 us or more for an epilogue on
// the tiles' SMs alone, 2 us for the kernel that adds the partial results of `elems`
// values, and their bytes at 5 TB/s.  (12 tokens, N = 1968, K = 368, two parts: dx
// 24.7 us unsplit, 12 so; 772 tokens, N = 9: dw 21 and 13; 226 x 2275 x 904, fp32:
// 23.1 and 13.4; 8331 tokens, K = 200: two splits' bytes would cost dx 2 us more
// than they save.)
int best_splits(int64_t tiles, int64_t slots, int64_t nkb, int parts, int64_t elems,
                int most) {
  int best = 1;
  int64_t least = nkb * parts * 260 + 1500;
  for (int64_t ks = 2; ks <= slots / tiles && ks <= nkb && ks <= most; ++ks) {
    const int64_t kb = (nkb + ks - 1) / ks;
    const int64_t t = kb * parts * 260 + 2000 + (ks + 1) * elems * 4 / 5000;
    if (t >= least || (nkb + kb - 1) / kb != ks) continue;  // (no empty split)
    least = t;
    best = static_cast<int>(ks);
  }
  return best;
}

// K splits of an engine product C [M, N], reduction K: the tiles' CTAs or CTA
// pairs are those of a GB300 (152, 76), whatever the device, so that sums do not
// depend on it.
int engine_splits(int64_t M, int64_t N, int64_t K, int parts) {
  const int64_t rows = M > 128 ? 256 : 128, cols = M > 128 || parts < 3 ? 256 : 128;
  const int64_t tiles = ((M + rows - 1) / rows) * ((N + cols - 1) / cols);
  return best_splits(tiles, M > 128 ? kGb300Sms / 2 : kGb300Sms, (K + 63) / 64, parts, M * N,
                     16);
}

size_t part_bytes(int splits, int64_t M, int64_t N) {
  return splits > 1 ? static_cast<size_t>(splits) * ((M + 127) / 128 * 128) * ((N + 3) / 4) * 16
                    : 0;
}

}  // namespace

size_t linear_fwd_bytes(const mok_linear_desc& D) {
  return engine_takes(D) ? part_bytes(engine_splits(D.M, D.N, D.K, 1), D.M, D.N) : 0;
}

cudaError_t launch_linear(const mok_linear_desc& D, const void* x, const void* w,
                          const float* bias, const void* res, void* y, void* z, void* ws,
                          int* status, cudaStream_t st) {
  if (D.M == 0) return cudaSuccess;
  LinArgs a;
  a.bias = bias; a.res = res; a.y = y; a.z = z;
  a.M = static_cast<int>(D.M);
  a.N = static_cast<int>(D.N);
  a.nkb = static_cast<int>((D.K + 63) / 64);
  a.act = D.act;
  a.status = status;
  const bool f32 = D.y_elem == MOK_ELEM_F32;
  // an fp32 result: at most 36 MMAs (9 blocks) in one accumulation, as in the
  // persistent engine; a bf16 one hides what the accumulation truncates
  a.chunk_kb = f32 ? 9 : a.nkb;
  const uintptr_t bits = reinterpret_cast<uintptr_t>(bias) | reinterpret_cast<uintptr_t>(res) |
                         reinterpret_cast<uintptr_t>(y) | reinterpret_cast<uintptr_t>(z);
  a.vec = D.N % 4 == 0 && (bits & 15) == 0;
  if (engine_takes(D)) {
    const int splits = engine_splits(D.M, D.N, D.K, 1);
    const bool direct = D.N % 8 != 0 || (bits & 15) != 0;
    if (splits == 1)
      return gemm_linear_fwd(D.M, D.N, D.K, D.ld_x, x, w, bias, res, D.act, y, z, f32, direct,
                             status, st);
    float* part = static_cast<float*>(ws);
    const cudaError_t e =
        gemm_linear_part(D.M, D.N, D.K, D.ld_x, x, w, part, splits, status, st);
    if (e != cudaSuccess) return e;
    return launch_finish(a, part, splits, (D.M + 127) / 128 * 128, f32, st);
  }
  // few tokens: on the CUDA cores while their products (M N K) do not take
  // longer than the tensor-core kernel's setup (measured even at 6e7: M = 4,
  // N = 2048, K = 7168, both 9 us; M = 8: 15 against 9)
  if (D.M <= 2 || (D.M <= kFewTokens && D.M * D.N * D.K <= 50000000)) {
    ProfScope prof("linear_few", st);
    const auto* xb = static_cast<const __nv_bfloat16*>(x);
    const auto* wb = static_cast<const __nv_bfloat16*>(w);
    const int K = static_cast<int>(D.K);
    cudaError_t e = cudaSuccess;
    // warps along K while each has its chunks in flight full, or while the rows
    // alone would leave SMs idle
    auto launch = [&](auto MT, auto WK, auto F) {
      constexpr int wk = decltype(WK)::value, rows = 4 * (8 / wk);
      e = launch_dependent(linear_few_kernel<decltype(MT)::value, 4, wk, decltype(F)::value>,
                           dim3(static_cast<unsigned>((D.N + rows - 1) / rows)),
                           dim3(kFewThreads), 0, st, xb, D.ld_x, wb, K, a);
    };
    auto run = [&](auto MT, auto F) {
      using std::integral_constant;
      constexpr int64_t many = 2 * kGb300Sms;
      if (K <= 2048 && D.N >= 16 * many) launch(MT, integral_constant<int, 2>(), F);
      else if (K <= 4096 && D.N >= 8 * many) launch(MT, integral_constant<int, 4>(), F);
      else launch(MT, integral_constant<int, 8>(), F);
    };
    auto by_tokens = [&](auto F) {
      using std::integral_constant;
      if (D.M == 1) run(integral_constant<int, 1>(), F);
      else if (D.M == 2) run(integral_constant<int, 2>(), F);
      else if (D.M <= 4) run(integral_constant<int, 4>(), F);
      else run(integral_constant<int, 8>(), F);
    };
    if (f32) by_tokens(std::true_type());
    else by_tokens(std::false_type());
    count_launch();
    return e != cudaSuccess ? e : cudaGetLastError();
  }
  if (D.M <= 16) return f32 ? run_linear<16, true>(D, x, w, a, st) : run_linear<16, false>(D, x, w, a, st);
  if (D.M <= 64) return f32 ? run_linear<64, true>(D, x, w, a, st) : run_linear<64, false>(D, x, w, a, st);
  return f32 ? run_linear<128, true>(D, x, w, a, st) : run_linear<128, false>(D, x, w, a, st);
}

// ----------------------------------------------------------------- backward --

namespace {

struct DzArgs {
  const void *dy, *z;
  __nv_bfloat16* dz[3];    // parts [M, n_pad], zero past N (NULL: not stored)
  float* part;             // [ceil(M / kDzRows), N] column sums (NULL: none)
  long long M;
  int N, n_pad;
};

constexpr int kDzRows = 32;  // rows of a block

// Eight consecutive elements of row r from column c.
template <bool F32, bool VEC>
struct Dz8 {
  float f[8];
  __device__ __forceinline__ void load(const void* base, long long r, int c, int N) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = 0.f;
    if (VEC) {
      if (c >= N) return;
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + r * N + c);
      const float4 x = p[0], y = p[1];
      f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w;
      f[4] = y.x; f[5] = y.y; f[6] = y.z; f[7] = y.w;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + j < N) f[j] = load1<F32>(base, r * N + c + j);
    }
  }
  __device__ __forceinline__ void get(float (&o)[8]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = f[j];
  }
};
template <>
struct Dz8<false, true> {
  uint4 u;
  __device__ __forceinline__ void load(const void* base, long long r, int c, int N) {
    u = make_uint4(0u, 0u, 0u, 0u);
    if (c < N)
      u = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + r * N + c);
  }
  __device__ __forceinline__ void get(float (&o)[8]) const {
    o[0] = bf16lo(u.x); o[1] = bf16hi(u.x); o[2] = bf16lo(u.y); o[3] = bf16hi(u.y);
    o[4] = bf16lo(u.z); o[5] = bf16hi(u.z); o[6] = bf16lo(u.w); o[7] = bf16hi(u.w);
  }
};

// Bound by its bytes (4096 x 1024, silu, three parts: 42 MB, 11.8 us with cold
// caches and alone on the GPU):
// dz = dy act'(z) as the sum of bf16 parts (each the rounding of what those
// before it leave), and its column sums over the block's rows.  A block takes
// kDzRows rows by 8 * `lanes` columns, a lane 8 columns of every 256/lanes-th
// row, in batches of four rows whose loads are in flight together.  The blocks of
// a grid of one dimension go round the `cols` column blocks first (two million
// tokens are more row blocks than a second dimension holds).
template <bool F32, bool VEC, int ACT>
__global__ void __launch_bounds__(256) linear_dz_kernel(DzArgs a, int lanes, int cols) {
  __shared__ float s_sum[256 * 9];
  grid_dep_launch();
  grid_dep_wait();
  const int l = threadIdx.x & (lanes - 1), row0 = threadIdx.x / lanes, rows = 256 / lanes;
  const int col_block = blockIdx.x % cols;
  const long long row_block = blockIdx.x / cols;
  const int c = (col_block * lanes + l) * 8;
  const long long r0 = row_block * kDzRows;
  float sum[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) sum[j] = 0.f;
  if (c < a.n_pad) {
    for (int i0 = row0; i0 < kDzRows; i0 += 4 * rows) {
      Dz8<F32, VEC> dy[4], z[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = i0 + i * rows;
        if (row < kDzRows && r0 + row < a.M) {
          dy[i].load(a.dy, r0 + row, c, a.N);
          if (ACT != MOK_ACT_NONE) z[i].load(a.z, r0 + row, c, a.N);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = i0 + i * rows;
        if (row >= kDzRows || r0 + row >= a.M) break;
        // (past N dy and z are zeros, and so is dz)
        float v[8], zz[8];
        dy[i].get(v);
        if (ACT != MOK_ACT_NONE) z[i].get(zz);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (ACT != MOK_ACT_NONE) v[j] *= act_slope(zz[j], ACT);
          sum[j] += v[j];
        }
#pragma unroll
        for (int p = 0; p < 3; ++p) {
          if (!a.dz[p]) break;
          uint32_t h[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            h[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
            v[2 * j] -= bf16lo(h[j]);
            v[2 * j + 1] -= bf16hi(h[j]);
          }
          st_global_v4(a.dz[p] + (r0 + row) * a.n_pad + c, make_uint4(h[0], h[1], h[2], h[3]));
          if (p == 0) {
            // a value that is infinite (or NaN) in the first part leaves nothing:
            // inf - inf would make the sum of the parts NaN
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = fabsf(v[j]) < INFINITY ? v[j] : 0.f;
          }
        }
      }
    }
  }
  if (!a.part) return;
  // the row groups' sums of a column in order
#pragma unroll
  for (int j = 0; j < 8; ++j) s_sum[(row0 * lanes + l) * 9 + j] = sum[j];
  __syncthreads();
  for (int i = threadIdx.x; i < lanes * 8; i += 256) {
    const int col = col_block * lanes * 8 + i;
    if (col >= a.N) break;
    float t = 0.f;
    for (int r = 0; r < rows; ++r) t += s_sum[(r * lanes + (i >> 3)) * 9 + (i & 7)];
    a.part[row_block * a.N + col] = t;
  }
}

// dw[i] (+)= sum over s < n of part[s * stride4 + i], float4s, in order
__global__ void __launch_bounds__(256) split_sum_kernel(const float4* part, int n,
                                                        long long stride4, long long n4,
                                                        float4* dw, int accumulate) {
  grid_dep_launch();
  grid_dep_wait();
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < n4; i += gridDim.x * 256LL) {
    float4 v = part[i];
#pragma unroll 8
    for (int s = 1; s < n; ++s) {
      const float4 p = part[s * stride4 + i];
      v.x += p.x; v.y += p.y; v.z += p.z; v.w += p.w;
    }
    if (accumulate) {
      const float4 p = dw[i];
      v.x += p.x; v.y += p.y; v.z += p.z; v.w += p.w;
    }
    dw[i] = v;
  }
}

// The parts of dz that a product with a result of fp32 (or bf16) takes.  A bf16
// dy without an activation is dz; else an fp32 result takes all 24 bits in three
// parts (16 bits of two parts leave it 2.4e-6 off, the fp32 sums 5e-7), a bf16
// result two.
int dz_parts(const mok_linear_desc& D, bool f32) {
  return D.y_elem != MOK_ELEM_F32 && D.act == MOK_ACT_NONE ? 1 : (f32 ? 3 : 2);
}

// ... of the weight gradient (over the tokens).
int dw_splits(const mok_linear_desc& D) {
  const int64_t mt = (D.N + 127) / 128;
  const int64_t tiles = (mt + 1) / 2 * ((D.K + 255) / 256);
  return best_splits(tiles, mt > 1 ? kGb300Sms / 2 : kGb300Sms, (D.M + 63) / 64, dz_parts(D, true), D.N * D.K,
                     32);
}

// Up to kFewTokens tokens, on the CUDA cores: dz, dbias, dx and dw in one pass
// over w and dw, whose bytes bound it.  A block takes 128 columns of K (a lane
// four) and a slice of the rows n, which its warps share: per row a lane has
// dz[m][n] (fp32, shared memory) for dw[n] = sum_m dz[m][n] x[m], stored at
// once, and for its sums dx[m] += dz[m][n] w[n].  The warps' sums are added in
// order; where there are several slices, a second kernel adds theirs.  (One token,
// N = 2048, K = 7168: 17.3 us, floor 13.0; N = 6351, K = 6072: two tokens 47 us,
// eight 66, 72 by the tensor cores in six launches; floor 34; one token, N = 37,
// K = 2520: 2.6 and 13.  At eight tokens the products on the CUDA cores show.)
constexpr int kFewDz = 512;  // rows whose dz a block holds
struct FewBwd {
  const void *dy, *z;
  const __nv_bfloat16 *x, *w;
  void* dx;      // (NULL: not wanted; so dw and dbias)
  float *dw, *dbias;
  float* part;   // [slices, M, K], several slices
  long long ld_x;
  int M, N, K, rows, act;  // rows: of a slice
  bool dx_f32, add_dx;
};

template <int MT, bool F32, bool ADD>
__global__ void __launch_bounds__(kFewThreads, 2) linear_bwd_few_kernel(FewBwd a) {
  constexpr int U = ADD ? 4 : 8;  // rows of a warp in flight
  constexpr int kWarps = kFewThreads / 32;
  union Shared {
    float dz[kFewDz][MT];
    float4 dx[kWarps][MT][32];
  };
  __shared__ __align__(16) Shared s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = (blockIdx.x * 32 + lane) * 4;
  const bool in = c < a.K;
  const int n0 = blockIdx.y * a.rows, n1 = n0 + a.rows < a.N ? n0 + a.rows : a.N;
  grid_dep_launch();
  grid_dep_wait();
  float xf[MT][4], acc[MT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
#pragma unroll
    for (int j = 0; j < 4; ++j) xf[m][j] = acc[m][j] = 0.f;
    if (in && a.dw && m < a.M) load4<false>(a.x, m * a.ld_x + c, xf[m]);
  }
  for (int t0 = n0; t0 < n1; t0 += kFewDz) {
    const int cnt = n1 - t0 < kFewDz ? n1 - t0 : kFewDz;
    __syncthreads();  // the rows before have been used
    for (int i = threadIdx.x; i < cnt; i += kFewThreads) {
      float d[MT], sum = 0.f;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const long long o = static_cast<long long>(m) * a.N + t0 + i;
        d[m] = m < a.M ? load1<F32>(a.dy, o) : 0.f;
        if (a.act != MOK_ACT_NONE && m < a.M) d[m] *= act_slope(load1<F32>(a.z, o), a.act);
        sum += d[m];
      }
#pragma unroll
      for (int m = 0; m < MT; m += 2)
        *reinterpret_cast<float2*>(&s.dz[i][m]) = make_float2(d[m], d[m + 1]);
      if (a.dbias && blockIdx.x == 0) a.dbias[t0 + i] = ADD ? a.dbias[t0 + i] + sum : sum;
    }
    __syncthreads();
    if (!in || (!a.dx && !a.dw)) continue;
    for (int i = warp; i < cnt; i += U * kWarps) {
      uint2 wv[U];
      float4 old[ADD ? U : 1];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int row = i + u * kWarps;
        const long long o = static_cast<long long>(t0 + row) * a.K + c;
        wv[u] = make_uint2(0u, 0u);
        if (a.dx && row < cnt) wv[u] = *reinterpret_cast<const uint2*>(a.w + o);
        if (ADD && a.dw && row < cnt) old[u] = *reinterpret_cast<const float4*>(a.dw + o);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int row = i + u * kWarps;
        if (row >= cnt) break;
        const float wf[4] = {bf16lo(wv[u].x), bf16hi(wv[u].x), bf16lo(wv[u].y), bf16hi(wv[u].y)};
        float v[4] = {0.f, 0.f, 0.f, 0.f}, dz[MT];
#pragma unroll
        for (int m = 0; m < MT; m += 2) {
          const float2 t = *reinterpret_cast<const float2*>(&s.dz[row][m]);
          dz[m] = t.x;
          dz[m + 1] = t.y;
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const float d = dz[m];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            v[j] = fmaf(d, xf[m][j], v[j]);
            acc[m][j] = fmaf(d, wf[j], acc[m][j]);
          }
        }
        if (ADD) {
          const float4 t = old[ADD ? u : 0];
          v[0] += t.x; v[1] += t.y; v[2] += t.z; v[3] += t.w;
        }
        if (a.dw) store4<true>(a.dw, static_cast<long long>(t0 + row) * a.K + c, v);
      }
    }
  }
  if (!a.dx) return;
  __syncthreads();
#pragma unroll
  for (int m = 0; m < MT; ++m)
    s.dx[warp][m][lane] = make_float4(acc[m][0], acc[m][1], acc[m][2], acc[m][3]);
  __syncthreads();
  for (int m = warp; m < a.M; m += kWarps) {
    if (!in) break;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int q = 0; q < kWarps; ++q) {
      const float4 t = s.dx[q][m][lane];
      v[0] += t.x; v[1] += t.y; v[2] += t.z; v[3] += t.w;
    }
    const long long o = static_cast<long long>(m) * a.K + c;
    if (gridDim.y > 1) {
      store4<true>(a.part, (static_cast<long long>(blockIdx.y) * a.M) * a.K + o, v);
    } else if (a.dx_f32) {
      float t[4] = {0.f, 0.f, 0.f, 0.f};
      if (a.add_dx) load4<true>(a.dx, o, t);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] += t[j];
      store4<true>(a.dx, o, v);
    } else {
      store4<false>(a.dx, o, v);
    }
  }
}

// Rows of a slice: two blocks per SM (of a GB300, whatever the device), at
// least eight rows per warp.
int64_t few_rows(const mok_linear_desc& D) {
  const int64_t cols = (D.K + 127) / 128;
  int64_t slices = 2 * kGb300Sms / cols;
  if (slices < 1) slices = 1;
  const int64_t rows = ((D.N + slices - 1) / slices + 7) / 8 * 8;
  return rows < 64 ? 64 : rows;
}

bool few_bwd(const mok_linear_desc& D) { return D.M <= kFewTokens; }

}  // namespace

bool linear_dz_is_dy(const mok_linear_desc& D, const void* dy) {
  return D.y_elem != MOK_ELEM_F32 && D.act == MOK_ACT_NONE && D.N % 8 == 0 &&
         (reinterpret_cast<uintptr_t>(dy) & 15) == 0;
}

void linear_layout(const mok_linear_desc& D, bool dz_is_dy, LinearWs* W) {
  auto al = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  if (few_bwd(D)) {
    *W = LinearWs{};
    const int64_t slices = (D.N + few_rows(D) - 1) / few_rows(D);
    W->total = slices > 1 ? al(static_cast<size_t>(slices) * D.M * D.K * 4) : 0;
    return;
  }
  W->n_pad = (D.N + 63) / 64 * 64;
  W->bias_rows = (D.M + kDzRows - 1) / kDzRows;
  W->dw_splits = dw_splits(D);
  // dz in as many parts as a product takes
  const size_t dz = al(static_cast<size_t>(D.M) * W->n_pad * 2);
  const int parts = dz_is_dy ? 0 : dz_parts(D, true);
  for (int p = 0; p < 3; ++p) W->dz[p] = p < parts ? p * dz : 0;
  W->part_bias = parts * dz;
  W->part_dw = W->part_bias + al(static_cast<size_t>(W->bias_rows) * D.N * 4);
  // partial products of dx, then of dw: one region
  W->dx_splits = engine_splits(D.M, D.K, W->n_pad, dz_parts(D, D.dx_elem == MOK_ELEM_F32));
  const size_t rows = static_cast<size_t>((D.N + 127) / 128 * 128);
  const size_t a = part_bytes(W->dx_splits, D.M, D.K);
  const size_t b = W->dw_splits > 1 ? W->dw_splits * rows * D.K * 4 : 0;
  W->total = W->part_dw + al(a > b ? a : b);
}

namespace {

cudaError_t launch_few_bwd(const mok_linear_desc& D, const void* dy, const void* x, const void* w,
                           const void* z, void* dx, float* dw, float* dbias, float* part,
                           cudaStream_t st) {
  FewBwd a;
  a.dy = dy; a.z = z;
  a.x = static_cast<const __nv_bfloat16*>(x);
  a.w = static_cast<const __nv_bfloat16*>(w);
  a.dx = dx; a.dw = dw; a.dbias = dbias; a.part = part;
  a.ld_x = D.ld_x;
  a.M = static_cast<int>(D.M); a.N = static_cast<int>(D.N); a.K = static_cast<int>(D.K);
  a.rows = static_cast<int>(few_rows(D));
  a.act = D.act;
  a.dx_f32 = D.dx_elem == MOK_ELEM_F32;
  a.add_dx = (D.accumulate & MOK_ADD_DX) != 0;
  const int64_t slices = (D.N + a.rows - 1) / a.rows;
  const int64_t cols = dx || dw ? (D.K + 127) / 128 : 1;
  cudaError_t e = cudaSuccess;
  {
    ProfScope prof("linear_bwd_few", st);
    auto run = [&](auto MT, auto F) {
      constexpr int mt = decltype(MT)::value;
      constexpr bool f32 = decltype(F)::value;
      e = launch_dependent((D.accumulate & MOK_ADD_DW) ? linear_bwd_few_kernel<mt, f32, true>
                                                       : linear_bwd_few_kernel<mt, f32, false>,
                           dim3(static_cast<unsigned>(cols), static_cast<unsigned>(slices)),
                           dim3(kFewThreads), 0, st, a);
    };
    auto by_tokens = [&](auto F) {
      using std::integral_constant;
      if (D.M <= 2) run(integral_constant<int, 2>(), F);
      else if (D.M <= 4) run(integral_constant<int, 4>(), F);
      else run(integral_constant<int, kFewTokens>(), F);
    };
    if (D.y_elem == MOK_ELEM_F32) by_tokens(std::true_type());
    else by_tokens(std::false_type());
    count_launch();
  }
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess || slices == 1 || !dx) return e;
  LinArgs f = {};
  f.y = dx;
  f.res = a.add_dx ? dx : nullptr;  // (fp32)
  f.M = a.M;
  f.N = a.K;
  f.act = MOK_ACT_NONE;
  f.vec = 1;
  return launch_finish(f, part, static_cast<int>(slices), D.M, a.dx_f32, st);
}

}  // namespace

cudaError_t launch_linear_bwd(const mok_linear_desc& D, const void* dy, const void* x,
                              const void* w, const void* z, void* dx, float* dw, float* dbias,
                              void* ws, int* status, cudaStream_t st) {
  // a bf16 dy without an activation is dz already
  const bool direct = linear_dz_is_dy(D, dy);
  LinearWs W;
  linear_layout(D, direct, &W);
  char* b = static_cast<char*>(ws);
  const bool f32 = D.y_elem == MOK_ELEM_F32;
  const bool add_dx = (D.accumulate & MOK_ADD_DX) != 0, add_dw = (D.accumulate & MOK_ADD_DW) != 0;
  const bool vec = D.N % 8 == 0 && ((reinterpret_cast<uintptr_t>(dy) | reinterpret_cast<uintptr_t>(z)) & 15) == 0;
  const bool dxf = D.dx_elem == MOK_ELEM_F32;
  const int parts = direct ? 0 : dz_parts(D, dw || dxf);
  const bool products = D.M > 0 && (dx || dw);
  if (D.M > 0 && few_bwd(D))
    return launch_few_bwd(D, dy, x, w, z, dx, dw, dbias, static_cast<float*>(ws), st);
  float* part_bias = reinterpret_cast<float*>(b + W.part_bias);
  if (D.M > 0 && ((products && !direct) || dbias)) {
    DzArgs a;
    a.dy = dy;
    a.z = z;
    for (int p = 0; p < 3; ++p)
      a.dz[p] = products && p < parts ? reinterpret_cast<__nv_bfloat16*>(b + W.dz[p]) : nullptr;
    a.part = dbias ? part_bias : nullptr;
    a.M = D.M;
    a.N = static_cast<int>(D.N);
    a.n_pad = static_cast<int>(W.n_pad);
    // lanes of a row: 8 columns each, up to a warp
    const int lanes = W.n_pad >= 256 ? 32 : (W.n_pad > 64 ? 16 : 8);
    const int64_t cols = (W.n_pad + lanes * 8 - 1) / (lanes * 8);
    const dim3 grid(static_cast<unsigned>(cols * W.bias_rows));
    ProfScope prof("linear_dz", st);
    cudaError_t e = cudaSuccess;
    auto run = [&](auto F, auto V, auto A) {
      e = launch_dependent(
          linear_dz_kernel<decltype(F)::value, decltype(V)::value, decltype(A)::value>, grid,
          dim3(256), 0, st, a, lanes, static_cast<int>(cols));
    };
    auto by_act = [&](auto F, auto V) {
      if (D.act == MOK_ACT_NONE) run(F, V, std::integral_constant<int, MOK_ACT_NONE>());
      else if (D.act == MOK_ACT_RELU) run(F, V, std::integral_constant<int, MOK_ACT_RELU>());
      else if (D.act == MOK_ACT_SILU) run(F, V, std::integral_constant<int, MOK_ACT_SILU>());
      else run(F, V, std::integral_constant<int, MOK_ACT_GELU>());
    };
    if (f32) vec ? by_act(std::true_type(), std::true_type()) : by_act(std::true_type(), std::false_type());
    else vec ? by_act(std::false_type(), std::true_type()) : by_act(std::false_type(), std::false_type());
    count_launch();
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (dbias) {
    const cudaError_t e = launch_column_sum(part_bias, W.bias_rows, D.N, dbias, add_dw, st);
    if (e != cudaSuccess) return e;
  }
  if (D.M == 0) {
    if (dw && !add_dw) return cudaMemsetAsync(dw, 0, static_cast<size_t>(D.N) * D.K * 4, st);
    return cudaSuccess;
  }
  BfParts dz;
  dz.n = dz_parts(D, true);
  dz.ld = direct ? D.N : W.n_pad;
  for (int p = 0; p < 3; ++p) dz.part[p] = b + W.dz[p];
  if (direct) dz.part[0] = dy;
  if (dx) {
    BfParts d = dz;
    d.n = dz_parts(D, dxf);
    const bool sum = W.dx_splits > 1;
    float* part = reinterpret_cast<float*>(b + W.part_dw);
    cudaError_t e = gemm_linear_dx(D.M, D.N, D.K, d, w, sum ? part : dx, sum || dxf,
                                   !sum && add_dx, W.dx_splits, status, st);
    if (e != cudaSuccess) return e;
    if (sum) {
      LinArgs f = {};
      f.y = dx;
      f.res = add_dx ? dx : nullptr;  // (fp32)
      f.M = static_cast<int>(D.M);
      f.N = static_cast<int>(D.K);
      f.act = MOK_ACT_NONE;
      f.vec = 1;
      e = launch_finish(f, part, W.dx_splits, (D.M + 127) / 128 * 128, dxf, st);
      if (e != cudaSuccess) return e;
    }
  }
  if (dw) {
    float* part = reinterpret_cast<float*>(b + W.part_dw);
    const bool sum = W.dw_splits > 1;
    cudaError_t e = gemm_linear_dw(D.M, D.N, D.K, dz, x, D.ld_x, sum ? part : dw,
                                   !sum && add_dw, W.dw_splits, status, st);
    if (e != cudaSuccess || !sum) return e;
    const long long n4 = D.N * D.K / 4;
    const long long stride4 = (D.N + 127) / 128 * 128 * D.K / 4;
    long long blocks = (n4 + 255) / 256;
    const long long cap = 8LL * num_sms_current_device();
    if (blocks > cap) blocks = cap;
    ProfScope prof("linear_dw_sum", st);
    e = launch_dependent(split_sum_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, st,
                         reinterpret_cast<const float4*>(part), W.dw_splits, stride4, n4,
                         reinterpret_cast<float4*>(dw), add_dw ? 1 : 0);
    count_launch();
    return e != cudaSuccess ? e : cudaGetLastError();
  }
  return cudaSuccess;
}

}  // namespace mok
