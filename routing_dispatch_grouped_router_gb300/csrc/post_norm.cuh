// What the kernels of the norms after and before a block share (post_norm.cu,
// post_norm_bwd.cu): sums over a row, the ring of rows in shared memory and its
// shapes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "mok_internal.h"
#include "ptx.cuh"
#include "rows.cuh"

namespace mok {

template <int N>
struct Ring {
  const void* p[N];   // the inputs' first rows (a NULL one: none)
  long long ld[N];
  int f32[N];
  uint32_t off[N];    // of an input within a slot
  uint32_t row_bytes, depth;
  int ld8;            // SHIFT: elements from one row to the next, mod 8
};

// Threads of a row, blocks and ring of the ring kernels.
struct RingShape {
  int tpr;
  uint32_t vec_bytes;  // of a row's bf16 input (an fp32 one's: twice)
  uint32_t row_bytes, depth;
  int64_t blocks;
};
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
// The backward through the ring of rows (post_norm_ring.cu).
cudaError_t launch_post_pre_bwd_ring(const PostPreBwd& a, Ring<4>& g, const RingShape& b, bool yf,
                                     bool xf, bool sf, bool shift, cudaStream_t st);

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

// The ring kernels' rows: a ring of `depth` rows in shared memory, each input of a
// row one bulk copy, requested a row or more ahead, so that a row's reductions do not
// interrupt the stream of loads.  What an SM issues and waits for counts as well
// here: a thread holds two vectors (one: half of the instructions are the
// reductions'), its elements in pairs for the packed fp32 instructions, and each row
// has one barrier, shared with the next row's first sums.  (8192 x 7168 backward with
// one vector a thread and two barriers a row: 226 us, floor 105.)
//
// SHIFT: rows of any length in aligned tensors.  Row r begins r ld8 elements (mod 8)
// past a multiple of eight, in all of them alike; a block's rows are a multiple of
// eight apart, so all of its rows begin at the same h, and a thread's eight columns
// are 8 v - h .. + 7: aligned words everywhere.  The copies take whole 16-byte words
// (a few elements of the rows next to it with them), except past the end of the last
// row.
constexpr int kRingMaxDepth = 4;
constexpr int kRingSmem = 212 * 1024;  // of an SM's shared memory, for all its blocks
constexpr int kRingThreads = 512;      // the most of a block
// threads of an SM, by the kernels' registers
constexpr int kFwdRingThreads = 768, kFwdShiftThreads = 512, kBwdRingThreads = 512;
// (rows at a shift of up to 384 threads: 168 registers instead of 128, 3000 x 5001
// with fp32 x 66 us instead of 83)
constexpr int kBwdShiftThreads = 384;
constexpr int kRingMinD = 1024, kShiftMinD = 512;

// Row r into `slot` (one thread).
template <int N, bool SHIFT>
__device__ __forceinline__ void ring_fill(const Ring<N>& g, uint8_t* slot, uint64_t* full,
                                          long long r, long long rows, int d, int h) {
  uint32_t total = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (!g.p[i]) continue;
    const int es = g.f32[i] ? 4 : 2;
    const uint8_t* src = static_cast<const uint8_t*>(g.p[i]) + (r * g.ld[i] - h) * es;
    uint32_t bytes = static_cast<uint32_t>((d + h + 7) / 8 * 8 * es);
    if (SHIFT && r == rows - 1) {
      const uint32_t end = static_cast<uint32_t>((d + h) * es);
      bytes = end & ~15u;
      for (uint32_t j = bytes; j < end; j += 2)  // (the last row's last elements)
        *reinterpret_cast<uint16_t*>(slot + g.off[i] + j) =
            *reinterpret_cast<const uint16_t*>(src + j);
    }
    if (bytes) bulk_load(slot + g.off[i], src, bytes, full);
    total += bytes;
  }
  mbar_arrive_expect_tx(full, total);
}

// Pairs of fp32 values and the packed instructions on them.
using F2 = unsigned long long;
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ F2 f2(float v) { return f2(v, v); }
__device__ __forceinline__ float lo_of(F2 v) { return __uint_as_float(static_cast<uint32_t>(v)); }
__device__ __forceinline__ float hi_of(F2 v) {
  return __uint_as_float(static_cast<uint32_t>(v >> 32));
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// The pair's elements that are the row's own (bits 0 and 1 of `own`), the others 0.
__device__ __forceinline__ F2 keep(F2 v, uint32_t own) {
  return v & ((own & 1u ? 0xffffffffull : 0ull) | (own & 2u ? 0xffffffffull << 32 : 0ull));
}

// Vector v of input i in a slot; elements that are not the row's own are 0.
template <bool F32, bool SHIFT, int N>
__device__ __forceinline__ void ring_get(const Ring<N>& g, const uint8_t* slot, int i, int v,
                                         uint32_t own, F2 (&o)[4]) {
  if (F32) {
    const ulonglong2* p = reinterpret_cast<const ulonglong2*>(slot + g.off[i]) + 2 * v;
    const ulonglong2 a = p[0], b = p[1];
    o[0] = a.x; o[1] = a.y; o[2] = b.x; o[3] = b.y;
  } else {
    const uint4 u = reinterpret_cast<const uint4*>(slot + g.off[i])[v];
    o[0] = f2(bf16lo(u.x), bf16hi(u.x));
    o[1] = f2(bf16lo(u.y), bf16hi(u.y));
    o[2] = f2(bf16lo(u.z), bf16hi(u.z));
    o[3] = f2(bf16lo(u.w), bf16hi(u.w));
  }
  if (SHIFT && own != 0xffu) {
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = keep(o[j], own >> (2 * j));
  }
}

__device__ __forceinline__ uint4 pack_bf16(const F2 (&o)[4]) {
  return make_uint4(pack_bf16x2(lo_of(o[0]), hi_of(o[0])), pack_bf16x2(lo_of(o[1]), hi_of(o[1])),
                    pack_bf16x2(lo_of(o[2]), hi_of(o[2])), pack_bf16x2(lo_of(o[3]), hi_of(o[3])));
}

// ... and to an output row that begins h elements after `row`.
template <bool SHIFT>
__device__ __forceinline__ void ring_put(uint8_t* row, int f32, int v, uint32_t own,
                                         const F2 (&o)[4]) {
  if (SHIFT && own != 0xffu) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (!(own >> j & 1u)) continue;
      const float x = j & 1 ? hi_of(o[j >> 1]) : lo_of(o[j >> 1]);
      if (f32) reinterpret_cast<float*>(row)[8 * v + j] = x;
      else reinterpret_cast<__nv_bfloat16*>(row)[8 * v + j] = __float2bfloat16_rn(x);
    }
  } else if (f32) {
    ulonglong2* p = reinterpret_cast<ulonglong2*>(row) + 2 * v;
    p[0] = make_ulonglong2(o[0], o[1]);
    p[1] = make_ulonglong2(o[2], o[3]);
  } else {
    reinterpret_cast<uint4*>(row)[v] = pack_bf16(o);
  }
}
__device__ __forceinline__ uint8_t* out_row(void* base, long long r, long long ld, int h, int f32) {
  return static_cast<uint8_t*>(base) + (r * ld - h) * (f32 ? 4 : 2);
}

// Which elements of vector v are columns 0 .. d - 1, and a weight's values there.
__device__ __forceinline__ uint32_t ring_own(int v, int h, int d) {
  uint32_t own = 0xffu;
  const int e = 8 * v - h;  // element 0's column
  if (e < 0) own &= 0xffu << -e;
  if (e + 8 > d) own &= e < d ? 0xffu >> (e + 8 - d) : 0u;
  return own;
}
// (WIDE, rows without a shift: by aligned vectors.)
template <bool WIDE>
__device__ __forceinline__ void ring_weight(const void* w, int f32, int v, int h, uint32_t own,
                                            F2 (&o)[4]) {
  float x[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = 0.f;
  if (WIDE) {
    if (own) load_weight<true>(w, f32, v, 0, x);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (own >> j & 1u) x[j] = elem_at(w, 8 * v - h + j, f32);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) o[j] = f2(x[2 * j], x[2 * j + 1]);
}

// The warp's sums of N <= 8 values (a power of two): of value lane / (32 / N).  Each
// step halves the values that a lane holds.
template <int N>
__device__ __forceinline__ float warp_sums(float (&v)[N], int lane) {
  int bit = 16;
#pragma unroll
  for (int n = N / 2; n > 0; n /= 2, bit /= 2) {
    const bool up = (lane & bit) != 0;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float give = up ? v[i] : v[i + n], mine = up ? v[i + n] : v[i];
      v[i] = mine + __shfl_xor_sync(0xffffffffu, give, bit);
    }
  }
  float s = v[0];
  for (; bit > 0; bit /= 2) s += __shfl_xor_sync(0xffffffffu, s, bit);
  return s;
}
// The block's, from the `nw` warps' in red[value][warp].
template <int N>
__device__ __forceinline__ void block_sums(const float (*red)[16], int nw, int lane,
                                           float (&out)[N]) {
  constexpr int L = 32 / N;  // lanes of a value
  float s = 0.f;
  for (int w = lane & (L - 1); w < nw; w += L) s += red[lane / L][w];
#pragma unroll
  for (int o = L / 2; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
#pragma unroll
  for (int i = 0; i < N; ++i) out[i] = __shfl_sync(0xffffffffu, s, L * i);
}

inline int esize(bool f32) { return f32 ? 4 : 2; }

// f(std::bool_constant ...) of run-time truth values.
template <typename F>
cudaError_t with_types(const F& f, bool a) {
  return a ? f(std::true_type()) : f(std::false_type());
}
template <typename F, typename... B>
cudaError_t with_types(const F& f, bool a, B... rest) {
  return with_types([&](auto... R) { return a ? f(std::true_type(), R...) : f(std::false_type(), R...); },
                    rest...);
}

// Threads of a row, blocks and ring of the ring kernels, by the descriptor and the
// rows' kind alone (the backward's sums do not depend on the device); blocks = 0
// where they do not serve: rows too short or too long, fewer than the ring is good
// for.  per_elem: bytes of an element's inputs.  threads: what an SM holds (its
// registers).
inline RingShape ring_shape(int64_t rows, int64_t d, bool shift, int64_t per_elem, int threads) {
  RingShape b = {};
  const int64_t nvec = shift ? (d + 14) / 8 : d / 8;
  if (nvec > 2 * kRingThreads || d < (shift ? kShiftMinD : kRingMinD)) return b;
  b.tpr = static_cast<int>((nvec + 63) / 64 * 32);
  b.vec_bytes = static_cast<uint32_t>(nvec * 16);
  b.row_bytes = static_cast<uint32_t>(nvec * 8 * per_elem);
  int64_t per_sm = threads / b.tpr;
  if (per_sm < 1) per_sm = 1;
  if (per_sm > 8) per_sm = 8;
  while (per_sm > 1 && per_sm * 3 * b.row_bytes > kRingSmem) --per_sm;  // three rows each
  b.depth = static_cast<uint32_t>(kRingSmem / per_sm / b.row_bytes);
  if (b.depth > kRingMaxDepth) b.depth = kRingMaxDepth;
  if (b.depth < 2) return b;
  const int64_t blocks = kGb300Sms * per_sm;  // (a multiple of eight)
  if (rows > blocks) b.blocks = blocks;
  return b;
}

// Every tensor's rows begin alike: aligned bases, lengths that agree mod 8 (fp32
// alone: mod 4).
inline bool alike(const void* p, int64_t ld, bool f32, int64_t step) {
  return !p || ((reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld - step) % (f32 ? 4 : 8) == 0);
}

template <typename K, typename A, int N>
cudaError_t ring_launch(K kern, const A& a, Ring<N>& g, const RingShape& b, cudaStream_t st) {
  uint32_t off = 0;
  g.row_bytes = b.row_bytes;
  g.depth = b.depth;
  for (int i = 0; i < N; ++i) {
    g.off[i] = off;
    if (g.p[i]) off += b.vec_bytes * (g.f32[i] ? 2 : 1);
  }
  const int smem = static_cast<int>(b.depth * b.row_bytes);
  // (the limit is the kernel's, not the call's: the most that any call takes, so that
  // no host thread lowers it between another's setting and launch)
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingSmem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, dim3(static_cast<unsigned>(b.blocks)), dim3(b.tpr), smem, st, a, g);
}

}  // namespace

}  // namespace mok
