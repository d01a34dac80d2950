// Products grouped by expert over ragged rows, on tcgen05 (sm_103a): rows
// off[e] <= r < off[e+1] belong to expert e,
//
//   forward  y_r = w_e x_r,   dx  dx_r = w_e^T dy_r,   dw  dw_e = sum of dy_r x_r^T
//
// Groups begin and end at any row.  In the forward and dx they are the rows of
// the product: a tile's rows past its group's end are other groups' or none, their
// products go nowhere, and its stores are cut at the end.  In dw they are the sum:
// the last K block of a group is cut to whole MMAs of 16 rows, and its last rows
// below 16 go through a slot of their own, where the rows past the end are zeroed
// in both operands (so that no Inf or NaN of the next group comes in).  The maps of
// the weights are cut at each expert's end.
//
// One CTA per SM, or one pair of CTAs on two (tcgen05.mma.cta_group::2, tiles of
// 256 rows), walks the tiles that the offsets on the device give, at a stride of
// the grid: warp 0 fills a ring of stages by TMA, warp 1 issues the MMAs into two
// accumulators in TMEM, warps 2..9 take the one in TMEM to memory while the other
// is being summed.  Every tile has one owner and one order of its sum.
//
// Large groups are bound by the tensor cores, a few rows per group by the bytes of
// the weights, dw by its own: 32768 rows in 8 groups, N = K = 2048, 158 us forward (1735
// TFLOP/s) and 157 dx; in 64 groups of any size 212 and 211 (tiles round rows up by a
// quarter) and dw 280 (4.8 TB/s); 320 rows of 64 groups 88 us (6.1 TB/s).
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <type_traits>

#include "mok_internal.h"
#include "ptx.cuh"

namespace mok {

enum GroupedMode : int { GRP_FWD = 0, GRP_DX = 1, GRP_DW = 2 };

struct GroupedArgs {
  const int* offsets;
  int E, R;
  int rows_w;     // DW: N (rows of C); else unused
  int cols;       // columns of C
  int num_kb;     // FWD, DX: 64-value blocks of the sum
  int m_tiles;    // DW: row tiles of C (PAIR: of 256 rows)
  int splits;     // DW: parts of a group's rows, each with a C of its own
  int n_tiles;
  long long ld_out;  // row stride of C
  void* out;
  int wide;          // C's rows begin on 32 bytes, and so do their ends
  int round16;       // F32: C is bf16 all the same (a long sum, see kOneSumKb)
  int chunk_kb;      // F32: K blocks of one accumulation
  // DX, DW: w's, x's (K) and dy's (N) 64-column blocks are a dimension of their maps:
  // one copy brings a stage's blocks.  (One thread issues the copies; one per 64
  // columns or 32 rows made it the slowest part: 64 groups of 512 rows, N = K = 2048,
  // single CTAs: forward 217 -> 206 us, dx 232 -> 197.  Of whole blocks: a last one
  // cut at the row's end would reach past the tensor's.)
  int blocks_k, blocks_n;
  int accumulate;
  int* status;
};

namespace {

constexpr int kEpiWarps = 8;
// DW: one more warp, for the groups' last rows
constexpr int threads_of(int mode) { return 320 + (mode == GRP_DW ? 32 : 0); }
constexpr int kTailWarp = 10;
// An fp32 result is summed on the tensor cores, whose accumulation truncates, over
// at most 36 MMAs (9 K blocks; 37 where dw's last chunk also takes the group's last rows)
// at a time, and the chunks' sums are added in
// registers with correct rounding (one accumulation over 2048 values is 2e-6 off,
// these 6e-7).
constexpr int kChunkKb = 9;
// A bf16 result is one accumulation while that is short: values of one sign lose 1e-7
// of their sum per MMA, 1e-4 over 256 K blocks (a bf16 half step is 2e-3 to 4e-3).
// Longer sums are taken in chunks of 64 K blocks and rounded at the end (2^20 values of
// one sign were 6.7e-3 off in one accumulation).  8192 rows of 8 groups, N = 2048, K =
// 16448: 356 us, in chunks of nine 378, in one accumulation 362.
constexpr int kOneSumKb = 256, kLongChunkKb = 64;

template <int MODE, int BN, bool PAIR>
struct Cfg {
  static constexpr int B_ROWS = PAIR ? BN / 2 : BN;  // of B staged by one CTA
  static constexpr int A_BYTES = 128 * 64 * 2, B_BYTES = B_ROWS * 64 * 2;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int TABLE_BYTES = 2 * 514 * 4 + 64;
  static constexpr int BAR_BYTES = 256;
  // DW stores C through shared memory: 32 rows of 128 bytes per warp.  (Two buffers
  // each cost a stage: 300 us instead of 274 for 64 groups of 512 rows, N = K =
  // 2048; stores from registers, a sector or a row's line at a time, 310 to 340.)
  static constexpr int STAGING = MODE == GRP_DW ? kEpiWarps * 4096 : 0;
  // ... and has two slots for groups' last rows below 16, of A and of B
  static constexpr int TAIL_BYTES = MODE == GRP_DW ? (128 + B_ROWS) * 32 : 0;
  static constexpr int ROOM =
      232448 - 1024 - BAR_BYTES - TABLE_BYTES - STAGING - 2 * TAIL_BYTES;
  static constexpr int STAGES = ROOM / STAGE_BYTES < 8 ? ROOM / STAGE_BYTES : 8;
  static constexpr int TAIL_OFF = STAGES * STAGE_BYTES;
  static constexpr int STAGING_OFF = TAIL_OFF + 2 * TAIL_BYTES;
  static constexpr int BAR_OFF = STAGING_OFF + STAGING;
  static constexpr int TABLE_OFF = BAR_OFF + BAR_BYTES;
  static constexpr int SMEM_BYTES = 1024 + TABLE_OFF + TABLE_BYTES;
};
static_assert(Cfg<GRP_FWD, 256, false>::STAGES == 4 && Cfg<GRP_FWD, 256, true>::STAGES == 6 &&
                  Cfg<GRP_FWD, 128, false>::STAGES == 6 && Cfg<GRP_DW, 256, false>::STAGES == 3 &&
                  Cfg<GRP_DW, 256, true>::STAGES == 5,
              "stages");
static_assert(Cfg<GRP_FWD, 256, false>::SMEM_BYTES <= 232448 &&
                  Cfg<GRP_DW, 256, true>::SMEM_BYTES <= 232448,
              "smem");
static_assert((2 * 8 + 11) * 8 + 8 <= Cfg<GRP_FWD, 128, false>::BAR_BYTES, "barriers");
static_assert(2 * 320 >= 514, "two offsets per thread");

// The groups' first rows (monotone, within [0, R], whatever the offsets hold) into
// off[0 .. E] and the prefix of their tiles of `tile` rows into pre[0 .. E]; without
// a tile, the groups in the order of their sizes, the largest first.
__device__ __forceinline__ void group_table(const GroupedArgs& a, int tile, int* off, int* pre,
                                            int* red) {
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, i = 2 * t;
  auto value = [&](int j) { return j <= a.E ? __ldg(a.offsets + j) : 0; };
  const int raw0 = value(i), raw1 = value(i + 1);
  const int v0 = min(max(raw0, 0), a.R), v1 = min(max(raw1, 0), a.R);
  int m = max(v0, v1);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(0xffffffffu, m, o);
    if (lane >= o) m = max(m, n);
  }
  if (lane == 31) red[warp] = m;
  __syncthreads();
  int before = __shfl_up_sync(0xffffffffu, m, 1);
  if (lane == 0) before = 0;
  for (int w = 0; w < warp; ++w) before = max(before, red[w]);
  const int o0 = max(before, v0), o1 = max(o0, v1);
  if (i <= a.E) off[i] = o0;
  if (i + 1 <= a.E) off[i + 1] = o1;
  if (blockIdx.x == 0 && ((i <= a.E && raw0 != o0) || (i + 1 <= a.E && raw1 != o1)))
    set_status(a.status, MOK_ERR_DEVICE_INDEX);
  __syncthreads();
  if (tile == 0) {  // pre[r]: the group that r groups are larger than (or before)
    for (int e = t; e < a.E; e += blockDim.x) {
      const int n = off[e + 1] - off[e];
      int r = 0, last = off[0];
      for (int f = 0; f < a.E; ++f) {
        const int next = off[f + 1], m = next - last;
        r += m > n || (m == n && f < e);
        last = next;
      }
      pre[r] = e;
    }
    __syncthreads();
    return;
  }
  const int c0 = i < a.E ? (off[i + 1] - off[i] + tile - 1) / tile : 0;
  const int c1 = i + 1 < a.E ? (off[i + 2] - off[i + 1] + tile - 1) / tile : 0;
  int s = c0 + c1;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += n;
  }
  if (lane == 31) red[warp] = s;
  __syncthreads();
  int sum = s - c0 - c1;
  for (int w = 0; w < warp; ++w) sum += red[w];
  if (i <= a.E) pre[i] = sum;
  if (i + 1 <= a.E) pre[i + 1] = sum + c0;
  __syncthreads();
}

struct Tile {
  int e, n_tile;
  int row0;    // FWD, DX: first row of this CTA's 128; DW: first row of C_e
  int rows;    // FWD, DX: this CTA's rows (0 .. 128), DW: likewise of C_e
  int other;   // FWD, DX, PAIR: the rows of the pair's other CTA
  int k0, kn;  // DW: first row of the group and its rows in whole sixteens,
  int tail;    // and the others
  int num_kb;
};

// Tile `local` of a group of mt x nt tiles: bands of kBand row tiles, in each column
// tiles from the left, so that the tiles that run at one time share rows and
// weights (and a band's rows stay in L2 until its last column).
constexpr int kBand = 8;
__device__ __forceinline__ void place(int local, int mt, int nt, int* m, int* n) {
  const int band = local / (kBand * nt), r = local - band * (kBand * nt);
  const int rows = min(kBand, mt - band * kBand);
  *n = r / rows;
  *m = band * kBand + r - *n * rows;
}

template <int MODE, bool PAIR>
__device__ __forceinline__ Tile tile_of(const GroupedArgs& a, const int* off, const int* pre,
                                        long long t, int rank) {
  constexpr int TM = PAIR ? 256 : 128;
  Tile tl;
  if (MODE == GRP_DW) {
    const int per = a.m_tiles * a.n_tiles;
    const int part = static_cast<int>(t / per);
    const int nth = part / a.splits, split = part - nth * a.splits;
    const int local = static_cast<int>(t - static_cast<long long>(part) * per);
    int m;
    place(local, a.m_tiles, a.n_tiles, &m, &tl.n_tile);
    const int e = pre[nth];
    tl.e = split * a.E + e;
    tl.row0 = m * TM + rank * 128;
    tl.rows = min(max(a.rows_w - tl.row0, 0), 128);
    tl.other = 0;
    tl.k0 = off[e];
    tl.kn = off[e + 1] - tl.k0;
    tl.tail = tl.kn & 15;
    tl.kn -= tl.tail;
    tl.num_kb = (tl.kn + 63) / 64;
    if (a.splits > 1) {  // its share of the K blocks; the last one also has the tail
      const int lo = static_cast<int>(static_cast<long long>(tl.num_kb) * split / a.splits);
      const int hi = static_cast<int>(static_cast<long long>(tl.num_kb) * (split + 1) / a.splits);
      const bool last = split == a.splits - 1;
      tl.kn = (last ? tl.kn : hi * 64) - lo * 64;
      tl.k0 += lo * 64;
      tl.num_kb = hi - lo;
      if (!last) tl.tail = 0;
    }
    return tl;
  }
  int lo = 0, hi = a.E;  // pre[lo] n_tiles <= t < pre[hi] n_tiles
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (static_cast<long long>(pre[mid]) * a.n_tiles <= t) lo = mid; else hi = mid;
  }
  const int p0 = pre[lo], mt = pre[lo + 1] - p0;
  const int local = static_cast<int>(t - static_cast<long long>(p0) * a.n_tiles);
  tl.e = lo;
  int m;
  place(local, mt, a.n_tiles, &m, &tl.n_tile);
  const int first = off[lo] + m * TM, end = off[lo + 1];
  tl.row0 = first + rank * 128;
  tl.rows = min(max(end - tl.row0, 0), 128);
  tl.other = PAIR ? min(max(end - (first + (rank ^ 1) * 128), 0), 128) : 0;
  tl.k0 = tl.kn = tl.tail = 0;
  tl.num_kb = a.num_kb;
  return tl;
}

// Bytes of A that a stage of `rows` rows holds: whole boxes of 32 rows.
__device__ __forceinline__ uint32_t a_bytes(int rows) { return (rows + 31) / 32 * 4096u; }

}  // namespace

// tmA, tmB: the stages' boxes.  FWD, DX: tmA2 has boxes of 32 rows of A.  DW: tmA2
// and tmB2 have boxes of 16 rows, tmC is C's.
template <int MODE, int BN, bool F32, bool PAIR>
__global__ void __launch_bounds__(threads_of(MODE), 1)
    grouped_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ CUtensorMap tmA2,
                   const __grid_constant__ CUtensorMap tmB2,
                   const __grid_constant__ CUtensorMap tmC,
                   const __grid_constant__ GroupedArgs args) {
  using C = Cfg<MODE, BN, PAIR>;
  constexpr bool A_MN = MODE == GRP_DW, B_MN = MODE != GRP_FWD;
  static_assert(MODE != GRP_DW || F32, "fp32 weight gradients");
  static_assert(!PAIR || BN == 256, "pairs");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
  uint64_t* empty = full + C::STAGES;
  uint64_t* tfull = empty + C::STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  // tail slots: copied, zeroed past the group's end (PAIR: in both CTAs), free
  uint64_t* tail_full = drain + 1;
  uint64_t* tail_ready = tail_full + 2;
  uint64_t* tail_empty = tail_ready + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tail_empty + 2);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  int* off = reinterpret_cast<int*>(smem + C::TABLE_OFF);
  int* pre = off + 514;
  int* red = pre + 514;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = PAIR ? static_cast<int>(cluster_ctarank()) : 0;
  const bool leader = rank == 0;
  const int first = PAIR ? static_cast<int>(cluster_id_x()) : static_cast<int>(blockIdx.x);
  const int step = PAIR ? static_cast<int>(cluster_count_x()) : static_cast<int>(gridDim.x);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], PAIR ? 2 * kEpiWarps : kEpiWarps);
      mbar_init(&tail_full[i], 1);
      mbar_init(&tail_ready[i], PAIR ? 2 : 1);
      mbar_init(&tail_empty[i], 1);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (threadIdx.x == 32) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmA2);
    if (MODE == GRP_DW) {
      tma_prefetch_desc(&tmB2);
      tma_prefetch_desc(&tmC);
    }
  }
  if (warp == 1) {
    if (PAIR) {
      tmem_alloc_pair(tmem_slot, 2 * BN);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, 2 * BN);
      tmem_relinquish();
    }
  }
  tc_fence_before_sync();
  if (PAIR) cluster_sync(); else __syncthreads();
  tc_fence_after_sync();
  // from here on the results of the kernel before this one are visible
  grid_dep_wait();
  grid_dep_launch();
  group_table(args, MODE == GRP_DW ? 0 : (PAIR ? 256 : 128), off, pre, red);
  const uint32_t tmem_base = *tmem_slot;
  volatile int* vabort = abort_flag;
  const long long total = MODE == GRP_DW
                              ? static_cast<long long>(args.E) * args.splits * args.m_tiles *
                                    args.n_tiles
                              : static_cast<long long>(pre[args.E]) * args.n_tiles;
  auto tile_at = [&](long long t) { return tile_of<MODE, PAIR>(args, off, pre, t, rank); };
  // this CTA's (pair's) units: one of every `step`, from alternate ends for the
  // weight gradients, whose tiles go from the longest to the shortest
  auto unit = [&](int i) {
    return static_cast<long long>(i) * step +
           (MODE == GRP_DW && (i & 1) ? step - 1 - first : first);
  };
  auto wait = [&](uint64_t* bar, uint32_t par) -> bool {
    return PAIR ? mbar_wait_cluster(bar, par, vabort) : mbar_wait(bar, par, vabort);
  };
  // DW: K rows y .. of `n` blocks of 64 columns from x (whole: by one copy)
  auto load_cols = [&](uint8_t* dst, const CUtensorMap* tm, uint64_t* bar, uint32_t bar_pair,
                       int x, int y, int n, uint32_t block, int whole) {
    if (whole) {
      if (bar_pair) tma_load_3d_pair(dst, tm, bar_pair, 0, y, x >> 6);
      else tma_load_3d(dst, tm, bar, 0, y, x >> 6);
      return;
    }
    for (int j = 0; j < n; ++j) {
      if (bar_pair) tma_load_2d_pair(dst + j * block, tm, bar_pair, x + 64 * j, y);
      else tma_load_2d(dst + j * block, tm, bar, x + 64 * j, y);
    }
  };

  if (warp == 0) {
    if (lane == 0) {
      // --------------------------------------------------------- producer --
      // PAIR: both CTAs' copies are counted on the leader's `full` barrier
      const uint32_t full_leader = PAIR ? mapa_shared(smem_addr(full), 0) : 0u;
      int stage = 0;
      uint32_t phase = 0;
      uint32_t steps = 0;  // stages filled
      bool ok = true;
      for (int i = 0; unit(i) < total && ok; ++i) {
        const Tile tl = tile_at(unit(i));
        const int n0 = tl.n_tile * BN + rank * C::B_ROWS;
        uint32_t bytes = (MODE == GRP_DW ? C::A_BYTES : a_bytes(tl.rows)) + C::B_BYTES;
        if (PAIR) bytes += (MODE == GRP_DW ? C::A_BYTES : a_bytes(tl.other)) + C::B_BYTES;
        for (int kb = 0; kb < tl.num_kb; ++kb, ++steps) {
          if (!wait(&empty[stage], phase ^ 1u)) {
            ok = false;
            break;
          }
          uint8_t* sA = smem + stage * C::STAGE_BYTES;
          uint8_t* sB = sA + C::A_BYTES;
          const uint32_t bar_c = full_leader + 8u * stage;
          if (leader) mbar_arrive_expect_tx(&full[stage], bytes);
          if (MODE != GRP_DW) {
            auto rows = [&](const CUtensorMap* tm, int r) {
              uint8_t* dst = sA + r * 128;
              if (PAIR) tma_load_2d_pair(dst, tm, bar_c, kb * 64, tl.row0 + r);
              else tma_load_2d(dst, tm, &full[stage], kb * 64, tl.row0 + r);
            };
            if (tl.rows > 96) {
              rows(&tmA, 0);
            } else {
              for (int r = 0; r < tl.rows; r += 32) rows(&tmA2, r);
            }
            if (MODE == GRP_FWD) {
              if (PAIR) tma_load_3d_pair(sB, &tmB, bar_c, kb * 64, n0, tl.e);
              else tma_load_3d(sB, &tmB, &full[stage], kb * 64, n0, tl.e);
            } else if (args.blocks_k) {
              if (PAIR) tma_load_4d_pair(sB, &tmB, bar_c, 0, kb * 64, n0 >> 6, tl.e);
              else tma_load_4d(sB, &tmB, &full[stage], 0, kb * 64, n0 >> 6, tl.e);
            } else {
#pragma unroll
              for (int j = 0; j < C::B_ROWS / 64; ++j) {
                uint8_t* dst = sB + j * 8192;
                if (PAIR) tma_load_3d_pair(dst, &tmB, bar_c, n0 + 64 * j, kb * 64, tl.e);
                else tma_load_3d(dst, &tmB, &full[stage], n0 + 64 * j, kb * 64, tl.e);
              }
            }
          } else {
            const int y = tl.k0 + kb * 64;
            load_cols(sA, &tmA, &full[stage], PAIR ? bar_c : 0u, tl.row0, y, 2, 8192,
                      args.blocks_n);
            load_cols(sB, &tmB, &full[stage], PAIR ? bar_c : 0u, n0, y, C::B_ROWS / 64, 8192,
                      args.blocks_k);
          }
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {
        *vabort = 1;
        set_status(args.status, MOK_ERR_DEVICE_TIMEOUT);
        // let the copies already issued land before the CTA can exit
        const int zero = 0;
        if (leader) {
          for (uint32_t s = 0; s < C::STAGES && s < steps; ++s)
            mbar_wait(&full[s], (steps - 1 - s) / C::STAGES & 1u, &zero);
        } else {
          spin_ns(1000000ull);
        }
      }
    }
  } else if (warp == 1) {
    // --------------------------------------------------------------- MMA --
    if (lane == 0 && leader) {
      constexpr uint32_t idesc = idesc_bf16_f32(PAIR ? 256 : 128, BN, A_MN, B_MN);
      constexpr uint32_t lbo_a = A_MN ? 8192u : 16u, lbo_b = B_MN ? 8192u : 16u;
      // One thread issues the MMAs, and what it does per K block counts (a select of
      // two descriptors made 64 groups of 512 rows, N = K = 2048, 182 -> 193 us):
      // descriptors are their first stage's, whose low words take the stage's and the
      // step's offsets in sixteens.
      constexpr uint32_t kstep_a = A_MN ? 128u : 2u, kstep_b = B_MN ? 128u : 2u;
      const uint32_t base = smem_addr(smem);
      const uint64_t ad0 = smem_desc_sw128(base, lbo_a, 1024);
      const uint64_t bd0 = smem_desc_sw128(base + C::A_BYTES, lbo_b, 1024);
      auto word = [](uint64_t d, uint32_t lo) {
        return (d & 0xffffffff00000000ull) | lo;
      };
      auto commit = [&](uint64_t* bar) {
        if (PAIR) mma_commit_pair(bar);
        else mma_commit(bar);
      };
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      int it = 0;     // accumulations
      int tails = 0;  // tail slots used
      for (int i = 0; unit(i) < total && ok; ++i) {
        const Tile tl = tile_at(unit(i));
        uint32_t d_tmem = 0;
        int kb0 = 0;
        // (a group of less than 16 rows has its tail alone)
        const int last = tl.num_kb > 0 || tl.tail == 0 ? tl.num_kb : 1;
        for (int kb = 0; kb < last; ++kb) {
          if (kb == 0 || (F32 && kb == kb0 + args.chunk_kb)) {
            if (kb > 0) {  // the next chunk's sum goes to the other accumulator
              commit(&tfull[it & 1]);
              ++it;
            }
            kb0 = kb;
            if (!wait(&tempty[it & 1], (static_cast<uint32_t>(it >> 1) & 1u) ^ 1u)) {
              ok = false;
              break;
            }
            tc_fence_after_sync();
            d_tmem = tmem_base + static_cast<uint32_t>((it & 1) * BN);
          }
          if (kb == tl.num_kb) break;
          if (!wait(&full[stage], phase)) {
            ok = false;
            break;
          }
          int mmas = 4;
          if (MODE == GRP_DW && kb == tl.num_kb - 1 && (tl.kn & 63)) mmas = (tl.kn & 63) >> 4;
          tc_fence_after_sync();
          const uint32_t x = static_cast<uint32_t>(ad0) + stage * (C::STAGE_BYTES / 16);
          const uint32_t y = static_cast<uint32_t>(bd0) + stage * (C::STAGE_BYTES / 16);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (MODE == GRP_DW && j >= mmas) break;
            const uint64_t ad = word(ad0, x + j * kstep_a), bd = word(bd0, y + j * kstep_b);
            const uint32_t acc = j > 0 ? 1u : (kb != kb0 ? 1u : 0u);
            if (PAIR) mma_bf16_pair(d_tmem, ad, bd, idesc, acc);
            else mma_bf16(d_tmem, ad, bd, idesc, acc);
          }
          commit(&empty[stage]);
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        if (MODE == GRP_DW && tl.tail) {
          const int slot = tails & 1;
          if (!wait(&tail_ready[slot], static_cast<uint32_t>(tails >> 1) & 1u)) {
            ok = false;
            break;
          }
          ++tails;
          tc_fence_after_sync();
          // (16 rows: blocks of 64 columns 2 KB apart)
          const uint32_t a_base = smem_addr(smem + C::TAIL_OFF + slot * C::TAIL_BYTES);
          const uint64_t ad = smem_desc_sw128(a_base, 2048, 1024);
          const uint64_t bd = smem_desc_sw128(a_base + 4096, 2048, 1024);
          if (PAIR) mma_bf16_pair(d_tmem, ad, bd, idesc, tl.num_kb > 0);
          else mma_bf16(d_tmem, ad, bd, idesc, tl.num_kb > 0);
          commit(&tail_empty[slot]);
        }
        if (last > 0) {
          commit(&tfull[it & 1]);
          ++it;
        }
      }
      if (!ok) {
        *vabort = 1;
        set_status(args.status, MOK_ERR_DEVICE_TIMEOUT);
        const int zero = 0;
        commit(drain);
        mbar_wait(drain, 0, &zero);
      }
    }
  } else if (warp == kTailWarp) {
    // -------------------------------------------------------------- tails --
    // A warp of their own brings the groups' last rows, two tiles ahead, and zeroes
    // those past the end.  (In the ring's own stage, by the MMA warp or another
    // between copy and MMA, it cost 1.4 us a tile: 32768 rows in 64 groups, N = K =
    // 2048: 350 us; 276 with groups of whole sixteens.)
    const uint32_t ready_leader = PAIR ? mapa_shared(smem_addr(tail_ready), 0) : 0u;
    int tails = 0;
    for (int i = 0; unit(i) < total; ++i) {
      const Tile tl = tile_at(unit(i));
      if (tl.tail == 0) continue;
      const int slot = tails & 1;
      const uint32_t par = static_cast<uint32_t>(tails >> 1) & 1u;
      ++tails;
      uint8_t* p = smem + C::TAIL_OFF + slot * C::TAIL_BYTES;
      // (a tile of 2^24 rows takes a good part of a wait's limit: up to 64 of them)
      // (the warp's lanes give up together: one may see a phase or the flag later)
      bool ok = false;
      for (int tries = 0; tries < 64 && !ok; ++tries) {
        ok = __all_sync(0xffffffffu, wait(&tail_empty[slot], par ^ 1u));
        if (!ok && __any_sync(0xffffffffu, *vabort)) break;
      }
      if (ok) {
        if (lane == 0) {
          mbar_arrive_expect_tx(&tail_full[slot], C::TAIL_BYTES);
          const int y = tl.k0 + tl.kn;
          load_cols(p, &tmA2, &tail_full[slot], 0u, tl.row0, y, 2, 2048, args.blocks_n);
          load_cols(p + 4096, &tmB2, &tail_full[slot], 0u, tl.n_tile * BN + rank * C::B_ROWS, y,
                    C::B_ROWS / 64, 2048, args.blocks_k);
        }
        __syncwarp();
        ok = __all_sync(0xffffffffu, wait(&tail_full[slot], par));
      }
      if (!ok) {
        *vabort = 1;
        if (lane == 0) set_status(args.status, MOK_ERR_DEVICE_TIMEOUT);
        spin_ns(1000000ull);  // copies in flight land before the CTA can exit
        break;
      }
      for (int b = 0; b < C::TAIL_BYTES / 2048; ++b)
        for (int j = tl.tail * 8 + lane; j < 128; j += 32)
          *reinterpret_cast<uint4*>(p + b * 2048 + j * 16) = make_uint4(0u, 0u, 0u, 0u);
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) {
        if (PAIR) mbar_arrive_cluster(ready_leader + 8u * slot);
        else mbar_arrive(&tail_ready[slot]);
      }
    }
  } else {
    // ----------------------------------------------------------- epilogue --
    const int q = warp & 3;            // TMEM lane quarter this warp may read
    const int half = (warp - 2) >> 2;  // column half of the tile
    const uint32_t tempty_leader = PAIR ? mapa_shared(smem_addr(tempty), 0) : 0u;
    constexpr int HC = BN / 2;           // columns of this warp
    constexpr int ES = F32 ? 4 : 2;
    // whole sectors of 32 bytes where C's rows begin on one
    const bool wide = args.wide != 0;
    uint8_t* const out = static_cast<uint8_t*>(args.out);
    // DW: 32 x 32 values (this lane's row) through shared memory and the TMA
    uint8_t* const buf = smem + C::STAGING_OFF + (warp - 2) * 4096;
    auto put_dw = [&](const Tile& tl, int x, const float* v) {
      if (lane == 0) bulk_wait_read<0>();
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 8; ++j)
        *reinterpret_cast<float4*>(buf + lane * 128 + ((j ^ (lane & 7)) << 4)) =
            make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (args.accumulate) tma_reduce_add_3d(&tmC, buf, x, tl.row0 + q * 32, tl.e);
        else tma_store_3d(&tmC, buf, x, tl.row0 + q * 32, tl.e);
        bulk_commit();
      }
    };
    // 32 columns of this lane's row (words of 16 bytes) to C's columns x ..
    auto put = [&](const Tile& tl, int x, const uint4* w, int words) {
      const long long row = tl.row0 + q * 32 + lane;
      const int es = ES == 4 && args.round16 ? 2 : ES;
      uint8_t* p = out + (row * args.ld_out + x) * es;
      const int left = min((args.cols - x) * es / 16, words);  // words within the row
      if (wide) {
#pragma unroll
        for (int j = 0; j < words; j += 2)
          if (j < left) st_global_v8(p + 16 * j, w[j], w[j + 1]);
      } else {
#pragma unroll
        for (int j = 0; j < words; ++j)
          if (j < left) *reinterpret_cast<uint4*>(p + 16 * j) = w[j];
      }
    };
    int it = 0;
    for (int i = 0; unit(i) < total; ++i) {
      const Tile tl = tile_at(unit(i));
      const int valid = min(max(tl.rows - q * 32, 0), 32);
      const bool in = lane < valid;
      const int x0 = tl.n_tile * BN + half * HC;
      const int chunks =
          !F32 || (tl.num_kb == 0 && tl.tail) ? 1 : (tl.num_kb + args.chunk_kb - 1) / args.chunk_kb;
      float sum[F32 ? HC : 1];
      if constexpr (F32) {
#pragma unroll
        for (int j = 0; j < HC; ++j) sum[j] = 0.f;
      }
      bool ok = true;
      for (int ch = 0; ch < chunks; ++ch, ++it) {
        ok = __all_sync(0xffffffffu,
                        wait(&tfull[it & 1], static_cast<uint32_t>(it >> 1) & 1u));
        if (!ok) {
          *vabort = 1;
          set_status(args.status, MOK_ERR_DEVICE_TIMEOUT);
          break;
        }
        tc_fence_after_sync();
        __syncwarp();
        const uint32_t src = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                             static_cast<uint32_t>((it & 1) * BN + half * HC);
        if (valid > 0) {
          if constexpr (F32) {
#pragma unroll
            for (int c = 0; c < HC; c += 32) {
              uint32_t r0[16], r1[16];
              tmem_ld16(src + c, r0);
              tmem_ld16(src + c + 16, r1);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                sum[c + j] += __uint_as_float(r0[j]);
                sum[c + 16 + j] += __uint_as_float(r1[j]);
              }
            }
          } else {
#pragma unroll 1
            for (int c = 0; c < HC && x0 + c < args.cols; c += 32) {
              uint32_t r[2][16];
              tmem_ld16(src + c, r[0]);
              tmem_ld16(src + c + 16, r[1]);
              tmem_ld_wait();
              uint4 w[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint32_t* v = r[j >> 1] + 8 * (j & 1);
                w[j] = make_uint4(
                    pack_bf16x2(__uint_as_float(v[0]), __uint_as_float(v[1])),
                    pack_bf16x2(__uint_as_float(v[2]), __uint_as_float(v[3])),
                    pack_bf16x2(__uint_as_float(v[4]), __uint_as_float(v[5])),
                    pack_bf16x2(__uint_as_float(v[6]), __uint_as_float(v[7])));
              }
              if (in) put(tl, x0 + c, w, 4);
            }
          }
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          if (PAIR) mbar_arrive_cluster(tempty_leader + 8u * (it & 1));
          else mbar_arrive(&tempty[it & 1]);
        }
      }
      if (!ok) break;
      if constexpr (F32) {
        if (MODE == GRP_DW) {
          if (valid > 0 && !(args.accumulate && chunks == 0)) {
#pragma unroll
            for (int c = 0; c < HC; c += 32)
              if (x0 + c < args.cols) put_dw(tl, x0 + c, sum + c);
          }
        } else if (in && args.round16) {
#pragma unroll
          for (int c = 0; c < HC; c += 32) {
            if (x0 + c >= args.cols) continue;
            uint4 w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float* v = sum + c + 8 * j;
              w[j] = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
            }
            put(tl, x0 + c, w, 4);
          }
        } else if (in) {
#pragma unroll
          for (int c = 0; c < HC; c += 32) {
            if (x0 + c >= args.cols) continue;
            uint4 w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
              w[j] = make_uint4(
                  __float_as_uint(sum[c + 4 * j]), __float_as_uint(sum[c + 4 * j + 1]),
                  __float_as_uint(sum[c + 4 * j + 2]), __float_as_uint(sum[c + 4 * j + 3]));
            put(tl, x0 + c, w, 8);
          }
        }
      }
    }
    if (MODE == GRP_DW && lane == 0) bulk_wait_all<0>();  // stores complete before exit
  }

  // the leader's MMAs read the other CTA's shared memory: neither CTA of a pair
  // leaves (or frees TMEM) before both are done
  tc_fence_before_sync();
  if (PAIR) cluster_sync(); else __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after_sync();
    if (PAIR) tmem_dealloc_pair(tmem_base, 2 * BN);
    else tmem_dealloc(tmem_base, 2 * BN);
  }
}

namespace {

template <int MODE, int BN, bool F32, bool PAIR>
cudaError_t launch(const char* name, const CUtensorMap& ta, const CUtensorMap& tb,
                   const CUtensorMap& ta2, const CUtensorMap& tb2, const CUtensorMap& tc,
                   const GroupedArgs& a,
                   long long max_units, cudaStream_t st) {
  auto kern = grouped_kernel<MODE, BN, F32, PAIR>;
  constexpr int smem = Cfg<MODE, BN, PAIR>::SMEM_BYTES;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int sms = num_sms_current_device();
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(threads_of(MODE), 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (!PAIR) {
    cfg.gridDim = dim3(static_cast<unsigned>(max_units < sms ? max_units : sms), 1, 1);
  } else {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(sms / 2 * 2), 1, 1);
    // clusters that can be resident at once, per instantiation and process (one
    // device type); racing first launches compute the same value
    static std::atomic<int> resident{-1};
    int n = resident.load(std::memory_order_relaxed);
    if (n < 0) {
      cudaLaunchConfig_t q = cfg;  // the cluster shape alone
      q.attrs = &attr[1];
      e = cudaOccupancyMaxActiveClusters(&n, kern, &q);
      if (e != cudaSuccess) return e;
      resident.store(n, std::memory_order_relaxed);
    }
    if (n < 1) return cudaErrorInvalidConfiguration;
    cfg.numAttrs = 2;
    cfg.gridDim = dim3(static_cast<unsigned>(2 * (max_units < n ? max_units : n)), 1, 1);
  }
  ProfScope prof(name, st);
  e = cudaLaunchKernelEx(&cfg, kern, ta, tb, ta2, tb2, tc, a);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

constexpr CUtensorMapDataType kBf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
constexpr CUtensorMapSwizzle kSw128 = CU_TENSOR_MAP_SWIZZLE_128B;

// The row tiles of `tile` rows that R rows in E groups can make.
long long most_tiles(const mok_grouped_desc& D, int tile) {
  return D.rows / tile + (D.E < D.rows ? D.E : D.rows);
}

// Forward and dx: C [R, cols] = A [R, sum] w.
template <int MODE>
cudaError_t rows_product(const char* name, const mok_grouped_desc& D, const void* A,
                         long long ld_a, int64_t sum, const void* w, void* out, long long ld_out,
                         int64_t cols, bool f32, const int32_t* offsets, int* status,
                         cudaStream_t st) {
  if (D.rows == 0) return cudaSuccess;
  GroupedArgs a = {};
  a.offsets = offsets;
  a.E = D.E;
  a.R = static_cast<int>(D.rows);
  a.cols = static_cast<int>(cols);
  a.num_kb = static_cast<int>((sum + 63) / 64);
  a.ld_out = ld_out;
  a.out = out;
  a.status = status;
  CUtensorMap ta, ta2, tb;
  const int es = f32 ? 4 : 2;
  a.wide = (reinterpret_cast<uintptr_t>(out) & 31) == 0 && ld_out * es % 32 == 0 &&
           cols * es % 32 == 0;
  a.blocks_k = MODE == GRP_DX && D.K % 64 == 0;
  a.round16 = !f32 && a.num_kb > kOneSumKb;
  a.chunk_kb = a.round16 ? kLongChunkKb : kChunkKb;
  if (!make_tensor_map_2d(&ta, kBf, 2, A, sum, D.rows, ld_a, 64, 128, kSw128) ||
      !make_tensor_map_2d(&ta2, kBf, 2, A, sum, D.rows, ld_a, 64, 32, kSw128))
    return cudaErrorInvalidValue;
  auto run = [&](auto BNC, auto P) {
    constexpr int BN = decltype(BNC)::value;
    constexpr bool PAIR = decltype(P)::value;
    constexpr int rows = PAIR ? BN / 2 : BN;
    const uint64_t K = D.K, N = D.N, E = D.E;
    bool ok;
    if (a.blocks_k) {
      const uint64_t dims[4] = {64, N, K / 64, E}, strides[3] = {K * 2, 128, N * K * 2};
      const uint32_t box[4] = {64, 64, rows / 64, 1};
      ok = make_tensor_map(&tb, kBf, w, 4, dims, strides, box, kSw128);
    } else {
      const uint64_t dims[3] = {K, N, E}, strides[2] = {K * 2, N * K * 2};
      const uint32_t box[3] = {64, MODE == GRP_FWD ? rows : 64, 1};
      ok = make_tensor_map(&tb, kBf, w, 3, dims, strides, box, kSw128);
    }
    if (!ok) return cudaErrorInvalidValue;
    a.n_tiles = static_cast<int>((cols + BN - 1) / BN);
    const long long units = most_tiles(D, PAIR ? 256 : 128) * a.n_tiles;
    return f32 || a.round16
               ? launch<MODE, BN, true, PAIR>(name, ta, tb, ta2, tb, ta, a, units, st)
               : launch<MODE, BN, false, PAIR>(name, ta, tb, ta2, tb, ta, a, units, st);
  };
  using Yes = std::true_type;
  using No = std::false_type;
  // Narrow tiles where wide ones would leave SMs without work (256 rows in 4 groups,
  // N = K = 1024: 14.5 us, wide 16.8; 16384 in 64, N = K = 2048: 176 and 146).
  if (most_tiles(D, 128) * ((cols + 255) / 256) < kGb300Sms)
    return run(std::integral_constant<int, 128>(), No());
  // Pairs halve what an SM reads per product, and round a group up to 256 rows (N = K
  // = 2048, even groups of 192 rows: 121 us, one CTA a tile 128; 256: alike; 512: 211
  // and 222; 4096: 160 and 173; zipf groups of 128 rows on average, 4096 x 1536: 335
  // and 314).  (Short tiles with the weights as the MMA's M, or all of them so, won 2%
  // where groups end in them and lost 4% elsewhere.)
  if (D.rows >= 160LL * D.E) return run(std::integral_constant<int, 256>(), Yes());
  return run(std::integral_constant<int, 256>(), No());
}

}  // namespace

cudaError_t launch_grouped_fwd(const mok_grouped_desc& D, const void* x, const void* w,
                               const int32_t* offsets, void* y, int* status, cudaStream_t st) {
  return rows_product<GRP_FWD>("grouped_linear", D, x, D.ld_x, D.K, w, y, D.ld_y, D.N,
                               D.y_elem == MOK_ELEM_F32, offsets, status, st);
}

cudaError_t launch_grouped_dx(const mok_grouped_desc& D, const void* dy, const void* w,
                              const int32_t* offsets, void* dx, int* status, cudaStream_t st) {
  return rows_product<GRP_DX>("grouped_linear_dx", D, dy, D.ld_y, D.N, w, dx, D.ld_dx, D.K,
                              D.dx_elem == MOK_ELEM_F32, offsets, status, st);
}

// out (+)= the sum of `n` parts, in a fixed order.  Each warp sums every eighth part of
// 32 words (W = 8, for few words) or each thread all parts of one (W = 1).
template <int W>
__global__ void __launch_bounds__(256)
    grouped_sum_kernel(const float4* part, int n, long long words, float4* out, int accumulate) {
  __shared__ float4 s_sum[8][32];
  grid_dep_launch();
  grid_dep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, first = W == 8 ? warp : 0;
  const long long i = W == 8 ? blockIdx.x * 32ll + lane : blockIdx.x * 256ll + threadIdx.x;
  const auto add = [](float4& v, const float4& u) {
    v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
  };
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (i < words) {
#pragma unroll 10
    for (int s = first; s < n; s += W) add(v, part[s * words + i]);
  }
  if (W == 8) {
    s_sum[warp][lane] = v;
    __syncthreads();
    if (warp != 0) return;
#pragma unroll
    for (int w = 1; w < 8; ++w) add(v, s_sum[w][lane]);
  }
  if (i >= words) return;
  if (accumulate) add(v, out[i]);
  out[i] = v;
}

// Parts of the groups' rows that dw is summed in: as many as give every SM a tile
// where there are fewer tiles of 128 x 128, none of less than 512 rows on average.  (A
// group of 131072 rows, N = K = 64: one CTA's 2048 K blocks in a row otherwise.)
static int dw_splits(const mok_grouped_desc& D) {
  const long long tiles = D.E * ((D.N + 127) / 128) * ((D.K + 127) / 128);
  long long s = kGb300Sms / tiles;
  if (s > D.rows / (512LL * D.E)) s = D.rows / (512LL * D.E);
  return static_cast<int>(s < 1 ? 1 : s);
}

size_t grouped_ws_bytes(const mok_grouped_desc& D) {
  const int s = dw_splits(D);
  return s > 1 ? static_cast<size_t>(s) * D.E * D.N * D.K * 4 : 0;
}

cudaError_t launch_grouped_dw(const mok_grouped_desc& D, const void* dy, const void* x,
                              const int32_t* offsets, float* dw, void* ws, int* status,
                              cudaStream_t st) {
  const bool add = (D.accumulate & MOK_ADD_DW) != 0;
  if (D.rows == 0)
    return add ? cudaSuccess : cudaMemsetAsync(dw, 0, static_cast<size_t>(D.E) * D.N * D.K * 4, st);
  GroupedArgs a = {};
  a.offsets = offsets;
  a.E = D.E;
  a.R = static_cast<int>(D.rows);
  a.rows_w = static_cast<int>(D.N);
  a.cols = static_cast<int>(D.K);
  a.splits = dw_splits(D);
  a.accumulate = add && a.splits == 1;
  a.chunk_kb = kChunkKb;
  a.status = status;
  CUtensorMap ta, tb, ta2, tb2, tc;
  const uint64_t K = D.K, N = D.N, E = D.E;
  a.blocks_n = N % 64 == 0;
  a.blocks_k = K % 64 == 0;
  // boxes of `rows` rows and one or (whole) n blocks of 64 columns
  auto col_map = [&](CUtensorMap* m, const void* p, uint64_t cols, int64_t ld, int whole, int n,
                     uint32_t rows) {
    const uint64_t stride = static_cast<uint64_t>(ld) * 2, R = D.rows;
    const uint64_t dims[3] = {whole ? 64 : cols, R, cols / 64}, strides[2] = {stride, 128};
    const uint32_t box[3] = {64, rows, static_cast<uint32_t>(n)};
    return make_tensor_map(m, kBf, p, whole ? 3 : 2, dims, strides, box, kSw128);
  };
  const uint64_t dims[3] = {K, N, E * a.splits}, strides[2] = {K * 4, N * K * 4};
  const uint32_t box[3] = {32, 32, 1};
  if (!col_map(&ta, dy, N, D.ld_y, a.blocks_n, 2, 64) ||
      !col_map(&ta2, dy, N, D.ld_y, a.blocks_n, 2, 16) ||
      !make_tensor_map(&tc, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, a.splits > 1 ? ws : dw, 3, dims,
                       strides, box, kSw128))
    return cudaErrorInvalidValue;
  auto run = [&](auto BNC, auto P) {
    constexpr int BN = decltype(BNC)::value;
    constexpr bool PAIR = decltype(P)::value;
    constexpr int blocks = (PAIR ? BN / 2 : BN) / 64;
    if (!col_map(&tb, x, K, D.ld_x, a.blocks_k, blocks, 64) ||
        !col_map(&tb2, x, K, D.ld_x, a.blocks_k, blocks, 16))
      return cudaErrorInvalidValue;
    a.m_tiles = static_cast<int>((D.N + (PAIR ? 255 : 127)) / (PAIR ? 256 : 128));
    a.n_tiles = static_cast<int>((D.K + BN - 1) / BN);
    return launch<GRP_DW, BN, true, PAIR>("grouped_linear_dw", ta, tb, ta2, tb2, tc, a,
                                          static_cast<long long>(D.E) * a.splits * a.m_tiles *
                                              a.n_tiles,
                                          st);
  };
  using Yes = std::true_type;
  using No = std::false_type;
  if (a.splits > 1) {
    cudaError_t e = run(std::integral_constant<int, 128>(), No());
    if (e != cudaSuccess) return e;
    const long long words = D.E * D.N * D.K / 4;  // (at most 152 tiles of 128 x 128)
    ProfScope prof("grouped_linear_dw_sum", st);
    const bool few = words < 64LL * kGb300Sms;
    e = launch_dependent(few ? grouped_sum_kernel<8> : grouped_sum_kernel<1>,
                         dim3(static_cast<unsigned>(few ? (words + 31) / 32 : (words + 255) / 256)),
                         dim3(256), 0, st, static_cast<const float4*>(ws), a.splits, words,
                         reinterpret_cast<float4*>(dw), add ? 1 : 0);
    count_launch();
    return e != cudaSuccess ? e : cudaGetLastError();
  }
  if (static_cast<long long>(D.E) * ((D.N + 127) / 128) * ((D.K + 255) / 256) < kGb300Sms)
    return run(std::integral_constant<int, 128>(), No());
  // Short groups are bound by the stores of dw, which single CTAs do better (64
  // groups, N = K = 2048: 64 rows each 194 us, pairs 201; 256 rows 221 and 265; 384
  // alike; 512 rows 328 and 279, 4096 rows 227 and 199).
  if (D.rows >= 384LL * D.E && D.N > 128) return run(std::integral_constant<int, 256>(), Yes());
  return run(std::integral_constant<int, 256>(), No());
}

}  // namespace mok
