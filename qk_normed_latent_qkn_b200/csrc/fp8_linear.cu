// qkn_fp8_linear: out = A W^T for rows and a weight in 8 bits with a scale for each block of 128.
//
// Mathematics.  out[i, n] = sum_b sa[b, i] sw[n / 128, b] sum_{k in b} a[i, k] w[n, k].  The products
// of two e4m3 values are exact in fp32; the tensor core sums the 128 of a block into a fresh TMEM
// accumulator, and the epilogue warps enter it into the fp32 total that they keep in registers, with
// the block's two scales.  One rounding, at the end.
//
// Two kernels, both fed by TMA (128-byte swizzled boxes of 128 codes, which zero-fill whatever lies
// behind the last row or column, so no size needs to be a multiple of anything):
//   * linear_pair_kernel, many rows: pairs of CTAs share a tile of 256 rows x 256 or 128 columns
//     (cta_group::2), persistent over the tiles;
//   * linear_split_kernel, few tiles: a tile is 128 columns of the product x 16 to 128 rows.  Up to 64
//     rows the weight's columns take the tensor core's M and the rows its N; 128 rows take M themselves,
//     because a row's scale is then one factor of the lane's.  A cluster of up to 8 CTAs splits K and
//     joins through distributed shared memory.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <atomic>

#include "common.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace qkn {

using namespace sm100;

struct LinearMaps {
  CUtensorMap a, w, a_scale;
};

namespace {

constexpr int kRowBytes = 128;                  // codes of one block of K in a tile row
constexpr int kTileBytes = 128 * kRowBytes;     // 128 rows of a tile
constexpr int kKStep = 32;                      // K of one MMA
constexpr uint32_t kDescStep = kKStep >> 4;     // the same in descriptor units

// Whether runs of E columns that start at multiples of E can be written as one piece.
template <typename O, int E>
__device__ __forceinline__ bool wide_ok(const OutCols& o) {
  return reinterpret_cast<uintptr_t>(o.out) % (E * sizeof(O)) == 0 && o.ld % E == 0 && o.begin % E == 0;
}

// A scale.  The kernel before this one may still be writing it when this one starts, so it is neither read
// through the read-only path (which __ldg takes: what it reads must not change while the kernel runs) nor
// moved: not above the wait for that kernel, nor, where it is asked for early, down to its use.
__device__ __forceinline__ float load_scale(const float* p) {
  float v;
  asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}

// One warp's 32 rows x ROW / sizeof(O) columns of the product pass through `box` (ROW = 128 or 256 bytes a row)
// from lanes that hold a row each to lanes that write ROW consecutive bytes of a row: straight from the
// registers every lane's 16 bytes would be a half-written sector of another row.  The 16-byte pieces of
// row r are permuted by r % 8, which keeps both sides free of bank conflicts.
constexpr int kBoxBytes = 32 * 256;

template <typename O, int ROW>
__device__ __forceinline__ void fill_box(uint8_t* box, const float* v) {
  constexpr int E = 16 / (int)sizeof(O);
  const int lane = threadIdx.x & 31;
  uint8_t* row = box + lane * ROW;
#pragma unroll
  for (int u = 0; u < ROW / 16; ++u) {
    uint4 w;
    if constexpr (sizeof(O) == 4) {
      w = make_uint4(__float_as_uint(v[u * E]), __float_as_uint(v[u * E + 1]), __float_as_uint(v[u * E + 2]),
                     __float_as_uint(v[u * E + 3]));
    } else {
      __nv_bfloat162 t[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) t[i] = __floats2bfloat162_rn(v[u * E + 2 * i], v[u * E + 2 * i + 1]);
      w = make_uint4(*reinterpret_cast<uint32_t*>(&t[0]), *reinterpret_cast<uint32_t*>(&t[1]),
                     *reinterpret_cast<uint32_t*>(&t[2]), *reinterpret_cast<uint32_t*>(&t[3]));
    }
    *reinterpret_cast<uint4*>(row + ((u ^ (lane & 7)) << 4)) = w;
  }
  __syncwarp();
}

template <typename O, int ROW>
__device__ __forceinline__ void write_box(const Fp8LinearArgs& p, const uint8_t* box, int row0, int col0) {
  constexpr int E = 16 / (int)sizeof(O), PIECES = ROW / 16, COLS = PIECES * E;
  const int lane = threadIdx.x & 31;
  if (col0 < p.n) {
    int o = 0;
    while (col0 >= p.outs[o].end) ++o;
    const int rows = min(32, p.m - row0);
    if (col0 + COLS <= p.outs[o].end && wide_ok<O, E>(p.outs[o])) {
      const int u = lane % PIECES;
      O* dst = static_cast<O*>(p.outs[o].out) + (col0 - p.outs[o].begin) + u * E;
      for (int r = lane / PIECES; r < rows; r += 32 / PIECES)
        *reinterpret_cast<uint4*>(dst + (row0 + r) * p.outs[o].ld) =
            *reinterpret_cast<const uint4*>(box + r * ROW + ((u ^ (r & 7)) << 4));
    } else if (col0 + COLS <= p.outs[o].end) {
      // Rows off the 16-byte grid: lane u writes the u-th aligned 16 bytes of a row, shifted out of two pieces,
      // and the E elements at the row's two ends go one to a lane.
      const int u = lane % PIECES;
      for (int r = lane / PIECES; r < rows; r += 32 / PIECES) {
        O* dst = static_cast<O*>(p.outs[o].out) + (row0 + r) * p.outs[o].ld + (col0 - p.outs[o].begin);
        const uint8_t* from = box + r * ROW;
        const uint32_t s = (0u - (uint32_t)reinterpret_cast<uintptr_t>(dst)) & 15;   // bytes before the grid
        if (u < PIECES - 1 || s == 0) {
          const uint4 a = *reinterpret_cast<const uint4*>(from + ((u ^ (r & 7)) << 4));
          const uint4 b = *reinterpret_cast<const uint4*>(from + ((min(u + 1, PIECES - 1) ^ (r & 7)) << 4));
          uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
          if (s & 8) {
#pragma unroll
            for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
          }
          if (s & 4) {
#pragma unroll
            for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
          }
          if constexpr (sizeof(O) == 2) {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], (s & 2) * 8);
          }
          *reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(dst) + s + 16 * u) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        if (s != 0 && u < E) {
          const int e = u < (int)(s / sizeof(O)) ? u : COLS - E + u;
          dst[e] = *reinterpret_cast<const O*>(from + (((e / E) ^ (r & 7)) << 4) + (e % E) * sizeof(O));
        }
      }
    } else {   // a destination ends inside the box: element by element
      for (int e = lane; e < COLS && col0 + e < p.n; e += 32) {
        while (col0 + e >= p.outs[o].end) ++o;
        O* dst = static_cast<O*>(p.outs[o].out) + (col0 + e - p.outs[o].begin);
        for (int r = 0; r < rows; ++r)
          dst[(row0 + r) * p.outs[o].ld] =
              *reinterpret_cast<const O*>(box + r * ROW + (((e / E) ^ (r & 7)) << 4) + (e % E) * sizeof(O));
      }
    }
  }
  __syncwarp();
}

// ---------------------------------------------------------------- many rows: CTA pairs
// A pair's tile halves what each SM has to fetch of the weight (32 KB a block of K for 256 x 256 outputs,
// and the L2 link of an SM brings about 64 bytes a cycle).  The scales of a block enter in fp32, so every
// block's sums leave tensor memory: the MMAs of a block (512 cycles of an SM at 256 columns) fill one
// accumulator while eight warps promote the other.  The promotion's latency bounds the kernel, not a unit's rate: 835
// cycles a block on a B200, 683 without its FMAs, 607 without it, while the tensor pipe is 58 % busy, the issue
// slots 53 % and the FMA pipe 33 %.  8192 x 25152 x 4096: 890 to 940 us, 1.8 to 1.9 PFLOP/s at 1.4 GHz, the
// power cap's doing (765 us in bursts at 1.6); 4096 x 4096 x 16384: 295 to 315 us.  Sixteen promoting warps were
// slower (they leave 96 registers each), as were half-width accumulators and packed FMAs.
constexpr int kPairM = 256;                     // rows of a pair's tile
constexpr int kPairWarps = 8;                   // epilogue warps, each 32 rows x half the tile's columns
constexpr int kPairThreads = 64 + 32 * kPairWarps;
constexpr int kPairGroupM = 16;                 // row tiles that are walked before the next column tile
constexpr int kLoadCols = 16;                   // columns of one TMEM load

// N columns of a pair's tile: 256, or 128 where that fills the waves better.
template <int N>
struct PairCfg {
  static constexpr int kHalfBytes = N / 2 * kRowBytes;            // this CTA's half of the tile's weight rows
  static constexpr int kStageBytes = kTileBytes + kHalfBytes;     // and its 128 rows of A
  static constexpr int kStages = N == 256 ? 5 : 6;
  static constexpr int kAccs = 512 / N;                           // accumulators in tensor memory
  static constexpr int kCols = N / 2;                             // columns of an epilogue warp
  static constexpr int kBoxOff = kStages * kStageBytes;
  static constexpr int kBarOff = kBoxOff + kPairWarps * kBoxBytes;
  static constexpr int kSmem = 1024 + kBarOff + 256;
  static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
};

template <int S, int A>
struct PairBars {
  uint64_t full[S], empty[S];
  uint64_t t_full[A], t_empty[A];
  uint32_t tmem;
  // For the way out after a wait that ran out, in both CTAs of the pair alike: whether one did, the blocks
  // that each CTA's producer asked for, and the blocks that went to the tensor core.
  uint32_t failed, issued[2], computed;
};

// Waits for the last uses, up to `uses`, of a ring of n mbarriers.  (A call: the loops that are never gone
// through stay out of the kernels' registers.)
__device__ __noinline__ void wait_last(uint32_t bars, int n, int uses) {
  for (int u = uses > n ? uses - n : 0; u < uses; ++u)
    (void)mbar_wait_warp(bars + (uint32_t)(u % n) * 8, (uint32_t)(u / n) & 1u, kLinearWaitCycles);
}

template <int N>
struct TileWalk {
  int mt, nt;
  __device__ __forceinline__ explicit TileWalk(const Fp8LinearArgs& p)
      : mt((p.m + kPairM - 1) / kPairM), nt((p.n + N - 1) / N) {}
  __device__ __forceinline__ void of(int t, int& m, int& n) const {
    const int g = t / (kPairGroupM * nt);
    const int rows = min(kPairGroupM, mt - g * kPairGroupM);
    const int r = t - g * kPairGroupM * nt;
    m = g * kPairGroupM + r % rows;
    n = r / rows;
  }
};

// Warps: 0 producer, 1 MMA (the even CTA issues for both), 2-9 epilogue (each CTA its 128 rows; warps
// 2-5 the first half of the tile's columns, 6-9 the second).
template <int N, typename O, bool STOP>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    linear_pair_kernel(const __grid_constant__ Fp8LinearArgs p, const __grid_constant__ LinearMaps maps) {
  using C = PairCfg<N>;
  extern __shared__ __align__(16) uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t{1023});
  auto& bars = *reinterpret_cast<PairBars<C::kStages, C::kAccs>*>(smem + C::kBarOff);
  static_assert(sizeof(bars) <= 256, "barriers");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const uint32_t stages = smem_u32(smem);

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(smem_u32(&bars.full[i]), 1);
      mbar_init(smem_u32(&bars.empty[i]), 1);
    }
    for (int i = 0; i < C::kAccs; ++i) {
      mbar_init(smem_u32(&bars.t_full[i]), 1);
      mbar_init(smem_u32(&bars.t_empty[i]), 2 * kPairWarps);   // of both CTAs
    }
    bars.failed = bars.issued[0] = bars.issued[1] = bars.computed = 0;
    mbar_fence_init();
    prefetch_tmap(&maps.a);
    prefetch_tmap(&maps.w);
  }
  __syncthreads();
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(&bars.tmem), 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = bars.tmem;
  pdl_trigger();
  pdl_wait();

  const TileWalk<N> walk(p);
  const int tiles = walk.mt * walk.nt;   // (the launcher checks that they fit)
  const int blocks = (p.k + kFp8Group - 1) / kFp8Group;
  const int pairs = gridDim.x >> 1;
  bool ok = true;

  const auto tell = [&](uint32_t& word, uint32_t v) {   // both CTAs (the cluster barrier below orders it)
    for (uint32_t r = 0; r < 2; ++r) st_shared_remote_u32(mapa_shared(smem_u32(&word), r), v);
  };

  if (warp == 0) {
    const int stop = STOP && p.test_stop == 1 + (int)rank ? p.test_at : INT32_MAX;
    RingPos<C::kStages> ring;
    int uses = 0;
    for (int t = blockIdx.x >> 1; ok && t < tiles; t += pairs) {
      int m, n;
      walk.of(t, m, n);
      const int y_a = m * kPairM + (int)rank * 128, y_w = n * N + (int)rank * (N / 2);
      int b = 0;
      for (const int to = min(blocks, stop - uses); b < to; ++b) {
        if (!mbar_wait_warp(smem_u32(&bars.empty[ring.slot]), ring.phase ^ 1u, p.wait_limit)) break;
        const uint32_t full = smem_u32(&bars.full[ring.slot]);
        if (rank == 0) mbar_arrive_expect_tx_elect(full, 2 * C::kStageBytes);
        const uint32_t dst = stages + ring.slot * C::kStageBytes;
        const uint32_t bar = mapa_shared(full, 0);
        tma_load_2d_pair_elect(dst, &maps.a, b * kFp8Group, y_a, bar);
        tma_load_2d_pair_elect(dst + kTileBytes, &maps.w, b * kFp8Group, y_w, bar);
        ring.next();
      }
      uses += b;
      ok = b == blocks;
    }
    // the last uses of the stages end before this CTA does: their commits arrive here
    for (int i = 0; i < C::kStages; ++i) {
      if (ok && !mbar_wait_warp(smem_u32(&bars.empty[ring.slot]), ring.phase ^ 1u, p.wait_limit)) ok = false;
      ring.next();
    }
    if (lane == 0) tell(bars.issued[rank], uses);
  } else if (warp == 1 && rank == 0) {
    constexpr uint32_t idesc = idesc_e4m3(256, N);
    const uint64_t d_a = smem_desc(stages, 16, 1024), d_w = smem_desc(stages + kTileBytes, 16, 1024);
    const int stop = STOP && p.test_stop == 3 ? p.test_at : INT32_MAX;
    RingPos<C::kStages> ring;
    RingPos<C::kAccs> acc;
    int uses = 0;
    for (int t = blockIdx.x >> 1; ok && t < tiles; t += pairs) {
      int b = 0;
      for (const int to = min(blocks, stop - uses); b < to; ++b) {
        if (!mbar_wait_warp(smem_u32(&bars.full[ring.slot]), ring.phase, p.wait_limit) ||
            !mbar_wait_warp(smem_u32(&bars.t_empty[acc.slot]), acc.phase ^ 1u, p.wait_limit))
          break;
        tc_fence_after();
        const uint64_t at = (uint64_t)((ring.slot * C::kStageBytes) >> 4);
#pragma unroll
        for (int s = 0; s < kFp8Group / kKStep; ++s)
          mma_e4m3_pair_elect(tmem + acc.slot * N, d_a + at + s * kDescStep, d_w + at + s * kDescStep, idesc,
                              s > 0);
        mma_commit_group2_elect(smem_u32(&bars.empty[ring.slot]), 3);
        mma_commit_group2_elect(smem_u32(&bars.t_full[acc.slot]), 3);
        ring.next();
        acc.next();
      }
      uses += b;
      ok = b == blocks;
    }
    if (lane == 0) tell(bars.computed, uses);
  } else if (warp >= 2) {
    const int quad = warp & 3, half = (warp - 2) >> 2;
    uint8_t* box = smem + C::kBoxOff + (warp - 2) * kBoxBytes;
    const uint32_t tq = tmem + ((uint32_t)(quad * 32) << 16) + half * C::kCols;
    if (STOP && p.test_stop == 4 && warp == 2) ok = false;
    RingPos<C::kAccs> acc;
    float total[C::kCols];
    // One block of K: its sums leave TMEM 16 columns at a time, the next ones on their way while these
    // enter the total.  (Single FMAs: as packed pairs they need the same FMA cycles and, with the moves
    // that pair up registers, more instructions.)
    auto enter = [&](float s) {
      if (ok && !mbar_wait_warp(smem_u32(&bars.t_full[acc.slot]), acc.phase, p.wait_limit)) ok = false;
      tc_fence_after();
      const uint32_t at = tq + acc.slot * N;
      constexpr int L = C::kCols / kLoadCols;
      uint32_t v[2][kLoadCols];
      tmem_ld16(at, v[0]);
      tmem_wait_ld(v[0]);
#pragma unroll
      for (int c = 0; c < L; ++c) {
        if (c < L - 1) tmem_ld16(at + (c + 1) * kLoadCols, v[(c + 1) & 1]);
#pragma unroll
        for (int e = 0; e < kLoadCols; ++e)
          total[c * kLoadCols + e] = fmaf(__uint_as_float(v[c & 1][e]), s, total[c * kLoadCols + e]);
        if (c < L - 1) tmem_wait_ld(v[(c + 1) & 1]);
        if (c == L - 2) {   // everything is out of TMEM
          tc_fence_before();
          __syncwarp();
          // (relaxed: what the arrival stands for, the loads from TMEM, is complete, and a release would
          // wait for the scales' loads too)
          if (lane == 0) mbar_arrive_remote(mapa_shared(smem_u32(&bars.t_empty[acc.slot]), 0));
        }
      }
      acc.next();
    };
    // The scales of a tile's blocks, one of this lane's row and one of the warp's 128 columns, are asked
    // for two blocks ahead.
    for (int t = blockIdx.x >> 1; ok && t < tiles; t += pairs) {
      int m, n;
      walk.of(t, m, n);
      const float* sa = p.a_scale + min(m * kPairM + (int)rank * 128 + quad * 32 + lane, p.m - 1);
      const float* sw = p.w_scale + (int64_t)min((n * N + half * C::kCols) / kFp8Group, (p.n - 1) / kFp8Group) * blocks;
      const int b1 = blocks > 1 ? 1 : 0;
      float s0 = load_scale(sa) * load_scale(sw), s1 = load_scale(sa + b1 * p.ld_as) * load_scale(sw + b1);
#pragma unroll
      for (int i = 0; i < C::kCols; ++i) total[i] = 0.f;
      for (int b = 0; b < blocks; b += 2) {
        const int b2 = min(b + 2, blocks - 1), b3 = min(b + 3, blocks - 1);
        const float a2 = load_scale(sa + b2 * p.ld_as), w2 = load_scale(sw + b2);
        enter(s0);
        const float a3 = load_scale(sa + b3 * p.ld_as), w3 = load_scale(sw + b3);
        if (b + 1 < blocks) enter(s1);
        s0 = a2 * w2;
        s1 = a3 * w3;
      }
      if (ok) {
        walk.of(t, m, n);
        constexpr int ROW = C::kCols * (int)sizeof(O) < 256 ? C::kCols * (int)sizeof(O) : 256;
        constexpr int COLS = ROW / (int)sizeof(O);
#pragma unroll
        for (int c = 0; c < C::kCols; c += COLS) {
          fill_box<O, ROW>(box, total + c);
          write_box<O, ROW>(p, box, m * kPairM + (int)rank * 128 + quad * 32, n * N + half * C::kCols + c);
        }
      }
    }
  }
  __syncwarp();
  if (!ok && lane == 0) {
    record_status(p.status, QKN_ERR_TIMEOUT);
    tell(bars.failed, 1);
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  if (__builtin_expect(bars.failed, 0)) {
    // A role gave up, and the others after it, at blocks of their own.  Nothing may be in flight when a CTA
    // leaves.  First the MMAs, and with them their arrivals in both CTAs.  Then the copies: all of a block's
    // complete on the even CTA's mbarrier, which was told to expect both CTAs' bytes, so a block that one CTA
    // has asked for and the other has not would never be complete.  The other asks for it now.  (A producer
    // that asked for a block had seen its stage's last use end, so that use's copies have arrived in both
    // CTAs, the two are at most a ring apart, and no MMA reads the stage any more.  Which bytes come is
    // all the same; the same tile corner is in bounds, or zeros.)
    if (warp == 0) {
      wait_last(smem_u32(bars.empty), C::kStages, bars.computed);
      wait_last(smem_u32(bars.t_full), C::kAccs, bars.computed);
    }
    cluster_sync();
    if (warp == 0) {
      const int uses = max(bars.issued[0], bars.issued[1]);
      for (int u = bars.issued[rank]; u < uses; ++u) {
        const int slot = u % C::kStages;
        const uint32_t full = smem_u32(&bars.full[slot]), dst = stages + slot * C::kStageBytes;
        if (rank == 0) mbar_arrive_expect_tx_elect(full, 2 * C::kStageBytes);
        tma_load_2d_pair_elect(dst, &maps.a, 0, 0, mapa_shared(full, 0));
        tma_load_2d_pair_elect(dst + kTileBytes, &maps.w, 0, 0, mapa_shared(full, 0));
      }
      if (rank == 0) wait_last(smem_u32(bars.full), C::kStages, uses);
    }
    cluster_sync();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// ---------------------------------------------------------------- few rows: K split over a cluster
template <int NT>
struct SplitCfg {
  static constexpr bool kRows = NT == 128;                               // the rows take the tensor core's M
  static constexpr int kWarps = NT == 16 ? 4 : 8;                         // epilogue warps, each 32 lanes x
  static constexpr int kPart = NT * 4 / kWarps;                          // kPart columns of the accumulator
  static constexpr int kPitch = kRows ? 132 : 128;                       // floats of a row of partial sums
  static constexpr int kThreads = 64 + 32 * kWarps;                       // (and the producer, the MMA)
  static constexpr int kPerSm = NT == 128 ? 1 : 2;                       // CTAs on an SM (registers, shared memory)
  // CTAs that the registers are shared out for; 64 rows are faster without (19.2 us for 18.4 at 64 x 4096 x 16384),
  // the others with (32 x 25152 x 4096: 21.2 for 22.3; 128 x 4096 x 16384: 18.1 for 19.6)
  static constexpr int kBound = NT == 64 ? 0 : kPerSm;
  static constexpr int kStageBytes = kTileBytes + NT * kRowBytes;         // weight, rows
  static constexpr int kStages = NT == 128 ? 6 : NT == 64 ? 4 : 5;
  static constexpr int kCols = NT < 32 ? 32 : NT;                        // TMEM columns of one accumulator
  static constexpr int kAccs = 4;
  // The rows' scales have a ring of their own, so that a stage is free as soon as the tensor core has
  // read it.  Its slots need no "empty" barrier: block b is loaded after the MMAs of block b - kStages
  // were issued, hence after the epilogue has left block b - kStages - kAccs.
  static constexpr int kScaleSlots = 16;
  static constexpr int kScaleBytes = NT * 4 < 128 ? 128 : NT * 4;        // a slot; copies land on 128-byte boundaries
  static_assert(kScaleSlots > kStages + kAccs, "scale slots are reused too early");
  static constexpr int kScaleOff = kStages * kStageBytes;
  static constexpr int kBarOff = kScaleOff + kScaleSlots * kScaleBytes;
  static constexpr int kSmem = 1024 + kBarOff + 512;
  static_assert(kSmem * kPerSm <= (227 - kPerSm) * 1024, "shared memory of an SM");
  static_assert(NT * kPitch * 4 <= kScaleOff, "the partial sums reuse the stages");
  static_assert(kScaleOff % 128 == 0 && kScaleBytes % 128 == 0, "a copy's destination");
  static_assert(kTileBytes % 1024 == 0 && kStageBytes % 1024 == 0, "swizzled tiles start on 1024 bytes");
};

template <int S, int A>
struct SplitBars {
  uint64_t full[S], empty[S];
  uint64_t t_full[A], t_empty[A];
  uint32_t tmem;
  uint32_t failed, issued, computed;   // as in PairBars
};

// Bound by memory or, in short calls, by the chain of one load, MMA, promotion and join: 32 x 25152 x 4096
// takes 21 us on a B200 (103 MB of weight; 7 TB/s once it streams, 5 us to start and end), 1 x 576 x 2048 3.6, and
// 64 x 4096 x 16384 18.4 (256 CTAs on 148 SMs: 108 of these carry two).  Splitting K over a cluster needs no workspace and no atomics, and the parts are
// added in rank order: the same bits every time.
// One tile: 128 columns of the product for NT rows.  Cluster rank r takes the r-th part of K's blocks.
// Warps: 0 producer, 1 MMA, 2 on: epilogue.
template <int NT, typename O, bool STOP>
__global__ void __launch_bounds__(SplitCfg<NT>::kThreads, SplitCfg<NT>::kBound)
    linear_split_kernel(const __grid_constant__ Fp8LinearArgs p, const __grid_constant__ LinearMaps maps, int split,
                        int row_tiles) {
  using C = SplitCfg<NT>;
  extern __shared__ __align__(16) uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t{1023});
  auto& bars = *reinterpret_cast<SplitBars<C::kStages, C::kAccs>*>(smem + C::kBarOff);
  static_assert(sizeof(bars) <= 512, "barriers");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x % split;                     // (clusters lie along x)
  const int tile = blockIdx.x / split;
  const int row0 = (tile % row_tiles) * NT, n0 = (tile / row_tiles) * 128;
  const int rows = min(NT, p.m - row0);
  const int blocks = (p.k + kFp8Group - 1) / kFp8Group;
  const int b0 = (int)((int64_t)blocks * rank / split), b1 = (int)((int64_t)blocks * (rank + 1) / split);
  const uint32_t stages = smem_u32(smem);

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(smem_u32(&bars.full[i]), 1);
      mbar_init(smem_u32(&bars.empty[i]), 1);
    }
    for (int i = 0; i < C::kAccs; ++i) {
      mbar_init(smem_u32(&bars.t_full[i]), 2);             // the MMA warp, and its MMAs when they are done
      mbar_init(smem_u32(&bars.t_empty[i]), C::kWarps);
    }
    bars.failed = 0;
    mbar_fence_init();
    prefetch_tmap(&maps.a);
    prefetch_tmap(&maps.w);
    prefetch_tmap(&maps.a_scale);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&bars.tmem), C::kCols * C::kAccs);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem;
  pdl_trigger();
  pdl_wait();

  float total[C::kPart];
  if (warp == 0) {
    RingPos<C::kStages> ring;
    RingPos<C::kScaleSlots> sring;
    int b = b0;
    for (const int to = STOP && (p.test_stop == 1 || p.test_stop == 2) ? min(b1, b0 + p.test_at) : b1; b < to; ++b) {
      if (!mbar_wait_warp(smem_u32(&bars.empty[ring.slot]), ring.phase ^ 1u, p.wait_limit)) break;
      const uint32_t full = smem_u32(&bars.full[ring.slot]);
      const uint32_t dst = stages + ring.slot * C::kStageBytes;
      mbar_arrive_expect_tx_elect(full, C::kStageBytes + NT * 4);
      tma_load_2d_elect(dst, &maps.w, b * kFp8Group, n0, full);
      tma_load_2d_elect(dst + kTileBytes, &maps.a, b * kFp8Group, row0, full);
      tma_load_2d_elect(stages + C::kScaleOff + sring.slot * C::kScaleBytes, &maps.a_scale, row0, b, full);
      ring.next();
      sring.next();
    }
    if (lane == 0) bars.issued = b - b0;
    bool ok = b == b1;
    for (int i = 0; ok && i < C::kStages; ++i) {            // nothing of this CTA's is in flight after this
      ok = mbar_wait_warp(smem_u32(&bars.empty[ring.slot]), ring.phase ^ 1u, p.wait_limit);
      ring.next();
    }
    if (!ok && lane == 0) bars.failed = 1;
  } else if (warp == 1) {
    constexpr uint32_t idesc = idesc_e4m3(128, NT);
    const uint64_t d_w = smem_desc(stages, 16, 1024), d_a = smem_desc(stages + kTileBytes, 16, 1024);
    const uint64_t d_m = C::kRows ? d_a : d_w, d_n = C::kRows ? d_w : d_a;
    RingPos<C::kStages> ring;
    RingPos<C::kAccs> acc;
    int b = b0;
    for (const int to = STOP && p.test_stop == 3 ? min(b1, b0 + p.test_at) : b1; b < to; ++b) {
      if (!mbar_wait_warp(smem_u32(&bars.t_empty[acc.slot]), acc.phase ^ 1u, p.wait_limit) ||
          !mbar_wait_warp(smem_u32(&bars.full[ring.slot]), ring.phase, p.wait_limit))
        break;
      tc_fence_after();
      const uint64_t at = (uint64_t)((ring.slot * C::kStageBytes) >> 4);
#pragma unroll
      for (int s = 0; s < kFp8Group / kKStep; ++s)
        mma_e4m3_elect(tmem + acc.slot * C::kCols, d_m + at + s * kDescStep, d_n + at + s * kDescStep, idesc, s > 0);
      mma_commit_elect(smem_u32(&bars.empty[ring.slot]));
      mma_commit_elect(smem_u32(&bars.t_full[acc.slot]));
      mbar_arrive_elect(smem_u32(&bars.t_full[acc.slot]));   // passes on the scales, which came with the stage
      ring.next();
      acc.next();
    }
    if (lane == 0) bars.computed = b - b0;
    if (b < b1 && lane == 0) bars.failed = 1;
  } else {
    const int quad = warp & 3, part = (warp - 2) >> 2;
    const float* sw = p.w_scale + (int64_t)(n0 / kFp8Group) * blocks;
    RingPos<C::kScaleSlots> sring;
    RingPos<C::kAccs> acc;
#pragma unroll
    for (int i = 0; i < C::kPart; ++i) total[i] = 0.f;
    float sw_lane = 0.f;             // the weight's scales of 32 blocks, one per lane
    int b = b0;
    for (const int to = STOP && p.test_stop == 4 && warp == 2 ? b0 : b1; b < to; ++b) {
      if (((b - b0) & 31) == 0) sw_lane = load_scale(sw + min(b + lane, b1 - 1));
      const float s = __shfl_sync(0xffffffffu, sw_lane, (b - b0) & 31);
      if (!mbar_wait_warp(smem_u32(&bars.t_full[acc.slot]), acc.phase, p.wait_limit)) break;
      tc_fence_after();
      const uint8_t* sa = smem + C::kScaleOff + sring.slot * C::kScaleBytes;
      const uint32_t at = tmem + ((uint32_t)(quad * 32) << 16) + acc.slot * C::kCols + part * C::kPart;
      // 16 sums at a time; the factors are formed, and the next sums asked for, while these are on their way
      uint32_t v[2][16];
      tmem_ld16(at, v[0]);
      const float row_f = C::kRows ? reinterpret_cast<const float*>(sa)[quad * 32 + lane] * s : 0.f;
#pragma unroll
      for (int c = 0; c < C::kPart; c += 16) {
        uint32_t(&u)[16] = v[(c >> 4) & 1];
        float f[16];
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
          if constexpr (C::kRows) {
            f[e] = f[e + 1] = f[e + 2] = f[e + 3] = row_f;
          } else {
            const float4 q = reinterpret_cast<const float4*>(sa)[(part * C::kPart + c + e) >> 2];
            f[e] = q.x * s, f[e + 1] = q.y * s, f[e + 2] = q.z * s, f[e + 3] = q.w * s;
          }
        }
        tmem_wait_ld(u);
        if (c + 16 < C::kPart) tmem_ld16(at + c + 16, v[((c >> 4) & 1) ^ 1]);
#pragma unroll
        for (int e = 0; e < 16; ++e) total[c + e] = fmaf(__uint_as_float(u[e]), f[e], total[c + e]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars.t_empty[acc.slot]));
      sring.next();
      acc.next();
    }
    if (b < b1 && lane == 0) bars.failed = 1;
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  // every stage is free, and the partial sums take their place; after a wait that ran out, once the copies and
  // MMAs in flight have ended
  if (__builtin_expect(bars.failed, 0)) {
    if (threadIdx.x == 0) record_status(p.status, QKN_ERR_TIMEOUT);
    if (warp == 0) {
      wait_last(smem_u32(bars.full), C::kStages, bars.issued);
      wait_last(smem_u32(bars.empty), C::kStages, bars.computed);
      wait_last(smem_u32(bars.t_full), C::kAccs, bars.computed);
    }
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols * C::kAccs);
  }
  float* sums = reinterpret_cast<float*>(smem);             // [rows][kPitch]
  if (warp >= 2) {
    const int i = (warp & 3) * 32 + lane, j0 = ((warp - 2) >> 2) * C::kPart;   // this thread's TMEM lane and columns
    if constexpr (C::kRows) {
      if (i < rows) {
#pragma unroll
        for (int j = 0; j < C::kPart; j += 4)
          *reinterpret_cast<float4*>(sums + i * C::kPitch + j0 + j) =
              make_float4(total[j], total[j + 1], total[j + 2], total[j + 3]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < C::kPart; ++j)
        if (j0 + j < rows) sums[(j0 + j) * C::kPitch + i] = total[j];
    }
  }
  cluster_sync();
  // rank r joins and writes the rows r, r + split, ... : 4 columns per lane, the parts in rank order
  const int col = n0 + lane * 4;
  int o = 0;
  while (o < p.n_outs - 1 && col >= p.outs[o].end) ++o;
  const bool four = col + 4 <= p.outs[o].end && wide_ok<O, 4>(p.outs[o]);
  O* const dst = static_cast<O*>(p.outs[o].out) + (col - p.outs[o].begin);
  for (int j = rank + split * warp; j < rows; j += split * (C::kThreads / 32)) {
    const uint32_t at = smem_u32(sums + j * C::kPitch + lane * 4);
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    for (int r = 0; r < split; ++r) {
      const float4 f = ld_shared_remote_f4(mapa_shared(at, r));
      v[0] += f.x;
      v[1] += f.y;
      v[2] += f.z;
      v[3] += f.w;
    }
    if (four) {
      if constexpr (sizeof(O) == 4) {
        *reinterpret_cast<float4*>(dst + (row0 + j) * p.outs[o].ld) = make_float4(v[0], v[1], v[2], v[3]);
      } else {
        __nv_bfloat162 t[2] = {__floats2bfloat162_rn(v[0], v[1]), __floats2bfloat162_rn(v[2], v[3])};
        *reinterpret_cast<uint2*>(dst + (row0 + j) * p.outs[o].ld) =
            make_uint2(*reinterpret_cast<uint32_t*>(&t[0]), *reinterpret_cast<uint32_t*>(&t[1]));
      }
    } else {   // a destination ends among the four, or its rows are not aligned for them
      for (int e = 0, oe = o; e < 4 && col + e < p.n; ++e) {
        while (col + e >= p.outs[oe].end) ++oe;
        static_cast<O*>(p.outs[oe].out)[(row0 + j) * p.outs[oe].ld + (col + e - p.outs[oe].begin)] = from_f32<O>(v[e]);
      }
    }
  }
  cluster_sync();                                           // no CTA leaves while its parts are read
}

// ---------------------------------------------------------------- host side
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}

bool make_map(CUtensorMap* m, CUtensorMapDataType type, const void* base, uint64_t inner, uint64_t rows,
              uint64_t row_bytes, uint32_t box_inner, uint32_t box_rows, CUtensorMapSwizzle swizzle) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {inner, rows};
  cuuint64_t strides[1] = {row_bytes};
  cuuint32_t box[2] = {box_inner, box_rows};
  cuuint32_t es[2] = {1, 1};
  return fn(m, type, 2, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Codes [rows, k] in boxes of 128 codes x box_rows rows.
bool codes_map(CUtensorMap* m, const uint8_t* codes, int k, int rows, int64_t ld, int box_rows) {
  return make_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, codes, k, rows, ld, kRowBytes, box_rows,
                  CU_TENSOR_MAP_SWIZZLE_128B);
}

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

template <int N, typename O, bool STOP>
cudaError_t launch_pair_as(const Fp8LinearArgs& a, int sms, cudaStream_t st) {
  LinearMaps maps;
  if (!codes_map(&maps.a, a.a, a.k, a.m, a.lda, 128) || !codes_map(&maps.w, a.w, a.k, a.n, a.ldw, N / 2))
    return cudaErrorInvalidValue;
  static PerDeviceOnce attrs;
  cudaError_t e = once_per_device(attrs, [] {
    return cudaFuncSetAttribute(linear_pair_kernel<N, O, STOP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                PairCfg<N>::kSmem);
  });
  if (e != cudaSuccess) return e;
  const int64_t tiles = (int64_t)ceil_div(a.m, kPairM) * ceil_div(a.n, N);
  if (tiles > (1 << 30)) return cudaErrorInvalidConfiguration;
  const int pairs = (int)(tiles < sms / 2 ? tiles : sms / 2);
  return launch_chained(linear_pair_kernel<N, O, STOP>, dim3(2 * pairs), dim3(kPairThreads), PairCfg<N>::kSmem, st, a, maps);
}

// (The instances with STOP are for tests; what they add to the loops would cost up to a twentieth.)
template <int N, typename O>
cudaError_t launch_pair(const Fp8LinearArgs& a, int sms, cudaStream_t st) {
  return a.test_stop ? launch_pair_as<N, O, true>(a, sms, st) : launch_pair_as<N, O, false>(a, sms, st);
}

// Clusters of `size` CTAs that the device holds at once, one CTA per SM: fewer than its SMs' worth, because a
// cluster stays within a group of SMs (148 SMs: 148, 148, 132 and 120 CTAs in clusters of 1, 2, 4 and 8).
template <int NT, typename O>
int clusters_of(int size, int sms) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(size * sms);
  cfg.blockDim = dim3(SplitCfg<NT>::kThreads);
  cfg.dynamicSmemBytes = SplitCfg<NT>::kSmem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = size;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, linear_split_kernel<NT, O, false>, &cfg) != cudaSuccess || n < 1) {
    (void)cudaGetLastError();
    n = 1;
  }
  return n;
}

// CTAs of a split kernel that the device holds at once in clusters of `split` (2, 4 or 8); a cluster too many
// costs a whole wave (32 x 9472 x 4096: 17.8 us in 74 clusters of 4, 11.1 in 74 of 2).  The runtime counts one
// CTA of a kernel with tensor memory per SM.  Where two run there, a cluster needs split / 2 SMs at best and
// split at worst: an estimate two thirds of the way between the two counts, 285 and 256 CTAs for 4 and 8 (B200 runs
// took 272 but not 288, and 264 but not 280, without another wave: for clusters of 8 it is on the safe side).
// Asked once per device.
template <int NT, typename O>
int resident_of(int split, int dev, int sms) {
  static std::atomic<int> known[64][3];
  std::atomic<int>* slot = dev >= 0 && dev < 64 ? &known[dev][split / 4] : nullptr;
  int n = slot ? slot->load(std::memory_order_relaxed) : 0;
  if (n > 0) return n;
  n = clusters_of<NT, O>(split, sms) * split;
  if (SplitCfg<NT>::kPerSm == 2) n = (2 * n + 2 * clusters_of<NT, O>(split / 2, sms) * split) / 3;
  if (slot) slot->store(n, std::memory_order_relaxed);
  return n;
}

// How many parts of K a cluster takes: as many as the SMs hold at once, each with a block at least.
template <int NT, typename O>
int split_of(int64_t tiles, int blocks, int dev, int sms) {
  int split = 1;
  while (split < 8 && split * 2 <= blocks && tiles * split * 2 <= resident_of<NT, O>(split * 2, dev, sms)) split *= 2;
  return split;
}

template <int NT, typename O, bool STOP = false>
cudaError_t split_attrs() {
  static PerDeviceOnce attrs;
  return once_per_device(attrs, [] { return set_smem_attrs(linear_split_kernel<NT, O, STOP>, SplitCfg<NT>::kSmem); });
}

template <int NT, typename O>
cudaError_t launch_split(const Fp8LinearArgs& a, int dev, int sms, cudaStream_t st) {
  using C = SplitCfg<NT>;
  LinearMaps maps;
  if (!codes_map(&maps.a, a.a, a.k, a.m, a.lda, NT) || !codes_map(&maps.w, a.w, a.k, a.n, a.ldw, 128) ||
      !make_map(&maps.a_scale, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, a.a_scale, a.m, ceil_div(a.k, kFp8Group), a.ld_as * 4,
                NT, 1, CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorInvalidValue;
  const cudaError_t e = split_attrs<NT, O>();
  if (e != cudaSuccess) return e;
  const int row_tiles = ceil_div(a.m, NT), blocks = ceil_div(a.k, kFp8Group);
  const int64_t tiles = (int64_t)row_tiles * ceil_div(a.n, 128);
  const int split = split_of<NT, O>(tiles, blocks, dev, sms);
  if (tiles * split > INT32_MAX) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * split));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (a.test_stop) {
    const cudaError_t t = split_attrs<NT, O, true>();
    if (t != cudaSuccess) return t;
    return cudaLaunchKernelEx(&cfg, linear_split_kernel<NT, O, true>, a, maps, split, row_tiles);
  }
  return cudaLaunchKernelEx(&cfg, linear_split_kernel<NT, O, false>, a, maps, split, row_tiles);
}

// Which kernel takes more than 64 rows.  All three walk their tiles in waves over the SMs; the constants
// (nanoseconds for a start, for a tile's start and end, and for a block of K) are from B200 runs: the
// estimates are within a fifth of the times below, and the choice falls on the shortest but for near ties.
//   rows x columns x K       pairs of 256   pairs of 128   split
//    65 x 25152 x 4096            37 us          36 us      32 us
//   128 x 25152 x 4096            38             37         35
//   256 x 25152 x 4096            39             38         50
//   512 x  4096 x 16384           63             47         46
//   256 x  4096 x 16384           63             46         27
//   1024 x 4096 x 16384           68             99         94
//   2048 x  576 x 4096            21             15         18
//   333 x  1000 x 1960            14             10         7.4
//   8192 x 8000 x 512             60             68          -
//   4096 x 4096 x 16384          306            384          -
template <typename O>
int choose(int64_t m, int64_t n, int blocks, int dev, int sms) {
  const int64_t row_tiles = ceil_div(m, kPairM);
  const int64_t wide = 4000 + ceil_div(row_tiles * ceil_div(n, 256), sms / 2) * (1500 + (int64_t)blocks * 480);
  const int64_t narrow = 4000 + ceil_div(row_tiles * ceil_div(n, 128), sms / 2) * (1500 + (int64_t)blocks * 335);
  const int64_t tiles = (int64_t)ceil_div(m, 128) * ceil_div(n, 128);
  const int parts = split_of<128, O>(tiles, blocks, dev, sms);
  const int64_t split = ceil_div(tiles * parts, sms) * (5000 + (int64_t)ceil_div(blocks, parts) * 380);
  if (split <= wide && split <= narrow) return QKN_LINEAR_SPLIT;
  return narrow < wide ? QKN_LINEAR_PAIR_128 : QKN_LINEAR_PAIR_256;
}

template <typename O>
cudaError_t launch(const Fp8LinearArgs& a, cudaStream_t st) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  int kernel = a.kernel;
  if (kernel == QKN_LINEAR_AUTO) {
    kernel = QKN_LINEAR_SPLIT;
    if (a.m > 64) {
      if ((e = split_attrs<128, O>()) != cudaSuccess) return e;   // (the estimate asks for the kernel's occupancy)
      kernel = choose<O>(a.m, a.n, ceil_div(a.k, kFp8Group), dev, sms);
    }
  }
  if (kernel == QKN_LINEAR_PAIR_256) return launch_pair<256, O>(a, sms, st);
  if (kernel == QKN_LINEAR_PAIR_128) return launch_pair<128, O>(a, sms, st);
  if (a.m > 64) return launch_split<128, O>(a, dev, sms, st);
  // the smallest of 16, 32 and 64 rows that holds them all: every tile reads its weight rows once
  if (a.m > 32) return launch_split<64, O>(a, dev, sms, st);
  if (a.m > 16) return launch_split<32, O>(a, dev, sms, st);
  return launch_split<16, O>(a, dev, sms, st);
}

}  // namespace

cudaError_t launch_fp8_linear(const Fp8LinearArgs& a, bool bf16_out, cudaStream_t st) {
  return bf16_out ? launch<__nv_bfloat16>(a, st) : launch<float>(a, st);
}

}  // namespace qkn
