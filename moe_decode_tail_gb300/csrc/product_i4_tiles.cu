// The 4-bit product on the 5th-generation tensor cores (sm_103a): tiles of 128 channels by up to 64 rows, or of 256 by 128.
//
// Persistent, one thread block an SM.  The packed weights cross memory once, by TMA (128 bytes of a channel, 256 columns of
// the reduction: a pair of blocks); converting warps, 32 channels each, turn them into BF16 in registers, their groups' scales
// multiplied in, and store them into tensor memory, from where the MMA takes its A operand (a thread's channel is a TMEM lane,
// so nothing is shuffled or written back to shared memory).  The rows arrive by TMA as the B operand; epilogue warps read
// finished accumulators, scale them by channel and write BF16.  The weight stream runs on across tiles.
//
// A gated tile has its gate channels, then the up channels that go with them.  In a narrow one they are in one accumulator
// and meet in shared memory; a wide one has an accumulator for each, and a thread both factors of a result.
//
// With few rows the weights' way from memory is the bound, and before it what a step costs the warps that issue MMAs and that
// convert.  64 tokens x 8 routes over 128 experts of 2048 x 4096 take 93 us (0.54 GB, 0.87 of the measured copy rate), of
// 4096 x 1024 with groups of 32 columns 58 us (0.74).  On the way there: a block a step with two barriers and commits 180 us;
// a pair a step, one barrier and one commit 112; three sets of converting warps that take whole steps instead of two that
// share them 102; rows asked for further ahead 100; tiles found by one warp for those that have no time to 94.
// With many rows the MMAs are the bound, with A in tensor memory about a third slower than their operations: 32768 rows over
// 128 experts of 4096 x 2048 take 390 to 440 us, as the GPU's clock under that load is, 1.25 to 1.41 PFLOP/s (0.65 to 0.74 of a
// library BF16 product).
//
// Every wait is bounded in time; on expiry the kernel raises a bit in the device error word, lets its copies and MMAs
// finish, frees its tensor memory and returns.
#include "kernels.h"
#include "layer.h"
#include "product_i4.cuh"

namespace moetail {

namespace {

__device__ unsigned int g_i4_tiles_error = 0;
__device__ __forceinline__ void raise_error(unsigned bit) { atomicOr(&g_i4_tiles_error, bit); }

constexpr int kRun = 16;                  // accumulator columns (rows of the result) written at a time
constexpr int kStaging = kRun * 128 * 4;  // of an epilogue set
constexpr int kTileRing = 32;             // tiles that the weights' warp has described: more than it can be ahead

// The forms of a tile: NT rows by 128 stored channels, or, wide, 128 rows by 256 of them: two MMAs for the same rows, whose
// way from L2 is halved (1999 tokens x 6 routes, half of them here, over 60 gated experts of 2832 x 2056: 82 us, without
// 106).
template <int NT_, bool WIDE_>
struct Form {
  static constexpr int NT = NT_;
  static constexpr bool WIDE = WIDE_;
  static constexpr int kSubs = WIDE ? 2 : 1;                        // tiles of 128 stored channels, the MMA's M
  static constexpr int kWStage = kSubs * 128 * 128;                 // bytes of a pair of blocks of them
  static constexpr int kBlocks = WIDE ? 1 : 2;                      // of a step of the MMA warp
  static constexpr int kStepsOfPair = 2 / kBlocks;
  static constexpr int kSlotColumns = 64 * kBlocks * kSubs;         // of a step's A in tensor memory: two BF16 each
  static constexpr int kAccs = WIDE ? 1 : 2;                        // accumulators, taken in turn
  static constexpr int kTmemA = kAccs * kSubs * NT;                 // first column of the A ring
  static constexpr int kSlots = (512 - kTmemA) / kSlotColumns;      // steps in it
  // Sets of converting warps take the pairs in turn, a warp for 32 channels.
  static constexpr int kSets = WIDE ? 1 : 3;
  static constexpr int kSetWarps = 4 * kSubs;
  static constexpr int kReaders = WIDE ? 2 : 1;                     // sets of four epilogue warps (one accumulator: it waits)
  static constexpr int kEpilogueWarps = 4 * kReaders;
  static constexpr int kThreads = 32 * (kEpilogueWarps + kSets * kSetWarps + 3);
  // Rows come a step at a time, and their arrival is seen by the converting warps, so that the MMA warp has one barrier to
  // wait for.  But for 64 rows (shared memory) they have twice as many slots as the step ring, so that their copy is asked
  // for well before it is needed; the set that finds a step's slot free again passes that on.
  static constexpr bool kRelayed = WIDE || NT <= 32;
  static constexpr int kXColumns = 128 * kBlocks;
  static constexpr int kXStages = kRelayed ? 2 * kSlots : kSlots;
  static constexpr int kXHalf = NT * 128, kXStage = NT * kXColumns * 2;  // bytes of 64 columns, and of a stage
  static_assert(kSlots % kSets == 0, "a set meets the same slots in every round");
};

struct Args {
  const uint8_t* group_scale;  // e4m3 [E][channels][pitch]
  const float* channel_scale;  // [E][channels]
  const int32_t* offsets;      // [E + 1] or null
  uint16_t* out;               // [R][N]
  int64_t R;
  int E, N;                    // N: channels of the result
  int blocks;                  // of 128 columns: ceil(D / 128)
  int groups, pitch;           // scales of a channel, and their distance to the next channel's
  int w_stages;
  bool whole;                  // D is a multiple of 64: map_x has the columns in sixty-fours
  unsigned long long stage_wait_ns;
};

// A tile: `rows` rows from r0 by channels from n0 (of the result) of expert e.
struct Tile {
  int e, n0, r0, rows;
};

template <class F, int GROUP, bool GATED>
__global__ void __launch_bounds__(F::kThreads, 1)
    product_i4_tiles_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, const Args a) {
  extern __shared__ uint8_t smem_raw[];
  constexpr int NT = F::NT, kSubs = F::kSubs, kWStage = F::kWStage, kBlocks = F::kBlocks, kStepsOfPair = F::kStepsOfPair;
  constexpr int kSlotColumns = F::kSlotColumns, kAccs = F::kAccs, kTmemA = F::kTmemA, kSlots = F::kSlots, kSets = F::kSets;
  constexpr int kSetWarps = F::kSetWarps, kReaders = F::kReaders, kEpilogueWarps = F::kEpilogueWarps;
  constexpr int kThreads = F::kThreads, kXColumns = F::kXColumns, kXStages = F::kXStages, kXHalf = F::kXHalf;
  constexpr int kXStage = F::kXStage;
  constexpr bool WIDE = F::WIDE, kRelayed = F::kRelayed;
  constexpr int kWarpW = kEpilogueWarps + kSets * kSetWarps, kWarpX = kWarpW + 1, kWarpMma = kWarpW + 2;
  constexpr int kPer = 128 / GROUP;              // groups of a block
  constexpr int kHalf = 64 * kSubs;              // of a gated tile: gate channels, then up channels
  constexpr int kOut = GATED ? kHalf : 2 * kHalf;  // channels of the result of a tile

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* base_ptr = smem_raw + (base - raw);
  const uint32_t x_ring = base, w_ring = x_ring + (uint32_t)(kXStages * kXStage);
  uint32_t at = w_ring + (uint32_t)(a.w_stages * kWStage);
  const uint32_t staging = at + (warp >> 2) % kReaders * kStaging;  // of an epilogue set
  at += kReaders * kStaging;
  auto bars = [&](int n) {
    const uint32_t first = at;
    at += 8u * n;
    return first;
  };
  const uint32_t w_full = bars(a.w_stages), w_empty = bars(a.w_stages), x_full = bars(kXStages);
  const uint32_t step_full = bars(kSlots), step_empty = bars(kSlots);
  const uint32_t x_empty = kRelayed ? bars(kXStages) : step_empty;
  const uint32_t acc_full = bars(kAccs), acc_empty = bars(kAccs), mma_done = bars(1);
  at = (at + 15u) & ~15u;
  volatile uint32_t* word = reinterpret_cast<volatile uint32_t*>(base_ptr + (at - base));  // TMEM base, abort
  volatile uint32_t* abort_ptr = word + 1;
  const uint32_t slot = at;
  Tile* s_tile = reinterpret_cast<Tile*>(base_ptr + (at - base) + 16);
  int32_t* s_first = reinterpret_cast<int32_t*>(s_tile + kTileRing);           // [E + 1] row tiles before an expert
  int32_t* s_row = s_first + a.E + 1;                                           // [E] its first row
  int32_t* s_count = s_row + a.E;                                               // [E] its rows

  if (warp == 0) {
    for (int s = lane; s < a.w_stages; s += 32) {
      mbar_init(w_full + 8 * s, 1);
      mbar_init(w_empty + 8 * s, kSetWarps);  // one set reads it
    }
    for (int s = lane; s < kXStages; s += 32) {
      mbar_init(x_full + 8 * s, 1);
      if (kRelayed) mbar_init(x_empty + 8 * s, 1);
    }
    if (lane < kSlots) {
      mbar_init(step_full + 8 * lane, kSetWarps);
      mbar_init(step_empty + 8 * lane, 1);
    }
    if (lane < kAccs) {
      mbar_init(acc_full + 8 * lane, 1);
      mbar_init(acc_empty + 8 * lane, kEpilogueWarps);
    }
    if (lane == 0) {
      mbar_init(mma_done, 1);
      *abort_ptr = 0;
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  } else if (warp == kWarpW && lane == 0) {
    prefetch_map(&map_w);
    prefetch_map(&map_x);
  }
  if (warp == kWarpMma) tmem_alloc(slot, 512);
  grid_dependency_wait();
  for (int e = threadIdx.x; e < a.E; e += kThreads) {
    const int begin = a.offsets ? clamp_row(a.offsets[e], a.R) : 0;
    const int end = a.offsets ? clamp_row(a.offsets[e + 1], a.R) : (int)a.R;
    s_row[e] = begin;
    s_count[e] = end > begin ? end - begin : 0;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  launch_dependents();
  const uint32_t tmem = word[0];
  if (warp == 0) row_tiles_before(s_count, s_first, a.E, NT);
  __syncthreads();

  const int n_tiles = (a.N + kOut - 1) / kOut;
  const int64_t tiles = (int64_t)s_first[a.E] * n_tiles;
  // Tiles in the order (expert, channel tile, row tile).  Finding one takes a thousand cycles: the warps that have none to
  // spare, those that convert and the one that issues MMAs, take it from the ring where the weights' warp leaves it; its
  // weights' arrival tells that it is there.
  auto tile_at = [&](int64_t i, Tile& q, bool* again = nullptr) {
    if (i >= tiles) return false;
    const int e = expert_of_tile(s_first, a.E, n_tiles, i);
    const int row_tiles = s_first[e + 1] - s_first[e];
    const int left = (int)(i - (int64_t)s_first[e] * n_tiles);
    const int n = left / row_tiles, t = left - n * row_tiles;
    q.e = e;
    q.n0 = n * kOut;
    // an expert's row tiles are equal but for a few rows
    const int share = ((s_count[e] + row_tiles - 1) / row_tiles + 15) & ~15;
    q.r0 = s_row[e] + t * share;
    q.rows = min(share, s_count[e] - t * share);  // at least one: NT * (row_tiles - 1) < s_count
    if (again) *again = row_tiles > 1;  // more than one row tile reads these weights
    return true;
  };
  // An odd last block has one of zeros beside it where a step takes both.
  const int pairs = (a.blocks + 1) / 2, steps = kStepsOfPair == 1 ? pairs : a.blocks;
  auto give_up = [&](unsigned bit) {
    if (!*abort_ptr) raise_error(bit);
    *abort_ptr = 1;
  };

  if (warp == kWarpW) {
    // ---------------- packed weights ----------------
    // The warps that issue copies and MMAs walk their loops whole, so that the addresses stay in uniform registers, and
    // one lane issues.
    const uint64_t once = policy_evict_first(), again = policy_evict_last();
    int64_t g = 0;
    Ring w;
    bool ok = true, shared = false;
    Tile q;
    int k = 0;
    for (int64_t i = blockIdx.x; ok && tile_at(i, q, &shared); i += gridDim.x, ++k) {
      const uint64_t policy = shared ? again : once;
      if (lane == 0) s_tile[k % kTileRing] = q;
      __syncwarp();
      for (int b = 0; b < pairs; ++b, ++g, w.step(a.w_stages)) {
        if (!warp_wait(w_empty + 8 * w.slot, w.parity ^ 1u, abort_ptr)) {  // the first round finds it free
          if (lane == 0) give_up(kErrWaitEmpty);
          ok = false;
          break;
        }
        if (elect_one()) {
          const uint32_t dst = w_ring + w.slot * kWStage, bar = w_full + 8 * w.slot;
          mbar_expect_tx(bar, kWStage);
          if (GATED) tma_load_4d(dst, &map_w, bar, 128 * b, q.n0, 0, q.e, policy);
          else tma_load_3d(dst, &map_w, bar, 128 * b, q.n0, q.e, policy);
        }
        __syncwarp();
      }
    }
    if (lane == 0)
      for (int64_t i = g > a.w_stages ? g - a.w_stages : 0; i < g; ++i)  // copies in flight land before the block ends
        if (!mbar_wait(w_full + 8 * (i % a.w_stages), (uint32_t)(i / a.w_stages) & 1u)) raise_error(kErrWaitDrain);
    __syncwarp();
  } else if (warp == kWarpX) {
    // ---------------- rows ----------------
    const uint64_t keep = policy_evict_last();
    int64_t g = 0;
    Ring x;
    bool ok = true;
    Tile q;
    for (int64_t i = blockIdx.x; ok && tile_at(i, q); i += gridDim.x) {
      for (int b = 0; b < steps; ++b, ++g, x.step(kXStages)) {
        if (!warp_wait(x_empty + 8 * x.slot, x.parity ^ 1u, abort_ptr)) {
          if (lane == 0) give_up(kErrWaitEmpty);
          ok = false;
          break;
        }
        if (elect_one()) {
          const uint32_t dst = x_ring + x.slot * kXStage, bar = x_full + 8 * x.slot;
          mbar_expect_tx(bar, kXStage);
          if (a.whole) {
            tma_load_3d(dst, &map_x, bar, 0, q.r0, kXColumns / 64 * b, keep);
          } else {
#pragma unroll
            for (int h = 0; h < kXColumns / 64; ++h)
              tma_load_2d(dst + h * kXHalf, &map_x, bar, kXColumns * b + 64 * h, q.r0, keep);
          }
        }
        __syncwarp();
      }
    }
    if (lane == 0)
      for (int64_t i = g > kXStages ? g - kXStages : 0; i < g; ++i)
        if (!mbar_wait(x_full + 8 * (i % kXStages), (uint32_t)(i / kXStages) & 1u)) raise_error(kErrWaitDrain);
    __syncwarp();
  } else if (warp == kWarpMma) {
    // ---------------- MMA issuer ----------------
    const unsigned long long limit = a.stage_wait_ns ? a.stage_wait_ns : kWaitLimitNs;
    Ring x, s, acc;
    bool ok = true;
    int k = 0;
    for (int64_t i = blockIdx.x; ok && i < tiles; i += gridDim.x, ++k, acc.step(kAccs)) {
      if (!warp_wait(acc_empty + 8 * acc.slot, acc.parity ^ 1u, abort_ptr)) {
        if (lane == 0) give_up(kErrWaitAccum);
        break;
      }
      const uint32_t d = tmem + acc.slot * (kSubs * NT);
      Tile q = {};
      if (k == 0) {
        tile_at(blockIdx.x, q);
      } else {  // once its first step is there
        if (!warp_wait(step_full + 8 * s.slot, s.parity, abort_ptr, limit)) {
          if (lane == 0) give_up(kErrWaitFull);
          break;
        }
        q = s_tile[k % kTileRing];
      }
      const uint32_t idesc = idesc_bf16(128, (q.rows + 15) & ~15);
      for (int b = 0; b < steps; ++b, s.step(kSlots), x.step(kXStages)) {
        if (!warp_wait(step_full + 8 * s.slot, s.parity, abort_ptr, limit)) {
          if (lane == 0) give_up(kErrWaitFull);
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t w = tmem + kTmemA + s.slot * kSlotColumns;
        const uint64_t bdesc = smem_desc_sw128(x_ring + x.slot * kXStage);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kXColumns / 16; ++kk)  // 16 columns: 8 TMEM columns of A, 32 bytes along B's swizzled row
#pragma unroll
            for (int m = 0; m < kSubs; ++m)
              mma_ts(d + m * NT, w + 64 * kBlocks * m + 8 * kk, bdesc + (kk / 4) * (kXHalf >> 4) + 2 * (kk % 4), idesc,
                     (b > 0 || kk > 0) ? 1u : 0u);
          mma_commit(step_empty + 8 * s.slot);
          if (b == steps - 1) mma_commit(acc_full + 8 * acc.slot);
        }
        __syncwarp();
      }
    }
    if (elect_one()) mma_commit(mma_done);  // the MMAs that were issued are done before tensor memory is freed
    __syncwarp();
    if (lane == 0 && !mbar_wait(mma_done, 0)) raise_error(kErrWaitAccum);
    __syncwarp();
  } else if (warp >= kEpilogueWarps) {
    // ---------------- 4 bits to BF16, one TMEM lane a thread ----------------
    // Set s takes the pairs s, s + kSets, ... of the stream, a step each, or two (wide).
    const int set = (warp - kEpilogueWarps) / kSetWarps, sub = (warp - kEpilogueWarps) % kSetWarps >> 2, quarter = warp & 3;
    const int row = sub * 128 + quarter * 32 + lane;   // of the staged tile
    const int channels = GATED ? 2 * a.N : a.N;
    constexpr int kGroups = 2 * kPer, kWords = (kGroups + 3) / 4;  // of a pair: their scales, in words of four
    Ring w, s, x;
    int ahead = set;  // pairs until this set's next one
    w.step(a.w_stages, ahead);
    s.step(kSlots, set);
    x.step(kXStages, set);
    bool ok = true;
    int fresh = kSlots / kSets;  // this set's slots that no step has had yet
    int k = 0;
    for (int64_t i = blockIdx.x; ok && i < tiles; i += gridDim.x, ++k) {
      Tile q = {};
      if (k == 0) {  // found here, and its scales asked for while its weights are on their way
        tile_at(blockIdx.x, q);
      } else if (ahead < pairs) {
        if (!warp_wait(w_full + 8 * w.slot, w.parity, abort_ptr)) {
          if (lane == 0) give_up(kErrWaitFull);
          ok = false;
          break;
        }
        q = s_tile[k % kTileRing];
      }
      // this thread's channel; past the last: the last
      const int n = min(q.n0 + (GATED ? row % kHalf : row), a.N - 1) + (GATED && row >= kHalf ? a.N : 0);
      const uint8_t* scales = a.group_scale + ((int64_t)q.e * channels + n) * a.pitch;
      auto load_scales = [&](int pair, uint32_t (&to)[kWords]) {  // the words with those of a pair
        const int first = pair * kGroups & ~3;
#pragma unroll
        for (int k = 0; k < kWords; ++k)
          to[k] = pair < pairs && first + 4 * k < a.groups ? __ldg(reinterpret_cast<const uint32_t*>(scales + first + 4 * k)) : 0u;
      };
      uint32_t next[kWords];
      load_scales(ahead, next);
      for (; ahead < pairs; ahead += kSets, w.step(a.w_stages, kSets)) {
        if (!warp_wait(w_full + 8 * w.slot, w.parity, abort_ptr)) {
          if (lane == 0) give_up(kErrWaitFull);
          ok = false;
          break;
        }
        const int first = ahead * kGroups;  // group
        uint32_t gs[kWords];
#pragma unroll
        for (int k = 0; k < kWords; ++k) {
          gs[k] = next[k];
          const int left = a.groups - (first & ~3) - 4 * k;  // behind the last group may stand anything: it counts as zero
          if (left < 4) gs[k] &= left > 0 ? (1u << (8 * left)) - 1u : 0u;
        }
        if (kGroups < 4) gs[0] >>= 8 * (first & 3);
        load_scales(ahead + kSets, next);  // not before a wait: that would wait for them too
        Factors f;
        uint4 v[4];  // words 4 t + i: columns 32 i + 8 t .. of a block
#pragma unroll
        for (int step = 0; step < kStepsOfPair; ++step, s.step(kSlots, kSets), x.step(kXStages, kSets)) {
          if (step > 0 && 2 * ahead + step >= a.blocks) break;
          const uint32_t dst = tmem + ((uint32_t)(quarter * 32) << 16) + kTmemA + s.slot * kSlotColumns + sub * 64 * kBlocks;
#pragma unroll
          for (int h = 0; h < 2 * kBlocks; ++h) {  // 64 columns
            if (h % 2 == 0) {
#pragma unroll
              for (int t = 0; t < 4; ++t)
                v[t] = ld_shared_v4(w_ring + w.slot * kWStage + sw128_offset(row, 4 * (step + h / 2) + t));
            }
            uint32_t r[32];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int c = 4 * step + 2 * h + j, group = 32 * c / GROUP;
              if (32 * c % GROUP == 0) f = scaled(gs[group / 4] >> (8 * (group % 4)));
#pragma unroll
              for (int t = 0; t < 4; ++t)
                int4x8_to_bf16(c % 4 == 0 ? v[t].x : c % 4 == 1 ? v[t].y : c % 4 == 2 ? v[t].z : v[t].w, f, r + 16 * j + 4 * t);
            }
            if (h == 0) {
              ok = warp_wait(step_empty + 8 * s.slot, s.parity ^ 1u, abort_ptr);
              if (!ok) break;
              tc_fence_after();
              // the step that had this slot before is done, and so are its rows
              if (fresh > 0) --fresh;
              else if (kRelayed && sub == 0 && quarter == 0 && lane == 0)
                mbar_arrive(x_empty + 8 * (x.slot < kSlots ? x.slot + kSlots : x.slot - kSlots));
            }
            tmem_st32(dst + 32 * h, r);
          }
          if (!ok) {
            if (lane == 0) give_up(kErrWaitEmpty);
            break;
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          // only now: the stores have taken what the loads brought, so nothing of the slot is still being read
          if ((step == kStepsOfPair - 1 || 2 * ahead + 1 >= a.blocks) && lane == 0) mbar_arrive(w_empty + 8 * w.slot);
          // one warp of the set sees the rows arrive too, so that the MMA warp has one barrier to wait for
          if (sub == 0 && quarter == 0 && !warp_wait(x_full + 8 * x.slot, x.parity, abort_ptr)) {
            if (lane == 0) give_up(kErrWaitFull);
            ok = false;
            break;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(step_full + 8 * s.slot);
        }
        if (!ok) break;
      }
      ahead -= pairs;
    }
  } else {
    // ---------------- accumulators to BF16 ----------------
    // A wide tile's result stays in registers until the accumulators have been read and given back.  Its two sets of four
    // warps read one of the two accumulators each, or, gated, every second run of 16 columns of both.
    const int reader = warp >> 2, quarter = warp & 3, row = 32 * quarter + lane;
    const int channels = GATED ? 2 * a.N : a.N;
    // this thread's channel of the result, and from which accumulator, of the tile's first
    const int column = WIDE ? row + (GATED ? 0 : 128 * reader) : GATED ? row & 63 : row;
    auto value = [](uint32_t bits) { return __uint_as_float(bits); };
    // 16 rows of 128 channels (of a narrow gated tile, 64) of this set, as they lie in shared memory, to the result
    auto store = [&](const Tile& q, int c, int n0, auto eight) {
      constexpr int kVectors = GATED && !WIDE ? 8 : 16;  // of a row
#pragma unroll
      for (int k = row; k < kRun * kVectors; k += 128) {
        const int r = k / kVectors, u = k % kVectors;
        const uint4 out = eight(r, u);
        if (c + r < q.rows && n0 + 8 * u < a.N) st_v4(a.out + (int64_t)(q.r0 + c + r) * a.N + n0 + 8 * u, out);
      }
    };
    auto bf16_rows = [&](int r, int u) { return ld_shared_v4(staging + (r * 128 + 8 * u) * 2); };
    Ring acc;
    bool ok = true;
    Tile q;
    for (int64_t i = blockIdx.x; ok && tile_at(i, q); i += gridDim.x, acc.step(kAccs)) {
      const float* cs_at = a.channel_scale + (int64_t)q.e * channels + q.n0 + column;
      const bool there = q.n0 + column < a.N;
      const float cs = there ? kScaled * __ldg(cs_at + (GATED && !WIDE && row >= 64 ? a.N : 0)) : 0.0f;
      const float cs_up = GATED && WIDE && there ? kScaled * __ldg(cs_at + a.N) : 0.0f;
      ok = warp_wait(acc_full + 8 * acc.slot, acc.parity, abort_ptr);
      ok = all_of<32 * kEpilogueWarps>(ok);  // one answer for the warps that meet at barriers below
      if (!ok) {
        if (lane == 0) give_up(kErrWaitAccum);
        break;
      }
      tc_fence_after();
      const uint32_t src = tmem + ((uint32_t)(quarter * 32) << 16) + acc.slot * (kSubs * NT);
      if constexpr (WIDE) {
        constexpr int kRuns = NT / kRun / (GATED ? 2 : 1);  // of a set
        uint32_t two[kRuns][kRun / 2];                      // two rows of this thread's channel
        auto first_row = [&](int k) { return kRun * (GATED ? 2 * k + reader : k); };
#pragma unroll
        for (int k = 0; k < kRuns; ++k) {
          const int c = first_row(k);
          if (c >= q.rows) continue;
          float v[kRun];
          together();
          tmem_ld16(src + (GATED ? 0 : reader * NT) + c, v);
          if (GATED) {
            float u[kRun];
            together();
            tmem_ld16(src + NT + c, u);
#pragma unroll
            for (int j = 0; j < kRun; ++j) v[j] = silu_times(v[j] * cs, u[j] * cs_up);
          } else {
#pragma unroll
            for (int j = 0; j < kRun; ++j) v[j] *= cs;
          }
#pragma unroll
          for (int j = 0; j < kRun; j += 2) two[k][j / 2] = bf16x2_pz(v[j], v[j + 1]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_empty + 8 * acc.slot);
#pragma unroll
        for (int k = 0; k < kRuns; ++k) {
          const int c = first_row(k);
          if (c >= q.rows) continue;
#pragma unroll
          for (int j = 0; j < kRun; j += 2) {
            st_shared_u16(staging + (j * 128 + row) * 2, two[k][j / 2]);
            st_shared_u16(staging + ((j + 1) * 128 + row) * 2, two[k][j / 2] >> 16);
          }
          set_bar(reader);
          store(q, c, q.n0 + (GATED ? 0 : 128 * reader), bf16_rows);
          set_bar(reader);
        }
      } else {
#pragma unroll 1
        for (int c = 0; c < q.rows; c += kRun) {
          float v[kRun];
          together();
          tmem_ld16(src + c, v);
#pragma unroll
          for (int j = 0; j < kRun; ++j) v[j] *= cs;
          // By shared memory, so that a row's channels leave as whole lines, and a gate meets its up.
          if (GATED) {
#pragma unroll
            for (int j = 0; j < kRun; ++j) st_shared_f32(staging + (j * 128 + row) * 4, v[j]);
          } else {
#pragma unroll
            for (int j = 0; j < kRun; j += 2) {
              const uint32_t two = bf16x2_pz(v[j], v[j + 1]);
              st_shared_u16(staging + (j * 128 + row) * 2, two);
              st_shared_u16(staging + ((j + 1) * 128 + row) * 2, two >> 16);
            }
          }
          set_bar(reader);
          if (GATED) {
            store(q, c, q.n0, [&](int r, int u) {
              uint32_t y[4];
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const uint4 g = ld_shared_v4(staging + (r * 128 + 8 * u + 4 * j) * 4);
                const uint4 up = ld_shared_v4(staging + (r * 128 + 64 + 8 * u + 4 * j) * 4);
                y[2 * j] = bf16x2_pz(silu_times(value(g.x), value(up.x)), silu_times(value(g.y), value(up.y)));
                y[2 * j + 1] = bf16x2_pz(silu_times(value(g.z), value(up.z)), silu_times(value(g.w), value(up.w)));
              }
              return make_uint4(y[0], y[1], y[2], y[3]);
            });
          } else {
            store(q, c, q.n0, bf16_rows);
          }
          set_bar(reader);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_empty + 8 * acc.slot);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpMma) tmem_dealloc(tmem, 512);
}

// ---- host --------------------------------------------------------------------------------------------------------------

template <class F, int GROUP, bool GATED>
cudaError_t launch_form(const ProductI4Args& p, const CUtensorMap& map_w, const CUtensorMap& map_x, int sms, cudaStream_t stream) {
  constexpr int kLimit = 227 * 1024, kXRing = F::kXStages * F::kXStage, kOut = (GATED ? 64 : 128) * F::kSubs;
  Args a;
  a.group_scale = p.group_scale;
  a.channel_scale = p.channel_scale;
  a.offsets = p.offsets;
  a.out = p.out;
  a.R = p.R;
  a.E = p.E;
  a.N = p.N;
  a.blocks = (p.D + 127) / 128;
  a.groups = (p.D + GROUP - 1) / GROUP;
  a.pitch = (a.groups + 3) / 4 * 4;
  a.stage_wait_ns = stage_wait_limit_ns();
  const int fixed = 1024 + F::kReaders * kStaging + 8 * (2 * 12 + 2 * 6 + 2 * 4 + 2 * 2 + 1) + 32 + kTileRing * 16 + 4 * (3 * p.E + 1);
  a.w_stages = (kLimit - fixed - kXRing) / F::kWStage;
  if (a.w_stages > 12) a.w_stages = 12;
  // A set of converting warps that takes every third pair must meet the same slots in every round: else it could ask for
  // a slot's next round while another set's copy in it is still on its way, and the parity of the round before would tell
  // it that its own had landed.
  a.w_stages -= a.w_stages % F::kSets;
  a.whole = p.D % 64 == 0;
  auto kernel = product_i4_tiles_kernel<F, GROUP, GATED>;
  cudaError_t e = ensure_smem_limit((const void*)kernel, kLimit);
  if (e != cudaSuccess) return e;
  // no more thread blocks than there can be tiles
  const int64_t row_tiles = p.E == 1 ? (p.R + F::NT - 1) / F::NT : p.R / F::NT + (p.R < p.E ? p.R : p.E);
  const int64_t most = row_tiles * ((p.N + kOut - 1) / kOut);
  return launch_pdl(kernel, dim3((unsigned)(most < sms ? most : sms)), dim3(F::kThreads),
                    (size_t)fixed + kXRing + (size_t)a.w_stages * F::kWStage, stream, map_w, map_x, a);
}

template <int GROUP, bool GATED>
cudaError_t launch_rows(const ProductI4Args& p, const ProductI4Plan& plan, const CUtensorMap& map_w, const CUtensorMap& map_x,
                        int sms, cudaStream_t stream) {
  if (plan.wide) return launch_form<Form<128, true>, GROUP, GATED>(p, map_w, map_x, sms, stream);
  switch (plan.rows) {
    case 16: return launch_form<Form<16, false>, GROUP, GATED>(p, map_w, map_x, sms, stream);
    case 32: return launch_form<Form<32, false>, GROUP, GATED>(p, map_w, map_x, sms, stream);
    default: return launch_form<Form<64, false>, GROUP, GATED>(p, map_w, map_x, sms, stream);
  }
}

}  // namespace

cudaError_t launch_product_i4_tiles(const ProductI4Args& p, const ProductI4Plan& plan, const CUtensorMap& map_w,
                                    const CUtensorMap& map_x, int sms, cudaStream_t stream) {
  if (p.gated)
    return p.group == 32   ? launch_rows<32, true>(p, plan, map_w, map_x, sms, stream)
           : p.group == 64 ? launch_rows<64, true>(p, plan, map_w, map_x, sms, stream)
                           : launch_rows<128, true>(p, plan, map_w, map_x, sms, stream);
  return p.group == 32   ? launch_rows<32, false>(p, plan, map_w, map_x, sms, stream)
         : p.group == 64 ? launch_rows<64, false>(p, plan, map_w, map_x, sms, stream)
                         : launch_rows<128, false>(p, plan, map_w, map_x, sms, stream);
}

cudaError_t take_product_i4_tiles_error(unsigned* bits) {
  unsigned v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_i4_tiles_error, sizeof v);
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_i4_tiles_error, &zero, sizeof zero);
  *bits = v;
  return e;
}

}  // namespace moetail
