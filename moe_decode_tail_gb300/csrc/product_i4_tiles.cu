// The 4-bit product on the 5th-generation tensor cores (sm_103a): tiles of 128 channels by 16 to 256 rows.
//
// Persistent, one thread block an SM.  The packed weights cross memory once, by TMA (128 channels x 64 bytes, 128 columns of
// the reduction: a block); sets of four warps turn a block into BF16 in registers, its groups' scales multiplied in, and store
// it into tensor memory, from where the MMA takes its A operand (a thread's channel is a TMEM lane, so nothing is shuffled
// or written back to shared memory).  The rows arrive by TMA as the B operand; four warps (eight at 256 rows) read finished
// accumulators, scale them by channel and write BF16.  The weight stream runs on across tiles.
//
// A gated tile has 64 gate and the 64 up channels that go with them, 16 and 16 in each quarter of the TMEM lanes, so that a
// pair of lanes 16 apart has both factors of a result.
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

constexpr int kTileM = 128;               // stored channels of a tile
constexpr int kWStage = kTileM * 64;      // bytes of a block of them
constexpr int kAColumns = 64;             // TMEM columns of a block: two BF16 each
constexpr int kASlots = 4;                // blocks in tensor memory
constexpr int kRun = 16;                  // accumulator columns (rows of the result) written at a time
constexpr int kStaging = kRun * kTileM * 2;

// With few rows the weights' way is the bound and more warps convert; with many the tensor cores.
constexpr int sets_of(int nt) { return nt > 64 ? 2 : 4; }
constexpr int readers_of(int nt) { return nt > 128 ? 2 : 1; }  // sets of four epilogue warps (one accumulator: it waits)
constexpr int threads_of(int nt) { return 32 * (4 * readers_of(nt) + 4 * sets_of(nt) + 3); }
constexpr int x_columns_of(int nt) { return nt > 128 ? 64 : 128; }  // of the reduction in a stage of rows
constexpr int x_stages_of(int nt) { return nt > 64 ? 4 : nt == 64 ? 6 : 8; }

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
  unsigned long long stage_wait_ns;
};

// A tile: `rows` rows from r0 by channels from n0 (of the result) of expert e.
struct Tile {
  int e, n0, r0, rows;
  bool shared;  // more than one row tile reads these weights
};

// NT: rows of a tile (the accumulator's columns).
template <int NT, int GROUP, bool GATED>
__global__ void __launch_bounds__(threads_of(NT), 1)
    product_i4_tiles_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, const Args a) {
  extern __shared__ uint8_t smem_raw[];
  constexpr int kReaders = readers_of(NT), kEpilogueWarps = 4 * kReaders, kSets = sets_of(NT), kThreads = threads_of(NT);
  constexpr int kWarpW = kEpilogueWarps + 4 * kSets, kWarpX = kWarpW + 1, kWarpMma = kWarpW + 2;
  constexpr int kXColumns = x_columns_of(NT), kXOfBlock = 128 / kXColumns, kXStages = x_stages_of(NT);
  constexpr int kXHalf = NT * 128, kXStage = NT * kXColumns * 2;  // bytes of 64 columns, and of a stage
  constexpr int kBox = NT < 64 ? NT : 64;        // rows of one TMA box
  constexpr int kAccs = NT > 128 ? 1 : 2;        // accumulators, taken in turn
  constexpr uint32_t kTmemA = kAccs * NT;        // first column of the A ring
  constexpr int kPer = 128 / GROUP;              // groups of a block
  constexpr int kOut = GATED ? 64 : 128;         // channels of the result of a tile
  static_assert(kTmemA + kASlots * kAColumns <= 512, "tensor memory");
  static_assert(kASlots % kSets == 0, "a set meets the same slots in every round");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* base_ptr = smem_raw + (base - raw);
  const uint32_t x_ring = base, w_ring = x_ring + (uint32_t)(kXStages * kXStage);
  uint32_t at = w_ring + (uint32_t)(a.w_stages * kWStage);
  const uint32_t staging = at + (warp >> 2) % kReaders * kStaging;  // an epilogue set's BF16
  at += kReaders * kStaging;
  auto bars = [&](int n) {
    const uint32_t first = at;
    at += 8u * n;
    return first;
  };
  const uint32_t w_full = bars(a.w_stages), w_empty = bars(a.w_stages), x_full = bars(kXStages), x_empty = bars(kXStages);
  const uint32_t a_full = bars(kASlots), a_empty = bars(kASlots);
  const uint32_t acc_full = bars(kAccs), acc_empty = bars(kAccs), mma_done = bars(1);
  at = (at + 15u) & ~15u;
  volatile uint32_t* word = reinterpret_cast<volatile uint32_t*>(base_ptr + (at - base));  // TMEM base, abort
  volatile uint32_t* abort_ptr = word + 1;
  const uint32_t slot = at;
  int32_t* s_first = reinterpret_cast<int32_t*>(base_ptr + (at - base) + 16);  // [E + 1] row tiles before an expert
  int32_t* s_row = s_first + a.E + 1;                                           // [E] its first row
  int32_t* s_count = s_row + a.E;                                               // [E] its rows

  if (warp == 0) {
    for (int s = lane; s < a.w_stages; s += 32) {
      mbar_init(w_full + 8 * s, 1);
      mbar_init(w_empty + 8 * s, 4);  // a set of four warps reads it
    }
    for (int s = lane; s < kXStages; s += 32) {
      mbar_init(x_full + 8 * s, 1);
      mbar_init(x_empty + 8 * s, 1);
    }
    if (lane < kASlots) {
      mbar_init(a_full + 8 * lane, 4);
      mbar_init(a_empty + 8 * lane, 1);
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
  auto tile_at = [&](int64_t i, Tile& q) {  // in the order (expert, channel tile, row tile)
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
    q.shared = row_tiles > 1;
    return true;
  };
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
    bool ok = true;
    Tile q;
    for (int64_t i = blockIdx.x; ok && tile_at(i, q); i += gridDim.x) {
      const uint64_t policy = q.shared ? again : once;
      for (int b = 0; b < a.blocks; ++b, ++g, w.step(a.w_stages)) {
        if (!warp_wait(w_empty + 8 * w.slot, w.parity ^ 1u, abort_ptr)) {  // the first round finds it free
          if (lane == 0) give_up(kErrWaitEmpty);
          ok = false;
          break;
        }
        if (elect_one()) {
          const uint32_t dst = w_ring + w.slot * kWStage, bar = w_full + 8 * w.slot;
          mbar_expect_tx(bar, kWStage);
          if (GATED) {
#pragma unroll
            for (int p = 0; p < 4; ++p) tma_load_4d(dst + p * (kWStage / 4), &map_w, bar, 64 * b, q.n0 + 16 * p, 0, q.e, policy);
          } else {
            tma_load_3d(dst, &map_w, bar, 64 * b, q.n0, q.e, policy);
          }
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
      const int boxes = NT <= kBox ? 1 : (q.rows + kBox - 1) / kBox;
      for (int b = 0; b < kXOfBlock * a.blocks; ++b, ++g, x.step(kXStages)) {
        if (!warp_wait(x_empty + 8 * x.slot, x.parity ^ 1u, abort_ptr)) {
          if (lane == 0) give_up(kErrWaitEmpty);
          ok = false;
          break;
        }
        if (elect_one()) {
          mbar_expect_tx(x_full + 8 * x.slot, (uint32_t)(kXColumns / 64 * boxes * kBox * 128));
#pragma unroll
          for (int h = 0; h < kXColumns / 64; ++h)
            for (int c = 0; c < boxes; ++c)
              tma_load_2d(x_ring + x.slot * kXStage + h * kXHalf + c * kBox * 128, &map_x, x_full + 8 * x.slot,
                          kXColumns * b + 64 * h, q.r0 + c * kBox, keep);
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
    Tile q;
    for (int64_t i = blockIdx.x; ok && tile_at(i, q); i += gridDim.x, acc.step(kAccs)) {
      if (!warp_wait(acc_empty + 8 * acc.slot, acc.parity ^ 1u, abort_ptr)) {
        if (lane == 0) give_up(kErrWaitAccum);
        break;
      }
      const uint32_t idesc = idesc_bf16(kTileM, (q.rows + 15) & ~15);
      const uint32_t d = tmem + acc.slot * NT;
      for (int b = 0; ok && b < a.blocks; ++b, s.step(kASlots)) {
        ok = warp_wait(a_full + 8 * s.slot, s.parity, abort_ptr, limit);
        const uint32_t w = tmem + kTmemA + s.slot * kAColumns;
#pragma unroll
        for (int h = 0; h < kXOfBlock; ++h) {
          ok = ok && warp_wait(x_full + 8 * x.slot, x.parity, abort_ptr, limit);
          if (!ok) break;
          tc_fence_after();
          const uint64_t bdesc = smem_desc_sw128(x_ring + x.slot * kXStage);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < kXColumns / 16; ++kk)  // 16 columns: 8 TMEM columns of A, 32 bytes along B's swizzled row
              mma_ts(d, w + 32 * h + 8 * kk, bdesc + (kk / 4) * (kXHalf >> 4) + 2 * (kk % 4), idesc,
                     (b > 0 || h > 0 || kk > 0) ? 1u : 0u);
            mma_commit(x_empty + 8 * x.slot);
            if (h == kXOfBlock - 1) {
              mma_commit(a_empty + 8 * s.slot);
              if (b == a.blocks - 1) mma_commit(acc_full + 8 * acc.slot);
            }
          }
          __syncwarp();
          x.step(kXStages);
        }
        if (!ok && lane == 0) give_up(kErrWaitFull);
      }
    }
    if (elect_one()) mma_commit(mma_done);  // the MMAs that were issued are done before tensor memory is freed
    __syncwarp();
    if (lane == 0 && !mbar_wait(mma_done, 0)) raise_error(kErrWaitAccum);
    __syncwarp();
  } else if (warp >= kEpilogueWarps) {
    // ---------------- 4 bits to BF16, one TMEM lane a thread ----------------
    // Set s takes the blocks s, s + kSets, ... of the stream.
    const int set = (warp - kEpilogueWarps) >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane, swizzle = (row >> 1) & 3;  // 16-byte units of a 64-byte row, as the copy lays them
    const int channels = GATED ? 2 * a.N : a.N;
    Ring w;
    w.step(a.w_stages, set);
    uint32_t parity = 0;  // of the set's rounds through its slots in tensor memory
    int slot_a = set;
    int ahead = set;      // blocks until this set's next one
    bool ok = true;
    Tile q;
    for (int64_t i = blockIdx.x; ok && tile_at(i, q); i += gridDim.x) {
      // this thread's channel; past the last: the last
      const int past = GATED && (lane & 16) ? a.N : 0;
      const int n = min(q.n0 + (GATED ? 16 * quarter + (lane & 15) : row), a.N - 1) + past;
      const uint8_t* scales = a.group_scale + ((int64_t)q.e * channels + n) * a.pitch;
      auto four_scales = [&](int block) {  // of them those of a block
        return block < a.blocks ? __ldg(reinterpret_cast<const uint32_t*>(scales + (block * kPer & ~3))) : 0u;
      };
      uint32_t next = four_scales(ahead);
      for (; ahead < a.blocks; ahead += kSets, w.step(a.w_stages, kSets)) {
        uint32_t gs = next;
        next = four_scales(ahead + kSets);
        const int left = a.groups - (ahead * kPer & ~3);  // behind the last group may stand anything: it counts as zero
        if (left < 4) gs &= (1u << (8 * left)) - 1u;
        gs >>= 8 * (ahead * kPer & 3);
        if (!warp_wait(w_full + 8 * w.slot, w.parity, abort_ptr)) {
          if (lane == 0) give_up(kErrWaitFull);
          ok = false;
          break;
        }
        const uint32_t src = w_ring + w.slot * kWStage + row * 64;
        uint4 v[4];  // words 4 t + i: columns 32 i + 8 t ..
#pragma unroll
        for (int t = 0; t < 4; ++t) v[t] = ld_shared_v4(src + ((t ^ swizzle) << 4));
        const uint32_t dst = tmem + ((uint32_t)(quarter * 32) << 16) + kTmemA + slot_a * kAColumns;
        Factors f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // 64 columns
          uint32_t r[32];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int c = 2 * h + j;
            if (32 * c % GROUP == 0) f = scaled(gs >> (8 * (32 * c / GROUP)));
#pragma unroll
            for (int t = 0; t < 4; ++t)
              int4x8_to_bf16(c == 0 ? v[t].x : c == 1 ? v[t].y : c == 2 ? v[t].z : v[t].w, f, r + 16 * j + 4 * t);
          }
          if (h == 0) {
            ok = warp_wait(a_empty + 8 * slot_a, parity ^ 1u, abort_ptr);
            if (!ok) break;
            tc_fence_after();
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
        if (lane == 0) {
          mbar_arrive(w_empty + 8 * w.slot);
          mbar_arrive(a_full + 8 * slot_a);
        }
        slot_a += kSets;
        if (slot_a >= kASlots) {
          slot_a -= kASlots;
          parity ^= 1u;
        }
      }
      ahead -= a.blocks;
    }
  } else {
    // ---------------- accumulators to BF16 ----------------
    // A set of four warps reads every kReaders-th run of 16 columns.
    const int reader = warp >> 2, quarter = warp & 3;
    const int channels = GATED ? 2 * a.N : a.N;
    const int mine = GATED ? 16 * quarter + (lane & 15) : 32 * quarter + lane;  // of the tile's channels of the result
    Ring acc;
    bool ok = true;
    Tile q;
    for (int64_t i = blockIdx.x; ok && tile_at(i, q); i += gridDim.x, acc.step(kAccs)) {
      const int past = GATED && (lane & 16) ? a.N : 0;
      const float cs = q.n0 + mine < a.N ? kScaled * __ldg(a.channel_scale + (int64_t)q.e * channels + q.n0 + mine + past) : 0.0f;
      ok = warp_wait(acc_full + 8 * acc.slot, acc.parity, abort_ptr);
      ok = all_of<32 * kEpilogueWarps>(ok);  // one answer for the warps that meet at barriers below
      if (!ok) {
        if (lane == 0) give_up(kErrWaitAccum);
        break;
      }
      tc_fence_after();
      const uint32_t src = tmem + ((uint32_t)(quarter * 32) << 16) + acc.slot * NT;
#pragma unroll 1
      for (int c = kRun * reader; c < q.rows; c += kRun * kReaders) {
        float v[kRun];
        together();
        tmem_ld16(src + c, v);
#pragma unroll
        for (int j = 0; j < kRun; ++j) v[j] *= cs;
        // By shared memory, so that a row's channels leave as whole lines.
        if (GATED) {
          // the lower lanes take the first eight rows, the upper ones the others: each sends the factors the other lacks
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float other = __shfl_xor_sync(0xffffffffu, lane & 16 ? v[j] : v[8 + j], 16);
            const float y = silu_times(lane & 16 ? other : v[j], lane & 16 ? v[8 + j] : other);
            st_shared_u16(staging + ((j + (lane & 16 ? 8 : 0)) * 64 + mine) * 2, bf16x2_pz(y, y));
          }
        } else {
#pragma unroll
          for (int j = 0; j < kRun; j += 2) {
            const uint32_t two = bf16x2_pz(v[j], v[j + 1]);
            st_shared_u16(staging + (j * kTileM + mine) * 2, two);
            st_shared_u16(staging + ((j + 1) * kTileM + mine) * 2, two >> 16);
          }
        }
        set_bar(reader);
        constexpr int kVectors = kOut / 8;  // of a row
#pragma unroll
        for (int k = quarter * 32 + lane; k < kRun * kVectors; k += 128) {
          const int r = k / kVectors, u = k % kVectors;
          const uint4 eight = ld_shared_v4(staging + 16 * k);
          if (c + r < q.rows && q.n0 + 8 * u < a.N) st_v4(a.out + (int64_t)(q.r0 + c + r) * a.N + q.n0 + 8 * u, eight);
        }
        set_bar(reader);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_empty + 8 * acc.slot);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpMma) tmem_dealloc(tmem, 512);
}

// ---- host --------------------------------------------------------------------------------------------------------------

template <int NT, int GROUP, bool GATED>
cudaError_t launch_nt(const ProductI4Args& p, const CUtensorMap& map_w, const CUtensorMap& map_x, int sms, cudaStream_t stream) {
  constexpr int kLimit = 227 * 1024, kXRing = x_stages_of(NT) * NT * x_columns_of(NT) * 2, kOut = GATED ? 64 : 128;
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
  const int fixed = 1024 + readers_of(NT) * kStaging + 8 * (2 * 16 + 2 * 8 + 2 * kASlots + 2 * 2 + 1) + 32 + 4 * (3 * p.E + 1);
  a.w_stages = (kLimit - fixed - kXRing) / kWStage;
  if (a.w_stages > 16) a.w_stages = 16;
  // A set of converting warps must meet the same slots in every round: else it could ask for a slot's next round while
  // another set's copy in it is still on its way, and the parity of the round before would tell it that its own had landed.
  a.w_stages -= a.w_stages % sets_of(NT);
  auto kernel = product_i4_tiles_kernel<NT, GROUP, GATED>;
  cudaError_t e = ensure_smem_limit((const void*)kernel, kLimit);
  if (e != cudaSuccess) return e;
  // no more thread blocks than there can be tiles
  const int64_t row_tiles = p.E == 1 ? (p.R + NT - 1) / NT : p.R / NT + (p.R < p.E ? p.R : p.E);
  const int64_t most = row_tiles * ((p.N + kOut - 1) / kOut);
  return launch_pdl(kernel, dim3((unsigned)(most < sms ? most : sms)), dim3(threads_of(NT)),
                    (size_t)fixed + kXRing + (size_t)a.w_stages * kWStage, stream, map_w, map_x, a);
}

template <int GROUP, bool GATED>
cudaError_t launch_rows(const ProductI4Args& p, int rows, const CUtensorMap& map_w, const CUtensorMap& map_x, int sms,
                        cudaStream_t stream) {
  switch (rows) {
    case 16: return launch_nt<16, GROUP, GATED>(p, map_w, map_x, sms, stream);
    case 32: return launch_nt<32, GROUP, GATED>(p, map_w, map_x, sms, stream);
    case 64: return launch_nt<64, GROUP, GATED>(p, map_w, map_x, sms, stream);
    case 128: return launch_nt<128, GROUP, GATED>(p, map_w, map_x, sms, stream);
    default: return launch_nt<256, GROUP, GATED>(p, map_w, map_x, sms, stream);
  }
}

}  // namespace

cudaError_t launch_product_i4_tiles(const ProductI4Args& p, int rows, const CUtensorMap& map_w, const CUtensorMap& map_x,
                                    int sms, cudaStream_t stream) {
  if (p.gated)
    return p.group == 32   ? launch_rows<32, true>(p, rows, map_w, map_x, sms, stream)
           : p.group == 64 ? launch_rows<64, true>(p, rows, map_w, map_x, sms, stream)
                           : launch_rows<128, true>(p, rows, map_w, map_x, sms, stream);
  return p.group == 32   ? launch_rows<32, false>(p, rows, map_w, map_x, sms, stream)
         : p.group == 64 ? launch_rows<64, false>(p, rows, map_w, map_x, sms, stream)
                         : launch_rows<128, false>(p, rows, map_w, map_x, sms, stream);
}

cudaError_t take_product_i4_tiles_error(unsigned* bits) {
  unsigned v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_i4_tiles_error, sizeof v);
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_i4_tiles_error, &zero, sizeof zero);
  *bits = v;
  return e;
}

}  // namespace moetail
