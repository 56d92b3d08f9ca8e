// Product of 8-bit integers with a scale for each row and each channel, by expert (sm_103a).
//
//   out[r][n] = bf16((sum over k of x[r][k] * w[e][n][k]) * w_scale[e][n] * x_scale[r]),
//   r in [offsets[e], offsets[e + 1])
//
// sm_103a's tensor cores have no fast 8-bit integer form, but every int8 is an FP16 number and a product of two
// is exact in FP32, so the product runs as kind::f16: exact while the magnitudes add up to less than 2^24, and
// rounded to FP32 beyond.  The weights cross memory once, as bytes, and become FP16 on the way to the tensor core:
//
//   expand   (own kernel) the rows x in FP16 into the workspace: small beside the weights, and every channel
//            tile reads them again
//   product  persistent, one thread block an SM.  A tile is 128 channels of an expert (the MMA's M) by up to NT
//            of its rows (its N).  The weight bytes arrive by TMA (128 channels x 128 bytes a stage); eight warps
//            turn them into FP16 in registers and store them into tensor memory, from where the MMA takes its A
//            operand (a thread's row is a TMEM lane, so nothing is shuffled or written back to shared memory);
//            the FP16 rows arrive by TMA as the B operand; four warps (eight at 256 rows) read finished
//            accumulators, scale them and write BF16.  The weight stream runs on across tiles.
//
// With few rows for an expert the weights' way from memory is the bound: 64 tokens x 8 routes over 128 experts of
// 2048 x 4096 take 175 us (1.06 GB, 0.90 of the measured copy rate; the product kernel alone 157 us, all of it).
// With many, the tensor cores and what feeds them: 8192 rows by 8192 channels x 4096 in 353 us, 1.56 PFLOP/s (0.84
// of a library BF16 product); 32768 rows over the 128 experts in 500 us, of which expand takes 75.
//
// The tiles that are no multiple of the thread blocks (with few rows, all of them) are dealt out by reduction
// blocks, the same number to each thread block, so such a tile may begin in one and end in another.  A part's FP32
// sums go to the workspace, and the thread block that finishes a tile's last missing part adds them, in the order
// of the reduction.  The other tiles follow whole, neighbours at the same time, so that they share what L2 holds.
//
// Every wait is bounded in time; on expiry the kernel raises a bit in the device error word, lets its copies and
// MMAs finish, frees its tensor memory and returns.
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"
#include "layer.h"
#include "tensor_core.cuh"

namespace moetail {

namespace {

__device__ unsigned int g_product_error = 0;
__device__ __forceinline__ void raise_error(unsigned bit) { atomicOr(&g_product_error, bit); }

constexpr int kTileM = 128;                    // channels of a tile
constexpr int kWBlock = 128;                   // reduction bytes of a weight stage: one swizzle row
constexpr int kWStage = kTileM * kWBlock;      // 16 KB
constexpr int kXBlock = 64;                    // FP16 of a row stage: one swizzle row
constexpr int kAColumns = kXBlock / 2;         // TMEM columns of a weight half stage: two FP16 each
constexpr int kSets = 2;                       // sets of four converting warps, a warp for each TMEM quarter (four: no faster)
constexpr int kMaxGrid = 160;                  // thread blocks: each has at most two parts of a tile
constexpr int kLeastBlocks = 4;                // reduction blocks a thread block is worth

struct Args {
  const float* x_scale;
  const float* w_scale;
  const int32_t* offsets;
  uint16_t* out;
  float* partial;      // [2 kMaxGrid][NT][128]: a block's continued tile, then the one it begins and does not end
  unsigned* counters;  // [kMaxGrid]: finished parts of the tile that a block begins, zeroed by the expand kernel
  int64_t R;
  int E, N;
  int w_blocks;        // ceil(D / 128)
  int w_stages;
  unsigned long long stage_wait_ns;
};

// Offsets come from the device: whatever they hold, no row outside [0, R) is touched.
__device__ __forceinline__ int clamp_row(int r, int64_t rows) { return r < 0 ? 0 : r > rows ? (int)rows : r; }

// ---- int8 to FP16 -----------------------------------------------------------------

// Four int8 as two pairs of FP16.  The byte v + 128 under the exponent of 1024 is the FP16 number 1152 + v, and
// the subtraction is exact.
__device__ __forceinline__ void int8x4_to_f16(uint32_t v, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = v ^ 0x80808080u;
  const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
  const __half2 base = __half2half2(__ushort_as_half((unsigned short)0x6480));  // 1152
  const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), base);
  const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), base);
  lo = *reinterpret_cast<const uint32_t*>(&x);
  hi = *reinterpret_cast<const uint32_t*>(&y);
}

constexpr int kExpand = 4;  // loads of a thread in flight

__global__ void __launch_bounds__(256) expand_rows_kernel(const int8_t* x, uint16_t* x16, const int32_t* offsets, int E,
                                                          int64_t R, int D, unsigned* counters) {
  grid_dependency_wait();
  // Only now: when the product's blocks start, everything before this call is complete, so they may read the
  // weights, scales and offsets at once and wait for this kernel before they touch what it writes.
  launch_dependents();
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < kMaxGrid; i += blockDim.x) counters[i] = 0;
  const int64_t rows = offsets ? clamp_row(offsets[E], R) : R;
  const int64_t n = rows * D / 16;
  for (int64_t i0 = (int64_t)blockIdx.x * (kExpand * 256) + threadIdx.x; i0 < n; i0 += (int64_t)gridDim.x * (kExpand * 256)) {
    uint4 v[kExpand];
#pragma unroll
    for (int j = 0; j < kExpand; ++j)
      if (i0 + 256 * j < n) v[j] = ld_stream_v4(x + 16 * (i0 + 256 * j));
#pragma unroll
    for (int j = 0; j < kExpand; ++j) {
      const int64_t i = i0 + 256 * j;
      if (i >= n) break;
      uint4 a, b;
      int8x4_to_f16(v[j].x, a.x, a.y);
      int8x4_to_f16(v[j].y, a.z, a.w);
      int8x4_to_f16(v[j].z, b.x, b.y);
      int8x4_to_f16(v[j].w, b.z, b.w);
      st_v4(x16 + 16 * i, a);
      st_v4(x16 + 16 * i + 8, b);
    }
  }
}

// Brings the warp's lanes together: before instructions that all of them have to execute at once (".aligned"), which
// the compiler does not know of inside inline assembly and might place in the branches before them.
__device__ __forceinline__ void together() { __syncwarp(); }

// ---- PTX of this kernel -------------------------------------------------------------

// D[tmem_d] (+)= A[tmem_a] * B[bdesc], FP16 operands, FP32 sums.
__device__ __forceinline__ void mma_f16_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
      "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// kind::f16 with FP16 operands: FP32 accumulate (bits 4-5 = 1), both K-major, N >> 3 at bit 17, M >> 4 at bit 24.
__device__ __forceinline__ uint32_t idesc_f16(int m, int n) {
  return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
// 32 consecutive TMEM columns of this thread's lane (to be waited for).
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  together();
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  together();
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void st_shared_u16(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"((uint16_t)v) : "memory");
}
// A barrier over the four warps of an epilogue set.
__device__ __forceinline__ void set_bar(int set) {
  together();
  asm volatile("bar.sync %0, 128;" ::"r"(2 + set) : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar), "l"(policy)
      : "memory");
}

// Barrier 1 over `threads`; whether `ok` holds in all of them.
template <int THREADS>
__device__ __forceinline__ bool all_of(bool ok) {
  uint32_t all;
  together();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"((uint32_t)ok), "n"(THREADS)
      : "memory");
  return all != 0;
}
// By a whole warp, with one answer for all its lanes.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag,
                                          unsigned long long limit_ns = kWaitLimitNs) {
  if (limit_ns > 1 && __all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, limit_ns, abort_flag));
}
// True in one lane of a converged warp.  The issuing warps walk their loops whole and issue under it: with one lane in
// the loop every operand of a copy or an MMA went from vector to uniform registers first (411 -> 211 us in decode).
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}

// A place in a ring of `stages` slots and the parity of its current round (counted, not divided: an integer
// division a step was most of the MMA thread's time).
struct Ring {
  int slot = 0;
  uint32_t parity = 0;  // of the round: a consumer waits for it on "full", a producer for its opposite on "empty"
  __device__ __forceinline__ void step(int stages, int by = 1) {
    slot += by;
    if (slot >= stages) {
      slot -= stages;
      parity ^= 1u;
    }
  }
};

// ---- the product ----------------------------------------------------------------------

// A part: reduction blocks [k0, k0 + blocks) of 128 channels from m0 by rows [r0, r0 + rows) of expert e.
struct Part {
  int e, m0, r0, rows, k0, blocks;
  int64_t tile;
  bool shared;  // more than one row tile reads this expert's weights
};

// A tile whose parts are all in the workspace, by the thread blocks first .. last.
struct Split {
  int e, m0, r0, rows, first, last;
};

// NT: rows of a tile (the accumulator's columns).
// A step of the MMA warp takes `halves` of a weight stage, 64 of the reduction each: what a step costs besides its
// MMAs (a wait, a commit) is then paid half as often (decode: 180 us, 200 with one).  With 256 rows shared memory has
// no room for two.
constexpr int halves_of(int nt) { return nt > 128 ? 1 : 2; }
// Steps in flight: what tensor memory has beside the accumulators; with 256 rows shared memory is the limit.
constexpr int steps_of(int nt) { return nt > 128 ? 5 : (512 - 2 * nt) / (2 * kAColumns); }
constexpr int readers_of(int nt) { return nt > 128 ? 2 : 1; }  // sets of four epilogue warps (one accumulator: it waits)
constexpr int threads_of(int nt) { return 32 * (4 * readers_of(nt) + 4 * kSets + 3); }
constexpr int kRun = 16;                             // accumulator columns (rows of the result) written at a time
constexpr int kStaging = kRun * kTileM * 2;          // their BF16, of a set

template <int NT>
__global__ void __launch_bounds__(threads_of(NT), 1)
    expert_product_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                          const Args a) {
  extern __shared__ uint8_t smem_raw[];
  constexpr int kReaders = readers_of(NT), kEpilogueWarps = 4 * kReaders, kThreads = threads_of(NT);
  constexpr int kWarpW = kEpilogueWarps + 4 * kSets, kWarpX = kWarpW + 1, kWarpMma = kWarpW + 2;
  constexpr int kHalves = halves_of(NT), kStepsOfStage = 2 / kHalves;
  constexpr int kXHalf = NT * kXBlock * 2, kXStage = kHalves * kXHalf;
  constexpr int kStepColumns = kHalves * kAColumns;  // of A in tensor memory
  constexpr int kBox = NT < 64 ? NT : 64;          // rows of one TMA box
  constexpr int kAccs = NT > 128 ? 1 : 2;          // accumulators, taken in turn
  constexpr int kSteps = steps_of(NT);             // ring of MMA steps: A in tensor memory, B in shared memory
  constexpr uint32_t kTmemA = kAccs * NT;          // first column of the A ring
  static_assert(kTmemA + kSteps * kStepColumns <= 512, "tensor memory");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* base_ptr = smem_raw + (base - raw);
  const uint32_t w_ring = base, x_ring = w_ring + (uint32_t)(a.w_stages * kWStage);
  uint32_t at = x_ring + (uint32_t)(kSteps * kXStage);
  auto bars = [&](int n) {
    const uint32_t first = at;
    at += 8u * n;
    return first;
  };
  const uint32_t w_full = bars(a.w_stages), w_empty = bars(a.w_stages);
  const uint32_t x_full = bars(kSteps), step_full = bars(kSteps), step_empty = bars(kSteps);
  const uint32_t acc_full = bars(kAccs), acc_empty = bars(kAccs), mma_done = bars(1);
  at = (at + 15u) & ~15u;
  // TMEM base, abort, parts finished before this one, tiles in s_split
  volatile uint32_t* word = reinterpret_cast<volatile uint32_t*>(base_ptr + (at - base));
  volatile uint32_t* abort_ptr = word + 1;
  const uint32_t slot = at;
  Split* s_split = reinterpret_cast<Split*>(base_ptr + (at - base) + 16);  // [2] that this thread block is to add up
  at += 64;
  // an epilogue warp's scales of the rows it writes [NT / kReaders], and its set's BF16 [kRun][128]
  const uint32_t scales = at + 16 + (warp % kEpilogueWarps) * (NT / kReaders) * 4;
  float* s_scale = reinterpret_cast<float*>(base_ptr + (scales - base));
  const uint32_t staging = at + 16 + 16 * NT + (warp >> 2) % kReaders * kStaging;
  int32_t* s_first = reinterpret_cast<int32_t*>(base_ptr + (at - base) + 16 + 16 * NT + kReaders * kStaging);  // [E + 1]
  int32_t* s_row = s_first + a.E + 1;                                    // row tiles before an expert; [E] its first row
  int32_t* s_count = s_row + a.E;                                        // [E] its rows

  if (warp == 0) {
    for (int s = lane; s < a.w_stages; s += 32) {
      mbar_init(w_full + 8 * s, 1);
      mbar_init(w_empty + 8 * s, 4 * kStepsOfStage);  // a set of four warps reads what it makes a step of
    }
    for (int s = lane; s < kSteps; s += 32) {
      mbar_init(x_full + 8 * s, 1);
      mbar_init(step_full + 8 * s, 4);
      mbar_init(step_empty + 8 * s, 1);
    }
    if (lane < kAccs) {
      mbar_init(acc_full + 8 * lane, 1);
      mbar_init(acc_empty + 8 * lane, kEpilogueWarps);
    }
    if (lane == 0) {
      mbar_init(mma_done, 1);
      *abort_ptr = 0;
      word[3] = 0;
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  } else if (warp == kWarpW && lane == 0) {
    prefetch_map(&map_w);
    prefetch_map(&map_x);
  }
  if (warp == kWarpMma) tmem_alloc(slot, 512);
  // The experts' rows and row tiles.  The offsets were complete before the expand kernel let this one start.
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
  if (warp == 0) {
    int before = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      const int e = e0 + lane;
      const int tiles = e < a.E ? (s_count[e] + NT - 1) / NT : 0;
      int sum = tiles;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, sum, off);
        if (lane >= off) sum += o;
      }
      if (e < a.E) s_first[e] = before + sum - tiles;
      before += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (lane == 0) s_first[a.E] = before;
  }
  __syncthreads();

  const int m_tiles = (a.N + kTileM - 1) / kTileM;
  // Tiles in the order (expert, channel tile, row tile).  The first `dealt` are dealt out by reduction blocks,
  // [my_begin, my_end) of them to this thread block; then come whole tiles, one in gridDim.x.
  const int64_t tiles = (int64_t)s_first[a.E] * m_tiles;
  // Dealing saves the idle part of a last wave, w_blocks * (1 - odd / grid) reduction blocks, and costs the FP32
  // sums' way through memory, measured as about ten blocks' time and one for 8 rows: 16 tiles of 32 blocks (2048 x
  // 4096) took 15 us dealt out and 19 not with 8 rows, 20 and 25 with 100; 56 tiles of 28 blocks (7168 x 3584) 17.8 and
  // 18.6 with 8 rows, 26 and 23 with 100; 64 tiles of 16 blocks were never better dealt out.
  const int odd = (int)(tiles % gridDim.x);
  const int64_t dealt = (int64_t)a.w_blocks * (gridDim.x - odd) > (int64_t)(10 + NT / 8) * gridDim.x ? odd : 0;
  const int64_t total = dealt * a.w_blocks;
  const int64_t worth = (total + kLeastBlocks - 1) / kLeastBlocks;
  const int64_t grid = worth < gridDim.x ? worth : gridDim.x;  // thread blocks with dealt work
  const int64_t my_begin = blockIdx.x < grid ? blockIdx.x * total / grid : 0;
  const int64_t my_end = blockIdx.x < grid ? (blockIdx.x + 1) * total / grid : 0;
  auto owner = [&](int64_t b) { return (int)(((b + 1) * grid + total - 1) / total) - 1; };  // the block that has b
  struct Walk {  // of this thread block's parts: the next dealt reduction block, the next whole tile
    int64_t dealt, tile;
  };
  const Walk start = {my_begin, dealt + blockIdx.x};
  auto next_part = [&](Walk& at, Part& q) {
    int64_t tile;
    if (at.dealt < my_end) {
      tile = at.dealt / a.w_blocks;
      q.k0 = (int)(at.dealt - tile * a.w_blocks);
      q.blocks = (int)min((int64_t)(a.w_blocks - q.k0), my_end - at.dealt);
      at.dealt += q.blocks;
    } else if (at.tile < tiles) {
      tile = at.tile;
      q.k0 = 0;
      q.blocks = a.w_blocks;
      at.tile += gridDim.x;
    } else {
      return false;
    }
    int lo = 0, hi = a.E - 1;  // the last expert whose tiles start at or before this one
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((int64_t)s_first[mid] * m_tiles <= tile) lo = mid;
      else hi = mid - 1;
    }
    const int row_tiles = s_first[lo + 1] - s_first[lo];
    const int left = (int)(tile - (int64_t)s_first[lo] * m_tiles);
    const int m = left / row_tiles, t = left - m * row_tiles;
    q.e = lo;
    q.m0 = m * kTileM;
    // an expert's row tiles are equal but for a few rows
    const int share = ((s_count[lo] + row_tiles - 1) / row_tiles + 15) & ~15;
    q.r0 = s_row[lo] + t * share;
    q.rows = min(share, s_count[lo] - t * share);  // at least one: NT * (row_tiles - 1) < s_count
    q.tile = tile;
    q.shared = row_tiles > 1;
    return true;
  };
  // The parts of a tile added up in the order of the reduction, scaled and written by warp w of `warps`: four rows at a
  // time, four channels a lane, four parts' loads in flight.
  auto add_parts = [&](const Split& q, int w, int warps) {
    const int n4 = q.m0 + 4 * lane;
    const float* scale4 = a.w_scale + (int64_t)q.e * a.N + n4;
    float ws[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) ws[i] = n4 < a.N ? scale4[i] : 0.0f;
#pragma unroll 1
    for (int r = 4 * w; r < q.rows; r += 4 * warps) {
      float4 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int s = q.first; s <= q.last; s += 4) {
        float4 u[4][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float* sums =
              a.partial + ((int64_t)(2 * (s + k) + (s + k == q.first ? 1 : 0)) * NT + r) * kTileM + 4 * lane;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            u[k][j] = s + k <= q.last ? __ldcg(reinterpret_cast<const float4*>(sums + j * kTileM))
                                      : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            v[j].x += u[k][j].x;
            v[j].y += u[k][j].y;
            v[j].z += u[k][j].z;
            v[j].w += u[k][j].w;
          }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (r + j >= q.rows || n4 >= a.N) continue;
        const float xs = a.x_scale[q.r0 + r + j];
        *reinterpret_cast<uint2*>(a.out + (int64_t)(q.r0 + r + j) * a.N + n4) =
            make_uint2(bf16x2_pz(v[j].x * ws[0] * xs, v[j].y * ws[1] * xs),
                       bf16x2_pz(v[j].z * ws[2] * xs, v[j].w * ws[3] * xs));
      }
    }
  };
  auto give_up = [&](unsigned bit) {
    if (!*abort_ptr) raise_error(bit);
    *abort_ptr = 1;
  };

  if (warp == kWarpW) {
    // ---------------- weight bytes ----------------
    // The warps that issue copies and MMAs walk their loops whole, so that the addresses stay in uniform
    // registers, and one lane issues.
    const uint64_t once = policy_evict_first(), again = policy_evict_last();
    int64_t g = 0;
    Ring w;
    bool ok = true;
    Part q;
    for (Walk at = start; ok && next_part(at, q);) {
      const uint64_t policy = q.shared ? again : once;
      for (int i = 0; i < q.blocks; ++i, ++g, w.step(a.w_stages)) {
        if (!warp_wait(w_empty + 8 * w.slot, w.parity ^ 1u, abort_ptr)) {  // the first round finds it free
          if (lane == 0) give_up(kErrWaitEmpty);
          ok = false;
          break;
        }
        if (elect_one()) {
          mbar_expect_tx(w_full + 8 * w.slot, kWStage);
          tma_load_3d(w_ring + w.slot * kWStage, &map_w, w_full + 8 * w.slot, (q.k0 + i) * kWBlock, q.m0, q.e, policy);
        }
        __syncwarp();
      }
    }
    if (lane == 0)
      for (int64_t i = g > a.w_stages ? g - a.w_stages : 0; i < g; ++i)  // copies in flight land before the block ends
        if (!mbar_wait(w_full + 8 * (i % a.w_stages), (uint32_t)(i / a.w_stages) & 1u)) raise_error(kErrWaitDrain);
    __syncwarp();
  } else if (warp == kWarpX) {
    // ---------------- FP16 rows ----------------
    grid_dependency_wait();  // the expand kernel's rows
    const uint64_t keep = policy_evict_last();
    int64_t g = 0;
    Ring x;
    bool ok = true;
    Part q;
    for (Walk at = start; ok && next_part(at, q);) {
      const int boxes = NT <= kBox ? 1 : (q.rows + kBox - 1) / kBox;
      for (int i = 0; i < kStepsOfStage * q.blocks; ++i, ++g, x.step(kSteps)) {
        if (!warp_wait(step_empty + 8 * x.slot, x.parity ^ 1u, abort_ptr)) {
          if (lane == 0) give_up(kErrWaitEmpty);
          ok = false;
          break;
        }
        if (elect_one()) {
          mbar_expect_tx(x_full + 8 * x.slot, (uint32_t)(kHalves * boxes * kBox * kXBlock * 2));
#pragma unroll
          for (int h = 0; h < kHalves; ++h)
            for (int c = 0; c < boxes; ++c)
              tma_load_2d(x_ring + x.slot * kXStage + h * kXHalf + c * kBox * kXBlock * 2, &map_x, x_full + 8 * x.slot,
                          (2 * q.k0 + kHalves * i + h) * kXBlock, q.r0 + c * kBox, keep);
        }
        __syncwarp();
      }
    }
    if (lane == 0)
      for (int64_t i = g > kSteps ? g - kSteps : 0; i < g; ++i)
        if (!mbar_wait(x_full + 8 * (i % kSteps), (uint32_t)(i / kSteps) & 1u)) raise_error(kErrWaitDrain);
    __syncwarp();
  } else if (warp == kWarpMma) {
    // ---------------- MMA issuer ----------------
    const unsigned long long limit = a.stage_wait_ns ? a.stage_wait_ns : kWaitLimitNs;
    Ring step, acc;
    bool ok = true;
    Part q;
    for (Walk at = start; ok && next_part(at, q); acc.step(kAccs)) {
      if (!warp_wait(acc_empty + 8 * acc.slot, acc.parity ^ 1u, abort_ptr)) {
        if (lane == 0) give_up(kErrWaitAccum);
        break;
      }
      const uint32_t idesc = idesc_f16(kTileM, (q.rows + 15) & ~15);
      const uint32_t d = tmem + acc.slot * NT;
      const int steps = kStepsOfStage * q.blocks;
      for (int i = 0; i < steps; ++i, step.step(kSteps)) {
        if (!warp_wait(step_full + 8 * step.slot, step.parity, abort_ptr, limit)) {
          if (lane == 0) give_up(kErrWaitFull);
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t bdesc = smem_desc_sw128(x_ring + step.slot * kXStage);
        const uint32_t w = tmem + kTmemA + step.slot * kStepColumns;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kHalves * kXBlock / 16; ++kk)  // 16 FP16: 8 columns of A, 32 bytes along B's swizzled row
            mma_f16_ts(d, w + 8 * kk, bdesc + (kk / 4) * (kXHalf >> 4) + 2 * (kk % 4), idesc, (i > 0 || kk > 0) ? 1u : 0u);
          mma_commit(step_empty + 8 * step.slot);
          if (i == steps - 1) mma_commit(acc_full + 8 * acc.slot);
        }
        __syncwarp();
      }
    }
    if (elect_one()) mma_commit(mma_done);  // the MMAs that were issued are done before tensor memory is freed
    __syncwarp();
    if (lane == 0 && !mbar_wait(mma_done, 0)) raise_error(kErrWaitAccum);
    __syncwarp();
  } else if (warp >= kEpilogueWarps) {
    // ---------------- int8 to FP16, one TMEM lane a thread ----------------
    // Set s takes the MMA steps s, s + kSets, ...: of a step that is half a weight stage, always the same half.
    constexpr int kStride = kSets / kStepsOfStage;  // weight stages from one step of a set to its next
    const int set = (warp - kEpilogueWarps) >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane, first_half = kHalves == 1 ? set % 2 : 0;
    Ring w, step;
    int ahead = set / kStepsOfStage;  // weight stages until this set's next one
    w.step(a.w_stages, ahead);
    step.slot = set;
    bool ok = true;
    Part q;
    for (Walk at = start; ok && next_part(at, q);) {
      for (; ahead < q.blocks; ahead += kStride, w.step(a.w_stages, kStride), step.step(kSteps, kSets)) {
        const uint32_t st = w_ring + w.slot * kWStage;
        const uint32_t dst = tmem + ((uint32_t)(quarter * 32) << 16) + kTmemA + step.slot * kStepColumns;
        if (!warp_wait(w_full + 8 * w.slot, w.parity, abort_ptr)) {
          if (lane == 0) give_up(kErrWaitFull);
          ok = false;
          break;
        }
#pragma unroll
        for (int h = 0; h < kHalves; ++h) {
          uint32_t r[32];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const uint4 v = ld_shared_v4(st + sw128_offset(row, 4 * (first_half + h) + u));
            int8x4_to_f16(v.x, r[8 * u], r[8 * u + 1]);
            int8x4_to_f16(v.y, r[8 * u + 2], r[8 * u + 3]);
            int8x4_to_f16(v.z, r[8 * u + 4], r[8 * u + 5]);
            int8x4_to_f16(v.w, r[8 * u + 6], r[8 * u + 7]);
          }
          if (h == 0) {
            ok = warp_wait(step_empty + 8 * step.slot, step.parity ^ 1u, abort_ptr);
            if (!ok) break;
            tc_fence_after();
          }
          tmem_st32(dst + h * kAColumns, r);
        }
        if (!ok) {
          if (lane == 0) give_up(kErrWaitEmpty);
          break;
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        // only now: the stores have taken what the loads brought, so nothing of the slot is still being read
        if (lane == 0) mbar_arrive(w_empty + 8 * w.slot);
        // one warp of the four sees the rows arrive too, so that the MMA warp has one barrier to wait for
        if (quarter == 0 && !warp_wait(x_full + 8 * step.slot, step.parity, abort_ptr)) {
          if (lane == 0) give_up(kErrWaitFull);
          ok = false;
          break;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(step_full + 8 * step.slot);
      }
      ahead -= q.blocks;
    }
  } else {
    // ---------------- accumulators to BF16 ----------------
    // A set of four warps reads every kReaders-th run of 16 columns.
    const int reader = warp >> 2, quarter = warp & 3;
    grid_dependency_wait();  // the counters
    Ring acc;
    bool ok = true;
    Part q;
    for (Walk at = start; ok && next_part(at, q); acc.step(kAccs)) {
      const int buf = acc.slot;
      const int n = q.m0 + quarter * 32 + lane;
      // the scales, while the MMAs run
      const float ws = n < a.N ? a.w_scale[(int64_t)q.e * a.N + n] : 0.0f;
      for (int i = lane; i < NT / kReaders; i += 32) {
        const int r = (i / kRun * kReaders + reader) * kRun + i % kRun;
        s_scale[i] = r < q.rows ? a.x_scale[q.r0 + r] : 0.0f;
      }
      __syncwarp();
      ok = warp_wait(acc_full + 8 * buf, acc.parity, abort_ptr);
      const bool whole = q.blocks == a.w_blocks;
      ok = all_of<32 * kEpilogueWarps>(ok);  // one answer for the warps that meet at barriers below
      if (!ok) {
        if (lane == 0) give_up(kErrWaitAccum);
        break;
      }
      tc_fence_after();
      const uint32_t src = tmem + ((uint32_t)(quarter * 32) << 16) + buf * NT;
      // FP32 sums [row][channel] of this thread block's part of a tile, this thread's channel
      float* mine = a.partial + (int64_t)(2 * blockIdx.x + (q.k0 == 0 ? 1 : 0)) * NT * kTileM + quarter * 32 + lane;
      // Columns c .. c + 15 of the set's accumulator rows, scaled, to the result: by shared memory, so that a row's
      // 128 channels leave as whole lines (two bytes a lane left 64 bytes at a time, and the tensor cores waited).
      auto finish16 = [&](const float (&v)[16], int c) {
        const uint32_t mine16 = staging + 2 * (quarter * 32 + lane);
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const uint4 s = ld_shared_v4(scales + 4 * (c / (kRun * kReaders) * kRun + i));
          const float sc[4] = {__uint_as_float(s.x), __uint_as_float(s.y), __uint_as_float(s.z), __uint_as_float(s.w)};
#pragma unroll
          for (int j = 0; j < 4; j += 2) {
            const uint32_t two = bf16x2_pz(v[i + j] * ws * sc[j], v[i + j + 1] * ws * sc[j + 1]);
            st_shared_u16(mine16 + (i + j) * (2 * kTileM), two);
            st_shared_u16(mine16 + (i + j + 1) * (2 * kTileM), two >> 16);
          }
        }
        set_bar(reader);
        const int u = (quarter * 32 + lane) & 15;  // 8 channels of rows quarter * 2 + lane / 16 and 8 further
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = 8 * i + quarter * 2 + (lane >> 4);
          const uint4 eight = ld_shared_v4(staging + r * (2 * kTileM) + 16 * u);
          if (c + r < q.rows && q.m0 + 8 * u < a.N) st_v4(a.out + (int64_t)(q.r0 + c + r) * a.N + q.m0 + 8 * u, eight);
        }
        set_bar(reader);
      };
#pragma unroll 1
      for (int c = 16 * reader; c < q.rows; c += 16 * kReaders) {
        float v[16];
        together();
        tmem_ld16(src + c, v);
        if (whole) {
          finish16(v, c);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) mine[(c + i) * kTileM] = v[i];
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_empty + 8 * buf);
      if (!whole) {
        const int first = owner(q.tile * a.w_blocks), last = owner((q.tile + 1) * a.w_blocks - 1);
        __threadfence();
        all_of<32 * kEpilogueWarps>(true);
        if (threadIdx.x == 0) word[2] = atomicAdd(&a.counters[first], 1u);
        all_of<32 * kEpilogueWarps>(true);
        if (word[2] == (unsigned)(last - first)) {  // the tile's last missing part: add them all, in order
          __threadfence();
          const Split tile = {q.e, q.m0, q.r0, q.rows, first, last};
          if (tiles >= gridDim.x) add_parts(tile, warp, kEpilogueWarps);  // whole tiles follow: their MMAs go on meanwhile
          else if (threadIdx.x == 0) s_split[word[3]++] = tile;           // nothing does: every warp helps, at the end
        }
        all_of<32 * kEpilogueWarps>(true);  // before word[2] is written again
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpMma) tmem_dealloc(tmem, 512);
  if (!*abort_ptr) {
    __threadfence();
    for (unsigned i = 0; i < word[3]; ++i) add_parts(s_split[i], warp, kThreads / 32);
  }
}

// ---- host ----------------------------------------------------------------------------

// Rows of a tile: all of them where one expert has few, else twice an expert's average share, so that an uneven
// batch still has one row tile for most experts.  Tiles of 128 go further, up to twice as many rows: they have a
// second accumulator and half the steps (128 experts of 2048 x 4096: 128 rows each on average 316 us, 349 with tiles of
// 256; 32 rows each 200 us with 64, 243 with 256; 256 rows each 508 us with 256, 537 with 128).
int rows_of_tile(int64_t R, int E) {
  const int64_t want = E == 1 ? R : 2 * ((R + E - 1) / E);
  return want <= 16 ? 16 : want <= 32 ? 32 : want <= 64 ? 64 : want <= 256 ? 128 : 256;
}

size_t round_up(size_t n, size_t to) { return (n + to - 1) / to * to; }

struct Layout {  // of the workspace, from its 256-aligned start
  size_t x16, counters, partial, bytes;
};
Layout layout(int64_t R, int E, int D) {
  Layout l;
  l.x16 = 0;
  l.counters = round_up((size_t)R * D * 2, 256);
  l.partial = l.counters + round_up(kMaxGrid * 4, 256);
  l.bytes = l.partial + (size_t)2 * kMaxGrid * kTileM * rows_of_tile(R, E) * 4;
  return l;
}

template <int NT>
cudaError_t launch_nt(const CUtensorMap& map_w, const CUtensorMap& map_x, Args& a, int sms, cudaStream_t stream) {
  constexpr int kLimit = 227 * 1024;
  constexpr int kXStage = halves_of(NT) * NT * kXBlock * 2;
  const int fixed = 1024 + 96 + 16 * NT + readers_of(NT) * kStaging + 4 * (3 * a.E + 1) + 8 * (2 * 12 + 3 * 15 + 2 * 2 + 1);
  constexpr int kSteps = steps_of(NT);
  a.w_stages = (kLimit - fixed - kSteps * kXStage) / kWStage;
  if (a.w_stages > 12) a.w_stages = 12;
  // A set of converting warps that takes every second stage must meet the same slots in every round: else it could ask
  // for a slot's next round while the other set's copy in it is still on its way, and the parity of the round before
  // would tell it that its own had landed.
  constexpr int kStride = kSets * halves_of(NT) / 2;
  a.w_stages -= a.w_stages % kStride;
  auto kernel = expert_product_kernel<NT>;
  cudaError_t e = ensure_smem_limit((const void*)kernel, kLimit);
  if (e != cudaSuccess) return e;
  const size_t smem = fixed + (size_t)kSteps * kXStage + (size_t)a.w_stages * kWStage;
  return launch_pdl(kernel, dim3(sms < kMaxGrid ? sms : kMaxGrid), dim3(threads_of(NT)), smem, stream, map_w, map_x, a);
}

}  // namespace

size_t expert_product_workspace(int64_t R, int E, int, int D) { return layout(R, E, D).bytes; }

int product_rows_of_tile(int64_t R, int E) { return rows_of_tile(R, E); }

cudaError_t launch_expert_product(const ProductArgs& p, const CUtensorMap& map_w, const CUtensorMap& map_x,
                                  void* workspace, int sms, cudaStream_t stream) {
  const Layout l = layout(p.R, p.E, p.D);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  Args a;
  a.x_scale = p.x_scale;
  a.w_scale = p.w_scale;
  a.offsets = p.offsets;
  a.out = p.out;
  a.partial = reinterpret_cast<float*>(ws + l.partial);
  a.counters = reinterpret_cast<unsigned*>(ws + l.counters);
  a.R = p.R;
  a.E = p.E;
  a.N = p.N;
  a.w_blocks = (p.D + kWBlock - 1) / kWBlock;
  a.stage_wait_ns = stage_wait_limit_ns();
  const int64_t vectors = p.R * p.D / 16;
  const int64_t blocks = (vectors + 256 * kExpand - 1) / (256 * kExpand);
  // at most as many blocks as run at once, so that none is left to start when the product's blocks take the SMs
  const int most = 5 * sms;
  cudaError_t e = launch_pdl(expand_rows_kernel, dim3((unsigned)(blocks < most ? blocks : most)), dim3(256), 0, stream, p.x,
                             reinterpret_cast<uint16_t*>(ws + l.x16), p.offsets, p.E, p.R, p.D, a.counters);
  if (e != cudaSuccess) return e;
  switch (rows_of_tile(p.R, p.E)) {
    case 16: return launch_nt<16>(map_w, map_x, a, sms, stream);
    case 32: return launch_nt<32>(map_w, map_x, a, sms, stream);
    case 64: return launch_nt<64>(map_w, map_x, a, sms, stream);
    case 128: return launch_nt<128>(map_w, map_x, a, sms, stream);
    default: return launch_nt<256>(map_w, map_x, a, sms, stream);
  }
}

cudaError_t take_product_error(unsigned* bits) {
  unsigned v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_product_error, sizeof v);
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_product_error, &zero, sizeof zero);
  *bits = v;
  return e;
}

}  // namespace moetail
