// Product with 4-bit weights, a scale for each group of columns and each channel, dense or by expert (sm_103a).
//
//   p[r][n] = (sum over k of x[r][k] * (gs[e][n][k / G] * q[e][n][k])) * cs[e][n],  r in [offsets[e], offsets[e + 1])
//   out = bf16(p),  or for a gated weight of 2 I channels  bf16(silu(p[r][i]) * p[r][I + i])
//
// x BF16, q in [-8, 7], gs e4m3, cs FP32.  A BF16 times a q is exact in FP32, and a q times a gs (three and four
// significant bits) is exact in BF16, so the tensor cores' products are exact either way and only their FP32 sums round.
//
// Most calls take the tiles of product_i4_tiles.cu.  Here is the kernel for at most eight rows and too few tiles to occupy
// the SMs: one dense weight and a token or a few.  A thread block takes 32 channels, its eight warps a block of 128 columns
// each, as mma.sync operands made in registers; two copies bring a step of 1024 columns, weights and rows, so that the first
// bytes are asked for at once and latency is what is left: one token by 7168 x 3584 takes 7.2 us on the device (a call from
// Python 8), 1.8 TB/s of packed weights
// (24 copies a step took 8.2, the tiles 9.3).  Wider, the tiles are faster (one token by 12288 x 4096: 11.1 us, 11.8 here).
#include "kernels.h"
#include "layer.h"
#include "product_i4.cuh"

namespace moetail {

namespace {

__device__ unsigned int g_i4_error = 0;
__device__ __forceinline__ void raise_error(unsigned bit) { atomicOr(&g_i4_error, bit); }

struct Args {
  const uint8_t* group_scale;  // e4m3 [E][channels][pitch]
  const float* channel_scale;  // [E][channels]
  const int32_t* offsets;      // [E + 1] or null
  uint16_t* out;               // [R][N]
  int64_t R;
  int E, N;                    // N: channels of the result
  int blocks;                  // of 128 columns: ceil(D / 128)
  int groups, pitch;           // scales of a channel, and their distance to the next channel's
  bool whole;                  // D is a multiple of 64: map_x has the columns in sixty-fours
  unsigned long long stage_wait_ns;
};

// D = A (16 channels x 16 columns) * B (16 columns x 8 rows) + C, BF16, FP32 sums.
__device__ __forceinline__ void mma_16x8x16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The same with C = 0.
__device__ __forceinline__ void mma_16x8x16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}

// ---- few rows and few tiles ------------------------------------------------------------------------------------------

constexpr int kWarps = 8;                       // that multiply; one more brings the data
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kRows = 8;                        // of a tile: the MMA's N
constexpr int kChannels = 32;                   // stored ones of a tile: two MMAs' 16
constexpr int kRowBytes = kWarps * 64;          // of a channel in a stage: a block for each warp
constexpr int kWeights = kChannels * kRowBytes, kXBlock = kRows * 256, kStage = kWeights + kWarps * kXBlock;
constexpr int kStages = 3;                      // 96 KB: two thread blocks an SM
constexpr int kWideFrom = 256;                  // rows of a tile that would be wanted from which wide ones pay: see the plan
constexpr int kMostExperts = 256;               // whose rows fit shared memory beside the stages
constexpr int kPadded = 40;                     // floats of a row of a warp's 32 channels: no two lanes in one bank

// A tile: `rows` rows from r0 by channels from n0 (of the result) of expert e.
struct Tile {
  int e, n0, r0, rows;
};

template <int GROUP, bool GATED>
__global__ void __launch_bounds__(kThreads, 2)
    product_i4_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, const Args a) {
  constexpr int kPer = 128 / GROUP;             // groups of a block
  constexpr int kOut = GATED ? kChannels / 2 : kChannels;
  extern __shared__ uint8_t smem_raw[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* base_ptr = smem_raw + (base - raw);
  uint32_t at = kStages * kStage;
  float* s_red = reinterpret_cast<float*>(base_ptr + at);  // [warps][8 rows][kPadded]
  at += kWarps * kRows * kPadded * 4;
  const uint32_t full = base + at, empty = full + 8 * kStages;
  at += 16 * kStages;
  volatile uint32_t* abort_ptr = reinterpret_cast<volatile uint32_t*>(base_ptr + at);
  int32_t* s_first = reinterpret_cast<int32_t*>(base_ptr + at + 16);  // [E + 1] row tiles before an expert
  int32_t* s_row = s_first + a.E + 1;                                  // [E] its first row
  int32_t* s_count = s_row + a.E;                                      // [E] its rows

  if (warp == kWarps) {
    if (lane < kStages) {
      mbar_init(full + 8 * lane, 1);
      mbar_init(empty + 8 * lane, kWarps);
    }
    if (lane == 0) *abort_ptr = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    if (lane == 0) {
      prefetch_map(&map_w);
      prefetch_map(&map_x);
    }
  }
  grid_dependency_wait();
  launch_dependents();
  for (int e = threadIdx.x; e < a.E; e += kThreads) {
    const int begin = a.offsets ? clamp_row(a.offsets[e], a.R) : 0;
    const int end = a.offsets ? clamp_row(a.offsets[e + 1], a.R) : (int)a.R;
    s_row[e] = begin;
    s_count[e] = end > begin ? end - begin : 0;
  }
  __syncthreads();
  if (warp == 0) row_tiles_before(s_count, s_first, a.E, kRows);
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
    q.r0 = s_row[e] + t * kRows;
    q.rows = min(kRows, s_count[e] - t * kRows);
    return true;
  };
  auto give_up = [&](unsigned bit) {
    if (!*abort_ptr) raise_error(bit);
    *abort_ptr = 1;
  };
  const int steps = (a.blocks + kWarps - 1) / kWarps;

  if (warp == kWarps) {
    // ---------------- copies ----------------
    const uint64_t once = policy_evict_first(), keep = policy_evict_last();
    int64_t g = 0;
    Ring ring;
    bool ok = true;
    Tile q;
    for (int64_t i = blockIdx.x; ok && tile_at(i, q); i += gridDim.x) {
      for (int s = 0; s < steps; ++s, ++g, ring.step(kStages)) {
        if (!warp_wait(empty + 8 * ring.slot, ring.parity ^ 1u, abort_ptr)) {  // the first round finds it free
          if (lane == 0) give_up(kErrWaitEmpty);
          ok = false;
          break;
        }
        const uint32_t bar = full + 8 * ring.slot, w = base + ring.slot * kStage, x = w + kWeights;
        if (elect_one()) {
          mbar_expect_tx(bar, kStage);  // what is out of range arrives as zeros
          if (GATED) tma_load_4d(w, &map_w, bar, s * (kRowBytes / 4), q.n0, 0, q.e, once);
          else tma_load_3d(w, &map_w, bar, s * (kRowBytes / 4), q.n0, q.e, once);
          if (a.whole) {
            tma_load_3d(x, &map_x, bar, 0, q.r0, 2 * kWarps * s, keep);
          } else {
            for (int k = 0; k < 2 * kWarps; ++k)
              tma_load_2d(x + k * (kXBlock / 2), &map_x, bar, 128 * kWarps * s + 64 * k, q.r0, keep);
          }
        }
        __syncwarp();
      }
    }
    if (lane == 0)
      for (int64_t i = g > kStages ? g - kStages : 0; i < g; ++i)  // copies in flight land before the block ends
        if (!mbar_wait(full + 8 * (i % kStages), (uint32_t)(i / kStages) & 1u)) raise_error(kErrWaitDrain);
    return;
  }

  // ---------------- products ----------------
  // Lane 4 g + t holds channels g and g + 8 of the MMA's A, columns of 8 t .. 8 t + 7 of every 32, and of B the row that
  // is column g of the result.  A word's eight columns feed two MMAs, four columns a lane each: the order in which the
  // columns are summed is free as long as both operands have the same.
  const unsigned long long limit = a.stage_wait_ns ? a.stage_wait_ns : kWaitLimitNs;
  const int g = lane >> 2, t = lane & 3;
  const int channels = GATED ? 2 * a.N : a.N;
  const int x_row = (g >> 1) | ((g & 1) << 2);  // columns 2 t and 2 t + 1 of the result are rows t and t + 4: no bank conflicts
  // a lane's channels: of the stage at 8 g' + g, g' = 0 .. 3 as the MMAs' halves (gated: the gates, then their ups)
  auto staged = [&](int j, int h) { return GATED ? 8 * j + 16 * h + g : 16 * j + 8 * h + g; };
  auto channel = [&](const Tile& q, int j, int h) {  // past the last: the last
    return GATED ? min(q.n0 + 8 * j + g, a.N - 1) + h * a.N : min(q.n0 + 16 * j + 8 * h + g, a.N - 1);
  };
  // Four of the scales of each, those of a block among them; what stands behind the last group counts as zero.
  auto load_scales = [&](const Tile& q, int block, uint32_t (&s)[2][2]) {
    const int first = block * kPer & ~3, left = a.groups - first;
    if (left <= 0) return;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        s[j][h] = __ldg(reinterpret_cast<const uint32_t*>(a.group_scale + ((int64_t)q.e * channels + channel(q, j, h)) * a.pitch + first));
        if (left < 4) s[j][h] &= (1u << (8 * left)) - 1u;
      }
  };
  const Factors factors = unscaled();
  Ring ring;
  bool ok = true;
  Tile q;
  for (int64_t i = blockIdx.x; tile_at(i, q); i += gridDim.x) {
    float acc[2][4], cs[2][2];
    uint32_t ahead[2][2] = {{0, 0}, {0, 0}};
    load_scales(q, warp, ahead);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) cs[j][h] = kScaled * __ldg(a.channel_scale + (int64_t)q.e * channels + channel(q, j, h));
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[j][c] = 0.0f;
    for (int s = 0; s < steps; ++s, ring.step(kStages)) {
      const int block = s * kWarps + warp;
      uint32_t scales[2][2];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) scales[j][h] = ahead[j][h] >> (8 * (block * kPer & 3));
      if (ok && !warp_wait(full + 8 * ring.slot, ring.parity, abort_ptr, limit)) {
        if (lane == 0) give_up(kErrWaitFull);
        ok = false;
      }
      if (!ok) continue;  // the tiles are walked to the end: the warps meet at barriers
      load_scales(q, block + kWarps, ahead);  // not before a wait: that would wait for them too
      if (block < a.blocks) {
        const uint32_t w = base + ring.slot * kStage + warp * 64 + 16 * t;
        const uint32_t x = base + ring.slot * kStage + kWeights + warp * kXBlock + x_row * 128;
        uint4 rows[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) rows[c] = ld_shared_v4(x + (c >> 1) * (kXBlock / 2) + (((4 * (c & 1) + t) ^ x_row) << 4));
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint4 wl = ld_shared_v4(w + staged(j, 0) * kRowBytes), wh = ld_shared_v4(w + staged(j, 1) * kRowBytes);
          float sum[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {  // 32 columns
            uint32_t l[4], h[4];
            int4x8_to_bf16(c == 0 ? wl.x : c == 1 ? wl.y : c == 2 ? wl.z : wl.w, factors, l);
            int4x8_to_bf16(c == 0 ? wh.x : c == 1 ? wh.y : c == 2 ? wh.z : wh.w, factors, h);
            const uint32_t a0[4] = {l[0], h[0], l[1], h[1]}, a1[4] = {l[2], h[2], l[3], h[3]};
            if (32 * c % GROUP == 0) mma_16x8x16_first(sum, a0, rows[c].x, rows[c].y);
            else mma_16x8x16(sum, a0, rows[c].x, rows[c].y);
            mma_16x8x16(sum, a1, rows[c].z, rows[c].w);
            if ((32 * c + 32) % GROUP == 0) {  // the group ends
              const int shift = 8 * (32 * c / GROUP);
              const float sl = e4m3_value(scales[j][0] >> shift), sh = e4m3_value(scales[j][1] >> shift);
              acc[j][0] += sl * sum[0];
              acc[j][1] += sl * sum[1];
              acc[j][2] += sh * sum[2];
              acc[j][3] += sh * sum[3];
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + 8 * ring.slot);  // its products have taken what the loads brought
    }
    // The warps' sums to shared memory, then added in the order of the warps, a channel of a row a thread.
    float* to = s_red + warp * kRows * kPadded;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      to[t * kPadded + staged(j, 0)] = acc[j][0] * cs[j][0];
      to[(t + 4) * kPadded + staged(j, 0)] = acc[j][1] * cs[j][0];
      to[t * kPadded + staged(j, 1)] = acc[j][2] * cs[j][1];
      to[(t + 4) * kPadded + staged(j, 1)] = acc[j][3] * cs[j][1];
    }
    asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory");
    const int n = lane % kOut;
    float v = 0.0f, u = 0.0f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      v += s_red[(k * kRows + warp) * kPadded + n];
      if (GATED) u += s_red[(k * kRows + warp) * kPadded + kOut + n];
    }
    if (GATED) v = silu_times(v, u);
    if (ok && warp < q.rows && lane < kOut && q.n0 + n < a.N) a.out[(int64_t)(q.r0 + warp) * a.N + q.n0 + n] = (uint16_t)bf16_bits_pz(v);
    asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory");
  }
}

// ---- host --------------------------------------------------------------------------------------------------------------

template <int GROUP, bool GATED>
cudaError_t launch(const ProductI4Args& p, const CUtensorMap& map_w, const CUtensorMap& map_x, int sms, cudaStream_t stream) {
  constexpr int kLimit = 113 * 1024, kOut = GATED ? kChannels / 2 : kChannels;  // two thread blocks an SM
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
  a.whole = p.D % 64 == 0;
  a.stage_wait_ns = stage_wait_limit_ns();
  auto kernel = product_i4_kernel<GROUP, GATED>;
  cudaError_t e = ensure_smem_limit((const void*)kernel, kLimit);
  if (e != cudaSuccess) return e;
  // no more thread blocks than there can be tiles
  const int64_t row_tiles = p.E == 1 ? (p.R + kRows - 1) / kRows : p.R / kRows + (p.R < p.E ? p.R : p.E);
  const int64_t most = row_tiles * ((p.N + kOut - 1) / kOut);
  const size_t smem = 1024 + kStages * kStage + kWarps * kRows * kPadded * 4 + 16 * kStages + 16 + 4 * (3 * p.E + 1);
  return launch_pdl(kernel, dim3((unsigned)(most < 2 * sms ? most : 2 * sms)), dim3(kThreads), smem, stream, map_w, map_x, a);
}

}  // namespace

ProductI4Plan product_i4_plan(int64_t R, int E, int N, int D, bool gated, int sms) {
  ProductI4Plan p;
  // Rows of a tile: all of them where one expert has few, else twice an expert's average share, so that an uneven batch
  // still has one row tile for most experts.
  const int64_t want = E == 1 ? R : 2 * ((R + E - 1) / E);
  const int64_t hit = R < E ? R : E;  // experts with a row, at most
  p.tiles = want > kRows || hit * ((N + 127) / 128) * (gated ? 2 : 1) >= sms / 2 || E > kMostExperts;
  p.wide = false;
  if (p.tiles) {
    // Wide tiles pay from about 128 rows an expert on, where there is one for each SM, by 10 to 20%: 128 experts of 4096 x 2048
    // with 256 rows each take 421 us in wide tiles and 520 in tiles of 64, with 137 each 270 and 320; 60 of 1408 x 2048 with
    // 192 each 63 and 71, gated 114 and 135.  Near the border it depends on how the tiles fill the rounds: those 60 with 137
    // rows each 58 and 56.5, gated 98 and 109; 8 of 4096 x 4096 with 160 each 49 and 53.5, with 129 51 and 39.  The rows
    // counted are the buffer's: where an eighth of them have an expert here (512 tokens x 8 routes, 16 experts of 128), wide
    // ones take 23 us and the others 21 (gated 1024 x 4096), 15 and 13 (4096 x 1024).  One expert's 1024 rows by 4096 x 4096
    // (128 wide tiles) take 35 us in tiles of 64 and would take 28.5.
    const int64_t row_tiles = E == 1 ? (R + 127) / 128 : R / 128 + hit;  // of a wide tile's rows
    p.wide = want > kWideFrom && row_tiles * ((N + 255) / 256) * (gated ? 2 : 1) >= sms;
    p.rows = p.wide ? 128 : want <= 16 ? 16 : want <= 32 ? 32 : 64;
    p.box_columns = 128;
    p.box_channels = (gated ? 64 : 128) * (p.wide ? 2 : 1);
    p.box_rows = p.rows;
    p.box_chunks = D % 64 ? 0 : p.wide ? 2 : 4;
  } else {
    p.rows = kRows;
    p.box_columns = kRowBytes;
    p.box_channels = gated ? kChannels / 2 : kChannels;
    p.box_rows = kRows;
    p.box_chunks = D % 64 ? 0 : 2 * kWarps;
  }
  return p;
}

cudaError_t launch_product_i4(const ProductI4Args& p, const ProductI4Plan& plan, const CUtensorMap& map_w,
                              const CUtensorMap& map_x, int sms, cudaStream_t stream) {
  if (plan.tiles) return launch_product_i4_tiles(p, plan, map_w, map_x, sms, stream);
  if (p.gated)
    return p.group == 32   ? launch<32, true>(p, map_w, map_x, sms, stream)
           : p.group == 64 ? launch<64, true>(p, map_w, map_x, sms, stream)
                           : launch<128, true>(p, map_w, map_x, sms, stream);
  return p.group == 32   ? launch<32, false>(p, map_w, map_x, sms, stream)
         : p.group == 64 ? launch<64, false>(p, map_w, map_x, sms, stream)
                         : launch<128, false>(p, map_w, map_x, sms, stream);
}

cudaError_t take_product_i4_error(unsigned* bits) {
  unsigned v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_i4_error, sizeof v);
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_i4_error, &zero, sizeof zero);
  *bits = v;
  return e;
}

}  // namespace moetail
