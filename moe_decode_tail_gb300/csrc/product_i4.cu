// Product with 4-bit weights, a scale for each group of columns and each channel, dense or by expert (sm_103a).
//
//   p[r][n] = (sum over k of x[r][k] * (gs[e][n][k / G] * q[e][n][k])) * cs[e][n],  r in [offsets[e], offsets[e + 1])
//   out = bf16(p),  or for a gated weight of 2 I channels  bf16(silu(p[r][i]) * p[r][I + i])
//
// x BF16, q in [-8, 7], gs e4m3, cs FP32.  A BF16 times a q is exact in FP32, and a q times a gs (three and four
// significant bits) is exact in BF16, so the tensor cores' products are exact either way and only their FP32 sums round.
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
  int stages;
  int splits;                  // warps along the reduction
  int depth;                   // blocks of a warp in a stage
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

// ---- few rows for an expert ------------------------------------------------------------------------------------------

constexpr int kWarps = 8;                       // that multiply; one more brings the data
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kWarpTile = 32;                   // channels of a warp: two MMAs' 16
constexpr int kWeightBlock = kWarpTile * 64;    // bytes of 128 columns of them
constexpr int blocks_per_sm(int nt) { return nt > 2 ? 1 : 2; }  // as registers allow
constexpr int kPadded = 40;                     // floats of a row of a warp's 32 channels: no two lanes in one bank

// A tile: `rows` rows from r0 by channels from n0 (of the result) of expert e.
struct Tile {
  int e, n0, r0, rows;
};

template <int NT, int GROUP, bool GATED>
__global__ void __launch_bounds__(kThreads, blocks_per_sm(NT))
    product_i4_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, const Args a) {
  constexpr int kRows = 8 * NT;
  constexpr int kPer = 128 / GROUP;             // groups of a block
  constexpr int kXBlock = kRows * 256;          // bytes of 128 columns of a tile's rows
  extern __shared__ uint8_t smem_raw[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* base_ptr = smem_raw + (base - raw);
  const int across = kWarps / a.splits;         // warps along the channels
  const int step_blocks = a.splits * a.depth;   // of a stage; a warp has every splits-th of them
  const int weights_bytes = a.depth * kWarps * kWeightBlock, stage_bytes = weights_bytes + step_blocks * kXBlock;
  uint32_t at = base + (uint32_t)(a.stages * stage_bytes);
  const uint32_t red = at;
  float* s_red = reinterpret_cast<float*>(base_ptr + (red - base));  // [warps][8 rows][kPadded]
  at += kWarps * 8 * kPadded * 4;
  const uint32_t full = at, empty = at + 8 * a.stages;
  at += 16 * a.stages;
  volatile uint32_t* abort_ptr = reinterpret_cast<volatile uint32_t*>(base_ptr + (at - base));
  int32_t* s_first = reinterpret_cast<int32_t*>(base_ptr + (at - base) + 16);  // [E + 1] row tiles before an expert
  int32_t* s_row = s_first + a.E + 1;                                           // [E] its first row
  int32_t* s_count = s_row + a.E;                                               // [E] its rows

  if (warp == kWarps) {
    for (int s = lane; s < a.stages; s += 32) {
      mbar_init(full + 8 * s, 1);
      mbar_init(empty + 8 * s, kWarps);
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

  const int per_tile = (GATED ? 16 : kWarpTile) * across;  // channels of the result of a tile
  const int n_tiles = (a.N + per_tile - 1) / per_tile;
  const int64_t tiles = (int64_t)s_first[a.E] * n_tiles;
  auto tile_at = [&](int64_t i, Tile& q) {  // in the order (expert, channel tile, row tile)
    if (i >= tiles) return false;
    const int e = expert_of_tile(s_first, a.E, n_tiles, i);
    const int row_tiles = s_first[e + 1] - s_first[e];
    const int left = (int)(i - (int64_t)s_first[e] * n_tiles);
    const int n = left / row_tiles, t = left - n * row_tiles;
    q.e = e;
    q.n0 = n * per_tile;
    q.r0 = s_row[e] + t * kRows;
    q.rows = min(kRows, s_count[e] - t * kRows);
    return true;
  };
  auto give_up = [&](unsigned bit) {
    if (!*abort_ptr) raise_error(bit);
    *abort_ptr = 1;
  };
  const int steps = (a.blocks + step_blocks - 1) / step_blocks;

  if (warp == kWarps) {
    // ---------------- copies ----------------
    const uint64_t once = policy_evict_first(), keep = policy_evict_last();
    int64_t g = 0;
    Ring ring;
    bool ok = true;
    Tile q;
    for (int64_t i = blockIdx.x; ok && tile_at(i, q); i += gridDim.x) {
      for (int s = 0; s < steps; ++s, ++g, ring.step(a.stages)) {
        if (!warp_wait(empty + 8 * ring.slot, ring.parity ^ 1u, abort_ptr)) {  // the first round finds it free
          if (lane == 0) give_up(kErrWaitEmpty);
          ok = false;
          break;
        }
        const int here = min(step_blocks, a.blocks - s * step_blocks);  // blocks of this step
        const uint32_t bar = full + 8 * ring.slot, w = base + ring.slot * stage_bytes, x = w + weights_bytes;
        if (elect_one()) {
          mbar_expect_tx(bar, (uint32_t)(here * (across * kWeightBlock + kXBlock)));
          for (int k = 0; k < here; ++k) {
            const int block = s * step_blocks + k;
            if (GATED) tma_load_4d(w + k * across * kWeightBlock, &map_w, bar, 64 * block, q.n0, 0, q.e, once);
            else tma_load_3d(w + k * across * kWeightBlock, &map_w, bar, 64 * block, q.n0, q.e, once);
            tma_load_2d(x + k * kXBlock, &map_x, bar, 128 * block, q.r0, keep);
            tma_load_2d(x + k * kXBlock + kXBlock / 2, &map_x, bar, 128 * block + 64, q.r0, keep);
          }
        }
        __syncwarp();
      }
    }
    if (lane == 0)
      for (int64_t i = g > a.stages ? g - a.stages : 0; i < g; ++i)  // copies in flight land before the block ends
        if (!mbar_wait(full + 8 * (i % a.stages), (uint32_t)(i / a.stages) & 1u)) raise_error(kErrWaitDrain);
    return;
  }

  // ---------------- products ----------------
  // Lane 4 g + t holds channels g and g + 8 of the MMA's A, columns of 8 t .. 8 t + 7 of every 32, and of B the row that
  // is column g of the result.  A word's eight columns feed two MMAs, four columns a lane each: the order in which the
  // columns are summed is free as long as both operands have the same.
  const unsigned long long limit = a.stage_wait_ns ? a.stage_wait_ns : kWaitLimitNs;
  const int g = lane >> 2, t = lane & 3;
  const int mine = warp / a.splits, split = warp - mine * a.splits;
  const int channels = GATED ? 2 * a.N : a.N;
  const int x_row = (g >> 1) | ((g & 1) << 2);  // columns 2 t and 2 t + 1 of the result are rows t and t + 4: no bank conflicts
  int local[2][2], channel0[2][2];              // a lane's channels in the staged tile, and from the tile's first
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    local[j][0] = GATED ? 16 * mine + 8 * j + g : kWarpTile * mine + 16 * j + g;
    local[j][1] = local[j][0] + (GATED ? 16 * across : 8);
    channel0[j][0] = local[j][0];
    channel0[j][1] = local[j][0] + (GATED ? a.N : 8);
  }
  // Where the lane's channels' scales begin.  Channels past the last read the last one's.
  const uint8_t* scale_base = nullptr;
  uint32_t scale_at[2][2];
  auto scales_of = [&](const Tile& q) {
    scale_base = a.group_scale + (int64_t)q.e * channels * a.pitch;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int past = GATED && h ? a.N : 0;
        scale_at[j][h] = (uint32_t)(min(q.n0 + channel0[j][h] - past, a.N - 1) + past) * (uint32_t)a.pitch;
      }
  };
  // Four of the scales of each: word i of them; what stands behind the last group counts as zero.
  auto load_scales = [&](int i, uint32_t (&s)[2][2]) {
    const int left = a.groups - 4 * i;
    if (left <= 0) return;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        s[j][h] = __ldg(reinterpret_cast<const uint32_t*>(scale_base + (scale_at[j][h] + 4u * i)));
    if (left < 4) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) s[j][h] &= (1u << (8 * left)) - 1u;
    }
  };
  const uint32_t w_lane = base + split * across * kWeightBlock + local[0][0] * 64 + 16 * t;
  const uint32_t w_half = (local[0][1] - local[0][0]) * 64;  // from a lane's channel in the upper half of A's rows to the lower
  const uint32_t x_lane = base + weights_bytes + split * kXBlock + x_row * 128;
  const uint32_t x_unit[2] = {x_lane + ((t ^ x_row) << 4), x_lane + (((4 + t) ^ x_row) << 4)};
  const Factors factors = unscaled();
  int slot = 0;
  uint32_t parity = 0, slot_at = 0;
  bool ok = true;
  Tile q, next;
  uint32_t scales[2][2], ahead[2][2];  // of the block at hand, and the words after them
  int64_t i = blockIdx.x;
  bool more = tile_at(i, q);
  if (more) {
    scales_of(q);
    load_scales(split * kPer / 4, ahead);
  }
  while (more) {
    i += gridDim.x;
    more = tile_at(i, next);
    const int row_groups = (q.rows + 7) >> 3;
    float acc[2][NT][4];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[j][n][c] = 0.0f;
    int word = -1;
    for (int block = split; block - split < a.blocks;) {
      if (ok && !warp_wait(full + 8 * slot, parity, abort_ptr, limit)) {
        if (lane == 0) give_up(kErrWaitFull);
        ok = false;
      }
#pragma unroll 1
      for (int k = 0; k < a.depth; ++k, block += a.splits) {
        if (!ok || block >= a.blocks) continue;  // the tiles are walked to the end: the warps meet at barriers
        if (block * kPer / 4 != word) {
          word = block * kPer / 4;
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) scales[j][h] = ahead[j][h];
          // the warp's next block whose scales are in another word
          const int after = a.splits * kPer >= 4 ? block + a.splits : (word + 1) * (4 / kPer) + split;
          if (after < a.blocks) {
            load_scales(after * kPer / 4, ahead);
          } else if (more) {
            scales_of(next);
            load_scales(split * kPer / 4, ahead);
          }
        }
        const uint32_t w = w_lane + slot_at + k * (kWarps * kWeightBlock), x = slot_at + k * a.splits * kXBlock;
        const int first_byte = kPer == 4 ? 0 : 8 * (block * kPer & 3);
        uint4 rows[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (NT == 1 || n < row_groups) rows[n][c] = ld_shared_v4(x_unit[c & 1] + x + (c >> 1) * (kXBlock / 2) + n * 1024);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint4 wl = ld_shared_v4(w + j * (GATED ? 512 : 1024)), wh = ld_shared_v4(w + w_half + j * (GATED ? 512 : 1024));
          float sum[NT][4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {  // 32 columns
            uint32_t l[4], h[4];
            int4x8_to_bf16(c == 0 ? wl.x : c == 1 ? wl.y : c == 2 ? wl.z : wl.w, factors, l);
            int4x8_to_bf16(c == 0 ? wh.x : c == 1 ? wh.y : c == 2 ? wh.z : wh.w, factors, h);
            const uint32_t a0[4] = {l[0], h[0], l[1], h[1]}, a1[4] = {l[2], h[2], l[3], h[3]};
            const bool last = (32 * c + 32) % GROUP == 0;  // of a group
            const int shift = first_byte + 8 * (32 * c / GROUP);
            const float sl = e4m3_value(scales[j][0] >> shift), sh = e4m3_value(scales[j][1] >> shift);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              if (NT > 1 && n >= row_groups) continue;
              if (32 * c % GROUP == 0) mma_16x8x16_first(sum[n], a0, rows[n][c].x, rows[n][c].y);
              else mma_16x8x16(sum[n], a0, rows[n][c].x, rows[n][c].y);
              mma_16x8x16(sum[n], a1, rows[n][c].z, rows[n][c].w);
              if (last) {
                acc[j][n][0] += sl * sum[n][0];
                acc[j][n][1] += sl * sum[n][1];
                acc[j][n][2] += sh * sum[n][2];
                acc[j][n][3] += sh * sum[n][3];
              }
            }
          }
        }
      }
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(empty + 8 * slot);  // its products have taken what the loads brought
      slot_at += stage_bytes;
      if (++slot == a.stages) {
        slot = 0;
        slot_at = 0;
        parity ^= 1u;
      }
    }
    if (word < 0 && more) {  // no block for this warp
      scales_of(next);
      load_scales(split * kPer / 4, ahead);
    }
    float cs[2][2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        cs[j][h] = q.n0 + (GATED ? channel0[j][0] : channel0[j][h]) < a.N
                       ? kUnscaled * __ldg(a.channel_scale + (int64_t)q.e * channels + q.n0 + channel0[j][h])
                       : 0.0f;
    // Eight rows at a time: the warps' sums to shared memory, those along the reduction added in their order, whole lines
    // of 16 bytes to the result.
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (n >= row_groups) break;
      float* to = s_red + warp * 8 * kPadded;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        to[t * kPadded + 16 * j + g] = acc[j][n][0] * cs[j][0];
        to[(t + 4) * kPadded + 16 * j + g] = acc[j][n][1] * cs[j][0];
        to[t * kPadded + 16 * j + 8 + g] = acc[j][n][2] * cs[j][1];
        to[(t + 4) * kPadded + 16 * j + 8 + g] = acc[j][n][3] * cs[j][1];
      }
      if (a.splits > 1) asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory");
      else __syncwarp();
      const int r = lane >> 2, part = lane & 3;
      const int row = 8 * n + r, column = q.n0 + (GATED ? 16 : kWarpTile) * mine + 8 * part;
      if (split == 0 && ok && row < q.rows && column < a.N && (!GATED || part < 2)) {
        float v[8], u[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] = u[c] = 0.0f;
        for (int k = 0; k < a.splits; ++k) {
          const float* from = to + k * 8 * kPadded + r * kPadded + (GATED ? 16 : 8) * part;
          const float4 v0 = *reinterpret_cast<const float4*>(from), v1 = *reinterpret_cast<const float4*>(from + 4);
          v[0] += v0.x; v[1] += v0.y; v[2] += v0.z; v[3] += v0.w;
          v[4] += v1.x; v[5] += v1.y; v[6] += v1.z; v[7] += v1.w;
          if (GATED) {
            const float4 u0 = *reinterpret_cast<const float4*>(from + 8), u1 = *reinterpret_cast<const float4*>(from + 12);
            u[0] += u0.x; u[1] += u0.y; u[2] += u0.z; u[3] += u0.w;
            u[4] += u1.x; u[5] += u1.y; u[6] += u1.z; u[7] += u1.w;
          }
        }
        if (GATED) {
#pragma unroll
          for (int c = 0; c < 8; ++c) v[c] = silu_times(v[c], u[c]);
        }
        st_v4(a.out + (int64_t)(q.r0 + row) * a.N + column,
              make_uint4(bf16x2_pz(v[0], v[1]), bf16x2_pz(v[2], v[3]), bf16x2_pz(v[4], v[5]), bf16x2_pz(v[6], v[7])));
      }
      if (a.splits > 1) asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory");
      else __syncwarp();
    }
    q = next;
  }
}

// ---- host --------------------------------------------------------------------------------------------------------------

constexpr int kFewRows = 8;

// Rows of a tile: all of them where one expert has few, else twice an expert's average share, so that an uneven batch still
// has one row tile for most experts.
int64_t rows_wanted(int64_t R, int E) { return E == 1 ? R : 2 * ((R + E - 1) / E); }

// Warps along the reduction: as few as leave every thread block at least three tiles.
int splits_of(int64_t R, int E, int N, int blocks, bool gated, int rows, int grid) {
  const int64_t row_tiles = E == 1 ? (R + rows - 1) / rows : R < E ? R : E;
  for (int splits = 1; splits < kWarps; splits *= 2) {
    const int per_tile = (gated ? 16 : kWarpTile) * (kWarps / splits);
    if (2 * splits > blocks || row_tiles * ((N + per_tile - 1) / per_tile) >= 3 * (int64_t)grid) return splits;
  }
  return kWarps;
}

}  // namespace

ProductI4Plan product_i4_plan(int64_t R, int E, int N, int D, bool gated, int sms) {
  ProductI4Plan p;
  const int64_t want = rows_wanted(R, E);
  p.tiles = want > kFewRows;
  p.wide = false;
  if (p.tiles) {
    p.rows = want <= 16 ? 16 : want <= 32 ? 32 : want <= 64 ? 64 : 128;
    const int64_t row_tiles = E == 1 ? (R + 127) / 128 : R / 128 + (R < E ? R : E);
    p.wide = want > 128 && row_tiles * ((N + 255) / 256) * (gated ? 2 : 1) >= sms;
    p.splits = 0;
    p.box_channels = (gated ? 64 : 128) * (p.wide ? 2 : 1);
    p.box_rows = p.rows < 64 ? p.rows : 64;
    p.box_chunks = D % 64 ? 0 : p.rows > 64 ? 1 : 4;
  } else {
    p.rows = want <= 8 ? 8 : want <= 16 ? 16 : 32;
    p.splits = splits_of(R, E, N, (D + 127) / 128, gated, p.rows, blocks_per_sm(p.rows / 8) * sms);
    p.box_channels = (gated ? 16 : kWarpTile) * (kWarps / p.splits);
    p.box_rows = p.rows;
    p.box_chunks = 0;
  }
  return p;
}

namespace {

template <int NT, int GROUP, bool GATED>
cudaError_t launch_few(const ProductI4Args& p, const ProductI4Plan& plan, const CUtensorMap& map_w, const CUtensorMap& map_x,
                       int sms, cudaStream_t stream) {
  constexpr int kBlocks = blocks_per_sm(NT), kLimit = (kBlocks > 1 ? 113 : 226) * 1024;
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
  a.splits = plan.splits;
  a.depth = plan.splits == 1 ? 2 : 1;
  a.stage_wait_ns = stage_wait_limit_ns();
  const int stage = a.depth * (kWarps * kWeightBlock + plan.splits * 8 * NT * 256);
  const int fixed = 1024 + kWarps * 8 * kPadded * 4 + 16 * 8 + 16 + 4 * (3 * p.E + 1);
  a.stages = (kLimit - fixed) / stage;
  if (a.stages > 8) a.stages = 8;
  auto kernel = product_i4_kernel<NT, GROUP, GATED>;
  cudaError_t e = ensure_smem_limit((const void*)kernel, kLimit);
  if (e != cudaSuccess) return e;
  // no more thread blocks than there can be tiles
  const int64_t row_tiles = p.E == 1 ? (p.R + 8 * NT - 1) / (8 * NT) : p.R / (8 * NT) + (p.R < p.E ? p.R : p.E);
  const int64_t most = row_tiles * ((p.N + plan.box_channels - 1) / plan.box_channels);
  const int grid = most < kBlocks * sms ? (int)most : kBlocks * sms;
  return launch_pdl(kernel, dim3(grid), dim3(kThreads), (size_t)fixed + (size_t)a.stages * stage, stream, map_w, map_x, a);
}

template <int GROUP, bool GATED>
cudaError_t launch_rows(const ProductI4Args& p, const ProductI4Plan& plan, const CUtensorMap& map_w, const CUtensorMap& map_x,
                        int sms, cudaStream_t stream) {
  switch (plan.rows) {
    case 8: return launch_few<1, GROUP, GATED>(p, plan, map_w, map_x, sms, stream);
    case 16: return launch_few<2, GROUP, GATED>(p, plan, map_w, map_x, sms, stream);
    default: return launch_few<4, GROUP, GATED>(p, plan, map_w, map_x, sms, stream);
  }
}

}  // namespace

cudaError_t launch_product_i4(const ProductI4Args& p, const ProductI4Plan& plan, const CUtensorMap& map_w,
                              const CUtensorMap& map_x, int sms, cudaStream_t stream) {
  if (plan.tiles) return launch_product_i4_tiles(p, plan, map_w, map_x, sms, stream);
  if (p.gated)
    return p.group == 32   ? launch_rows<32, true>(p, plan, map_w, map_x, sms, stream)
           : p.group == 64 ? launch_rows<64, true>(p, plan, map_w, map_x, sms, stream)
                           : launch_rows<128, true>(p, plan, map_w, map_x, sms, stream);
  return p.group == 32   ? launch_rows<32, false>(p, plan, map_w, map_x, sms, stream)
         : p.group == 64 ? launch_rows<64, false>(p, plan, map_w, map_x, sms, stream)
                         : launch_rows<128, false>(p, plan, map_w, map_x, sms, stream);
}

cudaError_t take_product_i4_error(unsigned* bits) {
  unsigned v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_i4_error, sizeof v);
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_i4_error, &zero, sizeof zero);
  *bits = v;
  return e;
}

}  // namespace moetail
