// Product of 8-bit integers with a scale for each row and each channel, by expert (sm_103a).
//
//   out[r][n] = bf16((sum over k of x[r][k] * w[e][n][k]) * w_scale[e][n] * x_scale[r]),
//   r in [offsets[e], offsets[e + 1])
#include "common.cuh"
#include "layer.h"

namespace moetail {

namespace {

// Offsets come from the device: whatever they hold, no row outside [0, R) is touched.
__device__ __forceinline__ int clamp_row(int r, int64_t rows) { return r < 0 ? 0 : r > rows ? (int)rows : r; }

constexpr int kTileN = 64, kTileR = 32, kTileD = 64;

__global__ void __launch_bounds__(256) expert_product_kernel(const ProductArgs a) {
  __shared__ int s_w[kTileN][kTileD / 4 + 1], s_x[kTileR][kTileD / 4 + 1];
  __shared__ int s_tile[2];
  grid_dependency_wait();
  launch_dependents();
  // the block's tile: row tiles are counted expert by expert
  if (threadIdx.x == 0) {
    int left = blockIdx.x, e = -1, first = 0;
    if (!a.offsets) {
      e = 0;
      first = left * kTileR;
    } else {
      for (int i = 0; i < a.E; ++i) {
        const int begin = clamp_row(a.offsets[i], a.R), end = clamp_row(a.offsets[i + 1], a.R);
        const int tiles = end > begin ? (end - begin + kTileR - 1) / kTileR : 0;
        if (left < tiles) {
          e = i;
          first = begin + left * kTileR;
          break;
        }
        left -= tiles;
      }
    }
    s_tile[0] = e;
    s_tile[1] = first;
  }
  __syncthreads();
  const int e = s_tile[0];
  if (e < 0) return;
  const int64_t first = s_tile[1], end = a.offsets ? clamp_row(a.offsets[e + 1], a.R) : a.R;
  const int n0 = blockIdx.y * kTileN;
  const int tn = threadIdx.x & 31, tr = threadIdx.x >> 5;  // 2 channels x 4 rows a thread
  int acc[4][2] = {};
  for (int k0 = 0; k0 < a.D; k0 += kTileD) {
    for (int i = threadIdx.x; i < (kTileN + kTileR) * (kTileD / 16); i += 256) {
      const int row = i / (kTileD / 16), c = i % (kTileD / 16), k = k0 + 16 * c;
      int4 v = make_int4(0, 0, 0, 0);
      if (row < kTileN) {
        if (n0 + row < a.N && k < a.D)
          v = *reinterpret_cast<const int4*>(a.w + ((int64_t)e * a.N + n0 + row) * a.D + k);
      } else if (first + row - kTileN < end && k < a.D) {
        v = *reinterpret_cast<const int4*>(a.x + (first + row - kTileN) * a.D + k);
      }
      int* dst = row < kTileN ? &s_w[row][4 * c] : &s_x[row - kTileN][4 * c];
      dst[0] = v.x;
      dst[1] = v.y;
      dst[2] = v.z;
      dst[3] = v.w;
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < kTileD / 4; ++c) {
      const int w0 = s_w[tn][c], w1 = s_w[tn + 32][c];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int x = s_x[tr + 8 * i][c];
        acc[i][0] = __dp4a(w0, x, acc[i][0]);
        acc[i][1] = __dp4a(w1, x, acc[i][1]);
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = first + tr + 8 * i;
    if (r >= end) continue;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int n = n0 + tn + 32 * j;
      if (n < a.N)
        a.out[r * a.N + n] =
            (uint16_t)bf16_bits_pz((float)acc[i][j] * a.w_scale[(int64_t)e * a.N + n] * a.x_scale[r]);
    }
  }
}

}  // namespace

size_t expert_product_workspace(int64_t, int, int, int) { return 256; }

cudaError_t launch_expert_product(const ProductArgs& a, void*, int, cudaStream_t stream) {
  // row tiles: the full ones, and at most one more for every expert with a row
  const int64_t tiles = a.R / kTileR + (a.offsets ? (a.E < a.R ? a.E : a.R) : 1);
  return launch_pdl(expert_product_kernel, dim3((unsigned)tiles, (a.N + kTileN - 1) / kTileN), dim3(256), 0, stream, a);
}

}  // namespace moetail
