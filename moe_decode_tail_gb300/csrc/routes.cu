// Routes sorted by expert, rows copied into that order and back with weights, and the gradients (sm_103a).
//
//   sort      a stable counting sort of the routes r = t * K + k by expert id
//   dispatch  rows[idx[t][k]] = x[t]
//   combine   out[t] = bf16(sum over k, in order, of w[t][k] * rows[idx[t][k]])      (FP32 from +0)
//   gradient  d_rows[idx[t][k]] = bf16(w[t][k] * d_out[t]),  d_w[t][k] = sum(d_out[t] * rows[idx[t][k]])
//
// A route has a row iff 0 <= idx < num_rows; a route without one is skipped, whatever its weight.
//
// The row kernels are bound by memory.  Each reads and writes a row once: dispatch reads a token's row once for all
// its routes (8192 tokens x 8 routes x 4096 BF16: 89 us, 6.8 TB/s), combine keeps eight route rows of a column in
// flight (8191 tokens x 16 routes, half of them with a row, x 3584: 83 us, 6.4 TB/s), the gradient keeps d_out's row
// in registers and the next route's row in flight (4096 x 8 x 4096: 95 us, 6.0 TB/s).  The sort of a decode step is
// one small kernel (512 routes: 4.5 us); 65536 routes take two, 8 us.
#include "common.cuh"
#include "kernels.h"
#include "layer.h"

namespace moetail {

namespace {

constexpr int kSortThreads = 1024, kSortWarps = 32;

// Routes of each expert in every chunk of PER * 1024 routes.
template <int PER>
__global__ void __launch_bounds__(kSortThreads) count_routes_kernel(const SortArgs a) {
  extern __shared__ int32_t s_count[];
  for (int e = threadIdx.x; e < a.E; e += kSortThreads) s_count[e] = 0;
  grid_dependency_wait();
  launch_dependents();
  __syncthreads();
  const int r0 = blockIdx.x * PER * kSortThreads;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int r = r0 + j * kSortThreads + threadIdx.x;
    const int e = r < a.routes ? a.ids[r] : -1;
    if (e >= 0 && e < a.E) atomicAdd(&s_count[e], 1);  // whole numbers: the order does not matter
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += kSortThreads) a.counts[(int64_t)blockIdx.x * a.E + e] = s_count[e];
}

// Exclusive sum over the 1024 threads; *all: the total.
__device__ __forceinline__ int block_exclusive_sum(int v, int* all) {
  __shared__ int s_warp[kSortWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int sum = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, sum, off);
    if (lane >= off) sum += o;
  }
  if (lane == 31) s_warp[warp] = sum;
  __syncthreads();
  int w = s_warp[lane];
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, w, off);
    if (lane >= off) w += o;
  }
  *all = __shfl_sync(0xffffffffu, w, 31);
  const int before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
  __syncthreads();
  return sum - v + (warp > 0 ? before : 0);
}

// The lanes of the warp with this lane's value, by its bits: a ballot each (a match of 32 mostly different values
// takes longer).
__device__ __forceinline__ unsigned lanes_with(int value, int bits) {
  unsigned same = 0xffffffffu;
  for (int i = 0; i < bits; ++i) {
    const bool one = (value >> i) & 1;
    const unsigned ones = __ballot_sync(0xffffffffu, one);
    same &= one ? ones : ~ones;
  }
  return same;
}

// Places of a chunk's routes.  A warp takes 32 * PER consecutive routes, 32 at a time, so the order
// within an expert is: earlier chunks, earlier warps, earlier rounds, lower lanes.
template <int PER>
__global__ void __launch_bounds__(kSortThreads) place_routes_kernel(const SortArgs a) {
  // [warps][E] counts, then the routes of the warps before; [E] first place; [E], [E] routes of all chunks, of those
  // before this one
  extern __shared__ int32_t s_mem[];
  int32_t *s_first = s_mem + kSortWarps * a.E, *s_total = s_first + a.E, *s_before = s_total + a.E;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < (kSortWarps + 3) * a.E; i += kSortThreads) s_mem[i] = 0;
  grid_dependency_wait();
  launch_dependents();
  __syncthreads();
  const int r0 = (blockIdx.x * kSortThreads + warp * 32) * PER + lane;
  int32_t* mine = s_mem + warp * a.E;
  const int id_bits = 32 - __clz(a.E);
  int id[PER], rank[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int r = r0 + 32 * j;
    id[j] = r < a.routes ? a.ids[r] : -1;
    if (id[j] >= a.E) id[j] = -1;
  }
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const unsigned same = lanes_with(id[j] < 0 ? a.E : id[j], id_bits);
    const unsigned below = same & ((1u << lane) - 1u);
    rank[j] = 0;
    if (id[j] >= 0) rank[j] = mine[id[j]] + __popc(below);
    __syncwarp();
    if (id[j] >= 0 && below == 0) mine[id[j]] += __popc(same);
    __syncwarp();
  }
  if (gridDim.x > 1) {  // every thread takes an expert's counts of some chunks
    const int groups = kSortThreads / a.E, e = threadIdx.x % a.E, g = threadIdx.x / a.E;
    if (g < groups) {
      int total = 0, before = 0;
#pragma unroll 4
      for (int c = g; c < (int)gridDim.x; c += groups) {
        const int n = a.counts[(int64_t)c * a.E + e];
        if (c < (int)blockIdx.x) before += n;
        total += n;
      }
      atomicAdd(&s_total[e], total);  // whole numbers: the order does not matter
      atomicAdd(&s_before[e], before);
    }
  }
  __syncthreads();
  const int e = threadIdx.x;  // E <= 1024
  int total = 0, before = 0;
  if (e < a.E) {
#pragma unroll 8
    for (int w = 0; w < kSortWarps; ++w) {
      const int n = s_mem[w * a.E + e];
      s_mem[w * a.E + e] = total;
      total += n;
    }
    if (gridDim.x > 1) {
      total = s_total[e];
      before = s_before[e];
    }
  }
  int all;
  const int first = block_exclusive_sum(total, &all);
  if (e < a.E) {
    s_first[e] = first + before;
    if (blockIdx.x == 0) a.offsets[e] = first;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) a.offsets[a.E] = all;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int r = r0 + 32 * j;
    if (r >= a.routes) continue;
    int place = -1;
    if (id[j] >= 0) {
      place = s_first[id[j]] + mine[id[j]] + rank[j];
      a.source[place] = r;
    }
    a.permuted_idx[r] = place;
    if (r >= all) a.source[r] = -1;  // places past the last row
  }
}

// ---- rows ---------------------------------------------------------------------------

// V: 16 or 8 bytes.  A thread copies one vector of a token's row to the places of all its routes.
template <typename V>
__global__ void __launch_bounds__(256) dispatch_rows_kernel(const DispatchArgs a) {
  grid_dependency_wait();
  launch_dependents();
  const int64_t t = blockIdx.x;
  const int nv = a.row_bytes / (int)sizeof(V), lane = threadIdx.x & 31;
  const int v = blockIdx.y * blockDim.x + threadIdx.x;
  // lane k keeps route k's row, -1 without one
  int mine = lane < a.K ? a.idx[t * a.K + lane] : -1;
  if (mine >= a.num_rows) mine = -1;
  V d = {};
  if (v < nv) d = static_cast<const V*>(a.x)[t * nv + v];
  for (int k = 0; k < a.K; ++k) {
    const int64_t j = __shfl_sync(0xffffffffu, mine, k);
    if (j >= 0 && v < nv) static_cast<V*>(a.rows)[j * nv + v] = d;
  }
  if (a.scale && v < 32 && mine >= 0) a.row_scale[mine] = a.scale[t];
}

template <int WMODE>
__device__ __forceinline__ float route_weight(const void* w, int64_t i) {
  if (WMODE == kWeightUnit) return 1.0f;
  if (WMODE == kWeightBF16) return bf16_lo(static_cast<const uint16_t*>(w)[i]);
  return static_cast<const float*>(w)[i];
}

// A route's row (or -1) and weight, kept by the lane of its number: lane k holds route k of token t.
struct Route {
  int row;
  float w;
};
template <int WMODE>
__device__ __forceinline__ Route route_of_lane(const CombineArgs& a, int64_t t) {
  const int lane = threadIdx.x & 31;
  Route r = {-1, 0.0f};
  if (lane < a.K) {
    r.row = a.idx[t * a.K + lane];
    r.w = route_weight<WMODE>(a.w, t * a.K + lane);
    if (r.row >= a.num_rows) r.row = -1;
  }
  return r;
}

constexpr int kRoutesAtOnce = 8;  // rows in flight of a thread
constexpr int kCombineThreads = 64;

template <int WMODE>
__global__ void __launch_bounds__(kCombineThreads) combine_rows_kernel(const CombineArgs a) {
  grid_dependency_wait();
  launch_dependents();
  const int64_t t = blockIdx.x;
  const int nv = a.H >> 3;
  const int v = blockIdx.y * blockDim.x + threadIdx.x;
  const Route mine = route_of_lane<WMODE>(a, t);
  float acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
  unsigned left = __ballot_sync(0xffffffffu, mine.row >= 0);  // routes with a row, in order
  while (left) {
    uint4 d[kRoutesAtOnce];
    float w[kRoutesAtOnce];
#pragma unroll
    for (int i = 0; i < kRoutesAtOnce; ++i) {
      const int k = left ? __ffs(left) - 1 : 0;
      const int j = __shfl_sync(0xffffffffu, mine.row, k);
      w[i] = __shfl_sync(0xffffffffu, mine.w, k);
      d[i] = make_uint4(0, 0, 0, 0);
      if (left == 0) w[i] = 0.0f;  // no route: zeros times zero
      else if (v < nv) d[i] = ld_stream_v4(a.rows + (int64_t)j * a.H + 8 * v);
      left &= left - 1;
    }
#pragma unroll
    for (int i = 0; i < kRoutesAtOnce; ++i) {
      float f[8];
      unpack8(d[i], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] += w[i] * f[e];
    }
  }
  if (v < nv)
    st_v4(a.out + t * a.H + 8 * v, make_uint4(bf16x2_pz(acc[0], acc[1]), bf16x2_pz(acc[2], acc[3]), bf16x2_pz(acc[4], acc[5]),
                                              bf16x2_pz(acc[6], acc[7])));
}

// A block per token: d_out's row stays in registers while the routes' rows pass, the next route's loads in flight.
template <int WMODE, int VPT>
__global__ void __launch_bounds__(1024) combine_grad_kernel(const CombineArgs a) {
  __shared__ float s_dot[kMaxK][32];
  grid_dependency_wait();
  launch_dependents();
  const int64_t t = blockIdx.x;
  const int nv = a.H >> 3, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Route mine = route_of_lane<WMODE>(a, t);
  uint4 d[VPT], next[VPT];
  auto load = [&](int j) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (j >= 0 && v < nv) next[i] = ld_stream_v4(a.rows + (int64_t)j * a.H + 8 * v);
    }
  };
  int j = __shfl_sync(0xffffffffu, mine.row, 0);
  load(j);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    if (v < nv) d[i] = ld_stream_v4(a.d_out + t * a.H + 8 * v);
  }
  for (int k = 0; k < a.K; ++k) {
    uint4 row[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) row[i] = next[i];
    const int here = j;
    const float w = __shfl_sync(0xffffffffu, mine.w, k);
    if (k + 1 < a.K) {
      j = __shfl_sync(0xffffffffu, mine.row, k + 1);
      load(j);
    }
    float dot = 0.0f;
    if (here >= 0) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v >= nv) continue;
        float f[8], g[8];
        unpack8(row[i], f);
        unpack8(d[i], g);
#pragma unroll
        for (int e = 0; e < 8; ++e) dot += f[e] * g[e];
        st_v4(a.d_rows + (int64_t)here * a.H + 8 * v,
              make_uint4(bf16x2_pz(w * g[0], w * g[1]), bf16x2_pz(w * g[2], w * g[3]), bf16x2_pz(w * g[4], w * g[5]),
                         bf16x2_pz(w * g[6], w * g[7])));
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
    if (lane == 0) s_dot[k][warp] = dot;
  }
  __syncthreads();
  if ((int)threadIdx.x < a.K) {
    float dot = 0.0f;
    for (int w = 0; w < (int)(blockDim.x >> 5); ++w) dot += s_dot[threadIdx.x][w];
    a.d_w[t * a.K + threadIdx.x] = dot;
  }
}

}  // namespace

namespace {

template <int PER>
cudaError_t launch_sort(const SortArgs& a, cudaStream_t stream) {
  const int blocks = sort_blocks(a.routes);
  cudaError_t e = ensure_smem_limit((const void*)place_routes_kernel<PER>, (kSortWarps + 3) * kMaxExperts * 4);
  if (e != cudaSuccess) return e;
  if (blocks > 1) {
    e = launch_pdl(count_routes_kernel<PER>, dim3(blocks), dim3(kSortThreads), (size_t)a.E * 4, stream, a);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(place_routes_kernel<PER>, dim3(blocks), dim3(kSortThreads), (size_t)(kSortWarps + 3) * a.E * 4, stream,
                    a);
}

constexpr int kMostBlocks = 128;  // each thread block adds up the counts of all

// Routes of a lane: few, until there would be more blocks.
int routes_of_lane(int routes) {
  return routes <= kMostBlocks * kSortThreads ? 1 : routes <= 4 * kMostBlocks * kSortThreads ? 4 : 16;
}

}  // namespace

int sort_blocks(int routes) {
  const int chunk = kSortThreads * routes_of_lane(routes);
  return routes > chunk ? (routes + chunk - 1) / chunk : 1;
}

int sort_blocks_up_to(int routes) {
  const int64_t of_one = ((int64_t)routes + kSortThreads - 1) / kSortThreads;  // chunks of one route a lane
  return of_one < 1 ? 1 : of_one < kMostBlocks ? (int)of_one : kMostBlocks;
}

cudaError_t launch_sort_routes(const SortArgs& a, cudaStream_t stream) {
  switch (routes_of_lane(a.routes)) {
    case 1: return launch_sort<1>(a, stream);
    case 4: return launch_sort<4>(a, stream);
    default: return launch_sort<16>(a, stream);
  }
}

cudaError_t launch_dispatch_rows(const DispatchArgs& a, cudaStream_t stream) {
  const bool wide = a.row_bytes % 16 == 0;
  const int nv = a.row_bytes / (wide ? 16 : 8);
  const dim3 grid(a.b, (nv + 255) / 256);
  if (wide) return launch_pdl(dispatch_rows_kernel<uint4>, grid, dim3(256), 0, stream, a);
  return launch_pdl(dispatch_rows_kernel<uint2>, grid, dim3(256), 0, stream, a);
}

cudaError_t launch_combine_rows(const CombineArgs& a, int wmode, cudaStream_t stream) {
  const int nv = a.H >> 3;
  // Small blocks: 64 threads took 83 us where 256 took 86 (8191 tokens, 16 routes, 3584 columns), and at 64 tokens
  // they spread a row over more SMs.
  const int threads = kCombineThreads;
  const dim3 grid(a.b, (nv + threads - 1) / threads);
  if (wmode == kWeightUnit) return launch_pdl(combine_rows_kernel<kWeightUnit>, grid, dim3(threads), 0, stream, a);
  if (wmode == kWeightBF16) return launch_pdl(combine_rows_kernel<kWeightBF16>, grid, dim3(threads), 0, stream, a);
  return launch_pdl(combine_rows_kernel<kWeightF32>, grid, dim3(threads), 0, stream, a);
}

cudaError_t launch_combine_grad(const CombineArgs& a, int wmode, cudaStream_t stream) {
  const int nv = a.H >> 3;
  // Two vectors a thread: 96 us for 4096 tokens, 8 routes, 4096 columns; one or four: 103 and 104.  More only where
  // a block of 1024 threads needs them.
  const int vpt = nv <= 2048 ? 2 : 4;
  const dim3 threads(((nv + vpt - 1) / vpt + 31) / 32 * 32);
  if (wmode == kWeightBF16)
    return vpt == 2 ? launch_pdl(combine_grad_kernel<kWeightBF16, 2>, dim3(a.b), threads, 0, stream, a)
                    : launch_pdl(combine_grad_kernel<kWeightBF16, 4>, dim3(a.b), threads, 0, stream, a);
  return vpt == 2 ? launch_pdl(combine_grad_kernel<kWeightF32, 2>, dim3(a.b), threads, 0, stream, a)
                  : launch_pdl(combine_grad_kernel<kWeightF32, 4>, dim3(a.b), threads, 0, stream, a);
}

}  // namespace moetail
