// Helpers of the kernels that hold a row of columns in a thread block's registers (sm_103a).
#pragma once

#include "common.cuh"

namespace moetail {

// The larger magnitude; a NaN stays one, so that a group's result tells whether all of it was finite.
__device__ __forceinline__ float larger(float top, float v) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(top), "f"(fabsf(v)));
  return m;
}
// The same of two results: as whole numbers, infinities are above every finite value and NaNs above them.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

__device__ __forceinline__ uint32_t max8(const float (&y)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = larger(m, y[i]);
  return magnitude(m);
}

// Rows that the kernel may write in place: through L1 they would not be coherent, so no read-only loads.
__device__ __forceinline__ uint4 ld_rows(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// Sum and maximum over the thread block, in a fixed order, known to every thread; a barrier between two calls of one ID.
struct RowSums {
  float sum;
  uint32_t top;
};
template <int ID = 0>
__device__ __forceinline__ RowSums block_reduce(float sum, uint32_t top) {
  __shared__ float s_sum[32];
  __shared__ uint32_t s_top[32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  top = __reduce_max_sync(0xffffffffu, top);
  if (warps > 1) {
    if (lane == 0) {
      s_sum[warp] = sum;
      s_top[warp] = top;
    }
    __syncthreads();
    sum = lane < warps ? s_sum[lane] : 0.0f;
    top = lane < warps ? s_top[lane] : 0u;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    top = __reduce_max_sync(0xffffffffu, top);
  }
  return RowSums{sum, top};
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(pair_bits(a)), "l"(pair_bits(b)), "l"(pair_bits(c)));
  return pair_of(d);
}

// Eight values in BF16, -0 made +0.
__device__ __forceinline__ uint4 pack8_pz(const float (&v)[8]) {
  return make_uint4(bf16x2_pz(v[0], v[1]), bf16x2_pz(v[2], v[3]), bf16x2_pz(v[4], v[5]), bf16x2_pz(v[6], v[7]));
}

// A row's vectors over the threads of a block: VPT vectors each, whole warps.
inline int threads_for(int nv, int vpt) { return ((nv + vpt - 1) / vpt + 31) / 32 * 32; }

// Vectors a thread: one where the rows are fewer than the SMs can take at once (a row's latency counts), else `many`,
// more where the row does not fit a block otherwise.
inline int vectors_for(int nv, int64_t rows, int sms, int many) {
  if (rows <= 2 * sms && nv <= 1024) return 1;
  int vpt = many;
  while (threads_for(nv, vpt) > 512) vpt *= 2;
  return vpt;
}

}  // namespace moetail
