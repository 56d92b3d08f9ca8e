// What the products by expert share (sm_103a): rings of slots, waits by whole warps, PTX wrappers.
#pragma once

#include "tensor_core.cuh"

namespace moetail {

// Offsets come from the device: whatever they hold, no row outside [0, R) is touched.
__device__ __forceinline__ int clamp_row(int r, int64_t rows) { return r < 0 ? 0 : r > rows ? (int)rows : r; }

// Brings the warp's lanes together: before instructions that all of them have to execute at once (".aligned"), which
// the compiler does not know of inside inline assembly and might place in the branches before them.
__device__ __forceinline__ void together() { __syncwarp(); }

// D[tmem_d] (+)= A[tmem_a] * B[bdesc], operands of idesc's type, FP32 sums.
__device__ __forceinline__ void mma_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
      "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
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
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar), "l"(policy)
      : "memory");
}

__device__ __forceinline__ void st_shared_u16(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"((uint16_t)v) : "memory");
}
__device__ __forceinline__ void st_shared_f32(uint32_t addr, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
// A barrier over the four warps of an epilogue set.
__device__ __forceinline__ void set_bar(int set) {
  together();
  asm volatile("bar.sync %0, 128;" ::"r"(2 + set) : "memory");
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

// first[e]: row tiles of `rows` rows of the experts before e, first[E]: of all.  By one warp; counts and first in shared memory.
__device__ __forceinline__ void row_tiles_before(const int32_t* count, int32_t* first, int E, int rows) {
  const int lane = threadIdx.x & 31;
  int before = 0;
  for (int e0 = 0; e0 < E; e0 += 32) {
    const int e = e0 + lane;
    const int tiles = e < E ? (count[e] + rows - 1) / rows : 0;
    int sum = tiles;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, sum, off);
      if (lane >= off) sum += o;
    }
    if (e < E) first[e] = before + sum - tiles;
    before += __shfl_sync(0xffffffffu, sum, 31);
  }
  if (lane == 0) first[E] = before;
}

// The expert of a tile, with `across` channel tiles for each row tile: the last whose tiles start at or before it.
__device__ __forceinline__ int expert_of_tile(const int32_t* first, int E, int across, int64_t tile) {
  int lo = 0, hi = E - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((int64_t)first[mid] * across <= tile) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

}  // namespace moetail
