// What the kernels of the 4-bit products share (sm_103a).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "product.cuh"

namespace moetail {

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z, int u,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(u), "r"(bar), "l"(policy)
      : "memory");
}

// ---- 4 bits to BF16 ------------------------------------------------------------------------------------------------
//
// The whole numbers 0 .. 255 in the low byte of a BF16 are the numbers n * 2^-133: below the smallest normal number and in
// the first binade above it the format is linear.  So nibbles need no exponent put in front of them: one mask takes the
// nibble n in bits 0 .. 3 of both halves of a word as n * 2^-133, another the one in bits 4 .. 7 as n * 2^-129, and a
// multiply-add brings either into range, subtracts 8 and multiplies by a scale.  Its result has at most seven significant
// bits and is exact.  Five integer operations (of which an SM does half as many as of the others) and four multiply-adds for
// eight weights; with an exponent put in front it were seven and four.
struct Factors {
  __nv_bfloat162 low, high, term;  // for the two nibbles of a byte, and what is added
  __device__ static __nv_bfloat162 both(uint16_t bits) { return __bfloat162bfloat162(__ushort_as_bfloat16(bits)); }
};

// Both kernels keep their sums as multiples of 2^-15, so that a row has the same range in either.
constexpr float kScaled = 32768.0f;
// For q * 2^-15: 2^118, 2^114 and -8 * 2^-15.
__device__ __forceinline__ Factors unscaled() { return Factors{Factors::both(0x7a80), Factors::both(0x7880), Factors::both(0xb980)}; }

__device__ __forceinline__ float e4m3_value(uint32_t byte) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)(byte & 0xffu), __NV_E4M3)));
}

// For q * gs * 2^-15: gs * 2^118, gs * 2^114 and -8 gs * 2^-15 (gs has four significant bits and is below 2^9).
__device__ __forceinline__ Factors scaled(uint32_t e4m3) {
  const float gs = e4m3_value(e4m3);
  const __nv_bfloat162 v = __floats2bfloat162_rn(gs, gs);
  return Factors{__hmul2(v, Factors::both(0x7a80)), __hmul2(v, Factors::both(0x7880)), __hmul2(v, Factors::both(0xb980))};
}

// Columns c = 0 .. 7 of a stored word as four pairs.
__device__ __forceinline__ void int4x8_to_bf16(uint32_t word, const Factors& f, uint32_t* pair) {
  const uint32_t upper = word >> 8;
  const uint32_t n[4] = {word & 0x000f000fu, word & 0x00f000f0u, upper & 0x000f000fu, upper & 0x00f000f0u};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 v = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&n[i]), i & 1 ? f.high : f.low, f.term);
    pair[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
}

// silu(g) * up.  With e = exp(-|g| / 2) the divisor is 1 + e^2; for g < 0 the fraction is multiplied by e^2 above and
// below, one e with each factor, so that nothing leaves FP32's range before the result does.  The exponent of two, rounded to
// FP32, and what the rounding left of it, which multiplies the power of two by 1 + (rest) ln 2: one rounded exponent would be
// off by up to |g| units.  Powers below FP32's normal numbers are kept: a large up brings the result back into range down to
// gates of -180.
__device__ __forceinline__ float silu_times(float g, float up) {
  constexpr float kHalfLog2e = 0.72134752f, kBeyond = (float)(0.72134752044448170368 - (double)0.72134752f);
  constexpr float kLn2 = 0.69314718f;
  const float m = fminf(fabsf(g), 512.0f), t = -kHalfLog2e * m;  // from 208 on the power is zero
  const float rest = fmaf(-kBeyond, m, fmaf(-kHalfLog2e, m, -t));
  float e, r;
  asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(t));
  e = fmaf(e, rest * kLn2, e);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fmaf(e, e, 1.0f)));
  const float p = g < 0.0f ? e : 1.0f;
  return ((g * p) * (up * p)) * r;
}

}  // namespace moetail
