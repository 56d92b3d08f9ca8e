// Rows in 8 bits with scales: residual addition + RMS norm, and silu(gate) * up (sm_103a).
//
//   norm_quant   h = x + residual (FP32); residual_out = bf16(h);
//                y = (h * inv) * (gamma + gain_center), inv = 1 / sqrt(sum(h^2) * (1/H) + eps)
//   silu_quant   y = (gate / (1 + exp(-gate))) * up
//   both         per group (a whole row, or 128 columns): scale = max|y| / M, q = round(y * (M / max|y|)),
//                M = 127 (int8) or 448 (e4m3), to nearest even; a group of zeros has scale 0 and zeros,
//                a group with a NaN or an infinity scale NaN and zeros.
//
// A thread block per row, 16-byte loads of 8 columns; the values stay in registers between the reduction and
// the rounding, so every input is read once.  The norm is bound by memory, 4 + 2 + 1 bytes a column: 16384 rows of
// 4096 in 75.5 us, 6.2 TB/s (0.92 of the measured copy rate).  silu reads and writes 4 + 1 bytes a column and is
// bound by its exponential, reciprocal and conversions as much: 28672 rows of 2048 in 55 us in int8 with a scale a
// row, 59 us, 5.0 TB/s (0.73), in e4m3 with a scale for every 128 columns.  One token of 7168 columns takes 4.5 us, a
// launch and two trips to memory.
#include <cuda_fp8.h>
#include <float.h>

#include "layer.h"
#include "rows.cuh"

namespace moetail {

namespace {

// What a group's largest magnitude gives: its scale, and the factors of the rounding.  Below 2^-100, M / top
// could overflow, so the values are lifted by 2^100 first (exact); elsewhere that factor is 1.
struct Rounding {
  float scale, lift, factor;
  bool finite;
  __device__ Rounding(uint32_t top_bits, float most) {
    const float top = __uint_as_float(top_bits);
    lift = top < 0x1p-100f ? 0x1p100f : 1.0f;
    factor = top_bits == 0 ? 0.0f : most / (top * lift);
    scale = top / most;
    finite = top_bits < 0x7f800000u;
    if (!finite) scale = __uint_as_float(0x7fffffffu);
  }
};

// Four values, at most 127 (1 + 2^-22) in magnitude after the factor, as int8: the sum with 1.5 * 2^23 rounds to the
// nearest even whole number, which stands in the low byte (one instruction, where a conversion takes several slots).
__device__ __forceinline__ uint32_t int8x4(float a, float b, float c, float d, float factor) {
  constexpr float kMagic = 12582912.0f;
  const uint32_t ia = __float_as_uint(__fmaf_rn(a, factor, kMagic)), ib = __float_as_uint(__fmaf_rn(b, factor, kMagic));
  const uint32_t ic = __float_as_uint(__fmaf_rn(c, factor, kMagic)), id = __float_as_uint(__fmaf_rn(d, factor, kMagic));
  return __byte_perm(__byte_perm(ia, ib, 0x0040), __byte_perm(ic, id, 0x0040), 0x5410);
}

// Eight values rounded to 8 bits; a group that is not finite gives zeros.
template <int KIND>
__device__ __forceinline__ uint2 round8(const float (&y)[8], const Rounding& r) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = y[i];
  if (r.lift != 1.0f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= r.lift;
  }
  uint2 q;
  if (KIND == kQuantInt8) {
    q.x = int8x4(v[0], v[1], v[2], v[3], r.factor);
    q.y = int8x4(v[4], v[5], v[6], v[7], r.factor);
  } else {
    auto pair = [&](float lo, float hi) {
      return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(lo * r.factor, hi * r.factor), __NV_SATFINITE, __NV_E4M3);
    };
    q.x = pair(v[0], v[1]) | (pair(v[2], v[3]) << 16);
    q.y = pair(v[4], v[5]) | (pair(v[6], v[7]) << 16);
  }
  return r.finite ? q : make_uint2(0, 0);
}

constexpr float most_of(int kind) { return kind == kQuantInt8 ? 127.0f : 448.0f; }

// The maximum over the 16 lanes of a 128-column group.
__device__ __forceinline__ uint32_t max_of_group(uint32_t m) {
#pragma unroll
  for (int off = 1; off < 16; off <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
  return m;
}

// The rounding of a thread's vectors and the scales: y[i] holds vector threadIdx.x + i * blockDim.x of the row,
// `top` the row's largest magnitude (one scale a row).
template <int KIND, bool GROUPED, int VPT>
__device__ __forceinline__ void store_rows(const float (&y)[VPT][8], uint32_t top, int64_t row, int nv, uint8_t* q,
                                           float* scale, int groups) {
  const Rounding whole(top, most_of(KIND));
  if (!GROUPED && threadIdx.x == 0) scale[row] = whole.scale;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    const Rounding r = GROUPED ? Rounding(max_of_group(max8(y[i])), most_of(KIND)) : whole;
    if (v < nv) {
      *reinterpret_cast<uint2*>(q + 8 * (row * nv + v)) = round8<KIND>(y[i], r);
      if (GROUPED && (v & 15) == 0) scale[row * groups + (v >> 4)] = r.scale;
    }
  }
}

// VPT: vectors of 8 columns of a thread; thread t holds vectors t, t + blockDim, ...  One reduction gives the sum
// of squares and max|h * gain|, whose product with 1/rms is max|y|.
template <int KIND, bool GROUPED, int VPT>
__global__ void __launch_bounds__(VPT == 1 ? 1024 : 512) norm_quant_kernel(const NormQuantArgs a) {
  grid_dependency_wait();
  launch_dependents();
  const int64_t row = blockIdx.x;
  const int nv = a.H >> 3;
  uint4 x[VPT], res[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    x[i] = res[i] = make_uint4(0, 0, 0, 0);
    if (v < nv) {
      x[i] = ld_rows(a.x + row * a.H + 8 * v);
      if (a.residual) res[i] = ld_rows(a.residual + row * a.H + 8 * v);
    }
  }
  float h[VPT][8], sum = 0.0f, top = 0.0f, most_gain = 0.0f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    float r[8], g[8];
    unpack8(x[i], h[i]);
    unpack8(res[i], r);
    if (!GROUPED) unpack8(v < nv ? ld_v4(a.gamma + 8 * v) : make_uint4(0, 0, 0, 0), g);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (a.residual) h[i][e] += r[e];
      sum += h[i][e] * h[i][e];
      if (!GROUPED) {
        top = larger(top, h[i][e] * (g[e] + a.gain_center));
        most_gain = fmaxf(most_gain, fabsf(g[e] + a.gain_center));
      }
    }
    if (v < nv && a.residual_out) st_v4(a.residual_out + row * a.H + 8 * v, pack8_pz(h[i]));
  }
  if (most_gain >= 0x1p64f) top = __uint_as_float(0x7fffffffu);  // a NaN: see below
  const RowSums sums = block_reduce(sum, magnitude(top));
  float mean = sums.sum * a.rcpH + a.eps;
  bool by_values = false;  // the row's maximum is to be taken of the values themselves
  // Squares or their sum beyond FP32, or so small that they lost bits (a row near 1e19 or 1e-19): once more with the row
  // brought near one by a power of two, which changes no bit and cancels in h * inv.
  if (!(mean >= 0x1p-100f && mean <= FLT_MAX)) {
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) most = larger(most, __uint_as_float(max8(h[i])));
    __syncthreads();
    most = __uint_as_float(block_reduce(0.0f, magnitude(most)).top);
    const float size = fmaxf(most, __fsqrt_rn(a.eps));
    if (most <= FLT_MAX && size > 0.0f) {  // else the row has no finite norm
      const int exponent = min(max((int)(magnitude(size) >> 23), 1), 253);
      const float unit = __uint_as_float((uint32_t)(254 - exponent) << 23);  // size * unit is in [1, 4), or below one
      sum = 0.0f;
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          h[i][e] *= unit;
          sum += h[i][e] * h[i][e];
        }
      __syncthreads();
      mean = block_reduce(sum, 0u).sum * a.rcpH + a.eps * unit * unit;
      by_values = true;
    }
  }
  const float inv = __fdiv_rn(1.0f, __fsqrt_rn(mean));
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    float g[8];
    unpack8(v < nv ? ld_v4(a.gamma + 8 * v) : make_uint4(0, 0, 0, 0), g);
#pragma unroll
    for (int e = 0; e < 8; ++e) h[i][e] = (h[i][e] * inv) * (g[e] + a.gain_center);
    if (v < nv && a.y) st_v4(a.y + row * a.H + 8 * v, pack8_pz(h[i]));
  }
  // max|h * gain| * inv is max|(h * inv) * gain| but for a few units in the last place, as long as neither product leaves
  // FP32's range nor loses bits below it: with inv in [2^-64, 2^50] and gains below 2^64 for results in these bounds.
  const float estimate = __uint_as_float(sums.top) * inv;
  uint32_t largest = magnitude(estimate);
  if (!GROUPED && (by_values || !(estimate >= 0x1p-60f && estimate <= 0x1p126f))) {
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) most = max(most, max8(h[i]));
    __syncthreads();
    largest = block_reduce(0.0f, most).top;
  }
  store_rows<KIND, GROUPED, VPT>(h, largest, row, nv, a.q, a.scale, a.groups);
}

// silu(g) * up = g * up / (1 + exp(-g)) for two columns, within 10 units in the last place.  With e = exp(-|g| / 2): for
// g >= 0 the divisor is 1 + e^2; for g < 0 the fraction is multiplied by e^2 above and below, one e with each factor, so
// that nothing leaves FP32's range before the result does.
// The exponential: a BF16 |g| times the upper 16 bits of log2(e) / 2 is exact (t), and what that leaves of the exponent,
// at most 175 * 3.6e-6, multiplies the power of two by 1 + (rest) ln 2; zero from |g| = 175 on.  One exponent rounded to
// FP32 would be off by up to |g| units.
__device__ __forceinline__ float2 silu_times(float2 g, float2 up) {
  constexpr double kHalfLog2e = 0.72134752044448170368, kLn2 = 0.69314718055994530942;
  constexpr float kUpper = 47274.0f / 65536.0f;
  constexpr float kRest = (float)((kHalfLog2e / kUpper - 1.0) * kLn2);  // of t
  const float2 t = make_float2(-kUpper * fabsf(g.x), -kUpper * fabsf(g.y));
  float2 e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
  e = fma2(e, mul2(t, splat2(kRest)), e);
  const float2 divisor = fma2(e, e, splat2(1.0f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(divisor.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(divisor.y));
  const float2 p = make_float2(g.x < 0.0f ? e.x : 1.0f, g.y < 0.0f ? e.y : 1.0f);
  return mul2(mul2(mul2(g, p), mul2(up, p)), r);
}

template <int KIND, bool GROUPED, int VPT>
__global__ void __launch_bounds__(VPT == 1 ? 1024 : 512) silu_quant_kernel(const SiluQuantArgs a) {
  grid_dependency_wait();
  launch_dependents();
  const int64_t row = blockIdx.x;
  if (a.used && row >= *a.used) return;
  const int nv = a.I >> 3;
  uint4 gate[VPT], up[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    gate[i] = up[i] = make_uint4(0, 0, 0, 0);
    if (v < nv) {
      const uint16_t* src = a.gate_up + row * 2 * a.I + 8 * v;
      gate[i] = ld_stream_v4(src);
      up[i] = ld_stream_v4(src + a.I);
    }
  }
  float y[VPT][8];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    float2 g[4], u[4];
    unpack8p(gate[i], g);
    unpack8p(up[i], u);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 v = silu_times(g[e], u[e]);
      y[i][2 * e] = v.x;
      y[i][2 * e + 1] = v.y;
    }
    if (!GROUPED) top = max(top, max8(y[i]));
  }
  if (!GROUPED) top = block_reduce(0.0f, top).top;
  store_rows<KIND, GROUPED, VPT>(y, top, row, nv, a.q, a.scale, a.groups);
}

}  // namespace

cudaError_t launch_norm_quant(const NormQuantArgs& a, int kind, bool grouped, int sms, cudaStream_t stream) {
  const int nv = a.H >> 3;
  auto launch = [&](auto kernel, int vpt) {
    return launch_pdl(kernel, dim3(a.b), dim3(threads_for(nv, vpt)), 0, stream, a);
  };
#define MOE_PICK(VPT)                                                                                        \
  (kind == kQuantInt8 ? (grouped ? launch(norm_quant_kernel<kQuantInt8, true, VPT>, VPT)                     \
                                 : launch(norm_quant_kernel<kQuantInt8, false, VPT>, VPT))                   \
                      : (grouped ? launch(norm_quant_kernel<kQuantE4M3, true, VPT>, VPT)                     \
                                 : launch(norm_quant_kernel<kQuantE4M3, false, VPT>, VPT)))
  // 16384 rows of 4096: 75.5 us with four vectors a thread, 81 with two, 88 with one.
  const int vpt = vectors_for(nv, a.b, sms, 4);
  return vpt == 1 ? MOE_PICK(1) : vpt == 4 ? MOE_PICK(4) : MOE_PICK(8);
#undef MOE_PICK
}

cudaError_t launch_silu_quant(const SiluQuantArgs& a, int kind, bool grouped, int sms, cudaStream_t stream) {
  const int nv = a.I >> 3;
  auto launch = [&](auto kernel, int vpt) {
    return launch_pdl(kernel, dim3((unsigned)a.rows), dim3(threads_for(nv, vpt)), 0, stream, a);
  };
#define MOE_PICK(VPT)                                                                                        \
  (kind == kQuantInt8 ? (grouped ? launch(silu_quant_kernel<kQuantInt8, true, VPT>, VPT)                     \
                                 : launch(silu_quant_kernel<kQuantInt8, false, VPT>, VPT))                   \
                      : (grouped ? launch(silu_quant_kernel<kQuantE4M3, true, VPT>, VPT)                     \
                                 : launch(silu_quant_kernel<kQuantE4M3, false, VPT>, VPT)))
  // 28672 rows of 2048 in e4m3 groups: 59 us with two vectors a thread, 60.5 with one, 62.5 with four.
  const int vpt = vectors_for(nv, a.rows, sms, 2);
  return vpt == 1 ? MOE_PICK(1) : vpt == 2 ? MOE_PICK(2) : vpt == 4 ? MOE_PICK(4) : MOE_PICK(8);
#undef MOE_PICK
}

}  // namespace moetail
