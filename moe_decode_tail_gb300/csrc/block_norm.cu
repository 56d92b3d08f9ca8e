// The norms after and before a block, fused with its gate and the scaled residual, and their gradients (sm_103a).
//
//   forward   n = (x * rstd0) * (post_gamma + c)            (without a norm after the block: n = x)
//             h = residual_scale * residual + (token_gate * channel_gate) * n
//             residual_out = bf16(h),  y = bf16((h * rstd1) * (pre_gamma + c)),  rstd = 1 / sqrt(mean of squares + eps)
//   gradient  with u = x * rstd0, v = h * rstd1, g = token_gate * channel_gate, and h formed again from x and residual
//             in FP32 (the norm is of h, not of its BF16 rounding):
//               d_v  = d_y * (pre_gamma + c)
//               d_h  = d_residual_out + rstd1 * (d_v - v * mean(d_v * v))
//               d_residual = residual_scale * d_h,  d_n = g * d_h,  d_u = d_n * (post_gamma + c)
//               d_x  = rstd0 * (d_u - u * mean(d_u * u))          (without a norm after the block: d_x = d_n)
//               d_token_gate = sum of d_h * channel_gate * n      (a row's; mean(d_u * u) is token_gate / H times it)
//               d_pre_gamma = sum of d_y * v,  d_post_gamma = sum of d_n * u,  d_channel_gate = sum of d_h * token_gate * n
//                                                                 (a column's, over the rows)
//
// Both are bound by memory: 8 and 12 bytes a column, every input read once.  The forward takes a thread block a row, as
// the norm in 8-bit rows does.
// The gradient is persistent: a thread keeps eight columns and their column sums in registers while the rows pass, the
// next row's loads in flight, so that the sums cost one FP32 row of each kind for a thread block at the end, and a second
// small kernel adds those in a fixed order (no atomics: results do not change from run to run).  Rows of at most 2048
// columns share a thread block, each by a group of warps; rows of more than 4096 are spread over a cluster of thread
// blocks, whose warps write their sums into one another's shared memory.
#include <float.h>

#include "kernels.h"
#include "layer.h"
#include "rows.cuh"

namespace moetail {

namespace {

// ---- forward -------------------------------------------------------------------------------------------------------

// 1 / rms of a row held in h (threads past its end hold zeros).  Where its squares leave FP32's range or lose bits below
// it, the row is brought near one by a power of two first, which changes no bit of h * result.  *rstd: of the row as it was.
// Two calls with different IDs need no barrier between them.
template <int ID, int VPT>
__device__ __forceinline__ float row_rstd(float (&h)[VPT][8], float rcpH, float eps, float* rstd) {
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) sum += h[i][e] * h[i][e];
  float mean = block_reduce<2 * ID>(sum, 0u).sum * rcpH + eps;
  float unit = 1.0f;
  if (!(mean >= 0x1p-100f && mean <= FLT_MAX)) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) top = max(top, max8(h[i]));
    const float most = __uint_as_float(block_reduce<2 * ID + 1>(0.0f, top).top);
    const float size = fmaxf(most, __fsqrt_rn(eps));
    if (most <= FLT_MAX && size > 0.0f) {  // else the row has no finite norm
      const int exponent = min(max((int)(magnitude(size) >> 23), 1), 253);
      unit = __uint_as_float((uint32_t)(254 - exponent) << 23);  // size * unit is in [1, 4), or below one
      sum = 0.0f;
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          h[i][e] *= unit;
          sum += h[i][e] * h[i][e];
        }
      mean = block_reduce<2 * ID>(sum, 0u).sum * rcpH + eps * unit * unit;  // the reduction between kept the first apart
    }
  }
  const float inv = __fdiv_rn(1.0f, __fsqrt_rn(mean));
  *rstd = inv * unit;
  return inv;
}

// VPT: vectors of 8 columns of a thread; thread t holds vectors t, t + blockDim, ...
template <bool POST, int VPT>
__global__ void __launch_bounds__(VPT == 1 ? 1024 : 512) block_norm_kernel(const BlockNormArgs a) {
  grid_dependency_wait();
  launch_dependents();
  const int64_t row = blockIdx.x;
  const int nv = a.H >> 3;
  uint4 res[VPT];
  float h[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    uint4 x = make_uint4(0, 0, 0, 0);
    res[i] = x;
    if (v < nv) {
      x = ld_rows(a.x + row * a.H + 8 * v);
      res[i] = ld_rows(a.residual + row * a.H + 8 * v);
    }
    unpack8(x, h[i]);
  }
  const float token = a.token_gate ? a.token_gate[row] : 1.0f;
  float rstd0 = 1.0f, rstd1;
  float inv = 1.0f;
  if (POST) inv = row_rstd<0, VPT>(h, a.rcpH, a.eps, &rstd0);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    if (v >= nv) continue;  // zeros
    float r[8], g[8], c[8];
    unpack8(res[i], r);
    if (POST) {
      unpack8(ld_v4(a.post_gamma + 8 * v), g);
#pragma unroll
      for (int e = 0; e < 8; ++e) h[i][e] = (h[i][e] * inv) * (g[e] + a.gain_center);
    }
    if (a.channel_gate) {
      unpack8(ld_v4(a.channel_gate + 8 * v), c);
#pragma unroll
      for (int e = 0; e < 8; ++e) h[i][e] *= token * c[e];
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) h[i][e] *= token;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) h[i][e] += a.residual_scale * r[e];
    st_v4(a.residual_out + row * a.H + 8 * v, pack8_pz(h[i]));
  }
  inv = row_rstd<1, VPT>(h, a.rcpH, a.eps, &rstd1);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    if (v >= nv) continue;
    float g[8];
    unpack8(ld_v4(a.pre_gamma + 8 * v), g);
#pragma unroll
    for (int e = 0; e < 8; ++e) h[i][e] = (h[i][e] * inv) * (g[e] + a.gain_center);
    st_v4(a.y + row * a.H + 8 * v, pack8_pz(h[i]));
  }
  if (a.rstd && threadIdx.x == 0) *reinterpret_cast<float2*>(a.rstd + 2 * row) = make_float2(rstd0, rstd1);
}

// ---- gradient ------------------------------------------------------------------------------------------------------

constexpr int kGradThreads = 512, kGradWarps = kGradThreads / 32;
constexpr int kGradColumns = 8 * kGradThreads;  // columns of a thread block
constexpr int kMaxCluster = 8;                  // thread blocks of a row: 32768 columns
constexpr int kMaxGradBlocks = 160;

// How a call's rows lie on thread blocks.
struct GradShape {
  int cluster;    // thread blocks of a row
  int vectors;    // of 8 columns, of a thread block
  int warps;      // of a row in a thread block
  int groups;     // rows at a time of a thread block
  int row_sets;   // clusters: sets of rows with their own column sums
};
GradShape grad_shape(int b, int H, int blocks) {
  GradShape s;
  const int nv = H >> 3;
  s.cluster = 1;
  while (s.cluster * kGradThreads < nv) s.cluster *= 2;
  s.vectors = (nv + s.cluster - 1) / s.cluster;
  s.warps = (s.vectors + 31) / 32;
  s.groups = s.cluster > 1 ? 1 : kGradWarps / s.warps;
  const int most = blocks / s.cluster, needed = (b + s.groups - 1) / s.groups;
  s.row_sets = needed < most ? needed : most;
  return s;
}

// The sum over a row's threads, the same in all of them: a warp's by shuffles, then the warps' in a fixed order.  The warps'
// sums meet in slots 0 and 1 in turn: a thread that has passed the barrier of one knows that the other has been read.
template <bool CLUSTER>
__device__ __forceinline__ float row_sum(float v, int& turn, int group, int warps, int warp, float (*s_sum)[kMaxCluster * kGradWarps]) {
  const int lane = threadIdx.x & 31, slot = turn;
  turn ^= 1;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  if (CLUSTER) {
    const int ranks = (int)cluster_size();
    if (lane < ranks) st_cluster_f32(map_to_rank(smem_addr(&s_sum[slot][cluster_rank() * kGradWarps + warp]), lane), v);
    cluster_sync_all();
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < kMaxCluster * kGradWarps; i += 32) {
      const int w = i + lane;
      if (w < ranks * kGradWarps && w % kGradWarps < warps) v += s_sum[slot][w];
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  } else if (warps > 1) {
    if (lane == 0) s_sum[slot][group * warps + warp] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(32 * warps) : "memory");
    v = lane < warps ? s_sum[slot][group * warps + lane] : 0.0f;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  }
  return v;
}

template <bool POST, bool CHANNEL, bool CLUSTER>
__global__ void __launch_bounds__(kGradThreads, 1) block_norm_grad_kernel(const BlockNormGradArgs a, const GradShape s) {
  __shared__ float s_sum[2][kMaxCluster * kGradWarps];
  __shared__ float s_columns[kGradWarps][256];  // a warp's columns
  const int group = (threadIdx.x >> 5) / s.warps, warp = (threadIdx.x >> 5) - group * s.warps;
  const int t = threadIdx.x - 32 * group * s.warps;  // the thread's vector in its thread block's part of the row
  const int part = CLUSTER ? (int)cluster_rank() : 0;
  const int64_t set = CLUSTER ? blockIdx.x / cluster_size() : blockIdx.x;
  const int v = part * s.vectors + t;
  const bool live = t < s.vectors && 8 * v < a.H;
  if (CLUSTER) cluster_sync_all();  // its thread blocks have started, so that their shared memory can be written
  grid_dependency_wait();
  launch_dependents();

  const uint4 zero = make_uint4(0, 0, 0, 0);
  uint4 post = zero, pre = zero, channel = zero;
  if (live) {
    pre = ld_v4(a.pre_gamma + 8 * v);
    if (POST) post = ld_v4(a.post_gamma + 8 * v);
    if (CHANNEL) channel = ld_v4(a.channel_gate + 8 * v);
  }
  float sum_pre[8], sum_post[8], sum_channel[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) sum_pre[e] = sum_post[e] = sum_channel[e] = 0.0f;

  struct Row {
    uint4 x, residual, d_y, d_residual;
    float rstd0, rstd1, token;
  };
  const int64_t stride = (int64_t)s.row_sets * s.groups;
  auto load = [&](int64_t row, Row& r) {
    r = Row{zero, zero, zero, zero, 0.0f, 0.0f, 1.0f};
    if (row >= a.b) return;
    if (live) {
      const int64_t at = row * a.H + 8 * v;
      r.x = ld_rows(a.x + at);
      r.residual = ld_rows(a.residual + at);
      r.d_y = ld_rows(a.d_y + at);
      if (a.d_residual_out) r.d_residual = ld_rows(a.d_residual_out + at);
    }
    r.rstd0 = a.rstd[2 * row];
    r.rstd1 = a.rstd[2 * row + 1];
    if (a.token_gate) r.token = a.token_gate[row];
  };
  Row next;
  int64_t row = set * s.groups + group;
  int turn = 0;
  load(row, next);
  for (; row < a.b; row += stride) {
    const Row r = next;
    load(row + stride, next);
    float x[8], n[8], c[8], h[8], d[8], g[8];
    unpack8(r.x, x);
    unpack8(r.residual, h);
    unpack8(r.d_y, d);
    unpack8(pre, g);
    if (CHANNEL) unpack8(channel, c);
    if (POST) {
      float p[8];
      unpack8(post, p);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] *= r.rstd0;  // u
        n[e] = x[e] * (p[e] + a.gain_center);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) n[e] = x[e];
    }
    float dot = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float gate = CHANNEL ? r.token * c[e] : r.token;
      h[e] = (a.residual_scale * h[e] + gate * n[e]) * r.rstd1;  // v
      sum_pre[e] += d[e] * h[e];
      d[e] *= g[e] + a.gain_center;  // d_v
      dot += d[e] * h[e];
    }
    const float mean = row_sum<CLUSTER>(dot, turn, group, s.warps, warp, s_sum) * a.rcpH;
    const int64_t at = row * a.H + 8 * v;
    unpack8(r.d_residual, g);
#pragma unroll
    for (int e = 0; e < 8; ++e) d[e] = g[e] + r.rstd1 * (d[e] - h[e] * mean);  // d_h
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = a.residual_scale * d[e];
    if (live) st_v4(a.d_residual + at, pack8_pz(h));
    dot = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float dn = d[e] * n[e];
      if (CHANNEL) sum_channel[e] += r.token * dn;
      dot += CHANNEL ? c[e] * dn : dn;
    }
    float d_token = 0.0f;
    if (POST || a.d_token_gate) d_token = row_sum<CLUSTER>(dot, turn, group, s.warps, warp, s_sum);
    if (a.d_token_gate && t == 0 && part == 0) a.d_token_gate[row] = d_token;
    const float mean_u = r.token * d_token * a.rcpH;
    if (POST) {
      float p[8];
      unpack8(post, p);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        d[e] *= CHANNEL ? r.token * c[e] : r.token;  // d_n
        sum_post[e] += d[e] * x[e];
        d[e] = r.rstd0 * (d[e] * (p[e] + a.gain_center) - x[e] * mean_u);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) d[e] *= CHANNEL ? r.token * c[e] : r.token;
    }
    if (live) st_v4(a.d_x + at, pack8_pz(d));
  }

  // The column sums of the thread block's groups, in their order, to this set's rows of the workspace.
  float* out = a.partial + set * 3 * a.H;
  auto leave = [&](float (&sum)[8], float* to) {
    __syncthreads();
    if (group > 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) s_columns[threadIdx.x >> 5][32 * e + (threadIdx.x & 31)] = sum[e];
    }
    __syncthreads();
    if (group == 0 && live) {
      for (int i = 1; i < s.groups; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] += s_columns[i * s.warps + warp][32 * e + (threadIdx.x & 31)];
      *reinterpret_cast<float4*>(to + 8 * v) = make_float4(sum[0], sum[1], sum[2], sum[3]);
      *reinterpret_cast<float4*>(to + 8 * v + 4) = make_float4(sum[4], sum[5], sum[6], sum[7]);
    }
  };
  if (POST && a.d_post_gamma) leave(sum_post, out);
  if (a.d_pre_gamma) leave(sum_pre, out + a.H);
  if (CHANNEL && a.d_channel_gate) leave(sum_channel, out + 2 * a.H);
}

// The sets' column sums added in their order: a warp takes every eighth set for 128 columns.
__global__ void __launch_bounds__(256) column_sums_kernel(const float* partial, int sets, int H, float* d_post, float* d_pre,
                                                          float* d_channel) {
  __shared__ float4 s_part[8][32];
  grid_dependency_wait();
  launch_dependents();
  float* out = blockIdx.y == 0 ? d_post : blockIdx.y == 1 ? d_pre : d_channel;
  if (!out) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x * 128 + 4 * lane;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c < H) {
#pragma unroll 4
    for (int i = warp; i < sets; i += 8) {
      const float4 p = __ldcg(reinterpret_cast<const float4*>(partial + ((int64_t)i * 3 + blockIdx.y) * H + c));
      sum.x += p.x;
      sum.y += p.y;
      sum.z += p.z;
      sum.w += p.w;
    }
  }
  s_part[warp][lane] = sum;
  __syncthreads();
  if (warp == 0 && c < H) {
#pragma unroll
    for (int w = 1; w < 8; ++w) {
      const float4 p = s_part[w][lane];
      sum.x += p.x;
      sum.y += p.y;
      sum.z += p.z;
      sum.w += p.w;
    }
    *reinterpret_cast<float4*>(out + c) = sum;
  }
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormArgs& a, int sms, cudaStream_t stream) {
  const int nv = a.H >> 3;
  auto launch = [&](auto kernel, int vpt) {
    return launch_pdl(kernel, dim3(a.b), dim3(threads_for(nv, vpt)), 0, stream, a);
  };
  const int vpt = vectors_for(nv, a.b, sms, 2);
  if (a.post_gamma)
    return vpt == 1   ? launch(block_norm_kernel<true, 1>, 1)
           : vpt == 2 ? launch(block_norm_kernel<true, 2>, 2)
           : vpt == 4 ? launch(block_norm_kernel<true, 4>, 4)
                      : launch(block_norm_kernel<true, 8>, 8);
  return vpt == 1   ? launch(block_norm_kernel<false, 1>, 1)
         : vpt == 2 ? launch(block_norm_kernel<false, 2>, 2)
         : vpt == 4 ? launch(block_norm_kernel<false, 4>, 4)
                    : launch(block_norm_kernel<false, 8>, 8);
}

size_t block_norm_grad_workspace(int b, int H) {
  return (size_t)grad_shape(b, H, kMaxGradBlocks).row_sets * 3 * H * sizeof(float);
}

cudaError_t launch_block_norm_grad(const BlockNormGradArgs& a, int sms, cudaStream_t stream) {
  const GradShape s = grad_shape(a.b, a.H, sms < kMaxGradBlocks ? sms : kMaxGradBlocks);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(s.row_sets * s.cluster);
  cfg.blockDim = dim3(32 * s.warps * s.groups);  // every thread takes part in a row: the cluster's barriers count them all
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {(unsigned)s.cluster, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = s.cluster > 1 ? 2 : 1;
  cudaError_t e = cudaSuccess;
  if (a.b > 0) {
    auto launch = [&](auto kernel) { return cudaLaunchKernelEx(&cfg, kernel, a, s); };
#define MOE_PICK(POST, CHANNEL) \
  (s.cluster > 1 ? launch(block_norm_grad_kernel<POST, CHANNEL, true>) : launch(block_norm_grad_kernel<POST, CHANNEL, false>))
    e = a.post_gamma ? (a.channel_gate ? MOE_PICK(true, true) : MOE_PICK(true, false))
                     : (a.channel_gate ? MOE_PICK(false, true) : MOE_PICK(false, false));
#undef MOE_PICK
    if (e != cudaSuccess) return e;
  }
  if (!a.d_post_gamma && !a.d_pre_gamma && !a.d_channel_gate) return e;
  // no rows: no sets, and the sums are zeros
  return launch_pdl(column_sums_kernel, dim3((a.H + 127) / 128, 3), dim3(256), 0, stream, (const float*)a.partial, s.row_sets,
                    a.H, a.d_post_gamma, a.d_pre_gamma, a.d_channel_gate);
}

}  // namespace moetail
