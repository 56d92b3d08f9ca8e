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
// the norm in 8-bit rows does: 16384 rows of 4096 in 86.2 us, 6.2 TB/s (0.93 of the measured copy rate), one token of 7168
// columns in 3.1 us.
// The gradient is persistent: a thread keeps eight columns and their column sums in registers while the rows pass, so that
// the sums cost one FP32 row of each kind for a thread block at the end, and a second small kernel adds those in a fixed
// order (no atomics: results do not change from run to run).  8192 rows of 4096 with every gradient take 71 us, 5.7 TB/s
// (0.85); 1500 rows of 18432, over clusters, 78 us (0.64: 138 of 152 SMs have a thread block of six).
#include <float.h>

#include <atomic>

#include "kernels.h"
#include "layer.h"
#include "product.cuh"
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

__device__ unsigned int g_norm_error = 0;

constexpr int kGradThreads = 512, kGradWarps = kGradThreads / 32;
constexpr int kGroupColumns = 2048;  // of a row that shares its thread block with others
constexpr int kMaxCluster = 8;       // thread blocks of a row: 32768 columns, eight a thread
constexpr int kMaxGradBlocks = 160;
constexpr int kAloneBytes = 116 * 1024;    // of which an SM has room for one thread block: two on one would leave others idle
constexpr int kStagedBytes = 200 * 1024;  // of rows in shared memory

// How a call's rows lie on thread blocks.
struct GradShape {
  int cluster;    // thread blocks of a row
  int vectors;    // of 8 columns, of a thread block
  int warps;      // of a row in a thread block
  int groups;     // rows at a time of a thread block
  int row_sets;   // clusters: sets of rows with their own column sums
  int stages;     // of rows in shared memory, 0: rows go to registers
};
int least_cluster(int H) { return (H + 8 * kGradThreads - 1) / (8 * kGradThreads); }
GradShape grad_shape(int H, int cluster) {
  GradShape s;
  s.cluster = cluster;
  s.vectors = ((H >> 3) + cluster - 1) / cluster;
  s.warps = (s.vectors + 31) / 32;
  const bool staged = H > kGroupColumns;
  s.groups = staged ? 1 : kGradWarps / s.warps;
  s.stages = staged ? kStagedBytes / (64 * s.vectors) : 0;
  if (s.stages > 8) s.stages = 8;
  s.row_sets = 0;
  return s;
}
int row_sets(int b, int groups, int most) {
  const int needed = (b + groups - 1) / groups;
  return needed < most ? needed : most;
}

// The columns' factors, as they are stored.
template <bool POST, bool CHANNEL>
struct Columns {
  uint4 post, pre, channel;
  __device__ __forceinline__ void load(const BlockNormGradArgs& a, int v, bool live) {
    post = pre = channel = make_uint4(0, 0, 0, 0);
    if (!live) return;
    pre = ld_v4(a.pre_gamma + 8 * v);
    if (POST) post = ld_v4(a.post_gamma + 8 * v);
    if (CHANNEL) channel = ld_v4(a.channel_gate + 8 * v);
  }
};
template <bool POST, bool CHANNEL>
struct Sums {
  float2 pre[4], post[4], channel[4];
  __device__ __forceinline__ Sums() {
#pragma unroll
    for (int e = 0; e < 4; ++e) pre[e] = post[e] = channel[e] = make_float2(0.0f, 0.0f);
  }
};
struct Row {
  float rstd0, rstd1, token;
  __device__ __forceinline__ void load(const BlockNormGradArgs& a, int64_t row) {
    rstd0 = rstd1 = 0.0f;
    token = 1.0f;
    if (row >= a.b) return;
    rstd0 = a.rstd[2 * row];
    rstd1 = a.rstd[2 * row + 1];
    if (a.token_gate) token = a.token_gate[row];
  }
};

// Eight columns of a row, two at a time.
template <bool POST, bool CHANNEL>
struct Values {
  float2 u[4], n[4], v[4], d_v[4];
  // From x, residual and d_y; returns the columns' part of the sum of d_v * v.
  __device__ __forceinline__ float form(const BlockNormGradArgs& a, const Row& r, const Columns<POST, CHANNEL>& c, uint4 x,
                                        uint4 residual, uint4 d_y) {
    float2 g[4], h[4], dot = make_float2(0.0f, 0.0f);
    unpack8p(x, u);
    if (POST) {
      unpack8p(c.post, g);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        u[e] = mul2(u[e], splat2(r.rstd0));
        n[e] = mul2(u[e], add2(g[e], splat2(a.gain_center)));
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) n[e] = u[e];
    }
    unpack8p(residual, h);
    if (CHANNEL) unpack8p(c.channel, g);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 gate = CHANNEL ? mul2(g[e], splat2(r.token)) : splat2(r.token);
      v[e] = mul2(fma2(gate, n[e], mul2(h[e], splat2(a.residual_scale))), splat2(r.rstd1));
    }
    unpack8p(d_y, d_v);
    unpack8p(c.pre, g);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      d_v[e] = mul2(d_v[e], add2(g[e], splat2(a.gain_center)));
      dot = fma2(d_v[e], v[e], dot);
    }
    return dot.x + dot.y;
  }
  // d_h in the place of d_v, given the mean of d_v * v; returns the columns' part of the sum of d_h * channel_gate * n.
  __device__ __forceinline__ float inner(const BlockNormGradArgs& a, const Row& r, const Columns<POST, CHANNEL>& c,
                                         Sums<POST, CHANNEL>& sums, float mean, uint4 d_y, uint4 d_residual) {
    float2 g[4], dot = make_float2(0.0f, 0.0f);
    unpack8p(d_y, g);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      sums.pre[e] = fma2(g[e], v[e], sums.pre[e]);
      d_v[e] = fma2(v[e], splat2(-mean), d_v[e]);
    }
    unpack8p(d_residual, g);
#pragma unroll
    for (int e = 0; e < 4; ++e) d_v[e] = fma2(d_v[e], splat2(r.rstd1), g[e]);
    if (CHANNEL) unpack8p(c.channel, g);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 d_n = mul2(d_v[e], n[e]);
      if (CHANNEL) {
        sums.channel[e] = fma2(d_n, splat2(r.token), sums.channel[e]);
        dot = fma2(d_n, g[e], dot);
      } else {
        dot = add2(dot, d_n);
      }
    }
    return dot.x + dot.y;
  }
};
__device__ __forceinline__ uint4 packed(const float2 (&v)[4]) {
  return make_uint4(bf16x2_pz(v[0].x, v[0].y), bf16x2_pz(v[1].x, v[1].y), bf16x2_pz(v[2].x, v[2].y), bf16x2_pz(v[3].x, v[3].y));
}
__device__ __forceinline__ uint4 packed(const float2 (&v)[4], float scale) {
  float2 w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) w[e] = mul2(v[e], splat2(scale));
  return packed(w);
}
// d_x of eight columns from their d_h and u, given the mean of d_u * u.
template <bool POST, bool CHANNEL>
__device__ __forceinline__ uint4 outer(const BlockNormGradArgs& a, const Row& r, const Columns<POST, CHANNEL>& c,
                                       Sums<POST, CHANNEL>& sums, const float2 (&d_h)[4], const float2 (&u)[4], float mean) {
  float2 g[4], d[4];
  if (CHANNEL) unpack8p(c.channel, g);
#pragma unroll
  for (int e = 0; e < 4; ++e) d[e] = mul2(d_h[e], CHANNEL ? mul2(g[e], splat2(r.token)) : splat2(r.token));  // d_n
  if (POST) {
    unpack8p(c.post, g);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      sums.post[e] = fma2(d[e], u[e], sums.post[e]);
      d[e] = mul2(fma2(d[e], add2(g[e], splat2(a.gain_center)), mul2(u[e], splat2(-mean))), splat2(r.rstd0));
    }
  }
  return packed(d);
}

__device__ __forceinline__ void st_columns(float* to, const float2 (&sum)[4]) {
  *reinterpret_cast<float4*>(to) = make_float4(sum[0].x, sum[0].y, sum[1].x, sum[1].y);
  *reinterpret_cast<float4*>(to + 4) = make_float4(sum[2].x, sum[2].y, sum[3].x, sum[3].y);
}

// Rows of at most 2048 columns: a group of warps each, the next row's loads in flight.
template <bool POST, bool CHANNEL>
__global__ void __launch_bounds__(kGradThreads, 1) grad_groups_kernel(const BlockNormGradArgs a, const GradShape s) {
  __shared__ float s_sum[2][kGradWarps];
  __shared__ float2 s_columns[kGradWarps][4 * 32];  // a warp's columns
  const int lane = threadIdx.x & 31, group = (threadIdx.x >> 5) / s.warps, warp = (threadIdx.x >> 5) - group * s.warps;
  const int v = 32 * warp + lane;  // this thread's vector of a row
  const bool live = v < s.vectors;
  grid_dependency_wait();
  launch_dependents();
  // The sum over a row's threads, the same in all of them, the warps' in a fixed order.  They meet in slots 0 and 1 in turn:
  // a thread that has passed the barrier of one knows that the other has been read.
  int slot = 0;
  auto row_sum = [&](float x) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    if (s.warps > 1) {
      if (lane == 0) s_sum[slot][group * s.warps + warp] = x;
      asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(32 * s.warps) : "memory");
      x = lane < s.warps ? s_sum[slot][group * s.warps + lane] : 0.0f;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
      slot ^= 1;
    }
    return x;
  };
  Columns<POST, CHANNEL> columns;
  columns.load(a, v, live);
  Sums<POST, CHANNEL> sums;
  struct Loads {
    uint4 x, residual, d_y, d_residual;
    Row row;
  } next;
  auto load = [&](int64_t row) {
    next.x = next.residual = next.d_y = next.d_residual = make_uint4(0, 0, 0, 0);
    next.row.load(a, row);
    if (row >= a.b || !live) return;
    const int64_t at = row * a.H + 8 * v;
    next.x = ld_rows(a.x + at);
    next.residual = ld_rows(a.residual + at);
    next.d_y = ld_rows(a.d_y + at);
    if (a.d_residual_out) next.d_residual = ld_rows(a.d_residual_out + at);
  };
  const int64_t stride = (int64_t)s.row_sets * s.groups;
  int64_t row = (int64_t)blockIdx.x * s.groups + group;
  load(row);
  for (; row < a.b; row += stride) {
    const Loads l = next;
    load(row + stride);
    Values<POST, CHANNEL> w;
    const float mean = row_sum(w.form(a, l.row, columns, l.x, l.residual, l.d_y)) * a.rcpH;
    float dot = w.inner(a, l.row, columns, sums, mean, l.d_y, l.d_residual);
    const int64_t at = row * a.H + 8 * v;
    if (live) st_v4(a.d_residual + at, packed(w.d_v, a.residual_scale));
    if (POST || a.d_token_gate) dot = row_sum(dot);
    if (a.d_token_gate && v == 0) a.d_token_gate[row] = dot;
    const uint4 d_x = outer(a, l.row, columns, sums, w.d_v, w.u, l.row.token * dot * a.rcpH);
    if (live) st_v4(a.d_x + at, d_x);
  }
  // The groups' column sums in their order, to this thread block's rows of the workspace.
  float* out = a.partial + (int64_t)blockIdx.x * 3 * a.H;
  auto leave = [&](float2 (&sum)[4], float* to) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 4; ++e) s_columns[threadIdx.x >> 5][32 * e + lane] = sum[e];
    __syncthreads();
    if (group > 0 || !live) return;
    for (int i = 1; i < s.groups; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] = add2(sum[e], s_columns[i * s.warps + warp][32 * e + lane]);
    st_columns(to + 8 * v, sum);
  };
  if (POST && a.d_post_gamma) leave(sums.post, out);
  if (a.d_pre_gamma) leave(sums.pre, out + a.H);
  if (CHANNEL && a.d_channel_gate) leave(sums.channel, out + 2 * a.H);
}

__device__ __forceinline__ void copy_bulk(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(bar)
               : "memory");
}
// Two values into shared memory of a thread block of the cluster, counted by a barrier there.
__device__ __forceinline__ void st_async_f32x2(uint32_t addr, float a, float b, uint32_t bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];" ::"r"(addr),
               "r"(__float_as_uint(a)), "r"(__float_as_uint(b)), "r"(bar)
               : "memory");
}

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
// Without an order of the memory accesses before it: does not wait for results on their way to memory.
__device__ __forceinline__ void cluster_sync_relaxed() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ unsigned long long limit(const BlockNormGradArgs& a, int times) {
  return a.stage_wait_ns ? a.stage_wait_ns : times * kWaitLimitNs;
}

// Wider rows: a row's (or a cluster's part of a row's) x, residual, d_y and d_residual_out arrive in shared memory, several
// rows ahead, and each row has one barrier: the second sum of a row and the first of the next meet at it.  In a cluster the
// warps send their sums to every thread block of it, and a barrier there counts their bytes: a barrier of the whole cluster
// would also wait for the row's results on their way to memory (8192 columns: 5.5 us a row).
//
// Every wait is bounded in time.  A thread whose wait runs out raises a bit in the device error word, tells its cluster (so that
// the others' waits end too) and asks for no more copies; what is written is undefined from there on.  Alone, a thread block
// walks on without the rows, since its barriers count every warp.  In a cluster a warp to which a row's sums have not come
// sends no more, and leaves.  No thread block ends before what is on its way to its shared memory has arrived: phases of
// barriers that stayed open because some of their threads stopped earlier are completed first.
template <bool POST, bool CHANNEL, bool CLUSTER>
__global__ void __launch_bounds__(kGradThreads, 1) grad_staged_kernel(const BlockNormGradArgs a, const GradShape s) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  __shared__ float2 s_sum[2][kMaxCluster * kGradWarps];
  __shared__ __align__(8) uint64_t s_bar[8], s_sent[2];
  __shared__ uint32_t s_abort;  // set in all thread blocks of a cluster
  __shared__ int s_brought[4], s_sends[kGradWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = CLUSTER ? (int)cluster_rank() : 0, ranks = CLUSTER ? (int)cluster_size() : 1;
  const int64_t set = CLUSTER ? blockIdx.x / ranks : blockIdx.x;
  const int first = part * s.vectors, vectors = min(s.vectors, (a.H >> 3) - first);
  const uint32_t row_bytes = 16u * vectors, stage_bytes = 64u * s.vectors, base = smem_addr(smem_raw), bars = smem_addr(s_bar);
  const int tensors = a.d_residual_out ? 4 : 3;
  if (threadIdx.x == 0) {
    for (int i = 0; i < s.stages; ++i) mbar_init(bars + 8 * i, tensors);
    for (int i = 0; i < 2; ++i) mbar_init(smem_addr(s_sent + i), 1);
    s_abort = a.stage_wait_ns == 1;  // to give up whatever comes
    if (s_abort) atomicOr(&g_norm_error, kErrWaitFull);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (CLUSTER) cluster_sync_all();  // its thread blocks have started, so that their shared memory can be written
  else __syncthreads();
  grid_dependency_wait();
  launch_dependents();

  const int64_t stride = (int64_t)s.row_sets * a.H;            // elements from one row of this set to its next
  const int rows = (int)((a.b - set + s.row_sets - 1) / s.row_sets);  // at least one
  // One lane of each of the first warps brings a tensor's part of a row (one thread for all of them kept its warp, and so
  // every barrier, waiting).
  const uint16_t* source = nullptr;
  if (lane == 0 && warp < tensors)
    source = (warp == 0 ? a.x : warp == 1 ? a.residual : warp == 2 ? a.d_y : a.d_residual_out) + set * a.H + 8 * first;
  const uint32_t apart = 16u * s.vectors;
  int brought = 0;
  auto bring = [&](uint32_t stage) {
    if (source == nullptr || brought >= rows) return;
    mbar_expect_tx(bars + 8 * stage, row_bytes);
    copy_bulk(base + stage * stage_bytes + warp * apart, source, row_bytes, bars + 8 * stage);
    source += stride;
    ++brought;
  };
  for (int i = 0; i < s.stages; ++i) bring(i);

  // This thread's vector of the thread block's part.  Threads past the last read what is there and add nothing to the sums.
  const int v = threadIdx.x;
  const bool live = v < vectors;
  Columns<POST, CHANNEL> columns;
  columns.load(a, first + v, live);
  Sums<POST, CHANNEL> sums;
  // Both waits look at the barrier before anything else: what follows is for those that run out.
  if (a.stage_wait_ns == 1) source = nullptr;
  auto give_up = [&] {
    if (!*(volatile uint32_t*)&s_abort) atomicOr(&g_norm_error, kErrWaitFull);
    if (CLUSTER)
      for (int i = 0; i < ranks; ++i) st_cluster_u32(map_to_rank(smem_addr(&s_abort), i), 1u);
    else
      *(volatile uint32_t*)&s_abort = 1u;
    source = nullptr;
  };
  auto wait = [&](uint32_t bar, uint32_t parity) {  // for a row
    if (mbar_try_wait(bar, parity) || mbar_wait(bar, parity, limit(a, 1), &s_abort)) return;
    give_up();
  };
  // One warp's sums of a row to all thread blocks of the cluster.
  auto send = [&](int to, float x, float y) {
    const uint32_t bar = smem_addr(s_sent + to);
    if (threadIdx.x == 0) mbar_expect_tx(bar, 8u * ranks * s.warps);
    if (lane < ranks)
      st_async_f32x2(map_to_rank(smem_addr(&s_sum[to][part * kGradWarps + warp]), lane), x, y, map_to_rank(bar, lane));
  };
  // Two sums over the row, the same in every thread, in a fixed order; slots in turn as for the groups.
  int slot = 0;
  uint32_t sent_parity = 0;
  bool lost = a.stage_wait_ns == 1;
  auto row_sums = [&](float x, float y) {
    bool here = true;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      x += __shfl_xor_sync(0xffffffffu, x, off);
      y += __shfl_xor_sync(0xffffffffu, y, off);
    }
    if (CLUSTER) {
      // A warp sends again after it has read what came for this row, so that a slot is never overtaken.
      send(slot, x, y);
      // Longer than the others wait for a row before they send on without it.
      const uint32_t bar = smem_addr(s_sent + slot);
      here = mbar_try_wait(bar, sent_parity) || mbar_wait(bar, sent_parity, limit(a, 2), &s_abort);
      if (slot == 1) sent_parity ^= 1u;
    } else {
      if (lane == 0) s_sum[slot][warp] = make_float2(x, y);
      __syncthreads();
    }
    float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < (CLUSTER ? kMaxCluster : 1) * kGradWarps; i += 32) {
      const int w = i + lane;
      if (w < ranks * kGradWarps && w % kGradWarps < s.warps) sum = add2(sum, s_sum[slot][w]);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      sum.x += __shfl_xor_sync(0xffffffffu, sum.x, off);
      sum.y += __shfl_xor_sync(0xffffffffu, sum.y, off);
    }
    slot ^= 1;
    if (CLUSTER && !here) {
      give_up();
      lost = true;
    }
    return sum;
  };
  Values<POST, CHANNEL> w;  // of the row at hand
  // The rows' scalars: a lane loads those of one row in 32 (loads in flight across the waits below made every row wait for them).
  Row of_lane;
  auto row_at = [&](int k) {  // called for 0, 1, 2, ..
    if (k % 32 == 0) of_lane.load(a, k + lane < rows ? set + (int64_t)(k + lane) * s.row_sets : a.b);
    Row row;
    row.rstd0 = __shfl_sync(0xffffffffu, of_lane.rstd0, k % 32);
    row.rstd1 = __shfl_sync(0xffffffffu, of_lane.rstd1, k % 32);
    row.token = __shfl_sync(0xffffffffu, of_lane.token, k % 32);
    return row;
  };
  Row r = row_at(0);
  const uint32_t mine = base + 16u * v;
  auto form = [&](const Row& row, uint32_t at) {
    const float dot = w.form(a, row, columns, ld_shared_v4(at), ld_shared_v4(at + apart), ld_shared_v4(at + 2 * apart));
    return live ? dot : 0.0f;
  };
  wait(bars, 0);
  float mean = row_sums(0.0f, form(r, mine)).y * a.rcpH;
  uint32_t stage = 0, parity = 0, at = mine;
  uint16_t *d_x = a.d_x + set * a.H + 8 * (first + v), *d_residual = a.d_residual + set * a.H + 8 * (first + v);
  float* d_token = a.d_token_gate && threadIdx.x == 0 && part == 0 ? a.d_token_gate + set : nullptr;
  int k = 0;
  for (; k < rows; ++k) {
    if (CLUSTER && __any_sync(0xffffffffu, lost)) break;  // after k + 1 rows' sums have been sent
    const uint4 d_out = a.d_residual_out ? ld_shared_v4(at + 3 * apart) : make_uint4(0, 0, 0, 0);
    float dot = w.inner(a, r, columns, sums, mean, ld_shared_v4(at + 2 * apart), d_out);
    if (!live) dot = 0.0f;
    if (live) st_v4(d_residual, packed(w.d_v, a.residual_scale));
    d_residual += stride;
    float2 d_h[4], u[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      d_h[e] = w.d_v[e];
      u[e] = w.u[e];
    }
    const Row here = r;
    const uint32_t read = stage;
    at += stage_bytes;
    if (++stage == (uint32_t)s.stages) {
      stage = 0;
      at = mine;
      parity ^= 1u;
    }
    float dot_next = 0.0f;
    if (k + 1 < rows) {
      r = row_at(k + 1);
      wait(bars + 8 * stage, parity);
      dot_next = form(r, at);
    }
    const float2 both = row_sums(dot, dot_next);
    bring(read);  // past the barrier every thread has read this row
    if (d_token) {
      *d_token = both.x;
      d_token += s.row_sets;
    }
    const uint4 out = outer(a, here, columns, sums, d_h, u, here.token * both.x * a.rcpH);
    if (live) st_v4(d_x, out);
    d_x += stride;
    mean = both.y * a.rcpH;
  }
  float* out = a.partial + set * 3 * a.H + 8 * (first + v);
  if (live) {
    if (POST && a.d_post_gamma) st_columns(out, sums.post);
    if (a.d_pre_gamma) st_columns(out + a.H, sums.pre);
    if (CHANNEL && a.d_channel_gate) st_columns(out + 2 * a.H, sums.channel);
  }

  // What is on its way to shared memory arrives before the thread block ends; where no wait ran out nothing is.
  if (CLUSTER) {
    together();
    if (*(volatile uint32_t*)&s_abort) asm volatile("fence.acq_rel.cluster;" ::: "memory");  // the flags before the barrier
    together();
    cluster_sync_relaxed();
  } else {
    __syncthreads();
  }
  if (!s_abort) return;  // the same in all thread blocks of the cluster: nobody waits any more
  const bool brings = lane == 0 && warp < tensors;
  if (brings) s_brought[warp] = brought;
  if (lane == 0) s_sends[warp] = k + 1;
  together();
  if (CLUSTER) cluster_sync_all();
  else __syncthreads();
  // A lane brings a row into a stage only once the stage's last one was complete, so that each stage lacks at most one
  // arrival of a lane.
  int most = 0;
  for (int i = 0; i < tensors; ++i) most = max(most, s_brought[i]);
  if (brings)
    for (int i = brought; i < most; ++i) mbar_arrive(bars + 8 * (i % s.stages));
  auto drain = [&](uint32_t bar, int round) {
    if (!mbar_wait(bar, (uint32_t)round & 1u)) atomicOr(&g_norm_error, kErrWaitDrain);
  };
  if (threadIdx.x == 0)
    for (int i = max(0, most - s.stages); i < most; ++i) drain(bars + 8 * (i % s.stages), i / s.stages);
  if (CLUSTER) {
    // A warp sends a row's sums only once all have sent the last row's: it lacks at most one row of those that most have.
    together();
    most = 0;
    for (int i = lane; i < ranks * s.warps; i += 32)
      most = max(most, (int)ld_cluster_u32(map_to_rank(smem_addr(&s_sends[i % s.warps]), i / s.warps)));
    most = __reduce_max_sync(0xffffffffu, most);
    if (k + 1 < most) send((k + 1) & 1, 0.0f, 0.0f);
    if (threadIdx.x == 0)
      for (int i = max(0, most - 2); i < most; ++i) drain(smem_addr(s_sent + (i & 1)), i >> 1);
    together();
    cluster_sync_all();
  }
}

// The sets' column sums added in their order: a warp takes every 32nd set for 128 columns, their loads in flight together.
__global__ void __launch_bounds__(1024) column_sums_kernel(const float* partial, int sets, int H, float* d_post, float* d_pre,
                                                           float* d_channel) {
  __shared__ float4 s_part[32][32];
  grid_dependency_wait();
  launch_dependents();
  float* out = blockIdx.y == 0 ? d_post : blockIdx.y == 1 ? d_pre : d_channel;
  if (!out) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x * 128 + 4 * lane;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c < H) {
#pragma unroll 5
    for (int i = warp; i < sets; i += 32) {
      const float4 p = __ldcg(reinterpret_cast<const float4*>(partial + ((int64_t)i * 3 + blockIdx.y) * H + c));
      sum.x += p.x;
      sum.y += p.y;
      sum.z += p.z;
      sum.w += p.w;
    }
  }
  s_part[warp][lane] = sum;
  __syncthreads();
  const int column = blockIdx.x * 128 + threadIdx.x;
  if (threadIdx.x < 128 && column < H) {
    float total = 0.0f;
#pragma unroll
    for (int w = 0; w < 32; ++w) total += reinterpret_cast<const float*>(s_part[w])[threadIdx.x];
    out[column] = total;
  }
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormArgs& a, int sms, cudaStream_t stream) {
  const int nv = a.H >> 3;
  auto launch = [&](auto kernel, int vpt) {
    return launch_pdl(kernel, dim3(a.b), dim3(threads_for(nv, vpt)), 0, stream, a);
  };
  // 16384 rows of 4096: 86.8 us with four vectors a thread, 92.5 with two, 102 with one.
  const int vpt = vectors_for(nv, a.b, sms, 4);
  if (a.post_gamma)
    return vpt == 1   ? launch(block_norm_kernel<true, 1>, 1)
           : vpt == 4 ? launch(block_norm_kernel<true, 4>, 4)
                      : launch(block_norm_kernel<true, 8>, 8);
  return vpt == 1   ? launch(block_norm_kernel<false, 1>, 1)
         : vpt == 4 ? launch(block_norm_kernel<false, 4>, 4)
                    : launch(block_norm_kernel<false, 8>, 8);
}

size_t block_norm_grad_workspace(int b, int H) {
  const GradShape s = grad_shape(H, least_cluster(H));
  return (size_t)row_sets(b, s.groups, kMaxGradBlocks / s.cluster) * 3 * H * sizeof(float);
}

namespace {

// The clusters of a launch that fit the current device at once: they lie within a part of the GPU, so that there are fewer
// of some sizes than the SMs divided by their size.  With one thread block an SM that depends on the size and the device
// alone, and is asked once for each.
cudaError_t clusters_at_once(const void* kernel, const cudaLaunchConfig_t& cfg, int cluster, int* n) {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices][kMaxCluster + 1];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool kept = dev < kDevices;
  if (kept && (*n = known[dev][cluster].load(std::memory_order_relaxed)) > 0) return cudaSuccess;
  cudaLaunchConfig_t only = cfg;  // without the other attribute
  only.attrs = cfg.attrs + 1;
  only.numAttrs = 1;
  e = cudaOccupancyMaxActiveClusters(n, kernel, &only);
  if (e == cudaSuccess && kept) known[dev][cluster].store(*n, std::memory_order_relaxed);
  return e;
}

template <bool POST, bool CHANNEL>
cudaError_t launch_grad(const BlockNormGradArgs& a, int most, int* sets, cudaStream_t stream) {
  GradShape s = grad_shape(a.H, least_cluster(a.H));
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  cfg.attrs = attr;
  cfg.stream = stream;
  auto shape = [&](int cluster) {
    s = grad_shape(a.H, cluster);
    attr[1].val.clusterDim = {(unsigned)cluster, 1, 1};
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    cfg.gridDim = dim3(cluster);
    cfg.blockDim = dim3(32 * s.warps * s.groups);  // every thread takes part in a row: its barriers count them all
    if (s.stages) {
      const int bytes = s.stages * 64 * s.vectors + 512;  // threads past the last vector read on
      cfg.dynamicSmemBytes = bytes < kAloneBytes ? kAloneBytes : bytes;
    }
  };
  shape(s.cluster);
  auto kernel = s.stages == 0 ? grad_groups_kernel<POST, CHANNEL>
                : s.cluster > 1 ? grad_staged_kernel<POST, CHANNEL, true>
                                : grad_staged_kernel<POST, CHANNEL, false>;
  if (s.stages > 0) {
    const cudaError_t e = ensure_smem_limit((const void*)kernel, kStagedBytes + 512);
    if (e != cudaSuccess) return e;
  }
  int at_once = most / s.cluster;
  if (s.cluster > 1) {  // the size of which the most SMs have a thread block
    int best = s.cluster, best_blocks = 0;
    // Only even sizes: of five, the clusters that should fit did not all run at once (1820 rows of 18432 columns: 128 us
    // with five, 90 with six).  At least a warp for each tensor of a row.
    for (int c = s.cluster + s.cluster % 2; c <= kMaxCluster && a.H >= 8 * 32 * 4 * c; c += 2) {
      shape(c);
      int fit = 0;
      const cudaError_t e = clusters_at_once((const void*)kernel, cfg, c, &fit);
      if (e != cudaSuccess) return e;  // another number would be another order of the sums
      const int n = fit < most / c ? fit : most / c;
      if (n * c > best_blocks) {
        best = c;
        best_blocks = n * c;
        at_once = n;
      }
    }
    if (best_blocks == 0) return cudaErrorLaunchOutOfResources;  // no size fits
    shape(best);
  }
  s.row_sets = *sets = row_sets(a.b, s.groups, at_once);
  cfg.gridDim = dim3(s.row_sets * s.cluster);
  return cudaLaunchKernelEx(&cfg, kernel, a, s);
}

}  // namespace

cudaError_t launch_block_norm_grad(const BlockNormGradArgs& a, int sms, cudaStream_t stream) {
  const int most = sms < kMaxGradBlocks ? sms : kMaxGradBlocks;
  int sets = 0;  // no rows: no sets, and the sums are zeros
  cudaError_t e = cudaSuccess;
  if (a.b > 0) {
    e = a.post_gamma ? (a.channel_gate ? launch_grad<true, true>(a, most, &sets, stream) : launch_grad<true, false>(a, most, &sets, stream))
                     : (a.channel_gate ? launch_grad<false, true>(a, most, &sets, stream) : launch_grad<false, false>(a, most, &sets, stream));
    if (e != cudaSuccess) return e;
  }
  if (!a.d_post_gamma && !a.d_pre_gamma && !a.d_channel_gate) return e;
  return launch_pdl(column_sums_kernel, dim3((a.H + 127) / 128, 3), dim3(1024), 0, stream, (const float*)a.partial, sets,
                    a.H, a.d_post_gamma, a.d_pre_gamma, a.d_channel_gate);
}

cudaError_t take_block_norm_error(unsigned* bits) {
  unsigned v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_norm_error, sizeof v);
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_norm_error, &zero, sizeof zero);
  *bits = v;
  return e;
}

}  // namespace moetail
