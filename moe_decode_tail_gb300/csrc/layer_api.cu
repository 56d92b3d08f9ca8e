// C ABI of the operators around the tail (8-bit rows, routes, the 8-bit product): argument checks and launches.
// Every check runs before the first CUDA call, so a refused call touches no device state.
#include "host_util.h"
#include "kernels.h"
#include "layer.h"

namespace {

using moetail::device_sms;
using moetail::kMaxExperts;
using moetail::kMaxK;
using moetail::kMaxP;
using moetail::kQuantGroup;

constexpr int64_t kMaxRows = (int64_t)1 << 22;    // rows (or routes) of one call
constexpr int64_t kMaxRoutes = (int64_t)1 << 21;  // routes of one sort
constexpr int kMaxD = 1 << 16, kMaxN = 1 << 20;   // the product's reduction length and channels

// One operand of a call: its range, and whether it may be null.
struct Operand {
  const void* p;
  size_t bytes;
  uintptr_t align;
  bool optional;
};

bool valid(const Operand& o) { return o.p ? aligned(o.p, o.align) : (o.optional || o.bytes == 0); }

// All operands valid, and no output overlapping an input or another output.
template <int NI, int NO>
bool operands_ok(const Operand (&in)[NI], const Operand (&out)[NO]) {
  for (const Operand& i : in)
    if (!valid(i)) return false;
  for (int o = 0; o < NO; ++o) {
    if (!valid(out[o])) return false;
    if (!out[o].p) continue;
    const Range r = span(out[o].p, out[o].bytes);
    for (const Operand& i : in)
      if (i.p && overlaps(r, span(i.p, i.bytes))) return false;
    for (int q = 0; q < o; ++q)
      if (out[q].p && overlaps(r, span(out[q].p, out[q].bytes))) return false;
  }
  return true;
}

bool width_ok(int w) { return w >= 8 && w <= kMaxP && w % 8 == 0; }

// Scales of a row of `width` columns; 0 for an unknown grouping.
int groups_of(int width, int group) {
  return group == 0 ? 1 : group == kQuantGroup ? (width + kQuantGroup - 1) / kQuantGroup : 0;
}

bool routes_ok(int b, int K) { return b >= 0 && K >= 1 && K <= kMaxK && (int64_t)b * K <= kMaxRows; }

bool weights_ok(int dtype) { return dtype == MOE_TAIL_W_FP32 || dtype == MOE_TAIL_W_BF16; }
size_t weight_size(int dtype) { return dtype == MOE_TAIL_W_FP32 ? 4 : 2; }

}  // namespace

// ============================================================================ 8-bit rows

MOE_API int moe_tail_norm_quant(const void* x, const void* residual, const void* gamma, float gain_center, float eps,
                                int b, int H, int q_dtype, int group, void* residual_out, void* y, void* q, void* scale,
                                void* stream) {
  const int groups = groups_of(H, group);
  if (b < 0 || b > kMaxRows || !width_ok(H) || groups == 0) return MOE_TAIL_EINVAL;
  if (q_dtype != MOE_TAIL_Q_INT8 && q_dtype != MOE_TAIL_Q_E4M3) return MOE_TAIL_EINVAL;
  if (b == 0) return MOE_TAIL_OK;
  const size_t n = (size_t)b * H;
  // the new residual may take x's or the residual's own place: each element is read before it is written
  const bool in_x = residual_out && residual_out == x, in_residual = residual_out && residual_out == residual;
  const Operand in[] = {{in_x ? nullptr : x, 2 * n, 16, in_x},
                        {in_residual ? nullptr : residual, 2 * n, 16, true},
                        {gamma, 2 * (size_t)H, 16, false}};
  const Operand out[] = {{residual_out, 2 * n, 16, true}, {y, 2 * n, 16, true}, {q, n, 16, false},
                         {scale, 4 * (size_t)b * groups, 4, false}};
  if (!operands_ok(in, out)) return MOE_TAIL_EINVAL;
  moetail::NormQuantArgs a;
  a.x = static_cast<const uint16_t*>(x);
  a.residual = static_cast<const uint16_t*>(residual);
  a.gamma = static_cast<const uint16_t*>(gamma);
  a.gain_center = gain_center;
  a.eps = eps;
  a.rcpH = (float)(1.0 / (double)H);
  a.b = b;
  a.H = H;
  a.residual_out = static_cast<uint16_t*>(residual_out);
  a.y = static_cast<uint16_t*>(y);
  a.q = static_cast<uint8_t*>(q);
  a.scale = static_cast<float*>(scale);
  a.groups = groups;
  return finish(moetail::launch_norm_quant(a, q_dtype, group != 0, device_sms(), static_cast<cudaStream_t>(stream)));
}

MOE_API int moe_tail_silu_quant(const void* gate_up, const int32_t* used_rows, int rows, int I, int q_dtype, int group,
                                void* q, void* scale, void* stream) {
  const int groups = groups_of(I, group);
  if (rows < 0 || rows > kMaxRows || !width_ok(I) || groups == 0) return MOE_TAIL_EINVAL;
  if (q_dtype != MOE_TAIL_Q_INT8 && q_dtype != MOE_TAIL_Q_E4M3) return MOE_TAIL_EINVAL;
  if (rows == 0) return MOE_TAIL_OK;
  const size_t n = (size_t)rows * I;
  const Operand in[] = {{gate_up, 4 * n, 16, false}, {used_rows, 4, 4, true}};
  const Operand out[] = {{q, n, 16, false}, {scale, 4 * (size_t)rows * groups, 4, false}};
  if (!operands_ok(in, out)) return MOE_TAIL_EINVAL;
  moetail::SiluQuantArgs a;
  a.gate_up = static_cast<const uint16_t*>(gate_up);
  a.used = used_rows;
  a.rows = rows;
  a.I = I;
  a.q = static_cast<uint8_t*>(q);
  a.scale = static_cast<float*>(scale);
  a.groups = groups;
  return finish(moetail::launch_silu_quant(a, q_dtype, group != 0, device_sms(), static_cast<cudaStream_t>(stream)));
}

// ============================================================================ norms around a block

MOE_API int moe_tail_block_norm(const void* x, const void* residual, const void* post_gamma, const void* pre_gamma,
                                const float* token_gate, const void* channel_gate, float residual_scale,
                                float gain_center, float eps, int b, int H, void* residual_out, void* y, float* rstd,
                                void* stream) {
  if (b < 0 || b > kMaxRows || !width_ok(H)) return MOE_TAIL_EINVAL;
  if (b == 0) return MOE_TAIL_OK;
  const size_t n = (size_t)b * H, row = 2 * (size_t)H;
  // the new residual may take x's or the residual's own place: each element is read before it is written
  const bool in_x = residual_out && residual_out == x, in_residual = residual_out && residual_out == residual;
  const Operand in[] = {{in_x ? nullptr : x, 2 * n, 16, in_x},
                        {in_residual ? nullptr : residual, 2 * n, 16, in_residual},
                        {post_gamma, row, 16, true},
                        {pre_gamma, row, 16, false},
                        {token_gate, 4 * (size_t)b, 4, true},
                        {channel_gate, row, 16, true}};
  const Operand out[] = {{residual_out, 2 * n, 16, false}, {y, 2 * n, 16, false}, {rstd, 8 * (size_t)b, 8, true}};
  if (!operands_ok(in, out)) return MOE_TAIL_EINVAL;
  moetail::BlockNormArgs a;
  a.x = static_cast<const uint16_t*>(x);
  a.residual = static_cast<const uint16_t*>(residual);
  a.post_gamma = static_cast<const uint16_t*>(post_gamma);
  a.pre_gamma = static_cast<const uint16_t*>(pre_gamma);
  a.token_gate = token_gate;
  a.channel_gate = static_cast<const uint16_t*>(channel_gate);
  a.residual_scale = residual_scale;
  a.gain_center = gain_center;
  a.eps = eps;
  a.rcpH = (float)(1.0 / (double)H);
  a.b = b;
  a.H = H;
  a.residual_out = static_cast<uint16_t*>(residual_out);
  a.y = static_cast<uint16_t*>(y);
  a.rstd = rstd;
  return finish(moetail::launch_block_norm(a, device_sms(), static_cast<cudaStream_t>(stream)));
}

MOE_API size_t moe_tail_block_norm_grad_workspace_bytes(int b, int H) {
  if (b < 0 || b > kMaxRows || !width_ok(H)) return 0;
  return round256(moetail::block_norm_grad_workspace(b < 1 ? 1 : b, H));
}

MOE_API int moe_tail_block_norm_grad(const void* d_y, const void* d_residual_out, const void* x, const void* residual,
                                     const void* post_gamma, const void* pre_gamma, const float* token_gate,
                                     const void* channel_gate, const float* rstd, float residual_scale,
                                     float gain_center, int b, int H, void* d_x, void* d_residual, float* d_post_gamma,
                                     float* d_pre_gamma, float* d_token_gate, float* d_channel_gate, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  if (b < 0 || b > kMaxRows || !width_ok(H)) return MOE_TAIL_EINVAL;
  // a gradient of what is not there
  if ((d_post_gamma && !post_gamma) || (d_token_gate && !token_gate) || (d_channel_gate && !channel_gate))
    return MOE_TAIL_EINVAL;
  const size_t n = (size_t)b * H, row = 2 * (size_t)H, tokens = 4 * (size_t)b;
  // d_x may take d_y's place and d_residual d_residual_out's: each element is read before it is written
  const bool in_y = d_x && d_x == d_y, in_residual = d_residual && d_residual == d_residual_out;
  const Operand in[] = {{in_y ? nullptr : d_y, 2 * n, 16, in_y},
                        {in_residual ? nullptr : d_residual_out, 2 * n, 16, true},
                        {x, 2 * n, 16, false},
                        {residual, 2 * n, 16, false},
                        {post_gamma, row, 16, true},
                        {pre_gamma, row, 16, false},
                        {token_gate, tokens, 4, true},
                        {channel_gate, row, 16, true},
                        {rstd, 2 * tokens, 8, false}};
  const Operand out[] = {{d_x, 2 * n, 16, false},
                         {d_residual, 2 * n, 16, false},
                         {d_post_gamma, 4 * (size_t)H, 16, true},
                         {d_pre_gamma, 4 * (size_t)H, 16, true},
                         {d_token_gate, tokens, 4, true},
                         {d_channel_gate, 4 * (size_t)H, 16, true},
                         {workspace, workspace_bytes, 16, false}};
  if (workspace_bytes < moe_tail_block_norm_grad_workspace_bytes(b, H) || !operands_ok(in, out)) return MOE_TAIL_EINVAL;
  if (b == 0 && !d_post_gamma && !d_pre_gamma && !d_channel_gate) return MOE_TAIL_OK;
  moetail::BlockNormGradArgs a;
  a.d_y = static_cast<const uint16_t*>(d_y);
  a.d_residual_out = static_cast<const uint16_t*>(d_residual_out);
  a.x = static_cast<const uint16_t*>(x);
  a.residual = static_cast<const uint16_t*>(residual);
  a.post_gamma = static_cast<const uint16_t*>(post_gamma);
  a.pre_gamma = static_cast<const uint16_t*>(pre_gamma);
  a.token_gate = token_gate;
  a.channel_gate = static_cast<const uint16_t*>(channel_gate);
  a.rstd = rstd;
  a.residual_scale = residual_scale;
  a.gain_center = gain_center;
  a.rcpH = (float)(1.0 / (double)H);
  a.b = b;
  a.H = H;
  a.d_x = static_cast<uint16_t*>(d_x);
  a.d_residual = static_cast<uint16_t*>(d_residual);
  a.d_post_gamma = d_post_gamma;
  a.d_pre_gamma = d_pre_gamma;
  a.d_channel_gate = d_channel_gate;
  a.d_token_gate = d_token_gate;
  a.partial = static_cast<float*>(workspace);
  a.stage_wait_ns = moetail::stage_wait_limit_ns();
  return finish(moetail::launch_block_norm_grad(a, device_sms(), static_cast<cudaStream_t>(stream)));
}

// ============================================================================ routes

MOE_API size_t moe_tail_sort_workspace_bytes(int b, int K, int num_experts) {
  if (!routes_ok(b, K) || (int64_t)b * K > kMaxRoutes || num_experts < 1 || num_experts > kMaxExperts) return 0;
  return round256((size_t)4 * moetail::sort_blocks_up_to(b * K) * num_experts);
}

MOE_API int moe_tail_sort_routes(const int32_t* expert_ids, int b, int K, int num_experts, int32_t* expert_offsets,
                                 int32_t* permuted_idx, int32_t* source, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  if (!routes_ok(b, K) || (int64_t)b * K > kMaxRoutes || num_experts < 1 || num_experts > kMaxExperts)
    return MOE_TAIL_EINVAL;
  const size_t n = (size_t)b * K;
  const Operand in[] = {{expert_ids, 4 * n, 4, false}};
  const Operand out[] = {{expert_offsets, 4 * ((size_t)num_experts + 1), 4, false},
                         {permuted_idx, 4 * n, 4, false},
                         {source, 4 * n, 4, false},
                         {workspace, workspace_bytes, 16, false}};
  if (workspace_bytes < moe_tail_sort_workspace_bytes(b, K, num_experts) || !operands_ok(in, out))
    return MOE_TAIL_EINVAL;
  moetail::SortArgs a;
  a.ids = expert_ids;
  a.offsets = expert_offsets;
  a.permuted_idx = permuted_idx;
  a.source = source;
  a.counts = static_cast<int32_t*>(workspace);
  a.routes = (int)n;
  a.E = num_experts;
  return finish(moetail::launch_sort_routes(a, static_cast<cudaStream_t>(stream)));
}

MOE_API int moe_tail_dispatch_rows(const void* x, const void* scale, const int32_t* permuted_idx, int b, int K, int H,
                                   int elem_bytes, int64_t num_rows, void* rows, void* row_scale, void* stream) {
  if (!routes_ok(b, K) || !width_ok(H) || (elem_bytes != 1 && elem_bytes != 2)) return MOE_TAIL_EINVAL;
  if (num_rows < 0 || num_rows > kMaxRows || (scale != nullptr) != (row_scale != nullptr)) return MOE_TAIL_EINVAL;
  if (b == 0 || num_rows == 0) return MOE_TAIL_OK;
  const size_t row = (size_t)H * elem_bytes;
  const Operand in[] = {{x, b * row, 16, false}, {scale, 4 * (size_t)b, 4, true}, {permuted_idx, 4 * (size_t)b * K, 4, false}};
  const Operand out[] = {{rows, num_rows * row, 16, false}, {row_scale, 4 * (size_t)num_rows, 4, true}};
  if (!operands_ok(in, out)) return MOE_TAIL_EINVAL;
  moetail::DispatchArgs a;
  a.x = x;
  a.scale = static_cast<const float*>(scale);
  a.idx = permuted_idx;
  a.rows = rows;
  a.row_scale = static_cast<float*>(row_scale);
  a.num_rows = num_rows;
  a.b = b;
  a.K = K;
  a.row_bytes = (int)row;
  return finish(moetail::launch_dispatch_rows(a, static_cast<cudaStream_t>(stream)));
}

MOE_API int moe_tail_combine_rows(const void* rows, int64_t num_rows, const int32_t* permuted_idx,
                                  const void* route_weights, int weight_dtype, int b, int K, int H, void* out,
                                  void* stream) {
  if (!routes_ok(b, K) || !width_ok(H) || !weights_ok(weight_dtype)) return MOE_TAIL_EINVAL;
  if (num_rows < 0 || num_rows > kMaxRows) return MOE_TAIL_EINVAL;
  if (b == 0) return MOE_TAIL_OK;
  const size_t ws = weight_size(weight_dtype);
  const Operand in[] = {{rows, (size_t)num_rows * H * 2, 16, false},
                        {permuted_idx, 4 * (size_t)b * K, 4, false},
                        {route_weights, ws * b * K, ws, true}};
  const Operand outs[] = {{out, (size_t)b * H * 2, 16, false}};
  if (!operands_ok(in, outs)) return MOE_TAIL_EINVAL;
  moetail::CombineArgs a = {};
  a.rows = static_cast<const uint16_t*>(rows);
  a.idx = permuted_idx;
  a.w = route_weights;
  a.num_rows = num_rows;
  a.b = b;
  a.K = K;
  a.H = H;
  a.out = static_cast<uint16_t*>(out);
  const int wmode = !route_weights ? moetail::kWeightUnit
                    : weight_dtype == MOE_TAIL_W_BF16 ? moetail::kWeightBF16
                                                      : moetail::kWeightF32;
  return finish(moetail::launch_combine_rows(a, wmode, static_cast<cudaStream_t>(stream)));
}

MOE_API int moe_tail_combine_grad(const void* d_out, const void* rows, int64_t num_rows, const int32_t* permuted_idx,
                                  const void* route_weights, int weight_dtype, int b, int K, int H, void* d_rows,
                                  void* d_weights, void* stream) {
  if (!routes_ok(b, K) || !width_ok(H) || !weights_ok(weight_dtype)) return MOE_TAIL_EINVAL;
  if (num_rows < 0 || num_rows > kMaxRows) return MOE_TAIL_EINVAL;
  if (b == 0) return MOE_TAIL_OK;
  const size_t ws = weight_size(weight_dtype);
  const size_t bytes = (size_t)num_rows * H * 2;
  const Operand in[] = {{d_out, (size_t)b * H * 2, 16, false},
                        {rows, bytes, 16, false},
                        {permuted_idx, 4 * (size_t)b * K, 4, false},
                        {route_weights, ws * b * K, ws, false}};
  const Operand outs[] = {{d_rows, bytes, 16, false}, {d_weights, 4 * (size_t)b * K, 4, false}};
  if (!operands_ok(in, outs)) return MOE_TAIL_EINVAL;
  moetail::CombineArgs a = {};
  a.rows = static_cast<const uint16_t*>(rows);
  a.idx = permuted_idx;
  a.w = route_weights;
  a.num_rows = num_rows;
  a.b = b;
  a.K = K;
  a.H = H;
  a.d_out = static_cast<const uint16_t*>(d_out);
  a.d_rows = static_cast<uint16_t*>(d_rows);
  a.d_w = static_cast<float*>(d_weights);
  const int wmode = weight_dtype == MOE_TAIL_W_BF16 ? moetail::kWeightBF16 : moetail::kWeightF32;
  return finish(moetail::launch_combine_grad(a, wmode, static_cast<cudaStream_t>(stream)));
}

// ============================================================================ 8-bit product

namespace {

// int8 [E][N][D] read in boxes of 128 channels x 128 bytes, and FP16 [R][D] in boxes of box_rows x 64 (128 bytes
// each: the swizzle span); out-of-range parts of a box read zeros.
bool encode_product_maps(CUtensorMap* map_w, CUtensorMap* map_x, const void* w, const void* x16, int64_t R, int E, int N,
                         int D, int box_rows) {
  EncodeTiled enc = encoder();
  if (!enc) return false;
  const cuuint64_t wd[3] = {(cuuint64_t)D, (cuuint64_t)N, (cuuint64_t)E};
  const cuuint64_t wst[2] = {(cuuint64_t)D, (cuuint64_t)D * N};
  const cuuint32_t wb[3] = {128, 128, 1}, ones[3] = {1, 1, 1};
  const cuuint64_t xd[2] = {(cuuint64_t)D, (cuuint64_t)R};
  const cuuint64_t xst[1] = {(cuuint64_t)D * 2};
  const cuuint32_t xb[2] = {64, (cuuint32_t)box_rows};
  return enc(map_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(w), wd, wst, wb, ones,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS &&
         enc(map_x, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void*>(x16), xd, xst, xb, ones,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool product_sizes_ok(int64_t R, int E, int N, int D) {
  return R >= 0 && R <= kMaxRows && E >= 1 && E <= kMaxExperts && N >= 8 && N <= kMaxN && N % 8 == 0 && D >= 16 &&
         D <= kMaxD && D % 16 == 0;
}

}  // namespace

MOE_API size_t moe_tail_expert_product_workspace_bytes(int64_t rows, int num_experts, int N, int D) {
  if (!product_sizes_ok(rows, num_experts, N, D)) return 0;
  return round256(moetail::expert_product_workspace(rows, num_experts, N, D));
}

MOE_API int moe_tail_expert_product(const void* x, const void* x_scale, const void* w, const void* w_scale,
                                    const int32_t* expert_offsets, int64_t rows, int num_experts, int N, int D,
                                    void* out, void* workspace, size_t workspace_bytes, void* stream) {
  if (!product_sizes_ok(rows, num_experts, N, D)) return MOE_TAIL_EINVAL;
  if (!expert_offsets && num_experts != 1) return MOE_TAIL_EINVAL;
  if (rows == 0) return MOE_TAIL_OK;
  const Operand in[] = {{x, (size_t)rows * D, 16, false},
                        {x_scale, 4 * (size_t)rows, 4, false},
                        {w, (size_t)num_experts * N * D, 16, false},
                        {w_scale, 4 * (size_t)num_experts * N, 4, false},
                        {expert_offsets, 4 * ((size_t)num_experts + 1), 4, true}};
  const Operand outs[] = {{out, (size_t)rows * N * 2, 16, false}, {workspace, workspace_bytes, 256, false}};
  if (workspace_bytes < moe_tail_expert_product_workspace_bytes(rows, num_experts, N, D) || !operands_ok(in, outs))
    return MOE_TAIL_EINVAL;
  moetail::ProductArgs a;
  a.x = static_cast<const int8_t*>(x);
  a.x_scale = static_cast<const float*>(x_scale);
  a.w = static_cast<const int8_t*>(w);
  a.w_scale = static_cast<const float*>(w_scale);
  a.offsets = expert_offsets;
  a.R = rows;
  a.E = num_experts;
  a.N = N;
  a.D = D;
  a.out = static_cast<uint16_t*>(out);
  const int tile = moetail::product_rows_of_tile(rows, num_experts);
  CUtensorMap map_w, map_x;
  if (!encode_product_maps(&map_w, &map_x, w, workspace, rows, num_experts, N, D, tile < 64 ? tile : 64))
    return MOE_TAIL_ECUDA;
  return finish(
      moetail::launch_expert_product(a, map_w, map_x, workspace, device_sms(), static_cast<cudaStream_t>(stream)));
}

// ============================================================================ 4-bit product

namespace {

bool i4_sizes_ok(int64_t R, int E, int N, int D, int group) {
  return R >= 0 && R <= kMaxRows && E >= 1 && E <= kMaxExperts && N >= 8 && N <= kMaxN && N % 8 == 0 && D >= 8 &&
         D <= kMaxD && D % 8 == 0 && (group == 32 || group == 64 || group == 128);
}

bool encode_i4_maps(CUtensorMap* map_w, CUtensorMap* map_x, const void* w, const void* x, int64_t R, int E, int N, int D,
                    bool gated, const moetail::ProductI4Plan& plan) {
  EncodeTiled enc = encoder();
  if (!enc) return false;
  const cuuint64_t bytes = 64 * (cuuint64_t)((D + 127) / 128), element = plan.tiles ? 1 : 4, columns = bytes / element;
  const cuuint64_t channels = (cuuint64_t)N, experts = (cuuint64_t)E;
  const cuuint32_t box = (cuuint32_t)plan.box_channels, ones[4] = {1, 1, 1, 1};
  const cuuint64_t wd3[3] = {columns, channels, experts}, wst3[2] = {bytes, bytes * channels};
  const cuuint64_t wd4[4] = {columns, channels, 2, experts}, wst4[3] = {bytes, bytes * channels, 2 * bytes * channels};
  const cuuint32_t width = (cuuint32_t)(plan.box_columns / element);
  const cuuint32_t wb3[3] = {width, box, 1}, wb4[4] = {width, box, 2, 1};
  const cuuint64_t row = (cuuint64_t)D * 2;
  const cuuint64_t xd2[2] = {(cuuint64_t)D, (cuuint64_t)R}, xst2[1] = {row};
  const cuuint64_t xd3[3] = {64, (cuuint64_t)R, (cuuint64_t)(D / 64)}, xst3[2] = {row, 128};
  const cuuint32_t xb2[2] = {64, (cuuint32_t)plan.box_rows};
  const cuuint32_t xb3[3] = {64, (cuuint32_t)plan.box_rows, (cuuint32_t)plan.box_chunks};
  const bool chunks = plan.box_chunks > 0;
  return enc(map_w, plan.tiles ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT32, gated ? 4 : 3,
             const_cast<void*>(w), gated ? wd4 : wd3,
             gated ? wst4 : wst3, gated ? wb4 : wb3, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
             plan.tiles ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS &&
         enc(map_x, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, chunks ? 3 : 2, const_cast<void*>(x), chunks ? xd3 : xd2,
             chunks ? xst3 : xst2, chunks ? xb3 : xb2, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int product_i4(const void* x, const void* w, const void* group_scale, const float* channel_scale,
               const int32_t* expert_offsets, int64_t rows, int num_experts, int N, int D, int group, bool gated, void* out,
               void* stream) {
  if (!i4_sizes_ok(rows, num_experts, N, D, group) || (!expert_offsets && num_experts != 1)) return MOE_TAIL_EINVAL;
  if (rows == 0) return MOE_TAIL_OK;
  const size_t channels = (size_t)num_experts * N * (gated ? 2 : 1), pitch = ((D + group - 1) / group + 3) / 4 * 4;
  const Operand in[] = {{x, (size_t)rows * D * 2, 16, false},
                        {w, channels * 64 * ((D + 127) / 128), 16, false},
                        {group_scale, channels * pitch, 4, false},
                        {channel_scale, 4 * channels, 4, false},
                        {expert_offsets, 4 * ((size_t)num_experts + 1), 4, true}};
  const Operand outs[] = {{out, (size_t)rows * N * 2, 16, false}};
  if (!operands_ok(in, outs)) return MOE_TAIL_EINVAL;
  moetail::ProductI4Args a;
  a.group_scale = static_cast<const uint8_t*>(group_scale);
  a.channel_scale = channel_scale;
  a.offsets = expert_offsets;
  a.out = static_cast<uint16_t*>(out);
  a.R = rows;
  a.E = num_experts;
  a.N = N;
  a.D = D;
  a.group = group;
  a.gated = gated;
  const moetail::ProductI4Plan plan = moetail::product_i4_plan(rows, num_experts, N, D, gated, device_sms());
  CUtensorMap map_w, map_x;
  if (!encode_i4_maps(&map_w, &map_x, w, x, rows, num_experts, N, D, gated, plan)) return MOE_TAIL_ECUDA;
  return finish(moetail::launch_product_i4(a, plan, map_w, map_x, device_sms(), static_cast<cudaStream_t>(stream)));
}

}  // namespace

MOE_API int moe_tail_expert_product_i4(const void* x, const void* w, const void* group_scale, const float* channel_scale,
                                       const int32_t* expert_offsets, int64_t rows, int num_experts, int N, int D,
                                       int group, void* out, void* stream) {
  return product_i4(x, w, group_scale, channel_scale, expert_offsets, rows, num_experts, N, D, group, false, out, stream);
}

MOE_API int moe_tail_gated_product_i4(const void* x, const void* w, const void* group_scale, const float* channel_scale,
                                      const int32_t* expert_offsets, int64_t rows, int num_experts, int I, int D, int group,
                                      void* out, void* stream) {
  return product_i4(x, w, group_scale, channel_scale, expert_offsets, rows, num_experts, I, D, group, true, out, stream);
}

MOE_API int moe_tail_product_i4_tile_rows(int64_t rows, int num_experts, int N, int D, int gated) {
  if (!i4_sizes_ok(rows, num_experts, N, D, 128)) return 0;
  return moetail::product_i4_plan(rows, num_experts, N, D, gated != 0, device_sms()).rows;
}
