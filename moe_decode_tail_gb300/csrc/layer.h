// Internal interface between the C ABI of the operators around the tail and their kernels (not exported).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <utility>

namespace moetail {

constexpr int kMaxExperts = 1024;

// Launch with programmatic dependent launch: the kernel touches no global memory that another kernel
// writes before griddepcontrol.wait, and every thread block executes that wait.
template <typename... Params, typename... Args>
cudaError_t launch_pdl(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                       Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// ---- 8-bit rows (row_quant.cu) -------------------------------------------------

enum { kQuantInt8 = 0, kQuantE4M3 = 1 };
constexpr int kQuantGroup = 128;  // columns of a group where a row has several scales

struct NormQuantArgs {
  const uint16_t* x;         // BF16 [b][H]
  const uint16_t* residual;  // BF16 [b][H] or null
  const uint16_t* gamma;     // BF16 [H]
  float gain_center, eps, rcpH;
  int b, H;
  uint16_t* residual_out;    // BF16 [b][H] or null (may be x or residual)
  uint16_t* y;               // BF16 [b][H] or null
  uint8_t* q;                // [b][H]
  float* scale;              // [b] or [b][groups]
  int groups;                // scales of a row
};
cudaError_t launch_norm_quant(const NormQuantArgs& a, int kind, bool grouped, int sms, cudaStream_t stream);

struct SiluQuantArgs {
  const uint16_t* gate_up;  // BF16 [rows][2 I]
  const int32_t* used;      // rows in use (device), or null: all
  int64_t rows;
  int I;
  uint8_t* q;
  float* scale;
  int groups;
};
cudaError_t launch_silu_quant(const SiluQuantArgs& a, int kind, bool grouped, int sms, cudaStream_t stream);

// ---- norms around a block (block_norm.cu) ----------------------------------------

struct BlockNormArgs {
  const uint16_t* x;             // BF16 [b][H]
  const uint16_t* residual;      // BF16 [b][H]
  const uint16_t* post_gamma;    // BF16 [H] or null: no norm after the block
  const uint16_t* pre_gamma;     // BF16 [H]
  const float* token_gate;       // [b] or null
  const uint16_t* channel_gate;  // BF16 [H] or null
  float residual_scale, gain_center, eps, rcpH;
  int b, H;
  uint16_t* residual_out;        // BF16 [b][H] (may be x or residual)
  uint16_t* y;                   // BF16 [b][H]
  float* rstd;                   // [b][2] or null
};
cudaError_t launch_block_norm(const BlockNormArgs& a, int sms, cudaStream_t stream);

struct BlockNormGradArgs {
  const uint16_t *d_y, *d_residual_out;  // BF16 [b][H]; d_residual_out may be null
  const uint16_t *x, *residual, *post_gamma, *pre_gamma;
  const float* token_gate;
  const uint16_t* channel_gate;
  const float* rstd;
  float residual_scale, gain_center, rcpH;
  int b, H;
  uint16_t *d_x, *d_residual;            // BF16 [b][H] (may be d_y and d_residual_out)
  float *d_post_gamma, *d_pre_gamma, *d_channel_gate;  // [H] or null
  float* d_token_gate;                   // [b] or null
  float* partial;                        // workspace [row sets][3][H]
  unsigned long long stage_wait_ns;      // of moe_tail_set_stage_wait_limit, 0: the default
};
cudaError_t launch_block_norm_grad(const BlockNormGradArgs& a, int sms, cudaStream_t stream);
size_t block_norm_grad_workspace(int b, int H);
cudaError_t take_block_norm_error(unsigned* bits);

// ---- routes (routes.cu) ----------------------------------------------------------

int sort_blocks(int routes);  // thread blocks of a sort, each with a row of counts in the workspace
// The most of any sort of so many routes or fewer: sort_blocks falls from 128 to 33 where a lane takes four times as many.
int sort_blocks_up_to(int routes);

struct SortArgs {
  const int32_t* ids;     // [routes]
  int32_t* offsets;       // [E + 1]
  int32_t* permuted_idx;  // [routes]
  int32_t* source;        // [routes]
  int32_t* counts;        // workspace [blocks][E] (more than one block)
  int routes, E;
};
cudaError_t launch_sort_routes(const SortArgs& a, cudaStream_t stream);

struct DispatchArgs {
  const void* x;             // [b][row_bytes]
  const float* scale;        // [b] or null
  const int32_t* idx;        // [b][K]
  void* rows;                // [num_rows][row_bytes]
  float* row_scale;          // [num_rows] or null
  int64_t num_rows;
  int b, K, row_bytes;
};
cudaError_t launch_dispatch_rows(const DispatchArgs& a, cudaStream_t stream);

struct CombineArgs {
  const uint16_t* rows;   // BF16 [num_rows][H]
  const int32_t* idx;     // [b][K]
  const void* w;          // [b][K] or null (unit weights)
  int64_t num_rows;
  int b, K, H;
  uint16_t* out;          // combine: BF16 [b][H]
  const uint16_t* d_out;  // gradient: BF16 [b][H]
  uint16_t* d_rows;       // gradient: BF16 [num_rows][H]
  float* d_w;             // gradient: [b][K]
};
cudaError_t launch_combine_rows(const CombineArgs& a, int wmode, cudaStream_t stream);
cudaError_t launch_combine_grad(const CombineArgs& a, int wmode, cudaStream_t stream);

// ---- 8-bit product (expert_product.cu) -------------------------------------------

struct ProductArgs {
  const int8_t* x;         // [R][D]
  const float* x_scale;    // [R]
  const int8_t* w;         // [E][N][D]
  const float* w_scale;    // [E][N]
  const int32_t* offsets;  // [E + 1] or null (E = 1: all rows)
  int64_t R;
  int E, N, D;
  uint16_t* out;           // BF16 [R][N]
};
// map_w: w as [E][N][D] bytes, boxes of 128 channels x 128 bytes; map_x: the FP16 rows at the workspace's start,
// [R][D], boxes of min(product_rows_of_tile, 64) rows x 64; both with the 128-byte swizzle, zeros out of range.
cudaError_t launch_expert_product(const ProductArgs& a, const CUtensorMap& map_w, const CUtensorMap& map_x,
                                  void* workspace, int sms, cudaStream_t stream);
size_t expert_product_workspace(int64_t R, int E, int N, int D);
int product_rows_of_tile(int64_t R, int E);
// Read and clear the product's device error word (synchronises).
cudaError_t take_product_error(unsigned* bits);

// ---- 4-bit product (product_i4.cu) -----------------------------------------------

struct ProductI4Args {
  const uint8_t* group_scale;  // e4m3 [E][channels][pitch]; channels: N, gated 2 N
  const float* channel_scale;  // [E][channels]
  const int32_t* offsets;      // [E + 1] or null (E = 1: all rows)
  uint16_t* out;               // BF16 [R][N]
  int64_t R;
  int E, N, D, group;
  bool gated;
};
// Which kernel a call takes and how its operands are read.
struct ProductI4Plan {
  bool tiles, wide;  // tiles on the tensor cores (product_i4_tiles.cu); else warps that multiply (product_i4.cu)
  int rows;          // of a tile
  int box_columns;   // bytes of a channel in a box of w
  int box_channels;  // of one half of a gated weight, or of a plain one, in a box of w
  int box_rows;      // in a box of x
  int box_chunks;    // of 64 columns in a box of x, or 0: x is read as two dimensions
};
ProductI4Plan product_i4_plan(int64_t R, int E, int N, int D, bool gated, int sms);
// map_w: w as [E][channels][64 ceil(D / 128)] bytes, gated as [E][2][N][...], in boxes of (2 x) box_channels x box_columns
// bytes; with tiles in bytes with the 128-byte swizzle, else in words of four bytes without one.  map_x: x as [R][D] in boxes
// of box_rows x 64, or as [D / 64][R][64] in boxes of box_chunks x box_rows x 64, with the 128-byte swizzle.  Zeros out of
// range.
cudaError_t launch_product_i4(const ProductI4Args& p, const ProductI4Plan& plan, const CUtensorMap& map_w,
                              const CUtensorMap& map_x, int sms, cudaStream_t stream);
cudaError_t launch_product_i4_tiles(const ProductI4Args& p, const ProductI4Plan& plan, const CUtensorMap& map_w,
                                    const CUtensorMap& map_x, int sms, cudaStream_t stream);
cudaError_t take_product_i4_tiles_error(unsigned* bits);
cudaError_t take_product_i4_error(unsigned* bits);

}  // namespace moetail
