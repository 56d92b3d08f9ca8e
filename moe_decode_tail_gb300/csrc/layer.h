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

}  // namespace moetail
