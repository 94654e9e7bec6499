// Launchers of the block operators: routing with groups, combine gradient, block
// norms, linear layer.
#pragma once

#include "common.cuh"
#include "linear_epilogue.cuh"

namespace moe {

// Choice-only bias, expert groups (route.cu). logits may hold n_parts partial
// sums, part_stride elements apart; logits_out (nullable) receives their sum.
cudaError_t launch_route(const moe_route_desc& d, const float* logits, int n_parts,
                         size_t part_stride, const float* bias, int32_t* idx, float* w,
                         float* logits_out, cudaStream_t st);
cudaError_t launch_route_backward(const moe_route_desc& d, const float* logits,
                                  const int32_t* idx, const float* d_w, float* d_logits,
                                  cudaStream_t st);
cudaError_t launch_combine_backward(const moe_layer_desc& d, const void* dy, const float* y_rows,
                                    const float* w, const int32_t* inv, void* d_rows, float* d_w,
                                    cudaStream_t st);
// Norms around a block (block_norm.cu); null pointers leave their part out.
cudaError_t launch_block_norm(const moe_norm_desc& d, const void* h, const void* y,
                              const void* w_post, const void* gate, const void* w_pre,
                              void* h_out, void* x, int sms, cudaStream_t st);
// Blocks of the backward pass on `sms` SMs; parts holds [blocks, 3, H] fp32.
int block_norm_backward_grid(const moe_norm_desc& d, int sms);
cudaError_t launch_block_norm_backward(const moe_norm_desc& d, const void* d_h_out,
                                       const void* d_x, const void* h_out, const void* y,
                                       const void* w_post, const void* gate, const void* w_pre,
                                       void* d_h, void* d_y, float* d_w_post, void* d_gate,
                                       float* d_w_pre, float* parts, int sms, cudaStream_t st);
// out[i][c] = sum over n_blocks rows of parts [n_blocks, n_out, H], in a fixed order.
struct ColumnSums {
  float* out[3];
};
cudaError_t launch_column_sums(const float* parts, int n_blocks, int n_out, int H,
                               const ColumnSums& o, cudaStream_t st);
// Linear layer (linear.cu, linear_tc.cu). SMs that the plans reckon with: a
// constant, so that the workspace size depends on the shape alone.
constexpr int kPlanSms = 148;
constexpr int kMaxSharedTiles = kPlanSms;   // shared tiles of a product, at most
struct LinearPlan {
  bool pair;
  int bn, m_tiles, n_tiles, k_stages, units, whole, parts, a_rows, a_bytes, stage_bytes, n_stages;
  size_t partial_bytes;
};
LinearPlan linear_plan(int M, int N, int K, bool a_mn, bool b_mn, int sms);
// C [M, N] = A B^T: a_mn / b_mn say that an operand is stored [K, M] / [K, N].
cudaError_t launch_linear_tc(const LinearPlan& p, int M, int N, int K, const void* A, bool a_mn,
                             const void* B, bool b_mn, const LinearEpilogue& epi,
                             float* partials, int* arrivals, uint32_t* status,
                             cudaStream_t st);
// A few tokens at a time: W streamed through CUDA cores (linear_few.cu).
bool linear_few_tokens(const moe_linear_desc& d);
cudaError_t launch_linear_few(const moe_linear_desc& d, const void* x, const void* w,
                              const LinearEpilogue& epi, cudaStream_t st);
cudaError_t launch_linear_simt(int M, int N, int K, const float* A, bool a_mn, const float* B,
                               bool b_mn, const LinearEpilogue& epi, cudaStream_t st);
// dz = dy * act'(pre) (dz null: not stored) and its column sums, one row of
// sums for each kGradRows rows (parts null: none).
constexpr int kGradRows = 64;
cudaError_t launch_linear_act_grad(const moe_linear_desc& d, const void* dy, const void* pre,
                                   void* dz, float* parts, cudaStream_t st);

}  // namespace moe
