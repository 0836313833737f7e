// Host-side internals of the operators around the path (router, experts'
// products, low-rank adapters; balance loss, layer norm, shared product): the
// checked arguments each launcher takes.
// Not part of the public interface.
#pragma once

#include "ep_internal.h"

namespace ep {

// ---- router (ep_route.cu)
struct RouteArgs {
  const void *logits;
  bool bf16;
  int64_t row_stride;  // elements between rows
  int num_tokens, num_experts, num_topk;
  bool sigmoid;
  const float *bias;  // [E] or null
  int num_groups, topk_groups, group_top;
  bool renormalize;
  float weight_scale;
  int64_t *topk_idx;
  float *topk_weights;
};
ep_status_t launch_route(const RouteArgs &a, cudaStream_t stream);

struct RouteBackwardArgs {
  const float *grad_weights;
  const void *logits;
  bool bf16;
  int64_t row_stride;
  const int64_t *topk_idx;
  int num_tokens, num_experts, num_topk;
  bool sigmoid, renormalize;
  float weight_scale;
  void *grad_logits;  // logits' type, rows E apart
};
ep_status_t launch_route_backward(const RouteBackwardArgs &a, cudaStream_t stream);

// ---- experts' products (ep_product.cu)
struct ProductArgs {
  const uint16_t *x;  // [cap, hidden]
  int recv_capacity, num_tokens, hidden, num_experts;
  const int32_t *num_rows_per_expert, *expert_offset;
  uint32_t *error_word;
  const uint16_t *w;  // [E, wide, hidden], wide = gated ? 2 * width : width
  int width;
  bool gated;
  uint16_t *out;     // [cap, width]
  uint16_t *preact;  // [cap, wide] or null
};
ep_status_t launch_product(const ProductArgs &a, cudaStream_t stream);

struct ProductBackwardArgs {
  const uint16_t *grad;  // [cap, width]
  const uint16_t *x, *w;
  int recv_capacity, num_tokens, hidden, num_experts;
  const int32_t *num_rows_per_expert, *expert_offset;
  uint32_t *error_word;
  int width;
  bool gated;
  const uint16_t *preact;  // [cap, 2 * width] (gated)
  uint16_t *grad_preact;   // [cap, 2 * width] (gated): written, then read
  uint16_t *grad_x;        // [cap, hidden] or null
  uint16_t *grad_w;        // [E, wide, hidden] or null
};
ep_status_t launch_product_backward(const ProductBackwardArgs &a, cudaStream_t stream);

// ---- low-rank adapters (ep_adapter.cu)
size_t adapter_workspace_bytes(int num_rows, int hidden, int rank);
struct AdapterArgs {
  const uint16_t *x;  // [T, hidden]
  int num_rows, hidden;
  const uint16_t *w;  // [width, hidden]
  int width;
  const uint16_t *lora_a;  // [A, rank, hidden]
  const uint16_t *lora_b;  // [A, width, rank]
  int num_adapters, rank;
  const int64_t *adapter_idx;  // [T]
  const float *adapter_scale;  // [A] or null
  uint16_t *out;               // [T, width]
  void *workspace;
  uint32_t *error_word;  // or null
};
ep_status_t launch_adapter(const AdapterArgs &a, cudaStream_t stream);

// ---- balance loss (ep_balance.cu)
size_t balance_workspace_bytes(int num_tokens, int num_experts, int num_sequences);
struct BalanceArgs {
  const void *logits;
  bool bf16;
  int64_t row_stride;
  const int64_t *topk_idx;
  int num_tokens, num_experts, num_topk;
  bool sigmoid;
  const int32_t *seq_offsets;  // [S + 1] or null: one sequence
  int num_sequences;
  float *losses;
  int32_t *counts;
  float *probs, *slopes;
  void *workspace;
};
ep_status_t launch_balance(const BalanceArgs &a, cudaStream_t stream);

struct BalanceBackwardArgs {
  const float *grad_losses;
  const void *logits;
  bool bf16;
  int64_t row_stride;
  int num_tokens, num_experts;
  bool sigmoid;
  const int32_t *seq_offsets;
  int num_sequences;
  const float *slopes;
  const void *add;    // logits' type, rows E apart, or null
  void *grad_logits;  // the same
};
ep_status_t launch_balance_backward(const BalanceBackwardArgs &a, cudaStream_t stream);

// ---- layer norm (ep_norm.cu)
struct NormArgs {
  const void *x;
  bool bf16;
  int64_t row_stride;
  int num_rows, hidden;
  const void *weight, *bias;  // or null
  bool param_bf16;
  float eps;
  void *out;
  float *mean, *rstd;  // or null
};
ep_status_t launch_norm(const NormArgs &a, cudaStream_t stream);

size_t norm_workspace_bytes(int num_rows, int hidden);
struct NormBackwardArgs {
  const void *grad, *x;
  bool bf16;
  int64_t row_stride;  // of x
  int num_rows, hidden;
  const float *mean, *rstd;
  const void *weight;  // or null
  bool param_bf16;
  const void *add;                         // or null
  void *grad_x, *grad_weight, *grad_bias;  // or null
  float *workspace;
};
ep_status_t launch_norm_backward(const NormBackwardArgs &a, cudaStream_t stream);

// ---- product shared by all rows (ep_dense.cu)
struct DenseArgs {
  const uint16_t *x;
  int64_t row_stride;
  int num_rows, hidden;
  const uint16_t *w;  // [wide, hidden], wide = width, or 2 * width (EP_ACT_SWIGLU)
  int width;
  const void *bias;  // [wide] or null
  bool bias_bf16;
  ep_activation_t activation;
  const uint16_t *residual;  // [T, width] or null
  void *out;
  bool out_bf16;
  uint16_t *preact;  // [T, wide] or null
  uint32_t *error_word;
};
ep_status_t launch_dense(const DenseArgs &a, cudaStream_t stream);

size_t dense_workspace_bytes(int num_rows, int hidden, int width, ep_activation_t activation);
struct DenseBackwardArgs {
  const void *grad;
  bool grad_bf16;
  const uint16_t *x;
  int64_t row_stride;
  int num_rows, hidden;
  const uint16_t *w;
  int width;
  ep_activation_t activation;
  const uint16_t *preact;
  uint16_t *grad_preact, *grad_x, *grad_w;  // grad_x, grad_w or null
  void *grad_bias;                          // or null
  bool bias_bf16;
  void *workspace;
  uint32_t *error_word;
};
ep_status_t launch_dense_backward(const DenseBackwardArgs &a, cudaStream_t stream);

}  // namespace ep
