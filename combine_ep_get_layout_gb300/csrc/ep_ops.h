// Host-side internals of the operators around the path (router, experts'
// products, low-rank adapters): the checked arguments each launcher takes.
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

}  // namespace ep
