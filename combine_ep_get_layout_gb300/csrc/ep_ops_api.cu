// The C ABI of the operators around the path (router, experts' products,
// low-rank adapters): argument checks on the host, before any CUDA call.
#include "ep_ops.h"

using namespace ep;

#define EP_CHECK(expr)             \
  do {                             \
    const ep_status_t _s = (expr); \
    if (_s != EP_OK) return _s;    \
  } while (0)

namespace {

// A size that has to be a multiple of 8 in [8, most].
ep_status_t check_eights(const char *fn, const char *name, int v, int most) {
  if (v < 8) return fail(EP_ERR_INVALID_ARG, "%s: %s=%d < 8", fn, name, v);
  if (v > most) return fail(EP_ERR_UNSUPPORTED, "%s: %s=%d > %d", fn, name, v, most);
  if (v % 8 != 0) return fail(EP_ERR_INVALID_ARG, "%s: %s=%d is not a multiple of 8", fn, name, v);
  return EP_OK;
}

ep_status_t check_route_sizes(const char *fn, int T, int E, int K, int score, int type, int64_t stride) {
  if (T < 0) return fail(EP_ERR_INVALID_ARG, "%s: num_tokens=%d < 0", fn, T);
  if (E < 1) return fail(EP_ERR_INVALID_ARG, "%s: num_experts=%d < 1", fn, E);
  if (E > EP_MAX_EXPERTS) return fail(EP_ERR_UNSUPPORTED, "%s: num_experts=%d > %d", fn, E, EP_MAX_EXPERTS);
  if (K < 1 || K > E) return fail(EP_ERR_INVALID_ARG, "%s: num_topk=%d not in [1, num_experts=%d]", fn, K, E);
  if (K > EP_MAX_TOPK) return fail(EP_ERR_UNSUPPORTED, "%s: num_topk=%d > %d", fn, K, EP_MAX_TOPK);
  if (score != EP_SCORE_SOFTMAX && score != EP_SCORE_SIGMOID)
    return fail(EP_ERR_INVALID_ARG, "%s: unknown score %d", fn, score);
  if (type != EP_LOGITS_FP32 && type != EP_LOGITS_BF16)
    return fail(EP_ERR_INVALID_ARG, "%s: unknown logits_type %d", fn, type);
  if (stride < E)
    return fail(EP_ERR_INVALID_ARG, "%s: row_stride=%lld < num_experts=%d", fn, (long long)stride, E);
  return EP_OK;
}

ep_status_t check_product(const char *fn, int cap, int T, int E, int hidden, int width, int act,
                          const ep_expanded_layout_t *layout) {
  if (cap < 0) return fail(EP_ERR_INVALID_ARG, "%s: recv_capacity=%d < 0", fn, cap);
  if (T < 0) return fail(EP_ERR_INVALID_ARG, "%s: num_tokens=%d < 0", fn, T);
  if (E < 1) return fail(EP_ERR_INVALID_ARG, "%s: num_experts=%d < 1", fn, E);
  if (E > EP_MAX_EXPERTS) return fail(EP_ERR_UNSUPPORTED, "%s: num_experts=%d > %d", fn, E, EP_MAX_EXPERTS);
  EP_CHECK(check_eights(fn, "hidden", hidden, EP_MAX_HIDDEN));
  EP_CHECK(check_eights(fn, "width", width, EP_MAX_HIDDEN));
  if (act != EP_ACT_NONE && act != EP_ACT_SWIGLU)
    return fail(EP_ERR_INVALID_ARG, "%s: unknown activation %d", fn, act);
  if (layout == nullptr) return fail(EP_ERR_INVALID_ARG, "%s: layout is NULL", fn);
  EP_CHECK(check_ptr(fn, "layout.num_rows_per_expert", layout->num_rows_per_expert, 4, true));
  EP_CHECK(check_ptr(fn, "layout.expert_offset", layout->expert_offset, 4, true));
  EP_CHECK(check_ptr(fn, "layout.error_word", layout->error_word, 4, true));
  return EP_OK;
}

}  // namespace

extern "C" {

ep_status_t ep_route(const ep_route_args_t *args, ep_stream_t stream) {
  static const char *fn = "ep_route";
  clear_error();
  if (args == nullptr) return fail(EP_ERR_INVALID_ARG, "%s: args is NULL", fn);
  const ep_route_args_t &x = *args;
  EP_CHECK(check_route_sizes(fn, x.num_tokens, x.num_experts, x.num_topk, x.score, x.logits_type, x.row_stride));
  if (x.num_groups < 1) return fail(EP_ERR_INVALID_ARG, "%s: num_groups=%d < 1", fn, x.num_groups);
  if (x.num_groups > EP_MAX_RANKS)
    return fail(EP_ERR_UNSUPPORTED, "%s: num_groups=%d > %d", fn, x.num_groups, EP_MAX_RANKS);
  if (x.num_experts % x.num_groups != 0)
    return fail(EP_ERR_INVALID_ARG, "%s: num_experts=%d is not a multiple of num_groups=%d", fn, x.num_experts,
                x.num_groups);
  if (x.topk_groups < 1 || x.topk_groups > x.num_groups)
    return fail(EP_ERR_INVALID_ARG, "%s: topk_groups=%d not in [1, num_groups=%d]", fn, x.topk_groups, x.num_groups);
  if (x.group_top < 1 || x.group_top > 2)
    return fail(EP_ERR_INVALID_ARG, "%s: group_top=%d is not 1 or 2", fn, x.group_top);
  const bool any = x.num_tokens > 0;
  const bool bf16 = x.logits_type == EP_LOGITS_BF16;
  EP_CHECK(check_ptr(fn, "logits", x.logits, bf16 ? 2 : 4, any));
  EP_CHECK(check_ptr(fn, "bias", x.bias, 4, false));
  EP_CHECK(check_ptr(fn, "topk_idx", x.topk_idx, 8, any));
  EP_CHECK(check_ptr(fn, "topk_weights", x.topk_weights, 4, any));
  const RouteArgs a{x.logits,     bf16,          x.row_stride, x.num_tokens,       x.num_experts,
                    x.num_topk,   x.score == EP_SCORE_SIGMOID, x.bias, x.num_groups, x.topk_groups,
                    x.group_top,  x.renormalize != 0, x.weight_scale, x.topk_idx, x.topk_weights};
  return launch_route(a, reinterpret_cast<cudaStream_t>(stream));
}

ep_status_t ep_route_backward(const ep_route_backward_args_t *args, ep_stream_t stream) {
  static const char *fn = "ep_route_backward";
  clear_error();
  if (args == nullptr) return fail(EP_ERR_INVALID_ARG, "%s: args is NULL", fn);
  const ep_route_backward_args_t &x = *args;
  EP_CHECK(check_route_sizes(fn, x.num_tokens, x.num_experts, x.num_topk, x.score, x.logits_type, x.row_stride));
  const bool any = x.num_tokens > 0;
  const bool bf16 = x.logits_type == EP_LOGITS_BF16;
  EP_CHECK(check_ptr(fn, "grad_weights", x.grad_weights, 4, any));
  EP_CHECK(check_ptr(fn, "logits", x.logits, bf16 ? 2 : 4, any));
  EP_CHECK(check_ptr(fn, "topk_idx", x.topk_idx, 8, any));
  EP_CHECK(check_ptr(fn, "grad_logits", x.grad_logits, bf16 ? 2 : 4, any));
  const RouteBackwardArgs a{x.grad_weights, x.logits,   bf16,       x.row_stride,
                            x.topk_idx,     x.num_tokens, x.num_experts, x.num_topk,
                            x.score == EP_SCORE_SIGMOID, x.renormalize != 0, x.weight_scale, x.grad_logits};
  return launch_route_backward(a, reinterpret_cast<cudaStream_t>(stream));
}

ep_status_t ep_expert_product(const ep_expert_product_args_t *args, ep_stream_t stream) {
  static const char *fn = "ep_expert_product";
  clear_error();
  if (args == nullptr) return fail(EP_ERR_INVALID_ARG, "%s: args is NULL", fn);
  const ep_expert_product_args_t &x = *args;
  EP_CHECK(check_product(fn, x.recv_capacity, x.num_tokens, x.num_experts, x.hidden, x.width, x.activation, x.layout));
  const bool any = x.recv_capacity > 0 && x.num_tokens > 0;
  EP_CHECK(check_ptr(fn, "x", x.x, 16, any));
  EP_CHECK(check_ptr(fn, "w", x.w, 16, true));
  EP_CHECK(check_ptr(fn, "out", x.out, 16, any));
  EP_CHECK(check_ptr(fn, "preact", x.preact, 16, false));
  const ProductArgs a{static_cast<const uint16_t *>(x.x), x.recv_capacity, x.num_tokens, x.hidden, x.num_experts,
                      x.layout->num_rows_per_expert, x.layout->expert_offset, x.layout->error_word,
                      static_cast<const uint16_t *>(x.w), x.width, x.activation == EP_ACT_SWIGLU,
                      static_cast<uint16_t *>(x.out), static_cast<uint16_t *>(x.preact)};
  return launch_product(a, reinterpret_cast<cudaStream_t>(stream));
}

ep_status_t ep_expert_product_backward(const ep_expert_product_backward_args_t *args, ep_stream_t stream) {
  static const char *fn = "ep_expert_product_backward";
  clear_error();
  if (args == nullptr) return fail(EP_ERR_INVALID_ARG, "%s: args is NULL", fn);
  const ep_expert_product_backward_args_t &x = *args;
  EP_CHECK(check_product(fn, x.recv_capacity, x.num_tokens, x.num_experts, x.hidden, x.width, x.activation, x.layout));
  const bool any = x.recv_capacity > 0 && x.num_tokens > 0;
  const bool gated = x.activation == EP_ACT_SWIGLU;
  EP_CHECK(check_ptr(fn, "grad", x.grad, 16, any));
  EP_CHECK(check_ptr(fn, "x", x.x, 16, any && x.grad_w != nullptr));
  EP_CHECK(check_ptr(fn, "w", x.w, 16, x.grad_x != nullptr));
  EP_CHECK(check_ptr(fn, "preact", x.preact, 16, any && gated));
  EP_CHECK(check_ptr(fn, "grad_preact", x.grad_preact, 16, any && gated));
  EP_CHECK(check_ptr(fn, "grad_x", x.grad_x, 16, false));
  EP_CHECK(check_ptr(fn, "grad_w", x.grad_w, 16, false));
  const ProductBackwardArgs a{static_cast<const uint16_t *>(x.grad), static_cast<const uint16_t *>(x.x),
                              static_cast<const uint16_t *>(x.w), x.recv_capacity, x.num_tokens, x.hidden,
                              x.num_experts, x.layout->num_rows_per_expert, x.layout->expert_offset,
                              x.layout->error_word, x.width, gated, static_cast<const uint16_t *>(x.preact),
                              static_cast<uint16_t *>(x.grad_preact), static_cast<uint16_t *>(x.grad_x),
                              static_cast<uint16_t *>(x.grad_w)};
  return launch_product_backward(a, reinterpret_cast<cudaStream_t>(stream));
}

size_t ep_adapter_workspace_bytes(int num_rows, int hidden, int rank) {
  if (num_rows < 0 || hidden < 8 || hidden > EP_MAX_HIDDEN || rank < 8 || rank > EP_MAX_RANK) return 0;
  return adapter_workspace_bytes(num_rows, hidden, rank);
}

ep_status_t ep_adapter_product(const ep_adapter_product_args_t *args, ep_stream_t stream) {
  static const char *fn = "ep_adapter_product";
  clear_error();
  if (args == nullptr) return fail(EP_ERR_INVALID_ARG, "%s: args is NULL", fn);
  const ep_adapter_product_args_t &x = *args;
  if (x.num_rows < 0) return fail(EP_ERR_INVALID_ARG, "%s: num_rows=%d < 0", fn, x.num_rows);
  EP_CHECK(check_eights(fn, "hidden", x.hidden, EP_MAX_HIDDEN));
  EP_CHECK(check_eights(fn, "width", x.width, EP_MAX_HIDDEN));
  EP_CHECK(check_eights(fn, "rank", x.rank, EP_MAX_RANK));
  if (x.num_adapters < 1) return fail(EP_ERR_INVALID_ARG, "%s: num_adapters=%d < 1", fn, x.num_adapters);
  if (x.num_adapters > EP_MAX_EXPERTS)
    return fail(EP_ERR_UNSUPPORTED, "%s: num_adapters=%d > %d", fn, x.num_adapters, EP_MAX_EXPERTS);
  const bool any = x.num_rows > 0;
  EP_CHECK(check_ptr(fn, "x", x.x, 16, any));
  EP_CHECK(check_ptr(fn, "w", x.w, 16, true));
  EP_CHECK(check_ptr(fn, "lora_a", x.lora_a, 16, true));
  EP_CHECK(check_ptr(fn, "lora_b", x.lora_b, 16, true));
  EP_CHECK(check_ptr(fn, "adapter_idx", x.adapter_idx, 8, any));
  EP_CHECK(check_ptr(fn, "adapter_scale", x.adapter_scale, 4, false));
  EP_CHECK(check_ptr(fn, "out", x.out, 16, any));
  EP_CHECK(check_ptr(fn, "error_word", x.error_word, 4, false));
  EP_CHECK(check_ptr(fn, "workspace", x.workspace, 16, any));
  const size_t need = adapter_workspace_bytes(x.num_rows, x.hidden, x.rank);
  if (any && x.workspace_bytes < need)
    return fail(EP_ERR_INVALID_ARG, "%s: workspace_bytes=%zu < %zu needed", fn, x.workspace_bytes, need);
  const AdapterArgs a{static_cast<const uint16_t *>(x.x), x.num_rows, x.hidden, static_cast<const uint16_t *>(x.w),
                      x.width, static_cast<const uint16_t *>(x.lora_a), static_cast<const uint16_t *>(x.lora_b),
                      x.num_adapters, x.rank, x.adapter_idx, x.adapter_scale, static_cast<uint16_t *>(x.out),
                      x.workspace, x.error_word};
  return launch_adapter(a, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
