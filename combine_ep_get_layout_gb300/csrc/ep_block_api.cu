// The C ABI of the operators of the block around the layer (balance loss,
// layer norm, shared product): argument checks on the host, before any CUDA
// call.
#include <cmath>

#include "ep_ops.h"

using namespace ep;

#define EP_CHECK(expr)             \
  do {                             \
    const ep_status_t _s = (expr); \
    if (_s != EP_OK) return _s;    \
  } while (0)

namespace {

ep_status_t check_type(const char *fn, const char *name, int type) {
  if (type != EP_TYPE_FP32 && type != EP_TYPE_BF16) return fail(EP_ERR_INVALID_ARG, "%s: unknown %s %d", fn, name, type);
  return EP_OK;
}

// A size in [least, most].
ep_status_t check_size(const char *fn, const char *name, int v, int least, int most) {
  if (v < least) return fail(EP_ERR_INVALID_ARG, "%s: %s=%d < %d", fn, name, v, least);
  if (v > most) return fail(EP_ERR_UNSUPPORTED, "%s: %s=%d > %d", fn, name, v, most);
  return EP_OK;
}

ep_status_t check_stride(const char *fn, int64_t stride, const char *name, int least) {
  if (stride < least) return fail(EP_ERR_INVALID_ARG, "%s: row_stride=%lld < %s=%d", fn, (long long)stride, name, least);
  return EP_OK;
}

ep_status_t check_workspace(const char *fn, const void *p, size_t bytes, size_t need) {
  EP_CHECK(check_ptr(fn, "workspace", p, 16, need > 0));
  if (bytes < need) return fail(EP_ERR_INVALID_ARG, "%s: workspace_bytes=%zu < %zu needed", fn, bytes, need);
  return EP_OK;
}

ep_status_t check_balance(const char *fn, int T, int E, int score, int type, int64_t stride, const int32_t *offsets, int S) {
  EP_CHECK(check_size(fn, "num_tokens", T, 0, EP_MAX_ROWS));
  EP_CHECK(check_size(fn, "num_experts", E, 1, EP_MAX_EXPERTS));
  if (score != EP_SCORE_SOFTMAX && score != EP_SCORE_SIGMOID)
    return fail(EP_ERR_INVALID_ARG, "%s: unknown score %d", fn, score);
  EP_CHECK(check_type(fn, "logits_type", type));
  EP_CHECK(check_stride(fn, stride, "num_experts", E));
  EP_CHECK(check_size(fn, "num_sequences", S, 1, EP_MAX_SEQUENCES));
  EP_CHECK(check_ptr(fn, "seq_offsets", offsets, 4, S > 1));
  return EP_OK;
}

ep_status_t check_norm(const char *fn, int T, int H, int type, int param_type, int64_t stride) {
  EP_CHECK(check_size(fn, "num_rows", T, 0, EP_MAX_ROWS));
  EP_CHECK(check_size(fn, "hidden", H, 1, EP_MAX_HIDDEN));
  EP_CHECK(check_type(fn, "type", type));
  EP_CHECK(check_type(fn, "param_type", param_type));
  return check_stride(fn, stride, "hidden", H);
}

ep_status_t check_eights(const char *fn, const char *name, int v) {
  EP_CHECK(check_size(fn, name, v, 8, EP_MAX_HIDDEN));
  if (v % 8 != 0) return fail(EP_ERR_INVALID_ARG, "%s: %s=%d is not a multiple of 8", fn, name, v);
  return EP_OK;
}

ep_status_t check_dense(const char *fn, int T, int H, int width, int act, int64_t stride) {
  EP_CHECK(check_size(fn, "num_rows", T, 0, EP_MAX_ROWS));
  EP_CHECK(check_eights(fn, "hidden", H));
  EP_CHECK(check_size(fn, "width", width, 1, EP_MAX_HIDDEN));
  if (act < EP_ACT_NONE || act > EP_ACT_GELU_TANH) return fail(EP_ERR_INVALID_ARG, "%s: unknown activation %d", fn, act);
  EP_CHECK(check_stride(fn, stride, "hidden", H));
  if (stride % 8 != 0)
    return fail(EP_ERR_INVALID_ARG, "%s: row_stride=%lld is not a multiple of 8", fn, (long long)stride);
  return EP_OK;
}

// What a call writes or reads (`p` null: not given).
struct Named {
  const char *name;
  const void *p;
};

// An output that begins where another output or an operand does, which others
// may still read or write then.
template <int M, int N>
ep_status_t check_apart(const char *fn, const Named (&outputs)[M], const Named (&operands)[N]) {
  for (int i = 0; i < M; ++i) {
    const Named &out = outputs[i];
    if (out.p == nullptr) continue;
    for (int j = i + 1; j < M; ++j)
      if (outputs[j].p == out.p) return fail(EP_ERR_INVALID_ARG, "%s: %s is %s", fn, out.name, outputs[j].name);
    for (const Named &in : operands)
      if (in.p == out.p) return fail(EP_ERR_INVALID_ARG, "%s: %s is %s", fn, out.name, in.name);
  }
  return EP_OK;
}

size_t size_of(int type) { return type == EP_TYPE_BF16 ? 2 : 4; }

}  // namespace

extern "C" {

size_t ep_balance_workspace_bytes(int T, int E, int S) {
  if (T < 0 || T > EP_MAX_ROWS || E < 1 || E > EP_MAX_EXPERTS || S < 1 || S > EP_MAX_SEQUENCES) return 0;
  return balance_workspace_bytes(T, E, S);
}

ep_status_t ep_balance_loss(const ep_balance_loss_args_t *args, ep_stream_t stream) {
  static const char *fn = "ep_balance_loss";
  clear_error();
  if (args == nullptr) return fail(EP_ERR_INVALID_ARG, "%s: args is NULL", fn);
  const ep_balance_loss_args_t &x = *args;
  EP_CHECK(check_balance(fn, x.num_tokens, x.num_experts, x.score, x.logits_type, x.row_stride, x.seq_offsets,
                         x.num_sequences));
  if (x.num_topk < 1 || x.num_topk > x.num_experts)
    return fail(EP_ERR_INVALID_ARG, "%s: num_topk=%d not in [1, num_experts=%d]", fn, x.num_topk, x.num_experts);
  if (x.num_topk > EP_MAX_TOPK) return fail(EP_ERR_UNSUPPORTED, "%s: num_topk=%d > %d", fn, x.num_topk, EP_MAX_TOPK);
  const bool any = x.num_tokens > 0;
  EP_CHECK(check_ptr(fn, "logits", x.logits, size_of(x.logits_type), any));
  EP_CHECK(check_ptr(fn, "topk_idx", x.topk_idx, 8, any));
  EP_CHECK(check_ptr(fn, "losses", x.losses, 4, true));
  EP_CHECK(check_ptr(fn, "counts", x.counts, 4, true));
  EP_CHECK(check_ptr(fn, "probs", x.probs, 4, true));
  EP_CHECK(check_ptr(fn, "slopes", x.slopes, 4, true));
  EP_CHECK(check_workspace(fn, x.workspace, x.workspace_bytes,
                           balance_workspace_bytes(x.num_tokens, x.num_experts, x.num_sequences)));
  const BalanceArgs a{x.logits, x.logits_type == EP_LOGITS_BF16, x.row_stride, x.topk_idx, x.num_tokens, x.num_experts,
                      x.num_topk, x.score == EP_SCORE_SIGMOID, x.seq_offsets, x.num_sequences, x.losses, x.counts,
                      x.probs, x.slopes, x.workspace};
  return launch_balance(a, reinterpret_cast<cudaStream_t>(stream));
}

ep_status_t ep_balance_loss_backward(const ep_balance_loss_backward_args_t *args, ep_stream_t stream) {
  static const char *fn = "ep_balance_loss_backward";
  clear_error();
  if (args == nullptr) return fail(EP_ERR_INVALID_ARG, "%s: args is NULL", fn);
  const ep_balance_loss_backward_args_t &x = *args;
  EP_CHECK(check_balance(fn, x.num_tokens, x.num_experts, x.score, x.logits_type, x.row_stride, x.seq_offsets,
                         x.num_sequences));
  const bool any = x.num_tokens > 0;
  const size_t size = size_of(x.logits_type);
  EP_CHECK(check_ptr(fn, "grad_losses", x.grad_losses, 4, any));
  EP_CHECK(check_ptr(fn, "logits", x.logits, size, any));
  EP_CHECK(check_ptr(fn, "slopes", x.slopes, 4, any));
  EP_CHECK(check_ptr(fn, "add", x.add, size, false));
  EP_CHECK(check_ptr(fn, "grad_logits", x.grad_logits, size, any));
  if (any && x.grad_logits == x.logits && x.row_stride != x.num_experts && x.num_tokens > 1)
    return fail(EP_ERR_INVALID_ARG, "%s: grad_logits is logits, whose rows are %lld apart", fn, (long long)x.row_stride);
  const BalanceBackwardArgs a{x.grad_losses, x.logits, x.logits_type == EP_LOGITS_BF16, x.row_stride, x.num_tokens,
                              x.num_experts, x.score == EP_SCORE_SIGMOID, x.seq_offsets, x.num_sequences, x.slopes,
                              x.add, x.grad_logits};
  return launch_balance_backward(a, reinterpret_cast<cudaStream_t>(stream));
}

ep_status_t ep_layer_norm(const ep_layer_norm_args_t *args, ep_stream_t stream) {
  static const char *fn = "ep_layer_norm";
  clear_error();
  if (args == nullptr) return fail(EP_ERR_INVALID_ARG, "%s: args is NULL", fn);
  const ep_layer_norm_args_t &x = *args;
  EP_CHECK(check_norm(fn, x.num_rows, x.hidden, x.type, x.param_type, x.row_stride));
  if (!(x.eps > 0.0f) || std::isinf(x.eps)) return fail(EP_ERR_INVALID_ARG, "%s: eps=%g is not positive", fn, x.eps);
  const bool any = x.num_rows > 0;
  EP_CHECK(check_ptr(fn, "x", x.x, size_of(x.type), any));
  EP_CHECK(check_ptr(fn, "weight", x.weight, size_of(x.param_type), false));
  EP_CHECK(check_ptr(fn, "bias", x.bias, size_of(x.param_type), false));
  EP_CHECK(check_ptr(fn, "out", x.out, size_of(x.type), any));
  EP_CHECK(check_ptr(fn, "mean", x.mean, 4, false));
  EP_CHECK(check_ptr(fn, "rstd", x.rstd, 4, false));
  if (any && x.out == x.x && x.row_stride != x.hidden && x.num_rows > 1)
    return fail(EP_ERR_INVALID_ARG, "%s: out is x, whose rows are %lld apart", fn, (long long)x.row_stride);
  const NormArgs a{x.x, x.type == EP_TYPE_BF16, x.row_stride, x.num_rows, x.hidden, x.weight, x.bias,
                   x.param_type == EP_TYPE_BF16, x.eps, x.out, x.mean, x.rstd};
  return launch_norm(a, reinterpret_cast<cudaStream_t>(stream));
}

size_t ep_layer_norm_workspace_bytes(int num_rows, int hidden) {
  if (num_rows < 0 || num_rows > EP_MAX_ROWS || hidden < 1 || hidden > EP_MAX_HIDDEN) return 0;
  return norm_workspace_bytes(num_rows, hidden);
}

ep_status_t ep_layer_norm_backward(const ep_layer_norm_backward_args_t *args, ep_stream_t stream) {
  static const char *fn = "ep_layer_norm_backward";
  clear_error();
  if (args == nullptr) return fail(EP_ERR_INVALID_ARG, "%s: args is NULL", fn);
  const ep_layer_norm_backward_args_t &x = *args;
  EP_CHECK(check_norm(fn, x.num_rows, x.hidden, x.type, x.param_type, x.row_stride));
  const bool any = x.num_rows > 0, params = x.grad_weight != nullptr || x.grad_bias != nullptr;
  EP_CHECK(check_ptr(fn, "grad", x.grad, size_of(x.type), any));
  EP_CHECK(check_ptr(fn, "x", x.x, size_of(x.type), any));
  EP_CHECK(check_ptr(fn, "mean", x.mean, 4, any));
  EP_CHECK(check_ptr(fn, "rstd", x.rstd, 4, any));
  EP_CHECK(check_ptr(fn, "weight", x.weight, size_of(x.param_type), false));
  EP_CHECK(check_ptr(fn, "add", x.add, size_of(x.type), false));
  EP_CHECK(check_ptr(fn, "grad_x", x.grad_x, size_of(x.type), false));
  EP_CHECK(check_ptr(fn, "grad_weight", x.grad_weight, size_of(x.param_type), false));
  EP_CHECK(check_ptr(fn, "grad_bias", x.grad_bias, size_of(x.param_type), false));
  if (any && x.grad_x != nullptr && x.grad_x == x.x && x.row_stride != x.hidden && x.num_rows > 1)
    return fail(EP_ERR_INVALID_ARG, "%s: grad_x is x, whose rows are %lld apart", fn, (long long)x.row_stride);
  EP_CHECK(check_workspace(fn, x.workspace, x.workspace_bytes, params ? norm_workspace_bytes(x.num_rows, x.hidden) : 0));
  const NormBackwardArgs a{x.grad, x.x, x.type == EP_TYPE_BF16, x.row_stride, x.num_rows, x.hidden, x.mean, x.rstd,
                           x.weight, x.param_type == EP_TYPE_BF16, x.add, x.grad_x, x.grad_weight, x.grad_bias,
                           static_cast<float *>(x.workspace)};
  return launch_norm_backward(a, reinterpret_cast<cudaStream_t>(stream));
}

ep_status_t ep_dense_product(const ep_dense_product_args_t *args, ep_stream_t stream) {
  static const char *fn = "ep_dense_product";
  clear_error();
  if (args == nullptr) return fail(EP_ERR_INVALID_ARG, "%s: args is NULL", fn);
  const ep_dense_product_args_t &x = *args;
  EP_CHECK(check_dense(fn, x.num_rows, x.hidden, x.width, x.activation, x.row_stride));
  EP_CHECK(check_type(fn, "bias_type", x.bias_type));
  EP_CHECK(check_type(fn, "out_type", x.out_type));
  const bool any = x.num_rows > 0;
  EP_CHECK(check_ptr(fn, "x", x.x, 16, any));
  EP_CHECK(check_ptr(fn, "w", x.w, 16, true));
  EP_CHECK(check_ptr(fn, "bias", x.bias, size_of(x.bias_type), false));
  EP_CHECK(check_ptr(fn, "residual", x.residual, 16, false));
  EP_CHECK(check_ptr(fn, "out", x.out, 16, any));
  EP_CHECK(check_ptr(fn, "preact", x.preact, 16, false));
  EP_CHECK(check_ptr(fn, "error_word", x.error_word, 4, false));
  if (any && x.residual == x.out && x.out_type == EP_TYPE_FP32)
    return fail(EP_ERR_INVALID_ARG, "%s: residual (bf16) is out (fp32)", fn);
  if (any) {
    const Named operands[] = {{"x", x.x}, {"w", x.w}, {"bias", x.bias}, {"error_word", x.error_word},
                              {"residual", x.residual == x.out ? nullptr : x.residual}};
    const Named outputs[] = {{"out", x.out}, {"preact", x.preact}};
    EP_CHECK(check_apart(fn, outputs, operands));
  }
  const DenseArgs a{static_cast<const uint16_t *>(x.x), x.row_stride, x.num_rows, x.hidden,
                    static_cast<const uint16_t *>(x.w), x.width, x.bias, x.bias_type == EP_TYPE_BF16, x.activation,
                    static_cast<const uint16_t *>(x.residual), x.out, x.out_type == EP_TYPE_BF16,
                    static_cast<uint16_t *>(x.preact), x.error_word};
  return launch_dense(a, reinterpret_cast<cudaStream_t>(stream));
}

size_t ep_dense_workspace_bytes(int num_rows, int hidden, int width, ep_activation_t activation) {
  if (num_rows < 0 || num_rows > EP_MAX_ROWS || hidden < 8 || hidden > EP_MAX_HIDDEN || hidden % 8 != 0 || width < 1 ||
      width > EP_MAX_HIDDEN)
    return 0;
  return dense_workspace_bytes(num_rows, hidden, width, activation);
}

ep_status_t ep_dense_product_backward(const ep_dense_product_backward_args_t *args, ep_stream_t stream) {
  static const char *fn = "ep_dense_product_backward";
  clear_error();
  if (args == nullptr) return fail(EP_ERR_INVALID_ARG, "%s: args is NULL", fn);
  const ep_dense_product_backward_args_t &x = *args;
  EP_CHECK(check_dense(fn, x.num_rows, x.hidden, x.width, x.activation, x.row_stride));
  EP_CHECK(check_type(fn, "grad_type", x.grad_type));
  EP_CHECK(check_type(fn, "bias_type", x.bias_type));
  const bool any = x.num_rows > 0, act = x.activation != EP_ACT_NONE;
  const bool products = x.grad_x != nullptr || x.grad_w != nullptr;
  EP_CHECK(check_ptr(fn, "grad", x.grad, 16, any));
  EP_CHECK(check_ptr(fn, "x", x.x, 16, any && x.grad_w != nullptr));
  EP_CHECK(check_ptr(fn, "w", x.w, 16, any && x.grad_x != nullptr));
  EP_CHECK(check_ptr(fn, "preact", x.preact, 16, any && act));
  EP_CHECK(check_ptr(fn, "grad_preact", x.grad_preact, 16,
                     any && products && (act || x.grad_type == EP_TYPE_FP32 || x.width % 8 != 0)));
  EP_CHECK(check_ptr(fn, "grad_x", x.grad_x, 16, false));
  EP_CHECK(check_ptr(fn, "grad_w", x.grad_w, 16, false));
  EP_CHECK(check_ptr(fn, "grad_bias", x.grad_bias, size_of(x.bias_type), false));
  EP_CHECK(check_ptr(fn, "error_word", x.error_word, 4, false));
  EP_CHECK(check_workspace(fn, x.workspace, x.workspace_bytes,
                           dense_workspace_bytes(x.num_rows, x.hidden, x.width, x.activation)));
  // (without rows only the parameters' gradients are written)
  const auto rows = [&](const void *p) { return any ? p : nullptr; };
  const Named outputs[] = {{"grad_x", rows(x.grad_x)}, {"grad_w", x.grad_w}, {"grad_bias", x.grad_bias},
                           {"grad_preact", rows(x.grad_preact)}, {"workspace", x.workspace}};
  const Named operands[] = {{"grad", rows(x.grad)}, {"x", rows(x.x)}, {"w", x.w}, {"preact", rows(x.preact)},
                            {"error_word", x.error_word}};
  EP_CHECK(check_apart(fn, outputs, operands));
  const DenseBackwardArgs a{x.grad, x.grad_type == EP_TYPE_BF16, static_cast<const uint16_t *>(x.x), x.row_stride,
                            x.num_rows, x.hidden, static_cast<const uint16_t *>(x.w), x.width, x.activation,
                            static_cast<const uint16_t *>(x.preact), static_cast<uint16_t *>(x.grad_preact),
                            static_cast<uint16_t *>(x.grad_x), static_cast<uint16_t *>(x.grad_w), x.grad_bias,
                            x.bias_type == EP_TYPE_BF16, x.workspace, x.error_word};
  return launch_dense_backward(a, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
