// A product shared by all rows, x w^T, with bias, activation and residual in
// its epilogue, and its gradients.
//
//   z = x w^T + b,  out = act(z) + residual
//   d = act'(z) grad,  grad_x = d w,  grad_w = d^T x,  grad_bias = sum of d
//
// bf16 operands, sums in fp32, results rounded once.  d is an operand of two
// products and kept in bf16; the bias's gradient is summed before that.
#include "ep_pair.cuh"

namespace ep {

namespace {

constexpr int kMaxSlices = 64;  // of the rows, for the bias's gradient

__device__ __forceinline__ float value_of(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ uint16_t rounded(float v) { return (uint16_t)(pack_bf16x2(v, 0.0f) & 0xffffu); }
__device__ __forceinline__ void store_value(void *p, bool bf16, int64_t i, float v) {
  if (bf16)
    static_cast<uint16_t *>(p)[i] = rounded(v);
  else
    static_cast<float *>(p)[i] = v;
}

// act'(z)
__device__ __forceinline__ float slope_of(ep_activation_t act, float z) {
  float s;
  switch (act) {
    case EP_ACT_RELU:
      return z > 0.0f ? 1.0f : 0.0f;
    case EP_ACT_SILU:
      s = sigmoid_of(z);
      return s * (1.0f + z * (1.0f - s));
    case EP_ACT_GELU:
      return 0.5f * erfcf(-z * kRootHalf) + z * kRootOneTwoPi * __expf(-0.5f * z * z);
    case EP_ACT_GELU_TANH:
      s = tanh_gate(z);
      z = fminf(fmaxf(z, -16.0f), 16.0f);  // s (1 - s) is 0 there; z^2 stays finite
      return s + z * s * (1.0f - s) * 2.0f * kRootTwoPi * (1.0f + 3.0f * kCubic * z * z);
    default:
      return 1.0f;
  }
}

// d, rounded, and a slice of the rows' part of the bias's gradient; a column
// a thread.
__global__ void __launch_bounds__(256) dense_gradient_kernel(DenseBackwardArgs p, float *sums, int slices) {
  griddep_wait();
  griddep_launch_dependents();
  const bool gated = p.activation == EP_ACT_SWIGLU;
  const int64_t wide = gated ? 2 * p.width : p.width;
  const int blocks = (p.width - 1) / 256 + 1, slice = blockIdx.x / blocks, n = blockIdx.x % blocks * 256 + threadIdx.x;
  if (n >= p.width) return;
  float sum = 0.0f, other = 0.0f;
  for (int64_t t = slice; t < p.num_rows; t += slices) {
    float d = load_param(p.grad, p.grad_bf16, t * p.width + n);
    if (gated) {
      const float g = value_of(p.preact[t * wide + n]), u = value_of(p.preact[t * wide + p.width + n]), s = sigmoid_of(g);
      const float du = d * g * s;
      d *= u * s * (1.0f + g * (1.0f - s));
      other += du;
      if (p.grad_preact != nullptr) p.grad_preact[t * wide + p.width + n] = rounded(du);
    } else if (p.activation != EP_ACT_NONE) {
      d *= slope_of(p.activation, value_of(p.preact[t * wide + n]));
    }
    if (p.grad_preact != nullptr) p.grad_preact[t * wide + n] = rounded(d);
    sum += d;
  }
  if (p.grad_bias == nullptr) return;
  sums[slice * wide + n] = sum;
  if (gated) sums[slice * wide + p.width + n] = other;
}

__global__ void __launch_bounds__(256) dense_bias_kernel(const float *sums, int slices, int wide, void *out, bool bf16) {
  griddep_wait();
  griddep_launch_dependents();
  const int n = blockIdx.x * 256 + threadIdx.x;
  if (n >= wide) return;
  float sum = 0.0f;
  for (int i = 0; i < slices; ++i) sum += sums[(int64_t)i * wide + n];
  store_value(out, bf16, n, sum);
}

int slices_of(int rows) { return rows < kMaxSlices ? rows : kMaxSlices; }

// What the products of a call share: one expert with every row.
Params params_of(int rows, int wide, int width, int hidden, uint32_t *error_word) {
  Params p = {};
  p.most_rows = p.cap = rows;
  p.error_word = error_word;
  p.E = 1;
  p.wide = wide;
  p.width = width;
  p.hidden = hidden;
  return p;
}

}  // namespace

ep_status_t launch_dense(const DenseArgs &a, cudaStream_t stream) {
  if (a.num_rows == 0) return EP_OK;
  const bool pairs = a.activation == EP_ACT_SWIGLU;
  Params p = params_of(a.num_rows, pairs ? 2 * a.width : a.width, a.width, a.hidden, a.error_word);
  p.inner = a.hidden;
  p.a_tiles = up(a.width, pairs ? 128 : 256);
  p.out = static_cast<uint16_t *>(a.out);
  p.preact = a.preact;
  p.bias = a.bias;
  p.bias_bf16 = a.bias_bf16;
  p.residual = a.residual;
  p.activation = a.activation;
  p.out_fp32 = !a.out_bf16;
  const ep_status_t s = weight_map(p, pairs ? kDenseGated : kDense, a.w, p.wide, a.hidden);
  if (s != EP_OK) return s;
  return pairs ? launch_rows_form<kDenseGated>(p, a.x, a.row_stride, stream)
               : launch_rows_form<kDense>(p, a.x, a.row_stride, stream);
}

size_t dense_workspace_bytes(int num_rows, int hidden, int width, ep_activation_t activation) {
  return (size_t)slices_of(num_rows) * (activation == EP_ACT_SWIGLU ? 2 : 1) * width * sizeof(float);
}

ep_status_t launch_dense_backward(const DenseBackwardArgs &a, cudaStream_t stream) {
  const int wide = a.activation == EP_ACT_SWIGLU ? 2 * a.width : a.width, slices = slices_of(a.num_rows);
  const bool made = a.activation != EP_ACT_NONE || !a.grad_bf16;  // d is not `grad` itself
  float *sums = static_cast<float *>(a.workspace);
  cudaError_t e = cudaSuccess;
  if (a.num_rows > 0 && (a.grad_bias != nullptr || (made && a.grad_preact != nullptr)))
    e = launch_kernel(dense_gradient_kernel, ((a.width - 1) / 256 + 1) * slices, 256, 0, stream, false, a, sums, slices);
  if (e == cudaSuccess && a.grad_bias != nullptr)
    e = launch_kernel(dense_bias_kernel, (wide - 1) / 256 + 1, 256, 0, stream, false, (const float *)sums, slices, wide,
                      a.grad_bias, a.bias_bf16);
  if (e != cudaSuccess) return cuda_fail(e, "dense_backward launch");
  const uint16_t *d = made ? a.grad_preact : static_cast<const uint16_t *>(a.grad);
  if (a.grad_x != nullptr && a.num_rows > 0) {
    Params p = params_of(a.num_rows, wide, a.hidden, a.hidden, a.error_word);
    p.inner = wide;
    p.a_tiles = up(a.hidden, 256);
    p.out = a.grad_x;
    ep_status_t s = weight_map(p, kDenseGradX, a.w, wide, a.hidden);
    if (s == EP_OK) s = launch_rows_form<kDenseGradX>(p, d, wide, stream);
    if (s != EP_OK) return s;
  }
  if (a.grad_w != nullptr) {
    Params p = params_of(a.num_rows, wide, a.width, a.hidden, a.error_word);
    p.parts = 1;
    p.max_cols = kMaxCols;
    p.a_tiles = up(wide, 256);
    p.b_tiles = up(a.hidden, 256);
    p.out = a.grad_w;
    // without rows nothing is copied: the maps only need an address
    const bool any = a.num_rows > 0;
    const int rows = any ? a.num_rows : 1;
    ep_status_t s = block_map(&p.a, &p.a_blocks, any ? d : a.grad_w, wide, rows, wide);
    const uint64_t dims[] = {(uint64_t)a.hidden, (uint64_t)wide, 1};
    const uint64_t strides[] = {a.hidden * kSize, (uint64_t)wide * a.hidden * kSize};
    const uint32_t box[] = {64, 32, 1};
    if (s == EP_OK) s = encode_map(&p.grad, a.grad_w, 3, dims, strides, box);
    if (s == EP_OK) s = block_map(&p.b[0], &p.b_blocks, any ? a.x : a.grad_w, a.hidden, rows, any ? a.row_stride : a.hidden);
    if (s == EP_OK) s = launch_form<kDenseGradW>(p, (int64_t)p.a_tiles * p.b_tiles, stream);
    if (s != EP_OK) return s;
  }
  return EP_OK;
}

}  // namespace ep
