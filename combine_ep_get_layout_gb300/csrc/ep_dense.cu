// A product shared by all rows, x w^T, with bias, activation and residual in
// its epilogue, and its gradients.
//
//   z = x w^T + b,  out = act(z) + residual
//   d = act'(z) grad,  grad_x = d w,  grad_w = d^T x,  grad_bias = sum of d
//
// bf16 operands, sums in fp32, results rounded once.  d is an operand of two
// products and kept in bf16; the bias's gradient is summed before that.
#include "ep_device.cuh"
#include "ep_ops.h"

namespace ep {

namespace {

constexpr int kTile = 32;
constexpr int kMaxSlices = 64;  // of the rows, for the bias's gradient

__device__ __forceinline__ float value_of(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ uint16_t rounded(float v) { return (uint16_t)(pack_bf16x2(v, 0.0f) & 0xffffu); }
__device__ __forceinline__ float load_value(const void *p, bool bf16, int64_t i) {
  return bf16 ? value_of(static_cast<const uint16_t *>(p)[i]) : static_cast<const float *>(p)[i];
}
__device__ __forceinline__ void store_value(void *p, bool bf16, int64_t i, float v) {
  if (bf16)
    static_cast<uint16_t *>(p)[i] = rounded(v);
  else
    static_cast<float *>(p)[i] = v;
}

constexpr float kRootHalf = 0.70710678118654752f;      // 1 / sqrt 2
constexpr float kRootTwoPi = 0.79788456080286536f;     // sqrt(2 / pi)
constexpr float kRootOneTwoPi = 0.39894228040143268f;  // 1 / sqrt(2 pi)
constexpr float kCubic = 0.044715f;

__device__ __forceinline__ float sigmoid(float z) { return 1.0f / (1.0f + __expf(-z)); }

__device__ __forceinline__ float activate(ep_activation_t act, float z) {
  switch (act) {
    case EP_ACT_RELU:
      return z < 0.0f ? 0.0f : z;
    case EP_ACT_SILU:
      return z * sigmoid(z);
    case EP_ACT_GELU:
      return 0.5f * z * erfcf(-z * kRootHalf);
    case EP_ACT_GELU_TANH:
      return z * sigmoid(2.0f * kRootTwoPi * (z + kCubic * z * z * z));
    default:
      return z;
  }
}

__device__ __forceinline__ float slope(ep_activation_t act, float z) {
  float s;
  switch (act) {
    case EP_ACT_RELU:
      return z > 0.0f ? 1.0f : 0.0f;
    case EP_ACT_SILU:
      s = sigmoid(z);
      return s * (1.0f + z * (1.0f - s));
    case EP_ACT_GELU:
      return 0.5f * erfcf(-z * kRootHalf) + z * kRootOneTwoPi * __expf(-0.5f * z * z);
    case EP_ACT_GELU_TANH:
      s = sigmoid(2.0f * kRootTwoPi * (z + kCubic * z * z * z));
      z = fminf(fmaxf(z, -16.0f), 16.0f);  // s (1 - s) is 0 there; z^2 stays finite
      return s + z * s * (1.0f - s) * 2.0f * kRootTwoPi * (1.0f + 3.0f * kCubic * z * z);
    default:
      return 1.0f;
  }
}

// sum over k of a(row, k) b(col, k), each matrix by its two strides.
struct Operand {
  const uint16_t *p;
  int64_t outer, inner;
  int count;
};

__device__ float tile_sum(const Operand &a, const Operand &b, int row0, int col0, int K) {
  __shared__ float s_a[kTile][kTile + 1], s_b[kTile][kTile + 1];
  const int x = threadIdx.x, y = threadIdx.y;
  float sum = 0.0f;
  for (int k0 = 0; k0 < K; k0 += kTile) {
    s_a[y][x] = row0 + y < a.count && k0 + x < K ? value_of(a.p[(row0 + y) * a.outer + (k0 + x) * a.inner]) : 0.0f;
    s_b[y][x] = col0 + y < b.count && k0 + x < K ? value_of(b.p[(col0 + y) * b.outer + (k0 + x) * b.inner]) : 0.0f;
    __syncthreads();
    for (int k = 0; k < kTile; ++k) sum += s_a[y][k] * s_b[x][k];
    __syncthreads();
  }
  return sum;
}

__global__ void __launch_bounds__(kTile *kTile) dense_kernel(DenseArgs p) {
  griddep_wait();
  griddep_launch_dependents();
  const bool gated = p.activation == EP_ACT_SWIGLU;
  const int tiles = (p.width - 1) / kTile + 1;
  const int row0 = blockIdx.x / tiles * kTile, col0 = blockIdx.x % tiles * kTile;
  const Operand x{p.x, p.row_stride, 1, p.num_rows}, w{p.w, p.hidden, 1, p.width};
  const int64_t t = row0 + threadIdx.y;
  const int n = col0 + threadIdx.x;
  float z = tile_sum(x, w, row0, col0, p.hidden), u = 0.0f;
  if (gated) {
    const Operand other{p.w + (int64_t)p.width * p.hidden, p.hidden, 1, p.width};
    u = tile_sum(x, other, row0, col0, p.hidden);
  }
  if (t >= p.num_rows || n >= p.width) return;
  const int64_t wide = gated ? 2 * p.width : p.width;
  if (p.bias != nullptr) z += load_value(p.bias, p.bias_bf16, n);
  if (p.bias != nullptr && gated) u += load_value(p.bias, p.bias_bf16, p.width + n);
  if (p.preact != nullptr) p.preact[t * wide + n] = rounded(z);
  if (p.preact != nullptr && gated) p.preact[t * wide + p.width + n] = rounded(u);
  float y = gated ? z * sigmoid(z) * u : activate(p.activation, z);
  if (p.residual != nullptr) y += value_of(p.residual[t * p.width + n]);
  store_value(p.out, p.out_bf16, t * p.width + n, y);
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
    float d = load_value(p.grad, p.grad_bf16, t * p.width + n);
    if (gated) {
      const float g = value_of(p.preact[t * wide + n]), u = value_of(p.preact[t * wide + p.width + n]), s = sigmoid(g);
      const float du = d * g * s;
      d *= u * s * (1.0f + g * (1.0f - s));
      other += du;
      if (p.grad_preact != nullptr) p.grad_preact[t * wide + p.width + n] = rounded(du);
    } else if (p.activation != EP_ACT_NONE) {
      d *= slope(p.activation, value_of(p.preact[t * wide + n]));
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

__global__ void __launch_bounds__(kTile *kTile) dense_product_kernel(Operand a, Operand b, int K, uint16_t *out) {
  griddep_wait();
  griddep_launch_dependents();
  const int tiles = (b.count - 1) / kTile + 1;
  const int row0 = blockIdx.x / tiles * kTile, col0 = blockIdx.x % tiles * kTile;
  const float v = tile_sum(a, b, row0, col0, K);
  const int64_t row = row0 + threadIdx.y;
  const int col = col0 + threadIdx.x;
  if (row < a.count && col < b.count) out[row * b.count + col] = rounded(v);
}

int slices_of(int rows) { return rows < kMaxSlices ? rows : kMaxSlices; }

cudaError_t launch_tiles(const Operand &a, const Operand &b, int K, uint16_t *out, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(((a.count - 1) / kTile + 1) * ((b.count - 1) / kTile + 1));
  cfg.blockDim = dim3(kTile, kTile);
  cfg.stream = stream;
  return cudaLaunchKernelEx(&cfg, dense_product_kernel, a, b, K, out);
}

}  // namespace

ep_status_t launch_dense(const DenseArgs &a, cudaStream_t stream) {
  if (a.num_rows == 0) return EP_OK;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(((a.num_rows - 1) / kTile + 1) * ((a.width - 1) / kTile + 1));
  cfg.blockDim = dim3(kTile, kTile);
  cfg.stream = stream;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, dense_kernel, a);
  return e == cudaSuccess ? EP_OK : cuda_fail(e, "dense launch");
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
  const uint16_t *d = made ? a.grad_preact : static_cast<const uint16_t *>(a.grad);
  if (e == cudaSuccess && a.grad_x != nullptr && a.num_rows > 0)
    e = launch_tiles(Operand{d, wide, 1, a.num_rows}, Operand{a.w, 1, a.hidden, a.hidden}, wide, a.grad_x, stream);
  if (e == cudaSuccess && a.grad_w != nullptr)
    e = launch_tiles(Operand{d, 1, wide, wide}, Operand{a.x, 1, a.row_stride, a.hidden}, a.num_rows, a.grad_w, stream);
  return e == cudaSuccess ? EP_OK : cuda_fail(e, "dense_backward launch");
}

}  // namespace ep
