// Layer norm of rows and its gradients.
//
//   mean = sum x / H, rstd = 1 / sqrt(sum (x - mean)^2 / H + eps), n = (x - mean) rstd
//   out = n w + b
//   grad_x = rstd (g w - mean(g w) - n mean(g w n)) + add
//   grad_weight = sum over rows of g n, grad_bias = sum over rows of g
//
// Statistics and sums in fp32, results rounded once.
#include "ep_device.cuh"
#include "ep_ops.h"

namespace ep {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxSlices = 304;  // blocks that sum rows for the parameters' gradients

__device__ __forceinline__ float load_value(const void *p, bool bf16, int64_t i) {
  return bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t *>(p)[i] << 16) : static_cast<const float *>(p)[i];
}

__device__ __forceinline__ void store_value(void *p, bool bf16, int64_t i, float v) {
  if (bf16)
    static_cast<uint16_t *>(p)[i] = (uint16_t)(pack_bf16x2(v, 0.0f) & 0xffffu);
  else
    static_cast<float *>(p)[i] = v;
}

__device__ __forceinline__ float block_sum(float v, float *s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0f;
  for (int i = 0; i < kThreads / 32; ++i) v += s[i];
  return v;
}

__global__ void __launch_bounds__(kThreads) norm_kernel(NormArgs p) {
  __shared__ float s[kThreads / 32];
  griddep_wait();
  griddep_launch_dependents();
  for (int64_t t = blockIdx.x; t < p.num_rows; t += gridDim.x) {
    const int H = p.hidden;
    float sum = 0.0f;
    for (int h = threadIdx.x; h < H; h += kThreads) sum += load_value(p.x, p.bf16, t * p.row_stride + h);
    const float mean = block_sum(sum, s) / H;
    sum = 0.0f;
    for (int h = threadIdx.x; h < H; h += kThreads) {
      const float d = load_value(p.x, p.bf16, t * p.row_stride + h) - mean;
      sum += d * d;
    }
    const float rstd = 1.0f / sqrtf(block_sum(sum, s) / H + p.eps);
    if (threadIdx.x == 0 && p.mean != nullptr) p.mean[t] = mean;
    if (threadIdx.x == 0 && p.rstd != nullptr) p.rstd[t] = rstd;
    for (int h = threadIdx.x; h < H; h += kThreads) {
      float v = (load_value(p.x, p.bf16, t * p.row_stride + h) - mean) * rstd;
      if (p.weight != nullptr) v *= load_value(p.weight, p.param_bf16, h);
      if (p.bias != nullptr) v += load_value(p.bias, p.param_bf16, h);
      store_value(p.out, p.bf16, t * H + h, v);
    }
  }
}

__global__ void __launch_bounds__(kThreads) norm_backward_kernel(NormBackwardArgs p) {
  __shared__ float s[kThreads / 32];
  griddep_wait();
  griddep_launch_dependents();
  for (int64_t t = blockIdx.x; t < p.num_rows; t += gridDim.x) {
    const int H = p.hidden;
    const float mean = p.mean[t], rstd = p.rstd[t];
    const auto of = [&](int h, float &n, float &g) {
      n = (load_value(p.x, p.bf16, t * p.row_stride + h) - mean) * rstd;
      g = load_value(p.grad, p.bf16, t * H + h);
      if (p.weight != nullptr) g *= load_value(p.weight, p.param_bf16, h);
    };
    float a = 0.0f, b = 0.0f, n, g;
    for (int h = threadIdx.x; h < H; h += kThreads) {
      of(h, n, g);
      a += g;
      b += g * n;
    }
    a = block_sum(a, s) / H;
    b = block_sum(b, s) / H;
    for (int h = threadIdx.x; h < H; h += kThreads) {
      of(h, n, g);
      float v = (g - a - n * b) * rstd;
      if (p.add != nullptr) v += load_value(p.add, p.bf16, t * H + h);
      store_value(p.grad_x, p.bf16, t * H + h, v);
    }
  }
}

// A slice of the rows' share of the parameters' gradients, a column a thread.
__global__ void __launch_bounds__(kThreads) norm_params_kernel(NormBackwardArgs p, int slices) {
  griddep_wait();
  griddep_launch_dependents();
  const int h = blockIdx.x * kThreads + threadIdx.x, slice = blockIdx.y, H = p.hidden;
  if (h >= H) return;
  float w = 0.0f, b = 0.0f;
  for (int64_t t = slice; t < p.num_rows; t += slices) {
    const float g = load_value(p.grad, p.bf16, t * H + h);
    w += g * (load_value(p.x, p.bf16, t * p.row_stride + h) - p.mean[t]) * p.rstd[t];
    b += g;
  }
  p.workspace[(int64_t)slice * 2 * H + h] = w;
  p.workspace[((int64_t)slice * 2 + 1) * H + h] = b;
}

__global__ void __launch_bounds__(kThreads) norm_join_kernel(NormBackwardArgs p, int slices) {
  griddep_wait();
  griddep_launch_dependents();
  const int h = blockIdx.x * kThreads + threadIdx.x, H = p.hidden;
  if (h >= H) return;
  float w = 0.0f, b = 0.0f;
  for (int i = 0; i < slices; ++i) {
    w += p.workspace[(int64_t)i * 2 * H + h];
    b += p.workspace[((int64_t)i * 2 + 1) * H + h];
  }
  if (p.grad_weight != nullptr) store_value(p.grad_weight, p.param_bf16, h, w);
  if (p.grad_bias != nullptr) store_value(p.grad_bias, p.param_bf16, h, b);
}

int slices_of(int num_rows) { return num_rows < kMaxSlices ? num_rows : kMaxSlices; }

}  // namespace

ep_status_t launch_norm(const NormArgs &a, cudaStream_t stream) {
  if (a.num_rows == 0) return EP_OK;
  const int grid = a.num_rows < 65536 ? a.num_rows : 65536;
  const cudaError_t e = launch_kernel(norm_kernel, grid, kThreads, 0, stream, false, a);
  return e == cudaSuccess ? EP_OK : cuda_fail(e, "norm launch");
}

size_t norm_workspace_bytes(int num_rows, int hidden) { return (size_t)slices_of(num_rows) * 2 * hidden * sizeof(float); }

ep_status_t launch_norm_backward(const NormBackwardArgs &a, cudaStream_t stream) {
  const int grid = a.num_rows < 65536 ? a.num_rows : 65536, columns = (a.hidden - 1) / kThreads + 1;
  cudaError_t e = cudaSuccess;
  if (a.grad_weight != nullptr || a.grad_bias != nullptr) {
    const int slices = slices_of(a.num_rows);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(columns, slices);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    if (slices > 0) e = cudaLaunchKernelEx(&cfg, norm_params_kernel, a, slices);
    if (e == cudaSuccess) e = launch_kernel(norm_join_kernel, columns, kThreads, 0, stream, false, a, slices);
  }
  if (e == cudaSuccess && a.grad_x != nullptr && a.num_rows > 0)
    e = launch_kernel(norm_backward_kernel, grid, kThreads, 0, stream, false, a);
  return e == cudaSuccess ? EP_OK : cuda_fail(e, "norm_backward launch");
}

}  // namespace ep
