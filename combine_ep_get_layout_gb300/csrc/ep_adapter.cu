// A shared projection with low-rank adapters of many requests beside it:
//
//   y[t] = x[t] w^T + scale[a] (x[t] A_a^T) B_a^T,    a = adapter_idx[t]
//
// (no second term where a = -1).  bf16 in and out, sums in fp32.
#include "ep_device.cuh"
#include "ep_ops.h"

namespace ep {

namespace {

constexpr int kThreads = 256;

struct Params {
  AdapterArgs a;
};

__device__ __forceinline__ float bf16_at(const uint16_t *p) { return __uint_as_float((uint32_t)*p << 16); }

// low[t] = scale[a] x[t] A_a^T, fp32 [T, rank]: one block a row, one warp an output.
__global__ void __launch_bounds__(kThreads) adapter_low_kernel(Params q) {
  const AdapterArgs &p = q.a;
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int t = blockIdx.x; t < p.num_rows; t += gridDim.x) {
    const int64_t a = p.adapter_idx[t];
    const bool none = a < 0 || a >= p.num_adapters;
    if (none && a != -1 && threadIdx.x == 0) set_error(p.error_word, EP_ERRBIT_BAD_INDEX);
    float *low = static_cast<float *>(p.workspace) + (int64_t)t * p.rank;
    for (int r = warp; r < p.rank; r += kThreads / 32) {
      float s = 0.0f;
      if (!none) {
        const uint16_t *row = p.lora_a + ((int64_t)a * p.rank + r) * p.hidden;
        for (int k = lane; k < p.hidden; k += 32) s += bf16_at(p.x + (int64_t)t * p.hidden + k) * bf16_at(row + k);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        s *= p.adapter_scale == nullptr ? 1.0f : p.adapter_scale[a];
      }
      if (lane == 0) low[r] = s;
    }
  }
}

constexpr int kTile = 64, kStep = 16;

__global__ void __launch_bounds__(kThreads) adapter_product_kernel(Params q) {
  const AdapterArgs &p = q.a;
  __shared__ float sa[kStep][kTile], sb[kStep][kTile];
  griddep_wait();
  griddep_launch_dependents();
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int t0 = blockIdx.x * kTile, n0 = blockIdx.y * kTile;
  float c[4][4] = {};
  for (int k0 = 0; k0 < p.hidden; k0 += kStep) {
    for (int i = threadIdx.x; i < kTile * kStep; i += kThreads) {
      const int r = i / kStep, k = k0 + i % kStep;
      sa[i % kStep][r] = t0 + r < p.num_rows && k < p.hidden ? bf16_at(p.x + (int64_t)(t0 + r) * p.hidden + k) : 0.0f;
      sb[i % kStep][r] = n0 + r < p.width && k < p.hidden ? bf16_at(p.w + (int64_t)(n0 + r) * p.hidden + k) : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kStep; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) c[i][j] += sa[k][4 * ty + i] * sb[k][4 * tx + j];
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i) {
    const int t = t0 + 4 * ty + i;
    if (t >= p.num_rows) continue;
    const int64_t a = p.adapter_idx[t];
    const float *low = static_cast<const float *>(p.workspace) + (int64_t)t * p.rank;
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + 4 * tx + j;
      if (n >= p.width) continue;
      float s = 0.0f;
      if (a >= 0 && a < p.num_adapters)
        for (int r = 0; r < p.rank; ++r) s += low[r] * bf16_at(p.lora_b + ((int64_t)a * p.width + n) * p.rank + r);
      p.out[(int64_t)t * p.width + n] = (uint16_t)(pack_bf16x2(c[i][j] + s, 0.0f) & 0xffffu);
    }
  }
}

}  // namespace

size_t adapter_workspace_bytes(int num_rows, int hidden, int rank) {
  (void)hidden;
  return ((size_t)num_rows * rank * 4 + 255) / 256 * 256;
}

ep_status_t launch_adapter(const AdapterArgs &a, cudaStream_t stream) {
  if (a.num_rows == 0) return EP_OK;
  const DeviceInfo *di = current_device_info();
  if (di == nullptr) return EP_ERR_CUDA;
  const int most = di->num_sms * 8;
  cudaError_t e = launch_kernel(adapter_low_kernel, a.num_rows < most ? a.num_rows : most, kThreads, 0, stream, false,
                                Params{a});
  if (e != cudaSuccess) return cuda_fail(e, "adapter_low launch");
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.num_rows + kTile - 1) / kTile, (a.width + kTile - 1) / kTile);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = kUsePdl ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, adapter_product_kernel, Params{a});
  return e == cudaSuccess ? EP_OK : cuda_fail(e, "adapter_product launch");
}

}  // namespace ep
