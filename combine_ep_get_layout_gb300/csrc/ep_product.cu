// The experts' products over the rows of an expanded layout, and their
// gradients.  Expert e's rows are the segment [expert_offset[e],
// expert_offset[e] + num_rows_per_expert[e]); its weights are w[e], one row
// of `hidden` inputs per output.
//
//   out[s]    = x[s] w[e]^T                             (plain)
//   out[s]    = silu(x[s] wg^T) * (x[s] wu^T)           (gated: w[e] = [wg; wu])
//   grad_x[s] = g[s] w[e],   grad_w[e] = sum over e's rows of g[s]^T x[s]
//
// with g the gradient of x w^T.  bf16 in and out, sums in fp32, rounded once.
#include "ep_device.cuh"
#include "ep_ops.h"

namespace ep {

namespace {

constexpr int kTile = 64, kStep = 16, kThreads = 256;

struct Segment {
  int first, rows;
};

__device__ __forceinline__ Segment segment(const int32_t *offset, const int32_t *rows, int e, int cap) {
  const int a = offset[e];
  const int n = rows[e];
  Segment s;
  s.first = a;
  s.rows = a < 0 || a >= cap ? 0 : max(0, min(n, cap - a));
  return s;
}

__device__ __forceinline__ float bf16_at(const uint16_t *p) { return __uint_as_float((uint32_t)*p << 16); }

__device__ __forceinline__ uint16_t to_bf16(float v) { return (uint16_t)(pack_bf16x2(v, 0.0f) & 0xffffu); }

__device__ __forceinline__ float silu_of(float g) { return g / (1.0f + expf(-g)); }

// c[i][j] += sum over k < depth of a(m0 + 4 ty + i, k) * b(n0 + 4 tx + j, k)
template <typename A, typename B>
__device__ __forceinline__ void tile_product(float (&c)[4][4], int depth, A a, B b, float (*sa)[kTile], float (*sb)[kTile]) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  for (int k0 = 0; k0 < depth; k0 += kStep) {
    for (int i = threadIdx.x; i < kTile * kStep; i += kThreads) {
      const int r = i / kStep, k = i % kStep;
      sa[k][r] = k0 + k < depth ? a(r, k0 + k) : 0.0f;
      sb[k][r] = k0 + k < depth ? b(r, k0 + k) : 0.0f;
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
}

struct Params {
  ProductArgs a;
};
struct BackwardParams {
  ProductBackwardArgs a;
};

__global__ void __launch_bounds__(kThreads) product_kernel(Params q) {
  const ProductArgs &p = q.a;
  __shared__ float sa[kStep][kTile], sb[kStep][kTile];
  const int e = blockIdx.z, n0 = blockIdx.y * kTile, H = p.hidden;
  griddep_wait();
  griddep_launch_dependents();
  const Segment s = segment(p.expert_offset, p.num_rows_per_expert, e, p.recv_capacity);
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0 && s.rows != p.num_rows_per_expert[e])
    set_error(p.error_word, EP_ERRBIT_CAPACITY);
  const int wide = p.gated ? 2 * p.width : p.width;
  const uint16_t *w = p.w + (int64_t)e * wide * H;
  for (int m0 = blockIdx.x * kTile; m0 < s.rows; m0 += gridDim.x * kTile) {
    const auto x = [&](int r, int k) {
      return m0 + r < s.rows ? bf16_at(p.x + (int64_t)(s.first + m0 + r) * H + k) : 0.0f;
    };
    float c[4][4] = {}, u[4][4] = {};
    tile_product(c, H, x, [&](int r, int k) { return n0 + r < p.width ? bf16_at(w + (int64_t)(n0 + r) * H + k) : 0.0f; },
                 sa, sb);
    if (p.gated)
      tile_product(u, H, x, [&](int r, int k) {
        return n0 + r < p.width ? bf16_at(w + (int64_t)(p.width + n0 + r) * H + k) : 0.0f;
      }, sa, sb);
    for (int i = 0; i < 4; ++i)
      for (int j = 0; j < 4; ++j) {
        const int m = m0 + 4 * (threadIdx.x >> 4) + i, n = n0 + 4 * (threadIdx.x & 15) + j;
        if (m >= s.rows || n >= p.width) continue;
        const int64_t at = s.first + m;
        p.out[at * p.width + n] = to_bf16(p.gated ? silu_of(c[i][j]) * u[i][j] : c[i][j]);
        if (p.preact != nullptr) {
          p.preact[at * wide + n] = to_bf16(c[i][j]);
          if (p.gated) p.preact[at * wide + p.width + n] = to_bf16(u[i][j]);
        }
      }
  }
}

// The gradient of silu(g) * u for the rows of the layout.
__global__ void __launch_bounds__(kThreads) gate_backward_kernel(BackwardParams q) {
  const ProductBackwardArgs &p = q.a;
  griddep_wait();
  griddep_launch_dependents();
  const int e = blockIdx.y;
  const Segment s = segment(p.expert_offset, p.num_rows_per_expert, e, p.recv_capacity);
  const int64_t n = (int64_t)s.rows * p.width;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) {
    const int64_t row = s.first + i / p.width;
    const int col = (int)(i % p.width);
    const float g = bf16_at(p.preact + row * 2 * p.width + col);
    const float u = bf16_at(p.preact + row * 2 * p.width + p.width + col);
    const float d = bf16_at(p.grad + row * p.width + col);
    const float sig = 1.0f / (1.0f + expf(-g));
    p.grad_preact[row * 2 * p.width + col] = to_bf16(d * u * sig * (1.0f + g * (1.0f - sig)));
    p.grad_preact[row * 2 * p.width + p.width + col] = to_bf16(d * g * sig);
  }
}

__global__ void __launch_bounds__(kThreads) product_grad_x_kernel(BackwardParams q) {
  const ProductBackwardArgs &p = q.a;
  __shared__ float sa[kStep][kTile], sb[kStep][kTile];
  griddep_wait();
  griddep_launch_dependents();
  const int e = blockIdx.z, h0 = blockIdx.y * kTile, H = p.hidden;
  const Segment s = segment(p.expert_offset, p.num_rows_per_expert, e, p.recv_capacity);
  const int wide = p.gated ? 2 * p.width : p.width;
  const uint16_t *g = p.gated ? p.grad_preact : p.grad;
  const uint16_t *w = p.w + (int64_t)e * wide * H;
  for (int m0 = blockIdx.x * kTile; m0 < s.rows; m0 += gridDim.x * kTile) {
    float c[4][4] = {};
    tile_product(c, wide, [&](int r, int k) {
      return m0 + r < s.rows ? bf16_at(g + (int64_t)(s.first + m0 + r) * wide + k) : 0.0f;
    }, [&](int r, int k) { return h0 + r < H ? bf16_at(w + (int64_t)k * H + h0 + r) : 0.0f; }, sa, sb);
    for (int i = 0; i < 4; ++i)
      for (int j = 0; j < 4; ++j) {
        const int m = m0 + 4 * (threadIdx.x >> 4) + i, h = h0 + 4 * (threadIdx.x & 15) + j;
        if (m < s.rows && h < H) p.grad_x[(int64_t)(s.first + m) * H + h] = to_bf16(c[i][j]);
      }
  }
}

__global__ void __launch_bounds__(kThreads) product_grad_w_kernel(BackwardParams q) {
  const ProductBackwardArgs &p = q.a;
  __shared__ float sa[kStep][kTile], sb[kStep][kTile];
  griddep_wait();
  griddep_launch_dependents();
  const int e = blockIdx.z, n0 = blockIdx.x * kTile, h0 = blockIdx.y * kTile, H = p.hidden;
  const Segment s = segment(p.expert_offset, p.num_rows_per_expert, e, p.recv_capacity);
  const int wide = p.gated ? 2 * p.width : p.width;
  const uint16_t *g = p.gated ? p.grad_preact : p.grad;
  float c[4][4] = {};
  tile_product(c, s.rows, [&](int r, int k) {
    return n0 + r < wide ? bf16_at(g + (int64_t)(s.first + k) * wide + n0 + r) : 0.0f;
  }, [&](int r, int k) { return h0 + r < H ? bf16_at(p.x + (int64_t)(s.first + k) * H + h0 + r) : 0.0f; }, sa, sb);
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + 4 * (threadIdx.x >> 4) + i, h = h0 + 4 * (threadIdx.x & 15) + j;
      if (n < wide && h < H) p.grad_w[((int64_t)e * wide + n) * H + h] = to_bf16(c[i][j]);
    }
}

int tiles(int n) { return (n + kTile - 1) / kTile; }

template <typename P>
ep_status_t launch3(void (*kernel)(P), dim3 grid, const P &p, cudaStream_t stream, const char *what) {
  if (grid.x == 0 || grid.y == 0 || grid.z == 0) return EP_OK;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = kUsePdl ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  return e == cudaSuccess ? EP_OK : cuda_fail(e, what);
}

}  // namespace

ep_status_t launch_product(const ProductArgs &a, cudaStream_t stream) {
  if (current_device_info() == nullptr) return EP_ERR_CUDA;
  const int most = a.num_tokens < a.recv_capacity ? a.num_tokens : a.recv_capacity;  // rows of one expert
  return launch3(product_kernel, dim3(tiles(most), tiles(a.width), a.num_experts), Params{a}, stream, "product launch");
}

ep_status_t launch_product_backward(const ProductBackwardArgs &a, cudaStream_t stream) {
  const DeviceInfo *di = current_device_info();
  if (di == nullptr) return EP_ERR_CUDA;
  const int most = a.num_tokens < a.recv_capacity ? a.num_tokens : a.recv_capacity;
  const int wide = a.gated ? 2 * a.width : a.width;
  const BackwardParams p{a};
  ep_status_t s = EP_OK;
  if (a.gated) {
    s = launch3(gate_backward_kernel, dim3(most > 0 ? 64 : 0, a.num_experts), p, stream, "gate_backward launch");
    if (s != EP_OK) return s;
  }
  if (a.grad_x != nullptr) {
    s = launch3(product_grad_x_kernel, dim3(tiles(most), tiles(a.hidden), a.num_experts), p, stream,
                "product_grad_x launch");
    if (s != EP_OK) return s;
  }
  if (a.grad_w != nullptr)
    s = launch3(product_grad_w_kernel, dim3(tiles(wide), tiles(a.hidden), a.num_experts), p, stream,
                "product_grad_w launch");
  return s;
}

}  // namespace ep
