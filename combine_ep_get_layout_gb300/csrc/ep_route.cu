// The router: a token's logits to its experts and their weights, and the
// gradient of the weights with respect to the logits.
//
//   p   = softmax(l) or sigmoid(l)
//   key = p + bias          (the bias steers the choice, never the weight)
//   a group's score = the sum of its best one or two keys; only the experts
//   of the best topk_groups groups are offered
//   idx = the K largest keys, descending, ties to the lowest index
//   w   = p[idx], divided by its sum if renormalised, times a constant
//
// The softmax of the chosen ones alone equals their renormalised share of
// the softmax of all, so renormalised softmax weights need K exponentials.
// Everything is held in fp32.  A masked expert (-infinity or NaN) is never
// chosen.
#include "ep_device.cuh"
#include "ep_ops.h"

namespace ep {

namespace {

constexpr int kRouteWarps = 4;
constexpr float kNegInf = -__builtin_huge_valf();

struct RouteParams {
  const void *logits;
  int64_t row_stride;
  int T, E, K;
  const float *bias;
  int G, Gk;
  float scale;
  int64_t *idx;
  float *w;
  int group_top;
  bool sigmoid, renorm, by_logit;
};

// A logit in fp32: NaN counts as masked, +infinity as the largest number.
template <bool BF16>
__device__ __forceinline__ float load_logit(const void *row, int j) {
  float v = BF16 ? __uint_as_float((uint32_t)static_cast<const uint16_t *>(row)[j] << 16)
                 : static_cast<const float *>(row)[j];
  v = v != v ? kNegInf : v;
  return fminf(v, 3.402823466e38f);
}

__device__ __forceinline__ float sigmoid_of(float l) { return 1.0f / (1.0f + expf(-l)); }

// Order-preserving map of a float (no NaN) to an unsigned integer.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);  // -0 counts as +0
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Warp-collective: the index of the largest value (ties to the lowest
// index), or -1 when every value is -infinity.  `i` < 0 where a lane has none.
__device__ __forceinline__ int warp_argmax(float v, int i) {
  const bool none = i < 0 || v == kNegInf;
  const uint32_t b = none ? 0u : ordered(v);
  const uint32_t top = __reduce_max_sync(0xffffffffu, b);
  const uint32_t at = __reduce_min_sync(0xffffffffu, (!none && b == top) ? (uint32_t)i : 0xffffffffu);
  return (int)at;
}

// The weight of lane k's choice (l = its logit, none: no choice).  m and sum
// are the row's maximum and its sum of exp(l - m), used by the softmax that
// is not renormalised.  Renormalised weights are shares, so the largest
// exponential of the chosen is taken out and none of them can underflow
// together: sigmoid(l) = exp(min(l, 0)) / (1 + exp(-|l|)).
__device__ __forceinline__ float choice_weight(bool none, float l, bool sigmoid, bool renorm, float m, float sum) {
  float p;
  if (sigmoid) {
    const float low = fminf(l, 0.0f);
    const float top = renorm ? warp_max(none ? kNegInf : low) : 0.0f;
    p = none ? 0.0f : expf(low - top) / (1.0f + expf(-fabsf(l)));
  } else {
    const float top = renorm ? warp_max(none ? kNegInf : l) : m;
    p = none ? 0.0f : expf(l - top);
    if (!renorm) p = none ? 0.0f : p / sum;
  }
  if (renorm) {
    const float total = warp_sum(p);
    p = total > 0.0f ? p / total : 0.0f;
  }
  return p;
}

// One warp a token; the keys of its row in shared memory.
template <bool BF16>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(RouteParams p) {
  extern __shared__ float s_keys[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float *key = s_keys + (size_t)warp * p.E;
  griddep_wait();
  griddep_launch_dependents();
  for (int t = blockIdx.x * kRouteWarps + warp; t < p.T; t += gridDim.x * kRouteWarps) {
    const void *row = static_cast<const char *>(p.logits) + (int64_t)t * p.row_stride * (BF16 ? 2 : 4);
    float m = kNegInf, sum = 0.0f;
    for (int j = lane; j < p.E; j += 32) {
      const float l = load_logit<BF16>(row, j);
      key[j] = l;
      m = fmaxf(m, l);
    }
    m = warp_max(m);
    if (!p.sigmoid && (!p.by_logit || !p.renorm)) {
      for (int j = lane; j < p.E; j += 32) sum += key[j] == kNegInf ? 0.0f : expf(key[j] - m);
      sum = warp_sum(sum);
    }
    if (!p.by_logit)
      for (int j = lane; j < p.E; j += 32) {
        const float l = key[j];
        float v = p.sigmoid ? sigmoid_of(l) : expf(l - m) / sum;
        if (p.bias != nullptr) v += p.bias[j];
        key[j] = l == kNegInf || v != v ? kNegInf : v;
      }
    __syncwarp();
    uint64_t groups = ~0ull;
    const int per = p.E / p.G;
    if (p.G > 1) {
      float score[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int g = lane + 32 * h;
        float a = kNegInf, b = kNegInf;
        if (g < p.G)
          for (int j = g * per; j < (g + 1) * per; ++j) {
            const float v = key[j];
            if (v > a) {
              b = a;
              a = v;
            } else if (v > b) {
              b = v;
            }
          }
        score[h] = p.group_top == 2 && b != kNegInf ? a + b : a;
      }
      groups = 0ull;
      for (int k = 0; k < p.Gk; ++k) {
        const bool second = score[1] > score[0];
        const int g = warp_argmax(second ? score[1] : score[0], lane + (second ? 32 : 0));
        if (g < 0) break;
        groups |= 1ull << g;
        if (g == lane) score[0] = kNegInf;
        if (g == lane + 32) score[1] = kNegInf;
      }
    }
    int mine = -1;
    for (int k = 0; k < p.K; ++k) {
      float v = kNegInf;
      int at = -1;
      for (int j = lane; j < p.E; j += 32)
        if (key[j] > v && ((groups >> (j / per)) & 1ull)) {
          v = key[j];
          at = j;
        }
      const int best = warp_argmax(v, at);
      if (best < 0) break;
      if (lane == k) mine = best;
      if ((best & 31) == lane) key[best] = kNegInf;
      __syncwarp();
    }
    const bool none = mine < 0;
    const float l = none ? kNegInf : load_logit<BF16>(row, mine);
    const float w = choice_weight(none, l, p.sigmoid, p.renorm, m, sum);
    if (lane < p.K) {
      p.idx[(int64_t)t * p.K + lane] = mine;
      p.w[(int64_t)t * p.K + lane] = w * p.scale;
    }
    __syncwarp();
  }
}

struct RouteBackwardParams {
  const float *grad;
  const void *logits;
  int64_t row_stride;
  const int64_t *idx;
  int T, E, K;
  float scale;
  void *out;
  bool sigmoid, renorm;
};

template <bool BF16>
__device__ __forceinline__ void store_grad(void *row, int j, float v) {
  if (BF16)
    static_cast<uint16_t *>(row)[j] = (uint16_t)(pack_bf16x2(v, 0.0f) & 0xffffu);
  else
    static_cast<float *>(row)[j] = v;
}

// One warp a token; the row of gradients in shared memory.
template <bool BF16>
__global__ void __launch_bounds__(kRouteWarps * 32) route_backward_kernel(RouteBackwardParams p) {
  extern __shared__ float s_rows[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float *dense = s_rows + (size_t)warp * p.E;
  griddep_wait();
  griddep_launch_dependents();
  for (int t = blockIdx.x * kRouteWarps + warp; t < p.T; t += gridDim.x * kRouteWarps) {
    const void *row = static_cast<const char *>(p.logits) + (int64_t)t * p.row_stride * (BF16 ? 2 : 4);
    void *out = static_cast<char *>(p.out) + (int64_t)t * p.E * (BF16 ? 2 : 4);
    for (int j = lane; j < p.E; j += 32) dense[j] = 0.0f;
    float m = kNegInf, sum = 0.0f;
    if (!p.sigmoid && !p.renorm) {
      for (int j = lane; j < p.E; j += 32) m = fmaxf(m, load_logit<BF16>(row, j));
      m = warp_max(m);
      for (int j = lane; j < p.E; j += 32) {
        const float l = load_logit<BF16>(row, j);
        sum += l == kNegInf ? 0.0f : expf(l - m);
      }
      sum = warp_sum(sum);
    }
    const int64_t at64 = lane < p.K ? p.idx[(int64_t)t * p.K + lane] : -1;
    const int at = at64 >= 0 && at64 < p.E ? (int)at64 : -1;
    const float l = at < 0 ? kNegInf : load_logit<BF16>(row, at);
    const bool none = l == kNegInf;
    float d = none ? 0.0f : p.grad[(int64_t)t * p.K + lane] * p.scale;
    float dot = 0.0f;
    if (p.renorm) {
      // u = p / sum p; du_k/dl_k' carries p' / sum = u (1 - p) for a sigmoid,
      // and u for a softmax (its share of the chosen alone)
      const float u = choice_weight(none, l, p.sigmoid, true, 0.0f, 1.0f);
      d = u * (d - warp_sum(d * u));
      if (p.sigmoid) d *= none ? 0.0f : 1.0f / (1.0f + expf(l));
    } else if (p.sigmoid) {
      const float e = expf(-fabsf(l));  // p (1 - p) = e / (1 + e)^2
      d = none ? 0.0f : d * (e / ((1.0f + e) * (1.0f + e)));
    } else {
      dot = warp_sum(none ? 0.0f : d * (expf(l - m) / sum));
    }
    __syncwarp();
    for (int k = 0; k < p.K; ++k) {  // one lane after the other: an index named twice adds up
      if (lane == k && !none) dense[at] += d;
      __syncwarp();
    }
    for (int j = lane; j < p.E; j += 32) {
      float v = dense[j];
      if (!p.sigmoid && !p.renorm) {
        const float lj = load_logit<BF16>(row, j);
        v = lj == kNegInf ? 0.0f : (expf(lj - m) / sum) * (v - dot);
      }
      store_grad<BF16>(out, j, v);
    }
    __syncwarp();
  }
}

template <typename K>
ep_status_t route_grid(K kernel, int T, int E, const DeviceInfo *di, int *grid, size_t *smem) {
  *smem = (size_t)kRouteWarps * E * sizeof(float);
  if (*smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)*smem);
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
  }
  const int64_t need = ((int64_t)T + kRouteWarps - 1) / kRouteWarps;
  const int64_t most = (int64_t)di->num_sms * 16;
  *grid = (int)(need < most ? need : most);
  return EP_OK;
}

}  // namespace

ep_status_t launch_route(const RouteArgs &a, cudaStream_t stream) {
  if (a.num_tokens == 0) return EP_OK;
  const DeviceInfo *di = current_device_info();
  if (di == nullptr) return EP_ERR_CUDA;
  RouteParams p;
  p.logits = a.logits;
  p.row_stride = a.row_stride;
  p.T = a.num_tokens;
  p.E = a.num_experts;
  p.K = a.num_topk;
  p.bias = a.bias;
  p.G = a.num_groups;
  p.Gk = a.topk_groups;
  p.group_top = a.group_top;
  p.scale = a.weight_scale;
  p.idx = a.topk_idx;
  p.w = a.topk_weights;
  p.sigmoid = a.sigmoid;
  p.renorm = a.renormalize;
  // Scores rise with their logits, so without biases, and where groups are
  // judged by their best expert, the logits themselves are compared: exact,
  // where scores far below the largest would round together.
  p.by_logit = a.bias == nullptr && (a.num_groups == 1 || a.group_top == 1);
  auto kernel = a.bf16 ? route_kernel<true> : route_kernel<false>;
  int grid;
  size_t smem;
  const ep_status_t s = route_grid(kernel, a.num_tokens, a.num_experts, di, &grid, &smem);
  if (s != EP_OK) return s;
  const cudaError_t e = launch_kernel(kernel, grid, kRouteWarps * 32, smem, stream, false, p);
  return e == cudaSuccess ? EP_OK : cuda_fail(e, "route launch");
}

ep_status_t launch_route_backward(const RouteBackwardArgs &a, cudaStream_t stream) {
  if (a.num_tokens == 0) return EP_OK;
  const DeviceInfo *di = current_device_info();
  if (di == nullptr) return EP_ERR_CUDA;
  RouteBackwardParams p{a.grad_weights, a.logits, a.row_stride,   a.topk_idx, a.num_tokens, a.num_experts,
                        a.num_topk,     a.weight_scale, a.grad_logits, a.sigmoid,  a.renormalize};
  auto kernel = a.bf16 ? route_backward_kernel<true> : route_backward_kernel<false>;
  int grid;
  size_t smem;
  const ep_status_t s = route_grid(kernel, a.num_tokens, a.num_experts, di, &grid, &smem);
  if (s != EP_OK) return s;
  const cudaError_t e = launch_kernel(kernel, grid, kRouteWarps * 32, smem, stream, false, p);
  return e == cudaSuccess ? EP_OK : cuda_fail(e, "route_backward launch");
}

}  // namespace ep
