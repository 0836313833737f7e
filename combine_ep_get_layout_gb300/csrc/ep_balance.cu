// The losses that balance a router, each expert's counts, and their gradient
// for the logits.
//
//   p = softmax(l), or sigmoid(l) / sum sigmoid(l)
//   balance = 1/S' sum over sequences of E sum_e share[e] mean_t p[t,e]
//   z = 1/N sum_t log(sum_e exp(l[t,e]))^2
//   d balance / d p[t,e] = slope[s,e] = E share[s,e] / (S' n_s)
//   d l: softmax p (slope - sum p slope), sigmoid the same times 1 - sigmoid(l)
//        + 2/N log-sum-exp softmax(l)
//
// The sums over tokens run in a fixed order: a block's part of a sequence
// first (a "segment"; block b's of sequence s is segment b + s, since later
// blocks hold later sequences), then the segments.
#include "ep_device.cuh"
#include "ep_ops.h"

namespace ep {

namespace {

constexpr int kThreads = 256;
constexpr float kNegInf = -__builtin_huge_valf();

// A logit in fp32: NaN counts as masked, +infinity as the largest number.
__device__ __forceinline__ float load_logit(const void *p, bool bf16, int64_t i) {
  float v = bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t *>(p)[i] << 16) : static_cast<const float *>(p)[i];
  v = v != v ? kNegInf : v;
  return fminf(v, 3.402823466e38f);
}

template <typename Op>
__device__ __forceinline__ float block_reduce(float v, float *s, Op op) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  v = s[0];
  for (int i = 1; i < (int)blockDim.x / 32; ++i) v = op(v, s[i]);
  return v;
}

struct Sum {
  __device__ float operator()(float a, float b) const { return a + b; }
};
struct Max {
  __device__ float operator()(float a, float b) const { return fmaxf(a, b); }
};

// What a row's scores need: softmax e^(l - m) / soft, sigmoid scores
// e^(min(l, 0) - k) / (1 + e^-|l|) / sig.
struct Row {
  float m, soft, k, sig;
  __device__ float softmax(float l) const { return soft > 0.0f ? expf(l - m) / soft : 0.0f; }
  __device__ float sigmoid(float l) const {
    return sig > 0.0f && l > kNegInf ? expf(fminf(l, 0.0f) - k) / (1.0f + expf(-fabsf(l))) / sig : 0.0f;
  }
  __device__ float lse() const { return soft > 0.0f ? m + logf(soft) : 0.0f; }
};

__device__ Row row_of(const void *logits, bool bf16, int64_t at, int E, bool sigmoid, float *s) {
  Row r;
  float m = kNegInf, sum = 0.0f, sig = 0.0f;
  for (int e = threadIdx.x; e < E; e += kThreads) m = fmaxf(m, load_logit(logits, bf16, at + e));
  r.m = block_reduce(m, s, Max());
  r.k = fminf(r.m, 0.0f);
  if (r.m > kNegInf) {
    for (int e = threadIdx.x; e < E; e += kThreads) {
      const float l = load_logit(logits, bf16, at + e);
      sum += expf(l - r.m);
      if (sigmoid) sig += l > kNegInf ? expf(fminf(l, 0.0f) - r.k) / (1.0f + expf(-fabsf(l))) : 0.0f;
    }
  }
  r.soft = block_reduce(sum, s, Sum());
  r.sig = block_reduce(sig, s, Sum());
  return r;
}

__device__ __forceinline__ int offset_of(const int32_t *offsets, int T, int s) {
  return offsets == nullptr ? (s == 0 ? 0 : T) : min(max(offsets[s], 0), T);
}

constexpr int kTokens = 64;  // of a block

int blocks_of(int T) { return (T + kTokens - 1) / kTokens; }

struct Parts {
  float *probs;    // [segments][E]
  int32_t *counts; // [segments][E]
  float *z;        // [segments]
};

__global__ void __launch_bounds__(kThreads) balance_kernel(BalanceArgs p, Parts parts) {
  __shared__ float s_reduce[kThreads / 32];
  __shared__ float s_probs[EP_MAX_EXPERTS];
  __shared__ int32_t s_counts[EP_MAX_EXPERTS];
  griddep_wait();
  griddep_launch_dependents();
  const int t0 = blockIdx.x * kTokens, t1 = min(p.num_tokens, t0 + kTokens);
  for (int s = 0; s < p.num_sequences; ++s) {
    const int a = max(t0, offset_of(p.seq_offsets, p.num_tokens, s));
    const int b = min(t1, offset_of(p.seq_offsets, p.num_tokens, s + 1));
    if (a >= b) continue;
    for (int e = threadIdx.x; e < p.num_experts; e += kThreads) {
      s_probs[e] = 0.0f;
      s_counts[e] = 0;
    }
    __syncthreads();
    float z = 0.0f;
    for (int t = a; t < b; ++t) {
      const int64_t at = t * p.row_stride;
      const Row r = row_of(p.logits, p.bf16, at, p.num_experts, p.sigmoid, s_reduce);
      for (int e = threadIdx.x; e < p.num_experts; e += kThreads) {
        const float l = load_logit(p.logits, p.bf16, at + e);
        s_probs[e] += p.sigmoid ? r.sigmoid(l) : r.softmax(l);
      }
      z += r.lse() * r.lse();
    }
    for (int64_t i = (int64_t)a * p.num_topk + threadIdx.x; i < (int64_t)b * p.num_topk; i += kThreads) {
      const int64_t e = p.topk_idx[i];
      if (e >= 0 && e < p.num_experts) atomicAdd(&s_counts[e], 1);
    }
    __syncthreads();
    const int64_t segment = blockIdx.x + s;
    for (int e = threadIdx.x; e < p.num_experts; e += kThreads) {
      parts.probs[segment * p.num_experts + e] = s_probs[e];
      parts.counts[segment * p.num_experts + e] = s_counts[e];
    }
    if (threadIdx.x == 0) parts.z[segment] = z;
    __syncthreads();
  }
}

__global__ void __launch_bounds__(kThreads) balance_join_kernel(BalanceArgs p, Parts parts) {
  __shared__ float s_reduce[kThreads / 32];
  __shared__ int s_bad;
  griddep_wait();
  griddep_launch_dependents();
  const int E = p.num_experts, S = p.num_sequences;
  if (threadIdx.x == 0) s_bad = 0;
  __syncthreads();
  int full = 0;
  bool bad = false;
  for (int s = 0; s < S; ++s) {
    const int a = offset_of(p.seq_offsets, p.num_tokens, s), b = offset_of(p.seq_offsets, p.num_tokens, s + 1);
    full += b > a;
    if (p.seq_offsets != nullptr)
      bad = bad || p.seq_offsets[s] < 0 || p.seq_offsets[s] > p.seq_offsets[s + 1] || p.seq_offsets[s + 1] > p.num_tokens;
  }
  float balance = 0.0f, z = 0.0f;
  int tokens = 0;
  for (int s = 0; s < S; ++s) {
    const int a = offset_of(p.seq_offsets, p.num_tokens, s), b = offset_of(p.seq_offsets, p.num_tokens, s + 1);
    const int b0 = a / kTokens, b1 = b > a ? (b - 1) / kTokens : b0 - 1;
    float chosen = 0.0f;
    for (int e = threadIdx.x; e < E; e += kThreads) {
      float prob = 0.0f;
      int count = 0;
      for (int i = b0; i <= b1; ++i) {
        prob += parts.probs[(int64_t)(i + s) * E + e];
        count += parts.counts[(int64_t)(i + s) * E + e];
      }
      p.probs[(int64_t)s * E + e] = b > a ? prob / (b - a) : 0.0f;
      p.counts[(int64_t)s * E + e] = count;
      chosen += count;
    }
    if (b > a) {
      tokens += b - a;
      for (int i = b0; i <= b1; ++i) z += parts.z[i + s];
    }
    chosen = block_reduce(chosen, s_reduce, Sum());
    float part = 0.0f;
    for (int e = threadIdx.x; e < E; e += kThreads) {
      const float share = chosen > 0.0f ? (float)E * p.counts[(int64_t)s * E + e] / chosen / full : 0.0f;
      p.slopes[(int64_t)s * E + e] = b > a ? share / (b - a) : 0.0f;
      part += share * p.probs[(int64_t)s * E + e];
    }
    balance += block_reduce(part, s_reduce, Sum());
  }
  if (threadIdx.x == 0) {
    const float nan = __int_as_float(0x7fffffff);
    p.losses[0] = bad ? nan : balance;
    p.losses[1] = bad ? nan : tokens > 0 ? z / tokens : 0.0f;
  }
}

__device__ __forceinline__ void store_grad(void *p, bool bf16, int64_t i, float v) {
  if (bf16)
    static_cast<uint16_t *>(p)[i] = (uint16_t)(pack_bf16x2(v, 0.0f) & 0xffffu);
  else
    static_cast<float *>(p)[i] = v;
}

__global__ void __launch_bounds__(kThreads) balance_backward_kernel(BalanceBackwardArgs p) {
  __shared__ float s_reduce[kThreads / 32];
  griddep_wait();
  griddep_launch_dependents();
  const int E = p.num_experts, S = p.num_sequences;
  const int first = offset_of(p.seq_offsets, p.num_tokens, 0), last = offset_of(p.seq_offsets, p.num_tokens, S);
  const float db = p.grad_losses[0], dz = p.grad_losses[1] * 2.0f / max(1, last - first);
  for (int64_t t = blockIdx.x; t < p.num_tokens; t += gridDim.x) {
    int s = 0;
    while (s < S && offset_of(p.seq_offsets, p.num_tokens, s + 1) <= t) ++s;
    const bool inside = s < S && t >= first;
    Row r = {};
    float dot = 0.0f;
    const float *slope = p.slopes + (int64_t)min(s, S - 1) * E;
    const auto score = [&](float l) { return p.sigmoid ? r.sigmoid(l) : r.softmax(l); };
    if (inside) {
      r = row_of(p.logits, p.bf16, t * p.row_stride, E, p.sigmoid, s_reduce);
      for (int e = threadIdx.x; e < E; e += kThreads)
        dot += score(load_logit(p.logits, p.bf16, t * p.row_stride + e)) * slope[e];
      dot = block_reduce(dot, s_reduce, Sum());
    }
    for (int e = threadIdx.x; e < E; e += kThreads) {
      float d = 0.0f;
      if (inside) {
        const float l = load_logit(p.logits, p.bf16, t * p.row_stride + e);
        d = db * score(l) * (slope[e] - dot);
        if (p.sigmoid) d *= 1.0f / (1.0f + expf(l));
        d += dz * r.lse() * r.softmax(l);
      }
      if (p.add != nullptr)
        d += p.bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t *>(p.add)[t * E + e] << 16)
                    : static_cast<const float *>(p.add)[t * E + e];
      store_grad(p.grad_logits, p.bf16, t * E + e, d);
    }
  }
}

size_t round16(size_t n) { return (n + 15) / 16 * 16; }

}  // namespace

size_t balance_workspace_bytes(int T, int E, int S) {
  const size_t segments = (size_t)blocks_of(T) + S;
  return 2 * round16(segments * E * 4) + round16(segments * 4);
}

ep_status_t launch_balance(const BalanceArgs &a, cudaStream_t stream) {
  const size_t segments = (size_t)blocks_of(a.num_tokens) + a.num_sequences, matrix = round16(segments * a.num_experts * 4);
  char *at = static_cast<char *>(a.workspace);
  const Parts parts{reinterpret_cast<float *>(at), reinterpret_cast<int32_t *>(at + matrix),
                    reinterpret_cast<float *>(at + 2 * matrix)};
  cudaError_t e = cudaSuccess;
  if (a.num_tokens > 0) e = launch_kernel(balance_kernel, blocks_of(a.num_tokens), kThreads, 0, stream, false, a, parts);
  if (e == cudaSuccess) e = launch_kernel(balance_join_kernel, 1, kThreads, 0, stream, false, a, parts);
  return e == cudaSuccess ? EP_OK : cuda_fail(e, "balance launch");
}

ep_status_t launch_balance_backward(const BalanceBackwardArgs &a, cudaStream_t stream) {
  if (a.num_tokens == 0) return EP_OK;
  const int grid = a.num_tokens < 65536 ? a.num_tokens : 65536;
  const cudaError_t e = launch_kernel(balance_backward_kernel, grid, kThreads, 0, stream, false, a);
  return e == cudaSuccess ? EP_OK : cuda_fail(e, "balance_backward launch");
}

}  // namespace ep
