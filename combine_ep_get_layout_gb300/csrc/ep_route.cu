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
#include <atomic>

#include "ep_device.cuh"
#include "ep_ops.h"

namespace ep {

namespace {

constexpr int kRouteWarps = 4;
constexpr int kLanesTokens = 2048;
constexpr int kLaneWarps = 4;
constexpr int kLoads = 8;  // of 16 bytes in flight a lane
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

// ------------------------------------------------------------- many tokens
// A lane a token: no exchange between lanes, and a selection by sorting
// networks, whose steps are one minimum and one maximum.  32 rows lie in
// shared memory, pieces of 16 bytes at (piece ^ (row & 7)), so that the lanes
// read the same place of their rows without conflicts.  The networks sort
// words of a key's upper bits over the complement of its index (ties go to
// the lowest); the few words found are then ordered by their keys, and where
// the upper bits alone cannot tell the last choice from what was left out, the
// row is searched again by whole keys.

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

constexpr float kLog2e = 1.4426950408889634f;

// Scores for keys, a few units in the last place from the weights' own.
__device__ __forceinline__ float sigmoid_key(float l) { return rcp_approx(1.0f + exp2_approx(-l * kLog2e)); }

template <int N>
__device__ __forceinline__ void merge_words(uint32_t (&w)[N]) {  // a bitonic sequence, to descending order
#pragma unroll
  for (int d = N / 2; d > 0; d >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i)
      if ((i & d) == 0) {
        const uint32_t a = w[i], b = w[i + d];
        w[i] = max(a, b);
        w[i + d] = min(a, b);
      }
}

template <int N>
__device__ __forceinline__ void sort_words(uint32_t (&w)[N]) {  // to descending order
#pragma unroll
  for (int size = 2; size <= N; size <<= 1)
#pragma unroll
    for (int d = size / 2; d > 0; d >>= 1)
#pragma unroll
      for (int i = 0; i < N; ++i)
        if ((i & d) == 0) {
          const bool down = (i & size) == 0 || size == N;
          const uint32_t a = w[i], b = w[i + d];
          w[i] = down ? max(a, b) : min(a, b);
          w[i + d] = down ? min(a, b) : max(a, b);
        }
}

// top: the N largest of top and w (both descending); out: the largest of the others.
template <int N>
__device__ __forceinline__ void join_words(uint32_t (&top)[N], uint32_t (&w)[N], uint32_t &out) {
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const uint32_t a = w[N - 1 - i], b = w[i];
    out = max(out, max(min(top[i], a), min(top[N - 1 - i], b)));
    top[i] = max(top[i], a);
    top[N - 1 - i] = max(top[N - 1 - i], b);
  }
  merge_words(top);
}

// kLaneWarps warps take 32 tokens together: each looks through a share of
// every row, the first joins what they found.  p.logits' rows are `aligned`
// where all of them are made of whole 16-byte pieces.
template <bool BF16, int N>
__global__ void __launch_bounds__(kLaneWarps * 32) route_lanes_kernel(RouteParams p, int pitch, int bits, bool aligned) {
  extern __shared__ float4 s_rows4[];
  float *rows = reinterpret_cast<float *>(s_rows4);
  uint32_t *words = reinterpret_cast<uint32_t *>(rows + 32 * pitch);  // [kLaneWarps][N + 1][32]
  float *bias = reinterpret_cast<float *>(words + kLaneWarps * (N + 1) * 32);  // [pitch]
  float *scores = bias + pitch;                                                // [groups][32]
  __shared__ float s_part[2][kLaneWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, quads = (p.E + 3) / 4;
  const int t0 = blockIdx.x * 32, count = min(32, p.T - t0);
  const auto quad_at = [&](int row, int q) { return row * pitch + ((q ^ (row & 7)) << 2); };
  griddep_wait();
  griddep_launch_dependents();

  // the rows, as fp32; NaN counts as masked, +infinity as the largest number
  const auto clean = [](float v) { return fminf(v != v ? kNegInf : v, 3.402823466e38f); };
  const int64_t step = p.row_stride * (BF16 ? 2 : 4);
  const char *base = static_cast<const char *>(p.logits) + (int64_t)t0 * step;
  if (aligned) {
    const int pieces = BF16 ? p.E / 8 : quads;
    for (int i = threadIdx.x; i < count * pieces; i += kLaneWarps * 32 * kLoads) {
      int4 v[kLoads];
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        const int at = i + kLaneWarps * 32 * j, r = at / pieces, c = at - r * pieces;
        if (at < count * pieces) v[j] = __ldcs(reinterpret_cast<const int4 *>(base + r * step + c * 16));
      }
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        const int at = i + kLaneWarps * 32 * j, r = at / pieces, c = at - r * pieces;
        if (at >= count * pieces) break;
        const uint32_t *w = reinterpret_cast<const uint32_t *>(&v[j]);
        if (BF16) {
          *reinterpret_cast<float4 *>(rows + quad_at(r, 2 * c)) =
              make_float4(clean(bf16_lo(w[0])), clean(bf16_hi(w[0])), clean(bf16_lo(w[1])), clean(bf16_hi(w[1])));
          *reinterpret_cast<float4 *>(rows + quad_at(r, 2 * c + 1)) =
              make_float4(clean(bf16_lo(w[2])), clean(bf16_hi(w[2])), clean(bf16_lo(w[3])), clean(bf16_hi(w[3])));
        } else {
          *reinterpret_cast<float4 *>(rows + quad_at(r, c)) =
              make_float4(clean(__uint_as_float(w[0])), clean(__uint_as_float(w[1])), clean(__uint_as_float(w[2])),
                          clean(__uint_as_float(w[3])));
        }
      }
    }
  } else {
#pragma unroll 8
    for (int i = threadIdx.x; i < count * quads * 4; i += kLaneWarps * 32) {
      const int r = i / (quads * 4), e = i - r * quads * 4;
      rows[quad_at(r, e >> 2) + (e & 3)] = e < p.E ? load_logit<BF16>(base + r * step, e) : kNegInf;
    }
  }
  for (int i = threadIdx.x; i < pitch; i += kLaneWarps * 32) bias[i] = p.bias != nullptr && i < p.E ? p.bias[i] : 0.0f;
  __syncthreads();

  const bool here = lane < count;
  const int q0 = quads * warp / kLaneWarps, q1 = quads * (warp + 1) / kLaneWarps;  // this warp's share of a row
  const auto read4 = [&](int q, float (&v)[4]) {
    const float4 f = *reinterpret_cast<const float4 *>(rows + quad_at(lane, q));
    v[0] = f.x;
    v[1] = f.y;
    v[2] = f.z;
    v[3] = f.w;
  };
  float m = 0.0f, sum = 1.0f;
  if (!p.sigmoid && !(p.by_logit && p.renorm)) {
    m = kNegInf;
    if (here)
#pragma unroll 4
      for (int q = q0; q < q1; ++q) {
        float v[4];
        read4(q, v);
        m = fmaxf(fmaxf(m, fmaxf(v[0], v[1])), fmaxf(v[2], v[3]));
      }
    s_part[0][warp][lane] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kLaneWarps; ++w) m = fmaxf(m, s_part[0][w][lane]);
    sum = 0.0f;
    if (here && m != kNegInf)
#pragma unroll 4
      for (int q = q0; q < q1; ++q) {
        float v[4];
        read4(q, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) sum += exp2_approx((v[j] - m) * kLog2e);
      }
    s_part[1][warp][lane] = sum;
    __syncthreads();
    sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kLaneWarps; ++w) sum += s_part[1][w][lane];
  }
  // keys in place of logits, and the groups' scores: a warp some groups, or
  // of a single group its share of the row
  const int per = p.E / p.G / 4;  // quads of a group
  if (!p.by_logit || p.G > 1) {
    const float inv = 1.0f / sum;
    for (int g = p.G == 1 ? 0 : warp; here && g < p.G; g += kLaneWarps) {
      float a = kNegInf, b = kNegInf;
      const int from = p.G == 1 ? q0 : g * per, to = p.G == 1 ? q1 : (g + 1) * per;
#pragma unroll 4
      for (int q = from; q < to; ++q) {
        float v[4];
        read4(q, v);
        if (!p.by_logit) {
          const float4 c = *reinterpret_cast<const float4 *>(bias + q * 4);
          const float more[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float key = (p.sigmoid ? sigmoid_key(v[j]) : exp2_approx((v[j] - m) * kLog2e) * inv) + more[j];
            v[j] = v[j] == kNegInf || key != key ? kNegInf : key;
          }
          *reinterpret_cast<float4 *>(rows + quad_at(lane, q)) = make_float4(v[0], v[1], v[2], v[3]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          b = fmaxf(b, fminf(a, v[j]));
          a = fmaxf(a, v[j]);
        }
      }
      if (p.G == 1) break;
      scores[g * 32 + lane] = p.group_top == 2 && b != kNegInf ? a + b : a;
    }
    __syncthreads();
  }
  uint64_t offered = p.G == 1 && here ? 1ull : 0ull;
  if (p.G > 1 && here)
    for (int k = 0; k < p.Gk; ++k) {
      float best = kNegInf;
      int at = -1;
#pragma unroll 4
      for (int g = 0; g < p.G; ++g) {
        const float v = scores[g * 32 + lane];
        if (v > best && !((offered >> g) & 1ull)) {
          best = v;
          at = g;
        }
      }
      if (at < 0) break;
      offered |= 1ull << at;
    }

  // this warp's share of the offered groups, one after the other: the N
  // largest words, and the largest of the others
  const uint32_t low = (1u << bits) - 1u;
  uint32_t top[N] = {}, out = 0u;
  const int length = p.G == 1 ? quads : per, all = length * p.Gk;
  const int i1 = all * (warp + 1) / kLaneWarps;
  int i = all * warp / kLaneWarps, in = i % length;
  uint64_t left = offered;
  for (int k = i / length; k > 0; --k) left &= left - 1ull;
  while (i < i1) {
    uint32_t w[N];
#pragma unroll
    for (int n = 0; n < N / 4; ++n) {
      float v[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
      int at = 0;
      if (i < i1) {
        if (left != 0ull) {
          at = (__ffsll((long long)left) - 1) * length + in;
          read4(at, v);
        }
        ++i;
        if (++in == length) {
          in = 0;
          left &= left - 1ull;
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[n * 4 + j] = v[j] == kNegInf ? 0u : (ordered(v[j]) & ~low) | (low - (uint32_t)(at * 4 + j));
    }
    sort_words(w);
    join_words(top, w, out);
  }
  uint32_t *mine = words + warp * (N + 1) * 32 + lane;
  if (warp > 0) {
#pragma unroll
    for (int n = 0; n < N; ++n) mine[n * 32] = top[n];
    mine[N * 32] = out;
  }
  __syncthreads();
  if (warp == 0) {
    for (int o = 1; o < kLaneWarps; ++o) {
      const uint32_t *other = words + o * (N + 1) * 32 + lane;
      uint32_t w[N];
#pragma unroll
      for (int n = 0; n < N; ++n) w[n] = other[n * 32];
      out = max(out, other[N * 32]);
      join_words(top, w, out);
    }

    float key[N];
    int idx[N];
    bool alike = false;  // words of the same upper bits
    uint32_t last = 0u;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      idx[n] = top[n] == 0u ? -1 : (int)(low - (top[n] & low));
      if (n > 0) alike = alike || (top[n] != 0u && (top[n] & ~low) == (top[n - 1] & ~low));
      if (n == p.K - 1) last = top[n];
    }
    if (alike) {
      // by whole keys: descending, ties to the lowest index
#pragma unroll
      for (int n = 0; n < N; ++n) key[n] = idx[n] < 0 ? kNegInf : rows[quad_at(lane, idx[n] >> 2) + (idx[n] & 3)];
#pragma unroll
      for (int round = 0; round < N; ++round)
#pragma unroll
        for (int n = round & 1; n + 1 < N; n += 2)
          if (key[n + 1] > key[n] || (key[n + 1] == key[n] && (uint32_t)idx[n + 1] < (uint32_t)idx[n])) {
            const float k = key[n];
            const int x = idx[n];
            key[n] = key[n + 1];
            idx[n] = idx[n + 1];
            key[n + 1] = k;
            idx[n + 1] = x;
          }
    }
    if (out != 0u && (out & ~low) == (last & ~low) && !(BF16 && p.by_logit)) {
#pragma unroll
      for (int n = 0; n < N; ++n) {
        key[n] = kNegInf;
        idx[n] = -1;
      }
      for (left = offered; left != 0ull; left &= left - 1ull) {
        const int g = __ffsll((long long)left) - 1;
        for (int e = g * length * 4; e < (g + 1) * length * 4; ++e) {
          const float v = rows[quad_at(lane, e >> 2) + (e & 3)];
          if (!(v > key[N - 1])) continue;
#pragma unroll
          for (int n = N - 1; n > 0; --n) {
            const bool up = v > key[n - 1], here_in = v > key[n];
            idx[n] = up ? idx[n - 1] : here_in ? e : idx[n];
            key[n] = up ? key[n - 1] : here_in ? v : key[n];
          }
          if (v > key[0]) {
            key[0] = v;
            idx[0] = e;
          }
        }
      }
    }

    // weights, as in choice_weight
    float l[N], w[N], most = kNegInf;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const bool some = here && n < p.K && idx[n] >= 0;
      l[n] = !some          ? kNegInf
             : p.by_logit ? rows[quad_at(lane, idx[n] >> 2) + (idx[n] & 3)]
                          : load_logit<BF16>(base + lane * step, idx[n]);
    }
#pragma unroll
    for (int n = 0; n < N; ++n) most = fmaxf(most, p.sigmoid ? fminf(l[n], 0.0f) : l[n]);
    if (!p.renorm) most = p.sigmoid ? 0.0f : m;
    float total = 0.0f;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const bool some = l[n] != kNegInf;
      if (p.sigmoid)
        w[n] = some ? expf(fminf(l[n], 0.0f) - most) / (1.0f + expf(-fabsf(l[n]))) : 0.0f;
      else
        w[n] = some ? expf(l[n] - most) : 0.0f;
      total += w[n];
    }
    if (!p.renorm) total = p.sigmoid ? 1.0f : sum;
    __syncwarp();
    // through shared memory: the rows' choices are one run of memory
    int64_t *s_idx = reinterpret_cast<int64_t *>(rows);
    float *s_w = reinterpret_cast<float *>(s_idx + 32 * N);
#pragma unroll
    for (int n = 0; n < N; ++n)
      if (n < p.K) {
        s_idx[lane * p.K + n] = here ? idx[n] : -1;
        s_w[lane * p.K + n] = total > 0.0f ? w[n] / total * p.scale : 0.0f;
      }
    __syncwarp();
    for (int n = lane; n < count * p.K; n += 32) {
      p.idx[(int64_t)t0 * p.K + n] = s_idx[n];
      p.w[(int64_t)t0 * p.K + n] = s_w[n];
    }
  }
}

// Where a lane a token is used: enough tokens that their warps fill the SMs
// (with fewer, a warp a token answers sooner), rows that fit beside each
// other, at most 16 choices, groups of whole quads.
bool lanes_fit(const RouteArgs &a) {
  return a.num_tokens >= kLanesTokens && a.num_experts <= 1024 && a.num_topk <= 16 &&
         (a.num_groups == 1 || a.num_experts / a.num_groups % 4 == 0);
}

template <bool BF16, int N>
ep_status_t launch_lanes(const RouteParams &p, cudaStream_t stream) {
  const int pitch = (p.E + 31) / 32 * 32;
  int bits = 1;
  while ((1 << bits) < pitch) ++bits;
  size_t smem = ((size_t)33 * pitch + kLaneWarps * (N + 1) * 32 + (p.G > 1 ? p.G * 32 : 0)) * 4;
  if (smem < 32 * N * 12) smem = 32 * N * 12;
  static std::atomic<bool> ready[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && !ready[dev]) {
    e = cudaFuncSetAttribute(route_lanes_kernel<BF16, N>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (33 * 1024 + kLaneWarps * (N + 1) * 32 + EP_MAX_RANKS * 32) * 4);
    if (e == cudaSuccess) ready[dev] = true;
  }
  const bool aligned = reinterpret_cast<uintptr_t>(p.logits) % 16 == 0 &&
                       p.row_stride % (BF16 ? 8 : 4) == 0 && p.E % (BF16 ? 8 : 4) == 0;
  if (e == cudaSuccess)
    e = launch_kernel(route_lanes_kernel<BF16, N>, (p.T + 31) / 32, kLaneWarps * 32, smem, stream, false, p, pitch,
                      bits, aligned);
  return e == cudaSuccess ? EP_OK : cuda_fail(e, "route launch");
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
  if (lanes_fit(a)) {
    if (a.num_topk <= 8) return a.bf16 ? launch_lanes<true, 8>(p, stream) : launch_lanes<false, 8>(p, stream);
    return a.bf16 ? launch_lanes<true, 16>(p, stream) : launch_lanes<false, 16>(p, stream);
  }
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
