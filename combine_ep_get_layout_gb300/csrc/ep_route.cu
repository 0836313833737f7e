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
constexpr int kLaneWarps = 4;
constexpr int kManyExperts = 64;  // from here on a lane takes a token whatever their number
constexpr float kMost = 3.402823466e38f;
constexpr uint32_t kLeast = 0x00800000u;  // order_of the lowest number, its low bits cleared
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

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

constexpr float kLog2e = 1.4426950408889634f;

// Keys, the same in both kernels, so that a token's choice does not hang on
// the size of its batch.  The approximations are a few units in the last
// place from the weights' own exponentials (rounding l - m alone moves a
// softmax as much); scores below 2^-126 count as 0.
__device__ __forceinline__ float sigmoid_key(float l, float bias) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + exp2_approx(-l * kLog2e)));
  return r + bias;
}

__device__ __forceinline__ float softmax_part(float l, float m) { return l == kNegInf ? 0.0f : exp2_approx((l - m) * kLog2e); }
__device__ __forceinline__ float softmax_key(float l, float m, float inv, float bias) {
  return fmaf(exp2_approx((l - m) * kLog2e), inv, bias);
}

// Order-preserving map of a float (no NaN) to an unsigned integer.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);  // -0 counts as +0
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// The same for a float that is not -0.
__device__ __forceinline__ uint32_t order_of(float v) {
  const int b = __float_as_int(v);
  return (uint32_t)(b ^ ((b >> 31) | (int)0x80000000));
}

__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Over L neighbouring lanes; the whole warp calls them.
template <int L = 32>
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int L = 32>
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
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
template <int L = 32>
__device__ __forceinline__ float choice_weight(bool none, float l, bool sigmoid, bool renorm, float m, float sum) {
  float p;
  if (sigmoid) {
    const float low = fminf(l, 0.0f);
    const float top = renorm ? warp_max<L>(none ? kNegInf : low) : 0.0f;
    p = none ? 0.0f : expf(low - top) / (1.0f + expf(-fabsf(l)));
  } else {
    const float top = renorm ? warp_max<L>(none ? kNegInf : l) : m;
    p = none ? 0.0f : expf(l - top);
    if (!renorm) p = none ? 0.0f : p / sum;
  }
  if (renorm) {
    const float total = warp_sum<L>(p);
    p = total > 0.0f ? p / total : 0.0f;
  }
  return p;
}

// One warp a token; the keys of its row in shared memory, a round of argmax a
// choice.  8 experts, top-2: 2.7 us up to 2048 tokens, latency.
template <bool BF16>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(RouteParams p) {
  extern __shared__ float s_keys[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float *key = s_keys + (size_t)warp * p.E;
  griddep_wait();
  griddep_launch_dependents();
  for (int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp; t < p.T; t += (int64_t)gridDim.x * kRouteWarps) {
    const void *row = static_cast<const char *>(p.logits) + (int64_t)t * p.row_stride * (BF16 ? 2 : 4);
    float m = kNegInf, sum = 0.0f;
    for (int j = lane; j < p.E; j += 32) {
      const float l = load_logit<BF16>(row, j);
      key[j] = l;
      m = fmaxf(m, l);
    }
    m = warp_max(m);
    if (!p.sigmoid && (!p.by_logit || !p.renorm)) {
      if (p.E < kManyExperts && !p.by_logit) {
        // keys: in the order of route_lanes_kernel, which takes the larger
        // batches (4096 tokens, 60 experts: 10.9 us, in the warp's order 10.5)
        __syncwarp();
        const int quads = (p.E + 3) / 4;
        if (lane < kLaneWarps)
          for (int j = quads * lane / kLaneWarps * 4; j < min(quads * (lane + 1) / kLaneWarps * 4, p.E); ++j)
            sum += softmax_part(key[j], m);
        const float own = sum;
        sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kLaneWarps; ++w) sum += __shfl_sync(0xffffffffu, own, w);
        __syncwarp();  // before the keys take the logits' place
      } else {
        for (int j = lane; j < p.E; j += 32) sum += softmax_part(key[j], m);
        sum = warp_sum(sum);
      }
    }
    const float inv = 1.0f / sum;
    if (!p.by_logit)
      for (int j = lane; j < p.E; j += 32) {
        const float l = key[j], bias = p.bias != nullptr ? p.bias[j] : 0.0f;
        const float v = p.sigmoid ? sigmoid_key(l, bias) : softmax_key(l, m, inv, bias);
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

// ---------------------------------------------------------- a lane a token
// A lane a token: no exchange between lanes, and a selection by sorting
// networks, whose steps are one minimum and one maximum.  32 rows lie in
// shared memory an odd number of 16-byte pieces apart, so that the lanes read
// the same place of their rows without conflicts.  The networks sort words:
// a key's place below the row's largest, in fixed point (23 bits of a window
// of kWindow; bf16 logits: their own 16 bits), over the complement of its
// index, so that ties go to the lowest.  Words of the same place are then
// ordered by their keys, and where the places alone cannot tell the last
// choice from what was left out (some 1e-4 of the tokens), or the window does
// not reach it, the row is searched again by whole keys.  Both hang on the
// logits: N(0, 1.5^2) for the 1e-4; ten times as wide, groups judged by two
// scores without biases take 66 us instead of 35, logits as keys 42 instead of
// 30, and scores with biases no longer.

enum KeyKind { kLogitKey, kSigmoidKey, kSoftmaxKey };

__device__ __forceinline__ void order_words(uint32_t &a, uint32_t &b) {
  const uint32_t x = max(a, b);
  b = min(a, b);
  a = x;
}

// Words L ... L + N - 1, a bitonic sequence, to descending order.
template <int L, int N, int M>
__device__ __forceinline__ void merge_words(uint32_t (&w)[M]) {
  if constexpr (N > 1) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) order_words(w[L + i], w[L + N / 2 + i]);
    merge_words<L, N / 2>(w);
    merge_words<L + N / 2, N / 2>(w);
  }
}

// Words L ... L + 7 to descending order, Batcher's odd-even merge sort.
template <int L, int M>
__device__ __forceinline__ void sort_eight(uint32_t (&w)[M]) {
  order_words(w[L + 0], w[L + 1]); order_words(w[L + 2], w[L + 3]); order_words(w[L + 4], w[L + 5]);
  order_words(w[L + 6], w[L + 7]); order_words(w[L + 0], w[L + 2]); order_words(w[L + 1], w[L + 3]);
  order_words(w[L + 4], w[L + 6]); order_words(w[L + 5], w[L + 7]); order_words(w[L + 1], w[L + 2]);
  order_words(w[L + 5], w[L + 6]); order_words(w[L + 0], w[L + 4]); order_words(w[L + 1], w[L + 5]);
  order_words(w[L + 2], w[L + 6]); order_words(w[L + 3], w[L + 7]); order_words(w[L + 2], w[L + 4]);
  order_words(w[L + 3], w[L + 5]); order_words(w[L + 1], w[L + 2]); order_words(w[L + 3], w[L + 4]);
  order_words(w[L + 5], w[L + 6]);
}

template <int N>
__device__ __forceinline__ void sort_words(uint32_t (&w)[N]) {
  sort_eight<0>(w);
  if constexpr (N == 16) {
    sort_eight<8>(w);
#pragma unroll
    for (int i = 0; i < 8; ++i) order_words(w[i], w[15 - i]);
    merge_words<0, 8>(w);
    merge_words<8, 8>(w);
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
  merge_words<0, N>(top);
}

// kLaneWarps warps take 32 tokens together: each looks through a share of
// every row, the first joins what they found.  65536 tokens, 256 experts in 8
// groups, top-8: 33 us (rounds of argmax, a warp a token: 276; one warp for
// the 32 tokens: 114; eight warps: 37).  The reads would take 11 us; it is
// bound by the integer pipe, which makes the networks' comparisons.  Few
// tokens: 7 us, mostly latency.  p.logits' rows are `aligned`
// where all of them are made of whole 16-byte pieces.
template <bool BF16, int N, KeyKind KIND>
__global__ void __launch_bounds__(kLaneWarps * 32) route_lanes_kernel(RouteParams p, int pitch, int tail, int bits,
                                                                       bool aligned) {
  extern __shared__ float4 s_rows4[];
  float *rows = reinterpret_cast<float *>(s_rows4);
  float *raw = rows + 32 * pitch;                          // bf16 rows before they are fp32
  uint32_t *words = reinterpret_cast<uint32_t *>(raw);     // [kLaneWarps][N + 1][32]
  float *scores = raw + kLaneWarps * (N + 1) * 32;         // [groups][32]
  float *bias = raw + tail;                                // [pitch]
  __shared__ float s_part[3][kLaneWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, quads = (p.E + 3) / 4;
  const int t0 = blockIdx.x * 32, count = min(32, p.T - t0);
  const auto quad_at = [&](int row, int q) { return row * pitch + q * 4; };
  griddep_wait();
  griddep_launch_dependents();

  // the rows, as fp32 (NaN and +infinity as they are); rows of whole pieces
  // are copied, bf16 ones first to where the scores and words come later
  const int64_t step = p.row_stride * (BF16 ? 2 : 4);
  const char *base = static_cast<const char *>(p.logits) + (int64_t)t0 * step;
  if (aligned) {
    const int pieces = BF16 ? p.E / 8 : quads, apart = BF16 ? pieces | 1 : pitch / 4;
    char *to = reinterpret_cast<char *>(BF16 ? raw : rows);
    for (int r = warp; r < count; r += kLaneWarps)
#pragma unroll 2
      for (int c = lane; c < pieces; c += 32) copy16(smem_addr(to + (r * apart + c) * 16), base + r * step + c * 16);
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (BF16) {
      __syncthreads();
      const int c0 = pieces * warp / kLaneWarps, c1 = pieces * (warp + 1) / kLaneWarps;
      for (int c = c0; c < c1; ++c) {
        const uint4 w = *reinterpret_cast<const uint4 *>(to + (lane * apart + c) * 16);
        float4 *f = reinterpret_cast<float4 *>(rows + quad_at(lane, 2 * c));
        f[0] = make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
        f[1] = make_float4(bf16_lo(w.z), bf16_hi(w.z), bf16_lo(w.w), bf16_hi(w.w));
      }
    }
  } else {
#pragma unroll 8
    for (int i = threadIdx.x; i < count * quads * 4; i += kLaneWarps * 32) {
      const int r = i / (quads * 4), e = i - r * quads * 4;
      rows[quad_at(r, e >> 2) + (e & 3)] = e < p.E ? load_logit<BF16>(base + r * step, e) : kNegInf;
    }
  }
  for (int i = threadIdx.x; i < pitch; i += kLaneWarps * 32) {
    const float v = p.bias != nullptr && i < p.E ? p.bias[i] : 0.0f;
    bias[i] = v != v ? kNegInf : v;
  }
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
  if (!p.sigmoid && !(KIND == kLogitKey && p.renorm)) {
    m = kNegInf;
    if (here)
#pragma unroll 4
      for (int q = q0; q < q1; ++q) {
        float v[4];
        read4(q, v);
        m = fmaxf(fmaxf(m, fmaxf(v[0], v[1])), fmaxf(v[2], v[3]));  // NaN gives way to a number
      }
    m = fminf(m, kMost);
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
        for (int j = 0; j < 4; ++j) sum += v[j] > kNegInf ? softmax_part(fminf(v[j], kMost), m) : 0.0f;
      }
    s_part[1][warp][lane] = sum;
    __syncthreads();
    sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kLaneWarps; ++w) sum += s_part[1][w][lane];
  }
  // Keys in place of logits (a logit that is its own key is only cleaned), and
  // the groups' scores: a warp some groups, or of a single group its share.
  const int per = p.E / p.G / 4;  // quads of a group
  const float inv = 1.0f / sum;
  float most_key = kNegInf;
  if (here)
    for (int g = p.G == 1 ? 0 : warp; g < p.G; g += kLaneWarps) {
      float a = kNegInf, b = kNegInf;
      const int from = p.G == 1 ? q0 : g * per, to = p.G == 1 ? q1 : (g + 1) * per;
#pragma unroll 4
      for (int q = from; q < to; ++q) {
        float v[4];
        read4(q, v);
        const float4 c = KIND == kLogitKey ? make_float4(0.0f, 0.0f, 0.0f, 0.0f)
                                           : *reinterpret_cast<const float4 *>(bias + q * 4);
        const float more[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float key;
          if (KIND == kLogitKey)
            key = fminf(v[j], kMost) + 0.0f;  // -0 counts as +0
          else if (KIND == kSigmoidKey)
            key = sigmoid_key(v[j], more[j]);
          else
            key = softmax_key(fminf(v[j], kMost), m, inv, more[j]);
          v[j] = v[j] > kNegInf ? key : kNegInf;
        }
        *reinterpret_cast<float4 *>(rows + quad_at(lane, q)) = make_float4(v[0], v[1], v[2], v[3]);
        if (p.G > 1) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            b = fmaxf(b, fminf(a, v[j]));
            a = fmaxf(a, v[j]);
          }
        } else {
          a = fmaxf(fmaxf(a, fmaxf(v[0], v[1])), fmaxf(v[2], v[3]));
        }
      }
      most_key = fmaxf(most_key, a);
      if (p.G == 1) break;
      scores[g * 32 + lane] = p.group_top == 2 && b != kNegInf ? a + b : a;
    }
  s_part[2][warp][lane] = most_key;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kLaneWarps; ++w) most_key = fmaxf(most_key, s_part[2][w][lane]);
  uint64_t offered = p.G == 1 && here ? 1ull : 0ull;
  if (p.G > 1 && p.G <= 8 && here) {
    // a group's rank among the few: how many come before it
    float s[8];
#pragma unroll
    for (int g = 0; g < 8; ++g) s[g] = g < p.G ? scores[g * 32 + lane] : kNegInf;
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      int rank = 0;
#pragma unroll
      for (int h = 0; h < 8; ++h) rank += h < g ? s[h] >= s[g] : h > g ? s[h] > s[g] : 0;
      if (s[g] != kNegInf && rank < p.Gk) offered |= 1ull << g;
    }
  } else if (p.G > 8 && here) {
    for (int k = 0; k < p.Gk; ++k) {
      float best = kNegInf;
      int at = -1;
#pragma unroll 8
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
  }

  // this warp's share of the offered groups, one after the other: the N
  // largest words, and the largest of the others
  constexpr bool kExact = BF16 && KIND == kLogitKey;
  constexpr float kWindow = KIND == kLogitKey ? 32.0f : 4.0f;
  const uint32_t low = (1u << bits) - 1u;
  const float steps = (float)((1u << (32 - bits)) - 1u), scale = steps * (1.0f / kWindow);
  // A key's place in a word's upper bits.  8388608 + the place, as a float,
  // has it in its low bits, and the shift drops the others.
  const auto place_of = [&](float v, float from) {
    return kExact ? order_of(v) & ~low : __float_as_uint(fmaxf(fmaf(v - from, scale, 8388608.0f + steps), 8388608.0f)) << bits;
  };
  const uint32_t least = kExact ? kLeast : 1u << bits;  // smaller words: none, or below the window
  uint32_t top[N] = {}, out = 0u;
  const int length = p.G == 1 ? quads : per, all = length * p.Gk;
  const int i1 = all * (warp + 1) / kLaneWarps;
  int i = all * warp / kLaneWarps, in = i % length;
  uint64_t left = offered;
  for (int k = i / length; k > 0; --k) left &= left - 1ull;
  while (i < i1) {
    // a run of quads of one group (a lane may have none left)
    const int run = min(i1 - i, length - in);
    const bool some = left != 0ull;
    const int from = (some ? __ffsll((long long)left) - 1 : 0) * length + in;
    for (int q = 0; q < run; q += N / 4) {
      uint32_t w[N];
#pragma unroll
      for (int n = 0; n < N / 4; ++n) {
        float v[4];
        const int at = from + min(q + n, run - 1);
        read4(at, v);
        const uint32_t index = low - (uint32_t)(at * 4);
        const bool use = some && q + n < run;
#pragma unroll
        for (int j = 0; j < 4; ++j) w[n * 4 + j] = use ? place_of(v[j], most_key) + (index - j) : 0u;
      }
      sort_words(w);
      join_words(top, w, out);
    }
    i += run;
    in = 0;
    left &= left - 1ull;
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
      idx[n] = top[n] < least ? -1 : (int)(low - (top[n] & low));
      if (n > 0) alike = alike || (!kExact && top[n] >= least && (top[n] & ~low) == (top[n - 1] & ~low));
      last = n < p.K ? top[n] : last;
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
    if (!kExact && (last < least || (out & ~low) == (last & ~low))) {
      // the last choices go by whole keys among all of that place
      const uint32_t bits_of = last & ~low;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        if ((top[n] & ~low) == bits_of) idx[n] = -1;
        key[n] = idx[n] < 0 ? kNegInf : rows[quad_at(lane, idx[n] >> 2) + (idx[n] & 3)];
      }
      for (left = offered; left != 0ull; left &= left - 1ull) {
        const int g = __ffsll((long long)left) - 1;
#pragma unroll 2
        for (int q = g * length; q < (g + 1) * length; ++q) {
          float v[4];
          read4(q, v);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (place_of(v[j], most_key) != bits_of || !(v[j] > key[N - 1])) continue;
            const float x = v[j];
            const int e = q * 4 + j;
#pragma unroll
            for (int n = N - 1; n > 0; --n) {
              const bool up = x > key[n - 1], at = x > key[n];
              idx[n] = up ? idx[n - 1] : at ? e : idx[n];
              key[n] = up ? key[n - 1] : at ? x : key[n];
            }
            if (x > key[0]) {
              key[0] = x;
              idx[0] = e;
            }
          }
        }
      }
    }

    __syncwarp();  // the other warps' words have been read
#pragma unroll
    for (int n = 0; n < N; ++n)
      if (n < p.K) reinterpret_cast<int *>(words)[lane * p.K + n] = here ? idx[n] : -1;
    s_part[0][0][lane] = m;
    s_part[1][0][lane] = sum;
  }
  __syncthreads();

  // weights, as in choice_weight: kLaneWarps threads a token
  const int *choice = reinterpret_cast<const int *>(words);
  const int t = threadIdx.x / kLaneWarps, own = threadIdx.x % kLaneWarps;
  m = s_part[0][0][t];
  sum = s_part[1][0][t];
  float l[N / kLaneWarps], w[N / kLaneWarps], most = kNegInf, total = 0.0f;
#pragma unroll
  for (int n = 0; n < N / kLaneWarps; ++n) {
    const int k = n * kLaneWarps + own, e = t < count && k < p.K ? choice[t * p.K + k] : -1;
    l[n] = e < 0               ? kNegInf
           : KIND == kLogitKey ? rows[quad_at(t, e >> 2) + (e & 3)]
                               : load_logit<BF16>(base + t * step, e);
    most = fmaxf(most, p.sigmoid ? fminf(l[n], 0.0f) : l[n]);
  }
  most = warp_max<kLaneWarps>(most);
  if (!p.renorm) most = p.sigmoid ? 0.0f : m;
#pragma unroll
  for (int n = 0; n < N / kLaneWarps; ++n) {
    if (p.sigmoid)
      w[n] = l[n] == kNegInf ? 0.0f : expf(fminf(l[n], 0.0f) - most) / (1.0f + expf(-fabsf(l[n])));
    else
      w[n] = l[n] == kNegInf ? 0.0f : expf(l[n] - most);
    total += w[n];
  }
  total = warp_sum<kLaneWarps>(total);
  if (!p.renorm) total = p.sigmoid ? 1.0f : sum;
#pragma unroll
  for (int n = 0; n < N / kLaneWarps; ++n) {
    const int k = n * kLaneWarps + own;
    if (t < count && k < p.K) p.w[(int64_t)(t0 + t) * p.K + k] = total > 0.0f ? w[n] / total * p.scale : 0.0f;
  }
  for (int i = threadIdx.x; i < count * p.K; i += kLaneWarps * 32) p.idx[(int64_t)t0 * p.K + i] = choice[i];
}

// Where a lane a token is used: rows that fit beside each other, at most 16
// choices, groups of whole quads.  Few tokens with few experts are answered
// sooner by a warp a token (8 experts: 2.8 us against 4.8; 64 experts: 4.7 to
// 5.4 against 4.9 to 5.2; 256 in groups: 13.7 against 6.4).
bool lanes_fit(const RouteArgs &a) {
  return (a.num_experts >= kManyExperts || a.num_tokens > 4096) && a.num_experts <= 1024 && a.num_topk <= 16 &&
         (a.num_groups == 1 || a.num_experts / a.num_groups % 4 == 0);
}

template <bool BF16, int N, KeyKind KIND>
ep_status_t launch_lanes_as(const RouteParams &p, cudaStream_t stream) {
  const int pitch = (((p.E + 3) / 4) | 1) * 4;
  int bits = 9;  // of a word, for the index
  while ((1 << bits) < (p.E + 3) / 4 * 4) ++bits;
  const bool aligned = reinterpret_cast<uintptr_t>(p.logits) % 16 == 0 &&
                       p.row_stride % (BF16 ? 8 : 4) == 0 && p.E % (BF16 ? 8 : 4) == 0;
  int tail = kLaneWarps * (N + 1) * 32 + (p.G > 1 ? p.G * 32 : 0);
  const int raw = BF16 && aligned ? 32 * (p.E / 8 | 1) * 4 : 0;
  if (tail < raw) tail = raw;
  const size_t smem = ((size_t)32 * pitch + tail + pitch) * 4;
  static std::atomic<bool> ready[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && !ready[dev]) {
    e = cudaFuncSetAttribute(route_lanes_kernel<BF16, N, KIND>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (33 * 1028 + 32 * 129 * 4) * 4);
    if (e == cudaSuccess) ready[dev] = true;
  }
  if (e == cudaSuccess)
    e = launch_kernel(route_lanes_kernel<BF16, N, KIND>, (p.T - 1) / 32 + 1, kLaneWarps * 32, smem, stream, false, p, pitch,
                      tail, bits, aligned);
  return e == cudaSuccess ? EP_OK : cuda_fail(e, "route launch");
}

template <bool BF16, int N>
ep_status_t launch_lanes(const RouteParams &p, cudaStream_t stream) {
  if (p.by_logit) return launch_lanes_as<BF16, N, kLogitKey>(p, stream);
  return p.sigmoid ? launch_lanes_as<BF16, N, kSigmoidKey>(p, stream) : launch_lanes_as<BF16, N, kSoftmaxKey>(p, stream);
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

constexpr int kBackwardWarps = 8;

// L lanes a token (8, 16 or 32, as its choices need), lane k its k-th choice.  Only a softmax over all experts
// (not renormalised) gives every logit a gradient, -p (sum d p), and needs
// the whole row of logits; otherwise the row is zeros but for the choices,
// and only their logits are read.  Either is written 16 bytes at a time
// (`wide`: rows of whole pieces) and the choices' values after it: writes to
// L2, which are one to memory.  The full softmax takes approximate
// exponentials: a few units in the last place, and the rounding of
// (l - m) log2 e, which is no more than that of l - m; a p below 2^-126, and
// its gradient, is 0.  65536 tokens, 256 experts, top-8, not a full
// softmax: 19 us, 7.3 TB/s of the bytes that would also read the logits
// (rows in shared memory, a warp a token: 41 us; 16-byte zeros: 31 us).
template <bool BF16, int L>
__global__ void __launch_bounds__(kBackwardWarps * 32) route_backward_kernel(RouteBackwardParams p, bool wide) {
  constexpr int kPiece = BF16 ? 8 : 4;
  constexpr int kTokens = kBackwardWarps * 32 / L;  // of a block
  const int lane = threadIdx.x % L;
  const bool dense = !p.sigmoid && !p.renorm;
  griddep_wait();
  griddep_launch_dependents();
  for (int64_t t0 = (int64_t)blockIdx.x * kTokens; t0 < p.T; t0 += (int64_t)gridDim.x * kTokens) {
    const int64_t own = t0 + threadIdx.x / L;
    const bool here = own < p.T;
    const int64_t t = here ? own : p.T - 1;  // all lanes take part in the exchanges
    const void *row = static_cast<const char *>(p.logits) + t * p.row_stride * (BF16 ? 2 : 4);
    void *out = static_cast<char *>(p.out) + t * p.E * (BF16 ? 2 : 4);
    const int64_t at64 = here && lane < p.K ? p.idx[t * p.K + lane] : -1;
    const float g = here && lane < p.K ? p.grad[t * p.K + lane] * p.scale : 0.0f;
    const int at = at64 >= 0 && at64 < p.E ? (int)at64 : -1;
    const float l = at < 0 ? kNegInf : load_logit<BF16>(row, at);
    const bool none = l == kNegInf;
    float d = none ? 0.0f : g, dot = 0.0f, m = kNegInf, inv = 0.0f;
    const auto piece = [&](int c, float (&v)[kPiece]) {
      const int4 f = __ldg(static_cast<const int4 *>(row) + c);
      const uint32_t *w = reinterpret_cast<const uint32_t *>(&f);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (BF16) {
          v[2 * j] = bf16_lo(w[j]);
          v[(2 * j + 1) % kPiece] = bf16_hi(w[j]);
        } else {
          v[j] = __uint_as_float(w[j]);
        }
      }
#pragma unroll
      for (int j = 0; j < kPiece; ++j) v[j] = fminf(v[j] != v[j] ? kNegInf : v[j], 3.402823466e38f);
    };
    if (dense) {
      float sum = 0.0f;
      if (wide) {
        for (int c = lane; c < p.E / kPiece; c += L) {
          float v[kPiece];
          piece(c, v);
#pragma unroll
          for (int j = 0; j < kPiece; ++j) m = fmaxf(m, v[j]);
        }
        m = warp_max<L>(m);
        if (m != kNegInf)
          for (int c = lane; c < p.E / kPiece; c += L) {
            float v[kPiece];
            piece(c, v);
#pragma unroll
            for (int j = 0; j < kPiece; ++j) sum += exp2_approx((v[j] - m) * kLog2e);
          }
      } else {
        for (int j = lane; j < p.E; j += L) m = fmaxf(m, load_logit<BF16>(row, j));
        m = warp_max<L>(m);
        if (m != kNegInf)
          for (int j = lane; j < p.E; j += L) sum += exp2_approx((load_logit<BF16>(row, j) - m) * kLog2e);
      }
      sum = warp_sum<L>(sum);
      inv = sum > 0.0f ? 1.0f / sum : 0.0f;
      dot = warp_sum<L>(none ? 0.0f : d * (exp2_approx((l - m) * kLog2e) * inv));
    } else if (p.renorm) {
      // u = p / sum p; du_k/dl_k' carries p' / sum = u (1 - p) for a sigmoid,
      // and u for a softmax (its share of the chosen alone)
      const float u = choice_weight<L>(none, l, p.sigmoid, true, 0.0f, 1.0f);
      d = u * (d - warp_sum<L>(d * u));
      if (p.sigmoid) d *= none ? 0.0f : 1.0f / (1.0f + expf(l));
    } else {
      const float e = expf(-fabsf(l));  // p (1 - p) = e / (1 + e)^2
      d = none ? 0.0f : d * (e / ((1.0f + e) * (1.0f + e)));
    }
    // an expert named twice receives both: every one of its lanes adds all
    const uint32_t same = __match_any_sync(0xffffffffu, none ? -1 - (int)(threadIdx.x & 31) : at | (int)(threadIdx.x & 31) / L << 16);
    if (__any_sync(0xffffffffu, !none && (same & (same - 1u)) != 0u)) {
      float all = 0.0f;
      for (int k = 0; k < p.K; ++k) {
        const int from = (int)(threadIdx.x & 31) / L * L + k;
        const float v = __shfl_sync(0xffffffffu, d, from);
        if ((same >> from) & 1u) all += v;
      }
      d = all;
    }
    if (here && wide) {
      for (int c = lane; c < p.E / kPiece; c += L) {
        int4 f = make_int4(0, 0, 0, 0);
        if (dense && m != kNegInf) {
          float v[kPiece];
          piece(c, v);
#pragma unroll
          for (int j = 0; j < kPiece; ++j) v[j] = -(exp2_approx((v[j] - m) * kLog2e) * inv) * dot;
          int *w = reinterpret_cast<int *>(&f);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            w[j] = BF16 ? (int)pack_bf16x2(v[2 * j % kPiece], v[(2 * j + 1) % kPiece]) : __float_as_int(v[j]);
        }
        static_cast<int4 *>(out)[c] = f;
      }
    } else if (here) {
      for (int j = lane; j < p.E; j += L) {
        const float v = dense && m != kNegInf ? -(exp2_approx((load_logit<BF16>(row, j) - m) * kLog2e) * inv) * dot : 0.0f;
        store_grad<BF16>(out, j, v);
      }
    }
    __syncwarp();
    if (!none) store_grad<BF16>(out, at, dense ? (exp2_approx((l - m) * kLog2e) * inv) * (d - dot) : d);
  }
}

// The limit of dynamic shared memory belongs to the kernel, not to a launch:
// it is set to the most that any call needs, so a call in another thread with
// fewer experts cannot lower it between this one's check and its launch.
template <bool BF16>
ep_status_t launch_warps(const RouteParams &p, const DeviceInfo *di, cudaStream_t stream) {
  const size_t smem = (size_t)kRouteWarps * p.E * sizeof(float);
  static std::atomic<bool> ready[64];
  if (smem > 48 * 1024 && !ready[di->device]) {
    const cudaError_t e = cudaFuncSetAttribute(route_kernel<BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kRouteWarps * EP_MAX_EXPERTS * (int)sizeof(float));
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
    ready[di->device] = true;
  }
  const int64_t need = ((int64_t)p.T + kRouteWarps - 1) / kRouteWarps, most = (int64_t)di->num_sms * 16;
  const cudaError_t e = launch_kernel(route_kernel<BF16>, (int)(need < most ? need : most), kRouteWarps * 32, smem, stream,
                                      false, p);
  return e == cudaSuccess ? EP_OK : cuda_fail(e, "route launch");
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
  return a.bf16 ? launch_warps<true>(p, di, stream) : launch_warps<false>(p, di, stream);
}

ep_status_t launch_route_backward(const RouteBackwardArgs &a, cudaStream_t stream) {
  if (a.num_tokens == 0) return EP_OK;
  const DeviceInfo *di = current_device_info();
  if (di == nullptr) return EP_ERR_CUDA;
  RouteBackwardParams p{a.grad_weights, a.logits, a.row_stride,   a.topk_idx, a.num_tokens, a.num_experts,
                        a.num_topk,     a.weight_scale, a.grad_logits, a.sigmoid,  a.renormalize};
  const int lanes = a.num_topk <= 8 ? 8 : a.num_topk <= 16 ? 16 : 32;
  const auto kernel = lanes == 8    ? (a.bf16 ? route_backward_kernel<true, 8> : route_backward_kernel<false, 8>)
                      : lanes == 16 ? (a.bf16 ? route_backward_kernel<true, 16> : route_backward_kernel<false, 16>)
                                    : (a.bf16 ? route_backward_kernel<true, 32> : route_backward_kernel<false, 32>);
  const int piece = a.bf16 ? 8 : 4;
  const bool wide = a.num_experts % piece == 0 && a.row_stride % piece == 0 &&
                    reinterpret_cast<uintptr_t>(a.logits) % 16 == 0 && reinterpret_cast<uintptr_t>(a.grad_logits) % 16 == 0;
  const int tokens = kBackwardWarps * 32 / lanes;  // of a block
  const int64_t need = ((int64_t)a.num_tokens + tokens - 1) / tokens, most = (int64_t)di->num_sms * 32;
  const cudaError_t e =
      launch_kernel(kernel, (int)(need < most ? need : most), kBackwardWarps * 32, 0, stream, false, p, wide);
  return e == cudaSuccess ? EP_OK : cuda_fail(e, "route_backward launch");
}

}  // namespace ep
