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
// Bound by memory: one pass over the logits.  A row belongs to L lanes of a
// warp (beyond 1024 experts to a whole block), V columns each, so that a row's
// sums take log2 L exchanges and the columns' sums stay in registers over all
// rows of a lane.  A lane copies its
// pieces of the rows ahead (cp.async) to shared memory that only it reads,
// so they need no barrier.  The sums over
// tokens run in a fixed order: a block's part of a sequence first (a
// "segment"; block b's of sequence s is segment b + s, since later blocks
// hold later sequences), then the segments.
#include <algorithm>
#include <atomic>

#include "ep_ops.h"
#include "ep_tc.cuh"

namespace ep {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTokenStep = 32;    // a block's tokens come in these
constexpr int kLanesMost = 1024;  // experts that a warp's lanes hold
constexpr int kChoices = 4;       // of a thread in a pass: EP_MAX_TOPK rows of 8 lanes
constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kMost = 3.402823466e38f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kTiny = -200.0f;  // 2^-200 is 0

__device__ __forceinline__ float value_of(const void *p, bool bf16, int64_t i) {
  return bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t *>(p)[i] << 16) : static_cast<const float *>(p)[i];
}

// A logit in fp32: NaN counts as masked, +infinity as the largest number.
__device__ __forceinline__ float offered(float v) { return fminf(v != v ? kNegInf : v, kMost); }

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ int offset_of(const int32_t *offsets, int T, int s) {
  return offsets == nullptr ? (s == 0 ? 0 : T) : min(max(offsets[s], 0), T);
}

// The first sequence that ends behind token t (S: none).  Within the bounds
// of `offsets` whatever they hold.
__device__ __forceinline__ int sequence_of(const int32_t *offsets, int T, int S, int t) {
  int low = 0, high = S;
  while (low < high) {
    const int mid = (low + high) / 2;
    if (offset_of(offsets, T, mid + 1) > t)
      high = mid;
    else
      low = mid + 1;
  }
  return low;
}

constexpr uint32_t kWarpLanes = 0xffffffffu;

// The lanes of the warp that hold this lane's row.
template <int L>
__device__ __forceinline__ uint32_t row_lanes() {
  return L < 32 ? ((1u << (L % 32)) - 1u) << (threadIdx.x % 32 / L * L) : kWarpLanes;
}

// Over a row's lanes, the same in all of them; L = kThreads: the block.
// `lanes`: those that call it, whole rows.
template <int L>
__device__ __forceinline__ float lanes_sum(float v, uint32_t lanes = kWarpLanes) {
#pragma unroll
  for (int o = (L < 32 ? L : 32) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(lanes, v, o);
  if (L > 32) {
    __shared__ float s[kWarps];
    __syncthreads();
    if (threadIdx.x % 32 == 0) s[threadIdx.x / 32] = v;
    __syncthreads();
    v = s[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) v += s[w];
  }
  return v;
}

template <int L>
__device__ __forceinline__ float lanes_max(float v, uint32_t lanes = kWarpLanes) {
#pragma unroll
  for (int o = (L < 32 ? L : 32) / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(lanes, v, o));
  if (L > 32) {
    __shared__ float s[kWarps];
    __syncthreads();
    if (threadIdx.x % 32 == 0) s[threadIdx.x / 32] = v;
    __syncthreads();
    v = s[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) v = fmaxf(v, s[w]);
  }
  return v;
}

__device__ __forceinline__ void copy_piece(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Until at most N of this thread's groups are in flight.
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A row's V columns of a lane: by pieces of 16 bytes where rows allow it
// (WIDE: through shared memory, `here` the lane's place, a block's threads
// apart), else one by one, neighbours in neighbouring lanes.
template <bool BF16, int L, int V, bool WIDE>
struct Columns {
  static constexpr int kPiece = BF16 ? 8 : 4, kCount = V / kPiece;
  int E, lane;
  __device__ int column(int i, int j) const { return WIDE ? (i * L + lane) * kPiece + j : (i * kPiece + j) * L + lane; }
  __device__ void fetch(char *here, const char *row) const {
    if (!WIDE) return;
#pragma unroll
    for (int i = 0; i < kCount; ++i)
      if (column(i, 0) < E) copy_piece(smem_addr(here) + i * kThreads * 16, row + column(i, 0) * (BF16 ? 2 : 4));
  }
  // Where no copy comes: past the last expert -infinity, or 0 of either type,
  // and 0 in a row that is not `there` (its lanes take part in exchanges and
  // in the warp's vote on how scores are computed).
  __device__ void clear(char *here, bool masked, bool there) const {
#pragma unroll
    for (int i = 0; i < kCount; ++i) {
      const bool past = column(i, 0) >= E;
      const int w = !(masked && past) ? 0 : BF16 ? (int)0xff80ff80u : (int)0xff800000u;
      if (WIDE && (past || !there)) *reinterpret_cast<int4 *>(here + i * kThreads * 16) = make_int4(w, w, w, w);
    }
  }
  // Columns past the last expert read what `clear` put there, or `none`; a row
  // that is not `there` is not read (its place may be one that another warp
  // writes, where the gradient goes over the logits).
  __device__ void load(const char *here, const char *row, bool there, float none, float (&v)[V]) const {
#pragma unroll
    for (int i = 0; i < kCount; ++i) {
      if (WIDE) {
        const int4 f = *reinterpret_cast<const int4 *>(here + i * kThreads * 16);
        const int w[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
        for (int j = 0; j < kPiece; ++j)
          v[i * kPiece + j] = !BF16 ? __int_as_float(w[j % 4]) : j % 2 ? bf16_hi(w[j / 2]) : bf16_lo(w[j / 2]);
      } else {
#pragma unroll
        for (int j = 0; j < kPiece; ++j)
          v[i * kPiece + j] = column(i, j) >= E ? none : there ? value_of(row, BF16, column(i, j)) : 0.0f;
      }
    }
  }
  __device__ void store(char *row, const float (&v)[V]) const {
#pragma unroll
    for (int i = 0; i < kCount; ++i) {
      if (WIDE) {
        int w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          w[j] = BF16 ? (int)pack_bf16x2(v[i * kPiece + 2 * j % kPiece], v[i * kPiece + (2 * j + 1) % kPiece])
                      : __float_as_int(v[i * kPiece + j % kPiece]);
        if (column(i, 0) < E)
          *reinterpret_cast<int4 *>(row + column(i, 0) * (BF16 ? 2 : 4)) = make_int4(w[0], w[1], w[2], w[3]);
      } else {
#pragma unroll
        for (int j = 0; j < kPiece; ++j) {
          if (column(i, j) >= E) continue;
          const float x = v[i * kPiece + j];
          if (BF16)
            reinterpret_cast<uint16_t *>(row)[column(i, j)] = (uint16_t)(pack_bf16x2(x, 0.0f) & 0xffffu);
          else
            reinterpret_cast<float *>(row)[column(i, j)] = x;
        }
      }
    }
  }
  __device__ void floats(const float *row, float (&v)[V]) const {
#pragma unroll
    for (int i = 0; i < kCount; ++i)
#pragma unroll
      for (int j = 0; j < kPiece; ++j) v[i * kPiece + j] = column(i, j) < E ? __ldg(row + column(i, j)) : 0.0f;
  }
};

// A row's scores over L lanes: p = e inv; softmax = soft inv_soft (kSigmoid;
// else e inv too), side = 1 - sigmoid.
template <int V, bool SIGMOID, bool GRAD>
struct Scores {
  float e[V];
  float soft[SIGMOID && GRAD ? V : 1], side[SIGMOID && GRAD ? V : 1];
  float inv, inv_soft, lse;
};

// Rows whose largest logit is huge, or by sigmoid whose sum of e^l is near the
// ends of fp32: everything relative to the largest.  The lanes of such a row
// alone come here, so no row's bits hang on another.
template <int L, int V, bool SIGMOID, bool GRAD>
__device__ __forceinline__ void far_scores(const float (&l)[V], Scores<V, SIGMOID, GRAD> &s) {
  const uint32_t lanes = row_lanes<L>();
  float m = kNegInf, sum = 0.0f, soft = 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) m = fmaxf(m, offered(l[j]));
  m = lanes_max<L>(m, lanes);
  const float k = fminf(m, 0.0f);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const float x = offered(l[j]);
    const bool there = x > kNegInf;
    const float e = there ? exp2_approx(fmaxf((x - m) * kLog2e, kTiny)) : 0.0f;
    soft += e;
    if (SIGMOID) {
      const float u = exp2_approx(fmaxf(-fabsf(x) * kLog2e, kTiny)), r = 1.0f / (1.0f + u);
      s.e[j] = there ? exp2_approx(fmaxf((fminf(x, 0.0f) - k) * kLog2e, kTiny)) * r : 0.0f;
      if (GRAD) {
        s.soft[GRAD ? j : 0] = e;
        s.side[GRAD ? j : 0] = x >= 0.0f ? u * r : r;
      }
    } else {
      s.e[j] = e;
    }
    sum += s.e[j];
  }
  sum = lanes_sum<L>(sum, lanes);
  soft = lanes_sum<L>(soft, lanes);
  s.inv = sum > 0.0f ? 1.0f / sum : 0.0f;
  s.inv_soft = soft > 0.0f ? 1.0f / soft : 0.0f;
  s.lse = soft > 0.0f ? m + logf(soft) : 0.0f;
}

// All lanes of the warp (L = kThreads: of the block) call it.  Exponentials are approximate (2 ulp, and
// the rounding of their argument); -infinity becomes 0; NaN makes the sum NaN,
// which is not near either.
//   softmax: 2^(l log2 e - c), c = m log2 e rounded once, which cancels in p
//            (below 2^24 it is off by 1 at most, so no power overflows)
//   sigmoid: E = e^l, sigmoid E / (1 + E); one exponential serves both scores
template <int L, int V, bool SIGMOID, bool GRAD>
__device__ __forceinline__ void scores_of(const float (&l)[V], Scores<V, SIGMOID, GRAD> &s) {
  float sum = 0.0f, soft = 0.0f, c = 0.0f;
  bool near;
  if (SIGMOID) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float e = exp2_approx(l[j] * kLog2e), r = rcp_normal(1.0f + e);
      s.e[j] = e * r;
      sum += s.e[j];
      soft += e;
      if (GRAD) {
        s.soft[GRAD ? j : 0] = e;
        s.side[GRAD ? j : 0] = r;
      }
    }
    sum = lanes_sum<L>(sum);
    soft = lanes_sum<L>(soft);
    near = soft > 1e-30f && soft < 1e30f;
  } else {
    float m = kNegInf;
#pragma unroll
    for (int j = 0; j < V; ++j) m = fmaxf(m, l[j]);
    m = lanes_max<L>(m);
    c = m * kLog2e;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      s.e[j] = exp2_approx(fmaf(l[j], kLog2e, -c));
      sum += s.e[j];
    }
    sum = lanes_sum<L>(sum);
    soft = sum;
    near = fabsf(m) < 16777216.0f && sum > 0.0f;
  }
  const auto finish = [&] {
    s.inv = rcp_normal(sum);
    s.inv_soft = SIGMOID ? rcp_normal(soft) : s.inv;
    s.lse = fmaf(c, kLn2, logf(soft));
  };
  // `near` is the same for all of a row's lanes.  The warp's vote keeps the
  // branches below out of the way of warps without such a row (65 536 tokens,
  // 256 experts by sigmoid: 23.0 us, without the vote 27.2).
  if (L > 32 ? !near : !__all_sync(kWarpLanes, near)) {
    if (near)
      finish();
    else
      far_scores<L, V, SIGMOID, GRAD>(l, s);
    __syncwarp();
    return;
  }
  finish();
}

// How the tokens are shared.  Many: by blocks that are all on the SMs at once,
// two each of 152, or three where a lane has 16 columns or fewer (65 536
// tokens, 256 experts: 411 blocks 28 us; 293, at most two an SM, 22).  In fp32
// that holds up to some 450 experts: at 512 a block takes 118 KB of shared
// memory, so an SM has one, and the blocks two turns (32 768 tokens, 256 blocks:
// 25.7 us, floor 10.2).  Few, up to five passes of a block's rows: by one cluster, which joins its parts itself and
// saves a launch, 3.4 us of the host's (1021 tokens, 64 experts in a graph 6.8
// us, 7.0 with the launch).
struct Cut {
  int tokens, blocks;  // of a block, and blocks
  bool joined;
};

constexpr int kPasses = 5;
constexpr int kJoinedCounts = 65536;  // sequences times experts, at most, of a cluster

Cut cut_of(int T, int E, int S) {
  if (T == 0) return Cut{kTokenStep, 0, false};
  const int rows = E <= 256 ? 32 : E <= 512 ? 16 : 8;  // of a pass
  const int each = ((T - 1) / kClusterMost + rows) / rows * rows;
  if (E <= kLanesMost && each <= kPasses * rows && (int64_t)S * E <= kJoinedCounts) return Cut{each, (T - 1) / each + 1, true};
  const int blocks = E <= 128 ? 456 : 304;
  const int tokens = std::max(kTokenStep, ((T - 1) / blocks + kTokenStep) / kTokenStep * kTokenStep);
  return Cut{tokens, (T - 1) / tokens + 1, false};
}

struct Parts {
  float *probs;     // [segments][E]
  int32_t *counts;  // [segments][E]
  int32_t *chosen;  // [segments]
  float *z;         // [blocks]
  float *balance;   // [S][column blocks]
  int32_t *head;    // sequences with tokens, whether offsets are out of order, tickets of the join
  int tokens, blocks;
  bool joined;
};

// Sequences with tokens (x), and whether the offsets are out of order (y),
// for all threads of a block.
__device__ int2 look_at_offsets(const int32_t *offsets, int T, int S) {
  int full = 0, bad = 0;
  for (int s = threadIdx.x; s < S; s += blockDim.x) {
    full += offset_of(offsets, T, s + 1) > offset_of(offsets, T, s);
    if (offsets != nullptr) bad |= offsets[s] < 0 || offsets[s] > offsets[s + 1] || offsets[s + 1] > T;
  }
  __shared__ int s_full[32], s_bad;
  if (threadIdx.x == 0) s_bad = 0;
  full = __reduce_add_sync(0xffffffffu, full);
  if ((threadIdx.x & 31) == 0) s_full[threadIdx.x / 32] = full;
  __syncthreads();
  if (bad) atomicOr(&s_bad, 1);
  __syncthreads();
  full = 0;
  for (int i = 0; i < (int)blockDim.x / 32; ++i) full += s_full[i];
  return make_int2(full, s_bad);
}

// The same for the joining kernel, whose tickets start at 0.
__device__ void write_head(const BalanceArgs &p, const Parts &parts) {
  const int2 v = look_at_offsets(p.seq_offsets, p.num_tokens, p.num_sequences);
  if (threadIdx.x != 0) return;
  parts.head[0] = v.x;
  parts.head[1] = v.y;
  parts.head[2] = 0;
}

// An expert's count and mean score in a sequence, and its share of the loss,
// from the segments' sums.  A sequence may have more choices than 32 bits
// count, and by indices named twice an expert too: its count stops there.
template <typename COUNT>
__device__ __forceinline__ float finish_expert(const BalanceArgs &p, int s, int e, int tokens, float prob, COUNT count,
                                               COUNT chosen, int full) {
  const int64_t at = (int64_t)s * p.num_experts + e;
  const float mean = tokens > 0 ? prob / tokens : 0.0f;
  const float share = chosen > 0 ? (float)p.num_experts * count / chosen / full : 0.0f;
  p.probs[at] = mean;
  p.counts[at] = (int32_t)min(count, (COUNT)INT32_MAX);
  p.slopes[at] = tokens > 0 ? share / tokens : 0.0f;
  return share * mean;
}

__device__ __forceinline__ float loss_of(float v, int bad) { return bad != 0 ? __int_as_float(0x7fffffff) : v; }

// The whole grid is one cluster: its blocks join the segments and the losses.
__device__ void join_in_cluster(const BalanceArgs &p, const Parts &parts, float z) {
  __shared__ float s_losses[2], s_balance[kWarps];
  const int E = p.num_experts, T = p.num_tokens, S = p.num_sequences;
  const int2 head = look_at_offsets(p.seq_offsets, T, S);
  cluster_sync();  // the segments in global memory
  float balance = 0.0f;
  for (int i = blockIdx.x * kThreads + threadIdx.x; i < S * E; i += gridDim.x * kThreads) {
    const int s = i / E, e = i - s * E;
    const int a = offset_of(p.seq_offsets, T, s), b = offset_of(p.seq_offsets, T, s + 1);
    const int b0 = a / parts.tokens, b1 = b > a ? (b - 1) / parts.tokens : b0 - 1;
    float prob = 0.0f;
    int count = 0, chosen = 0;
#pragma unroll 4
    for (int k = b0; k <= b1; ++k) {
      prob += __ldcg(parts.probs + (int64_t)(k + s) * E + e);
      count += __ldcg(parts.counts + (int64_t)(k + s) * E + e);
      chosen += __ldcg(parts.chosen + k + s);
    }
    balance += finish_expert(p, s, e, b - a, prob, count, chosen, head.x);
  }
  balance = lanes_sum<32>(balance);
  if (threadIdx.x % 32 == 0) s_balance[threadIdx.x / 32] = balance;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kWarps; ++w) balance += s_balance[w];
    s_losses[0] = balance;
    s_losses[1] = z;
  }
  cluster_sync();
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    balance = z = 0.0f;
    for (int b = 0; b < (int)gridDim.x; ++b) {
      balance += load_cluster(map_shared(smem_addr(&s_losses[0]), b));
      z += load_cluster(map_shared(smem_addr(&s_losses[1]), b));
    }
    const int tokens = offset_of(p.seq_offsets, T, S) - offset_of(p.seq_offsets, T, 0);
    p.losses[0] = loss_of(balance, head.y);
    p.losses[1] = loss_of(tokens > 0 ? z / tokens : 0.0f, head.y);
  }
  cluster_sync();  // before a block whose losses are read ends
}

// Passes of rows in shared memory: up to 64 KB (16 columns a lane in fp32),
// 96 KB (32).
template <bool BF16, int V>
constexpr int ahead() { return V > 16 && !BF16 ? 3 : 4; }
template <bool BF16, int V>
constexpr int pass_bytes() { return kThreads * V * (BF16 ? 2 : 4); }

template <bool BF16, int L, int V, bool WIDE, bool SIGMOID>
__global__ void __launch_bounds__(kThreads, V > 16 ? 2 : 3) balance_kernel(BalanceArgs p, Parts parts) {
  // [ahead][pieces][threads], then [warps][experts] sums (within a warp's rows) and [experts] counts
  extern __shared__ int4 s_rows[];
  __shared__ float s_z[kWarps];
  __shared__ int s_chosen[kWarps];
  constexpr int kRows = kThreads / L, kAhead = ahead<BF16, V>(), kPass = pass_bytes<BF16, V>();
  const int E = p.num_experts, T = p.num_tokens, S = p.num_sequences, K = p.num_topk;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const Columns<BF16, L, V, WIDE> columns{E, (int)threadIdx.x % L};
  float *s_probs = reinterpret_cast<float *>(reinterpret_cast<char *>(s_rows) + (WIDE ? kAhead * kPass : 0));
  int *s_counts = reinterpret_cast<int *>(s_probs + (L > 32 ? 0 : kWarps * E));
  char *mine = reinterpret_cast<char *>(s_rows + threadIdx.x);
  const int t0 = (int)blockIdx.x < parts.blocks ? blockIdx.x * parts.tokens : 0, count = min(T - t0, parts.tokens), row = threadIdx.x / L;
  const int64_t apart = p.row_stride * (BF16 ? 2 : 4);
  const char *from = static_cast<const char *>(p.logits) + (t0 + row) * apart;
  for (int e = threadIdx.x; e < E; e += kThreads) s_counts[e] = 0;
  for (int i = 0; i < kAhead; ++i) columns.clear(mine + i * kPass, true, row + i * kRows < count);
  griddep_wait();
  griddep_launch_dependents();
  if (blockIdx.x == parts.blocks) {  // the last block has no rows
    write_head(p, parts);
    return;
  }
  // passes number the rows from t0 on
  const int64_t pass_apart = kRows * apart;
  int to_fetch = row;
  const char *next = from;
  const auto fetch = [&](int slot) {
    if (to_fetch < count) columns.fetch(mine + slot * kPass, next);
    to_fetch += kRows;
    next += pass_apart;
    copies_commit();
  };
  for (int i = 0; WIDE && i < kAhead; ++i) fetch(i);
  // the choices of a pass's rows, kThreads apart: read a pass ahead
  int64_t choice[kChoices];
  int choice_row[kChoices];
  const int64_t *choices = p.topk_idx + (int64_t)t0 * K + threadIdx.x;
#pragma unroll
  for (int i = 0; i < kChoices; ++i) {
    const int at = threadIdx.x + i * kThreads;
    choice_row[i] = at < kRows * K ? at / K : count;
  }
  const auto read_choices = [&](int first) {
#pragma unroll
    for (int i = 0; i < kChoices; ++i) {
      if (i * kThreads >= kRows * K) break;
      choice[i] = choice_row[i] < count - first ? choices[i * kThreads] : -1;
    }
    choices += kRows * K;
  };
  read_choices(0);
  int s = sequence_of(p.seq_offsets, T, S, t0), chosen = 0;
  // this block's rows of sequence s, from t0 on
  int a = s < S ? max(t0, offset_of(p.seq_offsets, T, s)) - t0 : count;
  int b = s < S ? min(t0 + count, offset_of(p.seq_offsets, T, s + 1)) - t0 : count;
  float acc[V], z = 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) acc[j] = 0.0f;
  __syncthreads();
  int slot = 0;
  for (int done = 0; done < count; done += kRows, from += pass_apart) {
    const int r = done + row, behind = done + kRows;
    float l[V];
    if (WIDE) copies_wait<kAhead - 1>();
    columns.load(mine + slot * kPass, from, r < count, kNegInf, l);
    if (WIDE) fetch(slot);
    if (++slot == kAhead) slot = 0;
    int now[kChoices];
#pragma unroll
    for (int i = 0; i < kChoices; ++i) {
      if (i * kThreads >= kRows * K) break;
      now[i] = choice[i] >= 0 && choice[i] < E ? (int)choice[i] : -1;
    }
    if (behind < count) read_choices(behind);
    Scores<V, SIGMOID, false> sc;
    scores_of<L>(l, sc);
    // the sequences that the pass's rows belong to: mostly one
    while (a < behind && s < S) {
      const bool here = r >= a && r < b;
      const float inv = here ? sc.inv : 0.0f;
#pragma unroll
      for (int j = 0; j < V; ++j) acc[j] = fmaf(sc.e[j], inv, acc[j]);
      if (here && columns.lane == 0) z = fmaf(sc.lse, sc.lse, z);
#pragma unroll
      for (int i = 0; i < kChoices; ++i) {
        if (i * kThreads >= kRows * K) break;
        const int of = done + choice_row[i];
        if (now[i] >= 0 && of >= a && of < b) {
          atomicAdd(&s_counts[now[i]], 1);
          ++chosen;
        }
      }
      if (b > behind || (b == behind && b < count)) break;
      // the sequence, or the block, ends here: its segment.  The warp's rows,
      // then the warps.
#pragma unroll
      for (int j = 0; j < V; ++j) {
#pragma unroll
        for (int o = L; o < 32; o <<= 1) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], o);
      }
      const int64_t segment = (int64_t)blockIdx.x + s;
      if (lane < L) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int c = columns.column(j / columns.kPiece, j % columns.kPiece);
          if (L > 32 && c < E) parts.probs[segment * E + c] = acc[j];
          if (L <= 32 && c < E) s_probs[warp * E + c] = acc[j];
        }
      }
      chosen = __reduce_add_sync(0xffffffffu, chosen);
      if (lane == 0) s_chosen[warp] = chosen;
      __syncthreads();
      for (int e = threadIdx.x; e < E; e += kThreads) {
        if (L <= 32) {
          float sum = s_probs[e];
#pragma unroll
          for (int w = 1; w < kWarps; ++w) sum += s_probs[w * E + e];
          parts.probs[segment * E + e] = sum;
        }
        parts.counts[segment * E + e] = s_counts[e];
        s_counts[e] = 0;
      }
      if (threadIdx.x == 0) {
        for (int w = 1; w < kWarps; ++w) chosen += s_chosen[w];
        parts.chosen[segment] = chosen;
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < V; ++j) acc[j] = 0.0f;
      chosen = 0;
      do {  // the next one with rows
        ++s;
        a = s < S ? max(t0, offset_of(p.seq_offsets, T, s)) - t0 : count;
        b = s < S ? min(t0 + count, offset_of(p.seq_offsets, T, s + 1)) - t0 : count;
      } while (s < S && a < count && a >= b);
      if (a >= count) s = S;
    }
  }
  // (only a row's first lane has added to z)
  z = lanes_sum<32>(z);
  if (lane == 0) s_z[warp] = z;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kWarps; ++w) z += s_z[w];
    if (!parts.joined) parts.z[blockIdx.x] = z;
  }
  if (parts.joined) join_in_cluster(p, parts, z);
}

__device__ __forceinline__ int warp_sum(int v) { return __reduce_add_sync(0xffffffffu, v); }
__device__ __forceinline__ int64_t warp_sum(int64_t v) {  // not negative, below 2^52
  const uint32_t low = (uint32_t)v & 0x3ffffffu, high = (uint32_t)(v >> 26);  // neither one's sum leaves 32 bits
  return (int64_t)__reduce_add_sync(0xffffffffu, low) + ((int64_t)__reduce_add_sync(0xffffffffu, high) << 26);
}

constexpr int kJoinThreads = 1024, kJoinWarps = kJoinThreads / 32;
constexpr int kAtOnce = 15;  // segments that a lane reads at once: 480 of a sequence by 32 warps

// How the segments are joined: 32 experts of a sequence are a job of `warps`
// warps (a power of two).  Few segments are joined by one cluster, whose
// blocks add up the losses in its shared memory; else the block that ends last
// does it, 2 us later, where eight SMs would take longer to read them (65 536
// tokens, 256 experts, one sequence, 0.6 MB: the whole call 17.9 us, the other
// way 20.7; 16 384 of 1000, 2.4 MB: 29.8 and 28.5).
constexpr int64_t kClusterBytes = 1 << 20;

struct Join {
  int warps, blocks;
  bool cluster;
};

Join join_of(const Cut &cut, int E, int S) {
  const int64_t jobs = (int64_t)S * ((E + 31) / 32);
  Join j;
  j.cluster = jobs <= kClusterMost * kJoinWarps && ((int64_t)cut.blocks + S) * E * 8 <= kClusterBytes;
  j.warps = 1;
  if (j.cluster) {
    const int each = (int)((jobs + kClusterMost - 1) / kClusterMost);  // jobs of a block
    while (2 * j.warps * each <= kJoinWarps) j.warps *= 2;
  } else {
    const int mean = cut.blocks / S + 1;
    while (j.warps < kJoinWarps && j.warps * kAtOnce < mean) j.warps *= 2;
  }
  const int of_block = kJoinWarps / j.warps;
  j.blocks = (int)((jobs + of_block - 1) / of_block);
  return j;
}

// Block 0 adds up z too.  COUNT: what holds the choices of a sequence, 64 bits
// where a batch has 2^31 or more (65 536 tokens, 256 experts: 0.7 us longer).
template <typename COUNT>
__global__ void __launch_bounds__(kJoinThreads) balance_join_kernel(BalanceArgs p, Parts parts, Join join) {
  __shared__ float s_probs[kJoinWarps][32], s_part[kJoinWarps], s_z[kJoinWarps], s_loss;
  __shared__ COUNT s_counts[kJoinWarps][32], s_chosen[kJoinWarps];
  __shared__ int s_last;
  const int E = p.num_experts, T = p.num_tokens, S = p.num_sequences, tiles = (E + 31) / 32;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int of_block = kJoinWarps / join.warps, sub = warp % join.warps;
  const int64_t job = (int64_t)blockIdx.x * of_block + warp / join.warps;
  const bool some = job < (int64_t)S * tiles;
  const int s = some ? (int)(job / tiles) : 0, e = some ? (int)(job % tiles) * 32 + lane : E;
  // (the offsets are no work of the kernel ahead, which started after all that
  // was before it had ended; from L2, which that reached)
  int a = 0, b = T;
  if (p.seq_offsets != nullptr) {
    a = min(max(__ldcg(p.seq_offsets + s), 0), T);
    b = min(max(__ldcg(p.seq_offsets + s + 1), 0), T);
  }
  const int b0 = a / parts.tokens, b1 = some && b > a ? (b - 1) / parts.tokens : b0 - 1;
  griddep_wait();
  griddep_launch_dependents();
  const int full = parts.head[0], bad = parts.head[1];
  float prob = 0.0f, z = 0.0f;
  COUNT count = 0, chosen = 0;
  for (int i = b0 + sub * 32 + lane; i <= b1; i += join.warps * 32) chosen += parts.chosen[i + s];
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < parts.blocks; i += kJoinThreads) z += parts.z[i];
  const int64_t from = (int64_t)s * E + e;
  for (int i = b0 + sub; i <= b1; i += join.warps * kAtOnce) {
    float v[kAtOnce];
    int c[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int at = i + k * join.warps;
      const bool there = e < E && at <= b1;
      v[k] = there ? parts.probs[from + (int64_t)at * E] : 0.0f;
      c[k] = there ? parts.counts[from + (int64_t)at * E] : 0;
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      prob += v[k];
      count += c[k];
    }
  }
  s_probs[warp][lane] = prob;
  s_counts[warp][lane] = count;
  chosen = warp_sum(chosen);
  z = lanes_sum<32>(z);
  if (lane == 0) {
    s_chosen[warp] = chosen;
    s_z[warp] = z;
  }
  __syncthreads();
  float part = 0.0f;
  if (sub == 0 && some) {  // the job's warps in their order
    for (int w = 1; w < join.warps; ++w) {
      prob += s_probs[warp + w][lane];
      count += s_counts[warp + w][lane];
      chosen += s_chosen[warp + w];
    }
    if (e < E) part = finish_expert(p, s, e, b - a, prob, count, chosen, full);
  }
  part = lanes_sum<32>(part);
  if (lane == 0) s_part[warp] = part;
  __syncthreads();
  if (warp == 0) {
    part = lanes_sum<32>(s_part[lane]);
    z = lanes_sum<32>(s_z[lane]);
    if (lane == 0 && blockIdx.x == 0) {
      const int tokens = offset_of(p.seq_offsets, T, S) - offset_of(p.seq_offsets, T, 0);
      p.losses[1] = loss_of(tokens > 0 ? z / tokens : 0.0f, bad);
    }
  }
  float balance = 0.0f;
  if (join.cluster) {
    if (threadIdx.x == 0) s_loss = part;
    cluster_sync();
    if (blockIdx.x == 0 && threadIdx.x == 0) {
      float v[kClusterMost];
#pragma unroll
      for (int k = 0; k < kClusterMost; ++k)
        v[k] = k < (int)gridDim.x ? load_cluster(map_shared(smem_addr(&s_loss), k)) : 0.0f;
#pragma unroll
      for (int k = 0; k < kClusterMost; ++k) balance += v[k];
      p.losses[0] = loss_of(balance, bad);
    }
    cluster_sync();  // before a block whose loss is read ends
    return;
  }
  if (threadIdx.x == 0) {
    parts.balance[blockIdx.x] = part;
    __threadfence();
    s_last = atomicAdd(parts.head + 2, 1) == (int)gridDim.x - 1;
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  for (int64_t i = threadIdx.x; i < (int64_t)gridDim.x; i += kJoinThreads) balance += __ldcg(parts.balance + i);
  balance = lanes_sum<32>(balance);
  if (lane == 0) s_part[warp] = balance;
  __syncthreads();
  if (warp != 0) return;
  balance = lanes_sum<32>(s_part[lane]);
  if (lane == 0) p.losses[0] = loss_of(balance, bad);
}

// Without tokens nobody else looks at the offsets.
__global__ void __launch_bounds__(kThreads) balance_empty_kernel(BalanceArgs p, Parts parts) {
  griddep_wait();
  griddep_launch_dependents();
  write_head(p, parts);
}

template <bool BF16, int L, int V, bool WIDE, bool SIGMOID>
__global__ void __launch_bounds__(kThreads, 2) balance_backward_kernel(BalanceBackwardArgs p, int tokens) {
  extern __shared__ int4 s_rows[];  // [ahead][logits, add][pieces][threads]
  constexpr int kRows = kThreads / L, kSize = BF16 ? 2 : 4, kPass = pass_bytes<BF16, V>();
  constexpr int kAhead = V > 16 && !BF16 ? 1 : 3;
  const int E = p.num_experts, T = p.num_tokens, S = p.num_sequences;
  const Columns<BF16, L, V, WIDE> columns{E, (int)threadIdx.x % L};
  char *mine = reinterpret_cast<char *>(s_rows + threadIdx.x);
  const int t0 = blockIdx.x * tokens, count = min(T - t0, tokens), row = threadIdx.x / L;
  const int64_t apart = p.row_stride * kSize, packed = (int64_t)E * kSize;
  const char *from = static_cast<const char *>(p.logits) + (t0 + row) * apart;
  const char *add_from = static_cast<const char *>(p.add) + (t0 + row) * packed;
  char *out = static_cast<char *>(p.grad_logits) + (t0 + row) * packed;
  for (int i = 0; i < kAhead; ++i) {
    columns.clear(mine + i * 2 * kPass, true, row + i * kRows < count);
    columns.clear(mine + (i * 2 + 1) * kPass, false, true);
  }
  griddep_wait();
  griddep_launch_dependents();
  const int64_t pass_apart = kRows * apart, pass_packed = kRows * packed;
  int to_fetch = row;
  const char *next = from, *next_add = add_from;
  const auto fetch = [&](int slot) {
    if (to_fetch < count) {
      columns.fetch(mine + slot * 2 * kPass, next);
      if (p.add != nullptr) columns.fetch(mine + (slot * 2 + 1) * kPass, next_add);
    }
    to_fetch += kRows;
    next += pass_apart;
    next_add += pass_packed;
    copies_commit();
  };
  for (int i = 0; WIDE && i < kAhead; ++i) fetch(i);
  const int first = offset_of(p.seq_offsets, T, 0), last = offset_of(p.seq_offsets, T, S);
  const float db = p.grad_losses[0], dz = p.grad_losses[1] * 2.0f / max(1, last - first);
  float slope[V];
  int end = -1, slot = 0;  // of the sequence whose slopes are held
  for (int done = 0; done < count; done += kRows, from += pass_apart, add_from += pass_packed, out += pass_packed) {
    const int r = done + row, t = t0 + r;
    const bool there = r < count;
    if (there && t >= end) {
      const int s = sequence_of(p.seq_offsets, T, S, t);
      end = s < S ? offset_of(p.seq_offsets, T, s + 1) : INT32_MAX;
      if (s < S) columns.floats(p.slopes + (int64_t)s * E, slope);
    }
    const bool inside = there && end < INT32_MAX && t >= first;
    const char *here = mine + slot * 2 * kPass;
    float l[V], add[V];
    if (WIDE) copies_wait<kAhead - 1>();
    columns.load(here, from, there, kNegInf, l);
    if (p.add != nullptr) columns.load(here + kPass, add_from, there, 0.0f, add);
    if (WIDE) fetch(slot);
    if (++slot == kAhead) slot = 0;
    Scores<V, SIGMOID, true> sc;
    scores_of<L>(l, sc);
    float dot = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) dot = fmaf(sc.e[j], slope[j], dot);
    dot = lanes_sum<L>(dot) * sc.inv;
    const float scale = db * sc.inv, tail = fminf(fmaxf(dz * sc.lse * sc.inv_soft, -kMost), kMost);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float d = sc.e[j] * scale * (slope[j] - dot);
      if (SIGMOID) d *= sc.side[SIGMOID ? j : 0];
      d = fmaf(SIGMOID ? sc.soft[SIGMOID ? j : 0] : sc.e[j], tail, d);
      d = inside ? d : 0.0f;
      l[j] = p.add != nullptr ? add[j] + d : d;
    }
    if (there) columns.store(out, l);
  }
}

size_t round16(size_t n) { return (n + 15) / 16 * 16; }

Parts parts_of(const BalanceArgs &a) {
  const Cut cut = cut_of(a.num_tokens, a.num_experts, a.num_sequences);
  const size_t E = a.num_experts, segments = (size_t)cut.blocks + a.num_sequences;
  char *at = static_cast<char *>(a.workspace);
  const auto take = [&](size_t bytes) {
    char *p = at;
    at += round16(bytes);
    return p;
  };
  Parts p;
  p.head = reinterpret_cast<int32_t *>(take(16));
  p.probs = reinterpret_cast<float *>(take(segments * E * 4));
  p.counts = reinterpret_cast<int32_t *>(take(segments * E * 4));
  p.chosen = reinterpret_cast<int32_t *>(take(segments * 4));
  p.z = reinterpret_cast<float *>(take(segments * 4));
  p.balance = reinterpret_cast<float *>(take(a.num_sequences * ((E + 31) / 32) * 4));
  p.tokens = cut.tokens;
  p.blocks = cut.blocks;
  p.joined = cut.joined;
  return p;
}

// Rows of whole 16 bytes.
bool wide_rows(const void *p, int64_t stride, int E, bool bf16) {
  const int piece = bf16 ? 8 : 4;
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride % piece == 0 && E % piece == 0;
}

// The limit of shared memory belongs to the kernel: set once, to the most that
// any call needs.
template <typename Kernel>
cudaError_t allow_shared(Kernel *kernel, size_t bytes, std::atomic<bool> *ready) {
  if (*ready) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  *ready = e == cudaSuccess;
  return e;
}

template <bool BF16, int L, int V, bool WIDE, bool SIGMOID>
cudaError_t launch_lanes_as(const BalanceArgs &a, const Parts &parts, int device, cudaStream_t stream) {
  static std::atomic<bool> ready[64];
  const auto smem = [](int experts) {
    return (size_t)(WIDE ? ahead<BF16, V>() * pass_bytes<BF16, V>() : 0) + (size_t)(L > 32 ? 1 : kWarps + 1) * experts * 4;
  };
  const auto kernel = balance_kernel<BF16, L, V, WIDE, SIGMOID>;
  const cudaError_t e = allow_shared(kernel, smem(L * V), &ready[device]);
  if (e != cudaSuccess) return e;
  if (parts.joined) return launch_clusters(kernel, parts.blocks, kThreads, smem(a.num_experts), stream, parts.blocks, a, parts);
  return launch_kernel(kernel, parts.blocks + 1, kThreads, smem(a.num_experts), stream, false, a, parts);
}

template <bool BF16, int L, int V>
cudaError_t launch_lanes(const BalanceArgs &a, const Parts &parts, bool wide, int device, cudaStream_t stream) {
  if (wide)
    return a.sigmoid ? launch_lanes_as<BF16, L, V, true, true>(a, parts, device, stream)
                     : launch_lanes_as<BF16, L, V, true, false>(a, parts, device, stream);
  return a.sigmoid ? launch_lanes_as<BF16, L, V, false, true>(a, parts, device, stream)
                   : launch_lanes_as<BF16, L, V, false, false>(a, parts, device, stream);
}

template <bool BF16>
cudaError_t launch_lanes_of(const BalanceArgs &a, const Parts &parts, int device, cudaStream_t stream) {
  const bool wide = wide_rows(a.logits, a.row_stride, a.num_experts, a.bf16);
  const int E = a.num_experts;
  if (E <= 64) return launch_lanes<BF16, 8, 8>(a, parts, wide, device, stream);
  if (E <= 128) return launch_lanes<BF16, 8, 16>(a, parts, wide, device, stream);
  if (E <= 256) return launch_lanes<BF16, 8, 32>(a, parts, wide, device, stream);
  if (E <= 512) return launch_lanes<BF16, 16, 32>(a, parts, wide, device, stream);
  if (E <= kLanesMost) return launch_lanes<BF16, 32, 32>(a, parts, wide, device, stream);
  return launch_lanes<BF16, kThreads, EP_MAX_EXPERTS / kThreads>(a, parts, wide, device, stream);
}

constexpr int kGradBlocks = 304;  // two an SM

template <bool BF16, int L, int V, bool WIDE, bool SIGMOID>
cudaError_t launch_grad_as(const BalanceBackwardArgs &a, int device, cudaStream_t stream) {
  static std::atomic<bool> ready[64];
  const size_t smem = WIDE ? (size_t)(V > 16 && !BF16 ? 1 : 3) * 2 * pass_bytes<BF16, V>() : 0;
  const auto kernel = balance_backward_kernel<BF16, L, V, WIDE, SIGMOID>;
  const cudaError_t e = allow_shared(kernel, smem, &ready[device]);
  if (e != cudaSuccess) return e;
  const int tokens = std::max(kTokenStep, ((a.num_tokens - 1) / kGradBlocks + kTokenStep) / kTokenStep * kTokenStep);
  return launch_kernel(kernel, (a.num_tokens - 1) / tokens + 1, kThreads, smem, stream, false, a, tokens);
}

template <bool BF16, int L, int V>
cudaError_t launch_grad(const BalanceBackwardArgs &a, bool wide, int device, cudaStream_t stream) {
  if (wide)
    return a.sigmoid ? launch_grad_as<BF16, L, V, true, true>(a, device, stream)
                     : launch_grad_as<BF16, L, V, true, false>(a, device, stream);
  return a.sigmoid ? launch_grad_as<BF16, L, V, false, true>(a, device, stream)
                   : launch_grad_as<BF16, L, V, false, false>(a, device, stream);
}

template <bool BF16>
cudaError_t launch_grad_of(const BalanceBackwardArgs &a, int device, cudaStream_t stream) {
  const int E = a.num_experts;
  const bool wide = wide_rows(a.logits, a.row_stride, E, a.bf16) && wide_rows(a.add, E, E, a.bf16) &&
                    wide_rows(a.grad_logits, E, E, a.bf16);
  if (E <= 64) return launch_grad<BF16, 8, 8>(a, wide, device, stream);
  if (E <= 128) return launch_grad<BF16, 8, 16>(a, wide, device, stream);
  if (E <= 256) return launch_grad<BF16, 16, 16>(a, wide, device, stream);
  if (E <= 512) return launch_grad<BF16, 32, 16>(a, wide, device, stream);
  if (E <= kLanesMost) return launch_grad<BF16, 32, 32>(a, wide, device, stream);
  return launch_grad<BF16, kThreads, EP_MAX_EXPERTS / kThreads>(a, wide, device, stream);
}

}  // namespace

size_t balance_workspace_bytes(int T, int E, int S) {
  const size_t segments = (size_t)cut_of(T, E, S).blocks + S;
  return 16 + 2 * round16(segments * E * 4) + 2 * round16(segments * 4) + round16((size_t)S * ((E + 31) / 32) * 4);
}

ep_status_t launch_balance(const BalanceArgs &a, cudaStream_t stream) {
  const Parts parts = parts_of(a);
  const DeviceInfo *di = current_device_info();
  if (di == nullptr) return EP_ERR_CUDA;
  cudaError_t e;
  if (a.num_tokens == 0)
    e = launch_kernel(balance_empty_kernel, 1, kThreads, 0, stream, false, a, parts);
  else
    e = a.bf16 ? launch_lanes_of<true>(a, parts, di->device, stream) : launch_lanes_of<false>(a, parts, di->device, stream);
  if (e == cudaSuccess && parts.joined) return EP_OK;
  const Join join = join_of(cut_of(a.num_tokens, a.num_experts, a.num_sequences), a.num_experts, a.num_sequences);
  const auto kernel = (int64_t)a.num_tokens * a.num_topk > INT32_MAX ? balance_join_kernel<int64_t> : balance_join_kernel<int>;
  if (e == cudaSuccess)
    e = join.cluster ? launch_clusters(kernel, join.blocks, kJoinThreads, 0, stream, join.blocks, a, parts, join)
                     : launch_kernel(kernel, join.blocks, kJoinThreads, 0, stream, false, a, parts, join);
  return e == cudaSuccess ? EP_OK : cuda_fail(e, "balance launch");
}

ep_status_t launch_balance_backward(const BalanceBackwardArgs &a, cudaStream_t stream) {
  if (a.num_tokens == 0) return EP_OK;
  const DeviceInfo *di = current_device_info();
  if (di == nullptr) return EP_ERR_CUDA;
  const cudaError_t e = a.bf16 ? launch_grad_of<true>(a, di->device, stream) : launch_grad_of<false>(a, di->device, stream);
  return e == cudaSuccess ? EP_OK : cuda_fail(e, "balance_backward launch");
}

}  // namespace ep
