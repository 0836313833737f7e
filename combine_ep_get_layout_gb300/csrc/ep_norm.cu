// Layer norm of rows and its gradients.
//
//   mean = sum x / H, rstd = 1 / sqrt(sum (x - mean)^2 / H + eps), n = (x - mean) rstd
//   out = n w + b
//   grad_x = rstd (g w - mean(g w) - n mean(g w n)) + add
//   grad_weight = sum over rows of g n, grad_bias = sum over rows of g
//
// Statistics and sums in fp32, results rounded once; the variance from the
// differences, in a second pass over the row in shared memory.
//
// Bound by memory.  Persistent blocks of 16 or 32 warps; a row belongs to the
// W warps that hold it with 8 U elements a thread, and a block has as many
// such groups as fit.  A thread always has the same columns: the parameters stay in its registers, the parameters'
// gradients are summed there, and it copies the next rows' pieces (cp.async)
// to shared memory that only it reads, so rows ahead need no barrier.  Only a
// row's sums cross threads; the forward pass takes two rows at a time, so
// that they share the two barriers.  Arithmetic on pairs of fp32 (one
// instruction for two).
#include <atomic>

#include "ep_ops.h"
#include "ep_tc.cuh"

namespace ep {

namespace {

constexpr int kMaxWarps = 32;    // of a block of the forward pass with U = 1; others have half
constexpr int kMaxBlocks = 152;  // that sum rows for the parameters' gradients

__device__ __forceinline__ float load_value(const void *p, bool bf16, int64_t i) {
  return bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t *>(p)[i] << 16) : static_cast<const float *>(p)[i];
}

__device__ __forceinline__ void store_value(void *p, bool bf16, int64_t i, float v) {
  if (bf16)
    static_cast<uint16_t *>(p)[i] = (uint16_t)(pack_bf16x2(v, 0.0f) & 0xffffu);
  else
    static_cast<float *>(p)[i] = v;
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

// Two fp32 values in 64 bits: one instruction for both.
typedef unsigned long long Pair;

__device__ __forceinline__ Pair pair_of(float lo, float hi) {
  Pair v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
__device__ __forceinline__ float2 halves(Pair v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
  Pair d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ float total(Pair v) {
  const float2 f = halves(v);
  return f.x + f.y;
}

// 8 elements, from 16 or 32 bytes.
template <bool BF16>
__device__ __forceinline__ void unpack(const int4 &a, const int4 &b, Pair (&v)[4]) {
  if (BF16) {
    const uint32_t w[4] = {(uint32_t)a.x, (uint32_t)a.y, (uint32_t)a.z, (uint32_t)a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = pair_of(bf16_lo(w[j]), bf16_hi(w[j]));
  } else {
    const int w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = pair_of(__int_as_float(w[2 * j]), __int_as_float(w[2 * j + 1]));
  }
}

template <bool BF16>
__device__ __forceinline__ void pack(int4 *p, const Pair (&v)[4]) {
  float2 f[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] = halves(v[j]);
  if (BF16) {
    p[0] = make_int4((int)pack_bf16x2(f[0].x, f[0].y), (int)pack_bf16x2(f[1].x, f[1].y), (int)pack_bf16x2(f[2].x, f[2].y),
                     (int)pack_bf16x2(f[3].x, f[3].y));
  } else {
    p[0] = make_int4(__float_as_int(f[0].x), __float_as_int(f[0].y), __float_as_int(f[1].x), __float_as_int(f[1].y));
    p[1] = make_int4(__float_as_int(f[2].x), __float_as_int(f[2].y), __float_as_int(f[3].x), __float_as_int(f[3].y));
  }
}

// How a call's rows meet its threads.
struct Shape {
  int warps;    // of a row
  int groups;   // of a block
  bool joined;  // the gradients' blocks are a cluster, which adds up the parameters' itself
};

// How a thread meets a row: its elements one by one, a row's threads apart;
// or, where rows come in 16 bytes, by pieces of 16, a row's threads apart
// too: straight from memory, or through the rows ahead in shared memory.
enum Mode { kElements, kPieces, kRing };

// A thread's place, and its 8 U columns.
template <bool BF16, int U, Mode M>
struct Place {
  static constexpr bool kWide = M != kElements;
  static constexpr int kSize = BF16 ? 2 : 4;
  static constexpr int kCount = BF16 ? 1 : 2;    // pieces of 8 elements
  static constexpr int kLength = 8 / kCount;     // of a piece
  int hidden, threads, group, at;

  __device__ Place(const Shape &s, int hidden_) : hidden(hidden_), threads(s.warps * 32) {
    group = s.groups == 1 ? 0 : (int)threadIdx.x / threads;
    at = threadIdx.x - group * threads;
  }
  __device__ int column(int u, int j) const {
    return kWide ? ((u * kCount + j / kLength) * threads + at) * kLength + j % kLength : (u * 8 + j) * threads + at;
  }
  __device__ bool there(int u, int j) const { return column(u, j) < hidden; }
  // Copies this thread's pieces of a row (`from` its first column) to `to`,
  // a block's threads apart.
  __device__ void fetch(uint32_t to, const char *from) const {
#pragma unroll
    for (int i = 0; i < U * kCount; ++i)
      if ((i * threads + at) * kLength < hidden) copy_piece(to + i * blockDim.x * 16, from + (size_t)i * threads * 16);
  }
  // Zeros there for the pieces past the row's end, which no copy brings.
  __device__ void clear(char *here) const {
#pragma unroll
    for (int i = 0; i < U * kCount; ++i)
      if ((i * threads + at) * kLength >= hidden) *reinterpret_cast<int4 *>(here + i * blockDim.x * 16) = make_int4(0, 0, 0, 0);
  }
  // ... and reads them there.
  __device__ void fetched(const char *here, int u, Pair (&v)[4]) const {
    int4 f[kCount];
#pragma unroll
    for (int i = 0; i < kCount; ++i) f[i] = *reinterpret_cast<const int4 *>(here + (u * kCount + i) * blockDim.x * 16);
    unpack<BF16>(f[0], f[kCount - 1], v);
  }
  // `row` not modified while it is read (but by its reader, later).
  __device__ void raw(const char *row, int u, int4 (&f)[kCount]) const {
#pragma unroll
    for (int i = 0; i < kCount; ++i) {
      f[i] = make_int4(0, 0, 0, 0);
      if (there(u, i * kLength)) f[i] = *reinterpret_cast<const int4 *>(row + (size_t)column(u, i * kLength) * kSize);
    }
  }
  __device__ void load(const char *row, int u, Pair (&v)[4]) const {
    if (kWide) {
      int4 f[kCount];
      raw(row, u, f);
      unpack<BF16>(f[0], f[kCount - 1], v);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[j] = pair_of(there(u, 2 * j) ? load_value(row, BF16, column(u, 2 * j)) : 0.0f,
                       there(u, 2 * j + 1) ? load_value(row, BF16, column(u, 2 * j + 1)) : 0.0f);
    }
  }
  __device__ void store(char *row, int u, const Pair (&v)[4]) const {
    if (kWide) {
      int4 f[2];
      pack<BF16>(f, v);
#pragma unroll
      for (int i = 0; i < kCount; ++i)
        if (there(u, i * kLength)) *reinterpret_cast<int4 *>(row + (size_t)column(u, i * kLength) * kSize) = f[i];
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = halves(v[j]);
        if (there(u, 2 * j)) store_value(row, BF16, column(u, 2 * j), f.x);
        if (there(u, 2 * j + 1)) store_value(row, BF16, column(u, 2 * j + 1), f.y);
      }
    }
  }
  // The sum of squares, of the columns that are there.
  __device__ Pair squares(int u, const Pair (&v)[4], Pair sum) const {
    if (kWide) {
#pragma unroll
      for (int i = 0; i < kCount; ++i) {
        Pair part = sum;
#pragma unroll
        for (int j = i * 4 / kCount; j < (i + 1) * 4 / kCount; ++j) part = fma2(v[j], v[j], part);
        if (there(u, i * kLength)) sum = part;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = halves(v[j]);
        const Pair only = pair_of(there(u, 2 * j) ? f.x : 0.0f, there(u, 2 * j + 1) ? f.y : 0.0f);
        sum = fma2(only, only, sum);
      }
    }
    return sum;
  }
  // fp32 at the thread's columns, in a row of `hidden` (16-byte aligned with
  // pieces).
  __device__ void store_floats(float *row, int u, const Pair (&v)[4]) const {
#pragma unroll
    for (int j = 0; j < 8; j += 4) {
      const float2 a = halves(v[j / 2]), b = halves(v[j / 2 + 1]);
      if (kWide) {
        if (there(u, j)) *reinterpret_cast<float4 *>(row + column(u, j)) = make_float4(a.x, a.y, b.x, b.y);
      } else {
        const float f[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (there(u, j + k)) row[column(u, j + k)] = f[k];
      }
    }
  }
  __device__ void add_floats(const float *row, int u, Pair (&v)[4]) const {
#pragma unroll
    for (int j = 0; j < 8; j += 4) {
      float f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      if (kWide) {
        if (there(u, j)) *reinterpret_cast<float4 *>(f) = *reinterpret_cast<const float4 *>(row + column(u, j));
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (there(u, j + k)) f[k] = row[column(u, j + k)];
      }
      v[j / 2] = add2(v[j / 2], pair_of(f[0], f[1]));
      v[j / 2 + 1] = add2(v[j / 2 + 1], pair_of(f[2], f[3]));
    }
  }
  // Parameters: fp32 or bf16, aligned to their elements (`p` null: `none`).
  __device__ void params(const void *p, bool bf16, float none, int u, Pair (&v)[4]) const {
    float f[8];
    if (kWide && p != nullptr && reinterpret_cast<uintptr_t>(p) % 16 == 0) {
#pragma unroll
      for (int j = 0; j < 8; j += 4) {
        float4 w = make_float4(none, none, none, none);
        if (there(u, j)) {
          if (bf16) {
            const uint2 h = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + column(u, j)));
            w = make_float4(bf16_lo(h.x), bf16_hi(h.x), bf16_lo(h.y), bf16_hi(h.y));
          } else {
            w = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(p) + column(u, j)));
          }
        }
        f[j] = w.x;
        f[j + 1] = w.y;
        f[j + 2] = w.z;
        f[j + 3] = w.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = p != nullptr && there(u, j) ? load_value(p, bf16, column(u, j)) : none;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = pair_of(f[2 * j], f[2 * j + 1]);
  }
};

// a and b summed over the warp: a in lanes 0 to 15, b in the others.
__device__ __forceinline__ float warp_totals(float a, float b) {
  const bool low = (threadIdx.x & 16) == 0;
  float v = (low ? a : b) + __shfl_xor_sync(0xffffffffu, low ? b : a, 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The warps' sums of a row: of its group's warps, in two buffers that calls
// take in turn, so one barrier a call is enough.
struct Sums {
  float v[2][kMaxWarps][2];
};

// a and b summed over a row's threads, the same in all of them.
__device__ __forceinline__ void row_totals(float &a, float &b, Sums &s, int turn, int warps, int group) {
  float v = warp_totals(a, b);
  if (warps > 1) {
    const int lane = threadIdx.x & 31;
    if ((lane & 15) == 0) s.v[turn][threadIdx.x / 32][lane >> 4] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(warps * 32) : "memory");
    float2 f = make_float2(0.0f, 0.0f);
    if (lane < warps) f = *reinterpret_cast<const float2 *>(s.v[turn][group * warps + lane]);
    v = warp_totals(f.x, f.y);
  }
  a = __shfl_sync(0xffffffffu, v, 0);
  b = __shfl_sync(0xffffffffu, v, 16);
}

// Rows that a group takes at a time.  Twice as many are in shared memory, up
// to 32 KB each time (bf16, two rows of 8192; four times as many: 8192 rows of
// 7168 41.6 us instead of 41.0, 65 536 of 512 24.5 instead of 22.9).
constexpr int rows_at_once(int pieces) { return pieces == 1 ? 2 : 1; }
constexpr int kForwardAhead = 2;
constexpr int most_warps(int pieces) { return pieces == 1 ? kMaxWarps : kMaxWarps / 2; }

template <bool BF16, int U, Mode M>
__global__ void __launch_bounds__(most_warps(U) * 32, 1) norm_kernel(NormArgs p, Shape shape) {
  extern __shared__ int4 s_ring[];
  constexpr int R = rows_at_once(U), kAhead = kForwardAhead;
  __shared__ Sums s_sums;
  using At = Place<BF16, U, M>;
  const At at(shape, p.hidden);
  constexpr int kSize = At::kSize;
  const uint32_t T = p.num_rows, step = gridDim.x * shape.groups * R;
  uint32_t t = (blockIdx.x * shape.groups + at.group) * R;
  // what one time of fetching takes, and this thread's place in it
  const uint32_t row_bytes = U * At::kCount * blockDim.x * 16, slot_bytes = R * row_bytes;
  char *mine = reinterpret_cast<char *>(s_ring + threadIdx.x);
  int slot = 0;
  uint32_t next = t;
  const int64_t apart = p.row_stride * kSize, packed = (int64_t)p.hidden * kSize;
  const char *from = static_cast<const char *>(p.x) + next * apart + at.column(0, 0) * kSize;
  char *out = static_cast<char *>(p.out) + t * packed;
  const auto fetch = [&](int into) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (next + r < T) at.fetch(smem_addr(mine) + into * slot_bytes + r * row_bytes, from + r * apart);
    next += step;
    from += step * apart;
    copies_commit();
  };
  if (M == kRing) {
    for (int i = 0; i < kAhead * R; ++i) at.clear(mine + i * row_bytes);
  }
  griddep_wait();
  griddep_launch_dependents();
  if (M == kRing) {
    for (int i = 0; i < kAhead; ++i) fetch(i);
  }
  Pair w[U][4], b[U][4];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    at.params(p.weight, p.param_bf16, 1.0f, u, w[u]);
    at.params(p.bias, p.param_bf16, 0.0f, u, b[u]);
  }
  const float share = 1.0f / p.hidden;
  for (; t < T; t += step, out += step * packed) {
    Pair x[R][U][4];
    float v[2] = {0.0f, 0.0f};
    if (M == kRing) copies_wait<kAhead - 1>();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      Pair sum = pair_of(0.0f, 0.0f);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (M == kRing)
          at.fetched(mine + slot * slot_bytes + r * row_bytes, u, x[r][u]);
        else
          at.load(static_cast<const char *>(p.x) + (t + r < T ? t + r : t) * apart, u, x[r][u]);
#pragma unroll
        for (int j = 0; j < 4; ++j) sum = add2(sum, x[r][u][j]);
      }
      v[r] = total(sum);
    }
    if (M == kRing) {
      fetch(slot);
      if (++slot == kAhead) slot = 0;
    }
    row_totals(v[0], v[1], s_sums, 0, shape.warps, at.group);
    float mean[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mean[r] = v[r] * share;
      const Pair minus = pair_of(-mean[r], -mean[r]);
      Pair sum = pair_of(0.0f, 0.0f);
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[r][u][j] = add2(x[r][u][j], minus);
        sum = at.squares(u, x[r][u], sum);
      }
      v[r] = total(sum);
    }
    row_totals(v[0], v[1], s_sums, 1, shape.warps, at.group);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (t + r >= T) break;
      const float rstd = rsqrtf(v[r] * share + p.eps);
      if (at.at == 0) {
        if (p.mean != nullptr) p.mean[t + r] = mean[r];
        if (p.rstd != nullptr) p.rstd[t + r] = rstd;
      }
      const Pair scale = pair_of(rstd, rstd);
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[r][u][j] = fma2(mul2(x[r][u][j], scale), w[u][j], b[u][j]);
        at.store(out + r * packed, u, x[r][u]);
      }
    }
  }
}

// Rows of the backward pass (x, grad and add of each) in shared memory: up to
// 48 KB a row of 8192 in bf16, 96 KB in fp32; fp32 rows beyond 8192 come
// straight from memory.  (Four rows of 7168 in bf16 were slower, 83 us against
// 81.6, and two of 16 384, 155 against 142.)
constexpr int backward_ahead(int pieces) { return pieces == 4 ? 1 : 2; }

// grad_x, and this block's part of the parameters' gradients: [block][2][hidden].
template <bool BF16, int U, Mode M>
__global__ void __launch_bounds__(kMaxWarps * 16, 1) norm_backward_kernel(NormBackwardArgs p, Shape shape) {
  extern __shared__ int4 s_ring[];
  constexpr int kAhead = backward_ahead(U);
  __shared__ Sums s_sums;
  using At = Place<BF16, U, M>;
  const At at(shape, p.hidden);
  constexpr int kSize = At::kSize;
  const uint32_t T = p.num_rows, step = gridDim.x * shape.groups;
  uint32_t t = blockIdx.x * shape.groups + at.group;
  const bool added = p.add != nullptr && p.grad_x != nullptr;
  const uint32_t row_bytes = U * At::kCount * blockDim.x * 16, slot_bytes = 3 * row_bytes;
  char *mine = reinterpret_cast<char *>(s_ring + threadIdx.x);
  uint32_t next = t;
  const int64_t apart = p.row_stride * kSize, packed = (int64_t)p.hidden * kSize;
  const char *from_x = static_cast<const char *>(p.x) + next * apart + at.column(0, 0) * kSize;
  int64_t from = next * packed + at.column(0, 0) * kSize, row = t * packed;  // of grad and add
  const auto fetch = [&](int into) {
    if (next < T) {
      const uint32_t to = smem_addr(mine) + into * slot_bytes;
      at.fetch(to, from_x);
      at.fetch(to + row_bytes, static_cast<const char *>(p.grad) + from);
      if (added) at.fetch(to + 2 * row_bytes, static_cast<const char *>(p.add) + from);
    }
    next += step;
    from_x += step * apart;
    from += step * packed;
    copies_commit();
  };
  if (M == kRing) {
    for (int i = 0; i < kAhead * 3; ++i) at.clear(mine + i * row_bytes);
  }
  griddep_wait();
  griddep_launch_dependents();
  if (M == kRing) {
    for (int i = 0; i < kAhead; ++i) fetch(i);
  }
  constexpr bool kKeep = U < 4;  // the weight, and a row's y and h w, stay in registers
  constexpr int kKept = kKeep ? U : 1;
  const Pair zero = pair_of(0.0f, 0.0f);
  Pair w[kKept][4], dw[U][4], db[U][4];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (kKeep) at.params(p.weight, p.param_bf16, 1.0f, u, w[u % kKept]);
#pragma unroll
    for (int j = 0; j < 4; ++j) dw[u][j] = db[u][j] = zero;
  }
  const float share = 1.0f / p.hidden;
  int slot = 0, turn = 0;
  float mean = 0.0f, rstd = 0.0f;
  if (t < T) {
    mean = p.mean[t];
    rstd = p.rstd[t];
  }
  for (; t < T; t += step, row += step * packed) {
    // With y = x - mean and h = grad rstd, so n grad = h y:
    //   grad_x = h w - mean(h w) - y rstd (rstd mean(h w y)) + add,  grad_weight = sum h y
    // As many instructions as with n, which x rstd - (mean rstd) would give in
    // one, off by the rounding of mean rstd in a whole row alike.  (Where a row
    // is read again, g = grad w instead of h w, and rstd at the end: less to do
    // the second time.)
    const float factor = rstd;
    const Pair scale = pair_of(rstd, rstd), minus = pair_of(-mean, -mean);
    if (t + step < T) {  // the next row's, ahead
      mean = p.mean[t + step];
      rstd = p.rstd[t + step];
    }
    if (M == kRing) copies_wait<kAhead - 1>();
    const char *here = mine + slot * slot_bytes;
    const auto piece = [&](int a, int u, Pair (&v)[4]) {
      if (M == kRing)
        at.fetched(here + a * row_bytes, u, v);
      else
        at.load(a == 0   ? static_cast<const char *>(p.x) + t * apart
                : a == 1 ? static_cast<const char *>(p.grad) + row
                         : static_cast<const char *>(p.add) + row,
                u, v);
    };
    Pair y[kKept][4], gw[kKept][4], a = zero, b = zero;  // of this row; gw with kKeep times rstd
#pragma unroll
    for (int u = 0; u < U; ++u) {
      Pair x[4], g[4];
      piece(0, u, x);
      piece(1, u, g);
      const int k = u % kKept;
      if (!kKeep) at.params(p.weight, p.param_bf16, 1.0f, u, w[k]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const Pair h = mul2(g[j], scale);
        y[k][j] = add2(x[j], minus);
        gw[k][j] = mul2(kKeep ? h : g[j], w[k][j]);
        a = add2(a, gw[k][j]);
        b = fma2(gw[k][j], y[k][j], b);
        dw[u][j] = fma2(h, y[k][j], dw[u][j]);
        db[u][j] = add2(db[u][j], g[j]);
      }
    }
    if (p.grad_x != nullptr) {
      float av = total(a), bv = total(b);
      row_totals(av, bv, s_sums, turn, shape.warps, at.group);
      turn ^= 1;
      av *= -share;
      bv = bv * -share * factor * factor;  // (one after the other: the square alone may not be finite)
      a = pair_of(av, av);
      b = pair_of(bv, bv);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = u % kKept;
        Pair plus[4] = {zero, zero, zero, zero};
        if (!kKeep) {
          piece(0, u, y[k]);
          piece(1, u, gw[k]);
          at.params(p.weight, p.param_bf16, 1.0f, u, w[k]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            y[k][j] = add2(y[k][j], minus);
            gw[k][j] = mul2(gw[k][j], w[k][j]);
          }
        }
        if (added) piece(2, u, plus);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const Pair d = add2(fma2(y[k][j], b, gw[k][j]), a);
          plus[j] = !kKeep ? fma2(d, scale, plus[j]) : added ? add2(d, plus[j]) : d;
        }
        at.store(static_cast<char *>(p.grad_x) + row, u, plus);
      }
    }
    if (M == kRing) {
      fetch(slot);
      if (++slot == kAhead) slot = 0;
    }
  }
  if (p.grad_weight == nullptr && p.grad_bias == nullptr) return;
  // the groups one after the other
  float *s_params = reinterpret_cast<float *>(s_ring);  // [2][hidden]
  float *mine_of = p.workspace + (int64_t)blockIdx.x * 2 * p.hidden;
  copies_wait<0>();
  for (int i = 0; i < shape.groups; ++i) {
    __syncthreads();
    if (at.group != i) continue;
    float *to = i + 1 == shape.groups && !shape.joined ? mine_of : s_params;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i > 0) {
        at.add_floats(s_params, u, dw[u]);
        at.add_floats(s_params + p.hidden, u, db[u]);
      }
      at.store_floats(to, u, dw[u]);
      at.store_floats(to + p.hidden, u, db[u]);
    }
  }
  if (!shape.joined) return;
  cluster_sync();
  // each block a share of the columns, in the blocks' order
  const int blocks = gridDim.x, most = 2 * p.hidden;
  for (int c = (blockIdx.x * blockDim.x + threadIdx.x) * 4; c < most; c += blocks * blockDim.x * 4) {
    // (the last four of a length that is no multiple of four end past it)
    float4 v[kClusterMost];
#pragma unroll
    for (int b = 0; b < kClusterMost; ++b)
      if (b < blocks) v[b] = load_cluster4(map_shared(smem_addr(s_params + c), b));
    float sum[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
    for (int b = 1; b < kClusterMost; ++b) {
      if (b >= blocks) break;
      sum[0] += v[b].x, sum[1] += v[b].y, sum[2] += v[b].z, sum[3] += v[b].w;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int at = c + j;
      void *out = at < p.hidden ? p.grad_weight : p.grad_bias;
      if (at < most && out != nullptr) store_value(out, p.param_bf16, at < p.hidden ? at : at - p.hidden, sum[j]);
    }
  }
  cluster_sync();  // before a block whose sums are read ends
}

constexpr int kJoinWarps = 16;

// The blocks' parts, added in their order by sixteen warps, then those; a
// column a lane.
__global__ void __launch_bounds__(kJoinWarps * 32) norm_join_kernel(NormBackwardArgs p, int blocks) {
  __shared__ float s[kJoinWarps][32];
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, c = blockIdx.x * 32 + lane;
  constexpr int kEach = (kMaxBlocks + kJoinWarps - 1) / kJoinWarps;  // a warp's, all read at once
  float v[kEach], sum = 0.0f;
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int i = warp + k * kJoinWarps;
    v[k] = i < blocks && c < 2 * p.hidden ? p.workspace[(int64_t)i * 2 * p.hidden + c] : 0.0f;
  }
#pragma unroll
  for (int k = 0; k < kEach; ++k) sum += v[k];
  s[warp][lane] = sum;
  __syncthreads();
  if (warp != 0 || c >= 2 * p.hidden) return;
  for (int i = 1; i < kJoinWarps; ++i) sum += s[i][lane];
  void *out = c < p.hidden ? p.grad_weight : p.grad_bias;
  if (out != nullptr) store_value(out, p.param_bf16, c < p.hidden ? c : c - p.hidden, sum);
}

int up(int a, int b) { return (a + b - 1) / b; }

// Dynamic shared memory of a block, beside its warps' sums.
size_t shared_limit(const DeviceInfo *di) { return di->max_smem_per_block_optin - 8192; }

// Pieces of 8 elements a thread.  The forward pass does with 64 registers,
// so with 32 warps; the backward pass does not.
int forward_pieces(int hidden) { return hidden <= kMaxWarps * 256 ? 1 : 4; }
int backward_pieces(int hidden) { return hidden <= 256 ? 1 : hidden <= 8192 ? 2 : 4; }

// Rows are spread over the blocks before they share one.  Named barriers are
// few, so at most 15 groups that need one.
Shape shape_of(int rows, int hidden, int pieces, int warps, int blocks) {
  Shape s;
  s.warps = up(up(hidden, 8), 32 * pieces);
  s.joined = false;
  s.groups = warps / s.warps;
  if (s.warps > 1 && s.groups > 15) s.groups = 15;
  const int spread = up(rows, blocks);
  if (s.groups > spread) s.groups = spread;
  return s;
}

// 16-byte rows: the pointer, and the distance of rows.
bool wide_rows(const void *p, int64_t stride, bool bf16) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride * (bf16 ? 2 : 4) % 16 == 0;
}

// Few rows: their gradients are computed by one cluster, which saves the
// kernel that joins the blocks' sums, 3.4 us of the host's, up to where the
// device takes 1 to 2 us longer for it, which a graph's replay does not win back
// (in a graph, one cluster and two
// kernels: 13 rows of 4096 5.5 and 4.6 us, 48 of 1024 5.1 and 3.5, 8 of 1024
// 3.1 and 3.4; 96 of 1024 would be 7.1 and 3.7).
int cluster_rows(int groups) { return 16 + 4 * groups; }

template <typename Args>
ep_status_t launch_rows(void (*kernel)(Args, Shape), const Args &a, const Shape &s, size_t smem, int rows, int most, const DeviceInfo *di,
                        std::atomic<bool> (&ready)[64], const char *what, cudaStream_t stream) {
  // the limit belongs to the kernel, so it is the most that any call needs
  if (smem > 40 * 1024 && !ready[di->device]) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)shared_limit(di));
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
    ready[di->device] = true;
  }
  const int need = up(rows, s.groups), grid = need < most ? need : most, threads = s.groups * s.warps * 32;
  const cudaError_t e = s.joined ? launch_clusters(kernel, grid, threads, smem, stream, grid, a, s)
                                 : launch_kernel(kernel, grid, threads, smem, stream, false, a, s);
  return e == cudaSuccess ? EP_OK : cuda_fail(e, what);
}

template <bool BF16, int U, Mode M>
ep_status_t launch_norm_as(const NormArgs &a, const DeviceInfo *di, cudaStream_t stream) {
  static std::atomic<bool> ready[64];
  constexpr int R = rows_at_once(U);
  const int most = di->num_sms, rows = up(a.num_rows, R);
  const Shape s = shape_of(rows, a.hidden, U, most_warps(U), most);
  const size_t smem = M == kRing ? (size_t)kForwardAhead * R * U * (BF16 ? 16 : 32) * s.warps * s.groups * 32 : 0;
  return launch_rows(norm_kernel<BF16, U, M>, a, s, smem, rows, most, di, ready, "norm launch", stream);
}

template <bool BF16, int U, Mode M>
ep_status_t launch_norm_backward_as(const NormBackwardArgs &a, const DeviceInfo *di, int *blocks, cudaStream_t stream) {
  static std::atomic<bool> ready[64];
  int sms = di->num_sms < kMaxBlocks ? di->num_sms : kMaxBlocks;
  const bool params = a.grad_weight != nullptr || a.grad_bias != nullptr;
  Shape s = shape_of(a.num_rows, a.hidden, U, kMaxWarps / 2, sms);
  if (params) {
    const Shape few = shape_of(a.num_rows, a.hidden, U, kMaxWarps / 2, kClusterMost);
    if (a.num_rows <= cluster_rows(few.groups)) {
      s = few;
      s.joined = true;
      sms = kClusterMost;
    }
  }
  size_t smem = M == kRing ? (size_t)backward_ahead(U) * 3 * U * (BF16 ? 16 : 32) * s.warps * s.groups * 32 : 0;
  const size_t sums = (size_t)a.hidden * 8 + 16;  // the groups', with room for a last four
  if ((s.groups > 1 || s.joined) && smem < sums) smem = sums;
  *blocks = s.joined ? 0 : up(a.num_rows, s.groups) < sms ? up(a.num_rows, s.groups) : sms;
  return launch_rows(norm_backward_kernel<BF16, U, M>, a, s, smem, a.num_rows, sms, di, ready, "norm_backward launch", stream);
}

template <int U>
ep_status_t launch_norm_of(const NormArgs &a, bool wide, const DeviceInfo *di, cudaStream_t stream) {
  if (a.bf16) return wide ? launch_norm_as<true, U, kRing>(a, di, stream) : launch_norm_as<true, U, kElements>(a, di, stream);
  return wide ? launch_norm_as<false, U, kRing>(a, di, stream) : launch_norm_as<false, U, kElements>(a, di, stream);
}

template <int U>
ep_status_t launch_norm_backward_of(const NormBackwardArgs &a, bool wide, const DeviceInfo *di, int *blocks, cudaStream_t stream) {
  constexpr Mode kLong = U == 4 ? kPieces : kRing;
  if (a.bf16)
    return wide ? launch_norm_backward_as<true, U, kRing>(a, di, blocks, stream)
                : launch_norm_backward_as<true, U, kElements>(a, di, blocks, stream);
  return wide ? launch_norm_backward_as<false, U, kLong>(a, di, blocks, stream)
              : launch_norm_backward_as<false, U, kElements>(a, di, blocks, stream);
}

}  // namespace

ep_status_t launch_norm(const NormArgs &a, cudaStream_t stream) {
  if (a.num_rows == 0) return EP_OK;
  const bool wide = a.hidden % 8 == 0 && wide_rows(a.x, a.row_stride, a.bf16) && wide_rows(a.out, a.hidden, a.bf16);
  const DeviceInfo *di = current_device_info();
  if (di == nullptr) return EP_ERR_CUDA;
  return forward_pieces(a.hidden) == 1 ? launch_norm_of<1>(a, wide, di, stream) : launch_norm_of<4>(a, wide, di, stream);
}

size_t norm_workspace_bytes(int num_rows, int hidden) {
  return (size_t)(num_rows < kMaxBlocks ? num_rows : kMaxBlocks) * 2 * hidden * sizeof(float);
}

ep_status_t launch_norm_backward(const NormBackwardArgs &a, cudaStream_t stream) {
  const bool params = a.grad_weight != nullptr || a.grad_bias != nullptr;
  int blocks = 0;
  if (a.num_rows > 0 && (params || a.grad_x != nullptr)) {
    const DeviceInfo *di = current_device_info();
    if (di == nullptr) return EP_ERR_CUDA;
    const bool wide = a.hidden % 8 == 0 && wide_rows(a.x, a.row_stride, a.bf16) && wide_rows(a.grad, a.hidden, a.bf16) &&
                      wide_rows(a.add, a.hidden, a.bf16) && wide_rows(a.grad_x, a.hidden, a.bf16);
    const int pieces = backward_pieces(a.hidden);
    const ep_status_t s = pieces == 1   ? launch_norm_backward_of<1>(a, wide, di, &blocks, stream)
                          : pieces == 2 ? launch_norm_backward_of<2>(a, wide, di, &blocks, stream)
                                        : launch_norm_backward_of<4>(a, wide, di, &blocks, stream);
    if (s != EP_OK) return s;
  }
  if (!params || (a.num_rows > 0 && blocks == 0)) return EP_OK;
  const cudaError_t e = launch_kernel(norm_join_kernel, up(2 * a.hidden, 32), kJoinWarps * 32, 0, stream, false, a, blocks);
  return e == cudaSuccess ? EP_OK : cuda_fail(e, "norm_join launch");
}

}  // namespace ep
