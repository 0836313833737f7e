// Products of ragged groups of rows on the tensor cores, for pairs of CTAs:
// the kernel behind the experts' products, their gradients, the adapters'
// projection and the product shared by all rows (each includes the forms it
// launches).
//
// A pair of CTAs computes a tile of 256 x up to 256: A, the operand with 256
// rows, is the weights (so the ragged number of an expert's rows meets the
// dimension that comes in steps of 32, not of 256), B the rows:
//   kPlain, kGated   A = w[e] (inner dimension hidden),  B = rows of x
//   kGradX           A = w[e]^T (inner dimension wide),  B = rows of g
//   kGradW           A = g^T, B = x^T (inner dimension the expert's rows)
//   kAdapter         kPlain with one expert, and more inner steps: A = the
//                    up-projections of the adapters that the tile's rows name,
//                    side by side, B = the rows' low-rank factors in their
//                    adapter's columns, zero in the others
//   kDense, kDenseGated, kDenseGradX, kDenseGradW
//                    the first four with one expert that has every row, and
//                    the first two with bias, activation and residual
//   kDense32, kDenseGated32
//                    those two for results kept in fp32.  The tensor cores
//                    cut off what does not fit beside a growing sum: over
//                    7168 inner elements an error of 8e-6.  So their sums of
//                    kRun steps are added up in registers, rounded: 6e-7.
//   kDenseGradWPart  kDenseGradW by segments of the rows, p.rows_each long:
//                    the sums of each in fp32, joined by another kernel
// An inner step is 64 elements, a 128-byte row of shared memory in the
// 128-byte swizzle; the transposed operands are read with their outer
// dimension contiguous, so nothing is ever transposed in memory.
//
// Roles (warps) of a CTA: two copy (A and B, a copy a step each), one issues
// the products for the pair (in the leading CTA), eight bring results from
// tensor memory through a staging buffer to memory while the next tile is
// computed, one trims the rows' ends (kGradW), four gather (kAdapter).
//
// Bounds and measurements (one GB300; 6669 GB/s copy, 1905 TFLOP/s in the
// library's product).  A step of 64 x 256 columns takes the tensor cores 512
// cycles; the copies, the issue and the results have to stay below that.
// Dense 8192 x 4096 x 4096: 148 us, 1859 TFLOP/s (burst).  Few rows: reading
// the weights, 24 tokens top-6 of 64 experts, 4096 -> 2 x 1408, 191 to 198 us,
// 6.7 to 6.9 TB/s.  Many: the power limit (1370 W), 4096 tokens 421 to 457 us
// sustained at 1.3 GHz, 358 to 371 us in a burst.  8192 tokens top-8 of 256
// experts, 512 -> 7168: 477 to 505 us, 6 TB/s.
#pragma once

#include <atomic>
#include <cmath>

#include "ep_cut.h"
#include "ep_ops.h"
#include "ep_tc.cuh"

namespace ep {

namespace {

enum Form { kPlain, kGated, kGradX, kGradW, kAdapter, kDense, kDenseGated, kDense32, kDenseGated32, kDenseGradX, kDenseGradW, kDenseGradWPart };
__host__ __device__ constexpr bool gated(Form f) { return f == kGated || f == kDenseGated || f == kDenseGated32; }
__host__ __device__ constexpr bool grad_x(Form f) { return f == kGradX || f == kDenseGradX; }
__host__ __device__ constexpr bool grad_w(Form f) { return f == kGradW || f == kDenseGradW || f == kDenseGradWPart; }
__host__ __device__ constexpr bool dense(Form f) { return f >= kDense && f <= kDenseGated32; }  // with the epilogue
__host__ __device__ constexpr bool runs(Form f) { return f == kDense32 || f == kDenseGated32; }
__host__ __device__ constexpr bool single(Form f) { return f >= kAdapter; }  // one expert, its rows known to the host

// Warps: 0 and 3 copies of A and B, 1 products, 2 row ends (kGradW), 4-11
// results; kAdapter: 12-15 gather the adapters.
constexpr int kGatherWarps = 4;
__host__ __device__ constexpr int threads_of(Form f) { return f == kAdapter ? 384 + 32 * kGatherWarps : 384; }
constexpr int kInner = 64;           // elements of an inner step
constexpr int kABytes = 128 * 128;   // a CTA's half of A for one step
constexpr int kMaxCols = 256;        // columns of a tile
constexpr int kRun = 8;              // steps that kDense32 sums in tensor memory
__host__ __device__ constexpr int most_cols_of_form(Form f) { return runs(f) ? 128 : kMaxCols; }  // sums in 64 registers
constexpr int kTmemCols = 512;       // two tiles: one computed, one read out
constexpr int kMaxStages = 12;
constexpr int kSideStages = 4;
constexpr int kBoxes = kMaxCols / 2 / 16;  // heights of a half of B
// kAdapter, a tile: its number of adapters, their indices, each row's place among them or -1
constexpr int kPlanWords = 1 + 2 * kMaxCols;
constexpr int kPitch = 80;                       // bytes of a staged row: 64 and 16 against bank conflicts
constexpr int kStagedRows = 16;                  // of a result warp at a time
constexpr int kExchangeBytes = 8 * 32 * 4;       // kGated: 8 columns of a warp, fp32
__host__ __device__ constexpr int staging_of(Form f) { return grad_w(f) ? 32 * 128 : kStagedRows * kPitch; }
constexpr int kResultWarps = 8;
constexpr int kMaxParts = 4;         // pairs of a cluster, which share the inner dimension of one tile

struct Params {
  // One copy a step and operand (a copy costs its issuing thread about 200
  // cycles, so their number bounds a step of 512): A's 128 rows (kGated: 64
  // of the gate and the 64 that they multiply), and a half of B of any
  // height, b[i] of 16 (i + 1) rows.  Transposed operands are blocks of 64
  // outer elements; b[0] is kGradW's, of two.
  CUtensorMap a, b[kBoxes];
  bool a_blocks, b_blocks;  // both blocks in one copy (their length is a multiple of 64), else in two
  const int32_t *rows, *offset;
  uint32_t *error_word;
  int E, cap;
  int wide;      // outputs of an expert: rows of A (kPlain, kGated, kGradW), inner (kGradX)
  int width;     // kGated: wide / 2; else the outputs of a row
  int inner;     // length of the inner dimension (not kGradW)
  int a_tiles;   // tiles along A
  int b_tiles;   // kGradW: tiles along B (hidden)
  int hidden;    // kGradW
  int segments, rows_each;  // kDenseGradWPart
  CUtensorMap grad;  // kGradW: the gradient [E][wide][hidden], boxes of 64 x 32; kDenseGradWPart: [segments][wide][2 hidden]
  uint16_t *out, *preact;
  int max_cols;         // rows of a tile, at most
  int most_rows;        // of an expert, at most
  int parts;            // pairs that share a tile's inner dimension
  int ring_bytes;       // of the ring (kAdapter: both rings)
  // kAdapter
  const uint16_t *up;    // the up-projections [adapters][width][rank]
  const int32_t *plan;   // kPlanWords a tile of rows
  const uint16_t *low;   // [rows][rank], scaled
  int rank;
  // kDense and the like
  const void *bias;          // [wide] or null
  const uint16_t *residual;  // [rows][width] or null
  int activation;
  bool bias_bf16;
};

struct Barriers {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t ends[kMaxStages];   // kGradW: the last step of an expert has landed
  uint64_t fixed[kMaxStages];  // and was trimmed
  uint64_t side_full[kSideStages], side_empty[kSideStages];  // kAdapter's further steps
  uint64_t acc_full[2], acc_empty[2];
  uint64_t part_full, part_empty;  // the other pairs' results in the first one's shared memory
  uint32_t tmem;
  int odd;  // kAdapter, the first pair's: the last tile with an up-projection that is not finite
};

struct Tile {
  int e, first, count;  // rows of the tile (kGradW: all rows of the expert)
  int cols;             // columns of the product (multiple of 32: what a pair's product takes)
  int part;             // which of the expert's tiles of rows
  int a0, b0;           // first row of A; kGradW: first column
  int steps;
};

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Walks the tiles of a pair, 32 experts at a time (a whole warp calls it).
// Tiles are ordered by expert, then along A, then along the expert's rows, so
// pairs that run at the same time read the same weights.
template <Form F>
struct Walker {
  const Params &p;
  int lane, chunk = -1, base = 0, total = 0;
  int rows = 0, first = 0, prefix = 0, mine = 0;

  __device__ Walker(const Params &p_) : p(p_), lane(threadIdx.x & 31) {}

  // The most columns that a tile has (the whole warp calls it).
  __device__ static int most_cols(const Params &p) {
    if (grad_w(F)) return kMaxCols;
    // with so few rows the counts need not be read
    if (single(F) || p.most_rows <= 64) return most_cols_of(limits(p));
    const int n = widest_tile(limits(p), p.offset, p.rows, p.E, threadIdx.x & 31, 32);
    return max(kColumnStep, __reduce_max_sync(0xffffffffu, n));
  }

  __device__ static RowLimits limits(const Params &p) { return RowLimits{p.cap, p.most_rows, p.max_cols}; }

  __device__ void load(int c) {
    chunk = c;
    const int e = c * 32 + lane;
    rows = first = mine = 0;
    if (single(F)) {
      rows = e == 0 ? p.cap : 0;
      if (e == 0) {
        mine = !grad_w(F) ? p.a_tiles * tiles_of(limits(p), rows) : p.a_tiles * p.b_tiles;
        if (F == kDenseGradWPart) mine *= p.segments;
      }
    } else if (e < p.E) {
      first = p.offset[e];
      const int n = p.rows[e];
      rows = rows_within(limits(p), first, n);
      if (rows != n && blockIdx.x == 0 && threadIdx.x < 32) set_error(p.error_word, EP_ERRBIT_CAPACITY);
      mine = grad_w(F) ? p.a_tiles * p.b_tiles : p.a_tiles * tiles_of(limits(p), rows);
    }
    prefix = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, prefix, o);
      if (lane >= o) prefix += v;
    }
    total = __shfl_sync(0xffffffffu, prefix, 31);
  }

  // The tile with this number (numbers only grow); false past the last.
  __device__ bool find(int number, Tile &t) {
    while (chunk < 0 || number >= base + total) {
      base += total;
      if ((chunk + 1) * 32 >= p.E) {
        total = 0;
        return false;
      }
      load(chunk + 1);
    }
    const int local = number - base;
    const int src = __ffs(__ballot_sync(0xffffffffu, prefix > local)) - 1;
    const int at = local - __shfl_sync(0xffffffffu, prefix - mine, src);
    const int n = __shfl_sync(0xffffffffu, rows, src);
    t.e = chunk * 32 + src;
    t.first = __shfl_sync(0xffffffffu, first, src);
    if (grad_w(F)) {
      const int tiles = p.a_tiles * p.b_tiles, in = F == kDenseGradWPart ? at % tiles : at;
      t.a0 = in / p.b_tiles * 256;
      t.b0 = in % p.b_tiles * 256;
      t.count = n;
      if (F == kDenseGradWPart) {
        t.e = at / tiles;
        t.first = t.e * p.rows_each;
        t.count = min(p.rows_each, n - t.first);
      }
      t.cols = kMaxCols;
      t.steps = ceil_div(t.count, kInner);
    } else {
      const int tiles = tiles_of(limits(p), n);
      if (single(F)) {
        // eight tiles of rows go along A together, so the pairs running at
        // once share rows as well as weights
        const int band = at / (8 * p.a_tiles), in = at - band * 8 * p.a_tiles, high = min(8, tiles - band * 8);
        t.part = band * 8 + in % high;
        t.a0 = in / high * (gated(F) ? 128 : 256);
      } else {
        t.part = at % tiles;
        t.a0 = at / tiles * (gated(F) ? 128 : 256);
      }
      t.b0 = 0;
      int from;
      t.count = tile_rows(limits(p), n, t.part, &from);
      t.first += from;
      t.cols = ceil_div(t.count, kColumnStep) * kColumnStep;
      t.steps = ceil_div(p.inner, kInner);
    }
    return true;
  }
};

// __expf errs by up to 2 + 1.17 |g| units in the last place (its documented
// bound): 2^-16 before it overflows, where the result is rounded to 2^-9.
__device__ __forceinline__ float silu_of(float g) { return g / (1.0f + __expf(-g)); }

// Barriers of two warps; the first also gives whether both say `ok`.
__device__ __forceinline__ bool pair_agree(int id, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\t"
      "barrier.cta.red.and.pred q, %1, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"((uint32_t)ok)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ void pair_barrier(int id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); }

// A warp's 32 lanes hold outputs n (one a lane) of COUNT rows v[0..), `rows`
// of them real: out[row][n] through the staging buffer, 64 bytes of a row at
// a time; or, where rows are not of whole 16 bytes (ANY: they may not be),
// straight from the registers, 2 bytes a lane.
template <int COUNT, bool ANY = false>
__device__ __forceinline__ void store_transposed(const float *v, char *stage, uint16_t *out, int64_t pitch, int rows,
                                                 int n, int limit, int lane) {
  if (ANY && pitch % 8 != 0) {
#pragma unroll
    for (int c = 0; c < COUNT; ++c)
      if (c < rows && n + lane < limit) out[c * pitch + n + lane] = (uint16_t)(pack_bf16x2(v[c], 0.0f) & 0xffffu);
    return;
  }
  constexpr int kRows = COUNT < kStagedRows ? COUNT : kStagedRows;
  const int part = lane & 3;
#pragma unroll
  for (int r = 0; r < COUNT; r += kRows) {
    if (r >= rows) return;
#pragma unroll
    for (int c = 0; c < kRows; ++c)
      *reinterpret_cast<uint16_t *>(stage + c * kPitch + lane * 2) = (uint16_t)(pack_bf16x2(v[r + c], 0.0f) & 0xffffu);
    __syncwarp();
#pragma unroll
    for (int c = lane >> 2; c < kRows; c += 8) {
      if (r + c < rows && n + part * 8 < limit)
        *reinterpret_cast<int4 *>(out + (int64_t)(r + c) * pitch + n + part * 8) =
            *reinterpret_cast<const int4 *>(stage + c * kPitch + part * 16);
    }
    __syncwarp();
  }
}

// What the kernel ahead made, after the wait for it: kept in its place by the
// compiler, read from L2.
__device__ __forceinline__ int load_made(const int32_t *p) {
  int v;
  asm volatile("ld.global.cg.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ int4 load_made(const int4 *p) {
  int4 v;
  asm volatile("ld.global.cg.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// The halves of a word of two bf16 that are not finite: their top bits.
__device__ __forceinline__ uint32_t not_finite(uint32_t w) { return ((w & 0x7fff7fffu) + 0x00800080u) & 0x80008000u; }
__device__ __forceinline__ uint32_t not_finite(const uint4 &w) {
  return not_finite(w.x) | not_finite(w.y) | not_finite(w.z) | not_finite(w.w);
}

// kAdapter: the infinities and NaN of the up-projections, which the gathering
// warps replaced, added to 32 rows c ... of output `at` that this warp wrote
// (a sum with one of them is that one, whatever the rest was rounded to).
__device__ __forceinline__ void add_odd(const Params &p, const Tile &t, int c, int at) {
  const int32_t *plan = p.plan + (int64_t)t.part * kPlanWords;
  for (int j = c; j < c + 32 && j < t.count; ++j) {
    const int place = load_made(plan + 1 + kMaxCols + j);
    if (place < 0 || at >= p.width) continue;
    const uint16_t *up = p.up + ((int64_t)load_made(plan + 1 + place) * p.width + at) * p.rank;
    const uint16_t *low = p.low + (int64_t)(t.first + j) * p.rank;
    float more = 0.0f;
    bool some = false;
    for (int i = 0; i < p.rank; i += 8) {
      const uint4 u = __ldg(reinterpret_cast<const uint4 *>(up + i));
      if (not_finite(u) == 0u) continue;
      const int4 l = load_made(reinterpret_cast<const int4 *>(low + i));
      const uint32_t uw[4] = {u.x, u.y, u.z, u.w};
      const uint32_t lw[4] = {(uint32_t)l.x, (uint32_t)l.y, (uint32_t)l.z, (uint32_t)l.w};
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const uint32_t odd = not_finite(uw[h]);
        if (odd & 0x8000u) more += bf16_lo(uw[h]) * bf16_lo(lw[h]);
        if (odd & 0x80000000u) more += bf16_hi(uw[h]) * bf16_hi(lw[h]);
      }
      some = true;
    }
    if (some) {
      uint16_t *o = p.out + (int64_t)(t.first + j) * p.width + at;
      *o = (uint16_t)(pack_bf16x2(bf16_lo(*o) + more, 0.0f) & 0xffffu);
    }
  }
}

// ------------------------------------------------ the epilogue of kDense

constexpr float kRootTwoPi = 0.79788456080286536f;     // sqrt(2 / pi)
constexpr float kRootOneTwoPi = 0.39894228040143268f;  // 1 / sqrt(2 pi)
constexpr float kCubic = 0.044715f;

__device__ __forceinline__ float load_param(const void *p, bool bf16, int64_t i) {
  return bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t *>(p)[i] << 16) : static_cast<const float *>(p)[i];
}

// e^z by the hardware's power of two (2 ulp), whose argument is rounded: off
// by 2^-24 (4 + |z|), 2^-17 before it overflows; below 2^-126 it is 0.  With
// it and rcp_normal a sigmoid is five instructions; with a division and
// __expf, which scale what is not normal, it was some twenty, and results took
// longer than their products where the inner dimension is short (8192 rows
// 512 -> 2 x 512, SwiGLU: 13.8 us, before 20.5; 1024 rows 2048 -> 2048, SiLU:
// 11.4, before 14.2).
__device__ __forceinline__ float exp2_quick(float z) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(z));
  return r;
}
__device__ __forceinline__ float exp_quick(float z) { return exp2_quick(z * 1.4426950408889634f); }

__device__ __forceinline__ float sigmoid_of(float z) { return rcp_normal(1.0f + exp_quick(-z)); }

// The normal distribution's integral up to z, and e^(-z^2 / 2).  At z <= 0 it is
// the tail, which is that power times a function that falls slowly: t P(t) with
// t = 1 / (1 + c |z|), a polynomial fitted here (least squares, weighted until
// the largest relative error is least) to 10^-7 of the value for |z| <= 13.4,
// where the power leaves fp32's normal numbers.  So the tail is right relative
// to itself: with roundings and the power, whose argument has two, to
// 2^-24 (24 + 2 z^2).
__device__ __forceinline__ float normal_integral(float z, float &density) {
  const float t = rcp_normal(fmaf(0.3028125f, fabsf(z), 1.0f));
  float poly = fmaf(0.0366312386f, t, -0.1563754371f);
  poly = fmaf(poly, t, 0.1971785558f);
  poly = fmaf(poly, t, -0.0469131846f);
  poly = fmaf(poly, t, 0.1253758886f);
  poly = fmaf(poly, t, 0.1015798380f);
  poly = fmaf(poly, t, 0.1217660435f);
  poly = fmaf(poly, t, 0.1207570326f);
  density = exp2_quick(z * z * -0.72134752044448170f);  // log2(e) / 2
  const float tail = poly * t * density;
  return z < 0.0f ? tail : 1.0f - tail;
}

// tanh(u) = 2 sigmoid(2 u) - 1
__device__ __forceinline__ float tanh_gate(float z) { return sigmoid_of(2.0f * kRootTwoPi * (z + kCubic * z * z * z)); }

__device__ __forceinline__ void activate(int act, float (&v)[32]) {
  if (act == EP_ACT_RELU) {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = v[j] < 0.0f ? 0.0f : v[j];
  } else if (act == EP_ACT_SILU) {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] *= sigmoid_of(v[j]);
  } else if (act == EP_ACT_GELU) {
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      float density;
      v[j] *= normal_integral(v[j], density);
    }
  } else if (act == EP_ACT_GELU_TANH) {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] *= tanh_gate(v[j]);
  }
}

// The residual of COUNT rows of 32 outputs from `at` on, 16 bytes a lane and
// row: four lanes a row.
template <int COUNT>
__device__ __forceinline__ void load_residual(int4 (&r)[4], const Params &p, int64_t row, int rows, int at, int lane) {
  const int n = at + (lane & 3) * 8;
  if (p.width % 8 != 0) return;
#pragma unroll
  for (int i = 0; i < COUNT / 8; ++i) {
    const int c = (lane >> 2) + i * 8;
    if (c < rows && n < p.width) r[i] = *reinterpret_cast<const int4 *>(p.residual + (row + c) * p.width + n);
  }
}

// ... added to a row's value a lane and output, through the staging buffer
// (or, where rows are not of whole 16 bytes, read here).
template <int COUNT>
__device__ __forceinline__ void add_residual(float *v, const int4 (&r)[4], char *stage, const Params &p, int64_t row, int rows,
                                             int at, int lane) {
  if (p.width % 8 != 0) {
#pragma unroll
    for (int c = 0; c < COUNT; ++c)
      if (c < rows && at + lane < p.width) v[c] += __uint_as_float((uint32_t)p.residual[(row + c) * p.width + at + lane] << 16);
    return;
  }
#pragma unroll
  for (int h = 0; h < COUNT / 16; ++h) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      *reinterpret_cast<int4 *>(stage + ((lane >> 2) + i * 8) * kPitch + (lane & 3) * 16) = r[2 * h + i];
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 16; ++c)
      v[h * 16 + c] += __uint_as_float((uint32_t) * reinterpret_cast<const uint16_t *>(stage + c * kPitch + lane * 2) << 16);
    __syncwarp();
  }
}

template <Form F, int COUNT>
__device__ __forceinline__ void store_out(const float *v, char *stage, const Params &p, int64_t row, int rows, int at,
                                          int lane) {
  if (!runs(F)) {
    store_transposed<COUNT, true>(v, stage, p.out + row * p.width, p.width, rows, at, p.width, lane);
    return;
  }
  float *out = reinterpret_cast<float *>(p.out) + row * p.width;
  if (p.width % 4 != 0) {
#pragma unroll
    for (int c = 0; c < COUNT; ++c)
      if (c < rows && at + lane < p.width) out[(int64_t)c * p.width + at + lane] = v[c];
    return;
  }
  constexpr int kRows = 8, kWide = 144;  // of 128 bytes; 16 against bank conflicts
  static_assert(kRows * kWide <= kStagedRows * kPitch, "");
  const int n = at + (lane & 7) * 4;
#pragma unroll
  for (int r = 0; r < COUNT; r += kRows) {
    if (r >= rows) return;
#pragma unroll
    for (int c = 0; c < kRows; ++c) *reinterpret_cast<float *>(stage + c * kWide + lane * 4) = v[r + c];
    __syncwarp();
#pragma unroll
    for (int c = lane >> 3; c < kRows; c += 4) {
      if (r + c < rows && n < p.width)
        *reinterpret_cast<float4 *>(out + (int64_t)(r + c) * p.width + n) =
            *reinterpret_cast<const float4 *>(stage + c * kWide + (lane & 7) * 16);
    }
    __syncwarp();
  }
}

template <Form F>
__global__ void __launch_bounds__(threads_of(F), 1) product_kernel(const __grid_constant__ Params p) {
  extern __shared__ char s_raw[];
  __shared__ Barriers s_bar;
  char *ring = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(s_raw) + 1023) & ~uintptr_t(1023));
  char *staging = ring + p.ring_bytes / 1024 * 1024;
  char *exchange = staging + kResultWarps * staging_of(F);
  // [parts - 1][columns / 4][128][4]: the other pairs' results
  float4 *joined = reinterpret_cast<float4 *>(exchange + (gated(F) ? kResultWarps * kExchangeBytes : 0));
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  // A cluster is one pair, or the pairs that share a tile (`part`: which of them).
  const uint32_t rank = cluster_rank() & 1u, lead = cluster_rank() & ~1u, both = 3u << lead;
  const int part = (int)(cluster_rank() >> 1);
  const int pair = blockIdx.x / (2 * p.parts), pairs = gridDim.x / (2 * p.parts);
  const auto first_step = [&](const Tile &t) { return t.steps * part / p.parts; };
  const auto last_step = [&](const Tile &t) { return t.steps * (part + 1) / p.parts; };

  if (threadIdx.x == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(&s_bar.full[i], 1);
      mbar_init(&s_bar.empty[i], 1);
      mbar_init(&s_bar.ends[i], 1);
      mbar_init(&s_bar.fixed[i], 2);  // one arrival from each CTA
    }
    for (int i = 0; i < kSideStages; ++i) {
      mbar_init(&s_bar.side_full[i], 2 * kGatherWarps);
      mbar_init(&s_bar.side_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_bar.acc_full[i], 1);
      mbar_init(&s_bar.acc_empty[i], 2 * kResultWarps);
    }
    mbar_init(&s_bar.part_full, kResultWarps * (p.parts > 1 ? p.parts - 1 : 1));
    mbar_init(&s_bar.part_empty, kResultWarps);
    s_bar.odd = -1;
    fence_barrier_init();
    prefetch_map(&p.a);
  }
  __syncwarp();
  if (warp == 2) tmem_alloc_pair(&s_bar.tmem, kTmemCols);
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = s_bar.tmem;
  // kAdapter: only the low rows and the plan come from the kernel ahead, which
  // started after all that was before it had ended; who reads them waits.
  if (F != kAdapter || warp == 2) {
    griddep_wait();
    griddep_launch_dependents();
  }

  // A stage holds 128 rows of A and half of the most columns that a tile of
  // this call has (every CTA finds the same): the fewer, the deeper the ring,
  // which has to cover the latency of memory (gated product of 384 rows an
  // expert: 499, 442, 385 us with 3, 4, 5 stages).  kAdapter: a second ring
  // for the adapters' steps, so that the first waits for nothing.
  const int b_bytes = Walker<F>::most_cols(p) / 2 * 128, stage_bytes = kABytes + b_bytes;
  int stages = p.ring_bytes / 1024 * 1024 / stage_bytes;
  // (a stage less in the first costs 10% with six in all, so one is enough
  // for the second then: long runs of rows need a step or two a tile.  A tile
  // that pairs share is their only one, and its adapters' steps come last:
  // two, 1021 rows of 40 adapters 21.3 us against 22.3)
  const int side_stages = stages >= 8 ? kSideStages : p.parts > 1 ? 2 : 1;
  if (F == kAdapter) stages -= side_stages;
  stages = min(stages, kMaxStages);
  char *side = ring + stages * stage_bytes;

  bool ok = true;  // false: a wait gave up
  if (warp == 0 || warp == 3) {
    // ------------------------------------------------------------ copies
    const bool is_a = warp == 0;
    Walker<F> walk(p);
    Tile t;
    int stage = 0;
    uint32_t phase = 0;
    for (int n = pair; ok && walk.find(n, t); n += pairs) {
      const int b_rows = t.cols / 2;
      const uint32_t bytes = kABytes + b_rows * 128;
      const int a0 = t.a0 + (int)rank * (gated(F) ? 64 : 128);
      const int b0 = (grad_w(F) ? t.b0 : t.first) + (int)rank * b_rows;
      const int k1 = last_step(t);
      for (int k = first_step(t); k < k1; ++k) {
        if (!__all_sync(0xffffffffu, mbar_wait_pair(&s_bar.empty[stage], phase ^ 1))) {
          ok = false;
          break;
        }
        if (elect_one()) {
          const uint32_t a = smem_addr(ring + (size_t)stage * stage_bytes), b = a + kABytes;
          // both CTAs' copies complete on the leading CTA's barrier, but those
          // of a last step whose rows end raggedly go by the row ends
          const bool last = grad_w(F) && t.count % 16 != 0 && k == t.steps - 1;
          const uint32_t bar = last ? map_shared(smem_addr(&s_bar.ends[stage]), lead | rank)
                                    : map_shared(smem_addr(&s_bar.full[stage]), lead);
          if (is_a) {
            if (last) mbar_arrive_expect_tx(&s_bar.ends[stage], bytes);
            if (rank == 0) {
              if (last)
                mbar_arrive(&s_bar.full[stage]);
              else
                mbar_arrive_expect_tx(&s_bar.full[stage], 2 * bytes);
            }
          }
          const int at = k * kInner;
          if (is_a) {
            if (F == kPlain || F == kAdapter || (dense(F) && !gated(F))) {
              tile_load_3d(a, &p.a, at, a0, t.e, bar);
            } else if (gated(F)) {
              tile_load_4d(a, &p.a, at, a0, 0, t.e, bar);
            } else if (grad_x(F)) {
              if (p.a_blocks) {
                tile_load_4d(a, &p.a, 0, at, a0 / 64, t.e, bar);
              } else {
                tile_load_3d(a, &p.a, a0, at, t.e, bar);
                tile_load_3d(a + 8192, &p.a, a0 + 64, at, t.e, bar);
              }
            } else if (p.a_blocks) {
              tile_load_3d(a, &p.a, 0, t.first + at, a0 / 64, bar);
            } else {
              tile_load_2d(a, &p.a, a0, t.first + at, bar);
              tile_load_2d(a + 8192, &p.a, a0 + 64, t.first + at, bar);
            }
          } else if (!grad_w(F)) {
            tile_load_2d(b, &p.b[b_rows / 16 - 1], at, b0, bar);
          } else if (p.b_blocks) {
            tile_load_3d(b, &p.b[0], 0, t.first + at, b0 / 64, bar);
          } else {
            tile_load_2d(b, &p.b[0], b0, t.first + at, bar);
            tile_load_2d(b + 8192, &p.b[0], b0 + 64, t.first + at, bar);
          }
        }
        __syncwarp();
        if (++stage == stages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    // the products' last arrivals on this CTA's barriers come before it ends
    for (int i = 0; ok && i < stages; ++i) {
      ok = __all_sync(0xffffffffu, mbar_wait_pair(&s_bar.empty[stage], phase ^ 1));
      if (++stage == stages) {
        stage = 0;
        phase ^= 1;
      }
    }
  } else if (warp == 1 && rank == 0) {
    // ---------------------------------------------------------- products
    Walker<F> walk(p);
    Tile t;
    int stage = 0, acc = 0;
    uint32_t phase = 0, acc_phase = 0, trims = 0;
    int side_stage = 0;
    uint32_t side_phase = 0;
    const uint32_t ring_addr = smem_addr(ring);
    for (int n = pair; ok && walk.find(n, t); n += pairs) {
      if (t.steps == 0) continue;  // an expert without rows (kGradW): zeros are written
      const uint32_t idesc = mma_desc(t.cols, grad_x(F) || grad_w(F), grad_w(F));
      const int end = last_step(t);
      for (int k0 = first_step(t), k1; ok && k0 < end; k0 = k1) {  // one run, or runs of kRun
        k1 = runs(F) ? min(end, k0 + kRun) : end;
        const uint32_t d = tmem + acc * kMaxCols;
        ok = __all_sync(0xffffffffu, mbar_wait_pair(&s_bar.acc_empty[acc], acc_phase ^ 1));
        tc_fence_after();
        for (int k = k0; ok && k < k1; ++k) {
          ok = __all_sync(0xffffffffu, mbar_wait_pair(&s_bar.full[stage], phase));
          if (grad_w(F) && ok && k == t.steps - 1 && t.count % 16 != 0) {
            ok = __all_sync(0xffffffffu, mbar_wait_pair(&s_bar.fixed[stage], (trims >> stage) & 1u));
            trims ^= 1u << stage;
          }
          if (!ok) break;
          tc_fence_after();
          const uint32_t addr = ring_addr + (uint32_t)(stage * stage_bytes);
          const uint32_t a = grad_x(F) || grad_w(F) ? outer_desc(addr, 8192) : inner_desc(addr);
          const uint32_t b = grad_w(F) ? outer_desc(addr + kABytes, 8192) : inner_desc(addr + kABytes);
          const int parts = grad_w(F) ? min(4, ceil_div(t.count - k * kInner, 16)) : 4;
          if (elect_one()) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (j < parts)
                mma_pair(d, a + j * ((grad_x(F) || grad_w(F) ? 2048 : 32) >> 4), b + j * ((grad_w(F) ? 2048 : 32) >> 4),
                         idesc, k > k0 || j > 0);
            commit_pair(&s_bar.empty[stage], both);
            if (F != kAdapter && k == k1 - 1) commit_pair(&s_bar.acc_full[acc], both);
          }
          __syncwarp();
          if (++stage == stages) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (F == kAdapter && ok) {
          if (n == pair) griddep_wait();
          const int length = p.rank * load_made(p.plan + (int64_t)t.part * kPlanWords);  // of the adapters side by side
          for (int k = part; ok && k * kInner < length; k += p.parts) {
            ok = __all_sync(0xffffffffu, mbar_wait_pair(&s_bar.side_full[side_stage], side_phase));
            if (!ok) break;
            tc_fence_after();
            const uint32_t addr = smem_addr(side) + (uint32_t)(side_stage * stage_bytes);
            const uint32_t a = inner_desc(addr), b = inner_desc(addr + kABytes);
            const int parts = min(4, ceil_div(length - k * kInner, 16));
            if (elect_one()) {
              for (int j = 0; j < parts; ++j) mma_pair(d, a + j * 2, b + j * 2, idesc, true);
              commit_pair(&s_bar.side_empty[side_stage], both);
            }
            __syncwarp();
            if (++side_stage == side_stages) {
              side_stage = 0;
              side_phase ^= 1;
            }
          }
          if (ok && elect_one()) commit_pair(&s_bar.acc_full[acc], both);
          __syncwarp();
        }
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1;
      }
    }
  } else if (warp == 2 && grad_w(F)) {
    // ---------------------------------------------------------- row ends
    // The last step of an expert reads rows of the next one: they are zeroed
    // in both operands (both, since what lies there may be NaN).
    Walker<F> walk(p);
    Tile t;
    int stage = 0;
    uint32_t parities = 0;
    for (int n = pair; ok && walk.find(n, t); n += pairs) {
      stage = (stage + t.steps) % stages;
      if (t.count % 16 == 0) continue;
      const int s = (stage + stages - 1) % stages;
      ok = mbar_wait_pair(&s_bar.ends[s], (parities >> s) & 1u);
      if (!ok) break;
      parities ^= 1u << s;
      // four blocks of 64 outer elements (A's two and B's), 128 bytes of each
      // a row: one store of the warp
      char *row = ring + (size_t)s * stage_bytes + (lane >> 3) * 8192 + (lane & 7) * 16;
      const int from = t.count % kInner, to = ceil_div(from, 16) * 16;
      for (int r = from; r < to; ++r) *reinterpret_cast<int4 *>(row + r * 128) = make_int4(0, 0, 0, 0);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_local(map_shared(smem_addr(&s_bar.fixed[s]), lead));
    }
  } else if (F == kAdapter && warp >= 12) {
    // ---------------------------------------------------------- adapters
    // Both operands of a further step are gathered 16 bytes at a time, in the
    // swizzled order that a tile's copy would give them: eight lanes take the
    // eight pieces of a row, so a lane stays with one adapter in a step.  An
    // up-projection meets every row of the tile, and in other adapters' rows
    // zeros, which would make NaN of what is not finite: 2^-64 of its sign
    // takes its place here, the tile is noted, and the results' warps add it
    // to its own rows.  (Not zero: an infinite low value would make NaN of
    // that; times 2^-64 it is the infinity that the product is, and a finite
    // one is too little to be seen beside an infinity.)
    griddep_wait();
    Walker<F> walk(p);
    Tile t;
    const int rows = (warp - 12) * 32;  // this warp's of A, and of B
    int stage = 0, hand = 0;  // hand: the stage handed over next
    uint32_t phase = 0;
    int flying = 0;
    const int piece = lane & 7;
    const auto hand_over = [&](int n, int left) {  // left: of the inner dimension from this step on
      if (piece * 8 < left) {
        char *a = side + (size_t)hand * stage_bytes;
        const auto at = [&](int j) {
          const int r = rows + j * 4 + (lane >> 3);
          return reinterpret_cast<uint4 *>(a + r * 128 + ((piece ^ (r & 7)) << 4));
        };
        uint32_t odd = 0u;
#pragma unroll
        for (int j = 0; j < 8; ++j) odd |= not_finite(*at(j));
        if (odd != 0u) {
          for (int j = 0; j < 8; ++j) {
            uint32_t *w = reinterpret_cast<uint32_t *>(at(j));
            for (int i = 0; i < 4; ++i) {
              const uint32_t which = (not_finite(w[i]) >> 15) * 0xffffu;
              w[i] = (w[i] & ~(which & 0x7fff7fffu)) | (which & 0x1f801f80u);
            }
          }
          atom_max_cluster(map_shared(smem_addr(&s_bar.odd), rank), n);  // where the results are finished
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_local(map_shared(smem_addr(&s_bar.side_full[hand]), lead));
      if (++hand == side_stages) hand = 0;
      --flying;
    };
    for (int n = pair; ok && walk.find(n, t); n += pairs) {
      const int32_t *plan = p.plan + (int64_t)t.part * kPlanWords;
      const int count = load_made(plan), length = count * p.rank, b_rows = t.cols / 2;
      const int place = rows + lane < b_rows ? load_made(plan + 1 + kMaxCols + (int)rank * b_rows + rows + lane) : -1;
      const int a0 = t.a0 + (int)rank * 128;
      const uint16_t *low = p.low + (int64_t)(t.first + (int)rank * b_rows) * p.rank;
      // the adapter of this lane's columns, read a step ahead
      const auto adapter_of = [&](int k) {
        const int col = k * kInner + piece * 8;
        return col < length ? load_made(plan + 1 + col / p.rank) : 0;
      };
      int last = part, next = adapter_of(part);
      for (int k = part; k * kInner < length; k += p.parts) {
        const int adapter = next;
        next = adapter_of(k + p.parts);
        ok = __all_sync(0xffffffffu, mbar_wait_pair(&s_bar.side_empty[stage], phase ^ 1));
        if (!ok) break;
        const uint32_t a = smem_addr(side + (size_t)stage * stage_bytes), b = a + kABytes;
        const int col = k * kInner + piece * 8, mine = col / p.rank, in = col - mine * p.rank;
        const bool there = col < length;
        if (piece * 8 < ceil_div(min(length - k * kInner, kInner), 16) * 16) {
          const uint16_t *up = p.up + ((int64_t)adapter * p.width + a0) * p.rank + in;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int r = rows + j * 4 + (lane >> 3);
            const bool some = there && a0 + r < p.width;
            copy16(a + r * 128 + ((piece ^ (r & 7)) << 4), some ? up + (int64_t)r * p.rank : p.up, some);
          }
        }
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int r = rows + j * 4 + (lane >> 3);
          const bool some = __shfl_sync(0xffffffffu, place, j * 4 + (lane >> 3)) == mine && there;
          if (r < b_rows)
            copy16(b + r * 128 + ((piece ^ (r & 7)) << 4), some ? low + (int64_t)r * p.rank + in : p.low, some);
        }
        copy_commit();
        ++flying;
        if (side_stages == 1) {
          copy_wait<0>();
          hand_over(n, length - k * kInner);
        } else if (flying == 2) {
          copy_wait<1>();
          hand_over(n, length - (k - p.parts) * kInner);
        }
        last = k;
        if (++stage == side_stages) {
          stage = 0;
          phase ^= 1;
        }
      }
      if (flying > 0) {
        copy_wait<0>();
        hand_over(n, length - last * kInner);
      }
    }
    for (int i = 0; ok && i < side_stages; ++i) {
      ok = __all_sync(0xffffffffu, mbar_wait_pair(&s_bar.side_empty[stage], phase ^ 1));
      if (++stage == side_stages) {
        stage = 0;
        phase ^= 1;
      }
    }
  } else if (warp >= 4) {
    // ----------------------------------------------------------- results
    // Warp w reads the tensor-memory lanes 32 (w % 4) ...; the two groups of
    // four warps take every other 32 columns.
    Walker<F> walk(p);
    Tile t;
    const int w = warp - 4, quarter = w & 3, half = w >> 2;
    char *stage_buf = staging + w * staging_of(F);
    int acc = 0;
    uint32_t acc_phase = 0, part_phase = 0;
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const auto store_block = [&](char *from, const Tile &t, int c) {  // kGradW: 32 rows of 64 columns
      const int col = t.b0 + c, row = t.a0 + (int)rank * 128 + quarter * 32;
      if (col < p.hidden && row < p.wide)
        tile_store_3d(&p.grad, smem_addr(from), F == kDenseGradWPart ? 2 * col : col, row, t.e);
      bulk_commit();
    };
    const auto release = [&](int a) {  // this warp has read its columns of accumulator a
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_relaxed(map_shared(smem_addr(&s_bar.acc_empty[a]), lead));
    };
    for (int n = pair; ok && walk.find(n, t); n += pairs) {
      if (grad_w(F) && t.steps == 0) {  // an expert without rows
        if (lane == 0) bulk_wait_read<0>();
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j)
          *reinterpret_cast<int4 *>(stage_buf + (j * 32 + lane) * 16) = make_int4(0, 0, 0, 0);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0)
          for (int c = half * 64; c < t.cols; c += 128)
            store_block(stage_buf, t, c);
        continue;
      }
      float bias = 0.0f;
      int4 ahead[4];  // kDense: the residual of the next 32 rows
      if (dense(F) && part == 0) {
        const int at = gated(F) ? t.a0 + (int)rank * 64 + (quarter & 1) * 32 : t.a0 + (int)rank * 128 + quarter * 32;
        if (p.bias != nullptr && at + lane < p.width)
          bias = load_param(p.bias, p.bias_bf16, (gated(F) && quarter >= 2 ? p.width : 0) + at + lane);
        if (!gated(F) && p.residual != nullptr) load_residual<32>(ahead, p, t.first + half * 32, t.count - half * 32, at, lane);
      }
      constexpr int kHeld = runs(F) ? most_cols_of_form(F) / 64 : 1;
      float held[kHeld][32];  // kDense32: this warp's sums of the runs so far
      if (runs(F)) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
#pragma unroll
          for (int j = 0; j < 32; ++j) held[i][j] = 0.0f;
        const int end = last_step(t);
        for (int k = first_step(t); ok && k < end; k += kRun) {
          ok = __all_sync(0xffffffffu, mbar_wait_pair(&s_bar.acc_full[acc], acc_phase));
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int i = 0; i < kHeld; ++i) {
            const int c = half * 32 + i * 64;
            if (c >= t.cols) break;
            float v[32];
            tmem_load32(tmem + acc * kMaxCols + c + lane_base, v);
#pragma unroll
            for (int j = 0; j < 32; ++j) held[i][j] += v[j];
          }
          release(acc);
          acc ^= 1;
          if (acc == 0) acc_phase ^= 1;
        }
      } else {
        ok = mbar_wait_pair(&s_bar.acc_full[acc], acc_phase);
      }
      if (!grad_w(F) && p.parts > 1) {
        if (part > 0) {
          // this pair's sums go to the first pair's CTA with the same rows
          ok = ok && mbar_wait_cluster(&s_bar.part_empty, part_phase ^ 1);
          if (!__all_sync(0xffffffffu, ok)) break;
          tc_fence_after();
          const uint32_t to = map_shared(smem_addr(joined + (part - 1) * p.max_cols * 32 + quarter * 32 + lane), rank);
#pragma unroll(runs(F) ? kHeld : 1)
          for (int i = 0; i < (runs(F) ? kHeld : kMaxCols / 64); ++i) {
            const int c = half * 32 + i * 64;
            if (c >= t.cols) break;
            float v[32];
            if (runs(F)) {
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] = held[i % kHeld][j];
            } else {
              tmem_load32(tmem + acc * kMaxCols + c + lane_base, v);
            }
#pragma unroll
            for (int j = 0; j < 32; j += 4)
              store_cluster(to + (uint32_t)(c + j) * 512, make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]));
          }
          if (!runs(F)) release(acc);
          __syncwarp();
          fence_cluster();  // every lane's stores, before one arrives for all
          if (lane == 0) mbar_arrive_cluster_relaxed(map_shared(smem_addr(&s_bar.part_full), rank));
          part_phase ^= 1;
          if (runs(F)) continue;
          acc ^= 1;
          if (acc == 0) acc_phase ^= 1;
          continue;
        }
        ok = ok && mbar_wait_cluster(&s_bar.part_full, part_phase);
      }
      ok = gated(F) ? pair_agree(1 + half * 2 + (quarter & 1), ok) : __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      if (F == kDenseGradWPart) {
        // as below, 32 columns of fp32 at a time
        for (int c = half * 32; c < t.cols; c += 64) {
          float v[32];
          tmem_load32(tmem + acc * kMaxCols + c + lane_base, v);
          if (c + 64 >= t.cols) release(acc);
          if (lane == 0) bulk_wait_read<0>();
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<float4 *>(stage_buf + lane * 128 + ((j ^ (lane & 7)) << 4)) =
                make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) store_block(stage_buf, t, c);
        }
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1;
        continue;
      }
      if (grad_w(F)) {
        // a row of the gradient a lane; 64 columns are staged in the swizzled
        // order and stored as a tile
        for (int c = half * 64; c < t.cols; c += 128) {
          float v[64];
          tmem_load32(tmem + acc * kMaxCols + c + lane_base, reinterpret_cast<float (&)[32]>(v[0]));
          tmem_load32(tmem + acc * kMaxCols + c + 32 + lane_base, reinterpret_cast<float (&)[32]>(v[32]));
          if (c + 128 >= t.cols) release(acc);
          if (lane == 0) bulk_wait_read<0>();
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<uint4 *>(stage_buf + lane * 128 + ((j ^ (lane & 7)) << 4)) =
                make_uint4(pack_bf16x2(v[8 * j], v[8 * j + 1]), pack_bf16x2(v[8 * j + 2], v[8 * j + 3]),
                           pack_bf16x2(v[8 * j + 4], v[8 * j + 5]), pack_bf16x2(v[8 * j + 6], v[8 * j + 7]));
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) store_block(stage_buf, t, c);
        }
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1;
        continue;
      }
#pragma unroll(runs(F) ? kHeld : 1)
      for (int i = 0; i < (runs(F) ? kHeld : kMaxCols / 64); ++i) {
        const int c = half * 32 + i * 64;
        if (c >= t.cols) break;
        float v[32];
        if (runs(F)) {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = held[i % kHeld][j];
        } else {
          tmem_load32(tmem + acc * kMaxCols + c + lane_base, v);
          if (c + 64 >= t.cols) release(acc);
        }
        if (!grad_w(F) && p.parts > 1) {
          // the parts are added in their order
          for (int q = 0; q + 1 < p.parts; ++q) {
            const float4 *more = joined + (q * p.max_cols + c) * 32 + quarter * 32 + lane;
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              const float4 m = more[j * 32];
              v[j] += m.x;
              v[j + 1] += m.y;
              v[j + 2] += m.z;
              v[j + 3] += m.w;
            }
          }
        }
        const int left = t.count - c;  // rows of this chunk (not kGradW)
        if (dense(F) && !gated(F)) {
          const int at = t.a0 + (int)rank * 128 + quarter * 32;
          const int64_t row = t.first + c;
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] += bias;
          if (p.preact != nullptr)
            store_transposed<32, true>(v, stage_buf, p.preact + row * p.width, p.width, left, at, p.width, lane);
          activate(p.activation, v);
          if (p.residual != nullptr) {
            add_residual<32>(v, ahead, stage_buf, p, row, left, at, lane);
            load_residual<32>(ahead, p, row + 64, left - 64, at, lane);
          }
          store_out<F, 32>(v, stage_buf, p, row, left, at, lane);
        } else if (F == kPlain || grad_x(F) || F == kAdapter) {
          const int at = t.a0 + (int)rank * 128 + quarter * 32;
          const int64_t row = t.first + c;
          store_transposed<32>(v, stage_buf, p.out + row * p.width, p.width, left, at, p.width, lane);
          if (F == kPlain && p.preact != nullptr)
            store_transposed<32>(v, stage_buf, p.preact + row * p.width, p.width, left, at, p.width, lane);
        } else if (gated(F)) {
          // lanes 0-63 hold the gate, lanes 64-127 what it multiplies: warps
          // w and w + 2 exchange half of their columns and finish half each
          const int at = t.a0 + (int)rank * 64 + (quarter & 1) * 32;
          const int64_t row = t.first + c;
          const bool gate = quarter < 2;
          if (dense(F)) {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] += bias;
          }
          if (p.preact != nullptr) {
            // (a half may start off 16 bytes where a row does not)
            uint16_t *to = p.preact + row * p.wide + (gate ? 0 : p.width);
            if (dense(F) && p.width % 8 != 0) {
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (j < left && at + lane < p.width)
                  to[(int64_t)j * p.wide + at + lane] = (uint16_t)(pack_bf16x2(v[j], 0.0f) & 0xffffu);
            } else {
              store_transposed<32>(v, stage_buf, to, p.wide, left, at, p.width, lane);
            }
          }
          float *give = reinterpret_cast<float *>(exchange + w * kExchangeBytes);
          const float *take = reinterpret_cast<const float *>(exchange + (w ^ 2) * kExchangeBytes);
          const int id = 1 + half * 2 + (quarter & 1);
          const int skip = gate ? 0 : 16;  // the rows that this warp finishes
          if (dense(F) && p.residual != nullptr) load_residual<16>(ahead, p, row + skip, left - skip, at, lane);
          float o[16];
#pragma unroll
          for (int r = 0; r < 16; r += 8) {
#pragma unroll
            for (int j = 0; j < 8; ++j) give[j * 32 + lane] = gate ? v[16 + r + j] : v[r + j];
            pair_barrier(id);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float other = take[j * 32 + lane];
              const float z = gate ? v[r + j] : other, u = gate ? other : v[16 + r + j];
              o[r + j] = (dense(F) ? z * sigmoid_of(z) : silu_of(z)) * u;
            }
            pair_barrier(id);  // before the next columns overwrite what the other warp reads
          }
          if (dense(F)) {
            if (p.residual != nullptr) add_residual<16>(o, ahead, stage_buf, p, row + skip, left - skip, at, lane);
            store_out<F, 16>(o, stage_buf, p, row + skip, left - skip, at, lane);
          } else {
            store_transposed<16>(o, stage_buf, p.out + (row + skip) * p.width, p.width, left - skip, at, p.width, lane);
          }
        }
      }
      if (!runs(F) && t.cols <= half * 32) release(acc);  // no columns for this warp
      if (F == kAdapter && *static_cast<volatile int *>(&s_bar.odd) >= n) {
        __syncwarp();  // what other lanes wrote
        for (int c = half * 32; c < t.cols; c += 64) add_odd(p, t, c, t.a0 + (int)rank * 128 + quarter * 32 + lane);
      }
      if (!grad_w(F) && p.parts > 1) {
        __syncwarp();
        if (lane == 0)
          for (int q = 1; q < p.parts; ++q)
            mbar_arrive_cluster_relaxed(map_shared(smem_addr(&s_bar.part_empty), 2 * q + rank));
        part_phase ^= 1;
      }
      if (runs(F)) continue;
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1;
    }
  }
  if (grad_w(F) && warp >= 4 && lane == 0) bulk_wait<0>();
  if (!ok) {
    // A wait gave up (it never should): what this CTA started lands well
    // within the time waited here, then everything is given back.
    set_error(p.error_word, EP_ERRBIT_TIMEOUT);
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 2000000ull) __nanosleep(1000);
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  if (warp == 2) {
    tc_fence_after();
    tmem_free_pair(tmem, kTmemCols);
  }
}

// Dynamic shared memory of the kernel: all that a block may have.
int shared_limit(const DeviceInfo *di) { return (int)di->max_smem_per_block_optin - (int)sizeof(Barriers) - 1024; }

// Clusters of `parts` pairs that fit the device at once.
template <Form F>
ep_status_t most_clusters(const DeviceInfo *di, int parts, int *clusters) {
  const size_t smem = shared_limit(di);
  static std::atomic<int> known[64][kMaxParts + 1];  // per device; the same for every call
  if (known[di->device][parts] == 0) {
    cudaError_t e = cudaFuncSetAttribute(product_kernel<F>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(di->num_sms / (2 * parts) * (2 * parts));
    cfg.blockDim = dim3(threads_of(F));
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2 * parts;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, product_kernel<F>, &cfg);
    if (e != cudaSuccess) return cuda_fail(e, "cudaOccupancyMaxActiveClusters");
    known[di->device][parts] = n > 0 ? n : 1;
  }
  *clusters = known[di->device][parts];
  return EP_OK;
}

constexpr uint64_t kSize = 2;  // bytes of an element

int up(int a, int b) { return a / b + (a % b != 0); }

// Pairs that may share a tile of so many columns: their sums wait in the
// first pair's shared memory, beside its ring.
int parts_for(int cols) { return cols <= 64 ? kMaxParts : cols <= 128 ? 2 : 1; }

// How a call is cut: the most columns of a tile, the pairs that share its
// inner dimension.
struct Cut {
  int cols, parts;
};

// Tiles of rows, at most: an expert with n rows has n / cols rounded up.
int64_t most_tiles(int rows, int experts, int cols) { return (rows - 1) / cols + (rows < experts ? rows : experts); }

// The cheapest of a few cuts by its cycles: a step costs its products (two
// cycles a column) or its copies (58 bytes a cycle of A's half and B's half), a
// tile its results, a shared tile its joining.  Few tiles leave SMs idle, so
// they are narrower, or shared by up to four pairs where there is a pair for
// each even if every expert wastes most of a tile.  The rows of an expert are
// known on the device only; what is reckoned with is their mean and twice its
// root more.  Gated products: 1024 tokens top-2 of 4 experts 4096 -> 2 x 512
// tiles of 256 29.2 us, cut here 20.2; 1021 rows of one expert 4096 -> 2 x 1000
// 34.7, 20.5.  `most`: rows of an expert, at most.
template <Form F>
ep_status_t choose(const DeviceInfo *di, int rows, int experts, int most, int a_tiles, int inner, Cut *best) {
  const int steps = up(inner, kInner);
  const int used = rows < experts ? rows : experts, mean = up(rows, used);
  const int64_t likely = experts == 1 ? most : mean + (int64_t)(2.0f * sqrtf((float)mean));
  int64_t least = -1;
  for (int cut = most_cols_of_form(F); cut >= 32; cut -= 32) {
    // the rows of a single expert go to tiles of about equal size
    const int need = experts == 1 ? up(most, up(most, cut)) : most < cut ? most : cut;
    const int cols = up(need, 32) * 32;
    const int64_t tiles = most_tiles(rows, experts, cols) * a_tiles;
    for (int parts = 1; parts <= parts_for(cols); ++parts) {
      int clusters = 0;
      const ep_status_t s = most_clusters<F>(di, parts, &clusters);
      if (s != EP_OK) return s;
      if (parts > 1 && (tiles > clusters || steps < 2 * parts)) break;
      const int64_t copies = (kABytes + cols / 2 * 128) / 58, products = 2 * cols;
      const int64_t count = used * ((likely + cols - 1) / cols) * a_tiles, waves = (count + clusters - 1) / clusters;
      if (experts > 1 && waves > 1 && cut < most_cols_of_form(F)) continue;  // too uncertain to leave the widest for
      const int64_t cost =
          waves * (up(steps, parts) * (copies > products ? copies : products) + 2000 + 10 * cols) +
          (parts > 1 ? 1000 + parts * 10 * cols : 0);
      if (least < 0 || cost < least) {
        least = cost;
        *best = Cut{cols, parts};
      }
    }
  }
  return EP_OK;
}

// With p.max_cols, p.parts and p.most_rows set.
template <Form F>
ep_status_t launch_form(Params &p, int64_t tiles, cudaStream_t stream) {
  const DeviceInfo *di = current_device_info();
  if (di == nullptr) return EP_ERR_CUDA;
  const int cols = p.max_cols;
  // The ring takes what is left of shared memory.
  const int limit = shared_limit(di);
  const int fixed = 1024 + kResultWarps * staging_of(F) + (gated(F) ? kResultWarps * kExchangeBytes : 0) +
                    (p.parts - 1) * cols * 128 * 4;
  p.ring_bytes = limit - fixed;
  const size_t smem = (size_t)limit;
  int clusters = 0;
  const ep_status_t s = most_clusters<F>(di, p.parts, &clusters);
  if (s != EP_OK) return s;
  if (tiles < clusters) clusters = (int)tiles;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * p.parts * clusters);
  cfg.blockDim = dim3(threads_of(F));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2 * p.parts;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kUsePdl ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, product_kernel<F>, p);
  return e == cudaSuccess ? EP_OK : cuda_fail(e, "product launch");
}

// Rows of `length`, `pitch` elements apart, by halves of B of every height
// that a tile may have.
ep_status_t row_maps(Params &p, const void *rows, int length, int cap, int64_t pitch) {
  const uint64_t dims[] = {(uint64_t)length, (uint64_t)cap}, strides[] = {pitch * kSize};
  for (int i = 0; i < p.max_cols / 32; ++i) {
    const uint32_t box[] = {kInner, 16u * (i + 1)};
    const ep_status_t s = encode_map(&p.b[i], rows, 2, dims, strides, box);
    if (s != EP_OK) return s;
  }
  return EP_OK;
}

// Rows of `length`, `pitch` elements apart, read with the outer dimension
// contiguous: blocks of 64 of a row by 64 rows, two blocks a copy where the
// length allows it.
[[maybe_unused]] ep_status_t block_map(CUtensorMap *map, bool *blocks, const void *rows, int length, int cap, int64_t pitch) {
  *blocks = length % 64 == 0;
  if (*blocks) {
    const uint64_t dims[] = {64, (uint64_t)cap, (uint64_t)length / 64}, strides[] = {pitch * kSize, 64 * kSize};
    const uint32_t box[] = {64, kInner, 2};
    return encode_map(map, rows, 3, dims, strides, box);
  }
  const uint64_t dims[] = {(uint64_t)length, (uint64_t)cap}, strides[] = {pitch * kSize};
  const uint32_t box[] = {64, kInner};
  return encode_map(map, rows, 2, dims, strides, box);
}

// The weights [E][wide][hidden] as A of a form.
[[maybe_unused]] ep_status_t weight_map(Params &p, Form form, const void *w, int wide, int hidden) {
  const uint64_t E = p.E, n = wide, h = hidden;
  if (form == kPlain || (dense(form) && !gated(form))) {
    const uint64_t dims[] = {h, n, E}, strides[] = {h * kSize, n * h * kSize};
    const uint32_t box[] = {kInner, 128, 1};
    return encode_map(&p.a, w, 3, dims, strides, box);
  }
  if (gated(form)) {
    const uint64_t dims[] = {h, n / 2, 2, E}, strides[] = {h * kSize, n / 2 * h * kSize, n * h * kSize};
    const uint32_t box[] = {kInner, 64, 2, 1};
    return encode_map(&p.a, w, 4, dims, strides, box);
  }
  p.a_blocks = hidden % 64 == 0;
  if (p.a_blocks) {
    const uint64_t dims[] = {64, n, h / 64, E}, strides[] = {h * kSize, 64 * kSize, n * h * kSize};
    const uint32_t box[] = {64, kInner, 2, 1};
    return encode_map(&p.a, w, 4, dims, strides, box);
  }
  const uint64_t dims[] = {h, n, E}, strides[] = {h * kSize, n * h * kSize};
  const uint32_t box[] = {64, kInner, 1};
  return encode_map(&p.a, w, 3, dims, strides, box);
}

// A product whose columns are the experts' rows (`pitch` elements apart), cut
// and launched.
template <Form F>
ep_status_t launch_rows_form(Params &p, const void *rows, int64_t pitch, cudaStream_t stream) {
  const DeviceInfo *di = current_device_info();
  if (di == nullptr) return EP_ERR_CUDA;
  Cut c;
  ep_status_t s = choose<F>(di, p.cap, p.E, p.most_rows, p.a_tiles, p.inner, &c);
  if (s != EP_OK) return s;
  p.max_cols = c.cols;
  p.parts = c.parts;
  s = row_maps(p, rows, p.inner, p.cap, pitch);
  if (s != EP_OK) return s;
  return launch_form<F>(p, most_tiles(p.cap, p.E, c.cols) * p.a_tiles, stream);
}

}  // namespace

}  // namespace ep
