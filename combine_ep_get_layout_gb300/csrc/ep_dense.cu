// A product shared by all rows, x w^T, with bias, activation and residual in
// its epilogue, and its gradients.
//
//   z = x w^T + b,  out = act(z) + residual
//   d = act'(z) grad,  grad_x = d w,  grad_w = d^T x,  grad_bias = sum of d
//
// bf16 operands, sums in fp32, results rounded once.  d is an operand of two
// products and kept in bf16; the bias's gradient is summed before that.
#include "ep_pair.cuh"

namespace ep {

namespace {

// act'(z), but for ReLU
__device__ __forceinline__ float slope_of(int act, float z) {
  float s;
  switch (act) {
    case EP_ACT_SILU:
      s = sigmoid_of(z);
      return s * (1.0f + z * (1.0f - s));
    case EP_ACT_GELU: {
      float density;
      s = normal_integral(z, density);
      return fmaf(z * kRootOneTwoPi, density, s);
    }
    case EP_ACT_GELU_TANH:
      s = tanh_gate(z);
      z = fminf(fmaxf(z, -16.0f), 16.0f);  // s (1 - s) is 0 there; z^2 stays finite
      return s + z * s * (1.0f - s) * 2.0f * kRootTwoPi * (1.0f + 3.0f * kCubic * z * z);
    default:
      return 1.0f;
  }
}

// act'(z) grad.  ReLU's is a choice, not a product: what is cut off stays 0
// whatever came back to it.
__device__ __forceinline__ float through(int act, float z, float grad) {
  if (act == EP_ACT_RELU) return z > 0.0f ? grad : 0.0f;
  return slope_of(act, z) * grad;
}

// d = act'(z) grad for the products, rounded, and the bias's gradient: one
// pass over flat rows by eight columns a thread, whose sums a block keeps for
// a slice of the rows; a second kernel adds the slices in their order.
constexpr int kWide = 32 * 8;     // columns of a block
constexpr int kRowLanes = 8;      // rows of a block at a time
constexpr int kGradBlocks = 608;  // four an SM (of 152)
constexpr int kLeastRows = 32;    // of a slice

constexpr int kJoinedRows = 384;  // at most, whose slices are a cluster (set for calls outside graphs)

// A column block's slices are neighbours.  Few rows: as many slices as a
// cluster has blocks, which add them up themselves and save a launch, 3.4 us
// of the host's (in a graph, 128 rows 1024 -> 1024: 13.1 us, 14.4 with the
// launch; 333 rows 512 -> 1408 16.7 and 16.0; of 1024 rows 11 more).
struct Slices {
  int columns, slices, rows;  // blocks of columns, of rows, and a slice's rows
  bool joined;
};

Slices slices_of(int rows, int width) {
  Slices s;
  s.columns = up(width, kWide);
  s.joined = rows <= kJoinedRows && width % 8 == 0;
  if (s.joined) {
    s.rows = up(up(rows, kClusterMost), 2 * kRowLanes) * 2 * kRowLanes;
    s.slices = up(rows, s.rows > 0 ? s.rows : 1);
    return s;
  }
  const int most = s.columns < kGradBlocks ? kGradBlocks / s.columns : 1;
  s.rows = up(up(rows, most), kRowLanes) * kRowLanes;
  if (s.rows < kLeastRows) s.rows = kLeastRows;
  s.slices = up(rows, s.rows);
  return s;
}

__device__ __forceinline__ void unpack8(const int4 &f, float (&v)[8]) {
  const uint32_t w[4] = {(uint32_t)f.x, (uint32_t)f.y, (uint32_t)f.z, (uint32_t)f.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = bf16_lo(w[j]);
    v[2 * j + 1] = bf16_hi(w[j]);
  }
}

__device__ __forceinline__ int4 pack8(const float (&v)[8]) {
  return make_int4((int)pack_bf16x2(v[0], v[1]), (int)pack_bf16x2(v[2], v[3]), (int)pack_bf16x2(v[4], v[5]),
                   (int)pack_bf16x2(v[6], v[7]));
}

// 4096 rows x 4096 (gelu) 20 us, 8192 x 2 x 2048 (SwiGLU) 20 us, 168 MB, of
// which some stay in L2; with divisions in the sigmoid 25 and 25, then with
// three blocks an SM, so in more than one wave, 28 and 32.
template <bool GATED, bool BF16>
__global__ void __launch_bounds__(32 * kRowLanes, 4) dense_gradient_kernel(DenseBackwardArgs p, float *sums, Slices cut) {
  constexpr int kHalves = GATED ? 2 : 1, kUnroll = 2;
  __shared__ float s_sums[kRowLanes][kWide], s_total[kHalves][kWide];
  const int slice = blockIdx.x % cut.slices, lane = threadIdx.x % 32, row = threadIdx.x / 32;
  const int column0 = blockIdx.x / cut.slices * kWide, n = column0 + lane * 8;
  const int64_t wide = (int64_t)kHalves * p.width;
  const bool there = n < p.width;
  const int64_t first = (int64_t)slice * cut.rows, last = min(first + cut.rows, (int64_t)p.num_rows);
  float sum[kHalves][8] = {};
  griddep_wait();
  griddep_launch_dependents();
  for (int64_t t = first + row; there && t < last; t += kRowLanes * kUnroll) {
    int4 g[kUnroll][BF16 ? 1 : 2], z[kUnroll][kHalves];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int64_t r = min(t + i * kRowLanes, last - 1);
      const char *from = static_cast<const char *>(p.grad) + (r * p.width + n) * (BF16 ? 2 : 4);
#pragma unroll
      for (int h = 0; h < (BF16 ? 1 : 2); ++h) g[i][h] = __ldcs(reinterpret_cast<const int4 *>(from) + h);
      if (GATED || p.activation != EP_ACT_NONE) {
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
          z[i][h] = __ldcs(reinterpret_cast<const int4 *>(p.preact + r * wide + h * p.width + n));
      }
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int64_t r = t + i * kRowLanes;
      if (r >= last) break;
      float d[8], a[8], other[8];
      if (BF16) {
        unpack8(g[i][0], d);
      } else {
        const int4 lo = g[i][0], hi = g[i][BF16 ? 0 : 1];
        const int w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = __int_as_float(w[j]);
      }
      if (GATED) {
        unpack8(z[i][0], a);
        float u[8];
        unpack8(z[i][GATED ? 1 : 0], u);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float s = sigmoid_of(a[j]);
          other[j] = d[j] * (a[j] * s);
          d[j] *= u[j] * s * (1.0f + a[j] * (1.0f - s));
          sum[GATED ? 1 : 0][j] += other[j];
        }
      } else if (p.activation != EP_ACT_NONE) {
        unpack8(z[i][0], a);
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = through(p.activation, a[j], d[j]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[0][j] += d[j];
      if (p.grad_preact != nullptr) {
        *reinterpret_cast<int4 *>(p.grad_preact + r * wide + n) = pack8(d);
        if (GATED) *reinterpret_cast<int4 *>(p.grad_preact + r * wide + p.width + n) = pack8(other);
      }
    }
  }
  if (p.grad_bias == nullptr) return;
#pragma unroll
  for (int h = 0; h < kHalves; ++h) {
#pragma unroll
    for (int j = 0; j < 8; ++j) s_sums[row][j * 32 + lane] = sum[h][j];  // without bank conflicts
    __syncthreads();
    const int c = threadIdx.x, column = column0 + c % 32 * 8 + c / 32;
    float total = s_sums[0][c];
#pragma unroll
    for (int i = 1; i < kRowLanes; ++i) total += s_sums[i][c];
    if (cut.joined)
      s_total[h][c] = total;
    else if (column < p.width)
      sums[slice * wide + h * p.width + column] = total;
    __syncthreads();
  }
  if (!cut.joined) return;
  cluster_sync();
  // every block of the cluster adds up a share of the columns, in the slices' order
  for (int i = slice * kWide * kHalves / cut.slices + threadIdx.x; i < (slice + 1) * kWide * kHalves / cut.slices;
       i += 32 * kRowLanes) {
    const int h = i / kWide, c = i % kWide, column = column0 + c % 32 * 8 + c / 32;
    float v[kClusterMost], total = 0.0f;
#pragma unroll
    for (int s = 0; s < kClusterMost; ++s)
      v[s] = s < cut.slices ? load_cluster(map_shared(smem_addr(&s_total[h][c]), s)) : 0.0f;
#pragma unroll
    for (int s = 0; s < kClusterMost; ++s) total += v[s];
    if (column >= p.width) continue;
    const int64_t at = (int64_t)h * p.width + column;
    if (p.bias_bf16)
      static_cast<uint16_t *>(p.grad_bias)[at] = (uint16_t)(pack_bf16x2(total, 0.0f) & 0xffffu);
    else
      static_cast<float *>(p.grad_bias)[at] = total;
  }
  cluster_sync();  // before a block whose sums are read ends
}

// Rows that are not of whole 16 bytes: a column a thread, a slice's rows a
// block (32 or more).
template <bool GATED>
__global__ void __launch_bounds__(kWide) dense_gradient_any_kernel(DenseBackwardArgs p, float *sums, Slices cut, int64_t pitch) {
  const int slice = blockIdx.x % cut.slices, n = blockIdx.x / cut.slices * kWide + threadIdx.x;
  const int64_t wide = (GATED ? 2 : 1) * (int64_t)p.width;
  const int64_t first = (int64_t)slice * cut.rows, last = min(first + cut.rows, (int64_t)p.num_rows);
  griddep_wait();
  griddep_launch_dependents();
  if (n >= p.width) return;
  const auto put = [&](int64_t i, float v) { p.grad_preact[i] = (uint16_t)(pack_bf16x2(v, 0.0f) & 0xffffu); };
  float sum = 0.0f, other = 0.0f;
#pragma unroll 4
  for (int64_t t = first; t < last; ++t) {
    float d = load_param(p.grad, p.grad_bf16, t * p.width + n);
    if (GATED) {
      const float g = load_param(p.preact, true, t * wide + n), u = load_param(p.preact, true, t * wide + p.width + n);
      const float s = sigmoid_of(g), du = d * (g * s);
      d *= u * s * (1.0f + g * (1.0f - s));
      other += du;
      if (p.grad_preact != nullptr) put(t * pitch + p.width + n, du);
    } else if (p.activation != EP_ACT_NONE) {
      d = through(p.activation, load_param(p.preact, true, t * wide + n), d);
    }
    if (p.grad_preact != nullptr) put(t * pitch + n, d);
    sum += d;
  }
  if (p.grad_bias == nullptr) return;
  sums[slice * wide + n] = sum;
  if (GATED) sums[slice * wide + p.width + n] = other;
}

constexpr int kJoinWarps = 16;

// The slices by sixteen warps, ten of each read at once, then those in their
// order; a column a lane.  (8192 rows, 256 columns, 256 slices: 4.9 us with
// the pass over the rows, by eight warps 5.4.)
__global__ void __launch_bounds__(32 * kJoinWarps) dense_bias_kernel(const float *sums, int slices, int wide, void *out, bool bf16) {
  __shared__ float s[kJoinWarps][32];
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, n = blockIdx.x * 32 + lane;
  constexpr int kAtOnce = 10;
  float sum = 0.0f;
  for (int first = warp; first < slices; first += kJoinWarps * kAtOnce) {
    float v[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int i = first + k * kJoinWarps;
      v[k] = i < slices && n < wide ? sums[(int64_t)i * wide + n] : 0.0f;
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) sum += v[k];
  }
  s[warp][lane] = sum;
  __syncthreads();
  if (warp != 0 || n >= wide) return;
#pragma unroll
  for (int i = 1; i < kJoinWarps; ++i) sum += s[i][lane];
  if (bf16)
    static_cast<uint16_t *>(out)[n] = (uint16_t)(pack_bf16x2(sum, 0.0f) & 0xffffu);
  else
    static_cast<float *>(out)[n] = sum;
}

// The weights' gradient of few tiles of 256 x 256: pairs take segments of the
// rows, whose sums a second kernel adds.  That costs about 16 steps of 64
// rows, so it has to save more (with the bias's kernel): 8192 rows 7168 -> 256
// (28 tiles) 42 us, by two segments 35; 512 -> 512 (4 tiles) 38 us, by
// sixteen 17; 128 -> 128 (one) 37 us, by sixteen 10; 333 rows 512 -> 1408
// stay whole, 8.5 us.
constexpr int kPairs = 76;          // that run at once (152 SMs)
constexpr int kLeastSteps = 8;      // of a segment
constexpr int kSegmentsCost = 16;   // steps

struct Segments {
  int count, rows;
};

Segments segments_of(int rows, int wide, int hidden) {
  const int tiles = up(wide, 256) * up(hidden, 256), steps = up(rows, kInner);
  int most = tiles < kPairs ? kPairs / tiles : 1;
  if (most > steps / kLeastSteps) most = steps / kLeastSteps;
  if (most < 2 || steps - up(steps, most) < kSegmentsCost) return Segments{1, rows};
  const int each = up(steps, most);
  return Segments{up(steps, each), each * kInner};
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

size_t sums_bytes(int rows, int width, int wide) { return round256((size_t)slices_of(rows, width).slices * wide * sizeof(float)); }

// The segments' sums added up in their order, eight elements a thread.
__global__ void __launch_bounds__(256) dense_segments_kernel(const float *parts, int segments, int64_t count, uint16_t *out) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (at >= count) return;
  float v[8] = {};
#pragma unroll 4
  for (int i = 0; i < segments; ++i) {
    const float4 a = __ldcg(reinterpret_cast<const float4 *>(parts + i * count + at));
    const float4 b = __ldcg(reinterpret_cast<const float4 *>(parts + i * count + at) + 1);
    v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
    v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
  }
  *reinterpret_cast<int4 *>(out + at) = pack8(v);
}

// What the products of a call share: one expert with every row.
Params params_of(int rows, int wide, int width, int hidden, uint32_t *error_word) {
  Params p = {};
  p.most_rows = p.cap = rows;
  p.error_word = error_word;
  p.E = 1;
  p.wide = wide;
  p.width = width;
  p.hidden = hidden;
  return p;
}

}  // namespace

ep_status_t launch_dense(const DenseArgs &a, cudaStream_t stream) {
  if (a.num_rows == 0) return EP_OK;
  const bool pairs = a.activation == EP_ACT_SWIGLU;
  Params p = params_of(a.num_rows, pairs ? 2 * a.width : a.width, a.width, a.hidden, a.error_word);
  p.inner = a.hidden;
  p.a_tiles = up(a.width, pairs ? 128 : 256);
  p.out = static_cast<uint16_t *>(a.out);
  p.preact = a.preact;
  p.bias = a.bias;
  p.bias_bf16 = a.bias_bf16;
  p.residual = a.residual;
  p.activation = a.activation;
  const ep_status_t s = weight_map(p, pairs ? kDenseGated : kDense, a.w, p.wide, a.hidden);
  if (s != EP_OK) return s;
  if (!a.out_bf16)
    return pairs ? launch_rows_form<kDenseGated32>(p, a.x, a.row_stride, stream)
                 : launch_rows_form<kDense32>(p, a.x, a.row_stride, stream);
  return pairs ? launch_rows_form<kDenseGated>(p, a.x, a.row_stride, stream)
               : launch_rows_form<kDense>(p, a.x, a.row_stride, stream);
}

size_t dense_workspace_bytes(int num_rows, int hidden, int width, ep_activation_t activation) {
  const int wide = activation == EP_ACT_SWIGLU ? 2 * width : width;
  const int segments = segments_of(num_rows, wide, hidden).count;
  return sums_bytes(num_rows, width, wide) + (segments > 1 ? (size_t)segments * wide * hidden * sizeof(float) : 0);
}

ep_status_t launch_dense_backward(const DenseBackwardArgs &a, cudaStream_t stream) {
  const bool pairs = a.activation == EP_ACT_SWIGLU;
  const int wide = pairs ? 2 * a.width : a.width;
  const Slices cut = slices_of(a.num_rows, a.width);
  const bool any_width = a.width % 8 != 0;
  const bool made = a.activation != EP_ACT_NONE || !a.grad_bf16 || wide % 8 != 0;  // d is not `grad` itself
  const int64_t pitch = made ? up(wide, 8) * 8 : wide;                             // between d's rows
  float *sums = static_cast<float *>(a.workspace);
  cudaError_t e = cudaSuccess;
  if (a.num_rows > 0 && (a.grad_bias != nullptr || a.grad_preact != nullptr)) {
    const auto kernel = pairs ? (a.grad_bf16 ? dense_gradient_kernel<true, true> : dense_gradient_kernel<true, false>)
                              : (a.grad_bf16 ? dense_gradient_kernel<false, true> : dense_gradient_kernel<false, false>);
    if (any_width)
      e = launch_kernel(pairs ? dense_gradient_any_kernel<true> : dense_gradient_any_kernel<false>, cut.columns * cut.slices,
                        kWide, 0, stream, false, a, sums, cut, pitch);
    else if (cut.joined)
      e = launch_clusters(kernel, cut.columns * cut.slices, 32 * kRowLanes, 0, stream, cut.slices, a, sums, cut);
    else
      e = launch_kernel(kernel, cut.columns * cut.slices, 32 * kRowLanes, 0, stream, false, a, sums, cut);
  }
  if (e == cudaSuccess && a.grad_bias != nullptr && !(cut.joined && a.num_rows > 0))
    e = launch_kernel(dense_bias_kernel, up(wide, 32), 32 * kJoinWarps, 0, stream, false, (const float *)sums, cut.slices,
                      wide, a.grad_bias, a.bias_bf16);
  if (e != cudaSuccess) return cuda_fail(e, "dense_backward launch");
  const uint16_t *d = made ? a.grad_preact : static_cast<const uint16_t *>(a.grad);
  if (a.grad_x != nullptr && a.num_rows > 0) {
    Params p = params_of(a.num_rows, wide, a.hidden, a.hidden, a.error_word);
    p.inner = wide;
    p.a_tiles = up(a.hidden, 256);
    p.out = a.grad_x;
    ep_status_t s = weight_map(p, kDenseGradX, a.w, wide, a.hidden);
    if (s == EP_OK) s = launch_rows_form<kDenseGradX>(p, d, pitch, stream);
    if (s != EP_OK) return s;
  }
  if (a.grad_w != nullptr) {
    Params p = params_of(a.num_rows, wide, a.width, a.hidden, a.error_word);
    p.parts = 1;
    p.max_cols = kMaxCols;
    p.a_tiles = up(wide, 256);
    p.b_tiles = up(a.hidden, 256);
    p.out = a.grad_w;
    // without rows nothing is copied: the maps only need an address
    const bool any = a.num_rows > 0;
    const int rows = any ? a.num_rows : 1;
    const Segments seg = segments_of(a.num_rows, wide, a.hidden);
    const bool parts = seg.count > 1;
    float *part = reinterpret_cast<float *>(static_cast<char *>(a.workspace) + sums_bytes(a.num_rows, a.width, wide));
    ep_status_t s = block_map(&p.a, &p.a_blocks, any ? d : a.grad_w, wide, rows, any ? pitch : up(wide, 8) * 8);
    // (fp32 as two bf16 each)
    const uint64_t each = parts ? 2 : 1, columns = each * a.hidden;
    const uint64_t dims[] = {columns, (uint64_t)wide, (uint64_t)seg.count};
    const uint64_t strides[] = {columns * kSize, (uint64_t)wide * columns * kSize};
    const uint32_t box[] = {64, 32, 1};
    if (s == EP_OK) s = encode_map(&p.grad, parts ? (const void *)part : a.grad_w, 3, dims, strides, box);
    if (s == EP_OK) s = block_map(&p.b[0], &p.b_blocks, any ? a.x : a.grad_w, a.hidden, rows, any ? a.row_stride : a.hidden);
    const int64_t tiles = (int64_t)p.a_tiles * p.b_tiles * seg.count;
    p.segments = seg.count;
    p.rows_each = seg.rows;
    if (s == EP_OK) s = parts ? launch_form<kDenseGradWPart>(p, tiles, stream) : launch_form<kDenseGradW>(p, tiles, stream);
    if (s == EP_OK && parts) {
      const int64_t count = (int64_t)wide * a.hidden;
      e = launch_kernel(dense_segments_kernel, (int)((count / 8 + 255) / 256), 256, 0, stream, false, (const float *)part,
                        seg.count, count, a.grad_w);
      if (e != cudaSuccess) return cuda_fail(e, "dense_segments launch");
    }
    if (s != EP_OK) return s;
  }
  return EP_OK;
}

}  // namespace ep
