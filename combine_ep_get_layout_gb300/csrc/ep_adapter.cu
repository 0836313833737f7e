// A shared projection with low-rank adapters of many requests beside it:
//
//   y[t] = x[t] w^T + scale[a] (x[t] A_a^T) B_a^T,    a = adapter_idx[t]
//
// (no second term where a = -1).  bf16 in and out, sums in fp32.
//
// Two kernels.  adapter_low_kernel computes low[t] = scale[a] x[t] A_a^T for
// a tile of rows: the down-projections of the adapters that the tile names are
// stacked, 128 rows of them at a time, and multiplied with all its rows on the
// tensor cores; of every column only its own adapter's part is kept.  For the
// projection (ep_pair.cuh, kAdapter) the adapters of a tile, side by side, are
// a longer inner dimension: 64 / rank of them a step, their B_a against low[t]
// in its adapter's columns and zeros in the others, so the second term is
// summed in tensor memory with the first.
//
// low is kept in bf16, as the tensor cores take it: 2^-8 of the low term, the
// size of the result's own rounding.
//
// Measured: 8192 rows 7168 -> 4096, rank 32: 313 to 325 us, of which the low
// rows 32 (the projection's power limit bounds it); 1021 rows 4096 -> 1000, 40
// adapters of rank 8: 20 to 21 us in a graph; 32 rows 4096 -> 4096, 24 adapters
// of rank 16: 10.5 us in a graph, where reading the weights takes 6 (the low
// rows and the gather come one after the other).
#include "ep_pair.cuh"

namespace ep {

namespace {

constexpr int kLowThreads = 192;  // warps 0-3 copy A and read the results, 4 copies x, 5 issues the products
constexpr int kLowMaxStages = 8;
constexpr int kLowChunk = 32 * 128 * 4;  // 32 columns of the results, fp32
constexpr int kMaxSplits = 8;     // CTAs of a cluster

struct LowParams {
  CUtensorMap x;  // boxes of 64 x cols
  const uint16_t *a, *rows_x;
  const int64_t *index;
  const float *scale;
  uint32_t *error_word;
  int T, hidden, rank, adapters;
  int cols;    // rows of a tile
  int splits;  // of the inner dimension: the CTAs of a cluster
  float *part;      // [splits][T][rank]
  uint16_t *low;    // [T][rank]
  int32_t *plan;    // [tiles][kPlanWords]
};

struct LowBarriers {
  uint64_t full[kLowMaxStages], empty[kLowMaxStages];
  uint64_t acc_full, acc_empty;
  uint32_t tmem;
};

// The adapters of a tile in the order in which its rows name them (*list),
// each row's place among them or -1 (*place), their number; written to the
// plan if `write`.  table[adapters] holds kMaxCols in every entry.  The whole
// block calls it.
__device__ __forceinline__ int list_adapters(const LowParams &p, int tile, int *table, int *place, int *list,
                                             uint32_t *first_of, bool write) {
  const int first = tile * p.cols, rows = min(p.cols, p.T - first);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < p.cols; i += blockDim.x) {
    int a = -1;
    if (i < rows) {
      const int64_t v = p.index[first + i];
      if (v >= 0 && v < p.adapters)
        a = (int)v;
      else if (v != -1)
        set_error(p.error_word, EP_ERRBIT_BAD_INDEX);
    }
    place[i] = a;
    if (a >= 0) atomicMin(&table[a], i);
  }
  __syncthreads();
  for (int b = warp; b < kMaxCols / 32; b += blockDim.x / 32) {
    const int i = b * 32 + lane;
    const int a = i < p.cols ? place[i] : -1;
    const uint32_t m = __ballot_sync(0xffffffffu, a >= 0 && table[a] == i);
    if (lane == 0) first_of[b] = m;
  }
  __syncthreads();
  int count = 0;
#pragma unroll
  for (int b = 0; b < kMaxCols / 32; ++b) count += __popc(first_of[b]);
  for (int i = threadIdx.x; i < p.cols; i += blockDim.x) {
    const int a = place[i];
    if (a < 0) continue;
    const int f = table[a];
    int n = 0;  // rows before f that name an adapter first
#pragma unroll
    for (int b = 0; b < kMaxCols / 32; ++b)
      n += __popc(first_of[b] & (b < f >> 5 ? ~0u : b == f >> 5 ? (1u << (f & 31)) - 1u : 0u));
    if (f == i) list[n] = a;
    place[i] = n;
  }
  __syncthreads();
  if (write) {
    int32_t *plan = p.plan + (int64_t)tile * kPlanWords;
    if (threadIdx.x == 0) plan[0] = count;
    for (int i = threadIdx.x; i < count; i += blockDim.x) plan[1 + i] = list[i];
    for (int i = threadIdx.x; i < p.cols; i += blockDim.x) plan[1 + kMaxCols + i] = place[i];
  }
  return count;
}

// The low rows of few rows: SHARE warps for two low values of a row, which
// read their part of the adapter's down-projection by themselves (rows of one
// adapter meet it in L2); the first blocks make the tiles' plans.
constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;
constexpr int64_t kRowBytes = 256 << 20;

template <int SHARE>
__global__ void __launch_bounds__(kRowThreads) adapter_row_kernel(const __grid_constant__ LowParams p, int tiles) {
  extern __shared__ int s_dyn[];  // [adapters]
  __shared__ float2 s_sum[kRowWarps];
  __shared__ int s_place[kMaxCols], s_list[kMaxCols];
  __shared__ uint32_t s_first[kMaxCols / 32];
  if ((int)blockIdx.x < tiles)
    for (int i = threadIdx.x; i < p.adapters; i += kRowThreads) s_dyn[i] = kMaxCols;
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  if ((int)blockIdx.x < tiles) {
    list_adapters(p, blockIdx.x, s_dyn, s_place, s_list, s_first, true);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = warp % SHARE;
  const int item = ((int)blockIdx.x - tiles) * (kRowWarps / SHARE) + warp / SHARE;
  const int t = item / (p.rank / 2), i = item % (p.rank / 2) * 2;
  const int64_t a = t < p.T ? p.index[t] : -1;
  const bool some = a >= 0 && a < p.adapters;
  if (SHARE == 1 && !some) return;
  const float f = p.scale == nullptr || !some ? 1.0f : __ldg(p.scale + a);
  const uint16_t *x = p.rows_x + (int64_t)t * p.hidden;
  const uint16_t *v = p.a + (a * p.rank + i) * p.hidden;
  float sum[2] = {0.0f, 0.0f};
#pragma unroll 4
  for (int k = some ? (part * 32 + lane) * 8 : p.hidden; k < p.hidden; k += SHARE * 256) {
    const int4 xv = __ldg(reinterpret_cast<const int4 *>(x + k));
    const int4 a0 = __ldg(reinterpret_cast<const int4 *>(v + k));
    const int4 a1 = __ldg(reinterpret_cast<const int4 *>(v + p.hidden + k));
    const uint32_t *xw = reinterpret_cast<const uint32_t *>(&xv);
    const uint32_t *w0 = reinterpret_cast<const uint32_t *>(&a0), *w1 = reinterpret_cast<const uint32_t *>(&a1);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      sum[0] += bf16_lo(xw[j]) * bf16_lo(w0[j]);
      sum[0] += bf16_hi(xw[j]) * bf16_hi(w0[j]);
      sum[1] += bf16_lo(xw[j]) * bf16_lo(w1[j]);
      sum[1] += bf16_hi(xw[j]) * bf16_hi(w1[j]);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], o);
    sum[1] += __shfl_xor_sync(0xffffffffu, sum[1], o);
  }
  if constexpr (SHARE > 1) {  // the parts in their order
    if (lane == 0) s_sum[warp] = make_float2(sum[0], sum[1]);
    __syncthreads();
#pragma unroll
    for (int q = 1; q < SHARE; ++q) {
      if (part > 0) break;
      sum[0] += s_sum[warp + q].x;
      sum[1] += s_sum[warp + q].y;
    }
  }
  if (some && part == 0 && lane == 0)
    *reinterpret_cast<uint32_t *>(p.low + (int64_t)t * p.rank + i) = pack_bf16x2(sum[0] * f, sum[1] * f);
}

// A barrier of the first four warps; whether all of them say `ok`.
__device__ __forceinline__ bool four_agree(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)ok)
      : "memory");
  return r != 0;
}

// STAGES: of the ring; STAGES - 1 steps of A are in flight.
template <int STAGES>
__global__ void __launch_bounds__(kLowThreads) adapter_low_kernel(const __grid_constant__ LowParams p) {
  extern __shared__ char s_raw[];
  __shared__ LowBarriers s_bar;
  __shared__ int s_place[kMaxCols];  // of a row's adapter in the tile's list, or -1
  __shared__ int s_list[kMaxCols];
  __shared__ uint32_t s_first[kMaxCols / 32];
  char *ring = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(s_raw) + 1023) & ~uintptr_t(1023));
  const int stage_bytes = kABytes + p.cols * 128;
  // [adapters]: first row that names it; later 32 columns of the results
  int *s_table = reinterpret_cast<int *>(ring + STAGES * stage_bytes);
  float *s_chunk = reinterpret_cast<float *>(s_table);
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int first = blockIdx.x * p.cols, rows = min(p.cols, p.T - first);
  const int split = blockIdx.y;

  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&s_bar.full[i], 4 * 32 + 1);
      mbar_init(&s_bar.empty[i], 1);
    }
    mbar_init(&s_bar.acc_full, 1);
    mbar_init(&s_bar.acc_empty, 4);
    fence_barrier_init();
    prefetch_map(&p.x);
  }
  __syncwarp();
  if (warp == 5) tmem_alloc_one(&s_bar.tmem, kMaxCols);
  for (int i = threadIdx.x; i < p.adapters; i += kLowThreads) s_table[i] = kMaxCols;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_bar.tmem;
  griddep_wait();
  griddep_launch_dependents();

  const int count = list_adapters(p, blockIdx.x, s_table, s_place, s_list, s_first, split == 0 && blockIdx.z == 0);

  const int per = 128 / p.rank;  // adapters of a stack
  const int stacks = ceil_div(count, per);
  const int all_steps = ceil_div(p.hidden, kInner);
  const int k0 = all_steps * split / p.splits, k1 = all_steps * (split + 1) / p.splits;
  bool ok = true;
  int stage = 0;
  uint32_t phase = 0, acc_phase = 0;
  const auto advance = [&] {
    if (++stage == STAGES) {
      stage = 0;
      phase ^= 1;
    }
  };
  for (int s = blockIdx.z; s < stacks; s += gridDim.z) {
    const int stacked = min(per, count - s * per);
    if (warp < 4) {
      // this warp's 32 rows of the stack, four at a time, eight lanes a row
      const uint16_t *src[8];
      uint32_t to[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = warp * 32 + i * 4 + (lane >> 3), j = r / p.rank;
        src[i] = j < stacked ? p.a + ((int64_t)s_list[s * per + j] * p.rank + (r - j * p.rank)) * p.hidden + (lane & 7) * 8
                             : nullptr;
        to[i] = r * 128 + (((lane & 7) ^ (r & 7)) << 4);
      }
      int filled = 0;
      int hand = stage;  // the stage handed over next
      for (int k = k0; k < k1 + (STAGES - 1); ++k) {
        if (k < k1) {
          if (ok) ok = __all_sync(0xffffffffu, mbar_wait_pair(&s_bar.empty[stage], phase ^ 1));
          const uint32_t a = smem_addr(ring + stage * stage_bytes);
          const int at = k * kInner;
          const bool some = at + (lane & 7) * 8 < p.hidden;
          if (ok) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (src[i] != nullptr) copy16(a + to[i], some ? src[i] + at : src[i], some);
          }
          ++filled;
          advance();
        }
        copy_commit();
        if (k >= k0 + (STAGES - 1)) {
          copy_wait<(STAGES - 1)>();
          fence_proxy_async_smem();
          mbar_arrive(&s_bar.full[hand]);
          if (++hand == STAGES) hand = 0;
        }
      }
      copy_wait<0>();
      // results: lane l holds row l of the stack, of adapter l / rank
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait_pair(&s_bar.acc_full, acc_phase));
      acc_phase ^= 1;
      tc_fence_after();
      if (four_agree(ok)) {
        const int fours = p.rank / 4;
        for (int c = 0; c < p.cols; c += 32) {
          float v[32];
          tmem_load32(tmem + c + ((uint32_t)(warp * 32) << 16), v);
#pragma unroll
          for (int q = 0; q < 32; ++q) s_chunk[q * 128 + warp * 32 + lane] = v[q];
          asm volatile("bar.sync 1, 128;" ::: "memory");
          // of every row its own adapter's part, four values at a time
          for (int item = threadIdx.x; item < 32 * fours; item += 128) {
            const int q = item / fours, i = item - q * fours;
            const int place = c + q < p.cols ? s_place[c + q] : -1;
            if (place < s * per || place >= s * per + stacked) continue;
            const float4 f = *reinterpret_cast<const float4 *>(s_chunk + q * 128 + (place - s * per) * p.rank + i * 4);
            const int64_t at = (int64_t)(first + c + q) * p.rank + i * 4;
            if (p.splits == 1) {
              const float g = p.scale == nullptr ? 1.0f : __ldg(p.scale + s_list[place]);
              *reinterpret_cast<uint2 *>(p.low + at) =
                  make_uint2(pack_bf16x2(f.x * g, f.y * g), pack_bf16x2(f.z * g, f.w * g));
            } else {
              *reinterpret_cast<float4 *>(p.part + (int64_t)split * p.T * p.rank + at) = f;
            }
          }
          asm volatile("bar.sync 1, 128;" ::: "memory");
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s_bar.acc_empty);
    } else if (warp == 4) {
      for (int k = k0; ok && k < k1; ++k) {
        ok = __all_sync(0xffffffffu, mbar_wait_pair(&s_bar.empty[stage], phase ^ 1));
        if (!ok) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(&s_bar.full[stage], p.cols * 128);
          tile_load_one(smem_addr(ring + stage * stage_bytes) + kABytes, &p.x, k * kInner, first, &s_bar.full[stage]);
        }
        __syncwarp();
        advance();
      }
    } else {
      const uint32_t idesc = mma_desc_one(p.cols);
      ok = ok && __all_sync(0xffffffffu, mbar_wait_pair(&s_bar.acc_empty, acc_phase ^ 1));
      acc_phase ^= 1;
      tc_fence_after();
      for (int k = k0; ok && k < k1; ++k) {
        ok = __all_sync(0xffffffffu, mbar_wait_pair(&s_bar.full[stage], phase));
        if (!ok) break;
        tc_fence_after();
        const uint32_t at = smem_addr(ring) + (uint32_t)(stage * stage_bytes);
        const uint32_t a = inner_desc(at), b = inner_desc(at + kABytes);
        if (elect_one()) {
#pragma unroll
          for (int j = 0; j < 4; ++j) mma_one(tmem, a + j * 2, b + j * 2, idesc, k > k0 || j > 0);
          commit_one(&s_bar.empty[stage]);
          if (k == k1 - 1) commit_one(&s_bar.acc_full);
        }
        __syncwarp();
        advance();
      }
    }
    if (p.splits > 1) {
      // the splits' parts are added in their order, each row by one CTA
      cluster_sync();
      const int fours = p.rank / 4, mine = ceil_div(rows - split, p.splits);
      for (int item = threadIdx.x; item < mine * fours; item += kLowThreads) {
        const int c = split + item / fours * p.splits, i = item % fours * 4;
        const int place = s_place[c];
        if (place < s * per || place >= s * per + stacked) continue;
        const float f = p.scale == nullptr ? 1.0f : __ldg(p.scale + s_list[place]);
        const int64_t at = (int64_t)(first + c) * p.rank + i, pitch = (int64_t)p.T * p.rank;
        float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int q = 0; q < kMaxSplits; ++q) {
          if (q < p.splits) {
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(p.part + q * pitch + at));
            sum.x += v.x;
            sum.y += v.y;
            sum.z += v.z;
            sum.w += v.w;
          }
        }
        *reinterpret_cast<uint2 *>(p.low + at) =
            make_uint2(pack_bf16x2(sum.x * f, sum.y * f), pack_bf16x2(sum.z * f, sum.w * f));
      }
    }
  }
  if (!ok) {  // a wait gave up: what was started lands well within the time waited here
    set_error(p.error_word, EP_ERRBIT_TIMEOUT);
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 2000000ull) __nanosleep(1000);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_free_one(tmem, kMaxCols);
  }
}

int low_splits(int tiles, int hidden) {
  const int steps = up(hidden, kInner);
  int n = 128 / tiles;
  if (n > kMaxSplits) n = kMaxSplits;
  if (n > steps) n = steps;
  return n < 1 ? 1 : n;
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// Where every row may read its adapter by itself: up to 256 MB from L2
// (2048 rows of rank 16, 4096 -> 1024, 40 adapters: interleaved 42 us against 101
// by stacks, in runs 34 against 28).
bool row_kernel(const AdapterArgs &a) { return (int64_t)a.num_rows * a.rank * a.hidden * 2 <= kRowBytes; }

// Warps share a row's values while four blocks an SM hold them all, since a
// warp's rounds of loads come one after the other.  The whole call with inputs
// in memory: 32 rows of rank 16, 4096 -> 4096 25 us alone, 21 shared by eight;
// 300 of rank 8, 4096 -> 1000 27, 21 shared by four; 64 of rank 64, 7168 ->
// 2048 37, 33 shared by two.  With inputs in L2: 11.2 and 10.6; 12.4 to 15.0
// and 13.5 to 14.1; 16.8 and 17.8.
ep_status_t launch_rows(const LowParams &q, int tiles, const DeviceInfo *di, cudaStream_t stream) {
  const int items = q.T * (q.rank / 2);
  int share = 1;
  while (share < kRowWarps && 2 * items * share <= 4 * di->num_sms * kRowWarps && q.hidden > 512 * share) share *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(up(items, kRowWarps / share) + tiles);
  cfg.blockDim = dim3(kRowThreads);
  cfg.dynamicSmemBytes = (size_t)q.adapters * 4;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = kUsePdl ? 1 : 0;
  const auto kernel = share == 1   ? adapter_row_kernel<1>
                      : share == 2 ? adapter_row_kernel<2>
                      : share == 4 ? adapter_row_kernel<4>
                                   : adapter_row_kernel<8>;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, q, tiles);
  return e == cudaSuccess ? EP_OK : cuda_fail(e, "adapter_row launch");
}

ep_status_t launch_low(LowParams &q, const AdapterArgs &a, int tiles, const DeviceInfo *di, cudaStream_t stream) {
  const uint64_t dims[] = {(uint64_t)a.hidden, (uint64_t)a.num_rows}, strides[] = {a.hidden * kSize};
  const uint32_t box[] = {kInner, (uint32_t)q.cols};
  const ep_status_t s = encode_map(&q.x, a.x, 2, dims, strides, box);
  if (s != EP_OK) return s;
  // stacks of adapters side by side while there are SMs for them
  const int named = a.num_adapters < q.cols ? a.num_adapters : q.cols;
  const int stacks = up(named, 128 / a.rank);
  int side = di->num_sms / (tiles * q.splits);
  side = side < 1 ? 1 : side > stacks ? stacks : side;
  const bool shallow = q.cols > 64;  // a stage of x and A: up to 48 KB, or up to 24
  const auto kernel = shallow ? adapter_low_kernel<4> : adapter_low_kernel<kLowMaxStages>;
  const size_t table = (size_t)a.num_adapters * 4;
  const size_t smem = 1024 + (shallow ? 4 : kLowMaxStages) * (kABytes + (size_t)q.cols * 128) +
                      (table > kLowChunk ? table : kLowChunk);
  static std::atomic<bool> ready[64][2];
  if (!ready[di->device][shallow]) {
    const int most = 1024 + (shallow ? 4 * (kABytes + kMaxCols * 128) : kLowMaxStages * (kABytes + 64 * 128)) +
                     EP_MAX_EXPERTS * 4;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
    ready[di->device][shallow] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(tiles, q.splits, side);
  cfg.blockDim = dim3(kLowThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = attr[0].val.clusterDim.z = 1;
  attr[0].val.clusterDim.y = q.splits;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kUsePdl ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, q);
  return e == cudaSuccess ? EP_OK : cuda_fail(e, "adapter_low launch");
}

}  // namespace

size_t adapter_workspace_bytes(int num_rows, int hidden, int rank) {
  if (num_rows == 0) return 0;
  // whatever the cut: tiles of 32 columns or more, splits as for the fewest tiles
  const int splits = low_splits(up(num_rows, kMaxCols), hidden);
  return align256((size_t)up(num_rows, 32) * kPlanWords * 4) + align256((size_t)num_rows * rank * 2) +
         align256(splits > 1 ? (size_t)splits * num_rows * rank * 4 : 0);
}

ep_status_t launch_adapter(const AdapterArgs &a, cudaStream_t stream) {
  if (a.num_rows == 0) return EP_OK;
  const DeviceInfo *di = current_device_info();
  if (di == nullptr) return EP_ERR_CUDA;
  Cut c;
  ep_status_t s = choose<kAdapter>(di, a.num_rows, 1, a.num_rows, up(a.width, 256), a.hidden, &c);
  if (s != EP_OK) return s;
  const int tiles = up(a.num_rows, c.cols);
  char *ws = static_cast<char *>(a.workspace);
  LowParams q = {};
  q.a = a.lora_a;
  q.rows_x = a.x;
  q.index = a.adapter_idx;
  q.scale = a.adapter_scale;
  q.error_word = a.error_word;
  q.T = a.num_rows;
  q.hidden = a.hidden;
  q.rank = a.rank;
  q.adapters = a.num_adapters;
  q.cols = c.cols;
  q.splits = low_splits(tiles, a.hidden);
  q.plan = reinterpret_cast<int32_t *>(ws);
  ws += align256((size_t)up(a.num_rows, 32) * kPlanWords * 4);
  q.low = reinterpret_cast<uint16_t *>(ws);
  ws += align256((size_t)a.num_rows * a.rank * 2);
  q.part = reinterpret_cast<float *>(ws);
  s = row_kernel(a) ? launch_rows(q, tiles, di, stream) : launch_low(q, a, tiles, di, stream);
  if (s != EP_OK) return s;

  Params p = {};
  p.max_cols = c.cols;
  p.parts = c.parts;
  p.most_rows = a.num_rows;
  p.error_word = a.error_word;
  p.E = 1;
  p.cap = a.num_rows;
  p.wide = p.width = a.width;
  p.inner = a.hidden;
  p.a_tiles = up(a.width, 256);
  p.out = a.out;
  p.plan = q.plan;
  p.low = q.low;
  p.up = a.lora_b;
  p.rank = a.rank;
  const uint64_t wd[] = {(uint64_t)a.hidden, (uint64_t)a.width, 1};
  const uint64_t ws_[] = {a.hidden * kSize, (uint64_t)a.hidden * a.width * kSize};
  const uint32_t wb[] = {kInner, 128, 1};
  s = encode_map(&p.a, a.w, 3, wd, ws_, wb);
  if (s != EP_OK) return s;
  s = row_maps(p, a.x, a.hidden, a.num_rows, a.hidden);
  if (s != EP_OK) return s;
  return launch_form<kAdapter>(p, (int64_t)tiles * p.a_tiles, stream);
}

}  // namespace ep
