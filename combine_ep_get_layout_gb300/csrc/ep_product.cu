// The experts' products over the rows of an expanded layout, and their
// gradients.  Expert e's rows are the segment [expert_offset[e],
// expert_offset[e] + num_rows_per_expert[e]); its weights are w[e], one row
// of `hidden` inputs per output.
//
//   out[s]    = x[s] w[e]^T                             (plain)
//   out[s]    = silu(x[s] wg^T) * (x[s] wu^T)           (gated: w[e] = [wg; wu])
//   grad_x[s] = g[s] w[e],   grad_w[e] = sum over e's rows of g[s]^T x[s]
//
// with g the gradient of x w^T.  bf16 in and out, sums in fp32 in tensor
// memory, rounded once.  The kernel is in ep_pair.cuh.
//
// Gradients through the gate of 4096 tokens top-6 of 64 experts, 4096 -> 2 x
// 1408: 846 to 890 us sustained (789 to 814 the first time, before the power limit
// is met), of which the gate 43, the rows about 340, the weights about 400.
#include "ep_pair.cuh"

namespace ep {

namespace {

// The gradient of silu(g) * u for the rows of the layout, kept in bf16 as the
// preactivations are: it is an operand of two products on the tensor cores.
// (The gradients are then 2.3e-3 from 64 bits, with 32 bits between 1.7e-3;
// __expf is accurate to 2^-16, as in silu_of.)
// One pass over flat rows: 22 000 rows of 1408, 311 MB, 43 us (rows by expert
// and block: 73 us, since experts differ in their rows).
struct GateParams {
  const uint16_t *grad, *preact;
  uint16_t *out;
  const int32_t *offset;
  int E, cap, width;
};

__global__ void __launch_bounds__(256) gate_backward_kernel(GateParams p) {
  griddep_wait();
  griddep_launch_dependents();
  // every row up to the layout's last, padding rows too (nobody reads them)
  const int rows = min(max(p.offset[p.E], 0), p.cap), groups = p.width / 8;
  const int64_t n = (int64_t)rows * groups;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / groups;
    const int col = (int)(i - row * groups) * 8;
    const int4 g4 = __ldcs(reinterpret_cast<const int4 *>(p.preact + row * 2 * p.width + col));
    const int4 u4 = __ldcs(reinterpret_cast<const int4 *>(p.preact + row * 2 * p.width + p.width + col));
    const int4 d4 = __ldcs(reinterpret_cast<const int4 *>(p.grad + row * p.width + col));
    const uint32_t *gw = reinterpret_cast<const uint32_t *>(&g4), *uw = reinterpret_cast<const uint32_t *>(&u4);
    const uint32_t *dw = reinterpret_cast<const uint32_t *>(&d4);
    uint32_t og[4], ou[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float a[2], b[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float g = h ? bf16_hi(gw[j]) : bf16_lo(gw[j]);
        const float u = h ? bf16_hi(uw[j]) : bf16_lo(uw[j]);
        const float d = h ? bf16_hi(dw[j]) : bf16_lo(dw[j]);
        const float sig = 1.0f / (1.0f + __expf(-g));
        a[h] = d * u * sig * (1.0f + g * (1.0f - sig));
        b[h] = d * g * sig;
      }
      og[j] = pack_bf16x2(a[0], a[1]);
      ou[j] = pack_bf16x2(b[0], b[1]);
    }
    *reinterpret_cast<uint4 *>(p.out + row * 2 * p.width + col) = make_uint4(og[0], og[1], og[2], og[3]);
    *reinterpret_cast<uint4 *>(p.out + row * 2 * p.width + p.width + col) = make_uint4(ou[0], ou[1], ou[2], ou[3]);
  }
}

// Where no row may be computed: a layout that has some all the same is flagged.
__global__ void __launch_bounds__(256) flag_rows_kernel(const int32_t *rows, int E, uint32_t *error_word) {
  griddep_wait();
  griddep_launch_dependents();
  bool some = false;
  for (int e = threadIdx.x; e < E; e += 256) some = some || rows[e] != 0;
  if (some) set_error(error_word, EP_ERRBIT_CAPACITY);
}

ep_status_t launch_flag_rows(const Params &p, cudaStream_t stream) {
  const cudaError_t e = launch_kernel(flag_rows_kernel, 1, 256, 0, stream, false, p.rows, p.E, p.error_word);
  return e == cudaSuccess ? EP_OK : cuda_fail(e, "flag_rows launch");
}

}  // namespace

ep_status_t launch_product(const ProductArgs &a, cudaStream_t stream) {
  const int most = a.num_tokens < a.recv_capacity ? a.num_tokens : a.recv_capacity;  // rows of one expert
  Params p = {};
  p.most_rows = most;
  p.rows = a.num_rows_per_expert;
  p.offset = a.expert_offset;
  p.error_word = a.error_word;
  p.E = a.num_experts;
  if (most == 0) return launch_flag_rows(p, stream);
  p.cap = a.recv_capacity;
  p.width = a.width;
  p.wide = a.gated ? 2 * a.width : a.width;
  p.inner = a.hidden;
  p.a_tiles = up(a.width, a.gated ? 128 : 256);
  p.out = a.out;
  p.preact = a.preact;
  const ep_status_t s = weight_map(p, a.gated ? kGated : kPlain, a.w, p.wide, a.hidden);
  if (s != EP_OK) return s;
  return a.gated ? launch_rows_form<kGated>(p, a.x, a.hidden, stream) : launch_rows_form<kPlain>(p, a.x, a.hidden, stream);
}

ep_status_t launch_product_backward(const ProductBackwardArgs &a, cudaStream_t stream) {
  const int most = a.num_tokens < a.recv_capacity ? a.num_tokens : a.recv_capacity;
  const int wide = a.gated ? 2 * a.width : a.width;
  const uint16_t *g = a.gated ? a.grad_preact : a.grad;
  Params p = {};
  p.most_rows = most;
  p.rows = a.num_rows_per_expert;
  p.offset = a.expert_offset;
  p.error_word = a.error_word;
  p.E = a.num_experts;
  p.cap = a.recv_capacity;
  p.wide = wide;
  p.hidden = a.hidden;
  if (most == 0 && a.grad_w == nullptr) return launch_flag_rows(p, stream);  // else the weights' gradient flags them
  if (a.gated && most > 0) {
    const GateParams q{a.grad, a.preact, a.grad_preact, p.offset, a.num_experts, a.recv_capacity, a.width};
    const DeviceInfo *di = current_device_info();
    if (di == nullptr) return EP_ERR_CUDA;
    const int64_t need = ((int64_t)a.recv_capacity * (a.width / 8) + 255) / 256, fill = (int64_t)di->num_sms * 32;
    const cudaError_t e =
        launch_kernel(gate_backward_kernel, (int)(need < fill ? need : fill), 256, 0, stream, false, q);
    if (e != cudaSuccess) return cuda_fail(e, "gate_backward launch");
  }
  if (a.grad_x != nullptr && most > 0) {
    p.inner = wide;
    p.width = a.hidden;
    p.a_tiles = up(a.hidden, 256);
    p.out = a.grad_x;
    ep_status_t s = weight_map(p, kGradX, a.w, wide, a.hidden);
    if (s == EP_OK) s = launch_rows_form<kGradX>(p, g, wide, stream);
    if (s != EP_OK) return s;
  }
  if (a.grad_w != nullptr) {
    p.parts = 1;
    p.max_cols = kMaxCols;
    p.a_tiles = up(wide, 256);
    p.b_tiles = up(a.hidden, 256);
    p.out = a.grad_w;
    // without rows nothing is copied: the maps only need an address
    const int cap = most > 0 ? a.recv_capacity : 1;
    ep_status_t s = block_map(&p.a, &p.a_blocks, most > 0 ? g : a.grad_w, wide, cap, wide);
    const uint64_t dims[] = {(uint64_t)a.hidden, (uint64_t)wide, (uint64_t)a.num_experts};
    const uint64_t strides[] = {a.hidden * kSize, (uint64_t)wide * a.hidden * kSize};
    const uint32_t box[] = {64, 32, 1};
    if (s == EP_OK) s = encode_map(&p.grad, a.grad_w, 3, dims, strides, box);
    if (s == EP_OK) s = block_map(&p.b[0], &p.b_blocks, most > 0 ? a.x : a.grad_w, a.hidden, cap, a.hidden);
    if (s == EP_OK)
      s = launch_form<kGradW>(p, (int64_t)a.num_experts * p.a_tiles * p.b_tiles, stream);
    if (s != EP_OK) return s;
  }
  return EP_OK;
}

}  // namespace ep
