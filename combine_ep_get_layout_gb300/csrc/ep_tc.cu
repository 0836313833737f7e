// The host's tensor-map encoder (a driver function, found through the
// runtime, so nothing links against the driver).
#include "ep_tc.cuh"

namespace ep {

namespace {

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encoder() {
  static const EncodeFn fn = [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeFn>(f);
  }();
  return fn;
}

}  // namespace

ep_status_t encode_map(CUtensorMap *map, const void *base, uint64_t x, uint64_t y, uint64_t z, uint32_t box_x,
                       uint32_t box_y, CUtensorMapSwizzle swizzle) {
  const EncodeFn fn = encoder();
  if (fn == nullptr) return fail(EP_ERR_CUDA, "cuTensorMapEncodeTiled not found");
  const cuuint64_t dims[3] = {x, y, z};
  const cuuint64_t strides[2] = {x * 2, x * y * 2};
  const cuuint32_t box[3] = {box_x, box_y, 1}, steps[3] = {1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, z == 0 ? 2 : 3, const_cast<void *>(base), dims, strides,
                        box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(EP_ERR_CUDA, "cuTensorMapEncodeTiled: error %d", (int)r);
  return EP_OK;
}

}  // namespace ep
